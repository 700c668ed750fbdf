"""AdamW over a list of tensors with moments in 8 or 32 bits, microscaled 4-bit matrices, and a linear layer
on them whose weight gradient goes into a PowerSGD error buffer. All compute happens in libpsgd.so.
"""
from __future__ import annotations

from typing import Optional, Sequence

from . import binding as B

GROUP = 64                                   # elements under one exponent byte of the 8-bit moments


class AdamWGroup:
    """Tensors stepped together by AdamW.

    params, grads: lists of contiguous device tensors, one grad per param and of its size, each list of
                   one dtype (fp16, bf16 or fp32). The buffers are captured; the caller fills grads.
    bits: 8 (codes under an exponent per 64 elements) or 32, of both moments
    stochastic: stochastic rounding of 8-bit moments and 16-bit params, by bits hashed from `seed`, the
                step and the element. Default: with 8 bits, which rounding to nearest leaves standing still
    moments: state to continue from, as `state()` gives it (kept and updated in place); default zeros

    m1, m2 (and e1, e2): flat state, every tensor's part starting at a group of 64 (`offsets`)
    step_count, skip, norm: device words of the last step (t; 1 where it was skipped; norm, clipping factor)
    """

    def __init__(self, params: Sequence, grads: Sequence, bits: int = 8, stochastic: Optional[bool] = None, seed: int = 0,
                 moments: Optional[Sequence] = None):
        import torch
        call = "psgd_adamw_plan_create"
        self.ctx = self.plan = None
        self.params, self.grads = list(params), list(grads)
        if not self.params or len(self.params) != len(self.grads):
            raise B.PsgdError(call, B.PSGD_EINVAL, "need one grad per param, and at least one")
        if bits not in (8, 32):
            raise B.PsgdError(call, B.PSGD_EINVAL, f"moments have 8 or 32 bits, not {bits}")
        for ts in (self.params, self.grads):
            if any(t.dtype != ts[0].dtype for t in ts):
                raise B.PsgdError(call, B.PSGD_EDTYPE, "params and grads must each have one dtype")
        pt, gt = B._dtype(self.params[0], call), B._dtype(self.grads[0], call)
        self.bits, self.seed = bits, seed
        self.stochastic = bits == 8 if stochastic is None else bool(stochastic)
        dev = self.device = self.params[0].device
        self.offsets, room = [], 0
        for p in self.params:
            self.offsets.append(room)
            room += (p.numel() + GROUP - 1) // GROUP * GROUP
        if moments is None:
            kind = torch.uint8 if bits == 8 else torch.float32
            moments = [torch.zeros(room, dtype=kind, device=dev) for _ in range(2)]
            if bits == 8:
                moments += [torch.zeros(room // GROUP, dtype=torch.uint8, device=dev) for _ in range(2)]
        moments = list(moments)
        if len(moments) != (4 if bits == 8 else 2):
            raise B.PsgdError(call, B.PSGD_EINVAL, "moments are (m1, m2, e1, e2) with 8 bits, (m1, m2) with 32")
        for t, want in zip(moments, (room, room, room // GROUP, room // GROUP)):
            if t.dim() != 1 or t.numel() != want:
                raise B.PsgdError(call, B.PSGD_EINVAL, f"moments must be flat: {room} values, {room // GROUP} exponents")
        self.m1, self.m2 = moments[:2]
        self.e1, self.e2 = moments[2:] if bits == 8 else (None, None)
        B._same_device(call, *self.params, *self.grads, *moments)
        part = lambda t, o, n: t[o:o + (n + GROUP - 1) // GROUP * GROUP]  # noqa: E731
        ts = [B.make_adamw_tensor(p, g, part(self.m1, o, p.numel()), part(self.m2, o, p.numel()),
                                  *([self.e1[o // GROUP:], self.e2[o // GROUP:]] if bits == 8 else []))
              for p, g, o in zip(self.params, self.grads, self.offsets)]
        self.step_count = torch.zeros(1, dtype=torch.int32, device=dev)
        self.skip = torch.zeros(1, dtype=torch.int32, device=dev)
        self.norm = torch.zeros(2, dtype=torch.float32, device=dev)
        self.ctx = B.psgd_create(dev.index or 0, 1)
        self.plan = B.psgd_adamw_plan_create(self.ctx, ts, pt, gt, B.PSGD_STATE_BYTE if bits == 8 else B.PSGD_STATE_F32)

    def step(self, hp, max_norm: float = 0.0, skip=None, stream=None):
        """One step: skip word, norm and clipping factor from the gradients, then the update. skip: a skip word
        decided before (int32; PowerSGDGroup.skip, where the gradients are its decompressed ones), or None."""
        if skip is not None:
            B._words("psgd_adamw_prepare", self.ctx, None, skip_in=skip)
        h = B._hparams(hp)
        inf = float("inf")
        if not (0 <= h.beta1 < 1 and 0 <= h.beta2 < 1 and 0 <= h.lr < inf and 0 <= h.eps < inf and 0 <= h.weight_decay < inf):
            raise B.PsgdError("psgd_adamw_update", B.PSGD_EINVAL, "betas must lie in [0, 1), lr, eps and weight_decay be finite and >= 0")
        lib, st, ctx, plan = B.load_library(), B._stream(stream, self.device.index), self.ctx, self.plan
        words = self.skip.data_ptr(), self.step_count.data_ptr(), self.norm.data_ptr()
        B._check(ctx, "psgd_adamw_prepare", lib.psgd_adamw_prepare(ctx, plan, max_norm, B._ptr(skip), *words, st))
        B._check(ctx, "psgd_adamw_update", lib.psgd_adamw_update(ctx, plan, *words, B.ctypes.byref(h), int(self.stochastic),
                                                                 self.seed & 0xFFFFFFFFFFFFFFFF, st))

    def state(self):
        """The moments, for the constructor's `moments`; step_count belongs to a checkpoint as well, and is restored in
        place (step_count.copy_)."""
        return (self.m1, self.m2, self.e1, self.e2) if self.bits == 8 else (self.m1, self.m2)

    def moments(self, dtype=None, stream=None):
        """The moments' values, flat: new bf16 (or fp32) tensors of 8-bit moments, the fp32 ones themselves."""
        import torch
        if self.bits == 32:
            return self.m1, self.m2
        call, n = "psgd_adamw_moments", self.m1.numel()
        kind = dtype or torch.bfloat16
        out1, out2 = (B._workspace(n * kind.itemsize, self.device, stream).view(kind) for _ in range(2))
        B._check(self.ctx, call, B.load_library().psgd_adamw_moments(
            self.ctx, self.m1.data_ptr(), self.e1.data_ptr(), self.m2.data_ptr(), self.e2.data_ptr(), n, out1.data_ptr(), out2.data_ptr(),
            B._dtype(out1, call), B._stream(stream, self.device.index)))
        return out1, out2

    def close(self):
        if getattr(self, "plan", None):
            B.psgd_adamw_plan_destroy(self.plan)
            self.plan = None
        if getattr(self, "ctx", None):
            B.psgd_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class MxTensor:
    """A rows x k matrix in microscaled 4-bit elements, k the dimension its products sum over: `data`, one
    buffer of psgd_mx_bytes(rows, k) bytes, filled by psgd_mx_quantize."""

    def __init__(self, rows: int, k: int, device=None, data=None):
        import torch
        self.rows, self.k = rows, k = int(rows), int(k)
        # as the library counts (a refused size is its refusal)
        need = -(-k // 128) * (rows * 64 + -(-rows // 64) * 256) if 0 <= rows <= 1 << 25 and 0 <= k <= 1 << 25 else B.psgd_mx_bytes(rows, k)
        if data is None:
            data = torch.empty(need, dtype=torch.uint8, device=device or "cuda")
        elif data.dtype != torch.uint8 or not data.is_contiguous() or data.numel() < need:
            raise B.PsgdError("psgd_mx_bytes", B.PSGD_EINVAL, f"data must be {need} contiguous bytes")
        self.data = data
        self.struct = B.psgd_mx_tensor(data.data_ptr(), rows, k)


class MxLinear:
    """A linear layer y = x W whose three products run on 4-bit operands.

    weight: in x out device tensor (fp16, bf16 or fp32). Its 4-bit forms are made here and by refresh(),
            which follows every step on the weight
    seed: of the stochastic rounding of the output's gradient; another one for every layer

    Runs on the current stream of the weight's device. Holds one forward() for backward(): where a layer runs
    several times before, each but the last has to be run again before its backward().
    """

    def __init__(self, weight, seed: int = 0):
        self.ctx = None
        if weight.dim() != 2 or min(weight.shape) < 1:
            raise B.PsgdError("psgd_mx_quantize", B.PSGD_EINVAL, "weight must be an in x out tensor")
        B._dtype(weight, "psgd_mx_quantize")
        B._same_device("psgd_mx_quantize", weight)
        self.weight, self.seed, self.device = weight, seed, weight.device
        self.n_in, self.n_out = weight.shape
        self.w_row = MxTensor(self.n_in, self.n_out, self.device)
        self.w_col = MxTensor(self.n_out, self.n_in, self.device)
        self.x_col = None
        self.ctx = B.psgd_create(self.device.index or 0, 1)
        self.refresh()

    def refresh(self):
        """4-bit forms of the weight as it is now."""
        B.psgd_mx_quantize(self.ctx, self.weight, self.w_row, self.w_col)

    def _tokens(self, t, width, name):
        if t.shape[-1:] != (width,) or t.dim() < 2:
            raise B.PsgdError("psgd_mx_quantize", B.PSGD_EINVAL, f"{name} must hold one row of {width} values per token")
        return t if t.dim() == 2 else t.reshape(-1, width)

    # The calls of psgd_mx_quantize and psgd_mx_product, their tensors' device and shapes checked before.
    def _quantize(self, x, row, col, rounding, step, stream):
        call = "psgd_mx_quantize"
        m, n = x.shape
        B._check(self.ctx, call, B.load_library().psgd_mx_quantize(
            self.ctx, x.data_ptr(), B._row_stride(x, call), m, n, B._dtype(x, call), B._mx(row), B._mx(col), rounding,
            self.seed & 0xFFFFFFFFFFFFFFFF, B._ptr(step), stream))

    def _product(self, a, b, out, scale, accumulate, stream):
        call = "psgd_mx_product"
        need = B.psgd_mx_product_workspace(a.rows, b.rows, a.k)
        room = B._workspace(need, self.device, None) if need else None
        B._check(self.ctx, call, B.load_library().psgd_mx_product(
            self.ctx, B._mx(a), B._mx(b), B._ptr(scale), out.data_ptr(), B._row_stride(out, call), B._dtype(out, call), accumulate,
            B._ptr(room), need, stream))

    def forward(self, x, train: bool = True):
        """y = x W, in x's dtype; x [..., in] to nearest. With train, x's 4-bit transpose is kept for backward()."""
        import torch
        x2 = self._tokens(x, self.n_in, "x")
        B._same_device("psgd_mx_quantize", self.w_col.data, x2)
        t, stream = x2.shape[0], B._stream(None, self.device.index)
        row = MxTensor(t, self.n_in, self.device)
        col = MxTensor(self.n_in, t, self.device) if train else None
        y = torch.empty(t, self.n_out, dtype=x.dtype, device=self.device)
        self._quantize(x2, row, col, B.PSGD_NEAREST, None, stream)
        self._product(row, self.w_col, y, None, 0, stream)
        if train:
            self.x_col, self.x_stream = col, stream
        return y if x.dim() == 2 else y.view(*x.shape[:-1], self.n_out)

    def backward(self, dy, err=None, scale=None, step=None):
        """dx = dy W^T, in dy's dtype, and err += scale x^T dy (err: in x out fp32, the error buffer of an
        in-place matrix of a PowerSGDGroup; scale: its one-element fp32 multiplier, or None), which uses up
        the forward() before it: a second such call is refused. dy is rounded
        stochastically by seed and step (one-element int32 device tensor, which the caller advances; None: 0).
        Calls of one step draw the same bits: what is to average out, microbatches too, needs a step of its own."""
        import torch
        dy2 = self._tokens(dy, self.n_out, "dy")
        t, stream = dy2.shape[0], B._stream(None, self.device.index)
        B._same_device("psgd_mx_product", self.w_row.data, *[v for v in (dy2, err, scale, step) if v is not None])
        if step is not None and step.dtype != torch.int32:
            raise B.PsgdError("psgd_mx_quantize", B.PSGD_EDTYPE, "step must be int32")
        if step is not None and step.numel() < 1:
            raise B.PsgdError("psgd_mx_quantize", B.PSGD_EINVAL, "step must be one int32")
        if err is not None:
            if self.x_col is None or self.x_col.k != t:
                raise B.PsgdError("psgd_mx_product", B.PSGD_EINVAL, "backward() needs the forward() of the same tokens before it")
            if err.shape != self.weight.shape:
                raise B.PsgdError("psgd_mx_product", B.PSGD_EINVAL, f"err must be {self.n_in} x {self.n_out}")
            if err.dtype != torch.float32:
                raise B.PsgdError("psgd_mx_product", B.PSGD_EDTYPE, "products are added to fp32 only")
            if scale is not None and (scale.dtype != torch.float32 or scale.numel() < 1):
                raise B.PsgdError("psgd_mx_product", B.PSGD_EDTYPE, "scale must be one float32")
        row = MxTensor(t, self.n_out, self.device)
        col = MxTensor(self.n_out, t, self.device) if err is not None else None
        dx = torch.empty(t, self.n_in, dtype=dy.dtype, device=self.device)
        self._quantize(dy2, row, col, B.PSGD_STOCHASTIC, step, stream)
        self._product(row, self.w_row, dx, None, 0, stream)
        if err is not None:
            if self.x_stream != stream:                      # its memory is not handed out before this product is done
                self.x_col.data.record_stream(torch.cuda.current_stream(self.device))
            self._product(self.x_col, col, err, scale, 1, stream)
            self.x_col = None
        return dx if dy.dim() == 2 else dx.view(*dy.shape[:-1], self.n_in)

    def close(self):
        if getattr(self, "ctx", None):
            B.psgd_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

"""Groups of matrices over torch device tensors: gradients compressed together, and updates
orthogonalised together.

PowerSGDGroup holds the context, the plan and the per-step device words (flags, skip), and calls the three
entry points in order. All compute happens in libpsgd.so.
"""
from __future__ import annotations

from typing import List, Optional, Sequence

from . import binding as B


class PowerSGDGroup:
    """State of a group: per matrix G (caller-filled each step), E, Q, Q_next, P, optional D.

    grads: list of 2-D device tensors (fp16, bf16 or fp32, all the same dtype, unit row stride);
           an entry None makes that matrix in-place (its err tensor, which must then be given,
           already holds M = s_b G + E)
    blocks: per matrix index into `scale`
    scale: device fp32 tensor of per-resblock multipliers
    q0: list of n x r fp32 initial warm starts (copied)
    err: optional list of m x n fp32 device tensors used in place as the error buffers
         (unit row stride; default: new zero buffers)
    write_out: allocate D buffers and have the decompression write them
    """

    def __init__(self, grads: Sequence, blocks: Sequence[int], scale, rank: int, q0: Sequence,
                 err: Optional[Sequence] = None, write_out: bool = True, device: int = 0):
        import torch
        self.torch = torch
        self.rank = rank
        self.grads = list(grads)
        self.blocks = list(blocks)
        self.scale = scale
        if err is None and any(g is None for g in self.grads):
            raise ValueError("in-place matrices (grad None) need their err tensors")
        dev = (self.grads[0] if self.grads[0] is not None else err[0]).device
        self.err = ([torch.zeros(g.shape, dtype=torch.float32, device=dev) for g in self.grads]
                    if err is None else list(err))
        shapes = [tuple(e.shape) for e in self.err]
        self.q = [q.to(device=dev, dtype=torch.float32).contiguous().clone() for q in q0]
        self.q_next = [torch.empty_like(q) for q in self.q]
        self.p = [torch.empty((sh[0], rank), dtype=torch.float32, device=dev) for sh in shapes]
        self.out = [torch.empty(sh, dtype=torch.float32, device=dev) if write_out else None
                    for sh in shapes]
        self.flags = torch.zeros(len(self.grads), dtype=torch.uint8, device=dev)
        self.skip = torch.zeros(1, dtype=torch.int32, device=dev)
        self.ctx = B.psgd_create(device, rank)
        mats = [B.make_matrix(g, e, q, qn, p, b, o) for g, e, q, qn, p, b, o in
                zip(self.grads, self.err, self.q, self.q_next, self.p, self.blocks, self.out)]
        given = [g for g in self.grads if g is not None]
        self.plan = B.psgd_plan_create(self.ctx, mats,
                                       B.dtype_code(given[0].dtype) if given else B.PSGD_F32,
                                       int(scale.numel()))

    def compress(self, stream=None):
        B.psgd_compress(self.ctx, self.plan, self.scale, self.flags, stream)

    def check_finite(self, passthrough: Sequence = (), host: bool = False, stream=None):
        return B.psgd_check_finite(self.ctx, self.plan, self.flags, passthrough, self.scale,
                                   self.skip, host, stream)

    def decompress_update(self, stream=None):
        B.psgd_decompress_update(self.ctx, self.plan, self.scale, self.skip, stream)

    def counters(self):
        """(steps decompressed, steps skipped): the plan's device counters, copied to the host
        after a device synchronisation."""
        import ctypes
        self.torch.cuda.synchronize()
        addr = B.psgd_plan_counters(self.plan)
        out = (ctypes.c_int64 * 2)()
        hip = ctypes.CDLL("libamdhip64.so.7")
        hip.hipMemcpy.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int]
        err = hip.hipMemcpy(ctypes.addressof(out), addr, 16, 2)          # device to host
        if err != 0:
            raise RuntimeError(f"hipMemcpy of the step counters failed ({err})")
        return int(out[0]), int(out[1])

    def reset_errors(self, stream=None):
        """E = 0 for every matrix: resuming from a checkpoint, which holds no error buffers."""
        B.psgd_reset_errors(self.ctx, self.plan, stream)

    # ---- optimizer ---------------------------------------------------------------------
    def attach_adam(self, params: Sequence, m1: Sequence, m2: Sequence):
        """Attach per-matrix optimizer state (caller-owned device tensors, updated in place):
        params m x n (fp16, bf16 or fp32), m1 and m2 m x n 16-bit codes (bf16 and ue8m8)."""
        torch = self.torch
        self.params, self.m1, self.m2 = list(params), list(m1), list(m2)
        opt = [B.make_adam_matrix(p, a, b) for p, a, b in zip(self.params, self.m1, self.m2)]
        B.psgd_adam_attach(self.ctx, self.plan, opt, B.dtype_code(self.params[0].dtype))
        dev = self.flags.device
        self.adam_step = torch.zeros(1, dtype=torch.int32, device=dev)
        self.adam_norm = torch.zeros(2, dtype=torch.float32, device=dev)

    def step_adam(self, hp, passthrough: Sequence = (), hp_pass=None, max_norm: float = 0.0,
                  host: bool = False, stream=None):
        """One step with the optimizer: compress, finite check, global norm and clipping,
        decompression fused with the matrices' Adam update, fp32 Adam on the pass-through
        tensors. passthrough: (param, m1, m2, grad) fp32 tensors; their gradients take part in
        the finite check and the global norm."""
        self.compress(stream)
        grads = [t[3] for t in passthrough]
        s = self.check_finite(grads, host, stream)
        ts = [B.make_adam_tensor(*t) for t in passthrough]
        B.psgd_adam_prepare(self.ctx, self.plan, ts, max_norm, self.skip, self.adam_step, self.adam_norm, stream)
        B.psgd_decompress_adam(self.ctx, self.plan, self.scale, self.skip, self.adam_step, self.adam_norm, hp,
                               stream)
        if ts:
            B.psgd_adam_update(self.ctx, ts, self.skip, self.adam_step, self.adam_norm, hp_pass or hp, stream)
        return s

    def attach_muon(self, params: Sequence, momentum: Sequence, accurate: Optional[bool] = None):
        """Attach per-matrix Muon state (caller-owned device tensors, updated in place): params
        m x n (fp16, bf16 or fp32), momentum m x n fp32. The group needs its out buffers
        (write_out). accurate: products with the norm-wise error of fp32 ones; default: for fp32
        parameters, whose rounding the fast products' 2e-3 of the update would exceed. Each
        matrix is orthogonalised on its own: a shard of a weight gets its block's factor."""
        torch, call = self.torch, "psgd_muon_attach"
        params, momentum = list(params), list(momentum)
        if len(params) != len(self.err) or len(momentum) != len(self.err):
            raise B.PsgdError(call, B.PSGD_EINVAL, "one param and one momentum per matrix")
        if any(p.dtype != params[0].dtype for p in params):
            raise B.PsgdError(call, B.PSGD_EDTYPE, "parameters must have one dtype")
        for p, e in zip(params, self.err):
            if tuple(p.shape) != tuple(e.shape):
                raise B.PsgdError(call, B.PSGD_EINVAL, "param and matrix shapes differ")
        B._same_device(call, self.flags, *params, *momentum, ctx=self.ctx)
        if accurate is None:
            accurate = params[0].dtype == torch.float32
        opt = [B.make_muon_matrix(p, m) for p, m in zip(params, momentum)]
        B.psgd_muon_attach(self.ctx, self.plan, opt, B._dtype(params[0], call),
                           B.PSGD_NS_ACCURATE if accurate else B.PSGD_NS_FAST)
        # only now: a refused call leaves the attached tensors alive
        self.muon_params, self.momentum = params, momentum
        if not hasattr(self, "adam_step"):
            dev = self.flags.device
            self.adam_step = torch.zeros(1, dtype=torch.int32, device=dev)
            self.adam_norm = torch.zeros(2, dtype=torch.float32, device=dev)

    def step_muon(self, hp, passthrough: Sequence = (), hp_pass=None, max_norm: float = 0.0,
                  host: bool = False, stream=None):
        """One step with Muon on the matrices: compress, finite check, global norm and clipping,
        decompression, momentum and orthogonalised update, fp32 Adam (hp_pass) on the
        pass-through tensors. passthrough: (param, m1, m2, grad) fp32 tensors, e.g. an embedding
        with its psgd_embed_grad gradient."""
        if not hasattr(self, "muon_params"):
            raise B.PsgdError("psgd_muon_update", B.PSGD_EINVAL, "no Muon state attached (attach_muon)")
        if passthrough and hp_pass is None:
            raise ValueError("pass-through tensors need their Adam hyperparameters (hp_pass)")
        stream = B._stream(stream, self.flags.device)          # one stream, of the group's device, for all of them
        self.compress(stream)
        s = self.check_finite([t[3] for t in passthrough], host, stream)
        ts = [B.make_adam_tensor(*t) for t in passthrough]
        B.psgd_adam_prepare(self.ctx, self.plan, ts, max_norm, self.skip, self.adam_step, self.adam_norm, stream)
        self.decompress_update(stream)
        B.psgd_muon_update(self.ctx, self.plan, self.skip, self.adam_norm, hp, stream)
        if ts:
            B.psgd_adam_update(self.ctx, ts, self.skip, self.adam_step, self.adam_norm, hp_pass, stream)
        return s

    def step(self, passthrough: Sequence = (), host: bool = False, stream=None):
        self.compress(stream)
        s = self.check_finite(passthrough, host, stream)
        self.decompress_update(stream)
        return s

    def close(self):
        if getattr(self, "plan", None):
            B.psgd_plan_destroy(self.plan)
            self.plan = None
        if getattr(self, "ctx", None):
            B.psgd_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class NewtonSchulzGroup:
    """Update matrices orthogonalised together: out[i] = Newton-Schulz(updates[i]) on run().

    updates, outs: lists of 2-D device tensors (unit row stride), each list of one dtype (fp16,
                   bf16 or fp32); out may be its update itself. The buffers are captured.
    accurate: products with the norm-wise error of fp32 ones (1e-6 to 5e-6). Default: unless the
              outputs are bf16, whose rounding, 1.7e-3 of the norm, exceeds the fast products'
              error of about 1e-3 (both together: 2e-3)
    """

    def __init__(self, updates: Sequence, outs: Sequence, accurate: Optional[bool] = None):
        import torch
        self.ctx = self.plan = None
        self.updates, self.outs = list(updates), list(outs)
        call = "psgd_ns_plan_create"
        if not self.updates or len(self.updates) != len(self.outs):
            raise B.PsgdError(call, B.PSGD_EINVAL, "need one out per update, and at least one")
        for ts in (self.updates, self.outs):
            if any(t.dtype != ts[0].dtype for t in ts):
                raise B.PsgdError(call, B.PSGD_EDTYPE, "updates and outs must each have one dtype")
        if accurate is None:
            accurate = self.outs[0].dtype != torch.bfloat16
        mats = [B.make_ns_matrix(u, o) for u, o in zip(self.updates, self.outs)]
        it, ot = B._dtype(self.updates[0], call), B._dtype(self.outs[0], call)
        B._same_device(call, *self.updates, *self.outs)
        self.device = self.updates[0].device
        self.ctx = B.psgd_create(self.device.index or 0, 1)
        self.plan = B.psgd_ns_plan_create(self.ctx, mats, it, ot, B.PSGD_NS_ACCURATE if accurate else B.PSGD_NS_FAST)

    def run(self, hp=None, stream=None):
        B.psgd_newton_schulz(self.ctx, self.plan, hp, B._stream(stream, self.device))

    def close(self):
        if getattr(self, "plan", None):
            B.psgd_ns_plan_destroy(self.plan)
            self.plan = None
        if getattr(self, "ctx", None):
            B.psgd_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

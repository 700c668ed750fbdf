"""Refusals, layout, devices and streams of the many-tensor AdamW and 4-bit matrix calls that need no GPU: the
binding's checks, the C checks without a context, and a library that records its calls."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from rank_gradient_compression_powersgd_amd import binding as B
from rank_gradient_compression_powersgd_amd import lowbit
from tests.test_muon_args import ROOT, _raises
from tests.test_muon_devices import _On, lib  # noqa: F401


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not available")
def test_struct_layout_matches_c(tmp_path):
    structs = (B.psgd_adamw_tensor, B.psgd_mx_tensor)
    body = "".join(f' printf("%zu\\n", sizeof({s.__name__}));\n'
                   + "".join(f' printf("%zu\\n", offsetof({s.__name__}, {f[0]}));\n' for f in s._fields_) for s in structs)
    body += ' printf("%d\\n%d\\n%d\\n%d\\n", PSGD_NEAREST, PSGD_STOCHASTIC, PSGD_STATE_F32, PSGD_STATE_BYTE);\n'
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "psgd.h"\nint main(void){\n' + body + " return 0; }\n")
    exe = tmp_path / "layout"
    r = subprocess.run(["gcc", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", "/opt/rocm/include",
                        str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    vals = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for s in structs:
        want += [ctypes.sizeof(s)] + [getattr(s, f[0]).offset for f in s._fields_]
    assert vals == want + [B.PSGD_NEAREST, B.PSGD_STOCHASTIC, B.PSGD_STATE_F32, B.PSGD_STATE_BYTE]


def test_calls_without_a_context():
    lib = B.load_library()
    n = ctypes.c_int64(-1)
    assert lib.psgd_adamw_plan_create(None, None, 0, 3, 3, 1, None) == B.PSGD_EINVAL
    assert lib.psgd_adamw_plan_destroy(None) == B.PSGD_OK
    assert lib.psgd_adamw_prepare(None, None, 0.0, None, None, None, None, None) == B.PSGD_EINVAL
    assert lib.psgd_adamw_update(None, None, None, None, None, None, 0, 0, None) == B.PSGD_EINVAL
    assert lib.psgd_adamw_moments(None, None, None, None, None, 0, None, None, 3, None) == B.PSGD_EINVAL
    assert lib.psgd_mx_quantize(None, None, 1, 1, 1, 3, None, None, 0, 0, None, None) == B.PSGD_EINVAL
    assert lib.psgd_mx_dequantize(None, None, None, 1, 3, None) == B.PSGD_EINVAL
    assert lib.psgd_mx_product(None, None, None, None, None, 1, 3, 0, None, 0, None) == B.PSGD_EINVAL
    assert lib.psgd_mx_bytes(1, 1, None) == B.PSGD_EINVAL
    assert lib.psgd_mx_product_workspace(1, 1, 1, None) == B.PSGD_EINVAL
    for bad in ((-1, 1), (1, -1), (2 ** 25 + 1, 1), (1, 2 ** 25 + 1)):
        assert lib.psgd_mx_bytes(*bad, ctypes.byref(n)) == B.PSGD_EINVAL
        assert lib.psgd_mx_product_workspace(bad[0], 1, bad[1], ctypes.byref(n)) == B.PSGD_EINVAL
        assert lib.psgd_mx_product_workspace(1, *bad, ctypes.byref(n)) == B.PSGD_EINVAL


def test_sizes_of_matrices():
    assert B.psgd_mx_bytes(0, 100) == B.psgd_mx_bytes(100, 0) == 0
    assert B.psgd_mx_bytes(1, 1) == 64 + 256
    assert B.psgd_mx_bytes(65, 129) == 2 * (65 * 64 + 2 * 256)
    assert B.psgd_mx_bytes(2 ** 25, 2 ** 20) == 2 ** 13 * (2 ** 25 * 64 + 2 ** 19 * 256)


@pytest.mark.parametrize("m", [0, 1, 16, 64, 65, 200, 1000, 4096, 20480])
@pytest.mark.parametrize("n", [0, 1, 64, 333, 1488, 3968, 11904])
def test_workspaces_are_whole_parts(m, n):
    """A workspace holds a whole number of fp32 results, at most one per 8 panels."""
    for k in (0, 1, 128, 1000, 3968, 20480, 200000):
        need = B.psgd_mx_product_workspace(m, n, k)
        if need:
            parts, rest = divmod(need, 4 * m * n)
            assert rest == 0 and 2 <= parts <= -(-k // 128) // 4


def test_adamw_binding_checks():
    f, h, g = torch.zeros(100), torch.zeros(100, dtype=torch.float16), torch.zeros(100)
    make = lowbit.AdamWGroup
    _raises(B.PSGD_EINVAL, lambda: make([], []))
    _raises(B.PSGD_EINVAL, lambda: make([f], [g, g]))
    _raises(B.PSGD_EINVAL, lambda: make([f], [g], bits=4), "8 or 32")
    _raises(B.PSGD_EDTYPE, lambda: make([f, h], [g, g]))
    _raises(B.PSGD_EDTYPE, lambda: make([f.double()], [g]))
    _raises(B.PSGD_EINVAL, lambda: make([f], [g]), "GPU")
    c, e = torch.zeros(128, dtype=torch.uint8), torch.zeros(2, dtype=torch.uint8)
    tensor = B.make_adamw_tensor
    assert tensor(f, g, c, c.clone(), e, e.clone()).numel == 100
    assert tensor(f, g, torch.zeros(128), torch.zeros(128)).e1 is None
    _raises(B.PSGD_EINVAL, lambda: tensor(f, g[:99], c, c, e, e))
    _raises(B.PSGD_EINVAL, lambda: tensor(torch.zeros(200)[::2], g, c, c, e, e), "contiguous")
    _raises(B.PSGD_EINVAL, lambda: tensor(f, g, c[:127], c, e, e))
    _raises(B.PSGD_EINVAL, lambda: tensor(f, g, c, c, e[:1], e))
    _raises(B.PSGD_EINVAL, lambda: tensor(f, g, c, c, e))
    _raises(B.PSGD_EDTYPE, lambda: tensor(f, g, c.float(), c, e, e))
    _raises(B.PSGD_EDTYPE, lambda: tensor(f, g, c, c))
    out = torch.zeros(100)
    moments = B.psgd_adamw_moments
    _raises(B.PSGD_EINVAL, lambda: moments(0, c[:100], e, c, e, out, out))
    _raises(B.PSGD_EINVAL, lambda: moments(0, c, e, c, e, out, out[:50]))
    _raises(B.PSGD_EDTYPE, lambda: moments(0, c.int(), e, c, e, out, out))
    _raises(B.PSGD_EINVAL, lambda: moments(0, c, e, c, e, out, out), "GPU")


def test_a_group_takes_its_moments_whole(lib):  # noqa: F811
    f, g = _On(torch.zeros(100), 0), _On(torch.zeros(100), 0)
    c, e = torch.zeros(128, dtype=torch.uint8), torch.zeros(2, dtype=torch.uint8)
    make = lambda *m: lowbit.AdamWGroup([f], [g], moments=m)  # noqa: E731
    _raises(B.PSGD_EINVAL, lambda: make(c, c), "m1, m2, e1, e2")
    _raises(B.PSGD_EINVAL, lambda: make(c, c[:64], e, e), "flat")
    _raises(B.PSGD_EINVAL, lambda: make(c, c, e, e[:1]), "flat")
    _raises(B.PSGD_EINVAL, lambda: lowbit.AdamWGroup([f], [g], bits=32, moments=(c, c, e, e)))


class _Data:
    """An operand whose bytes say which device they are on."""

    def __init__(self, rows, k, index):
        self.rows, self.k, self.data = rows, k, _On(torch.zeros(B.psgd_mx_bytes(rows, k), dtype=torch.uint8), index)
        self.struct = B.psgd_mx_tensor(0, rows, k)


def test_calls_take_the_stream_of_their_device_and_refuse_another(lib, monkeypatch):  # noqa: F811
    monkeypatch.setattr(B, "psgd_mx_bytes", lambda rows, k: 4096)
    monkeypatch.setattr(B, "psgd_mx_product_workspace", lambda m, n, k: 0)
    ctx = B.psgd_create(1, 1)
    word, norm = (_On(torch.zeros(2, dtype=d), 1) for d in (torch.int32, torch.float32))
    hp = B.psgd_adam_hparams(0.1, 0.9, 0.9, 1e-8, 0.0)
    B.psgd_adamw_prepare(ctx, 7, 0.0, None, word, word, norm)
    B.psgd_adamw_update(ctx, 7, word, word, norm, hp, True, -1)
    assert lib.args("psgd_adamw_prepare")[0][-1] == lib.args("psgd_adamw_update")[0][-1] == 101
    assert lib.args("psgd_adamw_update")[0][-3:-1] == (B.PSGD_STOCHASTIC, 2 ** 64 - 1)
    a, b, x = _Data(10, 20, 1), _Data(20, 10, 1), _On(torch.zeros(10, 20), 1)
    B.psgd_mx_quantize(ctx, x, a, b)
    B.psgd_mx_dequantize(ctx, a, x)
    B.psgd_mx_product(ctx, a, _Data(30, 20, 1), _On(torch.zeros(10, 30), 1))
    for call in ("psgd_mx_quantize", "psgd_mx_dequantize", "psgd_mx_product"):
        assert lib.args(call)[0][-1] == 101
    B.psgd_mx_quantize(ctx, x, a, stream=55)
    assert lib.args("psgd_mx_quantize")[1][-1] == 55
    here = _On(torch.zeros(10, 20), 0)
    _raises(B.PSGD_EINVAL, lambda: B.psgd_mx_quantize(ctx, here, _Data(10, 20, 0)), "context on device 1")
    _raises(B.PSGD_EINVAL, lambda: B.psgd_mx_quantize(ctx, x, _Data(10, 20, 0)), "one GPU")
    _raises(B.PSGD_EINVAL, lambda: B.psgd_mx_dequantize(ctx, a, here), "one GPU")
    _raises(B.PSGD_EINVAL, lambda: B.psgd_mx_product(ctx, a, _Data(30, 20, 0), _On(torch.zeros(10, 30), 1)), "one GPU")
    assert len(lib.args("psgd_mx_quantize")) == 2 and len(lib.args("psgd_mx_product")) == 1


def _group_of(lib):  # noqa: F811
    """A group on device 1 of the recording library."""
    group = lowbit.AdamWGroup.__new__(lowbit.AdamWGroup)
    group.ctx, group.plan, group.device, group.stochastic, group.seed = B.psgd_create(1, 1), 7, torch.device("cuda", 1), True, 0
    group.skip, group.step_count = (_On(torch.zeros(1, dtype=torch.int32), 1) for _ in range(2))
    group.norm = _On(torch.zeros(2), 1)
    return group


def test_the_words_of_a_step_have_their_type_size_and_device(lib):  # noqa: F811
    """The kernels read and write 4 bytes per word and 8 for the norm, whatever the tensor holds."""
    ctx = B.psgd_create(1, 1)
    on = lambda n, dtype, device=1: _On(torch.zeros(n, dtype=dtype), device)  # noqa: E731
    word, norm, hp = on(1, torch.int32), on(2, torch.float32), B.psgd_adam_hparams(0.1, 0.9, 0.9, 1e-8, 0.0)
    group = _group_of(lib)
    wrong = [(B.PSGD_EDTYPE, on(1, d), "int32") for d in (torch.bool, torch.uint8, torch.float32, torch.int64)]
    wrong += [(B.PSGD_EINVAL, on(0, torch.int32), "1 contiguous"), (B.PSGD_EINVAL, on(1, torch.int32, 0), ""),
              (B.PSGD_EINVAL, torch.zeros(1, dtype=torch.int32), "GPU")]
    for status, bad, text in wrong:
        _raises(status, lambda: B.psgd_adamw_prepare(ctx, 7, 0.0, bad, word, word, norm), text)
        _raises(status, lambda: B.psgd_adamw_prepare(ctx, 7, 0.0, None, bad, word, norm), text)
        _raises(status, lambda: B.psgd_adamw_prepare(ctx, 7, 0.0, None, word, bad, norm), text)
        _raises(status, lambda: B.psgd_adamw_update(ctx, 7, bad, word, norm, hp), text)
        _raises(status, lambda: B.psgd_adamw_update(ctx, 7, word, bad, norm, hp), text)
        _raises(status, lambda: group.step(hp, skip=bad), text)
    for status, bad in ((B.PSGD_EINVAL, on(1, torch.float32)), (B.PSGD_EDTYPE, on(2, torch.float64)), (B.PSGD_EINVAL, on(2, torch.float32, 0)),
                        (B.PSGD_EINVAL, _On(torch.zeros(4)[::2], 1))):
        _raises(status, lambda: B.psgd_adamw_prepare(ctx, 7, 0.0, None, word, word, bad))
        _raises(status, lambda: B.psgd_adamw_update(ctx, 7, word, word, bad, hp))
    assert not lib.args("psgd_adamw_prepare") and not lib.args("psgd_adamw_update")
    B.psgd_adamw_prepare(ctx, 7, 0.0, word, word, word, norm)
    B.psgd_adamw_update(ctx, 7, word, word, None, hp)
    group.step(hp, skip=word)
    group.step(hp)
    assert len(lib.args("psgd_adamw_prepare")) == len(lib.args("psgd_adamw_update")) == 3
    group.plan = group.ctx = None


def test_a_list_has_the_types_and_the_device_of_its_tensors(lib):  # noqa: F811
    """A code of another type than the tensors' would have the kernels step past their ends."""
    ctx = B.psgd_create(1, 1)
    on = lambda n, dtype, device=1: _On(torch.zeros(n, dtype=dtype), device)  # noqa: E731

    def tensor(param, grad, device=1, bits=8):
        p, g = on(100, param, device), on(100, grad, device)
        if bits == 32:
            return B.make_adamw_tensor(p, g, on(128, torch.float32, device), on(128, torch.float32, device))
        return B.make_adamw_tensor(p, g, on(128, torch.uint8, device), on(128, torch.uint8, device), on(2, torch.uint8, device),
                                   on(2, torch.uint8, device))

    f32, f16, bf16 = torch.float32, torch.float16, torch.bfloat16
    create = lambda ts, p, g, s: B.psgd_adamw_plan_create(ctx, ts, p, g, s)  # noqa: E731
    good = tensor(bf16, f32)
    create([good], B.PSGD_BF16, B.PSGD_F32, B.PSGD_STATE_BYTE)
    create([tensor(f16, f16, bits=32)], B.PSGD_F16, B.PSGD_F16, B.PSGD_STATE_F32)
    create([B.psgd_adamw_tensor.from_buffer_copy(good)], B.PSGD_F32, B.PSGD_F32, B.PSGD_STATE_BYTE)   # a struct of the caller's own
    for codes in ((B.PSGD_F32, B.PSGD_F32), (B.PSGD_F16, B.PSGD_F32), (B.PSGD_BF16, B.PSGD_BF16)):
        _raises(B.PSGD_EDTYPE, lambda: create([good], *codes, B.PSGD_STATE_BYTE))
    _raises(B.PSGD_EDTYPE, lambda: create([good, tensor(f32, f32)], B.PSGD_BF16, B.PSGD_F32, B.PSGD_STATE_BYTE))
    _raises(B.PSGD_EINVAL, lambda: create([good], B.PSGD_BF16, B.PSGD_F32, B.PSGD_STATE_F32), "state")
    _raises(B.PSGD_EINVAL, lambda: create([good, tensor(bf16, f32, bits=32)], B.PSGD_BF16, B.PSGD_F32, B.PSGD_STATE_BYTE), "state")
    _raises(B.PSGD_EINVAL, lambda: create([tensor(bf16, f32, 0)], B.PSGD_BF16, B.PSGD_F32, B.PSGD_STATE_BYTE), "device 1")
    _raises(B.PSGD_EINVAL, lambda: create([good, tensor(bf16, f32, 0)], B.PSGD_BF16, B.PSGD_F32, B.PSGD_STATE_BYTE), "device 1")
    _raises(B.PSGD_EINVAL, lambda: B.make_adamw_tensor(on(64, f32), on(64, f32), on(64, f32, 0), on(64, f32)), "one GPU")
    _raises(B.PSGD_EDTYPE, lambda: tensor(torch.float64, f32))
    _raises(B.PSGD_EDTYPE, lambda: tensor(f32, torch.int32))
    assert len(lib.args("psgd_adamw_plan_create")) == 3


def test_an_empty_step_count_is_refused(lib):  # noqa: F811
    """Its address is NULL, which means step 0."""
    ctx = B.psgd_create(1, 1)
    x, row, none = _On(torch.zeros(10, 20), 1), _Data(10, 20, 1), _On(torch.zeros(0, dtype=torch.int32), 1)
    _raises(B.PSGD_EINVAL, lambda: B.psgd_mx_quantize(ctx, x, row, stochastic=True, step=none), "one int32")
    layer = lowbit.MxLinear.__new__(lowbit.MxLinear)
    layer.ctx, layer.n_in, layer.n_out, layer.device, layer.w_row = None, 20, 30, torch.device("cuda", 1), _Data(20, 30, 1)
    _raises(B.PSGD_EINVAL, lambda: layer.backward(_On(torch.zeros(10, 30), 1), step=none), "one int32")
    assert not lib.args("psgd_mx_quantize")


def test_few_rows_and_columns_share_a_long_sum():
    """The kernel for few rows gives 16 columns of C one workgroup for all of k. Where these are few and k is long, tiles in
    parts are several times as fast; where k is short or workgroups are many, the one launch is."""
    parts = lambda m, n, k: B.psgd_mx_product_workspace(m, n, k) // (4 * m * n)  # noqa: E731
    for m, n, k in ((64, 64, 327680), (64, 512, 81920), (16, 64, 163840), (1, 1, 2 ** 20), (33, 64, 40960), (64, 1984, 20480)):
        assert parts(m, n, k) >= 2, (m, n, k)
    for m, n, k in ((64, 64, 3968), (16, 64, 20480), (1, 496, 15872), (64, 1984, 3968), (16, 11904, 3968), (1, 32768, 4096), (17, 512, 8192)):
        assert parts(m, n, k) == 0, (m, n, k)


@pytest.mark.parametrize("m", [1, 16, 64, 65, 1000, 4096])
@pytest.mark.parametrize("n", [1, 64, 1488, 11904])
def test_a_part_has_eight_panels_at_least(m, n):
    for k in (1, 1000, 3968, 20480, 200000, 2 ** 20):
        parts = B.psgd_mx_product_workspace(m, n, k) // (4 * m * n)
        assert parts <= -(-k // 128) // 8

"""Refusals and layout of the Newton-Schulz, Muon and embedding calls. The binding's checks and the
C checks that need no context run on the CPU; the C checks of a context's calls need a device."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from rank_gradient_compression_powersgd_amd import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _raises(status, fn, text=""):
    with pytest.raises(B.PsgdError) as ei:
        fn()
    assert ei.value.status == status and text in str(ei.value), str(ei.value)


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not available")
def test_struct_layout_matches_c(tmp_path):
    structs = (B.psgd_ns_hparams, B.psgd_ns_matrix, B.psgd_muon_hparams, B.psgd_muon_matrix)
    body = "".join(f' printf("%zu\\n", sizeof({s.__name__}));\n'
                   + "".join(f' printf("%zu\\n", offsetof({s.__name__}, {f[0]}));\n' for f in s._fields_) for s in structs)
    body += ' printf("%d\\n%d\\n%d\\n%d\\n", PSGD_NS_FAST, PSGD_NS_ACCURATE, PSGD_I32, PSGD_I64);\n'
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "psgd.h"\nint main(void){\n' + body + " return 0; }\n")
    exe = tmp_path / "layout"
    r = subprocess.run(["gcc", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", "/opt/rocm/include",
                        str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    vals = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for s in structs:
        want.append(ctypes.sizeof(s))
        want += [getattr(s, f[0]).offset for f in s._fields_]
    assert vals == want + [B.PSGD_NS_FAST, B.PSGD_NS_ACCURATE, B.PSGD_I32, B.PSGD_I64]


def test_calls_without_a_context():
    lib = B.load_library()
    n = ctypes.c_int64(-1)
    assert lib.psgd_newton_schulz(None, None, None, None) == B.PSGD_EINVAL
    assert lib.psgd_ns_plan_create(None, None, 0, 3, 3, 0, None) == B.PSGD_EINVAL
    assert lib.psgd_ns_plan_destroy(None) == B.PSGD_OK
    assert lib.psgd_muon_attach(None, None, None, 3, 0) == B.PSGD_EINVAL
    assert lib.psgd_muon_update(None, None, None, None, None, None) == B.PSGD_EINVAL
    assert lib.psgd_embed_lookup(None, None, 1, 1, 1, 3, None, 8, 1, 1.0, None, 1, 3, None) == B.PSGD_EINVAL
    assert lib.psgd_embed_grad(None, None, 1, 3, None, 8, 1, 1, 1, 1.0, None, 1, 0, None, 0, None) == B.PSGD_EINVAL
    assert lib.psgd_embed_grad_workspace(1, 1, 1, None) == B.PSGD_EINVAL
    for bad in ((-1, 1, 1), (2 ** 25 + 1, 1, 1), (2 ** 31, 1, 1), (1, 0, 1), (1, 2 ** 20 + 1, 1), (1, 1, 0), (1, 1, 2 ** 23 + 1)):
        assert lib.psgd_embed_grad_workspace(*bad, ctypes.byref(n)) == B.PSGD_EINVAL
    assert lib.psgd_embed_grad_workspace(0, 1, 1, ctypes.byref(n)) == B.PSGD_OK and n.value > 0


def test_workspace_grows_past_32_bits():
    assert B.psgd_embed_grad_workspace(2 ** 25, 2 ** 20, 2 ** 14) > 2 ** 36


@pytest.mark.parametrize("vocab,dim", [(1, 1), (1031, 1000), (8195, 24), (32768, 3968), (262144, 7), (2 ** 20, 64)])
def test_a_workspace_serves_shorter_batches(vocab, dim):
    ns = sorted({max(0, x + d) for x in [0, 8, 32, 1000, 4096, 8192, 24576, 65536, 262144, 300000, 2 ** 22] + [(1 << 22) // dim] if x < 2 ** 24
                 for d in (-33, -1, 0, 1, 2, 31, 127, 129)})
    sizes = [B.psgd_embed_grad_workspace(n, vocab, dim) for n in ns]
    assert sizes == sorted(sizes), [(n, s) for n, s in zip(ns, sizes)]


def test_newton_schulz_binding_checks():
    from rank_gradient_compression_powersgd_amd import NewtonSchulzGroup
    f32, f16 = torch.zeros(4, 6), torch.zeros(4, 6, dtype=torch.float16)
    _raises(B.PSGD_EINVAL, lambda: NewtonSchulzGroup([], []))
    _raises(B.PSGD_EINVAL, lambda: NewtonSchulzGroup([f32], []))
    _raises(B.PSGD_EDTYPE, lambda: NewtonSchulzGroup([f32, f16], [f32, f32]))
    _raises(B.PSGD_EDTYPE, lambda: NewtonSchulzGroup([f32.double()], [f32]))
    _raises(B.PSGD_EINVAL, lambda: NewtonSchulzGroup([f32], [torch.zeros(6, 4)]))
    _raises(B.PSGD_EINVAL, lambda: NewtonSchulzGroup([torch.zeros(6, 4).t()], [f32]), "unit stride")
    _raises(B.PSGD_EINVAL, lambda: NewtonSchulzGroup([torch.zeros(6).expand(4, 6)], [f32]), "overlap")
    _raises(B.PSGD_EINVAL, lambda: NewtonSchulzGroup([f32], [f32]), "one GPU")
    _raises(B.PSGD_EINVAL, lambda: B.make_ns_matrix(torch.zeros(2, 3, 4), torch.zeros(2, 3, 4)))


def test_muon_binding_checks():
    p = torch.zeros(4, 8)
    _raises(B.PSGD_EINVAL, lambda: B.make_muon_matrix(p, torch.zeros(8, 4)))
    _raises(B.PSGD_EDTYPE, lambda: B.make_muon_matrix(p, p.half()))
    _raises(B.PSGD_EINVAL, lambda: B.make_muon_matrix(p, torch.zeros(4, 16)[:, :8]))
    _raises(B.PSGD_EINVAL, lambda: B.make_muon_matrix(torch.zeros(8, 4).t(), p))


def test_embedding_binding_checks():
    table, ids, out = torch.zeros(5, 8), torch.zeros(3, dtype=torch.int64), torch.zeros(3, 8)
    look = lambda t=table, i=ids, o=out: B.psgd_embed_lookup(0, t, i, o)                       # noqa: E731
    grad = lambda dx=out, i=ids, d=table, **kw: B.psgd_embed_grad(0, dx, i, d, **kw)           # noqa: E731
    _raises(B.PSGD_EINVAL, lambda: look(t=torch.zeros(8)))
    _raises(B.PSGD_EINVAL, lambda: look(t=torch.zeros(0, 8)))
    _raises(B.PSGD_EINVAL, lambda: look(o=torch.zeros(4, 8)))
    _raises(B.PSGD_EINVAL, lambda: look(o=torch.zeros(3, 7)))
    _raises(B.PSGD_EINVAL, lambda: look(o=torch.zeros(8, 3).t()))
    _raises(B.PSGD_EINVAL, lambda: look(o=torch.zeros(8).expand(3, 8)))
    _raises(B.PSGD_EINVAL, look, "one GPU")
    _raises(B.PSGD_EINVAL, lambda: grad(dx=torch.zeros(3, 9)))
    _raises(B.PSGD_EDTYPE, lambda: grad(d=table.half()))
    _raises(B.PSGD_EDTYPE, lambda: grad(i=ids.float()))
    _raises(B.PSGD_EINVAL, lambda: grad(i=torch.zeros(6, dtype=torch.int64)[::2]))
    _raises(B.PSGD_EDTYPE, lambda: grad(dx=out.double()))
    _raises(B.PSGD_EINVAL, grad, "one GPU")


@pytest.mark.gpu
def test_c_refusals():
    """Argument errors the library finds itself; nothing is launched, and each leaves its message."""
    from rank_gradient_compression_powersgd_amd import NewtonSchulzGroup, PowerSGDGroup, muon_hparams, ns_hparams
    x = torch.zeros(16, 16, device="cuda")
    ctx = B.psgd_create(0, 1)
    good = B.make_ns_matrix(x, torch.empty_like(x))
    create = lambda m, i=3, o=3, p=0: B.psgd_ns_plan_create(ctx, m, i, o, p)                   # noqa: E731
    _raises(B.PSGD_EINVAL, lambda: create([]))
    _raises(B.PSGD_EDTYPE, lambda: create([good], i=9))
    _raises(B.PSGD_EDTYPE, lambda: create([good], o=0))
    _raises(B.PSGD_EINVAL, lambda: create([good], p=2))
    for change in (dict(m=0), dict(n=0), dict(ld_in=15), dict(ld_out=15), dict(out=None), dict(m=2 ** 22 + 1),
                   {"in": x.data_ptr() + 2}):
        bad = B.make_ns_matrix(x, x)
        for k, v in change.items():
            setattr(bad, k, v)
        _raises(B.PSGD_EINVAL, lambda: create([good, bad]), "matrix 1")
    g = NewtonSchulzGroup([x], [torch.empty_like(x)])
    for bad, status in ((ns_hparams(steps=0), B.PSGD_EINVAL), (ns_hparams(steps=33), B.PSGD_EINVAL), (ns_hparams(eps=0.0), B.PSGD_EINVAL),
                        (ns_hparams(a=float("nan")), B.PSGD_EINVAL), (ns_hparams(a=5.0, b=0.0, c=0.0), B.PSGD_EUNSUPPORTED),
                        (ns_hparams(c=100.0), B.PSGD_EUNSUPPORTED), (ns_hparams(a=61.0, b=0.0, c=0.0, steps=1), B.PSGD_EUNSUPPORTED),
                        (ns_hparams(a=-61.0, b=1.0, c=0.0, steps=1), B.PSGD_EUNSUPPORTED)):
        _raises(status, lambda: g.run(bad))
    _raises(B.PSGD_EINVAL, lambda: B.psgd_newton_schulz(ctx, g.plan), "context")
    g.close()
    lib, null = B.load_library(), None
    look = lambda **k: lib.psgd_embed_lookup(ctx, *{**dict(t=x.data_ptr(), lt=16, v=16, d=16, td=3, i=x.data_ptr(), it=8, n=2, s=1.0,  # noqa: E731
                                                           o=x.data_ptr(), lo=16, od=3, st=None), **k}.values())
    for k in (dict(t=null), dict(o=null), dict(i=null), dict(lt=15), dict(lo=15), dict(n=-1), dict(v=0), dict(d=0), dict(s=float("inf")), dict(n=2 ** 25 + 1), dict(v=2 ** 31),
              dict(i=x.data_ptr() + 4), dict(t=x.data_ptr() + 2)):
        assert look(**k) == B.PSGD_EINVAL, k
    for k in (dict(td=7), dict(od=0), dict(it=3)):
        assert look(**k) == B.PSGD_EDTYPE, k
    ws = torch.empty(B.psgd_embed_grad_workspace(2, 16, 16), dtype=torch.uint8, device="cuda")
    grad = lambda **k: lib.psgd_embed_grad(ctx, *{**dict(dx=x.data_ptr(), ldx=16, dd=3, i=x.data_ptr(), it=8, n=2, v=16, d=16, s=1.0,  # noqa: E731
                                                         dt=x.data_ptr(), ldt=16, acc=0, w=ws.data_ptr(), wb=ws.numel(), st=None), **k}.values())
    for k in (dict(dx=null), dict(dt=null), dict(w=null), dict(wb=ws.numel() - 1), dict(w=ws.data_ptr() + 8), dict(ldx=15), dict(ldt=15)):
        assert grad(**k) == B.PSGD_EINVAL, k
    assert grad(dd=0) == B.PSGD_EDTYPE
    # Muon: an out buffer, attached state and sound scalars
    kw = dict(blocks=[0], scale=torch.ones(1, device="cuda"), rank=4, q0=[torch.zeros(16, 4)])
    no_out = PowerSGDGroup([x.half()], write_out=False, **kw)
    _raises(B.PSGD_EINVAL, lambda: no_out.attach_muon([x], [x.clone()]), "out buffer")
    no_out.close()
    grp = PowerSGDGroup([x.half()], **kw)
    _raises(B.PSGD_EINVAL, lambda: B.psgd_muon_update(grp.ctx, grp.plan, grp.skip, None, muon_hparams(0.1)), "psgd_muon_attach")
    _raises(B.PSGD_EINVAL, lambda: grp.attach_muon([x], []))
    _raises(B.PSGD_EINVAL, lambda: grp.attach_muon([torch.zeros(8, 16, device="cuda")], [torch.zeros(8, 16, device="cuda")]))
    _raises(B.PSGD_EINVAL, lambda: grp.step_muon(muon_hparams(0.1)), "attach_muon")
    grp.attach_muon([x], [x.clone()])
    kept = grp.muon_params[0], grp.momentum[0]
    _raises(B.PSGD_EINVAL, lambda: grp.attach_muon([], []))
    _raises(B.PSGD_EDTYPE, lambda: grp.attach_muon([x.double()], [x.clone()]))
    _raises(B.PSGD_EDTYPE, lambda: grp.attach_muon([x.clone()], [x.half()]))
    assert grp.muon_params[0] is kept[0] and grp.momentum[0] is kept[1]        # the library still points to them
    for bad in (muon_hparams(-1.0), muon_hparams(0.1, momentum=1.0), muon_hparams(0.1, weight_decay=float("inf")),
                muon_hparams(0.1, adjust=2), muon_hparams(0.1, steps=0)):
        _raises(B.PSGD_EINVAL, lambda: B.psgd_muon_update(grp.ctx, grp.plan, grp.skip, None, bad))
    _raises(B.PSGD_EINVAL, lambda: B.psgd_muon_update(grp.ctx, grp.plan, None, None, muon_hparams(0.1)), "skip_dev")
    torch.cuda.synchronize()
    assert bool((x == 0).all())
    grp.close()
    B.psgd_destroy(ctx)

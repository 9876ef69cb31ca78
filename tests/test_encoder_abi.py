"""C ABI of the embedding head's operators (include/maxsim_encoder.h) on a host
without a GPU: every declared function is exported with the binding's argument
count, and every refusal comes back before any device work.  Also the checks
that the binding makes itself, on host tensors."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "maxsim_encoder.h")
LIB = os.path.join(ROOT, "late_interaction_retrieval_amd", "libmaxsim.so")

if not os.path.exists(LIB):
    from late_interaction_retrieval_amd import build
    build.build()
from late_interaction_retrieval_amd import binding as bd  # noqa: E402

L = bd.lib()
A = ctypes.c_void_p(0x10000)  # aligned non-null fake pointers: never dereferenced
M = ctypes.c_void_p(0x10001)  # misaligned
OK, NULL, SHAPE, UNSUPPORTED, ALIGN, WORKSPACE = 0, 1, 2, 3, 4, 5
F16, BF16, F32, I8, E4M3 = 0, 1, 2, 3, 4


def test_every_declared_symbol_is_exported_with_binding_arity():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    decl = {m.group(1): len([p for p in m.group(2).split(",") if p.strip() and p.strip() != "void"])
            for m in re.finditer(r"^[A-Za-z_][\w \*]*?\b(maxsim_\w+)\s*\(([^)]*)\)\s*;", text, flags=re.M)}
    assert set(decl) == {"maxsim_rmsnorm_fwd", "maxsim_rmsnorm_bwd", "maxsim_rmsnorm_bwd_workspace_bytes",
                         "maxsim_quant_fp8", "maxsim_gemm_fp8", "maxsim_gemm_fp8_workspace_bytes", "maxsim_adamw"}
    raw = ctypes.CDLL(LIB)
    for name, nargs in decl.items():
        assert hasattr(raw, name), name
        assert len(bd.SIGNATURES[name][1]) == nargs, name
    assert bd._TENSOR.itemsize == 64


def norm_fwd(**kw):
    a = dict(x=A, ldx=64, res=A, ldr=64, w=A, wdt=BF16, R=3, H=64, dt=BF16, eps=1e-6, odt=BF16, y=A, ldy=64, scale=None,
             sum=A, lds=64, rstd=A, stream=None)
    a.update(kw)
    return L.maxsim_rmsnorm_fwd(*a.values())


@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(R=-1)), (SHAPE, dict(H=0)), (SHAPE, dict(eps=-1.0)), (SHAPE, dict(eps=float("nan"))),
    (SHAPE, dict(ldx=63)), (SHAPE, dict(ldy=63)), (SHAPE, dict(ldr=63)), (SHAPE, dict(lds=63)),
    (SHAPE, dict(ldx=1 << 32)), (UNSUPPORTED, dict(H=32769, ldx=40000, ldy=40000, ldr=40000, lds=40000)),
    (UNSUPPORTED, dict(dt=I8)), (UNSUPPORTED, dict(dt=7)), (UNSUPPORTED, dict(odt=9)), (UNSUPPORTED, dict(wdt=F16)),
    (NULL, dict(x=None)), (NULL, dict(y=None)), (NULL, dict(odt=I8)), (NULL, dict(odt=E4M3)),
    (ALIGN, dict(x=M)), (ALIGN, dict(res=M)), (ALIGN, dict(sum=M)), (ALIGN, dict(y=M)), (ALIGN, dict(w=M)),
    (ALIGN, dict(rstd=M)), (ALIGN, dict(odt=I8, scale=M)), (OK, dict(R=0)), (OK, dict(R=0, x=None, y=None)),
], ids=str)
def test_rmsnorm_fwd_refusals(want, kw):
    assert norm_fwd(**kw) == want


def norm_bwd(**kw):
    a = dict(dy=A, lddy=64, h=A, ldh=64, rstd=A, w=A, wdt=F32, ds=A, ldds=64, R=3, H=64, dt=F16, dx=A, lddx=64, dw=A,
             ws=A, nbytes=1 << 20, stream=None)
    a.update(kw)
    return L.maxsim_rmsnorm_bwd(*a.values())


@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(R=-1)), (SHAPE, dict(H=0)), (SHAPE, dict(lddy=1)), (SHAPE, dict(ldh=1)), (SHAPE, dict(lddx=1)),
    (SHAPE, dict(ldds=1)), (UNSUPPORTED, dict(dt=E4M3)), (UNSUPPORTED, dict(wdt=BF16)),
    (NULL, dict(dy=None)), (NULL, dict(h=None)), (NULL, dict(rstd=None)), (NULL, dict(dx=None)),
    (NULL, dict(R=5000, ws=None)), (ALIGN, dict(dy=M)), (ALIGN, dict(h=M)), (ALIGN, dict(ds=M)), (ALIGN, dict(dx=M)), (ALIGN, dict(dw=M)),
    (ALIGN, dict(ws=M)), (WORKSPACE, dict(R=5000, nbytes=64)), (OK, dict(R=0, dw=None)),
], ids=str)
def test_rmsnorm_bwd_refusals(want, kw):
    assert norm_bwd(**kw) == want


def quant(**kw):
    a = dict(x=A, ldx=64, R=3, C=64, dt=F32, br=1, q=A, ldq=64, s=A, qt=A, ldqt=16, st=A, stream=None)
    a.update(kw)
    return L.maxsim_quant_fp8(*a.values())


@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(R=-1)), (SHAPE, dict(C=-1)), (SHAPE, dict(ldx=63)), (SHAPE, dict(ldq=63)), (SHAPE, dict(ldqt=2)),
    (UNSUPPORTED, dict(dt=I8)), (UNSUPPORTED, dict(br=2)), (UNSUPPORTED, dict(br=0)),
    (SHAPE, dict(R=(1 << 31) - 1, C=(1 << 31) - 1, ldx=1 << 31, ldq=1 << 31, ldqt=1 << 31)),
    (NULL, dict(x=None)), (NULL, dict(q=None, qt=None)), (NULL, dict(s=None)), (NULL, dict(st=None)),
    (ALIGN, dict(x=M)), (ALIGN, dict(s=M)), (ALIGN, dict(st=M)), (OK, dict(R=0)), (OK, dict(C=0)),
], ids=str)
def test_quant_refusals(want, kw):
    assert quant(**kw) == want


def gemm(**kw):
    a = dict(A=A, lda=64, sa=A, B=A, ldb=64, sb=A, br=128, M=3, N=5, K=50, dt=BF16, c=A, ldc=5, ws=None, nbytes=0,
             stream=None)
    a.update(kw)
    return L.maxsim_gemm_fp8(*a.values())


@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(M=-1)), (SHAPE, dict(N=-1)), (SHAPE, dict(K=-1)), (SHAPE, dict(lda=48)), (SHAPE, dict(ldb=48)),
    (SHAPE, dict(ldc=4)), (UNSUPPORTED, dict(dt=E4M3)), (UNSUPPORTED, dict(br=64)),
    (UNSUPPORTED, dict(K=(1 << 22) + 1, lda=1 << 23, ldb=1 << 23)), (UNSUPPORTED, dict(lda=1 << 23)),
    (NULL, dict(A=None)), (NULL, dict(B=None)), (NULL, dict(sa=None)), (NULL, dict(sb=None)), (NULL, dict(c=None)),
    (ALIGN, dict(A=M)), (ALIGN, dict(B=M)), (ALIGN, dict(lda=72)), (ALIGN, dict(ldb=72)), (ALIGN, dict(c=M)),
    (ALIGN, dict(sa=M)), (ALIGN, dict(ws=M)), (OK, dict(M=0)), (OK, dict(N=0)),
], ids=str)
def test_gemm_refusals(want, kw):
    assert gemm(**kw) == want


def test_gemm_workspace_is_asked_for():
    need = L.maxsim_gemm_fp8_workspace_bytes(128, 128, 1 << 16)
    assert need > 0
    big = dict(M=128, N=128, K=1 << 16, lda=1 << 16, ldb=1 << 16, ldc=128)
    assert gemm(**big) == NULL
    assert gemm(ws=A, nbytes=need - 1, **big) == WORKSPACE
    for bad in ((-1, 5, 5), (5, 0, 5), (5, 5, 1 << 23)):
        assert L.maxsim_gemm_fp8_workspace_bytes(*bad) == 0


def adamw(entry=None, **kw):
    t = np.zeros(2, bd._TENSOR)
    for f in ("param", "grad", "m", "v", "m_scale", "v_scale"):
        t[f] = 0x10000
    t["n"] = 5
    for f, v in (entry or {}).items():
        t[f][1] = v
    a = dict(t=t.ctypes.data, n=2, pdt=F32, gdt=BF16, sdt=E4M3, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, step=1,
             dev=None, stream=None)
    a.update(kw)
    return L.maxsim_adamw(*a.values())


@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(n=-1)), (SHAPE, dict(step=0)), (SHAPE, dict(b1=1.0)), (SHAPE, dict(b1=-0.1)), (SHAPE, dict(b2=1.0)),
    (SHAPE, dict(b2=float("nan"))), (SHAPE, dict(eps=-1.0)), (SHAPE, dict(entry={"n": -1})),
    (UNSUPPORTED, dict(pdt=E4M3)), (UNSUPPORTED, dict(gdt=I8)), (UNSUPPORTED, dict(sdt=BF16)),
    (UNSUPPORTED, dict(entry={"master": 0x10000})), (NULL, dict(t=None)), (NULL, dict(entry={"param": 0})),
    (NULL, dict(entry={"grad": 0})), (NULL, dict(entry={"m": 0})), (NULL, dict(entry={"v": 0})),
    (NULL, dict(entry={"m_scale": 0})), (NULL, dict(entry={"v_scale": 0})), (ALIGN, dict(entry={"param": 0x10002})),
    (ALIGN, dict(entry={"grad": 0x10001})), (ALIGN, dict(sdt=F32, entry={"m": 0x10001})), (ALIGN, dict(dev=M)),
    (OK, dict(n=0)),
], ids=str)
def test_adamw_refusals(want, kw):
    assert adamw(**kw) == want


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 128)
    with pytest.raises(ValueError):
        bd.maxsim_rmsnorm_fwd(x)
    with pytest.raises(ValueError):
        bd.maxsim_rmsnorm_bwd(x, x, torch.zeros(4))
    with pytest.raises(ValueError):
        bd.maxsim_quant_fp8(x)
    q = x.to(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        bd.maxsim_gemm_fp8(q, torch.ones(4, 1), q, torch.ones(4, 1))


def test_binding_row_pitches():
    """_rows: the one pitch of all rows, or a refusal."""
    dev, f = torch.device("cpu"), torch.float32
    t = torch.zeros(6, 40)
    assert bd._rows(t, "t", t.shape, f, dev) == 40
    assert bd._rows(t[:, :8], "t", (6, 8), f, dev) == 40
    assert bd._rows(t[::2, 1:9], "t", (3, 8), f, dev) == 80
    assert bd._rows(t.reshape(2, 3, 40)[..., :8], "t", (2, 3, 8), f, dev) == 40
    assert bd._rows(t[2:3, :8], "t", (1, 8), f, dev) == 8
    assert bd._rows(t[:0], "t", (0, 40), f, dev) == 40
    for bad, shape in ((t.t(), (40, 6)), (t[:1].expand(6, 40), (6, 40)), (t.reshape(2, 3, 40)[:, :2], (2, 2, 40)),
                       (t[:, ::2], (6, 20)), (torch.zeros(64).as_strided((4, 8), (4, 1)), (4, 8))):
        with pytest.raises(ValueError):
            bd._rows(bad, "t", torch.Size(shape), f, dev)
    with pytest.raises(ValueError):
        bd._rows(t, "t", torch.Size((6, 41)), f, dev)
    with pytest.raises(TypeError):
        bd._rows(t, "t", t.shape, torch.float16, dev)


def test_binding_optimiser_table_refusals():
    p = [torch.zeros(5), torch.zeros(130)]
    s = [torch.zeros(5), torch.zeros(130)]
    q = [t.to(torch.float8_e4m3fn) for t in s]
    c = [torch.zeros(1), torch.zeros(2)]
    other = lambda ts: [t.clone() for t in ts]  # noqa: E731
    assert bd.AdamWTensors(p, s, other(s)).sizes == [5, 130]
    bd.AdamWTensors(p, q, other(q), c, other(c))
    with pytest.raises(ValueError):
        bd.AdamWTensors([], [], [])
    with pytest.raises(ValueError):
        bd.AdamWTensors(p, s[:1], s)
    with pytest.raises(ValueError):
        bd.AdamWTensors(p, q, q)             # 8 bits without scales
    with pytest.raises(ValueError):
        bd.AdamWTensors(p, s, s, c, c)       # scales without 8 bits
    with pytest.raises(ValueError):
        bd.AdamWTensors(p, q, q, c, [c[0], c[0]])
    with pytest.raises(ValueError):
        bd.AdamWTensors(p, s, s, masters=s)  # fp32 parameters have no masters
    with pytest.raises(TypeError):
        bd.AdamWTensors(p, q, s, c, c)
    with pytest.raises(TypeError):
        bd.AdamWTensors([t.int() for t in p], s, s)
    z = bd.AdamWTensors.zeros([t.bfloat16() for t in p], torch.float8_e4m3fn)
    assert z.masters[1].dtype == torch.float32 and z.m_scales[1].numel() == 2


def test_binding_optimiser_memory():
    """Tensors that share memory are refused when the table is made, and ones that have moved when it is used."""
    make = lambda *sizes: [torch.zeros(n) for n in sizes]  # noqa: E731
    p = make(5, 130)
    for bad in ([p[0], p[0]], [torch.zeros(200)[:130], p[0]]):
        with pytest.raises(ValueError):
            bd.AdamWTensors(bad, make(5, 5), make(5, 5))
    both = torch.zeros(200)
    with pytest.raises(ValueError, match="share memory"):
        bd.AdamWTensors([p[0], p[0]], make(5, 5), make(5, 5))
    with pytest.raises(ValueError, match="share memory"):
        bd.AdamWTensors([both[:100], both[99:]], make(100, 101), make(100, 101))
    with pytest.raises(ValueError, match="share memory"):
        bd.AdamWTensors(p, p, make(5, 130))
    bd.AdamWTensors([both[:100], both[100:]], make(100, 100), make(100, 100))  # neighbours
    bd.AdamWTensors([torch.zeros(0), p[0], torch.zeros(0)], make(0, 5, 0), make(0, 5, 0))
    w = torch.nn.Parameter(torch.zeros(7))
    tab = bd.AdamWTensors.zeros([w])
    tab._check_memory()
    w.data = torch.ones(7)
    with pytest.raises(ValueError, match="moved"):
        tab._check_memory()
    tab = bd.AdamWTensors.zeros([w])
    tab.m[0].untyped_storage().resize_(0)
    with pytest.raises(ValueError, match="moved"):
        tab._check_memory()

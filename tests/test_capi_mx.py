"""The C ABI of the microscaled operators: it exports what include/slope_mx.h
declares and refuses bad arguments on the host, before the GPU is touched."""
import ctypes
import os
import re

import pytest
import torch

import sparse_gemm_02_amd as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # aligned, never dereferenced: every call below fails its checks first
F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(S.library_path):
        from sparse_gemm_02_amd.build import build
        build()
    return S.library()


def test_exports_every_declared_symbol(lib):
    txt = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "slope_mx.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(slope_[a-z0-9_]+)\s*\(", txt))
    assert names == set(S.EXPORTED_SYMBOLS_MX)
    assert not names & (set(S.EXPORTED_SYMBOLS) | set(S.EXPORTED_SYMBOLS_INT8))
    for n in names:
        assert hasattr(lib, n) and callable(getattr(S, n)) and n in S.__all__


def _multi(lib, bits=8, count=2, pdt=(BF16, F32), gdt=(BF16, F32), p=(FAKE, 2 * FAKE), g=(3 * FAKE, 4 * FAKE),
           m=(5 * FAKE, 6 * FAKE), v=(7 * FAKE, 8 * FAKE), me=(9 * FAKE, 10 * FAKE), ve=(11 * FAKE, 12 * FAKE),
           n=(64, 65), hp=(1e-3, 0.9, 0.999, 1e-8, 0.01, 1)):
    vp = lambda a: None if a is None else (ctypes.c_void_p * len(a))(*a)
    i32 = lambda a: None if a is None else (ctypes.c_int32 * len(a))(*a)
    h = None if hp is None else ctypes.byref(S.AdamWParams(*hp))
    arrays = [i32(pdt), i32(gdt), vp(p), vp(g), vp(m), vp(v), vp(me), vp(ve), None if n is None else (ctypes.c_int64 * len(n))(*n)]
    return lib.slope_adamw_multi(bits, count, *[None if a is None else ctypes.addressof(a) for a in arrays], h, 0, None)


def test_adamw_multi_refusals(lib):
    f = lambda **k: _multi(lib, **k)
    for bits in (0, 4, 16, 64, -8):
        assert f(bits=bits) == -1
    assert f(count=-1) == -1 and f(hp=None) == -1
    for k in ("pdt", "gdt", "p", "g", "m", "v", "n"):
        assert f(**{k: None}) == -1, k
    assert f(me=None) == -1 and f(ve=None) == -1
    assert f(pdt=(BF16, 3)) == -1 and f(gdt=(-1, BF16)) == -1 and f(n=(64, -1)) == -1
    for k in ("p", "g", "m", "v", "me", "ve"):
        assert f(**{k: (FAKE * 20, 0)}) == -1, k                     # a tensor that is not there
    for hp in [(1e-3, 0.9, 0.999, 1e-8, 0.01, 0), (1e-3, 1.0, 0.999, 1e-8, 0.01, 1), (1e-3, 0.9, -0.1, 1e-8, 0.01, 1),
               (1e-3, 0.9, 0.999, -1.0, 0.01, 1), (float("nan"), 0.9, 0.999, 1e-8, 0.01, 1),
               (1e-3, 0.9, 0.999, 1e-8, float("inf"), 1)]:
        assert f(hp=hp) == -1, hp
    # addresses: an element's alignment is enough, less is not
    assert f(p=(FAKE + 1, 2 * FAKE)) == -3 and f(p=(FAKE, 2 * FAKE + 2)) == -3 and f(g=(3 * FAKE + 1, 4 * FAKE)) == -3
    assert f(bits=32, m=(5 * FAKE + 2, 6 * FAKE)) == -3 and f(bits=32, v=(7 * FAKE, 8 * FAKE + 1)) == -3
    assert f(n=(64, (1 << 34) + 1)) == -6


def test_adamw_multi_refuses_tensors_that_share_memory(lib):
    f = lambda **k: _multi(lib, **k)
    assert f(p=(FAKE, FAKE), pdt=(BF16, BF16)) == -1                 # the same weight twice
    assert f(p=(FAKE, FAKE + 126), pdt=(BF16, BF16)) == -1           # its last value
    assert f(m=(5 * FAKE, 5 * FAKE + 63)) == -1 and f(v=(7 * FAKE, 5 * FAKE)) == -1
    assert f(me=(9 * FAKE, 9 * FAKE + 1)) == -1 and f(ve=(9 * FAKE, 12 * FAKE)) == -1
    assert f(bits=32, m=(5 * FAKE, 5 * FAKE + 252)) == -1
    assert f(m=(FAKE, 6 * FAKE)) == -1                               # a moment over a weight
    assert f(g=(FAKE, 4 * FAKE)) == -1 and f(g=(3 * FAKE, 2 * FAKE + 124)) == -1   # a gradient over a weight
    assert f(g=(7 * FAKE - 126, 4 * FAKE)) == -1                     # the last value of a gradient over a moment


def test_adamw8_double_prune_refusals(lib):
    names = ("vals", "meta", "dw", "m", "me", "v", "ve", "ps", "pd")
    def f(dt=BF16, gdt=BF16, N=64, K=128, hp=(1e-3, 0.9, 0.999, 1e-8, 0.01, 1), pb=1 << 40, qb=1 << 40, **k):
        a = {n: k.get(n, (i + 1) * FAKE) for i, n in enumerate(names)}
        h = None if hp is None else ctypes.byref(S.AdamWParams(*hp))
        return lib.slope_adamw8_double_prune_packed(dt, gdt, a["vals"], a["meta"], a["dw"], a["m"], a["me"], a["v"], a["ve"],
                                                    N, K, h, 0, a["ps"], pb, a["pd"], qb, None)
    for n in names:
        assert f(**{n: None}) == -1, n
        if n not in ("me", "ve"):                                    # (scales may lie anywhere)
            assert f(**{n: 20 * FAKE + 8}) == -3, n
    assert f(dt=3) == -1 and f(gdt=7) == -1 and f(N=-1) == -1 and f(K=-1) == -1 and f(pb=-1) == -1 and f(qb=-1) == -1
    assert f(hp=None) == -1 and f(hp=(1e-3, 0.9, 0.999, 1e-8, 0.01, 0)) == -1
    assert f(dt=F32) == -6 and f(N=(1 << 21) + 16) == -6 and f(K=(1 << 21) + 64) == -6
    assert f(N=24) == -2 and f(K=96) == -2 and f(K=48) == -2
    assert f(pb=100) == -4 and f(qb=100) == -4
    assert f(N=0) == 0 and f(K=0) == 0


def test_adamw_moments_refusals(lib):
    f = lambda dt=BF16, m=FAKE, me=2 * FAKE, v=3 * FAKE, ve=4 * FAKE, n=64, mo=5 * FAKE, vo=6 * FAKE: \
        lib.slope_adamw_moments(dt, m, me, v, ve, n, mo, vo, None)
    assert f(dt=3) == -1 and f(n=-1) == -1 and f(mo=7 * FAKE, vo=7 * FAKE) == -1
    for k in ("m", "me", "mo", "v", "ve", "vo"):
        assert f(**{k: None}) == -1, k
    assert f(m=None, me=None, mo=None, v=None, ve=None, vo=None) == -1
    assert f(mo=5 * FAKE + 1) == -3 and f(dt=F32, vo=6 * FAKE + 2) == -3
    assert f(dt=F16) == -6 and f(n=(1 << 34) + 1) == -6


def test_binding_checks_lists():
    """The Python calls refuse lists that do not fit before anything reaches the library."""
    bf, u8 = torch.bfloat16, torch.uint8
    p = [torch.zeros(40, dtype=bf), torch.zeros(3, 5)]
    g = [torch.zeros(40), torch.zeros(3, 5, dtype=torch.float16)]
    m32 = [torch.zeros(40), torch.zeros(3, 5)]
    v32 = [torch.zeros(40), torch.zeros(3, 5)]
    m8 = [torch.zeros(40, dtype=u8), torch.zeros(3, 5, dtype=u8)]
    v8 = [torch.zeros(40, dtype=u8), torch.zeros(3, 5, dtype=u8)]
    e = [torch.zeros(2, dtype=u8), torch.zeros(1, dtype=u8)]
    step = dict(step=1, lr=1e-3)
    with pytest.raises(ValueError, match="GPU memory"):
        S.slope_adamw_multi(p, g, m32, v32, **step)
    with pytest.raises(ValueError, match="GPU memory"):
        S.slope_adamw_multi(p, g, m8, v8, m_exp=e, v_exp=e, **step)
    for lists in ((p, g[:1], m32, v32), (p, g, m32[:1], v32), (p[:1], g, m32, v32), ([], g, m32, v32)):
        with pytest.raises(ValueError, match="same length"):
            S.slope_adamw_multi(*lists, **step)
    with pytest.raises(ValueError, match="both m_exp and v_exp"):
        S.slope_adamw_multi(p, g, m8, v8, m_exp=e, **step)
    with pytest.raises(ValueError, match="same length"):
        S.slope_adamw_multi(p, g, m8, v8, m_exp=e, v_exp=e[:1], **step)
    with pytest.raises(TypeError, match=r"m\[0\] must be torch.float32"):
        S.slope_adamw_multi(p, g, m8, v32, **step)
    with pytest.raises(TypeError, match=r"v\[1\] must be torch.uint8"):
        S.slope_adamw_multi(p, g, m8, [v8[0], v32[1]], m_exp=e, v_exp=e, **step)
    with pytest.raises(ValueError, match=r"grads\[1\] must have 15 elements, got 14"):
        S.slope_adamw_multi(p, [g[0], g[1].view(-1)[:14]], m32, v32, **step)
    with pytest.raises(ValueError, match=r"m_exp\[0\] must have 2 elements, got 1"):
        S.slope_adamw_multi(p, g, m8, v8, m_exp=[e[1], e[1]], v_exp=e, **step)
    with pytest.raises(ValueError, match=r"params\[1\] must be contiguous"):
        S.slope_adamw_multi([p[0], torch.zeros(5, 3).t()], g, m32, v32, **step)
    with pytest.raises(TypeError, match="expected bfloat16"):
        S.slope_adamw_multi([p[0], torch.zeros(3, 5, dtype=torch.float64)], g, m32, v32, **step)
    S.slope_adamw_multi([], [], [], [], **step)                      # no tensors: nothing to do
    with pytest.raises(ValueError, match="one moment"):
        S.slope_adamw_moments(None, None, None, None)
    with pytest.raises(ValueError, match="m_exp must have shape"):
        S.slope_adamw_moments(m8[0], e[1], None, None, torch.zeros(40))
    with pytest.raises(ValueError, match="GPU memory"):
        S.slope_adamw_moments(m8[0], e[0], None, None, torch.zeros(40))


def test_4_bit_size_queries(lib):
    assert S.slope_mxfp4_row_bytes(0) == (0, 0) and S.slope_mxfp4_row_bytes(1) == (64, 16)
    assert S.slope_mxfp4_row_bytes(128) == (64, 16) and S.slope_mxfp4_row_bytes(4999) == (40 * 64, 160)
    assert S.slope_mxfp4_row_bytes(513) == (5 * 64, 32)
    assert S.slope_packed_sparse_mxfp4_bytes(27648, 9216) == 432 * 72 * 3328
    assert S.slope_packed_sparse_mxfp4_bytes(300, 272) == 5 * 3 * 3328 and S.slope_packed_sparse_mxfp4_bytes(0, 16) == 0
    for rows, cols in [(4, 8), (4, (1 << 21) + 16), (-1, 16), ((1 << 22) + 1, 16)]:
        with pytest.raises(S.SlopeError):
            S.slope_packed_sparse_mxfp4_bytes(rows, cols)
    for k in (-1, (1 << 22) + 1):
        with pytest.raises(S.SlopeError):
            S.slope_mxfp4_row_bytes(k)
    c = ctypes.c_int64()
    assert lib.slope_mxfp4_row_bytes(4, None, ctypes.byref(c)) == -1
    assert lib.slope_mxfp4_row_bytes(4, ctypes.byref(c), None) == -1
    assert lib.slope_packed_sparse_mxfp4_bytes(4, 16, None) == -1


def test_4_bit_refusals(lib):
    q = lambda dt=BF16, X=FAKE, T=4, K=64, c=FAKE, e=FAKE: lib.slope_quantize_mxfp4(dt, X, T, K, c, e, None)
    v = lambda dt=BF16, c=FAKE, e=FAKE, T=4, K=64, o=FAKE: lib.slope_mxfp4_values(dt, c, e, T, K, o, None)
    for f in (q, v):
        assert f(dt=3) == -1 and f(T=-1) == -1 and f(K=-1) == -1 and f(c=None) == -1 and f(e=None) == -1
        assert f(c=FAKE + 8) == -3 and f(e=FAKE + 4) == -3
        assert f(T=(1 << 22) + 1) == -6 and f(K=(1 << 22) + 1) == -6
    assert q(X=None) == -1 and q(X=FAKE + 1) == -3 and q(dt=F32, X=FAKE + 2) == -3
    assert v(o=None) == -1 and v(o=FAKE + 1) == -3 and v(dt=F32, o=FAKE + 2) == -3
    big = 1 << 40
    p = lambda dt=BF16, vals=FAKE, meta=FAKE, rows=64, cols=64, out=FAKE, nb=big: \
        lib.slope_pack_sparse_mxfp4(dt, vals, meta, rows, cols, out, nb, None)
    assert p(dt=5) == -1 and p(vals=None) == -1 and p(meta=None) == -1 and p(out=None) == -1
    assert p(rows=-1) == -1 and p(cols=-1) == -1 and p(nb=-1) == -1
    assert p(vals=FAKE + 2) == -3 and p(meta=FAKE + 4) == -3 and p(out=FAKE + 8) == -3
    assert p(cols=24) == -2 and p(dt=F32) == -6 and p(cols=(1 << 21) + 16) == -6 and p(rows=(1 << 22) + 1) == -6
    assert p(nb=3327) == -4
    y = lambda dt=BF16, c=FAKE, e=FAKE, T=4, K=64, w=FAKE, nb=big, N=64, Y=FAKE, ws=None, wb=0: \
        lib.slope_spmm_mxfp4_packed(dt, c, e, T, K, w, nb, N, Y, ws, wb, None)
    assert y(dt=3) == -1 and y(c=None) == -1 and y(e=None) == -1 and y(w=None) == -1 and y(Y=None) == -1
    assert y(T=-1) == -1 and y(K=-1) == -1 and y(N=-1) == -1 and y(nb=-1) == -1
    assert y(c=FAKE + 8) == -3 and y(e=FAKE + 8) == -3 and y(w=FAKE + 4) == -3 and y(Y=FAKE + 8) == -3
    assert y(K=24) == -2 and y(N=66) == -2
    assert y(T=(1 << 22) + 1) == -6 and y(N=(1 << 22) + 4) == -6 and y(K=(1 << 21) + 16) == -6
    assert y(nb=3327) == -4 and y(wb=-1) == -1 and y(ws=FAKE + 8, wb=64) == -3


def test_product_workspace_sizes(lib):
    """Parts of K for few tokens of a long K and few outputs: whole float32 [T, N] arrays, eight at most."""
    size = S.slope_spmm_mxfp4_workspace_bytes
    for T, K, N in [(64, 20480, 5120), (61, 20480, 5120), (64, 36864, 9216), (33, 65536, 64)]:
        parts, rest = divmod(size(T, K, N), 4 * T * N)
        assert rest == 0 and 2 <= parts <= 8, (T, K, N)
    for T, K, N in [(0, 64, 64), (4, 0, 64), (4, 64, 0), (65, 20480, 5120), (1, 9216, 27648), (64, 9216, 27648), (64, 16, 4),
                    (64, 1 << 21, 4)]:
        assert size(T, K, N) == 0, (T, K, N)
    b = ctypes.c_int64()
    f = lambda T=4, K=64, N=64, p=ctypes.byref(b): lib.slope_spmm_mxfp4_workspace_bytes(T, K, N, p)
    assert f(T=-1) == -1 and f(K=-1) == -1 and f(N=-1) == -1 and f(p=None) == -1
    assert f(K=24) == -2 and f(N=66) == -2
    assert f(T=(1 << 22) + 1) == -6 and f(N=(1 << 22) + 4) == -6 and f(K=(1 << 21) + 16) == -6


def test_binding_checks_4_bit_tensors():
    u8 = torch.uint8
    x, c, e = torch.zeros(3, 40), torch.zeros(3, 64, dtype=u8), torch.zeros(3, 16, dtype=u8)
    with pytest.raises(ValueError, match="GPU memory"):
        S.slope_quantize_mxfp4(x, c, e)
    with pytest.raises(ValueError, match="two dimensions"):
        S.slope_quantize_mxfp4(x.view(-1), c, e)
    with pytest.raises(ValueError, match="codes must have shape"):
        S.slope_quantize_mxfp4(x, c[:2], e)
    with pytest.raises(TypeError, match="exps must be torch.uint8"):
        S.slope_quantize_mxfp4(x, c, e.float())
    with pytest.raises(TypeError, match="expected bfloat16"):
        S.slope_quantize_mxfp4(x.double(), c, e)
    with pytest.raises(ValueError, match="X must be contiguous"):
        S.slope_quantize_mxfp4(torch.zeros(40, 3).t(), c, e)
    with pytest.raises(ValueError, match="exps must have shape"):
        S.slope_mxfp4_values(c, e[:, :2].contiguous(), x)
    w = torch.zeros(3328, dtype=u8)
    with pytest.raises(ValueError, match="Y must have shape"):
        S.slope_spmm_mxfp4_packed(c, e, 48, w, 64, torch.zeros(3, 60))
    with pytest.raises(ValueError, match="codes must have shape"):
        S.slope_spmm_mxfp4_packed(c, e, 144, w, 64, torch.zeros(3, 64))
    with pytest.raises(ValueError, match="GPU memory"):
        S.slope_spmm_mxfp4_packed(c, e, 48, w, 64, torch.zeros(3, 64))
    with pytest.raises(ValueError, match="values must have shape"):
        S.slope_pack_sparse_mxfp4(torch.zeros(64, 20, dtype=torch.bfloat16), torch.zeros(64, 2, dtype=torch.int32), 64, 48, w)

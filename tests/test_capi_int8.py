"""The C ABI of the RMS norm and the int8 products: it exports what
include/slope_int8.h declares and refuses bad arguments on the host, before the
GPU is touched (no compute calls)."""
import os
import re

import pytest
import torch

import sparse_gemm_02_amd as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # aligned, never dereferenced: every call below fails its checks first
BIG = 1 << 40   # a byte count that passes every size check
F32, BF16, F16 = 0, 1, 2
EPS = 1e-5


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(S.library_path):
        from sparse_gemm_02_amd.build import build
        build()
    return S.library()


def test_exports_every_declared_symbol(lib):
    txt = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "slope_int8.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(slope_[a-z0-9_]+)\s*\(", txt))
    assert names == set(S.EXPORTED_SYMBOLS_INT8) and not names & set(S.EXPORTED_SYMBOLS)
    for n in names:
        assert hasattr(lib, n) and callable(getattr(S, n)) and n in S.__all__


def test_size_queries(lib):
    assert S.slope_packed_sparse_i8_bytes(27648, 9216) == 108 * 72 * 20480
    assert S.slope_packed_sparse_i8_bytes(300, 272) == 2 * 3 * 20480
    assert S.slope_packed_sparse_i8_bytes(0, 16) == 0
    for rows, cols in [(4, 8), (4, S.I8_MAX_COLS + 16), (-1, 16), ((1 << 22) + 1, 16)]:
        with pytest.raises(S.SlopeError):
            S.slope_packed_sparse_i8_bytes(rows, cols)
    assert S.slope_rmsnorm_bwd_workspace_bytes(0, 768) == 0
    assert 3 * 771 * 4 <= S.slope_rmsnorm_bwd_workspace_bytes(3, 771) <= 3 * 771 * 4 + 256
    assert S.slope_rmsnorm_bwd_workspace_bytes(1 << 20, 9216) <= 1024 * 9216 * 4      # bounded in T
    with pytest.raises(S.SlopeError):
        S.slope_rmsnorm_bwd_workspace_bytes(-1, 8)
    assert lib.slope_rmsnorm_bwd_workspace_bytes(4, 8, None) == -1


def _norm(lib, dt=BF16, X=FAKE, res=None, gdt=BF16, gamma=FAKE, T=4, K=64, eps=EPS, H=None, Y=FAKE, q=None, qs=None,
          rstd=None):
    return lib.slope_rmsnorm(dt, X, res, gdt, gamma, T, K, eps, H, Y, q, qs, rstd, None)


def test_rmsnorm_refusals(lib):
    n = lambda **k: _norm(lib, **k)
    assert n(dt=3) == -1 and n(gdt=9) == -1 and n(X=None) == -1 and n(T=-1) == -1 and n(K=-1) == -1
    assert n(Y=None) == -1                                          # no output at all
    assert n(q=FAKE) == -1 and n(qs=FAKE) == -1                     # codes without scales, scales without codes
    assert n(H=FAKE, Y=FAKE) == -1                                  # h and y in one buffer
    assert n(q=FAKE, qs=FAKE, rstd=FAKE) == -1                      # scales and rstd in one buffer
    for eps in (0.0, -1e-5, float("nan"), float("inf"), 1e-40, 1e39):
        assert n(eps=eps) == -1, eps
    assert n(X=FAKE + 2) == -3 and n(res=FAKE + 8) == -3 and n(gamma=FAKE + 4) == -3 and n(H=FAKE + 8) == -3
    assert n(Y=FAKE + 2) == -3 and n(rstd=FAKE + 2) == -3 and n(q=FAKE, qs=FAKE + 1) == -3
    assert n(gdt=F16) == -6 and n(dt=F16, gdt=BF16) == -6 and n(dt=F32, gdt=BF16) == -6
    assert n(dt=F32, gdt=F32, q=FAKE, qs=FAKE) == -6                # codes come from 16-bit values
    assert n(T=(1 << 22) + 1) == -6 and n(K=(1 << 22) + 1) == -6


def _bwd(lib, dt=BF16, dY=FAKE, H=FAKE, rstd=FAKE, gdt=BF16, gamma=FAKE, dH=None, T=4, K=64, dX=2 * FAKE, dg=FAKE,
         ws=FAKE, wb=BIG):
    return lib.slope_rmsnorm_bwd(dt, dY, H, rstd, gdt, gamma, dH, T, K, dX, dg, 0, ws, wb, None)


def test_rmsnorm_bwd_refusals(lib):
    b = lambda **k: _bwd(lib, **k)
    assert b(dt=7) == -1 and b(gdt=-1) == -1 and b(dY=None) == -1 and b(H=None) == -1 and b(rstd=None) == -1
    assert b(T=-1) == -1 and b(K=-1) == -1 and b(wb=-1) == -1 and b(dX=None, dg=None) == -1
    assert b(gdt=F16) == -6 and b(dt=F32) == -6 and b(T=(1 << 22) + 1) == -6
    for k in ("dY", "H", "gamma", "dH", "dX", "dg", "ws"):
        assert b(**{k: FAKE + 8}) == -3, k
    assert b(rstd=FAKE + 2) == -3
    need = S.slope_rmsnorm_bwd_workspace_bytes(4, 64)
    assert b(wb=need - 1) == -4 and b(ws=None, wb=0) == -4
    assert b(dX=FAKE) == -1                                         # dX over H


def test_quantize_and_pack_refusals(lib):
    qr = lambda dt=BF16, X=FAKE, T=4, K=64, q=FAKE, s=FAKE: lib.slope_quantize_rows_i8(dt, X, T, K, q, s, None)
    assert qr(dt=5) == -1 and qr(X=None) == -1 and qr(q=None) == -1 and qr(s=None) == -1 and qr(T=-1) == -1
    assert qr(dt=F32) == -6 and qr(K=(1 << 22) + 1) == -6 and qr(X=FAKE + 2) == -3 and qr(s=FAKE + 2) == -3
    pk = lambda dt=BF16, v=FAKE, m=FAKE, r=256, c=256, s=FAKE, p=FAKE, b=BIG: lib.slope_pack_sparse_i8(
        dt, v, m, r, c, s, p, b, None)
    assert pk(dt=5) == -1 and pk(v=None) == -1 and pk(m=None) == -1 and pk(s=None) == -1 and pk(p=None) == -1
    assert pk(r=-1) == -1 and pk(b=-1) == -1 and pk(dt=F32) == -6 and pk(c=264) == -2
    assert pk(c=S.I8_MAX_COLS + 16) == -6 and pk(b=S.slope_packed_sparse_i8_bytes(256, 256) - 1) == -4
    assert pk(v=FAKE + 8) == -3 and pk(m=FAKE + 4) == -3 and pk(p=FAKE + 8) == -3 and pk(s=FAKE + 2) == -3


@pytest.mark.parametrize("fn", ["slope_spmm_i8_packed", "slope_spmm_i8_decode"])
def test_product_refusals(lib, fn):
    f = getattr(lib, fn)
    m = lambda out=BF16, x=FAKE, xs=FAKE, T=8, K=256, w=FAKE, b=BIG, ws=FAKE, N=64, y=FAKE: f(out, x, xs, T, K, w, b, ws,
                                                                                             N, y, None)
    assert m(out=4) == -1 and m(x=None) == -1 and m(xs=None) == -1 and m(w=None) == -1 and m(ws=None) == -1
    assert m(y=None) == -1 and m(T=-1) == -1 and m(K=-16) == -1 and m(N=-4) == -1 and m(b=-1) == -1
    assert m(K=264) == -2 and m(N=66) == -2
    assert m(K=S.I8_MAX_COLS + 16) == -6 and m(N=1 << 23) == -6
    assert m(x=FAKE + 8) == -3 and m(xs=FAKE + 2) == -3 and m(w=FAKE + 4) == -3 and m(ws=FAKE + 1) == -3
    assert m(y=FAKE + 8) == -3 and m(b=S.slope_packed_sparse_i8_bytes(64, 256) - 1) == -4
    assert m(T=S.I8_DECODE_MAX_TOKENS + 1 if fn.endswith("decode") else (1 << 22) + 1) == -6


def test_binding_refuses_shapes_types_and_places(lib):
    """Python-side checks, on host tensors: none of these reaches the library."""
    x = torch.zeros((4, 32), dtype=torch.bfloat16)
    g = torch.ones(32, dtype=torch.bfloat16)
    i8 = lambda *s: torch.zeros(s, dtype=torch.int8)
    f = lambda *s: torch.zeros(s, dtype=torch.float32)
    with pytest.raises(ValueError, match="GPU"):
        S.slope_rmsnorm(x, g, EPS, Y=torch.empty_like(x))
    with pytest.raises(ValueError, match="gamma"):
        S.slope_rmsnorm(x, g[:16].contiguous(), EPS, Y=torch.empty_like(x))
    with pytest.raises(ValueError, match="contiguous"):
        S.slope_rmsnorm(torch.zeros((32, 4), dtype=torch.bfloat16).t(), g, EPS, Y=torch.empty_like(x))
    with pytest.raises(ValueError, match="dimensions"):
        S.slope_rmsnorm(x[0], g, EPS, Y=torch.empty_like(x))
    with pytest.raises(TypeError, match="residual"):
        S.slope_rmsnorm(x, g, EPS, residual=x.float(), Y=torch.empty_like(x))
    with pytest.raises(TypeError, match="q must"):
        S.slope_rmsnorm(x, g, EPS, q=torch.zeros((4, 32), dtype=torch.uint8), q_scale=f(4))
    with pytest.raises(ValueError, match="q_scale"):
        S.slope_rmsnorm(x, g, EPS, q=i8(4, 32), q_scale=f(5))
    with pytest.raises(TypeError):
        S.slope_rmsnorm(x.double(), None, EPS, Y=x.double())
    with pytest.raises(ValueError, match="rstd"):
        S.slope_rmsnorm_bwd(x, x, f(3), g, dX=torch.empty_like(x))
    with pytest.raises(ValueError, match="H must"):
        S.slope_rmsnorm_bwd(x, x[:2].contiguous(), f(4), g, dX=torch.empty_like(x))
    with pytest.raises(TypeError, match="dgamma"):
        S.slope_rmsnorm_bwd(x, x, f(4), g, dgamma=f(32))
    with pytest.raises(ValueError, match="scale"):
        S.slope_quantize_rows_i8(x, i8(4, 32), f(1))
    with pytest.raises(ValueError, match="values"):
        S.slope_pack_sparse_i8(x, torch.zeros((4, 1), dtype=torch.int32), 4, 32, f(4), i8(20480))
    with pytest.raises(TypeError, match="meta"):
        S.slope_pack_sparse_i8(x[:, :16].contiguous(), f(4, 1), 4, 32, f(4), i8(20480))
    with pytest.raises(ValueError, match="w_scale"):
        S.slope_spmm_i8_packed(i8(4, 32), f(4), i8(20480), f(7), 8, f(4, 8))
    with pytest.raises(ValueError, match="Y must"):
        S.slope_spmm_i8_decode(i8(4, 32), f(4), i8(20480), f(8), 8, f(8, 4))


def test_adapter_of_the_int8_linear_runs_on_its_tensors_device(monkeypatch):
    """With another device current, the adapter's call (which takes the current
    device's stream) is made with the tensors' device current."""
    import contextlib
    from sparse_gemm_02_amd import layer as M
    made = []
    current = ["another"]

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d
        yield
        current[0] = before
    monkeypatch.setattr(torch.cuda, "device", device)
    for name in ("slope_quantize_rows_i8", "slope_spmm_i8_decode", "slope_spmm_i8_packed"):
        monkeypatch.setattr(M, name, lambda *a: None)
    monkeypatch.setattr(M, "slope_lowrank_workspace_bytes", lambda *a: 16)
    monkeypatch.setattr(M, "slope_lowrank_add", lambda *a, **k: made.append(current[0]))
    lin = M.Int8SparseLinear.__new__(M.Int8SparseLinear)
    torch.nn.Module.__init__(lin)
    lin.in_features, lin.out_features, lin.rank, lin.dtype = 32, 16, 4, torch.bfloat16
    for name, shape in (("packed", 16), ("w_scale", 16), ("L", (32, 4)), ("R", (4, 16))):
        lin.register_buffer(name, torch.zeros(shape))
    x = torch.zeros((3, 32), dtype=torch.bfloat16)
    lin(x)
    lin(M.Int8Rows(torch.zeros((3, 32), dtype=torch.int8), torch.zeros(3)), x)
    assert made == [x.device, x.device] and current == ["another"]

"""GPU parity of the RMS norm with residual addition and int8 codes, its
gradient, and the row quantizer, against the float64 oracle.

Tolerances.  h and the codes are exact functions of the inputs and must be equal
bit for bit.  Everything else carries fp32 rounding (2^-24 a step) and one
rounding to the output's format, at most half a step: HALF below.
* rstd: a sum of K squares by per-thread chains of at most 64 (70 in the long
  kernel's tests), 6 shuffle steps and 16 wave sums, each adding 2^-24 of a sum
  of positive terms; halved by the root; a few more roundings: below 2^-17.
* y: rstd's error and two products, then HALF of the value (plus half the
  smallest subnormal of the format).
* dX: (chain + 8) roundings of each of its three terms, with c's error a sum of
  signed products bounded by the mean of their magnitudes: 2^-17 of the terms'
  magnitudes, then HALF of the value.
* dgamma: chains of T / groups + 100 <= 256 steps: 2^-16 of the sum of
  magnitudes, then HALF of the value.
"""
import numpy as np
import pytest
import torch

import oracle
import sparse_gemm_02_amd as S

from gpu_util import say

pytestmark = pytest.mark.gpu
EPS = 1e-5
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}
GUARD = 64                                            # elements behind every output, left as they were


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    S.library()
    yield
    torch.cuda.synchronize()


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def rand(seed, *shape, sigma=1.0, dt="bf16", mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (mean + sigma * torch.randn(shape, generator=g)).to(DT[dt]).cuda()


class Out:
    """An output of the given shape with a guard behind it."""

    def __init__(self, shape, dtype):
        n = int(np.prod(shape))
        self.all = torch.full((n + GUARD,), 77, dtype=dtype, device="cuda")
        self.t = self.all[:n].view(shape)
        self.n = n

    def get(self):
        assert bool((self.all[self.n:] == 77).all()), "written past the end"
        return f64(self.t)


def close(got, ref, bound):
    bad = np.abs(got - ref) > bound
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], ref[bad][:3])


def check_norm(x, res, gamma, dt, codes=True, y=True, h=True, rstd=True):
    T, K = x.shape
    oH, oY, oq, oqs, orr = (Out((T, K), x.dtype), Out((T, K), x.dtype), Out((T, K), torch.int8),
                            Out((T,), torch.float32), Out((T,), torch.float32))
    S.slope_rmsnorm(x, gamma, EPS, residual=res, H=oH.t if h else None, Y=oY.t if y else None,
                    q=oq.t if codes else None, q_scale=oqs.t if codes else None, rstd=orr.t if rstd else None)
    torch.cuda.synchronize()
    href = oracle.residual_sum(f64(x), f64(res), dt)
    yref, rref = oracle.rmsnorm(href, f64(gamma), EPS)
    if h:
        assert np.array_equal(oH.get(), href)
    if rstd:
        close(orr.get(), rref, 2.0 ** -17 * rref)
    if y:
        close(oY.get(), yref, (HALF[dt] + 2.0 ** -16) * np.abs(yref) + TINY[dt])
    if codes:
        q, amax = oracle.row_codes_i8(href if gamma is None else href * f64(gamma))
        assert np.array_equal(oq.get(), q.astype(np.float64))
        close(oqs.get(), amax / 127 * rref, 2.0 ** -16 * amax / 127 * rref)


# every row layout: below a vector, one to four vectors of a wave, blocks of 1 to
# 8 vectors a thread, widths that are no multiple of a vector, the long kernel
WIDTHS = [1, 2, 7, 8, 9, 64, 65, 100, 511, 512, 520, 771, 1024, 2047, 2048, 2049, 4095, 4096, 5120, 8191, 9216, 12288,
          16383, 20480, 36864, 65536]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("K", WIDTHS)
def test_norm_widths(K, dt):
    say(f"[rmsnorm] K={K} {dt}")
    T = 5 if K > 4096 else 9
    x, res = rand(K, T, K, dt=dt), rand(K + 1, T, K, dt=dt)
    gamma = rand(K + 2, K, sigma=0.2, mean=1.0, dt=dt if K % 2 else "f32")
    check_norm(x, res, gamma, dt)


@pytest.mark.parametrize("K", [1, 3, 4, 5, 255, 256, 771, 1024, 4100, 9216, 32768])
def test_norm_f32(K):
    say(f"[rmsnorm] K={K} f32")
    check_norm(rand(1, 6, K, dt="f32"), rand(2, 6, K, dt="f32"), rand(3, K, mean=1.0, sigma=0.1, dt="f32"), "f32",
               codes=False)


@pytest.mark.parametrize("dt,K", [("bf16", 70000), ("f16", 65544), ("f32", 40001)])
def test_norm_rows_beyond_registers(dt, K):
    say(f"[rmsnorm long] {dt} K={K}")
    x, res = rand(1, 3, K, dt=dt), rand(2, 3, K, dt=dt)
    check_norm(x, res, rand(3, K, mean=1.0, sigma=0.1, dt="f32"), dt, codes=dt != "f32")
    check_norm(x, None, None, dt, codes=dt != "f32", h=False)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 63, 257, 1000])
def test_norm_token_counts(T):
    check_norm(rand(T, T, 768), rand(T + 1, T, 768), rand(5, 768, mean=1.0, sigma=0.1, dt="f32"), "bf16")
    check_norm(rand(T, T, 2304), None, rand(5, 2304, mean=1.0, sigma=0.1), "bf16")


@pytest.mark.parametrize("codes,y,h,rstd", [(1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1), (1, 0, 1, 0),
                                            (0, 1, 1, 1), (1, 1, 0, 1)])
@pytest.mark.parametrize("K", [96, 5120])
def test_norm_any_choice_of_outputs(K, codes, y, h, rstd):
    check_norm(rand(1, 7, K), rand(2, 7, K), rand(3, K, mean=1.0, sigma=0.1), "bf16", codes, y, h, rstd)


def test_norm_without_gamma_or_residual():
    check_norm(rand(1, 7, 640), None, None, "bf16")
    check_norm(rand(2, 7, 640, dt="f16"), rand(3, 7, 640, dt="f16"), None, "f16")


@pytest.mark.parametrize("K,dt", [(40, "bf16"), (771, "bf16"), (9216, "bf16"), (70000, "bf16"), (1445, "bf16"),
                                  (2049, "bf16"), (5121, "bf16"), (8191, "bf16"), (12301, "bf16"), (30001, "bf16"),
                                  (1001, "f32"), (4099, "f32"), (6001, "f32"), (12285, "f32")])
@pytest.mark.parametrize("place", ["H=X", "H=res", "Y=X", "Y=res", "H=res,Y=X", "H=X,Y=res"])
def test_norm_in_place(K, dt, place):
    x, res, g = rand(1, 300, K, dt=dt), rand(2, 300, K, dt=dt), rand(3, K, mean=1.0, sigma=0.1, dt=dt)
    hr, yr = torch.empty_like(x), torch.empty_like(x)
    S.slope_rmsnorm(x, g, EPS, residual=res, H=hr, Y=yr)
    where = dict(p.split("=") for p in place.split(","))
    a, b = x.clone(), res.clone()
    bufs = {"X": a, "res": b}
    outs = {k: bufs[v] for k, v in where.items()}
    S.slope_rmsnorm(a, g, EPS, residual=b, **outs)
    torch.cuda.synchronize()
    for k, t in outs.items():
        assert torch.equal(t, {"H": hr, "Y": yr}[k]), (place, k)


@pytest.mark.parametrize("K", [24, 1000, 5120, 70000])
def test_rows_without_a_scale(K):
    """Rows of zeros, with an infinity, with a NaN, in the residual, and one ordinary row between them."""
    x = rand(1, 6, K)
    x[0] = 0
    x[1, K - 1] = float("inf")
    x[2, 0] = float("nan")
    x[4] = -0.0
    res = torch.zeros_like(x)
    res[5, K // 2] = float("-inf")
    q = torch.full((6, K), 5, dtype=torch.int8, device="cuda")
    sc = torch.full((6,), 5.0, device="cuda")
    y = torch.empty_like(x)
    S.slope_rmsnorm(x, rand(2, K, mean=1.0, sigma=0.1), EPS, residual=res, q=q, q_scale=sc, Y=y)
    qp, sp = torch.full_like(q, 5), torch.full_like(sc, 5.0)
    S.slope_quantize_rows_i8(x, qp, sp)
    torch.cuda.synchronize()
    for codes, s, none in ((q, sc, (1, 2, 5)), (qp, sp, (1, 2))):
        for r in (0, 4):
            assert s[r] == 0 and not codes[r].any()
        for r in none:
            assert torch.isnan(s[r]) and not codes[r].any()
        assert torch.isfinite(s[3]) and int(codes[3].abs().max()) == 127
    assert not y[0].any() and not y[4].any() and torch.isnan(y[1, K - 1]) and torch.isnan(y[2]).all()
    assert torch.isfinite(y[3]).all()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_codes_at_every_tie(dt):
    """amax 254: every odd value is a tie; amax 381: every odd multiple of 1.5;
    and tiny and huge rows, whose reciprocals leave fp32's normal range first."""
    odd = torch.arange(-253, 254, dtype=torch.float32)
    rows = [torch.cat([odd, torch.tensor([254.0])]), torch.cat([torch.arange(-253, 254) * 1.5, torch.tensor([381.0])])]
    x = torch.stack(rows)
    scales = [1.0, 2.0 ** -14, 2.0 ** 7] if dt == "f16" else [1.0, 2.0 ** -110, 2.0 ** 110]
    for s in scales:
        xs = (x * s).to(DT[dt]).cuda()
        q, sc = torch.empty(xs.shape, dtype=torch.int8, device="cuda"), torch.empty(2, device="cuda")
        S.slope_quantize_rows_i8(xs, q, sc)
        torch.cuda.synchronize()
        qr, amax = oracle.row_codes_i8(f64(xs))
        assert np.array_equal(f64(q), qr.astype(np.float64)), s
        assert np.array_equal(f64(sc), oracle.round_to(amax / 127, "f32"))


@pytest.mark.parametrize("gdt", [None, "bf16", "f32"])
def test_codes_next_to_borders(gdt):
    """Many rows of few distinct magnitudes, so that quotients crowd around the borders."""
    g = torch.Generator().manual_seed(11)
    x = (torch.randint(-300, 301, (400, 512), generator=g).float() / 2).bfloat16().cuda()
    gamma = None if gdt is None else (torch.randint(1, 40, (512,), generator=g).float() / 3).to(DT[gdt]).cuda()
    check_norm(x, None, gamma, "bf16", y=False, h=False, rstd=False)


@pytest.mark.parametrize("K", [5, 24, 1001, 5120, 20000, 70000])
@pytest.mark.parametrize("dt,gdt,sizes", [("bf16", "bf16", (-48, -52, -64, -72, -80, -100)),
                                          ("bf16", "f32", (-48, -55, -64, -72, -80)), ("f16", "f32", (-7, -12))])
def test_codes_of_vanishing_products(K, dt, gdt, sizes):
    """Rows whose products h gamma lie around and below fp32's smallest numbers,
    where h and gamma themselves do not.  A scale is one rounding of amax / 127
    rstd (half a step, or half of fp32's smallest number), and rstd's error."""
    g = torch.Generator().manual_seed(K)
    x = torch.stack([torch.randn(K, generator=g) * 2.0 ** s for s in sizes]).to(DT[dt]).cuda()
    gamma = (1 + 0.2 * torch.randn(K, generator=g)) * 2.0 ** (-126 if dt == "f16" else -62)
    gamma = gamma.to(DT[gdt]).cuda()
    q, sc = torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(len(sizes), device="cuda")
    S.slope_rmsnorm(x, gamma, EPS, q=q, q_scale=sc)
    torch.cuda.synchronize()
    qr, amax = oracle.row_codes_i8(f64(x) * f64(gamma))
    assert np.array_equal(f64(q), qr.astype(np.float64))
    want = amax / 127 * oracle.rmsnorm(f64(x), None, EPS)[1]
    close(f64(sc), want, 2.0 ** -17 * want + TINY["f32"])


def test_codes_of_products_past_float32():
    """A finite product that fp32 does not hold is an infinity to the row."""
    x = torch.full((2, 64), 2.0 ** 80, dtype=torch.bfloat16, device="cuda")
    x[1] = 1.0
    gamma = torch.full((64,), 2.0 ** 80, dtype=torch.bfloat16, device="cuda")
    q, sc = torch.full((2, 64), 5, dtype=torch.int8, device="cuda"), torch.empty(2, device="cuda")
    S.slope_rmsnorm(x, gamma, EPS, q=q, q_scale=sc)
    torch.cuda.synchronize()
    assert torch.isnan(sc[0]) and not q[0].any() and bool((q[1] == 127).all()) and torch.isfinite(sc[1])


def test_norm_of_as_many_rows_as_there_may_be():
    """More rows than one grid takes: the last rows as they are by themselves."""
    T, K = 1 << 22, 24
    x = rand(6, 4096, K).repeat(T // 4096, 1)
    x[-4096:] = rand(7, 4096, K)
    gamma = rand(8, K, mean=1.0, sigma=0.2)

    def run(v, res):
        H, Y, q = torch.empty_like(v), torch.empty_like(v), torch.empty(v.shape, dtype=torch.int8, device="cuda")
        sc, rstd = torch.empty(len(v), device="cuda"), torch.empty(len(v), device="cuda")
        S.slope_rmsnorm(v, gamma, EPS, residual=res, H=H, Y=Y, q=q, q_scale=sc, rstd=rstd)
        return H, Y, q, sc, rstd
    all_rows, last = run(x, x), run(x[-4096:], x[-4096:])
    first = run(x[:4096], x[:4096])
    torch.cuda.synchronize()
    for a, l, f in zip(all_rows, last, first):
        assert torch.equal(a[-4096:], l)
        for at in (0, T // 2 - 4096, T // 2):
            assert torch.equal(a[at:at + 4096], f)


def test_quantizer_takes_unaligned_code_rows():
    x = rand(4, 3, 48)
    buf = torch.zeros(3 * 48 + 5, dtype=torch.int8, device="cuda")
    q, sc = buf[5:].view(3, 48), torch.empty(3, device="cuda")
    S.slope_quantize_rows_i8(x, q, sc)
    torch.cuda.synchronize()
    assert np.array_equal(f64(q), oracle.row_codes_i8(f64(x))[0].astype(np.float64)) and not buf[:5].any()


def test_empty_calls_write_nothing():
    x, e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), torch.empty(0, device="cuda")
    g = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    S.slope_rmsnorm(x, g, EPS, Y=torch.empty_like(x), rstd=e)
    S.slope_quantize_rows_i8(x, torch.empty((0, 64), dtype=torch.int8, device="cuda"), e)
    dg = torch.full_like(g, 3.0)
    S.slope_rmsnorm_bwd(x, x, e, g, dX=torch.empty_like(x), dgamma=dg, accumulate=True)
    torch.cuda.synchronize()
    assert bool((dg == 3).all())
    S.slope_rmsnorm_bwd(x, x, e, g, dgamma=dg)
    torch.cuda.synchronize()
    assert not dg.any()
    none = torch.empty((4, 0), dtype=torch.bfloat16, device="cuda")
    S.slope_rmsnorm(none, None, EPS, Y=torch.empty_like(none))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T", [1, 5, 300])
def test_quantizer_of_rows_without_values(T, dt):
    """K = 0: the scales of rows of zeros, so that a product with them is zeros."""
    sc = torch.full((T + GUARD,), float("nan"), device="cuda")
    sc[T:] = 77
    q = torch.empty((T, 0), dtype=torch.int8, device="cuda")
    S.slope_quantize_rows_i8(torch.empty((T, 0), dtype=DT[dt], device="cuda"), q, sc[:T])
    torch.cuda.synchronize()
    assert not sc[:T].any() and bool((sc[T:] == 77).all())
    y = torch.full((T, 8), 4.0, device="cuda")
    S.slope_spmm_i8_packed(q, sc[:T], torch.empty(0, dtype=torch.uint8, device="cuda"), torch.ones(8, device="cuda"), 8, y)
    torch.cuda.synchronize()
    assert not y.any()


# ------------------------------------------------------------------ gradient

def check_bwd(T, K, dt, gdt, with_dh, seed=0, accumulate=False, in_place=None):
    h, dy = rand(seed + 1, T, K, dt=dt), rand(seed + 2, T, K, dt=dt)
    gamma = None if gdt is None else rand(seed + 3, K, mean=1.0, sigma=0.2, dt=gdt)
    dh = rand(seed + 4, T, K, dt=dt) if with_dh else None
    g64, h64, dy64, dh64 = f64(gamma), f64(h), f64(dy), f64(dh)
    rstd = torch.from_numpy(oracle.rmsnorm(h64, g64, EPS)[1]).float().cuda()
    dX, dg = Out((T, K), h.dtype), Out((K,), DT[gdt or dt])
    start = rand(seed + 5, K, dt=gdt or dt)
    dg.t.copy_(start)
    ws = torch.empty(max(16, S.slope_rmsnorm_bwd_workspace_bytes(T, K)), dtype=torch.uint8, device="cuda")
    out = {"dy": dy, "dh": dh}.get(in_place, dX.t)
    S.slope_rmsnorm_bwd(dy, h, rstd, gamma, out, dg.t, ws, dH=dh, accumulate=accumulate)
    torch.cuda.synchronize()
    r64 = f64(rstd)
    dx_ref, dg_ref = oracle.rmsnorm_bwd(dy64, h64, r64, g64, dh64)
    a, xh = dy64 if g64 is None else dy64 * g64, h64 * r64[:, None]
    terms = r64[:, None] * (np.abs(a) + np.abs(xh) * np.abs(a * xh).mean(axis=1, keepdims=True))
    terms += 0 if dh64 is None else np.abs(dh64)
    got = f64(out) if in_place else dX.get()
    close(got, dx_ref, HALF[dt] * np.abs(dx_ref) + 2.0 ** -17 * terms + TINY[dt])
    base = f64(start) if accumulate else 0.0
    dg_ref = dg_ref + base
    close(dg.get(), dg_ref, HALF[gdt or dt] * np.abs(dg_ref) + 2.0 ** -16 * (np.abs(dy64 * xh).sum(axis=0) + np.abs(base))
          + TINY[gdt or dt])


@pytest.mark.parametrize("dt,gdt", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("K", [1, 7, 8, 9, 100, 512, 513, 771, 1024, 1025, 2048, 5120, 9216, 12289, 16384, 20480])
def test_bwd_widths(K, dt, gdt):
    say(f"[rmsnorm bwd] K={K} {dt}")
    check_bwd(11, K, dt, gdt, with_dh=K % 2 == 0, seed=K)


@pytest.mark.parametrize("dt,K", [("bf16", 32768), ("f16", 33001), ("f32", 16500)])
@pytest.mark.parametrize("in_place", [None, "dy", "dh"])
def test_bwd_rows_beyond_registers(dt, K, in_place):
    say(f"[rmsnorm bwd long] {dt} K={K} {in_place}")
    check_bwd(7, K, dt, "f32", with_dh=True, in_place=in_place)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 511, 769, 2500])
def test_bwd_token_counts(T):
    check_bwd(T, 768, "bf16", "f32", with_dh=True, seed=T)
    check_bwd(T, 2304, "f16", "f16", with_dh=False, seed=T)


@pytest.mark.parametrize("K", [768, 771, 9216])
def test_bwd_accumulates_and_works_in_place(K):
    check_bwd(100, K, "bf16", "bf16", with_dh=True, accumulate=True)
    check_bwd(100, K, "bf16", "f32", with_dh=True, in_place="dy")
    check_bwd(100, K, "bf16", None, with_dh=True, in_place="dh", accumulate=True)


@pytest.mark.parametrize("in_place", ["dy", "dh"])
@pytest.mark.parametrize("K,dt", [(301, "bf16"), (771, "bf16"), (2049, "f16"), (3333, "bf16"), (5121, "bf16"), (20481, "bf16"),
                                  (201, "f32"), (1001, "f32"), (6001, "f32"), (12285, "f32")])
def test_bwd_in_place_at_odd_widths(K, dt, in_place):
    check_bwd(700, K, dt, "f32", with_dh=True, in_place=in_place)


def test_bwd_one_output_at_a_time():
    T, K = 33, 1536
    h, dy, g = rand(1, T, K), rand(2, T, K), rand(3, K, mean=1.0, sigma=0.1, dt="f32")
    rstd = torch.from_numpy(oracle.rmsnorm(f64(h), f64(g), EPS)[1]).float().cuda()
    ws = torch.empty(S.slope_rmsnorm_bwd_workspace_bytes(T, K), dtype=torch.uint8, device="cuda")
    dx, dg, dx1, dg1 = torch.empty_like(h), torch.empty_like(g), torch.empty_like(h), torch.empty_like(g)
    S.slope_rmsnorm_bwd(dy, h, rstd, g, dx, dg, ws)
    S.slope_rmsnorm_bwd(dy, h, rstd, g, dX=dx1)
    S.slope_rmsnorm_bwd(dy, h, rstd, g, dgamma=dg1, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(dx, dx1) and torch.equal(dg, dg1)


def test_bwd_is_the_derivative_of_the_forward():
    """Central differences of the GPU's own fp32 forward along random directions.
    With step d the difference is off by d^2 f''' / 6 (f''' of order 10 here) and
    by the sums' rounding, T K 2^-24 over d in the worst case and its root in
    the mean: 1e-3 of sqrt(T K) covers both at d = 1e-2."""
    T, K = 6, 771
    x, g, dy = rand(1, T, K, dt="f32"), rand(2, K, mean=1.0, sigma=0.1, dt="f32"), rand(3, T, K, dt="f32")
    v, w = rand(4, T, K, dt="f32"), rand(5, K, dt="f32")
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")

    def f(x_, g_):
        S.slope_rmsnorm(x_, g_, EPS, Y=y, rstd=rstd)
        return float((y.double() * dy.double()).sum())
    d = 1e-2
    num = (f(x + d * v, g + d * w) - f(x - d * v, g - d * w)) / (2 * d)
    f(x, g)
    dx, dg = torch.empty_like(x), torch.empty_like(g)
    ws = torch.empty(S.slope_rmsnorm_bwd_workspace_bytes(T, K), dtype=torch.uint8, device="cuda")
    S.slope_rmsnorm_bwd(dy, x, rstd, g, dx, dg, ws)
    ana = float((dx.double() * v.double()).sum() + (dg.double() * w.double()).sum())
    assert abs(num - ana) <= 1e-3 * (T * K) ** 0.5 + 1e-3 * abs(ana), (num, ana)


def test_repeated_calls_are_bitwise_equal_and_other_streams_agree():
    T, K = 700, 5120
    x, res, g = rand(1, T, K), rand(2, T, K), rand(3, K, mean=1.0, sigma=0.1, dt="f32")
    dy = rand(4, T, K)

    def once():
        h, y, q = torch.empty_like(x), torch.empty_like(x), torch.empty((T, K), dtype=torch.int8, device="cuda")
        qs, rs = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        S.slope_rmsnorm(x, g, EPS, residual=res, H=h, Y=y, q=q, q_scale=qs, rstd=rs)
        dx, dg = torch.empty_like(x), torch.empty_like(g)
        ws = torch.empty(S.slope_rmsnorm_bwd_workspace_bytes(T, K), dtype=torch.uint8, device="cuda")
        S.slope_rmsnorm_bwd(dy, h, rs, g, dx, dg, ws)
        return h, y, q, qs, rs, dx, dg
    a, b = once(), once()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c = once()
    torch.cuda.synchronize()
    for p, q_, r in zip(a, b, c):
        assert torch.equal(p, q_) and torch.equal(p, r)

"""GPU parity of the int8 2:4 products against the oracle.

The sum of products is an integer below 2^31 and the rest is three float32
roundings in a fixed order, so every output is a determined number: codes,
scales, chunks and products are compared bit for bit."""
import numpy as np
import pytest
import torch

import oracle
import sparse_gemm_02_amd as S

from gpu_util import dev_meta, say

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
GUARD = 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    S.library()
    yield
    torch.cuda.synchronize()


def f64(t):
    return t.detach().cpu().double().numpy()


def compressed(N, K, dt, seed):
    """Compressed random 2:4 weight: (values tensor, meta words, float64 values)."""
    g = torch.Generator().manual_seed(seed)
    w = (0.02 * torch.randn((N, K), generator=g)).to(DT[dt])
    bits = w.view(torch.int16).numpy().view(np.uint16) if dt == "bf16" else w.numpy()
    mask, _ = oracle.prune24(bits)
    v, meta, _ = oracle.compress24(bits, mask)
    vt = torch.from_numpy(v.view(np.int16)).view(torch.bfloat16) if dt == "bf16" else torch.from_numpy(v)
    return vt.cuda(), meta, oracle.widen(v)


def chunks_reference(codes, meta, rows, cols):
    """int8 tile chunks as include/slope_int8.h states them, built with numpy."""
    n, tiles = -(-cols // 128), -(-rows // 256)
    vb = np.zeros((tiles * 256, n * 64), np.uint8)
    vb[:rows, :cols // 2] = codes.view(np.uint8)
    mw = np.zeros((tiles * 256, 4 * n), np.uint32)
    mw[:rows, :meta.shape[1]] = meta
    out = np.zeros((tiles, n, 20480), np.uint8)
    r = np.arange(256)
    for t in range(tiles):
        for s in range(n):
            blk = vb[256 * t:256 * t + 256, 64 * s:64 * s + 64].reshape(256, 4, 16)
            a = np.zeros_like(blk)
            for c in range(4):
                a[r, c ^ ((r >> 2) & 3)] = blk[:, c]
            out[t, s, :16384] = a.reshape(-1)
            out[t, s, 16384:] = np.ascontiguousarray(mw[256 * t:256 * t + 256, 4 * s:4 * s + 4]).view(np.uint8).reshape(-1)
    return out.reshape(-1)


def pack(vt, meta, N, K):
    n = S.slope_packed_sparse_i8_bytes(N, K)
    buf = torch.full((n + GUARD,), 0x5A, dtype=torch.uint8, device="cuda")
    sc = torch.full((N + GUARD,), -3.0, device="cuda")
    S.slope_pack_sparse_i8(vt, dev_meta(meta), N, K, sc[:N], buf[:n])
    torch.cuda.synchronize()
    assert bool((buf[n:] == 0x5A).all()) and bool((sc[N:] == -3.0).all())
    return buf[:n], sc[:N].contiguous()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("N,K", [(256, 256), (300, 272), (16, 16), (1, 16), (520, 1040), (257, 128), (4, 4096)])
def test_pack_layout(N, K, dt):
    say(f"[i8 pack] N={N} K={K} {dt}")
    vt, meta, v64 = compressed(N, K, dt, N + K)
    packed, sc = pack(vt, meta, N, K)
    q, amax = oracle.row_codes_i8(v64)
    assert np.array_equal(f64(sc), oracle.round_to(amax / 127, "f32"))
    assert np.array_equal(packed.cpu().numpy(), chunks_reference(q, meta, N, K))


def test_pack_rows_without_a_scale():
    vt, meta, v64 = compressed(40, 64, "bf16", 1)
    vt[3] = 0
    vt[17, 5] = float("inf")
    vt[39, 31] = float("nan")
    packed, sc = pack(vt, meta, 40, 64)
    q, amax = oracle.row_codes_i8(f64(vt))
    s = f64(sc)
    assert s[3] == 0 and np.isnan(s[17]) and np.isnan(s[39]) and np.isfinite(np.delete(s, [17, 39])).all()
    assert np.array_equal(packed.cpu().numpy(), chunks_reference(q, meta, 40, 64))


class Case:
    def __init__(self, T, K, N, seed, dt="bf16", full_range=False):
        self.T, self.K, self.N = T, K, N
        vt, self.meta, v64 = compressed(N, K, dt, seed)
        self.packed, self.ws = pack(vt, self.meta, N, K)
        self.wq = oracle.row_codes_i8(v64)[0]
        g = torch.Generator().manual_seed(seed + 1)
        lo = -128 if full_range else -127
        self.xq = torch.randint(lo, 128, (T, K), generator=g, dtype=torch.int8)
        self.xs = torch.rand(T, generator=g) * 0.05
        self.ref = lambda fmt: oracle.spmm_i8(self.xq.numpy(), f64(self.xs), self.wq, self.meta, K, f64(self.ws), fmt)

    def run(self, fn, out):
        n = self.T * self.N
        buf = torch.full((n + GUARD,), 9.0, dtype=DT[out], device="cuda")
        fn(self.xq.cuda(), self.xs.cuda(), self.packed, self.ws, self.N, buf[:n].view(self.T, self.N))
        torch.cuda.synchronize()
        assert bool((buf[n:] == 9.0).all()), "written past the end"
        return f64(buf[:n].view(self.T, self.N))


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,K,N", [(1, 16, 4), (3, 48, 20), (17, 272, 300), (32, 128, 32), (33, 1040, 96), (64, 2064, 516),
                                   (5, 5120, 1024), (61, 656, 260), (1, 272, 16900), (32, 1040, 17000), (33, 656, 17004),
                                   (64, 16, 20480), (9, 400, 33000), (40, 272, 33004), (50, 784, 8300), (20, 272, 8300)])
def test_few_token_product(T, K, N, out):
    say(f"[i8 decode] T={T} K={K} N={N} {out}")
    c = Case(T, K, N, seed=T + K)
    ref = c.ref(out)
    assert np.array_equal(c.run(S.slope_spmm_i8_decode, out), ref)
    assert np.array_equal(c.run(S.slope_spmm_i8_packed, out), ref)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,N", [(65, 768, 768), (256, 256, 256), (257, 272, 260), (511, 1040, 1028), (1000, 768, 2304),
                                   (300, 16, 8), (70, 128, 4), (513, 400, 1540), (300, 400, 2308), (130, 272, 9220),
                                   (300, 16, 2500), (190, 656, 5060)])
def test_product(T, K, N, out):
    say(f"[i8 product] T={T} K={K} N={N} {out}")
    c = Case(T, K, N, seed=T * 3 + K, dt="f16")
    assert np.array_equal(c.run(S.slope_spmm_i8_packed, out), c.ref(out))


# grids of every kind: full tiles with a last rows of half tiles, half tiles
# alone, full tiles alone, small and narrow tiles (one stage to more than a ring's);
# ragged in all three sizes
@pytest.mark.parametrize("T,K,N", [(4100, 144, 4612), (500, 272, 9216), (1000, 400, 9220), (515, 656, 4100),
                                   (2050, 128, 9220), (1000, 16, 2304), (200, 16, 5124), (65, 400, 16384),
                                   (253, 656, 7004), (256, 2320, 5120), (33000, 48, 100)])
def test_product_on_many_tiles(T, K, N):
    say(f"[i8 product] T={T} K={K} N={N}")
    c = Case(T, K, N, seed=T + N)
    assert np.array_equal(c.run(S.slope_spmm_i8_packed, "bf16"), c.ref("bf16"))


# the full tiles' ring of three slots over 19 stages: full tiles alone, full tiles
# with a last rows of half tiles, and half tiles alone
@pytest.mark.parametrize("T,K,N", [(1000, 2320, 9220), (4100, 2320, 4612), (500, 2320, 9216)])
def test_product_of_large_tiles_over_many_stages(T, K, N):
    say(f"[i8 product] T={T} K={K} N={N}")
    c = Case(T, K, N, seed=T + N)
    assert np.array_equal(c.run(S.slope_spmm_i8_packed, "bf16"), c.ref("bf16"))


@pytest.mark.parametrize("T", [1 << 22, (1 << 22) - 64])
def test_product_of_as_many_tokens_as_there_may_be(T):
    K, N = 16, 4
    c = Case(8, K, N, seed=3)
    g = torch.Generator().manual_seed(1)
    pick = torch.randint(0, 8, (T,), generator=g)
    xq, xs = c.xq[pick].contiguous().cuda(), c.xs[pick].contiguous().cuda()
    y = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda")
    S.slope_spmm_i8_packed(xq, xs, c.packed, c.ws, N, y)
    ref = torch.from_numpy(c.ref("bf16")).bfloat16().cuda()
    torch.cuda.synchronize()
    assert bool((y == ref[pick.cuda()]).all())


@pytest.mark.parametrize("T", [2, 80])
def test_long_sums_stay_in_int32(T):
    """The widest reduction with codes at the ends of int8: sums next to 2^31."""
    K, N = S.I8_MAX_COLS, 8
    vt = torch.ones((N, K // 2), dtype=torch.bfloat16, device="cuda")
    vt[1] = -1
    vt[2, ::2] = 0
    meta = np.full((N, K // 32), 0x44444444, np.uint32)         # positions 0 and 1 of every group
    packed, ws = pack(vt, meta, N, K)
    xq = torch.full((T, K), -128, dtype=torch.int8, device="cuda")
    xq[1] = 127
    xs = torch.full((T,), 1.0, device="cuda")
    y = torch.empty((T, N), device="cuda")
    for fn in (S.slope_spmm_i8_packed, *([S.slope_spmm_i8_decode] if T <= 64 else [])):
        y.fill_(0)
        fn(xq, xs, packed, ws, N, y)
        torch.cuda.synchronize()
        one = float(np.float32(-128 * 127 * (K // 2)) * np.float32(1 / np.float32(127)))
        assert abs(float(y[0, 0]) - one) <= 2.0 ** -22 * abs(one) and float(y[0, 1]) == -float(y[0, 0])
        assert abs(float(y[0, 2]) - one / 2) <= 2.0 ** -22 * abs(one)
        assert abs(float(y[1, 0]) - 127 * (K // 2)) <= 2.0 ** -22 * 127 * (K // 2)


def test_any_int8_code_is_taken():
    c = Case(20, 512, 64, seed=9, full_range=True)
    assert int(c.xq.min()) == -128
    assert np.array_equal(c.run(S.slope_spmm_i8_decode, "f32"), c.ref("f32"))
    assert np.array_equal(c.run(S.slope_spmm_i8_packed, "f32"), c.ref("f32"))


def test_scales_without_a_value_reach_only_their_own_rows_and_columns():
    c = Case(70, 256, 64, seed=2)
    c.xs[3] = float("nan")
    c.ws[5] = float("nan")
    c.ws[6] = 0.0
    for T, fn in ((70, S.slope_spmm_i8_packed), (64, S.slope_spmm_i8_decode)):
        y = torch.empty((T, 64), dtype=torch.bfloat16, device="cuda")
        fn(c.xq[:T].contiguous().cuda(), c.xs[:T].contiguous().cuda(), c.packed, c.ws, 64, y)
        torch.cuda.synchronize()
        nan = torch.isnan(y.cpu())
        want = torch.zeros_like(nan)
        want[3] = True
        want[:, 5] = True
        assert torch.equal(nan, want) and not y[[0, 1, 2, 4]][:, 6].any()


def test_empty_products():
    packed, ws = torch.zeros(20480, dtype=torch.uint8, device="cuda"), torch.zeros(8, device="cuda")
    for fn in (S.slope_spmm_i8_packed, S.slope_spmm_i8_decode):
        fn(torch.empty((0, 32), dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"), packed, ws, 8,
           torch.empty((0, 8), device="cuda"))
        y = torch.full((3, 8), 4.0, device="cuda")      # no reduction at all: zeros
        fn(torch.empty((3, 0), dtype=torch.int8, device="cuda"), torch.ones(3, device="cuda"),
           torch.empty(0, dtype=torch.uint8, device="cuda"), ws, 8, y)
        torch.cuda.synchronize()
        assert not y.any()


def test_layer_run_norm_codes_products_both_directions():
    """The operators as a layer uses them: residual + norm + codes into the
    forward product, dY's codes into the dX product with the double-pruned
    weight; every intermediate is the oracle's, so the outputs are too."""
    T, K, N = 130, 272, 320
    g = torch.Generator().manual_seed(4)
    x, res = (torch.randn((T, K), generator=g).bfloat16() for _ in range(2))
    gamma = 1 + 0.1 * torch.randn(K, generator=g)
    vt, meta, v64 = compressed(N, K, "bf16", 8)
    packed, ws = pack(vt, meta, N, K)
    h = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    q, qs = torch.empty((T, K), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    S.slope_rmsnorm(x.cuda(), gamma.cuda(), 1e-5, residual=res.cuda(), H=h, q=q, q_scale=qs)
    y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    S.slope_spmm_i8_packed(q, qs, packed, ws, N, y)
    vdp = torch.empty((K, N // 2), dtype=torch.bfloat16, device="cuda")
    mdp = torch.empty((K, (N // 4 + 7) // 8), dtype=torch.int32, device="cuda")
    S.slope_double_prune(vt, dev_meta(meta), N, K, vdp, mdp)
    pdp, wdp = pack(vdp, mdp.cpu().numpy().view(np.uint32), K, N)
    dy = torch.randn((T, N), generator=g).bfloat16().cuda()
    dq, dqs = torch.empty((T, N), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    S.slope_quantize_rows_i8(dy, dq, dqs)
    dx = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    S.slope_spmm_i8_packed(dq, dqs, pdp, wdp, K, dx)
    torch.cuda.synchronize()
    href = oracle.residual_sum(f64(x), f64(res), "bf16")
    qr, _ = oracle.row_codes_i8(href * f64(gamma))
    assert np.array_equal(f64(h), href) and np.array_equal(f64(q), qr.astype(np.float64))
    wq = oracle.row_codes_i8(v64)[0]
    assert np.array_equal(f64(y), oracle.spmm_i8(qr, f64(qs), wq, meta, K, f64(ws), "bf16"))
    dqr, damax = oracle.row_codes_i8(f64(dy))
    assert np.array_equal(f64(dq), dqr.astype(np.float64)) and np.array_equal(f64(dqs), oracle.round_to(damax / 127, "f32"))
    mdp_h = mdp.cpu().numpy().view(np.uint32)
    assert np.array_equal(f64(dx), oracle.spmm_i8(dqr, f64(dqs), oracle.row_codes_i8(f64(vdp))[0], mdp_h, N, f64(wdp), "bf16"))


def test_graph_replays_equal_the_eager_calls():
    """Norm with codes, both products and the norm's gradient in one captured
    graph, replayed on new inputs with eager work between the replays."""
    K, N, g = 768, 2304, torch.Generator().manual_seed(6)
    vt, meta, _ = compressed(N, K, "bf16", 12)
    packed, ws = pack(vt, meta, N, K)
    gamma = (1 + 0.1 * torch.randn(K, generator=g)).cuda()
    bufs = {}
    for T in (7, 200):
        b = bufs[T] = dict(x=torch.empty((T, K), dtype=torch.bfloat16, device="cuda"))
        for n in ("res", "h", "y", "dx"):
            b[n] = torch.empty_like(b["x"])
        b.update(q=torch.empty((T, K), dtype=torch.int8, device="cuda"), qs=torch.empty(T, device="cuda"),
                 rs=torch.empty(T, device="cuda"), out=torch.empty((T, N), dtype=torch.bfloat16, device="cuda"),
                 dg=torch.empty_like(gamma),
                 ws=torch.empty(S.slope_rmsnorm_bwd_workspace_bytes(T, K), dtype=torch.uint8, device="cuda"))

    def step():
        for T, b in bufs.items():
            S.slope_rmsnorm(b["x"], gamma, 1e-5, residual=b["res"], H=b["h"], Y=b["y"], q=b["q"], q_scale=b["qs"], rstd=b["rs"])
            (S.slope_spmm_i8_decode if T <= 64 else S.slope_spmm_i8_packed)(b["q"], b["qs"], packed, ws, N, b["out"])
            S.slope_rmsnorm_bwd(b["y"], b["h"], b["rs"], gamma, b["dx"], b["dg"], b["ws"])

    def fill(seed):
        r = torch.Generator().manual_seed(seed)
        for T, b in bufs.items():
            b["x"].copy_(torch.randn((T, K), generator=r))
            b["res"].copy_(torch.randn((T, K), generator=r))

    outs = ("h", "y", "q", "qs", "rs", "out", "dx", "dg")
    fill(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(1, 5):
        fill(seed)
        step()
        torch.cuda.synchronize()
        want = {T: {n: b[n].clone() for n in outs} for T, b in bufs.items()}
        for b in bufs.values():
            for n in outs:
                b[n].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for T, b in bufs.items():
            for n in outs:
                assert torch.equal(b[n], want[T][n]), (seed, T, n)


def test_first_call_of_a_kernel_inside_a_capture():
    """fp16 outputs on every kind of grid, captured before any eager call of them:
    what a launch sets up once must not be a stream operation."""
    shapes = [(40, 272, 260), (500, 272, 9216), (515, 656, 4100), (130, 272, 520), (150, 272, 2900), (300, 272, 2308),
              (130, 272, 9220), (5, 272, 16900), (5, 272, 33000), (50, 272, 33000), (33000, 48, 100)]
    cases = [Case(*s, seed=5) for s in shapes]
    args = [(c.xq.cuda(), c.xs.cuda(), c.packed, c.ws, c.N, torch.zeros((c.T, c.N), dtype=torch.float16, device="cuda"))
            for c in cases]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for a in args:
            S.slope_spmm_i8_packed(*a)
    for _ in range(3):
        for a in args:
            a[-1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for c, a in zip(cases, args):
            assert np.array_equal(f64(a[-1]), c.ref("f16"))


@pytest.mark.parametrize("T", [1, 16, 64, 512])
def test_at_opt_13b_width_on_sampled_outputs(T):
    K, N = 5120, 15360
    say(f"[i8 full] T={T}")
    g = torch.Generator().manual_seed(T)
    w = (0.02 * torch.randn((N, K), generator=g)).bfloat16().cuda()
    v = torch.empty((N, K // 2), dtype=torch.bfloat16, device="cuda")
    m = torch.empty((N, K // 32), dtype=torch.int32, device="cuda")
    S.slope_prune_compress24(w, v, m)
    meta = m.cpu().numpy().view(np.uint32)
    packed, ws = pack(v, meta, N, K)
    xq = torch.randint(-127, 128, (T, K), generator=g, dtype=torch.int8).cuda()
    xs = (torch.rand(T, generator=g) * 0.01).cuda()
    y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    S.slope_spmm_i8_packed(xq, xs, packed, ws, N, y)
    if T <= 64:
        y2 = torch.empty_like(y)
        S.slope_spmm_i8_decode(xq, xs, packed, ws, N, y2)
        assert torch.equal(y, y2)
    torch.cuda.synchronize()
    rows = np.unique(np.random.default_rng(T).integers(0, N, 200))
    wq = oracle.row_codes_i8(f64(v)[rows])[0]
    ref = oracle.spmm_i8(xq.cpu().numpy(), f64(xs), wq, meta[rows], K, f64(ws)[rows], "bf16")
    assert np.array_equal(f64(y)[:, rows], ref)

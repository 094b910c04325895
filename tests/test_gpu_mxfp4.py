"""GPU parity of 4-bit floating point: codes, scales, values and tile chunks bit for bit
against the oracle; the product within a bound counted from its float32 sums, and bit
for bit where every partial sum is a float32 number.

The product's bound.  Within a block all is exact; a matrix instruction adds the sums
of two blocks to an accumulator, so an output takes K / 64 such additions and at most
16 more where waves' sums meet.  Each rounds a partial sum of at most S = sum |x w|,
allowed 2^-23 of it (a float32 spacing): (K / 64 + 17) 2^-23 S, and then half a step of the
output's format."""
import functools

import numpy as np
import pytest
import torch

import oracle
import sparse_gemm_02_amd as S
from sparse_gemm_02_amd.layer import Mxfp4Rows, Mxfp4SparseLinear, ResidualRMSNorm, SparseAdamW, SparseLinear
from workloads import layer_inputs

from gpu_util import dev, dev_meta, host_f64, say

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
U8 = torch.uint8
GUARD = 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    S.library()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def quantize(x):
    """(codes, exps) of x with guard bytes behind both."""
    T, K = x.shape
    nc, ne = S.slope_mxfp4_row_bytes(K)
    c, e = (torch.full((T * n + GUARD,), 0xA5, dtype=U8, device="cuda") for n in (nc, ne))
    codes, exps = c[:T * nc].view(T, nc), e[:T * ne].view(T, ne)
    S.slope_quantize_mxfp4(x, codes, exps)
    torch.cuda.synchronize()
    assert (c[T * nc:] == 0xA5).all() and (e[T * ne:] == 0xA5).all()
    return codes, exps


def check_codes(x, codes, exps):
    want_c, want_e = oracle.mxfp4_codes(host_f64(x))
    assert np.array_equal(exps.cpu().numpy(), want_e)
    assert np.array_equal(codes.cpu().numpy(), oracle.mxfp4_rows(want_c))
    return want_c, want_e


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("T,K", [(1, 1), (1, 31), (2, 32), (3, 33), (5, 127), (4, 128), (7, 129), (33, 771), (3, 4999),
                                 (257, 256), (1, 20480)])
def test_codes_scales_and_values(dt, T, K):
    g = torch.Generator(device="cuda").manual_seed(T * 31 + K)
    x = torch.randn((T, K), device="cuda", generator=g) * torch.exp(2 * torch.randn((T, K), device="cuda", generator=g))
    x = x.to(DT[dt])
    c, e = check_codes(x, *quantize(x))
    want = oracle.mxfp4_values(c, e, K)
    codes, exps = quantize(x)
    for out in ("f32", "bf16"):
        raw = torch.full((T * K + GUARD,), 3.0, dtype=DT[out], device="cuda")
        S.slope_mxfp4_values(codes, exps, raw[:T * K].view(T, K))
        assert np.array_equal(host_f64(raw[:T * K]).reshape(T, K), want) and (raw[T * K:] == 3.0).all()
    o = torch.empty((T, K), dtype=torch.float16, device="cuda")
    S.slope_mxfp4_values(codes, exps, o)
    assert np.array_equal(host_f64(o), want.astype(np.float16).astype(np.float64))


def test_addresses_of_any_element():
    for dt in DT.values():
        for shift in (1, 3):
            raw = torch.randn(5 * 700 + 8, device="cuda").to(dt)
            x = raw[shift:shift + 3500].view(5, 700)
            codes, exps = quantize(x)
            check_codes(x, codes, exps)
            out = torch.zeros(3500 + 8, dtype=dt, device="cuda")
            S.slope_mxfp4_values(codes, exps, out[shift:shift + 3500].view(5, 700))
            ref = torch.empty(5, 700, dtype=dt, device="cuda")
            S.slope_mxfp4_values(codes, exps, ref)
            assert torch.equal(out[shift:shift + 3500].view(5, 700), ref)
            assert not out[:shift].any() and not out[shift + 3500:].any()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_every_16_bit_value_at_every_rounding(dt):
    """Each of the 65536 patterns in a block whose largest value puts it at each of the format's binades."""
    bits = np.arange(65536, dtype=np.uint16)
    x = (torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16) if dt == "bf16" else
         torch.from_numpy(bits.view(np.float16))).cuda().view(-1, 16)
    # alone with its neighbours (16 patterns apart by their last bits) and beside a value 1, 2, 4, .. 2^6 times as large
    for k in range(7):
        row = torch.zeros((x.shape[0], 32), dtype=x.dtype, device="cuda")
        row[:, :16] = x
        row[:, 20] = (x[:, 3].float() * 2.0 ** k).to(x.dtype)
        check_codes(row, *quantize(row))


def test_ties_bounds_and_blocks_without_values():
    v = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 6.5, 7.0, 0.2500001, 0.2499999, 4.999999, 5.000001])
    for scale in (1.0, 2.0 ** -100, 2.0 ** -126, 2.0 ** -149, 2.0 ** 100, 2.0 ** 125):
        x = torch.zeros((2 * len(v), 64))
        for i, t in enumerate(v):
            x[2 * i, 3], x[2 * i, 7] = t * scale, -4.0 * scale                 # below the block's largest or beside it
            x[2 * i + 1, 40], x[2 * i + 1, 41] = -t * scale, 6.0 * scale
        x = x.cuda()
        codes, exps = quantize(x)
        c, e = check_codes(x, codes, exps)
        out = torch.empty_like(x)
        S.slope_mxfp4_values(codes, exps, out)
        want = oracle.mxfp4_values(c, e, 64)
        assert np.array_equal(host_f64(out), want.astype(np.float32).astype(np.float64))
    for dt in DT.values():
        x = torch.ones((4, 96), dtype=dt, device="cuda")
        x[0, 5], x[1, 40], x[2, 95] = float("nan"), float("inf"), float("-inf")
        codes, exps = quantize(x)
        check_codes(x, codes, exps)
        out = torch.empty((4, 96), device="cuda")
        S.slope_mxfp4_values(codes, exps, out)
        bad = out.isnan()
        assert bad[0, :32].all() and bad[1, 32:64].all() and bad[2, 64:].all() and bad.sum() == 96
        assert (out[~bad] == 1).all()


def test_empty_calls():
    for T, K in ((0, 64), (3, 0), (0, 0)):
        x = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
        nc, ne = S.slope_mxfp4_row_bytes(K)
        codes, exps = torch.empty((T, nc), dtype=U8, device="cuda"), torch.empty((T, ne), dtype=U8, device="cuda")
        S.slope_quantize_mxfp4(x, codes, exps)
        S.slope_mxfp4_values(codes, exps, x)
    w = torch.empty(0, dtype=U8, device="cuda")
    codes, exps = torch.empty((3, 0), dtype=U8, device="cuda"), torch.empty((3, 0), dtype=U8, device="cuda")
    y = torch.full((3, 8), 5.0, device="cuda")
    S.slope_spmm_mxfp4_packed(codes, exps, 0, w, 8, y)                 # nothing to add: zeros
    assert (y == 0).all()
    S.slope_spmm_mxfp4_packed(codes[:0], exps[:0], 0, w, 8, y[:0])
    torch.cuda.synchronize()


# ------------------------------------------------------------------ the weight

@functools.lru_cache(maxsize=4)
def compressed(N, K, dt, seed, sigma=0.02):
    """(values tensor, meta words, float64 values) of a random compressed 2:4 weight."""
    g = torch.Generator().manual_seed(seed)
    w = (sigma * torch.randn((N, K), generator=g) * torch.exp(torch.randn((N, K), generator=g))).to(DT[dt])
    bits = w.view(torch.int16).numpy().view(np.uint16) if dt == "bf16" else w.numpy()
    v, meta, _ = oracle.compress24(bits, oracle.prune24(bits)[0])
    vt = torch.from_numpy(v.view(np.int16)).view(torch.bfloat16) if dt == "bf16" else torch.from_numpy(v)
    return vt.cuda(), meta, oracle.widen(v)


def pack(vt, meta, N, K):
    nb = S.slope_packed_sparse_mxfp4_bytes(N, K)
    raw = torch.full((nb + GUARD,), 0xA5, dtype=U8, device="cuda")
    S.slope_pack_sparse_mxfp4(vt, dev_meta(meta), N, K, raw[:nb])
    torch.cuda.synchronize()
    assert (raw[nb:] == 0xA5).all()
    return raw[:nb]


def chunks_reference(codes, exps, meta, rows, cols):
    """Tile chunks as include/slope_mx.h states them, one value at a time."""
    tiles, stages = -(-rows // 64), -(-cols // 128)
    out = np.zeros((tiles, stages, 3328), np.uint8)
    for r in range(rows):
        for b in range(-(-cols // 32)):
            chunk = out[r // 64, b // 4]
            q, rr, b4 = meta[r, b], r % 64, b % 4
            first = second = kept = 0
            for g in range(min(8, cols // 4 - 8 * b)):
                nib = (int(q) >> (4 * g)) & 15
                first |= int(codes[r, 16 * b + 2 * g]) << (4 * g)
                second |= int(codes[r, 16 * b + 2 * g + 1]) << (4 * g)
                kept |= ((1 << (nib & 3)) | (1 << (nib >> 2))) << (4 * g)
            for g in range(cols // 4 - 8 * b, 8):    # groups past a short block's end: position 0, code 0
                kept |= 1 << (4 * g)
            at = ((b4 // 2) * 64 + rr)
            chunk[at * 16 + (b4 % 2) * 8:][:8] = np.array([first, second], "<u4").view(np.uint8)
            chunk[2048 + at * 8 + (b4 % 2) * 4:][:4] = np.array([kept], "<u4").view(np.uint8)
            chunk[3 * 1024 + rr * 4 + b4] = exps[r, b]
    return out.reshape(-1)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("N,K", [(4, 16), (64, 128), (65, 144), (12, 272), (130, 48), (3, 1040)])
def test_chunks_byte_for_byte(dt, N, K):
    vt, meta, v = compressed(N, K, dt, N + K)
    if N > 4:
        vt = vt.clone()
        vt[2, 1] = float("nan")
        v = host_f64(vt)
    codes, exps = oracle.mxfp4_kept_codes(v, K)
    assert np.array_equal(pack(vt, meta, N, K).cpu().numpy(), chunks_reference(codes, exps, meta, N, K))


# ------------------------------------------------------------------ the product

def product_case(T, K, N, out, seed, wdt="bf16"):
    vt, meta, v = compressed(N, K, wdt, seed)
    packed = pack(vt, meta, N, K)
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, K), device="cuda", generator=g) * torch.exp(torch.randn((T, 1), device="cuda", generator=g))
    codes, exps = quantize(x.to(DT[out]))
    return packed, codes, exps, meta, v


def run(codes, exps, K, packed, N, out):
    T = codes.shape[0]
    raw = torch.full((T * N + GUARD,), 7.0, dtype=DT[out], device="cuda")
    S.slope_spmm_mxfp4_packed(codes, exps, K, packed, N, raw[:T * N].view(T, N))
    torch.cuda.synchronize()
    assert (raw[T * N:] == 7.0).all()
    return raw[:T * N].view(T, N)


def dense_weight(v, meta, K, rows=slice(None)):
    kept, e = oracle.mxfp4_kept_codes(v[rows], K)
    dense = oracle.decompress24(kept, meta[rows], K)
    pad = -K % 128
    codes = np.pad(dense, ((0, 0), (0, pad)))
    exps = np.pad(e, ((0, 0), (0, (K + pad) // 32 - e.shape[1])))
    return oracle.mxfp4_values(codes, exps, K)


SHAPES = [(1, 16, 4), (1, 128, 64), (3, 144, 68), (5, 4096, 260), (16, 272, 1000), (17, 2048, 36), (32, 1040, 132),
          (33, 512, 2052), (48, 5120, 64), (63, 784, 516), (64, 2048, 1024), (65, 768, 2304), (100, 1024, 128),
          (129, 272, 516), (200, 2320, 300), (255, 640, 256), (300, 128, 4100), (513, 1168, 772), (1000, 768, 516),
          (2, 20480, 1028), (64, 9216, 520), (7, 1024, 8196), (600, 256, 8196),
          (40, 65552, 68), (20, 327680, 8), (3, 655360, 36), (250, 1168, 24004), (1100, 400, 9220), (2100, 144, 9220), (1030, 16, 9216)]


@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("out", list(DT))
def test_product(T, K, N, out):
    say(f"[spmm_mxfp4] T={T} K={K} N={N} {out}")
    packed, codes, exps, meta, v = product_case(T, K, N, out, T + K + N, "f16" if out == "f16" else "bf16")
    y = run(codes, exps, K, packed, N, out)
    xv = torch.empty((T, K), device="cuda")
    S.slope_mxfp4_values(codes, exps, xv)
    rows = np.unique(np.concatenate([np.arange(0, N, 1 + N // 400), np.arange(N - 4, N)]))
    want, mass = oracle.spmm_mxfp4(host_f64(xv), dense_weight(v, meta, K, rows))
    got = host_f64(y)[:, rows]
    bound = (K / 64 + 17) * 2.0 ** -23 * mass + HALF_STEP[out] * np.abs(want) + (2.0 ** -25 if out == "f16" else 0)
    bad = np.abs(got - want) > bound
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])
    assert torch.equal(run(codes, exps, K, packed, N, out), y)         # the same sums again


SPLIT = [(2, 65552, 260), (9, 32768, 132), (16, 40960, 516), (17, 24592, 68), (32, 20480, 516), (33, 16400, 1028),
         (61, 20480, 1540), (64, 20368, 300), (64, 65552, 64), (40, 131072, 4), (64, 36864, 9216)]


@pytest.mark.parametrize("T,K,N", SPLIT)
@pytest.mark.parametrize("out", list(DT))
def test_product_in_parts(T, K, N, out):
    """Every number of parts that a workspace may hold, and a workspace that holds none."""
    if K * N > 1 << 27 and out != "bf16":
        pytest.skip("one large case is enough")
    say(f"[spmm_mxfp4 parts] T={T} K={K} N={N} {out}")
    need = S.slope_spmm_mxfp4_workspace_bytes(T, K, N)
    assert need >= 2 * 4 * T * N
    packed, codes, exps, meta, v = product_case(T, K, N, out, T + K + N, "f16" if out == "f16" else "bf16")
    xv = torch.empty((T, K), device="cuda")
    S.slope_mxfp4_values(codes, exps, xv)
    rows = np.unique(np.concatenate([np.arange(0, N, 1 + N // 100), np.arange(N - 4, N)]))
    want, mass = oracle.spmm_mxfp4(host_f64(xv), dense_weight(v, meta, K, rows))
    bound = (K / 64 + 17) * 2.0 ** -23 * mass + HALF_STEP[out] * np.abs(want) + (2.0 ** -25 if out == "f16" else 0)
    for size in sorted({0, 4 * T * N, *range(2 * 4 * T * N, need + 1, 4 * T * N), need, need + 4096}):
        ws = torch.full((size + GUARD,), 0xA5, dtype=U8, device="cuda")
        y = torch.full((T, N), 7.0, dtype=DT[out], device="cuda")
        S.slope_spmm_mxfp4_packed(codes, exps, K, packed, N, y, workspace=ws[:size])
        torch.cuda.synchronize()
        bad = np.abs(host_f64(y)[:, rows] - want) > bound
        assert not bad.any(), (size, np.argwhere(bad)[:3])
        assert (ws[size:] == 0xA5).all()
    assert torch.equal(run(codes, exps, K, packed, N, out), y)         # what the call takes by itself


@pytest.mark.parametrize("T,K,N", SHAPES + SPLIT[:-1])
def test_product_of_small_integers_is_exact(T, K, N):
    """Codes of 0 and +-1 with equal scales: every partial sum is an integer below 2^24."""
    rng = np.random.default_rng(T * K + N)
    wv = rng.choice([-1.0, 1.0], size=(N, K // 2))
    bits = (wv.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    nib = np.array([0b0100, 0b1000, 0b1100, 0b1001, 0b1101, 0b1110], np.uint32)      # i0 | i1 << 2
    groups = np.zeros((N, -(-K // 32) * 8), np.uint32)
    groups[:, :K // 4] = rng.choice(nib, size=(N, K // 4))
    meta = (groups.reshape(N, -1, 8) << (4 * np.arange(8, dtype=np.uint32))).sum(axis=2, dtype=np.uint32)
    vt = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).cuda()
    packed = pack(vt, meta, N, K)
    xi = rng.choice([-1.0, 0.0, 1.0], size=(T, K))
    xi[:, ::32] = 1.0                                                  # no block of zeros
    x = torch.from_numpy(xi).float().cuda()
    codes, exps = quantize(x)
    y = run(codes, exps, K, packed, N, "f32")
    w = oracle.decompress24(wv, meta, K)
    assert np.array_equal(host_f64(y), xi @ w.T)


@pytest.mark.parametrize("K,N", [(16384, 10308), (36864, 5060)])
def test_large_weights_take_the_values_of_small_ones(K, N):
    """Weights of more than 64 MB, whose loads few tokens make non-temporal, against the same rows in small
    weights.  Integers: every order of the sums is exact."""
    g = torch.Generator(device="cuda").manual_seed(K)
    vt = (torch.randint(0, 2, (N, K // 2), device="cuda", generator=g) * 2 - 1).bfloat16()
    nib = torch.tensor([4, 8, 12, 9, 13, 14], device="cuda")[torch.randint(0, 6, (N, K // 32, 8), device="cuda", generator=g)]
    meta = (nib << (4 * torch.arange(8, device="cuda"))).sum(-1).to(torch.int32)
    nb = S.slope_packed_sparse_mxfp4_bytes(N, K)
    assert nb >= 64 << 20
    packed = torch.empty(nb, dtype=U8, device="cuda")
    S.slope_pack_sparse_mxfp4(vt, meta, N, K, packed)
    for T in (1, 8, 9, 16, 17, 30, 33, 64):
        say(f"[spmm_mxfp4 large weight] T={T} K={K} N={N}")
        xi = torch.randint(-1, 2, (T, K), device="cuda", generator=g).float()
        xi[:, ::32] = 1.0
        codes, exps = quantize(xi)
        y = run(codes, exps, K, packed, N, "f32")
        for at in range(0, N, 1280):                                   # 20 chunks of rows
            n, row = min(1280, N - at), K // 128 * 3328
            part = packed[at // 64 * row:(at + n + 63) // 64 * row]
            assert torch.equal(run(codes, exps, K, part, n, "f32"), y[:, at:at + n])


def test_blocks_without_values_reach_their_outputs_only():
    T, K, N = 70, 512, 200
    for t in (1, 40, T):
        packed, codes, exps, meta, v = product_case(t, K, N, "f32", 5)
        clean = run(codes, exps, K, packed, N, "f32")
        e = exps.clone()
        e[t // 2, 3] = 255                                             # a token's block
        y = run(codes, e, K, packed, N, "f32")
        assert y[t // 2].isnan().all() and torch.equal(y[:t // 2], clean[:t // 2]) and torch.equal(y[t // 2 + 1:], clean[t // 2 + 1:])
        vt = torch.from_numpy(v).cuda().to(torch.bfloat16)
        vt[77, 100] = float("inf")                                     # a weight's block
        y = run(codes, exps, K, pack(vt, meta, N, K), N, "f32")
        assert y[:, 77].isnan().all()
        keep = [i for i in range(N) if i != 77]
        assert torch.equal(y[:, keep], clean[:, keep])


def test_far_scales():
    """Scales whose product leaves float32's range end in infinities and zeros, like the values' product."""
    K, N = 128, 64
    packed, codes, exps, meta, v = product_case(2, K, N, "f32", 9)
    vt = torch.from_numpy(v).cuda().to(torch.bfloat16)
    big = pack((vt.float() * 2.0 ** 100).bfloat16(), meta, N, K)
    e = exps.clone()
    e[0] = 250
    e[1] = 3
    y = run(codes, e, K, big, N, "f32")
    assert y[0].isinf().any() and not y[0].isfinite().any()
    xv = torch.empty((2, K), device="cuda")
    S.slope_mxfp4_values(codes, e, xv)
    kept, we = oracle.mxfp4_kept_codes(host_f64((vt.float() * 2.0 ** 100).bfloat16()), K)
    w = oracle.mxfp4_values(oracle.decompress24(kept, meta, K), we, K)
    want, mass = oracle.spmm_mxfp4(host_f64(xv[1:]), w)
    assert np.all(np.abs(host_f64(y[1:]) - want) <= (K / 64 + 17) * 2.0 ** -23 * mass + 2.0 ** -149)


@pytest.mark.parametrize("T,K", [(100003, 1), (70001, 33), (9973, 513), (4099, 2049), (65537, 40), (1031, 20479)])
def test_many_rows(T, K):
    """Row numbers come from a multiplication: every row of awkward widths, in both directions."""
    say(f"[mxfp4 rows] T={T} K={K}")
    x = torch.arange(T, device="cuda")[:, None] * 7 + torch.arange(K, device="cuda")[None, :] * 3
    x = ((x % 13) - 6).float().clamp(-6, 6)
    x[x.abs() == 5] = 4.0                                              # E2M1 numbers, and every block has few others
    codes, exps = quantize(x)
    y = torch.full_like(x, 9.0)
    S.slope_mxfp4_values(codes, exps, y)
    top = 32 * (K // 32)                                               # whole blocks hold a 6 or a 4, 2^0 either way
    assert torch.equal(x[:, :top], y[:, :top])
    assert ((x - y).abs() <= x.abs() / 6).all()
    z = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    S.slope_mxfp4_values(codes, exps, z)
    assert torch.equal(z.float(), y)


def test_values_of_more_items_than_a_launch_takes():
    T, K = 524291, 16384                                               # 2^30 items of eight values are 524288 rows
    say(f"[mxfp4_values] T={T} K={K}")
    nc, ne = S.slope_mxfp4_row_bytes(K)
    codes = torch.zeros((T, nc), dtype=U8, device="cuda")
    exps = torch.full((T, ne), 127, dtype=U8, device="cuda")
    rows = [0, 1, T // 2, 524286, 524287, 524288, 524289, T - 1]
    c, e = quantize(torch.randn((len(rows), K), device="cuda"))
    codes[rows], exps[rows] = c, e
    y = torch.full((T, K), 3.0, dtype=torch.bfloat16, device="cuda")
    S.slope_mxfp4_values(codes, exps, y)
    want = torch.empty((len(rows), K), dtype=torch.bfloat16, device="cuda")
    S.slope_mxfp4_values(c, e, want)
    assert torch.equal(y[rows], want) and want.any()
    y[rows] = 0
    assert not y.view(torch.int16).any()


def test_offsets_past_31_bits():
    """Codes, chunks and outputs of more than 2^31 bytes, sampled."""
    T, K, N = 300000, 16384, 64                                        # 2.46 GB of codes
    say(f"[spmm_mxfp4] T={T} K={K} N={N}")
    vt, meta, v = compressed(N, K, "bf16", 1)
    packed = pack(vt, meta, N, K)
    nc, ne = S.slope_mxfp4_row_bytes(K)
    codes = torch.zeros((T, nc), dtype=U8, device="cuda")
    exps = torch.full((T, ne), 127, dtype=U8, device="cuda")
    rows = [0, 1, T // 2, T - 257, T - 1]
    x = torch.randn((len(rows), K), device="cuda")
    c, e = quantize(x)
    codes[rows], exps[rows] = c, e
    y = run(codes, exps, K, packed, N, "f32")
    xv = torch.empty((len(rows), K), device="cuda")
    S.slope_mxfp4_values(c, e, xv)
    want, mass = oracle.spmm_mxfp4(host_f64(xv), dense_weight(v, meta, K))
    assert np.all(np.abs(host_f64(y[rows]) - want) <= (K / 64 + 17) * 2.0 ** -23 * mass)
    y[rows] = 0
    assert not y.any()
    del codes, exps, y
    # many outputs: 2.3e9 bytes of fp32, a weight of 64-row chunks to the last
    T, K, N = 1100, 16, 524292
    nib = np.full((N, 1), 0x0000CCCC, np.uint32)                       # positions 0 and 3
    values = torch.ones((N, K // 2), dtype=torch.bfloat16, device="cuda")
    values[-5:] = 2.0
    packed = pack(values, nib, N, K)
    x = torch.zeros((T, K), device="cuda")
    x[:, 0], x[:, 3] = 1.0, torch.arange(T, device="cuda") % 2
    codes, exps = quantize(x)
    y = run(codes, exps, K, packed, N, "f32")
    want = (1.0 + torch.arange(T, device="cuda") % 2)[:, None]
    assert (y[:, :-5] == want).all() and (y[:, -5:] == 2 * want).all()


# ------------------------------------------------------------------ modules, graphs, streams

def test_linear_module_and_its_adapter():
    T, N, K, r = 37, 272, 528, 8
    d = layer_inputs(K, N, T, r, "bf16", seed=3)
    layer = SparseLinear(dev(d["W"]), dev(d["L"]), dev(d["R"]))
    plain = SparseLinear(dev(d["W"]))
    x = dev(d["X"])
    lin, lin0 = Mxfp4SparseLinear(layer), Mxfp4SparseLinear(plain)
    xq = Mxfp4Rows.of(x)
    want, mass = oracle.spmm_mxfp4(host_f64(xq.values()), dense_weight(host_f64(layer.values), layer.meta.cpu().numpy().view(np.uint32), K))
    y0 = lin0(x)
    tol = (K / 64 + 17) * 2.0 ** -23 * mass + 2.0 ** -8 * np.abs(want)
    assert np.all(np.abs(host_f64(y0) - want) <= tol)
    assert torch.equal(lin0(xq), y0) and torch.equal(lin0(x.view(1, T, K)), y0.view(1, T, N))
    y = lin(x)
    ad = host_f64(x) @ host_f64(layer.L) @ host_f64(layer.R)
    # the adapter's addition reads and rounds Y once more (half a step of bf16), its own sums within 2^-14 of its size
    assert np.all(np.abs(host_f64(y) - (want + ad)) <= tol + 2.0 ** -8 * np.abs(want + ad) + 2.0 ** -8 * np.abs(want) +
                  2.0 ** -14 * (np.abs(host_f64(x)) @ np.abs(host_f64(layer.L)) @ np.abs(host_f64(layer.R))))
    assert torch.equal(lin(xq, x), y)
    # rows cut from larger tensors, at any address; no rows
    wide = torch.zeros((T, K + 3), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:] = x
    assert torch.equal(lin0(wide[:, 3:]), y0)
    cut = Mxfp4Rows(xq.codes[5:9], xq.exps[5:9], K)
    assert torch.equal(lin0(cut), lin0(x[5:9])) and lin0(x[:0]).shape == (0, N)
    with pytest.raises(ValueError, match="adapter needs"):
        lin(xq)
    with pytest.raises(ValueError, match="one input"):
        lin(x, x.clone())
    with pytest.raises(ValueError, match="in_features"):
        lin0(x.half())
    with pytest.raises(ValueError, match="in_features"):
        lin0(Mxfp4Rows.of(x[:, :512].contiguous()))
    lin.half()
    assert lin.packed.dtype is U8 and lin.L.dtype is torch.bfloat16 and torch.equal(lin(x), y)


def test_a_model_trained_with_8_bit_moments_and_served_in_4_bits():
    """The operators as they are used together: training steps with 8-bit moments, then norm, codes and
    product of the trained layers on their 4-bit weights, in both directions."""
    T, D, H = 96, 256, 512
    d1, d2 = (layer_inputs(a, b, T, 8, "bf16", seed=4, index=i) for i, (a, b) in enumerate(((D, H), (H, D))))
    norm = ResidualRMSNorm(D, dtype=torch.bfloat16)
    l1, l2 = SparseLinear(dev(d1["W"]), dev(d1["L"]), dev(d1["R"])), SparseLinear(dev(d2["W"]))
    opt = SparseAdamW([norm, l1, l2], lr=1e-3, state_bits=8)
    x = dev(d1["X"])
    first = [p.detach().clone() for p in (norm.weight, l1.values, l1.L, l2.values)]
    for _ in range(3):
        out = l2(torch.nn.functional.silu(l1(norm(x))))
        out.backward(dev(d2["dY"]))
        opt.step()
        opt.zero_grad()
    # (the norm's weights stand at 1 in bfloat16, where a step of about lr = 0.001 is below half a spacing, 2^-9)
    for p, f in zip((norm.weight, l1.values, l1.L, l2.values), first):
        assert p.isfinite().all() and torch.equal(p.detach(), f) == (p is norm.weight)
    s1, s2 = Mxfp4SparseLinear(l1), Mxfp4SparseLinear(l2)
    with torch.no_grad():
        y = norm(x)
    h = s1(y)
    z = s2(torch.nn.functional.silu(h))
    meta = lambda l: l.meta.cpu().numpy().view(np.uint32)
    xv = host_f64(Mxfp4Rows.of(y).values())
    want, mass = oracle.spmm_mxfp4(xv, dense_weight(host_f64(l1.values), meta(l1), D))
    ad = host_f64(y) @ host_f64(l1.L) @ host_f64(l1.R)
    tol = 2.0 ** -23 * (D / 64 + 17) * mass + 2.0 ** -7 * (np.abs(want) + np.abs(want + ad)) + \
        2.0 ** -14 * (np.abs(host_f64(y)) @ np.abs(host_f64(l1.L)) @ np.abs(host_f64(l1.R)))
    assert np.all(np.abs(host_f64(h) - (want + ad)) <= tol)
    hv = host_f64(Mxfp4Rows.of(torch.nn.functional.silu(h)).values())
    want, mass = oracle.spmm_mxfp4(hv, dense_weight(host_f64(l2.values), meta(l2), H))
    assert np.all(np.abs(host_f64(z) - want) <= 2.0 ** -23 * (H / 64 + 17) * mass + 2.0 ** -8 * np.abs(want))
    # dX of the second layer on 4-bit codes of dY and W_dp^T
    vdp, mdp, _ = oracle.double_prune(l2.values.detach().cpu().view(torch.int16).numpy().view(np.uint16), meta(l2), D, H)
    vt = torch.from_numpy(vdp.view(np.int16)).view(torch.bfloat16).cuda()
    codes, exps = quantize(dev(d2["dY"]))
    dx = run(codes, exps, D, pack(vt, mdp, H, D), H, "bf16")
    dv = torch.empty((T, D), device="cuda")
    S.slope_mxfp4_values(codes, exps, dv)
    want, mass = oracle.spmm_mxfp4(host_f64(dv), dense_weight(oracle.widen(vdp), mdp, D))
    assert np.all(np.abs(host_f64(dx) - want) <= 2.0 ** -23 * (D / 64 + 17) * mass + 2.0 ** -8 * np.abs(want))


@pytest.mark.parametrize("T,K,N", [(1, 1040, 772), (40, 1040, 772), (300, 1040, 772), (64, 20480, 516)])
def test_captured_and_on_another_stream(T, K, N):
    packed, codes, exps, meta, v = product_case(T, K, N, "bf16", T)
    x = [torch.randn((T, K), device="cuda").bfloat16() for _ in range(3)]
    eager = []
    for t in x:
        c, e = quantize(t)
        eager.append(run(c, e, K, packed, N, "bf16").clone())
    side = torch.cuda.Stream()
    xin, y = torch.empty_like(x[0]), torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    c, e = torch.empty_like(codes), torch.empty_like(exps)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        xin.copy_(x[0])
        S.slope_quantize_mxfp4(xin, c, e)
        S.slope_spmm_mxfp4_packed(c, e, K, packed, N, y)
    side.synchronize()
    assert torch.equal(y, eager[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.slope_quantize_mxfp4(xin, c, e)
        S.slope_spmm_mxfp4_packed(c, e, K, packed, N, y)
    for i in (0, 1, 2, 1):
        xin.copy_(x[i])
        y.fill_(float("nan"))
        with torch.cuda.stream(side):                                  # (parts take a workspace each: another call beside it)
            other = torch.empty_like(y)
            S.slope_spmm_mxfp4_packed(codes, exps, K, packed, N, other)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager[i])
        torch.zeros(1 << 20, device="cuda").add_(1)

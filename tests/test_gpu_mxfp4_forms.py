"""The 4-bit product on every form of its kernels (tests/mxfp4_forms.py names the form that each size takes), exact.

All operands are E2M1 numbers times a power of two of their block, chosen for each block, so that codes and scales
of every place matter: with whole numbers 0 to 6 times 2^0 to 2^2 on either side all products are whole numbers,
and where the sum of their magnitudes stays below 2^24 every partial sum is a float32 number, in any order of
additions.  float32 outputs are then the exact sums, 16-bit ones their nearest numbers."""
import pytest
import torch

import sparse_gemm_02_amd as S
from gpu_util import say
from mxfp4_forms import FORMS

pytestmark = pytest.mark.gpu
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


def whole_numbers(rows, cols, block, gen, binades):
    """[rows, cols] E2M1 numbers, times 2^0 .. 2^(binades - 1) for each `block` columns, whose first one is 4."""
    grid = torch.tensor([-6.0, -4, -3, -2, -1, 0, 1, 2, 3, 4, 6], device="cuda")
    x = grid[torch.randint(0, 11, (rows, cols), device="cuda", generator=gen)]
    x[:, ::block] = 4.0
    scale = torch.randint(0, binades, (rows, -(-cols // block)), device="cuda", generator=gen)
    return x * torch.exp2(scale.float()).repeat_interleave(block, 1)[:, :cols]


def weight(N, K, gen, binades):
    """(4-bit chunks with guard bytes behind them, dense float32) of a random 2:4 weight."""
    vt = whole_numbers(N, K // 2, 16, gen, binades)
    groups = -(-K // 32) * 8
    at = torch.randint(0, 6, (N, groups), device="cuda", generator=gen)
    at[:, K // 4:] = 0
    nib = torch.tensor([4, 8, 12, 9, 13, 14], device="cuda")[at]
    nib[:, K // 4:] = 0
    meta = (nib.view(N, -1, 8) << (4 * torch.arange(8, device="cuda"))).sum(-1).to(torch.int32)
    nb = S.slope_packed_sparse_mxfp4_bytes(N, K)
    raw = torch.full((nb + GUARD,), 0xA5, dtype=U8, device="cuda")
    S.slope_pack_sparse_mxfp4(vt.bfloat16(), meta, N, K, raw[:nb])
    dense = torch.zeros((N, K // 4, 4), device="cuda")
    for i, shift in ((0, 0), (1, 2)):
        dense.scatter_(2, (nib[:, :K // 4, None] >> shift) & 3, vt.view(N, K // 4, 2)[:, :, i:i + 1])
    assert (raw[nb:] == 0xA5).all()
    return raw[:nb], dense.view(N, K)


def rows_of(x):
    T, K = x.shape
    nc, ne = S.slope_mxfp4_row_bytes(K)
    codes, exps = torch.empty((T, nc), dtype=U8, device="cuda"), torch.empty((T, ne), dtype=U8, device="cuda")
    S.slope_quantize_mxfp4(x, codes, exps)
    back = torch.empty_like(x)
    S.slope_mxfp4_values(codes, exps, back)
    assert torch.equal(back, x)                                      # 4-bit numbers already
    return codes, exps


@pytest.mark.parametrize("T,K,N,form", FORMS + [(3, 655376, 36, "tiles 128x64, without a workspace")])
def test_every_form_is_exact(T, K, N, form):
    say(f"[spmm_mxfp4 form] T={T} K={K} N={N}: {form}")
    gen = torch.Generator(device="cuda").manual_seed(T + K + N)
    binades = 3 if K < 1 << 18 else 2
    packed, dense = weight(N, K, gen, binades)
    x = whole_numbers(T, K, 32, gen, binades)
    codes, exps = rows_of(x)
    want = x @ dense.t().contiguous()
    assert (x.abs() @ dense.abs().t().contiguous()).max().item() < 2 ** 24
    del dense
    need = S.slope_spmm_mxfp4_workspace_bytes(T, K, N)
    if "without" in form:
        sizes = [0]
    else:                                                            # the call's own choice, then every number of parts
        sizes = [None] + ([0, *range(2 * 4 * T * N, need + 1, 4 * T * N)] if need else [])
    for out in (torch.float32, torch.bfloat16, torch.float16):
        for size in sizes if out is torch.float32 else sizes[:1]:
            raw = torch.full((T * N + GUARD,), 7.0, dtype=out, device="cuda")
            ws = None if size is None else torch.full((size + GUARD,), 0xA5, dtype=U8, device="cuda")
            S.slope_spmm_mxfp4_packed(codes, exps, K, packed, N, raw[:T * N].view(T, N),
                                      workspace=None if ws is None else ws[:size])
            torch.cuda.synchronize()
            y = raw[:T * N].view(T, N)
            assert torch.equal(y, want.to(out)), (out, size, (y != want.to(out)).nonzero()[:4].tolist())
            assert (raw[T * N:] == 7.0).all() and (ws is None or (ws[size:] == 0xA5).all())

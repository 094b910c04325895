"""The ends of the 4-bit rows' range: the largest float32 and bfloat16 values round to 2^128, the least code is
2^-128."""
import numpy as np
import pytest
import torch

import oracle
import sparse_gemm_02_amd as S

TOP = 2.0 ** 127
# value of a block's largest, what it is rounded to
CASES = [(1.5 * TOP, 1.5 * TOP), ((1.75 - 2.0 ** -23) * TOP, 1.5 * TOP), (1.75 * TOP, 2.0 * TOP),
         (float(np.finfo(np.float32).max), 2.0 * TOP), (2.0 ** -149, 0.0), (2.0 ** -128, 2.0 ** -128), (2.0 ** -127, 2.0 ** -127)]


def test_the_oracle():
    for x, want in CASES:
        row = np.zeros((1, 32))
        row[0, 5] = -x
        codes, exps = oracle.mxfp4_codes(row)
        assert oracle.mxfp4_values(codes, exps, 32)[0, 5] == -want


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_rows_and_products(dt):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    for x, want in CASES:
        t = torch.zeros((1, 64), dtype=dt, device="cuda")
        t[0, 5] = -x
        if t[0, 5].item() != -float(x):
            continue                                                 # no bfloat16 number
        codes, exps = torch.empty((1, 64), dtype=torch.uint8, device="cuda"), torch.empty((1, 16), dtype=torch.uint8, device="cuda")
        S.slope_quantize_mxfp4(t, codes, exps)
        for out in (torch.float32, torch.bfloat16):
            y = torch.empty((1, 64), dtype=out, device="cuda")
            S.slope_mxfp4_values(codes, exps, y)
            assert y[0, 5].item() == (-want if want <= 1.5 * TOP else float("-inf")) and not y[0, 6:].any()
        if want == 2.0 * TOP:                                        # in a product it counts as 2^128
            w = torch.full((4, 32), 2.0 ** -3, dtype=torch.bfloat16, device="cuda")
            meta = torch.full((4, 2), 0x44444444, dtype=torch.int32, device="cuda")    # positions 0 and 1
            packed = torch.empty(S.slope_packed_sparse_mxfp4_bytes(4, 64), dtype=torch.uint8, device="cuda")
            S.slope_pack_sparse_mxfp4(w, meta, 4, 64, packed)
            y = torch.empty((1, 4), device="cuda")
            S.slope_spmm_mxfp4_packed(codes, exps, 64, packed, 4, y)
            assert (y == -2.0 ** 125).all()

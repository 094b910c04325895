"""Entry points of the microscaled operators whose outputs would be written by one block of threads while
another one reads or writes them: refused on the host, before the GPU is touched."""
import ctypes
import os

import pytest

import sparse_gemm_02_amd as S

FAKE = 1 << 24  # aligned, never dereferenced: every call below is refused
F32, BF16, F16 = 0, 1, 2
INVALID = -1


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(S.library_path):
        from sparse_gemm_02_amd.build import build
        build()
    return S.library()


# bytes of each argument of a 64 x 128 weight's step, values and gradients in 16 bits
N, K = 64, 128
NAMES = ("vals", "meta", "dw", "m", "me", "v", "ve", "ps", "pd")
WRITTEN = ("vals", "m", "me", "v", "ve", "ps", "pd")


def _sizes(gdt):
    n = N * K // 2
    return dict(vals=2 * n, meta=N * K // 8, dw=n * (4 if gdt == F32 else 2), m=n, me=n // 32, v=n, ve=n // 32,
                ps=S.slope_packed_sparse_bytes(N, K), pd=S.slope_packed_sparse_bytes(K, N))


@pytest.mark.parametrize("gdt", [BF16, F16, F32])
def test_fused_8_bit_step_refuses_shared_memory(lib, gdt):
    hp = ctypes.byref(S.AdamWParams(1e-3, 0.9, 0.999, 1e-8, 0.01, 1))
    size = _sizes(gdt)

    def f(**k):
        a = {n: k.get(n, (i + 1) * FAKE) for i, n in enumerate(NAMES)}
        return lib.slope_adamw8_double_prune_packed(BF16, gdt, a["vals"], a["meta"], a["dw"], a["m"], a["me"], a["v"], a["ve"],
                                                    N, K, hp, 0, a["ps"], size["ps"], a["pd"], size["pd"], None)
    at = {n: (i + 1) * FAKE for i, n in enumerate(NAMES)}
    for a in NAMES:
        for b in WRITTEN:
            if a == b:
                continue
            assert f(**{a: at[b]}) == INVALID, (a, b)                # the same address
            step = 1 if a in ("me", "ve") else 16
            assert f(**{a: at[b] + (size[b] - 1) // step * step}) == INVALID, (a, b)   # over its last bytes


@pytest.mark.parametrize("dt", [BF16, F32])
def test_moments_refuse_shared_memory(lib, dt):
    n, e = 4096, 2 if dt == BF16 else 4
    names = ("m", "me", "v", "ve", "mo", "vo")
    at = {k: (i + 1) * FAKE for i, k in enumerate(names)}
    size = dict(m=n, me=n // 32, v=n, ve=n // 32, mo=n * e, vo=n * e)

    def f(n=n, **k):
        return lib.slope_adamw_moments(dt, *[k.get(x, at[x]) for x in names[:4]], n, k.get("mo", at["mo"]), k.get("vo", at["vo"]), None)
    for out in ("mo", "vo"):
        for other in names:
            if other == out:
                continue
            assert f(**{out: at[other]}) == INVALID, (out, other)
            assert f(**{out: at[other] + (size[other] - 1) // e * e}) == INVALID, (out, other)   # over its last bytes
            assert f(**{other: at[out] + size[out] - e}) == INVALID, (out, other)
    # one moment alone: an output over its own codes
    g = lambda mo: lib.slope_adamw_moments(dt, at["m"], at["me"], None, None, n, mo, None, None)
    assert g(at["m"]) == INVALID and g(at["m"] + n - e) == INVALID and g(at["m"] - e * n + e) == INVALID and g(at["me"]) == INVALID
    assert f(n=0, mo=at["m"], vo=at["m"]) == 0                       # no values: nothing to share

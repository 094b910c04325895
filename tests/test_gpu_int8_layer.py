"""The module wrappers of the RMS norm and the int8 linear layer: a norm and a
sparse linear trained together (gradients against float64), the inference path
norm -> codes -> int8 linear with its adapter, and their refusals."""
import numpy as np
import pytest
import torch

import oracle
import sparse_gemm_02_amd as S
from sparse_gemm_02_amd.layer import Int8Rows, Int8SparseLinear, ResidualRMSNorm, SparseAdamW, SparseLinear

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    S.library()
    yield
    torch.cuda.synchronize()


def rand(seed, *shape, dtype=torch.bfloat16, sigma=1.0):
    return (sigma * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()


def f64(t):
    return t.detach().cpu().double()


def norm64(x, g, eps):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * g


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("use", ["y", "h", "both", "none"])
def test_norm_gradients(dtype, use):
    """x, residual and weight against autograd in float64 on the same stored
    values (h is the stored, rounded sum there too).  Terms as in the kernels'
    own tests: 2^-16 of the magnitudes, then half a step of each output."""
    norm = ResidualRMSNorm(200, dtype=torch.float32)
    with torch.no_grad():
        norm.weight.copy_(1 + 0.2 * rand(1, 200, dtype=torch.float32))
    x, res = rand(2, 3, 5, 200, dtype=dtype).requires_grad_(), rand(3, 3, 5, 200, dtype=dtype).requires_grad_()
    cy, ch = rand(4, 3, 5, 200, dtype=dtype), rand(5, 3, 5, 200, dtype=dtype)
    if use == "none":
        y, h = norm(x), None
    else:
        y, h = norm(x, res)
    outs, grads = ([y], [cy]) if use in ("y", "none") else ([h], [ch]) if use == "h" else ([y, h], [cy, ch])
    torch.autograd.backward(outs, grads)
    # the same in float64 from the stored h
    hs = f64(x if h is None else h).requires_grad_()
    g = f64(norm.weight).requires_grad_()
    yr = norm64(hs, g, norm.eps)
    loss = 0.0
    if use != "h":
        loss = loss + (yr * f64(cy)).sum()
    if use in ("h", "both"):
        loss = loss + (hs * f64(ch)).sum()
    loss.backward()
    r = 1 / torch.sqrt((hs * hs).mean(-1, keepdim=True) + norm.eps)
    a, xh = f64(cy) * g, hs * r
    mag = (r * (a.abs() + xh.abs() * (a * xh).abs().mean(-1, keepdim=True)) + f64(ch).abs()).detach()
    bound = HALF[dtype] * hs.grad.abs() + 2.0 ** -16 * mag
    assert ((f64(x.grad) - hs.grad).abs() <= bound).all()
    if use == "none":
        assert res.grad is None
    else:
        same = torch.equal(x.grad, res.grad)
        shared = x.grad.data_ptr() == res.grad.data_ptr()
        assert same and not shared
    if use == "h":
        assert norm.weight.grad is None
    else:
        gm = (f64(cy) * xh).abs().sum((0, 1)).detach()
        assert ((f64(norm.weight.grad) - g.grad).abs() <= HALF[torch.float32] * g.grad.abs() + 2.0 ** -16 * gm).all()
    if use != "h":
        ref = yr.detach()
        assert ((f64(y) - ref).abs() <= (HALF[dtype] + 2.0 ** -16) * ref.abs() + 2.0 ** -25).all()


def test_gradients_accumulate_over_two_passes():
    norm = ResidualRMSNorm(64)
    x, r = rand(1, 3, 5, 64).requires_grad_(), rand(2, 3, 5, 64).requires_grad_()
    once = []
    for _ in range(2):
        y, h = norm(x, r)
        torch.autograd.backward([y, h], [torch.ones_like(y), torch.ones_like(h)])
        once.append((x.grad.clone(), r.grad.clone(), norm.weight.grad.clone()))
    for a, b in zip(*once):
        doubled = torch.equal(b, 2 * a)
        assert doubled


def test_norm_with_the_same_tensor_twice():
    """x as its own residual: both gradients reach the one leaf."""
    norm = ResidualRMSNorm(64)
    x = rand(1, 7, 64, dtype=torch.float32).requires_grad_()
    y, h = norm(x, x)
    y.backward(torch.ones_like(y))
    xs = f64(x).requires_grad_()
    norm64(2 * xs, f64(norm.weight), norm.eps).sum().backward()
    assert torch.allclose(f64(x.grad), xs.grad, rtol=1e-4, atol=1e-6)


def test_norm_frozen_weight_and_strided_input():
    norm = ResidualRMSNorm(48)
    norm.weight.requires_grad_(False)
    big = rand(1, 9, 2, 48, dtype=torch.float32)
    x = big[:, 0].requires_grad_()                       # rows with a gap between them
    y = norm(x)
    y.backward(torch.ones_like(y).t().contiguous().t())  # a gradient with other strides
    xs = f64(big[:, 0]).requires_grad_()
    norm64(xs, 1.0, norm.eps).sum().backward()
    assert norm.weight.grad is None
    assert torch.allclose(f64(x.grad if x.grad is not None else big.grad), xs.grad, rtol=1e-4, atol=1e-6)


def test_norm_and_sparse_linear_train_together():
    """One block h = x + r, y = W norm(h), trained for a few steps by the layer's
    optimizer: gradients exist for every parameter and all stay finite."""
    torch.manual_seed(0)
    norm = ResidualRMSNorm(256, dtype=torch.bfloat16)
    lin = SparseLinear(rand(7, 320, 256, sigma=0.05), rand(8, 256, 16, sigma=0.05), rand(9, 16, 320, sigma=0.05))
    opt = SparseAdamW([norm, lin], lr=1e-3)
    x, r = rand(10, 100, 256), rand(11, 100, 256)
    for _ in range(3):
        opt.zero_grad()
        y, h = norm(x, r)
        (lin(y).float().square().mean() + h.float().square().mean()).backward()
        for p in (norm.weight, lin.values, lin.L, lin.R):
            assert p.grad is not None and torch.isfinite(p.grad).all() and p.grad.abs().max() > 0
        opt.step()
    assert all(torch.isfinite(p).all() for p in (norm.weight, lin.values, lin.L, lin.R))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (2, 130)])
@pytest.mark.parametrize("rank", [0, 24])
def test_inference_path(dtype, shape, rank):
    """norm.codes -> Int8SparseLinear: codes equal the oracle's, the product is its
    float64 value within the two float32 roundings and half a step, the adapter's
    term (another rounding to the format) within the 16-bit adapter's own bound."""
    K, N = 272, 320
    norm = ResidualRMSNorm(K)
    with torch.no_grad():
        norm.weight.copy_(1 + 0.2 * rand(1, K, dtype=torch.float32))
    lin = SparseLinear(rand(2, N, K, dtype=dtype, sigma=0.05), *((rand(3, K, rank, dtype=dtype, sigma=0.05),
                                                               rand(4, rank, N, dtype=dtype, sigma=0.05)) if rank else ()))
    q8 = Int8SparseLinear(lin)
    x, res = rand(5, *shape, K, dtype=dtype), rand(6, *shape, K, dtype=dtype)
    rows, h, y = norm.codes(x, res, output=True)
    out = q8(rows, y) if rank else q8(rows)
    assert rows.q.shape == x.shape and rows.scale.shape == shape and out.shape == (*shape, N) and out.dtype == dtype
    fmt = "bf16" if dtype == torch.bfloat16 else "f16"
    href = oracle.residual_sum(f64(x).numpy().reshape(-1, K), f64(res).numpy().reshape(-1, K), fmt)
    qr, _ = oracle.row_codes_i8(href * f64(norm.weight).numpy())
    assert np.array_equal(f64(h).numpy().reshape(-1, K), href)
    assert np.array_equal(rows.q.cpu().numpy().reshape(-1, K), qr)
    wq = oracle.row_codes_i8(f64(lin.values).numpy())[0]
    meta = lin.meta.cpu().numpy().view(np.uint32)
    dense = oracle.decompress24(wq, meta, K).astype(np.float64) * f64(q8.w_scale).numpy()[:, None]
    ref = (qr.astype(np.float64) * f64(rows.scale).numpy().reshape(-1, 1)) @ dense.T
    got = f64(out).numpy().reshape(-1, N)
    if rank:
        y64 = f64(y).numpy().reshape(-1, K)
        L, R = f64(lin.L).numpy(), f64(lin.R).numpy()
        low = (y64 @ L) @ R
        # the product rounded, the sum rounded, and the adapter's float32 sums of magnitudes
        bound = HALF[dtype] * (np.abs(ref) + np.abs(ref + low)) + 2.0 ** -14 * (np.abs(y64) @ np.abs(L)) @ np.abs(R)
        assert (np.abs(got - ref - low) <= bound + 2.0 ** -20).all()
        # quantizing y itself gives other codes (y is rounded to 16 bits first), the same adapter term
        assert q8(y).shape == out.shape
    else:
        assert (np.abs(got - ref) <= (HALF[dtype] + 2.0 ** -21) * np.abs(ref) + 2.0 ** -25).all()


def test_int8_linear_quantizes_its_own_input():
    lin = SparseLinear(rand(1, 64, 128, sigma=0.05))
    q8 = Int8SparseLinear(lin)
    x = rand(2, 5, 128)
    q, s = torch.empty(5, 128, dtype=torch.int8, device="cuda"), torch.empty(5, device="cuda")
    S.slope_quantize_rows_i8(x, q, s)
    assert torch.equal(q8(x), q8(Int8Rows(q, s)))
    # every 16-bit value is within half a code of its row, every weight of its channel
    err = (f64(q8(x)) - f64(lin(x))).abs()
    xa, wa = f64(x).abs().amax(1, keepdim=True) / 254, f64(q8.w_scale)[None, :] / 2
    wsum = torch.from_numpy(np.abs(oracle.decompress24(f64(lin.values).numpy(), lin.meta.cpu().numpy().view(np.uint32), 128)).sum(1))
    bound = xa * wsum[None, :] + (f64(x).abs().sum(1, keepdim=True) + 128 * xa) * wa
    assert (err <= bound + 2.0 ** -7 * (f64(lin(x)).abs() + bound)).all()


def test_refusals():
    norm = ResidualRMSNorm(64)
    x = rand(1, 4, 64)
    with pytest.raises(ValueError, match="columns"):
        norm(rand(1, 4, 65))
    with pytest.raises(ValueError, match="residual"):
        norm(x, rand(1, 5, 64))
    with pytest.raises(ValueError, match="residual"):
        norm(x, x.float())
    with pytest.raises(S.SlopeError):
        norm.codes(x.float())
    lin = SparseLinear(rand(1, 32, 64), rand(2, 64, 8), rand(3, 8, 32))
    q8 = Int8SparseLinear(lin)
    rows, _ = norm.codes(x)
    with pytest.raises(ValueError, match="adapter"):
        q8(rows)
    with pytest.raises(ValueError, match="format"):
        q8(x.float())
    with pytest.raises(ValueError, match="codes"):
        q8(Int8Rows(rows.q, rows.scale[:2]), x)
    with pytest.raises(ValueError, match="codes"):
        q8(rows, rand(1, 3, 64))


def test_batches_without_rows():
    """Every call on [0, K]: outputs without rows, gradients of zeros."""
    norm = ResidualRMSNorm(256, dtype=torch.bfloat16)
    x = rand(1, 0, 3, 256).requires_grad_()
    r = rand(2, 0, 3, 256).requires_grad_()
    for args in ((x,), (x, r)):
        out = norm(*args)
        y, h = out if len(args) == 2 else (out, x)
        (y.sum() + h.sum()).backward()
    torch.cuda.synchronize()
    assert y.shape == h.shape == (0, 3, 256) and x.grad.shape == r.grad.shape == x.shape
    assert norm.weight.grad is not None and not norm.weight.grad.any()
    rows, h, y = norm.codes(x, r, output=True)
    assert rows.q.shape == x.shape and rows.scale.shape == (0, 3) and h.shape == y.shape == x.shape
    lin = Int8SparseLinear(SparseLinear(rand(3, 128, 256, sigma=0.02)))
    assert lin(rows).shape == (0, 3, 128) and lin(x.detach()).shape == (0, 3, 128)


def test_captured_forward_and_backward():
    """norm's y, h and all three gradients in a captured graph, replayed on changed
    inputs: equal to the eager calls, bit for bit."""
    norm = ResidualRMSNorm(1024, dtype=torch.bfloat16)
    static = [rand(i, 96, 1024).requires_grad_(i < 2) for i in range(4)]      # x, residual, dy, dh

    def step():
        y, h = norm(static[0], static[1])
        return y.detach(), h.detach(), *torch.autograd.grad((y, h), (static[0], static[1], norm.weight), static[2:])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        with torch.no_grad():
            for j, t in enumerate(static):
                t.copy_(rand(10 * i + j, 96, 1024))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b), i
        torch.cuda.synchronize()


def at_offset(t, n):
    """The same values, contiguous, n elements behind an aligned address."""
    v = torch.empty(t.numel() + n, dtype=t.dtype, device=t.device)[n:].view(t.shape)
    v.copy_(t)
    assert v.is_contiguous() and v.data_ptr() % 16
    return v


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("K", [768, 771])
def test_norm_of_tensors_at_any_address(K, dtype):
    """Contiguous inputs, weight and gradients that start at any element: the same
    bits as from aligned ones."""
    w, x, r, dy, dh = (rand(i, *s, dtype=dtype) for i, s in enumerate([(K,)] + [(5, K)] * 4))

    def outputs(place):
        norm = ResidualRMSNorm(K, dtype=dtype)
        norm.weight = torch.nn.Parameter(place(w))
        a, b = place(x).requires_grad_(), place(r).requires_grad_()
        y, h = norm(a, b)
        out = [y, h, *torch.autograd.grad([y, h], [a, b, norm.weight], [place(dy), place(dh)])]
        y = norm(a)
        out += [y, *torch.autograd.grad([y], [a, norm.weight], [place(dy)])]
        if dtype != torch.float32:
            rows, h, y = norm.codes(place(x), place(r), output=True)
            out += [*rows, h, y]
            rows, h = norm.codes(place(x))
            out += [*rows, h]
        return out
    for got, want in zip(outputs(lambda t: at_offset(t, 1)), outputs(lambda t: t)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norms_of_odd_width_under_a_concatenation(dtype):
    """cat's gradient reaches the second norm as rows of a larger tensor that start
    at any element, x[1:] its input likewise."""
    norm = ResidualRMSNorm(771, dtype=dtype)
    x, r, g = rand(1, 4, 771, dtype=dtype), rand(2, 3, 771, dtype=dtype), rand(3, 12, 771, dtype=dtype)
    a = x[1:].detach().requires_grad_()
    assert a.data_ptr() % 16
    b = r.clone().requires_grad_()
    y, h = norm(a, b)
    torch.cat([norm(a), y, norm(b), h]).backward(g)
    got = a.grad, b.grad, norm.weight.grad
    want = [torch.zeros(t.shape, dtype=torch.float64) for t in got]
    hs = f64(h).requires_grad_()                         # h as stored; its gradient is a's and b's
    a64, b64, w = f64(a).requires_grad_(), f64(b).requires_grad_(), f64(norm.weight).requires_grad_()
    cat = torch.cat([norm64(a64, w, norm.eps), norm64(hs, w, norm.eps), norm64(b64, w, norm.eps), hs])
    cat.backward(f64(g))
    want = a64.grad + hs.grad, b64.grad + hs.grad, w.grad
    # every gradient is a sum of two (weight: three) rounded terms: half a step of each
    # term and each partial sum, none above the magnitudes added here, and 2^-16 for
    # the kernels' sums (the terms of test_norm_gradients)
    def terms(v, d):
        rs = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + norm.eps)
        p, xh = f64(d) * f64(norm.weight), v * rs
        return (rs * (p.abs() + xh.abs() * (p * xh).abs().mean(-1, keepdim=True))).detach(), (f64(d) * xh).abs().sum(0).detach()
    (ma, wa), (mh, wh), (mb, wb) = (terms(v, d) for v, d in ((f64(a), g[:3]), (f64(h), g[3:6]), (f64(b), g[6:9])))
    mh = mh + f64(g[9:]).abs()
    for t, ref, mag, n in zip(got, want, (ma + mh, mb + mh, wa + wh + wb), (2, 2, 3)):
        assert ((f64(t) - ref).abs() <= (n * HALF[dtype] + 2.0 ** -16) * mag).all()


@pytest.mark.parametrize("rank", [0, 8])
def test_int8_linear_of_tensors_at_any_address(rank):
    lin = SparseLinear(rand(1, 64, 128, sigma=0.05), *((rand(2, 128, rank), rand(3, rank, 64)) if rank else ()))
    q8, x = Int8SparseLinear(lin), rand(4, 5, 128)
    q, s = torch.empty(5, 128, dtype=torch.int8, device="cuda"), torch.empty(5, device="cuda")
    S.slope_quantize_rows_i8(x, q, s)
    want = q8(x)
    assert torch.equal(q8(at_offset(x, 1)), want)
    assert torch.equal(q8(Int8Rows(at_offset(q, 3), at_offset(s, 1)), at_offset(x, 5)), want)


@pytest.mark.parametrize("rank", [0, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_int8_linear_under_conversions_of_its_model(dtype, rank):
    """A conversion of the model's floating-point tensors leaves the layer's scales
    in float32 and its adapter in the layer's format; moves between devices take
    everything along."""
    lin = SparseLinear(rand(1, 64, 128, dtype=dtype, sigma=0.05),
                       *((rand(2, 128, rank, dtype=dtype), rand(3, rank, 64, dtype=dtype)) if rank else ()))
    q8, x = Int8SparseLinear(lin), rand(4, 5, 128, dtype=dtype)
    want, scale = q8(x), q8.w_scale.clone()
    model = torch.nn.Sequential(q8)
    for convert in (lambda m: m.to(torch.bfloat16), lambda m: m.half(), lambda m: m.float(), lambda m: m.double(),
                    lambda m: m.to("cuda", torch.bfloat16), lambda m: m.cpu().cuda(),
                    lambda m: m.to("cpu", torch.float16).to("cuda", torch.float64)):
        convert(model)
        assert q8.w_scale.dtype == torch.float32 and torch.equal(q8.w_scale, scale)
        assert torch.equal(model(x), want)
    with pytest.raises(ValueError, match="format"):
        model(x.float())
    model.cpu()
    assert not any(b.is_cuda for b in model.buffers())


def test_int8_linear_refuses_a_second_input_it_would_not_read():
    q8, x = Int8SparseLinear(SparseLinear(rand(1, 64, 128, sigma=0.05))), rand(2, 5, 128)
    with pytest.raises(ValueError, match="one input"):
        q8(x, rand(3, 5, 128))
    assert torch.equal(q8(x, x), q8(x))

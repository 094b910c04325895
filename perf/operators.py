"""Cases and plain forms of the row-scaled 8-bit operators: the RMS norm with
the residual's addition and 8-bit codes, its gradient, and the 2:4 sparse
product on 8-bit integer codes with a scale for each token and channel.

The widths are those of the layers in `workloads` (GPT-2-small, BERT-Large,
OPT-13B, OPT-66B), with odd widths and ragged token counts beside them.
`run(state)` computes one operator in plain torch operations where `own` is
false, and through the package's entry points where it is true.
"""
import math

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one token of a generating OPT-66B layer: the norm before QKV, latency only
        dict(name="norm_i8_1x9216", op="norm_i8", T=1, K=9216, dt="bf16", gamma="bf16", residual=True),
        # a ragged prompt of OPT-13B width, fp16 activations with fp32 norm weights, first layer (no residual yet)
        dict(name="norm_i8_1021x5120_f16", op="norm_i8", T=1021, K=5120, dt="f16", gamma="f32", residual=False),
        # a full prompt batch of OPT-66B width
        dict(name="norm_i8_8192x9216", op="norm_i8", T=8192, K=9216, dt="bf16", gamma="bf16", residual=True),
        # BERT-Large training step: 32 sequences of 512 tokens, 16-bit output, statistics kept for the gradient
        dict(name="norm_16384x1024", op="norm", T=16384, K=1024, dt="bf16", gamma="f32", residual=True),
        # odd width in fp32 (rows not 16-byte aligned)
        dict(name="norm_2047x771_f32", op="norm", T=2047, K=771, dt="f32", gamma="f32", residual=True),
        # gradient of the norm in an OPT-66B training step, with the residual stream's own gradient
        dict(name="norm_bwd_8192x9216", op="norm_bwd", T=8192, K=9216, dt="bf16", gamma="bf16", residual=True),
        # GPT-2-small training step, fp16: narrow rows, many tokens, no second gradient
        dict(name="norm_bwd_8192x768_f16", op="norm_bwd", T=8192, K=768, dt="f16", gamma="f32", residual=False),
        # one generated token through OPT-66B's QKV: the weight's stream is all there is
        dict(name="linear_i8_1x9216x27648", op="linear_i8", T=1, K=9216, N=27648, dt="bf16"),
        # 61 sequences in flight through OPT-13B's FC2
        dict(name="linear_i8_61x20480x5120_f16", op="linear_i8", T=61, K=20480, N=5120, dt="f16"),
        # a short prompt through GPT-2-small's QKV, fp32 output: few tiles
        dict(name="linear_i8_1000x768x2304_f32", op="linear_i8", T=1000, K=768, N=2304, dt="f32"),
        # a full prompt batch through OPT-66B's attention output: matrix rate
        dict(name="linear_i8_8192x9216x9216", op="linear_i8", T=8192, K=9216, N=9216, dt="bf16"),
        # 16 sequences of OPT-13B: residual, norm, codes and the QKV product, as a serving step runs them
        dict(name="norm_linear_i8_16x5120x15360", op="norm_linear_i8", T=16, K=5120, N=15360, dt="bf16", gamma="bf16",
             residual=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Another case of the same ranges: one token to 16384, widths to 20480
    (any width for the norms, multiples of 16 for the product's reduction and
    of 4 for its outputs), within the largest listed case's cost."""
    op = rng.choice(["norm_i8", "norm", "norm_bwd", "linear_i8", "linear_i8", "norm_linear_i8"])
    dt = rng.choice(["bf16", "bf16", "f16"])
    if op in ("norm", "norm_bwd"):
        dt = rng.choice(["bf16", "f16", "f32"])
    if op.endswith("linear_i8"):
        few = rng.random() < 0.5
        T = rng.randint(1, 64) if few else _log_int(rng, 65, 8192)
        K = 16 * _log_int(rng, 16, 1280)
        most = min(27648, 8192 * 9216 * 9216 // (T * K), 9216 * 27648 // K)
        N = 4 * _log_int(rng, 16, max(17, most // 4))
        case = dict(op=op, T=T, K=K, N=N, dt=dt)
    else:
        K = _log_int(rng, 16, 16384)
        if rng.random() < 0.5:
            K = (K + 15) // 16 * 16
        T = _log_int(rng, 1, min(16384, 8192 * 9216 * 3 // (2 * SIZE[dt] * K)))
        case = dict(op=op, T=T, K=K, dt=dt)
    if op != "linear_i8":
        case.update(gamma=rng.choice([dt, "f32"]), residual=rng.random() < 0.7)
    return case


def work(case):
    T, K, dt = case["T"], case["K"], case["dt"]
    e, g = SIZE[dt], SIZE.get(case.get("gamma"), 0)
    res = 1 if case.get("residual") else 0
    nbytes = flops = 0
    if case["op"] in ("norm_i8", "norm_linear_i8"):
        # x (and the residual), the sum written where there is one, codes and scales, gamma
        nbytes += T * K * (e + 2 * res * e) + K * g
        nbytes += T * K + 4 * T if case["op"] == "norm_i8" else 0
        flops += 8 * T * K
    if case["op"] == "norm":
        nbytes += T * K * (e + 2 * res * e + e) + 4 * T + K * g
        flops += 6 * T * K
    if case["op"] == "norm_bwd":
        nbytes += T * K * e * (3 + res) + 4 * T + 2 * K * g
        flops += 10 * T * K
    if case["op"].endswith("linear_i8"):
        N = case["N"]
        # codes and scales of both sides, one 2-bit position per kept weight, the output once
        nbytes += N * K // 2 + N * K // 8 + 4 * N + T * N * e
        nbytes += T * K + 4 * T if case["op"] == "linear_i8" else 0
        flops += T * N * K
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, sigma, dtype):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, sigma, generator=g).to(dtype)


def _activations(g, T, K, dtype):
    """Hidden states: unit normals with a few wide channels, as trained layers have."""
    x = torch.empty((T, K), dtype=torch.float32, device="cuda").normal_(0.0, 1.0, generator=g)
    wide = torch.randint(0, K, (max(1, K // 256),), device="cuda", generator=g)
    x[:, wide] *= 6.0
    return x.to(dtype)


def _weight(g, N, K, dtype):
    """A 2:4 weight as a checkpoint holds it, [N, K] with two zeros in every
    four: the two smallest magnitudes of each group are cleared."""
    w = _normal(g, (N, K // 4, 4), 0.02, dtype)
    drop = w.abs().argsort(dim=2, stable=True)[:, :, :2]
    return w.scatter_(2, drop, 0.0).reshape(N, K)


def _channel_codes(w):
    """8-bit codes and scales of a weight's rows."""
    a = w.float().abs().amax(dim=1)
    q = (w.double() * 127 / a.double().clamp_min(1e-300)[:, None]).round().to(torch.int8)
    return q, a / 127


def prepare(case, seed):
    g = _generator(seed)
    T, K, dtype = case["T"], case["K"], DTYPES[case["dt"]]
    s = {"case": case}
    if case["op"] != "linear_i8":
        s["gamma"] = (1.0 + _normal(g, (K,), 0.1, torch.float32)).to(DTYPES[case["gamma"]])
        s["x"] = _activations(g, T, K, dtype)
        if case["op"] == "norm_bwd":
            # the forward's saved sum and statistics, and the arriving gradients
            s["rstd"] = (s["x"].double().square().mean(dim=1) + EPS).rsqrt().float()
            s["dy"] = _normal(g, (T, K), 1.0, dtype)
            s["dh"] = _normal(g, (T, K), 1.0, dtype) if case["residual"] else None
        else:
            s["res"] = _normal(g, (T, K), 1.0, dtype) if case["residual"] else None
    if case["op"].endswith("linear_i8"):
        N = case["N"]
        w = _weight(g, N, K, dtype if dtype != torch.float32 else torch.bfloat16)
        if own:
            s["w"], s["w_scale"] = _packed(w)
        else:
            s["w"], s["w_scale"] = _channel_codes(w)
        if case["op"] == "linear_i8":
            x = _activations(g, T, K, torch.float32)
            a = x.abs().amax(dim=1)
            s["xq"] = (x * (127 / a)[:, None]).round().to(torch.int8)
            s["x_scale"] = a / 127
    return s


def _packed(w):
    """The weight laid out once, as a serving program keeps it."""
    import sparse_gemm_02_amd as S
    N, K = w.shape
    values = torch.empty((N, K // 2), dtype=w.dtype, device="cuda")
    meta = torch.empty((N, (K // 4 + 7) // 8), dtype=torch.int32, device="cuda")
    S.slope_prune_compress24(w, values, meta)
    packed = torch.empty(S.slope_packed_sparse_i8_bytes(N, K), dtype=torch.uint8, device="cuda")
    scale = torch.empty(N, dtype=torch.float32, device="cuda")
    S.slope_pack_sparse_i8(values, meta, N, K, scale, packed)
    return packed, scale


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    if case["op"] == "norm_i8":
        h, q, scale = (_own_norm_i8 if own else _plain_norm_i8)(s)
        # the codes as the values they stand for
        values = torch.mul(q, scale[:, None])
        return {"h": h, "values": values} if s["res"] is not None else {"values": values}
    if case["op"] == "norm":
        return (_own_norm if own else _plain_norm)(s)
    if case["op"] == "norm_bwd":
        return (_own_norm_bwd if own else _plain_norm_bwd)(s)
    if case["op"] == "linear_i8":
        return {"y": (_own_linear if own else _plain_linear)(s, s["xq"], s["x_scale"])}
    h, q, scale = (_own_norm_i8 if own else _plain_norm_i8)(s)
    y = (_own_linear if own else _plain_linear)(s, q, scale)
    return {"h": h, "y": y} if s["res"] is not None else {"y": y}


def _plain_sum(s):
    return s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(s["x"].dtype)


def _plain_norm_i8(s):
    h = _plain_sum(s)
    f = h.float()
    rstd = torch.rsqrt(f.square().mean(dim=1) + EPS)
    # in 64 bits: values next to a border between two codes (the code of a
    # value is its own share of the row's largest; rstd is common to both)
    u = h.double() * s["gamma"].double()
    amax = u.abs().amax(dim=1)
    q = (u * 127 / amax[:, None]).round().to(torch.int8)
    return h, q, amax.float() / 127 * rstd


def _plain_norm(s):
    h = _plain_sum(s)
    f = h.float()
    rstd = torch.rsqrt(f.square().mean(dim=1) + EPS)
    y = (f * rstd[:, None] * s["gamma"].float()).to(h.dtype)
    return {"h": h, "y": y, "rstd": rstd} if s["res"] is not None else {"y": y, "rstd": rstd}


def _plain_norm_bwd(s):
    dy, xh = s["dy"].float(), s["x"].float() * s["rstd"][:, None]
    a = dy * s["gamma"].float()
    dx = (a - xh * (a * xh).mean(dim=1, keepdim=True)) * s["rstd"][:, None]
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    # in 64 bits: a long sum over tokens
    dgamma = (dy * xh).sum(dim=0, dtype=torch.float64)
    return {"dx": dx.to(s["x"].dtype), "dgamma": dgamma.to(s["gamma"].dtype)}


def _plain_linear(s, q, scale):
    acc = q.float() @ s["w"].float().t()
    return (acc * (scale[:, None] * s["w_scale"])).to(DTYPES[s["case"]["dt"]])


def _own_norm_i8(s):
    import sparse_gemm_02_amd as S
    x = s["x"]
    h = torch.empty_like(x) if s["res"] is not None else None
    q = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    scale = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
    S.slope_rmsnorm(x, s["gamma"], EPS, residual=s["res"], H=h, q=q, q_scale=scale)
    return h, q, scale


def _own_norm(s):
    import sparse_gemm_02_amd as S
    x = s["x"]
    h = torch.empty_like(x) if s["res"] is not None else None
    y = torch.empty_like(x)
    rstd = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
    S.slope_rmsnorm(x, s["gamma"], EPS, residual=s["res"], H=h, Y=y, rstd=rstd)
    return {"h": h, "y": y, "rstd": rstd} if h is not None else {"y": y, "rstd": rstd}


def _own_norm_bwd(s):
    import sparse_gemm_02_amd as S
    x, gamma = s["x"], s["gamma"]
    dx, dgamma = torch.empty_like(x), torch.empty_like(gamma)
    ws = torch.empty(S.slope_rmsnorm_bwd_workspace_bytes(*x.shape), dtype=torch.uint8, device=x.device)
    S.slope_rmsnorm_bwd(s["dy"], x, s["rstd"], gamma, dx, dgamma, ws, dH=s["dh"])
    return {"dx": dx, "dgamma": dgamma}


def _own_linear(s, q, scale):
    import sparse_gemm_02_amd as S
    T, N = q.shape[0], s["case"]["N"]
    y = torch.empty((T, N), dtype=DTYPES[s["case"]["dt"]], device=q.device)
    if T <= S.I8_DECODE_MAX_TOKENS:
        S.slope_spmm_i8_decode(q, scale, s["w"], s["w_scale"], N, y)
    else:
        S.slope_spmm_i8_packed(q, scale, s["w"], s["w_scale"], N, y)
    return y


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    out = {}
    if case["op"] in ("norm_i8", "norm", "norm_linear_i8"):
        h = s["x"].double()
        if s["res"] is not None:
            h = (h + s["res"].double()).to(s["x"].dtype)
            out["h"] = h
            h = h.double()
        r = 1.0 / torch.sqrt((h * h).sum(dim=1, keepdim=True) / case["K"] + EPS)
        y = h * s["gamma"].double()
        if case["op"] == "norm":
            out["y"], out["rstd"] = y * r, r[:, 0]
            return out
        # nearest code, ties to even: 127 y / top has no rounding before the
        # division where y is a product of two stored numbers
        top = y.abs().max(dim=1, keepdim=True).values
        codes = torch.round(127 * y / top)
        step = r * top / 127
        if case["op"] == "norm_i8":
            out["values"] = codes * step
            return out
    if case["op"] == "norm_bwd":
        # derivative of y_j = g_j h_j / r, r = sqrt(mean h^2 + eps), given 1 / r
        h, inv, gd = s["x"].double(), s["rstd"].double()[:, None], s["gamma"].double() * s["dy"].double()
        dx = gd * inv - h * inv ** 3 * (gd * h).sum(dim=1, keepdim=True) / case["K"]
        if s["dh"] is not None:
            dx = dx + s["dh"].double()
        return {"dx": dx, "dgamma": (s["dy"].double() * h * inv).sum(dim=0)}
    if case["op"] == "linear_i8":
        codes, step = s["xq"].double(), s["x_scale"].double()[:, None]
    out["y"] = torch.mm(codes, s["w"].double().t().contiguous()) * step * s["w_scale"].double()[None, :]
    return out

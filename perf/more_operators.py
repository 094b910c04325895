"""Cases and plain forms of the microscaled operators: an AdamW step over many
tensors at once with moments in 8 bits (blocks of 32 with a power-of-two scale,
stochastic rounding) or in 32; quantisation to 4-bit floating point (E2M1 codes,
one power-of-two scale for 32 values); and the product of 4-bit activations with
a 2:4 sparse 4-bit weight.

The widths are those of the layers in `workloads` (GPT-2-small, OPT-13B,
OPT-66B), with odd sizes and ragged token counts beside them.  `run(state)`
computes one operator in plain torch operations where `own` is false, and
through the package's entry points where it is true.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
STEP = 100
BLOCK = 32                                             # values with one scale


def listed():
    return [
        # the adapter of GPT-2-small's attention output and two norm weights, 32-bit moments: a call's latency
        dict(name="adamw32_small", op="adamw", bits=32, dt="bf16", gdt="bf16", sizes="12288,12288,768,768"),
        # fp32 tensors of odd sizes with fp16 gradients: biases, a head, an embedding of a small model
        dict(name="adamw32_odd_f32", op="adamw", bits=32, dt="f32", gdt="f16", sizes="1,31,33,771,5001,1000003,6000011"),
        # the same kind of list with 8-bit moments, fp16 weights and fp32 gradients
        dict(name="adamw8_odd_f16", op="adamw", bits=8, dt="f16", gdt="f32", sizes="1,31,33,771,5001,1000003,6000011"),
        # an OPT-13B layer in training: the kept halves of its four 2:4 linears and its eight adapter factors (rank 40)
        dict(name="adamw8_opt13b_layer", op="adamw", bits=8, dt="bf16", gdt="bf16",
             sizes="39321600,13107200,52428800,52428800,204800,614400,204800,204800,204800,819200,819200,204800"),
        # one token of a generating OPT-66B layer: latency only
        dict(name="quant_1x9216", op="quant", T=1, K=9216, dt="bf16"),
        # a ragged prompt, fp16 rows of an odd width (the last block is short)
        dict(name="quant_1021x4999_f16", op="quant", T=1021, K=4999, dt="f16"),
        # a full prompt batch of OPT-66B width
        dict(name="quant_8192x9216", op="quant", T=8192, K=9216, dt="bf16"),
        # one generated token through OPT-66B's QKV: the weight's stream is all there is
        dict(name="linear_1x9216x27648", op="linear", T=1, K=9216, N=27648, dt="bf16"),
        # 61 sequences in flight through OPT-13B's FC2, the longest reduction
        dict(name="linear_61x20480x5120_f16", op="linear", T=61, K=20480, N=5120, dt="f16"),
        # a short prompt through GPT-2-small's QKV, fp32 output: few tiles
        dict(name="linear_1000x768x2304_f32", op="linear", T=1000, K=768, N=2304, dt="f32"),
        # a full prompt batch through OPT-66B's attention output: matrix rate
        dict(name="linear_8192x9216x9216", op="linear", T=8192, K=9216, N=9216, dt="bf16"),
        # 16 sequences of OPT-13B: 16-bit activations quantised and multiplied, as a serving step runs them
        dict(name="quant_linear_16x5120x15360", op="quant_linear", T=16, K=5120, N=15360, dt="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Another case of the same ranges: 1 to 12 tensors of one value to tens of
    millions; one token to 8192, widths to 20480 (any for the quantiser,
    multiples of 16 for the product's reduction and of 4 for its outputs),
    within the largest listed case's cost."""
    op = rng.choice(["adamw", "adamw", "quant", "linear", "linear", "quant_linear"])
    dt = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "adamw":
        bits = rng.choice([8, 8, 32])
        count = rng.randint(1, 12)
        most = 40_000_000 // count
        sizes = [_log_int(rng, 1, most) for _ in range(count)]
        return dict(op=op, bits=bits, dt=dt, gdt=rng.choice([dt, "f32"]), sizes=",".join(str(n) for n in sizes))
    if op == "quant":
        K = _log_int(rng, 16, 20480)
        T = _log_int(rng, 1, min(16384, 8192 * 9216 * 2 // (SIZE[dt] * K)))
        return dict(op=op, T=T, K=K, dt=dt)
    few = rng.random() < 0.5
    T = rng.randint(1, 64) if few else _log_int(rng, 65, 8192)
    K = 16 * _log_int(rng, 16, 1280)
    most = min(27648, 8192 * 9216 * 9216 // (T * K), 9216 * 27648 // K)
    return dict(op=op, T=T, K=K, N=4 * _log_int(rng, 16, max(17, most // 4)), dt=dt)


def _sizes(case):
    return [int(n) for n in case["sizes"].split(",")]


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    if case["op"] == "adamw":
        n, e = sum(_sizes(case)), SIZE[case["dt"]]
        # weight and both moments read and written, the gradient read
        nbytes = n * (2 * e + SIZE[case["gdt"]])
        if case["bits"] == 32:
            return {"bytes": nbytes + 16 * n, "flops": 14 * n}
        scales = sum(_blocks(k) for k in _sizes(case))
        # codes and scales both ways, and the moments' values as bfloat16
        return {"bytes": nbytes + 4 * n + 4 * scales + 4 * n, "flops": 20 * n}
    T, K, e = case["T"], case["K"], SIZE[case["dt"]]
    codes = T * (-(-K // 2) + _blocks(K))
    if case["op"] == "quant":
        # the values in, codes and scales out, and what they stand for as bfloat16
        return {"bytes": T * K * e + codes + 2 * T * K, "flops": 4 * T * K}
    N = case["N"]
    # two codes and two positions a group of four weights, a scale for 32 of them; the output once
    weight = N * (K // 4 + K // 8 + _blocks(K))
    x = T * K * e if case["op"] == "quant_linear" else codes
    return {"bytes": weight + x + T * N * e, "flops": T * N * K}


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


def _places(sizes):
    """First element of each tensor in flat buffers where every one starts a new block."""
    at, places = 0, []
    for n in sizes:
        places.append(at)
        at += _blocks(n) * BLOCK
    return places, at


def _tensor_seeds(seed, count):
    """32 bits for each tensor of a call (SplitMix64 of Steele, Lea and Flood, 2014)."""
    out = []
    for i in range(count):
        z = (seed + (i + 1) * 0x9E3779B97F4A7C15) % 2 ** 64
        z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9 % 2 ** 64
        z = (z ^ (z >> 27)) * 0x94D049BB133111EB % 2 ** 64
        out.append((z ^ (z >> 31)) % 2 ** 32)
    return out


def _prepare_adamw(case, seed):
    g = _generator(seed)
    sizes = _sizes(case)
    places, total = _places(sizes)
    # weights, gradients whose size differs from channel to channel, and moments in mid-training
    live = torch.zeros(total, dtype=torch.bool, device="cuda")
    for o, n in zip(places, sizes):
        live[o:o + n] = True
    wide = torch.empty(total, dtype=torch.float32, device="cuda").log_normal_(-7.0, 1.5, generator=g)
    flat = {"p": (_normal(g, (total,), 0.02, torch.float32) * live).to(DTYPES[case["dt"]]),
            "g": (_normal(g, (total,), 1.0, torch.float32) * wide * live).to(DTYPES[case["gdt"]])}
    m = _normal(g, (total,), 0.3, torch.float32) * wide * live
    v = (wide * live).square_()
    del wide, live
    s = {"case": case, "flat": flat, "seed": 1000 + seed}
    if case["bits"] == 32:
        flat.update(m=m, v=v)
    else:
        me, ve = _exponent(m.view(-1, BLOCK), 7), _exponent(v.view(-1, BLOCK), 15)
        half = torch.full((), 1 << 19, dtype=torch.int64, device="cuda")
        flat.update(m=_encode(m, me, 120, half), v=_encode(v, ve, 112, half),
                    m_exp=(me + 127).to(torch.uint8), v_exp=(ve + 127).to(torch.uint8))
    if own:
        cut = lambda t: [t[o:o + n] for o, n in zip(places, sizes)]
        s["lists"] = {k: cut(flat[k]) for k in ("p", "g", "m", "v")}
        if case["bits"] == 8:
            s["lists"].update({k: [flat[k][o // BLOCK:o // BLOCK + _blocks(n)] for o, n in zip(places, sizes)]
                               for k in ("m_exp", "v_exp")})
    elif case["bits"] == 8:
        # the seed and the number of each run of eight values within its tensor
        runs = [_blocks(n) * BLOCK // 8 for n in sizes]
        s["run_seed"] = torch.cat([torch.full((r,), t, dtype=torch.int64, device="cuda")
                                   for r, t in zip(runs, _tensor_seeds(s["seed"], len(runs)))])
        s["run_number"] = torch.cat([torch.arange(r, dtype=torch.int64, device="cuda") for r in runs])
    return s


def prepare(case, seed):
    if case["op"] == "adamw":
        return _prepare_adamw(case, seed)
    g = _generator(seed)
    T, K, dtype = case["T"], case["K"], DTYPES[case["dt"]]
    s = {"case": case, "x": _activations(g, T, K, dtype)}
    if case["op"] == "quant":
        return s
    w = _weight(g, case["N"], K, dtype if dtype != torch.float32 else torch.bfloat16)
    s["w"] = _packed(w) if own else _codes(w)
    if case["op"] == "linear":
        x = s.pop("x")
        s["xq"] = _own_codes(x) if own else _codes(x)
    return s


def _packed(w):
    """The weight laid out once, as a serving program keeps it."""
    import sparse_gemm_02_amd as S
    N, K = w.shape
    values = torch.empty((N, K // 2), dtype=w.dtype, device="cuda")
    meta = torch.empty((N, (K // 4 + 7) // 8), dtype=torch.int32, device="cuda")
    S.slope_prune_compress24(w, values, meta)
    packed = torch.empty(S.slope_packed_sparse_mxfp4_bytes(N, K), dtype=torch.uint8, device="cuda")
    S.slope_pack_sparse_mxfp4(values, meta, N, K, packed)
    return packed


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    if case["op"] == "adamw":
        return (_own_adamw if own else _plain_adamw)(s)
    if case["op"] == "quant":
        return {"values": (_own_quant if own else _plain_quant)(s["x"])}
    if case["op"] == "linear":
        return {"y": (_own_linear if own else _plain_linear)(s, s["xq"])}
    return {"y": (_own_linear if own else _plain_linear)(s, (_own_codes if own else _codes)(s["x"]))}


def _power(e):
    """2^e as float32, for e in -126 .. 127."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _exponent(blocks, top):
    """Scale exponents of rows of a block: the largest magnitude lands in [2^top, 2^(top+1))."""
    return ((blocks.abs().amax(dim=1).view(torch.int32) >> 23) - 127 - top).clamp_min_(-127).to(torch.int64)


def _encode(x, e, down, noise):
    """Codes of x / 2^e with three bits after the leading one: `noise` (20 bits)
    is added below the last bit kept.  down: what brings the format's smallest
    normal number to float32's."""
    y = (x.abs().view(-1, BLOCK) * _power(-e)[:, None]).view(-1) * 2.0 ** -down
    code = (y.view(torch.int32) + noise) >> 20
    if down == 112:
        return torch.maximum(code, (x > 0).to(code.dtype)).to(torch.uint8)     # no positive number becomes zero
    return (code | (torch.signbit(x).to(code.dtype) << 7)).to(torch.uint8)


def _decode(code, e, up):
    mag = (code & 0x7F) if up == 120 else code
    x = (mag.to(torch.int32) << 20).view(torch.float32) * 2.0 ** up
    if up == 120:
        x = torch.where(code >= 128, -x, x)
    return (x.view(-1, BLOCK) * torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)[:, None]).view(-1)


def _noise(number, seed):
    """A 32-bit word for each value: a hashed start for each run of eight, then
    Marsaglia's xorshift (13, 17, 5)."""
    low = 0xFFFFFFFF
    s = ((number * 0x9E3779B1) & low) ^ seed
    s = ((s ^ (s >> 16)) * 0xBB67AE85) & low
    s = s ^ (s >> 15)
    words = []
    for _ in range(8):
        s = s ^ ((s << 13) & low)
        s = s ^ (s >> 17)
        s = s ^ ((s << 5) & low)
        words.append(s)
    return torch.stack(words, dim=1).view(-1)


def _moments(flat):
    me, ve = flat["m_exp"].to(torch.int64) - 127, flat["v_exp"].to(torch.int64) - 127
    return _decode(flat["m"], me, 120), _decode(flat["v"], ve, 112)


def _plain_adamw(s):
    flat, h = s["flat"], HYPER
    eight = s["case"]["bits"] == 8
    m, v = _moments(flat) if eight else (flat["m"], flat["v"])
    g, p = flat["g"].float(), flat["p"].float()
    m = m * h["beta1"] + g * (1 - h["beta1"])
    v = v * h["beta2"] + g * g * (1 - h["beta2"])
    den = v.sqrt() * (1 / math.sqrt(1 - h["beta2"] ** STEP)) + h["eps"]
    p = p * (1 - h["lr"] * h["weight_decay"]) - m / den * (h["lr"] / (1 - h["beta1"] ** STEP))
    flat["p"].copy_(p)
    if not eight:
        flat["m"].copy_(m)
        flat["v"].copy_(v)
        return {"p": flat["p"], "m": flat["m"], "v": flat["v"]}
    noise = _noise(s["run_number"], s["run_seed"])
    me, ve = _exponent(m.view(-1, BLOCK), 7), _exponent(v.view(-1, BLOCK), 15)
    flat["m"].copy_(_encode(m, me, 120, noise >> 12))
    flat["v"].copy_(_encode(v, ve, 112, noise & 0xFFFFF))
    flat["m_exp"].copy_(me + 127)
    flat["v_exp"].copy_(ve + 127)
    m, v = _moments(flat)
    return {"p": flat["p"], "m": m.bfloat16(), "v": v.bfloat16()}        # four significant bits: exact


def _own_adamw(s):
    import sparse_gemm_02_amd as S
    flat, lists = s["flat"], s["lists"]
    if s["case"]["bits"] == 32:
        S.slope_adamw_multi(lists["p"], lists["g"], lists["m"], lists["v"], STEP, **HYPER)
        return {"p": flat["p"], "m": flat["m"], "v": flat["v"]}
    S.slope_adamw_multi(lists["p"], lists["g"], lists["m"], lists["v"], STEP, m_exp=lists["m_exp"],
                        v_exp=lists["v_exp"], seed=s["seed"], **HYPER)
    m = torch.empty(flat["m"].shape, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(m)
    S.slope_adamw_moments(flat["m"], flat["m_exp"], flat["v"], flat["v_exp"], m, v)
    return {"p": flat["p"], "m": m, "v": v}


def _codes(x):
    """(values of E2M1 codes, scales' exponents) of rows x, blocks of 32 filled up with zeros."""
    x = torch.nn.functional.pad(x.float(), (0, -x.shape[1] % BLOCK)).view(x.shape[0], -1, BLOCK)
    # the exponent of the largest magnitude, rounded to E2M1's two bits, less two
    e = (((x.abs().amax(dim=2).view(torch.int32) + 0x200000) >> 23) - 129).clamp_min_(-127)
    y = x * _power(-e)[:, :, None]
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = ((a / step).round() * step).clamp_max(6.0)
    return torch.copysign(q, y), e


def _values(q, e, K):
    return (q * torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)[:, :, None]).view(q.shape[0], -1)[:, :K]


def _plain_quant(x):
    return _values(*_codes(x), x.shape[1]).bfloat16()                     # two significant bits: exact


def _plain_linear(s, xq):
    K = s["case"]["K"]
    return (_values(*xq, K) @ _values(*s["w"], K).t()).to(DTYPES[s["case"]["dt"]])


def _own_codes(x):
    import sparse_gemm_02_amd as S
    T, K = x.shape
    nc, ne = S.slope_mxfp4_row_bytes(K)
    codes = torch.empty((T, nc), dtype=torch.uint8, device=x.device)
    exps = torch.empty((T, ne), dtype=torch.uint8, device=x.device)
    S.slope_quantize_mxfp4(x, codes, exps)
    return codes, exps


def _own_quant(x):
    import sparse_gemm_02_amd as S
    codes, exps = _own_codes(x)
    out = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    S.slope_mxfp4_values(codes, exps, out)
    return out


def _own_linear(s, xq):
    import sparse_gemm_02_amd as S
    T, K, N = (s["case"][k] for k in ("T", "K", "N"))
    y = torch.empty((T, N), dtype=DTYPES[s["case"]["dt"]], device=xq[0].device)
    S.slope_spmm_mxfp4_packed(*xq, K, s["w"], N, y)
    return y


# ------------------------------------------------------------------ the definition in 64 bits

_BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)     # between neighbouring magnitudes of E2M1
_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_values(x):
    """What the 4-bit codes of rows x stand for."""
    T, K = x.shape
    out = torch.zeros((T, _blocks(K) * BLOCK), dtype=torch.float64, device=x.device)
    out[:, :K] = x
    out = out.view(-1, BLOCK)
    part, e = torch.frexp(out.abs().max(dim=1, keepdim=True).values)
    scale = torch.exp2((e - 3 + (part >= 0.875).to(e.dtype)).clamp(min=-127).double())
    a = out.abs() / scale
    code = torch.zeros(a.shape, dtype=torch.int64, device=x.device)
    for i, b in enumerate(_BORDERS):                   # a tie goes to the even code
        code += (a >= b) if i % 2 else (a > b)
    mags = torch.tensor(_MAGNITUDES, dtype=torch.float64, device=x.device)
    return (torch.sign(out) * mags[code] * scale).view(T, -1)[:, :K]


def _exact_words(seeds, sizes):
    """The 32-bit word of every value of the padded tensors, in numpy's unsigned arithmetic."""
    import numpy as np
    parts = []
    for seed, n in zip(seeds, sizes):
        s = np.arange(_blocks(n) * 4, dtype=np.uint32) * np.uint32(0x9E3779B1)
        s ^= np.uint32(seed)
        s ^= s >> np.uint32(16)
        s *= np.uint32(0xBB67AE85)
        s ^= s >> np.uint32(15)
        words = np.empty((s.size, 8), dtype=np.uint32)
        for j in range(8):
            s ^= s << np.uint32(13)
            s ^= s >> np.uint32(17)
            s ^= s << np.uint32(5)
            words[:, j] = s
        parts.append(words.reshape(-1))
    return torch.from_numpy(np.concatenate(parts).astype(np.int64)).cuda()


def _exact_rounded(x, bits, top, least):
    """x with each block's values on the 8-bit grid: the position among the
    codes, in 64 bits, plus a random part below one, rounded down."""
    x = x.view(-1, BLOCK)
    peak = x.abs().max(dim=1, keepdim=True).values
    e = (torch.frexp(peak)[1] - 1 - top).clamp(min=-127)
    a = x.abs() * torch.exp2(-e.double())
    binade = (torch.frexp(a)[1] - 1).clamp(min=least).double()
    # eighths of its binade, counted from the smallest normal number's binade
    at = 8 * (binade - least) + 8 * a * torch.exp2(-binade)
    code = torch.floor(at + bits.view(-1, BLOCK).double() / 2 ** 20)
    if top == 15:
        code = torch.maximum(code, (a > 0).double())
    low = (torch.floor(code / 8) - 1).clamp(min=0)
    value = (code - 8 * low) / 8 * torch.exp2(low + least)
    return (torch.sign(x) * value * torch.exp2(e.double())).view(-1)


def _exact_adamw(s):
    import numpy as np
    flat, h, eight = s["flat"], HYPER, s["case"]["bits"] == 8
    g = flat["g"].double()
    if eight:
        byte = np.arange(256)
        low = np.maximum(byte // 8 - 1, 0)
        table = torch.from_numpy((byte - 8 * low) / 8 * 2.0 ** low).cuda()
        wide = lambda k: torch.exp2(flat[k].double() - 127).repeat_interleave(BLOCK)
        code = flat["m"].long()
        m = table[code % 128] * 2.0 ** -6 * (1 - 2 * (code // 128)) * wide("m_exp")
        v = table[flat["v"].long()] * 2.0 ** -14 * wide("v_exp")
    else:
        m, v = flat["m"].double(), flat["v"].double()
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * g ** 2
    hat_m, hat_v = m / (1 - h["beta1"] ** STEP), v / (1 - h["beta2"] ** STEP)
    w = flat["p"].double()
    p = w - h["lr"] * h["weight_decay"] * w - h["lr"] * hat_m / (torch.sqrt(hat_v) + h["eps"])
    if eight:
        sizes = _sizes(s["case"])
        words = _exact_words(_tensor_seeds(s["seed"], len(sizes)), sizes)
        m = _exact_rounded(m, words // 4096, 7, -6)
        v = _exact_rounded(v, words % 2 ** 20, 15, -14)
    return {"p": p, "m": m, "v": v}


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
        if case["op"] == "adamw":
            return _exact_adamw(s)
        if case["op"] == "quant":
            return {"values": _exact_values(s["x"].double())}
        g = _generator(seed)
        x = _activations(g, case["T"], case["K"], DTYPES[case["dt"]]).double()
        w = _weight(g, case["N"], case["K"], torch.float16 if case["dt"] == "f16" else torch.bfloat16).double()
        return {"y": torch.mm(_exact_values(x), _exact_values(w).t().contiguous())}
    finally:
        own = kept

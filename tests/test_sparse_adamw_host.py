"""SparseAdamW's host side on the CPU: its checkpoints and load hooks, which calls a step
makes, in which order and with which numbers.  The library's calls are recorded in
place of run."""
import pytest
import torch

from sparse_gemm_02_amd import layer as M


def _parameter(n=40, dtype=torch.float32):
    return torch.nn.Parameter(torch.arange(n, dtype=torch.float32).to(dtype))


def _optimizer(params, **kw):
    return M.SparseAdamW([], extra_params=params, **kw)


def _filled(opt, value=3):
    """The optimizer with a state for each parameter, moments of `value`."""
    for g in opt.param_groups:
        for p in g["params"]:
            st = opt._state_of(p)
            st["step"] = 5
            for t in st.values():
                if isinstance(t, torch.Tensor):
                    t.fill_(value)
    return opt


# ------------------------------------------------------------------ checkpoints

@pytest.mark.parametrize("bits,dtype", [(32, torch.float32), (32, torch.bfloat16), (8, torch.bfloat16), (8, torch.float32)])
def test_load_hooks_have_their_effect(bits, dtype):
    """What a hook before the load puts into the dictionary is loaded, and what one after it puts into the
    state stays; the moments keep their own format."""
    saved = _filled(_optimizer([_parameter(dtype=dtype)], state_bits=bits)).state_dict()
    p = _parameter(dtype=dtype)
    opt = _optimizer([p], state_bits=bits)

    def before(_, given):
        state = {i: {**st, "exp_avg": torch.full_like(st["exp_avg"], 7)} for i, st in given["state"].items()}
        return {**given, "state": state}

    def after(o):
        o.state[p]["exp_avg_sq"].fill_(5)

    opt.register_load_state_dict_pre_hook(before)
    opt.register_load_state_dict_post_hook(after)
    opt.load_state_dict(saved)
    st = opt.state[p]
    want = torch.float32 if bits == 32 else torch.uint8
    assert st["step"] == 5 and st["exp_avg"].dtype is want and st["exp_avg_sq"].dtype is want
    assert (st["exp_avg"] == 7).all() and (st["exp_avg_sq"] == 5).all()
    if bits == 8:
        assert (st["exp_avg_exp"] == 3).all() and st["exp_avg_exp"].dtype is torch.uint8
    st["exp_avg"].zero_()                                            # the dictionary's tensors are not the state's
    assert (saved["state"][0]["exp_avg"] == 3).all()
    opt.load_state_dict(saved)                                       # the hooks are those that were registered, once more
    assert (opt.state[p]["exp_avg"] == 7).all() and (opt.state[p]["exp_avg_sq"] == 5).all()


def test_a_load_hook_may_convert_the_moments():
    """A checkpoint of 32-bit moments, turned into 8-bit ones (zeros here) by a hook before the load."""
    saved = _filled(_optimizer([_parameter()], state_bits=32)).state_dict()
    p = _parameter()
    opt = _optimizer([p], state_bits=8)
    with pytest.raises(ValueError, match="moments are"):
        opt.load_state_dict(saved)
    codes, exps = torch.full((40,), 9, dtype=torch.uint8), torch.full((2,), 100, dtype=torch.uint8)
    opt.register_load_state_dict_pre_hook(lambda _, given: {**given, "state": {0: {
        "step": 8, "exp_avg": codes, "exp_avg_exp": exps, "exp_avg_sq": codes, "exp_avg_sq_exp": exps}}})
    opt.load_state_dict(saved)
    assert opt.state[p]["step"] == 8 and torch.equal(opt.state[p]["exp_avg"], codes)
    assert torch.equal(opt.state[p]["exp_avg_sq_exp"], exps)


def test_saved_moments_of_other_formats():
    """Floating moments become float32 ones (torch's method makes them the parameter's format); codes do not;
    a refused load leaves the optimizer as it was."""
    for dtype in (torch.float64, torch.bfloat16, torch.float32):
        saved = _filled(_optimizer([_parameter()])).state_dict()
        st = saved["state"][0]
        st["exp_avg"], st["exp_avg_sq"] = st["exp_avg"].to(dtype), st["exp_avg_sq"].to(dtype)
        p = _parameter(dtype=torch.bfloat16)
        opt = _optimizer([p])
        opt.load_state_dict(saved)
        assert opt.state[p]["exp_avg"].dtype is torch.float32 and (opt.state[p]["exp_avg_sq"] == 3).all()
    codes = _filled(_optimizer([_parameter()], state_bits=8)).state_dict()
    with pytest.raises(ValueError, match="moments are torch.uint8"):
        opt.load_state_dict(codes)
    assert opt.state[p]["step"] == 5 and (opt.state[p]["exp_avg"] == 3).all()


@pytest.mark.parametrize("bits", [8, 32])
def test_a_saved_state_without_moments_is_refused(bits):
    names = ("exp_avg", "exp_avg_sq") + (("exp_avg_exp", "exp_avg_sq_exp") if bits == 8 else ())
    for name in names:
        saved = _filled(_optimizer([_parameter()], state_bits=bits)).state_dict()
        del saved["state"][0][name]
        with pytest.raises(ValueError, match=f"no {name}$"):
            _optimizer([_parameter()], state_bits=bits).load_state_dict(saved)
        # ... unless a hook after the load puts it there
        p = _parameter()
        opt = _optimizer([p], state_bits=bits)
        opt.register_load_state_dict_post_hook(lambda o: o.state[p].__setitem__(name, torch.zeros(1)))
        opt.load_state_dict(saved)
    saved = _filled(_optimizer([_parameter(), _parameter(7)], state_bits=bits)).state_dict()
    del saved["state"][0]                                            # a parameter that had no step yet
    opt = _optimizer([_parameter(), _parameter(7)], state_bits=bits)
    opt.load_state_dict(saved)
    assert len(opt.state) == 1


# ------------------------------------------------------------------ steps

class Recorded:
    """The library's calls of a step, in order: ("list" or "layer", parameters, step, seed).  A list is refused
    as the library refuses it; weights take a step along their gradient, so that the order shows."""

    def __init__(self, monkeypatch):
        self.calls, self.refuse = [], None
        monkeypatch.setattr(M, "slope_adamw_multi", self._list)
        monkeypatch.setattr(M, "slope_adamw_double_prune_packed", self._layer32)
        monkeypatch.setattr(M, "slope_adamw8_double_prune_packed", self._layer8)

    @staticmethod
    def _span(t):
        return t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()

    def _list(self, ps, gs, m, v, step, m_exp=None, v_exp=None, seed=0, **hp):
        meet = lambda a, b: max(a[0], b[0]) < min(a[1], b[1])
        written = [self._span(t) for t in (*ps, *m, *v, *(m_exp or ()), *(v_exp or ())) if t.numel()]
        read = [self._span(t) for t in gs if t.numel()]
        assert not any(meet(a, b) for i, a in enumerate(written) for b in written[:i] + read), "INVALID_ARG"
        self._step("list", ps, gs, step, seed)

    def _layer32(self, p, meta, g, m, v, N, K, ps, pd, step, **hp):
        self._step("layer", [p], [g], step, None)

    def _layer8(self, p, meta, g, m, me, v, ve, N, K, ps, pd, step, seed=0, **hp):
        self._step("layer", [p], [g], step, seed)

    def _step(self, kind, ps, gs, step, seed):
        if self.refuse is not None and any(p is self.refuse for p in ps):
            raise ValueError("refused")
        self.calls.append((kind, list(ps), step, seed))
        for p, g in zip(ps, gs):
            p.copy_(2 * p + g)


def _layer(N=16, K=64, dtype=torch.bfloat16):
    layer = M.SparseLinear.__new__(M.SparseLinear)
    torch.nn.Module.__init__(layer)
    layer.in_features, layer.out_features, layer.rank = K, N, 0
    layer.values = torch.nn.Parameter(torch.randn(N, K // 2).to(dtype))
    layer.meta = layer.packed_s = layer.packed_dpT = None
    return layer


def _in_turn(params, grads):
    """What a call for each parameter in their order leaves in the memory that `params` are views of."""
    for p, g in zip(params, grads):
        p.data.copy_(2 * p.data + g)


@pytest.mark.parametrize("bits", [8, 32])
def test_parameters_that_overlap_in_part_take_turns(monkeypatch, bits):
    rec = Recorded(monkeypatch)
    def make():
        flat = torch.arange(96, dtype=torch.float32)
        own = torch.arange(5, dtype=torch.float32)
        views = [flat, own, flat[10:40], flat[30:], flat[40:41], own[4:], flat[0:0]]
        return flat, own, [torch.nn.Parameter(v) for v in views]
    flat, own, params = make()
    grads = [torch.randn(p.shape) for p in params]
    opt = _optimizer(params, state_bits=bits)
    for p, g in zip(params, grads):
        p.grad = g
    opt.step()
    want, want_own, again = make()
    _in_turn(again, grads)
    assert torch.equal(flat, want) and torch.equal(own, want_own)
    # three turns: the wholes, then what overlaps them alone, then what overlaps a part of the second turn
    assert [[next(i for i, q in enumerate(params) if q is p) for p in ps] for _, ps, _, _ in rec.calls] == [[0, 1, 6], [2, 5], [3], [4]]


def test_gradients_that_are_weights_of_the_step(monkeypatch):
    """A gradient over its own weight, over one that is stepped before it and over one that is stepped after it."""
    Recorded(monkeypatch)
    a, b, c, d = (torch.randn(33) for _ in range(4))
    start = [t.clone() for t in (a, b, c, d)]
    params = [torch.nn.Parameter(t) for t in (a, b, c, d)]
    for p, g in zip(params, (a, a, d, torch.ones(33))):
        p.grad = g
    _optimizer(params).step()
    a0, b0, c0, d0 = start
    assert torch.equal(a, 2 * a0 + a0) and torch.equal(b, 2 * b0 + a) and torch.equal(c, 2 * c0 + d0) and torch.equal(d, 2 * d0 + 1)


@pytest.mark.parametrize("bits", [8, 32])
def test_layers_take_turns_with_what_overlaps_them(monkeypatch, bits):
    rec = Recorded(monkeypatch)
    layer, other = _layer(), _layer()
    row = torch.nn.Parameter(layer.values.data[3])
    params = [row, layer.values, other.values, torch.nn.Parameter(torch.randn(9))]
    start = layer.values.detach().clone()
    opt = M.SparseAdamW([], extra_params=params, state_bits=bits)
    opt._layer_of = {l.values: l for l in (layer, other)}
    for p in params:
        p.grad = torch.randn(p.shape).to(p.dtype)
    opt.step()
    start[3] = 2 * start[3] + row.grad
    assert torch.equal(layer.values, 2 * start + layer.values.grad)
    assert [kind for kind, *_ in rec.calls] == ["layer", "list", "layer"]
    # without a common byte: the layers, then one list
    rec.calls.clear()
    params[0].grad = None
    opt.state[layer.values]["step"] = 0
    opt.step()
    assert [(kind, len(ps)) for kind, ps, *_ in rec.calls] == [("layer", 1), ("layer", 1), ("list", 1)]


@pytest.mark.parametrize("bits", [8, 32])
def test_a_refused_call_counts_no_step(monkeypatch, bits):
    """Where the library refuses a call, the parameters' step numbers are those of the calls that it took."""
    rec = Recorded(monkeypatch)
    layers = [_layer(), _layer()]
    w = torch.randn(64)
    rest = [torch.nn.Parameter(torch.randn(9)), torch.nn.Parameter(w), torch.nn.Parameter(w[:32])]
    params = [l.values for l in layers] + rest
    opt = M.SparseAdamW([], extra_params=params, state_bits=bits)
    opt._layer_of = {l.values: l for l in layers}
    for p in params:
        p.grad = torch.zeros_like(p)
    steps = lambda: [opt.state[p].get("step", 0) for p in params]
    for refuse, want in [(params[1], [1, 0, 0, 0, 0]), (rest[0], [2, 1, 0, 0, 0]), (rest[2], [3, 2, 1, 1, 0])]:
        rec.refuse = refuse
        with pytest.raises(ValueError, match="refused"):
            opt.step()
        assert steps() == want
    rec.refuse = None
    rec.calls.clear()
    opt.step()
    assert steps() == [4, 3, 2, 2, 1]
    assert [(len(ps), t) for _, ps, t, _ in rec.calls] == [(1, 4), (1, 3), (2, 2), (1, 1)]


def test_a_step_number_that_is_a_tensor(monkeypatch):
    """As other optimizers' checkpoints have it: parameters of one number still take one call."""
    rec = Recorded(monkeypatch)
    params = [_parameter(), _parameter(7)]
    opt = _filled(_optimizer(params))
    saved = opt.state_dict()
    for st in saved["state"].values():
        st["step"] = torch.tensor(5.0)
    opt.load_state_dict(saved)
    for p in params:
        p.grad = torch.zeros_like(p)
    opt.step()
    assert [(len(ps), t) for _, ps, t, _ in rec.calls] == [(2, 6)] and opt.state[params[0]]["step"] == 6


def test_parameters_too_large_for_a_list(monkeypatch):
    """slope_adamw_multi takes tensors of at most 2^34 values; larger ones with 32-bit moments have a call of
    slope_adamw's each, as far as that goes.  (Tensors without memory stand for them.)"""
    calls = []
    monkeypatch.setattr(M, "slope_adamw_multi", lambda ps, *a, **k: calls.append([p.numel() for p in ps]))
    monkeypatch.setattr(M, "slope_adamw", lambda p, g, m, v, step, **hp: calls.append((p.numel(), step, hp["lr"])))
    sizes = [1 << 34, (1 << 34) + 1, 64]
    params = [torch.nn.Parameter(torch.empty(n, dtype=torch.bfloat16, device="meta")) for n in sizes]
    monkeypatch.setattr(M, "_turns", lambda ps, gs: [0] * len(ps))
    opt = _optimizer(params, lr=0.5)
    for p in params:
        p.grad = torch.empty_like(p)
    opt.step()
    opt.step()
    assert calls == [((1 << 34) + 1, 1, 0.5), [1 << 34, 64], ((1 << 34) + 1, 2, 0.5), [1 << 34, 64]]


# ------------------------------------------------------------------ random bits

def test_seeds_of_neighbouring_optimizers_and_lists_are_apart(monkeypatch):
    """No two of the lists of a step, of steps and of optimizers with other seeds have the same random bits:
    300 parameters over one tensor make 300 lists."""
    rec = Recorded(monkeypatch)
    w = torch.zeros(4)
    seen, first = set(), {}
    seeds = [0, 1, 2, (1 << 24) - 1, 1 << 24, (1 << 24) + 1, 1 << 40, (1 << 64) - 1, -2]
    for seed in seeds:
        params = [torch.nn.Parameter(w) for _ in range(300)]
        opt = _optimizer(params, state_bits=8, seed=seed, lr=0.0)
        for p in params:
            p.grad = torch.zeros(4)
        rec.calls.clear()
        opt.step()
        opt.step()
        got = [(s & (2 ** 64 - 1), t) for _, _, t, s in rec.calls]
        assert [t for _, t in got] == [1] * 300 + [2] * 300
        seen |= {s for s, _ in got}
        first[seed] = [s for s, _ in got]
    assert len(seen) == len(seeds) * 600
    # the numbers that they always had: seeds of 24 bits, the first 256 lists of a step
    for seed in (0, 1, 2, (1 << 24) - 1):
        assert first[seed][:256] == [(seed << 40) + (done << 32) + 1 for done in range(256)]


def test_layers_take_seeds_in_their_order(monkeypatch):
    rec = Recorded(monkeypatch)
    layers = [_layer(), _layer()]
    params = [l.values for l in layers] + [_parameter()]
    opt = M.SparseAdamW([], extra_params=params, state_bits=8, seed=6)
    opt._layer_of = {l.values: l for l in layers}
    for p in params:
        p.grad = torch.zeros_like(p)
    opt.step()
    assert [s for *_, s in rec.calls] == [(6 << 40) + (done << 32) + 1 for done in range(3)]


def test_the_seed_is_part_of_a_checkpoint(monkeypatch, tmp_path):
    """A resumed run goes on with the random bits of the uninterrupted one, whatever seed the new optimizer was
    made with."""
    rec = Recorded(monkeypatch)
    p = _parameter()
    def run(o):
        rec.calls.clear()
        p.grad = torch.zeros_like(p)
        o.step()
        return [s for *_, s in rec.calls]
    opt = _optimizer([p], state_bits=8, seed=77)
    run(opt)
    torch.save(opt.state_dict(), tmp_path / "opt.pt")
    want = run(opt)
    assert want == [(77 << 40) + 2]
    again = _optimizer([p], state_bits=8)
    again.load_state_dict(torch.load(tmp_path / "opt.pt", weights_only=True))
    assert run(again) == want and again.seed == 77
    # a checkpoint without one leaves the optimizer's own; a hook before the load may change it
    old = torch.load(tmp_path / "opt.pt", weights_only=True)
    del old["seed"]
    other = _optimizer([p], state_bits=8, seed=5)
    other.load_state_dict(old)
    assert run(other) == [(5 << 40) + 2]
    other.register_load_state_dict_pre_hook(lambda _, given: {**given, "seed": 9})
    other.load_state_dict(old)
    assert other.seed == 9
    # 32-bit moments take no random bits, and their checkpoints are as they were
    assert set(_optimizer([p]).state_dict()) == {"state", "param_groups"}


@pytest.mark.parametrize("bits", [8, 32])
def test_copies_of_an_optimizer(monkeypatch, bits):
    """A deep copy (and a pickled one) saves, loads and steps as the optimizer does, on its own parameters and layers."""
    import copy
    import pickle
    rec = Recorded(monkeypatch)
    layer = _layer()
    opt = M.SparseAdamW([layer], extra_params=[_parameter()], state_bits=bits, seed=3)
    _filled(opt)
    for make in (copy.deepcopy, lambda o: pickle.loads(pickle.dumps(o))):
        other = make(opt)
        saved = other.state_dict()
        assert saved.get("seed") == (3 if bits == 8 else None) and len(saved["state"]) == 2
        other.load_state_dict(opt.state_dict())
        params = other.param_groups[0]["params"]
        assert not any(p is q for p in params for q in opt.param_groups[0]["params"])
        for p in params:
            p.grad = torch.zeros_like(p)
        rec.calls.clear()
        other.step()
        assert [kind for kind, *_ in rec.calls] == ["layer", "list"] and rec.calls[0][1][0] is params[0]
        assert other.state[params[0]]["step"] == 6 and opt.state[layer.values]["step"] == 5

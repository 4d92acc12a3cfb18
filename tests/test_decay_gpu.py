"""gdn_decay_step and gdn_decay_prefill (linear attention with a decay per
head) against the rule in 64 bits, and the properties the interface states."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import commit_gated_delta_amd as gdn  # noqa: E402
from tests import serving_ref as ref  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _rand(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *shape: torch.randn(shape, device="cuda", generator=g)


def _gates(x, kind):
    """Log-decays from normal draws."""
    if kind == "slow":
        return -torch.nn.functional.softplus(x - 2)
    if kind == "fast":
        return -torch.nn.functional.softplus(x) * 8
    if kind == "cut":      # some tokens forget everything before them
        y = -torch.nn.functional.softplus(x - 2)
        return torch.where(x > 1.2, torch.where(x > 1.7, -math.inf, -5000.0), y)
    if kind == "mixed":    # long and short memories side by side
        return torch.where(x > 0, -90 * x, -1e-3 * x.abs())
    raise ValueError(kind)


def _near(x, want, mag, rel, what):
    err = (x.double() - want).abs()
    lim = rel * mag + 1e-30
    assert torch.isfinite(x).all(), what
    worst = float((err / lim).max()) if err.numel() else 0.0
    print("%s: %.3g of its bound" % (what, worst), flush=True)
    assert worst <= 1, (what, worst)


# ------------------------------------------------------------------ prompts
def _prompt(lens, h_v, h_k, d_k, d_v, kind, gates, per_head, init, seed=0,
            scale=0.25):
    rand = _rand(seed)
    n, t = sum(lens), TYPES[kind]
    x = dict(q=rand(n, h_k, d_k).to(t), k=rand(n, h_k, d_k).to(t),
             v=rand(n, h_v, d_v).to(t))
    x["g"] = _gates(rand(h_v) if per_head else rand(n, h_v), gates)
    x["S0"] = rand(len(lens), h_v, d_k, d_v) if init else None
    return x


def _run_prompt(lens, h_v, h_k, d_k, d_v, x, per_head, scale=0.25,
                S_final=None, want_o=True):
    ws = gdn.decay_prefill_workspace_bytes(lens, h_v, h_k, d_k, d_v)
    ws = torch.empty(ws, dtype=torch.uint8, device="cuda")
    S = torch.full((len(lens), h_v, d_k, d_v), math.nan, device="cuda") \
        if S_final is None else S_final
    o = torch.full((sum(lens), h_v, d_v), math.nan, device="cuda")
    gdn.decay_prefill(lens, h_v, h_k, d_k, d_v, x["q"] if want_o else None,
                      x["k"], x["v"], x["g"], x["S0"], S,
                      o if want_o else None, ws, scale=scale,
                      head_decay=per_head)
    torch.cuda.synchronize()
    return o, S


def _check_prompt(lens, h_v, h_k, d_k, d_v, x, per_head, o, S, scale=0.25):
    at = 0
    for i, T in enumerate(lens):
        rep = lambda y: y[at:at + T].double().repeat_interleave(h_v // h_k, 1)
        g = x["g"].expand(T, h_v) if per_head else x["g"][at:at + T]
        S0 = x["S0"][i] if x["S0"] is not None else torch.zeros(
            h_v, d_k, d_v, device="cuda")
        wo, wS, mo, mS = ref.decay_chain(rep(x["q"]), rep(x["k"]),
                                         x["v"][at:at + T], g, S0, scale)
        rel = ref.decay_bound(d_k, T)
        if T:
            _near(o[at:at + T], wo, mo, rel, "o of sequence %d" % i)
        _near(S[i], wS, mS, rel, "S of sequence %d" % i)
        at += T


@pytest.mark.parametrize("lens,h_v,h_k,d_k,d_v,kind,gates,per_head,init", [
    ([1], 1, 1, 16, 1, "f32", "slow", False, False),
    ([1], 2, 1, 128, 128, "bf16", "slow", False, True),
    ([64], 4, 4, 128, 128, "bf16", "slow", False, True),
    ([63, 0, 65], 4, 2, 128, 128, "bf16", "slow", False, True),
    ([200], 3, 1, 128, 100, "bf16", "slow", False, True),
    ([5, 130, 0, 1], 2, 2, 128, 33, "bf16", "fast", False, False),
    ([129], 4, 1, 64, 64, "bf16", "cut", False, True),
    ([333, 64], 2, 1, 32, 40, "bf16", "mixed", False, True),
    ([190], 2, 1, 16, 256, "bf16", "slow", True, True),
    ([777, 5], 2, 1, 128, 128, "f32", "slow", False, True),
    ([200, 200], 2, 2, 64, 96, "f32", "cut", False, False),
    ([100], 2, 1, 128, 130, "f32", "mixed", False, True),
    ([256], 4, 2, 128, 64, "f32", "fast", True, False),
    ([1200, 1, 2500], 2, 1, 128, 128, "bf16", "slow", True, True),
    ([4500], 1, 1, 128, 128, "bf16", "mixed", False, True),
    ([3000], 2, 2, 64, 64, "f32", "slow", False, False),
    ([150], 1, 1, 128, 1024, "bf16", "slow", False, True),
])
def test_prompts(lens, h_v, h_k, d_k, d_v, kind, gates, per_head, init):
    x = _prompt(lens, h_v, h_k, d_k, d_v, kind, gates, per_head, init)
    o, S = _run_prompt(lens, h_v, h_k, d_k, d_v, x, per_head)
    _check_prompt(lens, h_v, h_k, d_k, d_v, x, per_head, o, S)


def test_256_sequences():
    lens = [(i * 37) % 90 for i in range(256)]
    x = _prompt(lens, 2, 1, 64, 64, "bf16", "slow", False, True)
    o, S = _run_prompt(lens, 2, 1, 64, 64, x, False)
    _check_prompt(lens, 2, 1, 64, 64, x, False, o, S)


@pytest.mark.parametrize("lens", [[70, 0, 3], [5000, 0, 9]])
def test_states_only_and_in_place(lens):
    """o = NULL gives the same states bit for bit; S_final may be S_init;
    an empty sequence keeps its state."""
    x = _prompt(lens, 2, 1, 128, 128, "bf16", "slow", False, True)
    _, S = _run_prompt(lens, 2, 1, 128, 128, x, False)
    _, S2 = _run_prompt(lens, 2, 1, 128, 128, x, False, want_o=False)
    assert torch.equal(S, S2)
    assert torch.equal(S[1], x["S0"][1])
    x["S0"] = x["S0"].clone()
    _, S3 = _run_prompt(lens, 2, 1, 128, 128, x, False, S_final=x["S0"])
    assert torch.equal(S, S3)


def test_outputs_only():
    lens = [100, 2100]
    x = _prompt(lens, 2, 2, 128, 128, "bf16", "slow", False, True)
    o, _ = _run_prompt(lens, 2, 2, 128, 128, x, False)
    ws = torch.empty(gdn.decay_prefill_workspace_bytes(lens, 2, 2, 128, 128),
                     dtype=torch.uint8, device="cuda")
    o2 = torch.empty_like(o)
    gdn.decay_prefill(lens, 2, 2, 128, 128, x["q"], x["k"], x["v"], x["g"],
                      x["S0"], None, o2, ws, scale=0.25)
    assert torch.equal(o, o2)


def test_prompts_repeat_bit_for_bit():
    lens = [3000, 17, 640]
    x = _prompt(lens, 4, 2, 128, 128, "bf16", "slow", False, True)
    a = _run_prompt(lens, 4, 2, 128, 128, x, False)
    b = _run_prompt(lens, 4, 2, 128, 128, x, False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_what_lies_behind_the_tokens_does_not_matter():
    """Rows after the last token (NaN here) are neither read into a result
    nor written."""
    lens = [37, 70]
    n = sum(lens)
    x = _prompt(lens + [100], 2, 1, 128, 128, "bf16", "slow", False, False)
    for name in ("q", "k", "v", "g"):
        x[name][n:] = math.nan
    S = torch.empty(2, 2, 128, 128, device="cuda")
    o = torch.full((n + 100, 2, 128), 7.0, device="cuda")
    gdn.decay_prefill(lens, 2, 1, 128, 128, x["q"], x["k"], x["v"], x["g"],
                      None, S, o, torch.empty(
                          gdn.decay_prefill_workspace_bytes(lens, 2, 1, 128, 128),
                          dtype=torch.uint8, device="cuda"), scale=0.25)
    _check_prompt(lens, 2, 1, 128, 128, x, False, o[:n], S)
    assert (o[n:] == 7).all()


@pytest.mark.parametrize("kind,d_k,d_v", [("bf16", 128, 128), ("bf16", 128, 50),
                                          ("f32", 64, 64)])
def test_infinities_and_nan_reach_no_earlier_token(kind, d_k, d_v):
    """What a token's value row holds changes nothing before the token, in its
    chunk of the prompt or before it, nor other heads, columns or sequences."""
    lens, t = [700, 90], 333
    x = _prompt(lens, 2, 1, d_k, d_v, kind, "slow", False, True)
    clean, S = _run_prompt(lens, 2, 1, d_k, d_v, x, False)
    x["v"][t, 0, 5] = math.inf
    x["v"][t, 0, 9] = math.nan
    o, S2 = _run_prompt(lens, 2, 1, d_k, d_v, x, False)
    keep = torch.ones_like(o, dtype=torch.bool)
    keep[t:700, 0, 5] = keep[t:700, 0, 9] = False
    # (the chunk's sums are made in another order then)
    assert torch.isfinite(o[keep]).all()
    assert float((o - clean)[keep].abs().max()) <= 1e-4 * float(clean.abs().max())
    assert torch.equal(o[:, 1], clean[:, 1]) or float(
        (o - clean)[:, 1].abs().max()) <= 1e-4 * float(clean.abs().max())
    assert torch.equal(o[700:], clean[700:])
    assert (torch.isinf(o[t, 0, 5]) or torch.isnan(o[t, 0, 5])) and torch.isnan(o[t, 0, 9])
    assert torch.equal(S2[1], S[1]) and torch.equal(S2[0, 1], S[0, 1])
    assert torch.isfinite(S2[0, 0, :, :5]).all() and torch.isnan(S2[0, 0, :, 9]).all()


def test_no_tokens():
    """Sequences without tokens hand their states through."""
    S0 = torch.randn(2, 2, 64, 64, device="cuda")
    S = torch.empty_like(S0)
    e = torch.empty(0, 2, 64, device="cuda")
    gdn.decay_prefill([0, 0], 2, 2, 64, 64, e, e, e,
                      torch.empty(0, 2, device="cuda"), S0, S, e, None)
    assert torch.equal(S, S0)
    gdn.decay_prefill([0, 0], 2, 2, 64, 64, e, e, e,
                      torch.empty(0, 2, device="cuda"), None, S, e, None)
    assert (S == 0).all()


# ------------------------------------------------------------------ windows
def _window(layers, t_lane, h_v, h_k, d_k, d_v, T, kind, gates, per_head,
            seed=1):
    rand, t, N = _rand(seed), TYPES[kind], len(t_lane)
    x = dict(q=rand(layers, N, T, h_k, d_k).to(t),
             k=rand(layers, N, T, h_k, d_k).to(t),
             v=rand(layers, N, T, h_v, d_v).to(t),
             S=rand(layers, N, h_v, d_k, d_v))
    x["g"] = _gates(rand(layers, h_v) if per_head else rand(layers, N, T, h_v),
                    gates)
    for n, m in enumerate(t_lane):      # rows past a window are never read
        for name in ("q", "k", "v") + (() if per_head else ("g",)):
            x[name][:, n, m:] = math.nan
    return x


def _run_window(x, t_lane, per_head, keep=False, want_o=True, scale=0.5):
    layers, N, T, h_k, d_k = x["q"].shape
    h_v, d_v = x["v"].shape[3:]
    dims = gdn.Dims.of(layers, N, h_v, h_k, d_k, d_v, T)
    S = x["S"].clone()
    o = torch.full(x["v"].shape, 7.0, device="cuda")
    gdn.decay_step(dims, t_lane, x["q"] if want_o else None, x["k"], x["v"],
                   x["g"], S, o if want_o else None, scale=scale,
                   head_decay=per_head, keep_state=keep)
    torch.cuda.synchronize()
    return o, S


@pytest.mark.parametrize("layers,t_lane,h_v,h_k,d_k,d_v,T,kind,gates,per_head", [
    (1, [1], 1, 1, 16, 1, 1, "f32", "slow", False),
    (1, [1, 1, 0], 4, 2, 128, 128, 1, "bf16", "slow", False),
    (2, [3, 0, 7], 4, 1, 128, 128, 7, "bf16", "slow", False),
    (1, [16, 5], 2, 2, 128, 100, 16, "bf16", "cut", False),
    (1, [64], 2, 1, 128, 33, 64, "f32", "mixed", False),
    (3, [2], 2, 1, 64, 64, 2, "f32", "slow", True),
    (2, [4, 4], 6, 2, 32, 40, 4, "bf16", "fast", True),
    (1, [9, 1], 2, 1, 16, 256, 9, "bf16", "slow", False),
    (1, [2], 1, 1, 128, 1024, 2, "bf16", "slow", False),
])
def test_windows(layers, t_lane, h_v, h_k, d_k, d_v, T, kind, gates, per_head):
    x = _window(layers, t_lane, h_v, h_k, d_k, d_v, T, kind, gates, per_head)
    o, S = _run_window(x, t_lane, per_head)
    for y in range(layers):
        for n, m in enumerate(t_lane):
            rep = lambda z: z[y, n, :m].double().repeat_interleave(h_v // h_k, 1)
            g = x["g"][y].expand(m, h_v) if per_head else x["g"][y, n, :m]
            wo, wS, mo, mS = ref.decay_chain(rep(x["q"]), rep(x["k"]),
                                             x["v"][y, n, :m], g, x["S"][y, n], 0.5)
            rel = ref.step_bound(d_k, max(m, 1))
            _near(o[y, n, :m], wo, mo, rel, "o layer %d lane %d" % (y, n))
            _near(S[y, n], wS, mS, rel, "S layer %d lane %d" % (y, n))
            assert (o[y, n, m:] == 7).all()      # left as they were
            if m == 0:
                assert torch.equal(S[y, n], x["S"][y, n])


@pytest.mark.parametrize("kind,d_k,d_v", [("bf16", 128, 128), ("f32", 64, 50)])
def test_verify_commit_and_single_tokens_agree_bit_for_bit(kind, d_k, d_v):
    """A verify leaves the state alone; committing m tokens of it, the window
    in one call and its tokens one by one give the same bits."""
    T, t_lane, m = 13, [13, 6, 13], [4, 6, 0]
    x = _window(2, t_lane, 4, 2, d_k, d_v, T, kind, "slow", False)
    o, S = _run_window(x, t_lane, False, keep=True)
    assert torch.equal(S, x["S"])
    o2, S_T = _run_window(x, t_lane, False)
    assert torch.equal(o, o2)
    _, S_m = _run_window(x, m, False, want_o=False)
    dims = gdn.Dims.of(2, 3, 4, 2, d_k, d_v, 1)
    S1 = x["S"].clone()
    for t in range(T):
        y = {a: x[a][:, :, t:t + 1].contiguous() for a in ("q", "k", "v", "g")}
        o1 = torch.full((2, 3, 1, 4, d_v), 7.0, device="cuda")
        gdn.decay_step(dims, [int(t < n) for n in t_lane], y["q"], y["k"],
                       y["v"], y["g"], S1, o1, scale=0.5)
        assert torch.equal(o1[:, :, 0], o[:, :, t])
        for n in range(3):
            if m[n] == t + 1:
                assert torch.equal(S1[:, n], S_m[:, n])
    assert torch.equal(S1, S_T)
    assert torch.equal(S_m[:, 2], x["S"][:, 2])


def test_a_layer_of_the_gates():
    """One layer's constant decays out of all layers' (8-byte aligned)."""
    x = _window(1, [3, 2], 2, 1, 64, 64, 3, "bf16", "slow", True)
    want = _run_window(x, [3, 2], True)
    g = torch.stack([x["g"][0] - 1, x["g"][0], x["g"][0] + 1])
    got = _run_window(dict(x, g=g[1:2]), [3, 2], True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_256_lanes():
    t_lane = [i % 3 for i in range(256)]
    x = _window(1, t_lane, 2, 1, 64, 64, 2, "bf16", "slow", False)
    o, S = _run_window(x, t_lane, False)
    for n in (0, 1, 2, 127, 254, 255):
        m = t_lane[n]
        rep = lambda z: z[0, n, :m].double().repeat_interleave(2, 1)
        wo, wS, mo, mS = ref.decay_chain(rep(x["q"]), rep(x["k"]),
                                         x["v"][0, n, :m], x["g"][0, n, :m],
                                         x["S"][0, n], 0.5)
        _near(S[0, n], wS, mS, ref.step_bound(64, 2), "S lane %d" % n)
        if m:
            _near(o[0, n, :m], wo, mo, ref.step_bound(64, 2), "o lane %d" % n)


def test_prompt_agrees_with_steps():
    T = 50
    x = _window(1, [T], 2, 1, 128, 128, T, "bf16", "slow", False)
    o, S = _run_window(x, [T], False)
    y = {a: x[a][0, 0] for a in ("q", "k", "v", "g")}
    y["S0"] = x["S"][0]
    o2, S2 = _run_prompt([T], 2, 1, 128, 128, y, False, scale=0.5)
    _check_prompt([T], 2, 1, 128, 128, y, False, o2, S2, scale=0.5)
    assert float((o2 - o[0, 0]).abs().max()) < 1e-3 * float(o.abs().max())


def test_captured_calls_replay():
    """A prompt and a step in one captured graph, replayed on changed inputs
    with the program's own work between the replays."""
    lens = [2100, 70]
    x = _prompt(lens, 2, 1, 128, 128, "bf16", "slow", False, True)
    w = _window(1, [1, 1], 2, 1, 128, 128, 1, "bf16", "slow", False)
    dims = gdn.Dims.of(1, 2, 2, 1, 128, 128, 1)
    ws = torch.empty(gdn.decay_prefill_workspace_bytes(lens, 2, 1, 128, 128),
                     dtype=torch.uint8, device="cuda")
    S, o = torch.empty(2, 2, 128, 128, device="cuda"), torch.empty(
        sum(lens), 2, 128, device="cuda")
    o1 = torch.empty(1, 2, 1, 2, 128, device="cuda")

    def calls():
        gdn.decay_prefill(lens, 2, 1, 128, 128, x["q"], x["k"], x["v"], x["g"],
                          x["S0"], S, o, ws)
        gdn.decay_step(dims, [1, 1], w["q"], w["k"], w["v"], w["g"],
                       S.view(1, 2, 2, 128, 128), o1)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for i in range(3):
        x["v"].copy_(torch.randn_like(x["v"]))
        w["v"].copy_(torch.randn_like(w["v"]))
        calls()
        torch.cuda.synchronize()
        want = [y.clone() for y in (S, o, o1)]
        for y in (S, o, o1):
            y.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        for y, z in zip((S, o, o1), want):
            assert torch.equal(y, z), i


def test_another_stream():
    lens = [600, 5]
    x = _prompt(lens, 2, 1, 128, 128, "bf16", "slow", False, True)
    want = _run_prompt(lens, 2, 1, 128, 128, x, False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _run_prompt(lens, 2, 1, 128, 128, x, False)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])

"""gdn_draft_verify against the definition in 64 bits."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import commit_gated_delta_amd as gdn  # noqa: E402
from tests import cache_ref as ref  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _case(t_lane, V, kind, drafted, T=None, seed=0, pad=0, offset=0, right=0.8):
    """Logits with one token that stands out in every row; drafts that are it
    most of the time; the drafter's logits near the model's."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n, T, t = len(t_lane), T or max(max(t_lane), 1), TYPES[kind]
    rand = lambda *s: torch.rand(s, device="cuda", generator=g)
    x = 2 * torch.randn(n, T, V, device="cuda", generator=g)
    best = torch.randint(V, (n, T), device="cuda", generator=g)
    x.scatter_(2, best[..., None], 2 + math.log(V) + 2 * rand(n, T, 1))

    def rows(y):       # with a row stride past the vocabulary, at an odd element
        if not pad and not offset:
            return y.to(t)
        a = torch.full((y.shape[0], y.shape[1], V + pad), math.nan, device="cuda", dtype=t)
        a = torch.cat([torch.zeros(offset, device="cuda", dtype=t), a.view(-1)])[offset:].view(y.shape[0], y.shape[1], V + pad)
        a[..., :V] = y
        return a[..., :V]

    s = dict(t_lane=t_lane, logits=rows(x))
    s["draft"] = rows(x[:, :-1] + 0.7 * torch.randn(n, T - 1, V, device="cuda", generator=g)) if drafted else None
    other = torch.randint(V, (n, T), device="cuda", generator=g)
    tokens = torch.where(rand(n, T) < right, torch.roll(best, 1, 1), other)
    s["tokens"] = tokens.to(torch.int32)
    s["uniforms"] = rand(n, T)
    s["it"] = 0.7 + 0.6 * rand(n)
    return s


def _run(s, stream=None):
    n, T, V = s["logits"].shape
    m, token = (torch.full((n,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    accept = torch.full((n, T), 7.0, device="cuda")
    ws = torch.empty(gdn.draft_verify_workspace_bytes(n, T, V), dtype=torch.uint8, device="cuda")
    gdn.draft_verify(s["t_lane"], s["logits"], s["draft"], s["tokens"], s["uniforms"], s["it"], m, token, ws,
                     accept=accept, stream=stream)
    torch.cuda.synchronize()
    return m.tolist(), token.tolist(), accept.cpu().double()


def _check(s, got, at_least=0.9):
    m, token, accept = got
    want = ref.verify(s["t_lane"], s["logits"], s["draft"], s["tokens"], s["uniforms"], s["it"])
    tol = ref.chance_bound(s["logits"], s["draft"], s["it"])
    sure = 0
    for n, w in enumerate(want):
        if w is None:
            assert m[n] == token[n] == -9 and (accept[n] == 7).all()
            sure += 1
            continue
        for t, c in enumerate(w[2]):
            a = float(accept[n, t])
            assert math.isnan(a) if math.isnan(c) else abs(a - c) <= tol * c, (n, t, a, c)
        assert (accept[n, len(w[2]):] == 7).all()
        if w[3]:
            continue       # a decision within rounding of its border
        sure += 1
        assert (m[n], token[n]) == w[:2], (n, m[n], token[n], w[:2])
    assert sure >= at_least * len(want)


@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("t_lane,V,kind", [
    ([1], 1, "f32"),
    ([3, 1, 2], 2, "f32"),
    ([1], 1000, "bf16"),
    ([4, 0, 2, 1], 37, "bf16"),
    ([16, 5, 1, 9], 1111, "f32"),
    ([6] * 12, 5003, "bf16"),
    ([64, 33], 300, "f32"),
    ([2, 3], 131072, "f32"),
    ([3], 131072, "bf16"),
    ([1, 1], 262144, "bf16"),
    ([4, 2], 65537, "f32"),
])
def test_verify(t_lane, V, kind, drafted):
    s = _case(t_lane, V, kind, drafted)
    _check(s, _run(s), 0.5)


@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("V,pad,offset", [(1001, 7, 1), (1024, 8, 3), (40007, 1, 5)])
def test_padded_rows_at_odd_places(V, pad, offset, kind, drafted):
    s = _case([4, 2, 5], V, kind, drafted, pad=pad, offset=offset)
    _check(s, _run(s), 0.5)


@pytest.mark.parametrize("drafted", [False, True])
def test_256_lanes(drafted):
    s = _case([1 + n % 6 for n in range(256)], 501, "f32", drafted)
    _check(s, _run(s), 0.95)


@pytest.mark.parametrize("drafted", [False, True])
def test_every_prefix_and_token(drafted):
    """Uniforms that make exactly the first k drafts stand, and a sweep of the
    last one over the whole vocabulary."""
    T, V = 6, 50
    s = _case([T] * T, V, "f32", drafted, right=1.0)
    s["it"].fill_(1.0)
    s["uniforms"].fill_(0.0)
    for k in range(T):
        if k < T - 1:
            s["uniforms"][k, k] = 1.0 - 2.0 ** -24
            s["tokens"][k, k + 1] = (s["tokens"][k, k + 1] + 1) % V
    for u in torch.linspace(0, 1 - 2.0 ** -24, 41).tolist():
        s["uniforms"][:, T - 1] = u
        got = _run(s)
        assert got[0] == list(range(1, T + 1)) if not drafted else True
        _check(s, got, 0.3)


@pytest.mark.parametrize("drafted", [False, True])
def test_tokens_come_out_as_the_model_has_them(drafted):
    """The law that the procedure is for, on a grid of uniforms: the token
    after the anchor is distributed as p, whatever the drafter's q.  Midpoints
    of 16 x 16 cells: the accepted share and the look-up are each off by at
    most half a cell for every draft."""
    V, G = 5, 16
    logits = torch.tensor([0.3, 1.0, -0.5, 0.9, -2.0])
    draft = torch.tensor([1.0, -0.3, 0.2, 0.9, -1.0])
    p, q = torch.softmax(logits, 0), torch.softmax(draft, 0)
    u = (torch.arange(G) + 0.5) / G
    first = torch.zeros(V, dtype=torch.float64)
    for w in range(V):
        s = dict(t_lane=[2] * 256, logits=logits.expand(256, 2, V).contiguous().cuda(),
                 draft=draft.expand(256, 1, V).contiguous().cuda() if drafted else None,
                 tokens=torch.full((256, 2), w, dtype=torch.int32, device="cuda"),
                 uniforms=torch.cartesian_prod(u, u).cuda(), it=torch.ones(256, device="cuda"))
        m, token, _ = _run(s)
        for a, b in zip(m, token):
            first[w if a == 2 else b] += (float(q[w]) if drafted else 1 / V) / 256
    if not drafted:      # drafts that are given: any law of theirs is left
        q = torch.full((V,), 1 / V)
    assert ((first - p.double()).abs() <= 2 * (0.5 / G) + 1e-6).all()


def test_sampling_follows_the_running_sum():
    """Windows of the anchor alone: u over a grid gives every token its
    share, ids in order."""
    V, n = 7, 256
    logits = torch.tensor([0.0, 2.0, -1.0, -math.inf, 1.0, -3.0, 0.5])
    p = torch.softmax(logits.double(), 0)
    s = dict(t_lane=[1] * n, logits=logits.expand(n, 1, V).contiguous().cuda(), draft=None,
             tokens=torch.zeros(n, 1, dtype=torch.int32, device="cuda"),
             uniforms=((torch.arange(n) + 0.5) / n)[:, None].contiguous().cuda(), it=torch.ones(n, device="cuda"))
    m, token, _ = _run(s)
    assert m == [1] * n and token == sorted(token) and 3 not in token
    for i in range(V):
        assert abs(token.count(i) / n - float(p[i])) <= 1.0 / n


@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("V", [50, 20000])
def test_masked_logits(V, drafted):
    """-inf in most places, drafts on masked tokens, a row with one token."""
    s = _case([5, 4, 5], V, "f32", drafted, right=0.7)
    out = torch.rand(3, 5, V, device="cuda") < 0.9
    out[..., 3] = False
    s["logits"].masked_fill_(out, -math.inf)
    s["logits"][1, 1] = -math.inf
    s["logits"][1, 1, V - 1] = -4.0
    s["tokens"][1, 2] = V - 1
    if drafted:
        s["draft"].masked_fill_(out[:, :-1] & (torch.rand(3, 4, V, device="cuda") < 0.5), -math.inf)
        s["draft"][1, 1, V - 1] = 2.0
    _check(s, _run(s), 0.3)


@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("V", [30, 9000])
def test_rows_without_a_distribution(V, drafted):
    s = _case([4] * 8, V, "f32", drafted, right=1.0)
    s["uniforms"][:, :-1] = 0.0
    s["logits"][0, 1, V // 2] = math.nan
    s["logits"][1, 2, V - 1] = math.inf
    s["logits"][2, 0] = -math.inf
    s["logits"][3, 3, 0] = math.nan                # the last row
    s["logits"][5, 1, 0] = -math.nan
    if drafted:
        s["draft"][4, 1, 5] = math.nan
        s["draft"][6, 0] = -math.inf
    got = _run(s)
    assert got[0][:4] == [2, 3, 1, 4] and got[1][:4] == [-1] * 4 and got[0][5] == 2
    if drafted:
        assert (got[0][4], got[1][4], got[0][6], got[1][6]) == (2, -1, 1, -1)
    _check(s, got, 0.5)


def test_inverse_temperatures():
    s = _case([3] * 9, 400, "f32", True)
    s["it"].copy_(torch.tensor([0.0, -1.0, math.nan, math.inf, 1e-31, 1e31, 1e-30, 1e30, 40.0]))
    got = _run(s)
    assert got[0][:6] == [1] * 6 and got[1][:6] == [-1] * 6
    assert torch.isnan(got[2][:6, :2]).all()
    _check(s, got, 0.5)


def test_logits_far_apart():
    """The lowest and largest values of the types beside others."""
    for kind, big in (("f32", 3.4e38), ("bf16", 3.38e38)):
        s = _case([3, 2], 3000, kind, True)
        s["logits"][:, :, ::7] = -big
        s["draft"][:, :, ::5] = -big
        s["logits"][1, 0, 1] = big
        _check(s, _run(s), 0.5)


@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_greedy_limit_beside_masked_logits(kind, drafted):
    """Inverse temperatures that leave one token, and -inf beside it: the
    drafts that are it stand, the next one is it."""
    s = _case([4, 3, 4, 2], 9000, kind, drafted, right=1.0)
    out = torch.rand(4, 4, 9000, device="cuda") < 0.5
    best = s["logits"].float().argmax(2, keepdim=True)
    out.scatter_(2, best, False)
    s["logits"].masked_fill_(out, -math.inf)
    if drafted:
        s["draft"].masked_fill_(out[:, :-1], -math.inf)
        s["draft"].scatter_(2, best[:, :-1], 200.0)
    s["logits"].scatter_(2, best, 100.0)
    s["it"].copy_(torch.tensor([1e3, 1e8, 1e12, 1e30]))
    got = _run(s)
    assert got[0] == s["t_lane"]
    assert got[1] == [int(best[n, m - 1]) for n, m in enumerate(got[0])]
    _check(s, got, 0.5)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_a_draft_that_is_all_there_is(kind):
    """The one token with any probability, drafted: with a uniform of 1 it
    falls and is sampled again."""
    s = _case([2, 2], 5000, kind, False)
    s["logits"].fill_(-math.inf)
    s["logits"][:, :, 77] = 1.0
    s["tokens"][:, 1] = 77
    s["uniforms"][0, 0], s["uniforms"][1, 0] = 1.0, 0.99
    m, token, accept = _run(s)
    assert (m, token) == ([1, 2], [77, 77]) and (accept[:, 0] == 1).all()


@pytest.mark.parametrize("drafted", [False, True])
def test_drafts_outside_the_vocabulary_fall(drafted):
    s = _case([4, 4, 4], 90, "f32", drafted, right=1.0)
    s["uniforms"][:, :-1] = 0.0
    s["tokens"][:, 2] = torch.tensor([90, -1, -2**31], dtype=torch.int32)
    s["tokens"][:, 0] = 2**31 - 1                  # anchors are not read
    got = _run(s)
    assert got[0] == [2, 2, 2]
    _check(s, got, 0.5)


def test_uniforms_outside_their_range():
    s = _case([2, 2, 2, 2, 1, 1], 60, "f32", False, right=1.0)
    s["uniforms"].copy_(torch.tensor([[1.0, 0.5], [math.nan, 0.5], [-1.0, 2.0], [0.0, -3.0], [1.0, 0], [math.nan, 0]]))
    got = _run(s)
    assert got[0][:4] == [1, 1, 2, 2]
    rows = s["logits"].double().cpu()
    last = lambda p: int(torch.nonzero(p > 0)[-1])
    assert got[1][2] == last(torch.softmax(rows[2, 1] * float(s["it"][2]), 0))
    assert got[1][3] == 0 and got[1][5] == 0
    assert got[1][4] == last(torch.softmax(rows[4, 0] * float(s["it"][4]), 0))


def test_equal_distributions_always_stand():
    s = _case([9] * 5, 700, "bf16", True, right=0.3)
    s["draft"].copy_(s["logits"][:, :-1])
    s["uniforms"].fill_(1.0 - 2.0 ** -12)
    got = _run(s)
    assert got[0] == [9] * 5
    _check(s, got, 0.5)


def test_the_same_call_gives_the_same_bits_alone_or_in_a_batch():
    s = _case([5, 3, 6], 40000, "f32", True)
    a = _run(s)
    for _ in range(2):
        b = _run(s)
        assert a[:2] == b[:2] and torch.equal(a[2], b[2])
    for n in range(3):
        one = dict(s, t_lane=[s["t_lane"][n]], **{c: s[c][n:n + 1].contiguous() for c in
                                                  ("logits", "draft", "tokens", "uniforms", "it")})
        b = _run(one)
        assert b[0] == a[0][n:n + 1] and b[1] == a[1][n:n + 1]


def test_rows_past_31_bits():
    """Logits whose last rows lie past 2^31 elements."""
    T, V = 9, 262144
    n = (1 << 31) // (T * V) + 2
    t_lane = [0] * n
    big = torch.empty(n, T, V, dtype=torch.bfloat16, device="cuda")
    assert n <= 1024
    if n > gdn.GDN_MAX_LANES:
        n = gdn.GDN_MAX_LANES
        T = (1 << 31) // (n * V) + 1
        del big
        big = torch.empty(n, T, V, dtype=torch.bfloat16, device="cuda")
        t_lane = [0] * n
    small = _case([min(T, 4)], V, "bf16", False, T=T)
    big[n - 1] = small["logits"][0]
    t_lane[n - 1] = min(T, 4)
    s = dict(t_lane=t_lane, logits=big, draft=None,
             tokens=small["tokens"].repeat(n, 1), uniforms=small["uniforms"].repeat(n, 1), it=small["it"].repeat(n))
    m, token, accept = _run(s)
    b = _run(small)
    assert (m[-1], token[-1]) == (b[0][0], b[1][0]) and m[:-1] == [-9] * (n - 1)


def test_another_stream_and_graph():
    s = _case([4, 2], 30000, "f32", True)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    a = _run(s, stream=stream)
    b = _run(s)
    assert a[:2] == b[:2]
    m, token = (torch.empty(2, dtype=torch.int32, device="cuda") for _ in range(2))
    accept = torch.zeros(2, 4, device="cuda")
    ws = torch.empty(gdn.draft_verify_workspace_bytes(2, 4, 30000), dtype=torch.uint8, device="cuda")

    def call():
        gdn.draft_verify([4, 2], s["logits"], s["draft"], s["tokens"], s["uniforms"], s["it"], m, token, ws,
                         accept=accept)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (5, 6, 7):
        other = _case([4, 2], 30000, "f32", True, seed=seed)
        for c in ("logits", "draft", "tokens", "uniforms", "it"):
            s[c].copy_(other[c])
        ws.fill_(seed)
        graph.replay()
        torch.cuda.synchronize()
        got = (m.tolist(), token.tolist())
        assert got == _run(s)[:2]

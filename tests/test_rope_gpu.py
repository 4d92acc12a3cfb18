"""gdn_rope_append and gdn_rope_append_mxfp against the rotation in 64 bits and
the 4-bit format's definition."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import commit_gated_delta_amd as gdn  # noqa: E402
from tests import cache_ref as ref  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# half a step of the outputs' type, relative
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _case(t_lane, lens, h_q, h_kv, d, page, kind, rot, T=None, seed=0, fused=True, extra=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    N, T, t = len(lens), T or max(max(t_lane), 1), TYPES[kind]
    cols = max(1, max(-(-max(n, 0) // page) for n in lens)) + extra
    pages = N * cols + 3
    randn = lambda *s: torch.randn(s, device="cuda", generator=g).to(t)
    x = dict(dims=gdn.KvDims.of(N, T, h_q, h_kv, d, page, pages, cols), rot=rot, kind=kind,
             t_lane=t_lane, lens=lens)
    if fused:
        rows = randn(N, T, (h_q + 2 * h_kv) * d)
        q, k, v = torch.split(rows, [h_q * d, h_kv * d, h_kv * d], 2)
        x["q"], x["k"], x["v"] = q.view(N, T, h_q, d), k.view(N, T, h_kv, d), v.view(N, T, h_kv, d)
    else:
        x["q"], x["k"], x["v"] = randn(N, T, h_q, d), randn(N, T, h_kv, d), randn(N, T, h_kv, d)
    x["inv_freq"] = (1e4 ** (-torch.arange(rot // 2, device="cuda").double() * 2 / max(rot, 1))).float()
    x["table"] = torch.randperm(pages, device="cuda", generator=g)[:N * cols].view(N, cols).int()
    x["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for c in "kv":
        x[c + "_cache"] = randn(pages, h_kv, page, d)
        x[c + "_codes"] = torch.randint(256, (pages, h_kv, page, d // 2), device="cuda", generator=g, dtype=torch.uint8)
        x[c + "_scales"] = torch.randint(100, 140, (pages, h_kv, page, d // 32), device="cuda", generator=g, dtype=torch.uint8)
    return x


def _positions(x, given=None):
    if given is not None:
        return given.cpu()
    n, T = x["dims"].n_lanes, x["dims"].t_max
    at = torch.arange(T)[None].repeat(n, 1)
    return at + (x["kv_len"].cpu().long() - torch.tensor(x["t_lane"]))[:, None]


def _places(x):
    """(lane, token, page, row) of the new rows that have a place."""
    page, table = x["dims"].page_size, x["table"].cpu()
    cap = x["dims"].max_pages * page
    for n, m in enumerate(x["t_lane"]):
        for t in range(m):
            pos = int(x["kv_len"][n]) - m + t
            if 0 <= pos < cap:
                p = int(table[n, pos // page])
                if 0 <= p < x["dims"].n_pages:
                    yield n, t, p, pos % page


def _run(x, pairs=False, positions=None, q=True, inplace=False, stream=None):
    d = x["dims"]
    shape = (d.n_lanes, d.t_max, d.h_q, d.d)
    q_out = None
    if q:
        q_out = x["q"] if inplace else torch.full(shape, 7.0, device="cuda", dtype=TYPES[x["kind"]])
    gdn.rope_append(d, x["t_lane"], x["q"] if q else None, x["k"], x["v"],
                    x["inv_freq"] if x["rot"] else None, x["rot"], q_out, x["k_cache"], x["v_cache"],
                    x["table"], x["kv_len"], positions=positions, interleaved=pairs, stream=stream)
    return q_out


def _run4(x, pairs=False, positions=None, q=True, held=True):
    d = x["dims"]
    q_out = torch.full((d.n_lanes, d.t_max, d.h_q, d.d), 7.0, device="cuda", dtype=TYPES[x["kind"]]) if q else None
    k, v = (torch.full((d.n_lanes, d.t_max, d.h_kv, d.d), 7.0, device="cuda", dtype=torch.bfloat16)
            if held else None for _ in range(2))
    gdn.rope_append_mxfp(d, x["t_lane"], x["q"] if q else None, x["k"], x["v"],
                         x["inv_freq"] if x["rot"] else None, x["rot"], q_out, x["k_codes"], x["k_scales"],
                         x["v_codes"], x["v_scales"], x["table"], x["kv_len"], k_held=k, v_held=v,
                         positions=positions, interleaved=pairs)
    return q_out, k, v


def _check_q(x, q, got, pairs, pos):
    want, tol = ref.turned(q, pos, x["inv_freq"], x["rot"], pairs)
    got = got.double().cpu()
    for n, m in enumerate(x["t_lane"]):
        err = (got[n, :m] - want[n, :m]).abs()
        lim = tol[n, :m] * 1.01 + HALF[x["kind"]] * want[n, :m].abs()
        assert (err <= lim).all(), n
        assert (got[n, m:] == 7).all()
        rot = x["rot"]
        assert torch.equal(got[n, :m, :, rot:], q.double().cpu()[n, :m, :, rot:])


def _check(x, before, q, pairs, pos):
    """The caches: the new rows turned, the values as they are, the rest
    untouched."""
    want, tol = ref.turned(x["k"], pos, x["inv_freq"], x["rot"], pairs)
    left = {c: b.clone() for c, b in before.items()}
    for n, t, p, r in _places(x):
        got = x["k_cache"][p, :, r].double().cpu()
        assert ((got - want[n, t]).abs() <= tol[n, t] * 1.01 + HALF[x["kind"]] * want[n, t].abs()).all(), (n, t)
        left["k_cache"][p, :, r] = x["k_cache"][p, :, r]
        left["v_cache"][p, :, r] = x["v"][n, t]
    assert torch.equal(x["k_cache"], left["k_cache"])
    assert torch.equal(x["v_cache"], left["v_cache"])


def _check4(x, before, out, pairs, pos):
    q, k, v = out
    want, tol = ref.turned(x["k"], pos, x["inv_freq"], x["rot"], pairs)
    codes, scales = ref.encode(x["v"].double())
    left = {c: b.clone() for c, b in before.items()}
    for n, t, p, r in _places(x):
        a, b = x["k_codes"][p, :, r], x["k_scales"][p, :, r]
        assert ref.held_ok(want[n, t], tol[n, t] * 1.01, a, b), (n, t)
        if k is not None:
            assert torch.equal(k[n, t].double().cpu(), ref.decode(a, b))
            assert torch.equal(v[n, t].double().cpu(), ref.decode(codes[n, t], scales[n, t]))
        left["k_codes"][p, :, r], left["k_scales"][p, :, r] = a, b
        left["v_codes"][p, :, r], left["v_scales"][p, :, r] = codes[n, t].cuda(), scales[n, t].cuda()
    for c in left:
        assert torch.equal(x[c], left[c]), c
    if k is not None:
        for n, m in enumerate(x["t_lane"]):
            assert (k[n, m:] == 7).all() and (v[n, m:] == 7).all()


def _before(x, names):
    return {c: x[c].clone() for c in names}


ROWS, BITS = ("k_cache", "v_cache"), ("k_codes", "k_scales", "v_codes", "v_scales")

CASES = [
    # t_lane, lens, h_q, h_kv, d, page, kind, rot, pairs
    ([1], [1], 1, 1, 64, 1, "bf16", 64, False),
    ([1, 1, 1], [5, 17, 300], 8, 2, 128, 16, "bf16", 128, False),
    ([1, 0, 1], [33, 50, 64], 4, 4, 64, 7, "bf16", 32, True),
    ([3, 0, 5], [20, 9, 5], 6, 2, 128, 8, "bf16", 16, False),
    ([7, 2], [70, 31], 16, 1, 256, 24, "bf16", 64, False),
    ([64, 1], [64, 100], 5, 5, 64, 10, "bf16", 48, False),
    ([2, 4], [2, 9], 3, 3, 256, 4, "bf16", 256, True),
    ([4, 4], [2, 0], 4, 2, 64, 16, "bf16", 64, False),     # rows before position 0
    ([1, 1, 1], [5, 17, 300], 8, 2, 128, 16, "f32", 128, False),
    ([6, 2], [100, 2], 4, 2, 64, 5, "f32", 48, True),
    ([16], [200], 15, 3, 256, 16, "f32", 96, False),
    ([5, 1], [40, 7], 4, 2, 128, 16, "f32", 0, False),      # nothing turns
    ([5, 1], [40, 7], 4, 2, 128, 16, "bf16", 0, True),
]


@pytest.mark.parametrize("t_lane,lens,h_q,h_kv,d,page,kind,rot,pairs", CASES)
@pytest.mark.parametrize("fused", [True, False])
def test_append(t_lane, lens, h_q, h_kv, d, page, kind, rot, pairs, fused):
    x = _case(t_lane, lens, h_q, h_kv, d, page, kind, rot, fused=fused)
    before = _before(x, ROWS)
    pos = _positions(x)
    q = _run(x, pairs)
    _check_q(x, x["q"], q, pairs, pos)
    _check(x, before, q, pairs, pos)


@pytest.mark.parametrize("t_lane,lens,h_q,h_kv,d,page,kind,rot,pairs", CASES)
def test_append_in_four_bits(t_lane, lens, h_q, h_kv, d, page, kind, rot, pairs):
    x = _case(t_lane, lens, h_q, h_kv, d, page, kind, rot)
    before = _before(x, BITS)
    pos = _positions(x)
    out = _run4(x, pairs)
    _check_q(x, x["q"], out[0], pairs, pos)
    _check4(x, before, out, pairs, pos)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("lanes,T,h_q,h_kv,d,rot", [(40, 64, 16, 4, 128, 128), (96, 33, 20, 4, 64, 64),
                                                  (9, 64, 8, 8, 256, 64)])
def test_many_rows(lanes, T, h_q, h_kv, d, rot, kind):
    """Prompts in windows, ragged; q checked, and a few lanes' caches."""
    t_lane = [1 + (7 * n) % T for n in range(lanes)]
    t_lane[1] = T
    x = _case(t_lane, [T + 3 * n for n in range(lanes)], h_q, h_kv, d, 16, kind, rot, T=T)
    before = _before(x, ROWS + BITS)
    pos = _positions(x)
    q = _run(x)
    _check_q(x, x["q"], q, False, pos)
    out = _run4(x)
    assert torch.equal(out[0], q)
    _check(x, {c: before[c] for c in ROWS}, q, False, pos)
    _check4(x, {c: before[c] for c in BITS}, out, False, pos)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_given_and_far_positions(kind, pairs):
    """Positions up to the largest int and negative ones; the places do not
    follow them."""
    x = _case([4, 3], [40, 20], 6, 2, 128, 16, kind, 128)
    given = torch.tensor([[0, 2**31 - 1, -5, 1234567], [2**30, -2**31, 77, 3]], dtype=torch.int32, device="cuda")
    before = _before(x, ROWS + BITS)
    pos = _positions(x, given)
    q = _run(x, pairs, given)
    _check_q(x, x["q"], q, pairs, pos)
    _check(x, {c: before[c] for c in ROWS}, q, pairs, pos)
    _check4(x, {c: before[c] for c in BITS}, _run4(x, pairs, given), pairs, pos)


def test_zero_position_turns_nothing():
    x = _case([1], [1], 4, 2, 64, 16, "f32", 64)
    q = _run(x)
    assert torch.equal(q, x["q"])
    assert torch.equal(x["k_cache"][int(x["table"][0, 0]), :, 0], x["k"][0, 0])


def test_a_rotation_keeps_lengths_and_relative_angles():
    """Without the reference: |q| stays, and q . k depends on the distance."""
    x = _case([2], [1000], 2, 2, 128, 16, "f32", 128, fused=False)
    dots = []
    for p in (0, 5, 100000):
        given = torch.tensor([[p + 3, p]], dtype=torch.int32, device="cuda")
        x["q"][0, 1], x["k"][0, 0] = x["q"][0, 0], x["k"][0, 1]
        q = _run(x, positions=given).double()
        assert torch.allclose(q.norm(dim=-1), x["q"].double().norm(dim=-1), rtol=128 * 12 * 2.0 ** -24)
        dims = x["dims"]
        at = 1000 - 2 + 1
        k = x["k_cache"][int(x["table"][0, at // dims.page_size]), :, at % dims.page_size].double()
        dots.append((q[0, 0] * k).sum(-1))
    size = (x["q"][0, 0].double().abs().sum(-1) * x["k"].double().abs().max())
    for d in dots[1:]:
        assert ((d - dots[0]).abs() <= 4 * 12 * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("kind,pairs", [("bf16", False), ("bf16", True), ("f32", False), ("f32", True)])
def test_queries_in_place(kind, pairs):
    x = _case([5, 64], [40, 90], 7, 1, 128, 16, kind, 96, T=64, fused=False)
    want = _run(x, pairs).clone()
    q = x["q"].clone()
    got = _run(x, pairs, inplace=True)
    for n, m in enumerate(x["t_lane"]):
        assert torch.equal(got[n, :m], want[n, :m])
        assert torch.equal(got[n, m:], q[n, m:])


def test_keys_alone():
    x = _case([3, 1], [30, 7], 4, 2, 128, 16, "bf16", 64)
    before = _before(x, ROWS + BITS)
    pos = _positions(x)
    assert _run(x, q=False) is None
    _check(x, {c: before[c] for c in ROWS}, None, False, pos)
    _check4(x, {c: before[c] for c in BITS}, _run4(x, q=False, held=False), False, pos)


def test_rows_without_a_place_are_dropped_but_turned():
    x = _case([4] * 5, [10] * 5, 2, 2, 64, 8, "bf16", 64)
    cap = x["dims"].max_pages * 8
    x["kv_len"].copy_(torch.tensor([cap + 2, 1, 2**31 - 1, -2**31 + 3, 10], dtype=torch.int32))
    x["table"][4, 0], x["table"][4, 1] = x["dims"].n_pages, -1
    given = torch.arange(20, dtype=torch.int32, device="cuda").view(5, 4)
    before = _before(x, ROWS + BITS)
    pos = _positions(x, given)
    q = _run(x, positions=given)
    _check_q(x, x["q"], q, False, pos)
    _check(x, {c: before[c] for c in ROWS}, q, False, pos)
    out = _run4(x, positions=given)
    _check4(x, {c: before[c] for c in BITS}, out, False, pos)
    want, tol = ref.turned(x["k"], pos, x["inv_freq"], 64, False)
    for n in range(5):    # held rows of dropped tokens too
        got = out[1][n].double().cpu()
        assert ((got - want[n]).abs() <= tol[n] + want[n].abs().unflatten(-1, (-1, 32)).amax(-1).repeat_interleave(32, -1) / 3).all()


def test_every_code_and_border():
    """Values on and beside every border between codes, at several scales:
    ties to even, signs, zeros of both signs; largest values that sit on and
    beside the scale's border."""
    borders = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    vals = [0.0, -0.0, 6.0, -6.0]
    for b in borders:
        for y in (b, math.nextafter(b, 0), math.nextafter(b, 9)):
            y32 = float(torch.tensor(y, dtype=torch.float32))
            vals += [y32, -y32, b + 2.0 ** -20, b - 2.0 ** -20]
    rows = []
    for e in (-100, -20, -1, 0, 3, 90):
        for top in (6.0, 3.0 + 2.0 ** -21, 4.0, 5.9):
            v = [top] + vals
            for i in range(0, len(v), 31):
                r = [top] + v[i:i + 31]
                rows.append([x * 2.0 ** e for x in r + [0.0] * (32 - len(r))])
    for e in (-126, -100, 0, 60, 126):        # borders of the scale itself
        for f in (1.5, 1.5 + 2.0 ** -22, 1.0, 2.0 - 2.0 ** -23):
            rows.append([f * 2.0 ** e] + [0.3 * f * 2.0 ** e] * 31)
    rows.append([0.0] * 32)
    rows.append([1e-45, -1e-45] + [0.0] * 30)
    rows += [[0.0] * 32] * (-len(rows) % 4)
    x32 = torch.tensor(rows, dtype=torch.float64).float().view(-1, 1, 1, 128)
    n = x32.shape[0]
    x = _case([1] * n, [1] * n, 1, 1, 128, 1, "f32", 0, fused=False)
    x["k"].copy_(x32)
    x["v"].copy_(x32)
    _run4(x)
    codes, scales = ref.encode(x32.double())
    for i, t, p, r in _places(x):
        for c in "kv":
            assert torch.equal(x[c + "_scales"][p, :, r].cpu(), scales[i, 0]), i
            assert torch.equal(x[c + "_codes"][p, :, r].cpu(), codes[i, 0]), i


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_turned_keys_are_rounded_once(kind, pairs):
    """Four million turned keys come out as the nearest codes of the keys in 64
    bits, every one: keys off by 2^-24 of their size would give about one in a
    million the neighbouring code.  (The kernel's sines and the reference's are
    2e-14 apart, which would do that to one in 10^13.)"""
    x = _case([64] * 64, [64] * 64, 8, 8, 128, 16, kind, 128)
    given = torch.randint(0, 1 << 20, (64, 64), dtype=torch.int32, device="cuda")
    _, k, _ = _run4(x, pairs, given)
    want, _ = ref.turned(x["k"], _positions(x, given), x["inv_freq"], 128, pairs)
    assert torch.equal(k.double().cpu(), ref.decode(*ref.encode(want)))


def test_values_past_the_largest_scale_and_non_finite_blocks():
    x = _case([1], [1], 1, 1, 128, 1, "f32", 0, fused=False)
    big = 6 * 2.0 ** 124
    row = torch.randn(128)
    row[0], row[1], row[2] = 3.4e38, -3.0e38, big / 2
    row[40] = math.inf
    row[70] = math.nan
    row[100] = -math.inf
    x["k"][0, 0, 0] = row
    x["v"][0, 0, 0] = row
    _, k, v = _run4(x)
    for h in (k, v):
        h = h[0, 0, 0].double().cpu()
        assert h[0] == big and h[1] == -big and h[2] == big / 2
        assert torch.isnan(h[32:]).all()
    p = int(x["table"][0, 0])
    for c in "kv":
        assert x[c + "_scales"][p, 0, 0].tolist() == [251, 255, 255, 255]
        assert (x[c + "_codes"][p, 0, 0, 16:] == 0).all()


def test_non_finite_channels_stay_in_their_pair():
    x = _case([1], [9], 2, 2, 64, 16, "f32", 32, fused=False)
    x["q"][0, 0, 0, 3], x["k"][0, 0, 1, 40] = math.nan, math.inf
    q = _run(x)
    want = torch.zeros(64, dtype=torch.bool)
    want[3] = want[19] = True
    assert torch.equal(torch.isnan(q[0, 0, 0]).cpu(), want)
    assert torch.isfinite(q[0, 0, 1]).all()
    k = x["k_cache"][int(x["table"][0, 0]), :, 8]
    assert k[1, 40] == math.inf and torch.isfinite(k[0]).all() and int(torch.isfinite(k[1]).sum()) == 63


def test_another_stream_and_graph():
    """Captured once, replayed on other lengths, rows and tables, with eager
    work between the replays."""
    x = _case([2, 1], [40, 20], 4, 2, 128, 16, "bf16", 64, T=2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = _run(x)
    s.synchronize()
    b = _run(x)
    assert torch.equal(a, b)
    q_out = torch.full_like(a, 7.0)
    k, v = (torch.empty(2, 2, 2, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))

    def call():
        gdn.rope_append_mxfp(x["dims"], [2, 1], x["q"], x["k"], x["v"], x["inv_freq"], 64, q_out,
                             x["k_codes"], x["k_scales"], x["v_codes"], x["v_scales"], x["table"],
                             x["kv_len"], k_held=k, v_held=v)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([41, 21], [7, 48], [2, 1]):
        x["kv_len"].copy_(torch.tensor(lens, dtype=torch.int32))
        x["k"].copy_(torch.randn(2, 2, 2, 128, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (q_out, k, v, x["k_codes"], x["k_scales"], x["v_codes"], x["v_scales"])]
        call()
        torch.cuda.synchronize()
        now = (q_out, k, v, x["k_codes"], x["k_scales"], x["v_codes"], x["v_scales"])
        for g, w in zip(got, now):      # (held rows of the idle token are left as they were)
            assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))
        _check_q(x, x["q"], q_out, False, _positions(x))


def test_caches_longer_than_32_bits():
    page, h_kv, d = 256, 8, 256
    pages = (1 << 33) // (page * h_kv * d) + 40       # codes past 2^32 bytes
    at = [pages - 1, 3, pages - 30]
    codes = [torch.empty(pages, h_kv, page, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.empty(pages, h_kv, page, d // 32, dtype=torch.uint8, device="cuda") for _ in range(2)]
    x = _case([1], [700], 8, h_kv, d, page, "bf16", 64, fused=False)
    dims = gdn.KvDims.of(1, 1, 8, h_kv, d, page, pages, 3)
    table = torch.tensor([at], dtype=torch.int32, device="cuda")
    q_out = torch.empty_like(x["q"])
    k, v = (torch.empty(1, 1, h_kv, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    gdn.rope_append_mxfp(dims, [1], x["q"], x["k"], x["v"], x["inv_freq"], 64, q_out, codes[0], scales[0],
                         codes[1], scales[1], table, x["kv_len"], k_held=k, v_held=v)
    for c, s, held in zip(codes, scales, (k, v)):
        r = 699 - 512
        assert torch.equal(ref.decode(c[at[2], :, r], s[at[2], :, r]), held[0, 0].double().cpu())

"""gdn_paged_attention and gdn_kv_append against attention in 64 bits over
the gathered pages."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import commit_gated_delta_amd as gdn  # noqa: E402
from tests import serving_ref as ref  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _case(t_lane, lens, h_q, h_kv, d, page, kind, T=None, seed=0, extra=2):
    """Random pages; rows behind each lane's length and unused pages hold
    NaN, table entries behind it page numbers outside the cache."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    N, T, t = len(lens), T or max(max(t_lane), 1), TYPES[kind]
    cols = max(1, max(-(-max(n, 0) // page) for n in lens)) + extra
    pages = N * cols + 3
    randn = lambda *s: torch.randn(s, device="cuda", generator=g).to(t)
    x = dict(q=randn(N, T, h_q, d), k=randn(pages, h_kv, page, d),
             v=randn(pages, h_kv, page, d))
    order = torch.randperm(pages, device="cuda", generator=g)[:N * cols].view(N, cols)
    used = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    table = torch.full((N, cols), -1, dtype=torch.int32, device="cuda")
    table[:, 1::2] = 1 << 30
    for n, length in enumerate(lens):
        for j in range(-(-max(length, 0) // page)):
            table[n, j] = order[n, j]
            used[order[n, j], : min(page, length - j * page)] = True
    for c in ("k", "v"):
        x[c].masked_fill_(~used[:, None, :, None], math.nan)
    x["table"] = table
    x["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    x["dims"] = gdn.KvDims.of(N, T, h_q, h_kv, d, page, pages, cols)
    return x


def _run(x, t_lane, scale):
    o = torch.full(x["q"].shape, 7.0, device="cuda")
    ws = torch.empty(gdn.paged_attention_workspace_bytes(x["dims"]),
                     dtype=torch.uint8, device="cuda")
    gdn.paged_attention(x["dims"], t_lane, x["q"], x["k"], x["v"], x["table"],
                        x["kv_len"], o, ws, scale=scale)
    torch.cuda.synchronize()
    return o


def _check(x, t_lane, o, scale):
    want, tol = ref.attend(x["q"], x["k"], x["v"], x["table"], x["kv_len"],
                           t_lane, scale)
    o = o.cpu().double()
    for n, m in enumerate(t_lane):
        assert (o[n, m:] == 7).all()
        if m == 0:
            continue
        assert torch.isfinite(o[n, :m]).all(), n
        worst = float(((o[n, :m] - want[n, :m]).abs() / tol[n, :m]).max())
        print("lane %d: %.3g of its bound" % (n, worst), flush=True)
        assert worst <= 1, (n, worst)


@pytest.mark.parametrize("t_lane,lens,h_q,h_kv,d,page,kind", [
    ([1], [1], 1, 1, 64, 1, "bf16"),
    ([1, 1, 1], [1, 17, 300], 8, 2, 128, 16, "bf16"),
    ([1, 0, 1], [33, 50, 64], 4, 4, 64, 7, "bf16"),
    ([1, 1], [0, 5], 4, 2, 128, 8, "bf16"),            # nothing to see
    ([1, 1], [700, 31], 16, 1, 256, 24, "bf16"),
    ([1], [5000], 32, 2, 128, 64, "bf16"),
    ([4, 7, 0, 1], [40, 7, 9, 129], 6, 2, 128, 16, "bf16"),
    ([16, 3], [500, 700], 8, 1, 128, 32, "bf16"),
    ([64], [64], 5, 5, 64, 10, "bf16"),
    ([33, 64], [200, 65], 20, 2, 128, 256, "bf16"),
    ([16], [300], 16, 2, 256, 16, "bf16"),
    ([5], [3], 2, 1, 64, 4, "bf16"),                   # more tokens than rows
    ([1, 1, 1], [1, 17, 300], 8, 2, 128, 16, "f32"),
    ([6, 2], [100, 2], 4, 2, 64, 5, "f32"),
    ([16], [200], 16, 2, 256, 16, "f32"),
    ([1], [2049], 40, 1, 128, 128, "f32"),
])
def test_attention(t_lane, lens, h_q, h_kv, d, page, kind):
    x = _case(t_lane, lens, h_q, h_kv, d, page, kind)
    _check(x, t_lane, _run(x, t_lane, d ** -0.5), d ** -0.5)


@pytest.mark.parametrize("t_lane,lens,h_q,h_kv,d,kind", [
    ([1], [20001], 2, 1, 64, "bf16"),                  # many splits of few rows
    ([1, 2], [15000, 9], 3, 1, 128, "f32"),
    ([1], [12345], 1, 1, 256, "bf16"),
    ([1] * 40, [20000] + [30] * 39, 32, 1, 64, "bf16"),  # and of many rows
    ([1] * 18, [200] * 17 + [9000], 64, 2, 128, "bf16"),
])
def test_many_splits(t_lane, lens, h_q, h_kv, d, kind):
    x = _case(t_lane, lens, h_q, h_kv, d, 64, kind)
    x["q"][0, 0, 0] *= 4                               # weights far apart
    _check(x, t_lane, _run(x, t_lane, d ** -0.5), d ** -0.5)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_peaked_scores(kind):
    """Scores far apart: one position takes nearly everything, in any tile."""
    x = _case([2, 2], [900, 70], 4, 2, 128, 16, kind)
    x["q"].mul_(6)
    _check(x, [2, 2], _run(x, [2, 2], 0.3), 0.3)


def test_negative_and_zero_scale():
    x = _case([1, 2], [90, 30], 4, 2, 64, 16, "bf16")
    for scale in (-0.2, 0.0):
        _check(x, [1, 2], _run(x, [1, 2], scale), scale)


def test_lengths_outside_the_table_are_cut():
    x = _case([1, 2, 1], [40, 48, 20], 4, 2, 64, 16, "bf16", extra=0)
    x["kv_len"].copy_(torch.tensor([1 << 30, 48, -5], dtype=torch.int32))
    x["k"].nan_to_num_(0.5)
    x["v"].nan_to_num_(0.25)
    o = _run(x, [1, 2, 1], 0.1)
    _check(x, [1, 2, 1], o, 0.1)
    assert (o[2, 0] == 0).all()


def test_bad_page_numbers_are_masked():
    x = _case([1, 3], [200, 90], 4, 2, 128, 16, "bf16")
    x["table"][0, 2] = -7
    x["table"][0, 12] = x["dims"].n_pages
    x["table"][1, :] = -1                               # a lane with no page
    o = _run(x, [1, 3], 0.1)
    _check(x, [1, 3], o, 0.1)
    assert (o[1, :3] == 0).all()


@pytest.mark.parametrize("T,h_q,d,kind", [(4, 4, 128, "bf16"), (16, 16, 128, "bf16"),
                                          (3, 2, 64, "f32"), (40, 2, 256, "bf16")])
def test_later_tokens_of_a_window_do_not_matter(T, h_q, d, kind):
    """A draft token's key and value rows hold infinities and NaN: the tokens
    before it are as if they did not, it and the ones after it see them."""
    bad = T // 2
    x = _case([T, 1], [300, 77], h_q, 2, d, 16, kind)
    pos = 300 - T + bad
    page, row = int(x["table"][0, pos // 16]), pos % 16
    clean = _run(x, [T, 1], 0.1)
    x["v"][page, 0, row, ::3] = math.inf
    x["v"][page, 0, row, 1::3] = math.nan
    x["k"][page, 1, row] = math.nan
    o = _run(x, [T, 1], 0.1)
    assert torch.equal(o[0, :bad], clean[0, :bad]) and torch.equal(o[1], clean[1])
    first, second = o[0, bad:, :h_q // 2], o[0, bad:, h_q // 2:]
    assert (first[..., ::3] == math.inf).all()
    assert torch.isnan(first[..., 1::3]).all()
    assert torch.equal(first[..., 2::3], clean[0, bad:, :h_q // 2][..., 2::3])
    assert torch.isnan(second).all()


def test_nan_in_the_cache_reaches_the_rows_that_see_it():
    x = _case([1, 2], [3000, 77], 4, 2, 128, 16, "bf16")
    x["k"][int(x["table"][0, 3]), 0, 5] = math.nan
    o = _run(x, [1, 2], 0.1)
    assert torch.isnan(o[0, 0, :2]).all() and torch.isfinite(o[0, 0, 2:]).all()
    assert torch.isfinite(o[1]).all()


def test_shared_pages():
    """Two lanes with a common prefix, and a page twice in one lane."""
    x = _case([1, 1], [64, 64], 4, 2, 128, 16, "bf16")
    x["table"][1, :3] = x["table"][0, :3]
    x["table"][0, 1] = x["table"][0, 0]
    _check(x, [1, 1], _run(x, [1, 1], 0.1), 0.1)


def test_256_lanes():
    lens = [1 + (i * 29) % 150 for i in range(256)]
    t_lane = [i % 3 for i in range(256)]
    x = _case(t_lane, lens, 2, 1, 64, 16, "bf16")
    _check(x, t_lane, _run(x, t_lane, 0.125), 0.125)


def test_one_long_lane_among_short_ones():
    lens = [30000, 3, 100, 1]
    x = _case([1] * 4, lens, 4, 1, 64, 64, "bf16")
    _check(x, [1] * 4, _run(x, [1] * 4, 0.125), 0.125)


def test_a_cache_longer_than_32_bits():
    """Pages whose rows lie past 2^32 elements of the cache."""
    page, h_kv, d = 256, 8, 256
    pages = (1 << 32) // (page * h_kv * d) + 40          # 4.3e9 elements each
    x = dict(k=torch.empty(pages, h_kv, page, d, dtype=torch.bfloat16, device="cuda"),
             v=torch.empty(pages, h_kv, page, d, dtype=torch.bfloat16, device="cuda"))
    at = [pages - 1, 3, pages - 30]
    for c in ("k", "v"):
        for p in at:
            x[c][p] = torch.randn(h_kv, page, d, device="cuda")
    x["q"] = torch.randn(1, 1, 8, d, device="cuda").bfloat16()
    x["table"] = torch.tensor([at], dtype=torch.int32, device="cuda")
    x["kv_len"] = torch.tensor([700], dtype=torch.int32, device="cuda")
    x["dims"] = gdn.KvDims.of(1, 1, 8, h_kv, d, page, pages, 3)
    new = [torch.randn(1, 1, h_kv, d, device="cuda").bfloat16() for _ in range(2)]
    gdn.kv_append(x["dims"], [1], *new, x["k"], x["v"], x["table"], x["kv_len"])
    o = _run(x, [1], 0.0625)
    assert torch.equal(x["k"][at[2], :, 699 - 512], new[0][0, 0])
    small = dict(x, k=x["k"][at].clone(), v=x["v"][at].clone(),
                 table=torch.arange(3, dtype=torch.int32, device="cuda")[None])
    del x
    _check(small, [1], o, 0.0625)


# ------------------------------------------------------------------- append
@pytest.mark.parametrize("t_lane,lens,h_kv,d,page,kind", [
    ([1], [1], 1, 64, 1, "bf16"),
    ([3, 0, 5], [20, 9, 5], 2, 128, 8, "bf16"),
    ([64, 64], [64, 100], 3, 256, 7, "f32"),
    ([4, 4], [2, 0], 2, 64, 16, "f32"),                 # rows before position 0
])
def test_append(t_lane, lens, h_kv, d, page, kind):
    x = _case(t_lane, lens, h_kv, h_kv, d, page, kind)
    T = x["dims"].t_max
    k, v = (torch.randn(len(lens), T, h_kv, d, device="cuda").to(TYPES[kind])
            for _ in range(2))
    x["k"].nan_to_num_(3.0)
    x["v"].nan_to_num_(3.0)
    want = {"k": x["k"].clone(), "v": x["v"].clone()}
    for n, m in enumerate(t_lane):
        for t in range(m):
            pos = lens[n] - m + t
            if pos >= 0:
                p = int(x["table"][n, pos // page])
                want["k"][p, :, pos % page] = k[n, t]
                want["v"][p, :, pos % page] = v[n, t]
    gdn.kv_append(x["dims"], t_lane, k, v, x["k"], x["v"], x["table"], x["kv_len"])
    for c in ("k", "v"):
        assert torch.equal(x[c], want[c])


def test_append_drops_rows_without_a_page():
    x = _case([2, 2], [18, 10], 2, 2, 64, 8, "bf16")
    x["table"][0, 2] = x["dims"].n_pages
    x["table"][1, 1] = -1
    k = torch.ones(2, 2, 2, 64, device="cuda").bfloat16()
    before = x["k"].nan_to_num_(3.0).clone()
    x["v"].nan_to_num_(3.0)
    gdn.kv_append(x["dims"], [2, 2], k, k, x["k"], x["v"], x["table"], x["kv_len"])
    assert torch.equal(x["k"], before)


def test_append_drops_rows_past_the_table_and_before_the_cache():
    """Lengths beyond the table's positions and shorter than the window: the
    rows that have a position go there, the others nowhere."""
    x = _case([4, 4, 4, 4], [10, 10, 10, 10], 2, 2, 64, 8, "bf16")
    cols = x["dims"].max_pages
    cap = cols * 8
    x["table"].copy_(torch.randperm(x["dims"].n_pages, device="cuda")[:4 * cols].view(4, cols))
    x["k"].nan_to_num_(3.0)
    x["v"].nan_to_num_(3.0)
    lens = [cap + 2, 1, 2**31 - 1, -2**31]
    x["kv_len"].copy_(torch.tensor(lens, dtype=torch.int32))
    k, v = (torch.randn(4, 4, 2, 64, device="cuda").bfloat16() for _ in range(2))
    want = {c: x[c].clone() for c in ("k", "v")}
    for n, length in enumerate(lens):
        for t in range(4):
            pos = length - 4 + t
            if 0 <= pos < cap:
                page = int(x["table"][n, pos // 8])
                want["k"][page, :, pos % 8] = k[n, t]
                want["v"][page, :, pos % 8] = v[n, t]
    gdn.kv_append(x["dims"], [4] * 4, k, v, x["k"], x["v"], x["table"], x["kv_len"])
    for c in ("k", "v"):
        assert torch.equal(x[c], want[c])


def test_captured_calls_follow_the_lengths():
    """Append and attention captured once; the replays see the lengths and
    pages of their time."""
    x = _case([1, 1], [300, 150], 8, 2, 128, 16, "bf16", T=1)
    x["k"].nan_to_num_(0.5)
    x["v"].nan_to_num_(0.5)
    cols = x["dims"].max_pages
    x["table"].copy_(torch.randperm(x["dims"].n_pages, device="cuda")[:2 * cols].view(2, cols))
    o = torch.empty(x["q"].shape, device="cuda")
    ws = torch.empty(gdn.paged_attention_workspace_bytes(x["dims"]),
                     dtype=torch.uint8, device="cuda")
    k, v = (torch.randn(2, 1, 2, 128, device="cuda").bfloat16() for _ in range(2))

    def calls():
        gdn.kv_append(x["dims"], [1, 1], k, v, x["k"], x["v"], x["table"], x["kv_len"])
        gdn.paged_attention(x["dims"], [1, 1], x["q"], x["k"], x["v"],
                            x["table"], x["kv_len"], o, ws, scale=0.1)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for length in ([301, 151], [5, 320], [1, 1]):
        x["kv_len"].copy_(torch.tensor(length, dtype=torch.int32))
        k.copy_(torch.randn(2, 1, 2, 128, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        _check(x, [1, 1], o, 0.1)
        got = o.clone()
        calls()
        torch.cuda.synchronize()
        assert torch.equal(o, got)

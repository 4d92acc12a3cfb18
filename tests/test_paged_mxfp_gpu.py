"""gdn_paged_attention_mxfp against attention in 64 bits over the decoded
rows of the gathered pages."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import commit_gated_delta_amd as gdn  # noqa: E402
from tests import cache_ref as ref  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
NAMES = ("k_codes", "k_scales", "v_codes", "v_scales")


def _case(t_lane, lens, h_q, h_kv, d, page, kind, T=None, seed=0, extra=2, spread=4):
    """Random pages; rows behind each lane's length and unused pages hold
    NaN, table entries behind it page numbers outside the cache."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    N, T, t = len(lens), T or max(max(t_lane), 1), TYPES[kind]
    cols = max(1, max(-(-max(n, 0) // page) for n in lens)) + extra
    pages = N * cols + 3
    x = dict(q=torch.randn(N, T, h_q, d, device="cuda", generator=g).to(t))
    order = torch.randperm(pages, device="cuda", generator=g)[:N * cols].view(N, cols)
    used = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    table = torch.full((N, cols), -1, dtype=torch.int32, device="cuda")
    table[:, 1::2] = 1 << 30
    for n, length in enumerate(lens):
        for j in range(-(-max(length, 0) // page)):
            table[n, j] = order[n, j]
            used[order[n, j], : min(page, length - j * page)] = True
    for c in "kv":
        x[c + "_codes"] = torch.randint(256, (pages, h_kv, page, d // 2), device="cuda", generator=g, dtype=torch.uint8)
        s = torch.randint(128 - spread, 128, (pages, h_kv, page, d // 32), device="cuda", generator=g, dtype=torch.uint8)
        x[c + "_scales"] = s.masked_fill(~used[:, None, :, None], 255)
    x["table"] = table
    x["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    x["dims"] = gdn.KvDims.of(N, T, h_q, h_kv, d, page, pages, cols)
    return x


def _run(x, t_lane, scale, stream=None, ws=None):
    o = torch.full(x["q"].shape, 7.0, device="cuda")
    if ws is None:
        ws = torch.empty(gdn.paged_attention_mxfp_workspace_bytes(x["dims"]), dtype=torch.uint8, device="cuda")
    gdn.paged_attention_mxfp(x["dims"], t_lane, x["q"], *(x[n] for n in NAMES), x["table"], x["kv_len"], o, ws,
                             scale=scale, stream=stream)
    torch.cuda.synchronize()
    return o


def _want(x, t_lane, scale):
    k, v = (ref.decode(x[c + "_codes"], x[c + "_scales"]) for c in "kv")
    return ref.attend(x["q"], k, v, x["table"], x["kv_len"], t_lane, scale, x["dims"].page_size, x["dims"].n_pages)


def _check(x, t_lane, o, scale):
    want, tol = _want(x, t_lane, scale)
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
    ([1, 1], [300, 77], 6, 2, 256, 16, "f32"),
    ([1], [2049], 40, 1, 128, 128, "f32"),
    ([20, 4], [150, 90], 12, 2, 64, 24, "f32"),
    ([40], [333], 6, 2, 128, 16, "f32"),
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
    ([16], [7001], 8, 1, 128, "bf16"),
    ([9, 2], [5000, 2600], 16, 1, 256, "f32"),
    ([1] * 10, [20000] + [30] * 9, 32, 1, 64, "bf16"),   # and of some hundred
    ([1] * 10, [9999] + [300] * 9, 32, 1, 128, "f32"),
    ([1] * 20, [9001] + [30] * 19, 16, 1, 256, "bf16"),
    ([17, 9], [3001, 700], 5, 1, 128, "bf16"),           # rows past a wave's last
    ([23, 3], [2500, 70], 3, 1, 64, "f32"),
    ([22, 30], [900, 2100], 3, 1, 128, "f32"),
])
def test_many_splits(t_lane, lens, h_q, h_kv, d, kind):
    x = _case(t_lane, lens, h_q, h_kv, d, 64, kind)
    x["q"][0, 0, 0] *= 4                               # weights far apart
    _check(x, t_lane, _run(x, t_lane, d ** -0.5), d ** -0.5)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T", [2, 40])
def test_peaked_scores(kind, T):
    """Scores far apart: one position takes nearly everything, in any tile."""
    x = _case([T, 2], [900, 70], 4, 2, 128, 16, kind)
    x["q"].mul_(6)
    _check(x, [T, 2], _run(x, [T, 2], 0.3), 0.3)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_queries_of_any_size(kind):
    """Blocks of a query row from tiny to huge, zeros among them."""
    x = _case([1, 2], [90, 30], 4, 2, 128, 16, kind)
    for i, f in enumerate((1e-30, 1e-3, 0.0, 1e4)):
        x["q"][0, 0, :, 32 * i:32 * i + 32] *= f
    x["q"][1, 0] *= 1e-20
    x["q"][1, 1, :, ::2] *= 2.0 ** -14
    _check(x, [1, 2], _run(x, [1, 2], 1e-4), 1e-4)


@pytest.mark.parametrize("low,high", [(1, 9), (60, 90), (120, 190)])
def test_scales_of_any_size(low, high):
    """Scale bytes over a wide range; values small enough that sums stay in
    f32 (a value below 2^-126 may count as zero)."""
    x = _case([1, 3], [90, 30], 4, 2, 128, 16, "bf16")
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    for c in "kv":
        s = x[c + "_scales"]
        s.copy_(torch.where(s == 255, s, torch.randint(low, high, s.shape, device="cuda", generator=g, dtype=torch.uint8)))
    scale = 2.0 ** (120 - high)
    want, tol = _want(x, [1, 3], scale)
    o = _run(x, [1, 3], scale).cpu().double()
    for n, m in enumerate([1, 3]):
        err = (o[n, :m] - want[n, :m]).abs()
        assert (err <= tol[n, :m] + 2.0 ** -126).all(), float((err / tol[n, :m]).max())


def test_every_code():
    """One position: the output is its value row, every code exactly."""
    x = _case([1], [1], 1, 1, 128, 1, "bf16")
    p = int(x["table"][0, 0])
    for first in range(0, 256, 64):
        x["v_codes"][p, 0, 0] = torch.arange(first, first + 64, dtype=torch.uint8, device="cuda")
        x["v_scales"][p, 0, 0] = torch.tensor([10, 126, 127, 250], dtype=torch.uint8, device="cuda")
        o = _run(x, [1], 0.1)[0, 0, 0].cpu().double()
        assert torch.equal(o, ref.decode(x["v_codes"][p, 0, 0], x["v_scales"][p, 0, 0]) + 0.0)


def test_negative_and_zero_scale():
    x = _case([1, 2], [90, 30], 4, 2, 64, 16, "bf16")
    for scale in (-0.2, 0.0):
        _check(x, [1, 2], _run(x, [1, 2], scale), scale)


def test_lengths_outside_the_table_are_cut():
    x = _case([1, 2, 1], [40, 48, 20], 4, 2, 64, 16, "bf16", extra=0)
    x["kv_len"].copy_(torch.tensor([1 << 30, 48, -5], dtype=torch.int32))
    for c in "kv":
        x[c + "_scales"].masked_fill_(x[c + "_scales"] == 255, 125)
    o = _run(x, [1, 2, 1], 0.1)
    _check(x, [1, 2, 1], o, 0.1)
    assert (o[2, 0] == 0).all()


@pytest.mark.parametrize("T", [3, 50])
def test_bad_page_numbers_are_masked(T):
    x = _case([1, T], [200, 90], 4, 2, 128, 16, "bf16")
    x["table"][0, 2] = -7
    x["table"][0, 12] = x["dims"].n_pages
    x["table"][1, :] = -1                               # a lane with no page
    o = _run(x, [1, T], 0.1)
    _check(x, [1, T], o, 0.1)
    assert (o[1, :T] == 0).all()


@pytest.mark.parametrize("T,h_q,d,kind", [(4, 4, 128, "bf16"), (16, 16, 128, "bf16"), (3, 2, 64, "f32"),
                                          (40, 2, 256, "bf16"), (40, 2, 64, "bf16"), (12, 2, 256, "f32")])
def test_later_tokens_of_a_window_do_not_matter(T, h_q, d, kind):
    """A draft token's key and value rows hold NaN: the tokens before it are
    as if they did not, it and the ones after it see them."""
    bad = T // 2
    x = _case([T, 1], [300, 77], h_q, 2, d, 16, kind)
    pos = 300 - T + bad
    page, row = int(x["table"][0, pos // 16]), pos % 16
    clean = _run(x, [T, 1], 0.1)
    x["v_scales"][page, 0, row, 0] = 255
    x["k_scales"][page, 1, row] = 255
    o = _run(x, [T, 1], 0.1)
    assert torch.equal(o[0, :bad], clean[0, :bad]) and torch.equal(o[1], clean[1])
    first, second = o[0, bad:, :h_q // 2], o[0, bad:, h_q // 2:]
    assert torch.isnan(first[..., :32]).all()
    assert torch.equal(first[..., 32:], clean[0, bad:, :h_q // 2][..., 32:])
    assert torch.isnan(second).all()


@pytest.mark.parametrize("byte", [253, 254, 255])
@pytest.mark.parametrize("T,d", [(1, 64), (1, 128), (2, 256), (40, 64), (40, 128), (40, 256)])
def test_blocks_that_read_as_nan(byte, T, d):
    """Value blocks with the largest scale bytes, in one and in several
    places of a step: NaN in their channels for the tokens that see one, the
    other channels as before.  Key blocks: NaN in every channel."""
    x = _case([T], [500], 4, 2, d, 16, "bf16")
    clean = _run(x, [T], 0.1)
    bad = {0: [3, 17, 300], d // 32 - 1: [500 - T // 2 - 1, 499]}     # block: positions
    for b, where in bad.items():
        for pos in where:
            x["v_scales"][int(x["table"][0, pos // 16]), 1, pos % 16, b] = byte
    o = _run(x, [T], 0.1)
    assert torch.equal(o[0, :, :2], clean[0, :, :2])
    want = clean.clone()
    for b, where in bad.items():
        for t in range(T):
            if min(where) <= 500 - T + t:
                want[0, t, 2:, 32 * b:32 * b + 32] = math.nan
    assert torch.equal(torch.isnan(o), torch.isnan(want))
    assert torch.equal(o.nan_to_num(9.0), want.nan_to_num(9.0))
    x["k_scales"][int(x["table"][0, 400 // 16]), 0, 400 % 16, 1] = byte
    o = _run(x, [T], 0.1)
    assert torch.isnan(o[0, :, :2]).all() and torch.equal(o[0, :, 2:].nan_to_num(9.0), want[0, :, 2:].nan_to_num(9.0))


def test_nan_in_the_cache_reaches_the_rows_that_see_it():
    x = _case([1, 2], [3000, 77], 4, 2, 128, 16, "bf16")
    x["k_scales"][int(x["table"][0, 3]), 0, 5, 2] = 255
    o = _run(x, [1, 2], 0.1)
    assert torch.isnan(o[0, 0, :2]).all() and torch.isfinite(o[0, 0, 2:]).all()
    assert torch.isfinite(o[1]).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("what", [math.inf, -math.inf, math.nan])
def test_queries_that_are_not_finite(kind, what):
    x = _case([2, 1, 1], [300, 77, 0], 4, 2, 128, 16, kind)
    clean = _run(x, [2, 1, 1], 0.1)
    x["q"][0, 1, 2, 77] = what
    x["q"][2, 0] = what
    o = _run(x, [2, 1, 1], 0.1)
    assert torch.isnan(o[0, 1, 2]).all()
    assert (o[2, 0] == 0).all()                          # sees nothing
    keep = torch.ones(3, 2, 4, dtype=torch.bool)
    keep[0, 1, 2] = False
    assert torch.equal(o[keep.cuda()], clean[keep.cuda()])


@pytest.mark.parametrize("T", [1, 30])
def test_scores_of_minus_infinity_alone(T):
    """Scores past f32: -inf everywhere that a row sees gives NaN, and no
    weight beside finite ones."""
    x = _case([T, 1], [40, 7], 4, 2, 64, 16, "f32")
    x["q"].fill_(1e30)
    x["k_codes"].fill_(0x77)                             # 6, 6
    x["k_scales"].masked_fill_(x["k_scales"] != 255, 127)
    o = _run(x, [T, 1], -1e30)
    assert torch.isnan(o[0]).all() and torch.isnan(o[1, :1]).all()
    pos = 40 - T                                          # one position with scores of 0
    x["k_codes"][int(x["table"][0, pos // 16]), :, pos % 16] = 0
    o = _run(x, [T, 1], -1e30)
    v = ref.decode(x["v_codes"], x["v_scales"])[int(x["table"][0, pos // 16]), :, pos % 16]
    assert torch.equal(o[0].cpu().double(), v.repeat_interleave(2, 0)[None].expand(T, 4, 64) + 0.0)


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


@pytest.mark.parametrize("d,kind", [(64, "bf16"), (128, "f32"), (256, "bf16")])
def test_one_long_lane_among_short_ones(d, kind):
    lens = [30000, 3, 100, 1]
    x = _case([1] * 4, lens, 4, 1, d, 64, kind)
    _check(x, [1] * 4, _run(x, [1] * 4, 0.125), 0.125)


@pytest.mark.parametrize("T,h_q,d", [(1, 4, 128), (1, 4, 256), (1, 4, 64), (40, 8, 128), (40, 4, 64), (20, 8, 256)])
def test_every_position_counts_once(T, h_q, d):
    """Equal scores: outputs are the means of the values that a token sees."""
    length = 3333
    x = _case([T], [length], h_q, 2, d, 24, "bf16")
    x["q"].zero_()
    v = ref.decode(x["v_codes"], x["v_scales"])
    pos = torch.arange(length)
    rows = v[x["table"].cpu()[0, pos // 24].long(), :, pos % 24]          # [L, 2, d]
    sums, mag = rows.cumsum(0), rows.abs().cumsum(0)
    o = _run(x, [T], 1.0).cpu().double()
    for t in range(T):
        n = length - T + t + 1
        want = (sums[n - 1] / n).repeat_interleave(h_q // 2, 0)
        tol = (2 * n + 16) * ref.U32 * (mag[n - 1] / n).repeat_interleave(h_q // 2, 0)
        assert ((o[0, t] - want).abs() <= tol).all(), t


@pytest.mark.parametrize("T,kind", [(1, "bf16"), (1, "f32"), (40, "bf16"), (40, "f32")])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_scores_that_rise_and_fall_along_the_cache(T, kind, d):
    """Keys whose scores grow or shrink by 2^160 along the cache: the running
    maximum is raised many times, or early ones hold on."""
    length = 1500
    x = _case([T], [length], 4, 1, d, 16, kind)
    x["q"].zero_()
    x["q"][..., 0] = 1.0
    pos = torch.arange(length)
    pages, rows = x["table"].cpu()[0, pos // 16].long(), pos % 16
    step = (pos * 8 // length)
    for up in (True, False):
        level = step if up else 7 - step
        x["k_scales"][pages.cuda(), 0, rows.cuda(), 0] = (120 + level).to(torch.uint8).cuda()
        x["k_codes"][pages.cuda(), 0, rows.cuda(), 0] = 0x04                # 2 in channel 0
        _check(x, [T], _run(x, [T], 80.0), 80.0)


def test_a_cache_longer_than_32_bits():
    """Pages whose rows lie past 2^32 bytes of codes."""
    page, h_kv, d = 256, 8, 256
    pages = (1 << 33) // (page * h_kv * d) + 40
    x = {}
    at = [pages - 1, 3, pages - 30]
    for c in "kv":
        x[c + "_codes"] = torch.empty(pages, h_kv, page, d // 2, dtype=torch.uint8, device="cuda")
        x[c + "_scales"] = torch.empty(pages, h_kv, page, d // 32, dtype=torch.uint8, device="cuda")
        for p in at:
            x[c + "_codes"][p] = torch.randint(256, (h_kv, page, d // 2), device="cuda", dtype=torch.uint8)
            x[c + "_scales"][p] = torch.randint(124, 128, (h_kv, page, d // 32), device="cuda", dtype=torch.uint8)
    x["q"] = torch.randn(1, 1, 8, d, device="cuda").bfloat16()
    x["table"] = torch.tensor([at], dtype=torch.int32, device="cuda")
    x["kv_len"] = torch.tensor([700], dtype=torch.int32, device="cuda")
    x["dims"] = gdn.KvDims.of(1, 1, 8, h_kv, d, page, pages, 3)
    o = _run(x, [1], 0.0625)
    small = dict(x, **{n: x[n][at].clone() for n in NAMES},
                 table=torch.arange(3, dtype=torch.int32, device="cuda")[None],
                 dims=gdn.KvDims.of(1, 1, 8, h_kv, d, page, 3, 3))
    del x
    _check(small, [1], o, 0.0625)


def test_the_same_call_gives_the_same_bits():
    x = _case([2, 1, 1], [4000, 2500, 9], 16, 2, 128, 16, "bf16")
    a = _run(x, [2, 1, 1], 0.1)
    for _ in range(3):
        assert torch.equal(_run(x, [2, 1, 1], 0.1), a)


def test_captured_calls_on_two_streams_follow_the_lengths():
    """Two captured calls with workspaces of their own, replayed at once, and
    against eager calls, at other lengths."""
    xs = [_case([1, 1], [3000, 150], 8, 2, 128, 16, "bf16", T=1, seed=s) for s in (1, 2)]
    for x in xs:
        for c in "kv":
            x[c + "_scales"].masked_fill_(x[c + "_scales"] == 255, 125)
        cols = x["dims"].max_pages
        x["table"].copy_(torch.randperm(x["dims"].n_pages, device="cuda")[:2 * cols].view(2, cols))
    ws = [torch.empty(gdn.paged_attention_mxfp_workspace_bytes(x["dims"]), dtype=torch.uint8, device="cuda") for x in xs]
    outs = [torch.full(x["q"].shape, 7.0, device="cuda") for x in xs]
    graphs, streams = [], [torch.cuda.Stream() for _ in xs]

    def call(i, x):
        gdn.paged_attention_mxfp(x["dims"], [1, 1], x["q"], *(x[n] for n in NAMES), x["table"], x["kv_len"],
                                 outs[i], ws[i], scale=0.1)

    for i, x in enumerate(xs):
        call(i, x)
    torch.cuda.synchronize()
    for i, x in enumerate(xs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            call(i, x)
    for length in ([3001, 151], [5, 3000], [1, 1]):
        for x in xs:
            x["kv_len"].copy_(torch.tensor(length, dtype=torch.int32))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for i, x in enumerate(xs):
            got = outs[i].clone()
            assert torch.equal(got, _run(x, [1, 1], 0.1))
            if max(length) < 200:
                _check(x, [1, 1], got, 0.1)

"""gdn_paged_attention_mxfp where finite scores lie far from 0: past 2^24 a
step of f32 is a whole octave of a weight, and past f32 a scaled score is an
infinity."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests import cache_ref as ref  # noqa: E402
from tests.test_paged_mxfp_gpu import _case, _run, _want  # noqa: E402

# name: T, length, h_q, h_kv, d, page, kind
FORMS = {
    "one tile": (1, 60, 4, 2, 128, 16, "bf16"),
    "odd pages": (1, 200, 6, 2, 64, 7, "f32"),
    "splits": (1, 9000, 4, 1, 256, 24, "bf16"),
    "two tiles of rows": (5, 3000, 10, 2, 128, 16, "bf16"),
    "many rows": (16, 3000, 8, 1, 128, 32, "bf16"),
    "many rows f32": (16, 3000, 8, 1, 128, 32, "f32"),
    "wide heads": (20, 700, 8, 2, 256, 16, "f32"),
    "few of many": (3, 2000, 21, 1, 64, 64, "bf16"),
}


def _pointed(form, log2, signs=1):
    """A cache whose rows' signs are those of one direction a head (against
    it where `signs` is -1) and queries along it: every score's size is about
    2^log2 (of base 2), all of one sign, the sizes of a row's entries random."""
    T, length, h_q, h_kv, d, page, kind = form
    x = _case([T], [length], h_q, h_kv, d, page, kind, seed=int(log2 * 8), spread=1)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    minus = torch.rand(h_kv, d, device="cuda", generator=g) < 0.5
    q = torch.rand(1, T, h_q, d, device="cuda", generator=g) + 0.5
    # |entry| about 3.5, q about 1: a score about 3.5 d
    q *= 2.0 ** log2 / (3.5 * d) * math.log(2.0)
    q = torch.where(minus.repeat_interleave(h_q // h_kv, 0), -q, q)
    x["q"] = q.to(x["q"].dtype)
    # codes of the values 2, 3 or 4, and where it points against q the sign
    low = torch.randint(4, 7, x["k_codes"].shape, device="cuda", generator=g)
    high = torch.randint(4, 7, x["k_codes"].shape, device="cuda", generator=g)
    sign = 8 * (minus if signs > 0 else ~minus).int()
    x["k_codes"] = (low | sign[None, :, None, 0::2] | (high | sign[None, :, None, 1::2]) << 4).to(torch.uint8)
    x["sign"] = sign
    return x


def _point(x, pos, code):
    """Position pos's keys: every entry the value of `code`, its sign kept."""
    page = x["dims"].page_size
    at = (code | x["sign"])
    x["k_codes"][int(x["table"][0, pos // page]), :, pos % page] = (at[:, 0::2] | at[:, 1::2] << 4).to(torch.uint8)


def _values(x, pos):
    page = x["dims"].page_size
    v = ref.decode(x["v_codes"], x["v_scales"])[int(x["table"][0, pos // page]), :, pos % page]
    return v.repeat_interleave(x["dims"].h_q // x["dims"].h_kv, 0)


# A weight of the one position that counts, its product with a value (exact
# parts, two sums), a rescaling, the sums over waves and splits (one term is
# not 0), the reciprocal and the last product: a step each at most.
TOL = 8 * ref.U32


@pytest.mark.parametrize("scale", [1.0, -1.0, 0.125])
@pytest.mark.parametrize("log2", [20, 23.5, 24.5, 26, 28, 30, 31.5, 32, 32.5, 33, 34, 36, 40, 80])
@pytest.mark.parametrize("form", list(FORMS))
def test_one_clear_maximum(form, log2, scale):
    T, length = FORMS[form][:2]
    x = _pointed(FORMS[form], log2 - math.log2(abs(scale)), 1 if scale > 0 else -1)
    for pos in (length - T, length // 3):
        _point(x, pos, 7)                               # 6, others 4 at most
        o = _run(x, [T], scale).cpu().double()
        want = _values(x, pos)
        assert ((o[0] - want).abs() <= TOL * want.abs()).all(), pos
        _point(x, pos, 4)


@pytest.mark.parametrize("log2", [24.5, 31, 32, 33, 34, 36, 40, 80])
@pytest.mark.parametrize("form", list(FORMS))
def test_one_clear_maximum_below_zero(form, log2):
    T, length = FORMS[form][:2]
    x = _pointed(FORMS[form], log2, -1)
    for pos in (length - T, length // 3):
        _point(x, pos, 2)                               # 1, others 2 at least
        o = _run(x, [T], 1.0).cpu().double()
        want = _values(x, pos)
        assert ((o[0] - want).abs() <= TOL * want.abs()).all(), pos
        _point(x, pos, 5)


@pytest.mark.parametrize("log2", [20, 25, 30, 32, 33, 34, 36, 40, 80])
@pytest.mark.parametrize("form", list(FORMS))
def test_equal_maxima_share_the_weight(form, log2):
    """Two equal keys: the mean of their values."""
    T, length = FORMS[form][:2]
    x = _pointed(FORMS[form], log2)
    at = (length - T, length // 3)
    for pos in at:
        _point(x, pos, 7)
    o = _run(x, [T], 1.0).cpu().double()
    a, b = (_values(x, pos) for pos in at)
    assert ((o[0] - (a + b) / 2).abs() <= TOL * (a.abs() + b.abs()) / 2).all()


@pytest.mark.parametrize("form", list(FORMS))
def test_far_rows_beside_ordinary_ones(form):
    """Rows with far scores share a wave with ordinary ones, which stay within
    their bounds."""
    T, length, h_q = FORMS[form][:3]
    x = _case([T], [length], *FORMS[form][2:], seed=3)
    scale = FORMS[form][4] ** -0.5
    want, tol = _want(x, [T], scale)
    x["q"][0, ::2, 1] *= 2.0 ** 34
    o = _run(x, [T], scale).cpu().double()
    assert torch.isfinite(o).all()
    near = torch.ones(T, h_q, dtype=torch.bool)
    near[::2, 1] = False
    assert ((o[0] - want[0]).abs() <= tol[0])[near].all()


@pytest.mark.parametrize("T", [1, 30])
def test_scores_past_f32(T):
    """Finite products whose scaled score is +inf have no softmax: NaN for the
    rows that see one, and nothing for those that do not."""
    x = _case([T, 1], [40, 7], 4, 2, 64, 16, "f32")
    x["q"].fill_(1e30)
    x["k_codes"].fill_(0x77)                             # 6, 6
    x["k_scales"].masked_fill_(x["k_scales"] != 255, 127)
    o = _run(x, [T, 1], 1e30)
    assert torch.isnan(o[0]).all() and torch.isnan(o[1, :1]).all()
    x["k_codes"].zero_()                                 # scores of 0
    clean = _run(x, [T, 1], 1e30)
    assert torch.isfinite(clean[0]).all()
    pos = 39                                             # the last token sees it, no other
    x["k_codes"][int(x["table"][0, pos // 16]), 1, pos % 16] = 0x77
    o = _run(x, [T, 1], 1e30)
    assert torch.isnan(o[0, T - 1, 2:]).all()
    assert torch.equal(o[0, :, :2], clean[0, :, :2]) and torch.equal(o[0, :T - 1], clean[0, :T - 1])
    assert torch.equal(o[1, :1], clean[1, :1])


@pytest.mark.parametrize("T,h_q,d,kind", [(1, 4, 256, "bf16"), (2, 8, 128, "f32"), (24, 8, 64, "bf16"), (16, 16, 128, "f32")])
def test_a_score_past_f32_in_a_long_cache(T, h_q, d, kind):
    """One of many splits holds the score that scales to +inf: NaN for the heads
    that see it, and the others as before."""
    x = _case([T], [7000], h_q, 2, d, 16, kind)
    x["k_codes"].zero_()
    x["q"].fill_(1e30)
    clean = _run(x, [T], 1e30)
    assert torch.isfinite(clean).all()
    x["k_codes"][int(x["table"][0, 2001 // 16]), 1, 2001 % 16] = 0x77
    o = _run(x, [T], 1e30)
    assert torch.isnan(o[0, :, h_q // 2:]).all()
    assert torch.equal(o[0, :, :h_q // 2], clean[0, :, :h_q // 2])

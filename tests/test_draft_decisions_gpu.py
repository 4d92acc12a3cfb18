"""gdn_draft_verify: every lane's decision, and chances within the error that
their sums have, row by row."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests import cache_ref as ref  # noqa: E402
from tests.test_draft_verify_gpu import _case, _check, _run  # noqa: E402


def _row_error(row, it):
    """Relative error of a row's sum, in steps of 2^-24.  A logit's distance
    from the largest is rounded once and its exponent once, so that a weight
    2^-y is off by 2 y ln 2, and the instruction by two (a step of its last bit):
    the sum by their mean over the row's distribution.  31 additions in a
    thread, six in a wave and two over the waves round once each; what follows
    is f64."""
    x = row.double().cpu()
    y = (x.amax() - x) * float(it) * math.log2(math.e)
    w = torch.exp2(-y)
    mean = float((torch.where(w > 0, y, 0.0) * w).sum() / w.sum())
    return 2 * math.log(2) * mean + 2 + 31 + 6 + 2


def _errors(s, got):
    """(error of every chance below 1 in steps, its bound) of rows that have
    distributions."""
    out = []
    want = ref.verify(s["t_lane"], s["logits"], s["draft"], s["tokens"], s["uniforms"], s["it"])
    for n, w in enumerate(want):
        for t, c in enumerate(w[2] if w else ()):
            if not 0 < c < 1:
                continue
            bound = _row_error(s["logits"][n, t], s["it"][n]) + 1        # (the chance rounds once)
            if s["draft"] is not None:
                bound += _row_error(s["draft"][n, t], s["it"][n])
            out.append(((float(got[2][n, t]) - c) / c / ref.U32, bound))
    return out


@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("t_lane,V,kind,right", [
    ([4, 0, 2, 1], 37, "bf16", 0.8),
    ([16, 5, 1, 9], 1111, "f32", 0.8),
    ([6] * 12, 5003, "bf16", 0.8),
    ([64, 33], 300, "f32", 0.9),
    ([9] * 20, 20001, "f32", 0.3),
    ([2, 3], 131072, "f32", 0.8),
    ([3, 5, 4], 131072, "bf16", 0.0),
    ([1, 1, 2], 262144, "bf16", 0.8),
    ([4, 2], 65537, "f32", 0.8),
])
def test_every_lane_decides_as_the_definition(t_lane, V, kind, right, drafted):
    s = _case(t_lane, V, kind, drafted, right=right, seed=11)
    got = _run(s)
    _check(s, got, 1.0)
    errors = _errors(s, got)
    for e, bound in errors:
        assert abs(e) <= bound
    if len(errors) >= 30:
        # roundings that have no common sign: a step of some 80 at most
        rms = math.sqrt(sum(e * e for e, _ in errors) / len(errors))
        print("%d chances, %.2f steps rms, worst %.2f" % (len(errors), rms, max(abs(e) for e, _ in errors)), flush=True)
        assert rms <= math.sqrt(80)


@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("above", [0.3, 5.0, 11.7836, 17.3])
def test_flat_rows_with_one_logit_above(above, drafted):
    """Weights that all round the same way: the bound without any luck."""
    V = 131072
    s = _case([3, 3], V, "f32", drafted, seed=2)
    for c in ("logits", "draft"):
        if s[c] is not None:
            s[c].fill_(-0.7)
            s[c][..., 99] = -0.7 + above
    if drafted:
        s["draft"][..., 99] += 0.25
    s["tokens"][0, 1:], s["tokens"][1, 1:] = 99, 1234
    s["it"].copy_(torch.tensor([1.0, 0.83]))
    got = _run(s)
    errors = _errors(s, got)
    assert len(errors) >= 2
    for e, bound in errors:
        assert abs(e) <= bound
    _check(s, got, 1.0)


@pytest.mark.parametrize("V", [50, 3000, 20000])
@pytest.mark.parametrize("drafted", [False, True])
def test_exactly_the_first_drafts_stand(V, drafted):
    """Lane k's draft k is one that the model hardly has, and the drafter almost
    nothing else: it falls under a uniform next to 1, the ones before it stand
    under 0, and the next token comes from what is left there."""
    T = 6
    s = _case([T] * T, V, "f32", drafted, right=1.0, seed=4)
    s["it"].fill_(1.0)
    s["uniforms"].fill_(0.0)
    for k in range(T - 1):
        w = (int(s["tokens"][k, k + 1]) + 1) % V
        s["tokens"][k, k + 1] = w
        s["uniforms"][k, k] = 1.0 - 2.0 ** -24
        if drafted:
            s["draft"][k, k, w] = 30.0
    for i in range(21):
        s["uniforms"][:, T - 1] = (i + 0.5) / 21
        got = _run(s)
        assert got[0] == list(range(1, T + 1))
        _check(s, got, 1.0)

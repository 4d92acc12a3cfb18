"""gdn_token_scores on logits further apart than the largest f32: their
difference times a small inverse temperature is an ordinary number."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import commit_gated_delta_amd as gdn  # noqa: E402

U32 = 2.0 ** -24


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab", [(3, 7), (3, 9001), (130, 9001)])
def test_logits_further_apart_than_the_largest_number(rows, vocab, kind):
    """log p = (x - m) it: the difference and the product are rounded, log Z
    = log 2 is nothing beside it: 3 steps of 2^-24 of it."""
    it = 2.0 ** -99
    x = torch.full((rows, vocab), -2e38, device="cuda").to(kind)
    x[:, 2] = x[:, vocab - 2] = 3e38
    x[:, vocab - 3] = torch.finfo(kind).min
    x[:, 1] = -math.inf
    t = torch.zeros(rows, dtype=torch.int32, device="cuda")
    t[1], t[2] = vocab - 3, 1
    lp, ent = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ids = torch.empty(rows, 4, dtype=torch.int32, device="cuda")
    best = torch.empty(rows, 4, device="cuda")
    ws = torch.empty(gdn.token_scores_workspace_bytes(rows, vocab, 4), dtype=torch.uint8,
                     device="cuda")
    gdn.token_scores(x, t, 4, lp, ent, ids, best, ws, inv_temperature=it)
    y = x.double()
    logp = (y - y.amax(1, keepdim=True)) * it - math.log(2)
    want = logp.gather(1, t.long()[:, None])[:, 0]
    assert math.isfinite(float(want[0])) and float(want[1]) < float(want[0]) < -1e8
    assert torch.equal(torch.isinf(lp), torch.isinf(want))
    fine = torch.isfinite(want)
    assert ((lp - want).abs() <= 3 * U32 * want.abs())[fine].all()
    order = [2, vocab - 2] + [i for i in range(vocab) if i not in (1, 2, vocab - 2, vocab - 3)][:2]
    assert ids.tolist() == [order] * rows
    want = logp.gather(1, ids.long())
    assert torch.isfinite(best).all()
    assert ((best - want).abs() <= 3 * U32 * want.abs()).all()
    assert ((ent - math.log(2)).abs() <= 4 * U32).all()

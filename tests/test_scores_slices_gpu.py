"""gdn_token_scores where a thread takes 32 logits and a row is several
slices, as in large batches: ties, masked, empty and bad rows, the types'
lowest values, rows at odd offsets; that every logit counts exactly once; and
bounds derived row by row."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import commit_gated_delta_amd as gdn  # noqa: E402
from tests import serving_ref as ref  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
U32 = ref.U32
PER = 8192                    # logits of a slice at 32 a thread
# several slices a row, and at least 256 in all
SIZES = [(130, 9001), (130, 16384), (64, 40003), (29, 70001)]


def slices(rows, vocab):
    """Slices of a row (rows of any alignment), from the workspace: 16 bytes
    for the sums of each, and 8 for an alternative."""
    need = lambda top: gdn.token_scores_workspace_bytes(rows, vocab, top)
    return need(0) // 16 // rows


def assert_many(rows, vocab):
    n = slices(rows, vocab)
    assert n in (-(-vocab // PER), -(-(vocab + 8) // PER)) and n >= 2


def _run(x, tokens, top, it=1.0):
    rows = x.shape[0]
    lp, ent = (torch.full((rows,), 9.0, device="cuda") for _ in range(2))
    ids = torch.full((rows, top), 9, dtype=torch.int32, device="cuda")
    best = torch.full((rows, top), 9.0, device="cuda")
    ws = torch.empty(gdn.token_scores_workspace_bytes(rows, x.shape[1], top),
                     dtype=torch.uint8, device="cuda")
    gdn.token_scores(x, tokens, top, lp, ent, ids, best, ws, inv_temperature=it)
    torch.cuda.synchronize()
    return lp.cpu(), ent.cpu(), ids.cpu(), best.cpu()


def _row_bounds(x, it):
    """For a row of logits in f64 (finite or -inf): a function that bounds the
    error of a log p from its distance to the maximum, and the bound of the
    entropy.  With d = (m - x) it: exp2 of d is off by 4 d + 4 steps of 2^-24
    (the difference, the factor it log2 e and their product, twice where
    slices join, and one ulp of two exponentials), a sum by one for each of
    32 + 6 + 2 additions of a slice, of up to slices / 64 + 6 of the join and
    of 4 products; log by two ulp.  W = sum p d the same with two more."""
    m = x.max()
    d = (m - x) * it
    p = torch.softmax(-d, 0)
    dp = torch.where(p > 0, p * d, 0)
    eps = torch.where(p > 0, p * (4 * d + 4), 0)
    adds = 50 + x.numel() / PER / 64
    log_z = float(torch.logsumexp(-d, 0))
    rel = (float(eps.sum()) + adds) * U32
    err_log = rel + 4 * U32 * log_z
    w = float(dp.sum())
    err_w = U32 * float(torch.where(p > 0, dp * (4 * d + 8), 0).sum()) + w * (adds * U32 + rel)
    return (lambda y, lp: 2 * U32 * y + U32 * abs(lp) + err_log,
            err_log + err_w + 2 * U32 * (log_z + w), float(m))


def _check(x, tokens, top, it=1.0):
    lp, ent, ids, best = _run(x, tokens, top, it)
    want = ref.scores(x, tokens, top, it)
    assert torch.equal(ids, want[2])
    for a, b in ((lp, want[0]), (ent, want[1]), (best, want[3])):
        assert torch.equal(torch.isnan(a), torch.isnan(b))
        assert torch.equal(torch.isinf(a), torch.isinf(b))
    y = x.double().cpu()
    worst = 0.0
    for r in range(x.shape[0]):
        if not math.isfinite(float(y[r].max())):
            assert float(ent[r]) == 0 or math.isnan(float(ent[r]))
            continue
        bound, ent_bound, m = _row_bounds(y[r], it)
        worst = max(worst, abs(float(ent[r] - want[1][r])) / ent_bound)
        pairs = [(float(lp[r]), float(want[0][r]), int(tokens[r]))]
        pairs += [(float(best[r, i]), float(want[3][r, i]), int(want[2][r, i])) for i in range(top)]
        for got, exact, i in pairs:
            if math.isfinite(exact):
                worst = max(worst, abs(got - exact) / bound((m - float(y[r, i])) * it, exact))
    print("%.3g of the bounds" % worst, flush=True)
    assert worst <= 1, worst


def _logits(rows, vocab, kind, spread=3.0, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(rows, vocab, device="cuda", generator=g) * spread
    t = torch.randint(vocab, (rows,), device="cuda", generator=g, dtype=torch.int32)
    return x.to(TYPES[kind]), t


@pytest.mark.parametrize("rows,vocab", SIZES)
@pytest.mark.parametrize("kind,top,it", [("bf16", 20, 1.25), ("f32", 32, 0.75), ("f32", 1, 1.0)])
def test_scores(rows, vocab, kind, top, it):
    assert_many(rows, vocab)
    x, t = _logits(rows, vocab, kind)
    _check(x, t, top, it)


@pytest.mark.parametrize("rows,vocab", SIZES + [(3, 131072), (2, 600001)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("masked", [True, False])
def test_every_logit_counts_once(rows, vocab, kind, masked):
    """Row r holds equal logits at the ids that are r modulo some 150, and
    -inf or 60 less elsewhere: log Z is the logarithm of their number, to two
    ulp of it (sums of whole numbers are exact, and the others' weight is
    under 2^-60 each).  A logit lost or taken twice would move it by 1 /
    number.  The alternatives are the lowest of those ids."""
    rest = -math.inf if masked else -60.0
    mod = max(rows, vocab // 150)
    x = torch.full((rows, vocab), rest, device="cuda", dtype=TYPES[kind])
    ids = torch.arange(vocab, device="cuda")
    # (with fewer rows than residues, runs of residues: every id in some row)
    own = (ids % mod) * rows // mod if mod > rows else ids % rows
    for r in range(rows):
        x[r, own == r] = 2.0
    count = torch.bincount(own, minlength=rows).double().cpu()
    first = torch.tensor([int((own == r).nonzero()[0]) for r in range(rows)], dtype=torch.int32)
    lp, ent, top_ids, best = _run(x, first.cuda(), 20)
    log_z = torch.log(count)
    tol = 5 * U32 * log_z
    if vocab < 600001:
        assert (log_z - torch.log(count - 1) > 2 * tol).all()    # one logit lost
    assert ((lp.double() + log_z).abs() <= tol).all()
    assert ((best.double() + log_z[:, None]).abs() <= tol[:, None]).all()
    if masked:
        assert ((ent.double() - log_z).abs() <= tol).all()
    for r in range(rows):
        assert top_ids[r].tolist() == (own == r).nonzero()[:20, 0].tolist(), r


@pytest.mark.parametrize("rows,vocab", SIZES)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("top", [20, 32])
def test_ties(rows, vocab, kind, top):
    assert_many(rows, vocab)
    x = torch.zeros(rows, vocab, device="cuda")            # everything equal
    i = torch.arange(vocab, device="cuda")
    x[1::7, ::7] = 1.0
    x[2::7] = i % 5
    x[3::7] = -0.0
    x[3::7, ::2] = 0.0                                      # -0 equals 0
    x[4::7] = i / 1000.0                                    # ascending
    x[5::7] = -i / 1000.0
    x[6::7, PER - 3:PER + 3] = 2.0                          # over a border
    t = torch.arange(rows, device="cuda", dtype=torch.int32)
    _check(x.to(TYPES[kind]), t, top)


@pytest.mark.parametrize("rows,vocab", SIZES)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_masked_empty_and_bad_rows(rows, vocab, kind):
    assert_many(rows, vocab)
    x, t = _logits(rows, vocab, kind)
    low = torch.finfo(x.dtype).min
    x[0::14, 5:] = -math.inf            # five tokens left, fewer than the top
    x[1::14] = -math.inf                # nothing left
    x[2::14, 50] = math.nan
    x[3::14, vocab - 1] = math.inf
    x[4::14, 1:] = -math.inf            # one token left
    x[5::14] = low                      # the type's lowest value everywhere
    x[6::14, :vocab - 40] = low
    x[7::14, ::3] = -math.inf
    x[8::14, :PER] = -math.inf          # the first slice
    x[9::14, PER - 8:] = -math.inf      # every other slice
    x[10::14, :vocab - 3] = low
    x[11::14, vocab - 1] = -math.nan
    x[12::14, 9:] = low
    t[0::14], t[6::14], t[7::14] = 20, 3, 3
    for top in (4, 32):
        _check(x, t, top)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_rows_at_odd_offsets_and_strides(kind):
    rows, vocab = 130, 9001
    x, t = _logits(rows, vocab + 90, kind)
    for first in (1, 3, 6):
        part = x[:, first:first + vocab]
        assert_many(*part.shape)
        _check(part, t % vocab, 20)
    wide, _ = _logits(2 * rows, 16384, kind)
    _check(wide[::2], t, 32)


@pytest.mark.parametrize("rows,vocab", SIZES)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_without_alternatives(rows, vocab, kind):
    assert_many(rows, vocab)
    x, t = _logits(rows, vocab, kind)
    x[3::5, 11:] = -math.inf
    _check(x, t, 0, 1.25)

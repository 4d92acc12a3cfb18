"""gdn_token_scores against log probabilities in 64 bits."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import commit_gated_delta_amd as gdn  # noqa: E402
from tests import serving_ref as ref  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


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


def _check(x, tokens, top, it=1.0):
    got = _run(x, tokens, top, it)
    want = ref.scores(x, tokens, top, it)
    tol = ref.scores_bound(x, it)
    assert torch.equal(got[2], want[2])
    for a, b, what in ((got[0], want[0], "logprob"), (got[1], want[1], "entropy"),
                       (got[3], want[3], "best")):
        assert torch.equal(torch.isnan(a), torch.isnan(b)), what
        assert torch.equal(torch.isinf(a), torch.isinf(b)), what
        fine = torch.isfinite(b)
        err = (a.double() - b)[fine].abs()
        if err.numel():
            print("%s: %.3g of its bound" % (what, float(err.max()) / tol), flush=True)
            assert float(err.max()) <= tol, (what, float(err.max()), tol)


def _logits(rows, vocab, kind, spread=3.0, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(rows, vocab, device="cuda", generator=g) * spread
    t = torch.randint(vocab, (rows,), device="cuda", generator=g, dtype=torch.int32)
    return x.to(TYPES[kind]), t


@pytest.mark.parametrize("rows,vocab,top,kind,it", [
    (1, 1, 1, "f32", 1.0),
    (3, 2, 2, "bf16", 0.5),
    (5, 33, 32, "f32", 1.0),
    (2, 64, 0, "bf16", 1.0),
    (7, 1000, 5, "bf16", 2.0),
    (4, 4097, 20, "f32", 1.3),
    (1, 100003, 8, "bf16", 1.0),
    (2, 131072, 20, "f32", 0.8),
    (300, 5003, 3, "bf16", 1.0),
    (1, 262144, 32, "bf16", 1.0),
    (700, 1537, 1, "f32", 1.0),
    (2, 600001, 5, "bf16", 1.0),          # more slices than threads
    (53, 2214, 20, "bf16", 1.0),
    (3, 300007, 32, "f32", 1.0),
])
def test_scores(rows, vocab, top, kind, it):
    x, t = _logits(rows, vocab, kind)
    _check(x, t, top, it)


def test_ties_go_to_the_lowest_id():
    x = torch.zeros(4, 70001, device="cuda")            # everything equal
    x[1, ::7] = 1.0
    x[2] = torch.arange(70001, device="cuda") % 5
    x[3] = -0.0
    x[3, ::2] = 0.0                                      # -0 equals 0
    t = torch.zeros(4, dtype=torch.int32, device="cuda")
    for kind in ("bf16", "f32"):
        _check(x.to(TYPES[kind]), t, 32)
        _check(x.to(TYPES[kind])[:, :900], t, 20)


def test_slices_without_logits():
    """Slices of nothing but -inf between others, and too few logits left."""
    x, t = _logits(4, 40003, "bf16")
    x[0, 2000:30000] = -math.inf
    x[1, :39990] = -math.inf
    x[2, 7:] = -math.inf
    x[3, 1::2] = -math.inf
    _check(x, t, 32)
    _check(x.float(), t, 20)


def test_ascending_and_descending_rows():
    """The largest entries side by side at either end."""
    v = 50000
    up = torch.arange(v, device="cuda", dtype=torch.float32) / 1000
    x = torch.stack([up, up.flip(0)])
    _check(x, torch.tensor([v - 1, 5], dtype=torch.int32, device="cuda"), 32)


@pytest.mark.parametrize("vocab", [77, 20011, 140000])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_masked_empty_and_bad_rows(vocab, kind):
    x, t = _logits(8, vocab, kind)
    x[0, 5:] = -math.inf                # five tokens left, fewer than the top
    x[1] = -math.inf                    # nothing left
    x[2, 50] = math.nan
    x[3, vocab - 1] = math.inf
    x[4, 1:] = -math.inf                # one token left
    x[5] = torch.finfo(x.dtype).min     # the type's lowest value everywhere
    x[6, :40] = torch.finfo(x.dtype).min
    t[0], t[6] = 20, 3
    x[7, ::3] = -math.inf
    t[7] = 3
    _check(x[:5], t[:5], 20)
    _check(x[7:], t[7:], 20)
    lp, ent, ids, best = _run(x, t, 4)
    assert float(lp[0]) == -math.inf and float(lp[1]) == -math.inf
    # equal logits at the lowest value: a uniform row
    assert abs(float(ent[5]) - math.log(vocab)) < 1e-3
    assert ids[5].tolist() == [0, 1, 2, 3]
    assert float(lp[6]) < -1e30 and math.isfinite(float(ent[6]))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_whole_slices_at_the_lowest_value(kind):
    """All but one token masked with the type's lowest value: p = 1 for it,
    and nothing in the entropy from slices that hold nothing else."""
    x = torch.full((3, 140000), torch.finfo(TYPES[kind]).min, device="cuda", dtype=TYPES[kind])
    for r, i in enumerate((0, 70000, 139999)):
        x[r, i] = 2.0
    t = torch.tensor([0, 70000, 5], dtype=torch.int32, device="cuda")
    lp, ent, ids, best = _run(x, t, 2)
    assert ent.tolist() == [0, 0, 0] and lp[:2].tolist() == [0, 0]
    assert float(lp[2]) < -1e38 and best[:, 0].tolist() == [0, 0, 0]
    assert ids.tolist() == [[0, 1], [70000, 0], [139999, 0]]


@pytest.mark.parametrize("vocab", [5, 100, 20011])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_nan_of_either_sign(vocab, kind):
    x, t = _logits(4, vocab, kind)
    ints = x.view(torch.int16 if kind == "bf16" else torch.int32)
    plus, minus = (0x7fc0, 0x7fc0 - 2**15) if kind == "bf16" else (0x7fc00000, 0x7fc00000 - 2**31)
    ints[0] = plus
    ints[1] = minus
    ints[2, vocab // 2] = minus
    assert torch.isnan(x[:2]).all()
    _check(x, t, 5)


def test_given_tokens_that_are_not_in_the_vocabulary():
    x, _ = _logits(4, 300, "f32")
    t = torch.tensor([-1, 300, 299, -100], dtype=torch.int32, device="cuda")
    _check(x, t, 2)
    x[0, 0] = math.nan
    lp, ent, _, _ = _run(x, t, 2)
    assert float(lp[0]) == 0 and math.isnan(float(ent[0]))


@pytest.mark.parametrize("it", [1e-30, 1e-4, 1e4, 1e30])
def test_extreme_temperatures(it):
    x, t = _logits(3, 20000, "f32")
    x[1, ::2] = -math.inf
    lp, ent, ids, best = _run(x, t, 3, it)
    want = ref.scores(x, t, 3, it)
    assert torch.equal(ids, want[2])
    fine = torch.isfinite(want[0])
    assert torch.equal(torch.isfinite(lp), fine)
    assert float(((lp - want[0]).abs() / (1 + want[0].abs()))[fine].max()) < 1e-5
    assert float((ent - want[1]).abs().max()) < 1e-4


def test_sharp_and_flat_rows():
    x, t = _logits(4, 30000, "f32", spread=1.0)
    x[0] *= 40
    x[1] *= 1e-3
    x[2, 77] = 500.0
    t[2] = 77
    _check(x, t, 5)


def test_strided_rows_and_missing_outputs():
    x, t = _logits(6, 5000, "bf16")
    part = x[:, 1:4098]                 # rows at an odd offset and stride
    _check(part, t % 4000, 7)
    _check(x[::2], t[::2].contiguous(), 7)
    ws = torch.empty(gdn.token_scores_workspace_bytes(6, 5000, 3), dtype=torch.uint8, device="cuda")
    want = _run(x, t, 3)
    ent = torch.empty(6, device="cuda")
    gdn.token_scores(x, None, 0, None, ent, None, None, ws)
    assert torch.equal(ent.cpu(), want[1])
    lp = torch.empty(6, device="cuda")
    gdn.token_scores(x, t, 0, lp, None, None, None, ws)
    assert torch.equal(lp.cpu(), want[0])
    ids, best = torch.empty(6, 3, dtype=torch.int32, device="cuda"), torch.empty(6, 3, device="cuda")
    gdn.token_scores(x, None, 3, None, None, ids, best, ws)
    assert torch.equal(ids.cpu(), want[2]) and torch.equal(best.cpu(), want[3])


def test_rows_past_32_bits():
    """A row whose elements start past 2^31 of the logits."""
    stride = (1 << 31) + 8
    buf = torch.empty(stride + 5000, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (2, 5000), (stride, 1))
    y, t = _logits(2, 5000, "bf16")
    x.copy_(y)
    got, want = _run(x, t, 5), _run(y, t, 5)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_captured_calls_replay():
    x, t = _logits(3, 131072, "bf16")
    ws = torch.empty(gdn.token_scores_workspace_bytes(3, 131072, 6), dtype=torch.uint8, device="cuda")
    lp, ent = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    ids, best = torch.empty(3, 6, dtype=torch.int32, device="cuda"), torch.empty(3, 6, device="cuda")
    call = lambda: gdn.token_scores(x, t, 6, lp, ent, ids, best, ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(3):
        y, _ = _logits(3, 131072, "bf16", seed=i + 1)
        x.copy_(y)
        want = _run(x, t, 6)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((lp, ent, ids, best), want):
            assert torch.equal(a.cpu(), b), i

"""gdn_paged_attention where scores are -inf: such a position has no weight
beside others, and a token that sees nothing else has no softmax."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import commit_gated_delta_amd as gdn  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
U32 = 2.0 ** -24


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("length", [40, 3000])          # one split, and many
@pytest.mark.parametrize("T,h_q,d", [(1, 2, 64), (20, 2, 128), (3, 4, 256), (40, 2, 128),
                                     (16, 16, 64), (30, 2, 256)])
def test_scores_of_minus_infinity(T, h_q, d, length, kind):
    """Lane 0 holds keys whose every score is -inf for head 0 and for head 1
    whose scores are -inf in the first 2/3 only; lane 1's head 0 has -inf
    except at position 5; lane 2 has no page, and lane 3 -inf at the pages
    that it has."""
    page, n = 8, 4
    cols = -(-length // page)
    t = TYPES[kind]
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    k = torch.randn(n * cols, 2, page, d, device="cuda", generator=g).to(t)
    v = torch.randn(n * cols, 2, page, d, device="cuda", generator=g).to(t)
    q = torch.randn(n, T, h_q, d, device="cuda", generator=g).to(t)
    q[..., 0] = 1
    kl, vl = k.view(n, cols, 2, page, d), v.view(n, cols, 2, page, d)
    third = 2 * cols // 3
    kl[0, :, 0, :, 0] = -math.inf
    kl[0, :third, 1, :, 0] = -math.inf
    at5 = kl[1, 0, 0, 5].clone()
    kl[1, :, 0, :, 0] = -math.inf
    kl[1, 0, 0, 5] = at5
    kl[3, :, :, :, 0] = -math.inf
    table = torch.arange(n * cols, dtype=torch.int32, device="cuda").view(n, cols)
    table[2] = -1
    table[3, 1:] = -1
    kv_len = torch.full((n,), length, dtype=torch.int32, device="cuda")
    dims = gdn.KvDims.of(n, T, h_q, 2, d, page, n * cols, cols)
    o = torch.full((n, T, h_q, d), 7.0, device="cuda")
    ws = torch.empty(gdn.paged_attention_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    gdn.paged_attention(dims, [T] * n, q, k, v, table, kv_len, o, ws, scale=0.125)
    half = h_q // 2
    assert torch.isnan(o[0, :, :half]).all()
    # the rest of a lane whose first positions weigh nothing, in f64.  (The
    # bits are not those of a cache without them: the rows of a wave raise
    # their maxima together.)  In steps of 2^-24, a score is off by d + 8 of
    # the sum of its terms, the difference to a running maximum, 8 log 2 low
    # at most, and exp2: e; the output by e - sum p e of each position, by
    # three roundings (the parts of p) for each of a split's 128 positions,
    # one for each of 24 splits and 64 in their joins.
    first = third * page
    tail = length - T + torch.arange(T, device="cuda") >= first
    heads = slice(half, None)
    rest = [c[0, :, 1].reshape(-1, d)[first:length].double() for c in (kl, vl)]
    x = 0.125 * torch.matmul(q[0, tail, heads].double(), rest[0].t().contiguous())
    mag = 0.125 * torch.matmul(q[0, tail, heads].double().abs(), rest[0].t().contiguous().abs())
    at = torch.arange(first, length, device="cuda")
    sees = at <= (length - T + torch.arange(T, device="cuda")[tail])[:, None, None]
    x = torch.where(sees, x, -math.inf)
    p = torch.softmax(x, 2)
    e = torch.where(sees, U32 * ((d + 8) * mag + (x.amax(2, keepdim=True) - x).abs() + 16), 0)
    e = p * (e + (p * e).sum(2, keepdim=True))
    tol = torch.matmul(e + (3 * 128 + 24 + 64) * U32 * p, rest[1].abs())
    assert ((o[0, tail, heads].double() - torch.matmul(p, rest[1])).abs() <= tol).all()
    assert torch.isnan(o[0, ~tail, heads]).all()
    # one position left: its value (p = 1 exactly), where it is seen
    sees = length - T + torch.arange(T, device="cuda") >= 5
    assert torch.equal(o[1, sees, :half], vl[1, 0, 0, 5].float().expand(int(sees.sum()), half, d))
    assert torch.isnan(o[1, ~sees, :half]).all()
    assert torch.isfinite(o[1, :, half:]).all()
    assert (o[2] == 0).all()
    assert torch.isnan(o[3]).all()

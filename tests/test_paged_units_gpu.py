"""gdn_paged_attention where a split is several units of positions, so that
every wave takes several steps: each kernel in each type, the running maximum
raised along the cache, missing pages, infinities and NaN in later tiles; that
every position counts exactly once; and that the probabilities keep the 24
bits of f32."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import commit_gated_delta_amd as gdn  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
U32 = 2.0 ** -24
UNIT = 128                     # positions


class Case:
    """k, v [lanes][positions][h_kv][d] scattered over shuffled pages."""

    def __init__(self, q, k, v, lens, page, T):
        n, longest, h_kv, d = k.shape
        self.q, self.lens, self.h_kv, self.d, self.page = q, lens, h_kv, d, page
        cols = -(-longest // page)
        pages = n * cols + 3
        g = torch.Generator(device="cuda")
        g.manual_seed(5)
        self.table = torch.randperm(pages, device="cuda", generator=g)[:n * cols].view(n, cols).int()
        pad = cols * page - longest
        self.k, self.v = (torch.full((pages, h_kv, page, d), math.nan, device="cuda", dtype=k.dtype)
                          for _ in range(2))
        for c, x in ((self.k, k), (self.v, v)):
            x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)).view(n, cols, page, h_kv, d)
            c[self.table.long()] = x.transpose(2, 3)
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.dims = gdn.KvDims.of(n, T, q.shape[2], h_kv, d, page, pages, cols)

    def units(self):
        """Units of a split, from what the library says it needs: slots for
        twice the number of splits that are aimed at.  (It asks for bf16's
        splits; f32 may take fewer, up to three times as long.)"""
        need = gdn.paged_attention_workspace_bytes(self.dims)
        group = self.q.shape[2] // self.h_kv
        slots = need // (self.h_kv * self.dims.t_max * group * (self.d + 2) * 4)
        return -(-sum(-(-x // UNIT) for x in self.lens) // (slots // 2))

    def run(self, t_lane, scale):
        o = torch.full(self.q.shape, 7.0, device="cuda")
        ws = torch.empty(gdn.paged_attention_workspace_bytes(self.dims), dtype=torch.uint8,
                         device="cuda")
        gdn.paged_attention(self.dims, t_lane, self.q, self.k, self.v, self.table, self.kv_len,
                            o, ws, scale=scale)
        torch.cuda.synchronize()
        return o

    def visible(self, n, t_lane):
        """[t_lane, positions]: what the lane's tokens see."""
        pos = torch.arange(self.lens[n], device="cuda")
        page = self.table[n, pos // self.page].long()
        there = (page >= 0) & (page < self.dims.n_pages)
        ends = self.lens[n] - t_lane + torch.arange(t_lane, device="cuda")
        return there & (pos <= ends[:, None])

    def rows(self, cache, n):
        """[h_kv, positions, d] in f64; zeros where there is no page."""
        pos = torch.arange(self.lens[n], device="cuda")
        page = self.table[n, pos // self.page].long()
        there = (page >= 0) & (page < self.dims.n_pages)
        x = cache[page.clamp(0, self.dims.n_pages - 1), :, pos % self.page].double()
        return torch.where(there[:, None, None], x, 0).transpose(0, 1).contiguous()

    def check(self, o, t_lane, scale):
        """Against softmax in f64.  A score is off by a rounding per term of
        its sum and a few more of its size, (d + 8) U32 sum |q k| |scale|, by
        the subtraction of the running maximum, which is at most 8 log 2 below
        the largest score so far, and by exp2 (one ulp): e_i.  The output is
        then off by sum p_i (e_i + sum p e) |v_i|, by at most three roundings
        (the parts of P; f32 has one part and longer splits) per position of a
        split, one per split and 64 for the rescalings of its joins, relative
        to sum p |v|."""
        split = UNIT * self.units()
        for n, m in enumerate(t_lane):
            assert (o[n, m:] == 7).all()
            k, v = self.rows(self.k, n), self.rows(self.v, n)
            group = self.q.shape[2] // self.h_kv
            sees = self.visible(n, m).repeat_interleave(group, 0)
            worst = 0.0
            for h in range(self.h_kv):
                q = self.q[n, :m, h * group:(h + 1) * group].double().reshape(m * group, -1)
                kt = k[h].t().contiguous()
                x = scale * torch.matmul(q, kt)
                xa = abs(scale) * torch.matmul(q.abs(), kt.abs())
                x = torch.where(sees, x, -math.inf)
                top = x.amax(1, keepdim=True)
                p = torch.exp(x - top)
                p = p / p.sum(1, keepdim=True)
                e = torch.where(sees, U32 * ((self.d + 8) * xa + (top - x).abs() + 16), 0)
                e = p * (e + (p * e).sum(1, keepdim=True))
                want = torch.matmul(p, v[h])
                va = v[h].abs()
                steps = 3 * split + self.lens[n] / split + 64
                tol = torch.matmul(e, va) + steps * U32 * torch.matmul(p, va) + 1e-30
                got = o[n, :m, h * group:(h + 1) * group].double().reshape(m * group, -1)
                assert torch.isfinite(got).all(), (n, h)
                worst = max(worst, float(((got - want).abs() / tol).max()))
            print("lane %d: %.3g of its bound" % (n, worst), flush=True)
            assert worst <= 1, (n, worst)


def _heads(rows, d, kind):
    """Key-value heads that leave about 32 splits for a call."""
    size = 2 if kind == "bf16" else 4
    if rows <= (32 if d < 256 else 16):
        return 64 if d * size < 512 else 8
    return 16 if rows <= 64 or d < 256 and rows <= 128 else 8


# tokens a lane, group, d, type: every kernel of the library
SHAPES = [(T, group, d, kind)
          for kind in ("bf16", "f32")
          for T, group, d in ((1, 8, 64), (3, 3, 64), (5, 4, 64), (10, 4, 64), (20, 5, 64),
                              (1, 5, 128), (7, 4, 128), (9, 5, 128), (16, 8, 128), (33, 4, 128),
                              (1, 16, 256), (2, 4, 256), (5, 5, 256), (16, 6, 256))]


def _random(T, group, d, kind, lens=(5000, 3111), page=24, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h_kv = _heads(T * group, d, kind)
    n = len(lens)
    make = lambda *s: torch.randn(s, device="cuda", generator=g).to(TYPES[kind])
    return make(n, T, h_kv * group, d), make(n, max(lens), h_kv, d), make(n, max(lens), h_kv, d), h_kv


@pytest.mark.parametrize("T,group,d,kind", SHAPES)
def test_several_units_a_split(T, group, d, kind):
    lens = [5000, 3111]
    q, k, v, _ = _random(T, group, d, kind, lens)
    x = Case(q, k, v, lens, 24, T)
    assert x.units() >= 2
    x.table[0, 40] = -1                    # positions 960 .. 983
    x.table[0, 100:140] = x.dims.n_pages   # more than a split
    x.table[1, 7] = 1 << 30
    t_lane = [T, max(1, T - 1)]
    x.check(x.run(t_lane, d ** -0.5), t_lane, d ** -0.5)


@pytest.mark.parametrize("T,group,d,kind", SHAPES)
@pytest.mark.parametrize("up", [True, False])
def test_scores_that_rise_or_fall_along_the_cache(T, group, d, kind, up):
    """By 2^160 over the cache, 2^12 and more within a split, so that the
    maximum is raised again and again (or never after the first step)."""
    lens = [5000, 3111]
    q, k, v, _ = _random(T, group, d, kind, lens)
    q.mul_(0.25)
    q[..., 0] = 1
    ramp = torch.arange(max(lens), device="cuda") * (160 * math.log(2) / max(lens))
    if not up:
        ramp = ramp.flip(0)
    k.mul_(0.25)
    k[..., 0] = ramp[None, :, None].to(k.dtype)
    x = Case(q, k, v, lens, 24, T)
    assert x.units() >= 2
    x.check(x.run([T, T], 1.0), [T, T], 1.0)


@pytest.mark.parametrize("T,group,d,kind", SHAPES)
@pytest.mark.parametrize("page", [1, 24, 256])
def test_every_position_counts_once(T, group, d, kind, page):
    """Equal scores and value rows that are 1 in column (position mod d): an
    output is the number of seen positions of its column over that of all.
    Probabilities and sums are whole numbers, so only the quotient (1 / l to
    2.5 ulp, then one product) is rounded; a position lost or taken twice
    would be off by d / length, over 1e-2."""
    lens = [5000, 3111] if page != 1 else [1025, 643]
    h_kv = _heads(T * group, d, kind)
    pos = torch.arange(max(lens), device="cuda")
    v = torch.nn.functional.one_hot(pos % d, d).to(TYPES[kind])[None, :, None].expand(
        2, -1, h_kv, -1).contiguous()
    k = torch.randn(v.shape, device="cuda").to(TYPES[kind])
    q = torch.zeros(2, T, h_kv * group, d, device="cuda", dtype=TYPES[kind])
    x = Case(q, k, v, lens, page, T)
    x.table[0, x.table.shape[1] // 3] = -1
    o = x.run([T, T], 0.5).double()
    for n in range(2):
        sees = x.visible(n, T).double()
        count = torch.matmul(sees, torch.nn.functional.one_hot(pos[:lens[n]] % d, d).double())
        want = (count / sees.sum(1, keepdim=True))[:, None]
        # (one position of the last column lost)
        lost = count[:, -1] - 1, sees.sum(1) - 1
        assert (lost[0] / lost[1] < want[:, 0, -1] * (1 - 1e-3)).all()
        assert ((o[n] - want).abs() <= 6 * U32 * want).all(), n


@pytest.mark.parametrize("T,group,d,kind", SHAPES)
def test_infinities_and_nan_in_later_tiles(T, group, d, kind):
    """Value rows deep in a split: they reach their own columns and heads of
    the tokens that see them, and change nothing else."""
    lens = [5000, 3111]
    q, k, v, h_kv = _random(T, group, d, kind, lens)
    t_lane = [T, T]
    x = Case(q, k, v, lens, 24, T)
    clean = x.run(t_lane, 0.1)
    at = [300, 301, 2222, 4999 - T // 2]
    for pos in at:
        page, row = int(x.table[0, pos // 24]), pos % 24
        x.v[page, 1, row, 3] = math.inf
        x.v[page, 1, row, 10] = math.nan
        x.v[page, 1, row, d - 1] = -math.inf
    o = x.run(t_lane, 0.1)
    mine = torch.zeros_like(o, dtype=torch.bool)
    for c in (3, 10, d - 1):
        mine[0, :, group:2 * group, c] = True
    assert torch.equal(o[~mine], clean[~mine])
    own = o[0, :, group:2 * group]
    assert (own[..., 3] == math.inf).all() and (own[..., d - 1] == -math.inf).all()
    assert torch.isnan(own[..., 10]).all()
    # behind the window's middle only: the tokens before it do not see it
    x = Case(q, k, v, lens, 24, T)
    page, row = int(x.table[0, at[3] // 24]), at[3] % 24
    x.v[page, 1, row, 3] = math.inf
    o = x.run(t_lane, 0.1)
    first = T - 1 - T // 2                   # the first token that does
    assert torch.equal(o[0, :first], clean[0, :first])
    assert (o[0, first:, group:2 * group, 3] == math.inf).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,group,d", [(1, 2, 64), (20, 1, 64), (1, 4, 128), (10, 4, 128),
                                       (16, 8, 128), (1, 3, 256), (8, 4, 256)])
def test_probabilities_keep_24_bits(T, group, d, kind):
    """Value rows that pick one position each, so that an output is that
    position's p.  Scores a b are exact.  In steps of 2^-24: the argument
    x log2 e of exp2, at most 8, takes a rounding from scale log2 e, the
    product and the difference to the maximum each, exp2 two (one ulp), 3 * 8
    log 2 + 2 < 19; the weight of a split 8 log 2 + 3 < 9; both in p and in
    the sum of p, which adds at most 8 terms a lane and step over four steps,
    2 lane groups and 6 levels of a wave, 40; the quotient 6 and the rescaling
    of an output 2: 2 (19 + 9) + 48 = 104.  Two bf16 parts of p would be off
    by up to 510 and by 190 in the mean."""
    length = d
    t = TYPES[kind]
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    a = 1 + torch.rand(1, T, 2 * group, device="cuda", generator=g)
    b = 2.7 * torch.rand(1, length, 2, device="cuda", generator=g)
    q = torch.zeros(1, T, 2 * group, d, device="cuda", dtype=t)
    k = torch.zeros(1, length, 2, d, device="cuda", dtype=t)
    q[..., 5] = a.bfloat16().to(t)           # (products of 16 bits)
    k[..., 5] = b.bfloat16().to(t)
    v = torch.eye(d, device="cuda", dtype=t)[None, :, None].expand(1, -1, 2, -1).contiguous()
    x = Case(q, k, v, [length], 16, T)
    o = x.run([T], 1.0).double()[0]          # [T, heads, position]
    s = q[0, :, :, 5].double()[..., None] * k[0, :, :, 5].double().t().repeat_interleave(group, 0)
    s = torch.where(x.visible(0, T)[:, None], s, -math.inf)
    assert float(s.max()) * math.log2(math.e) <= 8
    want = torch.softmax(s, 2)
    two = (torch.exp(s - s.amax(2, keepdim=True)).float().view(torch.int32) & ~255).view(torch.float32)
    two = two.double() / two.double().sum(2, keepdim=True)
    assert not ((two - want).abs() <= 104 * U32 * want).all()      # two parts would not do
    assert ((o - want).abs() <= 104 * U32 * want).all(), float(
        ((o - want).abs() / want.clamp(min=1e-9)).max() / U32)

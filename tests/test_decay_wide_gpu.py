"""gdn_decay_prefill where a workgroup takes 128 columns of d_v, as in every
large prompt: both types, rows of any length, segments of several chunks,
states alone, infinities and NaN; and the exactness of its f32 operands."""
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
# one segment each (all but one of them one to four chunks long), and
# sequences of several segments of six chunks, with ragged ends
SHORT = [65, 0, 130, 1, 64, 200, 33, 5, 129, 250, 17, 96, 66, 2, 3, 31, 190]
LONG = [3000, 1, 700, 2049]


def segments(lens, h_v, h_k, d_k, d_v):
    """Segments of a call, from its workspace (a state and a decay per head
    and segment, none where every sequence is one segment)."""
    need = gdn.decay_prefill_workspace_bytes(lens, h_v, h_k, d_k, d_v)
    return need // (h_v * (d_k * d_v + 1) * 4) or len(lens)


def assert_wide(lens, h_v, h_k, d_k, d_v):
    """Narrow workgroups are for calls of less than one wide one per CU; two
    and more per CU are never narrow."""
    n = segments(lens, h_v, h_k, d_k, d_v)
    assert d_v > 64 and n * h_v * -(-d_v // 128) >= 512, n
    return n


class Prompt:
    def __init__(self, lens, h_v, h_k, d_k, d_v, kind, per_head=False, init=True, seed=0):
        self.shape = (h_v, h_k, d_k, d_v)
        self.lens, self.per_head, self.scale = lens, per_head, 0.25
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        n, t = sum(lens), TYPES[kind]
        rand = lambda *s: torch.randn(s, device="cuda", generator=g)
        self.q, self.k = rand(n, h_k, d_k).to(t), rand(n, h_k, d_k).to(t)
        self.v = rand(n, h_v, d_v).to(t)
        self.g = -torch.nn.functional.softplus(rand(h_v) if per_head else rand(n, h_v)) / 8
        self.S0 = rand(len(lens), h_v, d_k, d_v) if init else None

    def run(self, want_o=True, want_s=True, S_final=None):
        h_v, h_k, d_k, d_v = self.shape
        ws = torch.empty(gdn.decay_prefill_workspace_bytes(self.lens, *self.shape),
                         dtype=torch.uint8, device="cuda")
        o = torch.full((sum(self.lens), h_v, d_v), math.nan, device="cuda") if want_o else None
        S = S_final
        if S is None and want_s:
            S = torch.full((len(self.lens), h_v, d_k, d_v), math.nan, device="cuda")
        gdn.decay_prefill(self.lens, h_v, h_k, d_k, d_v, self.q if want_o else None, self.k,
                          self.v, self.g, self.S0, S, o, ws, scale=self.scale,
                          head_decay=self.per_head)
        torch.cuda.synchronize()
        return o, S

    def reference(self, i, at):
        """o, S of sequence i and the sums of their terms' absolute values."""
        h_v, h_k, d_k, d_v = self.shape
        T = self.lens[i]
        rep = lambda y: y[at:at + T].double().repeat_interleave(h_v // h_k, 1)
        g = self.g.expand(T, h_v) if self.per_head else self.g[at:at + T]
        S0 = self.S0[i] if self.S0 is not None else torch.zeros(h_v, d_k, d_v, device="cuda")
        return ref.decay_chain(rep(self.q), rep(self.k), self.v[at:at + T], g, S0, self.scale)

    def check(self, o, S, only=None):
        at = 0
        for i, T in enumerate(self.lens):
            wo, wS, mo, mS = self.reference(i, at)
            rel = ref.decay_bound(self.shape[2], T)
            for got, want, mag, what in ((o[at:at + T], wo, mo, "o"), (S[i], wS, mS, "S")):
                ok = torch.ones_like(got, dtype=torch.bool)
                if only is not None:
                    ok = only[0][at:at + T] if what == "o" else only[1][i]
                assert torch.isfinite(got[ok]).all(), (what, i)
                err = ((got.double() - want).abs() / (rel * mag + 1e-30))[ok]
                worst = float(err.max()) if err.numel() else 0.0
                print("%s of sequence %d: %.3g of its bound" % (what, i, worst), flush=True)
                assert worst <= 1, (what, i, worst)
            at += T


@pytest.mark.parametrize("lens,h_v,h_k,d_k,d_v,kind,per_head,init", [
    (SHORT, 32, 16, 128, 128, "bf16", False, True),
    (SHORT, 32, 32, 128, 100, "bf16", False, False),
    (SHORT, 32, 8, 64, 128, "f32", False, True),
    (SHORT, 32, 16, 128, 101, "f32", True, True),
    (SHORT, 32, 32, 32, 72, "bf16", True, False),
    (SHORT, 32, 4, 16, 130, "bf16", False, True),
    (SHORT, 16, 16, 16, 256, "f32", False, False),
    (SHORT, 32, 16, 64, 65, "f32", False, True),
    (LONG, 32, 8, 128, 128, "bf16", False, True),
    (LONG, 32, 32, 128, 100, "bf16", True, False),
    (LONG, 32, 16, 128, 130, "bf16", False, False),
    (LONG, 32, 16, 128, 128, "f32", False, True),
    (LONG, 32, 16, 64, 104, "f32", False, False),
    (LONG, 32, 32, 32, 99, "f32", True, True),
    (LONG, 32, 16, 16, 128, "bf16", False, True),
])
def test_prompts(lens, h_v, h_k, d_k, d_v, kind, per_head, init):
    n = assert_wide(lens, h_v, h_k, d_k, d_v)
    assert (n > len(lens)) == (lens is LONG)
    x = Prompt(lens, h_v, h_k, d_k, d_v, kind, per_head, init)
    x.check(*x.run())


@pytest.mark.parametrize("lens", [SHORT, LONG])
@pytest.mark.parametrize("d_k,d_v,kind", [(128, 128, "bf16"), (128, 100, "bf16"),
                                          (128, 128, "f32"), (64, 99, "f32")])
def test_states_alone_outputs_alone_and_in_place(lens, d_k, d_v, kind):
    assert_wide(lens, 32, 16, d_k, d_v)
    x = Prompt(lens, 32, 16, d_k, d_v, kind)
    o, S = x.run()
    assert torch.equal(x.run(want_o=False)[1], S)
    assert torch.equal(x.run(want_s=False)[0], o)
    x.S0 = x.S0.clone()
    o2, S2 = x.run(S_final=x.S0)
    assert torch.equal(o2, o) and torch.equal(S2, S)


@pytest.mark.parametrize("lens,seq,t", [(SHORT, 9, 130), (LONG, 0, 1000), (LONG, 3, 2048)])
@pytest.mark.parametrize("d_k,d_v,kind", [(128, 128, "bf16"), (128, 100, "bf16"),
                                          (128, 128, "f32"), (64, 99, "f32")])
def test_infinities_and_nan(lens, seq, t, d_k, d_v, kind):
    """In a value row of token t of a sequence: its columns hold them from
    the token on; what is before it, and every other column, head and
    sequence, is what it would be without."""
    assert_wide(lens, 32, 16, d_k, d_v)
    x = Prompt(lens, 32, 16, d_k, d_v, kind)
    at = sum(lens[:seq])
    cols = (5, 90)
    keep = (torch.ones(sum(lens), 32, d_v, dtype=torch.bool, device="cuda"),
            torch.ones(len(lens), 32, d_k, d_v, dtype=torch.bool, device="cuda"))
    for c in cols:
        keep[0][at + t:at + lens[seq], 3, c] = False
        keep[1][seq, 3, :, c] = False
    clean = x.v.clone()
    x.v[at + t, 3, 5] = math.inf
    x.v[at + t, 3, 90] = math.nan
    o, S = x.run()
    x.v = clean
    x.check(o, S, keep)
    assert not torch.isfinite(o[at + t:at + lens[seq], 3, 5]).any()
    assert torch.isnan(o[at + t:at + lens[seq], 3, 90]).all()
    assert not torch.isfinite(S[seq, 3, :, 5]).any() and torch.isnan(S[seq, 3, :, 90]).all()


# ------------------------------------------------------------- exactness
# f32 operands (state, P, W) keep their 24 bits in every product.  Two bf16
# parts would lose the last 8: up to 2^-16 of a value.
EXACT = [(128, 128, "bf16"), (128, 104, "bf16"), (128, 100, "bf16"), (64, 128, "f32"),
         (128, 101, "f32"), (128, 64, "bf16"), (128, 40, "f32")]


@pytest.mark.parametrize("lens", [SHORT, LONG])
@pytest.mark.parametrize("d_k,d_v,kind", EXACT)
def test_a_query_picks_a_state_row_exactly(lens, d_k, d_v, kind):
    """No decay, zero keys and a unit query: the outputs are rows of the
    initial state, bit for bit, over all chunks and segments."""
    x = Prompt(lens, 32, 32, d_k, d_v, kind)
    x.k.zero_()
    x.g.zero_()
    x.scale = 1.0
    n = sum(lens)
    row = (torch.arange(n, device="cuda")[:, None] * 7 + torch.arange(32, device="cuda")) % d_k
    x.q = torch.nn.functional.one_hot(row, d_k).to(TYPES[kind])
    o, S = x.run()
    assert torch.equal(S, x.S0)
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"),
                                  torch.tensor(lens, device="cuda"))
    want = x.S0[seq[:, None], torch.arange(32, device="cuda"), row]
    assert torch.equal(o, want)


@pytest.mark.parametrize("d_k,d_v,kind", EXACT)
def test_scores_of_24_bits_pass_exactly(d_k, d_v, kind):
    """No decay; q.k = a + b u with a of 8 bits and b u of 16 below them, 24
    bits in all; token s writes column s alone, so that an output is one
    score, through P in its own chunk and through the state in the next."""
    lens = [min(d_v, 100), 1, min(d_v, 64)] * 6
    n, t = sum(lens), TYPES[kind]
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = Prompt(lens, 32, 32, d_k, d_v, kind, init=False)
    whole = lambda *s: torch.randint(128, 256, s, device="cuda", generator=g).double()
    a, b, u = whole(n, 32) / 128, (whole(n, 32).long() | 1) / 128.0, (whole(n, 32).long() | 1) / 65536.0
    x.q, x.k, x.v = (torch.zeros(n, 32, d, device="cuda", dtype=t) for d in (d_k, d_k, d_v))
    x.q[..., 3], x.q[..., d_k - 2] = a.to(t), b.to(t)
    x.k[..., 3], x.k[..., d_k - 2] = 1, u.to(t)
    x.g.zero_()
    x.scale = 1.0
    want = torch.zeros(n, 32, d_v, dtype=torch.float64, device="cuda")
    at = 0
    for T in lens:
        for s in range(T):
            c = s % d_v
            x.v[at + s, :, c] = 1
            want[at + s:at + T, :, c] += a[at + s:at + T] + b[at + s:at + T] * u[at + s]
        at += T
    if d_v > 64:
        assert_wide(lens, 32, 32, d_k, d_v)
    assert torch.equal(want.float().double(), want)
    o, S = x.run()
    assert torch.equal(o.double(), want)


@pytest.mark.parametrize("lens", [SHORT, LONG])
@pytest.mark.parametrize("d_k,d_v,kind", EXACT)
def test_written_values_keep_24_bits(lens, d_k, d_v, kind):
    """Unit keys and positive values: a state entry is a sum of positive
    terms v exp(sum g).  In steps of 2^-24: a term's exponentials, of sums
    below 4 in all, are off by 4 for their arguments and by 3 each with the
    product they enter; there are two for its own chunk and one for every
    later chunk of a segment (of six) and every segment (of eight).  An
    addition per T / d_k tokens and part of the value, one per such chunk and
    segment."""
    if lens is LONG:
        assert segments(lens, 32, 32, d_k, d_v) == 8 + 1 + 2 + 6
    x = Prompt(lens, 32, 32, d_k, d_v, kind, init=False)
    n = sum(lens)
    x.g = -torch.rand(n, 32, device="cuda") * 4 / max(lens)
    row = (torch.arange(n, device="cuda")[:, None] + torch.arange(32, device="cuda")) % d_k
    x.k = torch.nn.functional.one_hot(row, d_k).to(TYPES[kind])
    x.v = x.v.abs() + 0.5
    _, S = x.run()
    at = 0
    for i, T in enumerate(lens):
        w = torch.exp(x.g[at:at + T].double().flip(0).cumsum(0).flip(0) - x.g[at:at + T].double())
        want = torch.zeros(32, d_k, d_v, dtype=torch.float64, device="cuda")
        head = torch.arange(32, device="cuda").expand(T, 32)
        want.index_put_((head, row[at:at + T]), w[..., None] * x.v[at:at + T].double(),
                        accumulate=True)
        steps = 4 + 3 * (2 + 6 + 8) + (3 if kind == "bf16" else 1) * T / d_k + 6 + 8
        err = (S[i].double() - want).abs() / (steps * U32 * want + 1e-30)
        assert float(err.max()) <= 1, (i, float(err.max()))
        if lens is SHORT and T >= d_k:       # two parts of a sum of one or two terms
            two = (want.float().view(torch.int32) & ~255).view(torch.float32).double()
            assert ((two - want).abs() > steps * U32 * want).any()
        at += T

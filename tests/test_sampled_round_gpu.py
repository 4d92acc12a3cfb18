"""The rotated 4-bit cache, the attention that reads it and the verification
of sampled drafts together: a two-layer hybrid model (linear attention with a
decay per head, then attention over the cache) run as a server runs it,
prompts in windows, then rounds of drafts whose accepted prefix is committed.

Checked in 64 bits: every row of the cache is a right code of the model's own
key or value, the logits are those of the model over the cache's decoded rows,
and a round's prefix and next token are what the definition makes of them.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import commit_gated_delta_amd as gdn  # noqa: E402
from tests import cache_ref as ref  # noqa: E402

E, HV, HK, D, HQ, HKV, V, ROT = 96, 4, 2, 64, 6, 2, 700, 32
# Relative to the largest magnitude: a logit is some 1250 roundings of 2^-24
# away from its inputs (sums of 96, 256, 384 and 96 terms, a state and a
# softmax over 60 positions, products of 64), and a sum's terms are together
# about 13 times what it comes to (the square root of their number).
NEAR = 2.0 ** -10


class Model:
    def __init__(self, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        w = lambda *s: torch.randn(s, device="cuda", generator=g) / s[0] ** 0.5
        self.embed = w(V, E) * V ** 0.5
        self.q, self.k, self.v = w(E, HK * D), w(E, HK * D), w(E, HV * D)
        self.g, self.out = w(E, HV), w(HV * D, E)
        # queries, keys and values of the attention layer in one product
        self.qkv = w(E, (HQ + 2 * HKV) * D)
        self.aout, self.head = w(HQ * D, E), w(E, V) * 2
        self.freq = 500.0 ** (-torch.arange(ROT // 2, device="cuda") * 2.0 / ROT)

    def decay_inputs(self, x):
        s = x.shape[:-1]
        return ((x @ self.q).view(*s, HK, D), (x @ self.k).view(*s, HK, D) / 8,
                (x @ self.v).view(*s, HV, D),
                -torch.nn.functional.softplus(x @ self.g - 2))

    def double(self):
        m = object.__new__(Model)
        m.__dict__ = {k: w.double().cpu() for k, w in self.__dict__.items()}
        m.freq = self.freq.cpu()
        return m

    def first_layer(self, tokens):
        """Hidden rows after the decay layer, token by token in f64."""
        m, S, out = self.double(), torch.zeros(HV, D, D, dtype=torch.float64), []
        for t in tokens:
            x = m.embed[t]
            q, k, v, g = m.decay_inputs(x)
            k, q = (y.repeat_interleave(HV // HK, 0) for y in (k, q))
            S = torch.exp(g)[:, None, None] * S + k[:, :, None] * v[:, None, :]
            out.append(x + (q[:, :, None] * S).sum(1).reshape(-1) @ m.out)
        return torch.stack(out), S

    def second_layer(self, x, K, W):
        """Logits from all hidden rows x [L, E] over the cache's rows K, W
        [L, HKV, D]; the keys and values that the cache is to hold."""
        m, L = self.double(), len(x)
        y = (x @ m.qkv).view(L, HQ + 2 * HKV, D)
        y[:, :HQ + HKV] = ref.turned(y[:, :HQ + HKV], torch.arange(L), m.freq, ROT, False)[0]
        q, k, v = y.split((HQ, HKV, HKV), 1)
        K, W = (r.repeat_interleave(HQ // HKV, 1) for r in (K, W))
        s = torch.einsum("ihd,jhd->hij", q, K) * D ** -0.5
        s = s.masked_fill(torch.ones(L, L).triu(1).bool(), -torch.inf)
        o = torch.einsum("hij,jhd->ihd", torch.softmax(s, 2), W)
        return (x + o.reshape(L, -1) @ m.aout) @ m.head, k, v


class Server:
    def __init__(self, model, N, T, page=8, cols=9):
        self.m, self.N, self.T, self.page = model, N, T, page
        self.S = torch.zeros(1, N, HV, D, D, device="cuda")
        self.kv = gdn.KvDims.of(N, T, HQ, HKV, D, page, N * cols, cols)
        # what was in the pages before: blocks of NaN
        self.cache = [torch.full((N * cols, HKV, page, D // w), 255, dtype=torch.uint8, device="cuda")
                      for w in (2, 32, 2, 32)]
        self.table = torch.randperm(N * cols, device="cuda").view(N, cols).int()
        size = max(gdn.paged_attention_mxfp_workspace_bytes(self.kv), gdn.draft_verify_workspace_bytes(N, T, V))
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        self.dims = gdn.Dims.of(1, N, HV, HK, D, D, T)
        self.length = [0] * N

    def forward(self, windows):
        """Logits [N, T, V] of the windows' rows; nothing is committed."""
        t_lane = [len(w) for w in windows]
        tok = torch.zeros(self.N, self.T, dtype=torch.long, device="cuda")
        for n, w in enumerate(windows):
            tok[n, :len(w)] = torch.tensor(w, dtype=torch.long)
        x = self.m.embed[tok]
        self.step = [y[None].contiguous() for y in self.m.decay_inputs(x)]
        o = torch.zeros(1, self.N, self.T, HV, D, device="cuda")
        gdn.decay_step(self.dims, t_lane, *self.step, self.S, o, keep_state=True)
        x = x + o.view(self.N, self.T, -1) @ self.m.out
        y = (x @ self.m.qkv).view(self.N, self.T, HQ + 2 * HKV, D)
        q, k, v = y.split((HQ, HKV, HKV), 2)
        kv_len = torch.tensor([a + b for a, b in zip(self.length, t_lane)], dtype=torch.int32, device="cuda")
        turned = torch.zeros(self.N, self.T, HQ, D, device="cuda")
        gdn.rope_append_mxfp(self.kv, t_lane, q, k, v, self.m.freq, ROT, turned, *self.cache, self.table, kv_len)
        o = torch.zeros(self.N, self.T, HQ, D, device="cuda")
        gdn.paged_attention_mxfp(self.kv, t_lane, turned, *self.cache, self.table, kv_len, o, self.ws,
                                 scale=D ** -0.5)
        return (x + o.view(self.N, self.T, -1) @ self.m.aout) @ self.m.head

    def verify(self, windows, logits, drafted, uniforms, it):
        tok = torch.full((self.N, self.T), -1, dtype=torch.int32, device="cuda")
        for n, w in enumerate(windows):
            tok[n, :len(w)] = torch.tensor(w, dtype=torch.int32)
        m, nxt = (torch.full((self.N,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
        gdn.draft_verify([len(w) for w in windows], logits, drafted, tok, uniforms, it, m, nxt, self.ws)
        return tok, m.tolist(), nxt.tolist()

    def commit(self, m):
        q, k, v, g = self.step
        gdn.decay_step(self.dims, m, None, k, v, g, self.S, None)
        self.length = [a + b for a, b in zip(self.length, m)]

    def rows(self, n, length):
        """Codes and scales of lane n's keys and values, [length, HKV, ..]."""
        pos = torch.arange(length, device="cuda")
        pages = self.table[n, pos // self.page].long()
        return [c[pages, :, pos % self.page].cpu() for c in self.cache]


def check_lane(srv, n, text, logits):
    """The cache of all of `text` and the logits of its last rows."""
    x, _ = srv.m.first_layer(text)
    kc, ks, vc, vs = srv.rows(n, len(text))
    K, W = ref.decode(kc, ks), ref.decode(vc, vs)
    want, k, v = srv.m.second_layer(x, K, W)
    for own, c, s in ((k, kc, ks), (v, vc, vs)):
        assert ref.held_ok(own, torch.full_like(own, NEAR * float(own.abs().max())), c, s), n
    want = want[len(text) - len(logits):]
    off = float((logits.cpu().double() - want).abs().max() / want.abs().max())
    print("lane %d, %d tokens: logits off by %.2g" % (n, len(text), off), flush=True)
    assert off <= NEAR


@pytest.mark.parametrize("given", [True, False])  # the drafter's distribution
def test_sampled_rounds_agree_with_the_model(given):
    torch.manual_seed(7)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    model, N, T = Model(23), 3, 6
    srv = Server(model, N, T)
    it = torch.tensor([1.0, 0.6, 3.0], device="cuda")
    prompts = [torch.randint(V, (n,)).tolist() for n in (1, 20, 9)]
    # all but each prompt's last token, in windows; that one is the first anchor
    done = [0] * N
    while any(a < len(p) - 1 for a, p in zip(done, prompts)):
        windows = [p[a:len(p) - 1][:T] for a, p in zip(done, prompts)]
        logits = srv.forward(windows)
        srv.commit([len(w) for w in windows])
        for n, w in enumerate(windows):
            done[n] += len(w)
            if w:
                check_lane(srv, n, prompts[n][:done[n]], logits[n, :len(w)])
    text, anchor = [p[:-1] for p in prompts], [p[-1] for p in prompts]
    for drafts in ([5, 3, 0], [2, None, 5], [4, 5, 1], [5, 5, 5]):  # None: idle
        windows, drafted = [], torch.zeros(N, T - 1, V, device="cuda")
        for n, count in enumerate(drafts):
            w = [] if count is None else [anchor[n]]
            for t in range(count or 0):
                # the drafter: the first layer alone, sampled as the model is
                x = model.first_layer(text[n] + w)[0][-1].float().cuda() @ model.head
                drafted[n, t] = x
                w.append(int(torch.multinomial(torch.softmax(x * it[n], 0), 1, generator=g)))
            windows.append(w)
        logits = srv.forward(windows)
        uniforms = torch.rand(N, T, device="cuda", generator=g)
        tok, m, nxt = srv.verify(windows, logits, drafted if given else None, uniforms, it)
        t_lane = [len(w) for w in windows]
        want = ref.verify(t_lane, logits, drafted if given else None, tok, uniforms, it)
        for n, w in enumerate(windows):
            if not w:
                assert (m[n], nxt[n]) == (-7, -7)
                m[n] = 0
                continue
            check_lane(srv, n, text[n] + w, logits[n, :len(w)])
            assert want[n][3] or (m[n], nxt[n]) == want[n][:2], (n, m[n], nxt[n], want[n])
            text[n] += w[:m[n]]
            anchor[n] = nxt[n]
        print("accepted", m, "of", t_lane, flush=True)
        srv.commit(m)
        assert srv.length == [len(t) for t in text]
        for n in range(N):
            if text[n]:
                S = model.first_layer(text[n])[1]
                off = float((srv.S[0, n].cpu().double() - S).abs().max() / S.abs().max())
                assert off <= NEAR, n

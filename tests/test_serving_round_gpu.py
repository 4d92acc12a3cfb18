"""The serving operators together: a two-layer hybrid model (linear attention
with a decay per head, then attention over a paged cache) run as a server
runs it, prompts, draft windows with their verify, token scores, accepted
prefix and commit, and checked against the model run token by token in 64
bits over the accepted text."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import commit_gated_delta_amd as gdn  # noqa: E402

E, HV, HK, D, HQ, HKV, V = 96, 4, 2, 64, 4, 2, 700


class Model:
    """Embedding, decay layer, attention layer, logits; the projections are
    plain products in the type of the weights."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        w = lambda *s: torch.randn(s, device="cuda", generator=g) / s[0] ** 0.5
        self.embed = w(V, E) * V ** 0.5
        self.q, self.k, self.v = w(E, HK * D), w(E, HK * D), w(E, HV * D)
        self.g, self.out = w(E, HV), w(HV * D, E)
        self.aq, self.ak, self.av = w(E, HQ * D), w(E, HKV * D), w(E, HKV * D)
        self.aout, self.head = w(HQ * D, E), w(E, V) * 3

    def decay_inputs(self, x):
        s = x.shape[:-1]
        return ((x @ self.q).view(*s, HK, D), (x @ self.k).view(*s, HK, D) / 8,
                (x @ self.v).view(*s, HV, D),
                -torch.nn.functional.softplus(x @ self.g - 2))

    def attention_inputs(self, x):
        s = x.shape[:-1]
        return ((x @ self.aq).view(*s, HQ, D), (x @ self.ak).view(*s, HKV, D),
                (x @ self.av).view(*s, HKV, D))

    def double(self):
        m = object.__new__(Model)
        m.__dict__ = {k: w.double() for k, w in self.__dict__.items()}
        return m

    def reference(self, tokens):
        """Logits after every token, token by token in f64."""
        m = self.double()
        S = torch.zeros(HV, D, D, dtype=torch.float64, device="cuda")
        keys, vals, out = [], [], []
        for t in tokens:
            x = m.embed[t]
            q, k, v, g = m.decay_inputs(x)
            k, q = (y.repeat_interleave(HV // HK, 0) for y in (k, q))
            S = torch.exp(g)[:, None, None] * S + k[:, :, None] * v[:, None, :]
            x = x + (q[:, :, None] * S).sum(1).reshape(-1) @ m.out
            q, k, v = m.attention_inputs(x)
            keys.append(k.repeat_interleave(HQ // HKV, 0))
            vals.append(v.repeat_interleave(HQ // HKV, 0))
            K, W = torch.stack(keys), torch.stack(vals)
            p = torch.softmax((K * q).sum(2) * D ** -0.5, 0)
            x = x + (p[:, :, None] * W).sum(0).reshape(-1) @ m.aout
            out.append(x @ m.head)
        return torch.stack(out)


class Server:
    def __init__(self, model, prompts, T, page=8, cols=12):
        self.m, self.N, self.T = model, len(prompts), T
        n = self.N
        self.S = torch.zeros(1, n, HV, D, D, device="cuda")
        self.kv = gdn.KvDims.of(n, T, HQ, HKV, D, page, n * cols, cols)
        self.k_cache, self.v_cache = (
            torch.full((n * cols, HKV, page, D), float("nan"), device="cuda")
            for _ in range(2))
        self.table = torch.randperm(n * cols, device="cuda").view(n, cols).int()
        self.ws = torch.empty(gdn.paged_attention_workspace_bytes(self.kv),
                              dtype=torch.uint8, device="cuda")
        self.length = [0] * n
        self.prefill(prompts)

    def attend(self, x, t_lane):
        """The attention layer on [N, T, E] hidden rows of new tokens."""
        q, k, v = (y.contiguous() for y in self.m.attention_inputs(x))
        kv_len = torch.tensor([a + b for a, b in zip(self.length, t_lane)],
                              dtype=torch.int32, device="cuda")
        gdn.kv_append(self.kv, t_lane, k, v, self.k_cache, self.v_cache,
                      self.table, kv_len)
        o = torch.zeros(self.N, self.T, HQ, D, device="cuda")
        gdn.paged_attention(self.kv, t_lane, q, self.k_cache, self.v_cache,
                            self.table, kv_len, o, self.ws, scale=D ** -0.5)
        return x + o.view(self.N, self.T, -1) @ self.m.aout

    def prefill(self, prompts):
        lens = [len(p) for p in prompts]
        flat = torch.tensor(sum(prompts, []), device="cuda")
        x = self.m.embed[flat]
        q, k, v, g = (y.contiguous() for y in self.m.decay_inputs(x))
        o = torch.empty(len(flat), HV, D, device="cuda")
        ws = torch.empty(gdn.decay_prefill_workspace_bytes(lens, HV, HK, D, D),
                         dtype=torch.uint8, device="cuda")
        gdn.decay_prefill(lens, HV, HK, D, D, q, k, v, g, None, self.S[0], o, ws)
        x = x + o.view(len(flat), -1) @ self.m.out
        # the attention layer takes the prompts in windows of up to T tokens
        rows = torch.split(x, lens)
        self.last = [None] * self.N
        while any(a < b for a, b in zip(self.length, lens)):
            t_lane = [min(self.T, b - a) for a, b in zip(self.length, lens)]
            y = torch.zeros(self.N, self.T, E, device="cuda")
            for n, m in enumerate(t_lane):
                y[n, :m] = rows[n][self.length[n]:self.length[n] + m]
            z = self.attend(y, t_lane)
            for n, m in enumerate(t_lane):
                self.length[n] += m
                if m:
                    self.last[n] = z[n, m - 1] @ self.m.head

    def verify(self, windows):
        """Scores of every window's rows; nothing is committed."""
        t_lane = [len(w) for w in windows]
        tok = torch.zeros(self.N, self.T, dtype=torch.long, device="cuda")
        for n, w in enumerate(windows):
            tok[n, :len(w)] = torch.tensor(w)
        x = self.m.embed[tok]
        self.step = [y[None].contiguous() for y in self.m.decay_inputs(x)]
        dims = gdn.Dims.of(1, self.N, HV, HK, D, D, self.T)
        o = torch.zeros(1, self.N, self.T, HV, D, device="cuda")
        gdn.decay_step(dims, t_lane, *self.step, self.S, o, keep_state=True)
        x = x + o.view(self.N, self.T, -1) @ self.m.out
        logits = (self.attend(x, t_lane) @ self.m.head).view(self.N * self.T, V)
        # row t scores the window's next token; the last row has none
        given = torch.full((self.N, self.T), -1, dtype=torch.int32, device="cuda")
        for n, w in enumerate(windows):
            given[n, :len(w) - 1] = torch.tensor(w[1:], dtype=torch.int32)
        R = self.N * self.T
        lp, ent, best = (torch.empty(s, device="cuda") for s in ((R,), (R,), (R, 2)))
        ids = torch.empty(R, 2, dtype=torch.int32, device="cuda")
        ws = torch.empty(gdn.token_scores_workspace_bytes(R, V, 2),
                         dtype=torch.uint8, device="cuda")
        gdn.token_scores(logits, given.view(-1), 2, lp, ent, ids, best, ws)
        return (logits.view(self.N, self.T, V), lp.view(self.N, self.T),
                ids.view(self.N, self.T, 2))

    def commit(self, m):
        dims = gdn.Dims.of(1, self.N, HV, HK, D, D, self.T)
        q, k, v, g = self.step
        gdn.decay_step(dims, m, None, k, v, g, self.S, None)
        self.length = [a + b for a, b in zip(self.length, m)]


def test_speculative_rounds_agree_with_the_model():
    torch.manual_seed(3)
    model = Model(11)
    prompts = [torch.randint(V, (n,)).tolist() for n in (1, 19, 7)]
    T = 6
    srv = Server(model, prompts, T)
    text = [list(p) for p in prompts]
    # greedy text in f64: drafts are right for a while, then wrong
    future = []
    for p in prompts:
        t = list(p)
        for _ in range(20):
            t.append(int(model.reference(t)[-1].argmax()))
        future.append(t)
    tops = [int(x.argmax()) for x in srv.last]
    near = 2e-4          # f32 products of a two-layer model against f64
    for r, right in enumerate(([3, 5, 0], [5, 1, 2], [0, 4, 5])):
        windows = []
        for n in range(3):
            at = len(text[n])
            assert tops[n] == future[n][at]
            w = future[n][at:at + 1 + right[n]]
            windows.append((w + [(x + 1) % V for x in future[n][at + 1 + right[n]:]])[:T])
        logits, lp, ids = srv.verify(windows)
        m = []
        for n, w in enumerate(windows):
            ref = model.reference(text[n] + w)[-len(w):]
            got = logits[n, :len(w)].double()
            assert float((got - ref).abs().max()) <= near * float(ref.abs().max())
            logp = torch.log_softmax(ref, 1)
            for t in range(len(w) - 1):
                assert abs(float(lp[n, t]) - float(logp[t, w[t + 1]])) <= near * float(ref.abs().max())
            assert float(lp[n, len(w) - 1]) == 0
            a = 1
            while a < len(w) and w[a] == int(ids[n, a - 1, 0]):
                a += 1
            m.append(a)
            assert a == min(1 + right[n], T)
            tops[n] = int(ids[n, a - 1, 0])
            text[n] += w[:a]
        srv.commit(m)
        assert srv.length == [len(t) for t in text]

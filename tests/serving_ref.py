"""64-bit references of the serving operators (linear attention with a decay
per head, paged attention, token scores), written from their definitions, and
the error bounds the tests hold the kernels to.

Unit: U32 = 2^-24, half a step of f32.  (The kernels carry f32 operands of
bf16 products as three parts of 8 bits, which is exact.)
"""
import math

import torch

U32 = 2.0 ** -24


def decay_chain(q, k, v, g, S0, scale):
    """One sequence of one batch of heads in f64: q, k [T, H, dk] (already
    one row per value head), v [T, H, dv], g [T, H], S0 [H, dk, dv].
    Returns o, S and the same sums with every term's absolute value, which
    bound the rounding errors."""
    q, k, v, g, S = (x.double() for x in (q, k, v, g, S0))
    A = S.abs()
    o, oa = [], []
    for t in range(q.shape[0]):
        a = torch.exp(g[t])[:, None, None]
        S = a * S + k[t][:, :, None] * v[t][:, None, :]
        A = a * A + k[t].abs()[:, :, None] * v[t].abs()[:, None, :]
        o.append(scale * (q[t][:, :, None] * S).sum(1))
        oa.append(abs(scale) * (q[t].abs()[:, :, None] * A).sum(1))
    shape = (0,) + tuple(v.shape[1:])
    stack = lambda x: torch.stack(x) if x else torch.zeros(
        shape, dtype=torch.float64, device=S.device)
    return stack(o), S, stack(oa), A


def decay_bound(d_k, tokens):
    """Largest error of an output or state entry relative to the sum of its
    terms' absolute values: a term's decays are a product of at most
    tokens / 64 + 2 rounded exponentials, each exact to 4 steps of f32; sums
    run over d_k entries and 64 tokens, at most a step of f32 for each, and
    one addition per 64 tokens."""
    steps = tokens / 64 + 2
    return (8 * steps + 2 * (d_k + 64) + steps) * U32


def step_bound(d_k, tokens):
    """The recurrent form: per token one rounding of the decay (4 ulp with
    its exponential), one multiply, one add; then a sum of d_k terms."""
    return (10 * tokens + d_k + 4) * U32


def attend(q, k_cache, v_cache, table, kv_len, t_lane, scale):
    """f64 paged attention: (o, bound): rows of idle tokens are NaN in o.
    Relative to sum p |v|, an output is off by the error e of its score (and
    of the largest score) twice through the softmax, by the sums (one step
    per position) and a few roundings.  A score's error is
    (d + 4) U32 times the sum of its terms' absolute values."""
    N, T, Hq, d = q.shape
    n_pages, Hkv, page, _ = k_cache.shape
    group = Hq // Hkv
    o = torch.full(q.shape, float("nan"), dtype=torch.float64)
    tol = torch.zeros(q.shape, dtype=torch.float64)
    q, kc, vc = q.double().cpu(), k_cache.double().cpu(), v_cache.double().cpu()
    table, kv_len = table.cpu(), kv_len.cpu()
    cap = table.shape[1] * page
    for n in range(N):
        length = min(max(int(kv_len[n]), 0), cap)
        pos = torch.arange(length)
        pages = table[n, pos // page].long()
        ok = (pages >= 0) & (pages < n_pages)
        pos, pages = pos[ok], pages[ok]
        for t in range(t_lane[n]):
            sees = pos <= length - t_lane[n] + t
            k = kc[pages[sees], :, pos[sees] % page]         # [L, Hkv, d]
            v = vc[pages[sees], :, pos[sees] % page]
            if k.shape[0] == 0:
                o[n, t] = 0
                continue
            for h in range(Hq):
                x = scale * (k[:, h // group] * q[n, t, h]).sum(1)
                xa = abs(scale) * (k[:, h // group] * q[n, t, h]).abs().sum(1)
                p = torch.softmax(x, 0)
                o[n, t, h] = (p[:, None] * v[:, h // group]).sum(0)
                e = (d + 4) * U32 * float(xa.max()) + 4 * U32
                mag = (p[:, None] * v[:, h // group].abs()).sum(0)
                tol[n, t, h] = mag * (4 * e + (2 * len(x) + 16) * U32)
    return o, tol + 1e-30


def scores(logits, tokens, n_top, it):
    """f64 (logprob, entropy, ids, top logprobs) with the rules for empty and
    bad rows."""
    x = logits.double().cpu()
    R, V = x.shape
    lp = torch.zeros(R, dtype=torch.float64)
    ent = torch.zeros(R, dtype=torch.float64)
    ids = torch.full((R, n_top), -1, dtype=torch.int32)
    best = torch.full((R, n_top), float("nan"), dtype=torch.float64)
    for r in range(R):
        t = int(tokens[r])
        bad = bool((torch.isnan(x[r]) | (x[r] == math.inf)).any())
        empty = bool((x[r] == -math.inf).all())
        order = sorted(range(V), key=lambda i: (-float(x[r, i]), i))[:n_top] \
            if not bad and V <= 4096 else None
        if order is None and not bad:
            s = torch.sort(x[r], descending=True, stable=True)
            order = s.indices[:n_top].tolist()
        if bad:
            lp[r], ent[r] = math.nan, math.nan
        else:
            y = x[r] * float(it)
            logp = torch.full_like(y, -math.inf) if empty else torch.log_softmax(y, 0)
            p = torch.exp(logp)
            ent[r] = 0.0 if empty else -torch.where(p > 0, p * logp, 0).sum()
            if n_top:
                ids[r] = torch.tensor(order, dtype=torch.int32)
                best[r] = logp[order]
            lp[r] = math.nan if t >= V else logp[max(t, 0)]
        if t < 0:
            lp[r] = 0.0
    return lp, ent, ids, best


def scores_bound(logits, it):
    """A log probability is x - m - log Z in f32: two roundings of x - m at
    most |x - m| large, log Z off by the relative error of Z (64 partial sums
    of at most V / 64 positive terms... each exact to 4 ulp) and its own
    rounding.  Entropy adds the same error in W / Z."""
    x = logits.double().cpu()
    fin = torch.where(torch.isfinite(x), x, 0)
    spread = float((fin.max() - fin.min()) * it) + 1
    V = x.shape[1]
    return (4 * spread + 2 * math.log(V + 1) + V / 64 + 64) * U32 * (spread + 1)

"""Timing cases of the serving operators: linear attention with a decay per
head (prompts and windows), attention over a paged key-value cache and the
cache's append, and token scores.

``run`` makes one pass: in plain torch operations (float32 and float64) while
``own`` is false, through the package's entry points while it is true.
``exact`` computes the same outputs in float64 from the definitions, token by
token or lane by lane.
"""
import math
import random

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------- cases
def listed():
    """Sizes of the repository's own workloads (32 value heads of 128, 16 key
    heads, 8 lanes, 48 layers, windows of 16, a 32,768-token prompt, a
    131,072-row vocabulary) and generic ones."""
    return [
        # one long prompt on every head of a layer
        dict(name="prompt 32k x 32 heads", op="prompt", lens="32768", h_v=32, h_k=32, d_k=128,
             d_v=128, type="bf16", per_head=False, init=False),
        # a head-sharded layer's share of a very long prompt, resumed from a
        # state, with one constant decay per head
        dict(name="prompt 128k x 4 heads", op="prompt", lens="131072", h_v=4, h_k=4, d_k=128,
             d_v=128, type="bf16", per_head=True, init=True),
        # a scheduler's batch of short prompts in f32, packed, one of them empty
        dict(name="prompts packed f32", op="prompt", lens="1,300,0,64,65,1000,17", h_v=8, h_k=2,
             d_k=64, d_v=64, type="f32", per_head=False, init=True),
        # the decode step of one layer: one token on each of 8 lanes
        dict(name="step 8 lanes", op="step", layers=1, lanes=8, window=1, h_v=32, h_k=16,
             d_k=128, d_v=128, type="bf16", per_head=False, ragged=False, keep=False),
        # the verify of draft windows over all layers, state left as it was
        dict(name="window 16 x 48 layers", op="step", layers=48, lanes=8, window=16, h_v=32,
             h_k=16, d_k=128, d_v=128, type="bf16", per_head=False, ragged=True, keep=True),
        # one token against short caches: latency
        dict(name="attend 8 lanes 1k", op="attend", lanes=8, window=1, h_q=16, h_kv=2, d=256,
             page=16, longest=1024, type="bf16"),
        # many requests with long caches: bandwidth
        dict(name="attend 32 lanes 32k", op="attend", lanes=32, window=1, h_q=32, h_kv=8, d=128,
             page=64, longest=32768, type="bf16"),
        # draft windows of 16 verified on a few lanes with long caches
        dict(name="attend window 16", op="attend", lanes=8, window=16, h_q=32, h_kv=4, d=128,
             page=32, longest=16001, type="bf16"),
        # the rows of one decode step into the caches
        dict(name="append 8 lanes", op="append", lanes=8, window=1, h_q=16, h_kv=2, d=256,
             page=16, longest=1024, type="bf16"),
        # prompts of 64 tokens a lane into the caches
        dict(name="append 128 lanes x 64", op="append", lanes=128, window=64, h_q=32, h_kv=8,
             d=128, page=64, longest=2048, type="bf16"),
        # the verify rows of one lane: anchor and 15 drafts
        dict(name="scores 16 rows", op="scores", rows=16, vocab=131072, top=5, type="f32",
             masked=False),
        # scoring a stretch of prompt, some tokens ruled out by a grammar
        dict(name="scores 1024 rows", op="scores", rows=1024, vocab=131072, top=20, type="bf16",
             masked=True),
    ]


def _log_between(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("prompt", "prompt", "step", "step", "attend", "attend", "append", "scores", "scores"))
    kind = rng.choice(("bf16", "bf16", "f32"))
    if op == "prompt":
        h_k = rng.choice((1, 2, 4, 8))
        h_v = h_k * rng.choice((1, 2, 4))
        d_k, d_v = rng.choice((16, 32, 64, 128, 128)), rng.choice((16, 40, 64, 100, 128, 128, 256))
        most = max(64, min(65536, 16384 * 16 * 128 // (h_v * max(d_v, 64))))
        n = rng.choice((1, 1, 2, 3, 5, 9))
        lens = [_log_between(rng, 1, max(2, most // n)) for _ in range(n)]
        return dict(op=op, lens=",".join(map(str, lens)), h_v=h_v, h_k=h_k, d_k=d_k, d_v=d_v,
                    type=kind, per_head=rng.random() < 0.4, init=rng.random() < 0.5)
    if op == "step":
        h_k = rng.choice((1, 2, 4, 8, 16))
        h_v = h_k * rng.choice((1, 2, 3))
        lanes, layers = _log_between(rng, 1, 64), rng.choice((1, 1, 1, 3, 12))
        window = rng.choice((1, 1, 1, 2, 6, 16, 33))
        while lanes * layers * h_v * max(window, 4) > 8 * 48 * 32 * 16:
            lanes = max(1, lanes // 2)
        return dict(op=op, layers=layers, lanes=lanes, window=window, h_v=h_v, h_k=h_k,
                    d_k=rng.choice((16, 32, 64, 128, 128)), d_v=rng.choice((32, 64, 100, 128, 128)),
                    type=kind, per_head=rng.random() < 0.4, ragged=rng.random() < 0.5,
                    keep=rng.random() < 0.4)
    if op in ("attend", "append"):
        h_kv = rng.choice((1, 2, 4, 8))
        h_q = h_kv * rng.choice((1, 2, 4, 5, 8, 16))
        d = rng.choice((64, 128, 128, 256))
        window = rng.choice((1, 1, 1, 2, 5, 16)) if op == "attend" else _log_between(rng, 1, 64)
        lanes = _log_between(rng, 1, 96)
        longest = _log_between(rng, 65, 32768)
        while lanes * longest * h_kv * d > 16 * 32768 * 8 * 128 or lanes * longest * h_q * window > 1 << 28:
            lanes, longest = max(1, lanes // 2), max(65, longest // 2 if lanes == 1 else longest)
        return dict(op=op, lanes=lanes, window=window, h_q=h_q, h_kv=h_kv, d=d,
                    page=rng.choice((1, 8, 16, 24, 64, 256)), longest=longest, type=kind)
    vocab = _log_between(rng, 1000, 262144)
    rows = _log_between(rng, 1, max(2, min(4096, (1 << 26) // vocab)))
    return dict(op=op, rows=rows, vocab=vocab, top=rng.choice((0, 1, 3, 8, 20, 32)), type=kind,
                masked=rng.random() < 0.4)


# -------------------------------------------------------------------- inputs
def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _windows(case):
    """Tokens of each lane's window."""
    if not case["ragged"]:
        return [case["window"]] * case["lanes"]
    r = random.Random(case["lanes"] * 1000 + case["window"])
    return [r.randint(1, case["window"]) for _ in range(case["lanes"])]


def _kv_lens(case):
    """Tokens of each lane's cache, its window included."""
    r = random.Random(case["lanes"] * 7919 + case["longest"])
    low = max(case["window"], case["longest"] // 2)
    lens = [r.randint(low, max(low, case["longest"])) for _ in range(case["lanes"])]
    lens[0] = max(low, case["longest"])
    return lens


def _gates(case, shape, g):
    """Log-decays: slow ones per token, or one constant per head."""
    if case["per_head"]:
        h = torch.arange(case["h_v"], device="cuda", dtype=torch.float32)
        return -torch.exp2(-8.0 * (h + 1) / case["h_v"]) * (0.5 + torch.rand((), device="cuda", generator=g))
    x = torch.randn(shape, device="cuda", generator=g) - 2.0
    return -torch.nn.functional.softplus(x)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=case)
    op, t = case["op"], _TYPES[case.get("type", "bf16")]

    def normal(*shape, dtype=t):
        return torch.randn(shape, device="cuda", generator=g).to(dtype)

    if op == "prompt":
        lens = s["lens"] = _lens(case)
        n, h_v, h_k, d_k, d_v = sum(lens), case["h_v"], case["h_k"], case["d_k"], case["d_v"]
        s["q"], s["k"], s["v"] = normal(n, h_k, d_k), normal(n, h_k, d_k), normal(n, h_v, d_v)
        s["g"] = _gates(case, (n, h_v), g)
        s["init"] = 0.1 * normal(len(lens), h_v, d_k, d_v, dtype=torch.float32) if case["init"] else None
    elif op == "step":
        y, n, w, h_v, h_k, d_k, d_v = (case[x] for x in ("layers", "lanes", "window", "h_v", "h_k", "d_k", "d_v"))
        s["t_lane"] = _windows(case)
        s["q"], s["k"], s["v"] = normal(y, n, w, h_k, d_k), normal(y, n, w, h_k, d_k), normal(y, n, w, h_v, d_v)
        s["g"] = _gates(case, (y, n, w, h_v), g)
        if case["per_head"]:
            s["g"] = s["g"].expand(y, h_v).contiguous()
        s["S"] = 0.1 * normal(y, n, h_v, d_k, d_v, dtype=torch.float32)
    elif op in ("attend", "append"):
        n, w, h_q, h_kv, d, page = (case[x] for x in ("lanes", "window", "h_q", "h_kv", "d", "page"))
        lens = _kv_lens(case)
        per_lane = -(-max(lens) // page)
        pages = n * per_lane + 3
        order = torch.randperm(pages, device="cuda", generator=g)[: n * per_lane].view(n, per_lane)
        used = torch.tensor([-(-x // page) for x in lens], device="cuda")
        holds = torch.arange(per_lane, device="cuda") < used[:, None]
        s["table"] = torch.where(holds, order, torch.full_like(order, -1)).to(torch.int32)
        s["kv_len"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
        s["t_lane"] = [w] * n
        s["k_cache"], s["v_cache"] = normal(pages, h_kv, page, d), normal(pages, h_kv, page, d)
        if op == "attend":
            s["q"] = normal(n, w, h_q, d)
        else:
            s["k"], s["v"] = normal(n, w, h_kv, d), normal(n, w, h_kv, d)
    else:
        rows, vocab = case["rows"], case["vocab"]
        x = torch.randn(rows, vocab, device="cuda", generator=g).mul_(3.0)
        if case["masked"]:  # every second row allows a tenth of the vocabulary
            out = torch.rand(rows, vocab, device="cuda", generator=g) < 0.9
            out[::2] = False
            x.masked_fill_(out, -math.inf)
        s["logits"] = x.to(t)
        s["tokens"] = torch.randint(vocab, (rows,), device="cuda", generator=g, dtype=torch.int32)
        s["tokens"][::2] = s["logits"][::2].float().argmax(1).to(torch.int32)
        s["inv_temperature"] = 1.25
    if own:
        _keep(s)
    return s


def _keep(s):
    """What a program of the package holds between calls: dims, workspaces."""
    c, op, gdn = s["case"], s["case"]["op"], _gdn()
    need = 0
    if op == "prompt":
        need = gdn.decay_prefill_workspace_bytes(s["lens"], c["h_v"], c["h_k"], c["d_k"], c["d_v"])
    elif op == "step":
        s["dims"] = gdn.Dims.of(c["layers"], c["lanes"], c["h_v"], c["h_k"], c["d_k"], c["d_v"], c["window"])
    elif op in ("attend", "append"):
        s["dims"] = gdn.KvDims.of(c["lanes"], c["window"], c["h_q"], c["h_kv"], c["d"], c["page"],
                                  s["k_cache"].shape[0], s["table"].shape[1])
        need = gdn.paged_attention_workspace_bytes(s["dims"])
    else:
        need = gdn.token_scores_workspace_bytes(c["rows"], c["vocab"], c["top"])
    s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")


def _gdn():
    import commit_gated_delta_amd
    return commit_gated_delta_amd


# ---------------------------------------------------------------------- work
def work(case):
    op, size = case["op"], 2 if case.get("type", "bf16") == "bf16" else 4
    if op in ("prompt", "step"):
        h_v, h_k, d_k, d_v = case["h_v"], case["h_k"], case["d_k"], case["d_v"]
        if op == "prompt":
            tokens, states = sum(_lens(case)), len(_lens(case)) * (2 if case["init"] else 1)
            gates = h_v if case["per_head"] else tokens * h_v
        else:
            tokens = case["layers"] * sum(_windows(case))
            states = case["layers"] * case["lanes"] * (1 if case["keep"] else 2)
            gates = case["layers"] * h_v if case["per_head"] else tokens * h_v
        row = 2 * h_k * d_k * size + h_v * d_v * (size + 4)
        return {"bytes": tokens * row + 4 * gates + 4 * states * h_v * d_k * d_v,
                "flops": 4 * tokens * h_v * d_k * d_v}
    if op in ("attend", "append"):
        lens, w = _kv_lens(case), case["window"]
        if op == "append":
            return {"bytes": 4 * case["lanes"] * w * case["h_kv"] * case["d"] * size, "flops": 0}
        seen = sum(sum(n - w + t + 1 for t in range(w)) for n in lens)
        return {"bytes": 2 * sum(lens) * case["h_kv"] * case["d"] * size
                + case["lanes"] * w * case["h_q"] * case["d"] * (size + 4),
                "flops": 4 * seen * case["h_q"] * case["d"]}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * size + case["rows"] * (12 + 8 * case["top"]), "flops": 6 * n}


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if op == "prompt":
        return _own_prompt(s) if own else _plain_prompt(s)
    if op == "step":
        return _own_step(s) if own else _plain_step(s)
    if op == "attend":
        return _own_attend(s) if own else _plain_attend(s)
    if op == "append":
        return _own_append(s) if own else _plain_append(s)
    return _own_scores(s) if own else _plain_scores(s)


def _own_prompt(s):
    c, lens = s["case"], s["lens"]
    shape = (c["h_v"], c["h_k"], c["d_k"], c["d_v"])
    o = torch.empty(sum(lens), c["h_v"], c["d_v"], device="cuda")
    last = torch.empty(len(lens), c["h_v"], c["d_k"], c["d_v"], device="cuda")
    _gdn().decay_prefill(lens, *shape, s["q"], s["k"], s["v"], s["g"], s["init"], last, o,
                         s["workspace"], scale=c["d_k"] ** -0.5, head_decay=c["per_head"])
    return {"o": o, "S": last}


def _own_step(s):
    c = s["case"]
    o = torch.zeros(s["v"].shape, device="cuda") if c["ragged"] else torch.empty(s["v"].shape, device="cuda")
    _gdn().decay_step(s["dims"], s["t_lane"], s["q"], s["k"], s["v"], s["g"], s["S"], o,
                      scale=c["d_k"] ** -0.5, head_decay=c["per_head"], keep_state=c["keep"])
    return {"o": o} if c["keep"] else {"o": o, "S": s["S"]}


def _own_attend(s):
    o = torch.empty(s["q"].shape, device="cuda")
    _gdn().paged_attention(s["dims"], s["t_lane"], s["q"], s["k_cache"], s["v_cache"], s["table"],
                           s["kv_len"], o, s["workspace"], scale=s["case"]["d"] ** -0.5)
    return o


def _own_append(s):
    _gdn().kv_append(s["dims"], s["t_lane"], s["k"], s["v"], s["k_cache"], s["v_cache"],
                     s["table"], s["kv_len"])
    return {"k": s["k_cache"], "v": s["v_cache"]}


def _own_scores(s):
    c = s["case"]
    rows, top = c["rows"], c["top"]
    logprob, entropy = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ids = torch.empty(rows, top, dtype=torch.int32, device="cuda")
    best = torch.empty(rows, top, device="cuda")
    _gdn().token_scores(s["logits"], s["tokens"], top, logprob, entropy, ids, best, s["workspace"],
                        inv_temperature=s["inv_temperature"])
    return {"logprob": logprob, "entropy": entropy, "ids": ids, "best": best}


# --------------------------------------------------------- the plain forms
_CHUNK = 64


def _plain_prompt(s):
    """Chunks of 64 tokens: a masked product inside each chunk, and the chunk
    states combined with their decays in one product."""
    c, lens = s["case"], s["lens"]
    h_v, h_k, d_k, d_v = c["h_v"], c["h_k"], c["d_k"], c["d_v"]
    dev, group = s["q"].device, h_v // h_k
    length = torch.tensor(lens, device=dev)
    first = torch.cumsum(length, 0) - length
    chunks = -(-length // _CHUNK)
    m = sum(-(-n // _CHUNK) for n in lens)
    seq = torch.repeat_interleave(torch.arange(len(lens), device=dev), chunks, output_size=m)
    nth = torch.arange(m, device=dev) - (torch.cumsum(chunks, 0) - chunks)[seq]
    at = nth[:, None] * _CHUNK + torch.arange(_CHUNK, device=dev)
    there = at < length[seq][:, None]
    token = torch.where(there, at + first[seq][:, None], 0)

    def rows(x, heads):  # [chunks, value heads, 64, d]
        y = x.float()[token] * there[:, :, None, None]
        y = y if heads == h_v else y.repeat_interleave(group, 2)
        return y.transpose(1, 2).contiguous()

    q, k, v = rows(s["q"], h_k), rows(s["k"], h_k), rows(s["v"], h_v)
    gate = s["g"].double() if not c["per_head"] else s["g"].double().expand(sum(lens), h_v)
    gate = (gate[token] * there[:, :, None]).transpose(1, 2)
    b = torch.cumsum(gate, 2)                                   # [chunks, heads, 64]
    total = b[:, :, -1]
    causal = torch.ones(_CHUNK, _CHUNK, dtype=torch.bool, device=dev).tril()
    decay = torch.exp(torch.where(causal, b[..., :, None] - b[..., None, :], -math.inf)).float()
    o = torch.matmul(torch.matmul(q, k.transpose(2, 3)) * decay, v)
    added = torch.matmul((k * torch.exp(total[..., None] - b).float()[..., None]).transpose(2, 3), v)
    # state before chunk i: the chunks j < i of its sequence, and its start
    run = torch.cumsum(total, 0)
    before = run - total
    same = (seq[:, None] == seq[None, :]) & (torch.arange(m, device=dev)[:, None] > torch.arange(m, device=dev))
    carry = torch.exp(torch.where(same[..., None], before[:, None] - run[None], -math.inf)).float()
    flat = added.permute(1, 0, 2, 3).reshape(h_v, m, d_k * d_v)
    state = torch.matmul(carry.permute(2, 0, 1).contiguous(), flat).view(h_v, m, d_k, d_v).transpose(0, 1)
    head = torch.zeros(len(lens), h_v, dtype=torch.float64, device=dev)
    head.index_add_(0, seq, torch.where((nth == 0)[:, None], before, 0))   # sum before each sequence
    whole = torch.zeros_like(head).index_add_(0, seq, total)
    last = torch.zeros(len(lens), h_v, d_k, d_v, device=dev)
    final = nth == chunks[seq] - 1
    to_end = torch.where(final[:, None, None, None], torch.exp(total).float()[..., None, None] * state + added, 0)
    last.index_add_(0, seq, to_end)
    if s["init"] is not None:
        state = state + torch.exp(before - head[seq]).float()[..., None, None] * s["init"][seq]
        last = last + torch.exp(whole).float()[..., None, None] * s["init"]
    o = o + torch.exp(b).float()[..., None] * torch.matmul(q, state)
    o = (o.transpose(1, 2) * d_k ** -0.5)[there]
    return {"o": o, "S": last}


def _plain_step(s):
    """The window at once: a masked product among its tokens, and the state."""
    c = s["case"]
    h_v, h_k, w = c["h_v"], c["h_k"], c["window"]
    group = h_v // h_k
    t_lane = torch.tensor(s["t_lane"], device="cuda")
    there = (torch.arange(w, device="cuda") < t_lane[:, None])[None, :, :, None]      # [1, lanes, w, 1]

    def rows(x, heads):
        y = torch.where(there[..., None], x.float(), 0)
        return (y if heads == h_v else y.repeat_interleave(group, 3)).transpose(2, 3).contiguous()

    q, k, v = rows(s["q"], h_k), rows(s["k"], h_k), rows(s["v"], h_v)                 # [y, n, h, w, d]
    gate = s["g"].double()
    gate = gate[:, None, None, :].expand(-1, c["lanes"], w, -1) if c["per_head"] else gate
    b = torch.cumsum(torch.where(there, gate, 0), 2).transpose(2, 3)                  # [y, n, h, w]
    causal = torch.ones(w, w, dtype=torch.bool, device="cuda").tril()
    decay = torch.exp(torch.where(causal, b[..., :, None] - b[..., None, :], -math.inf)).float()
    o = torch.matmul(torch.matmul(q, k.transpose(3, 4)) * decay, v)
    o = (o + torch.exp(b).float()[..., None] * torch.matmul(q, s["S"])) * c["d_k"] ** -0.5
    o = torch.where(there[..., None], o.transpose(2, 3), 0)
    if c["keep"]:
        return {"o": o}
    total = b[..., -1:]
    k = k * torch.exp(total - b).float()[..., None]
    s["S"].mul_(torch.exp(total).float()[..., None]).add_(torch.matmul(k.transpose(3, 4), v))
    return {"o": o, "S": s["S"]}


def _places(s):
    """Page and row of every position of every lane."""
    longest, page = s["table"].shape[1] * s["case"]["page"], s["case"]["page"]
    at = torch.arange(longest, device="cuda")
    return s["table"].long().clamp(min=0)[:, at // page], at % page


def _plain_attend(s):
    c = s["case"]
    n, w, h_kv, d, group = c["lanes"], c["window"], c["h_kv"], c["d"], c["h_q"] // c["h_kv"]
    page, row = _places(s)
    k = s["k_cache"][page, :, row].float().transpose(1, 2).contiguous()               # [n, h_kv, L, d]
    q = s["q"].float().view(n, w, h_kv, group, d).permute(0, 2, 1, 3, 4).reshape(n, h_kv, w * group, d)
    x = torch.matmul(q, k.transpose(2, 3)) * d ** -0.5
    del k
    ends = (s["kv_len"][:, None] - w + torch.arange(w, device="cuda") + 1).repeat_interleave(group, 1)
    at = torch.arange(x.shape[3], device="cuda")
    x = torch.where((at < ends[..., None])[:, None], x, -math.inf)
    x = torch.exp(x - x.amax(3, keepdim=True))
    x = x / x.sum(3, keepdim=True)
    v = s["v_cache"][page, :, row].float().transpose(1, 2).contiguous()
    return torch.matmul(x, v).view(n, h_kv, w, group, d).permute(0, 2, 1, 3, 4).reshape(n, w, c["h_q"], d)


def _plain_append(s):
    c = s["case"]
    at = s["kv_len"].long()[:, None] - c["window"] + torch.arange(c["window"], device="cuda")
    page, row = torch.gather(s["table"].long(), 1, at // c["page"]), at % c["page"]
    s["k_cache"][page, :, row] = s["k"]
    s["v_cache"][page, :, row] = s["v"]
    return {"k": s["k_cache"], "v": s["v_cache"]}


def _plain_scores(s):
    top, x = s["case"]["top"], s["logits"].float()
    best, ids = torch.sort(x, dim=1, descending=True, stable=True)
    best, ids = best[:, :top] * s["inv_temperature"], ids[:, :top].to(torch.int32)
    x = x * s["inv_temperature"]
    x = x - x.amax(1, keepdim=True)
    e = torch.exp(x)
    z = e.sum(1, keepdim=True)
    log_z = torch.log(z)
    given = torch.gather(x, 1, s["tokens"].long()[:, None])
    entropy = log_z - torch.where(e > 0, e * x, 0).sum(1, keepdim=True) / z
    best = best - (s["logits"].float().amax(1, keepdim=True) * s["inv_temperature"] + log_z)
    return {"logprob": (given - log_z)[:, 0], "entropy": entropy[:, 0], "ids": ids, "best": best}


# ------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "prompt":
        return _exact_prompt(s)
    if op == "step":
        return _exact_step(s)
    if op == "attend":
        return _exact_attend(s)
    if op == "append":
        return _exact_append(s)
    return _exact_scores(s)


def _exact_prompt(s):
    """Token by token: every sequence that is still running takes a step."""
    c, lens = s["case"], s["lens"]
    h_v, h_k, d_k, d_v = c["h_v"], c["h_k"], c["d_k"], c["d_v"]
    if max(lens) * (120e-6 + 1e-11 * len(lens) * h_v * d_k * d_v) > 25:
        return None
    starts = np.concatenate([[0], np.cumsum(lens)])[:-1]
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    S = torch.zeros(len(lens), h_v, d_k, d_v, dtype=torch.float64, device="cuda")
    if s["init"] is not None:
        S += s["init"][order].double()
    o = torch.zeros(sum(lens), h_v, d_v, dtype=torch.float64, device="cuda")
    key = torch.arange(h_v, device="cuda") // (h_v // h_k)
    at = torch.tensor(starts[order], device="cuda")
    alpha = torch.exp(s["g"].double())
    alpha = alpha.expand(sum(lens), h_v) if c["per_head"] else alpha
    running = len(lens)
    for t in range(max(lens)):
        while lens[order[running - 1]] <= t:
            running -= 1
        i = at[:running] + t
        k, q, v = s["k"][i].double()[:, key], s["q"][i].double()[:, key], s["v"][i].double()
        state = S[:running]
        state.mul_(alpha[i][:, :, None, None]).add_(k[..., :, None] * v[..., None, :])
        o[i] = torch.matmul(q[:, :, None, :], state)[:, :, 0]
    last = torch.empty_like(S)
    last[order] = S
    return {"o": o * d_k ** -0.5, "S": last}


def _exact_step(s):
    c = s["case"]
    group = c["h_v"] // c["h_k"]
    S, o = s["S"].double(), torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
    for t in range(c["window"]):
        on = torch.tensor([t < n for n in s["t_lane"]], device="cuda")
        k, q = (s[x][:, :, t].double().repeat_interleave(group, 2) for x in "kq")
        g = s["g"].double()[:, None] if c["per_head"] else s["g"][:, :, t].double()
        new = torch.exp(g)[..., None, None] * S + k[..., None] * s["v"][:, :, t].double()[..., None, :]
        S = torch.where(on[None, :, None, None, None], new, S)
        o[:, :, t] = (q[..., None] * new).sum(3) * on[None, :, None, None]
    o *= c["d_k"] ** -0.5
    return {"o": o} if c["keep"] else {"o": o, "S": S}


def _exact_attend(s):
    c = s["case"]
    w, h_kv, d, group = c["window"], c["h_kv"], c["d"], c["h_q"] // c["h_kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for n, length in enumerate(s["kv_len"].tolist()):
        pages = s["table"][n, : -(-length // c["page"])].long()
        k, v = (s[x][pages].double().transpose(0, 1).reshape(h_kv, -1, d)[:, :length] for x in ("k_cache", "v_cache"))
        for t in range(w):
            end = length - w + t + 1
            q = s["q"][n, t].double().view(h_kv, group, d)
            x = torch.softmax(torch.matmul(q, k[:, :end].transpose(1, 2).contiguous()) / math.sqrt(d), 2)
            out[n, t] = torch.matmul(x, v[:, :end]).view(-1, d)
    return out


def _exact_append(s):
    """Token by token."""
    c = s["case"]
    k, v, table = s["k_cache"].double(), s["v_cache"].double(), s["table"].tolist()
    for n, length in enumerate(s["kv_len"].tolist()):
        for t in range(c["window"]):
            at = length - c["window"] + t
            page, row = table[n][at // c["page"]], at % c["page"]
            k[page, :, row], v[page, :, row] = s["k"][n, t].double(), s["v"][n, t].double()
    return {"k": k, "v": v}


def _exact_scores(s):
    """Row by row."""
    c = s["case"]
    rows, top = c["rows"], c["top"]
    logprob, entropy = (torch.zeros(rows, dtype=torch.float64, device="cuda") for _ in range(2))
    best = torch.zeros(rows, top, dtype=torch.float64, device="cuda")
    for i in range(rows):
        x = torch.log_softmax(s["logits"][i].double() * s["inv_temperature"], 0)
        logprob[i] = x[s["tokens"][i].long()]
        p = torch.exp(x)
        entropy[i] = -torch.where(p > 0, p * x, 0).sum()
        best[i] = torch.sort(x, descending=True).values[:top]
    return {"logprob": logprob, "entropy": entropy, "ids": None, "best": best}

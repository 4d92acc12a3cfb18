"""Timing cases of the attention layer's 4-bit cache and of sampled
verification: position rotation with the cache's append (rows kept in their
type or in 4 bits), attention over the 4-bit cache, and the verification of
drafted tokens from given random numbers.

``run`` makes one pass: in plain torch operations (float32 and float64) while
``own`` is false, through the package's entry points while it is true.
``exact`` computes the same outputs in float64 from the definitions.

The 4-bit cache: a row's channels in blocks of 32, each with a scale 2^(b -
127) from a byte b and 32 codes of the values 0, 0.5, 1, 1.5, 2, 3, 4, 6 and
their negatives, two codes a byte, the even channel in the lower half.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------- cases
def listed():
    """Sizes of the repository's own workloads (8 lanes, windows of 16 with
    the anchor, 6-token windows, a vocabulary of 131,072) and generic ones."""
    return [
        # one token a lane, part of every head rotated: latency
        dict(name="rope append 8 lanes", op="append", bits=16, lanes=8, window=1, h_q=16, h_kv=2, d=256,
             page=16, longest=1024, type="bf16", rot=64, pairs=False, far=False),
        # prompts of 64 tokens a lane from one fused projection: bandwidth
        dict(name="rope append 128 lanes x 64", op="append", bits=16, lanes=128, window=64, h_q=32,
             h_kv=8, d=128, page=64, longest=2048, type="bf16", rot=128, pairs=False, far=False),
        # f32 rows, neighbouring channels rotated, far positions given, odd pages
        dict(name="rope append f32 far", op="append", bits=16, lanes=29, window=11, h_q=20, h_kv=4, d=64,
             page=24, longest=4001, type="f32", rot=48, pairs=True, far=True),
        # one token a lane into the 4-bit cache: latency
        dict(name="fp4 append 8 lanes", op="append", bits=4, lanes=8, window=1, h_q=16, h_kv=2, d=256,
             page=16, longest=1024, type="bf16", rot=64, pairs=False, far=False),
        # prompts of 64 tokens a lane into the 4-bit cache: bandwidth
        dict(name="fp4 append 128 lanes x 64", op="append", bits=4, lanes=128, window=64, h_q=32, h_kv=8,
             d=128, page=64, longest=2048, type="bf16", rot=128, pairs=False, far=False),
        # one token against short caches: latency
        dict(name="fp4 attend 8 lanes 1k", op="attend", lanes=8, window=1, h_q=16, h_kv=2, d=256,
             page=16, longest=1024, type="bf16"),
        # many requests with long caches: bandwidth
        dict(name="fp4 attend 32 lanes 32k", op="attend", lanes=32, window=1, h_q=32, h_kv=8, d=128,
             page=64, longest=32768, type="bf16"),
        # draft windows of 16 verified on a few lanes with long caches
        dict(name="fp4 attend window 16", op="attend", lanes=8, window=16, h_q=32, h_kv=4, d=128,
             page=32, longest=16001, type="bf16"),
        # f32 queries, small heads, pages that end inside a tile
        dict(name="fp4 attend f32 d 64", op="attend", lanes=13, window=3, h_q=15, h_kv=3, d=64, page=24,
             longest=9999, type="f32"),
        # one token sampled from one row: latency
        dict(name="sample 1 row", op="verify", lanes=1, window=1, vocab=131072, type="f32", drafted=False,
             ragged=False, masked=False),
        # a full round of anchor and 15 drafts, the drafter's logits given
        dict(name="verify 8 lanes x 16", op="verify", lanes=8, window=16, vocab=131072, type="f32",
             drafted=True, ragged=True, masked=False),
        # many requests with drafts that have no distribution, a grammar on some rows
        dict(name="verify 64 lanes x 6", op="verify", lanes=64, window=6, vocab=131072, type="bf16",
             drafted=False, ragged=True, masked=True),
    ]


def _log_between(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "append", "append", "attend", "attend", "attend", "verify", "verify"))
    kind = rng.choice(("bf16", "bf16", "f32"))
    if op == "verify":
        vocab, window = _log_between(rng, 1000, 262144), rng.choice((1, 1, 2, 4, 6, 11, 16, 33))
        lanes = _log_between(rng, 1, max(2, min(96, (1 << 24) // (vocab * window))))
        return dict(op=op, lanes=lanes, window=window, vocab=vocab, type=kind, drafted=rng.random() < 0.5,
                    ragged=rng.random() < 0.5, masked=rng.random() < 0.4)
    h_kv = rng.choice((1, 2, 3, 4, 8))
    h_q = h_kv * rng.choice((1, 2, 4, 5, 8, 16))
    d = rng.choice((64, 128, 128, 256))
    window = rng.choice((1, 1, 1, 2, 5, 16)) if op == "attend" else _log_between(rng, 1, 64)
    lanes = _log_between(rng, 1, 96)
    longest = _log_between(rng, 65, 32768)
    while (lanes * longest * h_kv * d > 8 * 32768 * 8 * 128 or lanes * longest * h_q * window > 1 << 27
           or lanes * window * (h_q + 2 * h_kv) * d > 128 * 64 * 48 * 128):
        lanes, longest = max(1, lanes // 2), max(65, longest // 2 if lanes == 1 else longest)
    case = dict(op=op, lanes=lanes, window=window, h_q=h_q, h_kv=h_kv, d=d,
                page=rng.choice((1, 8, 16, 24, 64, 256)), longest=longest, type=kind)
    if op == "append":
        case.update(bits=rng.choice((4, 16)), rot=16 * rng.randint(1, d // 16) if rng.random() < 0.5 else d,
                    pairs=rng.random() < 0.4, far=rng.random() < 0.4)
    return case


# -------------------------------------------------------------------- inputs
def _windows(case):
    """Tokens of each lane's window."""
    if not case.get("ragged"):
        return [case["window"]] * case["lanes"]
    r = random.Random(case["lanes"] * 1000 + case["window"])
    lens = [r.randint(1, case["window"]) for _ in range(case["lanes"])]
    lens[0] = case["window"]
    return lens


def _kv_lens(case):
    """Tokens of each lane's cache, its window included."""
    r = random.Random(case["lanes"] * 7919 + case["longest"])
    low = max(case["window"], case["longest"] // 2)
    lens = [r.randint(low, max(low, case["longest"])) for _ in range(case["lanes"])]
    lens[0] = max(low, case["longest"])
    return lens


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=case)
    op, t = case["op"], _TYPES[case["type"]]

    def normal(*shape, dtype=t):
        return torch.randn(shape, device="cuda", generator=g).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, device="cuda", generator=g)

    if op == "verify":
        n, w, vocab = case["lanes"], case["window"], case["vocab"]
        s["t_lane"] = _windows(case)
        # one token of every row stands out, as in text that a drafter follows
        x = normal(n, w, vocab, dtype=torch.float32).mul_(2.0)
        right = torch.randint(vocab, (n, w), device="cuda", generator=g)
        x.scatter_(2, right[..., None], 2.0 + math.log(vocab) + 2.5 * uniform(n, w, 1))
        out = uniform(n, w, vocab) < 0.9 if case["masked"] else None
        if case["masked"]:  # every second row allows a tenth of the vocabulary
            out[:, ::2] = False
            x.masked_fill_(out, -math.inf)
        s["logits"] = x.to(t)
        s["inv_temperature"] = 0.8 + 0.5 * uniform(n)
        s["tokens"] = torch.randint(vocab, (n, w), device="cuda", generator=g, dtype=torch.int32)
        if case["drafted"]:
            y = x[:, :-1] + 0.7 * normal(n, w - 1, vocab, dtype=torch.float32)
            s["draft_logits"] = y.to(t)
            noise = uniform(n, w - 1, vocab).clamp_(min=1e-30).log_().neg_().log_().neg_()
            pick = (s["draft_logits"].float() * s["inv_temperature"][:, None, None] + noise).argmax(2)
        else:
            s["draft_logits"] = None
            pick = torch.where(uniform(n, w - 1) < 0.85, right[:, :-1], s["tokens"][:, 1:].long())
        s["tokens"][:, 1:] = pick.to(torch.int32)
        s["uniforms"] = uniform(n, w)
    else:
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
        if op == "attend" or case["bits"] == 4:
            for c in "kv":
                s[c + "_codes"] = torch.randint(256, (pages, h_kv, page, d // 2), device="cuda", generator=g,
                                                dtype=torch.uint8)
                s[c + "_scales"] = torch.randint(124, 128, (pages, h_kv, page, d // 32), device="cuda",
                                                 generator=g, dtype=torch.uint8)
        else:
            s["k_cache"], s["v_cache"] = normal(pages, h_kv, page, d), normal(pages, h_kv, page, d)
        if op == "attend":
            s["q"] = normal(n, w, h_q, d)
        else:
            # the rows as one projection gives them: a token's q, k and v side by side
            rows = normal(n, w, (h_q + 2 * h_kv) * d)
            q, k, v = torch.split(rows, [h_q * d, h_kv * d, h_kv * d], 2)
            s["q"], s["k"], s["v"] = q.view(n, w, h_q, d), k.view(n, w, h_kv, d), v.view(n, w, h_kv, d)
            half = torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64)
            s["inv_freq"] = (1e6 ** (-2.0 * half / case["rot"])).float()
            at = s["kv_len"][:, None] - w + torch.arange(w, device="cuda", dtype=torch.int32)
            s["positions"] = (at + 1500000).to(torch.int32) if case["far"] else None
    if own:
        _keep(s)
    return s


def _keep(s):
    """What a program of the package holds between calls: dims, workspaces."""
    c, op, gdn = s["case"], s["case"]["op"], _gdn()
    need = 0
    if op == "verify":
        need = gdn.draft_verify_workspace_bytes(c["lanes"], c["window"], c["vocab"])
    else:
        cache = s["k_codes"] if "k_codes" in s else s["k_cache"]
        s["dims"] = gdn.KvDims.of(c["lanes"], c["window"], c["h_q"], c["h_kv"], c["d"], c["page"],
                                  cache.shape[0], s["table"].shape[1])
        if op == "attend":
            need = gdn.paged_attention_mxfp_workspace_bytes(s["dims"])
    s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")


def _gdn():
    import commit_gated_delta_amd
    return commit_gated_delta_amd


# ---------------------------------------------------------------------- work
def work(case):
    op, size = case["op"], 2 if case["type"] == "bf16" else 4
    if op == "verify":
        lens, vocab = _windows(case), case["vocab"]
        rows = sum(lens) + (sum(n - 1 for n in lens) if case["drafted"] else 0)
        return {"bytes": rows * vocab * size + sum(lens) * 12 + case["lanes"] * 12, "flops": 3 * rows * vocab}
    n, w, h_q, h_kv, d = (case[x] for x in ("lanes", "window", "h_q", "h_kv", "d"))
    if op == "append":
        rows = n * w
        held = 2 * h_kv * (d // 2 + d // 32 + 2 * d) if case["bits"] == 4 else 2 * h_kv * d * size
        return {"bytes": rows * ((2 * h_q + 2 * h_kv) * d * size + held) + (4 * rows if case["far"] else 4 * n),
                "flops": 3 * rows * (h_q + h_kv) * case["rot"]}
    lens = _kv_lens(case)
    seen = sum(sum(x - w + t + 1 for t in range(w)) for x in lens)
    return {"bytes": 2 * sum(lens) * h_kv * (d // 2 + d // 32) + n * w * h_q * d * (size + 4),
            "flops": 4 * seen * h_q * d}


# ---------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if c["op"] == "verify":
        return _own_verify(s) if own else _plain_verify(s)
    if c["op"] == "attend":
        return _own_attend(s) if own else _plain_attend(s)
    if c["bits"] == 4:
        return _own_append_fp4(s) if own else _plain_append_fp4(s)
    return _own_append(s) if own else _plain_append(s)


def _own_append(s):
    c = s["case"]
    q = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    _gdn().rope_append(s["dims"], s["t_lane"], s["q"], s["k"], s["v"], s["inv_freq"], c["rot"], q,
                       s["k_cache"], s["v_cache"], s["table"], s["kv_len"], positions=s["positions"],
                       interleaved=c["pairs"])
    return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}


def _own_append_fp4(s):
    c = s["case"]
    q = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    k, v = (torch.empty(s["k"].shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    _gdn().rope_append_mxfp(s["dims"], s["t_lane"], s["q"], s["k"], s["v"], s["inv_freq"], c["rot"], q,
                           s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["table"],
                           s["kv_len"], k_held=k, v_held=v, positions=s["positions"],
                           interleaved=c["pairs"])
    return {"q": q, "k": k, "v": v}


def _own_attend(s):
    o = torch.empty(s["q"].shape, device="cuda")
    _gdn().paged_attention_mxfp(s["dims"], s["t_lane"], s["q"], s["k_codes"], s["k_scales"], s["v_codes"],
                               s["v_scales"], s["table"], s["kv_len"], o, s["workspace"],
                               scale=s["case"]["d"] ** -0.5)
    return o


def _own_verify(s):
    n, w = s["tokens"].shape
    m, token = (torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(2))
    accept = torch.zeros(n, w, device="cuda")
    _gdn().draft_verify(s["t_lane"], s["logits"], s["draft_logits"], s["tokens"], s["uniforms"],
                        s["inv_temperature"], m, token, s["workspace"], accept=accept)
    return {"m": m, "token": token, "accept": accept}


# --------------------------------------------------------- the plain forms
def _rotated(s, x, wide):
    """x with the channels that turn turned; angles in 64 bits, the products
    in 32, or with wide in 64 too (what is rounded to 4 bits next)."""
    c = s["case"]
    n, w, rot = c["lanes"], c["window"], c["rot"]
    at = s["positions"]
    if at is None:
        at = s["kv_len"][:, None] - w + torch.arange(w, device="cuda")
    angle = at.double()[:, :, None, None] * s["inv_freq"].double()
    kind = torch.float64 if wide else torch.float32
    cos, sin, x = torch.cos(angle).to(kind), torch.sin(angle).to(kind), x.to(kind)
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["pairs"] else (x[..., : rot // 2], x[..., rot // 2: rot])
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((a, b), 4).flatten(3) if c["pairs"] else torch.cat((a, b), 3)
    return torch.cat((y, x[..., rot:]), 3)


def _new_places(s):
    """Page and row of every new token."""
    c = s["case"]
    at = s["kv_len"].long()[:, None] - c["window"] + torch.arange(c["window"], device="cuda")
    return torch.gather(s["table"].long(), 1, at // c["page"]), at % c["page"]


def _plain_append(s):
    page, row = _new_places(s)
    t = s["q"].dtype
    s["k_cache"][page, :, row] = _rotated(s, s["k"], False).to(t)
    s["v_cache"][page, :, row] = s["v"]
    return {"q": _rotated(s, s["q"], False).to(t), "k": s["k_cache"], "v": s["v_cache"]}


def _coded(x):
    """Codes and scale bytes of rows, and the values that they stand for."""
    x = x.unflatten(3, (-1, 32))
    most = x.abs().amax(4)
    mantissa, exponent = torch.frexp(most)              # most = mantissa 2^exponent, mantissa in [0.5, 1)
    e = (exponent - 3 + (mantissa > 0.75).to(exponent.dtype)).clamp(-126, 124)
    e = torch.where(most == 0, -126, e)
    y = torch.ldexp(x, -e[..., None])
    a = y.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int())
    table = torch.tensor(_VALUES, dtype=torch.float64, device=x.device)
    value = torch.ldexp(table[code.long()], e[..., None])
    value = torch.where(torch.signbit(x), -value, value).flatten(3)
    code = (code + 8 * torch.signbit(x).int()).flatten(3).to(torch.uint8)
    return code[..., 0::2] | code[..., 1::2] << 4, (e + 127).to(torch.uint8), value.to(torch.bfloat16)


def _plain_append_fp4(s):
    page, row = _new_places(s)
    held = {}
    for c, x in (("k", _rotated(s, s["k"], True)), ("v", s["v"].double())):
        codes, scales, held[c] = _coded(x)
        s[c + "_codes"][page, :, row] = codes
        s[c + "_scales"][page, :, row] = scales
    return {"q": _rotated(s, s["q"], False).to(s["q"].dtype), "k": held["k"], "v": held["v"]}


def _decoded(codes, scales):
    """float32 rows of codes and scale bytes."""
    table = torch.tensor(_VALUES + tuple(-x for x in _VALUES), device=codes.device)
    both = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), -1)
    x = both.flatten(-2).unflatten(-1, (-1, 32))
    return (x * torch.exp2(scales.float() - 127)[..., None]).flatten(-2)


def _plain_attend(s):
    c = s["case"]
    n, w, h_kv, d, group = c["lanes"], c["window"], c["h_kv"], c["d"], c["h_q"] // c["h_kv"]
    at = torch.arange(s["table"].shape[1] * c["page"], device="cuda")
    page, row = s["table"].long().clamp(min=0)[:, at // c["page"]], at % c["page"]

    def rows(x):                                        # [n, h_kv, positions, d]
        y = _decoded(s[x + "_codes"][page, :, row], s[x + "_scales"][page, :, row])
        return y.transpose(1, 2).contiguous()

    q = s["q"].float().view(n, w, h_kv, group, d).permute(0, 2, 1, 3, 4).reshape(n, h_kv, w * group, d)
    x = torch.matmul(q, rows("k").transpose(2, 3)) * d ** -0.5
    ends = (s["kv_len"][:, None] - w + torch.arange(w, device="cuda") + 1).repeat_interleave(group, 1)
    x = torch.where((at < ends[..., None])[:, None], x, -math.inf)
    x = torch.exp(x - x.amax(3, keepdim=True))
    x = x / x.sum(3, keepdim=True)
    o = torch.matmul(x, rows("v"))
    return o.view(n, h_kv, w, group, d).permute(0, 2, 1, 3, 4).reshape(n, w, c["h_q"], d)


def _plain_verify(s):
    """In 64 bits: a token is where a running sum passes a given number."""
    n, w = s["tokens"].shape
    t_lane = torch.tensor(s["t_lane"], device="cuda")
    it = s["inv_temperature"].double()[:, None, None]

    def chances(logits):
        x = logits.double() * it
        x = torch.exp(x - x.amax(2, keepdim=True))
        return x / x.sum(2, keepdim=True)

    p, drafts = chances(s["logits"]), s["tokens"][:, 1:].long()
    chance = torch.gather(p[:, :-1], 2, drafts[..., None])[..., 0]
    if s["draft_logits"] is None:
        q, drafted = None, torch.ones_like(chance)
    else:
        q = chances(s["draft_logits"])
        drafted = torch.gather(q, 2, drafts[..., None])[..., 0]
    there = torch.arange(w - 1, device="cuda") < t_lane[:, None] - 1
    taken = (s["uniforms"][:, :-1].double() * drafted < chance) & there
    m = 1 + torch.cumprod(taken.int(), 1).sum(1)
    accept = torch.zeros(n, w, device="cuda")
    accept[:, :-1] = torch.where(there, torch.clamp(chance / drafted, max=1.0), 0.0)
    last, lane = m == t_lane, torch.arange(n, device="cuda")
    whole = p[lane, m - 1]
    if w == 1:
        rest = whole
    elif q is None:
        at = (m - 1).clamp(max=w - 2)
        rest = whole.scatter(1, drafts[lane, at][:, None], 0.0)
    else:
        rest = torch.clamp(whole - q[lane, (m - 1).clamp(max=w - 2)], min=0.0)
    rest = torch.where((last | (rest.sum(1) == 0))[:, None], whole, rest)
    run_sum = torch.cumsum(rest, 1)
    border = s["uniforms"].double().gather(1, t_lane[:, None] - 1) * run_sum[:, -1:]
    token = torch.minimum((run_sum <= border).sum(1), rest.shape[1] - 1 - (rest > 0).int().flip(1).argmax(1))
    return {"m": m.to(torch.int32), "token": token.to(torch.int32), "accept": accept}


# ------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "verify":
        return _exact_verify(s)
    if case["op"] == "attend":
        return _exact_attend(s)
    return _exact_append(s)


def _exact_append(s):
    """Rotation as a product of complex numbers; the nearest multiple of the
    step that the codes have at a value's size."""
    c = s["case"]
    rot, where = c["rot"], s["positions"]

    def turned(x):
        x = x.double()
        z = x[..., :rot].unflatten(3, (rot // 2, 2)) if c["pairs"] else x[..., :rot].unflatten(3, (2, rot // 2)).transpose(3, 4)
        z = torch.complex(z[..., 0].contiguous(), z[..., 1].contiguous())
        for n in range(c["lanes"]):
            at = torch.arange(c["window"], device="cuda") + (s["kv_len"][n] - c["window"]) if where is None else where[n]
            angle = torch.outer(at.double(), s["inv_freq"].double())[:, None]
            z[n] *= torch.polar(torch.ones_like(angle), angle)
        parts = (z.real, z.imag)
        y = x.clone()
        y[..., :rot] = torch.stack(parts, 4).flatten(3) if c["pairs"] else torch.cat(parts, 3)
        return y

    q, k, v = turned(s["q"]), turned(s["k"]), s["v"].double()
    if c["bits"] == 4:
        held = []
        for x in (k, v):
            blocks = x.reshape(-1, 32)
            step = torch.exp2(torch.ceil(torch.log2(blocks.abs().amax(1, keepdim=True) / 6)))
            y = blocks.abs() / step
            unit = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
            held.append((torch.round(y / unit) * unit * step * torch.sign(blocks)).view(x.shape))
        return {"q": q, "k": held[0], "v": held[1]}
    caches = {}
    for name, x in (("k", k), ("v", v)):
        cache, table = s[name + "_cache"].double(), s["table"].tolist()
        for n, length in enumerate(s["kv_len"].tolist()):
            for t in range(c["window"]):
                at = length - c["window"] + t
                cache[table[n][at // c["page"]], :, at % c["page"]] = x[n, t]
        caches[name] = cache
    return {"q": q, "k": caches["k"], "v": caches["v"]}


def _exact_attend(s):
    """Lane by lane."""
    c = s["case"]
    w, h_kv, d, group = c["window"], c["h_kv"], c["d"], c["h_q"] // c["h_kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")

    def rows(x, pages, length):
        codes, b = s[x + "_codes"][pages].int(), s[x + "_scales"][pages].int()
        nibble = torch.stack((codes % 16, codes // 16), 4).flatten(3)
        e, f = nibble % 8 // 2, nibble % 2                # exponent and fraction bit
        value = torch.where(e == 0, 0.5 * f.double(), torch.ldexp(1 + 0.5 * f.double(), e - 1))
        value = torch.where(nibble >= 8, -value, value)
        value = torch.ldexp(value, (b - 127).repeat_interleave(32, 3))
        return value.transpose(0, 1).reshape(h_kv, -1, d)[:, :length]

    for n, length in enumerate(s["kv_len"].tolist()):
        pages = s["table"][n, : -(-length // c["page"])].long()
        k, v = rows("k", pages, length), rows("v", pages, length)
        for t in range(w):
            end = length - w + t + 1
            q = s["q"][n, t].double().view(h_kv, group, d)
            x = torch.softmax(torch.matmul(q, k[:, :end].transpose(1, 2).contiguous()) / math.sqrt(d), 2)
            out[n, t] = torch.matmul(x, v[:, :end]).view(-1, d)
    return out


def _exact_verify(s):
    """Chances of acceptance, draft by draft."""
    n, w = s["tokens"].shape
    accept = torch.zeros(n, w, dtype=torch.float64, device="cuda")
    for i, length in enumerate(s["t_lane"]):
        for t in range(length - 1):
            token, it = s["tokens"][i, t + 1].long(), s["inv_temperature"][i].double()
            log_p = torch.log_softmax(s["logits"][i, t].double() * it, 0)[token]
            if s["draft_logits"] is not None:
                log_p = log_p - torch.log_softmax(s["draft_logits"][i, t].double() * it, 0)[token]
            accept[i, t] = torch.exp(torch.clamp(log_p, max=0.0))
    return {"m": None, "token": None, "accept": accept}

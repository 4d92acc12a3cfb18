"""64-bit references of the position rotation, the 4-bit cache, attention over
it and the verification of drafted tokens, written from their definitions,
with the error bounds the tests hold the kernels to.

Unit: U32 = 2^-24, half a step of f32.
"""
import math

import torch

U32 = 2.0 ** -24
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------- rotation
def turned(x, pos, inv_freq, rot, pairs):
    """x [.., h, d] (any type) at positions pos [..]: the turned rows in f64
    and the bound of their f32 error.  Cosine and sine are off by at most 4
    U32: the reduced angle (below 0.79) is rounded to f32 once, the series'
    last two operations round once each, earlier terms and the cut-off add
    less than one U32 together.  Two products and a sum round once more each:
    6 U32 of |a| + |b|."""
    x = x.double().cpu()
    pos, f = pos.double().cpu(), inv_freq.double().cpu()
    angle = (pos[..., None] * f)[..., None, :]
    c, s = torch.cos(angle), torch.sin(angle)
    y, tol = x.clone(), torch.zeros_like(x)
    if pairs:
        ia, ib = slice(0, rot, 2), slice(1, rot, 2)
    else:
        ia, ib = slice(0, rot // 2), slice(rot // 2, rot)
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    tol[..., ia] = tol[..., ib] = 6 * U32 * (a.abs() + b.abs())
    return y, tol


# -------------------------------------------------------------- 4-bit cache
def decode(codes, scales):
    """f64 rows of codes [.., d / 2] and scale bytes [.., d / 32]."""
    codes, scales = codes.cpu(), scales.cpu()
    grid = torch.tensor(GRID + tuple(-g for g in GRID), dtype=torch.float64)
    x = grid[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()]
    s = torch.exp2(scales.double() - 127).masked_fill(scales == 255, math.nan)
    return x * s.repeat_interleave(32, -1)


def encode(x):
    """Codes and scale bytes of f64 rows [.., d], finite or not."""
    blocks = x.double().cpu().unflatten(-1, (-1, 32))
    most = blocks.abs().amax(-1)
    finite = torch.isfinite(blocks).all(-1)
    safe = torch.where(finite & (most > 0), most, 1.0)
    e = torch.ceil(torch.log2(safe / 6))
    # (log2 rounds: step to the smallest power of two with most <= 6 s)
    e = torch.where(safe > 6 * torch.exp2(e), e + 1, e)
    e = torch.where(safe <= 6 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(most == 0, torch.full_like(e, -126), e).clamp(-126, 124)
    y = torch.where(finite[..., None], blocks, 0.0) * torch.exp2(-e)[..., None]
    a = y.abs().clamp(max=6.0)
    unit = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    near = torch.round(a / unit) * unit          # (round takes ties to even)
    grid = torch.tensor(GRID, dtype=torch.float64)
    code = torch.searchsorted(grid, near.contiguous())
    code = code + 8 * torch.signbit(y)
    code = torch.where(finite[..., None], code, 0).flatten(-2)
    codes = (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)
    return codes, torch.where(finite, e + 127, 255.0).to(torch.uint8)


def held_ok(x, tol, codes, scales):
    """Whether codes and scales are a right answer for rows within tol of x:
    the scale fits a largest magnitude within tol, and every value lies in
    its code's rounding cell, moved by tol."""
    b = scales.cpu().double()
    most, slack = x.abs().unflatten(-1, (-1, 32)), tol.unflatten(-1, (-1, 32))
    hi, lo = (most + slack).amax(-1), (most - slack).amax(-1)
    s = torch.exp2(b - 127)
    ok = (lo <= 6 * s) & ((hi > 3 * s) | (b == 1))
    v = decode(codes, scales)
    s = s.repeat_interleave(32, -1)
    a = (v / s).abs()
    grid = torch.tensor(GRID + (math.inf,), dtype=torch.float64)
    at = torch.searchsorted(grid, a.contiguous())
    above = torch.where(at < 7, (grid[at] + grid[(at + 1).clamp(max=7)]) / 2, math.inf)
    below = torch.where(at > 0, (grid[at] + grid[(at - 1).clamp(min=0)]) / 2, -math.inf)
    y = torch.where(torch.signbit(v), -x, x) / s
    d = tol / s
    # (a value that rounds to zero may carry either sign)
    y = torch.where(at == 0, y.abs(), y)
    return bool(ok.all()) and bool(((y <= above + d) & (y >= below - d)).all())


# ---------------------------------------------------------------- attention
def attend(q, k, v, table, kv_len, t_lane, scale, page, n_pages):
    """f64 attention over decoded rows k, v [n_pages, h_kv, page, d]: (o,
    bound); rows of idle tokens are NaN in o.

    A score is off by (d + 8) U32 of the sum of its terms' sizes (the codes'
    values and the bf16 parts of an f32 query are exact).  Through the softmax
    an error e of the scores (and of the largest one) moves an output by 4 e of
    sum p |v|, the sums by one step a position, and a few roundings."""
    N, T, Hq, d = q.shape
    Hkv = k.shape[1]
    group = Hq // Hkv
    q, table, kv_len = q.double().cpu(), table.cpu(), kv_len.cpu()
    o = torch.full(q.shape, math.nan, dtype=torch.float64)
    tol = torch.zeros(q.shape, dtype=torch.float64)
    cap = table.shape[1] * page
    for n in range(N):
        length = min(max(int(kv_len[n]), 0), cap)
        pos = torch.arange(length)
        pages = table[n, pos // page].long()
        ok = (pages >= 0) & (pages < n_pages)
        pos, pages = pos[ok], pages[ok]
        kk, vv = k[pages, :, pos % page], v[pages, :, pos % page]   # [L, Hkv, d]
        for t in range(t_lane[n]):
            sees = pos <= length - t_lane[n] + t
            if not bool(sees.any()):
                o[n, t] = 0
                continue
            for h in range(Hkv):
                a, b = kk[sees, h], vv[sees, h]                     # [L, d]
                rows = slice(h * group, (h + 1) * group)
                x = scale * q[n, t, rows] @ a.T                     # [group, L]
                size = abs(scale) * q[n, t, rows].abs() @ a.abs().T
                p = torch.softmax(x, 1)
                o[n, t, rows] = p @ b
                e = (d + 8) * U32 * size.amax(1) + 4 * U32
                mag = p @ b.abs()
                tol[n, t, rows] = mag * (4 * e[:, None] + (2 * a.shape[0] + 16) * U32)
    return o, tol + 1e-30


# ------------------------------------------------------------- verification
def usable(it):
    """Inverse temperatures within 1e-30 .. 1e30 (as f32)."""
    lo, hi = torch.tensor([1e-30, 1e30])
    return (it.cpu() >= lo) & (it.cpu() <= hi)


def verify(t_lane, logits, draft, tokens, uniforms, it):
    """Per lane (m, next token, [chances], near): from the definition in f64,
    id by id.  near: a decision lies within what the kernels' rounding may
    turn (a chance within 2^-16 relative of its uniform, a running sum within
    1e-12 of its border)."""
    out = []
    V = logits.shape[2]
    fine = usable(it)
    for n, T in enumerate(t_lane):
        if T == 0:
            out.append(None)
            continue
        f = float(it[n])

        def dist(x):
            x = x.double().cpu()
            top = float(x.max())
            if not fine[n] or not math.isfinite(top) or bool(torch.isnan(x).any()):
                return None
            e = torch.exp((x - top) * f)
            return e / e.sum()

        m, chances, near, open_ = 1, [], False, True
        for t in range(T - 1):
            w, u = int(tokens[n, t + 1]), float(uniforms[n, t])
            p = dist(logits[n, t])
            q = dist(draft[n, t]) if draft is not None else None
            if p is None or (draft is not None and q is None):
                chances.append(math.nan)
                open_ = False
                continue
            inside = 0 <= w < V
            pw = float(p[w]) if inside else 0.0
            qw = (float(q[w]) if inside else 1.0) if draft is not None else 1.0
            chances.append(0.0 if pw == 0 else min(1.0, pw / qw) if qw > 0 else 1.0)
            if open_:
                near |= pw > 0 and abs(u * qw - pw) <= 2.0 ** -16 * pw
                if u * qw < pw:
                    m += 1
                else:
                    open_ = False
        t = m - 1
        p = dist(logits[n, t])
        bad = p is None
        rest = p
        if m < T and not bad:
            w = int(tokens[n, t + 1])
            if draft is not None:
                q = dist(draft[n, t])
                bad = q is None
                rest = None if bad else torch.clamp(p - q, min=0)
            elif 0 <= w < V:
                rest = p.clone()
                rest[w] = 0
        if bad:
            out.append((m, -1, chances, near))
            continue
        if float(rest.sum()) == 0:
            rest = p
        run = torch.cumsum(rest, 0)
        border = min(max(float(uniforms[n, T - 1]), 0.0), 1.0) * float(run[-1])
        hit = torch.nonzero((run > border) & (rest > 0))
        token = int(hit[0]) if len(hit) else int(torch.nonzero(rest > 0)[-1])
        gap = float((run - border).abs().min())
        near |= gap <= 1e-12 * float(run[-1])
        out.append((m, token, chances, near))
    return out


def chance_bound(logits, draft, it):
    """Relative error of a chance p / q whose sums are f32: each side's
    exponentials are exact to 4 steps plus the rounding of their arguments (at
    most the spread of the logits that count, 104), 32 are added up a thread
    and six times two halves, one step each; the chance's own exponentials are
    f64, and it is rounded once."""
    spread = 0.0
    it = torch.where(usable(it), it.cpu(), 0.0)
    for x in (logits, draft):
        if x is not None:
            x = x.double()
            x = torch.where(torch.isfinite(x), x, 0.0)
            if x.numel():
                spread = max(spread, float((x.amax() - x.amin()) * it.max()))
    return (2 * (4 + 2 * min(spread, 104.0) + 32 + 8) + 1) * U32

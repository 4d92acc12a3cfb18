"""Argument checks of the serving operators (linear attention with a decay per
head, paged attention and append, token scores) without a GPU: every call here
is refused on the host, or has nothing to launch."""
import ctypes
import math

import pytest
import torch

import commit_gated_delta_amd as gdn

OK, EINVAL, EUNSUP, EWORK = (gdn.GDN_OK, gdn.GDN_EINVAL, gdn.GDN_EUNSUPPORTED,
                             gdn.GDN_EWORKSPACE)
P = 1 << 20      # an aligned address that no refused call touches


def _i32(vals):
    return (ctypes.c_int32 * max(len(vals), 1))(*vals)


def _message():
    return gdn.lib.gdn_last_error().decode()


# --------------------------------------------------------------------- step
def _step(t=(1, 1), q=P, k=P, v=P, dt=gdn.GDN_BF16, g=P, S=P, o=P, flags=0,
          t_null=False, **dims):
    d = dict(n_layers=1, n_lanes=2, h_v=4, h_k=2, d_k=128, d_v=128, t_max=8)
    d.update(dims)
    return gdn.lib.gdn_decay_step(
        ctypes.byref(gdn.Dims.of(**d)), None if t_null else _i32(t), q, k, v,
        dt, g, S, o, 1.0, flags, None)


def test_step_refusals():
    assert _step(d_k=24) == EUNSUP
    for bad in (dict(h_v=3), dict(t_max=0), dict(t_max=65), dict(d_v=0),
                dict(d_v=1025), dict(n_lanes=0), dict(n_lanes=257),
                dict(n_layers=0), dict(t=(9, 1)), dict(t=(-1, 1)),
                dict(t_null=True), dict(q=None), dict(k=None), dict(v=None),
                dict(g=None), dict(S=None), dict(dt=2), dict(flags=1),
                dict(flags=4), dict(flags=32), dict(q=P + 8), dict(S=P + 4),
                dict(o=P + 2), dict(g=P + 2),
                dict(o=None, flags=gdn.GDN_FLAG_KEEP_STATE)):
        assert _step(**bad) == EINVAL, bad
        assert _message()
    both = gdn.GDN_FLAG_KEEP_STATE | gdn.GDN_FLAG_HEAD_DECAY
    assert _step(t=(0, 0), flags=both) == OK
    assert _step(t=(0, 0), o=None, q=None) == OK
    assert gdn.lib.gdn_decay_step(None, _i32([1]), P, P, P, 0, P, P, P, 1.0, 0,
                                  None) == EINVAL


# ------------------------------------------------------------------- prompt
def _prompt(lens=(5, 7), n=None, h_v=4, h_k=2, d_k=128, d_v=128, q=P, k=P, v=P,
            dt=gdn.GDN_BF16, g=P, S0=None, S=P, o=P, ws=P, ws_bytes=1 << 40,
            flags=0, lens_null=False):
    return gdn.lib.gdn_decay_prefill(
        len(lens) if n is None else n, None if lens_null else _i32(lens), h_v,
        h_k, d_k, d_v, q, k, v, dt, g, S0, S, o, ws, ws_bytes, 1.0, flags, None)


def test_prompt_refusals():
    assert _prompt(d_k=48) == EUNSUP
    for bad in (dict(n=0), dict(n=257), dict(lens=(5, -1)), dict(lens_null=True),
                dict(lens=(1 << 30, 1 << 30, 5)), dict(h_v=3), dict(h_k=0),
                dict(d_v=0), dict(d_v=2000), dict(q=None), dict(k=None),
                dict(v=None), dict(g=None), dict(dt=5), dict(flags=16),
                dict(flags=1), dict(S=None, o=None), dict(S0=P + 4),
                dict(S=P + 8), dict(o=P + 4), dict(v=P + 2), dict(g=P + 2)):
        assert _prompt(**bad) == EINVAL, bad
        assert _message()
    # nothing to do
    assert _prompt(lens=(0, 0), S=None) == OK


def test_prompt_workspace():
    w = lambda lens, *s: gdn.decay_prefill_workspace_bytes(lens, *s)
    assert w([5, -1], 4, 2, 128, 128) == 0
    assert w([5], 4, 3, 128, 128) == 0
    assert w([5], 4, 2, 100, 128) == 0
    big = w([100000], 4, 2, 128, 128)
    if big:
        assert _prompt(lens=(100000,), ws_bytes=big - 1) == EWORK
        assert _prompt(lens=(100000,), ws=None) == EWORK
        assert _prompt(lens=(100000,), ws=P + 8) == EINVAL


def test_prompt_without_tokens_needs_no_inputs():
    none = dict(q=None, k=None, v=None, g=None, o=None)
    assert _prompt(lens=(0, 0), S=None, **none) == EINVAL    # nothing is wanted
    assert _prompt(lens=(0, 1), **none) == EINVAL


# -------------------------------------------------------------------- paged
def _kv(**over):
    d = dict(n_lanes=2, t_max=4, h_q=8, h_kv=2, d=128, page_size=16,
             n_pages=100, max_pages=10)
    d.update(over)
    return gdn.KvDims.of(**d)


BAD_KV = [dict(n_lanes=0), dict(n_lanes=257), dict(t_max=0), dict(t_max=65),
          dict(h_q=7), dict(h_q=0), dict(h_kv=0), dict(page_size=0),
          dict(n_pages=0), dict(max_pages=0),
          dict(page_size=1 << 15, max_pages=1 << 15), dict(d=0)]


def _attend(t=(1, 1), q=P, k=P, v=P, dt=gdn.GDN_BF16, table=P, lens=P, o=P,
            ws=P, ws_bytes=1 << 40, t_null=False, **dims):
    return gdn.lib.gdn_paged_attention(
        ctypes.byref(_kv(**dims)), None if t_null else _i32(t), q, k, v, dt,
        table, lens, o, ws, ws_bytes, 1.0, None)


def _append(t=(1, 1), k=P, v=P, dt=gdn.GDN_BF16, kc=P, vc=P, table=P, lens=P,
            t_null=False, **dims):
    return gdn.lib.gdn_kv_append(
        ctypes.byref(_kv(**dims)), None if t_null else _i32(t), k, v, dt, kc,
        vc, table, lens, None)


def test_attention_refusals():
    assert _attend(d=96) == EUNSUP
    for bad in BAD_KV + [dict(t=(5, 1)), dict(t=(-1, 1)), dict(t_null=True),
                         dict(q=None), dict(k=None), dict(v=None),
                         dict(table=None), dict(lens=None), dict(o=None),
                         dict(dt=3), dict(q=P + 8), dict(k=P + 2),
                         dict(v=P + 4), dict(o=P + 4), dict(ws=P + 8),
                         dict(table=P + 2), dict(lens=P + 1)]:
        assert _attend(**bad) == EINVAL, bad
        assert _message()
    need = gdn.paged_attention_workspace_bytes(_kv())
    if need:
        assert _attend(ws_bytes=need - 1) == EWORK
        assert _attend(ws=None) == EWORK
    assert _attend(t=(0, 0)) == OK
    for bad in BAD_KV + [dict(d=96)]:
        assert gdn.paged_attention_workspace_bytes(_kv(**bad)) == 0
    assert gdn.lib.gdn_paged_attention_workspace_bytes(None) == 0


def test_page_division():
    """The multiplier the kernels divide positions by the page size with, for
    every page size class and positions up to its limit."""
    for page in list(range(1, 130)) + [255, 256, 257, 1000, 4095, 65537, (1 << 28) + 1]:
        shift = 0
        while 1 << shift < page:
            shift += 1
        mul = ((((1 << shift) - page) << 32) // page + 1) & 0xffffffff
        for q in (0, 1, 2, 3, 7, 1000, (1 << 29) // page):
            for pos in (q * page - 1, q * page, q * page + page // 2):
                if 0 <= pos < 1 << 29:
                    assert (((pos * mul) >> 32) + pos) >> shift == pos // page


def test_append_refusals():
    assert _append(d=80) == EUNSUP
    for bad in BAD_KV + [dict(t=(5, 1)), dict(t=(0, -1)), dict(t_null=True),
                         dict(k=None), dict(v=None), dict(kc=None),
                         dict(vc=None), dict(table=None), dict(lens=None),
                         dict(dt=2), dict(k=P + 8), dict(vc=P + 4),
                         dict(table=P + 2)]:
        assert _append(**bad) == EINVAL, bad
    assert _append(t=(0, 0)) == OK


# ------------------------------------------------------------------- scores
def _scores(rows=4, vocab=1000, stride=1000, logits=P, dt=gdn.GDN_F32,
            tokens=P, top=5, it=1.0, lp=P, ent=P, ids=P, best=P, ws=P,
            ws_bytes=1 << 40):
    return gdn.lib.gdn_token_scores(rows, vocab, stride, logits, dt, tokens,
                                    top, it, lp, ent, ids, best, ws, ws_bytes,
                                    None)


def test_scores_refusals():
    for bad in (dict(rows=0), dict(rows=-1), dict(vocab=0), dict(stride=999),
                dict(vocab=2**30 + 1, stride=2**31), dict(top=-1), dict(top=33), dict(vocab=4, stride=4),
                dict(logits=None), dict(dt=2), dict(it=0.0), dict(it=-1.0),
                dict(it=math.inf), dict(it=math.nan), dict(it=1e-31), dict(it=1e31), dict(tokens=None),
                dict(lp=None), dict(ids=None), dict(best=None),
                dict(lp=None, tokens=None, ent=None, top=0),
                dict(logits=P + 2), dict(dt=gdn.GDN_BF16, logits=P + 1),
                dict(tokens=P + 2), dict(ids=P + 1), dict(ws=P + 8)):
        assert _scores(**bad) == EINVAL, bad
        assert _message()
    for rows, vocab, top in ((1, 200000, 5), (64, 131072, 0), (5000, 1000, 32)):
        need = gdn.token_scores_workspace_bytes(rows, vocab, top)
        if need:
            a = dict(rows=rows, vocab=vocab, stride=vocab, top=top)
            assert _scores(ws_bytes=need - 1, **a) == EWORK
            assert _scores(ws=None, **a) == EWORK
    assert gdn.token_scores_workspace_bytes(0, 5, 1) == 0
    assert gdn.token_scores_workspace_bytes(3, 5, 6) == 0


# ------------------------------------------------------------------ binding
def test_binding_refuses_tensors_that_do_not_fit():
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)
    with pytest.raises(ValueError):
        gdn._lanes([1], 2)
    with pytest.raises(TypeError):
        gdn._code(torch.float64)
    for t in (z(5, t=torch.float32), z(4, 2)[:, 0], z(3)):   # type, order, size
        with pytest.raises(ValueError):
            gdn._tensor(t, "x", torch.bfloat16, 4, -1)
    with pytest.raises(ValueError):                          # not on a device
        gdn._tensor(z(4), "x", torch.bfloat16, 4, 0)
    x = z(4)     # (a host tensor's device number is -1)
    assert gdn._tensor(x, "x", torch.bfloat16, 4, -1) == x.data_ptr()
    assert gdn._optional(None, "x", torch.bfloat16, 4, 0) is None

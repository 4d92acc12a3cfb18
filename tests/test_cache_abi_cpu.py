"""Argument checks of the rotating cache writers, the attention over the 4-bit
cache and the verification of drafts, without a GPU: every call here is
refused on the host, or has nothing to launch.  The references' own pins."""
import ctypes
import math

import pytest
import torch

import commit_gated_delta_amd as gdn
from tests import cache_ref as ref

OK, EINVAL, EUNSUP, EWORK = (gdn.GDN_OK, gdn.GDN_EINVAL, gdn.GDN_EUNSUPPORTED,
                             gdn.GDN_EWORKSPACE)
P = 1 << 20      # an aligned address that no refused call touches


def _i32(vals):
    return (ctypes.c_int32 * max(len(vals), 1))(*vals)


def _message():
    return gdn.lib.gdn_last_error().decode()


def _kv(**over):
    d = dict(n_lanes=2, t_max=4, h_q=8, h_kv=2, d=128, page_size=16,
             n_pages=100, max_pages=10)
    d.update(over)
    return gdn.KvDims.of(**d)


BAD_KV = [dict(n_lanes=0), dict(n_lanes=257), dict(t_max=0), dict(t_max=65),
          dict(h_q=7), dict(h_q=0), dict(h_kv=0), dict(page_size=0),
          dict(n_pages=0), dict(max_pages=0),
          dict(page_size=1 << 15, max_pages=1 << 15), dict(d=0)]


# ----------------------------------------------------------------- rotation
def _rope(fp4, t=(1, 1), q=P, qs=1024, k=P, ks=256, v=P, vs=256,
          dt=gdn.GDN_BF16, f=P, rot=64, pos=None, q_out=P, caches=None,
          held=(None, None), table=P, lens=P, flags=0, t_null=False, **dims):
    head = (ctypes.byref(_kv(**dims)), None if t_null else _i32(t), q, qs, k,
            ks, v, vs, dt, f, rot, pos, q_out)
    caches = caches or [P] * (4 if fp4 else 2)
    if fp4:
        return gdn.lib.gdn_rope_append_mxfp(*head, *caches, table, lens, *held,
                                            flags, None)
    return gdn.lib.gdn_rope_append(*head, *caches, table, lens, flags, None)


@pytest.mark.parametrize("fp4", [False, True])
def test_rope_refusals(fp4):
    n = 4 if fp4 else 2
    assert _rope(fp4, d=80) == EUNSUP
    bad = BAD_KV + [
        dict(t=(5, 1)), dict(t=(-1, 1)), dict(t_null=True), dict(k=None),
        dict(v=None), dict(q_out=None), dict(q=None), dict(f=None),
        dict(table=None), dict(lens=None), dict(dt=2), dict(flags=1),
        dict(flags=64), dict(rot=-16), dict(rot=8), dict(rot=144),
        dict(rot=72), dict(qs=1023), dict(qs=1016), dict(qs=1028),
        dict(qs=1 << 41), dict(ks=255), dict(ks=260), dict(vs=248),
        dict(vs=1 << 50), dict(dt=gdn.GDN_F32, ks=258), dict(q=P + 8),
        dict(k=P + 4), dict(v=P + 2), dict(q_out=P + 8), dict(f=P + 2),
        dict(pos=P + 1), dict(table=P + 2), dict(lens=P + 3), dict(h_kv=3)]
    for i in range(n):
        for what in (None, P + 8):
            c = [P] * n
            c[i] = what
            bad.append(dict(caches=c))
    if fp4:
        bad += [dict(held=(P + 8, None)), dict(held=(None, P + 2)),
                dict(n_pages=1 << 27)]                   # 2^32 rows
    for b in bad:
        assert _rope(fp4, **b) == EINVAL, b
        assert _message()
    assert _rope(fp4, t=(0, 0)) == OK
    assert _rope(fp4, t=(0, 0), q=None, q_out=None, f=None, rot=0, qs=0) == OK
    assert _rope(fp4, t=(0, 0), flags=gdn.GDN_FLAG_ROPE_PAIRS, dt=gdn.GDN_F32, ks=260) == OK


# ---------------------------------------------------------------- attention
def _attend(t=(1, 1), q=P, dt=gdn.GDN_BF16, caches=(P, P, P, P), table=P,
            lens=P, o=P, ws=P, ws_bytes=1 << 40, t_null=False, **dims):
    return gdn.lib.gdn_paged_attention_mxfp(
        ctypes.byref(_kv(**dims)), None if t_null else _i32(t), q, dt, *caches,
        table, lens, o, ws, ws_bytes, 1.0, None)


def test_attention_refusals():
    assert _attend(d=96) == EUNSUP
    bad = BAD_KV + [dict(t=(5, 1)), dict(t=(-1, 1)), dict(t_null=True),
                    dict(q=None), dict(table=None), dict(lens=None),
                    dict(o=None), dict(dt=3), dict(q=P + 8), dict(o=P + 4),
                    dict(ws=P + 8), dict(table=P + 2), dict(lens=P + 1),
                    dict(n_pages=1 << 27)]               # 2^32 rows
    for i in range(4):
        for what in (None, P + 8):
            c = [P] * 4
            c[i] = what
            bad.append(dict(caches=c))
    for b in bad:
        assert _attend(**b) == EINVAL, b
        assert _message()
    need = gdn.paged_attention_mxfp_workspace_bytes(_kv())
    assert need > 0
    assert _attend(ws_bytes=need - 1) == EWORK
    assert _attend(ws=None) == EWORK
    assert _attend(t=(0, 0)) == OK
    for b in BAD_KV + [dict(d=96), dict(n_pages=1 << 27)]:
        assert gdn.paged_attention_mxfp_workspace_bytes(_kv(**b)) == 0
    assert gdn.lib.gdn_paged_attention_mxfp_workspace_bytes(None) == 0
    assert gdn.lib.gdn_paged_attention_mxfp(
        None, _i32([1]), P, 0, P, P, P, P, P, P, P, P, 1 << 40, 1.0, None) == EINVAL


# ------------------------------------------------------------- verification
def _verify(n=2, T=4, t=(1, 1), V=1000, x=P, xs=1000, y=P, ys=1000,
            dt=gdn.GDN_F32, tokens=P, u=P, it=P, m=P, token=P, accept=P, ws=P,
            ws_bytes=1 << 40, t_null=False):
    return gdn.lib.gdn_draft_verify(n, T, None if t_null else _i32(t), V, x,
                                    xs, y, ys, dt, tokens, u, it, m, token,
                                    accept, ws, ws_bytes, None)


def test_verify_refusals():
    for bad in (dict(n=0), dict(n=257), dict(T=0), dict(T=65), dict(V=0),
                dict(V=2**30 + 1, xs=2**31, ys=2**31), dict(xs=999),
                dict(ys=999), dict(xs=2**41), dict(ys=2**41), dict(dt=2),
                dict(t=(5, 1)), dict(t=(1, -1)), dict(t_null=True),
                dict(x=None), dict(tokens=None), dict(u=None), dict(it=None),
                dict(m=None), dict(token=None), dict(x=P + 2), dict(y=P + 2),
                dict(dt=gdn.GDN_BF16, x=P + 1), dict(tokens=P + 2),
                dict(u=P + 1), dict(it=P + 2), dict(m=P + 2),
                dict(token=P + 1), dict(accept=P + 2), dict(ws=P + 8)):
        assert _verify(**bad) == EINVAL, bad
        assert _message()
    assert _verify(t=(0, 0)) == OK
    assert _verify(t=(0, 0), y=None, ys=0, accept=None) == OK
    for n, T, V in ((1, 1, 131072), (8, 16, 131072), (64, 6, 5000)):
        need = gdn.draft_verify_workspace_bytes(n, T, V)
        if need:
            a = dict(n=n, T=T, t=(1,) * n, V=V, xs=V, ys=V)
            assert _verify(ws_bytes=need - 1, **a) == EWORK
            assert _verify(ws=None, **a) == EWORK
    # more threads than a launch may have
    a = dict(n=256, T=64, t=(1,) * 256, V=2**23, xs=2**23, ys=2**23)
    assert _verify(ws_bytes=gdn.draft_verify_workspace_bytes(256, 64, 2**23), **a) == EINVAL
    assert b"grid too large" in gdn.lib.gdn_last_error()
    for sizes in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (257, 1, 1), (1, 65, 1), (1, 1, 2**30 + 1)):
        assert gdn.draft_verify_workspace_bytes(*sizes) == 0


# ------------------------------------------------------------------ binding
def test_binding_refuses_rows_that_do_not_fit():
    with pytest.raises(ValueError):
        gdn._lane_ints([1, 2, 3], 2)
    with pytest.raises(OverflowError):
        gdn._lane_ints([1, 1 << 31], 2)
    with pytest.raises(TypeError):
        gdn._lane_ints([1, 0.5], 2)
    assert list(gdn._lane_ints((3, -1), 2)) == [3, -1]
    rows = torch.zeros(2, 4, 6 * 64, dtype=torch.bfloat16)
    take = lambda t, dev=-1, **o: gdn._rows(t, "q", torch.bfloat16, *[o.get(a, b) for a, b in (
        ("n", 2), ("T", 4), ("h", 2), ("d", 64))], dev)
    q = rows[..., :128].view(2, 4, 2, 64)
    assert take(q) == (q.data_ptr(), 384)                # a part of wider rows
    assert take(q.contiguous())[1] == 128
    assert take(rows[:1, :1, :128].view(1, 1, 2, 64), n=1, T=1)[1] == 128
    assert take(rows[:, 0, :128].view(2, 1, 2, 64), T=1)[1] == 4 * 384
    for t in (q.float(), q[:, :3], q.transpose(0, 1), q.transpose(1, 2), q[..., ::2],
              torch.zeros(3, 4, 2, 64, dtype=torch.bfloat16)[::2],
              torch.zeros(8, 2, 64, dtype=torch.bfloat16).expand(2, 8, 2, 64)[:, ::2],
              q.view(8, 2, 64)):
        with pytest.raises(ValueError):
            take(t)
    with pytest.raises(ValueError):
        take(q, dev=0)
    x = torch.zeros(2, 3, 10)
    take = lambda t, rows=3, dev=-1: gdn._logit_rows(t, "logits", torch.float32, 2, rows, 8, dev)
    assert take(x[..., :8]) == (x.data_ptr(), 10)
    assert take(x[..., 1:9])[1] == 10
    for t in (x, x[..., :8].bfloat16(), x[:, ::2, :8], x[:, :2, :8], x.transpose(0, 1)[..., :8],
              x.view(2, 3, 5, 2)[..., 0], x[:, :1, :8].expand(2, 3, 8)):
        with pytest.raises(ValueError):
            take(t)
    with pytest.raises(ValueError):
        take(x[..., :8], dev=0)


# --------------------------------------------------------------- references
def test_reference_of_the_format():
    """Hand-made rows: codes, scales and values by the definition."""
    row = torch.zeros(32)
    row[:8] = torch.tensor([6.0, -0.25, 0.75, 5.0, -3.5, 0.3, -6.0, 1.25])
    codes, scales = ref.encode(row)
    assert scales.tolist() == [127]
    assert codes[:4].tolist() == [0x87, 0x62, 0x1e, 0x2f]
    assert ref.decode(codes, scales)[:8].tolist() == [6, -0.0, 1, 4, -4, 0.5, -6, 1]
    codes, scales = ref.encode(row * 2.0 ** -7)
    assert scales.tolist() == [120] and codes[0] == 0x87
    row[0] = 6.1        # past 6: the next power of two
    assert ref.encode(row)[1].tolist() == [128]
    for x, b in ((torch.zeros(32), 1), (torch.full((32,), math.inf), 255), (torch.full((32,), 3e38), 251)):
        assert ref.encode(x)[1].tolist() == [b]


def test_reference_of_the_verification():
    """Two tokens, chances known by hand."""
    two = torch.tensor([[[math.log(0.75), math.log(0.25)]] * 2])
    draft = torch.tensor([[[math.log(0.5), math.log(0.5)]]])
    one = lambda w, u, v, d: ref.verify([2], two, d, torch.tensor([[0, w]]), torch.tensor([[u, v]]), torch.ones(1))[0]
    assert one(0, 0.99, 0.7, draft)[:2] == (2, 0)
    assert one(1, 0.49, 0.8, draft)[:2] == (2, 1)        # chance 0.5
    assert one(1, 0.51, 0.0, draft)[:2] == (1, 0)        # what is left is token 0
    assert one(0, 0.74, 0.0, None)[:2] == (2, 0)         # chance 0.75
    assert one(0, 0.76, 0.5, None)[:2] == (1, 1)
    assert abs(one(1, 0.1, 0.5, draft)[2][0] - 0.5) < 1e-6

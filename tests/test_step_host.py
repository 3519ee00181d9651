"""The calls around the attention of a step on a host without a GPU: rotary descriptors, refusals and
no-ops (nothing reaches a launch), and the references the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest
import torch

import affix_kv_cache_gb300 as ac
from affix_kv_cache_gb300 import _lib

from step_reference import frequencies, masked_attention, rotate, token_scores

BOGUS = 1 << 40
E, UNS = _lib.ACACHE_ERR_INVALID_ARG, _lib.ACACHE_ERR_UNSUPPORTED
NAN, INF = float("nan"), float("inf")


def _desc(hq=4, hkv=2, d=128, dtype="bf16", scale=0.088):
    return ac.attn_desc(hq, hkv, d, scale, dtype)


def _ref(x):
    return None if x is None else ctypes.byref(x)


def _rotate(dsc, rope=None, rows=4, pos=BOGUS, q=BOGUS, qs=512, k=BOGUS + (1 << 30), ks=256, qw=None, kw=None, eps=1e-6,
            qo=BOGUS + (2 << 30), qos=512, ko=BOGUS + (3 << 30), kos=256):
    return ac.lib().acache_rotate_qk(_ref(dsc), _ref(rope), rows, pos, q, qs, k, ks, qw, kw, eps, qo, qos, ko, kos, None)


def _store(dsc, rope=None, batch=1, rows=4, pos=BOGUS, slot=BOGUS, q=BOGUS, qs=512, k=BOGUS, ks=256, v=BOGUS, vs=256, qw=None,
           kw=None, eps=1e-6, qo=BOGUS + (2 << 30), kc=BOGUS, vc=BOGUS, ns=10, pb=0):
    return ac.lib().acache_rotate_store(_ref(dsc), _ref(rope), batch, rows, pos, slot, q, qs, k, ks, v, vs, qw, kw, eps, qo,
                                        kc, vc, ns, pb, None, None)


def _store8(dsc, rope=None, batch=1, rows=4, pos=BOGUS, slot=BOGUS, q=BOGUS, qs=512, k=BOGUS, ks=256, v=BOGUS, vs=256, qw=None,
            kw=None, eps=1e-6, qo=BOGUS + (2 << 30), kc=BOGUS, vc=BOGUS, sc=BOGUS, ns=10, pb=0):
    return ac.lib().acache_rotate_store_q8(_ref(dsc), _ref(rope), batch, rows, pos, slot, q, qs, k, ks, v, vs, qw, kw, eps, qo,
                                           kc, vc, sc, ns, pb, None, None)


def _masked(dsc, mask=None, batch=1, n_q=4, q=BOGUS, T=4, rs=BOGUS, kc=BOGUS, vc=BOGUS, ns=10, out=BOGUS):
    return ac.lib().acache_slot_attention_masked(_ref(dsc), _ref(mask), batch, n_q, q, T, rs, kc, vc, ns, out, None, None)


def _ragged(dsc, mask=None, batch=1, qs=BOGUS, n_q=4, tq=4, q=BOGUS, ks=BOGUS, T=4, rs=BOGUS, kc=BOGUS, vc=BOGUS, ns=10,
            out=BOGUS):
    return ac.lib().acache_slot_attention_masked_varlen(_ref(dsc), _ref(mask), batch, qs, n_q, tq, q, ks, T, rs, kc, vc, ns, out,
                                                        None, None)


def _scores(dtype=_lib.ACACHE_BF16, rows=2, vocab=100, x=BOGUS, stride=100, temp=1.0, tok=BOGUS, lp=BOGUS, ent=BOGUS, k=2,
            tt=BOGUS, tl=BOGUS):
    return ac.lib().acache_token_scores(dtype, rows, vocab, x, stride, temp, tok, lp, ent, k, tt, tl, None, None)


def test_struct_layouts():
    assert ctypes.sizeof(_lib.Rope) == 16 + 64 * 8
    assert ctypes.sizeof(_lib.Mask) == 32


@pytest.mark.parametrize("call", [_rotate, _store, _store8, _masked, _ragged])
def test_descriptor_refusals(call):
    for bad, want in ((ac.attn_desc(3, 2, 128, 0.1, "bf16"), E), (ac.attn_desc(0, 1, 128, 0.1, "bf16"), E),
                      (ac.attn_desc(4, 2, 96, 0.1, "bf16"), UNS), (_lib.AttnDesc(4, 2, 128, 0.1, 7), UNS),
                      (ac.attn_desc(4, 2, 128, INF, "bf16"), E)):
        assert call(bad) == want
    assert call(None) == E


@pytest.mark.parametrize("call,pointers", [
    (_rotate, ("qo", "ko")), (_store, ("slot", "k", "v", "qo", "kc", "vc")),
    (_store8, ("slot", "k", "v", "qo", "kc", "vc", "sc")), (_masked, ("q", "rs", "kc", "vc", "out")),
    (_ragged, ("qs", "q", "ks", "rs", "kc", "vc", "out"))])
def test_pointer_refusals(call, pointers):
    for name in pointers:
        assert call(_desc(), **{name: None}) == E, name
        if name not in ("slot", "rs", "qs", "ks", "sc"):
            assert call(_desc(), **{name: BOGUS + 8}) == E, name        # 16-byte alignment
    if call is _store8:
        assert call(_desc(), sc=BOGUS + 1) == E


@pytest.mark.parametrize("call", [_rotate, _store, _store8])
def test_rotation_refusals(call):
    r = ac.rope_desc(128)
    d = _desc()
    assert call(d, rope=r, pos=None) == E                              # a rotation needs positions
    assert call(d, rope=r, pos=BOGUS + 2) == E
    assert call(_desc(d=64), rope=r) == E                              # more than the head
    for field, value in (("rotary_dim", 63), ("rotary_dim", 0), ("rotary_dim", 130), ("amplitude", NAN)):
        bad = ac.rope_desc(128)
        setattr(bad, field, value)
        assert call(d, rope=bad) == E, field
    for eps in (-1e-6, NAN, INF):
        assert call(d, eps=eps) == E
    for name in ("qw", "kw"):
        assert call(d, **{name: BOGUS + 8}) == E
    assert call(d, qs=511) == E and call(d, qs=516) == E               # shorter than a row; not 16 bytes
    assert call(d, ks=255) == E and call(d, ks=-256) == E
    assert call(d, rows=-1) == E
    assert call(d, rows=0, q=None, k=None) == 0
    assert call(d, qo=BOGUS + 32) == E                                 # an output across its input
    assert call(d, qo=BOGUS, qs=1024) == E                             # the same place, another stride
    if call is _rotate:
        assert call(d, ks=1024, ko=BOGUS + (1 << 30)) == E
        assert call(d, q=None, k=None, qo=None, ko=None) == 0
    else:
        assert call(d, vs=250) == E and call(d, pb=11) == E and call(d, pb=-1) == E and call(d, ns=-1) == E
        assert call(d, batch=-1) == E and call(d, batch=0) == 0


@pytest.mark.parametrize("call", [_masked, _ragged])
def test_mask_refusals(call):
    d = _desc()
    for mask in (_lib.Mask(None, None, None, -1.0, 0), _lib.Mask(None, None, None, NAN, 0), _lib.Mask(None, None, None, INF, 0),
                 _lib.Mask(None, None, BOGUS, 0.0, 0),                 # slopes without positions
                 _lib.Mask(BOGUS + 2, None, None, 0.0, 0), _lib.Mask(None, BOGUS + 1, BOGUS, 0.0, 0)):
        assert call(d, mask=mask) == E
    assert call(d, T=0) == E and call(d, T=-1) == E and call(d, n_q=-1) == E and call(d, batch=-1) == E and call(d, ns=-1) == E
    assert call(d, batch=65536) == E and call(d, n_q=1 << 21) == E and call(d, T=0x7fffffff) == E and call(d, ns=1 << 30) == E
    none = dict(q=None, rs=None, kc=None, vc=None, out=None)
    assert call(d, n_q=0, **none) == 0 and call(d, batch=0, **none) == 0
    if call is _ragged:
        assert call(d, tq=-1) == E and call(d, tq=0, qs=None, ks=None, **none) == 0


def test_score_refusals():
    assert _scores(dtype=5) == UNS
    for bad in (dict(rows=-1), dict(vocab=-1), dict(vocab=0), dict(k=-1), dict(k=33), dict(k=3, vocab=2), dict(x=None),
                dict(x=BOGUS + 1), dict(stride=99), dict(temp=0.0), dict(temp=-1.0), dict(temp=NAN), dict(temp=INF),
                dict(temp=1e-45), dict(tok=None), dict(lp=None), dict(tt=None)):
        if "vocab" in bad and bad["vocab"] == 0:
            bad["k"] = 0
        assert _scores(**bad) == E, bad
    assert _scores(rows=0, x=None) == 0
    assert _scores(tok=None, lp=None, ent=None, k=0, tt=None, tl=None) == 0      # nothing is asked for


def test_binding_refuses_rows_that_are_not_evenly_spaced():
    d, r = _desc(), ac.rope_desc(128)
    k, pos = torch.zeros(6, 2, 128, dtype=torch.bfloat16), torch.zeros(6, dtype=torch.int32)
    with pytest.raises(ValueError):
        ac.acache_rotate_qk(d, r, 6, pos, torch.zeros(2, 4, 4, 128, dtype=torch.bfloat16)[:, :3], k, k, k)
    with pytest.raises(ValueError):
        ac.acache_rotate_qk(d, r, 6, pos, torch.zeros(6, 8, 128, dtype=torch.bfloat16)[:, ::2], k, k, k)
    with pytest.raises(ValueError):
        ac.acache_token_scores(2, 4, torch.zeros(4, 2).T)
    # a slice of a wider projection is evenly spaced
    qkv = torch.zeros(2, 5, 8, 128, dtype=torch.bfloat16)
    assert _lib._row_stride(qkv[:, :, :4], 4, 128) == 1024
    assert _lib._row_stride(qkv[:1, :1, :4], 4, 128) == 512           # a single row has no next one
    assert _lib._row_stride(qkv[:, 1:2, :4], 4, 128) == 5120


# ------------------------------------------------------------------------------------- rotary descriptors
@pytest.mark.parametrize("rd,theta", [(2, 1e4), (36, 1e4), (64, 5e5), (128, 1e6), (128, 1e4)])
@pytest.mark.parametrize("scaling,factor,n", [("none", 1.0, 0), ("linear", 4.0, 0), ("ntk", 4.0, 0), ("yarn", 16.0, 8192),
                                              ("yarn", 1.5, 100), ("yarn", 4.0, 3), ("bands", 8.0, 8192), ("bands", 2.0, 50)])
def test_descriptor_holds_the_frequencies(rd, theta, scaling, factor, n):
    if scaling == "ntk" and rd == 2:
        with pytest.raises(ac.AcacheError):
            ac.rope_desc(rd, theta, scaling=scaling, factor=factor)
        return
    r = ac.rope_desc(rd, theta, interleaved=True, scaling=scaling, factor=factor, trained_len=n)
    want, amp = frequencies(rd, theta, scaling, factor, n)
    assert r.rotary_dim == rd and r.interleaved == 1 and abs(r.amplitude - amp) <= 2.0 ** -24 * amp
    for i, f in enumerate(want):
        got = r.phase[i] * 2.0 ** -64 * 2 * math.pi
        # double powers and logarithms on both sides; a phase is a whole number of 2^-64 turns
        assert abs(got - f) <= 1e-13 * f + 2 * math.pi * 2.0 ** -64, i


def test_descriptor_from_frequencies_is_exact_modulo_a_turn():
    f = [0.0, 1.0, 2 * math.pi, -0.25, 1e-12, 7.5, 1e15]
    r = ac.rope_desc_frequencies(f, amplitude=2.0)
    assert r.rotary_dim == 14 and r.amplitude == 2.0 and r.interleaved == 0
    for i, x in enumerate(f):
        turns = x / (2 * math.pi)
        want = turns - math.floor(turns)
        got = r.phase[i] * 2.0 ** -64
        assert abs(got - want) <= 2.0 ** -53 or abs(abs(got - want) - 1) <= 2.0 ** -53, x
    # a tiny negative frequency's fraction rounds to a whole turn, which is none
    assert ac.rope_desc_frequencies([-1e-300]).phase[0] == 0


def test_descriptor_refusals_of_values():
    L = ac.lib()
    r = _lib.Rope()
    ok = dict(out=r, rd=64, theta=1e4, kind=0, factor=1.0, n=0, low=0.0, high=0.0)

    def init(**kw):
        a = dict(ok, **kw)
        return L.acache_rope_init(_ref(a["out"]), a["rd"], 0, a["theta"], a["kind"], a["factor"], a["n"], a["low"], a["high"])

    assert init() == 0
    for bad in (dict(out=None), dict(rd=0), dict(rd=63), dict(rd=130), dict(theta=0.0), dict(theta=NAN), dict(theta=INF), dict(kind=5),
                dict(kind=-1), dict(kind=1, factor=0.0), dict(kind=1, factor=NAN), dict(kind=2, rd=2, factor=2.0),
                dict(kind=3, factor=1.0, n=10), dict(kind=3, factor=2.0, n=0), dict(kind=3, factor=2.0, n=9, low=2.0, high=1.0),
                dict(kind=3, factor=2.0, n=9, theta=1.0), dict(kind=4, factor=2.0, n=-1), dict(kind=4, factor=2.0, n=9, low=0.0, high=3.0)):
        assert init(**bad) == E, bad
    f = (ctypes.c_double * 2)(1.0, INF)
    assert L.acache_rope_init_frequencies(_ref(r), 4, 0, f, 1.0) == E
    f[1] = 0.5
    assert L.acache_rope_init_frequencies(_ref(r), 4, 0, f, NAN) == E
    assert L.acache_rope_init_frequencies(_ref(r), 4, 0, None, 1.0) == E
    assert L.acache_rope_init_frequencies(_ref(r), 4, 0, f, 1.0) == 0


# ------------------------------------------------------------------------------------- the references
def test_reference_rotation_composes_and_keeps_lengths():
    g = torch.Generator().manual_seed(1)
    x = torch.randn((3, 2, 64), generator=g, dtype=torch.float64)
    f, _ = frequencies(48, 1e4)
    for inter in (False, True):
        a, _ = rotate(x, None, 0.0, [5, -7, 1000], f, 1.0, inter)
        b, _ = rotate(torch.from_numpy(a), None, 0.0, [3, 7, 2 ** 30], f, 1.0, inter)
        c, _ = rotate(x, None, 0.0, [8, 0, 2 ** 30 + 1000], f, 1.0, inter)
        assert np.abs(b - c).max() < 1e-9
        assert np.allclose((a ** 2).sum(-1), (x.numpy() ** 2).sum(-1))
        assert np.array_equal(a[..., 48:], x.numpy()[..., 48:])


def test_reference_attention_and_scores_agree_with_torch():
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn((n, 2, 64), generator=g) for n in (5, 9, 9))
    lo, hi = [0, 2, 4, 3, 9], [9, 5, 4, 4, 20]
    got, tol = masked_attention(q, np.arange(9), k, v, 0.2, lo, hi, pos=[3] * 5, slopes=[0.5, -0.25], cap=2.0)
    s = torch.einsum("ihd,thd->hit", q.double(), k.double()) * 0.2
    s = 2 * torch.tanh(s / 2) - torch.tensor([0.5, -0.25]).view(2, 1, 1) * (3 - torch.arange(9)).abs()
    t = torch.arange(9)
    see = (t >= torch.tensor(lo)[:, None]) & (t < torch.tensor(hi)[:, None])
    p = torch.softmax(s.masked_fill(~see, -math.inf), -1).nan_to_num()
    assert np.allclose(got, torch.einsum("hit,thd->ihd", p, v.double()).numpy(), atol=1e-12)
    assert (got[2] == 0).all() and (got[4] == 0).all() and (tol[0] > 0).all()
    x = torch.randn((4, 50), generator=g)
    x[1, 7], x[2, 3] = -math.inf, 9.0
    lp, H, order, _, _ = token_scores(x, 0.7)
    want = torch.log_softmax(x.double() / 0.7, -1)
    assert np.allclose(lp, want.numpy()) and np.allclose(H, torch.special.entr(want.exp()).sum(-1).numpy())
    assert order[2, 0] == 3 and order[1, -1] == 7

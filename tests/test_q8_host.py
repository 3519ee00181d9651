"""The 8-bit pool's entry points on a host without a GPU: refusals and no-ops (nothing reaches a
launch), and the reference the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import affix_kv_cache_gb300 as ac
from affix_kv_cache_gb300 import _lib

from q8_reference import VALUES, quantise, values

BOGUS = 1 << 40
E, U = _lib.ACACHE_ERR_INVALID_ARG, _lib.ACACHE_ERR_UNSUPPORTED


def _desc(hq=4, hkv=2, d=128, dtype="bf16"):
    return ac.attn_desc(hq, hkv, d, 0.088, dtype)


def _write(dsc, batch=1, rows=4, slot=BOGUS, kn=BOGUS, vn=BOGUS, kc=BOGUS, vc=BOGUS, sc=BOGUS, ns=10, pb=0):
    return ac.lib().acache_write_slots_q8(ctypes.byref(dsc) if dsc else None, batch, rows, slot, kn, vn, kc, vc, sc, ns, pb, None, None)


def _gather(dsc, batch=1, T=4, rs=BOGUS, kc=BOGUS, vc=BOGUS, sc=BOGUS, ns=10, ko=BOGUS, vo=BOGUS):
    return ac.lib().acache_gather_slots_q8(ctypes.byref(dsc), batch, T, rs, kc, vc, sc, ns, ko, vo, None, None)


def _attend(dsc, batch=1, n_q=4, q=BOGUS, T=4, rs=BOGUS, kc=BOGUS, vc=BOGUS, sc=BOGUS, ns=10, out=BOGUS, drop=0):
    return ac.lib().acache_slot_attention_q8(ctypes.byref(dsc), batch, n_q, q, T, rs, kc, vc, sc, ns, out, drop, None, None)


def _varlen(dsc, batch=1, qs=BOGUS, mq=4, tq=4, q=BOGUS, ks=BOGUS, mt=4, rs=BOGUS, kc=BOGUS, vc=BOGUS, sc=BOGUS, ns=10, out=BOGUS):
    return ac.lib().acache_slot_attention_varlen_q8(ctypes.byref(dsc), batch, qs, mq, tq, q, ks, mt, rs, kc, vc, sc, ns, out, 0, None, None)


def _both(dsc, batch=1, rows=4, slot=BOGUS, kn=BOGUS, vn=BOGUS, kc=BOGUS, vc=BOGUS, sc=BOGUS, ns=10, pb=0, n_q=4, q=BOGUS,
          T=4, rs=BOGUS, out=BOGUS):
    return ac.lib().acache_store_attend_q8(ctypes.byref(dsc), batch, rows, slot, kn, vn, kc, vc, sc, ns, pb, n_q, q, T, rs,
                                           out, 0, None, None)


@pytest.mark.parametrize("call", [_write, _gather, _attend, _varlen, _both])
def test_descriptor_refusals(call):
    for bad, want in ((ac.attn_desc(3, 2, 128, 0.1, "bf16"), E), (ac.attn_desc(0, 1, 128, 0.1, "bf16"), E),
                      (ac.attn_desc(4, 2, 96, 0.1, "bf16"), U), (_lib.AttnDesc(4, 2, 128, 0.1, 7), U),
                      (ac.attn_desc(4, 2, 128, float("inf"), "bf16"), E)):
        assert call(bad) == want


@pytest.mark.parametrize("call,pointers", [
    (_write, ("slot", "kn", "vn", "kc", "vc", "sc")), (_gather, ("rs", "kc", "vc", "sc", "ko", "vo")),
    (_attend, ("q", "rs", "kc", "vc", "sc", "out")), (_varlen, ("qs", "q", "ks", "rs", "kc", "vc", "sc", "out")),
    (_both, ("slot", "kn", "vn", "kc", "vc", "sc", "q", "rs", "out"))])
def test_pointer_refusals(call, pointers):
    for name in pointers:
        assert call(_desc(), **{name: None}) == E, name
        if name not in ("slot", "rs", "qs", "ks", "sc"):
            assert call(_desc(), **{name: BOGUS + 8}) == E, name        # 16-byte alignment
    assert call(_desc(), sc=BOGUS + 1) == E                             # scale pairs are 2-byte words


def test_scalar_refusals_and_noops():
    d = _desc()
    assert _write(None) == E
    assert _write(d, rows=-1) == E and _write(d, batch=-1) == E and _write(d, ns=-1) == E
    assert _write(d, pb=11) == E and _write(d, pb=-1) == E
    assert _attend(d, T=0) == E and _attend(d, n_q=-1) == E and _attend(d, T=-1) == E
    assert _varlen(d, mt=0) == E and _varlen(d, mq=-1) == E and _varlen(d, tq=-1) == E
    assert _both(d, T=0) == E and _both(d, pb=11) == E
    assert _gather(d, T=-1) == E
    none = dict(kc=None, vc=None, sc=None)
    assert _write(d, rows=0, slot=None, kn=None, vn=None, **none) == 0
    assert _gather(d, T=0, rs=None, ko=None, vo=None, **none) == 0
    assert _attend(d, n_q=0, q=None, rs=None, out=None, **none) == 0
    assert _attend(d, batch=0, q=None, rs=None, out=None, **none) == 0
    assert _varlen(d, tq=0, qs=None, ks=None, q=None, rs=None, out=None, **none) == 0
    assert _both(d, batch=0, slot=None, kn=None, vn=None, q=None, rs=None, out=None, **none) == 0
    assert _both(d, rows=0, n_q=0, slot=None, kn=None, vn=None, q=None, rs=None, out=None, **none) == 0


def test_sizes_past_the_launch_limits_are_refused():
    """Before anything is launched: a store in the same call would write through these pointers."""
    for call in (_attend, _both):
        assert call(_desc(), batch=65536) == E
        assert call(_desc(), ns=(2 ** 31 - 1) // 2) == E
        assert call(_desc(), n_q=65535 * 64 // 2 + 1) == E
    assert _varlen(_desc(), batch=65536) == E and _varlen(_desc(), ns=2 ** 30) == E
    assert _varlen(_desc(), mq=65535 * 32 + 1) == E


def test_binding_raises():
    with pytest.raises(ac.AcacheError) as e:
        ac.acache_slot_attention_q8(_desc(), 1, 4, None, 4, None, None, None, None, 8, None)
    assert e.value.status == E


def test_reference_matches_the_torch_format():
    codes = torch.arange(256, dtype=torch.uint8)
    t = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(VALUES, t, equal_nan=True)
    # rows whose exponent is known: torch's own conversion is the rounding
    g = torch.Generator().manual_seed(0)
    x = torch.rand((200, 64), generator=g) * 400
    x[:, 0] = 448.0
    c, s, bad = quantise(x)
    assert (s == 127).all() and not bad.any()
    assert np.array_equal(c, x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_reference_scales_at_their_borders():
    top = torch.tensor([448.0, float(np.nextafter(np.float32(448), np.float32(500))), 1.75, 0.0, 1e-30, 2.0 ** 46,
                        448 * 2.0 ** 38, 2.0 ** 47, float("inf"), float("nan")])
    c, s, bad = quantise(top[:, None])
    assert s.tolist() == [127, 128, 119, 77, 77, 165, 165, 255, 255, 255]
    assert bad.tolist() == [False] * 7 + [True] * 3
    assert np.isnan(values(c, s)[-1]).all()


CALLS = {  # the arguments of each call behind the descriptor, in order; tensors by name
    "acache_write_slots_q8": (1, 4, "write_slot", "k_new", "v_new", "k_cache", "v_cache", "kv_scale", 10, 0),
    "acache_gather_slots_q8": (1, 4, "read_slot", "k_cache", "v_cache", "kv_scale", 10, "k_out", "v_out"),
    "acache_slot_attention_q8": (1, 4, "q", 4, "read_slot", "k_cache", "v_cache", "kv_scale", 10, "out"),
    "acache_slot_attention_varlen_q8": (1, "q_start", 4, 4, "q", "kv_start", 4, "read_slot", "k_cache", "v_cache", "kv_scale", 10,
                                        "out"),
    "acache_store_attend_q8": (1, 4, "write_slot", "k_new", "v_new", "k_cache", "v_cache", "kv_scale", 10, 0, 4, "q", 4,
                               "read_slot", "out")}
TENSORS = [(c, a) for c, args in CALLS.items() for a in args + ("dev_status",) if isinstance(a, str)]


@pytest.mark.parametrize("call,name", TENSORS)
def test_a_host_tensor_in_any_argument_is_refused(call, name):
    """It would reach a kernel as an address.  (The other arguments are plain addresses, which are the caller's.)"""
    host = torch.zeros(64)
    args = [host if a == name else BOGUS if isinstance(a, str) else a for a in CALLS[call]]
    with pytest.raises(ValueError, match="current device"):
        getattr(ac, call)(_desc(), *args, dev_status=host if name == "dev_status" else None)


def test_sizes_past_32_bit_indices_are_refused():
    """Their tile and item numbers would wrap: keys were rounded up to a negative number of tiles, and the
    call returned without an output or a status.  (One less passes the checks and reaches a host without a
    GPU.)"""
    longest = 2 ** 31 - 1024
    for call, name in ((_attend, "T"), (_both, "T"), (_varlen, "mt")):
        for n in (longest + 1, 2 ** 31 - 1):
            assert call(_desc(), **{name: n}) == E
        if not torch.cuda.is_available():
            assert call(_desc(), **{name: longest}) == _lib.ACACHE_ERR_CUDA
    wide = 2 ** 24 + 1
    for call in (_write, _gather, _attend, _varlen):
        assert call(_desc(hq=wide, hkv=wide), ns=1) == E
    assert _both(_desc(hq=wide, hkv=wide), ns=1, n_q=0) == E and _both(_desc(hq=wide, hkv=wide), ns=1, rows=0) == E
    if not torch.cuda.is_available():
        for call in (_write, _gather):
            assert call(_desc(hq=2 ** 24, hkv=2 ** 24), ns=1) == _lib.ACACHE_ERR_CUDA

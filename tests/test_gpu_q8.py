"""GPU parity of the 8-bit KV pool: quantising store, read-back, read-slot attention (fixed and
ragged), store-then-attend, and a run of them together, against 64-bit references."""
import numpy as np
import pytest
import torch

import affix_kv_cache_gb300 as ac
from affix_kv_cache_gb300 import _lib

from gpu_helpers import dev
from q8_reference import assert_attention, attention, quantise, random_pool, values
from test_q8_host import CALLS, TENSORS

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _desc(hq, hkv, d, dtype, scale=None):
    return ac.attn_desc(hq, hkv, d, d ** -0.5 if scale is None else scale, dtype)


# ------------------------------------------------------------------------------------- store
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("hkv,d", [(1, 64), (3, 64), (4, 128), (32, 128), (1, 128)])
@pytest.mark.parametrize("B,rows", [(1, 1), (3, 37), (2, 600)])
def test_store_is_bit_exact(dtype, hkv, d, B, rows):
    g = torch.Generator().manual_seed(hkv * 1000 + d + rows)
    ns, priv0 = B * rows + 90, 50
    slots = (priv0 + torch.randperm(ns - priv0, generator=g)[:B * rows]).to(torch.int32).view(B, rows)
    new = [(torch.randn((B, rows, hkv, d), generator=g) * torch.exp(3 * torch.randn((B, rows, hkv, 1), generator=g))).to(dtype)
           for _ in range(2)]
    new[0][0, 0, 0] = 0.0                                        # a zero row
    kc, vc = (torch.randint(0, 256, (ns, hkv, d), generator=g, dtype=torch.uint8) for _ in range(2))
    sc = torch.randint(0, 256, (ns, hkv, 2), generator=g, dtype=torch.uint8)
    gk, gv, gs, st = dev(kc), dev(vc), dev(sc), _status()
    ac.acache_write_slots_q8(_desc(hkv, hkv, d, dtype), B, rows, dev(slots), dev(new[0]), dev(new[1]), gk, gv, gs, ns, priv0,
                             dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    at = slots.view(-1).long()
    for i, (c, x) in enumerate(((kc, new[0]), (vc, new[1]))):
        codes, scale, _ = quantise(x.view(B * rows, hkv, d))
        c[at], sc[at, :, i] = torch.from_numpy(codes), torch.from_numpy(scale)
    assert torch.equal(gk.cpu(), kc) and torch.equal(gv.cpu(), vc) and torch.equal(gs.cpu(), sc)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_store_at_the_borders_of_the_format(dtype):
    d, hkv = 64, 1
    tops = [448.0, 450.0, 3.5, 3.515625, 2.0 ** 46, 448 * 2.0 ** 38, 2.0 ** 47, 3e38, float("inf"), -float("inf"), float("nan"),
            1e-20, 2.0 ** -59, 2.0 ** -60, 2.0 ** -130, 0.0]
    x = torch.zeros((1, len(tops), hkv, d))
    g = torch.Generator().manual_seed(4)
    for i, t in enumerate(tops):
        x[0, i, 0] = (torch.rand(d, generator=g) * 2 - 1) * (t if np.isfinite(t) else 1.0)
        x[0, i, 0, 17] = t
    x = x.to(dtype)
    n = len(tops)
    kc, vc = (torch.zeros((n, hkv, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    sc, st = torch.zeros((n, hkv, 2), dtype=torch.uint8, device="cuda"), _status()
    slots = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    ac.acache_write_slots_q8(_desc(1, 1, d, dtype), 1, n, slots, dev(x), dev(x), kc, vc, sc, n, 0, dev_status=st)
    torch.cuda.synchronize()
    codes, scale, bad = quantise(x[0])
    assert bad.any() and st.item() == _lib.DEV_BAD_VALUE
    assert np.array_equal(kc.cpu().numpy(), codes) and np.array_equal(vc.cpu().numpy(), codes)
    assert np.array_equal(sc.cpu().numpy()[..., 0], scale) and np.array_equal(sc.cpu().numpy()[..., 1], scale)


def test_store_skips_and_flags_bad_and_shared_slots():
    d, hkv, ns = 128, 2, 40
    x = torch.randn((1, 4, hkv, d), generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    for slot, bit in ((-1, _lib.DEV_BAD_SLOT), (ns, _lib.DEV_BAD_SLOT), (2 ** 31 - 1, _lib.DEV_BAD_SLOT),
                      (9, _lib.DEV_SHARED_WRITE)):
        kc, vc = (torch.full((ns, hkv, d), 7, dtype=torch.uint8, device="cuda") for _ in range(2))
        sc, st = torch.full((ns, hkv, 2), 9, dtype=torch.uint8, device="cuda"), _status()
        slots = torch.tensor([[20, slot, 11, 39]], dtype=torch.int32, device="cuda")
        ac.acache_write_slots_q8(_desc(2, 2, d, BF16), 1, 4, slots, x, x, kc, vc, sc, ns, 10, dev_status=st)
        torch.cuda.synchronize()
        assert st.item() == bit
        wrote = torch.zeros(ns, dtype=torch.bool)
        wrote[[20, 11, 39]] = True
        for t, v in ((kc, 7), (vc, 7), (sc, 9)):
            assert (t.cpu()[~wrote] == v).all()
        codes, _, _ = quantise(x[0].cpu())
        assert np.array_equal(kc.cpu().numpy()[[20, 11, 39]], codes[[0, 2, 3]])


# ------------------------------------------------------------------------------------- read-back
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("hkv,d,B,T", [(1, 64, 1, 1), (3, 64, 2, 77), (4, 128, 3, 513), (32, 128, 2, 300)])
def test_read_back_is_exact_and_storing_it_again_changes_nothing(dtype, hkv, d, B, T):
    g = torch.Generator().manual_seed(hkv + d + T)
    ns = B * T + 31
    kc, vc, sc, kv, vv = random_pool(ns, hkv, d, g, spread=4.0)
    rs = torch.randperm(ns, generator=g)[:B * T].to(torch.int32).view(B, T)
    ko, vo = (torch.full((B, T, hkv, d), 5.0, dtype=dtype, device="cuda") for _ in range(2))
    st = _status()
    desc = _desc(hkv, hkv, d, dtype)
    k, v, s = dev(kc), dev(vc), dev(sc)
    ac.acache_gather_slots_q8(desc, B, T, dev(rs), k, v, s, ns, ko, vo, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    assert np.array_equal(ko.double().cpu().numpy(), kv[rs.numpy()])
    assert np.array_equal(vo.double().cpu().numpy(), vv[rs.numpy()])
    # Values, not bytes: a row whose largest element was rounded down to 224 * 2^e gets exponent
    # e - 1 the second time, and every code of it exactly doubles.
    ac.acache_write_slots_q8(desc, B, T, dev(rs), ko, vo, k, v, s, ns, 0, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    k, v, s = k.cpu().numpy(), v.cpu().numpy(), s.cpu().numpy()
    assert np.array_equal(values(k, s[..., 0]), kv) and np.array_equal(values(v, s[..., 1]), vv)


def test_read_back_skips_bad_slots_and_shows_poison():
    d, hkv, ns = 128, 2, 30
    kc, vc, sc, kv, vv = random_pool(ns, hkv, d, torch.Generator().manual_seed(2))
    sc[4, 1, 0], sc[5, 0, 1], sc[6] = 255, 200, 0
    rs = torch.tensor([[3, -1, 4, 5, ns, 6]], dtype=torch.int32)
    ko, vo = (torch.full((1, 6, hkv, d), 5.0, dtype=BF16, device="cuda") for _ in range(2))
    st = _status()
    ac.acache_gather_slots_q8(_desc(2, 2, d, BF16), 1, 6, dev(rs), dev(kc), dev(vc), dev(sc), ns, ko, vo, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == _lib.DEV_BAD_SLOT
    k, v = ko.double().cpu().numpy()[0], vo.double().cpu().numpy()[0]
    assert (k[[1, 4]] == 5).all() and (v[[1, 4]] == 5).all()
    for row, slot in ((0, 3), (2, 4), (3, 5), (5, 6)):
        assert np.array_equal(k[row], values(kc[slot].numpy(), sc[slot, :, 0].numpy()), equal_nan=True)
        assert np.array_equal(v[row], values(vc[slot].numpy(), sc[slot, :, 1].numpy()), equal_nan=True)


# ------------------------------------------------------------------------------------- attention
def _attend_case(B, n_q, hq, hkv, d, dtype, T, drop, seed, paged=False):
    g = torch.Generator().manual_seed(seed)
    ns = max(T + 40, 200)
    pool = random_pool(ns, hkv, d, g)
    q = (1.5 * torch.randn((B, n_q, hq, d), generator=g)).to(dtype)
    if paged:          # runs of consecutive slots, as a request's own pages are
        rs = torch.stack([(torch.arange(T) + 7 * b) % ns for b in range(B)]).to(torch.int32)
    else:
        rs = torch.stack([torch.randperm(ns, generator=g)[:T] for _ in range(B)]).to(torch.int32)
    if drop:
        rs[torch.rand((B, T), generator=g) < 0.35] = -1
    return pool, q, rs, ns


SHAPES = [  # B, n_q, hq, hkv, d, T
    (1, 1, 1, 1, 128, 1), (1, 1, 8, 2, 128, 127), (2, 1, 32, 8, 128, 128), (3, 1, 4, 4, 128, 129), (2, 5, 12, 4, 128, 300),
    (1, 32, 4, 4, 128, 1408), (2, 32, 28, 4, 128, 700), (1, 128, 2, 2, 128, 260), (1, 129, 2, 1, 128, 257),
    (1, 300, 2, 2, 128, 513), (2, 97, 7, 1, 128, 640), (1, 589, 3, 1, 128, 1000), (1, 256, 1, 1, 128, 2000),
    (1, 2, 160, 1, 128, 333), (1, 1, 4, 2, 64, 1), (2, 33, 8, 2, 64, 129), (1, 260, 4, 4, 64, 700), (1, 40, 28, 4, 64, 255),
]


@pytest.mark.parametrize("B,n_q,hq,hkv,d,T", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("drop", [False, True])
def test_attention_parity(B, n_q, hq, hkv, d, T, dtype, drop):
    (kc, vc, sc, kv, vv), q, rs, ns = _attend_case(B, n_q, hq, hkv, d, dtype, T, drop, 31 * T + n_q, paged=T % 2 == 0)
    out, st = torch.full(q.shape, float("nan"), dtype=dtype, device="cuda"), _status()
    args = (_desc(hq, hkv, d, dtype), B, n_q, dev(q), T, dev(rs), dev(kc), dev(vc), dev(sc), ns)
    ac.acache_slot_attention_q8(*args, out, drop_none=drop, dev_status=st)
    again = torch.empty_like(out)
    ac.acache_slot_attention_q8(*args, again, drop_none=drop, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    assert torch.equal(out, again)                             # the same bits every time
    for b in range(B):
        want, tol = attention(q[b], rs[b].numpy(), kv, vv, d ** -0.5, drop)
        assert_attention(out[b].double().cpu().numpy(), want, tol, f"request {b}")


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 128)])
@pytest.mark.parametrize("n_q", [1, 40, 300])
def test_attention_over_a_long_context(dtype, d, n_q):
    B, hq, hkv, T = 1, 2, 1, 9000
    (kc, vc, sc, kv, vv), q, rs, ns = _attend_case(B, n_q, hq, hkv, d, dtype, T, False, n_q + d)
    out = torch.empty(q.shape, dtype=dtype, device="cuda")
    ac.acache_slot_attention_q8(_desc(hq, hkv, d, dtype), B, n_q, dev(q), T, dev(rs), dev(kc), dev(vc), dev(sc), ns, out)
    want, tol = attention(q[0], rs[0].numpy(), kv, vv, d ** -0.5)
    assert_attention(out[0].double().cpu().numpy(), want, tol)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("n_q", [1, 200])
def test_attention_with_rows_of_very_different_size(dtype, d, n_q):
    """Query rows, keys and values of a head that differ by factors of 2^20: one large row must not
    cost its neighbours their precision."""
    B, hq, hkv, T = 1, 2, 2, 300
    g = torch.Generator().manual_seed(77)
    ns = 400
    x = [torch.randn((ns, hkv, d), generator=g) for _ in range(2)]
    x[0] *= 2.0 ** torch.randint(-20, 3, (ns, hkv, 1), generator=g)
    x[1] *= 2.0 ** torch.randint(-20, 21, (ns, hkv, 1), generator=g)
    (kc, ks, _), (vc, vs, _) = quantise(x[0]), quantise(x[1])
    kv, vv = values(kc, ks), values(vc, vs)
    sc = torch.from_numpy(np.stack((ks, vs), -1)).contiguous()
    q = (torch.randn((B, n_q, hq, d), generator=g) * 2.0 ** torch.randint(-20, 3, (B, n_q, hq, 1), generator=g)).to(dtype)
    q[0, -1, 0] = 0.0
    rs = torch.randperm(ns, generator=g)[None, :T].to(torch.int32)
    out = torch.empty(q.shape, dtype=dtype, device="cuda")
    ac.acache_slot_attention_q8(_desc(hq, hkv, d, dtype), B, n_q, dev(q), T, dev(rs), dev(torch.from_numpy(kc)),
                                dev(torch.from_numpy(vc)), dev(sc), ns, out)
    want, tol = attention(q[0], rs[0].numpy(), kv, vv, d ** -0.5)
    assert_attention(out[0].double().cpu().numpy(), want, tol)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("n_q,T", [(1, 200), (3, 1300), (300, 400)])
def test_masked_bad_and_poisoned_keys(dtype, d, n_q, T):
    hq, hkv = 4, 2
    (kc, vc, sc, kv, vv), q, rs, ns = _attend_case(3, n_q, hq, hkv, d, dtype, T, False, 5 + T)
    q, rs = q[:3], rs[:3].clone()
    rs[0] = -1                                                  # every key discarded: zeros
    rs[1, :T // 2] = -1                                         # whole tiles discarded
    poison = ns - 1                                             # NaN in K of head 0 and V of head 1
    sc[poison, 0, 0] = sc[poison, 1, 1] = 255
    kv[poison, 0], vv[poison, 1] = np.nan, np.nan
    rs[rs == poison] = 0
    st = _status()

    def run(rs, drop):
        out = torch.full(q.shape, float("nan"), dtype=dtype, device="cuda")
        ac.acache_slot_attention_q8(_desc(hq, hkv, d, dtype), 3, n_q, dev(q), T, dev(rs), dev(kc), dev(vc), dev(sc), ns, out,
                                    drop_none=drop, dev_status=st)
        torch.cuda.synchronize()
        return out.double().cpu().numpy()

    got = run(rs, True)
    assert st.item() == 0 and (got[0] == 0).all()
    for b in (1, 2):
        want, tol = attention(q[b], rs[b].numpy(), kv, vv, d ** -0.5, True)
        assert_attention(got[b], want, tol, f"discarded keys, request {b}")
    # without drop_none, and for other slots outside the pool: zero rows, flagged
    rs[2, T // 3], rs[2, -1] = ns, -7
    got = run(rs, False)
    assert st.item() == _lib.DEV_BAD_SLOT
    for b in range(3):
        want, tol = attention(q[b], rs[b].numpy(), kv, vv, d ** -0.5)
        assert_attention(got[b], want, tol, f"bad slots, request {b}")
    # a poisoned row reaches the heads that read it in the request that reads it, and nothing else
    rs[2, T // 3], rs[2, -1] = poison, 1
    got = run(rs, True)
    assert np.isnan(got[2]).all()
    want, tol = attention(q[1], rs[1].numpy(), kv, vv, d ** -0.5, True)
    assert_attention(got[1], want, tol, "beside a poisoned request")


# few rows, so that the keys are split over as many CTAs as there are tiles of 128 (or chunks of 64), up to 8
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_q", [1, 70, 150])
@pytest.mark.parametrize("T", [129, 330, 600, 750, 890, 1100])
@pytest.mark.parametrize("drop", [False, True])
def test_any_number_of_parts(d, n_q, T, drop):
    hq, hkv = 1, 1
    (kc, vc, sc, kv, vv), q, rs, ns = _attend_case(1, n_q, hq, hkv, d, BF16, T, drop, 7 * T + n_q)
    if drop:
        rs[0, 128:256] = -1                                     # a part that may hold no key at all
    args = (_desc(hq, hkv, d, BF16), 1, n_q, dev(q), T, dev(rs), dev(kc), dev(vc), dev(sc), ns)
    out, again = (torch.empty(q.shape, dtype=BF16, device="cuda") for _ in range(2))
    for o in (out, again):
        ac.acache_slot_attention_q8(*args, o, drop_none=drop)
    want, tol = attention(q[0], rs[0].numpy(), kv, vv, d ** -0.5, drop)
    assert_attention(out[0].double().cpu().numpy(), want, tol)
    assert torch.equal(out, again)                              # parts are merged in a fixed order


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("n_q", [1, 40, 300])
def test_a_poisoned_key_among_discarded_ones_is_not_lost(dtype, d, n_q):
    """The parts a row's keys are split into: one holds only discarded keys and the poisoned one."""
    hq, hkv, T = 2, 1, 2000
    (kc, vc, sc, kv, vv), q, rs, ns = _attend_case(1, n_q, hq, hkv, d, dtype, T, False, 21)
    sc[7, 0, 0] = 255
    rs[0, 64:] = -1
    rs[0][rs[0] == 7] = 1
    for at in (700, 1999):
        one = rs.clone()
        one[0, at] = 7
        out = torch.zeros(q.shape, dtype=dtype, device="cuda")
        ac.acache_slot_attention_q8(_desc(hq, hkv, d, dtype), 1, n_q, dev(q), T, dev(one), dev(kc), dev(vc), dev(sc), ns, out,
                                    drop_none=True)
        assert torch.isnan(out).all()


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 64)])
def test_non_finite_queries_stay_in_their_rows(dtype, d):
    hq, hkv, T, n_q = 2, 1, 260, 20
    (kc, vc, sc, kv, vv), q, rs, ns = _attend_case(1, n_q, hq, hkv, d, dtype, T, False, 3)
    q[0, 3, 0, 5], q[0, 9, 1, 0] = float("nan"), float("inf")
    out = torch.empty(q.shape, dtype=dtype, device="cuda")
    ac.acache_slot_attention_q8(_desc(hq, hkv, d, dtype), 1, n_q, dev(q), T, dev(rs), dev(kc), dev(vc), dev(sc), ns, out)
    got = out[0].double().cpu().numpy()
    assert np.isnan(got[3, 0]).all() and np.isnan(got[9, 1]).all()
    q[0, 3, 0], q[0, 9, 1] = 0.0, 0.0
    want, tol = attention(q[0], rs[0].numpy(), kv, vv, d ** -0.5)
    keep = np.ones((n_q, hq), bool)
    keep[3, 0] = keep[9, 1] = False
    assert_attention(got[keep], want[keep], tol[keep])


@pytest.mark.parametrize("scale", [0.0, -0.1, 2.0])
def test_any_finite_softmax_scale(scale):
    hq, hkv, T, n_q, d = 2, 1, 150, 9, 128
    (kc, vc, sc, kv, vv), q, rs, ns = _attend_case(1, n_q, hq, hkv, d, BF16, T, False, 8)
    out = torch.empty(q.shape, dtype=BF16, device="cuda")
    ac.acache_slot_attention_q8(_desc(hq, hkv, d, BF16, scale), 1, n_q, dev(q), T, dev(rs), dev(kc), dev(vc), dev(sc), ns, out)
    want, tol = attention(q[0], rs[0].numpy(), kv, vv, scale)
    assert_attention(out[0].double().cpu().numpy(), want, tol)


@pytest.mark.parametrize("scale", [1e-10, 1e-30, 1e-42])
@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("n_q", [1, 50, 300])
def test_tiny_scales_and_empty_query_rows(dtype, d, n_q, scale):
    """Every logit is next to zero, however small the factor that makes it so; masked keys stay out."""
    hq, hkv, T = 2, 1, 100
    (kc, vc, sc, kv, vv), q, rs, ns = _attend_case(1, n_q, hq, hkv, d, dtype, T, True, 13)
    q[0, 0, 0], q[0, -1, 1] = 0.0, 1e-37
    rs[0, :70] = -1
    rs[0, 71] = 5
    out = torch.empty(q.shape, dtype=dtype, device="cuda")
    ac.acache_slot_attention_q8(_desc(hq, hkv, d, dtype, scale), 1, n_q, dev(q), T, dev(rs), dev(kc), dev(vc), dev(sc), ns, out,
                                drop_none=True)
    want, tol = attention(q[0], rs[0].numpy(), kv, vv, scale, True)
    assert_attention(out[0].double().cpu().numpy(), want, tol)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("n_q", [1, 40, 300])
def test_buffers_at_odd_16_byte_addresses(dtype, d, n_q):
    """16 bytes is all the alignment that is asked for, and nothing before or behind a buffer is written."""
    B, hq, hkv, T = 2, 4, 2, 333
    (kc, vc, sc, kv, vv), q, rs, ns = _attend_case(B, n_q, hq, hkv, d, dtype, T, False, 17)

    def at16(x, fill=0):
        lead = 16 // x.element_size()
        room = torch.full((x.numel() + 2 * lead,), fill, dtype=x.dtype, device="cuda")
        assert room.data_ptr() % 32 == 0
        view = room[lead:lead + x.numel()].view(x.shape)
        view.copy_(x)
        return view, room

    (gq, _), (gk, _), (gv, _) = at16(q), at16(kc), at16(vc)
    out, room = at16(torch.zeros_like(q), fill=7)
    ac.acache_slot_attention_q8(_desc(hq, hkv, d, dtype), B, n_q, gq, T, dev(rs), gk, gv, dev(sc), ns, out)
    lead = 16 // q.element_size()
    assert (room[:lead] == 7).all() and (room[-lead:] == 7).all()
    for b in range(B):
        want, tol = attention(q[b], rs[b].numpy(), kv, vv, d ** -0.5)
        assert_attention(out[b].double().cpu().numpy(), want, tol)
    ko, kroom = at16(torch.zeros((B, T, hkv, d), dtype=dtype), fill=7)
    vo, vroom = at16(torch.zeros((B, T, hkv, d), dtype=dtype), fill=7)
    ac.acache_gather_slots_q8(_desc(hq, hkv, d, dtype), B, T, dev(rs), gk, gv, dev(sc), ns, ko, vo)
    assert np.array_equal(ko.double().cpu().numpy(), kv[rs.numpy()]) and np.array_equal(vo.double().cpu().numpy(), vv[rs.numpy()])
    assert all((x[:lead] == 7).all() and (x[-lead:] == 7).all() for x in (kroom, vroom))
    # storing what was read back keeps the values
    (nk, _), (nv, _) = at16(ko[0]), at16(vo[0])
    (gk2, kroom), (gv2, vroom), s2 = at16(torch.zeros_like(kc), 9), at16(torch.zeros_like(vc), 9), torch.zeros_like(dev(sc))
    ac.acache_write_slots_q8(_desc(hq, hkv, d, dtype), 1, T, dev(rs[:1]), nk[None], nv[None], gk2, gv2, s2, ns, 0)
    at = rs[0].long()
    assert np.array_equal(values(gk2.cpu()[at].numpy(), s2.cpu()[at, :, 0].numpy()), kv[at])
    assert np.array_equal(values(gv2.cpu()[at].numpy(), s2.cpu()[at, :, 1].numpy()), vv[at])
    assert all((x[:16] == 9).all() and (x[-16:] == 9).all() for x in (kroom, vroom))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n_q", [1, 40])
def test_offsets_past_32_bits(dtype, n_q):
    """A pool of 5 GB a side: slots on both sides of 2^32 bytes and of 2^31."""
    hq, hkv, d, ns = 8, 8, 128, 5 << 20
    g = torch.Generator().manual_seed(2)
    near = [0, (1 << 21) - 1, 1 << 21, (1 << 22) - 1, 1 << 22, ns - 1]
    slots = torch.tensor(near + list(range((1 << 22) + 7, (1 << 22) + 301)) + list(range(ns - 200, ns - 10)), dtype=torch.int32)
    T = len(slots)
    new = [torch.randn((1, T, hkv, d), generator=g).to(dtype) for _ in range(2)]
    kc, vc = (torch.empty((ns, hkv, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    sc = torch.empty((ns, hkv, 2), dtype=torch.uint8, device="cuda")
    q = (1.5 * torch.randn((1, n_q, hq, d), generator=g)).to(dtype)
    rs, desc, st = dev(slots[None]), _desc(hq, hkv, d, dtype), _status()
    out = torch.empty(q.shape, dtype=dtype, device="cuda")
    ac.acache_store_attend_q8(desc, 1, T, rs, dev(new[0]), dev(new[1]), kc, vc, sc, ns, 0, n_q, dev(q), T, rs, out, dev_status=st)
    vals = []
    for x in new:
        c, e, _ = quantise(x[0])
        vals.append(values(c, e))
    want, tol = attention(q[0], np.arange(T), vals[0], vals[1], d ** -0.5)
    assert_attention(out[0].double().cpu().numpy(), want, tol)
    ko, vo = (torch.empty((1, T, hkv, d), dtype=dtype, device="cuda") for _ in range(2))
    ac.acache_gather_slots_q8(desc, 1, T, rs, kc, vc, sc, ns, ko, vo, dev_status=st)
    assert np.array_equal(ko[0].double().cpu().numpy(), vals[0]) and np.array_equal(vo[0].double().cpu().numpy(), vals[1])
    assert st.item() == 0


# clusters of 8 CTAs, with two row tiles each and with one (split keys); single CTAs.  Each has more key tiles
# (of 128) than its K ring's 3 or 4, so that the ring's producer has to wait.
@pytest.mark.parametrize("B,n_q,hq,hkv,T,d", [(2, 300, 4, 2, 5000, 128), (1, 100, 2, 2, 6000, 64), (4, 600, 16, 4, 700, 128)])
def test_a_wait_that_runs_out_is_flagged_and_leaves_the_context_usable(B, n_q, hq, hkv, T, d):
    """With a budget of a few hundred cycles that wait runs out on a healthy kernel: it flags the timeout and
    exits; the same call then matches."""
    (kc, vc, sc, kv, vv), q, rs, ns = _attend_case(B, n_q, hq, hkv, d, BF16, T, False, 41)
    args = (_desc(hq, hkv, d, BF16), B, n_q, dev(q), T, dev(rs), dev(kc), dev(vc), dev(sc), ns)
    out, st = torch.zeros(q.shape, dtype=BF16, device="cuda"), _status()
    prev = ac.acache_wait_budget(300)
    try:
        ac.acache_slot_attention_q8(*args, out, dev_status=st)
        torch.cuda.synchronize()
    finally:
        ac.acache_wait_budget(prev)
    assert st.item() & _lib.DEV_TIMEOUT, f"device status {st.item()}"
    st.zero_()
    for _ in range(2):
        ac.acache_slot_attention_q8(*args, out, dev_status=st)
    assert st.item() == 0
    want, tol = attention(q[0], rs[0].numpy(), kv, vv, d ** -0.5)
    assert_attention(out[0].double().cpu().numpy(), want, tol)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_an_empty_pool_holds_zero_rows(dtype):
    """num_slots = 0: every entry is a bad slot, or with drop_none and no slot no key at all."""
    hq, hkv, d, T, n_q = 2, 1, 64, 70, 3
    kc = vc = torch.zeros((1, hkv, d), dtype=torch.uint8, device="cuda")
    sc = torch.zeros((1, hkv, 2), dtype=torch.uint8, device="cuda")
    q = torch.randn((1, n_q, hq, d)).to(dtype).cuda()
    rs = torch.zeros((1, T), dtype=torch.int32, device="cuda")
    for fill, drop, flags in ((0, False, _lib.DEV_BAD_SLOT), (-1, True, 0)):
        rs.fill_(fill)
        out, st = torch.full(q.shape, 3.0, dtype=dtype, device="cuda"), _status()
        ac.acache_slot_attention_q8(_desc(hq, hkv, d, dtype), 1, n_q, q, T, rs, kc, vc, sc, 0, out, drop_none=drop, dev_status=st)
        assert (out == 0).all() and st.item() == flags


# ------------------------------------------------------------------------------------- ragged
RAGGED = [
    ("mixed", BF16, 128, 8, 2, [(300, 700), (0, 50), (5, 1), (589, 1408), (128, 129)]),
    ("tokens", BF16, 128, 8, 2, [(1, 2500), (1, 1), (0, 0), (1, 128), (1, 129), (1, 40), (1, 1000)]),
    ("d64", BF16, 64, 4, 4, [(32, 1480), (1, 37), (257, 256)]),
    ("f32", F32, 64, 2, 2, [(40, 200), (0, 0), (7, 33), (1, 1)]),
]


@pytest.mark.parametrize("name,dtype,d,hq,hkv,reqs", RAGGED, ids=[c[0] for c in RAGGED])
@pytest.mark.parametrize("drop", [False, True])
def test_ragged_parity(name, dtype, d, hq, hkv, reqs, drop):
    rows, keys = [r for r, _ in reqs], [k for _, k in reqs]
    g = torch.Generator().manual_seed(len(name))
    ns, B = 3000, len(reqs)
    kc, vc, sc, kv, vv = random_pool(ns, hkv, d, g)
    tail = 11                                                   # rows behind the last sequence
    q = (1.5 * torch.randn((sum(rows) + tail, hq, d), generator=g)).to(dtype)
    rs = torch.randint(0, ns, (sum(keys),), generator=g, dtype=torch.int32)
    if drop:
        rs[torch.rand(rs.shape, generator=g) < 0.4] = -1
    qs = torch.tensor([0] + list(np.cumsum(rows)), dtype=torch.int32)
    ks = torch.tensor([0] + list(np.cumsum(keys)), dtype=torch.int32)
    out, st = torch.full(q.shape, 9.0, dtype=dtype, device="cuda"), _status()
    ac.acache_slot_attention_varlen_q8(_desc(hq, hkv, d, dtype), B, dev(qs), max(rows), sum(rows), dev(q), dev(ks), max(keys),
                                       dev(rs), dev(kc), dev(vc), dev(sc), ns, out, drop_none=drop, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    got = out.double().cpu().numpy()
    assert (got[sum(rows):] == 9).all()
    for b in range(B):
        a, z = int(qs[b]), int(qs[b + 1])
        want, tol = attention(q[a:z], rs[int(ks[b]):int(ks[b + 1])].numpy(), kv, vv, d ** -0.5, drop)
        assert_attention(got[a:z], want, tol, f"request {b}")


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 64)])
def test_ragged_bad_lengths_are_skipped_and_flagged(dtype, d):
    rows, keys = [40, 50, 30, 10], [300, 300, 0, 301]           # requests 1 to 3: too many rows, no key, too many keys
    g = torch.Generator().manual_seed(3)
    kc, vc, sc, kv, vv = random_pool(500, 2, d, g)
    q = torch.randn((sum(rows), 2, d), generator=g).to(dtype)
    rs = torch.randint(0, 500, (sum(keys),), generator=g, dtype=torch.int32)
    qs = torch.tensor([0] + list(np.cumsum(rows)), dtype=torch.int32)
    ks = torch.tensor([0] + list(np.cumsum(keys)), dtype=torch.int32)
    out, st = torch.full(q.shape, 9.0, dtype=dtype, device="cuda"), _status()
    ac.acache_slot_attention_varlen_q8(_desc(2, 2, d, dtype), 4, dev(qs), 45, sum(rows), dev(q), dev(ks), 300, dev(rs), dev(kc),
                                       dev(vc), dev(sc), 500, out, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == _lib.DEV_BAD_LENGTH
    got = out.double().cpu().numpy()
    assert (got[40:] == 9).all()
    want, tol = attention(q[:40], rs[:300].numpy(), kv, vv, d ** -0.5)
    assert_attention(got[:40], want, tol)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("max_q", [20, 60])
def test_ragged_rows_outside_q_are_skipped_and_flagged(dtype, d, max_q):
    """Only the first total_q_rows rows of q and out are the call's."""
    rows, total = [15, 4, 11], 25                               # the last request's rows reach past them
    g = torch.Generator().manual_seed(6)
    kc, vc, sc, kv, vv = random_pool(200, 1, d, g)
    q = torch.randn((sum(rows), 2, d), generator=g).to(dtype)
    rs = torch.randint(0, 200, (3 * 100,), generator=g, dtype=torch.int32)
    qs = torch.tensor([0] + list(np.cumsum(rows)), dtype=torch.int32)
    ks = torch.tensor([0, 100, 200, 300], dtype=torch.int32)
    out, st = torch.full(q.shape, 9.0, dtype=dtype, device="cuda"), _status()
    ac.acache_slot_attention_varlen_q8(_desc(2, 1, d, dtype), 3, dev(qs), max_q, total, dev(q), dev(ks), 100, dev(rs), dev(kc),
                                       dev(vc), dev(sc), 200, out, dev_status=st)
    got = out.double().cpu().numpy()
    assert st.item() == _lib.DEV_BAD_LENGTH and (got[19:] == 9).all()
    for b in range(2):
        at = slice(int(qs[b]), int(qs[b + 1]))
        want, tol = attention(q[at], rs[100 * b:100 * b + 100].numpy(), kv, vv, d ** -0.5)
        assert_attention(got[at], want, tol)


# ------------------------------------------------------------------------------- store and attend
def _step(B, rows, n_q, hq, hkv, d, dtype, T, seed):
    g = torch.Generator().manual_seed(seed)
    priv0 = T
    ns = priv0 + B * rows + 9
    kc, vc, sc, _, _ = random_pool(ns, hkv, d, g)
    ws = (priv0 + torch.randperm(ns - priv0, generator=g)[:B * rows]).to(torch.int32).view(B, rows)
    rs = torch.stack([torch.randperm(priv0, generator=g)[:T] for _ in range(B)]).to(torch.int32)
    for b in range(B):
        at = torch.randperm(T, generator=g)[:min(rows, T)]
        rs[b, at] = ws[b, :len(at)]
    kn, vn = (torch.randn((B, rows, hkv, d), generator=g).to(dtype) for _ in range(2))
    q = torch.randn((B, n_q, hq, d), generator=g).to(dtype)
    return kc, vc, sc, ns, priv0, ws, rs, kn, vn, q


@pytest.mark.parametrize("B,rows,n_q,hq,hkv,d,dtype,T", [
    (2, 300, 300, 4, 4, 128, BF16, 700), (3, 32, 32, 8, 4, 128, BF16, 600), (2, 1, 1, 8, 2, 128, BF16, 1500),
    (2, 33, 40, 4, 2, 64, BF16, 300), (2, 40, 40, 2, 2, 64, F32, 150)])
def test_store_attend_is_the_store_and_the_attention(B, rows, n_q, hq, hkv, d, dtype, T):
    kc, vc, sc, ns, priv0, ws, rs, kn, vn, q = _step(B, rows, n_q, hq, hkv, d, dtype, T, rows + T)
    desc, st = _desc(hq, hkv, d, dtype), _status()
    outs, pools = [], []
    for one_call in (True, False):
        pool = [dev(x) for x in (kc, vc, sc)]
        out = torch.empty(q.shape, dtype=dtype, device="cuda")
        if one_call:
            ac.acache_store_attend_q8(desc, B, rows, dev(ws), dev(kn), dev(vn), *pool, ns, priv0, n_q, dev(q), T, dev(rs), out,
                                      dev_status=st)
        else:
            ac.acache_write_slots_q8(desc, B, rows, dev(ws), dev(kn), dev(vn), *pool, ns, priv0, dev_status=st)
            ac.acache_slot_attention_q8(desc, B, n_q, dev(q), T, dev(rs), *pool, ns, out, dev_status=st)
        torch.cuda.synchronize()
        outs.append(out)
        pools.append(pool)
    assert st.item() == 0 and torch.equal(*outs)
    assert all(torch.equal(a, b) for a, b in zip(*pools))
    k, v, s = [x.cpu().numpy() for x in pools[0]]
    for b in range(B):
        want, tol = attention(q[b], rs[b].numpy(), values(k, s[..., 0]), values(v, s[..., 1]), d ** -0.5)
        assert_attention(outs[0][b].double().cpu().numpy(), want, tol)


def test_store_only_and_attend_only():
    kc, vc, sc, ns, priv0, ws, rs, kn, vn, q = _step(1, 5, 6, 4, 2, 128, BF16, 130, 1)
    desc, pool = _desc(4, 2, 128, BF16), [dev(x) for x in (kc, vc, sc)]
    ac.acache_store_attend_q8(desc, 1, 5, dev(ws), dev(kn), dev(vn), *pool, ns, priv0, 0, None, 0, None, None)
    codes, scale, _ = quantise(kn[0])
    at = ws[0].numpy()
    assert np.array_equal(pool[0].cpu().numpy()[at], codes) and np.array_equal(pool[2].cpu().numpy()[at, :, 0], scale)
    out = torch.empty(q.shape, dtype=BF16, device="cuda")
    ac.acache_store_attend_q8(desc, 1, 0, None, None, None, *pool, ns, priv0, 6, dev(q), 130, dev(rs), out)
    k, v, s = [x.cpu().numpy() for x in pool]
    want, tol = attention(q[0], rs[0].numpy(), values(k, s[..., 0]), values(v, s[..., 1]), 128 ** -0.5)
    assert_attention(out[0].double().cpu().numpy(), want, tol)


@pytest.mark.parametrize("n_q,dtype,d", [(1, BF16, 128), (300, BF16, 128), (33, F32, 64)])
def test_captured_steps_replay_on_new_inputs(n_q, dtype, d):
    """Two steps in one graph on a side stream; a replay reads what the buffers hold then."""
    args = [_step(2, min(n_q, 40), n_q, 4, 2, d, dtype, 500, seed) for seed in (1, 2)]
    desc = _desc(4, 2, d, dtype)
    dead = [[dev(x) if torch.is_tensor(x) else x for x in a] for a in args]
    outs = [torch.empty(a[9].shape, dtype=dtype, device="cuda") for a in args]

    def step(i):
        kc, vc, sc, ns, priv0, ws, rs, kn, vn, q = dead[i]
        ac.acache_store_attend_q8(desc, 2, ws.shape[1], ws, kn, vn, kc, vc, sc, ns, priv0, n_q, q, 500, rs, outs[i])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(0), step(1)                                        # first launches outside the capture
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(0), step(1)
    new = _step(2, min(n_q, 40), n_q, 4, 2, d, dtype, 500, 9)
    for i in (0, 1):
        dead[i][9].copy_(new[9])
        dead[i][7].copy_(new[7])
        outs[i].zero_()
    graph.replay()
    torch.cuda.synchronize()
    for i in (0, 1):
        k, v, s = [x.cpu().numpy() for x in dead[i][:3]]
        at = dead[i][5].cpu().view(-1).numpy()
        codes, _, _ = quantise(new[7].view((-1,) + new[7].shape[2:]))
        assert np.array_equal(k[at], codes)
        for b in range(2):
            want, tol = attention(new[9][b], args[i][6][b].numpy(), values(k, s[..., 0]), values(v, s[..., 1]), d ** -0.5)
            assert_attention(outs[i][b].double().cpu().numpy(), want, tol)


def test_two_streams_at_once():
    desc = _desc(8, 4, 128, BF16)
    args = [_step(2, 40, 200, 8, 4, 128, BF16, 900, seed) for seed in (5, 6)]
    gpu = [[dev(x) if torch.is_tensor(x) else x for x in a] for a in args]
    outs = [torch.empty(a[9].shape, dtype=BF16, device="cuda") for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in gpu]
    for _ in range(3):
        for (kc, vc, sc, ns, priv0, ws, rs, kn, vn, q), o, s in zip(gpu, outs, streams):
            ac.acache_store_attend_q8(desc, 2, 40, ws, kn, vn, kc, vc, sc, ns, priv0, 200, q, 900, rs, o, stream=s)
    torch.cuda.synchronize()
    for a, g, o in zip(args, gpu, outs):
        k, v, s = [x.cpu().numpy() for x in g[:3]]
        want, tol = attention(a[9][1], a[6][1].numpy(), values(k, s[..., 0]), values(v, s[..., 1]), 128 ** -0.5)
        assert_attention(o[1].double().cpu().numpy(), want, tol)


def test_the_whole_path_over_an_8_bit_pool():
    """A shared affix stored in 8 bits and read back for the probe, anchors, maps, a recompute point
    and a decode block over the pool."""
    import oracle
    from affix_kv_cache_gb300 import workloads as wl
    w = wl.Workload(name="q8_path", dtype="bf16", layers=1, hq=4, hkv=2, d=128, batch=2,
                    segments=((wl.SEG_AFFIX, 300), (wl.SEG_REQ, 60), (wl.SEG_MASK, 70)), ratio_permille=200,
                    recompute_points=1, plant="aligned", plant_count=15, plant_scale=1.5, page=64)
    lay, inp, rec = wl.slot_layout(w), wl.probe_inputs(w, 0), wl.recompute_inputs(w, 0)
    desc, st = _desc(w.hq, w.hkv, w.d, BF16), _status()
    pool = [torch.zeros((lay.num_slots, w.hkv, x), dtype=torch.uint8, device="cuda") for x in (w.d, w.d, 2)]
    ac.acache_write_slots_q8(desc, 1, w.L, dev(lay.shared_slot), dev(inp["k_aff"]), dev(inp["v_aff"]), *pool, lay.num_slots, 0,
                             dev_status=st)
    ka, va = (torch.empty_like(inp["k_aff"], device="cuda") for _ in range(2))
    ac.acache_gather_slots_q8(desc, 1, w.L, dev(lay.shared_slot), *pool, lay.num_slots, ka, va, dev_status=st)
    masked = torch.tensor(w.masked_rows(), dtype=torch.int32).expand(w.batch, -1).contiguous()
    scores = torch.zeros((w.batch, w.L), device="cuda")
    space = torch.empty(ac.acache_probe_workspace_bytes(desc, w.batch, w.T, w.L, w.m), dtype=torch.uint8, device="cuda")
    ac.acache_probe_scores(desc, w.batch, w.T, w.l, w.L, dev(masked), w.m, dev(inp["q"]), dev(inp["k_req"]), dev(inp["v_req"]),
                           ka, va, None, scores, space, dev_status=st)
    ref = oracle.probe_layer(inp["q"], inp["k_req"], inp["v_req"], ka.cpu(), va.cpu(), T=w.T, l=w.l,
                             masked_rows=w.masked_rows(), scale=w.scale, want_out=False)["scores"]
    assert np.abs(scores.cpu().numpy() / ref - 1).max() < 1e-3
    anchors = torch.empty((w.batch, w.K), dtype=torch.int32, device="cuda")
    ac.acache_topk_anchors(scores, w.batch, w.L, w.K, anchors, dev_status=st)
    wp = torch.empty((w.batch, w.R), dtype=torch.int32, device="cuda")
    rs = torch.empty((w.batch, w.T), dtype=torch.int32, device="cuda")
    priv = dev(lay.private_slots)
    ac.acache_build_slot_maps(w.batch, w.T, w.l, w.L, w.K, anchors, dev(lay.shared_slot), priv, wp, rs, dev_status=st)
    out = torch.empty(rec["q_r"].shape, dtype=BF16, device="cuda")
    ac.acache_store_attend_q8(desc, w.batch, w.R, priv, dev(rec["k_new"]), dev(rec["v_new"]), *pool, lay.num_slots,
                              lay.private_begin, w.R, dev(rec["q_r"]), w.T, rs, out, dev_status=st)
    dec = wl.decode_inputs(w, 0)
    n = dec["q_blk"].shape[1]
    pos = {int(p): i for i, p in enumerate(wp[0].tolist())}
    at = torch.tensor([pos[p] for p in wl.decode_block_positions(w, 0)])
    blk = dev(lay.private_slots[:, at])
    dout = torch.empty(dec["q_blk"].shape, dtype=BF16, device="cuda")
    kept = [x.clone() for x in pool]
    ac.acache_store_attend_q8(desc, w.batch, n, blk, dev(dec["k_blk"]), dev(dec["v_blk"]), *pool, lay.num_slots,
                              lay.private_begin, n, dev(dec["q_blk"]), w.T, rs, dout, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for q, o, p in ((rec["q_r"], out, kept), (dec["q_blk"], dout, pool)):
        k, v, s = [x.cpu().numpy() for x in p]
        for b in range(w.batch):
            want, tol = attention(q[b], rs[b].cpu().numpy(), values(k, s[..., 0]), values(v, s[..., 1]), w.scale)
            assert_attention(o[b].double().cpu().numpy(), want, tol, f"request {b}")


def test_a_tensor_off_the_current_device_is_refused():
    args = _step(1, 5, 6, 4, 2, 128, BF16, 130, 1)
    kc, vc, sc, ns, priv0, ws, rs, kn, vn, q = args
    out = torch.empty(q.shape, dtype=BF16, device="cuda")
    with pytest.raises(ValueError, match="current device"):
        ac.acache_slot_attention_q8(_desc(4, 2, 128, BF16), 1, 6, dev(q), 130, dev(rs), kc, vc, sc, ns, out)


@pytest.mark.parametrize("dtype,scale", [(F32, None), (BF16, -0.125)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_q", [1, 3, 5, 17, 33])
def test_merges_whose_lanes_take_different_numbers_of_turns(dtype, scale, d, n_q):
    """CUDA-core kernel, keys split over a cluster, an odd number of rows: in the merge some lanes of a
    warp finalise one item more than the others before the whole warp reaches the cluster's barrier."""
    hq, hkv, T = 1, 1, 1100
    scale = d ** -0.5 if scale is None else scale
    (kc, vc, sc, kv, vv), q, rs, ns = _attend_case(2, n_q, hq, hkv, d, dtype, T, False, 3 * n_q + d)
    args = (_desc(hq, hkv, d, dtype, scale), 2, n_q, dev(q), T, dev(rs), dev(kc), dev(vc), dev(sc), ns)
    outs = [torch.empty(q.shape, dtype=dtype, device="cuda") for _ in range(3)]
    for o in outs:
        ac.acache_slot_attention_q8(*args, o)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    for b in range(2):
        want, tol = attention(q[b], rs[b].numpy(), kv, vv, scale)
        assert_attention(outs[0][b].double().cpu().numpy(), want, tol, f"request {b}")


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("n_q", [1, 32, 40, 300])
@pytest.mark.parametrize("size", [1.0, 1e-4, 1e-6, 1e-12])
def test_bad_slots_beside_small_values(dtype, d, n_q, size):
    """A zero row has no size: however small the other rows' values are, it takes only its share of the
    softmax."""
    hq, hkv, T, ns = 2, 1, 70, 200
    g = torch.Generator().manual_seed(23)
    x = [torch.randn((ns, hkv, d), generator=g) * f for f in (1.0, size)]
    (kc, ks, _), (vc, vs, _) = quantise(x[0]), quantise(x[1])
    kv, vv = values(kc, ks), values(vc, vs)
    sc = torch.from_numpy(np.stack((ks, vs), -1)).contiguous()
    q = (1.5 * torch.randn((1, n_q, hq, d), generator=g)).to(dtype)
    rs = torch.randperm(ns, generator=g)[None, :T].to(torch.int32)
    rs[0, [0, 17, 40, T - 1]] = torch.tensor([-1, ns, -9, 2 ** 31 - 1], dtype=torch.int32)
    out, st = torch.empty(q.shape, dtype=dtype, device="cuda"), _status()
    ac.acache_slot_attention_q8(_desc(hq, hkv, d, dtype), 1, n_q, dev(q), T, dev(rs), dev(torch.from_numpy(kc)),
                                dev(torch.from_numpy(vc)), dev(sc), ns, out, dev_status=st)
    want, tol = attention(q[0], rs[0].numpy(), kv, vv, d ** -0.5)
    assert_attention(out[0].double().cpu().numpy(), want, tol)
    assert st.item() == _lib.DEV_BAD_SLOT


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("n_q", [1, 32, 40, 300])
@pytest.mark.parametrize("drop", [False, True])
@pytest.mark.parametrize("slot", [-2 ** 31, -2 ** 31 + 1, -2, 2 ** 31 - 1])
def test_every_value_outside_the_pool_is_a_flagged_zero_row(dtype, d, n_q, drop, slot):
    """Nine keys, so that one key too few in a softmax shows; also the last of them, next to the keys that
    are past the end."""
    hq, hkv, T = 2, 1, 9
    (kc, vc, sc, kv, vv), q, rs, ns = _attend_case(2, n_q, hq, hkv, d, dtype, T, False, 19)
    rs[0, 3], rs[0, 8], rs[1, 0] = slot, slot, slot
    if drop:
        rs[0, 5] = -1
    desc, pool = _desc(hq, hkv, d, dtype), (dev(kc), dev(vc), dev(sc), ns)
    starts = [torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda") for n in (n_q, T)]
    for ragged in (False, True):
        out, st = torch.empty(q.shape, dtype=dtype, device="cuda"), _status()
        if ragged:
            ac.acache_slot_attention_varlen_q8(desc, 2, starts[0], n_q, 2 * n_q, dev(q), starts[1], T, dev(rs), *pool, out,
                                               drop_none=drop, dev_status=st)
        else:
            ac.acache_slot_attention_q8(desc, 2, n_q, dev(q), T, dev(rs), *pool, out, drop_none=drop, dev_status=st)
        for b in range(2):
            want, tol = attention(q[b], rs[b].numpy(), kv, vv, d ** -0.5, drop)
            assert_attention(out[b].double().cpu().numpy(), want, tol, f"request {b}")
        assert st.item() == _lib.DEV_BAD_SLOT


# single CTAs of two row tiles and of one (split keys); clusters of both
@pytest.mark.parametrize("B,n_q,hq,hkv,T,d", [(4, 600, 16, 4, 700, 128), (8, 100, 32, 32, 900, 128), (2, 300, 4, 2, 5000, 128),
                                              (1, 100, 2, 2, 6000, 64)])
def test_no_unfinished_row_is_written_after_a_timeout(B, n_q, hq, hkv, T, d):
    """Waits that run out at any stage of the kernel: a row of the output is right, or it is as it was."""
    (kc, vc, sc, kv, vv), q, rs, ns = _attend_case(B, n_q, hq, hkv, d, BF16, T, False, 43)
    args = (_desc(hq, hkv, d, BF16), B, n_q, dev(q), T, dev(rs), dev(kc), dev(vc), dev(sc), ns)
    both = [attention(q[b], rs[b].numpy(), kv, vv, d ** -0.5) for b in range(B)]
    want, tol = (torch.from_numpy(np.stack([x[i] for x in both])).cuda() for i in (0, 1))
    out, st = torch.empty(q.shape, dtype=BF16, device="cuda"), _status()
    seen = 0
    for budget in [300] * 8 + list(range(1000, 40000, 1500)):
        out.fill_(9.0)
        st.zero_()
        prev = ac.acache_wait_budget(budget)
        try:
            ac.acache_slot_attention_q8(*args, out, dev_status=st)
            torch.cuda.synchronize()
        finally:
            ac.acache_wait_budget(prev)
        got = out.double()
        left = (got == 9).all(-1)
        right = ((got - want).abs() <= tol).all(-1)
        assert (left | right).all(), f"budget {budget}: {(~(left | right)).sum().item()} rows"
        assert st.item() in (0, _lib.DEV_TIMEOUT) and (st.item() or right.all())
        seen += st.item() != 0
    assert seen


@pytest.mark.parametrize("call,name", TENSORS)
def test_a_host_tensor_beside_device_tensors_is_refused(call, name):
    """Raised before the library is called: nothing is launched."""
    host, there = torch.zeros(64), torch.zeros(64, device="cuda")
    args = [host if a == name else there if isinstance(a, str) else a for a in CALLS[call]]
    with pytest.raises(ValueError, match="current device"):
        getattr(ac, call)(_desc(4, 2, 128, BF16), *args, dev_status=host if name == "dev_status" else there)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("max_q", [1, 60])
def test_ragged_counts_that_wrap_32_bits_are_skipped_and_flagged(dtype, d, max_q):
    """Offsets whose difference is -(2^32 - 1): cut to 32 bits that is a count of one."""
    g = torch.Generator().manual_seed(8)
    kc, vc, sc, kv, vv = random_pool(50, 1, d, g)
    q = torch.randn((3, 2, d), generator=g).to(dtype)
    rs = torch.randint(0, 50, (40,), generator=g, dtype=torch.int32)
    top, low = 2 ** 31 - 1, -2 ** 31
    for qs, ks, right in (((0, 1, 2), (0, 40, low), 1), ((0, 1, 2), (top, low, 3), 0), ((top, low, 2), (0, 40, 40), 0)):
        out, st = torch.full(q.shape, 9.0, dtype=dtype, device="cuda"), _status()
        qs, ks = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (qs, ks))
        ac.acache_slot_attention_varlen_q8(_desc(2, 1, d, dtype), 2, qs, max_q, 3, dev(q), ks, 40, dev(rs), dev(kc), dev(vc), dev(sc),
                                           50, out, dev_status=st)
        got = out.double().cpu().numpy()
        assert st.item() == _lib.DEV_BAD_LENGTH and (got[right:] == 9).all()
        if right:
            want, tol = attention(q[:1], rs.numpy(), kv, vv, d ** -0.5)
            assert_attention(got[:1], want, tol)


def _counted_keys(T, hkv, d, g):
    """A pool of T slots whose attention outputs are counts: head h's key t has logit 0 or, for a random half,
    one that no weight is left of; and a value row that is zero but for one element of one head."""
    t = torch.arange(T)
    alive = torch.rand(T, generator=g) < 0.5
    alive[torch.tensor([0, T - 1])] = True
    k, v = torch.zeros((T, hkv, d)), torch.zeros((T, hkv, d))
    k[:, :, 0] = torch.where(alive, 0.0, -64.0)[:, None]
    v[t, t % hkv, t // hkv % d] = 1.0
    return k, v, alive


@pytest.mark.parametrize("dtype,hkv,d", [(BF16, 8, 128), (BF16, 16, 64), (F32, 8, 128)])
@pytest.mark.parametrize("n_q", [1, 9, 32, 40, 300])
@pytest.mark.parametrize("T", [4097, 9000])
@pytest.mark.parametrize("ragged", [False, True])
def test_every_key_of_a_long_context_counts_once(dtype, hkv, d, n_q, T, ragged):
    """Weights are 1 or 0, so an output element is a number of keys over the number of all: one key lost or
    read twice, anywhere, changes it by far more than its rounding."""
    g = torch.Generator().manual_seed(T + n_q)
    k, v, alive = _counted_keys(T, hkv, d, g)
    n, count = int(alive.sum()), v[alive].sum(0).double().numpy()         # [hkv][d]
    want = count / n
    rel = {BF16: 2.0 ** -8, F32: 2.0 ** -20}[dtype] + 2.0 ** -20          # the output's rounding; exp2, sum and 1/sum
    for other in ((count - 1) / (n - 1), (count + 1) / (n + 1)):
        changed = np.abs(other - want)[count > 0]
        assert (changed > 2.5 * rel * want[count > 0]).all()
    slots = torch.randperm(T, generator=g)
    slots[: T // 2] = torch.sort(slots[: T // 2]).values                  # (runs of neighbours as well)
    kc, vc = (torch.empty((T, hkv, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    sc = torch.empty((T, hkv, 2), dtype=torch.uint8, device="cuda")
    desc, rs = _desc(hkv, hkv, d, dtype, 1.0), slots.to(torch.int32).cuda()[None]
    ac.acache_write_slots_q8(desc, 1, T, rs, dev(k.to(dtype))[None], dev(v.to(dtype))[None], kc, vc, sc, T, 0)
    q = torch.zeros((1, n_q, hkv, d), dtype=dtype, device="cuda")
    q[..., 0] = 8.0
    out, st = torch.empty_like(q), _status()
    if ragged:                              # behind a request of one key and before an idle one
        qs, ks = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ((0, 1, n_q + 1, n_q + 1), (0, 1, T + 1, T + 1)))
        q, rs = torch.cat((q[0, :1], q[0])), torch.cat((rs[0, :1], rs[0]))
        o = torch.empty_like(q)
        ac.acache_slot_attention_varlen_q8(desc, 3, qs, n_q, n_q + 1, q, ks, T, rs, kc, vc, sc, T, o, dev_status=st)
        out = o[1:][None]
    else:
        ac.acache_slot_attention_q8(desc, 1, n_q, q, T, rs, kc, vc, sc, T, out, dev_status=st)
    got = out[0].double().cpu().numpy()
    assert st.item() == 0
    assert (np.abs(got - want) <= rel * want).all(), np.abs(got / np.maximum(want, 1e-30) - (want > 0)).max()


@pytest.mark.parametrize("B,rows,n_q,hq,hkv,d,dtype,T", [
    (2, 300, 300, 4, 4, 128, BF16, 700), (3, 32, 32, 8, 4, 128, BF16, 600), (2, 1, 1, 8, 2, 128, BF16, 1500),
    (2, 33, 40, 4, 2, 64, BF16, 300), (2, 40, 40, 2, 2, 64, F32, 150)])
def test_store_attend_with_discarded_keys(B, rows, n_q, hq, hkv, d, dtype, T):
    kc, vc, sc, ns, priv0, ws, rs, kn, vn, q = _step(B, rows, n_q, hq, hkv, d, dtype, T, rows + 2 * T)
    rs[(torch.rand(rs.shape, generator=torch.Generator().manual_seed(T)) < 0.4) & (rs < priv0)] = -1
    rs[1] = -1                                                  # stored, and nothing to attend to
    pool, st = [dev(x) for x in (kc, vc, sc)], _status()
    out = torch.full(q.shape, 9.0, dtype=dtype, device="cuda")
    ac.acache_store_attend_q8(_desc(hq, hkv, d, dtype), B, rows, dev(ws), dev(kn), dev(vn), *pool, ns, priv0, n_q, dev(q), T,
                              dev(rs), out, drop_none=True, dev_status=st)
    k, v, s = [x.cpu().numpy() for x in pool]
    at = ws.view(-1).numpy()
    for i, (c, x) in enumerate(((k, kn), (v, vn))):
        codes, scale, _ = quantise(x.view((-1,) + x.shape[2:]))
        assert np.array_equal(c[at], codes) and np.array_equal(s[at, :, i], scale)
    for b in range(B):
        want, tol = attention(q[b], rs[b].numpy(), values(k, s[..., 0]), values(v, s[..., 1]), d ** -0.5, True)
        assert_attention(out[b].double().cpu().numpy(), want, tol, f"request {b}")
    assert (out[1] == 0).all() and st.item() == 0


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 128), (F32, 64)])
@pytest.mark.parametrize("n_q", [1, 20, 40, 300])
def test_logits_of_minus_infinity(dtype, d, n_q):
    """A row whose every logit is -infinity has no softmax: NaN, not the zeros of a row without keys.  Beside one
    finite logit, wherever it is, they weigh nothing."""
    hq, hkv, T = 2, 1, 2000
    (kc, vc, sc, kv, vv), q, rs, ns = _attend_case(2, n_q, hq, hkv, d, dtype, T, False, 33)
    kc[:, :, 0], sc[..., 0] = 0x60, 127                         # element 0 of every key: 2^5
    free = ns - 1
    kc[free] = 0
    rs[rs == free] = 0
    desc, pool = _desc(hq, hkv, d, dtype, 1.0), (dev(kc), dev(vc), dev(sc), ns)

    def run(q, rs, drop=True):
        out = torch.full(q.shape, 9.0, dtype=dtype, device="cuda")
        ac.acache_slot_attention_q8(desc, 2, n_q, dev(q), T, dev(rs), *pool, out, drop_none=drop)
        return out.double().cpu().numpy()

    q[..., 0] = -float("inf")
    one = torch.full_like(rs, -1)
    one[:, 900] = rs[:, 900]
    for r in (rs, one):
        assert np.isnan(run(q, r)).all()
    assert np.isnan(run(q, rs, drop=False)).all()
    if dtype == F32:
        assert (run(q, torch.full_like(rs, -1)) == 0).all()
        # products that overflow to -infinity
        q[..., 0] = -3e38
        for at in (0, 700, T - 1):
            r = rs.clone()
            r[:, at] = free
            got, want = run(q, r), vv[free, 0]
            assert np.abs(got - want).max() <= 2.0 ** -20 * np.abs(want).max()


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("n_q", [1, 12, 40, 300])
def test_non_finite_queries_without_a_key_give_zeros(dtype, d, n_q):
    """The rows of a padded request may hold anything; a query row with a key is NaN if it is not finite, however
    many parts of the keys hold none."""
    B, hq, hkv, T = 4, 2, 1, 2000
    (kc, vc, sc, kv, vv), q, rs, ns = _attend_case(B, n_q, hq, hkv, d, dtype, T, False, 27)
    q[:, -1, 0, 3], q[:, 0, 1, 0] = float("nan"), -float("inf")
    rs[0], rs[1:3] = -1, -1
    rs[1, 700], rs[2, T - 1] = 5, 6
    out, st = torch.full(q.shape, 9.0, dtype=dtype, device="cuda"), _status()
    ac.acache_slot_attention_q8(_desc(hq, hkv, d, dtype), B, n_q, dev(q), T, dev(rs), dev(kc), dev(vc), dev(sc), ns, out,
                                drop_none=True, dev_status=st)
    got = out.double().cpu().numpy()
    assert st.item() == 0 and (got[0] == 0).all()
    gone = ~torch.isfinite(q).all(-1).numpy()
    assert gone.any() and np.isnan(got[1:][gone[1:]]).all()
    q[~torch.isfinite(q)] = 0.0
    for b in range(1, B):
        want, tol = attention(q[b], rs[b].numpy(), kv, vv, d ** -0.5, True)
        assert_attention(got[b][~gone[b]], want[~gone[b]], tol[~gone[b]], f"request {b}")

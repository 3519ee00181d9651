"""GPU parity of the steps around the attention: norm and rotation, the stores that apply them, attention
under a mask (fixed and ragged), token scores, and a run of them together, against 64-bit references."""
import numpy as np
import pytest
import torch

import affix_kv_cache_gb300 as ac
from affix_kv_cache_gb300 import _lib

from gpu_helpers import dev
from q8_reference import HALF, assert_attention, values
from step_reference import frequencies, masked_attention, rotate, token_scores

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _desc(hq, hkv, d, dtype, scale=None):
    return ac.attn_desc(hq, hkv, d, d ** -0.5 if scale is None else scale, dtype)


def _np(t):
    return t.detach().double().cpu().numpy()


def _close(got, want, tol, what=""):
    got = np.asarray(got, np.float64)
    assert got.shape == want.shape
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN pattern differs"
    with np.errstate(invalid="ignore"):
        over = np.where(np.isnan(want) | (got == want), 0.0, np.abs(got - want) - tol)
    assert not (over > 0).any(), f"{what}: {np.sum(over > 0)} elements, worst {over.max():.3e} over its bound"


# ------------------------------------------------------------------------------------- norm and rotation
ROPES = [(128, 128, False), (128, 128, True), (128, 64, False), (128, 36, False), (128, 2, False), (128, 100, True),
         (64, 64, False), (64, 64, True), (64, 32, False), (64, 20, False), (64, 6, True)]


def _rope(rd, inter, kind="none"):
    args = {"none": dict(theta=1e4), "yarn": dict(theta=5e5, scaling="yarn", factor=16.0, trained_len=8192),
            "bands": dict(theta=5e5, scaling="bands", factor=8.0, trained_len=8192)}[kind]
    f, amp = frequencies(rd, args["theta"], args.get("scaling", "none"), args.get("factor", 1.0), args.get("trained_len", 0))
    return ac.rope_desc(rd, interleaved=inter, **args), f, amp


def _new(n, hq, hkv, d, dtype, g, fused):
    """q, k, v [n, heads, d] (CPU) and the same on the GPU, slices of one buffer when fused."""
    x = (torch.randn((n, hq + 2 * hkv, d), generator=g) * torch.exp(torch.randn((n, hq + 2 * hkv, 1), generator=g))).to(dtype)
    parts = x.split((hq, hkv, hkv), 1)
    on = dev(x).split((hq, hkv, hkv), 1) if fused else [dev(p) for p in parts]
    return parts, on


def _check_rows(got, x, w, pos, f, amp, inter, dtype, what):
    want, tol = rotate(x, w, 1e-6, pos, f, amp, inter)
    _close(_np(got), want, tol + HALF[dtype] * (np.abs(want) + tol) * 1.001, what)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,rd,inter", ROPES)
@pytest.mark.parametrize("n,hq,hkv,norm,fused,kind", [(1, 4, 2, True, True, "none"), (37, 7, 1, True, False, "yarn"),
                                                      (5, 3, 3, False, True, "bands")])
def test_rotation(dtype, d, rd, inter, n, hq, hkv, norm, fused, kind):
    g = torch.Generator().manual_seed(d + rd + n)
    (q, k, _), (gq, gk, _) = _new(n, hq, hkv, d, dtype, g, fused)
    rope, f, amp = _rope(rd, inter, kind)
    pos = torch.randint(-1000, 1000000, (n,), generator=g, dtype=torch.int32)
    pos[0] = 2 ** 31 - 1 if norm else -2 ** 31
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(dtype) if norm else None for _ in range(2)]
    gw = [None if x is None else dev(x) for x in w]
    qo, ko = (torch.full((n + 1, h, d), 7.0, dtype=dtype, device="cuda") for h in (hq, hkv))
    ac.acache_rotate_qk(_desc(hq, hkv, d, dtype), rope, n, dev(pos), gq, gk, qo[:n], ko[:n], q_weight=gw[0], k_weight=gw[1])
    torch.cuda.synchronize()
    _check_rows(qo[:n], q, w[0], pos.numpy(), f, amp, inter, dtype, "queries")
    _check_rows(ko[:n], k, w[1], pos.numpy(), f, amp, inter, dtype, "keys")
    assert (qo[n] == 7).all() and (ko[n] == 7).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rd,inter", [(128, False), (36, False), (128, True)])
def test_rotation_in_place_in_a_fused_row_leaves_the_values(dtype, rd, inter):
    g = torch.Generator().manual_seed(5)
    n, hq, hkv, d = 300, 8, 2, 128
    (q, k, v), (gq, gk, gv) = _new(n, hq, hkv, d, dtype, g, True)
    rope, f, amp = _rope(rd, inter)
    pos = torch.arange(n, dtype=torch.int32) * 37
    ac.acache_rotate_qk(_desc(hq, hkv, d, dtype), rope, n, dev(pos), gq, gk, gq, gk)
    torch.cuda.synchronize()
    _check_rows(gq, q, None, pos.numpy(), f, amp, inter, dtype, "queries")
    _check_rows(gk, k, None, pos.numpy(), f, amp, inter, dtype, "keys")
    assert torch.equal(gv.cpu(), v)


def test_rotation_of_one_matrix_and_norm_alone():
    g = torch.Generator().manual_seed(6)
    n, hq, hkv, d = 9, 4, 2, 64
    (q, k, _), (gq, gk, _) = _new(n, hq, hkv, d, BF16, g, False)
    rope, f, amp = _rope(64, False)
    pos, w = torch.arange(n, dtype=torch.int32), (1 + 0.3 * torch.randn(d, generator=g)).to(BF16)
    qo, ko = (torch.full_like(x, 7) for x in (gq, gk))
    desc = _desc(hq, hkv, d, BF16)
    ac.acache_rotate_qk(desc, rope, n, dev(pos), gq, None, qo, None, k_weight=dev(w))
    ac.acache_rotate_qk(desc, None, n, None, None, gk, None, ko, k_weight=dev(w))
    torch.cuda.synchronize()
    _check_rows(qo, q, None, pos.numpy(), f, amp, False, BF16, "queries")
    _check_rows(ko, k, w, pos.numpy(), [], 1.0, False, BF16, "keys")


def test_rotation_keeps_what_is_not_finite_in_its_head():
    g = torch.Generator().manual_seed(7)
    n, hq, hkv, d = 3, 4, 2, 128
    (q, k, _), (gq, gk, _) = _new(n, hq, hkv, d, BF16, g, False)
    gq[1, 2, 5], gk[0, 1, 127] = NAN, INF
    rope, f, amp = _rope(128, False)
    pos, w = torch.arange(n, dtype=torch.int32), torch.ones(d, dtype=BF16)
    qo, ko = torch.empty_like(gq), torch.empty_like(gk)
    ac.acache_rotate_qk(_desc(hq, hkv, d, BF16), rope, n, dev(pos), gq, gk, qo, ko, q_weight=dev(w))
    torch.cuda.synchronize()
    bad = torch.zeros((n, hq), dtype=torch.bool)
    bad[1, 2] = True
    assert torch.equal(qo.isfinite().all(-1).cpu(), ~bad)
    assert torch.equal((~ko.isfinite()).sum((0, 1)).nonzero().flatten().cpu(), torch.tensor([63, 127]))


def test_rotation_of_many_rows():
    """Several rows to a CTA, an odd last one, and heads spread over CTAs when rows are few."""
    g = torch.Generator().manual_seed(8)
    for n, hq, hkv in ((9001, 2, 1), (3, 96, 32), (1217, 28, 4)):
        (q, k, _), (gq, gk, _) = _new(n, hq, hkv, 64, F32, g, True)
        rope, f, amp = _rope(64, False)
        pos = torch.randint(0, 100000, (n,), generator=g, dtype=torch.int32)
        qo, ko = (torch.empty((n, h, 64), device="cuda") for h in (hq, hkv))
        ac.acache_rotate_qk(_desc(hq, hkv, 64, F32), rope, n, dev(pos), gq, gk, qo, ko)
        torch.cuda.synchronize()
        _check_rows(qo, q, None, pos.numpy(), f, amp, False, F32, "queries")
        _check_rows(ko, k, None, pos.numpy(), f, amp, False, F32, "keys")


# ------------------------------------------------------------------------------------- stores
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("hq,hkv,d,rd,inter", [(4, 2, 128, 128, False), (7, 1, 128, 64, True), (3, 3, 64, 20, False), (32, 32, 64, 64, False)])
@pytest.mark.parametrize("B,rows,fused", [(1, 1, True), (3, 37, False), (2, 600, True)])
def test_rotating_store(dtype, hq, hkv, d, rd, inter, B, rows, fused):
    g = torch.Generator().manual_seed(hq + d + rows)
    n, priv0 = B * rows, 20
    ns = n + 60
    (q, k, v), (gq, gk, gv) = _new(n, hq, hkv, d, dtype, g, fused)
    shaped = [x.unflatten(0, (B, rows)) for x in (gq, gk, gv)]
    rope, f, amp = _rope(rd, inter)
    pos = torch.randint(0, 50000, (n,), generator=g, dtype=torch.int32)
    w = (1 + 0.3 * torch.randn(d, generator=g)).to(dtype)
    slots = (priv0 + torch.randperm(ns - priv0, generator=g)[:n]).to(torch.int32)
    kc, vc = (torch.randn((ns, hkv, d), generator=g).to(dtype) for _ in range(2))
    gkc, gvc, st = dev(kc), dev(vc), _status()
    qo = torch.empty((n, hq, d), dtype=dtype, device="cuda")
    ac.acache_rotate_store(_desc(hq, hkv, d, dtype), rope, B, rows, dev(pos), dev(slots), *shaped, qo, gkc, gvc, ns, priv0,
                           k_weight=dev(w), dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    at = slots.long()
    _check_rows(qo, q, None, pos.numpy(), f, amp, inter, dtype, "queries")
    _check_rows(gkc.cpu()[at], k, w, pos.numpy(), f, amp, inter, dtype, "keys")
    vc[at] = v
    kc[at] = gkc.cpu()[at]
    assert torch.equal(gvc.cpu(), vc) and torch.equal(gkc.cpu(), kc)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("hq,hkv,d,rd,inter", [(4, 2, 128, 128, False), (7, 1, 128, 36, False), (3, 3, 64, 64, True)])
@pytest.mark.parametrize("B,rows", [(1, 1), (2, 301)])
def test_rotating_store_8_bit(dtype, hq, hkv, d, rd, inter, B, rows):
    g = torch.Generator().manual_seed(hq + d + rows)
    n, ns = B * rows, B * rows + 13
    (q, k, v), (gq, gk, gv) = _new(n, hq, hkv, d, dtype, g, True)
    rope, f, amp = _rope(rd, inter)
    pos = torch.randint(0, 50000, (n,), generator=g, dtype=torch.int32)
    w = (1 + 0.3 * torch.randn(d, generator=g)).to(dtype)
    slots = torch.randperm(ns, generator=g)[:n].to(torch.int32)
    pool = [torch.full((ns, hkv, x), 5, dtype=torch.uint8, device="cuda") for x in (d, d, 2)]
    qo, st = torch.empty((n, hq, d), dtype=dtype, device="cuda"), _status()
    ac.acache_rotate_store_q8(_desc(hq, hkv, d, dtype), rope, B, rows, dev(pos), dev(slots), gq, gk, gv, qo, *pool, ns, 0,
                              k_weight=dev(w), dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    _check_rows(qo, q, None, pos.numpy(), f, amp, inter, dtype, "queries")
    at = slots.numpy()
    kc, vc, sc = (x.cpu().numpy() for x in pool)
    want, tol = rotate(k, w, 1e-6, pos.numpy(), f, amp, inter)
    for got, y, t in ((values(kc[at], sc[at, :, 0]), want, tol), (values(vc[at], sc[at, :, 1]), _np(v), np.zeros_like(tol))):
        # a code is off by half a step: 2^-4 of the value, or half of the smallest step 2^-9 of the row's power of
        # two, which is at most 2^-7 of its largest value (at least 224 of it, or the exponent were smaller)
        top = np.abs(y).max(-1, keepdims=True) + t.max(-1, keepdims=True)
        _close(got, y, t + np.maximum(2.0 ** -4 * (np.abs(y) + t), 2.0 ** -10 * top * 2.0 ** -7), "values")
    # the values are those of the plain store, byte for byte
    plain = [torch.full((ns, hkv, x), 5, dtype=torch.uint8, device="cuda") for x in (d, d, 2)]
    ac.acache_write_slots_q8(_desc(hq, hkv, d, dtype), B, rows, dev(slots), gk.contiguous(), gv.contiguous(), *plain, ns, 0)
    torch.cuda.synchronize()
    assert torch.equal(pool[1], plain[1]) and torch.equal(pool[2][..., 1], plain[2][..., 1])
    rest = np.setdiff1d(np.arange(ns), at)
    assert (kc[rest] == 5).all() and (vc[rest] == 5).all() and (sc[rest] == 5).all()


def test_store_with_nothing_to_turn_is_the_plain_store():
    g = torch.Generator().manual_seed(9)
    n, hkv, d, ns = 50, 4, 128, 60
    (_, k, v), (_, gk, gv) = _new(n, 4, hkv, d, F32, g, False)
    slots = dev(torch.randperm(ns, generator=g)[:n].to(torch.int32))
    for q8 in (False, True):
        pools = []
        for turn in (False, True):
            pool = [torch.full((ns, hkv, d), 5, dtype=torch.uint8 if q8 else F32, device="cuda") for _ in range(2)]
            if q8:
                pool.append(torch.full((ns, hkv, 2), 5, dtype=torch.uint8, device="cuda"))
            desc = _desc(4, hkv, d, F32)
            if turn:
                call = ac.acache_rotate_store_q8 if q8 else ac.acache_rotate_store
                call(desc, None, 1, n, None, slots, None, gk, gv, None, *pool, ns, 0)
            else:
                call = ac.acache_write_slots_q8 if q8 else ac.acache_write_slots
                call(desc, 1, n, slots, gk, gv, *pool, ns, 0)
            pools.append(pool)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(*pools))


@pytest.mark.parametrize("q8", [False, True])
def test_store_skips_and_flags_bad_and_shared_slots(q8):
    g = torch.Generator().manual_seed(3)
    d, hq, hkv, ns = 128, 4, 2, 40
    (q, k, v), (gq, gk, gv) = _new(4, hq, hkv, d, BF16, g, True)
    rope, f, amp = _rope(128, False)
    pos = torch.tensor([4, 5, 6, 7], dtype=torch.int32)
    for slot, bit in ((-1, _lib.DEV_BAD_SLOT), (ns, _lib.DEV_BAD_SLOT), (2 ** 31 - 1, _lib.DEV_BAD_SLOT), (9, _lib.DEV_SHARED_WRITE)):
        pool = [torch.full((ns, hkv, d), 7, dtype=torch.uint8 if q8 else BF16, device="cuda") for _ in range(2)]
        if q8:
            pool.append(torch.full((ns, hkv, 2), 7, dtype=torch.uint8, device="cuda"))
        st, qo = _status(), torch.empty((4, hq, d), dtype=BF16, device="cuda")
        slots = torch.tensor([20, slot, 11, 39], dtype=torch.int32, device="cuda")
        call = ac.acache_rotate_store_q8 if q8 else ac.acache_rotate_store
        call(_desc(hq, hkv, d, BF16), rope, 1, 4, dev(pos), slots, gq, gk, gv, qo, *pool, ns, 10, dev_status=st)
        torch.cuda.synchronize()
        assert st.item() == bit
        _check_rows(qo, q, None, pos.numpy(), f, amp, False, BF16, "queries")
        wrote = torch.zeros(ns, dtype=torch.bool)
        wrote[[20, 11, 39]] = True
        for t in pool:
            assert (t.cpu()[~wrote].float() == 7).all() and (t.cpu()[wrote].float() != 7).any()


def test_store_8_bit_poisons_rows_that_are_not_finite():
    d, hkv = 64, 2
    x = torch.randn((1, 3, hkv, d), generator=torch.Generator().manual_seed(4)).to(BF16).cuda()
    k, v = x.clone(), x.clone()
    k[0, 0, 1, 3], v[0, 2, 0, 9] = NAN, INF
    pool = [torch.zeros((3, hkv, n), dtype=torch.uint8, device="cuda") for n in (d, d, 2)]
    st, slots = _status(), torch.arange(3, dtype=torch.int32, device="cuda")
    ac.acache_rotate_store_q8(_desc(2, hkv, d, BF16), _rope(64, False)[0], 1, 3, slots, slots, None, k, v, None, *pool, 3, 0, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == _lib.DEV_BAD_VALUE
    sc = pool[2].cpu()
    assert sc[0, 1, 0] == 255 and sc[2, 0, 1] == 255 and (sc == 255).sum() == 2
    assert (pool[0][0, 1] == 0).all() and (pool[1][2, 0] == 0).all()


# ------------------------------------------------------------------------------------- masked attention
def _ranges(kind, n, T, g):
    """lo, hi of the last n positions (they may lie before the first key when n > T)."""
    p = torch.arange(T - n, T)
    zero, full = torch.zeros(n, dtype=torch.long), torch.full((n,), T)
    if kind == "causal":
        return zero, p + 1
    if kind == "window":
        return (p - 20).clamp_min(0), p + 1
    if kind == "blocks":
        return zero, ((p.div(32, rounding_mode="floor") + 1) * 32)
    if kind == "documents":
        cuts = torch.cat((torch.tensor([0]), torch.randint(0, T + 1, (4,), generator=g).sort()[0], torch.tensor([T])))
        doc = (torch.searchsorted(cuts, p, right=True) - 1).clamp(0, 4)
        return cuts[doc], cuts[doc + 1]
    if kind == "any":              # ends beyond the keys, before them, the wrong way round
        lo, hi = torch.randint(-20, T + 20, (n,), generator=g), torch.randint(-20, T + 20, (n,), generator=g)
        return lo, hi
    if kind == "none":
        return zero, zero
    return zero, full


def _attend_case(dtype, hq, hkv, d, B, n, T, kind, cap=0.0, bias=False, drop=False, seed=0, scale=None, poison=True):
    g = torch.Generator().manual_seed(1000 * seed + n + T + hq)
    ns = B * T + 9
    q = (1.5 * torch.randn((B, n, hq, d), generator=g)).to(dtype)
    kp, vp = (torch.randn((ns, hkv, d), generator=g).to(dtype) for _ in range(2))
    rs = torch.randperm(ns, generator=g)[:B * T].to(torch.int32).view(B, T)
    if seed % 2:
        rs[:, : T // 2] = torch.arange(T // 2, dtype=torch.int32)          # shared, consecutive
    if drop:
        rs[torch.rand((B, T), generator=g) < 0.3] = -1
    rr = torch.stack([torch.stack(_ranges(kind, n, T, g), -1) for _ in range(B)]).to(torch.int32)
    pos = torch.randint(0, T + 5, (B, n), generator=g, dtype=torch.int32) if bias else None
    slopes = torch.exp2(-8 * torch.arange(1, hq + 1) / hq) if bias else None
    if poison and kind not in ("full",):
        # keys that no row of their request sees hold what must not be looked at
        for b in range(B):
            t = torch.arange(T)
            unseen = ~((t >= rr[b, :, :1]) & (t < rr[b, :, 1:])).any(0)
            others = torch.cat([rs[c][((t >= rr[c, :, :1]) & (t < rr[c, :, 1:])).any(0)] for c in range(B)])
            for x, s in enumerate(rs[b][unseen].tolist()):
                if s >= 0 and s not in others:
                    kp[s], vp[s] = (NAN, INF, -INF)[x % 3], (INF, NAN, NAN)[x % 3]
    out = torch.full((B, n, hq, d), 7.0, dtype=dtype, device="cuda")
    st = _status()
    ac.acache_slot_attention_masked(_desc(hq, hkv, d, dtype, scale), B, n, dev(q), T, dev(rs), dev(kp), dev(vp), ns, out,
                                    row_range=None if kind == "full" else dev(rr), q_pos=None if pos is None else dev(pos),
                                    slopes=None if slopes is None else dev(slopes), softcap=cap, drop_none=drop, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for b in range(B):
        want, tol = masked_attention(q[b], rs[b].numpy(), kp, vp, d ** -0.5 if scale is None else scale, rr[b, :, 0], rr[b, :, 1],
                                     None if pos is None else pos[b].numpy(), None if slopes is None else slopes.numpy(), cap, drop)
        assert_attention(_np(out[b]), want, tol, f"request {b}")


KINDS = ["full", "causal", "window", "blocks", "documents", "any", "none"]


@pytest.mark.parametrize("dtype,hq,hkv,d", [(BF16, 4, 1, 128), (BF16, 2, 2, 64), (F32, 2, 1, 128), (F32, 3, 3, 64)])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,n,T", [(1, 1, 1), (2, 1, 300), (1, 8, 129), (2, 45, 200), (1, 150, 130)])
def test_masked_attention(dtype, hq, hkv, d, kind, B, n, T):
    _attend_case(dtype, hq, hkv, d, B, n, T, kind, seed=B)


@pytest.mark.parametrize("dtype,hq,hkv,d", [(BF16, 7, 1, 128), (BF16, 4, 2, 64), (F32, 2, 2, 64)])
@pytest.mark.parametrize("kind", ["causal", "any"])
@pytest.mark.parametrize("cap,bias,drop", [(1.5, False, False), (0.0, True, False), (30.0, True, True), (0.0, False, True)])
@pytest.mark.parametrize("n,T", [(1, 700), (4, 65), (70, 257)])
def test_masked_attention_caps_biases_and_discarded_keys(dtype, hq, hkv, d, kind, cap, bias, drop, n, T):
    _attend_case(dtype, hq, hkv, d, 2, n, T, kind, cap=cap, bias=bias, drop=drop, seed=3)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("cap", [0.01, 511.0, 513.0, 2e5, 1e12])
def test_masked_attention_with_small_and_large_caps(dtype, n, cap):
    """Up to a cap of 512 the score is off by 2^-22 of the cap, above by 2^-20 of itself."""
    _attend_case(dtype, 4, 2, 128, 1, n, 160, "causal", cap=cap, seed=6)


@pytest.mark.parametrize("n", [1, 40, 130])
@pytest.mark.parametrize("scale", [-0.1, 0.0])
def test_masked_attention_with_a_scale_that_is_not_positive(n, scale):
    _attend_case(BF16, 4, 2, 128, 1, n, 160, "causal", cap=3.0, scale=scale, seed=4)


@pytest.mark.parametrize("hq,hkv,d", [(7, 1, 128), (4, 2, 64)])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,n,T", [(1, 40, 700), (3, 60, 1500), (1, 33, 2700), (2, 150, 2600)])
def test_masked_attention_of_few_blocks_over_many_keys(hq, hkv, d, kind, B, n, T):
    """Blocks that a cluster of 2, 4 or 8 CTAs shares, each with a part of the keys; some parts hold none of a row's."""
    _attend_case(BF16, hq, hkv, d, B, n, T, kind, seed=B)


@pytest.mark.parametrize("hq,hkv,d", [(7, 1, 128), (16, 2, 64)])
@pytest.mark.parametrize("kind", ["causal", "any"])
@pytest.mark.parametrize("cap,bias,drop", [(1.5, False, False), (0.0, True, False), (80.0, True, True), (700.0, False, True)])
@pytest.mark.parametrize("n,T", [(37, 900), (70, 2700)])
def test_masked_attention_of_few_blocks_caps_biases_and_discarded_keys(hq, hkv, d, kind, cap, bias, drop, n, T):
    _attend_case(BF16, hq, hkv, d, 1, n, T, kind, cap=cap, bias=bias, drop=drop, seed=5)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [700, 2700])
def test_what_one_row_sees_does_not_reach_its_neighbours_over_many_keys(d, T):
    """NaN and infinities in keys and values of some parts of a block's keys, which some rows see and others do not."""
    g = torch.Generator().manual_seed(T)
    hq, hkv, n = 4, 2, 100
    q = torch.randn((1, n, hq, d), generator=g).to(BF16)
    kp, vp = (torch.randn((T, hkv, d), generator=g).to(BF16) for _ in range(2))
    rs = torch.randperm(T, generator=g).to(torch.int32)[None]
    kp[rs[0, T - 2], 0, 3] = NAN
    vp[rs[0, T - 1], 1, 5] = INF
    vp[rs[0, 40], 0, 7] = NAN
    kp[rs[0, 41], 1] = INF
    vp[rs[0, T // 2], :, 9] = -INF
    lo, hi = torch.zeros(n, dtype=torch.int32), torch.full((n,), T, dtype=torch.int32)
    hi[::2] = T - 2
    lo[::3] = 42
    hi[1::5] = T // 2
    lo[n // 2] = hi[n // 2] = 10
    out, st = torch.empty((1, n, hq, d), dtype=BF16, device="cuda"), _status()
    ac.acache_slot_attention_masked(_desc(hq, hkv, d, BF16), 1, n, dev(q), T, dev(rs), dev(kp), dev(vp), T, out,
                                    row_range=dev(torch.stack((lo, hi), -1)[None]), dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    want, tol = masked_attention(q[0], rs[0].numpy(), kp, vp, d ** -0.5, lo, hi)
    assert np.isnan(want).any() and (want[n // 2] == 0).all()
    got = _np(out[0])
    fine = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), fine)
    assert (np.abs(got[fine] - want[fine]) - tol[fine]).max(initial=0.0) <= 0


@pytest.mark.parametrize("n,cap", [(40, 0.0), (200, 30.0)])
def test_masked_waits_of_shared_blocks_that_run_out(n, cap):
    """One request whose blocks are shared by clusters: no row is written that lacks a part."""
    g = torch.Generator().manual_seed(n)
    hq, hkv, d, T = 8, 1, 128, 2700
    q = torch.randn((1, n, hq, d), generator=g).to(BF16)
    kp, vp = (torch.randn((T, hkv, d), generator=g).to(BF16) for _ in range(2))
    args = (_desc(hq, hkv, d, BF16), 1, n, dev(q), T, dev(torch.randperm(T, generator=g).to(torch.int32)[None]), dev(kp), dev(vp), T)

    def call():
        out, st = torch.full((1, n, hq, d), 7.0, dtype=BF16, device="cuda"), _status()
        ac.acache_slot_attention_masked(*args, out, softcap=cap, dev_status=st)
        torch.cuda.synchronize()
        return out, st.item()

    want, st = call()
    assert st == 0
    timed_out = 0
    for budget in (1, 300, 1000, 2000, 4000, 8000):
        prev = ac.acache_wait_budget(budget)
        try:
            out, st = call()
        finally:
            ac.acache_wait_budget(prev)
        assert st in (0, _lib.DEV_TIMEOUT)
        timed_out += st != 0
        same = (out == want).all(-1)
        assert (same | (out == 7.0).all(-1)).all()
        assert st != 0 or same.all()
    assert timed_out
    out, st = call()
    assert st == 0 and torch.equal(out, want)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 128)])
@pytest.mark.parametrize("n", [1, 5, 100, 300])
def test_what_one_row_sees_does_not_reach_its_neighbours(dtype, d, n):
    """NaN and infinities in keys and values that some rows see and others do not."""
    g = torch.Generator().manual_seed(n)
    hq, hkv, T = 4, 2, 310
    q = torch.randn((1, n, hq, d), generator=g).to(dtype)
    kp, vp = (torch.randn((T, hkv, d), generator=g).to(dtype) for _ in range(2))
    rs = torch.randperm(T, generator=g).to(torch.int32)[None]
    kp[rs[0, 300], 0, 3] = NAN
    vp[rs[0, 301], 1, 5] = INF
    vp[rs[0, 40], 0, 7] = NAN
    kp[rs[0, 41], 1] = INF
    lo, hi = torch.zeros(n, dtype=torch.int32), torch.full((n,), T, dtype=torch.int32)
    hi[::2] = 300
    lo[::3] = 42
    lo[n // 2] = hi[n // 2] = 10                               # and a row that sees nothing
    out, st = torch.empty((1, n, hq, d), dtype=dtype, device="cuda"), _status()
    ac.acache_slot_attention_masked(_desc(hq, hkv, d, dtype), 1, n, dev(q), T, dev(rs), dev(kp), dev(vp), T, out,
                                    row_range=dev(torch.stack((lo, hi), -1)[None]), dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    want, tol = masked_attention(q[0], rs[0].numpy(), kp, vp, d ** -0.5, lo, hi)
    assert np.isnan(want).any() or n == 1
    # a weight of an infinite or NaN value or key: NaN or infinite there; the sign of infinities is the formula's
    got = _np(out[0])
    fine = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), fine)
    assert (np.abs(got[fine] - want[fine]) - tol[fine]).max(initial=0.0) <= 0


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("n", [1, 33, 200])
def test_query_rows_that_are_not_finite(dtype, d, n):
    g = torch.Generator().manual_seed(n)
    T = 140
    q = torch.randn((1, n, 2, d), generator=g).to(dtype)
    q[0, n - 1, 0, 3], q[0, 0, 1, 1] = NAN, INF
    kp, vp = (torch.randn((T, 1, d), generator=g).to(dtype) for _ in range(2))
    rs = torch.arange(T, dtype=torch.int32)[None]
    for empty in (False, True):
        rr = torch.tensor([0, 0 if empty else T], dtype=torch.int32).expand(1, n, 2).contiguous()
        out = torch.empty((1, n, 2, d), dtype=dtype, device="cuda")
        ac.acache_slot_attention_masked(_desc(2, 1, d, dtype), 1, n, dev(q), T, dev(rs), dev(kp), dev(vp), T, out, row_range=dev(rr))
        torch.cuda.synchronize()
        bad = torch.zeros((n, 2), dtype=torch.bool)
        if not empty:
            bad[n - 1, 0] = bad[0, 1] = True
        assert torch.equal(out[0].isnan().all(-1).cpu(), bad) and torch.equal(out[0].isnan().any(-1).cpu(), bad)
        assert not empty or (out == 0).all()


def test_masked_attention_flags_and_zeroes_bad_slots():
    g = torch.Generator().manual_seed(11)
    for dtype in (BF16, F32):
        for n in (1, 40, 200):
            hq, hkv, d, T, ns = 4, 2, 128, 200, 210
            q = torch.randn((1, n, hq, d), generator=g).to(dtype)
            kp, vp = (torch.randn((ns, hkv, d), generator=g).to(dtype) for _ in range(2))
            rs = torch.randperm(ns, generator=g)[:T].to(torch.int32)[None]
            rs[0, 7], rs[0, 150], rs[0, 199] = -5, ns, 2 ** 31 - 1
            lo, hi = torch.zeros(n, dtype=torch.int32), torch.full((n,), T, dtype=torch.int32)
            out, st = torch.empty((1, n, hq, d), dtype=dtype, device="cuda"), _status()
            ac.acache_slot_attention_masked(_desc(hq, hkv, d, dtype), 1, n, dev(q), T, dev(rs), dev(kp), dev(vp), ns, out,
                                            row_range=dev(torch.stack((lo, hi), -1)[None]), softcap=5.0, dev_status=st)
            torch.cuda.synchronize()
            assert st.item() == _lib.DEV_BAD_SLOT
            want, tol = masked_attention(q[0], rs[0].numpy(), kp, vp, d ** -0.5, lo, hi, cap=5.0)
            assert_attention(_np(out[0]), want, tol)
    # an empty pool: every key is a row of zeros
    out, st = torch.full((1, 3, 4, 128), 7.0, dtype=BF16, device="cuda"), _status()
    x = torch.ones((1, 3, 4, 128), dtype=BF16, device="cuda")
    ac.acache_slot_attention_masked(_desc(4, 2, 128, BF16), 1, 3, x, 5, dev(torch.zeros(5, dtype=torch.int32)), x, x, 0, out, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == _lib.DEV_BAD_SLOT and (out == 0).all()


@pytest.mark.parametrize("dtype,hq,hkv,d", [(BF16, 4, 1, 128), (BF16, 8, 8, 64), (F32, 2, 1, 64)])
@pytest.mark.parametrize("cap,bias,drop", [(0.0, False, False), (4.0, True, True)])
def test_masked_attention_over_a_ragged_batch(dtype, hq, hkv, d, cap, bias, drop):
    g = torch.Generator().manual_seed(hq + d)
    rows, keys = [300, 1, 0, 17, 1, 128, 5, 3, 2], [310, 700, 40, 17, 1, 500, 90, 4, 30]
    keys[8] = 0                                     # rows without keys
    max_q, max_T, B = 300, 700, len(rows)
    qs, ks = (np.concatenate(([0], np.cumsum(x))).astype(np.int32) for x in (rows, keys))
    total, nk = int(qs[-1]), int(ks[-1])
    ns = nk + 5
    q = torch.randn((total, hq, d), generator=g).to(dtype)
    kp, vp = (torch.randn((ns, hkv, d), generator=g).to(dtype) for _ in range(2))
    rs = torch.randperm(ns, generator=g)[:nk].to(torch.int32)
    if drop:
        rs[torch.rand(nk, generator=g) < 0.3] = -1
    lo, hi = (torch.zeros(total, dtype=torch.int32) for _ in range(2))
    pos = torch.zeros(total, dtype=torch.int32)
    for b in range(B):
        a, z = int(qs[b]), int(qs[b + 1])
        p = torch.arange(keys[b] - rows[b], keys[b])
        pos[a:z], lo[a:z], hi[a:z] = p.int(), (p - 100).clamp_min(0).int(), (p + 1).int()
    slopes = torch.exp2(-8 * torch.arange(1, hq + 1) / hq) if bias else None
    out, st = torch.full((total + 2, hq, d), 7.0, dtype=dtype, device="cuda"), _status()
    ac.acache_slot_attention_masked_varlen(
        _desc(hq, hkv, d, dtype), B, dev(torch.from_numpy(qs)), max_q, total, dev(q), dev(torch.from_numpy(ks)), max_T, dev(rs),
        dev(kp), dev(vp), ns, out, row_range=dev(torch.stack((lo, hi), -1)), q_pos=dev(pos) if bias else None,
        slopes=dev(slopes) if bias else None, softcap=cap, drop_none=drop, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == _lib.DEV_BAD_LENGTH          # the request with rows and no key
    for b in range(B):
        a, z = int(qs[b]), int(qs[b + 1])
        if keys[b] == 0:
            assert (out[a:z] == 7).all()
            continue
        want, tol = masked_attention(q[a:z], rs[ks[b]:ks[b + 1]].numpy(), kp, vp, d ** -0.5, lo[a:z], hi[a:z], pos[a:z].numpy(),
                                     slopes.numpy() if bias else None, cap, drop)
        assert_attention(_np(out[a:z]), want, tol, f"request {b}")
    assert (out[total:] == 7).all()


@pytest.mark.parametrize("max_q", [4, 300])
def test_ragged_requests_outside_their_bounds_are_skipped(max_q):
    g = torch.Generator().manual_seed(12)
    hq, hkv, d = 4, 2, 128
    total, T = 12, 50
    q = torch.randn((total, hq, d), generator=g).to(BF16)
    kp, vp = (torch.randn((T, hkv, d), generator=g).to(BF16) for _ in range(2))
    rs = torch.arange(T, dtype=torch.int32)
    for qs, ks, fine in (([0, 4, 8], [0, 20, 200], [True, False]),          # more keys than max_seq_len
                         ([0, 4, 2], [0, 20, 40], [True, False]),           # a negative count
                         ([-4, 0, 4], [0, 20, 40], [False, True]),          # rows in front of q
                         ([0, 4, 8 + max_q], [0, 20, 40], [True, False]),   # behind q, or above the bound
                         ([0, 4, 8], [20, 10, 40], [False, True])):
        out, st = torch.full((total, hq, d), 7.0, dtype=BF16, device="cuda"), _status()
        ac.acache_slot_attention_masked_varlen(_desc(hq, hkv, d, BF16), 2, dev(torch.tensor(qs, dtype=torch.int32)), max_q, total, dev(q),
                                               dev(torch.tensor(ks, dtype=torch.int32)), 40, dev(rs), dev(kp), dev(vp), T, out, dev_status=st)
        torch.cuda.synchronize()
        assert st.item() == _lib.DEV_BAD_LENGTH, (qs, ks)
        written = torch.zeros(total, dtype=torch.bool)
        for b in range(2):
            if fine[b]:
                a, z = qs[b], qs[b + 1]
                written[a:z] = True
                want, tol = masked_attention(q[a:z], rs[ks[b]:ks[b + 1]].numpy(), kp, vp, d ** -0.5, [0] * 4, [T] * 4)
                assert_attention(_np(out[a:z]), want, tol)
        assert (out.cpu()[~written] == 7).all()


def test_masked_attention_without_a_mask_is_the_plain_call():
    """No range, cap or bias: within rounding of acache_slot_attention, at a recompute point and a single token."""
    g = torch.Generator().manual_seed(13)
    hq, hkv, d, T = 28, 4, 128, 900
    kp, vp = (torch.randn((T, hkv, d), generator=g).to(BF16).cuda() for _ in range(2))
    rs = dev(torch.randperm(T, generator=g).to(torch.int32)[None])
    for n in (1, 32, 400):
        q = torch.randn((1, n, hq, d), generator=g).to(BF16).cuda()
        a, b = (torch.empty_like(q) for _ in range(2))
        ac.acache_slot_attention(_desc(hq, hkv, d, BF16), 1, n, q, T, rs, kp, vp, T, a)
        ac.acache_slot_attention_masked(_desc(hq, hkv, d, BF16), 1, n, q, T, rs, kp, vp, T, b)
        torch.cuda.synchronize()
        # two bf16 roundings of the output, and of the weights on both sides: |o| <= max |v| < 5 here
        assert (a.float() - b.float()).abs().max().item() <= 4 * 2.0 ** -8 * 1.0


# ------------------------------------------------------------------------------------- token scores
def _score(x, tokens, k, temperature=1.0, entropy=True, x_gpu=None):
    R, V = x.shape
    gx = dev(x) if x_gpu is None else x_gpu
    st = _status()
    lp = torch.full((R,), 7.0, device="cuda") if tokens is not None else None
    H = torch.full((R,), 7.0, device="cuda") if entropy else None
    tt = torch.full((R, k), -7, dtype=torch.int32, device="cuda") if k else None
    tl = torch.full((R, k), 7.0, device="cuda") if k else None
    ac.acache_token_scores(R, V, gx, tokens=None if tokens is None else dev(tokens), token_logprob=lp, entropy=H, top_tokens=tt,
                           top_logprob=tl, temperature=temperature, dev_status=st)
    torch.cuda.synchronize()
    return lp, H, tt, tl, st.item()


def _check_scores(x, k, temperature=1.0, seed=0, x_gpu=None, status=0):
    R, V = x.shape
    tokens = torch.randint(0, V, (R,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
    lp, H, tt, tl, st = _score(x, tokens, k, temperature, x_gpu=x_gpu)
    assert st == status
    wl, wh, order, tol, tol_h = token_scores(x, temperature)
    at = np.arange(R)
    _close(_np(lp), wl[at, tokens.numpy()], tol[at, tokens.numpy()], "given")
    _close(_np(H), wh, tol_h, "entropy")
    if k:
        assert np.array_equal(tt.cpu().numpy(), order[:, :k])
        _close(_np(tl), np.take_along_axis(wl, order[:, :k], 1), np.take_along_axis(tol, order[:, :k], 1), "alternatives")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [1, 2, 7, 31, 64, 257, 1000, 4097, 9001, 50021, 131072])
@pytest.mark.parametrize("R,k", [(1, 1), (3, 5), (2, 32), (5, 0)])
def test_scores(dtype, V, R, k):
    g = torch.Generator().manual_seed(V + R)
    x = (3 * torch.randn((R, V), generator=g)).to(dtype)
    x[0, V // 2] += 20
    _check_scores(x, min(k, V), seed=V)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R,V", [(1900, 1100), (1900, 4003), (1900, 8190), (930, 8200), (930, 16385), (930, 32760)])
@pytest.mark.parametrize("k", [0, 1, 8, 9, 32])
def test_scores_of_many_short_rows(dtype, R, V, k):
    """Enough rows to fill the SMs with small CTAs."""
    V = V if dtype == BF16 else V // 2
    g = torch.Generator().manual_seed(V + k)
    few = (3 * torch.randn((24, V), generator=g)).to(dtype)
    few[1] = (few[1] * 0.5).round()                       # many alike
    few[2, 7:] = -INF
    few[3] = 1.0
    few[4, V - 60:] = 40.0
    x = few.repeat((R + 23) // 24, 1)[:R]
    lp, H, tt, tl, st = _score(x, torch.arange(R, dtype=torch.int32) % 7, k)
    assert st == 0
    wl, wh, order, tol, tol_h = token_scores(few, 1.0)
    at = np.arange(R) % 24
    _close(_np(lp), wl[at, np.arange(R) % 7], tol[at, np.arange(R) % 7], "given")
    _close(_np(H), wh[at], tol_h[at], "entropy")
    if k:
        assert np.array_equal(tt.cpu().numpy(), order[at, :k])
        _close(_np(tl), np.take_along_axis(wl, order[:, :k], 1)[at], np.take_along_axis(tol, order[:, :k], 1)[at], "alternatives")


@pytest.mark.parametrize("temperature", [0.05, 0.7, 1.5, 40.0])
def test_scores_with_a_temperature(temperature):
    g = torch.Generator().manual_seed(5)
    _check_scores((4 * torch.randn((3, 5003), generator=g)).to(F32), 8, temperature)
    _check_scores((4 * torch.randn((300, 700), generator=g)).to(BF16), 3, temperature)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V,pad,lead", [(1003, 5, 0), (5, 3, 1), (33000, 1, 3), (32, 1, 7), (8191, 64, 2)])
def test_scores_of_rows_that_are_not_aligned(dtype, V, pad, lead):
    """What lies beside the rows must not be read into them: it is larger than anything in them."""
    g = torch.Generator().manual_seed(V)
    R = 6
    buf = torch.full((R * (V + pad) + lead,), 1000.0)
    x = buf[lead:lead + R * (V + pad)].view(R, V + pad)[:, :V]
    x.copy_(3 * torch.randn((R, V), generator=g))
    buf = buf.to(dtype)
    on = dev(buf)
    view = on[lead:lead + R * (V + pad)].view(R, V + pad)[:, :V]
    _check_scores(buf[lead:lead + R * (V + pad)].view(R, V + pad)[:, :V], min(4, V), x_gpu=view)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [40, 600, 20011, 70001])
def test_ties_go_to_the_lower_token(dtype, V):
    g = torch.Generator().manual_seed(V)
    low = torch.finfo(dtype).min
    x = torch.stack([torch.zeros(V), torch.full((V,), low), torch.randint(0, 3, (V,), generator=g).float(), -torch.zeros(V),
                     torch.arange(V).float() // 8, (torch.arange(V) % 512 == 5).float() * 3]).to(dtype)
    x[3, ::2] = 0.0                                     # +0.0 and -0.0 are one value
    _check_scores(x, 32)


@pytest.mark.parametrize("k", [2, 32])
def test_candidates_of_one_thread_and_of_all(k):
    """More candidates than the list holds: the largest logits sit in the pieces of a few threads."""
    g = torch.Generator().manual_seed(k)
    V, N = 512 * 8 * 60, 8
    piece = torch.arange(V) // N
    for threads in (1, k - 1, k):
        x = torch.randn((1, V), generator=g)
        x[0] += 50.0 * (piece % 512 < threads)
        _check_scores(x.to(BF16).expand(400, V).contiguous()[:1], k)
        # (many rows: no cluster, so a thread has all of its 60 pieces)
        y = dev(x.to(BF16).expand(400, V).contiguous())
        tt = torch.empty((400, k), dtype=torch.int32, device="cuda")
        ac.acache_token_scores(400, V, y, top_tokens=tt)
        torch.cuda.synchronize()
        _, _, order, _, _ = token_scores(x.to(BF16), 1.0)
        assert (tt.cpu().numpy() == order[0, :k]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [300, 5003, 130001])
@pytest.mark.parametrize("k", [1, 5, 32])
def test_few_tokens_left_and_many_alike(dtype, V, k):
    """Rows of which a handful can be chosen (the rest -infinity, in front and behind), and rows with thousands of
    logits at the k-th best value, few or many above it."""
    g = torch.Generator().manual_seed(V + k)
    x = torch.full((8, V), -INF)
    x[0, [V // 2, V - 1, 3]] = torch.tensor([1.0, 2.0, 1.0])
    x[1] = torch.randint(0, 2, (V,), generator=g).float()
    x[2] = 1.0
    x[2, torch.randint(0, V, (3,), generator=g)] = 2.0
    x[3] = torch.randint(0, 200, (V,), generator=g).clamp_max(190).float()
    x[4, V - 60:] = 4.0                                   # the alike lie at the end
    x[5] = torch.where(torch.arange(V) % 3 == 0, 5.0, torch.randn(V, generator=g))
    x[6, :40], x[6, 40:] = NAN, -INF
    x[7, ::2] = NAN
    x[7, V - 1] = 0.5
    st = _lib.DEV_NAN
    _check_scores(x.to(dtype), min(k, V), status=st)
    _check_scores(x[:6].to(dtype).repeat(60, 1), min(k, V))      # many rows: no cluster


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [9, 3000, 40000])
def test_scores_of_what_is_not_finite(dtype, V):
    g = torch.Generator().manual_seed(V)
    x = torch.randn((6, V), generator=g)
    x[0] = -INF
    x[1, :V - 2] = -INF                                  # two tokens left
    x[2, V // 3] = NAN
    x[3, V // 2] = INF
    x[4] = NAN
    x[5, 1::2] = -INF
    _check_scores(x.to(dtype), min(5, V), status=_lib.DEV_NAN)
    _check_scores(x[[0, 1, 5]].to(dtype), min(32, V))    # no NaN, no +infinity: nothing to flag


def test_tokens_outside_the_vocabulary_are_left_and_flagged():
    x = torch.randn((5, 300), generator=torch.Generator().manual_seed(1))
    tokens = torch.tensor([0, -1, 299, 300, 2 ** 31 - 1], dtype=torch.int32)
    lp, _, _, _, st = _score(x, tokens, 0)
    assert st == _lib.DEV_BAD_TOKEN
    assert [i for i in range(5) if lp[i].item() == 7.0] == [1, 3, 4]
    # k alone, and an entropy alone
    _, H, tt, _, st = _score(x, None, 3, entropy=False)
    assert H is None and st == 0 and torch.equal(tt.cpu().long(), x.topk(3, 1).indices)
    _, H, _, _, _ = _score(x, None, 0)
    assert torch.isfinite(H).all()


def test_scores_of_rows_beyond_32_bit_offsets():
    V, stride = 1001, (1 << 28) + 3
    buf = torch.empty(9 * stride + V, dtype=BF16, device="cuda")
    rows = buf.as_strided((10, V), (stride, 1))
    x = (3 * torch.randn((10, V), generator=torch.Generator().manual_seed(2))).to(BF16)
    rows.copy_(x)
    _check_scores(x, 4, x_gpu=rows)


# ------------------------------------------------------------------------------------- together
def _step(B, n, hq, hkv, d, T, V, q8):
    """A decoding step's inputs: new rows out of a fused projection, a pool with the request's earlier keys."""
    g = torch.Generator().manual_seed(B + n + T)
    ns = B * T + 16
    qkv = torch.randn((B, n, hq + 2 * hkv, d), generator=g).to(BF16)
    slots = torch.randperm(ns, generator=g)[:B * T].to(torch.int32).view(B, T)
    pos = torch.arange(T - n, T, dtype=torch.int32).expand(B, n).contiguous()
    blocks = torch.stack((torch.zeros_like(pos), ((pos // 8 + 1) * 8).clamp_max(T)), -1)
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(BF16)
    head = (torch.randn((hq * d, V), generator=g) * (hq * d) ** -0.5 * 3).to(BF16)
    kp, vp = (torch.randn((ns, hkv, d), generator=g).to(BF16) for _ in range(2))
    return qkv, slots, pos, blocks, w, head, kp, vp, ns


@pytest.mark.parametrize("B,n,T", [(2, 1, 90), (2, 24, 160)])
def test_a_decoding_step_eager_and_captured(B, n, T):
    """Norm, rotation and store, attention under a block mask with a cap, logits, scores: eager, then the same captured
    into a graph and replayed on new inputs; each stage against the 64-bit reference of what the stage before gave."""
    hq, hkv, d, V = 8, 2, 128, 3001
    qkv, slots, pos, rr, w, head, kp, vp, ns = _step(B, n, hq, hkv, d, T, V, False)
    rope, f, amp = _rope(128, False)
    desc = _desc(hq, hkv, d, BF16)
    x = dev(qkv)
    gk, gv, gs, gp, gr, gw, gh = (dev(t) for t in (kp, vp, slots, pos, rr, w, head))
    new_slots = gs[:, T - n:].contiguous()
    qo, out, st = torch.empty((B, n, hq, d), dtype=BF16, device="cuda"), torch.empty((B, n, hq, d), dtype=BF16, device="cuda"), _status()
    logits = torch.empty((B * n, V), dtype=BF16, device="cuda")
    H, tt, tl = torch.empty(B * n, device="cuda"), torch.empty((B * n, 3), dtype=torch.int32, device="cuda"), torch.empty((B * n, 3), device="cuda")

    def step():
        q, k, v = x.split((hq, hkv, hkv), 2)
        ac.acache_rotate_store(desc, rope, B, n, gp, new_slots, q, k, v, qo, gk, gv, ns, 0, q_weight=gw, k_weight=gw, dev_status=st)
        ac.acache_slot_attention_masked(desc, B, n, qo, T, gs, gk, gv, ns, out, row_range=gr, softcap=20.0, dev_status=st)
        torch.matmul(out.view(B * n, hq * d), gh, out=logits)
        ac.acache_token_scores(B * n, V, logits, entropy=H, top_tokens=tt, top_logprob=tl, dev_status=st)

    def check():
        torch.cuda.synchronize()
        assert st.item() == 0
        q, k, v = x.cpu().split((hq, hkv, hkv), 2)
        p = pos.reshape(-1).numpy()
        _check_rows(qo.view(-1, hq, d), q.reshape(-1, hq, d), w, p, f, amp, False, BF16, "queries")
        at = new_slots.cpu().view(-1).long()
        _check_rows(gk.cpu()[at], k.reshape(-1, hkv, d), w, p, f, amp, False, BF16, "keys")
        assert torch.equal(gv.cpu()[at], v.reshape(-1, hkv, d))
        for b in range(B):
            want, tol = masked_attention(qo[b].cpu(), slots[b].numpy(), gk.cpu(), gv.cpu(), d ** -0.5, rr[b, :, 0], rr[b, :, 1], cap=20.0)
            assert_attention(_np(out[b]), want, tol)
        wl, wh, order, tol, tol_h = token_scores(logits.cpu(), 1.0)
        assert np.array_equal(tt.cpu().numpy(), order[:, :3])
        _close(_np(tl), np.take_along_axis(wl, order[:, :3], 1), np.take_along_axis(tol, order[:, :3], 1))
        _close(_np(H), wh, tol_h)

    step()
    check()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)).to(BF16))
        graph.replay()
        check()


def test_a_step_over_the_8_bit_pool():
    """The rotating store into an 8-bit pool, then the pool's own attention, against the plain path."""
    B, n, hq, hkv, d, T = 2, 24, 8, 2, 128, 160
    qkv, slots, pos, _, w, _, kp, vp, ns = _step(B, n, hq, hkv, d, T, 100, True)
    rope, _, _ = _rope(128, True)
    desc, gs, st = _desc(hq, hkv, d, BF16), dev(slots), _status()
    pool = [torch.zeros((ns, hkv, x), dtype=torch.uint8, device="cuda") for x in (d, d, 2)]
    every = torch.arange(ns, dtype=torch.int32, device="cuda")
    ac.acache_write_slots_q8(desc, 1, ns, every, dev(kp), dev(vp), *pool, ns, 0, dev_status=st)
    new_slots = gs[:, T - n:].contiguous()
    q, k, v = dev(qkv).split((hq, hkv, hkv), 2)
    qo, out, ref = (torch.empty((B, n, hq, d), dtype=BF16, device="cuda") for _ in range(3))
    ac.acache_rotate_store_q8(desc, rope, B, n, dev(pos), new_slots, q, k, v, qo, *pool, ns, 0, q_weight=dev(w), k_weight=dev(w), dev_status=st)
    ac.acache_slot_attention_q8(desc, B, n, qo, T, gs, *pool, ns, out, dev_status=st)
    # the same keys read back to 16 bits (exact), under no mask
    k16, v16 = (torch.empty((B, T, hkv, d), dtype=BF16, device="cuda") for _ in range(2))
    ac.acache_gather_slots_q8(desc, B, T, gs, *pool, ns, k16, v16, dev_status=st)
    rows = torch.arange(B * T, dtype=torch.int32, device="cuda").view(B, T)
    ac.acache_slot_attention_masked(desc, B, n, qo, T, rows, k16, v16, B * T, ref, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for b in range(B):
        want, tol = masked_attention(qo[b].cpu(), np.arange(T), k16[b].cpu(), v16[b].cpu(), d ** -0.5, [0] * n, [T] * n)
        assert_attention(_np(ref[b]), want, tol)
        # the 8-bit kernels carry queries to 2^-17 of the row's largest
        assert_attention(_np(out[b]), want, 2 * tol + 2.0 ** -10)


def test_tensors_on_the_host_are_refused():
    d, r = _desc(4, 2, 128, BF16), _rope(128, False)[0]
    x, k = (torch.zeros((2, h, 128), dtype=BF16, device="cuda") for h in (4, 2))
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        ac.acache_rotate_qk(d, r, 2, pos.cpu(), x, k, x, k)
    with pytest.raises(ValueError):
        ac.acache_slot_attention_masked(d, 1, 2, x, 2, pos, k, k, 2, x, row_range=torch.zeros((1, 2, 2), dtype=torch.int32))
    with pytest.raises(ValueError):
        ac.acache_token_scores(2, 128, x[:, 0].float(), entropy=torch.zeros(2))


@pytest.mark.parametrize("n", [40, 300])
@pytest.mark.parametrize("size", [4.0, 30.0, 300.0])
def test_scores_that_jump_between_tiles(n, size):
    """Scores that rise by up to hundreds from one tile of keys to the next, and rows whose first key is far below
    the others: what the softmax is taken against has to keep up."""
    g = torch.Generator().manual_seed(int(size))
    hq, hkv, d, T = 2, 1, 128, 700
    q = torch.randn((1, n, hq, d), generator=g)
    q[..., 0] = 1.0 * d ** 0.5
    kp, vp = (torch.randn((T, hkv, d), generator=g) * 0.2 for _ in range(2))
    t = torch.arange(T)
    kp[:, 0, 0] = size * torch.tensor([-1.0, 0.0, 1.0, -0.5, 2.0, 0.5])[t // 128]
    kp[0, 0, 0] = -2 * size
    kp[127, 0, 0] = -2 * size
    q, kp, vp = q.to(BF16), kp.to(BF16), vp.to(BF16)
    lo = torch.randint(0, 3, (n,), generator=g) * 127
    hi = torch.randint(200, T + 1, (n,), generator=g)
    out, st = torch.empty((1, n, hq, d), dtype=BF16, device="cuda"), _status()
    rs = t.to(torch.int32)[None]
    ac.acache_slot_attention_masked(_desc(hq, hkv, d, BF16), 1, n, dev(q), T, dev(rs), dev(kp), dev(vp), T, out,
                                    row_range=dev(torch.stack((lo, hi), -1).to(torch.int32)[None]), dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    want, tol = masked_attention(q[0], rs[0].numpy(), kp, vp, d ** -0.5, lo, hi)
    assert_attention(_np(out[0]), want, tol)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 128)])
@pytest.mark.parametrize("n", [1, 20, 150])
def test_rows_whose_scores_are_all_minus_infinity(dtype, d, n):
    """A softmax over keys that all score -infinity is 0 / 0; over no key it is zeros."""
    g = torch.Generator().manual_seed(n)
    T = 200
    q = torch.rand((1, n, 2, d), generator=g).to(dtype) + 0.5
    kp, vp = (torch.randn((T, 1, d), generator=g).to(dtype) for _ in range(2))
    kp[:, 0, 0] = -INF
    kp[150, 0, 0] = 1.0
    lo = torch.zeros(n, dtype=torch.int32)
    hi = torch.where(torch.arange(n) % 3 == 0, 150, torch.where(torch.arange(n) % 3 == 1, 200, 0)).to(torch.int32)
    out = torch.empty((1, n, 2, d), dtype=dtype, device="cuda")
    ac.acache_slot_attention_masked(_desc(2, 1, d, dtype), 1, n, dev(q), T, dev(torch.arange(T, dtype=torch.int32)[None]), dev(kp), dev(vp), T,
                                    out, row_range=dev(torch.stack((lo, hi), -1)[None]))
    torch.cuda.synchronize()
    o = out[0].float().cpu()
    assert o[::3].isnan().all()
    assert torch.equal(o[1::3], vp[150].float().expand_as(o[1::3])) and (o[2::3] == 0).all()


@pytest.mark.parametrize("n,cap", [(600, 0.0), (600, 30.0), (20, 0.0)])
def test_masked_waits_that_run_out(n, cap):
    """Waits of the tensor-core kernel that run out: flagged, no row is written that lacks a product, and the same call
    with the default budget gives what it gave before."""
    g = torch.Generator().manual_seed(n)
    B, hq, hkv, d, T = 8, 32, 8, 128, 1500
    q = torch.randn((B, n, hq, d), generator=g).to(BF16)
    kp, vp = (torch.randn((T, hkv, d), generator=g).to(BF16) for _ in range(2))
    rs = torch.randperm(T, generator=g).to(torch.int32).expand(B, T)
    args = (_desc(hq, hkv, d, BF16), B, n, dev(q), T, dev(rs), dev(kp), dev(vp), T)
    rr = torch.stack((torch.zeros(n, dtype=torch.int32), torch.arange(T - n + 1, T + 1, dtype=torch.int32)), -1)
    rr = dev(rr.expand(B, n, 2))

    def call():
        out, st = torch.full((B, n, hq, d), 7.0, dtype=BF16, device="cuda"), _status()
        ac.acache_slot_attention_masked(*args, out, row_range=rr, softcap=cap, dev_status=st)
        torch.cuda.synchronize()
        return out, st.item()

    want, st = call()
    assert st == 0
    timed_out = 0
    for budget in (1, 300, 1000, 2000, 4000, 8000):
        prev = ac.acache_wait_budget(budget)
        try:
            out, st = call()
        finally:
            ac.acache_wait_budget(prev)
        assert st in (0, _lib.DEV_TIMEOUT)
        timed_out += st != 0
        same = (out == want).all(-1)
        assert (same | (out == 7.0).all(-1)).all()
        assert st != 0 or same.all()
    assert timed_out
    out, st = call()
    assert st == 0 and torch.equal(out, want)


def test_calls_on_two_streams_at_once():
    """The calls hold nothing between them: two streams in turn give what one gives."""
    g = torch.Generator().manual_seed(21)
    hq, hkv, d, T, n = 8, 2, 128, 600, 64
    kp, vp = (torch.randn((T, hkv, d), generator=g).to(BF16).cuda() for _ in range(2))
    rs = dev(torch.randperm(T, generator=g).to(torch.int32)[None])
    qs = [torch.randn((1, n, hq, d), generator=g).to(BF16).cuda() for _ in range(4)]
    xs = [torch.randn((40, 70001), generator=g).cuda() for _ in range(4)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    results = []
    for two in (False, True):
        torch.cuda.synchronize()
        got = []
        for i in range(4):
            with torch.cuda.stream(streams[i & 1] if two else streams[0]):
                o, tt, tl = torch.empty_like(qs[i]), torch.empty((40, 20), dtype=torch.int32, device="cuda"), torch.empty((40, 20), device="cuda")
                ac.acache_slot_attention_masked(_desc(hq, hkv, d, BF16), 1, n, qs[i], T, rs, kp, vp, T, o, softcap=9.0)
                ac.acache_token_scores(40, 70001, xs[i], top_tokens=tt, top_logprob=tl)
                got += [o, tt, tl]
        torch.cuda.synchronize()
        results.append(got)
    assert all(torch.equal(a, b) for a, b in zip(*results))

"""Corners of the steps around the attention on the GPU: temperatures and logits at the ends of float32, sums of softmax
weights at its end, caps far from the scale, and buffers wider than the rows that a call takes of them."""
import numpy as np
import pytest
import torch

import affix_kv_cache_gb300 as ac

from gpu_helpers import dev
from q8_reference import assert_attention
from step_reference import masked_attention, token_scores

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
INF = float("inf")


def _desc(hq, hkv, d, dtype, scale=None):
    return ac.attn_desc(hq, hkv, d, d ** -0.5 if scale is None else scale, dtype)


def _np(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------------------------- token scores
def _check_extreme(x, k, temperature, on=None):
    """Scores whose log probabilities may lie beyond float32 (then they are -infinity); the given tokens are the likeliest."""
    T = float(np.float32(temperature))
    R, V = x.shape
    lp, H, order, tol, tol_h = token_scores(x, T)
    with np.errstate(over="ignore"):
        lp = lp.astype(np.float32).astype(np.float64)
    first = np.ascontiguousarray(order[:, 0]).astype(np.int32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    given, ent = torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
    tt, tl = torch.empty((R, k), dtype=torch.int32, device="cuda"), torch.empty((R, k), device="cuda")
    ac.acache_token_scores(R, V, dev(x) if on is None else on, tokens=dev(torch.from_numpy(first)), token_logprob=given, entropy=ent, top_tokens=tt,
                           top_logprob=tl, temperature=T, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    assert np.array_equal(tt.cpu().numpy(), order[:, :k])
    at = np.arange(R)
    for got, want, bound in ((_np(ent), H, tol_h), (_np(given), lp[at, first], tol[at, first]),
                             (_np(tl), np.take_along_axis(lp, order[:, :k], 1), np.take_along_axis(tol, order[:, :k], 1))):
        assert not np.isnan(got).any()
        with np.errstate(invalid="ignore"):
            assert not (np.where(got == want, 0.0, np.abs(got - want)) > bound).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [8, 13, 1003, 5000, 70001])
@pytest.mark.parametrize("top,temperature", [(200.0, 1.18e-38), (-200.0, 1.18e-38), (1e30, 1e-6), (3.38e38, 0.01), (-3.3e38, 0.01)])
def test_scores_of_logits_far_from_the_temperature(dtype, V, top, temperature):
    """The largest logit over the temperature lies beyond float32: the weights are those of the largest ones alone."""
    g = torch.Generator().manual_seed(V)
    x = torch.randn((5, V), generator=g).abs().clamp(0.1, 3.0) * -0.25 * abs(top) + top
    x = x.clamp(-3.3e38, 3.3e38).to(dtype)
    at = torch.randint(0, V, (5, 3), generator=g)
    for r in range(5):                                  # one to three that are the largest
        x[r, at[r, :1 + r % 3]] = top
    x[4, V // 2 + 1:] = -INF
    _check_extreme(x, min(3, V), temperature)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [8, 13, 1003, 5000, 70001])
@pytest.mark.parametrize("temperature", [3e37, 1e38, 3.4e38])
def test_scores_of_logits_whose_differences_leave_float32(dtype, V, temperature):
    """Logits at both ends of float32 over a temperature of their size: the differences divided by it are small numbers."""
    g = torch.Generator().manual_seed(V)
    x = (torch.rand((5, V), generator=g) * 2 - 1) * 3.3e38
    x[1] = x[1].abs() * -1.0
    x[1, V // 2] = 3.3e38                                # one far above the others
    x[2, ::2] = -INF
    x[3] = torch.where(x[3] > 0, 3.3e38, -3.3e38)
    _check_extreme(x.to(dtype), min(5, V), temperature)


# ------------------------------------------------------------------------------------- masked attention
def _attend(n, T, hq, k, v, q, scale, cap=0.0):
    """All rows see all keys, slots in order."""
    d = q.shape[-1]
    out, st = torch.full((1, n, hq, d), 7.0, dtype=q.dtype, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    rr = torch.tensor([0, T], dtype=torch.int32).expand(1, n, 2).contiguous()
    ac.acache_slot_attention_masked(_desc(hq, k.shape[1], d, q.dtype, scale), 1, n, dev(q), T,
                                    dev(torch.arange(T, dtype=torch.int32)[None]), dev(k), dev(v), T, out, row_range=dev(rr),
                                    softcap=cap, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    want, tol = masked_attention(q[0], np.arange(T), k, v, scale, [0] * n, [T] * n, cap=cap)
    assert_attention(_np(out[0]), want, tol)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,T", [(40, 512), (200, 512), (40, 3328), (200, 3328)])
@pytest.mark.parametrize("size", [0.25, 1.0, 3.0])
def test_sums_of_weights_at_the_end_of_float32(d, n, T, size):
    """Scores 120 powers of two above the first tile's in a tile behind which nothing raises the reference, in every chain
    and every CTA that shares the keys: each sum of weights is below 2^128, all of them together are not."""
    g = torch.Generator().manual_seed(T + n)
    q = torch.zeros((1, n, 1, d))
    q[..., 0] = 8.0
    q[..., 1:] = 0.01 * torch.randn((1, n, 1, d - 1), generator=g)
    k = 0.01 * torch.randn((T, 1, d), generator=g)
    tile = torch.arange(T) // 128
    k[:, 0, 0] = 0.0
    parts = 8 if T == 3328 else 1
    n_all = T // 128
    high = []
    for r in range(parts):                              # the last tiles of a part's chains, as the kernel lays them out
        j0, j1 = n_all * r // parts, n_all * (r + 1) // parts
        high += [j1 - 1] if n > 128 else [j0 + (j1 - j0 + 1) // 2 - 1, j1 - 1]
    for j in high:
        k[tile == j, 0, 0] = 10.4375                    # 83.5 = 120.46 ln 2
    v = size * (1.0 + 0.5 * torch.rand((T, 1, d), generator=g))
    _attend(n, T, 1, k.to(BF16), v.to(BF16), q.to(BF16), 1.0)


@pytest.mark.parametrize("n", [1, 40, 300])
@pytest.mark.parametrize("scale,cap", [(2.0 ** -20, 1e38), (2.0 ** -12, 2e38), (1e-3, 1e37)])
def test_caps_whose_quotient_with_the_scale_is_next_to_nothing(n, scale, cap):
    """2 log2e scale / cap is a float32 number of few bits or none: the score is the uncapped one."""
    g = torch.Generator().manual_seed(n)
    d, T = 128, 300
    q = (torch.randn((1, n, 2, d), generator=g) * (0.2 / scale) ** 0.5).to(BF16)
    k, v = ((torch.randn((T, 1, d), generator=g) * s).to(BF16) for s in ((0.2 / scale) ** 0.5, 1.0))
    _attend(n, T, 2, k, v, q, scale, cap)


# ------------------------------------------------------------------------------------- buffers wider than the rows
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", [(6, 1088), (2, 3, 1088), (6, 1003), (8, 1024)])
def test_scores_of_a_padded_buffer(dtype, shape):
    """The whole buffer of a padded LM head is handed over: its rows lie as far apart as it says."""
    R, V = 6, 1003
    x = torch.randn(shape, generator=torch.Generator().manual_seed(shape[-1])).to(dtype)
    x[..., V:] = 1000.0
    _check_extreme(x.view(-1, shape[-1])[:R, :V], 4, 0.7, on=dev(x))


def test_rotation_of_a_whole_fused_buffer():
    """The queries of rows of queries, keys and values, unsliced: the first heads of each row."""
    g = torch.Generator().manual_seed(3)
    B, n, hq, hkv, d = 2, 5, 4, 2, 128
    qkv = torch.randn((B, n, hq + 2 * hkv, d), generator=g).to(BF16).cuda()
    q, k, v = qkv.split((hq, hkv, hkv), 2)
    pos = torch.arange(B * n, dtype=torch.int32, device="cuda") * 100
    rope, desc = ac.rope_desc(d), _desc(hq, hkv, d, BF16)
    want, got = (torch.empty((B, n, hq, d), dtype=BF16, device="cuda") for _ in range(2))
    wide = torch.full((B, n, hq + 3, d), 7.0, dtype=BF16, device="cuda")
    ac.acache_rotate_qk(desc, rope, B * n, pos, q.contiguous(), None, want, None)
    ac.acache_rotate_qk(desc, rope, B * n, pos, qkv, None, got, None)
    ac.acache_rotate_qk(desc, rope, B * n, pos, q, None, wide, None)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(wide[:, :, :hq], want) and (wide[:, :, hq:] == 7).all()
    pools = [[torch.zeros((B * n, hkv, d), dtype=BF16, device="cuda") for _ in range(2)] for _ in range(2)]
    slots = torch.arange(B * n, dtype=torch.int32, device="cuda")
    ac.acache_rotate_store(desc, rope, B, n, pos, slots, qkv, k, v, got, *pools[0], B * n, 0)
    ac.acache_rotate_store(desc, rope, B, n, pos, slots, *(x.contiguous() for x in (q, k, v)), want, *pools[1], B * n, 0)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(*pools))


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("n", [1, 7])
def test_rotation_into_the_gaps_between_its_rows(first, n):
    """Rows before and after the rotation side by side in one buffer."""
    g = torch.Generator().manual_seed(n)
    hq, hkv, d = 4, 2, 64
    buf = torch.randn((n, 2 * (hq + hkv), d), generator=g).to(BF16).cuda()
    keep = buf.clone()
    half = slice(0, hq + hkv), slice(hq + hkv, None)
    x, y = (buf[:, half[not first]], buf[:, half[first]])
    pos, rope, desc = torch.arange(n, dtype=torch.int32, device="cuda") + 5, ac.rope_desc(d), _desc(hq, hkv, d, BF16)
    want = [x[:, :hq].clone(), x[:, hq:].clone()]
    ac.acache_rotate_qk(desc, rope, n, pos, *want, *want)
    ac.acache_rotate_qk(desc, rope, n, pos, x[:, :hq], x[:, hq:], y[:, :hq], y[:, hq:])
    torch.cuda.synchronize()
    assert torch.equal(y[:, :hq], want[0]) and torch.equal(y[:, hq:], want[1])
    assert torch.equal(x, keep[:, half[not first]])
    if n > 1:                                            # an output that shares a head with its input
        with pytest.raises(ac.AcacheError):
            ac.acache_rotate_qk(desc, rope, n, pos, buf[:, 1:1 + hq], None, buf[:, :hq], None)


# ------------------------------------------------------------------------------------- few rows over many keys
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,hkv", [(2, 8), (17, 1), (10, 2), (21, 1), (3, 8), (4, 8), (5, 8), (1, 3)])
def test_single_tokens_split_over_clusters_of_any_size(d, B, hkv):
    """From 3 to 40 (request, KV head) units over 1,500 keys: clusters of 6 to 16 CTAs, as many as run at once."""
    g = torch.Generator().manual_seed(B + hkv)
    T, hq = 1500, 2 * hkv
    ns = B * T
    q = torch.randn((B, 1, hq, d), generator=g).to(BF16)
    k, v = (torch.randn((ns, hkv, d), generator=g).to(BF16) for _ in range(2))
    rs = torch.randperm(ns, generator=g).to(torch.int32).view(B, T)
    lo = torch.randint(0, 700, (B,), generator=g)
    hi = torch.randint(600, T + 1, (B,), generator=g)
    out, st = torch.full((B, 1, hq, d), 7.0, dtype=BF16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ac.acache_slot_attention_masked(_desc(hq, hkv, d, BF16), B, 1, dev(q), T, dev(rs), dev(k), dev(v), ns, out,
                                    row_range=dev(torch.stack((lo, hi), -1).to(torch.int32)[:, None]), dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for b in range(B):
        want, tol = masked_attention(q[b], rs[b].numpy(), k, v, d ** -0.5, lo[b:b + 1], hi[b:b + 1])
        assert_attention(_np(out[b]), want, tol, f"request {b}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,hkv", [(4, 8), (16, 4), (33, 8)])
def test_ragged_single_tokens_split_over_clusters(d, B, hkv):
    g = torch.Generator().manual_seed(B)
    hq = 2 * hkv
    keys = [2000] + [int(2000 ** x) for x in torch.rand(B - 1, generator=g).tolist()]
    ks = np.concatenate(([0], np.cumsum(keys))).astype(np.int32)
    ns = int(ks[-1])
    q = torch.randn((B, hq, d), generator=g).to(BF16)
    k, v = (torch.randn((ns, hkv, d), generator=g).to(BF16) for _ in range(2))
    rs = torch.randperm(ns, generator=g).to(torch.int32)
    out, st = torch.full((B, hq, d), 7.0, dtype=BF16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ac.acache_slot_attention_masked_varlen(_desc(hq, hkv, d, BF16), B, dev(torch.arange(B + 1, dtype=torch.int32)), 1, B, dev(q),
                                           dev(torch.from_numpy(ks)), 2000, dev(rs), dev(k), dev(v), ns, out, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for b in range(B):
        want, tol = masked_attention(q[b:b + 1], rs[ks[b]:ks[b + 1]].numpy(), k, v, d ** -0.5, [0], [keys[b]])
        assert_attention(_np(out[b:b + 1]), want, tol, f"request {b}")

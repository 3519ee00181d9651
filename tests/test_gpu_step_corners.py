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
def _check_extreme(x, k, temperature):
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
    ac.acache_token_scores(R, V, dev(x), tokens=dev(torch.from_numpy(first)), token_logprob=given, entropy=ent, top_tokens=tt,
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

"""Outputs of the rotation and of the rotating stores that would be written over one another or over an input are refused
before anything is launched."""
import ctypes

import pytest

import affix_kv_cache_gb300 as ac
from affix_kv_cache_gb300 import _lib

AT, FAR, E = 1 << 40, 1 << 30, _lib.ACACHE_ERR_INVALID_ARG
D, HEAD = 128, 256                        # elements and bytes of a bf16 head


def _rotate(rows, q, qs, k, ks, qo, qos, ko, kos, hq=4, hkv=2):
    d = ac.attn_desc(hq, hkv, D, 0.1, "bf16")
    return ac.lib().acache_rotate_qk(ctypes.byref(d), None, rows, None, q, qs * D, k, ks * D, None, None, 1e-6, qo, qos * D, ko, kos * D,
                                     None)


@pytest.mark.parametrize("rows", [1, 5])
def test_outputs_across_one_another_and_across_inputs(rows):
    # rows of 12 heads: queries at 0, keys at 4, and free ones from 6 on
    q, k, free, w = AT, AT + 4 * HEAD, AT + 6 * HEAD, 12
    for qo, ko in ((k, free), (k + HEAD, free), (free, q), (free, q + 2 * HEAD), (free, free), (free, free + 3 * HEAD),
                   (free + 3 * HEAD, free + 2 * HEAD), (q, free - HEAD), (q, q)):
        assert _rotate(rows, q, w, k, w, qo, w, ko, w) == E, (qo - q, ko - q)
    # a row further on, where the gap of the row before would have room for part of the output only
    assert _rotate(5, q, w, k, w, AT + 9 * HEAD, w, AT + FAR, w) == E
    assert _rotate(5, q, w, k, w, AT + 2 * w * HEAD + 4 * HEAD, w, AT + FAR, w) == E


@pytest.mark.parametrize("q8", [False, True])
def test_queries_of_a_store_across_the_keys_and_values(q8):
    hq, hkv = 4, 4
    d = ac.attn_desc(hq, hkv, D, 0.1, "bf16")

    def store(q, k, v, qo, rows=3, s=4 * D):
        far = [AT + i * FAR for i in range(8, 12)]
        pool = far[:2] + ([far[2]] if q8 else [])
        f = ac.lib().acache_rotate_store_q8 if q8 else ac.lib().acache_rotate_store
        return f(ctypes.byref(d), None, 1, rows, None, far[3], q, s, k, s, v, s, None, None, 1e-6, qo, *pool, 10, 0, None, None)

    q, k, v = AT, AT + FAR, AT + 2 * FAR
    for qo in (k, v, k + HEAD, v - HEAD):
        assert store(q, k, v, qo) == E
    assert store(q, k, v, k, rows=1, s=12 * D) == E

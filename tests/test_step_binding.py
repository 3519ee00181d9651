"""What the binding of the steps around the attention hands on: strides of tensors that are wider than the rows a call
takes of them, and refusals of tensors that do not lie as the call reads them.  A stand-in for the library records the
arguments; nothing is launched."""
import pytest
import torch

import affix_kv_cache_gb300 as ac
from affix_kv_cache_gb300 import _lib

BF16 = torch.bfloat16


class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def calls(monkeypatch):
    """Calls that reach the library, as (name, arguments); tensors on the host pass for the current device's."""
    lib = _Recorder()
    monkeypatch.setattr(_lib, "lib", lambda: lib)
    monkeypatch.setattr(_lib, "_current_device", lambda: -1)
    monkeypatch.setattr(_lib, "_stream", lambda *a: None)
    return lib.calls


# ------------------------------------------------------------------------------------- logits
SCORE_STRIDE = 4                              # of acache_token_scores(dtype, rows, vocab, logits, row_stride, ...)


@pytest.mark.parametrize("shape,rows,vocab,want", [
    ((6, 100), 6, 100, 100), ((6, 128), 6, 100, 128), ((6, 128), 4, 100, 128), ((2, 3, 128), 6, 100, 128), ((2, 3, 128), 5, 128, 128),
    ((1, 128), 1, 100, 100), ((600,), 6, 100, 100), ((700,), 6, 100, 100), ((3, 200), 6, 100, 100), ((128,), 1, 100, 100)])
def test_logits_in_a_buffer_wider_than_the_vocabulary(calls, shape, rows, vocab, want):
    ac.acache_token_scores(rows, vocab, torch.zeros(shape), entropy=torch.zeros(rows))
    got = calls[0][1][SCORE_STRIDE]
    assert got == want or (rows == 1 and got >= vocab)


def test_logits_that_are_slices(calls):
    buf = torch.zeros(2, 6, 128)
    for x, rows, want in ((buf[0, :, :100], 6, 128), (buf[:, :, :100], 12, 128), (buf[:, 2, :100], 2, 768), (buf[:, 2], 2, 768),
                          (buf[0, ::2, 5:105], 3, 256)):
        calls.clear()
        ac.acache_token_scores(rows, 100, x, entropy=torch.zeros(rows))
        assert calls[0][1][SCORE_STRIDE] == want


@pytest.mark.parametrize("shape,rows,vocab", [((6, 90), 6, 100), ((5, 100), 6, 100), ((5, 128), 6, 100), ((90,), 1, 100), ((590,), 6, 100),
                                              ((2, 2, 128), 6, 100)])
def test_logits_of_too_few_rows_or_tokens_are_refused(calls, shape, rows, vocab):
    with pytest.raises(ValueError):
        ac.acache_token_scores(rows, vocab, torch.zeros(shape), entropy=torch.zeros(rows))
    assert not calls


# ------------------------------------------------------------------------------------- rows of heads
HQ, HKV, D = 4, 2, 128


def _desc():
    return ac.attn_desc(HQ, HKV, D, 0.1, "bf16")


def _rows(*shape):
    return torch.zeros(shape, dtype=BF16)


def _rotate(q, k, rows=6, q_out=None, k_out=None):
    ac.acache_rotate_qk(_desc(), None, rows, None, q, k, _rows(rows, HQ, D) if q_out is None else q_out,
                        _rows(rows, HKV, D) if k_out is None else k_out)


def _strides(args):
    """q, k, q_out, k_out of acache_rotate_qk(desc, rope, rows, positions, q, stride, k, stride, weights, eps, ...)."""
    return args[5], args[7], args[12], args[14]


@pytest.mark.parametrize("shape,rows,want", [
    ((6, HQ, D), 6, 512), ((2, 3, HQ, D), 6, 512), ((6, 8, D), 6, 1024), ((2, 3, 8, D), 6, 1024), ((2, 3, 8, D), 5, 1024),
    ((9, HQ, D), 6, 512), ((6, HQ * D), 6, 512), ((9, HQ * D), 6, 512), ((6 * HQ, D), 6, 512), ((2, 3 * HQ, D), 6, 512),
    ((6 * HQ * D,), 6, 512), ((7 * HQ * D,), 6, 512), ((1, 2, 3, 8, D), 6, 1024)])
def test_rows_in_a_buffer_of_more_heads(calls, shape, rows, want):
    """A whole fused projection in place of its slice of queries, and dense rows of any shape."""
    _rotate(_rows(*shape), None, rows)
    assert _strides(calls[0][1])[0] == want
    calls.clear()
    _rotate(None, None, rows, q_out=_rows(*shape))
    assert _strides(calls[0][1])[2] == want


def test_rows_of_every_matrix(calls):
    qkv, out = _rows(2, 3, HQ + 2 * HKV, D), _rows(2, 3, 2 * HQ, D)
    q, k, v = qkv.split((HQ, HKV, HKV), 2)
    _rotate(qkv, k, 6, out, out[:, :, HQ:HQ + HKV])
    assert _strides(calls[0][1]) == (1024, 1024, 1024, 1024)
    for call in (ac.acache_rotate_store, ac.acache_rotate_store_q8):
        calls.clear()
        pool = [_rows(9, HKV, D)] * (2 if call is ac.acache_rotate_store else 3)
        call(_desc(), None, 2, 3, None, torch.zeros(6, dtype=torch.int32), qkv, k, _rows(6, 5, D), _rows(6, HQ, D), *pool, 9, 0)
        a = calls[0][1]
        assert (a[7], a[9], a[11]) == (1024, 1024, 640)


@pytest.mark.parametrize("shape", [(6, HQ, D + 16), (6, HQ - 1, D + 8), (5, HQ, D), (2, 2, HQ, D), (5, 2 * HQ * D), (6, 2 * HQ * D)])
def test_rows_that_are_too_few_or_lie_otherwise_are_refused(calls, shape):
    with pytest.raises(ValueError):
        _rotate(_rows(*shape), None)
    with pytest.raises(ValueError):
        _rotate(None, None, q_out=_rows(*shape))
    assert not calls


@pytest.mark.parametrize("call", [ac.acache_rotate_store, ac.acache_rotate_store_q8])
def test_queries_of_a_store_come_out_dense(calls, call):
    """The stores write q_out as [rows][Hq][d]: rows that lie further apart are refused, not written in between."""
    pool = [_rows(9, HKV, D)] * (2 if call is ac.acache_rotate_store else 3)

    def store(batch, rows, q, q_out):
        call(_desc(), None, batch, rows, None, torch.zeros(batch * rows, dtype=torch.int32), q, _rows(batch, rows, HKV, D),
             _rows(batch, rows, HKV, D), q_out, *pool, 9, 0)

    wide = _rows(2, 3, HQ + 2, D)
    for q_out in (wide[:, :, :HQ], wide, _rows(6, HQ + 1, D), _rows(2, 6, HQ, D)[:, ::2], _rows(5, HQ, D)):
        with pytest.raises(ValueError):
            store(2, 3, _rows(2, 3, HQ, D), q_out)
    assert not calls
    for q_out in (_rows(2, 3, HQ, D), _rows(6, HQ * D), _rows(8, HQ, D)):
        store(2, 3, _rows(2, 3, HQ, D), q_out)
    store(1, 1, _rows(1, 1, HQ, D), wide[:1, :1, :HQ])             # a single row has no next one
    store(2, 3, None, wide[:, :, :HQ])                             # no queries: not used
    assert len(calls) == 5


# ------------------------------------------------------------------------------------- everything else is dense
def _apart(t):
    """The same shape and values with gaps between the elements."""
    return torch.stack((t, t), -1)[..., 0]


def _calls():
    """(name, call, arguments by name) of every call that takes tensors as one dense block."""
    i32 = torch.int32
    pos, slot, w = torch.zeros(6, dtype=i32), torch.zeros(6, dtype=i32), torch.zeros(D, dtype=BF16)
    q, k, v = _rows(2, 3, HQ, D), _rows(2, 3, HKV, D), _rows(2, 3, HKV, D)
    pool = dict(k_cache=_rows(9, HKV, D), v_cache=_rows(9, HKV, D), num_slots=9)
    turn = dict(desc=_desc(), rope=_lib.Rope(), positions=pos, q=q, k=k, q_weight=w, k_weight=w, q_out=_rows(2, 3, HQ, D))
    store = dict(turn, batch=2, rows=3, write_slot=slot, v=v, private_begin=0, **pool)
    mask = dict(row_range=torch.zeros((2, 3, 2), dtype=i32), q_pos=pos, slopes=torch.zeros(HQ))
    attend = dict(desc=_desc(), batch=2, q=q, read_slot=torch.zeros((2, 8), dtype=i32), out=_rows(2, 3, HQ, D), **pool, **mask)
    start = torch.zeros(3, dtype=i32)
    return [
        (ac.acache_rotate_qk, dict(turn, rows=6, k_out=_rows(2, 3, HKV, D)), ("positions", "q_weight", "k_weight")),
        (ac.acache_rotate_store, store, ("positions", "write_slot", "q_weight", "k_weight", "k_cache", "v_cache")),
        (ac.acache_rotate_store_q8, dict(store, kv_scale=torch.zeros(9, HKV, 2)), ("positions", "write_slot", "k_cache", "v_cache", "kv_scale")),
        (ac.acache_slot_attention_masked, dict(attend, n_q=3, seq_len=8),
         ("q", "read_slot", "k_cache", "v_cache", "out", "row_range", "q_pos", "slopes")),
        (ac.acache_slot_attention_masked_varlen, dict(attend, q_start=start, kv_start=start, max_q_rows=3, total_q_rows=6, max_seq_len=8),
         ("q", "read_slot", "q_start", "kv_start", "k_cache", "v_cache", "out", "row_range", "q_pos", "slopes")),
        (ac.acache_token_scores, dict(rows=6, vocab=50, logits=torch.zeros(6, 50), tokens=pos, token_logprob=torch.zeros(6),
                                      entropy=torch.zeros(6), top_tokens=torch.zeros((6, 4), dtype=i32), top_logprob=torch.zeros(6, 4), k=4),
         ("tokens", "token_logprob", "entropy", "top_tokens", "top_logprob"))]


@pytest.mark.parametrize("at", range(6))
def test_tensors_with_gaps_or_repeats_are_refused(calls, at):
    """A column of a wider tensor, or one row's positions expanded to a batch, does not lie as the kernels read it: they would
    take other values, or read behind its memory."""
    call, args, names = _calls()[at]
    call(**args)
    assert len(calls) == 1
    for name in names:
        for bad in (_apart(args[name]), args[name][:1].expand(args[name].shape)):
            with pytest.raises(ValueError):
                call(**dict(args, **{name: bad}))
        call(**dict(args, **{name: 1 << 40}))                       # a plain address is the caller's own
    assert len(calls) == 1 + len(names)


def test_alternatives_of_another_width_are_refused(calls):
    """The alternatives of a row follow those of the row before: k columns in each output."""
    i32, x = torch.int32, torch.zeros(6, 50)
    for tt, tl, k in (((6, 8), None, 4), ((6, 4), (6, 8), None), ((6, 4), (6, 2), 4), ((2, 3, 8), None, 4)):
        with pytest.raises(ValueError):
            ac.acache_token_scores(6, 50, x, top_tokens=torch.zeros(tt, dtype=i32), top_logprob=None if tl is None else torch.zeros(tl), k=k)
    assert not calls
    for tt, tl, k in (((6, 4), (6, 4), None), ((2, 3, 4), (6, 4), 4), ((24,), (24,), 4), ((8, 4), None, 4)):
        ac.acache_token_scores(6, 50, x, top_tokens=torch.zeros(tt, dtype=i32), top_logprob=None if tl is None else torch.zeros(tl), k=k)
    ac.acache_token_scores(1, 50, x[:1], top_tokens=torch.zeros((1, 32), dtype=i32), k=4)
    assert [c[1][9] for c in calls] == [4] * 5

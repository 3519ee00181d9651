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

"""Strided and expanded views at the serving entry points, on the CPU: the helpers that turn a
tensor's strides into those of the C ABI. There 0 stands for a dense tensor, so a tensor that is
expanded along its tokens or pages (stride 0, and the memory of one) must never get so far."""
import pytest
import torch

from gated_deltanet_mixer_causal_b200 import _lib


def test_token_strides():
    rows = lambda t, lead: _lib._token_rows(t, "x", lead)  # noqa: E731
    assert rows(torch.zeros(4, 2, 16), 1) == 0 and rows(torch.zeros(4, 3, 32), 2) == 0
    assert rows(torch.zeros(4, 48)[:, 16:].unflatten(1, (2, 16)), 1) == 48
    assert rows(torch.zeros(4, 3, 48)[:, :, :32], 2) == 48
    assert rows(torch.zeros(4, 3, 48)[:, :1, :32], 2) == 144          # one token a sequence
    assert rows(torch.zeros(1, 3, 48)[:, :, :32], 2) == 48
    # one token, whatever its strides say
    assert rows(torch.zeros(1, 1, 64)[:, :, ::1].expand(1, 1, 64), 2) == 0
    assert rows(torch.zeros(64).as_strided((1, 2, 16), (0, 16, 1)), 1) in (0, 32)


@pytest.mark.parametrize("t,lead", [
    (torch.zeros(1, 1, 64).expand(8, 1, 64), 2),                     # one token for many samples
    (torch.zeros(1, 1, 64).expand(8, 4, 64), 2), (torch.zeros(1, 1, 64).expand(1, 4, 64), 2),
    (torch.zeros(1, 2, 16).expand(5, 2, 16), 1),                     # one gate for all tokens
    (torch.zeros(2, 16).expand(2, 2, 16), 1),
    (torch.zeros(100).as_strided((4, 2, 16), (16, 16, 1)), 1),       # windows that overlap
    (torch.zeros(100).as_strided((2, 2, 32), (32, 16, 1)), 2), (torch.zeros(100).as_strided((2, 1, 32), (8, 8, 1)), 2),
])
def test_tokens_that_share_memory_are_refused(t, lead):
    with pytest.raises(ValueError, match="share memory"):
        _lib._token_rows(t, "x", lead)


def test_prefill_tokens_that_share_memory_are_refused():
    one = torch.zeros(1, 2, 16)
    with pytest.raises(ValueError, match="share memory"):
        _lib._row_view(one.expand(9, 2, 16), "q")
    assert _lib._row_view(one, "q") == 32 and _lib._row_view(torch.zeros(4, 64)[:, :32].unflatten(1, (2, 16)), "q") == 64


def test_pages_that_share_memory_are_refused():
    pool = torch.zeros(1, 2, 16)
    for t in (pool.expand(5, 2, 16), torch.zeros(99).as_strided((5, 2, 8), (8, 8, 1))):
        with pytest.raises(ValueError, match="share memory"):
            _lib._page_stride(t, "pool")
        with pytest.raises(ValueError, match="share memory"):
            _lib._pool_layout(t, "pool", 0)
    assert _lib._page_stride(torch.zeros(5, 40)[:, :32].unflatten(1, (2, 16)), "pool") == 40
    assert _lib._pool_layout(torch.zeros(5, 40)[:, :32], "pool", 0) == (5, 1, 128, 160, 0)
    many = torch.zeros(1, 1, 32)
    for t in (many.expand(3, 5, 32), torch.zeros(3, 1, 32).expand(3, 5, 32), torch.zeros(1, 5, 32).expand(3, 5, 32)):
        with pytest.raises(ValueError, match="share memory"):
            _lib._pool_layout(t, "pool", 1)
    layout = _lib._pool_layout(torch.zeros(5, 3, 32).movedim(1, 0), "pool", 1)      # [layers, P, page] by strides
    assert layout == (5, 3, 128, 384, 128)

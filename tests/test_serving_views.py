"""Strided and expanded views at the serving entry points, on the CPU: the helpers that turn a
tensor's strides into those of the C ABI. There 0 stands for a dense tensor, so a tensor that is
expanded along its tokens or pages (stride 0, and the memory of one) must never get so far."""
import ctypes
import random

import pytest
import torch

import gated_deltanet_mixer_causal_b200 as gdn
from gated_deltanet_mixer_causal_b200 import _lib
from gated_deltanet_mixer_causal_b200.build import build


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


# --------------------------------------------------------------------- pools in one buffer
#
# A call whose arguments pass every other check, but whose copy one launch cannot number (pages of
# 2^44 bytes, fake addresses), is refused as unsupported, before anything is launched.

UNIT = 1 << 44
BASE = 0x7f0000000000


def copied(first, second):
    """The status of a copy inside each of two pools (at, bytes, page, layer, layers in units), 5 pages each."""
    build()
    arr = (_lib._PagePool * 2)()
    for d, (at, size, page, layer, layers) in zip(arr, (first, second)):
        d.src = d.dst = BASE + at * UNIT
        d.page_bytes, d.layers = size * UNIT, layers
        d.src_page_stride = d.dst_page_stride = page * UNIT
        d.src_layer_stride = d.dst_layer_stride = layer * UNIT
    return _lib.lib().gdn_pages_copy(ctypes.addressof(arr), 2, 5, 5, 64, 128, 4, 1, None)


@pytest.mark.parametrize("first,second", [
    ((0, 1, 3, 0, 1), (1, 2, 3, 0, 1)),                    # a record a page: [taps | state]
    ((1, 2, 4, 0, 1), (0, 1, 4, 0, 1)),                    # the state first in the list, a gap behind
    ((0, 1, 3, 15, 2), (1, 2, 3, 15, 2)),                  # [layer][page][taps | state]
    ((0, 1, 6, 3, 2), (1, 2, 6, 3, 2)),                    # [page][layer][taps | state]
    ((0, 1, 6, 1, 2), (2, 2, 6, 2, 2)),                    # [page][taps of all layers | states of all layers]
    ((0, 1, 1, 15, 2), (5, 2, 2, 15, 2)),                  # [layer][taps of all pages | states of all pages]
    ((0, 1, 1, 5, 2), (10, 2, 2, 10, 2)),                  # one behind the other
])
def test_copy_takes_pools_that_share_a_buffer(first, second):
    assert copied(first, second) == _lib.GDN_ERR_UNSUPPORTED
    assert copied(second, first) == _lib.GDN_ERR_UNSUPPORTED


def test_copy_takes_no_pools_that_overlap():
    """Random layouts of two pools: what passes has no unit of memory in both."""
    rng, passed = random.Random(7), 0
    for _ in range(4000):
        page, layers = rng.randint(1, 8), rng.randint(1, 3)
        specs = []
        for _ in range(2):
            size = rng.randint(1, 3)
            p = page if rng.random() < 0.6 else rng.randint(size, 8)
            specs.append((rng.randint(0, 12), size, p, rng.choice([p * 5, page * 5, page, size, rng.randint(1, 40)]), layers))
        held = [{at + l * layer + p * stride + i for l in range(n) for p in range(5) for i in range(size)}
                for at, size, stride, layer, n in specs]
        status = copied(*specs)
        assert status in (_lib.GDN_ERR_INVALID_ARG, _lib.GDN_ERR_UNSUPPORTED)
        if status == _lib.GDN_ERR_UNSUPPORTED:
            assert not held[0] & held[1], specs
            passed += 1
    assert passed > 200


# ------------------------------------------------- forks and compactions that are refused
#
# The counts are changed before the pages are copied, so a call that the copy would refuse must end
# before its first launch. Without a GPU a launch fails with a CUDA error, so a refusal shows that
# none was tried; with one, the arguments below are all refused and none is launched either.

def refused(kind, *specs, P=8, n=3, refs=1 << 20, src=2 << 20, out=3 << 20, table=4 << 20):
    build()
    L = _lib.lib()
    arr = (_lib._PagePool * max(len(specs), 1))()
    for d, s in zip(arr, specs):
        v = dict(src=BASE, dst=BASE, page_bytes=4096, src_page_stride=0, src_layer_stride=0, dst_page_stride=0,
                 dst_layer_stride=0, layers=1)
        v.update(s)
        for k, x in v.items():
            setattr(d, k, x)
    at = ctypes.addressof(arr)
    if kind == "fork":
        return L.gdn_pages_fork(refs, P, src, n, out, at, len(specs), None)
    return L.gdn_pages_compact(refs, P, table, 4, src, out, 5 << 20, 6 << 20, at, len(specs), None)


@pytest.mark.parametrize("kind", ["fork", "compact"])
def test_refused_before_the_counts_change(kind):
    INVALID, UNSUPPORTED = _lib.GDN_ERR_INVALID_ARG, _lib.GDN_ERR_UNSUPPORTED
    far = BASE + (1 << 40)
    assert refused(kind, {}, {}) == INVALID                                   # one pool twice
    assert refused(kind, {}, dict(src=BASE + 4096, dst=BASE + 4096)) == INVALID
    assert refused(kind, dict(src=BASE + 8, dst=BASE + 8)) == INVALID and refused(kind, dict(page_bytes=40)) == INVALID
    assert refused(kind, dict(src=far)) == INVALID                            # from another pool
    assert refused(kind, dict(src=None, dst=None)) == INVALID and refused(kind) == INVALID
    assert refused(kind, dict(src_page_stride=64, dst_page_stride=64)) == INVALID
    assert refused(kind, dict(layers=2, src_layer_stride=16, dst_layer_stride=16)) == INVALID
    assert refused(kind, dict(page_bytes=UNIT)) == UNSUPPORTED                # too much for one launch
    assert refused(kind, dict(page_bytes=4 * UNIT)) == UNSUPPORTED            # 2^32 tiles
    assert refused(kind, {}, refs=BASE + 64) == INVALID and refused(kind, {}, src=BASE + 64) == INVALID
    assert refused(kind, {}, out=BASE + 64) == INVALID and refused(kind, {}, out=(1 << 20) + 4) == INVALID
    assert refused(kind, {}, refs=None) == INVALID and refused(kind, {}, src=None) == INVALID
    assert refused(kind, {}, out=None) == INVALID and refused(kind, {}, P=-1) == INVALID
    if kind == "fork":
        assert refused(kind, {}, n=2049) == UNSUPPORTED and refused(kind, {}, n=-1) == INVALID
        assert refused(kind, {}, n=0) == _lib.GDN_OK
    else:
        assert refused(kind, {}, table=BASE + 64) == INVALID and refused(kind, {}, table=(1 << 20) + 4) == INVALID
        # 4,096 entries in two parts of 64 groups each, 16 tiles a layer, and 992 more, 31 tiles a layer
        deep = dict(page_bytes=512, src_layer_stride=512 * 20000, dst_layer_stride=512 * 20000, layers=100_000_000)
        assert refused(kind, deep, P=2 * (4096 + 992), refs=1 << 58, src=1 << 59, out=3 << 58, table=5 << 58) == UNSUPPORTED


def test_gates_and_lists_need_only_their_own_alignment():
    """A slice of 10 heads' g begins on 8 bytes. The call goes on to the refusal behind the
    alignment (o lies in the conv's pool), so nothing is launched."""
    build()
    L = _lib.lib()
    at = lambda i, off=0: BASE + (i << 36) + off  # noqa: E731

    def call(g, beta, read):
        status = L.gdn_decode_paged(at(0), 0, at(1), at(2), 0, at(3), 0, 0, 16, read, None, None, g, beta, None, 0, None,
                                    1e-6, at(2), 1, 4, 2, 2, 10, 32, 32, 1.0, None)
        assert status == _lib.GDN_ERR_INVALID_ARG
        return L.gdn_last_error().decode()

    assert "overlaps" in call(at(5, 40), at(6, 40), at(4, 4))
    assert "aligned" in call(at(5, 42), at(6), at(4)) and "aligned" in call(at(5), at(6, 1), at(4))
    assert "aligned" in call(at(5), at(6), at(4, 2))


def test_counts_that_pass_32_bits():
    """Refused, where ctypes would pass on their lower half: 2^32 + 1 pages as one page."""
    i = torch.zeros(4, dtype=torch.int32)
    many = torch.empty((2 ** 32 + 1, 16), dtype=torch.uint8, device="meta")
    for call in (lambda: gdn.gdn_pages_ref(i, i, 2 ** 32 - 1), lambda: gdn.gdn_pages_take(i, n=2 ** 32 + 1),
                 lambda: _lib._pool_layout(many, "pool", 0), lambda: _lib._pool_layout(many[:, None], "pool", 1),
                 lambda: _lib._int32(2 ** 31, "n"), lambda: _lib._int32(-2 ** 31 - 1, "n")):
        with pytest.raises(ValueError, match="32 bits"):
            call()
    assert _lib._int32(2 ** 31 - 1, "n") == 2 ** 31 - 1


def test_counts_keep_within_their_range():
    """Entries times delta below 2^31: the sum of a page listed by all of them does not wrap."""
    build()
    ref = lambda n, delta: _lib.lib().gdn_pages_ref(None, 8, 64, n, delta, None)  # noqa: E731
    assert ref(2, -2 ** 31) == ref(2 ** 30, 2) == ref(3, 2 ** 30) == ref(1, -2 ** 31) == _lib.GDN_ERR_UNSUPPORTED
    assert ref(1, 2 ** 31 - 1) == ref(2 ** 31 - 1, -1) == _lib.GDN_ERR_INVALID_ARG     # on to the null counts

"""Host-side checks of the paged decode, the page operations and the norms that need no GPU:
invalid arguments come back as a status before any CUDA call, so fake addresses are safe here."""
import ctypes

import pytest
import torch

import gated_deltanet_mixer_causal_b200 as gdn
import serving_ref as R
from gated_deltanet_mixer_causal_b200 import _lib
from gated_deltanet_mixer_causal_b200.build import build

INVALID, UNSUPPORTED, WORKSPACE = _lib.GDN_ERR_INVALID_ARG, _lib.GDN_ERR_UNSUPPORTED, _lib.GDN_ERR_WORKSPACE
BASE = 0x7f0000000000
GB = 1 << 30


@pytest.fixture(scope="module")
def L():
    build()
    return _lib.lib()


def at(i, off=0):
    return BASE + i * 64 * GB + off


def paged(L, **kw):
    a = dict(x=at(0), xs=0, w=at(1), cp=at(2), cs=0, sp=at(3), ss=0, sdt=0, P=16, read=at(4), write=None, valid=None,
             g=at(5), b=at(6), z=None, zs=0, nw=None, eps=1e-6, o=at(7), dt=1, B=4, n=2, Hk=2, Hv=4, dk=32, dv=32)
    a.update(kw)
    return L.gdn_decode_paged(a["x"], a["xs"], a["w"], a["cp"], a["cs"], a["sp"], a["ss"], a["sdt"], a["P"], a["read"],
                              a["write"], a["valid"], a["g"], a["b"], a["z"], a["zs"], a["nw"], a["eps"], a["o"],
                              a["dt"], a["B"], a["n"], a["Hk"], a["Hv"], a["dk"], a["dv"], 1.0, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), UNSUPPORTED), (dict(sdt=5), UNSUPPORTED), (dict(B=-1), INVALID), (dict(n=0), INVALID),
    (dict(n=9), INVALID), (dict(Hk=0), INVALID), (dict(Hv=5), UNSUPPORTED), (dict(dk=24, dv=24), UNSUPPORTED),
    (dict(dk=64, dv=32), UNSUPPORTED), (dict(P=-1), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(xs=248), INVALID), (dict(xs=260), INVALID),                      # below a row of 256, not a multiple of 8
    (dict(cs=760), INVALID), (dict(ss=4100), INVALID), (dict(ss=4088), INVALID),
    (dict(x=None), INVALID), (dict(read=None), INVALID), (dict(sp=None), INVALID), (dict(o=None), INVALID),
    (dict(o=at(7, 8)), INVALID), (dict(x=at(0, 2)), INVALID), (dict(read=at(4, 2)), INVALID),
    (dict(z=at(8)), INVALID), (dict(nw=at(8)), INVALID),                   # one without the other
    (dict(z=at(8), nw=at(9), zs=120), INVALID),
    (dict(o=at(3, 4096)), INVALID), (dict(o=at(2)), INVALID), (dict(o=at(0, 512)), INVALID),
    (dict(sp=at(2, 1024)), INVALID),                                       # pools overlap
    (dict(x=at(3, 64)), INVALID), (dict(write=at(3, 4)), INVALID),         # an input inside a pool
    (dict(Hk=1, Hv=60, dk=128, dv=128, n=8), UNSUPPORTED),                 # shared memory
    (dict(B=1 << 30, Hk=4, Hv=4), INVALID),
    (dict(B=0), _lib.GDN_OK),
])
def test_paged_refusals(L, kw, status):
    assert paged(L, **kw) == status
    if status != _lib.GDN_OK:
        assert "decode_paged" in L.gdn_last_error().decode()


def test_paged_interleaved_pools_are_told_from_overlapping_ones(L):
    """One record a page, [taps | state]: bf16 taps of 768 and fp32 states of 4,096 elements. Equal
    strides in bytes and states behind the taps pass (to the launch, which has no GPU here)."""
    taps, state = 768 * 2, 4096 * 4
    step = taps + state
    ok = dict(cp=at(2), cs=step // 2, sp=at(2, taps), ss=step // 4)
    assert paged(L, **ok) != INVALID if not torch.cuda.is_available() else True
    assert paged(L, **{**ok, "sp": at(2, taps - 16)}) == INVALID
    assert paged(L, **{**ok, "cs": step // 2 + 8}) == INVALID
    assert paged(L, **{**ok, "sp": at(2, taps + 16)}) == INVALID           # runs into the next record


def pools(*specs):
    arr = (_lib._PagePool * len(specs))()
    for d, s in zip(arr, specs):
        v = dict(src=at(0), dst=at(0), page_bytes=4096, src_page_stride=0, src_layer_stride=0, dst_page_stride=0,
                 dst_layer_stride=0, layers=1)
        v.update(s)
        for k, x in v.items():
            setattr(d, k, x)
    return arr


def copy(L, *specs, sp=8, dp=8, src=at(5), dst=at(6), n=4, plain=0, n_pools=None):
    arr = pools(*specs)
    return L.gdn_pages_copy(ctypes.addressof(arr), len(specs) if n_pools is None else n_pools, sp, dp, src, dst, n, plain,
                            None)


@pytest.mark.parametrize("spec,kw,status", [
    (dict(page_bytes=0), {}, INVALID), (dict(page_bytes=40), {}, INVALID), (dict(layers=-1), {}, INVALID),
    (dict(src_page_stride=4000, dst_page_stride=4000), {}, INVALID),       # pages overlap
    (dict(src_page_stride=4104, dst_page_stride=4104), {}, INVALID),
    (dict(layers=2, src_layer_stride=4096, dst_layer_stride=4096), {}, INVALID),   # layers cross pages
    (dict(layers=2, src_layer_stride=8 * 4096, dst_layer_stride=8 * 4096 + 16), {}, INVALID),
    (dict(src=at(0, 8), dst=at(0, 8)), {}, INVALID), (dict(src=None), {}, INVALID),
    (dict(dst=at(0, 4096)), {}, INVALID),                                  # overlaps, not the same pool
    (dict(), dict(dp=9), INVALID), (dict(), dict(n=-1), INVALID), (dict(), dict(sp=-1), INVALID),
    (dict(), dict(n=2049), UNSUPPORTED), (dict(), dict(src=at(5, 2)), INVALID), (dict(), dict(src=None), INVALID),
    (dict(), dict(dst=at(0, 64)), INVALID),                                # the list lies in the pool
    (dict(), dict(n_pools=0), INVALID), (dict(), dict(n_pools=5), INVALID),
    (dict(), dict(n=0), _lib.GDN_OK), (dict(layers=0), {}, _lib.GDN_OK), (dict(), dict(sp=0, dp=0), _lib.GDN_OK),
])
def test_copy_refusals(L, spec, kw, status):
    assert copy(L, spec, **kw) == status


def test_copy_of_two_pools_that_overlap(L):
    assert copy(L, {}, dict(src=at(0, 4096), dst=at(0, 4096))) == INVALID
    assert "overlap" in L.gdn_last_error().decode()
    assert copy(L, {}, dict(src=at(0), dst=at(1))) == INVALID              # reads what the first pool writes


def test_counts_refusals(L):
    take = lambda refs=at(0), P=8, src=None, n=4, out=at(1): L.gdn_pages_take(refs, P, src, n, out, None)  # noqa: E731
    assert take(n=-1) == INVALID and take(P=-1) == INVALID and take(refs=None) == INVALID and take(out=None) == INVALID
    assert take(n=2049) == UNSUPPORTED and take(out=at(0, 8)) == INVALID and take(out=at(1, 2)) == INVALID
    assert take(src=at(1, 4)) == INVALID and take(n=0) == _lib.GDN_OK
    ref = lambda refs=at(0), P=8, pages=at(1), n=4: L.gdn_pages_ref(refs, P, pages, n, 1, None)  # noqa: E731
    assert ref(n=-1) == INVALID and ref(refs=None) == INVALID and ref(pages=at(0, 28)) == INVALID
    assert ref(n=0) == _lib.GDN_OK and ref(P=0) == _lib.GDN_OK
    plan = lambda refs=at(0), P=8, tab=at(1), nt=3, s=at(2), d=at(3), m=at(4), live=at(5): L.gdn_pages_plan(  # noqa: E731
        refs, P, tab, nt, s, d, m, live, None)
    assert plan(P=-1) == INVALID and plan(nt=-1) == INVALID and plan(tab=None) == INVALID and plan(live=None) == INVALID
    assert plan(m=at(0, 4)) == INVALID and plan(s=at(2), d=at(2, 8)) == INVALID and plan(live=at(1, 8)) == INVALID
    assert plan(refs=at(0, 1)) == INVALID


def gated(L, back=False, **kw):
    a = dict(o=at(0), z=at(1), zs=0, w=at(2), eps=1e-6, y=at(3), dy=at(4), do=at(5), dz=at(6), dzs=0, dw=at(7), dt=1, T=100,
             H=4, d=64, ws=at(8), wsb=1 << 20)
    a.update(kw)
    if not back:
        return L.gdn_gated_norm(a["o"], a["z"], a["zs"], a["w"], a["eps"], a["y"], a["dt"], a["T"], a["H"], a["d"], None)
    return L.gdn_gated_norm_bwd(a["o"], a["z"], a["zs"], a["w"], a["eps"], a["dy"], a["do"], a["dz"], a["dzs"], a["dw"],
                                a["dt"], a["T"], a["H"], a["d"], a["ws"], a["wsb"], None)


def test_gated_norm_refusals(L):
    for back in (False, True):
        r = lambda **kw: gated(L, back, **kw)  # noqa: E731
        assert r(dt=4) == UNSUPPORTED and r(d=48) == UNSUPPORTED and r(T=-1) == INVALID and r(H=0) == INVALID
        assert r(T=1 << 30, H=4) == UNSUPPORTED and r(eps=-1.0) == INVALID
        assert r(zs=248) == INVALID and r(zs=260) == INVALID and r(o=None) == INVALID and r(z=at(1, 4)) == INVALID
    assert gated(L, y=at(1, 64)) == INVALID and gated(L, y=at(0, 64)) == INVALID and gated(L, T=0) == _lib.GDN_OK
    assert gated(L, True, wsb=64) == WORKSPACE and gated(L, True, ws=None) == WORKSPACE
    assert gated(L, True, do=at(0)) == INVALID and gated(L, True, dz=at(5, 64)) == INVALID
    assert gated(L, True, dw=at(4)) == INVALID and gated(L, True, ws=at(7)) == INVALID and gated(L, True, dzs=12) == INVALID
    assert gated(L, True, T=0, dw=None) == _lib.GDN_OK


def add(L, back=False, **kw):
    a = dict(x=at(0), r=at(1), w=at(2), s=1.0, c=0.0, eps=1e-6, h=at(3), rdt=0, n=at(4), dt=1, T=100, D=1000, dn=at(5),
             dh=at(6), dres=at(7), dx=at(8), dw=at(9), ws=at(10), wsb=1 << 26)
    a.update(kw)
    if not back:
        return L.gdn_add_norm(a["x"], a["r"], a["w"], a["s"], a["c"], a["eps"], a["h"], a["rdt"], a["n"], a["dt"], a["T"],
                              a["D"], None)
    return L.gdn_add_norm_bwd(a["h"], a["w"], a["dn"], a["dh"], a["s"], a["c"], a["eps"], a["dres"], a["rdt"], a["dx"],
                              a["dw"], a["dt"], a["T"], a["D"], a["ws"], a["wsb"], None)


def test_add_norm_refusals(L):
    for back in (False, True):
        r = lambda **kw: add(L, back, **kw)  # noqa: E731
        assert r(dt=4) == UNSUPPORTED and r(rdt=2) == UNSUPPORTED and r(T=-1) == INVALID and r(T=1 << 31) == INVALID
        assert r(D=0) == INVALID and r(D=16385) == UNSUPPORTED and r(eps=-1.0) == INVALID
        assert r(w=None) == INVALID and r(h=at(3, 8)) == INVALID
    assert add(L, x=None) == INVALID and add(L, n=at(0, 64)) == INVALID and add(L, h=at(1, 64)) == INVALID
    assert add(L, n=at(3, 64)) == INVALID and add(L, T=0) == _lib.GDN_OK
    assert add(L, True, wsb=100) == WORKSPACE and add(L, True, dres=at(6, 64)) == INVALID
    assert add(L, True, dx=at(5)) == INVALID and add(L, True, dx=at(7)) == INVALID and add(L, True, dw=at(2)) == INVALID
    assert add(L, True, T=0, dw=None) == _lib.GDN_OK
    assert L.gdn_norm_bwd_workspace_size(-3) == 0 and L.gdn_norm_bwd_workspace_size(128) > 0


def test_bindings_refuse_cpu_tensors():
    e = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype)  # noqa: E731
    i = lambda *s: e(*s, dtype=torch.int32)  # noqa: E731
    calls = [lambda: gdn.gdn_decode_paged(e(1, 1, 48), e(48, 4), e(2, 3, 48), e(2, 1, 16, 16), i(1), e(1, 1, 1), e(1, 1, 1), 1),
             lambda: gdn.gdn_pages_copy(e(4, 16), i(1), i(1)), lambda: gdn.gdn_pages_take(i(4), n=1),
             lambda: gdn.gdn_pages_ref(i(4), i(1), 1), lambda: gdn.gdn_pages_compact(i(4), None, e(4, 16)),
             lambda: gdn.gdn_pages_fork(i(4), i(1), e(4, 16)),
             lambda: gdn.gdn_gated_norm(e(1, 1, 16), e(1, 1, 16), e(16)),
             lambda: gdn.gdn_gated_norm_bwd(e(1, 1, 16), e(1, 1, 16), e(16), e(1, 1, 16)),
             lambda: gdn.gdn_add_norm(e(1, 16), e(1, 16), e(16)), lambda: gdn.gdn_add_norm_bwd(e(1, 16), e(16), e(1, 16))]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_plain_forms_of_the_counts():
    """The forms that the GPU tests compare with, on pages that exist and pages that do not."""
    assert R.taken([1, 0, -2, 0, 3], [0, 4, 1, 9, -1, 0, 0]) == ([1, 1, 1, 1, 3], [1, 2, -1, -1, -1, 3, -1])
    assert R.taken([0, 0], [None, None, None]) == ([1, 1], [0, 1, -1])
    new, table, where, n_live, back, holes = R.planned([0, 2, 0, 1, -1, 5], [5, 3, 0, 7, -1])
    assert (new, n_live, back, holes) == ([1, 2, 5, 0, 0, 0], 3, [3, 5], [0, 2])
    assert where == [-1, 1, -1, 0, -1, 2] and table == [2, 0, -1, 7, -1]
    pool = torch.arange(4.0)[:, None]
    assert R.copied(pool, pool, [0, 1, 9, 2], [1, 0, 2, 0], 0).reshape(-1).tolist() == [2, 0, 2, 3]

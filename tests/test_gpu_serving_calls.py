"""Calls of the paged decode, the page operations and the norms that their documentation allows or
refuses at its edges: views, refusals that leave everything as it was, optional outputs, every
dispatch. Error bounds are counted as in serving_ref.py."""
import numpy as np
import pytest
import torch

import gated_deltanet_mixer_causal_b200 as gdn
import oracle
import serving_ref as R
from parity import check
from test_gpu_norms import add_case, add_terms, gated_case, gated_terms, slack
from test_gpu_paged import case, ints, pool_of, run_and_check

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


def test_expanded_tensors_are_refused(cuda_device):
    """One token, gate, gradient buffer or page in place of many has the memory of one."""
    dev = cuda_device
    c = case(dev, 4, 1, 1, 2, 16, FP, FP, 6, seed=1)
    args = dict(x=c["x"], conv_w=c["conv_w"], conv_pool=c["conv"], state_pool=c["state"], read_pages=ints([0, 1, 2, 3], dev),
                g=c["g"], beta=c["beta"], Hk=1)
    gate = dict(z=torch.zeros(1, 1, 2, 16, device=dev).expand(4, 1, 2, 16), norm_w=torch.ones(16, device=dev))
    kept = c["state"].clone(), c["conv"].clone()
    for kw in (dict(x=c["x"][:1].expand(4, 1, 64)), gate, dict(conv_pool=c["conv"][:1].expand(6, 3, 64)),
               dict(state_pool=c["state"][:1].expand(6, 2, 16, 16))):
        with pytest.raises(ValueError, match="share memory"):
            gdn.gdn_decode_paged(**{**args, **kw})
    assert torch.equal(kept[0], c["state"]) and torch.equal(kept[1], c["conv"])
    o = torch.zeros(5, 2, 16, device=dev)
    one = torch.zeros(1, 2, 16, device=dev).expand(5, 2, 16)
    w = torch.ones(16, device=dev)
    for call in (lambda: gdn.gdn_gated_norm(o, one, w), lambda: gdn.gdn_gated_norm_bwd(o, one, w, o),
                 lambda: gdn.gdn_gated_norm_bwd(o, o, w, o, dz=one)):
        with pytest.raises(ValueError, match="share memory"):
            call()
    template, pool = torch.ones(1, 16, device=dev), torch.zeros(6, 16, device=dev)
    lists, refs = ints([0, 5], dev), ints([1, 0, 0, 0, 0, 0], dev)
    for call in (lambda: gdn.gdn_pages_copy(template.expand(6, 16), lists, lists, dst_pool=pool),
                 lambda: gdn.gdn_pages_copy(pool, lists, lists, dst_pool=template.expand(6, 16)),
                 lambda: gdn.gdn_pages_fork(refs, ints([0], dev), template.expand(6, 16)),
                 lambda: gdn.gdn_pages_compact(refs, None, template.expand(6, 16))):
        with pytest.raises(ValueError, match="share memory"):
            call()
    assert (pool == 0).all() and refs.tolist() == [1, 0, 0, 0, 0, 0]


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("T,H,d", [(1, 1, 128), (7, 5, 128), (33, 5, 64), (9, 3, 16), (601, 5, 32)])
def test_gated_norm_without_eps(cuda_device, dt, T, H, d):
    """eps = 0 with no row of zeros: the rows that fill up the last group add nothing to dw."""
    o, z, w, dy = gated_case(T, H, d, dt, T + H, False)
    ref = gated_terms(o, z, w, dy, 0.0)
    do, dz, dw = gdn.gdn_gated_norm_bwd(*(t.to(cuda_device) for t in (o, z, w, dy)), eps=0.0)
    y = gdn.gdn_gated_norm(*(t.to(cuda_device) for t in (o, z, w)), eps=0.0)
    name, c, fast = f"gated eps 0 {dt} {T}x{H}x{d}", 160 * R.U + 2 * slack(dt), slack(dt)
    check(name, "y", R.worst(y, ref["y"], ref["y"].abs() * (R.HALF[dt] + 100 * R.U + fast) + 1e-30), 1.0)
    check(name, "do", R.worst(do, ref["do"], ref["do"].abs() * R.HALF[dt] + ref["do_abs"] * c + 1e-30), 1.0)
    check(name, "dz", R.worst(dz, ref["dz"], ref["dz"].abs() * R.HALF[dt] + ref["dz_abs"] * c + 1e-30), 1.0)
    check(name, "dw", R.worst(dw, ref["dw"], ref["dw_abs"] * ((T * H / 592 + 200) * R.U + 2 * fast) + 1e-30), 1.0)


@pytest.mark.parametrize("dt,res", [(BF, BF), (BF, FP), (FP, FP)])
@pytest.mark.parametrize("T,D", [(1, 64), (3, 1024), (5, 16), (7, 1001), (601, 200), (3, 7), (3, 9), (2, 16384)])
def test_add_norm_without_eps(cuda_device, dt, res, T, D):
    x, r, w, dn, dh = add_case(T, D, dt, res, T + D)
    ref = add_terms(r, w, dn, dh, 1.0, 0.0, 0.0)
    dx, dres, dw = gdn.gdn_add_norm_bwd(*(t.to(cuda_device) for t in (r, w, dn, dh)), eps=0.0)
    name, k = f"add eps 0 {dt} {res} {T}x{D}", 160 * R.U
    check(name, "dres", R.worst(dres, ref["dres"], ref["dres"].abs() * R.HALF[res] + ref["dres_abs"] * k + 1e-30), 1.0)
    check(name, "dx", R.worst(dx, ref["dx"], ref["dx"].abs() * R.HALF[dt] + ref["dres_abs"] * k + 1e-30), 1.0)
    check(name, "dw", R.worst(dw, ref["dw"], ref["dw_abs"] * (T / 592 + 200) * R.U + 1e-30), 1.0)


def shared_buffer(dev, layout, P, L, taps, vals, seed):
    """(buffer, taps pool, states pool), [L, P, page] views that lie in one buffer of fp32."""
    gen = torch.Generator().manual_seed(seed)
    make = lambda *s: torch.randint(-99, 99, s, generator=gen).float().to(dev)  # noqa: E731
    if layout == "layer, page, record":
        buf = make(L, P, taps + vals + 4)
        return buf, buf[..., :taps], buf[..., taps:taps + vals]
    if layout == "page, layer, record":
        buf = make(P, L, taps + vals)
        return buf, buf[..., :taps].movedim(0, 1), buf[..., taps:].movedim(0, 1)
    if layout == "page, kind, layer":
        buf = make(P, L * (taps + vals))
        return (buf, buf[:, :L * taps].unflatten(1, (L, taps)).movedim(0, 1),
                buf[:, L * taps:].unflatten(1, (L, vals)).movedim(0, 1))
    buf = make(L, P * (taps + vals))                        # layer, kind, page
    return buf, buf[:, :P * taps].unflatten(1, (P, taps)), buf[:, P * taps:].unflatten(1, (P, vals))


LAYOUTS = ["layer, page, record", "page, layer, record", "page, kind, layer", "layer, kind, page"]


@pytest.mark.parametrize("L", [1, 3])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_pages_of_pools_in_one_buffer(cuda_device, layout, L):
    """Copies, forks and compactions of taps and states that are interleaved as the decode takes them."""
    P, dev = 9, cuda_device
    for kind in ("copy", "fork", "compact"):
        buf, taps, vals = shared_buffer(dev, layout, P, L, 24, 100, seed=L)
        before = [t.clone() for t in (taps, vals)]
        gap = buf[..., 124:].clone() if layout == LAYOUTS[0] else None
        refs = ints([0, 2, 0, 1, 1, 0, 0, 3, 0], dev)
        if kind == "copy":
            src, dst = [1, 2, 3, 4, 4], [2, 3, 1, 0, 8]
            gdn.gdn_pages_copy([taps, vals], ints(src, dev), ints(dst, dev), page_dim=1)
        elif kind == "fork":
            src, dst = [3, 7, 3], [0, 2, 5]
            assert gdn.gdn_pages_fork(refs, ints(src, dev), [taps, vals], page_dim=1).tolist() == dst
            assert refs.tolist() == [1, 2, 1, 1, 1, 1, 0, 3, 0]
        else:
            new, _, m, n_live, src, dst = R.planned(refs.tolist(), [])
            table = ints([7, 4, 3, 1, 0, -1, 9], dev)
            got_map, live = gdn.gdn_pages_compact(refs, table, [taps, vals], page_dim=1)
            assert got_map.tolist() == m and live.tolist() == [n_live] and refs.tolist() == new
            assert table.tolist() == [m[7], m[4], m[3], m[1], -1, -1, 9]
        for pool, was in zip((taps, vals), before):
            assert torch.equal(pool.cpu(), R.copied(was, was, src, dst, 1)), kind
        assert gap is None or torch.equal(buf[..., 124:], gap)


@pytest.mark.parametrize("kind", ["fork", "compact"])
def test_refused_forks_and_compactions_change_nothing(cuda_device, kind):
    """What only the copy's own checks find: the same pool twice, pools that overlap, layers that do."""
    dev = cuda_device
    buf = torch.arange(8 * 64, dtype=FP, device=dev)
    pool, kept = buf[:256].view(8, 32), buf.clone()
    refs, table = ints([0, 1, 0, 2, 1, 0, 0, 1], dev), ints([7, 4, 3, 1], dev)
    for bad, dim in (([pool, pool], 0), ([pool, buf[128:384].view(8, 32)], 0),
                     (buf.as_strided((2, 8, 32), (32, 32, 1)), 1), ([pool[:, :16], pool[:, 12:28]], 0)):
        with pytest.raises(gdn.GDNError):
            if kind == "fork":
                gdn.gdn_pages_fork(refs, ints([3, 1], dev), bad, page_dim=dim)
            else:
                gdn.gdn_pages_compact(refs, table, bad, page_dim=dim)
        assert refs.tolist() == [0, 1, 0, 2, 1, 0, 0, 1] and table.tolist() == [7, 4, 3, 1] and torch.equal(buf, kept)


@pytest.mark.parametrize("act", [BF, FP])
def test_prefill_layer_refuses_a_gate_before_it_computes(cuda_device, act):
    dev, Hk, Hv, d, T = cuda_device, 2, 4, 32, 24
    c = case(dev, 1, T, Hk, Hv, d, act, FP, 2, seed=5, gate=True)
    x, z, g, beta = (c[k].squeeze(0) for k in ("x", "z", "g", "beta"))
    w, zeros = c["norm_w"], torch.zeros(T * Hv * d + 8, dtype=act, device=dev)
    state, conv = torch.full((1, Hv, d, d), 3.0, device=dev), torch.full((1, 3, 8 * d), 3.0, dtype=act, device=dev)
    bad = [dict(z=z[1:]), dict(z=z.half()), dict(z=z.cpu()), dict(z=z.transpose(1, 2).contiguous().transpose(1, 2)),
           dict(z=z[:1].expand(T, Hv, d)), dict(norm_w=w[:16]), dict(norm_w=w.double()), dict(eps=-1.0), dict(norm_w=None),
           dict(z=zeros[1:T * Hv * d + 1].view(T, Hv, d)), dict(o=z), dict(z=None),
           dict(z=torch.zeros(T, Hv * d + 4, dtype=act, device=dev)[:, :Hv * d].unflatten(1, (Hv, d)))]
    run = lambda **kw: gdn.prefill_layer(x, c["conv_w"], g, beta, Hk, Hv, d, final_state=state, conv_state_out=conv,  # noqa: E731
                                         **{**dict(z=z, norm_w=w), **kw})
    for kw in bad:
        with pytest.raises((ValueError, gdn.GDNError)):
            run(**kw)
    torch.cuda.synchronize()
    assert (state == 3.0).all() and (conv == 3.0).all()
    o = run()
    assert torch.equal(run(o=torch.empty_like(o)), o) and not (state == 3.0).any()
    empty = gdn.prefill_layer(x[:0], c["conv_w"], g[:0], beta[:0], Hk, Hv, d, z=z[:0], norm_w=w)
    assert empty.shape == (0, Hv, d)


def test_paged_decode_of_slices(cuda_device):
    """Sequences behind the first of a batch: with 10 value heads their g and beta begin on 8 bytes."""
    c = case(cuda_device, 4, 1, 2, 10, 16, FP, FP, 6, seed=12)
    for key in ("x", "g", "beta"):
        c[key] = c[key][1:]
    assert c["g"].data_ptr() % 16 == 8
    run_and_check("paged slices", c, [4, 0, 2], None, None, cuda_device)


@pytest.mark.parametrize("dt", [BF, FP])
def test_norms_fed_by_the_launch_before(cuda_device, dt):
    """Each call's inputs are the outputs of the launch just before it in the stream, whose end it
    overlaps: 30 rounds of forward and backward passes, against the same rounds with a wait behind
    every call."""
    T, H, d, rounds = 600, 4, 128, 30
    gen = torch.Generator().manual_seed(11)
    o, z, x = (torch.randn(T, H * d, generator=gen).to(dt).to(cuda_device) for _ in range(3))
    w, wide = (torch.rand(n, generator=gen).to(dt).to(cuda_device) for n in (d, H * d))

    def chain(wait):
        a, res, kept = o.clone(), x.clone(), []
        for _ in range(rounds):
            y = gdn.gdn_gated_norm(a.view(T, H, d), z.view(T, H, d), w).view(T, H * d)
            wait()
            n, h = gdn.gdn_add_norm(y, res, wide, scale=0.5)
            wait()
            dx, dres, dwide = gdn.gdn_add_norm_bwd(h, wide, n, n, scale=0.5)
            wait()
            do, dz, dw = gdn.gdn_gated_norm_bwd(dx.view(T, H, d), dres.view(T, H, d), w, dx.view(T, H, d))
            wait()
            # the weight gradients of this round are weights of the next call
            y2 = gdn.gdn_gated_norm(do, dz, dw.to(dt))
            wait()
            n2, _ = gdn.gdn_add_norm(y2.view(T, H * d), h, dwide.to(dt))
            wait()
            a, res = n2, h
            kept += [dw, dwide, n2]
        return kept

    once = chain(lambda: None)
    slow = chain(torch.cuda.synchronize)
    assert all(torch.equal(p, q) for p, q in zip(once, slow))
    assert all(torch.isfinite(t).all() for t in once)


def test_lists_of_nearly_2_to_the_31(cuda_device):
    """The longest list and table that a call takes: an index that steps over the end of 32 bits."""
    n, dev = 2 ** 31 - 512, cuda_device
    pages = torch.full((n,), -1, dtype=torch.int32, device=dev)
    pages[0], pages[-1] = 5, 3
    refs = ints([0, 0, 0, 1, 0, 2], dev)
    gdn.gdn_pages_ref(refs, pages, 1)
    assert refs.tolist() == [0, 0, 0, 2, 0, 3]
    gdn.gdn_pages_plan(refs, pages)
    assert refs.tolist() == [2, 3, 0, 0, 0, 0] and pages[0].item() == 1 and pages[-1].item() == 0
    assert int((pages == -1).sum()) == n - 2


@pytest.mark.parametrize("page,n,L", [(16, 1, 1), (16, 2048, 2), (528, 700, 1), (528, 1100, 3), (16384, 31, 1), (16384, 32, 2),
                                      (16400, 40, 1), (40960, 200, 2), (1 << 20, 33, 1), (8208, 65, 1)])
def test_plain_copies(cuda_device, page, n, L):
    """Every shape of a plain copy's tiles: parts of a page, a whole one, several; groups of entries
    below and above the number from which a CTA takes four (32). Entries that are void, and that stay."""
    P, gen = 2 * n + 3, torch.Generator().manual_seed(n)
    order = torch.randperm(P, generator=gen).tolist()
    src, dst = order[:n], order[n:2 * n]
    for i in range(0, n, 7):
        src[i] = (-1, P, dst[i])[i // 7 % 3]                            # void, void, stays
    for i in range(3, n, 11):
        dst[i] = -5
    pools = [pool_of(cuda_device, (L, P, page // 4), FP, 1), pool_of(cuda_device, (L, P, 24), BF, 2)]
    want = [p.clone() for p in pools]                                   # no order matters: copy on the device
    pairs = [(s, d) for s, d in zip(src, dst) if 0 <= s < P and 0 <= d < P]
    if pairs:
        s, d = (torch.tensor(v, device=cuda_device) for v in zip(*pairs))
        for w, p in zip(want, pools):
            w[:, d] = p[:, s]
    gdn.gdn_pages_copy(pools, ints(src, cuda_device), ints(dst, cuda_device), page_dim=1, plain=True)
    assert all(torch.equal(p, w) for p, w in zip(pools, want))


@pytest.mark.parametrize("P,page", [(200, 20000), (5000, 16400), (300, 528)])
def test_compactions_of_larger_pages(cuda_device, P, page):
    gen = torch.Generator().manual_seed(P)
    refs = torch.randint(0, 3, (P,), generator=gen).tolist()
    pool = pool_of(cuda_device, (P, page // 4), FP, 3)
    new, _, m, n_live, back, holes = R.planned(refs, [])
    want = R.copied(pool, pool, back, holes, 0)
    t = ints(refs, cuda_device)
    got_map, live = gdn.gdn_pages_compact(t, None, pool)
    assert t.tolist() == new and got_map.tolist() == m and live.tolist() == [n_live] and torch.equal(pool.cpu(), want)


@pytest.mark.parametrize("act,st,d,n,gate", [(BF, FP, 128, 1, False), (FP, FP, 64, 3, False), (BF, BF, 32, 2, False),
                                             (FP, BF, 128, 2, False), (BF, FP, 128, 2, True)])
def test_paged_scale(cuda_device, act, st, d, n, gate):
    c = case(cuda_device, 4, n, 2, 4, d, act, st, 6, seed=13, gate=gate)
    run_and_check(f"paged scale {act} {d} {n}", c, [5, 0, 3, -1], None, None, cuda_device, eps=1e-3, scale=0.0884)


def sizes_against_outputs(c, read, n_valid):
    """(alpha |S before| + |u|) / |o before its norm| for every valid token and head, [B, n, Hv], else 1.

    o = alpha S q + u (k.q) is a sum of products of a unit vector with S and of u, so its fp32 error is
    in proportion to |S| and |u| and not to what is left of them in o. A sequence that begins here has
    o = u (k.q): with k.q = 1e-4 it carries 1e4 times the error of k.q, which the output norm then
    takes over where eps binds. |u| = |S after - alpha S before|, since |k| = 1."""
    B, n, _ = c["x"].shape
    P, Hv, d, _ = c["state"].shape
    ratio = torch.ones(B, n, Hv, dtype=torch.float64)
    for b in range(B):
        fresh = not 0 <= read[b] < P
        S = np.zeros((1, Hv, d, d)) if fresh else R.f64(c["state"][read[b]])[None].numpy()
        taps = np.zeros((1, 3, c["x"].shape[2])) if fresh else R.f64(c["conv"][read[b]])[None].numpy()
        for t in range(min(max(n_valid[b], 0), n)):
            old = np.exp(R.f64(c["g"][b, t]).numpy())[:, None, None] * S[0]
            o, S, taps = oracle.decode_step(R.f64(c["x"][b, t])[None].numpy(), R.f64(c["conv_w"]).numpy(), taps,
                                            R.f64(c["g"][b, t])[None].numpy(), R.f64(c["beta"][b, t])[None].numpy(), S,
                                            c["Hk"], Hv, d, d, 1.0)
            size = np.linalg.norm(old, axis=(1, 2)) + np.linalg.norm(S[0] - old, axis=(1, 2))
            ratio[b, t] = torch.from_numpy(np.maximum(size / np.maximum(np.linalg.norm(o[0], axis=1), 1e-30), 1.0))
    return ratio


@pytest.mark.parametrize("B,Hk,Hv,d,n,act,st", [
    (150, 16, 32, 64, 2, BF, FP), (150, 16, 32, 64, 2, BF, BF), (150, 16, 32, 64, 2, FP, FP), (150, 16, 32, 64, 2, FP, BF),
    (160, 16, 48, 32, 3, BF, BF), (160, 16, 48, 32, 3, FP, FP), (300, 16, 16, 16, 3, BF, FP), (300, 16, 16, 16, 3, FP, BF),
    (80, 16, 16, 64, 1, BF, BF)])
def test_paged_many_narrow_heads_with_everything(cuda_device, act, st, B, Hk, Hv, d, n):
    """CTAs of several key heads (heads below 128 in batches that fill the GPU): gate and norm,
    scattered pages, sequences that begin here, a page for each token or none, ragged counts."""
    P, gen = B * (n + 1) + 5, torch.Generator().manual_seed(B + d)
    order = torch.randperm(P, generator=gen).tolist()
    read = [-1 if b % 13 == 4 else order[b] for b in range(B)]
    write = [[-1 if (b + t) % 5 == 3 else order[B + b * n + t] for t in range(n)] for b in range(B)]
    valid = torch.randint(0, n + 2, (B,), generator=gen).tolist()
    c = case(cuda_device, B, n, Hk, Hv, d, act, st, P, seed=B, wide=True, gate=True)
    ratio = sizes_against_outputs(c, read, valid)
    o = torch.full((B, n, Hv, d), 7.0, dtype=act, device=cuda_device)
    want_o, want_s, want_c = R.paged(c["x"], c["conv_w"], c["conv"], c["state"], read, c["g"], c["beta"], Hk, write, valid,
                                     c["z"], c["norm_w"], 1e-6, o)
    gdn.gdn_decode_paged(c["x"], c["conv_w"], c["conv"], c["state"], ints(read, cuda_device), c["g"], c["beta"], Hk,
                         write_pages=ints(write, cuda_device), n_valid=ints(valid, cuda_device), z=c["z"],
                         norm_w=c["norm_w"], o=o)
    name, fp32 = f"paged KH {act} {st} {Hk}/{Hv}x{d} n{n}", n * (3 * d + 40) * R.U
    fast = 0.0 if act == FP else 2.0 ** -20
    assert torch.equal(R.f64(c["conv"]), want_c)
    off = lambda got, want, dims: (R.f64(got) - want).norm(dim=dims) / want.norm(dim=dims).clamp(min=1e-300)  # noqa: E731
    kept = torch.tensor([p not in {q for row in write for q in row} for p in range(P)])
    assert torch.equal(R.f64(c["state"])[kept], want_s[kept])
    check(name, "state", off(c["state"], want_s, (2, 3)).max(), R.HALF[st] + fp32 + 4 * fast)
    live = torch.arange(n) < torch.tensor(valid)[:, None]
    assert (R.f64(o)[~live] == 7.0).all()
    bound = R.HALF[act] + 2 * (fp32 + 4 * fast) * ratio
    check(name, "o / bound", (off(o, want_o, -1) / bound)[live].max(), 1.0)


@pytest.mark.parametrize("dt,res,D", [(BF, FP, 1024), (BF, BF, 1001), (FP, FP, 16384), (FP, BF, 40), (BF, FP, 9001)])
def test_norm_backward_without_weight_or_input_gradient(cuda_device, dt, res, D):
    """dw = NULL (with no workspace) and dx = NULL of the C entry points: the other gradients are the
    same as with them."""
    L, dev, T, stream = gdn.lib(), cuda_device, 37, torch.cuda.current_stream().cuda_stream
    code = lambda t: 0 if t.dtype == FP else 1  # noqa: E731
    x, r, w, dn, dh = (t.to(dev) for t in add_case(T, D, dt, res, D))
    dx, dres, dw = gdn.gdn_add_norm_bwd(r, w, dn, dh, scale=0.5, w_add=1.0)
    ws = torch.empty(gdn.gdn_norm_bwd_workspace_size(D), dtype=torch.uint8, device=dev)
    for want_dx, want_dw in ((False, True), (True, False), (False, False)):
        dx2, dres2, dw2 = torch.full_like(dx, 7), torch.full_like(dres, 7), torch.full_like(dw, 7)
        status = L.gdn_add_norm_bwd(r.data_ptr(), w.data_ptr(), dn.data_ptr(), dh.data_ptr(), 0.5, 1.0, 1e-6, dres2.data_ptr(),
                                    code(r), dx2.data_ptr() if want_dx else None, dw2.data_ptr() if want_dw else None,
                                    code(dn), T, D, ws.data_ptr() if want_dw else None, ws.numel() if want_dw else 0, stream)
        assert status == 0 and torch.equal(dres2, dres)
        assert torch.equal(dx2, dx) if want_dx else (dx2 == 7).all()
        assert torch.equal(dw2, dw) if want_dw else (dw2 == 7).all()
    o, z, w, dy = (t.to(dev) for t in gated_case(T, 3, 64, dt, 9, False))
    do, dz, _ = gdn.gdn_gated_norm_bwd(o, z, w, dy)
    do2, dz2 = torch.empty_like(do), torch.empty_like(dz)
    assert L.gdn_gated_norm_bwd(o.data_ptr(), z.data_ptr(), 0, w.data_ptr(), 1e-6, dy.data_ptr(), do2.data_ptr(),
                                dz2.data_ptr(), 0, None, code(o), T, 3, 64, None, 0, stream) == 0
    assert torch.equal(do2, do) and torch.equal(dz2, dz)


def test_pages_captured(cuda_device):
    """A captured fork and compaction, replayed over counts and tables that change."""
    dev, P = cuda_device, 12
    pool, src = pool_of(dev, (P, 40), FP, 4), ints([2, 2, 7, -1], dev)
    refs, table = ints([0] * P, dev), ints([0, 0, 0], dev)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = gdn.gdn_pages_fork(refs, src, pool)
        where, live = gdn.gdn_pages_compact(refs, table, pool)
    for counts, names in (([0, 0, 3, 1, 0, 0, 0, 2, 0, 0, 0, 1], [2, 7, 11]), ([1] * 9 + [0, 0, 0], [8, 7, 2]),
                          ([0] * P, [3, -1, 0]), ([1] * P, [0, 5, 11])):
        refs.copy_(torch.tensor(counts)), table.copy_(torch.tensor(names))
        new, got = R.taken(counts, src.tolist())
        want = R.copied(pool, pool, src.tolist(), got, 0)
        new, named, m, n_live, back, holes = R.planned(new, names)
        want = R.copied(want, want, back, holes, 0)
        graph.replay()
        torch.cuda.synchronize()
        assert out.tolist() == got and refs.tolist() == new and table.tolist() == named
        assert where.tolist() == m and live.tolist() == [n_live] and torch.equal(pool.cpu(), want)


def test_calls_on_two_streams_at_once(cuda_device):
    """Decodes, forks and norms of two servers on a stream each, interleaved call by call, against the
    same calls one server after the other."""
    def server(seed):
        c = case(cuda_device, 30, 1, 4, 8, 64, BF, FP, 64, seed=seed, gate=True)
        c["refs"] = ints([1] * 30 + [0] * 34, cuda_device)
        c["pages"] = ints(list(range(30)), cuda_device)
        c["kept"] = []
        return c

    def step(c, i):
        o = gdn.gdn_decode_paged(c["x"], c["conv_w"], c["conv"], c["state"], c["pages"], c["g"], c["beta"], 4, z=c["z"],
                                 norm_w=c["norm_w"])
        new = gdn.gdn_pages_fork(c["refs"], c["pages"], [c["state"], c["conv"]])
        gdn.gdn_pages_ref(c["refs"], c["pages"], -1)
        c["pages"] = new
        do, dz, dw = gdn.gdn_gated_norm_bwd(o[:, 0], o[:, 0].contiguous() * 0.5, c["norm_w"], o[:, 0])
        c["kept"] += [o, new, do, dz, dw]

    alone = [server(1), server(2)]
    for c in alone:
        for i in range(12):
            step(c, i)
    torch.cuda.synchronize()
    both, streams = [server(1), server(2)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(12):
        for c, s in zip(both, streams):
            with torch.cuda.stream(s):
                step(c, i)
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert all(torch.equal(p, q) for p, q in zip(a["kept"], b["kept"]))
        assert torch.equal(a["state"], b["state"]) and torch.equal(a["conv"], b["conv"]) and torch.equal(a["refs"], b["refs"])

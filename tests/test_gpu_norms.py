"""The gated norm and the add norm, forward and backward, against fp64 formulas and differences.

Bounds, in fp32 roundings U = 2^-24: a row's sum of squares is added in at most 100 steps (a
thread's values, a warp's tree, the warps), so 1 / rms is off by at most 60 U, and each product
behind it by a few more: 100 U of the terms that are added (160 U backward, where two such sums
enter), and half a step of the output's type. The fast exponential of the bf16 form adds 2^-20. A
weight gradient adds rows in a chain of at most (rows / CTAs + 100) steps."""
import pytest
import torch

import gated_deltanet_mixer_causal_b200 as gdn
import serving_ref as R
from parity import check

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


def slack(dt):
    return 0.0 if dt == FP else 2.0 ** -20


def rnd(gen, *shape, std=1.0):
    return torch.randn(shape, generator=gen) * std


def gated_case(T, H, d, dt, seed, wide):
    gen = torch.Generator().manual_seed(seed)
    o, dy = rnd(gen, T, H, d, std=0.3).to(dt), rnd(gen, T, H, d).to(dt)
    z = rnd(gen, T, (2 if wide else 1) * H * d, std=3.0).to(dt)
    return o, z[:, -H * d:].unflatten(1, (H, d)), (1 + 0.1 * rnd(gen, d)).to(dt), dy


def gated_terms(o, z, w, dy, eps):
    o, z, w, dy = (R.f64(t) for t in (o, z, w, dy))
    r = (o.square().mean(-1, keepdim=True) + eps) ** -0.5
    p = torch.sigmoid(z)
    xh, gate, slope = o * r, z * p, p * (1 + z * (1 - p))
    a = dy * gate * w
    mean = (a * xh).mean(-1, keepdim=True)
    mean_abs = (a * xh).abs().mean(-1, keepdim=True)
    return dict(y=xh * w * gate, do=r * (a - xh * mean), do_abs=r * (a.abs() + xh.abs() * mean_abs),
                dz=dy * xh * w * slope, dz_abs=(dy * xh * w * p).abs() * (1 + z.abs()),
                dw=(dy * xh * gate).sum((0, 1)), dw_abs=(dy * xh * gate).abs().sum((0, 1)))


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("T,H,d,wide", [(1, 1, 16, False), (7, 3, 32, True), (33, 5, 64, True), (65, 6, 128, False),
                                        (300, 48, 128, True), (2, 1, 128, True)])
def test_gated_norm(cuda_device, dt, T, H, d, wide):
    o, z, w, dy = gated_case(T, H, d, dt, T + H + d, wide)
    eps = 1e-6
    ref = gated_terms(o, z, w, dy, eps)
    dev = [t.to(cuda_device) for t in (o, z, w, dy)]
    od, zd, wd, dyd = dev
    if wide:                                              # .to() keeps no strides of a view
        zw = torch.zeros(T, 2 * H * d, dtype=dt, device=cuda_device)
        zw[:, -H * d:] = zd.reshape(T, -1)
        zd = zw[:, -H * d:].unflatten(1, (H, d))
    name, fast = f"gated {dt} {T}x{H}x{d}", slack(dt)
    y = gdn.gdn_gated_norm(od, zd, wd, eps=eps)
    check(name, "y", R.worst(y, ref["y"], ref["y"].abs() * (R.HALF[dt] + 100 * R.U + fast) + 1e-30), 1.0)
    do, dz, dw = gdn.gdn_gated_norm_bwd(od, zd, wd, dyd, eps=eps)
    c = 160 * R.U + 2 * fast
    check(name, "do", R.worst(do, ref["do"], ref["do"].abs() * R.HALF[dt] + ref["do_abs"] * c + 1e-30), 1.0)
    check(name, "dz", R.worst(dz, ref["dz"], ref["dz"].abs() * R.HALF[dt] + ref["dz_abs"] * c + 1e-30), 1.0)
    steps = T * H / 592 + 200
    check(name, "dw", R.worst(dw, ref["dw"], ref["dw_abs"] * (steps * R.U + 2 * fast) + 1e-30), 1.0)
    again = gdn.gdn_gated_norm_bwd(od, zd, wd, dyd, eps=eps)
    assert all(torch.equal(a, b) for a, b in zip(again, (do, dz, dw)))
    # in place: y over o, do over dy, dz into a strided view
    wide_dz = torch.full((T, H * d + 8), 5.0, dtype=dt, device=cuda_device)
    into = wide_dz[:, 8:].unflatten(1, (H, d))
    dy2, o2 = dyd.clone(), od.clone()
    gdn.gdn_gated_norm_bwd(od, zd, wd, dy2, eps=eps, do=dy2, dz=into)
    assert torch.equal(dy2, do) and torch.equal(into, dz) and (wide_dz[:, :8] == 5.0).all()
    gdn.gdn_gated_norm(o2, zd, wd, eps=eps, y=o2)
    assert torch.equal(o2, y)


def test_gated_norm_zero_rows_and_extremes(cuda_device):
    """A row of zeros has norm 0 (under eps), gates of +-100 saturate, an infinite gate gives
    what the formula's limit does on the negative side: 0."""
    for dt in (BF, FP):
        o, z, w, dy = (t.to(cuda_device) for t in gated_case(4, 2, 64, dt, 3, False))
        o[0], z[1], z[2] = 0, 100.0, -100.0
        y = gdn.gdn_gated_norm(o, z, w)
        do, dz, dw = gdn.gdn_gated_norm_bwd(o, z, w, dy)
        assert (y[0] == 0).all() and all(torch.isfinite(t).all() for t in (y, do, dz, dw))
        ref = gated_terms(o.cpu(), z.cpu(), w.cpu(), dy.cpu(), 1e-6)
        assert (R.f64(y[2]).abs() <= 1e-30).all() and (R.f64(dz[2]).abs() <= 1e-30).all()
        c = 160 * R.U + 2 * slack(dt)
        check("gated extremes", "y", R.worst(y, ref["y"], ref["y"].abs() * (R.HALF[dt] + c) + 1e-30), 1.0)
        check("gated extremes", "do", R.worst(do, ref["do"], ref["do"].abs() * R.HALF[dt] + ref["do_abs"] * c + 1e-30), 1.0)


def add_case(T, D, dt, res, seed):
    gen = torch.Generator().manual_seed(seed)
    return (rnd(gen, T, D).to(dt), rnd(gen, T, D, std=2.0).to(res), rnd(gen, D, std=0.2).to(dt), rnd(gen, T, D).to(dt),
            rnd(gen, T, D).to(res))


def add_terms(h, w, dn, dh, scale, c, eps):
    h, w, dn = R.f64(h), R.f64(w) + c, R.f64(dn)
    r = (h.square().mean(-1, keepdim=True) + eps) ** -0.5
    a, hh = dn * w, h * r
    mean, mean_abs = (a * hh).mean(-1, keepdim=True), (a * hh).abs().mean(-1, keepdim=True)
    dh = torch.zeros_like(h) if dh is None else R.f64(dh)
    dres = dh + r * (a - hh * mean)
    return dict(dres=dres, dx=scale * dres, dres_abs=dh.abs() + r * (a.abs() + hh.abs() * mean_abs),
                dw=(dn * hh).sum(0), dw_abs=(dn * hh).abs().sum(0))


@pytest.mark.parametrize("dt,res", [(BF, BF), (BF, FP), (FP, FP), (FP, BF)])
@pytest.mark.parametrize("T,D", [(1, 1), (3, 7), (5, 64), (4, 1001), (300, 40), (129, 2048), (3, 4096), (2, 8200),
                                 (2, 9001), (3, 16384), (700, 256), (17, 7001), (5000, 9), (900, 70), (5, 16383),
                                 (310, 16380), (33, 15), (1300, 130)])
def test_add_norm(cuda_device, dt, res, T, D):
    x, r, w, dn, dh = add_case(T, D, dt, res, T + D)
    scale, c, eps = 0.7, 1.0, 1e-5
    s32 = float(torch.tensor(scale))                       # the scale the kernel gets, in fp32
    h64 = R.f64(r) + s32 * R.f64(x)
    n64 = h64 * (h64.square().mean(-1, keepdim=True) + eps) ** -0.5 * (R.f64(w) + c)
    size = R.f64(r).abs() + s32 * R.f64(x).abs()
    n_size = size * (h64.square().mean(-1, keepdim=True) + eps) ** -0.5 * (R.f64(w).abs() + c)
    xd, rd, wd, dnd, dhd = (t.to(cuda_device) for t in (x, r, w, dn, dh))
    name = f"add {dt} {res} {T}x{D}"
    n, h = gdn.gdn_add_norm(xd, rd, wd, scale=scale, w_add=c, eps=eps)
    check(name, "h", R.worst(h, h64, h64.abs() * R.HALF[res] + size * 2 * R.U + 1e-30), 1.0)
    check(name, "n", R.worst(n, n64, n64.abs() * R.HALF[dt] + n_size * 100 * R.U + 1e-30), 1.0)
    r2 = rd.clone()
    n2, _ = gdn.gdn_add_norm(xd, r2, wd, scale=scale, w_add=c, eps=eps, h=r2)
    assert torch.equal(n2, n) and torch.equal(r2, h)
    for grad in (dh, None):
        ref = add_terms(h.cpu(), w, dn, grad, s32, c, eps)
        dx, dres, dw = gdn.gdn_add_norm_bwd(h, wd, dnd, None if grad is None else dhd, scale=scale, w_add=c, eps=eps)
        k = 160 * R.U
        check(name, "dres", R.worst(dres, ref["dres"], ref["dres"].abs() * R.HALF[res] + ref["dres_abs"] * k + 1e-30), 1.0)
        check(name, "dx", R.worst(dx, ref["dx"], ref["dx"].abs() * R.HALF[dt] + ref["dres_abs"] * k + 1e-30), 1.0)
        check(name, "dw", R.worst(dw, ref["dw"], ref["dw_abs"] * (T / 592 + 200) * R.U + 1e-30), 1.0)
    dh2 = dhd.clone()
    dx2, dres2, dw2 = gdn.gdn_add_norm_bwd(h, wd, dnd, dh2, scale=scale, w_add=c, eps=eps, dres=dh2)
    one = gdn.gdn_add_norm_bwd(h, wd, dnd, dhd, scale=scale, w_add=c, eps=eps)
    assert dres2 is dh2 and all(torch.equal(a, b) for a, b in zip((dx2, dres2, dw2), one))


@pytest.mark.parametrize("T,D", [(3, 5), (7, 1001), (2, 8203), (9, 12), (4, 64)])
def test_add_norm_keeps_to_its_rows(cuda_device, T, D):
    """Rows that neither begin nor end on 16 bytes, at the end of their buffers: nothing behind them
    is written, and what lies there (NaN) is not used."""
    x, r, w, dn, dh = add_case(T, D, BF, FP, T + D)
    def behind(t):                                         # t in front of 64 NaN
        buf = torch.full((t.numel() + 64,), float("nan"), dtype=t.dtype, device=cuda_device)
        buf[:t.numel()] = t.reshape(-1).to(cuda_device)
        return buf, buf[:t.numel()].view(t.shape)
    bufs, views = zip(*(behind(t) for t in (x, r, w, dn, dh, torch.zeros_like(x), torch.zeros_like(r),
                                            torch.zeros_like(x), torch.zeros_like(r))))
    xd, rd, wd, dnd, dhd, n, h, dx, dres = views
    gdn.gdn_add_norm(xd, rd, wd, h=h, n=n)
    n2, h2 = gdn.gdn_add_norm(x.to(cuda_device), r.to(cuda_device), w.to(cuda_device))
    assert torch.equal(n, n2) and torch.equal(h, h2)
    dwb, dw = behind(torch.zeros(D))
    gdn.gdn_add_norm_bwd(h, wd, dnd, dhd, dres=dres, dx=dx, dw=dw)
    one = gdn.gdn_add_norm_bwd(h2, w.to(cuda_device), dn.to(cuda_device), dh.to(cuda_device))
    assert all(torch.equal(a, b) for a, b in zip((dx, dres, dw), one))
    for buf, t in zip((*bufs, dwb), (*views, dw)):
        assert torch.isnan(buf[t.numel():]).all()


@pytest.mark.parametrize("D", range(1, 8))
@pytest.mark.parametrize("dt,res", [(BF, FP), (FP, BF)])
def test_add_norm_of_rows_shorter_than_a_run(cuda_device, D, dt, res):
    """Several rows lie in one run of eight elements, and the last runs pass the end of the tensor,
    which lies at the end of its buffer."""
    for T in (1, 2, 7, 9, 16, 1201):
        ts = add_case(T, D, dt, res, T + D)
        x, r, w, dn, dh = (t.to(cuda_device) for t in ts)
        h64 = R.f64(r) + R.f64(x)
        size = R.f64(r).abs() + R.f64(x).abs()
        rms = (h64.square().mean(-1, keepdim=True) + 1e-6) ** -0.5
        n, h = gdn.gdn_add_norm(x, r, w)
        name, k = f"add {dt} {T}x{D}", 160 * R.U
        n64 = h64 * rms * R.f64(w)
        check(name, "h", R.worst(h, h64, h64.abs() * R.HALF[res] + size * 2 * R.U + 1e-30), 1.0)
        check(name, "n", R.worst(n, n64, n64.abs() * R.HALF[dt] + size * rms * R.f64(w).abs() * k + 1e-30), 1.0)
        ref = add_terms(h, w, dn, dh, 1.0, 0.0, 1e-6)
        dx, dres, dw = gdn.gdn_add_norm_bwd(h, w, dn, dh)
        check(name, "dres", R.worst(dres, ref["dres"], ref["dres"].abs() * R.HALF[res] + ref["dres_abs"] * k + 1e-30), 1.0)
        check(name, "dx", R.worst(dx, ref["dx"], ref["dx"].abs() * R.HALF[dt] + ref["dres_abs"] * k + 1e-30), 1.0)
        check(name, "dw", R.worst(dw, ref["dw"], ref["dw_abs"] * (T / 592 + 200) * R.U + 1e-30), 1.0)


def test_gradients_against_differences(cuda_device):
    """Directional derivatives by central differences of the fp64 forward formulas: with a step
    of 1e-5 they are exact to about 1e-9, so the kernels' fp32 error (counted above, summed over
    the elements) is what is left."""
    gen = torch.Generator().manual_seed(1)
    o, z, w, dy = gated_case(9, 3, 64, FP, 5, False)
    do, dz, dw = (R.f64(t) for t in gdn.gdn_gated_norm_bwd(*(t.to(cuda_device) for t in (o, z, w, dy))))
    f = lambda a, b, c: (R.gated(a, b, c, 1e-6) * R.f64(dy)).sum()  # noqa: E731
    args = [R.f64(t) for t in (o, z, w)]
    for i, grad in enumerate((do, dz, dw)):
        v = rnd(gen, *grad.shape).double()
        up, down = ([a + s * 1e-5 * v if j == i else a for j, a in enumerate(args)] for s in (1, -1))
        diff, got = (f(*up) - f(*down)) / 2e-5, (grad * v).sum()
        assert abs(diff - got) <= 400 * R.U * (grad * v).abs().sum() + 1e-7
    x, r, w, dn, dh = add_case(6, 50, FP, FP, 6)
    h = (R.f64(r) + 0.5 * R.f64(x)).float()
    dx, dres, dw = (R.f64(t) for t in gdn.gdn_add_norm_bwd(h.to(cuda_device), w.to(cuda_device), dn.to(cuda_device),
                                                           dh.to(cuda_device), scale=0.5, w_add=1.0))
    f = lambda a, b, c: (((b + 0.5 * a) * ((b + 0.5 * a).square().mean(-1, keepdim=True) + 1e-6) ** -0.5 * (c + 1)  # noqa: E731
                          * R.f64(dn)).sum() + ((b + 0.5 * a) * R.f64(dh)).sum())
    args = [R.f64(x), R.f64(h) - 0.5 * R.f64(x), R.f64(w)]
    for i, grad in enumerate((dx, dres, dw)):
        v = rnd(gen, *grad.shape).double()
        up, down = ([a + s * 1e-5 * v if j == i else a for j, a in enumerate(args)] for s in (1, -1))
        diff, got = (f(*up) - f(*down)) / 2e-5, (grad * v).sum()
        assert abs(diff - got) <= 400 * R.U * (grad * v).abs().sum() + 1e-7


def test_norms_without_tokens(cuda_device):
    e = lambda *s: torch.empty(s, device=cuda_device)  # noqa: E731
    assert gdn.gdn_gated_norm(e(0, 3, 16), e(0, 3, 16), e(16)).shape == (0, 3, 16)
    _, _, dw = gdn.gdn_gated_norm_bwd(e(0, 3, 16), e(0, 3, 16), e(16), e(0, 3, 16))
    assert (dw == 0).all()
    gdn.gdn_add_norm(e(0, 9), e(0, 9), e(9))
    _, _, dw = gdn.gdn_add_norm_bwd(e(0, 9), e(9), e(0, 9))
    assert (dw == 0).all()


def test_norm_backward_captured(cuda_device):
    """Two captured backward passes with a workspace each, replayed in turn over new gradients."""
    o, z, w, dy = (t.to(cuda_device) for t in gated_case(40, 4, 128, BF, 7, False))
    x, r, w2, dn, dh = (t.to(cuda_device) for t in add_case(40, 512, BF, FP, 8))
    ws = [torch.empty(gdn.gdn_norm_bwd_workspace_size(n), dtype=torch.uint8, device=cuda_device) for n in (128, 512)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        a = gdn.gdn_gated_norm_bwd(o, z, w, dy, workspace=ws[0])
        b = gdn.gdn_add_norm_bwd(r, w2, dn, dh, workspace=ws[1])
    for k in range(2):
        dy.mul_(-1.5), dn.mul_(0.5)
        graph.replay()
        ea, eb = gdn.gdn_gated_norm_bwd(o, z, w, dy), gdn.gdn_add_norm_bwd(r, w2, dn, dh)
        assert all(torch.equal(p, q) for p, q in zip((*a, *b), (*ea, *eb)))

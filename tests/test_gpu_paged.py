"""The paged decode and the page operations against plain fp64 and CPU forms.

Bounds: every output passes through at most three sums of D products (the norms of q and k, S k,
S q) and about 40 further fp32 roundings a token, so per (sequence, head) the fp32 error is at
most n_tok (3 D + 40) 2^-24 of the norm; the value's own storage adds its type's half step. The
gated output is a quotient of two such values: twice that."""
import numpy as np
import pytest
import torch

import gated_deltanet_mixer_causal_b200 as gdn
import oracle
import serving_ref as R
from parity import check, frob_rel

pytestmark = pytest.mark.gpu


def case(dev, B, n, Hk, Hv, d, act, st, P, seed, wide=False, gate=False):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s, std=1.0: torch.randn(s, generator=gen) * std  # noqa: E731
    Cc = (2 * Hk + Hv) * d
    proj = rnd(B, n, Cc + (Hv * d if wide else 0)).to(act).to(dev)
    c = dict(x=proj[:, :, :Cc], conv_w=rnd(Cc, 4, std=0.5).to(act).to(dev), conv=rnd(P, 3, Cc).to(act).to(dev),
             state=rnd(P, Hv, d, d, std=0.05).to(st).to(dev),
             g=(-0.3 * torch.rand((B, n, Hv), generator=gen)).to(dev),
             beta=torch.sigmoid(rnd(B, n, Hv)).to(dev), Hk=Hk, z=None, norm_w=None)
    if gate:
        z = rnd(B, n, Hv, d).to(act).to(dev)
        c["z"] = proj[:, :, Cc:].unflatten(2, (Hv, d)) if wide else z
        c["norm_w"] = (1 + 0.1 * rnd(d)).to(act).to(dev)
    return c


def ints(v, dev):
    return None if v is None else torch.tensor([int(i) for i in v] if isinstance(v, np.ndarray) else v, dtype=torch.int32, device=dev)


def run_and_check(name, c, read, write, n_valid, dev, eps=1e-6, scale=1.0):
    B, n, _ = c["x"].shape
    P, Hv, d, _ = c["state"].shape
    o = torch.full((B, n, Hv, d), 7.0, dtype=c["x"].dtype, device=dev)
    want_o, want_s, want_c = R.paged(c["x"], c["conv_w"], c["conv"], c["state"], read, c["g"], c["beta"], c["Hk"],
                                     write, n_valid, c["z"], c["norm_w"], eps, o, scale)
    kept_o = (want_o == 7.0).all(-1)
    got = gdn.gdn_decode_paged(c["x"], c["conv_w"], c["conv"], c["state"], ints(read, dev), c["g"], c["beta"],
                               c["Hk"], write_pages=ints(write, dev), n_valid=ints(n_valid, dev), z=c["z"],
                               norm_w=c["norm_w"], eps=eps, o=o, scale=scale)
    torch.cuda.synchronize()
    assert got.data_ptr() == o.data_ptr()
    fp32 = n * (3 * d + 40) * R.U
    fast = 0.0 if c["x"].dtype == torch.float32 else 2.0 ** -20     # SiLU by the fast exponential
    assert torch.equal(c["conv"].double().cpu(), want_c)            # taps move, no arithmetic
    wrote = {p for row in (write or [[r] for r in read]) for p in row}
    worst = 0.0
    tol = R.HALF[c["state"].dtype] + fp32 + 4 * fast
    for p in range(P):
        if p not in wrote:
            assert torch.equal(R.f64(c["state"][p]), want_s[p])
        else:
            worst = max([worst] + [frob_rel(R.f64(c["state"][p, h]), want_s[p, h]) for h in range(Hv)])
    if worst:
        check(name, "state", worst, tol)
    tol = R.HALF[o.dtype] + (2 if c["z"] is not None else 1) * fp32 + 4 * fast
    worst = 0.0
    for b in range(B):
        for t in range(n):
            for h in range(Hv):
                if kept_o[b, t, h]:
                    assert (o[b, t, h] == 7.0).all()
                elif want_o[b, t, h].norm() > 0:
                    worst = max(worst, frob_rel(R.f64(o[b, t, h]), want_o[b, t, h]))
                else:
                    assert (o[b, t, h] == 0).all()
    if worst:
        check(name, "o", worst, tol)


BF, FP = torch.bfloat16, torch.float32


@pytest.mark.parametrize("act", [BF, FP])
@pytest.mark.parametrize("st", [BF, FP])
@pytest.mark.parametrize("Hk,Hv,d,n", [(2, 6, 128, 1), (2, 4, 128, 4), (1, 1, 64, 3), (2, 10, 32, 8), (3, 3, 16, 5),
                                       (1, 7, 16, 2), (1, 3, 128, 8), (2, 2, 128, 5), (4, 12, 128, 2), (1, 9, 128, 3)])
def test_paged_types_and_heads(cuda_device, act, st, Hk, Hv, d, n):
    B, P = 5, 24
    c = case(cuda_device, B, n, Hk, Hv, d, act, st, P, seed=Hv * d + n, wide=True, gate=n % 2 == 0)
    read = [3, 17, -1, 0, 23]
    run_and_check(f"paged {act} {st} {Hk}/{Hv}x{d} n{n}", c, read, None, None, cuda_device)


@pytest.mark.parametrize("st", [BF, FP])
def test_paged_verify_with_a_page_per_token(cuda_device, st):
    """Ragged drafts, every token's state kept, two readers of one page, pages outside the pool,
    one page named by two tokens of a sequence (the later one's state stays)."""
    B, n, P = 6, 4, 20
    c = case(cuda_device, B, n, 2, 4, 128, BF, st, P, seed=3, gate=True)
    read = [0, 0, 1, -5, P, 2]
    write = [[3, 4, 5, 6], [7, 8, 9, 10], [-1, 1, 1, -1], [11, P, 12, -1], [13, 13, 13, 13], [14, 15, 16, 17]]
    run_and_check(f"paged verify {st}", c, read, write, [4, 3, 4, 2, 9, 0], cuda_device)


def test_paged_nothing_valid_touches_nothing(cuda_device):
    c = case(cuda_device, 3, 2, 1, 2, 32, BF, FP, 4, seed=4)
    run_and_check("paged none valid", c, [0, 1, 2], None, [0, -3, 0], cuda_device)


@pytest.mark.parametrize("act,d", [(FP, 64), (BF, 128)])
def test_paged_nan_in_unused_places(cuda_device, act, d):
    """NaN in tokens behind n_valid, in pages nobody reads and in the page of a fresh sequence's
    neighbour reaches no output."""
    c = case(cuda_device, 3, 3, 2, 4, d, act, FP, 6, seed=5, gate=True)
    for key in ("x", "g", "beta", "z"):
        c[key][0, 1:] = float("nan")
        c[key][2] = float("nan")
    c["state"][3:] = float("nan")
    c["conv"][3:] = float("nan")
    read, valid, write = [0, -1, 1], [1, 3, 0], [[4, 4, 4], [2, -1, 5], [1, 1, 1]]
    o = torch.zeros(3, 3, 4, d, dtype=act, device=cuda_device)
    gdn.gdn_decode_paged(c["x"], c["conv_w"], c["conv"], c["state"], ints(read, cuda_device), c["g"], c["beta"], 2,
                         write_pages=ints(write, cuda_device), n_valid=ints(valid, cuda_device), z=c["z"],
                         norm_w=c["norm_w"], o=o)
    assert torch.isfinite(o).all() and torch.isfinite(c["state"][[0, 1, 2, 4, 5]]).all()
    assert torch.isfinite(c["conv"][[0, 1, 2, 4, 5]]).all() and torch.isnan(c["state"][3]).all()


@pytest.mark.parametrize("act,d,n", [(FP, 32, 3), (BF, 128, 3), (BF, 128, 8), (BF, 64, 4)])
def test_paged_extremes_of_the_gates(cuda_device, act, d, n):
    """alpha = 0 (g = -inf) drops the state, decays of e^-25 a token pass the range that a factor is
    carried in, beta = 0 writes nothing, all beside ordinary heads; a zero k or q stays zero under
    the norm's eps."""
    c = case(cuda_device, 3, n, 1, 4, d, act, FP, 4, seed=6)
    c["g"][0, 1] = float("-inf")
    c["g"][2, :, :2] = -25.0
    c["beta"][1, :, 2] = 0
    c["x"][1, :, :2 * d] = 0
    c["conv"][1, :, :2 * d] = 0
    run_and_check(f"paged gates {act} {d} {n}", c, [0, 1, 2], None, None, cuda_device)


def test_paged_equals_the_dense_decode(cuda_device):
    """Pages in order, no write list: the same call as gdn_decode_tokens."""
    c = case(cuda_device, 4, 4, 16, 48, 128, BF, FP, 4, seed=7)
    conv, state = c["conv"].clone(), c["state"].clone()
    o = gdn.gdn_decode_paged(c["x"], c["conv_w"], c["conv"], c["state"], ints([0, 1, 2, 3], cuda_device), c["g"],
                             c["beta"], 16)
    ref = gdn.gdn_decode_tokens(c["x"].contiguous(), c["conv_w"], conv, c["g"], c["beta"], state, 16)
    assert torch.equal(conv, c["conv"])
    assert frob_rel(R.f64(c["state"]), R.f64(state)) <= 8 * (3 * 128 + 40) * R.U
    assert frob_rel(R.f64(o), R.f64(ref)) <= 2 * R.HALF[BF]


@pytest.mark.parametrize("B,Hk,Hv,d,n,st", [(150, 16, 32, 64, 2, FP), (160, 16, 48, 32, 3, BF), (620, 8, 8, 16, 1, FP),
                                              (300, 16, 16, 16, 5, BF), (700, 16, 48, 16, 2, FP)])
def test_paged_equals_the_dense_decode_for_many_narrow_heads(cuda_device, B, Hk, Hv, d, n, st):
    """Batches that fill the GPU with heads below 128, where a CTA takes several key heads."""
    c = case(cuda_device, B, n, Hk, Hv, d, BF, st, B, seed=d + n)
    conv, state = c["conv"].clone(), c["state"].clone()
    o = gdn.gdn_decode_paged(c["x"], c["conv_w"], c["conv"], c["state"], ints(list(range(B)), cuda_device), c["g"],
                             c["beta"], Hk)
    ref = gdn.gdn_decode_tokens(c["x"].contiguous(), c["conv_w"], conv, c["g"], c["beta"], state, Hk)
    assert torch.equal(conv, c["conv"])
    # either is off by n (3 d + 40) roundings at most, and the fast SiLU, before it is stored
    tol = 2 * (n * (3 * d + 40) * R.U + 4 * 2.0 ** -20)
    assert frob_rel(R.f64(c["state"]), R.f64(state)) <= tol + 2 * (R.HALF[BF] if st == BF else 0)
    assert frob_rel(R.f64(o), R.f64(ref)) <= tol + 2 * R.HALF[BF]


def test_paged_interleaved_pools(cuda_device):
    """Taps and state of a page side by side in one buffer, at page strides that are not dense."""
    c = case(cuda_device, 3, 2, 1, 2, 16, FP, FP, 5, seed=8)
    taps, vals, gap = 3 * 64, 2 * 16 * 16, 24
    buf = torch.full((5, taps + vals + gap), 9.0, device=cuda_device)
    buf[:, :taps] = c["conv"].reshape(5, -1)
    buf[:, taps:taps + vals] = c["state"].reshape(5, -1)
    c["conv"] = buf[:, :taps].unflatten(1, (3, 64))
    c["state"] = buf[:, taps:taps + vals].unflatten(1, (2, 16, 16))
    run_and_check("paged interleaved", c, [4, 0, 2], [[1, 4], [-1, 0], [3, 3]], None, cuda_device)
    assert (buf[:, taps + vals:] == 9.0).all()


def test_paged_far_page(cuda_device):
    """A page that begins behind 2^31 elements of the pool."""
    P, Hv, d = 2800, 48, 128
    state = torch.zeros(P, Hv, d, d, dtype=BF, device=cuda_device)       # 2.2e9 elements
    c = case(cuda_device, 2, 1, 16, Hv, d, BF, BF, 2, seed=9)
    conv = torch.zeros(P, 3, c["conv"].shape[2], dtype=BF, device=cuda_device)
    state[P - 1], conv[P - 1] = c["state"][0], c["conv"][0]
    o = gdn.gdn_decode_paged(c["x"], c["conv_w"], conv, state, ints([P - 1, -1], cuda_device), c["g"], c["beta"], 16,
                             write_pages=ints([[P - 2], [0]], cuda_device))
    near = gdn.gdn_decode_paged(c["x"], c["conv_w"], c["conv"], c["state"], ints([0, -1], cuda_device), c["g"],
                                c["beta"], 16, write_pages=ints([[0], [1]], cuda_device))
    assert torch.equal(o, near) and torch.equal(state[P - 2], c["state"][0]) and torch.equal(state[0], c["state"][1])
    assert torch.equal(conv[P - 2], c["conv"][0])
    gdn.gdn_pages_copy(state, ints([P - 2], cuda_device), ints([P - 1], cuda_device))
    assert torch.equal(state[P - 1], c["state"][0])


def test_paged_captured_and_on_a_stream(cuda_device):
    """Two captured calls replayed over changing page lists equal eager ones, on another stream."""
    c = case(cuda_device, 4, 1, 2, 4, 64, BF, FP, 12, seed=10, gate=True)
    eager = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    read, write = ints([0, 1, 2, 3], cuda_device), ints([[4], [5], [6], [7]], cuda_device)
    run = lambda q, o: gdn.gdn_decode_paged(q["x"], q["conv_w"], q["conv"], q["state"], read, q["g"], q["beta"], 2,  # noqa: E731
                                            write_pages=write, z=q["z"], norm_w=q["norm_w"], o=o)
    o, o_e = (torch.zeros(4, 1, 4, 64, dtype=BF, device=cuda_device) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            run(c, o)
        for a, b in (([0, 1, 2, 3], [4, 5, 6, 7]), ([4, 5, 6, 7], [8, 9, -1, 7])):
            read.copy_(torch.tensor(a)); write.copy_(torch.tensor(b)[:, None])
            graph.replay()
            run(eager, o_e)
            side.synchronize()
            assert torch.equal(o, o_e) and torch.equal(c["state"], eager["state"]) and torch.equal(c["conv"], eager["conv"])


# ---------------------------------------------------------------------------------- pages

def pool_of(dev, shape, dtype, seed):
    return torch.randint(-1000, 1000, shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(dev)


@pytest.mark.parametrize("page_dim", [0, 1])
@pytest.mark.parametrize("page", [(16,), (3, 8), (2, 100, 40), (9, 4096)])
@pytest.mark.parametrize("kind", ["apart", "permute", "chain", "fan", "repeats", "bad"])
def test_pages_copy(cuda_device, page_dim, page, kind):
    P, rng = 37, np.random.default_rng(len(page) * 7 + page_dim)
    shape = (P, *page) if page_dim == 0 else (3, P, *page)
    pool = pool_of(cuda_device, shape, FP, seed=len(kind))
    order = rng.permutation(P)
    if kind == "apart":
        src, dst = order[:15], order[15:30]
    elif kind == "permute":
        src, dst = order, np.arange(P)
    elif kind == "chain":
        src, dst = np.arange(P - 1), np.arange(1, P)
    elif kind == "fan":
        src, dst = np.full(20, order[0]), order[:20]
    elif kind == "repeats":
        src, dst = rng.integers(0, P, 60), rng.integers(0, P, 60)
    else:
        src, dst = np.array([0, -1, 5, P, 2, 3, 2**31 - 1]), np.array([1, 2, -1, 4, P + 3, 3, 6])
    src, dst = [int(v) for v in src], [int(v) for v in dst]
    want = R.copied(pool, pool, src, dst, page_dim)
    gdn.gdn_pages_copy(pool, ints(src, cuda_device), ints(dst, cuda_device), page_dim=page_dim)
    assert torch.equal(pool.cpu(), want)


@pytest.mark.parametrize("n", [1, 2, 33, 1000, 1025, 2048])
def test_pages_copy_long_lists_in_place(cuda_device, n):
    """Every length of list that one call takes, all entries depending on one another."""
    pool = pool_of(cuda_device, (n + 1, 52), FP, seed=n)
    order = np.random.default_rng(n).permutation(n + 1)[:n]
    want = R.copied(pool, pool, [int(v) for v in order], list(range(n)), 0)
    gdn.gdn_pages_copy(pool, ints(order.tolist(), cuda_device), ints(list(range(n)), cuda_device))
    assert torch.equal(pool.cpu(), want)


@pytest.mark.parametrize("n,moves", [(48, 30), (700, 600)])
def test_pages_copy_large_pages(cuda_device, n, moves):
    """More tiles than CTAs: every CTA must see the same moves in the same order."""
    pool = pool_of(cuda_device, (n, 100_000 if n < 100 else 5_000), FP, seed=n)
    order = np.random.default_rng(n).permutation(n)
    src, dst = [int(v) for v in order[:moves // 2]], [int(v) for v in order[moves // 2:moves // 2 * 2]]
    for s, d in ((src, dst), (src + dst, dst + src)):
        want = R.copied(pool, pool, s, d, 0)
        gdn.gdn_pages_copy(pool, ints(s, cuda_device), ints(d, cuda_device))
        assert torch.equal(pool.cpu(), want)


def test_pages_copy_between_pools_and_strided(cuda_device):
    a = pool_of(cuda_device, (6, 5, 2, 24), BF, seed=1)[:, :, :, :16][:, :, :1]     # pages of 16 in wider rows
    b = pool_of(cuda_device, (9, 5, 1, 16), BF, seed=2)
    src, dst = [0, 3, 5, 5], [8, 1, 2, 8]
    a0 = a.movedim(1, 0)                                    # [layers, P, ...] by strides
    b0 = b.movedim(1, 0)
    want = R.copied(a0, b0, src, dst, 1)
    gdn.gdn_pages_copy(a0, ints(src, cuda_device), ints(dst, cuda_device), dst_pool=b0, page_dim=1)
    assert torch.equal(b0.cpu(), want)


@pytest.mark.parametrize("P,n", [(1, 1), (5, 3), (40, 64), (3000, 700), (70000, 2048)])
def test_pages_take_and_ref(cuda_device, P, n):
    rng = np.random.default_rng(P)
    refs = rng.integers(-1, 3, P)
    src = [int(v) for v in rng.integers(-2, P + 2, n)]
    t = ints(refs.tolist(), cuda_device)
    want, out = R.taken(refs.tolist(), src) if P < 10000 else (None, None)
    got = gdn.gdn_pages_take(t, src=ints(src, cuda_device))
    if want is None:
        free = np.flatnonzero(refs <= 0)
        ok = [0 <= s < P and refs[s] > 0 for s in src]
        out = [int(free[sum(ok[:i])]) if ok[i] else -1 for i in range(n)]
        want = refs.copy()
        want[[p for p in out if p >= 0]] = 1
        want = want.tolist()
    assert got.tolist() == out and t.tolist() == want
    pages = [int(v) for v in rng.integers(-2, P + 2, 3 * n)]
    for delta in (1, -1, -2):
        count = np.array(t.tolist())
        for p in pages:
            if 0 <= p < P:
                count[p] += delta
        for p in pages:
            if 0 <= p < P:
                count[p] = max(count[p], 0)
        gdn.gdn_pages_ref(t, ints(pages, cuda_device), delta)
        assert t.tolist() == count.tolist()


@pytest.mark.parametrize("P,share", [(1, 0.5), (2, 0.5), (9, 0.0), (9, 1.0), (64, 0.5), (1025, 0.2), (5000, 0.7)])
def test_pages_compact(cuda_device, P, share):
    rng = np.random.default_rng(P)
    refs = np.where(rng.random(P) < share, rng.integers(1, 4, P), rng.integers(-1, 1, P))
    table = [int(v) for v in rng.integers(-2, P + 2, (7, 5)).reshape(-1)]
    pools = [pool_of(cuda_device, (2, P, 12), FP, 1), pool_of(cuda_device, (2, P, 3, 8), BF, 2)]
    new, tab, m, n_live, back, holes = R.planned(refs.tolist(), table)
    want = [R.copied(p, p, back, holes, 1) for p in pools]
    t, tb = ints(refs.tolist(), cuda_device), ints(table, cuda_device).reshape(7, 5)
    got_map, got_live = gdn.gdn_pages_compact(t, tb, pools, page_dim=1)
    assert got_live.tolist() == [n_live] and got_map.tolist() == m
    assert t.tolist() == new and tb.reshape(-1).tolist() == tab
    for a, b in zip(pools, want):
        assert torch.equal(a.cpu(), b)


def test_nothing_to_do(cuda_device):
    """Empty batches, lists and pools are no-ops."""
    dev = cuda_device
    e = lambda *s, dtype=FP: torch.empty(s, dtype=dtype, device=dev)  # noqa: E731
    none = ints([], dev)
    pool = pool_of(dev, (3, 16), FP, 1)
    before = pool.clone()
    gdn.gdn_pages_copy(pool, none, none)
    gdn.gdn_pages_copy(pool, none, none, plain=True)
    assert gdn.gdn_pages_take(ints([0, 0], dev), n=0).numel() == 0
    assert gdn.gdn_pages_fork(ints([1, 0, 0], dev), none, pool).numel() == 0
    gdn.gdn_pages_ref(ints([1], dev), none, -1)
    new, live = gdn.gdn_pages_compact(none, None, e(0, 16))
    assert new.numel() == 0 and live.tolist() == [0]
    new, live = gdn.gdn_pages_compact(ints([0, 0, 0], dev), ints([2, -1], dev), pool)
    assert new.tolist() == [-1, -1, -1] and live.tolist() == [0] and torch.equal(pool, before)
    o = gdn.gdn_decode_paged(e(0, 2, 64), e(64, 4), e(3, 3, 64), e(3, 2, 16, 16), none, e(0, 2, 2), e(0, 2, 2), 1)
    assert o.shape == (0, 2, 2, 16)
    # a pool without pages: every sequence begins here, nothing is stored
    c = case(dev, 2, 2, 1, 2, 16, FP, FP, 1, seed=2)
    a = gdn.gdn_decode_paged(c["x"], c["conv_w"], c["conv"][:0], c["state"][:0], ints([0, 5], dev), c["g"], c["beta"], 1)
    b = gdn.gdn_decode_paged(c["x"], c["conv_w"], c["conv"], c["state"], ints([-1, -1], dev), c["g"], c["beta"], 1)
    assert torch.equal(a, b)


def test_binding_refusals(cuda_device):
    """Wrong shapes, types and layouts are refused before anything changes."""
    dev = cuda_device
    c = case(dev, 2, 2, 1, 2, 16, FP, FP, 4, seed=3)
    args = lambda **kw: {**dict(x=c["x"], conv_w=c["conv_w"], conv_pool=c["conv"], state_pool=c["state"],  # noqa: E731
                                read_pages=ints([0, 1], dev), g=c["g"], beta=c["beta"], Hk=1), **kw}
    for kw in (dict(x=c["x"][:, :, ::2]), dict(x=c["x"].half()), dict(read_pages=ints([0], dev)),
               dict(read_pages=ints([0, 1], dev).long()), dict(g=c["g"][:, :1]), dict(conv_pool=c["conv"][:3]),
               dict(state_pool=c["state"].transpose(2, 3)), dict(z=c["x"][..., :32].unflatten(2, (2, 16))),
               dict(write_pages=ints([0, 1], dev)), dict(o=torch.empty(2, 2, 2, 8, device=dev)), dict(Hk=2)):
        with pytest.raises((ValueError, TypeError)):
            gdn.gdn_decode_paged(**args(**kw))
    with pytest.raises(gdn.GDNError):
        gdn.gdn_decode_paged(**args(o=c["state"].view(-1)[:128].view(2, 2, 2, 16)))
    refs, pool = ints([1, 0, 1], dev), torch.zeros(3, 8, device=dev)
    for bad in (torch.zeros(4, 8, device=dev), torch.zeros(3, 6, device=dev), torch.zeros(3, 8), [pool] * 5,
                torch.zeros(3, 2, 8, device=dev)[:, :, ::2]):
        with pytest.raises(ValueError):
            gdn.gdn_pages_fork(refs, ints([0], dev), bad)
        with pytest.raises(ValueError):
            gdn.gdn_pages_compact(refs, None, bad)
    with pytest.raises(gdn.GDNError):
        gdn.gdn_pages_copy([pool, pool], ints([0], dev), ints([1], dev))
    with pytest.raises(gdn.GDNError):
        gdn.gdn_pages_copy(pool, ints([0] * 2049, dev), ints([1] * 2049, dev))
    assert refs.tolist() == [1, 0, 1]


def test_serving_run(cuda_device):
    """As a server uses them together: a prompt's prefill leaves its state in a page, the page is
    forked for two samples, each decodes in its own page, one drafts two tokens and keeps the
    first, the other leaves, the pool is compacted, and decoding goes on -- against the oracle's
    run of each sample's whole sequence."""
    dev, Hk, Hv, d, P, T = cuda_device, 2, 4, 128, 16, 128
    gen = torch.Generator().manual_seed(21)
    Cc = (2 * Hk + Hv) * d
    x = torch.randn(T + 8, 2, Cc, generator=gen).to(BF)
    x[:T, 1] = x[:T, 0]
    g = -0.3 * torch.rand(T + 8, 2, Hv, generator=gen)
    beta = torch.sigmoid(torch.randn(T + 8, 2, Hv, generator=gen))
    g[:T, 1], beta[:T, 1] = g[:T, 0], beta[:T, 0]
    w = (0.5 * torch.randn(Cc, 4, generator=gen)).to(BF)
    xd, gd, bd, wd = x.to(dev), g.to(dev), beta.to(dev), w.to(dev)
    conv, state = torch.zeros(P, 3, Cc, dtype=BF, device=dev), torch.zeros(P, Hv, d, d, device=dev)
    refs = ints([1, 0, 1] + [0] * (P - 3), dev)                 # pages 0 and 2 belong to others
    prompt = gdn.gdn_pages_take(refs, n=1)
    assert prompt.tolist() == [1]
    taps = torch.empty(1, 3, Cc, dtype=BF, device=dev)
    y = gdn.gdn_conv1d_silu(xd[:T, 0].contiguous(), wd, conv_state_out=taps)
    q, k, v = gdn.qkv_views(y, Hk, Hv, d)
    gdn.gdn_chunk_prefill(q, k, v, gd[:T, 0].contiguous(), bd[:T, 0].contiguous(), block_tokens=T,
                          block_states=state, block_rows=prompt)
    gdn.gdn_pages_copy(taps, ints([0], dev), prompt, dst_pool=conv)
    pages = gdn.gdn_pages_fork(refs, ints([1, 1], dev), [state, conv])
    gdn.gdn_pages_ref(refs, prompt, -1)
    assert pages.tolist() == [3, 4] and refs.tolist()[:5] == [1, 0, 1, 1, 1]
    step = lambda a, b, rows, read, **kw: gdn.gdn_decode_paged(  # noqa: E731
        xd[a:b, rows].transpose(0, 1).contiguous(), wd, conv, state, read, gd[a:b, rows].transpose(0, 1).contiguous(),
        bd[a:b, rows].transpose(0, 1).contiguous(), Hk, **kw)
    outs = [step(T, T + 1, [0, 1], pages)]
    draft = gdn.gdn_pages_take(refs, n=2)                       # pages 1 and 5 for two drafted tokens
    assert draft.tolist() == [1, 5]
    outs.append(step(T + 1, T + 3, [1], pages[1:], write_pages=draft[None]))
    gdn.gdn_pages_ref(refs, torch.cat([pages, draft[1:]]), -1)  # sample 0 leaves; sample 1 lives in page 1
    table = draft[:1].clone()
    gdn.gdn_pages_ref(refs, ints([0], dev), -1)                 # and another request: page 2 moves to 0
    _, n_live = gdn.gdn_pages_compact(refs, table, [state, conv])
    assert n_live.tolist() == [2] and refs.tolist() == [1, 1] + [0] * (P - 2) and table.tolist() == [1]
    outs.append(step(T + 2, T + 4, [1], table))
    last = R.f64(state[1])
    for s, (rows, got) in enumerate([(T + 1, [outs[0][0, 0]]),
                                     (T + 4, [outs[0][1, 0], outs[1][0, 0], outs[2][0, 0], outs[2][0, 1]])]):
        o, S, _ = oracle.layer_prefill(R.f64(x[:rows, s]).numpy(), R.f64(w).numpy(), R.f64(g[:rows, s]).numpy(),
                                       R.f64(beta[:rows, s]).numpy(), Hk, Hv, d, d)
        for a, b in zip(got, o[T:]):
            check("serving run", "o", max(frob_rel(R.f64(a[h]), b[h]) for h in range(Hv)), 2e-2)
    check("serving run", "state", max(frob_rel(last[h], S[0, h]) for h in range(Hv)), 2e-2)


@pytest.mark.parametrize("act", [BF, FP])
def test_prefill_layer_with_the_output_norm(cuda_device, act):
    """A prefilled prompt's last token equals the same token decoded from a page, gate and norm
    included, and the prefill's whole output is gdn_gated_norm's of the plain one."""
    dev, Hk, Hv, d, T = cuda_device, 2, 4, 64, 40
    c = case(dev, 1, T, Hk, Hv, d, act, FP, 2, seed=31, gate=True)
    x, z, g, beta = (c[k].squeeze(0) for k in ("x", "z", "g", "beta"))
    plain = gdn.prefill_layer(x, c["conv_w"], g, beta, Hk, Hv, d)
    o = gdn.prefill_layer(x, c["conv_w"], g, beta, Hk, Hv, d, z=z, norm_w=c["norm_w"])
    assert torch.equal(o, gdn.gdn_gated_norm(plain, z, c["norm_w"]))
    conv, state = torch.zeros_like(c["conv"]), torch.zeros_like(c["state"])
    gdn.prefill_layer(x[:-1], c["conv_w"], g[:-1], beta[:-1], Hk, Hv, d, final_state=state[1:], conv_state_out=conv[1:])
    last = gdn.gdn_decode_paged(x[None, -1:], c["conv_w"], conv, state, ints([1], dev), g[None, -1:], beta[None, -1:], Hk,
                                z=z[None, -1:], norm_w=c["norm_w"])
    # both pass through T tokens of fp32 sums and one storage rounding; o is rounded before its norm
    # in the prefill, behind it in the decode
    tol = 3 * R.HALF[act] + 2 * (3 * d + 40) * R.U * 8 + (2.0 ** -18 if act == BF else 2e-6)
    check(f"prefill norm {act}", "o", frob_rel(R.f64(last[0, 0]), R.f64(o[-1])), tol)

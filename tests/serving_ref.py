"""Plain fp64 forms of the paged decode, the page operations and the norms, for the tests.

Error bounds are counted in roundings: U = 2^-24 is the most that one fp32 rounding is off by,
relative to its result; storing bf16 is off by at most 2^-8."""
import numpy as np
import torch

import oracle

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def f64(t):
    return t.detach().double().cpu()


def gated(o, z, w, eps):
    return o * (o.square().mean(-1, keepdim=True) + eps) ** -0.5 * w * z * torch.sigmoid(z)


def paged(x, conv_w, conv, state, read, g, beta, Hk, write, n_valid, z, norm_w, eps, o, scale=1.0):
    """x [B, n, Cc] ... (torch, any device); read/write/n_valid as lists. Returns fp64 copies of
    (o, state, conv) after the call, not rounded to the storage types."""
    B, n, Cc = x.shape
    P, Hv, d, _ = state.shape
    state_in, conv_in = f64(state), f64(conv)
    state, conv, o = state_in.clone(), conv_in.clone(), f64(o).clone()
    for b in range(B):
        fresh = not 0 <= read[b] < P
        S = np.zeros((1, Hv, d, d)) if fresh else state_in[read[b]][None].numpy()
        taps = np.zeros((1, 3, Cc)) if fresh else conv_in[read[b]][None].numpy()
        valid = n if n_valid is None else min(max(n_valid[b], 0), n)
        for t in range(valid):
            ot, S, taps = oracle.decode_step(f64(x[b, t])[None].numpy(), f64(conv_w).numpy(), taps,
                                             f64(g[b, t])[None].numpy(), f64(beta[b, t])[None].numpy(), S,
                                             Hk, Hv, d, d, scale)
            ot = torch.from_numpy(ot[0])
            if z is not None:
                ot = gated(ot, f64(z[b, t]), f64(norm_w), eps)
            o[b, t] = ot
            to = (read[b] if t == valid - 1 else -1) if write is None else write[b][t]
            if 0 <= to < P:
                state[to], conv[to] = torch.from_numpy(S[0]), torch.from_numpy(taps[0])
    return o, state, conv


def copied(src_pool, dst_pool, src, dst, page_dim):
    """dst_pool after a page copy, on the CPU."""
    a, b = src_pool.cpu(), dst_pool.cpu().clone()
    for s, d in zip(src, dst):
        if 0 <= s < a.shape[page_dim] and 0 <= d < b.shape[page_dim]:
            b.select(page_dim, d).copy_(a.select(page_dim, s))
    return b


def taken(refs, src):
    refs, before, out = list(refs), list(refs), []
    for s in src:
        free = [p for p, r in enumerate(refs) if r <= 0]
        ok = (s is None or (0 <= s < len(refs) and before[s] > 0)) and bool(free)
        out.append(free[0] if ok else -1)
        if ok:
            refs[free[0]] = 1
    return refs, out


def planned(refs, table):
    refs = list(refs)
    P, n_live = len(refs), sum(r > 0 for r in refs)
    holes = [p for p in range(n_live) if refs[p] <= 0]
    back = [p for p in range(n_live, P) if refs[p] > 0]
    where = {p: p for p in range(P) if refs[p] > 0}
    new = [max(r, 0) for r in refs]
    for d, s in zip(holes, back):
        where[s], new[d], new[s] = d, refs[s], 0
    m = [where.get(p, -1) for p in range(P)]
    return new, [m[p] if 0 <= p < P else p for p in table], m, n_live, back, holes


def worst(x, ref, bound):
    """Largest |x - ref| / bound over the elements (bound > 0 wherever they may differ)."""
    err = (f64(x) - ref).abs()
    assert torch.isfinite(f64(x)).all()
    return float((err / bound.clamp(min=1e-300)).max()) if err.numel() else 0.0

"""What the serving and training operators around the mixer cost: cases, inputs, plain forms.

Four operators: the gated delta rule's recurrent form over a pool of state pages ("paged"), the
copying, forking and compacting of those pages ("pages"), the gated norm of the mixer's output
with its backward pass ("gated"), and the residual add with the norm before a block, with its
backward pass ("add"). ``run`` computes them in elementary torch operations in fp32, or, with
``own`` set, by the library's calls; ``exact`` computes them in fp64 on its own.
"""
import math

import torch

own = False

F = {"bf16": torch.bfloat16, "fp32": torch.float32}
DEV = "cuda"
EPS = 1e-6
SIZE = {"bf16": 2, "fp32": 4}


def listed():
    return [
        # one user's next token in a 27B-shaped layer: latency, few bytes; fused output norm
        dict(name="decode 1", op="paged", B=1, n=1, Hk=16, Hv=48, d=128, act="bf16", state="fp32",
             P=8, write="place", ragged=False, gate=True),
        # a full decode batch of the same layer, pages in scattered order; fused output norm
        dict(name="decode 256 fp32 pages", op="paged", B=256, n=1, Hk=16, Hv=48, d=128, act="bf16",
             state="fp32", P=271, write="place", ragged=False, gate=True),
        # a 9B-shaped decode batch whose states are stored in bf16
        dict(name="decode 192 bf16 pages", op="paged", B=192, n=1, Hk=16, Hv=32, d=128, act="bf16",
             state="bf16", P=200, write="place", ragged=False, gate=False),
        # a speculative verify step: up to 4 drafted tokens a sequence, a page for each token's state
        dict(name="verify 48 x 4", op="paged", B=48, n=4, Hk=16, Hv=48, d=128, act="bf16",
             state="fp32", P=250, write="each", ragged=True, gate=False),
        # parallel sampling: one prompt's state page into 8 new pages, in 4 layers
        dict(name="fork 1 into 8", op="pages", kind="fork", P=24, n=8, L=4, Hk=16, Hv=48, d=128,
             state="fp32"),
        # a beam search step: 64 beams take their parents' pages, in place, parents repeated
        dict(name="beam reorder 64", op="pages", kind="reorder", P=72, n=64, L=4, Hk=16, Hv=32, d=128,
             state="bf16"),
        # the pool is squeezed to its front after half of its requests have left
        dict(name="compact 256", op="pages", kind="compact", P=256, n=131, L=1, Hk=16, Hv=48, d=128,
             state="fp32"),
        # the output norm of a decode batch
        dict(name="gated norm 64", op="gated", T=64, H=48, d=128, act="bf16", back=False, wide=True),
        # the output norm of a long prefill
        dict(name="gated norm 65536", op="gated", T=65536, H=48, d=128, act="bf16", back=False, wide=True),
        # its backward pass for a training batch
        dict(name="gated norm backward 8192", op="gated", T=8192, H=48, d=128, act="bf16", back=True,
             wide=False),
        # residual add and norm of a decode batch
        dict(name="add norm 64", op="add", T=64, D=4096, act="bf16", res="bf16", back=False),
        # its backward pass for a training batch with the residual stream in fp32
        dict(name="add norm backward 16384", op="add", T=16384, D=4096, act="bf16", res="fp32", back=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["paged", "paged", "pages", "pages", "gated", "add"])
    if op == "paged":
        d = rng.choice([128, 128, 128, 64, 32, 16])
        Hk, Hv = rng.choice([(16, 48), (16, 32), (4, 12), (8, 8), (2, 10), (1, 4)])
        act = rng.choice(["bf16", "bf16", "fp32"])
        c = dict(op=op, B=_log(rng, 1, 160), n=rng.randint(1, 8), Hk=Hk, Hv=Hv, d=d, act=act,
                 state=rng.choice(["fp32", "bf16"]), P=0, write=rng.choice(["place", "each"]),
                 ragged=rng.random() < 0.5, gate=rng.random() < 0.5)
        if c["write"] == "each":
            c["B"] = min(c["B"], 40)
        c["P"] = c["B"] * ((1 + c["n"]) if c["write"] == "each" else 1) + rng.randint(1, 9)
        return c
    if op == "pages":
        kind = rng.choice(["fork", "reorder", "compact"])
        d = rng.choice([128, 128, 64, 16])
        n = _log(rng, 1, 160 if d == 128 else 700)
        P = n + rng.randint(2, 40) + (n if kind == "fork" else 0)
        Hk, Hv = rng.choice([(16, 48), (16, 32), (4, 12)])
        L = rng.choice([1, 2, 3])
        if d == 128 and P * L > 300:
            L = 1
        return dict(op=op, kind=kind, P=P, n=n, L=L, Hk=Hk, Hv=Hv, d=d, state=rng.choice(["fp32", "bf16"]))
    if op == "gated":
        return dict(op=op, T=_log(rng, 1, 30000), H=rng.choice([48, 32, 12, 5, 1]), d=rng.choice([128, 128, 64, 32, 16]),
                    act=rng.choice(["bf16", "bf16", "fp32"]), back=rng.random() < 0.6, wide=rng.random() < 0.5)
    return dict(op=op, T=_log(rng, 1, 20000), D=rng.choice([4096, 8192, 2048, _log(rng, 64, 8192), _log(rng, 64, 8192)]),
                act=rng.choice(["bf16", "bf16", "fp32"]), res=rng.choice(["bf16", "fp32"]), back=rng.random() < 0.6)


class State:
    pass


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _order(n, seed):
    return torch.randperm(n, generator=torch.Generator().manual_seed(seed)).tolist()


def prepare(case, seed):
    s, g, c = State(), _gen(seed), case
    s.case = c
    if c["op"] == "paged":
        B, n, P, Cc = c["B"], c["n"], c["P"], (2 * c["Hk"] + c["Hv"]) * c["d"]
        act = F[c["act"]]
        # x is the front of a projection that also gives the output gate z
        proj = _normal(g, (B, n, Cc + c["Hv"] * c["d"]), act)
        s.x, s.z = proj[:, :, :Cc], proj[:, :, Cc:].unflatten(2, (c["Hv"], c["d"]))
        s.conv_w = _normal(g, (Cc, 4), act, 0.5)
        # the plain form writes what is to be dropped to a page behind the pool
        s.conv_all = _normal(g, (P + 1, 3, Cc), act)
        s.state_all = torch.empty((P + 1, c["Hv"], c["d"], c["d"]), dtype=F[c["state"]], device=DEV)
        for p in range(0, P + 1, 64):
            part = s.state_all[p:p + 64]
            part.copy_(torch.randn(part.shape, generator=g, device=DEV) * 0.02)
        s.conv_pool, s.state_pool = s.conv_all[:P], s.state_all[:P]
        s.g = -0.3 * torch.rand((B, n, c["Hv"]), generator=g, device=DEV)
        s.beta = torch.sigmoid(torch.randn((B, n, c["Hv"]), generator=g, device=DEV))
        s.norm_w = (1 + 0.1 * torch.randn(c["d"], generator=g, device=DEV)).to(act)
        pages = _order(P, seed)
        read = pages[:B]
        if B > 4:
            read[B // 2] = -1                       # a request that begins here
        s.read = _ints(read)
        s.write = None
        if c["write"] == "each":
            w = torch.tensor(pages[B:B + B * n], dtype=torch.int32).reshape(B, n)
            if B > 2:
                w[B // 3, 0] = -1                   # a token whose state nobody needs
            s.write = w.to(DEV)
        s.valid = None
        if c["ragged"]:
            s.valid = torch.randint(0, n + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
            s.valid[0] = n
        s.o = torch.zeros((B, n, c["Hv"], c["d"]), dtype=act, device=DEV)
    elif c["op"] == "pages":
        P, n, L, Cc = c["P"], c["n"], c["L"], (2 * c["Hk"] + c["Hv"]) * c["d"]
        s.state_pool = torch.empty((L, P, c["Hv"], c["d"], c["d"]), dtype=F[c["state"]], device=DEV)
        for l in range(L):
            for p in range(0, P, 64):
                part = s.state_pool[l, p:p + 64]
                part.copy_(torch.randn(part.shape, generator=g, device=DEV) * 0.02)
        s.conv_pool = _normal(g, (L, P, 3, Cc), torch.bfloat16)
        pages = _order(P, seed)
        refs = torch.zeros(P, dtype=torch.int32)
        if c["kind"] == "fork":                     # n children of one page (or of a few), others in use
            used = pages[:P - n - 1]
            refs[used] = 1
            s.src = _ints([used[i % max(1, n // 8)] if used else 0 for i in range(n)])
        elif c["kind"] == "reorder":
            beams = pages[:n]
            pick = torch.randint(0, n, (n,), generator=torch.Generator().manual_seed(seed + 1)).tolist()
            s.dst, s.src = _ints(beams), _ints([beams[i] for i in pick])
        else:
            live = pages[:n]
            refs[live] = 1 + torch.arange(n, dtype=torch.int32) % 3
            s.table = _ints(live + [-1])
        s.refs = refs.to(DEV)
    elif c["op"] == "gated":
        T, H, d, act = c["T"], c["H"], c["d"], F[c["act"]]
        s.o = _normal(g, (T, H, d), act, 0.2)
        proj = _normal(g, (T, (2 if c["wide"] else 1) * H * d), act)
        s.z = proj[:, -H * d:].unflatten(1, (H, d))
        s.w = (1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(act)
        s.dy = _normal(g, (T, H, d), act) if c["back"] else None
    else:
        T, D, act, res = c["T"], c["D"], F[c["act"]], F[c["res"]]
        s.x = _normal(g, (T, D), act)
        s.res = _normal(g, (T, D), res, 2.0)
        s.w = (0.1 * torch.randn(D, generator=g, device=DEV)).to(act)
        s.dn = _normal(g, (T, D), act) if c["back"] else None
        s.dh = _normal(g, (T, D), res) if c["back"] else None
    return s


# ------------------------------------------------------------------- the plain forms (fp32)

def _paged(s):
    c = s.case
    B, n, P, Hk, Hv, d = c["B"], c["n"], c["P"], c["Hk"], c["Hv"], c["d"]
    read = s.read.long()
    there = (read >= 0) & (read < P)
    at = read.clamp(0, P - 1)
    zero = torch.zeros((), device=DEV)
    taps = torch.where(there[:, None, None], s.conv_pool.index_select(0, at).float(), zero)
    S = torch.where(there[:, None, None, None], s.state_pool.index_select(0, at).float(), zero)
    win = torch.cat([taps, s.x.float()], 1)
    w = s.conv_w.float()
    y = sum(w[:, j] * win[:, j:j + n] for j in range(4))
    y = y / (1 + torch.exp(-y))
    q, k, v = (t.unflatten(2, (-1, d)) for t in y.split([Hk * d, Hk * d, Hv * d], 2))
    q = (q / torch.sqrt((q * q).sum(-1, keepdim=True) + EPS)).repeat_interleave(Hv // Hk, 2)
    k = (k / torch.sqrt((k * k).sum(-1, keepdim=True) + EPS)).repeat_interleave(Hv // Hk, 2)
    valid = torch.full((B,), n, device=DEV) if s.valid is None else s.valid.long()
    outs = []
    for t in range(n):
        kt, live = k[:, t, :, None, :], t < valid
        Sd = S * torch.exp(s.g[:, t])[..., None, None]
        u = s.beta[:, t, :, None] * (v[:, t] - (Sd * kt).sum(-1))
        Sd = Sd + u[..., None] * kt
        outs.append((Sd * q[:, t, :, None, :]).sum(-1))
        S = torch.where(live[:, None, None, None], Sd, S)
        if s.write is not None:
            to = s.write[:, t].long()
            to = torch.where(live & (to >= 0) & (to < P), to, P)
            s.state_all.index_copy_(0, to, S.to(s.state_all.dtype))
            s.conv_all.index_copy_(0, to, win[:, t + 1:t + 4].to(s.conv_all.dtype))
    if s.write is None:
        to = torch.where(there & (valid > 0), at, P)
        s.state_all.index_copy_(0, to, S.to(s.state_all.dtype))
        last = (valid[:, None] + torch.arange(3, device=DEV))[:, :, None].expand(B, 3, win.shape[2])
        s.conv_all.index_copy_(0, to, win.gather(1, last).to(s.conv_all.dtype))
    o = torch.stack(outs, 1)
    if c["gate"]:
        z = s.z.float()
        o = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS) * s.norm_w.float() * (z / (1 + torch.exp(-z)))
    rows = torch.arange(n, device=DEV)[None] < valid[:, None]
    s.o.copy_(torch.where(rows[..., None, None], o.to(s.o.dtype), s.o))
    return {"o": s.o, "state": s.state_pool, "conv": s.conv_pool}


def _pages(s):
    c, P = s.case, s.case["P"]
    pools = (s.state_pool, s.conv_pool)
    if c["kind"] == "reorder":
        for pool in pools:
            pool.index_copy_(1, s.dst.long(), pool.index_select(1, s.src.long()))
        return {"state": s.state_pool, "conv": s.conv_pool}
    refs = s.refs.clone()
    if c["kind"] == "fork":
        out = torch.argsort((refs > 0).int(), stable=True)[:c["n"]]       # the lowest free pages
        refs.index_fill_(0, out, 1)
        for pool in pools:
            pool.index_copy_(1, out, pool.index_select(1, s.src.long()))
        return {"pages": out.int(), "refs": refs, "state": s.state_pool, "conv": s.conv_pool}
    at, live = torch.arange(P, device=DEV), refs > 0
    n_live = live.sum()
    holes, movers = ~live & (at < n_live), live & (at >= n_live)
    m, half = holes.sum(), P // 2
    dst = torch.argsort((~holes).int(), stable=True)[:half]
    src = torch.argsort((~movers).int(), stable=True)[:half]
    moved = at[:half] < m
    frm = at.clone()                                                      # what each page is to hold
    frm.scatter_(0, dst, torch.where(moved, src, dst))
    for pool in pools:
        pool.copy_(pool.index_select(1, frm))
    new = torch.where(live, at, -1)
    new.scatter_(0, src, torch.where(moved, dst, new.gather(0, src)))
    table = s.table.long()
    table = torch.where(table >= 0, new[table.clamp(min=0)], table)
    refs = torch.where(at < n_live, refs[frm], 0)
    return {"map": new.int(), "table": table.int(), "refs": refs, "live": n_live.int().reshape(1),
            "state": s.state_pool, "conv": s.conv_pool}


def _gated(s):
    o, z, w = s.o.float(), s.z.float(), s.w.float()
    r = torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS)
    xh = o * r
    sg = 1 / (1 + torch.exp(-z))
    if not s.case["back"]:
        return (xh * w * (z * sg)).to(s.o.dtype)
    dy = s.dy.float()
    a = dy * w * (z * sg)
    do = r * (a - xh * (a * xh).mean(-1, keepdim=True))
    dz = dy * xh * w * (sg * (1 + z * (1 - sg)))
    dw = (dy * xh * (z * sg)).sum((0, 1), dtype=torch.float64).float()
    return {"do": do.to(s.o.dtype), "dz": dz.to(s.o.dtype), "dw": dw}


SCALE, W_ADD = 0.5, 1.0      # residual scale, and norm weights kept as their distance from one


def _add(s):
    w = s.w.float() + W_ADD
    if not s.case["back"]:
        h = s.res.float() + SCALE * s.x.float()
        n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * w
        return {"n": n.to(s.x.dtype), "h": h.to(s.res.dtype)}
    h, dn = s.res.float(), s.dn.float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    hh = h * r
    a = dn * w
    dres = s.dh.float() + r * (a - hh * (a * hh).mean(-1, keepdim=True))
    dw = (dn * hh).sum(0, dtype=torch.float64).float()
    return {"dx": (SCALE * dres).to(s.x.dtype), "dres": dres.to(s.res.dtype), "dw": dw}


# ------------------------------------------------------------------- the library's calls

def _own(s):
    import gated_deltanet_mixer_causal_b200 as gdn
    c = s.case
    if c["op"] == "paged":
        gdn.gdn_decode_paged(s.x, s.conv_w, s.conv_pool, s.state_pool, s.read, s.g, s.beta, c["Hk"],
                             write_pages=s.write, n_valid=s.valid, z=s.z if c["gate"] else None,
                             norm_w=s.norm_w if c["gate"] else None, eps=EPS, o=s.o)
        return {"o": s.o, "state": s.state_pool, "conv": s.conv_pool}
    if c["op"] == "pages":
        pools = [s.state_pool, s.conv_pool]
        if c["kind"] == "reorder":
            for pool in pools:
                gdn.gdn_pages_copy(pool, s.src, s.dst, page_dim=1)
            return {"state": s.state_pool, "conv": s.conv_pool}
        refs = s.refs.clone()
        if c["kind"] == "fork":
            out = gdn.gdn_pages_fork(refs, s.src, pools, page_dim=1)
            return {"pages": out, "refs": refs, "state": s.state_pool, "conv": s.conv_pool}
        table = s.table.clone()
        new, n_live = gdn.gdn_pages_compact(refs, table, pools, page_dim=1)
        return {"map": new, "table": table, "refs": refs, "live": n_live,
                "state": s.state_pool, "conv": s.conv_pool}
    if c["op"] == "gated":
        if not c["back"]:
            return gdn.gdn_gated_norm(s.o, s.z, s.w, eps=EPS)
        do, dz, dw = gdn.gdn_gated_norm_bwd(s.o, s.z, s.w, s.dy, eps=EPS)
        return {"do": do, "dz": dz, "dw": dw}
    if not c["back"]:
        n, h = gdn.gdn_add_norm(s.x, s.res, s.w, scale=SCALE, w_add=W_ADD, eps=EPS)
        return {"n": n, "h": h}
    dx, dres, dw = gdn.gdn_add_norm_bwd(s.res, s.w, s.dn, s.dh, scale=SCALE,
                                        w_add=W_ADD, eps=EPS)
    return {"dx": dx, "dres": dres, "dw": dw}


def run(state):
    if own:
        return _own(state)
    return {"paged": _paged, "pages": _pages, "gated": _gated, "add": _add}[state.case["op"]](state)


# ------------------------------------------------------------------- what the work is

def work(case):
    c = case
    if c["op"] == "paged":
        B, n, Cc = c["B"], c["n"], (2 * c["Hk"] + c["Hv"]) * c["d"]
        es, tok = SIZE[c["act"]], n / 2 if c["ragged"] else n            # tokens a sequence, on average
        out = tok if c["write"] == "each" else 1
        vals = c["Hv"] * c["d"]
        page = vals * c["d"] * SIZE[c["state"]] + 3 * Cc * es
        by = B * ((1 + out) * page + tok * (Cc * es + vals * es * (2 if c["gate"] else 1) + 8 * c["Hv"])) + Cc * 4 * es
        return {"bytes": by, "flops": 8 * B * tok * vals * c["d"]}
    if c["op"] == "pages":
        Cc = (2 * c["Hk"] + c["Hv"]) * c["d"]
        page = c["Hv"] * c["d"] * c["d"] * SIZE[c["state"]] + 3 * Cc * 2
        if c["kind"] == "fork":
            pages = c["n"] + max(1, c["n"] // 8)
        elif c["kind"] == "reorder":
            pages = c["n"] * (1 + 0.63)                                   # about 1 - 1/e of the parents are distinct
        else:
            pages = 2 * c["n"] * (c["P"] - c["n"]) / c["P"]               # live pages expected behind the border
        return {"bytes": pages * page * c["L"] + 8 * c["P"], "flops": 0}
    if c["op"] == "gated":
        n = c["T"] * c["H"] * c["d"]
        return {"bytes": n * SIZE[c["act"]] * (5 if c["back"] else 3), "flops": n * (20 if c["back"] else 9)}
    n = c["T"] * c["D"]
    a, r = SIZE[c["act"]], SIZE[c["res"]]
    if c["back"]:                                                         # h, dn, dh in; dres, dx out
        return {"bytes": n * (3 * r + 2 * a), "flops": 14 * n}
    return {"bytes": n * (2 * r + 2 * a), "flops": 6 * n}


# ------------------------------------------------------------------- the definitions in fp64

def _exact_paged(s):
    c = s.case
    n, Hk, Hv, d, G = c["n"], c["Hk"], c["Hv"], c["d"], c["Hv"] // c["Hk"]
    state, conv, o = s.state_pool.double(), s.conv_pool.double(), s.o.double()
    state_in, conv_in = s.state_pool, s.conv_pool
    x, w, z, nw = s.x.double(), s.conv_w.double(), s.z.double(), s.norm_w.double()
    write = None if s.write is None else s.write.tolist()
    valid = [n] * c["B"] if s.valid is None else s.valid.tolist()
    for b, page in enumerate(s.read.tolist()):
        fresh = not 0 <= page < c["P"]
        S = torch.zeros((Hv, d, d), dtype=torch.float64, device=DEV) if fresh else state_in[page].double()
        rows = [torch.zeros_like(w[:, 0])] * 3 if fresh else list(conv_in[page].double())
        for t in range(valid[b]):
            rows = rows[-3:] + [x[b, t]]
            m = w[:, 0] * rows[0] + w[:, 1] * rows[1] + w[:, 2] * rows[2] + w[:, 3] * rows[3]
            m = m * torch.sigmoid(m)
            q, k, v = m[:Hk * d].view(Hk, d), m[Hk * d:2 * Hk * d].view(Hk, d), m[2 * Hk * d:].view(Hv, d)
            q = (q * (q.square().sum(1, keepdim=True) + EPS) ** -0.5)[:, None].expand(Hk, G, d).reshape(Hv, d)
            k = (k * (k.square().sum(1, keepdim=True) + EPS) ** -0.5)[:, None].expand(Hk, G, d).reshape(Hv, d)
            S = S * s.g[b, t].double().exp().view(Hv, 1, 1)
            S = S + torch.einsum("hv,hk->hvk", s.beta[b, t].double()[:, None] * (v - torch.einsum("hvk,hk->hv", S, k)), k)
            out = torch.einsum("hvk,hk->hv", S, q)
            if c["gate"]:
                out = out * (out.square().mean(1, keepdim=True) + EPS) ** -0.5 * nw * z[b, t] * torch.sigmoid(z[b, t])
            o[b, t] = out
            to = page if write is None and t == valid[b] - 1 else -1 if write is None else write[b][t]
            if 0 <= to < c["P"]:
                state[to], conv[to] = S, torch.stack(rows[-3:])
    return {"o": o, "state": state, "conv": conv}


def _exact_pages(s):
    c = s.case
    pools = {"state": s.state_pool.double(), "conv": s.conv_pool.double()}
    before = {"state": s.state_pool, "conv": s.conv_pool}
    refs = s.refs.tolist()
    moves, more = [], {}
    if c["kind"] == "reorder":
        moves = list(zip(s.src.tolist(), s.dst.tolist()))
    elif c["kind"] == "fork":
        new = []
        for page in s.src.tolist():
            to = refs.index(0)
            refs[to] = 1
            new.append(to)
            moves.append((page, to))
        more = {"pages": _ints(new), "refs": _ints(refs)}
    else:
        n_live = sum(r > 0 for r in refs)
        holes = [p for p in range(n_live) if refs[p] == 0]
        back = [p for p in range(n_live, c["P"]) if refs[p] > 0]
        where = {p: p for p in range(c["P"]) if refs[p] > 0}
        for to, page in zip(holes, back):
            moves.append((page, to))
            where[page], refs[to], refs[page] = to, refs[page], 0
        more = {"map": _ints([where.get(p, -1) for p in range(c["P"])]), "refs": _ints(refs),
                "table": _ints([where.get(p, -1) for p in s.table.tolist()]), "live": _ints([n_live])}
    for name, pool in pools.items():
        for page, to in moves:
            pool[:, to] = before[name][:, page].double()
    return {**more, **pools}


def _sum_of_blocks(T, part):
    return sum(part(slice(a, a + 4096)) for a in range(0, T, 4096))


def _exact_gated(s):
    T, w = s.case["T"], s.w.double()
    outs = {"y": [], "do": [], "dz": []}

    def part(rows):
        o, z = s.o[rows].double(), s.z[rows].double()
        rms = (o.square().sum(-1, keepdim=True) / o.shape[-1] + EPS).sqrt()
        gate, slope = z * torch.sigmoid(z), torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)
        if not s.case["back"]:
            outs["y"].append(o / rms * w * gate)
            return 0
        dy = s.dy[rows].double()
        a = dy * gate * w
        outs["do"].append(a / rms - o * (a * o).sum(-1, keepdim=True) / (o.shape[-1] * rms ** 3))
        outs["dz"].append(dy * (o / rms) * w * slope)
        return (dy * gate * o / rms).sum((0, 1))

    dw = _sum_of_blocks(T, part)
    if not s.case["back"]:
        return torch.cat(outs["y"])
    return {"do": torch.cat(outs["do"]), "dz": torch.cat(outs["dz"]), "dw": dw}


def _exact_add(s):
    T, D, w = s.case["T"], s.case["D"], s.w.double() + W_ADD
    outs = {"n": [], "h": [], "dx": [], "dres": []}

    def part(rows):
        h = s.res[rows].double() + (0 if s.case["back"] else SCALE * s.x[rows].double())
        rms = (h.square().sum(-1, keepdim=True) / D + EPS).sqrt()
        if not s.case["back"]:
            outs["n"].append(h / rms * w)
            outs["h"].append(h)
            return 0
        a = s.dn[rows].double() * w
        dres = s.dh[rows].double() + a / rms - h * (a * h).sum(-1, keepdim=True) / (D * rms ** 3)
        outs["dres"].append(dres)
        outs["dx"].append(SCALE * dres)
        return (s.dn[rows].double() * h / rms).sum(0)

    dw = _sum_of_blocks(T, part)
    if not s.case["back"]:
        return {"n": torch.cat(outs["n"]), "h": torch.cat(outs["h"])}
    return {"dx": torch.cat(outs["dx"]), "dres": torch.cat(outs["dres"]), "dw": dw}


def exact(case, seed):
    s = prepare(case, seed)
    return {"paged": _exact_paged, "pages": _exact_pages, "gated": _exact_gated, "add": _exact_add}[case["op"]](s)

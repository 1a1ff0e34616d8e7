"""Cases, plain forms and 64-bit values of the cross-attention and drafted-token operators.

Four operators, by a case's "op":

  cross      attention of n_q decoder rows to an encoder's states of another length (shared heads,
             a length for each sequence), from one row (a generation step) to a whole target
  cross_bwd  its gradients, from the forward's stored out and lse
  tree       one verification step: every node of a tree of drafted tokens attends to its window
             and skips in the cache and to its own ancestors among the drafted tokens
  commit     the accepted path's keys and values go from the drafted tokens into the cache

Lengths, trees and paths are a function of the case; the numbers are a function of the seed.
"""
import math
import random

import torch

own = False


# ---- cases ---------------------------------------------------------------------------------------
def listed():
    return [
        # one generation step of one sentence against its source: nothing but latency
        dict(name="cross_step_1", op="cross", dtype="bf16", B=1, H=8, Hkv=8, nq=1, nkv=1021, d=64, ragged=False),
        # a generation step of a full batch, four query heads to a key head, sources of unequal length
        dict(name="cross_step_64", op="cross", dtype="bf16", B=64, H=32, Hkv=8, nq=1, nkv=4096, d=128, ragged=True),
        # a small fp32 target against a source of odd length: the precise path
        dict(name="cross_f32", op="cross", dtype="f32", B=2, H=4, Hkv=2, nq=193, nkv=301, d=32, ragged=True),
        # a whole target against a long document: the compute-bound end
        dict(name="cross_long", op="cross", dtype="bf16", B=1, H=16, Hkv=16, nq=8192, nkv=16384, d=128, ragged=False),
        # training in fp32 on short pairs
        dict(name="bwd_f32", op="cross_bwd", dtype="f32", B=1, H=2, Hkv=2, nq=257, nkv=384, d=32, ragged=False),
        # a training batch of padded pairs, shared key heads, odd target length
        dict(name="bwd_batch", op="cross_bwd", dtype="bf16", B=4, H=16, Hkv=4, nq=509, nkv=1024, d=64, ragged=True),
        # training on long documents: the compute-bound end
        dict(name="bwd_long", op="cross_bwd", dtype="bf16", B=1, H=16, Hkv=16, nq=4096, nkv=16384, d=128, ragged=False),
        # a short draft for one sequence: latency
        dict(name="tree_1", op="tree", dtype="bf16", B=1, H=8, T=9, cap=4096, d=64, k=128, pi=64, S=4, ring=False, ragged=False),
        # an ordinary draft for a batch over a compact ring cache
        dict(name="tree_batch", op="tree", dtype="bf16", B=64, H=32, T=16, cap=4096, d=128, k=1024, pi=128, S=31, ring=True, ragged=True),
        # the widest draft: most of the cache is read, by 64 rows a head
        dict(name="tree_wide", op="tree", dtype="bf16", B=64, H=32, T=64, cap=4096, d=128, k=1024, pi=128, S=31, ring=False, ragged=True),
        # a step's accepted tokens of one sequence: latency
        dict(name="commit_1", op="commit", dtype="bf16", B=1, H=8, T=9, L=4, cap=1024, d=64),
        # a step's accepted tokens of a batch
        dict(name="commit_64", op="commit", dtype="bf16", B=64, H=32, T=32, L=8, cap=1025, d=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cross", "cross", "cross_bwd", "cross_bwd", "tree", "tree", "commit"])
    f32 = rng.random() < 0.25
    dtype = "f32" if f32 else "bf16"
    if op in ("cross", "cross_bwd"):
        H = rng.choice([2, 4, 8] if f32 else [4, 8, 16, 32])
        Hkv = H // rng.choice([g for g in (1, 2, 4, 8) if H % g == 0])
        d = rng.choice([32, 64, 100, 128]) if f32 else rng.choice([64, 128])
        B = _log(rng, 1, 4 if f32 else 32)
        nkv = _log(rng, 16, 1000 if f32 else 16384)
        nq = 1 if op == "cross" and rng.random() < 0.3 else _log(rng, 2, 600 if f32 else 8192)
        top = 2 ** 24 if f32 else 2 ** (30 if op == "cross_bwd" else 31)
        while (B * H * nq * nkv > top or B * H * nq > 2 ** 19) and nq > 16:  # what the largest listed case costs
            nq //= 2
        while B * H * nq * nkv > top or B * Hkv * nkv * d > 2 ** 28:
            B = max(1, B // 2)
            nkv = nkv // 2 if B == 1 else nkv
        return dict(op=op, dtype=dtype, B=B, H=H, Hkv=Hkv, nq=nq, nkv=nkv, d=d, ragged=rng.random() < 0.7)
    d = rng.choice([32, 64, 128]) if f32 else rng.choice([64, 128])
    B, H = _log(rng, 1, 4 if f32 else 64), rng.choice([2, 4, 8] if f32 else [8, 16, 32])
    if op == "tree":
        T = _log(rng, 1, 16 if f32 else 64)
        pi, S = rng.choice([(16, 2), (64, 4), (256, 8), (128, 31), (96, 5)])
        k = _log(rng, 8, 256 if f32 else 1024)
        cap = max(_log(rng, 256, 4096), k + 1, S * pi + 1)
        return dict(op=op, dtype=dtype, B=B, H=H, T=T, cap=cap, d=d, k=k, pi=pi, S=S, ring=rng.random() < 0.5, ragged=rng.random() < 0.7)
    T = _log(rng, 1, 64)
    return dict(op=op, dtype=dtype, B=B, H=H, T=T, L=rng.randint(1, min(T, 16)), cap=_log(rng, 64, 2048), d=d)


# ---- what a case fixes: lengths, trees, paths ------------------------------------------------------
def _fixed(case):
    """Lengths, parents and paths of a case, as plain lists."""
    c = {k: v for k, v in case.items() if k != "name"}
    rng = random.Random(repr(sorted(c.items())))
    B = c["B"]
    if c["op"] in ("cross", "cross_bwd"):
        full = c["nkv"]
        return dict(kv_len=[rng.randint(full // 2, full) if c["ragged"] else full for _ in range(B)])
    T = c["T"]
    if c["op"] == "tree":
        # sequences some way into their generation; a ring has wrapped for some of them
        top = 2 * c["cap"] if c["ring"] else c["cap"]
        lens = [rng.randint(top // 2, top) for _ in range(B)]
        nodes = [rng.randint(max(1, T // 2), T) if c["ragged"] else T for _ in range(B)]
        # a node's parent is one of the few drafted before it: chains with side branches
        parents = [[-1 if t == 0 else max(-1, t - 1 - _branch(rng)) for t in range(T)] for _ in range(B)]
        return dict(cache_len=lens, tree_len=nodes, parent=parents)
    L = c["L"]
    lens = [rng.randint(0, 2 * c["cap"]) for _ in range(B)]
    count = [rng.randint(1, L) for _ in range(B)]
    paths = [sorted(rng.sample(range(T), L)) for _ in range(B)]
    return dict(cache_len=lens, n_path=count, path=paths)


def _branch(rng):
    return 0 if rng.random() < 0.4 else rng.randint(1, 6)


def _depths(parent):
    out = []
    for p in parent:
        out.append(0 if p < 0 else out[p] + 1)
    return out


def _keys(i, k, pi, S):
    """Window keys and skip keys of position i."""
    return list(range(max(0, i - k), i + 1)), [i - m * pi for m in range(1, S + 1) if m * pi > k and i - m * pi >= 0]


# ---- inputs ----------------------------------------------------------------------------------------
def prepare(case, seed):
    c, f = case, _fixed(case)
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32

    def normal(*shape, std=1.0, dtype=dt):
        return torch.empty(shape, dtype=dtype, device=dev).normal_(0.0, std, generator=g)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    s = dict(case=dict(c))
    B, H, d = c["B"], c["H"], c["d"]
    if c["op"] in ("cross", "cross_bwd"):
        s["q"] = normal(B, H, c["nq"], d)
        s["k"] = normal(B, c["Hkv"], c["nkv"], d)
        s["v"] = normal(B, c["Hkv"], c["nkv"], d)
        s["kv_len"] = ints(f["kv_len"]) if c["ragged"] else None
        if c["op"] == "cross_bwd":  # a training step has the forward's out and lse at hand
            s["dout"] = normal(B, H, c["nq"], d)
            s["out"], s["lse"] = _cross(s)
        return s
    if c["op"] == "tree":
        s["q"], s["k_tree"], s["v_tree"] = (normal(B, H, c["T"], d) for _ in range(3))
        s["kcache"], s["vcache"] = normal(B, H, c["cap"], d), normal(B, H, c["cap"], d)
        s["w_g"] = normal(H, d, std=1 / math.sqrt(d), dtype=torch.float32)
        s["b_g"] = normal(H, std=0.7, dtype=torch.float32)
        s["parent"], s["cache_len"] = ints(f["parent"]), ints(f["cache_len"])
        s["tree_len"] = ints(f["tree_len"]) if c["ragged"] else None
        # rows past a sequence's nodes keep what they hold
        s["out"] = torch.zeros(B, H, c["T"], d, dtype=dt, device=dev)
        s["lse"] = torch.zeros(B, H, c["T"], dtype=torch.float32, device=dev)
        return s
    s["k_tree"], s["v_tree"] = normal(B, H, c["T"], d), normal(B, H, c["T"], d)
    s["kcache"], s["vcache"] = normal(B, H, c["cap"], d), normal(B, H, c["cap"], d)
    s["path"], s["n_path"], s["cache_len"] = ints(f["path"]), ints(f["n_path"]), ints(f["cache_len"])
    return s


# ---- the plain forms ---------------------------------------------------------------------------------
def _scores(s):
    """Scaled scores [B, Hkv, G nq, nkv] in fp32, -inf behind each source's end."""
    q, k = s["q"], s["k"]
    B, H, nq, d = q.shape
    Hkv, nkv = k.shape[1], k.shape[2]
    x = (q.float().reshape(B, Hkv, -1, d) * (1.0 / math.sqrt(d))) @ k.float().transpose(2, 3)
    if s["kv_len"] is not None:
        past = torch.arange(nkv, device=q.device)[None, :] >= s["kv_len"][:, None]
        x.masked_fill_(past[:, None, None, :], -math.inf)
    return x


def _cross(s):
    q, v = s["q"], s["v"]
    B, H, nq, d = q.shape
    x = _scores(s)
    m = x.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x.sub_(m))
    tot = p.sum(dim=-1, keepdim=True)
    out = (p @ v.float()) / torch.where(tot == 0, 1.0, tot)
    lse = m + torch.log(tot)
    return out.reshape(B, H, nq, d).to(q.dtype), lse.reshape(B, H, nq)


def _cross_bwd(s):
    q, k, v = s["q"], s["k"], s["v"]
    B, H, nq, d = q.shape
    Hkv = k.shape[1]
    qf, do = (t.float().reshape(B, Hkv, -1, d) for t in (q, s["dout"]))
    lse = s["lse"].reshape(B, Hkv, -1, 1)
    p = torch.exp(_scores(s).sub_(torch.where(lse == -math.inf, 0.0, lse)))
    dv = p.transpose(2, 3) @ do
    row = (do * s["out"].float().reshape(B, Hkv, -1, d)).sum(dim=-1, keepdim=True)
    ds = (do @ v.float().transpose(2, 3)).sub_(row).mul_(p).mul_(1.0 / math.sqrt(d))
    dq = (ds @ k.float()).reshape(B, H, nq, d)
    dk = ds.transpose(2, 3) @ qf
    return dq.to(q.dtype), dk.to(q.dtype), dv.to(q.dtype)


def _tree(s):
    c = s["case"]
    q, kt, vt, kc, vc = (s[n].float() for n in ("q", "k_tree", "v_tree", "kcache", "vcache"))
    B, H, T, d = q.shape
    dev, C = q.device, c["cap"]
    parent, length = s["parent"].long(), s["cache_len"].long()
    node = torch.arange(T, device=dev)
    above = ((parent[:, :, None] == node) | (node[:, None] == node)).float()  # itself and its parent
    for _ in range(max(1, T - 1).bit_length()):  # reach doubles: itself and all its ancestors
        above = (above @ above).clamp_(max=1.0)
    depth = above.sum(dim=-1).long() - 1
    pos = length[:, None] + depth  # [B, T]
    slot = torch.arange(C, device=dev)
    at = slot + C * torch.div(length[:, None] - 1 - slot, C, rounding_mode="floor") if c["ring"] else slot.expand(B, C)
    held = (at >= 0) & (at < length[:, None])
    key_at = torch.cat([at, pos], dim=1)[:, None, :]  # [B, 1, C + T]
    seen = torch.cat([held[:, None, :].expand(B, T, C), above > 0], dim=2)
    back = pos[:, :, None] - key_at
    window = seen & (back >= 0) & (back <= c["k"])
    skip = seen & (back > c["k"]) & (back % c["pi"] == 0) & (back <= c["S"] * c["pi"])
    z = (q * s["w_g"][:, None, :]).sum(dim=-1) + s["b_g"][:, None]
    tail = torch.log1p(torch.exp(-z.abs()))  # log sigmoid(z) = min(z, 0) - log(1 + e^-|z|)
    lo, hi = (torch.clamp(z, max=0.0) - tail)[..., None], (torch.clamp(-z, max=0.0) - tail)[..., None]
    x = torch.cat([q @ kc.transpose(2, 3), q @ kt.transpose(2, 3)], dim=3) * (1.0 / math.sqrt(d))
    x = torch.where(window[:, None], x + lo, torch.where(skip[:, None], x + hi, -math.inf))
    m = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x.sub_(m))
    tot = p.sum(dim=-1, keepdim=True)
    out = (p[..., :C] @ vc + p[..., C:] @ vt) / tot
    lse = (m + torch.log(tot))[..., 0]
    if s["tree_len"] is not None:
        live = (node[None, :] < s["tree_len"][:, None])[:, None, :]
        out = torch.where(live[..., None], out, s["out"].float())
        lse = torch.where(live, lse, s["lse"])
    return out.to(s["q"].dtype), lse


def _commit(s):
    kc, vc, n = s["kcache"], s["vcache"], s["cache_len"]
    B, H, C, d = kc.shape
    L = s["path"].shape[1]
    e = torch.arange(L, device=kc.device)
    b = torch.arange(B, device=kc.device)[:, None]
    slot, node = (n[:, None].long() + e) % C, s["path"].long()
    live = (e < s["n_path"][:, None])[:, :, None, None]
    kc[b, :, slot] = torch.where(live, s["k_tree"][b, :, node], kc[b, :, slot])
    vc[b, :, slot] = torch.where(live, s["v_tree"][b, :, node], vc[b, :, slot])
    n += s["n_path"]
    return kc, vc, n


def run(state):
    s, c = state, state["case"]
    if own:
        import periodic_sparse_attention_b200 as pia

        if c["op"] == "cross":
            return pia.pi_attn_cross_fwd(s["q"], s["k"], s["v"], kv_len=s["kv_len"])
        if c["op"] == "cross_bwd":
            return pia.pi_attn_cross_bwd(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], kv_len=s["kv_len"])
        if c["op"] == "tree":
            return pia.pi_attn_decode_tree(s["q"], s["k_tree"], s["v_tree"], s["kcache"], s["vcache"], s["w_g"], s["b_g"], s["parent"], s["cache_len"],
                                           c["k"], c["pi"], c["S"], tree_len=s["tree_len"], ring=c["ring"], out=s["out"], lse=s["lse"])
        pia.pi_attn_cache_commit(s["kcache"], s["vcache"], s["k_tree"], s["v_tree"], s["path"], s["n_path"], s["cache_len"], ring=True)
        return s["kcache"], s["vcache"], s["cache_len"]
    return {"cross": _cross, "cross_bwd": _cross_bwd, "tree": _tree, "commit": _commit}[c["op"]](s)


# ---- what a pass cannot do without -------------------------------------------------------------------
def work(case):
    c, f = case, _fixed(case)
    e = 2 if c["dtype"] == "bf16" else 4
    B, H, d = c["B"], c["H"], c["d"]
    if c["op"] in ("cross", "cross_bwd"):
        rows, keys = B * H * c["nq"], sum(f["kv_len"])
        pairs = H * c["nq"] * keys
        if c["op"] == "cross":
            return dict(bytes=2 * rows * d * e + 4 * rows + 2 * c["Hkv"] * keys * d * e, flops=4 * pairs * d)
        # q, out, dout, lse, k, v in; dq, dk, dv out (whole, the padding's zeros too)
        return dict(bytes=4 * rows * d * e + 4 * rows + 2 * c["Hkv"] * (keys + B * c["nkv"]) * d * e, flops=10 * pairs * d)
    if c["op"] == "tree":
        bytes_, pairs = 4 * H * (d + 1), 0
        for n, t, parent in zip(f["cache_len"], f["tree_len"], f["parent"]):
            depth = _depths(parent[:t])
            rows = set()
            by_depth = {}
            for x in sorted(set(depth)):
                w, p = _keys(n + x, c["k"], c["pi"], c["S"])
                held = [j for j in w + p if j < n]
                rows.update(held)
                by_depth[x] = len(held)
            pairs += sum(by_depth[x] + x + 1 for x in depth)
            bytes_ += H * (2 * len(rows) * d * e + 4 * t * d * e + 4 * t)
        return dict(bytes=bytes_, flops=4 * H * pairs * d)
    return dict(bytes=4 * H * sum(f["n_path"]) * d * e, flops=0)


# ---- the same outputs from the definition, in 64 bits ------------------------------------------------
def exact(case, seed):
    c, f = case, _fixed(case)
    s = prepare(case, seed)
    B, H, d = c["B"], c["H"], c["d"]
    t64 = dict(dtype=torch.float64, device="cuda")
    if c["op"] in ("cross", "cross_bwd"):
        share = H // c["Hkv"]
        nq, nkv = c["nq"], c["nkv"]
        out, lse, dq = torch.zeros(B, H, nq, d, **t64), torch.full((B, H, nq), -math.inf, **t64), torch.zeros(B, H, nq, d, **t64)
        dk, dv = torch.zeros(B, c["Hkv"], nkv, d, **t64), torch.zeros(B, c["Hkv"], nkv, d, **t64)
        for b in range(B):
            n = f["kv_len"][b]
            if n == 0:
                continue
            for h in range(H):
                q, k, v = s["q"][b, h].double(), s["k"][b, h // share, :n].double(), s["v"][b, h // share, :n].double()
                x = torch.einsum("ic,jc->ij", q, k) / math.sqrt(d)
                lse[b, h] = torch.logsumexp(x, dim=1)
                w = torch.exp(x - lse[b, h][:, None])
                out[b, h] = torch.einsum("ij,jc->ic", w, v)
                if c["op"] == "cross_bwd":
                    go = s["dout"][b, h].double()
                    gx = w * (torch.einsum("ic,jc->ij", go, v) - (go * out[b, h]).sum(dim=1, keepdim=True)) / math.sqrt(d)
                    dq[b, h] = torch.einsum("ij,jc->ic", gx, k)
                    dk[b, h // share, :n] += torch.einsum("ij,ic->jc", gx, q)
                    dv[b, h // share, :n] += torch.einsum("ij,ic->jc", w, go)
        return (out, lse) if c["op"] == "cross" else (dq, dk, dv)
    if c["op"] == "tree":
        out, lse = torch.zeros(B, H, c["T"], d, **t64), torch.zeros(B, H, c["T"], **t64)
        w_g, b_g = s["w_g"].double(), s["b_g"].double()
        for b in range(B):
            n, parent = f["cache_len"][b], f["parent"][b]
            for t in range(f["tree_len"][b] if c["ragged"] else c["T"]):
                line = [t]  # the node and its ancestors, deepest first
                while parent[line[-1]] >= 0:
                    line.append(parent[line[-1]])
                i = n + len(line) - 1
                win, skp = _keys(i, c["k"], c["pi"], c["S"])
                rows_c = [j % c["cap"] for j in win + skp if j < n]
                rows_t = [line[i - j] for j in win + skp if j >= n]
                is_win = torch.tensor([j >= i - c["k"] for j in win + skp if j < n] + [j >= i - c["k"] for j in win + skp if j >= n], device="cuda")
                kk = torch.cat([s["kcache"][b][:, rows_c], s["k_tree"][b][:, rows_t]], dim=1).double()
                vv = torch.cat([s["vcache"][b][:, rows_c], s["v_tree"][b][:, rows_t]], dim=1).double()
                q = s["q"][b, :, t].double()
                z = (q * w_g).sum(dim=1) + b_g
                prior = torch.where(is_win[None, :], -torch.log1p(torch.exp(-z))[:, None], -torch.log1p(torch.exp(z))[:, None])
                x = torch.einsum("hc,hjc->hj", q, kk) / math.sqrt(d) + prior
                lse[b, :, t] = torch.logsumexp(x, dim=1)
                out[b, :, t] = torch.einsum("hj,hjc->hc", torch.exp(x - lse[b, :, t][:, None]), vv)
        return out, lse
    kc, vc = s["kcache"].clone(), s["vcache"].clone()
    for b in range(B):
        for e in range(f["n_path"][b]):
            kc[b, :, (f["cache_len"][b] + e) % c["cap"]] = s["k_tree"][b, :, f["path"][b][e]]
            vc[b, :, (f["cache_len"][b] + e) % c["cap"]] = s["v_tree"][b, :, f["path"][b][e]]
    return kc.double(), vc.double(), None

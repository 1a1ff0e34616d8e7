"""Cross attention, its gradients, the tree of drafted tokens and the cache commit in 64 bits, from
their definitions, with the error bounds the kernels are held to.

Bounds.  Let u be the unit roundoff of the operands of the last products (bf16 2^-8 on the tensor
cores, where p and ds are rounded to bf16; 2^-24 else), w that of the output's type and
e = (terms + 16) 2^-24 the worst relative error of an fp32 sum of so many terms (against the sum of
the terms' magnitudes).  With s the score, a score is off by at most e_d S, S = tau sum_c |q_c k_c|;
p by that times p (twice: once in the weight, once in the sum it is divided by).  Then, elementwise,
  out   (u + 2 e S + e) sum_j p |v| + w |out|
  lse   e S + 2^-20 (1 + |lse|)          (2^-20: the exponential and logarithm instructions)
  D     dD = sum_c |dout_c| (error of out_c) + e sum_c |dout_c out_c|
  ds    d_ij = p (|g| + |D|) (u + 2 e S + 2 e) + p (dD + e sum_c |dout_c v_c|),  g = dout . v
  Underflow adds to these: the exponential gives 0 below 2^-126, the least normal fp32 (and bf16)
  number, so a weight p is off by up to t = 2^-126 besides, ds by t (|g| + |D|), and what a weight or
  an output loses in its own type's subnormal range is below t again: 2 t a weight, t an output.
  dq    tau sum_j d_ij |k_j| + e tau sum_j |ds k| + w |dq|;  dk alike;  dv  (u + 2 e S + e) sum p |dout| + w |dv|
"""
import math

import torch

TINY = 2.0 ** -126
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _e(terms):
    return (terms + 16) * 2.0 ** -24


def cross(q, k, v, kv_len=None, dout=None, u=None):
    """Values and bounds: dict of name -> (value, bound) for out, lse and, with dout, dq, dk, dv."""
    B, H, nq, d = q.shape
    Hkv, nkv = k.shape[1], k.shape[2]
    G, tau, w = H // Hkv, 1.0 / math.sqrt(d), U[q.dtype]
    u = U[q.dtype] if u is None else u
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device=q.device)  # noqa: E731
    val = dict(out=z(B, H, nq, d), lse=torch.full((B, H, nq), -math.inf, dtype=torch.float64, device=q.device),
               dq=z(B, H, nq, d), dk=z(B, Hkv, nkv, d), dv=z(B, Hkv, nkv, d))
    tol = {n: torch.zeros_like(t) for n, t in val.items()}
    eb, en, er = _e(d), _e(nkv), _e(G * nq)
    for b in range(B):
        n = nkv if kv_len is None else int(kv_len[b])
        if n == 0:
            continue
        for h in range(H):
            Q, K, V = q[b, h].double(), k[b, h // G, :n].double(), v[b, h // G, :n].double()
            s = tau * Q @ K.T
            S = tau * Q.abs() @ K.abs().T
            lse = torch.logsumexp(s, dim=1)
            p = torch.exp(s - lse[:, None])
            out = p @ V
            val["out"][b, h], val["lse"][b, h] = out, lse
            dp = 2 * eb * S.amax(dim=1, keepdim=True) + 2.0 ** -20  # relative error of a weight
            to = (p * (u + dp + en) + 2 * TINY) @ V.abs() + w * out.abs() + TINY
            tol["out"][b, h] = to
            tol["lse"][b, h] = eb * S.amax(dim=1) + 2.0 ** -20 * (1 + lse.abs())
            if dout is None:
                continue
            G_ = dout[b, h].double()
            D = (G_ * out).sum(dim=1, keepdim=True)
            dD = (G_.abs() * to).sum(dim=1, keepdim=True) + eb * (G_ * out).abs().sum(dim=1, keepdim=True)
            g = G_ @ V.T
            ds = p * (g - D)
            te = (p * (dp + 2 * eb) + 2 * TINY) * (g.abs() + D.abs()) + ds.abs() * u + p * (dD + eb * (G_.abs() @ V.abs().T))
            val["dq"][b, h] = tau * ds @ K
            tol["dq"][b, h] = tau * (te + en * ds.abs()) @ K.abs()
            val["dk"][b, h // G, :n] += tau * ds.T @ Q
            tol["dk"][b, h // G, :n] += tau * (te + er * ds.abs()).T @ Q.abs()
            val["dv"][b, h // G, :n] += p.T @ G_
            tol["dv"][b, h // G, :n] += (p * (u + dp + er) + 2 * TINY).T @ G_.abs()
    for n in ("dq", "dk", "dv"):
        tol[n] += w * val[n].abs() + TINY * (val[n] != 0)  # rows behind the states are exactly zero
    return {n: (val[n], tol[n]) for n in val if dout is not None or n in ("out", "lse")}


def depth_of(parent, t):
    x = 0
    while parent[t] >= 0:
        t, x = parent[t], x + 1
    return x


def tree(q, kt, vt, kc, vc, w_g, b_g, parent, cache_len, k, pi, S, tree_len=None, ring=False, u=None):
    """out and lse of the nodes of every tree, (value, bound) each; NaN where a row is not computed."""
    B, H, T, d = q.shape
    C, tau, w = kc.shape[2], 1.0 / math.sqrt(d), U[q.dtype]
    u = U[q.dtype] if u is None else u
    nan = lambda *s: torch.full(s, math.nan, dtype=torch.float64, device=q.device)  # noqa: E731
    val = dict(out=nan(B, H, T, d), lse=nan(B, H, T))
    tol = dict(out=nan(B, H, T, d), lse=nan(B, H, T))
    eb = _e(d)
    for b in range(B):
        n, par = int(cache_len[b]), [int(x) for x in parent[b]]
        for t in range(T if tree_len is None else int(tree_len[b])):
            line = [t]
            while par[line[-1]] >= 0:
                line.append(par[line[-1]])
            i = n + len(line) - 1
            keys = [(j, True) for j in range(max(0, i - k), i + 1)]
            keys += [(i - m * pi, False) for m in range(1, S + 1) if m * pi > k and i - m * pi >= 0]
            old = [(j, win) for j, win in keys if j < n]
            new = [(line[i - j], win) for j, win in keys if j >= n]
            rows = [j % C if ring else j for j, _ in old]
            K = torch.cat([kc[b][:, rows], kt[b][:, [j for j, _ in new]]], dim=1).double()
            V = torch.cat([vc[b][:, rows], vt[b][:, [j for j, _ in new]]], dim=1).double()
            win = torch.tensor([x for _, x in old + new], device=q.device)
            Q = q[b, :, t].double()
            z = (Q * w_g.double()).sum(dim=1) + b_g.double()
            Z = (Q * w_g.double()).abs().sum(dim=1) + b_g.double().abs()
            ls = lambda x: torch.where(x > 0, 0.0, x) - torch.log1p(torch.exp(-x.abs()))  # noqa: E731
            s = tau * torch.einsum("hc,hjc->hj", Q, K) + torch.where(win, ls(z)[:, None], ls(-z)[:, None])
            Sa = tau * torch.einsum("hc,hjc->hj", Q.abs(), K.abs()) + 2 * Z[:, None]
            lse = torch.logsumexp(s, dim=1)
            p = torch.exp(s - lse[:, None])
            out = torch.einsum("hj,hjc->hc", p, V)
            dp = 2 * eb * Sa.amax(dim=1)[:, None] + 2.0 ** -20
            val["out"][b, :, t], val["lse"][b, :, t] = out, lse
            tol["out"][b, :, t] = torch.einsum("hj,hjc->hc", p * (u + dp + _e(len(keys))) + 2 * TINY, V.abs()) + w * out.abs() + TINY
            tol["lse"][b, :, t] = eb * Sa.amax(dim=1) + 2.0 ** -20 * (1 + lse.abs())
    return {n: (val[n], tol[n]) for n in val}


def check(got, want, what):
    """Every element of `got` within the bound of (value, bound); infinities equal."""
    value, bound = want
    g = got.double()
    fin = torch.isfinite(value)
    assert torch.equal(torch.isfinite(g), fin), f"{what}: not finite where it should be, or the other way round"
    assert torch.equal(g[~fin], value[~fin]), f"{what}: wrong infinities"
    over = ((g - value).abs() - bound * 1.02)[fin]  # 1.02: products of two roundings
    worst = float(over.max()) if over.numel() else -1.0
    assert worst <= 0.0, f"{what}: {int((over > 0).sum())} of {over.numel()} elements past their bound, by up to {worst:.3g}"

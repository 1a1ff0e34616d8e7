"""Rows whose keys go through the workspace in more than eight shares (B200 only): trees with rows behind
the nodes, refused lengths and parents, and guards around a workspace that is used."""
import math
import random

import pytest
import torch

import periodic_sparse_attention_b200 as pia
from periodic_sparse_attention_b200 import build as pbuild
from tests import rows_ref as ref
from tests.test_gpu_tree import ints, make_tree

pytestmark = pytest.mark.gpu

B, H, T, CAP, D, K, PI, S = 3, 1, 9, 4200, 64, 4000, 512, 8
TOP = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def _library():
    pbuild.build()
    pia.load()
    yield
    torch.cuda.synchronize()


def workspace_bytes():
    return pia.load().pi_attn_decode_tree_workspace_bytes(B, H, T, D, K, PI, S, pia.PI_ATTN_BF16, 0)


def inputs(seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, kt, vt, kc, vc = (r(B, H, n, D).to(torch.bfloat16) for n in (T, T, T, CAP, CAP))
    rng = random.Random(seed)
    return [q, kt, vt, kc, vc, r(H, D) / 8, r(H)], [make_tree("random", T, rng) for _ in range(B)]


def run(x, parent, lens, nodes, ring, **kw):
    out, lse = torch.full_like(x[0], 7.0), torch.full((B, H, T), 7.0, device="cuda")
    kw = {"out": out, "lse": lse, **kw}
    return pia.pi_attn_decode_tree(*x, ints(parent), ints(lens), K, PI, S, tree_len=ints(nodes), ring=ring, **kw)


def same(x, parent, lens, nodes, ring, out, lse, rows):
    good = [n if b in rows else 1 for b, n in enumerate(lens)]
    par = [p if b in rows else [-1] * T for b, p in enumerate(parent)]
    live = [n if b in rows else 1 for b, n in enumerate(nodes)]
    want = ref.tree(*x, par, good, K, PI, S, live, ring, u=2.0 ** -8)
    for b in rows:
        for name, got in (("out", out), ("lse", lse)):
            ref.check(got[b, :, :nodes[b]], tuple(t[b, :, :nodes[b]] for t in want[name]), f"{name} of sequence {b}")
            assert (got[b, :, nodes[b]:] == 7.0).all(), "rows behind the nodes were written"


@pytest.mark.parametrize("ring", [False, True])
def test_rows_behind_the_nodes(ring):
    assert workspace_bytes() > 0  # (more shares than a cluster joins)
    x, parent = inputs()
    lens, nodes = [4100, 70, 9000 if ring else 4200], [9, 0, 5]
    out, lse = run(x, parent, lens, nodes, ring)
    pia.pi_attn_check()
    same(x, parent, lens, nodes, ring, out, lse, (0, 1, 2))


@pytest.mark.parametrize("what", ["length", "negative", "last length", "nodes", "parent"])
@pytest.mark.parametrize("ring", [False, True])
def test_refused_values(what, ring):
    """The error word, and NaN in every row of the sequence (a wrong parent: in every node of it)."""
    assert workspace_bytes() > 0
    x, parent = inputs(1)
    lens, nodes = [4100, 4000, 3000], [9, 5, 7]
    want = list(lens), [list(p) for p in parent], list(nodes)
    if what == "length":
        if ring:
            return  # a ring takes any length, the last few below 2^31 aside
        lens[1] = CAP + 1
    if what == "negative":
        lens[1] = -1
    if what == "last length":
        lens[1] = TOP
    if what == "nodes":
        nodes[1] = T + 1
    if what == "parent":
        parent[1][3] = 3
    out, lse = run(x, parent, lens, nodes, ring)
    with pytest.raises(pia.PiAttnError, match="tree-or-path" if what == "parent" else "cache_len"):
        pia.pi_attn_check()
    n = 5 if what == "parent" else T
    assert out[1, :, :n].isnan().all() and lse[1, :, :n].isnan().all()
    assert (out[1, :, n:] == 7.0).all() and (lse[1, :, n:] == 7.0).all()
    same(x, want[1], want[0], want[2], ring, out, lse, (0, 2))


def test_nothing_is_written_outside_a_used_workspace():
    from tests.test_gpu_guards import Guarded

    x, parent = inputs(2)
    lens, nodes = [4100, 4000, 3000], [9, 5, 7]
    need = workspace_bytes()
    assert need > 0
    out, lse, ws = Guarded(x[0].shape, torch.bfloat16), Guarded((B, H, T), torch.float32), Guarded((need,), torch.uint8)
    out.t.fill_(7.0), lse.t.fill_(7.0)
    run(x, parent, lens, nodes, False, out=out.t, lse=lse.t, workspace=ws.t)
    pia.pi_attn_check()
    for name, t in (("out", out), ("lse", lse), ("workspace", ws)):
        t.check(name)
    same(x, parent, lens, nodes, False, out.t, lse.t, (0, 1, 2))
    # cross attention of few rows over many states
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(1, h, n, 128, generator=g, device="cuda").to(torch.bfloat16) for h, n in ((4, 3), (2, 9100), (2, 9100)))
    need = pia.load().pi_attn_cross_fwd_workspace_bytes(1, 4, 2, 3, 9100, 128, pia.PI_ATTN_BF16, 0)
    assert need > 0
    out, lse, ws = Guarded(q.shape, torch.bfloat16), Guarded((1, 4, 3), torch.float32), Guarded((need,), torch.uint8)
    pia.pi_attn_cross_fwd(q, k, v, out=out.t, lse=lse.t, workspace=ws.t)
    pia.pi_attn_check()
    for name, t in (("out", out), ("lse", lse), ("workspace", ws)):
        t.check(name)
    want = ref.cross(q, k, v, None, u=2.0 ** -8)
    ref.check(out.t, want["out"], "out")
    ref.check(lse.t, want["lse"], "lse")

"""Calls of cross attention, the tree of drafted tokens and the cache commit (B200 only) that the
documentation allows beside the ordinary ones."""
import random

import pytest
import torch

import periodic_sparse_attention_b200 as pia
from periodic_sparse_attention_b200 import build as pbuild
from tests.test_gpu_tree import ints, make_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    pbuild.build()
    pia.load()
    yield
    torch.cuda.synchronize()


def inside(t, at):
    """t as a contiguous view `at` elements into a larger buffer (a parameter of a flat buffer)."""
    buf = torch.zeros(t.numel() + at, dtype=t.dtype, device=t.device)
    view = buf[at:].view(t.shape)
    return view.copy_(t)


def tree_problem(B, H, T, cap, d, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, kt, vt, kc, vc = (r(B, H, n, d).to(dtype) for n in (T, T, T, cap, cap))
    rng = random.Random(seed)
    return [q, kt, vt, kc, vc, r(H, d) / 8, r(H), ints([make_tree("random", T, rng) for _ in range(B)]),
            ints([rng.randint(cap // 2, cap) for _ in range(B)])]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,path", [(torch.bfloat16, "tc"), (torch.bfloat16, "simt"), (torch.float32, "auto")])
@pytest.mark.parametrize("T", [1, 9, 40])
def test_gate_parameters_and_integers_of_any_alignment(T, dtype, path, d):
    """w_g and b_g, the lengths, the parents and lse need their element's alignment only."""
    x = tree_problem(2, 3, T, 300, d, dtype)
    want = pia.pi_attn_decode_tree(*x, 40, 32, 6, path=path)
    for at in (1, 2, 3):
        y = x[:5] + [inside(t, at) for t in x[5:]]
        assert y[5].data_ptr() % 16 == 4 * at and y[5].is_contiguous()
        out, lse = pia.pi_attn_decode_tree(*y, 40, 32, 6, path=path, lse=inside(torch.zeros_like(want[1]), at))
        pia.pi_attn_check()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("dtype,path", [(torch.bfloat16, "tc"), (torch.bfloat16, "simt"), (torch.float32, "auto")])
@pytest.mark.parametrize("nq,nkv", [(1, 3000), (75, 500), (400, 500)])
def test_lengths_and_lse_of_any_alignment(nq, nkv, dtype, path):
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k, v, dout = (torch.randn(2, h, n, 64, generator=g, device="cuda").to(dtype) for h, n in ((4, nq), (2, nkv), (2, nkv), (4, nq)))
    lens = ints([nkv, nkv // 3])
    want = pia.pi_attn_cross_fwd(q, k, v, kv_len=lens, path=path)
    grads = pia.pi_attn_cross_bwd(q, k, v, *want, dout, kv_len=lens, path=path)
    for at in (1, 2, 3):
        odd = inside(lens, at)
        out, lse = pia.pi_attn_cross_fwd(q, k, v, kv_len=odd, path=path, lse=inside(torch.zeros_like(want[1]), at))
        got = pia.pi_attn_cross_bwd(q, k, v, out, lse, dout, kv_len=odd, path=path)
        pia.pi_attn_check()
        for a, b in zip((out, lse, *got), (*want, *grads)):
            assert torch.equal(a, b)


def test_clusters_of_several_kernels_on_several_streams():
    """Clusters of the many-rows and the few-rows kernels that meet on the SMs: a CTA that waits for its
    cluster must not keep another's from starting.  Each call gives the bits it gives alone."""
    g = torch.Generator(device="cuda").manual_seed(0)
    states = [[torch.randn(1, 16, n, 64, generator=g, device="cuda").to(torch.bfloat16) for n in (nq, 2000, 2000)] for nq in (256, 1, 40)]
    trees = [tree_problem(1, 2, T, 2000, 64, torch.bfloat16, seed=T) for T in (9, 24, 64)]
    jobs = [lambda x=x: pia.pi_attn_cross_fwd(*x) for x in states]
    jobs += [lambda x=x: pia.pi_attn_decode_tree(*x, 900, 64, 20) for x in trees]
    alone = [j() for j in jobs]
    pia.pi_attn_check()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[] for _ in jobs]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(jobs[i]())
    torch.cuda.synchronize()
    pia.pi_attn_check()
    for a, runs in zip(alone, got):
        for r in runs:
            assert torch.equal(r[0], a[0]) and torch.equal(r[1], a[1])


@pytest.mark.parametrize("cap", [64, 700])
def test_a_window_wider_than_the_cache_takes_the_shares_of_the_cache(cap):
    """k_win meant as "everything": as many shares of the keys as a window of the cache's size takes, none of
    them through the workspace, and the same bits."""
    x = tree_problem(1, 2, 5, cap, 64, torch.bfloat16)
    assert pia.load().pi_attn_decode_tree_workspace_bytes(1, 2, 5, 64, 2 ** 30, 64, 4, pia.PI_ATTN_BF16, 0) > 0
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    out, lse = pia.pi_attn_decode_tree(*x, 2 ** 30, 64, 4, workspace=ws)
    pia.pi_attn_check()
    want = pia.pi_attn_decode_tree(*x, cap + 5, 64, 4)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert (ws == 0).all()


def test_first_calls_from_several_threads():
    """Host threads that make a process's first calls of every kernel at once, each on its own stream, get
    the results of one thread (in a process of its own, so that these are first calls)."""
    import os
    import subprocess
    import sys

    code = """
import threading
import torch
import periodic_sparse_attention_b200 as pia
from tests.test_gpu_rows_calls import tree_problem

pia.load()
g = torch.Generator(device="cuda").manual_seed(0)
jobs = []
for dtype in (torch.bfloat16, torch.float32):
    for nq in (1, 20, 400):
        x = [torch.randn(1, 4, n, 64, generator=g, device="cuda").to(dtype) for n in (nq, 900, 900, nq)]

        def both(q, k, v, dout):
            out, lse = pia.pi_attn_cross_fwd(q, k, v)
            return (out, lse, *pia.pi_attn_cross_bwd(q, k, v, out, lse, dout))

        jobs.append((both, x))
    for T in (5, 24, 60):
        jobs.append((lambda *x: pia.pi_attn_decode_tree(*x, 90, 64, 6), tree_problem(1, 3, T, 500, 64, dtype, seed=T)))
torch.cuda.synchronize()
start, got = threading.Barrier(4), [None] * 4

def work(i):
    with torch.cuda.stream(torch.cuda.Stream()):
        start.wait()
        got[i] = [f(*x) for f, x in jobs]
    torch.cuda.synchronize()

threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
[t.start() for t in threads]
[t.join() for t in threads]
want = [f(*x) for f, x in jobs]
pia.pi_attn_check()
for r in got:
    assert r is not None and all(torch.equal(a, b) for x, y in zip(r, want) for a, b in zip(x, y))
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]


def test_a_full_plain_cache_is_reported_by_default():
    kc, vc = (torch.zeros(1, 2, 10, 64, device="cuda") for _ in range(2))
    kt, vt = (torch.ones(1, 2, 4, 64, device="cuda") for _ in range(2))
    n = ints([8])
    pia.pi_attn_cache_commit(kc, vc, kt, vt, ints([[0, 1, 2]]), ints([3]), n)
    with pytest.raises(pia.PiAttnError, match="cache_len"):
        pia.pi_attn_check()
    assert (kc == 0).all() and (vc == 0).all() and int(n) == 8
    pia.pi_attn_cache_commit(kc, vc, kt, vt, ints([[0, 1, 2]]), ints([3]), n, ring=True)
    pia.pi_attn_check()
    assert int(n) == 11 and (kc[0, :, [8, 9, 0]] == 1).all() and (kc[0, :, 1:8] == 0).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,nq,nkv,lens", [(1, 4, 2, 700, 1500, [1437]), (2, 2, 2, 1300, 900, [900, 385]), (2, 6, 1, 257, 1100, [1, 1025]),
                                                 (1, 1, 1, 2049, 2177, None)], ids=str)
def test_gradients_of_many_tiles_on_both_sides(B, H, Hkv, nq, nkv, lens, d):
    """Many tiles of rows and of keys in each CTA's stream, against the definition."""
    from tests import rows_ref as ref

    g = torch.Generator(device="cuda").manual_seed(nq)
    q, k, v, dout = (torch.randn(B, h, n, d, generator=g, device="cuda").to(torch.bfloat16) for h, n in ((H, nq), (Hkv, nkv), (Hkv, nkv), (H, nq)))
    kv_len = None if lens is None else ints(lens)
    out, lse = pia.pi_attn_cross_fwd(q, k, v, kv_len=kv_len)
    grads = pia.pi_attn_cross_bwd(q, k, v, out, lse, dout, kv_len=kv_len)
    pia.pi_attn_check()
    want = ref.cross(q, k, v, lens, dout)
    for name, t in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        ref.check(t, want[name], name)


def test_offsets_past_32_bits():
    """Caches and states of more than 2^31 elements, the rows that are read behind that point."""
    from tests import rows_ref as ref

    g = torch.Generator(device="cuda").manual_seed(0)
    d, T, k, pi, S = 128, 6, 300, 64, 8
    cap = 2 ** 23 + 4001
    kc, vc = (torch.empty(1, 3, cap, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    assert kc.numel() > 2 ** 31 + 2 ** 30
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, kt, vt = (r(1, 3, T, d).to(torch.bfloat16) for _ in range(3))
    w_g, b_g = r(3, d) / 11, r(3)
    parent = [[-1, 0, 1, 1, 3, -1]]
    for path, u in (("tc", 2.0 ** -8), ("simt", 2.0 ** -24)):
        for ring, n in ((False, cap), (True, 2 ** 31 - 513), (True, cap + 100)):  # the last length that a ring may have
            out, lse = pia.pi_attn_decode_tree(q, kt, vt, kc, vc, w_g, b_g, ints(parent), ints([n]), k, pi, S, ring=ring, path=path)
            pia.pi_attn_check()
            want = ref.tree(q, kt, vt, kc, vc, w_g, b_g, parent, [n], k, pi, S, None, ring, u=u)
            ref.check(out, want["out"], "out")
            ref.check(lse, want["lse"], "lse")
    n = ints([cap - 2])
    before = kc[0, :, :cap - 2].sum(dtype=torch.float64)
    pia.pi_attn_cache_commit(kc, vc, kt, vt, ints([[1, 4]]), ints([2]), n)
    pia.pi_attn_check()
    assert torch.equal(kc[:, :, cap - 2:], kt[:, :, [1, 4]]) and torch.equal(vc[:, :, cap - 2:], vt[:, :, [1, 4]]) and int(n) == cap
    assert kc[0, :, :cap - 2].sum(dtype=torch.float64) == before
    # the same memory as the states of three key heads; a sequence's last rows count for nothing but its last keys
    lens = ints([cap - 1])
    for nq, path in ((1, "tc"), (1, "simt"), (100, "tc")):
        x, dout = r(1, 3, nq, d).to(torch.bfloat16), r(1, 3, nq, d).to(torch.bfloat16)
        kc[0, :, :, 0], x[..., 0] = -512.0, 64.0  # every key but the last few: a score below -2048
        kc[0, :, cap - 500:, 0] = 0.0
        out, lse = pia.pi_attn_cross_fwd(x, kc, vc, kv_len=lens, path=path)
        dq, dk, dv = pia.pi_attn_cross_bwd(x, kc, vc, out, lse, dout, kv_len=lens, path=path)
        pia.pi_attn_check()
        last = [t[:, :, cap - 500:].contiguous() for t in (kc, vc)]
        want = ref.cross(x, *last, [499], dout, u=2.0 ** -8 if path == "tc" else 2.0 ** -24)
        for name, t in (("out", out), ("lse", lse), ("dq", dq), ("dk", dk[:, :, cap - 500:]), ("dv", dv[:, :, cap - 500:])):
            ref.check(t, want[name], name)
        assert not dk[:, :, :cap - 500].any() and not dv[:, :, :cap - 500].any()
        del dk, dv

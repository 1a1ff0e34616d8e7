"""Cross attention, drafted tokens and the cache commit without a GPU: refused arguments (no call here
launches a kernel), the 64-bit definitions against differences, and the key list of a tree."""
import ctypes
import itertools
import os
import random
import subprocess

import pytest
import torch

import periodic_sparse_attention_b200 as pia
from periodic_sparse_attention_b200 import build as pbuild
from tests import rows_ref as ref

HERE = os.path.dirname(os.path.abspath(__file__))
F = ctypes.c_void_p(0x10000)  # aligned, never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return pia.load()


CROSS = dict(q=F, k=F, v=F, kv_len=None, out=F, lse=F, B=1, H=4, H_kv=2, n_q=3, n_kv=5, d=64, dt=1, path=0, ws=None, wb=0, st=None)
BWD = dict(q=F, k=F, v=F, kv_len=None, out=F, lse=F, dout=F, dq=F, dk=F, dv=F, B=1, H=4, H_kv=2, n_q=3, n_kv=5, d=64, dt=1,
           path=0, ws=None, wb=0, st=None)
TREE = dict(q=F, kt=F, vt=F, kc=F, vc=F, w=F, b=F, parent=F, tree_len=None, cache_len=F, out=F, lse=F, B=1, H=2, T=4, cap=64,
            d=64, k=16, pi=8, S=4, dt=1, ring=0, path=0, ws=None, wb=0, st=None)
COMMIT = dict(kc=F, vc=F, kt=F, vt=F, path=F, n_path=F, cache_len=F, B=1, H=2, cap=64, T=4, L=2, d=64, dt=1, ring=1, st=None)
SIZES = [dict(B=0), dict(H=0), dict(d=0), dict(d=300), dict(d=12), dict(dt=7), dict(dt=0, d=6)]
CASES = (
    [("pi_attn_cross_fwd", CROSS, c) for c in SIZES + [dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(q=ODD), dict(out=ODD),
                                                       dict(H_kv=0), dict(H_kv=3), dict(n_q=0), dict(n_kv=0), dict(path=3), dict(path=4),
                                                       dict(path=9), dict(ws=ODD, wb=1 << 30), dict(n_q=2 ** 31 - 1, H=64, H_kv=64)]]
    + [("pi_attn_cross_bwd", BWD, c) for c in SIZES + [dict([(n, None)]) for n in ("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv")]
       + [dict(dq=ODD), dict(dv=ODD), dict(H_kv=3), dict(n_q=0), dict(path=3), dict(ws=F, wb=32)]]
    + [("pi_attn_decode_tree", TREE, c) for c in SIZES + [dict([(n, None)]) for n in ("q", "kt", "vt", "kc", "vc", "w", "b", "parent", "cache_len", "out")]
       + [dict(T=0), dict(T=257), dict(cap=0), dict(k=-1), dict(pi=0), dict(S=-1), dict(ring=1, cap=31), dict(ring=1, k=65), dict(path=4), dict(k=2 ** 31 - 1, pi=1), dict(k=2 ** 30 + 1),
          dict(kc=ODD), dict(B=1 << 20, H=1 << 20)]]
    + [("pi_attn_cache_commit", COMMIT, c) for c in SIZES + [dict([(n, None)]) for n in ("kc", "vc", "kt", "vt", "path", "n_path", "cache_len")]
       + [dict(T=0), dict(T=257), dict(L=0), dict(L=257), dict(cap=0), dict(vt=ODD)]])


@pytest.mark.parametrize("name,base,change", CASES, ids=lambda x: str(x) if isinstance(x, (str, dict)) and len(str(x)) < 60 else "")
def test_refused(lib, name, base, change):
    args = {**base, **change}
    assert getattr(lib, name)(*args.values()) == pia.PI_ATTN_EINVAL
    assert lib.pi_attn_last_error() != b""


def test_tensor_core_coverage_is_explicit(lib):
    for name, base in (("pi_attn_cross_fwd", CROSS), ("pi_attn_cross_bwd", BWD), ("pi_attn_decode_tree", TREE)):
        for c in (dict(dt=0), dict(d=96), dict(d=256)):
            assert getattr(lib, name)(*{**base, **c, "path": 2}.values()) == pia.PI_ATTN_EUNSUPPORTED


def test_workspace_sizes(lib):
    assert lib.pi_attn_cross_bwd_workspace_bytes(2, 4, 5, 64, 1, 0) == 160
    assert lib.pi_attn_cross_bwd_workspace_bytes(2, 4, 5, 64, 0, 0) == 0
    assert lib.pi_attn_cross_bwd_workspace_bytes(0, 4, 5, 64, 1, 0) == -1
    assert lib.pi_attn_cross_fwd_workspace_bytes(1, 4, 3, 1, 64, 64, 1, 0) == -1
    assert lib.pi_attn_cross_fwd_workspace_bytes(64, 32, 32, 64, 64, 64, 0, 0) == 0
    assert lib.pi_attn_decode_tree_workspace_bytes(1, 4, 300, 64, 8, 8, 2, 1, 0) == -1
    # few rows over very many keys are split more often than a cluster joins: a workspace one byte short is refused
    assert lib.pi_attn_cross_fwd_workspace_bytes(1, 1, 1, 1, 1024, 64, 1, 0) == 0
    need = lib.pi_attn_cross_fwd_workspace_bytes(1, 1, 1, 1, 65536, 64, 1, 0)
    assert need > 0
    assert lib.pi_attn_cross_fwd(*{**CROSS, "H": 1, "H_kv": 1, "n_q": 1, "n_kv": 65536, "ws": F, "wb": need - 1}.values()) == \
        pia.PI_ATTN_EINVAL
    assert str(need).encode() in lib.pi_attn_last_error()


def test_host_tensors_are_refused():
    t = torch.zeros(1, 2, 4, 64)
    i = torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pia.pi_attn_cross_fwd(t, t, t)
    with pytest.raises(ValueError, match="CUDA"):
        pia.pi_attn_cross_bwd(t, t, t, t, t[..., 0], t)
    with pytest.raises(ValueError, match="CUDA"):
        pia.pi_attn_decode_tree(t, t, t, t, t, t[0, :, 0], t[0, :, 0, 0], i, i[:, 0], 4, 4, 2)
    with pytest.raises(ValueError, match="CUDA"):
        pia.pi_attn_cache_commit(t, t, t, t, i, i[:, 0], i[:, 0])


def test_definition_of_the_gradients():
    """The 64-bit gradients against central differences of the 64-bit forward."""
    g = torch.Generator().manual_seed(0)
    q, k, v, do = (torch.randn(*s, generator=g) for s in [(2, 4, 3, 8), (2, 2, 6, 8), (2, 2, 6, 8), (2, 4, 3, 8)])
    lens = [6, 4]
    want = ref.cross(q, k, v, lens, do)
    t = 2.0 ** -6

    def loss(*x):
        return float((ref.cross(*x, lens)["out"][0] * do.double()).sum())

    for at, name in enumerate(("dq", "dk", "dv")):
        e = torch.randn((q, k, v)[at].shape, generator=g)
        hi, lo = [q, k, v], [q, k, v]
        hi[at], lo[at] = hi[at] + t * e, lo[at] - t * e
        diff = (loss(*hi) - loss(*lo)) / (2 * t)
        assert abs(diff - float((want[name][0] * e).sum())) <= 1e-3 * float((want[name][0] * e).abs().sum() + 1)


def test_definition_of_a_chain_is_causal_attention():
    """A chain drafted on an empty cache against the prefill oracle."""
    import numpy as np

    import oracle

    g = torch.Generator().manual_seed(1)
    n, d, k, pi, S = 30, 8, 4, 3, 5
    q, kk, v = (torch.randn(1, 2, n, d, generator=g) for _ in range(3))
    w, b = torch.randn(2, d, generator=g), torch.randn(2, generator=g)
    empty = torch.zeros(1, 2, 1, d)
    got = ref.tree(q, kk, v, empty, empty, w, b, [list(range(-1, n - 1))], [0], k, pi, S)
    out, lse, _ = oracle.fwd(*(x.numpy() for x in (q, kk, v, w, b)), k, pi, S)
    assert np.abs(got["out"][0].numpy().reshape(out.shape) - out).max() < 1e-12
    assert np.abs(got["lse"][0].numpy().reshape(lse.shape) - lse).max() < 1e-12


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("tree") / "tree_rule_harness")
    csrc = os.path.join(os.path.dirname(HERE), "periodic_sparse_attention_b200", "csrc")
    r = subprocess.run([pbuild.nvcc(), "-std=c++17", "-O1", "-I", csrc, os.path.join(HERE, "tree_rule_harness.cu"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


def test_key_list_of_a_tree(harness):
    """Every (node, position) of the rule is one entry of the list with its kind, once; no entry reads a
    row that is not there."""
    rng = random.Random(5)
    runs = [(n, D, T, k, pi, S, cap, ring)
            for n, D, k, pi, S in itertools.product((0, 1, 5, 17, 40), (1, 2, 4, 9), (0, 1, 6, 30), (1, 2, 5, 11), (0, 1, 3, 7))
            for T, cap, ring in ((D, max(40, n), 0),)]
    runs += [(rng.randint(0, 2000), rng.randint(1, 256), 256, rng.randint(0, 300), rng.randint(1, 200), rng.randint(0, 20), 0, 1) for _ in range(60)]
    text = ""
    for n, D, T, k, pi, S, cap, ring in runs:
        if ring:
            cap = max(k, S * pi, 1)
        text += f"{n} {D} {T} {k} {pi} {S} {cap} {ring}\n"
    r = subprocess.run([harness], input=text, capture_output=True, text=True, timeout=300)
    lines = r.stdout.split("\n")[:-1]
    assert r.returncode == 0 and len(lines) == len(runs), r.stderr[-500:]
    for run, line in zip(runs, lines):
        n, D, T, k, pi, S, cap, ring = run
        if ring:
            cap = max(k, S * pi, 1)
        got = [tuple(int(x) for x in e.split(",")) for e in line.split()]
        want = set()
        for x in range(D):
            i = n + x
            keys = [(j, 1) for j in range(max(0, i - k), i + 1)] + [(i - m * pi, 2) for m in range(1, S + 1) if m * pi > k and i - m * pi >= 0]
            want |= {(x, j, kind) for j, kind in keys if j < n}
        assert len(got) == len(set(got)), run
        assert {(x, j, kind) for x, j, kind, _ in got} == want, run
        assert all(row == (j % cap if ring else j) and 0 <= row < cap for _, j, _, row in got), run

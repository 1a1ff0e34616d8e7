"""The tree of drafted tokens and the cache commit (B200 only) against the definition in 64 bits, and
a run of them as a generation loop uses them."""
import math
import random

import pytest
import torch

import periodic_sparse_attention_b200 as pia
from periodic_sparse_attention_b200 import build as pbuild
from tests import rows_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    pbuild.build()
    pia.load()
    yield
    torch.cuda.synchronize()


def ints(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")


def make_tree(kind, T, rng):
    if kind == "chain":
        return list(range(-1, T - 1))
    if kind == "flat":
        return [-1] * T
    if kind == "binary":
        return [(t - 1) // 2 if t else -1 for t in range(T)]
    return [rng.randint(-1, t - 1) for t in range(T)]


def problem(B, H, T, cap, d, dtype, lens, kind, k, pi, S, ring, seed=0, nodes=None):
    """Inputs whose cache holds NaN in every row that no node may read."""
    rng = random.Random(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = dict(q=r(B, H, T, d).to(dtype), k_tree=r(B, H, T, d).to(dtype), v_tree=r(B, H, T, d).to(dtype),
             kcache=r(B, H, cap, d).to(dtype), vcache=r(B, H, cap, d).to(dtype), w_g=r(H, d) / math.sqrt(d), b_g=r(H))
    parent = [make_tree(kind, T, rng) for _ in range(B)]
    for b in range(B):
        n, read = lens[b], set()
        live = T if nodes is None else nodes[b]
        for t in range(live):
            i = n + ref.depth_of(parent[b], t)
            keys = list(range(max(0, i - k), i + 1)) + [i - m * pi for m in range(1, S + 1) if m * pi > k and i - m * pi >= 0]
            read.update(j % cap if ring else j for j in keys if j < n)
        stale = [j for j in range(cap) if j not in read]
        x["kcache"][b, :, stale] = math.nan
        x["vcache"][b, :, stale] = math.nan
        x["k_tree"][b, :, live:] = math.nan
        x["v_tree"][b, :, live:] = math.nan
    x["parent"], x["cache_len"], x["tree_len"] = parent, lens, nodes
    return x


def call(x, k, pi, S, ring, path, **kw):
    return pia.pi_attn_decode_tree(x["q"], x["k_tree"], x["v_tree"], x["kcache"], x["vcache"], x["w_g"], x["b_g"],
                                   ints(x["parent"]), ints(x["cache_len"]), k, pi, S, tree_len=ints(x["tree_len"]),
                                   ring=ring, path=path, **kw)


# B, H, T, cap, d, cache lengths, kind, k, pi, S, ring, nodes
SHAPES = [
    (1, 1, 1, 8, 64, [0], "chain", 4, 4, 2, False, None),                # nothing cached
    (1, 2, 1, 300, 128, [300], "chain", 16, 32, 4, False, None),         # a decode step, the cache full
    (2, 2, 5, 300, 64, [1, 200], "flat", 0, 7, 9, False, None),          # window of the token itself
    (2, 2, 9, 512, 64, [511, 130], "random", 128, 64, 4, False, None),   # skips inside the window dropped
    (3, 2, 16, 700, 128, [700, 33, 0], "binary", 100, 96, 5, False, [16, 7, 16]),
    (2, 1, 33, 400, 64, [390, 17], "chain", 5, 3, 60, False, [33, 1]),   # deeper than the period
    (1, 2, 64, 900, 128, [900], "random", 300, 50, 16, False, None),
    (2, 1, 70, 300, 64, [280, 299], "chain", 20, 40, 6, False, [70, 65]),
    (1, 1, 256, 400, 64, [350], "chain", 37, 100, 3, False, None),       # ancestors past the window, by skips
    (1, 1, 256, 500, 128, [123], "random", 64, 1, 90, False, [200]),     # every position a skip
    (2, 2, 8, 257, 64, [1000, 256], "random", 256, 64, 4, True, None),   # a ring that has wrapped, no slot spare
    (2, 2, 12, 1300, 128, [99999, 5], "binary", 64, 128, 10, True, [12, 3]),
    (1, 2, 24, 100, 64, [73], "random", 1000, 5, 3, False, None),        # the window longer than the cache
    (2, 2, 6, 64, 64, [30, 50], "random", 10, 12, 0, False, [0, 6]),     # no skips; a sequence without nodes
]
KINDS = [(torch.bfloat16, p) for p in ("auto", "simt", "tc")] + [(torch.float32, "auto")]


def unit(dtype, path, d):
    return 2.0 ** -8 if dtype == torch.bfloat16 and d in (64, 128) and path != "simt" else 2.0 ** -24


def compare(x, out, lse, k, pi, S, ring, dtype, path, before=None):
    want = ref.tree(x["q"], x["k_tree"], x["v_tree"], x["kcache"], x["vcache"], x["w_g"], x["b_g"], x["parent"],
                    x["cache_len"], k, pi, S, x["tree_len"], ring, u=unit(dtype, path, x["q"].shape[3]))
    T = x["q"].shape[2]
    for b in range(x["q"].shape[0]):
        n = T if x["tree_len"] is None else x["tree_len"][b]
        for name, got in (("out", out), ("lse", lse)):
            ref.check(got[b, :, :n], tuple(t[b, :, :n] for t in want[name]), f"{name} of sequence {b}")
            if before is not None and n < T:
                assert torch.equal(got[b, :, n:], before[name][b, :, n:]), "rows behind the nodes were written"


@pytest.mark.parametrize("dtype,path", KINDS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_tree(shape, dtype, path):
    B, H, T, cap, d, lens, kind, k, pi, S, ring, nodes = shape
    x = problem(B, H, T, cap, d, dtype, lens, kind, k, pi, S, ring, seed=T, nodes=nodes)
    out, lse = torch.full_like(x["q"], 7.0), torch.full((B, H, T), 7.0, device="cuda")
    before = dict(out=out.clone(), lse=lse.clone())
    call(x, k, pi, S, ring, path, out=out, lse=lse)
    pia.pi_attn_check()
    compare(x, out, lse, k, pi, S, ring, dtype, path, before)


@pytest.mark.parametrize("d", [4, 36, 256])
def test_fp32_head_sizes(d):
    x = problem(2, 2, 10, 200, d, torch.float32, [180, 33], "random", 40, 30, 5, False, seed=d)
    out, lse = call(x, 40, 30, 5, False, "auto")
    pia.pi_attn_check()
    compare(x, out, lse, 40, 30, 5, False, torch.float32, "auto")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_sequences_and_splits(dtype):
    """One sequence (its keys split over blocks) and very many."""
    x = problem(1, 1, 4, 4096, 128, dtype, [4000], "random", 2000, 60, 40, False, seed=1)
    out, lse = call(x, 2000, 60, 40, False, "auto")
    pia.pi_attn_check()
    compare(x, out, lse, 2000, 60, 40, False, dtype, "auto")
    lens = [37 * b % 50 for b in range(40)]
    x = problem(40, 16, 3, 50, 64, dtype, lens, "random", 9, 11, 3, False, seed=2, nodes=[b % 4 for b in range(40)])
    out, lse = call(x, 9, 11, 3, False, "auto")
    pia.pi_attn_check()
    compare(x, out, lse, 9, 11, 3, False, dtype, "auto")


@pytest.mark.parametrize("d", [128, 256])
def test_many_sequences_of_other_head_sizes(d):
    """The 64-row tiles of the CUDA-core kernel with 70 nodes, at its largest shared memory."""
    x = problem(19, 8, 70, 90, d, torch.float32, [4 * b for b in range(19)], "random", 30, 7, 4, False, seed=d,
                nodes=[70 - 3 * b for b in range(19)])
    out, lse = call(x, 30, 7, 4, False, "auto")
    pia.pi_attn_check()
    compare(x, out, lse, 30, 7, 4, False, torch.float32, "auto")


def test_far_skips_and_wide_windows():
    """Windows and periods near the limits of 32 bits, which reach nothing."""
    for k, pi, S in ((2 ** 30, 1, 5), (3, 2 ** 31 - 1, 2 ** 31 - 1), (0, 2 ** 30, 7), (2 ** 30, 2 ** 31 - 1, 3)):
        x = problem(1, 2, 9, 200, 64, torch.bfloat16, [190], "random", min(k, 200), pi, min(S, 1), False, seed=2)
        for path in ("tc", "simt"):
            out, lse = call(x, k, pi, S, False, path)
            pia.pi_attn_check()
            compare(x, out, lse, min(k, 200), pi, min(S, 1), False, torch.bfloat16, path)


@pytest.mark.parametrize("gate", [60.0, -60.0])
@pytest.mark.parametrize("path", ["simt", "tc"])
def test_saturated_gate(gate, path):
    """A prior that all but removes the skips, or the window: the weights of one side vanish."""
    x = problem(1, 2, 20, 500, 64, torch.bfloat16, [480], "random", 30, 32, 12, False, seed=4)
    x["b_g"].fill_(gate)
    out, lse = call(x, 30, 32, 12, False, path)
    pia.pi_attn_check()
    compare(x, out, lse, 30, 32, 12, False, torch.bfloat16, path)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_node_is_a_decode_step(dtype):
    """T = 1 against pi_attn_decode over a cache that holds the token."""
    B, H, d, k, pi, S = 2, 4, 64, 50, 64, 5
    g = torch.Generator(device="cuda").manual_seed(0)
    kc, vc = (torch.randn(B, H, 400, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    q = torch.randn(B, H, d, generator=g, device="cuda").to(dtype)
    w_g, b_g = torch.randn(H, d, generator=g, device="cuda") / 8, torch.randn(H, generator=g, device="cuda")
    lens = [400, 77]
    out, lse = pia.pi_attn_decode(q, kc, vc, w_g, b_g, k, pi, S, cache_len=ints(lens))
    pick = lambda t: torch.stack([t[b, :, lens[b] - 1] for b in range(B)])[:, :, None].contiguous()  # noqa: E731
    o2, l2 = pia.pi_attn_decode_tree(q[:, :, None].contiguous(), pick(kc), pick(vc), kc, vc, w_g, b_g, ints([[-1]] * B),
                                     ints([n - 1 for n in lens]), k, pi, S)
    pia.pi_attn_check()
    # both are within their bound of the same value: bf16 outputs differ by at most two roundings of
    # out and one of p each way, fp32 ones by the sums' roundings
    tol = 4 * 2.0 ** -8 if dtype == torch.bfloat16 else 1e-5
    assert (out.float() - o2[:, :, 0].float()).abs().max() <= tol * vc.float().abs().max()
    assert (lse - l2[:, :, 0]).abs().max() <= 1e-4


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_bad_lengths_and_parents_are_reported(dtype):
    for what, match in (("len", "cache_len"), ("neg", "cache_len"), ("nodes", "cache_len"), ("later", "tree"), ("low", "tree")):
        x = problem(3, 2, 6, 64, 64, dtype, [60, 60, 5], "random", 10, 12, 3, False, seed=1, nodes=[6, 5, 6])
        good = {n: (list(v) if n != "parent" else [list(r) for r in v]) for n, v in x.items() if n in ("parent", "cache_len", "tree_len")}
        if what == "len":
            x["cache_len"][1] = 65
        if what == "neg":
            x["cache_len"][1] = -1
        if what == "nodes":
            x["tree_len"][1] = 7
        if what == "later":
            x["parent"][1][2] = 2
        if what == "low":
            x["parent"][1][4] = -2
        out, lse = torch.zeros_like(x["q"]), torch.zeros(3, 2, 6, device="cuda")
        call(x, 10, 12, 3, False, "auto", out=out, lse=lse)
        with pytest.raises(pia.PiAttnError, match=match):
            pia.pi_attn_check()
        n = 5 if match == "tree" else 6
        assert out[1, :, :n].isnan().all() and lse[1, :, :n].isnan().all()
        assert (out[1, :, n:] == 0).all()
        x.update(good)
        want = ref.tree(x["q"], x["k_tree"], x["v_tree"], x["kcache"], x["vcache"], x["w_g"], x["b_g"], x["parent"],
                        x["cache_len"], 10, 12, 3, x["tree_len"], u=unit(dtype, "auto", 64))
        for b in (0, 2):
            ref.check(out[b], tuple(t[b] for t in want["out"]), "out")
    # a bad parent behind the nodes of a sequence is not read
    x = problem(1, 2, 6, 64, 64, dtype, [60], "random", 10, 12, 3, False, seed=1, nodes=[4])
    x["parent"][0][5] = 99
    call(x, 10, 12, 3, False, "auto")
    pia.pi_attn_check()


@pytest.mark.parametrize("path", ["simt", "tc"])
def test_replay_and_second_stream(path):
    k, pi, S = 200, 64, 8
    x = problem(1, 2, 12, 600, 64, torch.bfloat16, [550], "random", k, pi, S, False, seed=3)
    dev = {n: ints(x[n]) for n in ("parent", "cache_len")}

    def one(**kw):
        return pia.pi_attn_decode_tree(x["q"], x["k_tree"], x["v_tree"], x["kcache"], x["vcache"], x["w_g"], x["b_g"],
                                       dev["parent"], dev["cache_len"], k, pi, S, path=path, **kw)

    first = one()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = one(stream=side)
    side.synchronize()
    for a, b in zip(first, other):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = one()
    for seed in (1, 2):  # other values, another tree and length in the captured call
        y = problem(1, 2, 12, 600, 64, torch.bfloat16, [550 - 40 * seed], "random", k, pi, S, False, seed=seed)
        for n in ("q", "k_tree", "v_tree", "kcache", "vcache"):
            x[n].copy_(y[n])
        for n in dev:
            dev[n].copy_(ints(y[n]))
        x["parent"], x["cache_len"] = y["parent"], y["cache_len"]
        graph.replay()
        pia.pi_attn_check()
        compare(x, *held, k, pi, S, False, torch.bfloat16, path)


@pytest.mark.parametrize("path", ["simt", "tc"])
def test_nothing_is_written_outside(path):
    from tests.test_gpu_guards import Guarded

    x = problem(1, 2, 11, 900, 64, torch.bfloat16, [880], "random", 500, 64, 8, False, seed=3)
    out, lse = Guarded(x["q"].shape, torch.bfloat16), Guarded(x["q"].shape[:3], torch.float32)
    need = pia.load().pi_attn_decode_tree_workspace_bytes(1, 2, 11, 64, 500, 64, 8, pia.PI_ATTN_BF16, pia.PATHS[path])
    ws = Guarded((max(need, 16),), torch.uint8)
    call(x, 500, 64, 8, False, path, out=out.t, lse=lse.t, workspace=ws.t)
    pia.pi_attn_check()
    for name, t in (("out", out), ("lse", lse), ("workspace", ws)):
        t.check(name)
    compare(x, out.t, lse.t, 500, 64, 8, False, torch.bfloat16, path)


# ---- commit --------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,H,T,L,cap,d,ring", [(1, 1, 1, 1, 1, 64, True), (3, 4, 9, 5, 70, 64, True), (2, 3, 256, 256, 300, 8, False),
                                                (70, 2, 16, 4, 40, 128, True), (2, 8, 5, 5, 5, 32, True), (3, 2, 7, 7, 50, 100, False)])
def test_commit(B, H, T, L, cap, d, ring, dtype):
    if dtype == torch.bfloat16 and d % 8:
        d += 4
    rng = random.Random(T + cap)
    g = torch.Generator(device="cuda").manual_seed(1)
    kc, vc = (torch.randn(B, H, cap, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    kt, vt = (torch.randn(B, H, T, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    count = [rng.randint(0, min(L, cap)) for _ in range(B)]
    count[0] = min(L, cap)
    lens = [rng.randint(0, 5 * cap) if ring else rng.randint(0, cap - c) for c in count]
    path = [[rng.randrange(T) for _ in range(L)] for _ in range(B)]
    want_k, want_v = kc.clone(), vc.clone()
    for b in range(B):
        for e in range(count[b]):
            at = (lens[b] + e) % cap if ring else lens[b] + e
            want_k[b, :, at], want_v[b, :, at] = kt[b, :, path[b][e]], vt[b, :, path[b][e]]
        path[b][count[b]:] = [T + 5] * (L - count[b])  # entries behind the count are not read
    n = ints(lens)
    pia.pi_attn_cache_commit(kc, vc, kt, vt, ints(path), ints(count), n, ring=ring)
    pia.pi_attn_check()
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)
    assert n.tolist() == [x + c for x, c in zip(lens, count)]


def test_commit_reports_and_leaves_alone():
    g = torch.Generator(device="cuda").manual_seed(1)
    B, H, T, L, cap, d = 2, 2, 4, 3, 10, 64
    base = [torch.randn(B, H, m, d, generator=g, device="cuda") for m in (cap, cap, T, T)]
    for lens, count, path, ring, match in [([0, 8], [1, 3], [0, 1, 2], False, "cache_len"), ([0, -1], [1, 1], [0, 1, 2], True, "cache_len"),
                                           ([0, 0], [1, 4], [0, 1, 2], True, "cache_len"), ([0, 0], [1, -1], [0, 1, 2], True, "cache_len"),
                                           ([0, 0], [1, 3], [0, 1, 4], True, "tree"), ([0, 0], [1, 2], [0, -1, 2], True, "tree")]:
        kc, vc, kt, vt = (t.clone() for t in base)
        n = ints(lens)
        pia.pi_attn_cache_commit(kc, vc, kt, vt, ints([[0, 1, 2], path]), ints(count), n, ring=ring)
        with pytest.raises(pia.PiAttnError, match=match):
            pia.pi_attn_check()
        assert torch.equal(kc[1], base[0][1]) and torch.equal(vc[1], base[1][1]) and int(n[1]) == lens[1]
        assert torch.equal(kc[0, :, 0], kt[0, :, 0]) and int(n[0]) == 1


# ---- together ------------------------------------------------------------------------------------
@pytest.mark.parametrize("ring", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_verification_loop(dtype, ring):
    """Steps of drafting, verifying (the tree over the cache, then cross attention of its nodes to an
    encoder's states) and committing give, node by node of the accepted path, what the causal prefill
    and cross attention of the whole accepted sequence give."""
    B, H, d, k, pi, S, T, total = 2, 2, 64, 24, 16, 5, 7, 140
    cap = 96 if ring else 256
    rng = random.Random(3)
    g = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    w_g, b_g = torch.randn(H, d, generator=g, device="cuda") / 8, torch.randn(H, generator=g, device="cuda")
    enc_k, enc_v, enc_len = r(B, 1, 90, d), r(B, 1, 90, d), ints([90, 41])
    seq = [r(B, H, total, d) for _ in range(3)]  # q, k, v of the accepted sequence
    kc, vc = (torch.full((B, H, cap, d), math.nan, device="cuda").to(dtype) for _ in range(2))
    n, lens = ints([0] * B), [0] * B
    got = [[], []]
    while max(lens) < total - T:
        parent = [make_tree("random", T, rng) for _ in range(B)]
        q, kt, vt = (r(B, H, T, d) for _ in range(3))
        paths, counts = [], []
        for b in range(B):  # the accepted path: a random node and its ancestors, in order
            line = [rng.randrange(T)]
            while parent[b][line[-1]] >= 0:
                line.append(parent[b][line[-1]])
            line = line[::-1]
            for e, t in enumerate(line):
                for x, y in zip((q, kt, vt), seq):
                    x[b, :, t] = y[b, :, lens[b] + e]
            paths.append(line + [0] * (T - len(line)))
            counts.append(len(line))
        o, l = pia.pi_attn_decode_tree(q, kt, vt, kc, vc, w_g, b_g, ints(parent), n, k, pi, S, ring=ring)
        co, cl = pia.pi_attn_cross_fwd(o, enc_k, enc_v, kv_len=enc_len)
        pia.pi_attn_cache_commit(kc, vc, kt, vt, ints(paths), ints(counts), n, ring=ring)
        for b in range(B):
            for e in range(counts[b]):
                t = paths[b][e]
                got[b].append((o[b, :, t], l[b, :, t], co[b, :, t]))
            lens[b] += counts[b]
        assert n.tolist() == lens
    pia.pi_attn_check()
    out, lse = pia.pi_attn_fwd(*(t.contiguous() for t in seq), w_g, b_g, k, pi, S)
    # two kernels of the same operator: each within (rounding of p, rounding of out) of the exact row
    tol = 4 * 2.0 ** -8 if dtype == torch.bfloat16 else 1e-5
    for b in range(B):
        m = len(got[b])
        assert m == lens[b] <= total
        o, l, co = (torch.stack([x[i] for x in got[b]], dim=1) for i in range(3))
        assert (o.float() - out[b, :, :m].float()).abs().max() <= tol * seq[2].float().abs().max()
        assert (l - lse[b, :, :m]).abs().max() <= 1e-3
        want = ref.cross(o[None].contiguous(), enc_k[b:b + 1], enc_v[b:b + 1], [int(enc_len[b])], u=unit(dtype, "auto", d))
        ref.check(co, tuple(x[0] for x in want["out"]), "cross")

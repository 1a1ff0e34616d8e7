"""Cross attention and its gradients (B200 only) against the definition in 64 bits."""
import math

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


def inputs(B, H, Hkv, nq, nkv, d, dtype, seed=0, poison=None, kv_len=None, scale=1.0):
    """q, k, v, dout; what k and v hold behind kv_len is `poison`."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = [torch.randn(*s, generator=g, device="cuda").mul_(scale).to(dtype)
         for s in [(B, H, nq, d), (B, Hkv, nkv, d), (B, Hkv, nkv, d), (B, H, nq, d)]]
    if kv_len is not None and poison is not None:
        for b, n in enumerate(kv_len):
            t[1][b, :, n:] = poison
            t[2][b, :, n:] = poison
    return t


def ints(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")


def unit(dtype, path, d):
    """The roundoff of p and ds in the last products: bf16 on the tensor cores, fp32 else."""
    tc = dtype == torch.bfloat16 and d in (64, 128) and path != "simt"
    return 2.0 ** -8 if tc else 2.0 ** -24


# B, H, Hkv, nq, nkv, d, kv_len
SHAPES = [
    (1, 1, 1, 1, 1, 64, None),                 # one row, one key
    (1, 2, 2, 1, 63, 128, None),
    (2, 4, 1, 1, 129, 64, [129, 1]),           # a step, four heads a key head
    (3, 8, 2, 1, 1000, 128, [0, 999, 64]),     # a sequence without states
    (2, 4, 4, 17, 65, 64, [65, 0]),
    (1, 8, 2, 5, 2111, 128, [2050]),
    (2, 2, 1, 127, 128, 64, [127, 128]),
    (1, 2, 2, 129, 257, 128, None),
    (2, 4, 2, 300, 191, 64, [191, 3]),
    (1, 2, 1, 513, 640, 128, [577]),
    (1, 1, 1, 1025, 33, 64, None),
    (1, 2, 2, 257, 1100, 128, None),
    (5, 3, 3, 40, 70, 128, [70, 69, 64, 1, 0]),
]
BF16 = [(torch.bfloat16, p) for p in ("auto", "simt", "tc")]


@pytest.mark.parametrize("dtype,path", BF16 + [(torch.float32, "auto")])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_gradients(shape, dtype, path):
    B, H, Hkv, nq, nkv, d, lens = shape
    q, k, v, dout = inputs(B, H, Hkv, nq, nkv, d, dtype, seed=nq + nkv, poison=math.nan, kv_len=lens)
    out, lse = pia.pi_attn_cross_fwd(q, k, v, kv_len=ints(lens), path=path)
    pia.pi_attn_check()
    want = ref.cross(q, k, v, lens, dout, u=unit(dtype, path, d))
    ref.check(out, want["out"], "out")
    ref.check(lse, want["lse"], "lse")
    grads = pia.pi_attn_cross_bwd(q, k, v, out, lse, dout, kv_len=ints(lens), path=path)
    pia.pi_attn_check()
    for name, g in zip(("dq", "dk", "dv"), grads):
        ref.check(g, want[name], name)


@pytest.mark.parametrize("d", [4, 20, 32, 100, 160, 256])
def test_fp32_head_sizes(d):
    q, k, v, dout = inputs(2, 4, 2, 37, 150, d, torch.float32, seed=d, poison=math.inf, kv_len=[150, 77])
    out, lse = pia.pi_attn_cross_fwd(q, k, v, kv_len=ints([150, 77]))
    grads = pia.pi_attn_cross_bwd(q, k, v, out, lse, dout, kv_len=ints([150, 77]))
    pia.pi_attn_check()
    want = ref.cross(q, k, v, [150, 77], dout)
    for name, g in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        ref.check(g, want[name], name)


@pytest.mark.parametrize("d", [8, 96, 192, 256])
def test_bf16_other_head_sizes_take_the_cuda_cores(d):
    q, k, v, dout = inputs(1, 4, 2, 70, 130, d, torch.bfloat16, seed=d)
    out, lse = pia.pi_attn_cross_fwd(q, k, v)
    grads = pia.pi_attn_cross_bwd(q, k, v, out, lse, dout)
    pia.pi_attn_check()
    want = ref.cross(q, k, v, None, dout, u=2.0 ** -24)
    for name, g in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        ref.check(g, want[name], name)


def test_many_tiles_take_the_large_row_tiles():
    """Enough rows for the 64-row tiles of the CUDA-core kernels, at each column count."""
    for d in (32, 100, 128, 200, 256):
        q, k, v, dout = inputs(4, 8, 8, 300, 130, d, torch.float32, seed=d)
        out, lse = pia.pi_attn_cross_fwd(q, k, v)
        grads = pia.pi_attn_cross_bwd(q, k, v, out, lse, dout)
        pia.pi_attn_check()
        want = ref.cross(q, k, v, None, dout)
        for name, g in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
            ref.check(g, want[name], name)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("nq", [1, 200, 700])
def test_scores_of_every_size(dtype, nq):
    """Scores in the hundreds, far apart from tile to tile: the running maximum moves often."""
    q, k, v, dout = inputs(1, 2, 1, nq, 700, 64, dtype, seed=3)
    k *= torch.linspace(0.1, 24, 700, device="cuda")[None, None, :, None].to(dtype)
    out, lse = pia.pi_attn_cross_fwd(q, k, v)
    grads = pia.pi_attn_cross_bwd(q, k, v, out, lse, dout)
    pia.pi_attn_check()
    want = ref.cross(q, k, v, None, dout, u=unit(dtype, "auto", 64))
    for name, g in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        ref.check(g, want[name], name)


def test_gradients_against_differences():
    """(loss(x + t e) - loss(x - t e)) / 2t of the kernel's own fp32 forward along random directions."""
    q, k, v, dout = inputs(1, 4, 2, 9, 50, 32, torch.float32, seed=8)
    lens = ints([47])
    out, lse = pia.pi_attn_cross_fwd(q, k, v, kv_len=lens)
    grads = pia.pi_attn_cross_bwd(q, k, v, out, lse, dout, kv_len=lens)
    loss = lambda *x: float((pia.pi_attn_cross_fwd(*x, kv_len=lens)[0].double() * dout.double()).sum())  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(1)
    t = 2.0 ** -7
    for at in range(3):
        e = torch.randn(grads[at].shape, generator=g, device="cuda")
        hi, lo = [q, k, v], [q, k, v]
        hi[at], lo[at] = hi[at] + t * e, lo[at] - t * e
        diff = (loss(*hi) - loss(*lo)) / (2 * t)
        want = float((grads[at].double() * e.double()).sum())
        # the difference carries t^2 / 6 of the third derivative and the forwards' rounding over t
        scale = float((grads[at].double().abs() * e.double().abs()).sum())
        assert abs(diff - want) <= 2e-3 * scale, (at, diff, want, scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("nq,nkv", [(1, 40), (300, 40), (1, 3000), (200, 3000)])
def test_bad_length_is_reported(dtype, nq, nkv):
    q, k, v, dout = inputs(3, 2, 2, nq, nkv, 64, dtype)
    for bad in (-1, nkv + 1):
        lens = ints([nkv, bad, 7])
        out, lse = pia.pi_attn_cross_fwd(q, k, v, kv_len=lens)
        with pytest.raises(pia.PiAttnError, match="cache_len-out-of-range"):
            pia.pi_attn_check()
        assert out[1].isnan().all() and lse[1].isnan().all()
        want = ref.cross(q, k, v, [nkv, 0, 7], dout, u=unit(dtype, "auto", 64))
        for b in (0, 2):
            ref.check(out[b], tuple(x[b] for x in want["out"]), "out")
        grads = pia.pi_attn_cross_bwd(q, k, v, out, lse, dout, kv_len=lens)
        with pytest.raises(pia.PiAttnError, match="cache_len-out-of-range"):
            pia.pi_attn_check()
        for name, g in zip(("dq", "dk", "dv"), grads):
            assert g[1].isnan().all()
            for b in (0, 2):
                ref.check(g[b], tuple(x[b] for x in want[name]), name)


@pytest.mark.parametrize("path", ["simt", "tc"])
@pytest.mark.parametrize("nq,nkv", [(1, 3000), (400, 300)])
def test_replay_and_second_stream(path, nq, nkv):
    """A captured call and a call on another stream give the eager call's bits; new values in the
    captured inputs give theirs."""
    q, k, v, dout = inputs(2, 4, 2, nq, nkv, 128, torch.bfloat16, seed=5)
    lens = ints([nkv, nkv // 2])

    def both():
        out, lse = pia.pi_attn_cross_fwd(q, k, v, kv_len=lens, path=path)
        return (out, lse, *pia.pi_attn_cross_bwd(q, k, v, out, lse, dout, kv_len=lens, path=path))

    first = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = pia.pi_attn_cross_fwd(q, k, v, kv_len=lens, path=path, stream=side)
    grads = pia.pi_attn_cross_bwd(q, k, v, out, lse, dout, kv_len=lens, path=path, stream=side)
    side.synchronize()
    for a, b in zip(first, (out, lse, *grads)):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = both()
    for seed in (6, 7):
        new = inputs(2, 4, 2, nq, nkv, 128, torch.bfloat16, seed=seed)
        for a, b in zip((q, k, v, dout), new):
            a.copy_(b)
        lens.copy_(ints([nkv - seed, 3]))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, both()):
            assert torch.equal(a, b)


@pytest.mark.parametrize("path", ["simt", "tc"])
@pytest.mark.parametrize("nq,nkv", [(1, 700), (3, 129), (130, 77)])
def test_nothing_is_written_outside(path, nq, nkv):
    from tests.test_gpu_guards import Guarded

    q, k, v, dout = inputs(1, 4, 2, nq, nkv, 64, torch.bfloat16, seed=2)
    out, lse = Guarded(q.shape, torch.bfloat16), Guarded(q.shape[:3], torch.float32)
    g = [Guarded(t.shape, torch.bfloat16) for t in (q, k, v)]
    need = pia.load().pi_attn_cross_fwd_workspace_bytes(1, 4, 2, nq, nkv, 64, pia.PI_ATTN_BF16, pia.PATHS[path])
    ws = Guarded((max(need, 16),), torch.uint8)
    need_b = pia.load().pi_attn_cross_bwd_workspace_bytes(1, 4, nq, 64, pia.PI_ATTN_BF16, pia.PATHS[path])
    wb = Guarded((max(need_b, 16),), torch.uint8)
    pia.pi_attn_cross_fwd(q, k, v, out=out.t, lse=lse.t, path=path, workspace=ws.t)
    pia.pi_attn_cross_bwd(q, k, v, out.t, lse.t, dout, grads=tuple(x.t for x in g), path=path, workspace=wb.t)
    pia.pi_attn_check()
    for name, x in zip(("out", "lse", "dq", "dk", "dv", "workspace", "backward workspace"), (out, lse, *g, ws, wb)):
        x.check(name)
    want = ref.cross(q, k, v, None, dout, u=unit(torch.bfloat16, path, 64))
    for name, x in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *g)):
        ref.check(x.t, want[name], name)


@pytest.mark.parametrize("shape", [
    (4, 16, 16, 130, 200, 64, [200, 0, 129, 128]),
    (5, 16, 16, 128, 385, 128, [385, 1, 127, 0, 256]),
    (2, 64, 32, 100, 128, 128, None),              # two heads' rows in one tile
    (1, 25, 25, 300, 1000, 64, [999]),             # a second CTA with one row tile
    (1, 52, 52, 65, 700, 128, [700]),
    (1, 13, 13, 1030, 513, 128, [513]),
    (1, 7, 7, 2000, 260, 64, [130]),
    (1, 3, 3, 500, 2500, 128, [2450]),             # clusters of eight, some without keys of a short sequence
    (2, 4, 2, 200, 2100, 64, [100, 0]),
    (3, 8, 8, 70, 1100, 128, [1100, 513, 2]),      # clusters of four
    (2, 75, 75, 140, 300, 64, [300, 257]),         # a full wave, then pairs
], ids=str)
def test_many_rows(shape):
    """Enough row tiles for the 256-row CTAs."""
    B, H, Hkv, nq, nkv, d, lens = shape
    q, k, v, dout = inputs(B, H, Hkv, nq, nkv, d, torch.bfloat16, seed=nq, poison=math.nan, kv_len=lens)
    k *= torch.linspace(0.5, 3, nkv, device="cuda")[None, None, :, None].to(torch.bfloat16)  # the maximum moves
    out, lse = pia.pi_attn_cross_fwd(q, k, v, kv_len=ints(lens))
    pia.pi_attn_check()
    want = ref.cross(q, k, v, lens, u=2.0 ** -8)
    ref.check(out, want["out"], "out")
    ref.check(lse, want["lse"], "lse")


def test_many_rows_bad_length():
    q, k, v, _ = inputs(3, 20, 20, 130, 40, 64, torch.bfloat16)
    out, lse = pia.pi_attn_cross_fwd(q, k, v, kv_len=ints([40, 41, 7]))
    with pytest.raises(pia.PiAttnError, match="cache_len-out-of-range"):
        pia.pi_attn_check()
    assert out[1].isnan().all() and lse[1].isnan().all()
    want = ref.cross(q, k, v, [40, 0, 7], u=2.0 ** -8)
    for b in (0, 2):
        ref.check(out[b], tuple(x[b] for x in want["out"]), "out")


@pytest.mark.parametrize("nq,nkv,lens", [(1, 9000, None), (3, 20000, [17011]), (40, 12000, None), (64, 16400, [129])])
def test_more_shares_than_a_cluster(nq, nkv, lens):
    """Few rows of one or two heads over many keys: the shares go through the workspace."""
    q, k, v, dout = inputs(1, 2, 1, nq, nkv, 128, torch.bfloat16, seed=nq, poison=math.nan, kv_len=lens)
    assert nq > 32 or pia.load().pi_attn_cross_fwd_workspace_bytes(1, 2, 1, nq, nkv, 128, pia.PI_ATTN_BF16, 0) > 0
    out, lse = pia.pi_attn_cross_fwd(q, k, v, kv_len=ints(lens))
    pia.pi_attn_check()
    want = ref.cross(q, k, v, lens, u=2.0 ** -8)
    ref.check(out, want["out"], "out")
    ref.check(lse, want["lse"], "lse")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_two_streams_at_once(dtype):
    """Calls that overlap on two streams give the bits they give alone."""
    jobs = []
    for seed, (nq, nkv) in enumerate([(1, 5000), (70, 3000)]):
        q, k, v, dout = inputs(2, 4, 2, nq, nkv, 64, dtype, seed=seed)
        jobs.append((q, k, v, dout, ints([nkv, nkv // 3])))

    def one(q, k, v, dout, lens):
        out, lse = pia.pi_attn_cross_fwd(q, k, v, kv_len=lens)
        return (out, lse, *pia.pi_attn_cross_bwd(q, k, v, out, lse, dout, kv_len=lens))

    alone = [one(*j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(one(*jobs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, alone[i]))


def test_without_lse():
    for nq, dtype in ((1, torch.bfloat16), (300, torch.bfloat16), (9, torch.float32)):
        q, k, v, _ = inputs(1, 2, 2, nq, 700, 64, dtype)
        a, lse = pia.pi_attn_cross_fwd(q, k, v, want_lse=False)
        assert lse is None
        assert torch.equal(a, pia.pi_attn_cross_fwd(q, k, v)[0])


def test_many_heads():
    """More (batch, key head) pairs than a grid's second dimension takes."""
    for nq in (1, 2):
        q, k, v, dout = inputs(8200, 8, 8, nq, 3, 64, torch.bfloat16, seed=nq)
        lens = [x % 4 for x in range(8200)]
        out, lse = pia.pi_attn_cross_fwd(q, k, v, kv_len=ints(lens))
        grads = pia.pi_attn_cross_bwd(q, k, v, out, lse, dout, kv_len=ints(lens))
        pia.pi_attn_check()
        pick = [0, 1, 2, 3, 4099, 8190, 8199]
        cut = lambda t: t[pick]  # noqa: E731
        want = ref.cross(cut(q), cut(k), cut(v), [lens[x] for x in pick], cut(dout))
        for name, g in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
            ref.check(cut(g), want[name], name)

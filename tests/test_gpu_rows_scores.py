"""Cross attention and trees of drafted tokens (B200 only) where scores or priors are infinite: a gate
whose bias is infinite (the window or the skips alone remain), keys whose scores are all -inf in a
tile, a share or altogether."""
import math
import random

import pytest
import torch

import periodic_sparse_attention_b200 as pia
from periodic_sparse_attention_b200 import build as pbuild
from tests import rows_ref as ref
from tests.test_gpu_tree import ints, make_tree, unit

pytestmark = pytest.mark.gpu

KINDS = [(torch.bfloat16, "tc"), (torch.bfloat16, "simt"), (torch.float32, "auto")]


@pytest.fixture(scope="module", autouse=True)
def _library():
    pbuild.build()
    pia.load()
    yield
    torch.cuda.synchronize()


# ---- an infinite gate bias -----------------------------------------------------------------------
# B, H, T, cap, d, cache lengths, k, pi, S, ring
TREES = [
    (1, 2, 9, 700, 64, [690], 200, 64, 9, False),           # few heads: the keys in several shares
    (1, 2, 1, 4096, 128, [4000], 2500, 60, 60, False),      # more shares than a cluster joins
    (32, 16, 2, 300, 64, [280] * 32, 130, 32, 8, False),    # one share, a tile of window keys first
    (1, 2, 5, 600, 128, [590], 0, 2, 250, False),           # no window but the token, tiles of skips first
    (30, 16, 5, 600, 64, [590] * 30, 0, 2, 250, False),
    (2, 2, 24, 512, 64, [1000, 512], 140, 64, 8, True),
    (2, 1, 64, 900, 128, [880, 600], 250, 50, 11, False),
]


def tree_inputs(shape, dtype, seed=0):
    B, H, T, cap, d, lens, k, pi, S, ring = shape
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    rng = random.Random(seed)
    return dict(q=r(B, H, T, d).to(dtype), kt=r(B, H, T, d).to(dtype), vt=r(B, H, T, d).to(dtype), kc=r(B, H, cap, d).to(dtype),
                vc=r(B, H, cap, d).to(dtype), w_g=r(H, d) / math.sqrt(d), parent=[make_tree("random", T, rng) for _ in range(B)])


def tree_call(x, shape, b_g, path):
    B, H, T, cap, d, lens, k, pi, S, ring = shape
    got = pia.pi_attn_decode_tree(x["q"], x["kt"], x["vt"], x["kc"], x["vc"], x["w_g"], torch.full((H,), b_g, device="cuda"),
                                  ints(x["parent"]), ints(lens), k, pi, S, ring=ring, path=path)
    pia.pi_attn_check()
    return got


@pytest.mark.parametrize("dtype,path", KINDS)
@pytest.mark.parametrize("gate", [-math.inf, math.inf])
@pytest.mark.parametrize("shape", TREES, ids=str)
def test_infinite_gate(shape, gate, dtype, path):
    """A bias of -inf leaves the skips, +inf the window, each with a prior of 0.  The definition is taken with a
    bias of -60 or 60 and w_g = 0: the other side's weights are then e^-60 of these, far below any bound."""
    B, H, T, cap, d, lens, k, pi, S, ring = shape
    x = tree_inputs(shape, dtype)
    out, lse = tree_call(x, shape, gate, path)
    some = sorted({0, B - 1})
    pick = lambda t: t[some]  # noqa: E731
    want = ref.tree(*(pick(x[n]) for n in ("q", "kt", "vt", "kc", "vc")), torch.zeros_like(x["w_g"]),
                    torch.full((H,), math.copysign(60.0, gate), device="cuda"), [x["parent"][b] for b in some], [lens[b] for b in some],
                    k, pi, S, None, ring, u=unit(dtype, path, d))
    ref.check(pick(out), want["out"], "out")
    ref.check(pick(lse), want["lse"], "lse")
    assert out.isfinite().all() and lse.isfinite().all()


@pytest.mark.parametrize("dtype,gate", [(torch.bfloat16, -math.inf), (torch.bfloat16, math.inf), (torch.float32, math.inf)])
def test_infinite_gate_of_one_node_is_a_decode_step(dtype, gate):
    B, H, d, k, pi, S, lens = 2, 4, 64, 150, 64, 5, [400, 350]
    g = torch.Generator(device="cuda").manual_seed(0)
    kc, vc = (torch.randn(B, H, 400, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    q = torch.randn(B, H, d, generator=g, device="cuda").to(dtype)
    w_g, b_g = torch.randn(H, d, generator=g, device="cuda") / 8, torch.full((H,), gate, device="cuda")
    out, lse = pia.pi_attn_decode(q, kc, vc, w_g, b_g, k, pi, S, cache_len=ints(lens))
    pick = lambda t: torch.stack([t[b, :, lens[b] - 1] for b in range(B)])[:, :, None].contiguous()  # noqa: E731
    o2, l2 = pia.pi_attn_decode_tree(q[:, :, None].contiguous(), pick(kc), pick(vc), kc, vc, w_g, b_g, ints([[-1]] * B),
                                     ints([n - 1 for n in lens]), k, pi, S)
    pia.pi_attn_check()
    # each side is within a rounding of p (2^-8 with bf16 products) and of out of the same value, at most
    # max |v|, so they differ by at most twice two roundings; fp32: sums of fewer than 256 terms, 2 * 280 * 2^-24
    tol = 4 * 2.0 ** -8 if dtype == torch.bfloat16 else 4e-5
    assert out.isfinite().all() and o2.isfinite().all()
    assert (out.float() - o2[:, :, 0].float()).abs().max() <= tol * vc.float().abs().max()
    assert (lse - l2[:, :, 0]).abs().max() <= 1e-4


def test_infinite_gate_of_one_node_is_a_decode_step_in_fp32():
    test_infinite_gate_of_one_node_is_a_decode_step(torch.float32, -math.inf)


@pytest.mark.parametrize("d", [32, 64])
def test_infinite_gate_of_a_chain_is_the_fp32_prefill(d):
    """Rows of the CUDA-core prefill whose first keys have a prior of -inf, against a chain drafted on an
    empty cache (the first pi rows have no skip and are left out)."""
    B, H, n, k, pi, S = 1, 2, 100, 20, 16, 6
    g = torch.Generator(device="cuda").manual_seed(2)
    q, kk, v = (torch.randn(B, H, n, d, generator=g, device="cuda") for _ in range(3))
    w_g, b_g = torch.randn(H, d, generator=g, device="cuda") / 8, torch.full((H,), -math.inf, device="cuda")
    out, lse = pia.pi_attn_fwd(q, kk, v, w_g, b_g, k, pi, S)
    empty = torch.zeros(B, H, 1, d, device="cuda")
    o2, l2 = pia.pi_attn_decode_tree(q, kk, v, empty, empty, w_g, b_g, ints([list(range(-1, n - 1))]), ints([0]), k, pi, S)
    pia.pi_attn_check()
    first = 2 * pi  # the first skip outside the window: 2 * 16 > 20
    assert out[:, :, first:].isfinite().all() and lse[:, :, first:].isfinite().all()
    # sums of at most 6 weights and dot products of d terms: 2 (d + 22) 2^-24 (1 + |score|), far below
    assert (out - o2)[:, :, first:].abs().max() <= 1e-4 and (lse - l2)[:, :, first:].abs().max() <= 1e-4


# ---- scores of -inf --------------------------------------------------------------------------------
# nq of 4 heads to a key head; the first `gone` of nkv keys score -inf
ROWS = [(1, 700, 128), (1, 700, 600), (4, 3000, 400), (5, 700, 130), (16, 9000, 1200), (75, 700, 300), (400, 700, 128), (400, 2000, 1111)]


def scored_inputs(nq, nkv, gone, dtype, how, seed=0, heads=(8, 2)):
    """Keys below `gone` score -inf in every row: by a coordinate of -inf against 1, or by a product of
    finite numbers that overflows; the others' is 0."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    H, Hkv = heads
    q, k, v, dout = (torch.randn(1, h, n, 64, generator=g, device="cuda").to(dtype) for h, n in ((H, nq), (Hkv, nkv), (Hkv, nkv), (H, nq)))
    q[..., 0] = 1.0 if how == "inf" else 2.0 ** 70
    k[..., 0] = 0.0
    k[:, :, :gone, 0] = -math.inf if how == "inf" else -(2.0 ** 70)
    return q, k, v, dout


@pytest.mark.parametrize("how", ["inf", "overflow"])
@pytest.mark.parametrize("dtype,path", KINDS)
@pytest.mark.parametrize("nq,nkv,gone", ROWS)
def test_keys_that_score_minus_infinity(nq, nkv, gone, dtype, path, how):
    """They are keys of weight 0, wherever they lie: the rest's attention remains."""
    q, k, v, _ = scored_inputs(nq, nkv, gone, dtype, how)
    out, lse = pia.pi_attn_cross_fwd(q, k, v, path=path)
    pia.pi_attn_check()
    q0 = q.clone()
    q0[..., 0] = 0.0  # (its partner is 0 in every key that counts)
    want = ref.cross(q0, k[:, :, gone:].contiguous(), v[:, :, gone:].contiguous(), u=unit(dtype, path, 64))
    ref.check(out, want["out"], "out")
    ref.check(lse, want["lse"], "lse")


@pytest.mark.parametrize("how", ["inf", "overflow"])
@pytest.mark.parametrize("dtype,path", KINDS)
@pytest.mark.parametrize("nq,nkv,gone", ROWS)
def test_gradients_with_keys_that_score_minus_infinity(nq, nkv, gone, dtype, path, how):
    """Those keys have no gradient, and leave no trace in the others': rows and keys that only fill up a
    tile must not multiply them."""
    q, k, v, dout = scored_inputs(nq, nkv, gone, dtype, how)
    out, lse = pia.pi_attn_cross_fwd(q, k, v, path=path)
    dq, dk, dv = pia.pi_attn_cross_bwd(q, k, v, out, lse, dout, path=path)
    pia.pi_attn_check()
    want = ref.cross(q, k[:, :, gone:].contiguous(), v[:, :, gone:].contiguous(), None, dout, u=unit(dtype, path, 64))
    for name, t in (("dk", dk), ("dv", dv)):
        assert (t[:, :, :gone] == 0).all(), name
        ref.check(t[:, :, gone:], want[name], name)
    at = 1 if how == "inf" else 0  # (0 times the infinite coordinate is not a number)
    ref.check(dq[..., at:], tuple(t[..., at:] for t in want["dq"]), "dq")


@pytest.mark.parametrize("dtype,path", KINDS)
@pytest.mark.parametrize("nq", [1, 33, 75, 300])
def test_an_infinite_value_of_a_key_that_weighs_nothing(nq, dtype, path):
    """v may hold an infinity where every weight is 0: dv is 0 there, and the others' gradients are theirs
    alone (its dk and every dq are 0 times an infinity)."""
    q, k, v, dout = scored_inputs(nq, 300, 5, dtype, "overflow")
    out, lse = pia.pi_attn_cross_fwd(q, k, v, path=path)
    clean = pia.pi_attn_cross_bwd(q, k, v, out, lse, dout, path=path)
    v[:, :, 2, 3] = math.inf
    _, dk, dv = pia.pi_attn_cross_bwd(q, k, v, out, lse, dout, path=path)
    pia.pi_attn_check()
    assert torch.equal(dv, clean[2]) and torch.equal(dk[:, :, 3:], clean[1][:, :, 3:])


@pytest.mark.parametrize("how", ["inf", "overflow"])
@pytest.mark.parametrize("dtype,path", KINDS)
@pytest.mark.parametrize("nq,nkv", [(1, 700), (5, 128), (16, 9000), (75, 700), (400, 700), (400, 2000)])
def test_rows_without_a_finite_score(nq, nkv, dtype, path, how):
    """A row whose scores are all -inf is one without keys: out 0, lse -inf, and (where no infinity
    enters a product) no gradient, on every path; another head's rows are not touched by it."""
    q, k, v, dout = scored_inputs(nq, nkv, nkv, dtype, how)
    q[:, 4:, :, 0] = 0.0
    k[:, 1, :, 0] = 0.0
    out, lse = pia.pi_attn_cross_fwd(q, k, v, path=path)
    pia.pi_attn_check()
    assert (out[:, :4] == 0).all() and (lse[:, :4] == -math.inf).all()
    want = ref.cross(q[:, 4:].contiguous(), k[:, 1:].contiguous(), v[:, 1:].contiguous(), None, dout[:, 4:].contiguous(), u=unit(dtype, path, 64))
    ref.check(out[:, 4:], want["out"], "out")
    ref.check(lse[:, 4:], want["lse"], "lse")
    dq, dk, dv = pia.pi_attn_cross_bwd(q, k, v, out, lse, dout, path=path)
    pia.pi_attn_check()
    for name, t in (("dq", dq[:, 4:]), ("dk", dk[:, 1:]), ("dv", dv[:, 1:])):
        ref.check(t, want[name], name)
    assert (dk[:, 0] == 0).all() and (dv[:, 0] == 0).all()
    if how == "overflow":
        assert (dq[:, :4] == 0).all()


@pytest.mark.parametrize("dtype,path", KINDS)
def test_nodes_without_a_finite_score(dtype, path):
    """The window off and no skip in reach: out 0 and lse -inf, as cross attention has it."""
    shape = (2, 2, 9, 300, 64, [250, 3], 40, 64, 3, False)  # the second sequence has no skip
    x = tree_inputs(shape, dtype)
    out, lse = tree_call(x, shape, -math.inf, path)
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
    assert out[0].isfinite().all() and lse[0].isfinite().all() and (out[0] != 0).any(dim=-1).all()


@pytest.mark.parametrize("dtype,path", KINDS)
@pytest.mark.parametrize("nq", [1, 20, 75, 400])
def test_a_nan_stays(nq, dtype, path):
    """A NaN in a query is a NaN in its row and in no other; one in a key is a NaN in every row."""
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(1, h, n, 64, generator=g, device="cuda").to(dtype) for h, n in ((2, nq), (2, 900), (2, 900)))
    clean = pia.pi_attn_cross_fwd(q, k, v, path=path)
    q[0, 0, nq // 2, 3] = math.nan
    k[0, 1, 333, 5] = math.nan
    out, lse = pia.pi_attn_cross_fwd(q, k, v, path=path)
    pia.pi_attn_check()
    bad = torch.zeros(2, nq, dtype=torch.bool, device="cuda")
    bad[0, nq // 2] = bad[1] = True
    assert torch.equal(out[0].isnan().all(dim=-1), bad) and torch.equal(lse[0].isnan(), bad)
    assert torch.equal(out[0][~bad], clean[0][0][~bad]) and torch.equal(lse[0][~bad], clean[1][0][~bad])

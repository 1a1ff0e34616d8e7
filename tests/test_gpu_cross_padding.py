"""Gradients of cross attention (B200 only) behind a sequence's states: exact zeros, whatever the
other operands hold."""
import math

import pytest
import torch

import periodic_sparse_attention_b200 as pia
from periodic_sparse_attention_b200 import build as pbuild

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    pbuild.build()
    pia.load()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype,path", [(torch.bfloat16, "tc"), (torch.bfloat16, "simt"), (torch.float32, "auto")])
@pytest.mark.parametrize("nq,nkv,n,d", [(1, 130, 129, 64), (40, 300, 77, 128), (200, 300, 290, 64), (700, 260, 1, 128)])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("where", ["q", "dout"])
def test_padding_has_no_gradient(where, bad, nq, nkv, n, d, dtype, path):
    """dk and dv are zero behind kv_len even where a row of q or dout is not finite (a step of a
    diverging run): 0 times an infinity must not get in."""
    g = torch.Generator(device="cuda").manual_seed(nq)
    q, k, v, dout = (torch.randn(2, h, m, d, generator=g, device="cuda").to(dtype) for h, m in ((4, nq), (2, nkv), (2, nkv), (4, nq)))
    lens = torch.tensor([n, nkv], dtype=torch.int32, device="cuda")
    out, lse = pia.pi_attn_cross_fwd(q, k, v, kv_len=lens, path=path)
    clean = pia.pi_attn_cross_bwd(q, k, v, out, lse, dout, kv_len=lens, path=path)
    dict(q=q, dout=dout)[where][0, 1, nq // 2, 5] = bad
    dq, dk, dv = pia.pi_attn_cross_bwd(q, k, v, out, lse, dout, kv_len=lens, path=path)
    pia.pi_attn_check()
    for name, t in (("dk", dk), ("dv", dv)):
        assert (t[0, :, n:] == 0).all(), name
    for a, b in zip((dq, dk, dv), clean):  # the other sequence is not touched
        assert torch.equal(a[1], b[1])

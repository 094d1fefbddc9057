"""Linear attention over rows of up to 64 tokens in bf16: the products under the decay keep 16 bits, so that one
token's outputs are not off as a whole.

Tolerance: the result's rounding, 2^-8 |o| at most; the products as two bf16 numbers are off by 2^-16 of each term; the
state as an operand is rounded to bf16, 2^-8 of each of its terms q_r S_rc.  Element by element, with fp32 sums of up
to 128 + 64 terms at 2^-24 each."""
import pytest
import torch

import chunk_wise_weight_gate_b200 as pkg
from tests import block_ref as ref
from tests.test_gpu_block_ops import attn_case, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,H,Hkv,Dk,Dv,docs", [
    (1, 1, 1, 1, 128, 128, ()), (3, 1, 2, 1, 64, 64, ()), (1, 1, 20, 20, 128, 64, ()), (2, 7, 3, 3, 64, 128, (9,)),
    (1, 33, 2, 1, 128, 128, (0, 5, 31, 32)), (1, 64, 2, 2, 64, 64, ()), (2, 64, 1, 1, 128, 128, (63, 100)), (1, 40, 4, 4, 128, 64, ()),
])
@pytest.mark.parametrize("state", [False, True])
def test_short_rows(B, T, H, Hkv, Dk, Dv, docs, state):
    cfg, q, k, v, ld, S0, ds = attn_case(B, T, H, Hkv, Dk, Dv, "bf16", docs, state)
    x = ref.leaves(q, k, v, S0)
    want, _ = ref.linear_attention(x[0], x[1], x[2], ld.cpu(), cfg.scale, docs, x[3])
    O = pkg.linear_attention(cfg, q, k, v, ld, ds, S0=S0)

    def within(got, want, terms, from_state):
        got, want = got.double().cpu(), want.detach()
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -15 + 192 * 2.0 ** -24) * terms + 2.0 ** -8 * 1.01 * from_state
        assert bool(((got - want).abs() <= tol).all())

    a = [t.detach().abs() for t in x[:3]]
    s = None if S0 is None else x[3].detach().abs()
    terms, _ = ref.linear_attention(*a, ld.cpu(), cfg.scale, docs, s)
    alone, _ = ref.linear_attention(*a, ld.cpu(), cfg.scale, docs)
    within(O, want, terms, terms - alone)
    # the gradients are the same passes over other operands: gq sees gO, v and k, gk and gv see the tokens after
    gO = ref.rand(20, B, T, H, Dv, dtype=torch.bfloat16).cuda()
    g = pkg.linear_attention_backward(cfg, q, k, v, ld, ds, gO, S0=S0)
    grads = torch.autograd.grad((want * gO.double().cpu()).sum(), x[:3])
    y = ref.leaves(q.abs(), k.abs(), v.abs(), None if S0 is None else S0.abs())
    most, _ = ref.linear_attention(y[0], y[1], y[2], ld.cpu(), cfg.scale, docs, y[3])
    bounds = torch.autograd.grad((most * gO.abs().double().cpu()).sum(), y[:3])
    y0 = ref.leaves(q.abs(), k.abs(), v.abs())
    most0, _ = ref.linear_attention(y0[0], y0[1], y0[2], ld.cpu(), cfg.scale, docs)
    bounds0 = torch.autograd.grad((most0 * gO.abs().double().cpu()).sum(), y0[:3])
    for n, w, m, m0 in zip("qkv", grads, bounds, bounds0):
        within(g[n], w, m, m - m0)
    assert status() == 0

"""The accuracy of the fp32 states that linear attention gives out on the tensor cores.

Tolerance 1e-6 of the 2-norm.  A key times its weight w goes into the product as three bf16 parts: the key times
the power of two nearest to w, exact, and two parts of the key times the rest y, |y| <= w/3.  A rounding to
bf16 is off by 0.42 * 2^-8 = 1.6e-3 of the value (rms, half a step at most), so y as two bf16 numbers by
the square, 2.6e-6 of y, and the second part, up to twice as large as a rounding leaves, by some 3.5e-6 of y; over w's
mantissas y is 0.19 of w (rms): 0.19 * 4.4e-6 = 8.3e-7 of each term, independent from term to term.  The fp32 sums
over a chunk and the chunks add some 1e-7."""
import pytest
import torch

import chunk_wise_weight_gate_b200 as pkg
from tests import block_ref as ref
from tests.test_gpu_block_ops import attn_case, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,H,Hkv,Dk,Dv,docs", [
    (2, 700, 4, 2, 128, 128, ()), (1, 1300, 2, 2, 64, 64, (500,)), (2, 300, 3, 1, 64, 128, (20, 450)), (1, 900, 2, 1, 128, 64, ()),
    (1, 127, 8, 8, 128, 128, ()), (1, 1, 4, 4, 64, 64, ()),
])
def test_states_are_good_to_a_millionth(B, T, H, Hkv, Dk, Dv, docs):
    decay = [-(2.0 ** -(1 + 11 * h / H)) for h in range(H)]
    cfg, q, k, v, ld, S0, ds = attn_case(B, T, H, Hkv, Dk, Dv, "bf16", docs, True, decay)
    x = ref.leaves(q, k, v, S0)
    want, want_S = ref.linear_attention(x[0], x[1], x[2], ld.cpu(), cfg.scale, docs, x[3])
    _, S = pkg.linear_attention(cfg, q, k, v, ld, ds, S0=S0, S_final=True)
    assert ref.relative(S, want_S) <= 1e-6
    gO, gS = ref.rand(20, B, T, H, Dv, dtype=torch.bfloat16).cuda(), ref.rand(21, B, H, Dk, Dv, std=0.1).cuda()
    g = pkg.linear_attention_backward(cfg, q, k, v, ld, ds, gO, S0=S0, gS_final=gS)
    loss = (want * gO.double().cpu()).sum() + (want_S * gS.double().cpu()).sum()
    assert ref.relative(g["S0"], torch.autograd.grad(loss, x[3])[0]) <= 1e-6
    assert status() == 0


@pytest.mark.parametrize("B,T,H,Dk,Dv", [(1, 8192, 20, 128, 128), (1, 20000, 2, 128, 64), (1, 9000, 4, 64, 128), (1, 2500, 150, 64, 64)])
def test_states_of_rows_in_segments(B, T, H, Dk, Dv):
    # against the fp32 pass, whose products and sums round at 2^-24: some 2e-7
    decay = [-(2.0 ** -(2 + 9 * h / H)) for h in range(H)]
    for docs in ((), (T // 3, T // 2)):
        cfg, q, k, v, ld, S0, ds = attn_case(B, T, H, H, Dk, Dv, "bf16", docs, True, decay)
        f32 = pkg.LinearAttentionConfig(B, T, H, H, Dk, Dv, cfg.scale, "f32")
        gO = ref.rand(20, B, T, H, Dv, dtype=torch.bfloat16).cuda()
        _, S = pkg.linear_attention(cfg, q, k, v, ld, ds, S0=S0, S_final=True)
        _, want = pkg.linear_attention(f32, q.float(), k.float(), v.float(), ld, ds, S0=S0, S_final=True)
        assert ref.relative(S, want.cpu()) <= 1.2e-6
        g = pkg.linear_attention_backward(cfg, q, k, v, ld, ds, gO, S0=S0)
        w = pkg.linear_attention_backward(f32, q.float(), k.float(), v.float(), ld, ds, gO.float(), S0=S0)
        assert ref.relative(g["S0"], w["S0"].cpu()) <= 1.2e-6
    assert status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H,D", [(1, 16384, 16, 64), (1, 8192, 40, 128), (2, 3000, 160, 64)])
def test_states_of_long_memories(B, T, H, D, dtype):
    # decays of any mantissa, that remember up to 16k tokens: the same factor is multiplied on up to 512 times.
    # S_T = sum of gamma^{T-1-t} k_t v_t^T, by its closed form in 64 bits; fp32: sums of up to 512 chunks, each rounded at
    # 2^-24 of a state that grows as its root: 1e-6
    cfg, q, k, v, _, _, _ = attn_case(B, T, H, H, D, D, dtype)
    ld = -torch.exp2(-13.0 * torch.rand(H, generator=torch.Generator().manual_seed(6))).cuda()
    _, S = pkg.linear_attention(cfg, q, k, v, ld, S_final=True)
    t = torch.arange(T - 1, -1, -1, device="cuda", dtype=torch.float64)
    for h in range(H):
        w = torch.exp(ld[h].double() * t)[None, :, None]
        want = torch.matmul((k[:, :, h].double() * w).transpose(1, 2), v[:, :, h].double())
        assert ref.relative(S[:, h], want.cpu()) <= 1.2e-6, h
    assert status() == 0


def test_states_after_a_walk_by_tokens():
    # a bad value in a finished document: the state after 4000 more tokens, each times gamma, is as exact
    T, H, D = 4500, 12, 64
    cfg, q, k, v, _, _, ds = attn_case(1, T, H, H, D, D, "bf16", (500,))
    ld = -torch.exp2(-4.0 - 9.0 * torch.rand(H, generator=torch.Generator().manual_seed(7))).cuda()
    k[0, 3, :, 1] = float("nan")
    _, S = pkg.linear_attention(cfg, q, k, v, ld, ds, S_final=True)
    t = torch.arange(T - 501, -1, -1, device="cuda", dtype=torch.float64)
    for h in range(H):
        w = torch.exp(ld[h].double() * t)[:, None]
        want = (k[0, 500:, h].double() * w).t() @ v[0, 500:, h].double()
        assert ref.relative(S[0, h], want.cpu()) <= 2e-6, h
    assert status() == 0

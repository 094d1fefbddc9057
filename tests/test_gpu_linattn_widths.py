"""Linear attention where widths differ and heads are shared, over rows of many chunks and segments, and
gradients written into views of one projection's gradient.  Tolerances as in test_gpu_block_ops.py."""
import pytest
import torch

import chunk_wise_weight_gate_b200 as pkg
from tests import block_ref as ref
from tests.test_gpu_block_ops import attn_case, check_attn, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [
    (2, 600, 4, 2, 64, 128, (130, 700, 1199), True), (1, 1300, 4, 1, 128, 64, (640, 641), True),
    (1, 1000, 2, 1, 64, 128, (), False), (2, 300, 6, 3, 128, 64, (0, 128, 427), True), (1, 515, 2, 2, 64, 128, (511,), True),
    (1, 515, 2, 2, 128, 64, (384,), False),
])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_widths_that_differ(case, dtype):
    check_attn(case, dtype)


# rows in one segment, in up to eight (summed by each segment), in more (k_prefix); whole rows beside cut ones
@pytest.mark.parametrize("B,T,H,Hkv", [(1, 1500, 150, 50), (2, 5000, 20, 20), (1, 4100, 32, 8), (1, 20000, 2, 1), (3, 2500, 60, 60)])
@pytest.mark.parametrize("Dk,Dv", [(64, 128), (128, 64)])
def test_widths_that_differ_over_many_segments(B, T, H, Hkv, Dk, Dv):
    docs = sorted(set(torch.randint(0, B * T, (9,), generator=torch.Generator().manual_seed(4)).tolist()))
    for d, state in ((docs, True), ((), True), (docs, False)):
        cfg, q, k, v, _, S0, ds = attn_case(B, T, H, Hkv, Dk, Dv, "bf16", d, state)
        ld = torch.log1p(-torch.exp2(-4.0 - 7.0 * torch.arange(H) / H)).cuda()
        f32 = pkg.LinearAttentionConfig(B, T, H, Hkv, Dk, Dv, cfg.scale, "f32")
        gO = ref.rand(20, B, T, H, Dv, dtype=torch.bfloat16).cuda()
        gS = ref.rand(21, B, H, Dk, Dv).cuda() if state else None
        O, S = pkg.linear_attention(cfg, q, k, v, ld, ds, S0=S0, S_final=True)
        want, want_S = pkg.linear_attention(f32, q.float(), k.float(), v.float(), ld, ds, S0=S0, S_final=True)
        assert ref.relative(O, want.cpu()) <= 6e-3 and ref.relative(S, want_S.cpu()) <= 1e-5
        g = pkg.linear_attention_backward(cfg, q, k, v, ld, ds, gO, S0=S0, gS_final=gS)
        w = pkg.linear_attention_backward(f32, q.float(), k.float(), v.float(), ld, ds, gO.float(), S0=S0, gS_final=gS)
        for n in g:
            assert ref.relative(g[n], w[n].cpu()) <= (1e-5 if n == "S0" else 6e-3), n
    assert status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,H,Hkv,Dk,Dv", [(2, 400, 4, 4, 64, 64), (1, 1300, 4, 2, 128, 64), (2, 90, 4, 1, 40, 56), (3, 1, 2, 2, 128, 128)])
def test_gradients_into_one_projections_gradient(B, T, H, Hkv, Dk, Dv, dtype):
    cfg, q, k, v, ld, S0, ds = attn_case(B, T, H, Hkv, Dk, Dv, dtype, (T // 2,), True)
    gO = ref.rand(20, B, T, H, Dv, dtype=q.dtype).cuda()
    want = pkg.linear_attention_backward(cfg, q, k, v, ld, ds, gO, S0=S0)
    widths = (H * Dk, Hkv * Dk, Hkv * Dv, 24)
    fused = torch.full((B, T, sum(widths)), 7.0, dtype=q.dtype, device="cuda")
    gq, gk, gv, rest = fused.split(widths, -1)
    gq, gk, gv = gq.unflatten(-1, (H, Dk)), gk.unflatten(-1, (Hkv, Dk)), gv.unflatten(-1, (Hkv, Dv))
    got = pkg.linear_attention_backward(cfg, q, k, v, ld, ds, gO, S0=S0, gq=gq, gk=gk, gv=gv)
    assert got["q"] is gq and got["k"] is gk and got["v"] is gv
    assert all(torch.equal(got[n], want[n]) for n in want) and bool((rest == 7.0).all())
    for bad in (gq.float() if dtype == "bf16" else gq.bfloat16(), gq[:, :, :1], gq.transpose(2, 3)):
        with pytest.raises(ValueError):
            pkg.linear_attention_backward(cfg, q, k, v, ld, ds, gO, S0=S0, gq=bad)
    with pytest.raises(pkg.IptttError):  # q's own place: later passes still read it
        pkg.linear_attention_backward(cfg, q, k, v, ld, ds, gO, S0=S0, gq=q)
    assert status() == 0

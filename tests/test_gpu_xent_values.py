"""Logits that are not finite in the softmax cross entropy: lse and loss are what their definition
gives (NaN from a NaN, an infinity from infinities), and other tokens are as ever."""
import math

import pytest
import torch

import chunk_wise_weight_gate_b200 as pkg
from tests.test_gpu_block_ops import status, xent_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("word", [0, 5, 255, 256, 700, 999])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_cross_entropy_of_a_head_that_is_not_finite(word, bad, dtype):
    N, V, d = 150, 1000, 64
    cfg, H, W, t = xent_case(N, V, d, dtype)
    W[word, 7] = bad  # that word's logit: NaN, or an infinity of H[:, 7]'s sign
    t[3] = word
    loss, lse = pkg.cross_entropy(cfg, H, W, t)
    logits = H.double().cpu() @ W.double().cpu().t()
    want = logits.logsumexp(1)
    want_loss = torch.where(t.cpu() >= 0, want - logits.gather(1, t.cpu().clamp(min=0)[:, None])[:, 0], 0.0)
    for got, w in ((lse, want), (loss, want_loss)):
        got = got.double().cpu()
        assert torch.equal(got.isnan(), w.isnan()) and torch.equal(got.isinf(), w.isinf())
        assert torch.equal(got[got.isinf()], w[w.isinf()])
        ok = w.isfinite()
        if bool(ok.any()):
            assert float((got[ok] - w[ok]).abs().max()) <= 1e-5 * max(1.0, float(w[ok].abs().max()))
    assert status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V", [(40, 300), (300, 3)])
def test_cross_entropy_of_a_token_that_is_not_finite(N, V, dtype):
    cfg, H, W, t = xent_case(N, V, 64, dtype)
    t[1], t[N // 2] = 2, -100
    loss, lse = pkg.cross_entropy(cfg, H, W, t)
    gl = torch.full((N,), 1.0 / N, device="cuda")
    want = pkg.cross_entropy_backward(cfg, H, W, t, lse, gl)["H"]
    h = H.clone()
    h[1], h[N // 2] = math.nan, math.nan  # one that takes part, one that does not
    loss2, lse2 = pkg.cross_entropy(cfg, h, W, t)
    assert bool(lse2[1].isnan()) and bool(loss2[1].isnan()) and bool(lse2[N // 2].isnan()) and float(loss2[N // 2]) == 0.0
    keep = torch.ones(N, dtype=torch.bool)
    keep[1] = keep[N // 2] = False
    assert torch.equal(loss2[keep], loss[keep]) and torch.equal(lse2[keep], lse[keep])
    g = pkg.cross_entropy_backward(cfg, h, W, t, lse2, gl)
    keep[N // 2] = True
    assert torch.equal(g["H"][keep], want[keep]) and bool(g["H"][1].isnan().all()) and bool(g["W"].isnan().all())
    assert status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,d,piece", [(150, 1000, 64, 256), (5, 300, 320, 0), (700, 2000, 96, 512)])
def test_cross_entropy_rows_left_out_of_a_head_that_is_not_finite(N, V, d, piece, dtype):
    cfg, H, W, t = xent_case(N, V, d, dtype, piece=piece)
    for bad in (math.nan, math.inf):
        w = W.clone()
        w[V // 2, 1] = bad
        loss, lse = pkg.cross_entropy(cfg, H, w, t)
        g = pkg.cross_entropy_backward(cfg, H, w, t, lse, torch.full((N,), 1.0 / N, device="cuda"))
        out = t == -100
        assert bool(out.any()) and not loss[out].any() and not g["H"][out].any()
    assert status() == 0

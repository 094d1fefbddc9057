"""The operators around the layer together with the layer, as a block of a model uses them:
norms and rotation -> linear attention -> the TTT layer -> loss, and the gradients back
through all of them; decoding against the prompt; the calls captured into graphs.

Tolerances.  fp32: each operator's error is at most 1e-5 (test_gpu_block_ops.py; the layer's is
1e-5 too), four of them in a chain and their gradients back: 1e-4 of the 2-norm.  bf16: the
layer's bar is 2e-2, the others' 6e-3 each, so the chain's is 2e-2 + 3 * 6e-3 < 4e-2."""
import numpy as np
import pytest
import torch

import chunk_wise_weight_gate_b200 as pkg
from chunk_wise_weight_gate_b200 import ipttt as ip
from oracle import ipttt_backward as obwd
from oracle import ipttt_oracle as orc
from tests import block_ref as ref
from tests.gpu_util import WEIGHTS, case, to_np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,B,T,heads,D,F,C,V,tol", [("f32", 2, 45, 4, 16, 96, 16, 301, 1e-4),
                                                        ("bf16", 2, 300, 4, 64, 512, 128, 1001, 4e-2)])
def test_a_block_and_its_loss_with_gradients(dtype, B, T, heads, D, F, C, V, tol):
    d, dt = heads * D, torch.float32 if dtype == "f32" else torch.bfloat16
    docs = [7, 20, T - 1, T + 11]
    lcfg, inp = case(B, T, C, d, F, dtype=dtype, eta=2e-2, clip=0.0, docs=docs)
    layer = {k: inp[k].cuda() for k in WEIGHTS}
    X0, starts = inp["X0"].cuda(), inp["doc_starts"].cuda()
    qkv = ref.rand(1, B, T, 3 * d, dtype=dt).cuda()
    q, k, v = (t.unflatten(-1, (heads, D)) for t in qkv.split(d, -1))
    wq, wk = ((1 + ref.rand(2 + i, D, std=0.2)).to(dt).cuda() for i in range(2))
    inv = (1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).cuda()
    pos = torch.arange(T, device="cuda").expand(B, T).contiguous()
    ld = torch.log1p(-torch.exp2(-3.0 - torch.arange(heads))).float().cuda()
    W = ref.rand(9, V, d, std=2.0 * d ** -0.5, dtype=dt).cuda()
    targets = torch.randint(0, V, (B * T,), generator=torch.Generator().manual_seed(3))
    targets[::7] = -100
    gloss = torch.full((B * T,), 1.0 / int((targets >= 0).sum())).cuda()
    scale = D ** -0.5

    # the program: forwards
    qcfg = pkg.QKNormRopeConfig(B, T, heads, heads, D, D, 1e-6, dtype=dtype)
    acfg = pkg.LinearAttentionConfig(B, T, heads, heads, D, D, scale, dtype)
    xcfg = pkg.CrossEntropyConfig(B * T, V, d, dtype=dtype)
    t = targets.cuda()
    qn, kn = pkg.qk_norm_rope(qcfg, q, k, wq, wk, inv, pos)
    A = pkg.linear_attention(acfg, qn, kn, v, ld, starts)
    H = A.view(B, T, d)
    O = ip.forward(lcfg, H, X0, *(layer[n] for n in WEIGHTS), starts)
    y = O.view(B * T, d)
    loss, lse = pkg.cross_entropy(xcfg, y, W, t)
    # and back
    gx = pkg.cross_entropy_backward(xcfg, y, W, t, lse, gloss)
    gl = ip.backward(lcfg, H, X0, *(layer[n] for n in WEIGHTS), starts, gx["H"].view(B, T, d))
    ga = pkg.linear_attention_backward(acfg, qn, kn, v, ld, starts, gl["H"].to(dt).view(B, T, heads, D))
    gq = pkg.qk_norm_rope_backward(qcfg, q, k, wq, wk, inv, pos, ga["q"], ga["k"])
    torch.cuda.synchronize()
    assert pkg.get_status() == 0

    # the same in 64 bits
    x = ref.leaves(q, k, v, wq, wk)
    qr, kr = (ref.qk_one(x[i], x[3 + i], inv.cpu(), pos.cpu(), D, 1e-6, False) for i in range(2))
    Ar, _ = ref.linear_attention(qr, kr, x[2], ld.cpu(), scale, docs)
    Hr = Ar.detach().reshape(B, T, d).numpy()
    w = {n: to_np(inp[n]) for n in WEIGHTS}
    a = (Hr, to_np(inp["X0"]), w["Wgate"], w["Wup"], w["Wdown0"], w["conv_w"], w["Wtarget"], C, np.asarray(docs), 2e-2, 0.0)
    yr = torch.tensor(orc.layer_forward(*a)["O"]).view(B * T, d).requires_grad_()
    Wr = W.double().cpu().requires_grad_()
    lr, _ = ref.cross_entropy(yr, Wr, targets)
    gy, gW = torch.autograd.grad((lr * gloss.double().cpu()).sum(), (yr, Wr))
    glr = obwd.layer_backward(*a, gy.view(B, T, d).numpy())
    grads = torch.autograd.grad((Ar * torch.tensor(glr["H"]).view(B, T, heads, D)).sum(), x)
    kept = targets >= 0
    assert ref.relative(loss[kept.cuda()], lr[kept]) <= tol
    # Behind the softmax errors grow: an error of y by tol of its 2-norm moves a logit l = y . w, sums of
    # d products of which each moves by tol, by tol times the logits' own size (rms), and p = exp(l -
    # lse) by that much of itself.  Every gradient is linear in p, so their bar is tol (1 + rms l).
    tol *= 1.0 + float((yr.detach() @ Wr.detach().t()).square().mean().sqrt())
    assert ref.relative(gx["W"], gW) <= tol
    for n in WEIGHTS:
        assert ref.relative(gl[n], torch.tensor(glr[n])) <= tol, n
    for name, got, want in zip(("q", "k", "v", "wq", "wk"), (gq["q"], gq["k"], ga["v"], gq["wq"], gq["wk"]), grads):
        assert ref.relative(got, want) <= tol, name


def test_tokens_one_by_one_are_the_prompt():
    # a prompt of 200 tokens, then 20 more one by one, against one call over the 220
    B, T, n, heads, Hk, D = 3, 220, 200, 8, 4, 128
    q, k, v = (ref.rand(i, B, T, h, D, dtype=torch.bfloat16).cuda() for i, h in enumerate((heads, Hk, Hk)))
    wq, wk = ((1 + ref.rand(5 + i, D, std=0.2)).bfloat16().cuda() for i in range(2))
    inv = (1e6 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).cuda()
    pos = (torch.arange(T, device="cuda") + 100000).expand(B, T).contiguous()
    ld = torch.linspace(-0.2, -0.001, heads).cuda()

    def norm(lo, hi):
        cfg = pkg.QKNormRopeConfig(B, hi - lo, heads, Hk, D, D)
        return pkg.qk_norm_rope(cfg, q[:, lo:hi].contiguous(), k[:, lo:hi].contiguous(), wq, wk, inv, pos[:, lo:hi].contiguous())

    def cfg(t):
        return pkg.LinearAttentionConfig(B, t, heads, Hk, D, D, D ** -0.5)

    qa, ka = norm(0, T)
    whole, S_whole = pkg.linear_attention(cfg(T), qa, ka, v, ld, S_final=True)
    qp, kp = norm(0, n)
    assert torch.equal(qp, qa[:, :n]) and torch.equal(kp, ka[:, :n])
    _, S = pkg.linear_attention(cfg(n), qp, kp, v[:, :n].contiguous(), ld, S_final=True)
    for t in range(n, T):
        qt, kt = norm(t, t + 1)
        o = pkg.linear_attention_step(cfg(1), S, qt[:, 0], kt[:, 0], v[:, t], ld)
        assert ref.relative(o, whole[:, t].double().cpu()) <= 6e-3
    assert ref.relative(S, S_whole.double().cpu()) <= 1e-5
    assert pkg.get_status() == 0


def test_captured_and_replayed_calls_share_a_workspace():
    B, T, heads, D, N, V = 2, 700, 4, 128, 1400, 3001
    acfg = pkg.LinearAttentionConfig(B, T, heads, heads, D, D, D ** -0.5)
    xcfg = pkg.CrossEntropyConfig(N, V, heads * D, piece=1024)
    qcfg = pkg.QKNormRopeConfig(B, T, heads, heads, D, D)
    ws = torch.empty(max(pkg.linear_attention_workspace_size(acfg, backward=True),
                         pkg.cross_entropy_workspace_size(xcfg), pkg.cross_entropy_workspace_size(xcfg, backward=True)),
                     dtype=torch.uint8, device="cuda")
    q, k, v, gO = (ref.rand(i, B, T, heads, D, dtype=torch.bfloat16).cuda() for i in range(4))
    w = torch.ones(D, device="cuda", dtype=torch.bfloat16)
    inv = (1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).cuda()
    pos = torch.arange(T, device="cuda").expand(B, T).contiguous()
    ld = torch.full((heads,), -0.02, device="cuda")
    docs = torch.tensor([100, 900], dtype=torch.int32, device="cuda")
    W = ref.rand(8, V, heads * D, std=0.1, dtype=torch.bfloat16).cuda()
    t = torch.randint(0, V, (N,), generator=torch.Generator().manual_seed(1)).cuda()
    S0 = ref.rand(9, B, heads, D, D).cuda()
    g1 = torch.full((N,), 1.0 / N, device="cuda")

    def attention():
        a, b = pkg.qk_norm_rope(qcfg, q, k, w, w, inv, pos)
        O, S = pkg.linear_attention(acfg, a, b, v, ld, docs, S0=S0, S_final=True, workspace=ws)
        g = pkg.linear_attention_backward(acfg, a, b, v, ld, docs, gO, S0=S0, gS_final=S, workspace=ws)
        h = pkg.qk_norm_rope_backward(qcfg, q, k, w, w, inv, pos, g["q"], g["k"])
        return [O, S, g["v"], g["S0"], h["q"], h["wk"]]

    def loss():
        H = v.view(N, heads * D)
        l, lse = pkg.cross_entropy(xcfg, H, W, t, workspace=ws)
        g = pkg.cross_entropy_backward(xcfg, H, W, t, lse, g1, workspace=ws)
        return [l, lse, g["H"], g["W"]]

    graphs = []
    for f in (attention, loss):
        f()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = f()
        graphs.append((g, out, f))
    for seed in (20, 40):  # other inputs in the same places; the graphs in turn, on one workspace
        for i, x in enumerate((q, k, v, gO)):
            x.copy_(ref.rand(seed + i, *x.shape, dtype=torch.bfloat16))
        for _ in range(2):
            for g, _, _ in graphs:
                g.replay()
        torch.cuda.synchronize()
        for g, out, f in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, f()))
    torch.cuda.synchronize()
    assert pkg.get_status() == 0
    del graphs


@pytest.mark.parametrize("dtype,B,T,heads,D", [("bf16", 1, 4000, 2, 128), ("bf16", 1, 1100, 150, 64), ("f32", 1, 1500, 3, 96)])
def test_captured_rows_in_many_segments(dtype, B, T, heads, D):
    # states of segments, their prefix and the pass (which may start early) in one graph; rows cut and whole
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    cfg = pkg.LinearAttentionConfig(B, T, heads, heads, D, D, D ** -0.5, dtype)
    q, k, v, gO = (ref.rand(i, B, T, heads, D, dtype=dt).cuda() for i in range(4))
    ld = torch.full((heads,), -0.003, device="cuda")
    docs = torch.tensor([T // 3, T - 7], dtype=torch.int32, device="cuda")
    S0 = ref.rand(9, B, heads, D, D).cuda()

    def run(S):
        O, S = pkg.linear_attention(cfg, q, k, v, ld, docs, S0=S, S_final=S)
        g = pkg.linear_attention_backward(cfg, q, k, v, ld, docs, gO, S0=S0, gS_final=S)
        return [O, S, *g.values()]

    S = S0.clone()
    run(S)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(S)
    for seed in (20, 40):
        for i, x in enumerate((q, k, v, gO)):
            x.copy_(ref.rand(seed + i, *x.shape, dtype=dt))
        for _ in range(3):  # the state in place: each replay starts anew
            S.copy_(S0)
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, run(S0.clone())))
    assert pkg.get_status() == 0
    del graph


def test_two_calls_at_once():
    B, T, heads, D, N, V = 1, 6000, 8, 128, 1200, 9000
    acfg = pkg.LinearAttentionConfig(B, T, heads, heads, D, D, D ** -0.5)
    xcfg = pkg.CrossEntropyConfig(N, V, 256)
    q, k, v, gO = (ref.rand(i, B, T, heads, D, dtype=torch.bfloat16).cuda() for i in range(4))
    ld = torch.full((heads,), -0.01, device="cuda")
    H, W = (ref.rand(i, n, 256, std=0.3, dtype=torch.bfloat16).cuda() for i, n in ((5, N), (6, V)))
    t = torch.randint(0, V, (N,), generator=torch.Generator().manual_seed(1)).cuda()
    g1 = torch.full((N,), 1.0 / N, device="cuda")

    def attention(stream=None):
        O, S = pkg.linear_attention(acfg, q, k, v, ld, S_final=True, stream=stream)
        return [O, S, *pkg.linear_attention_backward(acfg, q, k, v, ld, None, gO, stream=stream).values()]

    def loss(stream=None):
        l, lse = pkg.cross_entropy(xcfg, H, W, t, stream=stream)
        return [l, lse, *pkg.cross_entropy_backward(xcfg, H, W, t, lse, g1, stream=stream).values()]

    want_a, want_l = attention(), loss()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(5):
        got += [(want_a, attention(streams[0])), (want_l, loss(streams[1])), (want_a, attention(streams[2]))]
    torch.cuda.synchronize()
    for want, out in got:
        assert all(torch.equal(a, b) for a, b in zip(want, out))
    assert pkg.get_status() == 0

"""The operators around the layer against plain 64-bit implementations (block_ref).

Tolerances.  A stored value is off by at most half a step of its type: 2^-8 relative for
bf16, 2^-24 for fp32.  fp32 sums of n terms in blocks add a few 2^-24 per doubling of n.
 * fp32 calls: 2e-6 of the 2-norm for one pass (some ten roundings of 2^-24 = 6e-8 in
   sequence, sums in blocks), 1e-5 where a state or a loss is summed over many tokens.
 * norms and rotation, bf16: only the result is rounded: element by element 2^-8 |y|, and
   1e-5 of the vector's norm for the fp32 arithmetic and the angle (2^-24 of a turn).
 * linear attention, bf16: the products under the decay, the state (as operands) and the
   result are each rounded once, so element by element at most 2^-8 (|o| + 2 sum |terms|),
   where sum |terms| is the same pass over absolute values; roundings are independent,
   so the 2-norm of the error is at most sqrt(2) 2^-8 of the result's where the terms are
   (3 times 2^-8 / sqrt(3) covers it): 6e-3.  Its fp32 states carry operands split
   in two bf16 halves (2^-17 a term) and fp32 sums: 1e-5.
 * cross entropy, bf16: products of bf16 are exact in fp32, sums over d in fp32: loss and lse
   1e-5; p is rounded to bf16 (2^-8) before its two products, and the result (2^-8):
   independent, so 2^-8 sqrt(2) = 5.6e-3 of the 2-norm.
"""
import math

import pytest
import torch

import chunk_wise_weight_gate_b200 as pkg
from tests import block_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def status():
    torch.cuda.synchronize()
    return pkg.get_status()


# ---------------------------------------------------------------- norms and rotation

def qk_case(B, T, Hq, Hk, D, R, dtype, interleaved=False, far=0, seed=1):
    cfg = pkg.QKNormRopeConfig(B=B, T=T, Hq=Hq, Hk=Hk, D=D, R=R, eps=1e-5, interleaved=interleaved, dtype=dtype)
    dt = DT[dtype]
    qkv = ref.rand(seed, B, T, (Hq + 2 * Hk) * D, std=1.5, dtype=dt).cuda()
    q = qkv[..., :Hq * D].unflatten(-1, (Hq, D))
    k = qkv[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D))
    wq, wk = (1 + ref.rand(seed + 1, D, std=0.3)).to(dt).cuda(), (1 + ref.rand(seed + 2, D, std=0.3)).to(dt).cuda()
    inv = (1e4 ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1))).cuda()
    pos = (far + torch.arange(B * T).view(B, T) * 3 % max(2 * T, 5)).cuda()
    return cfg, q, k, wq, wk, inv, pos



QK_SHAPES = [
    (1, 1, 1, 1, 64, 64, False, 0), (2, 1, 20, 4, 128, 128, False, 10), (16, 1, 3, 3, 8, 8, True, 5),
    (3, 37, 5, 1, 96, 96, False, 1000), (1, 130, 4, 2, 256, 128, True, 0), (2, 65, 2, 2, 128, 64, False, 2 ** 31 + 5),
    (1, 700, 6, 5, 72, 24, True, 10 ** 6), (1, 5, 2, 1, 128, 0, False, 0), (2, 1500, 1, 1, 64, 64, False, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", QK_SHAPES)
def test_qk_norm_rope_and_its_gradients(shape, dtype):
    B, T, Hq, Hk, D, R, inter, far = shape
    cfg, q, k, wq, wk, inv, pos = qk_case(B, T, Hq, Hk, D, R, dtype, inter, far)
    got = pkg.qk_norm_rope(cfg, q, k, wq, wk, inv, pos)
    x = ref.leaves(q, k, wq, wk)
    want = [ref.qk_one(x[j], x[j + 2], inv.cpu(), pos.cpu(), R, cfg.eps, inter) for j in range(2)]
    for y, z in zip(got, want):
        tol = STEP[dtype] * z.abs() + 1e-5 * z.norm(dim=-1, keepdim=True) / math.sqrt(D)
        assert bool(((y.double().cpu() - z).abs() <= tol).all())
    gy = [ref.rand(50 + j, *y.shape, dtype=DT[dtype]).cuda() for j, y in enumerate(got)]
    g = pkg.qk_norm_rope_backward(cfg, q, k, wq, wk, inv, pos, *gy)
    grads = torch.autograd.grad(sum((z * h.double().cpu()).sum() for z, h in zip(want, gy)), x)
    for name, w in zip(("q", "k", "wq", "wk"), grads):
        tol = 4e-6 if dtype == "f32" or name[0] == "w" else 2.0 ** -8
        assert ref.relative(g[name], w) <= tol, name
    assert status() == 0


def test_qk_in_place_strided_and_zero_rows():
    cfg, q, k, wq, wk, inv, pos = qk_case(2, 19, 4, 2, 128, 128, "bf16")
    q[0, 3] = 0  # a head of zeros stays zeros
    before_v = q.as_strided((2, 19, 2 * 128), (19 * 8 * 128, 8 * 128, 1), 6 * 128).clone()
    want = pkg.qk_norm_rope(cfg, q, k, wq, wk, inv, pos)
    out = pkg.qk_norm_rope(cfg, q, k, wq, wk, inv, pos, q_out=q, k_out=k)
    assert out[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert not want[0][0, 3].any()
    assert torch.equal(before_v, q.as_strided((2, 19, 2 * 128), (19 * 8 * 128, 8 * 128, 1), 6 * 128))
    gq = pkg.qk_norm_rope_backward(cfg, q, k, wq, wk, inv, pos, want[0], want[1])
    a, b = want[0].clone(), want[1].clone()
    g2 = pkg.qk_norm_rope_backward(cfg, q, k, wq, wk, inv, pos, a, b, gq=a, gk=b)
    assert all(torch.equal(gq[n], g2[n]) for n in gq) and g2["q"] is a
    # in the inputs' own places, one projection's views
    g3 = pkg.qk_norm_rope_backward(cfg, q, k, wq, wk, inv, pos, want[0], want[1], gq=q, gk=k)
    assert all(torch.equal(gq[n], g3[n]) for n in gq) and g3["q"] is q
    assert status() == 0


# ---------------------------------------------------------------- linear attention

def attn_case(B, T, H, Hkv, Dk, Dv, dtype, docs=(), state=False, decay=None, seed=3):
    cfg = pkg.LinearAttentionConfig(B=B, T=T, H=H, Hkv=Hkv, Dk=Dk, Dv=Dv, scale=Dk ** -0.5, dtype=dtype)
    dt = DT[dtype]
    q, k, v = (ref.rand(seed + n, B, T, h, w, dtype=dt).cuda() for n, (h, w) in enumerate(((H, Dk), (Hkv, Dk), (Hkv, Dv))))
    ld = torch.log1p(-torch.exp2(-2.0 - 6.0 * torch.arange(H) / H)) if decay is None else torch.tensor(decay).float()
    S0 = ref.rand(seed + 5, B, H, Dk, Dv, std=2.0).cuda() if state else None
    return cfg, q, k, v, ld.cuda(), S0, torch.tensor(docs, dtype=torch.int32)


# rows of one token up to several chunks and segments; documents that start at the first token,
# at chunk borders, twice in a row, at the last token
ATTN = [
    # B, T, H, Hkv, Dk, Dv, docs, state
    (1, 1, 1, 1, 64, 64, (), False), (2, 1, 2, 1, 128, 128, (0,), True), (1, 2, 1, 1, 64, 128, (1,), True),
    (1, 31, 2, 2, 128, 64, (), True), (2, 32, 1, 1, 64, 64, (5, 31, 32, 63), True), (1, 33, 2, 1, 128, 128, (32,), False),
    (1, 127, 1, 1, 128, 128, (126,), True), (1, 128, 2, 1, 128, 128, (), True), (2, 129, 2, 2, 64, 64, (128, 129), True),
    (1, 257, 3, 1, 128, 128, (0, 100, 101, 255, 256), True), (2, 600, 2, 2, 128, 128, (130, 700, 1199), True),
    (1, 1300, 2, 1, 64, 64, (), True), (1, 1300, 1, 1, 128, 128, (640, 641), False),
    (1, 300, 2, 2, 40, 56, (64, 65), True), (1, 290, 1, 1, 256, 136, (), True), (1, 70, 4, 2, 8, 8, (3,), True),
]


def check_attn(case, dtype, decay=None):
    B, T, H, Hkv, Dk, Dv, docs, state = case
    cfg, q, k, v, ld, S0, ds = attn_case(*case[:6], dtype, docs, state, decay)
    O, S = pkg.linear_attention(cfg, q, k, v, ld, ds, S0=S0, S_final=True)
    x = ref.leaves(q, k, v, S0)
    want, want_S = ref.linear_attention(x[0], x[1], x[2], ld.cpu(), cfg.scale, docs, x[3])
    if dtype == "f32":
        assert ref.relative(O, want) <= 1e-5
    else:
        terms, _ = ref.linear_attention(*(t.detach().abs() for t in x[:3]), ld.cpu(), cfg.scale, docs,
                                        None if S0 is None else x[3].detach().abs())
        tol = 2.0 ** -8 * (want.abs() + 2 * terms) + 1e-6
        assert bool(((O.double().cpu() - want).abs() <= tol).all())
        assert ref.relative(O, want) <= 6e-3
    assert ref.relative(S, want_S) <= 1e-5
    gO = ref.rand(20, *O.shape, dtype=DT[dtype]).cuda()
    gS = ref.rand(21, *S.shape).cuda() if state else None
    g = pkg.linear_attention_backward(cfg, q, k, v, ld, ds, gO, S0=S0, gS_final=gS)
    loss = (want * gO.double().cpu()).sum() + (0 if gS is None else (want_S * gS.double().cpu()).sum())
    names = ["q", "k", "v"] + (["S0"] if state else [])
    for name, w in zip(names, torch.autograd.grad(loss, [t for t in x if t is not None])):
        tol = 1e-5 if dtype == "f32" or name == "S0" else 6e-3
        assert ref.relative(g[name], w) <= tol, name
    assert status() == 0


@pytest.mark.parametrize("case", ATTN)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_attention_and_its_gradients(case, dtype):
    check_attn(case, dtype)


@pytest.mark.parametrize("decay", [[0.0, -1e-4], [-3.0, -40.0], [-math.inf, -0.5]])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_attention_decays(decay, dtype):
    # no decay; a past that fades within the chunk, and below the smallest number; no past at all
    check_attn((2, 300, 2, 1, 64, 64, (50, 450), True), dtype, decay)


def test_linear_attention_many_segments_and_long_rows():
    # few heads and a long row: the row is cut into segments whose states are joined; the state of one
    # call over the row is that of two calls over its halves
    for docs in ([], [1000, 5000, 5001, 7000]):
        cfg, q, k, v, ld, _, ds = attn_case(1, 8192, 2, 2, 128, 128, "bf16", docs, False, [-1e-3, -0.1])
        O, S = pkg.linear_attention(cfg, q, k, v, ld, ds, S_final=True)
        half = pkg.LinearAttentionConfig(1, 4096, 2, 2, 128, 128, cfg.scale)
        state, parts = None, []
        for lo in (0, 4096):
            d = [x - lo for x in docs if lo <= x < lo + 4096]
            o, state = pkg.linear_attention(half, *(x[:, lo:lo + 4096].contiguous() for x in (q, k, v)), ld, d, S0=state,
                                            S_final=True if state is None else state)
            parts.append(o)
        assert ref.relative(S, state.double().cpu()) <= 1e-5
        assert ref.relative(O, torch.cat(parts, 1).double().cpu()) <= 6e-3
        # and the last rows against the definition over the tail that they can see
        tail = 600
        x = [t[:, -tail:].double().cpu() for t in (q, k, v)]
        want, _ = ref.linear_attention(*x, ld.cpu(), cfg.scale, [d - (8192 - tail) for d in docs])
        far = O[:, -64:, 1].double().cpu()  # gamma = 0.9: what lies 500 tokens back is below 1e-22
        assert ref.relative(far, want[:, -64:, 1]) <= 6e-3
    assert status() == 0


@pytest.mark.parametrize("B,T,H,D", [(1, 32768, 20, 128), (1, 5100, 150, 64), (2, 9000, 30, 128)])
def test_linear_attention_long_items(B, T, H, D):
    # many chunks to a work item, cut rows and whole ones: the tensor-core pass against the fp32 pass (held
    # to the definition above) on the same values
    docs = sorted(set(torch.randint(0, B * T, (15,), generator=torch.Generator().manual_seed(4)).tolist()))
    cfg, q, k, v, _, S0, ds = attn_case(B, T, H, H, D, D, "bf16", docs, True)
    ld = torch.log1p(-torch.exp2(-4.0 - 7.0 * torch.arange(H) / H)).cuda()
    f32 = pkg.LinearAttentionConfig(B, T, H, H, D, D, cfg.scale, "f32")
    gO = ref.rand(20, B, T, H, D, dtype=torch.bfloat16).cuda()
    O, S = pkg.linear_attention(cfg, q, k, v, ld, ds, S0=S0, S_final=True)
    want, want_S = pkg.linear_attention(f32, q.float(), k.float(), v.float(), ld, ds, S0=S0, S_final=True)
    assert ref.relative(O, want.cpu()) <= 6e-3 and ref.relative(S, want_S.cpu()) <= 1e-5
    g = pkg.linear_attention_backward(cfg, q, k, v, ld, ds, gO, S0=S0, gS_final=S0)
    w = pkg.linear_attention_backward(f32, q.float(), k.float(), v.float(), ld, ds, gO.float(), S0=S0, gS_final=S0)
    for n in g:
        assert ref.relative(g[n], w[n].cpu()) <= (1e-5 if n == "S0" else 6e-3), n
    assert status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 64, 64), (3, 4, 2, 128, 128), (2, 3, 3, 40, 56), (20, 16, 4, 128, 128),
                                   (2, 2, 1, 256, 136)])
def test_linear_attention_step_by_step_is_the_prompt(shape, dtype):
    B, H, Hkv, Dk, Dv = shape
    T = 6
    cfg, q, k, v, ld, S0, ds = attn_case(B, T, H, Hkv, Dk, Dv, dtype, (2, 4), True)
    x = ref.leaves(q, k, v, S0)
    want, want_S = ref.linear_attention(x[0], x[1], x[2], ld.cpu(), cfg.scale, (2, 4), x[3])
    S = S0.clone()
    for t in range(T):
        starts = torch.zeros(B, dtype=torch.int32, device="cuda")
        if t in (2, 4):
            starts[0] = 1
        o = pkg.linear_attention_step(cfg, S, q[:, t], k[:, t], v[:, t], ld, starts)
        # a fp32 sum of Dk products in any order is off by at most Dk 2^-24 sum |terms| (u = 2^-24 a product
        # and an addition, Dk of them in a chain at most), S itself by 3 u a token more; then the one
        # rounding of o.  (Of the result alone no bound holds: after a start o = scale (q . k) v, and q . k
        # may be far smaller than its terms: 0.03 out of 64 terms of size 1 at t = 2 of the first shape.)
        y = [z[:, :t + 1].detach().abs() for z in x[:3]]
        terms, _ = ref.linear_attention(*y, ld.cpu(), cfg.scale, [b * (t + 1) + u for b in (0,) for u in (2, 4) if u <= t],
                                        x[3].detach().abs())
        tol = STEP[dtype] * want[:, t].abs() + (Dk + 3 * T) * 2.0 ** -24 * terms[:, t]
        assert bool(((o.double().cpu() - want[:, t]).abs() <= tol).all())
    assert ref.relative(S, want_S) <= 1e-6
    assert status() == 0


def test_linear_attention_views_streams_and_state_in_place():
    B, T, H, Hkv, D = 2, 450, 4, 2, 128
    cfg, q, k, v, ld, S0, _ = attn_case(B, T, H, Hkv, D, D, "bf16", (), True)
    want, want_S = pkg.linear_attention(cfg, q, k, v, ld, S0=S0, S_final=True)
    qkv = torch.cat((q.flatten(2), k.flatten(2), v.flatten(2)), -1)
    views = [t.unflatten(-1, (-1, D)) for t in qkv.split([H * D, Hkv * D, Hkv * D], -1)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    S = S0.clone()
    side.wait_stream(torch.cuda.current_stream())
    O, S2 = pkg.linear_attention(cfg, *views, ld, S0=S, S_final=S, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert S2 is S and torch.equal(S, want_S) and torch.equal(O, want)
    g = pkg.linear_attention_backward(cfg, q, k, v, ld, None, want, S0=S0)
    h = pkg.linear_attention_backward(cfg, *views, ld, None, want, S0=S0)
    assert all(torch.equal(g[n], h[n]) for n in g)
    assert status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,H,D", [(1, 3000, 2, 64), (1, 700, 4, 128), (2, 40, 1, 64), (1, 1100, 150, 64)])
def test_linear_attention_state_in_place(B, T, H, D, dtype):
    # one segment, few and many, whole rows beside cut ones: S_final in S0's place is S_final elsewhere
    cfg, q, k, v, ld, S0, ds = attn_case(B, T, H, H, D, D, dtype, (T // 2,), True)
    for docs in (None, ds):
        want, want_S = pkg.linear_attention(cfg, q, k, v, ld, docs, S0=S0, S_final=True)
        S = S0.clone()
        O, _ = pkg.linear_attention(cfg, q, k, v, ld, docs, S0=S, S_final=S)
        assert torch.equal(O, want) and torch.equal(S, want_S)
    assert status() == 0


def test_linear_attention_bad_starts_and_decays_are_reported():
    cfg, q, k, v, ld, _, _ = attn_case(1, 40, 1, 1, 64, 64, "bf16")
    for bad in ([40], [-1], [5, 5], [9, 3]):
        pkg.linear_attention(cfg, q, k, v, ld, bad)
        assert status() == 1
    for x in (0.1, math.nan):
        pkg.linear_attention(cfg, q, k, v, torch.full_like(ld, x))
        assert status() == 1
    assert status() == 0


# ---------------------------------------------------------------- cross entropy

def xent_case(N, V, d, dtype, seed=11, std=2.0, piece=0):
    cfg = pkg.CrossEntropyConfig(N=N, V=V, d=d, dtype=dtype, piece=piece)
    H = ref.rand(seed, N, d, dtype=DT[dtype]).cuda()
    W = ref.rand(seed + 1, V, d, std=std * d ** -0.5, dtype=DT[dtype]).cuda()
    t = torch.randint(0, V, (N,), generator=torch.Generator().manual_seed(seed))
    t[N // 2::3] = -100
    t[0] = V - 1
    return cfg, H, W, t.cuda()


XENT = [(1, 1, 32, 0), (1, 300, 64, 0), (5, 257, 96, 256), (129, 1000, 128, 256), (300, 2049, 160, 512),
        (256, 512, 64, 0), (77, 40007, 32, 0), (600, 700, 320, 256)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,d,piece", XENT)
def test_cross_entropy_and_its_gradients(N, V, d, piece, dtype):
    cfg, H, W, t = xent_case(N, V, d, dtype, piece=piece)
    loss, lse = pkg.cross_entropy(cfg, H, W, t)
    h, w = ref.leaves(H, W)
    want, want_lse = ref.cross_entropy(h, w, t.cpu())
    assert float((loss.double().cpu() - want).abs().max()) <= 1e-5 * max(1.0, float(want.abs().max()))
    assert float((lse.double().cpu() - want_lse).abs().max()) <= 1e-5 * max(1.0, float(want_lse.abs().max()))
    assert not loss[t == -100].any()
    gl = ref.rand(5, N).cuda()
    g = pkg.cross_entropy_backward(cfg, H, W, t, lse, gl)
    for name, x in zip(("H", "W"), torch.autograd.grad((want * gl.double().cpu()).sum(), (h, w))):
        # one vocabulary word: p - 1 = 0 up to the rounding of lse
        if V == 1:
            assert float(g[name].abs().max()) <= 1e-5
        else:
            assert ref.relative(g[name], x) <= (1e-5 if dtype == "f32" else 5.6e-3), name
    assert not g["H"][t == -100].any()
    assert status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cross_entropy_far_logits_and_empty_batches(dtype):
    # logits of some +-2000: exp of any of them alone would overflow or vanish
    cfg, H, W, t = xent_case(70, 900, 64, dtype, std=700.0)
    loss, lse = pkg.cross_entropy(cfg, H, W, t)
    want, want_lse = ref.cross_entropy(H.double().cpu(), W.double().cpu(), t.cpu())
    assert float((lse.double().cpu() - want_lse).abs().max()) <= 1e-5 * float(want_lse.abs().max())
    assert float((loss.double().cpu() - want).abs().max()) <= 1e-5 * float(want_lse.abs().max())
    none = torch.full_like(t, -100)
    loss, lse = pkg.cross_entropy(cfg, H, W, none)
    assert not loss.any()
    g = pkg.cross_entropy_backward(cfg, H, W, none, lse, torch.ones_like(lse))
    assert not g["H"].any() and not g["W"].any()
    assert status() == 0
    for bad in (900, -1, 2 ** 40):  # reported, and the row left out
        b = t.clone()
        b[2] = bad
        loss, lse = pkg.cross_entropy(cfg, H, W, b)
        assert status() == 1 and float(loss[2]) == 0.0
        g = pkg.cross_entropy_backward(cfg, H, W, b, lse, torch.ones_like(lse))
        assert status() == 1 and not g["H"][2].any()
    pad = pkg.CrossEntropyConfig(N=70, V=900, d=64, dtype=dtype, ignore_index=7)
    t[t < 0] = 7
    assert not pkg.cross_entropy(pad, H, W, t)[0][t == 7].any() and status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,d,piece", [(3, 300, 64, 256), (300, 1000, 128, 512)])
def test_cross_entropy_rows_left_out_reach_nothing(N, V, d, piece, dtype):
    cfg, H, W, t = xent_case(N, V, d, dtype, piece=piece)
    gl = ref.rand(5, N).cuda()
    loss, lse = pkg.cross_entropy(cfg, H, W, t)
    want = pkg.cross_entropy_backward(cfg, H, W, t, lse, gl)
    out = t == -100
    assert bool(out.any())
    for bad in (math.nan, math.inf):
        h, g = H.clone(), gl.clone()
        h[out], g[out] = bad, bad
        loss2, lse2 = pkg.cross_entropy(cfg, h, W, t)
        assert torch.equal(loss2, loss) and torch.equal(lse2[~out], lse[~out])
        got = pkg.cross_entropy_backward(cfg, h, W, t, lse2, g)
        assert torch.equal(got["H"], want["H"]) and torch.equal(got["W"], want["W"])
    assert status() == 0


def test_offsets_beyond_32_bits():
    # tokens so far apart that the last ones lie more than 2^31 elements on: the packed call's values
    T, wide = 110000, 20480
    for H, D, dtype in ((2, 64, "bf16"), (2, 40, "bf16")):
        cfg, q, k, v, ld, S0, ds = attn_case(1, T, H, H, D, D, dtype, (70001,), True)
        far = torch.empty(1, T, wide, dtype=torch.bfloat16, device="cuda")
        views = []
        for i, x in enumerate((q, k, v, torch.empty_like(q))):
            y = far[..., wide - (i + 1) * H * D: wide - i * H * D].unflatten(-1, (H, D))
            y.copy_(x)
            views.append(y)
        O, S = pkg.linear_attention(cfg, q, k, v, ld, ds, S0=S0, S_final=True)
        O2, S2 = pkg.linear_attention(cfg, *views[:3], ld, ds, S0=S0, O=views[3], S_final=True)
        assert torch.equal(O, O2) and torch.equal(S, S2)
        g = pkg.linear_attention_backward(cfg, q, k, v, ld, ds, O, S0=S0)
        h = pkg.linear_attention_backward(cfg, *views[:3], ld, ds, views[3], S0=S0)
        assert all(torch.equal(g[n], h[n]) for n in g)
        qc = pkg.QKNormRopeConfig(1, T, H, H, D, D)
        w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
        inv = torch.logspace(0, -4, D // 2, dtype=torch.float64).cuda()
        pos = torch.arange(T, device="cuda")[None]
        a = pkg.qk_norm_rope(qc, q, k, w, w, inv, pos)
        ga = pkg.qk_norm_rope_backward(qc, q, k, w, w, inv, pos, k, v)
        gb = pkg.qk_norm_rope_backward(qc, *views[:2], w, w, inv, pos, *views[1:3])
        assert all(torch.equal(ga[n], gb[n]) for n in ga)
        b = pkg.qk_norm_rope(qc, *views[:2], w, w, inv, pos, q_out=views[0], k_out=views[1])
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert status() == 0


def test_cross_entropy_head_beyond_32_bits():
    N, V, d = 16, 850000, 2560  # 2.2e9 weights
    gen = torch.Generator("cuda").manual_seed(3)
    W = torch.empty(V, d, dtype=torch.bfloat16, device="cuda").normal_(0, d ** -0.5, generator=gen)
    H = torch.empty(N, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    t = torch.randint(V - 2000, V, (N,), generator=torch.Generator().manual_seed(1)).cuda()
    cfg = pkg.CrossEntropyConfig(N, V, d)
    loss, lse = pkg.cross_entropy(cfg, H, W, t)
    logits = torch.cat([H.double() @ W[i:i + 50000].double().T for i in range(0, V, 50000)], 1)
    want_lse = logits.logsumexp(1)
    want = want_lse - logits.gather(1, t[:, None])[:, 0]
    assert float((lse - want_lse).abs().max()) <= 1e-5 * float(want_lse.abs().max())
    assert float((loss - want).abs().max()) <= 1e-5 * float(want.abs().max())
    g = pkg.cross_entropy_backward(cfg, H, W, t, lse, torch.full((N,), 1 / N, device="cuda"))
    p = (logits - want_lse[:, None]).exp()
    p[torch.arange(N), t] -= 1
    p /= N
    gH = sum(p[:, i:i + 50000] @ W[i:i + 50000].double() for i in range(0, V, 50000))
    assert ref.relative(g["H"], gH.cpu()) <= 5.6e-3
    for lo in (0, V // 2, V - 2000):
        assert ref.relative(g["W"][lo:lo + 2000], (p[:, lo:lo + 2000].T @ H.double()).cpu()) <= 5.6e-3
    assert status() == 0

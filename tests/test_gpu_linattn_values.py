"""Values that are not finite in the linear attention: they reach what the definition makes
depend on them, and nothing else, whatever the order and grouping of the sums.

A place that depends on such a value is compared by kind only: it is not finite (a sum in
another order may give an infinity where the definition gives NaN).  Every other place is held to
the tolerances of test_gpu_block_ops.py."""
import math

import pytest
import torch

import chunk_wise_weight_gate_b200 as pkg
from tests import block_ref as ref
from tests.test_gpu_block_ops import attn_case, status

pytestmark = pytest.mark.gpu


def same_but_for_bad(got, want, tol, name=""):
    """Not finite in the same places; elsewhere the error's 2-norm is at most tol of the finite part's."""
    got, want = got.detach().double().cpu(), want.detach().double().cpu()
    bad = ~want.isfinite()
    assert torch.equal(~got.isfinite(), bad), (name, int((got.isfinite() == bad).sum()))
    assert ref.relative(got.masked_fill(bad, 0), want.masked_fill(bad, 0)) <= tol, name


ATTN = [
    # B, T, H, Hkv, Dk, Dv, docs, state; tokens that turn bad in turn
    (1, 300, 2, 1, 64, 64, (100, 200, 201), True, (0, 50, 99, 150, 200, 299)),
    (2, 200, 2, 2, 128, 128, (60, 130), False, (30, 129, 199)),
    (1, 1300, 1, 1, 64, 128, (640, 1200), True, (100, 639, 1290)),
    (1, 700, 1, 1, 128, 64, (), True, (0, 511, 699)),
    (1, 90, 2, 1, 40, 56, (31, 32, 64), True, (5, 31, 63, 89)),
]


def attn_bad(case, dtype, bad, which, token, decay=None):
    B, T, H, Hkv, Dk, Dv, docs, state, _ = case
    cfg, q, k, v, ld, S0, ds = attn_case(B, T, H, Hkv, Dk, Dv, dtype, docs, state, decay)
    gO = ref.rand(20, B, T, H, Dv, dtype=q.dtype).cuda()
    gS = ref.rand(21, B, H, Dk, Dv).cuda() if state else None
    x = {"q": q, "k": k, "v": v, "gO": gO}[which]
    x[0, token, 0, 3] = bad
    return cfg, q, k, v, ld, S0, ds, gO, gS, docs


def attn_ref(cfg, q, k, v, ld, S0, gO, gS, docs):
    x = ref.leaves(q, k, v, S0)
    want, want_S = ref.linear_attention(x[0], x[1], x[2], ld.cpu(), cfg.scale, docs, x[3])
    loss = (want * gO.double().cpu()).sum() + (0 if gS is None else (want_S * gS.double().cpu()).sum())
    names = ["q", "k", "v"] + ([] if S0 is None else ["S0"])
    return want, want_S, dict(zip(names, torch.autograd.grad(loss, [t for t in x if t is not None])))


@pytest.mark.parametrize("case", ATTN)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("which,bad", [("v", math.nan), ("v", math.inf), ("k", -math.inf), ("q", math.nan), ("gO", math.nan)])
def test_linear_attention_bad_values_stay_with_what_depends_on_them(case, dtype, which, bad):
    for token in case[-1]:
        cfg, q, k, v, ld, S0, ds, gO, gS, docs = attn_bad(case, dtype, bad, which, token)
        want, want_S, grads = attn_ref(cfg, q, k, v, ld, S0, gO, gS, docs)
        tol = 1e-5 if dtype == "f32" else 6e-3
        for in_place in (False, True) if S0 is not None else (False,):
            S = S0.clone() if in_place else S0
            O, Sf = pkg.linear_attention(cfg, q, k, v, ld, ds, S0=S, S_final=S if in_place else True)
            same_but_for_bad(O, want, tol, (token, "O"))
            same_but_for_bad(Sf, want_S, 1e-5, (token, "S"))
        g = pkg.linear_attention_backward(cfg, q, k, v, ld, ds, gO, S0=S0, gS_final=gS)
        for n, w in grads.items():
            same_but_for_bad(g[n], w, 1e-5 if n == "S0" else tol, (token, n))
    assert status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", [[-math.inf, -200.0], [-1.0, -30.0]])
def test_linear_attention_bad_values_under_strong_decays(dtype, decay):
    # no past at all (gamma = 0): the bad token's own outputs alone; a decay that underflows within a chunk
    # still carries an infinity on
    case = (1, 500, 2, 1, 64, 64, (400,), True, None)
    for which, bad, token in (("v", math.inf, 10), ("k", math.nan, 200), ("v", math.nan, 399), ("v", math.inf, 499)):
        cfg, q, k, v, ld, S0, ds, gO, gS, docs = attn_bad(case, dtype, bad, which, token, decay)
        tol = 1e-5 if dtype == "f32" else 6e-3
        O, S = pkg.linear_attention(cfg, q, k, v, ld, ds, S0=S0, S_final=True)
        x = ref.leaves(q, k, v, S0)
        want, want_S = definition(*x, ld, cfg.scale, docs)
        same_but_for_bad(O, want, tol, (token, "O"))
        same_but_for_bad(S, want_S, 1e-5, (token, "S"))
        g = pkg.linear_attention_backward(cfg, q, k, v, ld, ds, gO, S0=S0, gS_final=gS)
        loss = (want * gO.double().cpu()).sum() + (want_S * gS.double().cpu()).sum()
        for n, w in zip(("q", "k", "v", "S0"), torch.autograd.grad(loss, x)):
            same_but_for_bad(g[n], w, 1e-5 if n == "S0" else tol, (token, n))
    assert status() == 0


def definition(q, k, v, S, ld, scale, docs):
    """The recurrence for one row, with no past at all where gamma is 0 (below the smallest fp32)."""
    gamma = torch.exp(ld.cpu().float()).double().view(1, -1, 1, 1)
    k, v = (x.repeat_interleave(q.shape[2] // x.shape[2], 2) for x in (k, v))
    out = []
    for t in range(q.shape[1]):
        old = torch.where(gamma == 0, 0.0, gamma * S)
        S = (torch.zeros_like(S) if t in docs else old) + k[:, t, :, :, None] * v[:, t, :, None, :]
        out.append(scale * torch.einsum("bhk,bhkv->bhv", q[:, t], S))
    return torch.stack(out, 1), S


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_attention_bad_initial_states(dtype):
    # a state that is not finite ends where a document starts, and where there is no past
    for B, T, H, D, docs, decay in ((2, 300, 2, 64, (40,), [-0.1, -0.01]), (1, 1500, 1, 128, (1400,), [-0.5]),
                                    (1, 300, 2, 64, (), [-math.inf, -3.0])):
        cfg, q, k, v, ld, S0, ds = attn_case(B, T, H, H, D, D, dtype, docs, True, decay)
        S0[0, 0, 2, 5] = math.inf
        S0[0, 0, 4, 6] = math.nan
        want, want_S = [], []
        for b in range(B):
            o, s = definition(*(x[b:b + 1].double().cpu() for x in (q, k, v, S0)), ld, cfg.scale,
                              [d - b * T for d in docs if b * T <= d < b * T + T])
            want.append(o)
            want_S.append(s)
        O, S = pkg.linear_attention(cfg, q, k, v, ld, ds, S0=S0, S_final=True)
        same_but_for_bad(O, torch.cat(want), 1e-5 if dtype == "f32" else 6e-3)
        same_but_for_bad(S, torch.cat(want_S), 1e-5)
    assert status() == 0


@pytest.mark.parametrize("B,T,H,Dk,Dv", [(1, 9000, 2, 128, 128), (1, 6000, 2, 64, 128), (1, 3000, 8, 128, 64), (1, 700, 150, 64, 64)])
def test_linear_attention_bad_values_in_long_rows(B, T, H, Dk, Dv):
    # segments joined directly and by their prefix, whole rows beside cut ones: against the fp32 pass (held to
    # the definition above)
    docs = [T // 3, T // 2 + 1, T - 100]
    cfg, q, k, v, _, S0, ds = attn_case(B, T, H, H, Dk, Dv, "bf16", docs, True)
    ld = torch.log1p(-torch.exp2(-4.0 - 5.0 * torch.arange(H) / H)).cuda()
    gO = ref.rand(20, B, T, H, Dv, dtype=torch.bfloat16).cuda()
    f32 = pkg.LinearAttentionConfig(B, T, H, H, Dk, Dv, cfg.scale, "f32")
    v[0, T // 3 - 2, 0, 7] = math.nan     # the first document's last tokens
    k[0, T // 2 + 5, 1, 9] = math.inf     # the third document's first ones
    gO[0, T - 1, H - 1, 1] = -math.inf
    for S in (True, S0.clone()):
        O, Sf = pkg.linear_attention(cfg, q, k, v, ld, ds, S0=S0 if S is True else S, S_final=S)
        want, want_S = pkg.linear_attention(f32, q.float(), k.float(), v.float(), ld, ds, S0=S0, S_final=True)
        same_but_for_bad(O, want, 6e-3)
        same_but_for_bad(Sf, want_S, 1e-5)
    g = pkg.linear_attention_backward(cfg, q, k, v, ld, ds, gO, S0=S0, gS_final=S0)
    w = pkg.linear_attention_backward(f32, q.float(), k.float(), v.float(), ld, ds, gO.float(), S0=S0, gS_final=S0)
    for n in g:
        same_but_for_bad(g[n], w[n], 1e-5 if n == "S0" else 6e-3, n)
    assert status() == 0


def test_linear_attention_large_finite_values():
    # products of masked pairs beyond fp32's range: what sees none of them is as ever
    cfg, q, k, v, ld, S0, ds = attn_case(1, 300, 1, 1, 128, 128, "bf16", (150,), False)
    q[0, 20], k[0, 140] = 1e25, 1e25   # token 140 is later than 20, and in a document before 150
    want, want_S = ref.linear_attention(*(x.double().cpu() for x in (q, k, v)), ld.cpu(), cfg.scale, (150,))
    O, S = pkg.linear_attention(cfg, q, k, v, ld, ds, S_final=True)
    quiet = [t for t in range(300) if t != 20 and not 140 <= t < 150]
    assert bool(O.isfinite().all())
    assert ref.relative(O[:, quiet], want[:, quiet]) <= 6e-3 and ref.relative(S, want_S) <= 1e-5
    assert status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", [-math.inf, -200.0])
def test_linear_attention_step_without_a_past(dtype, decay):
    # gamma = 0: the state before is not read into the result, whatever it holds; as in the prompt
    cfg, q, k, v, ld, S0, _ = attn_case(3, 1, 2, 2, 64, 64, dtype, (), True, [decay, -0.5])
    S0[1, 0, 3], S0[2, 0] = math.inf, math.nan
    S = S0.clone()
    o = pkg.linear_attention_step(cfg, S, q[:, 0], k[:, 0], v[:, 0], ld)
    want = torch.einsum("bk,bv->bkv", k[:, 0, 0].double(), v[:, 0, 0].double())
    assert ref.relative(S[:, 0], want.cpu()) <= 1e-6
    O, S2 = pkg.linear_attention(cfg, q, k, v, ld, S0=S0, S_final=True)
    # products of bf16 are exact in fp32; in bf16 the prompt's state goes through two halves (2^-17)
    assert ref.relative(S2, S.double().cpu()) <= 1e-5
    # o = scale (q . k) v: fp32 sums of 64 terms either way, and the prompt's P rounded to bf16
    terms = torch.einsum("bhk,bhk->bh", q[:, 0].abs().double(), k[:, 0].abs().double())[..., None] * v[:, 0].abs().double()
    tol = (2.0 ** -7 if dtype == "bf16" else 2.0 ** -16) * cfg.scale * terms
    assert bool(((o.double() - O[:, 0].double()).abs() <= tol)[:, 0].all())
    assert status() == 0


def test_linear_attention_bad_values_in_some_of_many_short_rows():
    # some forty items a block, of which a few hold a bad value; state in place, captured and replayed
    B, T, H, D = 300, 3, 20, 64
    cfg, q, k, v, _, S0, _ = attn_case(B, T, H, H, D, D, "bf16", (), True)
    ld = torch.log1p(-torch.exp2(-1.0 - 5.0 * torch.arange(H) / H)).cuda()
    docs = torch.arange(2, B * T, 7, dtype=torch.int32).cuda()
    gen = torch.Generator().manual_seed(8)
    for x in (k, v):
        rows, toks, heads = (torch.randint(0, n, (60,), generator=gen).cuda() for n in (B, T, H))
        x[rows, toks, heads, 5] = math.nan
    S0[7, 3, 2, 1] = math.inf
    f32 = pkg.LinearAttentionConfig(B, T, H, H, D, D, cfg.scale, "f32")
    want, want_S = pkg.linear_attention(f32, q.float(), k.float(), v.float(), ld, docs, S0=S0, S_final=True)
    assert not bool(want.isfinite().all()) and bool(want.isfinite().any())
    O, S = pkg.linear_attention(cfg, q, k, v, ld, docs, S0=S0, S_final=True)
    same_but_for_bad(O, want, 6e-3)
    same_but_for_bad(S, want_S, 1e-5)
    S2 = S0.clone()
    O2, _ = pkg.linear_attention(cfg, q, k, v, ld, docs, S0=S2, S_final=S2)
    assert torch.equal(O.nan_to_num(7.0), O2.nan_to_num(7.0)) and torch.equal(S.nan_to_num(7.0), S2.nan_to_num(7.0))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O3, _ = pkg.linear_attention(cfg, q, k, v, ld, docs, S0=S2, S_final=S2)
    for _ in range(2):
        S2.copy_(S0)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(O.nan_to_num(7.0), O3.nan_to_num(7.0)) and torch.equal(S.nan_to_num(7.0), S2.nan_to_num(7.0))
    assert status() == 0
    del graph

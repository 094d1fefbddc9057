"""The operators around the TTT layer, as a user's program runs them: norms of queries
and keys with the position rotation, linear attention with a decay for each head, and
the softmax cross entropy over a large vocabulary.

A case names an operator and its sizes.  `run` takes one pass through it: in plain torch
operations (`own` false) or through the package's entry points (`own` true).  `exact`
gives the same outputs from the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of 16 sequences that decode together: latency counts
        {"name": "qk_step", "op": "qk_fwd", "B": 16, "T": 1, "Hq": 20, "Hk": 20, "D": 128, "R": 128,
         "interleaved": False, "far": 100000, "dtype": "bf16"},
        # a 32k-token prompt with four query heads to a key head, out of one fused projection
        {"name": "qk_prompt", "op": "qk_fwd", "B": 1, "T": 32768, "Hq": 32, "Hk": 8, "D": 128, "R": 128,
         "interleaved": False, "far": 1000000, "dtype": "bf16"},
        # a training batch of odd length, half of each head rotated, pairs side by side
        {"name": "qk_train", "op": "qk_bwd", "B": 3, "T": 4099, "Hq": 20, "Hk": 4, "D": 128, "R": 64,
         "interleaved": True, "far": 4099, "dtype": "bf16"},
        # a small model trained in fp32, head width no power of two
        {"name": "qk_train_f32", "op": "qk_bwd", "B": 2, "T": 1000, "Hq": 12, "Hk": 12, "D": 96, "R": 96,
         "interleaved": False, "far": 1000, "dtype": "f32"},
        # one token of 32 sequences against their states
        {"name": "attn_step", "op": "attn_step", "B": 32, "T": 1, "H": 20, "Hkv": 20, "Dk": 128, "Dv": 128,
         "docs": 0, "state": True, "dtype": "bf16"},
        # one long prompt of packed documents (lengths of 256 to 4096 tokens)
        {"name": "attn_prompt", "op": "attn_fwd", "B": 1, "T": 32768, "H": 20, "Hkv": 20, "Dk": 128, "Dv": 128,
         "docs": 15, "state": False, "dtype": "bf16"},
        # the next piece of eight long sequences: the state comes in and goes out; odd length, shared key heads
        {"name": "attn_piece", "op": "attn_fwd", "B": 8, "T": 2047, "H": 24, "Hkv": 8, "Dk": 128, "Dv": 128,
         "docs": 0, "state": True, "dtype": "bf16"},
        # a training batch: gradients of queries, keys and values
        {"name": "attn_train", "op": "attn_bwd", "B": 2, "T": 8192, "H": 20, "Hkv": 20, "Dk": 128, "Dv": 128,
         "docs": 8, "state": False, "dtype": "bf16"},
        # a small model in fp32, gradients of everything, head widths that differ
        {"name": "attn_train_f32", "op": "attn_bwd", "B": 2, "T": 777, "H": 6, "Hkv": 3, "Dk": 64, "Dv": 96,
         "docs": 3, "state": True, "dtype": "f32"},
        # the loss of a held-out batch, vocabulary of odd size
        {"name": "loss_eval", "op": "loss_fwd", "N": 2000, "V": 50001, "d": 2560, "dtype": "bf16"},
        # a training step's loss with its gradients
        {"name": "loss_train", "op": "loss_grad", "N": 8192, "V": 65536, "d": 2560, "dtype": "bf16"},
        # the same for a small model in fp32
        {"name": "loss_train_f32", "op": "loss_grad", "N": 300, "V": 10007, "d": 512, "dtype": "f32"},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk_fwd", "qk_bwd", "attn_step", "attn_fwd", "attn_bwd", "loss_fwd", "loss_grad"])
    f32 = rng.random() < 0.2
    dtype = "f32" if f32 else "bf16"
    if op.startswith("qk"):
        D = rng.choice([64, 96, 128, 128, 256])
        Hk = rng.choice([1, 2, 4, 8, 20])
        Hq = Hk * rng.choice([1, 1, 2, 4])
        tokens = _spread(rng, 1, min(65536 if op == "qk_fwd" else 16384, (1 << 28) // ((Hq + Hk) * D)))
        B = min(tokens, rng.choice([1, 2, 3, 8, 16]))
        return {"op": op, "B": B, "T": max(1, tokens // B), "Hq": Hq, "Hk": Hk, "D": D,
                "R": rng.choice([D, D, D // 2]), "interleaved": rng.random() < 0.3, "far": _spread(rng, 100, 1000000),
                "dtype": dtype}
    if op.startswith("attn"):
        G = rng.choice([1, 1, 1, 2, 4])
        Hkv = rng.choice([1, 2, 5, 8, 16, 20])
        H = Hkv * G
        if f32:
            Dk, Dv = rng.choice([(32, 32), (64, 64), (64, 96), (128, 128), (40, 56)])
            most = 16384
        else:
            Dk, Dv = rng.choice([(64, 64), (128, 128), (128, 128), (64, 128), (128, 64)])
            most = 655360 if op == "attn_fwd" else 327680
        if op == "attn_step":
            B, T = _spread(rng, 1, 64), 1
        else:
            tokens = _spread(rng, 1, max(2, min(32768, most // H)))
            B = min(tokens, rng.choice([1, 1, 2, 4, 8]))
            T = max(1, tokens // B)
        return {"op": op, "B": B, "T": T, "H": H, "Hkv": Hkv, "Dk": Dk, "Dv": Dv,
                "docs": 0 if T < 8 else rng.choice([0, 0, 1, 5, 20]), "state": op == "attn_step" or rng.random() < 0.5,
                "dtype": dtype}
    d = rng.choice([256, 512, 1024, 2560])
    if f32:
        N, V = _spread(rng, 1, 512), _spread(rng, 1000, 20000)
    else:
        V = _spread(rng, 2000, 131072)
        N = _spread(rng, 1, min(8192, 8192 * 65536 * 2560 // (V * d)))
    return {"op": op, "N": N, "V": V, "d": d, "dtype": dtype}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def prepare(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    s = dict(case)
    if case["op"].startswith("qk"):
        B, T, Hq, Hk, D, R = (case[k] for k in ("B", "T", "Hq", "Hk", "D", "R"))
        # queries and keys are views of one projection's output, as a model has them
        qkv = _randn(g, B, T, (Hq + 2 * Hk) * D, dtype=dt, std=1.5)
        s["q"] = qkv[..., :Hq * D].unflatten(-1, (Hq, D))
        s["k"] = qkv[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D))
        s["wq"] = (1 + _randn(g, D, std=0.2)).to(dt)
        s["wk"] = (1 + _randn(g, D, std=0.2)).to(dt)
        s["inv_freq"] = 1e6 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
        first = torch.randint(0, max(1, case["far"] - T + 1), (B, 1), generator=g, device="cuda")
        s["positions"] = first + torch.arange(T, device="cuda")
        if case["op"] == "qk_bwd":
            s["gq"] = _randn(g, B, T, Hq, D, dtype=dt)
            s["gk"] = _randn(g, B, T, Hk, D, dtype=dt)
    elif case["op"].startswith("attn"):
        B, T, H, Hkv, Dk, Dv = (case[k] for k in ("B", "T", "H", "Hkv", "Dk", "Dv"))
        if case["op"] == "attn_step":
            s["q"], s["k"], s["v"] = (_randn(g, B, n, w, dtype=dt) for n, w in ((H, Dk), (Hkv, Dk), (Hkv, Dv)))
        else:
            s["q"], s["k"], s["v"] = (_randn(g, B, T, n, w, dtype=dt) for n, w in ((H, Dk), (Hkv, Dk), (Hkv, Dv)))
        # heads that forget after some 30 tokens up to heads that remember for thousands
        s["log_decay"] = torch.log1p(-torch.exp2(-5 - 7 * torch.arange(H, device="cuda", dtype=torch.float64) / H)).float()
        s["scale"] = Dk ** -0.5
        s["S0"] = _randn(g, B, H, Dk, Dv, std=4.0) if case["state"] else None
        starts = torch.randint(0, B * T, (case["docs"],), generator=g, device="cuda")
        s["doc_starts"] = torch.unique(starts).to(torch.int32) if case["docs"] else None
        if case["op"] == "attn_bwd":
            s["gO"] = _randn(g, B, T, H, Dv, dtype=dt)
            s["gS"] = _randn(g, B, H, Dk, Dv, std=0.5) if case["state"] else None
    else:
        N, V, d = case["N"], case["V"], case["d"]
        s["H"] = _randn(g, N, d, dtype=dt)
        s["W"] = _randn(g, V, d, dtype=dt, std=2.0 * d ** -0.5)
        t = torch.randint(0, V, (N,), generator=g, device="cuda")
        # one token in ten takes no part (prompt or padding); the first always does
        drop = torch.rand(N, generator=g, device="cuda") < 0.1
        drop[0] = False
        s["targets"] = torch.where(drop, -100, t)
        s["gloss"] = torch.full((N,), 1.0, device="cuda") / (~drop).sum()
    return s


# ------------------------------------------------------------------ plain forms

def _angles(s):
    th = s["positions"].double()[..., None] * s["inv_freq"]          # [B, T, R/2], in 64 bits: positions are far
    return torch.cos(th).float()[:, :, None], torch.sin(th).float()[:, :, None]


def _pairs(x, s):
    """The two halves of every rotated pair, and what is not rotated."""
    R = s["R"]
    if s["interleaved"]:
        return x[..., 0:R:2], x[..., 1:R:2], x[..., R:]
    return x[..., :R // 2], x[..., R // 2:R], x[..., R:]


def _joined(a, b, rest, s):
    ab = torch.stack((a, b), -1).flatten(-2) if s["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((ab, rest), -1)


def _plain_qk(s):
    c, n = _angles(s)

    def one(x, w):
        x = x.float()
        z = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
        a, b, rest = _pairs(z, s)
        return _joined(a * c - b * n, a * n + b * c, rest, s).to(DTYPES[s["dtype"]])

    return one(s["q"], s["wq"]), one(s["k"], s["wk"])


def _plain_qk_backward(s):
    c, n = _angles(s)

    def one(x, w, gy):
        x, w, gy = x.float(), w.float(), gy.float()
        a, b, rest = _pairs(gy, s)
        gz = _joined(a * c + b * n, b * c - a * n, rest, s)
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        xh, gw = x * r, gz * w
        gx = r * (gw - xh * (gw * xh).mean(-1, keepdim=True))
        return gx.to(DTYPES[s["dtype"]]), (gz * xh).sum((0, 1, 2))

    (gq, gwq), (gk, gwk) = one(s["q"], s["wq"], s["gq"]), one(s["k"], s["wk"], s["gk"])
    return {"q": gq, "k": gk, "wq": gwq, "wk": gwk}


def _plain_scan(a, b, c, log_decay, doc, first, last=None, C=128):
    """o_t = sum_{s <= t, same document} gamma^{t-s} (a_t . b_s) c_s, and the state after the last token, by
    chunks of C tokens: a [B,T,H,Da], b [B,T,H,Da], c [B,T,H,Dc] in fp32, doc [B,T] document numbers,
    first [B,H,Da,Dc] the state before the first token (of document 0) or None."""
    B, T, H, Da = a.shape
    n = (T + C - 1) // C
    pad = n * C - T
    a, b, c = (torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)).view(B, n, C, H, -1).permute(0, 3, 1, 2, 4)
               for x in (a, b, c))                                     # [B,H,n,C,D]
    doc = torch.nn.functional.pad(doc, (0, pad), mode="replicate").view(B, 1, n, C)
    g = log_decay.view(1, H, 1, 1)
    i = torch.arange(C, device=a.device)
    inside = (i[:, None] >= i) & (doc[..., :, None] == doc[..., None, :])
    w = torch.exp(g[..., None] * (i[:, None] - i).clamp(min=0)) * inside
    o = torch.matmul(torch.matmul(a, b.transpose(-1, -2)) * w, c)
    # what each chunk adds to the state at its end, and how much of each chunk's end reaches a later chunk's start
    ends = doc[..., -1:]
    add = torch.matmul((b * (torch.exp(g * (C - 1 - i)) * (doc == ends))[..., None]).transpose(-1, -2), c)
    m = torch.arange(n + 1, device=a.device)
    if first is None:
        first = torch.zeros(B, H, Da, c.shape[-1], device=a.device)
    e = torch.cat((torch.zeros_like(ends[:, :, :1, 0]), ends[..., 0]), -1)  # [B,1,n+1] document at each boundary
    x = torch.cat((first[:, :, None], add), 2)
    reach = torch.exp(g * (C * (m[:, None] - m)).clamp(min=0)) * (m[:, None] >= m) * (e[..., :, None] == e[..., None, :])
    state = torch.matmul(reach, x.flatten(3)).view_as(x)              # [B,H,n+1,Da,Dc] at the chunk boundaries
    seen = torch.exp(g * (i + 1)) * (doc == e[..., :-1, None])
    o = o + seen[..., None] * torch.matmul(a, state[:, :, :-1])
    o = o.permute(0, 2, 3, 1, 4).reshape(B, n * C, H, -1)[:, :T]
    # the padded tokens only let the last state fade: undone here, from the state before the last chunk
    j = T - (n - 1) * C
    tail = (torch.exp(g[..., 0] * (j - 1 - i).clamp(min=0)) * (doc[:, :, -1] == ends[:, :, -1]) * (i < j))[..., None]
    end = torch.matmul((b[:, :, -1] * tail).transpose(-1, -2), c[:, :, -1])
    keep = torch.exp(g * j) * (e[..., -1] == e[..., -2])[..., None, None]
    return o, state[:, :, -2] * keep + end


def _documents(s, device):
    flags = torch.zeros(s["B"] * s["T"], dtype=torch.int64, device=device)
    if s["doc_starts"] is not None:
        flags[s["doc_starts"].long()] = 1
    return flags.view(s["B"], s["T"]).cumsum(1)


def _heads(x, s):
    return x.float().repeat_interleave(s["H"] // s["Hkv"], -2)


def _plain_attn(s):
    o, S = _plain_scan(s["q"].float(), _heads(s["k"], s), _heads(s["v"], s), s["log_decay"], _documents(s, "cuda"), s["S0"])
    o = (o * s["scale"]).to(DTYPES[s["dtype"]])
    return (o, S) if s["state"] else o


def _plain_attn_backward(s):
    q, k, v, go = s["q"].float(), _heads(s["k"], s), _heads(s["v"], s), s["gO"].float()
    doc, ld, sc = _documents(s, "cuda"), s["log_decay"], s["scale"]
    S0 = None if s["S0"] is None else s["S0"].transpose(-1, -2)
    gq, _ = _plain_scan(go, v, k, ld, doc, S0)
    # backwards in time; the gradient of the last state belongs to the last document and enters without a decay
    back = doc[:, -1:] - doc.flip(1)
    qf, kf, vf, gf = (x.flip(1) for x in (q, k, v, go))
    first = None
    if s["gS"] is not None:
        first = s["gS"] / sc * torch.exp(-ld).view(1, -1, 1, 1)
    gv, R = _plain_scan(kf, qf, gf, ld, back, first)
    gk, _ = _plain_scan(vf, gf, qf, ld, back, None if first is None else first.transpose(-1, -2))
    G = s["H"] // s["Hkv"]
    dt = DTYPES[s["dtype"]]
    out = {"q": (gq * sc).to(dt), "k": (gk.flip(1) * sc).unflatten(2, (-1, G)).sum(3).to(dt),
           "v": (gv.flip(1) * sc).unflatten(2, (-1, G)).sum(3).to(dt)}
    if s["S0"] is not None:
        out["S0"] = R * (sc * torch.exp(ld)).view(1, -1, 1, 1) * (doc[:, 0] == 0).view(-1, 1, 1, 1)
    return out


def _plain_attn_step(s):
    S = s["S0"]
    k, v = _heads(s["k"], s), _heads(s["v"], s)
    S.mul_(torch.exp(s["log_decay"]).view(1, -1, 1, 1)).add_(k[..., :, None] * v[..., None, :])
    o = torch.matmul(s["q"].float()[..., None, :], S)[..., 0, :] * s["scale"]
    return o.to(DTYPES[s["dtype"]]), S


def _plain_loss(s, grads):
    H, W, t = s["H"].float(), s["W"].float(), s["targets"]
    logits = torch.matmul(H, W.t())
    lse = torch.logsumexp(logits, -1)
    kept = t >= 0
    at = t.clamp(min=0)[:, None]
    loss = torch.where(kept, lse - logits.gather(1, at)[:, 0], 0.0)
    if not grads:
        return loss, lse
    p = logits.sub_(lse[:, None]).exp_()
    p.scatter_add_(1, at, torch.full_like(lse, -1.0)[:, None])
    p.mul_(torch.where(kept, s["gloss"], 0.0)[:, None])
    dt = DTYPES[s["dtype"]]
    return {"loss": loss, "H": torch.matmul(p, W).to(dt), "W": torch.matmul(p.t(), H).to(dt)}


# ------------------------------------------------------------------ the package's entry points

def _own(s):
    import chunk_wise_weight_gate_b200 as pkg

    op = s["op"]
    if op.startswith("qk"):
        cfg = pkg.QKNormRopeConfig(B=s["B"], T=s["T"], Hq=s["Hq"], Hk=s["Hk"], D=s["D"], R=s["R"], eps=1e-6,
                                   interleaved=s["interleaved"], dtype=s["dtype"])
        x = (s["q"], s["k"], s["wq"], s["wk"], s["inv_freq"], s["positions"])
        if op == "qk_fwd":
            return pkg.qk_norm_rope(cfg, *x)
        return pkg.qk_norm_rope_backward(cfg, *x, s["gq"], s["gk"])
    if op.startswith("attn"):
        cfg = pkg.LinearAttentionConfig(B=s["B"], T=s["T"], H=s["H"], Hkv=s["Hkv"], Dk=s["Dk"], Dv=s["Dv"],
                                        scale=s["scale"], dtype=s["dtype"])
        if op == "attn_step":
            return pkg.linear_attention_step(cfg, s["S0"], s["q"], s["k"], s["v"], s["log_decay"]), s["S0"]
        if op == "attn_fwd":
            return pkg.linear_attention(cfg, s["q"], s["k"], s["v"], s["log_decay"], s["doc_starts"], S0=s["S0"],
                                        S_final=s["state"])
        return pkg.linear_attention_backward(cfg, s["q"], s["k"], s["v"], s["log_decay"], s["doc_starts"], s["gO"],
                                             S0=s["S0"], gS_final=s["gS"])
    cfg = pkg.CrossEntropyConfig(N=s["N"], V=s["V"], d=s["d"], dtype=s["dtype"])
    loss, lse = pkg.cross_entropy(cfg, s["H"], s["W"], s["targets"])
    if op == "loss_fwd":
        return loss, lse
    g = pkg.cross_entropy_backward(cfg, s["H"], s["W"], s["targets"], lse, s["gloss"])
    return {"loss": loss, "H": g["H"], "W": g["W"]}


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "qk_fwd":
        return _plain_qk(state)
    if op == "qk_bwd":
        return _plain_qk_backward(state)
    if op == "attn_step":
        return _plain_attn_step(state)
    if op == "attn_fwd":
        return _plain_attn(state)
    if op == "attn_bwd":
        return _plain_attn_backward(state)
    return _plain_loss(state, op == "loss_grad")


# ------------------------------------------------------------------ work

def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if op.startswith("qk"):
        n = case["B"] * case["T"] * (case["Hq"] + case["Hk"]) * case["D"]
        tail = case["B"] * case["T"] * 8 + case["R"] * 4 + 2 * case["D"] * e
        if op == "qk_fwd":
            return {"bytes": 2 * n * e + tail, "flops": 8 * n}
        return {"bytes": 3 * n * e + tail + 8 * case["D"], "flops": 16 * n}
    if op.startswith("attn"):
        B, T, H, Hkv, Dk, Dv = (case[k] for k in ("B", "T", "H", "Hkv", "Dk", "Dv"))
        q, k, v, o = (B * T * h * w * e for h, w in ((H, Dk), (Hkv, Dk), (Hkv, Dv), (H, Dv)))
        state = 4 * B * H * Dk * Dv
        mac = 2 * B * T * H * Dk * Dv
        if op == "attn_bwd":
            # q, k, v, gO in, gq, gk, gv out; the two states' updates and the three products with them
            return {"bytes": 2 * (q + k + v) + o + (3 * state if case["state"] else 0), "flops": 5 * mac}
        return {"bytes": q + k + v + o + (2 * state if case["state"] else 0), "flops": 2 * mac}
    N, V, d = case["N"], case["V"], case["d"]
    if op == "loss_fwd":
        return {"bytes": (N + V) * d * e + 16 * N, "flops": 2 * N * V * d}
    return {"bytes": 2 * (N + V) * d * e + 16 * N, "flops": 6 * N * V * d}


# ------------------------------------------------------------------ the definition, in 64 bits

def _exact_qk(s, backward):
    """Pair by pair as a complex number: y = z e^{i th}."""
    D, R = s["D"], s["R"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["positions"].double()[..., None] * s["inv_freq"]).unsqueeze(2)
    idx = torch.arange(R, device="cuda")
    order = idx.view(-1, 2) if s["interleaved"] else idx.view(2, -1).t()     # [R/2, 2]

    def rotate(z, e):
        y = z.clone()
        c = torch.complex(z[..., order[:, 0]], z[..., order[:, 1]]) * e
        y[..., order[:, 0]], y[..., order[:, 1]] = c.real, c.imag
        return y

    out = {}
    for n, x, w in (("q", s["q"], s["wq"]), ("k", s["k"], s["wk"])):
        x, w = x.double(), w.double()
        norm = (x.square().sum(-1, keepdim=True) / D + 1e-6).sqrt()
        if not backward:
            out[n] = rotate(x / norm * w, turn)
            continue
        gz = rotate(s["g" + n].double(), turn.conj())
        u = gz * w
        out[n] = u / norm - x * (u * x).sum(-1, keepdim=True) / (D * norm ** 3)
        out["w" + n] = torch.einsum("bthd,bthd->d", gz, x / norm)
    return {k: out[k] for k in ("q", "k", "wq", "wk")} if backward else (out["q"], out["k"])


def _exact_walk(a, b, c, decay, cut, S, times, enters):
    """Token by token: S <- (cut ? 0 : decay S) + b c^T, o = a S, over `times`; `enters`: the first token of the walk
    takes S without the decay."""
    o = torch.empty(*a.shape[:3], c.shape[-1], dtype=torch.float64, device=a.device)
    B, _, H, Da = a.shape
    S = torch.zeros(B, H, Da, c.shape[-1], dtype=torch.float64, device=a.device) if S is None else S.double()
    fade = torch.where(cut[:, :, None], 0.0, decay)[..., None, None]          # [B,T,H,1,1]
    for n, t in enumerate(times):
        S = torch.addcmul(S if n == 0 and enters else S * fade[:, t], b[:, t, :, :, None], c[:, t, :, None, :])
        o[:, t] = torch.matmul(a[:, t, :, None, :], S)[..., 0, :]
    return o, S


def _exact_attn(s):
    G, T = s["H"] // s["Hkv"], s["T"]
    q = s["q"].double()
    k, v = (x.double().repeat_interleave(G, -2) for x in (s["k"], s["v"]))
    decay = s["log_decay"].double().exp()
    if s["op"] == "attn_step":
        S = s["S0"].double() * decay[None, :, None, None] + torch.einsum("bhk,bhv->bhkv", k, v)
        return torch.einsum("bhk,bhkv->bhv", q, S) * s["scale"], S
    cut = torch.zeros(s["B"] * T, dtype=torch.bool, device="cuda")
    if s["doc_starts"] is not None:
        cut[s["doc_starts"].long()] = True
    cut = cut.view(s["B"], T)
    if s["op"] == "attn_fwd":
        o, S = _exact_walk(q, k, v, decay, cut, s["S0"], range(T), False)
        return (o * s["scale"], S) if s["state"] else o * s["scale"]
    go, sc = s["gO"].double(), s["scale"]
    S0 = None if s["S0"] is None else s["S0"].transpose(-1, -2)
    gq, _ = _exact_walk(go, v, k, decay, cut, S0, range(T), False)
    # from the last token down, a token is cut off from the next one where that one starts a document
    after = torch.cat((cut[:, 1:], torch.zeros_like(cut[:, :1])), 1)
    R = None if s["gS"] is None else s["gS"].double() / sc
    down = range(T - 1, -1, -1)
    gv, first = _exact_walk(k, q, go, decay, after, R, down, True)
    gk, _ = _exact_walk(v, go, q, decay, after, None if R is None else R.transpose(-1, -2), down, True)
    out = {"q": gq * sc, "k": (gk * sc).unflatten(2, (-1, G)).sum(3), "v": (gv * sc).unflatten(2, (-1, G)).sum(3)}
    if s["S0"] is not None:
        out["S0"] = first * sc * torch.where(cut[:, 0, None], 0.0, decay)[..., None, None]
    return out


def _exact_loss(s, grads):
    H, W, t = s["H"].double(), s["W"].double(), s["targets"]
    N = H.shape[0]
    loss, lse = (torch.zeros(N, dtype=torch.float64, device="cuda") for _ in range(2))
    gH, gW = (torch.zeros_like(H), torch.zeros_like(W)) if grads else (None, None)
    for lo in range(0, N, 1024):
        rows = slice(lo, min(N, lo + 1024))
        p = H[rows] @ W.t()
        top = p.max(1, keepdim=True).values
        e = p.sub(top).exp_()
        total = e.sum(1, keepdim=True)
        lse[rows] = (top + total.log())[:, 0]
        use = torch.nonzero(t[rows] >= 0)[:, 0]
        loss[rows][use] = lse[rows][use] - p[use, t[rows][use]]
        if grads:
            e /= total
            e[use, t[rows][use]] -= 1
            e *= torch.where(t[rows] >= 0, s["gloss"][rows].double(), 0.0)[:, None]
            gH[rows] = e @ W
            gW += e.t() @ H[rows]
    return {"loss": loss, "H": gH, "W": gW} if grads else (loss, lse)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("qk"):
        return _exact_qk(s, case["op"] == "qk_bwd")
    if case["op"].startswith("attn"):
        return _exact_attn(s)
    return _exact_loss(s, case["op"] == "loss_grad")

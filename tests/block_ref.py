"""Plain 64-bit implementations (torch, CPU) of the operators around the layer, token by
token from their definitions, differentiable by autograd; and the tests' inputs."""
import torch


def rand(seed, *shape, std=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def qk_one(x, w, inv_freq, positions, R, eps, interleaved):
    """x [B,T,H,D] float64: norm per head, then every pair turned by its angle."""
    z = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w
    y = [z[..., i] for i in range(z.shape[-1])]
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        th = (positions.double() * inv_freq[i])[..., None]
        c, s = torch.cos(th), torch.sin(th)
        y[a], y[b] = z[..., a] * c - z[..., b] * s, z[..., b] * c + z[..., a] * s
    return torch.stack(y, -1)


def linear_attention(q, k, v, log_decay, scale, starts=(), S0=None):
    """The recurrence, token by token; starts: offsets b*T + t.  Returns O, S_T."""
    B, T, H, Dk = q.shape
    G = H // k.shape[2]
    k, v = k.repeat_interleave(G, 2), v.repeat_interleave(G, 2)
    gamma = torch.exp(log_decay.double()).view(1, H, 1, 1)
    S = torch.zeros(B, H, Dk, v.shape[-1], dtype=torch.float64) if S0 is None else S0
    starts = set(int(s) for s in starts)
    out = []
    for t in range(T):
        keep = torch.tensor([0.0 if b * T + t in starts else 1.0 for b in range(B)], dtype=torch.float64).view(B, 1, 1, 1)
        S = torch.where(keep > 0, gamma * S, torch.zeros_like(S)) + k[:, t, :, :, None] * v[:, t, :, None, :]
        out.append(scale * torch.einsum("bhk,bhkv->bhv", q[:, t], S))
    return torch.stack(out, 1), S


def cross_entropy(H, W, targets, ignore_index=-100):
    logits = H @ W.t()
    lse = torch.logsumexp(logits, -1)
    keep = targets != ignore_index
    at = torch.where(keep, targets, 0)
    return torch.where(keep, lse - logits.gather(1, at[:, None])[:, 0], 0.0), lse


def leaves(*ts):
    return [None if t is None else t.detach().double().cpu().requires_grad_() for t in ts]


def relative(x, ref):
    """2-norm of the difference over the 2-norm of the reference."""
    x, ref = x.detach().double().cpu(), ref.detach().double()
    n = ref.norm()
    return float((x - ref).norm() / n) if n > 0 else float(x.norm())

"""Binding of libipttt.so's operators around the TTT MLP layer: norms of queries and keys
with the position rotation, linear attention with a decay for each head (prompts, single
tokens, gradients), and the softmax cross entropy of a linear head with its gradients.

As in ipttt.py: argument marshalling only, no fallback.  Every function checks its tensors
(device, type, shape, strides), runs on the tensors' device and on `stream` (default: that
device's current stream), and takes what it allocates from that stream.  Token tensors
[B, T, heads, width] may be views whose tokens lie apart (q, k and v of one fused
projection): heads and width packed, any token stride that is a multiple of 8 elements.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from .ipttt import BF16, F32, LinattnParams, QKParams, XentParams, _check, lib

_DTYPES = {"bf16": (BF16, torch.bfloat16), "f32": (F32, torch.float32)}
_byref = ctypes.byref


def _dtype(name: str):
    if name not in _DTYPES:
        raise ValueError(f"dtype {name!r}, expected 'bf16' or 'f32'")
    return _DTYPES[name]


class _On:
    """Runs its block on t's device and on `stream` (default: that device's current one), so that what
    is allocated inside belongs to that stream; gives the stream's handle."""
    __slots__ = ("device", "stream", "inner")

    def __init__(self, t: torch.Tensor, stream):
        if not t.is_cuda:
            raise ValueError("the tensors must be CUDA tensors")
        self.device, self.stream, self.inner = t.device, stream, ()
        if stream is not None and stream.device != self.device:
            raise ValueError(f"stream of {stream.device}, tensors on {self.device}")

    def __enter__(self):
        index = self.device.index
        if self.stream is not None:
            self.inner = (torch.cuda.device(index), torch.cuda.stream(self.stream))
        elif index != torch._C._cuda_getDevice():
            self.inner = (torch.cuda.device(index),)
        for c in self.inner:
            c.__enter__()
        return self.stream.cuda_stream if self.stream is not None else torch._C._cuda_getCurrentRawStream(index)

    def __exit__(self, *error):
        for c in reversed(self.inner):
            c.__exit__(*error)


def _mismatch(t, name, shape, dtype, device):
    return ValueError(f"{name}: {tuple(t.shape)} {t.dtype} on {t.device}, expected {shape} {dtype} on {device}")


def _flat(t, name, shape, dtype, device):
    """Pointer of a packed tensor (None: None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        raise _mismatch(t, name, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _tokens(t, name, shape, dtype, device):
    """(pointer, token stride) of a token tensor [B, T, heads, width]; stride 0: packed."""
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        raise _mismatch(t, name, shape, dtype, device)
    if t.is_contiguous():
        return t.data_ptr(), 0
    B, T, H, D = shape
    sb, st, sh, sd = t.stride()
    ld = st if T > 1 else sb if B > 1 else H * D
    if (sd != 1 and D > 1) or (sh != D and H > 1) or (B > 1 and sb != T * ld) or ld < H * D or ld % 8:
        raise ValueError(f"{name}: strides {t.stride()}; heads and width must be packed, tokens a constant multiple of "
                         "8 elements apart")
    return t.data_ptr(), ld


_packed = torch.contiguous_format


def _starts(doc_starts, device):
    """(pointer, count, tensor to keep) of document starts b*T + t on `device`."""
    if doc_starts is None:
        return None, 0, None
    ds = doc_starts if isinstance(doc_starts, torch.Tensor) else torch.as_tensor(doc_starts, dtype=torch.int32)
    if ds.dtype == torch.int64:  # an offset beyond 32 bits stays out of range: the call reports it
        ds = ds.clamp(-1, 2 ** 31 - 1)
    elif ds.dtype != torch.int32:
        raise ValueError(f"doc_starts: {ds.dtype}, expected int32 or int64 offsets")
    ds = ds.to(device=device, dtype=torch.int32).contiguous()
    return (ds.data_ptr() if ds.numel() else None), ds.numel(), ds


def _workspace(workspace, need, device):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if workspace.dtype != torch.uint8 or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
    return workspace


def _size(fn, params, what):
    n = fn(_byref(params))
    if n == 0:
        raise ValueError(f"invalid configuration {what}")
    return n


# ---------------------------------------------------------------- norms and rotation

@dataclass
class QKNormRopeConfig:
    """B sequences of T tokens; Hq query and Hk key heads of width D, of which the first R
    elements are rotated (pairs (i, i + R/2), or (2i, 2i+1) when interleaved)."""
    B: int
    T: int
    Hq: int
    Hk: int
    D: int
    R: int
    eps: float = 1e-6
    interleaved: bool = False
    dtype: str = "bf16"

    def params(self, ldq=0, ldk=0, ldqo=0, ldko=0, ldgq=0, ldgk=0) -> QKParams:
        return QKParams(self.B, self.T, self.Hq, self.Hk, self.D, self.R, _dtype(self.dtype)[0], int(self.interleaved),
                        self.eps, ldq, ldk, ldqo, ldko, ldgq, ldgk)


def _qk_inputs(cfg, q, k, wq, wk, inv_freq, positions):
    dt, dev = _dtype(cfg.dtype)[1], q.device
    B, T, D = cfg.B, cfg.T, cfg.D
    sq, sk = (B, T, cfg.Hq, D), (B, T, cfg.Hk, D)
    pq, ldq = _tokens(q, "q", sq, dt, dev)
    pk, ldk = _tokens(k, "k", sk, dt, dev)
    turned = (_flat(inv_freq, "inv_freq", (cfg.R // 2,), torch.float64, dev),
              _flat(positions, "positions", (B, T), torch.int64, dev)) if cfg.R else (None, None)
    return (pq, pk, _flat(wq, "wq", (D,), dt, dev), _flat(wk, "wk", (D,), dt, dev), *turned), ldq, ldk, sq, sk, dt, dev


def qk_norm_rope(cfg: QKNormRopeConfig, q, k, wq, wk, inv_freq, positions, *, q_out=None, k_out=None, stream=None):
    """RMS norm of every head of q [B,T,Hq,D] and k [B,T,Hk,D] with weights wq, wk [D], then
    the rotation by positions [B,T] (int64) * inv_freq [R/2] (float64, radians a
    position).  Returns (q_out, k_out), packed unless given; q_out may be q, k_out k."""
    ptrs, ldq, ldk, sq, sk, dt, dev = _qk_inputs(cfg, q, k, wq, wk, inv_freq, positions)
    with _On(q, stream) as st:
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=_packed)
            pq, ldqo = q_out.data_ptr(), 0
        else:
            pq, ldqo = _tokens(q_out, "q_out", sq, dt, dev)
        if k_out is None:
            k_out = torch.empty_like(k, memory_format=_packed)
            pk, ldko = k_out.data_ptr(), 0
        else:
            pk, ldko = _tokens(k_out, "k_out", sk, dt, dev)
        rc = lib().ipttt_qk_norm_rope(_byref(cfg.params(ldq, ldk, ldqo, ldko)), *ptrs, pq, pk, st)
        if rc:
            _check(rc, "ipttt_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_backward(cfg: QKNormRopeConfig, q, k, wq, wk, inv_freq, positions, gq_out, gk_out, *, gq=None,
                          gk=None, workspace=None, stream=None):
    """Gradients of <gq_out, q_out> + <gk_out, k_out>: a dict with q and k (the call's dtype,
    packed unless gq, gk are given; they may be gq_out, gk_out, or q, k) and wq, wk (fp32)."""
    ptrs, ldq, ldk, sq, sk, dt, dev = _qk_inputs(cfg, q, k, wq, wk, inv_freq, positions)
    pgq, ldqo = _tokens(gq_out, "gq_out", sq, dt, dev)
    pgk, ldko = _tokens(gk_out, "gk_out", sk, dt, dev)
    with _On(q, stream) as st:
        gq = torch.empty_like(q, memory_format=_packed) if gq is None else gq
        gk = torch.empty_like(k, memory_format=_packed) if gk is None else gk
        po, ldgq = _tokens(gq, "gq", sq, dt, dev)
        pk, ldgk = _tokens(gk, "gk", sk, dt, dev)
        gw = torch.empty(2, cfg.D, dtype=torch.float32, device=dev)
        p = cfg.params(ldq, ldk, ldqo, ldko, ldgq, ldgk)
        ws = _workspace(workspace, _size(lib().ipttt_qk_norm_rope_backward_workspace_size, p, cfg), dev)
        _check(lib().ipttt_qk_norm_rope_backward(_byref(p), *ptrs, pgq, pgk, po, pk, gw.data_ptr(),
                                                 gw.data_ptr() + 4 * cfg.D, ws.data_ptr(), ws.numel(), st),
               "ipttt_qk_norm_rope_backward")
    return {"q": gq, "k": gk, "wq": gw[0], "wk": gw[1]}


# ---------------------------------------------------------------- linear attention

@dataclass
class LinearAttentionConfig:
    """B sequences of T tokens; H query heads over Hkv key/value heads, widths Dk and Dv."""
    B: int
    T: int
    H: int
    Hkv: int
    Dk: int
    Dv: int
    scale: float
    dtype: str = "bf16"

    def params(self, ldq=0, ldk=0, ldv=0, ldo=0, ldgq=0, ldgk=0, ldgv=0, T=None) -> LinattnParams:
        return LinattnParams(self.B, self.T if T is None else T, self.H, self.Hkv, self.Dk, self.Dv,
                             _dtype(self.dtype)[0], self.scale, ldq, ldk, ldv, ldo, ldgq, ldgk, ldgv)

    def shapes(self):
        B, T = self.B, self.T
        return {"q": (B, T, self.H, self.Dk), "k": (B, T, self.Hkv, self.Dk), "v": (B, T, self.Hkv, self.Dv),
                "O": (B, T, self.H, self.Dv), "S": (B, self.H, self.Dk, self.Dv)}


def linear_attention_workspace_size(cfg: LinearAttentionConfig, backward: bool = False) -> int:
    L = lib()
    return _size(L.ipttt_linattn_backward_workspace_size if backward else L.ipttt_linattn_workspace_size, cfg.params(),
                 cfg)


def linear_attention(cfg: LinearAttentionConfig, q, k, v, log_decay, doc_starts=None, *, S0=None, O=None,
                     S_final=False, workspace=None, stream=None):
    """o_t = scale q_t S_t with S_t = exp(log_decay) S_{t-1} + k_t v_t^T, S reset at document
    starts (offsets b*T + t).  S0: the state before the first token, fp32 [B,H,Dk,Dv]
    (None: zero).  Returns O [B,T,H,Dv], or (O, S_T) with S_final=True or with S_final an
    fp32 [B,H,Dk,Dv] tensor to write (S0 itself may be it)."""
    dt, dev, sh = _dtype(cfg.dtype)[1], q.device, cfg.shapes()
    f32 = torch.float32
    pq, ldq = _tokens(q, "q", sh["q"], dt, dev)
    pk, ldk = _tokens(k, "k", sh["k"], dt, dev)
    pv, ldv = _tokens(v, "v", sh["v"], dt, dev)
    pd = _flat(log_decay, "log_decay", (cfg.H,), f32, dev)
    p0 = _flat(S0, "S0", sh["S"], f32, dev)
    with _On(q, stream) as st:
        if O is None:
            O = q.new_empty(sh["O"])
        Sf = torch.empty(sh["S"], dtype=f32, device=dev) if S_final is True else S_final if S_final is not False else None
        po, ldo = _tokens(O, "O", sh["O"], dt, dev)
        p = cfg.params(ldq, ldk, ldv, ldo)
        ws = _workspace(workspace, _size(lib().ipttt_linattn_workspace_size, p, cfg), dev)
        dp, nd, keep = _starts(doc_starts, dev)
        _check(lib().ipttt_linattn_forward(_byref(p), pq, pk, pv, pd, dp, nd, p0, po,
                                           _flat(Sf, "S_final", sh["S"], f32, dev), ws.data_ptr(), ws.numel(), st),
               "ipttt_linattn_forward")
    return O if Sf is None else (O, Sf)


def linear_attention_backward(cfg: LinearAttentionConfig, q, k, v, log_decay, doc_starts, gO, *, S0=None,
                              gS_final=None, gq=None, gk=None, gv=None, workspace=None, stream=None):
    """Gradients of <gO, O> + <gS_final, S_T>: a dict with q, k and v (the call's dtype, packed unless
    gq, gk, gv are given: views of one projection's gradient, say) and, when S0 is given, S0 (fp32)."""
    dt, dev, sh = _dtype(cfg.dtype)[1], q.device, cfg.shapes()
    f32 = torch.float32
    pq, ldq = _tokens(q, "q", sh["q"], dt, dev)
    pk, ldk = _tokens(k, "k", sh["k"], dt, dev)
    pv, ldv = _tokens(v, "v", sh["v"], dt, dev)
    pg, ldo = _tokens(gO, "gO", sh["O"], dt, dev)
    pd = _flat(log_decay, "log_decay", (cfg.H,), f32, dev)
    p0 = _flat(S0, "S0", sh["S"], f32, dev)
    ps = _flat(gS_final, "gS_final", sh["S"], f32, dev)
    with _On(q, stream) as st:
        out, grads, lds = {}, [], []
        for n, t, g in (("q", q, gq), ("k", k, gk), ("v", v, gv)):
            if g is None:
                g = torch.empty_like(t, memory_format=_packed)
                at, ld = g.data_ptr(), 0
            else:
                at, ld = _tokens(g, "g" + n, sh[n], dt, dev)
            out[n] = g
            grads.append(at)
            lds.append(ld)
        if S0 is not None:
            out["S0"] = torch.empty(sh["S"], dtype=f32, device=dev)
        p = cfg.params(ldq, ldk, ldv, ldo, *lds)
        ws = _workspace(workspace, _size(lib().ipttt_linattn_backward_workspace_size, p, cfg), dev)
        dp, nd, keep = _starts(doc_starts, dev)
        _check(lib().ipttt_linattn_backward(_byref(p), pq, pk, pv, pd, dp, nd, p0, pg, ps, *grads,
                                            out["S0"].data_ptr() if S0 is not None else None, ws.data_ptr(),
                                            ws.numel(), st), "ipttt_linattn_backward")
    return out


def _rows(t, name, shape, dtype, device):
    """_tokens for one token a row: t [B, heads, width]."""
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        raise _mismatch(t, name, shape, dtype, device)
    if t.is_contiguous():
        return t.data_ptr(), 0
    B, H, D = shape
    return _tokens(t.unsqueeze(1), name, (B, 1, H, D), dtype, device)


def linear_attention_step(cfg: LinearAttentionConfig, S, q, k, v, log_decay, starts=None, *, o=None, stream=None):
    """One token of every row on the state S (fp32 [B,H,Dk,Dv], updated in place): q [B,H,Dk],
    k [B,Hkv,Dk], v [B,Hkv,Dv]; starts: int32 [B] on the device, nonzero where the row's token
    starts a document.  Returns o [B,H,Dv].  cfg.T is ignored."""
    dt, dev = _dtype(cfg.dtype)[1], q.device
    B, H, Hkv, Dk, Dv = cfg.B, cfg.H, cfg.Hkv, cfg.Dk, cfg.Dv

    pq, ldq = _rows(q, "q", (B, H, Dk), dt, dev)
    pk, ldk = _rows(k, "k", (B, Hkv, Dk), dt, dev)
    pv, ldv = _rows(v, "v", (B, Hkv, Dv), dt, dev)
    ps = _flat(S, "S", (B, H, Dk, Dv), torch.float32, dev)
    pd = _flat(log_decay, "log_decay", (H,), torch.float32, dev)
    pn = _flat(starts, "starts", (B,), torch.int32, dev)
    if ps is None:
        raise ValueError("S is missing")
    with _On(q, stream) as st:
        if o is None:
            o = q.new_empty((B, H, Dv))
            po, ldo = o.data_ptr(), 0
        else:
            po, ldo = _rows(o, "o", (B, H, Dv), dt, dev)
        rc = lib().ipttt_linattn_step(_byref(cfg.params(ldq, ldk, ldv, ldo, T=1)), ps, pq, pk, pv, pd, pn, po, st)
        if rc:
            _check(rc, "ipttt_linattn_step")
    return o


# ---------------------------------------------------------------- softmax cross entropy

@dataclass
class CrossEntropyConfig:
    """N tokens, a vocabulary of V, width d; targets equal to ignore_index take no part.
    piece: vocabulary rows the backward handles at a time (0: chosen by the library)."""
    N: int
    V: int
    d: int
    ignore_index: int = -100
    dtype: str = "bf16"
    piece: int = 0

    def params(self) -> XentParams:
        return XentParams(self.N, self.V, self.d, _dtype(self.dtype)[0], self.piece, self.ignore_index)


def cross_entropy_workspace_size(cfg: CrossEntropyConfig, backward: bool = False) -> int:
    L = lib()
    return _size(L.ipttt_xent_backward_workspace_size if backward else L.ipttt_xent_workspace_size, cfg.params(), cfg)


def cross_entropy(cfg: CrossEntropyConfig, H, W, targets, *, workspace=None, stream=None):
    """Per-token loss of the head W [V,d] on H [N,d] for targets [N] (int64): returns (loss,
    lse), fp32 [N]; lse goes to cross_entropy_backward.  The logits are never kept."""
    dt, dev, f32 = _dtype(cfg.dtype)[1], H.device, torch.float32
    ptrs = [_flat(H, "H", (cfg.N, cfg.d), dt, dev), _flat(W, "W", (cfg.V, cfg.d), dt, dev),
            _flat(targets, "targets", (cfg.N,), torch.int64, dev)]
    with _On(H, stream) as st:
        loss, lse = torch.empty(cfg.N, dtype=f32, device=dev), torch.empty(cfg.N, dtype=f32, device=dev)
        ws = _workspace(workspace, cross_entropy_workspace_size(cfg), dev)
        p = cfg.params()
        _check(lib().ipttt_xent_forward(_byref(p), *ptrs, loss.data_ptr(), lse.data_ptr(), ws.data_ptr(),
                                        ws.numel(), st), "ipttt_xent_forward")
    return loss, lse


def cross_entropy_backward(cfg: CrossEntropyConfig, H, W, targets, lse, gloss, *, gH=None, gW=None, workspace=None,
                           stream=None):
    """Gradients of <gloss, loss> (gloss fp32 [N]; 1/count everywhere for a mean): a dict
    with H and W in the call's dtype, from the lse that cross_entropy returned."""
    dt, dev, f32 = _dtype(cfg.dtype)[1], H.device, torch.float32
    ptrs = [_flat(H, "H", (cfg.N, cfg.d), dt, dev), _flat(W, "W", (cfg.V, cfg.d), dt, dev),
            _flat(targets, "targets", (cfg.N,), torch.int64, dev), _flat(lse, "lse", (cfg.N,), f32, dev),
            _flat(gloss, "gloss", (cfg.N,), f32, dev)]
    with _On(H, stream) as st:
        gH = torch.empty(cfg.N, cfg.d, dtype=dt, device=dev) if gH is None else gH
        gW = torch.empty(cfg.V, cfg.d, dtype=dt, device=dev) if gW is None else gW
        ws = _workspace(workspace, cross_entropy_workspace_size(cfg, backward=True), dev)
        p = cfg.params()
        _check(lib().ipttt_xent_backward(_byref(p), *ptrs, _flat(gH, "gH", (cfg.N, cfg.d), dt, dev),
                                         _flat(gW, "gW", (cfg.V, cfg.d), dt, dev), ws.data_ptr(), ws.numel(), st),
               "ipttt_xent_backward")
    return {"H": gH, "W": gW}

"""Refusals of the operators around the layer that need no GPU: argument errors come back
before any CUDA call, and the binding raises for tensors it cannot take."""
import ctypes

import pytest
import torch

import chunk_wise_weight_gate_b200 as pkg
from chunk_wise_weight_gate_b200 import ipttt as ip

FAKE = [0x100000 + 4096 * i for i in range(16)]  # never dereferenced: the checks fail first


def qk(**kw):
    d = dict(B=2, T=5, Hq=4, Hk=2, D=128, R=64, dtype=ip.BF16, interleaved=0, eps=1e-6)
    d.update(kw)
    return ip.QKParams(**d)


def qk_call(p, ptrs=FAKE[:8]):
    return ip.lib().ipttt_qk_norm_rope(ctypes.byref(p), *ptrs, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(Hq=0), 1), (dict(Hk=0), 1), (dict(D=0), 1), (dict(R=-8), 1), (dict(dtype=5), 4),
    (dict(eps=0.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(interleaved=2), 1),
    (dict(D=100), 5), (dict(R=12), 5), (dict(R=136), 5), (dict(D=264), 5), (dict(B=1 << 20, T=1 << 20), 2),
    (dict(ldq=504), 1), (dict(ldq=516), 1), (dict(ldk=8), 1), (dict(ldqo=100), 1), (dict(ldgk=250), 1),
])
def test_qk_norm_rope_refuses(kw, code):
    assert qk_call(qk(**kw)) == code
    L = ip.lib()
    assert L.ipttt_qk_norm_rope_backward_workspace_size(ctypes.byref(qk(**kw))) == 0
    assert L.ipttt_qk_norm_rope_backward(ctypes.byref(qk(**kw)), *FAKE[:13], 1 << 30, None) == code


def test_qk_norm_rope_refuses_pointers():
    for i in range(8):
        assert qk_call(qk(), FAKE[:i] + [None] + FAKE[i + 1:8]) == 1
    for i in (0, 1, 2, 3, 6, 7):
        assert qk_call(qk(), FAKE[:i] + [FAKE[i] + 8] + FAKE[i + 1:8]) == 3
    assert qk_call(qk(), FAKE[:5] + [FAKE[5] + 4] + FAKE[6:8]) == 3
    # in place with another stride
    assert qk_call(qk(ldq=1024), FAKE[:6] + [FAKE[0], FAKE[7]]) == 1
    L = ip.lib()
    need = L.ipttt_qk_norm_rope_backward_workspace_size(ctypes.byref(qk()))
    assert need > 0 and need % 256 == 0
    args = FAKE[:12]
    assert L.ipttt_qk_norm_rope_backward(ctypes.byref(qk()), *args, FAKE[12], need - 1, None) == 8
    assert L.ipttt_qk_norm_rope_backward(ctypes.byref(qk()), *args, None, need, None) == 8
    assert L.ipttt_qk_norm_rope_backward(ctypes.byref(qk()), *args, FAKE[12] + 16, need, None) == 3
    assert L.ipttt_qk_norm_rope_backward(ctypes.byref(qk()), *FAKE[:10], None, FAKE[11], FAKE[12], need, None) == 1


def la(**kw):
    d = dict(B=2, T=300, H=4, Hkv=2, Dk=128, Dv=64, dtype=ip.BF16, scale=0.1)
    d.update(kw)
    return ip.LinattnParams(**d)


def la_forward(p, q=FAKE[0], ds=None, n=0, ws=FAKE[9], size=1 << 40, O=FAKE[6], S0=None):
    return ip.lib().ipttt_linattn_forward(ctypes.byref(p), q, *FAKE[1:4], ds, n, S0, O, None, ws, size, None)


def la_backward(p, gq=FAKE[6], gS=None, gS0=None, size=1 << 40):
    return ip.lib().ipttt_linattn_backward(ctypes.byref(p), *FAKE[:4], None, 0, None, FAKE[5], gS, gq, *FAKE[7:9], gS0,
                                           FAKE[9], size, None)


def la_step(p, S=FAKE[4], o=FAKE[5]):
    return ip.lib().ipttt_linattn_step(ctypes.byref(p), S, *FAKE[:4], None, o, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(T=0), 1), (dict(H=0), 1), (dict(Hkv=0), 1), (dict(Dk=0), 1), (dict(Dv=-8), 1), (dict(Hkv=3), 1),
    (dict(dtype=2), 4), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(Dk=100), 5), (dict(Dv=264), 5), (dict(B=1 << 20, T=1 << 11), 2), (dict(B=40000), 2), (dict(ldq=256), 1),
    (dict(ldk=260), 1), (dict(ldv=4), 1), (dict(ldo=252), 1), (dict(ldgq=8), 1), (dict(ldgk=8), 1), (dict(ldgv=8), 1),
])
def test_linear_attention_refuses(kw, code):
    L = ip.lib()
    assert L.ipttt_linattn_workspace_size(ctypes.byref(la(**kw))) == 0
    assert L.ipttt_linattn_backward_workspace_size(ctypes.byref(la(**kw))) == 0
    assert la_forward(la(**kw)) == code
    assert la_backward(la(**kw)) == code
    if "T" not in kw:
        assert la_step(la(T=1, **kw)) == code


def test_linear_attention_refuses_pointers():
    L = ip.lib()
    p = la()
    need = L.ipttt_linattn_workspace_size(ctypes.byref(p))
    assert need > 0 and need % 256 == 0
    assert la_forward(p, q=None) == 1
    assert la_forward(p, O=None) == 1
    assert la_forward(p, q=FAKE[0] + 8) == 3
    assert la_forward(p, S0=FAKE[10] + 4) == 3
    assert la_forward(p, n=-1) == 1
    assert la_forward(p, n=2) == 1
    assert la_forward(p, size=need - 1) == 8
    assert la_forward(p, ws=None) == 8
    assert la_forward(p, ws=FAKE[9] + 16) == 3
    assert la_backward(p, gq=None) == 1
    assert la_backward(p, gq=FAKE[6] + 2) == 3
    assert la_backward(p, size=0) == 8
    assert la_backward(p, gS=FAKE[10], gS0=FAKE[10]) == 1
    assert la_step(p) == 1  # T is not 1
    assert la_step(la(T=1), S=None) == 1
    assert la_step(la(T=1), o=FAKE[5] + 4) == 3


def xe(**kw):
    d = dict(N=10, V=1000, d=64, dtype=ip.BF16, piece=0, ignore_index=-100)
    d.update(kw)
    return ip.XentParams(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(N=0), 1), (dict(V=0), 1), (dict(d=-32), 1), (dict(piece=100), 1), (dict(piece=-256), 1), (dict(dtype=9), 4),
    (dict(d=40), 5), (dict(d=66, dtype=ip.F32), 5), (dict(V=(1 << 26) + 1), 2), (dict(N=(1 << 24) + 1), 2),
])
def test_cross_entropy_refuses(kw, code):
    L = ip.lib()
    p = xe(**kw)
    assert L.ipttt_xent_workspace_size(ctypes.byref(p)) == 0
    assert L.ipttt_xent_backward_workspace_size(ctypes.byref(p)) == 0
    assert L.ipttt_xent_forward(ctypes.byref(p), *FAKE[:6], 1 << 40, None) == code
    assert L.ipttt_xent_backward(ctypes.byref(p), *FAKE[:8], 1 << 40, None) == code


def test_cross_entropy_refuses_pointers():
    L = ip.lib()
    p = xe()
    need, need_b = (f(ctypes.byref(p)) for f in (L.ipttt_xent_workspace_size, L.ipttt_xent_backward_workspace_size))
    assert need > 0 and need_b > 0
    for i in range(5):
        assert L.ipttt_xent_forward(ctypes.byref(p), *FAKE[:i], None, *FAKE[i + 1:6], need, None) == 1
    for i in range(7):
        assert L.ipttt_xent_backward(ctypes.byref(p), *FAKE[:i], None, *FAKE[i + 1:8], need_b, None) == 1
    assert L.ipttt_xent_forward(ctypes.byref(p), FAKE[0] + 8, *FAKE[1:6], need, None) == 3
    assert L.ipttt_xent_forward(ctypes.byref(p), *FAKE[:2], FAKE[2] + 4, *FAKE[3:6], need, None) == 3
    assert L.ipttt_xent_forward(ctypes.byref(p), *FAKE[:6], need - 1, None) == 8
    assert L.ipttt_xent_forward(ctypes.byref(p), *FAKE[:5], FAKE[5] + 64, need, None) == 3
    assert L.ipttt_xent_backward(ctypes.byref(p), *FAKE[:8], need_b - 1, None) == 8
    # smaller pieces take less room
    small = L.ipttt_xent_backward_workspace_size(ctypes.byref(xe(N=4096, V=100000, piece=256)))
    assert small < L.ipttt_xent_backward_workspace_size(ctypes.byref(xe(N=4096, V=100000, piece=8192)))


def test_binding_refuses_what_it_cannot_take():
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    ld = torch.zeros(2)
    cfg = pkg.LinearAttentionConfig(1, 4, 2, 2, 64, 64, 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.linear_attention(cfg, x, x, x, ld)
    for bad in (x.float(), x[:, :3], x.transpose(1, 2), torch.zeros(1, 4, 2, 68)[..., :64].to(torch.bfloat16)):
        with pytest.raises(ValueError):
            pkg.linear_attention(cfg, bad, x, x, ld)
    apart = torch.zeros(1, 4, 2 * 64 + 4, dtype=torch.bfloat16)[..., :128].unflatten(-1, (2, 64))
    with pytest.raises(ValueError, match="strides"):  # tokens 132 elements apart
        pkg.linear_attention(cfg, apart, x, x, ld)
    with pytest.raises(ValueError, match="log_decay"):
        pkg.linear_attention(cfg, x, x, x, ld.double())
    with pytest.raises(ValueError, match="dtype"):
        pkg.linear_attention(pkg.LinearAttentionConfig(1, 4, 2, 2, 64, 64, 1.0, "f16"), x, x, x, ld)
    with pytest.raises(ValueError):
        pkg.linear_attention_step(cfg, None, x[:, 0], x[:, 0], x[:, 0], ld)
    with pytest.raises(ValueError, match="invalid configuration"):
        pkg.linear_attention_workspace_size(pkg.LinearAttentionConfig(1, 4, 3, 2, 64, 64, 1.0))
    with pytest.raises(ValueError, match="invalid configuration"):
        pkg.cross_entropy_workspace_size(pkg.CrossEntropyConfig(1, 0, 64))
    H, W, t = torch.zeros(3, 64), torch.zeros(9, 64), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="targets"):
        pkg.cross_entropy(pkg.CrossEntropyConfig(3, 9, 64, dtype="f32"), H, W, t.int())
    with pytest.raises(ValueError, match="CUDA"):
        pkg.cross_entropy(pkg.CrossEntropyConfig(3, 9, 64, dtype="f32"), H, W, t)


def test_outputs_that_are_inputs_are_refused():
    for i in range(3):  # q, k, v
        assert la_forward(la(), O=FAKE[i]) == 1
        assert la_step(la(T=1), o=FAKE[i]) == 1
        assert la_backward(la(), gq=FAKE[i]) == 1
    assert la_backward(la(), gq=FAKE[5]) == 1  # gO
    L = ip.lib()
    assert qk_call(qk(), FAKE[:6] + [FAKE[1], FAKE[7]]) == 1  # q_out is k
    assert qk_call(qk(), FAKE[:6] + [FAKE[6], FAKE[0]]) == 1  # k_out is q
    for gq, gk in ((FAKE[1], FAKE[9]), (FAKE[7], FAKE[9]), (FAKE[8], FAKE[0]), (FAKE[8], FAKE[6])):
        assert L.ipttt_qk_norm_rope_backward(ctypes.byref(qk()), *FAKE[:8], gq, gk, *FAKE[10:13], 1 << 30, None) == 1
    # gq in q's place with another stride
    assert L.ipttt_qk_norm_rope_backward(ctypes.byref(qk(ldq=1024)), *FAKE[:8], FAKE[0], *FAKE[9:13], 1 << 30, None) == 1
    for gH, gW in ((FAKE[0], FAKE[6]), (FAKE[1], FAKE[6]), (FAKE[5], FAKE[0]), (FAKE[5], FAKE[1])):
        assert L.ipttt_xent_backward(ctypes.byref(xe()), *FAKE[:5], gH, gW, FAKE[7], 1 << 40, None) == 1

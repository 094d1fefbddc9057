"""No output of an operator around the layer may be an input's pointer, another output's or the
workspace's, except where the call says that it may be one: refused before any CUDA call."""
import ctypes

import pytest

from chunk_wise_weight_gate_b200 import ipttt as ip

HUGE = 1 << 40


def calls():
    """name: (function, parameters, argument names in order, outputs, pairs that may be one)."""
    L = ip.lib()
    qk = ip.QKParams(B=2, T=5, Hq=2, Hk=2, D=128, R=64, dtype=ip.F32, interleaved=0, eps=1e-6)
    la = ip.LinattnParams(B=2, T=300, H=2, Hkv=2, Dk=64, Dv=64, dtype=ip.F32, scale=0.1)
    one = ip.LinattnParams(B=2, T=1, H=2, Hkv=2, Dk=64, Dv=64, dtype=ip.F32, scale=0.1)
    xe = ip.XentParams(N=64, V=64, d=64, dtype=ip.F32, piece=0, ignore_index=-100)
    return {
        "qk_norm_rope": (L.ipttt_qk_norm_rope, qk, "q k wq wk inv_freq positions q_out k_out".split(), {"q_out", "k_out"},
                         {("q_out", "q"), ("k_out", "k")}),
        "qk_norm_rope_backward": (L.ipttt_qk_norm_rope_backward, qk,
                                  "q k wq wk inv_freq positions gqo gko gq gk gwq gwk ws".split(),
                                  {"gq", "gk", "gwq", "gwk", "ws"},
                                  {("gq", "q"), ("gq", "gqo"), ("gk", "k"), ("gk", "gko")}),
        "linattn_forward": (L.ipttt_linattn_forward, la, "q k v log_decay doc_starts #n S0 O S_final ws".split(),
                            {"O", "S_final", "ws"}, {("S_final", "S0")}),
        "linattn_backward": (L.ipttt_linattn_backward, la,
                             "q k v log_decay doc_starts #n S0 gO gS_final gq gk gv gS0 ws".split(),
                             {"gq", "gk", "gv", "gS0", "ws"}, set()),
        "linattn_step": (L.ipttt_linattn_step, one, "S q k v log_decay starts o".split(), {"S", "o"}, set()),
        "xent_forward": (L.ipttt_xent_forward, xe, "H W targets loss lse ws".split(), {"loss", "lse", "ws"}, set()),
        "xent_backward": (L.ipttt_xent_backward, xe, "H W targets lse gloss gH gW ws".split(), {"gH", "gW", "ws"}, set()),
    }


@pytest.mark.parametrize("name", ["qk_norm_rope", "qk_norm_rope_backward", "linattn_forward", "linattn_backward",
                                  "linattn_step", "xent_forward", "xent_backward"])
def test_outputs_are_no_inputs_and_not_one_another(name):
    fn, params, names, outs, allowed = calls()[name]
    ptr = {n: 0x100000 + 4096 * i for i, n in enumerate(names)}  # never dereferenced

    def call(**other):
        args = [3 if n == "#n" else {**ptr, **other}[n] for n in names]
        tail = [HUGE] if names[-1] == "ws" else []
        return fn(ctypes.byref(params), *args, *tail, None)

    refused = 0
    for out in sorted(outs):
        for n in names:
            if n == out or n == "#n" or (out, n) in allowed or (n in outs and n < out):
                continue
            assert call(**{out: ptr[n]}) == 1, (out, n)
            refused += 1
    assert refused > len(names)

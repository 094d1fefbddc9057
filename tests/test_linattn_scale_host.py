"""The scales that linear attention takes."""
import ctypes

import pytest

from chunk_wise_weight_gate_b200 import ipttt as ip

P = [0x100000 + 4096 * i for i in range(16)]  # never dereferenced: no call here gets as far


@pytest.mark.parametrize("scale,with_state,without", [(1e-39, 1, 8), (-1e-42, 1, 8), (1e-30, 8, 8), (0.125, 8, 8), (-2.0, 8, 8)])
def test_a_scale_without_a_reciprocal_is_refused_with_a_states_gradient(scale, with_state, without):
    # gS_final / scale is what the reverse recurrence starts from; 8: the call goes on to miss its workspace
    p = ip.LinattnParams(B=1, T=10, H=1, Hkv=1, Dk=64, Dv=64, dtype=ip.F32, scale=scale)
    for gS, code in ((P[12], with_state), (None, without)):
        assert ip.lib().ipttt_linattn_backward(ctypes.byref(p), *P[:4], None, 0, P[11], P[5], gS, *P[6:9], P[10], None, 0, None) == code

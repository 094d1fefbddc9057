"""How the operators around the layer are called: as a process's first call and captured at once, from
several host threads, with document starts that do not fit 32 bits."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import chunk_wise_weight_gate_b200 as pkg
from tests.test_gpu_block_ops import attn_case, qk_case, status, xent_case

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST = """
import sys, torch
import chunk_wise_weight_gate_b200 as pkg
from tests.test_gpu_block_ops import attn_case, qk_case, xent_case
what, dtype = sys.argv[1], sys.argv[2]
if what == "qk":
    a = qk_case(2, 50, 4, 2, 128, 64, dtype)
    def run():
        y = pkg.qk_norm_rope(*a)
        return [*y, *pkg.qk_norm_rope_backward(*a, *y).values()]
elif what == "attention":
    cfg, q, k, v, ld, S0, ds = attn_case(1, 3000, 2, 1, 64, 128, dtype, (700,), True)
    ds = ds.cuda()
    def run():
        O, S = pkg.linear_attention(cfg, q, k, v, ld, ds, S0=S0, S_final=True)
        return [O, S, *pkg.linear_attention_backward(cfg, q, k, v, ld, ds, O, S0=S0, gS_final=S).values()]
else:
    cfg, H, W, t = xent_case(300, 1000, 128, dtype)
    g1 = torch.full((300,), 1 / 300).cuda()
    def run():
        loss, lse = pkg.cross_entropy(cfg, H, W, t)
        return [loss, lse, *pkg.cross_entropy_backward(cfg, H, W, t, lse, g1).values()]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = run()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, run()))
assert pkg.get_status() == 0
print("first call captured")
"""


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["qk", "attention", "loss"])
def test_a_process_captures_its_first_call(what, dtype):
    env = dict(os.environ, PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", FIRST, what, dtype], capture_output=True, text=True, timeout=300, env=env, cwd=ROOT)
    assert r.returncode == 0 and "first call captured" in r.stdout, r.stdout + r.stderr[-2000:]


def test_calls_from_several_host_threads():
    qk = qk_case(2, 300, 4, 2, 128, 128, "bf16")
    cfg, q, k, v, ld, S0, ds = attn_case(1, 4000, 4, 2, 128, 64, "bf16", (1000,), True)
    ds = ds.cuda()
    xc, H, W, t = xent_case(500, 3000, 256, "bf16")
    g1 = torch.full((500,), 1 / 500).cuda()

    def work(stream=None):
        y = pkg.qk_norm_rope(*qk, stream=stream)
        O, S = pkg.linear_attention(cfg, q, k, v, ld, ds, S0=S0, S_final=True, stream=stream)
        g = pkg.linear_attention_backward(cfg, q, k, v, ld, ds, O, S0=S0, gS_final=S, stream=stream)
        loss, lse = pkg.cross_entropy(xc, H, W, t, stream=stream)
        h = pkg.cross_entropy_backward(xc, H, W, t, lse, g1, stream=stream)
        return [*y, O, S, *g.values(), loss, lse, *h.values()]

    want = work()
    torch.cuda.synchronize()
    got, errors = {}, []

    def thread(i):
        try:
            s = torch.cuda.Stream()
            got[i] = [work(s) for _ in range(4)]
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(4)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not errors, errors
    for outs in got.values():
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(want, out))
    assert len(got) == 4 and status() == 0


def test_document_starts_beyond_32_bits_are_reported():
    cfg, q, k, v, ld, _, _ = attn_case(1, 40, 1, 1, 64, 64, "bf16")
    for device in ("cpu", "cuda"):
        for bad in (2 ** 32 + 5, -2 ** 32 + 5):  # 5, if only the lower half were read
            pkg.linear_attention(cfg, q, k, v, ld, torch.tensor([bad], dtype=torch.int64, device=device))
            assert status() == 1
        want = pkg.linear_attention(cfg, q, k, v, ld, [5])
        assert torch.equal(pkg.linear_attention(cfg, q, k, v, ld, torch.tensor([5], device=device)), want)
    assert status() == 0


def test_document_starts_of_other_types_are_refused():
    cfg, q, k, v, ld, _, _ = attn_case(1, 40, 1, 1, 64, 64, "bf16")
    for bad in (torch.tensor([5.0]), torch.tensor([True])):
        with pytest.raises(ValueError, match="doc_starts"):
            pkg.linear_attention(cfg, q, k, v, ld, bad)

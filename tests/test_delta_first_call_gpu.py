"""The first call of a process may be a captured one: nothing is loaded, set or looked up that a capture forbids."""

import subprocess
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu

PROGRAM = """
import torch, gated_delta_rule_56_gb300 as kda
dtype, what = getattr(torch, "{dtype}"), "{what}"
r = lambda *s: torch.randn(*s, device="cuda")
q, k = (torch.nn.functional.normalize(r(1, 200, 2, 128), dim=-1).to(dtype) for _ in range(2))
v, g, b = r(1, 200, 4, 128).to(dtype), -torch.rand(1, 200, 4, device="cuda"), torch.rand(1, 200, 4, device="cuda")
state = torch.zeros(200, 4, 128, 128, device="cuda")
call = dict(prompt=lambda: kda.delta_prefill(q, k, v, g, b), gradients=lambda: kda.delta_backward(q, k, v, g, b, v),
            token=lambda: kda.delta_decode_step(q[0], k[0], v[0], g[0], b[0], state), norm=lambda: kda.layer_norm(v, gate=v),
            norm_gradients=lambda: kda.layer_norm_backward(v, None, v, gate=v))[what]
flat = lambda x: [x] if isinstance(x, torch.Tensor) else [t for y in (x.values() if isinstance(x, dict) else x) if y is not None for t in flat(y)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = flat(call())
graph.replay()
captured = [t.clone() for t in captured]
state.zero_()
assert all(torch.equal(x, y) for x, y in zip(captured, flat(call()), strict=True))
kda.check_status()
print("same")
"""


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("what", ["prompt", "gradients", "token", "norm", "norm_gradients"])
def test_a_first_call_can_be_captured(dtype, what):
    p = subprocess.run([sys.executable, "-c", PROGRAM.format(dtype=dtype, what=what)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and p.stdout.strip() == "same", p.stderr

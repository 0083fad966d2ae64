"""add_norm's logistic function of gates over their whole range, against 64 bits.

1 / (1 + exp(-g)) in binary32 is off by the exponential's error, 2 + 1.173 |g| units in the last place, and a few of the
sum, the quotient and the products; below 2^-126, where binary32 is subnormal, by half of 2^-149 and as much again for each
of the two operations."""
import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["token", "channel", "value"])
@pytest.mark.parametrize("gate_type", [torch.float32, torch.bfloat16])
def test_gates_of_any_size(kind, gate_type):
    require_gpu()
    from moe_nvfp4_gemv_gb300 import fp4gemv
    gates = torch.cat([torch.arange(-104.0, 105.0, 0.25), torch.tensor([-3e38, 3e38, -1e4])]).to(gate_type).cuda()
    n = len(gates)
    big = torch.tensor([2.0 ** 126, -1.0, 3.0], dtype=torch.bfloat16, device="cuda")
    if kind == "token":
        y, gate = big.expand(n, 3).contiguous(), gates[:, None].contiguous()
    elif kind == "channel":
        y, gate = big[:, None].expand(3, n).contiguous(), gates
    else:
        y, gate = big[:, None].expand(3, n).contiguous(), gates.expand(3, n).contiguous()
    x = torch.zeros(y.shape, dtype=torch.float32, device="cuda")
    _, r = fp4gemv.add_norm(x, y, torch.ones(y.shape[1], dtype=torch.bfloat16, device="cuda"), gate=gate, gate_sigmoid=True)
    g = (gate if kind != "channel" else gate.expand(3, n)).double()
    want = y.double() * torch.sigmoid(g)
    tol = want.abs() * (8 + 1.2 * g.abs()) * 2.0 ** -23 + y.double().abs() * 2.0 ** -148
    off = (r.double() - want).abs() > tol
    assert not off.any(), (g.expand_as(want)[off][:5], r[off][:5], want[off][:5])

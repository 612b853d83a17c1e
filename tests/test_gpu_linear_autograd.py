"""Training through the linear attention calls, as their documentation says: the two sides of a
torch.autograd.Function, against torch's own differentiation of the 64-bit recurrence."""
import pytest
import torch

import linear_reference as ref
from gated_delta_rule_90_b200 import binding
from linear_bounds import DECAYS, STATE, out_bound
from test_gpu_linear import F32, PATHS, d64, inputs, rel

pytestmark = pytest.mark.gpu


class Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, S0, path):
        ctx.save_for_backward(q, k, v, g, S0)
        ctx.path = path
        return binding.gdr_fwd_linear(q, k, v, g, S0, path=path)

    @staticmethod
    def backward(ctx, dout, dS):
        return *binding.gdr_bwd_linear(*ctx.saved_tensors[:4], dout.contiguous(), ctx.saved_tensors[4],
                                       dS.contiguous(), path=ctx.path), None


@pytest.mark.parametrize("path,dtype", PATHS)
@pytest.mark.parametrize("side", [False, True])
def test_two_layers(cuda_device, path, dtype, side):
    """Two calls in a row, the second's state from the first and its inputs through elementwise work, on the
    current stream and on another one.  Each of the four calls adds its own error to what passes through it."""
    x = inputs(cuda_device, 61, 2, 200, 4, 2, 64, 64, dtype)
    leaves = [x[n].clone().requires_grad_() for n in ("q", "k", "v", "g", "S0")]
    plain = [t.detach().double().requires_grad_() for t in leaves]

    def loss(call, q, k, v, g, S0, dout, dS):
        o1, S1 = call(q, k, v, g, S0)
        o2, S2 = call(k, q, o1, 0.5 * g, S1)
        return (o2 * dout).sum() + (S2 * dS).sum() + (o1 * dout).sum()

    s = torch.cuda.Stream() if side else torch.cuda.current_stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        loss(lambda *a: Linear.apply(*a, path), *leaves, x["dout"], x["dS"]).backward()
    torch.cuda.current_stream().wait_stream(s)
    assert binding.device_status() == binding.GDR_OK
    loss(ref.forward, *plain, *d64(x["dout"], x["dS"])).backward()
    for name, a, b in zip(("q", "k", "v", "g", "S0"), leaves, plain):
        assert a.grad.dtype == a.dtype and a.grad.shape == a.shape
        tol = 4 * out_bound(dtype == F32, path) + (DECAYS if name == "g" else STATE)
        assert rel(a.grad, b.grad) <= tol, (name, rel(a.grad, b.grad))


def test_results_do_not_require_gradients(cuda_device):
    x = inputs(cuda_device, 62, 1, 20, 2, 2, 32, 32, F32)
    out, S = binding.gdr_fwd_linear(*(x[n].requires_grad_() for n in ("q", "k", "v", "g", "S0")))
    assert not out.requires_grad and not S.requires_grad

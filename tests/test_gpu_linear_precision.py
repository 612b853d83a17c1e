"""The precision that the linear attention calls state, on the GPU against the
64-bit token recurrence, with the bounds of linear_bounds.py."""
import pytest
import torch

import linear_reference as ref
from linear_bounds import DECAYS, STATE, out_bound
from test_gpu_linear import BF, F32, PATHS, bwd, d64, fwd, inputs, rel

pytestmark = pytest.mark.gpu

# B, T, H, Hk, dk, dv, gate, cu
SHAPES = [(1, 200, 2, 2, 64, 64, "token", None), (1, 640, 6, 2, 128, 128, "token", None),
          (2, 333, 8, 8, 128, 64, "head", None), (1, 2500, 1, 1, 64, 128, "token", None),
          (1, 2048, 2, 1, 128, 96, "token", [0, 700, 2000, 2048])]


@pytest.mark.parametrize("path,dtype", PATHS)
@pytest.mark.parametrize("B,T,H,Hk,dk,dv,gate,cu", SHAPES)
def test_outputs_and_states(cuda_device, path, dtype, B, T, H, Hk, dk, dv, gate, cu):
    x = inputs(cuda_device, 31, B, T, H, Hk, dk, dv, dtype, gate, cu)
    out, S = fwd(x, path=path)
    r, Sr = ref.forward(*d64(x["q"], x["k"], x["v"], x["g"], x["S0"]), cu=cu)
    assert rel(out, r) <= out_bound(dtype == F32, path)
    assert rel(S, Sr) <= STATE


@pytest.mark.parametrize("path,dtype", PATHS)
@pytest.mark.parametrize("B,T,H,Hk,dk,dv,gate,cu", SHAPES)
def test_gradients(cuda_device, path, dtype, B, T, H, Hk, dk, dv, gate, cu):
    x = inputs(cuda_device, 32, B, T, H, Hk, dk, dv, dtype, gate, cu)
    got = dict(zip(("dq", "dk", "dv", "dg", "dS0"), bwd(x, path=path)))
    want = ref.gradients(*d64(x["q"], x["k"], x["v"], x["g"], x["dout"], x["S0"], x["dS"]), cu=cu)
    for (name, a), b in zip(got.items(), want):
        tol = {"dg": DECAYS, "dS0": STATE}.get(name, out_bound(dtype == F32, path))
        if name == "dg" and gate == "head":  # a sum over all tokens, with signs: its terms' size counts
            each = ref.gradients(*d64(x["q"], x["k"], x["v"]), x["g"].double().expand(B, T, H).contiguous(),
                                 *d64(x["dout"], x["S0"], x["dS"]), cu=cu)[3]
            assert float((a.double() - b).norm()) <= tol * float(each.norm()) * (B * T) ** 0.5, name
        else:
            assert rel(a, b) <= tol, (name, rel(a, b))


@pytest.mark.parametrize("path,dtype", PATHS)
@pytest.mark.parametrize("kind", ["every 4th", "three at a block's start", "one of -20 in a block"])
def test_decays_after_a_strong_one(cuda_device, path, dtype, kind):
    """The gradient of ordinary decays in a block of 32 tokens that also has strong ones: as exact as
    without them.  One chunk of 128 tokens, so sums of up to 128 differences, a memory of at least two
    tokens between resets: 8 x 2^-22 (see linear_bounds), held to four times that."""
    x = inputs(cuda_device, 33, 2, 128, 4, 4, 64, 64, dtype, "token")
    t = torch.arange(128, device=cuda_device)
    at, to = {"every 4th": (t % 4 == 1, float("-inf")), "three at a block's start": (t % 32 < 3, float("-inf")),
              "one of -20 in a block": (t % 32 == 1, -20.0)}[kind]
    x["g"][:, at] = to
    got = bwd(x, path=path)[3].double()
    g64 = x["g"].double().clamp(min=-800)  # e^-800 is 0 in 64 bits; -inf has no gradient there
    want = ref.gradients(*d64(x["q"], x["k"], x["v"]), g64, *d64(x["dout"], x["S0"], x["dS"]))[3]
    assert float((got - want).norm()) <= 2.0 ** -17 * float(want.norm())

"""CPU checks of the linear attention entry points: the host refuses bad
arguments before any launch, the workspace sizes, and the test's own 64-bit
gradients against differences of its forward."""
import ctypes

import pytest
import torch

import linear_reference as ref
from gated_delta_rule_90_b200 import binding

nogpu = pytest.mark.skipif(torch.cuda.is_available(), reason="host-validation tests use fake pointers")
P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
BASE = dict(q=P, k=P, v=P, g=P, S0=None, out=P, S_final=None, dout=P, dS=None, dq=P, dk=P, dv=P,
            dg=P, dS0=None, S=P, B=2, T=64, N=3, H=4, Hk=2, d_k=64, d_v=64, cu=None, n_seq=0, dtype=1,
            gate=0, path=0, ws=P, wsb=1 << 40, stream=None)


def fwd(**kw):
    a = dict(BASE, **kw)
    return binding.lib().gdr_fwd_linear(
        a["q"], a["k"], a["v"], a["g"], a["S0"], a["out"], a["S_final"], a["B"], a["T"], a["H"],
        a["Hk"], a["d_k"], a["d_v"], a["cu"], a["n_seq"], a["dtype"], a["gate"], a["path"], a["ws"],
        a["wsb"], a["stream"])


def bwd(**kw):
    a = dict(BASE, **kw)
    return binding.lib().gdr_bwd_linear(
        a["q"], a["k"], a["v"], a["g"], a["S0"], a["dout"], a["dS"], a["dq"], a["dk"], a["dv"],
        a["dg"], a["dS0"], a["B"], a["T"], a["H"], a["Hk"], a["d_k"], a["d_v"], a["cu"], a["n_seq"],
        a["dtype"], a["gate"], a["path"], a["ws"], a["wsb"], a["stream"])


def decode(**kw):
    a = dict(BASE, **kw)
    return binding.lib().gdr_decode_step_linear(a["q"], a["k"], a["v"], a["g"], a["S"], a["out"],
                                                a["N"], a["H"], a["Hk"], a["d_k"], a["d_v"],
                                                a["dtype"], a["gate"], a["stream"])


COMMON = [(dict(q=None), 1), (dict(v=None), 1), (dict(g=None), 1), (dict(H=0), 1), (dict(Hk=0), 1),
          (dict(H=4, Hk=3), 1), (dict(Hk=8), 1), (dict(dtype=2), 1), (dict(gate=3), 1),
          (dict(gate=-1), 1), (dict(k=ODD), 1), (dict(g=ODD), 1), (dict(gate=1), 2),
          (dict(d_k=24), 2), (dict(d_v=144), 2), (dict(d_k=0), 1), (dict(H=65536, Hk=1), 2)]
WHOLE = [(dict(B=0), 1), (dict(T=-1), 1), (dict(path=3), 1), (dict(cu=P, B=2, n_seq=2), 1),
         (dict(cu=P, B=1, n_seq=0), 1), (dict(ws=None, wsb=0), 1), (dict(wsb=16), 1),
         (dict(ws=ctypes.c_void_p(0x10010)), 1), (dict(S0=ODD), 1), (dict(path=2, dtype=0), 2),
         (dict(B=1 << 16, T=1 << 16), 1)]


@nogpu
@pytest.mark.parametrize("kw,expect", COMMON + WHOLE + [(dict(out=None), 1), (dict(S_final=ODD), 1)])
def test_fwd_linear_rejects_on_host(kw, expect):
    assert fwd(**kw) == expect


@nogpu
@pytest.mark.parametrize("kw,expect", COMMON + WHOLE + [
    (dict(dout=None), 1), (dict(dq=None), 1), (dict(dg=None), 1), (dict(dS=ODD), 1),
    (dict(dS0=ODD), 1), (dict(dv=ODD), 1)])
def test_bwd_linear_rejects_on_host(kw, expect):
    assert bwd(**kw) == expect


@nogpu
@pytest.mark.parametrize("kw,expect", COMMON + [(dict(N=0), 1), (dict(S=None), 1), (dict(S=ODD), 1),
                                                (dict(out=None), 1)])
def test_decode_step_linear_rejects_on_host(kw, expect):
    assert decode(**kw) == expect


def test_workspace_sizes():
    a = (2, 1000, 8, 4, 64, 128, 0, False)
    for size in (binding.fwd_linear_workspace_size, binding.bwd_linear_workspace_size):
        assert size(*a, binding.GDR_BF16, binding.GDR_GATE_SCALAR) > 0
        assert size(*a, binding.GDR_F32, binding.GDR_GATE_HEAD, "simt") > 0
        assert size(*a, binding.GDR_F32, binding.GDR_GATE_SCALAR, "tc") == 0
        assert size(2, 1000, 8, 3, 64, 128, 0, False, 1, 0) == 0   # refused: 8 heads, 3 shared
        assert size(2, 1000, 8, 4, 64, 128, 0, False, 1, 1) == 0   # refused: per-channel decay
        # linear in the heads, whatever the path
        assert size(1, 640, 16, 16, 64, 64, 0, False, 0, 0) >= size(1, 640, 8, 8, 64, 64, 0, False, 0, 0)


def test_binding_rejects_host_tensors():
    q = torch.zeros(1, 4, 2, 16)
    g = torch.zeros(1, 4, 2)
    with pytest.raises(ValueError, match="CUDA"):
        binding.gdr_fwd_linear(q, q, q, g)
    with pytest.raises(ValueError, match="CUDA"):
        binding.gdr_bwd_linear(q, q, q, g, q)
    with pytest.raises(ValueError, match="CUDA"):
        binding.gdr_decode_step_linear(q[0], q[0], q[0], g[0], torch.zeros(4, 2, 16, 16))


def test_reference_gradients_against_differences():
    """The tests' own gradients (of the recurrence, by differentiation) against
    central differences of its forward: step 1e-5, error O(step^2) + 2^-52 / step."""
    gen = torch.Generator().manual_seed(7)
    cu = [0, 3, 3, 7]

    def rand(*s):
        return torch.randn(*s, generator=gen, dtype=torch.float64)

    x = [rand(1, 7, 1, 3), rand(1, 7, 1, 3), rand(1, 7, 2, 2), -rand(1, 7, 2).abs(), rand(3, 2, 2, 3)]
    dout, dS = rand(1, 7, 2, 2), rand(3, 2, 2, 3)

    def loss(y):
        out, S = ref.forward(*y, cu=cu)
        return float((out * dout).sum() + (S * dS).sum())

    got = ref.gradients(x[0], x[1], x[2], x[3], dout, x[4], dS, cu)
    step = 1e-5
    for i, (t, d) in enumerate(zip(x, got)):
        for j in range(t.numel()):
            up, dn = [y.clone() for y in x], [y.clone() for y in x]
            up[i].view(-1)[j] += step
            dn[i].view(-1)[j] -= step
            assert abs((loss(up) - loss(dn)) / (2 * step) - float(d.reshape(-1)[j])) < 1e-7

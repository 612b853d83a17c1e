"""CPU checks of what the linear attention calls hand to the library: tensors
that pass for CUDA ones, and a library that records its arguments instead of
launching."""
import pytest
import torch

from gated_delta_rule_90_b200 import binding

F32 = torch.float32


class OnGpu(torch.Tensor):
    """A host tensor that says it is on cuda:0."""
    __torch_function__ = torch._C._disabled_torch_function_impl
    device = property(lambda self: torch.device("cuda:0"))
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return binding.GDR_OK
        return call


@pytest.fixture
def library(monkeypatch):
    rec = Library()
    monkeypatch.setattr(binding, "lib", lambda: rec)
    monkeypatch.setattr(binding, "fwd_linear_workspace_size", lambda *a: 256)
    monkeypatch.setattr(binding, "bwd_linear_workspace_size", lambda *a: 256)
    monkeypatch.setattr(binding, "_linear_call", lambda dev, stream, n, ws, call: call(0, n, 0))
    return rec


def made(*shape):
    return torch.zeros(*shape, dtype=F32).as_subclass(OnGpu)


def tensors(lead, H=4, Hk=2, dk=32, dv=16):
    return made(*lead, Hk, dk), made(*lead, Hk, dk), made(*lead, H, dv), made(*lead, H)


def states(n, H=4, dk=32, dv=16):
    return made(n, H, dv, dk)


def fwd(lead, n):
    q, k, v, g = tensors(lead)
    return binding.gdr_fwd_linear(q, k, v, g, out=made(*v.shape), S_final=states(n))


def bwd(lead, n):
    q, k, v, g = tensors(lead)
    return binding.gdr_bwd_linear(q, k, v, g, made(*v.shape), dq=made(*q.shape), dk=made(*q.shape),
                                  dv=made(*v.shape), dg=made(*g.shape), dS0=states(n))


def decode(lead, n):
    q, k, v, g = tensors(lead)
    return binding.gdr_decode_step_linear(q, k, v, g, states(n), out=made(*v.shape), stream=0)


@pytest.mark.parametrize("call,lead,at,counts", [
    (fwd, (3, 8), 7, (3, 8, 4, 2, 32, 16)), (bwd, (3, 8), 12, (3, 8, 4, 2, 32, 16)),
    (decode, (3,), 6, (3, 4, 2, 32, 16))])
def test_counts_that_reach_the_library(library, call, lead, at, counts):
    call(lead, 3)
    (_, args), = library.calls
    assert args[at:at + len(counts)] == counts


@pytest.mark.parametrize("call,lead", [
    (fwd, (8,)), (fwd, (3, 8, 2)), (fwd, ()), (bwd, (8,)), (bwd, (3, 8, 2)), (bwd, ()),
    (decode, ()), (decode, (3, 8)), (decode, (3, 1))])
def test_tensors_of_another_rank_are_refused(library, call, lead):
    """Unbatched tensors, a further axis, decode tensors with a token axis: each agrees with the
    others in shape, and the library would read its counts from the wrong axes."""
    with pytest.raises(ValueError, match="axes"):
        call(lead, lead[0] if lead else 1)
    assert not library.calls


@pytest.mark.parametrize("name", ["k", "v", "g"])
@pytest.mark.parametrize("call", [binding.gdr_fwd_linear, binding.gdr_decode_step_linear])
def test_one_tensor_of_another_rank_is_refused(library, call, name):
    lead = (3, 8) if call is binding.gdr_fwd_linear else (3,)
    x = dict(zip("qkvg", tensors(lead)))
    x[name] = x[name].reshape(1, *x[name].shape)
    with pytest.raises(ValueError):
        call(x["q"], x["k"], x["v"], x["g"], states(3))
    assert not library.calls


@pytest.mark.parametrize("H,Hk,dk,dv", [(16, 16, 128, 128), (32, 8, 128, 64), (4, 4, 64, 64), (2, 1, 48, 112)])
@pytest.mark.parametrize("T", [2048, 65536, 131072])
def test_workspace_of_packed_gradients_is_linear_in_the_sequences(H, Hk, dk, dv, T):
    """A further sequence adds at most its own part: for each head the states of its block, forward
    and backward, and its last state (fp32, d_v x d_k), the state at one run's start (128 x 64 fp32
    for each 64 columns of d_k) with 8 partial products, a few words of its plan, and the rounding
    of the arrays to 256 bytes."""
    groups = -(-dk // 64)
    a = H * (3 * dk * dv * 4 + groups * (128 * 64 * 4 + 8 * 4) + 64) + 64

    def size(n):
        return binding.bwd_linear_workspace_size(1, T, H, Hk, dk, dv, n, True, binding.GDR_BF16,
                                                 binding.GDR_GATE_HEAD, "tc")

    base = size(1)
    for n in (2, 16, 256, 2000):
        assert base < size(n) <= base + (n - 1) * a + 20 * 256


@pytest.mark.parametrize("dtype", [binding.GDR_F32, binding.GDR_BF16])
@pytest.mark.parametrize("gate", [binding.GDR_GATE_SCALAR, binding.GDR_GATE_HEAD])
@pytest.mark.parametrize("varlen", [False, True])
def test_a_call_without_tokens_has_a_workspace_size(dtype, gate, varlen):
    """0 stands for a refused call; a call of no tokens is a valid one."""
    a = (1 if varlen else 2, 0, 3, 1, 32, 16, 2, varlen, dtype, gate)
    assert binding.fwd_linear_workspace_size(*a) > 0
    assert binding.bwd_linear_workspace_size(*a) > 0


@pytest.mark.parametrize("dtype,path,block", [(binding.GDR_F32, "simt", 32), (binding.GDR_BF16, "simt", 32),
                                              (binding.GDR_BF16, "tc", 128)])
@pytest.mark.parametrize("B,T,H,Hk", [(1, 640, 16, 8), (2, 4096, 16, 16), (4, 1000, 64, 4), (1, 65536, 32, 32)])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (16, 48)])
def test_workspace_of_equal_sequences_is_bounded(dtype, path, block, B, T, H, Hk, dk, dv):
    """At the shortest blocks: a state for each block and head; of the gradients two, with the state
    (128 x 64 for each 64 columns) and 8 products at a run's start, the last states, four fp32 rows of
    partial sums for dq and for dk each and two more of the pairs, and fp32 dq and dk where value heads
    share them; words for each block, and 16 roundings to 256 bytes."""
    blocks, rows, nel, groups = B * -(-T // block) * H, B * T * H, dk * dv, -(-dk // 64)
    a = (B, T, H, Hk, dk, dv, 0, False, dtype, binding.GDR_GATE_SCALAR, path)
    assert 0 < binding.fwd_linear_workspace_size(*a) <= blocks * (4 * nel + 16) + 16 * 256
    most = blocks * (8 * nel + groups * (128 * 64 * 4 + 32) + 16) + B * H * nel * 4 + rows * (2 * 16 + 16)
    most += rows * dk * 8 if Hk < H else 0
    assert 0 < binding.bwd_linear_workspace_size(*a) <= most + 16 * 256

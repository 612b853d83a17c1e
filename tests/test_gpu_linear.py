"""Linear attention with a decay for each head on the GPU, against the 64-bit
token recurrence (linear_reference).

Tolerances are relative 2-norms of an output.  A value stored in bf16 is off by
at most half a step, 2^-8 of itself; the tensor-core path also rounds two
operands of each product to bf16 (the pair weights or the scaled state), 2^-8
each, so its bf16 outputs are held to 3 x 2^-8 and those of the CUDA cores to
2^-8 plus the fp32 sums.  fp32 sums of n terms are off by at most n 2^-24 of
the terms' sizes: with up to 128 + 256 terms, and rounding errors that mostly
cancel, fp32 outputs are held to 384 x 2^-24 = 2.3e-5 (dg, a sum of such sums
over up to 256 tokens with signs, to twice that)."""
import pytest
import torch

import linear_reference as ref
from gated_delta_rule_90_b200 import binding

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TOL32 = 384 * 2.0 ** -24


def tol_out(dtype, path):
    return TOL32 if dtype == F32 else (2.0 ** -8 if path == "simt" else 3 * 2.0 ** -8) + TOL32


def rel(x, r):
    x, r = x.double(), r.double()
    d = float(r.norm())
    return float((x - r).norm()) / d if d > 0 else float(x.norm())


def inputs(dev, seed, B, T, H, Hk, dk, dv, dtype=BF, gate="token", cu=None, s0=True, scale=0.1):
    gen = torch.Generator(device=dev).manual_seed(seed)

    def rand(*s):
        return torch.randn(*s, generator=gen, device=dev)

    n = B if cu is None else len(cu) - 1
    x = dict(q=torch.nn.functional.normalize(rand(B, T, Hk, dk), dim=-1).to(dtype),
             k=torch.nn.functional.normalize(rand(B, T, Hk, dk), dim=-1).to(dtype),
             v=rand(B, T, H, dv).to(dtype),
             g=-scale * torch.nn.functional.softplus(rand(H) if gate == "head" else rand(B, T, H)))
    x["S0"] = 0.3 * rand(n, H, dv, dk) if s0 else None
    x["dout"] = rand(B, T, H, dv).to(dtype)
    x["dS"] = 0.3 * rand(n, H, dv, dk) if s0 else None
    x["cu"] = cu
    return x


def cu_of(x):
    return None if x["cu"] is None else torch.tensor(x["cu"], dtype=torch.int32, device=x["q"].device)


def fwd(x, **kw):
    r = binding.gdr_fwd_linear(x["q"], x["k"], x["v"], x["g"], x["S0"], cu_seqlens=cu_of(x), **kw)
    assert binding.device_status() == binding.GDR_OK
    return r


def bwd(x, **kw):
    r = binding.gdr_bwd_linear(x["q"], x["k"], x["v"], x["g"], x["dout"], x["S0"], x["dS"],
                               cu_seqlens=cu_of(x), **kw)
    assert binding.device_status() == binding.GDR_OK
    return r


def d64(*ts):
    return [None if t is None else t.double() for t in ts]


PATHS = [("simt", F32), ("simt", BF), ("tc", BF)]
# B, T, H, Hk, dk, dv, gate, S0
SHAPES = [(1, 1, 1, 1, 16, 16, "token", True), (2, 37, 4, 2, 64, 64, "token", True),
          (1, 128, 2, 2, 128, 128, "head", False), (1, 129, 3, 1, 128, 64, "token", True),
          (3, 300, 2, 2, 48, 96, "token", False), (1, 513, 4, 1, 64, 128, "head", True),
          (1, 257, 2, 2, 112, 80, "token", True)]


@pytest.mark.parametrize("path,dtype", PATHS)
@pytest.mark.parametrize("shape", SHAPES)
def test_fwd_matches_the_recurrence(cuda_device, path, dtype, shape):
    B, T, H, Hk, dk, dv, gate, s0 = shape
    x = inputs(cuda_device, 1, B, T, H, Hk, dk, dv, dtype, gate, None, s0)
    out, S = fwd(x, path=path)
    r, Sr = ref.forward(*d64(x["q"], x["k"], x["v"], x["g"], x["S0"]))
    assert out.dtype == dtype and S.dtype == F32
    assert rel(out, r) <= tol_out(dtype, path)
    assert rel(S, Sr) <= TOL32


@pytest.mark.parametrize("path,dtype", PATHS)
@pytest.mark.parametrize("shape", SHAPES)
def test_bwd_matches_the_gradient(cuda_device, path, dtype, shape):
    B, T, H, Hk, dk, dv, gate, s0 = shape
    x = inputs(cuda_device, 2, B, T, H, Hk, dk, dv, dtype, gate, None, s0)
    got = bwd(x, path=path)
    want = ref.gradients(*d64(x["q"], x["k"], x["v"], x["g"], x["dout"], x["S0"], x["dS"]))
    for name, a, b in zip(("dq", "dk", "dv", "dg", "dS0"), got, want):
        tol = tol_out(dtype, path) if name in ("dq", "dk", "dv") else 2 * TOL32
        assert a.shape == b.shape and rel(a, b) <= tol, (name, rel(a, b))


@pytest.mark.parametrize("path,dtype", PATHS)
@pytest.mark.parametrize("cu", [[0, 0, 1, 130, 130, 258, 300], [0, 300], [0, 128, 256, 300],
                                [0, 299, 300, 300]])
def test_packed_sequences(cuda_device, path, dtype, cu):
    x = inputs(cuda_device, 3, 1, 300, 4, 2, 64, 48, dtype, "token", cu)
    out, S = fwd(x, path=path)
    r, Sr = ref.forward(*d64(x["q"], x["k"], x["v"], x["g"], x["S0"]), cu=cu)
    assert rel(out, r) <= tol_out(dtype, path)
    for s in range(len(cu) - 1):
        assert rel(S[s], Sr[s]) <= TOL32
    got = bwd(x, path=path)
    want = ref.gradients(*d64(x["q"], x["k"], x["v"], x["g"], x["dout"], x["S0"], x["dS"]), cu=cu)
    for name, a, b in zip(("dq", "dk", "dv", "dg", "dS0"), got, want):
        tol = tol_out(dtype, path) if name in ("dq", "dk", "dv") else 2 * TOL32
        assert rel(a, b) <= tol, (name, rel(a, b))


@pytest.mark.parametrize("path,dtype", PATHS)
def test_rows_of_no_sequence_are_left(cuda_device, path, dtype):
    cu = [5, 140, 190]  # rows 0..4 and 190..199 belong to nobody
    x = inputs(cuda_device, 4, 1, 200, 2, 1, 64, 64, dtype, "token", cu)
    out = torch.full_like(x["v"], 7.0)
    fwd(x, path=path, out=out)
    dq, dv = torch.full_like(x["q"], 7.0), torch.full_like(x["v"], 7.0)
    dg = torch.full_like(x["g"], 7.0)
    bwd(x, path=path, dq=dq, dk=dq.clone(), dv=dv, dg=dg)
    for t in (out, dq, dv, dg):
        assert (t[0, :5] == 7).all() and (t[0, 190:] == 7).all()
        assert not (t[0, 5:190] == 7).all(-1).any()


@pytest.mark.parametrize("path,dtype", PATHS)
def test_bad_values_stay_in_their_sequence(cuda_device, path, dtype):
    """NaN and infinities of one sequence reach no other, nor do those of rows of no sequence."""
    cu = [0, 100, 161, 300]
    x = inputs(cuda_device, 5, 1, 310, 2, 2, 64, 64, dtype, "token", cu)
    clean = fwd(x, path=path), bwd(x, path=path)
    y = {k: (t.clone() if torch.is_tensor(t) else t) for k, t in x.items()}
    for name in ("q", "k", "v", "dout"):
        y[name][0, 100:161] = float("nan")
        y[name][0, 300:] = float("inf")
    y["g"][0, 300:] = float("nan")
    dirty = fwd(y, path=path), bwd(y, path=path)
    keep = [t for t in range(300) if not 100 <= t < 161]
    assert torch.equal(clean[0][0][0, keep], dirty[0][0][0, keep])
    assert torch.equal(clean[0][1][[0, 2]], dirty[0][1][[0, 2]])
    for a, b in zip(clean[1][:4], dirty[1][:4]):
        assert torch.equal(a[0, keep], b[0, keep])
    assert torch.equal(clean[1][4][[0, 2]], dirty[1][4][[0, 2]])


@pytest.mark.parametrize("path,dtype", PATHS)
@pytest.mark.parametrize("kind", ["none", "strong", "reset"])
def test_extreme_decays(cuda_device, path, dtype, kind):
    """No decay at all; decays that forget within a token; a log-decay of -inf, which restarts the state."""
    x = inputs(cuda_device, 6, 1, 290, 2, 2, 64, 64, dtype, "token", None)
    if kind == "none":
        x["g"].zero_()
    elif kind == "strong":
        x["g"].mul_(200.0)
    else:
        x["g"][0, 3] = x["g"][0, 131] = x["g"][0, 132, 1] = float("-inf")
    out, S = fwd(x, path=path)
    r, Sr = ref.forward(*d64(x["q"], x["k"], x["v"], x["g"], x["S0"]))
    assert rel(out, r) <= tol_out(dtype, path) and rel(S, Sr) <= TOL32
    got = bwd(x, path=path)
    g64 = x["g"].double().clamp(min=-800)  # e^-800 is 0 in 64 bits; -inf has no gradient there
    want = ref.gradients(*d64(x["q"], x["k"], x["v"]), g64, *d64(x["dout"], x["S0"], x["dS"]))
    for name, a, b in zip(("dq", "dk", "dv", "dS0"), got[:3] + got[4:], want[:3] + want[4:]):
        tol = tol_out(dtype, path) if name != "dS0" else 2 * TOL32
        assert rel(a, b) <= tol, (name, rel(a, b))
    # dg cancels between large terms where the decays are strong: held to the size of those terms
    size = float((x["q"].double() * want[0]).sum(-1).abs().max())
    assert float((got[3].double() - want[3]).abs().max()) <= 2 * TOL32 * max(size, float(want[3].abs().max()))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,H,Hk,dk,dv,gate", [
    (1, 16, 16, 128, 128, "token"), (5, 6, 2, 64, 128, "head"), (3, 4, 1, 48, 80, "token"),
    (2, 3, 3, 16, 16, "token"), (4, 2, 2, 112, 96, "head"), (200, 4, 4, 80, 32, "token"),
    (2, 2, 1, 96, 112, "token"), (3, 2, 2, 32, 48, "token")])
def test_decode_step(cuda_device, dtype, N, H, Hk, dk, dv, gate):
    x = inputs(cuda_device, 7, N, 1, H, Hk, dk, dv, dtype, gate)
    S = x["S0"].clone()
    g = x["g"] if gate == "head" else x["g"][:, 0].contiguous()
    out = binding.gdr_decode_step_linear(x["q"][:, 0].contiguous(), x["k"][:, 0].contiguous(),
                                         x["v"][:, 0].contiguous(), g, S)
    r, Sr = ref.forward(*d64(x["q"], x["k"], x["v"], x["g"], x["S0"]))
    assert rel(out, r[:, 0]) <= tol_out(dtype, "simt") and rel(S, Sr) <= TOL32


@pytest.mark.parametrize("path,dtype", PATHS)
def test_prompt_then_tokens_then_gradient(cuda_device, path, dtype):
    """As they are used: a prompt in two pieces, single tokens after it, and the gradient of the whole."""
    T, n = 333, 9
    x = inputs(cuda_device, 8, 2, T + n, 4, 2, 64, 128, dtype)
    cut = lambda a, b: [x[s][:, a:b].contiguous() for s in ("q", "k", "v", "g")]  # noqa: E731
    o1, S = binding.gdr_fwd_linear(*cut(0, 150), x["S0"], path=path)
    o2, S = binding.gdr_fwd_linear(*cut(150, T), S, path=path, S_final=S)  # in place
    outs = [o1, o2]
    for t in range(T, T + n):
        outs.append(binding.gdr_decode_step_linear(*(y[:, 0].contiguous() for y in cut(t, t + 1)), S)[:, None])
    r, Sr = ref.forward(*d64(x["q"], x["k"], x["v"], x["g"], x["S0"]))
    assert rel(torch.cat(outs, 1), r) <= tol_out(dtype, path) and rel(S, Sr) <= TOL32
    # the gradient of the whole equals that of its two pieces, joined through the state
    whole = bwd(x, path=path)
    _, Sm = binding.gdr_fwd_linear(*cut(0, 150), x["S0"], path=path)
    do = x["dout"]
    late = binding.gdr_bwd_linear(*cut(150, T + n), do[:, 150:].contiguous(), Sm, x["dS"], path=path)
    early = binding.gdr_bwd_linear(*cut(0, 150), do[:, :150].contiguous(), x["S0"], late[4], path=path)
    for i, name in enumerate(("dq", "dk", "dv", "dg")):
        tol = 2 * tol_out(dtype, path) if name != "dg" else 4 * TOL32
        assert rel(torch.cat([early[i], late[i]], 1), whole[i]) <= tol, name
    assert rel(early[4], whole[4]) <= 2 * TOL32


@pytest.mark.parametrize("path,dtype", PATHS)
def test_runs_repeat_bit_for_bit(cuda_device, path, dtype):
    x = inputs(cuda_device, 9, 2, 700, 4, 2, 64, 64, dtype, "head")
    for call in (fwd, bwd):
        a, b = call(x, path=path), call(x, path=path)
        assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("path,dtype", PATHS)
def test_streams_and_graphs(cuda_device, path, dtype):
    """On a side stream, two calls at once with workspaces of their own, and captured and replayed with new inputs."""
    cu = [0, 77, 300, 401]
    x = inputs(cuda_device, 10, 1, 401, 2, 1, 64, 64, dtype, "token", cu)
    y = inputs(cuda_device, 11, 1, 401, 2, 1, 64, 64, dtype, "token", cu)
    c = cu_of(x)
    want = [(fwd(z, path=path), bwd(z, path=path)) for z in (x, y)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for z, s in zip((x, y), streams):
        got.append((binding.gdr_fwd_linear(z["q"], z["k"], z["v"], z["g"], z["S0"], cu_seqlens=c,
                                           path=path, stream=s),
                    binding.gdr_bwd_linear(z["q"], z["k"], z["v"], z["g"], z["dout"], z["S0"], z["dS"],
                                           cu_seqlens=c, path=path, stream=s)))
    torch.cuda.synchronize()
    for w, h in zip(want, got):
        assert all(torch.equal(p, q) for i in (0, 1) for p, q in zip(w[i], h[i]))
    z = {k: (t.clone() if torch.is_tensor(t) else t) for k, t in x.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = binding.gdr_fwd_linear(z["q"], z["k"], z["v"], z["g"], z["S0"], cu_seqlens=c, path=path)
        b = binding.gdr_bwd_linear(z["q"], z["k"], z["v"], z["g"], z["dout"], z["S0"], z["dS"],
                                   cu_seqlens=c, path=path)
    for src, w in ((y, want[1]), (x, want[0])):
        for name, t in z.items():
            if torch.is_tensor(t):
                t.copy_(src[name])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(w[0], f))
        assert all(torch.equal(p, q) for p, q in zip(w[1], b))


# one sequence long enough to be cut into blocks; a packed batch with an empty sequence, one token, and long ones
LONG = [(2500, 1, 1, 128, 128, "token", None), (2500, 2, 1, 64, 112, "head", None),
        (2600, 2, 1, 128, 48, "token", [0, 0, 1500, 1501, 2600]), (1800, 1, 1, 80, 128, "head", [0, 1537, 1800, 1800])]


@pytest.mark.parametrize("path,dtype", PATHS)
@pytest.mark.parametrize("T,H,Hk,dk,dv,gate,cu", LONG)
def test_long_sequences(cuda_device, path, dtype, T, H, Hk, dk, dv, gate, cu):
    x = inputs(cuda_device, 14, 1, T, H, Hk, dk, dv, dtype, gate, cu)
    out, S = fwd(x, path=path)
    r, Sr = ref.forward(*d64(x["q"], x["k"], x["v"], x["g"], x["S0"]), cu=cu)
    assert rel(out, r) <= tol_out(dtype, path) and rel(S, Sr) <= TOL32
    got = bwd(x, path=path)
    want = ref.gradients(*d64(x["q"], x["k"], x["v"], x["g"], x["dout"], x["S0"], x["dS"]), cu=cu)
    for name, a, b in zip(("dq", "dk", "dv", "dg", "dS0"), got, want):
        tol = tol_out(dtype, path) if name in ("dq", "dk", "dv") else 2 * TOL32
        assert rel(a, b) <= tol, (name, rel(a, b))


@pytest.mark.parametrize("path,dtype", PATHS)
def test_outputs_at_16_byte_offsets(cuda_device, path, dtype):
    """Output and input views that start 16 bytes into their storage give the same bits."""
    x = inputs(cuda_device, 15, 1, 150, 2, 2, 48, 80, dtype)

    def shifted(t):
        n = 16 // t.element_size()
        v = torch.empty(t.numel() + n, dtype=t.dtype, device=t.device)[n:].view(t.shape)
        v.copy_(t)
        return v

    y = {k: (shifted(t) if torch.is_tensor(t) else t) for k, t in x.items()}
    out, S = fwd(x, path=path)
    o2, S2 = fwd(y, path=path, out=shifted(out), S_final=shifted(S))
    assert torch.equal(out, o2) and torch.equal(S, S2)
    a = bwd(x, path=path)
    b = bwd(y, path=path, **{n: shifted(t) for n, t in zip(("dq", "dk", "dv", "dg", "dS0"), a)})
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_gradient_against_differences(cuda_device):
    """The fp32 gradients against central differences of the fp32 forward along one direction: step 2^-6,
    error O(step^2) of third derivatives of size about 1, and 2 sums of n terms rounded at 2^-24 over the step."""
    x = inputs(cuda_device, 16, 1, 40, 2, 1, 32, 16, F32, scale=0.3)
    got = dict(zip(("q", "k", "v", "g", "S0"), bwd(x)))
    gen = torch.Generator(device=cuda_device).manual_seed(17)
    for name, d in got.items():
        u = torch.randn(x[name].shape, generator=gen, device=cuda_device)
        u /= u.norm()
        loss = []
        for sign in (1, -1):
            y = dict(x)
            y[name] = x[name] + sign * 2.0 ** -6 * u
            out, S = fwd(y)
            loss.append(float((out.double() * x["dout"].double()).sum() + (S.double() * x["dS"].double()).sum()))
        slope, want = (loss[0] - loss[1]) * 2.0 ** 5, float((d.double() * u.double()).sum())
        assert abs(slope - want) <= 1e-3 * float(d.norm()), name


@pytest.mark.parametrize("path,dtype", PATHS)
@pytest.mark.parametrize("T", [70, 1300])
def test_state_gradient_in_place(cuda_device, path, dtype, T):
    """dS0 written over dS_final: the same results."""
    x = inputs(cuda_device, 18, 1, T, 2, 1, 64, 48, dtype, "head")
    a = bwd(x, path=path)
    y = dict(x, dS=x["dS"].clone())
    b = bwd(y, path=path, dS0=y["dS"])
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_empty_calls(cuda_device):
    """No tokens: S_final is S0 (or zero), dS0 is dS_final."""
    dev = cuda_device
    e = lambda h, d: torch.empty(2, 0, h, d, device=dev)  # noqa: E731
    S0 = torch.randn(2, 3, 16, 32, device=dev)
    out, S = binding.gdr_fwd_linear(e(3, 32), e(3, 32), e(3, 16), torch.empty(2, 0, 3, device=dev), S0)
    assert out.shape == (2, 0, 3, 16) and torch.equal(S, S0)
    _, S = binding.gdr_fwd_linear(e(3, 32), e(3, 32), e(3, 16), torch.empty(2, 0, 3, device=dev))
    assert not S.any()
    g = torch.full((3,), -0.1, device=dev)
    got = binding.gdr_bwd_linear(e(3, 32), e(3, 32), e(3, 16), g, e(3, 16), S0, S0)
    assert torch.equal(got[4], S0) and not got[3].any()


@pytest.mark.parametrize("path,dtype", PATHS)
def test_inputs_written_just_before_the_call(cuda_device, path, dtype):
    """Kernels that end right before the calls, in the same stream or in one joined to it, write the
    inputs; the gradients' inputs follow the forward pass.  Eager and captured: bit for bit the calls
    on inputs that were ready."""
    cu = [0, 300, 301, 900]
    x, y = (inputs(cuda_device, 60 + i, 1, 900, 4, 2, 64, 64, dtype, "token", cu) for i in (0, 1))
    want = [[t.clone() for t in fwd(z, path=path) + bwd(z, path=path)] for z in (x, y)]
    ts = [n for n in x if isinstance(x[n], torch.Tensor) and n != "cu"]
    live, src = dict(x), {n: x[n].clone() for n in ts}
    for n in ts:
        live[n] = torch.zeros_like(x[n])
    c = torch.tensor(cu, dtype=torch.int32, device=cuda_device)
    side = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            for n in ("k", "g"):
                torch.mul(src[n], 1, out=live[n])
        for n in ("v", "S0", "q"):
            torch.mul(src[n], 1, out=live[n])
        here.wait_stream(side)
        o = binding.gdr_fwd_linear(live["q"], live["k"], live["v"], live["g"], live["S0"], cu_seqlens=c, path=path)
        for n in ("dS", "dout"):
            torch.mul(src[n], 1, out=live[n])
        return o + binding.gdr_bwd_linear(live["q"], live["k"], live["v"], live["g"], live["dout"], live["S0"],
                                          live["dS"], cu_seqlens=c, path=path)

    def load(z):
        for n in ts:
            src[n].copy_(z[n])
            live[n].zero_()
        torch.cuda.synchronize()

    for _ in range(10):
        for z, w in zip((x, y), want):
            load(z)
            assert all(torch.equal(a, b) for a, b in zip(step(), w))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(10):
        for z, w in zip((x, y), want):
            load(z)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, w))
    assert binding.device_status() == binding.GDR_OK


@pytest.mark.parametrize("path,dtype", PATHS)
def test_malformed_offsets_stay_in_bounds(cuda_device, path, dtype):
    """Offsets that decrease or leave [0, T] are taken as their running maximum inside [0, T]."""
    x = inputs(cuda_device, 12, 1, 90, 2, 2, 32, 32, dtype, "token", [0, 50, 20, 70, 500])
    y = dict(x, cu=[0, 50, 50, 70, 90])
    for call in (fwd, bwd):
        assert all(torch.equal(a, b) for a, b in zip(call(x, path=path), call(y, path=path)))


def test_refusals(cuda_device):
    x = inputs(cuda_device, 13, 1, 8, 4, 2, 32, 32, F32)
    q, k, v, g = x["q"], x["k"], x["v"], x["g"]
    with pytest.raises(ValueError, match="shape"):
        binding.gdr_fwd_linear(q, k[:, :4].contiguous(), v, g)
    with pytest.raises(ValueError, match="contiguous"):
        binding.gdr_fwd_linear(q, k, v.transpose(1, 2).contiguous().transpose(1, 2), g)
    with pytest.raises(TypeError, match="g must be"):
        binding.gdr_fwd_linear(q, k, v, g.double())
    with pytest.raises(ValueError, match="key channel"):
        binding.gdr_fwd_linear(q, k, v, torch.zeros(1, 8, 4, 32, device=q.device))
    with pytest.raises(ValueError, match="share"):
        binding.gdr_fwd_linear(q, k, v[:, :, :3].contiguous(), g[..., :3].contiguous())
    with pytest.raises(ValueError, match="shape"):
        binding.gdr_bwd_linear(q, k, v, g, x["dout"][:, :4].contiguous())
    with pytest.raises(ValueError, match="cu_seqlens"):
        binding.gdr_fwd_linear(q, k, v, g, cu_seqlens=torch.zeros(1, dtype=torch.int32, device=q.device))
    with pytest.raises(TypeError, match="cu_seqlens"):
        binding.gdr_fwd_linear(q, k, v, g, cu_seqlens=torch.tensor([0, 8], device=q.device))
    with pytest.raises(binding.GdrError, match="UNSUPPORTED"):
        binding.gdr_fwd_linear(q, k, v, g, path="tc")

"""The linear-attention operators, as they are measured: cases, inputs, the plain form of each operator and its 64-bit definition.

The operators (S of one (sequence, head) is a d_v x d_k fp32 matrix; value head h reads query/key head h // (H / H_k)):

    forward   S_t = e^{g_t} S_{t-1} + v_t k_t^T,  o_t = S_t q_t, over whole sequences       (gdr_fwd_linear)
    decode    the same update for one token of each sequence, in place on S                 (gdr_decode_step_linear)
    backward  dq, dk, dv, dg and dS0 of the forward from dout and dS_final                  (gdr_bwd_linear)

g is the log-decay, one per token and head ("token") or one per head for all tokens ("head").
"""
import math

import torch

own = False

CHUNK = 128  # tokens of a chunk in the plain form


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # a short first prompt of one request: latency
        dict(name="fwd_first_prompt", op="fwd", dtype="bf16", B=1, T=37, H=16, Hk=16, dk=128, dv=128,
             gate="token", seqs=0, s0=False),
        # a batch of equal prompts that continue from a state: the framework's own prefill sizes
        dict(name="fwd_batch", op="fwd", dtype="bf16", B=4, T=4096, H=16, Hk=16, dk=128, dv=128,
             gate="token", seqs=0, s0=True),
        # a packed batch of requests of unequal length
        dict(name="fwd_packed", op="fwd", dtype="bf16", B=1, T=65536, H=16, Hk=16, dk=128, dv=128,
             gate="token", seqs=16, s0=False),
        # many value heads that share few query/key heads, each with a fixed decay; a ragged length
        dict(name="fwd_shared_heads", op="fwd", dtype="bf16", B=2, T=1000, H=32, Hk=4, dk=128, dv=64,
             gate="head", seqs=0, s0=False),
        # single-precision tokens (a check run, a small model), an odd length
        dict(name="fwd_fp32", op="fwd", dtype="f32", B=2, T=777, H=8, Hk=8, dk=64, dv=64,
             gate="token", seqs=0, s0=True),
        # one request that generates: latency
        dict(name="decode_one", op="decode", dtype="bf16", B=1, T=1, H=16, Hk=16, dk=128, dv=128,
             gate="token", seqs=0, s0=True),
        # a full serving batch: the framework's own decode sizes
        dict(name="decode_batch", op="decode", dtype="bf16", B=256, T=1, H=32, Hk=32, dk=128, dv=128,
             gate="token", seqs=0, s0=True),
        # an odd batch of single-precision tokens, shared heads, fixed decays
        dict(name="decode_shared_heads", op="decode", dtype="f32", B=37, T=1, H=24, Hk=8, dk=64, dv=128,
             gate="head", seqs=0, s0=True),
        # training: a batch of equal sequences
        dict(name="bwd_batch", op="bwd", dtype="bf16", B=4, T=4096, H=16, Hk=16, dk=128, dv=128,
             gate="token", seqs=0, s0=True),
        # training on packed documents, shared query/key heads
        dict(name="bwd_packed_shared", op="bwd", dtype="bf16", B=1, T=8191, H=16, Hk=4, dk=128, dv=64,
             gate="token", seqs=9, s0=False),
        # training with fixed decays
        dict(name="bwd_fixed_decay", op="bwd", dtype="bf16", B=2, T=1500, H=8, Hk=8, dk=64, dv=64,
             gate="head", seqs=0, s0=False),
        # a short single-precision step (a gradient check)
        dict(name="bwd_fp32", op="bwd", dtype="f32", B=1, T=100, H=4, Hk=4, dk=64, dv=64,
             gate="token", seqs=0, s0=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "decode", "bwd", "bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    hk = _log(rng, 1, 16)
    h = hk * rng.choice([1, 1, 2, 4])
    dims = [64, 128, 64, 128, 96, 48] if op != "decode" else [64, 128]
    dk, dv = rng.choice(dims), rng.choice(dims)
    gate, s0 = rng.choice(["token", "token", "head"]), rng.random() < 0.5
    if op == "decode":
        return dict(op=op, dtype=dtype, B=_log(rng, 1, 8192 // h), T=1, H=h, Hk=hk, dk=dk, dv=dv,
                    gate=gate, seqs=0, s0=True)
    # token-heads: up to the largest listed case of the operator; single precision up to 32768
    most = 32768 if dtype == "f32" else 1 << 20 if op == "fwd" else 1 << 18
    tokens = min(_log(rng, 1, max(2, most // h)), 1 << 16)
    if rng.random() < 0.4:  # packed sequences
        return dict(op=op, dtype=dtype, B=1, T=tokens, H=h, Hk=hk, dk=dk, dv=dv, gate=gate,
                    seqs=_log(rng, max(2, -(-tokens // 8192)), 48), s0=s0)
    b = max(_log(rng, 1, 8), -(-tokens // 8192))
    return dict(op=op, dtype=dtype, B=b, T=max(1, tokens // b), H=h, Hk=hk, dk=dk, dv=dv, gate=gate,
                seqs=0, s0=s0)


# ----------------------------------------------------------------------------- inputs
def _lengths(case, gen):
    """The lengths of a packed batch, all of them drawn, short ones and long ones (some may be empty); each at most 8192."""
    n, total = case["seqs"], case["T"]
    w = torch.rand(n, generator=gen).add_(0.15)
    cut = (w.cumsum(0) / w.sum() * total).round().long()
    cut[-1] = total
    lens = torch.diff(cut, prepend=torch.zeros(1, dtype=torch.long)).tolist()
    spare = 0
    for i, x in enumerate(lens):  # what is over the longest length goes to the others
        spare += max(0, x - 8192)
        lens[i] = min(x, 8192)
    for i, x in enumerate(lens):
        add = min(8192 - x, spare)
        lens[i], spare = x + add, spare - add
    return lens


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    tok = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    B, T, H, Hk, dk, dv = (case[x] for x in ("B", "T", "H", "Hk", "dk", "dv"))
    lead = (B,) if case["op"] == "decode" else (B, T)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    st = {"case": dict(case)}
    st["q"] = torch.nn.functional.normalize(normal(*lead, Hk, dk), dim=-1).to(tok)
    st["k"] = torch.nn.functional.normalize(normal(*lead, Hk, dk), dim=-1).to(tok)
    st["v"] = normal(*lead, H, dv).to(tok)
    if case["gate"] == "head":  # fixed decays 1 - 2^-x: memories of about 8 to 512 tokens
        st["g"] = torch.log1p(-torch.exp2(-(3 + 6 * torch.rand(H, generator=gen, device=dev))))
    else:
        st["g"] = torch.nn.functional.softplus(normal(*lead, H)).mul_(-0.1)
    lens = None
    if case["seqs"]:
        lens = _lengths(case, torch.Generator().manual_seed(seed))
        st["cu"] = torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32)
    st["lens"] = lens if lens is not None else [T] * B
    n = len(st["lens"])
    st["S"] = normal(n, H, dv, dk).mul_(0.1) if case["s0"] else None
    if case["op"] == "bwd":
        st["dout"] = normal(*lead, H, dv).to(tok)
        st["dS"] = normal(n, H, dv, dk).mul_(0.1) if case["s0"] else None
    return st


# ----------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        from gated_delta_rule_90_b200 import binding
        a = [state[x] for x in ("q", "k", "v", "g")]
        if op == "decode":
            out = binding.gdr_decode_step_linear(*a, state["S"])
            return {"out": out, "S": state["S"]}
        if op == "fwd":
            out, S = binding.gdr_fwd_linear(*a, state["S"], cu_seqlens=state.get("cu"))
            return {"out": out, "S_final": S}
        got = binding.gdr_bwd_linear(*a, state["dout"], state["S"], state["dS"],
                                     cu_seqlens=state.get("cu"))
        return dict(zip(("dq", "dk", "dv", "dg", "dS0"), got))
    return {"decode": _decode, "fwd": _forward, "bwd": _backward}[op](state)


def _decode(st):
    q, k, v, g, S = (st[x].float() for x in ("q", "k", "v", "g", "S"))
    r = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    S.mul_(g.exp().expand(v.shape[:2])[..., None, None])
    S.addcmul_(v[..., :, None], k[..., None, :])
    out = (S @ q[..., None])[..., 0].to(st["v"].dtype)
    return {"out": out, "S": S}


class _Chunks:
    """Sequences cut into chunks of CHUNK tokens, and what the chunked form needs of the decays: 64-bit running sums, so
    that the differences of far positions keep their digits."""

    def __init__(self, st):
        v, lens = st["v"], st["lens"]
        self.H, dev = v.shape[2], v.device
        self.tokens = v.shape[0] * v.shape[1]
        lens = torch.tensor(lens)
        count = (lens + CHUNK - 1) // CHUNK
        seq = torch.repeat_interleave(torch.arange(len(lens)), count)
        first = (torch.cumsum(count, 0) - count)[seq]
        at = (torch.arange(len(seq)) - first) * CHUNK
        left = (lens[seq] - at).clamp(max=CHUNK)
        self.seq, self.n_seq = seq.to(dev), len(lens)
        idx = ((torch.cumsum(lens, 0) - lens)[seq] + at)[:, None] + torch.arange(CHUNK)
        self.ok = (torch.arange(CHUNK) < left[:, None]).to(dev)          # [c, l]
        self.idx = idx.clamp(max=max(self.tokens - 1, 0)).to(dev)
        self.last = torch.cumsum(count, 0)[count > 0].sub(1).to(dev)     # last and first chunk of each sequence with tokens
        self.first = (torch.cumsum(count, 0) - count)[count > 0].to(dev)
        self.some = torch.nonzero(count > 0)[:, 0].to(dev)
        g = st["g"].double()
        g = g.expand(self.tokens, self.H) if g.dim() == 1 else g.reshape(self.tokens, self.H)
        g = (g[self.idx] * self.ok[..., None]).transpose(1, 2)           # [c, h, l]
        G = g.cumsum(-1)
        self.total = G[..., -1]                                          # [c, h]
        self.read = G.exp().float()                                      # of the state before the chunk, at l
        self.write = (self.total[..., None] - G).exp().float() * self.ok[:, None]  # of token l, at the chunk's end
        low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
        keep = low & self.ok[:, None, None, :]
        self.pair = torch.where(keep, G[..., :, None] - G[..., None, :], -math.inf).exp().float()  # [c, h, l, m]
        E = self.total.cumsum(0).t()                                     # [h, c]: over all chunks in a row
        same = self.seq[:, None] == self.seq[None, :]
        c = torch.arange(len(seq), device=dev)
        before = E - self.total.t()                                      # up to the chunk's start
        # state of chunk c from chunk j < c: the decay from j's end to c's start; from the sequence's first state
        self.carry = torch.where(same & (c[:, None] > c[None, :]), before[:, :, None] - E[:, None, :], -math.inf).exp().float()
        self.begin = (before - before[:, first.to(dev)]).exp().float()   # [h, c]
        ends = (torch.cumsum(count, 0) - 1)[seq].to(dev)
        self.finish = (E[:, ends] - E).exp().float()                     # from c's end to the sequence's end

    def cut(self, x, zero):
        """[B, T, h, d] -> [c, H, CHUNK, d] in 32 bits."""
        x = x.reshape(self.tokens, *x.shape[2:])[self.idx].float().transpose(1, 2)
        if zero:
            x = x * self.ok[:, None, :, None]
        return x.repeat_interleave(self.H // x.shape[1], 1)

    def join(self, x, like):
        """[c, H, CHUNK, d] -> the layout and type of `like`, shared heads summed."""
        h = like.shape[2]
        x = x.unflatten(1, (h, self.H // h)).sum(2).transpose(1, 2)
        out = torch.empty(self.tokens, h, x.shape[-1], dtype=like.dtype, device=like.device)
        out[self.idx[self.ok]] = x[self.ok].to(like.dtype)
        return out.view(like.shape[0], like.shape[1], h, -1)

    def states(self, P, S0):
        """The state before each chunk: P [c, H, dv, dk] of each chunk carried forward, and S0."""
        S = (self.carry @ P.transpose(0, 1).flatten(2)).view(self.H, -1, *P.shape[2:]).transpose(0, 1)
        if S0 is not None:
            S = S + self.begin.t()[..., None, None] * S0[self.seq]
        return S

    def adjoints(self, D, dS):
        """The gradient of the state after each chunk: D of each chunk carried backward, and dS."""
        A = (self.carry.transpose(1, 2) @ D.transpose(0, 1).flatten(2)).view(self.H, -1, *D.shape[2:]).transpose(0, 1)
        if dS is not None:
            A = A + self.finish.t()[..., None, None] * dS[self.seq]
        return A


def _forward(st):
    x = _Chunks(st)
    q, k, v = x.cut(st["q"], False), x.cut(st["k"], True), x.cut(st["v"], True)
    P = (v * x.write[..., None]).transpose(-1, -2) @ k
    S = x.states(P, st["S"])
    o = ((q @ k.transpose(-1, -2)) * x.pair) @ v + x.read[..., None] * (q @ S.transpose(-1, -2))
    dv, dk = v.shape[-1], k.shape[-1]
    S_final = torch.zeros(x.n_seq, x.H, dv, dk, device=v.device) if st["S"] is None else st["S"].clone()
    S_final[x.some] = (x.total.exp().float()[..., None, None] * S + P)[x.last]
    return {"out": x.join(o, st["v"]), "S_final": S_final}


def _backward(st):
    x = _Chunks(st)
    q, k, v, do = x.cut(st["q"], True), x.cut(st["k"], True), x.cut(st["v"], True), x.cut(st["dout"], True)
    end = x.total.exp().float()[..., None, None]
    P = (v * x.write[..., None]).transpose(-1, -2) @ k
    S = x.states(P, st["S"])
    D = (do * x.read[..., None]).transpose(-1, -2) @ q
    A = x.adjoints(D, st["dS"])
    pv = (do @ v.transpose(-1, -2)) * x.pair
    pk = (q @ k.transpose(-1, -2)) * x.pair
    old = x.read[..., None] * (do @ S)
    new = x.write[..., None] * (v @ A)
    dq = old + pv @ k
    dk = new + pv.transpose(-1, -2) @ q
    dv = x.write[..., None] * (k @ A.transpose(-1, -2)) + pk.transpose(-1, -2) @ do
    both = pv * (q @ k.transpose(-1, -2))
    rows = both.sum(-1) + (old * q).sum(-1) - both.sum(-2) - (new * k).sum(-1)     # [c, h, l]
    dg = rows.flip(-1).cumsum(-1).flip(-1) + ((end * S + P) * A).sum((-1, -2))[..., None]
    if st["g"].dim() == 1:
        dg = (dg.double() * x.ok[:, None]).sum((0, 2)).float()
    else:
        dg = x.join(dg[..., None], st["v"].float()).view(st["g"].shape)
    dS0 = torch.zeros(x.n_seq, x.H, v.shape[-1], k.shape[-1], device=v.device) if st["dS"] is None else st["dS"].clone()
    dS0[x.some] = (end * A + D)[x.first]
    return {"dq": x.join(dq, st["q"]), "dk": x.join(dk, st["k"]), "dv": x.join(dv, st["v"]), "dg": dg, "dS0": dS0}


# ----------------------------------------------------------------------------- cost
def work(case):
    B, T, H, Hk, dk, dv = (case[x] for x in ("B", "T", "H", "Hk", "dk", "dv"))
    e = 2 if case["dtype"] == "bf16" else 4
    n = case["seqs"] or B
    tokens = B * T
    gate = 4 * (tokens * H if case["gate"] == "token" else H)
    qk, vv, state = 2 * tokens * Hk * dk * e, tokens * H * dv * e, 4 * n * H * dk * dv
    # a token of a head: its rank-1 update of the state and one product with the state, 2 d_k d_v each
    step = 2.0 * tokens * H * dk * dv
    if case["op"] == "decode":
        return {"bytes": qk + 2 * vv + gate + 2 * state, "flops": 2 * step}
    s = state * (2 if case["s0"] else 1)
    if case["op"] == "fwd":
        return {"bytes": qk + 2 * vv + gate + s, "flops": 2 * step}
    # backward: both states' updates, and three products with them
    return {"bytes": 2 * qk + 3 * vv + 2 * gate + s + (state if case["s0"] else 0), "flops": 5 * step}


# ----------------------------------------------------------------------------- 64-bit definition
def exact(case, seed):
    """The token recurrence of the definition in 64 bits, all sequences side by side."""
    st = prepare(case, seed)
    dt = torch.float64
    v0, lens = st["v"], st["lens"]
    if case["op"] == "decode":
        q, k, v, S = (st[x].to(dt) for x in ("q", "k", "v", "S"))
        r = v.shape[1] // q.shape[1]
        a = st["g"].to(dt).exp()
        a = a.view(1, -1, 1, 1) if a.dim() == 1 else a[..., None, None]
        S = a * S + v.unsqueeze(-1) * k.repeat_interleave(r, 1).unsqueeze(-2)
        return {"out": torch.einsum("nhvk,nhk->nhv", S, q.repeat_interleave(r, 1)), "S": S}
    H, dev = v0.shape[2], v0.device
    N, L = len(lens), max(lens)
    tokens = v0.shape[0] * v0.shape[1]
    n = torch.tensor(lens, device=dev)
    start = torch.cumsum(n, 0) - n
    t = torch.arange(L, device=dev)
    inside = t < n[:, None]                                           # [N, L]
    at = (start[:, None] + t).clamp(max=tokens - 1)

    def rows(x):  # [L, N, H, d], zero past the end
        x = x.reshape(tokens, *x.shape[2:])[at].to(dt) * inside[..., None, None]
        return x.repeat_interleave(H // x.shape[2], 2).transpose(0, 1).contiguous()

    def back(x, heads):  # [L, N, H, d] -> [B, T, heads, d]
        x = x.transpose(0, 1)[inside]
        x = x.view(x.shape[0], heads, H // heads, x.shape[-1]).sum(2)
        return x.view(v0.shape[0], v0.shape[1], heads, -1)

    q, k, v = rows(st["q"]), rows(st["k"]), rows(st["v"])
    g = st["g"].to(dt)
    g = g.view(1, 1, H).expand(v0.shape[0], v0.shape[1], H) if g.dim() == 1 else g
    a = rows(g[..., None])[..., 0].exp()[..., None, None]             # [L, N, H, 1, 1]
    dk, dv = k.shape[-1], v.shape[-1]
    S = torch.zeros(N, H, dv, dk, dtype=dt, device=dev) if st["S"] is None else st["S"].to(dt)
    if case["op"] == "fwd":
        o = torch.empty_like(v)
        for i in range(L):
            S = S * a[i] + v[i].unsqueeze(-1) * k[i].unsqueeze(-2)
            o[i] = (S @ q[i].unsqueeze(-1)).squeeze(-1)
        return {"out": back(o, H), "S_final": S}
    do = rows(st["dout"])
    dq, dkk, dvv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for i in range(L):
        S = S * a[i] + v[i].unsqueeze(-1) * k[i].unsqueeze(-2)
        dq[i] = (do[i].unsqueeze(-2) @ S).squeeze(-2)
    A = torch.zeros_like(S) if st["dS"] is None else st["dS"].to(dt)
    # d loss / d g_t: the sum over s >= t of q_s . dq_s - k_s . dk_s, and the last state's own product with its gradient
    tail = (S * A).sum((-1, -2))
    for i in range(L - 1, -1, -1):
        A = A + do[i].unsqueeze(-1) * q[i].unsqueeze(-2)
        dkk[i] = (v[i].unsqueeze(-2) @ A).squeeze(-2)
        dvv[i] = (A @ k[i].unsqueeze(-1)).squeeze(-1)
        A = A * a[i]
    dg = ((q * dq).sum(-1) - (k * dkk).sum(-1)).flip(0).cumsum(0).flip(0) + tail
    dg = back(dg[..., None], H).squeeze(-1)
    if st["g"].dim() == 1:
        dg = dg.sum((0, 1))
    return {"dq": back(dq, case["Hk"]), "dk": back(dkk, case["Hk"]), "dv": back(dvv, H), "dg": dg, "dS0": A}

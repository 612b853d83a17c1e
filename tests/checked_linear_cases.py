"""Small calls of the linear attention entry points on both paths, shared by
the checked-build test: run through the normal library and, in a child process
with GDR_LIBRARY set, through the checked one."""
import sys

import numpy as np
import torch

from gated_delta_rule_90_b200 import binding


def run_cases(dev) -> dict:
    res = {}
    for name, B, T, H, Hk, dk, dv, dtype, path, gate, cu in (
            ("tc", 2, 300, 2, 1, 128, 64, torch.bfloat16, "tc", "token", None),
            ("tc_blocks", 1, 1200, 1, 1, 48, 96, torch.bfloat16, "tc", "head", None),
            ("tc_packed", 1, 700, 2, 2, 64, 128, torch.bfloat16, "tc", "token", [0, 0, 130, 131, 690]),
            ("simt_bf16", 1, 290, 2, 1, 64, 48, torch.bfloat16, "simt", "token", [3, 50, 290]),
            ("simt_fp32", 2, 100, 2, 2, 32, 112, torch.float32, "simt", "head", None)):
        gen = torch.Generator(device=dev).manual_seed(5)

        def rand(*s):
            return torch.randn(*s, generator=gen, device=dev)

        n = B if cu is None else len(cu) - 1
        q, k = (rand(B, T, Hk, dk).mul_(dk ** -0.5).to(dtype) for _ in range(2))
        v, dout = rand(B, T, H, dv).to(dtype), rand(B, T, H, dv).to(dtype)
        g = -0.1 * rand(*((H,) if gate == "head" else (B, T, H))).abs()
        S0, dS = rand(n, H, dv, dk), rand(n, H, dv, dk)
        c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=dev)
        out = torch.zeros_like(v)
        got = binding.gdr_fwd_linear(q, k, v, g, S0, cu_seqlens=c, path=path, out=out)
        z = [torch.zeros_like(t) for t in (q, k, v, g)]
        got += binding.gdr_bwd_linear(q, k, v, g, dout, S0, dS, cu_seqlens=c, path=path, dq=z[0],
                                      dk=z[1], dv=z[2], dg=z[3])
        S = S0.clone()
        if cu is None:
            g1 = g if g.dim() == 1 else g[:, 0].contiguous()
            got += (binding.gdr_decode_step_linear(*(t[:, 0].contiguous() for t in (q, k, v)), g1, S), S)
        st = binding.device_status()
        assert st == binding.GDR_OK, (name, binding.status_string(st))
        for i, t in enumerate(got):
            res["%s.%d" % (name, i)] = t.float().cpu().numpy()
    return res


if __name__ == "__main__":
    assert binding.checked_build(), binding.library_path()
    np.savez(sys.argv[1], **run_cases(torch.device("cuda:0")))

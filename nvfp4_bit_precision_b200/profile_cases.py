"""Single-case drivers for profiling one kernel launch under ncu.

    python -m nvfp4_bit_precision_b200.profile_cases gemm M N K [--warm W]
    python -m nvfp4_bit_precision_b200.profile_cases mxfp8-gemm M N K [--warm W]
    python -m nvfp4_bit_precision_b200.profile_cases grouped-gemm N K [--warm W]
    python -m nvfp4_bit_precision_b200.profile_cases quant-grad ROWS COLS [--warm W]
    python -m nvfp4_bit_precision_b200.profile_cases quant-act ROWS COLS [--warm W]
    python -m nvfp4_bit_precision_b200.profile_cases quant-weight ROWS COLS [--warm W]
    python -m nvfp4_bit_precision_b200.profile_cases mxfp4 ROWS COLS [--warm W]
    python -m nvfp4_bit_precision_b200.profile_cases dispatch TOKENS HIDDEN [--warm W]
    python -m nvfp4_bit_precision_b200.profile_cases combine TOKENS HIDDEN [--warm W]
    python -m nvfp4_bit_precision_b200.profile_cases norm ROWS COLS [--warm W]
    python -m nvfp4_bit_precision_b200.profile_cases norm-backward ROWS COLS [--warm W]
    python -m nvfp4_bit_precision_b200.profile_cases route TOKENS EXPERTS [--warm W]
    python -m nvfp4_bit_precision_b200.profile_cases weighted-combine TOKENS HIDDEN [--warm W]
    python -m nvfp4_bit_precision_b200.profile_cases gemv ROWS N K [--warm W]
    python -m nvfp4_bit_precision_b200.profile_cases kv-append TOKENS HEADS [--warm W]
    python -m nvfp4_bit_precision_b200.profile_cases kv-attention SEQUENCES LENGTH HEADS [--warm W]
    python -m nvfp4_bit_precision_b200.profile_cases expert-mlp TOKENS HIDDEN FFN [--warm W]

Each runs W untimed launches of the case, then one more, on synthetic operands
(codes and in-range scale bytes drawn on the device; bf16 inputs ~N(0, 1e-3)),
and exits 0 when the device status word is clear.  Pair with `ncu -s W -c 1`.
"""
from __future__ import annotations

import argparse
import sys


def _gemm(nv, torch, M, N, K, warm):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(0)
    u8 = dict(dtype=torch.uint8, device=dev)
    qa = torch.randint(0, 256, (M, K // 2), generator=g, **u8)
    qb = torch.randint(0, 256, (N, K // 2), generator=g, **u8)
    sa = torch.randint(0x30, 0x40, (nv.nvfp4_sf_mma_bytes(M, K),), generator=g, **u8)
    sb = torch.randint(0x30, 0x40, (nv.nvfp4_sf_mma_bytes(N, K),), generator=g, **u8)
    one = torch.ones(1, dtype=torch.float32, device=dev)
    D = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    ws = torch.zeros(256, **u8)
    for _ in range(warm + 1):
        nv.nvfp4_gemm(qa, sa, one, qb, sb, one, M, N, K, nv.NVFP4_OUT_BF16, D, N, None, ws, 256)
    return ws


def _mxfp8_gemm(nv, torch, M, N, K, warm):
    """MXFP8 GEMM on random E4M3 codes (NaN codes 0x7F/0xFF mapped to 0) and E8M0
    scale bytes near 127."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(0)
    u8 = dict(dtype=torch.uint8, device=dev)
    qa = torch.randint(0, 256, (M, K), generator=g, **u8)
    qb = torch.randint(0, 256, (N, K), generator=g, **u8)
    for q in (qa, qb):
        q[(q & 0x7F) == 0x7F] = 0
    sa = torch.randint(120, 134, (nv.mxfp8_sf_mma_bytes(M, K),), generator=g, **u8)
    sb = torch.randint(120, 134, (nv.mxfp8_sf_mma_bytes(N, K),), generator=g, **u8)
    D = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    ws = torch.zeros(256, **u8)
    for _ in range(warm + 1):
        nv.mxfp8_gemm(qa, sa, qb, sb, M, N, K, nv.NVFP4_OUT_BF16, D, N, None, ws, 256)
    return ws


def _grouped(nv, torch, N, K, warm):
    import numpy as np

    import workloads as W
    dev = torch.device("cuda")
    rng = np.random.default_rng(3)
    _, _, offsets = W.moe_routing(rng, 16384, 64, 4)
    R, G = int(offsets[-1]), 64
    u8 = dict(dtype=torch.uint8, device=dev)
    qa = torch.randint(0, 256, (R, K // 2), **u8)
    sa = torch.randint(0x30, 0x40, (nv.nvfp4_sf_mma_grouped_bytes(R, G, K),), **u8)
    qb = torch.randint(0, 256, (G, N, K // 2), **u8)
    sb = torch.randint(0x30, 0x40, (G * nv.nvfp4_sf_mma_bytes(N, K),), **u8)
    ga = torch.ones(1, dtype=torch.float32, device=dev)
    gb = torch.ones(G, dtype=torch.float32, device=dev)
    off = torch.from_numpy(offsets.astype(np.int32)).to(dev)
    D = torch.empty((R, N), dtype=torch.bfloat16, device=dev)
    ws = torch.zeros(256, **u8)
    for _ in range(warm + 1):
        nv.nvfp4_grouped_gemm(G, off, R, qa, sa, ga, qb, sb, gb, N, K, nv.NVFP4_OUT_BF16, D, None,
                              ws, 256)
    return ws


def _quant_grad(nv, torch, rows, cols, warm):
    """The gradient recipe: rowwise SR, columnwise Hadamard + SR, MXFP8 columnwise."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    x = (torch.randn((rows, cols), generator=g, device=dev) * 1e-3).to(torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    for _ in range(warm + 1):
        nv.quantize(x, rowwise=True, colwise=True, rounding=nv.NVFP4_SR, rht=True, seed=5,
                    mx_outputs=nv.NVFP4_COLWISE, sf_layout=nv.NVFP4_SF_MMA, workspace=ws)
    return ws


def _quant_act(nv, torch, rows, cols, warm):
    """The activation recipe: rowwise and columnwise Hadamard, both RNE."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(3)
    x = torch.randn((rows, cols), generator=g, device=dev).to(torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    for _ in range(warm + 1):
        nv.quantize(x, rowwise=True, colwise=True, rht=True, sf_layout=nv.NVFP4_SF_MMA, workspace=ws)
    return ws


def _quant_weight(nv, torch, rows, cols, warm):
    """The weight recipe: 16x16 2D scales, both directions, RNE."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(4)
    x = (torch.randn((rows, cols), generator=g, device=dev) * 0.02).to(torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev)
    for _ in range(warm + 1):
        nv.quantize(x, rowwise=True, colwise=True, scaling=nv.NVFP4_2D16x16, sf_layout=nv.NVFP4_SF_MMA,
                    workspace=ws)
    return ws


def _mxfp4(nv, torch, rows, cols, warm):
    """MXFP4 of a bf16 ~N(0, 1) tensor, both directions."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(2)
    x = torch.randn((rows, cols), generator=g, device=dev).to(torch.bfloat16)
    for _ in range(warm + 1):
        nv.mxfp4(x, nv.NVFP4_ROWWISE | nv.NVFP4_COLWISE)
    return None


def _dispatch(nv, torch, tokens, hidden, warm):
    """MoE dispatch of quantised token rows (top-4 Zipf(1.1) routing over 64 experts)
    into the grouped layout."""
    import numpy as np

    import workloads as W
    dev = torch.device("cuda")
    _, row_token, offsets = W.moe_routing(np.random.default_rng(3), tokens, 64, 4)
    R = int(offsets[-1])
    g = torch.Generator(device=dev)
    g.manual_seed(5)
    x = torch.randn((tokens, hidden), generator=g, device=dev).to(torch.bfloat16)
    t = nv.quantize(x, sf_layout=nv.NVFP4_SF_MMA)["row"]
    u8 = dict(dtype=torch.uint8, device=dev)
    qd = torch.empty((R, hidden // 2), **u8)
    sd = torch.zeros(nv.nvfp4_sf_mma_grouped_bytes(R, 64, hidden), **u8)
    rt = torch.from_numpy(row_token.astype(np.int32)).to(dev)
    off = torch.from_numpy(offsets.astype(np.int32)).to(dev)
    ws = torch.zeros(256, **u8)
    for _ in range(warm + 1):
        nv.nvfp4_gather_rows(t.q, t.sf, tokens, hidden, rt, R, off, 64, qd, sd, ws, 256)
    return ws


def _combine(nv, torch, tokens, hidden, warm):
    """MXFP8 combine of top-4 expert rows (in expert order) into tokens x hidden bf16."""
    import numpy as np
    dev = torch.device("cuda")
    R, k = 4 * tokens, 4
    g = torch.Generator(device=dev)
    g.manual_seed(6)
    out_rows = torch.randn((R, hidden), generator=g, device=dev).to(torch.bfloat16)
    u8 = dict(dtype=torch.uint8, device=dev)
    q, e8 = torch.empty((R, hidden), **u8), torch.empty((R, hidden // 32), **u8)
    nv.mxfp8_quantize(out_rows, R, hidden, hidden, nv.NVFP4_ROWWISE, 0, 0, 0, q, e8, None, None)
    slot = torch.from_numpy(np.random.default_rng(7).permutation(R).reshape(tokens, k).astype(np.int32)).to(dev)
    w = torch.full((tokens, k), 1.0 / k, dtype=torch.float32, device=dev)
    out = torch.empty((tokens, hidden), dtype=torch.bfloat16, device=dev)
    ws = torch.zeros(256, **u8)
    for _ in range(warm + 1):
        nv.mxfp8_combine(q, e8, R, hidden, slot, w, tokens, k, out, ws, 256)
    return ws


def _bf16(torch, shape, std, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _norm(nv, torch, rows, cols, warm):
    """The norm of x + residual as MXFP8 with tiled scales."""
    x, r, w = (_bf16(torch, s, 1.0, i) for i, s in enumerate(((rows, cols), (rows, cols), (cols,))))
    for _ in range(warm + 1):
        nv.rmsnorm(x, w, r, y=False, mx=True, mx_sf_layout=nv.NVFP4_SF_MMA)


def _norm_backward(nv, torch, rows, cols, warm):
    """The norm's gradients, with one of the sum coming in."""
    x, dy, dh, w = (_bf16(torch, s, 1.0, i) for i, s in enumerate(((rows, cols),) * 3 + ((cols,),)))
    rstd = nv.rmsnorm(x, w, rstd=True)["rstd"]
    for _ in range(warm + 1):
        nv.rmsnorm_backward(dy, x, w, rstd, dh)


def _route(nv, torch, tokens, experts, warm):
    """Softmax routing to four experts, renormalised."""
    logits = _bf16(torch, (tokens, experts), 1.5, 0).float()
    for _ in range(warm + 1):
        nv.route(logits, min(4, experts))


def _weighted_combine(nv, torch, tokens, hidden, warm):
    """The weighted sum of four bf16 rows per token, in random order."""
    rows = _bf16(torch, (4 * tokens, hidden), 1.0, 0)
    slot = torch.randperm(4 * tokens, device="cuda").to(torch.int32).reshape(tokens, 4)
    w = torch.full((tokens, 4), 0.25, device="cuda")
    for _ in range(warm + 1):
        nv.combine(rows, slot, w)


def _gemv(nv, torch, rows, N, K, warm):
    """A few bf16 rows times an NVFP4 matrix."""
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    u8 = dict(dtype=torch.uint8, device="cuda")
    w = nv.NVFP4Tensor(torch.randint(0, 256, (N, K // 2), generator=g, **u8),
                       torch.randint(0x30, 0x40, (nv.nvfp4_sf_mma_bytes(N, K),), generator=g, **u8),
                       torch.ones(1, device="cuda"), N, K, nv.NVFP4_SF_MMA)
    x = _bf16(torch, (rows, K), 1.0, 0)
    for _ in range(warm + 1):
        nv.gemv(x, w)


def _random_cache(nv, torch, pages, kv_heads, page, dim):
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    u8 = dict(dtype=torch.uint8, device="cuda", generator=g)
    c = nv.kv_cache(pages, kv_heads, page, dim, 8.0, 8.0)
    c.q.copy_(torch.randint(0, 256, tuple(c.q.shape), **u8))
    c.sf.copy_(torch.randint(0x30, 0x40, tuple(c.sf.shape), **u8))
    return c


def _kv_append(nv, torch, tokens, heads, warm):
    """Tokens of one sequence each 2048 long, 8 key heads of 128, keys and queries turned."""
    page, dim, kv, each = 64, 128, 8, min(tokens, 2048)
    n = -(-tokens // each)
    table = torch.randperm(n * -(-each // page), device="cuda").to(torch.int32).reshape(n, -1)
    cache = _random_cache(nv, torch, table.numel(), kv, page, dim)
    qkv = _bf16(torch, (tokens, heads + 2 * kv, dim), 1.0, 0)
    at = torch.arange(tokens, device="cuda")
    angle = (at[:each, None].double() * 10000.0 ** (-torch.arange(0, dim, 2, device="cuda").double() / dim))
    for _ in range(warm + 1):
        nv.kv_append(cache, qkv[:, heads:heads + kv], qkv[:, heads + kv:], table, (at % each).to(torch.int32),
                     (at // each).to(torch.int32), cos=angle.cos().float(), sin=angle.sin().float(), q=qkv[:, :heads])


def _kv_attention(nv, torch, sequences, length, heads, warm):
    """One query token of each sequence over its whole cache, 8 key heads of 128."""
    page, dim, kv = 64, 128, 8
    table = torch.randperm(sequences * -(-length // page), device="cuda").to(torch.int32).reshape(sequences, -1)
    cache = _random_cache(nv, torch, table.numel(), kv, page, dim)
    q = _bf16(torch, (sequences, 1, heads, dim), 1.0, 0)
    lengths = torch.full((sequences,), length, dtype=torch.int32, device="cuda")
    size = nv.nvfp4_kv_attention_workspace_size(sequences, 1, heads, kv, dim, table.shape[1] * page)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for _ in range(warm + 1):
        nv.kv_attention(q, cache, table, lengths, workspace=ws)
    return ws


def _expert_mlp(nv, torch, tokens, hidden, ffn, warm):
    """A few tokens through four of 64 gated experts."""
    from .moe import ExpertWeights
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    u8 = dict(dtype=torch.uint8, device="cuda", generator=g)

    def weights(n, k):
        return ExpertWeights(torch.randint(0, 256, (64, n, k // 2), **u8),
                             torch.randint(0x30, 0x40, (64 * nv.nvfp4_sf_mma_bytes(n, k),), **u8),
                             torch.full((64,), 0.01 / k ** 0.5, device="cuda"), n)

    up, gate, down = weights(ffn, hidden), weights(ffn, hidden), weights(hidden, ffn)
    x = _bf16(torch, (tokens, hidden), 1.0, 0)
    r = nv.route(_bf16(torch, (tokens, 64), 1.5, 1).float(), 4)
    ws = torch.zeros(nv.nvfp4_expert_mlp_workspace_size(4 * tokens, hidden, ffn), dtype=torch.uint8, device="cuda")
    for _ in range(warm + 1):
        nv.expert_mlp(x, r, up, down, gate, x, workspace=ws)
    return ws


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("case", choices=["gemm", "mxfp8-gemm", "grouped-gemm", "quant-grad", "quant-act",
                                         "quant-weight", "mxfp4", "dispatch", "combine", "norm",
                                         "norm-backward", "route", "weighted-combine", "gemv", "kv-append",
                                         "kv-attention", "expert-mlp"])
    ap.add_argument("dims", type=int, nargs="+")
    ap.add_argument("--warm", type=int, default=3)
    args = ap.parse_args(argv)
    import torch

    import nvfp4_bit_precision_b200 as nv
    if args.case == "gemm":
        ws = _gemm(nv, torch, *args.dims[:3], args.warm)
    elif args.case == "mxfp8-gemm":
        ws = _mxfp8_gemm(nv, torch, *args.dims[:3], args.warm)
    elif args.case == "grouped-gemm":
        ws = _grouped(nv, torch, *args.dims[:2], args.warm)
    elif args.case == "quant-grad":
        ws = _quant_grad(nv, torch, *args.dims[:2], args.warm)
    elif args.case == "quant-act":
        ws = _quant_act(nv, torch, *args.dims[:2], args.warm)
    elif args.case == "quant-weight":
        ws = _quant_weight(nv, torch, *args.dims[:2], args.warm)
    elif args.case == "dispatch":
        ws = _dispatch(nv, torch, *args.dims[:2], args.warm)
    elif args.case == "combine":
        ws = _combine(nv, torch, *args.dims[:2], args.warm)
    elif args.case == "gemv":
        ws = _gemv(nv, torch, *args.dims[:3], args.warm)
    elif args.case == "kv-append":
        ws = _kv_append(nv, torch, *args.dims[:2], args.warm)
    elif args.case == "kv-attention":
        ws = _kv_attention(nv, torch, *args.dims[:3], args.warm)
    elif args.case == "expert-mlp":
        ws = _expert_mlp(nv, torch, *args.dims[:3], args.warm)
    elif args.case in ("norm", "norm-backward", "route", "weighted-combine"):
        case = {"norm": _norm, "norm-backward": _norm_backward, "route": _route,
                "weighted-combine": _weighted_combine}[args.case]
        ws = case(nv, torch, *args.dims[:2], args.warm)
    else:
        ws = _mxfp4(nv, torch, *args.dims[:2], args.warm)
    torch.cuda.synchronize()
    status = nv.nvfp4_workspace_status(ws) if ws is not None else 0
    print(f"{args.case} {args.dims}: status {nv.status_string(status)}")
    return 0 if status == 0 else 1


if __name__ == "__main__":
    sys.exit(main())

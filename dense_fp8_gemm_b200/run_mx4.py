"""Run a few eager launches of one MXFP4 or expert operator, for profilers.

    python -m dense_fp8_gemm_b200.run_mx4 --op gemm --shape 51200x5120 --rows 16 --repeat 3
    python -m dense_fp8_gemm_b200.run_mx4 --op experts --shape 2560x5120 --experts 64 --rows 32 --repeat 3
    python -m dense_fp8_gemm_b200.run_mx4 --op quantize --shape 1x5120 --rows 8192 --top 4 --repeat 3
    python -m dense_fp8_gemm_b200.run_mx4 --op sort --rows 16384 --top 8 --experts 256 --repeat 3
    python -m dense_fp8_gemm_b200.run_mx4 --op combine --shape 1x5120 --rows 8192 --top 8 --repeat 3

`--shape NxK`: weight rows and columns (quantize and combine use the second).
`--rows`: rows of activations (experts: rows over all experts, evenly spread;
sort, combine, and the gather of quantize: tokens, with --top choices each).
Every launch goes through the C ABI; inputs are drawn on the GPU from a seed.
"""
from __future__ import annotations

import argparse
import sys

import torch

from . import spense


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--op", default="gemm", choices=["gemm", "experts", "quantize", "sort", "combine"])
    ap.add_argument("--shape", default="51200x5120", help="NxK")
    ap.add_argument("--rows", type=int, default=16)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--top", type=int, default=8)
    ap.add_argument("--repeat", type=int, default=3)
    args = ap.parse_args(argv)
    N, K = (int(v) for v in args.shape.lower().split("x"))
    M, E, k = args.rows, args.experts, args.top
    g = torch.Generator(device="cuda").manual_seed(1)

    def operands(rows):
        return spense.mx4_quantize(torch.randn(rows, K, device="cuda", generator=g), scale_rows=True)

    ids = torch.randint(E, (M, k), device="cuda", generator=g)
    status = 0
    if args.op in ("gemm", "experts"):
        count = 1 if args.op == "gemm" else E
        wq, ws = operands(count * N)
        pw = spense.mx4_pack(wq.view(count, N, -1), ws.view(count, N, -1))
        xq, xs = spense.mx4_quantize(torch.randn(M, K, device="cuda", generator=g))
        off = None if count == 1 else (torch.arange(E + 1, device="cuda") * M // E).to(torch.int32)
        work = spense.new_workspace(spense.mx4_workspace_size(pw, M))
        Y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        call = spense.PreparedMx4Gemm(pw, xq, xs, Y, work, offsets=off)
        for _ in range(args.repeat):
            call()
        status = spense.workspace_status(work)
    elif args.op == "quantize":
        X = torch.randn(M, K, device="cuda", generator=g).to(torch.bfloat16)
        rows = torch.randint(M, (M * k,), device="cuda", generator=g).to(torch.int32)
        for _ in range(args.repeat):
            spense.mx4_dequantize(*spense.mx4_quantize(X, rows=rows))
    elif args.op == "sort":
        for _ in range(args.repeat):
            spense.expert_sort(ids, E)
    else:
        Y = torch.randn(M * k, K, device="cuda", generator=g).to(torch.bfloat16)
        pos = spense.expert_sort(ids, E)[2]
        weights = torch.rand(M, k, device="cuda", generator=g)
        for _ in range(args.repeat):
            spense.expert_combine(Y, pos, weights)
    torch.cuda.synchronize()
    print(f"ran {args.repeat} x {args.op}, status {status:#x}")
    return 0 if status == 0 else 1


if __name__ == "__main__":
    sys.exit(main())

"""Runs the operators of include/moe_block.h for a profiler: every listed case of perf/more_operators.py
with the library's calls, and with --more sizes whose figures comments and documents quote. Then, from
the trace of such a run, prints a table of the kernels.

  rocprofv3 --kernel-trace --stats -f csv -d DIR -o block -- python3 profiles/block_cases.py [--more] [--only TEXT]
  python3 profiles/block_cases.py --table DIR/block_kernel_trace.csv
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from layer_cases import ROOT, table  # noqa: E402


def more(ops):
    plain = ("none", False, "bf16", 0.0, False, False, False)
    return [
        ops._product("product 8192 cubed", 8192, 1, 1, 8192, 8192, *plain),
        ops._back("back 8192 cubed", 8192, 1, 1, 8192, 8192, "none", False, "bf16", "f32", 0.0, False),
        ops._product("gate, 64 tokens", 64, 1, 1, 384, 7168, *plain),
        ops._product("gate, 4096 tokens", 4096, 1, 1, 384, 7168, *plain),
        ops._product("8 rows of 8 experts", 1, 8, 128, 1024, 2048, "swiglu", True, "bf16", 0.0, False, False, False),
        *(ops._product(f"4096 cubed, {act}{', residual' if res else ''}{', pre' if pre else ''}", 4096, 1, 1, 4096, 4096,
                       act, False, dtype, 0.0, True, res, pre)
          for act, dtype, res, pre in (("none", "bf16", False, False), ("none", "bf16", True, False),
                                       ("none", "f32", True, False), ("relu", "bf16", False, False),
                                       ("silu", "bf16", False, False), ("gelu", "bf16", False, False),
                                       ("gelu", "bf16", True, True))),
        *(ops._back(f"back 4096 cubed, {act}", 4096, 1, 1, 4096, 4096, act, False, "bf16", "f32", 0.0, False)
          for act in ("none", "relu", "gelu", "swiglu")),
        ops._combine("combine back, fp32", 4096, 8, 7168, "f32", "f32"),
        ops._combine("combine back, fp32 rows", 4096, 8, 7168, "f32", "bf16"),
        ops._combine("combine back, fp32 of 128 tokens", 128, 8, 7168, "f32", "f32"),
    ]


def run(args):
    import torch
    sys.path.insert(0, ROOT)
    from perf import more_operators as ops
    ops.own = True
    for case in more(ops) if args.more else ops.listed():
        if args.only and args.only not in case["name"]:
            continue
        state = ops.prepare(case, 1)
        for _ in range(args.passes):
            ops.run(state)
        torch.cuda.synchronize()
        print(case["name"], flush=True)
        del state
        torch.cuda.empty_cache()


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawTextHelpFormatter)
    p.add_argument("--table", metavar="CSV")
    p.add_argument("--more", action="store_true")
    p.add_argument("--only", default="")
    p.add_argument("--passes", type=int, default=20)
    args = p.parse_args()
    table(args.table, args.passes) if args.table else run(args)

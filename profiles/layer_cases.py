"""Runs the operators of include/moe_layer.h for a profiler: every listed case of perf/operators.py with
the library's calls, and with --more the larger shapes whose figures comments and documents quote.
Then, from the trace of such a run, prints the table of kernel_trace_layer.md.

  rocprofv3 --kernel-trace --stats -f csv -d DIR -o layer -- python3 profiles/layer_cases.py [--more] [--only TEXT]
  python3 profiles/layer_cases.py --table DIR/layer_kernel_trace.csv
"""
import argparse
import csv
import os
import re
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def more(ops):
    return [
        ops._quant("quant bf16 4096 x 7168", 4096, 7168, "bf16"),
        ops._quant("quant bf16 32768 x 2048", 32768, 2048, "bf16"),
        ops._quant("quant bf16 32768 x 4096", 32768, 4096, "bf16"),
        ops._quant("quant f32 4096 x 7168", 4096, 7168, "f32"),
        ops._quant("quant f32 32768 x 2048", 32768, 2048, "f32"),
        ops._quant("quant f32 32768 x 4096", 32768, 4096, "f32"),
        ops._balance("balance 4096 sequences of 16", 65536, 4096, 256, 8, False, "both", False),
        ops._product("product 8192 cubed", 8192, 1, 1, 8192, 8192, "none", False, "bf16", 0.0),
        # the rows of an expert-parallel rank: 8 sources of 512 tokens, 48 of 384 experts, about 85
        # rows each, alone and in a buffer for all rows that 8 sources could send
        ops._product("rank gate and up", 4096, 1, 48, 2048, 7168, "swiglu", False, "bf16", 0.0),
        {**ops._product("rank gate and up, capacity", 4096, 1, 48, 2048, 7168, "swiglu", False,
                        "bf16", 0.0), "rows": 8 * 512 * 8},
        ops._product("rank down", 4096, 1, 48, 7168, 2048, "none", False, "bf16", 0.0),
        {**ops._product("rank down, capacity", 4096, 1, 48, 7168, 2048, "none", False, "bf16", 0.0),
         "rows": 8 * 512 * 8},
    ]


def run(args):
    import torch
    sys.path.insert(0, ROOT)
    from perf import operators as ops
    ops.own = True
    for case in more(ops) if args.more else ops.listed():
        if args.only and args.only not in case["name"]:
            continue
        state = ops.prepare(case, 1)
        if "rows" in case:                       # a buffer of so many rows, the last ones empty
            for name in ("a", "a_scale", "out"):
                t = state[name]
                state[name] = torch.zeros((case["rows"], *t.shape[1:]), dtype=t.dtype, device="cuda")
                state[name][:len(t)] = t
        torch.cuda.synchronize()
        a, b = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        for i in range(args.passes):
            if i == args.passes // 2:
                a.record()
            ops.run(state)
        b.record()
        torch.cuda.synchronize()
        print(f"{case['name']}: {a.elapsed_time(b) * 1e3 / (args.passes - args.passes // 2):.1f} us",
              flush=True)
        del state
        torch.cuda.empty_cache()


def plain_name(name):
    """k_name<arguments> of one of the library's kernels, or None. Names with bf16 arguments come as the
    compiler mangles them."""
    name = name.replace("(anonymous namespace)::", "")
    plain = re.match(r"(?:void )?(k_\w+(?:<[^(]*>)?)\(", name)
    if plain:
        return plain.group(1)
    mangled = re.match(r"_ZN\d+_GLOBAL__N_1\d+(k_\w+?)I(.*?)EEvNS", name)
    if not mangled:
        return None
    args = re.sub(r"L[ib](\d+)E", r"\1, ", mangled.group(2)).replace("DF16b", "bf16")
    return f"{mangled.group(1)}<{args}>"


def table(path, passes):
    """A row for each kernel and grid of a case: a kernel's calls come `passes` to a case."""
    kernels, seen = {}, {}
    for r in sorted(csv.DictReader(open(path)), key=lambda r: int(r["Start_Timestamp"])):
        name = plain_name(r["Kernel_Name"])
        if not name:
            continue
        grid, wg = int(r["Grid_Size_X"]), int(r["Workgroup_Size_X"])
        key = name, grid // wg, wg
        seen[key] = seen.get(key, -1) + 1
        key += (seen[key] // passes,)
        kernels.setdefault(key, []).append((int(r["End_Timestamp"]) - int(r["Start_Timestamp"])) / 1e3)
    print("| kernel | workgroups | threads | calls | median | least |\n|---|---|---|---|---|---|")
    for (name, groups, wg, _), us in kernels.items():
        us.sort()
        print(f"| `{name}` | {groups} | {wg} | {len(us)} | {us[len(us) // 2]:.2f} | {us[0]:.2f} |")


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawTextHelpFormatter)
    p.add_argument("--table", metavar="CSV")
    p.add_argument("--more", action="store_true")
    p.add_argument("--only", default="")
    p.add_argument("--passes", type=int, default=20)
    args = p.parse_args()
    table(args.table, args.passes) if args.table else run(args)

"""What the planner of the linear and gated products chooses (csrc/linear_plan.h, host code
without HIP), compiled by itself.  A variant is a tuple that names the kernel's form:

  (type, product, "one row")
  (type, product, "few rows", blocks of 16 rows, waves a workgroup, split or whole)
  (type, product, tile rows, tile columns, split or whole)
  (type, product, "few-rows gradients", rows of the kernel, split or whole)

  (type, "dx and dw" or "glu dx and dw", "one grid" or "two grids")

type fp32 or bf16; product linear, glu (forward), and dx, dw, glu dx, glu dw.  With `deep`, the
tiled forms count only where a workgroup has at least 10 steps of its contraction, so that its
ring of operands goes round (it holds at most six).
"""
from __future__ import annotations

import ctypes
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SHIM = r"""
#include "linear_plan.h"
using namespace ada;
extern "C" {
// {tile rows, tile columns, splits, 1 for one row or 2 for few rows, two waves for few rows}
void forward(int64_t rows, int64_t n, int64_t k, int gated, int esz, int32_t* out) {
  const Plan p = plan_forward(rows, n, k, gated, esz);
  out[0] = kTileRows[p.tile], out[1] = kTileCols[p.tile], out[2] = p.splits;
  out[3] = rows == 1 ? 1 : few_rows_sizes(rows, n, k, gated, esz) ? 2 : 0;
  out[4] = few_rows_two_waves(n, k, gated, static_cast<int>((rows + 15) / 16), esz);
}
// {few-rows kernel, together, and for dx and dw: tile rows, tile columns, splits}
void gradients(int64_t rows, int64_t n, int64_t k, int act, int gated, int esz, int32_t* out, int64_t* bytes) {
  const GradPlan g = plan_grad(rows, n, k, act, gated, esz);
  out[0] = g.few, out[1] = g.pair.together;
  for (int i = 0; i < 2; ++i) {
    const Plan& p = g.pair.plan[i];
    out[2 + 3 * i] = kTileRows[p.tile], out[3 + 3 * i] = kTileCols[p.tile], out[4 + 3 * i] = p.splits;
  }
  *bytes = g.total;
}
}
"""


def compile_planner(folder):
    src, lib = os.path.join(folder, "planner.cpp"), os.path.join(folder, "planner.so")
    with open(src, "w") as f:
        f.write(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-Wno-unused-function", "-fPIC", "-shared", "-I",
                    os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "weight_merge_amd", "csrc"), src, "-o", lib],
                   check=True)
    so = ctypes.CDLL(lib)
    so.forward.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int32] * 2 + [ctypes.POINTER(ctypes.c_int32)]
    so.gradients.argtypes = ([ctypes.c_int64] * 3 + [ctypes.c_int32] * 3
                             + [ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int64)])
    so.forward.restype = so.gradients.restype = None
    return so


def _cut(splits):
    return "split" if splits > 1 else "whole"


def _steps(depth, dtype, splits):
    return -(-depth * (2 if dtype == "bf16" else 4) // 128) // splits


def forward_variants(so, rows, n, k, gated, dtype, deep=False):
    out = (ctypes.c_int32 * 5)()
    so.forward(rows, n, k, int(gated), 2 if dtype == "bf16" else 4, out)
    name = "glu" if gated else "linear"
    if out[3] == 1:
        return {(dtype, name, "one row")}
    if out[3] == 2:
        blocks = -(-rows // 16)
        waves = 2 if out[4] else 8 if blocks == 1 and not gated else 4
        return {(dtype, name, "few rows", blocks, waves, _cut(out[2]))}
    if deep and _steps(k, dtype, out[2]) < 10:
        return set()
    return {(dtype, name, out[0], out[1], _cut(out[2]))}


def gradient_variants(so, rows, n, k, gated, dtype, deep=False):
    out, total = (ctypes.c_int32 * 8)(), ctypes.c_int64()
    so.gradients(rows, n, k, 2, int(gated), 2 if dtype == "bf16" else 4, out, ctypes.byref(total))
    names = ("glu dx", "glu dw") if gated else ("dx", "dw")
    if out[0]:
        of = 16 if rows <= 16 else 32 if rows <= 32 else 64
        return {(dtype, names[0], "few-rows gradients", of, _cut(out[4])), (dtype, names[1], "few-rows gradients", of, "whole")}
    got = {(dtype, names[0] + " and dw", "one grid" if out[1] else "two grids")}
    for i, depth in enumerate(((2 if gated else 1) * n, rows)):
        if not deep or _steps(depth, dtype, out[4 + 3 * i]) >= 10:
            got.add((dtype, names[i], out[2 + 3 * i], out[3 + 3 * i], _cut(out[4 + 3 * i])))
    return got

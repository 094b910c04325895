"""Which kernel a 2:4 product on 4-bit codes takes: the library's own rule (csrc/mxfp4_plan.h, host code without
the GPU's), compiled by the host compiler, and sizes that reach every form of it."""
import ctypes
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
UNITS = 256                                                          # compute units of an MI355X

_SOURCE = """
#include "mxfp4_plan.h"
using namespace slope;
extern "C" void few(int64_t T, int64_t K, int64_t N, int64_t scratch, int64_t units, int64_t* out) {
  const int64_t stages = up(K, 128);
  const FewPlan p = few_plan(T, N, stages, most_parts(T, N, stages, scratch), units);
  out[0] = p.tokens; out[1] = p.wide; out[2] = p.one; out[3] = p.parts;
}
extern "C" void many(int64_t T, int64_t K, int64_t N, int64_t units, int64_t* out) {
  const ManyPlan p = many_plan(T, N, up(K, 128), units);
  out[0] = (int64_t)p.kernel; out[1] = p.rows_full;
}
"""


def compile_rule(folder):
    src, lib = os.path.join(folder, "plan.cpp"), os.path.join(folder, "plan.so")
    with open(src, "w") as f:
        f.write(_SOURCE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-Wall", "-Werror", "-Wno-unused-function",
                    "-I", os.path.join(ROOT, "sparse_gemm_02_amd", "csrc"), src, "-o", lib], check=True)
    rule = ctypes.CDLL(lib)
    i64, p64 = ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)
    rule.few.argtypes, rule.few.restype = [i64] * 5 + [p64], None
    rule.many.argtypes, rule.many.restype = [i64] * 4 + [p64], None
    return rule


def form(rule, T, K, N, scratch):
    """The form of a call as text: for up to 64 tokens tokens a block, rows a block (with "+" where a compute unit has
    more than one block and that matters), parts of K and whether the weight's loads are non-temporal; above, the
    kernel and which tiles of it there are."""
    out = (ctypes.c_int64 * 4)()
    nt = " nt" if -(-N // 64) * -(-K // 128) * 3328 >= 64 << 20 else ""
    if T <= 64:
        rule.few(T, K, N, scratch, UNITS, out)
        tokens, wide, one, parts = out
        if tokens == 0:
            return "tiles 128x64"
        more = not one and (tokens == 8 and not wide or tokens > 8 and wide)
        text = f"{tokens} tokens, {64 if wide else 32}{'+' if more else ''} rows" + (", parts" if parts > 1 else "")
        return text + (nt if T <= tokens else "")
    rule.many(T, K, N, UNITS, out)
    if out[0] < 2:
        return ("direct 32", "direct 64")[out[0]]
    if out[0] < 4:
        return ("tiles 128x64", "tiles 256x128")[out[0] - 2]
    rows = -(-N // 256)
    return "tiles 256x256" if out[1] == rows else "eight-wave tiles 256x128" if out[1] == 0 else "tiles 256x256, then 256x128"


# (T, K, N) and the form that the call takes with the workspace that it asks for.  K is long enough for every ring
# of LDS slots to go round several times, and odd in stages or ragged in rows and tokens where that matters.
FORMS = [
    (5, 4112, 260, "8 tokens, 32 rows"),
    (1, 28816, 6148, "8 tokens, 32 rows nt"),
    (3, 2064, 16452, "8 tokens, 32+ rows"),
    (8, 5136, 32772, "8 tokens, 32+ rows nt"),
    (7, 2064, 8260, "8 tokens, 64 rows"),
    (2, 20496, 8196, "8 tokens, 64 rows nt"),
    (6, 16400, 36, "8 tokens, 64 rows, parts"),
    (1, 327696, 516, "8 tokens, 64 rows, parts nt"),
    (9, 4112, 132, "16 tokens, 32 rows"),
    (9, 5136, 32772, "16 tokens, 32 rows nt"),
    (13, 4112, 8196, "16 tokens, 64 rows"),
    (11, 20496, 8196, "16 tokens, 64 rows nt"),
    (13, 12304, 36, "16 tokens, 64 rows, parts"),
    (15, 327696, 516, "16 tokens, 64 rows, parts nt"),
    (10, 4112, 27652, "16 tokens, 64+ rows"),
    (16, 9232, 27652, "16 tokens, 64+ rows nt"),
    (16, 28816, 8196, "16 tokens, 64+ rows, parts nt"),
    (19, 4112, 132, "32 tokens, 32 rows"),
    (17, 28816, 6148, "32 tokens, 32 rows nt"),
    (31, 4112, 8260, "32 tokens, 64 rows"),
    (18, 20496, 8196, "32 tokens, 64 rows nt"),
    (29, 9232, 36, "32 tokens, 64 rows, parts"),
    (21, 327696, 516, "32 tokens, 64 rows, parts nt"),
    (32, 4112, 16388, "32 tokens, 64+ rows"),
    (30, 9232, 27652, "32 tokens, 64+ rows nt"),
    (29, 20496, 8196, "32 tokens, 64+ rows, parts nt"),
    (50, 4112, 36, "64 tokens, 32 rows"),
    (33, 28816, 6148, "64 tokens, 32 rows nt"),
    (64, 4112, 8196, "64 tokens, 64 rows"),
    (35, 16400, 10308, "64 tokens, 64 rows nt"),
    (61, 16400, 260, "64 tokens, 64 rows, parts"),
    (47, 28816, 6148, "64 tokens, 64 rows, parts nt"),
    (60, 4112, 16388, "64 tokens, 64+ rows"),
    (64, 9232, 27652, "64 tokens, 64+ rows nt"),
    (61, 20496, 6148, "64 tokens, 64+ rows, parts"),
    (64, 20496, 8196, "64 tokens, 64+ rows, parts nt"),
    (200, 4624, 516, "direct 32"),
    (777, 2064, 2308, "direct 64"),
    (1000, 768, 2304, "tiles 128x64"),
    (257, 4624, 9220, "tiles 128x64"),
    (129, 1168, 24004, "tiles 128x64"),
    (520, 2320, 9220, "tiles 256x128"),
    (700, 2320, 16388, "tiles 256x256"),
    (1030, 1168, 9220, "tiles 256x256"),
    (2100, 2320, 9220, "tiles 256x256, then 256x128"),
    (1300, 4624, 9220, "tiles 256x256"),
]

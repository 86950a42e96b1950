"""The plan that the library takes for a size (csrc/fp4_plan.h, compiled by itself), and sizes that reach every variant of
the 4-bit kernels between them (test_fp4_plan_host.py says so)."""
import ctypes
import functools
import os
import subprocess
import tempfile

from conftest import ROOT

# (M, N, K, elements before a row of y, elements behind it); rows of y start on 16-byte boundaries where the two and N
# add up to a multiple of 8 and nothing is before them
PAIRS = [
    # one pair to a tile: 384, 256, 192, 128 and 64 weight rows, aligned and off, one tile to a pair and several
    (1700, 8027, 600, 0, 5), (300, 9541, 600, 0, 3), (260, 22144, 3621, 1, 0), (270, 10501, 3400, 0, 0),
    (400, 14701, 300, 0, 3), (70, 14328, 71, 0, 0), (1000, 9000, 4096, 1, 2), (130, 14710, 257, 0, 0),
    (1017, 7077, 72, 0, 3), (71, 10001, 300, 0, 7), (900, 7069, 130, 0, 0), (70, 10417, 129, 2, 1),
    (300, 9977, 130, 0, 7), (72, 4763, 129, 0, 5), (275, 9967, 129, 1, 0), (74, 4751, 300, 0, 0),
    (20000, 60, 100, 0, 4), (66, 77, 128, 0, 3), (3862, 530, 64, 0, 0), (65, 66, 300, 0, 1),
    # two and four pairs to a tile
    (69, 69, 1900, 0, 3), (73, 71, 2100, 1, 0), (66, 73, 4200, 0, 7), (66, 73, 4300, 0, 0),
    (67, 2100, 1900, 0, 4), (69, 2130, 1900, 0, 1), (73, 1161, 4300, 0, 7), (66, 1200, 4300, 1, 0),
]

# (M, N, K): 16, 32 and 64 token columns, one to eight CTAs to a tile
FEW = [(m, n, k) for ms in ((1, 5, 9, 16), (17, 24, 31, 32), (33, 41, 57, 64))
       for m, (n, k) in zip(ms, ((300, 500), (513, 1100), (129, 2100), (300, 4200)))]
FEW += [(16, 20000, 2560), (32, 20000, 1300), (64, 10000, 2560)]

# (rows, K, elements behind a row): quantised and read back in patches of 64 rows; off 16-byte boundaries, on 32-byte
# ones, and on 16-byte ones (of 16-bit types).  The last 128-row band holds 26 or 66 rows
PATCHES = [(18970, 257, 0), (19010, 300, 20), (19010, 300, 12)]

SHIM = """
#include "fp4_plan.h"
extern "C" {
int small_tokens() { return bitnet::kFp4SmallTokens; }
int split(int64_t M, int64_t N, int64_t K) { return bitnet::fp4_split(M, N, K); }
int pair(int64_t M, int64_t N, int64_t K, int format, int vec) {
    const bitnet::Fp4PairPlan p = bitnet::fp4_pair_plan(M, N, K, format, vec != 0);
    return p.width * 16 + p.split;
}
int patch_rows(int64_t rows, int64_t K) { return bitnet::fp4_patch_rows(rows, K); }
}
"""


@functools.lru_cache(None)
def library():
    with tempfile.TemporaryDirectory() as d:
        src, so = os.path.join(d, "plan.cpp"), os.path.join(d, "plan.so")
        with open(src, "w", encoding="utf-8") as f:
            f.write(SHIM)
        subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-Wall", "-Werror",
                        "-I", os.path.join(ROOT, "include"),
                        "-I", os.path.join(ROOT, "ternary_weight_bit_w2a8_b200", "csrc"), src, "-o", so], check=True)
        lib = ctypes.CDLL(so)
    i64 = ctypes.c_int64
    lib.split.argtypes = [i64, i64, i64]
    lib.pair.argtypes = [i64, i64, i64, ctypes.c_int, ctypes.c_int]
    lib.patch_rows.argtypes = [i64, i64]
    return lib


def pair_plan(M, N, K, fmt, aligned):
    """(weight rows of a tile, pairs to a tile, whether a pair of the 74 takes several tiles)."""
    width, split = divmod(library().pair(M, N, K, fmt, int(aligned)), 16)
    return width, split, split == 1 and -(-M // 256) * -(-N // width) > 74

"""Which kernel instances the 8-bit calls take (the rules of csrc/i8_gemm.hip, i8_thin.hip and i8_quant.hip, written
down once more, on 256 compute units), the cases that join those of test_gpu_i8.py and test_gpu_i8_instances.py, and the
instances that the built library holds.
"""
import re

from fp32_sgemm_f32_amd import LIB_PATH

F32, BF16, F16 = 0, 1, 2
TYPES = (F32, BF16, F16)
CUS = 256


def ld(cols):
    return -(-cols // 128) * 128


def piece_rows(n):
    return -(-n // 32) * 64


def built(kernel):
    """Template arguments of each instance of a kernel in the library, as whole numbers, tiles' first."""
    with open(LIB_PATH, "rb") as f:
        text = f.read()
    name = re.compile(rb"_ZN5sgemm12_GLOBAL__N_1%d%sI(\w+?)EEv" % (len(kernel), kernel.encode()))
    found = set()
    for m in set(name.findall(text)):
        args = tuple(int(v.replace(b"n", b"-")) for v in re.findall(rb"L[ib](n?\d+)E", m + b"E"))
        found.add(args[:6] + args if b"S3_" in m else args)      # the second tile is the first
    return found


# ---- the product: (BM, BN, waves, waves, stages, sets of waves), type, down, pieces ----

T256, T256x128, T128, T128_DEEP = (256, 256, 2, 4, 2, 1), (256, 128, 4, 4, 3, 1), (128, 128, 4, 2, 2, 1), (128, 128, 4, 2, 4, 1)
T64, T64x32, T32 = (64, 64, 2, 2, 4, 1), (64, 32, 2, 1, 4, 2), (32, 32, 1, 1, 4, 2)
PAIRS = {T256: T256, T128: (128, 128, 2, 4, 2, 1), T128_DEEP: (128, 128, 2, 4, 4, 1), T64: (128, 64, 2, 2, 3, 1)}
T64_THIRD, PAIRS_THIRD = (64, 64, 2, 2, 3, 1), (128, 64, 2, 2, 2, 1)
LARGE = (T256, T256x128, T128)


def tiles(m, n, bm, bn):
    return -(-m // bm) * -(-n // bn)


def tile(rows, n, pairs=False):
    """Of a product with `rows` rows of A (a pair counts as two)."""
    whole = tiles(rows, n, 256, 256)
    if whole >= CUS and 4 * -(-whole // CUS) * CUS <= 5 * whole:
        return T256
    if not pairs and min(rows, n) <= 32:
        return T32
    if tiles(rows, n, 128, 128) > CUS:
        return T256x128 if not pairs and tiles(rows, n, 256, 128) <= CUS else T128
    if 2 * tiles(rows, n, 128, 128) > CUS:
        return T128_DEEP
    return T64x32 if not pairs and tiles(rows, n, 64, 32) <= CUS else T64


def parts(rows, n, t):
    """Whether the grid of tiles is cut into a part for each XCD."""
    m, n = -(-rows // t[0]), -(-n // t[1])
    return m >= 32 and n >= 32 and m % 2 == 0 and n % 4 == 0


def thin(m, n, k):
    return min(m, n) <= 8 and max(m, n) * ld(k) <= 1 << 27


def product(m, n, k, type):
    """Launches of i8_gemm."""
    if thin(m, n, k):
        return {("i8_thin_kernel", (2 if max(m, n) <= 32 * CUS else 4, -1))}
    return {("i8_gemm_kernel", (*tile(m, n), type, 0, 1))}


def linear(m, n, k, type):
    if m <= 8 and m * ld(k) <= 16384 and n * ld(k) <= 1 << 27:
        return {("i8_thin_kernel", (2 if n <= 32 * CUS else 4, type))}
    return rows(k, type) | product(m, n, k, type)


def rows(cols, type):
    return {("i8_rows_kernel", (type, 1 if cols <= 2048 else 4 if cols <= 8192 else 16))}


def columns(m, n, type, pieces=1):
    """Of a row-major m x n matrix, by column."""
    cols = {("i8_cols_kernel", (type, pieces, 128 if ld(n) // 128 * (ld(m) // 128) >= 512 else 64))}
    return cols if pieces == 2 else cols | {("i8_part_kernel", (type,))}


def backward(m, n, k, type):
    """Launches of i8_train_backward, and how its two products share them."""
    all = {("i8_both_kernel", (type, int(n <= 4096)))} | columns(m, n, type, 2)
    a, b = tile(m, k), tile(piece_rows(n), k, True)
    if a == T256 and b == T256:
        shared = (T256, T256)
    elif a in (T128, T256x128) and b == T128:
        shared = (T128, PAIRS[T128])
    else:
        small = tiles(m, k, 64, 64) + tiles(piece_rows(n), k, 128, 64)
        shared = None
        if a not in LARGE and b not in LARGE and small <= 5 * CUS:
            shared = (T64, PAIRS[T64]) if small <= 2 * CUS else (T64_THIRD, PAIRS_THIRD)
    if shared:
        return all | {("i8_gemm_two_kernel", (*shared[0], *shared[1], type))}
    return all | {("i8_gemm_kernel", (*a, type, 1, 1)), ("i8_gemm_kernel", (*PAIRS[b], F32, 1, 2))}


KERNELS = ("i8_gemm_kernel", "i8_gemm_two_kernel", "i8_thin_kernel", "i8_rows_kernel", "i8_cols_kernel", "i8_part_kernel", "i8_both_kernel")

# Training steps beside those of test_gpu_i8_instances.py: tiles of 128 x 128 down K in a launch of their own; more than
# 512 groups of eight rows and several runs of columns; grids cut into a part for each XCD, down K alone, in pairs alone
# and both in one launch.
STEPS = [(2185, 181, 3913), (70000, 20, 40), (4105, 4100, 40), (8192, 130, 8192), (100, 4096, 8192), (8192, 4096, 8192)]
# Prompts and full batches through a layer.
PROMPTS = [(1000, 1111, 2050), (2048, 4096, 300), (4097, 4100, 515), (8192, 513, 1000)]
# Row-major matrices by column: few tiles, and many of 128 rows.
COLUMNS = [(333, 1000), (8197, 1100)]

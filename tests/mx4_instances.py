"""Which kernel instance of the 4-bit product, the thin product and the expert
layer a call takes (the rules of csrc/mx4_gemm.hip, mx4_linear.hip and
mx4_moe.hip, written down once more), the cases of the GPU tests that reach
every one of them, and the instances that the built library holds.
"""
import re

from fp32_sgemm_f32_amd import LIB_PATH

F32, BF16, F16 = 0, 1, 2
CUS = 256


def slabs(cols):
    return -(-cols // 128)


def built(kernel):
    """Template arguments of each instance of a kernel in the library, as whole numbers."""
    with open(LIB_PATH, "rb") as f:
        text = f.read()
    name = re.compile(rb"_ZN5sgemm12_GLOBAL__N_1%d%sI(\w+?)EEv" % (len(kernel), kernel.encode()))
    return {tuple(int(v) for v in re.findall(rb"L[ib](\d+)E", m + b"E")) for m in name.findall(text)}


# ---- the product: (BM, BN, BK, waves, waves, stages, type) ----

T256, T256_ODD = (256, 256, 256, 2, 4, 2), (256, 256, 128, 2, 4, 4)
T128, T64, T64_DEEP = (128, 128, 256, 2, 4, 2), (64, 64, 256, 2, 2, 2), (64, 64, 256, 2, 2, 4)


def tiles(m, n, b):
    return -(-m // b) * -(-n // b)


def gemm_tile(m, n, k, cus=CUS):
    whole = tiles(m, n, 256)
    if whole >= cus and 4 * -(-whole // cus) * cus <= 5 * whole:
        return T256 if slabs(k) % 2 == 0 else T256_ODD
    if tiles(m, n, 128) >= cus:
        return T128
    small = tiles(m, n, 64)
    return T64_DEEP if small <= cus or small <= 2 * cus and slabs(k) >= 32 else T64


def gemm_pair(m, n, k, cus=CUS):
    """Tile of the launch that both products of a backward pass share, or None: two launches."""
    a, b = gemm_tile(m, k, n, cus), gemm_tile(n, k, m, cus)
    small = (T64, T64_DEEP)
    if a in small and b in small:
        return T64_DEEP if tiles(m, k, 64) + tiles(n, k, 64) <= cus else T64
    return a if a == b and a in (T128, T256) else None


# (m, n, k): several chunks of K, more than the ring holds, the last one whole and in part; ragged edges; two adding to C.
GEMMS = {
    (4090, 4093, 1000): T256, (4090, 4093, 1100): T256_ODD, (4090, 4093, 1536): T256, (4090, 4093, 640): T256_ODD,
    (2100, 2050, 1000): T128, (2100, 2050, 1100): T128,
    (1111, 1500, 1000): T64, (1111, 1500, 1100): T64,
    (130, 520, 1536): T64_DEEP, (130, 520, 1700): T64_DEEP, (300, 4093, 4200): T64_DEEP,
}
ADDING = [(4090, 4093, 1000), (4090, 4093, 1100), (2100, 2050, 1100), (1111, 1500, 1000), (130, 520, 1700)]
# (m, n, k) of training steps, by the launch of the backward products.
STEPS = {(4090, 4093, 4091): T256, (2100, 2050, 2060): T128, (333, 1000, 1536): T64, (130, 257, 300): T64_DEEP,
         (2100, 300, 2050): None}


# ---- the thin product: (type, slabs of a wave, token tiles, row tiles at a time, folded) ----

def linear_instance(type, m, k):
    """Of a pass of m <= 64 tokens."""
    fold = m <= 8 if type == F16 else type == F32 and m <= 5
    mt = 1 if m <= 16 else 2 if m <= 32 or type == F32 else 4
    if type == F32:
        most = 2 if mt == 1 else 1
    elif type == BF16 or fold:
        most = 4 if mt == 1 else 2
    else:
        most = 2 if mt < 4 else 1
    need = -(-slabs(k) // 8)
    ks = most if need >= most else 4 if need > 2 else 2 if need > 1 else 1
    g = 2 if mt > 1 else 1 if ks == 4 else 4
    return type, ks, mt, g, int(fold)


# One, two and four slabs a wave; K in several parts, the last one short.
LINEAR_TOKENS = [1, 7, 13, 20, 50]
LINEAR_COLS = [600, 1500, 4000, 9001]


# ---- the expert layer ----

FEW = 16


def up_instance(type, tokens, top, hidden):
    """(type, slabs of a wave, waves along K, few choices, folded)"""
    pieces = {F32: 3, BF16: 1, F16: 2}[type]
    few = tokens * top <= FEW
    fold = pieces > 1 and (few or tokens <= 16 // pieces)
    p = 1 if fold and type != F32 else pieces
    n = slabs(hidden)

    def shape():
        if few:
            return (1, 8) if n <= 8 else (4, 8) if p == 1 and n > 16 else (2, 8)
        if n <= 4:
            return (1, 2) if n <= 2 else (1, 4)
        if n <= 8:
            return (1, 8) if p == 2 else (2, 4)
        return (4, 8) if type == BF16 and n > 24 else (2, 8)

    return (type, *shape(), int(few), int(fold))


def down_instance(tokens, top, inner):
    """(slabs of a wave, waves along K, folded); None: the kernel for few choices"""
    if tokens * top <= FEW:
        return None
    fold, n = tokens <= 16 // 3, slabs(inner)
    if n <= 1:
        return 1, 1, int(fold)
    if n <= 2:
        return 1, 2, int(fold)
    if not fold:
        return 1, 8, 0
    if n <= 4:
        return 2, 2, 1
    return (3, 2, 1) if n <= 6 else (2, 4, 1) if n <= 8 else (4, 4, 1) if n <= 16 else (4, 8, 1) if n > 24 else (3, 8, 1)


# (tokens, top) of 7 experts: few choices, folded, not folded, more tokens of an expert than a tile holds.
EXPERT_TOKENS = [(1, 2), (8, 2), (3, 6), (5, 7), (9, 3), (40, 4)]
EXPERT_HIDDEN = [200, 400, 900, 1100, 1400, 1900, 2500, 3300, 4300]
EXPERT_INNER = [100, 200, 400, 700, 900, 1500, 1700, 2300, 3500, 4300]

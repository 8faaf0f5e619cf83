// C = alpha A B^T + beta C for two matrices in the microscaled 4-bit format
// (A: M x K, B: N x K), sums in fp32, on the scaled matrix instruction
// v_mfma_scale_f32_32x32x64_f8f6f4: one lane's operand is 32 codes of a row,
// one block of the format, and its scale is one byte of a register, so a
// block's scale costs no arithmetic.
//
// A workgroup computes a BM x BN tile.  The codes and the scale words of a
// K chunk (BK columns) go from global memory straight into LDS, through a
// ring of S stages; the buffer resources end where the matrix does, so rows
// beyond it read as zeros and no mask is needed (K is padded with zeros in
// the format itself).
//
// LDS of a stage: A's rows (BK / 2 bytes each), B's rows, A's scale words,
// B's scale words (slab by slab).  A row's 16-byte quad q (one block) is kept
// at quad q ^ swz(row), so that the 32 rows of an operand read fall on
// different banks.  B's rows are kept in the order that gives a lane FN
// adjacent columns of C (fragment f holds columns FN l + f), which makes the
// stores FN values wide.
//
// K order: matrix step j of a chunk multiplies the blocks 2j (lanes 0-31) and
// 2j + 1 (lanes 32-63).  The scale word of a slab is shifted by one byte for
// the upper lanes, after which byte 0 serves the slab's first step and byte 2
// its second.
//
// Ring: before the last step of chunk c, whose operands are in registers by
// then, the waves meet once (loads of chunk c + 1 landed, LDS reads of chunk
// c done), read the first operands of chunk c + 1, and load chunk c + S into
// the stage of chunk c.
//
// Bound, on random codes, by the power the chip may draw: 16384^3 runs at
// 4.3 to 4.6 PFLOP/s on different chips, on zeros at 5.5, and the matrix instructions and barriers of
// the loop alone, without loads and LDS reads, at 5.7 and 7.8.
#include <type_traits>

#include "mx4.h"

namespace sgemm {
namespace {

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 16 (4) bytes per lane from the resource's base + voff into LDS at
// m0 + 16 (4) * lane; lanes out of the resource's range leave zeros.
__device__ __forceinline__ void dma16(i32v4 rsrc, uint32_t voff, uint32_t m0v) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(voff), "s"(rsrc), "s"(m0v)
                 : "memory", "m0");
}
__device__ __forceinline__ void dma4(i32v4 rsrc, uint32_t voff, uint32_t m0v) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds" ::"v"(voff), "s"(rsrc), "s"(m0v)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// No instruction moves across.
__device__ __forceinline__ void fence_order() { __builtin_amdgcn_sched_barrier(0); }

// f(0), f(1), ... with compile-time arguments FIRST .. END - 1.
template <int FIRST, int END, class F>
__device__ __forceinline__ void each(F f) {
    if constexpr (FIRST < END) {
        f(std::integral_constant<int, FIRST>{});
        each<FIRST + 1, END>(f);
    }
}

// At most VM of this wave's loads still in flight, its LDS reads done, and
// every wave of the workgroup here.
template <int VM>
__device__ __forceinline__ void meet() {
    static_assert(VM >= 0 && VM < 64, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(VM) : "memory");
}

__device__ __forceinline__ i32v4 resource(const void *p, int64_t bytes) {
    const uint64_t a = (uint64_t)p;
    return i32v4{(int)(uint32_t)a, (int)(uint32_t)(a >> 32), (int)(uint32_t)(bytes > 0 ? bytes : 0), 0x00020000};
}
__device__ __forceinline__ void advance(i32v4 &r, int64_t bytes) {
    const uint64_t a = (((uint64_t)(uint32_t)r[1] << 32) | (uint32_t)r[0]) + (uint64_t)bytes;
    r[0] = (int)(uint32_t)a;
    r[1] = (int)(uint32_t)(a >> 32);
}

struct Args {
    const uint8_t *a, *sa, *b, *sb;
    void *c;
    int64_t ldc;
    int M, N, slabs;
    int tiles_m, tiles_n;
    float alpha, beta;
};

template <int F, class T>
struct __attribute__((packed, aligned(sizeof(T)))) Vec {   // stored at any element's address
    T v[F];
};

// A result of 256 x 256 tiles is larger than the second-level caches (it fills
// every CU): past them it goes 1 to 2 % faster (4096^3: 41.2 us against 42.1).
template <bool PAST, class V>
__device__ __forceinline__ void store(V *p, const V &v) {
    typedef uint32_t u32_any __attribute__((aligned(2)));
    typedef uint32_t u32v2_any __attribute__((ext_vector_type(2), aligned(2)));
    if constexpr (PAST && sizeof(V) == 4) __builtin_nontemporal_store(__builtin_bit_cast(uint32_t, v), (u32_any *)p);
    else if constexpr (PAST && sizeof(V) == 8) __builtin_nontemporal_store(__builtin_bit_cast(u32v2_any, v), (u32v2_any *)p);
    else *p = v;
}

template <int BM_, int BN_, int BK_, int WM_, int WN_, int S_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, BK = BK_, WM = WM_, WN = WN_, S = S_;
    static constexpr int NW = WM * WN, NT = 64 * NW;
    static constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / 32, FN = WTN / 32;
    static constexpr int ROWB = BK / 2, QPR = ROWB / 16;     // bytes and quads of a row in a stage
    static constexpr int STEPS = BK / 64, SLABS = BK / kMxSlab;
    static constexpr int A_BYTES = BM * ROWB, B_BYTES = BN * ROWB;
    static constexpr int W_LOADS = (BM + BN) / 64 * SLABS;   // loads of scale words
    static constexpr int A_PW = A_BYTES / 1024 / NW, B_PW = B_BYTES / 1024 / NW, W_PW = (W_LOADS + NW - 1) / NW;
    static constexpr int STAGE = A_BYTES + B_BYTES + W_PW * NW * 256;
    static constexpr int L = A_PW + B_PW + W_PW;             // loads of a wave per chunk
    static_assert(A_PW * NW * 1024 == A_BYTES && B_PW * NW * 1024 == B_BYTES, "a chunk's loads split evenly over the waves");
    static_assert(S * STAGE <= 160 * 1024 && (S - 2) * L < 64 && S >= 2, "LDS and vmcnt budget");
    static_assert(BM % 64 == 0 && BN % 64 == 0, "a scale load covers 64 rows of one operand");

    __device__ __forceinline__ static int swz(int r) { return QPR == 4 ? (r >> 2) & 3 : (r ^ (r >> 3)) & 7; }
    // Column of the tile that B's LDS row r holds.
    __device__ __forceinline__ static int b_col(int r) { return r / WTN * WTN + FN * (r % 32) + r % WTN / 32; }
};

// The tile of workgroup `block` of the product g.
template <class TL, int TYPE>
__device__ __forceinline__ void compute_tile(const Args &g, int block) {
    typedef typename MxType<TYPE>::T T;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / TL::WN, wn = wave % TL::WN;

    // Workgroup -> tile: each XCD (workgroups w, w + 8, ...) takes a
    // contiguous run of tiles, which go down columns of 8-row groups.
    int tm, tn;
    {
        const int tiles = g.tiles_m * g.tiles_n, per = tiles >> 3, rest = tiles & 7;
        const int x = block & 7, y = block >> 3;
        const int t = x * per + (x < rest ? x : rest) + y;
        const int group = 8 * g.tiles_n, gi = t / group, first = gi * 8;
        const int rows = g.tiles_m - first < 8 ? g.tiles_m - first : 8;
        tm = first + (t - gi * group) % rows;
        tn = (t - gi * group) / rows;
    }
    const int m0 = tm * TL::BM, n0 = tn * TL::BN;
    const int64_t rowb = (int64_t)g.slabs * kMxSlabBytes;
    const int64_t plane_a = mx_plane_rows(g.M) * 4, plane_b = mx_plane_rows(g.N) * 4;
    const int chunks = (g.slabs + TL::SLABS - 1) / TL::SLABS;

    // Sources of this wave's loads.  The resources end with the tile's last
    // real row.  For BK = 256 a chunk may reach one slab past its rows' end
    // (odd slab counts): load_chunk masks those lanes.
    const int am = g.M - m0 < TL::BM ? g.M - m0 : TL::BM, bn = g.N - n0 < TL::BN ? g.N - n0 : TL::BN;
    i32v4 ra = resource(g.a + m0 * rowb, am * rowb), rb = resource(g.b + n0 * rowb, bn * rowb);
    uint32_t va[TL::A_PW], vb[TL::B_PW];
    bool ua[TL::A_PW], ub[TL::B_PW];   // BK = 256: the lane's block lies in the chunk's second slab
#pragma unroll
    for (int i = 0; i < TL::A_PW; ++i) {
        const int r = (wave * TL::A_PW + i) * (1024 / TL::ROWB) + lane / TL::QPR;
        const int q = (lane % TL::QPR) ^ TL::swz(r);
        va[i] = (uint32_t)(r * rowb) + 16 * q;
        ua[i] = q >= 4;
    }
#pragma unroll
    for (int i = 0; i < TL::B_PW; ++i) {
        const int r = (wave * TL::B_PW + i) * (1024 / TL::ROWB) + lane / TL::QPR;
        const int q = (lane % TL::QPR) ^ TL::swz(r);
        vb[i] = (uint32_t)(TL::b_col(r) * rowb) + 16 * q;
        ub[i] = q >= 4;
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;

    // Loads i = 0 .. L-1 of a chunk, A's first; `next_chunk` moves the
    // resources on by one chunk.  From the last chunk on they are empty.
    int lc = 0;   // the chunk that the resources stand at
    int left_a = (int)(am * rowb), left_b = (int)(bn * rowb);
    ra[2] = chunks > 0 ? left_a : 0;
    rb[2] = chunks > 0 ? left_b : 0;
    i32v4 rw[TL::W_PW];
    uint32_t vw[TL::W_PW];
    int64_t step_w[TL::W_PW];
#pragma unroll
    for (int i = 0; i < TL::W_PW; ++i) {
        // Load w of the scale words: 64 rows of one operand in one slab.
        const int w = wave * TL::W_PW + i;
        constexpr int PER = (TL::BM + TL::BN) / 64;
        const int slab = w / PER, u = w % PER;
        const bool is_a = u < TL::BM / 64;
        const int64_t plane = is_a ? plane_a : plane_b;
        rw[i] = resource((is_a ? g.sa + m0 * 4 : g.sb + n0 * 4) + slab * plane, plane - (is_a ? m0 : n0) * 4);
        vw[i] = 4 * (is_a ? u * 64 + lane : TL::b_col(u * 64 - TL::BM + lane));
        step_w[i] = plane * TL::SLABS;
        // (past the last slab, and past the chunk's words where the waves do not divide them: nothing)
        if (slab >= g.slabs || w >= TL::W_LOADS) rw[i][2] = 0;
    }
    auto load_one = [&](auto ic, int stage) {
        constexpr int i = decltype(ic)::value;
        const uint32_t base = lds0 + stage * TL::STAGE;
        // A slab past the row's end (BK = 256, odd slab counts): no lane loads it.
        const bool half = TL::SLABS == 2 && 2 * lc + 1 >= g.slabs;
        if constexpr (i < TL::A_PW) {
            uint32_t v = va[i];
            if constexpr (TL::SLABS == 2) v = half && ua[i] ? 0x80000000u : v;
            dma16(ra, v, base + (wave * TL::A_PW + i) * 1024);
        } else if constexpr (i < TL::A_PW + TL::B_PW) {
            constexpr int k = i - TL::A_PW;
            uint32_t v = vb[k];
            if constexpr (TL::SLABS == 2) v = half && ub[k] ? 0x80000000u : v;
            dma16(rb, v, base + TL::A_BYTES + (wave * TL::B_PW + k) * 1024);
        } else if constexpr (i < TL::L) {
            constexpr int k = i - TL::A_PW - TL::B_PW;
            dma4(rw[k], vw[k], base + TL::A_BYTES + TL::B_BYTES + (wave * TL::W_PW + k) * 256);
        }
    };
    auto next_chunk = [&] {
        ++lc;
        left_a -= TL::ROWB;
        left_b -= TL::ROWB;
        advance(ra, TL::ROWB);
        advance(rb, TL::ROWB);
        ra[2] = lc < chunks ? left_a : 0;
        rb[2] = lc < chunks ? left_b : 0;
#pragma unroll
        for (int i = 0; i < TL::W_PW; ++i) {
            advance(rw[i], step_w[i]);
            if (lc * TL::SLABS + (wave * TL::W_PW + i) / ((TL::BM + TL::BN) / 64) >= g.slabs) rw[i][2] = 0;
        }
    };
    auto load_chunk = [&](int stage) {
        each<0, TL::L>([&](auto i) { load_one(i, stage); });
        next_chunk();
    };

    f32v16 acc[TL::FM][TL::FN];
#pragma unroll
    for (int i = 0; i < TL::FM; ++i)
#pragma unroll
        for (int k = 0; k < TL::FN; ++k)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][k][r] = 0.0f;

    // Operand reads: lane l takes row l % 32 of a fragment, block 2 j + l / 32.
    const int fr = lane & 31, h = lane >> 5;
    struct Ops {
        i32v4 a[TL::FM], b[TL::FN];
    };
    struct Words {
        uint32_t a[TL::SLABS][TL::FM], b[TL::SLABS][TL::FN];
    };
    auto read_ops = [&](Ops &o, int stage, int j) {
        const uint8_t *st = lds + stage * TL::STAGE;
#pragma unroll
        for (int i = 0; i < TL::FM; ++i) {
            const int r = wm * TL::WTM + 32 * i + fr;
            o.a[i] = *(const i32v4 *)(st + r * TL::ROWB + 16 * ((2 * j + h) ^ TL::swz(r)));
        }
#pragma unroll
        for (int i = 0; i < TL::FN; ++i) {
            const int r = wn * TL::WTN + 32 * i + fr;
            o.b[i] = *(const i32v4 *)(st + TL::A_BYTES + r * TL::ROWB + 16 * ((2 * j + h) ^ TL::swz(r)));
        }
    };
    auto read_words = [&](Words &w, int stage) {
        const uint32_t *st = (const uint32_t *)(lds + stage * TL::STAGE + TL::A_BYTES + TL::B_BYTES);
#pragma unroll
        for (int s = 0; s < TL::SLABS; ++s) {
#pragma unroll
            for (int i = 0; i < TL::FM; ++i)
                w.a[s][i] = st[s * (TL::BM + TL::BN) + wm * TL::WTM + 32 * i + fr] >> (8 * h);
#pragma unroll
            for (int i = 0; i < TL::FN; ++i)
                w.b[s][i] = st[s * (TL::BM + TL::BN) + TL::BM + wn * TL::WTN + 32 * i + fr] >> (8 * h);
        }
    };
    // Products p = 0 .. FM FN - 1 of matrix step j, row by row.
    auto multiply = [&](const Ops &o, const Words &w, auto jc, auto pc) {
        constexpr int j = decltype(jc)::value, i = decltype(pc)::value / TL::FN, k = decltype(pc)::value % TL::FN;
        const i32v8 x = __builtin_shufflevector(o.a[i], o.a[i], 0, 1, 2, 3, -1, -1, -1, -1);
        const i32v8 y = __builtin_shufflevector(o.b[k], o.b[k], 0, 1, 2, 3, -1, -1, -1, -1);
        acc[i][k] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, acc[i][k], 4, 4, (j & 1) * 2, (int)w.a[j / 2][i],
                                                                    (j & 1) * 2, (int)w.b[j / 2][k]);
    };
    constexpr int NP = TL::FM * TL::FN;

    // Chunks 0 .. S-1 go out, the last of them only in part; from then on
    // every iteration adds one.  A wave that issues loads back to back waits
    // for the address unit with its products behind it: so a chunk's loads
    // are spread over the products of a last step (the first EARLY of them)
    // and of the next chunk's first.  Past the last chunk nothing is in
    // range, but the loads are issued all the same (they leave zeros): the
    // waits count them.
    constexpr int HEAD = NP / 4 > 0 ? NP / 4 : 1;
    constexpr int EARLY = TL::L * (NP - HEAD) / (2 * NP - HEAD);
    for (int c = 0; c < TL::S - 1; ++c) load_chunk(c);
    each<0, EARLY>([&](auto i) { load_one(i, TL::S - 1); });
    meet<(TL::S - 2) * TL::L + EARLY>();
    Ops o[2];
    Words w[2];
    read_ops(o[0], 0, 0);
    read_words(w[0], 0);
    int stage = 0, freed = TL::S - 1;
    for (int c = 0; c < chunks; ++c) {
        const int next = stage + 1 == TL::S ? 0 : stage + 1;
        each<0, TL::STEPS - 1>([&](auto jc) {
            constexpr int j = decltype(jc)::value;
            read_ops(o[(j + 1) & 1], stage, j + 1);
            fence_order();
            each<0, NP>([&](auto p) {
                multiply(o[j & 1], w[0], jc, p);
                if constexpr (j == 0) {
                    constexpr int first = EARLY + p * (TL::L - EARLY) / NP, end = EARLY + (p + 1) * (TL::L - EARLY) / NP;
                    each<first, end>([&](auto i) { load_one(i, freed); });
                    fence_order();
                }
            });
            if constexpr (j == 0) next_chunk();
            fence_order();
        });
        // The last step's operands are in registers once this wave has met
        // the others; behind its products go the next chunk's first operands
        // and the first loads into the stage that is free now.
        meet<(TL::S - 2) * TL::L>();
        constexpr int j = TL::STEPS - 1;
        constexpr std::integral_constant<int, j> last{};
        each<0, HEAD>([&](auto p) { multiply(o[j & 1], w[0], last, p); });
        fence_order();
        read_ops(o[0], next, 0);
        read_words(w[1], next);
        fence_order();
        each<HEAD, NP>([&](auto p) {
            multiply(o[j & 1], w[0], last, p);
            constexpr int first = (p - HEAD) * EARLY / (NP - HEAD), end = (p - HEAD + 1) * EARLY / (NP - HEAD);
            each<first, end>([&](auto i) { load_one(i, stage); });
            fence_order();
        });
        w[0] = w[1];
        freed = stage;
        stage = next;
    }
    // Loads still in flight write this workgroup's LDS: let them land.
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");

    // Lane l holds columns FN (l % 32) + 0 .. FN-1 of its wave's tile, rows
    // 8 (r / 4) + 4 (l / 32) + r % 4 of each fragment.
    const int col = n0 + wn * TL::WTN + TL::FN * fr;
    const bool wide = col + TL::FN <= g.N;
#pragma unroll
    for (int i = 0; i < TL::FM; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int row = m0 + wm * TL::WTM + 32 * i + 8 * (r / 4) + 4 * h + r % 4;
            if (row >= g.M) continue;
            T *p = (T *)g.c + row * g.ldc + col;
            if (wide) {
                Vec<TL::FN, T> out;
                if (g.beta != 0.0f) {
                    const Vec<TL::FN, T> old = *(const Vec<TL::FN, T> *)p;
#pragma unroll
                    for (int k = 0; k < TL::FN; ++k)
                        out.v[k] = MxType<TYPE>::from(g.alpha * acc[i][k][r] + g.beta * MxType<TYPE>::load(&old.v[k]));
                } else {
#pragma unroll
                    for (int k = 0; k < TL::FN; ++k) out.v[k] = MxType<TYPE>::from(g.alpha * acc[i][k][r]);
                }
                store<TL::BM >= 256>((Vec<TL::FN, T> *)p, out);
            } else {
#pragma unroll
                for (int k = 0; k < TL::FN; ++k)
                    if (col + k < g.N) {
                        float v = g.alpha * acc[i][k][r];
                        if (g.beta != 0.0f) v += g.beta * MxType<TYPE>::load(p + k);
                        p[k] = MxType<TYPE>::from(v);
                    }
            }
        }
}

template <class TL, int TYPE>
__global__ __launch_bounds__(TL::NT, 1) void mx4_gemm_kernel(Args g) {
    compute_tile<TL, TYPE>(g, blockIdx.x);
}

// Two products in one launch: the first `head` workgroups compute g, or k if
// k_first, the others the other.
template <class TL, int TYPE>
__global__ __launch_bounds__(TL::NT, 1) void mx4_gemm_two_kernel(Args g, Args k, int head, bool k_first) {
    const bool early = (int)blockIdx.x < head;
    const int block = early ? blockIdx.x : blockIdx.x - head;
    if (early == k_first) compute_tile<TL, SGEMM_TYPE_F32>(k, block);
    else compute_tile<TL, TYPE>(g, block);
}

// Waves 2 x 4 everywhere but in the smallest: two waves on a SIMD cover each
// other's waits (2 x 2 waves of 128 x 128 read a third less LDS and were 4 to
// 12 % slower).
typedef Tile<256, 256, 256, 2, 4, 2> T256;       // 8 waves of 128 x 64, 136 KiB
typedef Tile<256, 256, 128, 2, 4, 4> T256Odd;    // the same, 136 KiB
typedef Tile<128, 128, 256, 2, 4, 2> T128;       // 8 waves of 64 x 32, 68 KiB: two workgroups on a CU
typedef Tile<64, 64, 256, 2, 2, 2> T64;          // 4 waves of 32 x 32, 34 KiB: four workgroups on a CU
typedef Tile<64, 64, 256, 2, 2, 4> T64Deep;      // the same, 68 KiB

template <class TL>
Args arguments(const MxGemmJob &j) {
    return Args{j.a, j.sa, j.b, j.sb, j.c, j.ldc, j.M, j.N, mx_slabs(j.K), (int)(((int64_t)j.M + TL::BM - 1) / TL::BM),
                (int)(((int64_t)j.N + TL::BN - 1) / TL::BN), j.alpha, j.beta};
}

template <class TL, int TYPE>
hipError_t launch_tile(const MxGemmJob &j, hipStream_t s) {
    Args g = arguments<TL>(j);
    const void *k = (const void *)mx4_gemm_kernel<TL, TYPE>;
    const int bytes = TL::S * TL::STAGE;
    void *params[] = {&g};
    return hipLaunchKernel(k, dim3((unsigned)(g.tiles_m * g.tiles_n)), dim3(TL::NT), params, bytes, s);
}

template <class TL, int TYPE>
hipError_t launch_two(const MxGemmJob &first, const MxGemmJob &second, hipStream_t s) {
    Args g = arguments<TL>(first), h = arguments<TL>(second);
    bool h_first = h.slabs > g.slabs;   // the longer tiles begin
    const int tiles_g = g.tiles_m * g.tiles_n, tiles_h = h.tiles_m * h.tiles_n;
    int head = h_first ? tiles_h : tiles_g;
    void *params[] = {&g, &h, &head, &h_first};
    return hipLaunchKernel((const void *)mx4_gemm_two_kernel<TL, TYPE>, dim3((unsigned)(tiles_g + tiles_h)), dim3(TL::NT), params,
                           TL::S * TL::STAGE, s);
}

int64_t tiles_of(const MxGemmJob &j, int b) { return (((int64_t)j.M + b - 1) / b) * (((int64_t)j.N + b - 1) / b); }

enum Kind { k256, k256Odd, k128, k64, k64Deep };

Kind kind_of(const MxGemmJob &j, int num_cus) {
    const auto tiles = [&](int b) { return tiles_of(j, b); };
    // The largest tile that gives every CU one and whose rounds leave at most
    // a fifth of the CUs' time unused (272 tiles of 256 x 256, 4352 x 4096 x
    // 4096: 70 us, 60 in tiles of 128 x 128, two to a CU; 448 in two rounds,
    // 7000 x 4096 x 4096: 76 against 82).  A row of an even number of slabs is
    // whole 128-byte lines, which chunks of two slabs read at once (16384^3:
    // 1957 us, in chunks of one 2109); rows of an odd number split every line
    // between two such chunks (16000^3: 2042 against 1974).
    const int64_t rounds = (tiles(256) + num_cus - 1) / num_cus;
    if (tiles(256) >= num_cus && 4 * rounds * num_cus <= 5 * tiles(256))
        return mx_slabs(j.K) % 2 == 0 ? k256 : k256Odd;
    if (tiles(128) >= num_cus) return k128;
    // With one tile for a CU at most, a deep ring hides the memory's latency
    // (64 x 8192 x 8192: 13.0 us against 21.5).  Two deep rings fit on a CU: up to
    // as many tiles they pay for long K (300 x 4096 x 16384: 25.9 against 38.4, 1111
    // x 1500 x 4096: 10.5 against 12.9, 512 x 4096 x 4096: the same; but 300 x 4096 x
    // 1024: 6.3 against 6.1).  With more, further workgroups hide it (333 x 6000 x
    // 1536: 10.2 against 8.2).
    const bool deep = tiles(64) <= num_cus || (tiles(64) <= 2 * num_cus && mx_slabs(j.K) >= 32);
    return deep ? k64Deep : k64;
}

template <int TYPE>
hipError_t launch_type(const MxGemmJob &j, int num_cus, hipStream_t s) {
    switch (kind_of(j, num_cus)) {
    case k256: return launch_tile<T256, TYPE>(j, s);
    case k256Odd: return launch_tile<T256Odd, TYPE>(j, s);
    case k128: return launch_tile<T128, TYPE>(j, s);
    case k64: return launch_tile<T64, TYPE>(j, s);
    default: return launch_tile<T64Deep, TYPE>(j, s);
    }
}

// Two products that take the same tiles share a launch: no CU idles between the
// end of one and the beginning of the other (the backward pass of 2048 x 2048
// x 2048: 32.9 -> 26.3 us, of 2048 x 4096 x 2048 47.0 -> 41.6, of 16384 x 4096
// x 4096 353 -> 343).
template <int TYPE>
hipError_t launch_pair(const MxGemmJob &j, const MxGemmJob &k, int num_cus, hipStream_t s) {
    const Kind a = kind_of(j, num_cus), b = kind_of(k, num_cus);
    if (a >= k64 && b >= k64)
        return tiles_of(j, 64) + tiles_of(k, 64) <= num_cus ? launch_two<T64Deep, TYPE>(j, k, s) : launch_two<T64, TYPE>(j, k, s);
    if (a == k128 && b == k128) return launch_two<T128, TYPE>(j, k, s);
    if (a == k256 && b == k256) return launch_two<T256, TYPE>(j, k, s);
    const hipError_t e = launch_type<TYPE>(j, num_cus, s);
    return e == hipSuccess ? launch_type<SGEMM_TYPE_F32>(k, num_cus, s) : e;
}

}  // namespace

hipError_t launch_mx4_gemm(const MxGemmJob &j, int num_cus, hipStream_t s) {
    switch (j.type) {
    case SGEMM_TYPE_F32: return launch_type<SGEMM_TYPE_F32>(j, num_cus, s);
    case SGEMM_TYPE_BF16: return launch_type<SGEMM_TYPE_BF16>(j, num_cus, s);
    case SGEMM_TYPE_F16: return launch_type<SGEMM_TYPE_F16>(j, num_cus, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_mx4_gemm_two(const MxGemmJob &j, const MxGemmJob &k, int num_cus, hipStream_t s) {
    switch (j.type) {
    case SGEMM_TYPE_F32: return launch_pair<SGEMM_TYPE_F32>(j, k, num_cus, s);
    case SGEMM_TYPE_BF16: return launch_pair<SGEMM_TYPE_BF16>(j, k, num_cus, s);
    case SGEMM_TYPE_F16: return launch_pair<SGEMM_TYPE_F16>(j, k, num_cus, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace sgemm

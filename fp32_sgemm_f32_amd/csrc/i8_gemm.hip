// C = alpha A B^T + beta C for two matrices in the 8-bit integer format (A: M x
// K, B: N x K, a scale for each row), and C = alpha A B for B stored K x N
// (`down`), on v_mfma_i32_32x32x32_i8: exact 32-bit sums, scales in the
// epilogue.
//
// A workgroup computes a BM x BN tile.  Chunks of 128 along K go from global
// memory straight into LDS, through a ring of S stages; the buffer resources
// end where the matrix does, so what lies beyond reads as zeros and nothing is
// masked (A's rows are padded with zeros in the format itself; down B's rows
// beyond K meet those).
//
// LDS of a stage: A's rows (128 bytes), then B's rows (128 bytes of a column of
// C), or, down, 128 rows of BN bytes.  A lane's operand is 16 bytes along K.
// - Rows along K: quad q (16 bytes) of a row is kept at q ^ swz(row), so that
//   the 32 rows of an operand read fall on different banks.  B's rows are kept
//   in the order that gives a lane FN adjacent columns of C (fragment f holds
//   columns FN l + f): stores are FN values wide.
// - Down: ds_read_b64_tr_b8 reads 8 rows x 16 bytes across 16 lanes and gives
//   each of them a column's 8 bytes; two make an operand.  Quad q of row k is
//   kept at q ^ swz_down(k): the 8 rows x 32 columns that half a wave reads lie
//   in different banks.  A lane's columns are 32 apart.
//
// pieces = 2 (down): A's fragments come in pairs, the high and the low bytes of
// 16-bit whole numbers; a pair's sums are joined as 256 high + low.
//
// Small tiles slice K: KS sets of waves, each with a ring of its own, take every
// KS-th chunk, and the first adds up the sums.
//
// Bound, where tiles are large, by the power the chip may draw: 16384^3 runs in
// 3420 to 3700 us on different chips (2.4 to 2.6 POPS; the library's product of the
// same type, 8192^3, at 2.1), at 1.6 GHz with the matrix pipes busy in 76% of the
// cycles; on zeros, which draw less, in 2850 to 2900 (3.1), at 2.4 GHz and 61%.  The
// waves wait (for memory, at barriers) in 32% of their cycles, on zeros in 44%.
// Where tiles are small, by the loads: 60 to 85 GB/s reach a CU, of the 117 that
// such loads reach alone.  LDS conflicts: none (counters).
//
// K is not shared between workgroups: a small result of a long sum has few of
// them, and each goes through all of K (64 x 64 x 16384 18.6 us, 64 x 64 x 65536
// 61.4; a backward pass of 65536 x 64 x 64 273).
//
// Ring: before the last step of chunk c, whose operands are in registers by
// then, the waves meet once (loads of chunk c + 1 landed, LDS reads of chunk c
// done), read the first operands of chunk c + 1, and load chunk c + S into the
// stage of chunk c.
#include "i8.h"
#include "lds_dma.h"

namespace sgemm {
namespace {

typedef int i32v2 __attribute__((ext_vector_type(2)));
typedef int i32v16 __attribute__((ext_vector_type(16)));

constexpr int kChunk = 128;   // of K

struct Args {
    const int8_t *a;
    const float *sa;
    const int8_t *b;
    const float *sb;
    void *c;
    int64_t ldc;
    int M, N, K;        // M: rows of C
    int rows_a;         // rows of A (with two pieces more than M)
    int tiles_m, tiles_n;
    float alpha, beta;
};

template <int BM_, int BN_, int WM_, int WN_, int S_, int KS_ = 1>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, S = S_, KS = KS_;
    static constexpr int NW = WM * WN, NT = 64 * NW * KS;                            // waves of a set, threads of all
    static constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / 32, FN = WTN / 32;
    static constexpr int STEPS = kChunk / 32;
    static constexpr int A_BYTES = BM * kChunk, B_BYTES = BN * kChunk, STAGE = A_BYTES + B_BYTES, RING = S * STAGE;
    static constexpr int A_PW = A_BYTES / 1024 / NW, B_PW = B_BYTES / 1024 / NW, L = A_PW + B_PW;   // loads of a wave per chunk
    static_assert(A_PW * NW * 1024 == A_BYTES && B_PW * NW * 1024 == B_BYTES, "a chunk's loads split evenly over the waves");
    static_assert(KS * RING <= 160 * 1024 && (KS - 1) * BM * BN <= KS * RING / 4 && (S - 2) * L < 64 && S >= 2, "LDS and vmcnt budget");

    __device__ __forceinline__ static int swz(int r) { return (r ^ (r >> 3)) & 7; }
    // Column of the tile that B's LDS row r holds.
    __device__ __forceinline__ static int b_col(int r) { return r / WTN * WTN + FN * (r % 32) + r % WTN / 32; }
    // Rows of BN bytes: 256 / BN of them to all banks.
    __device__ __forceinline__ static int swz_down(int k) { return 2 * ((k / (256 / BN)) & (BN / 32 - 1)); }
};

// The tile of workgroup `block` of the product g.
template <class TL, int TYPE, bool DOWN, int PIECES>
__device__ __forceinline__ void compute_tile(const Args &g, int block) {
    typedef typename MxType<TYPE>::T T;
    extern __shared__ __attribute__((aligned(1024))) int8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int all = __builtin_amdgcn_readfirstlane(tid >> 6), set = all / TL::NW, wave = all % TL::NW;
    const int wm = wave / TL::WN, wn = wave % TL::WN;

    // Workgroup -> tile: each XCD (workgroups w, w + 8, ...) takes a
    // contiguous run of tiles, which go down columns of 8-row groups.  Large
    // grids are first cut into two by four parts, one for each XCD, where that
    // goes evenly: what the chip works on at a time is then as many rows as
    // columns, half of what it reads otherwise (16384^3: 3480 us against 3615; 16384
    // x 16384 x 4096 920 against 966; 8192^3 the same).
    int tm, tn;
    {
        const int x = block & 7, y = block >> 3;
        const bool parts = g.tiles_m >= 32 && g.tiles_n >= 32 && g.tiles_m % 2 == 0 && g.tiles_n % 4 == 0;
        const int pm = parts ? g.tiles_m / 2 : g.tiles_m, pn = parts ? g.tiles_n / 4 : g.tiles_n;
        const int tiles = pm * pn, per = tiles >> 3, rest = tiles & 7;
        const int t = parts ? y : x * per + (x < rest ? x : rest) + y;
        const int group = 8 * pn, gi = t / group, first = gi * 8;
        const int rows = pm - first < 8 ? pm - first : 8;
        tm = first + (t - gi * group) % rows + (parts ? (x & 1) * pm : 0);
        tn = (t - gi * group) / rows + (parts ? (x >> 1) * pn : 0);
    }
    const int m0 = tm * TL::BM, n0 = tn * TL::BN;
    const int chunks = (g.K + kChunk - 1) / kChunk;
    const int64_t rowb = (int64_t)chunks * kChunk;   // bytes of a row along K
    const int64_t downb = i8_ld(g.N);                // of a row down K

    // Sources of this wave's loads.  The resources end with the tile's last
    // real row along K; down, with the chunk's last real row.
    const int am = g.rows_a - m0 < TL::BM ? g.rows_a - m0 : TL::BM, bn = g.N - n0 < TL::BN ? g.N - n0 : TL::BN;
    i32v4 ra = resource(g.a + m0 * rowb, 0), rb = DOWN ? resource(g.b, 0) : resource(g.b + n0 * rowb, 0);
    uint32_t va[TL::A_PW], vb[TL::B_PW];
#pragma unroll
    for (int i = 0; i < TL::A_PW; ++i) {
        const int r = (wave * TL::A_PW + i) * 8 + lane / 8;
        va[i] = (uint32_t)(r * rowb) + 16 * ((lane % 8) ^ TL::swz(r));
    }
#pragma unroll
    for (int i = 0; i < TL::B_PW; ++i) {
        if constexpr (DOWN) {
            constexpr int QUADS = TL::BN / 16;
            const int at = (wave * TL::B_PW + i) * 64 + lane, k = at / QUADS;
            vb[i] = (uint32_t)(k * downb) + n0 + 16 * ((at % QUADS) ^ TL::swz_down(k));
        } else {
            const int r = (wave * TL::B_PW + i) * 8 + lane / 8;
            vb[i] = (uint32_t)(TL::b_col(r) * rowb) + 16 * ((lane % 8) ^ TL::swz(r));
        }
    }
    const int8_t *ring = lds + set * TL::RING;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) int8_t *)lds + set * TL::RING;

    // Loads i = 0 .. L-1 of a chunk, A's first; `next_chunk` moves the
    // resources on by one chunk.  From the last chunk on they are empty.
    int lc = set;   // the chunk that the resources stand at
    advance(ra, (int64_t)set * kChunk);
    advance(rb, set * (DOWN ? kChunk * downb : kChunk));
    int left_a = (int)(am * rowb) - set * kChunk, left_b = (int)(bn * rowb) - set * kChunk;
    const int whole = (int)(kChunk * downb), tail = (int)((g.K - (chunks - 1) * kChunk) * downb);   // down: bytes of a chunk, of the last
    auto limits = [&] {
        ra[2] = lc < chunks ? left_a : 0;
        if constexpr (DOWN) rb[2] = lc < chunks - 1 ? whole : lc < chunks ? tail : 0;
        else rb[2] = lc < chunks ? left_b : 0;
    };
    limits();
    auto load_one = [&](auto ic, int stage) {
        constexpr int i = decltype(ic)::value;
        const uint32_t base = lds0 + stage * TL::STAGE;
        if constexpr (i < TL::A_PW) dma16(ra, va[i], base + (wave * TL::A_PW + i) * 1024);
        else if constexpr (i < TL::L) dma16(rb, vb[i - TL::A_PW], base + TL::A_BYTES + (wave * TL::B_PW + i - TL::A_PW) * 1024);
    };
    auto next_chunk = [&] {
        lc += TL::KS;
        left_a -= TL::KS * kChunk;
        left_b -= TL::KS * kChunk;
        advance(ra, TL::KS * kChunk);
        advance(rb, TL::KS * (DOWN ? kChunk * downb : kChunk));
        limits();
    };
    auto load_chunk = [&](int stage) {
        each<0, TL::L>([&](auto i) { load_one(i, stage); });
        next_chunk();
    };

    i32v16 acc[TL::FM][TL::FN];
#pragma unroll
    for (int i = 0; i < TL::FM; ++i)
#pragma unroll
        for (int k = 0; k < TL::FN; ++k)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][k][r] = 0;

    // Operand reads: lane l takes row (down: column) l % 32 of a fragment,
    // bytes 32 j + 16 (l / 32) + 0 .. 15 of the chunk.
    const int fr = lane & 31, h = lane >> 5;
    const int tr_row = 16 * h + ((lane & 15) >> 1);   // down: the row of step 0 that this lane names
    const int tr_at = tr_row * TL::BN + 8 * (lane & 1);
    struct Ops {
        i32v4 a[TL::FM], b[TL::FN];
    };
    auto read_ops = [&](Ops &o, int stage, int j) {
        const int8_t *st = ring + stage * TL::STAGE;
#pragma unroll
        for (int i = 0; i < TL::FM; ++i) {
            const int r = wm * TL::WTM + 32 * i + fr;
            o.a[i] = *(const i32v4 *)(st + r * kChunk + 16 * ((2 * j + h) ^ TL::swz(r)));
        }
#pragma unroll
        for (int i = 0; i < TL::FN; ++i) {
            if constexpr (DOWN) {
                const int quad = (wn * TL::WTN + 32 * i) / 16 + (fr >> 4);
                typedef __attribute__((address_space(3))) i32v2 *Tr;
                const int8_t *p = st + TL::A_BYTES + 32 * j * TL::BN + tr_at + 16 * (quad ^ TL::swz_down(tr_row));
                const i32v2 lo = __builtin_amdgcn_ds_read_tr8_b64_v2i32((Tr)p);
                const i32v2 hi = __builtin_amdgcn_ds_read_tr8_b64_v2i32((Tr)(p + 8 * TL::BN));
                o.b[i] = i32v4{lo[0], lo[1], hi[0], hi[1]};
            } else {
                const int r = wn * TL::WTN + 32 * i + fr;
                o.b[i] = *(const i32v4 *)(st + TL::A_BYTES + r * kChunk + 16 * ((2 * j + h) ^ TL::swz(r)));
            }
        }
    };
    // Products p = 0 .. FM FN - 1 of a matrix step, row by row.
    auto multiply = [&](const Ops &o, auto pc) {
        constexpr int i = decltype(pc)::value / TL::FN, k = decltype(pc)::value % TL::FN;
        acc[i][k] = __builtin_amdgcn_mfma_i32_32x32x32_i8(o.a[i], o.b[k], acc[i][k], 0, 0, 0);
    };
    constexpr int NP = TL::FM * TL::FN;

    // Chunks 0 .. S-1 go out, the last of them only in part; from then on
    // every iteration adds one.  A chunk's loads are spread over the products
    // of a last step (the first EARLY of them) and of the next chunk's first:
    // a wave that issues loads back to back waits for the address unit with
    // its products behind it.  Past the last chunk nothing is in range, but
    // the loads are issued all the same (they leave zeros): the waits count
    // them.
    constexpr int HEAD = NP / 4 > 0 ? NP / 4 : 1;
    constexpr int EARLY = TL::L * (NP - HEAD) / (2 * NP - HEAD);
    for (int c = 0; c < TL::S - 1; ++c) load_chunk(c);
    each<0, EARLY>([&](auto i) { load_one(i, TL::S - 1); });
    meet<(TL::S - 2) * TL::L + EARLY>();
    Ops o[2];
    read_ops(o[0], 0, 0);
    int stage = 0, freed = TL::S - 1;
    for (int c = 0; c < chunks; c += TL::KS) {
        const int next = stage + 1 == TL::S ? 0 : stage + 1;
        each<0, TL::STEPS - 1>([&](auto jc) {
            constexpr int j = decltype(jc)::value;
            read_ops(o[(j + 1) & 1], stage, j + 1);
            fence_order();
            each<0, NP>([&](auto p) {
                multiply(o[j & 1], p);
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
        each<0, HEAD>([&](auto p) { multiply(o[j & 1], p); });
        fence_order();
        read_ops(o[0], next, 0);
        fence_order();
        each<HEAD, NP>([&](auto p) {
            multiply(o[j & 1], p);
            constexpr int first = (p - HEAD) * EARLY / (NP - HEAD), end = (p - HEAD + 1) * EARLY / (NP - HEAD);
            each<first, end>([&](auto i) { load_one(i, stage); });
            fence_order();
        });
        freed = stage;
        stage = next;
    }
    // Loads still in flight write this workgroup's LDS: let them land.  Then the
    // other sets' sums take their place, and then the scales: a lane that
    // fetched the scale of each of its rows from memory would wait for every
    // one of them.
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if constexpr (TL::KS > 1) {
        constexpr int OF_WAVE = TL::FM * TL::FN * 16 * 64;
        int *sums = (int *)lds + lane;
        if (set > 0) {
#pragma unroll
            for (int i = 0; i < TL::FM * TL::FN * 16; ++i)
                sums[((set - 1) * TL::NW + wave) * OF_WAVE + i * 64] = acc[i / 16 / TL::FN][i / 16 % TL::FN][i % 16];
        }
        __syncthreads();
        if (set == 0) {
            for (int k = 0; k < TL::KS - 1; ++k)
#pragma unroll
                for (int i = 0; i < TL::FM * TL::FN * 16; ++i)
                    acc[i / 16 / TL::FN][i / 16 % TL::FN][i % 16] += sums[(k * TL::NW + wave) * OF_WAVE + i * 64];
        }
        __syncthreads();
    }
    constexpr int ROWS = TL::BM / PIECES;
    float *scales = (float *)lds;
    for (int i = tid; i < ROWS; i += TL::NT) scales[i] = g.sa && m0 / PIECES + i < g.M ? g.sa[m0 / PIECES + i] : 1.0f;
    __syncthreads();

    // Lane l holds columns FN (l % 32) + 0 .. FN-1 of its wave's tile (down:
    // l % 32 + 32 k), rows 8 (r / 4) + 4 (l / 32) + r % 4 of each fragment.
    constexpr int APART = DOWN ? 32 : 1;   // columns between a lane's
    const int col = n0 + wn * TL::WTN + (DOWN ? 1 : TL::FN) * fr;
    float sb[TL::FN];
#pragma unroll
    for (int k = 0; k < TL::FN; ++k) sb[k] = g.sb && col + APART * k < g.N ? g.sb[col + APART * k] : 1.0f;
    // What is masked: nothing, rows, or rows and columns (then stores are one value wide).
    const auto write = [&](auto mask_c, auto beta_c) {
        constexpr int MASK = decltype(mask_c)::value;
        constexpr bool BETA = decltype(beta_c)::value, WIDE = !DOWN && MASK < 2;
        typedef Vec<TL::FN, T> V;
#pragma unroll
        for (int i = 0; i < TL::FM; i += PIECES)
#pragma unroll
            for (int r4 = 0; r4 < 4; ++r4) {
                const int first = (wm * TL::WTM + 32 * i) / PIECES + 8 * r4 + 4 * h, row = m0 / PIECES + first;
                const f32v4 sa = *(const f32v4 *)(scales + first);
                T *const p = (T *)g.c + row * g.ldc + col;
                V old[4] = {};
                if constexpr (BETA) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if (MASK > 0 && row + r >= g.M) continue;
                        if constexpr (WIDE) old[r] = *(const V *)(p + r * g.ldc);
                        else
#pragma unroll
                            for (int k = 0; k < TL::FN; ++k)
                                if (MASK < 2 || col + APART * k < g.N) old[r].v[k] = p[r * g.ldc + APART * k];
                    }
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    V out;
#pragma unroll
                    for (int k = 0; k < TL::FN; ++k) {
                        float sum = (float)acc[i][k][4 * r4 + r];
                        if constexpr (PIECES == 2) sum = fmaf(256.0f, sum, (float)acc[i + 1][k][4 * r4 + r]);
                        float v = g.alpha * i8_scaled(sum, sa[r], sb[k]);
                        if constexpr (BETA) v += g.beta * MxType<TYPE>::load(&old[r].v[k]);
                        out.v[k] = MxType<TYPE>::from(v);
                    }
                    if (MASK > 0 && row + r >= g.M) continue;
                    if constexpr (WIDE) *(V *)(p + r * g.ldc) = out;
                    else
#pragma unroll
                        for (int k = 0; k < TL::FN; ++k)
                            if (MASK < 2 || col + APART * k < g.N) p[r * g.ldc + APART * k] = out.v[k];
                }
            }
    };
    if (set > 0) return;
    const auto masked = [&](auto beta_c) {
        if (n0 + TL::BN > g.N) write(std::integral_constant<int, 2>{}, beta_c);
        else if (m0 / PIECES + ROWS > g.M) write(std::integral_constant<int, 1>{}, beta_c);
        else write(std::integral_constant<int, 0>{}, beta_c);
    };
    if (g.beta != 0.0f) masked(std::true_type{});
    else masked(std::false_type{});
}

template <class TL, int TYPE, bool DOWN, int PIECES>
__global__ __launch_bounds__(TL::NT, 1) void i8_gemm_kernel(Args g) {
    compute_tile<TL, TYPE, DOWN, PIECES>(g, blockIdx.x);
}

// Two products, down, the second of pairs with a result in fp32, in one launch:
// the first `head` workgroups compute g, or k if k_first, the others the other.
template <class TL, class PAIRS, int TYPE>
__global__ __launch_bounds__(TL::NT, 1) void i8_gemm_two_kernel(Args g, Args k, int head, bool k_first) {
    static_assert(TL::NT == PAIRS::NT, "one size of workgroups");
    const bool early = (int)blockIdx.x < head;
    const int block = early ? blockIdx.x : blockIdx.x - head;
    if (early == k_first) compute_tile<PAIRS, SGEMM_TYPE_F32, true, 2>(k, block);
    else compute_tile<TL, TYPE, true, 1>(g, block);
}

typedef Tile<256, 256, 2, 4, 2> T256;       // 8 waves of 128 x 64, 128 KiB
typedef Tile<256, 128, 4, 4, 3> T256x128;   // 16 waves of 64 x 32, 144 KiB
typedef Tile<128, 128, 4, 2, 2> T128;       // 8 waves of 32 x 64, 64 KiB: two workgroups on a CU
typedef Tile<128, 128, 4, 2, 4> T128Deep;   // the same, 128 KiB
typedef Tile<64, 64, 2, 2, 4> T64;          // 4 waves of 32 x 32, 64 KiB
typedef Tile<64, 32, 2, 1, 4, 2> T64x32;    // 2 x 2 waves of 32 x 32, 96 KiB
typedef Tile<32, 32, 1, 1, 4, 2> T32;       // 2 waves of 32 x 32, 64 KiB
// For fragments in pairs: waves of 64 x 32.
typedef Tile<128, 128, 2, 4, 2> T128Pairs;
typedef Tile<128, 128, 2, 4, 4> T128DeepPairs;
typedef Tile<128, 64, 2, 2, 3> T64Pairs;    // 72 KiB
// Both in 48 KiB: three workgroups on a CU.
typedef Tile<64, 64, 2, 2, 3> T64Third;
typedef Tile<128, 64, 2, 2, 2> T64PairsThird;

template <class TL>
Args arguments(const I8GemmJob &j) {
    const int rows_a = j.pieces == 2 ? (int)i8_piece_rows(j.M) : j.M;
    return Args{j.a, j.sa, j.b, j.sb, j.c, j.ldc, j.M, j.N, j.K, rows_a, (int)(((int64_t)rows_a + TL::BM - 1) / TL::BM),
                (int)(((int64_t)j.N + TL::BN - 1) / TL::BN), j.alpha, j.beta};
}

template <class TL, int TYPE, bool DOWN, int PIECES>
hipError_t launch_tile(const I8GemmJob &j, hipStream_t s) {
    Args g = arguments<TL>(j);
    void *params[] = {&g};
    return hipLaunchKernel((const void *)i8_gemm_kernel<TL, TYPE, DOWN, PIECES>, dim3((unsigned)(g.tiles_m * g.tiles_n)), dim3(TL::NT), params,
                           TL::KS * TL::RING, s);
}

enum Kind { k256, k256x128, k128, k128Deep, k64, k64x32, k32 };   // pairs: k256, k128, k128Deep, k64

// (Times: 1 GiB of different weights in turn, bf16 results, in us.)
Kind kind_of(const I8GemmJob &j, int num_cus) {
    const bool pairs = j.pieces == 2;
    const int64_t rows = pairs ? i8_piece_rows(j.M) : j.M;
    const auto tiles = [&](int m, int n) { return ((rows + m - 1) / m) * (((int64_t)j.N + n - 1) / n); };
    // The largest tile that gives every CU one and whose rounds leave at most
    // a fifth of the CUs' time unused (272 tiles of 256 x 256, 4352 x 4096 x
    // 4096: 95.1, 90.5 in tiles of 128 x 128, two to a CU; 8192 x 4096 x 4096: 116
    // against 156).
    const int64_t rounds = (tiles(256, 256) + num_cus - 1) / num_cus;
    if (tiles(256, 256) >= num_cus && 4 * rounds * num_cus <= 5 * tiles(256, 256)) return k256;
    // At most 32 rows or columns of C: 32 x 4096 x 4096 8.6, in tiles of 64 x 64
    // 14.2; 32 x 5001 x 16384 24.8 and 41; 32 x 16384 x 16384 54 and 61, but 32 x
    // 28672 x 8192 51 and 49.
    if (!pairs && (rows <= 32 || j.N <= 32)) return k32;
    // More tiles of 128 x 128 than CUs: two workgroups on a CU hide the memory's
    // latency, or, where tiles of 256 x 128 go round once, sixteen waves (1111 x
    // 4097 x 2050: 19.0, 20.8 in tiles of 128 x 128, 24.1 with the deep ring;
    // 2500 x 2500 x 1000: 14.9, 15.7, 19.0).
    if (tiles(128, 128) > num_cus) return !pairs && tiles(256, 128) <= num_cus ? k256x128 : k128;
    // One for a CU at most: a deep ring hides it (2048 x 2048 x 2048: 12.5 against
    // 17.7; 1024 x 4096 x 4096 22.7 against 32.4).  With less than half a tile for a
    // CU, smaller ones spread further (200 x 8192 x 4096, 128 tiles: 18.6 against
    // 24.3; 1000 x 1000 x 8192, 64: 21.8 against 38.6).
    if (2 * tiles(128, 128) > num_cus) return k128Deep;
    // Up to one tile of 64 x 32 for a CU: two sets of waves, each with a ring of
    // its own, take every other chunk of K (128 x 4096 x 4096: 10.4 against 12.8;
    // 400 x 1000 x 8192: 12.8 against 18.4; 200 x 300 x 700: 6.2 against 6.5).
    return !pairs && tiles(64, 32) <= num_cus ? k64x32 : k64;
}

template <int TYPE, bool DOWN>
hipError_t launch_form(const I8GemmJob &j, int num_cus, hipStream_t s) {
    switch (kind_of(j, num_cus)) {
    case k256: return launch_tile<T256, TYPE, DOWN, 1>(j, s);
    case k256x128: return launch_tile<T256x128, TYPE, DOWN, 1>(j, s);
    case k128: return launch_tile<T128, TYPE, DOWN, 1>(j, s);
    case k128Deep: return launch_tile<T128Deep, TYPE, DOWN, 1>(j, s);
    case k64: return launch_tile<T64, TYPE, DOWN, 1>(j, s);
    case k64x32: return launch_tile<T64x32, TYPE, DOWN, 1>(j, s);
    default: return launch_tile<T32, TYPE, DOWN, 1>(j, s);
    }
}

hipError_t launch_pairs(const I8GemmJob &j, int num_cus, hipStream_t s) {
    switch (kind_of(j, num_cus)) {
    case k256: return launch_tile<T256, SGEMM_TYPE_F32, true, 2>(j, s);
    case k128: return launch_tile<T128Pairs, SGEMM_TYPE_F32, true, 2>(j, s);
    case k128Deep: return launch_tile<T128DeepPairs, SGEMM_TYPE_F32, true, 2>(j, s);
    default: return launch_tile<T64Pairs, SGEMM_TYPE_F32, true, 2>(j, s);
    }
}

template <class TL, class PAIRS, int TYPE>
hipError_t launch_two(const I8GemmJob &first, const I8GemmJob &second, hipStream_t s) {
    Args g = arguments<TL>(first), k = arguments<PAIRS>(second);
    bool k_first = k.K > g.K;   // the longer tiles begin
    const int tiles_g = g.tiles_m * g.tiles_n, tiles_k = k.tiles_m * k.tiles_n;
    int head = k_first ? tiles_k : tiles_g;
    void *params[] = {&g, &k, &head, &k_first};
    constexpr int bytes = TL::KS * TL::RING > PAIRS::KS * PAIRS::RING ? TL::KS * TL::RING : PAIRS::KS * PAIRS::RING;
    return hipLaunchKernel((const void *)i8_gemm_two_kernel<TL, PAIRS, TYPE>, dim3((unsigned)(tiles_g + tiles_k)), dim3(TL::NT), params, bytes, s);
}

// The products of a backward pass share a launch where they take like tiles: no
// CU idles between the end of one and the beginning of the other (8192 x 4096 x
// 4096: 378 us against 244 and 139).
template <int TYPE>
hipError_t launch_pair(const I8GemmJob &j, const I8GemmJob &k, int num_cus, hipStream_t s) {
    const Kind a = kind_of(j, num_cus), b = kind_of(k, num_cus);
    if (a == k256 && b == k256) return launch_two<T256, T256, TYPE>(j, k, s);
    if ((a == k128 || a == k256x128) && b == k128) return launch_two<T128, T128Pairs, TYPE>(j, k, s);
    // Small tiles for both.  Up to two workgroups on a CU take the deeper rings
    // (the whole backward pass of 1024 x 1024 x 1024, 512 tiles: 23.5 us against
    // 24.2); more fit three to a CU (333 x 1000 x 1536, 528 tiles: 21.7 against 22.9;
    // 200 x 600 x 3000, 658: 20.0 against 21.8).  Up to some 1300 tiles that is also
    // faster than two launches (2000 x 500 x 2000, 1280: 37.5 against 41.2; 600 x
    // 900 x 3000, 1175, the same; 1000 x 800 x 4000, 1827: 43.3 against 42.2).
    const auto tiles = [](int64_t m, int64_t n, int bm, int bn) { return ((m + bm - 1) / bm) * ((n + bn - 1) / bn); };
    const int64_t small = tiles(j.M, j.N, 64, 64) + tiles(i8_piece_rows(k.M), k.N, 128, 64);
    if (a >= k128Deep && b >= k128Deep && small <= 5 * num_cus)
        return small <= 2 * num_cus ? launch_two<T64, T64Pairs, TYPE>(j, k, s) : launch_two<T64Third, T64PairsThird, TYPE>(j, k, s);
    const hipError_t e = launch_form<TYPE, true>(j, num_cus, s);
    return e == hipSuccess ? launch_pairs(k, num_cus, s) : e;
}

}  // namespace

hipError_t launch_i8_gemm(const I8GemmJob &j, int num_cus, hipStream_t s) {
    if (!j.down && j.K > 0 && i8_thin_takes(j.M, j.N, j.K)) return launch_i8_thin(j, nullptr, 0, num_cus, s);
    if (j.pieces == 2) return launch_pairs(j, num_cus, s);
    switch (j.type) {
    case SGEMM_TYPE_F32: return j.down ? launch_form<SGEMM_TYPE_F32, true>(j, num_cus, s) : launch_form<SGEMM_TYPE_F32, false>(j, num_cus, s);
    case SGEMM_TYPE_BF16: return j.down ? launch_form<SGEMM_TYPE_BF16, true>(j, num_cus, s) : launch_form<SGEMM_TYPE_BF16, false>(j, num_cus, s);
    case SGEMM_TYPE_F16: return j.down ? launch_form<SGEMM_TYPE_F16, true>(j, num_cus, s) : launch_form<SGEMM_TYPE_F16, false>(j, num_cus, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_i8_gemm_two(const I8GemmJob &j, const I8GemmJob &k, int num_cus, hipStream_t s) {
    switch (j.type) {
    case SGEMM_TYPE_F32: return launch_pair<SGEMM_TYPE_F32>(j, k, num_cus, s);
    case SGEMM_TYPE_BF16: return launch_pair<SGEMM_TYPE_BF16>(j, k, num_cus, s);
    case SGEMM_TYPE_F16: return launch_pair<SGEMM_TYPE_F16>(j, k, num_cus, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace sgemm

// chunk_tile.cu -- attention of chunks over a paged KV cache on the tcgen05 tensor
// cores, for calls whose (sequence, KV head) pairs have many query rows.
//
// Method: out = softmax_{j <= p} (scale q . k_j) v_j for the query at position p, query
// head h reading KV head h / g ("注意力变体与 MoE", GQA attention(); "attention",
// GroupQueryAttention), one pass over the keys with a running maximum and sum in fp32.
// The g heads of a group are rows of the same tile, so each K/V row is read once for
// all of them, and the causal border cuts few tiles.
//
// Work: chunk_plan.cuh.  A persistent CTA walks its stretch of (block, key tile)s.  A
// block of more than 128 rows is two Q tiles that share every K/V tile, so that the
// softmax of one overlaps the products of the other; a block of at most 128 rows is one
// Q tile whose key tiles' halves go to the two softmax groups, each with its own maximum,
// sum and accumulator, joined from tensor memory at the end.
//
// Warps: 0-7 / 8-15 softmax of the two buffers (16 rows a warp, 64 scores a thread: half the
// time of a thread per row, which the chain scores - softmax - P V - next scores waits for),
// 16 issues the scores' MMAs, 18 the values', 17 loads K/V pages (one box per page and
// 64-column half, page entries fetched one tile ahead), 19 hands out the pieces and loads Q.
// FP8: warps 20-27, or 20-23, turn the codes of each landed tile into fp16 (exact) in the
// layout that the MMAs read; the keys' scales multiply the scores and the values' scales
// the weights, in fp32.
// TMEM: S0 | S1 | O0 | O1.  Scores are computed 64 keys at a time in either half of their 128
// columns, one step ahead of the softmax; the weights (16 bits) overwrite the first half of
// their scores and the P V product takes them from there.  (128 keys at a time, where the
// next scores wait for the P V that reads the weights in their place, the chain scores -
// softmax - P V took 3960 cycles a tile against 2050 of the products alone.)
// Measured (d = 128): 3465 and 3759 tokens behind 4096 rows, 32 / 8 heads, 592 us = 1.18 PFLOP/s
// (680 in a stream of such calls: the power limit); bound by the MMAs' issue, as the scores' of
// 64 keys cost what 128 would.  FP8, 1021 tokens over 31K rows, 64 heads on one KV head: 1155 us
// = 0.91 PFLOP/s (1254 to 1274); no unit is near its limit (tcgen05 pipe 56%, issue slots 64%): the
// dependent steps widening - scores - softmax - P V set the pace.
#include <type_traits>

#include "chunk_plan.cuh"
#include "common.cuh"
#include "kernels.h"

namespace kvattn {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
// log2 units: the maximum moves only when it grows by more than this (at 8, where the values' scales moved it more
// often, 16 x 8 tokens over 8K rows took 110 us instead of 107)
constexpr float kRescaleThreshold = 12.0f;
// FP8: weights times the values' scales enter the product times this, up to 2^15 then, what fp16 has room for: a
// weight is lost below 2^-28 of the largest (2^-25 without it, a sum of which reaches 2^-11 over 16K rows)
constexpr float kWeightScale = 8.0f;

// A stretch of one unit's key tiles, as warp 19 hands it to the others (rows = 0: no more).
struct Piece {
    int b, kvh;
    int tok0;    // the block's first packed token
    int pos0;    // its position
    int rows, keys;
    int tb, te;  // tiles
    int keys0;   // keys that the first 128 rows see
    int qt;      // Q tiles of 128 rows: 1 or 2
    int count;   // pieces of the unit
    int first;   // whether this is the first of them
};
constexpr int PIECES = 4;
constexpr int CH_STEP = 64;  // keys whose scores are computed at a time

// Steps of a piece that buffer t takes.  Two Q tiles (buffer = tile): the steps of its tiles that its rows see.
// One: the halves of each tile go to the two buffers, so the last step may be buffer 0's alone.
template <typename P>
__device__ __forceinline__ int piece_steps(const P& u, int t)
{
    const int tiles = u.te - u.tb;
    auto upto = [&](int keys) { return max(min(2 * tiles, ((keys + CH_STEP - 1) >> 6) - 2 * u.tb), 0); };
    if (u.qt == 2) return upto(t ? u.keys : u.keys0);
    return (upto(u.keys) + 1 - t) >> 1;
}

// QT: the most Q tiles that a block of the call can have.  The room of the second one holds more of K/V where
// there is none (16 x 8 tokens over 8K rows, one tile / two: bf16 95.8 / 97.2 us, FP8 104.8 / 110.9; 2 x 9 over
// 300: 13.8 / 14.3, 17.1 / 17.9).
// WIDE: the warps that widen codes, 8 (40 registers each) or 4 (64); see launch_tiles.  All of them work on one
// tile: with half on K's and half on V's, a tile takes longer to come (16 x 8 tokens over 8K rows 117 us against
// 105, four 2K prompts 298 against 278).
template <int D, bool FP8, int QT, int WIDE>
struct TCfg {
    static constexpr int HALVES = D / 64;
    static constexpr int BOX = CH_KEYS * 128;          // 128 rows x 64 bf16
    static constexpr int TILE = HALVES * BOX;          // a Q, K or V tile
    static constexpr int CODES = CH_KEYS * D;          // a tile's codes
    static constexpr int NS = (FP8 ? 3 : 6 - QT) * 2 / HALVES;                    // 16-bit K/V slots
    static constexpr int LS = !FP8 ? 0 : QT == 2 ? 4 / HALVES : D == 128 ? 4 : 6;  // code slots
    static constexpr int RING = 8;  // tiles whose page flags (and scales) are kept: the loads run up to 6 ahead of the softmax
    static constexpr int CW = FP8 ? WIDE : 0;
    static constexpr int THREADS = 640 + 32 * CW;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_KV = QT * TILE;
    static constexpr int OFF_LAND = OFF_KV + NS * TILE;
    static constexpr int OFF_SC = OFF_LAND + LS * CODES;  // [RING][3][128]: K's scales; V's, as log2; V's times kWeightScale
    static constexpr int OFF_U = OFF_SC + (FP8 ? RING * 3 * CH_KEYS * 4 : 0);
    static constexpr int OFF_CU = OFF_U + (PAGED_MAX_B + 1) * 8;
    static constexpr int OFF_LEN = OFF_CU + (PAGED_MAX_B + 1) * 4;
    static constexpr int OFF_ML = (OFF_LEN + PAGED_MAX_B * 4 + 15) / 16 * 16;  // [2][128] (max, sum)
    // [PIECES][256] exponents of the powers of two that Q's rows were multiplied by (FP8).  A place per piece of the
    // ring: Q may be widened for a piece while a softmax warp still has to read them for the second or third one
    // before it; piece_empty, which every softmax warp releases when it is through with a piece, orders the reuse
    static constexpr int OFF_QS = OFF_ML + 2 * 128 * 8;
    static constexpr int OFF_PIECE = OFF_QS + (FP8 ? PIECES * CH_ROWS * 2 : 0);
    static constexpr int OFF_BAR = OFF_PIECE + PIECES * static_cast<int>(sizeof(Piece));
    // kv_full[NS], kv_empty[NS], land_full[LS], land_empty[LS], q_full, q_empty, s_full[4], p_full[4], pv_done[4],
    // joined[2], piece_full[PIECES], piece_empty[PIECES], done, q_ready
    static constexpr int NBAR = 2 * NS + 2 * LS + 18 + 2 * PIECES;
    // warps that take every piece: 16 of the softmax, both MMA warps, K/V loads, those of the widening
    static constexpr int TAKERS = 19 + CW;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM = OFF_MISC + 16 + RING * 4 + 1024;
    static_assert(SMEM <= 232448, "shared memory");
    // bf16, or fp16 with FP8 (formats 0 instead of 1 in bits 7 and 10)
    static constexpr uint32_t IDESC_S = umma_idesc_bf16(128, CH_STEP) & (FP8 ? ~((1u << 7) | (1u << 10)) : ~0u);
    static constexpr uint32_t IDESC_O = umma_idesc_bf16(128, D, false, true) & (FP8 ? ~((1u << 7) | (1u << 10)) : ~0u);
};

// Four E4M3 codes -> fp16 pairs, exactly.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^-up for an exponent of -253 .. 252, in two factors as one alone may leave fp32's range.
__device__ __forceinline__ float pow2_neg(int up)
{
    return __int_as_float((127 - (up >> 1)) << 23) * __int_as_float((127 - up + (up >> 1)) << 23);
}

// Two weights, as the MMAs take them.
template <bool FP8>
__device__ __forceinline__ uint32_t pack_weights(float2 w)
{
    if constexpr (FP8) {
        uint32_t h;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(w.y), "f"(w.x));
        return h;
    } else {
        return pack_bf16x2(w.x, w.y);
    }
}

// Store of 32 columns x 16 lanes: register 2j of thread t goes to lane t / 4, column 4j + t % 4,
// register 2j + 1 to lane t / 4 + 8 of it.
__device__ __forceinline__ void tmem_st_16x128b_x8(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// 16 lanes x 16 columns (see common.cuh for the shape).
__device__ __forceinline__ void tmem_ld_16x256b_x2(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

__device__ __forceinline__ void tmem_st_16x256b_x2(uint32_t taddr, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// warp_wait with a first look that asks for the phase alone.
__device__ __forceinline__ bool ready(uint64_t* bar, uint32_t parity, volatile int* abort_flag)
{
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || warp_wait(bar, parity, abort_flag);
}

// The MMA warp runs its loop with all lanes, so that the descriptors stay in uniform
// registers (under a one-lane branch each operand of each MMA is moved there first, about
// 100 cycles per instruction); only these instructions are for the elected lane.
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e;
}

__device__ __forceinline__ void mma_ss(uint32_t elect, uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(acc), "r"(elect)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t elect, uint32_t d, uint32_t at, uint64_t bd, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(at), "l"(bd), "r"(idesc), "r"(acc), "r"(elect)
        : "memory");
}

__device__ __forceinline__ void commit_to(uint32_t elect, uint64_t* bar)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(elect)
        : "memory");
}

template <int D, bool FP8, int QT, int WIDE>
__global__ void __launch_bounds__(TCfg<D, FP8, QT, WIDE>::THREADS, 1)
    chunk_tile_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, ChunkArgs a)
{
    using C = TCfg<D, FP8, QT, WIDE>;
    constexpr int NS = C::NS, LS = C::LS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);  // (stays a shared-memory address to the compiler)
    uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* kv_empty = kv_full + NS;
    uint64_t* land_full = kv_empty + NS;
    uint64_t* land_empty = land_full + LS;
    uint64_t* q_full = land_empty + LS;
    uint64_t* q_empty = q_full + 1;
    uint64_t* s_full = q_full + 2;
    uint64_t* p_full = q_full + 6;   // (each: buffer t, half h at 2 t + h)
    uint64_t* pv_done = q_full + 10;
    uint64_t* joined = q_full + 14;
    uint64_t* piece_full = q_full + 16;
    uint64_t* piece_empty = piece_full + PIECES;
    uint64_t* done = piece_empty + PIECES;
    uint64_t* q_ready = done + 1;  // FP8: Q's rows are fp16
    int16_t* s_qs = reinterpret_cast<int16_t*>(smem + C::OFF_QS);
    const Piece* s_piece = reinterpret_cast<const Piece*>(smem + C::OFF_PIECE);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
    volatile uint32_t* s_bad = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC + 16);  // [RING]: groups of 16 keys without a page
    float* s_sc = reinterpret_cast<float*>(smem + C::OFF_SC);
    float2* s_ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    int* s_cu = reinterpret_cast<int*>(smem + C::OFF_CU);
    int* s_len = reinterpret_cast<int*>(smem + C::OFF_LEN);
    long long* s_U = reinterpret_cast<long long*>(smem + C::OFF_U);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&kv_full[i], FP8 ? C::CW : 1);
            mbar_init(&kv_empty[i], 1);
        }
        for (int i = 0; i < LS; ++i) {
            mbar_init(&land_full[i], 1);
            mbar_init(&land_empty[i], C::CW);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s_full[i], 2);  // the products' commit, and their issuer
            mbar_init(&p_full[i], 8);
            mbar_init(&pv_done[i], 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&joined[i], 16);
        for (int i = 0; i < PIECES; ++i) {
            mbar_init(&piece_full[i], 1);
            mbar_init(&piece_empty[i], C::TAKERS);
        }
        mbar_init(done, 2);
        mbar_init(q_ready, FP8 ? C::CW : 1);
        *s_abort = 0;
        fence_barrier_init();
    }
    if (warp == 17 && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    if (warp == 16) {
        tmem_alloc(s_tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    pdl_wait();
    pdl_trigger();

    const PagedBatch& p = a.p;
    const int w = CH_ROWS / a.g;
    int gs = 0;
    while ((1 << gs) < a.g) ++gs;
    chunk_plan_build(p, 8 - gs, a.max_q, s_cu, s_len, s_U, blockIdx.x == 0);
    const ChunkPlan plan{s_cu, s_len, s_U, p.B, a.Hk, a.g, 8 - gs, a.max_q, &p};
    // tokens that stand before row 0 see nothing (their blocks may have no unit)
    bool any_blind = false;
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) any_blind |= plan.seq(b).base() < 0;
    any_blind = __syncthreads_or(any_blind);
    for (int b = 0; any_blind && b < p.B; ++b) {
        const ChunkSeq s = plan.seq(b);
        const int blind = min(-s.base(), s.take);
        for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
             i < static_cast<long long>(max(blind, 0)) * a.H * (D / 8); i += static_cast<long long>(gridDim.x) * blockDim.x) {
            const long long row = static_cast<long long>(s.t0) * a.H + i / (D / 8);
            reinterpret_cast<uint4*>(a.out)[row * (D / 8) + i % (D / 8)] = make_uint4(0, 0, 0, 0);
            if (a.lse && i % (D / 8) == 0) a.lse[row] = -INFINITY;
        }
    }
    const int c = blockIdx.x;
    // piece i of this CTA, for a whole warp; false: none left (or a wait ran out)
    auto take = [&](int i, Piece& pc) {
        const int k = i % PIECES;
        if (!warp_wait(&piece_full[k], (i / PIECES) & 1, s_abort)) return false;
        pc = s_piece[k];
        __syncwarp();
        if (lane == 0) mbar_arrive(&piece_empty[k]);
        return pc.rows > 0;
    };

    if (warp == 17) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;" ::: "memory");
        // ===== K/V pages: lane i takes box i of a tile (page, and for bf16 its 64-column half) =====
        const int bp_shift = min(p.page_shift, 7);  // rows of a box: a page's, 128 at most
        const int bp = 1 << bp_shift;
        const int per = FP8 ? 1 : C::HALVES;
        const int box = lane / per, half = lane % per;
        const int oob = p.n_pages * a.Hk;  // reads as zeros
        uint32_t x = 0;  // K and V tiles so far
        uint32_t it = 0;
        bool ok = true;
        Piece u;
        for (int n = 0; ok && take(n, u); ++n) {
            const int tb = u.tb, te = u.te;
            const int32_t* pt = p.page_table + static_cast<long long>(u.b) * p.max_pages;
            auto entry = [&](int j) {
                const int row = j * CH_KEYS + (box << bp_shift);
                return box < (CH_KEYS >> bp_shift) && row < u.keys ? __ldg(pt + (row >> p.page_shift)) : 0;
            };
            int e = entry(tb);
            for (int j = tb; j < te && ok; ++j, ++it) {
                const int row = j * CH_KEYS + (box << bp_shift);
                const bool mine = box < (CH_KEYS >> bp_shift) && row < u.keys;
                const int e_next = j + 1 < te ? entry(j + 1) : 0;
                const bool bad = mine && (e < 0 || e >= p.n_pages);
                const uint32_t bads = __ballot_sync(0xffffffffu, bad && half == 0);
                if (bad && half == 0) report_status(p.dev_status, KVATTN_STATUS_BAD_INDEX);
                uint32_t groups = 0;
                if (bads) {
                    for (int i = 0; i < (CH_KEYS >> bp_shift); ++i)
                        if (bads >> (i * per) & 1) groups |= ((1u << (bp >> 4)) - 1u) << (i * (bp >> 4));
                }
                if (lane == 0) s_bad[it % C::RING] = groups;
                const int z = bad ? oob : e * a.Hk + u.kvh;
                const int y = row & ((1 << p.page_shift) - 1);
                const int boxes = (min(u.keys - j * CH_KEYS, CH_KEYS) + bp - 1) >> bp_shift;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv, ++x) {
                    if constexpr (FP8) {
                        const uint32_t slot = x % (LS > 0 ? LS : 1);
                        if (x >= LS && !(ok = warp_wait(&land_empty[slot], (x / LS - 1) & 1, s_abort))) break;
                        // with the keys, the scales of both (no copy where the page is bad)
                        const uint32_t goods = boxes - __popc(bads);
                        if (lane == 0)
                            mbar_arrive_expect_tx(&land_full[slot], boxes * bp * D + (kv == 0 ? goods * bp * 8 : 0));
                        __syncwarp();
                        if (mine) {
                            tma_load_3d(smem + C::OFF_LAND + slot * C::CODES + (box << bp_shift) * D, kv == 0 ? &tm_k : &tm_v,
                                        &land_full[slot], 0, y, z);
                            if (kv == 0 && !bad) {
                                const long long r = (static_cast<long long>(z) << p.page_shift) + y;
                                float* dst = s_sc + (it % C::RING) * 3 * CH_KEYS + (box << bp_shift);
                                bulk_load(dst, a.k_scales + r, bp * 4, &land_full[slot]);
                                bulk_load(dst + 2 * CH_KEYS, a.v_scales + r, bp * 4, &land_full[slot]);
                            }
                        }
                    } else {
                        const uint32_t slot = x % NS;
                        if (x >= NS && !(ok = warp_wait(&kv_empty[slot], (x / NS - 1) & 1, s_abort))) break;
                        if (lane == 0) mbar_arrive_expect_tx(&kv_full[slot], boxes * bp * 128 * C::HALVES);
                        __syncwarp();
                        if (mine)
                            tma_load_3d(smem + C::OFF_KV + slot * C::TILE + half * C::BOX + (box << bp_shift) * 128,
                                        kv == 0 ? &tm_k : &tm_v, &kv_full[slot], half * 64, y, z);
                    }
                }
                e = e_next;
            }
        }
        __syncwarp();
        // copies in flight complete before the CTA leaves (bounded waits)
        if (lane == 0) {
            if (!ok) report_status(p.dev_status, KVATTN_STATUS_TIMEOUT);
            constexpr uint32_t R = FP8 ? LS : NS;
            uint64_t* full = FP8 ? land_full : kv_full;
            for (uint32_t i = x > R ? x - R : 0; i < x; ++i) mbar_wait(&full[i % R], (i / R) & 1);
        }
    } else if (warp == 16) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;" ::: "memory");
        // ===== scores: S_t = Q K^T, a step ahead of the softmax (while that works on step i, step i + 1 is
        // multiplied), into half g % 2 of buffer t for its step number g =====
        const uint32_t el = elect_one();
        const uint32_t sq = smem_u32(smem + C::OFF_Q), skv = smem_u32(smem + C::OFF_KV);
        bool ok = true;
        uint32_t x0 = 0;            // first K/V tile number of the piece
        uint32_t gn[2] = {0, 0};    // steps so far, per buffer
        Piece u;
        for (int np = 0; ok && take(np, u); ++np) {
            ok = ready(FP8 ? q_ready : q_full, np & 1, s_abort);
            const bool pair = QT == 2 && u.qt == 2;
            const int n0 = piece_steps(u, 0), n1 = piece_steps(u, 1), n = max(n0, n1);
#pragma unroll 1
            for (int i = 0; i < n && ok; ++i) {
                const uint32_t x = x0 + 2 * (pair ? i >> 1 : i), slot = x % NS;
                // (of a tile's steps, the first one waits for it)
                if (!pair || !(i & 1)) ok = ready(&kv_full[slot], (x / NS) & 1, s_abort);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const uint32_t g = gn[t];
                    if (!ok || i >= (t ? n1 : n0)) continue;
                    // the weights that stand in the place have been used
                    if (g >= 2 && !(ok = ready(&pv_done[2 * t + (g & 1)], ((g >> 1) - 1) & 1, s_abort))) continue;
                    tc_fence_after();
                    const uint32_t d = tmem + t * CH_KEYS + (g & 1) * CH_STEP;
                    const uint32_t qa = sq + (pair ? t * C::TILE : 0);
                    const uint32_t ka = skv + slot * C::TILE + (pair ? i & 1 : t) * (CH_STEP * 128);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t off = (ks >> 2) * C::BOX + (ks & 3) * 32;
                        mma_ss(el, d, umma_desc_k_sw128(qa + off), umma_desc_k_sw128(ka + off), C::IDESC_S, ks > 0 ? 1u : 0u);
                    }
                    commit_to(el, &s_full[2 * t + (g & 1)]);
                    if (el) mbar_arrive(&s_full[2 * t + (g & 1)]);
                    ++gn[t];
                }
                if (ok && (!pair || (i & 1) || i + 1 == n)) commit_to(el, &kv_empty[slot]);
            }
            if (ok) commit_to(el, q_empty);
            x0 += 2 * (u.te - u.tb);
        }
        if (*s_abort && el) report_status(p.dev_status, KVATTN_STATUS_TIMEOUT);
        commit_to(el, done);
        mbar_wait(done, 0);
        __syncwarp();
    } else if (warp == 18) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;" ::: "memory");
        // ===== O_t += P V, step by step =====
        const uint32_t el = elect_one();
        const uint32_t skv = smem_u32(smem + C::OFF_KV);
        bool ok = true;
        uint32_t x0 = 1;
        uint32_t gn[2] = {0, 0};
        Piece u;
        for (int np = 0; ok && take(np, u); ++np) {
            const bool pair = QT == 2 && u.qt == 2;
            const int n0 = piece_steps(u, 0), n1 = piece_steps(u, 1), n = max(n0, n1);
#pragma unroll 1
            for (int i = 0; i < n && ok; ++i) {
                const uint32_t x = x0 + 2 * (pair ? i >> 1 : i), slot = x % NS;
                if (!pair || !(i & 1)) ok = ready(&kv_full[slot], (x / NS) & 1, s_abort);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const uint32_t g = gn[t];
                    if (!ok || i >= (t ? n1 : n0) || !(ok = ready(&p_full[2 * t + (g & 1)], (g >> 1) & 1, s_abort))) continue;
                    tc_fence_after();
                    const uint32_t va = skv + slot * C::TILE + (pair ? i & 1 : t) * (CH_STEP * 128);
                    const uint32_t pa = tmem + t * CH_KEYS + (g & 1) * CH_STEP;
#pragma unroll
                    for (int ks = 0; ks < CH_STEP / 16; ++ks)
                        mma_ts(el, tmem + 256 + t * D, pa + ks * 8, umma_desc_mn_sw128(va + ks * 2048, C::BOX, 1024),
                               C::IDESC_O, (i > 0 || ks > 0) ? 1u : 0u);
                    commit_to(el, &pv_done[2 * t + (g & 1)]);
                    ++gn[t];
                }
                if (ok && (!pair || (i & 1) || i + 1 == n)) commit_to(el, &kv_empty[slot]);
            }
            x0 += 2 * (u.te - u.tb);
        }
        if (*s_abort && el) report_status(p.dev_status, KVATTN_STATUS_TIMEOUT);
        commit_to(el, done);
        mbar_wait(done, 0);
        __syncwarp();
    } else if (warp < 16) {
        // registers: 640 threads at 96 = 512 x 104 + 128 x 64; with FP8 896 at 72 >= 512 x 88 + 128 x 64 + 256 x 40,
        // or 768 at 80 = 512 x 88 + 128 x 64 + 128 x 64
        if constexpr (FP8) asm volatile("setmaxnreg.inc.sync.aligned.u32 88;" ::: "memory");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 104;" ::: "memory");
        // ===== softmax + epilogue: warps 0-7 buffer 0, warps 8-15 buffer 1, 16 rows each =====
        // A row's scores are spread over a lane quad: thread (g, q) = (lane / 4, lane % 4) holds, of rows g and
        // g + 8 of the warp's 16, the keys 8 j + 2 q and 8 j + 2 q + 1 of a step of 64.
        const int t = warp >> 3, quarter = warp & 3, half = (warp >> 2) & 1;
        const int r16 = quarter * 32 + half * 16;  // the warp's first row of the Q tile = TMEM lane
        const int q2 = 2 * (lane & 3);
        const uint32_t lane_off = static_cast<uint32_t>(r16) << 16;
        const uint32_t s_addr = tmem + lane_off + t * CH_KEYS;
        const uint32_t o_base = tmem + lane_off + 256;
        const float sl2 = a.scale * kLog2e;
        uint32_t it0 = 0;   // first tile number of the piece
        uint32_t cnt = 0;   // steps of this buffer so far
        uint32_t joins = 0;
        for (int n = 0;; ++n) {
            // the piece stays in shared memory, and is read where it is needed: registers are short here
            if (!ready(&piece_full[n % PIECES], (n / PIECES) & 1, s_abort)) break;
            const volatile Piece& u = s_piece[n % PIECES];
            if (u.rows == 0) break;
            const int tb = u.tb;
            const bool pair = QT == 2 && u.qt == 2;  // two Q tiles; else one, its keys dealt out in steps
            const int row0 = (pair ? t * 128 : 0) + r16;  // the warp's first row of the block
            const int pos_first = u.pos0 + (row0 >> gs);
            const bool active_warp = row0 < u.rows;
            const int n_my = piece_steps(u, t);
            float sl2a = sl2, sl2b = sl2;  // raw scores to log2 units
            float ma = -INFINITY, mb = -INFINITY, la = 0.f, lb = 0.f;  // maxima of the rows; this thread's share of their sums
            for (int k = 0; k < n_my; ++k, ++cnt) {
                const int jt = pair ? k >> 1 : k, hh = pair ? k & 1 : t;  // tile of the piece, half of it
                const int kb = (tb + jt) * CH_KEYS + hh * CH_STEP;         // first key of the step
                const uint32_t it = it0 + jt;
                const uint32_t sp = s_addr + (cnt & 1) * CH_STEP;
                if (!ready(&s_full[2 * t + (cnt & 1)], (cnt >> 1) & 1, s_abort)) continue;
                tc_fence_after();
                if (!FP8 && u.keys - kb < CH_STEP) {
                    // rows of V behind the last key in use were not loaded, or hold what nobody may see:
                    // zeros, so that 0 * garbage cannot reach a sum (the P V waits for these warps)
                    const uint32_t xv = 2 * it + 1;
                    if (!ready(&kv_full[xv % NS], (xv / NS) & 1, s_abort)) continue;
                    const int vr = (threadIdx.x & 255) >> 2;
                    if (vr >= u.keys - kb) {
                        uint8_t* v = smem + C::OFF_KV + (xv % NS) * C::TILE + (hh * CH_STEP + vr) * 128 + (lane & 3) * 32;
#pragma unroll
                        for (int i = 0; i < C::HALVES * 2; ++i)
                            *reinterpret_cast<uint4*>(v + (i >> 1) * C::BOX + (i & 1) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                if (FP8 && k == 0) {  // (the scores wait for the converted Q rows)
                    const int16_t* qs = s_qs + (n % PIECES) * CH_ROWS + row0 + (lane >> 2);
                    // not 0, as that times the -inf of a key out of sight is no number (a tiny or zero row: its
                    // scores are 0 either way)
                    sl2a = fmaxf(sl2 * pow2_neg(qs[0]), 0x1p-126f);
                    sl2b = fmaxf(sl2 * pow2_neg(qs[8]), 0x1p-126f);
                }
                if (active_warp) {
                    const uint32_t bad = s_bad[it % C::RING] >> (4 * hh) & 15u;
                    const float* ks = s_sc + (it % C::RING) * 3 * CH_KEYS + hh * CH_STEP + q2;
                    const bool masked = pos_first - kb < CH_STEP - 1 || bad != 0;  // warp-uniform
                    uint32_t sv[32];
                    tmem_ld_16x256b_x8(sp, sv);
                    tmem_wait_ld();
                    tmem_regs_ready(sv);
                    const float2 sca = make_float2(sl2a, sl2a), scb = make_float2(sl2b, sl2b);
                    if constexpr (FP8) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 f = *reinterpret_cast<const float2*>(ks + 8 * i);
                            uint32_t* x = sv + 4 * i;
                            const float2 y = __fmul2_rn(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), f);
                            const float2 z = __fmul2_rn(make_float2(__uint_as_float(x[2]), __uint_as_float(x[3])), f);
                            x[0] = __float_as_uint(y.x);
                            x[1] = __float_as_uint(y.y);
                            x[2] = __float_as_uint(z.x);
                            x[3] = __float_as_uint(z.y);
                        }
                    }
                    if (masked) {
                        // keys 0 .. lim of the step are seen
                        const int pos0 = u.pos0 - kb, ra = row0 + (lane >> 2);
                        const int lima = pos0 + (ra >> gs), limb = pos0 + ((ra + 8) >> gs);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const bool b = bad >> (i >> 1) & 1u;
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                if (b || 8 * i + q2 + e > lima) sv[4 * i + e] = 0xff800000u;  // -inf
                                if (b || 8 * i + q2 + e > limb) sv[4 * i + 2 + e] = 0xff800000u;
                            }
                        }
                    }
                    float xa[2] = {-INFINITY, -INFINITY}, xb[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t* x = sv + 4 * i;
                        float2 y = make_float2(__uint_as_float(x[0]), __uint_as_float(x[1]));
                        float2 z = make_float2(__uint_as_float(x[2]), __uint_as_float(x[3]));
                        if constexpr (FP8) {  // the maximum of s + log2 vs, in log2 units
                            const float2 lv = *reinterpret_cast<const float2*>(ks + CH_KEYS + 8 * i);
                            y = __ffma2_rn(y, sca, lv);
                            z = __ffma2_rn(z, scb, lv);
                        }
                        xa[i & 1] = fmax3(xa[i & 1], y.x, y.y);
                        xb[i & 1] = fmax3(xb[i & 1], z.x, z.y);
                    }
                    float mxa = fmaxf(xa[0], xa[1]), mxb = fmaxf(xb[0], xb[1]);
                    mxa = fmaxf(mxa, __shfl_xor_sync(0xffffffffu, mxa, 1));
                    mxb = fmaxf(mxb, __shfl_xor_sync(0xffffffffu, mxb, 1));
                    mxa = fmaxf(mxa, __shfl_xor_sync(0xffffffffu, mxa, 2)) * (FP8 ? 1.f : sl2a);
                    mxb = fmaxf(mxb, __shfl_xor_sync(0xffffffffu, mxb, 2)) * (FP8 ? 1.f : sl2b);
                    // the reference maximum moves (and O with it, for the warp together) only when the
                    // row's maximum has grown by more than 2^12: the weights stay below that
                    const bool mva = mxa > ma + kRescaleThreshold || ma == -INFINITY;
                    const bool mvb = mxb > mb + kRescaleThreshold || mb == -INFINITY;
                    if (__any_sync(0xffffffffu, mva || mvb)) {
                        const float na = mva ? fmaxf(mxa, ma) : ma, nb = mvb ? fmaxf(mxb, mb) : mb;
                        const bool rsa = mva && ma != -INFINITY, rsb = mvb && mb != -INFINITY;
                        if (__any_sync(0xffffffffu, rsa || rsb)) {
                            const float da = rsa ? ma - na : 0.f, db = rsb ? mb - nb : 0.f;
                            const float ala = fast_exp2(da), alb = fast_exp2(db);
                            la = sum_exp2(la, da);
                            lb = sum_exp2(lb, db);
                            // O must be still: the P V of the step before has finished
                            if (!ready(&pv_done[2 * t + ((cnt - 1) & 1)], ((cnt - 1) >> 1) & 1, s_abort)) continue;
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D / 16; ++c) {
                                uint32_t ov[8];
                                tmem_ld_16x256b_x2(o_base + t * D + c * 16, ov);
                                tmem_wait_ld();
                                tmem_regs_ready(ov);
#pragma unroll
                                for (int i = 0; i < 8; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * ((i & 2) ? alb : ala));
                                tmem_st_16x256b_x2(o_base + t * D + c * 16, ov);
                            }
                        }
                        ma = na;
                        mb = nb;
                    }
                    // weights 2^(s sl2 - m), to TMEM over the scores' first half.  Every exponential goes
                    // through the hardware unit, where 2^-inf is exactly 0: none / an eighth / a quarter / half of them
                    // as a polynomial on the FMA pipe took 592 / 601 / 607 / 647 us for two 3.5K-token chunks (and none
                    // at all 602: they are hidden behind the products)
                    const float mua = ma == -INFINITY ? 0.f : -ma, mub = mb == -INFINITY ? 0.f : -mb;
                    float2 acca = make_float2(0.f, 0.f), accb = acca;
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t* x = sv + 4 * i;
                        const float2 y = __ffma2_rn(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), sca, make_float2(mua, mua));
                        const float2 z = __ffma2_rn(make_float2(__uint_as_float(x[2]), __uint_as_float(x[3])), scb, make_float2(mub, mub));
                        float2 pa = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                        float2 pb = make_float2(fast_exp2(z.x), fast_exp2(z.y));
                        acca = __fadd2_rn(acca, pa);
                        accb = __fadd2_rn(accb, pb);
                        if constexpr (FP8) {
                            const float2 f = *reinterpret_cast<const float2*>(ks + 2 * CH_KEYS + 8 * i);
                            pa = __fmul2_rn(pa, f);
                            pb = __fmul2_rn(pb, f);
                        }
                        pk[2 * i] = pack_weights<FP8>(pa);
                        pk[2 * i + 1] = pack_weights<FP8>(pb);
                    }
                    tmem_st_16x128b_x8(sp, pk);
                    la += acca.x + acca.y;
                    lb += accb.x + accb.y;
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[2 * t + (cnt & 1)]);
            }
            it0 += u.te - tb;
            la += __shfl_xor_sync(0xffffffffu, la, 1);
            lb += __shfl_xor_sync(0xffffffffu, lb, 1);
            la += __shfl_xor_sync(0xffffffffu, la, 2);
            lb += __shfl_xor_sync(0xffffffffu, lb, 2);
            const bool ok = n_my == 0 || ready(&pv_done[2 * t + ((cnt - 1) & 1)], ((cnt - 1) >> 1) & 1, s_abort);
            tc_fence_after();
            // ---- the piece's rows: finished, or a partial for the merge ----
            float va = 0.f, vb = 0.f;  // weights of the other buffer's sums; ua, ub of this one's (nothing seen: 0, as
            constexpr float UNIT = FP8 ? 1.f / kWeightScale : 1.f;
            float ua = ma == -INFINITY ? 0.f : UNIT, ub = mb == -INFINITY ? 0.f : UNIT;  // it may never have been written)
            int c0 = 0, c1 = D / 16;   // column pieces of 16
            if (!pair) {
                // join the two buffers: each group writes half of the columns
                if ((lane & 3) == 0) {
                    s_ml[t * 128 + r16 + (lane >> 2)] = make_float2(ma, la);
                    s_ml[t * 128 + r16 + (lane >> 2) + 8] = make_float2(mb, lb);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&joined[0]);
                ready(&joined[0], joins & 1, s_abort);
                tc_fence_after();
                const float2 oa = s_ml[(t ^ 1) * 128 + r16 + (lane >> 2)], ob = s_ml[(t ^ 1) * 128 + r16 + (lane >> 2) + 8];
                const float Ma = fmaxf(ma, oa.x), Mb = fmaxf(mb, ob.x);
                const float fa = Ma == -INFINITY ? 0.f : Ma, fb = Mb == -INFINITY ? 0.f : Mb;
                ua = fast_exp2(ma - fa) * UNIT;
                ub = fast_exp2(mb - fb) * UNIT;
                va = fast_exp2(oa.x - fa) * UNIT;
                vb = fast_exp2(ob.x - fb) * UNIT;
                la = sum_exp2(la, ma - fa) + sum_exp2(oa.y, oa.x - fa);
                lb = sum_exp2(lb, mb - fb) + sum_exp2(ob.y, ob.x - fb);
                ma = Ma;
                mb = Mb;
                c0 = t * (D / 32);
                c1 = c0 + D / 32;
            }
            const bool whole = u.count == 1;
            const int rowa = row0 + (lane >> 2), rowb = rowa + 8, rows = u.rows;
            if (whole) {
                const float ia = la > 0.f ? 1.f / la : 0.f, ib = lb > 0.f ? 1.f / lb : 0.f;
                ua *= ia;
                va *= ia;
                ub *= ib;
                vb *= ib;
            }
            const long long base = static_cast<long long>(u.tok0) * a.H + static_cast<long long>(u.kvh) * a.g;
            const long long outa = base + static_cast<long long>(rowa >> gs) * a.H + (rowa & (a.g - 1));
            const long long outb = base + static_cast<long long>(rowb >> gs) * a.H + (rowb & (a.g - 1));
            const long long part = static_cast<long long>(2 * c + u.first) * CH_ROWS;
            const bool usea = ok && rowa < rows, useb = ok && rowb < rows;
            constexpr int EC = 16;  // columns at a time (more cost registers that the tile loop needs)
#pragma unroll 1
            for (int cc = c0; cc < c1; ++cc) {
                uint32_t ov[EC / 2], ow[EC / 2];
                tmem_ld_16x256b_x2(o_base + t * D + cc * EC, ov);
                if (!pair) tmem_ld_16x256b_x2(o_base + (t ^ 1) * D + cc * EC, ow);
                tmem_wait_ld();
                tmem_regs_ready(ov);
                if (!pair) tmem_regs_ready(ow);
                float x[EC / 2];
#pragma unroll
                for (int i = 0; i < EC / 2; ++i) {
                    const float f = (i & 2) ? ub : ua, h = (i & 2) ? vb : va;
                    x[i] = f == 0.f ? 0.f : __uint_as_float(ov[i]) * f;
                    if (!pair && h != 0.f) x[i] = fmaf(__uint_as_float(ow[i]), h, x[i]);
                }
#pragma unroll
                for (int i = 0; i < EC / 8; ++i) {
                    const int col = cc * EC + 8 * i + q2;
                    if (whole) {
                        if (usea) *reinterpret_cast<uint32_t*>(a.out + outa * D + col) = pack_bf16x2(x[4 * i], x[4 * i + 1]);
                        if (useb) *reinterpret_cast<uint32_t*>(a.out + outb * D + col) = pack_bf16x2(x[4 * i + 2], x[4 * i + 3]);
                    } else {
                        if (usea) *reinterpret_cast<float2*>(a.part_o + (part + rowa) * D + col) = make_float2(x[4 * i], x[4 * i + 1]);
                        if (useb) *reinterpret_cast<float2*>(a.part_o + (part + rowb) * D + col) = make_float2(x[4 * i + 2], x[4 * i + 3]);
                    }
                }
            }
            if ((lane & 3) == 0 && (pair || t == 0)) {
                if (whole) {
                    if (a.lse && usea) a.lse[outa] = la > 0.f ? (ma + __log2f(la)) * kLn2 : -INFINITY;
                    if (a.lse && useb) a.lse[outb] = lb > 0.f ? (mb + __log2f(lb)) * kLn2 : -INFINITY;
                } else {
                    if (usea) a.part_ml[part + rowa] = make_float2(ma, la);
                    if (useb) a.part_ml[part + rowb] = make_float2(mb, lb);
                }
            }
            // the other group reads this buffer's accumulator: the next piece waits for it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&piece_empty[n % PIECES]);
            if (!pair) {
                if (lane == 0) mbar_arrive(&joined[1]);
                ready(&joined[1], joins & 1, s_abort);
                ++joins;
            }
        }
    } else if (warp >= 20) {
        if constexpr (FP8) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(WIDE == 8 ? 40 : 64) : "memory");
            // ===== Q -> fp16 in place; codes -> fp16 tiles in the 128-byte-swizzled layout =====
            // fp16 is one conversion for two codes, exact, and three more bits of the weights than bf16 (the long
            // chunk's outputs are off by 0.0017 of their norm, their own rounding, where bf16 weights gave 0.0025).
            // Its range is enough: Q's rows are scaled into it, and a row's running reference is the maximum of
            // s + log2 vs over the keys it sees, so its weights times the values' scales stay below 2^12 (and the largest above 1),
            // below 2^15 with kWeightScale.
            const int tid = threadIdx.x - 640, cwarp = tid >> 5;
            // chunk of 16 codes: two rows by four chunks in eight neighbouring lanes, so that either half of their
            // 32 bytes falls on eight different bank groups
            const int ch0 = lane & 3, row0 = ((lane >> 2) & 1) + ((lane >> (D == 128 ? 4 : 3)) << 1);
            const int ch = ch0 + (D == 128 ? (lane >> 1) & 4 : 0);
            constexpr int RW = D == 128 ? 4 : 8;  // rows a warp takes at a time
            uint32_t x = 0;
            bool ok = true;
            Piece u;
            for (int n = 0; ok && take(n, u); ++n) {
                // a row's 16-byte pieces lie in D / 8 neighbouring lanes
                ok = ready(q_full, n & 1, s_abort);
                if (!ok) break;
#pragma unroll 2
                for (int i = 0; i < u.qt * (D / 8) * 4 / C::CW; ++i) {
                    const int id = i * (32 * C::CW) + tid, row = id / (D / 8), c8 = id % (D / 8);
                    uint4* q = reinterpret_cast<uint4*>(smem + C::OFF_Q + (row >> 7) * C::TILE + (c8 >> 3) * C::BOX + swz128(row & 127, c8 & 7));
                    const uint4 v = *q;
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    float m = 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) m = fmax3(m, fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e])));
#pragma unroll
                    for (int o = D / 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                    // largest element to [2^14, 2^15), by its exponent field (0 of a zero or subnormal row: taken as
                    // 1): exact down to 2^-31 of the largest (bf16's eight bits, steps of 2^-24 in fp16), below that
                    // rounded to a multiple of at most 2^-38 of it, far below the fp32 sums' own rounding.  Two factors, as one may leave fp32's range: 2^(141 - e) = fa fb.
                    const int e8 = max(static_cast<int>(__float_as_uint(m) >> 23), 1), up = 141 - e8;
                    const float fa = __int_as_float((127 + (up >> 1)) << 23), fb = __int_as_float((127 + up - (up >> 1)) << 23);
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(o[e]) : "f"(bf16_hi(w[e]) * fa * fb), "f"(bf16_lo(w[e]) * fa * fb));
                    *q = make_uint4(o[0], o[1], o[2], o[3]);
                    if (c8 == 0) s_qs[(n % PIECES) * CH_ROWS + row] = static_cast<int16_t>(up);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(q_ready);
                for (int j = u.tb; j < u.te && ok; ++j) {
                    const int nv = min(u.keys - j * CH_KEYS, CH_KEYS);
                    const uint32_t it = x / 2;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv, ++x) {
                        const uint32_t ls = x % (LS > 0 ? LS : 1), slot = x % NS;
                        ok = ready(&land_full[ls], (x / (LS > 0 ? LS : 1)) & 1, s_abort);
                        if (ok && x >= NS) ok = ready(&kv_empty[slot], (x / NS - 1) & 1, s_abort);
                        if (!ok) break;
                        const uint32_t bad = s_bad[it % C::RING];
                        const bool partial = nv < CH_KEYS || bad != 0;
                        if (kv == 0 && tid < CH_KEYS) {
                            float* sc = s_sc + (it % C::RING) * 3 * CH_KEYS + tid;
                            float lv = fmaxf(lg2(sc[2 * CH_KEYS]), CHUNK_MIN_LOG2_VS);
                            if (partial && (tid >= nv || (bad >> (tid / 16) & 1u))) {  // no key: anything may stand there
                                sc[0] = sc[2 * CH_KEYS] = 0.f;
                                lv = 0.f;
                            }
                            sc[CH_KEYS] = lv;
                            sc[2 * CH_KEYS] *= kWeightScale;
                        }
                        const uint8_t* src = smem + C::OFF_LAND + ls * C::CODES;
                        uint8_t* dst = smem + C::OFF_KV + slot * C::TILE + (ch >> 2) * C::BOX;
#pragma unroll 4
                        for (int i = 0; i < CH_KEYS / (C::CW * RW); ++i) {
                            const int row = (i * C::CW + cwarp) * RW + row0;
                            const uint4 v = *reinterpret_cast<const uint4*>(src + row * D + ch * 16);
                            uint4 o0, o1;
                            codes_to_f16(v.x, o0.x, o0.y);
                            codes_to_f16(v.y, o0.z, o0.w);
                            codes_to_f16(v.z, o1.x, o1.y);
                            codes_to_f16(v.w, o1.z, o1.w);
                            if (kv == 1 && partial && row >= nv) o0 = o1 = make_uint4(0, 0, 0, 0);
                            *reinterpret_cast<uint4*>(dst + swz128(row, 2 * ch0)) = o0;
                            *reinterpret_cast<uint4*>(dst + swz128(row, 2 * ch0 + 1)) = o1;
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&kv_full[slot]);
                            mbar_arrive(&land_empty[ls]);
                        }
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;" ::: "memory");
        // ===== warp 19: this CTA's pieces, and their Q: [128 / g tokens][g heads] boxes, one or two tiles =====
        if (lane == 0) {
            const long long N = plan.total();
            // every CTA's stretch holds a tile's points at least, so that it owns a tile of each unit it lies in
            const int G = static_cast<int>(min(static_cast<long long>(gridDim.x), max(N / CH_COST2, 1ll)));
            int4 split = make_int4(0, 0, 0, 0);
            int np = 0;
            bool ok = true;
            auto put = [&](const Piece& pc) {
                const int k = np % PIECES;
                if (np >= PIECES && !(ok = !*s_abort && mbar_wait(&piece_empty[k], (np / PIECES - 1) & 1))) {
                    *s_abort = 1;
                    return;
                }
                *reinterpret_cast<Piece*>(smem + C::OFF_PIECE + k * sizeof(Piece)) = pc;
                mbar_arrive(&piece_full[k]);
                ++np;
                if (pc.rows == 0) return;
                if (np > 1 && !(ok = !*s_abort && mbar_wait(q_empty, np & 1))) {  // the scores of the piece before are done
                    *s_abort = 1;
                    return;
                }
                mbar_arrive_expect_tx(q_full, pc.qt * C::TILE);
                for (int t = 0; t < pc.qt; ++t)
#pragma unroll
                    for (int h = 0; h < C::HALVES; ++h)
                        tma_load_3d(smem + C::OFF_Q + t * C::TILE + h * C::BOX, &tm_q, q_full, h * 64, pc.kvh * a.g,
                                    pc.tok0 + t * (w / 2));
            };
            if (N > 0 && c < G) {
                const long long lo = chunk_start(c, N, G), hi = chunk_start(c + 1, N, G);
                for (ChunkUnit u = plan.find(lo); ok && u.b < p.B && u.U < hi; plan.next(u)) {
                    Piece pc;
                    if (!plan.piece(u, lo, hi, pc.tb, pc.te)) continue;
                    const int f = chunk_owner(u.U, N, G);
                    pc.b = u.b;
                    pc.kvh = u.kvh;
                    pc.tok0 = u.s.t0 + u.rb * w;
                    pc.pos0 = u.s.base() + u.rb * w;
                    pc.rows = u.rows;
                    pc.keys = u.keys;
                    pc.keys0 = u.keys0;
                    pc.qt = u.qt;
                    pc.count = chunk_owner(u.U + static_cast<long long>(u.tiles - 1) * u.cost(), N, G) - f + 1;
                    pc.first = f == c;
                    if (pc.count > 1 && pc.first) split = make_int4(pc.tok0, pc.rows, pc.kvh, pc.count);
                    put(pc);
                }
            }
            // the merge finds a split unit at the CTA of its first tile
            a.split_info[c] = split;
            const int loaded = np;
            Piece none{};
            if (ok) put(none);
            if (loaded > 0) mbar_wait(q_full, (loaded - 1) & 1);  // no copy in flight when the CTA leaves
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---- merge of the split units ------------------------------------------------------
// One warp per query row: with M = max m_i over the partials and w_i = 2^(m_i - M),
// out = sum w_i O_i / sum w_i l_i and lse = ln 2 (M + log2 sum w_i l_i), in the
// partials' order.  Lane i holds (m, l) of partial i, 32 at a time, and eight partials'
// rows are in flight together, so a row waits for memory 2 + count / 8 times.  As many warps
// as the call's blocks can have rows; most units are whole, and their warps only look.
constexpr int TM_WARPS = 8;

template <int D>
__global__ void __launch_bounds__(TM_WARPS * 32) chunk_tile_merge_kernel(ChunkArgs a)
{
    constexpr int PL = D / 32, BATCH = 8;
    using Vec = typename std::conditional<PL == 4, float4, float2>::type;
    pdl_wait();
    pdl_trigger();
    const int f = blockIdx.x;
    const int4 info = a.split_info[f];
    const int lane = threadIdx.x & 31, row = blockIdx.y * TM_WARPS + (threadIdx.x >> 5), count = info.w;
    if (count < 2 || row >= info.y) return;
    auto slot = [&](int i) { return static_cast<long long>(i == 0 ? 2 * f + 1 : 2 * (f + i)) * CH_ROWS + row; };
    float M = -INFINITY, L = 0.f, acc[PL];
#pragma unroll
    for (int k = 0; k < PL; ++k) acc[k] = 0.f;
    for (int i0 = 0; i0 < count; i0 += 32) {
        const int n = min(32, count - i0);
        const float2 ml = lane < n ? __ldcg(a.part_ml + slot(i0 + lane)) : make_float2(-INFINITY, 0.f);
        float Mn = fmaxf(M, ml.x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) Mn = fmaxf(Mn, __shfl_xor_sync(0xffffffffu, Mn, o));
        const float mu = Mn == -INFINITY ? 0.f : Mn, c = fast_exp2(M - mu);
        L = sum_exp2(L, M - mu);
        M = Mn;
        const float wl = fast_exp2(ml.x - mu);
        float sum = sum_exp2(ml.y, ml.x - mu);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        L += sum;
#pragma unroll
        for (int k = 0; k < PL; ++k) acc[k] *= c;
        for (int i = 0; i < n; i += BATCH) {
            Vec v[BATCH];
#pragma unroll
            for (int j = 0; j < BATCH; ++j)
                if (i + j < n) v[j] = __ldcg(reinterpret_cast<const Vec*>(a.part_o + slot(i0 + i + j) * D) + lane);
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const float w = __shfl_sync(0xffffffffu, wl, (i + j) & 31);
                if (i + j < n) {
                    const float* x = reinterpret_cast<const float*>(&v[j]);
#pragma unroll
                    for (int k = 0; k < PL; ++k) acc[k] += w * x[k];
                }
            }
        }
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    const long long orow = (static_cast<long long>(info.x) + row / a.g) * a.H + static_cast<long long>(info.z) * a.g + row % a.g;
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + orow * D + lane * PL);
#pragma unroll
    for (int k = 0; k < PL; k += 2) dst[k / 2] = pack_bf16x2(acc[k] * inv, acc[k + 1] * inv);
    if (lane == 0 && a.lse) a.lse[orow] = L > 0.f ? (M + __log2f(L)) * kLn2 : -INFINITY;
}

template <int D, bool FP8, int QT, int WIDE>
cudaError_t launch_typed(const ChunkArgs& a, const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                         int num_sms, cudaStream_t stream)
{
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !attr_set[dev]) {
        e = cudaFuncSetAttribute(chunk_tile_kernel<D, FP8, QT, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, TCfg<D, FP8, QT, WIDE>::SMEM);
        if (e != cudaSuccess) return e;
        if (dev < 64) attr_set[dev] = true;
    }
    const int grid = num_sms < CHUNK_MAX_CTAS ? num_sms : CHUNK_MAX_CTAS;
    e = launch_pdl(chunk_tile_kernel<D, FP8, QT, WIDE>, dim3(grid), dim3(TCfg<D, FP8, QT, WIDE>::THREADS), TCfg<D, FP8, QT, WIDE>::SMEM, stream, tm_q,
                   tm_k, tm_v, a);
    if (e != cudaSuccess) return e;
    const int rows = a.max_q < CH_ROWS / a.g ? a.max_q * a.g : CH_ROWS;
    return launch_pdl(chunk_tile_merge_kernel<D>, dim3(grid, (rows + TM_WARPS - 1) / TM_WARPS), dim3(TM_WARPS * 32), 0, stream, a);
}

template <int D, bool FP8>
cudaError_t launch_tiles(const ChunkArgs& a, const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                         int num_sms, cudaStream_t stream)
{
    if (a.max_q * a.g <= CH_ROWS / 2) return launch_typed<D, FP8, 1, 8>(a, tm_q, tm_k, tm_v, num_sms, stream);
    if constexpr (FP8) {
        // Eight widening warps start a piece faster; in a long one, where they wait for the softmax, four take fewer
        // of its issue slots.  A piece has as many tiles as a sequence, or a CTA, at most.  8 / 4 warps: d = 128,
        // 2000 tokens over 0, 2000 and 8000 rows (32 and 8 heads) 109 / 121 us, 163 / 162, 396 / 374, 64 over 16000
        // 47.9 / 50; d = 64 (64 and 8 heads) 500 over 2000 70 / 66, 2000 over 8000 679 / 582, 300 over 0 22.4 / 23.
        const long long seq = (static_cast<long long>(a.p.max_pages) << a.p.page_shift) / CH_KEYS;
        const long long blocks = (static_cast<long long>(a.p.n_tokens) * a.g + CH_ROWS - 1) / CH_ROWS * a.Hk;
        if (seq >= D / 4 && blocks * seq / num_sms >= D / 4) return launch_typed<D, FP8, 2, 4>(a, tm_q, tm_k, tm_v, num_sms, stream);
    }
    return launch_typed<D, FP8, 2, 8>(a, tm_q, tm_k, tm_v, num_sms, stream);
}

}  // namespace

cudaError_t launch_chunk_tile(const ChunkArgs& a, bool fp8, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                              const CUtensorMap& tm_v, int num_sms, cudaStream_t stream)
{
    if (a.d == 128)
        return fp8 ? launch_tiles<128, true>(a, tm_q, tm_k, tm_v, num_sms, stream)
                   : launch_tiles<128, false>(a, tm_q, tm_k, tm_v, num_sms, stream);
    return fp8 ? launch_tiles<64, true>(a, tm_q, tm_k, tm_v, num_sms, stream)
               : launch_tiles<64, false>(a, tm_q, tm_k, tm_v, num_sms, stream);
}

}  // namespace kvattn

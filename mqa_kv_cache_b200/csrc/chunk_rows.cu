// chunk_rows.cu -- attention of chunks over a paged KV cache for calls with few query
// rows per (sequence, KV head): single tokens, or a few guessed ones to check.
//
// Method: out = softmax_{j <= p} (scale q . k_j) v_j for the query at position p, query
// head h reading KV head h / g ("注意力变体与 MoE", GQA attention(): the g heads of a
// group share one K/V); all rows of a (sequence, KV head), its tokens times g heads, 32
// at most, meet each cached row together, so every one is read once and the kernel is
// bound by that read.  The products run on mma.sync with the keys (then the columns of V)
// as M and 8 query rows as N: S^T = K Q^T, O^T = V^T P^T, so that 8 rows, a group of 8
// heads decoding, waste nothing; P^T's fragments are S^T's, transposed (movmatrix).
//
// Work: the 64-key tiles of all (sequence, KV head) units form one line, dealt out to the
// CTAs in equal stretches (as decode_plan.cuh does for contiguous caches); a stretch of a
// unit is a piece.  A unit in one piece is finished at once; otherwise each piece leaves
// an unnormalised partial and the CTA that finishes last joins them (up to 32 at once, more
// in groups of 16 and then the groups), always in the same order.
//
// Four warps per 8 or 16 query rows: 32 keys of every other tile each, with their own running
// maximum and sum, joined at the end of a piece.  One warp loads (one box per page and 64-column
// half, page entries fetched one tile ahead; the piece's query rows), the last one makes
// the pieces.
//
// FP8: the codes become fp16 in registers, one conversion for two of them (exact).  K: a
// thread's codes of a key are 16-byte loads, the k order of the MMA being free as long as Q
// follows it; Q is scaled per row by a power of two into fp16's range, its largest element to
// [2^14, 2^15) (bf16's eight bits are exact there down to 2^-31 of it; a smaller element rounds
// to a multiple of at most 2^-38 of it, far below the fp32 sums' own rounding).  V: transposed as pairs of bytes, the even columns of 16 being the first
// eight rows of V^T's tile and the odd ones the others.  Weights enter the product as
// 2^(14 + s_j + log2 vs_j - m), so the values' scales cost an addition and the product's largest
// weight is near 2^14 whatever they are: what is below 2^-39 of it is lost to fp16 (from 2^-25 on if it stood
// at 1, and 16K such weights of 2^-25 are 2^-11 of the sum).
//
// Measured (d = 128): one token each over 16 sequences of 1K - 8K rows, 32 / 8 heads, bf16 51.6 us =
// 5.5 TB/s; over 16 of 32K rows, 64 / 8 heads, FP8 204 us = 5.4 TB/s (the loads alone, without the
// arithmetic, 174).
#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"

namespace kvattn {

namespace {

constexpr int RK = 64;        // keys per tile
constexpr int RBATCH = 16;    // partials requested together
constexpr int RPIECES = 4;    // pieces handed out ahead
constexpr float kWeightLog2 = 14.f;  // FP8: the largest weight of the product, in log2 units
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

struct RowPiece {
    int b, kvh;
    int t0, n;      // packed tokens (n = 0: no more pieces)
    int pos0, keys; // position of the first token; keys in use
    int tb, te;     // tiles
    int first;      // CTA that holds the unit's first piece
    int count;      // pieces of the unit
};

// NQ: n-tiles of 8 query rows in a warp; NMT: sets of four warps, each with its own such rows.
template <int D, bool FP8, int NQ, int NMT>
struct RCfg {
    static constexpr int WR = 8 * NQ;      // query rows of a set of warps
    static constexpr int RM = WR * NMT;
    static constexpr int RW = 4 * NMT;
    static constexpr int THREADS = 32 * (RW + 2);
    static constexpr int CTAS = FP8 && NMT == 1 ? 2 : 1;  // per SM
    static constexpr int ROWB = D * (FP8 ? 1 : 2) < 128 ? 64 : 128;  // bytes of a row of a box, and its swizzle
    static constexpr int HALVES = D * (FP8 ? 1 : 2) / ROWB;           // boxes side by side
    static constexpr int BOXD = D / HALVES;                           // columns of one
    static constexpr int BOX = RK * ROWB;
    static constexpr int TILE = HALVES * BOX;          // K or V
    static constexpr int SCB = FP8 ? 2 * RK * 4 : 0;   // their scales
    static constexpr int STAGE = 2 * TILE;
    static constexpr int STAGES = (FP8 ? (NMT == 1 ? 4 : 8) : (NMT == 1 ? 6 : 4)) * (D == 128 ? 1 : 2);
    static_assert(STAGES % 2 == 0, "a stage always holds even tiles or always odd ones: its barriers count one half of the warps");
    static constexpr int SCR = D + 8;                  // floats per scratch row
    static constexpr int OFF_SC = STAGES * STAGE;
    static constexpr int OFF_Q = OFF_SC + STAGES * SCB;  // two pieces' query rows
    static constexpr int QB = RM * D * 2;
    static constexpr int OFF_O = OFF_Q + 2 * QB;         // [NMT][2][WR][SCR]
    static constexpr int OFF_ML = OFF_O + 2 * RM * SCR * 4;  // [RW][WR] (m, l)
    static constexpr int OFF_U = OFF_ML + RW * WR * 8;
    static constexpr int OFF_PIECE = OFF_U + (PAGED_MAX_B + 1) * 8;
    static constexpr int OFF_BAR = OFF_PIECE + (RPIECES * static_cast<int>(sizeof(RowPiece)) + 7) / 8 * 8;
    // full[STAGES], empty[STAGES], q_full[2], q_empty[2], piece_full[RPIECES], piece_empty[RPIECES], met
    static constexpr int NBAR = 2 * STAGES + 5 + 2 * RPIECES;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM = OFF_MISC + 64 + STAGES * 4 + 1024;
    static_assert(SMEM * CTAS <= 233472 - 1024 * CTAS, "shared memory");
};

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t h;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
    return h;
}

// The four codes of w, two fp16 pairs.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// warp_wait with a first look that asks for the phase alone.
__device__ __forceinline__ bool ready(uint64_t* bar, uint32_t parity, volatile int* abort_flag)
{
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || warp_wait(bar, parity, abort_flag);
}

// Pieces joined together: a unit of up to 32 at once, in two batches; one of more by 16, and then those.  (By 32
// throughout: 37 pieces of 8 rows 16.6 us instead of 13.7; by 16 throughout: 19 of them 14.0 instead of 12.7.)
__device__ __forceinline__ int group_size(int count) { return count <= 2 * RBATCH ? 2 * RBATCH : RBATCH; }

// Byte offset of 16-byte chunk `ch` (of 4) of row r in a 64-byte-swizzled block of 64-byte rows.
__device__ __forceinline__ uint32_t swz64(int r, int ch) { return static_cast<uint32_t>(r * 64 + ((ch ^ ((r >> 1) & 3)) << 4)); }

// The partial slots of pieces i0 .. i1 - 1 (every `step`-th) of the unit whose first piece is CTA f's,
// joined by `nthr` threads: into the unit's rows, or (unnormalised) into the slot of piece i0, with
// (maximum, sum) beside it, as other threads still read the slot's own.  A group's partials are all
// requested at once: a call waits for memory rows * D / 4 / nthr times.
template <int D, int RM>
__device__ void join_pieces(const ChunkArgs& a, int gs, int f, int i0, int i1, int step, const RowPiece& pc, bool last,
                            int tid, int nthr)
{
    constexpr int Q4 = D / 4;
    auto slot = [f](int i) { return static_cast<long long>(i == 0 ? 2 * f + 1 : 2 * (f + i)) * RM; };
    for (int idx = tid; idx < (pc.n << gs) * Q4; idx += nthr) {
        const int r = idx / Q4, q4 = idx - r * Q4;
        float M = -INFINITY, L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int i = i0; i < i1; i += RBATCH * step) {
            float2 ml[RBATCH];
            float4 o[RBATCH];
#pragma unroll
            for (int k = 0; k < RBATCH; ++k) {
                ml[k] = make_float2(-INFINITY, 0.f);
                o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i + k * step < i1) {
                    const long long s = slot(i + k * step) + r;
                    ml[k] = __ldcg(a.part_ml + s);
                    o[k] = __ldcg(reinterpret_cast<const float4*>(a.part_o + s * D) + q4);
                }
            }
            float Mn = M;
#pragma unroll
            for (int k = 0; k < RBATCH; ++k) Mn = fmaxf(Mn, ml[k].x);
            const float mu = Mn == -INFINITY ? 0.f : Mn;
            const float c = fast_exp2(M - mu);
            L = sum_exp2(L, M - mu);
            acc = make_float4(acc.x * c, acc.y * c, acc.z * c, acc.w * c);
            M = Mn;
#pragma unroll
            for (int k = 0; k < RBATCH; ++k) {
                const float e = fast_exp2(ml[k].x - mu);
                L += sum_exp2(ml[k].y, ml[k].x - mu);
                acc.x += e * o[k].x;
                acc.y += e * o[k].y;
                acc.z += e * o[k].z;
                acc.w += e * o[k].w;
            }
        }
        if (last) {
            const float inv = L > 0.f ? 1.f / L : 0.f;
            const long long row = static_cast<long long>(pc.t0 + (r >> gs)) * a.H + (static_cast<long long>(pc.kvh) << gs) + (r & ((1 << gs) - 1));
            *reinterpret_cast<uint2*>(a.out + row * D + 4 * q4) =
                make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
            if (q4 == 0 && a.lse) a.lse[row] = L > 0.f ? (M + __log2f(L)) * kLn2 : -INFINITY;
        } else {
            const long long s = slot(i0) + r;
            __stcg(reinterpret_cast<float4*>(a.part_o + s * D) + q4, acc);
            if (q4 == 0) __stcg(a.join_ml + s, make_float2(M, L));
        }
    }
}

template <int D, bool FP8, int NQ, int NMT>
__global__ void __launch_bounds__(RCfg<D, FP8, NQ, NMT>::THREADS, RCfg<D, FP8, NQ, NMT>::CTAS)
    chunk_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, ChunkArgs a)
{
    using C = RCfg<D, FP8, NQ, NMT>;
    constexpr int KS = D / 16, STAGES = C::STAGES, RM = C::RM, RW = C::RW, WR = C::WR;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);  // (stays a shared-memory address to the compiler)
    float* s_o = reinterpret_cast<float*>(smem + C::OFF_O);
    float2* s_ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    long long* s_U = reinterpret_cast<long long*>(smem + C::OFF_U);
    RowPiece* s_piece = reinterpret_cast<RowPiece*>(smem + C::OFF_PIECE);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* empty = full + STAGES;
    uint64_t* q_full = empty + STAGES;
    uint64_t* q_empty = q_full + 2;
    uint64_t* piece_full = q_empty + 2;
    uint64_t* piece_empty = piece_full + RPIECES;
    uint64_t* met = piece_empty + RPIECES;  // the consumer warps, at a barrier
    volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
    int* s_join = reinterpret_cast<int*>(smem + C::OFF_MISC) + 1;  // [2] whether this CTA joins its split units' groups
    volatile uint32_t* s_bad = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC + 64);  // [STAGES] 16-key groups without a page

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x;
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], RW / 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], RW);
        }
        for (int i = 0; i < RPIECES; ++i) {
            mbar_init(&piece_full[i], 1);
            mbar_init(&piece_empty[i], RW + 1);
        }
        mbar_init(met, RW);
        *s_abort = 0;
        fence_barrier_init();
    }
    if (warp == RW && lane == 0) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    pdl_wait();
    pdl_trigger();

    // ---- the line: tiles of every sequence (on one KV head), and their prefix ----
    const PagedBatch& p = a.p;
    auto seq = [&](int b, int c0, int c1, int len, int& take, int& keys) {
        const PagedSeq s = paged_seq(p, c0, c1, len);
        take = min(s.n, a.max_q);
        keys = take > 0 ? max(s.len - s.n + take, 0) : 0;  // up to the last computed token
        return s;
    };
    for (int b = threadIdx.x; b < p.B; b += C::THREADS) {
        int take, keys;
        const PagedSeq s = seq(b, p.cu[b], p.cu[b + 1], p.seq_lens[b], take, keys);
        if (c == 0 && (s.bad || s.n > a.max_q)) report_status(p.dev_status, KVATTN_STATUS_BAD_LENGTH);
        s_U[b + 1] = (keys + RK - 1) / RK;
        if (keys == 0 && b % gridDim.x == c) {  // nothing to see: zeros and -inf
            for (int i = 0; i < take * a.H * (D / 8); ++i)
                reinterpret_cast<uint4*>(a.out)[static_cast<long long>(s.t0) * a.H * (D / 8) + i] = make_uint4(0, 0, 0, 0);
            if (a.lse)
                for (int i = 0; i < take * a.H; ++i) a.lse[static_cast<long long>(s.t0) * a.H + i] = -INFINITY;
        }
    }
    if (threadIdx.x == 0) s_U[0] = 0;
    __syncthreads();
    if (threadIdx.x < 32 && p.B > 1) {
        const int per = (p.B + 31) / 32;
        const int beg = min(lane * per, p.B), end = min(beg + per, p.B);
        long long sum = 0;
        for (int b = beg; b < end; ++b) sum += s_U[b + 1];
        long long incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        long long run = incl - sum;
        for (int b = beg; b < end; ++b) {
            run += s_U[b + 1];
            s_U[b + 1] = run;
        }
    }
    __syncthreads();
    auto take_piece = [&](int i, RowPiece& pc) {
        const int k = i % RPIECES;
        if (!warp_wait(&piece_full[k], (i / RPIECES) & 1, s_abort)) return false;
        pc = s_piece[k];
        __syncwarp();
        if (lane == 0) mbar_arrive(&piece_empty[k]);
        return pc.n > 0;
    };

    if (warp == RW + 1) {
        // ===== the pieces of this CTA's stretch =====
        if (lane != 0) return;
        const long long N = s_U[p.B] * a.Hk;
        const int G = static_cast<int>(min(N, static_cast<long long>(gridDim.x)));
        int np = 0;
        bool ok = true;
        auto put = [&](const RowPiece& pc) {
            const int k = np % RPIECES;
            if (np >= RPIECES && !(ok = !*s_abort && mbar_wait(&piece_empty[k], (np / RPIECES - 1) & 1))) {
                *s_abort = 1;
                return;
            }
            s_piece[k] = pc;
            mbar_arrive(&piece_full[k]);
            ++np;
        };
        if (c < G) {
            const long long lo = (c * N + G - 1) / G, hi = ((c + 1) * N + G - 1) / G;
            int b = 0, z = p.B - 1;
            while (b < z) {
                const int mid = (b + z + 1) >> 1;
                if (s_U[mid] * a.Hk <= lo) b = mid;
                else z = mid - 1;
            }
            int n = static_cast<int>(s_U[b + 1] - s_U[b]);
            int kvh = static_cast<int>((lo - s_U[b] * a.Hk) / n);
            while (ok && b < p.B) {
                const long long U = s_U[b] * a.Hk + static_cast<long long>(kvh) * n;
                if (U >= hi) break;
                RowPiece pc;
                int keys;
                const PagedSeq s = seq(b, p.cu[b], p.cu[b + 1], p.seq_lens[b], pc.n, keys);
                pc.b = b;
                pc.kvh = kvh;
                pc.t0 = s.t0;
                pc.pos0 = s.len - s.n;
                pc.keys = keys;
                pc.tb = static_cast<int>(max(lo, U) - U);
                pc.te = static_cast<int>(min(hi, U + n) - U);
                pc.first = static_cast<int>(U * G / N);
                pc.count = static_cast<int>((U + n - 1) * G / N) - pc.first + 1;
                put(pc);
                if (++kvh == a.Hk) {
                    kvh = 0;
                    do ++b;
                    while (b < p.B && s_U[b + 1] == s_U[b]);
                    if (b < p.B) n = static_cast<int>(s_U[b + 1] - s_U[b]);
                }
            }
        }
        RowPiece none{};
        if (ok) put(none);
        return;
    }

    if (warp == RW) {
        // ===== loads: lanes 0-15 K, 16-31 V; lane i of 16 takes box i / HALVES, half i % HALVES =====
        const int bp_shift = min(p.page_shift, 6);
        const int bp = 1 << bp_shift;
        const int box = (lane & 15) / C::HALVES, half = (lane & 15) % C::HALVES;
        const bool is_v = lane >= 16;
        const int oob = p.n_pages * a.Hk;  // reads as zeros
        const uint64_t pol = l2_evict_first_policy();  // the cache is read once
        uint32_t it = 0;
        int np = 0;
        bool ok = true;
        RowPiece pc;
        for (; ok && take_piece(np, pc); ++np) {
            uint8_t* sq = smem + C::OFF_Q + (np & 1) * C::QB;
            if (np >= 2 && !(ok = warp_wait(&q_empty[np & 1], (np / 2 - 1) & 1, s_abort))) break;
            if (lane == 0) mbar_arrive_expect_tx(&q_full[np & 1], pc.n * a.g * D * 2);
            __syncwarp();
            if (lane < pc.n)
                bulk_load(sq + lane * a.g * D * 2,
                          a.q + (pc.t0 + lane) * a.q_st + static_cast<long long>(pc.kvh) * a.g * D, a.g * D * 2, &q_full[np & 1]);
            const int32_t* pt = p.page_table + static_cast<long long>(pc.b) * p.max_pages;
            auto entry = [&](int t) {
                const int row = t * RK + (box << bp_shift);
                return box < (RK >> bp_shift) && row < pc.keys ? __ldg(pt + (row >> p.page_shift)) : 0;
            };
            int e = entry(pc.tb);
            for (int t = pc.tb; t < pc.te; ++t, ++it) {
                const int row = t * RK + (box << bp_shift);
                const bool mine = box < (RK >> bp_shift) && row < pc.keys;
                const int e_next = t + 1 < pc.te ? entry(t + 1) : 0;
                const bool bad = mine && (e < 0 || e >= p.n_pages);
                const uint32_t bads = __ballot_sync(0xffffffffu, bad && half == 0 && !is_v);
                const uint32_t s = it % STAGES;
                if (it >= STAGES && !(ok = warp_wait(&empty[s], (it / STAGES - 1) & 1, s_abort))) break;
                const int boxes = (min(pc.keys - t * RK, RK) + bp - 1) >> bp_shift;
                if (lane == 0) {
                    uint32_t groups = 0;
                    if (bads) {
                        report_status(p.dev_status, KVATTN_STATUS_BAD_INDEX);
                        for (int i = 0; i < (RK >> bp_shift); ++i)
                            if (bads >> (i * C::HALVES) & 1) groups |= ((1u << (bp >> 4)) - 1u) << (i * (bp >> 4));
                    }
                    s_bad[s] = groups;
                    mbar_arrive_expect_tx(&full[s], boxes * bp * C::ROWB * C::HALVES * 2 +
                                                        (FP8 ? (boxes - __popc(bads)) * bp * 8 : 0));
                }
                __syncwarp();
                if (mine) {
                    const int z = bad ? oob : e * a.Hk + pc.kvh;
                    const int y = row & ((1 << p.page_shift) - 1);
                    tma_load_3d_hint(smem + s * C::STAGE + (is_v ? C::TILE : 0) + half * C::BOX + (box << bp_shift) * C::ROWB,
                                     is_v ? &tm_v : &tm_k, &full[s], half * C::BOXD, y, z, pol);
                    if (FP8 && half == 0 && !bad)
                        bulk_load(smem + C::OFF_SC + s * C::SCB + (is_v ? RK * 4 : 0) + (box << bp_shift) * 4,
                                  (is_v ? a.v_scales : a.k_scales) + ((static_cast<long long>(z) << p.page_shift) + y), bp * 4,
                                  &full[s]);
                }
                e = e_next;
            }
        }
        if (lane == 0) {
            if (!ok) report_status(p.dev_status, KVATTN_STATUS_TIMEOUT);
            // copies in flight complete before the CTA leaves (bounded waits)
            for (uint32_t i = it > STAGES ? it - STAGES : 0; i < it; ++i) mbar_wait(&full[i % STAGES], (i / STAGES) & 1);
            for (int i = np > 2 ? np - 2 : 0; i < np; ++i) mbar_wait(&q_full[i & 1], (i / 2) & 1);
        }
        return;
    }

    // ===== consumers =====
    const int r0 = lane >> 2, cq = lane & 3;
    const int mt = warp >> 2, sub = warp & 3;
    const uint32_t turn = sub >> 1;   // even or odd tiles
    const int tok0 = (sub & 1) * 32;  // this warp's keys of a tile
    const int mi = lane >> 3, rr = lane & 7;
    const float sl2 = a.scale * kLog2e;
    int gs = 0;
    while ((1 << gs) < a.g) ++gs;
    uint32_t it = 0, meets = 0;
    // barrier of the consumer warps: like every wait here, it gives up once a wait has run out
    auto meet = [&] {
        __syncwarp();
        if (lane == 0) mbar_arrive(met);
        ready(met, meets++ & 1, s_abort);
    };
    int n_split = 0;
    RowPiece pc, split[2];
    for (int np = 0; take_piece(np, pc); ++np) {
        const int rows = pc.n * a.g;
        // Q^T fragments: thread's query row r0 of each n-tile (rows past the last one: zero)
        uint32_t qb[NQ][KS][2];
        float qs[NQ][2];  // what turns a raw score of queries 2 cq, 2 cq + 1 into log2 units
        int pos[NQ][2];   // their positions
        {
            const bool have = warp_wait(&q_full[np & 1], (np / 2) & 1, s_abort);
            const uint8_t* sq = smem + C::OFF_Q + (np & 1) * C::QB;
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                const int row = mt * WR + n * 8 + r0;
                const bool v = have && row < rows;
                const uint8_t* qr = sq + row * D * 2;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    qs[n][e] = sl2;
                    pos[n][e] = pc.pos0 + ((mt * WR + n * 8 + 2 * cq + e) >> gs);
                }
                if constexpr (FP8) {
                    // k step x of thread cq: columns (D / 4) cq + 4 x + {0, 1 | 2, 3}
                    float m = 0.f;
#pragma unroll
                    for (int x = 0; x < KS; ++x) {
                        const uint2 y = v ? *reinterpret_cast<const uint2*>(qr + (cq * (D / 4) + 4 * x) * 2) : make_uint2(0, 0);
                        qb[n][x][0] = y.x;
                        qb[n][x][1] = y.y;
                        m = fmaxf(m, fmaxf(fmaxf(fabsf(bf16_lo(y.x)), fabsf(bf16_hi(y.x))), fmaxf(fabsf(bf16_lo(y.y)), fabsf(bf16_hi(y.y)))));
                    }
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                    // largest element to [2^14, 2^15): two factors, as one alone may leave fp32's range
                    const int ex = m > 0.f ? 14 - ilogbf(m) : 0;
                    const float fa = ldexpf(1.f, ex / 2), fb = ldexpf(1.f, ex - ex / 2);
#pragma unroll
                    for (int x = 0; x < KS; ++x)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            qb[n][x][e] = pack_f16x2(bf16_lo(qb[n][x][e]) * fa * fb, bf16_hi(qb[n][x][e]) * fa * fb);
#pragma unroll
                    for (int e = 0; e < 2; ++e) qs[n][e] = ldexpf(sl2, -__shfl_sync(0xffffffffu, ex, (2 * cq + e) * 4));
                } else {
#pragma unroll
                    for (int x = 0; x < KS; ++x) {
                        qb[n][x][0] = v ? *reinterpret_cast<const uint32_t*>(qr + (x * 16 + 2 * cq) * 2) : 0u;
                        qb[n][x][1] = v ? *reinterpret_cast<const uint32_t*>(qr + (x * 16 + 2 * cq + 8) * 2) : 0u;
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_empty[np & 1]);
        }
        const int pos_min = pc.pos0 + ((mt * WR) >> gs);
        float o[NQ][D / 16][4];  // O^T: 16 columns of V, 8 query rows
        float m[NQ][2], l[NQ][2];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
        }

        for (int t = pc.tb; t < pc.te; ++t, ++it) {
            if ((it & 1) != turn) continue;
            const uint32_t s = it % STAGES;
            if (ready(&full[s], (it / STAGES) & 1, s_abort)) {
                const uint8_t* kt = smem + s * C::STAGE;
                const uint32_t sk = smem_u32(kt), sv = sk + C::TILE;
                const uint32_t bad = s_bad[s] >> (tok0 / 16) & 3u;  // this warp's groups of 16 keys without a page
                const int nv = pc.keys - t * RK - tok0;             // keys of this warp's that are in use
                // ---- S^T: 2 m-tiles of 16 keys ----
                float sc[NQ][2][4];
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) sc[n][i][0] = sc[n][i][1] = sc[n][i][2] = sc[n][i][3] = 0.f;
                if constexpr (FP8) {
#pragma unroll
                    for (int y = 0; y < D / 64; ++y) {  // D = 128: the thread's 32 codes are chunks 2 cq and 2 cq + 1
                        uint4 ka[2], kb[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int row = tok0 + i * 16 + r0;
                            ka[i] = *reinterpret_cast<const uint4*>(kt + (D == 128 ? swz128(row, 2 * cq + y) : swz64(row, cq)));
                            kb[i] = *reinterpret_cast<const uint4*>(kt + (D == 128 ? swz128(row + 8, 2 * cq + y) : swz64(row + 8, cq)));
                        }
#pragma unroll
                        for (int x = 0; x < 4; ++x)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t wa = x == 0 ? ka[i].x : x == 1 ? ka[i].y : x == 2 ? ka[i].z : ka[i].w;
                                const uint32_t wb = x == 0 ? kb[i].x : x == 1 ? kb[i].y : x == 2 ? kb[i].z : kb[i].w;
                                uint32_t f[4];
                                codes_to_f16(wa, f[0], f[2]);
                                codes_to_f16(wb, f[1], f[3]);
#pragma unroll
                                for (int n = 0; n < NQ; ++n) mma_f16_16816(sc[n][i], f, qb[n][y * 4 + x][0], qb[n][y * 4 + x][1]);
                            }
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < KS; ++x) {
                        const int dim = x * 16 + ((mi >> 1) << 3);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t f[4];
                            ldsm_x4(sk + (dim >> 6) * C::BOX + swz128(tok0 + i * 16 + rr + ((mi & 1) << 3), (dim & 63) >> 3),
                                    f[0], f[1], f[2], f[3]);
#pragma unroll
                            for (int n = 0; n < NQ; ++n) mma_bf16_16816(sc[n][i], f, qb[n][x][0], qb[n][x][1]);
                        }
                    }
                }
                // ---- scores in log2 units; keys past a row's position (or without a page) -> -inf ----
                const bool masked = bad || t * RK + tok0 + 31 > pos_min;
                float ks[2][2], lv[2][2];  // (FP8) scales of keys r0 and r0 + 8 of each m-tile; log2 of the values'
                if constexpr (FP8) {
                    const float* scl = reinterpret_cast<const float*>(smem + C::OFF_SC + s * C::SCB) + tok0 + r0;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            ks[i][e] = scl[i * 16 + e * 8];
                            lv[i][e] = lg2(scl[RK + i * 16 + e * 8]);  // a zero row: -inf, its weight 0
                            // a scale that stands for no key may be anything, NaN included
                            if (masked && ((bad >> i & 1u) || i * 16 + e * 8 + r0 >= nv)) lv[i][e] = 0.f;
                        }
                }
                bool up = false;
                float mx[NQ][2];
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    mx[n][0] = mx[n][1] = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float x = sc[n][i][e] * (FP8 ? qs[n][e & 1] * ks[i][e >> 1] : sl2);
                            if (masked && ((bad >> i & 1u) || t * RK + tok0 + i * 16 + (e >> 1) * 8 + r0 > pos[n][e & 1])) x = -INFINITY;
                            sc[n][i][e] = x;
                            // FP8: the sums use the same reference as the weighted values
                            mx[n][e & 1] = fmaxf(mx[n][e & 1], FP8 ? fmaxf(x + lv[i][e >> 1], x + CHUNK_MIN_LOG2_VS) : x);
                        }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        mx[n][e] = fmaxf(mx[n][e], __shfl_xor_sync(0xffffffffu, mx[n][e], 4));
                        mx[n][e] = fmaxf(mx[n][e], __shfl_xor_sync(0xffffffffu, mx[n][e], 8));
                        mx[n][e] = fmaxf(mx[n][e], __shfl_xor_sync(0xffffffffu, mx[n][e], 16));
                        up |= mx[n][e] > m[n][e];
                    }
                }
                if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        float al[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float mn = fmaxf(m[n][e], mx[n][e]);
                            al[e] = m[n][e] == -INFINITY ? 0.f : fast_exp2(m[n][e] - mn);
                            if (m[n][e] != -INFINITY) l[n][e] = sum_exp2(l[n][e], m[n][e] - mn);
                            m[n][e] = mn;
                        }
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            o[n][i][0] *= al[0];
                            o[n][i][1] *= al[1];
                            o[n][i][2] *= al[0];
                            o[n][i][3] *= al[1];
                        }
                    }
                }
                // ---- P^T ----
                if constexpr (FP8) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e) lv[i][e] += kWeightLog2;
                }
                uint32_t pb[NQ][2][2];
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    const float mu[2] = {m[n][0] == -INFINITY ? 0.f : m[n][0], m[n][1] == -INFINITY ? 0.f : m[n][1]};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x = sc[n][i][e] - mu[e & 1], y = fast_exp2(x);
                            l[n][e & 1] += y;
                            w[e] = FP8 ? fast_exp2(x + lv[i][e >> 1]) : y;
                        }
                        pb[n][i][0] = transpose8x8(FP8 ? pack_f16x2(w[0], w[1]) : pack_bf16x2(w[0], w[1]));
                        pb[n][i][1] = transpose8x8(FP8 ? pack_f16x2(w[2], w[3]) : pack_bf16x2(w[2], w[3]));
                    }
                }
                // ---- O^T += V^T P^T; rows behind the last key in use may hold anything: zeros instead ----
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const bool b = bad >> j & 1u;
                    const bool tail = b || nv < j * 16 + 16;
                    uint32_t z0 = 0xffffffffu, z1 = 0xffffffffu;
                    if (tail) {
                        const int v0 = j * 16 + 2 * cq;
                        z0 = b ? 0u : (v0 < nv ? 0x0000ffffu : 0u) | (v0 + 1 < nv ? 0xffff0000u : 0u);
                        z1 = b ? 0u : (v0 + 8 < nv ? 0x0000ffffu : 0u) | (v0 + 9 < nv ? 0xffff0000u : 0u);
                    }
                    if constexpr (FP8) {
                        const int vrow = tok0 + j * 16 + rr + ((mi & 1) << 3);
#pragma unroll
                        for (int dg = 0; dg < D / 32; ++dg) {
                            // keys 0-7 | 8-15 of 16 columns, and of the next 16
                            const int ch = dg * 2 + (mi >> 1);
                            uint32_t v[4];
                            ldsm_x4_t(sv + (D == 128 ? swz128(vrow, ch) : swz64(vrow, ch)), v[0], v[1], v[2], v[3]);
                            if (tail) {
                                v[0] &= z0;
                                v[2] &= z0;
                                v[1] &= z1;
                                v[3] &= z1;
                            }
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint32_t f[4];
                                // even columns' pair of keys | odd columns'
                                codes_to_f16(__byte_perm(v[2 * h], 0u, 0x3120), f[0], f[1]);
                                codes_to_f16(__byte_perm(v[2 * h + 1], 0u, 0x3120), f[2], f[3]);
#pragma unroll
                                for (int n = 0; n < NQ; ++n) mma_f16_16816(o[n][2 * dg + h], f, pb[n][j][0], pb[n][j][1]);
                            }
                        }
                    } else {
                        const int vrow = tok0 + j * 16 + rr + ((mi >> 1) << 3);
#pragma unroll
                        for (int dp = 0; dp < D / 16; ++dp) {
                            const int dim = dp * 16 + ((mi & 1) << 3);
                            uint32_t f[4];
                            ldsm_x4_t(sv + (dim >> 6) * C::BOX + swz128(vrow, (dim & 63) >> 3), f[0], f[1], f[2], f[3]);
                            if (tail) {
                                f[0] &= z0;
                                f[1] &= z0;
                                f[2] &= z1;
                                f[3] &= z1;
                            }
#pragma unroll
                            for (int n = 0; n < NQ; ++n) mma_bf16_16816(o[n][dp], f, pb[n][j][0], pb[n][j][1]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
        }

        // ---- join the four warps: each row's common maximum, then sums over scratch memory ----
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 4);
                l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 8);
                l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 16);
                if (r0 == 0) s_ml[warp * WR + n * 8 + 2 * cq + e] = make_float2(m[n][e], l[n][e]);
            }
        meet();
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float2* ml = s_ml + mt * 4 * WR + n * 8 + 2 * cq + e;
                float M = -INFINITY, L = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) M = fmaxf(M, ml[j * WR].x);
                const float mu = M == -INFINITY ? 0.f : M;
#pragma unroll
                for (int j = 0; j < 4; ++j) L += sum_exp2(ml[j * WR].y, ml[j * WR].x - mu);
                const float w = fast_exp2(m[n][e] - mu - (FP8 ? kWeightLog2 : 0.f));
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    o[n][i][e] *= w;
                    o[n][i][2 + e] *= w;
                }
                m[n][e] = M;
                l[n][e] = L;
            }
        // (query row, first column, and the step to the second one) of o[n][i][e] and o[n][i][2 + e]
        constexpr int CS = FP8 ? 1 : 8;
        float* so = s_o + (mt * 2 + (sub & 1)) * WR * C::SCR + 2 * cq * C::SCR + (FP8 ? 2 * r0 : r0);
        if (sub >= 2) {
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) so[(n * 8 + (e & 1)) * C::SCR + i * 16 + (e >> 1) * CS] = o[n][i][e];
        }
        meet();
        if (sub < 2) {
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) so[(n * 8 + (e & 1)) * C::SCR + i * 16 + (e >> 1) * CS] += o[n][i][e];
        }
        if (sub == 0 && r0 == 0) {  // (every warp has read the sums)
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) s_ml[warp * WR + n * 8 + 2 * cq + e] = make_float2(m[n][e], l[n][e]);
        }
        meet();
        // ---- the rows: finished, or a partial ----
        const long long slot = static_cast<long long>(2 * c + (c == pc.first ? 1 : 0)) * RM;
        for (int idx = threadIdx.x; idx < rows * (D / 4); idx += RW * 32) {
            const int r = idx / (D / 4), q4 = idx - r * (D / 4);
            const float* sr = s_o + ((r / WR) * 2 * WR + r % WR) * C::SCR + 4 * q4;
            const float4 x = *reinterpret_cast<const float4*>(sr), y = *reinterpret_cast<const float4*>(sr + WR * C::SCR);
            const float4 v = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
            const float2 ml = s_ml[(r / WR) * 4 * WR + r % WR];
            if (pc.count == 1) {
                const float inv = ml.y > 0.f ? 1.f / ml.y : 0.f;
                const long long row = static_cast<long long>(pc.t0 + (r >> gs)) * a.H + static_cast<long long>(pc.kvh) * a.g + (r & (a.g - 1));
                *reinterpret_cast<uint2*>(a.out + row * D + 4 * q4) =
                    make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
                if (q4 == 0 && a.lse) a.lse[row] = ml.y > 0.f ? (ml.x + __log2f(ml.y)) * kLn2 : -INFINITY;
            } else {
                __stcg(reinterpret_cast<float4*>(a.part_o + (slot + r) * D) + q4, v);
                if (q4 == 0) __stcg(a.part_ml + slot + r, ml);
            }
        }
        meet();
        if (pc.count > 1) {  // at most the first and the last unit of the stretch
            // (counters, zero between calls: a group's, by its first piece's CTA, those behind a unit's first group in a
            // second array, as that CTA may begin another unit; the unit's in a third)
            // the partial is there: counted now, so that a piece that the stretch begins with does not keep its unit
            // waiting for the rest of it; who counts the last one of a group joins it below
            if (threadIdx.x == 0) {
                int go = 0;
                if (!*s_abort) {
                    const int size = group_size(pc.count), i0 = (c - pc.first) / size * size;
                    int* gcnt = a.counters + (i0 > 0 ? CHUNK_MAX_SLOTS : 0) + pc.first + i0;
                    __threadfence();
                    go = atomicAdd(gcnt, 1) == min(size, pc.count - i0) - 1;
                    if (go) {
                        *gcnt = 0;
                        __threadfence();
                    }
                }
                s_join[n_split & 1] = go;
            }
            split[n_split++ & 1] = pc;
        }
    }

    // ---- the split units of this CTA: the last piece of a group joins it, the last group the unit ----
    if (n_split > 0) meet();
    for (int k = 0; k < n_split; ++k) {
        if (!s_join[k]) continue;
        const RowPiece& s = split[k];
        const int size = group_size(s.count), groups = (s.count + size - 1) / size;
        const int i0 = (c - s.first) / size * size, i1 = min(i0 + size, s.count);
        if (i1 - i0 <= RBATCH)  // (one batch, to the compiler too)
            join_pieces<D, RM>(a, gs, s.first, i0, min(i1, i0 + RBATCH), 1, s, groups == 1, threadIdx.x, RW * 32);
        else
            join_pieces<D, RM>(a, gs, s.first, i0, i1, 1, s, groups == 1, threadIdx.x, RW * 32);
        if (groups == 1) continue;
        meet();  // everyone has read the group's (m, l)
        const long long lead = static_cast<long long>(i0 == 0 ? 2 * s.first + 1 : 2 * (s.first + i0)) * RM;
        for (int r = threadIdx.x; r < s.n * a.g; r += RW * 32) __stcg(a.part_ml + lead + r, __ldcg(a.join_ml + lead + r));
        meet();
        if (threadIdx.x == 0) {
            int* ucnt = a.counters + 2 * CHUNK_MAX_SLOTS + s.first;
            __threadfence();
            const int go = atomicAdd(ucnt, 1) == groups - 1;
            if (go) {
                *ucnt = 0;
                __threadfence();
            }
            s_join[k] = go;
        }
        meet();
        if (s_join[k]) join_pieces<D, RM>(a, gs, s.first, 0, s.count, size, s, true, threadIdx.x, RW * 32);
    }
}

template <int D, bool FP8, int NQ, int NMT>
cudaError_t launch_typed(const ChunkArgs& a, const CUtensorMap& tm_k, const CUtensorMap& tm_v, int num_sms,
                         cudaStream_t stream)
{
    using C = RCfg<D, FP8, NQ, NMT>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !attr_set[dev]) {
        e = cudaFuncSetAttribute(chunk_rows_kernel<D, FP8, NQ, NMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        if (dev < 64) attr_set[dev] = true;
    }
    int grid = num_sms * C::CTAS;
    if (grid > CHUNK_MAX_SLOTS) grid = CHUNK_MAX_SLOTS;
    return launch_pdl(chunk_rows_kernel<D, FP8, NQ, NMT>, dim3(grid), dim3(C::THREADS), C::SMEM, stream, tm_k, tm_v, a);
}

template <int D, bool FP8>
cudaError_t launch_rows(const ChunkArgs& a, const CUtensorMap& tm_k, const CUtensorMap& tm_v, int num_sms,
                        cudaStream_t stream)
{
    const int rows = a.max_q * a.g;
    return rows <= 8    ? launch_typed<D, FP8, 1, 1>(a, tm_k, tm_v, num_sms, stream)
           : rows <= 16 ? launch_typed<D, FP8, 2, 1>(a, tm_k, tm_v, num_sms, stream)
                        : launch_typed<D, FP8, 2, 2>(a, tm_k, tm_v, num_sms, stream);
}

}  // namespace

cudaError_t launch_chunk_rows(const ChunkArgs& a, bool fp8, const CUtensorMap& tm_k, const CUtensorMap& tm_v, int num_sms,
                              cudaStream_t stream)
{
    if (a.d == 128)
        return fp8 ? launch_rows<128, true>(a, tm_k, tm_v, num_sms, stream)
                   : launch_rows<128, false>(a, tm_k, tm_v, num_sms, stream);
    return fp8 ? launch_rows<64, true>(a, tm_k, tm_v, num_sms, stream)
               : launch_rows<64, false>(a, tm_k, tm_v, num_sms, stream);
}

}  // namespace kvattn

// chunk_rows.cu -- attention of chunks over a paged KV cache for calls with few query
// rows per (sequence, KV head): single tokens, or a few guessed ones to check.
//
// Method: out = softmax_{j <= p} (scale q . k_j) v_j for the query at position p, query
// head h reading KV head h / g ("注意力变体与 MoE", GQA attention(): the g heads of a
// group share one K/V); all rows of a (sequence, KV head), its tokens times g heads, 32
// at most, are the M rows of one or two mma.sync tiles, so every cached row is read once
// and the kernel is bound by that read.
//
// Work: the 64-key tiles of all (sequence, KV head) units form one line, dealt out to the
// CTAs in equal stretches (as decode_plan.cuh does for contiguous caches); a stretch of a
// unit is a piece.  A unit in one piece is finished at once; otherwise each piece leaves
// an unnormalised partial and the CTA that finishes last joins them, in groups of 16
// pieces and then the groups, always in the same order.
//
// Four warps per 16 query rows: 32 keys of every other tile each, with their own running
// maximum and sum, joined at the end of a piece.  One warp loads (one box per page and 64-column
// half, page entries fetched one tile ahead; the piece's query rows), the last one makes
// the pieces.
//
// FP8: the codes become fp16 in registers, one conversion for two of them (exact).  K: a
// thread's 16 codes of a key are one load, the k order of the MMA being free as long as Q
// follows it; Q is scaled per row by a power of two into fp16's range (an element below
// 2^-29 of its row's largest rounds to a multiple of 2^-40 of it, far below the fp32 sums'
// own rounding).  V: transposed as pairs of bytes, the even and the odd columns of 16 being
// two n-tiles.  Weights enter the product as 2^(s_j + log2 vs_j - m), so the values'
// scales cost an addition and the product's largest weight is near 1 whatever they are.
#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"

namespace kvattn {

namespace {

constexpr int RK = 64;        // keys per tile
constexpr int RGROUP = 16;    // pieces joined together
constexpr int RPIECES = 4;    // pieces handed out ahead
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

// NMT: 16-row tiles of query rows; each has four consumer warps
template <int D, bool FP8, int NMT>
struct RCfg {
    static constexpr int RM = 16 * NMT;
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
    static constexpr int OFF_O = OFF_Q + 2 * QB;         // [NMT][2][16][SCR]
    static constexpr int OFF_ML = OFF_O + 2 * RM * SCR * 4;  // [RW][16] (m, l)
    static constexpr int OFF_U = OFF_ML + RW * 16 * 8;
    static constexpr int OFF_PIECE = OFF_U + (PAGED_MAX_B + 1) * 8;
    static constexpr int OFF_BAR = OFF_PIECE + (RPIECES * static_cast<int>(sizeof(RowPiece)) + 7) / 8 * 8;
    // full[STAGES], empty[STAGES], q_full[2], q_empty[2], piece_full[RPIECES], piece_empty[RPIECES]
    static constexpr int NBAR = 2 * STAGES + 4 + 2 * RPIECES;
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

__device__ __forceinline__ uint32_t codes_to_f16x2(uint32_t w)  // the low two codes
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w)));
    return h;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t h;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
    return h;
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

// Byte offset of 16-byte chunk `ch` (of 4) of row r in a 64-byte-swizzled block of 64-byte rows.
__device__ __forceinline__ uint32_t swz64(int r, int ch) { return static_cast<uint32_t>(r * 64 + ((ch ^ ((r >> 1) & 3)) << 4)); }

// The partial slots of pieces i0 .. i1 - 1 (every `step`-th) of the unit whose first piece is CTA f's,
// joined by `nthr` threads: into the unit's rows, or (unnormalised) into the slot of piece i0.
template <int D, int RM>
__device__ void join_pieces(const ChunkArgs& a, int f, int i0, int i1, int step, const RowPiece& pc, bool last, int tid,
                            int nthr)
{
    constexpr int Q4 = D / 4, BATCH = 8;
    const int rows = pc.n * a.g;
    auto slot = [f](int i) { return static_cast<long long>(i == 0 ? 2 * f + 1 : 2 * (f + i)) * RM; };
    for (int idx = tid; idx < rows * Q4; idx += nthr) {
        const int r = idx / Q4, q4 = idx - r * Q4;
        float M = -INFINITY, L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = i0; i < i1; i += BATCH * step) {
            float2 ml[BATCH];
            float4 o[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                if (i + k * step < i1) {
                    const long long s = slot(i + k * step) + r;
                    ml[k] = __ldcg(a.part_ml + s);
                    o[k] = __ldcg(reinterpret_cast<const float4*>(a.part_o + s * D) + q4);
                }
            }
            float Mn = M;
#pragma unroll
            for (int k = 0; k < BATCH; ++k)
                if (i + k * step < i1) Mn = fmaxf(Mn, ml[k].x);
            const float mu = Mn == -INFINITY ? 0.f : Mn;
            const float c = M == -INFINITY ? 0.f : fast_exp2(M - mu);
            L *= c;
            acc = make_float4(acc.x * c, acc.y * c, acc.z * c, acc.w * c);
            M = Mn;
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                if (i + k * step < i1) {
                    const float e = ml[k].x == -INFINITY ? 0.f : fast_exp2(ml[k].x - mu);
                    L += e * ml[k].y;
                    acc.x += e * o[k].x;
                    acc.y += e * o[k].y;
                    acc.z += e * o[k].z;
                    acc.w += e * o[k].w;
                }
            }
        }
        if (last) {
            const float inv = L > 0.f ? 1.f / L : 0.f;
            const long long row = static_cast<long long>(pc.t0 + r / a.g) * a.H + static_cast<long long>(pc.kvh) * a.g + r % a.g;
            *reinterpret_cast<uint2*>(a.out + row * D + 4 * q4) =
                make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
            if (q4 == 0 && a.lse) a.lse[row] = L > 0.f ? (M + __log2f(L)) * kLn2 : -INFINITY;
        } else {
            // every thread of the row has read (m, l) before this one's place is rewritten: see the barrier
            // at the caller, which lets all threads finish their reads first
            const long long s = slot(i0) + r;
            __stcg(reinterpret_cast<float4*>(a.part_o + s * D) + q4, acc);
            if (q4 == 0) __stcg(a.join_ml + s, make_float2(M, L));
        }
    }
}

template <int D, bool FP8, int NMT>
__global__ void __launch_bounds__(RCfg<D, FP8, NMT>::THREADS, RCfg<D, FP8, NMT>::CTAS)
    chunk_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, ChunkArgs a)
{
    using C = RCfg<D, FP8, NMT>;
    constexpr int KS = D / 16, DT = D / 8, STAGES = C::STAGES, RM = C::RM, RW = C::RW;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
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
    volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
    int* s_join = reinterpret_cast<int*>(smem + C::OFF_MISC) + 1;  // what this CTA is to join
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
    uint32_t it = 0;
    int n_split = 0;
    RowPiece pc, split[2];
    for (int np = 0; take_piece(np, pc); ++np) {
        const int rows = pc.n * a.g;
        // Q fragments (rows past the last one: zero), and with FP8 the rows' powers of two
        uint32_t qa[KS][4];
        float qs0 = sl2, qs1 = sl2;
        {
            const bool have = warp_wait(&q_full[np & 1], (np / 2) & 1, s_abort);
            const uint8_t* sq = smem + C::OFF_Q + (np & 1) * C::QB;
            const int ra = mt * 16 + r0, rb = ra + 8;
            const bool va = have && ra < rows, vb = have && rb < rows;
            if constexpr (FP8) {
                // k step 4 h + s of thread cq: columns 64 h + 16 cq + 4 s + {0, 1 | 2, 3}
                float m0 = 0.f, m1 = 0.f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const int col = (ks >> 2) * 64 + cq * 16 + (ks & 3) * 4;
                    const uint2 x = va ? *reinterpret_cast<const uint2*>(sq + (ra * D + col) * 2) : make_uint2(0, 0);
                    const uint2 y = vb ? *reinterpret_cast<const uint2*>(sq + (rb * D + col) * 2) : make_uint2(0, 0);
                    qa[ks][0] = x.x;
                    qa[ks][1] = y.x;
                    qa[ks][2] = x.y;
                    qa[ks][3] = y.y;
                    m0 = fmaxf(m0, fmaxf(fmaxf(fabsf(bf16_lo(x.x)), fabsf(bf16_hi(x.x))), fmaxf(fabsf(bf16_lo(x.y)), fabsf(bf16_hi(x.y)))));
                    m1 = fmaxf(m1, fmaxf(fmaxf(fabsf(bf16_lo(y.x)), fabsf(bf16_hi(y.x))), fmaxf(fabsf(bf16_lo(y.y)), fabsf(bf16_hi(y.y)))));
                }
                m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, 1));
                m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, 2));
                m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, 1));
                m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, 2));
                // largest element to [2^14, 2^15): two factors, as one alone may leave fp32's range
                const int x0 = m0 > 0.f ? 14 - ilogbf(m0) : 0, x1 = m1 > 0.f ? 14 - ilogbf(m1) : 0;
                const float fa0 = ldexpf(1.f, x0 / 2), fb0 = ldexpf(1.f, x0 - x0 / 2);
                const float fa1 = ldexpf(1.f, x1 / 2), fb1 = ldexpf(1.f, x1 - x1 / 2);
                qs0 = ldexpf(sl2, -x0);
                qs1 = ldexpf(sl2, -x1);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float fa = (i & 1) ? fa1 : fa0, fb = (i & 1) ? fb1 : fb0;
                        qa[ks][i] = pack_f16x2(bf16_lo(qa[ks][i]) * fa * fb, bf16_hi(qa[ks][i]) * fa * fb);
                    }
                }
            } else {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const int col = ks * 16 + 2 * cq;
                    qa[ks][0] = va ? *reinterpret_cast<const uint32_t*>(sq + (ra * D + col) * 2) : 0u;
                    qa[ks][1] = vb ? *reinterpret_cast<const uint32_t*>(sq + (rb * D + col) * 2) : 0u;
                    qa[ks][2] = va ? *reinterpret_cast<const uint32_t*>(sq + (ra * D + col + 8) * 2) : 0u;
                    qa[ks][3] = vb ? *reinterpret_cast<const uint32_t*>(sq + (rb * D + col + 8) * 2) : 0u;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_empty[np & 1]);
        }
        const int pos_a = pc.pos0 + ((mt * 16 + r0) >> gs), pos_b = pc.pos0 + ((mt * 16 + r0 + 8) >> gs);
        float o[DT][4];
#pragma unroll
        for (int i = 0; i < DT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

        for (int t = pc.tb; t < pc.te; ++t, ++it) {
            if ((it & 1) != turn) continue;
            const uint32_t s = it % STAGES;
            if (ready(&full[s], (it / STAGES) & 1, s_abort)) {
                const uint8_t* kt = smem + s * C::STAGE;
                const uint8_t* vt = kt + C::TILE;
                const uint32_t bad = s_bad[s] >> (tok0 / 16) & 3u;  // this warp's groups of 16 keys without a page
                const int nv = pc.keys - t * RK - tok0;             // keys of this warp's that are in use
                float sc[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
                if constexpr (FP8) {
                    // D = 128: odd keys read their upper 64 codes first, so that two keys' reads fall
                    // on different banks
                    const int odd = r0 & 1;
                    uint4 k4[4][D / 64];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = tok0 + i * 8 + r0;
                        if constexpr (D == 128) {
                            const uint4 x = *reinterpret_cast<const uint4*>(kt + swz128(row, odd * 4 + cq));
                            const uint4 y = *reinterpret_cast<const uint4*>(kt + swz128(row, (odd ^ 1) * 4 + cq));
                            k4[i][0] = odd ? y : x;
                            k4[i][D / 64 - 1] = odd ? x : y;
                        } else {
                            k4[i][0] = *reinterpret_cast<const uint4*>(kt + swz64(row, cq));
                        }
                    }
#pragma unroll
                    for (int h = 0; h < D / 64; ++h)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t kw = x == 0 ? k4[i][h].x : x == 1 ? k4[i][h].y : x == 2 ? k4[i][h].z : k4[i][h].w;
                                mma_f16_16816(sc[i], qa[h * 4 + x], codes_to_f16x2(kw), codes_to_f16x2(kw >> 16));
                            }
                } else {
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        const int dim = ks * 16 + ((mi & 1) << 3);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            uint32_t b0, b1, b2, b3;
                            ldsm_x4(smem_u32(kt) + (dim >> 6) * C::BOX +
                                        swz128(tok0 + j * 16 + rr + ((mi >> 1) << 3), (dim & 63) >> 3),
                                    b0, b1, b2, b3);
                            mma_bf16_16816(sc[2 * j], qa[ks], b0, b1);
                            mma_bf16_16816(sc[2 * j + 1], qa[ks], b2, b3);
                        }
                    }
                }
                // ---- scores in log2 units; keys past a row's position (or without a page) -> -inf ----
                const bool masked = bad || t * RK + tok0 + 31 > pc.pos0 + ((mt * 16) >> gs);
                float2 lv[4];  // log2 of the values' scales (FP8)
                float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float2 kv = make_float2(1.f, 1.f);
                    if constexpr (FP8) {
                        const float* scl = reinterpret_cast<const float*>(smem + C::OFF_SC + s * C::SCB) + tok0 + i * 8 + 2 * cq;
                        kv = *reinterpret_cast<const float2*>(scl);
                        const float2 v = *reinterpret_cast<const float2*>(scl + RK);
                        lv[i] = make_float2(lg2(v.x), lg2(v.y));  // a zero row: -inf, its weight 0
                    }
                    sc[i][0] *= qs0 * kv.x;
                    sc[i][1] *= qs0 * kv.y;
                    sc[i][2] *= qs1 * kv.x;
                    sc[i][3] *= qs1 * kv.y;
                    if (masked) {
                        const int k = t * RK + tok0 + i * 8 + 2 * cq;
                        const bool b = bad >> (i >> 1) & 1u;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (b || k + (e & 1) > (e < 2 ? pos_a : pos_b)) sc[i][e] = -INFINITY;
                        if (FP8) {  // such a key's scale may be anything, NaN included
                            if (b || k >= pc.keys) lv[i].x = 0.f;
                            if (b || k + 1 >= pc.keys) lv[i].y = 0.f;
                        }
                    }
                    if constexpr (FP8) {
                        // the sums use the same reference as the weighted values: it may lie below the largest
                        // score (rows of tiny scale), but by no more than fp32 holds
                        mx0 = fmaxf(mx0, fmaxf(fmaxf(sc[i][0] + lv[i].x, sc[i][1] + lv[i].y), fmaxf(sc[i][0], sc[i][1]) - 100.f));
                        mx1 = fmaxf(mx1, fmaxf(fmaxf(sc[i][2] + lv[i].x, sc[i][3] + lv[i].y), fmaxf(sc[i][2], sc[i][3]) - 100.f));
                    } else {
                        mx0 = fmaxf(mx0, fmaxf(sc[i][0], sc[i][1]));
                        mx1 = fmaxf(mx1, fmaxf(sc[i][2], sc[i][3]));
                    }
                }
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
                if (__any_sync(0xffffffffu, mx0 > m0 || mx1 > m1)) {
                    const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
                    const float al0 = m0 == -INFINITY ? 0.f : fast_exp2(m0 - mn0), al1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 - mn1);
                    l0 *= al0;
                    l1 *= al1;
#pragma unroll
                    for (int i = 0; i < DT; ++i) {
                        o[i][0] *= al0;
                        o[i][1] *= al0;
                        o[i][2] *= al1;
                        o[i][3] *= al1;
                    }
                    m0 = mn0;
                    m1 = mn1;
                }
                const float mu0 = m0 == -INFINITY ? 0.f : m0, mu1 = m1 == -INFINITY ? 0.f : m1;
                uint32_t pa[2][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x = sc[i][e] - (e < 2 ? mu0 : mu1), y = fast_exp2(x);
                        if (e < 2) l0 += y;
                        else l1 += y;
                        w[e] = FP8 ? fast_exp2(x + ((e & 1) ? lv[i].y : lv[i].x)) : y;
                    }
                    pa[i >> 1][2 * (i & 1)] = FP8 ? pack_f16x2(w[0], w[1]) : pack_bf16x2(w[0], w[1]);
                    pa[i >> 1][2 * (i & 1) + 1] = FP8 ? pack_f16x2(w[2], w[3]) : pack_bf16x2(w[2], w[3]);
                }
                // ---- O += P V; rows behind the last key in use may hold anything: zeros instead ----
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
                    const int vrow = tok0 + j * 16 + rr + ((mi & 1) << 3);
                    if constexpr (FP8) {
#pragma unroll
                        for (int dg = 0; dg < D / 32; ++dg) {
                            // keys 0-7 | 8-15 of 16 columns, and of the next 16
                            const int ch = dg * 2 + (mi >> 1);
                            uint32_t v[4];
                            ldsm_x4_t(smem_u32(vt) + (D == 128 ? swz128(vrow, ch) : swz64(vrow, ch)), v[0], v[1], v[2], v[3]);
                            if (tail) {
                                v[0] &= z0;
                                v[2] &= z0;
                                v[1] &= z1;
                                v[3] &= z1;
                            }
#pragma unroll
                            for (int x = 0; x < 4; ++x) v[x] = __byte_perm(v[x], 0u, 0x3120);  // even columns' pair | odd columns'
                            mma_f16_16816(o[4 * dg], pa[j], codes_to_f16x2(v[0]), codes_to_f16x2(v[1]));
                            mma_f16_16816(o[4 * dg + 1], pa[j], codes_to_f16x2(v[0] >> 16), codes_to_f16x2(v[1] >> 16));
                            mma_f16_16816(o[4 * dg + 2], pa[j], codes_to_f16x2(v[2]), codes_to_f16x2(v[3]));
                            mma_f16_16816(o[4 * dg + 3], pa[j], codes_to_f16x2(v[2] >> 16), codes_to_f16x2(v[3] >> 16));
                        }
                    } else {
#pragma unroll
                        for (int dp = 0; dp < D / 16; ++dp) {
                            const int dim = dp * 16 + ((mi >> 1) << 3);
                            uint32_t v0, v1, v2, v3;
                            ldsm_x4_t(smem_u32(vt) + (dim >> 6) * C::BOX + swz128(vrow, (dim & 63) >> 3), v0, v1, v2, v3);
                            if (tail) {
                                v0 &= z0;
                                v2 &= z0;
                                v1 &= z1;
                                v3 &= z1;
                            }
                            mma_bf16_16816(o[2 * dp], pa[j], v0, v1);
                            mma_bf16_16816(o[2 * dp + 1], pa[j], v2, v3);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
        }

        // ---- join the four warps: each row's common maximum, then sums over scratch memory ----
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
        if (cq == 0) {
            s_ml[warp * 16 + r0] = make_float2(m0, l0);
            s_ml[warp * 16 + r0 + 8] = make_float2(m1, l1);
        }
        named_bar_sync(1, RW * 32);
        float M0 = -INFINITY, M1 = -INFINITY, L0 = 0.f, L1 = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            M0 = fmaxf(M0, s_ml[(mt * 4 + j) * 16 + r0].x);
            M1 = fmaxf(M1, s_ml[(mt * 4 + j) * 16 + r0 + 8].x);
        }
        const float mu0 = M0 == -INFINITY ? 0.f : M0, mu1 = M1 == -INFINITY ? 0.f : M1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 x = s_ml[(mt * 4 + j) * 16 + r0], y = s_ml[(mt * 4 + j) * 16 + r0 + 8];
            L0 += fast_exp2(x.x - mu0) * x.y;
            L1 += fast_exp2(y.x - mu1) * y.y;
        }
        const float w0 = fast_exp2(m0 - mu0), w1 = fast_exp2(m1 - mu1);
#pragma unroll
        for (int i = 0; i < DT; ++i) {
            o[i][0] *= w0;
            o[i][1] *= w0;
            o[i][2] *= w1;
            o[i][3] *= w1;
        }
        // column of o[i][e]: FP8: 16 (i / 2) + 4 cq + 2 (e & 1) + (i & 1); bf16: 8 i + 2 cq + (e & 1)
        auto col = [&](int i, int e) { return FP8 ? (i >> 1) * 16 + 4 * cq + 2 * e + (i & 1) : i * 8 + 2 * cq + e; };
        auto spill = [&](float* so) {
#pragma unroll
            for (int i = 0; i < DT; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    so[r0 * C::SCR + col(i, e)] = o[i][e];
                    so[(r0 + 8) * C::SCR + col(i, e)] = o[i][2 + e];
                }
        };
        auto fill = [&](const float* so) {
#pragma unroll
            for (int i = 0; i < DT; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    o[i][e] += so[r0 * C::SCR + col(i, e)];
                    o[i][2 + e] += so[(r0 + 8) * C::SCR + col(i, e)];
                }
        };
        float* so = s_o + (mt * 2 + (sub & 1)) * 16 * C::SCR;
        if (sub >= 2) spill(so);
        named_bar_sync(1, RW * 32);
        if (sub < 2) fill(so);
        if (sub < 2) spill(so);
        if (sub == 0 && cq == 0) {
            s_ml[warp * 16 + r0] = make_float2(M0, L0);  // (every warp has read the sums)
            s_ml[warp * 16 + r0 + 8] = make_float2(M1, L1);
        }
        named_bar_sync(1, RW * 32);
        // ---- the rows: finished, or a partial ----
        const long long slot = static_cast<long long>(2 * c + (c == pc.first ? 1 : 0)) * RM;
        for (int idx = threadIdx.x; idx < rows * (D / 4); idx += RW * 32) {
            const int r = idx / (D / 4), q4 = idx - r * (D / 4);
            const float* sr = s_o + ((r >> 4) * 32 + (r & 15)) * C::SCR + 4 * q4;
            const float4 x = *reinterpret_cast<const float4*>(sr), y = *reinterpret_cast<const float4*>(sr + 16 * C::SCR);
            const float4 v = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
            const float2 ml = s_ml[(r >> 4) * 64 + (r & 15)];
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
        named_bar_sync(1, RW * 32);
        if (pc.count > 1) split[n_split++ & 1] = pc;  // at most the first and the last unit of the stretch
    }

    // ---- the split units of this CTA: the last piece of a group of 16 joins it, the last group the unit ----
    for (int k = 0; k < n_split; ++k) {
        const RowPiece& s = split[k];
        const int me = c - s.first, grp = me / RGROUP, groups = (s.count + RGROUP - 1) / RGROUP;
        const int i0 = grp * RGROUP, i1 = min(i0 + RGROUP, s.count);
        // counters (zero between calls): a group's, by its first piece's CTA (those behind a unit's first
        // group in a second array, as that CTA may begin another unit), and the unit's
        int* gcnt = a.counters + (grp ? CHUNK_MAX_SLOTS : 0) + s.first + i0;
        int* ucnt = a.counters + 2 * CHUNK_MAX_SLOTS + s.first;
        if (threadIdx.x == 0) {
            int go = 0;
            if (!*s_abort) {
                __threadfence();
                go = atomicAdd(gcnt, 1) == i1 - i0 - 1;
                if (go) {
                    *gcnt = 0;
                    __threadfence();
                }
            }
            *s_join = go;
        }
        named_bar_sync(1, RW * 32);
        bool go = *s_join;
        named_bar_sync(1, RW * 32);
        if (!go) continue;
        join_pieces<D, RM>(a, s.first, i0, i1, 1, s, groups == 1, threadIdx.x, RW * 32);
        if (groups == 1) continue;
        named_bar_sync(1, RW * 32);  // everyone has read the group's (m, l)
        const long long lead = static_cast<long long>(i0 == 0 ? 2 * s.first + 1 : 2 * (s.first + i0)) * RM;
        for (int r = threadIdx.x; r < s.n * a.g; r += RW * 32) __stcg(a.part_ml + lead + r, __ldcg(a.join_ml + lead + r));
        named_bar_sync(1, RW * 32);
        if (threadIdx.x == 0) {
            __threadfence();
            go = atomicAdd(ucnt, 1) == groups - 1;
            if (go) {
                *ucnt = 0;
                __threadfence();
            }
            *s_join = go;
        }
        named_bar_sync(1, RW * 32);
        go = *s_join;
        named_bar_sync(1, RW * 32);
        if (go) join_pieces<D, RM>(a, s.first, 0, s.count, RGROUP, s, true, threadIdx.x, RW * 32);
    }
}

template <int D, bool FP8, int NMT>
cudaError_t launch_typed(const ChunkArgs& a, const CUtensorMap& tm_k, const CUtensorMap& tm_v, int num_sms,
                         cudaStream_t stream)
{
    using C = RCfg<D, FP8, NMT>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !attr_set[dev]) {
        e = cudaFuncSetAttribute(chunk_rows_kernel<D, FP8, NMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        if (dev < 64) attr_set[dev] = true;
    }
    int grid = num_sms * C::CTAS;
    if (grid > CHUNK_MAX_SLOTS) grid = CHUNK_MAX_SLOTS;
    return launch_pdl(chunk_rows_kernel<D, FP8, NMT>, dim3(grid), dim3(C::THREADS), C::SMEM, stream, tm_k, tm_v, a);
}

template <int D, bool FP8>
cudaError_t launch_rows(const ChunkArgs& a, const CUtensorMap& tm_k, const CUtensorMap& tm_v, int num_sms,
                        cudaStream_t stream)
{
    return a.max_q * a.g <= 16 ? launch_typed<D, FP8, 1>(a, tm_k, tm_v, num_sms, stream)
                               : launch_typed<D, FP8, 2>(a, tm_k, tm_v, num_sms, stream);
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

// paged_cache.cu -- writing new tokens into a paged KV cache, in bf16 or
// quantised to E4M3 as they are written, and reading an FP8 cache back.
//
// K of the token at position p is R(p) k ("Agentic RL 入门3" §1.1: the rotation is
// applied to k, never to v); it and v go to row p of the sequence ("注意力机制进化史",
// the cache append).  FP8: one group per row and head, the rule of the latent and
// indexer-key quantisers: s = absmax / 448 and E4M3(x / s), both fp32 divisions,
// taken from the rotated key in fp32 (it is rounded once, to its code).
// Memory-bound, and latency-bound for a decode step's few rows: a row's data is
// requested before its place is known, and the batch's offsets and lengths come in
// one round trip through shared memory.
// Measured (8 heads of 128): 10,612 tokens in bf16 17.1 us = 5.4 TB/s; 15,122 in FP8 27.4 us = 3.6 TB/s,
// bound by latency (100 registers: two blocks on an SM, six waves of them, each with three trips to memory in a
// row; issue slots 46%, DRAM 30% under ncu); 163,508 rows read back 161 us = 6.3 TB/s in a stream of such calls.
#include <type_traits>

#include "paged.cuh"

namespace kvattn {

namespace {

constexpr int AP_THREADS = 256;

__device__ __forceinline__ uint32_t codes_x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// One row's scale (absmax over the CPR lanes holding it) and this lane's E codes, four a word.
// Division by Markstein's method (P. Markstein, IBM J. Res. Dev. 34, 1990): r = RN(1 / s),
// q = RN(x r), and q + r (x - q s) with both products fused, whose error before its rounding is
// under 2^-23 ulp.  It can differ from RN(x / s) only where x / s lies that close to the middle of
// two floats, and the code only where that middle is also next to a border between codes, a
// number of five bits: for which s has to be within 2 ulp of a multiple of 2^-3 of its binade.
// tests/test_paged_quant_rule.py enumerates those: the code is the divided quotient's in all.
template <int CPR, int E>
__device__ __forceinline__ void quantise_row(const float (&x)[E], float& s, uint32_t (&c)[E / 4])
{
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < E; i += 2) a = fmax3(a, fabsf(x[i]), fabsf(x[i + 1]));
#pragma unroll
    for (int o = CPR / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    s = __fdiv_rn(a, 448.f);
    if (s > 0x1p-100f && s < 0x1p100f) {
        const float r = __frcp_rn(s);
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            uint32_t h[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float2 y = make_float2(x[4 * i + 2 * k], x[4 * i + 2 * k + 1]);
                const float2 q = __fmul2_rn(y, make_float2(r, r));
                const float2 e = __ffma2_rn(q, make_float2(-s, -s), y);
                const float2 z = __ffma2_rn(e, make_float2(r, r), q);
                h[k] = codes_x2(z.x, z.y);
            }
            c[i] = h[0] | (h[1] << 16);
        }
    } else {  // a zero row, or a scale whose reciprocal leaves the normal range
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            c[i] = 0u;
            if (s != 0.f)
                c[i] = codes_x2(__fdiv_rn(x[4 * i], s), __fdiv_rn(x[4 * i + 1], s)) |
                       (codes_x2(__fdiv_rn(x[4 * i + 2], s), __fdiv_rn(x[4 * i + 3], s)) << 16);
        }
    }
}

// The elements of N 16-byte pieces.
template <int N>
__device__ __forceinline__ void unpack(const uint4 (&v)[N], float (&x)[8 * N])
{
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[8 * k + 2 * i] = bf16_lo(w[i]);
            x[8 * k + 2 * i + 1] = bf16_hi(w[i]);
        }
    }
}

// CPR = D / E lanes take one token's rows of K and V for HB KV heads, E elements of each row a
// lane: its place and its cos / sin entries are looked up once for all of them, and the
// rows are requested before either is known.
template <int D, int E, int HB, bool FP8>
__global__ void __launch_bounds__(AP_THREADS) paged_append_kernel(PagedAppendArgs a)
{
    constexpr int CPR = D / E, N = E / 8;
    __shared__ int s_cu[PAGED_MAX_B + 1], s_len[PAGED_MAX_B];
    pdl_wait();
    pdl_trigger();
    const PagedBatch& p = a.p;
    const int ch = threadIdx.x % CPR;
    const int groups = (a.Hk + HB - 1) / HB;
    const long long item = static_cast<long long>(blockIdx.x) * (AP_THREADS / CPR) + threadIdx.x / CPR;
    const bool have = item < static_cast<long long>(p.n_tokens) * groups;
    const int t = have ? static_cast<int>(item / groups) : -1;
    const int h0 = have ? static_cast<int>(item - static_cast<long long>(t) * groups) * HB : 0;
    uint4 kx[HB][N], vx[HB][N];
#pragma unroll
    for (int i = 0; i < HB; ++i) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            kx[i][k] = vx[i][k] = make_uint4(0, 0, 0, 0);
            if (have && h0 + i < a.Hk) {
                kx[i][k] = __ldg(reinterpret_cast<const uint4*>(a.k_new + t * a.k_st + (h0 + i) * D) + ch * N + k);
                vx[i][k] = __ldg(reinterpret_cast<const uint4*>(a.v_new + t * a.v_st + (h0 + i) * D) + ch * N + k);
            }
        }
    }
    for (int b = threadIdx.x; b <= p.B; b += AP_THREADS) {
        s_cu[b] = p.cu[b];
        if (b < p.B) s_len[b] = p.seq_lens[b];
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < p.B; b += AP_THREADS)
            if (paged_seq(p, s_cu[b], s_cu[b + 1], s_len[b]).bad) report_status(p.dev_status, KVATTN_STATUS_BAD_LENGTH);
    // the sequence of token t: the last b with cu[b] <= t
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_cu[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    const PagedSeq s = paged_seq(p, s_cu[lo], s_cu[lo + 1], s_len[lo]);
    const bool mine = have && t >= s.t0 && t < s.t0 + s.n;  // not a token behind the last sequence
    const int pos = s.len - s.n + (t - s.t0);
    bool go = mine && pos >= 0 && pos < a.max_pos;
    if (mine && !go && ch == 0) report_status(p.dev_status, KVATTN_STATUS_BAD_POSITION);
    int page = 0;
    if (go) page = p.page_table[static_cast<long long>(lo) * p.max_pages + (pos >> p.page_shift)];
    // cos and sin of this lane's elements: its E / 2 pairs (2i, 2i + 1), or the E of its half
    float cc[E], ss[E];
    const bool first = ch < CPR / 2;  // half-split pairs: the lower half
    {
        const long long cs = static_cast<long long>(go ? pos : 0) * (D / 2) +
                             (a.pair_style == 0 ? ch * (E / 2) : (first ? ch : ch - CPR / 2) * E);
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            float4 c = make_float4(0.f, 0.f, 0.f, 0.f), n = c;
            if (i < E / 2 || a.pair_style != 0) {
                c = *reinterpret_cast<const float4*>(a.cos_tab + cs + i);
                n = *reinterpret_cast<const float4*>(a.sin_tab + cs + i);
            }
            cc[i] = c.x, cc[i + 1] = c.y, cc[i + 2] = c.z, cc[i + 3] = c.w;
            ss[i] = n.x, ss[i + 1] = n.y, ss[i + 2] = n.z, ss[i + 3] = n.w;
        }
    }
    if (go && (page < 0 || page >= p.n_pages)) {
        go = false;
        if (ch == 0) report_status(p.dev_status, KVATTN_STATUS_BAD_INDEX);
    }
#pragma unroll
    for (int j = 0; j < HB; ++j) {
        float kf[E], x[E];
        unpack(kx[j], x);
        if (a.pair_style == 0) {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                const float2 y = rope_pair(x[2 * i], x[2 * i + 1], cc[i], ss[i]);
                kf[2 * i] = y.x;
                kf[2 * i + 1] = y.y;
            }
        } else {
            // this lane's elements pair with those of the lane d/2 further on (or back)
            uint4 o[N];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                o[k].x = __shfl_xor_sync(0xffffffffu, kx[j][k].x, CPR / 2);
                o[k].y = __shfl_xor_sync(0xffffffffu, kx[j][k].y, CPR / 2);
                o[k].z = __shfl_xor_sync(0xffffffffu, kx[j][k].z, CPR / 2);
                o[k].w = __shfl_xor_sync(0xffffffffu, kx[j][k].w, CPR / 2);
            }
            float y[E];
            unpack(o, y);
#pragma unroll
            for (int i = 0; i < E; ++i)
                kf[i] = first ? rope_pair(x[i], y[i], cc[i], ss[i]).x : rope_pair(y[i], x[i], cc[i], ss[i]).y;
        }
        const bool put = go && h0 + j < a.Hk;
        const long long dst =
            ((static_cast<long long>(page) * a.Hk + h0 + j) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
        if constexpr (FP8) {
            using Codes = typename std::conditional<E == 16, uint4, uint2>::type;
            float vf[E], ks, vs;
            union {
                uint32_t w[E / 4];
                Codes v;
            } kc, vc;
            unpack(vx[j], vf);
            quantise_row<CPR>(kf, ks, kc.w);
            quantise_row<CPR>(vf, vs, vc.w);
            if (put) {
                reinterpret_cast<Codes*>(static_cast<uint8_t*>(a.k_pages) + dst * D)[ch] = kc.v;
                reinterpret_cast<Codes*>(static_cast<uint8_t*>(a.v_pages) + dst * D)[ch] = vc.v;
                if (ch == 0) {
                    a.k_scales[dst] = ks;
                    a.v_scales[dst] = vs;
                }
            }
        } else if (put) {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                reinterpret_cast<uint4*>(static_cast<kvattn_bf16*>(a.k_pages) + dst * D)[ch * N + k] =
                    make_uint4(pack_bf16x2(kf[8 * k], kf[8 * k + 1]), pack_bf16x2(kf[8 * k + 2], kf[8 * k + 3]),
                               pack_bf16x2(kf[8 * k + 4], kf[8 * k + 5]), pack_bf16x2(kf[8 * k + 6], kf[8 * k + 7]));
                reinterpret_cast<uint4*>(static_cast<kvattn_bf16*>(a.v_pages) + dst * D)[ch * N + k] = vx[j][k];
            }
        }
    }
}

// ---- FP8 pages -> contiguous bf16 rows ----------------------------------------------
// bf16(code * scale), one rounding.  D / 8 lanes per row, eight codes (an 8-byte load, a
// 16-byte store) each, so that a warp's stores are whole runs of 512 bytes; a thread takes
// RD_ROWS rows of K and V, all requested before the first is written.  Both streams pass
// once: they are marked so.  163,508 rows (8 x 128), 1.02 GB: 171 us as timed here (sixteen
// codes a lane, one row: 200; one row of eight: 190; two rows without the marks: 172).
constexpr int RD_THREADS = 256;
constexpr int RD_ROWS = 2;

template <int D>
__global__ void __launch_bounds__(RD_THREADS) paged_read_kernel(PagedReadArgs a)
{
    constexpr int LPR = D / 8;
    constexpr int RPB = RD_THREADS / LPR;  // rows per pass of a block
    pdl_wait();
    pdl_trigger();
    const PagedBatch& p = a.p;
    const int b = blockIdx.y / a.Hk, h = blockIdx.y - b * a.Hk;
    const int raw = p.seq_lens[b];
    const int len = min(max(raw, 0), min(a.T_max, p.max_pages << p.page_shift));
    if (raw != len && blockIdx.x == 0 && threadIdx.x == 0) report_status(p.dev_status, KVATTN_STATUS_BAD_LENGTH);
    const int r0 = blockIdx.x * (RPB * RD_ROWS) + threadIdx.x / LPR, ln = threadIdx.x % LPR;
    uint2 kc[RD_ROWS], vc[RD_ROWS];
    float ks[RD_ROWS], vs[RD_ROWS];
    bool have[RD_ROWS];
#pragma unroll
    for (int i = 0; i < RD_ROWS; ++i) {
        const int r = r0 + i * RPB;
        have[i] = r < len;
        if (!have[i]) continue;
        const int page = p.page_table[static_cast<long long>(b) * p.max_pages + (r >> p.page_shift)];
        if (page < 0 || page >= p.n_pages) {
            if (ln == 0) report_status(p.dev_status, KVATTN_STATUS_BAD_INDEX);
            have[i] = false;
            continue;
        }
        const long long src = ((static_cast<long long>(page) * a.Hk + h) << p.page_shift) + (r & ((1 << p.page_shift) - 1));
        kc[i] = __ldcs(reinterpret_cast<const uint2*>(a.k_codes + src * D) + ln);
        vc[i] = __ldcs(reinterpret_cast<const uint2*>(a.v_codes + src * D) + ln);
        ks[i] = __ldg(a.k_scales + src);
        vs[i] = __ldg(a.v_scales + src);
    }
#pragma unroll
    for (int i = 0; i < RD_ROWS; ++i) {
        if (!have[i]) continue;
        const long long dst = (static_cast<long long>(blockIdx.y) * a.T_max + r0 + i * RPB) * D + ln * 8;
        auto put = [&](kvattn_bf16* out, uint2 c, float s) {
            auto two = [s](uint32_t codes) {
                const float2 x = e4m3x2_to_f32(static_cast<uint16_t>(codes));
                return pack_bf16x2(x.x * s, x.y * s);
            };
            __stcs(reinterpret_cast<uint4*>(out + dst), make_uint4(two(c.x), two(c.x >> 16), two(c.y), two(c.y >> 16)));
        };
        put(a.k_out, kc[i], ks[i]);
        put(a.v_out, vc[i], vs[i]);
    }
}

}  // namespace

template <int E, int HB, bool FP8>
cudaError_t launch_append(const PagedAppendArgs& a, cudaStream_t stream)
{
    const int per_block = AP_THREADS / (a.d / E);
    const long long blocks = (static_cast<long long>(a.p.n_tokens) * ((a.Hk + HB - 1) / HB) + per_block - 1) / per_block;
    return launch_pdl(a.d == 128 ? paged_append_kernel<128, E, HB, FP8> : paged_append_kernel<64, E, HB, FP8>,
                      dim3(static_cast<unsigned>(blocks)), dim3(AP_THREADS), 0, stream, a);
}

cudaError_t launch_paged_append(const PagedAppendArgs& a, bool fp8, int num_sms, cudaStream_t stream)
{
    // Few rows: one row a lane group, for the shortest chain of one.  From the rows whose lanes take three eighths of
    // the card's thread slots on, several heads a group; in FP8 16 elements a lane, which halves the work per row (its
    // scale, the shuffles).  One / several, 8 heads of 128: 512 tokens 2.3 / 2.7 us (FP8 2.8 / 3.6), 1024 3.1 / 2.7
    // (4.0 / 3.6), 4096 6.8 / 5.9 (9.1 / 7.7); a single head 16384 4.4 / 6.2 (5.5 / 7.5).
    const bool few = static_cast<long long>(a.p.n_tokens) * a.Hk * (a.d / 8) < num_sms * 768ll || a.Hk < 2;
    if (fp8) return few ? launch_append<8, 1, true>(a, stream) : launch_append<16, 2, true>(a, stream);
    return few ? launch_append<8, 1, false>(a, stream) : launch_append<8, 4, false>(a, stream);
}

cudaError_t launch_paged_read(const PagedReadArgs& a, cudaStream_t stream)
{
    const int rows = RD_THREADS / (a.d / 8) * RD_ROWS;
    const int cap = a.p.max_pages << a.p.page_shift;
    const int most = a.T_max < cap ? a.T_max : cap;  // no row beyond both is read
    const dim3 grid((most + rows - 1) / rows, a.p.B * a.Hk);
    return launch_pdl(a.d == 128 ? paged_read_kernel<128> : paged_read_kernel<64>, grid, dim3(RD_THREADS), 0, stream, a);
}

}  // namespace kvattn

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

// One row's scale (absmax over the CPR lanes holding it) and this lane's eight codes.
template <int CPR>
__device__ __forceinline__ uint2 quantise_row(const float (&x)[8], float& s)
{
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(x[i]));
#pragma unroll
    for (int o = CPR / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    s = __fdiv_rn(a, 448.f);
    if (s == 0.f) return make_uint2(0u, 0u);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = codes_x2(__fdiv_rn(x[2 * i], s), __fdiv_rn(x[2 * i + 1], s));
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}

// CPR = d / 8 lanes hold one (token, head) row of K and the same row of V, eight
// elements each.
template <int CPR, bool FP8>
__global__ void __launch_bounds__(AP_THREADS) paged_append_kernel(PagedAppendArgs a)
{
    constexpr int D = CPR * 8;
    __shared__ int s_cu[PAGED_MAX_B + 1], s_len[PAGED_MAX_B];
    pdl_wait();
    pdl_trigger();
    const PagedBatch& p = a.p;
    const int ch = threadIdx.x % CPR;
    const long long rows = static_cast<long long>(p.n_tokens) * a.Hk;
    const long long step = static_cast<long long>(gridDim.x) * (AP_THREADS / CPR);
    long long row = static_cast<long long>(blockIdx.x) * (AP_THREADS / CPR) + threadIdx.x / CPR;
    uint4 kx = make_uint4(0, 0, 0, 0), vx = kx;
    auto fetch = [&](long long r) {
        const int t = static_cast<int>(r / a.Hk), h = static_cast<int>(r - static_cast<long long>(t) * a.Hk);
        kx = __ldg(reinterpret_cast<const uint4*>(a.k_new + t * a.k_st + h * D) + ch);
        vx = __ldg(reinterpret_cast<const uint4*>(a.v_new + t * a.v_st + h * D) + ch);
    };
    if (row < rows) fetch(row);
    for (int b = threadIdx.x; b <= p.B; b += AP_THREADS) {
        s_cu[b] = p.cu[b];
        if (b < p.B) s_len[b] = p.seq_lens[b];
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < p.B; b += AP_THREADS)
            if (paged_seq(p, s_cu[b], s_cu[b + 1], s_len[b]).bad) report_status(p.dev_status, KVATTN_STATUS_BAD_LENGTH);
    // every lane of a warp takes the same number of turns, for the shuffles
    for (long long r0 = row - threadIdx.x % 32 / CPR; r0 < rows; r0 += step, row += step) {
        const uint4 kr = kx, vr = vx;
        if (row + step < rows) fetch(row + step);
        const bool have = row < rows;
        const int t = have ? static_cast<int>(row / a.Hk) : -1;
        const int h = have ? static_cast<int>(row - static_cast<long long>(t) * a.Hk) : 0;
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
        if (go) {
            page = p.page_table[static_cast<long long>(lo) * p.max_pages + (pos >> p.page_shift)];
            if (page < 0 || page >= p.n_pages) {
                go = false;
                if (ch == 0) report_status(p.dev_status, KVATTN_STATUS_BAD_INDEX);
            }
        }
        float kf[8];
        {
            const long long cs = static_cast<long long>(go ? pos : 0) * (D / 2);
            float x[8];
            unpack8(kr, x);
            if (a.pair_style == 0) {
                const float4 c = *reinterpret_cast<const float4*>(a.cos_tab + cs + ch * 4);
                const float4 n = *reinterpret_cast<const float4*>(a.sin_tab + cs + ch * 4);
                const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 y = rope_pair(x[2 * i], x[2 * i + 1], cc[i], ss[i]);
                    kf[2 * i] = y.x;
                    kf[2 * i + 1] = y.y;
                }
            } else {
                // this lane's eight elements pair with those of the lane d/2 further on (or back)
                uint4 o;
                o.x = __shfl_xor_sync(0xffffffffu, kr.x, CPR / 2);
                o.y = __shfl_xor_sync(0xffffffffu, kr.y, CPR / 2);
                o.z = __shfl_xor_sync(0xffffffffu, kr.z, CPR / 2);
                o.w = __shfl_xor_sync(0xffffffffu, kr.w, CPR / 2);
                float y[8];
                unpack8(o, y);
                const bool first = ch < CPR / 2;
                const int ci = (first ? ch : ch - CPR / 2) * 8;
                const float4 c0 = *reinterpret_cast<const float4*>(a.cos_tab + cs + ci);
                const float4 c1 = *reinterpret_cast<const float4*>(a.cos_tab + cs + ci + 4);
                const float4 n0 = *reinterpret_cast<const float4*>(a.sin_tab + cs + ci);
                const float4 n1 = *reinterpret_cast<const float4*>(a.sin_tab + cs + ci + 4);
                const float cc[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
                const float ss[8] = {n0.x, n0.y, n0.z, n0.w, n1.x, n1.y, n1.z, n1.w};
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    kf[i] = first ? rope_pair(x[i], y[i], cc[i], ss[i]).x : rope_pair(y[i], x[i], cc[i], ss[i]).y;
            }
        }
        const long long dst = ((static_cast<long long>(page) * a.Hk + h) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
        if constexpr (FP8) {
            float vf[8], ks, vs;
            unpack8(vr, vf);
            const uint2 kc = quantise_row<CPR>(kf, ks), vc = quantise_row<CPR>(vf, vs);
            if (go) {
                reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.k_pages) + dst * D)[ch] = kc;
                reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v_pages) + dst * D)[ch] = vc;
                if (ch == 0) {
                    a.k_scales[dst] = ks;
                    a.v_scales[dst] = vs;
                }
            }
        } else if (go) {
            reinterpret_cast<uint4*>(static_cast<kvattn_bf16*>(a.k_pages) + dst * D)[ch] =
                make_uint4(pack_bf16x2(kf[0], kf[1]), pack_bf16x2(kf[2], kf[3]), pack_bf16x2(kf[4], kf[5]),
                           pack_bf16x2(kf[6], kf[7]));
            reinterpret_cast<uint4*>(static_cast<kvattn_bf16*>(a.v_pages) + dst * D)[ch] = vr;
        }
    }
}

// ---- FP8 pages -> contiguous bf16 rows ----------------------------------------------
// bf16(code * scale), one rounding.  D / 16 lanes per row, sixteen codes (one 16-byte
// load, two 16-byte stores) each; a block takes RD_ROWS consecutive rows of one (batch,
// KV head), K and V, so that their loads are all in flight together.
constexpr int RD_THREADS = 256;

template <int D>
__global__ void __launch_bounds__(RD_THREADS) paged_read_kernel(PagedReadArgs a)
{
    constexpr int LPR = D / 16;
    constexpr int RPB = RD_THREADS / LPR;  // rows per block
    pdl_wait();
    pdl_trigger();
    const PagedBatch& p = a.p;
    const int b = blockIdx.y / a.Hk, h = blockIdx.y - b * a.Hk;
    const int raw = p.seq_lens[b];
    const int len = min(max(raw, 0), min(a.T_max, p.max_pages << p.page_shift));
    if (raw != len && blockIdx.x == 0 && threadIdx.x == 0) report_status(p.dev_status, KVATTN_STATUS_BAD_LENGTH);
    const int r = blockIdx.x * RPB + threadIdx.x / LPR, ln = threadIdx.x % LPR;
    if (r >= len) return;
    const int page = p.page_table[static_cast<long long>(b) * p.max_pages + (r >> p.page_shift)];
    if (page < 0 || page >= p.n_pages) {
        if (ln == 0) report_status(p.dev_status, KVATTN_STATUS_BAD_INDEX);
        return;
    }
    const long long src = ((static_cast<long long>(page) * a.Hk + h) << p.page_shift) + (r & ((1 << p.page_shift) - 1));
    const uint4 kc = __ldg(reinterpret_cast<const uint4*>(a.k_codes + src * D) + ln);
    const uint4 vc = __ldg(reinterpret_cast<const uint4*>(a.v_codes + src * D) + ln);
    const float ks = __ldg(a.k_scales + src), vs = __ldg(a.v_scales + src);
    const long long dst = (static_cast<long long>(blockIdx.y) * a.T_max + r) * D + ln * 16;
    auto put = [&](kvattn_bf16* out, uint4 c, float s) {
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = e4m3x2_to_f32(static_cast<uint16_t>(w[i])), y = e4m3x2_to_f32(static_cast<uint16_t>(w[i] >> 16));
            o[2 * i] = pack_bf16x2(x.x * s, x.y * s);
            o[2 * i + 1] = pack_bf16x2(y.x * s, y.y * s);
        }
        uint4* d = reinterpret_cast<uint4*>(out + dst);
        d[0] = make_uint4(o[0], o[1], o[2], o[3]);
        d[1] = make_uint4(o[4], o[5], o[6], o[7]);
    };
    put(a.k_out, kc, ks);
    put(a.v_out, vc, vs);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, bool fp8, int num_sms, cudaStream_t stream)
{
    const int per_block = AP_THREADS / (a.d / 8);
    long long blocks = (static_cast<long long>(a.p.n_tokens) * a.Hk + per_block - 1) / per_block;
    if (blocks > num_sms * 8ll) blocks = num_sms * 8ll;  // 8 x 256 threads resident per SM
    if (blocks < 1) blocks = 1;                          // the lengths are still checked
    auto kern = a.d == 128 ? (fp8 ? paged_append_kernel<16, true> : paged_append_kernel<16, false>)
                           : (fp8 ? paged_append_kernel<8, true> : paged_append_kernel<8, false>);
    return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(AP_THREADS), 0, stream, a);
}

cudaError_t launch_paged_read(const PagedReadArgs& a, cudaStream_t stream)
{
    const int rows = RD_THREADS / (a.d / 16);
    const int cap = a.p.max_pages << a.p.page_shift;
    const int most = a.T_max < cap ? a.T_max : cap;  // no row beyond both is read
    const dim3 grid((most + rows - 1) / rows, a.p.B * a.Hk);
    return launch_pdl(a.d == 128 ? paged_read_kernel<128> : paged_read_kernel<64>, grid, dim3(RD_THREADS), 0, stream, a);
}

}  // namespace kvattn

// chunk.cu -- attention of a chunk of new tokens over a paged KV cache.
//
// Method: out = softmax_{j <= p} (scale q . k_j) v_j for the query at position p,
// query head h reading KV head h / g ("注意力变体与 MoE", GQA attention(); "attention",
// GroupQueryAttention), the keys and values being rows 0 .. p of the query's
// sequence.  FP8 rows stand for code * scale: the key's scale multiplies the score,
// the value's the weight.  One pass with a running maximum and sum in fp32.
//
// One warp per (token, head); the lanes split the head width.
#include "paged.cuh"

namespace kvattn {

namespace {

constexpr int CH_WARPS = 8;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

template <int D, bool FP8>
__global__ void __launch_bounds__(CH_WARPS * 32) chunk_kernel(ChunkArgs a)
{
    constexpr int PL = D / 32;  // dims per lane
    __shared__ int s_cu[PAGED_MAX_B + 1], s_len[PAGED_MAX_B];
    pdl_wait();
    pdl_trigger();
    const PagedBatch& p = a.p;
    for (int b = threadIdx.x; b <= p.B; b += blockDim.x) {
        s_cu[b] = p.cu[b];
        if (b < p.B) s_len[b] = p.seq_lens[b];
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
            const PagedSeq s = paged_seq(p, s_cu[b], s_cu[b + 1], s_len[b]);
            if (s.bad || s.n > a.max_q) report_status(p.dev_status, KVATTN_STATUS_BAD_LENGTH);
        }
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * CH_WARPS + (threadIdx.x >> 5);
    if (row >= static_cast<long long>(p.n_tokens) * a.H) return;
    const int t = static_cast<int>(row / a.H), h = static_cast<int>(row - static_cast<long long>(t) * a.H);
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_cu[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    const PagedSeq s = paged_seq(p, s_cu[lo], s_cu[lo + 1], s_len[lo]);
    if (t < s.t0 || t >= s.t0 + min(s.n, a.max_q)) return;
    const int pos = s.len - s.n + (t - s.t0);
    const int kvh = h / a.g;
    float q[PL], o[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) {
        q[i] = bf16_lo(a.q[t * a.q_st + h * D + lane * PL + i]);
        o[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j <= pos; ++j) {
        const int page = p.page_table[static_cast<long long>(lo) * p.max_pages + (j >> p.page_shift)];
        if (page < 0 || page >= p.n_pages) {
            if (lane == 0) report_status(p.dev_status, KVATTN_STATUS_BAD_INDEX);
            continue;
        }
        const long long r = ((static_cast<long long>(page) * a.Hk + kvh) << p.page_shift) + (j & ((1 << p.page_shift) - 1));
        float k[PL], v[PL], ks = 1.f, vs = 1.f;
        if constexpr (FP8) {
            const uint8_t* kp = static_cast<const uint8_t*>(a.k_pages) + r * D + lane * PL;
            const uint8_t* vp = static_cast<const uint8_t*>(a.v_pages) + r * D + lane * PL;
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                k[i] = e4m3x2_to_f32(kp[i]).x;
                v[i] = e4m3x2_to_f32(vp[i]).x;
            }
            ks = a.k_scales[r];
            vs = a.v_scales[r];
        } else {
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                k[i] = bf16_lo(static_cast<const kvattn_bf16*>(a.k_pages)[r * D + lane * PL + i]);
                v[i] = bf16_lo(static_cast<const kvattn_bf16*>(a.v_pages)[r * D + lane * PL + i]);
            }
        }
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < PL; ++i) x += q[i] * k[i];
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
        x *= ks * a.scale * kLog2e;
        const float mn = fmaxf(m, x);
        const float al = exp2f(m - mn), e = exp2f(x - mn);
        m = mn;
        l = l * al + e;
#pragma unroll
        for (int i = 0; i < PL; ++i) o[i] = o[i] * al + e * vs * v[i];
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int i = 0; i < PL; ++i)
        reinterpret_cast<__nv_bfloat16*>(a.out)[row * D + lane * PL + i] = __float2bfloat16_rn(o[i] * inv);
    if (a.lse && lane == 0) a.lse[row] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace

cudaError_t launch_chunk(const ChunkArgs& a, bool fp8, int num_sms, cudaStream_t stream)
{
    (void)num_sms;
    const long long blocks = (static_cast<long long>(a.p.n_tokens) * a.H + CH_WARPS - 1) / CH_WARPS;
    auto kern = a.d == 128 ? (fp8 ? chunk_kernel<128, true> : chunk_kernel<128, false>)
                           : (fp8 ? chunk_kernel<64, true> : chunk_kernel<64, false>);
    return launch_pdl(kern, dim3(static_cast<unsigned>(blocks > 0 ? blocks : 1)), dim3(CH_WARPS * 32), 0, stream, a);
}

}  // namespace kvattn

// paged.cuh -- ragged batches of new tokens over a paged KV cache: the launch
// arguments and the device helpers that the paged kernels share.
//
// A batch of B sequences brings n_tokens packed new tokens: sequence b's are
// tokens cu[b] .. cu[b+1]-1, and seq_lens[b] counts its cached rows with them,
// so its token i stands at position seq_lens[b] - n_b + i.  Row r of a sequence
// is row r % page_size of the page page_table[b][r / page_size]; a page holds
// page_size rows of every KV head, [n_pages][Hk][page_size][d].  Everything that
// only the device can see is range-checked here before it becomes an address.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace kvattn {

constexpr int PAGED_MAX_B = 1024;

struct PagedBatch {
    const int32_t* cu;          // [B + 1]
    const int32_t* seq_lens;    // [B]
    const int32_t* page_table;  // [B][max_pages]
    int B, n_tokens, max_pages, n_pages, page_shift;
    int32_t* dev_status;
};

struct PagedAppendArgs {
    PagedBatch p;
    const kvattn_bf16* k_new;  // token t, head h at k_new + t * k_st + h * d
    const kvattn_bf16* v_new;
    long long k_st, v_st;
    void* k_pages;  // bf16 rows, or E4M3 codes
    void* v_pages;
    float* k_scales;  // [n_pages][Hk][page_size], FP8 only
    float* v_scales;
    const float* cos_tab;
    const float* sin_tab;
    int Hk, d, max_pos, pair_style;
};
cudaError_t launch_paged_append(const PagedAppendArgs& a, bool fp8, int num_sms, cudaStream_t stream);

struct PagedReadArgs {
    PagedBatch p;  // cu unused
    const uint8_t* k_codes;
    const uint8_t* v_codes;
    const float* k_scales;
    const float* v_scales;
    kvattn_bf16* k_out;  // [B][Hk][T_max][d]
    kvattn_bf16* v_out;
    int Hk, d, T_max;
};
cudaError_t launch_paged_read(const PagedReadArgs& a, cudaStream_t stream);

struct ChunkArgs {
    PagedBatch p;
    const kvattn_bf16* q;  // token t, head h at q + t * q_st + h * d
    long long q_st;
    const void* k_pages;  // bf16 rows, or E4M3 codes
    const void* v_pages;
    const float* k_scales;  // [n_pages][Hk][page_size], FP8 only
    const float* v_scales;
    kvattn_bf16* out;  // [n_tokens][H][d]
    float* lse;        // [n_tokens][H] or null
    int H, Hk, g, d, max_q;
    float scale;
    // partials of units that several CTAs share: two slots of rows per CTA
    float2* part_ml;  // (maximum in log2 units, sum)
    float* part_o;    // unnormalised
    int4* split_info;  // tile kernel: split blocks, by the CTA of their first key tile (first token, rows, KV head, pieces)
    float2* join_ml;   // row kernel: (maximum, sum) of joined groups of partials
    int* counters;     // row kernel: pieces that have finished (zero between calls)
};
constexpr int CHUNK_MAX_CTAS = 148;     // tile kernel: at most this many CTAs, with slots of 256 rows
constexpr int CHUNK_SLOT_ROWS = 256;
constexpr int CHUNK_FEW_ROWS = 32;      // row kernel: query rows of a (sequence, KV head), and of a slot, at most
constexpr int CHUNK_MAX_SLOTS = 296;    // row kernel: at most this many CTAs
static_assert(3 * CHUNK_MAX_SLOTS * 4 <= KVATTN_DECODE_WS_ZERO_BYTES, "counters");
cudaError_t launch_chunk_rows(const ChunkArgs& a, bool fp8, const CUtensorMap& tm_k, const CUtensorMap& tm_v, int num_sms,
                              cudaStream_t stream);
cudaError_t launch_chunk_tile(const ChunkArgs& a, bool fp8, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                              const CUtensorMap& tm_v, int num_sms, cudaStream_t stream);

// A sequence's share of the packed tokens and its length, forced into range.
struct PagedSeq {
    int t0, n, len;
    bool bad;  // something was out of range
};

__host__ __device__ __forceinline__ PagedSeq paged_seq(const PagedBatch& p, int c0, int c1, int len_raw)
{
    PagedSeq s;
    s.t0 = min(max(c0, 0), p.n_tokens);
    const int t1 = min(max(c1, s.t0), p.n_tokens);
    s.n = t1 - s.t0;
    s.len = min(max(len_raw, 0), p.max_pages << p.page_shift);
    s.bad = s.t0 != c0 || t1 != c1 || s.len != len_raw;
    return s;
}

// FP8: a row's running reference is the maximum of s + max(log2 vs, this): a tiny or zero value row does not
// lower it further, so that its weight without vs, up to 2^96 of the reference, and sums of those fit fp32.
constexpr float CHUNK_MIN_LOG2_VS = -96.f;

// l 2^x for a sum l of weights that may be that large, and x that far below 0: 2^x alone may underflow.
__device__ __forceinline__ float sum_exp2(float l, float x)
{
    const float h = fast_exp2(0.5f * x);
    return l * h * h;
}

// E4M3 codes -> fp32, two at a time (every code is exact in fp16 and fp32).
__device__ __forceinline__ float2 e4m3x2_to_f32(uint16_t codes)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
    float2 r;
    asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(h));
    return r;
}

}  // namespace kvattn

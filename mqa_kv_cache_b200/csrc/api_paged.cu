// api_paged.cu -- the extern "C" boundary of the paged-cache operators: argument
// checks on the host (nothing is launched after a failed one), then the launch.
#include <cudaTypedefs.h>

#include <cmath>
#include <mutex>

#include "paged.cuh"

namespace {

using kvattn::record_error;

template <typename... P>
bool any_null(P... p)
{
    return ((p == nullptr) || ...);
}

template <typename... P>
bool all_aligned(unsigned to, P... p)
{
    return (((reinterpret_cast<uintptr_t>(p) & (to - 1u)) == 0) && ...);
}

int ok() { return record_error(KVATTN_OK, "%s", ""); }

int finish(cudaError_t e, const char* name)
{
    if (e != cudaSuccess) return record_error(KVATTN_ERR_CUDA, "%s launch: %s", name, cudaGetErrorString(e));
    return ok();
}

int sms_of_device(const char* name, int* sms)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return record_error(KVATTN_ERR_CUDA, "%s: no CUDA device", name);
    return KVATTN_OK;
}

// The sizes of a batch and its pages, common to every call.
int check_batch(const char* name, int B, int n_tokens, int heads, int n_kv_head, int head_dim, int page_size,
                int max_pages, int n_pages)
{
    if (B < 1 || B > kvattn::PAGED_MAX_B)
        return record_error(KVATTN_ERR_SHAPE, "%s: B %d outside 1..%d", name, B, kvattn::PAGED_MAX_B);
    if (n_tokens < 0) return record_error(KVATTN_ERR_SHAPE, "%s: n_tokens %d < 0", name, n_tokens);
    if (heads < 1 || n_kv_head < 1 || heads % n_kv_head)
        return record_error(KVATTN_ERR_SHAPE, "%s: n_head %d not a multiple of n_kv_head %d", name, heads, n_kv_head);
    if (head_dim != 64 && head_dim != 128) return record_error(KVATTN_ERR_UNSUPPORTED, "%s: head_dim %d", name, head_dim);
    if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)))
        return record_error(KVATTN_ERR_UNSUPPORTED, "%s: page_size %d is not a power of two in 16..1024", name, page_size);
    if (max_pages < 1 || static_cast<long long>(max_pages) * page_size > (1ll << 30))
        return record_error(KVATTN_ERR_SHAPE, "%s: max_pages %d (at most 2^30 rows a sequence)", name, max_pages);
    if (n_pages < 1 || static_cast<long long>(n_pages) * n_kv_head >= (1ll << 31))
        return record_error(KVATTN_ERR_SHAPE, "%s: n_pages %d", name, n_pages);
    if (static_cast<long long>(n_tokens) * heads >= (1ll << 31))
        return record_error(KVATTN_ERR_SHAPE, "%s: n_tokens %d x %d heads too large", name, n_tokens, heads);
    if (static_cast<long long>(B) * n_kv_head > KVATTN_DECODE_WS_ZERO_BYTES / 4)
        return record_error(KVATTN_ERR_UNSUPPORTED, "%s: B * n_kv_head = %lld above %u", name,
                            static_cast<long long>(B) * n_kv_head, KVATTN_DECODE_WS_ZERO_BYTES / 4);
    return KVATTN_OK;
}

int check_stride(const char* name, const char* what, int64_t stride, int heads, int head_dim)
{
    if (stride % 8) return record_error(KVATTN_ERR_ALIGN, "%s: %s stride must be a multiple of 8", name, what);
    if (stride < static_cast<int64_t>(heads) * head_dim || stride > (int64_t(1) << 32))
        return record_error(KVATTN_ERR_SHAPE, "%s: %s stride %lld below heads * head_dim (or above 2^32)", name, what,
                            static_cast<long long>(stride));
    return KVATTN_OK;
}

kvattn::PagedBatch batch(const int32_t* cu, const int32_t* seq_lens, const int32_t* page_table, int B, int n_tokens,
                         int page_size, int max_pages, int n_pages, int32_t* dev_status)
{
    kvattn::PagedBatch p{};
    p.cu = cu;
    p.seq_lens = seq_lens;
    p.page_table = page_table;
    p.B = B;
    p.n_tokens = n_tokens;
    p.max_pages = max_pages;
    p.n_pages = n_pages;
    while ((1 << p.page_shift) < page_size) ++p.page_shift;
    p.dev_status = dev_status;
    return p;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no libcuda link).
PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// Map of [z][y][x] with byte strides, boxes 128 bytes wide (64 bf16, 128-byte swizzle) or, over
// bytes, `byte_box_x` wide; the swizzle is given for bytes.  What lies outside reads as zero.
int encode_map(const char* name, CUtensorMap* map, const void* base, uint32_t byte_box_x, uint64_t x, uint64_t y,
               uint64_t z, uint64_t y_stride, uint64_t z_stride, uint32_t box_y, uint32_t box_z,
               CUtensorMapSwizzle byte_swizzle = CU_TENSOR_MAP_SWIZZLE_NONE)
{
    auto fn = encode_fn();
    if (!fn) return record_error(KVATTN_ERR_CUDA, "%s: cuTensorMapEncodeTiled is unavailable", name);
    const bool bytes = byte_box_x > 0;
    const cuuint64_t dims[3] = {x, y, z}, strides[2] = {y_stride, z_stride};
    const cuuint32_t box[3] = {bytes ? byte_box_x : 64u, box_y, box_z}, one[3] = {1, 1, 1};
    const CUresult r = fn(map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                          const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          bytes ? byte_swizzle : CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return record_error(KVATTN_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed (%d)", name, static_cast<int>(r));
    return KVATTN_OK;
}

constexpr size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

// Whether a call whose (sequence, KV head)s have up to max_q * g query rows goes to the row kernel: up to 8; 16 where
// the units, sequences times KV heads, are not shared by many CTAs each (as the last one of those joins a unit's rows);
// 32 where all the cached rows that it has room for are few, `units` times `room` of them.
// Row / tile kernel, d = 128: 9 query rows of 16 sequences over 300, 4000 and 32000 rows (16 KV heads) 22 / 23, 86 / 91,
// 626 / 606 us, FP8 23 / 28, 71 / 93, 416 / 575; 32 of 16 (8 KV heads) over 300, 4000 and 16000 27 / 17, 68 / 53,
// 192 / 167, FP8 30 / 21, 75 / 61, 217 / 182; 20 of 2 (8 KV heads) over 20, 100 and 250 8.3 / 13.0, 13.2 / 13.8,
// 13.8 / 12.9, FP8 9.3 / 15.8, 14.3 / 16.8, 14.8 / 14.8.  d = 64: 20 of 8 (2 KV heads) over 250, 500 and 1000
// 11.0 / 12.2, 11.4 / 11.9, 14.6 / 12.7, FP8 11.6 / 14.2, 12.1 / 13.9, 16.0 / 14.6.  16 query rows of 2 (4 KV heads) over
// 300, 1000 and 4000, d = 128: 12.4 / 12.8, 14.4 / 11.7, 22.1 / 13.8, FP8 15.5 / 15.5, 17.7 / 14.2, 23.7 / 16.3; d = 64, 8
// sequences of one KV head: 9.8 / 11.9, 11.0 / 11.6, 15.9 / 15.0.
long long most_rows(int n_tokens, int max_q, int g) { return static_cast<long long>(max_q <= 0 || max_q > n_tokens ? n_tokens : max_q) * g; }
bool few_rows(long long rows, long long units, long long room, int d)
{
    if (rows <= 8) return true;
    if (rows <= 16) return d == 64 || units > 16 || room < 1024;
    return rows <= kvattn::CHUNK_FEW_ROWS && units * room <= (d == 64 ? 8192 : 2048);
}

// The chunk workspace: the zero region (counters), then the partials.
struct ChunkWorkspace {
    size_t info = KVATTN_DECODE_WS_ZERO_BYTES, join, ml, o, total;
    ChunkWorkspace(bool few, int d)
    {
        const size_t rows = few ? size_t(2) * kvattn::CHUNK_MAX_SLOTS * kvattn::CHUNK_FEW_ROWS
                                : size_t(2) * kvattn::CHUNK_MAX_CTAS * kvattn::CHUNK_SLOT_ROWS;
        join = align_up(info + kvattn::CHUNK_MAX_CTAS * sizeof(int4));
        ml = align_up(join + (few ? rows * sizeof(float2) : 0));
        o = align_up(ml + rows * sizeof(float2));
        total = o + rows * d * sizeof(float);
    }
};

int append(const char* name, bool fp8, const kvattn_bf16* k_new, int64_t k_stride, const kvattn_bf16* v_new,
           int64_t v_stride, const int32_t* cu, const int32_t* seq_lens, const int32_t* page_table, int B,
           int n_tokens, int n_kv_head, int head_dim, int page_size, int max_pages, int n_pages, void* k_pages,
           float* k_scales, void* v_pages, float* v_scales, const float* cos_tab, const float* sin_tab, int max_pos,
           int pair_style, int32_t* dev_status, void* stream)
{
    int rc = check_batch(name, B, n_tokens, n_kv_head, n_kv_head, head_dim, page_size, max_pages, n_pages);
    if (rc != KVATTN_OK) return rc;
    if (pair_style != 0 && pair_style != 1) return record_error(KVATTN_ERR_UNSUPPORTED, "%s: pair_style %d", name, pair_style);
    if (max_pos < 1) return record_error(KVATTN_ERR_SHAPE, "%s: max_pos %d < 1", name, max_pos);
    if (n_tokens == 0) return ok();
    if (any_null(k_new, v_new, cu, seq_lens, page_table, k_pages, v_pages, cos_tab, sin_tab) ||
        (fp8 && any_null(k_scales, v_scales)))
        return record_error(KVATTN_ERR_NULL, "%s: NULL argument", name);
    if (!all_aligned(16, k_new, v_new, k_pages, v_pages, k_scales, v_scales, cos_tab, sin_tab) ||
        !all_aligned(4, cu, seq_lens, page_table, dev_status))
        return record_error(KVATTN_ERR_ALIGN, "%s: tensors must be 16-byte aligned", name);
    if ((rc = check_stride(name, "k_new", k_stride, n_kv_head, head_dim)) != KVATTN_OK) return rc;
    if ((rc = check_stride(name, "v_new", v_stride, n_kv_head, head_dim)) != KVATTN_OK) return rc;
    int sms = 0;
    if ((rc = sms_of_device(name, &sms)) != KVATTN_OK) return rc;
    kvattn::PagedAppendArgs a{};
    a.p = batch(cu, seq_lens, page_table, B, n_tokens, page_size, max_pages, n_pages, dev_status);
    a.k_new = k_new;
    a.v_new = v_new;
    a.k_st = k_stride;
    a.v_st = v_stride;
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.cos_tab = cos_tab;
    a.sin_tab = sin_tab;
    a.Hk = n_kv_head;
    a.d = head_dim;
    a.max_pos = max_pos;
    a.pair_style = pair_style;
    return finish(kvattn::launch_paged_append(a, fp8, sms, static_cast<cudaStream_t>(stream)), name);
}

int chunk(const char* name, bool fp8, const kvattn_bf16* q, int64_t q_stride, const int32_t* cu,
          const int32_t* seq_lens, const int32_t* page_table, int B, int n_tokens, int max_q, int n_head,
          int n_kv_head, int head_dim, int page_size, int max_pages, int n_pages, const void* k_pages,
          const float* k_scales, const void* v_pages, const float* v_scales, float scale, kvattn_bf16* out,
          float* lse, void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream)
{
    int rc = check_batch(name, B, n_tokens, n_head, n_kv_head, head_dim, page_size, max_pages, n_pages);
    if (rc != KVATTN_OK) return rc;
    const int g = n_head / n_kv_head;
    if (g > 64 || (g & (g - 1))) return record_error(KVATTN_ERR_UNSUPPORTED, "%s: group size %d", name, g);
    if (!(scale > 0.0f) || !std::isfinite(scale)) return record_error(KVATTN_ERR_SHAPE, "%s: scale must be finite > 0", name);
    if (n_tokens == 0) return ok();
    if (any_null(q, cu, seq_lens, page_table, k_pages, v_pages, out) || (fp8 && any_null(k_scales, v_scales)))
        return record_error(KVATTN_ERR_NULL, "%s: NULL argument", name);
    if (!all_aligned(16, q, k_pages, v_pages, k_scales, v_scales, out) ||
        !all_aligned(4, cu, seq_lens, page_table, lse, dev_status))
        return record_error(KVATTN_ERR_ALIGN, "%s: tensors must be 16-byte aligned", name);
    if ((rc = check_stride(name, "q", q_stride, n_head, head_dim)) != KVATTN_OK) return rc;
    const size_t need = attn_chunk_paged_workspace_bytes(B, n_tokens, max_q, n_head, n_kv_head, head_dim);
    if (!workspace || workspace_bytes < need)
        return record_error(KVATTN_ERR_WORKSPACE, "%s: workspace needs %zu bytes", name, need);
    if (!all_aligned(256, workspace)) return record_error(KVATTN_ERR_ALIGN, "%s: workspace must be 256-byte aligned", name);
    int sms = 0;
    if ((rc = sms_of_device(name, &sms)) != KVATTN_OK) return rc;
    kvattn::ChunkArgs a{};
    a.p = batch(cu, seq_lens, page_table, B, n_tokens, page_size, max_pages, n_pages, dev_status);
    a.q = q;
    a.q_st = q_stride;
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.out = out;
    a.lse = lse;
    a.H = n_head;
    a.Hk = n_kv_head;
    a.g = g;
    a.d = head_dim;
    a.max_q = max_q <= 0 || max_q > n_tokens ? n_tokens : max_q;
    a.scale = scale;
    const bool few = few_rows(most_rows(n_tokens, max_q, g), static_cast<long long>(B) * n_kv_head,
                              static_cast<long long>(max_pages) * page_size, head_dim);
    const ChunkWorkspace ws(few, head_dim);
    uint8_t* wp = static_cast<uint8_t*>(workspace);
    a.counters = reinterpret_cast<int*>(wp);
    a.split_info = reinterpret_cast<int4*>(wp + ws.info);
    a.join_ml = reinterpret_cast<float2*>(wp + ws.join);
    a.part_ml = reinterpret_cast<float2*>(wp + ws.ml);
    a.part_o = reinterpret_cast<float*>(wp + ws.o);
    const uint64_t row = head_dim * (fp8 ? 1 : 2), planes = static_cast<uint64_t>(n_pages) * n_kv_head;
    const uint32_t tile = few ? 64 : 128, box = page_size < static_cast<int>(tile) ? page_size : tile;
    const uint32_t byte_box = fp8 ? head_dim : 0;
    const CUtensorMapSwizzle sw = !few             ? CU_TENSOR_MAP_SWIZZLE_NONE
                                  : head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                                    : CU_TENSOR_MAP_SWIZZLE_64B;
    CUtensorMap mq, mk, mv;
    if ((rc = encode_map(name, &mk, k_pages, byte_box, head_dim, page_size, planes, row, row * page_size, box, 1, sw)) != KVATTN_OK ||
        (rc = encode_map(name, &mv, v_pages, byte_box, head_dim, page_size, planes, row, row * page_size, box, 1, sw)) != KVATTN_OK)
        return rc;
    if (few) return finish(kvattn::launch_chunk_rows(a, fp8, mk, mv, sms, static_cast<cudaStream_t>(stream)), name);
    if ((rc = encode_map(name, &mq, q, 0, head_dim, n_head, n_tokens, head_dim * 2, q_stride * 2, g, 128 / g)) != KVATTN_OK)
        return rc;
    return finish(kvattn::launch_chunk_tile(a, fp8, mq, mk, mv, sms, static_cast<cudaStream_t>(stream)), name);
}

}  // namespace

extern "C" {

int kv_append_paged_rope(const kvattn_bf16* k_new, int64_t k_stride, const kvattn_bf16* v_new, int64_t v_stride,
                         const int32_t* cu, const int32_t* seq_lens, const int32_t* page_table, int B, int n_tokens,
                         int n_kv_head, int head_dim, int page_size, int max_pages, int n_pages,
                         kvattn_bf16* k_pages, kvattn_bf16* v_pages, const float* cos_tab, const float* sin_tab,
                         int max_pos, int pair_style, int32_t* dev_status, void* stream)
{
    return append("kv_append_paged_rope", false, k_new, k_stride, v_new, v_stride, cu, seq_lens, page_table, B,
                  n_tokens, n_kv_head, head_dim, page_size, max_pages, n_pages, k_pages, nullptr, v_pages, nullptr,
                  cos_tab, sin_tab, max_pos, pair_style, dev_status, stream);
}

int kv_append_paged_rope_fp8(const kvattn_bf16* k_new, int64_t k_stride, const kvattn_bf16* v_new, int64_t v_stride,
                             const int32_t* cu, const int32_t* seq_lens, const int32_t* page_table, int B,
                             int n_tokens, int n_kv_head, int head_dim, int page_size, int max_pages, int n_pages,
                             uint8_t* k_codes, float* k_scales, uint8_t* v_codes, float* v_scales,
                             const float* cos_tab, const float* sin_tab, int max_pos, int pair_style,
                             int32_t* dev_status, void* stream)
{
    return append("kv_append_paged_rope_fp8", true, k_new, k_stride, v_new, v_stride, cu, seq_lens, page_table, B,
                  n_tokens, n_kv_head, head_dim, page_size, max_pages, n_pages, k_codes, k_scales, v_codes, v_scales,
                  cos_tab, sin_tab, max_pos, pair_style, dev_status, stream);
}

int kv_read_paged_fp8(const uint8_t* k_codes, const float* k_scales, const uint8_t* v_codes, const float* v_scales,
                      const int32_t* page_table, const int32_t* seq_lens, int B, int n_kv_head, int head_dim,
                      int page_size, int max_pages, int n_pages, int T_max, kvattn_bf16* k_out, kvattn_bf16* v_out,
                      int32_t* dev_status, void* stream)
{
    const char* name = "kv_read_paged_fp8";
    const int rc = check_batch(name, B, 0, n_kv_head, n_kv_head, head_dim, page_size, max_pages, n_pages);
    if (rc != KVATTN_OK) return rc;
    if (T_max < 1) return record_error(KVATTN_ERR_SHAPE, "%s: T_max %d", name, T_max);
    if (any_null(k_codes, k_scales, v_codes, v_scales, page_table, seq_lens, k_out, v_out))
        return record_error(KVATTN_ERR_NULL, "%s: NULL argument", name);
    if (!all_aligned(16, k_codes, k_scales, v_codes, v_scales, k_out, v_out) ||
        !all_aligned(4, page_table, seq_lens, dev_status))
        return record_error(KVATTN_ERR_ALIGN, "%s: tensors must be 16-byte aligned", name);
    kvattn::PagedReadArgs a{};
    a.p = batch(nullptr, seq_lens, page_table, B, 0, page_size, max_pages, n_pages, dev_status);
    a.k_codes = k_codes;
    a.v_codes = v_codes;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.k_out = k_out;
    a.v_out = v_out;
    a.Hk = n_kv_head;
    a.d = head_dim;
    a.T_max = T_max;
    return finish(kvattn::launch_paged_read(a, static_cast<cudaStream_t>(stream)), name);
}

size_t attn_chunk_paged_workspace_bytes(int B, int n_tokens, int max_q, int n_head, int n_kv_head, int head_dim)
{
    if (B < 1 || n_head < 1 || n_kv_head < 1 || n_head % n_kv_head || head_dim < 1) return 0;
    // (where either kernel may take the call, by its room: the tile kernel's partials are more)
    const long long rows = most_rows(n_tokens, max_q, n_head / n_kv_head);
    return ChunkWorkspace(rows <= 8 || (rows <= 16 && (head_dim == 64 || static_cast<long long>(B) * n_kv_head > 16)), head_dim).total;
}

int attn_chunk_paged(const kvattn_bf16* q, int64_t q_stride, const int32_t* cu, const int32_t* seq_lens,
                     const int32_t* page_table, int B, int n_tokens, int max_q, int n_head, int n_kv_head,
                     int head_dim, int page_size, int max_pages, int n_pages, const kvattn_bf16* k_pages,
                     const kvattn_bf16* v_pages, float scale, kvattn_bf16* out, float* lse, void* workspace,
                     size_t workspace_bytes, int32_t* dev_status, void* stream)
{
    return chunk("attn_chunk_paged", false, q, q_stride, cu, seq_lens, page_table, B, n_tokens, max_q, n_head,
                 n_kv_head, head_dim, page_size, max_pages, n_pages, k_pages, nullptr, v_pages, nullptr, scale, out,
                 lse, workspace, workspace_bytes, dev_status, stream);
}

int attn_chunk_paged_fp8(const kvattn_bf16* q, int64_t q_stride, const int32_t* cu, const int32_t* seq_lens,
                         const int32_t* page_table, int B, int n_tokens, int max_q, int n_head, int n_kv_head,
                         int head_dim, int page_size, int max_pages, int n_pages, const uint8_t* k_codes,
                         const float* k_scales, const uint8_t* v_codes, const float* v_scales, float scale,
                         kvattn_bf16* out, float* lse, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                         void* stream)
{
    return chunk("attn_chunk_paged_fp8", true, q, q_stride, cu, seq_lens, page_table, B, n_tokens, max_q, n_head,
                 n_kv_head, head_dim, page_size, max_pages, n_pages, k_codes, k_scales, v_codes, v_scales, scale, out,
                 lse, workspace, workspace_bytes, dev_status, stream);
}

}  // extern "C"

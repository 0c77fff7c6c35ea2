// chunk_plan.cuh -- how the tensor-core chunk kernel shares its work out.
//
// The query rows of (sequence b, KV head) are its tokens times the g heads of the
// group, token-major, cut into blocks of 256 rows (w = 256 / g tokens).  A block
// attends to the keys 0 .. (position of its last token), cut into tiles of 128: its
// unit has that many tiles, each costing 3 where the block has at most 128 rows and 4
// otherwise (the times that a tile takes then, about: 2600 and 3300 cycles; with 1 and 2 the
// CTAs of a mixed batch's decoding sequences took twice as long as those of its chunks).
// The costs of all units, in the order (sequence, head, block), form one
// line of length N; CTA c of G takes the stretch [c N / G, (c + 1) N / G) of it: the
// tiles whose first cost point lies there.  A unit that crosses a border is finished
// by the merge from one partial per CTA.  Everything is computed on the device, in
// closed form per sequence, so the host never waits for lengths.
#pragma once

#include "paged.cuh"

namespace kvattn {

constexpr int CH_ROWS = 256;  // query rows of a block
constexpr int CH_KEYS = 128;  // keys of a tile
constexpr int CH_COST1 = 3, CH_COST2 = 4;  // points of a tile with one and with two Q tiles

// Sums in closed form, by shifts: one thread walks the plan at the head of every call.
// Sum over i = 1 .. k of the tiles that base + i w keys fill, w = 1 << ws (4 .. 256).
__host__ __device__ inline long long chunk_tiles_prefix(int base, int ws, int k)
{
    int first = 1;  // the blocks before it end at or before row 0
    if (base < 0) first = (-base >> ws) + 1;
    if (k < first) return 0;
    const long long n = k - first + 1;
    const int x0 = base + ((first - 1) << ws);  // > -w, and x0 + w > 0
    if (ws >= 7) {
        const long long c0 = x0 > 0 ? (x0 + CH_KEYS - 1) >> 7 : -(-x0 >> 7);
        return n * c0 + ((n * (n + 1) / 2) << (ws - 7));
    }
    const int ms = 7 - ws;                                              // m = 1 << ms blocks per tile of keys
    const long long r = x0 > 0 ? (x0 + (1 << ws) - 1) >> ws : 0;        // ceil((x0 + i w) / 128) = ceil((r + i) / m)
    auto upto = [ms](long long x) {                                     // sum of ceil(i / m), i = 1 .. x
        const long long q = x >> ms;
        return ((q * (q + 1) / 2) << ms) + (x - (q << ms)) * (q + 1);
    };
    return upto(r + n) - upto(r);
}

struct ChunkSeq {
    int t0, n, take, len;  // packed tokens t0 .. t0 + take - 1 are computed (take = min(n, max_q))
    __host__ __device__ int base() const { return len - n; }
    // cost of this sequence's blocks 0 .. k - 1 on one KV head, blocks of 1 << ws tokens (256 rows)
    __host__ __device__ long long cost(int k, int ws) const
    {
        const int full = take >> ws;
        if (k <= full) return CH_COST2 * chunk_tiles_prefix(base(), ws, k);
        const int rest = take - (full << ws);
        const int keys = base() + take;
        const long long tiles = keys > 0 ? (keys + CH_KEYS - 1) >> 7 : 0;
        return CH_COST2 * chunk_tiles_prefix(base(), ws, full) + (2 * rest <= (1 << ws) ? CH_COST1 : CH_COST2) * tiles;
    }
    __host__ __device__ int blocks(int ws) const { return static_cast<int>((static_cast<long long>(take) + (1 << ws) - 1) >> ws); }
};

// floor(a / b) for quotients below 2^20, a < 2^62: a float guess, which is off by at most one, put right.
__host__ __device__ inline int small_quotient(long long a, long long b)
{
    int q = static_cast<int>(static_cast<float>(a) / static_cast<float>(b));
    if (static_cast<long long>(q + 1) * b <= a) ++q;
    if (static_cast<long long>(q) * b > a) --q;
    return q;
}

// One unit: a block of query rows of one sequence and KV head.
struct ChunkUnit {
    int b, kvh, rb;
    ChunkSeq s;
    long long U;     // its first point on the line
    int rows;        // query rows in use
    int keys;        // keys that its last token sees
    int tiles;       // 128-key tiles of them
    int keys0;       // keys that the last token of the first 128 rows sees
    int qt;          // Q tiles of 128 rows: 1 or 2
    __host__ __device__ int cost() const { return qt == 1 ? CH_COST1 : CH_COST2; }  // points per tile
};

// Where the batch lies in shared memory: raw offsets and lengths, and the line's prefix
// per sequence for one KV head.
struct ChunkPlan {
    const int* cu;
    const int* len;
    const long long* U;  // [B + 1]
    int B, Hk, g, ws, max_q;  // blocks of 1 << ws tokens
    const PagedBatch* p;

    __host__ __device__ ChunkSeq seq(int b) const
    {
        const PagedSeq s = paged_seq(*p, cu[b], cu[b + 1], len[b]);
        return ChunkSeq{s.t0, s.n, min(s.n, max_q), s.len};
    }
    __host__ __device__ long long total() const { return U[B] * Hk; }

    __host__ __device__ void fill(ChunkUnit& u) const  // rows, keys and tiles from b, rb
    {
        const int w = 1 << ws, i0 = u.rb << ws, left = min(u.s.take - i0, w);
        u.rows = left * g;
        u.keys = max(u.s.base() + i0 + left, 0);
        u.tiles = (u.keys + CH_KEYS - 1) >> 7;
        u.qt = u.rows <= CH_ROWS / 2 ? 1 : 2;
        // the first 128 rows end with token i0 + w / 2 - 1 (g <= 64: w / 2 >= 2); g = 1: w = 256
        u.keys0 = u.qt == 1 ? u.keys : max(u.s.base() + i0 + w / 2, 0);
    }

    // the unit holding point x (0 <= x < total())
    __host__ __device__ ChunkUnit find(long long x) const
    {
        int lo = 0, hi = B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (U[mid] * Hk <= x) lo = mid;
            else hi = mid - 1;
        }
        ChunkUnit u;
        u.b = lo;
        u.s = seq(lo);
        const long long per = U[lo + 1] - U[lo];
        x -= U[lo] * Hk;
        u.kvh = small_quotient(x, per);
        x -= u.kvh * per;
        int a = 0, z = u.s.blocks(ws) - 1;
        while (a < z) {
            const int mid = (a + z + 1) >> 1;
            if (u.s.cost(mid, ws) <= x) a = mid;
            else z = mid - 1;
        }
        u.rb = a;
        u.U = U[lo] * Hk + u.kvh * per + u.s.cost(a, ws);
        fill(u);
        return u;
    }

    // the next unit with tiles; b = B behind the last one
    __host__ __device__ void next(ChunkUnit& u) const
    {
        u.U += static_cast<long long>(u.cost()) * u.tiles;
        ++u.rb;
        while (u.b < B) {
            const int nb = u.s.blocks(ws);
            for (; u.rb < nb; ++u.rb) {
                fill(u);
                if (u.tiles > 0) return;
            }
            u.rb = 0;
            if (++u.kvh < Hk && U[u.b + 1] > U[u.b]) continue;
            u.kvh = 0;
            do ++u.b;
            while (u.b < B && U[u.b + 1] == U[u.b]);
            if (u.b < B) u.s = seq(u.b);
        }
    }

    // tiles [tb, te) of u whose first points lie in [lo, hi)
    __host__ __device__ bool piece(const ChunkUnit& u, long long lo, long long hi, int& tb, int& te) const
    {
        const uint32_t a = static_cast<uint32_t>(max(lo, u.U) - u.U);  // (a unit has less than 2^26 points)
        const uint32_t z = static_cast<uint32_t>(min(hi - u.U, static_cast<long long>(u.cost()) * u.tiles));
        auto tile = [&](uint32_t x) { return static_cast<int>(u.qt == 1 ? (x + CH_COST1 - 1) / CH_COST1 : (x + CH_COST2 - 1) / CH_COST2); };
        tb = tile(a);
        te = tile(z);
        return tb < te;
    }
};

__host__ __device__ __forceinline__ int chunk_owner(long long x, long long N, int G)
{
    // c with ceil(c N / G) <= x < ceil((c + 1) N / G)
    return small_quotient(x * G, N);
}

__host__ __device__ __forceinline__ long long chunk_start(int c, long long N, int G)
{
    // ceil(c N / G): a guess in double, put right
    const long long a = static_cast<long long>(c) * N;
    long long q = static_cast<long long>(static_cast<double>(a) * (1.0 / G));
    while (q * G < a) ++q;
    while ((q - 1) * G >= a) --q;
    return q;
}

// Block-wide: reads the batch, checks it, and builds the line's prefix.
__device__ inline void chunk_plan_build(const PagedBatch& p, int ws, int max_q, int* s_cu, int* s_len,
                                        long long* s_U, bool report)
{
    for (int b = threadIdx.x; b <= p.B; b += blockDim.x) {
        s_cu[b] = p.cu[b];
        if (b < p.B) s_len[b] = p.seq_lens[b];
    }
    __syncthreads();
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
        const PagedSeq s = paged_seq(p, s_cu[b], s_cu[b + 1], s_len[b]);
        if (report && (s.bad || s.n > max_q)) report_status(p.dev_status, KVATTN_STATUS_BAD_LENGTH);
        const ChunkSeq q{s.t0, s.n, min(s.n, max_q), s.len};
        s_U[b + 1] = q.cost(q.blocks(ws), ws);
    }
    if (threadIdx.x == 0) s_U[0] = 0;
    __syncthreads();
    if (threadIdx.x < 32 && p.B > 1) {
        const int lane = threadIdx.x;
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
}

}  // namespace kvattn

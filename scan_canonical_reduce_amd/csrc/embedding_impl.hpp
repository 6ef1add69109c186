// Embedding lookup, and its gradient as a canonical reduction by key.
//
// Lookup: 16-byte accesses, one row's vectors in neighbouring threads; bound
// by memory traffic (16384 rows of 4096 bf16: 34 us with ids that fall as 1/rank,
// whose frequent rows stay in the caches).
//
// Gradient: one kernel for few tokens (k_embed_direct, k_embed_one), else three:
//  1. k_embed_group: tokens by id, ascending within an id, without a sort
//     pass over memory.  Workgroup b owns the ids [b R, b R + R) and reads all
//     ids twice (they stay in cache): once to count its own ids, per wave, and
//     the ids below its range, which place it in the order; once to place its
//     tokens, each wave its own stretch, in token order.  No workgroup needs
//     another's result, so there is one launch and no wait.  It also lists the
//     work: (row, chunk of 64 occurrences).
//  2. k_embed_sum: a wave takes one entry and a slab of 64 vectors of columns,
//     and adds the rows of dout in the order of the pairwise tree (8 rows in
//     flight, a binary counter of complete subtrees above them).  An aligned
//     chunk of a sequence is a subtree of its pairwise tree, so the rows of an
//     id with more than 64 occurrences leave one partial value per chunk.  The
//     rows that no token names are set to zero by the same waves, some rows'
//     offsets at a time; every other workgroup does that first, so that the
//     writes overlap the others' gathers.
//  3. k_embed_finish: the tree over the partial values.
// 16384 tokens of 4096 bf16 into 65536 float32 rows: 13 + 227 + 8 us, 1.2 GB at 4.9
// TB/s, nearly all of them the zero rows' writes and the gathers.
#pragma once

#include <type_traits>

#include "embedding.hpp"
#include "launch.hpp"

namespace canon {
namespace seq {

__device__ __forceinline__ int64_t token_id(const void* ids, bool ids64, int64_t t)
{
    return ids64 ? static_cast<const int64_t*>(ids)[t]
                 : (int64_t) static_cast<const int32_t*>(ids)[t];
}

template <typename T, int V, bool AL>
__global__ __launch_bounds__(256) void k_embedding(EmbedArgs a)
{
    using E = typename T::store_t;
    const int64_t nv = (a.width + V - 1) / V;
    const int64_t n = a.tokens * nv;
    constexpr int U = 4;
    const int64_t i0 = (int64_t)blockIdx.x * (256 * U) + threadIdx.x;
    Vec<T, V> x[U];
    E* dst[U];
    float scale[U];  // 0 for an id outside the table, whatever the scale
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = i0 + u * 256;
        dst[u] = nullptr;
        x[u] = Vec<T, V>{};
        scale[u] = 0.f;
        if (i < n) {
            const int64_t t = i / nv, c = vec_col<V, AL>((i - t * nv) * V, a.width);
            const int64_t id = token_id(a.ids, a.ids64, t);
            dst[u] = static_cast<E*>(a.out) + t * a.ld_out + c;
            if (id >= 0 && id < a.rows) {
                x[u] = ld_any<T, V, AL>(static_cast<const E*>(a.weight) + id * a.ld_weight + c);
                scale[u] = a.scale;
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (!dst[u]) continue;
        float y[V];
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] = T::load(x[u].e[j]) * scale[u];
        st_any<T, V, AL>(dst[u], y);
    }
}

// The pairwise tree over rows that arrive eight at a time, V columns each: a
// binary counter of complete subtrees.  Missing rows of the last batch are -0,
// the exact identity of an addition.
template <int V, int LEVELS>
struct PairCounter {
    float sub[LEVELS][V] = {};  // subtrees of 8, 16, 32, ... rows
    uint32_t batches = 0;

    __device__ __forceinline__ void add(float (&x)[8][V])
    {
#pragma unroll
        for (int d = 1; d < 8; d *= 2)
#pragma unroll
            for (int r = 0; r < 8; r += 2 * d)
#pragma unroll
                for (int j = 0; j < V; ++j) x[r][j] += x[r + d][j];
        // the value goes up over the set bits of the count, to the first clear one
        bool done = false;
#pragma unroll
        for (int l = 0; l < LEVELS; ++l) {
            if (V == 1) {
                // selections: of branches that store one value the compiler makes
                // one store to an array in memory
                const bool up = batches >> l & 1, here = !up && !done;
                const float sum = sub[l][0] + x[0][0];
                sub[l][0] = here ? x[0][0] : sub[l][0];
                x[0][0] = up && !done ? sum : x[0][0];
                done |= here;
                continue;
            }
            if (done) continue;
            if (batches >> l & 1) {
#pragma unroll
                for (int j = 0; j < V; ++j) x[0][j] = sub[l][j] + x[0][j];
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) sub[l][j] = x[0][j];
                done = true;
            }
        }
        ++batches;
    }
    __device__ __forceinline__ void total(float (&acc)[V]) const
    {
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = -0.f;
#pragma unroll
        for (int l = 0; l < LEVELS; ++l)
            if (batches >> l & 1)
#pragma unroll
                for (int j = 0; j < V; ++j) acc[j] = sub[l][j] + acc[j];
    }
};

// Stores V columns from c on, all but the first `skip` (which the vector before
// has stored).
template <typename G, int V, bool AL>
__device__ __forceinline__ void store_grad(const EmbedGradArgs& a, int64_t v, int64_t c,
                                           const float (&sum)[V], int skip)
{
    typename G::store_t* p = static_cast<typename G::store_t*>(a.dw) + v * a.ld_dw + c;
    float y[V];
#pragma unroll
    for (int j = 0; j < V; ++j) y[j] = sum[j] * a.scale;
    if (!AL && skip) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j >= skip) p[j] = G::round(a.accumulate ? G::load(p[j]) + y[j] : y[j]);
        return;
    }
    if (a.accumulate) {
        const Vec<G, V> old = ld_any<G, V, AL>(p);
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] = G::load(old.e[j]) + y[j];
    }
    st_any<G, V, AL>(p, y);
}

// Groups whose prefix sums a workgroup keeps in LDS; callers walk more groups
// in blocks of that many.
constexpr int kGroupsInLds = 1024;

// Prefix sums of the counts of groups [first, first + kGroupsInLds), by the
// first 256 threads of the workgroup; returns the total to all.
__device__ __forceinline__ int64_t group_prefix(const int32_t* counts, int64_t first,
                                                int64_t groups, int32_t* prefix)
{
    __shared__ int32_t wave_sum[4];
    const int tid = threadIdx.x;
    int32_t c[4], s = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t g = first + tid * 4 + i;
        c[i] = tid < 256 && g < groups ? counts[g] : 0;
        s += c[i];
    }
    int32_t run = s;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int32_t o = __shfl_up(run, d, 64);
        if ((tid & 63) >= d) run += o;
    }
    __syncthreads();  // the previous block's prefix is no longer read
    if (tid < 256 && (tid & 63) == 63) wave_sum[tid >> 6] = run;
    __syncthreads();
    if (tid < 256) {
        int32_t base = run - s;
        for (int w = 0; w < (tid >> 6); ++w) base += wave_sum[w];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            prefix[tid * 4 + i] = base;
            base += c[i];
        }
        if (tid == 255) prefix[kGroupsInLds] = base;
    }
    __syncthreads();
    return prefix[kGroupsInLds];
}

// The group holding entry i of a block: the last g with prefix[g] <= i among
// those with entries.
__device__ __forceinline__ int find_group(const int32_t* prefix, int32_t i)
{
    int lo = 0, hi = kGroupsInLds - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= i)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Occurrences of an entry's chunk.
__device__ __forceinline__ int entry_tokens(int4 item)
{
    const int left = item.w - item.y * kEmbedChunk;
    return left < kEmbedChunk ? left : kEmbedChunk;
}

// Sums an entry (row, chunk, the row's offset and number of tokens): the tokens
// that the lanes hold in `mine`, V columns of this lane.
template <typename T, typename G, int V, bool AL>
__device__ __forceinline__ void sum_entry(const EmbedGradArgs& a, int4 item, int32_t mine,
                                          int64_t lane_col)
{
    const int64_t v = item.x, c = item.y;
    const int32_t off = item.z, n = item.w;
    const bool in = lane_col < a.width;
    const int64_t col = vec_col<V, AL>(lane_col, a.width);
    float acc[V];
    const int64_t p0 = off + c * kEmbedChunk;
    const int m = entry_tokens(item);
    const typename T::store_t* x = static_cast<const typename T::store_t*>(a.dout) + (in ? col : 0);
    auto row = [&](int k) {
        return ld_any<T, V, AL>(x + (int64_t)__builtin_amdgcn_readlane(mine, k) * a.ld_dout);
    };
    if (m == 1) {  // most rows of a large table
        const Vec<T, V> raw = row(0);
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = T::load(raw.e[j]);
    } else {
        PairCounter<V, 4> tree;
        for (int b = 0; b * 8 < m; ++b) {
            Vec<T, V> raw[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) raw[r] = row(b * 8 + r < m ? b * 8 + r : 0);
            float t[8][V];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const Vec<T, V> one = whole(raw[r]);
#pragma unroll
                for (int j = 0; j < V; ++j) t[r][j] = b * 8 + r < m ? T::load(one.e[j]) : -0.f;
            }
            tree.add(t);
        }
        tree.total(acc);
    }
    if (!in) return;
    if (n <= kEmbedChunk) {
        store_grad<G, V, AL>(a, v, col, acc, (int)(lane_col - col));
        return;
    }
    // Full chunks and last chunks of long rows each start at least 64
    // occurrences apart, so start / 64 numbers them.
    const bool last = (c + 1) * kEmbedChunk >= n;
    float* part = (last ? a.part_last + p0 / kEmbedChunk * a.ld_part
                        : a.part + (off / kEmbedChunk + c) * a.ld_part) + col;
#pragma unroll
    for (int j = 0; j < V; ++j) part[j] = acc[j];
}

// Sets columns [c0, c1) of the rows v0 + (set bits of left) to zero.
template <typename G, int V, bool AL>
__device__ __forceinline__ void zero_listed(const EmbedGradArgs& a, int64_t v0, uint64_t left,
                                            int64_t c0, int64_t c1, int lane)
{
    while (left) {
        const int64_t row = v0 + __builtin_ctzll(left);
        left &= left - 1;
        typename G::store_t* p = static_cast<typename G::store_t*>(a.dw) + row * a.ld_dw;
        if constexpr (V * sizeof(typename G::store_t) == 16) {
            typedef uint32_t u4 __attribute__((ext_vector_type(4)));
            const u4 zero = {0, 0, 0, 0};
            int64_t b = c0, e = c1;
            if (!AL) {
                // whole cache lines go past the caches; elements before the first one
                // and after the last, at most 63, share theirs with other rows
                constexpr int line = 128 / (int)sizeof(typename G::store_t);
                const int64_t head = (int64_t)((0 - reinterpret_cast<uintptr_t>(p + c0)) % 128) /
                                     (int64_t)sizeof(*p);
                b = head < c1 - c0 ? c0 + head : c1;
                e = c1 - (c1 - b) % line;
                if (lane < b - c0) p[c0 + lane] = 0;
                if (lane < c1 - e) p[e + lane] = 0;
            }
            for (int64_t c = b + lane * V; c < e; c += 64 * V)
                __builtin_nontemporal_store(zero, reinterpret_cast<u4*>(p + c));
        } else {
            for (int64_t c = c0 + lane; c < c1; c += 64) p[c] = 0;
        }
    }
}

// Rows a wave looks at at a time for ones to set to zero: few enough that a
// table of 65536 rows keeps 4096 waves busy.
constexpr int kZeroRows = 16;

// Rows to set to zero, kZeroRows at a time, and where they are few, cut into
// parts of their columns, of two accesses or more, so that every wave has some (4
// tokens, 118 rows of 3443 float32: 27 -> 10 us): f(first row, first column, end).
template <int V, class F>
__device__ __forceinline__ void each_zero_part(const EmbedGradArgs& a, int64_t wave,
                                               int64_t waves, F&& f)
{
    const uint32_t blocks = (uint32_t)((a.rows + kZeroRows - 1) / kZeroRows);
    const uint32_t steps = (uint32_t)((a.width + 64 * V - 1) / (64 * V));
    uint32_t parts = (uint32_t)waves / blocks;
    parts = parts < steps / 2 ? parts : steps / 2;
    if (parts < 1) parts = 1;
    const int64_t per = (int64_t)((steps + parts - 1) / parts) * (64 * V);
    for (uint32_t i = (uint32_t)wave; i < blocks * parts; i += (uint32_t)waves) {
        const uint32_t b = i / parts;
        const int64_t c0 = (i - b * parts) * per;
        f((int64_t)b * kZeroRows, c0, c0 + per < a.width ? c0 + per : a.width);
    }
}

// Zero rows for ids without tokens.
template <typename G, int V, bool AL>
__device__ __forceinline__ void zero_rows(const EmbedGradArgs& a, int64_t wave, int64_t waves,
                                          int lane)
{
    each_zero_part<V>(a, wave, waves, [&](int64_t v0, int64_t c0, int64_t c1) {
        const int64_t v = v0 + lane;
        const bool none =
            lane < kZeroRows && v < a.rows && a.offset[v] == a.offset[v + 1];
        zero_listed<G, V, AL>(a, v0, __ballot(none), c0, c1, lane);
    });
}

template <typename T, typename G, int V, bool AL>
__global__ __launch_bounds__(256, 4) void k_embed_sum(EmbedGradArgs a, int64_t groups)
{
    __shared__ int32_t prefix[kGroupsInLds + 1];
    const int lane = threadIdx.x & 63;
    const int64_t wave = (int64_t)blockIdx.x * 4 + uniform((int32_t)(threadIdx.x >> 6));
    const int64_t waves = gridDim.x * 4ll;
    const int64_t slabs = (a.width + 64 * V - 1) / (64 * V);
    // 16-byte stores of the gradient's type
    constexpr int VZ = V == 1 ? 1 : 16 / (int)sizeof(typename G::store_t);
    const bool zero = !a.accumulate;
    if (zero && (blockIdx.x & 1)) zero_rows<G, VZ, AL>(a, wave, waves, lane);
    for (int64_t g0 = 0; g0 < groups; g0 += kGroupsInLds) {
        const int64_t total = group_prefix(a.n_items, g0, groups, prefix);
        for (int64_t i = wave; i < total * slabs; i += waves) {
            const int32_t e = (int32_t)(i / slabs);
            const int64_t slab = i - e * slabs;
            const int k = find_group(prefix, e);
            int4 item = a.items[(int64_t)a.before[g0 + k] + (e - prefix[k])];
            item = make_int4(uniform(item.x), uniform(item.y), uniform(item.z), uniform(item.w));
            const int32_t at = item.z + item.y * kEmbedChunk;
            const int32_t mine = a.order[at + (lane < entry_tokens(item) ? lane : 0)];
            sum_entry<T, G, V, AL>(a, item, mine, slab * 64 * V + lane * V);
        }
    }
    if (zero && !(blockIdx.x & 1)) zero_rows<G, VZ, AL>(a, wave, waves, lane);
}

// Up to 128 tokens, one launch and no workspace: a wave keeps all ids, two a
// lane.  For each (token, slab of columns) it takes, the ballots of "same id" tell
// whether the token is its id's first, and are the list of occurrences, in order;
// rows of the table without a token are found the same way.  Measured against
// grouping in LDS (k_embed_one), us a call, frequencies falling as 1/rank (all tokens
// one id, whose rows one wave adds, 16 in flight): 64 x 1000 of 10007 rows bf16 9.1
// and 10.3 (12.5 and 15.5), 128 9.0 and 10.5 (18 and 17), 256 9.1 and 10.8 (40 and 17).
constexpr int kEmbedDirect = 128;

template <typename T, typename G, int V, bool AL>
__global__ __launch_bounds__(256) void k_embed_direct(EmbedGradArgs a)
{
    const int lane = threadIdx.x & 63;
    const int64_t wave = (int64_t)blockIdx.x * 4 + uniform((int32_t)(threadIdx.x >> 6));
    const int64_t waves = gridDim.x * 4ll;
    constexpr int C = kEmbedDirect / 64;
    int32_t id[C];  // of tokens 64 k + lane; -1: none
#pragma unroll
    for (int k = 0; k < C; ++k) {
        const int64_t t = k * 64 + lane;
        const int64_t v = t < a.tokens ? token_id(a.ids, a.ids64, t) : -1;
        id[k] = v >= 0 && v < a.rows && v != a.padding_id ? (int32_t)v : -1;
    }
    const int32_t slabs = (int32_t)((a.width + 64 * V - 1) / (64 * V));
    for (int64_t i = wave; i < a.tokens * slabs; i += waves) {
        const int32_t t = (int32_t)i / slabs, slab = (int32_t)i - t * slabs;
        int32_t v = -1;
#pragma unroll
        for (int k = 0; k < C; ++k)
            if (t >> 6 == k) v = __builtin_amdgcn_readlane(id[k], t & 63);
        if (v < 0) continue;
        uint64_t same[C];
        int32_t first = -1;
#pragma unroll
        for (int k = C - 1; k >= 0; --k) {
            same[k] = __ballot(id[k] == v);
            if (same[k]) first = k * 64 + __builtin_ctzll(same[k]);
        }
        if (first != t) continue;
        const int64_t lane_col = (int64_t)slab * 64 * V + lane * V;
        const bool in = lane_col < a.width;
        const int64_t col = vec_col<V, AL>(lane_col, a.width);
        const typename T::store_t* x =
            static_cast<const typename T::store_t*>(a.dout) + (in ? col : 0);
        PairCounter<V, 5> tree;
        int k = 0;
        uint64_t cur = same[0];
        bool more = true;
        while (more) {
            Vec<T, V> raw[2 * 8];
            int n = 0;
#pragma unroll
            for (int r = 0; r < 2 * 8; ++r) {
#pragma unroll
                for (int q = 1; q < C; ++q)
                    if (cur == 0 && k < q) {
                        k = q;
                        cur = same[q];
                    }
                if (cur) {
                    const int64_t row = k * 64 + __builtin_ctzll(cur);
                    cur &= cur - 1;
                    raw[r] = ld_any<T, V, AL>(x + row * a.ld_dout);
                    n = r + 1;
                }
            }
            more = n == 2 * 8;  // these may be the last: then there is no next one
#pragma unroll
            for (int half = 0; half < 2 * 8; half += 8) {
                if (n <= half) break;
                float s[8][V];
#pragma unroll
                for (int r = 0; r < 8; ++r)
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        s[r][j] = half + r < n ? T::load(raw[half + r].e[j]) : -0.f;
                tree.add(s);
            }
        }
        float acc[V];
        tree.total(acc);
        if (in) store_grad<G, V, AL>(a, v, col, acc, (int)(lane_col - col));
    }
    if (a.accumulate) return;
    // 16-byte stores of the gradient's type
    constexpr int VZ = V == 1 ? 1 : 16 / (int)sizeof(typename G::store_t);
    each_zero_part<VZ>(a, wave, waves, [&](int64_t v0, int64_t c0, int64_t c1) {
        uint64_t left = (1ull << (a.rows - v0 < kZeroRows ? a.rows - v0 : kZeroRows)) - 1;
#pragma unroll
        for (int k = 0; k < C; ++k) {
            uint64_t hit = __ballot(id[k] >= v0 && id[k] < v0 + kZeroRows);
            while (hit) {
                const int32_t v = __builtin_amdgcn_readlane(id[k], __builtin_ctzll(hit));
                hit &= hit - 1;
                left &= ~(1ull << (v - v0));
            }
        }
        zero_listed<G, VZ, AL>(a, v0, left, c0, c1, lane);
    });
}

// The pairwise tree over a long row's partial values [lo, hi) of m, eight in
// flight, four columns a lane.
template <int LEVELS>
__device__ __forceinline__ void tree_partials(const EmbedGradArgs& a, int32_t off, int32_t m,
                                              int32_t lo, int32_t hi, int64_t col,
                                              float (&acc)[4])
{
    const float* part = a.part + off / kEmbedChunk * a.ld_part + col;
    const float* last =
        a.part_last + (off + (m - 1) * kEmbedChunk) / kEmbedChunk * a.ld_part + col;
    PairCounter<4, LEVELS> tree;
    for (int32_t b = lo; b < hi; b += 8) {
        float x[8][4];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const int32_t j = b + r;
            float4 p = make_float4(-0.f, -0.f, -0.f, -0.f);
            if (j < hi)
                p = *reinterpret_cast<const float4*>(j == m - 1 ? last : part + j * a.ld_part);
            x[r][0] = p.x, x[r][1] = p.y, x[r][2] = p.z, x[r][3] = p.w;
        }
        tree.add(x);
    }
    tree.total(acc);
}

// Up to 4096 tokens, one launch: a workgroup groups the tokens of its ids in LDS
// (as k_embed_group; its ids are those equal to its number modulo a power of two,
// so that neighbouring frequent ones fall to different workgroups) and sums their
// rows in its part of the columns.  A frequent id is one workgroup's in each 512
// (16-bit) or 256 columns, so beyond 1024 tokens it is taken where it gains with
// spread ids: rows of fewer than 8 such parts, tables of up to 64 MiB.  Measured
// against three launches, us a call, bf16, frequencies falling as 1/rank (half the
// tokens one id; all):
//   1000 x 512 of 10007 rows    16 and 25 (18 and 25; 25 and 25)
//   1000 x 4096 of 10007 rows   27 and 33 (32 and 33; 35 and 34)
//   3001 x 1000 of 10007 rows   18 and 26 (39 and 26; 66 and 28)
//   4096 x 1000 of 10007 rows   20 and 27 (48 and 27; 86 and 30)
// and not taken:
//   4096 x 2048 of 32000 rows   42 and 44 (69 and 44; 99 and 43)
//   3001 x 4096 of 10007 rows   34 and 36 (53 and 37; 73 and 38)
//   4096 x 4096 of 32000 rows   78 and 70 (119 and 69; 138 and 68)
//   4096 x 8192 of 10007 rows   65 and 56 (116 and 56; 185 and 53)
// Nor above 1024 tokens for fewer than 256 rows or so, where few workgroups would
// have all tokens.
constexpr int kEmbedOne = 4096;
constexpr int kOneIds = 512;

struct OneShape {
    int log_groups, ids, parts;  // ids: of a workgroup; parts: of the columns
    int64_t blocks() const { return (int64_t)parts << log_groups; }
};

template <typename T, typename G, int V, bool AL>
__global__ __launch_bounds__(64 * kGroupWaves) void k_embed_one(EmbedGradArgs a, OneShape shape)
{
    extern __shared__ int32_t hist[];  // [wave][id]: count, then the next position
    __shared__ Pairs scan[kGroupWaves];
    __shared__ int32_t order[kEmbedOne], first_item[kOneIds + 1], first_token[kOneIds + 1];
    __shared__ int32_t longs[kEmbedOne / (kEmbedChunk + 1) + 1];
    const int tid = threadIdx.x, lane = tid & 63, w = uniform((int32_t)(tid >> 6));
    const int R = shape.ids;
    const uint32_t mask = (1u << shape.log_groups) - 1, own = blockIdx.x & mask;
    for (int i = tid; i < kGroupWaves * R; i += 64 * kGroupWaves) hist[i] = 0;
    __syncthreads();

    // Each wave's stretch of the tokens, whole batches of 64: ids in registers.
    constexpr int U = kEmbedOne / (64 * kGroupWaves);
    const int32_t batches = ((int32_t)a.tokens + 64 * kGroupWaves - 1) / (64 * kGroupWaves);
    const int32_t t0 = w * batches * 64 + lane;
    int32_t key[U];  // number of the id within the workgroup's, -1: none of them
    uint32_t below = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int32_t t = t0 + u * 64;
        const int64_t id =
            u < batches && t < a.tokens ? token_id(a.ids, a.ids64, t) : -1;
        const bool real = id >= 0 && id < a.rows && id != a.padding_id;
        const uint32_t group = (uint32_t)id & mask;
        below += real && group < own;
        key[u] = real && group == own ? (int32_t)(id >> shape.log_groups) : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (key[u] >= 0) atomicAdd(&hist[w * R + key[u]], 1);
    __syncthreads();

    // thread r: the counts of its id over the waves, in wave order
    int32_t n = 0;
    if (tid < R)
#pragma unroll
        for (int k = 0; k < kGroupWaves; ++k) {
            const int32_t c = hist[k * R + tid];
            hist[k * R + tid] = n;
            n += c;
        }
    const bool is_long = n > kEmbedChunk;
    uint64_t x = (uint64_t)(uint32_t)n |
                 (uint64_t)(uint32_t)((n + kEmbedChunk - 1) / kEmbedChunk) << 32;
    uint64_t y = (uint64_t)is_long | (uint64_t)below << 32;
    const Pairs at = block_exclusive(x, y, scan);
    const int32_t off = (int32_t)(uint32_t)at.x, n_items = (int32_t)(x >> 32);
    const int32_t n_long = (int32_t)(uint32_t)y, before = (int32_t)(y >> 32);
    if (tid < R) {
#pragma unroll
        for (int k = 0; k < kGroupWaves; ++k) hist[k * R + tid] += off;
        first_item[tid] = (int32_t)(at.x >> 32);
        first_token[tid] = off;
    }
    if (is_long) longs[(uint32_t)at.y] = tid;
    if (tid == 0) {
        first_item[R] = n_items;
        first_token[R] = (int32_t)(uint32_t)x;
    }
    __syncthreads();
    // Placing: a wave's lanes with the same id take consecutive positions.
#pragma unroll
    for (int u = 0; u < U; ++u) {
        uint64_t left = __ballot(key[u] >= 0);
        while (left) {
            const int lead = __builtin_amdgcn_readlane(key[u], __builtin_ctzll(left));
            const uint64_t same = __ballot(key[u] == lead);
            if (key[u] == lead)
                order[hist[w * R + lead] + __popcll(same & ((1ull << lane) - 1))] = t0 + u * 64;
            wave_lds_fence();
            if (lane == 0) hist[w * R + lead] += __popcll(same);
            wave_lds_fence();
            left &= ~same;
        }
    }
    __syncthreads();

    const int32_t part = (int32_t)(blockIdx.x >> shape.log_groups);
    const int32_t steps = (int32_t)((a.width + 64 * V - 1) / (64 * V));
    const int32_t per = (steps + shape.parts - 1) / shape.parts;
    const int64_t c0 = (int64_t)part * per * (64 * V);
    const int64_t c1 = c0 + per * (64 * V) < a.width ? c0 + per * (64 * V) : a.width;
    const int32_t slabs = c1 > c0 ? (int32_t)((c1 - c0 + 64 * V - 1) / (64 * V)) : 0;
    for (int32_t i = w; i < n_items * slabs; i += kGroupWaves) {
        const int32_t e = i / slabs;
        int r0 = 0, r1 = R - 1;  // the last id with first_item <= e
        while (r0 < r1) {
            const int mid = (r0 + r1 + 1) >> 1;
            if (first_item[mid] <= e)
                r0 = mid;
            else
                r1 = mid - 1;
        }
        const int32_t begin = uniform(first_token[r0]), chunk = e - uniform(first_item[r0]);
        const int4 item =
            make_int4((int32_t)(own + ((uint32_t)r0 << shape.log_groups)), chunk, before + begin,
                      uniform(first_token[r0 + 1]) - begin);
        const int32_t mine =
            order[begin + chunk * kEmbedChunk + (lane < entry_tokens(item) ? lane : 0)];
        sum_entry<T, G, V, AL>(a, item, mine, c0 + (i - e * slabs) * (64 * V) + lane * V);
    }
    if (!a.accumulate) {
        constexpr int VZ = V == 1 ? 1 : 16 / (int)sizeof(typename G::store_t);
        for (int r = w; r < R; r += kGroupWaves) {
            const int64_t v = own + ((int64_t)r << shape.log_groups);
            if (v < a.rows && uniform(first_token[r]) == uniform(first_token[r + 1]))
                zero_listed<G, VZ, AL>(a, v, 1, c0, c1, lane);
        }
    }
    if (n_long == 0) return;
    __syncthreads();
    const int32_t cols = c1 > c0 ? (int32_t)((c1 - c0 + 255) / 256) : 0;
    for (int32_t i = w; i < n_long * cols; i += kGroupWaves) {
        const int32_t e = i / cols, r = uniform(longs[e]);
        const int64_t col = c0 + (int64_t)(i - e * cols) * 256 + lane * 4;
        const int32_t begin = uniform(first_token[r]), count = uniform(first_token[r + 1]) - begin;
        const int32_t m = (count + kEmbedChunk - 1) / kEmbedChunk;
        float acc[4];
        tree_partials<4>(a, before + begin, m, 0, m, col < c1 ? col : c0, acc);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float one[1] = {acc[j]};
            if (col + j < c1)
                store_grad<G, 1, true>(a, own + ((int64_t)r << shape.log_groups), col + j, one, 0);
        }
    }
}

// Rows with more than 64 occurrences: the pairwise tree over the partial
// values, an aligned power-of-two range of them per wave, then over the
// waves.  A lane holds four neighbouring columns (the partial values' rows are
// padded to that).
constexpr int kFinishWaves = 8;

template <typename G>
__global__ __launch_bounds__(64 * kFinishWaves) void k_embed_finish(EmbedGradArgs a, int64_t groups)
{
    __shared__ int32_t prefix[kGroupsInLds + 1];
    __shared__ float4 waves[kFinishWaves][64];
    const int lane = threadIdx.x & 63, w = uniform((int32_t)(threadIdx.x >> 6));
    const int64_t slabs = (a.width + 255) / 256;
    for (int64_t g0 = 0; g0 < groups; g0 += kGroupsInLds) {
        const int64_t total = group_prefix(a.n_long, g0, groups, prefix);
        for (int64_t i = blockIdx.x; i < total * slabs; i += gridDim.x) {
            const int32_t e = (int32_t)(i / slabs);
            const int64_t col = (i - e * slabs) * 256 + lane * 4;
            const bool in = col < a.width;
            const int k = find_group(prefix, e);
            const int32_t v = uniform(a.longs[a.before[g0 + k] / (kEmbedChunk + 1) + (e - prefix[k])]);
            const int32_t off = uniform(a.offset[v]), n = uniform(a.offset[v + 1]) - off;
            const int32_t m = (n + kEmbedChunk - 1) / kEmbedChunk;
            int32_t range = 1;  // partial values per wave
            while (range * kFinishWaves < m) range *= 2;
            const int32_t lo = w * range, hi = lo + range < m ? lo + range : m;
            float acc[4];
            tree_partials<19>(a, off, m, lo, hi, in ? col : 0, acc);  // 2^30 / 64 / 8 / 8 batches
            waves[w][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
            __syncthreads();
            // wave w finishes its 256 / kFinishWaves columns, one a lane
            if (lane < 256 / kFinishWaves) {
                const int x = w * (256 / kFinishWaves) + lane;
                const int64_t at = (i - e * slabs) * 256 + x;
                float s[kFinishWaves];
#pragma unroll
                for (int j = 0; j < kFinishWaves; ++j)
                    s[j] = reinterpret_cast<const float*>(waves[j])[x];
#pragma unroll
                for (int d = 1; d < kFinishWaves; d *= 2)
#pragma unroll
                    for (int j = 0; j < kFinishWaves; j += 2 * d) s[j] += s[j + d];
                const float one[1] = {s[0]};
                if (at < a.width) store_grad<G, 1, true>(a, v, at, one, 0);
            }
            __syncthreads();
        }
    }
}

// f(V, AL): 16-byte accesses, at any alignment where rows are not aligned to
// that (16384 x 4095 bf16 rows: lookup 114 -> 41 us, gradient to 65536 float32
// rows 820 -> 340), or single elements where a row has fewer.
template <typename T, class F>
hipError_t with_access(bool aligned, int64_t width, F&& f)
{
    constexpr int V = 16 / (int)sizeof(typename T::store_t);
    if (aligned) return f(std::integral_constant<int, V>{}, std::true_type{});
    if (width >= V) return f(std::integral_constant<int, V>{}, std::false_type{});
    return f(std::integral_constant<int, 1>{}, std::true_type{});
}

template <typename T>
hipError_t launch_embedding(const EmbedArgs& a, hipStream_t st)
{
    return with_access<T>(a.vec, a.width, [&](auto v, auto al) {
        constexpr int V = decltype(v)::value;
        const int64_t n = a.tokens * ((a.width + V - 1) / V);
        static_assert(kEmbedGridAccesses == 4 * 256, "k_embedding: 4 a thread");
        k_embedding<T, V, decltype(al)::value>
            <<<dim3((unsigned)((n + kEmbedGridAccesses - 1) / kEmbedGridAccesses)), dim3(256), 0,
               st>>>(a);
        return hipGetLastError();
    });
}

inline OneShape one_shape(int64_t rows, int64_t slabs)
{
    OneShape s;
    s.parts = slabs < 16 ? (int)slabs : 16;
    // Groups are doubled up to 256 workgroups or down to 9 to 17 ids each, and on
    // until none has more than 512 ids, which may take more than 256 workgroups.
    s.log_groups = 0;
    while (((int64_t)2 * s.parts << s.log_groups) <= 256 && (rows >> s.log_groups) > 16)
        ++s.log_groups;
    while (s.log_groups < 24 && ((rows - 1) >> s.log_groups) + 1 > kOneIds) ++s.log_groups;
    s.ids = (int)(((rows - 1) >> s.log_groups) + 1);
    return s;
}

template <typename T, typename G>
hipError_t launch_embedding_grad(const EmbedGradArgs& a, hipStream_t st)
{
    return with_access<T>(a.vec, a.width, [&](auto v, auto al) {
        constexpr int V = decltype(v)::value;
        constexpr bool AL = decltype(al)::value;
        // four workgroups fit a compute unit (k_embed_sum's launch bound)
        const int64_t cus = (int64_t)device_cus(), cap = cus * 4;
        const int64_t slabs = (a.width + 64 * V - 1) / (64 * V);
        if (a.tokens <= kEmbedDirect) {
            const int64_t waves =
                a.tokens * slabs * (V > 1 ? 2 : 1) + (a.accumulate ? 0 : a.rows);
            const dim3 direct(
                (unsigned)capped_grid(waves < 4 ? 1 : waves / 4 < cap ? waves / 4 : cap));
            k_embed_direct<T, G, V == 1 ? 1 : V / 2, AL><<<direct, dim3(256), 0, st>>>(a);
            return hipGetLastError();
        }
        if (a.tokens <= kEmbedOne) {
            const OneShape one = one_shape(a.rows, slabs);
            const int64_t bytes = a.rows * a.width * (int64_t)sizeof(typename G::store_t);
            const bool spread = one.log_groups >= 4 && slabs < 8 && bytes <= (64 << 20);
            if (one.blocks() <= 512 && (spread || a.tokens <= 1024)) {
                k_embed_one<T, G, V, AL>
                    <<<dim3((unsigned)one.blocks()), dim3(64 * kGroupWaves),
                       (size_t)kGroupWaves * one.ids * sizeof(int32_t), st>>>(a, one);
                return hipGetLastError();
            }
        }
        const int64_t groups = id_groups(a.rows);
        if (hipError_t e = launch_embedding_group(a, st)) return e;
        const int64_t want = (a.tokens * slabs + (a.accumulate ? 0 : a.rows) + 3) / 4;
        const dim3 grid((unsigned)capped_grid(want < 1 ? 1 : want < cap ? want : cap));
        k_embed_sum<T, G, V, AL><<<grid, dim3(256), 0, st>>>(a, groups);
        if (hipError_t e = hipGetLastError()) return e;
        const int64_t most = a.tokens / (kEmbedChunk + 1) * ((a.width + 255) / 256);
        k_embed_finish<G><<<dim3((unsigned)capped_grid(most < cus ? most : cus)),
                            dim3(64 * kFinishWaves), 0, st>>>(a, groups);
        return hipGetLastError();
    });
}

}  // namespace seq
}  // namespace canon

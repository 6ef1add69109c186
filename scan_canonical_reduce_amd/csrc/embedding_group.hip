// Tokens grouped by id, in token order within an id (see embedding_impl.hpp).
#include "embedding.hpp"

namespace canon {
namespace seq {

namespace {

template <bool IDS64>
__device__ __forceinline__ int64_t id_at(const void* ids, int64_t t)
{
    return IDS64 ? static_cast<const int64_t*>(ids)[t]
                 : (int64_t) static_cast<const int32_t*>(ids)[t];
}

// R ids a workgroup (R <= 512); dynamic LDS: kGroupWaves x R counts.
template <bool IDS64>
__global__ __launch_bounds__(1024) void k_embed_group(EmbedGradArgs a, int R)
{
    extern __shared__ int32_t hist[];  // [wave][id]: count, then the next position
    __shared__ Pairs scan[kGroupWaves];
    __shared__ int32_t first_item[1025], first_token[1025];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int64_t b = blockIdx.x, lo = b * R;
    const int64_t hi = lo + R < a.rows ? lo + R : a.rows;
    for (int i = tid; i < kGroupWaves * R; i += 1024) hist[i] = 0;
    __syncthreads();

    // Each wave's stretch of the tokens, whole batches of 64.
    const int64_t per = ((a.tokens + kGroupWaves * 64 - 1) / (kGroupWaves * 64)) * 64;
    const int64_t t_lo = w * per < a.tokens ? w * per : a.tokens;
    const int64_t t_hi = t_lo + per < a.tokens ? t_lo + per : a.tokens;
    constexpr int U = 8;  // ids in flight per lane
    int64_t id[U];
    auto load = [&](int64_t t0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t t = t0 + u * 64 + lane;
            id[u] = t < t_hi ? id_at<IDS64>(a.ids, t) : -1;
        }
    };
    uint32_t below = 0;
    for (int64_t t0 = t_lo; t0 < t_hi; t0 += 64 * U) {
        load(t0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool real = id[u] >= 0 && id[u] < a.rows && id[u] != a.padding_id;
            below += real && id[u] < lo;
            if (real && id[u] >= lo && id[u] < hi)
                atomicAdd(&hist[w * R + (int)(id[u] - lo)], 1);
        }
    }
    __syncthreads();
    // thread r: the counts of id lo + r over the waves, in wave order
    int32_t n = 0;
    if (tid < R)
#pragma unroll
        for (int k = 0; k < kGroupWaves; ++k) {
            const int32_t c = hist[k * R + tid];
            hist[k * R + tid] = n;
            n += c;
        }
    const bool is_row = lo + tid < hi && tid < R;
    const int32_t chunks = (n + kEmbedChunk - 1) / kEmbedChunk;
    const int32_t items = is_row ? chunks : 0;
    const bool is_long = is_row && n > kEmbedChunk;
    uint64_t x = (uint64_t)(uint32_t)n | (uint64_t)(uint32_t)items << 32;
    uint64_t y = (uint64_t)is_long | (uint64_t)below << 32;
    const Pairs before = block_exclusive(x, y, scan);
    const uint64_t pos = before.x, both = x, long_pos = (uint32_t)before.y;
    const int64_t all_below = (int64_t)(y >> 32);
    const int32_t off = (int32_t)all_below + (int32_t)(uint32_t)pos;
    const int32_t item = (int32_t)(pos >> 32), n_items = (int32_t)(both >> 32);
    if (tid < R)
#pragma unroll
        for (int k = 0; k < kGroupWaves; ++k) hist[k * R + tid] += off;
    if (is_row) {
        a.offset[lo + tid] = off;
        if (lo + tid == a.rows - 1) a.offset[a.rows] = off + n;
    }
    // entries of rows >= kEmbedChunk + 1 tokens long, from before / 65 on
    if (is_long) a.longs[all_below / (kEmbedChunk + 1) + long_pos] = (int32_t)(lo + tid);
    first_item[tid] = item;
    first_token[tid] = off;
    if (tid == 0) {
        first_item[1024] = n_items;
        first_token[1024] = (int32_t)all_below + (int32_t)(uint32_t)both;
        a.n_items[b] = n_items;
        a.n_long[b] = (int32_t)(uint32_t)y;
        a.before[b] = (int32_t)all_below;
    }
    __syncthreads();
    // the list of work, from the tokens before this group on
    int4* list = a.items + all_below;
    for (int32_t i = tid; i < n_items; i += 1024) {
        int r0 = 0, r1 = 1023;  // the last id with first_item <= i
        while (r0 < r1) {
            const int mid = (r0 + r1 + 1) >> 1;
            if (first_item[mid] <= i)
                r0 = mid;
            else
                r1 = mid - 1;
        }
        list[i] = make_int4((int32_t)(lo + r0), i - first_item[r0], first_token[r0],
                            first_token[r0 + 1] - first_token[r0]);
    }

    // Placing: a wave's lanes with the same id take consecutive positions.  Ids of
    // a stretch of one batch are still in registers.
    for (int64_t t0 = t_lo; t0 < t_hi; t0 += 64 * U) {
        if (per > 64 * U) load(t0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            bool todo = id[u] >= lo && id[u] < hi && id[u] != a.padding_id;
            const int key = todo ? (int)(id[u] - lo) : -1;
            uint64_t left = __ballot(todo);
            while (left) {
                const int lead = __builtin_amdgcn_readlane(key, __builtin_ctzll(left));
                const uint64_t same = __ballot(key == lead);
                if (key == lead) {
                    const int rank = __popcll(same & ((1ull << lane) - 1));
                    const int32_t at = hist[w * R + lead];
                    a.order[at + rank] = (int32_t)(t0 + u * 64 + lane);
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
                if (lane == 0) hist[w * R + lead] += __popcll(same);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
                left &= ~same;
            }
        }
    }
}

}  // namespace

hipError_t launch_embedding_group(const EmbedGradArgs& a, hipStream_t st)
{
    const int R = (int)ids_per_group(a.rows);
    const dim3 grid((unsigned)id_groups(a.rows)), block(1024);
    const size_t lds = (size_t)kGroupWaves * R * sizeof(int32_t);
    if (a.ids64)
        k_embed_group<true><<<grid, block, lds, st>>>(a, R);
    else
        k_embed_group<false><<<grid, block, lds, st>>>(a, R);
    return hipGetLastError();
}

}  // namespace seq
}  // namespace canon

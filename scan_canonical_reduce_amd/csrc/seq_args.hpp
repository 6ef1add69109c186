// Argument checks and workspace layout that the C ABI's operators on sequences
// share (canon_seq.h, canon_layer.h).
#pragma once

#include "api_impl.hpp"
#include "seq_device.hpp"

namespace canon {
namespace seq {

inline size_t elem_bytes(int64_t dtype) { return dtype == CANON_F32 ? 4 : 2; }
inline bool is_dtype(int64_t d) { return d == CANON_F32 || d == CANON_BF16 || d == CANON_F16; }

// Launches are one-dimensional: fewer than 2^32 threads.  Row counts fit
// 32-bit indexes with room for a chunk; partial sums are kept below 2^47
// elements so that no size overflows.
constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int64_t kMaxGrid256 = (int64_t)1 << 24;

inline bool mul_fits(int64_t a, int64_t b, int64_t limit) { return a == 0 || b <= limit / a; }

template <class F>
inline canon_status_t with_dtype(int64_t dtype, F&& f)
{
    switch (dtype) {
        case CANON_F32: return f(F32{});
        case CANON_BF16: return f(BF16{});
        case CANON_F16: return f(F16{});
        default: return CANON_EINVAL;
    }
}

// Vectors of `bytes` at every row of r: base and strides.
inline bool rows_aligned(const canon_rows_t& r, size_t es, size_t bytes, bool one_row)
{
    if (r.p == nullptr) return true;
    const bool row_ok = one_row || (size_t)r.row * es % bytes == 0;
    return (uintptr_t)r.p % bytes == 0 && row_ok && (size_t)r.seq * es % bytes == 0;
}

inline bool ptr_aligned(const void* p, size_t bytes) { return (uintptr_t)p % bytes == 0; }

inline bool rows_valid(const canon_rows_t& r) { return r.p != nullptr && r.row >= 0 && r.seq >= 0; }
// rows of an output: no two may share elements, whether a sequence's rows lie
// together or the sequences are interleaved
inline bool out_valid(const canon_rows_t& r, int64_t cols, int64_t seqs, int64_t rows)
{
    if (!rows_valid(r)) return false;
    if (rows > 1 && r.row < cols) return false;
    if (seqs <= 1) return true;
    if (r.seq < cols) return false;
    return rows <= 1 || (r.seq - cols) / (rows - 1) >= r.row ||
           (r.row - cols) / (seqs - 1) >= r.seq;
}

// Bump allocation in the workspace.
struct Layout {
    size_t bytes = 0;
    size_t take(size_t n)
    {
        const size_t at = bytes;
        bytes += abi::round_up(n, 256);
        return at;
    }
    template <typename T>
    static T* at(void* ws, size_t off)
    {
        return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
    }
};

// Sizes that every kernel can index and launch.
inline canon_status_t seq_sizes(int64_t seqs, int64_t rows, int64_t channels, bool packed)
{
    if (seqs < 0 || rows < 0 || channels < 0) return CANON_EINVAL;
    if (rows >= kMaxRows || seqs >= kMaxRows || channels >= (1 << 24)) return CANON_EUNSUPPORTED;
    const int64_t slots = slot_count<8>(seqs, rows, packed);
    if (!mul_fits(slots, channels, (int64_t)1 << 40)) return CANON_EUNSUPPORTED;
    return CANON_OK;
}

}  // namespace seq
}  // namespace canon

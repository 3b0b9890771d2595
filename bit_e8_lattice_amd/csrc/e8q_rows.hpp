// Rows of logits: loads, stores and the split of few rows over blocks, shared
// by the operators on them.
#pragma once

#include "e8q_device.hpp"
#include "e8q_host.hpp"
#include "e8q_vec.hpp"

namespace e8q {

constexpr int kLpBlock = 256;         // threads per row, or per part of a row
constexpr int kLpWide = 1024;         // threads per row of the two-pass gradient
constexpr int kLpUnroll = 4;          // vectors in flight per thread
constexpr int kMaxSplits = 256;
constexpr int64_t kMaxRows = int64_t(1) << 24;   // a block of kLpBlock per row, fewer than 2^32 threads
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// A row as vectors of 16 bytes from its first element, whatever its alignment
// (gfx950 loads and stores dwordx4 at any element), so that the order of the
// sums does not depend on where a tensor lies.
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) RowVec {
    u32x4_t v;
};

template <typename T>
__device__ __forceinline__ void load_logits(const T* row, uint32_t vocab, uint32_t j, float (&v)[kVec<T>]) {
    constexpr int VE = kVec<T>;
    const uint32_t e0 = j * VE;
    if (e0 + VE <= vocab) {
        unpack(reinterpret_cast<const RowVec<T>*>(row + e0)->v, v);
    } else {
#pragma unroll
        for (int i = 0; i < VE; ++i) v[i] = e0 + i < vocab ? widen(row[e0 + i]) : -INFINITY;
    }
}

template <typename T>
__device__ __forceinline__ void store_grad(T* dx, uint32_t vocab, uint32_t e0, const float (&d)[kVec<T>]) {
    if (e0 + kVec<T> <= vocab) {
        // past the caches: it would push the rows' logits out, which are read again
        __builtin_nontemporal_store(pack(d), &reinterpret_cast<RowVec<T>*>(dx + e0)->v);
    } else {
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i)
            if (e0 + i < vocab) dx[e0 + i] = narrow<T>(d[i]);
    }
}

// Blocks per row: enough blocks for every CU to hold about four, each with
// kLpUnroll vectors a thread to read (one row of 131072 bf16 logits with 8
// alternatives: 14.4 us with 16 parts, 14.7 with 32, 16.4 with 32 joined by 1024
// threads).
inline uint32_t lp_splits(int64_t rows, int64_t vocab, size_t esz, uint32_t& per_split) {
    const uint64_t ve = 16 / esz, nvec = (uint64_t(vocab) + ve - 1) / ve;
    const uint64_t want = (uint64_t(device_cu_count()) * 4 + uint64_t(rows) - 1) / uint64_t(rows);
    const uint64_t most = (nvec + kLpBlock * kLpUnroll - 1) / (kLpBlock * kLpUnroll);
    uint64_t n = want < most ? want : most;
    if (n > kMaxSplits) n = kMaxSplits;
    if (n < 1) n = 1;
    per_split = uint32_t((nvec + n - 1) / n);
    return uint32_t((nvec + per_split - 1) / per_split);
}

}  // namespace e8q

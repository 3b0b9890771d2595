// e8q_adjust_logits: what a server does to a row of logits before a token is
// chosen from it.  With c_i the occurrences of token i among the row's made tokens
// and b_i the sum of its biases,
//   x' = x / r (x > 0) or x r        where i is in the history (prompt or made),
//   x'' = x' - (f c_i + p [c_i > 0]),   x''' = x'' + b_i,
//   out = x''' where the mask's bit is set, -inf where not (whatever x is).
//
// A block has a part of a row, and a word in LDS for each of its elements: the
// count, a bit for "in the history", a bit for "has a bias".  Its threads load their vectors
// of the part, and the first of the row's history, before anything is waited for; then
// the whole history is read (from L2: the row's other blocks read it too) and the ids of
// the part are counted with LDS atomics on integers, whose result does not depend on their
// order.  A vector whose words are all zero is copied; one that the mask empties is
// written without being read; in place, one that nothing touches is not met at all.
// Few elements are touched (2048 ids in a vocabulary of 131072), so a lane takes its
// touched elements one by one: all elements of every vector with a touched one, the wave
// through, made the arithmetic the bound (512 rows of 131072 bf16 logits with 2048 ids,
// biases and a mask: 81.5 us so, 70 one by one).  Biases of the part are
// chained in LDS by their elements; a lane walks the chain of its own, and the wave walks
// all of them together for an element that has very many (483 rows of 930 tokens, 300
// biases each: 218 us with the wave for every element, 18).  Several of one element
// are added in the order of their places.
//
// The bound is memory: logits in and out, history and mask are 60 us of the 70 at a
// large copy's rate.  One row takes 5 us, the wait for its length, its ids and its logits in turn.  In place, touched
// vectors are loaded after the history is counted: as fast with a mask that touches most of them (70.5 us a call, 69 out
// of place) as without one (71.6, 72.7).
#include <float.h>

#include "e8q_rows.hpp"

namespace e8q {

constexpr int64_t kMaxBias = 1024;
constexpr uint32_t kSeen = 0x80000000u, kBiased = 0x40000000u, kCount = 0x3FFFFFFFu;

struct AdjArgs {
    const void* x;
    int64_t stride;
    void* out;
    int64_t out_stride;
    uint32_t rows, vocab;
    const void* hist;
    int64_t hist_stride;
    uint32_t hist_cap;
    const int32_t* hist_len;
    const int32_t* prompt_len;
    const float* rep;
    const float* freq;
    const float* pres;
    const void* bias_idx;
    const float* bias;
    int64_t bias_stride;
    uint32_t n_bias;
    int i64;
    const uint32_t* mask;
    int64_t mask_stride;
    uint32_t chunk, chunks;     // elements of a block's part, parts of a row
    uint32_t* status;
};

__device__ __forceinline__ int64_t id_at(const void* p, int i64, int64_t i) {
    return i64 ? static_cast<const int64_t*>(p)[i] : int64_t(static_cast<const int32_t*>(p)[i]);
}

// x / r for positive x and r from inv = fl(1 / r'), r' = r up: correctly rounded where x is above 2^-100 (the
// remainder is exact).  up is a power of two that takes r' to where its reciprocal is a normal number, 0 for an infinite r.
struct Divisor {
    float r, inv, up;
};

__device__ __forceinline__ Divisor divisor(float r) {
    const float up = r < 0x1p-64f ? 0x1p64f : r > 0x1p64f ? 0x1p-64f : 1.0f;
    const float to = r * up > FLT_MAX ? FLT_MAX : r * up;      // (a NaN stays one)
    return {to, 1.0f / to, __builtin_isinf(r) ? 0.0f : up};
}

__device__ __forceinline__ float divide(float x, const Divisor& d) {
    const float q = x * d.inv;
    return (__builtin_isinf(q) ? q : fmaf(fmaf(-q, d.r, x), d.inv, q)) * d.up;
}

// Biases of a part, each in the slot of its place in the row's list: chains of slots by the
// element's low bits.  A node is the element (kNoElement: not of this part) and the next
// slot + 1 << 16.
struct BiasList {
    uint32_t* head;
    uint32_t* node;
    float* value;
    uint32_t n;
};
constexpr uint32_t kHeads = 1024, kNoElement = 0xFFFFu, kChain = 16;

// The sum of the element's biases in the order of their places, by its own lane; false: its chain is
// longer than kChain.
__device__ __forceinline__ bool bias_short(const BiasList& l, uint32_t local, float& sum) {
    const uint32_t first = l.head[local % kHeads];
    uint32_t at = first, m = 0u, one = 0u;
    for (uint32_t steps = 0u; at && steps < kChain; ++steps) {
        const uint32_t q = l.node[at - 1u];
        if ((q & 0xFFFFu) == local) {
            one = at - 1u;
            ++m;
        }
        at = q >> 16;
    }
    if (at) return false;
    sum = 0.0f;
    if (m == 1u) sum += l.value[one];
    for (uint32_t next = 0u; m > 1u && next < l.n;) {
        uint32_t best = l.n;
        for (at = first; at;) {
            const uint32_t q = l.node[at - 1u];
            if ((q & 0xFFFFu) == local && at - 1u >= next) best = min(best, at - 1u);
            at = q >> 16;
        }
        if (best < l.n) sum += l.value[best];
        next = best + 1u;
    }
    return true;
}

// The same by the whole wave, over all slots.
__device__ __forceinline__ float bias_long(const BiasList& l, uint32_t local, uint32_t lane) {
    float sum = 0.0f;
    for (uint32_t base = 0u; base < l.n; base += kWave) {
        const uint32_t j = base + lane;
        const float v = j < l.n ? l.value[j] : 0.0f;
        uint64_t who = __ballot(j < l.n && (l.node[min(j, l.n - 1u)] & 0xFFFFu) == local);
        while (who) {
            const int src = __ffsll((unsigned long long)who) - 1;
            who &= who - 1ull;
            sum += __uint_as_float(uint32_t(__builtin_amdgcn_readlane(int(__float_as_uint(v)), src)));
        }
    }
    return sum;
}

// Element i of a vector, i known at run time only.
template <typename T>
__device__ __forceinline__ float element(const u32x4_t& raw, uint32_t i) {
    const uint32_t k = sizeof(T) == 2 ? i >> 1 : i;
    const uint32_t r0 = raw[0], r1 = raw[1], r2 = raw[2], r3 = raw[3];
    const uint32_t r = k & 2u ? (k & 1u ? r3 : r2) : (k & 1u ? r1 : r0);
    if constexpr (sizeof(T) == 4) return __uint_as_float(r);
    return __uint_as_float(i & 1u ? r & 0xFFFF0000u : r << 16);
}

template <typename T>
__device__ __forceinline__ void put_element(u32x4_t& raw, uint32_t i, float y) {
#pragma unroll
    for (uint32_t k = 0u; k < 4u; ++k) {
        const uint32_t r = raw[k];
        if constexpr (sizeof(T) == 4) {
            raw[k] = i == k ? __float_as_uint(y) : r;
        } else {
            const uint32_t h = narrow<T>(y), with = i & 1u ? (r & 0xFFFFu) | h << 16 : (r & 0xFFFF0000u) | h;
            raw[k] = i >> 1 == k ? with : r;
        }
    }
}

// -inf where the mask has no bit.
template <typename T>
__device__ __forceinline__ u32x4_t masked(const u32x4_t& raw, uint32_t bits) {
    u32x4_t o;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t r = raw[k];
        if constexpr (sizeof(T) == 4) {
            o[k] = (bits >> k) & 1u ? r : 0xFF800000u;
        } else {
            const uint32_t keep = ((bits >> (2 * k)) & 1u ? 0xFFFFu : 0u) | ((bits >> (2 * k + 1)) & 1u ? 0xFFFF0000u : 0u);
            o[k] = (r & keep) | (0xFF80FF80u & ~keep);
        }
    }
    return o;
}

// A thread has kAdjElements of the part, as vectors that it loads before the history is
// read: their latency and the history's are one.
constexpr int kAdjElements = 16;

template <typename T, int BLOCK, bool TABLE>
__global__ __launch_bounds__(BLOCK) void adjust_kernel(AdjArgs a) {
    constexpr int VE = kVec<T>, NV = kAdjElements / VE;
    constexpr uint32_t kFull = (1u << VE) - 1u;
    extern __shared__ uint4 s_adjust[];
    const uint32_t tid = threadIdx.x, lane = tid & 63u;
    const uint32_t row = blockIdx.x / a.chunks, part = blockIdx.x - row * a.chunks;
    const uint32_t lo = part * a.chunk, n = min(a.chunk, a.vocab - lo);
    const T* x = static_cast<const T*>(a.x) + int64_t(row) * a.stride + lo;
    T* out = static_cast<T*>(a.out) + int64_t(row) * a.out_stride + lo;
    uint32_t* word = reinterpret_cast<uint32_t*>(s_adjust);
    const BiasList list = {word + a.chunk, word + a.chunk + kHeads,
                           reinterpret_cast<float*>(word + a.chunk + kHeads + a.n_bias), a.n_bias};
    const uint32_t* mask = a.mask ? a.mask + int64_t(row) * a.mask_stride : nullptr;
    const bool in_place = a.out == a.x;
    const uint32_t nvec = (n + VE - 1u) / VE;
    // the mask's bits of the thread's vectors; none where there is no vector
    uint32_t bits[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const uint32_t j = u * BLOCK + tid, e = lo + j * VE;
        bits[u] = j >= nvec ? 0u : mask ? (mask[e >> 5] >> (e & 31u)) & kFull : kFull;
    }
    u32x4_t raw[NV];
    const auto load = [&](int u) {
        const uint32_t e0 = (u * BLOCK + tid) * VE;
        if (e0 + VE <= n) {
            raw[u] = reinterpret_cast<const RowVec<T>*>(x + e0)->v;
        } else {
            float v[VE];
#pragma unroll
            for (int i = 0; i < VE; ++i) v[i] = e0 + i < n ? widen(x[e0 + i]) : 0.0f;
            raw[u] = pack(v);
        }
    };
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        raw[u] = u32x4_t{0u, 0u, 0u, 0u};
        if (bits[u] != 0u && !in_place) load(u);
    }
    float rep = 1.0f, freq = 0.0f, pres = 0.0f;
    Divisor by = {1.0f, 1.0f, 1.0f};
    if constexpr (TABLE) {
        constexpr int kIds = 2;                 // places in flight per thread
        const int64_t hrow = int64_t(row) * a.hist_stride;
        int64_t id[kIds];
        // the first ids before the length is known: they are in the tensor
#pragma unroll
        for (int u = 0; u < kIds; ++u) {
            const int64_t j = u * BLOCK + int64_t(tid);
            id[u] = j < int64_t(a.hist_cap) ? id_at(a.hist, a.i64, hrow + j) : -1;
        }
        for (uint32_t i = tid; i < (n + 7u) / 8u * 2u; i += BLOCK) s_adjust[i] = make_uint4(0u, 0u, 0u, 0u);
        if (a.n_bias)
            for (uint32_t i = tid; i < kHeads; i += BLOCK) list.head[i] = 0u;
        uint32_t flags = 0u;
        int64_t len = 0, prompt = 0;
        if (a.hist) {
            len = a.hist_len ? a.hist_len[row] : int64_t(a.hist_cap);
            len = min(len, int64_t(a.hist_cap));
            prompt = a.prompt_len ? max(a.prompt_len[row], 0) : 0;
            if (a.rep) rep = a.rep[row];
            if (a.freq) freq = a.freq[row];
            if (a.pres) pres = a.pres[row];
            by = divisor(rep);
        }
        __syncthreads();
        // a prompt counts for the repetition penalty only
        const int64_t from = a.rep ? 0 : prompt;
        for (int64_t base = 0; base < len; base += kIds * BLOCK) {
#pragma unroll
            for (int u = 0; u < kIds; ++u) {
                const int64_t j = base + u * BLOCK + int64_t(tid);
                if (base > 0) id[u] = j < len ? id_at(a.hist, a.i64, hrow + j) : -1;
            }
#pragma unroll
            for (int u = 0; u < kIds; ++u) {
                const int64_t j = base + u * BLOCK + int64_t(tid);
                // (512 rows of 131072 with 2048 ids: 76 us so, 102 where the check stands between the two ends of the next)
                if (j < len && id[u] >= int64_t(a.vocab)) flags |= E8Q_STATUS_BAD_INDEX;
                if (j < from || j >= len) continue;
                const int64_t e = id[u] - int64_t(lo);
                if (id[u] < 0 || e < 0 || e >= int64_t(n)) continue;
                if (j < prompt) atomicOr(&word[e], kSeen);
                else atomicAdd(&word[e], 1u);
            }
        }
        for (uint32_t j = tid; j < a.n_bias; j += BLOCK) {
            const int64_t at = int64_t(row) * a.bias_stride + j, t = id_at(a.bias_idx, a.i64, at);
            if (t >= int64_t(a.vocab)) flags |= E8Q_STATUS_BAD_INDEX;
            const int64_t e = t - int64_t(lo);
            const bool here = t >= 0 && e >= 0 && e < int64_t(n);
            uint32_t node = kNoElement;
            if (here) {
                atomicOr(&word[e], kBiased);
                node = uint32_t(e) | atomicExch(&list.head[uint32_t(e) % kHeads], j + 1u) << 16;
                list.value[j] = a.bias[at];
            }
            list.node[j] = node;
        }
        flush_status(flags, a.status);
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const uint32_t j = u * BLOCK + tid, e0 = j * VE;
        uint32_t left = 0u;                      // touched elements of the vector
        if constexpr (TABLE) {
            if (j < nvec) {
                uint32_t w[VE], any = 0u;
#pragma unroll
                for (int i = 0; i < VE; i += 4) {
                    const uint4 q = s_adjust[(e0 + i) / 4u];
                    w[i] = q.x;
                    w[i + 1] = q.y;
                    w[i + 2] = q.z;
                    w[i + 3] = q.w;
                }
#pragma unroll
                for (int i = 0; i < VE; ++i) any |= w[i];
                if (any) {
#pragma unroll
                    for (int i = 0; i < VE; ++i) left |= w[i] ? 1u << i : 0u;
                }
            }
        }
        const bool write = j < nvec && !(in_place && left == 0u && bits[u] == kFull);
        if (in_place && write && bits[u] != 0u) load(u);
        if constexpr (TABLE) {
            left &= bits[u];
            while (__ballot(left != 0u)) {
                // every lane its lowest one
                const uint32_t i0 = left ? uint32_t(__ffs(int(left)) - 1) : 0u, local = e0 + i0;
                const uint32_t w = left ? word[local] : 0u, c = w & kCount;
                float y = element<T>(raw[u], i0);
                if (w & ~kBiased) y = y > 0.0f ? divide(y, by) : y * rep;
                if (c) y -= freq * float(c) + pres;
                if (__ballot((w & kBiased) != 0u)) {
                    float b = 0.0f;
                    uint64_t who = __ballot((w & kBiased) && !bias_short(list, local, b));
                    while (who) {
                        const int src = __ffsll((unsigned long long)who) - 1;
                        who &= who - 1ull;
                        const float all = bias_long(list, uint32_t(__builtin_amdgcn_readlane(int(local), src)), lane);
                        if (lane == uint32_t(src)) b = all;
                    }
                    if (w & kBiased) y += b;
                }
                if (left) put_element<T>(raw[u], i0, y);
                left &= left - 1u;
            }
        }
        if (!write) continue;
        if (mask) raw[u] = masked<T>(raw[u], bits[u]);
        if (e0 + VE <= n) {
            __builtin_nontemporal_store(raw[u], &reinterpret_cast<RowVec<T>*>(out + e0)->v);
        } else {
            float v[VE];
            unpack(raw[u], v);
#pragma unroll
            for (int i = 0; i < VE; ++i)
                if (e0 + i < n) out[e0 + i] = narrow<T>(v[i]);
        }
    }
}

// Elements of a block's part: as many as leave two blocks' words in LDS, fewer where there would be less than two
// blocks a CU.
static uint32_t adjust_chunk(int64_t rows, int64_t vocab) {
    uint32_t chunk = 16384;
    while (chunk > 512 && chunk / 2 >= uint64_t(vocab)) chunk /= 2;
    while (chunk > 2048 && uint64_t(rows) * ((uint64_t(vocab) + chunk - 1) / chunk) < 2u * uint64_t(device_cu_count()))
        chunk /= 2;
    return chunk;
}

static uint32_t adjust_threads(uint32_t chunk) { return chunk > 4096 ? 1024u : 256u; }
static_assert(1024 * kAdjElements >= 16384 && 256 * kAdjElements >= 4096, "a block's threads hold its part");

template <typename T, bool TABLE>
static void adjust_launch(const AdjArgs& a, hipStream_t st) {
    const size_t lds = TABLE ? size_t(a.chunk) * 4 + (a.n_bias ? size_t(kHeads) * 4 + size_t(a.n_bias) * 8 : 0) : 0;
    const dim3 grid(a.rows * a.chunks);
    if (adjust_threads(a.chunk) == 1024u) launch(adjust_kernel<T, 1024, TABLE>, grid, dim3(1024), lds, st, a);
    else launch(adjust_kernel<T, 256, TABLE>, grid, dim3(256), lds, st, a);
}

}  // namespace e8q

extern "C" e8q_status_t e8q_adjust_logits(const void* logits, e8q_dtype_t dtype, int64_t rows, int64_t vocab,
                                          int64_t row_stride, e8q_index_t index_type, const void* history,
                                          int64_t history_cols, int64_t history_stride, const int32_t* history_len,
                                          const int32_t* prompt_len, const float* repetition, const float* frequency,
                                          const float* presence, const void* bias_idx, const float* bias,
                                          int64_t n_bias, int64_t bias_stride, const uint32_t* mask,
                                          int64_t mask_stride, void* out, int64_t out_stride, uint32_t* status_dev,
                                          void* stream) {
    using namespace e8q;
    if (!logits || !out || !status_dev || rows <= 0 || vocab <= 0 || row_stride < vocab || out_stride < vocab)
        return E8Q_ERR_INVALID;
    if (dtype != E8Q_F32 && dtype != E8Q_BF16) return E8Q_ERR_INVALID;
    if (index_type != E8Q_I32 && index_type != E8Q_I64) return E8Q_ERR_INVALID;
    const size_t esz = dtype == E8Q_BF16 ? 2 : 4, isz = index_type == E8Q_I64 ? 8 : 4;
    const auto off = [](const void* p, size_t unit) { return reinterpret_cast<uintptr_t>(p) % unit != 0; };
    if (off(logits, esz) || off(out, esz) || off(history, isz) || off(bias_idx, isz) || off(bias, 4) || off(mask, 4) ||
        off(history_len, 4) || off(prompt_len, 4) || off(repetition, 4) || off(frequency, 4) || off(presence, 4))
        return E8Q_ERR_INVALID;
    if (out == logits && out_stride != row_stride) return E8Q_ERR_INVALID;
    const bool penalties = repetition || frequency || presence;
    if (penalties != (history != nullptr)) return E8Q_ERR_INVALID;
    if (history && (history_cols <= 0 || history_stride < history_cols)) return E8Q_ERR_INVALID;
    if (!history && (history_len || prompt_len)) return E8Q_ERR_INVALID;
    if (n_bias < 0 || (n_bias > 0) != (bias_idx != nullptr) || (n_bias > 0) != (bias != nullptr)) return E8Q_ERR_INVALID;
    if (n_bias > 0 && bias_stride != 0 && bias_stride < n_bias) return E8Q_ERR_INVALID;
    if (mask && mask_stride != 0 && mask_stride < (vocab + 31) / 32) return E8Q_ERR_INVALID;
    if (vocab >= (int64_t(1) << 31) - 16 || rows >= kMaxRows || n_bias > kMaxBias ||
        (history && history_cols >= int64_t(kCount)))
        return E8Q_ERR_UNSUPPORTED;
    for (const int64_t s : {row_stride, out_stride, history_stride, bias_stride, mask_stride})
        if (s >= (int64_t(1) << 40)) return E8Q_ERR_UNSUPPORTED;
    AdjArgs a{};
    a.chunk = adjust_chunk(rows, vocab);
    a.chunks = uint32_t((uint64_t(vocab) + a.chunk - 1) / a.chunk);
    // a launch has fewer than 2^32 threads
    if (uint64_t(rows) * a.chunks * adjust_threads(a.chunk) >= uint64_t(1) << 32) return E8Q_ERR_UNSUPPORTED;
    a.x = logits;
    a.stride = row_stride;
    a.out = out;
    a.out_stride = out_stride;
    a.rows = uint32_t(rows);
    a.vocab = uint32_t(vocab);
    a.hist = history;
    a.hist_stride = history_stride;
    a.hist_cap = history ? uint32_t(history_cols) : 0u;
    a.hist_len = history_len;
    a.prompt_len = prompt_len;
    a.rep = repetition;
    a.freq = frequency;
    a.pres = presence;
    a.bias_idx = bias_idx;
    a.bias = bias;
    a.bias_stride = bias_stride;
    a.n_bias = uint32_t(n_bias);
    a.i64 = index_type == E8Q_I64;
    a.mask = mask;
    a.mask_stride = mask_stride;
    a.status = status_dev;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const bool table = history || n_bias > 0;
    if (dtype == E8Q_BF16) table ? adjust_launch<uint16_t, true>(a, s) : adjust_launch<uint16_t, false>(a, s);
    else table ? adjust_launch<float, true>(a, s) : adjust_launch<float, false>(a, s);
    return launch_status();
}

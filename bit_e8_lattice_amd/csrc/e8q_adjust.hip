// e8q_adjust_logits: what a server does to a row of logits before a token is
// chosen from it.  With c_i the occurrences of token i among the row's made tokens
// and b_i the sum of its biases,
//   x' = x / r (x > 0) or x r        where i is in the history (prompt or made),
//   x'' = x' - (f c_i + p [c_i > 0]),   x''' = x'' + b_i,
//   out = x''' where the mask's bit is set, -inf where not (whatever x is).
//
// A block has a part of a row, and a word in LDS for each of its elements: the
// count, a bit for "in the history", a bit for "has a bias".  It reads the whole history
// of the row (from L2: the row's other blocks read it too) and counts the ids of
// its part with LDS atomics on integers, whose result does not depend on their order.  Then
// it streams its part.  A vector whose words are all zero is copied; one that the
// mask empties is written without being read; in place, one that nothing touches
// is not met at all.  Biases of the part are listed in LDS, and the wave looks a
// biased element up together; several of one element are added in the order of
// their places.
//
// The bound is memory: the logits in and out.
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

// x / r, correctly rounded but for subnormal results: inv = fl(1 / r).
__device__ __forceinline__ float divide(float x, float r, float inv) {
    const float q = x * inv;
    return __builtin_isinf(q) ? q : fmaf(fmaf(-q, r, x), inv, q);
}

// Biases of a part: element | place << 16 and value, `n` of them, in any order.
struct BiasList {
    uint32_t* key;
    float* value;
    uint32_t* n;
};

// The sum of the element's biases in the order of their places, by the whole wave.
__device__ __forceinline__ float bias_of(const BiasList& l, uint32_t local, uint32_t lane) {
    float sum = 0.0f;
    uint32_t next = 0u;                                // places below are added
    for (;;) {
        uint32_t best = 0xFFFFFFFFu;
        float v = 0.0f;
        for (uint32_t j = lane; j < *l.n; j += kWave) {
            const uint32_t key = l.key[j], place = key >> 16;
            if ((key & 0xFFFFu) == local && place >= next && place < best) {
                best = place;
                v = l.value[j];
            }
        }
        uint32_t first = best;
        first = min(first, lane_xor<32>(first));
        first = min(first, lane_xor<16>(first));
        first = min(first, lane_xor<8>(first));
        first = min(first, lane_xor<4>(first));
        first = min(first, lane_xor<2>(first));
        first = min(first, lane_xor<1>(first));
        if (first == 0xFFFFFFFFu) return sum;
        const int src = __ffsll((unsigned long long)__ballot(best == first)) - 1;
        sum += __uint_as_float(uint32_t(__builtin_amdgcn_readlane(int(__float_as_uint(v)), src)));
        next = first + 1u;
    }
}

template <typename T, int BLOCK, bool TABLE>
__global__ __launch_bounds__(BLOCK) void adjust_kernel(AdjArgs a) {
    constexpr int VE = kVec<T>;
    extern __shared__ uint4 s_adjust[];
    __shared__ uint32_t s_n;
    const uint32_t tid = threadIdx.x, lane = tid & 63u;
    const uint32_t row = blockIdx.x / a.chunks, part = blockIdx.x - row * a.chunks;
    const uint32_t lo = part * a.chunk, n = min(a.chunk, a.vocab - lo);
    const T* x = static_cast<const T*>(a.x) + int64_t(row) * a.stride + lo;
    T* out = static_cast<T*>(a.out) + int64_t(row) * a.out_stride + lo;
    uint32_t* word = reinterpret_cast<uint32_t*>(s_adjust);
    const BiasList list = {word + a.chunk, reinterpret_cast<float*>(word + a.chunk + a.n_bias), &s_n};
    float rep = 1.0f, inv = 1.0f, freq = 0.0f, pres = 0.0f;
    if constexpr (TABLE) {
        for (uint32_t i = tid; i < (n + 7u) / 8u * 2u; i += BLOCK) s_adjust[i] = make_uint4(0u, 0u, 0u, 0u);
        if (tid == 0u) s_n = 0u;
        uint32_t flags = 0u;
        int64_t len = 0, prompt = 0;
        if (a.hist) {
            len = a.hist_len ? a.hist_len[row] : int64_t(a.hist_cap);
            len = min(len, int64_t(a.hist_cap));
            prompt = a.prompt_len ? max(a.prompt_len[row], 0) : 0;
            if (a.rep) rep = a.rep[row];
            if (a.freq) freq = a.freq[row];
            if (a.pres) pres = a.pres[row];
            inv = 1.0f / rep;
        }
        __syncthreads();
        const int64_t hrow = int64_t(row) * a.hist_stride;
        // a prompt counts for the repetition penalty only
        for (int64_t j = (a.rep ? 0 : prompt) + tid; j < len; j += BLOCK) {
            const int64_t id = id_at(a.hist, a.i64, hrow + j);
            if (id >= int64_t(a.vocab)) flags |= E8Q_STATUS_BAD_INDEX;
            const int64_t e = id - int64_t(lo);
            if (id < 0 || e < 0 || e >= int64_t(n)) continue;
            if (j < prompt) atomicOr(&word[e], kSeen);
            else atomicAdd(&word[e], 1u);
        }
        for (uint32_t j = tid; j < a.n_bias; j += BLOCK) {
            const int64_t at = int64_t(row) * a.bias_stride + j, id = id_at(a.bias_idx, a.i64, at);
            if (id >= int64_t(a.vocab)) flags |= E8Q_STATUS_BAD_INDEX;
            const int64_t e = id - int64_t(lo);
            if (id < 0 || e < 0 || e >= int64_t(n)) continue;
            atomicOr(&word[e], kBiased);
            const uint32_t k = atomicAdd(&s_n, 1u);
            list.key[k] = uint32_t(e) | (j << 16);
            list.value[k] = a.bias[at];
        }
        flush_status(flags, a.status);
        __syncthreads();
    }
    const uint32_t* mask = a.mask ? a.mask + int64_t(row) * a.mask_stride : nullptr;
    const bool in_place = a.out == a.x;
    const uint32_t nvec = (n + VE - 1u) / VE;
    // whole waves: biased elements are looked up by all lanes
    for (uint32_t base = 0u; base < nvec; base += BLOCK) {
        const uint32_t j = base + tid, e0 = j * VE;
        const bool mine = j < nvec;
        uint32_t bits = (1u << VE) - 1u, w[VE], any = 0u;
        if (mask && mine) bits = (mask[(lo + e0) >> 5] >> ((lo + e0) & 31u)) & ((1u << VE) - 1u);
#pragma unroll
        for (int i = 0; i < VE; ++i) w[i] = 0u;
        if constexpr (TABLE) {
            if (mine) {
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
            }
        }
        const bool write = mine && !(in_place && any == 0u && bits == (1u << VE) - 1u);
        float v[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i) v[i] = 0.0f;
        if (write && bits != 0u) load_logits<T>(x, n, j, v);
        if constexpr (TABLE) {
            if (any) {
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    const uint32_t c = w[i] & kCount;
                    float y = v[i];
                    if (w[i] & ~kBiased) y = y > 0.0f ? divide(y, rep, inv) : y * rep;
                    if (c) y -= freq * float(c) + pres;
                    v[i] = y;
                }
            }
            if (a.n_bias && __ballot((any & kBiased) != 0u)) {
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    uint64_t who = __ballot((w[i] & kBiased) != 0u);
                    while (who) {
                        const int src = __ffsll((unsigned long long)who) - 1;
                        who &= who - 1ull;
                        const float b = bias_of(list, uint32_t(__builtin_amdgcn_readlane(int(e0), src)) + i, lane);
                        if (lane == uint32_t(src)) v[i] += b;
                    }
                }
            }
        }
        if (!write) continue;
#pragma unroll
        for (int i = 0; i < VE; ++i) v[i] = (bits >> i) & 1u ? v[i] : -INFINITY;
        store_grad<T>(out, n, e0, v);
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

template <typename T, bool TABLE>
static void adjust_launch(const AdjArgs& a, hipStream_t st) {
    const size_t lds = TABLE ? size_t(a.chunk) * 4 + size_t(a.n_bias) * 8 : 0;
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

// e8q_token_logprobs, its gradient, and both in one call.
//
// Forward.  One pass over a row keeps, per thread, the running maximum m of the
// logits, s = sum exp2((x - m) k) and t = sum exp2((x - m) k) (x - m) k with
// k = scale log2 e; a new maximum rescales both.  At the end
//   lse = scale m + ln s,   entropy = ln s - ln 2 * t / s,
//   logprob = scale (x_t - m) - ln s,
// so every exponent is formed from a difference of logits, exact where it
// matters (near the maximum), and not from scale x - lse.  So is the gradient's,
// but for one that is handed a stored lse of moderate size (kLseMost).
//
// Alternatives.  Each wave keeps the 64 best keys of its part of the row,
// sorted, one per lane.  A key orders by value, then by lower index:
// (order-preserving bits of x) << 32 | ~index.  The k-th best key so far is
// the threshold; a vector without an element above it costs one comparison.
// Elements above it are appended to a list in LDS, and every 64 of them are
// sorted and merged (bitonic, in registers).  The first threshold is the k-th
// largest of the 64 lanes' maxima over their first vectors (at least k
// elements reach it), so that a row in random order appends about k ln(V / k)
// elements; one in ascending order appends every element and is still right.
//
// Few rows are split over blocks (partial m, s, t and keys in the workspace)
// and joined by a second kernel.
//
// What bounds it.  Long batches: memory, with about 11 vector instruction slots
// per logit close behind (v_exp_f32 takes four): 4096 x 32768 bf16 52 us, 5.1 TB/s;
// with 20 alternatives the search for them, 103 us.
// One row: two launches and their latencies (11 + 5 us for 131072 logits with 8
// alternatives, while the host needs 12 us to issue them).
#include <float.h>

#include "e8q_device.hpp"
#include "e8q_host.hpp"
#include "e8q_vec.hpp"

namespace e8q {

constexpr int kLpBlock = 256;         // threads per row, or per part of a row
constexpr int kLpWide = 1024;         // threads per row of the two-pass gradient
constexpr int kLpUnroll = 4;          // vectors in flight per thread
constexpr int kTopMax = 64;           // one key per lane
constexpr int kMaxTokens = 1024;
constexpr int kMaxSplits = 256;
constexpr int64_t kMaxRows = int64_t(1) << 24;   // a block of kLpBlock per row, fewer than 2^32 threads
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
// Stands in for an exponent of -inf where it is multiplied (0 * -inf is NaN):
// exp2 of it is 0, and times any sum it stays finite.
constexpr float kFloor = -1e9f;

struct LpArgs {
    const void* x;
    int64_t stride;
    uint32_t rows, vocab;
    float scale;
    const void* tokens;
    uint32_t ntok;
    int i64;                    // token ids are int64
    float* logprob;
    float* lse;
    float* ent;
    int32_t* top_idx;
    float* top_lp;
    uint32_t k;
    uint32_t splits;            // blocks per row
    uint32_t per_split;         // vectors per block
    float4* part;               // [rows, splits] m, s, t
    union {                     // (one more pointer costs a call of few rows 0.4 us)
        uint64_t* part_keys;    // with alternatives: [rows, splits, 64]
        float4* joined;         // without: [rows] m, s, t of whole rows, for the gradient, or null
    };
    const float* g_lp;
    const float* g_ent;
    const float* lse_in;
    const float* ent_in;
    void* dx;
    int64_t dx_stride;
    uint32_t* status;
};

__device__ __forceinline__ int64_t token_at(const LpArgs& a, uint64_t i) {
    return a.i64 ? static_cast<const int64_t*>(a.tokens)[i] : int64_t(static_cast<const int32_t*>(a.tokens)[i]);
}

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// ------------------------------------------------------------ softmax statistics

struct Stat {
    float m, s, t;
};

__device__ __forceinline__ Stat stat_empty() { return {-FLT_MAX, 0.0f, 0.0f}; }

__device__ __forceinline__ Stat stat_join(const Stat& a, const Stat& b, float k) {
    const float m = fmaxf(a.m, b.m);
    const float da = fmaxf((a.m - m) * k, kFloor), db = fmaxf((b.m - m) * k, kFloor);
    // a NaN in (a.m - m) can only come from m = inf, where s is a NaN already
    const float ea = exp2_fast(da), eb = exp2_fast(db);
    return {m, a.s * ea + b.s * eb, ea * (a.t + a.s * da) + eb * (b.t + b.s * db)};
}

template <int N>
__device__ __forceinline__ void stat_add(Stat& st, const float (&v)[N], float k) {
    float cm = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) cm = fmaxf(cm, v[i]);
    const float m = fmaxf(st.m, cm);
    const float d = fmaxf((st.m - m) * k, kFloor);
    const float r = exp2_fast(d);
    st.t = r * (st.t + st.s * d);
    st.s *= r;
    st.m = m;
    float s0 = 0.0f, s1 = 0.0f, t0 = 0.0f, t1 = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float d0 = (v[i] - m) * k, d1 = (v[i + 1] - m) * k;
        const float e0 = exp2_fast(d0), e1 = exp2_fast(d1);
        s0 += e0;
        s1 += e1;
        t0 = fmaf(e0, fmaxf(d0, kFloor), t0);
        t1 = fmaf(e1, fmaxf(d1, kFloor), t1);
    }
    st.s += s0 + s1;
    st.t += t0 + t1;
}

template <int MASK>
__device__ __forceinline__ void stat_xor(Stat& st, float k) {
    const Stat o = {lane_xor<MASK>(st.m), lane_xor<MASK>(st.s), lane_xor<MASK>(st.t)};
    // in the order of the lanes, so that both partners get the same bits
    st = (__lane_id() & uint32_t(MASK)) ? stat_join(o, st, k) : stat_join(st, o, k);
}

__device__ __forceinline__ Stat stat_wave(Stat st, float k) {
    stat_xor<32>(st, k);
    stat_xor<16>(st, k);
    stat_xor<8>(st, k);
    stat_xor<4>(st, k);
    stat_xor<2>(st, k);
    stat_xor<1>(st, k);
    return st;
}

// ------------------------------------------------------------ sorted keys

__device__ __forceinline__ uint64_t key_of(float v, uint32_t idx) {
    const uint32_t b = __float_as_uint(v + 0.0f);                // -0 counts as +0
    uint32_t h = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    h = v != v ? 0xFFFFFFFFu : h;                                // NaN above everything
    return (uint64_t(h) << 32) | uint32_t(~idx);
}

__device__ __forceinline__ float value_of(uint64_t key) {
    const uint32_t h = uint32_t(key >> 32);
    return __uint_as_float(h & 0x80000000u ? h & 0x7FFFFFFFu : ~h);
}

// Lane l gets lane l ^ 15.
__device__ __forceinline__ uint64_t row_mirror(uint64_t v) {
    const int lo = __builtin_amdgcn_mov_dpp(int(uint32_t(v)), 0x140, 0xF, 0xF, true);
    const int hi = __builtin_amdgcn_mov_dpp(int(uint32_t(v >> 32)), 0x140, 0xF, 0xF, true);
    return (uint64_t(uint32_t(hi)) << 32) | uint32_t(lo);
}

__device__ __forceinline__ uint64_t keep(uint64_t a, uint64_t b, bool larger) { return (a > b) == larger ? a : b; }

// One stage of a bitonic network: blocks of `block` lanes descend and ascend in turn.
template <int J>
__device__ __forceinline__ void exchange(uint64_t& v, uint32_t lane, uint32_t block) {
    v = keep(v, lane_xor<J>(v), ((lane & uint32_t(J)) == 0u) == ((lane & block) == 0u));
}

template <int J>
__device__ __forceinline__ void merge_stages(uint64_t& v, uint32_t lane, uint32_t block) {
    exchange<J>(v, lane, block);
    if constexpr (J > 1) merge_stages<J / 2>(v, lane, block);
}

// Descending over the lanes.
__device__ __forceinline__ uint64_t sort_desc(uint64_t v, uint32_t lane) {
    merge_stages<1>(v, lane, 2u);
    merge_stages<2>(v, lane, 4u);
    merge_stages<4>(v, lane, 8u);
    merge_stages<8>(v, lane, 16u);
    merge_stages<16>(v, lane, 32u);
    merge_stages<32>(v, lane, 64u);
    return v;
}

// The 64 largest of two descending lists, descending.
__device__ __forceinline__ uint64_t merge_desc(uint64_t a, uint64_t b, uint32_t lane) {
    uint64_t v = lane_xor<32>(lane_xor<16>(row_mirror(b)));          // lane 63 - l
    v = a > v ? a : v;
    merge_stages<32>(v, lane, 64u);
    return v;
}

// The k-th largest of the lanes' values, by the bits of the answer from the top.
__device__ __forceinline__ uint32_t kth_largest(uint32_t v, uint32_t k) {
    uint32_t t = 0u;
    for (int b = 31; b >= 0; --b) {
        const uint32_t c = t | (1u << b);
        if (uint32_t(__popcll(__ballot(v >= c))) >= k) t = c;
    }
    return t;
}

// A wave's alternatives: its 64 best keys so far, and candidates not merged yet.
struct TopList {
    uint64_t best;        // lane's place in the descending list
    uint64_t thr;         // k-th best key, at least (wave-uniform)
    float floor;          // its value; a NaN's lets everything pass to the keys
    uint32_t count;       // candidates in LDS (wave-uniform, < 64 between vectors)
    uint64_t* buf;        // [128] of this wave

    __device__ __forceinline__ void set(uint64_t key) {
        thr = key;
        floor = value_of(key);
    }

    __device__ __forceinline__ void flush(uint32_t n, uint32_t k, uint32_t lane) {
        const uint64_t c = lane < n ? buf[lane] : 0ull;
        best = merge_desc(best, sort_desc(c, lane), lane);
        const uint32_t lo = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(best)), int(k - 1)));
        const uint32_t hi = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(best >> 32)), int(k - 1)));
        const uint64_t kth = (uint64_t(hi) << 32) | lo;
        if (kth > thr) set(kth);
    }

    // Appends the lanes' keys above the threshold.
    __device__ __forceinline__ void offer(uint64_t key, uint32_t k, uint32_t lane) {
        const bool in = key > thr;
        const uint64_t who = __ballot(in);
        if (!who) return;
        if (in) buf[count + __popcll(who & ((1ull << lane) - 1ull))] = key;
        count += uint32_t(__popcll(who));
        if (count >= 64u) {
            __builtin_amdgcn_wave_barrier();
            flush(64u, k, lane);
            const uint64_t rest = buf[64u + lane];
            __builtin_amdgcn_wave_barrier();
            buf[lane] = rest;
            count -= 64u;
            __builtin_amdgcn_wave_barrier();
        }
    }
};

// ------------------------------------------------------------ one row's part

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

// The block's statistics, in every thread.  Opens with no barrier: `s` is this
// call's own LDS.
template <int BLOCK>
__device__ __forceinline__ Stat stat_block(Stat st, float k2, Stat* s) {
    st = stat_wave(st, k2);
    if ((threadIdx.x & 63u) == 0u) s[threadIdx.x >> 6] = st;
    __syncthreads();
    st = s[0];
#pragma unroll
    for (int w = 1; w < BLOCK / kWave; ++w) st = stat_join(st, s[w], k2);
    return st;
}

// The waves' lists (in `s`, STRIDE keys apart, and in `best`) in pairs; wave 0
// ends with the block's.
template <int BLOCK, int STRIDE>
__device__ __forceinline__ void merge_block(uint64_t& best, uint64_t* s, uint32_t wave, uint32_t lane) {
#pragma unroll
    for (int gap = 1; gap < BLOCK / kWave; gap *= 2) {
        if (wave % (2 * gap) == 0) {
            best = merge_desc(best, s[(wave + gap) * STRIDE + lane], lane);
            s[wave * STRIDE + lane] = best;
        }
        __syncthreads();
    }
}

// Statistics (all waves end with the block's) and alternatives (wave 0 ends
// with the block's) of the vectors [lo, hi) of a row.
template <typename T, bool TOP, int BLOCK>
__device__ __forceinline__ Stat row_part(const T* row, uint32_t vocab, uint32_t lo, uint32_t hi,
                                         float k2, uint32_t top_k, uint64_t& best) {
    constexpr int VE = kVec<T>, kWaves = BLOCK / kWave;
    __shared__ Stat s_stat[kWaves];
    __shared__ uint64_t s_keys[TOP ? kWaves * 128 : 1];
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
    Stat st = stat_empty();
    TopList top{0ull, 0ull, -INFINITY, 0u, s_keys + (TOP ? wave * 128 : 0)};
    bool first = true;
    for (uint32_t base = lo; base < hi; base += BLOCK * kLpUnroll) {
        float v[kLpUnroll * VE];
#pragma unroll
        for (int u = 0; u < kLpUnroll; ++u) {
            const uint32_t j = base + u * BLOCK + tid;
            float w[VE];
            if (j < hi) {
                load_logits<T>(row, vocab, j, w);
            } else {
#pragma unroll
                for (int i = 0; i < VE; ++i) w[i] = -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < VE; ++i) v[u * VE + i] = w[i];
        }
        stat_add(st, v, k2);
        if constexpr (TOP) {
            // per vector: its largest element, and whether it holds a NaN
            float most[kLpUnroll];
            bool nan[kLpUnroll];
#pragma unroll
            for (int u = 0; u < kLpUnroll; ++u) {
                most[u] = v[u * VE];
                nan[u] = false;
#pragma unroll
                for (int i = 1; i < VE; ++i) most[u] = fmaxf(most[u], v[u * VE + i]);
#pragma unroll
                for (int i = 0; i < VE; i += 2) nan[u] |= __builtin_isunordered(v[u * VE + i], v[u * VE + i + 1]);
            }
            if (first) {
                float m = most[0];
                bool any = nan[0];
#pragma unroll
                for (int u = 1; u < kLpUnroll; ++u) {
                    m = fmaxf(m, most[u]);
                    any |= nan[u];
                }
                const uint32_t mine = any ? 0xFFFFFFFFu : uint32_t(key_of(m, 0u) >> 32);
                top.set(uint64_t(kth_largest(mine, top_k)) << 32);
                first = false;
            }
#pragma unroll
            for (int u = 0; u < kLpUnroll; ++u) {
                if (!__ballot(nan[u] || !(most[u] < top.floor))) continue;
                const uint32_t j = base + u * BLOCK + tid;
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    const uint32_t e = j * VE + i;
                    top.offer(j < hi && e < vocab ? key_of(v[u * VE + i], e) : 0ull, top_k, lane);
                }
            }
        }
    }
    if constexpr (TOP) {
        __builtin_amdgcn_wave_barrier();
        if (top.count) top.flush(top.count, top_k, lane);
    }
    if constexpr (TOP) {
        __builtin_amdgcn_wave_barrier();
        top.buf[lane] = top.best;
    }
    st = stat_block<BLOCK>(st, k2, s_stat);
    if constexpr (TOP) {
        merge_block<BLOCK, 128>(top.best, s_keys, wave, lane);
        best = top.best;
    }
    return st;
}

struct RowEnd {
    float ln_s, lse, ent;
};

// Row of -inf only: s = 0.
__device__ __forceinline__ RowEnd row_end(const Stat& st, float scale) {
    if (st.s == 0.0f) return {0.0f, -INFINITY, 0.0f};
    const float l2 = __log2f(st.s);
    const float ln_s = l2 * kLn2;
    return {ln_s, scale * st.m + ln_s, (l2 - st.t / st.s) * kLn2};
}

__device__ __forceinline__ float logprob_of(float x, const Stat& st, const RowEnd& e, float scale) {
    return st.s == 0.0f ? -INFINITY : scale * (x - st.m) - e.ln_s;
}

// A thread's given token (the first of blockDim) and its logit, read ahead of
// the statistics.
struct OneToken {
    int64_t id;
    float x;
};

template <typename T>
__device__ __forceinline__ OneToken first_token(const LpArgs& a, uint32_t row, const T* x) {
    OneToken t = {-1, 0.0f};
    if (threadIdx.x < a.ntok) {
        t.id = token_at(a, uint64_t(row) * a.ntok + threadIdx.x);
        if (t.id >= 0 && t.id < int64_t(a.vocab)) t.x = widen(x[t.id]);
    }
    return t;
}

// Outputs of one row, by one block; `best` is wave 0's list.
template <typename T, bool TOP>
__device__ __forceinline__ void write_row(const LpArgs& a, uint32_t row, const T* x, const Stat& st, uint64_t best,
                                          OneToken tok) {
    const uint32_t tid = threadIdx.x;
    const RowEnd e = row_end(st, a.scale);
    uint32_t flags = 0u;
    if (tid == 0) {
        if (a.lse) a.lse[row] = e.lse;
        if (a.ent) a.ent[row] = e.ent;
        if (st.s != st.s) flags |= E8Q_STATUS_NONFINITE;
    }
    for (uint32_t j = tid; j < a.ntok; j += blockDim.x) {
        if (j != tid) {
            tok.id = token_at(a, uint64_t(row) * a.ntok + j);
            tok.x = tok.id >= 0 && tok.id < int64_t(a.vocab) ? widen(x[tok.id]) : 0.0f;
        }
        if (tok.id >= int64_t(a.vocab)) flags |= E8Q_STATUS_BAD_INDEX;
        if (a.logprob)
            a.logprob[uint64_t(row) * a.ntok + j] =
                tok.id >= 0 && tok.id < int64_t(a.vocab) ? logprob_of(tok.x, st, e, a.scale) : 0.0f;
    }
    if constexpr (TOP) {
        if (tid < a.k) {
            if (a.top_idx) a.top_idx[uint64_t(row) * a.k + tid] = int32_t(~uint32_t(best));
            if (a.top_lp) a.top_lp[uint64_t(row) * a.k + tid] = logprob_of(value_of(best), st, e, a.scale);
        }
    }
    flush_status(flags, a.status);
}

template <typename T, bool TOP>
__global__ __launch_bounds__(kLpBlock) void logprobs_kernel(LpArgs a) {
    const uint32_t row = a.splits == 1 ? blockIdx.x : blockIdx.x / a.splits;
    const uint32_t sp = blockIdx.x - row * a.splits;
    const T* x = static_cast<const T*>(a.x) + int64_t(row) * a.stride;
    const uint32_t nvec = (a.vocab + kVec<T> - 1) / kVec<T>;
    const uint32_t lo = min(sp * a.per_split, nvec), hi = min(lo + a.per_split, nvec);
    uint64_t best = 0ull;
    OneToken tok = {-1, 0.0f};
    if (a.splits == 1) tok = first_token(a, row, x);
    const Stat st = row_part<T, TOP, kLpBlock>(x, a.vocab, lo, hi, a.scale * kLog2e, a.k, best);
    if (a.splits == 1) {
        write_row<T, TOP>(a, row, x, st, best, tok);
        return;
    }
    if (threadIdx.x == 0) a.part[blockIdx.x] = make_float4(st.m, st.s, st.t, 0.0f);
    if constexpr (TOP) {
        if (threadIdx.x < kTopMax) a.part_keys[uint64_t(blockIdx.x) * kTopMax + threadIdx.x] = best;
    }
}

// Joins the parts of one row.
template <typename T, bool TOP>
__global__ __launch_bounds__(kLpBlock) void logprobs_join_kernel(LpArgs a) {
    constexpr int BLOCK = kLpBlock, kWaves = BLOCK / kWave;
    __shared__ Stat s_stat[kWaves];
    __shared__ uint64_t s_keys[TOP ? kWaves * kTopMax : 1];
    const uint32_t row = blockIdx.x, tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
    const T* x = static_cast<const T*>(a.x) + int64_t(row) * a.stride;
    const OneToken tok = first_token(a, row, x);
    Stat st = stat_empty();
    if (tid < a.splits) {
        const float4 p = a.part[uint64_t(row) * a.splits + tid];
        st = {p.x, p.y, p.z};
    }
    uint64_t best = 0ull;
    if constexpr (TOP) {
        const uint64_t* keys = a.part_keys + uint64_t(row) * a.splits * kTopMax + lane;
        if (wave < a.splits) best = keys[wave * kTopMax];
        for (uint32_t i = wave + kWaves; i < a.splits; i += kWaves) best = merge_desc(best, keys[i * kTopMax], lane);
        s_keys[tid] = best;
    }
    st = stat_block<BLOCK>(st, a.scale * kLog2e, s_stat);
    if constexpr (!TOP) {
        if (a.joined && tid == 0u) a.joined[row] = make_float4(st.m, st.s, st.t, 0.0f);
    }
    if constexpr (TOP) merge_block<BLOCK, kTopMax>(best, s_keys, wave, lane);
    write_row<T, TOP>(a, row, x, st, best, tok);
}

// ------------------------------------------------------------ gradient

// dx = p' (c0 + c1 d) with d = (x a - b) k, p' = exp2(d): the row's constants.
struct GradRow {
    float a, b, k, c0, c1;
};

__device__ __forceinline__ float grad_at(float x, const GradRow& g) {
    const float d = (x * g.a - g.b) * g.k;
    return exp2_fast(d) * fmaf(g.c1, fmaxf(d, kFloor), g.c0);
}

// The row's live tokens, their logits and upstream gradients in (dynamic) LDS.
struct RowTokens {
    int32_t* id;
    float* g;
    float* x;
};

__device__ __forceinline__ RowTokens row_tokens(uint32_t ntok) {
    extern __shared__ uint32_t s_tokens[];
    return {reinterpret_cast<int32_t*>(s_tokens), reinterpret_cast<float*>(s_tokens + ntok),
            reinterpret_cast<float*>(s_tokens + 2u * ntok)};
}

template <typename T>
__device__ __forceinline__ float load_tokens(const LpArgs& a, uint32_t row, const T* x, const RowTokens& s) {
    uint32_t flags = 0u;
    for (uint32_t j = threadIdx.x; j < a.ntok; j += blockDim.x) {
        const int64_t t = token_at(a, uint64_t(row) * a.ntok + j);
        const bool live = t >= 0 && t < int64_t(a.vocab);
        if (t >= int64_t(a.vocab)) flags |= E8Q_STATUS_BAD_INDEX;
        s.id[j] = live ? int32_t(t) : -1;
        s.g[j] = live ? a.g_lp[uint64_t(row) * a.ntok + j] : 0.0f;
        s.x[j] = live ? widen(x[t]) : 0.0f;
    }
    flush_status(flags, a.status);
    __syncthreads();
    float sum = 0.0f;
    for (uint32_t j = 0; j < a.ntok; ++j) sum += s.g[j];
    return sum;
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

// The given tokens among the elements [first, last), which this block has
// written (the logits of the tokens were read before: dx may be x).
template <typename T>
__device__ __forceinline__ void grad_tokens(const LpArgs& a, T* dx, int64_t first, int64_t last, const GradRow& g,
                                            bool zero, const RowTokens& s) {
    if (!a.ntok || zero) return;
    __syncthreads();
    for (uint32_t j = threadIdx.x; j < a.ntok; j += blockDim.x) {
        const int32_t t = s.id[j];
        if (t < 0 || t < first || t >= last) continue;
        float sum = 0.0f;                                  // equal tokens: the same sum for each
        for (uint32_t i = 0; i < a.ntok; ++i) sum += s.id[i] == t ? s.g[i] : 0.0f;
        dx[t] = narrow<T>(fmaf(a.scale, sum, grad_at(s.x[j], g)));
    }
}

// The vectors [lo, hi) of the gradient row.
template <typename T>
__device__ __forceinline__ void grad_part(const LpArgs& a, const T* x, T* dx, uint32_t lo, uint32_t hi,
                                          const GradRow& g, bool zero, const RowTokens& s) {
    constexpr int VE = kVec<T>;
    for (uint32_t j = lo + threadIdx.x; j < hi; j += blockDim.x) {
        float v[VE];
        load_logits<T>(x, a.vocab, j, v);
#pragma unroll
        for (int i = 0; i < VE; ++i) v[i] = zero ? 0.0f : grad_at(v[i], g);
        store_grad<T>(dx, a.vocab, j * VE, v);
    }
    grad_tokens<T>(a, dx, int64_t(lo) * VE, int64_t(hi) * VE, g, zero, s);
}

// The gradient's constants from the row's statistics.
__device__ __forceinline__ GradRow grad_row(const LpArgs& a, const Stat& st, float sum, float gh) {
    const RowEnd e = row_end(st, a.scale);
    const float c = a.scale / st.s;
    return {1.0f, st.m, a.scale * kLog2e, -c * (sum + gh * (e.ent - e.ln_s)), -c * gh * kLn2};
}

// Rows up to this |lse| take their p from lse.  It is stored to 24 bits, so p is
// off by a factor of at most 1 + |lse| 2^-24: here 2^-20 of itself (16 < |lse| <= 32),
// about what the rounding of an exponent of that size costs.  Past it the error would
// grow with whatever all logits of a row have in common (a row of the type's lowest
// value would have p = 1 everywhere), so the row's maximum and sum are formed
// again.  301 x 32003 float32: 14 us, with the second reading (by every part of a
// row) 35 us, in place 13 and 54 us; 8192 x 32768 bf16: 202 and 240 us.
constexpr float kLseMost = 32.0f;

// Statistics as they were joined (`joined`), or from lse as stored.
template <typename T>
__global__ __launch_bounds__(kLpBlock) void logprobs_backward_kernel(LpArgs a) {
    const RowTokens s_tok = row_tokens(a.ntok);
    const uint32_t row = a.splits == 1 ? blockIdx.x : blockIdx.x / a.splits;
    const uint32_t sp = blockIdx.x - row * a.splits;
    const T* x = static_cast<const T*>(a.x) + int64_t(row) * a.stride;
    T* dx = static_cast<T*>(a.dx) + int64_t(row) * a.dx_stride;
    const uint32_t nvec = (a.vocab + kVec<T> - 1) / kVec<T>;
    uint32_t lo = min(sp * a.per_split, nvec), hi = min(lo + a.per_split, nvec);
    // read beside the tokens: what branches below depends on it
    const float lse = a.joined ? 0.0f : a.lse_in[row];
    const float gh = a.g_ent ? a.g_ent[row] : 0.0f;
    const float h = a.g_ent && !a.joined ? a.ent_in[row] : 0.0f;
    const float sum = load_tokens<T>(a, row, x, s_tok);
    GradRow g;
    bool zero;
    if (a.joined) {
        const float4 p = a.joined[row];
        const Stat st = {p.x, p.y, p.z};
        g = grad_row(a, st, sum, gh);
        zero = st.s == 0.0f;
    } else {
        zero = lse == -INFINITY;
        if (fabsf(lse) > kLseMost && !zero) {
            // in place a row is read and written by its first block alone, whose threads
            // have all read (a barrier joins the statistics) before one of them writes
            if (a.dx == a.x) {
                if (sp > 0u) return;
                lo = 0u;
                hi = nvec;
            }
            uint64_t none = 0ull;
            const Stat st = row_part<T, false, kLpBlock>(x, a.vocab, 0u, nvec, a.scale * kLog2e, 0u, none);
            g = grad_row(a, st, sum, gh);
            zero = st.s == 0.0f;
        } else {
            g = {a.scale, lse, kLog2e, -a.scale * (sum + gh * h), -a.scale * gh * kLn2};
        }
    }
    grad_part<T>(a, x, dx, lo, hi, g, zero, s_tok);
}

// Statistics and gradient of a row that fits the registers of one block, NV
// vectors a thread: the row is read once.
template <typename T, int BLOCK, int NV>
__global__ __launch_bounds__(BLOCK) void logprobs_grad_kernel(LpArgs a) {
    constexpr int VE = kVec<T>, kGroup = 2;      // vectors unpacked at a time
    __shared__ Stat s_stat[BLOCK / kWave];
    const RowTokens s_tok = row_tokens(a.ntok);
    const uint32_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + int64_t(row) * a.stride;
    T* dx = static_cast<T*>(a.dx) + int64_t(row) * a.dx_stride;
    const uint32_t nvec = (a.vocab + VE - 1) / VE;
    const uint32_t wave0 = uint32_t(__builtin_amdgcn_readfirstlane(int(threadIdx.x & ~63u)));
    u32x4_t raw[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const uint32_t e0 = (n * BLOCK + threadIdx.x) * VE;
        if (e0 + VE <= a.vocab) {
            raw[n] = reinterpret_cast<const RowVec<T>*>(x + e0)->v;
        } else {
            float v[VE];
#pragma unroll
            for (int i = 0; i < VE; ++i) v[i] = e0 + i < a.vocab ? widen(x[e0 + i]) : -INFINITY;
            raw[n] = pack(v);
        }
    }
    const float sum = load_tokens<T>(a, row, x, s_tok);
    const float k2 = a.scale * kLog2e;
    Stat st = stat_empty();
#pragma unroll
    for (int n = 0; n < NV; n += kGroup) {
        if (uint32_t(n * BLOCK) + wave0 >= nvec) break;        // nothing of the row for this wave any more
        float v[kGroup * VE];
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
            float w[VE];
            unpack(raw[n + u], w);
#pragma unroll
            for (int i = 0; i < VE; ++i) v[u * VE + i] = w[i];
        }
        stat_add(st, v, k2);
        __builtin_amdgcn_sched_barrier(0);       // one group unpacked at a time
    }
    st = stat_block<BLOCK>(st, k2, s_stat);
    write_row<T, false>(a, row, x, st, 0ull, first_token(a, row, x));
    __syncthreads();                 // the tokens' logits are read before dx (maybe x) is written
    const GradRow g = grad_row(a, st, sum, a.g_ent ? a.g_ent[row] : 0.0f);
    const bool zero = st.s == 0.0f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        if (uint32_t(n * BLOCK) + wave0 >= nvec) break;
        const uint32_t e0 = (n * BLOCK + threadIdx.x) * VE;
        float v[VE];
        unpack(raw[n], v);
#pragma unroll
        for (int i = 0; i < VE; ++i) v[i] = zero ? 0.0f : grad_at(v[i], g);
        store_grad<T>(dx, a.vocab, e0, v);
        __builtin_amdgcn_sched_barrier(0);
    }
    grad_tokens<T>(a, dx, 0, int64_t(a.vocab), g, zero, s_tok);
}

// The same for longer rows: two passes over the row.
template <typename T>
__global__ __launch_bounds__(kLpWide) void logprobs_grad_long_kernel(LpArgs a) {
    const RowTokens s_tok = row_tokens(a.ntok);
    const uint32_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + int64_t(row) * a.stride;
    T* dx = static_cast<T*>(a.dx) + int64_t(row) * a.dx_stride;
    const uint32_t nvec = (a.vocab + kVec<T> - 1) / kVec<T>;
    const float sum = load_tokens<T>(a, row, x, s_tok);
    uint64_t none = 0ull;
    const Stat st = row_part<T, false, kLpWide>(x, a.vocab, 0u, nvec, a.scale * kLog2e, 0u, none);
    write_row<T, false>(a, row, x, st, 0ull, first_token(a, row, x));
    __syncthreads();                 // the tokens' logits are read before dx (maybe x) is written
    const GradRow g = grad_row(a, st, sum, a.g_ent ? a.g_ent[row] : 0.0f);
    grad_part<T>(a, x, dx, 0u, nvec, g, st.s == 0.0f, s_tok);
}

// ------------------------------------------------------------ host

// Blocks per row: enough blocks for every CU to hold about four, each with
// kLpUnroll vectors a thread to read (one row of 131072 bf16 logits with 8
// alternatives: 14.4 us with 16 parts, 14.7 with 32, 16.4 with 32 joined by 1024
// threads).
static uint32_t lp_splits(int64_t rows, int64_t vocab, size_t esz, uint32_t& per_split) {
    const uint64_t ve = 16 / esz, nvec = (uint64_t(vocab) + ve - 1) / ve;
    const uint64_t want = (uint64_t(device_cu_count()) * 4 + uint64_t(rows) - 1) / uint64_t(rows);
    const uint64_t most = (nvec + kLpBlock * kLpUnroll - 1) / (kLpBlock * kLpUnroll);
    uint64_t n = want < most ? want : most;
    if (n > kMaxSplits) n = kMaxSplits;
    if (n < 1) n = 1;
    per_split = uint32_t((nvec + n - 1) / n);
    return uint32_t((nvec + per_split - 1) / per_split);
}

static e8q_status_t lp_check(const void* logits, e8q_dtype_t dtype, int64_t rows, int64_t vocab, int64_t stride,
                             float scale, const void* tokens, e8q_index_t index_type, int64_t ntok,
                             uint32_t* status) {
    if (!logits || !status || rows <= 0 || vocab <= 0 || stride < vocab || ntok < 0) return E8Q_ERR_INVALID;
    if (dtype != E8Q_F32 && dtype != E8Q_BF16) return E8Q_ERR_INVALID;
    if (!(scale > 0.0f) || __builtin_isinf(scale)) return E8Q_ERR_INVALID;
    if ((ntok > 0) != (tokens != nullptr)) return E8Q_ERR_INVALID;
    if (index_type != E8Q_I32 && index_type != E8Q_I64) return E8Q_ERR_INVALID;
    const size_t esz = dtype == E8Q_BF16 ? 2 : 4, isz = index_type == E8Q_I64 ? 8 : 4;
    if (reinterpret_cast<uintptr_t>(logits) % esz || reinterpret_cast<uintptr_t>(tokens) % isz) return E8Q_ERR_INVALID;
    if (vocab >= (int64_t(1) << 31) - 16 || rows >= kMaxRows || ntok > kMaxTokens ||
        stride >= (int64_t(1) << 40))
        return E8Q_ERR_UNSUPPORTED;
    return E8Q_OK;
}

static LpArgs lp_args(const void* logits, int64_t rows, int64_t vocab, int64_t stride, float scale,
                      const void* tokens, e8q_index_t index_type, int64_t ntok, uint32_t* status) {
    LpArgs a{};
    a.x = logits;
    a.stride = stride;
    a.rows = uint32_t(rows);
    a.vocab = uint32_t(vocab);
    a.scale = scale;
    a.tokens = tokens;
    a.ntok = uint32_t(ntok);
    a.i64 = index_type == E8Q_I64;
    a.status = status;
    return a;
}

static size_t lp_part_bytes(uint64_t blocks) { return size_t((blocks * sizeof(float4) + 255) / 256 * 256); }

static size_t lp_workspace(int64_t rows, int64_t vocab, size_t esz, int64_t top_k) {
    uint32_t per = 0;
    const uint64_t splits = lp_splits(rows, vocab, esz, per);
    if (splits == 1) return 0;
    // without alternatives: room for the rows' statistics (e8q_token_logprobs_grad)
    return lp_part_bytes(uint64_t(rows) * splits) +
           (top_k ? size_t(uint64_t(rows) * splits * kTopMax * 8) : size_t(rows) * sizeof(float4));
}

// Forward launches; the arguments are checked.
template <typename T, bool TOP>
static void lp_forward(LpArgs& a, void* ws, hipStream_t st) {
    a.splits = lp_splits(a.rows, a.vocab, sizeof(T), a.per_split);
    a.part = static_cast<float4*>(ws);
    if (TOP)
        a.part_keys = reinterpret_cast<uint64_t*>(static_cast<char*>(ws) + lp_part_bytes(uint64_t(a.rows) * a.splits));
    launch(logprobs_kernel<T, TOP>, dim3(a.rows * a.splits), dim3(kLpBlock), 0, st, a);
    if (a.splits == 1) return;
    launch(logprobs_join_kernel<T, TOP>, dim3(a.rows), dim3(kLpBlock), 0, st, a);
}

template <typename T>
static void lp_backward(LpArgs& a, hipStream_t st) {
    a.splits = lp_splits(a.rows, a.vocab, sizeof(T), a.per_split);
    launch(logprobs_backward_kernel<T>, dim3(a.rows * a.splits), dim3(kLpBlock), a.ntok * 12u, st, a);
}

// Whole rows: the smallest block whose registers hold one, while that leaves
// several rows to a CU.  Longer rows are read twice by blocks of kLpWide threads,
// two to a CU: their rows (512 at a time, 128 MiB at 131072 bf16 logits) stay in
// the last-level cache until the second reading.  Measured, 2^28 logits, bytes
// read and written once: bf16 2048 wide 4.3 TB/s, 16384 5.2, 32768 5.0, 65536
// 4.3 (3.9 in the registers of 512 threads), 131072 4.3; float32 8192 wide 5.3,
// 32768 5.3 (4.7 read twice), 131072 4.3.  A copy reaches 4.9.
template <typename T, class Go>
static void lp_grad_kernel(int64_t vocab, Go&& go) {
    const uint64_t nvec = (uint64_t(vocab) + kVec<T> - 1) / kVec<T>;
    if (nvec <= 64 * 4) go(logprobs_grad_kernel<T, 64, 4>, 64u);
    else if (nvec <= 128 * 4) go(logprobs_grad_kernel<T, 128, 4>, 128u);
    else if (nvec <= 256 * 4) go(logprobs_grad_kernel<T, 256, 4>, 256u);
    else if (nvec <= 256 * 8) go(logprobs_grad_kernel<T, 256, 8>, 256u);
    else if (nvec <= 256 * 16) go(logprobs_grad_kernel<T, 256, 16>, 256u);
    else if (sizeof(T) == 4 && nvec <= 512 * 16) go(logprobs_grad_kernel<T, 512, 16>, 512u);
    else go(logprobs_grad_long_kernel<T>, unsigned(kLpWide));
}

template <typename T>
static void lp_grad(LpArgs& a, hipStream_t st) {
    a.splits = 1;
    lp_grad_kernel<T>(a.vocab, [&](auto kernel, unsigned block) {
        launch(kernel, dim3(a.rows), dim3(block), a.ntok * 12u, st, a);
    });
}

// A launch has fewer than 2^32 threads.
template <typename T>
static bool lp_grad_fits(int64_t rows, int64_t vocab) {
    bool fits = false;
    lp_grad_kernel<T>(vocab, [&](auto, unsigned block) { fits = uint64_t(rows) * block < uint64_t(1) << 32; });
    return fits;
}

}  // namespace e8q

extern "C" size_t e8q_token_logprobs_workspace_size(int64_t rows, int64_t vocab, int64_t top_k) {
    using namespace e8q;
    if (rows <= 0 || vocab <= 0 || top_k < 0 || top_k > kTopMax || rows >= kMaxRows ||
        vocab >= (int64_t(1) << 31) - 16)
        return 0;
    const size_t b = lp_workspace(rows, vocab, 2, top_k), f = lp_workspace(rows, vocab, 4, top_k);
    return b > f ? b : f;
}

extern "C" e8q_status_t e8q_token_logprobs(const void* logits, e8q_dtype_t dtype, int64_t rows, int64_t vocab,
                                           int64_t row_stride, float scale, const void* tokens,
                                           e8q_index_t index_type, int64_t n_tokens, float* logprob_out,
                                           float* lse_out, float* entropy_out, int64_t top_k, int32_t* top_idx_out,
                                           float* top_logprob_out, void* workspace, size_t workspace_bytes,
                                           uint32_t* status_dev, void* stream) {
    using namespace e8q;
    e8q_status_t st = lp_check(logits, dtype, rows, vocab, row_stride, scale, tokens, index_type, n_tokens, status_dev);
    if (st != E8Q_OK) return st;
    if (top_k < 0 || top_k > vocab || (top_k > 0) != (top_idx_out || top_logprob_out)) return E8Q_ERR_INVALID;
    if ((logprob_out && !n_tokens) || (!logprob_out && !lse_out && !entropy_out && !top_k)) return E8Q_ERR_INVALID;
    if (top_k > kTopMax) return E8Q_ERR_UNSUPPORTED;
    const size_t need = lp_workspace(rows, vocab, dtype == E8Q_BF16 ? 2 : 4, top_k);
    if (need && (!workspace || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 256))
        return E8Q_ERR_INVALID;
    LpArgs a = lp_args(logits, rows, vocab, row_stride, scale, tokens, index_type, n_tokens, status_dev);
    a.logprob = logprob_out;
    a.lse = lse_out;
    a.ent = entropy_out;
    a.k = uint32_t(top_k);
    a.top_idx = top_idx_out;
    a.top_lp = top_logprob_out;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (dtype == E8Q_BF16)
        top_k ? lp_forward<uint16_t, true>(a, workspace, s) : lp_forward<uint16_t, false>(a, workspace, s);
    else
        top_k ? lp_forward<float, true>(a, workspace, s) : lp_forward<float, false>(a, workspace, s);
    return launch_status();
}

namespace e8q {

static e8q_status_t lp_check_grad(const void* logits, int64_t vocab, int64_t row_stride, int64_t n_tokens,
                                  const float* grad_logprob, const void* grad_logits, int64_t grad_stride,
                                  e8q_dtype_t dtype) {
    if (!grad_logits || grad_stride < vocab || (n_tokens > 0 && !grad_logprob)) return E8Q_ERR_INVALID;
    if (grad_logits == logits && grad_stride != row_stride) return E8Q_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(grad_logits) % (dtype == E8Q_BF16 ? 2 : 4)) return E8Q_ERR_INVALID;
    return grad_stride >= (int64_t(1) << 40) ? E8Q_ERR_UNSUPPORTED : E8Q_OK;
}

}  // namespace e8q

extern "C" e8q_status_t e8q_token_logprobs_backward(const void* logits, e8q_dtype_t dtype, int64_t rows,
                                                    int64_t vocab, int64_t row_stride, float scale,
                                                    const void* tokens, e8q_index_t index_type, int64_t n_tokens,
                                                    const float* lse, const float* grad_logprob,
                                                    const float* entropy, const float* grad_entropy,
                                                    void* grad_logits, int64_t grad_stride, uint32_t* status_dev,
                                                    void* stream) {
    using namespace e8q;
    e8q_status_t st = lp_check(logits, dtype, rows, vocab, row_stride, scale, tokens, index_type, n_tokens, status_dev);
    if (st != E8Q_OK) return st;
    if (!lse || (entropy == nullptr) != (grad_entropy == nullptr)) return E8Q_ERR_INVALID;
    st = lp_check_grad(logits, vocab, row_stride, n_tokens, grad_logprob, grad_logits, grad_stride, dtype);
    if (st != E8Q_OK) return st;
    LpArgs a = lp_args(logits, rows, vocab, row_stride, scale, tokens, index_type, n_tokens, status_dev);
    a.lse_in = lse;
    a.g_lp = grad_logprob;
    a.ent_in = entropy;
    a.g_ent = grad_entropy;
    a.dx = grad_logits;
    a.dx_stride = grad_stride;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (dtype == E8Q_BF16) lp_backward<uint16_t>(a, s);
    else lp_backward<float>(a, s);
    return launch_status();
}

extern "C" e8q_status_t e8q_token_logprobs_grad(const void* logits, e8q_dtype_t dtype, int64_t rows, int64_t vocab,
                                                int64_t row_stride, float scale, const void* tokens,
                                                e8q_index_t index_type, int64_t n_tokens, const float* grad_logprob,
                                                const float* grad_entropy, float* logprob_out, float* lse_out,
                                                float* entropy_out, void* grad_logits, int64_t grad_stride,
                                                void* workspace, size_t workspace_bytes, uint32_t* status_dev,
                                                void* stream) {
    using namespace e8q;
    e8q_status_t st = lp_check(logits, dtype, rows, vocab, row_stride, scale, tokens, index_type, n_tokens, status_dev);
    if (st != E8Q_OK) return st;
    if (logprob_out && !n_tokens) return E8Q_ERR_INVALID;
    st = lp_check_grad(logits, vocab, row_stride, n_tokens, grad_logprob, grad_logits, grad_stride, dtype);
    if (st != E8Q_OK) return st;
    const size_t need = lp_workspace(rows, vocab, dtype == E8Q_BF16 ? 2 : 4, 0);
    if (!need && !(dtype == E8Q_BF16 ? lp_grad_fits<uint16_t>(rows, vocab) : lp_grad_fits<float>(rows, vocab)))
        return E8Q_ERR_UNSUPPORTED;
    if (need && (!workspace || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 256))
        return E8Q_ERR_INVALID;
    LpArgs a = lp_args(logits, rows, vocab, row_stride, scale, tokens, index_type, n_tokens, status_dev);
    a.logprob = logprob_out;
    a.lse = lse_out;
    a.ent = entropy_out;
    a.g_lp = grad_logprob;
    a.g_ent = grad_entropy;
    a.dx = grad_logits;
    a.dx_stride = grad_stride;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (!need) {
        if (dtype == E8Q_BF16) lp_grad<uint16_t>(a, s);
        else lp_grad<float>(a, s);
        return launch_status();
    }
    // few rows: the two split passes, with the rows' statistics in the workspace
    a.joined = reinterpret_cast<float4*>(static_cast<char*>(workspace) + need - size_t(rows) * sizeof(float4));
    if (dtype == E8Q_BF16) {
        lp_forward<uint16_t, false>(a, workspace, s);
        lp_backward<uint16_t>(a, s);
    } else {
        lp_forward<float, false>(a, workspace, s);
        lp_backward<float>(a, s);
    }
    return launch_status();
}

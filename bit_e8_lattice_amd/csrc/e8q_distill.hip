// e8q_distill, its gradient, and both in one call: the divergence of a row's
// distribution from a teacher's top logits.
//
// With y = scale x, q = softmax(y), the teacher's places i_j with probabilities
// w_j (as given, or divided by their sum: then of log probabilities less the row's largest, whose
// exponentials keep float32's range whatever the scale of the given ones) and K the set of the named tokens,
//   loss = sum_j w_j (log w_j - log q_{i_j})  [ + w_r (log w_r - log q_r) ],
//   w_r = max(0, 1 - sum_j w_j),  q_r = sum of q outside K  (tail "rest" only),
//   dloss/dy_i = P q_i - sum_{j: i_j = i} w_j              for i in K,
//                q_i (P - w_r / q_r)                       outside K,
// P = sum_j w_j + w_r (w_r = 0 but for "rest").
//
// q_r is never formed as 1 - sum of q over K, which would lose it where the
// student is sure of K: there are two pairs of a running maximum and a sum.  The others' comes from
// the pass over the row, where a bit for every element (in LDS, a byte for each vector) says
// whether the teacher names it; the named elements' from their own logits, gathered by
// the places, one place for each element however often the teacher names it.
// Outside K the gradient is exp2((x - m_r) k) (P q_r - w_r) / s_r, m_r and
// s_r the maximum and sum of the others, so its exponential is at most 1 and the
// division by q_r is gone.  It is written for every element, and then, after a barrier, the
// places write theirs over it: looking the named elements up in the stream took
// 1268 us where this takes 1015 (8192 rows of 131072 bf16 logits, 64 places).  Where
// no other element is left (all named, or -inf), w_r counts as 0.
//
// Rows that fit are kept in the registers of a block between the sums and the gradient.  Few
// longer ones are split over blocks (partial sums in the workspace) and joined by a second
// kernel; many are read twice: the second time from the end, which the caches still
// hold (8192 rows of 131072: 1015 us from the start, 973 from the end; in the
// registers of one block of 1024 threads, which has a CU to itself, 1176).  The bound
// is memory: the bytes of the logits, and of the gradient.  Reached of them:
// 4.6 TB/s with 32768 bf16 logits a row (4096 rows 117 us), 4.4 with 131072 (8192 rows 976 us); a copy 4.9.
#include <float.h>

#include "e8q_rows.hpp"

namespace e8q {

constexpr int64_t kMaxPlaces = 1024;     // teacher places of a row
constexpr uint32_t kSegment = 32768;     // vectors marked in LDS at a time

struct DsArgs {
    const void* x;
    int64_t stride;
    uint32_t rows, vocab;
    float scale;
    const void* idx;
    const float* lp;
    uint32_t k;
    int i64;
    int tail;
    float* loss;
    float* logprob;
    float4* stats;              // [rows]: written forward, read backward
    uint32_t splits, per_split;
    float4* part;               // [rows, splits] both pairs
    const float* g;
    void* dx;
    int64_t dx_stride;
    uint32_t* status;
};

// ------------------------------------------------------------ running sums

struct Sum {
    float m, s;
};

struct Sums {
    Sum other, named;
};

__device__ __forceinline__ Sum sum_empty() { return {-FLT_MAX, 0.0f}; }

__device__ __forceinline__ Sum sum_join(const Sum& a, const Sum& b, float k2) {
    const float m = fmaxf(a.m, b.m);
    // a NaN in (a.m - m) can only come from m = inf, where s is a NaN already
    return {m, a.s * exp2_fast((a.m - m) * k2) + b.s * exp2_fast((b.m - m) * k2)};
}

template <int N>
__device__ __forceinline__ void sum_add(Sum& st, const float (&v)[N], float k2) {
    float cm = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) cm = fmaxf(cm, v[i]);
    const float m = fmaxf(st.m, cm);
    st.s *= exp2_fast((st.m - m) * k2);
    st.m = m;
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        s0 += exp2_fast((v[i] - m) * k2);
        s1 += exp2_fast((v[i + 1] - m) * k2);
    }
    st.s += s0 + s1;
}

template <int MASK>
__device__ __forceinline__ void sum_xor(Sum& st, float k2) {
    const Sum o = {lane_xor<MASK>(st.m), lane_xor<MASK>(st.s)};
    // in the order of the lanes, so that both partners get the same bits
    st = (__lane_id() & uint32_t(MASK)) ? sum_join(o, st, k2) : sum_join(st, o, k2);
}

__device__ __forceinline__ Sum sum_wave(Sum st, float k2) {
    sum_xor<32>(st, k2);
    sum_xor<16>(st, k2);
    sum_xor<8>(st, k2);
    sum_xor<4>(st, k2);
    sum_xor<2>(st, k2);
    sum_xor<1>(st, k2);
    return st;
}

__device__ __forceinline__ float add_wave(float v) {
    v += lane_xor<32>(v);
    v += lane_xor<16>(v);
    v += lane_xor<8>(v);
    v += lane_xor<4>(v);
    v += lane_xor<2>(v);
    v += lane_xor<1>(v);
    return v;
}

// The block's sums, in every thread; `s` is this call's own LDS.
template <int BLOCK>
__device__ __forceinline__ Sums sums_block(Sums st, float k2, Sums* s) {
    st.other = sum_wave(st.other, k2);
    st.named = sum_wave(st.named, k2);
    if constexpr (BLOCK == kWave) return st;
    if ((threadIdx.x & 63u) == 0u) s[threadIdx.x >> 6] = st;
    __syncthreads();
    st = s[0];
#pragma unroll
    for (int w = 1; w < BLOCK / kWave; ++w) {
        st.other = sum_join(st.other, s[w].other, k2);
        st.named = sum_join(st.named, s[w].named, k2);
    }
    return st;
}

// ------------------------------------------------------------ the teacher's places

// A row's places in (dynamic) LDS: ids (-1: not used), logarithms of the probabilities as given, the probabilities
// (exp(lp - shift)), the student's logits, and the marks of the vectors of a part of the row.
struct Places {
    int32_t* id;
    float* p;
    float* lp;
    float* x;
    uint32_t* marks;
};

__device__ __forceinline__ Places places_lds(uint32_t k) {
    extern __shared__ uint32_t s_places[];
    float* f = reinterpret_cast<float*>(s_places + k);
    return {reinterpret_cast<int32_t*>(s_places), f, f + k, f + 2u * k, s_places + 4u * k};
}

static size_t places_bytes(uint32_t k, uint32_t vectors) {
    const uint32_t marked = vectors < kSegment ? vectors : kSegment;
    return size_t(k) * 16 + (marked + 3) / 4 * 4;
}

__device__ __forceinline__ int64_t place_id(const DsArgs& a, uint64_t i) {
    return a.i64 ? static_cast<const int64_t*>(a.idx)[i] : int64_t(static_cast<const int32_t*>(a.idx)[i]);
}

__device__ __forceinline__ float max_wave(float v) {
    v = fmaxf(v, lane_xor<32>(v));
    v = fmaxf(v, lane_xor<16>(v));
    v = fmaxf(v, lane_xor<8>(v));
    v = fmaxf(v, lane_xor<4>(v));
    v = fmaxf(v, lane_xor<2>(v));
    return fmaxf(v, lane_xor<1>(v));
}

// The thread's number, but nothing that is formed from it is kept for another use (no instruction): what the rare path
// of a call forms early would cost the kernel a register until its end, and the step to the next occupancy.
__device__ __forceinline__ uint32_t thread_here() {
    uint32_t t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}

// What the places' logarithms are less in their probabilities: the row's largest if these are divided by their sum
// (-FLT_MAX where all are -inf, whose exponentials stay 0), else 0.  By a wave.
__device__ __forceinline__ float places_shift(const DsArgs& a, const Places& pl) {
    if (a.tail != E8Q_TAIL_RENORM) return 0.0f;
    float most = -FLT_MAX;
    for (uint32_t j = thread_here() & 63u; j < a.k; j += kWave) most = pl.id[j] >= 0 ? fmaxf(most, pl.lp[j]) : most;
    return max_wave(most);
}

// Fills the places; whether one of them is used (a barrier for the whole block; the probabilities are there after the
// next one).
template <typename T>
__device__ __forceinline__ bool load_places(const DsArgs& a, uint32_t row, const T* x, const Places& pl) {
    uint32_t flags = 0u;
    int any = 0;
    for (uint32_t j = threadIdx.x; j < a.k; j += blockDim.x) {
        const int64_t t = place_id(a, uint64_t(row) * a.k + j);
        const float lp = a.lp[uint64_t(row) * a.k + j];
        const bool live = t >= 0 && t < int64_t(a.vocab);
        if (t >= int64_t(a.vocab)) flags |= E8Q_STATUS_BAD_INDEX;
        pl.id[j] = live ? int32_t(t) : -1;
        pl.p[j] = live ? expf(lp) : 0.0f;
        pl.lp[j] = lp;
        pl.x[j] = live ? widen(x[t]) : 0.0f;
        any |= int(live);
    }
    flush_status(flags, a.status);
    any = __syncthreads_or(any);
    if (a.tail == E8Q_TAIL_RENORM) {
        const float shift = places_shift(a, pl);
        for (uint32_t j = thread_here(); j < a.k; j += blockDim.x) pl.p[j] = pl.id[j] >= 0 ? expf(pl.lp[j] - shift) : 0.0f;
    }
    return any != 0;
}

// Marks the named elements of the vectors [lo, hi), at most kSegment of them; whether places share one.
template <typename T>
__device__ __forceinline__ bool mark_places(const Places& pl, uint32_t k, uint32_t lo, uint32_t hi) {
    constexpr uint32_t VE = kVec<T>;
    for (uint32_t w = threadIdx.x; w < (hi - lo + 3u) / 4u; w += blockDim.x) pl.marks[w] = 0u;
    __syncthreads();
    int shared = 0;
    for (uint32_t j = threadIdx.x; j < k; j += blockDim.x) {
        const int32_t id = pl.id[j];
        const uint32_t v = uint32_t(id) / VE;
        if (id < 0 || v < lo || v >= hi) continue;
        const uint32_t bit = 1u << (((v - lo) & 3u) * 8u + uint32_t(id) % VE);
        shared |= int((atomicOr(&pl.marks[(v - lo) >> 2], bit) & bit) != 0u);
    }
    return __syncthreads_or(shared) != 0;
}

// Whether places share an element, where nothing is marked: they are entered into an open table, in place
// of the marks.
__host__ __device__ inline uint32_t places_slots(uint32_t k) {
    uint32_t n = 4u;
    while (n < 2u * k) n *= 2u;
    return n;
}

__device__ __forceinline__ bool places_share(const Places& pl, uint32_t k) {
    const uint32_t slots = places_slots(k);
    for (uint32_t i = threadIdx.x; i < slots; i += blockDim.x) pl.marks[i] = 0u;
    __syncthreads();
    int shared = 0;
    for (uint32_t j = threadIdx.x; j < k; j += blockDim.x) {
        const uint32_t key = uint32_t(pl.id[j]) + 1u;      // 0: not used
        if (key == 0u) continue;
        for (uint32_t at = key * 2654435761u >> 16, old = 1u; old != 0u; ++at) {
            old = atomicCAS(&pl.marks[at % slots], 0u, key);
            if (old == key) {
                shared = 1;
                break;
            }
        }
    }
    return __syncthreads_or(shared) != 0;
}

// Whether no place before j names its element.
__device__ __forceinline__ bool first_of(const Places& pl, uint32_t j) {
    const int32_t id = pl.id[j];
    for (uint32_t i = 0u; i < j; ++i)
        if (pl.id[i] == id) return false;
    return true;
}

// Calls go(j) for a place of each named element of the vectors [lo, hi), a thread each.
template <typename T, class Go>
__device__ __forceinline__ void each_named(const Places& pl, uint32_t k, uint32_t lo, uint32_t hi, bool shared, Go&& go) {
    for (uint32_t j = threadIdx.x; j < k; j += blockDim.x) {
        const int32_t id = pl.id[j];
        const uint32_t v = uint32_t(id) / kVec<T>;
        if (id >= 0 && v >= lo && v < hi && !(shared && !first_of(pl, j))) go(j, id);
    }
}

__device__ __forceinline__ uint32_t marks_of(const Places& pl, uint32_t v) {
    return reinterpret_cast<const uint8_t*>(pl.marks)[v];
}

// Adds the elements of N vectors that no place names; `marks` has a byte for each vector.
template <typename T, int N>
__device__ __forceinline__ void add_others(Sum& st, float (&v)[N * kVec<T>], const uint32_t (&marks)[N], float k2) {
    constexpr int VE = kVec<T>;
#pragma unroll
    for (int u = 0; u < N; ++u) {
        if (!__ballot(marks[u] != 0u)) continue;
#pragma unroll
        for (int i = 0; i < VE; ++i) v[u * VE + i] = (marks[u] >> i) & 1u ? -INFINITY : v[u * VE + i];
    }
    sum_add(st, v, k2);
}

// Adds the named elements of the vectors [lo, hi).
template <typename T>
__device__ __forceinline__ void add_named(Sum& st, const Places& pl, uint32_t k, uint32_t lo, uint32_t hi, bool shared,
                                          float k2) {
    each_named<T>(pl, k, lo, hi, shared, [&](uint32_t j, int32_t) {
        const float x = pl.x[j], m = fmaxf(st.m, x);
        st.s = st.s * exp2_fast((st.m - m) * k2) + exp2_fast((x - m) * k2);
        st.m = m;
    });
}

// Vector j of a row; -inf behind its end.
template <typename T>
__device__ __forceinline__ u32x4_t load_raw(const T* x, uint32_t vocab, uint32_t j) {
    constexpr int VE = kVec<T>;
    const uint32_t e0 = j * VE;
    if (e0 + VE <= vocab) return reinterpret_cast<const RowVec<T>*>(x + e0)->v;
    float v[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) v[i] = e0 + i < vocab ? widen(x[e0 + i]) : -INFINITY;
    return pack(v);
}

// Both sums of the vectors [lo, hi) of a row (all threads end with the block's).
template <typename T, int BLOCK, int UNROLL>
__device__ __forceinline__ Sums row_sums(const DsArgs& a, const T* row, uint32_t lo, uint32_t hi, float k2,
                                         const Places& pl, bool& shared) {
    constexpr int VE = kVec<T>, kGroup = 2;      // vectors unpacked at a time
    __shared__ Sums s_sums[BLOCK / kWave];
    const uint32_t wave0 = uint32_t(__builtin_amdgcn_readfirstlane(int(threadIdx.x & ~63u)));
    Sums st = {sum_empty(), sum_empty()};
    for (uint32_t seg = lo; seg < hi; seg += kSegment) {
        const uint32_t end = min(hi, seg + kSegment);
        if (seg > lo) __syncthreads();               // the marks before are read
        const bool sh = mark_places<T>(pl, a.k, seg, end);
        shared |= sh;
        for (uint32_t base = seg; base < end; base += BLOCK * UNROLL) {
            u32x4_t raw[UNROLL];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                raw[u] = u32x4_t{0u, 0u, 0u, 0u};
                if (base + u * BLOCK + wave0 < end)
                    raw[u] = load_raw<T>(row, a.vocab, min(base + u * BLOCK + threadIdx.x, end - 1u));
            }
#pragma unroll
            for (int u = 0; u < UNROLL; u += kGroup) {
                if (base + u * BLOCK + wave0 >= end) break;      // nothing left for this wave
                float v[kGroup * VE];
                uint32_t marks[kGroup];
#pragma unroll
                for (int g = 0; g < kGroup; ++g) {
                    const uint32_t j = base + (u + g) * BLOCK + threadIdx.x;
                    float w[VE];
                    unpack(raw[u + g], w);
                    marks[g] = j < end ? marks_of(pl, j - seg) : 0xFFu;
#pragma unroll
                    for (int i = 0; i < VE; ++i) v[g * VE + i] = w[i];
                }
                add_others<T, kGroup>(st.other, v, marks, k2);
                __builtin_amdgcn_sched_barrier(0);       // one group unpacked at a time
            }
        }
        add_named<T>(st.named, pl, a.k, seg, end, sh, k2);
    }
    return sums_block<BLOCK>(st, k2, s_sums);
}

// ------------------------------------------------------------ a row's end

// What the gradient needs of a row: maxima and sums, of all elements and of those that no place names.  The sums
// themselves and not their logarithms, which would be rounded to 2^-20 of q for the whole row.
struct RowStats {
    float m, s, m_other, s_other;
};

__device__ __forceinline__ RowStats row_stats(const Sums& st, float k2) {
    const Sum all = sum_join(st.other, st.named, k2);
    return {all.m, all.s, st.other.m, st.other.s};
}

// The teacher's side of a row: sum of the probabilities (less the shift), the factor to the weights
// used, its logarithm, and the weight left to the rest.  The same in every wave.
struct Teacher {
    float mass, factor, log_factor, rest, total;
};

__device__ __forceinline__ Teacher teacher_row(const DsArgs& a, const Places& pl, const RowStats& st) {
    float mass = 0.0f;
    for (uint32_t j = threadIdx.x & 63u; j < a.k; j += kWave) mass += pl.p[j];
    mass = add_wave(mass);
    if (__builtin_isinf(mass)) mass = __uint_as_float(0x7FC00000u);
    Teacher t = {mass, 1.0f, 0.0f, 0.0f, mass};
    if (a.tail == E8Q_TAIL_RENORM) {
        t.factor = mass > 0.0f ? 1.0f / mass : mass;       // no mass: no weights (a NaN stays one)
        t.log_factor = -logf(mass);
        t.total = mass > 0.0f ? 1.0f : mass;
    } else if (a.tail == E8Q_TAIL_REST && st.s_other != 0.0f) {
        t.rest = fmaxf(0.0f, 1.0f - mass);
        t.total = mass + t.rest;
    }
    return t;
}

// log q_r.
__device__ __forceinline__ float log_rest(const RowStats& st, float scale) {
    return (st.m_other - st.m) * scale + logf(st.s_other / st.s);
}

// Loss and log probabilities of a row, by wave 0 of one block.
__device__ __forceinline__ void write_row(const DsArgs& a, uint32_t row, const RowStats& st, const Teacher& t,
                                          const Places& pl) {
    if (threadIdx.x >= kWave) return;
    const float ln_s = logf(st.s), shift = places_shift(a, pl);
    float loss = 0.0f;
    for (uint32_t j = threadIdx.x; j < a.k; j += kWave) {
        const int32_t id = pl.id[j];
        float lq = 0.0f;
        if (id >= 0) {
            lq = st.s == 0.0f ? -INFINITY : (pl.x[j] - st.m) * a.scale - ln_s;
            const float p = pl.p[j];
            if (!(p == 0.0f)) loss += p * t.factor * (pl.lp[j] - shift + t.log_factor - lq);
        }
        if (a.logprob) a.logprob[uint64_t(row) * a.k + j] = lq;
    }
    loss = add_wave(loss);
    if (t.mass != t.mass) loss = t.mass;
    if (st.s != st.s) loss = st.s;                         // (a NaN or +inf among the logits, also where every p is 0)
    if (t.rest > 0.0f) loss += t.rest * (logf(t.rest) - log_rest(st, a.scale));
    if (threadIdx.x == 0u) {
        if (a.loss) a.loss[row] = loss;
        if (a.stats) a.stats[row] = make_float4(st.m, st.s, st.m_other, st.s_other);
        if (loss != loss || st.s != st.s) atomicOr(a.status, uint32_t(E8Q_STATUS_NONFINITE));
    }
}

// A row without a used place: loss 0, gradient 0, whatever its logits.
__device__ __forceinline__ void write_empty(const DsArgs& a, uint32_t row) {
    if (a.logprob)
        for (uint32_t j = threadIdx.x; j < a.k; j += blockDim.x) a.logprob[uint64_t(row) * a.k + j] = 0.0f;
    if (threadIdx.x == 0u) {
        if (a.loss) a.loss[row] = 0.0f;
        if (a.stats) a.stats[row] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
}

// ------------------------------------------------------------ forward

template <typename T>
__global__ __launch_bounds__(kLpBlock) void distill_kernel(DsArgs a) {
    const Places pl = places_lds(a.k);
    const uint32_t row = a.splits == 1 ? blockIdx.x : blockIdx.x / a.splits;
    const uint32_t sp = blockIdx.x - row * a.splits;
    const T* x = static_cast<const T*>(a.x) + int64_t(row) * a.stride;
    const uint32_t nvec = (a.vocab + kVec<T> - 1) / kVec<T>;
    const uint32_t lo = min(sp * a.per_split, nvec), hi = min(lo + a.per_split, nvec);
    const float k2 = a.scale * kLog2e;
    if (!load_places<T>(a, row, x, pl)) {
        if (a.splits == 1) write_empty(a, row);
        return;
    }
    bool shared = false;
    const Sums st = row_sums<T, kLpBlock, kLpUnroll>(a, x, lo, hi, k2, pl, shared);
    if (a.splits > 1) {
        if (threadIdx.x == 0u) a.part[blockIdx.x] = make_float4(st.other.m, st.other.s, st.named.m, st.named.s);
        return;
    }
    const RowStats rs = row_stats(st, k2);
    write_row(a, row, rs, teacher_row(a, pl, rs), pl);
}

// Joins the parts of one row.
template <typename T>
__global__ __launch_bounds__(kLpBlock) void distill_join_kernel(DsArgs a) {
    __shared__ Sums s_sums[kLpBlock / kWave];
    const Places pl = places_lds(a.k);
    const uint32_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + int64_t(row) * a.stride;
    const float k2 = a.scale * kLog2e;
    Sums st = {sum_empty(), sum_empty()};
    if (!load_places<T>(a, row, x, pl)) {
        write_empty(a, row);
        return;
    }
    if (threadIdx.x < a.splits) {
        const float4 p = a.part[uint64_t(row) * a.splits + threadIdx.x];
        st = {{p.x, p.y}, {p.z, p.w}};
    }
    st = sums_block<kLpBlock>(st, k2, s_sums);
    const RowStats rs = row_stats(st, k2);
    write_row(a, row, rs, teacher_row(a, pl, rs), pl);
}

// ------------------------------------------------------------ gradient

// The row's constants: c exp2((x - m) k2) outside K; cq exp2((x - m_all) k2) - cw w inside.
struct GradRow {
    float c, m, cq, m_all, cw, k2;
    bool empty;                 // all logits are -inf
};

__device__ __forceinline__ GradRow grad_row(const DsArgs& a, const RowStats& st, const Teacher& t, float g) {
    const float up = a.scale * g;
    GradRow r = {up * t.total / st.s, st.m, up * t.total / st.s, st.m, up * t.factor, a.scale * kLog2e, st.s == 0.0f};
    if (st.s_other == 0.0f) {                          // all others are -inf: exp2 gives their 0, but for a NaN row's
        r.c = r.c == r.c || r.empty ? 0.0f : r.c;
        r.m = 0.0f;
    } else if (t.rest > 0.0f) {
        const float rest = exp2_fast((st.m_other - st.m) * r.k2) * (st.s_other / st.s);
        r.c = up * (t.total * rest - t.rest) / st.s_other;
        r.m = st.m_other;
    }
    return r;
}

// The gradient of one vector, as if no place named an element of it.
template <typename T>
__device__ __forceinline__ void grad_store(const DsArgs& a, T* dx, uint32_t e0, const u32x4_t& raw, const GradRow& r) {
    float v[kVec<T>];
    unpack(raw, v);
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i) v[i] = r.c * exp2_fast((v[i] - r.m) * r.k2);
    store_grad<T>(dx, a.vocab, e0, v);
}

// Then the named elements of the vectors [lo, hi), after a barrier: over what grad_store left there.
template <typename T>
__device__ __forceinline__ void grad_named(const DsArgs& a, T* dx, uint32_t lo, uint32_t hi, bool shared,
                                           const GradRow& r, const Places& pl) {
    __syncthreads();
    each_named<T>(pl, a.k, lo, hi, shared, [&](uint32_t j, int32_t id) {
        float w = pl.p[j];
        if (shared) {                                      // every place that names it
            double sum = 0.0;
            for (uint32_t i = 0u; i < a.k; ++i) sum += pl.id[i] == id ? pl.p[i] : 0.0f;
            w = float(sum);
        }
        const float q = exp2_fast((pl.x[j] - r.m_all) * r.k2);
        dx[id] = narrow<T>(r.empty ? 0.0f : r.cq * q - r.cw * w);
    });
}

// The vectors [lo, hi) of the gradient row.
template <typename T, int UNROLL>
__device__ __forceinline__ void grad_part(const DsArgs& a, const T* x, T* dx, uint32_t lo, uint32_t hi,
                                          const GradRow& r, const Places& pl, bool shared) {
    const uint32_t step = blockDim.x * UNROLL;
    for (uint32_t left = (hi - lo + step - 1u) / step; left-- > 0u;) {
        const uint32_t base = lo + left * step;
        u32x4_t raw[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const uint32_t j = base + u * blockDim.x + threadIdx.x;
            raw[u] = u32x4_t{0u, 0u, 0u, 0u};
            if (j < hi) raw[u] = load_raw<T>(x, a.vocab, j);
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const uint32_t j = base + u * blockDim.x + threadIdx.x;
            if (j < hi) grad_store<T>(a, dx, j * kVec<T>, raw[u], r);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    grad_named<T>(a, dx, lo, hi, shared, r, pl);
}

template <typename T>
__device__ __forceinline__ void zero_part(const DsArgs& a, T* dx, uint32_t lo, uint32_t hi) {
    float v[kVec<T>];
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i) v[i] = 0.0f;
    for (uint32_t j = lo + threadIdx.x; j < hi; j += blockDim.x) store_grad<T>(dx, a.vocab, j * kVec<T>, v);
}

// From the stored statistics.
template <typename T>
__global__ __launch_bounds__(kLpBlock) void distill_backward_kernel(DsArgs a) {
    const Places pl = places_lds(a.k);
    const uint32_t row = a.splits == 1 ? blockIdx.x : blockIdx.x / a.splits;
    const uint32_t sp = blockIdx.x - row * a.splits;
    const T* x = static_cast<const T*>(a.x) + int64_t(row) * a.stride;
    T* dx = static_cast<T*>(a.dx) + int64_t(row) * a.dx_stride;
    const uint32_t nvec = (a.vocab + kVec<T> - 1) / kVec<T>;
    const uint32_t lo = min(sp * a.per_split, nvec), hi = min(lo + a.per_split, nvec);
    const float4 s = a.stats[row];
    const float g = a.g[row];
    if (!load_places<T>(a, row, x, pl)) {
        zero_part<T>(a, dx, lo, hi);
        return;
    }
    const RowStats rs = {s.x, s.y, s.z, s.w};
    const bool shared = places_share(pl, a.k);
    grad_part<T, kLpUnroll>(a, x, dx, lo, hi, grad_row(a, rs, teacher_row(a, pl, rs), g), pl, shared);
}

// Sums (and gradient) of a row that fits the registers of one block, NV vectors a
// thread: the row is read once, and before the places are.
template <typename T, int BLOCK, int NV, bool GRAD>
__global__ __launch_bounds__(BLOCK) void distill_row_kernel(DsArgs a) {
    constexpr int VE = kVec<T>, kGroup = 2;      // vectors unpacked at a time
    __shared__ Sums s_sums[BLOCK / kWave];
    const Places pl = places_lds(a.k);
    const uint32_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + int64_t(row) * a.stride;
    T* dx = static_cast<T*>(a.dx) + int64_t(row) * a.dx_stride;
    const uint32_t nvec = (a.vocab + VE - 1) / VE;
    const uint32_t wave0 = uint32_t(__builtin_amdgcn_readfirstlane(int(threadIdx.x & ~63u)));
    u32x4_t raw[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) raw[n] = load_raw<T>(x, a.vocab, n * BLOCK + threadIdx.x);
    const float g = GRAD ? a.g[row] : 0.0f;
    if (!load_places<T>(a, row, x, pl)) {
        write_empty(a, row);
        if constexpr (GRAD) zero_part<T>(a, dx, 0u, nvec);
        return;
    }
    const bool shared = mark_places<T>(pl, a.k, 0u, nvec);
    const float k2 = a.scale * kLog2e;
    Sums st = {sum_empty(), sum_empty()};
#pragma unroll
    for (int n = 0; n < NV; n += kGroup) {
        if (uint32_t(n * BLOCK) + wave0 >= nvec) break;        // nothing of the row for this wave any more
        float v[kGroup * VE];
        uint32_t marks[kGroup];
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
            const uint32_t j = (n + u) * BLOCK + threadIdx.x;
            float w[VE];
            unpack(raw[n + u], w);
#pragma unroll
            for (int i = 0; i < VE; ++i) v[u * VE + i] = w[i];
            marks[u] = j < nvec ? marks_of(pl, j) : 0u;
        }
        add_others<T, kGroup>(st.other, v, marks, k2);
        __builtin_amdgcn_sched_barrier(0);       // one group unpacked at a time
    }
    add_named<T>(st.named, pl, a.k, 0u, nvec, shared, k2);
    st = sums_block<BLOCK>(st, k2, s_sums);
    const RowStats rs = row_stats(st, k2);
    const Teacher t = teacher_row(a, pl, rs);
    write_row(a, row, rs, t, pl);
    if constexpr (!GRAD) return;
    const GradRow r = grad_row(a, rs, t, g);
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        if (uint32_t(n * BLOCK) + wave0 >= nvec) break;
        const uint32_t j = n * BLOCK + threadIdx.x;
        if (j < nvec) grad_store<T>(a, dx, j * VE, raw[n], r);
        __builtin_amdgcn_sched_barrier(0);
    }
    grad_named<T>(a, dx, 0u, nvec, shared, r, pl);
}

// The same for longer rows: two passes over the row.
template <typename T>
__global__ __launch_bounds__(kLpWide, 8) void distill_grad_long_kernel(DsArgs a) {
    const Places pl = places_lds(a.k);
    const uint32_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + int64_t(row) * a.stride;
    T* dx = static_cast<T*>(a.dx) + int64_t(row) * a.dx_stride;
    const uint32_t nvec = (a.vocab + kVec<T> - 1) / kVec<T>;
    const float g = a.g[row];
    if (!load_places<T>(a, row, x, pl)) {
        write_empty(a, row);
        zero_part<T>(a, dx, 0u, nvec);
        return;
    }
    const float k2 = a.scale * kLog2e;
    bool shared = false;
    const Sums st = row_sums<T, kLpWide, kLpUnroll>(a, x, 0u, nvec, k2, pl, shared);
    const RowStats rs = row_stats(st, k2);
    const Teacher t = teacher_row(a, pl, rs);
    write_row(a, row, rs, t, pl);
    grad_part<T, kLpUnroll>(a, x, dx, 0u, nvec, grad_row(a, rs, t, g), pl, shared);
}

// ------------------------------------------------------------ host

static e8q_status_t ds_check(const void* logits, e8q_dtype_t dtype, int64_t rows, int64_t vocab, int64_t stride,
                             float scale, const void* idx, e8q_index_t index_type, const float* lp, int64_t k,
                             int32_t tail, uint32_t* status) {
    if (!logits || !idx || !lp || !status || rows <= 0 || vocab <= 0 || stride < vocab || k <= 0) return E8Q_ERR_INVALID;
    if (dtype != E8Q_F32 && dtype != E8Q_BF16) return E8Q_ERR_INVALID;
    if (!(scale > 0.0f) || __builtin_isinf(scale)) return E8Q_ERR_INVALID;
    if (index_type != E8Q_I32 && index_type != E8Q_I64) return E8Q_ERR_INVALID;
    if (tail != E8Q_TAIL_NONE && tail != E8Q_TAIL_RENORM && tail != E8Q_TAIL_REST) return E8Q_ERR_INVALID;
    const size_t esz = dtype == E8Q_BF16 ? 2 : 4, isz = index_type == E8Q_I64 ? 8 : 4;
    if (reinterpret_cast<uintptr_t>(logits) % esz || reinterpret_cast<uintptr_t>(idx) % isz ||
        reinterpret_cast<uintptr_t>(lp) % 4)
        return E8Q_ERR_INVALID;
    if (vocab >= (int64_t(1) << 31) - 16 || rows >= kMaxRows || k > kMaxPlaces || stride >= (int64_t(1) << 40))
        return E8Q_ERR_UNSUPPORTED;
    return E8Q_OK;
}

static e8q_status_t ds_check_grad(const void* logits, int64_t vocab, int64_t row_stride, const float* grad_loss,
                                  const void* grad_logits, int64_t grad_stride, e8q_dtype_t dtype) {
    if (!grad_loss || !grad_logits || grad_stride < vocab) return E8Q_ERR_INVALID;
    if (grad_logits == logits && grad_stride != row_stride) return E8Q_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(grad_logits) % (dtype == E8Q_BF16 ? 2 : 4)) return E8Q_ERR_INVALID;
    return grad_stride >= (int64_t(1) << 40) ? E8Q_ERR_UNSUPPORTED : E8Q_OK;
}

static DsArgs ds_args(const void* logits, int64_t rows, int64_t vocab, int64_t stride, float scale, const void* idx,
                      e8q_index_t index_type, const float* lp, int64_t k, int32_t tail, uint32_t* status) {
    DsArgs a{};
    a.x = logits;
    a.stride = stride;
    a.rows = uint32_t(rows);
    a.vocab = uint32_t(vocab);
    a.scale = scale;
    a.idx = idx;
    a.i64 = index_type == E8Q_I64;
    a.lp = lp;
    a.k = uint32_t(k);
    a.tail = tail;
    a.status = status;
    return a;
}

static uint32_t ds_vectors(int64_t vocab, size_t esz) { return uint32_t((uint64_t(vocab) * esz + 15) / 16); }

static size_t ds_part_bytes(uint64_t blocks) { return size_t((blocks * sizeof(float4) + 255) / 256 * 256); }

// Longest rows that every call keeps in registers, and that need no workspace.
constexpr uint32_t kRowVectors = 256 * 16;

// The parts' sums and the rows' statistics.  One size for the loss alone and for the one call with the gradient: the latter
// does not use it for rows of 512 x 16 vectors.
static size_t ds_workspace(int64_t rows, int64_t vocab, size_t esz) {
    uint32_t per = 0;
    const uint64_t splits = lp_splits(rows, vocab, esz, per);
    return splits == 1 || ds_vectors(vocab, esz) <= kRowVectors ? 0 : ds_part_bytes(uint64_t(rows) * splits) + size_t(rows) * sizeof(float4);
}

// Rows that the registers of one block hold: the smallest such block; whether there is one.  512 x 16 vectors are for
// float32 gradients only: the loss alone of such rows takes the split passes (301 rows of 32003: 11.7 + 4.5 us).
template <typename T, bool GRAD, class Go>
static bool ds_row_kernel(int64_t vocab, Go&& go) {
    const uint32_t nvec = ds_vectors(vocab, sizeof(T));
    if (nvec <= 64 * 4) go(distill_row_kernel<T, 64, 4, GRAD>, 64u);
    else if (nvec <= 128 * 4) go(distill_row_kernel<T, 128, 4, GRAD>, 128u);
    else if (nvec <= 256 * 4) go(distill_row_kernel<T, 256, 4, GRAD>, 256u);
    else if (nvec <= 256 * 8) go(distill_row_kernel<T, 256, 8, GRAD>, 256u);
    else if (nvec <= kRowVectors) go(distill_row_kernel<T, 256, 16, GRAD>, 256u);
    else if (sizeof(T) == 4 && GRAD && nvec <= 512 * 16) go(distill_row_kernel<T, 512, 16, GRAD>, 512u);
    else return false;
    return true;
}

template <typename T, bool GRAD>
static bool ds_rows(DsArgs& a, hipStream_t st) {
    return ds_row_kernel<T, GRAD>(a.vocab, [&](auto kernel, unsigned block) {
        launch(kernel, dim3(a.rows), dim3(block), places_bytes(a.k, ds_vectors(a.vocab, sizeof(T))), st, a);
    });
}

template <typename T>
static void ds_forward(DsArgs& a, void* ws, hipStream_t st) {
    a.splits = lp_splits(a.rows, a.vocab, sizeof(T), a.per_split);
    a.part = static_cast<float4*>(ws);
    // one launch for the rows that registers hold: few rows (16 of 9000 bf16 logits 12.3 us in two, 9.5) or short ones;
    // many longer ones are as fast in one pass without (4000 of 32000: 50.5 us, 53.5)
    const bool few = a.splits > 1 || ds_vectors(a.vocab, sizeof(T)) <= 256 * 4;
    if (few && ds_rows<T, false>(a, st)) return;
    launch(distill_kernel<T>, dim3(a.rows * a.splits), dim3(kLpBlock), places_bytes(a.k, a.per_split), st, a);
    if (a.splits > 1) launch(distill_join_kernel<T>, dim3(a.rows), dim3(kLpBlock), places_bytes(a.k, 0), st, a);
}

template <typename T>
static void ds_backward(DsArgs& a, hipStream_t st) {
    a.splits = lp_splits(a.rows, a.vocab, sizeof(T), a.per_split);
    launch(distill_backward_kernel<T>, dim3(a.rows * a.splits), dim3(kLpBlock),
           places_bytes(a.k, 0) + size_t(places_slots(a.k)) * 4, st, a);
}

// A launch has fewer than 2^32 threads.
template <typename T>
static bool ds_grad_fits(int64_t rows, int64_t vocab) {
    unsigned threads = kLpWide;
    ds_row_kernel<T, true>(vocab, [&](auto, unsigned block) { threads = block; });
    return uint64_t(rows) * threads < uint64_t(1) << 32;
}

template <typename T>
static e8q_status_t ds_both(DsArgs& a, void* ws, size_t need, hipStream_t st) {
    if (!ds_grad_fits<T>(a.rows, a.vocab)) return E8Q_ERR_UNSUPPORTED;
    // one launch wherever registers hold a row (16 rows of 9000 bf16 logits 18.2 us in three, 10.5; 500 of 32000 float32
    // ones 42.7, 25.4)
    if (ds_rows<T, true>(a, st)) return launch_status();
    if (!need) {
        launch(distill_grad_long_kernel<T>, dim3(a.rows), dim3(kLpWide), places_bytes(a.k, ds_vectors(a.vocab, sizeof(T))),
               st, a);
        return launch_status();
    }
    // few long rows: the split passes, with the rows' statistics in the workspace
    a.stats = reinterpret_cast<float4*>(static_cast<char*>(ws) + need - size_t(a.rows) * sizeof(float4));
    ds_forward<T>(a, ws, st);
    ds_backward<T>(a, st);
    return launch_status();
}

static bool ds_workspace_bad(const void* ws, size_t bytes, size_t need) {
    return need && (!ws || bytes < need || reinterpret_cast<uintptr_t>(ws) % 256);
}

}  // namespace e8q

extern "C" size_t e8q_distill_workspace_size(int64_t rows, int64_t vocab, int64_t k) {
    using namespace e8q;
    if (rows <= 0 || vocab <= 0 || k <= 0 || k > kMaxPlaces || rows >= kMaxRows || vocab >= (int64_t(1) << 31) - 16)
        return 0;
    const size_t b = ds_workspace(rows, vocab, 2), f = ds_workspace(rows, vocab, 4);
    return b > f ? b : f;
}

extern "C" e8q_status_t e8q_distill(const void* logits, e8q_dtype_t dtype, int64_t rows, int64_t vocab,
                                    int64_t row_stride, float scale, const void* teacher_idx, e8q_index_t index_type,
                                    const float* teacher_logprob, int64_t k, int32_t tail, float* loss_out,
                                    float* logprob_out, float* stats_out, void* workspace, size_t workspace_bytes,
                                    uint32_t* status_dev, void* stream) {
    using namespace e8q;
    const e8q_status_t st = ds_check(logits, dtype, rows, vocab, row_stride, scale, teacher_idx, index_type,
                                     teacher_logprob, k, tail, status_dev);
    if (st != E8Q_OK) return st;
    if (!loss_out && !logprob_out && !stats_out) return E8Q_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(stats_out) % 16) return E8Q_ERR_INVALID;
    if (ds_workspace_bad(workspace, workspace_bytes, ds_workspace(rows, vocab, dtype == E8Q_BF16 ? 2 : 4)))
        return E8Q_ERR_INVALID;
    DsArgs a = ds_args(logits, rows, vocab, row_stride, scale, teacher_idx, index_type, teacher_logprob, k, tail,
                       status_dev);
    a.loss = loss_out;
    a.logprob = logprob_out;
    a.stats = reinterpret_cast<float4*>(stats_out);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (dtype == E8Q_BF16) ds_forward<uint16_t>(a, workspace, s);
    else ds_forward<float>(a, workspace, s);
    return launch_status();
}

extern "C" e8q_status_t e8q_distill_backward(const void* logits, e8q_dtype_t dtype, int64_t rows, int64_t vocab,
                                             int64_t row_stride, float scale, const void* teacher_idx,
                                             e8q_index_t index_type, const float* teacher_logprob, int64_t k,
                                             int32_t tail, const float* stats, const float* grad_loss,
                                             void* grad_logits, int64_t grad_stride, uint32_t* status_dev,
                                             void* stream) {
    using namespace e8q;
    e8q_status_t st = ds_check(logits, dtype, rows, vocab, row_stride, scale, teacher_idx, index_type, teacher_logprob,
                               k, tail, status_dev);
    if (st != E8Q_OK) return st;
    if (!stats || reinterpret_cast<uintptr_t>(stats) % 16) return E8Q_ERR_INVALID;
    st = ds_check_grad(logits, vocab, row_stride, grad_loss, grad_logits, grad_stride, dtype);
    if (st != E8Q_OK) return st;
    DsArgs a = ds_args(logits, rows, vocab, row_stride, scale, teacher_idx, index_type, teacher_logprob, k, tail,
                       status_dev);
    a.stats = reinterpret_cast<float4*>(const_cast<float*>(stats));
    a.g = grad_loss;
    a.dx = grad_logits;
    a.dx_stride = grad_stride;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (dtype == E8Q_BF16) ds_backward<uint16_t>(a, s);
    else ds_backward<float>(a, s);
    return launch_status();
}

extern "C" e8q_status_t e8q_distill_grad(const void* logits, e8q_dtype_t dtype, int64_t rows, int64_t vocab,
                                         int64_t row_stride, float scale, const void* teacher_idx,
                                         e8q_index_t index_type, const float* teacher_logprob, int64_t k, int32_t tail,
                                         const float* grad_loss, float* loss_out, float* logprob_out,
                                         void* grad_logits, int64_t grad_stride, void* workspace,
                                         size_t workspace_bytes, uint32_t* status_dev, void* stream) {
    using namespace e8q;
    e8q_status_t st = ds_check(logits, dtype, rows, vocab, row_stride, scale, teacher_idx, index_type, teacher_logprob,
                               k, tail, status_dev);
    if (st != E8Q_OK) return st;
    st = ds_check_grad(logits, vocab, row_stride, grad_loss, grad_logits, grad_stride, dtype);
    if (st != E8Q_OK) return st;
    const size_t need = ds_workspace(rows, vocab, dtype == E8Q_BF16 ? 2 : 4);
    if (ds_workspace_bad(workspace, workspace_bytes, need)) return E8Q_ERR_INVALID;
    DsArgs a = ds_args(logits, rows, vocab, row_stride, scale, teacher_idx, index_type, teacher_logprob, k, tail,
                       status_dev);
    a.loss = loss_out;
    a.logprob = logprob_out;
    a.g = grad_loss;
    a.dx = grad_logits;
    a.dx_stride = grad_stride;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    return dtype == E8Q_BF16 ? ds_both<uint16_t>(a, workspace, need, s) : ds_both<float>(a, workspace, need, s);
}

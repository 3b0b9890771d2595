// e8q_moe_core_escape: a mixture-of-experts layer of a few tokens, straight from
// the exported form (16-bit core indices and escape records).
//
//   p = softmax(W_r x);  e_1 ... e_k the k largest, w_j = p_{e_j} (/ their sum)
//   y = sum_j w_j D_{e_j} ( act(G_{e_j} x) * (U_{e_j} x) ),   G, U, D = R^T (s z).
//
// R is orthogonal, so a product with an expert's matrix is s_r sum_g z_g . x~_g with
// x~ = R x = kappa H (sigma x), as in e8q_gemv_core_escape: x is rotated once, the
// weights never are.  x~ is held in fixed point, N = rint(x~ 2^(22 - e)) with
// 2^(e-1) <= max |x~| < 2^e, written as three signed base-256 digits, and the row sums
// sum 2z N are exact int32 sums on the int8 matrix cores:
//   A (16 x 64): 16 rows x 8 groups of points, a byte for each 2z;
//   B (64 x 16): the same groups' digits, column 3 j + d holding digit d of token j.
// So one sweep over an expert's indices serves five tokens.  The rounding to fixed point,
// |x~ - N 2^(e-22)| <= 2^(e-23) (2^-22 of the largest), is the only one in the product
// besides the last to float32: it keeps three digits because 2^-14 of the largest (two
// digits) would be more than a bfloat16 activation's own rounding in a vector with one
// strong channel.  An escaped slot's 2z has up to 16 bits: its low byte goes into A and,
// where there is one, its high byte into a second product.
//
// Launches: router products (float64: a tie or near-tie must not depend on the order of
// a sum) with the rotation of x beside them; the choice of experts; gate and up of the chosen
// experts with the activation; the rotation of its result; down; the weighted sum, in
// the order of the places.
#include <float.h>

#include "e8q_device.hpp"
#include "e8q_host.hpp"
#include "e8q_vec.hpp"

namespace e8q {

constexpr uint32_t kMoeThreads = 1024, kMoeWaves = 16;
constexpr uint32_t kMoeTile = 16;            // rows of a matrix instruction
constexpr uint32_t kMoeTokens = 5;           // tokens of a sweep: 3 of the 16 columns each
constexpr uint32_t kMoeSlab = 8;             // chunks of 256 columns whose digits are in LDS at a time
constexpr uint32_t kMoeTable = 9216;         // points whose table fits LDS beside them
constexpr int64_t kMoeExperts = 1024, kMoeTopK = 64, kMoeRoutes = 4096, kMoeCols = 32768;
constexpr int kDigitBits = 22;
constexpr int kBadExponent = 1 << 20;        // the exponent of a vector with a NaN or infinity

typedef int moe_i32x4 __attribute__((ext_vector_type(4)));
typedef unsigned short moe_u16x2 __attribute__((ext_vector_type(2)));

struct MoeMatrix {
    const uint16_t* idx;        // [experts, rows, gpr]
    const uint32_t* esc;
    const int64_t* esc_count;
    uint64_t esc_capacity;
    const float* scale;         // [experts, rows]
    const uint64_t* offsets;    // [experts + 1], in the workspace
};

struct MoeArgs {
    const void* x;
    int x_bf16;
    uint32_t tokens, experts, hidden, inter, k;
    const void* router;         // or null: the routes are given
    int router_bf16, normalize, act;
    int32_t* route;             // [tokens, k]
    float* weight;
    double* logits;             // [tokens, experts]
    const int8_t* signs_in;
    const int8_t* signs_down;
    uint32_t had_in, had_down;
    float kappa_in, kappa_down;
    MoeMatrix gate, up, down;
    uint64_t* offsets;          // [3, experts + 1]
    uint8_t* xd;                // digits of x: [tokens] x 3 bytes a (padded) column
    int* xe;                    // their exponents
    float* h;                   // [tokens k, inter]
    uint8_t* hd;
    int* he;
    float* part;                // [tokens k, hidden]
    void* y;
    int y_bf16;
    const uint32_t* pts;
    uint32_t npts;
    uint32_t rows_in, rows_down;     // rows of a block
    uint32_t parts_in, parts_down;   // blocks of an expert
    uint32_t* status;
};

__host__ __device__ inline uint32_t moe_chunks(uint32_t cols) { return (cols + 255u) / 256u; }
__host__ __device__ inline uint64_t moe_digit_bytes(uint32_t cols) { return uint64_t(moe_chunks(cols)) * 768u; }

// ------------------------------------------------------------ rotation and digits

// Eight values from element `i` of a vector of either type, at any element's alignment.
struct __attribute__((packed, aligned(2))) Bytes16 {
    u32x4_t v;
};

__device__ __forceinline__ void load8(const void* p, int bf16, uint64_t i, float (&v)[8]) {
    if (bf16) {
        unpack(reinterpret_cast<const Bytes16*>(static_cast<const uint16_t*>(p) + i)->v, v);
    } else {
        float a[4], b[4];
        const Bytes16* q = reinterpret_cast<const Bytes16*>(static_cast<const float*>(p) + i);
        unpack(q[0].v, a);
        unpack(q[1].v, b);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = a[k];
            v[4 + k] = b[k];
        }
    }
}

template <int MASK>
__device__ __forceinline__ void lane_stage(float (&v)[8], uint32_t lane) {
    const bool upper = lane & uint32_t(MASK);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float o = lane_xor<MASK>(v[i]);
        v[i] = upper ? o - v[i] : v[i] + o;
    }
}

// kappa H (sigma v) of a vector's group `g` (8 columns a thread, consecutive groups in
// consecutive lanes from a multiple of 64 on), blocks of `had` columns (0: none).  Blocks wider than a
// wave's 512 columns go through `s` (8 floats a thread); all threads call it then.
__device__ __forceinline__ void rotate8(float (&v)[8], const int8_t* signs, uint32_t had, float kappa, uint32_t g,
                                        bool live, float* s) {
    if (!had) return;
    const uint32_t lane = threadIdx.x & 63u;
    if (live) apply_signs(signs, g * 8u, v);
    fwht_inlane<8>(v);
    if (had > 8u) lane_stage<1>(v, lane);
    if (had > 16u) lane_stage<2>(v, lane);
    if (had > 32u) lane_stage<4>(v, lane);
    if (had > 64u) lane_stage<8>(v, lane);
    if (had > 128u) lane_stage<16>(v, lane);
    if (had > 256u) lane_stage<32>(v, lane);
    for (uint32_t step = 64u; step * 8u < had; step *= 2u) {         // threads apart
        float4* mine = reinterpret_cast<float4*>(s + threadIdx.x * 8u);
        const float4* other = reinterpret_cast<const float4*>(s + (threadIdx.x ^ step) * 8u);
        mine[0] = make_float4(v[0], v[1], v[2], v[3]);
        mine[1] = make_float4(v[4], v[5], v[6], v[7]);
        __syncthreads();
        const float4 a = other[0], b = other[1];
        const float o[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        const bool upper = threadIdx.x & step;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = upper ? o[i] - v[i] : v[i] + o[i];
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= kappa;
}

__device__ __forceinline__ uint32_t abs_bits(const float (&v)[8]) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return m;
}

// e with 2^(e-1) <= max < 2^e from the bits of the largest |value| (0: 0).
__device__ __forceinline__ int exponent_of(uint32_t bits) {
    if (bits >= 0x7F800000u) return kBadExponent;
    return bits == 0u ? 0 : __builtin_amdgcn_frexp_expf(__uint_as_float(bits));
}

// The three digits of a group, 8 bytes each.
__device__ __forceinline__ void digits8(const float (&v)[8], int e, uint2 (&d)[3]) {
    uint32_t w[3][2] = {{0u, 0u}, {0u, 0u}, {0u, 0u}};
    const bool fin = e != kBadExponent;          // digits of a non-finite vector are not used
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        int n = fin ? int(__builtin_rintf(__builtin_ldexpf(v[i], kDigitBits - e))) : 0;
        const int d2 = int(int8_t(uint8_t(n)));
        n = (n - d2) >> 8;
        const int d1 = int(int8_t(uint8_t(n)));
        const int d0 = (n - d1) >> 8;
        const uint32_t sh = 8u * uint32_t(i & 3);
        w[0][i >> 2] |= (uint32_t(d0) & 0xFFu) << sh;
        w[1][i >> 2] |= (uint32_t(d1) & 0xFFu) << sh;
        w[2][i >> 2] |= (uint32_t(d2) & 0xFFu) << sh;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) d[k] = make_uint2(w[k][0], w[k][1]);
}

// Digits in the order of the sweep: a lane of quarter q takes groups 32 c + 8 q + 2 s, + 1 at
// step s of chunk c, so entry ((c 4 + s) 4 + q) holds both groups' digits, 16 bytes for
// each digit.  Byte offset of a group's half of digit 0 in the vector's entries, `columns` digits apart.
__device__ __forceinline__ uint32_t digit_offset(uint32_t g, uint32_t columns) {
    const uint32_t entry = ((g >> 5) * 4u + ((g >> 1) & 3u)) * 4u + ((g >> 3) & 3u);
    return entry * columns * 16u + (g & 1u) * 8u;
}

// Rotation and digits of one vector by the block: `load` gives a group's values.
template <class Load>
__device__ __forceinline__ void vector_digits(Load&& load, uint32_t cols, const int8_t* signs, uint32_t had, float kappa,
                                              uint8_t* out, int* exponent) {
    constexpr int kPasses = int(kMoeCols / (kMoeThreads * 8));
    __shared__ float4 s_wide4[kMoeThreads * 2];
    float* s_wide = reinterpret_cast<float*>(s_wide4);
    __shared__ uint32_t s_max[kMoeWaves];
    const uint32_t tid = threadIdx.x, groups = cols / 8u, padded = moe_chunks(cols) * 32u;
    float v[kPasses][8];
    uint32_t m = 0u;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const uint32_t g = uint32_t(p) * kMoeThreads + tid;
        if (uint32_t(p) * kMoeThreads < padded) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[p][i] = 0.0f;
            if (g < groups) load(g, v[p]);
            rotate8(v[p], signs, had, kappa, g, g < groups, s_wide);
            m = max(m, abs_bits(v[p]));
        }
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = max(m, uint32_t(__shfl_xor(m, off, 64)));
    if ((tid & 63u) == 0u) s_max[tid >> 6] = m;
    __syncthreads();
#pragma unroll
    for (uint32_t w = 0; w < kMoeWaves; ++w) m = max(m, s_max[w]);
    const int e = exponent_of(m);
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const uint32_t g = uint32_t(p) * kMoeThreads + tid;
        if (g < padded) {
            uint2 d[3];
            digits8(v[p], e, d);
#pragma unroll
            for (uint32_t k = 0; k < 3u; ++k)
                *reinterpret_cast<uint2*>(out + digit_offset(g, 3u) + k * 16u) = d[k];
        }
    }
    if (tid == 0u) *exponent = e;
}

// Digits of x, one block a token; three more blocks scan the matrices' escape counts.
__global__ __launch_bounds__(kMoeThreads) void moe_prepare_kernel(MoeArgs a) {
    if (blockIdx.x < a.tokens) {
        const uint32_t t = blockIdx.x;
        vector_digits([&](uint32_t g, float (&v)[8]) { load8(a.x, a.x_bf16, uint64_t(t) * a.hidden + g * 8u, v); },
                      a.hidden, a.signs_in, a.had_in, a.kappa_in, a.xd + t * moe_digit_bytes(a.hidden), a.xe + t);
        return;
    }
    __shared__ uint64_t s_sum[kMoeWaves];
    const uint32_t which = blockIdx.x - a.tokens, tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
    const MoeMatrix& m = which == 0u ? a.gate : which == 1u ? a.up : a.down;
    const int64_t c = tid < a.experts ? m.esc_count[tid] : 0;
    uint64_t run = c > 0 ? uint64_t(c) : 0ull;
    const uint64_t own = run;
    for (uint32_t off = 1u; off < 64u; off *= 2u) {
        const uint64_t o = __shfl_up(run, off, 64);
        if (lane >= off) run += o;
    }
    if (lane == 63u) s_sum[wave] = run;
    __syncthreads();
    for (uint32_t w = 0; w < wave; ++w) run += s_sum[w];
    uint64_t* out = a.offsets + uint64_t(which) * (a.experts + 1u);
    if (tid < a.experts) out[tid] = min(run - own, m.esc_capacity);
    if (tid == a.experts - 1u) out[a.experts] = min(run, m.esc_capacity);
}

__global__ __launch_bounds__(kMoeThreads) void moe_digits_kernel(MoeArgs a) {
    const uint32_t r = blockIdx.x;
    const int32_t e = a.route[r];
    if (e < 0 || uint32_t(e) >= a.experts) return;
    vector_digits([&](uint32_t g, float (&v)[8]) { load8(a.h, 0, uint64_t(r) * a.inter + g * 8u, v); }, a.inter,
                  a.signs_down, a.had_down, a.kappa_down, a.hd + r * moe_digit_bytes(a.inter), a.he + r);
}

// ------------------------------------------------------------ router

constexpr uint32_t kRouteTokens = 4;     // tokens a wave multiplies with one expert's router row

__global__ __launch_bounds__(256) void moe_logits_kernel(MoeArgs a) {
    const uint32_t lane = threadIdx.x & 63u, e = blockIdx.x * 4u + (threadIdx.x >> 6), t0 = blockIdx.y * kRouteTokens;
    if (e >= a.experts) return;
    const uint32_t nt = min(kRouteTokens, a.tokens - t0);
    double acc[kRouteTokens] = {};
    for (uint32_t g = lane; g < a.hidden / 8u; g += kWave) {
        float w[8], x[8];
        load8(a.router, a.router_bf16, uint64_t(e) * a.hidden + g * 8u, w);
        double wd[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) wd[i] = double(w[i]);
#pragma unroll
        for (uint32_t t = 0; t < kRouteTokens; ++t) {
            if (t >= nt) break;
            load8(a.x, a.x_bf16, uint64_t(t0 + t) * a.hidden + g * 8u, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[t] = fma(wd[i], double(x[i]), acc[t]);
        }
    }
#pragma unroll
    for (uint32_t t = 0; t < kRouteTokens; ++t) {
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) acc[t] += __shfl_xor(acc[t], off, 64);
        if (t < nt && lane == 0u) a.logits[uint64_t(t0 + t) * a.experts + e] = acc[t];
    }
}

// The k largest logits of a token (equal ones by index, NaN as -inf) and their weights, one wave a token.
__global__ __launch_bounds__(256) void moe_choose_kernel(MoeArgs a) {
    constexpr int kEach = int(kMoeExperts / kWave);
    const uint32_t lane = threadIdx.x & 63u, t = blockIdx.x * 4u + (threadIdx.x >> 6);
    if (t >= a.tokens) return;
    const double* row = a.logits + uint64_t(t) * a.experts;
    double v[kEach];
    uint32_t taken = 0u, flags = 0u;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const uint32_t e = uint32_t(i) * kWave + lane;
        v[i] = -INFINITY;
        if (e < a.experts) {
            v[i] = row[e];
            if (!(v[i] - v[i] == 0.0)) flags |= E8Q_STATUS_NONFINITE;
            if (v[i] != v[i]) v[i] = -INFINITY;
        } else {
            taken |= 1u << i;
        }
    }
    flush_status(flags, a.status);
    double most = -INFINITY, mine = -INFINITY;       // the largest; the logit of place `lane`
    int32_t place = -1;
    for (uint32_t j = 0; j < a.k; ++j) {
        double best = -INFINITY;
        uint32_t at = 0xFFFFFFFFu;
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (!((taken >> i) & 1u) && (at == 0xFFFFFFFFu || v[i] > best)) {
                best = v[i];
                at = uint32_t(i) * kWave + lane;
            }
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) {
            const double ob = __shfl_xor(best, off, 64);
            const uint32_t oa = uint32_t(__shfl_xor(int(at), off, 64));
            if (oa != 0xFFFFFFFFu && (at == 0xFFFFFFFFu || ob > best || (ob == best && oa < at))) {
                best = ob;
                at = oa;
            }
        }
        if ((at & 63u) == lane) taken |= 1u << (at >> 6);
        if (j == 0u) most = best;
        if (lane == j) {
            mine = best;
            place = int32_t(at);
        }
    }
    float sum = 0.0f;
    const float own = lane < a.k ? expf(float(mine - most)) : 0.0f;
    if (a.normalize) {
        sum = own;
    } else {
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if (uint32_t(i) * kWave + lane < a.experts) sum += expf(float(v[i] - most));
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
    if (lane < a.k) {
        a.route[uint64_t(t) * a.k + lane] = place;
        a.weight[uint64_t(t) * a.k + lane] = own / sum;
    }
}

// ------------------------------------------------------------ the experts' products

// 2z of an escaped slot: by halves among the sorted records of its expert; the first probe where an even spread
// would have it.
__device__ __forceinline__ bool moe_record(const MoeMatrix& m, uint32_t expert, uint32_t group, uint32_t groups,
                                           uint32_t (&rec)[4]) {
    uint64_t lo = m.offsets[expert], hi = m.offsets[expert + 1];
    bool first = true;
    while (lo < hi) {
        const uint64_t mid = first && hi - lo <= 0xFFFFFFFFull ? lo + uint64_t(group) * (hi - lo) / groups
                                                               : lo + ((hi - lo) >> 1);
        first = false;
        const uint32_t key = m.esc[mid * 5];
        if (key == group) {
#pragma unroll
            for (int i = 0; i < 4; ++i) rec[i] = m.esc[mid * 5 + 1 + i];
            return true;
        }
        if (key < group) lo = mid + 1;
        else hi = mid;
    }
    return false;
}

// Points as signed bytes from the table's words of 2z + 64 (no borrow across bytes).
__device__ __forceinline__ uint32_t signed_bytes(uint32_t p) {
    return ((p | 0x80808080u) - 0x40404040u) ^ 0x80808080u;
}

// The eight indices of groups 8 n ... 8 n + 7 of a row; past its end 0, whose point meets digits of 0.
__device__ __forceinline__ u32x4_t load_indices(const uint16_t* row, uint32_t gpr, uint32_t n) {
    const uint32_t g = n * 8u;
    if (g + 8u <= gpr) return reinterpret_cast<const Bytes16*>(row + g)->v;
    u32x4_t w;
#pragma unroll
    for (uint32_t i = 0; i < 4u; ++i) {
        const uint32_t a = g + 2u * i < gpr ? row[g + 2u * i] : 0u, b = g + 2u * i + 1u < gpr ? row[g + 2u * i + 1u] : 0u;
        w[i] = a | (b << 16);
    }
    return w;
}

// One wave: chunks [lo, hi) of 16 rows against the digits in LDS (from chunk `base` on).
template <bool TAB>
struct Sweep {
    const uint16_t* row;        // this lane's row
    uint32_t gpr, npts, expert, groups, row_group;   // groups of a matrix; of the rows before this one
    bool row_ok;
    const uint2* table;         // LDS
    const uint2* pts;           // global
    const uint4* digits;        // LDS: [entries][16]
    moe_i32x4 acc, high;
    bool any_high;
    uint32_t flags;

    __device__ __forceinline__ uint2 point(uint32_t idx) const {
        if constexpr (TAB) return table[idx];
        if (idx >= npts) return make_uint2(0u, 0u);
        const uint2 p = pts[idx];
        return make_uint2(signed_bytes(p.x), signed_bytes(p.y));
    }

    __device__ __forceinline__ void chunk(const MoeMatrix& m, u32x4_t w, uint32_t c, uint32_t base) {
        const uint32_t lane = threadIdx.x & 63u, q = lane >> 4;
        uint2 p[8], ph[8];
        bool wide = false;
        // (scalars: a bit cast of a vector's element takes its first one)
        const uint32_t wd[4] = {w[0], w[1], w[2], w[3]};
        uint32_t cw[4] = {wd[0], wd[1], wd[2], wd[3]};
        const moe_u16x2 most = __builtin_elementwise_max(
            __builtin_elementwise_max(__builtin_bit_cast(moe_u16x2, wd[0]), __builtin_bit_cast(moe_u16x2, wd[1])),
            __builtin_elementwise_max(__builtin_bit_cast(moe_u16x2, wd[2]), __builtin_bit_cast(moe_u16x2, wd[3])));
        const bool big = uint32_t(most.x > most.y ? most.x : most.y) >= npts;
        if (big) {
            const moe_u16x2 lim = {uint16_t(npts), uint16_t(npts)};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                cw[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(moe_u16x2, wd[i]), lim));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p[2 * i] = point(cw[i] & 0xFFFFu);
            p[2 * i + 1] = point(cw[i] >> 16);
        }
        const uint32_t g0 = c * 32u + q * 8u;
        if (__ballot(big)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) ph[i] = make_uint2(0u, 0u);
            if (big && row_ok) {
#pragma unroll 1
                for (uint32_t i = 0; i < 8u; ++i) {
                    const uint32_t word = i < 4u ? (i < 2u ? wd[0] : wd[1]) : (i < 6u ? wd[2] : wd[3]);
                    const uint32_t id = (i & 1u) ? word >> 16 : word & 0xFFFFu;
                    if (id < npts) continue;
                    if (id != 0xFFFFu) {
                        flags |= E8Q_STATUS_BAD_INDEX;
                        continue;
                    }
                    uint32_t rec[4];
                    if (!moe_record(m, expert, row_group + g0 + i, groups, rec)) {
                        flags |= E8Q_STATUS_ESC_MISSING;
                        continue;
                    }
                    // 2z = 256 hi + lo, lo in [-128, 127]; |2z| <= 2^14 in an encoder's records
                    uint32_t l[2] = {0u, 0u}, h[2] = {0u, 0u};
                    bool ok = true;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int z = int(int16_t(uint16_t((k & 1) ? rec[k >> 1] >> 16 : rec[k >> 1] & 0xFFFFu)));
                        const int hi = (z + 128) >> 8;
                        ok = ok && z >= -16384 && z <= 16384;
                        l[k >> 2] |= (uint32_t(z) & 0xFFu) << (8 * (k & 3));
                        h[k >> 2] |= (uint32_t(hi) & 0xFFu) << (8 * (k & 3));
                    }
                    if (!ok) {
                        flags |= E8Q_STATUS_X_RANGE;
                        continue;
                    }
                    wide |= (h[0] | h[1]) != 0u;
#pragma unroll
                    for (uint32_t k = 0; k < 8u; ++k)
                        if (k == i) {
                            p[k] = make_uint2(l[0], l[1]);
                            ph[k] = make_uint2(h[0], h[1]);
                        }
                }
            }
            if (__ballot(wide)) {
                any_high = true;
#pragma unroll
                for (uint32_t s = 0; s < 4u; ++s) {
                    const uint4 d = digits[(((c - base) * 4u + s) * 4u + q) * 16u + (lane & 15u)];
                    const moe_i32x4 av = {int(ph[2 * s].x), int(ph[2 * s].y), int(ph[2 * s + 1].x), int(ph[2 * s + 1].y)};
                    const moe_i32x4 bv = {int(d.x), int(d.y), int(d.z), int(d.w)};
                    high = __builtin_amdgcn_mfma_i32_16x16x64_i8(av, bv, high, 0, 0, 0);
                }
            }
        }
#pragma unroll
        for (uint32_t s = 0; s < 4u; ++s) {
            const uint4 d = digits[(((c - base) * 4u + s) * 4u + q) * 16u + (lane & 15u)];
            const moe_i32x4 av = {int(p[2 * s].x), int(p[2 * s].y), int(p[2 * s + 1].x), int(p[2 * s + 1].y)};
            const moe_i32x4 bv = {int(d.x), int(d.y), int(d.z), int(d.w)};
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(av, bv, acc, 0, 0, 0);
        }
    }

    __device__ __forceinline__ void run(const MoeMatrix& m, uint32_t lo, uint32_t hi, uint32_t base) {
        constexpr uint32_t kAhead = 4u;
        const uint32_t q = (threadIdx.x & 63u) >> 4;
        u32x4_t w[kAhead];
#pragma unroll
        for (uint32_t i = 0; i < kAhead; ++i)
            if (lo + i < hi) w[i] = load_indices(row, gpr, (lo + i) * 4u + q);
        for (uint32_t c0 = lo; c0 < hi; c0 += kAhead) {
#pragma unroll
            for (uint32_t i = 0; i < kAhead; ++i) {
                const uint32_t c = c0 + i;
                if (c >= hi) break;
                const u32x4_t now = w[i];
                if (c + kAhead < hi) w[i] = load_indices(row, gpr, (c + kAhead) * 4u + q);
                chunk(m, now, c, base);
            }
        }
    }
};

__device__ __forceinline__ float activation(float g, int act) {
    if (act == E8Q_ACT_SILU) return g / (1.0f + expf(-g));
    return 0.5f * g * (1.0f + tanhf(0.7978845608028654f * (g + 0.044715f * g * g * g)));
}

// The rows [row0, row0 + n) of one expert for all its tokens.  IN: gate and up, the activation, into h; otherwise
// down, into part.
template <bool IN, bool TAB>
__global__ __launch_bounds__(kMoeThreads) void moe_product_kernel(MoeArgs a) {
    constexpr uint32_t kMats = IN ? 2u : 1u;
    extern __shared__ uint4 s_moe[];
    __shared__ uint32_t s_used[kMoeExperts / 32];
    __shared__ uint16_t s_list[kMoeRoutes];
    __shared__ int s_red[kMoeWaves][2][256];
    __shared__ uint32_t s_high[kMoeWaves], s_n;
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t cols = IN ? a.hidden : a.inter, rows = IN ? a.inter : a.hidden;
    const uint32_t parts = IN ? a.parts_in : a.parts_down, per = IN ? a.rows_in : a.rows_down;
    const uint32_t nth = blockIdx.x / parts, part = blockIdx.x - nth * parts;
    const uint32_t routes = a.tokens * a.k;

    // the nth expert that some token chose, and its routes in order
    if (tid < kMoeExperts / 32) s_used[tid] = 0u;
    __syncthreads();
    for (uint32_t r = tid; r < routes; r += kMoeThreads) {
        const int32_t e = a.route[r];
        if (e >= 0 && uint32_t(e) < a.experts) atomicOr(&s_used[uint32_t(e) >> 5], 1u << (e & 31));
    }
    __syncthreads();
    uint32_t expert = 0xFFFFFFFFu, left = nth;
    for (uint32_t w = 0; w < (a.experts + 31u) / 32u; ++w) {
        uint32_t bits = s_used[w];
        const uint32_t n = uint32_t(__popc(bits));
        if (left >= n) {
            left -= n;
            continue;
        }
        for (; left; --left) bits &= bits - 1u;
        expert = w * 32u + uint32_t(__ffs(int(bits)) - 1);
        break;
    }
    if (expert == 0xFFFFFFFFu) return;             // fewer are used
    if (wave == 0u) {
        uint32_t n = 0u;
        for (uint32_t r0 = 0; r0 < routes; r0 += kWave) {
            const uint32_t r = r0 + lane;
            const bool in = r < routes && a.route[r] == int32_t(expert);
            const uint64_t who = __ballot(in);
            if (in) s_list[n + uint32_t(__popcll(who & ((1ull << lane) - 1ull)))] = uint16_t(r);
            n += uint32_t(__popcll(who));
        }
        if (lane == 0u) s_n = n;
    }

    uint2* table = reinterpret_cast<uint2*>(s_moe);
    uint4* digits = s_moe + (TAB ? (a.npts + 2u) / 2u : 0u);
    if constexpr (TAB) {
        const uint2* src = reinterpret_cast<const uint2*>(a.pts);
        for (uint32_t i = tid; i <= a.npts; i += kMoeThreads) {
            const uint2 p = i < a.npts ? src[i] : make_uint2(0x40404040u, 0x40404040u);
            table[i] = make_uint2(signed_bytes(p.x), signed_bytes(p.y));
        }
    }
    __syncthreads();
    const uint32_t n = s_n, gpr = cols / 8u, chunks = moe_chunks(cols);
    const uint32_t row0 = part * per, row_end = min(rows, row0 + per);
    const uint32_t tiles = (row_end - row0 + kMoeTile - 1u) / kMoeTile;
    // waves share a tile's columns where there are fewer tiles than waves
    const uint32_t slab_chunks = min(chunks, kMoeSlab);
    uint32_t split = max(1u, kMoeWaves / (kMats * tiles));
    split = min(split, slab_chunks);
    const uint32_t at_once = kMoeWaves / (kMats * split);         // tiles of a round
    const uint8_t* xd = IN ? a.xd : a.hd;
    const int* xe = IN ? a.xe : a.he;
    const uint64_t vec_bytes = moe_digit_bytes(cols);
    uint32_t flags = 0u;

    for (uint32_t g0 = 0; g0 < n; g0 += kMoeTokens) {
        const uint32_t nt = min(kMoeTokens, n - g0);
        for (uint32_t t0 = 0; t0 < tiles; t0 += at_once) {
            const uint32_t item = wave / split, kp = wave - item * split;
            const uint32_t tile = t0 + item / kMats, mat = item % kMats;
            const bool busy = item < at_once * kMats && tile < tiles;
            const MoeMatrix& m = IN ? (mat ? a.up : a.gate) : a.down;
            const uint32_t r = row0 + tile * kMoeTile + (lane & 15u);
            const uint32_t rr = min(r, rows - 1u);
            Sweep<TAB> sw;
            sw.row = m.idx + (uint64_t(expert) * rows + rr) * gpr;
            sw.gpr = gpr;
            sw.npts = a.npts;
            sw.expert = expert;
            sw.groups = rows * gpr;
            sw.row_group = rr * gpr;
            sw.row_ok = r < row_end;
            sw.table = table;
            sw.pts = reinterpret_cast<const uint2*>(a.pts);
            sw.digits = digits;
            sw.acc = sw.high = moe_i32x4{0, 0, 0, 0};
            sw.any_high = false;
            sw.flags = 0u;
            for (uint32_t base = 0; base < chunks; base += kMoeSlab) {
                const uint32_t here = min(kMoeSlab, chunks - base);
                if (t0 == 0u || chunks > kMoeSlab) {             // (one slab stays for all tiles)
                    __syncthreads();
                    for (uint32_t i = tid; i < here * 16u * 3u * nt; i += kMoeThreads) {
                        const uint32_t j = i / (here * 48u), k = i - j * (here * 48u), entry = k / 3u, d = k - entry * 3u;
                        const uint32_t route = s_list[g0 + j], vec = IN ? route / a.k : route;
                        const uint4* src = reinterpret_cast<const uint4*>(xd + vec * vec_bytes) + base * 48u;
                        digits[entry * 16u + 3u * j + d] = src[k];
                    }
                    __syncthreads();
                }
                if (busy) sw.run(m, base + here * kp / split, base + here * (kp + 1u) / split, base);
            }
            flags |= sw.flags;
            if (busy) {
#pragma unroll
                for (uint32_t i = 0; i < 4u; ++i) {
                    s_red[wave][0][(4u * (lane >> 4) + i) * 16u + (lane & 15u)] = sw.acc[i];
                    if (sw.any_high) s_red[wave][1][(4u * (lane >> 4) + i) * 16u + (lane & 15u)] = sw.high[i];
                }
                if (lane == 0u) s_high[wave] = sw.any_high;
            }
            __syncthreads();
            const uint32_t here = min(at_once, tiles - t0);
            for (uint32_t o = tid; o < here * 16u * nt; o += kMoeThreads) {
                const uint32_t j = o / (here * 16u), k = o - j * (here * 16u), lt = k / 16u, i = k & 15u;
                const uint32_t row = row0 + (t0 + lt) * kMoeTile + i;
                if (row >= row_end) continue;
                const uint32_t route = s_list[g0 + j], vec = IN ? route / a.k : route;
                const int e = xe[vec];
                float v[kMats];
#pragma unroll
                for (uint32_t mt = 0; mt < kMats; ++mt) {
                    int64_t sum = 0;
                    for (uint32_t p = 0; p < split; ++p) {
                        const uint32_t w = (lt * kMats + mt) * split + p;
                        const int* s = &s_red[w][0][i * 16u + 3u * j];
                        sum += (int64_t(s[0]) * 256 + s[1]) * 256 + s[2];
                        if (s_high[w]) {
                            s += 256;
                            sum += ((int64_t(s[0]) * 256 + s[1]) * 256 + s[2]) * 256;
                        }
                    }
                    const MoeMatrix& mm = IN ? (mt ? a.up : a.gate) : a.down;
                    const float scale = mm.scale[uint64_t(expert) * rows + row];
                    if (!(scale > 0.0f) || __builtin_isinf(scale)) {
                        flags |= E8Q_STATUS_BAD_SCALE;
                        v[mt] = 0.0f;
                    } else if (e == kBadExponent) {
                        flags |= E8Q_STATUS_NONFINITE;
                        v[mt] = __uint_as_float(0x7FC00000u);
                    } else {
                        v[mt] = float((0.5 * double(scale)) * __builtin_ldexp(double(sum), e - kDigitBits));
                    }
                }
                if constexpr (IN) a.h[uint64_t(route) * a.inter + row] = activation(v[0], a.act) * v[1];
                else a.part[uint64_t(route) * a.hidden + row] = v[0];
            }
            __syncthreads();
        }
    }
    flush_status(flags, a.status);
}

// The weighted sum over the places, in their order.
__global__ __launch_bounds__(256) void moe_combine_kernel(MoeArgs a) {
    const uint32_t t = blockIdx.y, r = blockIdx.x * 256u + threadIdx.x;
    if (r >= a.hidden) return;
    float sum = 0.0f;
    uint32_t flags = 0u;
    for (uint32_t j = 0; j < a.k; ++j) {
        const uint32_t route = t * a.k + j;
        const int32_t e = a.route[route];
        if (e >= int32_t(a.experts)) flags |= E8Q_STATUS_BAD_INDEX;
        if (e < 0 || uint32_t(e) >= a.experts) continue;
        sum += a.weight[route] * a.part[uint64_t(route) * a.hidden + r];
    }
    if (a.y_bf16) static_cast<uint16_t*>(a.y)[uint64_t(t) * a.hidden + r] = narrow<uint16_t>(sum);
    else static_cast<float*>(a.y)[uint64_t(t) * a.hidden + r] = sum;
    flush_status(flags, a.status);
}

// ------------------------------------------------------------ host

static size_t moe_round(uint64_t bytes) { return size_t((bytes + 255) / 256 * 256); }

struct MoeLayout {
    size_t offsets, logits, xd, xe, h, hd, he, part, total;
};

static MoeLayout moe_layout(int64_t experts, int64_t hidden, int64_t inter, int64_t tokens, int64_t k) {
    MoeLayout l;
    size_t at = 0;
    const auto take = [&](uint64_t bytes) {
        const size_t here = at;
        at += moe_round(bytes);
        return here;
    };
    const uint64_t routes = uint64_t(tokens) * uint64_t(k);
    l.offsets = take(3 * uint64_t(experts + 1) * 8);
    l.logits = take(uint64_t(tokens) * uint64_t(experts) * 8);
    l.xd = take(uint64_t(tokens) * moe_digit_bytes(uint32_t(hidden)));
    l.xe = take(uint64_t(tokens) * 4);
    l.h = take(routes * uint64_t(inter) * 4);
    l.hd = take(routes * moe_digit_bytes(uint32_t(inter)));
    l.he = take(routes * 4);
    l.part = take(routes * uint64_t(hidden) * 4);
    l.total = at;
    return l;
}

static bool moe_sizes_ok(int64_t experts, int64_t hidden, int64_t inter, int64_t tokens, int64_t k) {
    return experts > 0 && hidden > 0 && inter > 0 && tokens > 0 && k > 0 && hidden % 8 == 0 && inter % 8 == 0 && k <= experts;
}

static bool moe_sizes_fit(int64_t experts, int64_t hidden, int64_t inter, int64_t tokens, int64_t k) {
    return experts <= kMoeExperts && hidden <= kMoeCols && inter <= kMoeCols && k <= kMoeTopK && tokens <= kMoeRoutes &&
           tokens * k <= kMoeRoutes;
}

// Rows of a block: whole tiles, so that the experts met (at most) fill the CUs once.
static uint32_t moe_rows(uint32_t rows, uint64_t met) {
    const uint64_t tiles = (rows + kMoeTile - 1) / kMoeTile, cus = uint64_t(device_cu_count());
    uint64_t parts = (cus + met - 1) / met;
    if (parts > tiles) parts = tiles;
    return uint32_t((tiles + parts - 1) / parts) * kMoeTile;
}

template <bool IN>
static void moe_product(const MoeArgs& a, bool tab, unsigned blocks, hipStream_t st) {
    const uint32_t chunks = moe_chunks(IN ? a.hidden : a.inter);
    const size_t lds = (tab ? size_t(a.npts + 2) / 2 * 16 : 0) + size_t(chunks < kMoeSlab ? chunks : kMoeSlab) * 16 * 256;
    if (tab) launch(moe_product_kernel<IN, true>, dim3(blocks), dim3(kMoeThreads), lds, st, a);
    else launch(moe_product_kernel<IN, false>, dim3(blocks), dim3(kMoeThreads), lds, st, a);
}

static e8q_status_t moe_matrix(const e8q_experts_t* m, MoeMatrix& out) {
    if (!m || !m->core_idx || !m->esc_count || !m->row_scale) return E8Q_ERR_INVALID;
    if (m->esc_capacity < 0 || (m->esc_capacity > 0 && !m->esc)) return E8Q_ERR_INVALID;
    const auto off = [](const void* p, size_t unit) { return reinterpret_cast<uintptr_t>(p) % unit != 0; };
    if (off(m->core_idx, 2) || off(m->esc, 4) || off(m->esc_count, 8) || off(m->row_scale, 4)) return E8Q_ERR_INVALID;
    out.idx = m->core_idx;
    out.esc = reinterpret_cast<const uint32_t*>(m->esc);
    out.esc_count = m->esc_count;
    out.esc_capacity = uint64_t(m->esc_capacity);
    out.scale = m->row_scale;
    return E8Q_OK;
}

}  // namespace e8q

extern "C" size_t e8q_moe_workspace_size(int64_t experts, int64_t hidden, int64_t inter, int64_t tokens, int64_t top_k) {
    using namespace e8q;
    if (!moe_sizes_ok(experts, hidden, inter, tokens, top_k) || !moe_sizes_fit(experts, hidden, inter, tokens, top_k))
        return 0;
    return moe_layout(experts, hidden, inter, tokens, top_k).total;
}

extern "C" e8q_status_t e8q_moe_core_escape(const e8q_experts_t* gate, const e8q_experts_t* up, const e8q_experts_t* down,
                                            int64_t experts, int64_t hidden, int64_t inter, int32_t core_bound,
                                            const int8_t* signs_in, int32_t had_block_in, const int8_t* signs_down,
                                            int32_t had_block_down, int32_t activation, const void* x,
                                            e8q_dtype_t x_dtype, int64_t tokens, const void* router,
                                            e8q_dtype_t router_dtype, int64_t top_k, int32_t normalize,
                                            int32_t* expert_idx, float* expert_weight, void* y_out, e8q_dtype_t y_dtype,
                                            void* workspace, size_t workspace_bytes, uint32_t* status_dev, void* stream) {
    using namespace e8q;
    if (!x || !expert_idx || !expert_weight || !y_out || !workspace || !status_dev) return E8Q_ERR_INVALID;
    if (!moe_sizes_ok(experts, hidden, inter, tokens, top_k)) return E8Q_ERR_INVALID;
    if (core_bound < 0 || core_bound > 40) return E8Q_ERR_INVALID;
    if (activation != E8Q_ACT_SILU && activation != E8Q_ACT_GELU_TANH) return E8Q_ERR_INVALID;
    for (const e8q_dtype_t t : {x_dtype, router_dtype, y_dtype})
        if (t != E8Q_F32 && t != E8Q_BF16) return E8Q_ERR_INVALID;
    const auto size = [](e8q_dtype_t t) { return t == E8Q_BF16 ? size_t(2) : size_t(4); };
    const auto off = [](const void* p, size_t unit) { return reinterpret_cast<uintptr_t>(p) % unit != 0; };
    if (off(x, size(x_dtype)) || off(router, size(router_dtype)) || off(y_out, size(y_dtype)) || off(expert_idx, 4) ||
        off(expert_weight, 4) || off(workspace, 256) || off(signs_in, 8) || off(signs_down, 8))
        return E8Q_ERR_INVALID;
    MoeArgs a{};
    for (const auto& [from, to] : {std::pair{gate, &a.gate}, std::pair{up, &a.up}, std::pair{down, &a.down}}) {
        const e8q_status_t st = moe_matrix(from, *to);
        if (st != E8Q_OK) return st;
    }
    if (signs_in && check_block(signs_in, had_block_in, hidden) != E8Q_OK) return E8Q_ERR_INVALID;
    if (signs_down && check_block(signs_down, had_block_down, inter) != E8Q_OK) return E8Q_ERR_INVALID;
    if (!moe_sizes_fit(experts, hidden, inter, tokens, top_k)) return E8Q_ERR_UNSUPPORTED;
    if (double(hidden) * double(inter / 8) >= 4294967295.0) return E8Q_ERR_UNSUPPORTED;
    const MoeLayout l = moe_layout(experts, hidden, inter, tokens, top_k);
    if (workspace_bytes < l.total) return E8Q_ERR_INVALID;
    e8q_status_t err = E8Q_OK;
    const DevTable* tab = get_table(core_bound, err);
    if (!tab) return err;
    char* ws = static_cast<char*>(workspace);
    a.x = x;
    a.x_bf16 = x_dtype == E8Q_BF16;
    a.tokens = uint32_t(tokens);
    a.experts = uint32_t(experts);
    a.hidden = uint32_t(hidden);
    a.inter = uint32_t(inter);
    a.k = uint32_t(top_k);
    a.router = router;
    a.router_bf16 = router_dtype == E8Q_BF16;
    a.normalize = normalize != 0;
    a.act = activation;
    a.route = expert_idx;
    a.weight = expert_weight;
    a.logits = reinterpret_cast<double*>(ws + l.logits);
    a.signs_in = signs_in;
    a.signs_down = signs_down;
    a.had_in = signs_in ? uint32_t(had_block_in) : 0u;
    a.had_down = signs_down ? uint32_t(had_block_down) : 0u;
    a.kappa_in = kappa_for(int32_t(a.had_in));
    a.kappa_down = kappa_for(int32_t(a.had_down));
    a.offsets = reinterpret_cast<uint64_t*>(ws + l.offsets);
    a.gate.offsets = a.offsets;
    a.up.offsets = a.offsets + (experts + 1);
    a.down.offsets = a.offsets + 2 * (experts + 1);
    a.xd = reinterpret_cast<uint8_t*>(ws + l.xd);
    a.xe = reinterpret_cast<int*>(ws + l.xe);
    a.h = reinterpret_cast<float*>(ws + l.h);
    a.hd = reinterpret_cast<uint8_t*>(ws + l.hd);
    a.he = reinterpret_cast<int*>(ws + l.he);
    a.part = reinterpret_cast<float*>(ws + l.part);
    a.y = y_out;
    a.y_bf16 = y_dtype == E8Q_BF16;
    a.pts = tab->dpoints;
    a.npts = uint32_t(tab->size);
    a.status = status_dev;
    const uint64_t routes = uint64_t(tokens) * uint64_t(top_k);
    const uint64_t met = routes < uint64_t(experts) ? routes : uint64_t(experts);
    a.rows_in = moe_rows(a.inter, met);
    a.rows_down = moe_rows(a.hidden, met);
    a.parts_in = (a.inter + a.rows_in - 1) / a.rows_in;
    a.parts_down = (a.hidden + a.rows_down - 1) / a.rows_down;
    const bool lds = a.npts < kMoeTable;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    launch(moe_prepare_kernel, dim3(a.tokens + 3u), dim3(kMoeThreads), 0, s, a);
    if (router) {
        launch(moe_logits_kernel, dim3((a.experts + 3u) / 4u, (a.tokens + kRouteTokens - 1u) / kRouteTokens), dim3(256), 0,
               s, a);
        launch(moe_choose_kernel, dim3((a.tokens + 3u) / 4u), dim3(256), 0, s, a);
    }
    moe_product<true>(a, lds, unsigned(met * a.parts_in), s);
    launch(moe_digits_kernel, dim3(unsigned(routes)), dim3(kMoeThreads), 0, s, a);
    moe_product<false>(a, lds, unsigned(met * a.parts_down), s);
    launch(moe_combine_kernel, dim3((a.hidden + 255u) / 256u, a.tokens), dim3(256), 0, s, a);
    return launch_status();
}

// e8q_moe_core_escape: a mixture-of-experts layer of a few tokens, straight from
// the exported form (16-bit core indices and escape records).
//
//   p = softmax(W_r x);  e_1 ... e_k the k largest, w_j = p_{e_j} (/ their sum)
//   y = sum_j w_j D_{e_j} ( act(G_{e_j} x) * (U_{e_j} x) ),   G, U, D = R^T (s z).
//
// R is orthogonal, so a product with an expert's matrix is s_r sum_g z_g . x~_g with
// x~ = R x = kappa H (sigma x), as in e8q_gemv_core_escape: x is rotated, the
// weights never are.  x~ is held in fixed point, N = rint(x~ S) with S = 8355000 / max |x~|,
// written as three signed base-256 digits, and the row sums sum 2z N are exact int32
// sums on the int8 matrix cores:
//   A (16 x 64): 16 rows x 8 groups of points, a byte for each 2z;
//   B (64 x 16): the same groups' digits, column 3 j + d holding digit d of token j.
// So one product serves five tokens, and a sweep over an expert's indices up to two
// such products (10 tokens; three left too few registers).  The step is 2^-23 of the largest |x~|,
// so that the rounding is of the size of float32's own (5 tokens in float32: 3.2e-7 of
// the result against float64, 5.1e-7 with float32 products of restored weights);
// two digits (2^-15) would be more than a bfloat16 activation's rounding in a vector with one
// strong channel.
// A core point's bytes are 2z + 8, from a table of four bytes a point: the sums lose
// 8 sum N at the end, and the LDS banks that a look-up takes are half of eight bytes'.
// An escaped slot's 2z has up to 16 bits: its low byte goes into A, and where one has a
// high byte the tile is swept once more for those.
//
// Two tiles of 16 rows go together (gate and up of the same rows; two neighbouring
// tiles of down): they share every read of the digits from LDS.
//
// Launches: the router's products (float64: a near-tie must not depend on the
// order of a sum) beside the digits of x; the choice of experts (a few logits: inside the
// third); the plan of sweeps over the chosen experts; gate and up of them with the
// activation; down, whose blocks rotate h and make its digits (past 2048 columns a launch before
// it); the weighted sum in the order of the places (up to 16 places: inside down).
//
// What bounds it (128 experts of 2048 x 768, 8 a token, C(16) and 3.0 x row RMS, medians of
// a kernel trace): for one token three dependent launches of 5.7 + 13.5 + 14.2 us, each a
// chain of waits (the choice, the table, the indices, the sum over waves) for 10 MB in
// all, the last one on 64 blocks of 32 rows for 256 CUs; for 64 tokens gate and up 43.7 us and down 41.7, where 151 MB of
// indices are 31 us at a large copy's rate: a turn of jobs on all CUs reads at 4.6 TB/s, but the second turn
// has jobs for half of them, and every job of down makes the digits of its tokens' h again.
//
// A chunk with escaped slots goes the plain way with zero points in them, then their records'
// bytes alone: resolving slot by slot in one path took 107 us for 64 tokens where this
// takes 100, and 127 instead of 86 where most chunks have one (89 experts of 896 x 544, 2.5 x
// row RMS, 25 tokens).
#include <float.h>

#include "e8q_device.hpp"
#include "e8q_host.hpp"
#include "e8q_vec.hpp"

namespace e8q {

constexpr uint32_t kMoeThreads = 1024, kMoeWaves = 16;
constexpr uint32_t kMoeTile = 16;            // rows of a matrix instruction
constexpr uint32_t kMoeTokens = 5;           // tokens of a product: 3 of the 16 columns each
constexpr uint32_t kMoeGroups = 2;           // products of a sweep, at most
constexpr uint32_t kMoeVectors = 16;         // vectors whose digits are in LDS, at most
constexpr uint32_t kMoeSlab = 8;             // chunks of 256 columns whose digits are in LDS at a time
constexpr uint32_t kMoeSmall = 4096;         // points of a table at a fixed place in LDS
constexpr uint32_t kMoeOwn = 32 * 1024;      // LDS of the kernels' own, at most
constexpr uint32_t kMoeLds = 160 * 1024;
constexpr uint32_t kMoeInline = 256;         // logits that every block of the next launch ranks itself
constexpr uint32_t kMoeDirect = 16;          // places that down's blocks sum up themselves
constexpr int64_t kMoeExperts = 1024, kMoeTopK = 64, kMoeRoutes = 4096, kMoeCols = 32768;
constexpr float kMoeFull = 8355000.0f;       // largest |N|: below 127 (2^16 + 2^8 + 1)
constexpr float kMoeLeast = 0x1p-100f;       // a vector's largest element, at least (S stays finite)

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

// One sweep: up to 5 G tokens of an expert, their routes from list[first] on.
struct MoeItem {
    uint32_t expert, first, n, pad;
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
    struct Vector* xs;          // their steps (NaN: a vector with a NaN or infinity) and sums
    float* h;                   // [tokens k, inter]
    uint8_t* hd;
    struct Vector* hs;
    float* part;                // [tokens k, hidden]
    void* y;
    int y_bf16;
    const uint32_t* pts;
    uint32_t npts;
    int table;                       // where the point table goes (Points)
    FastDiv k_div, experts_div;
    uint32_t split_direct;           // waves of a place
    int ready_down;                  // the digits of h are in the workspace
    MoeItem* items;                  // the sweeps
    uint4* plan;                     // sweeps, parts of a sweep's rows in gate and up and in down
    uint16_t* list;                  // [tokens k] routes by expert
    uint32_t most;                   // tokens of a sweep
    uint32_t blocks;                 // of a product's launch
    int choose;                      // the product's blocks choose the experts, without items
    int direct;                      // down sums over the places
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

// S from the bits of the largest |x~|, 0 where a value is not finite.
__device__ __forceinline__ float scale_of(uint32_t bits) {
    return bits >= 0x7F800000u ? 0.0f : kMoeFull / fmaxf(__uint_as_float(bits), kMoeLeast);
}

__device__ __forceinline__ double step_of(float s) { return s == 0.0f ? __builtin_nan("") : 1.0 / double(s); }

// The three digits of a group, 8 bytes each (0 where S is 0); returns the sum of N.
__device__ __forceinline__ int digits8(const float (&v)[8], float s, uint2 (&d)[3]) {
    int sum = 0;
    uint32_t w[3][2] = {{0u, 0u}, {0u, 0u}, {0u, 0u}};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        int n = s != 0.0f ? int(__builtin_rintf(v[i] * s)) : 0;
        sum += n;
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
    return sum;
}

// What a vector's products need beside its digits: 1 / S, and the sum of N.
struct Vector {
    double step, sum;
};

__device__ __forceinline__ int add_lanes(int v) {
    v += int(lane_xor<32>(uint32_t(v)));
    v += int(lane_xor<16>(uint32_t(v)));
    v += int(lane_xor<8>(uint32_t(v)));
    v += int(lane_xor<4>(uint32_t(v)));
    v += int(lane_xor<2>(uint32_t(v)));
    v += int(lane_xor<1>(uint32_t(v)));
    return v;
}

// The sum over a wave of values below 2^28: in halves that stay below 2^31.
__device__ __forceinline__ double sum_wave(int v) { return double(add_lanes(v >> 12)) * 4096.0 + double(add_lanes(v & 4095)); }

// Digits in the order of the sweep: a lane of quarter q takes groups 32 c + 8 q + 2 s, + 1 at
// step s of chunk c, so entry ((c 4 + s) 4 + q) holds both groups' digits, 16 bytes for
// each digit.  Byte offset of a group's half of digit 0 in the entries, `columns` digits apart.
__device__ __forceinline__ uint32_t digit_offset(uint32_t g, uint32_t columns) {
    const uint32_t entry = ((g >> 5) * 4u + ((g >> 1) & 3u)) * 4u + ((g >> 3) & 3u);
    return entry * columns * 16u + (g & 1u) * 8u;
}

__device__ __forceinline__ uint32_t max_wave(uint32_t m) {
    m = max(m, lane_xor<32>(m));
    m = max(m, lane_xor<16>(m));
    m = max(m, lane_xor<8>(m));
    m = max(m, lane_xor<4>(m));
    m = max(m, lane_xor<2>(m));
    m = max(m, lane_xor<1>(m));
    return m;
}

// Rotation and digits of one vector by the block, into memory: `load` gives a group's values.
template <class Load>
__device__ __forceinline__ void vector_digits(Load&& load, uint32_t cols, const int8_t* signs, uint32_t had, float kappa,
                                              uint8_t* out, Vector* vec) {
    constexpr int kPasses = int(kMoeCols / (kMoeThreads * 8));
    __shared__ float4 s_wide4[kMoeThreads * 2];
    __shared__ uint32_t s_max[kMoeWaves];
    float* s_wide = reinterpret_cast<float*>(s_wide4);
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
    m = max_wave(m);
    if ((tid & 63u) == 0u) s_max[tid >> 6] = m;
    __syncthreads();
#pragma unroll
    for (uint32_t w = 0; w < kMoeWaves; ++w) m = max(m, s_max[w]);
    const float s = scale_of(m);
    int total = 0;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const uint32_t g = uint32_t(p) * kMoeThreads + tid;
        if (g < padded) {
            uint2 d[3];
            total += digits8(v[p], s, d);
#pragma unroll
            for (uint32_t k = 0; k < 3u; ++k)
                *reinterpret_cast<uint2*>(out + digit_offset(g, 3u) + k * 16u) = d[k];
        }
    }
    __shared__ double s_sum[kMoeWaves];
    const double part = sum_wave(total);
    if ((tid & 63u) == 0u) s_sum[tid >> 6] = part;
    __syncthreads();
    if (tid == 0u) {
        double sum = 0.0;
        for (uint32_t w = 0; w < kMoeWaves; ++w) sum += s_sum[w];
        *vec = {step_of(s), sum};
    }
}

__global__ __launch_bounds__(kMoeThreads) void moe_inner_digits_kernel(MoeArgs a) {
    const uint32_t r = blockIdx.x;
    const int32_t e = a.route[r];
    if (e < 0 || uint32_t(e) >= a.experts) return;
    vector_digits([&](uint32_t g, float (&v)[8]) { load8(a.h, 0, uint64_t(r) * a.inter + g * 8u, v); }, a.inter,
                  a.signs_down, a.had_down, a.kappa_down, a.hd + r * moe_digit_bytes(a.inter), a.hs + r);
}

// The same for `n` vectors of at most 2048 columns and rotations within a wave, into LDS: vector j into columns
// 3 (j % 5) ... of part j / 5 of `digits`, its numbers into `vec`.  A wave takes 64 groups of a vector, the block as
// many vectors at a time as it has waves for (a loop, not unrolled: code that runs once costs its fetch).  Ends with a barrier.
template <class Load>
__device__ __forceinline__ void vectors_lds(Load&& load, uint32_t n, uint32_t cols, const int8_t* signs, uint32_t had,
                                            float kappa, uint4* digits, Vector* vec, uint32_t* s_max,
                                            double* s_sum) {
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t groups = cols / 8u, padded = moe_chunks(cols) * 32u, quarters = (padded + 63u) / 64u;
    const uint32_t at_once = kMoeWaves / quarters, mine = wave / quarters, first = mine * quarters;
    const uint32_t g = (wave - first) * 64u + lane, entries = moe_chunks(cols) * 16u;
#pragma unroll 1
    for (uint32_t j0 = 0; j0 < n; j0 += at_once) {
        const uint32_t j = j0 + mine;
        const bool live = mine < at_once && j < n;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.0f;
        if (live && g < groups) load(j, g, v);
        rotate8(v, signs, had, kappa, g, live && g < groups, nullptr);
        const uint32_t m = max_wave(abs_bits(v));
        if (j0 > 0u) __syncthreads();                // the maxima before are read
        if (lane == 0u) s_max[wave] = m;
        __syncthreads();
        uint32_t most = 0u;
        for (uint32_t q = 0; q < quarters; ++q) most = max(most, s_max[min(first + q, kMoeWaves - 1u)]);
        const float s = scale_of(most);
        int total = 0;
        if (live && g < padded) {
            uint2 d[3];
            total = digits8(v, s, d);
            char* out = reinterpret_cast<char*>(digits) + (j / kMoeTokens) * entries * 256u + (j % kMoeTokens) * 48u +
                        digit_offset(g, 16u);
#pragma unroll
            for (uint32_t k = 0; k < 3u; ++k) *reinterpret_cast<uint2*>(out + k * 16u) = d[k];
        }
        const double sum = sum_wave(total);
        if (lane == 0u) s_sum[wave] = sum;
        __syncthreads();
        if (live && g == 0u) {
            double all = 0.0;
            for (uint32_t q = 0; q < quarters; ++q) all += s_sum[first + q];
            vec[j] = {step_of(s), all};
        }
    }
    __syncthreads();
}

// ------------------------------------------------------------ router

constexpr uint32_t kRouteTokens = 2;     // tokens a wave multiplies with one expert's router row

// The first launch.  Blocks [0, 3): running sums of the matrices' escape counts; [3, 3 + tokens): the digits of x; the
// others: logits, a wave for an expert and up to kRouteTokens tokens.
__global__ __launch_bounds__(kMoeThreads) void moe_prepare_kernel(MoeArgs a) {
    __shared__ uint64_t s_sum[kMoeWaves];
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
    if (blockIdx.x < 3u) {
        const MoeMatrix& m = blockIdx.x == 0u ? a.gate : blockIdx.x == 1u ? a.up : a.down;
        const int64_t c = tid < a.experts ? m.esc_count[tid] : 0;
        // (a count past the records counts as all of them: the sums of 1024 stay in range, and the offsets in order)
        const uint64_t own = c > 0 ? min(uint64_t(c), m.esc_capacity) : 0ull;
        uint64_t run = own;
        for (uint32_t off = 1u; off < 64u; off *= 2u) {
            const uint64_t o = __shfl_up(run, off, 64);
            if (lane >= off) run += o;
        }
        if (lane == 63u) s_sum[wave] = run;
        __syncthreads();
        for (uint32_t w = 0; w < wave; ++w) run += s_sum[w];
        uint64_t* out = a.offsets + uint64_t(blockIdx.x) * (a.experts + 1u);
        if (tid < a.experts) out[tid] = min(run - own, m.esc_capacity);
        if (tid == a.experts - 1u) out[a.experts] = min(run, m.esc_capacity);
        return;
    }
    if (blockIdx.x < 3u + a.tokens) {
        const uint32_t t = blockIdx.x - 3u;
        vector_digits([&](uint32_t g, float (&v)[8]) { load8(a.x, a.x_bf16, uint64_t(t) * a.hidden + g * 8u, v); },
                      a.hidden, a.signs_in, a.had_in, a.kappa_in, a.xd + t * moe_digit_bytes(a.hidden), a.xs + t);
        return;
    }
    const uint32_t blocks = (a.experts + kMoeWaves - 1u) / kMoeWaves, b = blockIdx.x - 3u - a.tokens, chunk = b / blocks;
    const uint32_t e = (b - chunk * blocks) * kMoeWaves + wave, t0 = chunk * kRouteTokens;
    if (e >= a.experts) return;
    const uint32_t nt = min(kRouteTokens, a.tokens - t0);
    double acc[kRouteTokens] = {};
    constexpr uint32_t kEach = 2u;                   // groups of a lane whose loads go together
    for (uint32_t g0 = lane; g0 < a.hidden / 8u; g0 += kEach * kWave) {
        float w[kEach][8], x[kRouteTokens][kEach][8];
#pragma unroll
        for (uint32_t i = 0; i < kEach; ++i) {
            const uint32_t g = min(g0 + i * kWave, a.hidden / 8u - 1u);
            load8(a.router, a.router_bf16, uint64_t(e) * a.hidden + g * 8u, w[i]);
#pragma unroll
            for (uint32_t t = 0; t < kRouteTokens; ++t)
                load8(a.x, a.x_bf16, uint64_t(min(t0 + t, a.tokens - 1u)) * a.hidden + g * 8u, x[t][i]);
        }
#pragma unroll
        for (uint32_t i = 0; i < kEach; ++i) {
            if (g0 + i * kWave >= a.hidden / 8u) break;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const double wd = double(w[i][k]);
#pragma unroll
                for (uint32_t t = 0; t < kRouteTokens; ++t) acc[t] = fma(wd, double(x[t][i][k]), acc[t]);
            }
        }
    }
#pragma unroll
    for (uint32_t t = 0; t < kRouteTokens; ++t) {
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) acc[t] += __shfl_xor(acc[t], off, 64);
        // (a NaN counts as -inf: no weight, and its place among equal ones)
        if (t < nt && lane == 0u)
            a.logits[uint64_t(t0 + t) * a.experts + e] = acc[t] != acc[t] ? -__builtin_inf() : acc[t];
    }
}

// A logit's place in the order of the values.
__device__ __forceinline__ uint64_t logit_key(double v) {
    const uint64_t b = uint64_t(__double_as_longlong(v + 0.0));
    return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}

// Logits of a token that are greater than that of expert e, or equal and before it: by the keys' high halves, and by
// the whole keys where another has the same.  kRankLanes neighbouring lanes share an expert.
constexpr uint32_t kRankLanes = 4;

__device__ __forceinline__ uint32_t add_rank_lanes(uint32_t v) {
    v += lane_xor<1>(v);
    return v + lane_xor<2>(v);
}

__device__ __forceinline__ uint32_t logit_rank(const uint32_t* high, const uint32_t* low, uint32_t experts, uint32_t e) {
    const uint32_t own = high[e], sub = threadIdx.x % kRankLanes;
    uint32_t rank = 0u, same = 0u;
#pragma unroll 8
    for (uint32_t j = sub; j < experts; j += kRankLanes) {
        const uint32_t h = high[j];
        rank += h > own ? 1u : 0u;
        same += h == own ? 1u : 0u;
    }
    if (add_rank_lanes(same) > 1u) {
        const uint32_t mine = low[e];
#pragma unroll 4
        for (uint32_t j = sub; j < experts; j += kRankLanes) {
            const uint32_t l = low[j];
            rank += high[j] == own && (l > mine || (l == mine && j < e)) ? 1u : 0u;
        }
    }
    return add_rank_lanes(rank);
}

// The weights of a token's places from their logits (in LDS, by place), by one wave; NaN where all logits are -inf.
__device__ __forceinline__ float place_weight(const MoeArgs& a, const double* chosen, const double* logits, uint32_t lane) {
    const double most = chosen[0];
    const float own = lane < a.k ? expf(float(chosen[lane] - most)) : 0.0f;
    float sum = own;
    if (!a.normalize) {
        sum = 0.0f;
        for (uint32_t e = lane; e < a.experts; e += kWave) sum += expf(float(logits[e] - most));
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
    return own / sum;
}

// The choice of experts, a block a token.
constexpr uint32_t kChooseThreads = 512;

__global__ __launch_bounds__(kChooseThreads) void moe_choose_kernel(MoeArgs a) {
    __shared__ uint32_t s_high[kMoeExperts], s_low[kMoeExperts];
    __shared__ double s_chosen[kMoeTopK];
    const uint32_t t = blockIdx.x, tid = threadIdx.x, lane = tid & 63u;
    const double* row = a.logits + uint64_t(t) * a.experts;
    uint32_t flags = 0u;
    for (uint32_t e = tid; e < a.experts; e += kChooseThreads) {
        const double v = row[e];
        if (!(v - v == 0.0)) flags |= E8Q_STATUS_NONFINITE;
        const uint64_t key = logit_key(v);
        s_high[e] = uint32_t(key >> 32);
        s_low[e] = uint32_t(key);
    }
    flush_status(flags, a.status);
    __syncthreads();
    for (uint32_t e = tid / kRankLanes; e < a.experts; e += kChooseThreads / kRankLanes) {
        const uint32_t rank = logit_rank(s_high, s_low, a.experts, e);
        if (rank < a.k && tid % kRankLanes == 0u) {
            a.route[uint64_t(t) * a.k + rank] = int32_t(e);
            s_chosen[rank] = row[e];
        }
    }
    __syncthreads();
    if (tid >= kWave) return;
    const float w = place_weight(a, s_chosen, row, lane);
    if (lane < a.k) a.weight[uint64_t(t) * a.k + lane] = w;
}

// Time of a job of `units` units, in quarters of a chunk's (about 1 us): six chunks beside its sweep (its tokens' digits and
// records, 5 to 6.5 us), a round of sixteen units a chunk's for each and 1.3 for the sums, half as much again for two products.  A
// round of few units is split along the chunks.  Fitted to jobs of 2048 x 768 alone; elsewhere a guess that costs time, not results.
__device__ __forceinline__ uint32_t job_cost(uint32_t units, uint32_t chunks, bool two) {
    const uint32_t full = units / kMoeWaves, left = units % kMoeWaves;
    const uint32_t sweep = 4u * (full * chunks + (chunks * left + kMoeWaves - 1u) / kMoeWaves);
    return 24u + 5u * (full + (left ? 1u : 0u)) + sweep + (two ? sweep / 2u : 0u);
}

// How long the blocks take for `items` sweeps cut into `parts`, the first `heavy` ones of two products: the longest of the
// first block, the last, and the one with the last job.
__device__ __forceinline__ uint32_t plan_span(uint32_t items, uint32_t heavy, uint32_t parts, uint32_t each, uint32_t chunks,
                                              uint32_t blocks) {
    const uint32_t units = (each + parts - 1u) / parts, jobs = items * parts, turns = (jobs + blocks - 1u) / blocks;
    const uint32_t one = job_cost(units, chunks, false), two = job_cost(units, chunks, true);
    const uint32_t pos = jobs - 1u - (turns - 1u) * blocks;
    const uint32_t ends[3] = {0u, blocks - 1u, (turns - 1u) & 1u ? blocks - 1u - pos : pos};
    uint32_t span = 0u;
#pragma unroll
    for (uint32_t i = 0; i < 3u; ++i) {
        uint32_t sum = 0u;
        for (uint32_t t = 0; t < turns; ++t) {
            const uint32_t job = t * blocks + (t & 1u ? blocks - 1u - ends[i] : ends[i]);
            if (job < jobs) sum += job < heavy * parts ? two : one;
        }
        span = max(span, sum);
    }
    return span;
}

constexpr uint32_t kTurns = 4;               // jobs of a block that the plan considers

// The sweeps: the routes by expert (their order within one has no effect on any result), and an item for every `most` of
// them; those of two products come first, so that a block whose second job is a longer one had the shortest first.
__global__ __launch_bounds__(kMoeThreads) void moe_plan_kernel(MoeArgs a) {
    __shared__ uint32_t s_count[kMoeExperts], s_first[kMoeExperts], s_wave[3][kMoeWaves];
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6, routes = a.tokens * a.k;
    constexpr uint32_t kEach = uint32_t(kMoeRoutes) / kMoeThreads;
    s_count[tid] = 0u;
    int32_t e[kEach];
#pragma unroll
    for (uint32_t i = 0; i < kEach; ++i) {
        const uint32_t route = i * kMoeThreads + tid;
        e[i] = route < routes ? a.route[route] : -1;
        if (e[i] >= int32_t(a.experts)) e[i] = -1;
    }
    __syncthreads();
    uint32_t place[kEach];
#pragma unroll
    for (uint32_t i = 0; i < kEach; ++i) place[i] = e[i] >= 0 ? atomicAdd(&s_count[e[i]], 1u) : 0u;
    __syncthreads();
    // running sums over the experts: routes, items of one product, items of two
    const uint32_t n = s_count[tid], sweeps = (n + a.most - 1u) / a.most, last = n - (sweeps ? sweeps - 1u : 0u) * a.most;
    const uint32_t light = a.most > kMoeTokens ? (last > 0u && last <= kMoeTokens ? 1u : 0u) : sweeps;
    uint32_t run[3] = {n, light, sweeps - light};
    const uint32_t own[3] = {run[0], run[1], run[2]};
#pragma unroll
    for (uint32_t off = 1; off < 64u; off *= 2u)
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const uint32_t o = uint32_t(__shfl_up(int(run[k]), off, 64));
            if (lane >= off) run[k] += o;
        }
    if (lane == 63u)
#pragma unroll
        for (int k = 0; k < 3; ++k) s_wave[k][wave] = run[k];
    __syncthreads();
    uint32_t total[3] = {0u, 0u, 0u};
#pragma unroll
    for (uint32_t w = 0; w < kMoeWaves; ++w)
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const uint32_t v = s_wave[k][w];
            run[k] += w < wave ? v : 0u;
            total[k] += v;
        }
    const uint32_t first = run[0] - own[0];
    s_first[tid] = first;
    for (uint32_t i = 0; i < sweeps; ++i) {
        const bool one = i >= sweeps - light;
        const uint32_t at = one ? total[2] + run[1] - own[1] + i - (sweeps - light) : run[2] - own[2] + i;
        a.items[at] = {tid, first + i * a.most, min(n - i * a.most, a.most), 0u};
    }
    __syncthreads();
#pragma unroll
    for (uint32_t i = 0; i < kEach; ++i)
        if (e[i] >= 0) a.list[s_first[e[i]] + place[i]] = uint16_t(i * kMoeThreads + tid);
    // the parts of the items: as many as the blocks take in 1 ... kTurns turns (one part at least); a lane each, of gate and up and
    // of down
    if (wave != kMoeWaves - 1u) return;
    const uint32_t items = total[1] + total[2], turns = lane % kTurns + 1u;
    const bool down = lane / kTurns & 1u;
    const uint32_t each = down ? (a.hidden + 31u) / 32u : (a.inter + 15u) / 16u;
    const uint32_t parts = min(each, max(1u, turns * a.blocks / max(1u, items)));
    uint32_t best = plan_span(max(1u, items), total[2], parts, each, moe_chunks(down ? a.inter : a.hidden), a.blocks);
    uint32_t own_parts = parts;
#pragma unroll
    for (uint32_t off = 1; off < kTurns; off *= 2u) {
        const uint32_t other = uint32_t(__shfl_xor(int(best), int(off), 64)), p = uint32_t(__shfl_xor(int(own_parts), int(off), 64));
        if (other < best || (other == best && p < own_parts)) {
            best = other;
            own_parts = p;
        }
    }
    const uint32_t parts_down = uint32_t(__shfl(int(own_parts), int(kTurns), 64));
    if (lane == 0u) *a.plan = make_uint4(items, own_parts, parts_down, 0u);
}

// ------------------------------------------------------------ the experts' products

// 2z of an escaped slot among the sorted records of its expert.  `next`: where the record behind the last one found
// is, which is tried first (a lane's slots are consecutive groups); then probes where an even spread between
// the keys known would have it, and halves if those do not end.
constexpr uint32_t kNoRecord = 0xFFFFFFFFu;

__device__ __forceinline__ bool moe_record(const uint32_t* esc, uint64_t begin, uint64_t end, uint32_t group,
                                           uint32_t groups, uint32_t& next, uint32_t (&rec)[4]) {
    const uint32_t* list = esc + begin * 5u;
    uint32_t lo = 0u, hi = uint32_t(min(end - begin, uint64_t(groups))), from = 0u, to = groups;
    for (uint32_t probes = 0u; lo < hi; ++probes) {
        uint32_t mid = lo + ((hi - lo) >> 1);
        if (probes == 0u && next < hi) mid = next;
        else if (probes < 8u)
            mid = lo + min(uint32_t(float(group - from) * __builtin_amdgcn_rcpf(float(to - from)) * float(hi - lo)), hi - lo - 1u);
        const uint32_t* r = list + uint64_t(mid) * 5u;
        const uint32_t key = r[0];
#pragma unroll
        for (int i = 0; i < 4; ++i) rec[i] = r[1 + i];
        if (key == group) {
            next = mid + 1u;
            return true;
        }
        if (key < group) {
            lo = mid + 1u;
            from = key + 1u;
        } else {
            hi = mid;
            to = key;
        }
    }
    return false;
}

constexpr uint32_t kMoeRecords = 64;         // records of a block's rows that it keeps in LDS
constexpr uint32_t kManyRecords = 0xFFFFFFFFu;

// The records of an expert whose groups are in [first, last) into LDS (five words each), by one wave; how many, or
// kManyRecords if they are more than `cap` (or 64 or more).  Sorted keys: 64 probes at a time find the first one.
__device__ __forceinline__ uint32_t gather_records(const MoeMatrix& m, uint32_t expert, uint32_t first, uint32_t last,
                                                   uint32_t* to, uint32_t cap) {
    const uint32_t lane = threadIdx.x & 63u;
    uint64_t lo = m.offsets[expert], hi = m.offsets[expert + 1];
    const uint64_t end = hi;
    while (hi - lo > uint64_t(kWave)) {                    // keys before lo are below first, from hi on not
        const uint64_t step = (hi - lo + kWave - 1u) / kWave, at = min(lo + uint64_t(lane) * step, hi - 1u);
        const uint32_t below = uint32_t(__popcll(__ballot(m.esc[at * 5] < first)));      // of the probes, the first ones
        if (below == 0u) {
            hi = lo;
            break;
        }
        const uint64_t from = min(lo + uint64_t(below - 1u) * step, hi - 1u) + 1u;
        hi = below < uint32_t(kWave) ? min(lo + uint64_t(below) * step, hi) : hi;
        lo = from;
    }
    // (up to 64 keys that may be below, then the ones asked for)
    const uint64_t mine = lo + lane;
    const uint32_t key = mine < end ? m.esc[mine * 5] : 0xFFFFFFFFu;
    const uint32_t skip = uint32_t(__popcll(__ballot(key < first)));
    uint64_t at = mine;
    uint32_t own = key;
    if (skip) {                                            // 64 keys from the first one on
        at = mine + skip;
        own = at < end ? m.esc[at * 5] : 0xFFFFFFFFu;
    }
    const uint32_t n = uint32_t(__popcll(__ballot(own < last)));
    if (n > cap || n == kWave) return kManyRecords;
    if (lane < n) {
        to[lane * 5u] = own;
#pragma unroll
        for (uint32_t i = 1; i < 5u; ++i) to[lane * 5u + i] = m.esc[at * 5 + i];
    }
    return n;
}

// A point's eight 2z + 8 as nibbles (|2z| <= 6 in any core): coordinates 0 ... 3 in the low ones of the bytes, 4 ... 7 in
// the high ones; from the table's two words of 2z + 64.
__device__ __forceinline__ uint32_t point_word(const uint2& p) { return (p.x - 0x38383838u) | ((p.y - 0x38383838u) << 4); }

__device__ __forceinline__ uint2 point_bytes(uint32_t w) { return make_uint2(w & 0x0F0F0F0Fu, (w >> 4) & 0x0F0F0F0Fu); }

constexpr uint32_t kZeroPoint = 0x88888888u;

// The indices of eight groups from `at` on, in a matrix of `total` groups (eight at least): the words past its end are not
// read.  A row's last ones can be the next row's: they meet digits of 0.
__device__ __forceinline__ uint4 load_indices(const uint16_t* idx, uint32_t at, uint32_t total) {
    const uint32_t from = min(at, total - 8u);
    const u32x4_t v = reinterpret_cast<const Bytes16*>(reinterpret_cast<const char*>(idx) + from * 2u)->v;
    uint4 w = make_uint4(v[0], v[1], v[2], v[3]);
    if (at > from) {
#pragma unroll 1
        for (uint32_t d = min(at - from, 8u); d > 0u; --d) {
            w.x = (w.x >> 16) | (w.y << 16);
            w.y = (w.y >> 16) | (w.z << 16);
            w.z = (w.z >> 16) | (w.w << 16);
            w.w >>= 16;
        }
    }
    return w;
}

// LDS accesses of one wave, ordered across its lanes.
__device__ __forceinline__ void moe_wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The point table, four bytes a point: 0 read from memory, 1 at a fixed place in LDS (fewer than kMoeSmall points), 2 in
// LDS.  Four bytes a lane instead of eight halve the banks a read takes; three vector instructions make them operands
// (2z + 8 in every byte; the sums lose 8 sum N at the end).
template <int TAB>
struct Points {
    const uint32_t* lds;
    const uint2* mem;
    uint32_t n;

    __device__ __forceinline__ uint32_t word(uint32_t i) const {
        if constexpr (TAB == 0) return i < n ? point_word(mem[i]) : kZeroPoint;
        return lds[i];
    }
    __device__ __forceinline__ void pair(uint32_t w, uint32_t& a, uint32_t& b) const {
        if constexpr (TAB == 0) {
            a = word(w & 0xFFFFu);
            b = word(w >> 16);
        } else {
            const char* t = reinterpret_cast<const char*>(lds);
            a = *reinterpret_cast<const uint32_t*>(t + ((w << 2) & 0x3FFFCu));
            b = *reinterpret_cast<const uint32_t*>(t + ((w >> 14) & 0x3FFFCu));
        }
    }
    // Two points a thread at a time, four loads in flight.
    __device__ __forceinline__ void fill(uint32_t* to) const {
        if constexpr (TAB == 0) return;
        constexpr uint32_t kEach = TAB == 1 ? kMoeSmall / 2u / kMoeThreads : 4u;
        const uint4* from = reinterpret_cast<const uint4*>(mem);
        for (uint32_t i0 = threadIdx.x; 2u * i0 <= n; i0 += kEach * kMoeThreads) {
            uint4 p[kEach];
#pragma unroll
            for (uint32_t k = 0; k < kEach; ++k) {
                const uint32_t i = i0 + k * kMoeThreads;
                p[k] = make_uint4(0x40404040u, 0x40404040u, 0x40404040u, 0x40404040u);
                if (2u * i + 1u < n) p[k] = from[i];
                else if (2u * i < n) {
                    const uint2 last = mem[2u * i];
                    p[k].x = last.x;
                    p[k].y = last.y;
                }
            }
#pragma unroll
            for (uint32_t k = 0; k < kEach; ++k) {
                const uint32_t i = i0 + k * kMoeThreads;
                if (2u * i <= n)
                    reinterpret_cast<uint2*>(to)[i] = make_uint2(point_word(make_uint2(p[k].x, p[k].y)),
                                                                 point_word(make_uint2(p[k].z, p[k].w)));
            }
        }
    }
};

// The same value, but nothing that is formed from it is formed ahead of a loop (no instruction): what all of a kernel's
// rare paths need, formed at its start, would be spilled.
__device__ __forceinline__ uint32_t here_only(uint32_t v) {
    v = __builtin_amdgcn_readfirstlane(v);
    asm volatile("" : "+s"(v));
    return v;
}

template <typename T>
__device__ __forceinline__ T* here_only(T* p) {
    asm volatile("" : "+s"(p));
    return p;
}

// What a wave sweeps: two rows a lane, of one expert.
struct Rows {
    const uint16_t* idx[2];     // the expert's matrices
    const uint32_t* esc[2];
    const uint64_t* offsets[2]; // of its records
    uint32_t first[2];          // this lane's rows: groups of the matrix before them
    bool ok[2];
    uint32_t gpr, groups;
    const uint32_t* kept[2];    // records in LDS, their number
    uint32_t n_kept[2];
};

__device__ __forceinline__ void set_rows(Rows& r, int t, const MoeMatrix& m, uint32_t expert, uint32_t rows, uint32_t gpr,
                                         uint32_t row, uint32_t row_end) {
    r.gpr = gpr;
    r.groups = rows * gpr;
    r.idx[t] = m.idx + uint64_t(expert) * r.groups;
    r.esc[t] = m.esc;
    r.offsets[t] = m.offsets + expert;
    r.first[t] = min(row, rows - 1u) * gpr;
    r.ok[t] = row < row_end;
}

// The operand of an escaped slot: its record's low bytes, or high ones (2z = 256 high + low, low in [-128, 127]; |2z| <= 2^14 in
// an encoder's records).
__device__ __forceinline__ uint2 record_bytes(const Rows& r, bool second, uint32_t g, bool high, uint32_t (&next)[2], bool& wide,
                                              uint32_t& flags) {
    uint32_t rec[4], at_next = second ? next[1] : next[0];
    const uint32_t group = (second ? r.first[1] : r.first[0]) + g, kept = second ? r.n_kept[1] : r.n_kept[0];
    bool found = false;
    if (kept != kManyRecords) {
        const uint32_t* list = second ? r.kept[1] : r.kept[0];
        uint32_t lo = 0u, hi = kept, mid = at_next < kept ? at_next : kept / 2u;
        while (lo < hi) {
            const uint32_t key = list[mid * 5u];
            if (key == group) {
                found = true;
                at_next = mid + 1u;
#pragma unroll
                for (uint32_t k = 0; k < 4u; ++k) rec[k] = list[mid * 5u + 1u + k];
                break;
            }
            if (key < group) lo = mid + 1u;
            else hi = mid;
            mid = (lo + hi) / 2u;
        }
    } else {
        const uint64_t* at = second ? r.offsets[1] : r.offsets[0];
        found = moe_record(second ? r.esc[1] : r.esc[0], at[0], at[1], group, r.groups, at_next, rec);
    }
    (second ? next[1] : next[0]) = at_next;
    if (!found) {
        flags |= E8Q_STATUS_ESC_MISSING;
        return make_uint2(0u, 0u);
    }
    moe_u16x2 most = {0, 0};
    uint32_t above[4];                                     // 2z + 128: its upper byte is the high one
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t word = rec[k];
        const moe_u16x2 z = __builtin_bit_cast(moe_u16x2, word);
        most = __builtin_elementwise_max(most, moe_u16x2(z + moe_u16x2{16384, 16384}));
        above[k] = __builtin_bit_cast(uint32_t, moe_u16x2(z + moe_u16x2{128, 128}));
    }
    if (most.x > 32768u || most.y > 32768u) {
        flags |= E8Q_STATUS_X_RANGE;
        return make_uint2(0u, 0u);
    }
    const uint2 h = make_uint2(__builtin_amdgcn_perm(above[1], above[0], 0x07050301u),
                               __builtin_amdgcn_perm(above[3], above[2], 0x07050301u));
    wide |= (h.x | h.y) != 0u;
    return high ? h : make_uint2(__builtin_amdgcn_perm(rec[1], rec[0], 0x06040200u),
                                 __builtin_amdgcn_perm(rec[3], rec[2], 0x06040200u));
}

__device__ __forceinline__ uint32_t most_index(const uint4& w) {
    const moe_u16x2 m = __builtin_elementwise_max(
        __builtin_elementwise_max(__builtin_bit_cast(moe_u16x2, w.x), __builtin_bit_cast(moe_u16x2, w.y)),
        __builtin_elementwise_max(__builtin_bit_cast(moe_u16x2, w.z), __builtin_bit_cast(moe_u16x2, w.w)));
    return uint32_t(m.x > m.y ? m.x : m.y);
}

template <int G, int N>
__device__ __forceinline__ void step_products(const uint4* digits, uint32_t part, const uint2 (&p)[2][2],
                                              moe_i32x4 (&acc)[2][N]) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const uint4 d = digits[uint32_t(g) * part];
        const moe_i32x4 bv = {int(d.x), int(d.y), int(d.z), int(d.w)};
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const moe_i32x4 av = {int(p[t][0].x), int(p[t][0].y), int(p[t][1].x), int(p[t][1].y)};
            acc[t][g] = __builtin_amdgcn_mfma_i32_16x16x64_i8(av, bv, acc[t][g], 0, 0, 0);
        }
    }
}

// One chunk of both tiles, no slot escaped, against G products' digits, `part` apart.
template <int TAB, int G, int N>
__device__ __forceinline__ void plain_chunk(const Points<TAB>& pts, const uint4 (&word)[2], const uint4* digits, uint32_t part,
                                            moe_i32x4 (&acc)[2][N]) {
    uint32_t p[4][2][2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        pts.pair(word[t].x, p[0][t][0], p[0][t][1]);
        pts.pair(word[t].y, p[1][t][0], p[1][t][1]);
        pts.pair(word[t].z, p[2][t][0], p[2][t][1]);
        pts.pair(word[t].w, p[3][t][0], p[3][t][1]);
    }
#pragma unroll
    for (uint32_t s = 0; s < 4u; ++s) {
        const uint2 b[2][2] = {{point_bytes(p[s][0][0]), point_bytes(p[s][0][1])},
                               {point_bytes(p[s][1][0]), point_bytes(p[s][1][1])}};
        step_products<G>(digits + s * 64u, part, b, acc);
    }
}

// The escaped slots among a lane's sixteen of a chunk: bit 4 s + k for step s, tile k / 2, slot k % 2.  A malformed index is
// flagged, and its slot is 0.
__device__ __forceinline__ uint32_t escaped(const Rows& r, uint32_t n, const uint4 (&word)[2], uint32_t g0, uint32_t& flags) {
    uint32_t mask = 0u;
#pragma unroll
    for (uint32_t i = 0; i < 16u; ++i) {
        const uint32_t s = i >> 2, t = (i >> 1) & 1u;
        const uint32_t v = s == 0u ? word[t].x : s == 1u ? word[t].y : s == 2u ? word[t].z : word[t].w;
        const uint32_t id = (i & 1u) ? v >> 16 : v & 0xFFFFu;
        if (id < n || g0 + 2u * s + (i & 1u) >= r.gpr || !r.ok[t]) continue;
        if (id == 0xFFFFu) mask |= 1u << i;
        else flags |= E8Q_STATUS_BAD_INDEX;
    }
    return mask;
}

// Index n, the zero point, in place of every index past the core.
__device__ __forceinline__ uint32_t within(uint32_t w, uint32_t n) {
    const uint32_t most = n | (n << 16);
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(moe_u16x2, w),
                                                                  __builtin_bit_cast(moe_u16x2, most)));
}

// The products of the escaped slots of a chunk, by steps that have one.
template <int N>
__device__ __forceinline__ void escape_chunk(const Rows& r, uint32_t mask, uint32_t g0, bool high, const uint4* digits,
                                             uint32_t part, uint32_t groups, moe_i32x4 (&acc)[2][N], bool& wide,
                                             uint32_t& flags) {
    uint32_t next[2] = {kNoRecord, kNoRecord};
    Rows rare = r;
    rare.groups = here_only(r.groups);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        rare.esc[t] = here_only(r.esc[t]);
        rare.offsets[t] = here_only(r.offsets[t]);
    }
#pragma unroll 1
    for (uint32_t s = 0; s < 4u; ++s) {
        const uint32_t slots = (mask >> (4u * s)) & 15u;
        if (!__ballot(slots != 0u)) continue;
        uint2 p[2][2] = {};
#pragma unroll 1
        for (uint32_t k = 0; k < 4u; ++k) {
            const bool mine = (slots >> k) & 1u;
            if (!__ballot(mine)) continue;
            uint2 out = make_uint2(0u, 0u);
            if (mine) out = record_bytes(rare, k >= 2u, g0 + 2u * s + (k & 1u), high, next, wide, flags);
#pragma unroll
            for (uint32_t i = 0; i < 4u; ++i)
                if (k == i) p[i >> 1][i & 1u] = out;
        }
        // (the products of groups that have no digits are left out)
#pragma unroll
        for (int g = 0; g < N; ++g) {
            if (uint32_t(g) >= groups) break;
            moe_i32x4 one[2][1] = {{acc[0][g]}, {acc[1][g]}};
            step_products<1>(digits + uint32_t(g) * part + s * 64u, 0u, p, one);
            acc[0][g] = one[0][0];
            acc[1][g] = one[1][0];
        }
    }
}

// One chunk of both tiles against `groups` products' digits (N at most): the core's points, and the low bytes of escaped
// slots; or only the high bytes of those.
template <int TAB, int N, bool HIGH>
__device__ __forceinline__ void sweep_chunk(const Points<TAB>& pts, const Rows& r, uint4 (&word)[2], uint32_t c,
                                            const uint4* digits, uint32_t part, uint32_t groups, moe_i32x4 (&acc)[2][N],
                                            bool& wide, uint32_t& flags) {
    uint32_t mask = 0u;
    const bool rare = HIGH || __ballot(max(most_index(word[0]), most_index(word[1])) >= pts.n) != 0ull;
    if (rare) {
        const uint32_t g0 = c * 32u + (here_only(0u) + (threadIdx.x & 63u)) / 16u * 8u, n = here_only(pts.n);
        mask = escaped(r, n, word, g0, flags);
        if constexpr (!HIGH) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
                word[t] = make_uint4(within(word[t].x, n), within(word[t].y, n), within(word[t].z, n), within(word[t].w, n));
        }
    }
    if constexpr (!HIGH) {
        if constexpr (N == 1) {
            plain_chunk<TAB, 1>(pts, word, digits, part, acc);
        } else {
            if (groups == 1u) plain_chunk<TAB, 1>(pts, word, digits, part, acc);
            else plain_chunk<TAB, N>(pts, word, digits, part, acc);
        }
    }
    if (rare && __ballot(mask != 0u))
        escape_chunk<N>(r, mask, c * 32u + (here_only(0u) + (threadIdx.x & 63u)) / 16u * 8u, HIGH, digits, part, groups, acc,
                        wide, flags);
}

// Index words of both tiles, kAhead chunks ahead.
struct Words {
    static constexpr int kAhead = 2;
    uint4 w[kAhead][2];

    __device__ __forceinline__ static void load(uint4 (&to)[2], const Rows& r, uint32_t c) {
        const uint32_t q = (threadIdx.x & 63u) >> 4;
#pragma unroll
        for (int t = 0; t < 2; ++t) to[t] = load_indices(r.idx[t], r.first[t] + c * 32u + q * 8u, r.groups);
    }
    __device__ __forceinline__ void start(const Rows& r, uint32_t lo, uint32_t hi) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (lo + i < hi) load(w[i], r, lo + i);
    }
    // The words of chunk c; loads those of chunk c + kAhead.
    __device__ __forceinline__ void next(uint4 (&now)[2], const Rows& r, uint32_t c, uint32_t hi) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            now[t] = w[0][t];
#pragma unroll
            for (int i = 1; i < kAhead; ++i) w[i - 1][t] = w[i][t];
        }
        if (c + kAhead < hi) load(w[kAhead - 1], r, c + kAhead);
    }
};

// g sigmoid(g), or g (1 + tanh z) / 2 = g sigmoid(2 z) with z = sqrt(2 / pi) (g + 0.044715 g^3).
__device__ __forceinline__ float activation(float g, int act) {
    const float arg = act == E8Q_ACT_SILU ? g : 1.5957691216057308f * fmaf(0.044715f * g * g, g, g);
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * arg));
}

constexpr uint32_t kRedRow = 17;             // (16 columns; an odd stride for the reads by row)

// A wave's accumulators into LDS (added to what other waves put there: integers, in any order); then lane l has row l % 16
// of tokens l / 16 and l / 16 + 4, as float64 (exact).
template <bool ADD>
__device__ __forceinline__ void put_tile(int* red, const moe_i32x4& acc) {
    const uint32_t lane = threadIdx.x & 63u;
#pragma unroll
    for (uint32_t i = 0; i < 4u; ++i) {
        int* to = red + (4u * (lane >> 4) + i) * kRedRow + (lane & 15u);
        if constexpr (ADD) atomicAdd(to, acc[i]);
        else *to = acc[i];
    }
}

__device__ __forceinline__ double get_tile(const int* red, uint32_t row, uint32_t token) {
    const int* s = red + row * kRedRow + 3u * token;
    return (double(s[0]) * 256.0 + double(s[1])) * 256.0 + double(s[2]);
}

// A product from its exact sum of (2z + 8) N.
__device__ __forceinline__ float product_of(double sum, float scale, const Vector& v, uint32_t& flags) {
    if (!(scale > 0.0f) || __builtin_isinf(scale)) {
        flags |= E8Q_STATUS_BAD_SCALE;
        return 0.0f;
    }
    if (v.step != v.step) flags |= E8Q_STATUS_NONFINITE;
    return float((sum - 8.0 * v.sum) * (0.5 * double(scale) * v.step));
}

// x / y of small numbers (below 2^12), y's reciprocal given.
__device__ __forceinline__ uint32_t small_div(uint32_t x, float inv) {
    return __builtin_amdgcn_readfirstlane(uint32_t((float(x) + 0.5f) * inv));
}

// How a wave takes part in a round.  IN: a unit is 16 rows of gate and up; otherwise 32 rows of down.  Whole rounds
// have a unit for every wave; in the last one, where there are fewer, `split` waves share a unit's columns.
struct Round {
    uint32_t split, unit, kp;           // unit 0xFFFFFFFF: none
    float inv;

    __device__ __forceinline__ bool busy() const { return unit != 0xFFFFFFFFu; }
    // this wave's share of n chunks
    __device__ __forceinline__ uint32_t lo(uint32_t n) const { return small_div(n * kp, inv); }
    __device__ __forceinline__ uint32_t hi(uint32_t n) const { return small_div(n * (kp + 1u), inv); }
};

__device__ __forceinline__ Round round_of(uint32_t units, uint32_t first_chunks, uint32_t round) {
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Round r;
    const uint32_t left = units - round * kMoeWaves;       // (round * kMoeWaves < units)
    r.split = left > 8u ? 1u : left > 5u ? 2u : left == 5u ? 3u : left == 4u ? 4u : left == 3u ? 5u : left == 2u ? 8u : 16u;
    r.split = min(r.split, first_chunks);
    r.inv = __builtin_amdgcn_rcpf(float(r.split));
    const uint32_t slot = small_div(wave, r.inv);
    r.kp = wave - slot * r.split;
    r.unit = slot < left ? round * kMoeWaves + slot : 0xFFFFFFFFu;
    return r;
}

// What a block multiplies: its rows of one expert with `n` tokens.
struct Job {
    uint4* digits;
    const uint16_t* list;       // their routes
    Vector* vec;                // in LDS
    int (*red)[16 * kRedRow];
    const uint32_t* kept;       // records of the block's rows: [2][kMoeRecords][5], and their numbers
    const uint32_t* n_kept;
    uint32_t expert, row0, row_end, n;
};

template <bool IN>
__device__ __forceinline__ Rows unit_rows(const MoeArgs& a, uint32_t expert, uint32_t row0, uint32_t row_end, uint32_t unit) {
    const uint32_t gpr = (IN ? a.hidden : a.inter) / 8u, rows = IN ? a.inter : a.hidden, lane = threadIdx.x & 63u;
    Rows r;
    const uint32_t row = row0 + unit * (IN ? 16u : 32u) + (lane & 15u);
    set_rows(r, 0, IN ? a.gate : a.down, expert, rows, gpr, row, row_end);
    set_rows(r, 1, IN ? a.up : a.down, expert, rows, gpr, IN ? row : row + 16u, row_end);
    return r;
}

// The digits of chunks [base, base + here) of the job's tokens from the workspace, a half of the block a vector at a time:
// first to registers, then to LDS.
template <bool IN, int G>
struct Slab {
    static constexpr uint32_t kEach = (uint32_t(G) * kMoeTokens + 1u) / 2u;
    uint4 v[kEach];
    Vector vec;

    __device__ __forceinline__ static uint32_t word() { return threadIdx.x & (kMoeThreads / 2u - 1u); }
    __device__ __forceinline__ static uint32_t half() { return __builtin_amdgcn_readfirstlane(threadIdx.x / (kMoeThreads / 2u)); }
    __device__ __forceinline__ static uint32_t index(const MoeArgs& a, const Job& job, uint32_t j) {
        const uint32_t route = job.list[min(j, job.n - 1u)];
        return IN ? fdiv(route, a.k_div) : route;
    }

    // (past the last vector or word: the last ones again, which are not stored)
    __device__ __forceinline__ void load(const MoeArgs& a, const Job& job, uint32_t base, uint32_t here) {
        static_assert(kMoeSlab * 48u <= kMoeThreads / 2u, "a thread has one word of a vector's slab");
        const uint64_t vec_bytes = moe_digit_bytes(IN ? a.hidden : a.inter);
        const uint8_t* from = (IN ? a.xd : a.hd) + (base * 48u + min(word(), here * 48u - 1u)) * 16u;
#pragma unroll
        for (uint32_t k = 0; k < kEach; ++k)
            v[k] = *reinterpret_cast<const uint4*>(from + index(a, job, half() + 2u * k) * vec_bytes);
        vec = (IN ? a.xs : a.hs)[index(a, job, threadIdx.x)];
    }
    __device__ __forceinline__ void store(const Job& job, uint32_t here, uint32_t part) const {
        const uint32_t i = word(), entry = i / 3u, d = i - entry * 3u;
#pragma unroll
        for (uint32_t k = 0; k < kEach; ++k) {
            const uint32_t j = half() + 2u * k, group = j >= kMoeTokens ? 1u : 0u;
            if (j < job.n && i < here * 48u) job.digits[group * part + entry * 16u + 3u * (j - group * kMoeTokens) + d] = v[k];
        }
        if (threadIdx.x < job.n) job.vec[threadIdx.x] = vec;
    }
    // Both, vector by vector.
    __device__ __forceinline__ static void copy(const MoeArgs& a, const Job& job, uint32_t base, uint32_t here, uint32_t part) {
        const uint64_t vec_bytes = moe_digit_bytes(IN ? a.hidden : a.inter);
        const uint32_t i = word(), entry = i / 3u, d = i - entry * 3u;
#pragma unroll 1
        for (uint32_t j = half(); j < job.n; j += 2u) {
            const uint32_t vec = index(a, job, j);
            const uint32_t group = j >= kMoeTokens ? 1u : 0u;
            if (i < here * 48u)
                job.digits[group * part + entry * 16u + 3u * (j - group * kMoeTokens) + d] =
                    *reinterpret_cast<const uint4*>((IN ? a.xd : a.hd) + vec * vec_bytes + (base * 48u + i) * 16u);
            if (i == 0u) job.vec[j] = (IN ? a.xs : a.hs)[vec];
        }
    }
};

// A unit's chunks of every slab; `words` has the first ones of the first slab, whose digits are in LDS.
template <bool IN, int TAB, int N, bool HIGH>
__device__ __forceinline__ void sweep_unit(const MoeArgs& a, const Points<TAB>& pts, const Job& job, const Round& rd,
                                           uint32_t chunks, const Rows& r, uint32_t group, uint32_t groups, Words& words,
                                           moe_i32x4 (&acc)[2][N], bool& wide, uint32_t& flags) {
    const uint32_t part = min(chunks, kMoeSlab) * 256u;
    const uint4* from = job.digits + group * part + (threadIdx.x & 63u);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int g = 0; g < N; ++g) acc[t][g] = moe_i32x4{0, 0, 0, 0};
#pragma unroll 1
    for (uint32_t base = 0; base < chunks; base += kMoeSlab) {
        const uint32_t here = min(kMoeSlab, chunks - base);
        const uint32_t lo = base + rd.lo(here), hi = base + rd.hi(here);
        if (rd.busy() && (HIGH || base > 0u)) words.start(r, lo, hi);
        if (chunks > kMoeSlab) {
            __syncthreads();
            Slab<IN, 1>::copy(a, job, base, here, part);
            __syncthreads();
        }
        if (!rd.busy()) continue;
#pragma unroll 1
        for (uint32_t c = lo; c < hi; ++c) {
            uint4 now[2];
            words.next(now, r, c, hi);
            sweep_chunk<TAB, N, HIGH>(pts, r, now, c, from + (c - base) * 256u, part, groups, acc, wide, flags);
        }
    }
}

// The rows of a block for up to 5 G of its expert's tokens.
template <bool IN, int TAB, int G>
__device__ __forceinline__ void multiply(const MoeArgs& a, const Points<TAB>& pts, const Job& whole, uint32_t units,
                                         uint32_t chunks, uint32_t& flags, uint32_t* s_max, double* s_sum) {
    Job job = whole;
    job.expert = here_only(job.expert);
    job.row0 = here_only(job.row0);
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t rows = IN ? a.inter : a.hidden, first = min(chunks, kMoeSlab), part = first * 256u;
    const uint32_t groups = job.n > kMoeTokens ? 2u : 1u;
    const uint32_t rounds = (units + kMoeWaves - 1u) / kMoeWaves;
    // the digits, with the first indices on their way behind them
    Round rd = round_of(units, first, 0u);
    Words words;
    const auto start = [&](const Round& x) {
        words.start(unit_rows<IN>(a, job.expert, job.row0, job.row_end, x.unit), x.lo(first), x.hi(first));
    };
    if (!IN && !a.ready_down) {
        if (rd.busy()) start(rd);
        vectors_lds([&](uint32_t j, uint32_t g, float (&v)[8]) {
            load8(a.h, 0, uint64_t(job.list[j]) * a.inter + g * 8u, v);
        }, job.n, a.inter, a.signs_down, a.had_down, a.kappa_down, job.digits, job.vec, s_max, s_sum);
    } else if (chunks <= kMoeSlab) {
        Slab<IN, G> slab;
        slab.load(a, job, 0u, chunks);
        if (rd.busy()) start(rd);
        slab.store(job, chunks, part);
    } else if (rd.busy()) {
        start(rd);
    }
    for (uint32_t i = threadIdx.x; i < kMoeWaves * 16u * kRedRow; i += kMoeThreads) job.red[0][i] = 0;
    __syncthreads();
#pragma unroll 1
    for (uint32_t round = 0; round < rounds; ++round) {
        Rows r = unit_rows<IN>(a, job.expert, job.row0, job.row_end, rd.busy() ? rd.unit : 0u);
#pragma unroll
        for (uint32_t t = 0; t < 2u; ++t) {
            r.kept[t] = job.kept + (IN ? t * kMoeRecords * 5u : 0u);
            r.n_kept[t] = __builtin_amdgcn_readfirstlane(job.n_kept[IN ? t : 0u]);
        }
        const uint32_t row = job.row0 + (rd.busy() ? rd.unit : 0u) * (IN ? 16u : 32u) + (threadIdx.x & 15u);
        float scale[2];
#pragma unroll
        for (uint32_t t = 0; t < 2u; ++t)
            scale[t] = (IN ? (t ? a.up : a.gate) : a.down)
                           .scale[uint64_t(job.expert) * rows + min(IN ? row : row + t * 16u, rows - 1u)];
        moe_i32x4 acc[2][G];
        bool wide = false;
        sweep_unit<IN, TAB, G, false>(a, pts, job, rd, chunks, r, 0u, groups, words, acc, wide, flags);
        const bool together = rd.split > 1u || chunks > kMoeSlab;      // the block's waves keep step
        const bool again = together ? __syncthreads_or(wide) != 0 : __ballot(wide) != 0ull;
        const Round now = rd;
        const bool more = round + 1u < rounds;
        if (more) {
            rd = round_of(units, first, round + 1u);
            if (rd.busy() && !again) start(rd);
        }
        const uint32_t lane = here_only(0u) + (threadIdx.x & 63u), q = lane >> 4;
#pragma unroll 1
        for (uint32_t g = 0; g < groups; ++g) {
            moe_i32x4 tile[2], above[2][1];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                tile[t] = acc[t][0];
#pragma unroll
                for (int i = 1; i < G; ++i)
                    if (g == uint32_t(i)) tile[t] = acc[t][i];
            }
            if (again) {
                bool none = false;
                Rows same = unit_rows<IN>(a, here_only(job.expert), job.row0, job.row_end, now.busy() ? now.unit : 0u);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    same.kept[t] = r.kept[t];
                    same.n_kept[t] = r.n_kept[t];
                }
                sweep_unit<IN, TAB, 1, true>(a, pts, job, now, chunks, same, here_only(g), 1u, words, above, none, flags);
            }
            double sum[2][2] = {{0.0, 0.0}, {0.0, 0.0}};
#pragma unroll 1
            for (int pass = 0; pass < (again ? 2 : 1); ++pass) {
                const double times = pass ? 256.0 : 1.0;
                if (now.split > 1u) {
                    // the waves of a unit add up in the places of its first two
                    int (*red)[16 * kRedRow] = job.red + (wave - now.kp);
                    if (round + g + uint32_t(pass) > 0u) {
                        __syncthreads();
                        for (uint32_t i = threadIdx.x; i < kMoeWaves * 16u * kRedRow; i += kMoeThreads) job.red[0][i] = 0;
                        __syncthreads();
                    }
                    if (now.busy()) {
                        put_tile<true>(red[0], pass ? above[0][0] : tile[0]);
                        put_tile<true>(red[1], pass ? above[1][0] : tile[1]);
                    }
                    __syncthreads();
                    if (now.busy() && now.kp == 0u) {
#pragma unroll
                        for (int t = 0; t < 2; ++t)
#pragma unroll
                            for (uint32_t i = 0; i < 2u; ++i)
                                if (q + 4u * i < kMoeTokens) sum[t][i] += times * get_tile(red[t], lane & 15u, q + 4u * i);
                    }
                } else {
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (now.busy()) put_tile<false>(job.red[wave], pass ? above[t][0] : tile[t]);
                        moe_wave_sync();
                        if (now.busy()) {
#pragma unroll
                            for (uint32_t i = 0; i < 2u; ++i)
                                if (q + 4u * i < kMoeTokens)
                                    sum[t][i] += times * get_tile(job.red[wave], lane & 15u, q + 4u * i);
                        }
                        moe_wave_sync();
                    }
                }
            }
            if (!now.busy() || now.kp != 0u) continue;
#pragma unroll
            for (uint32_t i = 0; i < 2u; ++i) {
                const uint32_t j = g * kMoeTokens + q + 4u * i;
                if (q + 4u * i >= kMoeTokens || j >= job.n) continue;
                const uint32_t route = job.list[j];
                float v[2];
#pragma unroll
                for (int t = 0; t < 2; ++t) v[t] = r.ok[t] ? product_of(sum[t][i], scale[t], job.vec[j], flags) : 0.0f;
                if constexpr (IN) {
                    if (r.ok[0]) a.h[uint64_t(route) * a.inter + row] = activation(v[0], a.act) * v[1];
                } else {
                    if (r.ok[0]) a.part[uint64_t(route) * a.hidden + row] = v[0];
                    if (r.ok[1]) a.part[uint64_t(route) * a.hidden + row + 16u] = v[1];
                }
            }
        }
        if (more && rd.busy() && again) start(rd);
    }
}

template <bool IN, int TAB, int G>
__global__ __launch_bounds__(kMoeThreads) void moe_product_kernel(MoeArgs a) {
    extern __shared__ uint4 s_moe[];
    __shared__ uint2 s_table2[TAB == 1 ? kMoeSmall / 2 : 1];
    __shared__ int s_red[kMoeWaves][16 * kRedRow];
    __shared__ uint32_t s_max[kMoeWaves];
    __shared__ Vector s_vec[kMoeVectors];
    __shared__ double s_sum[kMoeWaves];
    __shared__ uint32_t s_high[IN ? kMoeInline : 1], s_low[IN ? kMoeInline : 1];
    __shared__ double s_chosen[IN ? kMoeDirect : 1];
    __shared__ int32_t s_route[IN ? kMoeDirect : 1];
    __shared__ uint16_t s_list[kMoeVectors];
    __shared__ uint32_t s_kept[2][kMoeRecords][5], s_n_kept[2];
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t cols = IN ? a.hidden : a.inter, rows = IN ? a.inter : a.hidden, gpr = cols / 8u;
    constexpr uint32_t kUnit = IN ? 16u : 32u;
    uint32_t flags = 0u, n_items, parts = 0u;
    uint32_t* table = TAB == 1 ? reinterpret_cast<uint32_t*>(s_table2) : reinterpret_cast<uint32_t*>(s_moe);
    const Points<TAB> pts = {table, reinterpret_cast<const uint2*>(a.pts), a.npts};
    uint4* digits = s_moe + (TAB == 2 ? a.npts / 4u + 1u : 0u);
    const bool choose = IN && a.choose;

    uint64_t firsts = 0ull;                        // places (of a choosing block) that are an expert's first
    if (choose) {
        // a few logits: every block ranks them; the first one writes the places
        const uint32_t cells = a.tokens * a.experts, routes = a.tokens * a.k;
        const bool writer = blockIdx.x == 0u;
        static_assert(kMoeInline * kRankLanes <= kMoeThreads, "the block ranks every logit at once");
        if (tid < cells) {
            const double logit = a.logits[tid];
            if (!(logit - logit == 0.0) && writer) flags |= E8Q_STATUS_NONFINITE;
            const uint64_t key = logit_key(logit);
            s_high[tid] = uint32_t(key >> 32);
            s_low[tid] = uint32_t(key);
        }
        pts.fill(table);
        __syncthreads();
        const uint32_t cell = tid / kRankLanes;
        if (cell < cells) {
            const uint32_t t = fdiv(cell, a.experts_div), e = cell - t * a.experts;
            const uint32_t rank = logit_rank(s_high + t * a.experts, s_low + t * a.experts, a.experts, e);
            if (rank < a.k && tid % kRankLanes == 0u) {
                s_route[t * a.k + rank] = int32_t(e);
                if (writer) s_chosen[t * a.k + rank] = a.logits[cell];
                if (writer) a.route[t * a.k + rank] = int32_t(e);
            }
        }
        __syncthreads();
        if (writer) {
            for (uint32_t t = wave; t < a.tokens; t += kMoeWaves) {
                const float w = place_weight(a, s_chosen + t * a.k, a.logits + t * a.experts, lane);
                if (lane < a.k) a.weight[t * a.k + lane] = w;
            }
        }
        bool first = lane < routes;
        for (uint32_t j = 0; j < routes; ++j) first = first && !(j < lane && s_route[j] == s_route[lane]);
        firsts = __ballot(first);
        n_items = uint32_t(__popcll(firsts));
    } else {
        const uint4 plan = *a.plan;
        n_items = plan.x;
        parts = IN ? plan.y : plan.z;
        pts.fill(table);
    }
    n_items = __builtin_amdgcn_readfirstlane(n_items);

    // jobs: equal parts of the items' units, the first ones longest; the blocks take them to and fro
    const uint32_t each = (rows + kUnit - 1u) / kUnit;
    parts = __builtin_amdgcn_readfirstlane(choose ? max(1u, min(each, gridDim.x / max(1u, n_items))) : parts);
    const uint32_t units = (each + parts - 1u) / parts, jobs = n_items * parts;
#pragma unroll 1
    for (uint32_t turn = 0u, at = blockIdx.x; at < jobs;
         ++turn, at = turn * gridDim.x + (turn & 1u ? gridDim.x - 1u - blockIdx.x : blockIdx.x)) {
        const uint32_t nth = __builtin_amdgcn_readfirstlane(at / parts), unit0 = (at - nth * parts) * units;
        if (unit0 >= each) continue;
        const uint32_t unit1 = min(each, unit0 + units), row0 = unit0 * kUnit, row_end = min(rows, unit1 * kUnit);
        if (turn) __syncthreads();
        uint32_t expert, n;
        if (choose) {
            // the nth first place's expert and its places
            uint64_t left = firsts;
            for (uint32_t k = nth; k; --k) left &= left - 1ull;
            const int32_t own = s_route[__ffsll((unsigned long long)left) - 1];
            const uint64_t who = __ballot(lane < a.tokens * a.k && s_route[min(lane, kMoeDirect - 1u)] == own);
            expert = uint32_t(own);
            n = uint32_t(__popcll(who));
            if (wave == 0u && ((who >> lane) & 1ull)) s_list[__popcll(who & ((1ull << lane) - 1ull))] = uint16_t(lane);
        } else {
            const MoeItem item = a.items[nth];
            expert = item.expert;
            n = item.n;
            if (tid < n) s_list[tid] = a.list[item.first + tid];
        }
        expert = __builtin_amdgcn_readfirstlane(expert);
        n = __builtin_amdgcn_readfirstlane(n);
        if (wave >= 1u && wave <= (IN ? 2u : 1u)) {
            // the records of the rows
            const uint32_t kept = gather_records(IN ? (wave == 1u ? a.gate : a.up) : a.down, expert, row0 * gpr, row_end * gpr,
                                                 &s_kept[wave - 1u][0][0], kMoeRecords);
            if (lane == 0u) s_n_kept[wave - 1u] = kept;
        }
        __syncthreads();
        const Job job = {digits, s_list, s_vec, s_red, &s_kept[0][0][0], s_n_kept, expert, row0, row_end, n};
        multiply<IN, TAB, G>(a, pts, job, unit1 - unit0, moe_chunks(cols), flags, s_max, s_sum);
    }
    flush_status(flags, a.status);
}

// Down and the weighted sum for few places: a block has 32 rows of every place's expert, a wave (or several that share
// the columns) a place.
template <int TAB>
__global__ __launch_bounds__(kMoeThreads) void moe_direct_kernel(MoeArgs a) {
    extern __shared__ uint4 s_moe[];
    __shared__ uint2 s_table2[TAB == 1 ? kMoeSmall / 2 : 1];
    __shared__ int s_red[kMoeWaves][16 * kRedRow];
    __shared__ uint32_t s_max[kMoeWaves];
    __shared__ Vector s_vec[kMoeVectors];
    __shared__ double s_sum[kMoeWaves];
    __shared__ float s_y[kMoeDirect][32];
    __shared__ uint32_t s_kept[kMoeWaves][kMoeRecords / 2][5];
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = __builtin_amdgcn_readfirstlane(tid >> 6), q = lane >> 4;
    const uint32_t routes = a.tokens * a.k, chunks = moe_chunks(a.inter), split = a.split_direct;
    const float inv = __builtin_amdgcn_rcpf(float(split));
    const uint32_t place = small_div(wave, inv), kp = wave - place * split;
    const int32_t chosen = place < routes ? a.route[place] : -1;
    const bool busy = chosen >= 0 && uint32_t(chosen) < a.experts;
    const uint32_t expert = __builtin_amdgcn_readfirstlane(busy ? uint32_t(chosen) : 0u), row0 = blockIdx.x * 32u;
    uint32_t flags = place < routes && chosen >= int32_t(a.experts) ? uint32_t(E8Q_STATUS_BAD_INDEX) : 0u;

    uint32_t* table = TAB == 1 ? reinterpret_cast<uint32_t*>(s_table2) : reinterpret_cast<uint32_t*>(s_moe);
    const Points<TAB> pts = {table, reinterpret_cast<const uint2*>(a.pts), a.npts};
    uint4* digits = s_moe + (TAB == 2 ? a.npts / 4u + 1u : 0u);
    Rows r;
    float scale[2];
#pragma unroll
    for (uint32_t t = 0; t < 2u; ++t) {
        const uint32_t row = row0 + t * 16u + (lane & 15u);
        set_rows(r, int(t), a.down, expert, a.hidden, a.inter / 8u, row, a.hidden);
        scale[t] = a.down.scale[uint64_t(expert) * a.hidden + min(row, a.hidden - 1u)];
    }
    const uint32_t lo = small_div(chunks * kp, inv), hi = small_div(chunks * (kp + 1u), inv);
    Words words;
    if (busy) words.start(r, lo, hi);
    const uint32_t gpr = a.inter / 8u;
    r.n_kept[0] = r.n_kept[1] = busy ? gather_records(a.down, expert, row0 * gpr, min(row0 + 32u, a.hidden) * gpr,
                                                      &s_kept[wave][0][0], kMoeRecords / 2) : 0u;
    r.kept[0] = r.kept[1] = &s_kept[wave][0][0];
    for (uint32_t i = tid; i < kMoeWaves * 16u * kRedRow; i += kMoeThreads) s_red[0][i] = 0;
    pts.fill(table);
    // (places that are not used leave what h held: their columns are not read)
    vectors_lds([&](uint32_t j, uint32_t g, float (&v)[8]) { load8(a.h, 0, uint64_t(j) * a.inter + g * 8u, v); }, routes,
                a.inter, a.signs_down, a.had_down, a.kappa_down, digits, s_vec, s_max, s_sum);
    double sum[2] = {0.0, 0.0};
    const uint4* mine = digits + (place / kMoeTokens) * chunks * 256u + q * 16u + (lane & 15u);
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        const bool high = pass == 1;
        bool wide = false;
        moe_i32x4 acc[2][1] = {{moe_i32x4{0, 0, 0, 0}}, {moe_i32x4{0, 0, 0, 0}}};
        if (busy) {
            if (high) words.start(r, lo, hi);
#pragma unroll 1
            for (uint32_t c = lo; c < hi; ++c) {
                uint4 now[2];
                words.next(now, r, c, hi);
                if (high) sweep_chunk<TAB, 1, true>(pts, r, now, c, mine + c * 256u, 0u, 1u, acc, wide, flags);
                else sweep_chunk<TAB, 1, false>(pts, r, now, c, mine + c * 256u, 0u, 1u, acc, wide, flags);
            }
        }
        // the waves of a place add up in one tile's place, one tile after the other
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if (t || high) {
                __syncthreads();
                for (uint32_t i = tid; i < kMoeWaves * 16u * kRedRow; i += kMoeThreads) s_red[0][i] = 0;
                __syncthreads();
            }
            if (busy) put_tile<true>(s_red[place], acc[t][0]);
            __syncthreads();
            if (busy && kp == 0u && q == 0u)
                sum[t] += (high ? 256.0 : 1.0) * get_tile(s_red[place], lane, place % kMoeTokens);
        }
        if (!__syncthreads_or(wide)) break;
    }
    if (busy && kp == 0u && q == 0u) {
#pragma unroll
        for (uint32_t t = 0; t < 2u; ++t)
            s_y[place][t * 16u + lane] = r.ok[t] ? product_of(sum[t], scale[t], s_vec[place], flags) : 0.0f;
    }
    __syncthreads();
    for (uint32_t o = tid; o < a.tokens * 32u; o += kMoeThreads) {
        const uint32_t t = o >> 5, row = row0 + (o & 31u);
        if (row >= a.hidden) continue;
        float y = 0.0f;
        for (uint32_t j = t * a.k; j < (t + 1u) * a.k; ++j) {
            const int32_t e = a.route[j];
            if (e >= 0 && uint32_t(e) < a.experts) y += a.weight[j] * s_y[j][o & 31u];
        }
        if (a.y_bf16) static_cast<uint16_t*>(a.y)[uint64_t(t) * a.hidden + row] = narrow<uint16_t>(y);
        else static_cast<float*>(a.y)[uint64_t(t) * a.hidden + row] = y;
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

// Sweeps at most: one for every expert that is met, and one more for every five tokens (the least that a sweep takes).
static uint64_t moe_items(uint64_t experts, uint64_t routes) {
    return (routes < experts ? routes : experts) + routes / kMoeTokens;
}

struct MoeLayout {
    size_t offsets, logits, items, list, xd, xs, h, hd, hs, part, total;
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
    l.items = take((1 + moe_items(experts, routes)) * sizeof(MoeItem));
    l.list = take(routes * 2);
    l.xd = take(uint64_t(tokens) * moe_digit_bytes(uint32_t(hidden)));
    l.xs = take(uint64_t(tokens) * sizeof(Vector));
    l.h = take(routes * uint64_t(inter) * 4);
    l.hd = take(routes * moe_digit_bytes(uint32_t(inter)));
    l.hs = take(routes * sizeof(Vector));
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

static size_t moe_group_lds(uint32_t cols) {
    const uint32_t chunks = moe_chunks(cols);
    return size_t(chunks < kMoeSlab ? chunks : kMoeSlab) * 4096;
}

// LDS of a table in it whose place is not fixed.
static size_t moe_table_bytes(uint32_t npts) { return (size_t(npts) / 4 + 1) * 16; }

// Where the table goes (Points): LDS, if the digits of one product fit beside it.
static int moe_table(uint32_t npts, uint32_t hidden, uint32_t inter) {
    if (npts < kMoeSmall) return 1;
    const size_t group = moe_group_lds(hidden > inter ? hidden : inter);
    return kMoeOwn + moe_table_bytes(npts) + group <= kMoeLds ? 2 : 0;
}

static size_t moe_table_lds(const MoeArgs& a) { return a.table == 2 ? moe_table_bytes(a.npts) : 0; }

// The kernels' LDS without the digits.
static size_t moe_own_lds(const MoeArgs& a) { return kMoeOwn + (a.table == 1 ? kMoeSmall * 4 : 0) + moe_table_lds(a); }

// Products of a sweep at most, where LDS has room for their digits: one for up to five tokens, two for more.
static uint32_t moe_groups(const MoeArgs& a, uint32_t cols) {
    return a.tokens > kMoeTokens && moe_own_lds(a) + kMoeGroups * moe_group_lds(cols) <= kMoeLds ? kMoeGroups : 1;
}

// Whether down's blocks make the digits of h themselves.
static bool moe_own_digits(uint32_t cols, uint32_t had) { return moe_chunks(cols) <= kMoeSlab && had <= 512; }

template <bool IN, int TAB>
static void moe_product(const MoeArgs& a, hipStream_t st) {
    const uint32_t groups = a.most / kMoeTokens;
    const size_t lds = moe_table_lds(a) + groups * moe_group_lds(IN ? a.hidden : a.inter);
    const dim3 grid{a.blocks};               // a block a CU: they share all sweeps' jobs
    if (groups == 1) launch(moe_product_kernel<IN, TAB, 1>, grid, dim3(kMoeThreads), lds, st, a);
    else launch(moe_product_kernel<IN, TAB, int(kMoeGroups)>, grid, dim3(kMoeThreads), lds, st, a);
}

template <bool IN>
static void moe_product(const MoeArgs& a, hipStream_t st) {
    switch (a.table) {
        case 1: moe_product<IN, 1>(a, st); break;
        case 2: moe_product<IN, 2>(a, st); break;
        default: moe_product<IN, 0>(a, st); break;
    }
}

static size_t moe_direct_lds(const MoeArgs& a) {
    return moe_table_lds(a) + (a.tokens * a.k + kMoeTokens - 1) / kMoeTokens * moe_group_lds(a.inter);
}

static void moe_direct(const MoeArgs& a, hipStream_t st) {
    const size_t lds = moe_direct_lds(a);
    const dim3 grid((a.hidden + 31u) / 32u);
    switch (a.table) {
        case 1: launch(moe_direct_kernel<1>, grid, dim3(kMoeThreads), lds, st, a); break;
        case 2: launch(moe_direct_kernel<2>, grid, dim3(kMoeThreads), lds, st, a); break;
        default: launch(moe_direct_kernel<0>, grid, dim3(kMoeThreads), lds, st, a); break;
    }
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
    a.xs = reinterpret_cast<Vector*>(ws + l.xs);
    a.h = reinterpret_cast<float*>(ws + l.h);
    a.hd = reinterpret_cast<uint8_t*>(ws + l.hd);
    a.hs = reinterpret_cast<Vector*>(ws + l.hs);
    a.part = reinterpret_cast<float*>(ws + l.part);
    a.plan = reinterpret_cast<uint4*>(ws + l.items);
    a.blocks = uint32_t(device_cu_count());
    a.items = reinterpret_cast<MoeItem*>(ws + l.items) + 1;
    a.list = reinterpret_cast<uint16_t*>(ws + l.list);
    a.y = y_out;
    a.y_bf16 = y_dtype == E8Q_BF16;
    a.pts = tab->dpoints;
    a.npts = uint32_t(tab->size);
    a.table = moe_table(a.npts, a.hidden, a.inter);
    a.status = status_dev;
    const uint64_t routes = uint64_t(tokens) * uint64_t(top_k);
    a.split_direct = uint32_t(routes >= kMoeWaves ? 1 : kMoeWaves / routes);
    if (a.split_direct > moe_chunks(a.inter)) a.split_direct = moe_chunks(a.inter);
    a.k_div = make_fastdiv(a.k);
    a.experts_div = make_fastdiv(a.experts);
    a.ready_down = !moe_own_digits(a.inter, a.had_down);
    const uint32_t groups_in = moe_groups(a, a.hidden), groups_down = moe_groups(a, a.inter);
    a.most = (groups_in < groups_down ? groups_in : groups_down) * kMoeTokens;
    a.direct = !a.ready_down && routes <= kMoeDirect && moe_direct_lds(a) + moe_own_lds(a) - moe_table_lds(a) <= kMoeLds;
    a.choose = router && a.direct && tokens * experts <= int64_t(kMoeInline) && a.tokens <= kMoeTokens;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const uint32_t logits = (a.experts + kMoeWaves - 1u) / kMoeWaves * ((a.tokens + kRouteTokens - 1u) / kRouteTokens);
    launch(moe_prepare_kernel, dim3(3u + a.tokens + (router ? logits : 0u)), dim3(kMoeThreads), 0, s, a);
    if (router && !a.choose) launch(moe_choose_kernel, dim3(a.tokens), dim3(kChooseThreads), 0, s, a);
    if (!a.choose) launch(moe_plan_kernel, dim3(1), dim3(kMoeThreads), 0, s, a);
    moe_product<true>(a, s);
    if (a.direct) {
        moe_direct(a, s);
        return launch_status();
    }
    if (a.ready_down) launch(moe_inner_digits_kernel, dim3(unsigned(routes)), dim3(kMoeThreads), 0, s, a);
    moe_product<false>(a, s);
    launch(moe_combine_kernel, dim3((a.hidden + 255u) / 256u, a.tokens), dim3(256), 0, s, a);
    return launch_status();
}

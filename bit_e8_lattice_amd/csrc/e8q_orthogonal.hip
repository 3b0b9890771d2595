// e8q_orthogonalize and e8q_orthogonal_step: Newton-Schulz products on the
// matrix cores.
//
// With n the smaller and m the larger side, X is n x m.  One step is three
// products: A = X X^T, then M = a I + b A + c A^2, then X <- M X.
//
// Rounding.  The operands of the matrix cores are float16.  Were X float16 too,
// its rounding (2^-12 of an entry) would land on every singular direction alike
// and grow with the small singular values (up to a^steps = 485 times): a
// gradient of low rank would come out with errors of 2 to 4 percent.  So X is
// kept to 22 bits, X_hi + X_lo, and the new X is M X_hi + g X_lo with one gain g of
// M = aI + bA + cA^2 for all directions.  What (M - g I) X_lo leaves out lands on
// every direction and grows in the weak ones, so g has to be theirs: the
// polynomial one standard deviation below the mean of the squared singular values
// (never below 0), both of which the trace and the norm of A give.  That is a for a
// spectrum of low rank, and the mean gain for a flat one, whose directions are all
// alike; the last step, after which nothing grows, takes the mean gain alpha.  (With
// alpha throughout, low rank came out with 1.9e-2 at 8 x 64 and 5e-3 at 257 x 1280; with
// a throughout, flat spectra with 1.6e-3 instead of 1.2e-3 at 769 x 1280.)  The rounding
// of M acts on the strong directions' columns alone.  Problems too small to fill the
// chip (64-wide tiles) wait for memory and launches, not for the matrix cores: there
// every operand has its low part and a product is three (hi hi, hi lo, lo hi), which
// leaves the rounding of the result.
//
// Measured against float64, of |O|_F, before the last rounding, five default steps:
// flat, falling, low-rank (1/8, 1/4, 1/2) and half-weak (1e-3) spectra, and a scan of
// 37 in clusters (a part at 1, the rest at 0.3 .. 1e-5), power laws and exponentials:
//                        flat    fall    1/8     1/4     1/2     half    worst
//   256 x    8 x   64    0.8e-3  0.9e-3  1.6e-3  2.0e-3  2.7e-3  3.3e-3  4.1e-3
//    64 x   32 x 1024    3.2e-3  1.4e-3  2.2e-3  1.7e-3  1.8e-3  1.8e-3  3.2e-3
//   140 x  257 x 1280    1.0e-3  0.7e-3  1.6e-3  1.6e-3  1.6e-3  1.7e-3  2.6e-3
//    20 x  769 x 1280    1.2e-3  1.0e-3  1.4e-3  1.4e-3  1.5e-3  2.4e-3  2.4e-3
//   128 x  768 x 2048    0.9e-3  2.7e-3  3.2e-3  3.2e-3  2.4e-3  2.3e-3  6.1e-3  in pairs
//        2048 x 8192     1.1e-3  2.3e-3  2.7e-3  2.2e-3  1.6e-3  1.6e-3  3.9e-3  in pairs
// Steps amplify roundings; eight default ones: worst of the scan 1.3e-2 at 8 x 64, else
// 9e-3, half of it below 2e-3.
//
// Two steps at once.  Where m is at least 2 n, two steps may take one A = X X^T and
// one product with X instead of two each: with M, M' the two steps' polynomials
// of A, A' = M A M and M' M are n x n and symmetric (all commute):
//   T = A M,  A' = M T,  X <- M' M X,
// three symmetric products of n^3 for 3 n^2 m saved.  These products are made of
// D = M - alpha I, the rest added in float32: a diagonal rounded with the rest
// would cost half as much again in accuracy.  A' comes out of two more roundings
// than X X^T of a new X would, which the table above shows; so pairs are kept for
// sides from 640 on, where those errors have averaged out to 6.4e-3 at worst (5.5e-3 and
// more for a half-weak spectrum at 64 x 256), and for steps that amplify by no more
// than five default ones do.  Time of five steps singly and in pairs, ms:
//   m / n   4096 x ..    128 of 768 x ..   16 of 1024 x ..  24, 32 of 640 x ..
//   1       1.45, 1.59   2.11, 2.36
//   1.33    1.86, 1.80   2.43, 2.54
//   1.5     2.07, 1.99   2.93, 2.82        0.69, 0.74       0.59, 0.67 (1.6)
//   2                    3.31, 3.09        0.82, 0.82       0.54, 0.55
//   2.67                 4.03, 3.54
//   3.5     4.14, 3.22                                      1.06, 0.93 (3.2)
// Below 2 what pairs gain (7% at most) is not worth their errors.  More than two
// steps at once would lose more (A' holds the squares of the singular values).
//
// Ranges.  X is stored times 2^s, s = floor(log2(sqrt(n m))) <= 15, A and T times
// 2^14, M and D times 2^12, E times 2^9: the entries' bounds (singular values
// <= 1.5, |M| <= 7) stay below 65504 and typical entries well above float16's
// smallest normal number.
//
// Layout.  Every product is C[p][q] = sum_k P[p][k] Q[q][k] with k contiguous
// in both operands: A = (X, X), A^2 = (A, A), M A = (M, A) (all symmetric).  Only
// M X = (M, X^T) has its second operand the other way round: its fragments are
// read out of X's rows by LDS reads that turn them, so X is kept (and moved)
// once, as [n, m].  Sides are padded with zeros to whole tiles, which every step
// maps to zeros.  The symmetric products compute the tiles on and below the
// diagonal and write each twice.
//
// What bounds it.  At 4096 x 14336 the product with X (481 GFLOP) takes 443 us
// (1.09 PFLOP/s; the library's float16 product of 8192^3 runs at 1.30), X X^T
// (half a product) 300 us and a square product 91 to 96 us: its 136 tiles leave 120
// of 256 CUs idle (on the others the matrix cores are busy 72% of the time, with
// no LDS bank conflict), and 528 tiles of 128 are as many rounds.
// At 128 x 768 x 2048 a tile's sum is 24 stages long and the moving of X (both
// parts read and written, 8 bytes an entry) counts as much: 483 us for 309 GFLOP.
#include <algorithm>
#include <cmath>

#include "e8q_device.hpp"
#include "e8q_host.hpp"
#include "e8q_vec.hpp"

namespace e8q {

typedef _Float16 half_t;
typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));

constexpr int kBK = 32;                 // elements of k per stage: one matrix product's
constexpr int kScaleA = 14, kScaleD = 12, kScaleE = 9;
constexpr int kNormBlocks = 1024;       // most partial sums of |G|^2 per matrix

// ------------------------------------------------------------ input

struct OrthoIn {
    const void* g;
    int g_f32;
    const float* mom_in;       // null: U = G
    float* mom_out;
    float mu;
    int nesterov;
    uint64_t cells;            // per matrix
    uint32_t rows, cols;
    uint32_t np, mp;
    int s;                     // X is scaled by 2^s
    half_t* x;                 // [batch, np, mp]
    half_t* x_lo;
    double* norm;              // [batch, norm_blocks]
    uint32_t norm_blocks;
    uint32_t* status;
};

// The update direction before orthogonalization.
__device__ __forceinline__ float direction(const OrthoIn& a, float g, float m1) {
    return a.mom_in ? (a.nesterov ? fmaf(a.mu, m1, g) : m1) : g;
}

__device__ __forceinline__ void load_g8(const OrthoIn& a, uint64_t i, float (&v)[8]) {
    if (a.g_f32) {
        const float* p = static_cast<const float*>(a.g) + i;
        float w[4];
        unpack(*reinterpret_cast<const u32x4_t*>(p), w);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = w[j];
        unpack(*reinterpret_cast<const u32x4_t*>(p + 4), w);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 + j] = w[j];
    } else {
        unpack(*reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(a.g) + i), v);
    }
}

__device__ __forceinline__ void load_f8(const float* p, float (&v)[8]) {
    float w[4];
    unpack(*reinterpret_cast<const u32x4_t*>(p), w);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = w[j];
    unpack(*reinterpret_cast<const u32x4_t*>(p + 4), w);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[4 + j] = w[j];
}

// New momentum, and partial sums of |U|^2 (float64: any magnitude of G).  A
// stream: 95 us for the momentum of 4096 x 14336 (6.2 TB/s).
__global__ __launch_bounds__(256) void ortho_norm_kernel(OrthoIn a) {
    __shared__ double s_sum[4];
    const uint64_t base = uint64_t(blockIdx.y) * a.cells;
    double sum = 0.0;
    for (uint64_t i = (uint64_t(blockIdx.x) * 256u + threadIdx.x) * 8u; i < a.cells; i += uint64_t(gridDim.x) * 2048u) {
        float g[8], m1[8] = {};
        load_g8(a, base + i, g);
        if (a.mom_in) {
            float m0[8];
            load_f8(a.mom_in + base + i, m0);
#pragma unroll
            for (int j = 0; j < 8; ++j) m1[j] = fmaf(a.mu, m0[j], g[j]);
            float lo[4] = {m1[0], m1[1], m1[2], m1[3]}, hi[4] = {m1[4], m1[5], m1[6], m1[7]};
            *reinterpret_cast<u32x4_t*>(a.mom_out + base + i) = pack(lo);
            *reinterpret_cast<u32x4_t*>(a.mom_out + base + i + 4) = pack(hi);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const double u = double(direction(a, g[j], m1[j]));
            sum = fma(u, u, sum);
        }
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
    if ((threadIdx.x & 63u) == 0u) s_sum[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0)
        a.norm[uint64_t(blockIdx.y) * a.norm_blocks + blockIdx.x] = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
}

// X = U / |U| (of U^T for a tall U) as float16 parts, by tiles of 64 x 64 of U's
// own layout; cells outside U are zeros.  A stream: 226 us for 128 x 768 x 2048 in
// bf16 (5.3 TB/s).
template <bool TALL>
__global__ __launch_bounds__(256) void ortho_split_kernel(OrthoIn a) {
    __shared__ half_t s_hi[TALL ? 64 : 1][72];
    __shared__ half_t s_lo[TALL ? 64 : 1][72];
    __shared__ double s_scale;
    const uint32_t tid = threadIdx.x, item = blockIdx.z;
    if (tid < 64u) {
        double sum = 0.0;
        for (uint32_t i = tid; i < a.norm_blocks; i += 64u) sum += a.norm[uint64_t(item) * a.norm_blocks + i];
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
        if (tid == 0u) {
            const bool bad = !(sum <= 1.7976931348623157e308);
            s_scale = bad ? __longlong_as_double(0x7FF8000000000000ll) : sum > 0.0 ? ldexp(1.0 / sqrt(sum), a.s) : 0.0;
            if (bad && blockIdx.x == 0u && blockIdx.y == 0u) atomicOr(a.status, uint32_t(E8Q_STATUS_NONFINITE));
        }
    }
    __syncthreads();
    const double scale = s_scale;
    const uint32_t r0 = blockIdx.y * 64u, c0 = blockIdx.x * 64u;
    const uint64_t item_g = uint64_t(item) * a.cells, item_x = uint64_t(item) * a.np * a.mp;
    const uint32_t c = (tid & 7u) * 8u;
#pragma unroll
    for (uint32_t it = 0; it < 2; ++it) {
        const uint32_t r = (tid >> 3) + it * 32u;
        half8_t hi = {}, lo = {};
        if (r0 + r < a.rows && c0 + c < a.cols) {
            const uint64_t i = item_g + uint64_t(r0 + r) * a.cols + c0 + c;
            float g[8], m1[8] = {};
            load_g8(a, i, g);
            if (a.mom_in) load_f8(a.mom_out + i, m1);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float x = float(double(direction(a, g[j], m1[j])) * scale);
                hi[j] = half_t(x);
                lo[j] = half_t(x - float(hi[j]));
            }
        }
        if constexpr (TALL) {
            *reinterpret_cast<half8_t*>(&s_hi[r][c]) = hi;
            *reinterpret_cast<half8_t*>(&s_lo[r][c]) = lo;
        } else {
            const uint64_t at = item_x + uint64_t(r0 + r) * a.mp + c0 + c;
            *reinterpret_cast<half8_t*>(a.x + at) = hi;
            *reinterpret_cast<half8_t*>(a.x_lo + at) = lo;
        }
    }
    if constexpr (TALL) {
        __syncthreads();
#pragma unroll
        for (uint32_t it = 0; it < 2; ++it) {
            const uint32_t r = (tid >> 3) + it * 32u;        // row of the turned tile
            half8_t hi, lo;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                hi[j] = s_hi[c + j][r];
                lo[j] = s_lo[c + j][r];
            }
            const uint64_t at = item_x + uint64_t(c0 + r) * a.mp + r0 + c;
            *reinterpret_cast<half8_t*>(a.x + at) = hi;
            *reinterpret_cast<half8_t*>(a.x_lo + at) = lo;
        }
    }
}

// ------------------------------------------------------------ products

// The 4 x 4 halves of four neighbouring lanes (two words each), turned: lane e
// gets half e of every lane, in the order of the lanes.
__device__ __forceinline__ uint2 quad_turn(uint2 v) {
    const uint32_t lane = __lane_id(), sel = lane & 1u ? 0x03020706u : 0x05040100u;
    const uint32_t a = __builtin_amdgcn_perm(lane_xor<1>(v.x), v.x, sel);
    const uint32_t b = __builtin_amdgcn_perm(lane_xor<1>(v.y), v.y, sel);
    const uint32_t got = lane_xor<2>(lane & 2u ? a : b);
    return lane & 2u ? make_uint2(got, b) : make_uint2(a, got);
}

// What a launch computes from C = P Q^T; the symmetric ones on the lower
// triangle's tiles.
//   kGram     A  = X X^T                                (P = Q = X)
//   kPoly     M  = a I + b A + c A^2, or D = M - alpha I for a pair   (P = Q = A)
//   kApply    X <- E X_hi + gain X_lo                   (P = E, Q = X turned; E = M or a pair's)
//   kLast     the same, as the result or the latents' step
// and for two steps at once
//   kMix      T  = alpha A + A D = A M                  (P = A, Q = D)
//   kMixSum   A' = alpha T + D T = M A M                (P = D, Q = T)
//   kJoin     E  = M' M = alpha alpha' I + alpha' D + alpha D' + D' D   (P = D', Q = D)
enum { kGram, kPoly, kMix, kMixSum, kJoin, kApply, kLast };

struct OrthoMul {
    const half_t* p;           // [batch, np, k]
    const half_t* q;           // [batch, np, k]; kApply, kLast: X [batch, k = np, mp]
    const half_t* p_lo;        // low parts (SPLIT)
    const half_t* q_lo;
    uint64_t p_item, q_item;   // elements per matrix
    uint32_t k;                // padded, a multiple of kBK
    uint32_t tiles_p, tiles_q; // kGram, kPoly: tiles_p on a side, lower triangle
    uint32_t per_item;         // tiles per matrix
    uint32_t n, np, mp;
    float ca, cb, cc;
    int s;
    half_t* out;               // kGram: A; kPoly: D; kApply: X [np, mp]
    half_t* out_lo;            // its low part (kApply, SPLIT); kApply: may be in, where that is no operand
    const half_t* in;          // added to C (kPoly: A, kMix: A, kMixSum: T, kJoin: D; kApply, kLast: X's low part)
    const half_t* in_lo;       // its low part (SPLIT); kJoin: D'
    float* sums;               // [batch, per-item tiles of the triangle, 2]: tr A, |A|^2 of a tile
    uint32_t sum_tiles;
    float* alpha;              // [4, batch]: alpha of the first and of the second step of a pair, then their low gains
    uint32_t batch;
    int second;                // kPoly: the pair's second step
    int pair;                  // two steps at once
    // kLast
    uint32_t rows, cols;
    int tall;
    uint16_t* update;          // or null: the latents' step
    const uint16_t* w;
    uint16_t* w_out;
    float keep, step;          // w_out = w * keep - step * O
};

// 64 lanes x 16 bytes straight to LDS at byte `to` (wave-uniform) + 16 * lane,
// from `base` (wave-uniform) + `offset`.  Written in assembly so that the
// compiler does not wait for it at the next LDS read: the stage that it fills
// is read only after wait_loads() and a barrier.  It has no result register.  The
// LDS address goes in m0, as an operand, so that the compiler knows what is there;
// the load needs a wait state after it is written.
__device__ __forceinline__ void load_lds16(const half_t* base, uint32_t offset, uint32_t to) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(to), "v"(offset), "s"(base) : "memory");
}

__device__ __forceinline__ uint32_t lds_address(const half_t* p) {
    return uint32_t(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) half_t*)p));
}

// Lane (t, c) of 16 reads 4 halves and lane (c, e) gets element e of the 4 that
// lanes (0, c) .. (3, c) read.
__device__ __forceinline__ half4_t read_turned(const half_t* p) {
    typedef short short4_t __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) short4_t lds_short4;
    return __builtin_bit_cast(half4_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4*)p));
}

// All but this wave's last N loads to LDS have landed, and its LDS reads have
// returned.
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// Waits for no memory operation of its own: after wait_loads() only.
__device__ __forceinline__ void block_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A barrier where LDS is about to be used for something else: what this wave read
// and wrote there is done (the writes too: a diagonal tile never reads its mirror).
__device__ __forceinline__ void reuse_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    block_barrier();
}

// Tile t of the lower triangle of side x side tiles: four rows of tiles at a
// time, column by column, so that tiles that run together share their operands.
__device__ __forceinline__ void tri_tile(uint32_t t, uint32_t side, uint32_t& ti, uint32_t& tj) {
    uint32_t g = uint32_t(sqrtf(float(t) * 0.125f));                 // 8 g^2 + 2 g tiles lie before group g
    while (8u * (g + 1u) * (g + 1u) + 2u * (g + 1u) <= t) ++g;
    while (8u * g * g + 2u * g > t) --g;
    uint32_t r = t - (8u * g * g + 2u * g);
    const uint32_t rows = min(4u, side - 4u * g);
    if (r < 4u * g * rows) {
        tj = r / rows;
        ti = 4u * g + r - tj * rows;
        return;
    }
    r -= 4u * g * rows;
    uint32_t d = 0u;
    while (r >= rows - d) r -= rows - d++;
    tj = 4u * g + d;
    ti = tj + r;
}

// Workgroups are dealt to the 8 XCDs in turn; this gives each XCD a contiguous
// range of tiles, whose operands then meet in its L2.
__device__ __forceinline__ uint32_t xcd_order(uint32_t b, uint32_t total) {
    const uint32_t each = total / 8u, rest = total % 8u, x = b % 8u, i = b / 8u;
    return x * each + min(x, rest) + i;
}

// A tile of BP x BQ by WP x WQ waves, RING stages in LDS.
template <int BP, int BQ, int WP, int WQ, int RING, bool SPLIT, int MODE>
__global__ __launch_bounds__(WP* WQ * 64, WP* WQ >= 4 ? 2 : 1) void ortho_mul_kernel(OrthoMul a) {
    constexpr bool kSquare = MODE != kApply && MODE != kLast;
    constexpr int kWaves = WP * WQ, FP = BP / WP / 16, FQ = BQ / WQ / 16;
    constexpr int kLoadsP = BP / 16 / kWaves, kLoadsQ = BQ / 16 / kWaves;    // wave loads per stage
    constexpr int kParts = SPLIT ? 2 : 1;
    constexpr int kSlot = kParts * (BP + BQ) * kBK;          // P's parts, then Q's
    __shared__ half_t s_op[RING * kSlot];
    const uint32_t tid = threadIdx.x, lane = tid & 63u;
    const uint32_t wave = uint32_t(__builtin_amdgcn_readfirstlane(int(tid >> 6)));
    const uint32_t tile = xcd_order(blockIdx.x, gridDim.x);
    const uint32_t item = tile / a.per_item, t = tile - item * a.per_item;
    uint32_t ti, tj;
    if constexpr (kSquare) {
        tri_tile(t, a.tiles_p, ti, tj);
    } else {
        // four columns of tiles at a time, row by row
        const uint32_t g = t / (4u * a.tiles_p), cols = min(4u, a.tiles_q - 4u * g), r = t - g * 4u * a.tiles_p;
        ti = r / cols;
        tj = 4u * g + r - ti * cols;
    }
    // Rows of a wave's fragments.  A lane's results are rows 4 (lane >> 4) .. + 3
    // of each P fragment and row lane & 15 of each Q fragment.  Row r of P
    // fragment i stands for row 32 (i / 2) + 8 (r / 4) + 4 (i % 2) + r % 4 of the
    // wave's P rows, and row r of Q fragment j for its Q row FQ r + j: two P
    // fragments give a lane 8 neighbours along P, the FQ Q fragments FQ
    // neighbours along Q, and both orders of the result go to memory in whole
    // vectors without passing through LDS again.
    // LDS holds the rows in fragment order (row 16 i + r for row r of fragment i),
    // and the 16-byte chunk c of LDS row r at position c ^ f(r), f = 0, 3, 2, 1 for
    // r / 4 mod 4: the 16 lanes that a fragment read serves at a time (rows 0-3
    // and 12-15 of one chunk, 4-11 of its neighbour, or the other way round) then
    // meet all 64 banks.
    const uint32_t lrow = lane >> 2;                 // a wave load fills 16 rows of 64 bytes
    auto place = [](uint32_t r) { return (0u - (r >> 2)) & 3u; };
    const uint64_t op = uint64_t(item) * a.p_item + uint64_t(ti * BP) * a.k;
    const uint64_t oq = uint64_t(item) * a.q_item + (kSquare ? uint64_t(tj * BQ) * a.k : uint64_t(tj * BQ));
    // The products with X take Q's fragments out of rows of X by LDS reads that
    // turn 4 x 4 blocks (read_turned).  Fragment j's column c = (c', e) is column
    // 32 (c' / 2) + 8 j + 4 (c' % 2) + e of the wave's, so that after a turn among
    // four lanes each holds 4 neighbours; turn() spreads the 8 rows and 4 places
    // that 32 lanes read over all banks.
    auto turn = [](uint32_t r) {
        return BQ >= 128 ? (r & 3u) | (r & 8u) : ((r >> 1) & 1u) | ((r >> 2) & 2u);
    };
    const uint32_t chunk = ((lane & 3u) ^ place(lrow)) * 8u;
    uint32_t off_p[kLoadsP], off_q[kLoadsQ];
#pragma unroll
    for (int i = 0; i < kLoadsP; ++i) {
        const uint32_t r = (wave * kLoadsP + i) * 16u + lrow;
        off_p[i] = (((r & ~31u) | ((r << 1) & 24u) | ((r >> 2) & 4u) | (r & 3u)) * a.k + chunk) * 2u;
    }
#pragma unroll
    for (int i = 0; i < kLoadsQ; ++i) {
        if constexpr (kSquare) {
            const uint32_t r = (wave * kLoadsQ + i) * 16u + lrow;
            off_q[i] = ((r / (FQ * 16) * (FQ * 16) + (r & 15u) * FQ + (r >> 4) % FQ) * a.k + chunk) * 2u;
        } else {
            // rows of X are Q's columns: whole rows of BQ elements, chunk c at c ^ turn(row)
            const uint32_t r = (wave * kLoadsQ + i) * (512 / BQ) + lane / (BQ / 8);
            off_q[i] = (r * a.mp + ((lane % (BQ / 8)) ^ turn(r)) * 8u) * 2u;
        }
    }
    const uint32_t lds = lds_address(s_op);
    const uint32_t to_p = lds + wave * (kLoadsP * 16 * kBK * 2);
    const uint32_t to_q = lds + kParts * (BP * kBK * 2) + wave * (kLoadsQ * 16 * kBK * 2);
    // load `l` of this wave's loads of the stage at k
    constexpr int kStageLoads = (kLoadsP + kLoadsQ) * kParts;
    auto load = [&](uint32_t slot, uint32_t k, int l) {
        const int h = l % kParts, i = l / kParts;
        if (i < kLoadsP)
            load_lds16((h ? a.p_lo : a.p) + op + k, off_p[i],
                       to_p + slot * (kSlot * 2) + h * (BP * kBK * 2) + i * (16 * kBK * 2));
        else
            load_lds16((h ? a.q_lo : a.q) + oq + (kSquare ? uint64_t(k) : uint64_t(k) * a.mp), off_q[i - kLoadsP],
                       to_q + slot * (kSlot * 2) + h * (BQ * kBK * 2) + (i - kLoadsP) * (16 * kBK * 2));
    };
    const uint32_t wp = wave / WQ, wq = wave - wp * WQ;
    const uint32_t frow = lane & 15u, fk = lane >> 4;
    struct Frags {
        half8_t p[kParts][FP], q[kParts][FQ];
    };
    // fragment `r` of the (FP + FQ) kParts fragments of a stage
    constexpr int kReads = (FP + FQ) * kParts;
    const uint32_t at_p = (wp * FP * 16 + frow) * kBK + (fk ^ place(frow)) * 8;
    const uint32_t at_q = (wq * FQ * 16 + frow) * kBK + (fk ^ place(frow)) * 8;
    // (products with X) this lane's part of the rows for fragment j
    uint32_t turn_q[FQ];
    if constexpr (!kSquare) {
#pragma unroll
        for (int j = 0; j < FQ; ++j) {
            const uint32_t r = fk * 8u + (frow >> 2), c = frow & 3u;
            turn_q[j] = r * BQ + ((wq * (FQ * 2) + (c >> 1) * 4u + j) ^ turn(r)) * 8u + (c & 1u) * 4u;
        }
    }
    auto read = [&](Frags& f, uint32_t slot, int r) {
        const int h = r % kParts, n = r / kParts;
        const half_t* at = s_op + slot * kSlot;
        if (n < FQ) {
            if constexpr (kSquare) {
                f.q[h][n] = *reinterpret_cast<const half8_t*>(at + (kParts * BP + h * BQ + n * 16) * kBK + at_q);
            } else {
                const half_t* q = at + (kParts * BP + h * BQ) * kBK + turn_q[n];
                f.q[h][n] = __builtin_shufflevector(read_turned(q), read_turned(q + 4 * BQ), 0, 1, 2, 3, 4, 5, 6, 7);
            }
        } else {
            f.p[h][n - FQ] = *reinterpret_cast<const half8_t*>(at + (h * BP + (n - FQ) * 16) * kBK + at_p);
        }
    };
    f32x4_t acc[FP][FQ] = {};
    auto multiply_row = [&](const Frags& f, int i) {
#pragma unroll
        for (int j = 0; j < FQ; ++j) {
            if constexpr (SPLIT) {
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f.p[1][i], f.q[0][j], acc[i][j], 0, 0, 0);
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f.p[0][i], f.q[1][j], acc[i][j], 0, 0, 0);
            }
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f.p[0][i], f.q[0][j], acc[i][j], 0, 0, 0);
        }
    };
    // A ring of stages in LDS and two fragment sets in registers.  In step s the
    // products of stage s run while the fragments of s + 1 are read and stage
    // s + RING is loaded into the slot of stage s, which every wave has read
    // (its fragments) before the barrier that opens step s.  A stage is so
    // loaded RING - 1 steps before it is read, and one barrier is met per step.
    // Past the end the last stage is loaded again and not used: no branch
    // stands between the products.
    auto step = [&](const Frags& f, Frags& next, uint32_t s, uint32_t slot) {
        wait_loads<(RING - 2) * kStageLoads>();
        block_barrier();
        const uint32_t k = min((s + RING) * kBK, a.k - kBK), read_slot = slot + 1 == RING ? 0 : slot + 1;
#pragma unroll
        for (int i = 0; i < FP; ++i) {
            multiply_row(f, i);
#pragma unroll
            for (int l = kStageLoads * i / FP; l < kStageLoads * (i + 1) / FP; ++l) load(slot, k, l);
#pragma unroll
            for (int r = kReads * i / FP; r < kReads * (i + 1) / FP; ++r) read(next, read_slot, r);
            __builtin_amdgcn_sched_barrier(0);
        }
        return read_slot;
    };
    Frags f0, f1;
#pragma unroll
    for (int s = 0; s < RING; ++s)
#pragma unroll
        for (int l = 0; l < kStageLoads; ++l) load(s, min(uint32_t(s * kBK), a.k - kBK), l);
    wait_loads<(RING - 1) * kStageLoads>();
    block_barrier();
#pragma unroll
    for (int r = 0; r < kReads; ++r) read(f0, 0u, r);
    uint32_t slot = 0u;
    for (uint32_t s = 0; s * kBK < a.k; s += 2) {        // k is a multiple of two stages
        slot = step(f0, f1, s, slot);
        slot = step(f1, f0, s + 1, slot);
    }
    wait_loads<0>();

    // the tile's first P and Q rows of this wave
    const uint32_t pw = ti * BP + wp * FP * 16, qw = tj * BQ + wq * FQ * 16;

    const float *alpha1 = a.alpha + item, *alpha2 = alpha1 + a.batch;
    const float *gain1 = alpha2 + a.batch, *gain2 = gain1 + a.batch;
    float alpha = 0.0f;
    if constexpr (MODE == kPoly) {
        // every block of a matrix adds the tiles' sums up in the same order
        block_barrier();
        float* s_sum = reinterpret_cast<float*>(s_op);
        const float* sums = a.sums + uint64_t(item) * a.sum_tiles * 2u;
        float tr = 0.0f, sq = 0.0f;
        for (uint32_t i = tid; i < a.sum_tiles; i += kWaves * 64u) {
            tr += sums[2u * i];
            sq += sums[2u * i + 1u];
        }
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) {
            tr += __shfl_xor(tr, off, 64);
            sq += __shfl_xor(sq, off, 64);
        }
        if (lane == 0u) {
            s_sum[wave] = tr;
            s_sum[kWaves + wave] = sq;
        }
        __syncthreads();
        tr = sq = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            tr += s_sum[w];
            sq += s_sum[kWaves + w];
        }
        alpha = a.ca + (a.cb * tr + a.cc * sq) / float(a.n);
        if (t == 0u && tid == 0u) {
            // the gain a standard deviation below the mean of the squared singular values
            const float mean = tr / float(a.n), spread = sqrtf(fmaxf(sq / float(a.n) - mean * mean, 0.0f));
            const float low = fmaxf(mean - spread, 0.0f);
            a.alpha[a.second * a.batch + item] = alpha;
            a.alpha[(2 + a.second) * a.batch + item] = a.ca + low * (a.cb + a.cc * low);
        }
    }

    // result = by_c C + by_hi in + by_lo in_lo + on_diagonal I, all in the scales
    // of what is stored
    const float back = ldexpf(1.0f, -a.s);
    float by_c = 0.0f, by_hi = 0.0f, by_lo = 0.0f, on_diagonal = 0.0f;
    if constexpr (MODE == kGram) by_c = ldexpf(1.0f, kScaleA - 2 * a.s);
    if constexpr (MODE == kPoly) {
        by_c = ldexpf(a.cc, kScaleD - 2 * kScaleA);
        by_hi = by_lo = ldexpf(a.cb, kScaleD - kScaleA);
        on_diagonal = ldexpf(a.pair ? a.ca - alpha : a.ca, kScaleD);
    }
    if constexpr (MODE == kMix || MODE == kMixSum) {
        by_c = ldexpf(1.0f, -kScaleD);
        by_hi = *alpha1;
    }
    if constexpr (MODE == kJoin) {
        by_c = ldexpf(1.0f, kScaleE - 2 * kScaleD);
        by_hi = ldexpf(*alpha2, kScaleE - kScaleD);
        by_lo = ldexpf(*alpha1, kScaleE - kScaleD);
        on_diagonal = ldexpf(*alpha1 * *alpha2, kScaleE);
    }
    if constexpr (MODE == kApply || MODE == kLast) {
        by_c = ldexpf(1.0f, a.pair ? -kScaleE : -kScaleD);
        // the last step takes the mean gain: nothing grows after it
        const float last = MODE == kLast ? (a.pair ? *alpha2 : *alpha1) : (a.pair ? *gain2 : *gain1);
        by_hi = SPLIT ? 0.0f : a.pair ? *gain1 * last : last;
    }
    constexpr bool kUseLo = MODE == kJoin || (MODE == kPoly && SPLIT);
    constexpr bool kSums = MODE == kGram || MODE == kMixSum;

    // (u, j): this lane's 8 results along P, from p0 on, at row q of Q
    const uint64_t item_out = uint64_t(item) * a.np * (kSquare ? a.np : a.mp);
    float tr = 0.0f, sq = 0.0f;
    auto value = [&](int u, int j, int e) { return acc[2 * u + e / 4][j][e % 4]; };
    if constexpr (kSquare) {
        half8_t in_hi[2][FQ], in_lo[2][FQ];       // what the results are added to, one pair of fragments ahead
        auto fetch = [&](int u) {
            const uint32_t p0 = pw + u * 32u + fk * 8u;
#pragma unroll
            for (int j = 0; j < FQ; ++j) {
                const uint64_t at = item_out + uint64_t(qw + frow * FQ + j) * a.np + p0;
                in_hi[u & 1][j] = *reinterpret_cast<const half8_t*>(a.in + at);
                if constexpr (kUseLo) in_lo[u & 1][j] = *reinterpret_cast<const half8_t*>(a.in_lo + at);
            }
        };
        // The mirrored tile goes through LDS (a part of its own for each wave, rows of
        // Q, chunk c of row r at c ^ (r / FQ)) to memory in rows of FP * 32 bytes:
        // stored from the registers, 64 bytes of a row at a time, it took three times
        // as long as the tile itself.
        constexpr uint32_t kChunks = FP * 2;
        half_t* mirror = s_op + wave * (kParts * FQ * 16 * FP * 16);
        reuse_barrier();                          // operands and (kPoly) sums are no longer read
        if constexpr (MODE != kGram) fetch(0);
#pragma unroll
        for (int u = 0; u < FP / 2; ++u) {
            const uint32_t p0 = pw + u * 32u + fk * 8u;
            if constexpr (MODE != kGram) {
                if (u + 1 < FP / 2) fetch(u + 1);
            }
            half8_t h[FQ], l[FQ];
#pragma unroll
            for (int j = 0; j < FQ; ++j) {
                const uint32_t q = qw + frow * FQ + j;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float r = by_c * value(u, j, e);
                    if constexpr (MODE != kGram) r = fmaf(by_hi, float(in_hi[u & 1][j][e]), r);
                    if constexpr (kUseLo) r = fmaf(by_lo, float(in_lo[u & 1][j][e]), r);
                    if constexpr (MODE == kPoly || MODE == kJoin) r += p0 + e == q ? on_diagonal : 0.0f;
                    if constexpr (kSums) {
                        sq = fmaf(r, r, sq);
                        tr += p0 + e == q ? r : 0.0f;
                    }
                    h[j][e] = half_t(r);
                    l[j][e] = half_t(r - float(h[j][e]));
                }
                half_t* at = mirror + (frow * FQ + j) * (FP * 16) + ((u * 4u + fk) ^ (frow & (kChunks - 1u))) * 8u;
                *reinterpret_cast<half8_t*>(at) = h[j];
                if constexpr (SPLIT) *reinterpret_cast<half8_t*>(at + FQ * 16 * FP * 16) = l[j];
            }
            typedef _Float16 row_t __attribute__((ext_vector_type(FQ)));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                row_t rh, rl;
#pragma unroll
                for (int j = 0; j < FQ; ++j) {
                    rh[j] = h[j][e];
                    rl[j] = l[j][e];
                }
                const uint64_t at = item_out + uint64_t(p0 + e) * a.np + qw + frow * FQ;
                *reinterpret_cast<row_t*>(a.out + at) = rh;
                if constexpr (SPLIT) *reinterpret_cast<row_t*>(a.out_lo + at) = rl;
            }
        }
        if (ti != tj) {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int n = 0; n < FP * FQ / 2; ++n) {
                const uint32_t r = n * (64u / kChunks) + lane / kChunks, c = lane % kChunks;
                const half_t* from = mirror + r * (FP * 16) + (c ^ ((r / FQ) & (kChunks - 1u))) * 8u;
                const uint64_t at = item_out + uint64_t(qw + r) * a.np + pw + c * 8u;
                *reinterpret_cast<half8_t*>(a.out + at) = *reinterpret_cast<const half8_t*>(from);
                if constexpr (SPLIT)
                    *reinterpret_cast<half8_t*>(a.out_lo + at) =
                        *reinterpret_cast<const half8_t*>(from + FQ * 16 * FP * 16);
            }
        } else if constexpr (MODE == kMix || MODE == kMixSum) {
            // Rounded factors commute only nearly, so these two products are not
            // symmetric by themselves, as X X^T and A^2 are, and what reads them takes
            // rows for columns: left so inside the diagonal tiles they gave errors of
            // 4.5e-3 to 5.6e-3.  The entries above the diagonal are overwritten with those below.
            static_assert(BP == BQ && !SPLIT, "square tiles");
            wait_loads<0>();                      // this wave's stores too
            block_barrier();
            constexpr uint32_t kRowChunks = BP / 8;
            for (uint32_t i = tid; i < BQ * kRowChunks; i += kWaves * 64u) {
                const uint32_t q = i / kRowChunks, p = i % kRowChunks * 8u;
                if (p + 7u <= q) continue;
                const uint32_t part = p / (FP * 16) * WQ + q / (FQ * 16), r = q % (FQ * 16), c = p % (FP * 16) / 8u;
                const half8_t v = *reinterpret_cast<const half8_t*>(
                    s_op + (part * (FQ * 16) + r) * (FP * 16) + (c ^ ((r / FQ) & (kChunks - 1u))) * 8u);
                half_t* to = a.out + item_out + uint64_t(tj * BQ + q) * a.np + ti * BP + p;
                if (p > q) {
                    *reinterpret_cast<half8_t*>(to) = v;
                } else {
#pragma unroll
                    for (uint32_t e = 1; e < 8; ++e)
                        if (p + e > q) to[e] = v[e];
                }
            }
        }
    } else {
        static_assert(FQ == 4, "columns turned four by four");
        // after a turn: columns m0 .. m0 + 3; before: column mj + 8 j in slot j
        const uint32_t quad = qw + (frow >> 3) * 32u + ((frow >> 2) & 1u) * 4u;
        const uint32_t m0 = quad + (frow & 3u) * 8u, mj = quad + (frow & 3u);
        uint2 in[2][8];                           // X's low part, one pair of fragments ahead
        auto fetch = [&](int u) {
            const uint64_t at = item_out + uint64_t(pw + u * 32u + fk * 8u) * a.mp + m0;
#pragma unroll
            for (int e = 0; e < 8; ++e) in[u & 1][e] = *reinterpret_cast<const uint2*>(a.in + at + uint64_t(e) * a.mp);
        };
        constexpr bool kAddLow = !SPLIT;          // with SPLIT the product has it
        if constexpr (kAddLow) fetch(0);
#pragma unroll
        for (int u = 0; u < FP / 2; ++u) {
            const uint32_t p0 = pw + u * 32u + fk * 8u;
            if constexpr (kAddLow) {
                if (u + 1 < FP / 2) fetch(u + 1);
            }
            float v[FQ][8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                half4_t low = {};
                if constexpr (kAddLow) low = __builtin_bit_cast(half4_t, quad_turn(in[u & 1][e]));
#pragma unroll
                for (int j = 0; j < FQ; ++j) {
                    float r = by_c * value(u, j, e);
                    if constexpr (kAddLow) r = fmaf(by_hi, float(low[j]), r);
                    v[j][e] = r;
                }
            }
            if constexpr (MODE == kApply) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    half4_t h, l;
#pragma unroll
                    for (int j = 0; j < FQ; ++j) {
                        h[j] = half_t(v[j][e]);
                        l[j] = half_t(v[j][e] - float(h[j]));
                    }
                    const uint64_t at = item_out + uint64_t(p0 + e) * a.mp + m0;
                    *reinterpret_cast<uint2*>(a.out + at) = quad_turn(__builtin_bit_cast(uint2, h));
                    *reinterpret_cast<uint2*>(a.out_lo + at) = quad_turn(__builtin_bit_cast(uint2, l));
                }
            } else if (a.tall) {
                // whole vectors of the result's rows lie inside or outside it: its columns are a multiple of 8
#pragma unroll
                for (int j = 0; j < FQ; ++j) {
                    const uint32_t q = mj + 8u * j;
                    if (q >= a.rows || p0 >= a.cols) continue;
                    const uint64_t o = (uint64_t(item) * a.rows + q) * a.cols + p0;
                    float r[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) r[e] = v[j][e] * back;
                    if (!a.update) {
                        float w[8];
                        unpack(*reinterpret_cast<const u32x4_t*>(a.w + o), w);
#pragma unroll
                        for (int e = 0; e < 8; ++e) r[e] = fmaf(-a.step, r[e], w[e] * a.keep);
                    }
                    *reinterpret_cast<u32x4_t*>((a.update ? a.update : a.w_out) + o) = pack(r);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const bool in_range = p0 + e < a.rows && m0 < a.cols;
                    const uint64_t o = (uint64_t(item) * a.rows + p0 + e) * a.cols + m0;
                    float r[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) r[j] = v[j][e] * back;
                    if (!a.update) {
                        uint2 w = make_uint2(0u, 0u);
                        if (in_range) w = *reinterpret_cast<const uint2*>(a.w + o);
                        w = quad_turn(w);
                        r[0] = fmaf(-a.step, r[0], __uint_as_float(w.x << 16) * a.keep);
                        r[1] = fmaf(-a.step, r[1], __uint_as_float(w.x & 0xFFFF0000u) * a.keep);
                        r[2] = fmaf(-a.step, r[2], __uint_as_float(w.y << 16) * a.keep);
                        r[3] = fmaf(-a.step, r[3], __uint_as_float(w.y & 0xFFFF0000u) * a.keep);
                    }
                    const uint2 b = quad_turn(make_uint2(cvt_bf16x2(r[0], r[1]), cvt_bf16x2(r[2], r[3])));
                    if (in_range) *reinterpret_cast<uint2*>((a.update ? a.update : a.w_out) + o) = b;
                }
            }
        }
    }
    if constexpr (kSums) {
        reuse_barrier();
        float* s_sum = reinterpret_cast<float*>(s_op);
        tr *= 0x1p-14f;
        sq *= ti != tj ? 0x1p-27f : 0x1p-28f;              // an entry off the diagonal stands for two
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) {
            tr += __shfl_xor(tr, off, 64);
            sq += __shfl_xor(sq, off, 64);
        }
        if (lane == 0u) {
            s_sum[wave] = tr;
            s_sum[kWaves + wave] = sq;
        }
        __syncthreads();
        if (tid == 0u) {
            tr = sq = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                tr += s_sum[w];
                sq += s_sum[kWaves + w];
            }
            float* out = a.sums + (uint64_t(item) * a.sum_tiles + t) * 2u;
            out[0] = tr;
            out[1] = sq;
        }
    }
}

// ------------------------------------------------------------ host

struct OrthoPlan {
    uint32_t n, m, np, mp;
    uint32_t square, rect, side;           // tiles of the square products and of those with X; square tiles along n
    uint32_t norm_blocks;
    int tall, s;
    size_t x0, x1, lo, a, d, sums, alpha, norm, total;
    size_t lo1, a_lo, d_lo;                 // 64-wide tiles only
    int pair;                               // two steps at once
    size_t t, d2;
};

static size_t ortho_align(size_t v) { return (v + 255) / 256 * 256; }

// 256-wide tiles, one a CU, or 128-wide ones, two a CU: whichever takes fewer
// rounds, a round of 128-wide tiles (half the work) counting 0.75, or 0.33 if
// there is at most one to a CU.  Five steps, ms, square / rectangular products by
// 256 / 256, 128 / 256 and 128 / 128, * what this rule takes:
//   4096 x 4096      1.48*  1.69   1.77     16 x 768 x 2048    0.68   0.58*  0.57
//   2048 x 8192      1.16   0.66*  0.68     128 x 768 x 2048   3.59*  3.97   4.26
//   1024 x 4096      0.65   0.34   0.30*    5503 x 4096        2.06*  2.36   2.34
//   2048 x 2048      0.68   0.44   0.33*    140 x 257 x 1280   1.68   1.74*  1.34
// (1024 x 4096 by 64 / 64 with low parts 0.46.)  The last is what the rule does not
// see: rows that a wider tile pads.
static uint32_t ortho_tile(uint64_t of256, uint64_t of128, uint64_t cus) {
    const double wide = double((of256 + cus - 1) / cus);
    const double small = of128 <= cus ? 0.33 : 0.75 * double((of128 + 2 * cus - 1) / (2 * cus));
    return wide <= small ? 256u : 128u;
}

// Bounds of the steps taken in pairs (see the top): what the steps can amplify a
// rounding by, the product of their largest gains |a + b s^2 + c s^4| (3.4445^5 = 485
// for five default steps), and the smaller side.
constexpr double kPairGrowth = 512.0;
constexpr uint32_t kPairSide = 640;

static OrthoPlan ortho_plan(int64_t batch, int64_t rows, int64_t cols, double growth) {
    OrthoPlan p{};
    p.tall = rows > cols;
    p.n = uint32_t(p.tall ? cols : rows);
    p.m = uint32_t(p.tall ? rows : cols);
    const uint64_t cus = uint64_t(device_cu_count());
    auto along = [](uint32_t v, uint32_t tile) { return uint64_t((v + tile - 1) / tile); };
    auto squares = [&](uint32_t tile) { const uint64_t s = along(p.n, tile); return batch * (s * (s + 1) / 2); };
    auto rects = [&](uint32_t tile) { return batch * along(p.n, tile) * along(p.m, tile); };
    p.rect = rects(128) < cus ? 64u : ortho_tile(rects(256), rects(128), cus);
    p.square = p.rect < 256u ? p.rect : ortho_tile(squares(256), squares(128), cus);
    const uint32_t pad = std::max(p.square, p.rect);
    p.np = (p.n + pad - 1) / pad * pad;
    p.mp = (p.m + pad - 1) / pad * pad;
    p.side = p.np / p.square;
    p.s = int(std::floor(0.5 * std::log2(double(p.n) * double(p.m))));
    if (p.s > 15) p.s = 15;
    const size_t rect = size_t(batch) * p.np * p.mp * 2, sq = size_t(batch) * p.np * p.np * 2;
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t o = at; at += ortho_align(bytes); return o; };
    p.x0 = take(rect);
    p.x1 = take(rect);
    p.lo = take(rect);
    p.a = take(sq);
    p.d = take(sq);
    p.sums = take(size_t(batch) * p.side * (p.side + 1) / 2 * 8);
    p.alpha = take(size_t(batch) * 16);
    // four vectors of 8 per thread and block, while that leaves blocks for every CU
    const uint64_t cells = uint64_t(p.n) * p.m, most = (cus * 8 + batch - 1) / uint64_t(batch);
    const uint64_t want = (cells + 8191) / 8192;
    p.norm_blocks = uint32_t(std::min<uint64_t>(std::min<uint64_t>(want, most), kNormBlocks));
    p.norm = take(size_t(batch) * p.norm_blocks * 8);
    p.pair = p.rect != 64 && p.n >= kPairSide && p.m >= 2u * p.n && growth <= kPairGrowth;
    if (p.pair) {
        p.t = take(sq);
        p.d2 = take(sq);
    }
    if (p.rect == 64) {
        p.lo1 = take(rect);
        p.a_lo = take(sq);
        p.d_lo = take(sq);
    }
    p.total = at;
    return p;
}

static e8q_status_t ortho_check(const void* g, e8q_dtype_t dtype, int64_t batch, int64_t rows, int64_t cols,
                                int32_t steps, float ca, float cb, float cc, const uint32_t* status, double& growth) {
    if (!g || !status || batch <= 0 || rows <= 0 || cols <= 0 || cols % 8) return E8Q_ERR_INVALID;
    if (dtype != E8Q_F32 && dtype != E8Q_BF16) return E8Q_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(g) % 16) return E8Q_ERR_INVALID;
    if (!std::isfinite(ca) || !std::isfinite(cb) || !std::isfinite(cc)) return E8Q_ERR_INVALID;
    if (steps < 1 || steps > 16 || rows > 65536 || cols > 65536 || batch > 65535) return E8Q_ERR_UNSUPPORTED;
    // largest singular value after each step, from [0, 1]: the polynomial at the
    // ends and where its derivative a + 3 b s^2 + 5 c s^4 vanishes
    double top = 1.0;
    growth = 1.0;
    for (int32_t i = 0; i < steps; ++i) {
        const double a = ca, b = cb, c = cc;
        double at[4] = {top, 0.0, 0.0, 0.0}, next = 0.0, gain = std::fabs(a);
        const double disc = 9.0 * b * b - 20.0 * a * c;
        if (c != 0.0 && disc >= 0.0) {
            at[1] = (-3.0 * b + std::sqrt(disc)) / (10.0 * c);
            at[2] = (-3.0 * b - std::sqrt(disc)) / (10.0 * c);
        } else if (c == 0.0 && b != 0.0) {
            at[1] = -a / (3.0 * b);
        }
        at[3] = c != 0.0 ? -b / (2.0 * c) : 0.0;                 // square where the gain is extreme
        for (int j = 0; j < 4; ++j) {
            const double x2 = j == 0 ? top * top : at[j];
            if (x2 < 0.0 || x2 > top * top) continue;
            const double f = a + b * x2 + c * x2 * x2;
            gain = std::fmax(gain, std::fabs(f));
            next = std::fmax(next, std::fabs(f) * std::sqrt(x2));
        }
        if (gain > 7.0 || next > 1.5) return E8Q_ERR_UNSUPPORTED;
        top = next;
        growth *= gain;
    }
    return E8Q_OK;
}

template <int BP, int BQ, int WP, int WQ, int RING, bool SPLIT>
struct OrthoTile {
    static constexpr int kBP = BP, kBQ = BQ, kThreads = WP * WQ * 64;
    static constexpr bool kSplit = SPLIT;
    template <int MODE>
    static constexpr auto kernel = ortho_mul_kernel<BP, BQ, WP, WQ, RING, SPLIT, MODE>;
};

// SQ: the kernels of the square products, RE: those of the products with X.
template <class SQ, class RE>
static void ortho_steps(const OrthoPlan& p, OrthoMul a, int64_t batch, int32_t steps, char* ws, hipStream_t st) {
    constexpr bool SPLIT = SQ::kSplit;
    half_t* x[2] = {reinterpret_cast<half_t*>(ws + p.x0), reinterpret_cast<half_t*>(ws + p.x1)};
    half_t* lo[2] = {reinterpret_cast<half_t*>(ws + p.lo), reinterpret_cast<half_t*>(ws + (SPLIT ? p.lo1 : p.lo))};
    half_t* a_lo = SPLIT ? reinterpret_cast<half_t*>(ws + p.a_lo) : nullptr;
    half_t* d_lo = SPLIT ? reinterpret_cast<half_t*>(ws + p.d_lo) : nullptr;
    half_t *ma = reinterpret_cast<half_t*>(ws + p.a), *md = reinterpret_cast<half_t*>(ws + p.d);
    const uint32_t tri = p.side * (p.side + 1) / 2, tq = p.mp / RE::kBQ;
    const uint64_t rect = uint64_t(p.np) * p.mp, sq = uint64_t(p.np) * p.np;
    a.n = p.n;
    a.np = p.np;
    a.mp = p.mp;
    a.s = p.s;
    a.sums = reinterpret_cast<float*>(ws + p.sums);
    a.sum_tiles = tri;
    a.alpha = reinterpret_cast<float*>(ws + p.alpha);
    a.batch = uint32_t(batch);
    auto square = [&](auto kernel, const half_t* pp, const half_t* pp_lo, const half_t* qq, const half_t* qq_lo,
                      const half_t* in, const half_t* in_lo, half_t* out, half_t* out_lo) {
        a.p = pp;
        a.p_lo = pp_lo;
        a.q = qq;
        a.q_lo = qq_lo;
        a.p_item = a.q_item = in ? sq : rect;
        a.k = in ? p.np : p.mp;
        a.in = in;
        a.in_lo = in_lo;
        a.out = out;
        a.out_lo = out_lo;
        a.tiles_p = p.side;
        a.per_item = tri;
        launch(kernel, dim3(uint32_t(batch) * tri), dim3(SQ::kThreads), 0, st, a);
    };
    int at = 0;                              // which of x, lo holds X
    for (int32_t i = 0; i < steps;) {
        a.second = 0;
        a.pair = p.pair && i + 1 < steps;
        const half_t *e = md, *e_lo = d_lo;
        square(SQ::template kernel<kGram>, x[at], lo[at], x[at], lo[at], nullptr, nullptr, ma, a_lo);
        square(SQ::template kernel<kPoly>, ma, a_lo, ma, a_lo, ma, a_lo, md, d_lo);
        if constexpr (!SPLIT) {
            if (a.pair) {
                half_t *mt = reinterpret_cast<half_t*>(ws + p.t), *md2 = reinterpret_cast<half_t*>(ws + p.d2);
                square(SQ::template kernel<kMix>, ma, nullptr, md, nullptr, ma, nullptr, mt, nullptr);
                square(SQ::template kernel<kMixSum>, md, nullptr, mt, nullptr, mt, nullptr, ma, nullptr);
                a.second = 1;
                square(SQ::template kernel<kPoly>, ma, nullptr, ma, nullptr, ma, nullptr, md2, nullptr);
                square(SQ::template kernel<kJoin>, md2, nullptr, md, nullptr, md, md2, mt, nullptr);
                e = mt;
            }
        }
        i += a.pair ? 2 : 1;
        a.p = e;
        a.p_lo = e_lo;
        a.q = x[at];
        a.q_lo = a.in = lo[at];
        a.p_item = sq;
        a.q_item = rect;
        a.k = p.np;
        a.tiles_p = p.np / RE::kBP;
        a.tiles_q = tq;
        a.per_item = (p.np / RE::kBP) * tq;
        at ^= 1;
        a.out = x[at];
        a.out_lo = lo[at];
        const dim3 grid(uint32_t(batch) * a.per_item);
        if (i < steps) launch(RE::template kernel<kApply>, grid, dim3(RE::kThreads), 0, st, a);
        else launch(RE::template kernel<kLast>, grid, dim3(RE::kThreads), 0, st, a);
    }
}

static void ortho_run(const OrthoPlan& p, OrthoIn in, const OrthoMul& mul, int64_t batch, int64_t rows, int64_t cols,
                      int32_t steps, char* ws, hipStream_t st) {
    in.cells = uint64_t(rows) * uint64_t(cols);
    in.rows = uint32_t(rows);
    in.cols = uint32_t(cols);
    in.np = p.np;
    in.mp = p.mp;
    in.s = p.s;
    in.x = reinterpret_cast<half_t*>(ws + p.x0);
    in.x_lo = reinterpret_cast<half_t*>(ws + p.lo);
    in.norm_blocks = p.norm_blocks;
    in.norm = reinterpret_cast<double*>(ws + p.norm);
    const uint32_t pr = p.tall ? p.mp : p.np, pc = p.tall ? p.np : p.mp;
    launch(ortho_norm_kernel, dim3(p.norm_blocks, uint32_t(batch)), dim3(256), 0, st, in);
    const dim3 split(pc / 64, pr / 64, uint32_t(batch));
    if (p.tall) launch(ortho_split_kernel<true>, split, dim3(256), 0, st, in);
    else launch(ortho_split_kernel<false>, split, dim3(256), 0, st, in);
    typedef OrthoTile<256, 256, 2, 4, 5, false> T256;
    typedef OrthoTile<128, 128, 2, 2, 5, false> T128;
    typedef OrthoTile<64, 64, 2, 1, 3, true> T64;
    if (p.rect == 64) ortho_steps<T64, T64>(p, mul, batch, steps, ws, st);
    else if (p.rect == 128) ortho_steps<T128, T128>(p, mul, batch, steps, ws, st);
    else if (p.square == 128) ortho_steps<T128, T256>(p, mul, batch, steps, ws, st);
    else ortho_steps<T256, T256>(p, mul, batch, steps, ws, st);
}

// The workspace holds the plan, and no launch has 2^32 threads.
static e8q_status_t ortho_fits(const OrthoPlan& p, int64_t batch, const void* ws, size_t bytes) {
    const double tiles = std::max(double(p.side) * (p.side + 1) / 2, double(p.np / p.rect) * (p.mp / p.rect));
    if (double(batch) * tiles >= double(1 << 22)) return E8Q_ERR_UNSUPPORTED;
    return ws && bytes >= p.total && reinterpret_cast<uintptr_t>(ws) % 256 == 0 ? E8Q_OK : E8Q_ERR_INVALID;
}

}  // namespace e8q

extern "C" size_t e8q_orthogonalize_workspace_size(int64_t batch, int64_t rows, int64_t cols) {
    if (batch <= 0 || batch > 65535 || rows <= 0 || rows > 65536 || cols <= 0 || cols > 65536 || cols % 8) return 0;
    return e8q::ortho_plan(batch, rows, cols, 1.0).total;      // with pairs, where the sides allow them
}

extern "C" e8q_status_t e8q_orthogonalize(const void* g, e8q_dtype_t g_dtype, int64_t batch, int64_t rows,
                                          int64_t cols, int32_t steps, float coeff_a, float coeff_b, float coeff_c,
                                          void* update_out, void* workspace, size_t workspace_bytes,
                                          uint32_t* status_dev, void* stream) {
    using namespace e8q;
    double growth = 1.0;
    const e8q_status_t c =
        ortho_check(g, g_dtype, batch, rows, cols, steps, coeff_a, coeff_b, coeff_c, status_dev, growth);
    if (c != E8Q_OK) return c;
    if (!update_out || reinterpret_cast<uintptr_t>(update_out) % 16) return E8Q_ERR_INVALID;
    const OrthoPlan p = ortho_plan(batch, rows, cols, growth);
    const e8q_status_t f = ortho_fits(p, batch, workspace, workspace_bytes);
    if (f != E8Q_OK) return f;
    OrthoIn in{};
    in.g = g;
    in.g_f32 = g_dtype == E8Q_F32;
    in.status = status_dev;
    OrthoMul mul{};
    mul.ca = coeff_a;
    mul.cb = coeff_b;
    mul.cc = coeff_c;
    mul.rows = uint32_t(rows);
    mul.cols = uint32_t(cols);
    mul.tall = p.tall;
    mul.update = static_cast<uint16_t*>(update_out);
    ortho_run(p, in, mul, batch, rows, cols, steps, static_cast<char*>(workspace), reinterpret_cast<hipStream_t>(stream));
    return launch_status();
}

extern "C" e8q_status_t e8q_orthogonal_step(const void* w, void* w_out, const void* grad, e8q_dtype_t grad_dtype,
                                            const float* momentum, float* momentum_out, float mu, int32_t nesterov,
                                            float lr, float decay, float gamma, int64_t batch, int64_t rows,
                                            int64_t cols, int32_t steps, float coeff_a, float coeff_b, float coeff_c,
                                            void* workspace, size_t workspace_bytes, uint32_t* status_dev,
                                            void* stream) {
    using namespace e8q;
    double growth = 1.0;
    const e8q_status_t c =
        ortho_check(grad, grad_dtype, batch, rows, cols, steps, coeff_a, coeff_b, coeff_c, status_dev, growth);
    if (c != E8Q_OK) return c;
    if (!w || !w_out || !momentum || !momentum_out) return E8Q_ERR_INVALID;
    for (const void* q : {w, static_cast<const void*>(w_out), static_cast<const void*>(momentum),
                          static_cast<const void*>(momentum_out)})
        if (reinterpret_cast<uintptr_t>(q) % 16) return E8Q_ERR_INVALID;
    if (w_out == grad || momentum_out == grad || static_cast<void*>(momentum_out) == w_out ||
        static_cast<const void*>(momentum_out) == w || static_cast<const void*>(momentum) == w_out)
        return E8Q_ERR_INVALID;
    if (!std::isfinite(mu) || !std::isfinite(lr) || !std::isfinite(decay) || !std::isfinite(gamma))
        return E8Q_ERR_INVALID;
    const OrthoPlan p = ortho_plan(batch, rows, cols, growth);
    const e8q_status_t f = ortho_fits(p, batch, workspace, workspace_bytes);
    if (f != E8Q_OK) return f;
    OrthoIn in{};
    in.g = grad;
    in.g_f32 = grad_dtype == E8Q_F32;
    in.mom_in = momentum;
    in.mom_out = momentum_out;
    in.mu = mu;
    in.nesterov = nesterov != 0;
    in.status = status_dev;
    OrthoMul mul{};
    mul.ca = coeff_a;
    mul.cb = coeff_b;
    mul.cc = coeff_c;
    mul.rows = uint32_t(rows);
    mul.cols = uint32_t(cols);
    mul.tall = p.tall;
    mul.w = static_cast<const uint16_t*>(w);
    mul.w_out = static_cast<uint16_t*>(w_out);
    mul.keep = 1.0f - lr * decay;
    mul.step = lr * gamma;
    ortho_run(p, in, mul, batch, rows, cols, steps, static_cast<char*>(workspace), reinterpret_cast<hipStream_t>(stream));
    return launch_status();
}

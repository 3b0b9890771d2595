// e8q_embed and its gradient.
//
// The lookup is a gather of rows: each lane takes the widest vector that the
// row length and the pointers allow, and a block as many rows as fill it.
//
// The gradient sums grad_out rows of equal tokens, without atomics on the
// sums: the token ids are sorted (stable, so that the rows of a token stay in
// their order), the sorted positions are cut into chunks of 8 to 128 rows, and a
// block sums the rows of one chunk token by token over a slice of the columns.
// A token whose rows lie inside one chunk is written at once; one that spans
// chunks leaves a float32 partial in each, and a second kernel joins them in
// order.  Every block reads the same number of rows, however often a token
// occurs, and the result does not depend on scheduling.
//
// Sort: least significant digit first, with a digit count and a stable
// placement per tile of 1024 ids; up to 4096 ids take one launch of one block.
//
// What bounds it: writing the table's gradient.  32768 x 4096 bf16 into 131072
// float32 rows: 433 us for the sums and zeros (2.4 GB, 5.6 TB/s), 32 us for the
// sort, 11 us for the joins, 97 us for the lookup (5.5 TB/s).
#include <algorithm>

#include "e8q_device.hpp"
#include "e8q_host.hpp"
#include "e8q_vec.hpp"

namespace e8q {

// ------------------------------------------------------------ lookup

struct EmbedArgs {
    const void* table;
    void* out;
    const void* tokens;
    int i64;
    uint32_t n, vocab;
    uint32_t units;          // vectors per row
    FastDiv units_div;
    uint64_t total;          // n * units
    float scale;
    uint32_t* status;
};

__device__ __forceinline__ int64_t id_at(const void* tokens, int i64, uint64_t i) {
    return i64 ? static_cast<const int64_t*>(tokens)[i] : int64_t(static_cast<const int32_t*>(tokens)[i]);
}

// N consecutive elements as float32, with the widest aligned access (N = 8, 4,
// 2 or 1; the caller has checked the alignment of N elements, up to 16 bytes).
template <typename T, int N>
__device__ __forceinline__ void load_n(const T* p, float (&v)[N]) {
    if constexpr (N * sizeof(T) >= 16) {
#pragma unroll
        for (int i = 0; i < N; i += kVec<T>) {
            float w[kVec<T>];
            unpack(*reinterpret_cast<const u32x4_t*>(p + i), w);
#pragma unroll
            for (int j = 0; j < kVec<T>; ++j) v[i + j] = w[j];
        }
    } else {
        struct alignas(N * sizeof(T)) Pack { T e[N]; };
        const Pack r = *reinterpret_cast<const Pack*>(p);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = widen(r.e[i]);
    }
}

template <typename T, int N>
__device__ __forceinline__ void store_n(T* p, const float (&v)[N]) {
    if constexpr (N * sizeof(T) >= 16) {
#pragma unroll
        for (int i = 0; i < N; i += kVec<T>) {
            float w[kVec<T>];
#pragma unroll
            for (int j = 0; j < kVec<T>; ++j) w[j] = v[i + j];
            *reinterpret_cast<u32x4_t*>(p + i) = pack(w);
        }
    } else {
        struct alignas(N * sizeof(T)) Pack { T e[N]; };
        Pack r;
#pragma unroll
        for (int i = 0; i < N; ++i) r.e[i] = narrow<T>(v[i]);
        *reinterpret_cast<Pack*>(p) = r;
    }
}

template <typename T, typename O, int N>
__global__ __launch_bounds__(256) void embed_kernel(EmbedArgs a) {
    uint32_t flags = 0u;
    for (uint64_t i = uint64_t(blockIdx.x) * 256u + threadIdx.x; i < a.total; i += uint64_t(gridDim.x) * 256u) {
        uint32_t row, u;
        if (a.total <= 0xFFFFFFFFull) {
            row = fdiv(uint32_t(i), a.units_div);
            u = uint32_t(i) - row * a.units;
        } else {
            row = uint32_t(i / a.units);
            u = uint32_t(i - uint64_t(row) * a.units);
        }
        const int64_t t = id_at(a.tokens, a.i64, row);
        float v[N];
        if (t >= 0 && t < int64_t(a.vocab)) {
            load_n<T, N>(static_cast<const T*>(a.table) + (uint64_t(t) * a.units + u) * N, v);
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] *= a.scale;
        } else {
            if (t >= int64_t(a.vocab)) flags |= E8Q_STATUS_BAD_INDEX;
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = 0.0f;
        }
        store_n<O, N>(static_cast<O*>(a.out) + (uint64_t(row) * a.units + u) * N, v);
    }
    flush_status(flags, a.status);
}

// ------------------------------------------------------------ sort

constexpr int kSortBlock = 256;
constexpr int kSortWaves = kSortBlock / kWave;
constexpr int kSortRounds = 4;                               // ids per lane and tile
constexpr uint32_t kSortTile = kSortBlock * kSortRounds;     // 1024
constexpr int kMaxBins = 1024;                               // 10-bit digits
constexpr uint32_t kFewTiles = 64;                           // every tile sums the counts of all
constexpr uint32_t kSmallIds = 4096;                         // one block sorts these
constexpr int kSmallBlock = 1024;

struct SortArgs {
    const void* tokens;
    int i64;
    uint32_t n, vocab;
    const uint32_t* key_in;      // null on the first pass: keys come from the tokens
    const uint32_t* pos_in;
    uint32_t* key_out;
    uint32_t* pos_out;
    uint32_t* counts;            // [bins, tiles] to be scanned, else [tiles, bins]
    uint32_t tiles;
    uint32_t shift, bits;
    int scanned;                 // counts hold the exclusive sums
    uint8_t* zero;               // sort_small_kernel: memory to clear, or null
    uint64_t zero_bytes;
    uint32_t* status;
};

// Ids that contribute nothing sort behind the vocabulary, as key `vocab`.
__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, uint32_t i, uint32_t& flags) {
    if (a.key_in) return a.key_in[i];
    const int64_t t = id_at(a.tokens, a.i64, i);
    if (t >= int64_t(a.vocab)) flags |= E8Q_STATUS_BAD_INDEX;
    return t >= 0 && t < int64_t(a.vocab) ? uint32_t(t) : a.vocab;
}

// Lanes of the wave whose digit equals this lane's (among the live ones).
__device__ __forceinline__ uint64_t same_digit(uint32_t d, uint32_t bits, bool live) {
    uint64_t m = __ballot(live);
    for (uint32_t b = 0; b < bits; ++b) {
        const bool one = (d >> b) & 1u;
        const uint64_t w = __ballot(one);
        m &= one ? w : ~w;
    }
    return m;
}

__global__ __launch_bounds__(kSortBlock) void sort_count_kernel(SortArgs a) {
    __shared__ uint32_t s_count[kMaxBins];
    const uint32_t bins = 1u << a.bits;
    for (uint32_t b = threadIdx.x; b < bins; b += kSortBlock) s_count[b] = 0u;
    __syncthreads();
    uint32_t flags = 0u;
    const uint32_t base = blockIdx.x * kSortTile;
    uint32_t key[kSortRounds];
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        const uint32_t i = base + r * kSortBlock + threadIdx.x;
        if (i < a.n) key[r] = sort_key(a, i, flags);
    }
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r)
        if (base + r * kSortBlock + threadIdx.x < a.n) atomicAdd(&s_count[(key[r] >> a.shift) & (bins - 1u)], 1u);
    flush_status(flags, a.status);
    __syncthreads();
    for (uint32_t b = threadIdx.x; b < bins; b += kSortBlock)
        a.counts[a.scanned ? uint64_t(b) * a.tiles + blockIdx.x : uint64_t(blockIdx.x) * bins + b] = s_count[b];
}

// Exclusive sums of `n` counts in place, by one block of 1024 threads.
__global__ __launch_bounds__(1024) void sort_scan_kernel(uint32_t* counts, uint32_t n) {
    __shared__ uint32_t s_wave[16];
    __shared__ uint32_t s_carry;
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
    if (tid == 0) s_carry = 0u;
    __syncthreads();
    for (uint32_t base = 0; base < n; base += 4096u) {
        uint32_t v[4], sum = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t j = base + tid * 4u + i;
            v[i] = j < n ? counts[j] : 0u;
            sum += v[i];
        }
        uint32_t inc = sum;
#pragma unroll
        for (uint32_t off = 1; off < 64; off <<= 1) {
            const uint32_t o = __shfl_up(inc, off, 64);
            if (lane >= off) inc += o;
        }
        if (lane == 63u) s_wave[wave] = inc;
        __syncthreads();
        uint32_t before = s_carry;
        for (uint32_t w = 0; w < wave; ++w) before += s_wave[w];
        uint32_t at = before + inc - sum;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t j = base + tid * 4u + i;
            if (j < n) counts[j] = at;
            at += v[i];
        }
        __syncthreads();
        if (tid == 1023u) s_carry = at;
        __syncthreads();
    }
}

__global__ __launch_bounds__(kSortBlock) void sort_place_kernel(SortArgs a) {
    __shared__ uint32_t s_at[kSortWaves][kMaxBins];
    const uint32_t bins = 1u << a.bits, tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
    for (uint32_t b = tid; b < bins; b += kSortBlock)
        for (int w = 0; w < kSortWaves; ++w) s_at[w][b] = 0u;
    __syncthreads();
    // wave w takes the tile's ids [w * 256, (w + 1) * 256) in order, 64 a round
    const uint32_t base = blockIdx.x * kSortTile + wave * (kSortTile / kSortWaves) + lane;
    uint32_t key[kSortRounds], pos[kSortRounds], rank[kSortRounds], none = 0u;
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        const uint32_t i = base + r * 64u;
        key[r] = i < a.n ? sort_key(a, i, none) : 0u;
        pos[r] = i < a.n && a.pos_in ? a.pos_in[i] : i;
    }
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        const bool live = base + r * 64u < a.n;
        const uint32_t d = (key[r] >> a.shift) & (bins - 1u);
        const uint64_t m = same_digit(d, a.bits, live);
        const uint32_t under = uint32_t(__popcll(m & ((1ull << lane) - 1ull)));
        if (live) {
            const uint32_t seen = s_at[wave][d];
            rank[r] = seen + under;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (under == 0u) s_at[wave][d] = seen + uint32_t(__popcll(m));
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    // where this tile's ids of each bin start: from the scanned counts, or, while
    // the tiles are few, summed up here (a launch less)
    uint32_t start[kMaxBins / kSortBlock];
    if (a.scanned) {
#pragma unroll
        for (int i = 0; i < kMaxBins / kSortBlock; ++i) {
            const uint32_t b = tid * (kMaxBins / kSortBlock) + i;
            start[i] = b < bins ? a.counts[uint64_t(b) * a.tiles + blockIdx.x] : 0u;
        }
    } else {
        __shared__ uint32_t s_wave[kSortWaves];
        static_assert(kMaxBins / kSortBlock == 4, "four neighbouring bins a thread (digits have two bits at least)");
        uint32_t total[4] = {}, sum = 0u;
        const uint32_t b0 = tid * 4u;
#pragma unroll
        for (int i = 0; i < 4; ++i) start[i] = 0u;
        if (b0 < bins) {
#pragma unroll 8
            for (uint32_t t = 0; t < a.tiles; ++t) {
                const uint4 c = *reinterpret_cast<const uint4*>(a.counts + uint64_t(t) * bins + b0);
                const uint32_t v[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    total[i] += v[i];
                    start[i] += t < blockIdx.x ? v[i] : 0u;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) sum += total[i];
        }
        uint32_t inc = sum;
#pragma unroll
        for (uint32_t off = 1; off < 64; off <<= 1) {
            const uint32_t o = __shfl_up(inc, off, 64);
            if (lane >= off) inc += o;
        }
        if (lane == 63u) s_wave[wave] = inc;
        __syncthreads();
        uint32_t before = inc - sum;
        for (uint32_t w = 0; w < wave; ++w) before += s_wave[w];
#pragma unroll
        for (int i = 0; i < kMaxBins / kSortBlock; ++i) {
            start[i] += before;
            before += total[i];
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMaxBins / kSortBlock; ++i) {
        const uint32_t b = tid * (kMaxBins / kSortBlock) + i;
        if (b >= bins) break;
        uint32_t at = start[i];
        for (int w = 0; w < kSortWaves; ++w) {
            const uint32_t c = s_at[w][b];
            s_at[w][b] = at;
            at += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        if (base + r * 64u < a.n) {
            const uint32_t to = s_at[wave][(key[r] >> a.shift) & (bins - 1u)] + rank[r];
            a.key_out[to] = key[r];
            a.pos_out[to] = pos[r];
        }
    }
}

// The whole sort of up to kSmallIds ids by one block: `passes` digits of
// `bits` bits, ids in LDS.  Wave w holds per_wave ids from w * per_wave on.
// The other blocks clear the table's gradient meanwhile (a few ids name few of
// its rows, and the sort keeps one CU busy).
__global__ __launch_bounds__(kSmallBlock) void sort_small_kernel(SortArgs a, uint32_t passes) {
    constexpr int kWaves = kSmallBlock / kWave, kRounds = int(kSmallIds) / kSmallBlock;
    const uint32_t per_wave = (a.n + kSmallBlock - 1u) / kSmallBlock * 64u;
    __shared__ uint32_t s_key[kSmallIds];
    __shared__ uint16_t s_pos[kSmallIds];
    __shared__ uint16_t s_at[kWaves][kMaxBins];
    __shared__ uint32_t s_wave[kWaves];
    const uint32_t bins = 1u << a.bits, tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
    if (blockIdx.x > 0u) {
        const uint64_t head = min(uint64_t(-reinterpret_cast<uintptr_t>(a.zero) & 15u), a.zero_bytes);
        const uint64_t vecs = (a.zero_bytes - head) / 16u, done = head + vecs * 16u;
        u32x4_t* to = reinterpret_cast<u32x4_t*>(a.zero + head);
        for (uint64_t i = uint64_t(blockIdx.x - 1u) * kSmallBlock + tid; i < vecs;
             i += uint64_t(gridDim.x - 1u) * kSmallBlock)
            to[i] = u32x4_t{};
        if (blockIdx.x == 1u) {
            if (tid < head) a.zero[tid] = 0;
            if (done + tid < a.zero_bytes) a.zero[done + tid] = 0;
        }
        return;
    }
    uint32_t flags = 0u;
    for (uint32_t i = tid; i < a.n; i += kSmallBlock) {
        s_key[i] = sort_key(a, i, flags);
        s_pos[i] = uint16_t(i);
    }
    flush_status(flags, a.status);
    for (uint32_t p = 0; p < passes; ++p) {
        const uint32_t shift = p * a.bits;
        for (uint32_t b = tid; b < bins * kWaves; b += kSmallBlock) s_at[b / bins][b % bins] = 0;
        __syncthreads();
        const uint32_t base = wave * per_wave + lane;
        uint32_t key[kRounds], pos[kRounds], rank[kRounds];
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            if (r * 64u >= per_wave) break;
            const uint32_t i = base + r * 64u;
            const bool live = i < a.n;
            key[r] = live ? s_key[i] : 0u;
            pos[r] = live ? s_pos[i] : 0u;
            const uint32_t d = (key[r] >> shift) & (bins - 1u);
            const uint64_t m = same_digit(d, a.bits, live);
            const uint32_t under = uint32_t(__popcll(m & ((1ull << lane) - 1ull)));
            if (live) {
                const uint32_t seen = s_at[wave][d];
                rank[r] = seen + under;
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                if (under == 0u) s_at[wave][d] = uint16_t(seen + uint32_t(__popcll(m)));
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
        __syncthreads();
        // thread b owns bin b: its total, the exclusive sum over the bins, the waves' offsets
        uint32_t total = 0u;
        if (tid < bins)
            for (int w = 0; w < kWaves; ++w) total += s_at[w][tid];
        uint32_t inc = total;
#pragma unroll
        for (uint32_t off = 1; off < 64; off <<= 1) {
            const uint32_t o = __shfl_up(inc, off, 64);
            if (lane >= off) inc += o;
        }
        if (lane == 63u) s_wave[wave] = inc;
        __syncthreads();
        uint32_t at = inc - total;
        for (uint32_t w = 0; w < wave; ++w) at += s_wave[w];
        if (tid < bins)
            for (int w = 0; w < kWaves; ++w) {
                const uint32_t c = s_at[w][tid];
                s_at[w][tid] = uint16_t(at);
                at += c;
            }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            if (r * 64u < per_wave && base + r * 64u < a.n) {
                const uint32_t to = s_at[wave][(key[r] >> shift) & (bins - 1u)] + rank[r];
                s_key[to] = key[r];
                s_pos[to] = uint16_t(pos[r]);
            }
        }
        __syncthreads();
    }
    for (uint32_t i = tid; i < a.n; i += kSmallBlock) {
        a.key_out[i] = s_key[i];
        a.pos_out[i] = s_pos[i];
    }
}

// ------------------------------------------------------------ sums

constexpr uint32_t kMaxChunk = 128;  // most sorted rows per block
constexpr uint32_t kZeroRows = 16;   // table rows per zero-filling block

struct EmbedBwdArgs {
    const void* g;
    void* gt;                // gradient of the table, or null
    uint16_t* w;             // latents, or null
    const uint32_t* key;     // sorted
    const uint32_t* pos;
    float* part;             // [chunks, 2, dim]: first and last token's partial of a chunk
    uint32_t n, vocab, chunks, chunk;
    uint32_t units;          // vectors per row
    uint32_t slices;         // blocks per chunk
    uint32_t sum_blocks;     // chunks * slices
    float scale, lr;
};

template <typename O, int N>
__device__ __forceinline__ void finish_row(const EmbedBwdArgs& a, uint32_t v, uint32_t u, const float (&acc)[N]) {
    float d[N];
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = a.scale * acc[i];
    const uint64_t at = (uint64_t(v) * a.units + u) * N;
    if (a.gt) store_n<O, N>(static_cast<O*>(a.gt) + at, d);
    if (a.w) {
        float w[N];
        load_n<uint16_t, N>(a.w + at, w);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            w[i] = w[i] - a.lr * d[i];
            w[i] = w[i] != w[i] ? __uint_as_float(0x7FC00000u) : w[i];
        }
        store_n<uint16_t, N>(a.w + at, w);
    }
}

template <typename T, typename O, int N>
__global__ __launch_bounds__(256) void embed_sum_kernel(EmbedBwdArgs a) {
    __shared__ uint32_t s_key[kMaxChunk + 2];
    __shared__ uint32_t s_pos[kMaxChunk];
    const uint32_t tid = threadIdx.x;
    if (blockIdx.x >= a.sum_blocks) {
        // rows that no id names: zeros
        const uint32_t v0 = (blockIdx.x - a.sum_blocks) * kZeroRows;
        if (tid < kZeroRows) {
            uint32_t lo = 0u, hi = a.n;
            const uint32_t v = v0 + tid;
            while (lo < hi) {
                const uint32_t mid = lo + (hi - lo) / 2u;
                if (a.key[mid] < v) lo = mid + 1u;
                else hi = mid;
            }
            s_key[tid] = v >= a.vocab || (lo < a.n && a.key[lo] == v);
        }
        __syncthreads();
        float z[N] = {};
        for (uint32_t r = 0; r < kZeroRows; ++r) {
            if (s_key[r]) continue;
            for (uint32_t u = tid; u < a.units; u += 256u)
                store_n<O, N>(static_cast<O*>(a.gt) + (uint64_t(v0 + r) * a.units + u) * N, z);
        }
        return;
    }
    const uint32_t chunk = blockIdx.x / a.slices, slice = blockIdx.x - chunk * a.slices;
    const uint32_t lo = chunk * a.chunk, cnt = min(a.chunk, a.n - lo);
    // s_key[i + 1] = key of row i; the neighbours' keys tell whether a token spans chunks
    if (tid < a.chunk + 2u) {
        const int64_t i = int64_t(lo) + tid - 1;
        s_key[tid] = i >= 0 && i < int64_t(lo + cnt + 1u) && i < int64_t(a.n) ? a.key[i] : 0xFFFFFFFFu;
    }
    if (tid < cnt) s_pos[tid] = a.pos[lo + tid];
    __syncthreads();
    const uint32_t u = slice * 256u + tid;
    if (u >= a.units) return;
    const T* g = static_cast<const T*>(a.g) + uint64_t(u) * N;
    float acc[N] = {};
    uint32_t start = 0u;
    constexpr uint32_t kBatch = 8;
    for (uint32_t i0 = 0; i0 < cnt; i0 += kBatch) {
        float v[kBatch][N];
#pragma unroll
        for (uint32_t q = 0; q < kBatch; ++q) {
            const uint32_t i = i0 + q;
            if (i < cnt && s_key[i + 1u] < a.vocab) load_n<T, N>(g + uint64_t(s_pos[i]) * a.units * N, v[q]);
        }
#pragma unroll
        for (uint32_t q = 0; q < kBatch; ++q) {
            const uint32_t i = i0 + q;
            if (i >= cnt) break;
            const uint32_t key = s_key[i + 1u];
            if (key >= a.vocab) break;
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] += v[q][j];
            const bool ends = i + 1u == cnt || s_key[i + 2u] != key;
            if (!ends) continue;
            const bool from_before = start == 0u && s_key[0] == key;
            const bool goes_on = i + 1u == cnt && s_key[i + 2u] == key;
            if (goes_on) store_n<float, N>(a.part + ((uint64_t(chunk) * 2u + 1u) * a.units + u) * N, acc);
            else if (from_before) store_n<float, N>(a.part + (uint64_t(chunk) * 2u * a.units + u) * N, acc);
            else finish_row<O, N>(a, key, u, acc);
            start = i + 1u;
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] = 0.0f;
        }
    }
}

// Joins the partials of the token that starts in chunk c and goes on after it.
template <typename O, int N>
__global__ __launch_bounds__(256) void embed_join_kernel(EmbedBwdArgs a) {
    const uint32_t chunk = blockIdx.x / a.slices, slice = blockIdx.x - chunk * a.slices;
    const uint32_t first = chunk * a.chunk, last = min(first + a.chunk, a.n) - 1u;
    const uint32_t key = a.key[last];
    if (last + 1u >= a.n || key >= a.vocab || a.key[last + 1u] != key) return;               // ends here
    if (chunk > 0u && a.key[first] == key && a.key[first - 1u] == key) return;               // started before
    uint32_t end = last + 1u, hi = a.n;                // first row of another token
    while (end < hi) {
        const uint32_t mid = end + (hi - end) / 2u;
        if (a.key[mid] == key) end = mid + 1u;
        else hi = mid;
    }
    const uint32_t u = slice * 256u + threadIdx.x;
    if (u >= a.units) return;
    // this chunk and those it covers whole left their sum as last partial, the
    // chunk where it ends as first
    const uint32_t final = (end - 1u) / a.chunk;
    float acc[N] = {};
    constexpr uint32_t kBatch = 8;
    for (uint32_t c0 = chunk; c0 <= final; c0 += kBatch) {
        float v[kBatch][N];
#pragma unroll
        for (uint32_t q = 0; q < kBatch; ++q)
            if (c0 + q <= final)
                load_n<float, N>(a.part + ((uint64_t(c0 + q) * 2u + (c0 + q < final ? 1u : 0u)) * a.units + u) * N, v[q]);
#pragma unroll
        for (uint32_t q = 0; q < kBatch; ++q)
            if (c0 + q <= final) {
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] += v[q][j];
            }
    }
    finish_row<O, N>(a, key, u, acc);
}

// ------------------------------------------------------------ host

// Elements per lane: the most that divide the row and keep every access
// aligned; at most 16 bytes of the wider type.
static int embed_vec(int64_t dim, size_t esz_a, const void* pa, size_t esz_b, const void* pb, size_t esz_c = 1,
                     const void* pc = nullptr) {
    size_t wide = esz_a > esz_b ? esz_a : esz_b;
    int n = int(16 / wide);
    auto fits = [&](const void* p, size_t e) {
        const size_t b = size_t(n) * e;
        return reinterpret_cast<uintptr_t>(p) % (b > 16 ? 16 : b) == 0;
    };
    while (n > 1 && (dim % n || !fits(pa, esz_a) || !fits(pb, esz_b) || (pc && !fits(pc, esz_c)))) n /= 2;
    return n;
}

static bool embed_index_ok(e8q_index_t t, const void* tokens) {
    return (t == E8Q_I32 || t == E8Q_I64) && reinterpret_cast<uintptr_t>(tokens) % (t == E8Q_I64 ? 8 : 4) == 0;
}

template <typename T, typename O>
static void launch_embed(int n, const EmbedArgs& a, hipStream_t st) {
    const dim3 grid(grid_for(a.total, 256, 32)), block(256);
    switch (n) {
        case 8:
            if constexpr (sizeof(T) == 2 && sizeof(O) == 2) launch(embed_kernel<T, O, 8>, grid, block, 0, st, a);
            break;
        case 4: launch(embed_kernel<T, O, 4>, grid, block, 0, st, a); break;
        case 2: launch(embed_kernel<T, O, 2>, grid, block, 0, st, a); break;
        default: launch(embed_kernel<T, O, 1>, grid, block, 0, st, a); break;
    }
}

struct EmbedPlan {
    uint32_t bits, passes, tiles, chunk, chunks;
    size_t key[2], pos[2], counts, part, total;   // byte offsets
};

static size_t a256(size_t v) { return (v + 255) / 256 * 256; }

static EmbedPlan embed_plan(int64_t n, int64_t vocab, int64_t dim) {
    EmbedPlan p{};
    uint32_t need = 2;
    while ((uint64_t(1) << need) <= uint64_t(vocab)) ++need;      // keys 0 .. vocab
    p.passes = (need + 9) / 10;
    p.bits = (need + p.passes - 1) / p.passes;
    p.tiles = uint32_t((uint64_t(n) + kSortTile - 1) / kSortTile);
    // chunks of 8 rows (one batch of loads) while they are few, longer ones (fewer
    // partials) once there are plenty of blocks: 999 ids of 1001 columns 18 us with
    // chunks of 32, 8 us with 8; 32768 ids of 4096 columns 46 us of joining with
    // chunks of 32, 12 us with 64
    p.chunk = 8;
    while (p.chunk < kMaxChunk && uint64_t(n) / p.chunk > 2 * uint64_t(device_cu_count())) p.chunk *= 2;
    p.chunks = uint32_t((uint64_t(n) + p.chunk - 1) / p.chunk);
    size_t at = 0;
    for (int i = 0; i < 2; ++i) {
        p.key[i] = at;
        at += a256(size_t(n) * 4);
        p.pos[i] = at;
        at += a256(size_t(n) * 4);
    }
    p.counts = at;
    at += a256((size_t(p.tiles) << p.bits) * 4);
    // room for the chunks of every smaller number of ids too (shorter chunks can be
    // more: 4096 ids make 512, 4104 make 257), so that one workspace serves a last,
    // smaller batch
    const uint64_t most = std::min((uint64_t(n) + 7) / 8, 2 * uint64_t(device_cu_count()) + 1);
    p.part = at;
    at += a256(size_t(std::max<uint64_t>(p.chunks, most)) * 2 * size_t(dim) * 4);
    p.total = at;
    return p;
}

template <typename T, typename O, int N>
static void launch_embed_sums(const EmbedBwdArgs& a, uint32_t zero_blocks, hipStream_t st) {
    launch(embed_sum_kernel<T, O, N>, dim3(a.sum_blocks + zero_blocks), dim3(256), 0, st, a);
    if (a.chunks > 1) launch(embed_join_kernel<O, N>, dim3(a.sum_blocks), dim3(256), 0, st, a);
}

template <typename T, typename O>
static void embed_sums(int n, EmbedBwdArgs& a, int64_t dim, bool cleared, hipStream_t st) {
    a.units = uint32_t(dim / n);
    a.slices = (a.units + 255u) / 256u;
    a.sum_blocks = a.chunks * a.slices;
    const uint32_t zero = a.gt && !cleared ? uint32_t((uint64_t(a.vocab) + kZeroRows - 1) / kZeroRows) : 0u;
    switch (n) {
        case 8:
            if constexpr (sizeof(T) == 2 && sizeof(O) == 2) launch_embed_sums<T, O, 8>(a, zero, st);
            break;
        case 4: launch_embed_sums<T, O, 4>(a, zero, st); break;
        case 2: launch_embed_sums<T, O, 2>(a, zero, st); break;
        default: launch_embed_sums<T, O, 1>(a, zero, st); break;
    }
}

}  // namespace e8q

extern "C" e8q_status_t e8q_embed(const void* table, e8q_dtype_t table_dtype, int64_t vocab, int64_t dim,
                                  const void* tokens, e8q_index_t index_type, int64_t n, float scale, void* out,
                                  e8q_dtype_t out_dtype, uint32_t* status_dev, void* stream) {
    using namespace e8q;
    if (!table || !tokens || !out || !status_dev || vocab <= 0 || dim <= 0 || n <= 0) return E8Q_ERR_INVALID;
    if ((table_dtype != E8Q_F32 && table_dtype != E8Q_BF16) || (out_dtype != E8Q_F32 && out_dtype != E8Q_BF16))
        return E8Q_ERR_INVALID;
    if (!embed_index_ok(index_type, tokens)) return E8Q_ERR_INVALID;
    const size_t te = table_dtype == E8Q_BF16 ? 2 : 4, oe = out_dtype == E8Q_BF16 ? 2 : 4;
    if (reinterpret_cast<uintptr_t>(table) % te || reinterpret_cast<uintptr_t>(out) % oe) return E8Q_ERR_INVALID;
    constexpr int64_t kMost = int64_t(1) << 31;
    if (vocab >= kMost || dim >= kMost || n >= kMost) return E8Q_ERR_UNSUPPORTED;
    const int v = embed_vec(dim, te, table, oe, out);
    EmbedArgs a{};
    a.table = table;
    a.out = out;
    a.tokens = tokens;
    a.i64 = index_type == E8Q_I64;
    a.n = uint32_t(n);
    a.vocab = uint32_t(vocab);
    a.units = uint32_t(dim / v);
    a.units_div = make_fastdiv(a.units);
    a.total = uint64_t(n) * a.units;
    a.scale = scale;
    a.status = status_dev;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (table_dtype == E8Q_BF16)
        out_dtype == E8Q_BF16 ? launch_embed<uint16_t, uint16_t>(v, a, s) : launch_embed<uint16_t, float>(v, a, s);
    else
        out_dtype == E8Q_BF16 ? launch_embed<float, uint16_t>(v, a, s) : launch_embed<float, float>(v, a, s);
    return launch_status();
}

extern "C" size_t e8q_embed_backward_workspace_size(int64_t n, int64_t vocab, int64_t dim) {
    constexpr int64_t kMost = int64_t(1) << 31;
    if (n <= 0 || vocab <= 0 || dim <= 0 || n >= kMost || vocab >= kMost || dim >= kMost) return 0;
    return e8q::embed_plan(n, vocab, dim).total;
}

extern "C" e8q_status_t e8q_embed_backward(const void* grad_out, e8q_dtype_t grad_dtype, int64_t n, int64_t dim,
                                           const void* tokens, e8q_index_t index_type, int64_t vocab, float scale,
                                           void* grad_table, e8q_dtype_t table_dtype, void* w_latent, float lr,
                                           void* workspace, size_t workspace_bytes, uint32_t* status_dev,
                                           void* stream) {
    using namespace e8q;
    if (!grad_out || !tokens || !status_dev || vocab <= 0 || dim <= 0 || n <= 0 || (!grad_table && !w_latent))
        return E8Q_ERR_INVALID;
    if ((grad_dtype != E8Q_F32 && grad_dtype != E8Q_BF16) || (table_dtype != E8Q_F32 && table_dtype != E8Q_BF16))
        return E8Q_ERR_INVALID;
    if (!embed_index_ok(index_type, tokens)) return E8Q_ERR_INVALID;
    const size_t ge = grad_dtype == E8Q_BF16 ? 2 : 4, te = table_dtype == E8Q_BF16 ? 2 : 4;
    if (reinterpret_cast<uintptr_t>(grad_out) % ge || reinterpret_cast<uintptr_t>(grad_table) % te ||
        reinterpret_cast<uintptr_t>(w_latent) % 2)
        return E8Q_ERR_INVALID;
    if (grad_table == grad_out || w_latent == grad_out || (w_latent && w_latent == grad_table)) return E8Q_ERR_INVALID;
    constexpr int64_t kMost = int64_t(1) << 31;
    if (vocab >= kMost || dim >= kMost || n >= kMost) return E8Q_ERR_UNSUPPORTED;
    const EmbedPlan p = embed_plan(n, vocab, dim);
    if (!workspace || workspace_bytes < p.total || reinterpret_cast<uintptr_t>(workspace) % 256) return E8Q_ERR_INVALID;
    // blocks of a launch and their threads stay below 2^32
    const double blocks = double(p.chunks) * double((dim + 255) / 256) + double(vocab) / kZeroRows + 1;
    if (blocks >= double(1 << 24)) return E8Q_ERR_UNSUPPORTED;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    SortArgs q{};
    q.tokens = tokens;
    q.i64 = index_type == E8Q_I64;
    q.n = uint32_t(n);
    q.vocab = uint32_t(vocab);
    q.counts = reinterpret_cast<uint32_t*>(ws + p.counts);
    q.tiles = p.tiles;
    q.bits = p.bits;
    q.scanned = p.tiles > kFewTiles;
    q.status = status_dev;
    uint32_t* key[2] = {reinterpret_cast<uint32_t*>(ws + p.key[0]), reinterpret_cast<uint32_t*>(ws + p.key[1])};
    uint32_t* pos[2] = {reinterpret_cast<uint32_t*>(ws + p.pos[0]), reinterpret_cast<uint32_t*>(ws + p.pos[1])};
    int at = 0;
    const bool cleared = uint64_t(n) <= kSmallIds;
    if (cleared) {
        q.key_out = key[0];
        q.pos_out = pos[0];
        q.zero = static_cast<uint8_t*>(grad_table);
        q.zero_bytes = grad_table ? uint64_t(vocab) * uint64_t(dim) * te : 0u;
        const unsigned blocks = 1u + (grad_table ? grid_for(q.zero_bytes / 16 + 1, kSmallBlock * 4, 8) : 0u);
        launch(sort_small_kernel, dim3(blocks), dim3(kSmallBlock), 0, s, q, p.passes);
    } else {
        for (uint32_t i = 0; i < p.passes; ++i) {
            q.shift = i * p.bits;
            q.key_in = i ? key[at] : nullptr;
            q.pos_in = i ? pos[at] : nullptr;
            if (i) at ^= 1;
            q.key_out = key[at];
            q.pos_out = pos[at];
            launch(sort_count_kernel, dim3(p.tiles), dim3(kSortBlock), 0, s, q);
            if (q.scanned) launch(sort_scan_kernel, dim3(1), dim3(1024), 0, s, q.counts, uint32_t(p.tiles << p.bits));
            launch(sort_place_kernel, dim3(p.tiles), dim3(kSortBlock), 0, s, q);
        }
    }
    const int v = embed_vec(dim, ge, grad_out, te, grad_table, 2, w_latent);
    EmbedBwdArgs a{};
    a.g = grad_out;
    a.gt = grad_table;
    a.w = static_cast<uint16_t*>(w_latent);
    a.key = key[at];
    a.pos = pos[at];
    a.part = reinterpret_cast<float*>(ws + p.part);
    a.n = uint32_t(n);
    a.vocab = uint32_t(vocab);
    a.chunks = p.chunks;
    a.chunk = p.chunk;
    a.scale = scale;
    a.lr = lr;
    if (grad_dtype == E8Q_BF16)
        table_dtype == E8Q_BF16 ? embed_sums<uint16_t, uint16_t>(v, a, dim, cleared, s) : embed_sums<uint16_t, float>(v, a, dim, cleared, s);
    else
        table_dtype == E8Q_BF16 ? embed_sums<float, uint16_t>(v, a, dim, cleared, s) : embed_sums<float, float>(v, a, dim, cleared, s);
    return launch_status();
}

// rows.hip -- the gradient of a table's rows from the tokens that looked them
// up, for CDNA4 (gfx950, wave64).
//
// G[v] = s * (sum of dy_t over the t with index_t = v), for every row v, or
// added to what G holds.  The tokens are sorted by row (a stable radix sort, so
// a row's tokens stay in order), and the sorted tokens are summed in tiles of
// equal length, however often a row occurs: a row whose tokens lie within a
// tile is finished there, the others leave a sum per tile that a second kernel
// joins in the tiles' order.  No sum depends on the order in which waves run,
// so equal calls give equal bits.  Sums are FP32, rounded once to G's type.
// An index outside the table sorts behind its last row and counts nowhere.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "lct_internal.h"

namespace lct {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// 16 bytes that start at any element
typedef uint32_t u32x4e __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ uint32_t lane() { return threadIdx.x & 63; }

// ------------------------------------------------------------------ sort by row

// A token's row, or `rows` for an index outside the table.
__device__ __forceinline__ uint32_t key_of(const SortParams &p, uint32_t i) {
    if (p.from) return p.from[i];
    if (p.wide) {
        const int64_t v = static_cast<const int64_t *>(p.index)[i];
        return v >= 0 && v < (int64_t)p.rows ? (uint32_t)v : p.rows;
    }
    const int32_t v = static_cast<const int32_t *>(p.index)[i];
    return v >= 0 && (uint32_t)v < p.rows ? (uint32_t)v : p.rows;
}

// The lanes of the wave with this lane's digit (of those that have one).
__device__ __forceinline__ uint64_t alike(uint32_t digit, uint32_t bits, bool have) {
    uint64_t m = __ballot(have);
    for (uint32_t b = 0; b < bits; ++b) {
        const bool set = digit >> b & 1;
        const uint64_t v = __ballot(set);
        m &= set ? v : ~v;
    }
    return m;
}

// A chunk's tokens of each digit: hist[digit][chunk].
__global__ __launch_bounds__(kSortThreads) void k_sort_count(const SortParams p) {
    __shared__ uint32_t h[kSortDigits];
    const uint32_t digits = 1u << p.bits;
    for (uint32_t d = threadIdx.x; d < digits; d += kSortThreads) h[d] = 0;
    __syncthreads();
    const uint32_t i0 = blockIdx.x * kSortChunk;
    for (uint32_t k = threadIdx.x; k < kSortChunk; k += kSortThreads)
        if (i0 + k < p.count) atomicAdd(&h[key_of(p, i0 + k) >> p.shift & (digits - 1)], 1u);
    __syncthreads();
    for (uint32_t d = threadIdx.x; d < digits; d += kSortThreads) p.hist[(uint64_t)d * p.chunks + blockIdx.x] = h[d];
}

// hist's exclusive running sum, in place, by one workgroup: a run of
// neighbours per thread.
__global__ __launch_bounds__(1024) void k_sort_scan(uint32_t *hist, uint32_t n) {
    __shared__ uint32_t s[16];
    const uint32_t per = (n + 1023) / 1024, a = min(n, threadIdx.x * per), e = min(n, a + per);
    uint32_t sum = 0;
    for (uint32_t i = a; i < e; ++i) sum += hist[i];
    uint32_t inc = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t t = __shfl_up(inc, d, 64);
        if ((int)lane() >= d) inc += t;
    }
    if (lane() == 63) s[threadIdx.x >> 6] = inc;
    __syncthreads();
    uint32_t at = inc - sum;
    for (uint32_t w = 0; w < threadIdx.x >> 6; ++w) at += s[w];
    for (uint32_t i = a; i < e; ++i) {
        const uint32_t v = hist[i];
        hist[i] = at;
        at += v;
    }
}

// The chunk's tokens to their places: a wave takes a run of them, 64 at a
// time, and counts its own digits before it, so that the order within a digit
// stays.
__global__ __launch_bounds__(kSortThreads) void k_sort_place(const SortParams p) {
    constexpr uint32_t W = kSortThreads / 64, R = kSortChunk / kSortThreads;
    __shared__ uint32_t h[W][kSortDigits];
    const uint32_t digits = 1u << p.bits, w = threadIdx.x >> 6, l = lane();
    for (uint32_t d = threadIdx.x; d < W * kSortDigits; d += kSortThreads) (&h[0][0])[d] = 0;
    __syncthreads();
    const uint32_t i0 = blockIdx.x * kSortChunk + w * (R * 64);
    uint32_t key[R], rank[R];
#pragma unroll
    for (uint32_t r = 0; r < R; ++r) {
        const uint32_t i = i0 + r * 64 + l;
        const bool have = i < p.count;
        key[r] = have ? key_of(p, i) : 0u;
        const uint32_t d = key[r] >> p.shift & (digits - 1);
        const uint64_t m = alike(d, p.bits, have);
        const uint32_t before = __popcll(m & ((1ull << l) - 1));
        rank[r] = have ? h[w][d] + before : 0u;
        __builtin_amdgcn_wave_barrier();
        if (have && before == 0) h[w][d] += __popcll(m);
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    // each wave's first place of each digit
    for (uint32_t d = threadIdx.x; d < digits; d += kSortThreads) {
        uint32_t at = p.hist[(uint64_t)d * p.chunks + blockIdx.x];
        for (uint32_t k = 0; k < W; ++k) {
            const uint32_t v = h[k][d];
            h[k][d] = at;
            at += v;
        }
    }
    __syncthreads();
#pragma unroll
    for (uint32_t r = 0; r < R; ++r) {
        const uint32_t i = i0 + r * 64 + l;
        if (i >= p.count) continue;
        const uint32_t to = h[w][key[r] >> p.shift & (digits - 1)] + rank[r];
        p.to[to] = key[r];
        p.to_token[to] = p.from ? p.from_token[i] : i;
    }
}

// ------------------------------------------------------------------ sums

// Eight neighbouring elements (fewer at a row's end: `have`) as floats.
template <int TYPE>
__device__ __forceinline__ void load8(const void *x, uint64_t at, uint32_t have, float (&f)[8]) {
    if (have == 8) {
        if constexpr (TYPE == LCT_FP32) {
            const u32x4 a = *reinterpret_cast<const u32x4e *>(static_cast<const float *>(x) + at);
            const u32x4 b = *reinterpret_cast<const u32x4e *>(static_cast<const float *>(x) + at + 4);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(k < 4 ? a[k] : b[k - 4]);
        } else {
            const u32x4 a = *reinterpret_cast<const u32x4e *>(static_cast<const uint16_t *>(x) + at);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t h = k % 2 ? a[k / 2] >> 16 : a[k / 2] & 0xFFFFu;
                f[k] = TYPE == LCT_BF16 ? __uint_as_float(h << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)h);
            }
        }
        return;
    }
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {
        f[k] = 0.0f;
        if (k >= have) continue;
        if constexpr (TYPE == LCT_FP32) {
            f[k] = static_cast<const float *>(x)[at + k];
        } else {
            const uint32_t h = static_cast<const uint16_t *>(x)[at + k];
            f[k] = TYPE == LCT_BF16 ? __uint_as_float(h << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)h);
        }
    }
}

template <int TYPE>
__device__ __forceinline__ uint32_t bits16(float f) {
    if constexpr (TYPE == LCT_FP16) return __builtin_bit_cast(uint16_t, (_Float16)f);
    return __builtin_bit_cast(uint16_t, (__bf16)f);
}

template <int TYPE>
__device__ __forceinline__ void store8(void *y, uint64_t at, uint32_t have, const float (&f)[8]) {
    if (have == 8) {
        if constexpr (TYPE == LCT_FP32) {
            u32x4 a, b;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                a[k] = __float_as_uint(f[k]);
                b[k] = __float_as_uint(f[k + 4]);
            }
            *reinterpret_cast<u32x4e *>(static_cast<float *>(y) + at) = a;
            *reinterpret_cast<u32x4e *>(static_cast<float *>(y) + at + 4) = b;
        } else {
            u32x4 a;
#pragma unroll
            for (int k = 0; k < 4; ++k) a[k] = bits16<TYPE>(f[2 * k]) | bits16<TYPE>(f[2 * k + 1]) << 16;
            *reinterpret_cast<u32x4e *>(static_cast<uint16_t *>(y) + at) = a;
        }
        return;
    }
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {
        if (k >= have) continue;
        if constexpr (TYPE == LCT_FP32)
            static_cast<float *>(y)[at + k] = f[k];
        else
            static_cast<uint16_t *>(y)[at + k] = (uint16_t)bits16<TYPE>(f[k]);
    }
}

// A finished row's piece: s * sum, or added to what is there.
template <int TO>
__device__ __forceinline__ void finish(const RowGradParams &p, uint64_t at, uint32_t have, float (&acc)[8]) {
    if (p.add) {
        float g[8];
        load8<TO>(p.g, at, have, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = __builtin_fmaf(p.scale, acc[k], g[k]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] *= p.scale;
    }
    store8<TO>(p.g, at, have, acc);
}

// The first of the sorted tokens whose row is at least v, by the whole wave:
// 64 places looked at in each of its steps.
__device__ __forceinline__ uint32_t lower_bound(const uint32_t *key, uint32_t n, uint32_t v) {
    uint32_t lo = 0, len = n;   // the answer lies in [lo, lo + len]
    while (len > 0) {
        const uint32_t step = (len + 63) / 64, i = lane() * step;
        const bool below = i < len && key[lo + i] < v;
        const uint32_t k = __popcll(__ballot(below));   // the first k places are below
        if (k == 0) return lo;
        const uint32_t at = (k - 1) * step + 1;         // past the last of them
        lo += at;
        len = min(step - 1, len - at);
    }
    return lo;
}

// Rows of the table that no token has, cleared: a wave looks at 16 rows.
template <int TO>
__device__ __forceinline__ void clear_rows(const RowGradParams &p, uint32_t wave) {
    const uint32_t v0 = wave * kClearRows;
    if (v0 >= p.rows) return;
    const uint32_t v1 = min(v0 + kClearRows, p.rows);
    uint32_t present = 0;
    uint32_t at = lower_bound(p.key, p.count, v0);
    while (at < p.count) {
        const uint32_t i = at + lane();
        const uint32_t k = i < p.count ? p.key[i] : 0xFFFFFFFFu;
#pragma unroll
        for (uint32_t b = 0; b < kClearRows; ++b) present |= (__ballot(k == v0 + b) != 0 ? 1u : 0u) << b;
        const uint32_t last = (uint32_t)__builtin_amdgcn_readlane((int)k, 63);
        if (last >= v1) break;
        // (a frequent row's tokens are passed over at once)
        at = lower_bound(p.key, p.count, last + 1);
    }
    constexpr uint32_t ES = TO == LCT_FP32 ? 4 : 2;
    for (uint32_t v = v0; v < v1; ++v) {
        if (present >> (v - v0) & 1) continue;
        char *g = static_cast<char *>(p.g) + (uint64_t)v * p.cols * ES;
        const uint64_t bytes = (uint64_t)p.cols * ES;
        uint64_t o = 16ull * lane();
        for (; o + 16 <= bytes; o += 1024) *reinterpret_cast<u32x4e *>(g + o) = u32x4{0u, 0u, 0u, 0u};
        if (o < bytes)
            for (; o < bytes; o += 2) *reinterpret_cast<uint16_t *>(g + o) = 0;
    }
}

// The sorted tokens in tiles of p.tile, 512 columns to a wave (blockIdx.y),
// and behind the tiles' workgroups those that clear rows.  A row that began
// in an earlier tile leaves its sum in part[tile][0], one that goes on into the
// next tile in part[tile][1].
template <int FROM, int TO>
__global__ __launch_bounds__(64) void k_row_sums(const RowGradParams p) {
    const uint32_t wg = blockIdx.x;
    if (wg >= p.tiles) {
        clear_rows<TO>(p, (wg - p.tiles) * gridDim.y + blockIdx.y);
        return;
    }
    const uint64_t c = (uint64_t)blockIdx.y * 512 + 8 * lane();
    const uint32_t have = c < p.cols ? (uint32_t)min<uint64_t>(8, p.cols - c) : 0;
    const uint32_t a = wg * p.tile, e = min(a + p.tile, p.count);
    if (p.key[a] >= p.rows) return;                       // only indices outside the table
    bool open = a > 0 && p.key[a - 1] == p.key[a];        // the present row began before
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    constexpr uint32_t B = 4;                             // rows in flight
    for (uint32_t i = a; i < e; i += B) {
        float x[B][8];
#pragma unroll
        for (uint32_t b = 0; b < B; ++b) {
            const uint32_t t = p.token[min(i + b, e - 1)];
            load8<FROM>(p.dy, t * p.cols + c, have, x[b]);
        }
#pragma unroll
        for (uint32_t b = 0; b < B; ++b) {
            if (i + b >= e) break;
            const uint32_t v = p.key[i + b];
            if (v >= p.rows) return;
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[k] += x[b][k];
            const bool ends = i + b + 1 == p.count || p.key[i + b + 1] != v;
            if (!ends && i + b + 1 < e) continue;
            if (ends && !open)
                finish<TO>(p, v * p.cols + c, have, acc);
            else
                store8<LCT_FP32>(p.part, (2ull * wg + (open ? 0 : 1)) * p.cols + c, have, acc);
            open = false;
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[k] = 0.0f;
        }
    }
}

// The rows that cross tiles, each by the tile in which it begins.
template <int TO>
__global__ __launch_bounds__(64) void k_row_join(const RowGradParams p) {
    const uint32_t wg = blockIdx.x;
    const uint64_t c = (uint64_t)blockIdx.y * 512 + 8 * lane();
    const uint32_t have = c < p.cols ? (uint32_t)min<uint64_t>(8, p.cols - c) : 0;
    const uint32_t a = wg * p.tile, e = min(a + p.tile, p.count);
    if (e == p.count) return;
    const uint32_t v = p.key[e - 1];
    if (v >= p.rows || p.key[e] != v) return;             // its last row ends with it
    if (p.key[a] == v && a > 0 && p.key[a - 1] == v) return;   // and began before it
    float acc[8];
    load8<LCT_FP32>(p.part, (2ull * wg + 1) * p.cols + c, have, acc);
    // tiles that begin with v, to the row's end
    const uint32_t end = lower_bound(p.key, p.count, v + 1);
    const uint32_t last = (end - 1) / p.tile;
    constexpr uint32_t B = 4;
    for (uint32_t t = wg + 1; t <= last; t += B) {
        float x[B][8];
#pragma unroll
        for (uint32_t b = 0; b < B; ++b) load8<LCT_FP32>(p.part, 2ull * min(t + b, last) * p.cols + c, have, x[b]);
#pragma unroll
        for (uint32_t b = 0; b < B; ++b)
            if (t + b <= last)
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[k] += x[b][k];
    }
    finish<TO>(p, v * p.cols + c, have, acc);
}

template <int FROM, int TO>
int launch_sums(const RowGradParams &p, void *stream) {
    const uint32_t cols = (uint32_t)((p.cols + 511) / 512);
    const uint32_t waves = p.add ? 0 : (p.rows + kClearRows - 1) / kClearRows;
    const dim3 grid(p.tiles + (waves + cols - 1) / cols, cols);
    if (grid.x == 0) return hipSuccess;
    hipLaunchKernelGGL((k_row_sums<FROM, TO>), grid, dim3(64), 0, (hipStream_t)stream, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.tiles < 2) return (int)e;
    hipLaunchKernelGGL((k_row_join<TO>), dim3(p.tiles, cols), dim3(64), 0, (hipStream_t)stream, p);
    return (int)hipGetLastError();
}
template <int FROM>
int launch_sums_from(const RowGradParams &p, uint32_t to, void *stream) {
    if (to == LCT_BF16) return launch_sums<FROM, LCT_BF16>(p, stream);
    if (to == LCT_FP16) return launch_sums<FROM, LCT_FP16>(p, stream);
    return launch_sums<FROM, LCT_FP32>(p, stream);
}

}  // namespace

// The tokens sorted by row; *key and *token get the sorted rows and tokens.
int launch_row_sort(SortParams p, const RowScratch &s, uint8_t *scratch, const uint32_t **key, const uint32_t **token,
                    void *stream) {
    uint32_t *keys[2] = {reinterpret_cast<uint32_t *>(scratch + s.key0), reinterpret_cast<uint32_t *>(scratch + s.key1)};
    uint32_t *toks[2] = {reinterpret_cast<uint32_t *>(scratch + s.tok0), reinterpret_cast<uint32_t *>(scratch + s.tok1)};
    uint32_t all = 0;   // bits of the largest key, `rows`
    while (all < 32 && p.rows >> all) ++all;
    const uint32_t passes = std::max(1u, (all + kSortBits - 1) / kSortBits);
    p.hist = reinterpret_cast<uint32_t *>(scratch + s.hist);
    p.chunks = (p.count + kSortChunk - 1) / kSortChunk;
    p.bits = (all + passes - 1) / passes;
    for (uint32_t k = 0; k < passes; ++k) {
        p.shift = k * p.bits;
        p.from = k ? keys[(k - 1) & 1] : nullptr;
        p.from_token = k ? toks[(k - 1) & 1] : nullptr;
        p.to = keys[k & 1];
        p.to_token = toks[k & 1];
        hipLaunchKernelGGL(k_sort_count, dim3(p.chunks), dim3(kSortThreads), 0, (hipStream_t)stream, p);
        hipLaunchKernelGGL(k_sort_scan, dim3(1), dim3(1024), 0, (hipStream_t)stream, p.hist, p.chunks << p.bits);
        hipLaunchKernelGGL(k_sort_place, dim3(p.chunks), dim3(kSortThreads), 0, (hipStream_t)stream, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return (int)e;
    }
    *key = keys[(passes - 1) & 1];
    *token = toks[(passes - 1) & 1];
    return hipSuccess;
}

int launch_row_grad(const RowGradParams &p, uint32_t from, uint32_t to, void *stream) {
    if (from == LCT_BF16) return launch_sums_from<LCT_BF16>(p, to, stream);
    if (from == LCT_FP16) return launch_sums_from<LCT_FP16>(p, to, stream);
    return launch_sums_from<LCT_FP32>(p, to, stream);
}

}  // namespace lct

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

// A chunk's tokens of each digit: hist[chunk][digit].
__global__ __launch_bounds__(kSortThreads) void k_sort_count(const SortParams p) {
    __shared__ uint32_t h[kSortDigits];
    const uint32_t digits = 1u << p.bits;
    for (uint32_t d = threadIdx.x; d < digits; d += kSortThreads) h[d] = 0;
    __syncthreads();
    const uint32_t i0 = blockIdx.x * kSortChunk;
#pragma unroll
    for (uint32_t k = 0; k < kSortChunk; k += kSortThreads) {
        const uint32_t i = i0 + k + threadIdx.x;
        if (i < p.count) atomicAdd(&h[key_of(p, i) >> p.shift & (digits - 1)], 1u);
    }
    __syncthreads();
    for (uint32_t d = threadIdx.x; d < digits; d += kSortThreads) p.hist[blockIdx.x * kSortDigits + d] = h[d];
}

// Many chunks: each digit's running sum over the chunks, in place, its total
// behind them (hist[chunks][digit]).
__global__ __launch_bounds__(64) void k_sort_prefix(uint32_t *hist, uint32_t chunks) {
    const uint32_t d = blockIdx.x * 64 + threadIdx.x;
    uint32_t sum = 0;
    for (uint32_t c = 0; c < chunks; c += 8) {
        uint32_t v[8];
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) v[k] = c + k < chunks ? hist[(uint64_t)(c + k) * kSortDigits + d] : 0u;
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) {
            if (c + k < chunks) hist[(uint64_t)(c + k) * kSortDigits + d] = sum;
            sum += v[k];
        }
    }
    hist[(uint64_t)chunks * kSortDigits + d] = sum;
}

// v's exclusive running sum over the workgroup's threads (T of them).
template <uint32_t T>
__device__ __forceinline__ uint32_t group_scan(uint32_t v, uint32_t (&s)[T / 64]) {
    uint32_t inc = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t t = __shfl_up(inc, d, 64);
        if ((int)lane() >= d) inc += t;
    }
    if (lane() == 63) s[threadIdx.x >> 6] = inc;
    __syncthreads();
    uint32_t at = inc - v;
    for (uint32_t w = 0; w < threadIdx.x >> 6; ++w) at += s[w];
    return at;
}

// Ranks of a wave's R keys a lane within their digits, h being the wave's
// counts (cleared before, its totals after): 64 keys at a time, so that the
// order within a digit stays.
template <uint32_t R>
__device__ __forceinline__ void ranks(const uint32_t (&key)[R], const bool (&have)[R], uint32_t shift, uint32_t bits,
                                      uint32_t *h, uint32_t (&rank)[R]) {
    const uint32_t l = lane();
#pragma unroll
    for (uint32_t r = 0; r < R; ++r) {
        const uint32_t d = key[r] >> shift & ((1u << bits) - 1);
        const uint64_t m = alike(d, bits, have[r]);
        const uint32_t before = __popcll(m & ((1ull << l) - 1));
        rank[r] = have[r] ? h[d] + before : 0u;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (have[r] && before == 0) h[d] += __popcll(m);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// The chunk's tokens to their places.
__global__ __launch_bounds__(kSortThreads) void k_sort_place(const SortParams p) {
    constexpr uint32_t W = kSortThreads / 64, R = kSortChunk / kSortThreads, D = kSortDigits / kSortThreads;
    __shared__ uint32_t h[W][kSortDigits];
    __shared__ uint32_t s[W];
    const uint32_t w = threadIdx.x >> 6, l = lane();
    for (uint32_t d = threadIdx.x; d < W * kSortDigits; d += kSortThreads) (&h[0][0])[d] = 0;
    // this thread's digits, neighbours: all tokens of each, and those of the
    // chunks before this one
    const uint32_t digits = 1u << p.bits, d0 = threadIdx.x * D;
    uint32_t all[D] = {}, mine[D] = {}, sum = 0;
    if (d0 < digits) {
        if (p.chunks <= kSortFew) {
            for (uint32_t c = 0; c < p.chunks; c += 8) {
                uint32_t v[8][D];
#pragma unroll
                for (uint32_t k = 0; k < 8; ++k)
#pragma unroll
                    for (uint32_t e = 0; e < D; ++e)
                        v[k][e] = c + k < p.chunks ? p.hist[(c + k) * kSortDigits + d0 + e] : 0u;
#pragma unroll
                for (uint32_t k = 0; k < 8; ++k)
#pragma unroll
                    for (uint32_t e = 0; e < D; ++e) {
                        if (c + k < blockIdx.x) mine[e] += v[k][e];
                        all[e] += v[k][e];
                    }
            }
        } else {
#pragma unroll
            for (uint32_t e = 0; e < D; ++e) {
                mine[e] = p.hist[(uint64_t)blockIdx.x * kSortDigits + d0 + e];
                all[e] = p.hist[(uint64_t)p.chunks * kSortDigits + d0 + e];
            }
        }
#pragma unroll
        for (uint32_t e = 0; e < D; ++e) {
            if (d0 + e >= digits) all[e] = 0;
            sum += all[e];
        }
    }
    uint32_t at = group_scan<kSortThreads>(sum, s);   // (its barrier: h is cleared)
    const uint32_t i0 = blockIdx.x * kSortChunk + w * (R * 64);
    uint32_t key[R], rank[R];
    bool have[R];
#pragma unroll
    for (uint32_t r = 0; r < R; ++r) {
        const uint32_t i = i0 + r * 64 + l;
        have[r] = i < p.count;
        key[r] = have[r] ? key_of(p, i) : 0u;
    }
    ranks<R>(key, have, p.shift, p.bits, h[w], rank);
    __syncthreads();
    // each wave's first place of each digit
#pragma unroll
    for (uint32_t e = 0; e < D; ++e) {
        if (d0 + e >= digits) break;
        uint32_t to = at + mine[e];
        for (uint32_t k = 0; k < W; ++k) {
            const uint32_t v = h[k][d0 + e];
            h[k][d0 + e] = to;
            to += v;
        }
        at += all[e];
    }
    __syncthreads();
#pragma unroll
    for (uint32_t r = 0; r < R; ++r) {
        const uint32_t i = i0 + r * 64 + l;
        if (!have[r]) continue;
        const uint32_t to = h[w][key[r] >> p.shift & (digits - 1)] + rank[r];
        p.to[to] = key[r];
        p.to_token[to] = p.from ? p.from_token[i] : i;
    }
}

// Few tokens: every pass by one workgroup, in LDS.
__global__ __launch_bounds__(1024) void k_sort_one(const SortParams p) {
    constexpr uint32_t W = 16, R = kSortOne / 1024;
    __shared__ uint32_t h[W][kSortDigits];
    __shared__ uint32_t keys[kSortOne], toks[kSortOne];
    __shared__ uint32_t s[W];
    const uint32_t w = threadIdx.x >> 6, l = lane(), i0 = w * (R * 64);
    const uint32_t digits = 1u << p.bits;
    uint32_t key[R], tok[R], rank[R];
    bool have[R];
#pragma unroll
    for (uint32_t r = 0; r < R; ++r) {
        tok[r] = i0 + r * 64 + l;
        have[r] = tok[r] < p.count;
        key[r] = have[r] ? key_of(p, tok[r]) : 0u;
    }
    for (uint32_t pass = 0; pass < p.passes; ++pass) {
        const uint32_t shift = pass * p.bits;
        for (uint32_t d = threadIdx.x; d < W * kSortDigits; d += 1024) (&h[0][0])[d] = 0;
        __syncthreads();
        ranks<R>(key, have, shift, p.bits, h[w], rank);
        __syncthreads();
        uint32_t sum = 0;
        if (threadIdx.x < digits)
            for (uint32_t k = 0; k < W; ++k) sum += h[k][threadIdx.x];
        uint32_t to = group_scan<1024>(sum, s);
        if (threadIdx.x < digits)
            for (uint32_t k = 0; k < W; ++k) {
                const uint32_t v = h[k][threadIdx.x];
                h[k][threadIdx.x] = to;
                to += v;
            }
        __syncthreads();
#pragma unroll
        for (uint32_t r = 0; r < R; ++r)
            if (have[r]) {
                const uint32_t at = h[w][key[r] >> shift & (digits - 1)] + rank[r];
                keys[at] = key[r];
                toks[at] = tok[r];
            }
        __syncthreads();
#pragma unroll
        for (uint32_t r = 0; r < R; ++r)
            if (have[r]) {
                key[r] = keys[i0 + r * 64 + l];
                tok[r] = toks[i0 + r * 64 + l];
            }
    }
#pragma unroll
    for (uint32_t r = 0; r < R; ++r)
        if (have[r]) {
            p.to[i0 + r * 64 + l] = key[r];
            p.to_token[i0 + r * 64 + l] = tok[r];
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
    p.passes = passes;
    if (p.count <= kSortOne) {
        p.to = keys[0];
        p.to_token = toks[0];
        hipLaunchKernelGGL(k_sort_one, dim3(1), dim3(1024), 0, (hipStream_t)stream, p);
        *key = keys[0];
        *token = toks[0];
        return (int)hipGetLastError();
    }
    for (uint32_t k = 0; k < passes; ++k) {
        p.shift = k * p.bits;
        p.from = k ? keys[(k - 1) & 1] : nullptr;
        p.from_token = k ? toks[(k - 1) & 1] : nullptr;
        p.to = keys[k & 1];
        p.to_token = toks[k & 1];
        hipLaunchKernelGGL(k_sort_count, dim3(p.chunks), dim3(kSortThreads), 0, (hipStream_t)stream, p);
        if (p.chunks > kSortFew)
            hipLaunchKernelGGL(k_sort_prefix, dim3(kSortDigits / 64), dim3(64), 0, (hipStream_t)stream, p.hist, p.chunks);
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

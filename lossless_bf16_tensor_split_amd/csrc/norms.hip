// norms.hip -- norms of many dense tensors, the clip coefficient, and the
// scaling of many tensors by it, for CDNA4 (gfx950, wave64).
//
// A list's tensors are cut into chunks of 2^11 to 2^14 elements, numbered
// through the list; a launch covers at most kListMax tensors, whose pointers
// and sizes travel as kernel arguments (no table to upload, so tensors may
// move from step to step).  Sums of squares are kept in 64 bits from the
// first product on: a BF16 or FP32 square does not fit 32 bits for values
// past 2^64 or below 2^-75, and the sum then needs no care for its order or
// length.  The order is fixed all the same (no atomics), so equal calls give
// equal bits.  The largest magnitude is an integer maximum of the values'
// bits without their sign, which puts infinity above every finite value and
// NaN above infinity: a NaN is never lost.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "lct_internal.h"

namespace lct {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// 16 bytes that start at any element (tensors may be views at any offset)
typedef uint32_t u32x4e __attribute__((ext_vector_type(4), aligned(2)));

constexpr uint32_t kWaves = kNormThreads / 64;

// ------------------------------------------------------------------ accumulators

// A running sum of squares (in 64 bits), or the running maximum of the
// magnitudes' bits.
struct SumSq {
    double a = 0.0, b = 0.0;
    __device__ __forceinline__ void add(float x, float y) {
        a = __builtin_fma((double)x, (double)x, a);
        b = __builtin_fma((double)y, (double)y, b);
    }
    __device__ __forceinline__ double value() const { return a + b; }
    __device__ static __forceinline__ double join(double x, double y) { return x + y; }
};
struct MaxAbs {
    uint32_t m = 0;
    __device__ __forceinline__ void add(float x, float y) {
        m = max(m, max(__float_as_uint(x) & 0x7FFFFFFFu, __float_as_uint(y) & 0x7FFFFFFFu));
    }
    __device__ __forceinline__ double value() const { return (double)__uint_as_float(m); }
    // of two magnitudes, NaN above all
    __device__ static __forceinline__ double join(double x, double y) {
        const uint64_t a = (uint64_t)__double_as_longlong(x) & ~(1ull << 63);
        const uint64_t b = (uint64_t)__double_as_longlong(y) & ~(1ull << 63);
        return __longlong_as_double((long long)(a > b ? a : b));
    }
};

template <class A>
__device__ __forceinline__ double wave_join(double v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v = A::join(v, __shfl_xor(v, d, 64));
    return v;
}

// The workgroup's value in every thread; `slots` holds one double per wave.
// A barrier before the first store lets slots be used again at once.
template <class A>
__device__ __forceinline__ double group_join(double v, double *slots) {
    v = wave_join<A>(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
    __syncthreads();
    double r = slots[0];
    for (uint32_t k = 1; k < blockDim.x / 64; ++k) r = A::join(r, slots[k]);
    return r;
}

// ------------------------------------------------------------------ values

template <int TYPE>
constexpr uint32_t per16() { return TYPE == LCT_FP32 ? 4 : 8; }

__device__ __forceinline__ float half_bits(uint32_t h) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}

template <int TYPE>
__device__ __forceinline__ float element(const void *x, uint64_t i) {
    if (TYPE == LCT_FP32) return static_cast<const float *>(x)[i];
    const uint32_t b = static_cast<const uint16_t *>(x)[i];
    return TYPE == LCT_BF16 ? __uint_as_float(b << 16) : half_bits(b);
}

// The elements of 16 bytes, as floats.
template <int TYPE>
__device__ __forceinline__ void unpack(u32x4 v, float (&f)[per16<TYPE>()]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (TYPE == LCT_FP32) {
            f[k] = __uint_as_float(v[k]);
        } else if constexpr (TYPE == LCT_BF16) {
            f[2 * k] = __uint_as_float(v[k] << 16);
            f[2 * k + 1] = __uint_as_float(v[k] & 0xFFFF0000u);
        } else {
            f[2 * k] = half_bits(v[k] & 0xFFFFu);
            f[2 * k + 1] = half_bits(v[k] >> 16);
        }
    }
}

template <int TYPE, class A>
__device__ __forceinline__ void add16(u32x4 v, A &acc) {
    float f[per16<TYPE>()];
    unpack<TYPE>(v, f);
#pragma unroll
    for (uint32_t k = 0; k < per16<TYPE>(); k += 2) acc.add(f[k], f[k + 1]);
}

// Elements [e0, e0 + m) of x into acc, by `threads` threads of which this is
// number t.
template <int TYPE, class A>
__device__ __forceinline__ void add_range(const void *x, uint64_t e0, uint32_t m, uint32_t t, uint32_t threads,
                                          A &acc) {
    constexpr uint32_t V = per16<TYPE>();
    constexpr uint32_t ES = TYPE == LCT_FP32 ? 4 : 2;
    const char *p = static_cast<const char *>(x) + e0 * ES;
    const uint32_t nv = m / V;
    uint32_t v = t;
    // B loads in flight per thread.  Non-temporal: read once, the values leave
    // the caches to others; 8 GB of BF16 then take 1.21 ms in place of 1.37,
    // and a clip that follows loses nothing it would still have found.
    auto batch = [&](auto B_) {
        constexpr uint32_t B = decltype(B_)::value;
        for (; v + (B - 1) * threads < nv; v += B * threads) {
            u32x4 r[B];
#pragma unroll
            for (uint32_t k = 0; k < B; ++k)
                r[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4e *>(p + 16ull * (v + k * threads)));
#pragma unroll
            for (uint32_t k = 0; k < B; ++k) add16<TYPE>(r[k], acc);
        }
    };
    if (TYPE == LCT_FP32) batch(std::integral_constant<uint32_t, 16>{});   // a whole chunk: 104 us for 110 at 0.65 GB
    batch(std::integral_constant<uint32_t, 8>{});
    batch(std::integral_constant<uint32_t, 4>{});
    for (; v < nv; v += threads) add16<TYPE>(*reinterpret_cast<const u32x4e *>(p + 16ull * v), acc);
    const uint32_t tail = m - nv * V;
    if (t < tail) acc.add(element<TYPE>(x, e0 + nv * V + t), 0.0f);
}

template <class A>
__device__ __forceinline__ void add_typed(uint32_t type, const void *x, uint64_t e0, uint32_t m, uint32_t t,
                                          uint32_t threads, A &acc) {
    if (type == LCT_BF16)
        add_range<LCT_BF16>(x, e0, m, t, threads, acc);
    else if (type == LCT_FP16)
        add_range<LCT_FP16>(x, e0, m, t, threads, acc);
    else
        add_range<LCT_FP32>(x, e0, m, t, threads, acc);
}

// ------------------------------------------------------------------ results

// The norm and the coefficient from the joined value (a sum of squares, or
// the largest magnitude).  A NaN quotient stays NaN: no comparison with it
// holds.
__device__ __forceinline__ lct_norm_t result(double v, const NormArgs &a, bool squares) {
    const double n = fabs(a.scale) * (squares ? sqrt(v) : v);
    const double q = a.max_norm / (n + 1e-6);
    lct_norm_t r;
    r.sum = v;
    r.norm = (float)n;
    r.coef = (float)(a.scale * (q >= 1.0 ? 1.0 : q));
    return r;
}

// The last tensor that starts at or before chunk c (tensors of no elements
// have no chunks, so it is the one that holds c): every lane looks at a few
// tensors, one round trip for all (a search by halves takes eight).
template <uint32_t N>
__device__ __forceinline__ uint32_t tensor_of(const ListArgs<N> &li, uint32_t c) {
    uint32_t k = 0;
#pragma unroll
    for (uint32_t b = 0; b < N; b += 64) {
        const uint32_t j = b + (threadIdx.x & 63);
        k += __popcll(__ballot(j < li.count && li.chunk0[min(j, N)] <= c));
    }
    return __builtin_amdgcn_readfirstlane(k) - 1;
}

// Workgroup i of G takes chunks [first(i), first(i + 1)); chunk c belongs to
// workgroup owner(c).
__device__ __forceinline__ uint32_t run_first(uint32_t i, uint32_t chunks, uint32_t G) {
    return (uint32_t)((uint64_t)i * chunks / G);
}
__device__ __forceinline__ uint32_t run_owner(uint32_t c, uint32_t chunks, uint32_t G) {
    return (uint32_t)((((uint64_t)c + 1) * G - 1) / chunks);
}

// ------------------------------------------------------------------ the list's norm

// Bound by reading: 8 GB of BF16 in 398 tensors take 1.21 ms (6.6 TB/s, 83 % of
// the memory's peak; a device copy reaches 4.8), 0.65 GB of FP32 105 us.  The
// 64-bit conversions and products hide behind the loads.
//
// Each workgroup walks its run of chunks and leaves the run's value in
// p.run[i]; where the tensors' own norms are wanted, the part of the run that
// lies in tensor k goes to p.piece[i + k] (runs and tensors both ascend, so no
// two pairs share a place).
template <class A, uint32_t N>
__global__ __launch_bounds__(kNormThreads) void k_list_norm(const ListNormParams<N> p) {
    __shared__ double slots[kWaves];
    const ListArgs<N> &li = p.list;
    const uint32_t i = blockIdx.x, G = gridDim.x;
    uint32_t c = run_first(i, li.chunks, G);
    const uint32_t end = run_first(i + 1, li.chunks, G);
    uint32_t k = tensor_of(li, c);
    double run = 0.0;
    A acc;
    while (c < end) {
        while (li.chunk0[k + 1] <= c) ++k;   // (the first is at hand)
        const uint32_t stop = min(end, li.chunk0[k + 1]);
        const uint64_t n = li.n[k] & kListElems;
        const uint32_t type = (uint32_t)(li.n[k] >> kListTypeShift);
        for (; c < stop; ++c) {
            const uint64_t at = (uint64_t)(c - li.chunk0[k]) << li.shift;
            add_typed(type, li.x[k], at, (uint32_t)min<uint64_t>(1u << li.shift, n - at), threadIdx.x, kNormThreads, acc);
        }
        if (p.piece) {
            const double v = group_join<A>(acc.value(), slots);
            if (threadIdx.x == 0) p.piece[i + k] = v;
            run = A::join(run, v);
            acc = A();
        }
    }
    if (!p.piece) run = group_join<A>(acc.value(), slots);
    if (threadIdx.x == 0) p.run[i] = run;
}

// After a launch: a wave per tensor joins its pieces (the workgroups after
// the first), and the first workgroup joins all runs into the result.
template <class A>
__global__ __launch_bounds__(1024) void k_list_finish(const ListFinishParams p) {
    __shared__ double slots[16];
    uint32_t b = blockIdx.x;
    if (p.out) {
        if (b == 0) {
            double v = 0.0;
            for (uint64_t j = threadIdx.x; j < p.runs; j += 1024) v = A::join(v, p.run[j]);
            v = group_join<A>(v, slots);
            if (threadIdx.x == 0) *p.out = result(v, p.args, p.squares);
            return;
        }
        --b;
    }
    const uint32_t k = b * 16 + (threadIdx.x >> 6), l = threadIdx.x & 63;
    if (k >= p.count) return;
    double v = 0.0;
    if (p.chunk0[k + 1] > p.chunk0[k]) {
        const uint32_t first = run_owner(p.chunk0[k], p.chunks, p.G);
        const uint32_t last = run_owner(p.chunk0[k + 1] - 1, p.chunks, p.G);
        for (uint32_t i = first + l; i <= last; i += 64) v = A::join(v, p.piece[i + k]);
    }
    v = wave_join<A>(v);
    if (l == 0) p.each[k] = result(v, p.args, p.squares).norm;
}

// A short list in one launch: every wave of a single workgroup takes chunks
// in turn and leaves their values in LDS.  Up to 64 chunks (131,072 elements):
// there a call takes 7.4 us among others and 20 alone, in the two-launch form
// 9.1 and 20; twice as many elements take 12.5 us in one workgroup.
template <class A, uint32_t N>
__global__ __launch_bounds__(kOneThreads) void k_list_one(const ListOneParams<N> p, bool squares) {
    __shared__ double vals[kOneMax];
    const ListArgs<N> &li = p.list;
    const uint32_t w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
    for (uint32_t c = w; c < li.chunks; c += kOneThreads / 64) {
        const uint32_t k = tensor_of(li, c);
        const uint64_t n = li.n[k] & kListElems, at = (uint64_t)(c - li.chunk0[k]) << kOneShift;
        A acc;
        add_typed((uint32_t)(li.n[k] >> kListTypeShift), li.x[k], at, (uint32_t)min<uint64_t>(1u << kOneShift, n - at), l,
                  64, acc);
        const double v = wave_join<A>(acc.value());
        if (l == 0) vals[c] = v;
    }
    __syncthreads();
    if (w == 0) {
        double v = 0.0;
        for (uint32_t c = l; c < li.chunks; c += 64) v = A::join(v, vals[c]);
        v = wave_join<A>(v);
        if (l == 0) *p.out = result(v, p.args, squares);
    }
    if (!p.each) return;
    for (uint32_t k = w; k < li.count; k += kOneThreads / 64) {
        double v = 0.0;
        for (uint32_t c = li.chunk0[k] + l; c < li.chunk0[k + 1]; c += 64) v = A::join(v, vals[c]);
        v = wave_join<A>(v);
        if (l == 0) p.each[k] = result(v, p.args, squares).norm;
    }
}

// The result from part values (every stride-th double), by one workgroup.
template <class A>
__global__ __launch_bounds__(1024) void k_norm_join(const NormJoinParams p) {
    __shared__ double slots[16];
    double v = 0.0;
    for (uint64_t j = threadIdx.x; j < p.count; j += 1024) v = A::join(v, p.part[j * p.stride]);
    v = group_join<A>(v, slots);
    if (threadIdx.x == 0) *p.out = result(v, p.args, p.squares);
}

// After the blocks' values of a compressed tensor or group: the first F
// workgroups join them all, into the result (F = 1) or a value each (fold),
// and each of the others makes the norm of a tensor of the group.
template <class A>
__global__ __launch_bounds__(1024) void k_code_finish(const CodeFinishParams p) {
    __shared__ double slots[16];
    const uint32_t F = p.fold ? kFoldGrid : 1u, i = blockIdx.x;
    uint64_t lo, hi;
    if (i < F) {
        lo = i * p.nblk / F;
        hi = (i + 1) * p.nblk / F;
    } else {
        const GroupEntry e = p.ent[i - F];
        lo = e.blk0;
        hi = lo + e.nblk;
    }
    double v = 0.0;
    for (uint64_t j = lo + threadIdx.x; j < hi; j += 1024) v = A::join(v, p.part[j]);
    v = group_join<A>(v, slots);
    if (threadIdx.x != 0) return;
    if (i >= F)
        p.each[i - F] = result(v, p.args, p.squares).norm;
    else if (p.fold)
        p.fold[i] = v;
    else
        *p.out = result(v, p.args, p.squares);
}

// ------------------------------------------------------------------ clip

// x * c rounded to fp32.  The empty statement keeps the product in a register
// of its own: the compiler otherwise makes one mixed-precision instruction of
// it and a rounding to FP16 that follows, which skips the fp32 rounding, so
// that the bits would depend on the code around.
__device__ __forceinline__ float product(float x, float c) {
    float p = x * c;
    asm("" : "+v"(p));
    return p;
}

// Two values rounded to a 16-bit type (nearest, ties to even; an overflow of
// FP16 gives infinity), the first in the low half.
template <int TYPE>
__device__ __forceinline__ uint32_t round16(float f, float g) {
    if (TYPE == LCT_FP16) {
        typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, f16x2{(_Float16)f, (_Float16)g});
    }
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)f, (__bf16)g});
}

// y[i] = c * x[i] for elements [e0, e0 + m).  Eight elements a thread and
// step: one or two 16-byte accesses on either side.
template <int FROM, int TO>
__device__ __forceinline__ void clip_range(const void *x, void *y, uint64_t e0, uint32_t m, float c) {
    constexpr uint32_t FS = FROM == LCT_FP32 ? 4 : 2, TS = TO == LCT_FP32 ? 4 : 2;
    const char *px = static_cast<const char *>(x) + e0 * FS;
    char *py = static_cast<char *>(y) + e0 * TS;
    const uint32_t nv = m / 8;
    auto load = [&](uint32_t v, u32x4 (&r)[FS / 2]) {
#pragma unroll
        for (uint32_t k = 0; k < FS / 2; ++k)
            r[k] = *reinterpret_cast<const u32x4e *>(px + 8ull * FS * v + 16 * k);
    };
    auto store = [&](uint32_t v, const u32x4 (&r)[FS / 2]) {
        float f[8];
        if constexpr (FROM == LCT_FP32) {
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(r[k / 4][k % 4]);
        } else {
            unpack<FROM>(r[0], f);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = product(f[k], c);
        char *q = py + 8ull * TS * v;
        if constexpr (TO == LCT_FP32) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4 o;
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k] = __float_as_uint(f[4 * h + k]);
                *reinterpret_cast<u32x4e *>(q + 16 * h) = o;
            }
        } else {
            u32x4 o;
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = round16<TO>(f[2 * k], f[2 * k + 1]);
            *reinterpret_cast<u32x4e *>(q) = o;
        }
    };
    uint32_t v = threadIdx.x;
    for (; v + 3 * kNormThreads < nv; v += 4 * kNormThreads) {
        u32x4 r[4][FS / 2];
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) load(v + k * kNormThreads, r[k]);
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) store(v + k * kNormThreads, r[k]);
    }
    for (; v < nv; v += kNormThreads) {
        u32x4 r[FS / 2];
        load(v, r);
        store(v, r);
    }
    const uint32_t t = nv * 8 + threadIdx.x;
    if (t < m) {
        const float f = product(element<FROM>(px, t), c);
        if constexpr (TO == LCT_FP32)
            reinterpret_cast<float *>(py)[t] = f;
        else
            reinterpret_cast<uint16_t *>(py)[t] = (uint16_t)round16<TO>(f, f);
    }
}

template <int FROM>
__device__ __forceinline__ void clip_from(uint32_t to, const void *x, void *y, uint64_t e0, uint32_t m, float c) {
    if (to == LCT_BF16)
        clip_range<FROM, LCT_BF16>(x, y, e0, m, c);
    else if (to == LCT_FP16)
        clip_range<FROM, LCT_FP16>(x, y, e0, m, c);
    else
        clip_range<FROM, LCT_FP32>(x, y, e0, m, c);
}

// A workgroup per chunk: 1.6 G elements from FP32 to BF16 in 1.81 ms (5.3
// TB/s), where 2048 workgroups that walk a run of chunks each take 1.88 ms.
template <uint32_t N>
__global__ __launch_bounds__(kNormThreads) void k_list_clip(const ListClipParams<N> p) {
    const float c = *p.coef;
    const ListArgs<N> &li = p.list;
    const uint32_t at = blockIdx.x;
    const uint32_t k = tensor_of(li, at);
    const uint32_t types = (uint32_t)(li.n[k] >> kListTypeShift);
    const uint32_t from = types & 3u, to = types >> 2;
    // in place, a coefficient of 1 leaves every value as it is
    if (c == 1.0f && li.x[k] == p.y[k]) return;
    const uint64_t e0 = (uint64_t)(at - li.chunk0[k]) << li.shift;
    const uint32_t m = (uint32_t)min<uint64_t>(1u << li.shift, (li.n[k] & kListElems) - e0);
    if (from == LCT_BF16)
        clip_from<LCT_BF16>(to, li.x[k], p.y[k], e0, m, c);
    else if (from == LCT_FP16)
        clip_from<LCT_FP16>(to, li.x[k], p.y[k], e0, m, c);
    else
        clip_from<LCT_FP32>(to, li.x[k], p.y[k], e0, m, c);
}

template <class F>
int launched(F f) {
    f();
    return (int)hipGetLastError();
}

}  // namespace

template <uint32_t N>
int launch_list_norm(const ListNormParams<N> &p, uint32_t grid, bool squares, void *stream) {
    return launched([&] {
        if (squares)
            hipLaunchKernelGGL((k_list_norm<SumSq, N>), dim3(grid), dim3(kNormThreads), 0, (hipStream_t)stream, p);
        else
            hipLaunchKernelGGL((k_list_norm<MaxAbs, N>), dim3(grid), dim3(kNormThreads), 0, (hipStream_t)stream, p);
    });
}
template int launch_list_norm(const ListNormParams<kListFew> &, uint32_t, bool, void *);
template int launch_list_norm(const ListNormParams<kListMax> &, uint32_t, bool, void *);

template <uint32_t N>
int launch_list_one(const ListOneParams<N> &p, bool squares, void *stream) {
    return launched([&] {
        if (squares)
            hipLaunchKernelGGL((k_list_one<SumSq, N>), dim3(1), dim3(kOneThreads), 0, (hipStream_t)stream, p, squares);
        else
            hipLaunchKernelGGL((k_list_one<MaxAbs, N>), dim3(1), dim3(kOneThreads), 0, (hipStream_t)stream, p,
                               squares);
    });
}
template int launch_list_one(const ListOneParams<kListFew> &, bool, void *);
template int launch_list_one(const ListOneParams<kListMax> &, bool, void *);

int launch_list_finish(const ListFinishParams &p, void *stream) {
    const dim3 grid((p.out ? 1 : 0) + (p.each ? (p.count + 15) / 16 : 0));
    return launched([&] {
        if (p.squares)
            hipLaunchKernelGGL(k_list_finish<SumSq>, grid, dim3(1024), 0, (hipStream_t)stream, p);
        else
            hipLaunchKernelGGL(k_list_finish<MaxAbs>, grid, dim3(1024), 0, (hipStream_t)stream, p);
    });
}

int launch_norm_join(const NormJoinParams &p, void *stream) {
    return launched([&] {
        if (p.squares)
            hipLaunchKernelGGL(k_norm_join<SumSq>, dim3(1), dim3(1024), 0, (hipStream_t)stream, p);
        else
            hipLaunchKernelGGL(k_norm_join<MaxAbs>, dim3(1), dim3(1024), 0, (hipStream_t)stream, p);
    });
}

int launch_code_finish(const CodeFinishParams &p, void *stream) {
    const dim3 grid((p.fold ? kFoldGrid : 1u) + (p.each ? p.count : 0u));
    return launched([&] {
        if (p.squares)
            hipLaunchKernelGGL(k_code_finish<SumSq>, grid, dim3(1024), 0, (hipStream_t)stream, p);
        else
            hipLaunchKernelGGL(k_code_finish<MaxAbs>, grid, dim3(1024), 0, (hipStream_t)stream, p);
    });
}

template <uint32_t N>
int launch_list_clip(const ListClipParams<N> &p, void *stream) {
    return launched([&] {
        hipLaunchKernelGGL(k_list_clip<N>, dim3(p.list.chunks), dim3(kNormThreads), 0, (hipStream_t)stream, p);
    });
}
template int launch_list_clip(const ListClipParams<kListFew> &, void *);
template int launch_list_clip(const ListClipParams<kClipMax> &, void *);

}  // namespace lct

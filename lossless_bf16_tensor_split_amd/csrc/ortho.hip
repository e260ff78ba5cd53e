// ortho.hip -- orthogonalising many matrices by Newton-Schulz products, for
// CDNA4 (gfx950, wave64).
//
// For a matrix X of m rows and n >= m columns (a taller one is taken
// transposed), X0 = x / (|x| + 1e-7) and then, `steps` times,
//     A = X X',  B = b A + c A A,  X <- a X + B X,
// an odd polynomial of X's singular values that drives them towards one.
//
// Number format.  The first steps multiply small singular values by a (3.4 a
// step, 485 in five), and what a rounding adds to directions that X barely
// has is multiplied with them.  Products of BF16 operands so leave errors of
// 2 % of the result, and 24 % where X is of low rank.  Here the matrix units
// work on FP16 operands (their rate is BF16's, their rounding eight times
// finer), all held scaled by a power of two that keeps them away from both
// ends of FP16's range, and three places keep what one FP16 number would lose:
//   - X is kept as a pair of FP16 numbers (22 bits), whose sum enters a X;
//   - A is kept as a pair too, and A A is summed as hi hi + hi lo + lo hi;
//   - sums are FP32 throughout.
// X's high part alone enters the products X X' and B X, and B is one FP16
// number: those roundings act within the rows that X has.  The result is then
// 1.7e-3 to 2.3e-3 off the exact one (norms), of which rounding it to BF16
// makes 1.66e-3.
//
// Layout.  Every operand of a product is read along its rows: X X' from X,
// A A from A (symmetric), and B X from B and X transposed, of which a copy is
// kept (written by the kernel that makes the new X).  Rows and columns are
// padded with zeros to whole tiles, so the inner loops check nothing.
#include <hip/hip_runtime.h>

#include <atomic>

#include "lct_internal.h"

namespace lct {
namespace {

typedef _Float16 f16;
typedef f16 f16x4 __attribute__((ext_vector_type(4)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(1))) const uint8_t glb_u8;

// Where a matrix's parts lie in the working memory (elements of FP16).
struct Parts {
    f16 *xh, *xl, *xt[2], *ah, *al, *bh;
};
__device__ __forceinline__ Parts parts_of(uint8_t *scratch, const OrthoMat &o) {
    f16 *p = reinterpret_cast<f16 *>(scratch + o.off);
    const uint64_t x = (uint64_t)o.mp * o.np, a = (uint64_t)o.mp * o.mp;
    Parts r;
    r.xh = p;
    r.xl = p + x;
    r.xt[0] = p + 2 * x;
    r.xt[1] = p + 3 * x;
    r.ah = p + 4 * x;
    r.al = r.ah + a;
    r.bh = r.al + a;
    return r;
}

// The matrix whose tiles of launch kind `f` include tile t.
template <class F>
__device__ __forceinline__ uint32_t matrix_of(const OrthoParams &p, uint32_t t, F f) {
    const uint32_t l = threadIdx.x & 63;
    const bool at = l < p.count && f(p.mat[l < p.count ? l : 0]) <= t;
    return __builtin_amdgcn_readfirstlane(__popcll(__ballot(at))) - 1;
}

// ------------------------------------------------------------------ the first X

constexpr uint32_t kPrepTile = 64;

__device__ __forceinline__ float value(const void *x, uint32_t type, uint64_t i) {
    if (type == LCT_FP32) return static_cast<const float *>(x)[i];
    const uint32_t b = static_cast<const uint16_t *>(x)[i];
    return type == LCT_BF16 ? __uint_as_float(b << 16) : (float)__builtin_bit_cast(f16, (uint16_t)b);
}

// X0, scaled, from the input and its norm: both orientations, a 64 x 64 tile
// per workgroup.  A matrix whose norm is not finite becomes NaN throughout.
__global__ __launch_bounds__(256) void k_ortho_prep(const OrthoParams p) {
    __shared__ float tile[kPrepTile][kPrepTile + 1];
    const uint32_t k = matrix_of(p, blockIdx.x, [](const OrthoMat &o) { return o.prep0; });
    const OrthoMat &o = p.mat[k];
    const Parts w = parts_of(p.scratch, o);
    const uint32_t t = blockIdx.x - o.prep0, nt = o.np / kPrepTile;
    const uint32_t i0 = t / nt * kPrepTile, j0 = t % nt * kPrepTile;
    const float norm = p.norm[o.index];
    const float inv = norm <= 3.0e38f ? (float)(p.xscale / ((double)norm + 1e-7)) : __builtin_nanf("");
    const uint32_t c = threadIdx.x % 64, r0 = threadIdx.x / 64;
    if (!o.tall) {
        for (uint32_t r = r0; r < kPrepTile; r += 4) {
            const uint32_t i = i0 + r, j = j0 + c;
            tile[r][c] = i < o.m && j < o.n ? value(o.x, o.type, (uint64_t)i * o.n + j) * inv : 0.0f;
        }
    } else {
        for (uint32_t r = r0; r < kPrepTile; r += 4) {
            const uint32_t j = j0 + r, i = i0 + c;
            tile[c][r] = i < o.m && j < o.n ? value(o.x, o.type, (uint64_t)j * o.m + i) * inv : 0.0f;
        }
    }
    __syncthreads();
    for (uint32_t r = r0; r < kPrepTile; r += 4) {
        const float v = tile[r][c];
        const f16 h = (f16)v;
        const uint64_t at = (uint64_t)(i0 + r) * o.np + j0 + c;
        w.xh[at] = h;
        w.xl[at] = (f16)(v - (float)h);
        w.xt[0][(uint64_t)(j0 + r) * o.mp + i0 + c] = (f16)tile[c][r];
    }
}

// ------------------------------------------------------------------ products

// The product of P's rows with Q's rows over K (both read along their rows),
// a T x T tile per workgroup of WM x WN waves.  K advances by 64 elements
// (128 bytes of a row) a step; two LDS buffers alternate, filled by loads that
// go to LDS directly.  A row's eight 16-byte pieces are stored rotated by an
// exclusive-or with the row's number modulo 8: the fragments' reads (32 rows
// of one column of pieces) then touch every bank equally.
constexpr uint32_t kRowB = 128;

template <uint32_t T, uint32_t WM, uint32_t WN>
struct Product {
    static constexpr uint32_t kWaves = WM * WN;
    static constexpr uint32_t FM = T / (32 * WM), FN = T / (32 * WN);
    static constexpr uint32_t kSide = T * kRowB;        // LDS bytes of one operand's step
    static constexpr uint32_t kBuf = 2 * kSide;
    f32x16 acc[FM][FN];

    // Rows r0.. of g (a step's 128 bytes of each, at column byte c) to LDS.
    __device__ __forceinline__ void fetch(const f16 *g, uint64_t ld, uint32_t c, uint8_t *lds) {
        const uint32_t l = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const uint8_t *src = reinterpret_cast<const uint8_t *>(g) + c + 16 * ((l & 7) ^ (l >> 3));
#pragma unroll
        for (uint32_t it = 0; it < T / (8 * kWaves); ++it) {
            const uint32_t r = (it * kWaves + w) * 8;
            __builtin_amdgcn_global_load_lds(
                reinterpret_cast<glb_u8 *>(reinterpret_cast<uintptr_t>(src + 2 * ld * (r + (l >> 3)))),
                (lds_u8 *)(lds + r * kRowB), 16, 0, 0);
        }
    }

    // segs pairs of operands (p[s], q[s]), each of `steps` steps of 64.
    __device__ __forceinline__ void run(const f16 *const *ps, const f16 *const *qs, uint32_t segs, uint32_t steps,
                                        uint64_t ldp, uint64_t ldq, uint8_t *lds) {
        const uint32_t l = threadIdx.x & 63, w = threadIdx.x >> 6;
        const uint32_t wm = w / WN, wn = w % WN;
#pragma unroll
        for (uint32_t a = 0; a < FM; ++a)
#pragma unroll
            for (uint32_t b = 0; b < FN; ++b) acc[a][b] = f32x16{0.0f};
        const uint32_t total = segs * steps;
        const uint32_t pr = (wm * FM * 32 + (l & 31)) * kRowB, qr = (wn * FN * 32 + (l & 31)) * kRowB + kSide;
        auto get = [&](uint32_t k, uint8_t *buf) {
            const uint32_t s = k / steps, c = (k - s * steps) * kRowB;
            fetch(ps[s], ldp, c, buf);
            fetch(qs[s], ldq, c, buf + kSide);
        };
        auto step = [&](const uint8_t *buf) {
#pragma unroll
            for (uint32_t ks = 0; ks < 4; ++ks) {
                const uint32_t slot = 16 * ((2 * ks + (l >> 5)) ^ (l & 7));
                f16x8 a[FM], b[FN];
#pragma unroll
                for (uint32_t f = 0; f < FM; ++f)
                    a[f] = *reinterpret_cast<const f16x8 *>(buf + pr + f * 32 * kRowB + slot);
#pragma unroll
                for (uint32_t f = 0; f < FN; ++f)
                    b[f] = *reinterpret_cast<const f16x8 *>(buf + qr + f * 32 * kRowB + slot);
#pragma unroll
                for (uint32_t f = 0; f < FM; ++f)
#pragma unroll
                    for (uint32_t g = 0; g < FN; ++g)
                        acc[f][g] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a[f], b[g], acc[f][g], 0, 0, 0);
            }
        };
        get(0, lds);
        for (uint32_t k = 0; k < total; ++k) {
            __builtin_amdgcn_s_waitcnt(0x0F70);   // the step's loads are in LDS (vmcnt 0)
            __syncthreads();
            if (k + 1 < total) get(k + 1, lds + ((k + 1) & 1) * kBuf);
            step(lds + (k & 1) * kBuf);
        }
    }

    // f(i, j, v): v are the values of rows i..i+3 of column j of the tile
    template <class F>
    __device__ __forceinline__ void each(F f) {
        const uint32_t l = threadIdx.x & 63, w = threadIdx.x >> 6;
        const uint32_t wm = w / WN, wn = w % WN;
#pragma unroll
        for (uint32_t a = 0; a < FM; ++a)
#pragma unroll
            for (uint32_t b = 0; b < FN; ++b)
#pragma unroll
                for (uint32_t r = 0; r < 4; ++r) {
                    const float v[4] = {acc[a][b][4 * r], acc[a][b][4 * r + 1], acc[a][b][4 * r + 2],
                                        acc[a][b][4 * r + 3]};
                    f((wm * FM + a) * 32 + 8 * r + 4 * (l >> 5), (wn * FN + b) * 32 + (l & 31), v);
                }
    }
};

// Tile t of the upper triangle of a square of s x s tiles, row by row.
__device__ __forceinline__ void triangle(uint32_t t, uint32_t s, uint32_t &i, uint32_t &j) {
    i = 0;
    uint32_t len = s;
    while (t >= len) {
        t -= len;
        --len;
        ++i;
    }
    j = i + t;
}

// A = X X' (SQUARE false) or B = b A + c A A: the tiles on and above the
// diagonal, each written to its mirror image too.
template <uint32_t T, uint32_t WM, uint32_t WN, bool SQUARE>
__global__ __launch_bounds__(64 * WM * WN) void k_ortho_sym(const OrthoParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t k = matrix_of(p, blockIdx.x, [](const OrthoMat &o) { return o.sym0; });
    const OrthoMat &o = p.mat[k];
    const Parts w = parts_of(p.scratch, o);
    uint32_t ti, tj;
    triangle(blockIdx.x - o.sym0, o.mp / T, ti, tj);
    const uint32_t i0 = ti * T, j0 = tj * T;
    Product<T, WM, WN> pr;
    const uint64_t ld = SQUARE ? o.mp : o.np;
    if (SQUARE) {
        const f16 *ps[3] = {w.ah + i0 * ld, w.ah + i0 * ld, w.al + i0 * ld};
        const f16 *qs[3] = {w.ah + j0 * ld, w.al + j0 * ld, w.ah + j0 * ld};
        pr.run(ps, qs, 3, o.mp / 64, ld, ld, smem);
    } else {
        const f16 *ps[1] = {w.xh + i0 * ld}, *qs[1] = {w.xh + j0 * ld};
        pr.run(ps, qs, 1, o.np / 64, ld, ld, smem);
    }
    pr.each([&](uint32_t i, uint32_t j, const float (&v)[4]) {
        const uint64_t at = (uint64_t)(i0 + i) * o.mp + j0 + j, mirror = (uint64_t)(j0 + j) * o.mp + i0 + i;
        f16x4 h, lo;
#pragma unroll
        for (uint32_t r = 0; r < 4; ++r) {
            if (SQUARE) {
                const uint64_t e = at + (uint64_t)r * o.mp;
                h[r] = (f16)(p.ka * ((float)w.ah[e] + (float)w.al[e]) + p.kaa * v[r]);
                w.bh[e] = h[r];
            } else {
                const float f = p.kx * v[r];
                h[r] = (f16)f;
                lo[r] = (f16)(f - (float)h[r]);
                w.ah[at + (uint64_t)r * o.mp] = h[r];
                w.al[at + (uint64_t)r * o.mp] = lo[r];
            }
        }
        if (ti != tj) {
            if (SQUARE) {
                *reinterpret_cast<f16x4 *>(w.bh + mirror) = h;
            } else {
                *reinterpret_cast<f16x4 *>(w.ah + mirror) = h;
                *reinterpret_cast<f16x4 *>(w.al + mirror) = lo;
            }
        }
    });
}

// X <- a X + B X; the last step writes y in its place.
template <uint32_t T, uint32_t WM, uint32_t WN>
__global__ __launch_bounds__(64 * WM * WN) void k_ortho_next(const OrthoParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t k = matrix_of(p, blockIdx.x, [](const OrthoMat &o) { return o.next0; });
    const OrthoMat &o = p.mat[k];
    const Parts w = parts_of(p.scratch, o);
    const uint32_t t = blockIdx.x - o.next0, mt = o.mp / T;
    const uint32_t i0 = t % mt * T, j0 = t / mt * T;
    Product<T, WM, WN> pr;
    const f16 *ps[1] = {w.bh + (uint64_t)i0 * o.mp}, *qs[1] = {w.xt[p.turn] + (uint64_t)j0 * o.mp};
    pr.run(ps, qs, 1, o.mp / 64, o.mp, o.mp, smem);
    const bool last = p.last;
    pr.each([&](uint32_t i, uint32_t j, const float (&v)[4]) {
        const uint64_t at = (uint64_t)(i0 + i) * o.np + j0 + j;
        f16x4 h;
#pragma unroll
        for (uint32_t r = 0; r < 4; ++r) {
            const uint64_t e = at + (uint64_t)r * o.np;
            const float x = p.a * ((float)w.xh[e] + (float)w.xl[e]) + p.kbx * v[r];
            if (!last) {
                h[r] = (f16)x;
                w.xh[e] = h[r];
                w.xl[e] = (f16)(x - (float)h[r]);
            } else if (i0 + i + r < o.m && j0 + j < o.n) {
                const uint64_t ye = o.tall ? (uint64_t)(j0 + j) * o.m + i0 + i + r : (uint64_t)(i0 + i + r) * o.n + j0 + j;
                static_cast<__bf16 *>(o.y)[ye] = (__bf16)(o.scale * x);
            }
        }
        if (!last) *reinterpret_cast<f16x4 *>(w.xt[p.turn ^ 1] + (uint64_t)(j0 + j) * o.mp + i0 + i) = h;
    });
}

std::atomic<size_t> g_granted[8];

int launch_tiles(const void *fn, uint32_t grid, uint32_t threads, size_t lds, const OrthoParams &p, void *stream,
                 std::atomic<size_t> &granted) {
    if (lds > 64 * 1024 && lds > granted.load()) {
        const hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return (int)e;
        granted.store(lds);
    }
    void *args[] = {const_cast<OrthoParams *>(&p)};
    const hipError_t e = hipLaunchKernel(fn, dim3(grid), dim3(threads), args, lds, (hipStream_t)stream);
    return (int)(e != hipSuccess ? e : hipGetLastError());
}

template <uint32_t T, uint32_t WM, uint32_t WN>
int run_batch(OrthoParams &p, const OrthoBatch &b, uint32_t steps, void *stream) {
    const void *gram = reinterpret_cast<const void *>(&k_ortho_sym<T, WM, WN, false>);
    const void *square = reinterpret_cast<const void *>(&k_ortho_sym<T, WM, WN, true>);
    const void *next = reinterpret_cast<const void *>(&k_ortho_next<T, WM, WN>);
    const size_t lds = 2 * Product<T, WM, WN>::kBuf;
    const uint32_t threads = 64 * WM * WN;
    for (uint32_t s = 0; s < steps; ++s) {
        p.turn = s & 1;
        p.last = s + 1 == steps;
        int e = launch_tiles(gram, b.sym_tiles, threads, lds, p, stream, g_granted[0]);
        if (e == hipSuccess) e = launch_tiles(square, b.sym_tiles, threads, lds, p, stream, g_granted[1]);
        if (e == hipSuccess) e = launch_tiles(next, b.next_tiles, threads, lds, p, stream, g_granted[2]);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

int launch_ortho(OrthoParams &p, const OrthoBatch &b, uint32_t steps, void *stream) {
    hipLaunchKernelGGL(k_ortho_prep, dim3(b.prep_tiles), dim3(256), 0, (hipStream_t)stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
    return run_batch<kOrthoTile, 2, 2>(p, b, steps, stream);
}

}  // namespace lct

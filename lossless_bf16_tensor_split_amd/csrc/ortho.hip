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
// number: those roundings act within the rows that X has.  Rounding the result
// to BF16 leaves 1.66e-3 of it (norms); with these roundings it is, after 1 to
// 3 steps, 1.7e-3 to 1.8e-3 off the exact one, 1.7e-3 to 2.1e-3 after 4, 1.8e-3
// to 2.4e-3 after 5, 2.4e-3 to 3.6e-3 after 8, 3.3e-3 to 4.7e-3 after 12 and
// 5e-3 to 3e-2 after 16 to 32 (257 x 257 to 4096 x 4096, full and low rank and
// with rows that fade by e^8): the usual coefficients drive no singular value to
// a fixed point, and what a step leaves goes on growing.  Those that do, (15,
// -10, 3) / 8 and (3, -1, 0) / 2, stay at 1.7e-3 to 1.8e-3 after 32.  Of short
// matrices (kOrthoPairs), whose few elements would leave 2.4e-3 to 5e-3 after
// five, every operand is a pair and every product three: 1.6e-3 to 1.7e-3 after
// any number of steps.
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
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(1))) const uint8_t glb_u8;

// Where a matrix's parts lie in the working memory (elements of FP16).
struct Parts {
    f16 *xh, *xl, *xt0, *xt1, *ah, *al, *bh;
    f16 *xtl0, *xtl1, *bl;   // low parts of X' and B, where every operand is a pair
};
__device__ __forceinline__ Parts parts_of(uint8_t *scratch, const OrthoMat &o) {
    f16 *p = reinterpret_cast<f16 *>(scratch + o.off);
    const uint64_t x = (uint64_t)o.mp * o.np, a = (uint64_t)o.mp * o.mp;
    Parts r;
    r.xh = p;
    r.xl = p + x;
    r.xt0 = p + 2 * x;
    r.xt1 = p + 3 * x;
    r.ah = p + 4 * x;
    r.al = r.ah + a;
    r.bh = r.al + a;
    r.bl = r.bh + a;
    r.xtl0 = r.bl + a;
    r.xtl1 = r.xtl0 + x;
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
    const uint32_t tl = blockIdx.x - o.prep0, nt = o.np / kPrepTile;
    const uint32_t i0 = tl / nt * kPrepTile, j0 = tl % nt * kPrepTile;
    const float norm = p.norm[o.index];
    // (false for NaN)
    const float inv = norm < __builtin_inff() ? (float)(p.xscale / ((double)norm + 1e-7)) : __builtin_nanf("");
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
        const uint64_t t = (uint64_t)(j0 + r) * o.mp + i0 + c;
        const float u = tile[c][r];
        w.xt0[t] = (f16)u;
        if (o.pairs) w.xtl0[t] = (f16)(u - (float)(f16)u);
    }
}

// ------------------------------------------------------------------ products

// The product of P's rows with Q's rows over K (both read along their rows),
// a TP x TQ tile per workgroup of four waves, a quarter each.  K advances by 32
// elements (64 bytes of a row) a step through NB buffers in LDS, filled by
// loads that go there directly.  A row's four 16-byte pieces are stored
// exchanged by an exclusive-or with the row's number over 4, so that the
// fragments' reads (32 rows of one column of pieces) touch every bank equally.
//
// The matrix units wait for nothing but the data: a wave reads the next
// fragments while it multiplies the present ones, asks for one load at a
// time among them (sixteen at once keep it from issuing products for half a
// step), and has NB - 2 steps' loads under way when it waits for the one after
// the present step.  The barrier lies between a step's halves: by then every
// read of the step is done, so its buffer is free for the loads that follow.
constexpr uint32_t kRowB = 64;
constexpr uint32_t kStep = kRowB / 2;
constexpr uint32_t kThreads = 256;

template <uint32_t TP, uint32_t TQ, uint32_t NB>
struct Product {
    static constexpr uint32_t FP = TP / 64, FQ = TQ / 64;   // fragments of 32 along the sides of a wave's part
    static constexpr uint32_t SP = TP / 2, SQ = TQ / 2;     // its sides
    static constexpr uint32_t kSide = TP * kRowB;           // LDS bytes of P's step; Q's follow
    static constexpr uint32_t kBuf = (TP + TQ) * kRowB;
    static constexpr uint32_t kLds = NB * kBuf;
    static constexpr uint32_t kPart = 2 * SP * SQ;          // bytes of a wave's part as 16-bit numbers
    static_assert(kLds >= 4 * kPart, "the waves' parts pass through LDS");
    // acc[a][b][4 r + q]: row a 32 + 8 r + 4 (lane / 32) + q of P's part, row
    // b 32 + lane % 32 of Q's
    f32x16 acc[FP][FQ];

    // at most n loads outstanding, no LDS read
    template <uint32_t N>
    __device__ __forceinline__ static void wait() {
        static_assert(N < 64, "six bits");
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0070);
        __builtin_amdgcn_sched_barrier(0);
    }

    // P Q' over `steps` steps; with three segments, P and Q being the first of
    // pairs, P Q' + P Ql' + Pl Q'.  Of all these steps part `part` of `parts`.
    __device__ __forceinline__ void run(const f16 *ph, const f16 *pl, const f16 *qh, const f16 *ql, uint32_t segs,
                                        uint32_t steps, uint64_t ld, uint8_t *lds, uint32_t part = 0,
                                        uint32_t parts = 1) {
        const uint32_t l = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
        for (uint32_t a = 0; a < FP; ++a)
#pragma unroll
            for (uint32_t b = 0; b < FQ; ++b) acc[a][b] = f32x16{0.0f};
        const uint32_t begin = segs * steps * part / parts, total = segs * steps * (part + 1) / parts - begin;
        if (total == 0) return;
        // a load: 16 rows of 64 bytes, a lane's row and (exchanged) piece
        const uint32_t ldb = 2 * (uint32_t)ld;   // (T rows span less than 2^32 bytes)
        const uint32_t mine = (16 * w + (l >> 2)) * ldb + 16 * ((l & 3) ^ (l >> 4));
        // the next load's step of its segment, in bytes
        uint32_t seg = begin / steps, at = (begin - seg * steps) * kRowB;
        __amdgpu_buffer_rsrc_t rp = rsrc(seg == 2 ? pl : ph, ldb), rq = rsrc(seg == 1 ? ql : qh, ldb);
        auto load = [&](bool side, uint32_t it, uint8_t *buf) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(side ? rq : rp,
                                                     (lds_u8 *)(buf + (side ? kSide : 0) + (it * 64 + 16 * w) * kRowB),
                                                     16, mine, at + it * 64 * ldb, 0, 0);
        };
        auto next_step = [&]() {
            at += kRowB;
            if (at == steps * kRowB && ++seg < segs) {
                at = 0;
                rp = rsrc(seg == 1 ? ph : pl, ldb);
                rq = rsrc(seg == 1 ? ql : qh, ldb);
            }
        };
        const uint32_t pr = ((w >> 1) * SP + (l & 31)) * kRowB, qr = ((w & 1) * SQ + (l & 31)) * kRowB + kSide;
        struct Frags {
            f16x8 p[FP], q[FQ];
        };
        auto read = [&](Frags &f, const uint8_t *buf, uint32_t ks) {
            const uint32_t slot = 16 * ((2 * ks + (l >> 5)) ^ ((l >> 2) & 3));
#pragma unroll
            for (uint32_t k = 0; k < FP; ++k) f.p[k] = *reinterpret_cast<const f16x8 *>(buf + pr + k * 32 * kRowB + slot);
#pragma unroll
            for (uint32_t k = 0; k < FQ; ++k) f.q[k] = *reinterpret_cast<const f16x8 *>(buf + qr + k * 32 * kRowB + slot);
            __builtin_amdgcn_sched_barrier(0);
        };
        // FP * FQ products, with the loads of one operand among them
        auto multiply = [&](const Frags &f, bool side, uint8_t *buf) {
#pragma unroll
            for (uint32_t a = 0; a < FP; ++a) {
#pragma unroll
                for (uint32_t b = 0; b < FQ; ++b)
                    acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.p[a], f.q[b], acc[a][b], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
                if (!side)
                    load(false, a, buf);
                else if (a % (FP / FQ) == 0)
                    load(true, a / (FP / FQ), buf);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        auto buffer = [&](uint32_t k) { return lds + (k % NB) * kBuf; };
        Frags x, y;
        // the first NB - 1 steps' loads (past the end the last step's again,
        // so that the counts of what is outstanding hold)
        for (uint32_t k = 0; k < NB - 1; ++k) {
#pragma unroll
            for (uint32_t it = 0; it < FP; ++it) load(false, it, buffer(k));
#pragma unroll
            for (uint32_t it = 0; it < FQ; ++it) load(true, it, buffer(k));
            if (k + 1 < total) next_step();
        }
        wait<(FP + FQ) * (NB - 2)>();
        __syncthreads();
        read(x, buffer(0), 0);
        for (uint32_t k = 0; k < total; ++k) {
            // (each wait is for fragments asked for half a step ago, before the
            // next are: the compiler's own wait, behind them, is for all)
            uint8_t *into = buffer(k + NB - 1);
            wait<(FP + FQ) * (NB - 2)>();
            read(y, buffer(k), 1);
            multiply(x, false, into);
            wait<(FP + FQ) * (NB - 3) + FP>();   // the next step's loads are in LDS
            asm volatile("" ::: "memory");        // (a workgroup fence would wait for every load)
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            read(x, buffer(k + 1), 0);
            multiply(y, true, into);
            if (k + NB < total) next_step();
        }
        wait<0>();
        __syncthreads();   // LDS is free for what follows
    }
    __device__ __forceinline__ static __amdgpu_buffer_rsrc_t rsrc(const f16 *g, uint32_t ldb) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<f16 *>(g), (short)0, (int)(max(TP, TQ) * ldb), 0x00020000);
    }

    // Parts of matrices on their way between memory and a wave's sums, through
    // the wave's own LDS, 16-byte pieces exchanged by row.  ALONG: the rows are
    // Q's (SQ of SP elements; a lane has four neighbours of a row); otherwise
    // P's (SP of SQ).
    template <bool ALONG>
    struct Rows {
        static constexpr uint32_t kLen = ALONG ? SP : SQ, kCount = ALONG ? SQ : SP;
        static constexpr uint32_t kPieces = kLen / 8, kPer = 64 / kPieces;   // of a row; rows a wave moves at once
        __device__ __forceinline__ static uint32_t at(uint32_t row, uint32_t piece) {
            return row * (2 * kLen) + 16 * (piece ^ (row & (kPieces - 1)));
        }
    };
    __device__ __forceinline__ static uint8_t *mine(uint8_t *lds) { return lds + (threadIdx.x >> 6) * kPart; }
    // The lane's number, anew for each pass over the sums: the compiler would
    // otherwise keep every pass's addresses in registers, of which the sums
    // take half, and spill.
    __device__ __forceinline__ static uint32_t lane_anew() {
        uint32_t l = threadIdx.x & 63;
        asm volatile("" : "+v"(l));
        return l;
    }
    template <class G>
    __device__ __forceinline__ void quads(G g) {
        const uint32_t l = lane_anew();
#pragma unroll
        for (uint32_t a = 0; a < FP; ++a)
#pragma unroll
            for (uint32_t b = 0; b < FQ; ++b) {
#pragma unroll
                for (uint32_t r = 0; r < 4; ++r) g(a, b, r, Rows<true>::at(b * 32 + (l & 31), 4 * a + r) + 8 * (l >> 5));
                __builtin_amdgcn_sched_barrier(0);
            }
    }
    // acc <- acc + f * g, g's rows along
    __device__ __forceinline__ void add_along(const f16 *g, uint64_t ld, float f, uint8_t *lds) {
        using R = Rows<true>;
        const uint32_t l = lane_anew();
        uint8_t *own = mine(lds);
#pragma unroll
        for (uint32_t it = 0; it < R::kCount / R::kPer; ++it) {
            const uint32_t v = it * R::kPer + l / R::kPieces, c = (l % R::kPieces) ^ (v & (R::kPieces - 1));
            __builtin_amdgcn_global_load_lds(
                reinterpret_cast<glb_u8 *>(reinterpret_cast<uintptr_t>(g + v * ld + 8 * c)),
                (lds_u8 *)(own + it * 1024), 16, 0, 0);
        }
        wave_wait<true>();
        quads([&](uint32_t a, uint32_t b, uint32_t r, uint32_t at) {
            const f16x4 x = *reinterpret_cast<const f16x4 *>(own + at);
#pragma unroll
            for (uint32_t q = 0; q < 4; ++q) acc[a][b][4 * r + q] += f * (float)x[q];
        });
        wave_wait();
    }
    // the wave's own LDS accesses (and, with LOADS, its loads to LDS) are done
    template <bool LOADS = false>
    __device__ __forceinline__ static void wave_wait() {
        __builtin_amdgcn_s_waitcnt(LOADS ? 0x0070 : 0xC07F);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    // 16-bit numbers v(value) to LDS
    template <bool ALONG, class V>
    __device__ __forceinline__ void put(uint8_t *lds, V v) {
        const uint32_t l = lane_anew();
        uint8_t *own = mine(lds);
        wave_wait();
        if (ALONG) {
            quads([&](uint32_t a, uint32_t b, uint32_t r, uint32_t at) {
                uint16_t h[4];
#pragma unroll
                for (uint32_t q = 0; q < 4; ++q) h[q] = v(acc[a][b][4 * r + q]);
                typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
                *reinterpret_cast<u32x2 *>(own + at) =
                    u32x2{h[0] | ((uint32_t)h[1] << 16), h[2] | ((uint32_t)h[3] << 16)};
            });
        } else {
#pragma unroll
            for (uint32_t a = 0; a < FP; ++a)
#pragma unroll
                for (uint32_t b = 0; b < FQ; ++b) {
#pragma unroll
                    for (uint32_t e = 0; e < 16; ++e) {
                        const uint32_t row = a * 32 + 8 * (e / 4) + 4 * (l >> 5) + e % 4;
                        *reinterpret_cast<uint16_t *>(own + Rows<false>::at(row, 4 * b + (l & 31) / 8) + 2 * (l & 7)) =
                            v(acc[a][b][e]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
        }
        wave_wait();
    }
    // f(row, column, 16 bytes) for every piece of the part in LDS
    template <bool ALONG, class G>
    __device__ __forceinline__ static void pieces(uint8_t *lds, G g) {
        using R = Rows<ALONG>;
        typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
        const uint32_t l = lane_anew();
        uint8_t *own = mine(lds);
#pragma unroll 8
        for (uint32_t it = 0; it < R::kCount / R::kPer; ++it) {
            const uint32_t row = it * R::kPer + l / R::kPieces, c = l % R::kPieces;
            g(row, 8 * c, *reinterpret_cast<const u32x4 *>(own + R::at(row, c)));
        }
    }
    // The sums as they lie, 16 bytes a lane at a time: to memory, and added
    // from there.
    __device__ __forceinline__ void leave(float *to) const {
#pragma unroll
        for (uint32_t a = 0; a < FP; ++a)
#pragma unroll
            for (uint32_t b = 0; b < FQ; ++b)
#pragma unroll
                for (uint32_t r = 0; r < 4; ++r)
                    *reinterpret_cast<f32x4 *>(to + (((a * FQ + b) * 4 + r) * kThreads + threadIdx.x) * 4) =
                        f32x4{acc[a][b][4 * r], acc[a][b][4 * r + 1], acc[a][b][4 * r + 2], acc[a][b][4 * r + 3]};
    }
    // acc = the sums of wave w of `parts` parts, one after another
    __device__ __forceinline__ void join(const float *from, uint32_t parts, uint32_t w) {
        constexpr uint32_t N = FP * FQ * 4;
        const float *mine = from + (w * 64 + (threadIdx.x & 63)) * 4;
        f32x4 sum[N], a[N], b[N];
        auto get = [&](f32x4 (&v)[N], uint32_t s) {
#pragma unroll
            for (uint32_t e = 0; e < N; ++e)
                v[e] = *reinterpret_cast<const f32x4 *>(mine + (uint64_t)s * (TP * TQ) + e * (kThreads * 4));
        };
        get(sum, 0);
        for (uint32_t s = 1; s < parts; s += 2) {
            get(a, s);
            get(b, min(s + 1, parts - 1));
#pragma unroll
            for (uint32_t e = 0; e < N; ++e) sum[e] += a[e];
            if (s + 1 < parts)
#pragma unroll
                for (uint32_t e = 0; e < N; ++e) sum[e] += b[e];
        }
#pragma unroll
        for (uint32_t e = 0; e < N; ++e)
#pragma unroll
            for (uint32_t q = 0; q < 4; ++q) acc[e / 4 / FQ][e / 4 % FQ][e % 4 * 4 + q] = sum[e][q];
    }
    // (the sums are hidden from the compiler between passes, or it keeps one
    // pass's conversions for the next)
    template <bool ALONG, class V>
    __device__ __forceinline__ void store(f16 *g, uint64_t ld, uint8_t *lds, V v) {
#pragma unroll
        for (auto &ra : acc)
#pragma unroll
            for (auto &x : ra) asm volatile("" : "+a"(x));
        put<ALONG>(lds, v);
        pieces<ALONG>(lds, [&](uint32_t row, uint32_t c, auto x) {
            *reinterpret_cast<decltype(x) *>(g + row * ld + c) = x;
        });
    }
};

__device__ __forceinline__ uint16_t high(float x) { return __builtin_bit_cast(uint16_t, (f16)x); }
__device__ __forceinline__ uint16_t low(float x) { return __builtin_bit_cast(uint16_t, (f16)(x - (float)(f16)x)); }

// Workgroups go to the eight XCDs in turn: of every 64 tiles an XCD gets eight
// consecutive ones, which share rows of their operands in its L2.  (A longer
// run each would give one XCD all of a batch's largest products.)
__device__ __forceinline__ uint32_t tile_number() {
    const uint32_t g = blockIdx.x;
    if ((g | 63) >= gridDim.x) return g;
    return (g & ~63u) + (g & 7) * 8 + (g >> 3 & 7);
}

// Tile t of the upper triangle of a square of s x s tiles: groups of four
// rows, a group column by column.
__device__ __forceinline__ void triangle(uint32_t t, uint32_t s, uint32_t &i, uint32_t &j) {
    uint32_t r0 = 0, rows, head;
    while (true) {
        rows = min(4u, s - r0);
        head = rows * (rows + 1) / 2;                  // the columns that the diagonal cuts
        const uint32_t n = head + (s - r0 - rows) * rows;
        if (t < n) break;
        t -= n;
        r0 += rows;
    }
    if (t >= head) {
        i = r0 + (t - head) % rows;
        j = r0 + rows + (t - head) / rows;
        return;
    }
    uint32_t c = 0;
    while (t > c) t -= ++c;
    i = r0 + t;
    j = r0 + c;
}

// A = X X' (SQUARE false) or B = b A + c A A: the tiles on and above the
// diagonal, each written to its mirror image too.
//
// With few tiles and long sums (one matrix of 777 x 2049 has 28 of them) K is
// cut into p.split parts, a workgroup each, which leave their sums in memory
// (PART); the launch that follows (JOIN) adds them, in order, and goes on as
// the whole kernel does, a workgroup for each wave's quarter of a tile.
enum Stage { WHOLE, PART, JOIN };
template <uint32_t TP, uint32_t TQ, uint32_t NB, bool SQUARE, Stage STAGE>
__global__ __launch_bounds__(STAGE == JOIN ? 64 : kThreads, STAGE == JOIN ? 1 : 2) void k_ortho_sym(const OrthoParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t g = STAGE == WHOLE ? tile_number() : blockIdx.x;
    const uint32_t t = STAGE == PART ? g / p.split : STAGE == JOIN ? g / 4 : g;
    const uint32_t k = matrix_of(p, t, [](const OrthoMat &o) { return o.sym0; });
    const OrthoMat &o = p.mat[k];
    const Parts w = parts_of(p.scratch, o);
    uint32_t ti, tj;
    constexpr uint32_t R = TP / TQ;   // tiles to a square one
    const uint32_t square = (t - o.sym0) / R;
    triangle(square, o.mp / TP, ti, tj);
    const bool mirror = ti != tj;
    tj = tj * R + (t - o.sym0) % R;
    const uint64_t ld = SQUARE ? o.mp : o.np, i0 = ti * TP * ld, j0 = tj * TQ * ld;
    Product<TP, TQ, NB> pr;
    if constexpr (STAGE != JOIN) {
        const uint32_t part = STAGE == PART ? g % p.split : 0, parts = STAGE == PART ? p.split : 1;
        if constexpr (SQUARE)
            pr.run(w.ah + i0, w.al + i0, w.ah + j0, w.al + j0, 3, o.mp / kStep, ld, smem, part, parts);
        else
            pr.run(w.xh + i0, w.xl + i0, w.xh + j0, w.xl + j0, o.pairs ? 3 : 1, o.np / kStep, ld, smem, part, parts);
    }
    if constexpr (STAGE == PART) {
        pr.leave(p.partial + (uint64_t)g * (TP * TQ));
        return;
    }
    // this wave's part: rows pi.. of P (of A), pj.. of Q
    const uint32_t wv = STAGE == JOIN ? g % 4 : threadIdx.x >> 6;
    if constexpr (STAGE == JOIN) pr.join(p.partial + (uint64_t)t * p.split * (TP * TQ), p.split, wv);
    const uint64_t pi = ti * TP + (wv >> 1) * (TP / 2), pj = tj * TQ + (wv & 1) * (TQ / 2);
    const uint64_t along = pj * o.mp + pi, across = pi * o.mp + pj;
    const float f = SQUARE ? p.kaa : p.kx;
#pragma unroll
    for (auto &ra : pr.acc)
#pragma unroll
        for (auto &v : ra) v *= f;
    if (SQUARE) {
        pr.add_along(w.ah + along, o.mp, p.ka, smem);
        pr.add_along(w.al + along, o.mp, p.ka, smem);
        pr.template store<true>(w.bh + along, o.mp, smem, high);
        if (mirror) pr.template store<false>(w.bh + across, o.mp, smem, high);
        if (o.pairs) {
            pr.template store<true>(w.bl + along, o.mp, smem, low);
            if (mirror) pr.template store<false>(w.bl + across, o.mp, smem, low);
        }
    } else {
        pr.template store<true>(w.ah + along, o.mp, smem, high);
        pr.template store<true>(w.al + along, o.mp, smem, low);
        if (mirror) {
            pr.template store<false>(w.ah + across, o.mp, smem, high);
            pr.template store<false>(w.al + across, o.mp, smem, low);
        }
    }
}

// X <- a X + B X; the last step writes y in its place.
template <uint32_t TP, uint32_t TQ, uint32_t NB, bool LAST>
__global__ __launch_bounds__(kThreads, 2) void k_ortho_next(const OrthoParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t tile = tile_number();
    const uint32_t k = matrix_of(p, tile, [](const OrthoMat &o) { return o.next0; });
    const OrthoMat &o = p.mat[k];
    const Parts w = parts_of(p.scratch, o);
    const uint32_t t = tile - o.next0, mt = o.mp / TQ;
    const uint64_t i0 = t % mt * TQ, j0 = t / mt * TP;
    Product<TP, TQ, NB> pr;
    pr.run((p.turn ? w.xt1 : w.xt0) + j0 * o.mp, (p.turn ? w.xtl1 : w.xtl0) + j0 * o.mp, w.bh + i0 * o.mp,
           w.bl + i0 * o.mp, o.pairs ? 3 : 1, o.mp / kStep, o.mp, smem);
    const uint32_t wv = threadIdx.x >> 6;
    const uint64_t pj = j0 + (wv >> 1) * (TP / 2), pi = i0 + (wv & 1) * (TQ / 2);
    const uint64_t along = pi * o.np + pj, across = pj * o.mp + pi;
#pragma unroll
    for (auto &ra : pr.acc)
#pragma unroll
        for (auto &v : ra) v *= p.kbx;
    pr.add_along(w.xh + along, o.np, p.a, smem);
    pr.add_along(w.xl + along, o.np, p.a, smem);
    if (!LAST) {
        pr.template store<true>(w.xh + along, o.np, smem, high);
        pr.template store<true>(w.xl + along, o.np, smem, low);
        pr.template store<false>((p.turn ? w.xt0 : w.xt1) + across, o.mp, smem, high);
        if (o.pairs) pr.template store<false>((p.turn ? w.xtl0 : w.xtl1) + across, o.mp, smem, low);
        return;
    }
    const float scale = o.scale;
    auto rounded = [&](float x) { return __builtin_bit_cast(uint16_t, (__bf16)(scale * x)); };
    if (o.tall)
        pr.template put<false>(smem, rounded);
    else
        pr.template put<true>(smem, rounded);
    // rows and columns of y as the caller has it
    const uint32_t rows = o.tall ? o.n : o.m, cols = o.tall ? o.m : o.n;
    const uint64_t r0 = o.tall ? pj : pi, c0 = o.tall ? pi : pj;
    uint16_t *y = static_cast<uint16_t *>(o.y);
    const bool whole = cols % 8 == 0 && (reinterpret_cast<uintptr_t>(y) & 15) == 0;
    auto out = [&](uint32_t row, uint32_t c, auto x) {
        const uint64_t r = r0 + row, q = c0 + c;
        if (r >= rows || q >= cols) return;
        uint16_t *to = y + r * cols + q;
        if (whole) {
            *reinterpret_cast<decltype(x) *>(to) = x;
        } else {
#pragma unroll
            for (uint32_t e = 0; e < 8; ++e)
                if (q + e < cols) to[e] = (uint16_t)(x[e / 2] >> (16 * (e % 2)));
        }
    };
    if (o.tall)
        pr.template pieces<false>(smem, out);
    else
        pr.template pieces<true>(smem, out);
}

// Dynamic LDS beyond 64 KiB must be requested per kernel, once.
std::atomic<bool> g_granted[4];

int launch_tiles(const void *fn, uint32_t grid, size_t lds, const OrthoParams &p, void *stream,
                 std::atomic<bool> &granted, uint32_t threads = kThreads) {
    if (lds > 64 * 1024 && !granted.load()) {
        const hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return (int)e;
        granted.store(true);
    }
    void *args[] = {const_cast<OrthoParams *>(&p)};
    const hipError_t e = hipLaunchKernel(fn, dim3(grid), dim3(threads), args, lds, (hipStream_t)stream);
    return (int)(e != hipSuccess ? e : hipGetLastError());
}

// A symmetric product, whole or (small tiles) in parts.
template <uint32_t TP, uint32_t TQ, uint32_t NB, bool SQUARE>
int run_sym(OrthoParams &p, uint32_t tiles, uint32_t split, void *stream, std::atomic<bool> &granted) {
    constexpr size_t lds = Product<TP, TQ, NB>::kLds;
    if constexpr (TP == kOrthoSmall) {
        static_assert(lds <= 64 * 1024, "granted without asking");
        if (split > 1) {
            p.split = split;
            int e = launch_tiles(reinterpret_cast<const void *>(&k_ortho_sym<TP, TQ, NB, SQUARE, PART>), tiles * split,
                                 lds, p, stream, granted);
            if (e == hipSuccess)
                e = launch_tiles(reinterpret_cast<const void *>(&k_ortho_sym<TP, TQ, NB, SQUARE, JOIN>), tiles * 4,
                                 Product<TP, TQ, NB>::kPart, p, stream, granted, 64);
            return e;
        }
    }
    return launch_tiles(reinterpret_cast<const void *>(&k_ortho_sym<TP, TQ, NB, SQUARE, WHOLE>), tiles, lds, p, stream,
                        granted);
}

template <uint32_t TP, uint32_t TQ, uint32_t NB>
int run_batch(OrthoParams &p, const OrthoBatch &b, uint32_t steps, void *stream) {
    const void *next = reinterpret_cast<const void *>(&k_ortho_next<TP, TQ, NB, false>);
    const void *last = reinterpret_cast<const void *>(&k_ortho_next<TP, TQ, NB, true>);
    constexpr size_t lds = Product<TP, TQ, NB>::kLds;
    for (uint32_t s = 0; s < steps; ++s) {
        p.turn = s & 1;
        const bool end = s + 1 == steps;
        if (end) {
            // the last sums stand for X itself: a tiny factor of the result
            // would be a subnormal number after kOrthoX is taken from it
            p.a = (float)(p.a / kOrthoX);
            p.kbx = (float)(p.kbx / kOrthoX);
        }
        int e = run_sym<TP, TQ, NB, false>(p, b.sym_tiles, b.split_gram, stream, g_granted[0]);
        if (e == hipSuccess) e = run_sym<TP, TQ, NB, true>(p, b.sym_tiles, b.split_square, stream, g_granted[1]);
        if (e == hipSuccess)
            e = end ? launch_tiles(last, b.next_tiles, lds, p, stream, g_granted[3])
                    : launch_tiles(next, b.next_tiles, lds, p, stream, g_granted[2]);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

int launch_ortho(OrthoParams &p, const OrthoBatch &b, uint32_t steps, void *stream) {
    hipLaunchKernelGGL(k_ortho_prep, dim3(b.prep_tiles), dim3(256), 0, (hipStream_t)stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
    return b.tile == kOrthoLarge ? run_batch<256, 128, 3>(p, b, steps, stream)
                                 : run_batch<128, 128, 4>(p, b, steps, stream);
}

}  // namespace lct

// lct_internal.h -- parameter blocks shared by the C ABI (api.cpp) and the
// HIP kernels (kernels.hip).  Not part of the public interface.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/lct.h"

namespace lct {

constexpr uint32_t kStreams = 256;          // streams per block
constexpr uint32_t kChunk = 16;             // positions per stream processed per loop step
constexpr uint32_t kMinBlock = kStreams * kChunk;
constexpr uint32_t kMaxBlock = 65536;
constexpr uint32_t kMaxCapWords = 64;

constexpr uint32_t kMaxUnits = 4;           // units a block is split into
constexpr uint32_t kUnitStreams = kStreams / kMaxUnits;   // streams per unit: one wave's lanes

// Scratch layout (bytes).  The header and the scan's look-back flags are
// cleared by a fill kernel before each encode / SGD launch.  Every unit of the
// main kernel writes its record (spilled bytes, where they sit in the second
// staging area, whether its counts were parked).  Spilled exponent fields are
// parked per stream in the first staging area while a unit runs, copied into
// one contiguous piece per unit at its end, and placed in the overflow region
// by the placing kernel once the scan has given every block its offset.  An
// in-place update parks its counts too, so that no unit overwrites counts
// another unit of the same block has yet to read; the placing kernel puts
// them in place.
constexpr uint64_t kScrTicket2 = 4;   // uint32: next group of the scan kernel
constexpr uint64_t kScrStage = 8;     // uint64: bytes claimed in the first staging area
constexpr uint64_t kScrStage2 = 16;   // uint64: bytes claimed in the second
constexpr uint64_t kScrParked = 24;   // uint32: nonzero when some unit parked its counts
constexpr uint64_t kScrFullUnits = 28;  // uint32: units the update ran on its full-block path
                                        // (read by tests to show which path ran)
constexpr uint64_t kScrFlags = 64;    // uint64[groups + 1]: the scan's look-back flags
constexpr uint32_t kScanGroup = 256;  // blocks per scan workgroup (the flags are sized for
                                      // one group per 256 units, more than it needs)
__host__ __device__ inline uint64_t scr_units(uint64_t nblk) { return kMaxUnits * nblk; }
__host__ __device__ inline uint64_t scr_clear_bytes(uint64_t nblk) {
    return kScrFlags + 8 * ((scr_units(nblk) + kScanGroup - 1) / kScanGroup + 1);
}
__host__ __device__ inline uint64_t align256(uint64_t v) { return (v + 255) & ~uint64_t(255); }
__host__ __device__ inline uint64_t scr_rec_offset(uint64_t nblk) { return align256(scr_clear_bytes(nblk)); }
__host__ __device__ inline uint64_t scr_cnt_offset(uint64_t nblk) {
    return align256(scr_rec_offset(nblk) + 16 * scr_units(nblk));
}
__host__ __device__ inline uint64_t scr_stage_offset(uint64_t nblk) {
    return align256(scr_cnt_offset(nblk) + 2 * kStreams * nblk);
}
__host__ __device__ inline uint64_t scr_stage2_offset(uint64_t nblk, uint64_t ovf_cap) {
    return align256(scr_stage_offset(nblk) + ovf_cap);
}
__host__ __device__ inline uint64_t scr_bytes(uint64_t nblk, uint64_t ovf_cap) {
    return scr_stage2_offset(nblk, ovf_cap) + ovf_cap;
}

// A unit's record: where its spilled bytes sit in the second staging area,
// how many there are, and flags (bit 0: its counts are parked in scratch).
struct UnitRec {
    uint64_t base;
    uint32_t total, flags;
};

// Encoder tables: stream bits of each exponent field and their count.
struct EncTab {
    uint32_t bits[256];
    uint8_t len[256];
};

// Decoder table: 8-bit peek -> field | bits << 8 | escape << 13 | invalid << 14
// (the kernels expand it in LDS).
struct DecTab {
    uint16_t dec[256];
    uint32_t esc_len;
};

// Tensor groups: tensor k's blocks follow tensor k-1's in one set of arrays
// (pay, cnt, obase indexed by the group's block number; sf at the tensor's
// own offset e0, a multiple of 256), one overflow region for all.  The device
// table holds a record per tensor, the tensor of every block and every
// tensor's code tables.
struct GroupEntry {
    uint16_t *dense;      // encode source and decode target (null: none)
    uint64_t n;           // elements
    uint64_t e0;          // first sign-fraction byte in the group's sf array
    uint32_t blk0, nblk;  // first block in the group, blocks
};
// blk_tab[b]: the first tensor whose code tables are byte-identical to those
// of block b's tensor (tensors with one model and one shift share tables, so
// an update that walks many tensors stages them only when they change).
struct GroupRef {
    const GroupEntry *ent;
    const EncTab *enc;
    const DecTab *dec;
    const uint32_t *blk_tensor;
    const uint32_t *blk_tab;
};
// Offsets of the parts of a group's device table.
struct GroupTableLayout {
    uint64_t ent, enc, dec, blk_tensor, blk_tab, bytes;
};
inline GroupTableLayout group_table_layout(uint64_t count, uint64_t nblk) {
    auto up = [](uint64_t v) { return (v + 255) & ~uint64_t(255); };
    GroupTableLayout t;
    t.ent = 0;
    t.enc = up(t.ent + count * sizeof(GroupEntry));
    t.dec = up(t.enc + count * sizeof(EncTab));
    t.blk_tensor = up(t.dec + count * sizeof(DecTab));
    t.blk_tab = up(t.blk_tensor + nblk * sizeof(uint32_t));
    t.bytes = up(t.blk_tab + nblk * sizeof(uint32_t));
    return t;
}

struct EncodeParams {
    const uint16_t *x;
    uint64_t n;
    uint32_t block_elems, cap_words, nblk, pad0;
    uint8_t *sf;
    uint32_t *pay;
    uint16_t *cnt;
    uint64_t *obase;
    uint8_t *ovf;
    uint64_t ovf_cap;
    uint32_t *status;
    uint8_t *scratch;
    GroupRef grp;         // used by the group kernels only
    EncTab enc;
};

struct DecodeParams {
    const uint8_t *sf;
    const uint32_t *pay;
    const uint16_t *cnt;
    const uint64_t *obase;
    const uint8_t *ovf;
    uint64_t ovf_cap;
    uint16_t *y;
    uint64_t n;
    uint32_t block_elems, cap_words, nblk, pad0;
    GroupRef grp;         // used by the group kernels only
    DecTab dec;
};

struct SgdParams {
    // inputs: W (codebook cw) and M (codebook cm)
    const uint8_t *w_sf;
    const uint32_t *w_pay;
    const uint16_t *w_cnt;
    const uint64_t *w_obase;
    const uint8_t *w_ovf;
    uint64_t w_ovf_cap;
    const uint8_t *m_sf;
    const uint32_t *m_pay;
    const uint16_t *m_cnt;
    const uint64_t *m_obase;
    const uint8_t *m_ovf;
    uint64_t m_ovf_cap;
    // output W'
    uint8_t *o_sf;
    uint32_t *o_pay;
    uint16_t *o_cnt;
    uint64_t *o_obase;
    uint8_t *o_ovf;
    uint64_t ovf_cap;
    uint32_t *status;
    uint8_t *scratch;
    uint64_t n;
    uint32_t block_elems, cap_words, nblk;
    float mul;           // the product's factor: -eta, for W - eta*M
    const float *coef;   // a device factor of mul (null: 1)
    uint32_t park_cnt;   // the result's counts overwrite W's: park them in scratch
    uint32_t all;        // the general kernel does every block
    GroupRef gw, gm;     // used by the group kernels only (W's codes for W and W';
                         // M's for M)
    EncTab wenc;
    DecTab wdec;
    DecTab mdec;
};

// The fused momentum step: W and M decoded, g dense; M' = rne(mu*M + g) and
// W' = rne(W - eta*M') (M' as rounded), both re-encoded in one pass.  Encode
// tables travel packed (stream bits | bit count << 24) to keep the arguments
// small.
struct MomParams {
    const uint8_t *w_sf;
    const uint32_t *w_pay;
    const uint16_t *w_cnt;
    const uint64_t *w_obase;
    const uint8_t *w_ovf;
    uint64_t w_ovf_cap;
    const uint8_t *m_sf;
    const uint32_t *m_pay;
    const uint16_t *m_cnt;
    const uint64_t *m_obase;
    const uint8_t *m_ovf;
    uint64_t m_ovf_cap;
    const uint16_t *g;
    // outputs W' (ow_*) and M' (om_*), each with its own overflow side
    uint8_t *ow_sf;
    uint32_t *ow_pay;
    uint16_t *ow_cnt;
    uint64_t *ow_obase;
    uint8_t *ow_ovf;
    uint64_t ow_ovf_cap;
    uint32_t *ow_status;
    uint8_t *ow_scratch;
    uint8_t *om_sf;
    uint32_t *om_pay;
    uint16_t *om_cnt;
    uint64_t *om_obase;
    uint8_t *om_ovf;
    uint64_t om_ovf_cap;
    uint32_t *om_status;
    uint8_t *om_scratch;
    uint64_t n;
    uint32_t block_elems, cap_words, nblk;
    float mu, neg_eta;
    uint32_t park_w, park_m;   // an output's counts overwrite its input's: park them
    uint32_t all;              // the general kernel does every block
    const float *coef;         // clip kernels only: a device factor of g
    GroupRef gw, gm, gg;       // group kernels: W's and M's codes, the gradients' buffers
    uint32_t wenc[256], menc[256];   // packed: bits | len << 24 (W' and M')
    DecTab wdec, mdec;
};

// The mix of a compressed tensor with a dense one: y' = rne(a * y + bx), bx =
// (b * coef) * x, y' encoded; d (null: not wanted) gets y', or ahead, rne(a *
// y' + bx).
struct MixParams {
    const uint8_t *sf;
    const uint32_t *pay;
    const uint16_t *cnt;
    const uint64_t *obase;
    const uint8_t *ovf;
    uint64_t ovf_cap;
    const uint16_t *x;
    uint16_t *d;
    uint8_t *o_sf;
    uint32_t *o_pay;
    uint16_t *o_cnt;
    uint64_t *o_obase;
    uint8_t *o_ovf;
    uint64_t o_ovf_cap;
    uint32_t *status;
    uint8_t *scratch;
    uint64_t n;
    uint32_t block_elems, cap_words, nblk;
    float a, b;
    uint32_t park_cnt;     // the result's counts overwrite the input's: park them in scratch
    uint32_t dense, ahead;
    const float *coef;     // null: 1
    GroupRef g, gx, gd;    // group kernels: y's codes, x's and d's buffers
    EncTab enc;
    DecTab dec;
};

// Rows of a compressed tensor taken as a table of `cols` columns.
struct RowsParams {
    const uint8_t *sf;
    const uint32_t *pay;
    const uint16_t *cnt;
    const uint64_t *obase;
    const uint8_t *ovf;
    uint64_t ovf_cap;
    uint64_t n, rows, cols, count;
    uint32_t block_elems, cap_words, wide, type;   // wide: 64-bit indices; type: the result's
    const void *index;
    const uint32_t *key, *token;   // many tokens: their rows, sorted, and the tokens (null: in order, by index)
    void *y;
    uint32_t run, piece;   // sorted tokens of a workgroup; bytes of LDS for a row's exponents (a multiple of 16)
    float scale;
    DecTab dec;
};
constexpr uint32_t kRowsRun = 16;          // sorted tokens that a workgroup takes at most,
constexpr uint32_t kRowsRoom = 12288;      // and bytes of LDS for their exponents
// Tokens are sorted from so many on, if there are two to a block of the table.
// In us, in order and (sorted, with the sort): 50,304 x 768 (590 blocks), 2048
// tokens 29 (36), 4096 45 (44), 16,384 139 (84); 151,936 x 2560 (5936 blocks),
// 4096 tokens 52 (56), 8192 91 (86), 100 (118) where none is frequent, 16,384
// 164 (134).
constexpr uint64_t kRowsSortFrom = 4096;

// The gradient of a table's rows (rows.hip).  Tokens are sorted by row in
// passes of at most kSortBits bits over chunks of kSortChunk tokens, then
// summed in tiles.
constexpr uint32_t kSortBits = 9, kSortDigits = 1u << kSortBits;
constexpr uint32_t kSortThreads = 256, kSortChunk = 1024;
// Up to so many tokens one workgroup sorts them.  A gradient's us by that kernel
// and (by a launch or more a pass): of 4001 x 331, 2048 tokens 27 (34), 4096 39
// (46), with a kernel for 8192 of them 47 (48); of 300,000 x 40, 4096 25 (35).
// One for 8192 takes 4 to 7 us more for the fewer, one for 1024 2 to 3 us less.
constexpr uint32_t kSortOne = 4096;
// Chunks whose counts the placing kernel adds up itself; (by a launch of their
// own): 50,304 x 40, 17 chunks 59 us (62), 64 118 (121), 98 134 (137), 256 229 (231).
constexpr uint32_t kSortFew = 64;
// (so that every launch's threads stay below 2^32 in a dimension)
constexpr uint64_t kMaxTokens = 1ull << 30, kMaxRows = 1ull << 29, kMaxCols = 1ull << 24;
// Tokens of a tile: four where there are few (each row that ends in a tile waits
// for what G holds), more where there are many (fewer sums to join).  A gradient's
// us with tiles of 4, 8, 16 and 32: 777 tokens added to 4001 x 331 21, 23, 31, 46;
// 4096 to 32,000 x 1024 31, 29, 32, 38 (25, 27, 32, 42 where none is frequent);
// 8192 53, 45, 47, 57 (39, 40, 45, 57); 16,384 to 50,304 x 768 109, 77, 69, 80;
// 65,536 371, 229, 156, 135; 16,384 of 151,936 x 2560, written, 259, 237, 225, 233.
constexpr uint32_t kRowTileFew = 4, kRowTile = 16, kRowTileMax = 256;
constexpr uint64_t kRowFew = 4096;                     // tokens up to which they are few
constexpr uint64_t kRowTiles = 4096;
constexpr uint32_t kClearRows = 16;                    // rows that a clearing wave looks at
inline uint32_t row_tile(uint64_t count) {
    if (count <= kRowFew) return kRowTileFew;
    uint64_t t = kRowTile;
    while (t < kRowTileMax && count > kRowTiles * t) t *= 2;
    return (uint32_t)t;
}
// The most tiles that up to `count` tokens make: memory for many tokens does for
// fewer, whose tiles are shorter.
inline uint64_t row_tiles_most(uint64_t count) {
    uint64_t most = (count + row_tile(count) - 1) / row_tile(count);
    if (count > kRowFew) most = std::max<uint64_t>(most, kRowFew / kRowTileFew);
    if (count > kRowTiles * kRowTile) most = std::max(most, kRowTiles);
    return most;
}
struct SortParams {
    const void *index;          // the first pass reads indices, the others keys
    const uint32_t *from, *from_token;
    uint32_t *to, *to_token, *hist;
    uint32_t count, rows, wide, bits, shift, chunks, passes;
};
struct RowGradParams {
    const uint32_t *key, *token;   // sorted
    const void *dy;
    void *g;
    float *part;                   // [tiles][2][cols]
    uint64_t cols;
    uint32_t count, rows, tile, tiles, add;
    float scale;
};
// The gradient's working memory.
struct RowScratch {
    uint64_t key0, key1, tok0, tok1, hist, part, bytes;
};
inline RowScratch row_scratch(uint64_t count, uint64_t cols) {
    RowScratch s;
    const uint64_t list = align256(4 * count), chunks = (count + kSortChunk - 1) / kSortChunk;
    s.key0 = 0;
    s.key1 = list;
    s.tok0 = 2 * list;
    s.tok1 = 3 * list;
    s.hist = 4 * list;
    s.part = s.hist + align256(4ull * kSortDigits * (chunks + 1));
    s.bytes = s.part + align256(8 * row_tiles_most(count) * cols);
    return s;
}

// Shift sample of a compressed tensor: the values at floor(i * n / m), i < m.
struct SampleParams {
    const uint8_t *sf;
    const uint32_t *pay;
    const uint16_t *cnt;
    const uint64_t *obase;
    const uint8_t *ovf;
    uint64_t ovf_cap;
    uint64_t n;
    uint32_t block_elems, cap_words, m, pad0;
    DecTab dec;
};

// Fit of a codebook on the device: the shift of x's sample over the base
// code, the shifted code's tables, and x's record, written as a one-tensor
// group table.
struct FitParams {
    uint16_t *x;
    uint64_t n;
    uint32_t m, nblk;        // sample size min(n, 4096); x's blocks
    uint32_t esc_len, pad0;
    uint8_t base[256];       // base code lengths (0: escaped)
    GroupEntry *ent;
    EncTab *enc;
    DecTab *dec;
    uint32_t *blk_tensor;
    uint32_t *blk_tab;
    int32_t *shift_out;      // may be null
};

// Norms: the scale of the values and the norm to clip to.
struct NormArgs {
    double max_norm, scale;
};

// Lists of dense tensors: cut into chunks of 2^shift elements, numbered
// through a launch's tensors (chunk0[k]: tensor k's first; chunk0[count]: all
// of them).  A size travels with its element types above kListTypeShift.
constexpr uint32_t kNormThreads = 256;
constexpr uint32_t kListChunkMax = 14, kListChunkMin = 11;   // shifts
constexpr uint32_t kListSpread = 512;     // chunks that a cut should make
constexpr uint32_t kListMax = 192;        // tensors per launch of the norm
constexpr uint32_t kListFew = 16;         // short lists take kernels with shorter arguments
constexpr uint32_t kClipMax = 128;        // and of the clip
constexpr uint32_t kListGrid = 2048;      // workgroups per launch at most: eight per CU
constexpr uint32_t kListTypeShift = 48;
constexpr uint64_t kListElems = (1ull << kListTypeShift) - 1;
constexpr uint64_t kListMaxElems = 1ull << 44;   // of a whole list: chunk numbers stay within 32 bits
constexpr uint32_t kListMaxCount = 1u << 24;     // tensors of a list
// Short lists in one launch: a workgroup of kOneThreads does every chunk of
// 2^kOneShift elements, a wave each.
constexpr uint32_t kOneThreads = 1024;
constexpr uint32_t kOneShift = 11;
constexpr uint32_t kOneMax = 64;          // chunks
template <uint32_t N>
struct ListArgs {
    uint32_t count, chunks, shift;
    const void *x[N];
    uint64_t n[N];
    uint32_t chunk0[N + 1];
};
template <uint32_t N>
struct ListNormParams {
    double *run;          // a value per workgroup
    double *piece;        // a value per workgroup and tensor that meet (null: not wanted)
    ListArgs<N> list;
};
template <uint32_t N>
struct ListOneParams {
    float *each;          // null: not wanted
    lct_norm_t *out;
    NormArgs args;
    ListArgs<N> list;
};
// What follows a launch of the norm: the tensors' own norms (each) and, after
// the last, the result of `runs` workgroups' values (out).
struct ListFinishParams {
    const double *piece, *run;
    float *each;          // null: not wanted
    lct_norm_t *out;      // null: not yet
    uint64_t runs;
    NormArgs args;
    uint32_t count, chunks, G;   // G: the norm launch's workgroups
    bool squares;
    uint32_t chunk0[kListMax + 1];
};
// Part values (every `stride`-th double) joined into the result.
struct NormJoinParams {
    const double *part;
    uint64_t count, stride;
    lct_norm_t *out;
    NormArgs args;
    bool squares;
};
// What follows the norm of codes (a value per block in part).
struct CodeFinishParams {
    const double *part;
    uint64_t nblk;
    double *fold;         // many blocks: kFoldGrid values first (null: the result)
    lct_norm_t *out;
    const GroupEntry *ent;
    float *each;          // null: not wanted
    NormArgs args;
    uint32_t count;       // a group's tensors
    bool squares;
};
template <uint32_t N>
struct ListClipParams {
    const float *coef;
    ListArgs<N> list;     // types: x's | y's << 2
    void *y[N];
};
// Norm of a compressed tensor (or a group's): a value per block.
struct CodeNormParams {
    const uint8_t *sf;
    const uint32_t *pay;
    const uint16_t *cnt;
    const uint64_t *obase;
    const uint8_t *ovf;
    uint64_t ovf_cap;
    uint64_t n;
    uint32_t block_elems, cap_words, nblk, pad0;
    double *part;
    GroupRef grp;         // used by the group kernels only
    DecTab dec;
};
// Scratch of the norms, in doubles: the blocks' (or launches' workgroups')
// values, then the values they are folded into when there are many.
constexpr uint64_t kFoldFrom = 4096;      // more part values than this are folded first
constexpr uint32_t kFoldGrid = 256;
inline uint64_t list_launches(uint64_t count) { return (count + kListMax - 1) / kListMax; }
inline uint64_t norm_scratch_bytes(uint64_t count, uint64_t nblk) {
    const uint64_t runs = list_launches(count) * kListGrid;
    const uint64_t list = runs + list_launches(count) * (kListGrid + kListMax);
    return align256(8 * ((list > nblk ? list : nblk) + kFoldGrid));
}

// Orthogonalising many matrices (ortho.hip): a launch's matrices travel as
// kernel arguments.  A matrix has m rows and n >= m columns (`tall`: the
// caller's is the transpose), padded to mp and np, whole tiles; its working
// memory starts at byte `off`: X as a pair, two copies of its transpose, A as a
// pair, B, all FP16; for short matrices (m at most kOrthoPairs) then the low
// parts of B and of X' too.  The error that this takes away stands in ortho.hip;
// what it takes, in us, with and (without): 64 x 64 140 (114), 200 x 300 226
// (169), 24 of 256 x 2048 565 (370); it would take 24 of 512 x 2048 1292 (671).
constexpr uint32_t kOrthoPairs = 256;
constexpr uint32_t kOrthoMax = 32;        // matrices per launch
constexpr uint32_t kOrthoSmall = 128, kOrthoLarge = 256;
// Tiles of 128 x 128, or (kOrthoLarge) of 256 x 128, whose operands take three
// quarters of the traffic but which leave more of the device idle in the last
// round.  In us, small and (large): 160 large tiles' worth (2560 x 4096) 1179
// (1576), 380 (2560 x 9728) 2025 (2378), 432 (24 matrices) 1204 (1299), 1540
// (seven matrices) 8457 (7604).
constexpr uint32_t kOrthoLargeFrom = 800;
// Large tiles pad more: they are taken if the padded work (m m n, of a batch)
// grows by a fifth at most.  In us, small and (large): 24 of 1000 x 2000, as
// much work in either, 2402 (2167); 2 of 4100 x 8200, 1.08 times as much, 9794
// (9333); 8 of 2100 x 4200, 1.16 times, 5993 (5917); 20 of 1100 x 2200, 1.23
// times, 2739 (3258); 32 of 600 x 2000, 1.44 times, 1409 (1789); 32 of 64 x
// 6400, 4 times, 805 (2963).
constexpr uint32_t kOrthoLargePad = 5;
// Few small tiles (kOrthoSplitTo parts of them at most, half of what the device
// holds at once) with long sums (kOrthoLong steps of 32 and more): K is cut into
// up to kOrthoSplitMax parts of at least kOrthoPart steps.  In us, cut and
// (whole): 128 x 4096 239 (527), 256 x 16,384 464 (1812), 400 x 2000 244 (288),
// 777 x 2049 317 (366), 1536 x 1536 406 (520), 2048 x 2048 (whole by the rule) 617,
// 4 of 777 x 2049 464 (490).  With other limits, for 777 x 2049, 1536 x 1536 and 9
// of 300 x 2000 (317, 406 and 301): 128 parts 291, 520 and 313, 512 parts 317, 440
// and 321; sums of 24 steps 317, 407 and 318, of 96 366, 414 and 332; parts of 4
// steps 317, 407 and 300, of 16 294, 406 and 301; at most 4 parts 291, 407 and 299
// (256 x 16,384 then 656), 16 308, 406 and 300.
constexpr uint32_t kOrthoSplitTo = 256, kOrthoSplitMax = 8, kOrthoPart = 8, kOrthoLong = 48;
// Elements that a batch of matrices gathers, with sides rounded up to small
// tiles: 2048 tiles of 256 x 256, eight per CU.
constexpr uint64_t kOrthoBatch = 1ull << 27;
// FP16 numbers stand for X, A and B times these powers of two.  Singular
// values stay below kOrthoBound (checked for the coefficients), so X's
// elements do, A's stay below its square and B's below kOrthoBoundB.
constexpr double kOrthoX = 32768.0, kOrthoA = 16384.0, kOrthoB = 8192.0;
constexpr double kOrthoBound = 1.9, kOrthoBoundB = 7.8;
constexpr uint64_t kOrthoMaxElems = 1ull << 32;   // of one matrix: its root mean square stays in FP16's range
constexpr uint32_t kOrthoMaxSide = 1u << 22;      // a tile's rows span less than 2^32 bytes
struct OrthoMat {
    const void *x;
    void *y;
    uint64_t off;
    uint32_t m, n, mp, np;
    uint32_t type, tall, pairs, index;   // pairs: every operand is one; index: in the whole list (its norm's place)
    float scale;
    uint32_t prep0, sym0, next0;  // first tile of each kind of launch
};
struct OrthoParams {
    uint8_t *scratch;
    const float *norm;
    double xscale;
    float a, ka, kaa, kx, kbx;    // factors of a X, A, A A, X X' and B X for numbers as held
    float *partial;               // sums of parts of K, where it is cut
    uint32_t count, turn, split;  // turn: which copy of X' is read; split: parts of K
    OrthoMat mat[kOrthoMax];
};
struct OrthoBatch {
    uint32_t tile, prep_tiles, sym_tiles, next_tiles;
    uint32_t split_gram, split_square;   // parts that the symmetric products' K is cut into
};

// The allocation-free update's static working memory (per device).
constexpr uint64_t kNoAllocScratch = LCT_NOALLOC_SCRATCH_BYTES;
constexpr int kMaxDevices = 64;
// Device address of the current device's static working memory, looked up
// once per device (hipGetSymbolAddress).  Returns a hipError_t.
int noalloc_scratch(uint8_t **out);

// The overflow side of a call's outputs (the momentum step has two).
struct OutSide {
    uint8_t *scratch;
    uint64_t *obase;
    uint8_t *ovf;
    uint64_t ovf_cap;
    uint32_t *status;
    uint16_t *cnt;
};
struct OutSides {
    OutSide side[2];
    uint32_t count;
    uint64_t nblk;
};

// Host-side launchers (kernels.hip).  Each returns the hipError_t of the launch.
int launch_clear(const OutSides &o, void *stream);
int launch_scan(const OutSides &o, void *stream);
int launch_encode(const EncodeParams &p, void *stream, bool group = false);
int launch_decode(const DecodeParams &p, void *stream, bool group = false);
int launch_sgd(const SgdParams &p, void *stream, bool group = false);
int launch_mom(const MomParams &p, void *stream, bool group = false);
int launch_mix(const MixParams &p, void *stream, bool group = false);
int launch_rows(const RowsParams &p, void *stream);
// A table's gradient (rows.hip).
int launch_row_sort(SortParams p, const RowScratch &s, uint8_t *scratch, const uint32_t **key, const uint32_t **token,
                    void *stream);
int launch_row_grad(const RowGradParams &p, uint32_t from, uint32_t to, void *stream);
int launch_gather(const uint16_t *x, uint64_t n, uint32_t m, void *stream, uint16_t *host_out);
// The shift sample of a compressed tensor, copied to host_out; synchronises.
int launch_sample(const SampleParams &p, void *stream, uint16_t *host_out);
// The device fit (enqueues only).
int launch_fit(const FitParams &p, void *stream);
// Norms and clipping (norms.hip; the codes' norm in kernels.hip).
template <uint32_t N>
int launch_list_norm(const ListNormParams<N> &p, uint32_t grid, bool squares, void *stream);
template <uint32_t N>
int launch_list_one(const ListOneParams<N> &p, bool squares, void *stream);
int launch_list_finish(const ListFinishParams &p, void *stream);
int launch_norm_join(const NormJoinParams &p, void *stream);
int launch_code_finish(const CodeFinishParams &p, void *stream);
template <uint32_t N>
int launch_list_clip(const ListClipParams<N> &p, void *stream);
int launch_code_norm(const CodeNormParams &p, bool group, bool squares, void *stream);
// Orthogonalising a batch of matrices (ortho.hip); changes p from step to step.
int launch_ortho(OrthoParams &p, const OrthoBatch &b, uint32_t steps, void *stream);

// Host codebook construction (codebook.cpp).
// The model's probability of each exponent field (its range of |x|).
void model_pmf(const lct_model &model, double p[256]);
lct_status build_codebook(const lct_model &model, const uint16_t *sample, uint32_t m,
                          lct_codebook *out);
lct_status codebook_from_lengths(const uint8_t len_base[256], uint8_t esc_len, int32_t shift,
                                 lct_codebook *out);
// cb's base code with the shift that minimises the sample's coded bits.
lct_status reshift_codebook(const lct_codebook &cb, const uint16_t *sample, uint32_t m,
                            lct_codebook *out);
// The ranges the kernels rely on hold in cb's lookup tables: an escape code
// of 1..8 bits, every field costing 1..16 bits with no bits past its length,
// every decode entry's length at most 16 (a codebook not made by the
// library, e.g. one left zeroed, fails).
bool tables_ok(const lct_codebook &cb);
void fill_enc(const lct_codebook &cb, EncTab *t);
void fill_enc_packed(const lct_codebook &cb, uint32_t t[256]);
void fill_dec(const lct_codebook &cb, DecTab *t);

}  // namespace lct

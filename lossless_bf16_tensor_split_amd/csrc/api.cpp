// api.cpp -- the extern "C" entry points declared in include/lct.h:
// argument checks, size accounting and kernel launches.
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <cmath>
#include <map>
#include <mutex>
#include <new>
#include <vector>

#include "lct_internal.h"

namespace {

using namespace lct;

thread_local char g_hip_msg[256] = "";

lct_status hip_fail(int err, const char *what) {
    snprintf(g_hip_msg, sizeof g_hip_msg, "%s: %s", what, hipGetErrorString((hipError_t)err));
    return LCT_EHIP;
}

// gfx950 check, cached per device.
lct_status check_arch() {
    static std::mutex mu;
    static int known[64] = {0};   // 0 unknown, 1 ok, -1 other arch
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
    if (dev < 0 || dev >= 64) return LCT_EARCH;
    std::lock_guard<std::mutex> lock(mu);
    if (known[dev] == 0) {
        hipDeviceProp_t prop;
        e = hipGetDeviceProperties(&prop, dev);
        if (e != hipSuccess) return hip_fail(e, "hipGetDeviceProperties");
        known[dev] = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : -1;
    }
    return known[dev] == 1 ? LCT_OK : LCT_EARCH;
}

bool layout_ok(const lct_layout &l) {
    return l.block_elems >= kMinBlock && l.block_elems <= kMaxBlock &&
           l.block_elems % kMinBlock == 0 && l.cap_words >= 1 && l.cap_words <= kMaxCapWords;
}

uint64_t nblocks(uint64_t n, const lct_layout &l) { return (n + l.block_elems - 1) / l.block_elems; }

// The largest sizes a call accepts, so that no size or address computed from
// them wraps: n elements (blocks are indexed by 32 bits) and ovf_cap bytes.
constexpr uint64_t kMaxElems = 1ull << 48;
constexpr uint64_t kMaxOvfCap = 1ull << 56;
bool sizes_ok(uint64_t n, const lct_layout &l, uint64_t ovf_cap) {
    return n <= kMaxElems && nblocks(n, l) <= 0xFFFFFFFFull && ovf_cap <= kMaxOvfCap;
}

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

struct Range {
    uintptr_t lo, hi;   // [lo, hi)
};
Range rng(const void *p, uint64_t bytes) { return {(uintptr_t)p, (uintptr_t)p + bytes}; }
bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

struct Parts {
    Range sf, pay, cnt, obase, ovf, status, scratch;
};

// The ranges of a tensor's buffers; nb overrides the block count (a group's
// storage has more blocks than its n implies).
Parts parts(const lct_tensor &t, uint64_t nb = ~0ull) {
    if (nb == ~0ull) nb = nblocks(t.n, t.layout);
    Parts p;
    p.sf = rng(t.sf, t.n);
    p.pay = rng(t.pay, nb * t.layout.cap_words * kStreams * 4);
    p.cnt = rng(t.cnt, nb * kStreams * 2);
    p.obase = rng(t.obase, (nb + 1) * 8);
    p.ovf = rng(t.ovf, t.ovf_cap);
    p.status = rng(t.status, 4);
    p.scratch = rng(t.scratch, scr_bytes(nb, t.ovf_cap));
    return p;
}

// Pointers a call reads or writes must be non-null and aligned.
lct_status check_tensor(const lct_tensor *t, bool writes, uint64_t nb = ~0ull) {
    if (!t || !layout_ok(t->layout) || !sizes_ok(t->n, t->layout, t->ovf_cap)) return LCT_EINVAL;
    if (nb != ~0ull && nb > 0xFFFFFFFFull) return LCT_EINVAL;
    if (!t->sf || !t->pay || !t->cnt || !t->obase) return LCT_EINVAL;
    if (t->ovf_cap && !t->ovf) return LCT_EINVAL;
    if (!aligned(t->sf, 16) || !aligned(t->pay, 16) || !aligned(t->cnt, 4) || !aligned(t->obase, 8))
        return LCT_EALIGN;
    if (writes) {
        if (!t->status || !t->scratch) return LCT_EINVAL;
        if (!aligned(t->status, 4) || !aligned(t->scratch, 256)) return LCT_EALIGN;
        // the output's own parts must be disjoint
        const Parts p = parts(*t, nb);
        const Range all[] = {p.sf, p.pay, p.cnt, p.obase, p.ovf, p.status, p.scratch};
        for (int i = 0; i < 7; ++i)
            for (int j = i + 1; j < 7; ++j)
                if (overlap(all[i], all[j])) return LCT_EALIAS;
    }
    return LCT_OK;
}

bool overlaps_any(Range r, const Parts &p, bool with_writable = true) {
    const Range all[] = {p.sf, p.pay, p.cnt, p.obase, p.ovf};
    for (const Range &a : all)
        if (overlap(r, a)) return true;
    if (with_writable && (overlap(r, p.status) || overlap(r, p.scratch))) return true;
    return false;
}

// A clipped step's coefficient (null: not a clipped step): aligned, and not
// in what the step writes.
lct_status check_coef(const float *coef, const Parts &out) {
    if (!coef) return LCT_OK;
    if (!aligned(coef, 4)) return LCT_EALIGN;
    return overlaps_any(rng(coef, 4), out) ? LCT_EALIAS : LCT_OK;
}

std::mutex g_sample_mu;

// ---- groups

uint64_t shape_hash(uint32_t count, const uint64_t *n, const lct_layout &l) {
    uint64_t h = 1469598103934665603ull;   // FNV-1a over the layout and sizes
    auto mix = [&](uint64_t v) {
        for (int i = 0; i < 8; ++i) {
            h ^= (v >> (8 * i)) & 0xFF;
            h *= 1099511628211ull;
        }
    };
    mix(l.block_elems);
    mix(l.cap_words);
    mix(count);
    for (uint32_t k = 0; k < count; ++k) mix(n[k]);
    return h;
}

uint64_t round256(uint64_t v) { return (v + 255) & ~uint64_t(255); }

// The group's block count and sf bytes; false on overflow of the 32-bit block index.
bool group_extent(uint32_t count, const uint64_t *n, const lct_layout &l, uint64_t *nblk, uint64_t *sf) {
    uint64_t nb = 0, s = 0;
    for (uint32_t k = 0; k < count; ++k) {
        if (n[k] > kMaxElems) return false;
        nb += nblocks(n[k], l);
        if (nb > 0xFFFFFFFFull) return false;   // checked as it grows: it cannot wrap
        s += round256(n[k]);
    }
    *nblk = nb;
    *sf = s;
    return true;
}

GroupRef group_ref(const lct_group &g) {
    const GroupTableLayout t = group_table_layout(g.count, g.nblk);
    const uint8_t *base = static_cast<const uint8_t *>(g.d_table);
    return {reinterpret_cast<const GroupEntry *>(base + t.ent), reinterpret_cast<const EncTab *>(base + t.enc),
            reinterpret_cast<const DecTab *>(base + t.dec), reinterpret_cast<const uint32_t *>(base + t.blk_tensor),
            reinterpret_cast<const uint32_t *>(base + t.blk_tab)};
}

// A bound group and storage sized for it.
lct_status check_group(const lct_group *g, const lct_tensor *all, bool writes) {
    if (!g || !all || !g->d_table || !g->n || g->count == 0 || !layout_ok(g->layout)) return LCT_EINVAL;
    if (all->n != g->sf_bytes || all->layout.block_elems != g->layout.block_elems ||
        all->layout.cap_words != g->layout.cap_words)
        return LCT_EINVAL;
    uint64_t nb = 0, sf = 0;
    if (!group_extent(g->count, g->n, g->layout, &nb, &sf) || nb != g->nblk || sf != g->sf_bytes ||
        shape_hash(g->count, g->n, g->layout) != g->shape_hash)
        return LCT_EINVAL;
    return check_tensor(all, writes, g->nblk);
}

// Every dense buffer of the group, disjoint from the storage's parts.
lct_status check_group_dense(const lct_group &g, const Parts &p) {
    if (!g.d_dense) return LCT_EINVAL;
    for (uint32_t k = 0; k < g.count; ++k) {
        if (g.n[k] == 0) continue;
        if (!g.d_dense[k]) return LCT_EINVAL;
        if (!aligned(g.d_dense[k], 16)) return LCT_EALIGN;
        if (overlaps_any(rng(g.d_dense[k], g.n[k] * 2), p)) return LCT_EALIAS;
    }
    return LCT_OK;
}

// The buffers of an update: W and M (both decoded) and the result.
void sgd_params(SgdParams &p, const lct_tensor &w_in, const lct_tensor &m, const lct_tensor &w_out,
                uint64_t nb, float mul) {
    p.w_sf = w_in.sf;
    p.w_pay = w_in.pay;
    p.w_cnt = w_in.cnt;
    p.w_obase = w_in.obase;
    p.w_ovf = w_in.ovf;
    p.w_ovf_cap = w_in.ovf_cap;
    p.m_sf = m.sf;
    p.m_pay = m.pay;
    p.m_cnt = m.cnt;
    p.m_obase = m.obase;
    p.m_ovf = m.ovf;
    p.m_ovf_cap = m.ovf_cap;
    p.o_sf = w_out.sf;
    p.o_pay = w_out.pay;
    p.o_cnt = w_out.cnt;
    p.o_obase = w_out.obase;
    p.o_ovf = w_out.ovf;
    p.ovf_cap = w_out.ovf_cap;
    p.status = w_out.status;
    p.scratch = (uint8_t *)w_out.scratch;
    p.n = w_in.n;
    p.block_elems = w_in.layout.block_elems;
    p.cap_words = w_in.layout.cap_words;
    p.nblk = (uint32_t)nb;
    p.mul = mul;
    p.park_cnt = p.o_cnt == p.w_cnt;
}

// Clear, update, scan.
lct_status sgd_launch(const SgdParams &p, uint64_t nb, bool group, void *stream) {
    const OutSides o{{{p.scratch, p.o_obase, p.o_ovf, p.ovf_cap, p.status, p.o_cnt}}, 1, nb};
    int e = launch_clear(o, stream);
    if (e != hipSuccess) return hip_fail(e, "clear launch");
    e = launch_sgd(p, stream, group);
    if (e != hipSuccess) return hip_fail(e, "sgd launch");
    e = launch_scan(o, stream);
    if (e != hipSuccess) return hip_fail(e, "scan launch");
    return LCT_OK;
}

// The buffers of a fused momentum step.
void mom_params(MomParams &p, const lct_tensor &w_in, const lct_tensor &m_in, const uint16_t *g,
                const lct_tensor &w_out, const lct_tensor &m_out, uint64_t nb, float mu, float eta) {
    p.w_sf = w_in.sf;
    p.w_pay = w_in.pay;
    p.w_cnt = w_in.cnt;
    p.w_obase = w_in.obase;
    p.w_ovf = w_in.ovf;
    p.w_ovf_cap = w_in.ovf_cap;
    p.m_sf = m_in.sf;
    p.m_pay = m_in.pay;
    p.m_cnt = m_in.cnt;
    p.m_obase = m_in.obase;
    p.m_ovf = m_in.ovf;
    p.m_ovf_cap = m_in.ovf_cap;
    p.g = g;
    p.ow_sf = w_out.sf;
    p.ow_pay = w_out.pay;
    p.ow_cnt = w_out.cnt;
    p.ow_obase = w_out.obase;
    p.ow_ovf = w_out.ovf;
    p.ow_ovf_cap = w_out.ovf_cap;
    p.ow_status = w_out.status;
    p.ow_scratch = (uint8_t *)w_out.scratch;
    p.om_sf = m_out.sf;
    p.om_pay = m_out.pay;
    p.om_cnt = m_out.cnt;
    p.om_obase = m_out.obase;
    p.om_ovf = m_out.ovf;
    p.om_ovf_cap = m_out.ovf_cap;
    p.om_status = m_out.status;
    p.om_scratch = (uint8_t *)m_out.scratch;
    p.n = w_in.n;
    p.block_elems = w_in.layout.block_elems;
    p.cap_words = w_in.layout.cap_words;
    p.nblk = (uint32_t)nb;
    p.mu = mu;
    p.neg_eta = -eta;
    p.park_w = p.ow_cnt == p.w_cnt;
    p.park_m = p.om_cnt == p.m_cnt;
}

// Clear both outputs' scratch headers and status words, the fused kernel,
// both outputs' overflow scans.
lct_status mom_launch(const MomParams &p, uint64_t nb, bool group, void *stream) {
    const OutSides o{{{p.ow_scratch, p.ow_obase, p.ow_ovf, p.ow_ovf_cap, p.ow_status, p.ow_cnt},
                      {p.om_scratch, p.om_obase, p.om_ovf, p.om_ovf_cap, p.om_status, p.om_cnt}},
                     2, nb};
    int e = launch_clear(o, stream);
    if (e != hipSuccess) return hip_fail(e, "clear launch");
    e = launch_mom(p, stream, group);
    if (e != hipSuccess) return hip_fail(e, "momentum launch");
    e = launch_scan(o, stream);
    if (e != hipSuccess) return hip_fail(e, "scan launch");
    return LCT_OK;
}

// The momentum step's aliasing rules (nb: the block count, ~0 for n's): the
// outputs are disjoint from each other; each output's fixed side is its own
// input's buffers, exactly, or disjoint from every input; its overflow,
// status and scratch overlap no input.
bool momentum_alias_ok(const lct_tensor &w_in, const lct_tensor &m_in, const lct_tensor &w_out,
                       const lct_tensor &m_out, uint64_t nb) {
    const Parts pw = parts(w_in, nb), pm = parts(m_in, nb), qw = parts(w_out, nb), qm = parts(m_out, nb);
    const Range qws[] = {qw.sf, qw.pay, qw.cnt, qw.obase, qw.ovf, qw.status, qw.scratch};
    for (const Range &r : qws)
        if (overlaps_any(r, qm)) return false;
    auto check_out = [&](const Parts &own, const Parts &other, const Parts &q) {
        const Range in[] = {own.sf, own.pay, own.cnt, own.obase};
        const Range out[] = {q.sf, q.pay, q.cnt, q.obase};
        for (int i = 0; i < 4; ++i) {
            for (int j = 0; j < 4; ++j) {
                const bool same = i == j && in[i].lo == out[j].lo;
                if (!same && overlap(in[i], out[j])) return false;
            }
            if (overlap(own.ovf, out[i])) return false;
            if (overlaps_any(out[i], other, false)) return false;
        }
        const Range rest[] = {q.ovf, q.status, q.scratch};
        for (const Range &r : rest)
            if (overlaps_any(r, own, false) || overlaps_any(r, other, false)) return false;
        return true;
    };
    return check_out(pw, pm, qw) && check_out(pm, pw, qm);
}

// Aliasing rules, parameters and launches of an update (a tensor, or a
// group's storage when `group`); p's tables (or group references) are set.
lct_status sgd_run(SgdParams &p, const lct_tensor &w_in, const lct_tensor &m, const lct_tensor &w_out,
                   uint64_t nb, float eta, const float *coef, bool group, void *stream) {
    const Parts pw = parts(w_in, nb), pm = parts(m, nb), po = parts(w_out, nb);
    // M is read-only and must not share memory with the output
    const Range mr[] = {pm.sf, pm.pay, pm.cnt, pm.obase, pm.ovf};
    for (const Range &r : mr)
        if (overlaps_any(r, po)) return LCT_EALIAS;
    // the output's fixed side may be W's own buffers, exactly, or disjoint from W
    const Range wf[] = {pw.sf, pw.pay, pw.cnt, pw.obase};
    const Range of[] = {po.sf, po.pay, po.cnt, po.obase};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 4; ++j) {
            const bool same = i == j && wf[i].lo == of[j].lo;
            if (!same && overlap(wf[i], of[j])) return LCT_EALIAS;
        }
        if (overlap(pw.ovf, of[i])) return LCT_EALIAS;
    }
    // overflow, status and scratch of the output never overlap an input
    const Range ow[] = {po.ovf, po.status, po.scratch};
    for (const Range &r : ow)
        if (overlaps_any(r, pw, false) || overlaps_any(r, pm, false)) return LCT_EALIAS;
    lct_status st = check_coef(coef, po);
    if (st != LCT_OK) return st;
    st = check_arch();
    if (st != LCT_OK) return st;
    sgd_params(p, w_in, m, w_out, nb, -eta);
    p.coef = coef;
    return sgd_launch(p, nb, group, stream);
}

// ---- mix

// Aliasing rules of a mix (nb: the block count, ~0 for n's): the output's
// fixed side is the input's own buffers, exactly, or disjoint from it; its
// overflow, status and scratch overlap no part of the input.
bool mix_alias_ok(const lct_tensor &in, const lct_tensor &out, uint64_t nb) {
    const Parts pi = parts(in, nb), po = parts(out, nb);
    const Range fi[] = {pi.sf, pi.pay, pi.cnt, pi.obase}, fo[] = {po.sf, po.pay, po.cnt, po.obase};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 4; ++j)
            if (!(i == j && fi[i].lo == fo[j].lo) && overlap(fi[i], fo[j])) return false;
        if (overlap(pi.ovf, fo[i])) return false;
    }
    for (const Range &r : {po.ovf, po.status, po.scratch})
        if (overlaps_any(r, pi, false)) return false;
    return true;
}

void mix_params(MixParams &p, const lct_tensor &in, const lct_tensor &out, uint64_t nb, float a, float b,
                const float *coef, bool dense, int32_t ahead) {
    p.sf = in.sf;
    p.pay = in.pay;
    p.cnt = in.cnt;
    p.obase = in.obase;
    p.ovf = in.ovf;
    p.ovf_cap = in.ovf_cap;
    p.o_sf = out.sf;
    p.o_pay = out.pay;
    p.o_cnt = out.cnt;
    p.o_obase = out.obase;
    p.o_ovf = out.ovf;
    p.o_ovf_cap = out.ovf_cap;
    p.status = out.status;
    p.scratch = (uint8_t *)out.scratch;
    p.n = in.n;
    p.block_elems = in.layout.block_elems;
    p.cap_words = in.layout.cap_words;
    p.nblk = (uint32_t)nb;
    p.a = a;
    p.b = b;
    p.coef = coef;
    p.park_cnt = out.cnt == in.cnt;
    p.dense = dense;
    p.ahead = ahead != 0;
}

lct_status mix_launch(const MixParams &p, uint64_t nb, bool group, void *stream) {
    const OutSides o{{{p.scratch, p.o_obase, p.o_ovf, p.o_ovf_cap, p.status, p.o_cnt}}, 1, nb};
    int e = launch_clear(o, stream);
    if (e != hipSuccess) return hip_fail(e, "clear launch");
    e = launch_mix(p, stream, group);
    if (e != hipSuccess) return hip_fail(e, "mix launch");
    e = launch_scan(o, stream);
    if (e != hipSuccess) return hip_fail(e, "scan launch");
    return LCT_OK;
}

// ---- norms and clipping

uint64_t type_bytes(int32_t type) { return type == LCT_FP32 ? 4 : 2; }

Range member(const lct_list &x, uint32_t k) { return rng(x.d_x[k], x.n[k] * type_bytes(x.type[k])); }

lct_status check_list(const lct_list *x) {
    if (!x || x->count > kListMaxCount || (x->count > 0 && (!x->n || !x->d_x || !x->type))) return LCT_EINVAL;
    uint64_t total = 0;
    for (uint32_t k = 0; k < x->count; ++k) {
        if (x->type[k] != LCT_BF16 && x->type[k] != LCT_FP16 && x->type[k] != LCT_FP32) return LCT_EINVAL;
        if (x->n[k] > kListMaxElems) return LCT_EINVAL;
        total += x->n[k];
        if (total > kListMaxElems) return LCT_EINVAL;   // checked as it grows: it cannot wrap
        if (x->n[k] == 0) continue;
        if (!x->d_x[k]) return LCT_EINVAL;
        if (!aligned(x->d_x[k], type_bytes(x->type[k]))) return LCT_EALIGN;
    }
    return LCT_OK;
}

lct_status check_norm_args(int32_t kind, double max_norm, double scale, const lct_norm_t *out) {
    if (kind != LCT_NORM_L2 && kind != LCT_NORM_MAX) return LCT_EINVAL;
    if (!(max_norm >= 0) || !std::isfinite(scale) || !out) return LCT_EINVAL;
    return aligned(out, 8) ? LCT_OK : LCT_EALIGN;
}

// A norm's arguments and outputs (each: `count` floats, or null).
lct_status check_norm(int32_t kind, double max_norm, double scale, const void *scratch, uint64_t scratch_bytes,
                      const float *each, uint32_t count, const lct_norm_t *out) {
    const lct_status st = check_norm_args(kind, max_norm, scale, out);
    if (st != LCT_OK) return st;
    if (!scratch) return LCT_EINVAL;
    if (!aligned(scratch, 256) || !aligned(each, 4)) return LCT_EALIGN;
    const Range s = rng(scratch, scratch_bytes), o = rng(out, sizeof *out), e = rng(each, each ? 4ull * count : 0);
    return overlap(s, o) || overlap(s, e) || overlap(o, e) ? LCT_EALIAS : LCT_OK;
}

// The result from `count` part values (every stride-th double).
lct_status norm_join(const double *part, uint64_t count, uint64_t stride, bool squares, NormArgs args,
                     lct_norm_t *out, void *stream) {
    NormJoinParams p;
    memset(&p, 0, sizeof p);
    p.part = part;
    p.count = count;
    p.stride = stride;
    p.out = out;
    p.args = args;
    p.squares = squares;
    const int e = launch_norm_join(p, stream);
    return e == hipSuccess ? LCT_OK : hip_fail(e, "norm join launch");
}

// The cut of a list's tensors [k0, k0 + count): the largest chunks that still
// make 512 of them (two per CU), so that a list of a megabyte is spread over
// the device (a clip of 1M FP16 elements takes 3.9 us, with chunks of 2^14
// elements 5.4) and a long one walked in long pieces.  More workgroups cost a
// short norm more than they read faster (a call on 9.6M FP16 elements: 9.1 us
// with 512 chunks, 10.0 with 1024, 11.5 with 2048).
uint32_t list_shift(const lct_list &x, uint32_t k0, uint32_t count) {
    uint64_t n = 0;
    for (uint32_t j = 0; j < count; ++j) n += x.n[k0 + j];
    uint32_t s = kListChunkMax;
    while (s > kListChunkMin && (n >> s) < kListSpread) --s;
    return s;
}

// Tensors [k0, k0 + count) of a list, in chunks of 2^shift elements.
template <uint32_t N>
void list_args(ListArgs<N> &a, const lct_list &x, uint32_t k0, uint32_t count, uint32_t shift) {
    uint64_t c = 0;
    const uint64_t chunk = 1ull << shift;
    a.shift = shift;
    for (uint32_t j = 0; j < count; ++j) {
        a.x[j] = x.d_x[k0 + j];
        a.n[j] = x.n[k0 + j] | ((uint64_t)x.type[k0 + j] << kListTypeShift);
        a.chunk0[j] = (uint32_t)c;
        c += (x.n[k0 + j] + chunk - 1) >> shift;
    }
    a.count = count;
    a.chunks = a.chunk0[count] = (uint32_t)c;
}

template <uint32_t N>
lct_status list_one(const lct_list &x, bool squares, NormArgs args, float *each, lct_norm_t *out, void *stream) {
    ListOneParams<N> p;
    memset(&p, 0, sizeof p);
    p.each = each;
    p.out = out;
    p.args = args;
    list_args(p.list, x, 0, x.count, kOneShift);
    const int e = launch_list_one(p, squares, stream);
    return e == hipSuccess ? LCT_OK : hip_fail(e, "list norm launch");
}

// One launch for tensors [k0, k0 + count); q gets its cut and workgroups.
template <uint32_t N>
int list_part(const lct_list &x, uint32_t k0, uint32_t count, bool squares, double *run, double *piece,
              ListFinishParams &q, void *stream) {
    ListNormParams<N> p;
    memset(&p, 0, sizeof p);
    list_args(p.list, x, k0, count, list_shift(x, k0, count));
    p.run = run;
    p.piece = piece;
    q.count = count;
    q.chunks = p.list.chunks;
    q.G = std::min(kListGrid, p.list.chunks);
    memcpy(q.chunk0, p.list.chunk0, sizeof p.list.chunk0);
    return q.G ? launch_list_norm(p, q.G, squares, stream) : (int)hipSuccess;
}

lct_status list_norm(const lct_list &x, bool squares, NormArgs args, double *run, float *each, lct_norm_t *out,
                     void *stream) {
    uint64_t ones = 0;   // chunks of the one-launch form
    for (uint32_t k = 0; k < x.count && ones <= kOneMax; ++k) ones += (x.n[k] + (1u << kOneShift) - 1) >> kOneShift;
    if (x.count <= kListMax && ones <= kOneMax)
        return x.count <= kListFew ? list_one<kListFew>(x, squares, args, each, out, stream)
                                   : list_one<kListMax>(x, squares, args, each, out, stream);
    ListFinishParams q;
    memset(&q, 0, sizeof q);
    q.args = args;
    q.squares = squares;
    q.run = run;
    // the launches' runs, one after another; then a place per launch for pieces
    double *piece = run + list_launches(x.count) * kListGrid;
    for (uint32_t k0 = 0; k0 < x.count; k0 += kListMax) {
        const uint32_t count = std::min(kListMax, x.count - k0);
        double *pc = each ? piece : nullptr;
        int e = count <= kListFew ? list_part<kListFew>(x, k0, count, squares, run + q.runs, pc, q, stream)
                                  : list_part<kListMax>(x, k0, count, squares, run + q.runs, pc, q, stream);
        if (e != hipSuccess) return hip_fail(e, "list norm launch");
        q.runs += q.G;
        q.piece = piece;
        q.each = each ? each + k0 : nullptr;
        q.out = k0 + count == x.count ? out : nullptr;
        if (q.each || q.out) {
            e = launch_list_finish(q, stream);
            if (e != hipSuccess) return hip_fail(e, "list norm launch");
        }
        piece += kListGrid + kListMax;
    }
    return LCT_OK;
}

// The norm of a compressed tensor, or (g set) of a group's storage; p's
// tables are set.
lct_status code_norm(CodeNormParams &p, const lct_tensor &t, uint64_t nb, const lct_group *g, int32_t kind,
                     double max_norm, double scale, void *scratch, float *each, lct_norm_t *out, void *stream) {
    const uint32_t count = g ? g->count : 1;
    const uint64_t scr = norm_scratch_bytes(0, nb);
    lct_status st = check_norm(kind, max_norm, scale, scratch, scr, each, count, out);
    if (st != LCT_OK) return st;
    // what is read: the codes, and a group's table (codebooks, members, blocks)
    const Range table = g ? rng(g->d_table, group_table_layout(count, nb).bytes) : Range{0, 0};
    const Range written[] = {rng(scratch, scr), rng(out, sizeof *out), rng(each, each ? 4ull * count : 0)};
    for (const Range &r : written)
        if ((nb > 0 && overlaps_any(r, parts(t, nb), false)) || overlap(r, table)) return LCT_EALIAS;
    st = check_arch();
    if (st != LCT_OK) return st;
    const bool squares = kind == LCT_NORM_L2;
    double *part = static_cast<double *>(scratch);
    if (nb > 0) {
        p.sf = t.sf;
        p.pay = t.pay;
        p.cnt = t.cnt;
        p.obase = t.obase;
        p.ovf = t.ovf;
        p.ovf_cap = t.ovf_cap;
        p.n = t.n;
        p.block_elems = t.layout.block_elems;
        p.cap_words = t.layout.cap_words;
        p.nblk = (uint32_t)nb;
        p.part = part;
        const int e = launch_code_norm(p, g != nullptr, squares, stream);
        if (e != hipSuccess) return hip_fail(e, "code norm launch");
    }
    CodeFinishParams q;
    memset(&q, 0, sizeof q);
    q.part = part;
    q.nblk = nb;
    q.fold = nb > kFoldFrom ? part + nb : nullptr;
    q.out = out;
    q.ent = p.grp.ent;
    q.each = each;
    q.args = {max_norm, scale};
    q.count = count;
    q.squares = squares;
    const int e = launch_code_finish(q, stream);
    if (e != hipSuccess) return hip_fail(e, "code norm launch");
    return q.fold ? norm_join(q.fold, kFoldGrid, 1, squares, q.args, out, stream) : LCT_OK;
}

// One launch of the clip for tensors [k0, k0 + count).
template <uint32_t N>
int clip_part(const lct_list &x, const lct_list &y, uint32_t k0, uint32_t count, const float *coef, void *stream) {
    ListClipParams<N> p;
    memset(&p, 0, sizeof p);
    list_args(p.list, x, k0, count, list_shift(x, k0, count));
    for (uint32_t j = 0; j < count; ++j) {
        p.list.n[j] |= (uint64_t)(y.type[k0 + j] << 2) << kListTypeShift;
        p.y[j] = y.d_x[k0 + j];
    }
    p.coef = coef;
    return p.list.chunks ? launch_list_clip(p, stream) : (int)hipSuccess;
}

// The aliasing rules of a call that reads the tensors of x and writes those
// of y, and that reads or writes one range more: with every range sorted by its
// start, none may begin inside a written one before it, and a written one
// inside none.  In place, x_k and y_k are one range; inputs may overlap each
// other.
lct_status check_list_alias(const lct_list &x, Range also, bool also_written, const lct_list &y) {
    struct Span {
        Range r;
        bool written;
    };
    try {
        std::vector<Span> v;
        v.reserve(2 * (size_t)x.count + 1);
        for (uint32_t k = 0; k < x.count; ++k) {
            if (x.n[k] == 0) continue;
            const Range rx = member(x, k), ry = member(y, k);
            const bool inplace = rx.lo == ry.lo && x.type[k] == y.type[k];
            if (!inplace) v.push_back({rx, false});
            v.push_back({ry, true});
        }
        if (also.lo != also.hi) v.push_back({also, also_written});
        std::sort(v.begin(), v.end(), [](const Span &a, const Span &b) { return a.r.lo < b.r.lo; });
        uintptr_t any = 0, written = 0;   // furthest end of all spans so far, of the written ones
        for (const Span &s : v) {
            if (s.r.lo < written || (s.written && s.r.lo < any)) return LCT_EALIAS;
            any = std::max(any, s.r.hi);
            if (s.written) written = std::max(written, s.r.hi);
        }
    } catch (const std::bad_alloc &) {
        return hip_fail(hipErrorOutOfMemory, "table of ranges");
    }
    return LCT_OK;
}

// ---- orthogonalisation

// A list of matrices: rows[k] divides n[k], and no side is too long.
lct_status check_matrices(const lct_list *x, const uint64_t *rows) {
    const lct_status st = check_list(x);
    if (st != LCT_OK) return st;
    if (x->count > 0 && !rows) return LCT_EINVAL;
    for (uint32_t k = 0; k < x->count; ++k) {
        const uint64_t n = x->n[k], r = rows[k];
        if (n == 0) continue;
        if (r == 0 || n % r || n > kOrthoMaxElems || r > kOrthoMaxSide || n / r > kOrthoMaxSide) return LCT_EINVAL;
    }
    return LCT_OK;
}

// The largest magnitude that p(s) = a s + b s^3 + c s^5 (odd), or with
// `square` b s + c s^2 (for s of A), takes on [0, hi]: at the end or where the
// derivative vanishes.
double poly_most(const float (&coef)[3], double hi, bool square) {
    const double a = coef[0], b = coef[1], c = coef[2];
    auto at = [&](double s) { return std::fabs(square ? b * s + c * s * s : s * (a + s * s * (b + c * s * s))); };
    double most = at(hi);
    auto look = [&](double s) {
        if (s > 0.0 && s < hi) most = std::max(most, at(s));
    };
    if (square) {
        if (c != 0.0) look(-b / (2.0 * c));
        return most;
    }
    // a + 3 b t + 5 c t^2 = 0 in t = s^2
    if (c == 0.0) {
        if (b != 0.0) look(std::sqrt(std::max(0.0, -a / (3.0 * b))));
        return most;
    }
    const double d = 9.0 * b * b - 20.0 * a * c;
    if (d >= 0.0)
        for (const double sign : {-1.0, 1.0}) look(std::sqrt(std::max(0.0, (-3.0 * b + sign * std::sqrt(d)) / (10.0 * c))));
    return most;
}

// Coefficients whose iterates stay within the range of the numbers that the
// kernels hold them in.
bool ortho_coef_ok(const float (&coef)[3], uint32_t steps) {
    for (const float c : coef)
        if (!std::isfinite(c)) return false;
    double hi = 1.001;   // a norm rounded down leaves a singular value slightly above one
    for (uint32_t s = 0; s < steps; ++s) {
        if (!(poly_most(coef, hi * hi, true) <= kOrthoBoundB)) return false;
        hi = poly_most(coef, hi, false) * 1.001;
        if (s + 1 < steps && !(hi <= kOrthoBound)) return false;   // (the last result is not held in FP16)
    }
    return true;
}

uint64_t up_to(uint64_t v, uint64_t step) { return (v + step - 1) / step * step; }

uint64_t ortho_bytes(uint64_t mp, uint64_t np, bool pairs) {
    return 2 * ((pairs ? 6 : 4) * mp * np + (pairs ? 4 : 3) * mp * mp);
}

// Batches of matrices, in list order: f(p, b, bytes) with the matrices' sizes
// and places in the working memory; the other fields are the caller's.  Stops
// at f's first failure.
template <class F>
lct_status ortho_batches(const lct_list &x, const uint64_t *rows, F f) {
    uint32_t k = 0;
    while (k < x.count) {
        OrthoParams p;
        memset(&p, 0, sizeof p);
        uint64_t elems = 0;   // with whole tiles' sides, which is what takes memory and time
        for (; k < x.count && p.count < kOrthoMax; ++k) {
            if (x.n[k] == 0) continue;
            const uint64_t r = rows[k], c = x.n[k] / r;
            const uint64_t padded = up_to(r, kOrthoSmall) * up_to(c, kOrthoSmall);
            if (p.count > 0 && elems + padded > kOrthoBatch) break;
            elems += padded;
            OrthoMat &o = p.mat[p.count++];
            o.m = (uint32_t)std::min(r, c);
            o.n = (uint32_t)std::max(r, c);
            o.type = (uint32_t)x.type[k];
            o.tall = r > c;
            o.pairs = o.m <= kOrthoPairs;
            o.index = k;
            o.x = x.d_x[k];
        }
        if (p.count == 0) break;
        // the longest products first: short ones fill what they leave
        std::stable_sort(p.mat, p.mat + p.count,
                         [](const OrthoMat &a, const OrthoMat &b) { return (uint64_t)a.m + a.n > (uint64_t)b.m + b.n; });
        OrthoBatch b = {kOrthoLarge, 0, 0, 0, 1, 1};
        uint64_t tiles = 0, large = 0, small = 0;   // (their work: m m n with whole tiles' sides)
        for (uint32_t j = 0; j < p.count; ++j) {
            const uint64_t m = p.mat[j].m, n = p.mat[j].n, ml = up_to(m, kOrthoLarge), ms = up_to(m, kOrthoSmall);
            tiles += ml / kOrthoLarge * (up_to(n, kOrthoLarge) / kOrthoLarge);
            large += ml * ml * up_to(n, kOrthoLarge);
            small += ms * ms * up_to(n, kOrthoSmall);
        }
        if (tiles < kOrthoLargeFrom || large > small + small / kOrthoLargePad) b.tile = kOrthoSmall;
        uint64_t bytes = 0;
        for (uint32_t j = 0; j < p.count; ++j) {
            OrthoMat &o = p.mat[j];
            const uint64_t mt = (o.m + b.tile - 1) / b.tile, nt = (o.n + b.tile - 1) / b.tile;
            o.mp = (uint32_t)(mt * b.tile);
            o.np = (uint32_t)(nt * b.tile);
            o.off = bytes;
            o.prep0 = b.prep_tiles;
            o.sym0 = b.sym_tiles;
            o.next0 = b.next_tiles;
            b.prep_tiles += o.mp / 64 * (o.np / 64);
            const uint64_t r = b.tile / kOrthoSmall;   // a large tile is two wide ones
            b.sym_tiles += (uint32_t)(mt * (mt + 1) / 2 * r);
            b.next_tiles += (uint32_t)(mt * nt * r);
            bytes += ortho_bytes(o.mp, o.np, o.pairs);
        }
        if (b.tile == kOrthoSmall) {
            // parts of K for the longest sums; what is shorter gets shorter parts
            uint32_t gram = 0, square = 0;
            for (uint32_t j = 0; j < p.count; ++j) {
                gram = std::max(gram, p.mat[j].np / 32 * (p.mat[j].pairs ? 3 : 1));
                square = std::max(square, p.mat[j].mp / 32 * 3);
            }
            const uint32_t room = std::min(kOrthoSplitMax, kOrthoSplitTo / b.sym_tiles);
            if (gram >= kOrthoLong) b.split_gram = std::max(1u, std::min(room, gram / kOrthoPart));
            if (square >= kOrthoLong) b.split_square = std::max(1u, std::min(room, square / kOrthoPart));
            const uint32_t parts = std::max(b.split_gram, b.split_square);
            p.partial = reinterpret_cast<float *>(bytes);   // (an offset so far)
            if (parts > 1) bytes += 4ull * kOrthoSmall * kOrthoSmall * b.sym_tiles * parts;
        }
        const lct_status st = f(p, b, bytes);
        if (st != LCT_OK) return st;
    }
    return LCT_OK;
}

// The working memory: every matrix's norm, the norms' result and scratch, then
// the largest batch's.
struct OrthoScratch {
    uint64_t out, norm, batch, bytes;
};
OrthoScratch ortho_scratch(const lct_list &x, const uint64_t *rows) {
    OrthoScratch s;
    s.out = align256(4ull * x.count);
    s.norm = s.out + 256;
    s.batch = s.norm + norm_scratch_bytes(x.count, 0);
    uint64_t most = 0;
    (void)ortho_batches(x, rows, [&](OrthoParams &, OrthoBatch &, uint64_t bytes) {
        most = std::max(most, bytes);
        return LCT_OK;
    });
    s.bytes = s.batch + most;
    return s;
}

}  // namespace

extern "C" {

lct_status lct_layout_init(int32_t mode, lct_layout *out) {
    if (!out) return LCT_EINVAL;
    switch (mode) {
    case LCT_CLEAN: *out = {65536, 25}; return LCT_OK;
    case LCT_MEDIUM: *out = {32768, 12}; return LCT_OK;
    case LCT_HIGH: *out = {32768, 11}; return LCT_OK;
    }
    return LCT_EINVAL;
}

lct_status lct_sizes(uint64_t n, const lct_layout *layout, uint64_t ovf_cap, lct_sizes_t *out) {
    if (!layout || !out || !layout_ok(*layout) || !sizes_ok(n, *layout, ovf_cap)) return LCT_EINVAL;
    const uint64_t nb = nblocks(n, *layout);
    out->nblk = nb;
    out->sf = n;
    out->pay = nb * layout->cap_words * kStreams * 4;
    out->cnt = nb * kStreams * 2;
    out->obase = (nb + 1) * 8;
    out->scratch = scr_bytes(nb, ovf_cap);
    out->fixed = out->sf + out->pay + out->cnt + out->obase;
    return LCT_OK;
}

lct_status lct_codebook_build(const lct_model *model, const uint16_t *d_x, uint64_t n, void *stream,
                              lct_codebook *out) {
    if (!model || !out || (n > 0 && !d_x) || n > kMaxElems) return LCT_EINVAL;
    const uint32_t m = (uint32_t)std::min<uint64_t>(n, 4096);
    uint16_t sample[4096];
    if (m > 0) {
        lct_status st = check_arch();
        if (st != LCT_OK) return st;
        std::lock_guard<std::mutex> lock(g_sample_mu);
        const int e = launch_gather(d_x, n, m, stream, sample);
        if (e != hipSuccess) return hip_fail(e, "sample gather");
    }
    return build_codebook(*model, sample, m, out);
}

lct_status lct_codebook_from_lengths(const uint8_t len_base[256], uint8_t esc_len, int32_t shift,
                                     lct_codebook *out) {
    return codebook_from_lengths(len_base, esc_len, shift, out);
}

lct_status lct_tensor_sample(const lct_codebook *cb, const lct_tensor *t, void *stream,
                             uint16_t *sample, uint32_t *m_out) {
    if (!cb || !t || !sample || !tables_ok(*cb)) return LCT_EINVAL;
    const uint32_t m = (uint32_t)std::min<uint64_t>(t->n, 4096);
    if (m > 0) {
        lct_status st = check_tensor(t, false);
        if (st != LCT_OK) return st;
        if (t->n >= (1ull << 52)) return LCT_EINVAL;   // i * n stays within 64 bits
        st = check_arch();
        if (st != LCT_OK) return st;
        SampleParams p;
        memset(&p, 0, sizeof p);
        p.sf = t->sf;
        p.pay = t->pay;
        p.cnt = t->cnt;
        p.obase = t->obase;
        p.ovf = t->ovf;
        p.ovf_cap = t->ovf_cap;
        p.n = t->n;
        p.block_elems = t->layout.block_elems;
        p.cap_words = t->layout.cap_words;
        p.m = m;
        fill_dec(*cb, &p.dec);
        std::lock_guard<std::mutex> lock(g_sample_mu);
        const int e = launch_sample(p, stream, sample);
        if (e != hipSuccess) return hip_fail(e, "compressed sample");
    }
    if (m_out) *m_out = m;
    return LCT_OK;
}

lct_status lct_codebook_reshift(const lct_codebook *cb, const lct_tensor *t, void *stream,
                                lct_codebook *out) {
    if (!cb || !t || !out || !tables_ok(*cb)) return LCT_EINVAL;
    uint16_t sample[4096];
    uint32_t m = 0;
    const lct_status st = lct_tensor_sample(cb, t, stream, sample, &m);
    if (st != LCT_OK) return st;
    return reshift_codebook(*cb, sample, m, out);
}

lct_status lct_codebook_reshift_dense(const lct_codebook *cb, const uint16_t *d_x, uint64_t n,
                                      void *stream, lct_codebook *out) {
    if (!cb || !out || (n > 0 && !d_x) || n > kMaxElems || !tables_ok(*cb)) return LCT_EINVAL;
    const uint32_t m = (uint32_t)std::min<uint64_t>(n, 4096);
    uint16_t sample[4096];
    if (m > 0) {
        lct_status st = check_arch();
        if (st != LCT_OK) return st;
        std::lock_guard<std::mutex> lock(g_sample_mu);
        const int e = launch_gather(d_x, n, m, stream, sample);
        if (e != hipSuccess) return hip_fail(e, "sample gather");
    }
    return reshift_codebook(*cb, sample, m, out);
}

lct_status lct_codebook_adapt(const lct_codebook *cb, const lct_tensor *t, double max_spill_per_elem,
                              void *stream, lct_codebook *out, int32_t *changed) {
    if (!cb || !t || !out || !(max_spill_per_elem >= 0) || !tables_ok(*cb)) return LCT_EINVAL;
    const lct_codebook in = *cb;   // out may be cb
    bool reshift = false;
    if (t->n > 0) {
        lct_status st = check_tensor(t, false);
        if (st != LCT_OK) return st;
        st = check_arch();
        if (st != LCT_OK) return st;
        uint64_t spilled = 0;
        hipStream_t hs = (hipStream_t)stream;
        hipError_t e = hipMemcpyAsync(&spilled, t->obase + nblocks(t->n, t->layout), sizeof spilled,
                                      hipMemcpyDeviceToHost, hs);
        if (e == hipSuccess) e = hipStreamSynchronize(hs);
        if (e != hipSuccess) return hip_fail(e, "spill total read");
        reshift = (double)spilled > max_spill_per_elem * (double)t->n;
    }
    if (reshift) {
        lct_status st = lct_codebook_reshift(&in, t, stream, out);
        if (st != LCT_OK) return st;
    } else {
        *out = in;
    }
    if (changed) *changed = out->shift != in.shift;
    return LCT_OK;
}

lct_status lct_encode(const lct_codebook *cb, const uint16_t *d_x, const lct_tensor *out,
                      void *stream) {
    if (!cb || !out || !tables_ok(*cb)) return LCT_EINVAL;
    if (out->n == 0) return LCT_OK;
    lct_status st = check_tensor(out, true);
    if (st != LCT_OK) return st;
    if (!d_x) return LCT_EINVAL;
    if (!aligned(d_x, 16)) return LCT_EALIGN;
    if (overlaps_any(rng(d_x, out->n * 2), parts(*out))) return LCT_EALIAS;
    st = check_arch();
    if (st != LCT_OK) return st;

    const uint64_t nb = nblocks(out->n, out->layout);
    if (nb > 0xFFFFFFFFull) return LCT_EINVAL;
    EncodeParams p;
    memset(&p, 0, sizeof p);
    p.x = d_x;
    p.n = out->n;
    p.block_elems = out->layout.block_elems;
    p.cap_words = out->layout.cap_words;
    p.nblk = (uint32_t)nb;
    p.sf = out->sf;
    p.pay = out->pay;
    p.cnt = out->cnt;
    p.obase = out->obase;
    p.ovf = out->ovf;
    p.ovf_cap = out->ovf_cap;
    p.status = out->status;
    p.scratch = (uint8_t *)out->scratch;
    fill_enc(*cb, &p.enc);
    const OutSides o{{{p.scratch, p.obase, p.ovf, p.ovf_cap, p.status, p.cnt}}, 1, nb};
    int e = launch_clear(o, stream);
    if (e != hipSuccess) return hip_fail(e, "clear launch");
    e = launch_encode(p, stream);
    if (e != hipSuccess) return hip_fail(e, "encode launch");
    e = launch_scan(o, stream);
    if (e != hipSuccess) return hip_fail(e, "scan launch");
    return LCT_OK;
}

lct_status lct_decode(const lct_codebook *cb, const lct_tensor *in, uint16_t *d_y, void *stream) {
    if (!cb || !in || !tables_ok(*cb)) return LCT_EINVAL;
    if (in->n == 0) return LCT_OK;
    lct_status st = check_tensor(in, false);
    if (st != LCT_OK) return st;
    if (!d_y) return LCT_EINVAL;
    if (!aligned(d_y, 16)) return LCT_EALIGN;
    if (overlaps_any(rng(d_y, in->n * 2), parts(*in), false)) return LCT_EALIAS;
    st = check_arch();
    if (st != LCT_OK) return st;
    const uint64_t nb = nblocks(in->n, in->layout);
    if (nb > 0xFFFFFFFFull) return LCT_EINVAL;
    DecodeParams p;
    memset(&p, 0, sizeof p);
    p.sf = in->sf;
    p.pay = in->pay;
    p.cnt = in->cnt;
    p.obase = in->obase;
    p.ovf = in->ovf;
    p.ovf_cap = in->ovf_cap;
    p.y = d_y;
    p.n = in->n;
    p.block_elems = in->layout.block_elems;
    p.cap_words = in->layout.cap_words;
    p.nblk = (uint32_t)nb;
    fill_dec(*cb, &p.dec);
    const int e = launch_decode(p, stream);
    if (e != hipSuccess) return hip_fail(e, "decode launch");
    return LCT_OK;
}

// The update of one tensor, plain (coef null) or clipped.
static lct_status sgd_one(const lct_codebook *cw, const lct_tensor *w_in, const lct_codebook *cm,
                          const lct_tensor *m, float eta, const float *coef, const lct_codebook *cw_out,
                          const lct_tensor *w_out, void *stream) {
    if (!cw || !cm || !cw_out || !w_in || !m || !w_out) return LCT_EINVAL;
    if (!tables_ok(*cw) || !tables_ok(*cm) || !tables_ok(*cw_out)) return LCT_EINVAL;
    if (w_in->n != m->n || w_in->n != w_out->n) return LCT_EINVAL;
    if (w_in->layout.block_elems != m->layout.block_elems ||
        w_in->layout.block_elems != w_out->layout.block_elems ||
        w_in->layout.cap_words != m->layout.cap_words ||
        w_in->layout.cap_words != w_out->layout.cap_words)
        return LCT_EINVAL;
    if (w_in->n == 0) return LCT_OK;
    lct_status st = check_tensor(w_in, false);
    if (st == LCT_OK) st = check_tensor(m, false);
    if (st == LCT_OK) st = check_tensor(w_out, true);
    if (st != LCT_OK) return st;
    const uint64_t nb = nblocks(w_in->n, w_in->layout);
    if (nb > 0xFFFFFFFFull) return LCT_EINVAL;
    SgdParams p;
    memset(&p, 0, sizeof p);
    fill_enc(*cw_out, &p.wenc);
    fill_dec(*cw, &p.wdec);
    fill_dec(*cm, &p.mdec);
    return sgd_run(p, *w_in, *m, *w_out, nb, eta, coef, false, stream);
}

lct_status lct_sgd_step(const lct_codebook *cw, const lct_tensor *w_in, const lct_codebook *cm,
                        const lct_tensor *m, float eta, const lct_tensor *w_out, void *stream) {
    return sgd_one(cw, w_in, cm, m, eta, nullptr, cw, w_out, stream);
}

lct_status lct_sgd_step_recode(const lct_codebook *cw, const lct_tensor *w_in, const lct_codebook *cm,
                               const lct_tensor *m, float eta, const lct_codebook *cw_out,
                               const lct_tensor *w_out, void *stream) {
    return sgd_one(cw, w_in, cm, m, eta, nullptr, cw_out, w_out, stream);
}

lct_status lct_sgd_step_clip(const lct_codebook *cw, const lct_tensor *w_in, const lct_codebook *cm,
                             const lct_tensor *m, float eta, const float *d_coef, const lct_tensor *w_out,
                             void *stream) {
    if (!d_coef) return LCT_EINVAL;
    return sgd_one(cw, w_in, cm, m, eta, d_coef, cw, w_out, stream);
}

lct_status lct_sgd_step_noalloc(const lct_codebook *cw, const lct_tensor *w_in, const lct_codebook *cm,
                                const lct_tensor *m, float eta, const lct_tensor *w_out, void *stream) {
    if (!cw || !cm || !w_in || !m || !w_out || !tables_ok(*cw) || !tables_ok(*cm)) return LCT_EINVAL;
    if (w_out->n == 0) return lct_sgd_step(cw, w_in, cm, m, eta, w_out, stream);
    if (!layout_ok(w_out->layout) || !sizes_ok(w_out->n, w_out->layout, w_out->ovf_cap)) return LCT_EINVAL;
    if (scr_bytes(nblocks(w_out->n, w_out->layout), w_out->ovf_cap) > kNoAllocScratch) return LCT_ESIZE;
    lct_status st = check_arch();
    if (st != LCT_OK) return st;
    uint8_t *scr = nullptr;
    const int e = noalloc_scratch(&scr);
    if (e != hipSuccess) return hip_fail(e, "static scratch address");
    lct_tensor out = *w_out;
    out.scratch = scr;
    return lct_sgd_step(cw, w_in, cm, m, eta, &out, stream);
}

// The momentum step of one tensor, plain (coef null) or clipped.
static lct_status momentum_one(const lct_codebook *cw, const lct_tensor *w_in, const lct_codebook *cm,
                               const lct_tensor *m_in, const uint16_t *d_g, const float *coef, float mu,
                               float eta, const lct_codebook *cw_out, const lct_codebook *cm_out,
                               const lct_tensor *w_out, const lct_tensor *m_out, void *stream) {
    if (!cw || !cm || !cw_out || !cm_out || !w_in || !m_in || !w_out || !m_out) return LCT_EINVAL;
    if (!tables_ok(*cw) || !tables_ok(*cm) || !tables_ok(*cw_out) || !tables_ok(*cm_out)) return LCT_EINVAL;
    const lct_tensor *all[] = {w_in, m_in, w_out, m_out};
    for (const lct_tensor *t : all)
        if (t->n != w_in->n || t->layout.block_elems != w_in->layout.block_elems ||
            t->layout.cap_words != w_in->layout.cap_words)
            return LCT_EINVAL;
    if (w_in->n == 0) return LCT_OK;
    if (!d_g) return LCT_EINVAL;
    if (!aligned(d_g, 16)) return LCT_EALIGN;
    lct_status st = check_tensor(w_in, false);
    if (st == LCT_OK) st = check_tensor(m_in, false);
    if (st == LCT_OK) st = check_tensor(w_out, true);
    if (st == LCT_OK) st = check_tensor(m_out, true);
    if (st != LCT_OK) return st;
    if (overlaps_any(rng(d_g, w_in->n * 2), parts(*w_out)) || overlaps_any(rng(d_g, w_in->n * 2), parts(*m_out)))
        return LCT_EALIAS;   // the gradient is read only: no output may overlap it
    if (!momentum_alias_ok(*w_in, *m_in, *w_out, *m_out, ~0ull)) return LCT_EALIAS;
    st = check_coef(coef, parts(*w_out));
    if (st == LCT_OK) st = check_coef(coef, parts(*m_out));
    if (st != LCT_OK) return st;
    st = check_arch();
    if (st != LCT_OK) return st;

    const uint64_t nb = nblocks(w_in->n, w_in->layout);
    if (nb > 0xFFFFFFFFull) return LCT_EINVAL;
    // One pass: W and M decoded, M' = rne(mu * M + g) and W' = rne(W - eta * M')
    // with M' as rounded, both re-encoded by the fused kernel.
    MomParams p;
    memset(&p, 0, sizeof p);
    mom_params(p, *w_in, *m_in, d_g, *w_out, *m_out, nb, mu, eta);
    p.coef = coef;
    fill_enc_packed(*cw_out, p.wenc);
    fill_enc_packed(*cm_out, p.menc);
    fill_dec(*cw, &p.wdec);
    fill_dec(*cm, &p.mdec);
    return mom_launch(p, nb, false, stream);
}

lct_status lct_momentum_step(const lct_codebook *cw, const lct_tensor *w_in, const lct_codebook *cm,
                             const lct_tensor *m_in, const uint16_t *d_g, float mu, float eta,
                             const lct_tensor *w_out, const lct_tensor *m_out, void *stream) {
    return momentum_one(cw, w_in, cm, m_in, d_g, nullptr, mu, eta, cw, cm, w_out, m_out, stream);
}

lct_status lct_momentum_step_recode(const lct_codebook *cw, const lct_tensor *w_in,
                                    const lct_codebook *cm, const lct_tensor *m_in,
                                    const uint16_t *d_g, float mu, float eta,
                                    const lct_codebook *cw_out, const lct_codebook *cm_out,
                                    const lct_tensor *w_out, const lct_tensor *m_out, void *stream) {
    return momentum_one(cw, w_in, cm, m_in, d_g, nullptr, mu, eta, cw_out, cm_out, w_out, m_out, stream);
}

lct_status lct_momentum_step_clip(const lct_codebook *cw, const lct_tensor *w_in, const lct_codebook *cm,
                                  const lct_tensor *m_in, const uint16_t *d_g, const float *d_coef, float mu,
                                  float eta, const lct_tensor *w_out, const lct_tensor *m_out, void *stream) {
    if (!d_coef) return LCT_EINVAL;
    return momentum_one(cw, w_in, cm, m_in, d_g, d_coef, mu, eta, cw, cm, w_out, m_out, stream);
}

// ---- groups

lct_status lct_group_table_bytes(uint32_t count, const uint64_t *n, const lct_layout *layout,
                                 uint64_t *bytes) {
    if (!layout || !bytes || !layout_ok(*layout) || (count > 0 && !n)) return LCT_EINVAL;
    uint64_t nb = 0, sf = 0;
    if (!group_extent(count, n, *layout, &nb, &sf)) return LCT_EINVAL;
    *bytes = group_table_layout(count, nb).bytes;
    return LCT_OK;
}

lct_status lct_group_bind(uint32_t count, const uint64_t *n, const lct_layout *layout,
                          const lct_codebook *cbs, uint16_t *const *d_dense, void *d_table,
                          lct_group *out) {
    if (!layout || !out || !cbs || !n || !d_table || count == 0 || !layout_ok(*layout))
        return LCT_EINVAL;
    for (uint32_t k = 0; k < count; ++k)
        if (!tables_ok(cbs[k])) return LCT_EINVAL;
    if (!aligned(d_table, 256)) return LCT_EALIGN;
    uint64_t nb = 0, sf = 0;
    if (!group_extent(count, n, *layout, &nb, &sf)) return LCT_EINVAL;
    if (d_dense) {
        std::vector<Range> rs;
        for (uint32_t k = 0; k < count; ++k) {
            if (n[k] == 0) continue;
            if (!d_dense[k]) return LCT_EINVAL;
            if (!aligned(d_dense[k], 16)) return LCT_EALIGN;
            rs.push_back(rng(d_dense[k], n[k] * 2));
        }
        std::sort(rs.begin(), rs.end(), [](const Range &a, const Range &b) { return a.lo < b.lo; });
        for (size_t i = 1; i < rs.size(); ++i)
            if (rs[i].lo < rs[i - 1].hi) return LCT_EALIAS;
    }
    lct_status st = check_arch();
    if (st != LCT_OK) return st;
    const GroupTableLayout t = group_table_layout(count, nb);
    std::vector<uint8_t> host(t.bytes, 0);
    auto *ent = reinterpret_cast<GroupEntry *>(host.data() + t.ent);
    auto *enc = reinterpret_cast<EncTab *>(host.data() + t.enc);
    auto *dec = reinterpret_cast<DecTab *>(host.data() + t.dec);
    auto *owner = reinterpret_cast<uint32_t *>(host.data() + t.blk_tensor);
    auto *tabs = reinterpret_cast<uint32_t *>(host.data() + t.blk_tab);
    // tensors whose tables are byte-identical share the first one's index
    std::map<std::vector<uint8_t>, uint32_t> first_with;
    uint64_t b0 = 0, e0 = 0;
    for (uint32_t k = 0; k < count; ++k) {
        const uint64_t nbk = nblocks(n[k], *layout);
        ent[k].dense = d_dense ? d_dense[k] : nullptr;
        ent[k].n = n[k];
        ent[k].e0 = e0;
        ent[k].blk0 = (uint32_t)b0;
        ent[k].nblk = (uint32_t)nbk;
        fill_enc(cbs[k], &enc[k]);
        fill_dec(cbs[k], &dec[k]);
        std::vector<uint8_t> key(sizeof(EncTab) + sizeof(DecTab));
        memcpy(key.data(), &enc[k], sizeof(EncTab));
        memcpy(key.data() + sizeof(EncTab), &dec[k], sizeof(DecTab));
        const uint32_t tab = first_with.emplace(std::move(key), k).first->second;
        for (uint64_t j = 0; j < nbk; ++j) {
            owner[b0 + j] = k;
            tabs[b0 + j] = tab;
        }
        b0 += nbk;
        e0 += round256(n[k]);
    }
    const hipError_t e = hipMemcpy(d_table, host.data(), t.bytes, hipMemcpyHostToDevice);
    if (e != hipSuccess) return hip_fail(e, "group table copy");
    out->count = count;
    out->layout = *layout;
    out->nblk = nb;
    out->sf_bytes = sf;
    out->shape_hash = shape_hash(count, n, *layout);
    out->n = n;
    out->d_dense = d_dense;
    out->d_table = d_table;
    return LCT_OK;
}

lct_status lct_group_fit(const lct_codebook *base, const uint64_t *n, uint16_t *const *d_dense,
                         const lct_layout *layout, void *d_table, int32_t *d_shift, void *stream,
                         lct_group *out) {
    if (!base || !n || !d_dense || !layout || !d_table || !out || !layout_ok(*layout)) return LCT_EINVAL;
    // the device builds the tables from the base code: its lengths must make one
    lct_codebook check;
    if (codebook_from_lengths(base->len_base, base->esc_len, 0, &check) != LCT_OK) return LCT_EINVAL;
    if (n[0] > 0 && !d_dense[0]) return LCT_EINVAL;
    if (!aligned(d_table, 256) || (n[0] > 0 && !aligned(d_dense[0], 16)) || (d_shift && !aligned(d_shift, 4)))
        return LCT_EALIGN;
    uint64_t nb = 0, sf = 0;
    if (!group_extent(1, n, *layout, &nb, &sf)) return LCT_EINVAL;
    lct_status st = check_arch();
    if (st != LCT_OK) return st;
    const GroupTableLayout t = group_table_layout(1, nb);
    uint8_t *tab = static_cast<uint8_t *>(d_table);
    FitParams p;
    memset(&p, 0, sizeof p);
    p.x = d_dense[0];
    p.n = n[0];
    p.m = (uint32_t)std::min<uint64_t>(n[0], 4096);
    p.nblk = (uint32_t)nb;
    p.esc_len = base->esc_len;
    memcpy(p.base, base->len_base, sizeof p.base);
    p.ent = reinterpret_cast<GroupEntry *>(tab + t.ent);
    p.enc = reinterpret_cast<EncTab *>(tab + t.enc);
    p.dec = reinterpret_cast<DecTab *>(tab + t.dec);
    p.blk_tensor = reinterpret_cast<uint32_t *>(tab + t.blk_tensor);
    p.blk_tab = reinterpret_cast<uint32_t *>(tab + t.blk_tab);
    p.shift_out = d_shift;
    const int e = launch_fit(p, stream);
    if (e != hipSuccess) return hip_fail(e, "fit launch");
    out->count = 1;
    out->layout = *layout;
    out->nblk = nb;
    out->sf_bytes = sf;
    out->shape_hash = shape_hash(1, n, *layout);
    out->n = n;
    out->d_dense = d_dense;
    out->d_table = d_table;
    return LCT_OK;
}

lct_status lct_group_sizes(const lct_group *g, uint64_t ovf_cap, lct_sizes_t *out) {
    if (!g || !out || !layout_ok(g->layout) || g->nblk > 0xFFFFFFFFull || ovf_cap > kMaxOvfCap)
        return LCT_EINVAL;
    out->nblk = g->nblk;
    out->sf = g->sf_bytes;
    out->pay = g->nblk * g->layout.cap_words * kStreams * 4;
    out->cnt = g->nblk * kStreams * 2;
    out->obase = (g->nblk + 1) * 8;
    out->scratch = scr_bytes(g->nblk, ovf_cap);
    out->fixed = out->sf + out->pay + out->cnt + out->obase;
    return LCT_OK;
}

lct_status lct_group_tensor(const lct_group *g, const lct_tensor *all, uint32_t k, lct_tensor *out) {
    if (!g || !all || !out || !g->n || k >= g->count) return LCT_EINVAL;
    uint64_t b0 = 0, e0 = 0;
    for (uint32_t j = 0; j < k; ++j) {
        b0 += nblocks(g->n[j], g->layout);
        e0 += round256(g->n[j]);
    }
    *out = *all;
    out->n = g->n[k];
    out->sf = all->sf + e0;
    out->pay = all->pay + b0 * g->layout.cap_words * kStreams;
    out->cnt = all->cnt + b0 * kStreams;
    out->obase = all->obase + b0;
    return LCT_OK;
}

lct_status lct_encode_group(const lct_group *g, const lct_tensor *all, void *stream) {
    lct_status st = check_group(g, all, true);
    if (st != LCT_OK) return st;
    st = check_group_dense(*g, parts(*all, g->nblk));
    if (st != LCT_OK) return st;
    st = check_arch();
    if (st != LCT_OK) return st;
    if (g->nblk == 0) return LCT_OK;
    EncodeParams p;
    memset(&p, 0, sizeof p);
    p.n = all->n;
    p.block_elems = g->layout.block_elems;
    p.cap_words = g->layout.cap_words;
    p.nblk = (uint32_t)g->nblk;
    p.sf = all->sf;
    p.pay = all->pay;
    p.cnt = all->cnt;
    p.obase = all->obase;
    p.ovf = all->ovf;
    p.ovf_cap = all->ovf_cap;
    p.status = all->status;
    p.scratch = (uint8_t *)all->scratch;
    p.grp = group_ref(*g);
    const OutSides o{{{p.scratch, p.obase, p.ovf, p.ovf_cap, p.status, p.cnt}}, 1, g->nblk};
    int e = launch_clear(o, stream);
    if (e != hipSuccess) return hip_fail(e, "clear launch");
    e = launch_encode(p, stream, true);
    if (e != hipSuccess) return hip_fail(e, "group encode launch");
    e = launch_scan(o, stream);
    if (e != hipSuccess) return hip_fail(e, "scan launch");
    return LCT_OK;
}

lct_status lct_decode_group(const lct_group *g, const lct_tensor *all, void *stream) {
    lct_status st = check_group(g, all, false);
    if (st != LCT_OK) return st;
    st = check_group_dense(*g, parts(*all, g->nblk));
    if (st != LCT_OK) return st;
    st = check_arch();
    if (st != LCT_OK) return st;
    if (g->nblk == 0) return LCT_OK;
    DecodeParams p;
    memset(&p, 0, sizeof p);
    p.sf = all->sf;
    p.pay = all->pay;
    p.cnt = all->cnt;
    p.obase = all->obase;
    p.ovf = all->ovf;
    p.ovf_cap = all->ovf_cap;
    p.n = all->n;
    p.block_elems = g->layout.block_elems;
    p.cap_words = g->layout.cap_words;
    p.nblk = (uint32_t)g->nblk;
    p.grp = group_ref(*g);
    const int e = launch_decode(p, stream, true);
    if (e != hipSuccess) return hip_fail(e, "group decode launch");
    return LCT_OK;
}

static lct_status sgd_group(const lct_group *gw, const lct_tensor *w_all, const lct_group *gm,
                            const lct_tensor *m_all, float eta, const float *coef, const lct_tensor *w_out,
                            void *stream) {
    lct_status st = check_group(gw, w_all, false);
    if (st == LCT_OK) st = check_group(gm, m_all, false);
    if (st == LCT_OK) st = check_group(gw, w_out, true);
    if (st != LCT_OK) return st;
    if (gm->shape_hash != gw->shape_hash || gm->count != gw->count || gm->nblk != gw->nblk ||
        gm->sf_bytes != gw->sf_bytes)
        return LCT_EINVAL;
    for (uint32_t k = 0; k < gw->count; ++k)
        if (gw->n[k] != gm->n[k]) return LCT_EINVAL;
    if (gw->nblk == 0) return LCT_OK;
    SgdParams p;
    memset(&p, 0, sizeof p);
    p.gw = group_ref(*gw);
    p.gm = group_ref(*gm);
    return sgd_run(p, *w_all, *m_all, *w_out, gw->nblk, eta, coef, true, stream);
}

lct_status lct_sgd_step_group(const lct_group *gw, const lct_tensor *w_all, const lct_group *gm,
                              const lct_tensor *m_all, float eta, const lct_tensor *w_out,
                              void *stream) {
    return sgd_group(gw, w_all, gm, m_all, eta, nullptr, w_out, stream);
}

lct_status lct_sgd_step_clip_group(const lct_group *gw, const lct_tensor *w_all, const lct_group *gm,
                                   const lct_tensor *m_all, float eta, const float *d_coef,
                                   const lct_tensor *w_out, void *stream) {
    if (!d_coef) return LCT_EINVAL;
    return sgd_group(gw, w_all, gm, m_all, eta, d_coef, w_out, stream);
}

static lct_status momentum_group(const lct_group *gw, const lct_tensor *w_all, const lct_group *gm,
                                 const lct_tensor *m_all, const lct_group *gg, const float *coef, float mu,
                                 float eta, const lct_tensor *w_out, const lct_tensor *m_out, void *stream) {
    lct_status st = check_group(gw, w_all, false);
    if (st == LCT_OK) st = check_group(gm, m_all, false);
    if (st == LCT_OK) st = check_group(gw, w_out, true);
    if (st == LCT_OK) st = check_group(gm, m_out, true);
    if (st != LCT_OK) return st;
    if (!gg || !gg->d_table || !gg->n) return LCT_EINVAL;
    for (const lct_group *o : {gm, gg}) {
        if (o->shape_hash != gw->shape_hash || o->count != gw->count || o->nblk != gw->nblk ||
            o->sf_bytes != gw->sf_bytes)
            return LCT_EINVAL;
        for (uint32_t k = 0; k < gw->count; ++k)
            if (o->n[k] != gw->n[k]) return LCT_EINVAL;
    }
    // the gradients (gg's dense buffers) are read only: no output may overlap them
    st = check_group_dense(*gg, parts(*w_out, gw->nblk));
    if (st == LCT_OK) st = check_group_dense(*gg, parts(*m_out, gw->nblk));
    if (st != LCT_OK) return st;
    if (!momentum_alias_ok(*w_all, *m_all, *w_out, *m_out, gw->nblk)) return LCT_EALIAS;
    st = check_coef(coef, parts(*w_out, gw->nblk));
    if (st == LCT_OK) st = check_coef(coef, parts(*m_out, gw->nblk));
    if (st != LCT_OK) return st;
    st = check_arch();
    if (st != LCT_OK) return st;
    if (gw->nblk == 0) return LCT_OK;
    const uint64_t nb = gw->nblk;
    MomParams p;
    memset(&p, 0, sizeof p);
    mom_params(p, *w_all, *m_all, nullptr, *w_out, *m_out, nb, mu, eta);
    p.gw = group_ref(*gw);
    p.gm = group_ref(*gm);
    p.gg = group_ref(*gg);
    p.coef = coef;
    return mom_launch(p, nb, true, stream);
}

lct_status lct_momentum_step_group(const lct_group *gw, const lct_tensor *w_all, const lct_group *gm,
                                   const lct_tensor *m_all, const lct_group *gg, float mu, float eta,
                                   const lct_tensor *w_out, const lct_tensor *m_out, void *stream) {
    return momentum_group(gw, w_all, gm, m_all, gg, nullptr, mu, eta, w_out, m_out, stream);
}

lct_status lct_momentum_step_clip_group(const lct_group *gw, const lct_tensor *w_all, const lct_group *gm,
                                        const lct_tensor *m_all, const lct_group *gg, const float *d_coef,
                                        float mu, float eta, const lct_tensor *w_out,
                                        const lct_tensor *m_out, void *stream) {
    if (!d_coef) return LCT_EINVAL;
    return momentum_group(gw, w_all, gm, m_all, gg, d_coef, mu, eta, w_out, m_out, stream);
}

// ---- norms and clipping

lct_status lct_norm_scratch(uint32_t count, uint64_t nblk, uint64_t *bytes) {
    if (!bytes || count > kListMaxCount || nblk > 0xFFFFFFFFull) return LCT_EINVAL;
    *bytes = norm_scratch_bytes(count, nblk);
    return LCT_OK;
}

lct_status lct_list_norm(const lct_list *x, int32_t kind, double max_norm, double scale, void *d_scratch,
                         float *d_each, lct_norm_t *d_out, void *stream) {
    lct_status st = check_list(x);
    if (st != LCT_OK) return st;
    const uint64_t scr = norm_scratch_bytes(x->count, 0);
    st = check_norm(kind, max_norm, scale, d_scratch, scr, d_each, x->count, d_out);
    if (st != LCT_OK) return st;
    const Range out[] = {rng(d_scratch, scr), rng(d_each, d_each ? 4ull * x->count : 0), rng(d_out, sizeof *d_out)};
    for (uint32_t k = 0; k < x->count; ++k)
        for (const Range &r : out)
            if (overlap(member(*x, k), r)) return LCT_EALIAS;
    st = check_arch();
    if (st != LCT_OK) return st;
    return list_norm(*x, kind == LCT_NORM_L2, {max_norm, scale}, static_cast<double *>(d_scratch), d_each, d_out,
                     stream);
}

lct_status lct_tensor_norm(const lct_codebook *cb, const lct_tensor *t, int32_t kind, double max_norm,
                           double scale, void *d_scratch, lct_norm_t *d_out, void *stream) {
    if (!cb || !t || !tables_ok(*cb)) return LCT_EINVAL;
    uint64_t nb = 0;
    if (t->n > 0) {
        const lct_status st = check_tensor(t, false);
        if (st != LCT_OK) return st;
        nb = nblocks(t->n, t->layout);
    }
    CodeNormParams p;
    memset(&p, 0, sizeof p);
    fill_dec(*cb, &p.dec);
    return code_norm(p, *t, nb, nullptr, kind, max_norm, scale, d_scratch, nullptr, d_out, stream);
}

lct_status lct_group_norm(const lct_group *g, const lct_tensor *all, int32_t kind, double max_norm,
                          double scale, void *d_scratch, float *d_each, lct_norm_t *d_out, void *stream) {
    const lct_status st = check_group(g, all, false);
    if (st != LCT_OK) return st;
    CodeNormParams p;
    memset(&p, 0, sizeof p);
    p.grp = group_ref(*g);
    return code_norm(p, *all, g->nblk, g, kind, max_norm, scale, d_scratch, d_each, d_out, stream);
}

lct_status lct_norm_join(const lct_norm_t *d_parts, uint32_t count, int32_t kind, double max_norm,
                         double scale, lct_norm_t *d_out, void *stream) {
    if (count > 0 && !d_parts) return LCT_EINVAL;
    if (!aligned(d_parts, 8)) return LCT_EALIGN;
    lct_status st = check_norm_args(kind, max_norm, scale, d_out);
    if (st != LCT_OK) return st;
    st = check_arch();
    if (st != LCT_OK) return st;
    static_assert(sizeof(lct_norm_t) == 16 && offsetof(lct_norm_t, sum) == 0, "sums are every second double");
    return norm_join(reinterpret_cast<const double *>(d_parts), count, 2, kind == LCT_NORM_L2, {max_norm, scale},
                     d_out, stream);
}

lct_status lct_list_clip(const lct_list *x, const float *d_coef, const lct_list *y, void *stream) {
    lct_status st = check_list(x);
    if (st == LCT_OK) st = check_list(y);
    if (st != LCT_OK) return st;
    if (!d_coef || x->count != y->count) return LCT_EINVAL;
    if (!aligned(d_coef, 4)) return LCT_EALIGN;
    for (uint32_t k = 0; k < x->count; ++k)
        if (x->n[k] != y->n[k]) return LCT_EINVAL;
    st = check_list_alias(*x, rng(d_coef, 4), false, *y);
    if (st != LCT_OK) return st;
    st = check_arch();
    if (st != LCT_OK) return st;
    for (uint32_t k0 = 0; k0 < x->count; k0 += kClipMax) {
        const uint32_t count = std::min(kClipMax, x->count - k0);
        const int e = count <= kListFew ? clip_part<kListFew>(*x, *y, k0, count, d_coef, stream)
                                        : clip_part<kClipMax>(*x, *y, k0, count, d_coef, stream);
        if (e != hipSuccess) return hip_fail(e, "clip launch");
    }
    return LCT_OK;
}

// ---- mix of a compressed tensor with a dense one

lct_status lct_mix_step(const lct_codebook *cb, const lct_tensor *y_in, float a, const uint16_t *d_x, float b,
                        const float *d_coef, const lct_codebook *cb_out, const lct_tensor *y_out,
                        uint16_t *d_dense, int32_t ahead, void *stream) {
    if (!cb || !y_in || !y_out || !cb_out || !tables_ok(*cb) || !tables_ok(*cb_out)) return LCT_EINVAL;
    if (y_in->n != y_out->n || y_in->layout.block_elems != y_out->layout.block_elems ||
        y_in->layout.cap_words != y_out->layout.cap_words || (ahead && !d_dense))
        return LCT_EINVAL;
    if (y_in->n == 0) return layout_ok(y_in->layout) ? LCT_OK : LCT_EINVAL;
    lct_status st = check_tensor(y_in, false);
    if (st == LCT_OK) st = check_tensor(y_out, true);
    if (st != LCT_OK) return st;
    if (!d_x) return LCT_EINVAL;
    if (!aligned(d_x, 16) || !aligned(d_dense, 16)) return LCT_EALIGN;
    const uint64_t nb = nblocks(y_in->n, y_in->layout);
    const Parts pi = parts(*y_in), po = parts(*y_out);
    const Range x = rng(d_x, 2 * y_in->n), d = rng(d_dense, d_dense ? 2 * y_in->n : 0);
    if (!mix_alias_ok(*y_in, *y_out, nb) || overlaps_any(x, po)) return LCT_EALIAS;
    if (overlaps_any(d, pi, false) || overlaps_any(d, po) || (overlap(d, x) && d.lo != x.lo)) return LCT_EALIAS;
    st = check_coef(d_coef, po);
    if (st != LCT_OK) return st;
    if (d_coef && overlap(rng(d_coef, 4), d)) return LCT_EALIAS;
    st = check_arch();
    if (st != LCT_OK) return st;
    MixParams p;
    memset(&p, 0, sizeof p);
    mix_params(p, *y_in, *y_out, nb, a, b, d_coef, d_dense != nullptr, ahead);
    p.x = d_x;
    p.d = d_dense;
    fill_dec(*cb, &p.dec);
    fill_enc(*cb_out, &p.enc);
    return mix_launch(p, nb, false, stream);
}

lct_status lct_mix_step_group(const lct_group *g, const lct_tensor *y_all, float a, const lct_group *gx, float b,
                              const float *d_coef, const lct_tensor *y_out, const lct_group *gd, int32_t ahead,
                              void *stream) {
    lct_status st = check_group(g, y_all, false);
    if (st == LCT_OK) st = check_group(g, y_out, true);
    if (st != LCT_OK) return st;
    if (!gx || (ahead && !gd)) return LCT_EINVAL;
    for (const lct_group *o : {gx, gd}) {
        if (!o) continue;
        if (!o->d_table || !o->n || o->shape_hash != g->shape_hash || o->count != g->count || o->nblk != g->nblk ||
            o->sf_bytes != g->sf_bytes)
            return LCT_EINVAL;
        for (uint32_t k = 0; k < g->count; ++k)
            if (o->n[k] != g->n[k]) return LCT_EINVAL;
    }
    st = check_group_dense(*gx, parts(*y_out, g->nblk));
    if (st != LCT_OK) return st;
    if (gd) {
        st = check_group_dense(*gd, parts(*y_out, g->nblk));
        if (st == LCT_OK) st = check_group_dense(*gd, parts(*y_all, g->nblk));
        if (st != LCT_OK) return st;
        // the dense results: x's own buffers, or disjoint from all of them
        // (status and scratch of the input, which the check above includes,
        // are not in use: an overlap with them is refused all the same)
        try {
            const std::vector<int32_t> types(g->count, LCT_BF16);
            const lct_list lx{g->count, gx->n, reinterpret_cast<void *const *>(gx->d_dense), types.data()};
            const lct_list ld{g->count, gd->n, reinterpret_cast<void *const *>(gd->d_dense), types.data()};
            st = check_list_alias(lx, rng(d_coef, d_coef ? 4 : 0), false, ld);
        } catch (const std::bad_alloc &) {
            return hip_fail(hipErrorOutOfMemory, "table of types");
        }
        if (st != LCT_OK) return st;
    }
    if (!mix_alias_ok(*y_all, *y_out, g->nblk)) return LCT_EALIAS;
    st = check_coef(d_coef, parts(*y_out, g->nblk));
    if (st != LCT_OK) return st;
    st = check_arch();
    if (st != LCT_OK) return st;
    if (g->nblk == 0) return LCT_OK;
    MixParams p;
    memset(&p, 0, sizeof p);
    mix_params(p, *y_all, *y_out, g->nblk, a, b, d_coef, gd != nullptr, ahead);
    p.g = group_ref(*g);
    p.gx = group_ref(*gx);
    if (gd) p.gd = group_ref(*gd);
    return mix_launch(p, g->nblk, true, stream);
}

// ---- rows of a compressed table, and their gradient

static int sort_rows(const void *index, int32_t wide, uint64_t count, uint64_t rows, const RowScratch &s,
                     void *scratch, const uint32_t **key, const uint32_t **token, void *stream) {
    SortParams q;
    memset(&q, 0, sizeof q);
    q.index = index;
    q.count = (uint32_t)count;
    q.rows = (uint32_t)rows;
    q.wide = wide != 0;
    return launch_row_sort(q, s, static_cast<uint8_t *>(scratch), key, token, stream);
}

static bool type_ok(int32_t t) { return t == LCT_BF16 || t == LCT_FP16 || t == LCT_FP32; }

lct_status lct_rows_scratch(uint64_t count, uint64_t cols, uint64_t *bytes) {
    if (!bytes || count > kMaxTokens || cols > kMaxCols) return LCT_EINVAL;
    *bytes = row_scratch(count, cols).bytes;
    return LCT_OK;
}

lct_status lct_tensor_rows(const lct_codebook *cb, const lct_tensor *t, uint64_t cols, const void *d_index,
                           int32_t wide, uint64_t count, float scale, void *d_y, int32_t type, void *d_scratch,
                           void *stream) {
    if (!cb || !t || !tables_ok(*cb) || cols == 0 || cols > kMaxCols || count > kMaxTokens || !type_ok(type))
        return LCT_EINVAL;
    if (!layout_ok(t->layout) || t->n % cols || t->n / cols > kMaxRows) return LCT_EINVAL;
    if (count == 0) return LCT_OK;
    if (t->n > 0) {
        const lct_status st = check_tensor(t, false);
        if (st != LCT_OK) return st;
    }
    if (!d_index || !d_y) return LCT_EINVAL;
    if (!aligned(d_index, wide ? 8 : 4) || !aligned(d_y, type_bytes(type))) return LCT_EALIGN;
    if (!aligned(d_scratch, 256)) return LCT_EALIGN;
    const RowScratch s = row_scratch(count, 0);
    const Range y = rng(d_y, count * cols * type_bytes(type)), idx = rng(d_index, count * (wide ? 8 : 4));
    const Range scr = rng(d_scratch, d_scratch ? s.bytes : 0);
    if (overlap(y, idx) || overlap(y, scr) || overlap(scr, idx)) return LCT_EALIAS;
    if (t->n > 0 && (overlaps_any(y, parts(*t), false) || overlaps_any(scr, parts(*t), false))) return LCT_EALIAS;
    const lct_status st = check_arch();
    if (st != LCT_OK) return st;
    RowsParams p;
    memset(&p, 0, sizeof p);
    p.sf = t->sf;
    p.pay = t->pay;
    p.cnt = t->cnt;
    p.obase = t->obase;
    p.ovf = t->ovf;
    p.ovf_cap = t->ovf_cap;
    p.n = t->n;
    p.rows = t->n / cols;
    p.cols = cols;
    p.count = count;
    p.block_elems = t->layout.block_elems;
    p.cap_words = t->layout.cap_words;
    p.wide = wide != 0;
    p.type = (uint32_t)type;
    p.index = d_index;
    p.y = d_y;
    p.scale = scale;
    fill_dec(*cb, &p.dec);
    int e = hipSuccess;
    p.run = 1;
    p.piece = (uint32_t)std::min<uint64_t>((cols + 15) / 16 * 16, kRowsRoom);
    if (d_scratch && count >= kRowsSortFrom && count >= 2 * nblocks(t->n, t->layout)) {
        for (uint32_t r = kRowsRun; r > 1 && p.run == 1; r /= 2)
            if (r * p.piece <= kRowsRoom) p.run = r;
        e = sort_rows(d_index, wide, count, p.rows, s, d_scratch, &p.key, &p.token, stream);
        if (e != hipSuccess) return hip_fail(e, "sort launch");
    }
    e = launch_rows(p, stream);
    return e == hipSuccess ? LCT_OK : hip_fail(e, "rows launch");
}

lct_status lct_rows_grad(const void *d_index, int32_t wide, uint64_t count, const void *d_dy, int32_t dy_type,
                         uint64_t rows, uint64_t cols, float scale, int32_t add, void *d_g, int32_t g_type,
                         void *d_scratch, void *stream) {
    if (count > kMaxTokens || rows > kMaxRows || cols > kMaxCols || !type_ok(dy_type) || !type_ok(g_type))
        return LCT_EINVAL;
    if (rows == 0 || cols == 0) return LCT_OK;
    if (!d_g || !d_scratch || (count > 0 && (!d_index || !d_dy))) return LCT_EINVAL;
    if (!aligned(d_index, wide ? 8 : 4) || !aligned(d_dy, type_bytes(dy_type)) ||
        !aligned(d_g, type_bytes(g_type)) || !aligned(d_scratch, 256))
        return LCT_EALIGN;
    const RowScratch s = row_scratch(count, cols);
    const Range idx = rng(d_index, count * (wide ? 8 : 4)), dy = rng(d_dy, count * cols * type_bytes(dy_type));
    const Range g = rng(d_g, rows * cols * type_bytes(g_type)), scr = rng(d_scratch, s.bytes);
    if (overlap(g, idx) || overlap(g, dy) || overlap(g, scr) || overlap(scr, idx) || overlap(scr, dy))
        return LCT_EALIAS;
    const lct_status st = check_arch();
    if (st != LCT_OK) return st;
    uint8_t *scratch = static_cast<uint8_t *>(d_scratch);
    RowGradParams p;
    memset(&p, 0, sizeof p);
    if (count > 0) {
        const int e = sort_rows(d_index, wide, count, rows, s, d_scratch, &p.key, &p.token, stream);
        if (e != hipSuccess) return hip_fail(e, "sort launch");
    }
    p.dy = d_dy;
    p.g = d_g;
    p.part = reinterpret_cast<float *>(scratch + s.part);
    p.cols = cols;
    p.count = (uint32_t)count;
    p.rows = (uint32_t)rows;
    p.tile = row_tile(count);
    p.tiles = (uint32_t)((count + p.tile - 1) / p.tile);
    p.add = add != 0;
    p.scale = scale;
    const int e = launch_row_grad(p, (uint32_t)dy_type, (uint32_t)g_type, stream);
    return e == hipSuccess ? LCT_OK : hip_fail(e, "row gradient launch");
}

// ---- orthogonalisation

lct_status lct_orthogonal_scratch(const lct_list *x, const uint64_t *rows, uint64_t *bytes) {
    if (!bytes) return LCT_EINVAL;
    const lct_status st = check_matrices(x, rows);
    if (st != LCT_OK) return st;
    *bytes = ortho_scratch(*x, rows).bytes;
    return LCT_OK;
}

lct_status lct_list_orthogonalize(const lct_list *x, const uint64_t *rows, const lct_list *y, uint32_t steps,
                                  const float coef[3], const float *scale, void *d_scratch, void *stream) {
    lct_status st = check_matrices(x, rows);
    if (st == LCT_OK) st = check_list(y);
    if (st != LCT_OK) return st;
    if (!coef || steps < 1 || steps > 32 || x->count != y->count || !d_scratch) return LCT_EINVAL;
    for (uint32_t k = 0; k < x->count; ++k)
        if (x->n[k] != y->n[k] || y->type[k] != LCT_BF16) return LCT_EINVAL;
    const float cf[3] = {coef[0], coef[1], coef[2]};
    if (!ortho_coef_ok(cf, steps)) return LCT_EINVAL;
    if (!aligned(d_scratch, 256)) return LCT_EALIGN;
    const OrthoScratch s = ortho_scratch(*x, rows);
    st = check_list_alias(*x, rng(d_scratch, s.bytes), true, *y);
    if (st != LCT_OK) return st;
    st = check_arch();
    if (st != LCT_OK) return st;
    uint8_t *scr = static_cast<uint8_t *>(d_scratch);
    float *norm = reinterpret_cast<float *>(scr);
    if (x->count > 0) {
        st = list_norm(*x, true, {INFINITY, 1.0}, reinterpret_cast<double *>(scr + s.norm), norm,
                       reinterpret_cast<lct_norm_t *>(scr + s.out), stream);
        if (st != LCT_OK) return st;
    }
    return ortho_batches(*x, rows, [&](OrthoParams &p, OrthoBatch &b, uint64_t) {
        p.scratch = scr + s.batch;
        p.partial = reinterpret_cast<float *>(p.scratch + reinterpret_cast<uint64_t>(p.partial));
        p.norm = norm;
        p.xscale = kOrthoX;
        p.a = cf[0];
        p.kx = (float)(kOrthoA / (kOrthoX * kOrthoX));
        p.ka = (float)(cf[1] * kOrthoB / kOrthoA);
        p.kaa = (float)(cf[2] * kOrthoB / (kOrthoA * kOrthoA));
        p.kbx = (float)(1.0 / kOrthoB);
        for (uint32_t j = 0; j < p.count; ++j) {
            OrthoMat &o = p.mat[j];
            o.y = const_cast<void *>(y->d_x[o.index]);
            o.scale = scale ? scale[o.index] : 1.0f;
        }
        const int e = launch_ortho(p, b, steps, stream);
        return e == hipSuccess ? LCT_OK : hip_fail(e, "orthogonalisation launch");
    });
}

const char *lct_strerror(lct_status st) {
    switch (st) {
    case LCT_OK: return "ok";
    case LCT_EINVAL: return "invalid argument";
    case LCT_EALIGN: return "misaligned device pointer";
    case LCT_EALIAS: return "illegal buffer overlap";
    case LCT_EHIP: return "HIP runtime error";
    case LCT_EARCH: return "device is not gfx950";
    case LCT_ESIZE: return "working memory needed exceeds the static scratch of the allocation-free call";
    }
    return "unknown status";
}

const char *lct_last_hip_error(void) { return g_hip_msg; }

}  // extern "C"

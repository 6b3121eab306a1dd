// C ABI of the delta-rule layer's operators: argument validation, workspace layout, launch
// dispatch. Declared in include/selscan_ops.h. Nothing here touches the device before all
// arguments have been validated, so a rejected call enqueues nothing.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "ops_check.h"
#include "ops_layer_internal.h"

namespace selscan {

// Segments that run at the same time: two workgroups a CU where it holds two (bf16, dk up to 128) and a segment
// then has 16 chunks at least, else one, which is faster alone, with fewer to join. 128 x 128 in bf16, none, two and one: 32768
// tokens of 16 heads 2916, 708 and 760 us, 8192 of 16 723, 281 and 243, 2048 of 40 203, 163 and 157 (in fp32, where a CU
// holds one: 5990, 1615 and 1560, 1508, 509 and 446, 399, 332 and 293). A segment has four chunks at least, as each is
// one more to join.
int64_t gdr_segment(int64_t BH, int64_t dv, int64_t nchunks, bool two) {
    const int64_t groups = BH * ((dv + 63) / 64);           // workgroups of one segment
    int64_t n = two ? 512 / groups : 0;
    if (nchunks < 16 * n || !two) n = 256 / groups;
    if (n < 2 || nchunks < 8) return nchunks;
    const int64_t seg = (nchunks + n - 1) / n;
    return seg < 4 ? 4 : seg;
}

// The backward's: one workgroup a CU, so that what a segment does for itself slows no other. 32768 tokens of 16 heads of
// 128 x 128, no segments, one and two workgroups a CU: 4.2, 1.84 and 1.89 ms in bf16, 8.9, 3.9 and 5.4 in fp32. Up to five chunks the
// two launches more cost what they save (4 heads of 128 x 128 in bf16 at 256, 384 and 512 tokens, with segments and without: 77 and
// 70 us, 77 and 81, 78 and 94, and 79, 88 and 98 with segments where decays are so slow that all chunks behind one count).
int64_t gdr_segment_back(int64_t BH, int64_t dv, int64_t nchunks) {
    const int64_t n = 256 / (BH * ((dv + 63) / 64));
    if (n < 2 || nchunks < 6) return nchunks;
    const int64_t seg = (nchunks + n - 1) / n;
    return seg < 2 ? 2 : seg;
}

}  // namespace selscan

namespace {

// ---------------------------------------------------------------------------
// gated delta rule

enum GdrCall { kFwd, kBwd, kStep };

ss_status check_gdr_dims(const ss_gdr_dims* d, GdrCall call) {
    if (!d) return fail(SS_ERR_INVALID_ARG, "dims is NULL");
    if (d->batch < 1 || d->k_heads < 1 || d->heads < 1 || d->dk < 1 || d->dv < 1 || (call != kStep && d->seqlen < 0))
        return fail(SS_ERR_INVALID_ARG, "batch, heads, dk and dv must be positive, seqlen not negative");
    if (d->heads % d->k_heads) return fail(SS_ERR_INVALID_ARG, "heads %d not a multiple of k_heads %d", d->heads, d->k_heads);
    if (d->dk > 256 || d->dv > 512) return fail(SS_ERR_UNSUPPORTED, "dk %d above 256 or dv %d above 512", d->dk, d->dv);
    if (d->io_dtype != SS_F32 && d->io_dtype != SS_BF16) return fail(SS_ERR_UNSUPPORTED, "io_dtype %d unknown", d->io_dtype);
    // 64 tokens of y, and of the gradients of q and k, lie within 32-bit offsets
    if ((int64_t)d->heads * d->dv > (int64_t(1) << 22) || (int64_t)d->k_heads * d->dk > (int64_t(1) << 22))
        return fail(SS_ERR_UNSUPPORTED, "heads x dv or k_heads x dk above 2^22");
    if (!std::isfinite(d->scale)) return fail(SS_ERR_INVALID_ARG, "scale must be finite");
    if (!(d->eps >= 0.0f) || !std::isfinite(d->eps)) return fail(SS_ERR_INVALID_ARG, "eps must be finite and not negative");
    if (d->reserved != 0) return fail(SS_ERR_INVALID_ARG, "reserved must be 0");
    if (call != kStep && d->seqlen >= (int64_t(1) << 31))
        return fail(SS_ERR_INVALID_ARG, "seqlen %lld not below 2^31", (long long)d->seqlen);
    // one launch holds fewer than 2^32 lanes: 256 a chunk and head, and up to 16 workgroups of them a head
    if (d->batch > INT32_MAX || d->batch * d->heads >= (int64_t(1) << 20))
        return fail(SS_ERR_INVALID_ARG, "batch x heads not below 2^20");
    if (call != kStep && d->batch * d->heads * ceil_div(d->seqlen, SS_GDR_CHUNK) >= (int64_t(1) << 23))
        return fail(SS_ERR_INVALID_ARG, "batch x heads x seqlen too large for one call");
    return SS_OK;
}

size_t ckpt_states(const ss_gdr_dims& d) {
    return (size_t)d.batch * d.heads * (size_t)ceil_div(d.seqlen, SS_GDR_CHUNK) * d.dk * d.dv;
}
size_t ckpt_floats(const ss_gdr_dims& d) { return ckpt_states(d) + (size_t)d.batch * (size_t)d.seqlen * d.heads * d.dv; }

// Per chunk and head: the tokens' factors and the inverse (a triangle, in three bf16 terms or fp32). The forward in
// segments: the states in front of them, what they make of these, and the states behind them. The backward: these of
// gradients, the state's gradient behind every chunk, the gradients of v in fp32, and those of q and k by head of v where heads share them.
struct GdrLayout { size_t co, wT, wS, wV, pq, pk, wE, wM, wF, wX, wQ, wG, total; int64_t seg, nseg; };
GdrLayout gdr_layout(const ss_gdr_dims& d, bool backward) {
    GdrLayout l{};
    if (d.seqlen == 0) return l;
    const size_t n = (size_t)d.batch * d.heads * (size_t)ceil_div(d.seqlen, SS_GDR_CHUNK);
    const size_t rows = (size_t)d.batch * (size_t)d.seqlen * d.heads;
    size_t off = 0;
    auto take = [&](size_t& at, size_t floats) { at = off; off = align256(off + floats * 4); };
    take(l.co, n * 10 * 64);
    take(l.wT, n * ((backward ? selscan::kGdrTri : selscan::kGdrLow) *
                    (d.io_dtype == SS_BF16 ? selscan::kGdrInverseBytes<true> : selscan::kGdrInverseBytes<false>) / 4));
    l.seg = ceil_div(d.seqlen, SS_GDR_CHUNK);
    l.nseg = 1;
    if (!backward) {
        const int64_t chunks = l.seg;
        l.seg = selscan::gdr_segment(d.batch * d.heads, d.dv, chunks, d.io_dtype == SS_BF16 && d.dk <= 128);
        l.nseg = ceil_div(chunks, l.seg);
        if (l.nseg > 1) {
            const size_t ends = (size_t)(l.nseg - 1) * d.batch * d.heads;
            take(l.wE, (size_t)l.nseg * d.batch * d.heads * d.dk * d.dv);
            take(l.wM, ends * d.dk * d.dk);
            take(l.wF, ends);
            take(l.wX, ends * d.dk * d.dv);
            take(l.wQ, (size_t)l.nseg * d.batch * d.heads * (size_t)ceil_div(d.dv, 64) * 4);
        }
    }
    if (backward) {
        l.seg = selscan::gdr_segment_back(d.batch * d.heads, d.dv, l.seg);
        l.nseg = ceil_div(ceil_div(d.seqlen, SS_GDR_CHUNK), l.seg);
        if (l.nseg > 1) {
            const size_t ends = (size_t)(l.nseg - 1) * d.batch * d.heads;
            take(l.wE, ends * d.dk * d.dv);
            take(l.wX, ends * d.dk * d.dv);
            take(l.wQ, (size_t)l.nseg * d.batch * d.heads * (size_t)ceil_div(d.dv, 64) * 4);
        }
        take(l.wS, n * d.dk * d.dv);
        take(l.wV, rows * d.dv);
        take(l.wG, n * 4);
        if (d.heads > d.k_heads) {
            take(l.pq, rows * d.dk);
            take(l.pk, rows * d.dk);
        }
    }
    l.total = off;
    return l;
}

ss_status check_view(const ss_head_view& v, int64_t B, int64_t L, int64_t H, int64_t d, size_t es, const char* name, Range* r) {
    if (!v.p) return fail(SS_ERR_INVALID_ARG, "%s is NULL", name);
    if ((uintptr_t)v.p % es) return fail(SS_ERR_INVALID_ARG, "%s not aligned to its element", name);
    if ((B > 1 && v.batch_stride < 0) || (L > 1 && v.token_stride < 0) || (H > 1 && v.head_stride < 0))
        return fail(SS_ERR_INVALID_ARG, "%s has a negative stride", name);
    const __int128 last = (__int128)(B > 1 ? B - 1 : 0) * v.batch_stride + (__int128)(L > 1 ? L - 1 : 0) * v.token_stride +
                          (__int128)(H > 1 ? H - 1 : 0) * v.head_stride + d;
    if (last > (__int128(1) << 60)) return fail(SS_ERR_INVALID_ARG, "%s spans too many bytes", name);
    *r = Range{v.p, (size_t)last * es, name};
    return SS_OK;
}

// every row of a view starts on 16 bytes and is whole accesses of 16 bytes, 64 tokens within 32-bit offsets
bool view_vec(const ss_head_view& v, int64_t B, int64_t L, int64_t H, int64_t d, int64_t es) {
    const int64_t per = 16 / es;
    return (uintptr_t)v.p % 16 == 0 && d % 8 == 0 && v.token_stride < (int64_t(1) << 24) && (B == 1 || v.batch_stride % per == 0) && (L == 1 || v.token_stride % per == 0) &&
           (H == 1 || v.head_stride % per == 0);
}

// a stride that does not matter is 0, so that no address is made from it
ss_head_view plain(ss_head_view v, int64_t B, int64_t L, int64_t H) {
    if (B == 1) v.batch_stride = 0;
    if (L == 1) v.token_stride = 0;
    if (H == 1) v.head_stride = 0;
    return v;
}

struct GdrInputs { Range q, k, v; };

ss_status check_gdr_args(const ss_gdr_dims& d, const ss_gdr_args* a, GdrCall call, GdrInputs* in, selscan::LaunchGdr* p) {
    if (!a) return fail(SS_ERR_INVALID_ARG, "args is NULL");
    const int64_t B = d.batch, L = call == kStep ? 1 : d.seqlen;
    const int64_t es = (int64_t)io_size(d.io_dtype);
    ss_status s = check_view(a->q, B, L, d.k_heads, d.dk, es, "q", &in->q);
    if (s == SS_OK) s = check_view(a->k, B, L, d.k_heads, d.dk, es, "k", &in->k);
    if (s == SS_OK) s = check_view(a->v, B, L, d.heads, d.dv, es, "v", &in->v);
    if (s != SS_OK) return s;
    if (!a->g || !a->beta) return fail(SS_ERR_INVALID_ARG, "g or beta is NULL");
    if (call != kBwd && !a->y) return fail(SS_ERR_INVALID_ARG, "y is NULL");
    if (call == kStep && !a->state) return fail(SS_ERR_INVALID_ARG, "state is NULL");
    if (call == kBwd && !a->ckpt) return fail(SS_ERR_INVALID_ARG, "ckpt is NULL");
    const Range f4[] = {{a->g, 4, "g"}, {a->beta, 4, "beta"}, {call == kBwd ? nullptr : a->state, 4, "state"},
                        {call == kStep ? nullptr : a->ckpt, 4, "ckpt"}};
    for (const Range& q : f4)
        if ((uintptr_t)q.p & 3u) return fail(SS_ERR_INVALID_ARG, "%s not 4-byte aligned", q.name);
    if (call != kBwd && (uintptr_t)a->y % es) return fail(SS_ERR_INVALID_ARG, "y not aligned to its element");
    p->bf16 = d.io_dtype == SS_BF16;
    p->vec = view_vec(a->q, B, L, d.k_heads, d.dk, es) && view_vec(a->k, B, L, d.k_heads, d.dk, es);
    p->vec_v = L == 1 || a->v.token_stride < (int64_t(1) << 24);
    p->vec_y = d.dv % 4 == 0 && (uintptr_t)a->y % (4 * es) == 0;
    p->vec_state = d.dv % 4 == 0 && (uintptr_t)a->state % 16 == 0;
    p->B = B;
    p->L = L;
    p->nchunks = ceil_div(L, SS_GDR_CHUNK);
    p->H = d.heads; p->Hk = d.k_heads; p->dk = d.dk; p->dv = d.dv;
    p->scale = d.scale; p->eps = d.eps;
    p->q = plain(a->q, B, L, d.k_heads);
    p->k = plain(a->k, B, L, d.k_heads);
    p->v = plain(a->v, B, L, d.heads);
    p->g = a->g; p->beta = a->beta; p->reset = a->reset; p->y = a->y; p->state = a->state;
    if (call != kStep && a->ckpt) {
        p->ckpt = a->ckpt;
        p->ckptX = a->ckpt + ckpt_states(d);
    }
    return SS_OK;
}

void gdr_attach(selscan::LaunchGdr& p, const ss_gdr_dims& d, const GdrLayout& l, void* workspace, bool backward) {
    char* ws = static_cast<char*>(workspace);
    auto at = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
    p.co = at(l.co); p.wT = at(l.wT);
    p.seg = l.seg;
    p.nseg = (int)l.nseg;
    p.wE = at(l.wE); p.wM = at(l.wM); p.wF = at(l.wF); p.wX = at(l.wX);
    p.wQ = reinterpret_cast<uint32_t*>(ws + l.wQ);
    if (backward) {
        p.wS = at(l.wS); p.wV = at(l.wV);
        p.wG = reinterpret_cast<uint32_t*>(ws + l.wG);
        if (d.heads > d.k_heads) { p.part_q = at(l.pq); p.part_k = at(l.pk); }
    }
}

// ---------------------------------------------------------------------------
// the norms around a layer

ss_status check_gnorm_dims(const ss_gnorm_dims* d) {
    if (!d) return fail(SS_ERR_INVALID_ARG, "dims is NULL");
    if (d->rows < 1 || d->cols < 1 || d->group < 1) return fail(SS_ERR_INVALID_ARG, "rows, cols and group must be positive");
    if (d->rows > INT32_MAX) return fail(SS_ERR_INVALID_ARG, "rows %lld not below 2^31", (long long)d->rows);
    if (d->cols > selscan::kGnormMaxCols) return fail(SS_ERR_UNSUPPORTED, "cols %lld above 16384", (long long)d->cols);
    if (d->cols % d->group) return fail(SS_ERR_INVALID_ARG, "group %lld does not divide cols %lld", (long long)d->group, (long long)d->cols);
    if (d->io_dtype != SS_F32 && d->io_dtype != SS_BF16) return fail(SS_ERR_UNSUPPORTED, "io_dtype %d unknown", d->io_dtype);
    if (!(d->eps > 0.0f) || !std::isfinite(d->eps)) return fail(SS_ERR_INVALID_ARG, "eps must be positive and finite");
    return SS_OK;
}

ss_status check_gnorm_args(const ss_gnorm_dims& d, const ss_gnorm_args* a) {
    if (!a) return fail(SS_ERR_INVALID_ARG, "args is NULL");
    if (!a->y || !a->w) return fail(SS_ERR_INVALID_ARG, "y or w is NULL");
    const size_t es = io_size(d.io_dtype);
    const void* io[] = {a->y, a->gate, a->residual};
    for (const void* p : io)
        if ((uintptr_t)p % es) return fail(SS_ERR_INVALID_ARG, "y, gate or residual not aligned to its element");
    const void* f4[] = {a->w, a->scale, a->w_next};
    for (const void* p : f4)
        if ((uintptr_t)p & 3u) return fail(SS_ERR_INVALID_ARG, "w, scale or w_next not 4-byte aligned");
    return SS_OK;
}

selscan::LaunchGnorm gnorm_launch(const ss_gnorm_dims& d, const ss_gnorm_args& a, void* stream) {
    selscan::LaunchGnorm p{};
    p.bf16 = d.io_dtype == SS_BF16;
    p.M = d.rows; p.K = d.cols; p.group = d.group; p.eps = d.eps;
    p.y = a.y; p.gate = a.gate; p.residual = a.residual; p.w = a.w; p.scale = a.scale; p.w_next = a.w_next;
    p.stream = stream;
    return p;
}

template <typename... P>
bool vec16(int64_t cols, int64_t group, const P*... ptrs) {
    bool v = cols % 8 == 0 && group % 8 == 0;
    ((v = v && ((uintptr_t)ptrs & 15u) == 0), ...);
    return v;
}

}  // namespace

extern "C" {

size_t ss_gdr_ckpt_floats(const ss_gdr_dims* dims) {
    return check_gdr_dims(dims, kFwd) == SS_OK ? ckpt_floats(*dims) : 0;
}

size_t ss_gdr_workspace_bytes(const ss_gdr_dims* dims, int backward) {
    return check_gdr_dims(dims, backward ? kBwd : kFwd) == SS_OK ? gdr_layout(*dims, backward != 0).total : 0;
}

ss_status ss_gdr_fwd(const ss_gdr_dims* d, const ss_gdr_args* a, void* workspace, size_t workspace_bytes, void* stream) {
    ss_status s = check_gdr_dims(d, kFwd);
    if (s != SS_OK) return s;
    if (d->seqlen == 0) return a ? SS_OK : fail(SS_ERR_INVALID_ARG, "args is NULL");
    GdrInputs in{};
    selscan::LaunchGdr p{};
    if ((s = check_gdr_args(*d, a, kFwd, &in, &p)) != SS_OK) return s;
    const GdrLayout l = gdr_layout(*d, false);
    if ((s = check_workspace(workspace, workspace_bytes, l.total)) != SS_OK) return s;
    const size_t B = (size_t)d->batch, rows = B * (size_t)d->seqlen, H = (size_t)d->heads;
    const Range ins[] = {in.q, in.k, in.v, {a->g, rows * H * 4, "g"}, {a->beta, rows * H * 4, "beta"}, {a->reset, rows, "reset"}};
    const Range outs[] = {{a->y, rows * H * d->dv * io_size(d->io_dtype), "y"}, {a->state, B * H * d->dk * d->dv * 4, "state"},
                          {a->ckpt, ckpt_floats(*d) * 4, "ckpt"}, {workspace, l.total, "workspace"}};
    if ((s = check_overlaps(outs, 4, ins, 6)) != SS_OK) return s;
    gdr_attach(p, *d, l, workspace, false);
    p.pass = selscan::LaunchGdr::kFwd;
    p.stream = stream;
    return launched(selscan::launch_gdr(p));
}

ss_status ss_gdr_step(const ss_gdr_dims* d, const ss_gdr_args* a, void* stream) {
    ss_status s = check_gdr_dims(d, kStep);
    if (s != SS_OK) return s;
    GdrInputs in{};
    selscan::LaunchGdr p{};
    if ((s = check_gdr_args(*d, a, kStep, &in, &p)) != SS_OK) return s;
    const size_t B = (size_t)d->batch, H = (size_t)d->heads;
    const Range ins[] = {in.q, in.k, in.v, {a->g, B * H * 4, "g"}, {a->beta, B * H * 4, "beta"}, {a->reset, B, "reset"}};
    const Range outs[] = {{a->y, B * H * d->dv * io_size(d->io_dtype), "y"}, {a->state, B * H * d->dk * d->dv * 4, "state"}};
    if ((s = check_overlaps(outs, 2, ins, 6)) != SS_OK) return s;
    p.pass = selscan::LaunchGdr::kStep;
    p.stream = stream;
    return launched(selscan::launch_gdr(p));
}

ss_status ss_gdr_bwd(const ss_gdr_dims* d, const ss_gdr_args* a, const ss_gdr_grads* g, void* workspace, size_t workspace_bytes,
                     void* stream) {
    ss_status s = check_gdr_dims(d, kBwd);
    if (s != SS_OK) return s;
    if (d->seqlen == 0) return fail(SS_ERR_INVALID_ARG, "seqlen must be positive for the gradients");
    GdrInputs in{};
    selscan::LaunchGdr p{};
    if ((s = check_gdr_args(*d, a, kBwd, &in, &p)) != SS_OK) return s;
    if (!g) return fail(SS_ERR_INVALID_ARG, "grads is NULL");
    const struct { const void* p; const char* name; size_t align; } need[] = {
        {g->dy, "dy", io_size(d->io_dtype)}, {g->dq, "dq", io_size(d->io_dtype)}, {g->dk, "dk", io_size(d->io_dtype)},
        {g->dv, "dv", io_size(d->io_dtype)}, {g->dg, "dg", 4}, {g->dbeta, "dbeta", 4}};
    for (const auto& q : need) {
        if (!q.p) return fail(SS_ERR_INVALID_ARG, "%s is NULL", q.name);
        if ((uintptr_t)q.p % q.align) return fail(SS_ERR_INVALID_ARG, "%s not aligned to its element", q.name);
    }
    if (((uintptr_t)g->dstate_final & 3u) || ((uintptr_t)g->dstate_init & 3u))
        return fail(SS_ERR_INVALID_ARG, "dstate_final or dstate_init not 4-byte aligned");
    const GdrLayout l = gdr_layout(*d, true);
    if ((s = check_workspace(workspace, workspace_bytes, l.total)) != SS_OK) return s;
    const size_t B = (size_t)d->batch, rows = B * (size_t)d->seqlen, H = (size_t)d->heads, es = io_size(d->io_dtype);
    const size_t st = B * H * d->dk * d->dv * 4, keys = rows * d->k_heads * d->dk * es, vals = rows * H * d->dv * es;
    const Range ins[] = {in.q, in.k, in.v, {a->g, rows * H * 4, "g"}, {a->beta, rows * H * 4, "beta"}, {a->reset, rows, "reset"},
                         {a->ckpt, ckpt_floats(*d) * 4, "ckpt"}, {g->dy, vals, "dy"}, {g->dstate_final, st, "dstate_final"}};
    const Range outs[] = {{g->dq, keys, "dq"}, {g->dk, keys, "dk"}, {g->dv, vals, "dv"}, {g->dg, rows * H * 4, "dg"},
                          {g->dbeta, rows * H * 4, "dbeta"}, {g->dstate_init, st, "dstate_init"}, {workspace, l.total, "workspace"}};
    if ((s = check_overlaps(outs, 7, ins, 9)) != SS_OK) return s;
    gdr_attach(p, *d, l, workspace, true);
    p.gr = *g;
    p.vec_dy = d->dv % 8 == 0 && (uintptr_t)g->dy % 16 == 0;
    p.vec_ck = d->dv % 4 == 0 && d->dk * d->dv % 4 == 0 && (uintptr_t)a->ckpt % 16 == 0;
    p.vec_dk = d->dk % 4 == 0 && (uintptr_t)g->dq % (4 * es) == 0 && (uintptr_t)g->dk % (4 * es) == 0;
    p.pass = selscan::LaunchGdr::kBwd;
    p.stream = stream;
    return launched(selscan::launch_gdr(p));
}

ss_status ss_gnorm_fwd(const ss_gnorm_dims* d, const ss_gnorm_args* a, void* stream) {
    ss_status st = check_gnorm_dims(d);
    if (st == SS_OK) st = check_gnorm_args(*d, a);
    if (st != SS_OK) return st;
    const size_t es = io_size(d->io_dtype), K = (size_t)d->cols, all = (size_t)d->rows * K * es;
    if (!a->s) return fail(SS_ERR_INVALID_ARG, "s is NULL");
    if (a->w_next && !a->n) return fail(SS_ERR_INVALID_ARG, "n is required with w_next");
    if (!a->w_next && a->n) return fail(SS_ERR_INVALID_ARG, "n given without w_next");
    if ((uintptr_t)a->s % es || (uintptr_t)a->n % es) return fail(SS_ERR_INVALID_ARG, "s or n not aligned to its element");
    const Range ins[] = {{a->s == a->y ? nullptr : a->y, all, "y"}, {a->s == a->gate ? nullptr : a->gate, all, "gate"},
                         {a->s == a->residual ? nullptr : a->residual, all, "residual"}, {a->w, (size_t)d->group * 4, "w"},
                         {a->scale, K * 4, "scale"}, {a->w_next, K * 4, "w_next"}};
    const Range outs[] = {{a->s, all, "s"}, {a->n, all, "n"}};
    if ((st = check_overlaps(outs, 2, ins, 6)) != SS_OK) return st;
    selscan::LaunchGnorm p = gnorm_launch(*d, *a, stream);
    p.s = a->s;
    p.n = a->n;
    p.vec = vec16(d->cols, d->group, a->y, a->gate, a->residual, a->s, a->n, a->w, a->scale, a->w_next);
    return launched(selscan::launch_gnorm(p));
}

size_t ss_gnorm_workspace_bytes(const ss_gnorm_dims* d) {
    return check_gnorm_dims(d) == SS_OK ? align256((size_t)selscan::gnorm_groups(d->rows, d->cols) * 3 * (size_t)d->cols * 4) : 0;
}

ss_status ss_gnorm_bwd(const ss_gnorm_dims* d, const ss_gnorm_args* a, const ss_gnorm_grads* g, void* workspace,
                       size_t workspace_bytes, void* stream) {
    ss_status st = check_gnorm_dims(d);
    if (st == SS_OK) st = check_gnorm_args(*d, a);
    if (st != SS_OK) return st;
    if (!g) return fail(SS_ERR_INVALID_ARG, "grads is NULL");
    if (!g->ds && !g->dn) return fail(SS_ERR_INVALID_ARG, "ds or dn is required");
    if (g->dn && !a->w_next) return fail(SS_ERR_INVALID_ARG, "dn given without w_next");
    const struct { const void* out; const void* in; const char* name; bool io; } outs_of[] = {
        {g->dy, a->y, "dy", true}, {g->dgate, a->gate, "dgate", true}, {g->dresidual, a->residual, "dresidual", true},
        {g->dw, a->w, "dw", false}, {g->dscale, a->scale, "dscale", false}, {g->dw_next, a->w_next, "dw_next", false}};
    const size_t es = io_size(d->io_dtype), K = (size_t)d->cols, all = (size_t)d->rows * K * es;
    for (const auto& q : outs_of) {
        if (q.in && !q.out) return fail(SS_ERR_INVALID_ARG, "%s is NULL", q.name);
        if (!q.in && q.out) return fail(SS_ERR_INVALID_ARG, "%s given without what it is the gradient of", q.name);
        if ((uintptr_t)q.out % (q.io ? es : 4)) return fail(SS_ERR_INVALID_ARG, "%s not aligned to its element", q.name);
    }
    if ((uintptr_t)g->ds % es || (uintptr_t)g->dn % es) return fail(SS_ERR_INVALID_ARG, "ds or dn not aligned to its element");
    const size_t need = ss_gnorm_workspace_bytes(d);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != SS_OK) return st;
    const Range ins[] = {{a->y, all, "y"}, {a->gate, all, "gate"}, {a->residual, all, "residual"}, {a->w, (size_t)d->group * 4, "w"},
                         {a->scale, K * 4, "scale"}, {a->w_next, K * 4, "w_next"}, {g->ds, all, "ds"}, {g->dn, all, "dn"}};
    const Range outs[] = {{g->dy, all, "dy"}, {g->dgate, all, "dgate"}, {g->dresidual, all, "dresidual"}, {g->dw, (size_t)d->group * 4, "dw"},
                          {g->dscale, K * 4, "dscale"}, {g->dw_next, K * 4, "dw_next"}, {workspace, need, "workspace"}};
    if ((st = check_overlaps(outs, 7, ins, 8)) != SS_OK) return st;
    selscan::LaunchGnorm p = gnorm_launch(*d, *a, stream);
    p.back = true;
    p.ds = g->ds; p.dn = g->dn;
    p.dy = g->dy; p.dgate = g->dgate; p.dresidual = g->dresidual;
    p.dw = g->dw; p.dscale = g->dscale; p.dw_next = g->dw_next;
    p.part = static_cast<float*>(workspace);
    p.vec = vec16(d->cols, d->group, a->y, a->gate, a->residual, g->ds, g->dn, g->dy, g->dgate, g->dresidual, a->w, a->scale, a->w_next);
    return launched(selscan::launch_gnorm(p));
}

}  // extern "C"

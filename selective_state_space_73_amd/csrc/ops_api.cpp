// C ABI of the operators around the scan: argument validation, workspace layout, launch
// dispatch. Declared in include/selscan_ops.h. Nothing here touches the device before all
// arguments have been validated, so a rejected call enqueues nothing.
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "ops_internal.h"

namespace {

ss_status fail(ss_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return selscan::set_error(s, buf);
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }
size_t io_size(int dt) { return dt == SS_BF16 ? 2 : 4; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Range { const void* p; size_t bytes; const char* name; };
bool overlap(const Range& a, const Range& b) {
    if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// Every output apart from every input, from every other output and from the workspace.
ss_status check_overlaps(const Range* outs, int n_out, const Range* ins, int n_in) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (overlap(outs[i], ins[j])) return fail(SS_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, ins[j].name);
        for (int j = i + 1; j < n_out; ++j)
            if (overlap(outs[i], outs[j])) return fail(SS_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, outs[j].name);
    }
    return SS_OK;
}

ss_status check_workspace(const void* workspace, size_t given, size_t need) {
    if (need > 0 && (!workspace || given < need))
        return fail(SS_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", given, need);
    if (need > 0 && ((uintptr_t)workspace & 255u)) return fail(SS_ERR_INVALID_ARG, "workspace not 256-byte aligned");
    return SS_OK;
}

// ---------------------------------------------------------------------------
// gated linear recurrence

enum GlrCall { kFwd, kBwd, kStep };

ss_status check_glr_dims(const ss_glr_dims* d, GlrCall call) {
    if (!d) return fail(SS_ERR_INVALID_ARG, "dims is NULL");
    if (d->batch < 1 || d->d < 1 || (call != kStep && d->seqlen < 1))
        return fail(SS_ERR_INVALID_ARG, "batch, seqlen and d must be positive");
    if (d->d > (int64_t(1) << 26)) return fail(SS_ERR_INVALID_ARG, "d %lld above 2^26", (long long)d->d);
    if (d->batch > INT32_MAX) return fail(SS_ERR_INVALID_ARG, "batch %lld not below 2^31", (long long)d->batch);
    if (call != kStep && d->seqlen >= (int64_t(1) << 31))
        return fail(SS_ERR_INVALID_ARG, "seqlen %lld not below 2^31", (long long)d->seqlen);
    if (d->io_dtype != SS_F32 && d->io_dtype != SS_BF16) return fail(SS_ERR_UNSUPPORTED, "io_dtype %d unknown", d->io_dtype);
    if (d->reserved != 0) return fail(SS_ERR_INVALID_ARG, "reserved must be 0");
    const int64_t chunk = call == kBwd ? selscan::glr_bwd_chunk(d->batch, d->seqlen, d->d)
                                       : selscan::glr_fwd_chunk(d->io_dtype == SS_BF16, d->batch, d->seqlen, d->d);
    const int64_t n = call == kStep ? 1 : ceil_div(d->seqlen, chunk);
    const int64_t cols = ceil_div(d->d, selscan::kGlrCols);
    if (d->batch > INT32_MAX / (n * cols)) return fail(SS_ERR_INVALID_ARG, "batch x seqlen x d too large");
    // one launch holds fewer than 2^32 lanes: 1024 a tile where a row is one chunk, 64 in a step
    if (n == 1 && d->batch * cols >= (int64_t(1) << (call == kStep ? 26 : 22)))
        return fail(SS_ERR_INVALID_ARG, "batch %lld too large for one call", (long long)d->batch);
    return SS_OK;
}

// Workspace of the chunked passes: the ticket, one word per chunk and channel (more than one
// chunk), the backward's parts of dA.
struct GlrLayout { int64_t chunk, nchunks; size_t off_slots, off_part, total; };
GlrLayout glr_layout(const ss_glr_dims& d, bool backward) {
    GlrLayout l{};
    l.chunk = backward ? selscan::glr_bwd_chunk(d.batch, d.seqlen, d.d) : selscan::glr_fwd_chunk(d.io_dtype == SS_BF16, d.batch, d.seqlen, d.d);
    l.nchunks = ceil_div(d.seqlen, l.chunk);
    const size_t words = (size_t)l.nchunks * (size_t)d.batch * (size_t)d.d;
    size_t off = 0;
    if (l.nchunks > 1) {
        l.off_slots = 256;
        off = align256(256 + words * sizeof(uint64_t));
    }
    if (backward) {
        l.off_part = off;
        off = align256(off + words * sizeof(float));
    }
    l.total = off;
    return l;
}

// A view's last element must lie at an offset that 62 bits hold, in bytes.
bool view_bytes(const ss_view& v, int64_t B, int64_t L, int64_t D, size_t es, size_t* bytes) {
    const __int128 last = (__int128)(B > 1 ? B - 1 : 0) * v.batch_stride + (__int128)(L > 1 ? L - 1 : 0) * v.token_stride + D;
    if (last > (__int128(1) << 60)) return false;
    *bytes = (size_t)last * es;
    return true;
}

struct GlrInputs { Range x, r, i; bool even; };

ss_status check_glr_args(const ss_glr_dims& d, const ss_glr_args* a, GlrCall call, GlrInputs* in) {
    if (!a) return fail(SS_ERR_INVALID_ARG, "args is NULL");
    const int64_t B = d.batch, L = call == kStep ? 1 : d.seqlen, D = d.d;
    const size_t es = io_size(d.io_dtype);
    const struct { const ss_view* v; Range* r; const char* name; } views[] = {
        {&a->x, &in->x, "x"}, {&a->r, &in->r, "r"}, {&a->i, &in->i, "i"}};
    in->even = D % 2 == 0;
    for (const auto& q : views) {
        if (!q.v->p) return fail(SS_ERR_INVALID_ARG, "%s is NULL", q.name);
        if ((uintptr_t)q.v->p % es) return fail(SS_ERR_INVALID_ARG, "%s not aligned to its element", q.name);
        if ((B > 1 && q.v->batch_stride < 0) || (L > 1 && q.v->token_stride < 0))
            return fail(SS_ERR_INVALID_ARG, "%s has a negative stride", q.name);
        size_t bytes = 0;
        if (!view_bytes(*q.v, B, L, D, es, &bytes)) return fail(SS_ERR_INVALID_ARG, "%s spans too many bytes", q.name);
        *q.r = Range{q.v->p, bytes, q.name};
        if ((uintptr_t)q.v->p % (2 * es) || (B > 1 && q.v->batch_stride % 2) || (L > 1 && q.v->token_stride % 2))
            in->even = false;
    }
    if (!a->A) return fail(SS_ERR_INVALID_ARG, "A is NULL");
    if (call != kBwd && !a->y) return fail(SS_ERR_INVALID_ARG, "y is NULL");
    if (call == kStep && !a->state) return fail(SS_ERR_INVALID_ARG, "state is NULL");
    if (call == kBwd && !a->ckpt) return fail(SS_ERR_INVALID_ARG, "ckpt is NULL");
    const Range f4[] = {{a->A, 4, "A"}, {a->state, 4, "state"}, {a->ckpt, 4, "ckpt"}};
    for (const Range& q : f4) {
        if ((uintptr_t)q.p & 3u) return fail(SS_ERR_INVALID_ARG, "%s not 4-byte aligned", q.name);
        if ((uintptr_t)q.p & 7u) in->even = false;
    }
    if (call != kBwd) {
        if ((uintptr_t)a->y % es) return fail(SS_ERR_INVALID_ARG, "y not aligned to its element");
        if ((uintptr_t)a->y % (2 * es)) in->even = false;
    }
    return SS_OK;
}

selscan::LaunchGlr glr_launch(const ss_glr_dims& d, const ss_glr_args& a, bool even, void* stream) {
    selscan::LaunchGlr p{};
    p.bf16 = d.io_dtype == SS_BF16;
    p.vec = even;
    p.batch = d.batch; p.L = d.seqlen; p.D = d.d;
    p.x = a.x; p.r = a.r; p.i = a.i;
    p.A = a.A; p.reset = a.reset; p.y = a.y; p.state = a.state; p.ckpt = a.ckpt;
    p.nchunks = 1;
    p.stream = stream;
    return p;
}

void glr_attach(selscan::LaunchGlr& p, const GlrLayout& l, void* workspace) {
    char* ws = static_cast<char*>(workspace);
    p.chunk = l.chunk;
    p.nchunks = l.nchunks;
    if (l.nchunks > 1) {
        p.ticket = reinterpret_cast<unsigned*>(ws);
        p.slots = reinterpret_cast<uint64_t*>(ws + l.off_slots);
    }
    p.part = reinterpret_cast<float*>(ws + l.off_part);
}

ss_status launched(hipError_t e) {
    return e == hipSuccess ? SS_OK : fail(SS_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
}

ss_status glr_forward(const ss_glr_dims* d, const ss_glr_args* a, void* workspace, size_t workspace_bytes, void* stream,
                      GlrCall call) {
    GlrInputs in{};
    ss_status s = check_glr_dims(d, call);
    if (s == SS_OK) s = check_glr_args(*d, a, call, &in);
    if (s != SS_OK) return s;
    const GlrLayout l = call == kStep ? GlrLayout{1, 1, 0, 0, 0} : glr_layout(*d, false);
    if ((s = check_workspace(workspace, workspace_bytes, l.total)) != SS_OK) return s;
    const size_t B = (size_t)d->batch, L = call == kStep ? 1 : (size_t)d->seqlen, D = (size_t)d->d;
    const size_t nck = call == kStep ? 0 : (size_t)ceil_div(d->seqlen, SS_GLR_CKPT);
    const Range ins[] = {in.x, in.r, in.i, {a->A, D * 4, "A"}, {a->reset, B * L, "reset"}};
    const Range outs[] = {{a->y, B * L * D * io_size(d->io_dtype), "y"}, {a->state, B * D * 4, "state"},
                          {a->ckpt, B * nck * D * 4, "ckpt"}, {workspace, l.total, "workspace"}};
    if ((s = check_overlaps(outs, 4, ins, 5)) != SS_OK) return s;
    selscan::LaunchGlr p = glr_launch(*d, *a, in.even, stream);
    p.pass = call == kStep ? selscan::LaunchGlr::kStep : selscan::LaunchGlr::kFwd;
    glr_attach(p, l, workspace);
    return launched(selscan::launch_glr(p));
}

// ---------------------------------------------------------------------------
// 8-bit floating point with block scales

constexpr int64_t kMaxGrid = INT32_MAX;

ss_status check_q8_dims(const ss_q8_dims* d, bool norm) {
    if (!d) return fail(SS_ERR_INVALID_ARG, "dims is NULL");
    if (d->rows < 1 || d->cols < 1) return fail(SS_ERR_INVALID_ARG, "rows and cols must be positive");
    if (d->cols > INT32_MAX || d->rows > kMaxGrid) return fail(SS_ERR_INVALID_ARG, "rows or cols too large");
    if (d->rows > INT64_MAX / 16 / d->cols) return fail(SS_ERR_INVALID_ARG, "rows x cols too large");
    if (d->io_dtype != SS_F32 && d->io_dtype != SS_BF16) return fail(SS_ERR_UNSUPPORTED, "io_dtype %d unknown", d->io_dtype);
    if (d->reserved != 0) return fail(SS_ERR_INVALID_ARG, "reserved must be 0");
    if (norm && !(d->eps > 0.0f)) return fail(SS_ERR_INVALID_ARG, "eps must be positive");
    if (norm && d->square != 0) return fail(SS_ERR_INVALID_ARG, "square must be 0 for the norm");
    if (d->square != 0 && d->square != 1) return fail(SS_ERR_INVALID_ARG, "square must be 0 or 1");
    if (d->square && (ceil_div(d->rows, 128) > 65535 || d->cols >= (int64_t(1) << 29)))
        return fail(SS_ERR_INVALID_ARG, "too many squares for one call");
    return SS_OK;
}

// whether a row of 8 elements can be one access wherever it starts
bool q8_vec(const ss_q8_dims& d, std::initializer_list<const void*> io16, const void* q) {
    bool v = d.cols % 8 == 0 && ((uintptr_t)q & 7u) == 0;
    for (const void* p : io16) v = v && ((uintptr_t)p & 15u) == 0;
    return v;
}

ss_status check_gemm_q8_dims(const ss_gemm_q8_dims* d) {
    if (!d) return fail(SS_ERR_INVALID_ARG, "dims is NULL");
    if (d->m < 1 || d->n < 1 || d->k < 1) return fail(SS_ERR_INVALID_ARG, "m, n and k must be positive");
    // rows of one tile are addressed by 32-bit offsets: 256 k < 2^32
    if (d->m > INT32_MAX || d->n > INT32_MAX || d->k > (int64_t(1) << 23)) return fail(SS_ERR_INVALID_ARG, "m, n or k too large");
    if (d->k % 16) return fail(SS_ERR_UNSUPPORTED, "k %lld is not a multiple of 16", (long long)d->k);
    if (d->y_dtype != SS_F32 && d->y_dtype != SS_BF16) return fail(SS_ERR_UNSUPPORTED, "y_dtype %d unknown", d->y_dtype);
    if (d->reserved != 0) return fail(SS_ERR_INVALID_ARG, "reserved must be 0");
    if (ceil_div(d->m, 128) > INT32_MAX / ceil_div(d->n, 128)) return fail(SS_ERR_INVALID_ARG, "m x n too large");
    return SS_OK;
}

}  // namespace

extern "C" {

size_t ss_glr_workspace_bytes(const ss_glr_dims* dims, int backward) {
    if (check_glr_dims(dims, backward ? kBwd : kFwd) != SS_OK) return 0;
    return glr_layout(*dims, backward != 0).total;
}

ss_status ss_glr_fwd(const ss_glr_dims* dims, const ss_glr_args* args, void* workspace, size_t workspace_bytes,
                     void* stream) {
    return glr_forward(dims, args, workspace, workspace_bytes, stream, kFwd);
}

ss_status ss_glr_step(const ss_glr_dims* dims, const ss_glr_args* args, void* stream) {
    return glr_forward(dims, args, nullptr, 0, stream, kStep);
}

ss_status ss_glr_bwd(const ss_glr_dims* dims, const ss_glr_args* args, const ss_glr_grads* grads, void* workspace,
                     size_t workspace_bytes, void* stream) {
    GlrInputs in{};
    ss_status s = check_glr_dims(dims, kBwd);
    if (s == SS_OK) s = check_glr_args(*dims, args, kBwd, &in);
    if (s != SS_OK) return s;
    const ss_glr_grads* g = grads;
    if (!g) return fail(SS_ERR_INVALID_ARG, "grads is NULL");
    const size_t es = io_size(dims->io_dtype);
    const size_t B = (size_t)dims->batch, L = (size_t)dims->seqlen, D = (size_t)dims->d;
    const size_t BLD = B * L * D * es;
    const GlrLayout l = glr_layout(*dims, true);
    const Range ins[] = {in.x, in.r, in.i, {args->A, D * 4, "A"}, {args->reset, B * L, "reset"},
                         {args->ckpt, B * (size_t)ceil_div(dims->seqlen, SS_GLR_CKPT) * D * 4, "ckpt"},
                         {g->dy, BLD, "dy"}, {g->dstate_final, B * D * 4, "dstate_final"}};
    const Range outs[] = {{g->dx, BLD, "dx"}, {g->dr, BLD, "dr"}, {g->di, BLD, "di"}, {g->dA, D * 4, "dA"},
                          {g->dstate_init, B * D * 4, "dstate_init"}, {workspace, l.total, "workspace"}};
    const Range req[] = {{g->dy, es, "dy"}, {g->dx, es, "dx"}, {g->dr, es, "dr"}, {g->di, es, "di"}, {g->dA, 4, "dA"}};
    for (const Range& q : req) {
        if (!q.p) return fail(SS_ERR_INVALID_ARG, "grads.%s is NULL", q.name);
        if ((uintptr_t)q.p % q.bytes) return fail(SS_ERR_INVALID_ARG, "grads.%s not aligned to its element", q.name);
        if (&q != &req[4] && (uintptr_t)q.p % (2 * es)) in.even = false;
    }
    const Range opt[] = {{g->dstate_final, 4, "dstate_final"}, {g->dstate_init, 4, "dstate_init"}};
    for (const Range& q : opt) {
        if ((uintptr_t)q.p & 3u) return fail(SS_ERR_INVALID_ARG, "grads.%s not 4-byte aligned", q.name);
        if ((uintptr_t)q.p & 7u) in.even = false;
    }
    if ((s = check_workspace(workspace, workspace_bytes, l.total)) != SS_OK) return s;
    if ((s = check_overlaps(outs, 6, ins, 8)) != SS_OK) return s;
    selscan::LaunchGlr p = glr_launch(*dims, *args, in.even, stream);
    p.pass = selscan::LaunchGlr::kBwd;
    p.g = *g;
    glr_attach(p, l, workspace);
    return launched(selscan::launch_glr(p));
}

ss_status ss_quant_q8(const ss_q8_dims* dims, const void* x, void* q, float* scale, void* stream) {
    ss_status s = check_q8_dims(dims, false);
    if (s != SS_OK) return s;
    if (!x || !q || !scale) return fail(SS_ERR_INVALID_ARG, "x, q or scale is NULL");
    const size_t es = io_size(dims->io_dtype), M = (size_t)dims->rows, K = (size_t)dims->cols, KB = (K + 127) / 128;
    if ((uintptr_t)x % es || ((uintptr_t)scale & 3u)) return fail(SS_ERR_INVALID_ARG, "x or scale not aligned to its element");
    const Range ins[] = {{x, M * K * es, "x"}};
    const Range outs[] = {{q, M * K, "q"}, {scale, (dims->square ? (M + 127) / 128 : M) * KB * 4, "scale"}};
    if ((s = check_overlaps(outs, 2, ins, 1)) != SS_OK) return s;
    selscan::LaunchQ8 p{};
    p.bf16 = dims->io_dtype == SS_BF16;
    p.square = dims->square != 0;
    p.vec = q8_vec(*dims, {x}, q);
    p.x = x; p.q = static_cast<uint8_t*>(q); p.scale = scale;
    p.M = dims->rows; p.K = dims->cols;
    p.stream = stream;
    return launched(selscan::launch_q8(p));
}

ss_status ss_norm_q8(const ss_q8_dims* dims, const ss_norm_q8_args* a, void* stream) {
    ss_status s = check_q8_dims(dims, true);
    if (s != SS_OK) return s;
    if (!a) return fail(SS_ERR_INVALID_ARG, "args is NULL");
    if (!a->x || !a->w || !a->q || !a->scale) return fail(SS_ERR_INVALID_ARG, "x, w, q or scale is NULL");
    if (a->residual && !a->sum) return fail(SS_ERR_INVALID_ARG, "sum is required with a residual");
    if (!a->residual && a->sum) return fail(SS_ERR_INVALID_ARG, "sum given without a residual");
    const size_t es = io_size(dims->io_dtype), M = (size_t)dims->rows, K = (size_t)dims->cols, KB = (K + 127) / 128;
    const void* io[] = {a->x, a->residual, a->sum};
    for (const void* p : io)
        if ((uintptr_t)p % es) return fail(SS_ERR_INVALID_ARG, "x, residual or sum not aligned to its element");
    if (((uintptr_t)a->w & 3u) || ((uintptr_t)a->scale & 3u)) return fail(SS_ERR_INVALID_ARG, "w or scale not 4-byte aligned");
    const Range ins[] = {{a->x, M * K * es, "x"}, {a->residual, M * K * es, "residual"}, {a->w, K * 4, "w"}};
    const Range outs[] = {{a->q, M * K, "q"}, {a->scale, M * KB * 4, "scale"}};
    const Range sum{a->sum, M * K * es, "sum"};
    if ((s = check_overlaps(outs, 2, ins, 3)) != SS_OK) return s;
    if ((s = check_overlaps(outs, 2, &sum, 1)) != SS_OK) return s;
    for (const Range& r : ins)
        if (overlap(sum, r) && !(a->sum == r.p && r.bytes == sum.bytes && r.p != (const void*)a->w))
            return fail(SS_ERR_INVALID_ARG, "sum overlaps %s (only sum == x or sum == residual is allowed)", r.name);
    selscan::LaunchQ8 p{};
    p.bf16 = dims->io_dtype == SS_BF16;
    p.vec = q8_vec(*dims, {a->x, a->residual, a->sum, a->w}, a->q);
    p.x = a->x; p.res = a->residual; p.w = a->w; p.eps = dims->eps;
    p.q = static_cast<uint8_t*>(a->q); p.scale = a->scale; p.sum = a->sum;
    p.M = dims->rows; p.K = dims->cols;
    p.stream = stream;
    return launched(selscan::launch_q8(p));
}

ss_status ss_gemm_q8(const ss_gemm_q8_dims* dims, const ss_gemm_q8_args* a, void* stream) {
    ss_status s = check_gemm_q8_dims(dims);
    if (s != SS_OK) return s;
    if (!a) return fail(SS_ERR_INVALID_ARG, "args is NULL");
    if (!a->xq || !a->xs || !a->wq || !a->ws || !a->y) return fail(SS_ERR_INVALID_ARG, "xq, xs, wq, ws or y is NULL");
    const void* al[] = {a->xq, a->wq, a->residual, a->y};
    for (const void* p : al)
        if ((uintptr_t)p & 15u) return fail(SS_ERR_INVALID_ARG, "xq, wq, residual and y must be 16-byte aligned");
    if (((uintptr_t)a->xs & 3u) || ((uintptr_t)a->ws & 3u)) return fail(SS_ERR_INVALID_ARG, "xs or ws not 4-byte aligned");
    const size_t M = (size_t)dims->m, N = (size_t)dims->n, K = (size_t)dims->k, KB = (K + 127) / 128;
    const size_t yb = M * N * io_size(dims->y_dtype);
    const Range ins[] = {{a->xq, M * K, "xq"}, {a->xs, M * KB * 4, "xs"}, {a->wq, N * K, "wq"},
                         {a->ws, (N + 127) / 128 * KB * 4, "ws"}, {a->residual == a->y ? nullptr : a->residual, yb, "residual"}};
    const Range y{a->y, yb, "y"};
    if ((s = check_overlaps(&y, 1, ins, 5)) != SS_OK) return s;
    selscan::LaunchGemmQ8 p{};
    p.y_bf16 = dims->y_dtype == SS_BF16;
    p.xq = static_cast<const uint8_t*>(a->xq); p.xs = a->xs;
    p.wq = static_cast<const uint8_t*>(a->wq); p.ws = a->ws;
    p.R = a->residual; p.Y[0] = a->y; p.Y[1] = nullptr;
    p.split = dims->n; p.M = dims->m; p.N = dims->n; p.K = dims->k;
    p.stream = stream;
    return launched(selscan::launch_gemm_q8(p));
}

}  // extern "C"

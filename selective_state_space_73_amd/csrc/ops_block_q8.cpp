// Host pipeline of the block with 8-bit projections (ss_block_q8_fwd / ss_block_q8_step).
//
// The block of ss_block_fwd, with its two wide projections as 8-bit products:
//   xq = e4m3 of RMSNorm(x) * norm_w           (norm and rounding in one pass over x)
//   xi, z = xq W_in^T                            (fp32, one launch into two matrices)
//   u, delta, B, C, the scan: as in the block, fp32 activations
//   out = x + e4m3(y) W_out^T                  (y rounded in one pass, residual in the epilogue)
// A decode step reads W_in and W_out once, which is most of what it reads: a byte a weight
// instead of two. x_proj and dt_proj stay in the I/O dtype: they are a few hundredths of the
// block's weights, and the step size and the decay leave through an exponential.
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "ops_internal.h"
#include "selscan_internal.h"

namespace {

ss_status fail(ss_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return selscan::set_error(s, buf);
}

int64_t blocks(int64_t n) { return (n + 127) / 128; }

// the scan inside the block: fp32 activations whatever the block's I/O dtype
ss_dims scan_dims(const ss_block_dims& d, bool step) {
    ss_dims s{};
    s.batch = d.batch;
    s.seqlen = step ? 1 : d.seqlen;
    s.d_inner = d.d_inner;
    s.d_state = d.d_state;
    s.d_conv = d.d_conv;
    s.io_dtype = SS_F32;
    s.discretization = d.discretization;
    return s;
}

ss_status check_dims(const ss_block_dims* d, bool step) {
    if (!d) return fail(SS_ERR_INVALID_ARG, "dims is NULL");
    if (d->batch < 1 || (!step && d->seqlen < 1) || d->d_model < 1 || d->d_inner < 1 || d->dt_rank < 1)
        return fail(SS_ERR_INVALID_ARG, "block sizes must be positive");
    if (d->d_model > (int64_t(1) << 20) || d->d_inner > (int64_t(1) << 23) || d->dt_rank > 4096)
        return fail(SS_ERR_INVALID_ARG, "d_model, d_inner or dt_rank out of range");
    if (d->d_model % 16 || d->d_inner % 16)
        return fail(SS_ERR_UNSUPPORTED, "d_model %lld or d_inner %lld is not a multiple of 16", (long long)d->d_model,
                    (long long)d->d_inner);
    if (!(d->norm_eps > 0.0f)) return fail(SS_ERR_INVALID_ARG, "norm_eps must be positive");
    if (d->d_conv != 4) return fail(SS_ERR_UNSUPPORTED, "d_conv %d: only 4 is built", d->d_conv);
    if (d->io_dtype != SS_F32 && d->io_dtype != SS_BF16) return fail(SS_ERR_UNSUPPORTED, "io_dtype %d unknown", d->io_dtype);
    const int64_t L = step ? 1 : d->seqlen, wide = 2 * d->d_inner > d->d_model ? 2 * d->d_inner : d->d_model;
    // (the small projections' grids have a row of 64 tokens per y)
    if (d->batch > INT32_MAX / L || d->batch * L > 65535 * 64 || blocks(d->batch * L) > INT32_MAX / blocks(wide))
        return fail(SS_ERR_INVALID_ARG, "batch x seqlen too large for these widths");
    const ss_dims sd = scan_dims(*d, step);
    return selscan::validate_dims(&sd, step);
}

struct Layout { size_t xq, xs, xi, z, u, dr, bm, cm, delta, y, yq, ys, scan, part, total; };

Layout layout(const ss_block_dims& d, bool step) {
    Layout l{};
    const int64_t M = d.batch * (step ? 1 : d.seqlen), dm = d.d_model, di = d.d_inner, N = d.d_state, R = d.dt_rank;
    size_t off = 0;
    auto take = [&](size_t bytes) { const size_t o = off; off = (off + bytes + 255) & ~size_t(255); return o; };
    auto rows = [&](int64_t n, size_t es) { return take((size_t)M * (size_t)n * es); };
    l.xq = rows(dm, 1); l.xs = rows(blocks(dm), 4);
    l.xi = rows(di, 4); l.z = rows(di, 4); l.u = rows(di, 4);
    l.dr = rows(R, 4); l.bm = rows(N, 4); l.cm = rows(N, 4);
    l.delta = rows(di, 4); l.y = rows(di, 4);
    l.yq = rows(di, 1); l.ys = rows(blocks(di), 4);
    const ss_dims sd = scan_dims(d, step);
    l.scan = take(step ? 0 : ss_workspace_bytes(&sd));
    const bool bf16 = d.io_dtype == SS_BF16;             // fp32 partials of the projections that split K
    const size_t px = selscan::gemm_plan(M, R + 2 * N, di, bf16).part_bytes, pd = selscan::gemm_plan(M, di, R, bf16).part_bytes;
    l.part = take(px > pd ? px : pd);
    l.total = off;
    return l;
}

struct Range { const void* p; size_t bytes; const char* name; };
bool overlap(const Range& a, const Range& b) {
    if (!a.p || !b.p) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

ss_status check(const ss_block_dims& d, const ss_block_q8_weights* q, const void* x, const void* out,
                const float* ssm_state, const float* conv_state, const void* workspace, size_t workspace_bytes, bool step) {
    if (!q) return fail(SS_ERR_INVALID_ARG, "weights is NULL");
    const ss_block_weights& w = q->w;
    const struct { const void* p; const char* name; unsigned align; } req[] = {
        {x, "x", 16}, {out, "out", 16}, {w.W_in, "W_in", 16}, {w.W_x, "W_x", 16}, {w.W_dt, "W_dt", 16}, {w.W_out, "W_out", 16},
        {q->S_in, "S_in", 4}, {q->S_out, "S_out", 4}, {w.norm_w, "norm_w", 4}, {w.conv_w, "conv_w", 4}, {w.A, "A", 4}};
    for (const auto& r : req) {
        if (!r.p) return fail(SS_ERR_INVALID_ARG, "%s is NULL", r.name);
        if ((uintptr_t)r.p % r.align) return fail(SS_ERR_INVALID_ARG, "%s not %u-byte aligned", r.name, r.align);
    }
    if (step && (!ssm_state || !conv_state)) return fail(SS_ERR_INVALID_ARG, "a step needs both states");
    const void* f4[] = {w.conv_b, w.dt_bias, w.Dskip, conv_state};
    for (const void* p : f4)
        if ((uintptr_t)p & 3u) return fail(SS_ERR_INVALID_ARG, "conv_b, dt_bias, Dskip or conv_state not 4-byte aligned");
    if ((uintptr_t)ssm_state & 15u) return fail(SS_ERR_INVALID_ARG, "ssm_state not 16-byte aligned");
    const Layout l = layout(d, step);
    if (!workspace || workspace_bytes < l.total)
        return fail(SS_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", workspace_bytes, l.total);
    if ((uintptr_t)workspace & 255u) return fail(SS_ERR_INVALID_ARG, "workspace not 256-byte aligned");
    const size_t es = d.io_dtype == SS_BF16 ? 2 : 4, B = (size_t)d.batch, M = B * (size_t)(step ? 1 : d.seqlen);
    const size_t dm = (size_t)d.d_model, di = (size_t)d.d_inner, N = (size_t)d.d_state, R = (size_t)d.dt_rank;
    const Range outs[] = {{out, M * dm * es, "out"}, {ssm_state, B * di * N * 4, "ssm_state"},
                          {conv_state, B * di * 12, "conv_state"}, {workspace, l.total, "workspace"}};
    const size_t KM = (size_t)blocks(d.d_model), KI = (size_t)blocks(d.d_inner);
    const Range ins[] = {{x == out ? nullptr : x, M * dm * es, "x"}, {w.W_in, 2 * di * dm, "W_in"}, {w.W_out, dm * di, "W_out"},
                         {q->S_in, (size_t)blocks(2 * d.d_inner) * KM * 4, "S_in"}, {q->S_out, KM * KI * 4, "S_out"},
                         {w.W_x, (R + 2 * N) * di * es, "W_x"}, {w.W_dt, di * R * es, "W_dt"}, {w.norm_w, dm * 4, "norm_w"},
                         {w.conv_w, di * 16, "conv_w"}, {w.conv_b, di * 4, "conv_b"}, {w.dt_bias, di * 4, "dt_bias"},
                         {w.A, di * N * 4, "A"}, {w.Dskip, di * 4, "Dskip"}};
    for (size_t i = 0; i < 4; ++i) {
        for (const Range& r : ins)
            if (overlap(outs[i], r)) return fail(SS_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, r.name);
        for (size_t j = i + 1; j < 4; ++j)
            if (overlap(outs[i], outs[j])) return fail(SS_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, outs[j].name);
    }
    return SS_OK;
}

ss_status run(const ss_block_dims* d, const ss_block_q8_weights* q, const void* x, void* out, float* ssm_state,
              float* conv_state, void* workspace, size_t workspace_bytes, void* stream, bool step) {
    ss_status s = check_dims(d, step);
    if (s == SS_OK) s = check(*d, q, x, out, ssm_state, conv_state, workspace, workspace_bytes, step);
    if (s != SS_OK) return s;
    const ss_block_weights& w = q->w;
    const Layout l = layout(*d, step);
    char* ws = static_cast<char*>(workspace);
    auto at = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
    const bool bf16 = d->io_dtype == SS_BF16;
    const int64_t L = step ? 1 : d->seqlen, M = d->batch * L, dm = d->d_model, di = d->d_inner, N = d->d_state, R = d->dt_rank;
    hipError_t e;
    auto failed = [&](const char* what) { return fail(SS_ERR_HIP, "%s launch failed: %s", what, hipGetErrorString(e)); };

    selscan::LaunchQ8 n{};
    n.bf16 = bf16;
    n.vec = ((uintptr_t)w.norm_w & 15u) == 0;            // rows of x and q are whole 16-byte pieces
    n.x = x; n.w = w.norm_w; n.eps = d->norm_eps;
    n.q = reinterpret_cast<uint8_t*>(ws + l.xq); n.scale = at(l.xs);
    n.M = M; n.K = dm; n.stream = stream;
    if ((e = selscan::launch_q8(n)) != hipSuccess) return failed("norm");

    selscan::LaunchGemmQ8 p{};
    p.xq = n.q; p.xs = n.scale;
    p.wq = static_cast<const uint8_t*>(w.W_in); p.ws = q->S_in;
    p.Y[0] = at(l.xi); p.Y[1] = at(l.z); p.split = di;
    p.M = M; p.N = 2 * di; p.K = dm; p.stream = stream;
    if ((e = selscan::launch_gemm_q8(p)) != hipSuccess) return failed("input projection");

    selscan::LaunchBlockOps c{};
    c.stream = stream;
    c.in = at(l.xi); c.out = at(l.u); c.conv_w = w.conv_w; c.conv_b = w.conv_b; c.hist = conv_state;
    c.cols = (int)di; c.L = L; c.batch = d->batch;
    c.op = step ? selscan::LaunchBlockOps::kConvStep : selscan::LaunchBlockOps::kConvSilu;
    if ((e = selscan::launch_block_op(c)) != hipSuccess) return failed("conv");
    c.op = selscan::LaunchBlockOps::kConvHistory;
    if (!step && conv_state && (e = selscan::launch_block_op(c)) != hipSuccess) return failed("conv history");

    selscan::LaunchGemm g{};
    g.bf16 = bf16;
    g.X = at(l.u); g.W = w.W_x; g.Y[0] = at(l.dr); g.Y[1] = at(l.bm); g.Y[2] = at(l.cm);
    g.cols[0] = R; g.cols[1] = g.cols[2] = N;
    g.M = M; g.N = R + 2 * N; g.K = di; g.part = at(l.part); g.stream = stream;
    if ((e = selscan::launch_gemm(g)) != hipSuccess) return failed("x_proj");
    g.X = at(l.dr); g.W = w.W_dt; g.Y[0] = at(l.delta); g.Y[1] = g.Y[2] = nullptr;
    g.cols[0] = di; g.cols[1] = g.cols[2] = 0;
    g.N = di; g.K = R;
    if ((e = selscan::launch_gemm(g)) != hipSuccess) return failed("dt_proj");

    const ss_dims sd = scan_dims(*d, step);
    ss_args a{};
    a.x = at(l.u); a.delta = at(l.delta); a.delta_bias = w.dt_bias; a.A = w.A; a.B = at(l.bm); a.C = at(l.cm);
    a.Dskip = w.Dskip; a.z = at(l.z); a.y = at(l.y); a.ssm_state = ssm_state;
    s = step ? ss_step(&sd, &a, stream) : ss_conv_scan_fwd(&sd, &a, ws + l.scan, ss_workspace_bytes(&sd), stream);
    if (s != SS_OK) return s;

    selscan::LaunchQ8 r{};
    r.vec = true;                                        // fp32 rows of a multiple of 16, aligned in the workspace
    r.x = at(l.y); r.q = reinterpret_cast<uint8_t*>(ws + l.yq); r.scale = at(l.ys);
    r.M = M; r.K = di; r.stream = stream;
    if ((e = selscan::launch_q8(r)) != hipSuccess) return failed("rounding");

    p.y_bf16 = bf16;
    p.xq = r.q; p.xs = r.scale;
    p.wq = static_cast<const uint8_t*>(w.W_out); p.ws = q->S_out;
    p.R = x; p.Y[0] = out; p.Y[1] = nullptr;
    p.split = p.N = dm; p.K = di;
    if ((e = selscan::launch_gemm_q8(p)) != hipSuccess) return failed("output projection");
    return SS_OK;
}

}  // namespace

extern "C" {

size_t ss_block_q8_workspace_bytes(const ss_block_dims* dims, int step) {
    if (check_dims(dims, step != 0) != SS_OK) return 0;
    return layout(*dims, step != 0).total;
}

ss_status ss_block_q8_fwd(const ss_block_dims* dims, const ss_block_q8_weights* weights, const void* x, void* out,
                          float* ssm_state, float* conv_state, void* workspace, size_t workspace_bytes, void* stream) {
    return run(dims, weights, x, out, ssm_state, conv_state, workspace, workspace_bytes, stream, false);
}

ss_status ss_block_q8_step(const ss_block_dims* dims, const ss_block_q8_weights* weights, const void* x, void* out,
                           float* ssm_state, float* conv_state, void* workspace, size_t workspace_bytes, void* stream) {
    return run(dims, weights, x, out, ssm_state, conv_state, workspace, workspace_bytes, stream, true);
}

}  // extern "C"

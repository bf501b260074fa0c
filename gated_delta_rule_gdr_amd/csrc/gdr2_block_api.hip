// gdr2_block_api.hip -- the C ABI of the operators around the mixer (layer norm, gated linear
// recurrence, sliding-window attention and its decode): host-side validation, then launch.
// Nothing here touches device memory before every check has passed, and every size is bounded
// before a product that depends on it is formed.
#include "gdr2.h"

#include <hip/hip_runtime.h>

#include "gdr2_block_kernels.hpp"
#include "gdr2_checks.hpp"

namespace {

constexpr int64_t kMaxInt = ((int64_t)1 << 31) - 1;   // counts that the kernels hold as ints

bool dtype_ok(gdr2_dtype dt) { return dt == GDR2_F32 || dt == GDR2_BF16; }
size_t esize(gdr2_dtype dt) { return dt == GDR2_F32 ? 4 : 2; }

template <size_t N>
bool all_aligned(const void* const (&ptrs)[N]) {
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return false;
    return true;
}
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

gdr2_status status_of(hipError_t e) { return e == hipSuccess ? GDR2_OK : GDR2_E_HIP; }

// ------------------------------------------------------------------ layer norm
gdr2_status check_norm(int64_t rows, int64_t D) {
    if (rows < 0 || D < 0 || rows > kMaxInt) return GDR2_E_SHAPE;
    if (D < 8 || D > gdr2::kNormMaxD || D % 8) return GDR2_E_UNSUPPORTED;
    return GDR2_OK;
}

// ------------------------------------------------------------------ gated linear recurrence
// Afterwards B * T * D <= 2^50 and one batch row's segments fit a launch.
gdr2_status check_glr(int64_t B, int64_t T, int64_t D) {
    if (B < 0 || T < 0 || D < 0 || T > ((int64_t)1 << 37) || D > ((int64_t)1 << 30)) return GDR2_E_SHAPE;
    if (D < 8 || D % 8) return GDR2_E_UNSUPPORTED;
    const int64_t nseg = gdr2::glr_segments(T, gdr2::kGlrBwdSeg), strips = gdr2::glr_strips(D);
    if (!prod_le(B, strips, kMaxInt) || !prod_le(B * strips, nseg, kMaxInt)) return GDR2_E_SHAPE;
    // (the backward has up to twice the segments and half the threads)
    if (!prod_le(strips, gdr2::glr_segments(T, gdr2::kGlrFwdSeg), gdr2::max_workgroups(gdr2::kGlrFwdThreads))) return GDR2_E_SHAPE;
    return GDR2_OK;
}
struct GlrWs {
    size_t states, pub, ticket, total;  // offsets; the forward's layout (the backward has no states)
};
GlrWs glr_layout(int64_t B, int64_t T, int64_t D, bool with_states) {
    const size_t nbwd = gdr2::glr_segments(T, gdr2::kGlrBwdSeg), ch = gdr2::glr_strips(D) * gdr2::kGlrCh;
    const size_t nseg = with_states ? gdr2::glr_segments(T, gdr2::kGlrFwdSeg) : nbwd;
    GlrWs w{};
    size_t off = 0;
    auto take = [&](size_t n) { const size_t o = off; off += round_up(n, 256); return o; };
    w.states = take(with_states ? (size_t)B * nbwd * D * 4 : 0);
    w.pub = take(nseg > 1 ? (size_t)B * (nseg + nseg / gdr2::kGlrGroup) * ch * 8 : 0);
    w.ticket = take(nseg > 1 ? 4 : 0);
    w.total = off;
    return w;
}

// ------------------------------------------------------------------ sliding-window attention
gdr2_status check_heads(int64_t H, int64_t Hkv, int64_t d, int64_t window, int64_t sinks) {
    if (H < 0 || Hkv < 0 || d < 0 || H > 32768) return GDR2_E_SHAPE;  // a token's row stays below 2^24 + 1 bytes
    if (!dims_ok(d)) return GDR2_E_UNSUPPORTED;
    if (H > 0 && (Hkv == 0 || H % Hkv)) return GDR2_E_SHAPE;
    if (H == 0 && Hkv != 0) return GDR2_E_SHAPE;
    if (window < 1 || sinks < 0 || sinks > gdr2::kSwaMaxSinks) return GDR2_E_VALUE;
    return GDR2_OK;
}
bool scale_ok(float s) { return s > 0.f && s < 1e30f; }
// Afterwards B * H <= 2^22, B * T * H <= 2^31 rows, and the launches of 256 threads fit: a workgroup per 128 queries or
// keys of a head, and one per key/value head for the sinks' far queries.  (Only launches of a few hundred such
// workgroups are cut finer.)
gdr2_status check_swa(int64_t B, int64_t T, int64_t H, int64_t Hkv, int64_t d, int64_t window, int64_t sinks) {
    const gdr2_status st = check_heads(H, Hkv, d, window, sinks);
    if (st != GDR2_OK) return st;
    if (B < 0 || T < 0 || T > ((int64_t)1 << 30)) return GDR2_E_SHAPE;
    if (!prod_le(B, H, (int64_t)1 << 22) || !prod_le(B * H, (T + 127) / 128 + 1, gdr2::max_workgroups(256))) return GDR2_E_SHAPE;
    return GDR2_OK;
}
gdr2::SwaParams swa_params(int64_t B, int64_t T, int64_t H, int64_t Hkv, int64_t d, int64_t window, int64_t sinks,
                           float scale, const void* q, const void* k, const void* v, const int32_t* lengths) {
    gdr2::SwaParams p{};
    p.B = (int)B; p.H = (int)H; p.Hkv = (int)Hkv; p.d = (int)d; p.sinks = (int)sinks;
    p.T = (int)T; p.window = (int)(window < T ? window : T);
    p.scale = scale; p.q = q; p.k = k; p.v = v; p.lengths = lengths;
    return p;
}
struct SwaBwdWs {
    size_t delta, sinks, keys, total;
    gdr2::SwaCut cut;
};
SwaBwdWs swa_bwd_layout(int64_t B, int64_t T, int64_t H, int64_t Hkv, int64_t d, int64_t window, int64_t sinks) {
    SwaBwdWs w{};
    if (B == 0 || T == 0 || H == 0) return w;
    w.cut = gdr2::swa_cut(B, T, H, Hkv, d, window < T ? window : T, (int)sinks);
    size_t off = 0;
    auto take = [&](size_t n) { const size_t o = off; off += round_up(n, 256); return o; };
    w.delta = take((size_t)B * H * T * 4);
    w.sinks = take((size_t)w.cut.pieces * B * Hkv * 2 * gdr2::kSwaMaxSinks * d * 4);
    w.keys = take((size_t)w.cut.splits * 2 * B * w.cut.part_rows * Hkv * d * 4);
    w.total = off;
    return w;
}
// The backward's last launch: four channels of every reduced row per thread.
gdr2_status check_swa_bwd(int64_t B, int64_t T, int64_t H, int64_t Hkv, int64_t d, int64_t window, int64_t sinks) {
    const gdr2_status st = check_swa(B, T, H, Hkv, d, window, sinks);
    if (st != GDR2_OK || B == 0 || T == 0 || H == 0) return st;
    const int64_t rows = gdr2::swa_cut(B, T, H, Hkv, d, window < T ? window : T, (int)sinks).part_rows;
    return prod_le(B * Hkv, rows * (d / 4), gdr2::max_workgroups(256) * 256) ? GDR2_OK : GDR2_E_SHAPE;
}
gdr2_status check_decode(int64_t N, int64_t H, int64_t Hkv, int64_t d, int64_t window, int64_t sinks) {
    const gdr2_status st = check_heads(H, Hkv, d, window, sinks);
    if (st != GDR2_OK) return st;
    if (N < 0 || window > ((int64_t)1 << 30)) return GDR2_E_SHAPE;
    // at most N * H jobs, each a workgroup (512 in parts where there are fewer); launches take whole sequences
    if (!prod_le(N, H, ((int64_t)1 << 30)) || !prod_le(N * Hkv, window + sinks, (int64_t)1 << 33)) return GDR2_E_SHAPE;
    return GDR2_OK;
}
int64_t decode_jobs(int64_t N, int64_t H, int64_t Hkv) { return Hkv ? N * Hkv * ((H / Hkv + 15) / 16) : 0; }
int decode_splits(int64_t N, int64_t H, int64_t Hkv, int64_t window, int64_t sinks) {
    return gdr2::swa_decode_splits(N, Hkv, Hkv ? (H / Hkv + 15) / 16 : 0, window + sinks);
}

}  // namespace

extern "C" {

gdr2_status gdr2_layer_norm_fwd(int64_t rows, int64_t D, gdr2_dtype dt, const void* x,
                                const float* weight, const float* bias, float eps, void* y,
                                float* mean, float* rstd, void* stream) {
    if (!dtype_ok(dt)) return GDR2_E_DTYPE;
    const gdr2_status st = check_norm(rows, D);
    if (st != GDR2_OK) return st;
    if (!(eps > 0.f) || !(eps < 1e30f)) return GDR2_E_VALUE;
    if (rows == 0) return GDR2_OK;
    if (!x || !weight || !y) return GDR2_E_NULL;
    if (!all_aligned({x, weight, bias, y}) || !aligned4(mean) || !aligned4(rstd)) return GDR2_E_ALIGN;
    const size_t n = (size_t)rows * D * esize(dt), w = (size_t)D * 4, r = (size_t)rows * 4;
    const Range ins[] = {{x, n}, {weight, w}, {bias, w}}, outs[] = {{y, n}, {mean, r}, {rstd, r}};
    if (any_alias(outs, 3, ins, 3)) return GDR2_E_ALIAS;
    gdr2::NormParams p{};
    p.rows = rows; p.D = (int)D; p.eps = eps; p.x = x; p.weight = weight; p.bias = bias; p.y = y;
    p.mean = mean; p.rstd = rstd;
    return status_of(gdr2::norm_dispatch(dt == GDR2_BF16, false, p, (hipStream_t)stream));
}

size_t gdr2_layer_norm_bwd_workspace_bytes(int64_t rows, int64_t D) {
    if (check_norm(rows, D) != GDR2_OK) return 0;
    return (size_t)gdr2::norm_bwd_blocks(rows, (int)D) * 2 * D * sizeof(float);
}

gdr2_status gdr2_layer_norm_bwd(int64_t rows, int64_t D, gdr2_dtype dt, const void* x,
                                const float* weight, const float* mean, const float* rstd,
                                const void* dy, void* dx, float* dweight, float* dbias,
                                void* workspace, size_t workspace_bytes, void* stream) {
    if (!dtype_ok(dt)) return GDR2_E_DTYPE;
    const gdr2_status st = check_norm(rows, D);
    if (st != GDR2_OK) return st;
    if (!dweight) return GDR2_E_NULL;
    if (rows > 0 && (!x || !weight || !mean || !rstd || !dy || !dx)) return GDR2_E_NULL;
    if (!all_aligned({x, weight, dy, dx, dweight, dbias, workspace}) || !aligned4(mean) || !aligned4(rstd)) return GDR2_E_ALIGN;
    const size_t need = gdr2_layer_norm_bwd_workspace_bytes(rows, D);
    if (rows > 0 && (!workspace || workspace_bytes < need)) return GDR2_E_WORKSPACE;
    const size_t n = (size_t)rows * D * esize(dt), w = (size_t)D * 4, r = (size_t)rows * 4;
    const Range ins[] = {{x, n}, {weight, w}, {mean, r}, {rstd, r}, {dy, n}};
    const Range outs[] = {{dx, n}, {dweight, w}, {dbias, w}, {workspace, need}};
    if (any_alias(outs, 4, ins, 5)) return GDR2_E_ALIAS;
    gdr2::NormParams p{};
    p.rows = rows; p.D = (int)D; p.x = x; p.weight = weight; p.mean = (float*)mean; p.rstd = (float*)rstd;
    p.dy = dy; p.dx = dx; p.dweight = dweight; p.dbias = dbias; p.part = (float*)workspace;
    return status_of(gdr2::norm_dispatch(dt == GDR2_BF16, true, p, (hipStream_t)stream));
}

size_t gdr2_glr_fwd_workspace_bytes(int64_t B, int64_t T, int64_t D) {
    return check_glr(B, T, D) == GDR2_OK ? glr_layout(B, T, D, true).total : 0;
}
size_t gdr2_glr_bwd_workspace_bytes(int64_t B, int64_t T, int64_t D) {
    return check_glr(B, T, D) == GDR2_OK ? glr_layout(B, T, D, false).total : 0;
}

static gdr2::GlrParams glr_params(int64_t B, int64_t T, int64_t D, const void* x, const float* la,
                                  int seg, const GlrWs& w, void* ws) {
    gdr2::GlrParams p{};
    p.B = (int)B; p.T = T; p.D = D; p.x = x; p.la = la;
    p.nseg = (int)gdr2::glr_segments(T, seg);
    p.nstrip = (int)gdr2::glr_strips(D);
    p.pub = (unsigned long long*)((char*)ws + w.pub);
    p.ticket = (unsigned*)((char*)ws + w.ticket);
    return p;
}

gdr2_status gdr2_glr_fwd(int64_t B, int64_t T, int64_t D, gdr2_dtype dt, const void* x,
                         const float* log_a, const float* h0, void* h, float* h_T,
                         void* workspace, size_t workspace_bytes, void* stream) {
    if (!dtype_ok(dt)) return GDR2_E_DTYPE;
    const gdr2_status st = check_glr(B, T, D);
    if (st != GDR2_OK) return st;
    if (B == 0) return GDR2_OK;
    if (T > 0 && (!x || !log_a || !h)) return GDR2_E_NULL;
    if (!all_aligned({x, log_a, h0, h, h_T, workspace})) return GDR2_E_ALIGN;
    const GlrWs w = glr_layout(B, T, D, true);
    if (!workspace || workspace_bytes < w.total) return GDR2_E_WORKSPACE;
    const size_t n = (size_t)B * T * D, s = (size_t)B * D * 4;
    const Range ins[] = {{x, n * esize(dt)}, {log_a, n * 4}, {h0, s}};
    const Range outs[] = {{h, n * esize(dt)}, {h_T, s}, {workspace, w.total}};
    if (any_alias(outs, 3, ins, 3)) return GDR2_E_ALIAS;
    gdr2::GlrParams p = glr_params(B, T, D, x, log_a, gdr2::kGlrFwdSeg, w, workspace);
    p.h0 = h0; p.h = h; p.hT = h_T; p.states = (float*)((char*)workspace + w.states);
    return status_of(gdr2::glr_dispatch(dt == GDR2_BF16, false, p, (hipStream_t)stream));
}

gdr2_status gdr2_glr_bwd(int64_t B, int64_t T, int64_t D, gdr2_dtype dt, const void* x,
                         const float* log_a, const void* fwd_workspace, size_t fwd_workspace_bytes,
                         const void* dh, const float* dh_T, void* dx, float* dlog_a, float* dh0,
                         void* workspace, size_t workspace_bytes, void* stream) {
    if (!dtype_ok(dt)) return GDR2_E_DTYPE;
    const gdr2_status st = check_glr(B, T, D);
    if (st != GDR2_OK) return st;
    if (B == 0) return GDR2_OK;
    if (T > 0 && (!x || !log_a || !dh || !dx || !dlog_a)) return GDR2_E_NULL;
    if (!all_aligned({x, log_a, fwd_workspace, dh, dh_T, dx, dlog_a, dh0, workspace})) return GDR2_E_ALIGN;
    const GlrWs f = glr_layout(B, T, D, true), w = glr_layout(B, T, D, false);
    if (!fwd_workspace || fwd_workspace_bytes < f.total) return GDR2_E_WORKSPACE;
    if (w.total > 0 && (!workspace || workspace_bytes < w.total)) return GDR2_E_WORKSPACE;
    const size_t n = (size_t)B * T * D, s = (size_t)B * D * 4;
    const Range ins[] = {{x, n * esize(dt)}, {log_a, n * 4}, {fwd_workspace, f.total}, {dh, n * esize(dt)}, {dh_T, s}};
    const Range outs[] = {{dx, n * esize(dt)}, {dlog_a, n * 4}, {dh0, s}, {workspace, w.total}};
    if (any_alias(outs, 4, ins, 5)) return GDR2_E_ALIAS;
    gdr2::GlrParams p = glr_params(B, T, D, x, log_a, gdr2::kGlrBwdSeg, w, workspace);
    p.states = (float*)((char*)fwd_workspace + f.states);
    p.dh = dh; p.dhT = dh_T; p.dx = dx; p.dla = dlog_a; p.dh0 = dh0;
    return status_of(gdr2::glr_dispatch(dt == GDR2_BF16, true, p, (hipStream_t)stream));
}

gdr2_status gdr2_glr_step(int64_t N, int64_t D, gdr2_dtype dt, const void* x, const float* log_a,
                          const float* h_in, float* h_out, void* h, void* stream) {
    if (!dtype_ok(dt)) return GDR2_E_DTYPE;
    if (N < 0 || D < 0) return GDR2_E_SHAPE;
    if (D < 8 || D % 8) return GDR2_E_UNSUPPORTED;
    if (!prod_le(N, D, (int64_t)1 << 34)) return GDR2_E_SHAPE;  // eight per thread of one launch
    if (N == 0) return GDR2_OK;
    if (!x || !log_a || !h_out || !h) return GDR2_E_NULL;
    if (!all_aligned({x, log_a, h_in, h_out, h})) return GDR2_E_ALIGN;
    const size_t n = (size_t)N * D;
    // h_in may be h_out exactly; any other overlap with an output is an error
    const Range ins[] = {{x, n * esize(dt)}, {log_a, n * 4}, {h_in == h_out ? nullptr : h_in, n * 4}};
    const Range outs[] = {{h_out, n * 4}, {h, n * esize(dt)}};
    if (any_alias(outs, 2, ins, 3)) return GDR2_E_ALIAS;
    gdr2::GlrStepParams p{(long)n, x, log_a, h_in, h_out, h};
    return status_of(gdr2::glr_step_dispatch(dt == GDR2_BF16, p, (hipStream_t)stream));
}

gdr2_status gdr2_swa_fwd(int64_t B, int64_t T, int64_t H, int64_t Hkv, int64_t d, gdr2_dtype dt,
                         int64_t window, int64_t sinks, float scale, const void* q, const void* k,
                         const void* v, const int32_t* lengths, void* o, float* lse, void* stream) {
    if (!dtype_ok(dt)) return GDR2_E_DTYPE;
    const gdr2_status st = check_swa(B, T, H, Hkv, d, window, sinks);
    if (st != GDR2_OK) return st;
    if (!scale_ok(scale)) return GDR2_E_VALUE;
    if (B == 0 || T == 0 || H == 0) return GDR2_OK;
    if (!q || !k || !v || !o || !lse) return GDR2_E_NULL;
    if (!all_aligned({q, k, v, o}) || !aligned4(lse) || !aligned4(lengths)) return GDR2_E_ALIGN;
    const size_t nq = (size_t)B * T * H * d * esize(dt), nk = (size_t)B * T * Hkv * d * esize(dt);
    const Range ins[] = {{q, nq}, {k, nk}, {v, nk}, {lengths, (size_t)B * 4}};
    const Range outs[] = {{o, nq}, {lse, (size_t)B * T * H * 4}};
    if (any_alias(outs, 2, ins, 4)) return GDR2_E_ALIAS;
    gdr2::SwaParams p = swa_params(B, T, H, Hkv, d, window, sinks, scale, q, k, v, lengths);
    p.o = o; p.lse = lse;
    return status_of(gdr2::swa_fwd_dispatch(dt == GDR2_BF16, p, (hipStream_t)stream));
}

size_t gdr2_swa_bwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Hkv, int64_t d,
                                    int64_t window, int64_t sinks) {
    if (check_swa_bwd(B, T, H, Hkv, d, window, sinks) != GDR2_OK) return 0;
    return swa_bwd_layout(B, T, H, Hkv, d, window, sinks).total;
}

gdr2_status gdr2_swa_bwd(int64_t B, int64_t T, int64_t H, int64_t Hkv, int64_t d, gdr2_dtype dt,
                         int64_t window, int64_t sinks, float scale, const void* q, const void* k,
                         const void* v, const int32_t* lengths, const void* o, const float* lse,
                         const void* dO, void* dq, void* dk, void* dv, void* workspace,
                         size_t workspace_bytes, void* stream) {
    if (!dtype_ok(dt)) return GDR2_E_DTYPE;
    const gdr2_status st = check_swa_bwd(B, T, H, Hkv, d, window, sinks);
    if (st != GDR2_OK) return st;
    if (!scale_ok(scale)) return GDR2_E_VALUE;
    if (B == 0 || T == 0 || H == 0) return GDR2_OK;
    if (!q || !k || !v || !o || !lse || !dO || !dq || !dk || !dv) return GDR2_E_NULL;
    if (!all_aligned({q, k, v, o, dO, dq, dk, dv, workspace}) || !aligned4(lse) || !aligned4(lengths)) return GDR2_E_ALIGN;
    const SwaBwdWs w = swa_bwd_layout(B, T, H, Hkv, d, window, sinks);
    if (!workspace || workspace_bytes < w.total) return GDR2_E_WORKSPACE;
    const size_t nq = (size_t)B * T * H * d * esize(dt), nk = (size_t)B * T * Hkv * d * esize(dt);
    const Range ins[] = {{q, nq}, {k, nk}, {v, nk}, {lengths, (size_t)B * 4}, {o, nq}, {lse, (size_t)B * T * H * 4}, {dO, nq}};
    const Range outs[] = {{dq, nq}, {dk, nk}, {dv, nk}, {workspace, w.total}};
    if (any_alias(outs, 4, ins, 7)) return GDR2_E_ALIAS;
    gdr2::SwaParams p = swa_params(B, T, H, Hkv, d, window, sinks, scale, q, k, v, lengths);
    p.o = (void*)o; p.lse = (float*)lse; p.dO = dO; p.dq = dq; p.dk = dk; p.dv = dv;
    p.delta = (float*)((char*)workspace + w.delta);
    p.sink_part = (float*)((char*)workspace + w.sinks);
    p.key_part = (float*)((char*)workspace + w.keys);
    p.splits = w.cut.splits; p.part_rows = w.cut.part_rows; p.pieces = w.cut.pieces;
    p.far0 = w.cut.far0; p.piece_len = w.cut.piece_len;
    return status_of(gdr2::swa_bwd_dispatch(dt == GDR2_BF16, p, (hipStream_t)stream));
}

gdr2_status gdr2_swa_cache_fill(int64_t B, int64_t T, int64_t Hkv, int64_t d, gdr2_dtype dt,
                                int64_t window, int64_t sinks, const void* k, const void* v,
                                const int32_t* lengths, void* k_cache, void* v_cache, void* stream) {
    if (!dtype_ok(dt)) return GDR2_E_DTYPE;
    gdr2_status st = check_swa(B, T, Hkv, Hkv, d, window, sinks);
    if (st == GDR2_OK) st = check_decode(B, Hkv, Hkv, d, window, sinks);
    if (st != GDR2_OK) return st;
    if (B == 0 || T == 0 || Hkv == 0) return GDR2_OK;
    if (!k || !v || !k_cache || !v_cache) return GDR2_E_NULL;
    if (!all_aligned({k, v, k_cache, v_cache}) || !aligned4(lengths)) return GDR2_E_ALIGN;
    const size_t n = (size_t)B * T * Hkv * d * esize(dt), nc = (size_t)B * (window + sinks) * Hkv * d * esize(dt);
    const Range ins[] = {{k, n}, {v, n}, {lengths, (size_t)B * 4}}, outs[] = {{k_cache, nc}, {v_cache, nc}};
    if (any_alias(outs, 2, ins, 3)) return GDR2_E_ALIAS;
    gdr2::SwaFillParams p{};
    p.B = (int)B; p.Hkv = (int)Hkv; p.sinks = (int)sinks; p.T = T; p.window = window;
    p.row16 = Hkv * d * (int64_t)esize(dt) / 16;
    p.k = k; p.v = v; p.kc = k_cache; p.vc = v_cache; p.lengths = lengths;
    return status_of(gdr2::swa_fill_dispatch(p, (hipStream_t)stream));
}

size_t gdr2_swa_decode_workspace_bytes(int64_t N, int64_t H, int64_t Hkv, int64_t d, int64_t window,
                                       int64_t sinks) {
    if (check_decode(N, H, Hkv, d, window, sinks) != GDR2_OK) return 0;
    const int splits = decode_splits(N, H, Hkv, window, sinks);
    return splits > 1 ? (size_t)decode_jobs(N, H, Hkv) * splits * 16 * (d + 4) * sizeof(float) : 0;
}

gdr2_status gdr2_swa_decode_step(int64_t N, int64_t H, int64_t Hkv, int64_t d, gdr2_dtype dt,
                                 int64_t window, int64_t sinks, float scale, const void* q,
                                 const void* k, const void* v, void* k_cache, void* v_cache,
                                 const int32_t* pos, void* o, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    if (!dtype_ok(dt)) return GDR2_E_DTYPE;
    const gdr2_status st = check_decode(N, H, Hkv, d, window, sinks);
    if (st != GDR2_OK) return st;
    if (!scale_ok(scale)) return GDR2_E_VALUE;
    if (N == 0 || H == 0) return GDR2_OK;
    if (!q || !k || !v || !k_cache || !v_cache || !pos || !o) return GDR2_E_NULL;
    if (!all_aligned({q, k, v, k_cache, v_cache, o, workspace}) || !aligned4(pos)) return GDR2_E_ALIGN;
    const size_t need = gdr2_swa_decode_workspace_bytes(N, H, Hkv, d, window, sinks);
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDR2_E_WORKSPACE;
    const size_t es = esize(dt), nq = (size_t)N * H * d * es, nk = (size_t)N * Hkv * d * es;
    const size_t nc = (size_t)N * (window + sinks) * Hkv * d * es;
    const Range ins[] = {{q, nq}, {k, nk}, {v, nk}, {pos, (size_t)N * 4}};
    const Range outs[] = {{k_cache, nc}, {v_cache, nc}, {o, nq}, {workspace, need}};
    if (any_alias(outs, 4, ins, 4)) return GDR2_E_ALIAS;
    gdr2::SwaDecodeParams p{};
    p.N = (int)N; p.H = (int)H; p.Hkv = (int)Hkv; p.d = (int)d; p.sinks = (int)sinks; p.window = window;
    p.scale = scale; p.q = q; p.k = k; p.v = v; p.kc = k_cache; p.vc = v_cache; p.pos = pos; p.o = o;
    p.splits = decode_splits(N, H, Hkv, window, sinks);
    p.part = (float*)workspace;
    return status_of(gdr2::swa_decode_dispatch(dt == GDR2_BF16, p, (hipStream_t)stream));
}

}  // extern "C"

// gdr2_hybrid_api.hip -- the C ABI of the RMS norm of a residual stream, linear attention with a decay per
// head and the paged key/value cache: host-side validation, then launch.  Nothing here touches device memory
// before every check has passed, and every size is bounded before a product that depends on it is formed.
#include "gdr2.h"

#include <hip/hip_runtime.h>

#include "gdr2_checks.hpp"
#include "gdr2_hybrid_kernels.hpp"

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

// ------------------------------------------------------------------ RMS norm
gdr2_status check_rms(int64_t rows, int64_t D) {
    if (rows < 0 || D < 0 || rows > kMaxInt) return GDR2_E_SHAPE;
    if (D < 8 || D > gdr2::kNormMaxD || D % 8) return GDR2_E_UNSUPPORTED;
    return GDR2_OK;
}
// Both forwards: `y` of ybytes per element, `stat` (rstd or scales) of nstat numbers per row.
gdr2_status rms_fwd(gdr2::RmsKind kind, int64_t rows, int64_t D, gdr2_dtype dt, int64_t group, const void* x,
                    const void* residual, const float* weight, float eps, void* h, void* y, float* stat, void* stream) {
    if (!dtype_ok(dt)) return GDR2_E_DTYPE;
    const gdr2_status st = check_rms(rows, D);
    if (st != GDR2_OK) return st;
    const bool q8 = kind == gdr2::kRmsQ8;
    if (q8 && group != 0 && group != 32 && group != 64 && group != 128) return GDR2_E_UNSUPPORTED;
    if (!(eps > 0.f) || !(eps < 1e30f) || (h && !residual)) return GDR2_E_VALUE;
    if (rows == 0) return GDR2_OK;
    if (!x || !weight || !y || (residual && !h) || (q8 && !stat)) return GDR2_E_NULL;
    if (!all_aligned({x, residual, weight, h, y}) || !aligned4(stat)) return GDR2_E_ALIGN;
    const size_t n = (size_t)rows * D, nstat = (size_t)rows * (q8 && group ? (D + group - 1) / group : 1);
    // h may be residual exactly; any other overlap with an output is an error
    const Range ins[] = {{x, n * esize(dt)}, {h == residual ? nullptr : residual, n * esize(dt)}, {weight, (size_t)D * 4}};
    const Range outs[] = {{h, n * esize(dt)}, {y, n * (q8 ? 1 : esize(dt))}, {stat, nstat * 4}};
    if (any_alias(outs, 3, ins, 3)) return GDR2_E_ALIAS;
    gdr2::RmsParams p{};
    p.rows = rows; p.D = (int)D; p.group = (int)group; p.eps = eps;
    p.x = x; p.residual = residual; p.weight = weight; p.h = h; p.y = y;
    (q8 ? p.scale : p.rstd) = stat;
    return status_of(gdr2::rms_dispatch(dt == GDR2_BF16, kind, p, (hipStream_t)stream));
}

// ------------------------------------------------------------------ linear attention with a decay per head
// Afterwards B * H <= 2^19, B * T * H <= 2^30, and every launch fits: at most twelve workgroups of 512 threads per
// chain, or (few chains, cut into segments) at most 256 in all.
gdr2_status check_dla(int64_t B, int64_t T, int64_t H, int64_t dk, int64_t dv) {
    if (B < 0 || T < 0 || H < 0 || dk < 0 || dv < 0 || T > ((int64_t)1 << 30) || H > 32768) return GDR2_E_SHAPE;
    if (!dims_ok(dk) || !dims_ok(dv)) return GDR2_E_UNSUPPORTED;
    if (!prod_le(B, H, (int64_t)1 << 19) || !prod_le(B * H, (T + 63) / 64 + 1, ((int64_t)1 << 24) - 1)) return GDR2_E_SHAPE;
    return GDR2_OK;
}
// The forward is one pass with dv columns; the backward's dq and dk have dk columns, dv has dv.
struct DlaPlan {
    gdr2::DlaCut cut;
    size_t total;
};
DlaPlan dla_plan(bool bwd, int64_t B, int64_t T, int64_t H, int64_t dk, int64_t dv, gdr2_dtype dt) {
    const bool f32 = dt == GDR2_F32;
    const int slots = gdr2::dla_slots((int)dv, f32) + (bwd ? 2 * gdr2::dla_slots((int)dk, f32) : 0);
    DlaPlan d{gdr2::dla_cut(B, T, H, slots, f32), 0};
    d.total = round_up((size_t)(bwd ? 3 : 1) * B * H * (d.cut.segs - 1) * dk * dv * sizeof(float), 256);
    return d;
}
template <size_t N>
gdr2_status dla_run(const DlaPlan& d, int64_t B, int64_t T, int64_t H, gdr2_dtype dt, const gdr2::DlaPass (&pass)[N],
                    const float* log_decay, const int32_t* lengths, void* ws, void* stream) {
    gdr2::DlaParams p{};
    p.B = (int)B; p.T = (int)T; p.H = (int)H; p.passes = (int)N;
    p.segs = d.cut.segs; p.seg_chunks = d.cut.seg_chunks;
    p.log_decay = log_decay; p.lengths = lengths; p.local = (float*)ws;
    for (size_t i = 0; i < N; ++i) {
        p.pass[i] = pass[i];
        p.pass[i].slot = p.slots;
        p.slots += gdr2::dla_slots(pass[i].V, dt == GDR2_F32);
    }
    return status_of(gdr2::dla_dispatch(dt == GDR2_BF16, p, (hipStream_t)stream));
}

// ------------------------------------------------------------------ paged cache
bool scale_ok(float s) { return s > 0.f && s < 1e30f; }
int shift_of(int64_t page) {  // -1: no power of two
    for (int s = 0; s <= 30; ++s)
        if (page == (int64_t)1 << s) return s;
    return -1;
}
gdr2_status check_pages(int64_t H, int64_t Hkv, int64_t d, int64_t page, int64_t pages, int64_t width) {
    if (H < 0 || Hkv < 0 || d < 0 || H > 32768 || pages < 0 || width < 0) return GDR2_E_SHAPE;
    if (!dims_ok(d)) return GDR2_E_UNSUPPORTED;
    if (H > 0 ? Hkv == 0 || H % Hkv : Hkv != 0) return GDR2_E_SHAPE;
    if (shift_of(page) < 0) return GDR2_E_VALUE;
    if (!prod_le(page, pages, kMaxInt) || !prod_le(page, width, (int64_t)1 << 30)) return GDR2_E_SHAPE;
    return GDR2_OK;
}
gdr2_status check_paged_decode(int64_t N, int64_t H, int64_t Hkv, int64_t d, int64_t page, int64_t pages, int64_t width) {
    const gdr2_status st = check_pages(H, Hkv, d, page, pages, width);
    if (st != GDR2_OK) return st;
    if (N < 0 || !prod_le(N, H, (int64_t)1 << 30) || !prod_le(N, width, (int64_t)1 << 40)) return GDR2_E_SHAPE;
    return GDR2_OK;
}
int64_t head_groups(int64_t H, int64_t Hkv) { return Hkv ? (H / Hkv + gdr2::kPagedHeads - 1) / gdr2::kPagedHeads : 0; }

}  // namespace

extern "C" {

gdr2_status gdr2_rms_norm_fwd(int64_t rows, int64_t D, gdr2_dtype dt, const void* x, const void* residual,
                              const float* weight, float eps, void* h, void* y, float* rstd, void* stream) {
    return rms_fwd(gdr2::kRmsFwd, rows, D, dt, 0, x, residual, weight, eps, h, y, rstd, stream);
}

gdr2_status gdr2_rms_norm_q8_fwd(int64_t rows, int64_t D, gdr2_dtype dt, int64_t group, const void* x,
                                 const void* residual, const float* weight, float eps, void* h, void* y8,
                                 float* scale, void* stream) {
    return rms_fwd(gdr2::kRmsQ8, rows, D, dt, group, x, residual, weight, eps, h, y8, scale, stream);
}

size_t gdr2_rms_norm_bwd_workspace_bytes(int64_t rows, int64_t D) {
    if (check_rms(rows, D) != GDR2_OK) return 0;
    return (size_t)gdr2::rms_bwd_blocks(rows, (int)D) * D * sizeof(float);
}

gdr2_status gdr2_rms_norm_bwd(int64_t rows, int64_t D, gdr2_dtype dt, const void* h, const float* weight,
                              const float* rstd, const void* dy, const void* dh, void* dx, float* dweight,
                              void* workspace, size_t workspace_bytes, void* stream) {
    if (!dtype_ok(dt)) return GDR2_E_DTYPE;
    const gdr2_status st = check_rms(rows, D);
    if (st != GDR2_OK) return st;
    if (!dweight) return GDR2_E_NULL;
    if (rows > 0 && (!h || !weight || !rstd || !dy || !dx)) return GDR2_E_NULL;
    if (!all_aligned({h, weight, dy, dh, dx, dweight, workspace}) || !aligned4(rstd)) return GDR2_E_ALIGN;
    const size_t need = gdr2_rms_norm_bwd_workspace_bytes(rows, D);
    if (rows > 0 && (!workspace || workspace_bytes < need)) return GDR2_E_WORKSPACE;
    const size_t n = (size_t)rows * D * esize(dt), w = (size_t)D * 4;
    const Range ins[] = {{h, n}, {weight, w}, {rstd, (size_t)rows * 4}, {dy, n}, {dh, n}};
    const Range outs[] = {{dx, n}, {dweight, w}, {workspace, need}};
    if (any_alias(outs, 3, ins, 5)) return GDR2_E_ALIAS;
    gdr2::RmsParams p{};
    p.rows = rows; p.D = (int)D; p.x = h; p.weight = weight; p.rstd = (float*)rstd; p.dy = dy; p.dh = dh;
    p.dx = dx; p.dweight = dweight; p.part = (float*)workspace;
    return status_of(gdr2::rms_dispatch(dt == GDR2_BF16, gdr2::kRmsBwd, p, (hipStream_t)stream));
}

size_t gdr2_dla_fwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t dk, int64_t dv, gdr2_dtype dt) {
    if (!dtype_ok(dt) || check_dla(B, T, H, dk, dv) != GDR2_OK) return 0;
    return dla_plan(false, B, T, H, dk, dv, dt).total;
}

gdr2_status gdr2_dla_fwd(int64_t B, int64_t T, int64_t H, int64_t dk, int64_t dv, gdr2_dtype dt, const void* q,
                         const void* k, const void* v, const float* log_decay, const float* S0, const int32_t* lengths,
                         void* o, float* S_T, void* workspace, size_t workspace_bytes, void* stream) {
    if (!dtype_ok(dt)) return GDR2_E_DTYPE;
    const gdr2_status st = check_dla(B, T, H, dk, dv);
    if (st != GDR2_OK) return st;
    if (B == 0 || H == 0) return GDR2_OK;
    if (!log_decay || (T > 0 && (!q || !k || !v || !o))) return GDR2_E_NULL;
    if (!all_aligned({q, k, v, S0, o, S_T, workspace}) || !aligned4(log_decay) || !aligned4(lengths)) return GDR2_E_ALIGN;
    const DlaPlan d = dla_plan(false, B, T, H, dk, dv, dt);
    if (d.total > 0 && (!workspace || workspace_bytes < d.total)) return GDR2_E_WORKSPACE;
    const size_t n = (size_t)B * T * H * esize(dt), ns = (size_t)B * H * dk * dv * 4;
    const Range ins[] = {{q, n * dk}, {k, n * dk}, {v, n * dv}, {log_decay, (size_t)H * 4}, {S0, ns}, {lengths, (size_t)B * 4}};
    const Range outs[] = {{o, n * dv}, {S_T, ns}, {workspace, d.total}};
    if (any_alias(outs, 3, ins, 6)) return GDR2_E_ALIAS;
    const int K = (int)dk, V = (int)dv;
    const gdr2::DlaPass pass[] = {{K, V, q, k, v, o, S0, S_T, 0, 0, 1, 0}};
    return dla_run(d, B, T, H, dt, pass, log_decay, lengths, workspace, stream);
}

size_t gdr2_dla_bwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t dk, int64_t dv, gdr2_dtype dt) {
    if (!dtype_ok(dt) || check_dla(B, T, H, dk, dv) != GDR2_OK) return 0;
    return dla_plan(true, B, T, H, dk, dv, dt).total;
}

gdr2_status gdr2_dla_bwd(int64_t B, int64_t T, int64_t H, int64_t dk, int64_t dv, gdr2_dtype dt, const void* q,
                         const void* k, const void* v, const float* log_decay, const float* S0, const int32_t* lengths,
                         const void* dO, const float* dS_T, void* dq, void* dk_, void* dv_, float* dS0, void* workspace,
                         size_t workspace_bytes, void* stream) {
    if (!dtype_ok(dt)) return GDR2_E_DTYPE;
    const gdr2_status st = check_dla(B, T, H, dk, dv);
    if (st != GDR2_OK) return st;
    if (B == 0 || H == 0) return GDR2_OK;
    if (!log_decay || (T > 0 && (!q || !k || !v || !dO || !dq || !dk_ || !dv_))) return GDR2_E_NULL;
    if (!all_aligned({q, k, v, S0, dO, dS_T, dq, dk_, dv_, dS0, workspace}) || !aligned4(log_decay) || !aligned4(lengths)) return GDR2_E_ALIGN;
    const DlaPlan d = dla_plan(true, B, T, H, dk, dv, dt);
    if (d.total > 0 && (!workspace || workspace_bytes < d.total)) return GDR2_E_WORKSPACE;
    const size_t n = (size_t)B * T * H * esize(dt), ns = (size_t)B * H * dk * dv * 4;
    const Range ins[] = {{q, n * dk}, {k, n * dk}, {v, n * dv}, {log_decay, (size_t)H * 4}, {S0, ns}, {lengths, (size_t)B * 4}, {dO, n * dv}, {dS_T, ns}};
    const Range outs[] = {{dq, n * dk}, {dk_, n * dk}, {dv_, n * dv}, {dS0, ns}, {workspace, d.total}};
    if (any_alias(outs, 5, ins, 8)) return GDR2_E_ALIAS;
    const int K = (int)dk, V = (int)dv;
    const gdr2::DlaPass pass[] = {{V, K, dO, v, k, dq, S0, nullptr, 0, 1, 0, 0},
                                  {V, K, v, dO, q, dk_, dS_T, nullptr, 1, 1, 0, 0},
                                  {K, V, k, q, dO, dv_, dS_T, dS0, 1, 0, 1, 0}};
    return dla_run(d, B, T, H, dt, pass, log_decay, lengths, workspace, stream);
}

gdr2_status gdr2_dla_step(int64_t N, int64_t H, int64_t dk, int64_t dv, gdr2_dtype dt, const void* q, const void* k,
                          const void* v, const float* log_decay, const float* S_in, float* S_out, void* o, void* stream) {
    if (!dtype_ok(dt)) return GDR2_E_DTYPE;
    if (N < 0 || H < 0 || dk < 0 || dv < 0) return GDR2_E_SHAPE;
    if (!dims_ok(dk) || !dims_ok(dv)) return GDR2_E_UNSUPPORTED;
    if (!prod_le(N, H, ((int64_t)1 << 24) - 1)) return GDR2_E_SHAPE;  // a workgroup of 256 threads per chain
    if (N == 0 || H == 0) return GDR2_OK;
    if (!q || !k || !v || !log_decay || !S_out || !o) return GDR2_E_NULL;
    if (!all_aligned({q, k, v, S_in, S_out, o}) || !aligned4(log_decay)) return GDR2_E_ALIGN;
    const size_t n = (size_t)N * H, es = esize(dt), ns = n * dk * dv * 4;
    // S_in may be S_out exactly; any other overlap with an output is an error
    const Range ins[] = {{q, n * dk * es}, {k, n * dk * es}, {v, n * dv * es}, {log_decay, (size_t)H * 4}, {S_in == S_out ? nullptr : S_in, ns}};
    const Range outs[] = {{S_out, ns}, {o, n * dv * es}};
    if (any_alias(outs, 2, ins, 5)) return GDR2_E_ALIAS;
    gdr2::DlaStepParams p{(long)n, (int)H, q, k, v, log_decay, S_in, S_out, o};
    return status_of(gdr2::dla_step_dispatch(dt == GDR2_BF16, (int)dk, (int)dv, p, (hipStream_t)stream));
}

gdr2_status gdr2_paged_cache_fill(int64_t B, int64_t T, int64_t Hkv, int64_t d, gdr2_dtype dt, int64_t page, int64_t pages,
                                  int64_t width, const void* k, const void* v, const int32_t* start, const int32_t* lengths,
                                  const int32_t* page_table, void* k_pages, void* v_pages, void* stream) {
    if (!dtype_ok(dt)) return GDR2_E_DTYPE;
    const gdr2_status st = check_pages(Hkv, Hkv, d, page, pages, width);
    if (st != GDR2_OK) return st;
    if (B < 0 || T < 0 || T > kMaxInt || B > kMaxInt || !prod_le(B, width, (int64_t)1 << 40)) return GDR2_E_SHAPE;
    if (Hkv > 0 && (!prod_le(B, T, (int64_t)1 << 32) || !prod_le(B * T, Hkv, (int64_t)1 << 32))) return GDR2_E_SHAPE;
    if (B == 0 || T == 0 || Hkv == 0 || pages == 0 || width == 0) return GDR2_OK;  // no row to store in
    if (!k || !v || !page_table || !k_pages || !v_pages) return GDR2_E_NULL;
    if (!all_aligned({k, v, k_pages, v_pages}) || !aligned4(start) || !aligned4(lengths) || !aligned4(page_table)) return GDR2_E_ALIGN;
    const size_t row = (size_t)Hkv * d * esize(dt), n = (size_t)B * T * row, nc = (size_t)pages * page * row;
    const Range ins[] = {{k, n}, {v, n}, {start, (size_t)B * 4}, {lengths, (size_t)B * 4}, {page_table, (size_t)B * width * 4}};
    const Range outs[] = {{k_pages, nc}, {v_pages, nc}};
    if (any_alias(outs, 2, ins, 5)) return GDR2_E_ALIAS;
    gdr2::PagedFillParams p{};
    p.B = (int)B; p.T = (int)T; p.shift = shift_of(page); p.pages = (int)pages; p.width = (int)width; p.row16 = (int)(row / 16);
    p.k = k; p.v = v; p.start = start; p.lengths = lengths; p.table = page_table; p.kp = k_pages; p.vp = v_pages;
    return status_of(gdr2::paged_fill_dispatch(p, (hipStream_t)stream));
}

size_t gdr2_paged_decode_workspace_bytes(int64_t N, int64_t H, int64_t Hkv, int64_t d, int64_t page, int64_t width) {
    if (check_paged_decode(N, H, Hkv, d, page, 0, width) != GDR2_OK) return 0;
    const int64_t groups = head_groups(H, Hkv);
    const int splits = gdr2::paged_splits(N, Hkv, groups, page * width);
    return splits > 1 ? (size_t)N * Hkv * groups * splits * gdr2::kPagedHeads * (d + 4) * sizeof(float) : 0;
}

gdr2_status gdr2_paged_decode_step(int64_t N, int64_t H, int64_t Hkv, int64_t d, gdr2_dtype dt, int64_t page, int64_t pages,
                                   int64_t width, float scale, const void* q, const void* k, const void* v,
                                   const int32_t* page_table, const int32_t* pos, void* k_pages, void* v_pages, void* o,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    if (!dtype_ok(dt)) return GDR2_E_DTYPE;
    const gdr2_status st = check_paged_decode(N, H, Hkv, d, page, pages, width);
    if (st != GDR2_OK) return st;
    if (!scale_ok(scale)) return GDR2_E_VALUE;
    if (N == 0 || H == 0) return GDR2_OK;
    if (!q || !k || !v || !pos || !o || (width > 0 && !page_table) || (pages > 0 && (!k_pages || !v_pages))) return GDR2_E_NULL;
    if (!all_aligned({q, k, v, k_pages, v_pages, o, workspace}) || !aligned4(page_table) || !aligned4(pos)) return GDR2_E_ALIGN;
    const size_t need = gdr2_paged_decode_workspace_bytes(N, H, Hkv, d, page, width);
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDR2_E_WORKSPACE;
    const size_t es = esize(dt), nq = (size_t)N * H * d * es, nk = (size_t)N * Hkv * d * es, nc = (size_t)pages * page * Hkv * d * es;
    const Range ins[] = {{q, nq}, {k, nk}, {v, nk}, {page_table, (size_t)N * width * 4}, {pos, (size_t)N * 4}};
    const Range outs[] = {{k_pages, nc}, {v_pages, nc}, {o, nq}, {workspace, need}};
    if (any_alias(outs, 4, ins, 5)) return GDR2_E_ALIAS;
    gdr2::PagedDecodeParams p{};
    p.N = (int)N; p.H = (int)H; p.Hkv = (int)Hkv; p.d = (int)d; p.shift = shift_of(page); p.pages = (int)pages; p.width = (int)width;
    p.scale = scale; p.q = q; p.k = k; p.v = v; p.table = page_table; p.pos = pos; p.kp = k_pages; p.vp = v_pages; p.o = o;
    p.splits = gdr2::paged_splits(N, Hkv, head_groups(H, Hkv), page * width); p.part = (float*)workspace;
    return status_of(gdr2::paged_decode_dispatch(dt == GDR2_BF16, p, (hipStream_t)stream));
}

}  // extern "C"

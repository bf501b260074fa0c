// Host-only driver for the C ABI of the residual stream's RMS norm, linear attention with a decay and the paged cache
// under AddressSanitizer and UndefinedBehaviorSanitizer: gdr2_hybrid_api.hip compiled as plain C++ against launch
// stand-ins that check what a launch would be given (sizes in range, parts inside the workspace) and touch no memory.
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "gdr2.h"
#include "gdr2_hybrid_kernels.hpp"

static long g_launches = 0;
static int g_fail = 0;
static uintptr_t g_ws = 0, g_ws_end = 0;  // the workspace of the running call
#define CHECK(c)                                                        \
    do {                                                                \
        if (!(c)) {                                                     \
            std::printf("FAIL line %d: %s\n", __LINE__, #c);            \
            ++g_fail;                                                   \
        }                                                               \
    } while (0)
static bool inside(const void* p, size_t n) { return !n || ((uintptr_t)p >= g_ws && (uintptr_t)p + n <= g_ws_end); }

namespace gdr2 {
// stand-ins for the sizing rules that live beside their kernels
long rms_bwd_blocks(long rows, int) { return rows < 512 ? rows : 512; }
int dla_slots(int V, bool f32) { return f32 ? V / 32 : 1; }
DlaCut dla_cut(long B, long T, long H, long slots, bool) {
    const long nch = (T + kDlaChunk - 1) / kDlaChunk, jobs = B * H * slots;
    long n = jobs > 0 ? 300 / jobs : 1;
    n = n < nch / 2 ? n : nch / 2;
    n = n < 1 ? 1 : n;
    const long per = (nch + n - 1) / n > 1 ? (nch + n - 1) / n : 1, segs = (nch + per - 1) / per;
    return DlaCut{(int)(segs < 1 ? 1 : segs), (int)per};
}
int paged_splits(long N, long Hkv, long groups, long capacity) {
    const long jobs = N * Hkv * groups, steps = (capacity + kPagedStep) / kPagedStep;
    if (jobs < 1 || jobs > 500) return 1;
    return (int)(500 / jobs < steps ? 500 / jobs : steps);
}
hipError_t rms_dispatch(int, RmsKind kind, const RmsParams& p, hipStream_t) {
    ++g_launches;
    CHECK(p.D >= 8 && p.D <= kNormMaxD && p.D % 8 == 0 && p.rows >= 0 && p.rows <= 0x7fffffff);
    if (kind == kRmsBwd) CHECK(inside(p.part, (size_t)rms_bwd_blocks(p.rows, p.D) * p.D * 4));
    else CHECK(p.y && (p.residual == nullptr) == (p.h == nullptr) && (kind == kRmsQ8) == (p.scale != nullptr));
    return hipSuccess;
}
hipError_t dla_dispatch(int bf, const DlaParams& p, hipStream_t) {
    ++g_launches;
    CHECK(p.passes == 1 || p.passes == 3);
    CHECK((int64_t)p.B * p.H <= 1 << 19 && (int64_t)p.B * p.T * p.H <= (int64_t)1 << 30 && p.H <= 32768);
    int slots = 0;
    for (int i = 0; i < p.passes; ++i) {
        CHECK((p.pass[i].K == 64 || p.pass[i].K == 128) && p.pass[i].slot == slots && p.pass[i].K * p.pass[i].V == p.pass[0].K * p.pass[0].V);
        slots += dla_slots(p.pass[i].V, !bf);
    }
    CHECK(slots == p.slots && (int64_t)p.segs * p.seg_chunks * kDlaChunk >= p.T);
    CHECK((int64_t)p.B * p.H * p.slots * p.segs < (int64_t)1 << 31);
    CHECK(inside(p.local, (size_t)p.passes * p.B * p.H * (p.segs - 1) * p.pass[0].K * p.pass[0].V * 4));
    return hipSuccess;
}
hipError_t dla_step_dispatch(int, int dk, int dv, const DlaStepParams& p, hipStream_t) {
    ++g_launches;
    CHECK(p.n > 0 && p.n < 1 << 24 && dk * dv >= 4096);
    return hipSuccess;
}
hipError_t paged_fill_dispatch(const PagedFillParams& p, hipStream_t) {
    ++g_launches;
    CHECK(p.B > 0 && p.T > 0 && p.row16 > 0 && ((int64_t)p.pages << p.shift) < (int64_t)1 << 31 && ((int64_t)p.width << p.shift) <= 1 << 30);
    return hipSuccess;
}
hipError_t paged_decode_dispatch(int, const PagedDecodeParams& p, hipStream_t) {
    ++g_launches;
    const size_t jobs = (size_t)p.N * p.Hkv * ((p.H / p.Hkv + kPagedHeads - 1) / kPagedHeads);
    CHECK(p.splits >= 1 && ((int64_t)p.pages << p.shift) < (int64_t)1 << 31 && ((int64_t)p.width << p.shift) <= 1 << 30);
    if (p.splits > 1) CHECK(inside(p.part, jobs * p.splits * kPagedHeads * (p.d + 4) * 4));
    return hipSuccess;
}
}  // namespace gdr2

#define EXPECT(call, want)                                                                              \
    do {                                                                                                \
        const long before = g_launches;                                                                 \
        const int got = (int)(call);                                                                    \
        if (got != (want) || (got != GDR2_OK && g_launches != before)) {                                \
            std::printf("FAIL line %d: %s -> %d (want %d)\n", __LINE__, #call, got, (int)(want));       \
            ++g_fail;                                                                                   \
        }                                                                                               \
    } while (0)

// addresses far apart, never dereferenced
static void* A(int i) { return (void*)((uintptr_t)(i + 1) << 48); }
static float* F(int i) { return (float*)A(i); }
static int32_t* I(int i) { return (int32_t*)A(i); }
static void* W(int i, size_t n) {
    g_ws = (uintptr_t)A(i);
    g_ws_end = g_ws + n;
    return n ? A(i) : nullptr;
}

int main() {
    const int64_t big[] = {0, 1, 7, 64, 4096, 1 << 20, (int64_t)1 << 31, (int64_t)1 << 40, INT64_MAX};
    // every size query and call over a grid of sizes, products that overflow 64 bits among them: no
    // sanitizer report, and a workspace of the queried size always holds what a launch is given
    for (int64_t a : big)
        for (int64_t b : big) {
            size_t n = gdr2_rms_norm_bwd_workspace_bytes(a, b);
            (void)gdr2_rms_norm_fwd(a, b, GDR2_BF16, A(0), A(1), F(2), 1e-6f, A(3), A(4), F(5), nullptr);
            (void)gdr2_rms_norm_q8_fwd(a, b, GDR2_F32, 64, A(0), A(1), F(2), 1e-6f, A(1), A(4), F(5), nullptr);
            (void)gdr2_rms_norm_bwd(a, b, GDR2_BF16, A(0), F(1), F(2), A(3), A(4), A(5), F(6), W(7, n), n, nullptr);
            (void)gdr2_dla_step(a, b, 64, 128, GDR2_F32, A(0), A(1), A(2), F(3), F(4), F(4), A(5), nullptr);
            for (int64_t c : {(int64_t)0, (int64_t)1, (int64_t)12, (int64_t)32768, (int64_t)1 << 40, INT64_MAX})
                for (gdr2_dtype dt : {GDR2_BF16, GDR2_F32})
                    for (int64_t dk : {64, 128}) {
                        n = gdr2_dla_fwd_workspace_bytes(a, b, c, dk, 128, dt);
                        (void)gdr2_dla_fwd(a, b, c, dk, 128, dt, A(0), A(1), A(2), F(3), F(4), I(5), A(6), F(7), W(8, n), n, nullptr);
                        n = gdr2_dla_bwd_workspace_bytes(a, b, c, dk, 128, dt);
                        (void)gdr2_dla_bwd(a, b, c, dk, 128, dt, A(0), A(1), A(2), F(3), F(4), I(5), A(6), F(7), A(8), A(9), A(10), F(11), W(12, n), n, nullptr);
                        for (int64_t page : {(int64_t)1, (int64_t)16, (int64_t)1 << 20, (int64_t)1 << 40})
                            for (int64_t width : {(int64_t)0, (int64_t)3, (int64_t)1 << 20, INT64_MAX}) {
                                (void)gdr2_paged_cache_fill(a, b, c, dk, dt, page, width, width, A(0), A(1), I(2), I(3), I(4), A(5), A(6), nullptr);
                                n = gdr2_paged_decode_workspace_bytes(a, c, c, dk, page, width);
                                (void)gdr2_paged_decode_step(a, c, c, dk, dt, page, b, width, 1.f, A(0), A(1), A(2), I(3), I(4), A(5), A(6), A(7), W(8, n), n, nullptr);
                            }
                    }
        }
    size_t n = gdr2_dla_bwd_workspace_bytes(2, 7777, 6, 64, 128, GDR2_BF16);
    CHECK(n > 0);
#define BWD(ws, bytes) gdr2_dla_bwd(2, 7777, 6, 64, 128, GDR2_BF16, A(0), A(1), A(2), F(3), F(4), I(5), A(6), F(7), A(8), A(9), A(10), F(11), ws, bytes, nullptr)
    EXPECT(BWD(W(12, n), n), GDR2_OK);
    EXPECT(BWD(W(12, n), n - 1), GDR2_E_WORKSPACE);
    EXPECT(BWD(nullptr, n), GDR2_E_WORKSPACE);
    n = gdr2_paged_decode_workspace_bytes(2, 8, 2, 64, 16, 100);
    CHECK(n > 0);
#define STEP(ws, bytes) gdr2_paged_decode_step(2, 8, 2, 64, GDR2_BF16, 16, 200, 100, 1.f, A(0), A(1), A(2), I(3), I(4), A(5), A(6), A(7), ws, bytes, nullptr)
    EXPECT(STEP(W(8, n), n), GDR2_OK);
    EXPECT(STEP(W(8, n), n - 1), GDR2_E_WORKSPACE);
    EXPECT(gdr2_rms_norm_fwd(3, 64, GDR2_BF16, A(0), nullptr, F(1), 1e-6f, nullptr, A(2), nullptr, nullptr), GDR2_OK);
    EXPECT(gdr2_rms_norm_fwd(3, 64, GDR2_BF16, A(0), nullptr, F(1), 0.f, nullptr, A(2), nullptr, nullptr), GDR2_E_VALUE);
    EXPECT(gdr2_dla_step(4, 3, 64, 64, GDR2_BF16, A(0), A(1), A(2), F(3), nullptr, F(4), A(5), nullptr), GDR2_OK);
    CHECK(g_launches > 100);
    if (g_fail) return 1;
    std::printf("ok %ld launches\n", g_launches);
    return 0;
}

// Host-only driver for the C ABI of the operators around the mixer under AddressSanitizer and
// UndefinedBehaviorSanitizer: gdr2_block_api.hip compiled as plain C++ against launch stand-ins that
// check what a launch would be given (positive sizes, parts inside the workspace) and touch no memory.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "gdr2.h"
#include "gdr2_block_kernels.hpp"

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
// stand-ins for the two sizing rules that live beside their kernels
long norm_bwd_blocks(long rows, int) { return rows < 512 ? rows : 512; }
int swa_decode_splits(long N, long Hkv, long groups, long slots) {
    const long jobs = N * Hkv * groups, steps = (slots + 127) / 128, want = jobs > 0 ? 512 / jobs : 1;
    const long s = want < steps ? want : steps;
    return (int)(s < 1 ? 1 : s);
}
hipError_t norm_dispatch(int, bool bwd, const NormParams& p, hipStream_t) {
    ++g_launches;
    CHECK(p.D >= 8 && p.D <= kNormMaxD && p.rows >= 0);
    if (bwd) CHECK(inside(p.part, (size_t)norm_bwd_blocks(p.rows, p.D) * 2 * p.D * 4));
    return hipSuccess;
}
hipError_t glr_dispatch(int, bool bwd, const GlrParams& p, hipStream_t) {
    ++g_launches;
    CHECK(p.nseg >= 1 && p.nstrip >= 1 && (int64_t)p.B * p.nseg * p.nstrip <= 0x7fffffff);
    const size_t words = (size_t)p.B * (p.nseg + p.nseg / kGlrGroup) * p.nstrip * kGlrCh;
    if (p.nseg > 1) CHECK(inside(p.pub, words * 8) && inside(p.ticket, 4));
    if (!bwd) CHECK(inside(p.states, (size_t)p.B * glr_segments(p.T, kGlrBwdSeg) * p.D * 4));
    return hipSuccess;
}
hipError_t glr_step_dispatch(int, const GlrStepParams& p, hipStream_t) {
    ++g_launches;
    CHECK(p.n > 0 && p.n % 8 == 0);
    return hipSuccess;
}
hipError_t swa_fwd_dispatch(int, const SwaParams& p, hipStream_t) {
    ++g_launches;
    CHECK(p.window >= 1 && p.window <= p.T && p.H % p.Hkv == 0);
    return hipSuccess;
}
hipError_t swa_bwd_dispatch(int, const SwaParams& p, hipStream_t) {
    ++g_launches;
    const size_t bk = (size_t)p.B * p.Hkv;
    CHECK(inside(p.delta, (size_t)p.B * p.H * p.T * 4));
    CHECK(inside(p.sink_part, (size_t)p.pieces * bk * 2 * kSwaMaxSinks * p.d * 4));
    CHECK(inside(p.key_part, (size_t)p.splits * 2 * bk * p.part_rows * p.d * 4));
    CHECK(p.splits >= 1 && p.pieces >= 0 && p.part_rows <= p.T);
    // the pieces cover the far queries, and none starts behind the end
    if (p.pieces) {
        CHECK(p.far0 + (long)p.pieces * p.piece_len >= p.T && p.far0 + (long)(p.pieces - 1) * p.piece_len < p.T);
        CHECK(p.piece_len % 64 == 0 && p.far0 % 64 == 0 && p.far0 >= kSwaKeyTile - 1 + p.window && p.part_rows >= p.sinks);
    }
    if (p.splits > 1) CHECK(p.part_rows == p.T);
    return hipSuccess;
}
hipError_t swa_fill_dispatch(const SwaFillParams& p, hipStream_t) {
    ++g_launches;
    CHECK((p.B * (p.window + p.sinks) * p.row16 + 255) / 256 <= 0x7fffffff);
    return hipSuccess;
}
hipError_t swa_decode_dispatch(int, const SwaDecodeParams& p, hipStream_t) {
    ++g_launches;
    const size_t jobs = (size_t)p.N * p.Hkv * ((p.H / p.Hkv + 15) / 16);
    CHECK(p.splits >= 1 && jobs * p.splits <= 0x7fffffff);
    if (p.splits > 1) CHECK(inside(p.part, jobs * p.splits * 16 * (p.d + 4) * 4));
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
static void* W(int i, size_t n) {
    g_ws = (uintptr_t)A(i);
    g_ws_end = g_ws + n;
    return A(i);
}

int main() {
    const int64_t big[] = {0, 1, 7, 64, 4096, 1 << 20, (int64_t)1 << 31, (int64_t)1 << 40, INT64_MAX};
    // every size query and call over a grid of sizes, products that overflow 64 bits among them: no
    // sanitizer report, and a workspace of the queried size always holds what a launch is given
    for (int64_t a : big)
        for (int64_t b : big)
            for (int64_t c : {(int64_t)8, (int64_t)64, (int64_t)1024, (int64_t)1 << 20, INT64_MAX}) {
                size_t n = gdr2_layer_norm_bwd_workspace_bytes(a, c);
                (void)gdr2_layer_norm_bwd(a, c, GDR2_BF16, A(0), F(1), F(2), F(3), A(4), A(5), F(6), F(7), W(8, n), n, nullptr);
                n = gdr2_glr_fwd_workspace_bytes(a, b, c);
                const size_t f = n;
                (void)gdr2_glr_fwd(a, b, c, GDR2_BF16, A(0), F(1), F(2), A(3), F(4), W(5, n), n, nullptr);
                n = gdr2_glr_bwd_workspace_bytes(a, b, c);
                (void)gdr2_glr_bwd(a, b, c, GDR2_F32, A(0), F(1), A(2), f, A(3), F(4), A(5), F(6), F(7), W(8, n), n, nullptr);
                (void)gdr2_glr_step(a, c, GDR2_F32, A(0), F(1), F(2), F(2), A(3), nullptr);
                for (int64_t H : {(int64_t)1, (int64_t)12, (int64_t)1 << 40})
                    for (int64_t Hkv : {(int64_t)1, (int64_t)4, (int64_t)0})
                        for (int64_t win : {(int64_t)1, (int64_t)500, INT64_MAX})
                            for (int64_t s : {(int64_t)0, (int64_t)64}) {
                                n = gdr2_swa_bwd_workspace_bytes(a, b, H, Hkv, 64, win, s);
                                (void)gdr2_swa_fwd(a, b, H, Hkv, 64, GDR2_BF16, win, s, 1.f, A(0), A(1), A(2), nullptr, A(3), F(4), nullptr);
                                (void)gdr2_swa_bwd(a, b, H, Hkv, 64, GDR2_BF16, win, s, 1.f, A(0), A(1), A(2), nullptr, A(3), F(4), A(5), A(6), A(7), A(8), W(9, n), n, nullptr);
                                (void)gdr2_swa_cache_fill(a, b, Hkv, 128, GDR2_F32, win, s, A(0), A(1), nullptr, A(2), A(3), nullptr);
                                n = gdr2_swa_decode_workspace_bytes(a, H, Hkv, 128, win, s);
                                (void)gdr2_swa_decode_step(a, H, Hkv, 128, GDR2_F32, win, s, 1.f, A(0), A(1), A(2), A(3), A(4), (int32_t*)A(5), A(6), W(7, n), n, nullptr);
                            }
            }
    size_t n = gdr2_swa_bwd_workspace_bytes(2, 777, 6, 2, 64, 256, 8);
    EXPECT(gdr2_swa_bwd(2, 777, 6, 2, 64, GDR2_F32, 256, 8, 1.f, A(0), A(1), A(2), nullptr, A(3), F(4), A(5), A(6), A(7), A(8), W(9, n), n, nullptr), GDR2_OK);
    EXPECT(gdr2_swa_bwd(2, 777, 6, 2, 64, GDR2_F32, 256, 8, 1.f, A(0), A(1), A(2), nullptr, A(3), F(4), A(5), A(6), A(7), A(8), W(9, n), n - 1, nullptr), GDR2_E_WORKSPACE);
    EXPECT(gdr2_layer_norm_fwd(3, 64, GDR2_BF16, A(0), F(1), nullptr, 1e-5f, A(2), nullptr, nullptr, nullptr), GDR2_OK);
    EXPECT(gdr2_layer_norm_fwd(3, 64, GDR2_BF16, A(0), F(1), nullptr, -1.f, A(2), nullptr, nullptr, nullptr), GDR2_E_VALUE);
    EXPECT(gdr2_glr_step(4, 64, GDR2_BF16, A(0), F(1), nullptr, F(2), A(3), nullptr), GDR2_OK);
    CHECK(g_launches > 100);
    if (g_fail) return 1;
    std::printf("ok %ld launches\n", g_launches);
    return 0;
}

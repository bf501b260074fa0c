// The launches that libgdr2.so makes for the residual stream's RMS norm, linear attention with a decay and the paged
// cache, seen from a host without a GPU: the runtime's entry points, and the checks that every launch passes, are those of
// launch_driver.cpp.  Checked here: the launches of one call cover the problem once, in order, and all that a grid writes
// of the workspace lies in what the size query returned.
#define main main_of_the_operators_around_the_mixer
#include "launch_driver.cpp"
#undef main

#include "gdr2_hybrid_kernels.hpp"

static int32_t* I(int i) { return (int32_t*)A(i); }
static int64_t g_rows_per, g_n, g_stage, g_group;

static void rms() {
    struct Case { int64_t rows, D, per; };  // rows of a workgroup of 512 threads, counted from D apart from the library
    for (Case c : {Case{1, 8, 64}, Case{4099, 1000, 8}, Case{((int64_t)1 << 31) - 1, 8, 64}, Case{((int64_t)1 << 26) + 1, 1024, 8}, Case{((int64_t)1 << 25) + 3, 2048, 4},
                   Case{(int64_t)1 << 24, 4096, 2}, Case{((int64_t)1 << 23) + 1, 8192, 1}, Case{((int64_t)1 << 23) + 5, 16384, 1}})
        for (gdr2_dtype dt : {GDR2_BF16, GDR2_F32})
            for (int64_t group : {-1, 0, 128}) {  // -1: the plain result
                g_call = text("rms_norm", {c.rows, c.D, dt, group});
                g_done = 0, g_D = c.D, g_es = dt == GDR2_BF16 ? 2 : 4, g_rows_per = c.per, g_group = group;
                g_seen = [](const Launch& l) {
                    const auto& p = params<gdr2::RmsParams>(l);
                    CHECK(is(l, "rms_fwd") && p.D == g_D && p.rows > 0 && l.block.x == 512);
                    CHECK((const char*)p.x == (const char*)A(0) + g_done * g_D * g_es);
                    CHECK((const char*)p.residual == (const char*)A(1) + g_done * g_D * g_es);
                    CHECK((const char*)p.h == (const char*)A(3) + g_done * g_D * g_es);
                    CHECK((const char*)p.y == (const char*)A(4) + g_done * g_D * (g_group < 0 ? g_es : 1));
                    CHECK((g_group < 0 ? p.rstd : p.scale) == F(5) + g_done * (g_group > 0 ? (g_D + g_group - 1) / g_group : 1));
                    CHECK((int64_t)l.grid.x == (p.rows + g_rows_per - 1) / g_rows_per);
                    g_done += p.rows;
                };
                const gdr2_status st = group < 0 ? LIB(gdr2_rms_norm_fwd)(c.rows, c.D, dt, A(0), A(1), F(2), 1e-6f, A(3), A(4), F(5), nullptr)
                                                 : LIB(gdr2_rms_norm_q8_fwd)(c.rows, c.D, dt, group, A(0), A(1), F(2), 1e-6f, A(3), A(4), F(5), nullptr);
                CHECK(st == GDR2_OK && g_done == c.rows);
            }
    for (int64_t D : {8, 72, 504, 1000, 2048, 4096, 16384})
        for (int64_t rows : {(int64_t)0, (int64_t)1, (int64_t)63, (int64_t)4099, (int64_t)100000, ((int64_t)1 << 31) - 1}) {
            g_call = text("rms_norm_bwd", {rows, D});
            const size_t n = LIB(gdr2_rms_norm_bwd_workspace_bytes)(rows, D);
            g_D = D, g_parts = 0, g_stage = 0;
            g_seen = [](const Launch& l) {
                const auto& p = params<gdr2::RmsParams>(l);
                if (is(l, "rms_reduce")) {
                    CHECK(*(long*)l.args[1] == g_parts && (int64_t)l.grid.x == (g_D + 63) / 64);
                    ++g_stage;
                    return;
                }
                CHECK(is(l, "rms_bwd") && g_parts == 0 && g_stage == 0);
                g_parts = l.grid.x;  // a row of D sums each
                CHECK(inside(p.part, g_parts * g_D * 4));
            };
            CHECK(LIB(gdr2_rms_norm_bwd)(rows, D, GDR2_BF16, A(0), F(1), F(2), A(3), A(4), A(5), F(6), W(7, n), n, nullptr) == GDR2_OK);
            CHECK(g_stage == 1 && (g_parts > 0) == (rows > 0));
        }
}

static int64_t g_dkdv;
static int g_passes;
// One launch of segments' own states where there are any, then one of everything.
static void dla_seen(const Launch& l) {
    const auto& p = params<gdr2::DlaParams>(l);
    const bool local = is(l, "Li0ELb1") || is(l, "Li64ELb1") || is(l, "Li128ELb1");  // <..., columns or 0, LOCAL, ...>
    if (is(l, "gdr2_dla_kernel")) CHECK(is(l, "ELb0ELb1E") == (p.T <= 128) && l.block.x >= 256u + 2 * p.pass[0].V);  // short sequences' own variant; waves
    const int64_t per = g_B * g_H * g_slots, n = *(int*)l.args[1];
    CHECK(is(l, "gdr2_dla_") && p.passes == g_passes && p.slots == g_slots && p.T == g_T);
    CHECK(p.segs >= 1 && p.seg_chunks >= 1 && (int64_t)p.segs * p.seg_chunks * 64 >= p.T);
    CHECK(p.segs == 1 || (int64_t)(p.segs - 1) * p.seg_chunks * 64 < p.T);
    CHECK(local ? g_stage == 0 && p.segs > 1 : g_stage == (p.segs > 1 ? 1 : 0));
    CHECK(n == per * (local ? p.segs - 1 : p.segs) && (int64_t)l.grid.x >= n && l.grid.x % 8 == 0 && l.grid.x < n + 8);
    CHECK(inside(p.local, p.passes * g_B * g_H * (p.segs - 1) * g_dkdv * 4));
    g_stage = local ? 1 : 2;
}
static void dla() {
    struct Case { int64_t B, T, H; };
    for (Case c : {Case{1, 0, 1}, Case{1, 1, 1}, Case{1, 64, 3}, Case{3, 777, 6}, Case{4, 4096, 16}, Case{1, 32768, 16}, Case{1, (int64_t)1 << 29, 1}, Case{1, ((int64_t)1 << 30) - 128, 1},
                   Case{16, 64, 32768}, Case{1 << 19, 1, 1}, Case{1 << 19, (int64_t)30 * 64, 1}, Case{2, 100000, 300}})
        for (gdr2_dtype dt : {GDR2_BF16, GDR2_F32})
            for (int64_t dk : {64, 128})
                for (int64_t dv : {64, 128}) {
                    auto slots = [&](int64_t columns) { return dt == GDR2_BF16 ? 1 : columns / 32; };  // workgroups of a pass
                    g_B = c.B, g_T = c.T, g_H = c.H, g_dkdv = dk * dv;
                    g_seen = dla_seen;
                    g_call = text("dla_fwd", {c.B, c.T, c.H, dk, dv, dt});
                    g_passes = 1, g_slots = slots(dv), g_stage = 0;
                    size_t n = LIB(gdr2_dla_fwd_workspace_bytes)(c.B, c.T, c.H, dk, dv, dt);
                    CHECK(LIB(gdr2_dla_fwd)(c.B, c.T, c.H, dk, dv, dt, A(0), A(1), A(2), F(3), F(4), I(5), A(6), F(7), W(8, n), n, nullptr) == GDR2_OK);
                    CHECK(g_stage == 2);
                    g_call = text("dla_bwd", {c.B, c.T, c.H, dk, dv, dt});
                    g_passes = 3, g_slots = slots(dv) + 2 * slots(dk), g_stage = 0;
                    n = LIB(gdr2_dla_bwd_workspace_bytes)(c.B, c.T, c.H, dk, dv, dt);
                    CHECK(LIB(gdr2_dla_bwd)(c.B, c.T, c.H, dk, dv, dt, A(0), A(1), A(2), F(3), F(4), I(5), A(6), F(7), A(8), A(9), A(10), F(11), W(12, n), n, nullptr) == GDR2_OK);
                    CHECK(g_stage == 2);
                }
    for (int64_t n : {(int64_t)1, (int64_t)4096, ((int64_t)1 << 24) - 1}) {
        g_call = text("dla_step", {n});
        g_n = n, g_done = 0;
        g_seen = [](const Launch& l) {
            CHECK(is(l, "dla_step") && (int64_t)l.grid.x == g_n);
            ++g_done;
        };
        CHECK(LIB(gdr2_dla_step)(n, 1, 128, 64, GDR2_BF16, A(0), A(1), A(2), F(3), F(4), F(4), A(5), nullptr) == GDR2_OK && g_done == 1);
    }
}

static int64_t g_heads, g_d, g_width;
static void paged() {
    struct Case { int64_t N, H, Hkv, page, width; };
    for (Case c : {Case{1, 16, 4, 64, 512}, Case{256, 16, 4, 16, 256}, Case{13, 12, 4, 32, 87}, Case{1, 1, 1, 1, 0}, Case{3, 32, 1, 1, 1000}, Case{64, 16, 4, 16, 24}, Case{64, 16, 4, 16, 25},
                   Case{1024, 1, 1, 1024, 1024}, Case{(int64_t)1 << 24, 64, 64, 16, 4}, Case{((int64_t)1 << 24) + 9, 1, 1, 16, 4}, Case{1, 32768, 32768, 16, 1000}, Case{2, 32768, 1, 16, 1000}})
        for (gdr2_dtype dt : {GDR2_BF16, GDR2_F32})
            for (int64_t d : {64, 128}) {
                g_call = text("paged_decode", {c.N, c.H, c.Hkv, c.page, c.width, dt, d});
                g_es = dt == GDR2_BF16 ? 2 : 4, g_n = c.N, g_heads = c.H, g_Hkv = c.Hkv, g_d = d, g_width = c.width, g_done = 0, g_stage = 0;
                const size_t n = LIB(gdr2_paged_decode_workspace_bytes)(c.N, c.H, c.Hkv, d, c.page, c.width);
                g_seen = [](const Launch& l) {
                    const auto& p = params<gdr2::PagedDecodeParams>(l);
                    const int64_t groups = (g_heads / g_Hkv + 15) / 16, jobs = p.N * g_Hkv * groups;
                    if (is(l, "paged_join")) {
                        CHECK(g_done == g_n && p.N == g_n && p.splits > 1 && (int64_t)l.grid.x == g_n * g_heads);
                        ++g_stage;
                        return;
                    }
                    CHECK(is(l, "paged_decode") && (int64_t)l.grid.x == jobs * p.splits && p.N > 0);
                    CHECK((const char*)p.q == (const char*)A(0) + g_done * g_heads * g_d * g_es && (const char*)p.o == (const char*)A(7) + g_done * g_heads * g_d * g_es);
                    CHECK((const char*)p.k == (const char*)A(1) + g_done * g_Hkv * g_d * g_es && (const char*)p.v == (const char*)A(2) + g_done * g_Hkv * g_d * g_es);
                    CHECK(p.table == I(3) + g_done * g_width && p.pos == I(4) + g_done);
                    if (p.splits > 1) CHECK(p.N == g_n && inside(p.part, jobs * p.splits * 16 * (g_d + 4) * 4));
                    else CHECK(g_ws == g_ws_end);
                    g_done += p.N;
                };
                CHECK(LIB(gdr2_paged_decode_step)(c.N, c.H, c.Hkv, d, dt, c.page, 1000, c.width, 1.f, A(0), A(1), A(2), I(3), I(4), A(5), A(6), A(7), W(8, n), n, nullptr) == GDR2_OK);
                CHECK(g_done == c.N && g_stage == (n ? 1 : 0));
            }
    struct Fill { int64_t B, T, Hkv; };
    for (Fill c : {Fill{1, 1, 1}, Fill{4, 4096, 4}, Fill{3, 777, 5}, Fill{2, (int64_t)1 << 30, 2}, Fill{(int64_t)1 << 30, 2, 2}, Fill{((int64_t)1 << 31) - 1, 1, 2}})
        for (gdr2_dtype dt : {GDR2_BF16, GDR2_F32}) {
            g_call = text("paged_fill", {c.B, c.T, c.Hkv, dt});
            g_done = 0, g_n = c.B * c.T * c.Hkv * 128 * (dt == GDR2_BF16 ? 2 : 4) / 16;
            g_seen = [](const Launch& l) {
                const auto& p = params<gdr2::PagedFillParams>(l);
                CHECK(is(l, "paged_fill") && p.first == g_done && p.n == g_n && l.block.x == 256);
                g_done = p.first + (int64_t)l.grid.x * 256;
            };
            CHECK(LIB(gdr2_paged_cache_fill)(c.B, c.T, c.Hkv, 128, dt, 16, 1000, 4, A(0), A(1), I(2), I(3), I(4), A(5), A(6), nullptr) == GDR2_OK);
            CHECK(g_done >= g_n && g_done < g_n + 256);
        }
}

int main(int argc, char** argv) {
    g_lib = argc > 1 ? dlopen(argv[1], RTLD_NOW) : nullptr;
    if (!g_lib) {
        std::printf("FAIL: %s\n", dlerror());
        return 1;
    }
    rms();
    dla();
    paged();
    if (g_fail) return 1;
    std::printf("ok %ld launches\n", g_launches);
    return 0;
}

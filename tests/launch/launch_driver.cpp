// The launches that libgdr2.so makes for the operators around the mixer, seen from a host without a GPU:
// this program defines the runtime's launch and registration entry points itself, so the library,
// loaded as built, hands every launch to the checks below and nothing runs.  Checked of each launch:
// HIP's limit of 2^32 - 1 work items, per operator that the launches of one call cover the problem
// once, in order, and that all a launch's grid writes of the workspace lies in what the size query
// returned (each kernel's needs are counted here from its grid, apart from the library's layouts).
#include <dlfcn.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <string>

#include "gdr2.h"
#include "gdr2_block_kernels.hpp"

static int g_fail = 0;
#define CHECK(c)                                                                   \
    do {                                                                           \
        if (!(c)) {                                                                \
            std::printf("FAIL line %d: %s  [%s]\n", __LINE__, #c, g_call.c_str()); \
            ++g_fail;                                                              \
        }                                                                          \
    } while (0)
static std::string g_call = "load";

// ---------------------------------------------------------------- the runtime's entry points
struct Launch {
    std::string name;  // the kernel's (mangled) name
    dim3 grid, block;
    void** args;
};
static std::map<const void*, std::string> g_names;
static void (*g_seen)(const Launch&) = nullptr;
static long g_launches = 0;
static dim3 g_grid, g_block;
static size_t g_shm;
static hipStream_t g_stream;

extern "C" {
static void* g_module;
void** __hipRegisterFatBinary(const void*) { return &g_module; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, dim3*, dim3*, int*) {
    g_names[host] = name;
}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shm, hipStream_t s) {
    g_grid = grid, g_block = block, g_shm = shm, g_stream = s;
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shm, hipStream_t* s) {
    *grid = g_grid, *block = g_block, *shm = g_shm, *s = g_stream;
    return hipSuccess;
}
hipError_t hipGetLastError(void) { return hipSuccess; }
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t, hipStream_t) {
    ++g_launches;
    const Launch l{g_names.count(f) ? g_names[f] : "?", grid, block, args};
    CHECK(l.name != "?");
    CHECK(grid.x >= 1 && grid.y >= 1 && grid.z == 1 && block.x >= 1 && block.x <= 1024 && block.y == 1 && block.z == 1);
    CHECK((uint64_t)grid.x * block.x < (uint64_t)1 << 32 && grid.y < 65536);  // work items
    if (g_seen) g_seen(l);
    return hipSuccess;
}
}

static bool is(const Launch& l, const char* part) { return l.name.find(part) != std::string::npos; }
template <typename P>
static const P& params(const Launch& l) {
    return *(const P*)l.args[0];
}

// ---------------------------------------------------------------- the library
static void* g_lib;
template <typename F>
static F* fn(const char* name) {
    void* p = dlsym(g_lib, name);
    if (!p) {
        std::printf("FAIL: %s is not exported\n", name);
        std::exit(1);
    }
    return (F*)p;
}
#define LIB(name) fn<decltype(name)>(#name)
// addresses far apart, never dereferenced
static void* A(int i) { return (void*)((uintptr_t)(i + 1) << 48); }
static float* F(int i) { return (float*)A(i); }
static std::string text(const char* f, std::initializer_list<int64_t> v) {
    std::string s = f;
    for (int64_t x : v) s += " " + std::to_string(x);
    return s;
}

static uintptr_t g_ws, g_ws_end;  // the workspace of the running call: W(i, queried bytes)
static void* W(int i, size_t n) {
    g_ws = (uintptr_t)A(i);
    g_ws_end = g_ws + n;
    return A(i);
}
static bool inside(const void* p, int64_t n) { return n == 0 || (n > 0 && (uintptr_t)p >= g_ws && (uintptr_t)p + n <= g_ws_end); }
static bool apart(const void* p, int64_t n, const void* q, int64_t m) {
    return n == 0 || m == 0 || (uintptr_t)p + n <= (uintptr_t)q || (uintptr_t)q + m <= (uintptr_t)p;
}

static int64_t g_done;      // rows, batch rows, sequences or pieces covered so far by the call's launches
static int64_t g_D, g_T, g_es;

static void norm_fwd() {
    struct Case { int64_t rows, D; };
    for (Case c : {Case{1, 8}, Case{4099, 1000}, Case{(int64_t)1 << 29, 8}, Case{((int64_t)1 << 31) - 1, 8}, Case{(int64_t)1 << 26, 512},
                   Case{((int64_t)1 << 26) + 1, 1024}, Case{((int64_t)1 << 25) + 3, 2048}, Case{(int64_t)1 << 24, 4096}, Case{((int64_t)1 << 23) + 1, 8192}, Case{(int64_t)1 << 23, 16384}})
        for (gdr2_dtype dt : {GDR2_BF16, GDR2_F32}) {
            g_call = text("layer_norm_fwd", {c.rows, c.D, dt});
            g_done = 0, g_D = c.D, g_es = dt == GDR2_BF16 ? 2 : 4;
            g_seen = [](const Launch& l) {
                const auto& p = params<gdr2::NormParams>(l);
                CHECK(is(l, "norm_fwd") && p.D == g_D && p.rows > 0);
                CHECK((const char*)p.x == (const char*)A(0) + g_done * g_D * g_es);
                CHECK((const char*)p.y == (const char*)A(3) + g_done * g_D * g_es);
                CHECK(p.mean == F(4) + g_done && p.rstd == nullptr && p.weight == F(1) && p.bias == F(2));
                // rows of a workgroup (512 threads): 64 / 32 / 16 / 8 / 8 / 4 / 2 / 1
                const int64_t lanes = g_D <= 64 ? 8 : g_D <= 128 ? 16 : g_D <= 256 ? 32 : 64;
                const int64_t waves = g_D <= 1024 ? 1 : g_D <= 2048 ? 2 : g_D <= 4096 ? 4 : 8, R = 8 / waves * (64 / lanes);
                CHECK(l.block.x == 512 && (int64_t)l.grid.x == (p.rows + R - 1) / R);
                g_done += p.rows;
            };
            CHECK(LIB(gdr2_layer_norm_fwd)(c.rows, c.D, dt, A(0), F(1), F(2), 1e-5f, A(3), F(4), nullptr, nullptr) == GDR2_OK);
            CHECK(g_done == c.rows);
        }
}

static int64_t g_parts;
static void norm_bwd() {
    for (int64_t D : {8, 64, 72, 128, 256, 512, 1000, 2048, 4096, 8192, 16384})
        for (int64_t rows : {(int64_t)0, (int64_t)1, (int64_t)63, (int64_t)511, (int64_t)4099, (int64_t)16384, (int64_t)100000, ((int64_t)1 << 31) - 1})
            for (bool bias : {false, true}) {
                g_call = text("layer_norm_bwd", {rows, D, bias});
                const size_t n = LIB(gdr2_layer_norm_bwd_workspace_bytes)(rows, D);
                g_D = D, g_parts = 0;
                g_seen = [](const Launch& l) {
                    const auto& p = params<gdr2::NormParams>(l);
                    if (is(l, "norm_reduce")) {  // columns of 64, one or two rows of them, over the parts just written
                        CHECK(*(long*)l.args[1] == g_parts && (int64_t)l.grid.x == (g_D + 63) / 64 && l.grid.y == (p.dbias ? 2 : 1));
                        return;
                    }
                    CHECK(is(l, "norm_bwd") && p.D == g_D && g_parts == 0);
                    g_parts = l.grid.x;  // every workgroup writes two rows of D sums
                    CHECK(inside(p.part, g_parts * 2 * g_D * 4));
                };
                const long before = g_launches;
                CHECK(LIB(gdr2_layer_norm_bwd)(rows, D, GDR2_BF16, A(0), F(1), F(2), F(3), A(4), A(5), F(6), bias ? F(7) : nullptr, W(8, n), n, nullptr) == GDR2_OK);
                CHECK(g_launches == before + (rows ? 2 : 1));
            }
}

static void glr() {
    struct Case { int64_t B, T, D; };
    for (Case c : {Case{1, 1, 8}, Case{3, 300, 136}, Case{(int64_t)1 << 23, 1, 8}, Case{((int64_t)1 << 30) + 1, 1, 8}, Case{((int64_t)1 << 20), 256, 1024},
                   Case{(int64_t)1 << 16, 257, 8192}, Case{((int64_t)1 << 23) + 1, 300, 8}, Case{3, (int64_t)1 << 30, 64}, Case{1, ((int64_t)1 << 31) - 256, 64}, Case{2, 1 << 20, 1 << 16}})
        for (bool bwd : {false, true}) {
            g_call = text(bwd ? "glr_bwd" : "glr_fwd", {c.B, c.T, c.D});
            const size_t f = LIB(gdr2_glr_fwd_workspace_bytes)(c.B, c.T, c.D), n = LIB(gdr2_glr_bwd_workspace_bytes)(c.B, c.T, c.D);
            CHECK(f > 0);
            g_done = 0, g_D = c.D, g_T = c.T;
            g_seen = [](const Launch& l) {
                if (is(l, "glr_clear")) {  // words and ticket of the launch behind it
                    CHECK(inside(*(void**)l.args[0], *(long*)l.args[1] * 8) && inside(*(void**)l.args[2], 4));
                    g_parts = *(long*)l.args[1];
                    return;
                }
                const auto& p = params<gdr2::GlrParams>(l);
                const bool back = is(l, "glr_bwd");
                const int64_t seg = back ? 128 : 256, first = g_done * g_T * g_D;
                CHECK((back || is(l, "glr_fwd")) && p.T == g_T && p.D == g_D && p.B > 0);
                CHECK(p.nseg == (g_T + seg - 1) / seg && p.nstrip == (g_D + 63) / 64);
                CHECK((int64_t)l.grid.x == (int64_t)p.B * p.nseg * p.nstrip && l.block.x == 2 * seg);
                CHECK(p.x == (const char*)A(0) + 2 * first && p.la == F(1) + first);
                CHECK(p.states == F(5) + g_done * ((g_T + 127) / 128) * g_D);
                if (p.nseg > 1) {  // one word per segment and channel of a strip, one per 16 whole segments
                    const int64_t words = (int64_t)p.B * (p.nseg + p.nseg / 16) * p.nstrip * 64;
                    CHECK(words == g_parts && inside(p.pub, words * 8) && inside(p.ticket, 4) && apart(p.pub, words * 8, p.ticket, 4));
                }
                if (!back) {
                    const int64_t kept = (int64_t)p.B * ((g_T + 127) / 128) * g_D * 4;
                    CHECK(inside(p.states, kept));
                    if (p.nseg > 1) CHECK(apart(p.states, kept, p.pub, g_parts * 8) && apart(p.states, kept, p.ticket, 4));
                }
                if (back) CHECK(p.dh == (char*)A(3) + 2 * first && p.dhT == F(4) + g_done * g_D && p.dx == (char*)A(6) + 2 * first && p.dla == F(7) + first && p.dh0 == F(8) + g_done * g_D);
                else CHECK(p.h0 == F(2) + g_done * g_D && p.h == (char*)A(3) + 2 * first && p.hT == F(4) + g_done * g_D);
                g_done += p.B;
            };
            if (bwd) CHECK(LIB(gdr2_glr_bwd)(c.B, c.T, c.D, GDR2_BF16, A(0), F(1), A(5), f, A(3), F(4), A(6), F(7), F(8), W(9, n), n, nullptr) == GDR2_OK);
            else CHECK(LIB(gdr2_glr_fwd)(c.B, c.T, c.D, GDR2_BF16, A(0), F(1), F(2), A(3), F(4), W(5, f), f, nullptr) == GDR2_OK);
            CHECK(g_done == c.B);
        }
    g_call = "glr: one batch row beyond a launch";
    g_seen = nullptr;
    const long before = g_launches;
    CHECK(LIB(gdr2_glr_fwd_workspace_bytes)(1, ((int64_t)1 << 31) - 256, 8) > 0 && LIB(gdr2_glr_bwd_workspace_bytes)(1, ((int64_t)1 << 31) - 256, 8) > 0);
    CHECK(LIB(gdr2_glr_fwd_workspace_bytes)(1, ((int64_t)1 << 31) - 255, 8) == 0);
    CHECK(LIB(gdr2_glr_fwd_workspace_bytes)(1, (int64_t)1 << 32, 64 << 8) == 0 && LIB(gdr2_glr_bwd_workspace_bytes)(1, (int64_t)1 << 32, 64 << 8) == 0);
    CHECK(LIB(gdr2_glr_fwd)(1, (int64_t)1 << 32, 64 << 8, GDR2_BF16, A(0), F(1), F(2), A(3), F(4), A(5), SIZE_MAX, nullptr) == GDR2_E_SHAPE);
    for (int64_t n : {(int64_t)1, (int64_t)1 << 31, (int64_t)1 << 32, (int64_t)1 << 36}) {
        g_call = text("glr_step", {n});
        const gdr2_status st = LIB(gdr2_glr_step)(n, 8, GDR2_BF16, A(0), F(1), nullptr, F(2), A(3), nullptr);
        CHECK(st == (n * 8 <= (int64_t)1 << 34 ? GDR2_OK : GDR2_E_SHAPE));
    }
    CHECK(g_launches == before + 2);
}

static int64_t g_H, g_Hkv, g_slots;
static void decode() {
    struct Case { int64_t N, H, Hkv, window, sinks; };
    for (Case c : {Case{1, 4, 1, 4096, 4}, Case{1, 1, 1, 1, 0}, Case{1, 40, 1, 1 << 20, 64}, Case{3, 4, 2, 129, 0}, Case{24, 16, 4, 8192, 0}, Case{40, 8, 4, 8192, 0},
                   Case{47, 16, 4, 2048, 4}, Case{48, 16, 4, 2048, 4}, Case{64, 16, 4, 2048, 4}, Case{191, 17, 1, 900, 0}, Case{192, 1, 1, 900, 0}, Case{256, 16, 4, 2048, 4}, Case{(int64_t)1 << 24, 1, 1, 1, 0}, Case{((int64_t)1 << 25) + 7, 4, 2, 1, 3},
                   Case{((int64_t)1 << 23) + 1, 34, 2, 2, 0}, Case{(int64_t)1 << 30, 1, 1, 8, 0}}) {
        g_call = text("swa_decode_step", {c.N, c.H, c.Hkv, c.window, c.sinks});
        const size_t n = LIB(gdr2_swa_decode_workspace_bytes)(c.N, c.H, c.Hkv, 64, c.window, c.sinks);
        g_done = 0, g_H = c.H, g_Hkv = c.Hkv, g_slots = c.window + c.sinks;
        g_seen = [](const Launch& l) {
            const auto& p = params<gdr2::SwaDecodeParams>(l);
            if (is(l, "decode_join")) {
                CHECK(p.splits > 1 && (int64_t)l.grid.x == p.N * g_H);
                return;
            }
            // a part: sixteen heads of a row and two statistics, the statistics 16 bytes
            if (p.splits > 1) CHECK(inside(p.part, (int64_t)l.grid.x * 16 * (64 + 4) * 4));
            const int64_t row = 64 * 2, kv = g_done * g_Hkv * row;
            CHECK(is(l, "swa_decode") && (int64_t)l.grid.x == (int64_t)p.N * g_Hkv * ((g_H / g_Hkv + 15) / 16) * p.splits);
            CHECK(p.q == (char*)A(0) + g_done * g_H * row && p.o == (char*)A(6) + g_done * g_H * row && p.k == (char*)A(1) + kv && p.v == (char*)A(2) + kv);
            CHECK(p.kc == (char*)A(3) + kv * g_slots && p.vc == (char*)A(4) + kv * g_slots && p.pos == (const int*)A(5) + g_done);
            g_done += p.N;
        };
        CHECK(LIB(gdr2_swa_decode_step)(c.N, c.H, c.Hkv, 64, GDR2_BF16, c.window, c.sinks, 1.f, A(0), A(1), A(2), A(3), A(4), (int32_t*)A(5), A(6), W(7, n), n, nullptr) == GDR2_OK);
        CHECK(g_done == c.N);
    }
}

static void fill() {
    struct Case { int64_t B, T, Hkv, window, sinks; };
    for (Case c : {Case{1, 1, 1, 1, 0}, Case{4, 4096, 16, 2048, 4}, Case{1100, 100, 8, 32768, 64}, Case{1 << 16, 3, 4, 16384, 0}, Case{2, 100, 2, 1 << 30, 0}}) {
        g_call = text("swa_cache_fill", {c.B, c.T, c.Hkv, c.window, c.sinks});
        g_done = 0;
        g_seen = [](const Launch& l) {
            const auto& p = params<gdr2::SwaFillParams>(l);
            CHECK(is(l, "swa_fill") && p.first == g_done && l.block.x == 256);
            g_done += (int64_t)l.grid.x * 256;
        };
        CHECK(LIB(gdr2_swa_cache_fill)(c.B, c.T, c.Hkv, 128, GDR2_BF16, c.window, c.sinks, A(0), A(1), nullptr, A(2), A(3), nullptr) == GDR2_OK);
        const int64_t pieces = c.B * (c.window + c.sinks) * c.Hkv * 128 * 2 / 16;
        CHECK(g_done >= pieces && g_done < pieces + 256);
    }
}

static void attention() {
    // accepted sizes launch, whatever they are; no size is accepted whose launch would be refused
    for (int64_t B : {(int64_t)1, (int64_t)3, (int64_t)1 << 10, (int64_t)1 << 16, (int64_t)1 << 20, (int64_t)1 << 22, (int64_t)1 << 24})
        for (int64_t T : {(int64_t)1, (int64_t)129, (int64_t)500, (int64_t)4096, (int64_t)1 << 20, (int64_t)1 << 30})
            for (int64_t H : {(int64_t)1, (int64_t)4, (int64_t)64, (int64_t)32768})
                for (int64_t win : {(int64_t)1, (int64_t)500, (int64_t)1 << 40})
                    for (int64_t sinks : {0, 64}) {
                        g_call = text("swa", {B, T, H, win, sinks});
                        g_seen = nullptr;
                        const long before = g_launches;
                        const gdr2_status f = LIB(gdr2_swa_fwd)(B, T, H, 1, 128, GDR2_BF16, win, sinks, 1.f, A(0), A(1), A(2), nullptr, A(3), F(4), nullptr);
                        CHECK(f == GDR2_OK || f == GDR2_E_SHAPE);
                        CHECK(g_launches == before + (f == GDR2_OK));
                        const size_t n = LIB(gdr2_swa_bwd_workspace_bytes)(B, T, H, 1, 128, win, sinks);
                        const gdr2_status b = LIB(gdr2_swa_bwd)(B, T, H, 1, 128, GDR2_BF16, win, sinks, 1.f, A(0), A(1), A(2), nullptr, A(3), F(4), A(5), A(6), A(7), A(8), A(9), n, nullptr);
                        CHECK(b == GDR2_OK || b == GDR2_E_SHAPE);
                        CHECK((b == GDR2_OK) == (n > 0));
                        // what fits a card of 288 GB is accepted: q, k, v, o and their gradients
                        const double bytes = 2. * B * T * 128 * (2. * H + 2);
                        if (H <= 32768 && B * H <= 4000000 && bytes < 288e9) CHECK(f == GDR2_OK);
                        if (H <= 32768 && B * H <= 4000000 && 2 * bytes < 288e9) CHECK(b == GDR2_OK);
                    }
}

// What the backward's launches keep in the workspace, at sizes that cut keys and far queries every way.
static int64_t g_win, g_sinks, g_B;
static void attention_parts() {
    for (int64_t B : {1, 3, 40})
        for (int64_t T : {1, 63, 128, 129, 777, 1537, 4096, 8192, 32768})
            for (int64_t Hkv : {1, 3, 16})
                for (int64_t G : {1, 4})
                    for (int64_t win : {1, 64, 256, 2048, 1 << 20})
                        for (int64_t sinks : {0, 1, 33, 64}) {
                            g_call = text("swa_bwd", {B, T, Hkv * G, Hkv, win, sinks});
                            g_B = B, g_T = T, g_Hkv = Hkv, g_H = Hkv * G, g_win = win < T ? win : T, g_sinks = sinks, g_parts = 0;
                            const size_t n = LIB(gdr2_swa_bwd_workspace_bytes)(B, T, g_H, Hkv, 64, win, sinks);
                            g_seen = [](const Launch& l) {
                                const auto& p = params<gdr2::SwaParams>(l);
                                const int64_t bk = g_B * g_Hkv, tiles = (g_T + 127) / 128 * bk, sums = 64 * 4;
                                CHECK(p.T == g_T && p.window == g_win && p.sinks == g_sinks);
                                if (is(l, "swa_dq")) {
                                    const int64_t wide = (g_T + 127) / 128 * g_B * g_H, narrow = (g_T + 63) / 64 * g_B * g_H;
                                    CHECK((int64_t)l.grid.x == wide || (int64_t)l.grid.x == narrow);
                                    CHECK(inside(p.delta, g_B * g_H * g_T * 4));
                                } else if (is(l, "swa_dkv")) {
                                    const int64_t sink_wgs = p.pieces * bk, parts = ((int64_t)l.grid.x - sink_wgs) / tiles;
                                    CHECK(parts * tiles + sink_wgs == (int64_t)l.grid.x && parts == p.splits && parts >= 1);
                                    // the far queries: behind the window of the first key tile, none lost, no piece empty
                                    CHECK((p.pieces > 0) == (g_sinks > 0 && g_T > (127 + g_win + 63) / 64 * 64));
                                    if (p.pieces) CHECK(p.far0 >= 127 + g_win && p.far0 + (int64_t)p.pieces * p.piece_len >= g_T && p.far0 + (int64_t)(p.pieces - 1) * p.piece_len < g_T);
                                    // written: dk and dv of every key per part, or of the first 64 keys where the far
                                    // queries' sums are added to them; dk and dv of 64 keys per piece
                                    const int64_t rows = parts > 1 ? g_T : p.pieces ? (g_T < 64 ? g_T : 64) : 0;
                                    const int64_t keys = parts * 2 * bk * rows * sums, far = sink_wgs * 2 * 64 * sums;
                                    CHECK(p.part_rows == rows && inside(p.key_part, keys) && inside(p.sink_part, far));
                                    CHECK(apart(p.key_part, keys, p.sink_part, far) && apart(p.key_part, keys, p.delta, g_B * g_H * g_T * 4) &&
                                          apart(p.sink_part, far, p.delta, g_B * g_H * g_T * 4));
                                    g_parts = rows;
                                } else {
                                    CHECK(is(l, "swa_reduce") && g_parts > 0 && (int64_t)l.grid.x == (bk * g_parts * 16 + 255) / 256);
                                }
                            };
                            const long before = g_launches;
                            CHECK(LIB(gdr2_swa_bwd)(B, T, g_H, Hkv, 64, GDR2_F32, win, sinks, 1.f, A(0), A(1), A(2), nullptr, A(3), F(4), A(5), A(6), A(7), A(8), W(9, n), n, nullptr) == GDR2_OK);
                            CHECK(g_launches == before + (g_parts ? 3 : 2));
                        }
}

int main(int argc, char** argv) {
    g_lib = argc > 1 ? dlopen(argv[1], RTLD_NOW) : nullptr;
    if (!g_lib) {
        std::printf("FAIL: %s\n", dlerror());
        return 1;
    }
    norm_fwd();
    norm_bwd();
    glr();
    decode();
    fill();
    attention();
    attention_parts();
    if (g_fail) return 1;
    std::printf("ok %ld launches\n", g_launches);
    return 0;
}

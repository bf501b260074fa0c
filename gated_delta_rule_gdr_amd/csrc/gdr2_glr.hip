// gdr2_glr.hip -- elementwise gated linear recurrence, forward, backward and single step (gfx950).
//
// Per channel, with a_t = exp(log_a_t):
//     h_t = a_t h_{t-1} + x_t
// and, for the cotangents dh_t of h_t and dh_T of the final state, with R_{T+1} = dh_T:
//     dx_t = G_t = dh_t + R_{t+1},   R_t = a_t G_t,   dlog_a_t = R_t h_{t-1},   dh_0 = R_1
// A run of tokens is an affine map of the state that enters it (forward: h -> A h + X, backward:
// R -> A R + Y, A the product of its a_t), and maps compose, so the time axis is split at three
// levels: a thread owns four tokens of eight channels, a wave eight such runs, a workgroup
// a segment (kGlrFwdSeg or kGlrBwdSeg tokens) of kGlrCh channels.  Everything is held in fp32.
//
// The pass is a stream (9 flops per 8 or more bytes): every element is read once and written once.
// B=4 T=4096 D=2048 bf16: forward 64 us for 268 MB and the kept states (4.2 TB/s), backward 108 us for 470 MB
// (4.3 TB/s; it reads x and log_a again), and 5 us each to preset the published words; B=1 T=32749 D=1024 fp32:
// 91 us (4.4 TB/s) and 137 us (4.9 TB/s).  The step kernel (256 x 2048) takes 3 us, a launch's latency.
// Segments of one channel strip are joined inside the same launch: a workgroup publishes the map of
// its segment (A, X in one 64-bit word per channel), then reads the maps before it, at most
// kGlrGroup of them behind the last published running state, and composes them in their order, so
// the result does not depend on timing.  Workgroups take their segment from a ticket counter in
// order of the scan and publish before they wait, so a workgroup only ever waits for workgroups
// that already run and that publish without waiting for it (running states: for a chain of such
// workgroups that ends at the first segment): every wait ends whatever the order of dispatch.
// The words are preset to a pattern that no published word has.
//
// The forward keeps the state that enters each of the backward's segments (1/128 of an fp32 output); the backward
// rebuilds every h_{t-1} from it in fp32, so that dlog_a does not see the rounding of a 16-bit h.
#include "gdr2_block_kernels.hpp"
#include "gdr2_common.hpp"

namespace gdr2 {

constexpr int kGlrRun = 4;  // tokens of a thread
constexpr int kGlrWaveTok = 8 * kGlrRun;
// Waves of a workgroup.  Longer segments mean fewer joins but fewer independent workgroups: measured at
// B=4 T=4096 D=2048 bf16, 4 / 8 / 16 waves take 79 / 66 / 75 us forward and 120 / 138 / 166 us backward
// (whose threads hold three tensors' tokens instead of two).
constexpr int kGlrFwdWaves = kGlrFwdSeg / kGlrWaveTok, kGlrBwdWaves = kGlrBwdSeg / kGlrWaveTok;
static_assert(kGlrFwdSeg % kGlrBwdSeg == 0 && kGlrCh == 64, "segment mapping");
static_assert(kGlrFwdThreads == 64 * kGlrFwdWaves && kGlrBwdThreads == 64 * kGlrBwdWaves, "threads of a segment");
constexpr unsigned long long kUnpublished = ~0ull;

typedef float f32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x8 ld8(const float* p) {
    const f32x4 a = *(const f32x4*)p, b = *(const f32x4*)(p + 4);
    return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
__device__ __forceinline__ f32x8 ld8(const bf16* p) {
    return __builtin_convertvector(*(const bf16x8*)p, f32x8);
}
__device__ __forceinline__ void st8(float* p, const f32x8& v) {
    *(f32x4*)p = f32x4{v[0], v[1], v[2], v[3]};
    *(f32x4*)(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void st8(bf16* p, const f32x8& v) { *(bf16x8*)p = __builtin_convertvector(v, bf16x8); }  // RNE
// The results leave past the L2, in whole lines: nothing here reads them again (B=4 T=4096 D=2048 bf16:
// forward 68 -> 65 us, backward 119 -> 114 us).
__device__ __forceinline__ void st8s(float* p, const f32x8& v) {
    store_stream((f32x4*)p, f32x4{v[0], v[1], v[2], v[3]});
    store_stream((f32x4*)(p + 4), f32x4{v[4], v[5], v[6], v[7]});
}
__device__ __forceinline__ void st8s(bf16* p, const f32x8& v) { store_stream((bf16x8*)p, __builtin_convertvector(v, bf16x8)); }

__device__ __forceinline__ float decay(float la) { return __builtin_amdgcn_exp2f(la * 1.4426950408889634f); }

// One 64-bit word: the map's product in the high half, its offset in the low half.  A NaN product
// is published as the plain quiet NaN, so no word equals kUnpublished.
__device__ __forceinline__ unsigned long long pack_map(float A, float X) {
    const unsigned a = A != A ? 0x7fc00000u : __builtin_bit_cast(unsigned, A);
    return (unsigned long long)a << 32 | __builtin_bit_cast(unsigned, X);
}
__device__ __forceinline__ float word_hi(unsigned long long w) { return __builtin_bit_cast(float, (unsigned)(w >> 32)); }
__device__ __forceinline__ float word_lo(unsigned long long w) { return __builtin_bit_cast(float, (unsigned)w); }
__device__ __forceinline__ void publish(unsigned long long* p, unsigned long long w) {
    __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Waits of a call that has its workspace to itself end within microseconds.  The bound (some tenths of a
// second) is for a workspace that another call uses meanwhile, which the interface forbids: such calls end, and
// what they and the other call leave in their outputs and in the workspace is undefined.
constexpr int kAwaitPolls = 1 << 18;
__device__ __forceinline__ unsigned long long await(unsigned long long* p) {
    unsigned long long w = kUnpublished;
    for (int i = 0; i < kAwaitPolls; ++i) {
        w = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (w != kUnpublished) break;
        __builtin_amdgcn_s_sleep(2);
    }
    return w;
}

template <int W>
struct GlrSmem {
    float A[W][kGlrCh], X[W][kGlrCh];                    // maps of the waves' tokens
    unsigned long long got[kGlrGroup][kGlrCh];           // maps of the segments before this one
    float carry[kGlrCh];                                 // state entering the segment
    unsigned ticket;
};

// Where the workgroup stands in the scan: its place `ord` (0 = first segment of the scan), strip
// and batch row.  Tickets count the strips of one place before the next place.  One behind the last
// (again: a workspace that another call uses) is nobody's: ord < 0, and its workgroup writes nothing.
struct GlrPlace {
    int ord, strip, b;
};
template <int W>
__device__ __forceinline__ GlrPlace glr_place(const GlrParams& p, GlrSmem<W>& sm) {
    unsigned t = blockIdx.x;
    if (p.nseg > 1) {
        if (threadIdx.x == 0)
            sm.ticket = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        t = sm.ticket;
    }
    if (t >= gridDim.x) return {-1, 0, 0};
    const unsigned per = (unsigned)p.nstrip * (unsigned)p.B, r = t % per;
    return {(int)(t / per), (int)(r % (unsigned)p.nstrip), (int)(r / (unsigned)p.nstrip)};
}

// Joins the segment to those before it in the scan: sm.A / sm.X hold the waves' maps in scan order
// (wave 0 first); publishes the segment's map, and leaves the state entering the segment in
// sm.carry.  `first` is the state entering the scan (null = zero).
template <int W>
__device__ __forceinline__ void glr_join(const GlrParams& p, GlrSmem<W>& sm, const GlrPlace& w, const float* first) {
    const int l = lane_id(), wv = wave_id();
    const long words = (long)p.nstrip * kGlrCh, chw = (long)w.strip * kGlrCh + l;
    const int groups = p.nseg / kGlrGroup;
    unsigned long long* maps = p.pub + (long)w.b * p.nseg * words + chw;
    unsigned long long* runs = p.pub + (long)p.B * p.nseg * words + (long)w.b * groups * words + chw;
    const int base = w.ord / kGlrGroup * kGlrGroup;  // segments base .. ord - 1 are folded here
    float A = 1.f, X = 0.f;
    if (wv == 0) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            X = sm.A[i][l] * X + sm.X[i][l];
            A *= sm.A[i][l];
        }
        if (w.ord + 1 < p.nseg) publish(maps + (long)w.ord * words, pack_map(A, X));
    }
    for (int j = base + wv; j < w.ord; j += W) sm.got[j - base][l] = await(maps + (long)j * words);
    __syncthreads();
    if (wv == 0) {
        const long ch = (long)w.strip * kGlrCh + l;
        // The maps of the segments base .. ord - 1 are composed among themselves before they meet the state,
        // whose sum is then rounded once per group, not once per segment (normwise error against 64 bits where
        // nothing decays, T=32749 fp32: h 1.7e-7 -> 1.4e-7, dx 2.3e-7 -> 1.2e-7, 232 -> 233 us in all; composing
        // the waves' maps in the same way 1.3e-7 and 1.2e-7, but 240 us).
        float ga = 1.f, gx = 0.f;
        for (int j = 0; j < w.ord - base; ++j) {
            const float a = word_hi(sm.got[j][l]);
            gx = a * gx + word_lo(sm.got[j][l]);
            ga *= a;
        }
        float h = 0.f;
        if (base > 0) h = word_lo(await(runs + (long)(base / kGlrGroup - 1) * words));
        else if (first && ch < p.D) h = first[(long)w.b * p.D + ch];
        sm.carry[l] = ga * h + gx;
        if (w.ord % kGlrGroup == kGlrGroup - 1 && w.ord + 1 < p.nseg)
            publish(runs + (long)(w.ord / kGlrGroup) * words, pack_map(0.f, A * ga * h + (A * gx + X)));
    }
    __syncthreads();
}

// Composes the maps of the lanes of one channel group in scan order: lane group g = l / 8 (UP: g
// ascending, else descending).  In: the thread's own map; out: the map of everything in the wave
// before the thread (exclusive); the wave's whole map goes to sm.A / sm.X at place `slot`.
template <bool UP, int W>
__device__ __forceinline__ void glr_wave_scan(f32x8& A, f32x8& X, GlrSmem<W>& sm, int slot) {
    const int l = lane_id(), g = UP ? l >> 3 : 7 - (l >> 3);
#pragma unroll
    for (int m = 1; m < 8; m <<= 1) {
        const bool use = g >= m;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float a = UP ? __shfl_up(A[e], 8 * m) : __shfl_down(A[e], 8 * m);
            const float x = UP ? __shfl_up(X[e], 8 * m) : __shfl_down(X[e], 8 * m);
            X[e] = use ? A[e] * x + X[e] : X[e];
            A[e] = use ? A[e] * a : A[e];
        }
    }
    if (g == 7) {
        const int c = 8 * (l & 7);
#pragma unroll
        for (int e = 0; e < 8; ++e) sm.A[slot][c + e] = A[e], sm.X[slot][c + e] = X[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float a = UP ? __shfl_up(A[e], 8) : __shfl_down(A[e], 8);
        const float x = UP ? __shfl_up(X[e], 8) : __shfl_down(X[e], 8);
        A[e] = g ? a : 1.f;
        X[e] = g ? x : 0.f;
    }
}

// The state entering the thread's tokens: sm.carry through the waves before, then the exclusive map.
template <int W>
__device__ __forceinline__ f32x8 glr_enter(const GlrSmem<W>& sm, int slot, const f32x8& A, const f32x8& X) {
    const int c = 8 * (lane_id() & 7);
    f32x8 h;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float s = sm.carry[c + e];
        for (int i = 0; i < slot; ++i) s = sm.A[i][c + e] * s + sm.X[i][c + e];
        h[e] = A[e] * s + X[e];
    }
    return h;
}

// The thread's tokens of a [B][T][D] tensor; element `off` is its first.  Zeros (which leave the state
// alone) behind the end: such loads go to the tensor's start, so that no branch parts the loads.
template <typename T>
__device__ __forceinline__ void glr_load(const GlrParams& p, bool live, long t0, long off, const T* src, f32x8 (&v)[kGlrRun]) {
    if (p.T == 0) {
#pragma unroll
        for (int s = 0; s < kGlrRun; ++s) v[s] = f32x8{0, 0, 0, 0, 0, 0, 0, 0};
        return;
    }
#pragma unroll
    for (int s = 0; s < kGlrRun; ++s) v[s] = ld8(src + (live && t0 + s < p.T ? off + s * p.D : 0));
#pragma unroll
    for (int s = 0; s < kGlrRun; ++s)
        if (!(live && t0 + s < p.T)) v[s] = f32x8{0, 0, 0, 0, 0, 0, 0, 0};
}

template <typename T>
__global__ __launch_bounds__(kGlrFwdThreads) void gdr2_glr_fwd_kernel(GlrParams p) {
    constexpr int W = kGlrFwdWaves;
    __shared__ GlrSmem<W> sm;
    const GlrPlace w = glr_place(p, sm);
    if (w.ord < 0) return;
    const int l = lane_id(), wv = wave_id();
    const long ch = (long)w.strip * kGlrCh + 8 * (l & 7);
    const long t0 = (long)w.ord * kGlrFwdSeg + (wv * 8 + (l >> 3)) * kGlrRun;
    const bool live = ch < p.D;  // D is a multiple of 8: all eight channels or none
    const long off = (w.b * p.T + t0) * p.D + ch;
    const T* x = (const T*)p.x;
    const float* la = p.la;
    f32x8 xv[kGlrRun], a[kGlrRun];
    glr_load(p, live, t0, off, x, xv);
    glr_load(p, live, t0, off, la, a);
    f32x8 A = {1, 1, 1, 1, 1, 1, 1, 1}, X = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < kGlrRun; ++s) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            a[s][e] = decay(a[s][e]);
            X[e] = a[s][e] * X[e] + xv[s][e];
            A[e] *= a[s][e];
        }
    }
    glr_wave_scan<true>(A, X, sm, wv);
    __syncthreads();
    glr_join(p, sm, w, p.h0);
    f32x8 h = glr_enter(sm, wv, A, X);
    if (!live) return;
    // the first tokens of the backward's segments keep the state that enters them
    if (wv % kGlrBwdWaves == 0 && l < 8) {
        const long seg = (long)w.ord * (kGlrFwdSeg / kGlrBwdSeg) + wv / kGlrBwdWaves, n = glr_segments(p.T, kGlrBwdSeg);
        if (seg < n) st8(p.states + (w.b * n + seg) * p.D + ch, h);
    }
    T* hp = (T*)p.h + off;
#pragma unroll
    for (int s = 0; s < kGlrRun; ++s) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = a[s][e] * h[e] + xv[s][e];
        if (t0 + s < p.T) st8s(hp + s * p.D, h);
    }
    if (p.hT && w.ord == p.nseg - 1 && wv == W - 1 && (l >> 3) == 7) st8(p.hT + w.b * p.D + ch, h);
}

template <typename T>
__global__ __launch_bounds__(kGlrBwdThreads) void gdr2_glr_bwd_kernel(GlrParams p) {
    constexpr int W = kGlrBwdWaves;
    __shared__ GlrSmem<W> sm;
    const GlrPlace w = glr_place(p, sm);
    if (w.ord < 0) return;
    const int l = lane_id(), wv = wave_id();
    const int seg = p.nseg - 1 - w.ord;  // the scan starts at the last segment
    const long ch = (long)w.strip * kGlrCh + 8 * (l & 7);
    const long t0 = (long)seg * kGlrBwdSeg + (wv * 8 + (l >> 3)) * kGlrRun;
    const bool live = ch < p.D;
    const long off = (w.b * p.T + t0) * p.D + ch;
    const T* x = (const T*)p.x;
    const T* dh = (const T*)p.dh;
    const float* la = p.la;
    f32x8 hp[kGlrRun], a[kGlrRun], g[kGlrRun];
    glr_load(p, live, t0, off, x, hp);
    glr_load(p, live, t0, off, la, a);
    glr_load(p, live, t0, off, dh, g);
    // forward inside the segment: hp[s] becomes h_{t-1}
    f32x8 A = {1, 1, 1, 1, 1, 1, 1, 1}, X = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < kGlrRun; ++s) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            a[s][e] = decay(a[s][e]);
            X[e] = a[s][e] * X[e] + hp[s][e];
            A[e] *= a[s][e];
        }
    }
    f32x8 Y = {0, 0, 0, 0, 0, 0, 0, 0}, Ar = A;
#pragma unroll
    for (int s = kGlrRun - 1; s >= 0; --s)
#pragma unroll
        for (int e = 0; e < 8; ++e) Y[e] = a[s][e] * (g[s][e] + Y[e]);
    glr_wave_scan<true>(A, X, sm, wv);
    if (threadIdx.x < kGlrCh) {
        const long c = (long)w.strip * kGlrCh + threadIdx.x;
        sm.carry[threadIdx.x] = c < p.D ? p.states[((long)w.b * p.nseg + seg) * p.D + c] : 0.f;
    }
    __syncthreads();
    f32x8 h = glr_enter(sm, wv, A, X);
#pragma unroll
    for (int s = 0; s < kGlrRun; ++s) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float next = a[s][e] * h[e] + hp[s][e];
            hp[s][e] = h[e];
            h[e] = next;
        }
    }
    __syncthreads();  // sm.A, sm.X and sm.carry are used again
    const int slot = W - 1 - wv;
    glr_wave_scan<false>(Ar, Y, sm, slot);
    __syncthreads();
    glr_join(p, sm, w, p.dhT);
    f32x8 R = glr_enter(sm, slot, Ar, Y);
    if (!live) return;
    T* dx = (T*)p.dx + off;
    float* dla = p.dla + off;
#pragma unroll
    for (int s = kGlrRun - 1; s >= 0; --s) {
        f32x8 d;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            g[s][e] += R[e];
            R[e] = a[s][e] * g[s][e];
            d[e] = R[e] * hp[s][e];
        }
        if (t0 + s < p.T) {
            st8s(dx + s * p.D, g[s]);
            st8s(dla + s * p.D, d);
        }
    }
    if (p.dh0 && seg == 0 && wv == 0 && l < 8) st8(p.dh0 + w.b * p.D + ch, R);
}

// Presets the published words and the ticket of the next launch on the same stream.
__global__ __launch_bounds__(256) void gdr2_glr_clear_kernel(unsigned long long* pub, long n, unsigned* ticket) {
    for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long)gridDim.x * 256) pub[i] = kUnpublished;
    if (blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0;
}

template <typename T>
__global__ __launch_bounds__(256) void gdr2_glr_step_kernel(GlrStepParams p) {
    const long i = 8 * ((long)blockIdx.x * 256 + threadIdx.x);
    if (i >= p.n) return;
    const f32x8 x = ld8((const T*)p.x + i), la = ld8(p.la + i);
    f32x8 h = p.h_in ? ld8(p.h_in + i) : f32x8{0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = decay(la[e]) * h[e] + x[e];
    st8(p.h_out + i, h);
    st8((T*)p.h + i, h);
}

template <typename T>
static hipError_t launch_glr(bool bwd, const GlrParams& p, hipStream_t s) {
    const long row = (long)p.nseg * p.nstrip, fit = max_workgroups(bwd ? kGlrBwdThreads : kGlrFwdThreads) / row;
    const long most = fit < p.B ? fit : p.B;  // batch rows of a launch
    if (most < 1) return hipErrorInvalidConfiguration;
    for (long b0 = 0; b0 < p.B; b0 += most) {
        GlrParams c = p;
        const long tok = b0 * p.T * p.D, st = b0 * p.D;
        c.B = (int)(p.B - b0 < most ? p.B - b0 : most);
        c.x = (const T*)p.x + tok;
        c.la = p.la + tok;
        c.states = p.states + b0 * glr_segments(p.T, kGlrBwdSeg) * p.D;
        if (bwd) {
            c.dh = (const T*)p.dh + tok;
            c.dx = (T*)p.dx + tok;
            c.dla = p.dla + tok;
            if (p.dhT) c.dhT = p.dhT + st;
            if (p.dh0) c.dh0 = p.dh0 + st;
        } else {
            c.h = (T*)p.h + tok;
            if (p.h0) c.h0 = p.h0 + st;
            if (p.hT) c.hT = p.hT + st;
        }
        if (c.nseg > 1) {
            const long n = (long)c.B * (c.nseg + c.nseg / kGlrGroup) * c.nstrip * kGlrCh;
            const long nb = (n + 1023) / 1024;
            hipLaunchKernelGGL(gdr2_glr_clear_kernel, dim3(nb < 2048 ? nb : 2048), dim3(256), 0, s, c.pub, n, c.ticket);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        const dim3 grid((unsigned)(c.B * row));
        if (bwd) hipLaunchKernelGGL((gdr2_glr_bwd_kernel<T>), grid, dim3(kGlrBwdThreads), 0, s, c);
        else hipLaunchKernelGGL((gdr2_glr_fwd_kernel<T>), grid, dim3(kGlrFwdThreads), 0, s, c);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t glr_dispatch(int bf, bool bwd, const GlrParams& p, hipStream_t s) {
    return bf ? launch_glr<bf16>(bwd, p, s) : launch_glr<float>(bwd, p, s);
}

hipError_t glr_step_dispatch(int bf, const GlrStepParams& p, hipStream_t s) {
    const dim3 grid((unsigned)((p.n / 8 + 255) / 256));
    if (bf) hipLaunchKernelGGL((gdr2_glr_step_kernel<bf16>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((gdr2_glr_step_kernel<float>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace gdr2

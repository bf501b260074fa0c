// gdr2_swa_decode.hip -- one token per sequence against the bounded cache of sliding-window
// attention, and the cache's filling from a prefill (gfx950).
//
// The cache of a sequence holds `sinks` fixed slots and a ring of `window` slots; position p lives
// in slot p (p < sinks) or sinks + (p - sinks) mod window.  The new token at position pos goes into
// its slot, over the one position that leaves the window, and sees every slot that has been
// written: min(pos + 1, sinks + window) of them, in any order, since softmax sums commute:
//     s_j = scale q . k_j,   o = sum_j exp(s_j) v_j / sum_j exp(s_j)
// The step is bound by reading the cache once (256 sequences of 2052 slots, 4 key/value heads of 128, bf16:
// 193 us when all are full, 5.6 TB/s, as a device copy; with a wave's next slots loaded ahead of its
// products 196); for one sequence (5.4 us, and 3.7 us for the join) by the latency of its two launches.  A workgroup takes up to sixteen query heads of one
// key/value head and a part of the slots; a wave takes 32 slots at a time: keys come as MFMA rows
// straight from the cache (scores: slots in rows, heads in columns), so a lane's eight
// probabilities are one head's, and the values it loads (its own slots, d / 16 channels) turn into
// the second product's operand inside its registers.  Waves, then parts, are joined at the end by
// their running maxima.  The new token's key and value are taken from the call's arguments, not
// from the cache, so its slot can be written by the same launch; that is done by one workgroup.
#include "gdr2_block_kernels.hpp"
#include "gdr2_common.hpp"

namespace gdr2 {

constexpr int kDecThreads = 256, kDecWaves = 4, kDecHeads = 16;
constexpr int kDecTile = 32;                        // slots of a wave's step
constexpr int kDecStep = kDecTile * kDecWaves;      // slots of a workgroup's step
constexpr float kDecLowest = -3.0e38f, kDecLog2e = 1.4426950408889634f;

template <typename T, int D>
__global__ __launch_bounds__(kDecThreads, 2) void gdr2_swa_decode_kernel(SwaDecodeParams p) {
    constexpr int ES = (int)sizeof(T), DPL = D / 16, KS = D * ES / 64;  // KS: 64-byte steps of a row
    constexpr int PITCH = D + 4;
    __shared__ float osum[kDecWaves][kDecHeads][PITCH];
    __shared__ float stat[kDecWaves][kDecHeads][2];
    const int l = lane_id(), wv = wave_id(), c = l & 15, g = l >> 4;
    const int G = p.H / p.Hkv, groups = (G + kDecHeads - 1) / kDecHeads;
    const int split = blockIdx.x % p.splits, job = blockIdx.x / p.splits;
    const int grp = job % groups, kvh = job / groups % p.Hkv, sq = job / groups / p.Hkv;
    const int h0 = kvh * G + grp * kDecHeads, heads = G - grp * kDecHeads < kDecHeads ? G - grp * kDecHeads : kDecHeads;
    const long slots = p.window + p.sinks, pos = p.pos[sq];
    const bool any = pos >= 0;
    const long held = any ? (pos + 1 < slots ? pos + 1 : slots) : 0;
    const long mine = any ? (pos < p.sinks ? pos : p.sinks + (pos - p.sinks) % p.window) : 0;
    const long rstr = (long)p.Hkv * D * ES;  // bytes from slot to slot
    const long noff = ((long)sq * p.Hkv + kvh) * D * ES, coff = ((long)sq * slots * p.Hkv + kvh) * D * ES;
    const char *kn = (const char*)p.k + noff, *vn = (const char*)p.v + noff;
    char *kc = (char*)p.kc + coff, *vc = (char*)p.vc + coff;
    const float sc = p.scale * kDecLog2e;

    // queries: column c is head h0 + c, pieces of 16 bytes in the order the keys are read
    i32x4 qf[KS];
    const char* q = (const char*)p.q + ((long)sq * p.H + h0 + c) * D * ES;
#pragma unroll
    for (int s = 0; s < KS; ++s) qf[s] = c < heads ? *(const i32x4*)(q + s * 64 + g * 16) : i32x4{0, 0, 0, 0};

    float m = kDecLowest, z = 0.f;
    f32x4 acc[DPL];
#pragma unroll
    for (int i = 0; i < DPL; ++i) acc[i] = f32x4{0, 0, 0, 0};
    // this part's slots: whole workgroup steps
    const long steps = (held + kDecStep - 1) / kDecStep, per = (steps + p.splits - 1) / p.splits;
    const long s_end = (split + 1) * per * kDecStep < held ? (split + 1) * per * kDecStep : held;
    for (long s0 = split * per * kDecStep + wv * kDecTile; s0 < s_end; s0 += kDecStep) {
        // slots that hold nothing yet are replaced by the new token's row and masked
        i32x4 kf[2][KS];
        T vf[2][4][DPL];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const long j = s0 + 16 * b + c;
            const char* kr = j == mine || j >= held ? kn : kc + j * rstr;
#pragma unroll
            for (int s = 0; s < KS; ++s) kf[b][s] = *(const i32x4*)(kr + s * 64 + g * 16);
        }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const long j = s0 + 16 * b + 4 * g + r;
                const char* vr = j == mine || j >= held ? vn : vc + j * rstr;
                __builtin_memcpy(vf[b][r], __builtin_assume_aligned(vr + c * DPL * ES, DPL * ES < 16 ? 8 : 16), DPL * ES);
            }
        f32x4 s[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                if constexpr (ES == 2) {
                    s[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, kf[b][k]), __builtin_bit_cast(bf16x8, qf[k]), s[b], 0, 0, 0);
                } else {
                    const f32x4 x = __builtin_bit_cast(f32x4, kf[b][k]), y = __builtin_bit_cast(f32x4, qf[k]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[b] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], y[e], s[b], 0, 0, 0);
                }
            }
        float mx = -INFINITY;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                s[b][r] = s0 + 16 * b + 4 * g + r < held ? s[b][r] * sc : -INFINITY;
                mx = fmaxf(mx, s[b][r]);
            }
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        const float mn = fmaxf(m, mx), f = __builtin_amdgcn_exp2f(m - mn);
        m = mn;
        z *= f;
#pragma unroll
        for (int i = 0; i < DPL; ++i) acc[i] *= f;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                s[b][r] = __builtin_amdgcn_exp2f(s[b][r] - m);
                z += s[b][r];
            }
        // probabilities rounded to bf16 for the bf16 product (its inputs' precision), sums in fp32
#pragma unroll
        for (int i = 0; i < DPL; ++i) {
            if constexpr (ES == 2) {
                const bf16x8 a = {vf[0][0][i], vf[0][1][i], vf[0][2][i], vf[0][3][i], vf[1][0][i], vf[1][1][i], vf[1][2][i], vf[1][3][i]};
                const bf16x8 w = {(bf16)s[0][0], (bf16)s[0][1], (bf16)s[0][2], (bf16)s[0][3], (bf16)s[1][0], (bf16)s[1][1], (bf16)s[1][2], (bf16)s[1][3]};
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, w, acc[i], 0, 0, 0);
            } else {
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(vf[b][r][i], s[b][r], acc[i], 0, 0, 0);
            }
        }
    }
    z += __shfl_xor(z, 16);
    z += __shfl_xor(z, 32);
    // lane (c, g) holds head c, channels (4 g + r) DPL + i
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < DPL; ++i) osum[wv][c][(4 * g + r) * DPL + i] = acc[i][r];
    if (g == 0) {
        stat[wv][c][0] = m;
        stat[wv][c][1] = z;
    }
    __syncthreads();
    for (int x = threadIdx.x; x < heads * (D / 4); x += kDecThreads) {
        const int hd = x / (D / 4), d = 4 * (x % (D / 4));
        float M = kDecLowest, Z = 0.f;
#pragma unroll
        for (int w = 0; w < kDecWaves; ++w) M = fmaxf(M, stat[w][hd][0]);
        f32x4 o = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kDecWaves; ++w) {
            const float f = __builtin_amdgcn_exp2f(stat[w][hd][0] - M);
            Z += stat[w][hd][1] * f;
            o += *(const f32x4*)&osum[w][hd][d] * f;
        }
        if (p.splits == 1) {
            const float inv = any ? 1.f / Z : 0.f;
            store4((T*)p.o + ((long)sq * p.H + h0 + hd) * D + d, any ? o * inv : f32x4{0, 0, 0, 0});
        } else {
            float* part = p.part + ((long)blockIdx.x * kDecHeads + hd) * (D + 4);
            *(f32x4*)(part + d) = o;
            if (d == 0) {
                part[D] = M;
                part[D + 1] = Z;
            }
        }
    }
    // the new token's row into its slot
    if (any && split == 0 && grp == 0 && threadIdx.x < 2 * D * ES / 16) {
        constexpr int U = D * ES / 16;
        const int x = threadIdx.x % U;
        *(i32x4*)((threadIdx.x < U ? kc : vc) + mine * rstr + x * 16) = *(const i32x4*)((threadIdx.x < U ? kn : vn) + x * 16);
    }
}

// Joins the parts of one head: thread groups of D / 4 lanes take every kGroups-th part, four channels per
// lane, then the groups in order.
template <typename T, int D>
__global__ __launch_bounds__(kDecThreads) void gdr2_swa_decode_join_kernel(SwaDecodeParams p) {
    constexpr int LANES = D / 4, kGroups = kDecThreads / LANES;
    __shared__ f32x4 osum[kGroups][LANES];
    __shared__ float stat[kGroups][2];
    const int G = p.H / p.Hkv, groups = (G + kDecHeads - 1) / kDecHeads;
    const int sq = blockIdx.x / p.H, head = blockIdx.x % p.H, kvh = head / G, in = head % G;
    const long job = ((long)sq * p.Hkv + kvh) * groups + in / kDecHeads, stride = (long)kDecHeads * (D + 4);
    const float* part = p.part + job * p.splits * stride + (in % kDecHeads) * (D + 4);
    const int grp = threadIdx.x / LANES, ln = threadIdx.x % LANES;
    const bool any = p.pos[sq] >= 0;
    float M = kDecLowest, Z = 0.f;
    f32x4 o = {0, 0, 0, 0};
#pragma unroll 4
    for (int s = grp; s < p.splits; s += kGroups) {
        const float* q = part + s * stride;
        const f32x4 x = *(const f32x4*)(q + 4 * ln);
        const float m = q[D], z = q[D + 1], mn = fmaxf(M, m);
        const float f0 = __builtin_amdgcn_exp2f(M - mn), f1 = __builtin_amdgcn_exp2f(m - mn);
        M = mn;
        Z = Z * f0 + z * f1;
        o = o * f0 + x * f1;
    }
    osum[grp][ln] = o;
    if (ln == 0) {
        stat[grp][0] = M;
        stat[grp][1] = Z;
    }
    __syncthreads();
    if (grp != 0) return;
    for (int g = 1; g < kGroups; ++g) {
        const float m = stat[g][0], mn = fmaxf(M, m), f0 = __builtin_amdgcn_exp2f(M - mn), f1 = __builtin_amdgcn_exp2f(m - mn);
        M = mn;
        Z = Z * f0 + stat[g][1] * f1;
        o = o * f0 + osum[g][ln] * f1;
    }
    store4((T*)p.o + ((long)sq * p.H + head) * D + 4 * ln, any ? o * (1.f / Z) : f32x4{0, 0, 0, 0});
}

// Parts per (sequence, key/value head, head group), none with less than one workgroup step of slots: as many
// as give one workgroup per compute unit (256), each a long stream; where that leaves more than a quarter of
// the units idle, two per unit.  N sequences of 4 key/value heads, d=128 bf16, us with one / two per unit:
// window 8192: N=8 30 / 32, N=16 46 / 51, N=24 85 / 81, N=40 (160 of 256 units) 144 / 128, N=50 151 / 176;
// window 2048: N=48 35 / 40, N=64 44 / 47 (one part needs no joining launch).
int swa_decode_splits(long N, long Hkv, long groups, long slots) {
    const long jobs = N * Hkv * groups, steps = (slots + kDecStep - 1) / kDecStep;
    long want = jobs > 0 ? 256 / jobs : 1;
    if (jobs > 0 && want * jobs < 192) want = 512 / jobs;
    const long s = want < steps ? want : steps;
    return (int)(s < 1 ? 1 : s);
}

template <typename T, int D>
static hipError_t launch_decode(const SwaDecodeParams& p, hipStream_t s) {
    const long per = (long)p.Hkv * ((p.H / p.Hkv + kDecHeads - 1) / kDecHeads);  // workgroups of a sequence's part
    const long fit = max_workgroups(kDecThreads) / (per * p.splits), most = fit < p.N ? fit : p.N;
    if (most < 1 || (p.splits > 1 && most < p.N)) return hipErrorInvalidConfiguration;  // parts: few jobs only
    for (long n0 = 0; n0 < p.N; n0 += most) {
        SwaDecodeParams c = p;
        const long row = D * (long)sizeof(T), kv = n0 * p.Hkv * row;
        c.N = (int)(p.N - n0 < most ? p.N - n0 : most);
        c.q = (const char*)p.q + n0 * p.H * row;
        c.o = (char*)p.o + n0 * p.H * row;
        c.k = (const char*)p.k + kv;
        c.v = (const char*)p.v + kv;
        c.kc = (char*)p.kc + kv * (p.window + p.sinks);
        c.vc = (char*)p.vc + kv * (p.window + p.sinks);
        c.pos = p.pos + n0;
        hipLaunchKernelGGL((gdr2_swa_decode_kernel<T, D>), dim3((unsigned)(c.N * per * p.splits)), dim3(kDecThreads), 0, s, c);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (p.splits == 1) return hipSuccess;
    hipLaunchKernelGGL((gdr2_swa_decode_join_kernel<T, D>), dim3((unsigned)((long)p.N * p.H)), dim3(kDecThreads), 0, s, p);
    return hipGetLastError();
}

hipError_t swa_decode_dispatch(int bf, const SwaDecodeParams& p, hipStream_t s) {
    if (bf) return p.d == 128 ? launch_decode<bf16, 128>(p, s) : launch_decode<bf16, 64>(p, s);
    return p.d == 128 ? launch_decode<float, 128>(p, s) : launch_decode<float, 64>(p, s);
}

// One 16-byte piece of a slot per thread, keys and values: the newest position below the length that
// lives in the slot; a slot none lives in keeps its contents.
__global__ __launch_bounds__(256) void gdr2_swa_fill_kernel(SwaFillParams p) {
    const long slots = p.window + p.sinks, x = p.first + (long)blockIdx.x * 256 + threadIdx.x;
    if (x >= p.B * slots * p.row16) return;
    const long piece = x % p.row16, slot = x / p.row16 % slots, b = x / p.row16 / slots;
    long L = p.lengths ? p.lengths[b] : p.T;
    L = L > p.T ? p.T : L;
    long pos = slot;
    if (slot >= p.sinks && pos < L) pos += (L - 1 - slot) / p.window * p.window;
    if (pos >= L) return;
    const long src = (b * p.T + pos) * p.row16 + piece;
    ((i32x4*)p.kc)[x] = ((const i32x4*)p.k)[src];
    ((i32x4*)p.vc)[x] = ((const i32x4*)p.v)[src];
}

hipError_t swa_fill_dispatch(const SwaFillParams& p, hipStream_t s) {
    const long n = p.B * (p.window + p.sinks) * p.row16, most = max_workgroups(256) * 256;
    for (long first = 0; first < n; first += most) {
        SwaFillParams c = p;
        c.first = first;
        const long m = n - first < most ? n - first : most;
        hipLaunchKernelGGL(gdr2_swa_fill_kernel, dim3((unsigned)((m + 255) / 256)), dim3(256), 0, s, c);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace gdr2

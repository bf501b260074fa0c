// gdr2_paged.hip -- one token per sequence against a key/value cache of pages, and the pages' filling from a
// prefill (gfx950).
//
// A sequence's positions 0 .. pos lie in the rows its page table names; the new token's own key and value come
// from the call's arguments, so its row is written by the same launch and read by none:
//     s_j = scale q . k_j,   o = sum_j exp(s_j) v_j / sum_j exp(s_j)
// The step is bound by reading the held rows once.  A workgroup takes up to sixteen query heads of one key/value
// head and a part of the positions, a wave 32 positions at a time.  Lane i of the wave looks up the row of position
// i, a step ahead of its use; the rows go around by cross-lane reads, so a page may end anywhere inside a step.
// Keys come as MFMA rows straight from memory (scores: positions in rows, heads in columns), so a lane's eight
// probabilities are one head's, and the values it loads (its own positions, d / 16 channels) are the second
// product's operand as they stand.  Waves, then parts, are joined by their running maxima.
//
// Measured (16 query heads over 4 of d = 128, bf16): 256 sequences of 1 to 4096 positions in pages of 16, 208 us with the
// join, the rows at 4.6 TB/s of the 5.0 that a copy reaches; one sequence of 32768 positions in pages of 64, 15 us for the
// rows (4.4 TB/s) and 6 for the join's launch.  The filling stores 4 prompts of up to 4096 tokens in 10 us, at a copy's rate.
#include "gdr2_common.hpp"
#include "gdr2_hybrid_kernels.hpp"

namespace gdr2 {

constexpr int kPagedThreads = 256, kPagedWaves = 4, kPagedTile = kPagedStep / kPagedWaves;
// Maxima start at the lowest finite number: below every finite score, and a masked one, -inf, leaves exp2(-inf) = 0 of it.
constexpr float kPagedLowest = -__FLT_MAX__, kPagedLog2e = 1.4426950408889634f;

// What a sequence sees: positions 0 .. old - 1 through the table, then the new token.  Parts of whole steps.
struct PagedSeq {
    int slots, per, live;   // old + 1 (0: no token), positions of a part, parts that hold any
    __device__ __forceinline__ PagedSeq(const PagedDecodeParams& p, int sq) {
        const int pos = p.pos[sq], cap = p.width << p.shift;
        slots = pos < 0 ? 0 : (pos < cap ? pos : cap) + 1;
        const int steps = (slots + kPagedStep - 1) / kPagedStep, n = (steps + p.splits - 1) / p.splits;
        per = n * kPagedStep;
        live = n > 0 ? (steps + n - 1) / n : 0;
    }
};

// The row of position j < cap of the sequence whose table is `t`; -1 where it has none.
__device__ __forceinline__ int paged_row(const PagedDecodeParams& p, const int* t, int j) {
    const int e = t[j >> p.shift];
    return (unsigned)e < (unsigned)p.pages ? (e << p.shift) + (j & ((1 << p.shift) - 1)) : -1;
}

template <typename T, int D>
__global__ __launch_bounds__(kPagedThreads, 2) void gdr2_paged_decode_kernel(PagedDecodeParams p) {
    constexpr int ES = (int)sizeof(T), DPL = D / 16, KS = D * ES / 64;  // KS: 64-byte steps of a row
    constexpr int PITCH = D + 4;
    __shared__ float osum[kPagedWaves][kPagedHeads][PITCH];
    __shared__ float stat[kPagedWaves][kPagedHeads][2];
    const int l = lane_id(), wv = wave_id(), c = l & 15, g = l >> 4;
    const int G = p.H / p.Hkv, groups = (G + kPagedHeads - 1) / kPagedHeads;
    const int split = blockIdx.x % p.splits, job = blockIdx.x / p.splits;
    const int grp = job % groups, kvh = job / groups % p.Hkv, sq = job / groups / p.Hkv;
    const PagedSeq seq(p, sq);
    if (split > 0 && split >= seq.live) return;
    const int h0 = kvh * G + grp * kPagedHeads, heads = G - grp * kPagedHeads < kPagedHeads ? G - grp * kPagedHeads : kPagedHeads;
    const int old = seq.slots - 1;              // the new token's slot
    const long rstr = (long)p.Hkv * D * ES;     // bytes from row to row
    const long noff = ((long)sq * p.Hkv + kvh) * D * ES, hoff = (long)kvh * D * ES;
    const char *kn = (const char*)p.k + noff, *vn = (const char*)p.v + noff;
    const char *kp = (const char*)p.kp + hoff, *vp = (const char*)p.vp + hoff;
    const int* table = p.table + (long)sq * p.width;
    const float sc = p.scale * kPagedLog2e;

    // queries: column c is head h0 + c, pieces of 16 bytes in the order the keys are read
    i32x4 qf[KS];
    const char* q = (const char*)p.q + ((long)sq * p.H + h0 + c) * D * ES;
#pragma unroll
    for (int s = 0; s < KS; ++s) qf[s] = c < heads ? *(const i32x4*)(q + s * 64 + g * 16) : i32x4{0, 0, 0, 0};

    float m = kPagedLowest, z = 0.f;
    f32x4 acc[DPL];
#pragma unroll
    for (int i = 0; i < DPL; ++i) acc[i] = f32x4{0, 0, 0, 0};
    const int s_end = (split + 1) * (long)seq.per < seq.slots ? (split + 1) * seq.per : seq.slots;
    // the row of the lane's position (lanes 32 and up as lane - 32); -1: none, -2: the new token
    auto look = [&](int s0) {
        const int j = s0 + (l & 31);
        return j < old ? paged_row(p, table, j) : j == old ? -2 : -1;
    };
    const int first = split * seq.per + wv * kPagedTile;
    int next = first < s_end ? look(first) : -1;
    for (int s0 = first; s0 < s_end; s0 += kPagedStep) {
        const int mine = next;
        if (s0 + kPagedStep < s_end) next = look(s0 + kPagedStep);
        // positions without a row are replaced by the new token's and masked
        i32x4 kf[2][KS];
        T vf[2][4][DPL];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int row = __builtin_amdgcn_ds_bpermute((16 * b + c) << 2, mine);
            const char* kr = row < 0 ? kn : kp + row * rstr;
#pragma unroll
            for (int s = 0; s < KS; ++s) kf[b][s] = *(const i32x4*)(kr + s * 64 + g * 16);
        }
        bool seen[2][4];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = __builtin_amdgcn_ds_bpermute((16 * b + 4 * g + r) << 2, mine);
                seen[b][r] = row != -1;
                const char* vr = row < 0 ? vn : vp + row * rstr;
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
                s[b][r] = seen[b][r] ? s[b][r] * sc : -INFINITY;
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
        // bf16: probabilities in two parts, 16 bits (with one, a few positions do not average its roundings out; the second
        // product is free beside the rows' arrival), sums in fp32
        bf16x8 w, rest;
        if constexpr (ES == 2) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                w[e] = (bf16)s[e / 4][e % 4];
                rest[e] = (bf16)(s[e / 4][e % 4] - (float)w[e]);
            }
        }
#pragma unroll
        for (int i = 0; i < DPL; ++i) {
            if constexpr (ES == 2) {
                const bf16x8 a = {vf[0][0][i], vf[0][1][i], vf[0][2][i], vf[0][3][i], vf[1][0][i], vf[1][1][i], vf[1][2][i], vf[1][3][i]};
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, w, acc[i], 0, 0, 0);
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, rest, acc[i], 0, 0, 0);
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
    const bool any = seq.slots > 0;
    for (int x = threadIdx.x; x < heads * (D / 4); x += kPagedThreads) {
        const int hd = x / (D / 4), d = 4 * (x % (D / 4));
        float M = kPagedLowest, Z = 0.f;
#pragma unroll
        for (int w = 0; w < kPagedWaves; ++w) M = fmaxf(M, stat[w][hd][0]);
        f32x4 o = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kPagedWaves; ++w) {
            const float f = __builtin_amdgcn_exp2f(stat[w][hd][0] - M);
            Z += stat[w][hd][1] * f;
            o += *(const f32x4*)&osum[w][hd][d] * f;
        }
        if (seq.live <= 1) {  // no part to join
            store4((T*)p.o + ((long)sq * p.H + h0 + hd) * D + d, any ? o * (1.f / Z) : f32x4{0, 0, 0, 0});
        } else {
            float* part = p.part + ((long)blockIdx.x * kPagedHeads + hd) * (D + 4);
            *(f32x4*)(part + d) = o;
            if (d == 0) {
                part[D] = M;
                part[D + 1] = Z;
            }
        }
    }
    // the new token's row into its page
    constexpr int U = D * ES / 16;
    const int pos = p.pos[sq];
    if (split == 0 && grp == 0 && threadIdx.x < 2 * U && any && pos < p.width << p.shift) {
        const int row = paged_row(p, table, pos), x = threadIdx.x % U;
        if (row >= 0)
            *(i32x4*)((threadIdx.x < U ? (char*)p.kp : (char*)p.vp) + hoff + row * rstr + x * 16) =
                *(const i32x4*)((threadIdx.x < U ? kn : vn) + x * 16);
    }
}

// Joins the parts of one head: thread groups of D / 4 lanes take every kGroups-th part, four channels per
// lane, then the groups in order.
template <typename T, int D>
__global__ __launch_bounds__(kPagedThreads) void gdr2_paged_join_kernel(PagedDecodeParams p) {
    constexpr int LANES = D / 4, kGroups = kPagedThreads / LANES;
    __shared__ f32x4 osum[kGroups][LANES];
    __shared__ float stat[kGroups][2];
    const int G = p.H / p.Hkv, groups = (G + kPagedHeads - 1) / kPagedHeads;
    const int sq = blockIdx.x / p.H, head = blockIdx.x % p.H, kvh = head / G, in = head % G;
    const PagedSeq seq(p, sq);
    if (seq.live <= 1) return;
    const long job = ((long)sq * p.Hkv + kvh) * groups + in / kPagedHeads, stride = (long)kPagedHeads * (D + 4);
    const float* part = p.part + job * p.splits * stride + (in % kPagedHeads) * (D + 4);
    const int grp = threadIdx.x / LANES, ln = threadIdx.x % LANES;
    float M = kPagedLowest, Z = 0.f;
    f32x4 o = {0, 0, 0, 0};
#pragma unroll 4
    for (int s = grp; s < seq.live; s += kGroups) {
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
    store4((T*)p.o + ((long)sq * p.H + head) * D + 4 * ln, o * (1.f / Z));
}

// Parts of the positions, by the table's width: only the device knows how many of them a sequence holds, and it spreads
// their steps over the parts.  As many as make 2048 workgroups with the sequences and heads, none below a step of 128.
// That is more than the device holds at once: lengths differ, and so do the parts' ends.  Measured for 256 / 512 / 1024 /
// 2048 / 4096 workgroups (16 query heads over 4 of d = 128, bf16): 256 sequences of 1 to 4096 positions 219 / 219 / 219 /
// 208 / 206 us, one of 32768 18 / 18 / 21 / 21 / 21, 32 of 1 to 4096 40 / 31 / 33 / 32 / 40; and 13 of 1 to 2777, fp32,
// 12 over 4 heads of d = 64, 20 / 19 / 17 / 14.5 / 15.  Tables of up to three steps stay one part, since the launch that joins
// parts costs as much as two steps: 64 sequences of 300 positions 7.7 us in one part each, 10.3 in three (as a wider table has
// them); one of 500 (four steps) 7.5 us in four parts, 9.1 in two.
int paged_splits(long N, long Hkv, long groups, long capacity) {
    const long jobs = N * Hkv * groups, steps = (capacity + kPagedStep) / kPagedStep;  // the new token included
    if (steps <= 3 || jobs < 1 || jobs > 1024) return 1;
    return (int)(2048 / jobs < steps ? 2048 / jobs : steps);
}

template <typename T, int D>
static hipError_t launch_decode(const PagedDecodeParams& p, hipStream_t s) {
    const long per = (long)p.Hkv * ((p.H / p.Hkv + kPagedHeads - 1) / kPagedHeads);  // workgroups of a sequence's part
    const long fit = max_workgroups(kPagedThreads) / (per * p.splits), most = fit < p.N ? fit : p.N;
    if (most < 1 || (p.splits > 1 && most < p.N)) return hipErrorInvalidConfiguration;  // parts: few jobs only
    for (long n0 = 0; n0 < p.N; n0 += most) {
        PagedDecodeParams c = p;
        const long row = D * (long)sizeof(T), kv = n0 * p.Hkv * row;
        c.N = (int)(p.N - n0 < most ? p.N - n0 : most);
        c.q = (const char*)p.q + n0 * p.H * row;
        c.o = (char*)p.o + n0 * p.H * row;
        c.k = (const char*)p.k + kv;
        c.v = (const char*)p.v + kv;
        c.table = p.table + n0 * p.width;
        c.pos = p.pos + n0;
        hipLaunchKernelGGL((gdr2_paged_decode_kernel<T, D>), dim3((unsigned)(c.N * per * p.splits)), dim3(kPagedThreads), 0, s, c);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (p.splits == 1) return hipSuccess;
    hipLaunchKernelGGL((gdr2_paged_join_kernel<T, D>), dim3((unsigned)((long)p.N * p.H)), dim3(kPagedThreads), 0, s, p);
    return hipGetLastError();
}

hipError_t paged_decode_dispatch(int bf, const PagedDecodeParams& p, hipStream_t s) {
    if (bf) return p.d == 128 ? launch_decode<bf16, 128>(p, s) : launch_decode<bf16, 64>(p, s);
    return p.d == 128 ? launch_decode<float, 128>(p, s) : launch_decode<float, 64>(p, s);
}

// One 16-byte piece of a token's row per thread, keys and values.
__global__ __launch_bounds__(256) void gdr2_paged_fill_kernel(PagedFillParams p) {
    const long x = p.first + (long)blockIdx.x * 256 + threadIdx.x;
    if (x >= p.n) return;
    const long tok = x / p.row16;
    const int piece = (int)(x % p.row16), t = (int)(tok % p.T), b = (int)(tok / p.T);
    if (p.lengths && t >= p.lengths[b]) return;
    const long j = (long)(p.start ? p.start[b] : 0) + t;
    if (j < 0 || j >= (long)p.width << p.shift) return;
    const int e = p.table[(long)b * p.width + (j >> p.shift)];
    if ((unsigned)e >= (unsigned)p.pages) return;
    const long row = ((long)e << p.shift) + (j & ((1 << p.shift) - 1)), dst = row * p.row16 + piece;
    ((i32x4*)p.kp)[dst] = ((const i32x4*)p.k)[x];
    ((i32x4*)p.vp)[dst] = ((const i32x4*)p.v)[x];
}

hipError_t paged_fill_dispatch(const PagedFillParams& p, hipStream_t s) {
    const long n = (long)p.B * p.T * p.row16, most = max_workgroups(256) * 256;
    for (long first = 0; first < n; first += most) {
        PagedFillParams c = p;
        c.first = first;
        c.n = n;
        const long m = n - first < most ? n - first : most;
        hipLaunchKernelGGL(gdr2_paged_fill_kernel, dim3((unsigned)((m + 255) / 256)), dim3(256), 0, s, c);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace gdr2

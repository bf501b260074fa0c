// gdr2_swa_fwd.hip -- forward of sliding-window attention with sinks (gfx950).
//
// Query i of a sequence of L tokens sees key j when j <= i < L and (i - j < window or j < sinks):
//     s_ij = scale q_i . k_j,   o_i = sum_j exp(s_ij) v_j / z_i,   z_i = sum_j exp(s_ij)
// and lse_i = ln z_i for the backward.  One pass over the keys with a running reference m_i of the
// exponent: the terms are exp(s_ij - m_i), and m_i moves (with one rescaling of the sums) only when
// a score exceeds it by more than 2^8, so the sums stay within fp32 and most tiles rescale nothing.
// A workgroup takes 128 queries of one head, 32 per wave, and walks the key tiles its queries may
// see through a double-buffered pair of LDS tiles; grouped heads share the tiles in L2.  Where that
// gives few workgroups for the card (kSwaNarrowMost), it takes 64 queries and its two halves (KS = 2)
// walk alternate 32-key blocks, joined at the end.
//
// No pipe is full: the matrix units are busy 37 % of the cycles at the first size below and 43 % at the second, the
// LDS pipe 29 and 33 %.  The bound is the chain of a tile, scores to exponentials to products, which two waves per SIMD
// (241 registers, 32 of them for tiles on their way to LDS) overlap only in part.
// B=4 T=4096 H=16 d=128 window 2048 bf16: 251 us, 823 TFLOP/s over the visible pairs (a library product of
// 8192^3 random bf16 reaches 1275 on the same card); T=32768, four heads to a key head: 610 us, 874 TFLOP/s.
// With the work between the products taken out, the products and their operands' reads in order still need 193 us.  Measured at the first size and
// not kept, against 257 us in the same runs: scores formed one tile ahead of their softmax in the same wave 313 us; 64 queries per wave
// (one wave per SIMD) 469; two wave groups alternating products and softmax behind barriers 286; three
// waves per SIMD with 32-key tiles 259.
#include "gdr2_swa.hpp"

namespace gdr2 {

template <typename T, int D, int KS>
__global__ __launch_bounds__(kSwaThreads, 2) void gdr2_swa_fwd_kernel(SwaParams p) {
    using S = Swa<T, D>;
    constexpr int BT = S::BT, NB = S::NB, QW = kSwaWaves / KS, BQ = 32 * QW;  // QW: waves side by side
    static_assert(NB % KS == 0, "whole key blocks per half");
    constexpr int KM = S::kRows, VM = S::kBoth;
    constexpr int KP = BT * S::template kPitch<KM>, VP = BT * S::template kPitch<VM>;
    __shared__ i32x4 lds[2 * KP + 2 * VP];  // two key tiles, two value tiles
    static_assert(sizeof(lds) >= (size_t)QW * S::kPut * 16, "output rows fit the tiles");
    const int l = lane_id(), wv = uniform_wave(), n = l & 31, h = l >> 5;
    const int nqt = (int)((p.T + BQ - 1) / BQ);
    const int work = xcd_swizzle(blockIdx.x, gridDim.x);
    const int qt = swa_query_tile(p, work % nqt, nqt), bh = work / nqt, b = bh / p.H, hd = bh % p.H, kvh = hd / (p.H / p.Hkv);
    const int L = swa_length(p, b);
    const int Q0 = qt * BQ, q0 = Q0 + 32 * (wv % QW), i = q0 + n, ks = wv / QW;
    const long qstr = (long)p.H * D * S::ES, kstr = (long)p.Hkv * D * S::ES;
    const char* kb = (const char*)p.k + ((long)b * p.T * p.Hkv + kvh) * D * S::ES;
    const char* vb = (const char*)p.v + ((long)b * p.T * p.Hkv + kvh) * D * S::ES;
    const bool live = i < L;
    const float c = p.scale * kLog2e;

    f32x16 acc[S::DB];
#pragma unroll
    for (int db = 0; db < S::DB; ++db) acc[db] = zero16();
    float m = kLowest, z = 0.f;
    if (Q0 < L) {
        i32x4 qf[S::KK];
        S::keep(qf, live ? (const char*)p.q + (((long)b * p.T + i) * p.H + hd) * D * S::ES : nullptr);
        const SwaTiles tl(p, BT, Q0, Q0 + BQ <= L ? Q0 + BQ - 1 : L - 1);
        i32x4 ku[S::UNITS], vu[S::UNITS];
        auto fetch = [&](int t) {
            const int j0 = tl.start(t, BT), rows = L - j0 < BT ? L - j0 : BT;
            S::fetch(ku, kb + j0 * kstr, kstr, rows);
            S::fetch(vu, vb + j0 * kstr, kstr, rows);
        };
        fetch(0);
        S::template stage<KM>(lds, ku);
        S::template stage<VM>(lds + 2 * KP, vu);
        lds_barrier();
        for_tiles(tl.n, [&](int t, auto buf_) {
            constexpr int cur = decltype(buf_)::value;
            if (t + 1 < tl.n) fetch(t + 1);
            const int j0 = tl.start(t, BT);
            if (j0 <= q0 + 31 && (q0 - (j0 + BT - 1) < p.window || j0 < p.sinks)) {
                f32x16 s[NB / KS];  // the half's key blocks, from row r0 of the tile
                const int r0 = ks * (BT / KS);
#pragma unroll
                for (int kb_ = 0; kb_ < NB / KS; ++kb_) s[kb_] = S::template dots<KM>(lds + cur * KP, r0 + 32 * kb_, qf);
                if (j0 + BT - 1 > q0 || q0 + 31 - j0 >= p.window) {
                    edge_tile();
#pragma unroll
                    for (int kb_ = 0; kb_ < NB / KS; ++kb_)
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            if (!swa_sees(p, i, j0 + r0 + 32 * kb_ + crow(r, h))) s[kb_][r] = -INFINITY;
                        }
                }
                float mx = s[0][0];
#pragma unroll
                for (int kb_ = 0; kb_ < NB / KS; ++kb_)
#pragma unroll
                    for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[kb_][r]);
                if (__any(mx * c > m + 8.f)) {  // rare once the reference has settled
                    const float mn = fmaxf(m, fmaxf(mx, __shfl_xor(mx, 32)) * c), f = exp2_f(m - mn);
                    m = mn;
                    z *= f;
#pragma unroll
                    for (int db = 0; db < S::DB; ++db)
#pragma unroll
                        for (int r = 0; r < 16; ++r) acc[db][r] *= f;
                }
#pragma unroll
                for (int kb_ = 0; kb_ < NB / KS; ++kb_) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        s[kb_][r] = exp2_f(s[kb_][r] * c - m);
                        z += s[kb_][r];
                    }
                    S::template add_rows<VM>(acc, lds + 2 * KP + cur * VP, r0 + 32 * kb_, s[kb_]);
                }
            }
            if (t + 1 < tl.n) {
                S::template stage<KM>(lds + (cur ^ 1) * KP, ku);
                S::template stage<VM>(lds + 2 * KP + (cur ^ 1) * VP, vu);
            }
            lds_barrier();
        });
    }
    z += __shfl_xor(z, 32);
    if constexpr (KS == 2) {
        // the second half's sums, through LDS: D + 2 floats per query (the tiles are no longer read)
        constexpr int PITCH = D + 4;
        static_assert(sizeof(lds) >= sizeof(float) * (size_t)QW * 32 * PITCH, "sums of one half fit the tiles");
        float* row = (float*)lds + ((wv % QW) * 32 + n) * PITCH;
        if (ks == 1) {
            S::each4([&](int db, int e, int d0) { *(f32x4*)(row + d0) = S::four(acc[db], e); });
            if (h == 0) row[D] = m, row[D + 1] = z;
        }
        __syncthreads();
        if (ks == 0) {
            const float m1 = row[D], z1 = row[D + 1], mn = fmaxf(m, m1), f0 = exp2_f(m - mn), f1 = exp2_f(m1 - mn);
            m = mn;
            z = z * f0 + z1 * f1;
            S::each4([&](int db, int e, int d0) {
                const f32x4 x = *(const f32x4*)(row + d0);
#pragma unroll
                for (int c4 = 0; c4 < 4; ++c4) acc[db][e + c4] = acc[db][e + c4] * f0 + x[c4] * f1;
            });
        }
        __syncthreads();
        if (ks == 1) return;
    }
    // a query at or behind the length saw nothing: zero output, lse = -inf
    const float inv = live ? 1.f / z : 0.f;
    if (!live) {
#pragma unroll
        for (int db = 0; db < S::DB; ++db) acc[db] = zero16();
    }
    const int rows = p.T - q0 >= 32 ? 32 : p.T > q0 ? p.T - q0 : 0;
    S::put_rows(acc, inv, lds + wv * S::kPut, (char*)p.o + (((long)b * p.T + q0) * p.H + hd) * D * S::ES,
                qstr, rows);
    if (h == 0 && n < rows) p.lse[(long)bh * p.T + i] = live ? (m + __builtin_amdgcn_logf(z)) * kLn2 : -INFINITY;
}

template <typename T, int D>
static hipError_t launch_swa_fwd(const SwaParams& p, hipStream_t s) {
    const long heads = (long)p.B * p.H, wide = (p.T + 127) / 128 * heads, narrow = (p.T + 63) / 64 * heads;
    if constexpr (Swa<T, D>::NB == 2) {
        if (wide <= kSwaNarrowMost) {
            hipLaunchKernelGGL((gdr2_swa_fwd_kernel<T, D, 2>), dim3((unsigned)narrow), dim3(kSwaThreads), 0, s, p);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((gdr2_swa_fwd_kernel<T, D, 1>), dim3((unsigned)wide), dim3(kSwaThreads), 0, s, p);
    return hipGetLastError();
}

hipError_t swa_fwd_dispatch(int bf, const SwaParams& p, hipStream_t s) {
    if (bf) return p.d == 128 ? launch_swa_fwd<bf16, 128>(p, s) : launch_swa_fwd<bf16, 64>(p, s);
    return p.d == 128 ? launch_swa_fwd<float, 128>(p, s) : launch_swa_fwd<float, 64>(p, s);
}

}  // namespace gdr2

// gdr2_swa_bwd.hip -- backward of sliding-window attention with sinks (gfx950).
//
// With p_ij = exp(scale q_i . k_j - lse_i) over the visible pairs and delta_i = dO_i . o_i:
//     dv_j = sum_i p_ij dO_i,   ds_ij = p_ij (dO_i . v_j - delta_i)
//     dq_i = scale sum_j ds_ij k_j,   dk_j = scale sum_i ds_ij q_i
// (dk_j, dv_j: summed over the query heads of the key/value head).  The probabilities are formed
// again from lse, in two passes that each own their outputs, so that nothing is added atomically
// and results do not change from run to run:
//   gdr2_swa_dq_kernel    128 queries of one head per workgroup, walking key tiles (three products
//                         per tile); also writes delta;
//   gdr2_swa_dkv_kernel   128 keys of one key/value head per workgroup, walking the query tiles of
//                         its heads (four products per tile).
// The sinks are seen by every later query: a key tile that walked them all would run many times
// longer than the others, so the queries behind its window are cut into at most kSwaSinkPieces
// pieces, each a workgroup of gdr2_swa_sink_kernel that leaves fp32 sums for the (at most 64)
// sinks; the first key tile's workgroup adds them in order.
#include "gdr2_swa.hpp"

namespace gdr2 {

template <typename T, int D>
__global__ __launch_bounds__(kSwaThreads, sizeof(T) * D > 256 ? 1 : 2) void gdr2_swa_dq_kernel(SwaParams p) {
    using S = Swa<T, D>;
    constexpr int BT = S::BT, NB = S::NB;
    constexpr int BQ = 32 * kSwaWaves;
    __shared__ typename S::tile lds[4];
    const int l = lane_id(), wv = uniform_wave(), n = l & 31, h = l >> 5;
    const int nqt = (int)((p.T + BQ - 1) / BQ);
    const int work = xcd_swizzle(blockIdx.x, gridDim.x);
    const int qt = work % nqt, bh = work / nqt, b = bh / p.H, hd = bh % p.H, kvh = hd / (p.H / p.Hkv);
    const int L = swa_length(p, b);
    const int Q0 = qt * BQ, q0 = Q0 + 32 * wv, i = q0 + n;
    const long qstr = (long)p.H * D * S::ES, kstr = (long)p.Hkv * D * S::ES;
    const char* kb = (const char*)p.k + ((long)b * p.T * p.Hkv + kvh) * D * S::ES;
    const char* vb = (const char*)p.v + ((long)b * p.T * p.Hkv + kvh) * D * S::ES;
    const bool live = i < L;
    const float c = p.scale * kLog2e;
    const long qoff = (((long)b * p.T + i) * p.H + hd) * D * S::ES;

    f32x16 acc[S::DB];
#pragma unroll
    for (int db = 0; db < S::DB; ++db) acc[db] = zero16();
    float delta = 0.f;
    if (Q0 < L) {
        // a dead query (at or behind the length) has zero rows and lse = inf: its probabilities are 0
        i32x4 qf[S::KK], gf[S::KK];
        S::keep(qf, live ? (const char*)p.q + qoff : nullptr);
        S::keep(gf, live ? (const char*)p.dO + qoff : nullptr);
        if (live) {
#pragma unroll
            for (int kk = 0; kk < S::KK; ++kk) {
                const i32x4 of = *(const i32x4*)((const char*)p.o + qoff + (2 * kk + h) * 16);
                if constexpr (S::ES == 2) {
                    const bf16x8 x = __builtin_bit_cast(bf16x8, of), y = __builtin_bit_cast(bf16x8, gf[kk]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) delta += (float)x[e] * (float)y[e];
                } else {
                    const f32x4 x = __builtin_bit_cast(f32x4, of), y = __builtin_bit_cast(f32x4, gf[kk]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) delta += x[e] * y[e];
                }
            }
        }
        delta += __shfl_xor(delta, 32);
        const float lse2 = live ? p.lse[(long)bh * p.T + i] * kLog2e : INFINITY;
        const SwaTiles tl(p, BT, Q0, Q0 + BQ <= L ? Q0 + BQ - 1 : L - 1);
        i32x4 ku[S::UNITS], vu[S::UNITS];
        auto fetch = [&](int t) {
            const int j0 = tl.start(t, BT);
            const int rows = L - j0 < BT ? L - j0 : BT;
            S::fetch(ku, kb + j0 * kstr, kstr, rows);
            S::fetch(vu, vb + j0 * kstr, kstr, rows);
        };
        fetch(0);
        S::stage(lds[0], ku);
        S::stage(lds[2], vu);
        lds_barrier();
        for_tiles(tl.n, [&](int t, auto buf_) {
            constexpr int cur = decltype(buf_)::value;
            if (t + 1 < tl.n) fetch(t + 1);
            const int j0 = tl.start(t, BT);
            if (j0 <= q0 + 31 && (q0 - (j0 + BT - 1) < p.window || j0 < p.sinks)) {
                const bool edge = j0 + BT - 1 > q0 || q0 + 31 - j0 >= p.window;
#pragma unroll
                for (int k_ = 0; k_ < NB; ++k_) {
                    f32x16 s = S::dots(lds[cur], 32 * k_, qf);
                    const f32x16 dp = S::dots(lds[2 + cur], 32 * k_, gf);
                    if (edge) {
                        edge_tile();
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            if (!swa_sees(p, i, j0 + 32 * k_ + crow(r, h))) s[r] = -INFINITY;
                    }
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = exp2_f(s[r] * c - lse2) * (dp[r] - delta);
                    S::add_rows(acc, lds[cur], 32 * k_, s);
                }
            }
            if (t + 1 < tl.n) {
                S::stage(lds[cur ^ 1], ku);
                S::stage(lds[2 + (cur ^ 1)], vu);
            }
            lds_barrier();
        });
    }
    const int rows = p.T - q0 >= 32 ? 32 : p.T > q0 ? p.T - q0 : 0;
    S::put_rows(acc, p.scale, &lds[0][0] + wv * 32 * S::CPR,
                (char*)p.dq + (((long)b * p.T + q0) * p.H + hd) * D * S::ES, qstr, rows);
    if (h == 0 && n < rows) p.delta[(long)bh * p.T + i] = delta;
}

// One 32-key block of a wave against one 32-query block of the staged tiles: adds to dk and dv
// (columns: keys).  ls / dl: lse (in units of log 2) and delta of the tile's queries.
template <typename T, int D>
struct SwaKeys {
    using S = Swa<T, D>;
    i32x4 kf[S::KK], vf[S::KK];
    f32x16 dk[S::DB], dv[S::DB];
    __device__ __forceinline__ void init(const char* k, const char* v) {
        S::keep(kf, k);
        S::keep(vf, v);
#pragma unroll
        for (int db = 0; db < S::DB; ++db) dk[db] = dv[db] = zero16();
    }
    __device__ __forceinline__ void step(const SwaParams& p, const i32x4* qt, const i32x4* gt, const float* ls, const float* dl,
                                         int r0, int i0, int j, bool edge, float c) {
        const int h = lane_id() >> 5;
        f32x16 s = S::dots(qt, r0, kf);
        f32x16 dp = S::dots(gt, r0, vf);
        if (edge) {  // some pairs of the block are hidden
            edge_tile();
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (!swa_sees(p, i0 + r0 + crow(r, h), j)) s[r] = -INFINITY;
        }
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
            const f32x4 x = *(const f32x4*)(ls + r0 + 8 * r4 + 4 * h), y = *(const f32x4*)(dl + r0 + 8 * r4 + 4 * h);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[4 * r4 + e] = exp2_f(s[4 * r4 + e] * c - x[e]);
                dp[4 * r4 + e] = s[4 * r4 + e] * (dp[4 * r4 + e] - y[e]);
            }
        }
        S::add_rows(dv, gt, r0, s);
        S::add_rows(dk, qt, r0, dp);
    }
};

// Query tiles of BT rows with their lse and delta, from registers into LDS.
template <typename T, int D>
struct SwaQueries {
    using S = Swa<T, D>;
    i32x4 qu[S::UNITS], gu[S::UNITS];
    float su;
    // threads 0 .. BT - 1: lse, BT .. 2 BT - 1: delta of the tile's rows
    __device__ __forceinline__ void fetch(const SwaParams& p, int b, int hd, int i0, int L) {
        const long qstr = (long)p.H * D * S::ES, off = (((long)b * p.T + i0) * p.H + hd) * D * S::ES;
        const int rows = L - i0 < S::BT ? L - i0 : S::BT;
        S::fetch(qu, (const char*)p.q + off, qstr, rows);
        S::fetch(gu, (const char*)p.dO + off, qstr, rows);
        const int x = threadIdx.x, r = x % S::BT;
        const long at = ((long)b * p.H + hd) * p.T + i0 + r;
        su = 0.f;
        if (x < S::BT) su = r < rows ? p.lse[at] * kLog2e : INFINITY;
        else if (x < 2 * S::BT && r < rows) su = p.delta[at];
    }
    __device__ __forceinline__ void stage(i32x4* qt, i32x4* gt, float* sc) const {
        S::stage(qt, qu);
        S::stage(gt, gu);
        if (threadIdx.x < 2 * S::BT) sc[threadIdx.x] = su;
    }
};

template <typename T, int D>
__global__ __launch_bounds__(kSwaThreads, sizeof(T) * D > 128 ? 1 : 2) void gdr2_swa_dkv_kernel(SwaParams p) {
    using S = Swa<T, D>;
    constexpr int BT = S::BT, NB = S::NB;
    static_assert(kSwaKeyTile == 32 * kSwaWaves, "a wave holds 32 keys");
    __shared__ typename S::tile lds[4];  // queries and cotangents, two of each
    __shared__ float sc[2][2 * BT];
    const int l = lane_id(), wv = uniform_wave(), n = l & 31, h = l >> 5;
    const int nkt = (int)((p.T + kSwaKeyTile - 1) / kSwaKeyTile);
    const int work = xcd_swizzle(blockIdx.x, gridDim.x);
    const int kt = work % nkt, bh = work / nkt, b = bh / p.Hkv, kvh = bh % p.Hkv, G = p.H / p.Hkv;
    const int L = swa_length(p, b);
    const int K0 = kt * kSwaKeyTile, k0 = K0 + 32 * wv, j = k0 + n;
    const long kstr = (long)p.Hkv * D * S::ES;
    const long koff = (((long)b * p.T + j) * p.Hkv + kvh) * D * S::ES;
    const float c = p.scale * kLog2e;
    SwaKeys<T, D> ks;
    ks.init(j < L ? (const char*)p.k + koff : nullptr, j < L ? (const char*)p.v + koff : nullptr);
    if (K0 < L) {
        // the queries that see the tile's last key; with sinks, the first tile's go on to the far ones
        const int seen = kt == 0 && p.sinks > 0 ? p.far0 : K0 + kSwaKeyTile - 1 + p.window;
        const int i_end = seen < L ? seen : L;
        const int t0 = K0 / BT, per = (i_end + BT - 1) / BT - t0, nt = per * G;
        SwaQueries<T, D> qs;
        auto fetch = [&](int t) { qs.fetch(p, b, kvh * G + t / per, (t0 + t % per) * BT, L); };
        fetch(0);
        qs.stage(lds[0], lds[2], sc[0]);
        lds_barrier();
        for_tiles(nt, [&](int t, auto buf_) {
            constexpr int cur = decltype(buf_)::value;
            if (t + 1 < nt) fetch(t + 1);
            const int i0 = (t0 + t % per) * BT;
#pragma unroll
            for (int r = 0; r < NB; ++r) {
                const int ia = i0 + 32 * r;
                if (ia + 31 >= k0 && (ia - (k0 + 31) < p.window || k0 < p.sinks))
                    ks.step(p, lds[cur], lds[2 + cur], sc[cur], sc[cur] + BT, 32 * r, i0, j,
                            ia < k0 + 31 || ia + 31 - k0 >= p.window, c);
            }
            if (t + 1 < nt) qs.stage(lds[cur ^ 1], lds[2 + (cur ^ 1)], sc[cur ^ 1]);
            lds_barrier();
        });
    }
    // the sinks' sums over the far queries, piece by piece
    if (kt == 0 && p.pieces > 0 && k0 < p.sinks) {
        for (int q = 0; q < p.pieces; ++q) {
            if (p.far0 + q * p.piece_len >= L) break;
            const float* part = p.sink_part + (((long)q * p.B * p.Hkv + bh) * 2 * kSwaMaxSinks + j) * D;
#pragma unroll
            for (int db = 0; db < S::DB; ++db)
#pragma unroll
                for (int r4 = 0; r4 < 4; ++r4) {
                    const f32x4 x = *(const f32x4*)(part + 32 * db + 8 * r4 + 4 * h);
                    const f32x4 y = *(const f32x4*)(part + (long)kSwaMaxSinks * D + 32 * db + 8 * r4 + 4 * h);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        ks.dk[db][4 * r4 + e] += x[e];
                        ks.dv[db][4 * r4 + e] += y[e];
                    }
                }
        }
    }
    const int rows = p.T - k0 >= 32 ? 32 : p.T > k0 ? p.T - k0 : 0;
    const long ooff = (((long)b * p.T + k0) * p.Hkv + kvh) * D * S::ES;
    i32x4* buf = &lds[0][0] + wv * 32 * S::CPR;
    S::put_rows(ks.dk, p.scale, buf, (char*)p.dk + ooff, kstr, rows);
    wave_sync();
    S::put_rows(ks.dv, 1.f, buf, (char*)p.dv + ooff, kstr, rows);
}

// Sums over one piece of the far queries for the sinks: wave w takes the queries of 32-row block
// w % NB of every tile and the keys of block w / NB (kSwaMaxSinks: two blocks).
template <typename T, int D>
__global__ __launch_bounds__(kSwaThreads, sizeof(T) * D > 128 ? 1 : 2) void gdr2_swa_sink_kernel(SwaParams p) {
    using S = Swa<T, D>;
    constexpr int BT = S::BT, NB = S::NB;
    __shared__ typename S::tile lds[4];
    __shared__ float sc[2][2 * BT];
    static_assert(sizeof(lds) >= 2 * 32 * D * 2 * sizeof(float), "partial sums of two waves fit the tiles");
    const int l = lane_id(), wv = uniform_wave(), n = l & 31, h = l >> 5;
    const int piece = blockIdx.x % p.pieces, bh = blockIdx.x / p.pieces, b = bh / p.Hkv, kvh = bh % p.Hkv, G = p.H / p.Hkv;
    const int L = swa_length(p, b);
    const int ia = p.far0 + piece * p.piece_len;
    if (ia >= L) return;  // the first key tile skips this piece too
    const int ib = ia + p.piece_len < L ? ia + p.piece_len : L;
    const int rb = wv % NB, key0 = 32 * (wv / NB);
    const int j = key0 + n;
    const bool mine = key0 < p.sinks;
    const float c = p.scale * kLog2e;
    const long koff = (((long)b * p.T + j) * p.Hkv + kvh) * D * S::ES;
    // far queries lie behind far0 > the sinks, so a sink's row exists; keys behind the sinks are zero
    const bool key = j < p.sinks && j < L;
    SwaKeys<T, D> ks;
    ks.init(key ? (const char*)p.k + koff : nullptr, key ? (const char*)p.v + koff : nullptr);
    const int per = (ib - ia + BT - 1) / BT, nt = per * G;
    SwaQueries<T, D> qs;
    auto fetch = [&](int t) { qs.fetch(p, b, kvh * G + t / per, ia + t % per * BT, L); };
    fetch(0);
    qs.stage(lds[0], lds[2], sc[0]);
    lds_barrier();
    for_tiles(nt, [&](int t, auto buf_) {
        constexpr int cur = decltype(buf_)::value;
        if (t + 1 < nt) fetch(t + 1);
        if (mine) ks.step(p, lds[cur], lds[2 + cur], sc[cur], sc[cur] + BT, 32 * rb, ia + t % per * BT, j, true, c);
        if (t + 1 < nt) qs.stage(lds[cur ^ 1], lds[2 + (cur ^ 1)], sc[cur ^ 1]);
        lds_barrier();
    });
    // two query blocks of one key block: the second wave's sums through LDS
    float* buf = (float*)&lds[0][0] + (wv / NB) * 2 * 32 * D;
    auto place = [&](int db, int r4) { return n * D + 32 * db + 8 * r4 + 4 * h; };
    if constexpr (NB == 2) {
        if (mine && rb == 1) {
#pragma unroll
            for (int db = 0; db < S::DB; ++db)
#pragma unroll
                for (int r4 = 0; r4 < 4; ++r4) {
                    const int e = 4 * r4;
                    *(f32x4*)(buf + place(db, r4)) = f32x4{ks.dk[db][e], ks.dk[db][e + 1], ks.dk[db][e + 2], ks.dk[db][e + 3]};
                    *(f32x4*)(buf + 32 * D + place(db, r4)) = f32x4{ks.dv[db][e], ks.dv[db][e + 1], ks.dv[db][e + 2], ks.dv[db][e + 3]};
                }
        }
        __syncthreads();
    }
    if (!mine || rb != 0) return;
    float* part = p.sink_part + (((long)piece * p.B * p.Hkv + bh) * 2 * kSwaMaxSinks + key0) * D;
#pragma unroll
    for (int db = 0; db < S::DB; ++db)
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
            const int e = 4 * r4;
            f32x4 x = {ks.dk[db][e], ks.dk[db][e + 1], ks.dk[db][e + 2], ks.dk[db][e + 3]};
            f32x4 y = {ks.dv[db][e], ks.dv[db][e + 1], ks.dv[db][e + 2], ks.dv[db][e + 3]};
            if constexpr (NB == 2) {
                x += *(const f32x4*)(buf + place(db, r4));
                y += *(const f32x4*)(buf + 32 * D + place(db, r4));
            }
            *(f32x4*)(part + place(db, r4)) = x;
            *(f32x4*)(part + (long)kSwaMaxSinks * D + place(db, r4)) = y;
        }
}

template <typename T, int D>
static hipError_t launch_swa_bwd(const SwaParams& p, hipStream_t s) {
    const long gq = (long)((p.T + 127) / 128) * p.B * p.H, gk = (long)((p.T + kSwaKeyTile - 1) / kSwaKeyTile) * p.B * p.Hkv;
    hipLaunchKernelGGL((gdr2_swa_dq_kernel<T, D>), dim3((unsigned)gq), dim3(kSwaThreads), 0, s, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (p.pieces > 0) {
        hipLaunchKernelGGL((gdr2_swa_sink_kernel<T, D>), dim3((unsigned)((long)p.pieces * p.B * p.Hkv)), dim3(kSwaThreads), 0, s, p);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((gdr2_swa_dkv_kernel<T, D>), dim3((unsigned)gk), dim3(kSwaThreads), 0, s, p);
    return hipGetLastError();
}

hipError_t swa_bwd_dispatch(int bf, const SwaParams& p, hipStream_t s) {
    if (bf) return p.d == 128 ? launch_swa_bwd<bf16, 128>(p, s) : launch_swa_bwd<bf16, 64>(p, s);
    return p.d == 128 ? launch_swa_bwd<float, 128>(p, s) : launch_swa_bwd<float, 64>(p, s);
}

}  // namespace gdr2

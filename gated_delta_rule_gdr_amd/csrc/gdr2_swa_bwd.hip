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
// longer than the others, so the queries behind its window are cut into pieces, each a workgroup of
// the second kernel that leaves fp32 sums for the (at most 64) sinks.  Where the key tiles alone do
// not fill the card, the queries of a tile are cut into parts too.  gdr2_swa_reduce_kernel adds such
// sums in a fixed order.
//
// No pipe is full: at the size below the matrix units are busy 43 % (dq) and 28 % (dkv) of the cycles, the LDS pipe
// 29 and 22 %.  The bound is the chain of a tile, probabilities to score gradients to products, over two waves per
// SIMD (dq, 247 registers) and one (dkv: dk, dv, k and v of 32 keys and the staged tiles take 416).  B=4 T=4096 H=16 d=128 window 2048 bf16: dq 339 us (914 TFLOP/s over its
// three products), dkv 596 us (693 over its four), reduction 5 us.  Measured there and not kept, for the
// whole backward (953-956 us): dv and dk on different waves, each forming the probabilities, 981; the
// same with the probabilities handed over through LDS 948, but 87 us instead of 69 at B=3 T=1537 H=12/3
// d=64; both query blocks of a tile side by side in one wave 1123.
#include "gdr2_swa.hpp"

namespace gdr2 {

// Key tiles (of 64) up to which delta is summed from the probabilities.  Normwise error of dq against fp64
// (d=128 bf16, no window), delta from o / summed: T=16 3.0e-3 / 2.6e-3, T=64 2.7e-3 / 2.5e-3, T=256 2.55e-3 /
// 2.43e-3, T=1024 2.50e-3 / 2.41e-3; the walk costs 38 -> 43 us of the backward at B=1 T=256 H=64, and
// 954 -> 1193 us at B=4 T=4096 H=16 window 2048 if every query walked (with four tiles: no change).  Windows of up to
// 129 tokens (193 with 64 queries per workgroup) and no sinks keep every query of any sequence at four tiles, so they
// always pay it: B=4 T=4096 H=16 window 64 / 128, backward 240 / 262 -> 265 / 298 us, dq's error 2.42e-3 -> 2.36e-3.
constexpr int kExactTiles = 4;

// Sequences of at most this many tokens form the bf16 gradients FINE, from probabilities and score gradients in two
// bf16 pieces: their outputs are sums of few terms, whose roundings do not average out.  Error of dq and dk
// against fp64 over that of rounding the exact result once, 1500 random problems, one piece: 1.41 on average, over 1.5
// in 6 % of all, up to 2.1, all of them with T <= 31; so in 0.1 %, up to 1.58 (with 64 tokens 0.05 %).  Backward in us,
// one piece / two: T=32 H=8 d=128 14.6 / 15.5, B=1024 T=32 H=16/4 d=128 566 / 585, B=512 T=32 H=16 d=64 154 / 176.
constexpr int kSwaFine = 32;

// KS = 2: 64 queries per workgroup, its halves walk alternate 32-key blocks (as in the forward).
template <typename T, int D, int KS, bool FINE>
__global__ __launch_bounds__(kSwaThreads, sizeof(T) * D > 256 ? 1 : 2) void gdr2_swa_dq_kernel(SwaParams p) {
    using S = Swa<T, D>;
    constexpr int BT = S::BT, NB = S::NB, QW = kSwaWaves / KS, BQ = 32 * QW;
    constexpr int KM = S::kBoth, VM = S::kRows;
    constexpr int KP = BT * S::template kPitch<KM>, VP = BT * S::template kPitch<VM>;
    __shared__ i32x4 lds[2 * KP + 2 * VP];  // two key tiles, two value tiles
    static_assert(sizeof(lds) >= (size_t)QW * S::kPut * 16, "output rows fit the tiles");
    __shared__ float dsum[KS == 2 ? kSwaWaves : 1][32];
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
            const int j0 = tl.start(t, BT), rows = L - j0 < BT ? L - j0 : BT;
            S::fetch(ku, kb + j0 * kstr, kstr, rows);
            S::fetch(vu, vb + j0 * kstr, kstr, rows);
        };
        fetch(0);
        S::template stage<KM>(lds, ku);
        S::template stage<VM>(lds + 2 * KP, vu);
        lds_barrier();
        // the probabilities of the half's 32-key block k_ of the tile at j0, and dO . v
        auto probs = [&](f32x16& s, f32x16& dp, int buf, int k_, int j0) {
            s = S::template dots<KM>(lds + buf * KP, 32 * k_, qf);
            dp = S::template dots<VM>(lds + 2 * KP + buf * VP, 32 * k_, gf);
            if (j0 + BT - 1 > q0 || q0 + 31 - j0 >= p.window) {
                edge_tile();
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (!swa_sees(p, i, j0 + 32 * k_ + crow(r, h))) s[r] = -INFINITY;
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = exp2_f(s[r] * c - lse2);
        };
        // the wave has pairs in the tile at j0
        auto meets = [&](int j0) { return j0 <= q0 + 31 && (q0 - (j0 + BT - 1) < p.window || j0 < p.sinks); };
        // delta = sum_j p_ij dO_i . v_j also; formed from a 16-bit o it carries that rounding into every
        // ds of the row, which shows where few keys share a row.  Queries with at most kExactTiles
        // key tiles therefore walk them once more, for delta alone.
        if (S::ES == 2 && tl.n <= kExactTiles) {
            float sum = 0.f;
#pragma unroll 1
            for (int t = 0; t < tl.n; ++t) {
                const int j0 = tl.start(t, BT);
                if (meets(j0)) {
#pragma unroll 1
                    for (int u = 0; u < NB / KS; ++u) {
                        f32x16 s, dp;
                        probs(s, dp, 0, ks * (NB / KS) + u, j0);
#pragma unroll
                        for (int r = 0; r < 16; ++r) sum += s[r] * dp[r];
                    }
                }
                const int next = t + 1 < tl.n ? t + 1 : 0;
                if (next != t) {
                    fetch(next);
                    lds_barrier();
                    S::template stage<KM>(lds, ku);
                    S::template stage<VM>(lds + 2 * KP, vu);
                    lds_barrier();
                }
            }
            sum += __shfl_xor(sum, 32);
            delta = sum;
            if constexpr (KS == 2) {
                if (h == 0) dsum[wv][n] = sum;
                __syncthreads();
                delta = dsum[wv % QW][n] + dsum[wv % QW + QW][n];
            }
        }
        for_tiles(tl.n, [&](int t, auto buf_) {
            constexpr int cur = decltype(buf_)::value;
            if (t + 1 < tl.n) fetch(t + 1);
            const int j0 = tl.start(t, BT);
            if (meets(j0)) {
#pragma unroll
                for (int u = 0; u < NB / KS; ++u) {
                    const int k_ = ks * (NB / KS) + u;
                    f32x16 s, dp;
                    probs(s, dp, cur, k_, j0);
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] *= dp[r] - delta;
                    S::template add_rows<KM, FINE>(acc, lds + cur * KP, 32 * k_, s);
                }
            }
            if (t + 1 < tl.n) {
                S::template stage<KM>(lds + (cur ^ 1) * KP, ku);
                S::template stage<VM>(lds + 2 * KP + (cur ^ 1) * VP, vu);
            }
            lds_barrier();
        });
    }
    if constexpr (KS == 2) {
        // the second half's sums, through LDS (the tiles are no longer read)
        constexpr int PITCH = D + 4;
        static_assert(sizeof(lds) >= sizeof(float) * (size_t)QW * 32 * PITCH, "sums of one half fit the tiles");
        float* row = (float*)lds + ((wv % QW) * 32 + n) * PITCH;
        if (ks == 1) S::each4([&](int db, int e, int d0) { *(f32x4*)(row + d0) = S::four(acc[db], e); });
        __syncthreads();
        if (ks == 0)
            S::each4([&](int db, int e, int d0) {
                const f32x4 x = *(const f32x4*)(row + d0);
#pragma unroll
                for (int c4 = 0; c4 < 4; ++c4) acc[db][e + c4] += x[c4];
            });
        __syncthreads();
        if (ks == 1) return;
    }
    const int rows = p.T - q0 >= 32 ? 32 : p.T > q0 ? p.T - q0 : 0;
    S::put_rows(acc, p.scale, lds + wv * S::kPut,
                (char*)p.dq + (((long)b * p.T + q0) * p.H + hd) * D * S::ES, qstr, rows);
    if (h == 0 && n < rows) p.delta[(long)bh * p.T + i] = delta;
}

// One 32-key block of a wave against one 32-query block of the staged tiles: adds to dk and dv
// (columns: keys).  ls / dl: lse (in units of log 2) and delta of the tile's queries.
template <typename T, int D, bool FINE>
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
        f32x16 s = S::template dots<S::kBoth>(qt, r0, kf);
        f32x16 dp = S::template dots<S::kBoth>(gt, r0, vf);
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
        S::template add_rows<S::kBoth, FINE>(dv, gt, r0, s);
        S::template add_rows<S::kBoth, FINE>(dk, qt, r0, dp);
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
        S::template stage<S::kBoth>(qt, qu);
        S::template stage<S::kBoth>(gt, gu);
        if (threadIdx.x < 2 * S::BT) sc[threadIdx.x] = su;
    }
};

// Two kinds of workgroups.  Main ones: 128 keys, 32 per wave, against part `split` of the tiles of the
// queries that see them, head by head.  The first sink_wgs ones: the sinks (at most 64 keys) against one
// piece of the far queries; a wave takes key block wv / NB and query block wv % NB of every tile.
template <typename T, int D, bool FINE>
__global__ __launch_bounds__(kSwaThreads, sizeof(T) * D > 128 ? 1 : 2) void gdr2_swa_dkv_kernel(SwaParams p) {
    using S = Swa<T, D>;
    constexpr int BT = S::BT, NB = S::NB;
    static_assert(kSwaKeyTile == 32 * kSwaWaves, "a wave holds 32 keys");
    __shared__ typename S::template tile<S::kBoth> lds[4];  // queries and cotangents, two of each
    __shared__ float sc[2][2 * BT];
    static_assert(sizeof(lds) >= (size_t)kSwaWaves * S::kPut * 16, "output rows fit the tiles");
    static_assert(sizeof(lds) >= 2 * 32 * D * 2 * sizeof(float), "partial sums of two waves fit the tiles");
    const int l = lane_id(), wv = uniform_wave(), n = l & 31, G = p.H / p.Hkv;
    const int sink_wgs = p.pieces * p.B * p.Hkv;
    const bool far = (int)blockIdx.x < sink_wgs;
    int bh, K0, split = 0, piece = 0;
    if (far) {
        piece = blockIdx.x % p.pieces;
        bh = blockIdx.x / p.pieces;
        K0 = 0;
    } else {
        const int nkt = (p.T + kSwaKeyTile - 1) / kSwaKeyTile;
        const int work = xcd_swizzle(blockIdx.x - sink_wgs, gridDim.x - sink_wgs), job = work / p.splits;
        split = work % p.splits;
        K0 = job % nkt * kSwaKeyTile;
        bh = job / nkt;
    }
    const int b = bh / p.Hkv, kvh = bh % p.Hkv, L = swa_length(p, b);
    const int k0 = K0 + 32 * (far ? wv / NB : wv), j = k0 + n;
    const bool mine = !far || k0 < p.sinks;  // a key block without a sink has no far queries
    const long kstr = (long)p.Hkv * D * S::ES;
    const float c = p.scale * kLog2e;
    const int ia = p.far0 + piece * p.piece_len;
    if (far && ia >= L) return;  // the reduction skips this piece too
    // queries from .. to, in `per` tiles per head; the queries that see the tile's last key, and, with
    // sinks, for the first tile those up to the far ones
    const int from = far ? ia : K0, seen = far ? ia + p.piece_len : K0 == 0 && p.sinks > 0 ? p.far0 : K0 + kSwaKeyTile - 1 + p.window;
    const int to = seen < L ? seen : L;
    const bool key = j < L && (!far || j < p.sinks);
    const long koff = (((long)b * p.T + j) * p.Hkv + kvh) * D * S::ES;
    SwaKeys<T, D, FINE> ks;
    ks.init(key ? (const char*)p.k + koff : nullptr, key ? (const char*)p.v + koff : nullptr);
    if (K0 < L) {
        const int per = (to - from + BT - 1) / BT, all = per * G;
        const int parts = far ? 1 : p.splits;
        const int t0 = (int)((long)all * split / parts), nt = (int)((long)all * (split + 1) / parts) - t0;
        SwaQueries<T, D> qs;
        auto fetch = [&](int t) { qs.fetch(p, b, kvh * G + (t0 + t) / per, from + (t0 + t) % per * BT, L); };
        if (nt > 0) {
            fetch(0);
            qs.stage(lds[0], lds[2], sc[0]);
        }
        lds_barrier();
        for_tiles(nt, [&](int t, auto buf_) {
            constexpr int cur = decltype(buf_)::value;
            if (t + 1 < nt) fetch(t + 1);
            const int i0 = from + (t0 + t) % per * BT;
#pragma unroll
            for (int r = 0; r < NB; ++r) {
                const int ib = i0 + 32 * r;
                if (mine && (!far || r == wv % NB) && ib + 31 >= k0 && (ib - (k0 + 31) < p.window || k0 < p.sinks))
                    ks.step(p, lds[cur], lds[2 + cur], sc[cur], sc[cur] + BT, 32 * r, i0, j,
                            ib < k0 + 31 || ib + 31 - k0 >= p.window, c);
            }
            if (t + 1 < nt) qs.stage(lds[cur ^ 1], lds[2 + (cur ^ 1)], sc[cur ^ 1]);
            lds_barrier();
        });
    }
    if (far) {
        // two query blocks of one key block: the second wave's sums through LDS
        float* buf = (float*)&lds[0][0] + (wv / NB) * 2 * 32 * D + n * D;
        if constexpr (NB == 2) {
            if (mine && wv % NB == 1)
                S::each4([&](int db, int e, int d0) {
                    *(f32x4*)(buf + d0) = S::four(ks.dk[db], e);
                    *(f32x4*)(buf + 32 * D + d0) = S::four(ks.dv[db], e);
                });
            __syncthreads();
        }
        if (!mine || wv % NB != 0) return;
        float* part = p.sink_part + (((long)piece * p.B * p.Hkv + bh) * 2 * kSwaMaxSinks + j) * D;
        S::each4([&](int db, int e, int d0) {
            f32x4 x = S::four(ks.dk[db], e), y = S::four(ks.dv[db], e);
            if constexpr (NB == 2) {
                x += *(const f32x4*)(buf + d0);
                y += *(const f32x4*)(buf + 32 * D + d0);
            }
            *(f32x4*)(part + d0) = x;
            *(f32x4*)(part + (long)kSwaMaxSinks * D + d0) = y;
        });
        return;
    }
    const int rows = p.T - k0 >= 32 ? 32 : p.T > k0 ? p.T - k0 : 0;
    if (p.splits > 1 || (p.pieces > 0 && k0 < kSwaMaxSinks)) {  // fp32 sums for the reduction
        if (n < rows) {
            const long set = (long)p.B * p.part_rows * p.Hkv * D;
            float* part = p.key_part + (long)split * 2 * set + (((long)b * p.part_rows + j) * p.Hkv + kvh) * D;
            S::each4([&](int db, int e, int d0) {
                *(f32x4*)(part + d0) = S::four(ks.dk[db], e);
                *(f32x4*)(part + set + d0) = S::four(ks.dv[db], e);
            });
        }
        return;
    }
    const long ooff = (((long)b * p.T + k0) * p.Hkv + kvh) * D * S::ES;
    i32x4* buf = &lds[0][0] + wv * S::kPut;
    S::put_rows(ks.dk, p.scale, buf, (char*)p.dk + ooff, kstr, rows);
    wave_sync();
    S::put_rows(ks.dv, 1.f, buf, (char*)p.dv + ooff, kstr, rows);
}

// dk and dv of the first part_rows rows: the parts of their queries in order, then, for the sinks, the
// pieces of the far queries.  Four channels per thread.
template <typename T>
__global__ __launch_bounds__(256) void gdr2_swa_reduce_kernel(SwaParams p) {
    const int d4 = p.d / 4;
    const long n4 = (long)p.B * p.part_rows * p.Hkv * d4, x = (long)blockIdx.x * 256 + threadIdx.x;
    if (x >= n4) return;
    const int d0 = (int)(x % d4) * 4, kvh = (int)(x / d4 % p.Hkv), j = (int)(x / d4 / p.Hkv % p.part_rows);
    const int b = (int)(x / d4 / p.Hkv / p.part_rows);
    f32x4 dk = {0, 0, 0, 0}, dv = {0, 0, 0, 0};
    for (int s = 0; s < p.splits; ++s) {
        const f32x4* part = (const f32x4*)p.key_part + (long)s * 2 * n4 + x;
        dk += part[0];
        dv += part[n4];
    }
    if (j < p.sinks) {
        const int L = swa_length(p, b);
        for (int q = 0; q < p.pieces && p.far0 + q * p.piece_len < L; ++q) {
            const float* part = p.sink_part + ((((long)q * p.B + b) * p.Hkv + kvh) * 2 * kSwaMaxSinks + j) * p.d + d0;
            dk += *(const f32x4*)part;
            dv += *(const f32x4*)(part + (long)kSwaMaxSinks * p.d);
        }
    }
    const long o = (((long)b * p.T + j) * p.Hkv + kvh) * p.d + d0;
    store4((T*)p.dk + o, dk * p.scale);
    store4((T*)p.dv + o, dv);
}

template <typename T, int D, bool FINE>
static hipError_t launch_swa_bwd(const SwaParams& p, hipStream_t s) {
    const long heads = (long)p.B * p.H, wide = (p.T + 127) / 128 * heads, narrow = (p.T + 63) / 64 * heads;
    bool done = false;
    if constexpr (Swa<T, D>::NB == 2) {
        if (FINE || wide <= kSwaNarrowMost) {  // (FINE: one workgroup per head either way)
            hipLaunchKernelGGL((gdr2_swa_dq_kernel<T, D, 2, FINE>), dim3((unsigned)narrow), dim3(kSwaThreads), 0, s, p);
            done = true;
        }
    }
    if constexpr (!FINE) {
        if (!done) hipLaunchKernelGGL((gdr2_swa_dq_kernel<T, D, 1, false>), dim3((unsigned)wide), dim3(kSwaThreads), 0, s, p);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const long bk = (long)p.B * p.Hkv, main = (p.T + kSwaKeyTile - 1) / kSwaKeyTile * bk * p.splits;
    hipLaunchKernelGGL((gdr2_swa_dkv_kernel<T, D, FINE>), dim3((unsigned)(main + p.pieces * bk)), dim3(kSwaThreads), 0, s, p);
    e = hipGetLastError();
    if (e != hipSuccess || p.part_rows == 0) return e;
    const long n4 = bk * p.part_rows * (D / 4);
    hipLaunchKernelGGL((gdr2_swa_reduce_kernel<T>), dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, s, p);
    return hipGetLastError();
}

hipError_t swa_bwd_dispatch(int bf, const SwaParams& p, hipStream_t s) {
    if (bf && p.T <= kSwaFine) return p.d == 128 ? launch_swa_bwd<bf16, 128, true>(p, s) : launch_swa_bwd<bf16, 64, true>(p, s);
    if (bf) return p.d == 128 ? launch_swa_bwd<bf16, 128, false>(p, s) : launch_swa_bwd<bf16, 64, false>(p, s);
    return p.d == 128 ? launch_swa_bwd<float, 128, false>(p, s) : launch_swa_bwd<float, 64, false>(p, s);
}

}  // namespace gdr2

// gdr2_swa.hpp -- tiles and products of the sliding-window attention kernels (gfx950).
//
// Every product runs on 32x32 MFMA with fp32 accumulators (bf16: v_mfma_f32_32x32x16_bf16, fp32:
// v_mfma_f32_32x32x2_f32).  Lane l = 32 h + n holds, of a 32x32 product C = A B,
//     C: column n, rows crow(r, h) = 8 (r / 4) + 4 h + r % 4 for its sixteen registers r
//     A: row n, B: column n; the contraction values of half h.
// Scores are formed with the side that is reduced over in the rows (keys for o and dq, queries for
// dk and dv), so that the probabilities a lane holds are contraction values of the next product's B
// operand as they stand: sixteen registers are rows 16 kk + {4h..4h+3, 8+4h..8+4h+3}, kk = 0, 1,
// and its A operand is gathered from the LDS tile in that same order (ds_read_b64_tr_b16 for bf16,
// one float per register for fp32).  No probability ever crosses lanes.
#pragma once
#include "gdr2_block_kernels.hpp"
#include "gdr2_common.hpp"

namespace gdr2 {

typedef float f32x16 __attribute__((ext_vector_type(16)));
constexpr int kSwaThreads = 256, kSwaWaves = 4;
// Workgroups of 128 queries: up to five for four compute units, 64 queries each and the keys in two halves (the
// busiest unit then has three half shares instead of two whole ones; past that the halves' joining costs more).
// Window 2048, T=4096, d=128 bf16, forward, us with 128 / 64 queries: 128 workgroups 51 / 38, 256 52 / 50,
// 288 69 / 59, 320 69 / 67, 384 70 / 85; backward 141 / 121, 151 / 147, 210 / 194, -, -, 512 260 / 275.  Window 512,
// T=8192, d=64: 256 18 / 19, 320 21 / 18, 448 21 / 24.  B=2 T=777 H=6 d=64 fp32 (84): 39 / 22 and 100 / 75.
constexpr long kSwaNarrowMost = 320;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.0e38f;

__device__ __forceinline__ int crow(int r, int h) { return 8 * (r / 4) + 4 * h + r % 4; }
__device__ __forceinline__ float exp2_f(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ f32x16 zero16() {
    return f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
}

template <typename T, int D>
struct Swa {
    static constexpr int ES = (int)sizeof(T), CPR = D * ES / 16;  // 16-byte pieces per row
    static constexpr int KK = CPR / 2;                            // contraction steps of a row
    static constexpr int DB = D / 32;                             // 32-column blocks of a row
    static constexpr int BT = D * ES > 256 ? 32 : 64;             // rows of a staged tile (at most 16 KB)
    static constexpr int NB = BT / 32;
    static constexpr int UNITS = BT * CPR / kSwaThreads;          // pieces a thread stages
    static_assert(UNITS * kSwaThreads == BT * CPR, "staging");

    // 16-byte piece (row, c) of a tile.  kRows tiles are read by whole pieces of 16 rows at a time: padded
    // by one piece, those rows fall in different banks.  kBoth tiles are also read by 64 bytes of four
    // rows (add_rows): padded by four pieces, and piece c kept at c ^ (row / 4 % 4) inside its group of
    // four, both reads are free of bank conflicts, at addresses that differ by constants.
    static constexpr int kRows = 1, kBoth = 4;
    template <int M> static constexpr int kPitch = CPR + M;
    template <int M> using tile = i32x4[BT * kPitch<M>];
    // piece 4 * group + c of a row
    template <int M>
    static __device__ __forceinline__ int at(int row, int group, int c) {
        return row * kPitch<M> + 4 * group + (M == kBoth ? c ^ ((row >> 2) & 3) : c);
    }

    // BT rows of a token tensor into registers: row r at base + r * stride bytes.  Only the first `rows`
    // (>= 1) exist; the last of them stands in for the others, which no live pair uses.
    static __device__ __forceinline__ void fetch(i32x4 (&u)[UNITS], const char* base, long stride, int rows) {
        constexpr int RSTEP = kSwaThreads / CPR;  // rows between a thread's pieces
        const unsigned st = (unsigned)stride, c = threadIdx.x % CPR * 16;  // strides stay below 2^24 + 1
        const unsigned off = threadIdx.x / CPR * st + c, last = (rows - 1) * st + c;
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            const unsigned o = off + i * RSTEP * st;
            u[i] = *(const i32x4*)(base + (o < last ? o : last));
        }
    }
    template <int M>
    static __device__ __forceinline__ void stage(i32x4* t, const i32x4 (&u)[UNITS]) {
        constexpr int RSTEP = kSwaThreads / CPR;
        const int r0 = threadIdx.x / CPR, c = threadIdx.x % CPR;
#pragma unroll
        for (int i = 0; i < UNITS; ++i) t[at<M>(r0 + i * RSTEP, c / 4, c % 4)] = u[i];
    }
    // the B operand of 32 rows, kept in registers: piece 2 kk + h of the lane's row (null: zeros)
    static __device__ __forceinline__ void keep(i32x4 (&f)[KK], const char* row) {
        const int h = lane_id() >> 5;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
            f[kk] = row ? *(const i32x4*)(row + (2 * kk + h) * 16) : i32x4{0, 0, 0, 0};
    }
    static __device__ __forceinline__ void mma(f32x16& c, const i32x4& a, const i32x4& b) {
        if constexpr (ES == 2) {
            c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
        } else {
            const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
            for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[e], y[e], c, 0, 0, 0);
        }
    }
    // rows r0 .. r0 + 31 of a tile times the kept rows: C[r][n] = tile row . kept row
    template <int M>
    static __device__ __forceinline__ f32x16 dots(const i32x4* t, int r0, const i32x4 (&f)[KK]) {
        const int l = lane_id(), row = r0 + (l & 31), h = l >> 5;
        f32x16 c = zero16();
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) mma(c, t[at<M>(row, kk / 2, 2 * (kk % 2) + h)], f[kk]);
        return c;
    }
    // acc[db][d][n] += sum over the rows r0 + crow(r, h) of tile[row][32 db + d] w[r] (for bf16 the
    // weights are rounded to bf16: the products' inputs, relative error 2^-8 each, summed in fp32; FINE adds the
    // product of what that rounding left, 2^-16 each)
    template <int M, bool FINE = false>
    static __device__ __forceinline__ void add_rows(f32x16 (&acc)[DB], const i32x4* t, int r0, const f32x16& w) {
        const int l = lane_id(), h = l >> 5;
        if constexpr (ES == 2) {
            const int p = l & 15, sub = (l >> 4) & 1;
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                bf16x8 b;
#pragma unroll
                for (int e = 0; e < 8; ++e) b[e] = (bf16)w[8 * kk + e];
                bf16x8 rest;
                if constexpr (FINE) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) rest[e] = (bf16)(w[8 * kk + e] - (float)b[e]);
                }
                const int ra = r0 + 16 * kk + 4 * h + (p >> 2), rb = ra + 8;
#pragma unroll
                for (int db = 0; db < DB; ++db) {
                    const int c = 2 * sub + ((p & 3) >> 1);
                    const bf16x4 lo = ds_read_tr4((const bf16*)(t + at<M>(ra, db, c)) + 4 * (p & 1));
                    const bf16x4 hi = ds_read_tr4((const bf16*)(t + at<M>(rb, db, c)) + 4 * (p & 1));
                    const bf16x8 a = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                    acc[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc[db], 0, 0, 0);
                    if constexpr (FINE) acc[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, rest, acc[db], 0, 0, 0);
                }
            }
        } else {
            const int n = l & 31;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = r0 + crow(r, h);
#pragma unroll
                for (int db = 0; db < DB; ++db) {
                    const float a = ((const float*)(t + at<M>(row, 2 * db + (n >> 4), (n >> 2) & 3)))[n & 3];
                    acc[db] = __builtin_amdgcn_mfma_f32_32x32x2f32(a, w[r], acc[db], 0, 0, 0);
                }
            }
        }
    }
    // The lane's values of its row (32 rows, lane column n = row), four channels at a time
    template <typename F>
    static __device__ __forceinline__ void each4(F&& f) {
        const int h = lane_id() >> 5;
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int j = 0; j < 4; ++j) f(db, 4 * j, 32 * db + 8 * j + 4 * h);  // block, first register, first channel
    }
    static __device__ __forceinline__ f32x4 four(const f32x16& a, int e) { return f32x4{a[e], a[e + 1], a[e + 2], a[e + 3]}; }

    // Writes 32 rows (lane column n = row) of D values, acc * mul, as whole rows through the wave's
    // own kPut pieces of LDS: row n goes to out + n * stride bytes for n < rows.
    static constexpr int kPut = 32 * kPitch<kRows>;
    static __device__ __forceinline__ void put_rows(const f32x16 (&acc)[DB], float mul, i32x4* buf, char* out,
                                                    long stride, int rows) {
        const int l = lane_id(), n = l & 31, h = l >> 5;
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f32x4 x = {acc[db][4 * j] * mul, acc[db][4 * j + 1] * mul, acc[db][4 * j + 2] * mul, acc[db][4 * j + 3] * mul};
                const int d0 = 32 * db + 8 * j + 4 * h, c = d0 * ES / 16;
                if constexpr (ES == 2)
                    *((bf16x4*)(buf + at<kRows>(n, c / 4, c % 4)) + h) = bf16x4{(bf16)x[0], (bf16)x[1], (bf16)x[2], (bf16)x[3]};
                else
                    *(f32x4*)(buf + at<kRows>(n, c / 4, c % 4)) = x;
            }
        wave_sync();
#pragma unroll
        for (int i = 0; i < 32 * CPR / 64; ++i) {
            const int x = l + i * 64, r = x / CPR, c = x % CPR;
            const i32x4 u = buf[at<kRows>(r, c / 4, c % 4)];
            if (r < rows) *(i32x4*)(out + r * stride + c * 16) = u;
        }
    }
};

// the wave's index as a wave-uniform value, so that conditions on its rows are scalar branches
__device__ __forceinline__ int uniform_wave() { return __builtin_amdgcn_readfirstlane(wave_id()); }

// Positions inside a sequence are ints (T <= 2^30); addresses are formed in 64 bits.
// Tokens of sequence b: its length clamped to [0, T].
__device__ __forceinline__ int swa_length(const SwaParams& p, int b) {
    if (!p.lengths) return p.T;
    const int L = p.lengths[b];
    return L < 0 ? 0 : L > p.T ? p.T : L;
}
// The x-th query tile of a head in the order of the launch.  Tiles inside the first window grow with their
// position; where they are half of the head or more, the last ones go first, so that the launch ends with
// short ones (B=4 T=1500 H=12 d=128 window 2048: forward 64 -> 50 us, backward 208 -> 191; B=4 T=4096 H=16 forward
// 259 -> 256).  Longer sequences go in order, each tile's keys just read by the one before (T=32768, H=16/4:
// 0.54 GB from memory and 610 us, against 1.31 GB and 615 us backwards).
__device__ __forceinline__ int swa_query_tile(const SwaParams& p, int x, int nqt) {
    return p.T - p.window <= p.window ? nqt - 1 - x : x;
}
// Keeps the masking of an edge tile behind its branch: most tiles are seen whole.
__device__ __forceinline__ void edge_tile() { asm volatile(""); }
// Calls f(t, IC<buffer>) for t = 0 .. n - 1 with the LDS buffer t % 2 as a constant.
template <typename F>
__device__ __forceinline__ void for_tiles(int n, F&& f) {
    for (int t = 0; t < n; t += 2) {
        f(t, IC<0>{});
        if (t + 1 < n) f(t + 1, IC<1>{});
    }
}
__device__ __forceinline__ bool swa_sees(const SwaParams& p, int i, int j) {
    return j <= i && (i - j < p.window || j < p.sinks);
}

// Key tiles (of BT keys) that queries qa .. qb may see: `extra` tiles with sinks from the start of
// the sequence, then tiles first .. last.
struct SwaTiles {
    int extra, first, n;
    __device__ __forceinline__ SwaTiles(const SwaParams& p, int bt, int qa, int qb) {
        const int lo = qa - p.window + 1;
        first = lo > 0 ? lo / bt : 0;
        const int s = (p.sinks + bt - 1) / bt;
        extra = s < first ? s : first;
        n = extra + qb / bt - first + 1;
    }
    __device__ __forceinline__ int start(int i, int bt) const { return (i < extra ? i : first + i - extra) * bt; }
};

}  // namespace gdr2

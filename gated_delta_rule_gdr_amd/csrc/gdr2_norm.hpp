// gdr2_norm.hpp -- rows in registers, shared by the norms (gfx950): how a row of D channels is laid over the
// lanes and waves of a workgroup, its loads and stores, and how many workgroups keep column sums.
#pragma once
#include "gdr2_block_kernels.hpp"
#include "gdr2_common.hpp"

namespace gdr2 {

constexpr int kNormThreads = 512, kNormWaves = kNormThreads / 64;
// Workgroups of the backward, each with one partial of the weight's gradient: one per compute unit,
// up to two where that leaves each at least four passes over its rows (16384 x 2048 bf16: 41 us with
// 256, 39 with 512, 42 with 1024; 4099 x 1000 fp32: 24 us with 256, 26 with 512).
constexpr long kNormBlocks = 256, kNormMaxBlocks = 512, kNormPasses = 4;

// sum over the LPR lanes that share a row (LPR a power of two, aligned groups), in all of them
template <int LPR>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int m = 1; m < LPR; m <<= 1) x += __shfl_xor(x, m);
    return x;
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* v) {
    if constexpr (sizeof(T) == 2) {
        const bf16x8 x = *(const bf16x8*)p;
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = (float)x[c];
    } else {
        const f32x4 a = *(const f32x4*)p, b = *(const f32x4*)(p + 4);
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = a[c], v[c + 4] = b[c];
    }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* v) {
    if constexpr (sizeof(T) == 2) {
        bf16x8 x;
#pragma unroll
        for (int c = 0; c < 8; ++c) x[c] = (bf16)v[c];  // RNE
        *(bf16x8*)p = x;
    } else {
        *(f32x4*)p = f32x4{v[0], v[1], v[2], v[3]};
        *(f32x4*)(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
}

// The row a thread works on and its columns: LPR lanes (WPR == 1) or WPR whole waves per row; a
// thread's piece u is the eight channels at col + u * stride.
template <int LPR, int WPR>
struct RowMap {
    static constexpr int kRows = WPR > 1 ? kNormWaves / WPR : kNormWaves * (64 / LPR);  // per pass
    static constexpr int kStride = WPR > 1 ? WPR * 64 * 8 : LPR * 8;
    int row, col, part;  // row of the pass, first column, wave's place in the row
    __device__ __forceinline__ RowMap() {
        const int l = lane_id(), w = wave_id();
        row = WPR > 1 ? w / WPR : w * (64 / LPR) + l / LPR;
        part = w % WPR;
        col = 8 * (WPR > 1 ? part * 64 + l : l % LPR);
    }
    // the row's sum of x (every thread of the workgroup calls it)
    __device__ __forceinline__ float sum(float x, float* red) const {
        x = lanes_sum<LPR>(x);
        if constexpr (WPR > 1) {
            if (lane_id() == 0) red[wave_id()] = x;
            __syncthreads();
            x = 0.f;
#pragma unroll
            for (int i = 0; i < WPR; ++i) x += red[row * WPR + i];
            __syncthreads();
        }
        return x;
    }
};

// Calls f(NV, LPR, WPR constants) for rows of D channels: the narrowest lane group whose single
// piece covers the row, then up to two pieces of 1, 2, 4 or 8 waves, then four of 8 (two pieces over two
// waves rather than four over one: 16384 x 2048 bf16 backward 47 -> 39 us, since the registers of
// four pieces leave two waves per SIMD).
template <typename F>
static auto with_row_shape(int D, F&& f) {
    if (D <= 64) return f(IC<1>{}, IC<8>{}, IC<1>{});
    if (D <= 128) return f(IC<1>{}, IC<16>{}, IC<1>{});
    if (D <= 256) return f(IC<1>{}, IC<32>{}, IC<1>{});
    if (D <= 512) return f(IC<1>{}, IC<64>{}, IC<1>{});
    if (D <= 1024) return f(IC<2>{}, IC<64>{}, IC<1>{});
    if (D <= 2048) return f(IC<2>{}, IC<64>{}, IC<2>{});
    if (D <= 4096) return f(IC<2>{}, IC<64>{}, IC<4>{});
    if (D <= 8192) return f(IC<2>{}, IC<64>{}, IC<8>{});
    return f(IC<4>{}, IC<64>{}, IC<8>{});
}

// Workgroups that walk `rows` rows with column sums in registers (one partial each).
inline long norm_part_blocks(long rows, int D) {
    return with_row_shape(D, [&](auto, auto lpr, auto wpr) -> long {
        constexpr int R = RowMap<decltype(lpr)::value, decltype(wpr)::value>::kRows;
        const long passes = (rows + R - 1) / R;
        long n = passes / kNormPasses;
        n = n < kNormBlocks ? kNormBlocks : n < kNormMaxBlocks ? n : kNormMaxBlocks;
        return n < passes ? n : passes;
    });
}

}  // namespace gdr2

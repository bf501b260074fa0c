// gdr2_norm.hip -- layer normalisation before a mixer, forward and backward (gfx950).
//
// Per row of D channels (D a multiple of 8):
//     mean = sum_j x_j / D,   rstd = 1 / sqrt(sum_j (x_j - mean)^2 / D + eps)
//     n_j = (x_j - mean) rstd,   y_j = n_j weight_j + bias_j
// and for the cotangent dy, with a_j = dy_j weight_j:
//     dx_j = rstd (a_j - sum_i a_i / D - n_j sum_i a_i n_i / D)
//     dweight_j = sum over rows of dy_j n_j,   dbias_j = sum over rows of dy_j
//
// Both passes are streams: a row is read once into registers (eight channels per lane and piece,
// at most four pieces), the variance is the second pass over those registers (no cancellation of
// large means), and the row leaves once.  A row belongs to 8..64 lanes of a wave, or, above 1024
// channels, to 2, 4 or 8 waves that exchange their sums through LDS; sums are fp32.  The weight's
// and bias' gradients are summed without atomics: every workgroup walks rows with its columns'
// partial sums in registers and writes one partial per column, and a second kernel adds the
// partials in a fixed order, so results do not change from run to run.
// 16384 x 2048 bf16: forward 25 us (134 MB, 5.4 TB/s), backward 35 us (201 MB, 5.7 TB/s) and 4 us for the second
// kernel; 4099 x 1000 fp32: 8.4 us and 11.6 + 3.9 us, launches and ramps; 256 x 2048 bf16 forward 4.1 us.
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

template <typename T, int NV, int LPR, int WPR>
__global__ __launch_bounds__(kNormThreads) void gdr2_norm_fwd_kernel(NormParams p) {
    using RM = RowMap<LPR, WPR>;
    __shared__ float red[kNormWaves];
    const RM m;
    const int D = p.D;
    const float inv = 1.f / (float)D;
    const long row = (long)blockIdx.x * RM::kRows + m.row;
    const long rl = row < p.rows ? row : p.rows - 1;  // rows past the end are read, not stored
    const T* __restrict__ x = (const T*)p.x + rl * D;
    float v[NV][8];
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int c = m.col + u * RM::kStride;
        load8(x + (c < D ? c : 0), v[u]);
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        if (m.col + u * RM::kStride < D) {
#pragma unroll
            for (int e = 0; e < 8; ++e) s += v[u][e];
        }
    }
    const float mean = m.sum(s, red) * inv;
    float ss = 0.f;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        if (m.col + u * RM::kStride < D) {
#pragma unroll
            for (int e = 0; e < 8; ++e) ss += (v[u][e] - mean) * (v[u][e] - mean);
        }
    }
    const float rstd = 1.f / sqrtf(m.sum(ss, red) * inv + p.eps);
    if (row >= p.rows) return;
    T* y = (T*)p.y + row * D;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int c = m.col + u * RM::kStride;
        if (c < D) {
            float w[8], b[8] = {}, r[8];
            load8(p.weight + c, w);
            if (p.bias) load8(p.bias + c, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) r[e] = (v[u][e] - mean) * rstd * w[e] + b[e];
            store8(y + c, r);
        }
    }
    if (m.col == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
}

template <typename T, int NV, int LPR, int WPR>
__global__ __launch_bounds__(kNormThreads) void gdr2_norm_bwd_kernel(NormParams p) {
    using RM = RowMap<LPR, WPR>;
    __shared__ float red[kNormWaves];
    __shared__ float cols[2][NV * RM::kStride];  // the workgroup's column sums
    const RM m;
    const int D = p.D;
    const float inv = 1.f / (float)D;
    float dw[NV][8], db[NV][8], w[NV][8];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int c = m.col + u * RM::kStride;
        load8(p.weight + (c < D ? c : 0), w[u]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[u][e] = db[u][e] = 0.f;
    }
    // the trip count is the same for every thread of the workgroup
    for (long r0 = (long)blockIdx.x * RM::kRows; r0 < p.rows; r0 += (long)gridDim.x * RM::kRows) {
        const long row = r0 + m.row;
        const bool live = row < p.rows;
        const long rl = live ? row : p.rows - 1;
        const T* __restrict__ x = (const T*)p.x + rl * D;
        const T* __restrict__ dy = (const T*)p.dy + rl * D;
        float n[NV][8], a[NV][8];
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int c = m.col + u * RM::kStride;
            load8(x + (c < D ? c : 0), n[u]);
            load8(dy + (c < D ? c : 0), a[u]);
        }
        const float mean = p.mean[rl], rstd = p.rstd[rl];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            if (live && m.col + u * RM::kStride < D) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    n[u][e] = (n[u][e] - mean) * rstd;
                    dw[u][e] += a[u][e] * n[u][e];
                    db[u][e] += a[u][e];
                    a[u][e] *= w[u][e];
                    s1 += a[u][e];
                    s2 += a[u][e] * n[u][e];
                }
            }
        }
        s1 = m.sum(s1, red) * inv;
        s2 = m.sum(s2, red) * inv;
        if (live) {
            T* dx = (T*)p.dx + row * D;
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                const int c = m.col + u * RM::kStride;
                if (c < D) {
                    float r[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) r[e] = rstd * (a[u][e] - s1 - n[u][e] * s2);
                    store8(dx + c, r);
                }
            }
        }
    }
    // lane groups of a wave that hold the same columns, then the waves in turn
    if constexpr (WPR == 1) {
#pragma unroll
        for (int k = LPR; k < 64; k <<= 1)
#pragma unroll
            for (int u = 0; u < NV; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dw[u][e] += __shfl_xor(dw[u][e], k);
                    db[u][e] += __shfl_xor(db[u][e], k);
                }
    }
    for (int t = 0; t < RM::kRows * (WPR > 1 ? 1 : LPR) / (WPR > 1 ? 1 : 64); ++t) {
        const bool mine = WPR > 1 ? m.row == t : wave_id() == t && lane_id() < LPR;
        if (mine) {
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                const int c = m.col + u * RM::kStride;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    cols[0][c + e] = t ? cols[0][c + e] + dw[u][e] : dw[u][e];
                    cols[1][c + e] = t ? cols[1][c + e] + db[u][e] : db[u][e];
                }
            }
        }
        __syncthreads();
    }
    float* part = p.part + (long)blockIdx.x * 2 * D;
    for (int c = threadIdx.x; c < D; c += kNormThreads) {
        part[c] = cols[0][c];
        part[D + c] = cols[1][c];
    }
}

// Column sums of the partials: 64 columns per workgroup, sixteen threads per column over strided
// subsets, then those sixteen in order.  blockIdx.y: 0 dweight, 1 dbias.
constexpr int kNormRedThreads = 1024, kNormRedGroups = kNormRedThreads / 64;
__global__ __launch_bounds__(kNormRedThreads) void gdr2_norm_reduce_kernel(NormParams p, long nparts) {
    __shared__ float red[kNormRedGroups][64];
    const int l = lane_id(), g = wave_id();
    const int c = blockIdx.x * 64 + l;
    const bool live = c < p.D;
    const float* src = p.part + (long)blockIdx.y * p.D + (live ? c : 0);
    float acc = 0.f;
#pragma unroll 8
    for (long i = g; i < nparts; i += kNormRedGroups) acc += src[i * 2 * p.D];
    red[g][l] = acc;
    __syncthreads();
    if (g == 0 && live) {
        acc = 0.f;
#pragma unroll
        for (int i = 0; i < kNormRedGroups; ++i) acc += red[i][l];
        (blockIdx.y ? p.dbias : p.dweight)[c] = acc;
    }
}

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

long norm_bwd_blocks(long rows, int D) {
    return with_row_shape(D, [&](auto, auto lpr, auto wpr) -> long {
        constexpr int R = RowMap<decltype(lpr)::value, decltype(wpr)::value>::kRows;
        const long passes = (rows + R - 1) / R;
        long n = passes / kNormPasses;
        n = n < kNormBlocks ? kNormBlocks : n < kNormMaxBlocks ? n : kNormMaxBlocks;
        return n < passes ? n : passes;
    });
}

template <typename T>
static hipError_t launch_norm(bool bwd, const NormParams& p, hipStream_t s) {
    return with_row_shape(p.D, [&](auto nv, auto lpr, auto wpr) -> hipError_t {
        constexpr int NV = decltype(nv)::value, LPR = decltype(lpr)::value, WPR = decltype(wpr)::value;
        constexpr int R = RowMap<LPR, WPR>::kRows;
        if (!bwd) {
            const long most = max_workgroups(kNormThreads) * R;
            for (long r0 = 0; r0 < p.rows; r0 += most) {
                NormParams c = p;
                c.rows = p.rows - r0 < most ? p.rows - r0 : most;
                c.x = (const T*)p.x + r0 * p.D;
                c.y = (T*)p.y + r0 * p.D;
                if (p.mean) c.mean = p.mean + r0;
                if (p.rstd) c.rstd = p.rstd + r0;
                hipLaunchKernelGGL((gdr2_norm_fwd_kernel<T, NV, LPR, WPR>), dim3((unsigned)((c.rows + R - 1) / R)),
                                   dim3(kNormThreads), 0, s, c);
                const hipError_t e = hipGetLastError();
                if (e != hipSuccess) return e;
            }
            return hipSuccess;
        }
        const long nb = norm_bwd_blocks(p.rows, p.D);
        if (nb > 0) {
            hipLaunchKernelGGL((gdr2_norm_bwd_kernel<T, NV, LPR, WPR>), dim3(nb), dim3(kNormThreads), 0, s, p);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        hipLaunchKernelGGL(gdr2_norm_reduce_kernel, dim3((p.D + 63) / 64, p.dbias ? 2 : 1), dim3(kNormRedThreads),
                           0, s, p, nb);
        return hipGetLastError();
    });
}

hipError_t norm_dispatch(int bf, bool bwd, const NormParams& p, hipStream_t s) {
    return bf ? launch_norm<bf16>(bwd, p, s) : launch_norm<float>(bwd, p, s);
}

}  // namespace gdr2

// gdr2_rms.hip -- RMS norm of a residual stream, forward, with an 8-bit result, and backward (gfx950).
//
// Per row of D channels (D a multiple of 8), h = x + residual rounded to the stream's type:
//     rstd = 1 / sqrt(sum_j h_j^2 / D + eps),   n_j = h_j rstd,   y_j = n_j weight_j
// and for the cotangents dy of y and dh of h, with a_j = dy_j weight_j:
//     dx_j = dh_j + rstd (a_j - n_j sum_i a_i n_i / D),   dweight_j = sum over rows of dy_j n_j
// The 8-bit result divides the row, or each group of channels, by its largest magnitude over 448 (e4m3's
// largest value), so that value is met exactly and nothing overflows; y is rounded once, from fp32.
//
// All are streams: a row is read once into registers (eight channels per lane and piece), and leaves once.
// A row belongs to 8..64 lanes of a wave or to 2, 4 or 8 waves (gdr2_norm.hpp); a group's eight channels per
// lane make its largest magnitude a maximum over 4, 8 or 16 neighbouring lanes.  The weight's gradient is
// summed as the layer norm's is: column sums in registers, one partial per workgroup, added in a fixed order.
//
// Measured (16384 rows of 2048, bf16, with a residual): forward 46 us, 5.8 TB/s with what the caches keep; with 8-bit
// values and a scale per 128 channels 40 us; backward 46 us and 5 for the partials.  A plain copy reaches 5.0 TB/s.
#include "gdr2_hybrid_kernels.hpp"
#include "gdr2_norm.hpp"

namespace gdr2 {

constexpr float kE4m3Max = 448.f, kLeastScale = 1e-37f;

// The larger magnitude as bits: a NaN's lie above infinity's, so one in the group is kept.
__device__ __forceinline__ unsigned magnitude(float x) { return __builtin_bit_cast(unsigned, x) & 0x7fffffffu; }
__device__ __forceinline__ unsigned lanes_max(unsigned x, int lanes) {
    for (int m = 1; m < lanes; m <<= 1) {
        const unsigned y = (unsigned)__shfl_xor((int)x, m);
        x = x > y ? x : y;
    }
    return x;
}

template <typename T, bool Q8, int NV, int LPR, int WPR>
__global__ __launch_bounds__(kNormThreads) void gdr2_rms_fwd_kernel(RmsParams p) {
    using RM = RowMap<LPR, WPR>;
    __shared__ float red[kNormWaves];
    const RM m;
    const int D = p.D;
    const long row = (long)blockIdx.x * RM::kRows + m.row;
    const bool live = row < p.rows;
    const long rl = live ? row : p.rows - 1;  // rows past the end are read, not stored
    const T* x = (const T*)p.x + rl * D;
    float v[NV][8];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int c = m.col + u * RM::kStride;
        load8(x + (c < D ? c : 0), v[u]);
    }
    if (p.residual) {
        const T* r = (const T*)p.residual + rl * D;
        float a[NV][8];
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int c = m.col + u * RM::kStride;
            load8(r + (c < D ? c : 0), a[u]);
        }
        // the stream is kept in its type: the norm goes on with the rounded sum
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int c = m.col + u * RM::kStride;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[u][e] = to_f(from_f<T>(v[u][e] + a[u][e]));
            if (live && c < D) store8((T*)p.h + row * D + c, v[u]);
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        if (m.col + u * RM::kStride < D) {
#pragma unroll
            for (int e = 0; e < 8; ++e) ss += v[u][e] * v[u][e];
        }
    }
    const float rstd = 1.f / sqrtf(m.sum(ss, red) * (1.f / (float)D) + p.eps);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int c = m.col + u * RM::kStride;
        float w[8];
        load8(p.weight + (c < D ? c : 0), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[u][e] *= rstd * w[e];
        if constexpr (!Q8) {
            if (live && c < D) store8((T*)p.y + row * D + c, v[u]);
        }
    }
    if constexpr (Q8) {
        unsigned top[NV];
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            top[u] = 0;
            if (m.col + u * RM::kStride < D) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const unsigned b = magnitude(v[u][e]);
                    top[u] = top[u] > b ? top[u] : b;
                }
            }
        }
        if (p.group) {
            const int lanes = p.group / 8 < LPR ? p.group / 8 : LPR;
#pragma unroll
            for (int u = 0; u < NV; ++u) top[u] = lanes_max(top[u], lanes);
        } else {
            unsigned t = 0;
#pragma unroll
            for (int u = 0; u < NV; ++u) t = t > top[u] ? t : top[u];
            t = lanes_max(t, LPR);
            if constexpr (WPR > 1) {
                __shared__ unsigned most[kNormWaves];
                if (lane_id() == 0) most[wave_id()] = t;
                __syncthreads();
#pragma unroll
                for (int i = 0; i < WPR; ++i) t = t > most[m.row * WPR + i] ? t : most[m.row * WPR + i];
            }
#pragma unroll
            for (int u = 0; u < NV; ++u) top[u] = t;
        }
        if (!live) return;
        const int per = p.group ? (D + p.group - 1) / p.group : 1;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int c = m.col + u * RM::kStride;
            if (c < D) {
                const float most = __builtin_bit_cast(float, top[u]);
                const bool fine = top[u] < 0x7f800000u;
                float s = most * (1.f / kE4m3Max);
                s = !fine ? __builtin_nanf("") : top[u] == 0 ? 0.f : fmaxf(s, kLeastScale);
                const float inv = top[u] == 0 ? 0.f : 1.f / s;
                float q[8];
                // |y| / scale is at most 448 (1 + 2^-22): within half a step of 448, never above it after rounding
#pragma unroll
                for (int e = 0; e < 8; ++e) q[e] = v[u][e] * inv;
                int lo = 0, hi = 0;
                lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], lo, false);
                lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
                hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], hi, false);
                hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
                int2 out = {lo, hi};
                *(int2*)((unsigned char*)p.y + row * D + c) = out;
                if (p.group ? c % p.group == 0 : c == 0) p.scale[row * per + (p.group ? c / p.group : 0)] = s;
            }
        }
    } else {
        if (live && m.col == 0 && p.rstd) p.rstd[row] = rstd;
    }
}

template <typename T, int NV, int LPR, int WPR>
__global__ __launch_bounds__(kNormThreads) void gdr2_rms_bwd_kernel(RmsParams p) {
    using RM = RowMap<LPR, WPR>;
    __shared__ float red[kNormWaves];
    __shared__ float cols[NV * RM::kStride];  // the workgroup's column sums
    const RM m;
    const int D = p.D;
    const float inv = 1.f / (float)D;
    float dw[NV][8], w[NV][8];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int c = m.col + u * RM::kStride;
        load8(p.weight + (c < D ? c : 0), w[u]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[u][e] = 0.f;
    }
    // the trip count is the same for every thread of the workgroup
    for (long r0 = (long)blockIdx.x * RM::kRows; r0 < p.rows; r0 += (long)gridDim.x * RM::kRows) {
        const long row = r0 + m.row;
        const bool live = row < p.rows;
        const long rl = live ? row : p.rows - 1;
        const T* __restrict__ h = (const T*)p.x + rl * D;
        const T* __restrict__ dy = (const T*)p.dy + rl * D;
        const T* __restrict__ dh = p.dh ? (const T*)p.dh + rl * D : nullptr;
        float n[NV][8], a[NV][8], g[NV][8] = {};
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int c = m.col + u * RM::kStride;
            load8(h + (c < D ? c : 0), n[u]);
            load8(dy + (c < D ? c : 0), a[u]);
            if (dh) load8(dh + (c < D ? c : 0), g[u]);
        }
        const float rstd = p.rstd[rl];
        float s = 0.f;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            if (live && m.col + u * RM::kStride < D) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    n[u][e] *= rstd;
                    dw[u][e] += a[u][e] * n[u][e];
                    a[u][e] *= w[u][e];
                    s += a[u][e] * n[u][e];
                }
            }
        }
        s = m.sum(s, red) * inv;
        if (live) {
            T* dx = (T*)p.dx + row * D;
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                const int c = m.col + u * RM::kStride;
                if (c < D) {
                    float r[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) r[e] = g[u][e] + rstd * (a[u][e] - n[u][e] * s);
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
                for (int e = 0; e < 8; ++e) dw[u][e] += __shfl_xor(dw[u][e], k);
    }
    constexpr int kTurns = WPR > 1 ? RM::kRows : kNormWaves;
    for (int t = 0; t < kTurns; ++t) {
        const bool mine = WPR > 1 ? m.row == t : wave_id() == t && lane_id() < LPR;
        if (mine) {
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                const int c = m.col + u * RM::kStride;
#pragma unroll
                for (int e = 0; e < 8; ++e) cols[c + e] = t ? cols[c + e] + dw[u][e] : dw[u][e];
            }
        }
        __syncthreads();
    }
    float* part = p.part + (long)blockIdx.x * D;
    for (int c = threadIdx.x; c < D; c += kNormThreads) part[c] = cols[c];
}

// Column sums of the partials: 64 columns per workgroup, sixteen threads per column over strided
// subsets, then those sixteen in order.
constexpr int kRmsRedThreads = 1024, kRmsRedGroups = kRmsRedThreads / 64;
__global__ __launch_bounds__(kRmsRedThreads) void gdr2_rms_reduce_kernel(RmsParams p, long nparts) {
    __shared__ float red[kRmsRedGroups][64];
    const int l = lane_id(), g = wave_id();
    const int c = blockIdx.x * 64 + l;
    const bool live = c < p.D;
    const float* src = p.part + (live ? c : 0);
    float acc = 0.f;
#pragma unroll 8
    for (long i = g; i < nparts; i += kRmsRedGroups) acc += src[i * p.D];
    red[g][l] = acc;
    __syncthreads();
    if (g == 0 && live) {
        acc = 0.f;
#pragma unroll
        for (int i = 0; i < kRmsRedGroups; ++i) acc += red[i][l];
        p.dweight[c] = acc;
    }
}

long rms_bwd_blocks(long rows, int D) { return norm_part_blocks(rows, D); }

template <typename T, bool Q8>
static hipError_t launch_rms_fwd(const RmsParams& p, hipStream_t s) {
    return with_row_shape(p.D, [&](auto nv, auto lpr, auto wpr) -> hipError_t {
        constexpr int NV = decltype(nv)::value, LPR = decltype(lpr)::value, WPR = decltype(wpr)::value;
        constexpr int R = RowMap<LPR, WPR>::kRows;
        const long most = max_workgroups(kNormThreads) * R;
        const long per = p.group ? (p.D + p.group - 1) / p.group : 1;
        for (long r0 = 0; r0 < p.rows; r0 += most) {
            RmsParams c = p;
            c.rows = p.rows - r0 < most ? p.rows - r0 : most;
            c.x = (const T*)p.x + r0 * p.D;
            if (p.residual) {
                c.residual = (const T*)p.residual + r0 * p.D;
                c.h = (T*)p.h + r0 * p.D;
            }
            c.y = (char*)p.y + r0 * p.D * (Q8 ? 1 : (long)sizeof(T));
            if (p.rstd) c.rstd = p.rstd + r0;
            if (p.scale) c.scale = p.scale + r0 * per;
            hipLaunchKernelGGL((gdr2_rms_fwd_kernel<T, Q8, NV, LPR, WPR>), dim3((unsigned)((c.rows + R - 1) / R)),
                               dim3(kNormThreads), 0, s, c);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    });
}

template <typename T>
static hipError_t launch_rms_bwd(const RmsParams& p, hipStream_t s) {
    return with_row_shape(p.D, [&](auto nv, auto lpr, auto wpr) -> hipError_t {
        constexpr int NV = decltype(nv)::value, LPR = decltype(lpr)::value, WPR = decltype(wpr)::value;
        const long nb = rms_bwd_blocks(p.rows, p.D);
        if (nb > 0) {
            hipLaunchKernelGGL((gdr2_rms_bwd_kernel<T, NV, LPR, WPR>), dim3((unsigned)nb), dim3(kNormThreads), 0, s, p);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        hipLaunchKernelGGL(gdr2_rms_reduce_kernel, dim3((p.D + 63) / 64), dim3(kRmsRedThreads), 0, s, p, nb);
        return hipGetLastError();
    });
}

template <typename T>
static hipError_t launch_rms(RmsKind kind, const RmsParams& p, hipStream_t s) {
    return kind == kRmsBwd ? launch_rms_bwd<T>(p, s) : kind == kRmsQ8 ? launch_rms_fwd<T, true>(p, s) : launch_rms_fwd<T, false>(p, s);
}

hipError_t rms_dispatch(int bf, RmsKind kind, const RmsParams& p, hipStream_t s) {
    return bf ? launch_rms<bf16>(kind, p, s) : launch_rms<float>(kind, p, s);
}

}  // namespace gdr2

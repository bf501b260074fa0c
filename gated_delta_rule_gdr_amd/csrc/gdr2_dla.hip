// gdr2_dla.hip -- linear attention with a fixed decay per head: prompts, gradients and single tokens (gfx950).
//
// With a = exp(log_decay), S_t = a S_{t-1} + k_t v_t^T, o_t = S_t^T q_t and R_t = a R_{t+1} + q_t dO_t^T,
//     dq_t = S_t dO_t,   dk_t = R_t v_t,   dv_t = R_t^T k_t,   dS0 = a R_0
// are, like o, all of the form (gdr2_hybrid_kernels.hpp)
//     out_t = sum over s <= t of a^(t - s) (x_t . y_s) z_s
// so one kernel computes each as a pass, with time turned round for dk and dv, and the backward needs nothing
// kept by the forward.  Chunks of 64 tokens: inside a chunk through the scores x_r . y_s, weighted a^(r - s);
// from before it through the state, out_r += a^(r + 1) x_r S; then S <- a^64 S + sum_s a^(63 - s) y_s z_s^T.
//
// A workgroup carries 32 or 64 columns of one chain's state in fp32 registers (columns are independent), over the
// whole sequence or, where there are few chains, over one segment of it, whose entering state is put together from
// the segments' own states (a first launch).  Scores are formed transposed (rows s, columns r), so that a lane's
// weighted scores are operand values of the next product as they stand; the state is read from a bf16 copy in LDS
// that each chunk writes for the next one.  Tiles are double buffered in LDS, one barrier per chunk.
//
// Rounding: S is carried in fp32, its decay as S + S (a^n - 1), so that slow decays lose nothing over long
// sequences; the decayed operand of its sums is split into two bf16 (16 bits).  Scores, and S as it is read, are
// rounded to bf16 once as inputs of their products, whose sums are fp32.  fp32 rounds nothing else.
#include "gdr2_common.hpp"
#include "gdr2_hybrid_kernels.hpp"

namespace gdr2 {

constexpr int kDlaThreads = 256, C = kDlaChunk;

// a^n for whole n >= 0; a^0 = 1 also where a = 0
__device__ __forceinline__ float dla_pow(float g, int n) { return n == 0 ? 1.f : expf((float)n * g); }

template <typename T, int K, int VS>
struct Dla {
    static constexpr int ES = (int)sizeof(T), E16 = 16 / ES;            // elements of a 16-byte piece
    static constexpr int KP = K * ES / 64;                              // operand pieces of a row per lane
    static constexpr int PY = K + E16, PZ = VS + E16;                   // LDS pitches, elements
    static constexpr int YU = C * K * ES / 16 / kDlaThreads, ZU = C * VS * ES / 16 / kDlaThreads;  // pieces a thread stages
    static constexpr int KB = K / 64, VB = VS / 16;                     // a wave's 16-row blocks of the state, and columns'
    static_assert(YU >= 1 && ZU >= 1, "staging");

    // products of 16 x 16 by 64 bytes of contraction
    static __device__ __forceinline__ void mma(f32x4& c, const i32x4& a, const i32x4& b) {
        if constexpr (ES == 2) {
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
        } else {
            const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
            for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], y[e], c, 0, 0, 0);
        }
    }
    // piece kk of row i0 + l % 16 of a tile
    static __device__ __forceinline__ i32x4 row(const T* t, int pitch, int i0, int kk) {
        const int l = lane_id();
        return *(const i32x4*)(t + (i0 + (l & 15)) * pitch + (kk * 4 + (l >> 4)) * E16);
    }
};

template <typename T, int K, int VS, bool LOCAL>
__global__ __launch_bounds__(kDlaThreads) void gdr2_dla_kernel(DlaParams p, int V, int nwork) {
    using W = Dla<T, K, VS>;
    constexpr int ES = W::ES, E16 = W::E16, KP = W::KP, KB = W::KB, VB = W::VB, PY = W::PY, PZ = W::PZ;
    __shared__ __align__(16) T Yl[2][C * PY];
    __shared__ __align__(16) T Zl[2][C * PZ];
    __shared__ __align__(16) T Sl[LOCAL ? 1 : 2][LOCAL ? 8 : VS * PY];

    // work items: slices of a chain's columns next to each other, then passes, segments, heads, sequences;
    // neighbours, which read the same rows, run on one XCD
    const int per = gridDim.x / 8, item = blockIdx.x % 8 * per + blockIdx.x / 8;
    if (item >= nwork) return;
    const int slices = V / VS, segs = LOCAL ? p.segs - 1 : p.segs;
    const int sl = item % slices, ip = item / slices % p.passes, sg = item / slices / p.passes % segs;
    const int bh = item / slices / p.passes / segs, h = bh % p.H, b = bh / p.H;
    const DlaPass& ps = p.pass[ip];
    const int l = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id()), c = l & 15, g = l >> 4, tid = threadIdx.x;

    int L = p.lengths ? p.lengths[b] : p.T;
    L = L < 0 ? 0 : L > p.T ? p.T : L;
    const int nch = (L + C - 1) / C, c0 = sg * p.seg_chunks;
    const int c1 = c0 + p.seg_chunks < nch ? c0 + p.seg_chunks : nch;
    if (LOCAL && c1 - c0 < p.seg_chunks) return;  // no later segment has a token: nobody reads this one's state
    const float ga = p.log_decay[h];
    const bool rev = ps.reverse;

    // rows: token t of the pass is row t, or L - 1 - t against time
    const long sx = (long)p.H * K * ES * (rev ? -1 : 1), sz = (long)p.H * V * ES * (rev ? -1 : 1);
    const long row0 = ((long)b * p.T + (rev ? L - 1 : 0)) * p.H + h;
    const char* X = (const char*)ps.x + row0 * K * ES;
    const char* Y = (const char*)ps.y + row0 * K * ES;
    const char* Z = (const char*)ps.z + (row0 * V + sl * VS) * ES;
    char* O = (char*)ps.out + (row0 * V + sl * VS) * ES;

    // The state: blocks of 16 x 16, rows k = 16 (w + 4 kb) + 4 g + i, columns v = 16 vb + c
    f32x4 S[KB][VB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int vb = 0; vb < VB; ++vb) S[kb][vb] = f32x4{0, 0, 0, 0};
    const int tsl = KB * VB * kDlaThreads * 4;  // numbers of a slice's state
    const long chain = ((long)ip * p.B + b) * p.H + h;
    auto each_state = [&](auto&& f) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int vb = 0; vb < VB; ++vb)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = 16 * (w + 4 * kb) + 4 * g + i, v = sl * VS + 16 * vb + c;
                    f(S[kb][vb], i, ((long)b * p.H + h) * K * V + (ps.flip ? (long)v * K + k : (long)k * V + v));
                }
    };
    // Against time the state before the first token is undecayed at that token: one power less (in the first chunk).
    const int early = rev ? 1 : 0;
    if constexpr (!LOCAL) {
        if (ps.init) each_state([&](f32x4& s, int i, long at) { s[i] = ps.init[at]; });
        for (int j = 0; j < sg; ++j) {
            if (c0 >= nch && sg > 0) break;  // no token here
            const float e = expm1f((float)(p.seg_chunks * C - (j == 0 ? early : 0)) * ga);
            const f32x4* src = (const f32x4*)(p.local + ((chain * (p.segs - 1) + j) * slices + sl) * tsl) + tid;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int vb = 0; vb < VB; ++vb) {
                    const f32x4 x = src[(kb * VB + vb) * kDlaThreads];
#pragma unroll
                    for (int i = 0; i < 4; ++i) S[kb][vb][i] = fmaf(S[kb][vb][i], e, S[kb][vb][i]) + x[i];
                }
        }
    }
    auto put_state = [&](T* dst) {  // as read by the next chunk: [v][k]
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int vb = 0; vb < VB; ++vb) store4(dst + (16 * vb + c) * PY + 16 * (w + 4 * kb) + 4 * g, S[kb][vb]);
    };

    // staging: piece u of a thread is row (tid + 256 u) / pieces of a row
    constexpr int YR = K * ES / 16, ZR = VS * ES / 16;
    i32x4 yr[W::YU], zr[W::ZU], xr[KP];
    const int xrow = 16 * w + c;
    auto fetch = [&](int ch) {
        const int n = L - ch * C;
#pragma unroll
        for (int u = 0; u < W::YU; ++u) {
            const int x = tid + u * kDlaThreads, r = x / YR, q = x % YR;
            yr[u] = r < n ? *(const i32x4*)(Y + (ch * C + r) * sx + q * 16) : i32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int u = 0; u < W::ZU; ++u) {
            const int x = tid + u * kDlaThreads, r = x / ZR, q = x % ZR;
            zr[u] = r < n ? *(const i32x4*)(Z + (ch * C + r) * sz + q * 16) : i32x4{0, 0, 0, 0};
        }
        if constexpr (!LOCAL) {
#pragma unroll
            for (int kk = 0; kk < KP; ++kk)
                xr[kk] = xrow < n ? *(const i32x4*)(X + (ch * C + xrow) * sx + (kk * 4 + g) * 16) : i32x4{0, 0, 0, 0};
        }
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int u = 0; u < W::YU; ++u) {
            const int x = tid + u * kDlaThreads, r = x / YR, q = x % YR;
            *(i32x4*)(Yl[buf] + r * PY + q * E16) = yr[u];
        }
#pragma unroll
        for (int u = 0; u < W::ZU; ++u) {
            const int x = tid + u * kDlaThreads, r = x / ZR, q = x % ZR;
            *(i32x4*)(Zl[buf] + r * PZ + q * E16) = zr[u];
        }
    };

    // weights that every chunk shares: near[b][i] = a^(r - s) of score block b, late[j] = a^(63 - s)
    float near[4][4], late[16];
#pragma unroll
    for (int sb = 0; sb < 4; ++sb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int lag = xrow - (16 * sb + 4 * g + i);
            near[sb][i] = lag < 0 ? 0.f : dla_pow(ga, lag);
        }
    // token of the lane's contraction value j of the state's products
    auto late_token = [&](int j) { return ES == 2 ? 32 * (j / 8) + 8 * g + j % 8 : 4 * j + g; };
#pragma unroll
    for (int j = 0; j < 16; ++j) late[j] = dla_pow(ga, C - 1 - late_token(j));
    float carry = expm1f((float)C * ga);

    if (c0 < c1) {
        fetch(c0);
        stage(0);
        if constexpr (!LOCAL) put_state(Sl[0]);
    }
    i32x4 xf[KP];
    int buf = 0;
    for (int ch = c0; ch < c1; ++ch, buf ^= 1) {
        lds_barrier();
        const int n = L - ch * C < C ? L - ch * C : C;
        if constexpr (!LOCAL) {
#pragma unroll
            for (int kk = 0; kk < KP; ++kk) xf[kk] = xr[kk];
        }
        if (ch + 1 < c1) fetch(ch + 1);
        const T *yl = Yl[buf], *zl = Zl[buf];
        if constexpr (!LOCAL) {
            const T* st = Sl[buf];
            // from before the chunk: out^T = S^T x, rows v, columns r
            f32x4 out[VB];
#pragma unroll
            for (int vb = 0; vb < VB; ++vb) out[vb] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int kk = 0; kk < KP; ++kk)
#pragma unroll
                for (int vb = 0; vb < VB; ++vb) W::mma(out[vb], W::row(st, PY, 16 * vb, kk), xf[kk]);
            const float before = dla_pow(ga, xrow + 1 - (ch == 0 ? early : 0));
#pragma unroll
            for (int vb = 0; vb < VB; ++vb) out[vb] *= before;
            // scores, rows s, columns r; blocks behind the wave's rows are not seen
            f32x4 sc[4];
#pragma unroll
            for (int sb = 0; sb < 4; ++sb) {
                sc[sb] = f32x4{0, 0, 0, 0};
                if (sb <= w) {
#pragma unroll
                    for (int kk = 0; kk < KP; ++kk) W::mma(sc[sb], W::row(yl, PY, 16 * sb, kk), xf[kk]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[sb][i] = near[sb][i] == 0.f ? 0.f : sc[sb][i] * near[sb][i];
                }
            }
            // out^T += z^T scores^T
            if constexpr (ES == 2) {
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    if (2 * kk <= w) {
                        bf16x8 pr;
#pragma unroll
                        for (int e = 0; e < 4; ++e) pr[e] = (bf16)sc[2 * kk][e], pr[4 + e] = (bf16)sc[2 * kk + 1][e];
#pragma unroll
                        for (int vb = 0; vb < VB; ++vb) {
                            const T* a = zl + (32 * kk + 4 * g + (c >> 2)) * PZ + 16 * vb + 4 * (c & 3);
                            const bf16x4 lo = ds_read_tr4(a), hi = ds_read_tr4(a + 16 * PZ);
                            out[vb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7), pr, out[vb], 0, 0, 0);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int sb = 0; sb < 4; ++sb) {
                    if (sb <= w) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int vb = 0; vb < VB; ++vb)
                                out[vb] = __builtin_amdgcn_mfma_f32_16x16x4f32(zl[(16 * sb + 4 * g + i) * PZ + 16 * vb + c], sc[sb][i], out[vb], 0, 0, 0);
                    }
                }
            }
            if (xrow < n) {
#pragma unroll
                for (int vb = 0; vb < VB; ++vb) store4((T*)(O + (ch * C + xrow) * sz) + 16 * vb + 4 * g, out[vb]);
            }
        }
        // the state behind the chunk
        if (n < C) {
#pragma unroll
            for (int j = 0; j < 16; ++j) late[j] = late_token(j) < n ? dla_pow(ga, n - 1 - late_token(j)) : 0.f;
        }
        const int decays = n - (ch == 0 ? early : 0);
        const float e = decays == C ? carry : decays == 0 ? 0.f : expm1f((float)decays * ga);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int vb = 0; vb < VB; ++vb)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[kb][vb][i] = fmaf(S[kb][vb][i], e, S[kb][vb][i]);
        if constexpr (ES == 2) {
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                bf16x8 hi[KB], lo[KB];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    const bf16x8 y = Frag<bf16>::tr(yl, PY, 32 * kk, 16 * (w + 4 * kb), l);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float f = (float)y[j] * late[8 * kk + j];
                        hi[kb][j] = (bf16)f;
                        lo[kb][j] = (bf16)(f - (float)hi[kb][j]);
                    }
                }
#pragma unroll
                for (int vb = 0; vb < VB; ++vb) {
                    const bf16x8 z = Frag<bf16>::tr(zl, PZ, 32 * kk, 16 * vb, l);
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb) {
                        Mfma<bf16>::mma(S[kb][vb], hi[kb], z);
                        Mfma<bf16>::mma(S[kb][vb], lo[kb], z);
                    }
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                float y[KB];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) y[kb] = yl[(4 * j + g) * PY + 16 * (w + 4 * kb) + c] * late[j];
#pragma unroll
                for (int vb = 0; vb < VB; ++vb) {
                    const float z = zl[(4 * j + g) * PZ + 16 * vb + c];
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb) mma32(S[kb][vb], y[kb], z);
                }
            }
        }
        if (ch + 1 < c1) {
            stage(buf ^ 1);
            if constexpr (!LOCAL) put_state(Sl[buf ^ 1]);
        }
    }

    if constexpr (LOCAL) {
        f32x4* dst = (f32x4*)(p.local + ((chain * (p.segs - 1) + sg) * slices + sl) * tsl) + tid;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int vb = 0; vb < VB; ++vb) dst[(kb * VB + vb) * kDlaThreads] = S[kb][vb];
    } else {
        // the final state, by the segment of the last token; against time it is decayed once more (dS0 = a R_0)
        if (ps.fin && (nch == 0 ? sg == 0 : c0 < nch && c1 == nch)) {
            const float f = rev && L > 0 ? dla_pow(ga, 1) : 1.f;
            each_state([&](f32x4& s, int i, long at) { ps.fin[at] = s[i] * f; });
        }
        // padding rows of the segment's part of the time axis
        const long t0 = L > (long)c0 * C ? L : (long)c0 * C, t1 = sg + 1 < p.segs ? (long)(c0 + p.seg_chunks) * C : p.T;
        char* out = (char*)ps.out + ((((long)b * p.T) * p.H + h) * V + sl * VS) * ES;
        for (long x = tid; x < (t1 - t0) * ZR; x += kDlaThreads)
            *(i32x4*)(out + (t0 + x / ZR) * p.H * V * ES + x % ZR * 16) = i32x4{0, 0, 0, 0};
    }
}

DlaCut dla_cut(long B, long T, long H, int passes, int K, int V, bool f32) {
    DlaCut c{32, 1, 1};
    const long nch = (T + C - 1) / C, jobs = B * H * passes * (V / c.slice);
    long segs = jobs > 0 ? 512 / jobs : 1;
    segs = segs < nch / 16 ? segs : nch / 16;
    segs = segs < 1 ? 1 : segs;
    c.seg_chunks = (int)((nch + segs - 1) / segs);
    c.seg_chunks = c.seg_chunks < 1 ? 1 : c.seg_chunks;
    c.segs = (int)((nch + c.seg_chunks - 1) / c.seg_chunks);
    c.segs = c.segs < 1 ? 1 : c.segs;
    return c;
}

template <typename T, int K, int VS>
static hipError_t launch_dla(int V, const DlaParams& p, hipStream_t s) {
    const long per = (long)p.passes * (V / VS);
    const long chains = (long)p.B * p.H;
    if (p.segs > 1) {
        const long n = chains * per * (p.segs - 1);
        hipLaunchKernelGGL((gdr2_dla_kernel<T, K, VS, true>), dim3((unsigned)((n + 7) / 8 * 8)), dim3(kDlaThreads), 0, s, p, V, (int)n);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const long n = chains * per * p.segs;
    hipLaunchKernelGGL((gdr2_dla_kernel<T, K, VS, false>), dim3((unsigned)((n + 7) / 8 * 8)), dim3(kDlaThreads), 0, s, p, V, (int)n);
    return hipGetLastError();
}

template <typename T>
static hipError_t launch_dla(int K, int V, const DlaCut& c, const DlaParams& p, hipStream_t s) {
    return K == 128 ? launch_dla<T, 128, 32>(V, p, s) : launch_dla<T, 64, 32>(V, p, s);
}

hipError_t dla_dispatch(int bf, int K, int V, const DlaCut& c, const DlaParams& p, hipStream_t s) {
    return bf ? launch_dla<bf16>(K, V, c, p, s) : launch_dla<float>(K, V, c, p, s);
}

// One token: S <- a S + k v^T, o = S^T q.  A pure stream over the fp32 state, in registers, 16-byte accesses.
template <typename T, int DK, int DV>
__global__ __launch_bounds__(kDlaThreads) void gdr2_dla_step_kernel(DlaStepParams p) {
    constexpr int CG = DV / 4, RG = kDlaThreads / CG, R = DK / RG;  // column groups, row groups, rows of a thread
    __shared__ f32x4 red[RG][CG];
    const long n = blockIdx.x;
    const int jg = threadIdx.x % CG, ig = threadIdx.x / CG;
    const T *q = (const T*)p.q + n * DK, *k = (const T*)p.k + n * DK, *v = (const T*)p.v + n * DV;
    const long at = n * DK * DV + 4 * jg;
    f32x4 s[R];
#pragma unroll
    for (int u = 0; u < R; ++u) s[u] = p.S_in ? *(const f32x4*)(p.S_in + at + (ig * R + u) * DV) : f32x4{0, 0, 0, 0};
    const float a = expf(p.log_decay[n % p.H]);
    const f32x4 vv = load4(v + 4 * jg);
    f32x4 o = {0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < R; ++u) {
        const int i = ig * R + u;
        const float ki = to_f(k[i]), qi = to_f(q[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[u][j] = fmaf(a, s[u][j], ki * vv[j]);
            o[j] = fmaf(qi, s[u][j], o[j]);
        }
        *(f32x4*)(p.S_out + at + i * DV) = s[u];
    }
    red[ig][jg] = o;
    __syncthreads();
    if (ig == 0) {
#pragma unroll
        for (int r = 1; r < RG; ++r) o += red[r][jg];
        store4((T*)p.o + n * DV + 4 * jg, o);
    }
}

template <typename T, int DK, int DV>
static hipError_t launch_step(const DlaStepParams& p, hipStream_t s) {
    hipLaunchKernelGGL((gdr2_dla_step_kernel<T, DK, DV>), dim3((unsigned)p.n), dim3(kDlaThreads), 0, s, p);
    return hipGetLastError();
}
template <typename T>
static hipError_t launch_step(int dk, int dv, const DlaStepParams& p, hipStream_t s) {
    if (dk == 128) return dv == 128 ? launch_step<T, 128, 128>(p, s) : launch_step<T, 128, 64>(p, s);
    return dv == 128 ? launch_step<T, 64, 128>(p, s) : launch_step<T, 64, 64>(p, s);
}
hipError_t dla_step_dispatch(int bf, int dk, int dv, const DlaStepParams& p, hipStream_t s) {
    return bf ? launch_step<bf16>(dk, dv, p, s) : launch_step<float>(dk, dv, p, s);
}

}  // namespace gdr2

// gdr2_block_kernels.hpp -- host-side launch interface of the operators around the GDR-2 mixer:
// layer norm, gated linear recurrence, sliding-window attention and its decode.
#pragma once
#include <hip/hip_runtime.h>

namespace gdr2 {

// Workgroups of one launch: HIP takes gridDim.x * blockDim.x up to 2^32 - 1.  Problems of more rows,
// batch rows or sequences than that are cut into several launches.
inline constexpr long max_workgroups(int threads) { return (((long)1 << 32) - 1) / threads; }

// Layer norm over the last axis: y = (x - mean) rstd weight + bias per row of D channels.
struct NormParams {
    long rows;
    int D;
    float eps;
    const void* x;        // [rows][D] input dtype
    const float* weight;  // [D]
    const float* bias;    // [D] or null
    void* y;              // forward output [rows][D]
    float *mean, *rstd;   // [rows] fp32: forward outputs (null = not wanted), backward inputs
    const void* dy;       // backward: cotangent of y
    void* dx;             // backward output [rows][D]
    float *dweight, *dbias;  // backward outputs [D] (dbias null = not wanted)
    float* part;          // backward workspace [norm_bwd_blocks(rows, D)][2][D] fp32
};
constexpr int kNormMaxD = 16384;
long norm_bwd_blocks(long rows, int D);
hipError_t norm_dispatch(int dtype_bf16, bool bwd, const NormParams& p, hipStream_t s);

// Gated linear recurrence h_t = exp(log_a_t) h_{t-1} + x_t per channel.
constexpr int kGlrFwdSeg = 256, kGlrBwdSeg = 128;  // tokens of a segment: a workgroup's share of the time axis
constexpr int kGlrCh = 64;      // channels of a workgroup
constexpr int kGlrGroup = 16;   // segments between two published running states
constexpr int kGlrFwdThreads = 2 * kGlrFwdSeg, kGlrBwdThreads = 2 * kGlrBwdSeg;  // eight channels of four tokens each
struct GlrParams {
    int B, nseg, nstrip;
    long T, D;
    const void* x;        // [B][T][D] input dtype
    const float* la;      // [B][T][D]
    const float* h0;      // [B][D] or null
    void* h;              // [B][T][D] input dtype
    float* hT;            // [B][D] or null
    float* states;        // [B][segments of the backward][D]: the state entering each
    const void* dh;       // backward: cotangent of h
    const float* dhT;     // [B][D] or null
    void* dx;             // [B][T][D] input dtype
    float* dla;           // [B][T][D]
    float* dh0;           // [B][D] or null
    unsigned long long* pub;  // [B][nseg][nstrip * kGlrCh] published segment maps, then
                              // [B][nseg / kGlrGroup][..] published running states
    unsigned* ticket;
};
inline __host__ __device__ long glr_segments(long T, int seg) { return T <= 0 ? 1 : (T + seg - 1) / seg; }
inline long glr_strips(long D) { return (D + kGlrCh - 1) / kGlrCh; }
// One batch row's segments have to fit a launch; batch rows are cut into launches that use pub and
// ticket in turn.
hipError_t glr_dispatch(int dtype_bf16, bool bwd, const GlrParams& p, hipStream_t s);
struct GlrStepParams {
    long n;               // N * D elements
    const void* x;
    const float* la;
    const float* h_in;    // may equal h_out; null = zero state
    float* h_out;
    void* h;
};
hipError_t glr_step_dispatch(int dtype_bf16, const GlrStepParams& p, hipStream_t s);

// Sliding-window attention with sinks: query i of a sequence of L tokens sees key j when
// j <= i < L and (i - j < window or j < sinks).
constexpr int kSwaMaxSinks = 64;
constexpr int kSwaKeyTile = 128;    // keys of a key/value-gradient workgroup
struct SwaParams {
    int B, H, Hkv, d, sinks;
    int T, window;          // T <= 2^30, window <= T
    float scale;
    const void *q, *k, *v;  // [B][T][H][d], [B][T][Hkv][d]
    const int* lengths;     // [B] or null (every sequence has T tokens)
    void* o;                // [B][T][H][d] (forward output, backward input)
    float* lse;             // [B][H][T] log of the softmax denominators (natural; -inf: nothing seen)
    const void* dO;         // backward
    void *dq, *dk, *dv;
    float* delta;           // [B][H][T] sum of dO o per query (backward workspace)
    // dk and dv in parts (backward workspace, fp32)
    float* sink_part;       // [pieces][B][Hkv][2][64][d]: the sinks' from the far queries
    float* key_part;        // [splits][2][B][part_rows][Hkv][d]
    int splits, part_rows;  // part_rows: rows that the reduction writes (0: it is not needed)
    int pieces;             // 0: no query lies behind the window, or no sinks
    int far0, piece_len;    // piece i covers queries far0 + i * piece_len ..
};
// How the key/value gradients are cut.  far0: the first query the first key tile's workgroups leave
// to the sinks' pieces.
struct SwaCut {
    int splits, part_rows, pieces, far0, piece_len;
};
// Workgroups of 128 keys fill the card once there are as many as compute units (256); with fewer, the
// queries of a tile are cut into up to eight parts of at least two tiles of 64, towards the workgroups the
// card holds: d=64 bf16 two per unit, d=128 one, unless whole parts leave an eighth of the units idle.  (The type
// is not asked: the workspace query does not know it.  fp32 d=64 holds one per unit and is cut for two.)
// Backward in us uncut / up to four / eight / sixteen parts: T=2048 H=16/4 d=128 window 2048 bf16 356 / 155 / 152 /
// 182, T=512 H=8/2 d=64 70 / 34 / 28 / 29, B=2 T=777 H=6/2 d=64 fp32 202 / 88 / 75 / 76; cut at 256 workgroups
// too: T=4096 H=8 d=128 162 -> 195.  Towards one / two per unit, T=4096 window 2048 d=128: 4 heads (128
// workgroups) 119 / 133, 5 heads 153 / 147, 7 heads 155 / 171; T=2048 H=8 window 512 50 / 65; d=64 T=1537 H=12/3 83 / 69.
// Pieces of the far queries: up to one workgroup per two compute units, at least 128 queries and at most 64
// pieces per head (us with 64 / 128 / 256 / 512 workgroups: B=4 T=4096 H=16 d=128 window 2048 947 / 949 / 954 / 959,
// T=8192 H=8 window 1024 195 / 189 / 190 / 202, T=16384 H=16/4 window 2048 1254 / 1196 / 1188 / 1187).
inline SwaCut swa_cut(long B, long T, long H, long Hkv, long d, long window, int sinks) {
    SwaCut c{1, 0, 0, 0, 0};
    const long heads = B * Hkv, jobs = (T + kSwaKeyTile - 1) / kSwaKeyTile * heads;
    const long seen = window + kSwaKeyTile < T ? window + kSwaKeyTile : T, tiles = (seen + 63) / 64 * (H / Hkv);
    if (jobs < 256) {
        const long one = 256 / jobs, want = d == 128 && one * jobs >= 224 ? one : 512 / jobs;
        const long s = want < tiles / 2 ? want : tiles / 2;
        c.splits = (int)(s < 1 ? 1 : s < 8 ? s : 8);
    }
    const long far0 = (kSwaKeyTile - 1 + window + 63) / 64 * 64;
    c.far0 = (int)far0;
    if (sinks > 0 && T > far0) {
        const long want = heads < 128 ? 128 / heads : 1, most = (T - far0 + 127) / 128;
        long n = want < most ? want : most;
        n = n < 64 ? n : 64;
        c.piece_len = (int)(((T - far0 + n - 1) / n + 63) / 64 * 64);
        c.pieces = (int)((T - far0 + c.piece_len - 1) / c.piece_len);
    }
    c.part_rows = c.splits > 1 ? (int)T : c.pieces > 0 ? (int)(T < kSwaMaxSinks ? T : kSwaMaxSinks) : 0;
    return c;
}
hipError_t swa_fwd_dispatch(int dtype_bf16, const SwaParams& p, hipStream_t s);
hipError_t swa_bwd_dispatch(int dtype_bf16, const SwaParams& p, hipStream_t s);

// The bounded cache: [N][sinks + window][Hkv][d]; position p lives in slot p (p < sinks) or
// sinks + (p - sinks) mod window.
struct SwaFillParams {
    int B, Hkv, sinks;
    long T, window, row16;  // row16: 16-byte pieces of a token's row (all heads)
    const void *k, *v;      // [B][T][Hkv][d]
    void *kc, *vc;
    const int* lengths;
    long first;             // the launch's first piece of the caches (set by the dispatch)
};
hipError_t swa_fill_dispatch(const SwaFillParams& p, hipStream_t s);
struct SwaDecodeParams {
    int N, H, Hkv, d, sinks;
    long window;
    float scale;
    const void *q, *k, *v;  // [N][H][d], [N][Hkv][d]
    void *kc, *vc;
    const int* pos;         // [N] position of the new token; negative: no token
    void* o;                // [N][H][d]
    int splits;             // parts of the slots per (sequence, key/value head, head group)
    float* part;            // splits > 1: [N][Hkv][groups][splits][16][d + 4] fp32 (a row, its maximum and sum)
};
int swa_decode_splits(long N, long Hkv, long groups, long slots);
hipError_t swa_decode_dispatch(int dtype_bf16, const SwaDecodeParams& p, hipStream_t s);

}  // namespace gdr2

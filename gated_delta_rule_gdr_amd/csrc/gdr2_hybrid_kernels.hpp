// gdr2_hybrid_kernels.hpp -- host-side launch interface of the RMS norm of a residual stream, linear
// attention with a decay per head, and the paged key/value cache.
#pragma once
#include <hip/hip_runtime.h>

#include "gdr2_block_kernels.hpp"

namespace gdr2 {

// RMS norm of h = x + residual per row of D channels, its result in dtype or in 8 bits with scales.
struct RmsParams {
    long rows;
    int D, group;         // group: channels per scale (0: the row)
    float eps;
    const void* x;        // forward [rows][D]; backward: the stream h
    const void* residual; // [rows][D] or null
    const float* weight;  // [D]
    void* h;              // [rows][D], with a residual; may equal it
    void* y;              // [rows][D] dtype or bytes
    float* rstd;          // [rows]: forward output (null = not wanted), backward input
    float* scale;         // [rows] or [rows][ceil(D / group)] (8-bit result)
    const void *dy, *dh;  // backward cotangents (dh null = zero)
    void* dx;
    float* dweight;
    float* part;          // backward workspace [rms_bwd_blocks(rows, D)][D] fp32
};
enum RmsKind { kRmsFwd, kRmsQ8, kRmsBwd };
long rms_bwd_blocks(long rows, int D);
hipError_t rms_dispatch(int dtype_bf16, RmsKind kind, const RmsParams& p, hipStream_t s);

// The paged key/value cache: k_pages and v_pages [pages][page][Hkv][d]; position p of sequence n is row p % page of
// page table[n][p / page], if that entry lies in [0, pages).
struct PagedFillParams {
    int B, T, shift, pages, width;  // page = 1 << shift rows
    int row16;              // 16-byte pieces of a token's row (all heads)
    const void *k, *v;      // [B][T][Hkv][d]
    const int *start, *lengths, *table;
    void *kp, *vp;
    long first, n;          // the launch's first piece, and the pieces of all tokens (set by the dispatch)
};
hipError_t paged_fill_dispatch(const PagedFillParams& p, hipStream_t s);

constexpr int kPagedHeads = 16;     // query heads of a workgroup: the columns of its products
constexpr int kPagedStep = 128;     // positions that a workgroup takes at a time
struct PagedDecodeParams {
    int N, H, Hkv, d, shift, pages, width;
    float scale;
    const void *q, *k, *v;  // [N][H][d], [N][Hkv][d]
    const int *table, *pos;
    void *kp, *vp;
    void* o;                // [N][H][d]
    int splits;             // parts of the positions per (sequence, key/value head, head group)
    float* part;            // splits > 1: [N][Hkv][groups][splits][16][d + 4] fp32 (a row, its maximum and sum)
};
int paged_splits(long N, long Hkv, long groups, long capacity);
hipError_t paged_decode_dispatch(int dtype_bf16, const PagedDecodeParams& p, hipStream_t s);

// Linear attention with a fixed decay per head.  Every result of the forward and of the backward is one pass of
//     out_t = sum over s <= t of a^(t - s) (x_t . y_s) z_s, and what the state before the first token adds,
// in the order of time or against it:
//     o: x, y, z = q, k, v     dq: dO, v, k     dk: v, dO, q (against time)     dv: k, q, dO (against time)
// with the state, sums of a^.. y_s z_s^T, carried in fp32.
struct DlaPass {
    int K, V;
    const void *x, *y, *z;  // [B][T][H][K], [B][T][H][K], [B][T][H][V]
    void* out;              // [B][T][H][V]
    const float* init;      // the state before the first token, [B][H][K][V] or (flip) [B][H][V][K]; null = zero
    float* fin;             // the state behind the last one, likewise; null = not wanted
    int reverse, flip;
    int state;              // whether the final state is a result of the operator, wanted or not
    int slot;               // slots of the passes before it
};
constexpr int kDlaChunk = 64;
struct DlaCut {
    int segs, seg_chunks;   // segments of the sequence, and their chunks
};
struct DlaParams {
    int B, T, H, passes;
    int slots;              // workgroups of a segment of one chain, over the passes
    int segs, seg_chunks;
    const float* log_decay;
    const int* lengths;     // [B] or null
    DlaPass pass[3];
    float* local;           // segs > 1: [passes][B][H][segs - 1][dk * dv] fp32, a segment's own state in the kernel's order
};
int dla_slots(int V, bool f32);  // of a pass
DlaCut dla_cut(long B, long T, long H, long slots, bool f32);
hipError_t dla_dispatch(int dtype_bf16, const DlaParams& p, hipStream_t s);
struct DlaStepParams {
    long n;                 // N * H chains
    int H;
    const void *q, *k, *v;
    const float* log_decay;
    const float* S_in;      // may equal S_out; null = zero
    float* S_out;
    void* o;
};
hipError_t dla_step_dispatch(int dtype_bf16, int dk, int dv, const DlaStepParams& p, hipStream_t s);

}  // namespace gdr2

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
// A workgroup carries the columns of one chain's state (fp32: 32 of them; columns are independent) in fp32 registers,
// over the whole sequence or, where there are few chains, over one segment of it, whose entering state is put together from
// the segments' own states (a first launch).  Scores are formed transposed (rows s, columns r), so that a lane's
// weighted scores are operand values of the next product as they stand, and so are its values of the state.
//
// Rounding: S is carried in fp32, its decay as S + S (a^n - 1) where a^n is above a half, so that slow decays lose nothing over
// long sequences, and as S a^n below, where a^n - 1 lies next to -1 and its rounding would leave 2^-25 of the old S.  For
// bf16 the decayed operand of its sums is split into bf16 parts: three (24 bits) where the state is a result, two where it is
// only read, as bf16.  Scores, and S as it is read, are rounded to bf16 once as inputs of their products (in short sequences:
// split in two), whose sums are fp32.  fp32 rounds nothing else.
//
// Measured in whole calls (dk = dv = 128, bf16): B = 4, T = 4096, H = 16 forward 98 us, backward 171 us (its tensors, each
// once, take 94 us at a copy's rate, its 99 GFLOP of products 80 us at the rate of a large one; traced launches of both are
// a tenth longer); B = 1, T = 32768, H = 16 191 us, the bytes of its two launches 168 us.  The chain of steps inside a
// chunk bounds the backward: the owners' 54 products of 32 cycles wait for operands from LDS, each other and two barriers, 5600
// cycles a chunk; the matrix units are busy for 25 % of the launch, the LDS pipe for 23 %.
// fp32 (B = 3, T = 777, H = 6, dk = 64, dv = 128): forward 30 us, backward 78 us, bound by the fp32 matrix rate: the
// busiest of four SIMDs has 288 products of 32 cycles per chunk, 9200 of its 13000 cycles.
#include "gdr2_common.hpp"
#include "gdr2_hybrid_kernels.hpp"

namespace gdr2 {

constexpr int kDlaThreads = 256, C = kDlaChunk;
// Columns of an fp32 workgroup's state: 64 would leave no register for the rows ahead.  (bf16 takes all columns: with 64 to
// a workgroup, two waves for the outputs, two for the state and that read from LDS, two workgroups to a compute unit, forward
// and backward of B = 4, T = 4096, H = 16 took 112 + 198 us against 103 + 176, a prompt of 32768 207 against 195.)
constexpr int kDlaF32VS = 32;
// In sequences of up to this length bf16 keeps 16 bits of the scores and of the state as it is read (two products each): sums
// that short do not average roundings out.  Normwise error over that of the exact result rounded once, 1 to 64 tokens of a few
// heads: 1.0 against up to 1.96; from 129 tokens on it is 1.41 to 1.44 with one rounding each.  It costs 64 prompts of 128 tokens
// (H = 16, dk = dv = 128) 67 us for 60, their backward 133 for 119; fewer chains less than a microsecond.
constexpr int kDlaFine = 128;

// a^n for whole n >= 0; a^0 = 1 also where a = 0
__device__ __forceinline__ float dla_pow(float g, int n) { return n == 0 ? 1.f : expf((float)n * g); }

// The decay of a state over n >= 0 tokens: S a^n, as S + S f (f = a^n - 1) where it is slow, else as S f.
template <bool SLOW>
__device__ __forceinline__ float dla_factor(float g, int n) {
    const float x = (float)n * g;
    if constexpr (SLOW) return n == 0 ? 0.f : expm1f(x);
    else return n == 0 ? 1.f : expf(x);
}
template <bool SLOW>
__device__ __forceinline__ float dla_decayed(float s, float f) { return SLOW ? fmaf(s, f, s) : s * f; }
// Slow: a^n > 1/2.  A head keeps to one form through its chunks, that of a whole one: of shorter ones, which may be slow
// where a whole one is not, a sequence has two.
__device__ __forceinline__ bool dla_slow(float g, int n) { return __builtin_amdgcn_readfirstlane(n == 0 || (float)n * g > -0.6931472f); }

// Tiles in LDS are rows of R 16-byte pieces without padding.  Operands with the contraction along a row are read as one
// piece of sixteen rows, operands with it down the rows as 64 bytes of four rows; an exclusive or on the piece's number
// spreads either over all banks.
template <typename T, int R>
__device__ __forceinline__ int tile_at(int row, int piece) {
    if constexpr (sizeof(T) == 2) {
        const int b = ((row >> 2) ^ (row >> 3)) & 1, t = row >> 1;
        if constexpr (R == 16) return row * R + (piece ^ ((row & 3) << 2 | b << 1 | ((row >> 2) & 1)));
        else return row * R + (piece ^ ((t & 1) << 2 | b << 1 | ((t >> 1) & 1)));
    } else {
        if constexpr (R >= 16) return row * R + (piece ^ (row & 15));
        else return (row * R + piece) ^ (((row >> 2) & 1) << 3 | ((row >> 3) & 1) << 2);
    }
}

// Through a buffer descriptor: lanes outside of it load zeros and store nothing.
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i32x4 load16(__amdgpu_buffer_rsrc_t t, int offset) {
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(t, offset, 0, 0));
}
__device__ __forceinline__ void store16(__amdgpu_buffer_rsrc_t t, int offset, const i32x4& v) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), t, offset, 0, 0);
}
__device__ __forceinline__ float uniform(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, x)));
}

// The rows of one tensor, chunk by chunk.  A chunk is reached through a buffer descriptor that starts at its lowest row and
// ends behind its highest, so the rows that a last chunk lacks lie outside of it (against time below it, at offsets that
// wrap): they load as zeros and are not stored, without a branch.
struct DlaStream {
    const char* p;          // the lowest row of the next chunk, if it were whole
    long step;
    int whole, part, lack;  // bytes of a whole and of the sequence's last chunk, and those the latter lacks below
    int end, last;          // chunks from `end` on are not touched
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t next(int ch, int& shift) {
        shift = ch == last ? lack : 0;
        const int bytes = ch == last ? part : whole;
        const char* at = p + shift;
        p += step;
        return __builtin_amdgcn_make_buffer_rsrc((void*)at, 0, ch < end ? bytes : 0, 0x27000);
    }
};

// Sequence b's length; wave-uniform, for the descriptors
__device__ __forceinline__ int dla_length(const DlaParams& p, int b) {
    const int n = p.lengths ? p.lengths[b] : p.T;
    return __builtin_amdgcn_readfirstlane(n < 0 ? 0 : n > p.T ? p.T : n);
}

// A workgroup's share: VS columns of one pass of one chain, chunks c0 .. c1 - 1 of the sequence.  Row r of chunk ch is
// token 64 ch + r, or L - 1 - (64 ch + r) against time.
template <typename T, int K, int VS, bool LOCAL>
struct DlaWork {
    static constexpr int ES = (int)sizeof(T), RY = K * ES / 16, RZ = VS * ES / 16;    // pieces of a row
    const DlaParams& p;
    const DlaPass& ps;
    int V, slices, ip, sl, sg, h, b;
    int L, nch, c0, c1;
    float ga;
    bool rev;
    int early;              // against time the state before the first token is undecayed at it: one power less, once
    int sx, sz;             // bytes from row to row (H <= 32768: 64 rows fit 32 bits)

    // Slices of a chain's columns lie next to each other, then passes, segments, heads, sequences: neighbours, which read
    // the same rows, run on one XCD.
    __device__ __forceinline__ DlaWork(const DlaParams& q, int item, int pass)
        : p(q), ps(q.pass[pass]), V(ps.V), slices(V / VS), ip(pass) {
        const int segs = LOCAL ? p.segs - 1 : p.segs;
        sl = item % p.slots - ps.slot, sg = item / p.slots % segs;
        const int bh = item / p.slots / segs;
        h = bh % p.H, b = bh / p.H;
        L = dla_length(p, b);
        nch = (L + C - 1) / C, c0 = sg * p.seg_chunks;
        c1 = c0 + p.seg_chunks < nch ? c0 + p.seg_chunks : nch;
        ga = uniform(p.log_decay[h]);
        rev = ps.reverse;
        early = rev ? 1 : 0;
        sx = p.H * K * ES, sz = p.H * V * ES;
    }
    __device__ __forceinline__ int off(int r, int stride) const { return (rev ? C - 1 - r : r) * stride; }
    __device__ __forceinline__ DlaStream stream(const void* t, int stride, int bytes, int width, int col) const {
        const long low = (long)b * p.T + (rev ? (long)L - (c0 + 1) * C : (long)c0 * C);
        const int tail = L - (nch - 1) * C;  // rows of the sequence's last chunk
        return DlaStream{(const char*)t + ((low * p.H + h) * width + col) * ES, (long)(rev ? -C : C) * stride, (C - 1) * stride + bytes,
                         (tail - 1) * stride + bytes, rev ? (C - tail) * stride : 0, c1, nch - 1};
    }
    __device__ __forceinline__ DlaStream rows_of_k(const void* t) const { return stream(t, sx, K * ES, K, 0); }
    __device__ __forceinline__ DlaStream rows_of_v(const void* t) const { return stream(t, sz, VS * ES, V, sl * VS); }
    // The number (k, column v of the slice) of the chain's state in memory, whose steps along k and v are chosen once for all
    // of a lane's numbers.
    __device__ __forceinline__ int step_k() const { return ps.flip ? 1 : V; }
    __device__ __forceinline__ int step_v() const { return ps.flip ? K : 1; }
    __device__ __forceinline__ long state_at(int k, int v, int sk, int sv) const {
        return ((long)b * p.H + h) * K * V + k * sk + (sl * VS + v) * sv;
    }
    // the own state of segment j
    __device__ __forceinline__ float* local(int j) const {
        return p.local + (((((long)ip * p.B + b) * p.H + h) * (p.segs - 1) + j) * slices + sl) * (K * VS);
    }
    __device__ __forceinline__ bool final_here() const { return nch == 0 ? sg == 0 : c0 < nch && c1 == nch; }
    // The state's decay over chunk ch, where `whole` is a whole one's.  The empty statement keeps the others' behind a branch:
    // formed in every chunk and then chosen, their exponential lies in the state's way (backward of dk = 128, dv = 64 +18 %).
    template <bool SLOW>
    __device__ __forceinline__ float decay(int ch, float whole) const {
        const int n = L - ch * C < C ? L - ch * C : C, m = n - (ch == 0 ? early : 0);
        if (m == C) return whole;
        asm volatile("");
        return dla_factor<SLOW>(ga, m);
    }
    // f(form, factor) with the decay over segment j
    template <typename F>
    __device__ __forceinline__ void segment_decay(int j, F&& f) const {
        const int n = p.seg_chunks * C - (j == 0 ? early : 0);
        if (dla_slow(ga, n)) f(IC<1>{}, dla_factor<true>(ga, n));
        else f(IC<0>{}, dla_factor<false>(ga, n));
    }
    // zeros behind the sequence, in the segment's part of the time axis
    __device__ __forceinline__ void pad(int tid, int threads) const {
        const long t0 = L > (long)c0 * C ? L : (long)c0 * C, t1 = sg + 1 < p.segs ? (long)(c0 + p.seg_chunks) * C : p.T;
        char* out = (char*)ps.out + ((((long)b * p.T) * p.H + h) * V + sl * VS) * ES;
        for (long x = tid; x < (t1 - t0) * RZ; x += threads)
            *(i32x4*)(out + (t0 + x / RZ) * p.H * V * ES + x % RZ * 16) = i32x4{0, 0, 0, 0};
    }
};

// The workgroup's share of the launch goes to `body` with the length of its pass' rows: KM, or (KM = 0, dk and dv differ in
// a backward) the pass' own.
template <int KM, typename F>
__device__ __forceinline__ void dla_share(const DlaParams& p, int nwork, F&& body) {
    const int per = gridDim.x / 8, item = blockIdx.x % 8 * per + blockIdx.x / 8;
    if (item >= nwork) return;
    int ip = 0;
    while (ip + 1 < p.passes && item % p.slots >= p.pass[ip + 1].slot) ++ip;
    if constexpr (KM) body(IC<KM>{}, item, ip);
    else if (p.pass[ip].K == 128) body(IC<128>{}, item, ip);
    else body(IC<64>{}, item, ip);
}

// ------------------------------------------------------------------ bf16
// 32 x 32 products.  A workgroup takes all columns of a pass: a wave per 32 of them owns their state and outputs, and four
// waves help: they bring the tiles, a chunk ahead, and form the scores, a block of 32 x 32 each of three.  Loops of
// their own meet at two barriers per chunk: before the first the owners read the state and carry it on while the helpers
// form this chunk's scores and write the next one's rows; behind it the owners add the scores' part and store, and the helpers
// write the next decayed operand.  (For a segment's own state alone, LOCAL, one barrier.)
typedef float f32x16 __attribute__((ext_vector_type(16)));
__device__ __forceinline__ int acc_row32(int i, int l) { return 8 * (i / 4) + 4 * (l >> 5) + i % 4; }
// operand of 32 columns from piece q of a tile, contraction down sixteen rows from r0: rows 4 h .. + 3 and 8 + 4 h .. + 3
template <int R>
__device__ __forceinline__ bf16x8 columns32(const i32x4* t, int r0, int q, int l) {
    const int p = l & 15, row = r0 + 4 * (l >> 5) + (p >> 2), piece = q + 2 * ((l >> 4) & 1) + ((p & 3) >> 1);
    const bf16x4 lo = ds_read_tr4((const bf16*)(t + tile_at<bf16, R>(row, piece)) + 4 * (p & 1));
    const bf16x4 hi = ds_read_tr4((const bf16*)(t + tile_at<bf16, R>(row + 8, piece)) + 4 * (p & 1));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ void mma32x32(f32x16& c, const bf16x8& a, const bf16x8& b) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 zeros16() { return f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0}; }

constexpr int kDlaHelp = 256;  // the helpers' threads
// Two buffers belong to chunks by turns.
template <int K, int V, bool LOCAL, bool FINE>
struct DlaTiles {
    i32x4 y[2][C * K / 8];
    i32x4 x[LOCAL ? 1 : 2][LOCAL ? 1 : C * K / 8];
    i32x4 z[LOCAL ? 1 : 2][LOCAL ? 1 : C * V / 8];
    i32x4 d[LOCAL ? 2 : 1][3][C * V / 8];                // z_s a^(63 - s) in parts of 8 bits
    i32x4 pr[FINE ? 2 : 1][LOCAL ? 1 : 6 * 64];          // weighted scores, as the owners' lanes take them
};

// A helper's share of the rows of one tensor: 16 bytes at a time.
template <int R>
struct DlaRows {
    static constexpr int U = C * R / kDlaHelp;
    DlaStream s;
    int off[U];
    i32x4 r[U];
    template <typename W>
    __device__ __forceinline__ DlaRows(const W& k, const DlaStream& stream, int stride, int th) : s(stream) {
#pragma unroll
        for (int u = 0; u < U; ++u) off[u] = k.off((th + u * kDlaHelp) / R, stride) + (th + u * kDlaHelp) % R * 16;
    }
    __device__ __forceinline__ void fetch(int ch) {
        int shift;
        const auto t = s.next(ch, shift);
#pragma unroll
        for (int u = 0; u < U; ++u) r[u] = load16(t, off[u] - shift);
    }
    // pieces 2 i and 2 i + 1 as their first halves and their second ones
    __device__ __forceinline__ void put_halves(i32x4* tile, int th) const {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = (th + u * kDlaHelp) / R, piece = (th + u * kDlaHelp) % R, even = piece & ~1;
            *((u32x2*)(tile + tile_at<bf16, R>(row, even)) + (piece & 1)) = u32x2{(unsigned)r[u][0], (unsigned)r[u][1]};
            *((u32x2*)(tile + tile_at<bf16, R>(row, even + 1)) + (piece & 1)) = u32x2{(unsigned)r[u][2], (unsigned)r[u][3]};
        }
    }
    __device__ __forceinline__ void put(i32x4* tile, int th) const {
#pragma unroll
        for (int u = 0; u < U; ++u) tile[tile_at<bf16, R>((th + u * kDlaHelp) / R, (th + u * kDlaHelp) % R)] = r[u];
    }
};
// f times two values, in parts: each time the upper eight bits of what is left; after three nothing remains of 24.
__device__ __forceinline__ void split2(int two, float f, int& p0, int& p1, int& p2) {
    auto upper = [](float x) { return __builtin_bit_cast(float, __builtin_bit_cast(unsigned, x) & 0xffff0000u); };
    auto pair = [](float lo, float hi) { return (int)__builtin_amdgcn_perm(__builtin_bit_cast(unsigned, hi), __builtin_bit_cast(unsigned, lo), 0x07060302); };
    float lo = __builtin_bit_cast(float, (unsigned)two << 16) * f, hi = __builtin_bit_cast(float, (unsigned)two & 0xffff0000u) * f;
    p0 = pair(lo, hi);
    lo -= upper(lo), hi -= upper(hi);
    p1 = pair(lo, hi);
    lo -= upper(lo), hi -= upper(hi);
    p2 = pair(lo, hi);
}

template <int K, int V, bool LOCAL, bool FINE>
__device__ __forceinline__ void dla_body(const DlaParams& p, i32x4* lds, int item, int ip) {
    typedef DlaWork<bf16, K, V, LOCAL> Work;
    constexpr int KK = K / 16, KB = K / 32, VB = V / 32, RK = K / 8, RV = V / 8;
    auto& t = *(DlaTiles<K, V, LOCAL, FINE>*)lds;
    const int l = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id()), n = l & 31, hf = l >> 5;
    if (w >= kDlaHelp / 64 + VB) return;  // a launch for wider passes too
    const Work k(p, item, ip);
    if (LOCAL && k.c1 - k.c0 < p.seg_chunks) return;  // no later segment has a token: nobody reads this one's state
    const bool exact = k.ps.state && (LOCAL || k.final_here());
    auto owner = [&](auto parts, auto slow) {
        constexpr int PARTS = decltype(parts)::value, SLOW = decltype(slow)::value;
        const int cv = w - kDlaHelp / 64;
        // unknown to the compiler: it would form all instances' addresses before choosing among them, more than fit the registers
        int sk = k.step_k(), sv = k.step_v();
        asm volatile("" : "+s"(sk), "+s"(sv));
        f32x16 S[KB];  // rows 32 kb + acc_row32(i), columns 32 cv + n
        auto each_four = [&](int j, auto&& f) {  // of the own state of segment j
            f32x4* at = (f32x4*)k.local(j) + l;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int i = 0; i < 4; ++i) f(S[kb], 4 * i, at[((kb * VB + cv) * 4 + i) * 64]);
        };
        auto decay_state = [&](auto form, float e) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int i = 0; i < 16; ++i) S[kb][i] = dla_decayed<decltype(form)::value>(S[kb][i], e);
        };
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) S[kb] = zeros16();
        if constexpr (!LOCAL) {
            if (k.ps.init)
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int i = 0; i < 16; ++i) S[kb][i] = k.ps.init[k.state_at(32 * kb + acc_row32(i, l), 32 * cv + n, sk, sv)];
            for (int j = 0; j < k.sg && k.c0 < k.nch; ++j) {
                k.segment_decay(j, decay_state);
                each_four(j, [&](f32x16& s, int i0, const f32x4& x) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[i0 + i] += x[i];
                });
            }
        }
        DlaStream os = k.rows_of_v(k.ps.out);
        int oo[2];
        float before[2], before0[2];
#pragma unroll
        for (int rb = 0; rb < 2; ++rb) {
            const int r = 32 * rb + n;
            oo[rb] = k.off(r, k.sz) + (32 * cv + 8 * hf) * 2;
            before[rb] = dla_pow(k.ga, r + 1);
            before0[rb] = k.early ? dla_pow(k.ga, r) : before[rb];
        }
        const float whole = dla_factor<SLOW>(k.ga, C);
        if (k.c0 < k.c1) lds_barrier();
        for (int ch = k.c0; ch < k.c1; ++ch) {
            const int P = (ch - k.c0) & 1;
            f32x16 out[2];
            if constexpr (!LOCAL) {
                // from before the chunk: out^T = S^T x, rows v, columns r.  A lane's values of S are operand values as they
                // stand, contraction rows 4 h .. + 3 and 8 + 4 h .. + 3 of sixteen; x is read in that order.
                out[0] = out[1] = zeros16();
                bf16x8 xb[2][2];
                auto takex = [&](int kk) {
#pragma unroll
                    for (int rb = 0; rb < 2; ++rb) xb[kk % 2][rb] = __builtin_bit_cast(bf16x8, t.x[P][tile_at<bf16, RK>(32 * rb + n, 2 * kk + hf)]);
                };
                takex(0);
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    if (kk + 1 < KK) takex(kk + 1);
                    __builtin_amdgcn_sched_barrier(0);
                    bf16x8 s, rest;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float v = S[kk / 2][8 * (kk % 2) + e];
                        s[e] = (bf16)v;
                        if constexpr (FINE) rest[e] = (bf16)(v - (float)s[e]);
                    }
#pragma unroll
                    for (int rb = 0; rb < 2; ++rb) {
                        mma32x32(out[rb], s, xb[kk % 2][rb]);
                        if constexpr (FINE) mma32x32(out[rb], rest, xb[kk % 2][rb]);
                    }
                }
            }
            decay_state(IC<SLOW>{}, k.template decay<SLOW>(ch, whole));
            bf16x8 y[2][KB], d[2][PARTS];  // operands a step ahead
            auto take = [&](int kk) {
#pragma unroll
                for (int q = 0; q < PARTS; ++q) d[kk % 2][q] = columns32<RV>(t.d[LOCAL ? P : 0][q], 16 * kk, 4 * cv, l);
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) y[kk % 2][kb] = columns32<RK>(t.y[P], 16 * kk, 4 * kb, l);
            };
            take(0);
#pragma unroll
            for (int kk = 0; kk < C / 16; ++kk) {
                if (kk + 1 < C / 16) take(kk + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int q = 0; q < PARTS; ++q)
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb) mma32x32(S[kb], y[kk % 2][kb], d[kk % 2][q]);
            }
            if constexpr (!LOCAL) {
#pragma unroll
                for (int rb = 0; rb < 2; ++rb) {
                    const float f = ch == 0 ? before0[rb] : before[rb];
#pragma unroll
                    for (int i = 0; i < 16; ++i) out[rb][i] *= f;
                }
                lds_barrier();
                // out^T += z^T scores^T: rows s of the first half for both halves of r, of the second for the second
#pragma unroll
                for (int kk = 0; kk < C / 16; ++kk) {
                    const bf16x8 z = columns32<RV>(t.z[P], 16 * kk, 4 * cv, l);
#pragma unroll
                    for (int q = 0; q < (FINE ? 2 : 1); ++q) {
                        if (kk < 2) mma32x32(out[0], z, __builtin_bit_cast(bf16x8, t.pr[q][kk * 64 + l]));
                        mma32x32(out[1], z, __builtin_bit_cast(bf16x8, t.pr[q][((kk < 2 ? 4 : 2) + kk % 2) * 64 + l]));
                    }
                }
                int shift;
                const auto o = os.next(ch, shift);
#pragma unroll
                for (int rb = 0; rb < 2; ++rb)
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        // lanes n and n + 32 hold fours of columns in turn: exchanged, each has eight in a row
                        const f32x16& v = out[rb];
                        const u32x2 a = __builtin_bit_cast(u32x2, Raw4<bf16>::narrow(f32x4{v[8 * m], v[8 * m + 1], v[8 * m + 2], v[8 * m + 3]}));
                        const u32x2 b = __builtin_bit_cast(u32x2, Raw4<bf16>::narrow(f32x4{v[8 * m + 4], v[8 * m + 5], v[8 * m + 6], v[8 * m + 7]}));
                        const auto p0 = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false), p1 = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
                        store16(o, oo[rb] - shift + 32 * m, i32x4{(int)p0[0], (int)p1[0], (int)p0[1], (int)p1[1]});
                    }
            }
            if (ch + 1 < k.c1) lds_barrier();
        }
        if constexpr (LOCAL) {
            each_four(k.sg, [&](const f32x16& s, int i0, f32x4& x) { x = f32x4{s[i0], s[i0 + 1], s[i0 + 2], s[i0 + 3]}; });
        } else if (k.ps.fin && k.final_here()) {
            // against time the final state is decayed once more (dS0 = a R_0)
            const float f = k.rev && k.L > 0 ? dla_pow(k.ga, 1) : 1.f;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int i = 0; i < 16; ++i) k.ps.fin[k.state_at(32 * kb + acc_row32(i, l), 32 * cv + n, sk, sv)] = S[kb][i] * f;
        }
    };
    if (w >= kDlaHelp / 64) {
        if (dla_slow(k.ga, C)) {
            if (exact) owner(IC<3>{}, IC<1>{});
            else owner(IC<2>{}, IC<1>{});
        } else {
            if (exact) owner(IC<3>{}, IC<0>{});
            else owner(IC<2>{}, IC<0>{});
        }
    } else {
        const int th = threadIdx.x;
        DlaRows<RK> xs(k, k.rows_of_k(k.ps.x), k.sx, th), ys(k, k.rows_of_k(k.ps.y), k.sx, th);
        DlaRows<RV> zs(k, k.rows_of_v(k.ps.z), k.sz, th);
        constexpr int ZU = DlaRows<RV>::U;
        float late[ZU];  // a^(63 - s) of the own rows of z
#pragma unroll
        for (int u = 0; u < ZU; ++u) late[u] = dla_pow(k.ga, C - 1 - (th + u * kDlaHelp) / RV);
        auto put_rows = [&](int P) {
            ys.put(t.y[P], th);
            if constexpr (!LOCAL) {
                xs.put_halves(t.x[P], th);
                zs.put(t.z[P], th);
            }
        };
        auto fetch_rows = [&](int ch) {  // all but z, which the decayed operand is still formed from
            if constexpr (!LOCAL) xs.fetch(ch);
            ys.fetch(ch);
        };
        i32x4 part0[ZU], part1[ZU], part2[ZU];
        auto split_late = [&](int ch) {
            const int m = k.L - ch * C;
            float f[ZU];
#pragma unroll
            for (int u = 0; u < ZU; ++u) f[u] = late[u];
            if (m < C) {
#pragma unroll
                for (int u = 0; u < ZU; ++u) {
                    const int r = (th + u * kDlaHelp) / RV;
                    f[u] = r < m ? dla_pow(k.ga, m - 1 - r) : 0.f;
                }
            }
#pragma unroll
            for (int u = 0; u < ZU; ++u) {
                int a[4], b[4], c[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) split2(zs.r[u][i], f[u], a[i], b[i], c[i]);
                part0[u] = i32x4{a[0], a[1], a[2], a[3]};
                part1[u] = i32x4{b[0], b[1], b[2], b[3]};
                part2[u] = i32x4{c[0], c[1], c[2], c[3]};
            }
        };
        auto put_late = [&](int P) {
#pragma unroll
            for (int u = 0; u < ZU; ++u) {
                const int at = tile_at<bf16, RV>((th + u * kDlaHelp) / RV, (th + u * kDlaHelp) % RV);
                t.d[P][0][at] = part0[u];
                t.d[P][1][at] = part1[u];
                if (exact) t.d[P][2][at] = part2[u];
            }
        };
        // Scores: waves 0 and 1 the blocks on the diagonal (rows r and s from 32 w), wave 2 the one before the second.  The lane's
        // values 4 j .. 4 j + 3 of a block are rows s = s_j .. s_j + 3 of column r, so a^(r - s) is a^(r - s_j - 3) times a^3, a^2,
        // a, 1; both are powers with an exponent >= 0 but where the diagonal passes through the four, which have weights of
        // their own.
        const int first = n - 4 * hf;     // r - s_0 on the diagonal
        const int xb = w == 0 ? 0 : 32, yb = w == 1 ? 32 : 0;
        float near[4], diag[4];
        const float a1 = uniform(dla_pow(k.ga, 1)), a2 = uniform(dla_pow(k.ga, 2)), a3 = uniform(dla_pow(k.ga, 3));
        const float fall[4] = {a3, a2, a1, 1.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int least = first + (w == 2 ? 32 : 0) - 8 * j - 3;
            near[j] = least < 0 ? 0.f : dla_pow(k.ga, least);
            const int lag = (n & 7) - 4 * hf - j;
            diag[j] = lag < 0 ? 0.f : dla_pow(k.ga, lag);
        }
        const int on = w == 2 || first < 0 || first % 8 > 2 ? -1 : first / 8;  // the four that the diagonal leaves in part
        auto scores = [&](int P) {
            f32x16 sc = zeros16();
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                const bf16x4 lo = *((const bf16x4*)(t.y[P] + tile_at<bf16, RK>(yb + n, 2 * kk)) + hf);
                const bf16x4 hi = *((const bf16x4*)(t.y[P] + tile_at<bf16, RK>(yb + n, 2 * kk + 1)) + hf);
                mma32x32(sc, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7),
                         __builtin_bit_cast(bf16x8, t.x[P][tile_at<bf16, RK>(xb + n, 2 * kk + hf)]));
            }
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                bf16x8 pr, rest;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int j = 2 * kk + e / 4, i = e % 4;
                    const float v = sc[8 * kk + e] * (j == on ? diag[i] : near[j] * fall[i]);
                    pr[e] = (bf16)v;
                    if constexpr (FINE) rest[e] = (bf16)(v - (float)pr[e]);
                }
                t.pr[0][(2 * w + kk) * 64 + l] = __builtin_bit_cast(i32x4, pr);
                if constexpr (FINE) t.pr[1][(2 * w + kk) * 64 + l] = __builtin_bit_cast(i32x4, rest);
            }
        };
        if (k.c0 < k.c1) {
            fetch_rows(k.c0);
            zs.fetch(k.c0);
            put_rows(0);
            fetch_rows(k.c0 + 1);
            split_late(k.c0);
            zs.fetch(k.c0 + 1);
            put_late(0);
            lds_barrier();
        }
        for (int ch = k.c0; ch < k.c1; ++ch) {
            const int P = (ch - k.c0) & 1;
            if constexpr (LOCAL) {
                if (ch + 1 < k.c1) {
                    put_rows(1 - P);
                    fetch_rows(ch + 2);
                    split_late(ch + 1);
                    zs.fetch(ch + 2);
                    put_late(1 - P);
                    lds_barrier();
                }
            } else {
                if (w < 3) scores(P);
                if (ch + 1 < k.c1) {
                    put_rows(1 - P);
                    fetch_rows(ch + 2);
                    split_late(ch + 1);
                    zs.fetch(ch + 2);
                }
                lds_barrier();
                if (ch + 1 < k.c1) {
                    put_late(0);
                    lds_barrier();
                }
            }
        }
        if constexpr (!LOCAL) k.pad(th, kDlaHelp);
    }
}
// K = 0: a backward whose dk and dv differ, passes of either kind.
template <int K, int V, bool LOCAL, bool FINE>
__global__ __launch_bounds__(512, 2) void gdr2_dla_kernel(DlaParams p, int nwork) {
    constexpr size_t A = sizeof(DlaTiles<K ? K : 128, K ? V : 64, LOCAL, FINE>), B = sizeof(DlaTiles<K ? K : 64, K ? V : 128, LOCAL, FINE>);
    __shared__ i32x4 lds[(A > B ? A : B) / 16];
    dla_share<K>(p, nwork, [&](auto k, int item, int ip) {
        constexpr int KP = decltype(k)::value;
        dla_body<KP, K ? V : 192 - KP, LOCAL, FINE>(p, lds, item, ip);
    });
}

// A padded batch of more: each sequence's variant by its own length, so that its result does not depend on its company.  The
// second variant's registers and LDS cost the others 0 to 4 % (B = 4, T = 4096, H = 16, dk = dv = 128, lengths from 4096 to 2048:
// forward 90 -> 91 us, backward 167 -> 170).
template <int K, int V>
__global__ __launch_bounds__(512, 2) void gdr2_dla_ragged_kernel(DlaParams p, int nwork) {
    constexpr size_t A = sizeof(DlaTiles<K ? K : 128, K ? V : 64, false, true>), B = sizeof(DlaTiles<K ? K : 64, K ? V : 128, false, true>);
    __shared__ i32x4 lds[(A > B ? A : B) / 16];
    dla_share<K>(p, nwork, [&](auto k, int item, int ip) {
        constexpr int KP = decltype(k)::value, VP = K ? V : 192 - KP;
        if (dla_length(p, item / p.slots / p.segs / p.H) <= kDlaFine) dla_body<KP, VP, false, true>(p, lds, item, ip);
        else dla_body<KP, VP, false, false>(p, lds, item, ip);
    });
}

// ------------------------------------------------------------------ fp32
// 16 x 16 products, of which this type's scores need eight times as many cycles: waves 0..3 read sixteen rows each,
// waves 4..7 carry every fourth sixteen of the state's rows.
// Staging of y and z, z also as the decayed operand z_s a^(63 - s) of the state's sums.  Set (ch - c0) % 2 of the registers
// and of the tiles belongs to chunk ch.  Behind the last chunk nothing is loaded.
template <int K, bool LOCAL>
struct DlaF32Stage {
    typedef DlaWork<float, K, kDlaF32VS, LOCAL> Work;
    static constexpr int NT = LOCAL ? 256 : 512, RY = Work::RY, RZ = Work::RZ, YU = C * RY / NT, ZU = C * RZ / NT;
    struct Tiles {
        i32x4 y[2][C * RY];
        i32x4 z[LOCAL ? 1 : 2][LOCAL ? 1 : C * RZ];
        i32x4 d[2][C * RZ];
        i32x4 s[LOCAL ? 1 : 2][LOCAL ? 1 : kDlaF32VS * RY];  // the state as the chunk reads it, [v][k]
    };
    const Work& k;
    Tiles& t;
    DlaStream ys, zs;
    i32x4 yr[2][YU], zr[2][ZU];
    int th, yo[YU], zo[ZU];
    float late[ZU];  // a^(63 - s) of the staged rows
    __device__ __forceinline__ DlaF32Stage(const Work& work, Tiles& tiles, int thread)
        : k(work), t(tiles), ys(work.rows_of_k(work.ps.y)), zs(work.rows_of_v(work.ps.z)), th(thread) {
#pragma unroll
        for (int u = 0; u < YU; ++u) yo[u] = k.off((th + u * NT) / RY, k.sx) + (th + u * NT) % RY * 16;
#pragma unroll
        for (int u = 0; u < ZU; ++u) {
            zo[u] = k.off((th + u * NT) / RZ, k.sz) + (th + u * NT) % RZ * 16;
            late[u] = dla_pow(k.ga, C - 1 - (th + u * NT) / RZ);
        }
    }
    template <int P>
    __device__ __forceinline__ void fetch(int ch) {
        int shift;
        const auto y = ys.next(ch, shift);
#pragma unroll
        for (int u = 0; u < YU; ++u) yr[P][u] = load16(y, yo[u] - shift);
        const auto z = zs.next(ch, shift);
#pragma unroll
        for (int u = 0; u < ZU; ++u) zr[P][u] = load16(z, zo[u] - shift);
    }
    template <int P>
    __device__ __forceinline__ void put(int ch) {
        const int n = k.L - ch * C;
#pragma unroll
        for (int u = 0; u < YU; ++u) t.y[P][tile_at<float, RY>((th + u * NT) / RY, (th + u * NT) % RY)] = yr[P][u];
#pragma unroll
        for (int u = 0; u < ZU; ++u) {
            const int r = (th + u * NT) / RZ, at = tile_at<float, RZ>(r, (th + u * NT) % RZ);
            if constexpr (!LOCAL) t.z[P][at] = zr[P][u];
            const float f = n >= C ? late[u] : r < n ? dla_pow(k.ga, n - 1 - r) : 0.f;
            *(f32x4*)(t.d[P] + at) = __builtin_bit_cast(f32x4, zr[P][u]) * f;
        }
    }
};
template <int K, bool LOCAL>
__device__ __forceinline__ void dla_f32_body(const DlaParams& p, i32x4* lds, int item, int ip) {
    typedef DlaWork<float, K, kDlaF32VS, LOCAL> Work;
    typedef DlaF32Stage<K, LOCAL> Stage;
    constexpr int KP = K / 16, KB = K / 64, VB = kDlaF32VS / 16, RY = Work::RY, RZ = Work::RZ;
    auto& t = *(typename Stage::Tiles*)lds;
    const Work k(p, item, ip);
    if (LOCAL && k.c1 - k.c0 < p.seg_chunks) return;
    const int l = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id()), c = l & 15, g = l >> 4;
    // operand value of column 16 block + l % 16, contraction down the rows
    auto column = [&](const i32x4* tile, auto pieces, int row, int block) {
        constexpr int R = decltype(pieces)::value;
        return ((const float*)(tile + tile_at<float, R>(row, 4 * block + (c >> 2))))[c & 3];
    };
    Stage st(k, t, threadIdx.x);
    if (k.c0 < k.c1) {
        st.template fetch<0>(k.c0);
        st.template fetch<1>(k.c0 + 1);
    }
    if (LOCAL || w >= 4) {
        // blocks of 16 x 16: rows 16 (cw + 4 kb) + 4 g + i, column 16 vb + c
        const int cw = LOCAL ? w : w - 4;
        const int sk = k.step_k(), sv = k.step_v();
        f32x4 S[KB][VB];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int vb = 0; vb < VB; ++vb) S[kb][vb] = f32x4{0, 0, 0, 0};
        auto each = [&](auto&& f) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int vb = 0; vb < VB; ++vb) f(S[kb][vb], 16 * (cw + 4 * kb) + 4 * g, 16 * vb + c, (kb * VB + vb) * 256 + cw * 64 + l);
        };
        auto decay_state = [&](auto form, float e) {
            each([&](f32x4& s, int, int, int) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[i] = dla_decayed<decltype(form)::value>(s[i], e);
            });
        };
        if constexpr (!LOCAL) {
            if (k.ps.init)
                each([&](f32x4& s, int row, int v, int) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[i] = k.ps.init[k.state_at(row + i, v, sk, sv)];
                });
            for (int j = 0; j < k.sg && k.c0 < k.nch; ++j) {
                k.segment_decay(j, decay_state);
                const f32x4* own = (const f32x4*)k.local(j);
                each([&](f32x4& s, int, int, int at) { s += own[at]; });
            }
        }
        auto put_state = [&](auto set) {
            constexpr int P = decltype(set)::value;
            if constexpr (!LOCAL) each([&](const f32x4& s, int row, int v, int) { *(f32x4*)(t.s[P] + tile_at<float, RY>(v, row / 4)) = s; });
        };
        if (k.c0 < k.c1) {
            put_state(IC<0>{});
            st.template put<0>(k.c0);
            st.template fetch<0>(k.c0 + 2);
        }
        auto chunk = [&](int ch, auto set, auto slow, float whole) {
            constexpr int P = decltype(set)::value;
            lds_barrier();
            decay_state(slow, k.template decay<decltype(slow)::value>(ch, whole));
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int r = 16 * (j / 4) + 4 * g + j % 4;
                float y[KB];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) y[kb] = column(t.y[P], IC<RY>{}, r, cw + 4 * kb);
#pragma unroll
                for (int vb = 0; vb < VB; ++vb) {
                    const float z = column(t.d[P], IC<RZ>{}, r, vb);
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb) mma32(S[kb][vb], y[kb], z);
                }
            }
            if (ch + 1 < k.c1) {
                put_state(IC<1 - P>{});
                st.template put<1 - P>(ch + 1);
            }
            st.template fetch<1 - P>(ch + 3);
        };
        auto chunks = [&](auto slow) {
            const float whole = dla_factor<decltype(slow)::value>(k.ga, C);
            for (int ch = k.c0; ch < k.c1; ch += 2) {
                chunk(ch, IC<0>{}, slow, whole);
                if (ch + 1 < k.c1) chunk(ch + 1, IC<1>{}, slow, whole);
            }
        };
        if (dla_slow(k.ga, C)) chunks(IC<1>{});
        else chunks(IC<0>{});
        if constexpr (LOCAL) {
            f32x4* own = (f32x4*)k.local(k.sg);
            each([&](const f32x4& s, int, int, int at) { own[at] = s; });
        } else if (k.ps.fin && k.final_here()) {
            const float f = k.rev && k.L > 0 ? dla_pow(k.ga, 1) : 1.f;
            each([&](const f32x4& s, int row, int v, int) {
#pragma unroll
                for (int i = 0; i < 4; ++i) k.ps.fin[k.state_at(row + i, v, sk, sv)] = s[i] * f;
            });
        }
    } else if constexpr (!LOCAL) {
        DlaStream xs = k.rows_of_k(k.ps.x), os = k.rows_of_v(k.ps.out);
        const int xrow = 16 * w + c, xo = k.off(xrow, k.sx) + g * 16, oo = k.off(xrow, k.sz) + g * 16;
        i32x4 xr[2][KP];
        auto fetch_x = [&](int ch, auto set) {
            constexpr int P = decltype(set)::value;
            int shift;
            const auto x = xs.next(ch, shift);
#pragma unroll
            for (int kk = 0; kk < KP; ++kk) xr[P][kk] = load16(x, xo - shift + kk * 64);
        };
        // products of 16 x 16 by sixteen values of contraction
        auto mma = [&](f32x4& acc, const i32x4& a, const i32x4& b) {
            const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
            for (int e = 0; e < 4; ++e) mma32(acc, x[e], y[e]);
        };
        // weights that every chunk shares: near[b][i] = a^(r - s) of score block b, before = a^(r + 1)
        float near[4][4];
#pragma unroll
        for (int sb = 0; sb < 4; ++sb)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int lag = xrow - (16 * sb + 4 * g + i);
                near[sb][i] = lag < 0 ? 0.f : dla_pow(k.ga, lag);
            }
        const float before = dla_pow(k.ga, xrow + 1), before0 = k.early ? dla_pow(k.ga, xrow) : before;
        if (k.c0 < k.c1) {
            fetch_x(k.c0, IC<0>{});
            fetch_x(k.c0 + 1, IC<1>{});
            st.template put<0>(k.c0);
            st.template fetch<0>(k.c0 + 2);
        }
        auto chunk = [&](int ch, auto set) {
            constexpr int P = decltype(set)::value;
            lds_barrier();
            f32x4 out[VB], sc[4];
#pragma unroll
            for (int vb = 0; vb < VB; ++vb) out[vb] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int kk = 0; kk < KP; ++kk)
#pragma unroll
                for (int vb = 0; vb < VB; ++vb) mma(out[vb], t.s[P][tile_at<float, RY>(16 * vb + c, 4 * kk + g)], xr[P][kk]);
            const float f = ch == 0 ? before0 : before;
#pragma unroll
            for (int vb = 0; vb < VB; ++vb) out[vb] *= f;
            // blocks of scores behind the wave's rows are not seen
#pragma unroll
            for (int sb = 0; sb < 4; ++sb) {
                if (sb <= w) {
                    sc[sb] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int kk = 0; kk < KP; ++kk) mma(sc[sb], t.y[P][tile_at<float, RY>(16 * sb + c, 4 * kk + g)], xr[P][kk]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float s = sc[sb][i] * near[sb][i];
#pragma unroll
                        for (int vb = 0; vb < VB; ++vb) mma32(out[vb], column(t.z[P], IC<RZ>{}, 16 * sb + 4 * g + i, vb), s);
                    }
                }
            }
            fetch_x(ch + 2, set);
            int shift;
            const auto o = os.next(ch, shift);
#pragma unroll
            for (int vb = 0; vb < VB; ++vb) store16(o, oo - shift + 64 * vb, __builtin_bit_cast(i32x4, out[vb]));
            if (ch + 1 < k.c1) st.template put<1 - P>(ch + 1);
            st.template fetch<1 - P>(ch + 3);
        };
        for (int ch = k.c0; ch < k.c1; ch += 2) {
            chunk(ch, IC<0>{});
            if (ch + 1 < k.c1) chunk(ch + 1, IC<1>{});
        }
        k.pad(threadIdx.x, 256);
    }
}
template <int KM, bool LOCAL>
__global__ __launch_bounds__(LOCAL ? 256 : 512, LOCAL ? 1 : 2) void gdr2_dla_f32_kernel(DlaParams p, int nwork) {
    __shared__ i32x4 lds[sizeof(typename DlaF32Stage<KM ? KM : 128, LOCAL>::Tiles) / 16];
    dla_share<KM>(p, nwork, [&](auto k, int item, int ip) { dla_f32_body<decltype(k)::value, LOCAL>(p, lds, item, ip); });
}

// Segments of the sequence: as many as fill the device once (a workgroup to a compute unit), none below two chunks (fp32:
// four).  Measured for 192 / 256 / 512 / 768 workgroups of bf16: B = 4, T = 4096, H = 16 forward 114 / 103 / 123 / 134 us,
// backward 174 / 176 / 218 / 239 (192 workgroups in one segment; then two and four), B = 1, T = 32768, H = 16 214 / 195 / 247 /
// 263.  At least two, four or eight chunks: B = 1, T = 1000, H = 8 backward 24 / 27 / 39 us.  fp32, B = 3, T = 777, H = 6: at
// least four chunks 29 us against 42 with at least sixteen (one segment) and 36 with two; 512 instead of 256 workgroups made
// its backward 84 us from 76.
DlaCut dla_cut(long B, long T, long H, long slots, bool f32) {
    const long nch = (T + C - 1) / C, jobs = B * H * slots, least = f32 ? 4 : 2;
    long segs = jobs > 0 ? 256 / jobs : 1;
    segs = segs < nch / least ? segs : nch / least;
    segs = segs < 1 ? 1 : segs;
    DlaCut c{};
    c.seg_chunks = (int)((nch + segs - 1) / segs);
    c.seg_chunks = c.seg_chunks < 1 ? 1 : c.seg_chunks;
    c.segs = (int)((nch + c.seg_chunks - 1) / c.seg_chunks);
    c.segs = c.segs < 1 ? 1 : c.segs;
    return c;
}

template <int K, int V, bool LOCAL>
static hipError_t launch_dla(bool bf, long n, const DlaParams& p, hipStream_t s) {
    const dim3 grid((unsigned)((n + 7) / 8 * 8)), block(kDlaHelp + 64 * (K ? V : 128) / 32);
    if (bf && !LOCAL && p.T <= kDlaFine) hipLaunchKernelGGL((gdr2_dla_kernel<K, V, false, true>), grid, block, 0, s, p, (int)n);
    else if (bf && !LOCAL && p.lengths) hipLaunchKernelGGL((gdr2_dla_ragged_kernel<K, V>), grid, block, 0, s, p, (int)n);
    else if (bf) hipLaunchKernelGGL((gdr2_dla_kernel<K, V, LOCAL, false>), grid, block, 0, s, p, (int)n);
    else hipLaunchKernelGGL((gdr2_dla_f32_kernel<K, LOCAL>), grid, dim3(LOCAL ? 256 : 512), 0, s, p, (int)n);
    return hipGetLastError();
}
template <bool LOCAL>
static hipError_t launch_dla_k(bool bf, long n, const DlaParams& p, hipStream_t s) {
    const int K = p.pass[0].K, V = p.pass[0].V;
    for (int i = 1; i < p.passes; ++i)
        if (p.pass[i].K != K) return launch_dla<0, 0, LOCAL>(bf, n, p, s);
    if (K == 128) return V == 128 ? launch_dla<128, 128, LOCAL>(bf, n, p, s) : launch_dla<128, 64, LOCAL>(bf, n, p, s);
    return V == 128 ? launch_dla<64, 128, LOCAL>(bf, n, p, s) : launch_dla<64, 64, LOCAL>(bf, n, p, s);
}

int dla_slots(int V, bool f32) { return f32 ? V / kDlaF32VS : 1; }

hipError_t dla_dispatch(int bf, const DlaParams& p, hipStream_t s) {
    const long per = (long)p.B * p.H * p.slots;  // workgroups of a segment
    if (p.segs > 1) {
        const hipError_t e = launch_dla_k<true>(bf, per * (p.segs - 1), p, s);
        if (e != hipSuccess) return e;
    }
    return launch_dla_k<false>(bf, per * p.segs, p, s);
}

// One token: S <- a S + k v^T, o = S^T q.  A pure stream over the fp32 state, in registers, 16-byte accesses.  Slow decays are
// added as S (a - 1): a itself, rounded, would be off to the same side at every token, by up to 2^-25 of S (10000 tokens at
// log_decay -1e-4: 2500 half steps of the state, against 25).
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
    const float ga = p.log_decay[n % p.H];
    const bool slow = dla_slow(ga, 1);
    const float f = slow ? dla_factor<true>(ga, 1) : dla_factor<false>(ga, 1);
    const f32x4 vv = load4(v + 4 * jg);
    f32x4 o = {0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < R; ++u) {
        const int i = ig * R + u;
        const float ki = to_f(k[i]), qi = to_f(q[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float x = fmaf(f, s[u][j], ki * vv[j]);
            s[u][j] = slow ? s[u][j] + x : x;
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

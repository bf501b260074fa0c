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
// A workgroup carries some columns of one chain's state in fp32 registers (columns are independent), over the
// whole sequence or, where there are few chains, over one segment of it, whose entering state is put together from
// the segments' own states (a first launch).  Scores are formed transposed (rows s, columns r), so that a lane's
// weighted scores are operand values of the next product as they stand; the state is read from a copy in LDS (bf16: rounded)
// that each chunk writes for the next one.
//
// Rounding: S is carried in fp32, its decay as S + S (a^n - 1), so that slow decays lose nothing over long
// sequences.  For bf16 the decayed operand of its sums is split into bf16 parts: three (24 bits) where the state is a
// result, two where it is only read, as bf16 (the third costs 3 % of a backward).  Scores, and S as it is read, are
// rounded to bf16 once as inputs of their products (in short sequences: split in two), whose sums are fp32.  fp32 rounds
// nothing else.
//
// Measured (dk = dv = 128, bf16): B = 4, T = 4096, H = 16 forward 114 us (1.2 TB/s of its rows), backward 200 us (its
// tensors, each once, would take 84 us; products 31 us); B = 1, T = 32768, H = 16 with its states 210 us.  The chain of steps
// inside a chunk bounds it: scores wait for rows, products for scores, the next tiles for the products; a chunk takes 2.3 us
// alone on a compute unit, two at once 3.5 us, with the matrix units a quarter busy, LDS a third, the caches' port a
// third.  fp32 (B = 3, T = 777, H = 6, dk = 64, dv = 128): forward 29 us, backward 76 us, bound by the fp32 matrix rate: the
// busiest of four SIMDs has 288 products of 32 cycles per chunk, 9200 of its 13000 cycles.
#include "gdr2_common.hpp"
#include "gdr2_hybrid_kernels.hpp"

namespace gdr2 {

constexpr int kDlaThreads = 256, C = kDlaChunk;
// Columns of a workgroup's state.  bf16: scores are formed again for every 64, and 64 is what registers hold with two
// workgroups to a compute unit; with 32, forward and backward of B = 4, T = 4096, H = 16 took 361 us against 331, a prompt of
// 32768 289 against 222.  fp32: 64 would leave no register for the rows ahead.
constexpr int kDlaVS = 64, kDlaF32VS = 32;
// Up to this length bf16 keeps 16 bits of the scores and of the state as it is read (two products each): sums that short do
// not average roundings out.  Normwise error over that of the exact result rounded once, 1 to 64 tokens of a few
// heads: 1.0 against up to 1.96; from 129 tokens on it is 1.41 to 1.44 with one rounding each.  It costs 64 prompts of 128 tokens
// (H = 16, dk = dv = 128) 66 us for 59, their backward 144 for 123; fewer chains less than a microsecond.
constexpr int kDlaFine = 128;

// a^n for whole n >= 0; a^0 = 1 also where a = 0
__device__ __forceinline__ float dla_pow(float g, int n) { return n == 0 ? 1.f : expf((float)n * g); }

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
template <typename T>
__device__ __forceinline__ typename Raw4<T>::t load4(__amdgpu_buffer_rsrc_t t, int offset) {
    if constexpr (sizeof(T) == 2) return __builtin_bit_cast(bf16x4, __builtin_amdgcn_raw_buffer_load_b64(t, offset, 0, 0));
    else return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(t, offset, 0, 0));
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

// A workgroup's share: VS columns of one pass of one chain, chunks c0 .. c1 - 1 of the sequence.  Row r of chunk ch is
// token 64 ch + r, or L - 1 - (64 ch + r) against time.
template <typename T, int K, int VS, bool LOCAL>
struct DlaWork {
    static constexpr int ES = (int)sizeof(T), E16 = 16 / ES;     // elements of a 16-byte piece
    static constexpr int RY = K * ES / 16, RZ = VS * ES / 16;    // pieces of a row
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
        const int n = p.lengths ? p.lengths[b] : p.T;
        L = __builtin_amdgcn_readfirstlane(n < 0 ? 0 : n > p.T ? p.T : n);  // wave-uniform, for the descriptors
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
    // the number (k, column v of the slice) of the chain's state in memory
    __device__ __forceinline__ long state_at(int k, int v) const {
        return ((long)b * p.H + h) * K * V + (ps.flip ? (long)(sl * VS + v) * K + k : (long)k * V + sl * VS + v);
    }
    // the own state of segment j
    __device__ __forceinline__ float* local(int j) const {
        return p.local + (((((long)ip * p.B + b) * p.H + h) * (p.segs - 1) + j) * slices + sl) * (K * VS);
    }
    __device__ __forceinline__ bool final_here() const { return nch == 0 ? sg == 0 : c0 < nch && c1 == nch; }
    // the state's decay over chunk ch less one: S <- S + S (a^n - 1)
    __device__ __forceinline__ float decay(int ch, float whole) const {
        const int n = L - ch * C < C ? L - ch * C : C, m = n - (ch == 0 ? early : 0);
        return m == C ? whole : m == 0 ? 0.f : expm1f((float)m * ga);
    }
    // zeros behind the sequence, in the segment's part of the time axis
    __device__ __forceinline__ void pad(int tid, int threads) const {
        const long t0 = L > (long)c0 * C ? L : (long)c0 * C, t1 = sg + 1 < p.segs ? (long)(c0 + p.seg_chunks) * C : p.T;
        char* out = (char*)ps.out + ((((long)b * p.T) * p.H + h) * V + sl * VS) * ES;
        for (long x = tid; x < (t1 - t0) * RZ; x += threads)
            *(i32x4*)(out + (t0 + x / RZ) * p.H * V * ES + x % RZ * 16) = i32x4{0, 0, 0, 0};
    }
};

// Staging of y (16 bytes at a time, by NY threads) and z (four columns at a time, by NZ), z also as the decayed operand
// z_s a^(63 - s) of the state's sums: for bf16 in parts of 8 bits each, three where the state is a result, two where it is only
// read as bf16.  With two buffers (NB) set (ch - c0) % 2 of the registers and of the tiles belongs to chunk ch.  Behind
// the last chunk nothing is loaded.
template <typename T, int K, int VS, bool LOCAL, int NY, int NZ, int NB>
struct DlaStage {
    typedef DlaWork<T, K, VS, LOCAL> Work;
    typedef typename Raw4<T>::t z4;
    static constexpr int ES = Work::ES, E16 = Work::E16, RY = Work::RY, RZ = Work::RZ;
    static constexpr int YU = C * RY / NY, ZU = C * VS / 4 / NZ, NP = ES == 2 ? 3 : 1;
    static constexpr int RS = ES == 2 ? RY + 1 : RY;  // pieces of a row of the state (bf16: read along rows only, padded by one)
    static_assert(YU >= 1 && ZU >= 1, "staging");
    struct Tiles {
        i32x4 y[NB][C * RY];
        i32x4 z[LOCAL ? 1 : NB][LOCAL ? 1 : C * RZ];
        i32x4 d[NB][NP][C * RZ];
        i32x4 s[LOCAL ? 1 : NB][LOCAL ? 1 : VS * RS];  // the state as the chunk reads it, [v][k]
    };
    const Work& k;
    Tiles& t;
    DlaStream ys, zs;
    i32x4 yr[NB][YU];
    z4 zr[NB][ZU];
    int yt, zt, yo[YU], zo[ZU];
    float late[ZU];  // a^(63 - s) of the staged rows
    bool exact;      // the third part too
    __device__ __forceinline__ DlaStage(const Work& work, Tiles& tiles, int ythread, int zthread)
        : k(work), t(tiles), ys(work.rows_of_k(work.ps.y)), zs(work.rows_of_v(work.ps.z)), yt(ythread), zt(zthread), exact(work.ps.state && (LOCAL || work.final_here())) {
#pragma unroll
        for (int u = 0; u < YU; ++u) yo[u] = k.off((yt + u * NY) / RY, k.sx) + (yt + u * NY) % RY * 16;
#pragma unroll
        for (int u = 0; u < ZU; ++u) {
            const int x = zt + u * NZ, r = x / (VS / 4);
            zo[u] = k.off(r, k.sz) + x % (VS / 4) * 4 * ES;
            late[u] = dla_pow(k.ga, C - 1 - r);
        }
    }
    template <int P>
    __device__ __forceinline__ void fetch_y(int ch) {
        int shift;
        const auto y = ys.next(ch, shift);
#pragma unroll
        for (int u = 0; u < YU; ++u) yr[P][u] = load16(y, yo[u] - shift);
    }
    template <int P>
    __device__ __forceinline__ void fetch_z(int ch) {
        int shift;
        const auto z = zs.next(ch, shift);
#pragma unroll
        for (int u = 0; u < ZU; ++u) zr[P][u] = load4<T>(z, zo[u] - shift);
    }
    template <int P>
    __device__ __forceinline__ void put_y() {
#pragma unroll
        for (int u = 0; u < YU; ++u) t.y[P][tile_at<T, RY>((yt + u * NY) / RY, (yt + u * NY) % RY)] = yr[P][u];
    }
    template <int P>
    __device__ __forceinline__ void put_z(int ch) {
        const int n = k.L - ch * C;
        float f[ZU];
#pragma unroll
        for (int u = 0; u < ZU; ++u) f[u] = late[u];
        if (n < C) {
#pragma unroll
            for (int u = 0; u < ZU; ++u) {
                const int r = (zt + u * NZ) / (VS / 4);
                f[u] = r < n ? dla_pow(k.ga, n - 1 - r) : 0.f;
            }
        }
        if constexpr (ES == 2) {
            if (exact) split_z<P, 3>(f);
            else split_z<P, 2>(f);
        } else {
            split_z<P, 1>(f);
        }
    }
    // z as it is, and z f in NP parts
    template <int P, int PARTS>
    __device__ __forceinline__ void split_z(const float (&f)[ZU]) {
#pragma unroll
        for (int u = 0; u < ZU; ++u) {
            const int x = zt + u * NZ, r = x / (VS / 4), col = x % (VS / 4) * 4;
            const int at = tile_at<T, RZ>(r, col / E16), in = col % E16;
            if constexpr (!LOCAL) *(z4*)((T*)(t.z[P] + at) + in) = zr[P][u];
            f32x4 rest = Raw4<T>::widen(zr[P][u]) * f[u];
            if constexpr (ES == 2) {
                // each time the upper eight bits of what is left: after three nothing remains of 24
#pragma unroll
                for (int q = 0; q < PARTS; ++q) {
                    u32x2 part;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float even = rest[2 * i], odd = rest[2 * i + 1];
                        const unsigned lo = __builtin_bit_cast(unsigned, even), hi = __builtin_bit_cast(unsigned, odd);
                        part[i] = __builtin_amdgcn_perm(hi, lo, 0x07060302);
                        rest[2 * i] = even - __builtin_bit_cast(float, lo & 0xffff0000u);
                        rest[2 * i + 1] = odd - __builtin_bit_cast(float, hi & 0xffff0000u);
                    }
                    *(u32x2*)((T*)(t.d[P][q] + at) + in) = part;
                }
            } else {
                *(f32x4*)(t.d[P][0] + at) = rest;
            }
        }
    }
    template <int P>
    __device__ __forceinline__ void fetch(int ch) {
        fetch_y<P>(ch);
        fetch_z<P>(ch);
    }
    template <int P>
    __device__ __forceinline__ void put(int ch) {
        put_y<P>();
        put_z<P>(ch);
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
// 32 x 32 products over 64 columns.  Two waves read: outputs of 32 rows each.  Two carry the state: every other 32 of its
// rows.  They run loops of their own that meet at two barriers per chunk, before and behind the products; between the second
// and the next first the next chunk's tiles are written.  (For a segment's own state alone, LOCAL, all four carry.)
__device__ __forceinline__ int acc_row32(int i, int l) { return 8 * (i / 4) + 4 * (l >> 5) + i % 4; }
// operand of 32 columns from piece q of a tile, contraction down sixteen rows from r0: rows 4 h .. + 3 and 8 + 4 h .. + 3
template <int R>
__device__ __forceinline__ bf16x8 columns32(const i32x4* t, int r0, int q, int l) {
    const int p = l & 15, row = r0 + 4 * (l >> 5) + (p >> 2), piece = q + 2 * ((l >> 4) & 1) + ((p & 3) >> 1);
    const bf16x4 lo = ds_read_tr4((const bf16*)(t + tile_at<bf16, R>(row, piece)) + 4 * (p & 1));
    const bf16x4 hi = ds_read_tr4((const bf16*)(t + tile_at<bf16, R>(row + 8, piece)) + 4 * (p & 1));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
typedef float f32x16 __attribute__((ext_vector_type(16)));
__device__ __forceinline__ void mma32x32(f32x16& c, const bf16x8& a, const bf16x8& b) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 zeros16() { return f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0}; }

template <int K, bool LOCAL>
struct DlaLds {
    typedef DlaStage<bf16, K, kDlaVS, LOCAL, LOCAL ? 256 : 128, 256, 1> Stage;
    typename Stage::Tiles t;
    i32x4 own[LOCAL ? 1 : 2][32 * 9];  // a reading wave's own: 64 channels of its rows, or its outputs
};
// FINE: scores and the state as it is read in two parts each; the state's second part takes the first one's place in LDS
// between two more barriers.
template <int K, bool LOCAL, bool FINE>
__device__ __forceinline__ void dla_body(const DlaParams& p, i32x4* lds, int item, int ip) {
    typedef DlaWork<bf16, K, kDlaVS, LOCAL> Work;
    typedef typename DlaLds<K, LOCAL>::Stage Stage;
    constexpr int KK = K / 16, RY = Work::RY, RZ = Work::RZ, VB = kDlaVS / 32;
    // carrying waves, and the blocks of 32 x 32 of each: rows cw % NK + NK kb, columns cv + vb (times 32)
    constexpr int NW = LOCAL ? 4 : 2, NK = NW < K / 32 ? NW : K / 32, KB = K / 32 / NK, CB = VB * NK / NW;
    auto& t = ((DlaLds<K, LOCAL>*)lds)->t;
    const Work k(p, item, ip);
    if (LOCAL && k.c1 - k.c0 < p.seg_chunks) return;  // no later segment has a token: nobody reads this one's state
    const int l = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id()), n = l & 31, hf = l >> 5;
    Stage st(k, t, (int)threadIdx.x - (LOCAL ? 0 : 128), threadIdx.x);
    if (LOCAL || w >= 2) {
        const int cw = LOCAL ? w : w - 2, ck = cw % NK, cv = cw / NK * CB;
        f32x16 S[KB][CB];  // rows 32 (ck + NK kb) + acc_row32(i), columns 32 (cv + vb) + n
        auto each_block = [&](auto&& f) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int vb = 0; vb < CB; ++vb) f(S[kb][vb], ck + NK * kb, cv + vb);
        };
        auto each_four = [&](int j, auto&& f) {  // of the own state of segment j
            f32x4* at = (f32x4*)k.local(j) + l;
            each_block([&](f32x16& s, int kb, int vb) {
#pragma unroll
                for (int i = 0; i < 4; ++i) f(s, 4 * i, at[((kb * VB + vb) * 4 + i) * 64]);
            });
        };
        each_block([&](f32x16& s, int, int) { s = zeros16(); });
        if constexpr (!LOCAL) {
            if (k.ps.init)
                each_block([&](f32x16& s, int kb, int vb) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[i] = k.ps.init[k.state_at(32 * kb + acc_row32(i, l), 32 * vb + n)];
                });
            for (int j = 0; j < k.sg && k.c0 < k.nch; ++j) {
                const float e = expm1f((float)(p.seg_chunks * C - (j == 0 ? k.early : 0)) * k.ga);
                each_four(j, [&](f32x16& s, int i0, const f32x4& x) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[i0 + i] = fmaf(s[i0 + i], e, s[i0 + i]) + x[i];
                });
            }
        }
        auto put_state = [&]() {
            if constexpr (!LOCAL)
                each_block([&](const f32x16& s, int kb, int vb) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        store4((bf16*)(t.s[0] + (32 * vb + n) * Stage::RS + 4 * kb + i) + 4 * hf, f32x4{s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]});
                });
        };
        auto put_rest = [&]() {  // what rounding left of it
            each_block([&](const f32x16& s, int kb, int vb) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f32x4 r;
#pragma unroll
                    for (int e = 0; e < 4; ++e) r[e] = s[4 * i + e] - (float)(bf16)s[4 * i + e];
                    store4((bf16*)(t.s[0] + (32 * vb + n) * Stage::RS + 4 * kb + i) + 4 * hf, r);
                }
            });
        };
        const float whole = expm1f((float)C * k.ga);
        if (k.c0 < k.c1) {
            st.template fetch<0>(k.c0);
            put_state();
            st.template put<0>(k.c0);
            st.template fetch<0>(k.c0 + 1);
        }
        for (int ch = k.c0; ch < k.c1; ++ch) {
            lds_barrier();
            if constexpr (FINE) {
                lds_barrier();
                put_rest();
                lds_barrier();
            }
            const float e = k.decay(ch, whole);
            each_block([&](f32x16& s, int, int) {
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i] = fmaf(s[i], e, s[i]);
            });
#pragma unroll
            for (int kk = 0; kk < C / 16; ++kk) {
                bf16x8 y[KB];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) y[kb] = columns32<RY>(t.y[0], 16 * kk, 4 * (ck + NK * kb), l);
#pragma unroll
                for (int q = 0; q < Stage::NP; ++q) {
                    if (q == 2 && !st.exact) break;
#pragma unroll
                    for (int vb = 0; vb < CB; ++vb) {
                        const bf16x8 z = columns32<RZ>(t.d[0][q], 16 * kk, 4 * (cv + vb), l);
#pragma unroll
                        for (int kb = 0; kb < KB; ++kb) mma32x32(S[kb][vb], y[kb], z);
                    }
                }
            }
            if (ch + 1 < k.c1) {
                lds_barrier();
                put_state();
                st.template put<0>(ch + 1);
                st.template fetch<0>(ch + 2);
            }
        }
        if constexpr (LOCAL) {
            each_four(k.sg, [&](const f32x16& s, int i0, f32x4& x) { x = f32x4{s[i0], s[i0 + 1], s[i0 + 2], s[i0 + 3]}; });
        } else if (k.ps.fin && k.final_here()) {
            // against time the final state is decayed once more (dS0 = a R_0)
            const float f = k.rev && k.L > 0 ? dla_pow(k.ga, 1) : 1.f;
            each_block([&](const f32x16& s, int kb, int vb) {
#pragma unroll
                for (int i = 0; i < 16; ++i) k.ps.fin[k.state_at(32 * kb + acc_row32(i, l), 32 * vb + n)] = s[i] * f;
            });
        }
    } else {
        // The wave's 32 rows arrive as whole lines (a lane's own pieces, as the products want them, would be 32 lines a
        // load), and outputs leave so; both turn round in the wave's own LDS.
        DlaStream xs = k.rows_of_k(k.ps.x), os = k.rows_of_v(k.ps.out);
        i32x4* own = ((DlaLds<K, LOCAL>*)lds)->own[w];
        constexpr int XR = 8, XH = K / 64;  // pieces of a row and rounds: 64 channels at a time
        const int xrow = 32 * w + n;
        const int xo = k.off(32 * w + l / XR, k.sx) + l % XR * 16, oo = k.off(32 * w + l / RZ, k.sz) + l % RZ * 16;
        const int xd = k.rev ? -8 * k.sx : 8 * k.sx, od = k.rev ? -8 * k.sz : 8 * k.sz;  // eight rows on
        int at[KK];  // row n of a tile, the lane's piece
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) at[kk] = tile_at<bf16, RY>(n, 2 * kk + hf);
        i32x4 xp[XH][4], xr[KK];
        auto fetch_x = [&](int ch) {
            int shift;
            const auto x = xs.next(ch, shift);
#pragma unroll
            for (int q = 0; q < XH; ++q)
#pragma unroll
                for (int u = 0; u < 4; ++u) xp[q][u] = load16(x, xo + (xd * u - shift) + q * 128);
        };
        auto take_x = [&]() {
#pragma unroll
            for (int q = 0; q < XH; ++q) {
                wave_sync();
#pragma unroll
                for (int u = 0; u < 4; ++u) own[(8 * u + l / XR) * (XR + 1) + l % XR] = xp[q][u];
                wave_sync();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) xr[4 * q + kk] = own[n * (XR + 1) + 2 * kk + hf];
            }
        };
        auto put_out = [&](int ch, const f32x16 (&out)[VB]) {
            static_assert(RZ == XR, "outputs turn round in the rows' place");
            wave_sync();
#pragma unroll
            for (int vb = 0; vb < VB; ++vb)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    store4((bf16*)(own + n * (XR + 1) + 4 * vb + i) + 4 * hf, f32x4{out[vb][4 * i], out[vb][4 * i + 1], out[vb][4 * i + 2], out[vb][4 * i + 3]});
            wave_sync();
            int shift;
            const auto o = os.next(ch, shift);
#pragma unroll
            for (int u = 0; u < 4; ++u) store16(o, oo + (od * u - shift), own[(8 * u + l / XR) * (XR + 1) + l % XR]);
        };
        // Weights that every chunk shares: a^(r - s) inside the wave's 32 rows and to the 32 before them.  The lane's values
        // 4 j .. 4 j + 3 of a block are rows s = s_j .. s_j + 3, so a^(r - s) is a^(r - s_j - 3) times a^3, a^2, a, 1; both are
        // powers with an exponent >= 0 but where the diagonal passes through the four, which have weights of their own.
        float self[4], prev[4], diag[4];
        const float a1 = uniform(dla_pow(k.ga, 1)), a2 = uniform(dla_pow(k.ga, 2)), a3 = uniform(dla_pow(k.ga, 3));
        const float fall[4] = {a3, a2, a1, 1.f};
        const int first = n - 4 * hf;     // r - s_0
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            self[j] = first - 8 * j < 3 ? 0.f : dla_pow(k.ga, first - 8 * j - 3);
            prev[j] = dla_pow(k.ga, first - 8 * j + 29);
            const int lag = (n & 7) - 4 * hf - j;
            diag[j] = lag < 0 ? 0.f : dla_pow(k.ga, lag);
        }
        const int on = first < 0 || first % 8 > 2 ? -1 : first / 8;  // the four that the diagonal leaves in part
        const float before = dla_pow(k.ga, xrow + 1), before0 = k.early ? dla_pow(k.ga, xrow) : before;
        if (k.c0 < k.c1) {
            fetch_x(k.c0);
            st.template fetch_z<0>(k.c0);
            take_x();
            st.template put_z<0>(k.c0);
            fetch_x(k.c0 + 1);
            st.template fetch_z<0>(k.c0 + 1);
        }
        for (int ch = k.c0; ch < k.c1; ++ch) {
            lds_barrier();
            // from before the chunk: out^T = S^T x, rows v, columns r; and scores, rows s, columns r
            f32x16 out[VB], sc = zeros16();
#pragma unroll
            for (int vb = 0; vb < VB; ++vb) out[vb] = zeros16();
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                const bf16x8 x = __builtin_bit_cast(bf16x8, xr[kk]);
                mma32x32(sc, __builtin_bit_cast(bf16x8, t.y[0][at[kk] + w * 32 * RY]), x);
#pragma unroll
                for (int vb = 0; vb < VB; ++vb)
                    mma32x32(out[vb], __builtin_bit_cast(bf16x8, t.s[0][(32 * vb + n) * Stage::RS + 2 * kk + hf]), x);
            }
            if constexpr (FINE) {
                lds_barrier();
                lds_barrier();
#pragma unroll
                for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                    for (int vb = 0; vb < VB; ++vb)
                        mma32x32(out[vb], __builtin_bit_cast(bf16x8, t.s[0][(32 * vb + n) * Stage::RS + 2 * kk + hf]), __builtin_bit_cast(bf16x8, xr[kk]));
            }
            const float f = ch == 0 ? before0 : before;
#pragma unroll
            for (int vb = 0; vb < VB; ++vb)
#pragma unroll
                for (int i = 0; i < 16; ++i) out[vb][i] *= f;
            // out^T += z^T scores^T
            auto add = [&](const f32x16& score, int r0, auto inside) {
                constexpr bool SELF = decltype(inside)::value;
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    bf16x8 pr, rest;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int j = 2 * kk + e / 4, i = e % 4;
                        const float wt = SELF ? j == on ? diag[i] : self[j] * fall[i] : prev[j] * fall[i];
                        const float x = score[8 * kk + e] * wt;
                        pr[e] = (bf16)x;
                        if constexpr (FINE) rest[e] = (bf16)(x - (float)pr[e]);
                    }
#pragma unroll
                    for (int vb = 0; vb < VB; ++vb) {
                        const bf16x8 z = columns32<RZ>(t.z[0], r0 + 16 * kk, 4 * vb, l);
                        mma32x32(out[vb], z, pr);
                        if constexpr (FINE) mma32x32(out[vb], z, rest);
                    }
                }
            };
            add(sc, 32 * w, IC<1>{});
            if (w) {
                sc = zeros16();
#pragma unroll
                for (int kk = 0; kk < KK; ++kk)
                    mma32x32(sc, __builtin_bit_cast(bf16x8, t.y[0][at[kk]]), __builtin_bit_cast(bf16x8, xr[kk]));
                add(sc, 0, IC<0>{});
            }
            put_out(ch, out);
            if (ch + 1 < k.c1) {
                take_x();
                fetch_x(ch + 2);
                lds_barrier();
                st.template put_z<0>(ch + 1);
                st.template fetch_z<0>(ch + 2);
            }
        }
        k.pad(threadIdx.x, 128);
    }
}
template <int KM, bool LOCAL, bool FINE>
__global__ __launch_bounds__(256, LOCAL ? 3 : 2) void gdr2_dla_kernel(DlaParams p, int nwork) {
    __shared__ i32x4 lds[sizeof(DlaLds<KM ? KM : 128, LOCAL>) / 16];
    dla_share<KM>(p, nwork, [&](auto k, int item, int ip) { dla_body<decltype(k)::value, LOCAL, FINE>(p, lds, item, ip); });
}

// ------------------------------------------------------------------ fp32
// 16 x 16 products, of which this type's scores need eight times as many cycles: waves 0..3 read sixteen rows each,
// waves 4..7 carry every fourth sixteen of the state's rows.
template <int K, bool LOCAL>
using DlaF32Stage = DlaStage<float, K, kDlaF32VS, LOCAL, LOCAL ? 256 : 512, LOCAL ? 256 : 512, 2>;
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
    Stage st(k, t, threadIdx.x, threadIdx.x);
    if (k.c0 < k.c1) {
        st.template fetch<0>(k.c0);
        st.template fetch<1>(k.c0 + 1);
    }
    if (LOCAL || w >= 4) {
        // blocks of 16 x 16: rows 16 (cw + 4 kb) + 4 g + i, column 16 vb + c
        const int cw = LOCAL ? w : w - 4;
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
        if constexpr (!LOCAL) {
            if (k.ps.init)
                each([&](f32x4& s, int row, int v, int) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[i] = k.ps.init[k.state_at(row + i, v)];
                });
            for (int j = 0; j < k.sg && k.c0 < k.nch; ++j) {
                const float e = expm1f((float)(p.seg_chunks * C - (j == 0 ? k.early : 0)) * k.ga);
                const f32x4* own = (const f32x4*)k.local(j);
                each([&](f32x4& s, int, int, int at) {
                    const f32x4 x = own[at];
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[i] = fmaf(s[i], e, s[i]) + x[i];
                });
            }
        }
        auto put_state = [&](auto set) {
            constexpr int P = decltype(set)::value;
            if constexpr (!LOCAL) each([&](const f32x4& s, int row, int v, int) { *(f32x4*)(t.s[P] + tile_at<float, RY>(v, row / 4)) = s; });
        };
        const float whole = expm1f((float)C * k.ga);
        if (k.c0 < k.c1) {
            put_state(IC<0>{});
            st.template put<0>(k.c0);
            st.template fetch<0>(k.c0 + 2);
        }
        auto chunk = [&](int ch, auto set) {
            constexpr int P = decltype(set)::value;
            lds_barrier();
            const float e = k.decay(ch, whole);
            each([&](f32x4& s, int, int, int) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[i] = fmaf(s[i], e, s[i]);
            });
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int r = 16 * (j / 4) + 4 * g + j % 4;
                float y[KB];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) y[kb] = column(t.y[P], IC<RY>{}, r, cw + 4 * kb);
#pragma unroll
                for (int vb = 0; vb < VB; ++vb) {
                    const float z = column(t.d[P][0], IC<RZ>{}, r, vb);
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
        for (int ch = k.c0; ch < k.c1; ch += 2) {
            chunk(ch, IC<0>{});
            if (ch + 1 < k.c1) chunk(ch + 1, IC<1>{});
        }
        if constexpr (LOCAL) {
            f32x4* own = (f32x4*)k.local(k.sg);
            each([&](const f32x4& s, int, int, int at) { own[at] = s; });
        } else if (k.ps.fin && k.final_here()) {
            const float f = k.rev && k.L > 0 ? dla_pow(k.ga, 1) : 1.f;
            each([&](const f32x4& s, int row, int v, int) {
#pragma unroll
                for (int i = 0; i < 4; ++i) k.ps.fin[k.state_at(row + i, v)] = s[i] * f;
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
__global__ __launch_bounds__(LOCAL ? 256 : 512, 2) void gdr2_dla_f32_kernel(DlaParams p, int nwork) {
    __shared__ i32x4 lds[sizeof(typename DlaF32Stage<KM ? KM : 128, LOCAL>::Tiles) / 16];
    dla_share<KM>(p, nwork, [&](auto k, int item, int ip) { dla_f32_body<decltype(k)::value, LOCAL>(p, lds, item, ip); });
}

// Segments of the sequence: as many as fill the device once (two workgroups of bf16 to a compute unit, one of fp32), none
// below four chunks.  Measured for 128 / 256 / 384 / 512 / 768 / 1024 workgroups of bf16: B = 4, T = 4096, H = 16 forward
// 152 / 140 / 130 / 123 / 131 / 137 us, B = 1, T = 32768, H = 16 467 / 254 / 245 / 225 / 245 / 252 (unsplit 1143); the
// backward of the first, 384 workgroups in one segment, took 199 us, in two segments 242.  fp32, B = 3, T = 777, H = 6: at least
// four chunks 29 us against 42 with at least sixteen (one segment); 512 instead of 256 workgroups made its backward 84 us
// from 76.
DlaCut dla_cut(long B, long T, long H, long slots, bool f32) {
    const long nch = (T + C - 1) / C, jobs = B * H * slots, least = 4;
    long segs = jobs > 0 ? (f32 ? 256 : 512) / jobs : 1;
    segs = segs < nch / least ? segs : nch / least;
    segs = segs < 1 ? 1 : segs;
    DlaCut c{};
    c.seg_chunks = (int)((nch + segs - 1) / segs);
    c.seg_chunks = c.seg_chunks < 1 ? 1 : c.seg_chunks;
    c.segs = (int)((nch + c.seg_chunks - 1) / c.seg_chunks);
    c.segs = c.segs < 1 ? 1 : c.segs;
    return c;
}

template <int KM, bool LOCAL>
static hipError_t launch_dla(bool bf, long n, const DlaParams& p, hipStream_t s) {
    const dim3 grid((unsigned)((n + 7) / 8 * 8));
    if (bf && !LOCAL && p.T <= kDlaFine) hipLaunchKernelGGL((gdr2_dla_kernel<KM, false, true>), grid, dim3(256), 0, s, p, (int)n);
    else if (bf) hipLaunchKernelGGL((gdr2_dla_kernel<KM, LOCAL, false>), grid, dim3(256), 0, s, p, (int)n);
    else hipLaunchKernelGGL((gdr2_dla_f32_kernel<KM, LOCAL>), grid, dim3(LOCAL ? 256 : 512), 0, s, p, (int)n);
    return hipGetLastError();
}
template <bool LOCAL>
static hipError_t launch_dla_k(bool bf, long n, const DlaParams& p, hipStream_t s) {
    for (int i = 1; i < p.passes; ++i)
        if (p.pass[i].K != p.pass[0].K) return launch_dla<0, LOCAL>(bf, n, p, s);
    return p.pass[0].K == 128 ? launch_dla<128, LOCAL>(bf, n, p, s) : launch_dla<64, LOCAL>(bf, n, p, s);
}

int dla_slots(int V, bool f32) { return V / (f32 ? kDlaF32VS : kDlaVS); }

hipError_t dla_dispatch(int bf, const DlaParams& p, hipStream_t s) {
    const long per = (long)p.B * p.H * p.slots;  // workgroups of a segment
    if (p.segs > 1) {
        const hipError_t e = launch_dla_k<true>(bf, per * (p.segs - 1), p, s);
        if (e != hipSuccess) return e;
    }
    return launch_dla_k<false>(bf, per * p.segs, p, s);
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

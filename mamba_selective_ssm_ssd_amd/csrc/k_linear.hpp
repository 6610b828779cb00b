// k_linear.hpp -- linear attention with a decay for each head: the chunked
// scan that serves the prompt pass and, with its operands exchanged or the
// tokens walked backwards, the three gradients, and its launch.
//
// One scan, with g = exp(log_decay) and rows x_i, y_i (DX channels) and z_i
// (DZ channels) in scan order, keeps a DX x DZ state S in fp32 and writes
//     out_i = a_in sum_{j<=i} g^{i-j} (x_i . y_j) z_j + a_init g^{i+e} x_i^T S,
//     S    <- g^C S + a_state sum_j g^{C-e-j} y_j z_j^T    behind C rows,
// with S the state at the start of the chunk and e = 1, or e = 0 where the
// scan runs from the last token to the first.  With s the scale of o:
//     o  : (q, k, v),  state S,    forwards,  s, s, 1
//     dq : (go, v, k), state S^T,  forwards,  s, s, 1
//     dk : (v, go, q), state G^T,  backwards, s, 1, s
//     dv : (k, q, go), state G,    backwards, s, 1, s
// where G_t = g G_{t+1} + s q_t go_t^T is the gradient of S_t.
//
// Four waves walk one sequence (or a segment of one) for one head, chunk by
// chunk, with the state in registers as fp32 accumulators of the matrix
// instruction: the products of a chunk are (rows x rows x channels) for the
// weights, (rows x rows x channels) and (rows x channels x channels) for the
// outputs, (channels x rows x channels) for the state.  The weights come out of
// the matrix instruction transposed, which is the layout that the next product
// takes as its operand, so they never leave the registers; only the rows and the
// state's bf16 image pass through LDS.  The next chunk's rows are in flight to
// registers meanwhile, one barrier before the products and one behind.
// Chunks of 64 rows: as many as two workgroups a compute unit have room for.
//
// Bound by memory where the chip is full, at 4.5 to 4.9 TB/s of the 5.2 that a
// large copy reaches: 32 x 1024 x 32 x 128 250 us (4.6 TB/s); of 65536 x 64 x 64
// cut into 64 segments the pre-pass 238 us (4.7) and the outputs 450 us (4.9).
// Matrix units are busy 23% of the time, LDS 25%, vector units 31%.  Few
// workgroups are bound by the chain of chunks: 3.3 us per 64 rows of 128 x 128.
#pragma once

#include "m3_device.hpp"

#include <stddef.h>
#include <type_traits>

namespace m3 {

// One scan of a launch.  Strides in elements.
struct LinRole {
    const void *x, *y, *z;
    void *out;
    int64_t xt, xh, yt, yh, zt, zh, ot, oh;
    int32_t xg, yg, zg;      // heads that share one row of x, y, z
    int32_t dx, dz;          // channels, multiples of 8
    int32_t rev;             // from the last token to the first
    int32_t out32;           // out is fp32 whatever the I/O type
    float a_in, a_init, a_state;
    const void *init;        // state pool, or null: zero
    void *fin;               // state pool, or null: not written
    int32_t init16, fin16;   // the pools' entries are bf16
    int32_t sm, sn;          // strides of the state's two axes (pools and seg alike)
    float *seg;              // [state slot][H][dx dz] fp32, for the start of each segment of a cut sequence
};

struct LinParams {
    LinRole role[3];
    int32_t nroles, H, ztiles;
    int32_t hg, group;       // heads that share rows; workgroups that do: hg x ztiles x nroles
    int32_t tail;            // extra workgroups per scan that zero the rows outside every sequence
    int32_t nwork;           // workgroups without the tail
    int32_t grad;            // the scans are gradients
    int64_t batch, tokens, each; // each: tokens of a sequence without cu
    const int32_t *cu;       // null: equal sequences
    const int32_t *slots;    // null: sequence b has state b
    int64_t nstates;
    const float *log_decay;
    int32_t segbits;         // log2 of the tokens per segment, 0: sequences are not cut
    int32_t fold;            // slots hold what each segment leaves, not yet joined
    int64_t nseg;            // segment slots (batch when not cut)
    int32_t sparse;          // states are kept for cut sequences alone
};

// First token of sequence b, clamped to the rows there are.
__device__ __forceinline__ int64_t lin_start(const LinParams &p, int64_t b) {
    if (!p.cu) return b * p.each;
    const int64_t c = p.cu[b];
    return c < 0 ? 0 : c > p.tokens ? p.tokens : c;
}

constexpr int64_t kSlotSkip = -1, kSlotTaken = -2;

// State of sequence b: its slot, kSlotSkip for padding, kSlotTaken where an
// earlier sequence of the call names the same slot.  All threads of the
// workgroup call it.  Every workgroup reads the slots before its own: prompts of
// 4096 x 16 tokens of 16 x 64 x 64 934 us, 1126 with slots, and 496 and 568 of
// 1024 x 32 of 32 x 64 x 64, most of it the states' order in memory.
__device__ __forceinline__ int64_t lin_slot(const int32_t *slots, int64_t nstates, int64_t b) {
    if (!slots) return b;
    const int64_t s = slots[b];
    if (s < 0 || s >= nstates) return kSlotSkip;
    int dup = 0;
    for (int64_t j = threadIdx.x; j < b; j += blockDim.x) dup |= slots[j] == s;
    return __syncthreads_or(dup) ? kSlotTaken : s;
}

// Segment slots.  A sequence of n tokens has ceil(n / L) segments of L tokens
// (one, empty, without a token) and gets the slots from start / L + b on:
// floor((start + n) / L) - floor(start / L) + 1 >= ceil(n / L), so the slots
// of two sequences never meet, there are at most tokens / L + batch of them,
// and the sequence of a slot is found by bisection without any table.
__device__ __forceinline__ int64_t lin_first_slot(const LinParams &p, int64_t b) { return (lin_start(p, b) >> p.segbits) + b; }

// Where the states of sequence b's segments lie: at their slots, or, where there
// are more sequences than segments of tokens, from 2 start / L on.  Only a cut
// sequence, of n > L tokens, has states, and floor(2 (start + n) / L) -
// floor(2 start / L) >= floor(2 n / L) >= ceil(n / L): two never meet, and there
// are at most 2 tokens / L, however many sequences.
__device__ __forceinline__ int64_t lin_state_slot(const LinParams &p, int64_t b, int64_t start) {
    return p.sparse ? 2 * start >> p.segbits : (start >> p.segbits) + b;
}

// ---------------------------------------------------------------------------
// Operands as PL planes of bf16 whose sum is the value: one plane for bf16
// values, three for fp32 ones (8 bits each: the 24 of an fp32 mantissa).  A
// product takes the pairs of planes whose weights stay within 2^-16 of the
// leading one, smallest first: 1, 3 (one side bf16) or 6 instructions, and is
// exact to about 2^-24.  Six bf16 instructions still do a product at 2.7 times
// the rate of the fp32 instruction.
// ---------------------------------------------------------------------------
template <int PL>
struct lfrag {
    bf16x8 v[PL];
};

template <int PA, int PB>
__device__ __forceinline__ floatx4 lmma(floatx4 acc, const lfrag<PA> &a, const lfrag<PB> &b) {
#pragma unroll
    for (int s = 2; s >= 0; --s)
#pragma unroll
        for (int i = PA - 1; i >= 0; --i)
            if (s - i >= 0 && s - i < PB) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[s - i], acc, 0, 0, 0);
    return acc;
}

// f(i, j) for the pairs of planes of a product, in that order.
template <int PA, int PB, typename F>
__device__ __forceinline__ void lpairs(F &&f) {
    auto pair = [&](auto i, auto j) {
        if constexpr (i.value < PA && j.value < PB) f(i, j);
    };
    typedef std::integral_constant<int, 0> c0;
    typedef std::integral_constant<int, 1> c1;
    typedef std::integral_constant<int, 2> c2;
    pair(c2(), c0());
    pair(c1(), c1());
    pair(c0(), c2());
    pair(c1(), c0());
    pair(c0(), c1());
    pair(c0(), c0());
}

template <int PL>
__device__ __forceinline__ lfrag<PL> lsplit(const float a[8]) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = a[i];
    lfrag<PL> f;
#pragma unroll
    for (int k = 0; k < PL; ++k) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = pack2_bf16(r[2 * i], r[2 * i + 1]);
            if (k + 1 < PL) {
                r[2 * i] -= __uint_as_float(w[i] << 16);
                r[2 * i + 1] -= __uint_as_float(w[i] & 0xffff0000u);
            }
        }
        f.v[k] = bf16x8_from_words(w[0], w[1], w[2], w[3]);
    }
    return f;
}

template <int PL>
__device__ __forceinline__ void lunsplit(const lfrag<PL> &f, float a[8]) {
#pragma unroll
    for (int k = PL - 1; k >= 0; --k) {
        const uint4 w = __builtin_bit_cast(uint4, f.v[k]);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float lo = __uint_as_float(ws[i] << 16), hi = __uint_as_float(ws[i] & 0xffff0000u);
            a[2 * i] = k + 1 < PL ? a[2 * i] + lo : lo;
            a[2 * i + 1] = k + 1 < PL ? a[2 * i + 1] + hi : hi;
        }
    }
}

// ---------------------------------------------------------------------------
// Tile of one scan.  Q rows per chunk, DX x DZ state columns of a workgroup of
// four waves; z columns beyond DZ are another workgroup's.
// ---------------------------------------------------------------------------
template <typename IO, int DX, int DZ, bool OUT>
struct LinCfg {
    static constexpr bool F32 = std::is_same<IO, float>::value;
    static constexpr int PL = F32 ? 3 : 1;
    // planes of the weights: a row of a few tokens is the sum of a few of them, so a
    // bf16 result would show one plane's rounding whole, beside its own
    static constexpr int WP = F32 ? 3 : 2;
    static constexpr int Q = F32 || (OUT && DX == 128 && DZ == 128) ? 32 : 64; // 64 rows of 128 x 128 spill (gradients of 4999 x 32 (8) x 128 442 us for 219)
    static constexpr int MP = DX / 32, NP = DZ / 32; // 32 x 32 blocks of the state, 16 x 16 tiles in pairs
    // the state's tiles over the waves: MW along x (MTW tiles each, a pair of
    // one block where it is two), NW along z
    static constexpr int W = 4, T = 64 * W;
    static constexpr int WAVES = OUT || DX * DZ > 64 * 128 ? 2 : DX * DZ > 64 * 64 ? 3 : 4; // a SIMD, as far as registers go round
    static constexpr int MW = 2 * MP < W ? 2 * MP : W, MTW = 2 * MP / MW, NW = W / MW, NTW = 2 * NP / NW;
    static_assert(MTW <= 2 && NTW >= 1, "tiles of a wave");
    // the output's 16-row tiles over the waves: RW along the rows, OW along z (NOT tiles each)
    static constexpr int RW = Q / 16, OW = W / RW, NOT = 2 * NP / OW;
    static_assert(NOT >= 1 && (F32 || NOT % 2 == 0), "output tiles of a wave, pairs where two share a store");
    static_assert(NW == 1 || OW == 1 || MW == RW, "a wave's tiles of the state and of the output start alike");
    static constexpr int KS = Q / 32; // 32-row steps of a product over the chunk's rows
    // LDS, in bf16 elements: x, y, z planes and the state's fragments
    static constexpr int XP = Q * DX, ZP = Q * DZ, SP = DX * DZ;
    static constexpr int XO = 0, YO = OUT ? PL * XP : 0, ZO = YO + PL * XP, SO = ZO + PL * ZP;
    static constexpr size_t bytes = 2 * size_t(SO + (OUT ? PL * SP : 0));
};

// A staged row's 16-byte units are permuted by the row, in pairs and within a
// pair, so that 16 rows at one unit (row reads), and eight rows at one pair (the
// transposing reads of 16 neighbouring columns), touch every bank once.
template <int D>
__device__ __forceinline__ int lin_at(int row, int unit) {
    constexpr int P = D / 16, SH = P >= 8 ? 0 : P == 4 ? 1 : 2;
    return row * D + (((((unit >> 1) ^ (row >> SH & (P - 1))) << 1) | ((unit & 1) ^ (row >> 3 & 1))) << 3);
}

// Eight k-slots of a column of a staged matrix: rows 16 t0 + 4 g + v, then
// 16 (t0 + 1) + 4 g + v, read transposed: lane j of a group addresses four
// columns of row j / 4, and gets column `j` of the group's 16.
template <int PL, int D, int PS>
__device__ __forceinline__ lfrag<PL> lin_tr(const uint16_t *m, int row, int unit, int part) {
    const uint16_t *p0 = m + lin_at<D>(row, unit) + 4 * part, *p1 = m + lin_at<D>(row + 16, unit) + 4 * part;
    lfrag<PL> f;
#pragma unroll
    for (int k = 0; k < PL; ++k) {
        const uint2 a = lds_tr4(p0 + k * PS), b = lds_tr4(p1 + k * PS);
        f.v[k] = bf16x8_from_words(a.x, a.y, b.x, b.y);
    }
    return f;
}
// Tile n of z: lane r has column 16 n + r.
template <int PL, int D, int PS>
__device__ __forceinline__ lfrag<PL> lin_zcol(const uint16_t *m, int t0, int n, int r16, int g) {
    return lin_tr<PL, D, PS>(m, 16 * t0 + 4 * g + (r16 >> 2), 2 * n + (r16 >> 1 & 1), r16 & 1);
}
// Tile t of y: lane r has column 32 (t / 2) + 8 (r / 4) + r % 4 + 4 (t % 2), so
// that the state's rows of two tiles are eight neighbours in one lane: the
// k-slots of a row of x.
template <int PL, int D, int PS>
__device__ __forceinline__ lfrag<PL> lin_ycol(const uint16_t *m, int t0, int t, int r16, int g) {
    return lin_tr<PL, D, PS>(m, 16 * t0 + 4 * g + (r16 >> 2), 4 * (t >> 1) + (r16 & 3), t & 1);
}
template <int PL, int D, int PS>
__device__ __forceinline__ lfrag<PL> lin_row(const uint16_t *m, int row, int unit) {
    const uint16_t *p = m + lin_at<D>(row, unit);
    lfrag<PL> f;
#pragma unroll
    for (int k = 0; k < PL; ++k) f.v[k] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4 *>(p + k * PS));
    return f;
}

// Bounded access to the rows of one chunk.  A chunk of fewer than Q rows lies at
// the end of its tile, so that what a row weighs at the chunk's end, and in the
// rows behind it, is the same in every chunk; the rows before it read as zero
// and are not written.  Offsets count from the chunk's lowest token: walking
// forwards a row before the chunk lies below zero, which as an unsigned number
// is beyond the end, walking backwards beyond the end itself.
constexpr uint32_t kNowhere = 0xffffffe0u; // beyond the end of every buffer, with the 16 bytes behind it

struct LinBuf {
    __amdgpu_buffer_rsrc_t r;
    __device__ __forceinline__ LinBuf(const void *base, uint32_t bytes)
        : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, bytes, 0x00027000)) {}
    __device__ __forceinline__ uint4 load(uint32_t at) const {
        const u32x4_v v = __builtin_bit_cast(u32x4_v, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
        return make_uint4(v.x, v.y, v.z, v.w);
    }
    __device__ __forceinline__ void store(uint32_t at, uint4 v) const {
        __builtin_amdgcn_raw_buffer_store_b128(u32x4_v{v.x, v.y, v.z, v.w}, r, at, 0, 0);
    }
    __device__ __forceinline__ float get(uint32_t at) const { return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0)); }
    __device__ __forceinline__ float get16(uint32_t at) const { return bits_to_f32(uint16_t(__builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0))); }
    __device__ __forceinline__ void put(uint32_t at, float v) const { __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, at, 0, 0); }
    __device__ __forceinline__ void put16(uint32_t at, float v) const { __builtin_amdgcn_raw_buffer_store_b16(f32_to_bits(v), r, at, 0, 0); }
};

// Eight consecutive elements as loaded.
template <typename IO>
struct lraw;
template <>
struct lraw<bf16> {
    uint4 a;
    __device__ __forceinline__ void load(const LinBuf &r, uint32_t at) { a = r.load(at); }
    template <int PS>
    __device__ __forceinline__ void stage(uint16_t *p) const { *reinterpret_cast<uint4 *>(p) = a; }
};
template <>
struct lraw<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const LinBuf &r, uint32_t at) { a = r.load(at); b = r.load(at + 16); }
    template <int PS>
    __device__ __forceinline__ void stage(uint16_t *p) const {
        const float v[8] = {__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w),
                            __uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w)};
        const lfrag<3> f = lsplit<3>(v);
#pragma unroll
        for (int k = 0; k < 3; ++k) *reinterpret_cast<uint4 *>(p + k * PS) = __builtin_bit_cast(uint4, f.v[k]);
    }
};

// A chunk's rows of one operand: issued to registers, staged to LDS later.
template <typename IO, int Q, int D, int T>
struct LinRegs {
    static constexpr int U = D / 8, PIECES = Q * U, N = (PIECES + T - 1) / T;
    lraw<IO> r[N];
    template <int PS>
    __device__ __forceinline__ void stage(uint16_t *m) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int piece = threadIdx.x + i * T;
            if (PIECES % T == 0 || piece < PIECES) r[i].template stage<PS>(m + lin_at<D>(piece / U, piece % U));
        }
    }
};

template <typename IO, int Q, int D, int T>
struct LinRows {
    static constexpr int U = D / 8;
    const char *base;  // the row of the next chunk's first token (walking backwards: last)
    uint32_t step;     // bytes from token to token
    uint32_t at;       // byte offset of this thread's first piece in a full chunk
    bool rev, on;
    __device__ __forceinline__ void init(const void *rows, int64_t t0, int64_t stride, int64_t off, int dim, bool back) {
        const int row = threadIdx.x / U, unit = threadIdx.x % U;
        step = uint32_t(stride) * sizeof(IO);
        rev = back;
        base = static_cast<const char *>(rows) + (t0 * stride + off) * int64_t(sizeof(IO));
        at = uint32_t(back ? Q - 1 - row : row) * step + unit * uint32_t(8 * sizeof(IO));
        on = unit * 8 < dim && row < Q;
    }
    // the next `rows` rows; Q of them where more follow
    __device__ __forceinline__ void load(LinRegs<IO, Q, D, T> &to, int rows) {
        const LinBuf b(base - (rev ? uint32_t(rows - 1) * step : 0u), uint32_t(rows) * step);
        base += rev ? -int64_t(Q) * step : int64_t(Q) * step;
        const uint32_t first = at - (rev ? 0u : uint32_t(Q - rows) * step), next = (rev ? 0u - step : step) * (T / U);
#pragma unroll
        for (int i = 0; i < to.N; ++i) to.r[i].load(b, on ? first + i * next : kNowhere);
    }
};

// g^n, 1 for n <= 0 rows: g = 0 (log_decay = -inf) keeps the row itself.  ld2 is
// log_decay / log 2; the exponent is off by two roundings of itself, 2^-22 of a
// factor of e^-2 and less where the factor is nearer to one.
__device__ __forceinline__ float lin_power(float ld2, int n) { return n > 0 ? __builtin_amdgcn_exp2f(ld2 * float(n)) : 1.f; }

// s g^n, rounded once.  A slow decay is taken as s + s (g^n - 1): g^n itself,
// rounded to 24 bits, would err the same way in every chunk of a long sequence.
// Of an infinite s that sum makes inf - inf: such a result is s again, an
// infinity as the product is, or the NaN that it was.  A decay that is NaN makes
// everything NaN.
struct LinDecay {
    float f;
    uint32_t keep; // all of s, or nothing, to add
    float poison;  // 0, or NaN where f is
    __device__ __forceinline__ LinDecay(float ld, double n) {
        const float x = n > 0 ? float(double(ld) * n) : 0.f;
        f = x > -0.5f ? expm1f(x) : expf(x);
        keep = x > -0.5f ? 0xffffffffu : 0u;
        poison = f - f;
    }
    __device__ __forceinline__ float operator()(float s) const {
        const float r = fmaf(s, f, __uint_as_float(__float_as_uint(s) & keep));
        return r != r ? s + poison : r;
    }
};

// The decay of a state chunk by chunk, one product an entry.  g^n rounded to 24
// bits would err the same way in every chunk of a long sequence; here each
// chunk's factor also makes up for the rounding of those before it, so that the
// product of all of them is right to 24 bits.
struct LinDecays {
    double exact, back, owed; // g^Q, 1 / g^Q, what the product of the factors so far lacks
    __device__ __forceinline__ LinDecays(float ld, int n) : exact(power(ld, n)), owed(1.0) { back = exact > 1e-30 ? 1.0 / exact : 0.0; }
    static __device__ __forceinline__ double power(float ld, int n) {
        const float x = ld * float(n); // n is a power of two, or the last chunk's
        return x > -0.5f ? 1.0 + double(expm1f(x)) : double(expf(x));
    }
    __device__ __forceinline__ float next() {
        const double t = owed * exact;
        const float f = float(t);
        owed = fma(t - double(f), back, 1.0);
        return f;
    }
    __device__ __forceinline__ float last(float ld, int n) const { return float(owed * power(ld, n)); }
};

// Zeroes a gradient's rows of tokens outside every sequence (the fp32 parts of
// a shared row are left to their sum).
template <typename IO>
__device__ __forceinline__ void lin_tail(const LinParams &p, const LinRole &R, int64_t wg) {
    if (R.out32) return;
    const int64_t lo = lin_start(p, 0), hi = lin_start(p, p.batch);
    const int64_t n = lo + (p.tokens > hi ? p.tokens - hi : 0);
    const int u = R.dz / 8, units = p.H * u;
    const float zero[4] = {};
    for (int64_t i = wg; i < n; i += p.tail) {
        IO *o = static_cast<IO *>(R.out) + (i < lo ? i : hi + (i - lo)) * R.ot;
        for (int e = threadIdx.x; e < units; e += blockDim.x) {
            IO *c = o + (e / u) * R.oh + e % u * 8;
            io<IO>::store4(c, zero);
            io<IO>::store4(c + 4, zero);
        }
    }
}

// The launch's parameters where the kernel's arguments lie, for an index known
// at run time: taken from the argument itself, the compiler copies it first.
__device__ __forceinline__ const LinParams &lin_args() {
    return *reinterpret_cast<const LinParams *>((const void *)__builtin_amdgcn_kernarg_segment_ptr());
}

// The scan.  OUT: outputs (and the final state); otherwise only the state that
// a segment's own rows leave, for the slot of the next segment.  UP: planes of
// the weighted y that join the state; three keep it to fp32 accuracy, two (2^-17)
// do where it is only rounded to bf16 and never handed out: in the gradients.  A
// prompt takes three whether its final state is asked for or not, so that its
// outputs are the same bits.
template <typename IO, int DX, int DZ, bool OUT, int UP>
__global__ __launch_bounds__((LinCfg<IO, DX, DZ, OUT>::T), (LinCfg<IO, DX, DZ, OUT>::WAVES)) void k_linear_scan(const LinParams p) {
    typedef LinCfg<IO, DX, DZ, OUT> C;
    constexpr int PL = C::PL, Q = C::Q, KS = C::KS;
    extern __shared__ __align__(16) uint16_t lds[];
    uint16_t *const xs = lds + C::XO, *const ys = lds + C::YO, *const zs = lds + C::ZO, *const sf = lds + C::SO;

    // Workgroups that share rows (the scans, column tiles and heads of a group)
    // follow each other on one XCD, whose L2 they share; ids go round the eight
    // XCDs, and so do the groups: segments and heads differ in work.
    const bool tail = OUT && blockIdx.x >= uint32_t(p.nwork);
    uint32_t id = tail ? blockIdx.x - p.nwork : blockIdx.x / 8 % uint32_t(p.group);
    const LinRole &R = lin_args().role[id % uint32_t(p.nroles)];
    id /= uint32_t(p.nroles);
    if (tail) {
        lin_tail<IO>(p, R, id);
        return;
    }
    const uint32_t unit = blockIdx.x / 8 / uint32_t(p.group) * 8 + blockIdx.x % 8, units = uint32_t(p.H / p.hg);
    const int z0 = int(id % uint32_t(p.ztiles)) * DZ;
    const int h = int(unit % units * p.hg + id / uint32_t(p.ztiles));
    const int64_t slot = unit / units;
    if (slot >= p.nseg) return;
    if (z0 >= R.dz) return;

    // the sequence of the slot, and the rows [pos, pos1) of it in scan order
    int64_t b = slot, pos = 0;
    if (p.segbits) {
        int64_t lo = 0, hi = p.batch - 1;
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) >> 1;
            if (lin_first_slot(p, mid) <= slot) lo = mid;
            else hi = mid - 1;
        }
        b = lo;
        pos = (slot - lin_first_slot(p, b)) << p.segbits;
    }
    const int64_t start = lin_start(p, b), next = lin_start(p, b + 1);
    const int64_t len = next > start ? next - start : 0;
    if (pos < 0 || (pos > 0 && pos >= len)) return;          // a slot without a segment
    const bool first = pos == 0;
    int64_t pos1 = len;
    if (p.segbits && pos + (int64_t(1) << p.segbits) < len) pos1 = pos + (int64_t(1) << p.segbits);
    const bool last = pos1 == len;
    if (!OUT && last) return;                                // nothing starts behind it
    const float ld = p.log_decay[h];
    const int64_t pool = lin_slot(p.slots, p.nstates, b);
    if (pool == kSlotSkip) return;

    // the wave's number as a scalar: matrix instructions ignore the lane mask, so
    // what only some waves do has to be branched around
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63, r16 = lane & 15, g = lane >> 4;
    if (pool == kSlotTaken) {
        if (OUT)
            for (int64_t e = tid; e < (pos1 - pos) * DZ; e += C::T)
                if (z0 + int(e % DZ) < R.dz)
                    io<IO>::put(static_cast<IO *>(R.out) + (start + pos + e / DZ) * R.ot + h * R.oh + z0 + e % DZ, __builtin_nanf(""));
        return;
    }
    const int64_t t0 = R.rev ? start + len - 1 - pos : start + pos; // token of the first row
    LinRows<IO, Q, DX, C::T> xr, yr;
    LinRows<IO, Q, DZ, C::T> zr;
    if (OUT) xr.init(R.x, t0, R.xt, (h / R.xg) * R.xh, R.dx, R.rev);
    yr.init(R.y, t0, R.yt, (h / R.yg) * R.yh, R.dx, R.rev);
    zr.init(R.z, t0, R.zt, (h / R.zg) * R.zh + z0, R.dz - z0, R.rev);
    LinRegs<IO, Q, DX, C::T> xq, yq; // the next chunk's rows, on their way
    LinRegs<IO, Q, DZ, C::T> zq;
    int left = int(pos1 - pos); // rows to go
    auto load = [&]() __attribute__((always_inline)) {
        if (left <= 0) return;
        const int rows = left < Q ? left : Q;
        if (OUT) xr.load(xq, rows);
        yr.load(yq, rows);
        zr.load(zq, rows);
    };
    load();

    const int es = R.rev ? 0 : 1;
    const float ld2 = ld * 1.44269504f;

    // This wave's tiles of the state, mt0 on along x and first on (round the end)
    // along z, and of the output, row tile rt and the tiles along z that start
    // alike: which of them a loop over all z tiles meets is then known when it is
    // unrolled.  State tile (i, j), register v, is
    // S[sm0 + 4 i + v][z0 + 16 ((first + j) % NT) + r16].
    constexpr int NT = 2 * C::NP;
    const int mt0 = w % C::MW * C::MTW, rt = w % C::RW;
    const int first_tile = C::NW > 1 ? w / C::MW * C::NTW : w / C::RW * C::NOT;
    auto tile = [&](int j) __attribute__((always_inline)) { return (first_tile + j) & (NT - 1); };
    floatx4 S[C::MTW][C::NTW];
    const int sm0 = 32 * (mt0 >> 1) + 8 * g + 4 * (mt0 & 1);
    const int dx = R.dx, dz = R.dz - z0;
    const uint32_t sm = R.sm, sn = R.sn, area = uint32_t(R.dx * R.dz);
    // every entry of this wave's tiles, with its index in an area (kNowhere / 4: none)
    auto each = [&](auto &&f) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < C::NTW; ++j) {
            const int n = 16 * tile(j) + r16;
            const uint32_t at = sm0 * sm + (z0 + n) * sn;
#pragma unroll
            for (int i = 0; i < C::MTW; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    S[i][j][v] = f(S[i][j][v], sm0 + 4 * i + v < dx && n < dz ? at + (4 * i + v) * sm : kNowhere / 4);
        }
    };
    // The state to start from.  A sequence that is not cut has it in its pool; of a
    // cut one the first segment's pass takes it along and leaves a copy in the
    // first slot, so that the last segment's may write the pool.  The slots behind
    // hold what the segments left, each without those before it where they are
    // still to be folded.
    const bool cut = p.segbits && !(first && last);
    const int64_t seg_at = ((lin_state_slot(p, b, start) + (pos >> p.segbits)) * p.H + h) * int64_t(area);
    if (OUT && cut && (!first || R.init)) {
        const int64_t from = OUT && p.fold && !first ? (pos >> p.segbits) - 1 : 0; // slots before this one to fold in
        LinBuf s0(R.seg + seg_at - from * p.H * int64_t(area), area * 4);
        each([&](float, uint32_t at) { return s0.get(4 * at); });
        const LinDecay d(ld, double(int64_t(1) << p.segbits));
        for (int64_t i = from - 1; i >= 0; --i) {
            const LinBuf s(R.seg + seg_at - i * p.H * int64_t(area), area * 4);
            each([&](float v, uint32_t at) { return d(v) + s.get(4 * at); });
        }
    } else if (R.init && first) {
        const int64_t at0 = (pool * p.H + h) * int64_t(area);
        if (R.init16) {
            const LinBuf s(static_cast<const bf16 *>(R.init) + at0, area * 2);
            each([&](float, uint32_t at) { return s.get16(2 * at); });
        } else {
            const LinBuf s(static_cast<const float *>(R.init) + at0, area * 4);
            each([&](float, uint32_t at) { return s.get(4 * at); });
        }
        if (!OUT) {
            const LinBuf s(R.seg + seg_at, area * 4);
            each([&](float v, uint32_t at) { s.put(4 * at, v); return v; });
        }
    } else {
        each([](float, uint32_t) { return 0.f; });
    }

    // decay factors, the same in every chunk: of row j = 16 t + 4 g + v in row
    // i = 16 rt + r16, and at the chunk's end.  No factor is a quotient: g^n may
    // be zero.
    float inner[2 * KS][4], weight[2 * KS][4];
    uint32_t upto[2] = {}; // in tile rt, the rows up to i, as masks of pairs of bf16 weights
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        const float diag = R.a_in * lin_power(ld2, r16 - 4 * g - v);
        upto[v >> 1] |= 4 * g + v <= r16 ? 0xffffu << 16 * (v & 1) : 0u;
        const float over = R.a_in * lin_power(ld2, 16 + r16 - 4 * g - v), end = R.a_state * lin_power(ld2, 16 - es - 4 * g - v);
#pragma unroll
        for (int t = 0; t < 2 * KS; ++t) {
            inner[t][v] = t < rt ? over * lin_power(ld2, 16 * (rt - 1 - t)) : diag;
            weight[t][v] = end * lin_power(ld2, 16 * (2 * KS - 1 - t));
        }
    }
    float from_start = R.a_init * lin_power(ld2, 16 * rt + r16 + es);
    LinDecays decays(ld, Q);
    char *out = static_cast<char *>(R.out);
    const int osize = C::F32 || R.out32 ? 4 : 2;
    const uint32_t ostep = uint32_t(R.ot) * osize;
    const uint32_t oat = uint32_t(R.rev ? Q - 1 - (16 * rt + r16) : 16 * rt + r16) * ostep + (osize == 4 ? 16 * g : 32 * (g & 1) + 16 * (g >> 1));
    const bool rev = R.rev;
    out += (t0 * R.ot + h * R.oh + z0) * osize;

    while (left > 0) {
        const int rows = left < Q ? left : Q;
        left -= rows;
        float decay;
        if (rows == Q) {
            decay = decays.next();
        } else { // the last one
            decay = decays.last(ld, rows);
            const int i = 16 * rt + r16 - (Q - rows);
            from_start = i >= 0 ? R.a_init * lin_power(ld2, i + es) : 0.f;
        }
        if (OUT) xq.template stage<C::XP>(xs);
        yq.template stage<C::XP>(ys);
        zq.template stage<C::ZP>(zs);
        if (OUT) {
#pragma unroll
            for (int j = 0; j < C::NTW; ++j) {
                // a bf16 result takes the state rounded to bf16 as operand: one
                // rounding per term, the size of the result's own, and a relative
                // error of 0.0022 where the result's rounding alone makes 0.0017.
                // A second plane would make it that, but leaves one workgroup a unit
                // at 128 x 128: 16 ragged sequences of 1024 x 32 x 128 207 -> 270 us,
                // gradients of 4 x 2048 x 64 x 64 144 -> 158
                uint16_t *const f = sf + (((mt0 >> 1) * NT + tile(j)) * 64 + lane) * 8;
                float a[8];
#pragma unroll
                for (int v = 0; v < 8; ++v) a[v] = v < 4 * C::MTW ? S[(v >> 2) % C::MTW][j][v & 3] : 0.f;
                const lfrag<PL> q = lsplit<PL>(a);
#pragma unroll
                for (int k = 0; k < PL; ++k) {
                    const uint4 u = __builtin_bit_cast(uint4, q.v[k]);
                    if (C::MTW == 2) *reinterpret_cast<uint4 *>(f + k * C::SP) = u;
                    else *reinterpret_cast<uint2 *>(f + k * C::SP + 4 * (mt0 & 1)) = make_uint2(u.x, u.y);
                }
            }
        }
        __syncthreads();
        load();

        floatx4 O[C::NOT]; // out^T, tile j: channel z0 + 16 tile(j) + 4 g + v of row 16 rt + r16
        lfrag<C::WP> pf[KS]; // weights of the chunk's rows in row 16 rt + r16
        if (OUT) {
            lfrag<PL> xf[C::MP];
#pragma unroll
            for (int m = 0; m < C::MP; ++m) xf[m] = lin_row<PL, DX, C::XP>(xs, 16 * rt + r16, 4 * m + g);
            // the weights, also of the rows behind row i, which are cleared as bits:
            // whatever they are, they must not reach it
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                floatx4 a[2] = {};
#pragma unroll
                for (int m = 0; m < C::MP; ++m)
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        a[u] = lmma(a[u], lin_row<PL, DX, C::XP>(ys, 32 * s + 16 * u + r16, 4 * m + g), xf[m]);
                float pr[8];
#pragma unroll
                for (int v = 0; v < 8; ++v) pr[v] = a[v >> 2][v & 3] * inner[2 * s + (v >> 2)][v & 3];
                pf[s] = lsplit<C::WP>(pr);
                const uint32_t at0 = 2 * s == rt ? ~0u : 0u, all0 = 2 * s < rt ? ~0u : 0u, at1 = 2 * s + 1 == rt ? ~0u : 0u, all1 = 2 * s + 1 < rt ? ~0u : 0u;
#pragma unroll
                for (int k = 0; k < C::WP; ++k) {
                    const uint4 u = __builtin_bit_cast(uint4, pf[s].v[k]);
                    pf[s].v[k] = bf16x8_from_words(u.x & ((upto[0] & at0) | all0), u.y & ((upto[1] & at0) | all0),
                                                   u.z & ((upto[0] & at1) | all1), u.w & ((upto[1] & at1) | all1));
                }
            }
#pragma unroll
            for (int j = 0; j < C::NOT; ++j) O[j] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int m = 0; m < C::MP; ++m)
#pragma unroll
                for (int j = 0; j < C::NOT; ++j) {
                    lfrag<PL> f;
#pragma unroll
                    for (int k = 0; k < PL; ++k)
                        f.v[k] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4 *>(
                            sf + k * C::SP + ((m * NT + tile(j)) * 64 + lane) * 8));
                    O[j] = lmma(O[j], f, xf[m]);
                }
#pragma unroll
            for (int j = 0; j < C::NOT; ++j) O[j] *= from_start;
        }
#pragma unroll
        for (int i = 0; i < C::MTW; ++i)
#pragma unroll
            for (int j = 0; j < C::NTW; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v) S[i][j][v] *= decay;
        // the rows join the output, and, weighted by what is left of them at the
        // chunk's end, in UP planes, the state
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            lfrag<UP> yf[C::MTW];
#pragma unroll
            for (int i = 0; i < C::MTW; ++i) {
                float a[8];
                lunsplit(lin_ycol<PL, DX, C::XP>(ys, 2 * s, mt0 + i, r16, g), a);
#pragma unroll
                for (int k = 0; k < 8; ++k) a[k] *= weight[2 * s + (k >> 2)][k & 3];
                yf[i] = lsplit<UP>(a);
            }
            // a few tiles of z at a time: the products of one plane over all of
            // them, so that no product waits for the one before it
            constexpr int NB = NT < 4 ? NT : 4;
#pragma unroll
            for (int j0 = 0; j0 < NT; j0 += NB) {
                if (j0 >= C::NTW && (!OUT || j0 >= C::NOT)) continue;
                lfrag<PL> zf[NB];
#pragma unroll
                for (int q = 0; q < NB; ++q)
                    if (j0 + q < C::NTW || (OUT && j0 + q < C::NOT)) zf[q] = lin_zcol<PL, DZ, C::ZP>(zs, 2 * s, tile(j0 + q), r16, g);
                if (OUT)
                    lpairs<PL, C::WP>([&](auto a, auto b) {
#pragma unroll
                        for (int q = 0; q < NB; ++q)
                            if (j0 + q < C::NOT)
                                O[(j0 + q) % C::NOT] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(zf[q].v[a.value], pf[s].v[b.value], O[(j0 + q) % C::NOT], 0, 0, 0);
                    });
                lpairs<UP, PL>([&](auto a, auto b) {
#pragma unroll
                    for (int q = 0; q < NB; ++q)
                        if (j0 + q < C::NTW)
#pragma unroll
                            for (int i = 0; i < C::MTW; ++i) {
                                floatx4 &o = S[i][(j0 + q) % C::NTW];
                                o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(yf[i].v[a.value], zf[q].v[b.value], o, 0, 0, 0);
                            }
                });
            }
        }
        if (OUT) {
            const LinBuf o(out - (rev ? uint32_t(rows - 1) * ostep : 0u), uint32_t(rows) * ostep);
            out += rev ? -int64_t(Q) * ostep : int64_t(Q) * ostep;
            const uint32_t at = oat - (rev ? 0u : uint32_t(Q - rows) * ostep);
            if (osize == 4) {
#pragma unroll
                for (int j = 0; j < C::NOT; ++j)
                    o.store(16 * tile(j) + 4 * g < dz ? at + 64 * tile(j) : kNowhere, __builtin_bit_cast(uint4, O[j]));
            } else if constexpr (!C::F32) {
                // lanes of neighbouring groups swap halves of two tiles: eight
                // neighbouring channels each
                if (C::NOT == 2 && C::NTW == 1 && first_tile) { // the one shape whose tiles may start at an odd one
                    const floatx4 a = O[0];
                    O[0] = O[1 % C::NOT];
                    O[1 % C::NOT] = a;
                }
#pragma unroll
                for (int j = 0; j < C::NOT; j += 2) {
                    const int n = tile(j) & ~1;
                    const auto a = __builtin_amdgcn_permlane16_swap(pack2_bf16(O[j][0], O[j][1]), pack2_bf16(O[j + 1][0], O[j + 1][1]), false, false);
                    const auto b = __builtin_amdgcn_permlane16_swap(pack2_bf16(O[j][2], O[j][3]), pack2_bf16(O[j + 1][2], O[j + 1][3]), false, false);
                    o.store(16 * n + 16 * (g & 1) + 8 * (g >> 1) < dz ? at + 32 * n : kNowhere, make_uint4(a[0], b[0], a[1], b[1]));
                }
            }
        }
        __syncthreads();
    }

    if (OUT && (!last || !R.fin)) return;
    if (OUT && R.fin16) {
        const LinBuf s(static_cast<bf16 *>(R.fin) + (pool * p.H + h) * int64_t(area), area * 2);
        each([&](float v, uint32_t at) { s.put16(2 * at, v); return v; });
    } else {
        const LinBuf s((OUT ? static_cast<float *>(R.fin) + (pool * p.H + h) * int64_t(area) : R.seg + seg_at + p.H * int64_t(area)),
                       area * 4);
        each([&](float v, uint32_t at) { s.put(4 * at, v); return v; });
    }
}

template <typename IO, int DX, int DZ, bool OUT, int UP>
hipError_t launch_linear_planes(const LinParams &p, hipStream_t s) {
    typedef LinCfg<IO, DX, DZ, OUT> C;
    if (C::bytes > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(&k_linear_scan<IO, DX, DZ, OUT, UP>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, int(C::bytes));
        if (e != hipSuccess) return e;
    }
    const int64_t grid = int64_t(p.nwork) + (OUT ? p.tail * p.nroles : 0);
    if (grid == 0) return hipSuccess;
    hipLaunchKernelGGL((k_linear_scan<IO, DX, DZ, OUT, UP>), dim3(unsigned(grid)), dim3(C::T), C::bytes, s, p);
    return hipGetLastError();
}

template <typename IO, int DX, int DZ, bool OUT>
hipError_t launch_linear_inst(const LinParams &p, hipStream_t s) {
    // gradients of 4 x 2048 x 64 x 64: 144 us with two planes, 153 with three
    if constexpr (OUT && !std::is_same<IO, float>::value) {
        bool three = !p.grad;
        for (int i = 0; i < p.nroles; ++i) three |= p.role[i].fin != nullptr;
        if (!three) return launch_linear_planes<IO, DX, DZ, OUT, 2>(p, s);
    }
    return launch_linear_planes<IO, DX, DZ, OUT, 3>(p, s);
}

// The compiled tile of a size: 32, 64 or 128 channels.
constexpr int lin_tile(int d) { return d <= 32 ? 32 : d <= 64 ? 64 : 128; }

// Launches with the tiles dx x dz (each 32, 64 or 128; dz at most 64 with fp32 I/O).
template <typename IO, int DX>
hipError_t launch_linear_dx(const LinParams &p, int dz, bool out, hipStream_t s) {
    switch (dz) {
    case 32: return out ? launch_linear_inst<IO, DX, 32, true>(p, s) : launch_linear_inst<IO, DX, 32, false>(p, s);
    case 64: return out ? launch_linear_inst<IO, DX, 64, true>(p, s) : launch_linear_inst<IO, DX, 64, false>(p, s);
    case 128:
        if constexpr (!std::is_same<IO, float>::value)
            return out ? launch_linear_inst<IO, DX, 128, true>(p, s) : launch_linear_inst<IO, DX, 128, false>(p, s);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_linear_bf16_32(const LinParams &p, int dz, bool out, hipStream_t s);
hipError_t launch_linear_bf16_64(const LinParams &p, int dz, bool out, hipStream_t s);
hipError_t launch_linear_bf16_128(const LinParams &p, int dz, bool out, hipStream_t s);
hipError_t launch_linear_f32_32(const LinParams &p, int dz, bool out, hipStream_t s);
hipError_t launch_linear_f32_64(const LinParams &p, int dz, bool out, hipStream_t s);
hipError_t launch_linear_f32_128(const LinParams &p, int dz, bool out, hipStream_t s);

} // namespace m3

// k_linear.hpp -- linear attention with a decay for each head: the chunked
// scan that serves the prompt pass and, with its operands exchanged or the
// tokens walked backwards, the three gradients; the join of a cut sequence's
// segment states; the sum of a shared row's gradients.
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
    float *seg;              // [segment slot][H][dx dz] fp32: state at the start of each segment
};

struct LinParams {
    LinRole role[3];
    int32_t nroles, H, ztiles;
    int32_t tail;            // extra workgroups per scan that zero the rows outside every sequence
    int64_t batch, tokens, nwork; // nwork: workgroups without the tail
    const int32_t *cu;       // null: equal sequences
    const int32_t *slots;    // null: sequence b has state b
    int64_t nstates;
    const float *log_decay;
    int64_t seglen;          // tokens per segment, 0: sequences are not cut
    int64_t nseg;            // segment slots (batch when not cut)
};

// First token of sequence b, clamped to the rows there are.
__device__ __forceinline__ int64_t lin_start(const LinParams &p, int64_t b) {
    if (!p.cu) return b * (p.tokens / p.batch);
    const int64_t c = p.cu[b];
    return c < 0 ? 0 : c > p.tokens ? p.tokens : c;
}

constexpr int64_t kSlotSkip = -1, kSlotTaken = -2;

// State of sequence b: its slot, kSlotSkip for padding, kSlotTaken where an
// earlier sequence of the call names the same slot.  All threads of the
// workgroup call it.
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
__device__ __forceinline__ int64_t lin_first_slot(const LinParams &p, int64_t b) { return lin_start(p, b) / p.seglen + b; }

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
    for (int i = 0; i < 8; ++i) a[i] = 0.f;
#pragma unroll
    for (int k = PL - 1; k >= 0; --k) {
        const uint4 w = __builtin_bit_cast(uint4, f.v[k]);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[2 * i] += __uint_as_float(ws[i] << 16);
            a[2 * i + 1] += __uint_as_float(ws[i] & 0xffff0000u);
        }
    }
}

// ---------------------------------------------------------------------------
// Tile of one scan.  Q rows per chunk, DX x DZ state columns of a workgroup of
// four waves; z columns beyond DZ are another workgroup's.
// ---------------------------------------------------------------------------
constexpr int kLT = 256; // threads

template <typename IO, int DX, int DZ, bool OUT>
struct LinCfg {
    static constexpr bool F32 = std::is_same<IO, float>::value;
    static constexpr int PL = F32 ? 3 : 1;
    static constexpr int Q = F32 ? 32 : 64;
    static constexpr int MP = DX / 32, NP = DZ / 32; // 32 x 32 blocks of the state
    // the state's blocks over the four waves: MW along x, the rest along z
    static constexpr int MW = MP < 4 ? MP : 4, NW = 4 / MW, NPW = (NP + NW - 1) / NW;
    // the output's 16-row tiles over the waves: RW along the rows, the rest along z
    static constexpr int RW = Q / 16, OW = 4 / RW, NPO = (NP + OW - 1) / OW;
    static constexpr int KS = Q / 32; // 32-row steps of a product over the chunk's rows
    // LDS, in bf16 elements: x, y, z planes and the state's fragments
    static constexpr int XP = Q * DX, ZP = Q * DZ, SP = DX * DZ;
    static constexpr int XO = 0, YO = OUT ? PL * XP : 0, ZO = YO + PL * XP, SO = ZO + PL * ZP;
    static constexpr size_t bytes = 2 * size_t(SO + (OUT ? PL * SP : 0));
};

// 16-byte units of a staged row are permuted by the row, so that 16 rows at
// one unit (row reads) and four rows at four neighbouring units (transposing
// reads) both touch every bank once.
template <int D>
__device__ __forceinline__ int lin_at(int row, int unit) {
    constexpr int U = D / 8;
    const int f = ((row & 3) << 2 | (row >> 2 & 3));
    const int h = U >= 16 ? f : U == 8 ? (((f >> 3) << 2) | (f & 3)) : (f & 3);
    return row * D + ((unit ^ h) << 3);
}

// Eight k-slots of one column of a staged matrix: rows 16 t0 + 4 g + v, then
// 16 (t0 + 1) + 4 g + v.  Lane r of a group gets column
// 32 blk + 8 (r / 4) + r % 4 + 4 half.
template <int PL, int D, int PS>
__device__ __forceinline__ lfrag<PL> lin_col(const uint16_t *m, int t0, int blk, int half, int r16, int g) {
    const int row = 16 * t0 + 4 * g + (r16 >> 2), unit = 4 * blk + (r16 & 3);
    const uint16_t *p0 = m + lin_at<D>(row, unit) + 4 * half;
    const uint16_t *p1 = m + lin_at<D>(row + 16, unit) + 4 * half;
    lfrag<PL> f;
#pragma unroll
    for (int k = 0; k < PL; ++k) {
        const uint2 a = lds_tr4(p0 + k * PS), b = lds_tr4(p1 + k * PS);
        f.v[k] = bf16x8_from_words(a.x, a.y, b.x, b.y);
    }
    return f;
}
template <int PL, int D, int PS>
__device__ __forceinline__ lfrag<PL> lin_row(const uint16_t *m, int row, int unit) {
    const uint16_t *p = m + lin_at<D>(row, unit);
    lfrag<PL> f;
#pragma unroll
    for (int k = 0; k < PL; ++k) f.v[k] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4 *>(p + k * PS));
    return f;
}

// Eight consecutive elements as loaded.
template <typename IO>
struct lraw;
template <>
struct lraw<bf16> {
    uint4 a;
    __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const bf16 *p) { a = ld16(p); }
    template <int PS>
    __device__ __forceinline__ void stage(uint16_t *p) const { *reinterpret_cast<uint4 *>(p) = a; }
};
template <>
struct lraw<float> {
    uint4 a, b;
    __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const float *p) { a = ld16(p); b = ld16(p + 4); }
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
template <typename IO, int Q, int D>
struct LinRows {
    static constexpr int U = D / 8, PIECES = Q * U, N = (PIECES + kLT - 1) / kLT;
    lraw<IO> r[N];
    // base: row 0 of the chunk; step: elements from one row to the next
    __device__ __forceinline__ void load(const IO *base, int64_t step, int rows, int dim) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int piece = threadIdx.x + i * kLT, row = piece / U, unit = piece % U;
            r[i].zero();
            if (row < rows && unit * 8 < dim) r[i].load(base + row * step + unit * 8);
        }
    }
    template <int PS>
    __device__ __forceinline__ void stage(uint16_t *m) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int piece = threadIdx.x + i * kLT;
            if (PIECES % kLT == 0 || piece < PIECES) r[i].template stage<PS>(m + lin_at<D>(piece / U, piece % U));
        }
    }
};

// g^n for n >= 0 rows; g = 0 (log_decay = -inf) keeps the row itself.
__device__ __forceinline__ float lin_power(float ld, int n) { return n > 0 ? expf(ld * float(n)) : 1.f; }

// s g^n.  A slow decay is applied as s + s (g^n - 1): rounding g^n itself to
// 24 bits would err the same way in every chunk of a long sequence.
struct LinDecay {
    float f;
    bool slow;
    __device__ __forceinline__ LinDecay(float ld, double n) {
        const float x = n > 0 ? float(double(ld) * n) : 0.f;
        slow = x > -0.5f;
        f = slow ? expm1f(x) : expf(x);
    }
    __device__ __forceinline__ float operator()(float s) const { return slow ? fmaf(s, f, s) : s * f; }
};

// Workgroup id -> work item, so that neighbouring items run on one XCD (ids go
// round the eight XCDs) and share its L2: the scans of one head and segment,
// and heads that share rows.
__device__ __forceinline__ int64_t lin_xcd(int64_t id, int64_t n) {
    const int64_t q = n / 8, r = n % 8, x = id % 8;
    return x * q + (x < r ? x : r) + id / 8;
}

// Zeroes a gradient's rows of tokens outside every sequence (the fp32 parts of
// a shared row are left to their sum).
template <typename IO>
__device__ __forceinline__ void lin_tail(const LinParams &p, const LinRole &R, int64_t wg) {
    if (R.out32) return;
    const int64_t lo = lin_start(p, 0), hi = lin_start(p, p.batch);
    const int64_t n = lo + (p.tokens > hi ? p.tokens - hi : 0);
    for (int64_t i = wg; i < n; i += p.tail) {
        IO *o = static_cast<IO *>(R.out) + (i < lo ? i : hi + (i - lo)) * R.ot;
        for (int e = threadIdx.x; e < p.H * R.dz; e += kLT) io<IO>::put(o + (e / R.dz) * R.oh + e % R.dz, 0.f);
    }
}

// The scan.  OUT: outputs (and the final state); otherwise only the state that
// a segment's own rows leave, for the slot of the next segment.
template <typename IO, int DX, int DZ, bool OUT>
__global__ __launch_bounds__(kLT) void k_linear_scan(const LinParams p) {
    typedef LinCfg<IO, DX, DZ, OUT> C;
    constexpr int PL = C::PL, Q = C::Q, KS = C::KS;
    extern __shared__ __align__(16) uint16_t lds[];
    uint16_t *const xs = lds + C::XO, *const ys = lds + C::YO, *const zs = lds + C::ZO, *const sf = lds + C::SO;

    const bool tail = OUT && int64_t(blockIdx.x) >= p.nwork;
    int64_t id = tail ? int64_t(blockIdx.x) - p.nwork : lin_xcd(blockIdx.x, p.nwork);
    const LinRole R = p.role[id % p.nroles];
    id /= p.nroles;
    if (tail) {
        lin_tail<IO>(p, R, id);
        return;
    }
    const int z0 = int(id % p.ztiles) * DZ;
    id /= p.ztiles;
    const int h = int(id % p.H);
    const int64_t slot = id / p.H;
    if (z0 >= R.dz) return;

    // the sequence of the slot, and the rows [pos, pos1) of it in scan order
    int64_t b = slot, pos = 0;
    if (p.seglen) {
        int64_t lo = 0, hi = p.batch - 1;
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) / 2;
            if (lin_first_slot(p, mid) <= slot) lo = mid;
            else hi = mid - 1;
        }
        b = lo;
        pos = (slot - lin_first_slot(p, b)) * p.seglen;
    }
    const int64_t start = lin_start(p, b), next = lin_start(p, b + 1);
    const int64_t len = next > start ? next - start : 0;
    if (pos < 0 || (pos > 0 && pos >= len)) return;          // a slot without a segment
    const bool first = pos == 0;
    int64_t pos1 = len;
    if (p.seglen && pos + p.seglen < len) pos1 = pos + p.seglen;
    const bool last = pos1 == len;
    if (!OUT && last) return;                                // nothing starts behind it
    const int64_t pool = lin_slot(p.slots, p.nstates, b);
    if (pool == kSlotSkip) return;

    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, r16 = lane & 15, g = lane >> 4;
    if (pool == kSlotTaken) {
        if (OUT)
            for (int64_t e = tid; e < (pos1 - pos) * DZ; e += kLT)
                if (z0 + int(e % DZ) < R.dz)
                    io<IO>::put(static_cast<IO *>(R.out) + (start + pos + e / DZ) * R.ot + h * R.oh + z0 + e % DZ, __builtin_nanf(""));
        return;
    }
    const int es = R.rev ? 0 : 1;
    const float ld = p.log_decay[h];

    // state: block (m, np) of this wave, fragment (mt, nt), register v is
    // S[32 m + 8 g + 4 mt + v][z0 + 32 np + 8 (r16 / 4) + r16 % 4 + 4 nt]
    const int mp = w % C::MW, np0 = (w / C::MW) * C::NPW;
    floatx4 S[C::NPW][2][2];
    const int sm0 = 32 * mp + 8 * g, sn0 = z0 + 8 * (r16 >> 2) + (r16 & 3);
    const int64_t area = int64_t(R.dx) * R.dz;
    auto each = [&](auto &&f) {
#pragma unroll
        for (int i = 0; i < C::NPW; ++i)
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const int m = sm0 + 4 * mt + v, n = sn0 + 32 * (np0 + i) + 4 * nt;
                        S[i][mt][nt][v] = f(S[i][mt][nt][v], np0 + i < C::NP && m < R.dx && n < R.dz, m * R.sm + n * R.sn);
                    }
    };
    bool live = false; // the state is not zero as a whole
    if (OUT && (p.seglen ? !first || R.init : R.init != nullptr)) {
        live = true;
        if (p.seglen) {
            const float *s = R.seg + (slot * p.H + h) * area;
            each([&](float, bool in, int at) { return in ? s[at] : 0.f; });
        } else if (R.init16) {
            const bf16 *s = static_cast<const bf16 *>(R.init) + (pool * p.H + h) * area;
            each([&](float, bool in, int at) { return in ? bits_to_f32(s[at].bits) : 0.f; });
        } else {
            const float *s = static_cast<const float *>(R.init) + (pool * p.H + h) * area;
            each([&](float, bool in, int at) { return in ? s[at] : 0.f; });
        }
    } else {
        each([](float, bool, int) { return 0.f; });
    }

    // decay factors that every full chunk shares
    const int rt = w % C::RW, no0 = (w / C::RW) * C::NPO;   // this wave's output rows and columns
    float inner[2 * KS][4], from_start = 0.f;               // rows j = 16 t + 4 g + v seen from row i = 16 rt + r16
    if (OUT) {
#pragma unroll
        for (int t = 0; t < 2 * KS; ++t)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int n = 16 * (rt - t) + r16 - 4 * g - v;
                inner[t][v] = n >= 0 ? R.a_in * lin_power(ld, n) : 0.f;
            }
        from_start = R.a_init * lin_power(ld, 16 * rt + r16 + es);
    }
    float weight[KS][8];                                    // rows 32 s + 16 (k / 4) + 4 g + k % 4 seen from the end
    auto weights = [&](int rows) {
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                weight[s][k] = R.a_state * lin_power(ld, rows - es - (32 * s + 16 * (k >> 2) + 4 * g + (k & 3)));
    };
    weights(Q);
    const LinDecay whole(ld, Q);

    const int64_t sgn = R.rev ? -1 : 1, t0 = R.rev ? start + len - 1 : start;
    const IO *xp = static_cast<const IO *>(R.x) + (t0 + sgn * pos) * R.xt + (h / R.xg) * R.xh;
    const IO *yp = static_cast<const IO *>(R.y) + (t0 + sgn * pos) * R.yt + (h / R.yg) * R.yh;
    const IO *zp = static_cast<const IO *>(R.z) + (t0 + sgn * pos) * R.zt + (h / R.zg) * R.zh + z0;
    LinRows<IO, Q, DX> xr, yr;
    LinRows<IO, Q, DZ> zr;
    auto load = [&]() {
        const int rows = int(pos1 - pos < Q ? pos1 - pos : Q);
        if (OUT) xr.load(xp, sgn * R.xt, rows, R.dx);
        yr.load(yp, sgn * R.yt, rows, R.dx);
        zr.load(zp, sgn * R.zt, rows, R.dz - z0);
        xp += sgn * Q * R.xt;
        yp += sgn * Q * R.yt;
        zp += sgn * Q * R.zt;
    };
    if (pos < pos1) load();
    while (pos < pos1) {
        const int rows = int(pos1 - pos < Q ? pos1 - pos : Q);
        const int64_t here = t0 + sgn * pos;
        pos += rows;
        if (OUT) xr.template stage<C::XP>(xs);
        yr.template stage<C::XP>(ys);
        zr.template stage<C::ZP>(zs);
        if (OUT && live) {
#pragma unroll
            for (int i = 0; i < C::NPW; ++i)
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    if (np0 + i >= C::NP) continue;
                    float a[8];
#pragma unroll
                    for (int v = 0; v < 8; ++v) a[v] = S[i][v >> 2][nt][v & 3];
                    // a bf16 result takes the state rounded to bf16 as operand: one
                    // rounding per term, the size of the result's own
                    const lfrag<PL> f = lsplit<PL>(a);
#pragma unroll
                    for (int k = 0; k < PL; ++k)
                        *reinterpret_cast<uint4 *>(sf + k * C::SP + (((mp * C::NP + np0 + i) * 2 + nt) * 64 + lane) * 8) =
                            __builtin_bit_cast(uint4, f.v[k]);
                }
        }
        __syncthreads();
        if (pos < pos1) load();

        if (OUT) {
            lfrag<PL> xf[C::MP];
#pragma unroll
            for (int m = 0; m < C::MP; ++m) xf[m] = lin_row<PL, DX, C::XP>(xs, 16 * rt + r16, 4 * m + g);
            // out^T, fragment nt: channel z0 + 32 np + 8 g + 4 nt + v of row 16 rt + r16
            floatx4 O[C::NPO][2];
#pragma unroll
            for (int i = 0; i < C::NPO; ++i) O[i][0] = O[i][1] = floatx4{0.f, 0.f, 0.f, 0.f};
            if (live) {
#pragma unroll
                for (int i = 0; i < C::NPO; ++i)
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        if (no0 + i >= C::NP) continue;
#pragma unroll
                        for (int m = 0; m < C::MP; ++m) {
                            lfrag<PL> f;
#pragma unroll
                            for (int k = 0; k < PL; ++k)
                                f.v[k] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4 *>(
                                    sf + k * C::SP + (((m * C::NP + no0 + i) * 2 + nt) * 64 + lane) * 8));
                            O[i][nt] = lmma(O[i][nt], f, xf[m]);
                        }
                        O[i][nt] *= from_start;
                    }
            }
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                if (2 * s > rt) continue; // rows behind this wave's
                float pr[8];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int t = 2 * s + u;
                    floatx4 a{0.f, 0.f, 0.f, 0.f};
                    if (t <= rt) {
#pragma unroll
                        for (int m = 0; m < C::MP; ++m)
                            a = lmma(a, lin_row<PL, DX, C::XP>(ys, 16 * t + r16, 4 * m + g), xf[m]);
                    }
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        pr[4 * u + v] = t < rt || (t == rt && 4 * g + v <= r16) ? a[v] * inner[t][v] : 0.f;
                }
                // the weights of a bf16 result are rounded to bf16, as above
                const lfrag<PL> pf = lsplit<PL>(pr);
#pragma unroll
                for (int i = 0; i < C::NPO; ++i)
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        if (no0 + i >= C::NP) continue;
                        O[i][nt] = lmma(O[i][nt], lin_col<PL, DZ, C::ZP>(zs, 2 * s, no0 + i, nt, r16, g), pf);
                    }
            }
            if (16 * rt + r16 < rows) {
                const int64_t at = (here + sgn * (16 * rt + r16)) * R.ot + h * R.oh + z0 + 8 * g;
#pragma unroll
                for (int i = 0; i < C::NPO; ++i) {
                    const int n = 32 * (no0 + i);
                    if (no0 + i >= C::NP || z0 + n + 8 * g >= R.dz) continue;
                    if (C::F32 || R.out32) {
                        float *o = static_cast<float *>(R.out) + at + n;
                        *reinterpret_cast<floatx4 *>(o) = O[i][0];
                        *reinterpret_cast<floatx4 *>(o + 4) = O[i][1];
                    } else {
                        bf16 *o = static_cast<bf16 *>(R.out) + at + n;
                        *reinterpret_cast<uint4 *>(o) =
                            make_uint4(pack2_bf16(O[i][0][0], O[i][0][1]), pack2_bf16(O[i][0][2], O[i][0][3]),
                                       pack2_bf16(O[i][1][0], O[i][1][1]), pack2_bf16(O[i][1][2], O[i][1][3]));
                    }
                }
            }
        }
        // the state behind the chunk, where anything reads it
        if (!OUT || pos < pos1 || (last && R.fin)) {
            if (rows < Q) weights(rows);
            if (live) {
                const LinDecay d = rows == Q ? whole : LinDecay(ld, rows);
                each([&](float v, bool, int) { return d(v); });
            }
            live = true;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                lfrag<3> yf[2];
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    float a[8];
                    lunsplit(lin_col<PL, DX, C::XP>(ys, 2 * s, mp, mt, r16, g), a);
#pragma unroll
                    for (int k = 0; k < 8; ++k) a[k] *= weight[s][k];
                    yf[mt] = lsplit<3>(a); // the state is kept to fp32 accuracy
                }
#pragma unroll
                for (int i = 0; i < C::NPW; ++i)
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        if (np0 + i >= C::NP) continue;
                        const lfrag<PL> zf = lin_col<PL, DZ, C::ZP>(zs, 2 * s, np0 + i, nt, r16, g);
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt) S[i][mt][nt] = lmma(S[i][mt][nt], yf[mt], zf);
                    }
            }
        }
        __syncthreads();
    }

    if (!OUT) {
        float *s = R.seg + ((slot + 1) * p.H + h) * area;
        each([&](float v, bool in, int at) { if (in) s[at] = v; return v; });
    } else if (last && R.fin) {
        if (R.fin16) {
            bf16 *s = static_cast<bf16 *>(R.fin) + (pool * p.H + h) * area;
            each([&](float v, bool in, int at) { if (in) s[at].bits = f32_to_bits(v); return v; });
        } else {
            float *s = static_cast<float *>(R.fin) + (pool * p.H + h) * area;
            each([&](float v, bool in, int at) { if (in) s[at] = v; return v; });
        }
    }
}

template <typename IO, int DX, int DZ, bool OUT>
hipError_t launch_linear_inst(const LinParams &p, hipStream_t s) {
    typedef LinCfg<IO, DX, DZ, OUT> C;
    if (C::bytes > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(&k_linear_scan<IO, DX, DZ, OUT>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, int(C::bytes));
        if (e != hipSuccess) return e;
    }
    const int64_t grid = p.nwork + (OUT ? p.tail * p.nroles : 0);
    if (grid == 0) return hipSuccess;
    hipLaunchKernelGGL((k_linear_scan<IO, DX, DZ, OUT>), dim3(unsigned(grid)), dim3(kLT), C::bytes, s, p);
    return hipGetLastError();
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

// m3_rotary.hip -- the norm of queries and keys for each head with the position
// rotation in the same pass, and its gradients (include/m3_rotary.h).
//
// A row of dim channels lies over LPR lanes, eight channels a lane, so a wave
// takes 64 / LPR rows at once, and the mean of squares is a sum over LPR lanes.
// A lane's channels are four rotation pairs whichever way the pairs lie, and
// they are the same pairs in every row: a wave takes up to kRows sets of rows
// of one token and forms the four angles' sine and cosine once for all of
// them.  Bound by reading and writing the rows: 16384 x 40 x 128 in bf16 54 us
// (6.2 TB/s); a few rows take 3 us, the time of a launch.
#include "m3_rotary.h"
#include "m3_device.hpp"

#include <algorithm>
#include <initializer_list>

namespace m3 {

constexpr int kRT = 256;   // threads, four waves
constexpr int kRows = 4;   // row sets per wave and token at most

struct RotRows {
    const void *x, *g;     // input rows; upstream gradient (backward)
    void *out;
    int64_t xt, xh, gt, gh, ot, oh;
    const float *w;
    int32_t heads, items;  // items: groups of kRows row sets
};
struct RotParams {
    RotRows r[2];          // q, k
    int64_t tokens;
    int32_t dim, rot, axes, pos64, norm;
    float eps, inv_dim;
    const void *pos;
    const float *freq;
    float *part;           // backward: [workgroup][dim] partial gradients of the weights
    int32_t split;         // backward: workgroups of q, the others are k's
};

// The channels and angles of one lane.  HALVES: pairs (i, i + rot / 2), across
// the two runs; else (2i, 2i + 1), and the runs are neighbours.
template <bool HALVES>
struct RotLane {
    int c0, c1;            // two runs of four channels
    bool in, turn;         // channels within the row; turned
    float cs[4], sn[4];

    __device__ __forceinline__ RotLane(const RotParams &p, int unit) {
        in = unit * 8 < p.dim;
        turn = unit * 8 < p.rot;
        c0 = HALVES && turn ? 4 * unit : 8 * unit;
        c1 = HALVES && turn ? p.rot / 2 + 4 * unit : 8 * unit + 4;
    }
    // Angles as fractions of a turn: far positions times fast frequencies lose
    // all of fp32.  position * frequency and its product with 1 / 2 pi are taken
    // as fp64 values with their remainders (fma), so that whole turns drop out
    // exactly and the rest is good to 2^-50 of a turn up to positions of 2^53.
    // It goes to the hardware's sine and cosine of turns (at most 1.3e-7 off).
    __device__ __forceinline__ void angles(const RotParams &p, int unit, int64_t token) {
#pragma clang fp contract(off) // u must be the rounded product where its remainder is added
        if (!turn) return;
        constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57; // 1 / 2 pi = kHi + kLo
        double a[4] = {};
        for (int x = 0; x < p.axes; ++x) {
            const int64_t i = x * p.tokens + token;
            const double t = p.pos64 ? double(static_cast<const int64_t *>(p.pos)[i]) : double(static_cast<const int32_t *>(p.pos)[i]);
            const float4 f = *reinterpret_cast<const float4 *>(p.freq + x * (p.rot / 2) + 4 * unit);
            const float fs[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const double m = t * double(fs[c]), u = m * kHi;
                const double rest = fma(m, kHi, -u) + fma(m, kLo, fma(t, double(fs[c]), -m) * kHi);
                a[c] += (u - rint(u)) + rest;
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float f = float(a[c] - rint(a[c]));
            sn[c] = __builtin_amdgcn_sinf(f);
            cs[c] = __builtin_amdgcn_cosf(f);
        }
    }
    // Turns the eight channels by the angles, or back by them.
    __device__ __forceinline__ void rotate(float v[8], bool back) const {
        if (!turn) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int a = HALVES ? i : 2 * i, b = HALVES ? 4 + i : 2 * i + 1;
            const float s = back ? -sn[i] : sn[i], u = v[a], w = v[b];
            v[a] = u * cs[i] - w * s;
            v[b] = u * s + w * cs[i];
        }
    }
};

// A lane's eight channels as loaded.  Rows are read once: past the cache, which
// is left to what is written.
template <typename IO, bool HALVES>
struct RotRaw {
    static constexpr int W = sizeof(IO) * 2; // words
    typedef uint32_t half __attribute__((ext_vector_type(W / 2 == 2 ? 2 : 4)));
    uint32_t w[W];
    __device__ __forceinline__ void load(const IO *p, const RotLane<HALVES> &l) {
        if constexpr (sizeof(IO) == 2 && !HALVES) {
            const u32x4_v v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_v *>(p + l.c0));
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = v[i];
        } else {
            const half a = __builtin_nontemporal_load(reinterpret_cast<const half *>(p + l.c0));
            const half b = __builtin_nontemporal_load(reinterpret_cast<const half *>(p + l.c1));
#pragma unroll
            for (int i = 0; i < W / 2; ++i) w[i] = a[i], w[W / 2 + i] = b[i];
        }
    }
    __device__ __forceinline__ void unpack(float v[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (sizeof(IO) == 4) v[i] = __uint_as_float(w[i]);
            else v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        }
    }
};
template <typename IO, bool HALVES>
__device__ __forceinline__ void rot_store(IO *p, const RotLane<HALVES> &l, const float v[8]) {
    if constexpr (sizeof(IO) == 2 && !HALVES) {
        *reinterpret_cast<uint4 *>(p + l.c0) = make_uint4(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]), pack2_bf16(v[4], v[5]), pack2_bf16(v[6], v[7]));
    } else {
        io<IO>::store4(p + l.c0, v);
        io<IO>::store4(p + l.c1, v + 4);
    }
}

template <typename IO, int LPR, bool HALVES, int NR>
__global__ __launch_bounds__(kRT) void k_norm_rotate(const RotParams p) {
    constexpr int RPW = 64 / LPR;
    const int lane = threadIdx.x & 63, unit = lane % LPR, sub = lane / LPR;
    // counts of tokens and rows together stay below 2^31
    const uint32_t items = p.r[0].items + p.r[1].items;
    const uint32_t item = blockIdx.x * (kRT / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t token = item / items;
    if (token >= p.tokens) return;
    int j = int(item % items);
    const bool is_q = j < p.r[0].items;
    if (!is_q) j -= p.r[0].items;
    const RotRows R = is_q ? p.r[0] : p.r[1];
    RotLane<HALVES> l(p, unit);
    const int h0 = j * NR * RPW + sub;
    const IO *x = static_cast<const IO *>(R.x) + token * R.xt;
    IO *o = static_cast<IO *>(R.out) + token * R.ot;
    RotRaw<IO, HALVES> raw[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i)
        if (l.in && h0 + i * RPW < R.heads) raw[i].load(x + (h0 + i * RPW) * R.xh, l);
    float w[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) w[c] = 1.f;
    if (R.w && l.in) {
        io<float>::load4(R.w + l.c0, w);
        io<float>::load4(R.w + l.c1, w + 4);
    }
    l.angles(p, unit, token);
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        if (i && j * NR * RPW + i * RPW >= R.heads) break; // the same for the whole wave
        const bool on = l.in && h0 + i * RPW < R.heads;
        float v[8] = {};
        if (on) raw[i].unpack(v);
        if (p.norm) {
            float ss = 0.f;
#pragma unroll
            for (int c = 0; c < 8; ++c) ss = fmaf(v[c], v[c], ss);
            const float r = __builtin_amdgcn_rsqf(fmaf(row_sum<LPR>(ss), p.inv_dim, p.eps));
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] *= r * w[c];
        }
        l.rotate(v, false);
        if (on) rot_store(o + (h0 + i * RPW) * R.oh, l, v);
    }
}

// With n = w r x, r = 1 / sqrt(mean x^2 + eps) and gn the gradient turned back:
//     dw = sum gn r x,    dx = r w gn - (r^3 / dim) x sum(x w gn).
// Workgroups are q's or k's, walk their items with a fixed stride and keep their
// share of dw in registers; k_norm_rotate_sum adds the shares in a fixed order.
// Bound by its rows: 8192 x 128 x 64 in bf16 73 us (5.5 TB/s); where q and k have
// unlike head counts, by the share of workgroups that each gets (backward_grid).
template <typename IO, int LPR, bool HALVES>
__global__ __launch_bounds__(kRT, 4) void k_norm_rotate_backward(const RotParams p) {
    constexpr int RPW = 64 / LPR, NW = kRT / 64;
    __shared__ float part[NW][LPR * 8];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), unit = lane % LPR, sub = lane / LPR;
    RotLane<HALVES> l(p, unit);
    const bool is_q = int(blockIdx.x) < p.split;
    const RotRows R = is_q ? p.r[0] : p.r[1];
    const uint32_t first = is_q ? blockIdx.x : blockIdx.x - p.split, stride = is_q ? p.split : gridDim.x - p.split;
    float w[8], dw[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) w[c] = 1.f, dw[c] = 0.f;
    if (R.w && l.in) {
        io<float>::load4(R.w + l.c0, w);
        io<float>::load4(R.w + l.c1, w + 4);
    }
    for (uint32_t item = first * NW + wave; item < uint32_t(p.tokens) * R.items; item += stride * NW) {
        const int64_t token = item / uint32_t(R.items);
        const int h0 = int(item % uint32_t(R.items)) * kRows * RPW + sub;
        const IO *x = static_cast<const IO *>(R.x) + token * R.xt;
        const IO *g = static_cast<const IO *>(R.g) + token * R.gt;
        IO *o = static_cast<IO *>(R.out) + token * R.ot;
        RotRaw<IO, HALVES> rx[kRows], rg[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (l.in && h0 + i * RPW < R.heads) {
                if (p.norm) rx[i].load(x + (h0 + i * RPW) * R.xh, l);
                rg[i].load(g + (h0 + i * RPW) * R.gh, l);
            }
        l.angles(p, unit, token);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (i && h0 - sub + i * RPW >= R.heads) break; // the same for the whole wave
            const bool on = l.in && h0 + i * RPW < R.heads;
            float a[8] = {};
            if (on) rg[i].unpack(a);
            l.rotate(a, true);
            if (p.norm) {
                float v[8] = {}, ss = 0.f, dot = 0.f;
                if (on) rx[i].unpack(v);
#pragma unroll
                for (int c = 0; c < 8; ++c) ss = fmaf(v[c], v[c], ss);
                // without a row nothing joins dw: eps may be 0, and then r would be infinite
                const float rms = __builtin_amdgcn_rsqf(fmaf(row_sum<LPR>(ss), p.inv_dim, p.eps)), r = on ? rms : 0.f;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    dw[c] = fmaf(a[c] * r, v[c], dw[c]);
                    a[c] *= w[c];
                    dot = fmaf(v[c], a[c], dot);
                }
                const float m = row_sum<LPR>(dot) * p.inv_dim * (r * r);
#pragma unroll
                for (int c = 0; c < 8; ++c) a[c] = r * (a[c] - m * v[c]);
            }
            if (on) rot_store(o + (h0 + i * RPW) * R.oh, l, a);
        }
    }
    if (!R.w) return;
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int m = LPR; m < 64; m <<= 1) dw[c] += __shfl_xor(dw[c], m);
    if (sub == 0)
#pragma unroll
        for (int c = 0; c < 8; ++c) part[wave][unit * 8 + c] = dw[c];
    __syncthreads();
    if (wave == 0 && sub == 0 && l.in) {
        float *o = p.part + int64_t(blockIdx.x) * p.dim;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            float s = 0.f;
#pragma unroll
            for (int v = 0; v < NW; ++v) s += part[v][unit * 8 + c];
            o[c < 4 ? l.c0 + c : l.c1 + c - 4] = s;
        }
    }
}

// Sum of the workgroups' shares, four channels of one weight per workgroup: a
// share to a thread, then the threads of a wave and the waves in turn.  4 us for
// 1024 shares of 64 channels: the latency of a load, the sums and the launch.
__global__ __launch_bounds__(1024) void k_norm_rotate_sum(const float *part, int split, int n, int dim, float *dq, float *dk) {
    __shared__ floatx4 s[16];
    const int c = blockIdx.x * 4;
    float *out = blockIdx.y ? dk : dq;
    if (!out) return;
    floatx4 a{0.f, 0.f, 0.f, 0.f};
    for (int i = (blockIdx.y ? split : 0) + threadIdx.x; i < (blockIdx.y ? n : split); i += 1024)
        a += *reinterpret_cast<const floatx4 *>(part + int64_t(i) * dim + c);
#pragma unroll
    for (int m = 32; m > 0; m >>= 1)
#pragma unroll
        for (int v = 0; v < 4; ++v) a[v] += __shfl_xor(a[v], m);
    if (threadIdx.x % 64 == 0) s[threadIdx.x / 64] = a;
    __syncthreads();
    if (threadIdx.x < 4) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < 16; ++w) t += s[w][threadIdx.x];
        out[c + threadIdx.x] = t;
    }
}

// Lanes of a row: the power of two that holds dim / 8.
constexpr int rot_lanes(int dim) {
    int n = 1;
    while (n * 8 < dim) n *= 2;
    return n;
}

template <typename IO, int LPR, bool HALVES>
hipError_t launch_rotary(RotParams &p, int64_t grid, bool back, hipStream_t s) {
    if (back) {
        hipLaunchKernelGGL((k_norm_rotate_backward<IO, LPR, HALVES>), dim3(unsigned(grid)), dim3(kRT), 0, s, p);
        return hipGetLastError();
    }
    // Below two waves a SIMD, or where a set holds all heads, a wave takes one set:
    // 512 x 40 x 128 4.8 us (5.4 with up to four sets), 32768 x 10 x 64 33 us (37).
    // Else its angles serve up to four: 16384 x 40 x 128 57 us a call, 54 the kernel
    // (calls of 79 with one, 60 with six), 1024 x 40 x 128 7.5 us (8.5 with one).
    if (grid < 512 || std::max(p.r[0].heads, p.r[1].heads) <= 64 / LPR) {
        for (RotRows &r : p.r) r.items = (r.heads + 64 / LPR - 1) / (64 / LPR);
        grid = (p.tokens * (p.r[0].items + p.r[1].items) + 3) / 4;
        hipLaunchKernelGGL((k_norm_rotate<IO, LPR, HALVES, 1>), dim3(unsigned(grid)), dim3(kRT), 0, s, p);
    } else {
        hipLaunchKernelGGL((k_norm_rotate<IO, LPR, HALVES, kRows>), dim3(unsigned(grid)), dim3(kRT), 0, s, p);
    }
    return hipGetLastError();
}

template <typename IO, bool HALVES>
hipError_t launch_rotary_lanes(RotParams &p, int64_t grid, bool back, hipStream_t s) {
    switch (rot_lanes(p.dim)) {
    case 1: return launch_rotary<IO, 1, HALVES>(p, grid, back, s);
    case 2: return launch_rotary<IO, 2, HALVES>(p, grid, back, s);
    case 4: return launch_rotary<IO, 4, HALVES>(p, grid, back, s);
    case 8: return launch_rotary<IO, 8, HALVES>(p, grid, back, s);
    case 16: return launch_rotary<IO, 16, HALVES>(p, grid, back, s);
    case 32: return launch_rotary<IO, 32, HALVES>(p, grid, back, s);
    }
    return hipErrorInvalidValue;
}
template <typename IO>
hipError_t launch_rotary_io(RotParams &p, bool halves, int64_t grid, bool back, hipStream_t s) {
    return halves ? launch_rotary_lanes<IO, true>(p, grid, back, s) : launch_rotary_lanes<IO, false>(p, grid, back, s);
}

} // namespace m3

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Items of one token: groups of kRows row sets.
int32_t items(const m3_rotary_shape_t *s, int32_t heads) {
    const int set = m3::kRows * (64 / m3::rot_lanes(s->dim));
    return (heads + set - 1) / set;
}

m3_status_t check_shape(const m3_rotary_shape_t *s) {
    if (!s) return M3_ERR_INVALID_ARGUMENT;
    if (s->io_dtype != M3_DTYPE_F32 && s->io_dtype != M3_DTYPE_BF16) return M3_ERR_INVALID_ARGUMENT;
    if (s->tokens < 0 || s->q_heads < 1 || s->k_heads < 0 || s->dim < 1 || s->rot < 1 || s->rot > s->dim || s->axes < 1)
        return M3_ERR_INVALID_ARGUMENT;
    if (s->norm && !(s->eps >= 0.f)) return M3_ERR_INVALID_ARGUMENT;
    if (s->dim % 8 || s->dim > 256 || s->rot % 8 || s->axes > 4) return M3_ERR_UNSUPPORTED;
    if (s->q_heads > (1 << 20) || s->k_heads > (1 << 20)) return M3_ERR_UNSUPPORTED;
    // rows are counted in 32 bits, and a launch has fewer than 2^32 threads: a wave of 64
    // for 64 / lanes rows or fewer
    if (double(s->tokens) * (double(s->q_heads) + s->k_heads + 2) > 2147483647.0) return M3_ERR_UNSUPPORTED;
    if ((double(s->tokens) * (items(s, s->q_heads) + items(s, s->k_heads)) + 4) * 64 > 4294967295.0) return M3_ERR_UNSUPPORTED;
    return M3_OK;
}

bool rows_ok(const m3_rows_t *r, int64_t tokens, int32_t heads, int32_t dim, bool out) {
    if (heads == 0) return true;
    if (!r) return false;
    if (tokens == 0) return true;
    const int64_t t = r->token_stride, h = r->head_stride;
    if (!r->data || !aligned16(r->data) || t < 0 || h < 0 || t >= (int64_t(1) << 24) || h >= (int64_t(1) << 40) || t % 8 || h % 8)
        return false;
    if (!out) return true;
    const bool by_token = (tokens == 1 || t >= (heads - 1) * h + dim) && (heads == 1 || h >= dim);
    const bool by_head = (heads == 1 || h >= (tokens - 1) * t + dim) && (tokens == 1 || t >= dim);
    return by_token || by_head;
}

// Whether an output's rows start where another operand does, or its own input's lie otherwise.
bool rows_overlap(const m3_rotary_shape_t *s, const m3_rows_t *q, const m3_rows_t *k, const m3_rows_t *qo, const m3_rows_t *ko,
                  const m3_rows_t *gq, const m3_rows_t *gk, std::initializer_list<const void *> others) {
    if (s->tokens == 0) return false;
    auto clash = [&](const m3_rows_t *out, const m3_rows_t *own, int32_t heads) {
        return own && out->data == own->data &&
               ((s->tokens > 1 && out->token_stride != own->token_stride) || (heads > 1 && out->head_stride != own->head_stride));
    };
    auto among = [&](const m3_rows_t *out) { return std::find(others.begin(), others.end(), out->data) != others.end(); };
    if (clash(qo, q, s->q_heads) || clash(qo, gq, s->q_heads) || among(qo)) return true;
    if (s->k_heads == 0) return false;
    if (clash(ko, k, s->k_heads) || clash(ko, gk, s->k_heads) || among(ko)) return true;
    return qo->data == ko->data || qo->data == k->data || ko->data == q->data ||
           (gq && (qo->data == gk->data || ko->data == gq->data));
}

// Workgroups of the gradients, for q and for k, in the ratio of their items: at
// most the four per compute unit that are resident at once (128 registers), so
// that they leave few partial sums.  Twice as many took as long (a call of 75 us at
// 8192 x 128 x 64) and their sum 1 us more.  An item holds one to four sets of
// rows, so the rows are shared evenly where q and k have as many heads; of 16 and
// 4 heads of 96 channels k gets half the workgroups for a fifth of the rows (3001
// tokens in fp32 17.5 us, 4.0 TB/s), of 32 and 8 of 128 a third for a fifth (16384
// in bf16 91 us, 5.5 TB/s).
struct BackGrid {
    int64_t q, k;
};
BackGrid backward_grid(const m3_rotary_shape_t *s) {
    const int64_t iq = items(s, s->q_heads), ik = items(s, s->k_heads), n = (s->tokens * (iq + ik) + 3) / 4;
    const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(n, 1024));
    if (ik == 0) return {grid, 0};
    const int64_t k = std::max<int64_t>(1, grid * ik / (iq + ik));
    return {std::max<int64_t>(1, grid - k), k};
}

m3::RotParams params(const m3_rotary_shape_t *s, const m3_rows_t *q, const m3_rows_t *k, const void *pos,
                     const float *freq, const float *qw, const float *kw, const m3_rows_t *qo, const m3_rows_t *ko) {
    m3::RotParams p{};
    const m3_rows_t *in[2] = {q, k}, *out[2] = {qo, ko};
    const int32_t heads[2] = {s->q_heads, s->k_heads};
    const float *w[2] = {qw, kw};
    for (int i = 0; i < 2; ++i) {
        if (heads[i] == 0) continue;
        p.r[i].x = in[i]->data; p.r[i].xt = in[i]->token_stride; p.r[i].xh = in[i]->head_stride;
        p.r[i].out = out[i]->data; p.r[i].ot = out[i]->token_stride; p.r[i].oh = out[i]->head_stride;
        p.r[i].w = w[i];
        p.r[i].heads = heads[i];
        p.r[i].items = items(s, heads[i]);
    }
    p.tokens = s->tokens;
    p.dim = s->dim;
    p.rot = s->rot;
    p.axes = s->axes;
    p.pos64 = s->pos_int64;
    p.norm = s->norm;
    p.eps = s->eps;
    p.inv_dim = 1.f / float(s->dim);
    p.pos = pos;
    p.freq = freq;
    return p;
}

m3_status_t check_common(const m3_rotary_shape_t *s, const void *pos, const float *freq, const float *qw, const float *kw) {
    if (s->tokens && (!pos || (reinterpret_cast<uintptr_t>(pos) & (s->pos_int64 ? 7 : 3)))) return M3_ERR_INVALID_ARGUMENT;
    if (!freq || !aligned16(freq) || !aligned16(qw) || !aligned16(kw)) return M3_ERR_INVALID_ARGUMENT;
    if ((qw || kw) && !s->norm) return M3_ERR_INVALID_ARGUMENT;
    if (kw && s->k_heads == 0) return M3_ERR_INVALID_ARGUMENT;
    return M3_OK;
}

} // namespace

extern "C" {

m3_status_t m3_norm_rotate(const m3_rotary_shape_t *shape, const m3_rows_t *q, const m3_rows_t *k,
                           const void *positions, const float *inv_freq, const float *q_weight,
                           const float *k_weight, const m3_rows_t *q_out, const m3_rows_t *k_out,
                           hipStream_t stream) {
    m3_status_t sc = check_shape(shape);
    if (sc != M3_OK) return sc;
    sc = check_common(shape, positions, inv_freq, q_weight, k_weight);
    if (sc != M3_OK) return sc;
    const int64_t T = shape->tokens;
    if (!rows_ok(q, T, shape->q_heads, shape->dim, false) || !rows_ok(k, T, shape->k_heads, shape->dim, false) ||
        !rows_ok(q_out, T, shape->q_heads, shape->dim, true) || !rows_ok(k_out, T, shape->k_heads, shape->dim, true))
        return M3_ERR_INVALID_ARGUMENT;
    if (T == 0) return M3_OK;
    if (rows_overlap(shape, q, k, q_out, k_out, nullptr, nullptr, {positions, inv_freq, q_weight, k_weight}))
        return M3_ERR_INVALID_ARGUMENT;
    m3::RotParams p = params(shape, q, k, positions, inv_freq, q_weight, k_weight, q_out, k_out);
    const int64_t grid = (T * (p.r[0].items + p.r[1].items) + 3) / 4;
    const hipError_t e = shape->io_dtype == M3_DTYPE_F32 ? m3::launch_rotary_io<float>(p, shape->halves, grid, false, stream)
                                                         : m3::launch_rotary_io<m3::bf16>(p, shape->halves, grid, false, stream);
    return e == hipSuccess ? M3_OK : M3_ERR_HIP;
}

size_t m3_norm_rotate_backward_workspace_bytes(const m3_rotary_shape_t *shape) {
    if (check_shape(shape) != M3_OK) return 0;
    const BackGrid g = backward_grid(shape);
    return size_t(g.q + g.k) * shape->dim * sizeof(float);
}

m3_status_t m3_norm_rotate_backward(const m3_rotary_shape_t *shape, const m3_rows_t *q, const m3_rows_t *k,
                                    const void *positions, const float *inv_freq, const float *q_weight,
                                    const float *k_weight, const m3_rows_t *gq, const m3_rows_t *gk,
                                    const m3_rows_t *dq, const m3_rows_t *dk, float *dq_weight, float *dk_weight,
                                    void *workspace, size_t workspace_bytes, hipStream_t stream) {
    m3_status_t sc = check_shape(shape);
    if (sc != M3_OK) return sc;
    sc = check_common(shape, positions, inv_freq, q_weight, k_weight);
    if (sc != M3_OK) return sc;
    const int64_t T = shape->tokens;
    if (!rows_ok(q, T, shape->q_heads, shape->dim, false) || !rows_ok(k, T, shape->k_heads, shape->dim, false) ||
        !rows_ok(gq, T, shape->q_heads, shape->dim, false) || !rows_ok(gk, T, shape->k_heads, shape->dim, false) ||
        !rows_ok(dq, T, shape->q_heads, shape->dim, true) || !rows_ok(dk, T, shape->k_heads, shape->dim, true))
        return M3_ERR_INVALID_ARGUMENT;
    if (!q_weight != !dq_weight || !k_weight != !dk_weight) return M3_ERR_INVALID_ARGUMENT;
    if ((reinterpret_cast<uintptr_t>(dq_weight) & 3) || (reinterpret_cast<uintptr_t>(dk_weight) & 3)) return M3_ERR_INVALID_ARGUMENT;
    if (!workspace || !aligned16(workspace) || workspace_bytes < m3_norm_rotate_backward_workspace_bytes(shape))
        return M3_ERR_WORKSPACE;
    if (rows_overlap(shape, q, k, dq, dk, gq, gk, {positions, inv_freq, q_weight, k_weight, dq_weight, dk_weight, workspace}))
        return M3_ERR_INVALID_ARGUMENT;
    // the weights' gradients and the workspace, each against every operand that is not a row of the gradients
    const void *const small[] = {dq_weight, dk_weight, workspace, q_weight, k_weight, inv_freq, T ? positions : nullptr,
                                 T ? q->data : nullptr, T ? gq->data : nullptr, T && shape->k_heads ? k->data : nullptr,
                                 T && shape->k_heads ? gk->data : nullptr};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 11; ++j)
            if (small[i] && small[i] == small[j]) return M3_ERR_INVALID_ARGUMENT;
    m3::RotParams p = params(shape, q, k, positions, inv_freq, q_weight, k_weight, dq, dk);
    p.r[0].g = gq->data; p.r[0].gt = gq->token_stride; p.r[0].gh = gq->head_stride;
    if (shape->k_heads) { p.r[1].g = gk->data; p.r[1].gt = gk->token_stride; p.r[1].gh = gk->head_stride; }
    p.part = static_cast<float *>(workspace);
    const BackGrid g = backward_grid(shape);
    const int64_t grid = g.q + g.k;
    p.split = int32_t(g.q);
    const hipError_t e = shape->io_dtype == M3_DTYPE_F32 ? m3::launch_rotary_io<float>(p, shape->halves, grid, true, stream)
                                                         : m3::launch_rotary_io<m3::bf16>(p, shape->halves, grid, true, stream);
    if (e != hipSuccess) return M3_ERR_HIP;
    if (dq_weight || dk_weight) {
        hipLaunchKernelGGL(m3::k_norm_rotate_sum, dim3(unsigned(shape->dim / 4), 2), dim3(1024), 0, stream,
                           p.part, p.split, int(grid), shape->dim, dq_weight, dk_weight);
        if (hipGetLastError() != hipSuccess) return M3_ERR_HIP;
    }
    return M3_OK;
}

} // extern "C"

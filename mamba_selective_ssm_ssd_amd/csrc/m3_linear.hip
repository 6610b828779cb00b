// m3_linear.hip -- C ABI of linear attention with a decay for each head
// (include/m3_linear.h): argument checks, plan, workspace and launch sequence,
// with the small kernels around the scan of k_linear.hpp: the join of segment
// states, the sum of a shared row's gradients, the single-token step.
#include "m3_linear.h"
#include "k_linear.hpp"
#include "lin_plan.hpp"
#include "m3_internal.hpp"

#include <algorithm>
#include <initializer_list>

namespace m3 {

// Joins the segment states of a cut sequence in place: a slot holds what the
// segment before it left from zero (the first one from the initial state) and
// gets the state that its own segment starts from: s_i <- g^L s_{i-1} + s_i.
// blockIdx.x: (sequence, head), blockIdx.y: 1024 entries of the state,
// blockIdx.z: scan.  A thread has four entries and eight segments' loads in
// flight: bound by reading and writing the states (64 segments of 64 x 64 x 64
// heads, 134 MB, 30 us: 4.5 TB/s), or by the chain of loads where they are few,
// which goes through the segments one after another: two unlike sequences,
// 8192 x 8 x 128 in all, in 32 segments, 12 us beside scans of 15 and 24.
__global__ __launch_bounds__(256) void k_linear_join(const LinParams p) {
    const LinRole &R = p.role[blockIdx.z];
    const int64_t b = blockIdx.x / p.H, h = blockIdx.x % p.H;
    const int64_t start = lin_start(p, b), next = lin_start(p, b + 1);
    const int64_t len = next > start ? next - start : 0, n = (len + (int64_t(1) << p.segbits) - 1) >> p.segbits;
    if (n <= 2) return;
    if (lin_slot(p.slots, p.nstates, b) < 0) return;
    const int64_t area = int64_t(R.dx) * R.dz, e = (int64_t(blockIdx.y) * 256 + threadIdx.x) * 4;
    if (e >= area) return;
    float *w = R.seg + (lin_state_slot(p, b, start) * p.H + h) * area + e;
    const int64_t step = p.H * area;
    floatx4 s = *reinterpret_cast<const floatx4 *>(w + step);
    const LinDecay d(p.log_decay[h], double(int64_t(1) << p.segbits));
    constexpr int U = 8; // loads in flight
    for (int64_t i = 2; i < n; i += U) {
        floatx4 a[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u < n) a[u] = *reinterpret_cast<const floatx4 *>(w + (i + u) * step);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u < n) {
#pragma unroll
                for (int k = 0; k < 4; ++k) s[k] = d(s[k]) + a[u][k];
                *reinterpret_cast<floatx4 *>(w + (i + u) * step) = s;
            }
    }
}

// Gradient rows that several heads share: the heads' parts [token][H][dim]
// fp32, summed in the heads' order and rounded once; zero for tokens outside
// every sequence.  Bound by reading the parts: 2 x 4999 x 32 x 128, 184 MB with
// the result, 29.5 us (6.2 TB/s, part of it from the last-level cache).
struct LinSum {
    const float *part;
    void *out;
    int64_t ot, oh;
    int32_t heads, group, dim; // rows of out, heads per row
};
struct LinSums {
    LinSum s[3];
    int32_t n;
    LinParams seq; // sequences only
};

template <typename IO>
__global__ __launch_bounds__(256) void k_linear_sum(const LinSums p) {
    const LinSum &s = p.s[blockIdx.y];
    const int u = s.dim / 8;
    const int64_t n = p.seq.tokens * s.heads * u;
    const int64_t lo = lin_start(p.seq, 0), hi = lin_start(p.seq, p.seq.batch);
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
        const int c = int(i % u) * 8, r = int(i / u % s.heads);
        const int64_t t = i / (int64_t(u) * s.heads);
        float a[8] = {};
        if (t >= lo && t < hi) {
            const float *q = s.part + ((t * s.heads + r) * s.group) * s.dim + c;
            for (int j = 0; j < s.group; ++j) {
                float v[8];
                io<float>::load8(q + int64_t(j) * s.dim, v);
#pragma unroll
                for (int k = 0; k < 8; ++k) a[k] += v[k];
            }
        }
        IO *o = static_cast<IO *>(s.out) + t * s.ot + r * s.oh + c;
        io<IO>::store4(o, a);
        io<IO>::store4(o + 4, a + 4);
    }
}

// ---------------------------------------------------------------------------
// Single-token step.  S <- g S + k v^T and o = scale q^T S over one state of
// Dk x Dv entries per sequence and head: bound by reading and writing it.  A
// workgroup takes W columns of one state, four columns per lane in rows of
// W / 4 lanes, and holds all its rows in registers: every load is issued before
// the first is used.  States are read and written past the caches, as the layers
// between two steps leave nothing of them there:
// 100 us (5.4 TB/s) against 111 us with reads alone and 114 us with neither, over
// 256 x 64 fp32 states of 64 x 64 taken in turn from more than the cache holds;
// bf16 states, of which a lane loads 8 bytes, 63 us (4.3 TB/s).
// With slots a workgroup also reads those before its own: as slots in order
// nothing to 1024 sequences, 4% of 4096 x 16 states of 64 x 64, 40% of 16384 x 4
// of them; in any order states lie apart, which costs 13% at 1024 x 64.
// ---------------------------------------------------------------------------
struct LinStepParams {
    const void *q, *k, *v;
    void *o, *state;
    int64_t qt, qh, kt, kh, vt, vh, ot, oh;
    int32_t qg, kg, vg, H, dk, dv, slices;
    int64_t batch, nstates;
    const int32_t *slots;
    const float *log_decay;
    float scale;
};

typedef uint32_t u32x2_v __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint4 step_load(const float *p) {
    const u32x4_v v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_v *>(p));
    return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ uint2 step_load(const bf16 *p) {
    const u32x2_v v = __builtin_nontemporal_load(reinterpret_cast<const u32x2_v *>(p));
    return make_uint2(v.x, v.y);
}
__device__ __forceinline__ void step_store(float *p, const float v[4]) {
    __builtin_nontemporal_store(floatx4{v[0], v[1], v[2], v[3]}, reinterpret_cast<floatx4 *>(p));
}
__device__ __forceinline__ void step_store(bf16 *p, const float v[4]) {
    __builtin_nontemporal_store(u32x2_v{pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3])}, reinterpret_cast<u32x2_v *>(p));
}

template <typename IO, typename ST, int W>
__global__ __launch_bounds__(256) void k_linear_step(const LinStepParams p) {
    constexpr int L = W / 4, RP = 256 / L, NP = 128 / RP; // lanes per row, rows per pass, passes
    __shared__ float part[4][W];
    int64_t id = blockIdx.x;
    const int slice = int(id % p.slices);
    id /= p.slices;
    const int h = int(id % p.H);
    const int64_t b = id / p.H;
    const int tid = threadIdx.x, c = slice * W + tid % L * 4, r0 = tid / L;
    const bool in = c < p.dv;
    IO *o = static_cast<IO *>(p.o) + b * p.ot + h * p.oh;

    int64_t slot = b;
    int taken = 0;
    if (p.slots) {
        slot = p.slots[b];
        if (slot < 0 || slot >= p.nstates) return;
        // an earlier sequence with the same slot has the state; looked for before
        // the state's loads, which answer in order, are issued
        for (int64_t j = tid; j < b; j += 256) taken |= p.slots[j] == int32_t(slot);
    }
    ST *st = static_cast<ST *>(p.state) + (slot * p.H + h) * p.dk * p.dv + c;
    typename io4<ST>::raw raw[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i)
        if (in && r0 + i * RP < p.dk) raw[i] = step_load(st + (r0 + i * RP) * p.dv);
    const IO *q = static_cast<const IO *>(p.q) + b * p.qt + (h / p.qg) * p.qh;
    const IO *k = static_cast<const IO *>(p.k) + b * p.kt + (h / p.kg) * p.kh;
    float qv[NP], kv[NP], v[4] = {};
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        qv[i] = kv[i] = 0.f;
        if (r0 + i * RP < p.dk) {
            qv[i] = io<IO>::get(q + r0 + i * RP);
            kv[i] = io<IO>::get(k + r0 + i * RP);
        }
    }
    if (in) io<IO>::load4(static_cast<const IO *>(p.v) + b * p.vt + (h / p.vg) * p.vh + c, v);
    if (p.slots && __syncthreads_or(taken)) {
        if (tid < L && in)
            for (int j = 0; j < 4; ++j) io<IO>::put(o + c + j, __builtin_nanf(""));
        return;
    }
    const LinDecay d(p.log_decay[h], 1.0);
    float a[4] = {};
#pragma unroll
    for (int i = 0; i < NP; ++i)
        if (in && r0 + i * RP < p.dk) {
            float s[4];
            io4<ST>::unpack(raw[i], s);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[j] = fmaf(kv[i], v[j], d(s[j]));
                a[j] = fmaf(qv[i], s[j], a[j]);
            }
            step_store(st + (r0 + i * RP) * p.dv, s);
        }
    // rows of one wave, then the four waves
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int m = L; m < 64; m <<= 1) a[j] += __shfl_xor(a[j], m);
    if (tid % 64 < L)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[tid / 64][tid % 64 * 4 + j] = a[j];
    __syncthreads();
    if (tid < L && in) {
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = p.scale * ((part[0][tid * 4 + j] + part[1][tid * 4 + j]) + (part[2][tid * 4 + j] + part[3][tid * 4 + j]));
        io<IO>::store4(o + c, a);
    }
}

template <typename IO, typename ST>
hipError_t launch_linear_step(LinStepParams &p, hipStream_t s) {
    // below two workgroups a compute unit, twice as many of half the columns: 32
    // states of 128 x 128 4.7 us (5.2 with 64 columns); 512 of 64 x 64 6.0 us (6.7 with 32)
    const bool wide = p.batch * p.H * ((p.dv + 63) / 64) >= 512;
    p.slices = wide ? (p.dv + 63) / 64 : (p.dv + 31) / 32;
    const dim3 grid(unsigned(p.batch * p.H * p.slices));
    if (wide) hipLaunchKernelGGL((k_linear_step<IO, ST, 64>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((k_linear_step<IO, ST, 32>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

} // namespace m3

namespace {

using m3::LinParams;
using m3::LinRole;

constexpr size_t kAlign = 256;
size_t round_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int32_t heads(const m3_linear_shape_t *s) { return std::max(s->q_heads, std::max(s->k_heads, s->v_heads)); }

m3_status_t check_shape(const m3_linear_shape_t *s, bool decode) {
    if (!s) return M3_ERR_INVALID_ARGUMENT;
    if (s->io_dtype != M3_DTYPE_F32 && s->io_dtype != M3_DTYPE_BF16) return M3_ERR_INVALID_ARGUMENT;
    if (s->state_dtype != M3_DTYPE_F32 && s->state_dtype != M3_DTYPE_BF16) return M3_ERR_INVALID_ARGUMENT;
    if (s->batch < 1 || s->q_heads < 1 || s->k_heads < 1 || s->v_heads < 1 || s->key_dim < 1 || s->value_dim < 1)
        return M3_ERR_INVALID_ARGUMENT;
    if (!decode && (s->tokens < 0 || s->max_seqlen < 0)) return M3_ERR_INVALID_ARGUMENT;
    const int32_t H = heads(s);
    if (H % s->q_heads || H % s->k_heads || H % s->v_heads) return M3_ERR_INVALID_ARGUMENT;
    if (s->key_dim % 8 || s->value_dim % 8 || s->key_dim > 128 || s->value_dim > 128) return M3_ERR_UNSUPPORTED;
    // counts of sequences and tokens are indexed in 32 bits (cu_seqlens, slots), workgroups too
    if (s->batch > (int64_t(1) << 31) - 2) return M3_ERR_UNSUPPORTED;
    // one token's rows of all heads, in parts of a gradient: a chunk of them within 2^32 bytes
    if (int64_t(H) * std::max(s->key_dim, s->value_dim) >= int64_t(1) << 24) return M3_ERR_UNSUPPORTED;
    if (!decode && s->tokens > (int64_t(1) << 31) - 1) return M3_ERR_UNSUPPORTED;
    // a launch has fewer than 2^32 threads: workgroups of 256 for each head, two column
    // tiles and three scans of a segment slot: one per sequence, and one per 1024 tokens
    // but where these are 512 at most
    const double slots = (double(s->batch) + 8 + (decode ? 0. : double(s->tokens) / 1024)) * H + 512;
    if (slots * 256 * (decode ? 2 : 6) > 4294967295.0) return M3_ERR_UNSUPPORTED;
    return M3_OK;
}

bool strides_ok(const m3_rows_t *r) {
    return r->token_stride >= 0 && r->head_stride >= 0 && r->token_stride < (int64_t(1) << 24) &&
           r->head_stride < (int64_t(1) << 40) && r->token_stride % 8 == 0 && r->head_stride % 8 == 0;
}
// Rows to read.  Without a row the pointer is not looked at.
bool rows_ok(const m3_rows_t *r, int64_t tokens, int32_t dim) {
    if (!r) return false;
    return tokens == 0 || (r->data && aligned16(r->data) && strides_ok(r) && (tokens == 1 || r->token_stride >= dim));
}
// Rows to write: no two may overlap, whichever axis is the outer one.
bool out_ok(const m3_rows_t *r, int64_t tokens, int32_t heads, int32_t dim) {
    if (!rows_ok(r, tokens, dim)) return false;
    if (tokens == 0) return true;
    const int64_t t = r->token_stride, h = r->head_stride;
    const bool by_token = (tokens == 1 || t >= (heads - 1) * h + dim) && (heads == 1 || h >= dim);
    const bool by_head = (heads == 1 || h >= (tokens - 1) * t + dim) && (tokens == 1 || t >= dim);
    return by_token || by_head;
}

// Where rows start (nowhere without a token).
const void *start(const m3_rows_t *r, int64_t tokens) { return tokens > 0 ? r->data : nullptr; }
// Whether one of the first `outputs` operands starts where another operand does (they may
// still overlap: views are not compared).  Absent ones are null.
bool starts_in(int outputs, std::initializer_list<const void *> operands) {
    const void *const *p = operands.begin();
    const int n = int(operands.size());
    for (int i = 0; i < outputs; ++i)
        for (int j = i + 1; j < n; ++j)
            if (p[i] && p[i] == p[j]) return true;
    return false;
}

// Columns of z a workgroup takes, up to `most`: 64 with fp32 I/O, which holds three planes of everything.
int z_tile(int dz, bool f32, int most = 128) { return std::min(m3::lin_tile(dz), std::min(most, f32 ? 64 : 128)); }
int z_tiles(int dz, bool f32, int most = 128) { return (dz + z_tile(dz, f32, most) - 1) / z_tile(dz, f32, most); }

// Tokens per segment, a power of two (0: sequences are not cut) for `scans` scans over `columns`
// column tiles in one launch.
int64_t segment(const m3_linear_shape_t *s, int scans, int columns) {
    const int64_t longest = s->max_seqlen > 0 && s->max_seqlen < s->tokens ? s->max_seqlen : s->tokens;
    const int64_t per = int64_t(heads(s)) * scans * columns;
    // Enough workgroups for most compute units, none much longer than the others:
    // the chip is full without cutting, and nothing is read twice (8 x 2048 x 32 x
    // 128 144 us, 177 cut by 1024; gradients of 4 x 2048 x 32 x 128 184 us, 222 cut).
    // It counts workgroups and not how long their chains are: gradients of one
    // sequence of 65536 x 64 x 64, 192 workgroups, take 1570 us, twice the time of
    // their bytes.
    if (longest <= 256 || (s->batch * per >= 192 && longest * s->batch < 2 * s->tokens)) return 0;
    // Else two workgroups a compute unit, all that fit at once: longer segments leave
    // some idle, shorter ones read and write states instead of rows (16 ragged
    // sequences of 1024 x 32 x 128: 207 us with segments of 1024, 227 of 512, 240 of
    // 2048).  The gradients' scans differ more: four (4096 x 32 x 128 135 us, 148 with
    // two).  1024 tokens at most: 65536 x 64 x 64 703 us, 729 with 2048.
    // From 256 on, or 128 of the slower fp32 rows (1000 x 8 x 128 34 us, 47 with 256;
    // in bf16 2000 x 32 x 128 53 us, 45 with 256).
    int64_t L = s->io_dtype == M3_DTYPE_F32 ? 128 : 256;
    while (L < 1024 && L * (scans > 1 ? 1024 : 512) < s->tokens * per) L *= 2;
    return longest > L ? L : 0;
}
// With four segments or fewer each folds the states before its own instead of a
// pass that joins them: 1000 x 32 x 128 36 us, 38 joined; gradients of 8192 x 32 x
// 128 242 us, 247 joined, but 292 where eight are folded.
int32_t few_segments(const m3_linear_shape_t *s, int64_t L) {
    const int64_t longest = s->max_seqlen > 0 && s->max_seqlen < s->tokens ? s->max_seqlen : s->tokens;
    return L && longest <= 4 * L;
}
int64_t segment_slots(const m3_linear_shape_t *s, int64_t L) { return L ? s->tokens / L + s->batch : s->batch; }
// States of segments that a workspace holds: one a slot, or, with more sequences than segments of
// tokens, those of cut sequences alone: 1000 sequences of 60000 tokens, the longest of 8192, take 117
// states of every head (245 MB of 32 x 128 x 128) instead of 1058.
bool sparse_states(const m3_linear_shape_t *s, int64_t L) { return L && s->tokens / L < s->batch; }
int64_t state_slots(const m3_linear_shape_t *s, int64_t L) {
    return sparse_states(s, L) ? 2 * s->tokens / L : segment_slots(s, L);
}

struct Layout {
    int64_t L, slots;
    int32_t most; // columns of z a workgroup takes at most
    int32_t fold; // few segments: each reads the slots before its own instead of a pass that joins them
    size_t seg_f, seg_b, part[3], total; // byte offsets: segment states forwards, backwards, the parts of gradients
};
// Narrower workgroups while there is at most one for each compute unit: the
// chain of chunks is as long, but a chunk's work, and the state to load and
// store, less.  77 x 16 x 128 12.1 us, 10.3 with 64 columns, 9.0 with 32;
// 1000 x 32 x 128 38, 30, 34; gradients of 250 x 16 x 128 17.8, 12.7, 11.6.
int most_columns(const m3_linear_shape_t *s, int64_t slots, const int *dz, int scans) {
    const bool f32 = s->io_dtype == M3_DTYPE_F32;
    int most = f32 ? 64 : 128;
    for (; most > 32; most /= 2) {
        int64_t columns = 0;
        for (int i = 0; i < scans; ++i) columns += z_tiles(dz[i], f32, most / 2);
        if (slots * heads(s) * columns > 256) break;
    }
    return most;
}
Layout prefill_layout(const m3_linear_shape_t *s) {
    Layout w{};
    w.L = segment(s, 1, z_tiles(s->value_dim, s->io_dtype == M3_DTYPE_F32));
    w.slots = segment_slots(s, w.L);
    w.most = most_columns(s, w.slots, &s->value_dim, 1);
    w.fold = few_segments(s, w.L);
    if (w.L) w.total = round_up(size_t(state_slots(s, w.L)) * heads(s) * s->key_dim * s->value_dim * 4);
    w.total = std::max(w.total, kAlign);
    return w;
}
Layout backward_layout(const m3_linear_shape_t *s) {
    Layout w{};
    const int32_t H = heads(s);
    w.L = segment(s, 3, 1);
    w.slots = segment_slots(s, w.L);
    const int dz[3] = {s->key_dim, s->key_dim, s->value_dim};
    w.most = most_columns(s, w.slots, dz, 3);
    w.fold = few_segments(s, w.L);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += round_up(bytes);
        return o;
    };
    if (w.L) {
        const size_t n = size_t(state_slots(s, w.L)) * H * s->key_dim * s->value_dim * 4;
        w.seg_f = take(n);
        w.seg_b = take(n);
    }
    const int32_t hs[3] = {s->q_heads, s->k_heads, s->v_heads}, ds[3] = {s->key_dim, s->key_dim, s->value_dim};
    for (int i = 0; i < 3; ++i)
        if (hs[i] < H) w.part[i] = take(size_t(s->tokens) * H * ds[i] * 4);
    w.total = std::max(at, kAlign);
    return w;
}

// Launches the scans p.role[0 .. n-1], which share their tile sizes.
hipError_t launch_scan(LinParams p, bool f32, int most, bool out, hipStream_t st) {
    const int dx = m3::lin_tile(p.role[0].dx), dz = z_tile(p.role[0].dz, f32, most);
    p.ztiles = 1;
    for (int i = 0; i < p.nroles; ++i) p.ztiles = std::max(p.ztiles, (p.role[i].dz + dz - 1) / dz);
    int32_t share = 1; // heads that have a row in common
    for (int i = 0; i < p.nroles; ++i) share = std::max(share, std::max(p.role[i].xg, std::max(p.role[i].yg, p.role[i].zg)));
    p.hg = m3::lin_head_group(share, p.H, p.nseg, p.ztiles, p.nroles, p.segbits != 0);
    p.group = p.hg * p.ztiles * p.nroles;
    p.nwork = int32_t((p.nseg * (p.H / p.hg) + 7) / 8 * 8 * p.group);
    switch (dx) {
    case 32: return f32 ? m3::launch_linear_f32_32(p, dz, out, st) : m3::launch_linear_bf16_32(p, dz, out, st);
    case 64: return f32 ? m3::launch_linear_f32_64(p, dz, out, st) : m3::launch_linear_bf16_64(p, dz, out, st);
    case 128: return f32 ? m3::launch_linear_f32_128(p, dz, out, st) : m3::launch_linear_bf16_128(p, dz, out, st);
    }
    return hipErrorInvalidValue;
}

// The scans in as few launches as their tile sizes allow.
hipError_t launch_scans(const LinParams &all, int n, bool f32, int most, bool out, hipStream_t st) {
    bool done[3] = {};
    for (int i = 0; i < n; ++i) {
        if (done[i]) continue;
        LinParams p = all;
        p.nroles = 0;
        for (int j = i; j < n; ++j)
            if (!done[j] && m3::lin_tile(all.role[j].dx) == m3::lin_tile(all.role[i].dx) &&
                z_tile(all.role[j].dz, f32, most) == z_tile(all.role[i].dz, f32, most)) {
                p.role[p.nroles++] = all.role[j];
                done[j] = true;
            }
        const hipError_t e = launch_scan(p, f32, most, out, st);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_join(LinParams p, int n, hipStream_t st) {
    p.nroles = n;
    const int64_t area = int64_t(p.role[0].dx) * p.role[0].dz;
    hipLaunchKernelGGL(m3::k_linear_join, dim3(unsigned(p.batch * p.H), unsigned((area + 1023) / 1024), unsigned(n)),
                       dim3(256), 0, st, p);
    return hipGetLastError();
}

// One operand of a scan.
struct Rows {
    const m3_rows_t *r;
    int32_t heads, dim;
    // the tokens' stride also bounds a chunk's rows: a single token's, which may be anything, must not cut its own
    int64_t pitch() const { return std::max<int64_t>(r->token_stride, dim); }
};
void set_x(LinRole &R, const Rows &a, int32_t H) { R.x = a.r->data; R.xt = a.pitch(); R.xh = a.r->head_stride; R.xg = H / a.heads; }
void set_y(LinRole &R, const Rows &a, int32_t H) { R.y = a.r->data; R.yt = a.pitch(); R.yh = a.r->head_stride; R.yg = H / a.heads; }
void set_z(LinRole &R, const Rows &a, int32_t H) { R.z = a.r->data; R.zt = a.pitch(); R.zh = a.r->head_stride; R.zg = H / a.heads; }

LinParams sequences(const m3_linear_shape_t *s, const int32_t *cu, const int32_t *slots, int64_t nstates, const float *ld,
                    const Layout &w) {
    LinParams p{};
    p.H = heads(s);
    p.ztiles = 1;
    p.batch = s->batch;
    p.tokens = s->tokens;
    p.cu = cu;
    p.slots = slots;
    p.nstates = nstates;
    p.log_decay = ld;
    p.each = s->tokens / s->batch;
    p.fold = w.fold;
    while (p.segbits < 30 && w.L >> p.segbits > 1) ++p.segbits;
    p.nseg = w.slots;
    p.sparse = sparse_states(s, w.L);
    return p;
}

m3_status_t check_sequences(const m3_linear_shape_t *s, const float *ld, const int32_t *cu, const int32_t *slots,
                            int64_t nstates, bool states) {
    if (!ld || (reinterpret_cast<uintptr_t>(ld) & 3)) return M3_ERR_INVALID_ARGUMENT;
    if (cu && (reinterpret_cast<uintptr_t>(cu) & 3)) return M3_ERR_INVALID_ARGUMENT;
    if (slots && (reinterpret_cast<uintptr_t>(slots) & 3)) return M3_ERR_INVALID_ARGUMENT;
    if (!cu && s->tokens % s->batch) return M3_ERR_INVALID_ARGUMENT;
    if (nstates < 0 || (states && !slots && nstates < s->batch)) return M3_ERR_INVALID_ARGUMENT;
    return M3_OK;
}

} // namespace

extern "C" {

size_t m3_linear_prefill_workspace_bytes(const m3_linear_shape_t *shape) {
    return check_shape(shape, false) == M3_OK ? prefill_layout(shape).total : 0;
}

size_t m3_linear_prefill_backward_workspace_bytes(const m3_linear_shape_t *shape) {
    return check_shape(shape, false) == M3_OK ? backward_layout(shape).total : 0;
}

m3_status_t m3_linear_plan(const m3_linear_shape_t *shape, int64_t *prefill_segment, int64_t *backward_segment) {
    const m3_status_t sc = check_shape(shape, false);
    if (sc != M3_OK) return sc;
    if (prefill_segment) *prefill_segment = prefill_layout(shape).L;
    if (backward_segment) *backward_segment = backward_layout(shape).L;
    return M3_OK;
}

m3_status_t m3_linear_prefill(const m3_linear_shape_t *shape, const m3_rows_t *q, const m3_rows_t *k,
                              const m3_rows_t *v, const float *log_decay, const int32_t *cu_seqlens,
                              const int32_t *slots, int64_t nstates, const void *init, void *final_state,
                              const m3_rows_t *o, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    m3_status_t sc = check_shape(shape, false);
    if (sc != M3_OK) return sc;
    const int32_t H = heads(shape);
    if (!rows_ok(q, shape->tokens, shape->key_dim) || !rows_ok(k, shape->tokens, shape->key_dim) ||
        !rows_ok(v, shape->tokens, shape->value_dim) ||
        !out_ok(o, shape->tokens, H, shape->value_dim))
        return M3_ERR_INVALID_ARGUMENT;
    sc = check_sequences(shape, log_decay, cu_seqlens, slots, nstates, init || final_state);
    if (sc != M3_OK) return sc;
    if (!aligned16(init) || !aligned16(final_state)) return M3_ERR_INVALID_ARGUMENT;
    const Layout w = prefill_layout(shape);
    if (!workspace || !aligned16(workspace) || workspace_bytes < w.total) return M3_ERR_WORKSPACE;
    const int64_t T = shape->tokens;
    if (starts_in(3, {start(o, T), final_state, workspace, start(q, T), start(k, T), start(v, T), log_decay, cu_seqlens, slots,
                      init == final_state ? nullptr : init}) ||
        starts_in(1, {init, start(o, T), workspace}))
        return M3_ERR_INVALID_ARGUMENT;

    LinParams p = sequences(shape, cu_seqlens, slots, nstates, log_decay, w);
    LinRole &R = p.role[0];
    set_x(R, {q, shape->q_heads, shape->key_dim}, H);
    set_y(R, {k, shape->k_heads, shape->key_dim}, H);
    set_z(R, {v, shape->v_heads, shape->value_dim}, H);
    R.out = o->data;
    R.dx = shape->key_dim;
    R.dz = shape->value_dim;
    R.ot = std::max<int64_t>(o->token_stride, R.dz);
    R.oh = o->head_stride;
    R.a_in = R.a_init = shape->scale;
    R.a_state = 1.f;
    R.init = init;
    R.fin = final_state;
    R.init16 = R.fin16 = shape->state_dtype == M3_DTYPE_BF16;
    R.sm = R.dz;
    R.sn = 1;
    R.seg = static_cast<float *>(workspace);
    const bool f32 = shape->io_dtype == M3_DTYPE_F32;
    if (w.L) {
        if (launch_scans(p, 1, f32, w.most, false, stream) != hipSuccess) return M3_ERR_HIP;
        if (!w.fold && launch_join(p, 1, stream) != hipSuccess) return M3_ERR_HIP;
    }
    return launch_scans(p, 1, f32, w.most, true, stream) == hipSuccess ? M3_OK : M3_ERR_HIP;
}

m3_status_t m3_linear_decode_step(const m3_linear_shape_t *shape, const m3_rows_t *q, const m3_rows_t *k,
                                  const m3_rows_t *v, const float *log_decay, const int32_t *slots, int64_t nstates,
                                  void *state, const m3_rows_t *o, hipStream_t stream) {
    const m3_status_t sc = check_shape(shape, true);
    if (sc != M3_OK) return sc;
    const int32_t H = heads(shape);
    if (!rows_ok(q, shape->batch, shape->key_dim) || !rows_ok(k, shape->batch, shape->key_dim) ||
        !rows_ok(v, shape->batch, shape->value_dim) ||
        !out_ok(o, shape->batch, H, shape->value_dim))
        return M3_ERR_INVALID_ARGUMENT;
    if (!log_decay || (reinterpret_cast<uintptr_t>(log_decay) & 3) || (reinterpret_cast<uintptr_t>(slots) & 3))
        return M3_ERR_INVALID_ARGUMENT;
    if (!state || !aligned16(state) || nstates < 0 || (!slots && nstates < shape->batch)) return M3_ERR_INVALID_ARGUMENT;
    if (starts_in(2, {o->data, state, q->data, k->data, v->data, log_decay, slots})) return M3_ERR_INVALID_ARGUMENT;
    m3::LinStepParams p{};
    p.q = q->data; p.qt = q->token_stride; p.qh = q->head_stride; p.qg = H / shape->q_heads;
    p.k = k->data; p.kt = k->token_stride; p.kh = k->head_stride; p.kg = H / shape->k_heads;
    p.v = v->data; p.vt = v->token_stride; p.vh = v->head_stride; p.vg = H / shape->v_heads;
    p.o = o->data; p.ot = o->token_stride; p.oh = o->head_stride;
    p.state = state;
    p.H = H;
    p.dk = shape->key_dim;
    p.dv = shape->value_dim;
    p.batch = shape->batch;
    p.nstates = nstates;
    p.slots = slots;
    p.log_decay = log_decay;
    p.scale = shape->scale;
    const bool f32 = shape->io_dtype == M3_DTYPE_F32, s16 = shape->state_dtype == M3_DTYPE_BF16;
    const hipError_t e = f32 ? (s16 ? m3::launch_linear_step<float, m3::bf16>(p, stream) : m3::launch_linear_step<float, float>(p, stream))
                             : (s16 ? m3::launch_linear_step<m3::bf16, m3::bf16>(p, stream) : m3::launch_linear_step<m3::bf16, float>(p, stream));
    return e == hipSuccess ? M3_OK : M3_ERR_HIP;
}

m3_status_t m3_linear_prefill_backward(const m3_linear_shape_t *shape, const m3_rows_t *q, const m3_rows_t *k,
                                       const m3_rows_t *v, const float *log_decay, const int32_t *cu_seqlens,
                                       const void *init, const m3_rows_t *go, const float *gfinal,
                                       const m3_rows_t *gq, const m3_rows_t *gk, const m3_rows_t *gv, float *ginit,
                                       void *workspace, size_t workspace_bytes, hipStream_t stream) {
    m3_status_t sc = check_shape(shape, false);
    if (sc != M3_OK) return sc;
    const int32_t H = heads(shape), dk = shape->key_dim, dv = shape->value_dim;
    const int64_t T = shape->tokens;
    if (!rows_ok(q, T, dk) || !rows_ok(k, T, dk) || !rows_ok(v, T, dv) || !rows_ok(go, T, dv) || !out_ok(gq, T, shape->q_heads, dk) ||
        !out_ok(gk, T, shape->k_heads, dk) || !out_ok(gv, T, shape->v_heads, dv))
        return M3_ERR_INVALID_ARGUMENT;
    sc = check_sequences(shape, log_decay, cu_seqlens, nullptr, shape->batch, true);
    if (sc != M3_OK) return sc;
    if (!aligned16(init) || !aligned16(gfinal) || !aligned16(ginit)) return M3_ERR_INVALID_ARGUMENT;
    const Layout w = backward_layout(shape);
    if (!workspace || !aligned16(workspace) || workspace_bytes < w.total) return M3_ERR_WORKSPACE;
    if (starts_in(5, {start(gq, T), start(gk, T), start(gv, T), ginit, workspace, start(q, T), start(k, T), start(v, T), start(go, T),
                      log_decay, cu_seqlens, init, gfinal}))
        return M3_ERR_INVALID_ARGUMENT;
    unsigned char *ws = static_cast<unsigned char *>(workspace);

    LinParams p = sequences(shape, cu_seqlens, nullptr, shape->batch, log_decay, w);
    p.tail = cu_seqlens ? 64 : 0;
    p.grad = 1;
    const Rows rq{q, shape->q_heads, shape->key_dim}, rk{k, shape->k_heads, shape->key_dim}, rv{v, shape->v_heads, shape->value_dim}, rg{go, H, dv};
    const Rows x[3] = {rg, rv, rk}, y[3] = {rv, rg, rq}, z[3] = {rk, rq, rg};
    const m3_rows_t *out[3] = {gq, gk, gv};
    const int32_t out_heads[3] = {shape->q_heads, shape->k_heads, shape->v_heads};
    m3::LinSums sums{};
    for (int i = 0; i < 3; ++i) {
        LinRole &R = p.role[i];
        set_x(R, x[i], H);
        set_y(R, y[i], H);
        set_z(R, z[i], H);
        R.dx = i < 2 ? dv : dk;
        R.dz = i < 2 ? dk : dv;
        if (out_heads[i] < H) {
            R.out = ws + w.part[i];
            R.out32 = 1;
            R.ot = int64_t(H) * R.dz;
            R.oh = R.dz;
            sums.s[sums.n++] = {static_cast<const float *>(R.out), out[i]->data, out[i]->token_stride, out[i]->head_stride,
                                out_heads[i], H / out_heads[i], R.dz};
        } else {
            R.out = out[i]->data;
            R.ot = std::max<int64_t>(out[i]->token_stride, R.dz);
            R.oh = out[i]->head_stride;
        }
        R.rev = i > 0;
        R.a_in = shape->scale;
        R.a_init = i > 0 ? 1.f : shape->scale;
        R.a_state = i > 0 ? shape->scale : 1.f;
        R.init = i > 0 ? static_cast<const void *>(gfinal) : init;
        R.init16 = i == 0 && shape->state_dtype == M3_DTYPE_BF16;
        // the pools hold [key][value]; dq and dk scan with the transposed state
        R.sm = i < 2 ? 1 : dv;
        R.sn = i < 2 ? dv : 1;
        R.seg = reinterpret_cast<float *>(ws + (i > 0 ? w.seg_b : w.seg_f));
        if (i == 2) R.fin = ginit;
    }
    const bool f32 = shape->io_dtype == M3_DTYPE_F32;
    if (w.L) {
        // the state forwards (of k and v) and its gradient backwards (of q and go), as [key][value]
        LinParams a = p;
        a.role[0] = p.role[2];
        set_y(a.role[0], rk, H);
        set_z(a.role[0], rv, H);
        a.role[0].rev = 0;
        a.role[0].a_state = 1.f;
        a.role[0].seg = p.role[0].seg;
        a.role[0].init = p.role[0].init;
        a.role[0].init16 = p.role[0].init16;
        a.role[1] = p.role[2];
        if (launch_scans(a, 2, f32, w.most, false, stream) != hipSuccess) return M3_ERR_HIP;
        if (!w.fold && launch_join(a, 2, stream) != hipSuccess) return M3_ERR_HIP;
    }
    if (launch_scans(p, 3, f32, w.most, true, stream) != hipSuccess) return M3_ERR_HIP;
    if (sums.n && T > 0) {
        sums.seq = p;
        const int64_t n = T * H * (std::max(dk, dv) / 8); // no row has more heads than H
        const dim3 grid(unsigned(std::min<int64_t>(2048, (n + 255) / 256)), unsigned(sums.n));
        if (f32) hipLaunchKernelGGL(m3::k_linear_sum<float>, grid, dim3(256), 0, stream, sums);
        else hipLaunchKernelGGL(m3::k_linear_sum<m3::bf16>, grid, dim3(256), 0, stream, sums);
        if (hipGetLastError() != hipSuccess) return M3_ERR_HIP;
    }
    return M3_OK;
}

} // extern "C"

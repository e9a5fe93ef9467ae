// block_norm.cu -- the norms after and before a block fused with its gate and
// residual scale (zero_block_norm_forward), and their gradient
// (zero_block_norm_backward).
//
//   n = post(h)                                 RMSNorm or LayerNorm, or h itself
//   y = a*x + b * gate[row / rows_per_gate, :] * n
//   u = pre(y)                                  the norm before the next block
//
// with v^ = (v - mean) * r, r = 1/sqrt(mean((v - mean)^2) + eps), mean = 0 for
// RMSNorm, and norm(v) = v^ * w + c.  The gradient, given dy and du:
//
//   g  = dy + J_pre(y)^T du                     J^T d = r*(d*w - m0 - v^*mean(d*w*v^)),
//   dx = a*g                                    m0 = mean(d*w) for LayerNorm, else 0
//   dh = J_post(h)^T (b*gate*g)
//   dgate = sum over its rows of b*g*n,  dw = sum of d*v^,  dc = sum of d
//
// The row statistics are formed again from y and h rather than kept: they
// ride in a reduction that the gradient needs anyhow.
//
// One group of warps holds a row in registers, 8 columns to a thread, reads
// every tensor once and writes every result once: 4 row lengths forward, 6
// backward, HBM-bound (and latency-bound for a few rows).  A thread keeps the
// same columns for all rows of its group, so the sums over rows (dw, dc,
// dgate) stay in its registers in fp32; the groups of a block are added in
// shared memory, and the blocks, whose number depends on the sizes alone, by
// reduce_kernel in order: the same bits in every run.
//
// Rows whose length is no multiple of 8 start at every alignment.  A thread
// then takes the 8 columns of an aligned 16-byte (bf16) or 32-byte (fp32)
// piece of memory, which begin at a column that depends on row*dim mod 8, and
// a group takes only rows that agree in it, so that its columns stay the same.
#include "typed.cuh"
#include "zero_internal.h"

namespace zero {
namespace {

using dev::Bf16;

constexpr int kThreads = 512;        // threads of a block, at most
constexpr int kMaxBlocks = 304;      // backward: two blocks for each of 152 SMs
constexpr int64_t kMaxDim = 16384;   // 512 threads, 4 vectors of 8 columns each
constexpr int kVectors = 4;          // parameter gradients: dw and dc of both norms

struct Geometry {
    int64_t rows, dim, span; // span: rows per gate row
    int32_t threads;         // of a group
    int32_t groups;          // in a block
    int32_t classes;         // rows are dealt by row mod classes (1: aligned, or taken as they are)
    int32_t blocks;
    int64_t run;             // backward: consecutive rows of a worker (of `classes` workers together)
};

struct Params {
    const void *gate, *post_w, *post_b, *pre_w, *pre_b;
    int32_t param_type, gate_type;
    int32_t layer, post, pre;
    float eps, res_scale, branch_scale;
};

// ------------------------------------------------------------- device helpers
struct Group {
    int id, thread, threads, warps, first_warp, buffer;
};

__device__ __forceinline__ Group make_group(int threads)
{
    Group g;
    g.id = static_cast<int>(threadIdx.x) / threads;
    g.thread = static_cast<int>(threadIdx.x) - g.id * threads;
    g.threads = threads;
    g.warps = threads >> 5;
    g.first_warp = g.id * g.warps;
    g.buffer = 0;
    return g;
}

// Sums of kN values over the group's threads, valid in all of them.  Two
// buffers in turn: one is written again only after the barrier of the other's
// use, which every thread reaches after it has read the first.
template <int kN>
__device__ __forceinline__ void group_sum(Group& g, float (&v)[kN])
{
    __shared__ float red[2][kThreads / 32][4];
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v[n] += __shfl_xor_sync(0xFFFFFFFFu, v[n], off);
    if (g.warps == 1) return;
    const int lane = threadIdx.x & 31;
    if (lane == 0) {
#pragma unroll
        for (int n = 0; n < kN; ++n) red[g.buffer][threadIdx.x >> 5][n] = v[n];
    }
    asm volatile("bar.sync %0, %1;" ::"r"(g.id + 1), "r"(g.threads) : "memory");
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        v[n] = lane < g.warps ? red[g.buffer][g.first_warp + lane][n] : 0.0f;
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) v[n] += __shfl_xor_sync(0xFFFFFFFFu, v[n], off);
        v[n] = __shfl_sync(0xFFFFFFFFu, v[n], 0);
    }
    g.buffer ^= 1;
}

// The 8 columns from col of the row that starts at p: columns outside [0, dim)
// are read as 0 and not written.
template <typename T>
__device__ __forceinline__ void load_cols(const T* p, int64_t col, int64_t dim, float (&x)[8])
{
    const T* q = p + col;
    if (col >= 0 && col + 8 <= dim && (reinterpret_cast<uintptr_t>(q) & 15) == 0) {
        dev::load_vec<8>(q, x);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        x[e] = col + e >= 0 && col + e < dim ? dev::load1(q + e) : 0.0f;
}
template <typename T>
__device__ __forceinline__ void store_cols(T* p, int64_t col, int64_t dim, const float (&x)[8])
{
    T* q = p + col;
    if (col >= 0 && col + 8 <= dim && (reinterpret_cast<uintptr_t>(q) & 15) == 0) {
        dev::store8(q, x);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (col + e >= 0 && col + e < dim) dev::store1(q + e, x[e]);
}
__device__ __forceinline__ void load_cols_any(const void* p, int32_t type, int64_t row,
                                              int64_t col, int64_t dim, float absent,
                                              float (&x)[8])
{
    if (!p) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = absent;
    } else if (type == ZERO_TYPE_BF16) {
        load_cols(static_cast<const Bf16*>(p) + row * dim, col, dim, x);
    } else {
        load_cols(static_cast<const float*>(p) + row * dim, col, dim, x);
    }
}

// Mean (0 for RMSNorm) and 1/sqrt(variance + eps) of a row.  LayerNorm's
// variance is taken about the mean in a second sum: the one-pass form
// mean(v^2) - mean^2 loses the digits that a large mean takes.
template <int kNV>
__device__ __forceinline__ void row_stats(Group& g, const float (&v)[kNV][8],
                                          const bool (&in)[kNV][8], int64_t dim, bool layer,
                                          float eps, float& mean, float& rstd)
{
    const float inv = 1.0f / static_cast<float>(dim);
    mean = 0.0f;
    if (layer) {
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < kNV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] += v[i][e];
        group_sum(g, s);
        mean = s[0] * inv;
    }
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = in[i][e] ? v[i][e] - mean : 0.0f;
            s[0] = fmaf(d, d, s[0]);
        }
    group_sum(g, s);
    rstd = 1.0f / sqrtf(fmaf(s[0], inv, eps));
}

// ------------------------------------------------------------------ forward
template <int kNV, typename Act, typename Res>
__global__ void __launch_bounds__(kThreads)
forward_kernel(const Geometry G, const Params P, const Res* __restrict__ x,
               const Act* __restrict__ h, Res* __restrict__ y, Act* __restrict__ u)
{
    Group g = make_group(G.threads);
    const int64_t worker = static_cast<int64_t>(blockIdx.x) * G.groups + g.id;
    const int64_t workers = static_cast<int64_t>(G.blocks) * G.groups / G.classes * G.classes;
    if (worker >= workers) return;
    const int64_t shift = G.classes == 1 ? 0 : worker % G.classes * G.dim % 8;
    int64_t col[kNV];
    bool in[kNV][8];
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        col[i] = (g.thread + static_cast<int64_t>(i) * g.threads) * 8 - shift;
#pragma unroll
        for (int e = 0; e < 8; ++e) in[i][e] = col[i] + e >= 0 && col[i] + e < G.dim;
    }
    for (int64_t row = worker; row < G.rows; row += workers) {
        float v[kNV][8];
#pragma unroll
        for (int i = 0; i < kNV; ++i) load_cols(x + row * G.dim, col[i], G.dim, v[i]);
        if (h) {
            float n[kNV][8];
#pragma unroll
            for (int i = 0; i < kNV; ++i) load_cols(h + row * G.dim, col[i], G.dim, n[i]);
            if (P.post) {
                float mean, rstd;
                row_stats(g, n, in, G.dim, P.layer, P.eps, mean, rstd);
#pragma unroll
                for (int i = 0; i < kNV; ++i) {
                    float w[8], c[8];
                    load_cols_any(P.post_w, P.param_type, 0, col[i], G.dim, 1.0f, w);
                    load_cols_any(P.post_b, P.param_type, 0, col[i], G.dim, 0.0f, c);
#pragma unroll
                    for (int e = 0; e < 8; ++e) n[i][e] = fmaf((n[i][e] - mean) * rstd, w[e], c[e]);
                }
            }
            const int64_t gate_row = P.gate ? row / G.span : 0;
#pragma unroll
            for (int i = 0; i < kNV; ++i) {
                float t[8];
                load_cols_any(P.gate, P.gate_type, gate_row, col[i], G.dim, 1.0f, t);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[i][e] = fmaf(P.res_scale, v[i][e], P.branch_scale * t[e] * n[i][e]);
                if (y) store_cols(y + row * G.dim, col[i], G.dim, v[i]);
            }
        }
        if (P.pre) {
            float mean, rstd;
            row_stats(g, v, in, G.dim, P.layer, P.eps, mean, rstd);
#pragma unroll
            for (int i = 0; i < kNV; ++i) {
                float w[8], c[8];
                load_cols_any(P.pre_w, P.param_type, 0, col[i], G.dim, 1.0f, w);
                load_cols_any(P.pre_b, P.param_type, 0, col[i], G.dim, 0.0f, c);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] = fmaf((v[i][e] - mean) * rstd, w[e], c[e]);
                store_cols(u + row * G.dim, col[i], G.dim, v[i]);
            }
        }
    }
}

// ----------------------------------------------------------------- backward
// Partial sums in the scratch: [blocks][vectors in use][dim] of the sums over
// all rows, then, with several gate rows, [workers][2][dim] of the gate rows
// that a worker shares with others: its first one, and its last one.
struct Grads {
    void *dgate;
    int32_t dgate_type;
    int32_t gate_rows;   // 0: no dgate wanted
    int32_t vectors;     // sums over all rows: kVectors, and the gate's where it has one row
    float* partial;
    float* gate_partial;
};

template <int kNV, typename Act, typename Res>
__global__ void __launch_bounds__(kThreads)
backward_kernel(const Geometry G, const Params P, const Grads D, const Res* __restrict__ dy,
                const Act* __restrict__ du, const Res* __restrict__ y, const Act* __restrict__ h,
                Res* __restrict__ dx, Act* __restrict__ dh)
{
    extern __shared__ float combine[]; // groups x dim, where a block has several groups
    Group g = make_group(G.threads);
    const int64_t worker = static_cast<int64_t>(blockIdx.x) * G.groups + g.id;
    const int64_t strip = worker / G.classes; // workers of a strip share its rows by class
    const int64_t cls = worker - strip * G.classes;
    const int64_t lo = strip * G.run + cls;
    int64_t hi = strip * G.run + G.run;
    if (hi > G.rows) hi = G.rows;
    const int64_t shift = G.classes == 1 ? 0 : cls * G.dim % 8;
    const float inv = 1.0f / static_cast<float>(G.dim);
    int64_t col[kNV];
    bool in[kNV][8];
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        col[i] = (g.thread + static_cast<int64_t>(i) * g.threads) * 8 - shift;
#pragma unroll
        for (int e = 0; e < 8; ++e) in[i][e] = col[i] + e >= 0 && col[i] + e < G.dim;
    }
    float sums[kVectors + 1][kNV][8]; // dw, dc of post, dw, dc of pre, dgate
#pragma unroll
    for (int a = 0; a <= kVectors; ++a)
#pragma unroll
        for (int i = 0; i < kNV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) sums[a][i][e] = 0.0f;

    const bool by_rows = D.gate_rows > 1;
    int64_t gate_row = P.gate && lo < hi ? lo / G.span : 0;
    const int64_t first_gate = gate_row;
    // The sum of one gate row: final where this worker has all its rows.
    auto leave_gate = [&] {
        const int64_t from = gate_row * G.span;
        const int64_t to = from + G.span < G.rows ? from + G.span : G.rows;
        const bool whole = G.classes == 1 ? from >= lo && to <= hi : to - from == 1;
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            if (whole) {
                if (D.dgate_type == ZERO_TYPE_BF16)
                    store_cols(static_cast<Bf16*>(D.dgate) + gate_row * G.dim, col[i], G.dim,
                               sums[kVectors][i]);
                else
                    store_cols(static_cast<float*>(D.dgate) + gate_row * G.dim, col[i], G.dim,
                               sums[kVectors][i]);
            } else {
                const int slot = gate_row == first_gate ? 0 : 1;
                store_cols(D.gate_partial + (2 * worker + slot) * G.dim, col[i], G.dim,
                           sums[kVectors][i]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sums[kVectors][i][e] = 0.0f;
        }
    };

    for (int64_t row = lo; row < hi; row += G.classes) {
        if (P.gate && row / G.span != gate_row) {
            if (by_rows) leave_gate();
            gate_row = row / G.span;
        }
        float t[kNV][8]; // the gradient that arrives at y
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            if (dy)
                load_cols(dy + row * G.dim, col[i], G.dim, t[i]);
            else
#pragma unroll
                for (int e = 0; e < 8; ++e) t[i][e] = 0.0f;
        }
        if (P.pre) {
            float v[kNV][8], d[kNV][8];
#pragma unroll
            for (int i = 0; i < kNV; ++i) {
                load_cols(y + row * G.dim, col[i], G.dim, v[i]);
                load_cols(du + row * G.dim, col[i], G.dim, d[i]);
            }
            float mean, rstd, m[2] = {0.0f, 0.0f};
            row_stats(g, v, in, G.dim, P.layer, P.eps, mean, rstd);
#pragma unroll
            for (int i = 0; i < kNV; ++i) {
                float w[8];
                load_cols_any(P.pre_w, P.param_type, 0, col[i], G.dim, 1.0f, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    v[i][e] = in[i][e] ? (v[i][e] - mean) * rstd : 0.0f;
                    sums[2][i][e] = fmaf(d[i][e], v[i][e], sums[2][i][e]);
                    sums[3][i][e] += d[i][e];
                    d[i][e] *= w[e];
                    m[0] += d[i][e];
                    m[1] = fmaf(d[i][e], v[i][e], m[1]);
                }
            }
            group_sum(g, m);
            const float m0 = P.layer ? m[0] * inv : 0.0f, m1 = m[1] * inv;
#pragma unroll
            for (int i = 0; i < kNV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    t[i][e] = fmaf(rstd, d[i][e] - m0 - v[i][e] * m1, t[i][e]);
        }
        if (dx) {
#pragma unroll
            for (int i = 0; i < kNV; ++i) {
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = P.res_scale * t[i][e];
                store_cols(dx + row * G.dim, col[i], G.dim, o);
            }
        }
        if (!h) continue;
        float n[kNV][8];
#pragma unroll
        for (int i = 0; i < kNV; ++i) load_cols(h + row * G.dim, col[i], G.dim, n[i]);
        float mean = 0.0f, rstd = 1.0f, m[2] = {0.0f, 0.0f};
        if (P.post) row_stats(g, n, in, G.dim, P.layer, P.eps, mean, rstd);
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            float w[8], c[8], s[8];
            load_cols_any(P.post_w, P.param_type, 0, col[i], G.dim, 1.0f, w);
            load_cols_any(P.post_b, P.param_type, 0, col[i], G.dim, 0.0f, c);
            load_cols_any(P.gate, P.gate_type, gate_row, col[i], G.dim, 1.0f, s);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = P.branch_scale * t[i][e];
                n[i][e] = in[i][e] ? (n[i][e] - mean) * rstd : 0.0f;
                sums[kVectors][i][e] = fmaf(d, fmaf(n[i][e], w[e], c[e]), sums[kVectors][i][e]);
                const float dn = d * s[e];
                sums[0][i][e] = fmaf(dn, n[i][e], sums[0][i][e]);
                sums[1][i][e] += dn;
                t[i][e] = dn * w[e];
                m[0] += t[i][e];
                m[1] = fmaf(t[i][e], n[i][e], m[1]);
            }
        }
        float m0 = 0.0f, m1 = 0.0f;
        if (P.post) {
            group_sum(g, m);
            m0 = P.layer ? m[0] * inv : 0.0f;
            m1 = m[1] * inv;
        }
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) t[i][e] = rstd * (t[i][e] - m0 - n[i][e] * m1);
            store_cols(dh + row * G.dim, col[i], G.dim, t[i]);
        }
    }
    if (by_rows && lo < hi) leave_gate();

    // The block's sums, its groups added in order.
#pragma unroll
    for (int a = 0; a <= kVectors; ++a) {
        if (a >= D.vectors) break;
        float* out = D.partial + (static_cast<int64_t>(blockIdx.x) * D.vectors + a) * G.dim;
        if (G.groups == 1) {
#pragma unroll
            for (int i = 0; i < kNV; ++i) store_cols(out, col[i], G.dim, sums[a][i]);
            continue;
        }
        __syncthreads();
        if (g.id < G.groups) {
#pragma unroll
            for (int i = 0; i < kNV; ++i)
                store_cols(combine + g.id * G.dim, col[i], G.dim, sums[a][i]);
        }
        __syncthreads();
        for (int64_t c = threadIdx.x; c < G.dim; c += blockDim.x) {
            float total = 0.0f;
            for (int k = 0; k < G.groups; ++k) total += combine[k * G.dim + c];
            out[c] = total;
        }
    }
}

// Sums the blocks' partials (blockIdx.y < vectors) and the shared gate rows'.
// 32 columns x kSlices threads; a slice adds a run of the partials in order,
// the slices are added in order.
constexpr int kSlices = 8;

struct Finals {
    void* out[kVectors + 1];
    int32_t type[kVectors + 1];
};

__global__ void __launch_bounds__(32 * kSlices)
reduce_kernel(const Geometry G, const Grads D, const Finals F)
{
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    __shared__ float sums[kSlices][32];
    const int64_t tasks = D.vectors + (D.gate_rows > 1 ? D.gate_rows : 0);
    for (int64_t task = blockIdx.y; task < tasks; task += gridDim.y) {
        const float* src;
        int64_t first, count, step;
        void* out;
        int32_t type;
        float acc = 0.0f;
        if (task < D.vectors) {
            out = F.out[task];
            type = F.type[task];
            if (!out) continue;
            src = D.partial + task * G.dim;
            first = 0;
            count = G.blocks;
            step = D.vectors * G.dim;
        } else {
            const int64_t q = task - D.vectors; // gate row
            const int64_t from = q * G.span;
            const int64_t to = from + G.span < G.rows ? from + G.span : G.rows;
            if (G.classes != 1) continue; // rows of one token: final already
            first = from / G.run;
            count = (to - 1) / G.run - first + 1;
            if (count == 1) continue; // one worker's: final already
            src = D.gate_partial;
            step = 2 * G.dim;
            // the first worker holds it as its last row, unless it is its first too
            if (slice == 0 && first * G.run / G.span != q) {
                if (col < G.dim) acc = src[(2 * first + 1) * G.dim + col];
                ++first;
                --count;
            } else if (first * G.run / G.span != q) {
                ++first;
                --count;
            }
            out = static_cast<char*>(D.dgate) +
                  q * G.dim * (D.dgate_type == ZERO_TYPE_BF16 ? 2 : 4);
            type = D.dgate_type;
        }
        const int64_t per = (count + kSlices - 1) / kSlices;
        const int64_t lo = slice * per, hi = lo + per < count ? lo + per : count;
        if (col < G.dim) {
#pragma unroll 4
            for (int64_t k = lo; k < hi; ++k) acc += src[(first + k) * step + col];
        }
        __syncthreads();
        sums[slice][lane] = acc;
        __syncthreads();
        if (slice == 0 && col < G.dim) {
            float total[1] = {0.0f};
#pragma unroll
            for (int s = 0; s < kSlices; ++s) total[0] += sums[s][lane];
            dev::store_any<1>(out, type, col, total);
        }
    }
}

// --------------------------------------------------------------------- host
bool sizes_ok(int64_t rows, int64_t dim, int64_t span)
{
    return rows >= 0 && rows <= (int64_t(1) << 40) && dim >= 1 && dim <= kMaxDim && span >= 1;
}

// aligned: every row tensor starts at a multiple of 16 bytes.
Geometry geometry(int64_t rows, int64_t dim, int64_t span, bool aligned, bool backward)
{
    Geometry G = {};
    G.rows = rows;
    G.dim = dim;
    G.span = span < rows ? span : (rows > 0 ? rows : 1);
    G.classes = 1;
    if (dim % 8 != 0 && aligned && dim + 7 <= kMaxDim &&
        (!backward || G.span == 1 || G.span >= rows))
        G.classes = dim % 4 == 0 ? 2 : dim % 2 == 0 ? 4 : 8;
    const int64_t vecs = (dim + (G.classes > 1 ? 7 : 0) + 7) / 8;
    const int64_t per_thread = vecs <= kThreads ? 1 : vecs <= 2 * kThreads ? 2 : 4;
    const int64_t lanes = (vecs + per_thread - 1) / per_thread;
    G.threads = static_cast<int32_t>((lanes + 31) / 32 * 32);
    G.groups = kThreads / G.threads;
    if (G.groups > 15 && G.threads > 32) G.groups = 15;
    while (G.groups > 1 && (rows + G.groups - 1) / G.groups < kMaxBlocks) G.groups /= 2;
    int64_t blocks = (rows + G.groups - 1) / G.groups;
    if (blocks > kMaxBlocks) blocks = kMaxBlocks;
    if (blocks < 1) blocks = 1;
    if (G.classes > 1) { // at least one worker of each class
        while (blocks * G.groups < G.classes) ++blocks;
    }
    G.blocks = static_cast<int32_t>(blocks);
    const int64_t strips = blocks * G.groups / G.classes;
    const int64_t run = (rows + strips - 1) / strips;
    G.run = (run + G.classes - 1) / G.classes * G.classes;
    if (G.run < 1) G.run = G.classes;
    return G;
}

int vectors_per_thread(const Geometry& G)
{
    const int64_t vecs = (G.dim + (G.classes > 1 ? 7 : 0) + 7) / 8;
    return vecs <= kThreads ? 1 : vecs <= 2 * kThreads ? 2 : 4;
}

// Scratch of the larger of the two shapes that the pointers' alignment may give.
int64_t scratch_floats(int64_t rows, int64_t dim, int64_t span)
{
    int64_t most = 0;
    for (int aligned = 0; aligned < 2; ++aligned) {
        const Geometry G = geometry(rows, dim, span, aligned != 0, true);
        const int64_t n = static_cast<int64_t>(G.blocks) * (kVectors + 1) * dim +
                          (G.span < rows ? static_cast<int64_t>(G.blocks) * G.groups * 2 * dim : 0);
        if (n > most) most = n;
    }
    return most;
}

int check_block(const zero_block_norm_t* n, const void* branch, const void* gate,
                const void* post_w, const void* post_b, const void* pre_w, const void* pre_b)
{
    if (!n || !sizes_ok(n->n_rows, n->dim, n->rows_per_gate) || !float_type(n->act_type) ||
        !float_type(n->res_type) || !float_type(n->param_type) || !float_type(n->gate_type) ||
        (n->act_type == ZERO_TYPE_F32 && n->res_type != ZERO_TYPE_F32) ||
        (n->kind != ZERO_NORM_RMS && n->kind != ZERO_NORM_LAYER) ||
        (n->post_norm != 0 && n->post_norm != 1) || (n->pre_norm != 0 && n->pre_norm != 1))
        return ZERO_EINVAL;
    if (!std::isfinite(n->eps) || n->eps <= 0 || static_cast<float>(n->eps) <= 0 ||
        !std::isfinite(n->residual_scale) || !std::isfinite(n->branch_scale))
        return ZERO_EINVAL;
    // with no rows the tensors of rows may have no address
    if (n->n_rows > 0 && !branch && (n->post_norm || gate || !n->pre_norm)) return ZERO_EINVAL;
    if ((!n->post_norm && (post_w || post_b)) || (!n->pre_norm && (pre_w || pre_b)))
        return ZERO_EINVAL;
    const int pb = type_bytes(n->param_type);
    if (!aligned_to(post_w, pb) || !aligned_to(post_b, pb) || !aligned_to(pre_w, pb) ||
        !aligned_to(pre_b, pb) || !aligned_to(gate, type_bytes(n->gate_type)))
        return ZERO_EALIGN;
    return ZERO_OK;
}

Params make_params(const zero_block_norm_t* n, const void* gate, const void* post_w,
                   const void* post_b, const void* pre_w, const void* pre_b)
{
    Params P = {};
    P.gate = gate;
    P.post_w = post_w;
    P.post_b = post_b;
    P.pre_w = pre_w;
    P.pre_b = pre_b;
    P.param_type = n->param_type;
    P.gate_type = n->gate_type;
    P.layer = n->kind == ZERO_NORM_LAYER;
    P.post = n->post_norm;
    P.pre = n->pre_norm;
    P.eps = static_cast<float>(n->eps);
    P.res_scale = static_cast<float>(n->residual_scale);
    P.branch_scale = static_cast<float>(n->branch_scale);
    return P;
}

template <typename Act, typename Res>
int launch_forward(const Geometry& G, const Params& P, const void* x, const void* h, void* y,
                   void* u, cudaStream_t stream)
{
    const auto* xp = static_cast<const Res*>(x);
    const auto* hp = static_cast<const Act*>(h);
    auto* yp = static_cast<Res*>(y);
    auto* up = static_cast<Act*>(u);
    const dim3 grid(static_cast<unsigned>(G.blocks)), block(static_cast<unsigned>(G.threads * G.groups));
    switch (vectors_per_thread(G)) {
    case 1: forward_kernel<1, Act, Res><<<grid, block, 0, stream>>>(G, P, xp, hp, yp, up); break;
    case 2: forward_kernel<2, Act, Res><<<grid, block, 0, stream>>>(G, P, xp, hp, yp, up); break;
    default: forward_kernel<4, Act, Res><<<grid, block, 0, stream>>>(G, P, xp, hp, yp, up);
    }
    return cuda_status(cudaGetLastError());
}

template <typename Act, typename Res>
int launch_backward(const Geometry& G, const Params& P, const Grads& D, const void* dy,
                    const void* du, const void* y, const void* h, void* dx, void* dh,
                    cudaStream_t stream)
{
    const auto* dyp = static_cast<const Res*>(dy);
    const auto* dup = static_cast<const Act*>(du);
    const auto* yp = static_cast<const Res*>(y);
    const auto* hp = static_cast<const Act*>(h);
    auto* dxp = static_cast<Res*>(dx);
    auto* dhp = static_cast<Act*>(dh);
    const dim3 grid(static_cast<unsigned>(G.blocks)), block(static_cast<unsigned>(G.threads * G.groups));
    const size_t smem = G.groups > 1 ? static_cast<size_t>(G.groups) * G.dim * sizeof(float) : 0;
    switch (vectors_per_thread(G)) {
    case 1:
        backward_kernel<1, Act, Res><<<grid, block, smem, stream>>>(G, P, D, dyp, dup, yp, hp, dxp, dhp);
        break;
    case 2:
        backward_kernel<2, Act, Res><<<grid, block, smem, stream>>>(G, P, D, dyp, dup, yp, hp, dxp, dhp);
        break;
    default:
        backward_kernel<4, Act, Res><<<grid, block, smem, stream>>>(G, P, D, dyp, dup, yp, hp, dxp, dhp);
    }
    return cuda_status(cudaGetLastError());
}

} // namespace
} // namespace zero

using namespace zero;

extern "C" int zero_block_norm_forward(const zero_block_norm_t* norm, const void* x,
                                       const void* branch, const void* gate,
                                       const void* post_weight, const void* post_bias,
                                       const void* pre_weight, const void* pre_bias, void* y,
                                       void* u, cudaStream_t stream)
{
    const int rc = check_block(norm, branch, gate, post_weight, post_bias, pre_weight, pre_bias);
    if (rc != ZERO_OK) return rc;
    if (norm->n_rows == 0) return ZERO_OK;
    if ((branch != nullptr) != (y != nullptr) || (norm->pre_norm != 0) != (u != nullptr))
        return ZERO_EINVAL;
    if (!x) return ZERO_EINVAL;
    const int ab = type_bytes(norm->act_type), rb = type_bytes(norm->res_type);
    if (!aligned_to(x, rb) || !aligned_to(y, rb) || !aligned_to(branch, ab) || !aligned_to(u, ab))
        return ZERO_EALIGN;
    const Geometry G = geometry(norm->n_rows, norm->dim, norm->rows_per_gate,
                                aligned16(x) && aligned16(branch) && aligned16(y) && aligned16(u),
                                false);
    const Params P = make_params(norm, gate, post_weight, post_bias, pre_weight, pre_bias);
    if (norm->act_type == ZERO_TYPE_F32)
        return launch_forward<float, float>(G, P, x, branch, y, u, stream);
    if (norm->res_type == ZERO_TYPE_F32)
        return launch_forward<Bf16, float>(G, P, x, branch, y, u, stream);
    return launch_forward<Bf16, Bf16>(G, P, x, branch, y, u, stream);
}

extern "C" int64_t zero_block_norm_scratch_bytes(int64_t n_rows, int64_t dim,
                                                 int64_t rows_per_gate)
{
    if (!sizes_ok(n_rows, dim, rows_per_gate)) return ZERO_EINVAL;
    return scratch_floats(n_rows, dim, rows_per_gate) * static_cast<int64_t>(sizeof(float));
}

extern "C" int zero_block_norm_backward(const zero_block_norm_t* norm, const void* dy,
                                        const void* du, const void* y, const void* branch,
                                        const void* gate, const void* post_weight,
                                        const void* post_bias, const void* pre_weight, void* dx,
                                        void* dbranch, const zero_block_norm_grads_t* grads,
                                        void* scratch, int64_t scratch_bytes, cudaStream_t stream)
{
    const int rc = check_block(norm, branch, gate, post_weight, post_bias, pre_weight, nullptr);
    if (rc != ZERO_OK) return rc;
    if (!grads || !scratch || !float_type(grads->grad_type) || !float_type(grads->dgate_type))
        return ZERO_EINVAL;
    if ((grads->dgate && !gate) ||
        (!norm->post_norm && (grads->dpost_weight || grads->dpost_bias)) ||
        (!norm->pre_norm && (grads->dpre_weight || grads->dpre_bias)))
        return ZERO_EINVAL;
    if (norm->n_rows > 0 &&
        ((norm->pre_norm != 0) != (du != nullptr) || (branch != nullptr) != (dbranch != nullptr) ||
         (!dy && !du) || (norm->pre_norm && !y)))
        return ZERO_EINVAL;
    if (scratch_bytes < zero_block_norm_scratch_bytes(norm->n_rows, norm->dim, norm->rows_per_gate))
        return ZERO_EINVAL;
    const int ab = type_bytes(norm->act_type), rb = type_bytes(norm->res_type);
    const int gb = type_bytes(grads->grad_type);
    if (!aligned_to(dy, rb) || !aligned_to(y, rb) || !aligned_to(dx, rb) || !aligned_to(du, ab) ||
        !aligned_to(branch, ab) || !aligned_to(dbranch, ab) || !aligned16(scratch) ||
        !aligned_to(grads->dpost_weight, gb) || !aligned_to(grads->dpost_bias, gb) ||
        !aligned_to(grads->dpre_weight, gb) || !aligned_to(grads->dpre_bias, gb) ||
        !aligned_to(grads->dgate, type_bytes(grads->dgate_type)))
        return ZERO_EALIGN;
    const Geometry G = geometry(norm->n_rows, norm->dim, norm->rows_per_gate,
                                aligned16(dy) && aligned16(du) && aligned16(y) &&
                                    aligned16(branch) && aligned16(dx) && aligned16(dbranch),
                                true);
    const Params P = make_params(norm, gate, post_weight, post_bias, pre_weight, nullptr);
    const int64_t gate_rows = (norm->n_rows + G.span - 1) / G.span;
    if (gate_rows > 0x7FFFFFFF) return ZERO_EINVAL;
    Grads D = {};
    D.dgate = grads->dgate;
    D.dgate_type = grads->dgate_type;
    D.gate_rows = grads->dgate ? static_cast<int32_t>(gate_rows > 0 ? gate_rows : 1) : 0;
    D.vectors = D.gate_rows == 1 ? kVectors + 1 : kVectors;
    D.partial = static_cast<float*>(scratch);
    D.gate_partial = D.partial + static_cast<int64_t>(G.blocks) * (kVectors + 1) * G.dim;
    int status;
    if (norm->act_type == ZERO_TYPE_F32)
        status = launch_backward<float, float>(G, P, D, dy, du, y, branch, dx, dbranch, stream);
    else if (norm->res_type == ZERO_TYPE_F32)
        status = launch_backward<Bf16, float>(G, P, D, dy, du, y, branch, dx, dbranch, stream);
    else
        status = launch_backward<Bf16, Bf16>(G, P, D, dy, du, y, branch, dx, dbranch, stream);
    if (status != ZERO_OK) return status;
    Finals F = {};
    F.out[0] = grads->dpost_weight;
    F.out[1] = grads->dpost_bias;
    F.out[2] = grads->dpre_weight;
    F.out[3] = grads->dpre_bias;
    F.out[4] = grads->dgate;
    for (int i = 0; i < kVectors; ++i) F.type[i] = grads->grad_type;
    F.type[kVectors] = grads->dgate_type;
    const int64_t tasks = D.vectors + (D.gate_rows > 1 ? D.gate_rows : 0);
    const dim3 grid(static_cast<unsigned>((G.dim + 31) / 32),
                    static_cast<unsigned>(tasks < 1024 ? tasks : 1024));
    reduce_kernel<<<grid, 32 * kSlices, 0, stream>>>(G, D, F);
    return cuda_status(cudaGetLastError());
}

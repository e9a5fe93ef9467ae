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
// backward, so HBM bounds it if the exchanges between a row's warps are kept few
// and other rows are under way meanwhile.  A thread keeps the same columns for
// all rows of its group, so the sums over rows (dw, dc, dgate) stay in its
// registers in fp32; the groups of a block are added in shared memory, and the
// blocks, whose number depends on the sizes alone, by reduce_kernel in order:
// the same bits in every run.
//
// Measured (device time, one GB300): forward 16384 x 4096 bf16 91 us, 5.9 TB/s, of
// 345 us with one row's loads, weights and exchanges after another; backward
// 16384 x 2048 with an fp32 residual 105 us, 5.8 TB/s (288 at first), 16384 x 4096
// bf16 159 us (a gate row for each token 390: 268 MB more, and a row at a time);
// 8191 x 768 LayerNorm with biases 32 us, of which 11 are the two
// launches, their first loads and the sums over blocks, and the rest is bound by
// instructions (three exchanges a row); a single row 3.7 us forward.  dim above 4096
// backward (one row at a time) and above 8192 at all does not fit the registers:
// 8192 x 8192 RMS forward 93 us, backward 328 (240 to 480 bytes of stack a thread; LayerNorm
// 132 and 576, up to 856 bytes), 8192 x 16384 968 and 3353 us (1.0 to 2.4 KB).
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
constexpr int kMaxBlocks = 304;      // forward: two blocks for each of 152 SMs
constexpr int kMaxPlainBlocks = 456; // forward, 80 registers: three blocks of 256 threads
constexpr int kMaxBackBlocks = 152;  // backward: its registers fill an SM with one block
constexpr int64_t kMaxDim = 16384;   // 512 threads, 4 vectors of 8 columns each
constexpr int kVectors = 4;          // parameter gradients: dw and dc of both norms

struct Geometry {
    int64_t rows, dim, span; // span: rows per gate row
    int32_t threads;         // of a group
    int32_t groups;          // in a block
    int32_t classes;         // rows are dealt by row mod classes (1: aligned, or taken as they are)
    int32_t wide;            // rows start (with their class) at 16-byte boundaries
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

// Sums of kN (1, 2 or 4) values over the group's threads, valid in all of
// them.  In a warp, kN values are halved along the first steps: a lane keeps
// half of them and gives the other half away, so that the 4 sums cost 6
// shuffles, not 20.  Across warps: one word per warp and value.  Two buffers in
// turn: one is written again only after the barrier of the other's use, which
// every thread reaches after it has read the first.
constexpr int kMaxWarps = kThreads / 32;

template <int kN>
__device__ __forceinline__ void group_sum(Group& g, float (&v)[kN])
{
    static_assert(kN == 1 || kN == 2 || kN == 4, "");
    constexpr uint32_t kAll = 0xFFFFFFFFu;
    __shared__ __align__(16) float red[2][kMaxWarps * kN];
    const int lane = threadIdx.x & 31;
    float mine; // the sum of value (lane >> 3) & 3, lane >> 4 or 0 over this lane's part
    if constexpr (kN == 1) {
        mine = v[0];
        mine += __shfl_xor_sync(kAll, mine, 16);
        mine += __shfl_xor_sync(kAll, mine, 8);
    } else if constexpr (kN == 2) {
        const bool up = lane & 16;
        mine = (up ? v[1] : v[0]) + __shfl_xor_sync(kAll, up ? v[0] : v[1], 16);
        mine += __shfl_xor_sync(kAll, mine, 8);
    } else {
        const bool up = lane & 16, odd = lane & 8;
        const float a = (up ? v[2] : v[0]) + __shfl_xor_sync(kAll, up ? v[0] : v[2], 16);
        const float b = (up ? v[3] : v[1]) + __shfl_xor_sync(kAll, up ? v[1] : v[3], 16);
        mine = (odd ? b : a) + __shfl_xor_sync(kAll, odd ? a : b, 8);
    }
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) mine += __shfl_xor_sync(kAll, mine, off);
    constexpr int kLanes = 32 / kN; // lanes that hold a value's sum
    if (g.warps > 1) {
        float* buf = red[g.buffer] + g.first_warp * kN;
        if (lane % kLanes == 0) buf[(lane / kLanes) * g.warps + (threadIdx.x >> 5) - g.first_warp] = mine;
        asm volatile("bar.sync %0, %1;" ::"r"(g.id + 1), "r"(g.threads) : "memory");
        // value n's warps by its kLanes lanes
        const float* of = buf + (lane / kLanes) * g.warps;
        mine = 0.0f;
#pragma unroll
        for (int w = 0; w < kMaxWarps; w += kLanes) {
            const int at = w + lane % kLanes;
            if (at < g.warps) mine += of[at];
        }
#pragma unroll
        for (int off = (kLanes < kMaxWarps ? kLanes : kMaxWarps) / 2; off > 0; off >>= 1)
            mine += __shfl_xor_sync(kAll, mine, off);
        g.buffer ^= 1;
    }
#pragma unroll
    for (int n = 0; n < kN; ++n) v[n] = __shfl_sync(kAll, mine, n * kLanes);
}

// The 8 columns from col of the row that starts at p, as loaded.  full: they
// all lie in the row, at a multiple of 16 bytes; else those inside are read
// one by one and the others are 0.
__device__ __forceinline__ void edge_cols(const Bf16* p, int col, int dim, dev::Raw8<Bf16>& r)
{
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int c = col + 2 * e;
        const uint32_t lo = c >= 0 && c < dim ? p[c].bits : 0u;
        const uint32_t hi = c + 1 >= 0 && c + 1 < dim ? p[c + 1].bits : 0u;
        w[e] = lo | (hi << 16);
    }
    r.a = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void edge_cols(const float* p, int col, int dim, dev::Raw8<float>& r)
{
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = col + e >= 0 && col + e < dim ? p[col + e] : 0.0f;
    r.a = make_float4(x[0], x[1], x[2], x[3]);
    r.b = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void clear(dev::Raw8<Bf16>& r) { r.a = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void clear(dev::Raw8<float>& r)
{
    r.a = r.b = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
}
__device__ __forceinline__ float part(const float2 (&x)[4], int e)
{
    return e & 1 ? x[e >> 1].y : x[e >> 1].x;
}
template <typename T>
__device__ __forceinline__ void store_edge(T* p, int col, int dim, const float2 (&x)[4])
{
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (col + e >= 0 && col + e < dim) dev::store1(p + col + e, part(x, e));
}
// 16 bytes at once where the address allows.
template <typename T>
__device__ __forceinline__ void store_cols(T* p, int col, int dim, const float2 (&x)[4])
{
    if ((reinterpret_cast<uintptr_t>(p + col) & 15) == 0 && col >= 0 && col + 8 <= dim)
        dev::store8_stream(p + col, x);
    else
        store_edge(p, col, dim, x);
}
// Weights, biases and gate rows: read seldom, at any alignment.
__device__ __forceinline__ void load_vector(const void* p, int32_t type, int64_t row, int col,
                                            int dim, float absent, float2 (&x)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = dev::pair(absent);
    if (!p) return;
    const int64_t at = row * dim + col;
    if (type == ZERO_TYPE_BF16) {
        const Bf16* q = static_cast<const Bf16*>(p) + at;
        dev::Raw8<Bf16> r;
        if (col >= 0 && col + 8 <= dim && (reinterpret_cast<uintptr_t>(q) & 15) == 0)
            dev::load_raw8(q, r);
        else
            edge_cols(q - col, col, dim, r);
        dev::unpack8(r, x);
    } else {
        const float* q = static_cast<const float*>(p) + at;
        dev::Raw8<float> r;
        if (col >= 0 && col + 8 <= dim && (reinterpret_cast<uintptr_t>(q) & 15) == 0)
            dev::load_raw8(q, r);
        else
            edge_cols(q - col, col, dim, r);
        dev::unpack8(r, x);
    }
}

// What a kernel is compiled for.
//   kPlain  RMSNorm without biases, rows at 16-byte boundaries, whole pieces
//   kWhole  LayerNorm or biases too, the same rows
//   kEdges  everything: pieces that reach over the row's ends, any alignment
// The tests for ends in kEdges' loads and stores cost it about a third of the
// other two's rate.
enum Mode { kPlain = 0, kWhole = 1, kEdges = 2 };

// The thread's columns: kNV pieces of 8.  A piece of kPlain and kWhole lies in
// the row as a whole, or outside.
template <int kNV, int kMode>
struct Columns {
    int col[kNV], dim;
    bool full[kNV]; // inside the row, at a multiple of 16 bytes

    __device__ __forceinline__ Columns(const Geometry& G, const Group& g, int shift)
    {
        dim = static_cast<int>(G.dim);
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            col[i] = (g.thread + i * g.threads) * 8 - shift;
            full[i] = col[i] + 8 <= dim;
            if (kMode == kEdges) full[i] = G.wide && full[i] && col[i] >= 0;
        }
    }
    __device__ __forceinline__ bool inside(int i, int e) const
    {
        return kMode != kEdges ? full[i] : col[i] + e >= 0 && col[i] + e < dim;
    }
    // The pieces' values at p, the row's start; 0 outside the row.
    template <typename T>
    __device__ __forceinline__ void load(const T* p, dev::Raw8<T> (&r)[kNV]) const
    {
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            if (full[i])
                dev::stream_raw8(p + col[i], r[i]);
            else if (kMode == kEdges)
                edge_cols(p, col[i], dim, r[i]);
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T* p, int i, const float2 (&x)[4]) const
    {
        if (full[i])
            dev::store8_stream(p + col[i], x);
        else if (kMode == kEdges)
            store_edge(p, col[i], dim, x);
    }
};

// x - mean inside the row, 0 outside.
template <int kNV, int kMode>
__device__ __forceinline__ void centre(const Columns<kNV, kMode>& c, float mean,
                                       float2 (&x)[kNV][4])
{
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        if (kMode != kEdges) {
            const float2 m = dev::pair(c.full[i] ? -mean : 0.0f);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][e] = dev::add2(x[i][e], m);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[i][e].x = c.inside(i, 2 * e) ? x[i][e].x - mean : 0.0f;
                x[i][e].y = c.inside(i, 2 * e + 1) ? x[i][e].y - mean : 0.0f;
            }
        }
    }
}
template <int kNV>
__device__ __forceinline__ float total(const float2 (&x)[kNV][4])
{
    float2 s = x[0][0];
#pragma unroll
    for (int i = 0; i < 4 * kNV; ++i)
        if (i) s = dev::add2(s, x[i / 4][i % 4]);
    return s.x + s.y;
}
template <int kNV>
__device__ __forceinline__ float dot(const float2 (&x)[kNV][4], const float2 (&y)[kNV][4])
{
    float2 s = dev::mul2(x[0][0], y[0][0]);
#pragma unroll
    for (int i = 0; i < 4 * kNV; ++i)
        if (i) s = dev::fma2(x[i / 4][i % 4], y[i / 4][i % 4], s);
    return s.x + s.y;
}

// ------------------------------------------------------------------ forward
// The row's centred values and 1/sqrt(variance + eps).  LayerNorm's variance
// is taken about the mean in a second sum: the one-pass form
// mean(v^2) - mean^2 loses the digits that a large mean takes.
template <int kNV, int kMode>
__device__ __forceinline__ float standardise(Group& g, const Columns<kNV, kMode>& c, const Params& P,
                                             float inv, float2 (&v)[kNV][4])
{
    if (kMode != kPlain && P.layer) {
        float s[1] = {total(v)};
        group_sum(g, s);
        centre(c, s[0] * inv, v);
    }
    float s[1] = {dot(v, v)};
    group_sum(g, s);
    return rsqrtf(fmaf(s[0], inv, P.eps));
}

// Rows are dealt to the groups in turn; the next row's loads are issued before this row is computed, and the
// weights stay in registers: branch_scale * gate * w of the branch's norm as one
// factor, formed again only where the gate's row changes.
template <int kNV, int kMode, typename Act, typename Res>
__global__ void __launch_bounds__(kThreads)
forward_kernel(const Geometry G, const Params P, const Res* __restrict__ x,
               const Act* __restrict__ h, Res* __restrict__ y, Act* __restrict__ u)
{
    Group g = make_group(G.threads);
    const int64_t worker = static_cast<int64_t>(blockIdx.x) * G.groups + g.id;
    const int64_t workers = static_cast<int64_t>(G.blocks) * G.groups / G.classes * G.classes;
    if (worker >= workers || worker >= G.rows) return;
    const int dim = static_cast<int>(G.dim);
    const float inv = 1.0f / static_cast<float>(dim);
    constexpr bool kFull = kMode != kPlain;
    const Columns<kNV, kMode> c(
        G, g, kMode == kEdges ? static_cast<int>(worker % G.classes * G.dim % 8) : 0);
    float2 pw[kNV][4], pb[kNV][4], qw[kNV][4], qb[kNV][4];
    auto factors = [&](int64_t gate_row) {
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            float2 t[4];
            load_vector(P.gate, P.gate_type, gate_row, c.col[i], dim, 1.0f, t);
            load_vector(P.post_w, P.param_type, 0, c.col[i], dim, 1.0f, pw[i]);
            if (kFull) load_vector(P.post_b, P.param_type, 0, c.col[i], dim, 0.0f, pb[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                t[e] = dev::mul2(t[e], dev::pair(P.branch_scale));
                pw[i][e] = dev::mul2(pw[i][e], t[e]);
                if (kFull) pb[i][e] = dev::mul2(pb[i][e], t[e]);
            }
        }
    };
    int64_t gate_row = P.gate ? worker / G.span : 0;
    int64_t gate_end = P.gate ? (gate_row + 1) * G.span : G.rows; // first row of the next gate row
    factors(gate_row);
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        load_vector(P.pre_w, P.param_type, 0, c.col[i], dim, 1.0f, qw[i]);
        if (kFull) load_vector(P.pre_b, P.param_type, 0, c.col[i], dim, 0.0f, qb[i]);
    }
    dev::Raw8<Res> rx[kNV];
    dev::Raw8<Act> rh[kNV];
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        clear(rx[i]);
        clear(rh[i]);
    }
    const int64_t step = workers * G.dim;
    int64_t at = worker * G.dim; // the row's first element
    c.load(x + at, rx);
    if (h) c.load(h + at, rh);
    for (int64_t row = worker; row < G.rows; row += workers, at += step) {
        float2 v[kNV][4], n[kNV][4];
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            dev::unpack8(rx[i], v[i]);
            dev::unpack8(rh[i], n[i]);
        }
        if (row + workers < G.rows) {
            c.load(x + at + step, rx);
            if (h) c.load(h + at + step, rh);
        }
        if (h) {
            const float2 r = dev::pair(P.post ? standardise(g, c, P, inv, n) : 1.0f);
            if (row >= gate_end) {
                gate_row = row / G.span;
                gate_end = (gate_row + 1) * G.span;
                factors(gate_row);
            }
            const float2 a = dev::pair(P.res_scale);
#pragma unroll
            for (int i = 0; i < kNV; ++i) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[i][e] = kFull ? dev::fma2(a, v[i][e], pb[i][e]) : dev::mul2(a, v[i][e]);
                    v[i][e] = dev::fma2(dev::mul2(n[i][e], r), pw[i][e], v[i][e]);
                }
                c.store(y + at, i, v[i]);
            }
        }
        if (P.pre) {
            const float2 r = dev::pair(standardise(g, c, P, inv, v));
#pragma unroll
            for (int i = 0; i < kNV; ++i) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[i][e] = dev::mul2(v[i][e], r);
                    v[i][e] = kFull ? dev::fma2(v[i][e], qw[i][e], qb[i][e])
                                    : dev::mul2(v[i][e], qw[i][e]);
                }
                c.store(u + at, i, v[i]);
            }
        }
    }
}

// ----------------------------------------------------------------- backward
// Per-column factors that a thread keeps in shared memory, where the sums take
// its registers: its own 8 columns of vector k, piece i, as two 16-byte words;
// consecutive threads have consecutive words, and a thread's words lie a constant
// kThreads apart.  No other thread reads them.
template <int kNV>
struct Slots {
    float4* base;
    __device__ __forceinline__ float4* at(int k, int i) const
    {
        return base + (k * kNV + i) * 2 * kThreads + threadIdx.x;
    }
    __device__ __forceinline__ void put(int k, int i, const float2 (&x)[4]) const
    {
        at(k, i)[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
        at(k, i)[kThreads] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
    }
    __device__ __forceinline__ void get(int k, int i, float2 (&x)[4]) const
    {
        const float4 a = at(k, i)[0], b = at(k, i)[kThreads];
        x[0] = make_float2(a.x, a.y), x[1] = make_float2(a.z, a.w);
        x[2] = make_float2(b.x, b.y), x[3] = make_float2(b.z, b.w);
    }
};
constexpr int kSlotPost = 0, kSlotPre = 1, kSlotGate = 2, kSlotBias = 3;
// With 4 pieces a thread four vectors do not fit; the bias is then read anew.
template <int kNV>
constexpr bool kBiasSlot = kNV < 4;

// Partial sums in the scratch: [blocks][vectors in use][dim] of the sums over
// all rows, then, with several gate rows, [workers][2][dim] of the gate rows
// that a worker shares with others: its first one, and its last one.
struct Grads {
    void *dgate;
    int32_t dgate_type;
    int32_t gate_rows;   // 0: no dgate wanted
    int32_t vectors;     // sums over all rows: kVectors, and the gate's where it has one row
    int32_t by_ends;     // how reduce_kernel finds the gate rows that workers share
    float* partial;
    float* gate_partial;
};

// The sums of a row come together as far as the formulas allow: RMSNorm takes
// { y^2, du w y, h^2 } and then { d w h }, two exchanges a row; LayerNorm
// { y, du w, h }, the centred { y^2, du w y, h^2 }, then { d w, d w h }.
template <int kNV, int kMode, typename Act, typename Res>
__global__ void __launch_bounds__(kThreads)
backward_kernel(const Geometry G, const Params P, const Grads D, const Res* __restrict__ dy,
                const Act* __restrict__ du, const Res* __restrict__ y, const Act* __restrict__ h,
                Res* __restrict__ dx, Act* __restrict__ dh)
{
    extern __shared__ float4 shared[];
    const Slots<kNV> slots = {shared};
    // after the rows: groups x dim, where a block has several groups
    float* combine = reinterpret_cast<float*>(shared);
    Group g = make_group(G.threads);
    const int64_t worker = static_cast<int64_t>(blockIdx.x) * G.groups + g.id;
    const int64_t strip = worker / G.classes; // workers of a strip share its rows by class
    const int64_t cls = worker - strip * G.classes;
    const int64_t lo = strip * G.run + cls;
    int64_t hi = strip * G.run + G.run;
    if (hi > G.rows) hi = G.rows;
    const int dim = static_cast<int>(G.dim);
    const float inv = 1.0f / static_cast<float>(dim);
    constexpr bool kFull = kMode != kPlain;
    const Columns<kNV, kMode> c(G, g, kMode == kEdges ? static_cast<int>(cls * G.dim % 8) : 0);
    constexpr int kSums = kFull ? kVectors + 1 : 3;
    // dw post, dw pre, dgate / branch_scale; dc post, dc pre
    float2 sums[kSums][kNV][4];
#pragma unroll
    for (int a = 0; a < kSums; ++a)
#pragma unroll
        for (int i = 0; i < kNV; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) sums[a][i][e] = dev::pair(0.0f);

    const bool by_rows = D.gate_rows > 1;
    int64_t gate_row = P.gate && lo < hi ? lo / G.span : 0;
    int64_t gate_end = P.gate ? (gate_row + 1) * G.span : G.rows;
    const int64_t first_gate = gate_row;
    auto load_gate = [&] { // branch_scale * gate
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            float2 w[4];
            load_vector(P.gate, P.gate_type, gate_row, c.col[i], dim, 1.0f, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = dev::mul2(w[e], dev::pair(P.branch_scale));
            slots.put(kSlotGate, i, w);
        }
    };
    // The sum of one gate row: final where this worker has all its rows.
    auto leave_gate = [&] {
        const int64_t from = gate_row * G.span;
        const int64_t to = from + G.span < G.rows ? from + G.span : G.rows;
        const bool whole = G.classes == 1 ? from >= lo && to <= hi : to - from == 1;
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            float2 t[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                t[e] = dev::mul2(dev::pair(P.branch_scale), sums[2][i][e]);
                sums[2][i][e] = dev::pair(0.0f);
            }
            if (!whole) {
                const int slot = gate_row == first_gate ? 0 : 1;
                store_edge(D.gate_partial + (2 * worker + slot) * G.dim, c.col[i], dim, t);
            } else if (D.dgate_type == ZERO_TYPE_BF16) {
                store_edge(static_cast<Bf16*>(D.dgate) + gate_row * G.dim, c.col[i], dim, t);
            } else {
                store_edge(static_cast<float*>(D.dgate) + gate_row * G.dim, c.col[i], dim, t);
            }
        }
    };
    dev::Raw8<Res> rdy[kNV], ry[kNV];
    dev::Raw8<Act> rdu[kNV], rh[kNV];
#pragma unroll
    for (int i = 0; i < kNV; ++i) { // what is absent, or outside the row, is 0
        clear(rdy[i]);
        clear(ry[i]);
        clear(rdu[i]);
        clear(rh[i]);
    }
    auto fetch = [&](int64_t from) {
        if (dy) c.load(dy + from, rdy);
        if (P.pre) {
            c.load(y + from, ry);
            c.load(du + from, rdu);
        }
        if (h) c.load(h + from, rh);
    };
    const int64_t step = G.classes * G.dim;
    int64_t at = lo * G.dim; // the row's first element
    if (lo < hi) {
        fetch(at);
        load_gate();
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            float2 w[4];
            load_vector(P.post_w, P.param_type, 0, c.col[i], dim, 1.0f, w);
            slots.put(kSlotPost, i, w);
            load_vector(P.pre_w, P.param_type, 0, c.col[i], dim, 1.0f, w);
            slots.put(kSlotPre, i, w);
            if (kFull && kBiasSlot<kNV>) {
                load_vector(P.post_b, P.param_type, 0, c.col[i], dim, 0.0f, w);
                slots.put(kSlotBias, i, w);
            }
        }
    }

    for (int64_t row = lo; row < hi; row += G.classes, at += step) {
        float2 t[kNV][4], v[kNV][4], d[kNV][4], n[kNV][4]; // dy, then g; y; du; branch
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            dev::unpack8(rdy[i], t[i]);
            dev::unpack8(ry[i], v[i]);
            dev::unpack8(rdu[i], d[i]);
            dev::unpack8(rh[i], n[i]);
        }
        if (row + G.classes < hi) fetch(at + step);
        if (row >= gate_end) {
            if (by_rows) leave_gate();
            gate_row = row / G.span;
            gate_end = (gate_row + 1) * G.span;
            load_gate();
        }
        float m0 = 0.0f;
        if (kFull && P.layer) {
            float2 dw = dev::pair(0.0f);
#pragma unroll
            for (int i = 0; i < kNV; ++i) {
                float2 w[4];
                slots.get(kSlotPre, i, w);
#pragma unroll
                for (int e = 0; e < 4; ++e) dw = dev::fma2(d[i][e], w[e], dw);
            }
            float s[4] = {total(v), dw.x + dw.y, total(n), 0.0f};
            group_sum(g, s);
            centre(c, s[0] * inv, v);
            m0 = s[1] * inv;
            if (P.post) centre(c, s[2] * inv, n);
        }
        float2 dwv = dev::pair(0.0f);
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            float2 w[4];
            slots.get(kSlotPre, i, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) dwv = dev::fma2(dev::mul2(d[i][e], w[e]), v[i][e], dwv);
        }
        float s[4] = {dot(v, v), dwv.x + dwv.y, dot(n, n), 0.0f};
        group_sum(g, s);
        if (P.pre) {
            const float rstd = rsqrtf(fmaf(s[0], inv, P.eps));
            const float2 r = dev::pair(rstd);
            // -r^2 mean(du w y^); a row of zeros has 0, though r^3 may be out of range
            const float2 k = dev::pair(-rstd * (rstd * (rstd * (s[1] * inv))));
#pragma unroll
            for (int i = 0; i < kNV; ++i) {
                const float2 k0 = dev::pair(kMode == kEdges || c.full[i] ? -rstd * m0 : 0.0f);
                float2 w[4];
                slots.get(kSlotPre, i, w);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (kFull) sums[4][i][e] = dev::add2(sums[4][i][e], d[i][e]);
                    d[i][e] = dev::mul2(d[i][e], r);
                    sums[1][i][e] = dev::fma2(d[i][e], v[i][e], sums[1][i][e]);
                    t[i][e] = dev::fma2(k, v[i][e], dev::fma2(d[i][e], w[e], t[i][e]));
                    if (kFull) t[i][e] = dev::add2(t[i][e], k0);
                }
            }
        }
        if (dx) {
#pragma unroll
            for (int i = 0; i < kNV; ++i) {
                float2 o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = dev::mul2(dev::pair(P.res_scale), t[i][e]);
                c.store(dx + at, i, o);
            }
        }
        if (!h) continue;
        const float rstd = P.post ? rsqrtf(fmaf(s[2], inv, P.eps)) : 1.0f;
        const float2 r = dev::pair(rstd);
        float2 m0s = dev::pair(0.0f), m1s = m0s;
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            float2 pb[4], pw[4], gate[4];
            slots.get(kSlotPost, i, pw);
            slots.get(kSlotGate, i, gate);
            if (kFull && kBiasSlot<kNV>)
                slots.get(kSlotBias, i, pb);
            else if (kFull)
                load_vector(P.post_b, P.param_type, 0, c.col[i], dim, 0.0f, pb);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                n[i][e] = dev::mul2(n[i][e], r);
                const float2 a =
                    kFull ? dev::fma2(n[i][e], pw[e], pb[e]) : dev::mul2(n[i][e], pw[e]);
                sums[2][i][e] = dev::fma2(t[i][e], a, sums[2][i][e]);
                t[i][e] = dev::mul2(t[i][e], gate[e]);
                if (kMode == kEdges) { // LayerNorm's mean was taken off outside the row too
                    if (!c.inside(i, 2 * e)) t[i][e].x = 0.0f;
                    if (!c.inside(i, 2 * e + 1)) t[i][e].y = 0.0f;
                }
                if (kFull) {
                    sums[3][i][e] = dev::add2(sums[3][i][e], t[i][e]);
                }
                sums[0][i][e] = dev::fma2(t[i][e], n[i][e], sums[0][i][e]);
                t[i][e] = dev::mul2(t[i][e], pw[e]);
                if (kFull) m0s = dev::add2(m0s, t[i][e]);
                m1s = dev::fma2(t[i][e], n[i][e], m1s);
            }
        }
        float k0 = 0.0f, k1 = 0.0f;
        if (P.post) {
            if (kFull) {
                float m[2] = {m0s.x + m0s.y, m1s.x + m1s.y};
                group_sum(g, m);
                if (P.layer) k0 = m[0] * inv;
                k1 = m[1] * inv;
            } else {
                float m[1] = {m1s.x + m1s.y};
                group_sum(g, m);
                k1 = m[0] * inv;
            }
        }
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float2 o = t[i][e];
                if (kFull) o = dev::add2(o, dev::pair(-k0));
                t[i][e] = dev::mul2(r, dev::fma2(dev::pair(-k1), n[i][e], o));
            }
            c.store(dh + at, i, t[i]);
        }
    }
    if (by_rows && lo < hi) leave_gate();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // The block's sums, its groups added in order.
#pragma unroll
    for (int a = 0; a < kSums; ++a) {
        constexpr int kPlace[kVectors + 1] = {0, 2, kVectors, 1, 3}; // in Finals' order
        if (kPlace[a] >= D.vectors) continue;
        if (a == 2) {
#pragma unroll
            for (int i = 0; i < kNV; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sums[a][i][e] = dev::mul2(sums[a][i][e], dev::pair(P.branch_scale));
        }
        float* out = D.partial + (static_cast<int64_t>(blockIdx.x) * D.vectors + kPlace[a]) * G.dim;
        if (G.groups == 1) {
#pragma unroll
            for (int i = 0; i < kNV; ++i) store_edge(out, c.col[i], dim, sums[a][i]);
            continue;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kNV; ++i)
            store_edge(combine + g.id * dim, c.col[i], dim, sums[a][i]);
        __syncthreads();
        for (int j = threadIdx.x; j < dim; j += blockDim.x) {
            float sum = 0.0f;
            for (int k = 0; k < G.groups; ++k) sum += combine[k * dim + j];
            out[j] = sum;
        }
    }
}

// ------------------------------------------- backward, two rows at a time
// For rows of whole 16-byte pieces, at most one piece a thread (dim <= 4096): the
// usual case.  A group takes two rows at once: their sums share the exchanges
// between the warps, whose latency is what a row costs most (measured, 16384 x
// 2048 with an fp32 residual: one row at a time 119 us).  The next two rows come to
// shared memory meanwhile (cp.async), each thread's pieces to its own slots,
// which no other thread touches, so no barrier is needed for them and no
// register is held.

// One tensor's two pieces of a thread: 16-byte words, kThreads apart.
template <typename T>
struct Pieces {
    static constexpr int kWords = sizeof(T) / 2; // of one piece
    uint4* base;                                 // word 0 of row 0

    __device__ __forceinline__ uint4* word(int row, int w) const
    {
        return base + (row * kWords + w) * kThreads;
    }
    __device__ __forceinline__ void fetch(int row, const T* p) const
    {
        const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(base));
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
            // the two words of an fp32 piece are half a sector each: through the L1,
            // where the second finds the first's
            if constexpr (kWords == 1)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                 to + (row * kWords + w) * (16 * kThreads)),
                             "l"(p)
                             : "memory");
            else
                asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(
                                 to + (row * kWords + w) * (16 * kThreads)),
                             "l"(reinterpret_cast<const uint4*>(p) + w)
                             : "memory");
        }
    }
    __device__ __forceinline__ void clear(int row) const
    {
#pragma unroll
        for (int w = 0; w < kWords; ++w) *word(row, w) = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(int row, float2 (&x)[4]) const
    {
        dev::Raw8<T> r;
        if constexpr (kWords == 1) {
            r.a = *word(row, 0);
        } else {
            r.a = *reinterpret_cast<const float4*>(word(row, 0));
            r.b = *reinterpret_cast<const float4*>(word(row, 1));
        }
        dev::unpack8(r, x);
    }
};

// Sums of 8 values over the group, valid in all its threads: 9 shuffles in the
// warp (a lane keeps half of its values at each of the first three steps), a
// word per warp and value in shared memory (`red`: two buffers of 8 x 16 words
// for the group, zero where there is no warp), and 8 to hand them round.
__device__ __forceinline__ void group_sum8(Group& g, float* red, float (&v)[8])
{
    constexpr uint32_t kAll = 0xFFFFFFFFu;
    const int lane = threadIdx.x & 31;
    float a[4], b[2];
    const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        a[i] = (b4 ? v[i + 4] : v[i]) + __shfl_xor_sync(kAll, b4 ? v[i] : v[i + 4], 16);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        b[i] = (b3 ? a[i + 2] : a[i]) + __shfl_xor_sync(kAll, b3 ? a[i] : a[i + 2], 8);
    float x = (b2 ? b[1] : b[0]) + __shfl_xor_sync(kAll, b2 ? b[0] : b[1], 4);
    x += __shfl_xor_sync(kAll, x, 2);
    x += __shfl_xor_sync(kAll, x, 1); // the sum of value lane >> 2
    if (g.warps > 1) {
        float* buf = red + g.buffer * (8 * kMaxWarps);
        if ((lane & 3) == 0)
            buf[(lane >> 2) * kMaxWarps + (threadIdx.x >> 5) - g.first_warp] = x;
        asm volatile("bar.sync %0, %1;" ::"r"(g.id + 1), "r"(g.threads) : "memory");
        const float4 w = *reinterpret_cast<const float4*>(buf + 4 * lane);
        x = (w.x + w.y) + (w.z + w.w);
        x += __shfl_xor_sync(kAll, x, 2);
        x += __shfl_xor_sync(kAll, x, 1);
        g.buffer ^= 1;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __shfl_sync(kAll, x, 4 * i);
}

template <int kMode, typename Act, typename Res>
__global__ void __launch_bounds__(kThreads)
backward_pair_kernel(const Geometry G, const Params P, const Grads D, const Res* __restrict__ dy,
                     const Act* __restrict__ du, const Res* __restrict__ y,
                     const Act* __restrict__ h, Res* __restrict__ dx, Act* __restrict__ dh)
{
    constexpr bool kFull = kMode != kPlain;
    constexpr int kSums = kFull ? kVectors + 1 : 3;
    constexpr int kFactors = kFull ? 4 : 3;
    extern __shared__ float4 shared[];
    // [kFactors x 2] words of factors, then the pieces of two rows, then the
    // groups' exchange words
    const Slots<1> slots = {shared};
    const int block = static_cast<int>(blockDim.x);
    constexpr int kRes = 2 * Pieces<Res>::kWords * kThreads, kAct = 2 * Pieces<Act>::kWords * kThreads;
    uint4* pieces = reinterpret_cast<uint4*>(shared) + kFactors * 2 * kThreads;
    const Pieces<Res> s_dy = {pieces + threadIdx.x};
    const Pieces<Res> s_y = {pieces + kRes + threadIdx.x};
    const Pieces<Act> s_du = {pieces + 2 * kRes + threadIdx.x};
    const Pieces<Act> s_h = {pieces + 2 * kRes + kAct + threadIdx.x};
    Group g = make_group(G.threads);
    float* red = reinterpret_cast<float*>(pieces + 2 * kRes + 2 * kAct) + g.id * (2 * 8 * kMaxWarps);
    for (int i = g.thread; i < 2 * 8 * kMaxWarps; i += g.threads) red[i] = 0.0f;

    const int64_t worker = static_cast<int64_t>(blockIdx.x) * G.groups + g.id;
    const int64_t lo = worker * G.run;
    const int64_t hi = lo + G.run < G.rows ? lo + G.run : G.rows;
    const int dim = static_cast<int>(G.dim);
    const float inv = 1.0f / static_cast<float>(dim);
    const int col = g.thread * 8;
    const bool full = col < dim;
    // dw post, dw pre, dgate / branch_scale; dc post, dc pre
    float2 sums[kSums][4];
#pragma unroll
    for (int a = 0; a < kSums; ++a)
#pragma unroll
        for (int e = 0; e < 4; ++e) sums[a][e] = dev::pair(0.0f);
#pragma unroll
    for (int r = 0; r < 2; ++r) { // what is absent, or outside the row, stays 0
        s_dy.clear(r);
        s_y.clear(r);
        s_du.clear(r);
        s_h.clear(r);
    }

    const bool by_rows = D.gate_rows > 1;
    int64_t gate_row = P.gate && lo < hi ? lo / G.span : 0;
    int64_t gate_end = P.gate ? (gate_row + 1) * G.span : G.rows;
    const int64_t first_gate = gate_row;
    auto load_gate = [&] { // branch_scale * gate
        float2 w[4];
        load_vector(P.gate, P.gate_type, gate_row, col, dim, 1.0f, w);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = dev::mul2(w[e], dev::pair(P.branch_scale));
        slots.put(kSlotGate, 0, w);
    };
    // The sum of one gate row: final where this worker has all its rows.
    auto leave_gate = [&] {
        const int64_t from = gate_row * G.span;
        const int64_t to = from + G.span < G.rows ? from + G.span : G.rows;
        float2 t[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            t[e] = dev::mul2(dev::pair(P.branch_scale), sums[2][e]);
            sums[2][e] = dev::pair(0.0f);
        }
        if (!full) return;
        if (!(from >= lo && to <= hi)) {
            const int slot = gate_row == first_gate ? 0 : 1;
            store_cols(D.gate_partial + (2 * worker + slot) * G.dim, col, dim, t);
        } else if (D.dgate_type == ZERO_TYPE_BF16) {
            store_cols(static_cast<Bf16*>(D.dgate) + gate_row * G.dim, col, dim, t);
        } else {
            store_cols(static_cast<float*>(D.dgate) + gate_row * G.dim, col, dim, t);
        }
    };
    // Rows of the pair that begins at `row`: one where the run or the gate row ends.
    auto pair_rows = [&](int64_t row, int64_t end_of_gate) {
        return row + 1 < hi && row + 1 < end_of_gate ? 2 : 1;
    };
    auto fetch = [&](int64_t row, int rows) {
        if (full) {
            for (int r = 0; r < rows; ++r) {
                const int64_t at = (row + r) * G.dim + col;
                if (dy) s_dy.fetch(r, dy + at);
                if (P.pre) {
                    s_y.fetch(r, y + at);
                    s_du.fetch(r, du + at);
                }
            }
        }
    };
    // The branch's pieces are read twice, and fetched once they are done with.
    auto fetch_branch = [&](int64_t row, int rows) {
        if (full && h)
            for (int r = 0; r < rows; ++r) s_h.fetch(r, h + (row + r) * G.dim + col);
    };
    auto clear_second = [&] { // a pair of one row
        s_dy.clear(1);
        s_y.clear(1);
        s_du.clear(1);
    };
    int rows = 0;
    if (lo < hi) {
        rows = pair_rows(lo, gate_end);
        fetch(lo, rows);
        fetch_branch(lo, rows);
        // the usual types and alignment: all four vectors' loads at once, not each
        // after the one before (a microsecond each at the kernel's start)
        const void* from[4] = {P.post_w, P.pre_w, P.gate, P.post_b};
        bool plain = full && P.param_type == ZERO_TYPE_BF16 && P.gate_type == ZERO_TYPE_BF16;
#pragma unroll
        for (int k = 0; k < 4; ++k) plain = plain && (reinterpret_cast<uintptr_t>(from[k]) & 15) == 0;
        if (plain) {
            dev::Raw8<Bf16> raw[4];
#pragma unroll
            for (int k = 0; k < kFactors; ++k) {
                const uint32_t one = k == 3 ? 0u : 0x3F803F80u; // absent: 1, or 0 of a bias
                raw[k].a = make_uint4(one, one, one, one);
                if (from[k])
                    dev::load_raw8(static_cast<const Bf16*>(from[k]) +
                                       (k == kSlotGate ? gate_row * G.dim : 0) + col,
                                   raw[k]);
            }
#pragma unroll
            for (int k = 0; k < kFactors; ++k) {
                float2 w[4];
                dev::unpack8(raw[k], w);
                if (k == kSlotGate) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = dev::mul2(w[e], dev::pair(P.branch_scale));
                }
                slots.put(k, 0, w);
            }
        } else {
            load_gate();
            float2 w[4];
            load_vector(P.post_w, P.param_type, 0, col, dim, 1.0f, w);
            slots.put(kSlotPost, 0, w);
            load_vector(P.pre_w, P.param_type, 0, col, dim, 1.0f, w);
            slots.put(kSlotPre, 0, w);
            if (kFull) {
                load_vector(P.post_b, P.param_type, 0, col, dim, 0.0f, w);
                slots.put(kSlotBias, 0, w);
            }
        }
    }
    __syncthreads(); // the exchange words are 0

    for (int64_t row = lo; row < hi;) {
        const int64_t next = row + rows;
        if (row >= gate_end) {
            if (by_rows) leave_gate();
            gate_row = row / G.span;
            gate_end = (gate_row + 1) * G.span;
            load_gate();
        }
        int next_rows = 0;
        if (next < hi) {
            const int64_t end = P.gate && next >= gate_end ? (next / G.span + 1) * G.span : gate_end;
            next_rows = pair_rows(next, end);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        float2 t[2][4], v[2][4], d[2][4]; // dy, then g; y; du
        float s[8] = {};                  // of row r: s[r], s[2 + r], s[4 + r]
        float mean_n[2] = {0.0f, 0.0f}, m0[2] = {0.0f, 0.0f};
        float2 w[4];
        slots.get(kSlotPre, 0, w);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            s_dy.get(r, t[r]);
            s_y.get(r, v[r]);
            s_du.get(r, d[r]);
        }
        if (kFull && P.layer) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float2 n[4], a = dev::pair(0.0f), b = a, c = a;
                s_h.get(r, n);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    a = dev::add2(a, v[r][e]);
                    b = dev::fma2(d[r][e], w[e], b);
                    c = dev::add2(c, n[e]);
                }
                s[r] = a.x + a.y;
                s[2 + r] = b.x + b.y;
                s[4 + r] = c.x + c.y;
            }
            group_sum8(g, red, s);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float2 mean = dev::pair(full ? -s[r] * inv : 0.0f);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[r][e] = dev::add2(v[r][e], mean);
                m0[r] = s[2 + r] * inv;
                mean_n[r] = full && P.post ? -s[4 + r] * inv : 0.0f;
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float2 n[4], a = dev::pair(0.0f), b = a, c = a;
            s_h.get(r, n);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (kFull) n[e] = dev::add2(n[e], dev::pair(mean_n[r]));
                a = dev::fma2(v[r][e], v[r][e], a);
                b = dev::fma2(dev::mul2(d[r][e], w[e]), v[r][e], b);
                c = dev::fma2(n[e], n[e], c);
            }
            s[r] = a.x + a.y;
            s[2 + r] = b.x + b.y;
            s[4 + r] = c.x + c.y;
        }
        s[6] = s[7] = 0.0f;
        // the three tensors are in registers: their slots take the next rows
        if (next_rows) {
            fetch(next, next_rows);
            if (next_rows == 1) clear_second();
        }
        group_sum8(g, red, s);
        if (P.pre) {
            slots.get(kSlotPre, 0, w);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float rstd = rsqrtf(fmaf(s[r], inv, P.eps));
                const float2 rr = dev::pair(rstd);
                // -r^2 mean(du w y^); a row of zeros, or no second row, has 0, though
                // r^3 may be out of range
                const float2 k = dev::pair(-rstd * (rstd * (rstd * (s[2 + r] * inv))));
                const float2 k0 = dev::pair(full ? -rstd * m0[r] : 0.0f);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (kFull) sums[4][e] = dev::add2(sums[4][e], d[r][e]);
                    d[r][e] = dev::mul2(d[r][e], rr);
                    sums[1][e] = dev::fma2(d[r][e], v[r][e], sums[1][e]);
                    t[r][e] = dev::fma2(k, v[r][e], dev::fma2(d[r][e], w[e], t[r][e]));
                    if (kFull) t[r][e] = dev::add2(t[r][e], k0);
                }
            }
        }
        if (dx && full) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float2 o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = dev::mul2(dev::pair(P.res_scale), t[r][e]);
                if (r < rows) dev::store8_stream(dx + (row + r) * G.dim + col, o);
            }
        }
        if (h) {
            float2 n[2][4], pw[4], gate[4], pb[4];
            slots.get(kSlotPost, 0, pw);
            slots.get(kSlotGate, 0, gate);
            if (kFull) slots.get(kSlotBias, 0, pb);
            float2 rr[2];
            float m[4] = {};
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                s_h.get(r, n[r]);
                rr[r] = dev::pair(P.post ? rsqrtf(fmaf(s[4 + r], inv, P.eps)) : 1.0f);
                float2 a = dev::pair(0.0f), b = a;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (kFull) n[r][e] = dev::add2(n[r][e], dev::pair(mean_n[r]));
                    n[r][e] = dev::mul2(n[r][e], rr[r]);
                    const float2 x =
                        kFull ? dev::fma2(n[r][e], pw[e], pb[e]) : dev::mul2(n[r][e], pw[e]);
                    sums[2][e] = dev::fma2(t[r][e], x, sums[2][e]);
                    t[r][e] = dev::mul2(t[r][e], gate[e]);
                    if (kFull) sums[3][e] = dev::add2(sums[3][e], t[r][e]);
                    sums[0][e] = dev::fma2(t[r][e], n[r][e], sums[0][e]);
                    t[r][e] = dev::mul2(t[r][e], pw[e]);
                    if (kFull) b = dev::add2(b, t[r][e]);
                    a = dev::fma2(t[r][e], n[r][e], a);
                }
                m[r] = a.x + a.y;
                m[2 + r] = b.x + b.y;
            }
            if (next_rows) {
                fetch_branch(next, next_rows);
                if (next_rows == 1) s_h.clear(1);
            }
            if (P.post) {
                if (kFull) {
                    group_sum(g, m);
                } else {
                    float two[2] = {m[0], m[1]};
                    group_sum(g, two);
                    m[0] = two[0];
                    m[1] = two[1];
                }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float2 k1 = dev::pair(P.post ? -m[r] * inv : 0.0f);
                const float2 k0 = dev::pair(kFull && P.post && P.layer ? -m[2 + r] * inv : 0.0f);
                float2 o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    o[e] = kFull ? dev::add2(t[r][e], k0) : t[r][e];
                    o[e] = dev::mul2(rr[r], dev::fma2(k1, n[r][e], o[e]));
                }
                if (full && r < rows) dev::store8_stream(dh + (row + r) * G.dim + col, o);
            }
        }
        row = next;
        rows = next_rows;
    }
    if (by_rows && lo < hi) leave_gate();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // The block's sums, its groups added in order: every thread's sums to shared
    // memory, 16-byte words of the same columns G.threads apart.
    __syncthreads();
#pragma unroll
    for (int a = 0; a < kSums; ++a) {
        const float k = a == 2 ? P.branch_scale : 1.0f;
        shared[(2 * a) * block + threadIdx.x] =
            make_float4(k * sums[a][0].x, k * sums[a][0].y, k * sums[a][1].x, k * sums[a][1].y);
        shared[(2 * a + 1) * block + threadIdx.x] =
            make_float4(k * sums[a][2].x, k * sums[a][2].y, k * sums[a][3].x, k * sums[a][3].y);
    }
    __syncthreads();
    constexpr int kPlace[kVectors + 1] = {0, 2, kVectors, 1, 3}; // in Finals' order
#pragma unroll
    for (int a = 0; a < kSums; ++a) {
        if (kPlace[a] >= D.vectors) continue;
        float* out = D.partial + (static_cast<int64_t>(blockIdx.x) * D.vectors + kPlace[a]) * G.dim;
        for (int i = threadIdx.x; i < 2 * G.threads; i += block) {
            const int half = i >= G.threads ? 1 : 0, thread = i - half * G.threads;
            if (thread * 8 >= dim) continue;
            const float4* p = shared + (2 * a + half) * block + thread;
            float4 x = p[0];
            for (int k = 1; k < G.groups; ++k) {
                const float4 z = p[k * G.threads];
                x.x += z.x, x.y += z.y, x.z += z.z, x.w += z.w;
            }
            *reinterpret_cast<float4*>(out + thread * 8 + half * 4) = x;
        }
    }
}

// Sums the blocks' partials, and those of the gate rows that several workers
// share: blockIdx.y is one of the sums over all rows, or, from D.vectors on, a
// gate row, or (by_ends, where those are fewer) the end of a worker's run that
// lies inside a gate row, the first such end of it.  kVec columns a lane, kSlices threads
// each: a slice adds a run of the partials in order, the slices are added in order.
constexpr int kSlices = 16;

struct Finals {
    void* out[kVectors + 1];
    int32_t type[kVectors + 1];
};

template <int kVec>
__global__ void __launch_bounds__(32 * kSlices)
reduce_kernel(const Geometry G, const Grads D, const Finals F)
{
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int dim = static_cast<int>(G.dim);
    const int col = (static_cast<int>(blockIdx.x) * 32 + lane) * kVec;
    const int task = static_cast<int>(blockIdx.y);
    __shared__ float sums[kSlices][32][kVec];
    // launched while the blocks of the kernel before drain; every block waits for
    // all of them, so that this kernel's end is also theirs
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float* src; // the slices' share: src + k * step, k < count
    const float* head = nullptr;
    int64_t step, count;
    void* out;
    int32_t type;
    int64_t out_row = 0;
    if (task < D.vectors) {
        out = F.out[task];
        type = F.type[task];
        if (!out) return;
        src = D.partial + task * G.dim;
        count = G.blocks;
        step = D.vectors * G.dim;
    } else {
        int64_t worker, q; // the gate row, and the first worker that has rows of it
        if (D.by_ends) {
            worker = task - D.vectors;
            const int64_t end = (worker + 1) * G.run;
            if (end >= G.rows || end % G.span == 0) return;
            q = end / G.span;
            if (q * G.span / G.run != worker) return; // it began before
        } else {
            q = task - D.vectors;
            worker = q * G.span / G.run;
        }
        const int64_t to = (q + 1) * G.span < G.rows ? (q + 1) * G.span : G.rows;
        if ((to - 1) / G.run == worker) return; // one worker's: final already
        // its first worker holds it as its last gate row, unless it is its first
        // too; the others as their first
        head = D.gate_partial + (2 * worker + (worker * G.run / G.span == q ? 0 : 1)) * G.dim;
        src = D.gate_partial + 2 * (worker + 1) * G.dim;
        step = 2 * G.dim;
        count = (to - 1) / G.run - worker;
        out = D.dgate;
        type = D.dgate_type;
        out_row = q * G.dim;
    }
    float acc[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v) acc[v] = 0.0f;
    auto add = [&](const float* p) {
        if constexpr (kVec == 4) {
            const float4 x = *reinterpret_cast<const float4*>(p + col);
            acc[0] += x.x, acc[1] += x.y, acc[2] += x.z, acc[3] += x.w;
        } else {
            acc[0] += p[col];
        }
    };
    const int64_t per = (count + kSlices - 1) / kSlices;
    const int64_t lo = slice * per, hi = lo + per < count ? lo + per : count;
    if (col < dim) {
        if (slice == 0 && head) add(head);
#pragma unroll 10
        for (int64_t k = lo; k < hi; ++k) add(src + k * step);
    }
#pragma unroll
    for (int v = 0; v < kVec; ++v) sums[slice][lane][v] = acc[v];
    __syncthreads();
    if (slice == 0 && col < dim) {
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            float all[1] = {0.0f};
#pragma unroll
            for (int w = 0; w < kSlices; ++w) all[0] += sums[w][lane][v];
            dev::store_any<1>(out, type, out_row + col + v, all);
        }
    }
}

// --------------------------------------------------------------------- host
bool sizes_ok(int64_t rows, int64_t dim, int64_t span)
{
    return rows >= 0 && rows <= (int64_t(1) << 40) && dim >= 1 && dim <= kMaxDim && span >= 1;
}

// Two vectors a thread halve the exchanges' share of the work, where that
// leaves no more threads idle (forward; the backward kernel's sums take the
// registers).
int vectors_per_thread(int64_t dim, int32_t classes, bool backward)
{
    const int64_t vecs = (dim + (classes > 1 ? 7 : 0) + 7) / 8;
    if (vecs > 2 * kThreads) return 4;
    if (vecs > kThreads) return 2;
    return !backward && vecs % 64 == 0 ? 2 : 1;
}

// aligned: every row tensor starts at a multiple of 16 bytes.  Depends on the
// sizes alone, so that the order of the sums does too.
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
    G.wide = aligned && (dim % 8 == 0 || G.classes > 1);
    const int64_t vecs = (dim + (G.classes > 1 ? 7 : 0) + 7) / 8;
    const int64_t per_thread = vectors_per_thread(dim, G.classes, backward);
    const int64_t lanes = (vecs + per_thread - 1) / per_thread;
    G.threads = static_cast<int32_t>((lanes + 31) / 32 * 32);
    // forward: blocks of 256, of which two or three fit an SM's registers
    const int32_t wanted = !backward && G.threads <= 256 ? 256 : kThreads;
    G.groups = wanted / G.threads;
    if (G.groups > 15 && G.threads > 32) G.groups = 15;
    const int64_t most = backward ? kMaxBackBlocks : kMaxBlocks;
    while (G.groups > 1 && (rows + G.groups - 1) / G.groups < most) G.groups /= 2;
    int64_t blocks = (rows + G.groups - 1) / G.groups;
    if (blocks > most) blocks = most;
    if (blocks < 1) blocks = 1;
    while (blocks * G.groups < G.classes) ++blocks; // a worker of each class
    G.blocks = static_cast<int32_t>(blocks);
    const int64_t strips = blocks * G.groups / G.classes;
    const int64_t run = (rows + strips - 1) / strips;
    G.run = (run + G.classes - 1) / G.classes * G.classes;
    if (G.run < 1) G.run = G.classes;
    return G;
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

Mode mode_of(const Geometry& G, bool full)
{
    return !G.wide || G.classes > 1 ? kEdges : full ? kWhole : kPlain;
}

template <int kNV, typename Act, typename Res>
void start_forward(const Geometry& G, const Params& P, const Res* x, const Act* h, Res* y, Act* u,
                   cudaStream_t stream)
{
    const unsigned grid = static_cast<unsigned>(G.blocks);
    const unsigned block = static_cast<unsigned>(G.threads * G.groups);
    const Mode mode = mode_of(G, P.layer || P.post_b || P.pre_b);
    constexpr int kP = kNV < 4 ? kPlain : kEdges, kW = kNV < 4 ? kWhole : kEdges;
    if (mode == kPlain)
        forward_kernel<kNV, kP, Act, Res><<<grid, block, 0, stream>>>(G, P, x, h, y, u);
    else if (mode == kWhole)
        forward_kernel<kNV, kW, Act, Res><<<grid, block, 0, stream>>>(G, P, x, h, y, u);
    else
        forward_kernel<kNV, kEdges, Act, Res><<<grid, block, 0, stream>>>(G, P, x, h, y, u);
}

template <typename Act, typename Res>
int launch_forward(const Geometry& G, const Params& P, const void* x, const void* h, void* y,
                   void* u, cudaStream_t stream)
{
    const auto* xp = static_cast<const Res*>(x);
    const auto* hp = static_cast<const Act*>(h);
    auto* yp = static_cast<Res*>(y);
    auto* up = static_cast<Act*>(u);
    switch (vectors_per_thread(G.dim, G.classes, false)) {
    case 1: start_forward<1>(G, P, xp, hp, yp, up, stream); break;
    case 2: start_forward<2>(G, P, xp, hp, yp, up, stream); break;
    default: start_forward<4>(G, P, xp, hp, yp, up, stream);
    }
    return cuda_status(cudaGetLastError());
}

template <int kNV, typename Act, typename Res>
int start_backward(const Geometry& G, const Params& P, const Grads& D, bool full, const Res* dy,
                    const Act* du, const Res* y, const Act* h, Res* dx, Act* dh,
                    cudaStream_t stream)
{
    const unsigned grid = static_cast<unsigned>(G.blocks);
    const unsigned block = static_cast<unsigned>(G.threads * G.groups);
    const Mode mode = mode_of(G, full);
    if (kNV == 1 && mode != kEdges) {
        auto* pairs = mode == kPlain ? backward_pair_kernel<kPlain, Act, Res>
                                     : backward_pair_kernel<kWhole, Act, Res>;
        const size_t words = (mode == kPlain ? 6 : 8) + 2 * sizeof(Res) + 2 * sizeof(Act);
        auto bytes_of = [&](int groups) {
            return words * 16 * kThreads + static_cast<size_t>(groups) * 2 * 8 * kMaxWarps * 4;
        };
        const size_t bytes = bytes_of(G.groups);
        if (!allow_shared(reinterpret_cast<const void*>(pairs), bytes_of(kMaxWarps))) return ZERO_ECUDA;
        pairs<<<grid, block, bytes, stream>>>(G, P, D, dy, du, y, h, dx, dh);
        return cuda_status(cudaGetLastError());
    }
    // one size for each kernel; the groups' sums at the end (G.groups x G.dim, where a
    // thread has one piece: 16 KB at most) fit into it
    const size_t smem = static_cast<size_t>((mode != kPlain || kNV != 2) && kBiasSlot<kNV> ? 4 : 3) * kNV * 32 * kThreads;
    // several pieces a thread, or ragged ends: one row at a time (kEdges does
    // what kWhole does; the sums' registers bound both)
    constexpr int kP = kNV == 2 ? kPlain : kEdges;
    auto* kernel = mode == kPlain ? backward_kernel<kNV, kP, Act, Res>
                                  : backward_kernel<kNV, kEdges, Act, Res>;
    if (!allow_shared(reinterpret_cast<const void*>(kernel), smem)) return ZERO_ECUDA;
    kernel<<<grid, block, smem, stream>>>(G, P, D, dy, du, y, h, dx, dh);
    return cuda_status(cudaGetLastError());
}

template <typename Act, typename Res>
int launch_backward(const Geometry& G, const Params& P, const Grads& D, bool full, const void* dy,
                    const void* du, const void* y, const void* h, void* dx, void* dh,
                    cudaStream_t stream)
{
    const auto* dyp = static_cast<const Res*>(dy);
    const auto* dup = static_cast<const Act*>(du);
    const auto* yp = static_cast<const Res*>(y);
    const auto* hp = static_cast<const Act*>(h);
    auto* dxp = static_cast<Res*>(dx);
    auto* dhp = static_cast<Act*>(dh);
    switch (vectors_per_thread(G.dim, G.classes, true)) {
    case 1: return start_backward<1>(G, P, D, full, dyp, dup, yp, hp, dxp, dhp, stream);
    case 2: return start_backward<2>(G, P, D, full, dyp, dup, yp, hp, dxp, dhp, stream);
    default: return start_backward<4>(G, P, D, full, dyp, dup, yp, hp, dxp, dhp, stream);
    }
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
    Geometry G = geometry(norm->n_rows, norm->dim, norm->rows_per_gate,
                                aligned16(x) && aligned16(branch) && aligned16(y) && aligned16(u),
                                false);
    const Params P = make_params(norm, gate, post_weight, post_bias, pre_weight, pre_bias);
    // As many blocks as are resident at once: 16384 x 1000 takes 27.2 us with 456
    // where three fit an SM, 31.5 with 304; where two fit, 16384 x 4096 takes 90 us
    // with 304, 104 with 456.  A row's result does not depend on it.
    if (vectors_per_thread(G.dim, G.classes, false) == 1 && G.threads <= 256 &&
        mode_of(G, P.layer || P.post_b || P.pre_b) == kPlain) {
        const int64_t blocks = (G.rows + G.groups - 1) / G.groups;
        G.blocks = static_cast<int32_t>(blocks < kMaxPlainBlocks ? blocks : kMaxPlainBlocks);
    }
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
    const bool full = P.layer || post_bias || grads->dpost_bias || grads->dpre_bias;
    int status;
    if (norm->act_type == ZERO_TYPE_F32)
        status = launch_backward<float, float>(G, P, D, full, dy, du, y, branch, dx, dbranch, stream);
    else if (norm->res_type == ZERO_TYPE_F32)
        status = launch_backward<Bf16, float>(G, P, D, full, dy, du, y, branch, dx, dbranch, stream);
    else
        status = launch_backward<Bf16, Bf16>(G, P, D, full, dy, du, y, branch, dx, dbranch, stream);
    if (status != ZERO_OK) return status;
    Finals F = {};
    F.out[0] = grads->dpost_weight;
    F.out[1] = grads->dpost_bias;
    F.out[2] = grads->dpre_weight;
    F.out[3] = grads->dpre_bias;
    F.out[4] = grads->dgate;
    for (int i = 0; i < kVectors; ++i) F.type[i] = grads->grad_type;
    F.type[kVectors] = grads->dgate_type;
    // gate rows of one token are final already
    const int64_t workers = static_cast<int64_t>(G.blocks) * G.groups;
    const int64_t shared = D.gate_rows > 1 && G.span > 1 ? D.gate_rows : 0;
    D.by_ends = shared > workers - 1;
    const int64_t tasks = D.vectors + (D.by_ends ? workers - 1 : shared);
    const bool four = G.dim % 4 == 0;
    const dim3 grid(static_cast<unsigned>((G.dim + (four ? 127 : 31)) / (four ? 128 : 32)),
                    static_cast<unsigned>(tasks));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(32 * kSlices);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cuda_status(four ? cudaLaunchKernelEx(&cfg, reduce_kernel<4>, G, D, F)
                            : cudaLaunchKernelEx(&cfg, reduce_kernel<1>, G, D, F));
}

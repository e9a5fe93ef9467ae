// group_norm.cu -- group norm with an activation, channels last
// (zero_group_norm_forward), and its gradient (zero_group_norm_backward).
//
//   h = (x - mean) * rstd, z = h * weight + bias, y = act(z)
//   d = dy * act'(z), dbias = sum d, dweight = sum d h
//   dx = rstd * (d * weight - s1 - h * s2),  s1 = mean of d * weight, s2 = mean of
//   d * weight * h over the group
//
// A sample's positions are cut into chunks, its channels into slabs of whole
// groups; a block takes the rows of one chunk of one slab, a thread one vector of
// channels (8 where rows and addresses allow 16-byte accesses, else 1) and every
// row_groups-th row.  Statistics: a thread sums each channel's differences from
// its own first value (at most kRows rows, so the squares of the differences are at
// most 2 + 2 * kRows times those about the mean and fp32 keeps the variance to
// kRows roundings even where that first value is an outlier); block, chunks and
// groups are joined by means and sums of squares about them.  The gradient's sums
// are per channel first: sums of d and d * h give dbias and dweight, and, weighed,
// s1 and s2.
#include <cmath>

#include "typed.cuh"
#include "zero_internal.h"

namespace zero {
namespace {

using dev::Bf16;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 32; // rows of a thread in a chunk, at most
constexpr int64_t kMaxChannels = 16384;
constexpr int64_t kMaxCount = int64_t(1) << 30;

struct Geometry {
    int64_t positions, x_stride, y_stride;
    const int32_t* lengths;
    int32_t samples, channels, groups, per; // per: channels of a group
    int32_t slab_groups, slabs;             // whole groups; the last slab may have fewer
    int32_t lanes, tiles;                   // vectors of a row that the block takes at once
    int32_t row_groups;                     // rows that it takes at once
    int32_t rows, chunks;                   // rows of a chunk, chunks of a sample
    int32_t vec;                            // channels of a vector: 8 or 1
};

struct Place { // a block's work
    int n, chunk, first_group, n_groups, c0, width; // channels c0 .. c0 + width - 1
    int row0, rows;                                 // 0 rows: nothing to do
};

__device__ __forceinline__ int length_of(const Geometry& G, int n)
{
    const int most = static_cast<int>(G.positions);
    if (!G.lengths) return most;
    const int len = G.lengths[n];
    return len < 0 ? 0 : len < most ? len : most;
}

__device__ __forceinline__ Place place_of(const Geometry& G, int64_t block)
{
    Place p;
    p.chunk = static_cast<int>(block % G.chunks);
    const int64_t unit = block / G.chunks;
    const int slab = static_cast<int>(unit % G.slabs);
    p.n = static_cast<int>(unit / G.slabs);
    p.first_group = slab * G.slab_groups;
    p.n_groups = min(G.slab_groups, G.groups - p.first_group);
    p.c0 = p.first_group * G.per;
    p.width = p.n_groups * G.per;
    p.row0 = p.chunk * G.rows;
    p.rows = max(0, min(G.rows, length_of(G, p.n) - p.row0));
    return p;
}

// ---------------------------------------------------------------- activation
template <int kAct>
__device__ __forceinline__ float activated(float z)
{
    if constexpr (kAct == ZERO_ACT_SILU) return z * __fdividef(1.0f, 1.0f + __expf(-z));
    if constexpr (kAct == ZERO_ACT_GELU) return z * fmaf(0.5f, erff(z * 0.70710678f), 0.5f);
    return z;
}
template <int kAct>
__device__ __forceinline__ float slope(float z)
{
    if constexpr (kAct == ZERO_ACT_SILU) {
        const float p = __fdividef(1.0f, 1.0f + __expf(-z));
        return p * fmaf(z, 1.0f - p, 1.0f);
    }
    if constexpr (kAct == ZERO_ACT_GELU) {
        const float cdf = fmaf(0.5f, erff(z * 0.70710678f), 0.5f);
        return fmaf(z * 0.39894228f, __expf(-0.5f * z * z), cdf);
    }
    return 1.0f;
}

template <int kVec>
__device__ __forceinline__ void load_param(const void* p, int32_t type, int c, float absent,
                                           float (&x)[kVec])
{
    if (p) {
        // a parameter may start at any of its elements
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            float one[1];
            dev::load_any<1>(p, type, c + e, one);
            x[e] = one[0];
        }
    } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) x[e] = absent;
    }
}

// ------------------------------------------------------------------- forward
// Mean and sum of squares about it of each group in each chunk.
template <int kVec, typename T>
__global__ void __launch_bounds__(kThreads)
chunk_stats_kernel(const __grid_constant__ Geometry G, const T* __restrict__ x,
                   float2* __restrict__ partial)
{
    __shared__ float means[kThreads * kVec], squares[kThreads * kVec];
    __shared__ float3 joined[8]; // where a slab takes several tiles: the groups so far
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Place p = place_of(G, blockIdx.x);
    if (p.rows == 0) return;
    const int rg = threadIdx.x / G.lanes, lane = threadIdx.x - rg * G.lanes;
    const int warp = threadIdx.x >> 5, wl = threadIdx.x & 31;
    const T* base = x + (static_cast<int64_t>(p.n) * G.positions + p.row0) * G.x_stride + p.c0;
    float2* out = partial + (static_cast<int64_t>(p.n) * G.chunks + p.chunk) * G.groups + p.first_group;
    for (int tile = 0; tile < G.tiles; ++tile) {
        const int tile_c = tile * G.lanes * kVec;
        const int c = tile_c + lane * kVec;
        const int tile_width = min(G.lanes * kVec, p.width - tile_c);
        if (rg < G.row_groups && c < p.width) {
            float shift[kVec], s[kVec], q[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e) shift[e] = s[e] = q[e] = 0.0f;
            const T* at = base + c + rg * G.x_stride;
            const int64_t step = G.row_groups * G.x_stride;
            if (rg < p.rows) dev::load_vec<kVec>(at, shift);
            int count = 0;
#pragma unroll 4
            for (int r = rg; r < p.rows; r += G.row_groups, at += step, ++count) {
                float v[kVec];
                dev::load_vec<kVec>(at, v);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const float d = v[e] - shift[e];
                    s[e] += d;
                    q[e] = fmaf(d, d, q[e]);
                }
            }
            const float inv = count > 0 ? 1.0f / static_cast<float>(count) : 0.0f;
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float m = s[e] * inv;
                means[rg * G.lanes * kVec + lane * kVec + e] = shift[e] + m;
                squares[rg * G.lanes * kVec + lane * kVec + e] = fmaxf(fmaf(-s[e], m, q[e]), 0.0f);
            }
        }
        __syncthreads();
        const int live = min(G.row_groups, p.rows); // row groups that have rows
        const int g_first = tile_c / G.per, g_last = (tile_c + tile_width - 1) / G.per;
        for (int g = g_first + warp; g <= g_last; g += kWarps) {
            const int lo = max(g * G.per - tile_c, 0);
            const int hi = min((g + 1) * G.per - tile_c, tile_width);
            const int w = hi - lo, entries = w * live;
            float sum = 0.0f;
            for (int i = wl; i < entries; i += 32) {
                const int r = i / w, k = r * G.lanes * kVec + lo + (i - r * w);
                const int count = (p.rows - r + G.row_groups - 1) / G.row_groups;
                sum = fmaf(static_cast<float>(count), means[k], sum);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
            const float n = static_cast<float>(w) * static_cast<float>(p.rows);
            const float mean = sum / n;
            float m2 = 0.0f;
            for (int i = wl; i < entries; i += 32) {
                const int r = i / w, k = r * G.lanes * kVec + lo + (i - r * w);
                const int count = (p.rows - r + G.row_groups - 1) / G.row_groups;
                const float d = means[k] - mean;
                m2 += fmaf(static_cast<float>(count) * d, d, squares[k]);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) m2 += __shfl_xor_sync(0xFFFFFFFFu, m2, off);
            if (wl == 0) {
                float3 a = make_float3(n, mean, m2);
                if (G.tiles > 1 && g * G.per < tile_c) { // begun in a tile before
                    const float3 b = joined[g];
                    const float all = a.x + b.x, d = a.y - b.y;
                    a = make_float3(all, fmaf(d, a.x / all, b.y),
                                    a.z + b.z + d * d * (a.x / all) * b.x);
                }
                if (G.tiles > 1 && (g + 1) * G.per > tile_c + tile_width)
                    joined[g] = a;
                else
                    out[g] = make_float2(a.y, a.z);
            }
        }
        if (G.tiles > 1) __syncthreads();
    }
}

// A warp joins the chunks of one group of one sample.
__global__ void __launch_bounds__(kThreads)
stats_kernel(const __grid_constant__ Geometry G, const float2* __restrict__ partial, float eps,
             float2* __restrict__ stats)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (unit >= static_cast<int64_t>(G.samples) * G.groups) return;
    const int n = static_cast<int>(unit / G.groups), g = static_cast<int>(unit % G.groups);
    const int len = length_of(G, n);
    const int chunks = (len + G.rows - 1) / G.rows;
    const float2* from = partial + static_cast<int64_t>(n) * G.chunks * G.groups + g;
    float sum = 0.0f;
    for (int k = lane; k < chunks; k += 32)
        sum = fmaf(static_cast<float>(min(G.rows, len - k * G.rows)),
                   from[static_cast<int64_t>(k) * G.groups].x, sum);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
    const float mean = len > 0 ? sum / static_cast<float>(len) : 0.0f;
    float m2 = 0.0f;
    for (int k = lane; k < chunks; k += 32) {
        const float2 a = from[static_cast<int64_t>(k) * G.groups];
        const float d = a.x - mean;
        const float w = static_cast<float>(min(G.rows, len - k * G.rows)) * static_cast<float>(G.per);
        m2 += fmaf(w * d, d, a.y);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m2 += __shfl_xor_sync(0xFFFFFFFFu, m2, off);
    if (lane == 0) {
        const float count = static_cast<float>(len) * static_cast<float>(G.per);
        const float var = len > 0 ? m2 / count : 0.0f;
        stats[unit] = make_float2(mean, 1.0f / sqrtf(var + eps));
    }
}

template <int kVec, typename T, int kAct>
__global__ void __launch_bounds__(kThreads)
apply_kernel(const __grid_constant__ Geometry G, const T* x, const void* __restrict__ weight,
             const void* __restrict__ bias, int32_t param_type,
             const float2* __restrict__ stats, T* y)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Place p = place_of(G, blockIdx.x);
    const int rg = threadIdx.x / G.lanes, lane = threadIdx.x - rg * G.lanes;
    if (rg >= G.row_groups || rg >= p.rows) return;
    const int64_t row = static_cast<int64_t>(p.n) * G.positions + p.row0 + rg;
    for (int c = lane * kVec; c < p.width; c += G.lanes * kVec) {
        float mean[kVec], a[kVec], b[kVec];
        load_param<kVec>(weight, param_type, p.c0 + c, 1.0f, a);
        load_param<kVec>(bias, param_type, p.c0 + c, 0.0f, b);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const float2 s = stats[static_cast<int64_t>(p.n) * G.groups + (p.c0 + c + e) / G.per];
            mean[e] = s.x;
            a[e] *= s.y;
        }
        const T* from = x + row * G.x_stride + p.c0 + c;
        T* to = y + row * G.y_stride + p.c0 + c;
        const int64_t x_step = G.row_groups * G.x_stride, y_step = G.row_groups * G.y_stride;
        constexpr int kAhead = 4;
        for (int r = rg; r < p.rows; r += kAhead * G.row_groups) {
            float v[kAhead][kVec];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (r + k * G.row_groups < p.rows) dev::load_vec<kVec>(from + k * x_step, v[k]);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (r + k * G.row_groups >= p.rows) break;
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    v[k][e] = activated<kAct>(fmaf(v[k][e] - mean[e], a[e], b[e]));
                if constexpr (kVec == 8)
                    dev::store8_stream(to + k * y_step, v[k]);
                else
                    dev::store1(to + k * y_step, v[k][0]);
            }
            from += kAhead * x_step;
            to += kAhead * y_step;
        }
    }
}

// ------------------------------------------------------------------ backward
// Sums of d and d * h of each channel in each chunk.
template <int kVec, typename T, int kAct>
__global__ void __launch_bounds__(kThreads)
chunk_sums_kernel(const __grid_constant__ Geometry G, const T* __restrict__ x,
                  const T* __restrict__ dy, const void* __restrict__ weight,
                  const void* __restrict__ bias, int32_t param_type,
                  const float2* __restrict__ stats, float2* __restrict__ partial)
{
    __shared__ float straight[kThreads * kVec], along[kThreads * kVec];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Place p = place_of(G, blockIdx.x);
    if (p.rows == 0) return;
    const int rg = threadIdx.x / G.lanes, lane = threadIdx.x - rg * G.lanes;
    const int64_t row = static_cast<int64_t>(p.n) * G.positions + p.row0 + rg;
    float2* out = partial + (static_cast<int64_t>(p.n) * G.chunks + p.chunk) * G.channels + p.c0;
    for (int tile_c = 0; tile_c < p.width; tile_c += G.lanes * kVec) {
        const int c = tile_c + lane * kVec;
        if (rg < G.row_groups && c < p.width) {
            float mean[kVec], rstd[kVec], w[kVec], b[kVec], s[kVec], q[kVec];
            load_param<kVec>(weight, param_type, p.c0 + c, 1.0f, w);
            load_param<kVec>(bias, param_type, p.c0 + c, 0.0f, b);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float2 st = stats[static_cast<int64_t>(p.n) * G.groups + (p.c0 + c + e) / G.per];
                mean[e] = st.x;
                rstd[e] = st.y;
                s[e] = q[e] = 0.0f;
            }
            const T* xp = x + row * G.x_stride + p.c0 + c;
            const T* dp = dy + row * G.y_stride + p.c0 + c;
            const int64_t x_step = G.row_groups * G.x_stride, y_step = G.row_groups * G.y_stride;
#pragma unroll 2
            for (int r = rg; r < p.rows; r += G.row_groups, xp += x_step, dp += y_step) {
                float v[kVec], d[kVec];
                dev::load_vec<kVec>(xp, v);
                dev::load_vec<kVec>(dp, d);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const float h = (v[e] - mean[e]) * rstd[e];
                    const float g = kAct ? d[e] * slope<kAct>(fmaf(h, w[e], b[e])) : d[e];
                    s[e] += g;
                    q[e] = fmaf(g, h, q[e]);
                }
            }
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                straight[rg * G.lanes * kVec + lane * kVec + e] = s[e];
                along[rg * G.lanes * kVec + lane * kVec + e] = q[e];
            }
        }
        __syncthreads();
        for (int k = threadIdx.x; k < min(G.lanes * kVec, p.width - tile_c); k += kThreads) {
            float s = 0.0f, q = 0.0f;
            for (int r = 0; r < G.row_groups; ++r) {
                s += straight[r * G.lanes * kVec + k];
                q += along[r * G.lanes * kVec + k];
            }
            out[tile_c + k] = make_float2(s, q);
        }
        __syncthreads();
    }
}

// The chunks' sums of one channel of one sample.
__global__ void __launch_bounds__(kThreads)
channel_sums_kernel(const __grid_constant__ Geometry G, const float2* __restrict__ partial,
                    float2* __restrict__ sums)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (at >= static_cast<int64_t>(G.samples) * G.channels) return;
    const int n = static_cast<int>(at / G.channels), c = static_cast<int>(at % G.channels);
    const int chunks = (length_of(G, n) + G.rows - 1) / G.rows;
    const float2* from = partial + static_cast<int64_t>(n) * G.chunks * G.channels + c;
    float s = 0.0f, q = 0.0f;
#pragma unroll 8
    for (int k = 0; k < chunks; ++k) {
        const float2 v = from[static_cast<int64_t>(k) * G.channels];
        s += v.x;
        q += v.y;
    }
    sums[at] = make_float2(s, q);
}

// Blocks below group_blocks: a warp for each group of each sample, its means of
// d * weight and d * weight * h; the others: a thread for each channel, dweight and
// dbias over the samples.
__global__ void __launch_bounds__(kThreads)
group_sums_kernel(const __grid_constant__ Geometry G, const float2* __restrict__ sums,
                  const void* __restrict__ weight, int32_t param_type, int64_t group_blocks,
                  float2* __restrict__ group_means, void* dweight, void* dbias, int32_t grad_type)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x < group_blocks) {
        const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
        const int lane = threadIdx.x & 31;
        if (unit >= static_cast<int64_t>(G.samples) * G.groups) return;
        const int n = static_cast<int>(unit / G.groups), g = static_cast<int>(unit % G.groups);
        const float2* from = sums + static_cast<int64_t>(n) * G.channels;
        float s = 0.0f, q = 0.0f;
        for (int c = g * G.per + lane; c < (g + 1) * G.per; c += 32) {
            float w[1];
            load_param<1>(weight, param_type, c, 1.0f, w);
            const float2 v = from[c];
            s = fmaf(w[0], v.x, s);
            q = fmaf(w[0], v.y, q);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
            q += __shfl_xor_sync(0xFFFFFFFFu, q, off);
        }
        if (lane == 0) {
            const float count = static_cast<float>(length_of(G, n)) * static_cast<float>(G.per);
            const float inv = count > 0.0f ? 1.0f / count : 0.0f;
            group_means[unit] = make_float2(s * inv, q * inv);
        }
        return;
    }
    const int c = static_cast<int>((blockIdx.x - group_blocks) * 32 + (threadIdx.x & 31));
    const int slice = threadIdx.x >> 5;
    __shared__ float2 slices[kWarps][32];
    float s = 0.0f, q = 0.0f;
    if (c < G.channels) {
#pragma unroll 4
        for (int n = slice; n < G.samples; n += kWarps) {
            const float2 v = sums[static_cast<int64_t>(n) * G.channels + c];
            s += v.x;
            q += v.y;
        }
    }
    slices[slice][threadIdx.x & 31] = make_float2(s, q);
    __syncthreads();
    if (slice == 0 && c < G.channels) {
        float a[1] = {0.0f}, b[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            a[0] += slices[k][threadIdx.x].x;
            b[0] += slices[k][threadIdx.x].y;
        }
        if (dbias) dev::store_any<1>(dbias, grad_type, c, a);
        if (dweight) dev::store_any<1>(dweight, grad_type, c, b);
    }
}

template <int kVec, typename T, int kAct>
__global__ void __launch_bounds__(kThreads)
apply_gradient_kernel(const __grid_constant__ Geometry G, const T* __restrict__ x, const T* dy,
                      const void* __restrict__ weight, const void* __restrict__ bias,
                      int32_t param_type, const float2* __restrict__ stats,
                      const float2* __restrict__ group_means, T* dx)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Place p = place_of(G, blockIdx.x);
    const int rg = threadIdx.x / G.lanes, lane = threadIdx.x - rg * G.lanes;
    if (rg >= G.row_groups || rg >= p.rows) return;
    const int64_t row = static_cast<int64_t>(p.n) * G.positions + p.row0 + rg;
    for (int c = lane * kVec; c < p.width; c += G.lanes * kVec) {
        float mean[kVec], rstd[kVec], w[kVec], b[kVec], s1[kVec], s2[kVec];
        load_param<kVec>(weight, param_type, p.c0 + c, 1.0f, w);
        load_param<kVec>(bias, param_type, p.c0 + c, 0.0f, b);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const int64_t unit = static_cast<int64_t>(p.n) * G.groups + (p.c0 + c + e) / G.per;
            const float2 st = stats[unit], m = group_means[unit];
            mean[e] = st.x;
            rstd[e] = st.y;
            s1[e] = m.x;
            s2[e] = m.y;
        }
        const T* xp = x + row * G.x_stride + p.c0 + c;
        const T* dp = dy + row * G.y_stride + p.c0 + c;
        T* to = dx + row * G.x_stride + p.c0 + c;
        const int64_t x_step = G.row_groups * G.x_stride, y_step = G.row_groups * G.y_stride;
#pragma unroll 2
        for (int r = rg; r < p.rows; r += G.row_groups, xp += x_step, dp += y_step, to += x_step) {
            float v[kVec], d[kVec];
            dev::load_vec<kVec>(xp, v);
            dev::load_vec<kVec>(dp, d);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float h = (v[e] - mean[e]) * rstd[e];
                const float g = kAct ? d[e] * slope<kAct>(fmaf(h, w[e], b[e])) : d[e];
                v[e] = rstd[e] * fmaf(-h, s2[e], fmaf(g, w[e], -s1[e]));
            }
            if constexpr (kVec == 8)
                dev::store8_stream(to, v);
            else
                dev::store1(to, v[0]);
        }
    }
}

// --------------------------------------------------------------------- host
bool sizes_ok(int64_t samples, int64_t positions, int64_t channels, int32_t groups)
{
    return samples >= 0 && samples <= kMaxCount && positions >= 0 && positions <= kMaxCount &&
           samples * positions <= (int64_t(1) << 40) && channels >= 1 &&
           channels <= kMaxChannels && samples * channels <= (int64_t(1) << 34) && groups >= 1 &&
           channels % groups == 0;
}

// By the sizes and whether 16-byte accesses are possible alone.
Geometry geometry(int64_t samples, int64_t positions, int64_t channels, int32_t groups, bool wide)
{
    Geometry G = {};
    const int vec = G.vec = wide ? 8 : 1;
    G.samples = static_cast<int32_t>(samples);
    G.positions = positions;
    G.channels = static_cast<int32_t>(channels);
    G.groups = groups;
    G.per = G.channels / groups;
    // groups that fill whole vectors together
    int unit = 1;
    while (unit * G.per % vec != 0) ++unit;
    G.slab_groups = kThreads * vec / (unit * G.per) * unit;
    if (G.slab_groups < unit) G.slab_groups = unit;
    if (G.slab_groups > groups) G.slab_groups = groups;
    G.slabs = (groups + G.slab_groups - 1) / G.slab_groups;
    const int vecs = G.slab_groups * G.per / vec;
    G.tiles = (vecs + kThreads - 1) / kThreads;
    G.lanes = (vecs + G.tiles - 1) / G.tiles;
    G.row_groups = kThreads / G.lanes;
    int64_t rows = samples * G.slabs * positions / (static_cast<int64_t>(G.row_groups) * 152 * 8);
    if (rows < 4) rows = 4;
    if (rows > kRows) rows = kRows;
    G.rows = static_cast<int32_t>(rows) * G.row_groups;
    G.chunks = static_cast<int32_t>((positions + G.rows - 1) / G.rows);
    return G;
}

int64_t blocks_of(const Geometry& G)
{
    return static_cast<int64_t>(G.samples) * G.slabs * G.chunks;
}

// Scratch: [partial][sums][group means or stats].
struct Scratch {
    float2 *partial, *sums, *groups;
    int64_t bytes;
};
Scratch scratch_of(void* base, int64_t samples, int64_t positions, int64_t channels, int32_t groups)
{
    int64_t chunks = 0;
    for (int wide = 0; wide < 2; ++wide) {
        if (wide && channels % 8 != 0) continue;
        const Geometry G = geometry(samples, positions, channels, groups, wide != 0);
        if (G.chunks > chunks) chunks = G.chunks;
    }
    Scratch s;
    s.partial = static_cast<float2*>(base);
    const int64_t n = samples * chunks * channels, m = samples * channels;
    s.sums = s.partial + n;
    s.groups = s.sums + m;
    s.bytes = (n + m + samples * groups) * 8;
    s.bytes = (s.bytes + 15) / 16 * 16;
    return s;
}

// A launch that may begin while the kernel before it on the stream drains; the
// kernel waits for that one's results itself.
template <typename... Params, typename... Given>
int launch(bool after, void (*kernel)(Params...), int64_t blocks, cudaStream_t stream, Given... given)
{
    if (blocks > 0x7FFFFFFF) return ZERO_EINVAL;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = after ? 1 : 0;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(given)...));
}

struct Call {
    const zero_group_norm_t* norm;
    Geometry G;
    Scratch s;
    const void *x, *dy, *weight, *bias;
    const float2* stats;
    void *y, *dx, *dweight, *dbias;
    cudaStream_t stream;
};

template <int kVec, typename T, int kAct>
int forward(const Call& c, float2* stats)
{
    const Geometry& G = c.G;
    const int64_t blocks = blocks_of(G);
    const int64_t units = static_cast<int64_t>(G.samples) * G.groups;
    int rc = ZERO_OK;
    if (blocks > 0)
        rc = launch(false, chunk_stats_kernel<kVec, T>, blocks, c.stream, G,
                    static_cast<const T*>(c.x), c.s.partial);
    if (rc == ZERO_OK)
        rc = launch(blocks > 0, stats_kernel, (units + kWarps - 1) / kWarps, c.stream, G, c.s.partial,
                    static_cast<float>(c.norm->eps), stats);
    if (rc == ZERO_OK && blocks > 0)
        rc = launch(true, apply_kernel<kVec, T, kAct>, blocks, c.stream, G,
                    static_cast<const T*>(c.x), c.weight, c.bias, c.norm->param_type, stats,
                    static_cast<T*>(c.y));
    return rc;
}

template <int kVec, typename T, int kAct>
int backward(const Call& c)
{
    const Geometry& G = c.G;
    const int64_t blocks = blocks_of(G);
    const int64_t units = static_cast<int64_t>(G.samples) * G.groups;
    const auto* x = static_cast<const T*>(c.x);
    const auto* dy = static_cast<const T*>(c.dy);
    int rc = ZERO_OK;
    if (blocks > 0)
        rc = launch(false, chunk_sums_kernel<kVec, T, kAct>, blocks, c.stream, G, x, dy, c.weight,
                    c.bias, c.norm->param_type, c.stats, c.s.partial);
    const int64_t channels = static_cast<int64_t>(G.samples) * G.channels;
    if (rc == ZERO_OK && channels > 0)
        rc = launch(blocks > 0, channel_sums_kernel, (channels + kThreads - 1) / kThreads, c.stream, G,
                    c.s.partial, c.s.sums);
    const int64_t group_blocks = c.dx ? (units + kWarps - 1) / kWarps : 0;
    const int64_t more = c.dweight || c.dbias ? (G.channels + 31) / 32 : 0;
    if (rc == ZERO_OK && group_blocks + more > 0)
        rc = launch(channels > 0, group_sums_kernel, group_blocks + more, c.stream, G, c.s.sums, c.weight,
                    c.norm->param_type, group_blocks, c.s.groups, c.dweight, c.dbias,
                    c.norm->grad_type);
    if (rc == ZERO_OK && c.dx && blocks > 0)
        rc = launch(true, apply_gradient_kernel<kVec, T, kAct>, blocks, c.stream, G, x, dy, c.weight,
                    c.bias, c.norm->param_type, c.stats, c.s.groups, static_cast<T*>(c.dx));
    return rc;
}

int check(const zero_group_norm_t* n, const void* weight, const void* bias, const int32_t* lengths,
          void* scratch, int64_t scratch_bytes)
{
    if (!n || !sizes_ok(n->samples, n->positions, n->channels, n->groups) || !float_type(n->type) ||
        !float_type(n->param_type) || n->act < ZERO_ACT_NONE || n->act > ZERO_ACT_GELU)
        return ZERO_EINVAL;
    if (n->x_stride < n->channels || n->x_stride > (int64_t(1) << 30) ||
        n->y_stride < n->channels || n->y_stride > (int64_t(1) << 30))
        return ZERO_EINVAL;
    if (!scratch || scratch_bytes < scratch_of(nullptr, n->samples, n->positions, n->channels,
                                               n->groups).bytes)
        return ZERO_EINVAL;
    if (!aligned_to(weight, type_bytes(n->param_type)) ||
        !aligned_to(bias, type_bytes(n->param_type)) || !aligned_to(lengths, 4) || !aligned16(scratch))
        return ZERO_EALIGN;
    return ZERO_OK;
}

Geometry of_call(const zero_group_norm_t* n, const int32_t* lengths, bool aligned)
{
    const int unit = 16 / type_bytes(n->type);
    const bool wide = aligned && n->channels % 8 == 0 && n->x_stride % unit == 0 &&
                      n->y_stride % unit == 0;
    Geometry G = geometry(n->samples, n->positions, n->channels, n->groups, wide);
    G.x_stride = n->x_stride;
    G.y_stride = n->y_stride;
    G.lengths = lengths;
    return G;
}


template <int kVec, typename T>
int forward_by_act(const Call& c, float2* stats)
{
    switch (c.norm->act) {
    case ZERO_ACT_SILU: return forward<kVec, T, ZERO_ACT_SILU>(c, stats);
    case ZERO_ACT_GELU: return forward<kVec, T, ZERO_ACT_GELU>(c, stats);
    default: return forward<kVec, T, ZERO_ACT_NONE>(c, stats);
    }
}

template <int kVec, typename T>
int backward_by_act(const Call& c)
{
    switch (c.norm->act) {
    case ZERO_ACT_SILU: return backward<kVec, T, ZERO_ACT_SILU>(c);
    case ZERO_ACT_GELU: return backward<kVec, T, ZERO_ACT_GELU>(c);
    default: return backward<kVec, T, ZERO_ACT_NONE>(c);
    }
}

} // namespace
} // namespace zero

using namespace zero;

extern "C" int64_t zero_group_norm_scratch_bytes(int64_t samples, int64_t positions,
                                                 int64_t channels, int32_t groups)
{
    if (!sizes_ok(samples, positions, channels, groups)) return ZERO_EINVAL;
    return scratch_of(nullptr, samples, positions, channels, groups).bytes;
}

extern "C" int zero_group_norm_forward(const zero_group_norm_t* norm, const void* x,
                                       const void* weight, const void* bias,
                                       const int32_t* lengths, void* y, float* stats,
                                       void* scratch, int64_t scratch_bytes, cudaStream_t stream)
{
    const int rc = check(norm, weight, bias, lengths, scratch, scratch_bytes);
    if (rc != ZERO_OK) return rc;
    if (!std::isfinite(norm->eps) || static_cast<float>(norm->eps) <= 0) return ZERO_EINVAL;
    if (norm->samples == 0) return ZERO_OK;
    if (norm->positions > 0 && (!x || !y || (x == y && norm->x_stride != norm->y_stride)))
        return ZERO_EINVAL;
    const int tb = type_bytes(norm->type);
    if (!aligned_to(x, tb) || !aligned_to(y, tb) || !aligned_to(stats, 8)) return ZERO_EALIGN;
    Call c = {};
    c.norm = norm;
    c.G = of_call(norm, lengths, aligned16(x) && aligned16(y));
    if (blocks_of(c.G) > 0x7FFFFFFF) return ZERO_EINVAL;
    c.s = scratch_of(scratch, norm->samples, norm->positions, norm->channels, norm->groups);
    c.x = x;
    c.weight = weight;
    c.bias = bias;
    c.y = y;
    c.stream = stream;
    auto* to = stats ? reinterpret_cast<float2*>(stats) : c.s.groups;
    if (norm->type == ZERO_TYPE_BF16)
        return c.G.vec == 8 ? forward_by_act<8, Bf16>(c, to) : forward_by_act<1, Bf16>(c, to);
    return c.G.vec == 8 ? forward_by_act<8, float>(c, to) : forward_by_act<1, float>(c, to);
}

extern "C" int zero_group_norm_backward(const zero_group_norm_t* norm, const void* x,
                                        const void* dy, const void* weight, const void* bias,
                                        const int32_t* lengths, const float* stats, void* dx,
                                        void* dweight, void* dbias, void* scratch,
                                        int64_t scratch_bytes, cudaStream_t stream)
{
    const int rc = check(norm, weight, bias, lengths, scratch, scratch_bytes);
    if (rc != ZERO_OK) return rc;
    if (!float_type(norm->grad_type)) return ZERO_EINVAL;
    if (norm->samples > 0 && norm->positions > 0 &&
        (!x || !dy || !stats || (dx == dy && norm->x_stride != norm->y_stride)))
        return ZERO_EINVAL;
    const int tb = type_bytes(norm->type), gb = type_bytes(norm->grad_type);
    if (!aligned_to(x, tb) || !aligned_to(dy, tb) || !aligned_to(dx, tb) ||
        !aligned_to(stats, 8) || !aligned_to(dweight, gb) || !aligned_to(dbias, gb))
        return ZERO_EALIGN;
    Call c = {};
    c.norm = norm;
    c.G = of_call(norm, lengths, aligned16(x) && aligned16(dy) && aligned16(dx));
    if (blocks_of(c.G) > 0x7FFFFFFF) return ZERO_EINVAL;
    c.s = scratch_of(scratch, norm->samples, norm->positions, norm->channels, norm->groups);
    c.x = x;
    c.dy = dy;
    c.weight = weight;
    c.bias = bias;
    c.stats = reinterpret_cast<const float2*>(stats);
    c.dx = dx;
    c.dweight = dweight;
    c.dbias = dbias;
    c.stream = stream;
    if (norm->type == ZERO_TYPE_BF16)
        return c.G.vec == 8 ? backward_by_act<8, Bf16>(c) : backward_by_act<1, Bf16>(c);
    return c.G.vec == 8 ? backward_by_act<8, float>(c) : backward_by_act<1, float>(c);
}

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
#include <type_traits>

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
// 2^x to 2 ulp and 1/x to 1 ulp, one instruction each; results below 2^-126 are 0.
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float reciprocal_fast(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.44269504f;

// 1 / (1 + exp(-z)); an exponential that overflows gives 0.
__device__ __forceinline__ float2 sigmoid2(float2 z)
{
    const float2 t = dev::mul2(z, dev::pair(-kLog2e));
    const float2 d = dev::add2(make_float2(exp2_fast(t.x), exp2_fast(t.y)), dev::pair(1.0f));
    return make_float2(reciprocal_fast(d.x), reciprocal_fast(d.y));
}
__device__ __forceinline__ float2 normal_cdf2(float2 z)
{
    const float2 t = dev::mul2(z, dev::pair(0.70710678f));
    return dev::fma2(make_float2(erff(t.x), erff(t.y)), dev::pair(0.5f), dev::pair(0.5f));
}

template <int kAct>
__device__ __forceinline__ float2 activated2(float2 z)
{
    if constexpr (kAct == ZERO_ACT_SILU) return dev::mul2(z, sigmoid2(z));
    if constexpr (kAct == ZERO_ACT_GELU) return dev::mul2(z, normal_cdf2(z));
    return z;
}
template <int kAct>
__device__ __forceinline__ float2 slope2(float2 z)
{
    if constexpr (kAct == ZERO_ACT_SILU) {
        const float2 p = sigmoid2(z);
        return dev::mul2(p, dev::fma2(z, dev::fma2(p, dev::pair(-1.0f), dev::pair(1.0f)), dev::pair(1.0f)));
    }
    if constexpr (kAct == ZERO_ACT_GELU) {
        const float2 t = dev::mul2(dev::mul2(z, z), dev::pair(-0.5f * kLog2e));
        const float2 density = dev::mul2(make_float2(exp2_fast(t.x), exp2_fast(t.y)), dev::pair(0.39894228f));
        return dev::fma2(z, density, normal_cdf2(z));
    }
    return dev::pair(1.0f);
}
template <int kAct>
__device__ __forceinline__ float activated(float z)
{
    return activated2<kAct>(dev::pair(z)).x;
}
template <int kAct>
__device__ __forceinline__ float slope(float z)
{
    return slope2<kAct>(dev::pair(z)).x;
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

// ------------------------------------------------- samples held in shared memory
// The whole pass in one launch that reads every value from HBM once: a team of
// blocks holds one slab of one sample in its shared memory between the sums and
// the result, so nothing is read twice.  Each thread copies its own vectors there
// (cp.async), as many rows ahead as fit, sums them as they lie there, and while it
// forms the results puts the next sample's vectors in the places that become free.
// A team of one block needs nothing of others; larger ones exchange their groups'
// sums through global memory, counted on a word that a thread of each waits for.
// Such launches are cooperative: all blocks are resident, or the launch fails.
//
// Rows are positions (x_stride apart) where 16-byte accesses are possible at every
// position.  Else, where the channels are contiguous, they are runs of `repeats`
// positions that fill whole vectors (flat): the sample is taken as one line of
// values that starts `lead` elements behind a 16-byte boundary; element e of vector
// l of a row is value 8 l + e - lead of it, of channel (8 l + e - lead) mod channels.
struct Held {
    int64_t x_stride, y_stride; // elements between rows
    int64_t x_sample, y_sample; // and between samples
    const int32_t* lengths;
    int32_t samples, positions, channels, groups, per;
    int32_t slab_groups, slabs, width;  // groups and channels of a slab
    int32_t lanes, row_groups, repeats; // vectors of a row, rows at once, positions of a row
    int32_t slots, members, teams;      // rows of a thread; blocks of a team
};

constexpr int kHeldMaxBlocks = 152 * 3;
constexpr int kHeldWidth = 8 * kThreads; // channels of a slab, at most

__device__ __forceinline__ void put(float2& to, float, float mean, float m2) { to = make_float2(mean, m2); }
__device__ __forceinline__ void put(float4& to, float count, float mean, float m2)
{
    to = make_float4(mean, m2, count, 0.0f);
}

// Threads that share a channel of a slab where the blocks' row groups are joined.
__host__ __device__ __forceinline__ int parts_of(const Held& H)
{
    const int most = kThreads / H.width;
    return most < 1 ? 1 : most < H.row_groups ? most : H.row_groups;
}

__device__ __forceinline__ void copy_async(void* to, const void* from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(to))),
                 "l"(from)
                 : "memory");
}
__device__ __forceinline__ void copies_here()
{
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// A thread's vectors in shared memory: planes of 16 bytes a thread, one for bf16,
// two for fp32.
template <typename T>
struct Slot;
template <>
struct Slot<Bf16> {
    static constexpr int kPlanes = 1;
    template <typename X>
    static __device__ __forceinline__ void read(const float4* p, X& x)
    {
        dev::Raw8<Bf16> r;
        r.a = *reinterpret_cast<const uint4*>(p);
        dev::unpack8(r, x);
    }
    static __device__ __forceinline__ void fetch(float4* p, const Bf16* from) { copy_async(p, from); }
};
template <>
struct Slot<float> {
    static constexpr int kPlanes = 2;
    template <typename X>
    static __device__ __forceinline__ void read(const float4* p, X& x)
    {
        dev::Raw8<float> r;
        r.a = p[0];
        r.b = p[kThreads];
        dev::unpack8(r, x);
    }
    static __device__ __forceinline__ void fetch(float4* p, const float* from)
    {
        copy_async(p, from);
        copy_async(p + kThreads, from + 4);
    }
};
// Elements f .. l - 1 of the vector, one by one; the others are left as they are.
__device__ __forceinline__ void fetch_some(float4* p, const Bf16* from, int f, int l)
{
    auto* to = reinterpret_cast<Bf16*>(p);
    for (int e = f; e < l; ++e) to[e] = from[e];
}
__device__ __forceinline__ void fetch_some(float4* p, const float* from, int f, int l)
{
    for (int e = f; e < l; ++e) reinterpret_cast<float*>(p + (e >> 2) * kThreads)[e & 3] = from[e];
}

// Where a thread stands in the sample that its team works on.
struct Here {
    int n;     // the sample
    int rows;  // the thread's rows in it
    int total; // flat: values of the sample
    int lead;  // flat: elements that its first vector starts before it
    int first; // flat: the value of element 0 of the thread's first vector
};

template <bool kFlat, typename T>
__device__ __forceinline__ Here here_of(const Held& H, int n, const T* x, int rg, int lane, int row0)
{
    Here h;
    h.n = n;
    int len = H.positions;
    if (H.lengths) len = max(0, min(len, H.lengths[n]));
    int all = len;
    h.total = h.lead = h.first = 0;
    if (kFlat) {
        const int64_t at = static_cast<int64_t>(reinterpret_cast<uintptr_t>(x) / sizeof(T)) + n * H.x_sample;
        h.lead = static_cast<int>(at & (16 / static_cast<int>(sizeof(T)) - 1));
        h.total = len * H.channels;
        const int row = 8 * H.lanes;
        all = len > 0 ? (h.total + h.lead + row - 1) / row : 0;
        h.first = (row0 + rg) * row + lane * 8 - h.lead;
    }
    const int left = all - row0 - rg;
    h.rows = rg < H.row_groups && left > 0 ? min((left + H.row_groups - 1) / H.row_groups, H.slots) : 0;
    return h;
}

// The first value of the thread's row k, flat.
__device__ __forceinline__ int value_of(const Held& H, const Here& h, int k)
{
    return h.first + k * H.row_groups * 8 * H.lanes;
}

template <bool kFlat, typename T>
__device__ __forceinline__ void fetch_row(const Held& H, const Here& h, int k, float4* slot,
                                          const T* base, int64_t sample, int64_t stride)
{
    const T* from = base + h.n * sample + k * H.row_groups * stride;
    if (kFlat) {
        const int64_t at = h.n * sample + value_of(H, h, k); // in the tensor
        const int64_t behind = H.samples * sample - at;
        if (at < 0 || behind < 8) {
            fetch_some(slot, from, at < 0 ? static_cast<int>(-at) : 0, behind < 8 ? static_cast<int>(behind) : 8);
            return;
        }
    }
    Slot<T>::fetch(slot, from);
}

// Waits until `count` has reached `target`; false after about a second.
__device__ __forceinline__ bool wait_count(const uint32_t* count, uint32_t target)
{
    for (int i = 0; i < (1 << 20); ++i) {
        uint32_t v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(count) : "memory");
        if (static_cast<int32_t>(v - target) >= 0) return true;
        if (i > 32) __nanosleep(64);
    }
    return false;
}

// All threads of all blocks of a team, after they wrote what the others are to read:
// counts the block, and waits for the others of this turn.  A block whose wait runs
// out is lost from then on: it does not wait any more, and its results are NaN.
__device__ __forceinline__ void team_barrier(uint32_t* count, uint32_t target, int* lost)
{
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(count) : "memory");
        if (!*lost && !wait_count(count, target)) *lost = 1;
    }
    __syncthreads();
}

// Lanes that share a group's segments: a whole warp for many.
__device__ __forceinline__ int lanes_of_group(const Held& H)
{
    return max(H.row_groups, (H.per + 7) / 8) >= 24 ? 32 : 8;
}
// Lanes that share a group's members: as many as leave all groups a place.
__device__ __forceinline__ int lanes_of_members(int groups)
{
    return groups <= kWarps ? 32 : groups <= 2 * kWarps ? 16 : 8;
}

__device__ __forceinline__ float sum_lanes(float x, int lanes)
{
    for (int off = lanes / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
    return x;
}

// The groups of 8 neighbouring channels from c on (flat: around the end).
template <bool kFlat>
struct GroupWalk {
    int c, g, left;
    __device__ __forceinline__ GroupWalk(const Held& H, int first) : c(first)
    {
        g = c / H.per;
        left = (g + 1) * H.per - c;
    }
    __device__ __forceinline__ void next(const Held& H)
    {
        ++c;
        if (--left == 0) {
            ++g;
            left = H.per;
            if (kFlat && c == H.channels) c = g = 0;
        }
    }
};
template <bool kFlat>
__device__ __forceinline__ int first_channel(const Held& H, const Here& h, int lane)
{
    return kFlat ? (lane * 8 + 8 * H.lanes - h.lead) % H.channels : lane * 8;
}

// Sums of a thread's 8 channels go by segments: of each of the (at most two) groups that
// the vector lies in where a group has 8 channels or more, else of each channel.
__host__ __device__ __forceinline__ int segments_of(const Held& H) { return H.per >= 8 ? 2 : 8; }

// Calls f(entry) for this lane's share of the segments of group g, an entry being segment *
// kThreads + thread; `firsts` holds the group of each thread's first channel.  Lanes go
// over whichever is more, vectors or row groups.
template <bool kFlat, typename F>
__device__ __forceinline__ void over_segments(const Held& H, int lead, const int* firsts, int g, int sub, int gl, F f)
{
    if (H.per >= 8) {
        const bool whole = kFlat && H.groups == 1; // rows of one group: all vectors, once
        for (int j = 0; j < (kFlat && !whole ? H.repeats : 1); ++j) {
            int p = g * H.per, nv = H.lanes;
            if (kFlat) {
                p = whole ? 0 : p + j * H.channels + lead;
                if (p >= 8 * H.lanes) p -= 8 * H.lanes;
            }
            const int v0 = p >> 3;
            if (!whole) nv = ((p & 7) + H.per + 7) >> 3;
            const bool by_vectors = nv >= H.row_groups;
            const int outer = by_vectors ? H.row_groups : nv, inner = by_vectors ? nv : H.row_groups;
            for (int a = 0; a < outer; ++a)
                for (int b = sub; b < inner; b += gl) {
                    int v = v0 + (by_vectors ? b : a);
                    if (kFlat && v >= H.lanes) v -= H.lanes;
                    const int t = (by_vectors ? a : b) * H.lanes + v;
                    f(whole || firsts[t] == g ? t : kThreads + t);
                }
        }
    } else {
        for (int j = 0; j < (kFlat ? H.repeats : 1); ++j)
            for (int c = 0; c < H.per; ++c) {
                int p = g * H.per + c;
                if (kFlat) {
                    p += j * H.channels + lead;
                    if (p >= 8 * H.lanes) p -= 8 * H.lanes;
                }
                for (int r = sub; r < H.row_groups; r += gl) f((p & 7) * kThreads + r * H.lanes + (p >> 3));
            }
    }
}

template <typename T, int kAct, bool kFlat>
__global__ void __launch_bounds__(kThreads, 2)
held_forward_kernel(const __grid_constant__ Held H, const T* x, const void* __restrict__ weight,
                    const void* __restrict__ bias, int32_t param_type, float eps, T* y,
                    float2* __restrict__ stats, uint32_t* counts, void* exchange_words)
{
    // mean, squares and, flat, values of a group in a member
    using Exchanged = std::conditional_t<kFlat, float4, float2>;
    auto* exchange = static_cast<Exchanged*>(exchange_words);
    constexpr int kPlanes = Slot<T>::kPlanes;
    extern __shared__ float4 shared[];
    __shared__ int lost;
    const int segments = segments_of(H);
    float4* slots = shared;
    float* means = reinterpret_cast<float*>(slots + H.slots * kPlanes * kThreads); // of the segments
    float* squares = means + segments * kThreads;
    float* sizes = squares + segments * kThreads;
    int* firsts = reinterpret_cast<int*>(sizes + segments * kThreads);
    float* weights = reinterpret_cast<float*>(firsts + kThreads);
    float* biases = weights + H.width;
    float2* group_stats = reinterpret_cast<float2*>(biases + H.width);

    const int team = blockIdx.x / H.members, member = blockIdx.x - team * H.members;
    const int slab = team % H.slabs, step = H.teams / H.slabs;
    const int c0 = slab * H.width;
    const int rg = threadIdx.x / H.lanes, lane = threadIdx.x - rg * H.lanes;
    const int row0 = member * H.slots * H.row_groups;
    float4* mine = slots + threadIdx.x;
    const T* xp = x + (row0 + rg) * H.x_stride + c0 + lane * 8;
    T* yp = y + (row0 + rg) * H.y_stride + c0 + lane * 8;

    if (threadIdx.x == 0) lost = 0;
    int n = team / H.slabs;
    Here next = here_of<kFlat>(H, n < H.samples ? n : 0, x, rg, lane, row0);
    if (n < H.samples)
        for (int k = 0; k < next.rows; ++k)
            fetch_row<kFlat>(H, next, k, mine + k * kPlanes * kThreads, xp - next.lead, H.x_sample, H.x_stride);
    for (int c = threadIdx.x; c < H.width; c += kThreads) {
        float one[1];
        load_param<1>(weight, param_type, c0 + c, 1.0f, one);
        weights[c] = one[0];
        load_param<1>(bias, param_type, c0 + c, 0.0f, one);
        biases[c] = one[0];
    }
    for (int turn = 0; n < H.samples; n += step, ++turn) {
        const Here h = next;
        // ---- sums about the thread's first value of each channel
        {
            float2 shift[4], s[4], q[4];
            const float count = static_cast<float>(h.rows);
#pragma unroll
            for (int i = 0; i < 4; ++i) shift[i] = s[i] = q[i] = make_float2(0.0f, 0.0f);
            copies_here();
            if (h.rows > 0) {
                Slot<T>::read(mine, shift);
                if (kFlat) { // a first vector that is not all the sample's: the row behind it
                    const int a = value_of(H, h, 0), b = value_of(H, h, 1);
                    if (a < 0 || a + 8 > h.total) {
                        float2 v[4] = {};
                        if (h.rows > 1) Slot<T>::read(mine + kPlanes * kThreads, v);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int e = 2 * i;
                            if (a + e < 0 || a + e >= h.total) shift[i].x = h.rows > 1 && b + e < h.total ? v[i].x : 0.0f;
                            if (a + e + 1 < 0 || a + e + 1 >= h.total)
                                shift[i].y = h.rows > 1 && b + e + 1 < h.total ? v[i].y : 0.0f;
                        }
                    }
                }
            }
#pragma unroll 4
            for (int k = 0; k < h.rows; ++k) {
                float2 v[4];
                Slot<T>::read(mine + k * kPlanes * kThreads, v);
                if (kFlat) {
                    const int f = value_of(H, h, k);
                    if (f < 0 || f + 8 > h.total) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int e = f + 2 * i;
                            if (e < 0 || e >= h.total) v[i].x = shift[i].x;
                            if (e + 1 < 0 || e + 1 >= h.total) v[i].y = shift[i].y;
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 d = dev::fma2(shift[i], dev::pair(-1.0f), v[i]);
                    s[i] = dev::add2(s[i], d);
                    q[i] = dev::fma2(d, d, q[i]);
                }
            }
            if (rg < H.row_groups) {
                const float inv = h.rows > 0 ? 1.0f / count : 0.0f;
                float mean[8] = {s[0].x, s[0].y, s[1].x, s[1].y, s[2].x, s[2].y, s[3].x, s[3].y};
                float square[8] = {q[0].x, q[0].y, q[1].x, q[1].y, q[2].x, q[2].y, q[3].x, q[3].y};
                const float from[8] = {shift[0].x, shift[0].y, shift[1].x, shift[1].y,
                                       shift[2].x, shift[2].y, shift[3].x, shift[3].y};
                float size[8];
                GroupWalk<kFlat> at(H, first_channel<kFlat>(H, h, lane));
                const int g = at.g;
                float n0 = 0.0f, n1 = 0.0f, sum0 = 0.0f, sum1 = 0.0f;
                unsigned second = 0; // channels of the second segment
#pragma unroll
                for (int e = 0; e < 8; ++e, at.next(H)) {
                    float of = count, by = inv;
                    if (kFlat && h.rows > 0) { // values before and behind the sample
                        const int a = value_of(H, h, 0), b = value_of(H, h, h.rows - 1);
                        const int out = (a + e < 0 ? 1 : 0) + (b + e >= h.total ? 1 : 0);
                        if (out > 0) {
                            of = fmaxf(count - static_cast<float>(out), 0.0f);
                            by = of > 0.0f ? 1.0f / of : 0.0f;
                        }
                    }
                    const float m = mean[e] * by;
                    square[e] = fmaf(-mean[e], m, square[e]);
                    if (square[e] < 0.0f) square[e] = 0.0f; // NaN stays
                    mean[e] = from[e] + m;
                    size[e] = of;
                    if (at.g != g) {
                        second |= 1u << e;
                        n1 += of;
                        sum1 = fmaf(of, mean[e], sum1);
                    } else {
                        n0 += of;
                        sum0 = fmaf(of, mean[e], sum0);
                    }
                }
                if (segments == 2) {
                    const float m0 = n0 > 0.0f ? sum0 / n0 : 0.0f, m1 = n1 > 0.0f ? sum1 / n1 : 0.0f;
                    float q0 = 0.0f, q1 = 0.0f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const bool two = second & (1u << e);
                        const float d = mean[e] - (two ? m1 : m0);
                        const float add = size[e] > 0.0f ? fmaf(size[e] * d, d, square[e]) : 0.0f;
                        if (two)
                            q1 += add;
                        else
                            q0 += add;
                    }
                    means[threadIdx.x] = m0;
                    squares[threadIdx.x] = q0;
                    sizes[threadIdx.x] = n0;
                    means[kThreads + threadIdx.x] = m1;
                    squares[kThreads + threadIdx.x] = q1;
                    sizes[kThreads + threadIdx.x] = n1;
                    firsts[threadIdx.x] = g;
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        means[e * kThreads + threadIdx.x] = mean[e];
                        squares[e * kThreads + threadIdx.x] = square[e];
                        sizes[e * kThreads + threadIdx.x] = size[e];
                    }
                }
            }
        }
        __syncthreads();
        // ---- groups: their segments joined
        const int len = H.lengths ? max(0, min(H.positions, H.lengths[n])) : H.positions;
        const int gl = lanes_of_group(H), sub = threadIdx.x & (gl - 1);
        const bool alone = H.members == 1;
        Exchanged* to = exchange + (static_cast<int64_t>(team) * 2 + (turn & 1)) * H.members * H.slab_groups;
        for (int g0 = 0; g0 < H.slab_groups; g0 += kThreads / gl) {
            const int g = g0 + threadIdx.x / gl;
            float count = 0.0f, sum = 0.0f, m2 = 0.0f;
            if (g < H.slab_groups)
                over_segments<kFlat>(H, h.lead, firsts, g, sub, gl, [&](int i) {
                    count += sizes[i];
                    sum = fmaf(sizes[i], means[i], sum);
                });
            count = sum_lanes(count, gl);
            sum = sum_lanes(sum, gl);
            const float mean = count > 0.0f ? sum / count : 0.0f;
            if (g < H.slab_groups)
                over_segments<kFlat>(H, h.lead, firsts, g, sub, gl, [&](int i) {
                    const float d = means[i] - mean;
                    m2 += sizes[i] > 0.0f ? fmaf(sizes[i] * d, d, squares[i]) : 0.0f;
                });
            m2 = sum_lanes(m2, gl);
            if (sub == 0 && g < H.slab_groups) {
                if (alone) {
                    const float2 st = make_float2(mean, 1.0f / sqrtf((count > 0.0f ? m2 / count : 0.0f) + eps));
                    group_stats[g] = st;
                    if (stats) stats[static_cast<int64_t>(n) * H.groups + slab * H.slab_groups + g] = st;
                } else {
                    put(to[g * H.members + member], count, mean, m2);
                }
            }
        }
        if (!alone) {
            // The members of a group, about the mean of its first ones (so the squares of the
            // differences are few times those about the mean of all).
            team_barrier(counts + team, static_cast<uint32_t>(H.members) * (turn + 1), &lost);
            constexpr int kAtOnce = 5;
            const int ml = lanes_of_members(H.slab_groups), ms = threadIdx.x & (ml - 1);
            const float per = static_cast<float>(H.per);
            for (int g0 = 0; g0 < H.slab_groups; g0 += kThreads / ml) {
                const int g = g0 + threadIdx.x / ml;
                float count = 0.0f, sum = 0.0f, m2 = 0.0f, shift = 0.0f;
                for (int m0 = 0; m0 < H.members; m0 += kAtOnce * ml) {
                    Exchanged v[kAtOnce];
#pragma unroll
                    for (int i = 0; i < kAtOnce; ++i) {
                        const int m = m0 + i * ml + ms;
                        if (g < H.slab_groups && m < H.members) v[i] = __ldcg(to + g * H.members + m);
                    }
                    auto size_of = [&](int i) { // values of the group that member i of these holds
                        const int m = m0 + i * ml + ms;
                        if (g >= H.slab_groups || m >= H.members) return 0.0f;
                        if constexpr (kFlat) return v[i].z;
                        return per * static_cast<float>(max(0, min(H.slots * H.row_groups, len - m * H.slots * H.row_groups)));
                    };
                    if (m0 == 0) {
                        float a = 0.0f, b = 0.0f;
#pragma unroll
                        for (int i = 0; i < kAtOnce; ++i) {
                            const float of = size_of(i);
                            a += of;
                            b += of > 0.0f ? of * v[i].x : 0.0f;
                        }
                        a = sum_lanes(a, ml);
                        b = sum_lanes(b, ml);
                        shift = a > 0.0f ? b / a : 0.0f;
                    }
#pragma unroll
                    for (int i = 0; i < kAtOnce; ++i) {
                        const float of = size_of(i);
                        if (of > 0.0f) {
                            const float d = v[i].x - shift;
                            count += of;
                            sum = fmaf(of, d, sum);
                            m2 += fmaf(of * d, d, v[i].y);
                        }
                    }
                }
                count = sum_lanes(count, ml);
                sum = sum_lanes(sum, ml);
                m2 = sum_lanes(m2, ml);
                if (ms == 0 && g < H.slab_groups) {
                    const float by = count > 0.0f ? 1.0f / count : 0.0f, d = sum * by;
                    float2 st = make_float2(shift + d, 1.0f / sqrtf(fmaxf(fmaf(-sum, d, m2), 0.0f) * by + eps));
                    if (isnan(m2) || lost) st.x = st.y = __int_as_float(0x7FC00000);
                    group_stats[g] = st;
                    if (stats && member == 0)
                        stats[static_cast<int64_t>(n) * H.groups + slab * H.slab_groups + g] = st;
                }
            }
        }
        __syncthreads();
        // ---- the result, and the next sample's vectors into the places that become free
        const int n2 = n + step;
        const bool more = n2 < H.samples;
        next = here_of<kFlat>(H, more ? n2 : n, x, rg, lane, row0);
        const int rows2 = more ? next.rows : 0;
        float2 minus_mean[4], a[4], b[4];
        if (rg < H.row_groups) {
            float mean[8], aa[8], bb[8];
            GroupWalk<kFlat> at(H, first_channel<kFlat>(H, h, lane));
#pragma unroll
            for (int e = 0; e < 8; ++e, at.next(H)) {
                const float2 st = group_stats[at.g];
                mean[e] = -st.x;
                aa[e] = weights[at.c] * st.y;
                bb[e] = biases[at.c];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                minus_mean[i] = make_float2(mean[2 * i], mean[2 * i + 1]);
                a[i] = make_float2(aa[2 * i], aa[2 * i + 1]);
                b[i] = make_float2(bb[2 * i], bb[2 * i + 1]);
            }
        }
        T* row = yp + h.n * H.y_sample - h.lead;
#pragma unroll 2
        for (int k = 0; k < h.rows; ++k) {
            float2 v[4];
            Slot<T>::read(mine + k * kPlanes * kThreads, v);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = activated2<kAct>(dev::fma2(dev::add2(v[i], minus_mean[i]), a[i], b[i]));
            T* out = row + k * H.row_groups * H.y_stride;
            const int f = kFlat ? value_of(H, h, k) : 0;
            if (!kFlat || (f >= 0 && f + 8 <= h.total)) {
                dev::store8_stream(out, v);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = f + 2 * i;
                    if (e >= 0 && e < h.total) dev::store1(out + 2 * i, v[i].x);
                    if (e + 1 >= 0 && e + 1 < h.total) dev::store1(out + 2 * i + 1, v[i].y);
                }
            }
            if (k < rows2)
                fetch_row<kFlat>(H, next, k, mine + k * kPlanes * kThreads, xp - next.lead, H.x_sample, H.x_stride);
        }
        for (int k = h.rows; k < rows2; ++k)
            fetch_row<kFlat>(H, next, k, mine + k * kPlanes * kThreads, xp - next.lead, H.x_sample, H.x_stride);
    }
}

// The gradient, likewise: x is held as it is and d in fp32, in dy's place, so that
// the activation's slope is formed once.  dx == nullptr: the parameters' sums alone.
template <typename T, int kAct, bool kFlat>
__global__ void __launch_bounds__(kThreads, 2)
held_backward_kernel(const __grid_constant__ Held H, const T* x, const T* dy,
                     const void* __restrict__ weight, const void* __restrict__ bias,
                     int32_t param_type, const float2* __restrict__ stats, T* dx,
                     uint32_t* counts, float2* exchange, float2* __restrict__ block_sums)
{
    constexpr int kPlanes = Slot<T>::kPlanes;
    extern __shared__ float4 shared[];
    __shared__ int lost;
    const int row_values = 8 * H.lanes, entries = H.row_groups * row_values, parts = parts_of(H);
    const int segments = segments_of(H);
    float4* xs = shared;
    float4* ds = xs + H.slots * kPlanes * kThreads; // two planes a row
    // sums of each channel in each row group, by element: over the samples, or (flat) of one
    float* straight = reinterpret_cast<float*>(ds + H.slots * 2 * kThreads);
    float* along = straight + entries;
    float* segment_s = along + entries;
    float* segment_q = segment_s + segments * kThreads;
    int* firsts = reinterpret_cast<int*>(segment_q + segments * kThreads);
    float* weights = reinterpret_cast<float*>(firsts + kThreads);
    float* biases = weights + H.width;
    float2* sums = reinterpret_cast<float2*>(biases + H.width); // of each channel, over the samples
    float2* group_means = sums + H.width;
    float2* group_stats = group_means + H.slab_groups; // of the sample at hand

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int team = blockIdx.x / H.members, member = blockIdx.x - team * H.members;
    const int slab = team % H.slabs, step = H.teams / H.slabs;
    const int c0 = slab * H.width;
    const int rg = threadIdx.x / H.lanes, lane = threadIdx.x - rg * H.lanes;
    const int row0 = member * H.slots * H.row_groups;
    float4* my_x = xs + threadIdx.x;
    float4* my_d = ds + threadIdx.x;
    const T* xp = x + (row0 + rg) * H.x_stride + c0 + lane * 8;
    const T* dp = dy + (row0 + rg) * H.y_stride + c0 + lane * 8;
    auto fetch = [&](const Here& h, int k) {
        fetch_row<kFlat>(H, h, k, my_x + k * kPlanes * kThreads, xp - h.lead, H.x_sample, H.x_stride);
        fetch_row<kFlat>(H, h, k, my_d + k * 2 * kThreads, dp - h.lead, H.y_sample, H.y_stride);
    };

    if (threadIdx.x == 0) lost = 0;
    int n = team / H.slabs;
    Here next = here_of<kFlat>(H, n < H.samples ? n : 0, x, rg, lane, row0);
    if (n < H.samples)
        for (int k = 0; k < next.rows; ++k) fetch(next, k);
    for (int c = threadIdx.x; c < H.width; c += kThreads) {
        float one[1];
        load_param<1>(weight, param_type, c0 + c, 1.0f, one);
        weights[c] = one[0];
        load_param<1>(bias, param_type, c0 + c, 0.0f, one);
        biases[c] = one[0];
        sums[c] = make_float2(0.0f, 0.0f);
    }
    auto fetch_stats = [&](int sample) {
        const float2* of = stats + static_cast<int64_t>(sample) * H.groups + slab * H.slab_groups;
        for (int g = threadIdx.x; g < H.slab_groups; g += kThreads) group_stats[g] = __ldg(of + g);
    };
    // The channels' sums from those by row group and element: each of `parts` threads adds
    // every parts-th row group (and a flat row's positions).
    auto join_channels = [&](int lead) {
        for (int t = threadIdx.x; t < H.width * parts; t += kThreads) {
            const int part = parts > 1 ? t / H.width : 0, c = t - part * H.width;
            const int begin = kFlat ? (c + lead) % row_values : c;
            float s = 0.0f, q = 0.0f;
#pragma unroll 4
            for (int r = part; r < H.row_groups; r += parts) {
                int i = r * row_values + begin;
                for (int j = 0; j < (kFlat ? H.repeats : 1); ++j) {
                    s += straight[i];
                    q += along[i];
                    if (kFlat) {
                        i += H.channels;
                        if (i >= (r + 1) * row_values) i -= row_values;
                    }
                }
            }
            straight[part * row_values + begin] = s;
            along[part * row_values + begin] = q;
        }
        __syncthreads();
        for (int c = threadIdx.x; c < H.width; c += kThreads) {
            const int begin = kFlat ? (c + lead) % row_values : c;
            float2 all = sums[c];
            for (int part = 0; part < parts; ++part) {
                all.x += straight[part * row_values + begin];
                all.y += along[part * row_values + begin];
            }
            sums[c] = all;
        }
    };
    if (n < H.samples) fetch_stats(n);
    __syncthreads();
    int turns = 0;
    for (int turn = 0; n < H.samples; n += step, ++turn, ++turns) {
        const Here h = next;
        float2 minus_mean[4], rstd[4], w[4];
        if (rg < H.row_groups) {
            float2 b[4], s[4], q[4];
            {
                float m[8], r[8], ww[8], bb[8];
                GroupWalk<kFlat> at(H, first_channel<kFlat>(H, h, lane));
#pragma unroll
                for (int e = 0; e < 8; ++e, at.next(H)) {
                    const float2 st = group_stats[at.g];
                    m[e] = -st.x;
                    r[e] = st.y;
                    ww[e] = weights[at.c];
                    bb[e] = biases[at.c];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    minus_mean[i] = make_float2(m[2 * i], m[2 * i + 1]);
                    rstd[i] = make_float2(r[2 * i], r[2 * i + 1]);
                    w[i] = make_float2(ww[2 * i], ww[2 * i + 1]);
                    b[i] = make_float2(bb[2 * i], bb[2 * i + 1]);
                    s[i] = q[i] = make_float2(0.0f, 0.0f);
                }
            }
            copies_here();
#pragma unroll 2
            for (int k = 0; k < h.rows; ++k) {
                float2 v[4], d[4];
                Slot<T>::read(my_x + k * kPlanes * kThreads, v);
                float4* place = my_d + k * 2 * kThreads;
                Slot<T>::read(place, d);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = dev::mul2(dev::add2(v[i], minus_mean[i]), rstd[i]);
                    if (kAct) d[i] = dev::mul2(d[i], slope2<kAct>(dev::fma2(v[i], w[i], b[i])));
                }
                if (kFlat) {
                    const int f = value_of(H, h, k);
                    if (f < 0 || f + 8 > h.total) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int e = f + 2 * i;
                            if (e < 0 || e >= h.total) v[i].x = d[i].x = 0.0f;
                            if (e + 1 < 0 || e + 1 >= h.total) v[i].y = d[i].y = 0.0f;
                        }
                    }
                }
                place[0] = make_float4(d[0].x, d[0].y, d[1].x, d[1].y);
                place[kThreads] = make_float4(d[2].x, d[2].y, d[3].x, d[3].y);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[i] = dev::add2(s[i], d[i]);
                    q[i] = dev::fma2(d[i], v[i], q[i]);
                }
            }
            auto* st = reinterpret_cast<float2*>(straight + rg * row_values + lane * 8);
            auto* al = reinterpret_cast<float2*>(along + rg * row_values + lane * 8);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                st[i] = kFlat || turn == 0 ? s[i] : dev::add2(st[i], s[i]);
                al[i] = kFlat || turn == 0 ? q[i] : dev::add2(al[i], q[i]);
                s[i] = dev::mul2(s[i], w[i]);
                q[i] = dev::mul2(q[i], w[i]);
            }
            const float ss[8] = {s[0].x, s[0].y, s[1].x, s[1].y, s[2].x, s[2].y, s[3].x, s[3].y};
            const float qq[8] = {q[0].x, q[0].y, q[1].x, q[1].y, q[2].x, q[2].y, q[3].x, q[3].y};
            if (segments == 2) {
                GroupWalk<kFlat> at(H, first_channel<kFlat>(H, h, lane));
                const int g = at.g;
                float s0 = 0.0f, s1 = 0.0f, q0 = 0.0f, q1 = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e, at.next(H)) {
                    if (at.g != g) {
                        s1 += ss[e];
                        q1 += qq[e];
                    } else {
                        s0 += ss[e];
                        q0 += qq[e];
                    }
                }
                segment_s[threadIdx.x] = s0;
                segment_q[threadIdx.x] = q0;
                segment_s[kThreads + threadIdx.x] = s1;
                segment_q[kThreads + threadIdx.x] = q1;
                firsts[threadIdx.x] = g;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    segment_s[e * kThreads + threadIdx.x] = ss[e];
                    segment_q[e * kThreads + threadIdx.x] = qq[e];
                }
            }
        }
        __syncthreads();
        if (kFlat) join_channels(h.lead);
        const int n2 = n + step;
        const bool more = n2 < H.samples;
        if (dx) {
            const int gl = lanes_of_group(H), sub = threadIdx.x & (gl - 1);
            const bool alone = H.members == 1;
            const int len = H.lengths ? max(0, min(H.positions, H.lengths[n])) : H.positions;
            const float size = static_cast<float>(len) * static_cast<float>(H.per);
            const float inv = len > 0 ? 1.0f / size : 0.0f;
            float2* to = exchange + (static_cast<int64_t>(team) * 2 + (turn & 1)) * H.members * H.slab_groups;
            for (int g0 = 0; g0 < H.slab_groups; g0 += kThreads / gl) {
                const int g = g0 + threadIdx.x / gl;
                float s = 0.0f, q = 0.0f;
                if (g < H.slab_groups)
                    over_segments<kFlat>(H, h.lead, firsts, g, sub, gl, [&](int i) {
                        s += segment_s[i];
                        q += segment_q[i];
                    });
                s = sum_lanes(s, gl);
                q = sum_lanes(q, gl);
                if (sub == 0 && g < H.slab_groups) {
                    if (alone)
                        group_means[g] = make_float2(s * inv, q * inv);
                    else
                        to[g * H.members + member] = make_float2(s, q);
                }
            }
            if (!alone) {
                team_barrier(counts + team, static_cast<uint32_t>(H.members) * (turn + 1), &lost);
                constexpr int kAtOnce = 5;
                const int ml = lanes_of_members(H.slab_groups), ms = threadIdx.x & (ml - 1);
                for (int g0 = 0; g0 < H.slab_groups; g0 += kThreads / ml) {
                    const int g = g0 + threadIdx.x / ml;
                    float s = 0.0f, q = 0.0f;
                    for (int m0 = 0; m0 < H.members; m0 += kAtOnce * ml) {
                        float2 v[kAtOnce];
#pragma unroll
                        for (int i = 0; i < kAtOnce; ++i) {
                            const int m = m0 + i * ml + ms;
                            v[i] = g < H.slab_groups && m < H.members ? __ldcg(to + g * H.members + m)
                                                                      : make_float2(0.0f, 0.0f);
                        }
#pragma unroll
                        for (int i = 0; i < kAtOnce; ++i) {
                            s += v[i].x;
                            q += v[i].y;
                        }
                    }
                    s = sum_lanes(s, ml);
                    q = sum_lanes(q, ml);
                    if (ms == 0 && g < H.slab_groups)
                        group_means[g] = lost ? make_float2(__int_as_float(0x7FC00000), __int_as_float(0x7FC00000))
                                              : make_float2(s * inv, q * inv);
                }
            }
            __syncthreads();
        }
        next = here_of<kFlat>(H, more ? n2 : n, x, rg, lane, row0);
        const int rows2 = more ? next.rows : 0;
        if (more) fetch_stats(n2);
        if (dx) {
            // rstd (d w - s1 - h s2) = d (rstd w) - rstd s1 - h (rstd s2)
            float2 wr[4], s1[4], s2[4];
            if (rg < H.row_groups) {
                float a[8], b[8];
                GroupWalk<kFlat> at(H, first_channel<kFlat>(H, h, lane));
#pragma unroll
                for (int e = 0; e < 8; ++e, at.next(H)) {
                    const float2 m = group_means[at.g];
                    a[e] = -m.x;
                    b[e] = -m.y;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    wr[i] = dev::mul2(w[i], rstd[i]);
                    s1[i] = dev::mul2(make_float2(a[2 * i], a[2 * i + 1]), rstd[i]);
                    s2[i] = dev::mul2(make_float2(b[2 * i], b[2 * i + 1]), rstd[i]);
                }
            }
            T* row = dx + (row0 + rg) * H.x_stride + c0 + lane * 8 + h.n * H.x_sample - h.lead;
#pragma unroll 2
            for (int k = 0; k < h.rows; ++k) {
                float2 v[4];
                Slot<T>::read(my_x + k * kPlanes * kThreads, v);
                const float4* place = my_d + k * 2 * kThreads;
                const float4 lo = place[0], hi = place[kThreads];
                const float2 d[4] = {make_float2(lo.x, lo.y), make_float2(lo.z, lo.w), make_float2(hi.x, hi.y),
                                     make_float2(hi.z, hi.w)};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = dev::fma2(dev::mul2(dev::add2(v[i], minus_mean[i]), rstd[i]), s2[i],
                                     dev::fma2(d[i], wr[i], s1[i]));
                T* out = row + k * H.row_groups * H.x_stride;
                const int f = kFlat ? value_of(H, h, k) : 0;
                if (!kFlat || (f >= 0 && f + 8 <= h.total)) {
                    dev::store8_stream(out, v);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int e = f + 2 * i;
                        if (e >= 0 && e < h.total) dev::store1(out + 2 * i, v[i].x);
                        if (e + 1 >= 0 && e + 1 < h.total) dev::store1(out + 2 * i + 1, v[i].y);
                    }
                }
                if (k < rows2) fetch(next, k);
            }
            for (int k = h.rows; k < rows2; ++k) fetch(next, k);
        } else {
            for (int k = 0; k < rows2; ++k) fetch(next, k);
        }
        __syncthreads();
    }
    copies_here();
    __syncthreads();
    if (!kFlat && turns > 0) join_channels(0);
    for (int c = threadIdx.x; c < H.width; c += kThreads) // each by the thread that summed it
        block_sums[static_cast<int64_t>(blockIdx.x) * H.width + c] = sums[c];
}

// dweight and dbias of 32 channels: the blocks' sums of their slab.
__global__ void __launch_bounds__(kThreads)
block_sums_kernel(const __grid_constant__ Held H, const float2* __restrict__ block_sums,
                  void* dweight, void* dbias, int32_t grad_type)
{
    __shared__ float2 slices[kWarps][32];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    // launched while the blocks of the kernel before drain
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float s = 0.0f, q = 0.0f;
    if (c < H.channels) {
        const int slab = c / H.width, blocks = H.teams / H.slabs * H.members;
        const float2* from = block_sums + c - slab * H.width;
#pragma unroll 8
        for (int j = slice; j < blocks; j += kWarps) {
            const int team = j / H.members * H.slabs + slab;
            const float2 v = from[(static_cast<int64_t>(team) * H.members + j % H.members) * H.width];
            s += v.x;
            q += v.y;
        }
    }
    slices[slice][lane] = make_float2(s, q);
    __syncthreads();
    if (slice == 0 && c < H.channels) {
        float a[1] = {0.0f}, b[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            a[0] += slices[k][lane].x;
            b[0] += slices[k][lane].y;
        }
        if (dbias) dev::store_any<1>(dbias, grad_type, c, a);
        if (dweight) dev::store_any<1>(dweight, grad_type, c, b);
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

int64_t held_scratch_bytes(int64_t channels, int64_t groups);

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
    const int64_t held = held_scratch_bytes(channels, groups);
    if (s.bytes < held) s.bytes = held;
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

// ---- samples held in shared memory
constexpr int kHeldResident = 152 * 2; // two blocks an SM
constexpr int64_t kHeldShared = 113 * 1024;

struct Plan {
    Held H;
    int64_t grid, shared;
};

// What a block needs beside its slots, in bytes.
int64_t held_tables(const Held& H, bool flat, bool backward)
{
    const int64_t entries = static_cast<int64_t>(H.row_groups) * 8 * H.lanes;
    return (backward ? 8 * entries : 0) + 4 * kThreads * (segments_of(H) * (backward ? 2 : 3) + 1) +
           8 * static_cast<int64_t>(H.width) * (backward ? 2 : 1) +
           8 * static_cast<int64_t>(H.slab_groups) * (backward ? 2 : 1);
}
int64_t slot_bytes(int32_t type, bool backward)
{
    return kThreads * 16 * (type == ZERO_TYPE_F32 ? (backward ? 4 : 2) : (backward ? 3 : 1));
}

// What a call costs where `teams` teams take all slabs of all samples in turn, in rows that a
// block streams: every turn takes about kTurn of them for its sums, its exchange and its wait.
constexpr int64_t kTurn = 8;
int64_t held_cost(const Held& H, int64_t rows, int64_t teams)
{
    const int64_t of_slab = teams / H.slabs, members = kHeldResident / teams;
    return ((H.samples + of_slab - 1) / of_slab) * ((rows + members * H.row_groups - 1) / (members * H.row_groups) + kTurn);
}

// Whether and how a call runs with its samples held: by its sizes, its type and whether
// 16-byte accesses are possible at every position (!flat) or along a sample (flat).
// A slab for one block where there is one that fits and is not narrower than 64 bytes (the
// widest that leaves every resident block one, or else the narrowest: few samples then
// spread over more blocks); else the narrowest of 128 bytes or more that the resident
// blocks can hold: the smaller a team, the sooner its members have exchanged their sums.
bool make_plan(const zero_group_norm_t* n, const int32_t* lengths, bool flat, bool backward, Plan* plan)
{
    if (n->positions * n->channels >= (int64_t(1) << 30)) return false;
    Held H = {};
    H.lengths = lengths;
    H.samples = static_cast<int32_t>(n->samples);
    H.positions = static_cast<int32_t>(n->positions);
    H.channels = static_cast<int32_t>(n->channels);
    H.groups = n->groups;
    H.per = H.channels / H.groups;
    H.repeats = 1;
    if (flat)
        while (H.repeats * H.channels % 8 != 0) ++H.repeats;
    auto with = [&](int slab_groups) {
        Held c = H;
        c.slab_groups = slab_groups;
        c.slabs = H.groups / slab_groups;
        c.width = slab_groups * H.per;
        c.lanes = H.repeats * c.width / 8;
        c.row_groups = kThreads / c.lanes;
        return c;
    };
    auto capacity = [&](const Held& c) {
        return (kHeldShared - held_tables(c, flat, backward)) / slot_bytes(n->type, backward);
    };
    auto rows_of = [&](const Held& c) { // of a sample, flat ones with a lead
        return flat ? (static_cast<int64_t>(c.positions) * c.channels + 7 + 8 * c.lanes - 1) / (8 * c.lanes)
                    : static_cast<int64_t>(c.positions);
    };
    auto possible = [&](int slab_groups) {
        if (H.groups % slab_groups != 0) return false;
        const int64_t width = static_cast<int64_t>(slab_groups) * H.per;
        return flat ? slab_groups == H.groups && H.repeats * width <= kHeldWidth
                    : width % 8 == 0 && width <= kHeldWidth;
    };
    const int bytes = type_bytes(n->type);
    Held one = {}, many = {};
    for (int g = 1; g <= H.groups && g * H.per <= kHeldWidth; ++g) {
        if (!possible(g)) continue;
        const Held c = with(g);
        if (c.slabs > kHeldResident) continue;
        const int64_t cap = capacity(c);
        if (cap < 1) continue;
        const int64_t rows = rows_of(c);
        if (rows <= cap * c.row_groups) {
            if ((c.width * bytes >= 64 || g == H.groups) &&
                (one.width == 0 || static_cast<int64_t>(c.samples) * c.slabs >= kHeldResident))
                one = c;
        } else if (rows <= cap * c.row_groups * (kHeldResident / c.slabs) &&
                   (many.width == 0 || many.width * bytes < 128)) {
            many = c;
        }
    }
    int64_t teams;
    if (one.width > 0) {
        H = one;
        H.members = 1;
        const int64_t rows = rows_of(H);
        H.slots = static_cast<int32_t>(rows < 1 ? 1 : (rows + H.row_groups - 1) / H.row_groups);
        teams = kHeldResident / H.slabs * H.slabs;
        if (teams > static_cast<int64_t>(H.samples) * H.slabs) teams = static_cast<int64_t>(H.samples) * H.slabs;
    } else if (many.width > 0) {
        H = many;
        const int64_t rows = rows_of(H), cap = capacity(H);
        const int64_t least = (rows + cap * H.row_groups - 1) / (cap * H.row_groups); // members
        teams = H.slabs;
        for (int64_t t = 2 * H.slabs; t * least <= kHeldResident; t += H.slabs)
            if (held_cost(H, rows, t) <= held_cost(H, rows, teams)) teams = t;
        const int64_t members = kHeldResident / teams;
        H.slots = static_cast<int32_t>((rows + members * H.row_groups - 1) / (members * H.row_groups));
        H.members = static_cast<int32_t>((rows + static_cast<int64_t>(H.slots) * H.row_groups - 1) /
                                         (static_cast<int64_t>(H.slots) * H.row_groups));
    } else {
        return false;
    }
    H.teams = static_cast<int32_t>(teams);
    H.x_sample = flat ? n->positions * n->channels : n->positions * n->x_stride;
    H.y_sample = flat ? n->positions * n->channels : n->positions * n->y_stride;
    H.x_stride = flat ? 8 * H.lanes : n->x_stride;
    H.y_stride = flat ? 8 * H.lanes : n->y_stride;
    plan->H = H;
    plan->grid = teams * H.members;
    plan->shared = held_tables(H, flat, backward) + slot_bytes(n->type, backward) * H.slots;
    return true;
}

// Scratch of the held kernels: counts, exchange, blocks' sums; for any plan of these sizes.
struct HeldScratch {
    uint32_t* counts;
    void* exchange;
    float2* block_sums;
    int64_t bytes;
};
HeldScratch held_scratch(void* base, int64_t channels, int64_t groups)
{
    HeldScratch s;
    auto* at = static_cast<char*>(base);
    s.counts = reinterpret_cast<uint32_t*>(at);
    at += kHeldResident * 4 / 16 * 16 + 16;
    s.exchange = at;
    at += int64_t(kHeldResident) * 2 * 16 * (groups < kHeldWidth ? groups : kHeldWidth);
    s.block_sums = reinterpret_cast<float2*>(at);
    at += int64_t(kHeldResident) * 8 * (channels < kHeldWidth ? channels : kHeldWidth);
    s.bytes = at - static_cast<char*>(base);
    return s;
}

int64_t held_scratch_bytes(int64_t channels, int64_t groups)
{
    return held_scratch(nullptr, channels, groups).bytes;
}

// Launches a held kernel: cooperatively where its blocks wait for one another.
template <typename... Params, typename... Given>
int launch_held(void (*kernel)(Held, Params...), const Plan& plan, uint32_t* counts, cudaStream_t stream,
                Given... given)
{
    if (!allow_shared(reinterpret_cast<const void*>(kernel), kHeldShared)) return ZERO_ECUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(plan.grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(plan.shared);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeCooperative;
    attr.val.cooperative = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = plan.H.members > 1 ? 1 : 0;
    if (plan.H.members > 1) {
        const int rc = cuda_status(cudaMemsetAsync(counts, 0, static_cast<size_t>(plan.H.teams) * 4, stream));
        if (rc != ZERO_OK) return rc;
    }
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, plan.H, static_cast<Params>(given)...));
}

struct Call {
    const zero_group_norm_t* norm;
    Geometry G;
    Scratch s;
    HeldScratch hs;
    Plan plan;
    bool held, flat;
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


template <typename T, int kAct>
int held_forward(const Call& c, float2* stats)
{
    auto* kernel = c.flat ? held_forward_kernel<T, kAct, true> : held_forward_kernel<T, kAct, false>;
    return launch_held(kernel, c.plan, c.hs.counts, c.stream, static_cast<const T*>(c.x), c.weight, c.bias,
                       c.norm->param_type, static_cast<float>(c.norm->eps), static_cast<T*>(c.y), stats,
                       c.hs.counts, c.hs.exchange);
}

template <typename T, int kAct>
int held_backward(const Call& c)
{
    auto* kernel = c.flat ? held_backward_kernel<T, kAct, true> : held_backward_kernel<T, kAct, false>;
    const int rc = launch_held(kernel, c.plan, c.hs.counts, c.stream, static_cast<const T*>(c.x),
                               static_cast<const T*>(c.dy), c.weight, c.bias, c.norm->param_type, c.stats,
                               static_cast<T*>(c.dx), c.hs.counts, static_cast<float2*>(c.hs.exchange),
                               c.hs.block_sums);
    if (rc != ZERO_OK || (!c.dweight && !c.dbias)) return rc;
    return launch(true, block_sums_kernel, (c.norm->channels + 31) / 32, c.stream, c.plan.H,
                  c.hs.block_sums, c.dweight, c.dbias, c.norm->grad_type);
}

template <typename T>
int held_forward_by_act(const Call& c, float2* stats)
{
    switch (c.norm->act) {
    case ZERO_ACT_SILU: return held_forward<T, ZERO_ACT_SILU>(c, stats);
    case ZERO_ACT_GELU: return held_forward<T, ZERO_ACT_GELU>(c, stats);
    default: return held_forward<T, ZERO_ACT_NONE>(c, stats);
    }
}

template <typename T>
int held_backward_by_act(const Call& c)
{
    switch (c.norm->act) {
    case ZERO_ACT_SILU: return held_backward<T, ZERO_ACT_SILU>(c);
    case ZERO_ACT_GELU: return held_backward<T, ZERO_ACT_GELU>(c);
    default: return held_backward<T, ZERO_ACT_NONE>(c);
    }
}

bool same_lead(const void* a, const void* b)
{
    return ((reinterpret_cast<uintptr_t>(a) ^ reinterpret_cast<uintptr_t>(b)) & 15u) == 0;
}

// Whether the samples are held, and how; `aligned` and `same_lead`: all row tensors start at
// multiples of 16 bytes, or equally far behind.
void choose(Call& c, const int32_t* lengths, bool aligned, bool same_lead, bool backward)
{
    const zero_group_norm_t* n = c.norm;
    const int unit = 16 / type_bytes(n->type);
    const bool rows = aligned && n->channels % 8 == 0 && n->x_stride % unit == 0 && n->y_stride % unit == 0;
    c.flat = !rows;
    c.held = (rows || (same_lead && n->x_stride == n->channels && n->y_stride == n->channels)) &&
             make_plan(n, lengths, c.flat, backward, &c.plan);
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
    c.hs = held_scratch(scratch, norm->channels, norm->groups);
    choose(c, lengths, aligned16(x) && aligned16(y), same_lead(x, y), false);
    if (c.held && norm->positions > 0) {
        auto* st = reinterpret_cast<float2*>(stats);
        return norm->type == ZERO_TYPE_BF16 ? held_forward_by_act<Bf16>(c, st) : held_forward_by_act<float>(c, st);
    }
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
    c.hs = held_scratch(scratch, norm->channels, norm->groups);
    choose(c, lengths, aligned16(x) && aligned16(dy) && aligned16(dx),
           same_lead(x, dy) && (!dx || same_lead(x, dx)), true);
    if (c.held && norm->samples > 0 && norm->positions > 0)
        return norm->type == ZERO_TYPE_BF16 ? held_backward_by_act<Bf16>(c) : held_backward_by_act<float>(c);
    if (norm->type == ZERO_TYPE_BF16)
        return c.G.vec == 8 ? backward_by_act<8, Bf16>(c) : backward_by_act<1, Bf16>(c);
    return c.G.vec == 8 ? backward_by_act<8, float>(c) : backward_by_act<1, float>(c);
}

// group_norm.cuh -- what the kernels of the group norm share: the activations, where a
// thread's rows lie, and the sums of groups.
//
// A block takes one slab (whole groups, at most 8 * kThreads channels) of a run of a
// sample's rows; a thread one vector of 8 channels of every row_groups-th row, `slots` of
// them at most.  Rows are positions (x_stride apart) where 16-byte accesses are possible at
// every position.  Else, where the channels are contiguous, they are runs of `repeats`
// positions that fill whole vectors (flat): the sample is taken as one line of values that
// starts `lead` elements behind a 16-byte boundary; element e of vector l of a row is value
// 8 l + e - lead of it, of channel (8 l + e - lead) mod channels.
//
// Statistics: a thread sums each channel's differences from its own first value, and their
// squares: with at most 64 rows those are at most 2 + 2 * 64 times the squares about the
// mean even where that first value is an outlier, so fp32 keeps the variance.  Threads and
// blocks are joined by means and sums of squares about them.
#pragma once

#include <cstdint>
#include <type_traits>

#include "typed.cuh"
#include "zero_internal.h"

namespace zero {
namespace gn {

using dev::Bf16;
using dev::Raw8;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kWidth = 8 * kThreads; // channels of a slab, at most

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
// The normal distribution's density and cumulative probability, from one exponential.  bf16
// tensors: Abramowitz and Stegun, 26.2.17 (absolute error below 7.5e-8).  fp32 ones, whose own
// rounding is no larger than that: for z < 0 the probability is exp(-z^2 / 2) t Q(t) with t = 1 / (1 +
// 0.34 |z|) and Q of degree 8, fitted here for the least relative error over |z| < 14 (Remez' exchange;
// 3.0e-8, 3.1e-7 with its fp32 roundings), for z > 0 the rest to 1.  32 x 4096 x 640 fp32 takes 190 us, its
// gradient 307; by erfcf 228 and 445; by erff, which loses the digits of small probabilities, 194 and
// 350.
template <typename T>
__device__ __forceinline__ void normal(float z, float& density, float& cdf)
{
    // Single operations: they take constants as they stand, pairs need them in registers.
    float p, t, tail;
    if constexpr (std::is_same_v<T, float>) {
        const float e = expf(-0.5f * z * z);
        t = reciprocal_fast(fmaf(fabsf(z), 0.34f, 1.0f));
        density = e * 0.39894228f;
        p = fmaf(t, -0.0261207484f, 0.139500543f);
        p = fmaf(p, t, -0.273134351f);
        p = fmaf(p, t, 0.202183843f);
        p = fmaf(p, t, -0.0447188057f);
        p = fmaf(p, t, 0.115359128f);
        p = fmaf(p, t, 0.115197711f);
        p = fmaf(p, t, 0.136112183f);
        p = fmaf(p, t, 0.135620505f) * t;
        tail = p * e;
    } else {
        t = reciprocal_fast(fmaf(fabsf(z), 0.2316419f, 1.0f));
        density = exp2_fast(z * z * (-0.5f * kLog2e)) * 0.39894228f;
        p = fmaf(t, 1.330274429f, -1.821255978f);
        p = fmaf(p, t, 1.781477937f);
        p = fmaf(p, t, -0.356563782f);
        p = fmaf(p, t, 0.319381530f) * t;
        tail = p * density;
    }
    cdf = z > 0.0f ? 1.0f - tail : tail;
}

template <typename T, int kAct>
__device__ __forceinline__ float2 activated2(float2 z)
{
    if constexpr (kAct == ZERO_ACT_SILU) return dev::mul2(z, sigmoid2(z));
    if constexpr (kAct == ZERO_ACT_GELU) {
        float density, a, b;
        normal<T>(z.x, density, a);
        normal<T>(z.y, density, b);
        return dev::mul2(z, make_float2(a, b));
    }
    return z;
}
template <typename T, int kAct>
__device__ __forceinline__ float2 slope2(float2 z)
{
    if constexpr (kAct == ZERO_ACT_SILU) {
        const float2 p = sigmoid2(z);
        return dev::mul2(p, dev::fma2(z, dev::fma2(p, dev::pair(-1.0f), dev::pair(1.0f)), dev::pair(1.0f)));
    }
    if constexpr (kAct == ZERO_ACT_GELU) {
        float2 density, cdf;
        normal<T>(z.x, density.x, cdf.x);
        normal<T>(z.y, density.y, cdf.y);
        return dev::fma2(z, density, cdf);
    }
    return dev::pair(1.0f);
}
template <typename T, int kAct>
__device__ __forceinline__ float activated(float z)
{
    return activated2<T, kAct>(dev::pair(z)).x;
}
template <typename T, int kAct>
__device__ __forceinline__ float slope(float z)
{
    return slope2<T, kAct>(dev::pair(z)).x;
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


// ------------------------------------------------------------------- layout
struct Layout {
    int64_t x_stride, y_stride; // elements between rows
    int64_t x_sample, y_sample; // and between samples
    const int32_t* lengths;
    int32_t samples, positions, channels;
    int32_t groups, per;                // groups and their channels; where a group is wider than a
    int32_t splits;                     // slab, its `splits` equal parts in their place
    int32_t slab_groups, slabs, width;  // groups and channels of a slab
    int32_t lanes, row_groups, repeats; // vectors of a row, rows at once, positions of a row
    int32_t slots, chunks;              // rows of a thread; runs of rows of a sample
};

// Where a thread stands in the rows that its block works on.
struct Here {
    int n;     // the sample
    int rows;  // the thread's rows
    int total; // flat: values of the sample
    int lead;  // flat: elements that its first vector starts before it
    int first; // flat: the value of element 0 of the thread's first vector
};

__device__ __forceinline__ int length_of(const Layout& H, int n)
{
    return H.lengths ? max(0, min(H.positions, H.lengths[n])) : H.positions;
}

// row0: the block's first row.  x gives the lead.
template <bool kFlat, typename T>
__device__ __forceinline__ Here here_of(const Layout& H, int n, const T* x, int rg, int lane, int row0)
{
    Here h;
    h.n = n;
    int all = length_of(H, n);
    h.total = h.lead = h.first = 0;
    if (kFlat) {
        const int64_t at = static_cast<int64_t>(reinterpret_cast<uintptr_t>(x) / sizeof(T)) + n * H.x_sample;
        h.lead = static_cast<int>(at & (16 / static_cast<int>(sizeof(T)) - 1));
        h.total = all * H.channels;
        const int row = 8 * H.lanes;
        all = all > 0 ? (h.total + h.lead + row - 1) / row : 0;
        h.first = (row0 + rg) * row + lane * 8 - h.lead;
    }
    const int left = all - row0 - rg;
    h.rows = rg < H.row_groups && left > 0 ? min((left + H.row_groups - 1) / H.row_groups, H.slots) : 0;
    return h;
}

// The first value of the thread's row k, flat.
__device__ __forceinline__ int value_of(const Layout& H, const Here& h, int k)
{
    return h.first + k * H.row_groups * 8 * H.lanes;
}
// Whether all of that row's vector is the sample's.
template <bool kFlat>
__device__ __forceinline__ bool whole(const Layout& H, const Here& h, int k)
{
    return !kFlat || (value_of(H, h, k) >= 0 && value_of(H, h, k) + 8 <= h.total);
}

// The groups of 8 neighbouring channels from c on (flat: around the end).
template <bool kFlat>
struct GroupWalk {
    int c, g, left;
    __device__ __forceinline__ GroupWalk(const Layout& H, const Here& h, int lane)
    {
        c = kFlat ? (lane * 8 + 8 * H.lanes - h.lead) % H.channels : lane * 8;
        g = c / H.per;
        left = (g + 1) * H.per - c;
    }
    __device__ __forceinline__ void next(const Layout& H)
    {
        ++c;
        if (--left == 0) {
            ++g;
            left = H.per;
            if (kFlat && c == H.channels) c = g = 0;
        }
    }
};

// A vector that this call reads once more, or not again.
template <bool kStream, typename T>
__device__ __forceinline__ void load_vector(const T* p, Raw8<T>& r)
{
    if constexpr (kStream)
        dev::stream_raw8(p, r);
    else
        dev::load_raw8(p, r);
}
__device__ __forceinline__ void set_element(Raw8<Bf16>& r, int e, Bf16 x)
{
    uint32_t* w = &r.a.x; // unrolled: known at compile time
    w[e / 2] = e % 2 ? (w[e / 2] & 0xFFFFu) | static_cast<uint32_t>(x.bits) << 16 : (w[e / 2] & 0xFFFF0000u) | x.bits;
}
__device__ __forceinline__ void set_element(Raw8<float>& r, int e, float x)
{
    (e < 4 ? &r.a.x : &r.b.x)[e & 3] = x;
}

// The thread's row k of a tensor; `base` is where its first row's vector would start in the
// first sample without a lead.  Elements outside the tensor are not read (any value).
template <bool kFlat, bool kStream, typename T>
__device__ __forceinline__ void load_row(const Layout& H, const Here& h, int k, const T* base, int64_t sample,
                                         int64_t stride, Raw8<T>& r)
{
    const T* from = base + h.n * sample + k * H.row_groups * stride - (kFlat ? h.lead : 0);
    if (kFlat && !whole<kFlat>(H, h, k)) {
        const int64_t at = h.n * sample + value_of(H, h, k), behind = H.samples * sample - at;
        if (at < 0 || behind < 8) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (at + e >= 0 && e < behind) set_element(r, e, from[e]);
            return;
        }
    }
    load_vector<kStream>(from, r);
}

template <bool kFlat, typename T>
__device__ __forceinline__ void store_row(const Layout& H, const Here& h, int k, T* base, int64_t sample,
                                          int64_t stride, const float2 (&v)[4])
{
    T* to = base + h.n * sample + k * H.row_groups * stride - (kFlat ? h.lead : 0);
    if (whole<kFlat>(H, h, k)) {
        dev::store8_stream(to, v);
    } else {
        const int f = value_of(H, h, k);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = f + 2 * i;
            if (e >= 0 && e < h.total) dev::store1(to + 2 * i, v[i].x);
            if (e + 1 >= 0 && e + 1 < h.total) dev::store1(to + 2 * i + 1, v[i].y);
        }
    }
}

// Elements of row k that are not the sample's.
template <typename F>
__device__ __forceinline__ void outside(const Layout& H, const Here& h, int k, F f)
{
    const int at = value_of(H, h, k);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (at + e < 0 || at + e >= h.total) f(e);
}
__device__ __forceinline__ float& of_pair(float2 (&v)[4], int e) { return e % 2 ? v[e / 2].y : v[e / 2].x; }

// ------------------------------------------------------------ sums of groups
__device__ __forceinline__ float sum_lanes(float x, int lanes) // 8 or 32
{
    if (lanes == 32) {
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 16);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 8);
    }
    x += __shfl_xor_sync(0xFFFFFFFFu, x, 4);
    x += __shfl_xor_sync(0xFFFFFFFFu, x, 2);
    return x + __shfl_xor_sync(0xFFFFFFFFu, x, 1);
}
// Lanes that share a group's segments: a whole warp for many.
__device__ __forceinline__ int lanes_of_group(const Layout& H)
{
    return max(H.row_groups, (H.per + 7) / 8) >= 24 ? 32 : 8;
}

// Sums of a thread's 8 channels go by segments: of each of the (at most two) groups that
// the vector lies in where a group has 8 channels or more, else of each channel.
__host__ __device__ __forceinline__ int segments_of(const Layout& H) { return H.per >= 8 ? 2 : 8; }

// Calls f(entry) for this lane's share of the segments of group g, an entry being segment *
// kThreads + thread; `firsts` holds the group of each thread's first channel.  Lanes go
// over whichever is more, vectors or row groups.
template <bool kFlat, typename F>
__device__ __forceinline__ void over_segments(const Layout& H, int lead, const int* firsts, int g, int sub, int gl, F f)
{
    if (H.per >= 8) {
        const bool all = kFlat && H.groups == 1; // rows of one group: all vectors, once
        for (int j = 0; j < (kFlat && !all ? H.repeats : 1); ++j) {
            int p = g * H.per, nv = H.lanes;
            if (kFlat) {
                p = all ? 0 : p + j * H.channels + lead;
                if (p >= 8 * H.lanes) p -= 8 * H.lanes;
            }
            const int v0 = p >> 3;
            if (!all) nv = ((p & 7) + H.per + 7) >> 3;
            if (nv >= H.row_groups) {
                for (int b = sub; b < nv; b += gl) {
                    int v = v0 + b;
                    if (kFlat && v >= H.lanes) v -= H.lanes;
                    const int i = all || firsts[v] == g ? v : kThreads + v;
#pragma unroll 2
                    for (int r = 0; r < H.row_groups; ++r) f(i + r * H.lanes);
                }
            } else {
                for (int b = 0; b < nv; ++b) {
                    int v = v0 + b;
                    if (kFlat && v >= H.lanes) v -= H.lanes;
                    const int i = all || firsts[v] == g ? v : kThreads + v;
#pragma unroll 2
                    for (int r = sub; r < H.row_groups; r += gl) f(i + r * H.lanes);
                }
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
#pragma unroll 2
                for (int r = sub; r < H.row_groups; r += gl) f((p & 7) * kThreads + r * H.lanes + (p >> 3));
            }
    }
}

// Mean of `count` parts of `size` values each and the squares about it, from the squares about a
// value `near` it and from rest, the sum of the parts' means less `near`.  A sum of the means
// themselves would round by 2^-24 of the mean at every step, and the same way where they are
// alike; these differences leave nothing large to round.  (Parts of unequal sizes: their
// differences weighted, count the values of all, size 1.)
__device__ __forceinline__ float2 corrected(float near, float squares, float rest, float by, float size)
{
    const float d = rest * by;
    const float m2 = fmaf(-size * rest, d, squares);
    return make_float2(near + d, m2 < 0.0f ? 0.0f : m2); // NaN stays
}

// In shared memory: words [segments][kThreads] each, and the groups of first channels.
struct Segments {
    float *a, *b, *c;
    int* firsts;
};
// Words that Segments take, with two or three kinds of sums.
__host__ __device__ __forceinline__ int segment_words(const Layout& H, int kinds)
{
    return kThreads * (kinds * segments_of(H) + 1);
}
__device__ __forceinline__ Segments segments_at(const Layout& H, int kinds, float* at)
{
    const int n = segments_of(H) * kThreads;
    return {at, at + n, at + 2 * n, reinterpret_cast<int*>(at + kinds * n)};
}

// A thread's rows of x: the sums of its channels about their first values, as means (a), sums
// of squares about them (b) and sizes (c) of its segments.  fetch(k, raw) loads row k.
template <bool kFlat, int kAhead, typename T, typename Fetch>
__device__ __forceinline__ void sum_rows(const Layout& H, const Here& h, int rg, int lane, const Segments& S, Fetch fetch)
{
    float2 shift[4], s[4], q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) shift[i] = s[i] = q[i] = make_float2(0.0f, 0.0f);
    auto add = [&](int k, const Raw8<T>& raw) {
        float2 v[4];
        dev::unpack8(raw, v);
        if (kFlat && !whole<kFlat>(H, h, k)) outside(H, h, k, [&](int e) { of_pair(v, e) = of_pair(shift, e); });
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 d = dev::fma2(shift[j], dev::pair(-1.0f), v[j]);
            s[j] = dev::add2(s[j], d);
            q[j] = dev::fma2(d, d, q[j]);
        }
    };
    int k = 0;
    if (h.rows > 0) {
        Raw8<T> raw;
        fetch(0, raw);
        dev::unpack8(raw, shift);
        if (kFlat && !whole<kFlat>(H, h, 0)) { // in the place of what is not the sample's: the next row's
            float2 next[4] = {};
            if (h.rows > 1) {
                Raw8<T> second = {};
                fetch(1, second);
                dev::unpack8(second, next);
            }
            const int b = value_of(H, h, 1);
            outside(H, h, 0, [&](int e) { of_pair(shift, e) = h.rows > 1 && b + e < h.total ? of_pair(next, e) : 0.0f; });
        }
    }
    for (; k + kAhead <= h.rows; k += kAhead) {
        Raw8<T> raw[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fetch(k + i, raw[i]);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) add(k + i, raw[i]);
    }
    for (; k < h.rows; ++k) {
        Raw8<T> raw;
        fetch(k, raw);
        add(k, raw);
    }
    if (rg >= H.row_groups) return;
    const float count = static_cast<float>(h.rows), inv = h.rows > 0 ? 1.0f / count : 0.0f;
    float size[8];
    GroupWalk<kFlat> at(H, h, lane);
    const int g = at.g;
    float n0 = 0.0f, n1 = 0.0f, sum0 = 0.0f, sum1 = 0.0f;
    unsigned second = 0; // channels of the second segment
#pragma unroll
    for (int e = 0; e < 8; ++e, at.next(H)) {
        float of = count, by = inv;
        if (kFlat && h.rows > 0) { // values before and behind the sample
            const int out = (value_of(H, h, 0) + e < 0 ? 1 : 0) + (value_of(H, h, h.rows - 1) + e >= h.total ? 1 : 0);
            if (out > 0) {
                of = fmaxf(count - static_cast<float>(out), 0.0f);
                by = of > 0.0f ? 1.0f / of : 0.0f;
            }
        }
        float &mean = of_pair(s, e), &square = of_pair(q, e);
        const float m = mean * by;
        square = fmaf(-mean, m, square);
        if (square < 0.0f) square = 0.0f; // NaN stays
        mean = of_pair(shift, e) + m;
        size[e] = of;
        if (at.g != g) {
            second |= 1u << e;
            n1 += of;
            sum1 = fmaf(of, mean, sum1);
        } else {
            n0 += of;
            sum0 = fmaf(of, mean, sum0);
        }
    }
    const int t = threadIdx.x;
    if (H.per < 8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            S.a[e * kThreads + t] = of_pair(s, e);
            S.b[e * kThreads + t] = of_pair(q, e);
            S.c[e * kThreads + t] = size[e];
        }
        return;
    }
    const float by0 = n0 > 0.0f ? 1.0f / n0 : 0.0f, by1 = n1 > 0.0f ? 1.0f / n1 : 0.0f;
    const float m0 = sum0 * by0, m1 = sum1 * by1;
    float q0 = 0.0f, q1 = 0.0f, rest0 = 0.0f, rest1 = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const bool two = second & (1u << e);
        const float d = of_pair(s, e) - (two ? m1 : m0), sized = size[e] * d;
        const float add = size[e] > 0.0f ? fmaf(sized, d, of_pair(q, e)) : 0.0f;
        if (two)
            q1 += add, rest1 += sized;
        else
            q0 += add, rest0 += sized;
    }
    const float2 one = corrected(m0, q0, rest0, by0, 1.0f), other = corrected(m1, q1, rest1, by1, 1.0f);
    S.a[t] = one.x, S.b[t] = one.y, S.c[t] = n0;
    S.a[kThreads + t] = other.x, S.b[kThreads + t] = other.y, S.c[kThreads + t] = n1;
    S.firsts[t] = g;
}

// After a barrier: done(g, size, mean, squares about it) for each of the slab's groups, by one
// thread.
template <bool kFlat, typename Done>
__device__ __forceinline__ void join_groups(const Layout& H, int lead, const Segments& S, Done done)
{
    const int gl = lanes_of_group(H), sub = threadIdx.x & (gl - 1);
    for (int g0 = 0; g0 < H.slab_groups; g0 += kThreads / gl) {
        const int g = g0 + threadIdx.x / gl;
        float count = 0.0f, sum = 0.0f, m2 = 0.0f;
        if (g < H.slab_groups)
            over_segments<kFlat>(H, lead, S.firsts, g, sub, gl, [&](int i) {
                count += S.c[i];
                sum = fmaf(S.c[i], S.a[i], sum);
            });
        count = sum_lanes(count, gl);
        sum = sum_lanes(sum, gl);
        const float by = count > 0.0f ? 1.0f / count : 0.0f, near = sum * by;
        float rest = 0.0f;
        if (g < H.slab_groups)
            over_segments<kFlat>(H, lead, S.firsts, g, sub, gl, [&](int i) {
                const float d = S.a[i] - near, sized = S.c[i] * d;
                rest += sized;
                m2 += S.c[i] > 0.0f ? fmaf(sized, d, S.b[i]) : 0.0f;
            });
        m2 = sum_lanes(m2, gl);
        rest = sum_lanes(rest, gl);
        if (sub == 0 && g < H.slab_groups) {
            const float2 all = corrected(near, m2, rest, by, 1.0f);
            done(g, count, all.x, all.y);
        }
    }
}

// A thread's factors of its 8 channels, from a slab's weights and biases and the groups'
// statistics (mean, rstd).
template <bool kFlat>
__device__ __forceinline__ void forward_factors(const Layout& H, const Here& h, int lane, const float* weights,
                                                const float* biases, const float2* stats, float2 (&minus_mean)[4],
                                                float2 (&a)[4], float2 (&b)[4])
{
    GroupWalk<kFlat> at(H, h, lane);
#pragma unroll
    for (int e = 0; e < 8; ++e, at.next(H)) {
        const float2 st = stats[at.g];
        of_pair(minus_mean, e) = -st.x;
        of_pair(a, e) = weights[at.c] * st.y;
        of_pair(b, e) = biases[at.c];
    }
}
// The same for the gradient's sums; a = weight * rstd.
template <typename T, int kAct>
__device__ __forceinline__ void form_d(float2 (&v)[4], float2 (&d)[4], const float2 (&minus_mean)[4],
                                       const float2 (&a)[4], const float2 (&b)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) { // x - mean in v's place, d in dy's
        v[i] = dev::add2(v[i], minus_mean[i]);
        if (kAct) d[i] = dev::mul2(d[i], slope2<T, kAct>(dev::fma2(v[i], a[i], b[i])));
    }
}

// The factors of dx = rstd (d w - s1 - h s2) = d a - rstd s1 - ((x - mean) rstd) (rstd s2).
template <bool kFlat>
__device__ __forceinline__ void result_factors(const Layout& H, const Here& h, int lane, const float2* stats,
                                               const float2* means, float2 (&rstd)[4], float2 (&s1)[4], float2 (&s2)[4])
{
    GroupWalk<kFlat> at(H, h, lane);
#pragma unroll
    for (int e = 0; e < 8; ++e, at.next(H)) {
        const float r = stats[at.g].y;
        const float2 m = means[at.g];
        of_pair(rstd, e) = r;
        of_pair(s1, e) = -m.x * r;
        of_pair(s2, e) = -m.y * r;
    }
}

// A thread's sums of d (s) and d * (x - mean) (q): the latter to those of d * h, and both,
// weighed, as the sums (a, b) of its segments.
template <bool kFlat>
__device__ __forceinline__ void put_weighed(const Layout& H, const Here& h, int lane, const float* weights,
                                            const float2* stats, float2 (&s)[4], float2 (&q)[4], const Segments& S)
{
    const int t = threadIdx.x;
    GroupWalk<kFlat> at(H, h, lane);
    const int g = at.g;
    float s0 = 0.0f, s1 = 0.0f, q0 = 0.0f, q1 = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e, at.next(H)) {
        const float w = weights[at.c];
        float& along = of_pair(q, e);
        along *= stats[at.g].y;
        const float ws = of_pair(s, e) * w, wq = along * w;
        if (H.per < 8) {
            S.a[e * kThreads + t] = ws;
            S.b[e * kThreads + t] = wq;
        } else if (at.g != g) {
            s1 += ws;
            q1 += wq;
        } else {
            s0 += ws;
            q0 += wq;
        }
    }
    if (H.per < 8) return;
    S.a[t] = s0, S.b[t] = q0;
    S.a[kThreads + t] = s1, S.b[kThreads + t] = q1;
    S.firsts[t] = g;
}
// After a barrier: done(g, sum of a, sum of b) for each of the slab's groups, by one thread.
template <bool kFlat, typename Done>
__device__ __forceinline__ void join_sums(const Layout& H, int lead, const Segments& S, Done done)
{
    const int gl = lanes_of_group(H), sub = threadIdx.x & (gl - 1);
    for (int g0 = 0; g0 < H.slab_groups; g0 += kThreads / gl) {
        const int g = g0 + threadIdx.x / gl;
        float s = 0.0f, q = 0.0f;
        if (g < H.slab_groups)
            over_segments<kFlat>(H, lead, S.firsts, g, sub, gl, [&](int i) {
                s += S.a[i];
                q += S.b[i];
            });
        s = sum_lanes(s, gl);
        q = sum_lanes(q, gl);
        if (sub == 0 && g < H.slab_groups) done(g, s, q);
    }
}

// Sums of d and d * h of each channel of a block's slab: kept by row group and element
// (straight, along; own words of each thread) and joined into `sums` at the end or, flat,
// whenever the lead changes.
struct ChannelSums {
    float *straight, *along;
    float2* sums;
};
__host__ __device__ __forceinline__ int channel_words(const Layout& H)
{
    return 2 * H.row_groups * 8 * H.lanes + 2 * H.width;
}
__device__ __forceinline__ ChannelSums channels_at(const Layout& H, float* at)
{
    const int entries = H.row_groups * 8 * H.lanes;
    return {at, at + entries, reinterpret_cast<float2*>(at + 2 * entries)};
}
__device__ __forceinline__ void add_channels(const Layout& H, const ChannelSums& C, int rg, int lane, bool first,
                                             const float2 (&s)[4], const float2 (&q)[4])
{
    auto* st = reinterpret_cast<float2*>(C.straight + rg * 8 * H.lanes + lane * 8);
    auto* al = reinterpret_cast<float2*>(C.along + rg * 8 * H.lanes + lane * 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        st[i] = first ? s[i] : dev::add2(st[i], s[i]);
        al[i] = first ? q[i] : dev::add2(al[i], q[i]);
    }
}
// Between barriers.  Each of `parts` threads adds every parts-th row group (and a flat row's
// positions) of a channel.
template <bool kFlat>
__device__ __forceinline__ void join_channels(const Layout& H, const ChannelSums& C, int lead)
{
    const int row_values = 8 * H.lanes;
    const int parts = max(1, min(H.row_groups, kThreads / H.width));
    for (int t = threadIdx.x; t < H.width * parts; t += kThreads) {
        const int part = parts > 1 ? t / H.width : 0, c = t - part * H.width;
        const int begin = kFlat ? (c + lead) % row_values : c;
        float s = 0.0f, q = 0.0f;
#pragma unroll 4
        for (int r = part; r < H.row_groups; r += parts) {
            int i = r * row_values + begin;
            for (int j = 0; j < (kFlat ? H.repeats : 1); ++j) {
                s += C.straight[i];
                q += C.along[i];
                if (kFlat) {
                    i += H.channels;
                    if (i >= (r + 1) * row_values) i -= row_values;
                }
            }
        }
        C.straight[part * row_values + begin] = s;
        C.along[part * row_values + begin] = q;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < H.width; c += kThreads) {
        const int begin = kFlat ? (c + lead) % row_values : c;
        float2 all = C.sums[c];
        for (int part = 0; part < parts; ++part) {
            all.x += C.straight[part * row_values + begin];
            all.y += C.along[part * row_values + begin];
        }
        C.sums[c] = all;
    }
}

// By a block: dweight and dbias of kSumChannels channels from blocks' sums of their slab's
// channels; block j of a slab has the index j * slabs + slab.
constexpr int kSumChannels = 8, kSumSlices = kThreads / kSumChannels;
__device__ __forceinline__ void sum_blocks_of(const Layout& H, int part, const float2* block_sums, int blocks,
                                              void* dweight, void* dbias, int32_t grad_type)
{
    __shared__ float2 slices[kSumSlices][kSumChannels];
    const int lane = threadIdx.x % kSumChannels, slice = threadIdx.x / kSumChannels;
    const int c = part * kSumChannels + lane;
    float s = 0.0f, q = 0.0f;
    if (c < H.channels) {
        const int slab = c / H.width;
        const float2* from = block_sums + static_cast<int64_t>(slab) * H.width + (c - slab * H.width);
#pragma unroll 10
        for (int j = slice; j < blocks; j += kSumSlices) {
            const float2 v = from[static_cast<int64_t>(j) * H.slabs * H.width];
            s += v.x;
            q += v.y;
        }
    }
    slices[slice][lane] = make_float2(s, q);
    __syncthreads();
    if (slice == 0 && c < H.channels) {
        float a[1] = {0.0f}, b[1] = {0.0f};
#pragma unroll 8
        for (int k = 0; k < kSumSlices; ++k) {
            a[0] += slices[k][lane].x;
            b[0] += slices[k][lane].y;
        }
        if (dbias) dev::store_any<1>(dbias, grad_type, c, a);
        if (dweight) dev::store_any<1>(dweight, grad_type, c, b);
    }
}

__device__ __forceinline__ float rstd_of(float count, float m2, float eps)
{
    return 1.0f / sqrtf((count > 0.0f ? m2 / count : 0.0f) + eps);
}

// A slab's weights and biases in fp32.
__device__ __forceinline__ void load_params(const Layout& H, int c0, const void* weight, const void* bias,
                                            int32_t type, float* weights, float* biases)
{
    for (int c = threadIdx.x; c < H.width; c += kThreads) {
        float one[1];
        load_param<1>(weight, type, c0 + c, 1.0f, one);
        weights[c] = one[0];
        load_param<1>(bias, type, c0 + c, 0.0f, one);
        biases[c] = one[0];
    }
}

// ---------------------------------------------------------------------- host
// What the entry points hand to the three ways of running.
struct Call {
    const zero_group_norm_t* norm;
    const void *x, *dy, *weight, *bias;
    const int32_t* lengths;
    const float2* stats_in;
    float2* stats; // may be nullptr
    void *y, *dx, *dweight, *dbias;
    void* scratch;
    cudaStream_t stream;
    bool aligned;   // all row tensors start at multiples of 16 bytes
    bool same_lead; // or equally far behind
};

inline bool rows_whole(const Call& c) // 16-byte accesses at every position
{
    const int unit = 16 / type_bytes(c.norm->type);
    return c.aligned && c.norm->channels % 8 == 0 && c.norm->x_stride % unit == 0 && c.norm->y_stride % unit == 0;
}
inline bool line_whole(const Call& c) // along a sample
{
    return c.same_lead && c.norm->x_stride == c.norm->channels && c.norm->y_stride == c.norm->channels;
}

// A launch that may begin while the kernel before it on the stream drains; the
// kernel waits for that one's results itself.
template <typename... Params, typename... Given>
int launch(bool after, void (*kernel)(Params...), int64_t blocks, size_t shared, cudaStream_t stream, Given... given)
{
    if (blocks > 0x7FFFFFFF) return ZERO_EINVAL;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = after ? 1 : 0;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(given)...));
}

// Two of the ways: the scratch for these sizes at any alignment and type, and the launches.
bool passes_take(const Call& c);
int64_t passes_bytes(const zero_group_norm_t& n);
int passes_forward(const Call& c);
int passes_backward(const Call& c);
int64_t single_bytes(const zero_group_norm_t& n);
int single_forward(const Call& c);
int single_backward(const Call& c);

} // namespace gn
} // namespace zero

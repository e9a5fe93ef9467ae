// group_norm_single.cu -- the group norm a channel at a time, for rows that 16-byte accesses
// cannot reach (channel slices at odd places, tensors unequally far behind a boundary, odd
// widths above 256).  A thread takes a channel and every row_groups-th row of a run; sums
// are [samples][chunks][channels], joined by runs and then by groups.  Loads of 2 or 4 bytes bound
// it: 32 x 4096 x 641 bf16 with rows of 642 takes 197 us (2.6 TB/s of both passes), its gradient 362;
// 32 x 4096 x 640, which does not come here, would take 196 and 363 (95 and 176 by passes).  The runs' join
// has a kernel of its own: 1 x 16384 x 1279 in one group takes 74 us, 2,754 with a warp for all of it.
#include "group_norm.cuh"

namespace zero {
namespace gn {
namespace {

constexpr int kRows = 32; // rows of a thread in a run, at most

struct Grid {
    int64_t x_stride, y_stride;
    const int32_t* lengths;
    int32_t samples, positions, channels, groups, per;
    int32_t lanes, tiles, row_groups; // channels of a block, blocks of a row, rows at once
    int32_t rows, chunks;             // rows of a run, runs of a sample
};

struct Spot { // a thread's channel and rows
    int n, chunk, c, rg, rows; // rows of the block's run
    int64_t row;               // the thread's first, among all samples'
};
__device__ __forceinline__ int length_of(const Grid& G, int n)
{
    return G.lengths ? max(0, min(G.positions, G.lengths[n])) : G.positions;
}
__device__ __forceinline__ Spot spot_of(const Grid& G)
{
    Spot s;
    int64_t i = blockIdx.x;
    const int tile = static_cast<int>(i % G.tiles);
    i /= G.tiles;
    s.chunk = static_cast<int>(i % G.chunks);
    s.n = static_cast<int>(i / G.chunks);
    s.rg = threadIdx.x / G.lanes;
    s.c = tile * G.lanes + threadIdx.x - s.rg * G.lanes;
    s.rows = max(0, min(G.rows, length_of(G, s.n) - s.chunk * G.rows));
    s.row = static_cast<int64_t>(s.n) * G.positions + s.chunk * G.rows + s.rg;
    if (s.rg >= G.row_groups || s.c >= G.channels) s.rg = G.rows; // no row
    return s;
}

// Mean and squares about it of each channel in each run.
template <typename T>
__global__ void __launch_bounds__(kThreads)
single_stats_kernel(const __grid_constant__ Grid G, const T* __restrict__ x, float2* __restrict__ partial)
{
    __shared__ float means[kThreads], squares[kThreads];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Spot p = spot_of(G);
    float mean = 0.0f, square = 0.0f;
    if (p.rg < p.rows) {
        const T* at = x + p.row * G.x_stride + p.c;
        const int64_t step = G.row_groups * G.x_stride;
        const float shift = dev::load1(at);
        float s = 0.0f, q = 0.0f;
        int count = 0;
#pragma unroll 8
        for (int r = p.rg; r < p.rows; r += G.row_groups, at += step, ++count) {
            const float d = dev::load1(at) - shift;
            s += d;
            q = fmaf(d, d, q);
        }
        const float m = s / static_cast<float>(count);
        mean = shift + m;
        square = fmaf(-s, m, q);
        if (square < 0.0f) square = 0.0f; // NaN stays
    }
    means[threadIdx.x] = mean;
    squares[threadIdx.x] = square;
    __syncthreads();
    if (p.rows > 0 && p.rg == 0) { // the row groups joined, about this thread's own mean
        float sum = 0.0f, m2 = 0.0f, rest = 0.0f;
        auto size = [&](int r) { return static_cast<float>((p.rows - r + G.row_groups - 1) / G.row_groups); };
        const int live = min(G.row_groups, p.rows);
        for (int r = 1; r < live; ++r) sum = fmaf(size(r), means[r * G.lanes + threadIdx.x] - mean, sum);
        const float by = 1.0f / static_cast<float>(p.rows);
        mean = fmaf(sum, by, mean);
        for (int r = 0; r < live; ++r) {
            const float d = means[r * G.lanes + threadIdx.x] - mean, n = size(r);
            rest = fmaf(n, d, rest);
            m2 += fmaf(n * d, d, squares[r * G.lanes + threadIdx.x]);
        }
        partial[(static_cast<int64_t>(p.n) * G.chunks + p.chunk) * G.channels + p.c] = corrected(mean, m2, rest, by, 1.0f);
    }
}

// The runs of 32 channels of samples joined, by a warp every kWarps-th run of each.
__global__ void __launch_bounds__(kThreads)
single_runs_kernel(const __grid_constant__ Grid G, const float2* __restrict__ partial, float2* __restrict__ joined)
{
    __shared__ float sums[kWarps][32], squares[kWarps][32], rests[kWarps][32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    const bool live = at < static_cast<int64_t>(G.samples) * G.channels;
    const int n = live ? static_cast<int>(at / G.channels) : 0;
    const int len = live ? length_of(G, n) : 0, chunks = (len + G.rows - 1) / G.rows;
    const float2* from = partial + static_cast<int64_t>(n) * G.chunks * G.channels + (at - static_cast<int64_t>(n) * G.channels);
    const float by = len > 0 ? 1.0f / static_cast<float>(len) : 0.0f;
    const float shift = len > 0 ? from->x : 0.0f;
    auto over = [&](auto f) { // f(rows of the run, its mean and squares)
#pragma unroll 4
        for (int k = warp; k < chunks; k += kWarps)
            f(static_cast<float>(min(G.rows, len - k * G.rows)), from[static_cast<int64_t>(k) * G.channels]);
    };
    float sum = 0.0f, m2 = 0.0f, rest = 0.0f;
    over([&](float rows, float2 v) { sum = fmaf(rows, v.x - shift, sum); });
    sums[warp][lane] = sum;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += sums[w][lane];
    const float mean = fmaf(sum, by, shift);
    over([&](float rows, float2 v) {
        const float d = v.x - mean;
        rest = fmaf(rows, d, rest);
        m2 += fmaf(rows * d, d, v.y);
    });
    squares[warp][lane] = m2;
    rests[warp][lane] = rest;
    __syncthreads();
    if (warp > 0 || len == 0) return;
    m2 = rest = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        m2 += squares[w][lane];
        rest += rests[w][lane];
    }
    joined[at] = corrected(mean, m2, rest, by, 1.0f);
}

// A warp joins the channels of one group of one sample.
__global__ void __launch_bounds__(kThreads)
single_join_kernel(const __grid_constant__ Grid G, const float2* __restrict__ channels, float eps,
                   float2* __restrict__ stats)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (unit >= static_cast<int64_t>(G.samples) * G.groups) return;
    const int n = static_cast<int>(unit / G.groups), g = static_cast<int>(unit - static_cast<int64_t>(n) * G.groups);
    const float len = static_cast<float>(length_of(G, n)), per = static_cast<float>(G.per);
    float2 all = make_float2(0.0f, 0.0f);
    if (len > 0.0f) {
        const float2* from = channels + static_cast<int64_t>(n) * G.channels + g * G.per;
        const float shift = from->x;
        float sum = 0.0f, m2 = 0.0f, rest = 0.0f;
#pragma unroll 8
        for (int c = lane; c < G.per; c += 32) sum += from[c].x - shift;
        sum = sum_lanes(sum, 32);
        const float by = 1.0f / per, mean = fmaf(sum, by, shift);
#pragma unroll 8
        for (int c = lane; c < G.per; c += 32) {
            const float2 v = from[c];
            const float d = v.x - mean;
            rest += d;
            m2 += fmaf(len * d, d, v.y);
        }
        m2 = sum_lanes(m2, 32);
        rest = sum_lanes(rest, 32);
        all = corrected(mean, m2, rest, by, len);
    }
    if (lane == 0) stats[unit] = make_float2(all.x, rstd_of(len * per, all.y, eps));
}

template <typename T, int kAct>
__global__ void __launch_bounds__(kThreads)
single_apply_kernel(const __grid_constant__ Grid G, const T* x, const void* __restrict__ weight,
                    const void* __restrict__ bias, int32_t param_type, const float2* stats, T* y)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Spot p = spot_of(G);
    if (p.rg >= p.rows) return;
    float w[1], b[1];
    load_param<1>(weight, param_type, p.c, 1.0f, w);
    load_param<1>(bias, param_type, p.c, 0.0f, b);
    const float2 st = stats[static_cast<int64_t>(p.n) * G.groups + p.c / G.per];
    const float a = w[0] * st.y;
    const T* from = x + p.row * G.x_stride + p.c;
    T* to = y + p.row * G.y_stride + p.c;
    const int64_t x_step = G.row_groups * G.x_stride, y_step = G.row_groups * G.y_stride;
    constexpr int kAhead = 8;
    for (int r = p.rg; r < p.rows; r += kAhead * G.row_groups) {
        float v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (r + k * G.row_groups < p.rows) v[k] = dev::load1(from + k * x_step);
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (r + k * G.row_groups < p.rows)
                dev::store1(to + k * y_step, activated<T, kAct>(fmaf(v[k] - st.x, a, b[0])));
        from += kAhead * x_step;
        to += kAhead * y_step;
    }
}

// ------------------------------------------------------------------ backward
// Sums of d and d * h of each channel in each run.
template <typename T, int kAct>
__global__ void __launch_bounds__(kThreads)
single_sums_kernel(const __grid_constant__ Grid G, const T* __restrict__ x, const T* __restrict__ dy,
                   const void* __restrict__ weight, const void* __restrict__ bias, int32_t param_type,
                   const float2* __restrict__ stats, float2* __restrict__ partial)
{
    __shared__ float2 sums[kThreads];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Spot p = spot_of(G);
    float s = 0.0f, q = 0.0f;
    if (p.rg < p.rows) {
        float w[1], b[1];
        load_param<1>(weight, param_type, p.c, 1.0f, w);
        load_param<1>(bias, param_type, p.c, 0.0f, b);
        const float2 st = stats[static_cast<int64_t>(p.n) * G.groups + p.c / G.per];
        const T* xp = x + p.row * G.x_stride + p.c;
        const T* dp = dy + p.row * G.y_stride + p.c;
        const int64_t x_step = G.row_groups * G.x_stride, y_step = G.row_groups * G.y_stride;
#pragma unroll 4
        for (int r = p.rg; r < p.rows; r += G.row_groups, xp += x_step, dp += y_step) {
            const float h = (dev::load1(xp) - st.x) * st.y, dy1 = dev::load1(dp);
            const float d = kAct ? dy1 * slope<T, kAct>(fmaf(h, w[0], b[0])) : dy1;
            s += d;
            q = fmaf(d, h, q);
        }
    }
    sums[threadIdx.x] = make_float2(s, q);
    __syncthreads();
    if (p.rows > 0 && p.rg == 0) {
        for (int r = 1; r < G.row_groups; ++r) {
            s += sums[r * G.lanes + threadIdx.x].x;
            q += sums[r * G.lanes + threadIdx.x].y;
        }
        partial[(static_cast<int64_t>(p.n) * G.chunks + p.chunk) * G.channels + p.c] = make_float2(s, q);
    }
}

// The runs' sums of one channel of one sample.
__global__ void __launch_bounds__(kThreads)
single_channels_kernel(const __grid_constant__ Grid G, const float2* __restrict__ partial, float2* __restrict__ sums)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (at >= static_cast<int64_t>(G.samples) * G.channels) return;
    const int n = static_cast<int>(at / G.channels), c = static_cast<int>(at - static_cast<int64_t>(n) * G.channels);
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

// Blocks below group_blocks: a warp for each group of each sample, its means of d * weight and
// d * weight * h; the others: dweight and dbias of kSumChannels channels over the samples.
__global__ void __launch_bounds__(kThreads)
single_groups_kernel(const __grid_constant__ Grid G, const float2* __restrict__ sums, const void* __restrict__ weight,
                     int32_t param_type, int64_t group_blocks, float2* __restrict__ means, void* dweight, void* dbias,
                     int32_t grad_type)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x >= group_blocks) {
        Layout one = {}; // the samples' sums as blocks of one slab
        one.channels = one.width = G.channels;
        one.slabs = 1;
        sum_blocks_of(one, static_cast<int>(blockIdx.x - group_blocks), sums, G.samples, dweight, dbias, grad_type);
        return;
    }
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (unit >= static_cast<int64_t>(G.samples) * G.groups) return;
    const int n = static_cast<int>(unit / G.groups), g = static_cast<int>(unit - static_cast<int64_t>(n) * G.groups);
    const float2* from = sums + static_cast<int64_t>(n) * G.channels;
    float s = 0.0f, q = 0.0f;
    for (int c = g * G.per + lane; c < (g + 1) * G.per; c += 32) {
        float w[1];
        load_param<1>(weight, param_type, c, 1.0f, w);
        s = fmaf(w[0], from[c].x, s);
        q = fmaf(w[0], from[c].y, q);
    }
    s = sum_lanes(s, 32);
    q = sum_lanes(q, 32);
    if (lane == 0) {
        const float size = static_cast<float>(length_of(G, n)) * static_cast<float>(G.per);
        const float inv = size > 0.0f ? 1.0f / size : 0.0f;
        means[unit] = make_float2(s * inv, q * inv);
    }
}

template <typename T, int kAct>
__global__ void __launch_bounds__(kThreads)
single_gradient_kernel(const __grid_constant__ Grid G, const T* __restrict__ x, const T* dy,
                       const void* __restrict__ weight, const void* __restrict__ bias, int32_t param_type,
                       const float2* __restrict__ stats, const float2* means, T* dx)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Spot p = spot_of(G);
    if (p.rg >= p.rows) return;
    float w[1], b[1];
    load_param<1>(weight, param_type, p.c, 1.0f, w);
    load_param<1>(bias, param_type, p.c, 0.0f, b);
    const int64_t unit = static_cast<int64_t>(p.n) * G.groups + p.c / G.per;
    const float2 st = stats[unit], m = means[unit];
    const T* xp = x + p.row * G.x_stride + p.c;
    const T* dp = dy + p.row * G.y_stride + p.c;
    T* to = dx + p.row * G.x_stride + p.c;
    const int64_t x_step = G.row_groups * G.x_stride, y_step = G.row_groups * G.y_stride;
    constexpr int kAhead = 4;
    for (int r = p.rg; r < p.rows; r += kAhead * G.row_groups) {
        float v[kAhead], d[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (r + k * G.row_groups < p.rows) {
                v[k] = dev::load1(xp + k * x_step);
                d[k] = dev::load1(dp + k * y_step);
            }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (r + k * G.row_groups < p.rows) {
                const float h = (v[k] - st.x) * st.y;
                const float g = kAct ? d[k] * slope<T, kAct>(fmaf(h, w[0], b[0])) : d[k];
                dev::store1(to + k * x_step, st.y * fmaf(-h, m.y, fmaf(g, w[0], -m.x)));
            }
        xp += kAhead * x_step;
        dp += kAhead * y_step;
        to += kAhead * x_step;
    }
}

// --------------------------------------------------------------------- host
Grid grid_of(const zero_group_norm_t& n, const int32_t* lengths)
{
    Grid G = {};
    G.x_stride = n.x_stride;
    G.y_stride = n.y_stride;
    G.lengths = lengths;
    G.samples = static_cast<int32_t>(n.samples);
    G.positions = static_cast<int32_t>(n.positions);
    G.channels = static_cast<int32_t>(n.channels);
    G.groups = n.groups;
    G.per = G.channels / G.groups;
    G.tiles = (G.channels + kThreads - 1) / kThreads;
    G.lanes = (G.channels + G.tiles - 1) / G.tiles;
    G.row_groups = kThreads / G.lanes;
    int64_t rows = n.samples * G.tiles * n.positions / (static_cast<int64_t>(G.row_groups) * 152 * 8);
    rows = rows < 4 ? 4 : rows > kRows ? kRows : rows;
    G.rows = static_cast<int32_t>(rows) * G.row_groups;
    G.chunks = static_cast<int32_t>((n.positions + G.rows - 1) / G.rows);
    return G;
}
int64_t blocks_of(const Grid& G) { return static_cast<int64_t>(G.samples) * G.chunks * G.tiles; }

struct Scratch {
    float2 *partial, *sums, *groups; // [samples][chunks][channels], [samples][channels], [samples][groups]
    int64_t bytes;
};
Scratch scratch_of(void* base, const Grid& G)
{
    const int64_t m = static_cast<int64_t>(G.samples) * G.channels, n = m * G.chunks;
    Scratch s;
    s.partial = static_cast<float2*>(base);
    s.sums = s.partial + n;
    s.groups = s.sums + m;
    s.bytes = (n + m + static_cast<int64_t>(G.samples) * G.groups) * 8;
    return s;
}

template <typename T, int kAct>
int forward(const Call& c)
{
    const Grid G = grid_of(*c.norm, c.lengths);
    const Scratch s = scratch_of(c.scratch, G);
    const int64_t blocks = blocks_of(G), units = static_cast<int64_t>(G.samples) * G.groups;
    if (blocks > 0x7FFFFFFF) return ZERO_EINVAL;
    float2* stats = c.stats ? c.stats : s.groups;
    const auto* x = static_cast<const T*>(c.x);
    int rc = ZERO_OK;
    if (blocks > 0) rc = launch(false, single_stats_kernel<T>, blocks, 0, c.stream, G, x, s.partial);
    const bool runs = G.chunks > 1; // else the one run's sums are the channels'
    if (rc == ZERO_OK && runs)
        rc = launch(true, single_runs_kernel, (static_cast<int64_t>(G.samples) * G.channels + 31) / 32, 0, c.stream, G,
                    s.partial, s.sums);
    if (rc == ZERO_OK)
        rc = launch(blocks > 0, single_join_kernel, (units + kWarps - 1) / kWarps, 0, c.stream, G,
                    runs ? s.sums : s.partial, static_cast<float>(c.norm->eps), stats);
    if (rc == ZERO_OK && blocks > 0)
        rc = launch(true, single_apply_kernel<T, kAct>, blocks, 0, c.stream, G, x, c.weight, c.bias,
                    c.norm->param_type, stats, static_cast<T*>(c.y));
    return rc;
}

template <typename T, int kAct>
int backward(const Call& c)
{
    const Grid G = grid_of(*c.norm, c.lengths);
    const Scratch s = scratch_of(c.scratch, G);
    const int64_t blocks = blocks_of(G), units = static_cast<int64_t>(G.samples) * G.groups;
    if (blocks > 0x7FFFFFFF) return ZERO_EINVAL;
    const auto* x = static_cast<const T*>(c.x);
    const auto* dy = static_cast<const T*>(c.dy);
    int rc = ZERO_OK;
    if (blocks > 0)
        rc = launch(false, single_sums_kernel<T, kAct>, blocks, 0, c.stream, G, x, dy, c.weight, c.bias,
                    c.norm->param_type, c.stats_in, s.partial);
    const int64_t channels = static_cast<int64_t>(G.samples) * G.channels;
    if (rc == ZERO_OK && channels > 0)
        rc = launch(blocks > 0, single_channels_kernel, (channels + kThreads - 1) / kThreads, 0, c.stream, G, s.partial,
                    s.sums);
    const int64_t group_blocks = c.dx ? (units + kWarps - 1) / kWarps : 0;
    const int64_t more = c.dweight || c.dbias ? (G.channels + kSumChannels - 1) / kSumChannels : 0;
    if (rc == ZERO_OK && group_blocks + more > 0)
        rc = launch(channels > 0, single_groups_kernel, group_blocks + more, 0, c.stream, G, s.sums, c.weight,
                    c.norm->param_type, group_blocks, s.groups, c.dweight, c.dbias, c.norm->grad_type);
    if (rc == ZERO_OK && c.dx && blocks > 0)
        rc = launch(true, single_gradient_kernel<T, kAct>, blocks, 0, c.stream, G, x, dy, c.weight, c.bias,
                    c.norm->param_type, c.stats_in, s.groups, static_cast<T*>(c.dx));
    return rc;
}

template <typename T>
int forward_by_act(const Call& c)
{
    switch (c.norm->act) {
    case ZERO_ACT_SILU: return forward<T, ZERO_ACT_SILU>(c);
    case ZERO_ACT_GELU: return forward<T, ZERO_ACT_GELU>(c);
    default: return forward<T, ZERO_ACT_NONE>(c);
    }
}
template <typename T>
int backward_by_act(const Call& c)
{
    switch (c.norm->act) {
    case ZERO_ACT_SILU: return backward<T, ZERO_ACT_SILU>(c);
    case ZERO_ACT_GELU: return backward<T, ZERO_ACT_GELU>(c);
    default: return backward<T, ZERO_ACT_NONE>(c);
    }
}

} // namespace

int64_t single_bytes(const zero_group_norm_t& n) { return scratch_of(nullptr, grid_of(n, nullptr)).bytes; }
int single_forward(const Call& c)
{
    return c.norm->type == ZERO_TYPE_BF16 ? forward_by_act<Bf16>(c) : forward_by_act<float>(c);
}
int single_backward(const Call& c)
{
    return c.norm->type == ZERO_TYPE_BF16 ? backward_by_act<Bf16>(c) : backward_by_act<float>(c);
}

} // namespace gn
} // namespace zero

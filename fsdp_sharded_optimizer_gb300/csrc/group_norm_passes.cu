// group_norm_passes.cu -- the group norm where a slab of a sample does not fit one block:
// sums of runs of rows, their join, and a second pass over the rows for the result.  The
// second pass takes the last rows first: the L2 may hold them still.
//
// What bounds it: HBM, with x (and dy) read twice.  32 x 16384 x 320 bf16 takes 184 us, 5.5 TB/s
// of the 1,007 MB of both passes (65 us for the sums, 115 for the result); the gradient of 32 x
// 4096 x 640 177 us, 4.7 TB/s of 839 MB (80 and 95 us: 16 warps an SM, as the factors of eight
// channels take 48 registers).  Parts of the samples that fit the L2, one after another, take
// longer (64 MB: 251 us): every part has three launches to wait for.  24 x 3001 x 81 with GELU and
// lengths down to half takes 40 us for 26 MB: a chain of loads, joins and launches in one round of
// blocks.
#include "group_norm.cuh"

namespace zero {
namespace gn {
namespace {

constexpr int kResident = 152 * 2; // blocks at once, two an SM
constexpr int kMostSlots = 64;     // rows of a thread in a run

struct Run { // a block's work
    int n, slab, chunk;
};
__device__ __forceinline__ Run run_of(const Layout& H, int64_t i)
{
    Run r;
    r.chunk = static_cast<int>(i % H.chunks);
    i /= H.chunks;
    r.slab = static_cast<int>(i % H.slabs);
    r.n = static_cast<int>(i / H.slabs);
    return r;
}

// Rows 0 .. rows - 1 by kAhead, without a branch between those.  kNext: the next ones are
// loaded before the last ones are used.  On 32 x 4096 x 640 bf16 the gradient's sums take 80 us
// by four and 95 by two and the next two; its result 110 and 95.
template <int kAhead, bool kNext, typename R, typename Fetch, typename Use>
__device__ __forceinline__ void over_rows(int rows, Fetch fetch, Use use)
{
    int k = 0;
    if constexpr (!kNext) {
        for (; k + kAhead <= rows; k += kAhead) {
            R r[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) fetch(k + i, r[i]);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) use(k + i, r[i]);
        }
    } else if (rows >= kAhead) {
        R a[kAhead], b[kAhead];
        auto load = [&](R(&r)[kAhead], int from) {
            if (from + kAhead > rows) return;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) fetch(from + i, r[i]);
        };
        auto take = [&](const R(&r)[kAhead]) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) use(k + i, r[i]);
            k += kAhead;
        };
        load(a, 0);
        for (;;) {
            load(b, k + kAhead);
            take(a);
            if (k + kAhead > rows) break;
            load(a, k + kAhead);
            take(b);
            if (k + kAhead > rows) break;
        }
    }
    for (; k < rows; ++k) {
        R r;
        fetch(k, r);
        use(k, r);
    }
}
template <typename T>
struct Pair { // a row of x and of dy
    Raw8<T> x, d;
};

// Mean, squares about it and size of each group in each run.
template <typename T, bool kFlat>
__global__ void __launch_bounds__(kThreads, 3)
stats_kernel(const __grid_constant__ Layout H, const T* __restrict__ x, float4* __restrict__ partial)
{
    extern __shared__ float4 shared[];
    const Segments S = segments_at(H, 3, reinterpret_cast<float*>(shared));
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Run run = run_of(H, blockIdx.x);
    const int rg = threadIdx.x / H.lanes, lane = threadIdx.x - rg * H.lanes;
    const int row0 = run.chunk * H.slots * H.row_groups;
    const Here h = here_of<kFlat>(H, run.n, x, rg, lane, row0);
    const T* xp = x + (row0 + rg) * H.x_stride + run.slab * H.width + lane * 8;
    sum_rows<kFlat, sizeof(T) == 2 ? 8 : 4, T>(H, h, rg, lane, S, [&](int k, Raw8<T>& r) {
        load_row<kFlat, false>(H, h, k, xp, H.x_sample, H.x_stride, r);
    });
    __syncthreads();
    float4* to = partial + (static_cast<int64_t>(run.n) * H.groups + run.slab * H.slab_groups) * H.chunks + run.chunk;
    join_groups<kFlat>(H, h.lead, S, [&](int g, float count, float mean, float m2) {
        to[static_cast<int64_t>(g) * H.chunks] = make_float4(mean, m2, count, 0.0f);
    });
}

// A warp joins the runs of one group of one sample.
__global__ void __launch_bounds__(kThreads)
join_stats_kernel(const __grid_constant__ Layout H, const float4* __restrict__ partial, float eps,
                  float2* __restrict__ stats)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, entries = H.splits * H.chunks;
    if (unit >= static_cast<int64_t>(H.samples) * (H.groups / H.splits)) return;
    const float4* from = partial + unit * entries;
    float count = 0.0f, sum = 0.0f, m2 = 0.0f;
#pragma unroll 4
    for (int k = lane; k < entries; k += 32) {
        const float4 v = from[k];
        count += v.z;
        sum = fmaf(v.z, v.x, sum);
    }
    count = sum_lanes(count, 32);
    sum = sum_lanes(sum, 32);
    const float by = count > 0.0f ? 1.0f / count : 0.0f, near = sum * by;
    float rest = 0.0f;
#pragma unroll 4
    for (int k = lane; k < entries; k += 32) {
        const float4 v = from[k];
        const float d = v.x - near, sized = v.z * d;
        rest += sized;
        m2 += v.z > 0.0f ? fmaf(sized, d, v.y) : 0.0f;
    }
    m2 = sum_lanes(m2, 32);
    rest = sum_lanes(rest, 32);
    const float2 all = corrected(near, m2, rest, by, 1.0f);
    if (lane == 0) stats[unit] = make_float2(all.x, rstd_of(count, all.y, eps));
}

// A slab's values by group (of which parts share one where groups are split).
__device__ __forceinline__ void load_groups(const Layout& H, const Run& run, const float2* from, float2* to)
{
    for (int g = threadIdx.x; g < H.slab_groups; g += kThreads) {
        const int all = run.slab * H.slab_groups + g;
        to[g] = from[static_cast<int64_t>(run.n) * (H.groups / H.splits) + all / H.splits];
    }
}

template <typename T, int kAct, bool kFlat>
__global__ void __launch_bounds__(kThreads, 4)
apply_kernel(const __grid_constant__ Layout H, const T* x, const void* __restrict__ weight,
             const void* __restrict__ bias, int32_t param_type, const float2* stats, T* y)
{
    extern __shared__ float4 shared[];
    float* weights = reinterpret_cast<float*>(shared);
    float* biases = weights + H.width;
    float2* group_stats = reinterpret_cast<float2*>(biases + H.width);
    const Run run = run_of(H, static_cast<int64_t>(gridDim.x) - 1 - blockIdx.x);
    const int rg = threadIdx.x / H.lanes, lane = threadIdx.x - rg * H.lanes;
    const int row0 = run.chunk * H.slots * H.row_groups;
    load_params(H, run.slab * H.width, weight, bias, param_type, weights, biases);
    const Here h = here_of<kFlat>(H, run.n, x, rg, lane, row0);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    load_groups(H, run, stats, group_stats);
    __syncthreads();
    if (h.rows == 0) return;
    float2 minus_mean[4], a[4], b[4];
    forward_factors<kFlat>(H, h, lane, weights, biases, group_stats, minus_mean, a, b);
    const T* xp = x + (row0 + rg) * H.x_stride + run.slab * H.width + lane * 8;
    T* yp = y + (row0 + rg) * H.y_stride + run.slab * H.width + lane * 8;
    auto put = [&](int k, const Raw8<T>& raw) {
        float2 v[4];
        dev::unpack8(raw, v);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = activated2<T, kAct>(dev::fma2(dev::add2(v[j], minus_mean[j]), a[j], b[j]));
        store_row<kFlat>(H, h, k, yp, H.y_sample, H.y_stride, v);
    };
    over_rows<sizeof(T) == 2 ? 2 : 1, true, Raw8<T>>(h.rows, [&](int k, Raw8<T>& raw) {
        load_row<kFlat, true>(H, h, k, xp, H.x_sample, H.x_stride, raw);
    }, put);
}

// ------------------------------------------------------------------ backward
// Sums of d * weight and d * weight * h of each group in each run, and the block's sums of d
// and d * h of each channel.  A block takes consecutive runs of one slab.
template <typename T, int kAct, bool kFlat>
__global__ void __launch_bounds__(kThreads, 2)
sums_kernel(const __grid_constant__ Layout H, const T* __restrict__ x, const T* __restrict__ dy,
            const void* __restrict__ weight, const void* __restrict__ bias, int32_t param_type,
            const float2* __restrict__ stats, float2* __restrict__ partial, float2* __restrict__ block_sums)
{
    extern __shared__ float4 shared[];
    float* words = reinterpret_cast<float*>(shared);
    const ChannelSums C = channels_at(H, words);
    words += channel_words(H);
    const Segments S = segments_at(H, 2, words);
    float2* group_stats = reinterpret_cast<float2*>(words + segment_words(H, 2));
    float* weights = reinterpret_cast<float*>(group_stats + H.slab_groups);
    float* biases = weights + H.width;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int rg = threadIdx.x / H.lanes, lane = threadIdx.x - rg * H.lanes;
    Run run;
    run.slab = blockIdx.x % H.slabs;
    const int64_t runs = static_cast<int64_t>(H.samples) * H.chunks, blocks = gridDim.x / H.slabs;
    const int64_t from = blockIdx.x / H.slabs * runs / blocks, to = (blockIdx.x / H.slabs + 1) * runs / blocks;
    load_params(H, run.slab * H.width, weight, bias, param_type, weights, biases);
    for (int c = threadIdx.x; c < H.width; c += kThreads) C.sums[c] = make_float2(0.0f, 0.0f);

    float2 minus_mean[4], a[4], b[4];
    Here h;
    bool first = true;
    int last_n = -1, lead = 0;
    for (int64_t i = from; i < to; ++i) {
        run.n = static_cast<int>(i / H.chunks);
        run.chunk = static_cast<int>(i - static_cast<int64_t>(run.n) * H.chunks);
        const int row0 = run.chunk * H.slots * H.row_groups;
        h = here_of<kFlat>(H, run.n, x, rg, lane, row0);
        if (run.n != last_n) {
            __syncthreads();
            if (kFlat && !first) {
                join_channels<kFlat>(H, C, lead);
                first = true;
            }
            load_groups(H, run, stats, group_stats);
            __syncthreads();
            if (rg < H.row_groups)
                forward_factors<kFlat>(H, h, lane, weights, biases, group_stats, minus_mean, a, b);
            last_n = run.n;
            lead = h.lead;
        }
        if (rg < H.row_groups) {
            const T* xp = x + (row0 + rg) * H.x_stride + run.slab * H.width + lane * 8;
            const T* dp = dy + (row0 + rg) * H.y_stride + run.slab * H.width + lane * 8;
            float2 s[4], q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] = q[j] = make_float2(0.0f, 0.0f);
            over_rows<sizeof(T) == 2 ? 4 : 2, false, Pair<T>>(h.rows, [&](int k, Pair<T>& r) {
                load_row<kFlat, false>(H, h, k, xp, H.x_sample, H.x_stride, r.x);
                load_row<kFlat, false>(H, h, k, dp, H.y_sample, H.y_stride, r.d);
            }, [&](int k, const Pair<T>& r) {
                float2 v[4], d[4];
                dev::unpack8(r.x, v);
                dev::unpack8(r.d, d);
                form_d<T, kAct>(v, d, minus_mean, a, b);
                if (kFlat && !whole<kFlat>(H, h, k))
                    outside(H, h, k, [&](int e) { of_pair(v, e) = of_pair(d, e) = 0.0f; });
#pragma unroll
                for (int l = 0; l < 4; ++l) {
                    s[l] = dev::add2(s[l], d[l]);
                    q[l] = dev::fma2(d[l], v[l], q[l]);
                }
            });
            put_weighed<kFlat>(H, h, lane, weights, group_stats, s, q, S);
            add_channels(H, C, rg, lane, first, s, q);
        }
        first = false;
        __syncthreads();
        float2* out = partial + (static_cast<int64_t>(run.n) * H.groups + run.slab * H.slab_groups) * H.chunks + run.chunk;
        join_sums<kFlat>(H, h.lead, S, [&](int g, float s, float q) {
            out[static_cast<int64_t>(g) * H.chunks] = make_float2(s, q);
        });
        __syncthreads();
    }
    __syncthreads();
    if (!first) join_channels<kFlat>(H, C, lead);
    for (int c = threadIdx.x; c < H.width; c += kThreads) // each by the thread that summed it
        block_sums[static_cast<int64_t>(blockIdx.x) * H.width + c] = C.sums[c];
}

// Blocks below group_blocks: a warp for each group of each sample, its means of d * weight and
// d * weight * h; the others dweight and dbias of kSumChannels channels each.
__global__ void __launch_bounds__(kThreads)
join_sums_kernel(const __grid_constant__ Layout H, const float2* __restrict__ partial, int64_t group_blocks,
                 float2* __restrict__ means, const float2* __restrict__ block_sums, int blocks_of_slab, void* dweight,
                 void* dbias, int32_t grad_type)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x >= group_blocks) {
        sum_blocks_of(H, static_cast<int>(blockIdx.x - group_blocks), block_sums, blocks_of_slab, dweight, dbias, grad_type);
        return;
    }
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, entries = H.splits * H.chunks;
    if (unit >= static_cast<int64_t>(H.samples) * (H.groups / H.splits)) return;
    const float2* from = partial + unit * entries;
    float s = 0.0f, q = 0.0f;
#pragma unroll 4
    for (int k = lane; k < entries; k += 32) {
        const float2 v = from[k];
        s += v.x;
        q += v.y;
    }
    s = sum_lanes(s, 32);
    q = sum_lanes(q, 32);
    if (lane == 0) {
        const int n = static_cast<int>(unit / (H.groups / H.splits));
        const float size = static_cast<float>(length_of(H, n)) * static_cast<float>(H.per * H.splits);
        const float inv = size > 0.0f ? 1.0f / size : 0.0f;
        means[unit] = make_float2(s * inv, q * inv);
    }
}

template <typename T, int kAct, bool kFlat>
__global__ void __launch_bounds__(kThreads, 2)
apply_gradient_kernel(const __grid_constant__ Layout H, const T* __restrict__ x, const T* dy,
                      const void* __restrict__ weight, const void* __restrict__ bias, int32_t param_type,
                      const float2* __restrict__ stats, const float2* means, T* dx)
{
    extern __shared__ float4 shared[];
    float* weights = reinterpret_cast<float*>(shared);
    float* biases = weights + H.width;
    float2* group_stats = reinterpret_cast<float2*>(biases + H.width);
    float2* group_means = group_stats + H.slab_groups;
    const Run run = run_of(H, static_cast<int64_t>(gridDim.x) - 1 - blockIdx.x);
    const int rg = threadIdx.x / H.lanes, lane = threadIdx.x - rg * H.lanes;
    const int row0 = run.chunk * H.slots * H.row_groups;
    load_params(H, run.slab * H.width, weight, bias, param_type, weights, biases);
    load_groups(H, run, stats, group_stats);
    const Here h = here_of<kFlat>(H, run.n, x, rg, lane, row0);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    load_groups(H, run, means, group_means);
    __syncthreads();
    if (h.rows == 0) return;
    float2 minus_mean[4], a[4], b[4], rstd[4], s1[4], s2[4];
    forward_factors<kFlat>(H, h, lane, weights, biases, group_stats, minus_mean, a, b);
    result_factors<kFlat>(H, h, lane, group_stats, group_means, rstd, s1, s2);
    const T* xp = x + (row0 + rg) * H.x_stride + run.slab * H.width + lane * 8;
    const T* dp = dy + (row0 + rg) * H.y_stride + run.slab * H.width + lane * 8;
    T* out = dx + (row0 + rg) * H.x_stride + run.slab * H.width + lane * 8;
    over_rows<sizeof(T) == 2 ? 2 : 1, true, Pair<T>>(h.rows, [&](int k, Pair<T>& r) {
        load_row<kFlat, true>(H, h, k, xp, H.x_sample, H.x_stride, r.x);
        load_row<kFlat, true>(H, h, k, dp, H.y_sample, H.y_stride, r.d);
    }, [&](int k, const Pair<T>& r) {
        float2 v[4], d[4];
        dev::unpack8(r.x, v);
        dev::unpack8(r.d, d);
        form_d<T, kAct>(v, d, minus_mean, a, b);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = dev::fma2(dev::mul2(v[j], rstd[j]), s2[j], dev::fma2(d[j], a[j], s1[j]));
        store_row<kFlat>(H, h, k, out, H.x_sample, H.x_stride, v);
    });
}

// --------------------------------------------------------------------- host
// false: a slab of these channels is not possible.
bool make_layout(const zero_group_norm_t& n, bool flat, bool backward, Layout* out)
{
    if (n.positions * n.channels >= (int64_t(1) << 30) && flat) return false;
    Layout H = {};
    H.samples = static_cast<int32_t>(n.samples);
    H.positions = static_cast<int32_t>(n.positions);
    H.channels = static_cast<int32_t>(n.channels);
    H.groups = n.groups;
    H.per = H.channels / H.groups;
    H.splits = H.repeats = 1;
    if (flat) {
        while (H.repeats * H.channels % 8 != 0) ++H.repeats;
        if (H.repeats * H.channels > kWidth) return false;
        H.slab_groups = H.groups;
    } else {
        if (H.channels % 8 != 0) return false;
        if (H.per > kWidth) {
            int splits = 2;
            while (splits <= H.per && (H.per % splits != 0 || H.per / splits > kWidth || H.per / splits % 8 != 0)) ++splits;
            if (splits > H.per) return false;
            H.splits = splits;
            H.per /= splits;
            H.groups *= splits;
        }
        for (int g = 1; g <= H.groups && g * H.per <= kWidth; ++g)
            if (H.groups % g == 0 && g * H.per % 8 == 0) H.slab_groups = g;
        if (H.slab_groups == 0) return false;
    }
    H.slabs = H.groups / H.slab_groups;
    H.width = H.slab_groups * H.per;
    H.lanes = H.repeats * H.width / 8;
    H.row_groups = kThreads / H.lanes;
    const int64_t rows = flat ? (n.positions * n.channels + 7 + 8 * H.lanes - 1) / (8 * H.lanes) : n.positions;
    const int64_t steps = (rows + H.row_groups - 1) / H.row_groups; // rows of a thread in a sample
    // As many rows to a run as leave a few rounds of blocks (backward one: a block takes several
    // runs then), and then as leave the last round full.
    const int64_t all = n.samples * H.slabs;
    int64_t slots = all * steps / (kResident * (backward ? 1 : 4));
    slots = slots < 4 ? 4 : slots > kMostSlots ? kMostSlots : slots;
    double best = 0;
    for (int64_t t = slots; t > slots / 2; --t) {
        const int64_t runs = all * ((steps + t - 1) / t);
        const double use = static_cast<double>(runs) / static_cast<double>((runs + kResident - 1) / kResident * kResident);
        if (use > best + 0.02) best = use, slots = t;
    }
    H.slots = static_cast<int32_t>(slots);
    H.chunks = static_cast<int32_t>((steps + slots - 1) / slots);
    *out = H;
    return true;
}

Layout layout_of(const Call& c, bool flat, bool backward)
{
    Layout H;
    make_layout(*c.norm, flat, backward, &H);
    H.lengths = c.lengths;
    H.x_sample = c.norm->positions * c.norm->x_stride;
    H.y_sample = c.norm->positions * c.norm->y_stride;
    H.x_stride = flat ? 8 * H.lanes : c.norm->x_stride;
    H.y_stride = flat ? 8 * H.lanes : c.norm->y_stride;
    return H;
}

int64_t runs_of(const Layout& H) { return static_cast<int64_t>(H.samples) * H.slabs * H.chunks; }

struct Scratch {
    float4* partial;    // [samples][groups][chunks], forward; float2 backward
    float2* groups;     // [samples][groups]: statistics, or means
    float2* block_sums; // [blocks][width]
    int64_t bytes;
};
Scratch scratch_of(void* base, const Layout& H)
{
    Scratch s;
    auto* at = static_cast<char*>(base);
    s.partial = reinterpret_cast<float4*>(at);
    at += static_cast<int64_t>(H.samples) * H.groups * H.chunks * 16;
    s.groups = reinterpret_cast<float2*>(at);
    at += (static_cast<int64_t>(H.samples) * H.groups * 8 + 15) / 16 * 16;
    s.block_sums = reinterpret_cast<float2*>(at);
    at += static_cast<int64_t>(kResident) * H.width * 8;
    s.bytes = at - static_cast<char*>(base);
    return s;
}

template <typename T, int kAct, bool kFlat>
int forward(const Call& c)
{
    const Layout H = layout_of(c, kFlat, false);
    const Scratch s = scratch_of(c.scratch, H);
    const int64_t runs = runs_of(H), units = static_cast<int64_t>(H.samples) * (H.groups / H.splits);
    float2* stats = c.stats ? c.stats : s.groups;
    const auto* x = static_cast<const T*>(c.x);
    int rc = launch(false, stats_kernel<T, kFlat>, runs, 4 * segment_words(H, 3), c.stream, H, x, s.partial);
    if (rc == ZERO_OK)
        rc = launch(true, join_stats_kernel, (units + kWarps - 1) / kWarps, 0, c.stream, H, s.partial,
                    static_cast<float>(c.norm->eps), stats);
    if (rc == ZERO_OK)
        rc = launch(true, apply_kernel<T, kAct, kFlat>, runs, 8 * (H.width + H.slab_groups), c.stream, H, x, c.weight,
                    c.bias, c.norm->param_type, stats, static_cast<T*>(c.y));
    return rc;
}

template <typename T, int kAct, bool kFlat>
int backward(const Call& c)
{
    const Layout H = layout_of(c, kFlat, true);
    const Scratch s = scratch_of(c.scratch, H);
    const int64_t runs = runs_of(H), units = static_cast<int64_t>(H.samples) * (H.groups / H.splits);
    const auto* x = static_cast<const T*>(c.x);
    const auto* dy = static_cast<const T*>(c.dy);
    auto* partial = reinterpret_cast<float2*>(s.partial);
    int64_t blocks = kResident / H.slabs; // of each slab
    if (blocks > runs / H.slabs) blocks = runs / H.slabs;
    auto* sums = sums_kernel<T, kAct, kFlat>;
    const int64_t words = channel_words(H) + segment_words(H, 2) + 2 * H.slab_groups + 2 * H.width;
    if (!allow_shared(reinterpret_cast<const void*>(sums), 113 * 1024)) return ZERO_ECUDA;
    int rc = launch(false, sums, blocks * H.slabs, static_cast<size_t>(4 * words), c.stream, H, x, dy, c.weight, c.bias,
                    c.norm->param_type, c.stats_in, partial, s.block_sums);
    const int64_t group_blocks = c.dx ? (units + kWarps - 1) / kWarps : 0;
    const int64_t more = c.dweight || c.dbias ? (H.channels + kSumChannels - 1) / kSumChannels : 0;
    if (rc == ZERO_OK && group_blocks + more > 0)
        rc = launch(true, join_sums_kernel, group_blocks + more, 0, c.stream, H, partial, group_blocks, s.groups,
                    s.block_sums, static_cast<int>(blocks), c.dweight, c.dbias, c.norm->grad_type);
    if (rc == ZERO_OK && c.dx)
        rc = launch(true, apply_gradient_kernel<T, kAct, kFlat>, runs, 8 * (H.width + 2 * H.slab_groups), c.stream, H, x,
                    dy, c.weight, c.bias, c.norm->param_type, c.stats_in, s.groups, static_cast<T*>(c.dx));
    return rc;
}

template <typename T, bool kFlat>
int forward_by_act(const Call& c)
{
    switch (c.norm->act) {
    case ZERO_ACT_SILU: return forward<T, ZERO_ACT_SILU, kFlat>(c);
    case ZERO_ACT_GELU: return forward<T, ZERO_ACT_GELU, kFlat>(c);
    default: return forward<T, ZERO_ACT_NONE, kFlat>(c);
    }
}
template <typename T, bool kFlat>
int backward_by_act(const Call& c)
{
    switch (c.norm->act) {
    case ZERO_ACT_SILU: return backward<T, ZERO_ACT_SILU, kFlat>(c);
    case ZERO_ACT_GELU: return backward<T, ZERO_ACT_GELU, kFlat>(c);
    default: return backward<T, ZERO_ACT_NONE, kFlat>(c);
    }
}

} // namespace

bool passes_take(const Call& c)
{
    Layout H;
    const bool flat = !rows_whole(c);
    return (!flat || line_whole(c)) && make_layout(*c.norm, flat, false, &H) && H.slabs <= kResident &&
           runs_of(H) <= 0x7FFFFFFF;
}

int64_t passes_bytes(const zero_group_norm_t& n)
{
    int64_t most = 0;
    Layout H;
    for (int way = 0; way < 4; ++way)
        if (make_layout(n, way % 2 != 0, way / 2 != 0, &H)) {
            const int64_t bytes = scratch_of(nullptr, H).bytes;
            if (bytes > most) most = bytes;
        }
    return most;
}

int passes_forward(const Call& c)
{
    if (c.norm->type == ZERO_TYPE_BF16)
        return rows_whole(c) ? forward_by_act<Bf16, false>(c) : forward_by_act<Bf16, true>(c);
    return rows_whole(c) ? forward_by_act<float, false>(c) : forward_by_act<float, true>(c);
}
int passes_backward(const Call& c)
{
    if (c.norm->type == ZERO_TYPE_BF16)
        return rows_whole(c) ? backward_by_act<Bf16, false>(c) : backward_by_act<Bf16, true>(c);
    return rows_whole(c) ? backward_by_act<float, false>(c) : backward_by_act<float, true>(c);
}

} // namespace gn
} // namespace zero

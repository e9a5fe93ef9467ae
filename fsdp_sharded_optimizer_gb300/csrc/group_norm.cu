// group_norm.cu -- group norm with an activation, channels last
// (zero_group_norm_forward), and its gradient (zero_group_norm_backward).
//
//   h = (x - mean) * rstd, z = h * weight + bias, y = act(z)
//   d = dy * act'(z), dbias = sum d, dweight = sum d h
//   dx = rstd * (d * weight - s1 - h * s2),  s1 = mean of d * weight, s2 = mean of
//   d * weight * h over the group
//
// Three ways, chosen by sizes, alignment and type:
//  - held (here): a slab of a whole sample fits the shared memory of one block, so that one
//    launch reads every value once;
//  - passes (group_norm_passes.cu): the sums of runs of rows, their join, and the result in a
//    second pass over the rows, the last ones first (they may be in the L2 still);
//  - single (group_norm_single.cu): channel by channel, for what 16-byte accesses cannot reach.
//
// Measured, bf16 with SiLU, microseconds (forward, gradient):
//                       held          passes        single
//   1 x 64 x 1280       5.8,  7.7     7.2, 11       8.3,  9.2
//   16 x 256 x 640      7.7, 12       12,  23       17,  22
//   64 x 256 x 1280     24,  61       53,  70       50,  82
//   32 x 1024 x 320     14,  32       32,  33       29,  46
//   32 x 4096 x 640     -             95, 176       196, 363
//   32 x 16384 x 320    -             184, 329      420, 820
// and where the channels fill no vectors (passes along a sample):
//   2 x 300000 x 33     -             62,  68       114, 234
//   1 x 1000000 x 15    -             82,  60       122, 271
//   32 x 5000 x 255     -             92, 131       98,  186
//   64 x 8000 x 81      -             106, 138      97,  169
//   32 x 16000 x 33     -             90,  63       43,  73
//   16 x 2000 x 201     -             59,  40       26,  40
//   64 x 1500 x 27      19,  40       37,  40       17,  21
// Passes are taken for all of those: up to 4.5 times faster over long samples and in most
// gradients, up to 2.3 times slower over many samples of few thousand rows and groups, where the
// joins of their runs cost more than the rows.
// A sample held by a team of blocks that exchange their sums through global memory (a cooperative
// launch) read every value once and took longer than two passes: 32 x 16384 x 320 216 us against
// 184, as a turn's exchange takes longer than its streaming.
#include <cmath>

#include "group_norm.cuh"

namespace zero {
namespace gn {
namespace {

// ------------------------------------------------- samples held in shared memory
// Each thread copies its own vectors there (cp.async), sums them as they lie there, and while
// it forms the results puts the block's next sample's in the places that become free.  No
// thread reads another's places.  64 x 256 x 1280 bf16 takes 24 us (3.6 TB/s): a turn's barriers
// and joins, which the other block of the SM covers only in part; the gradient 61 us (2.1 TB/s)
// with 48 bytes a vector held in the place of 16.
constexpr int kResident = 152 * 2;          // blocks at once, two an SM
constexpr int64_t kShared = 113 * 1024;     // bytes of each

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

// A thread's vector in shared memory: planes of 16 bytes a thread, one for bf16, two for fp32.
template <typename T>
constexpr int kPlanes = sizeof(T) / 2;

__device__ __forceinline__ void read_slot(const float4* p, Raw8<Bf16>& r) { r.a = *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void read_slot(const float4* p, Raw8<float>& r)
{
    r.a = p[0];
    r.b = p[kThreads];
}
__device__ __forceinline__ void write_slot(float4* p, const Raw8<Bf16>& r) { *reinterpret_cast<uint4*>(p) = r.a; }
__device__ __forceinline__ void write_slot(float4* p, const Raw8<float>& r)
{
    p[0] = r.a;
    p[kThreads] = r.b;
}

// Row k into its place; arguments as load_row's.
template <bool kFlat, typename T>
__device__ __forceinline__ void copy_row(const Layout& H, const Here& h, int k, float4* place, const T* base,
                                         int64_t sample, int64_t stride)
{
    if (kFlat && !whole<kFlat>(H, h, k)) {
        const int64_t at = h.n * sample + value_of(H, h, k);
        if (at < 0 || H.samples * sample - at < 8) { // not all of the vector is the tensor's
            Raw8<T> r = {};
            load_row<kFlat, true>(H, h, k, base, sample, stride, r);
            write_slot(place, r);
            return;
        }
    }
    const T* from = base + h.n * sample + k * H.row_groups * stride - (kFlat ? h.lead : 0);
    copy_async(place, from);
    if (sizeof(T) == 4) copy_async(place + kThreads, from + 4);
}

template <typename T, int kAct, bool kFlat>
__global__ void __launch_bounds__(kThreads, 2)
held_forward_kernel(const __grid_constant__ Layout H, const T* x, const void* __restrict__ weight,
                    const void* __restrict__ bias, int32_t param_type, float eps, T* y, float2* __restrict__ stats)
{
    extern __shared__ float4 shared[];
    float* words = reinterpret_cast<float*>(shared + H.slots * kPlanes<T> * kThreads);
    const Segments S = segments_at(H, 3, words);
    float2* group_stats = reinterpret_cast<float2*>(words + segment_words(H, 3));
    float* weights = reinterpret_cast<float*>(group_stats + H.slab_groups);
    float* biases = weights + H.width;

    const int slab = blockIdx.x % H.slabs, step = gridDim.x / H.slabs;
    const int rg = threadIdx.x / H.lanes, lane = threadIdx.x - rg * H.lanes;
    float4* mine = shared + threadIdx.x;
    const T* xp = x + rg * H.x_stride + slab * H.width + lane * 8;
    T* yp = y + rg * H.y_stride + slab * H.width + lane * 8;
    auto copy = [&](const Here& h, int k) {
        copy_row<kFlat>(H, h, k, mine + k * kPlanes<T> * kThreads, xp, H.x_sample, H.x_stride);
    };
    int n = blockIdx.x / H.slabs; // less than samples
    Here next = here_of<kFlat>(H, n, x, rg, lane, 0);
    for (int k = 0; k < next.rows; ++k) copy(next, k);
    load_params(H, slab * H.width, weight, bias, param_type, weights, biases);
    for (; n < H.samples; n += step) {
        const Here h = next;
        copies_here();
        sum_rows<kFlat, 4, T>(H, h, rg, lane, S, [&](int k, Raw8<T>& r) {
            read_slot(mine + k * kPlanes<T> * kThreads, r);
        });
        __syncthreads();
        join_groups<kFlat>(H, h.lead, S, [&](int g, float count, float mean, float m2) {
            const float2 st = make_float2(mean, rstd_of(count, m2, eps));
            group_stats[g] = st;
            if (stats) stats[static_cast<int64_t>(n) * H.groups + slab * H.slab_groups + g] = st;
        });
        __syncthreads();
        const bool more = n + step < H.samples;
        next = here_of<kFlat>(H, more ? n + step : n, x, rg, lane, 0);
        const int rows2 = more ? next.rows : 0;
        if (rg >= H.row_groups) continue;
        float2 minus_mean[4], a[4], b[4];
        forward_factors<kFlat>(H, h, lane, weights, biases, group_stats, minus_mean, a, b);
#pragma unroll 2
        for (int k = 0; k < h.rows; ++k) {
            Raw8<T> raw;
            float2 v[4];
            read_slot(mine + k * kPlanes<T> * kThreads, raw);
            dev::unpack8(raw, v);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = activated2<T, kAct>(dev::fma2(dev::add2(v[i], minus_mean[i]), a[i], b[i]));
            store_row<kFlat>(H, h, k, yp, H.y_sample, H.y_stride, v);
            if (k < rows2) copy(next, k);
        }
        for (int k = h.rows; k < rows2; ++k) copy(next, k);
    }
}

// The gradient, likewise: x is held as it is and d in fp32, in dy's place, so that the
// activation's slope is formed once.  dx == nullptr: the parameters' sums alone.
template <typename T, int kAct, bool kFlat>
__global__ void __launch_bounds__(kThreads, 2)
held_backward_kernel(const __grid_constant__ Layout H, const T* x, const T* dy, const void* __restrict__ weight,
                     const void* __restrict__ bias, int32_t param_type, const float2* __restrict__ stats, T* dx,
                     float2* __restrict__ block_sums)
{
    extern __shared__ float4 shared[];
    float4* ds = shared + H.slots * kPlanes<T> * kThreads; // two planes a row
    float* words = reinterpret_cast<float*>(ds + H.slots * 2 * kThreads);
    const ChannelSums C = channels_at(H, words);
    words += channel_words(H);
    const Segments S = segments_at(H, 2, words);
    float2* group_stats = reinterpret_cast<float2*>(words + segment_words(H, 2));
    float2* next_stats = group_stats + H.slab_groups; // they change places
    float2* group_means = next_stats + H.slab_groups;
    float* weights = reinterpret_cast<float*>(group_means + H.slab_groups);
    float* biases = weights + H.width;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int slab = blockIdx.x % H.slabs, step = gridDim.x / H.slabs;
    const int rg = threadIdx.x / H.lanes, lane = threadIdx.x - rg * H.lanes;
    float4* my_x = shared + threadIdx.x;
    float4* my_d = ds + threadIdx.x;
    const T* xp = x + rg * H.x_stride + slab * H.width + lane * 8;
    const T* dp = dy + rg * H.y_stride + slab * H.width + lane * 8;
    T* out = dx ? dx + rg * H.x_stride + slab * H.width + lane * 8 : nullptr;
    auto copy = [&](const Here& h, int k) {
        copy_row<kFlat>(H, h, k, my_x + k * kPlanes<T> * kThreads, xp, H.x_sample, H.x_stride);
        copy_row<kFlat>(H, h, k, my_d + k * 2 * kThreads, dp, H.y_sample, H.y_stride);
    };
    auto copy_stats = [&](int sample) {
        const float2* of = stats + static_cast<int64_t>(sample) * H.groups + slab * H.slab_groups;
        for (int g = threadIdx.x; g < H.slab_groups; g += kThreads) next_stats[g] = __ldg(of + g);
    };
    int n = blockIdx.x / H.slabs; // less than samples
    Here next = here_of<kFlat>(H, n, x, rg, lane, 0);
    for (int k = 0; k < next.rows; ++k) copy(next, k);
    load_params(H, slab * H.width, weight, bias, param_type, weights, biases);
    for (int c = threadIdx.x; c < H.width; c += kThreads) C.sums[c] = make_float2(0.0f, 0.0f);
    copy_stats(n);
    __syncthreads();
    bool first = true;
    for (; n < H.samples; n += step) {
        const Here h = next;
        float2* const old = group_stats;
        group_stats = next_stats;
        next_stats = old;
        float2 minus_mean[4], a[4];
        copies_here();
        if (rg < H.row_groups) {
            float2 b[4], s[4], q[4];
            forward_factors<kFlat>(H, h, lane, weights, biases, group_stats, minus_mean, a, b);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] = q[i] = make_float2(0.0f, 0.0f);
#pragma unroll 2
            for (int k = 0; k < h.rows; ++k) {
                Raw8<T> rx, rd;
                float2 v[4], d[4];
                float4* place = my_d + k * 2 * kThreads;
                read_slot(my_x + k * kPlanes<T> * kThreads, rx);
                read_slot(place, rd);
                dev::unpack8(rx, v);
                dev::unpack8(rd, d);
                form_d<T, kAct>(v, d, minus_mean, a, b);
                if (kFlat && !whole<kFlat>(H, h, k))
                    outside(H, h, k, [&](int e) { of_pair(v, e) = of_pair(d, e) = 0.0f; });
                place[0] = make_float4(d[0].x, d[0].y, d[1].x, d[1].y);
                place[kThreads] = make_float4(d[2].x, d[2].y, d[3].x, d[3].y);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[i] = dev::add2(s[i], d[i]);
                    q[i] = dev::fma2(d[i], v[i], q[i]);
                }
            }
            put_weighed<kFlat>(H, h, lane, weights, group_stats, s, q, S);
            add_channels(H, C, rg, lane, kFlat || first, s, q);
        }
        first = false;
        __syncthreads();
        if (kFlat) join_channels<kFlat>(H, C, h.lead);
        if (dx) {
            const float size = static_cast<float>(length_of(H, n)) * static_cast<float>(H.per);
            const float inv = size > 0.0f ? 1.0f / size : 0.0f;
            join_sums<kFlat>(H, h.lead, S, [&](int g, float s, float q) { group_means[g] = make_float2(s * inv, q * inv); });
            __syncthreads();
        }
        const bool more = n + step < H.samples;
        next = here_of<kFlat>(H, more ? n + step : n, x, rg, lane, 0);
        const int rows2 = more ? next.rows : 0;
        if (more) copy_stats(n + step);
        if (dx && rg < H.row_groups) {
            float2 rstd[4], s1[4], s2[4];
            result_factors<kFlat>(H, h, lane, group_stats, group_means, rstd, s1, s2);
#pragma unroll 2
            for (int k = 0; k < h.rows; ++k) {
                Raw8<T> raw;
                float2 v[4];
                read_slot(my_x + k * kPlanes<T> * kThreads, raw);
                dev::unpack8(raw, v);
                const float4* place = my_d + k * 2 * kThreads;
                const float4 lo = place[0], hi = place[kThreads];
                const float2 d[4] = {make_float2(lo.x, lo.y), make_float2(lo.z, lo.w), make_float2(hi.x, hi.y),
                                     make_float2(hi.z, hi.w)};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = dev::fma2(dev::mul2(dev::add2(v[i], minus_mean[i]), rstd[i]), s2[i],
                                     dev::fma2(d[i], a[i], s1[i]));
                store_row<kFlat>(H, h, k, out, H.x_sample, H.x_stride, v);
                if (k < rows2) copy(next, k);
            }
            for (int k = h.rows; k < rows2; ++k) copy(next, k);
        } else {
            for (int k = 0; k < rows2; ++k) copy(next, k);
        }
        __syncthreads();
    }
    if (!kFlat) join_channels<kFlat>(H, C, 0);
    for (int c = threadIdx.x; c < H.width; c += kThreads) // each by the thread that summed it
        block_sums[static_cast<int64_t>(blockIdx.x) * H.width + c] = C.sums[c];
}

__global__ void __launch_bounds__(kThreads)
sum_blocks_kernel(const __grid_constant__ Layout H, const float2* __restrict__ block_sums, int blocks, void* dweight,
                  void* dbias, int32_t grad_type)
{
    // launched while the blocks of the kernel before drain
    asm volatile("griddepcontrol.wait;" ::: "memory");
    sum_blocks_of(H, blockIdx.x, block_sums, blocks, dweight, dbias, grad_type);
}

// --------------------------------------------------------------------- host
int64_t held_words(const Layout& H, bool backward)
{
    return (backward ? channel_words(H) : 0) + segment_words(H, backward ? 2 : 3) + 2 * H.width +
           2 * H.slab_groups * (backward ? 3 : 1);
}
int64_t slot_bytes(int32_t type, bool backward)
{
    return kThreads * 16 * (type == ZERO_TYPE_F32 ? (backward ? 4 : 2) : (backward ? 3 : 1));
}

struct Plan {
    Layout H;
    int64_t grid, shared;
    bool flat;
};

// A slab of whole groups of a whole sample for each block: the widest that fits and leaves
// every resident block one, or else the narrowest that is not below 64 bytes (few samples
// then spread over more blocks).
bool make_plan(const Call& c, bool backward, Plan* plan)
{
    const zero_group_norm_t* n = c.norm;
    const bool flat = !rows_whole(c);
    if ((flat && !line_whole(c)) || n->positions * n->channels >= (int64_t(1) << 30)) return false;
    Layout H = {};
    H.lengths = c.lengths;
    H.samples = static_cast<int32_t>(n->samples);
    H.positions = static_cast<int32_t>(n->positions);
    H.channels = static_cast<int32_t>(n->channels);
    H.groups = n->groups;
    H.per = H.channels / H.groups;
    H.splits = H.repeats = H.chunks = 1;
    if (flat)
        while (H.repeats * H.channels % 8 != 0) ++H.repeats;
    const int bytes = type_bytes(n->type);
    bool found = false;
    for (int g = 1; g <= H.groups && g * H.per <= kWidth; ++g) {
        const int width = g * H.per;
        if (H.groups % g != 0 || (flat ? g != H.groups || H.repeats * width > kWidth : width % 8 != 0)) continue;
        Layout t = H;
        t.slab_groups = g;
        t.slabs = H.groups / g;
        t.width = width;
        t.lanes = H.repeats * width / 8;
        t.row_groups = kThreads / t.lanes;
        const int64_t rows = flat ? (n->positions * n->channels + 7 + 8 * t.lanes - 1) / (8 * t.lanes) : n->positions;
        const int64_t slots = rows < 1 ? 1 : (rows + t.row_groups - 1) / t.row_groups;
        const int64_t shared = held_words(t, backward) * 4 + slots * slot_bytes(n->type, backward);
        if (t.slabs > kResident || shared > kShared || (width * bytes < 64 && g != H.groups)) continue;
        if (found && static_cast<int64_t>(t.samples) * t.slabs < kResident) continue;
        t.slots = static_cast<int32_t>(slots);
        plan->H = t;
        plan->shared = shared;
        plan->flat = flat;
        found = true;
    }
    if (!found) return false;
    Layout& P = plan->H;
    P.x_sample = flat ? n->positions * n->channels : n->positions * n->x_stride;
    P.y_sample = flat ? P.x_sample : n->positions * n->y_stride;
    P.x_stride = flat ? 8 * P.lanes : n->x_stride;
    P.y_stride = flat ? 8 * P.lanes : n->y_stride;
    const int64_t units = static_cast<int64_t>(P.samples) * P.slabs, most = kResident / P.slabs * P.slabs;
    plan->grid = units < most ? units : most;
    return true;
}

template <typename T, int kAct>
int start_forward(const Call& c, const Plan& p)
{
    auto* kernel = p.flat ? held_forward_kernel<T, kAct, true> : held_forward_kernel<T, kAct, false>;
    if (!allow_shared(reinterpret_cast<const void*>(kernel), kShared)) return ZERO_ECUDA;
    return launch(false, kernel, p.grid, static_cast<size_t>(p.shared), c.stream, p.H, static_cast<const T*>(c.x),
                  c.weight, c.bias, c.norm->param_type, static_cast<float>(c.norm->eps), static_cast<T*>(c.y), c.stats);
}

template <typename T, int kAct>
int start_backward(const Call& c, const Plan& p)
{
    auto* kernel = p.flat ? held_backward_kernel<T, kAct, true> : held_backward_kernel<T, kAct, false>;
    if (!allow_shared(reinterpret_cast<const void*>(kernel), kShared)) return ZERO_ECUDA;
    return launch(false, kernel, p.grid, static_cast<size_t>(p.shared), c.stream, p.H, static_cast<const T*>(c.x),
                  static_cast<const T*>(c.dy), c.weight, c.bias, c.norm->param_type, c.stats_in,
                  static_cast<T*>(c.dx), static_cast<float2*>(c.scratch));
}

template <typename T>
int forward_by_act(const Call& c, const Plan& p)
{
    switch (c.norm->act) {
    case ZERO_ACT_SILU: return start_forward<T, ZERO_ACT_SILU>(c, p);
    case ZERO_ACT_GELU: return start_forward<T, ZERO_ACT_GELU>(c, p);
    default: return start_forward<T, ZERO_ACT_NONE>(c, p);
    }
}
template <typename T>
int backward_by_act(const Call& c, const Plan& p)
{
    switch (c.norm->act) {
    case ZERO_ACT_SILU: return start_backward<T, ZERO_ACT_SILU>(c, p);
    case ZERO_ACT_GELU: return start_backward<T, ZERO_ACT_GELU>(c, p);
    default: return start_backward<T, ZERO_ACT_NONE>(c, p);
    }
}

constexpr int64_t kMaxChannels = 16384;
constexpr int64_t kMaxCount = int64_t(1) << 30;

bool sizes_ok(int64_t samples, int64_t positions, int64_t channels, int32_t groups)
{
    return samples >= 0 && samples <= kMaxCount && positions >= 0 && positions <= kMaxCount &&
           samples * positions <= (int64_t(1) << 40) && channels >= 1 &&
           channels <= kMaxChannels && samples * channels <= (int64_t(1) << 34) && groups >= 1 &&
           channels % groups == 0;
}

// Scratch of a call of these sizes, whatever its type and alignment.
int64_t scratch_bytes_of(const zero_group_norm_t& n)
{
    int64_t most = static_cast<int64_t>(kResident) * 8 * (n.channels < kWidth ? n.channels : kWidth);
    const int64_t passes = passes_bytes(n), single = single_bytes(n);
    if (passes > most) most = passes;
    if (single > most) most = single;
    return (most + 15) / 16 * 16;
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
    if (!scratch || scratch_bytes < scratch_bytes_of(*n)) return ZERO_EINVAL;
    if (!aligned_to(weight, type_bytes(n->param_type)) ||
        !aligned_to(bias, type_bytes(n->param_type)) || !aligned_to(lengths, 4) || !aligned16(scratch))
        return ZERO_EALIGN;
    return ZERO_OK;
}

bool equally_far(const void* a, const void* b)
{
    return ((reinterpret_cast<uintptr_t>(a) ^ reinterpret_cast<uintptr_t>(b)) & 15u) == 0;
}

} // namespace

} // namespace gn
} // namespace zero

using namespace zero;

extern "C" int64_t zero_group_norm_scratch_bytes(int64_t samples, int64_t positions,
                                                 int64_t channels, int32_t groups)
{
    if (!gn::sizes_ok(samples, positions, channels, groups)) return ZERO_EINVAL;
    zero_group_norm_t n = {};
    n.samples = samples;
    n.positions = positions;
    n.channels = channels;
    n.groups = groups;
    return gn::scratch_bytes_of(n);
}

extern "C" int zero_group_norm_forward(const zero_group_norm_t* norm, const void* x,
                                       const void* weight, const void* bias,
                                       const int32_t* lengths, void* y, float* stats,
                                       void* scratch, int64_t scratch_bytes, cudaStream_t stream)
{
    const int rc = gn::check(norm, weight, bias, lengths, scratch, scratch_bytes);
    if (rc != ZERO_OK) return rc;
    if (!std::isfinite(norm->eps) || static_cast<float>(norm->eps) <= 0) return ZERO_EINVAL;
    if (norm->samples == 0) return ZERO_OK;
    if (norm->positions > 0 && (!x || !y || (x == y && norm->x_stride != norm->y_stride)))
        return ZERO_EINVAL;
    const int tb = type_bytes(norm->type);
    if (!aligned_to(x, tb) || !aligned_to(y, tb) || !aligned_to(stats, 8)) return ZERO_EALIGN;
    gn::Call c = {};
    c.norm = norm;
    c.x = x;
    c.y = y;
    c.weight = weight;
    c.bias = bias;
    c.lengths = lengths;
    c.stats = reinterpret_cast<float2*>(stats);
    c.scratch = scratch;
    c.stream = stream;
    c.aligned = aligned16(x) && aligned16(y);
    c.same_lead = gn::equally_far(x, y);
    gn::Plan p;
    if (norm->positions > 0 && gn::make_plan(c, false, &p))
        return norm->type == ZERO_TYPE_BF16 ? gn::forward_by_act<gn::Bf16>(c, p) : gn::forward_by_act<float>(c, p);
    return norm->positions > 0 && gn::passes_take(c) ? gn::passes_forward(c) : gn::single_forward(c);
}

extern "C" int zero_group_norm_backward(const zero_group_norm_t* norm, const void* x,
                                        const void* dy, const void* weight, const void* bias,
                                        const int32_t* lengths, const float* stats, void* dx,
                                        void* dweight, void* dbias, void* scratch,
                                        int64_t scratch_bytes, cudaStream_t stream)
{
    const int rc = gn::check(norm, weight, bias, lengths, scratch, scratch_bytes);
    if (rc != ZERO_OK) return rc;
    if (!float_type(norm->grad_type)) return ZERO_EINVAL;
    const bool any = norm->samples > 0 && norm->positions > 0;
    if (any && (!x || !dy || !stats || (dx == dy && norm->x_stride != norm->y_stride)))
        return ZERO_EINVAL;
    const int tb = type_bytes(norm->type), gb = type_bytes(norm->grad_type);
    if (!aligned_to(x, tb) || !aligned_to(dy, tb) || !aligned_to(dx, tb) ||
        !aligned_to(stats, 8) || !aligned_to(dweight, gb) || !aligned_to(dbias, gb))
        return ZERO_EALIGN;
    gn::Call c = {};
    c.norm = norm;
    c.x = x;
    c.dy = dy;
    c.weight = weight;
    c.bias = bias;
    c.lengths = lengths;
    c.stats_in = reinterpret_cast<const float2*>(stats);
    c.dx = dx;
    c.dweight = dweight;
    c.dbias = dbias;
    c.scratch = scratch;
    c.stream = stream;
    c.aligned = aligned16(x) && aligned16(dy) && aligned16(dx);
    c.same_lead = gn::equally_far(x, dy) && (!dx || gn::equally_far(x, dx));
    gn::Plan p;
    if (any && gn::make_plan(c, true, &p)) {
        const int status = norm->type == ZERO_TYPE_BF16 ? gn::backward_by_act<gn::Bf16>(c, p)
                                                        : gn::backward_by_act<float>(c, p);
        if (status != ZERO_OK || (!dweight && !dbias)) return status;
        return gn::launch(true, gn::sum_blocks_kernel, (norm->channels + gn::kSumChannels - 1) / gn::kSumChannels, 0,
                          stream, p.H, static_cast<const float2*>(scratch), static_cast<int>(p.grid / p.H.slabs),
                          dweight, dbias, norm->grad_type);
    }
    return any && gn::passes_take(c) ? gn::passes_backward(c) : gn::single_backward(c);
}

// tensors.cu -- gradients that do not lie in one flat buffer: the global norm
// over many tensors (zero_tensors_sqnorm), the clip and the copy into the flat
// gradient (zero_tensors_scale), and both at once (zero_tensors_clip).
//
//   norm = sqrt(sum over all tensors and elements of src^2)
//   coef = min(1, max_norm / (norm + 1e-6))
//   dst  = round(factor * src)
//
// Every tensor is cut into chunks of kChunk elements (fewer in small lists) at 16-byte boundaries of
// the tensor that the pass stores (dst) or only reads (src); a block takes the
// chunks blockIdx, blockIdx + grid, ... of the whole list, so a list of one large
// and hundreds of small tensors is spread evenly, and one launch does them all.
// The list travels in the kernel's parameters: nothing is copied to the device
// before the launch, and a captured graph holds the list itself.
//
// The norm's partial sums are those of zero_grad_sqnorm (kNormBlocks doubles), so
// both add into one scratch, and zero_clip_coef serves either.  A thread sums the
// squares of a chunk in fp32 (eight pairwise, then eight such sums) and adds that
// to an fp64 sum; eight squares whose sum leaves [1e-25, 1e30] are summed in fp64
// at once, so the norm neither overflows nor loses small gradients.
//
// What bounds it: HBM.  The gradients are needed twice, so the least is their bytes once and
// the result's, and what the L2 does not keep between the passes is read again; the scaling
// therefore starts at the end of the list, with loads that may hit.  200 tensors of 1.03 G fp32
// elements to bf16: 1,478 us, 7.0 TB/s of 10.3 GB with both reads (by evict-first loads 1,532);
// 182 of 124 M bf16: 121 us, 6.1 TB/s of 742 MB; 32 of 128 K fp32: 6.9 us, two launches (9.5
// with chunks of 16 K elements: fewer blocks, each longer).
#include "typed.cuh"
#include "zero_internal.h"

namespace zero {
namespace {

using dev::Bf16;
using dev::Raw8;

constexpr int kThreads = 256;
constexpr int kVecs = 8; // vectors of 8 elements that a thread takes of a chunk
constexpr int64_t kChunk = int64_t(kThreads) * kVecs * 8;
// Lists of fewer elements are cut into chunks of one vector a thread: more blocks, each done
// sooner.
constexpr int64_t kSmallList = int64_t(kNormBlocks) * kThreads * 8;
// A list of up to kFew tensors fits 4 KB of parameters; longer ones take the 32 KB form, and
// further launches.  The device takes as long with either; 32 tensors' call takes the host 8.5 us,
// and 11.9 in the long form.
constexpr int kFew = 120, kMany = 1000;
constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxLaunchChunks = int64_t(1) << 30;

struct Entry {
    const void* src;
    void* dst;
    int64_t n;
    int32_t first; // chunks of the entries before
    int16_t src_type, dst_type;
};
template <int kMost>
struct List {
    int32_t n, chunks;
    int64_t chunk; // elements of a chunk
    Entry e[kMost];
};

template <int kMost>
__device__ __forceinline__ int entry_of(const List<kMost>& L, int chunk)
{
    int lo = 0, hi = L.n; // the last entry whose first chunk is not behind `chunk`
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (L.e[mid].first <= chunk)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Elements between the 16-byte boundary at or before p, and p.
template <typename T>
__device__ __forceinline__ int lead(const T* p)
{
    return static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
}

__device__ __forceinline__ bool any_bits(const Raw8<Bf16>& r)
{
    return ((r.a.x | r.a.y | r.a.z | r.a.w) & 0x7FFF7FFFu) != 0;
}
__device__ __forceinline__ bool any_bits(const Raw8<float>& r)
{
    return ((__float_as_uint(r.a.x) | __float_as_uint(r.a.y) | __float_as_uint(r.a.z) |
             __float_as_uint(r.a.w) | __float_as_uint(r.b.x) | __float_as_uint(r.b.y) |
             __float_as_uint(r.b.z) | __float_as_uint(r.b.w)) &
            0x7FFFFFFFu) != 0;
}

template <typename T>
__device__ __forceinline__ void add_squares(const Raw8<T>& r, float& sum, double& wide)
{
    float x[8];
    dev::unpack8(r, x);
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = __fmaf_rn(x[2 * i], x[2 * i], x[2 * i + 1] * x[2 * i + 1]);
    const float s = (q[0] + q[1]) + (q[2] + q[3]);
    if (s >= 1e-25f && s <= 1e30f) {
        sum += s;
    } else if (any_bits(r)) { // also NaN
#pragma unroll
        for (int i = 0; i < 8; ++i) wide = fma(static_cast<double>(x[i]), static_cast<double>(x[i]), wide);
    }
}

// The squares of chunk `local` of one tensor.
template <typename T>
__device__ __forceinline__ void chunk_squares(const T* src, int64_t n, int64_t local, int64_t chunk, double& wide)
{
    const int64_t head = lead(src), end = n + head;
    const T* base = src - head;
    const int64_t lo = local * chunk, hi = lo + chunk < end ? lo + chunk : end;
    float sum = 0.0f;
    if (lo >= head && hi == lo + kChunk) {
        constexpr int kAhead = sizeof(T) == 2 ? kVecs : kVecs / 2;
        const T* p = base + lo + threadIdx.x * 8;
#pragma unroll
        for (int k = 0; k < kVecs; k += kAhead) {
            Raw8<T> r[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) dev::load_raw8(p + (k + i) * kThreads * 8, r[i]);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) add_squares(r[i], sum, wide);
        }
    } else {
        for (int64_t at = lo + threadIdx.x * 8; at < hi; at += kThreads * 8) {
            if (at >= head && at + 8 <= end) {
                Raw8<T> r;
                dev::load_raw8(base + at, r);
                add_squares(r, sum, wide);
            } else {
                for (int64_t i = at; i < at + 8; ++i)
                    if (i >= head && i < end) {
                        const double x = dev::load1(base + i);
                        wide = fma(x, x, wide);
                    }
            }
        }
    }
    wide += static_cast<double>(sum);
}

// Thread 0 gets the sum over the block, in a fixed order.
__device__ __forceinline__ double block_sum(double d)
{
    __shared__ double warps[kThreads / 32];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) d += __shfl_down_sync(0xFFFFFFFFu, d, off);
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = d;
    __syncthreads();
    double total = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < kThreads / 32; ++w) total += warps[w];
    return total;
}

template <int kMost>
__global__ void __launch_bounds__(kThreads)
sqnorm_kernel(const __grid_constant__ List<kMost> L, int accumulate, double* __restrict__ partials)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    double wide = 0.0;
    for (int c = blockIdx.x; c < L.chunks; c += gridDim.x) {
        const Entry& e = L.e[entry_of(L, c)];
        if (e.src_type == ZERO_TYPE_BF16)
            chunk_squares(static_cast<const Bf16*>(e.src), e.n, c - e.first, L.chunk, wide);
        else
            chunk_squares(static_cast<const float*>(e.src), e.n, c - e.first, L.chunk, wide);
    }
    const double b = block_sum(wide);
    if (threadIdx.x == 0) {
        partials[blockIdx.x] = (accumulate ? partials[blockIdx.x] : 0.0) + b;
        if (!accumulate)
            for (int i = blockIdx.x + gridDim.x; i < kNormBlocks; i += gridDim.x) partials[i] = 0.0;
    }
}

template <typename In, typename Out>
__device__ __forceinline__ void scale_vec(const In* s, Out* d, float factor, bool wide_in)
{
    float x[8];
    if (wide_in) {
        Raw8<In> r;
        dev::stream_raw8(s, r);
        dev::unpack8(r, x);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = dev::load1(s + i);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= factor;
    dev::store8_stream(d, x);
}

// Chunk `local` of one tensor, cut at 16-byte boundaries of dst.
template <typename In, typename Out>
__device__ __forceinline__ void chunk_scale(const In* src, Out* dst, int64_t n, int64_t local,
                                            int64_t chunk, float factor)
{
    const int64_t head = lead(dst), end = n + head;
    const In* from = src - head;
    Out* to = dst - head;
    const bool wide_in = (reinterpret_cast<uintptr_t>(from) & 15u) == 0;
    const int64_t lo = local * chunk, hi = lo + chunk < end ? lo + chunk : end;
    if (wide_in && lo >= head && hi == lo + kChunk) {
        constexpr int kAhead = sizeof(In) == 2 ? kVecs : kVecs / 2;
        const int64_t at = lo + threadIdx.x * 8;
#pragma unroll
        for (int k = 0; k < kVecs; k += kAhead) {
            Raw8<In> r[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                dev::load_raw8(from + at + (k + i) * kThreads * 8, r[i]);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                float x[8];
                dev::unpack8(r[i], x);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] *= factor;
                dev::store8_stream(to + at + (k + i) * kThreads * 8, x);
            }
        }
        return;
    }
    for (int64_t at = lo + threadIdx.x * 8; at < hi; at += kThreads * 8) {
        if (at >= head && at + 8 <= end) {
            scale_vec(from + at, to + at, factor, wide_in);
        } else {
            for (int64_t i = at; i < at + 8; ++i)
                if (i >= head && i < end) dev::store1(to + i, dev::load1(from + i) * factor);
        }
    }
}

// partials != nullptr: the coefficient is formed from them by every block, in
// zero_clip_coef's order, and norm_coef is written; otherwise norm_coef[1] is
// read, where there is one.
template <int kMost>
__global__ void __launch_bounds__(kThreads)
scale_kernel(const __grid_constant__ List<kMost> L, float scale,
             const double* __restrict__ partials, int n_partials, double max_norm,
             float* __restrict__ norm_coef)
{
    __shared__ float coef;
    // launched while the norm pass drains
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float factor = scale;
    if (partials) {
        double s = 0.0;
        for (int i = threadIdx.x; i < n_partials; i += kThreads) s += partials[i];
        const double total = block_sum(s);
        if (threadIdx.x == 0) {
            const double norm = sqrt(total);
            double c = max_norm / (norm + 1e-6);
            if (c > 1.0) c = 1.0;
            coef = static_cast<float>(c);
            if (blockIdx.x == 0) {
                norm_coef[0] = static_cast<float>(norm);
                norm_coef[1] = static_cast<float>(c);
            }
        }
        __syncthreads();
        factor *= coef;
    } else if (norm_coef) {
        factor *= norm_coef[1];
    }
    // from the end of the list: what the norm pass read last may be in the L2 still
    for (int c = L.chunks - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= gridDim.x) {
        const Entry& e = L.e[entry_of(L, c)];
        if (e.src == e.dst && factor == 1.0f) continue; // in place, nothing changes
        const int64_t local = c - e.first;
        if (e.src_type == ZERO_TYPE_BF16) {
            const auto* s = static_cast<const Bf16*>(e.src);
            if (e.dst_type == ZERO_TYPE_BF16)
                chunk_scale(s, static_cast<Bf16*>(e.dst), e.n, local, L.chunk, factor);
            else
                chunk_scale(s, static_cast<float*>(e.dst), e.n, local, L.chunk, factor);
        } else {
            const auto* s = static_cast<const float*>(e.src);
            if (e.dst_type == ZERO_TYPE_BF16)
                chunk_scale(s, static_cast<Bf16*>(e.dst), e.n, local, L.chunk, factor);
            else
                chunk_scale(s, static_cast<float*>(e.dst), e.n, local, L.chunk, factor);
        }
    }
}

// --------------------------------------------------------------------- host
int check_tensors(const zero_tensor_t* t, int64_t n, bool with_dst)
{
    if (n < 0 || n > (int64_t(1) << 30) || (n > 0 && !t)) return ZERO_EINVAL;
    bool aligned = true;
    for (int64_t i = 0; i < n; ++i) {
        if (t[i].n < 0 || t[i].n > kMaxElems || !float_type(t[i].src_type)) return ZERO_EINVAL;
        if (with_dst && (!float_type(t[i].dst_type) ||
                         (t[i].src == t[i].dst && t[i].src && t[i].src_type != t[i].dst_type)))
            return ZERO_EINVAL;
        if (t[i].n == 0) continue;
        if (!t[i].src || (with_dst && !t[i].dst)) return ZERO_EINVAL;
        aligned = aligned && aligned_to(t[i].src, type_bytes(t[i].src_type)) &&
                  (!with_dst || aligned_to(t[i].dst, type_bytes(t[i].dst_type)));
    }
    return aligned ? ZERO_OK : ZERO_EALIGN;
}

int64_t chunks_of(const zero_tensor_t& t, bool by_dst, int64_t chunk)
{
    const uintptr_t p = reinterpret_cast<uintptr_t>(by_dst ? t.dst : t.src);
    const int64_t head = static_cast<int64_t>(p & 15u) / type_bytes(by_dst ? t.dst_type : t.src_type);
    return (t.n + head + chunk - 1) / chunk;
}

// Elements of a chunk, for a whole list: the order of the sums goes by it.
int64_t chunk_of(const zero_tensor_t* t, int64_t n)
{
    int64_t all = 0;
    for (int64_t i = 0; i < n && all < kSmallList; ++i) all += t[i].n;
    return all < kSmallList ? kThreads * 8 : kChunk;
}

// Fills L from tensor `at` on; returns the first tensor that no longer fits.
template <int kMost>
int64_t fill(List<kMost>& L, const zero_tensor_t* t, int64_t n, int64_t at, bool by_dst)
{
    L.n = L.chunks = 0;
    for (; at < n && L.n < kMost; ++at) {
        if (t[at].n == 0) continue;
        const int64_t c = chunks_of(t[at], by_dst, L.chunk);
        if (L.n > 0 && L.chunks + c > kMaxLaunchChunks) break;
        L.e[L.n++] = {t[at].src, t[at].dst, t[at].n, L.chunks, static_cast<int16_t>(t[at].src_type),
                      static_cast<int16_t>(by_dst ? t[at].dst_type : 0)};
        L.chunks += static_cast<int32_t>(c);
    }
    return at;
}

// Adds the squares of all tensors into the partials; *used: how many of them the
// launches wrote with anything but zero.
template <int kMost>
int launch_sqnorm(const zero_tensor_t* t, int64_t n, int accumulate, double* partials,
                  cudaStream_t stream, int* used)
{
    List<kMost> L;
    L.chunk = chunk_of(t, n);
    int64_t at = 0;
    *used = 0;
    do {
        at = fill(L, t, n, at, false);
        if (L.n == 0 && accumulate) break;
        const int grid = L.chunks < 1 ? 1 : L.chunks < kNormBlocks ? L.chunks : kNormBlocks;
        sqnorm_kernel<kMost><<<grid, kThreads, 0, stream>>>(L, accumulate, partials);
        const int rc = cuda_status(cudaGetLastError());
        if (rc != ZERO_OK) return rc;
        accumulate = 1;
        if (grid > *used) *used = grid;
    } while (at < n);
    return ZERO_OK;
}

template <int kMost>
int launch_scale(const zero_tensor_t* t, int64_t n, float scale, const double* partials,
                 int n_partials, double max_norm, float* norm_coef, cudaStream_t stream)
{
    List<kMost> L;
    L.chunk = chunk_of(t, n);
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = partials ? 1 : 0;
    int64_t at = 0;
    bool first = true;
    do {
        at = fill(L, t, n, at, true);
        if (L.n == 0 && !(first && partials)) break; // the norm is written without tensors too
        const int blocks = persistent_blocks(reinterpret_cast<const void*>(scale_kernel<kMost>),
                                             kThreads, 0);
        if (blocks < 1) return ZERO_ECUDA;
        const int grid = L.chunks < 1 ? 1 : L.chunks < blocks ? L.chunks : blocks;
        cfg.gridDim = dim3(static_cast<unsigned>(grid));
        const int rc = cuda_status(cudaLaunchKernelEx(&cfg, scale_kernel<kMost>, L, scale, partials,
                                                      n_partials, max_norm, norm_coef));
        if (rc != ZERO_OK) return rc;
        cfg.numAttrs = 0;
        first = false;
    } while (at < n);
    return ZERO_OK;
}

} // namespace
} // namespace zero

using namespace zero;

extern "C" int zero_tensors_sqnorm(const zero_tensor_t* tensors, int64_t n_tensors,
                                   int32_t accumulate, double* scratch, int64_t scratch_bytes,
                                   cudaStream_t stream)
{
    if (!scratch || scratch_bytes < kNormScratchBytes || (accumulate != 0 && accumulate != 1))
        return ZERO_EINVAL;
    const int rc = check_tensors(tensors, n_tensors, false);
    if (rc != ZERO_OK) return rc;
    if (!aligned16(scratch)) return ZERO_EALIGN;
    int used;
    return n_tensors <= kFew
               ? launch_sqnorm<kFew>(tensors, n_tensors, accumulate, scratch, stream, &used)
               : launch_sqnorm<kMany>(tensors, n_tensors, accumulate, scratch, stream, &used);
}

extern "C" int zero_tensors_scale(const zero_tensor_t* tensors, int64_t n_tensors, double scale,
                                  const float* norm_coef, cudaStream_t stream)
{
    const float s = static_cast<float>(scale);
    if (!std::isfinite(s)) return ZERO_EINVAL;
    const int rc = check_tensors(tensors, n_tensors, true);
    if (rc != ZERO_OK) return rc;
    if (!aligned16(norm_coef)) return ZERO_EALIGN;
    auto* nc = const_cast<float*>(norm_coef); // read only, without partials
    return n_tensors <= kFew
               ? launch_scale<kFew>(tensors, n_tensors, s, nullptr, 0, 1.0, nc, stream)
               : launch_scale<kMany>(tensors, n_tensors, s, nullptr, 0, 1.0, nc, stream);
}

extern "C" int zero_tensors_clip(const zero_tensor_t* tensors, int64_t n_tensors, double max_norm,
                                 float* norm_coef, double* scratch, int64_t scratch_bytes,
                                 cudaStream_t stream)
{
    if (!scratch || scratch_bytes < kNormScratchBytes || !norm_coef || !(max_norm > 0) ||
        !std::isfinite(max_norm))
        return ZERO_EINVAL;
    int rc = check_tensors(tensors, n_tensors, true);
    if (rc != ZERO_OK) return rc;
    if (!aligned16(scratch) || !aligned16(norm_coef)) return ZERO_EALIGN;
    int used;
    if (n_tensors <= kFew) {
        rc = launch_sqnorm<kFew>(tensors, n_tensors, 0, scratch, stream, &used);
        return rc != ZERO_OK ? rc
                             : launch_scale<kFew>(tensors, n_tensors, 1.0f, scratch, used, max_norm,
                                                  norm_coef, stream);
    }
    rc = launch_sqnorm<kMany>(tensors, n_tensors, 0, scratch, stream, &used);
    return rc != ZERO_OK ? rc
                         : launch_scale<kMany>(tensors, n_tensors, 1.0f, scratch, used, max_norm,
                                               norm_coef, stream);
}

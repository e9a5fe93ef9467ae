// distill.cu -- distillation from a teacher's top logits: the loss of each row
// (zero_distill_forward), and the loss with the gradient of the student's
// logits (zero_distill_forward_backward).
//
// For a row with student logits s[0..V) and the teacher's K largest logits t
// at the ids i (entries whose id lies outside [0, V) are not counted):
//
//   p_k  = softmax(t / tau)_k over the counted entries
//   q    = softmax(s / tau),  q1 = softmax(s)
//   kl   = tau^2 * sum_k p_k (log p_k - log q[i_k])
//   ce   = -log q1[label]
//   ds_j = w * ( kl_weight * tau * (q_j - sum_{k: i_k = j} p_k)
//              + ce_weight * (q1_j - [j = label]) )
//
// Both softmaxes have the same maximum m, so one pass over the row keeps it
// and both sums of exponentials, rescaled when m grows.  Everything is fp32.
// Read and written: the logits once and the gradient once, where the row stays
// on the chip between the two (row_kernel); HBM bounds it as long as a logit
// costs about ten instructions, an exponential per pass among them.
//
// Measured (device time, one GB300): 4096 x 32000 fp32, soft targets only, 164 us,
// 6.4 TB/s; 8192 x 32000 bf16 at temperature 1 177 us, 5.9 TB/s, at 1.5 with
// labels 213 us (two exponentials a logit and pass); 8191 x 50257 bf16 at
// temperature 2 308 us, 5.4 TB/s (100 KB a row: two blocks to an SM, whose
// phases do not hide one another fully); 2000 x 131072 bf16 193 us, 5.4 TB/s; the loss
// alone of 8192 x 32000 bf16 95-96 us, 5.5 TB/s.  Reading the row twice instead
// (distill_kernel, for rows that no cluster holds) took 255, 553 and 212 us for the
// first, third and last of the four that a block or two hold; 200 x 800003 takes 304 us.
//
//   kl = tau * ( sum_k p_k ((t_k - tm) - (s_ik - so)) + m - so ) + tau^2 * (log Z - log Zt)
// with Zt the teacher's sum and so the student's largest logit at a counted entry:
// every block of a row can form the sum about it before it knows the row's maximum m,
// and neither so - s_ik nor m - so is negative, so that nothing cancels, however far
// below m the logits of a block's own part lie.  One block alone takes so = m.
#include "exchange.cuh"
#include "typed.cuh"
#include "zero_internal.h"

namespace zero {
namespace {

using dev::Bf16;
using dev::kMaxRanks;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTop = 1024;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// kl of a row from the sum of e_k ((t_k - tm) - (s_ik - so)), in units that keep kMaxTop
// terms of any finite size in range, the teacher's sum zt, m - so and log Z.  Nothing is
// divided by the temperature: a masked logit of the type's lowest value would overflow.
constexpr float kCrossUnit = 1.0f / kMaxTop;
__device__ __forceinline__ float kl_of(float tau, float cross, float zt, float above, float log_z)
{
    return fmaf(cross / zt, tau / kCrossUnit, fmaf(tau * tau, log_z - logf(zt), tau * above));
}

struct Args {
    const void *logits, *teacher, *ids, *labels;
    const float* row_weight;
    float *ce, *kl;
    void* dlogits;
    int64_t rows, vocab, stride, dstride;
    int32_t top, teacher_type, id_type, label_type;
    float tau, ce_weight, kl_weight;
};

__device__ __forceinline__ float block_max(float v, float* red)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) v = fmaxf(v, red[w]);
    return v;
}
__device__ __forceinline__ float block_sum(float v, float* red)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
    for (int w = 0; w < kWarps; ++w) v += red[w];
    return v;
}

// Calls f(index, values, count) over a row of n elements at p: single elements
// up to the first 16-byte boundary, vectors of 8, single elements.
template <typename T, typename F>
__device__ __forceinline__ void over_row(const T* p, int64_t n, F f)
{
    const int64_t mis = (reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T);
    const int64_t lead = mis == 0 ? 0 : 16 / static_cast<int64_t>(sizeof(T)) - mis;
    const int64_t head = lead < n ? lead : n;
    const int64_t body = (n - head) / 8;
    for (int64_t i = threadIdx.x; i < body; i += kThreads) {
        float x[8];
        dev::load_vec<8>(p + head + 8 * i, x);
        f(head + 8 * i, x);
    }
    float x[1];
    for (int64_t i = threadIdx.x; i < head; i += kThreads) {
        x[0] = dev::load1(p + i);
        f(i, x);
    }
    for (int64_t i = head + 8 * body + threadIdx.x; i < n; i += kThreads) {
        x[0] = dev::load1(p + i);
        f(i, x);
    }
}

template <typename T, bool kGrad>
__global__ void __launch_bounds__(kThreads)
distill_kernel(const Args A)
{
    __shared__ float red[kWarps];
    __shared__ float top_p[kMaxTop], top_s[kMaxTop]; // probabilities; the student's logits there
    __shared__ int32_t top_id[kMaxTop];              // -1: not counted
    const int tid = threadIdx.x;
    const float inv_tau = 1.0f / A.tau;
    const float c2 = kLog2e * inv_tau;
    for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x) {
        const T* s = static_cast<const T*>(A.logits) + row * A.stride;
        T* ds = static_cast<T*>(A.dlogits) + row * A.dstride;
        const float w = A.row_weight ? A.row_weight[row] : 1.0f;
        if (w == 0.0f) { // a masked row: not read
            if (tid == 0) {
                A.ce[row] = 0.0f;
                A.kl[row] = 0.0f;
            }
            if (kGrad)
                for (int64_t j = tid; j < A.vocab; j += kThreads) dev::store1(ds + j, 0.0f);
            continue;
        }
        __syncthreads(); // the last row's use of top_*
        float tm = -INFINITY;
        for (int k = tid; k < A.top; k += kThreads) {
            const int64_t id = dev::load_index(A.ids, A.id_type, row * A.top + k);
            const bool counted = id >= 0 && id < A.vocab;
            float t[1] = {-INFINITY};
            if (counted) {
                dev::load_any<1>(A.teacher, A.teacher_type, row * A.top + k, t);
                tm = fmaxf(tm, t[0]);
            }
            top_id[k] = counted ? static_cast<int32_t>(id) : -1;
            top_p[k] = t[0];
            top_s[k] = counted ? dev::load1(s + id) : 0.0f;
        }
        const int64_t label = A.labels ? dev::load_index(A.labels, A.label_type, row) : -1;
        const bool labelled = label >= 0 && label < A.vocab;
        const float s_label = labelled ? dev::load1(s + label) : 0.0f;

        float m = -INFINITY, z1 = 0.0f, z2 = 0.0f;
        over_row(s, A.vocab, [&](int64_t, auto& x) {
            constexpr int n = sizeof(x) / sizeof(float);
            float mx = x[0];
#pragma unroll
            for (int e = 1; e < n; ++e) mx = fmaxf(mx, x[e]);
            if (mx > m) {
                z1 *= exp2_approx((m - mx) * kLog2e);
                z2 *= exp2_approx((m - mx) * c2);
                m = mx;
            }
            const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
            for (int e = 0; e < n; ++e) {
                z1 += exp2_approx((x[e] - base) * kLog2e);
                z2 += exp2_approx((x[e] - base) * c2);
            }
        });
        const float row_m = block_max(m, red);
        const float base = row_m == -INFINITY ? 0.0f : row_m;
        const float own = m == -INFINITY ? 0.0f : m;
        const bool none = m == -INFINITY;
        z1 = block_sum(none ? z1 : z1 * exp2_approx((own - base) * kLog2e), red);
        z2 = block_sum(none ? z2 : z2 * exp2_approx((own - base) * c2), red);
        tm = block_max(tm, red);
        const float tbase = tm == -INFINITY ? 0.0f : tm;
        float zt = 0.0f, cross = 0.0f;
        for (int k = tid; k < A.top; k += kThreads) {
            const float e = exp2_approx((top_p[k] - tbase) * c2); // 0 where not counted
            zt += e;
            if (e != 0.0f) cross = fmaf(e * kCrossUnit, (top_p[k] - tbase) - (top_s[k] - base), cross);
            top_p[k] = e;
        }
        zt = block_sum(zt, red);
        cross = block_sum(cross, red);
        // a row whose logits are all -inf has no distribution, a teacher whose
        // counted entries are all -inf (or none) has none either; a NaN is neither
        const bool empty = z1 == 0.0f;
        const bool has_top = zt != 0.0f && !empty;
        const bool has_label = labelled && !empty;
        if (tid == 0) {
            A.ce[row] = has_label ? logf(z1) - (s_label - base) : 0.0f;
            A.kl[row] = has_top ? kl_of(A.tau, cross, zt, 0.0f, logf(z2)) : 0.0f;
        }
        if constexpr (kGrad) {
            const float a1 = has_label ? w * A.ce_weight / z1 : 0.0f;
            const float a2 = has_top ? w * A.kl_weight * A.tau / z2 : 0.0f;
            const float hit = has_label ? w * A.ce_weight : 0.0f;
            const float share = has_top ? w * A.kl_weight * A.tau / zt : 0.0f;
            auto dense = [&](float x) {
                float g = 0.0f;
                if (has_label) g = a1 * exp2_approx((x - base) * kLog2e);
                if (has_top) g = fmaf(a2, exp2_approx((x - base) * c2), g);
                return g;
            };
            over_row(s, A.vocab, [&](int64_t j, auto& x) {
                constexpr int n = sizeof(x) / sizeof(float);
                bool wide = false;
#pragma unroll
                for (int e = 0; e < n; ++e) x[e] = dense(x[e]);
                if constexpr (n == 8) {
                    wide = (reinterpret_cast<uintptr_t>(ds + j) & 15) == 0;
                    if (wide) dev::store8(ds + j, x);
                }
                if (!wide) {
#pragma unroll
                    for (int e = 0; e < n; ++e) dev::store1(ds + j + e, x[e]);
                }
            });
            __syncthreads(); // before the teacher's entries are written over
            bool label_in_top = false;
            for (int k = tid; k < A.top; k += kThreads) {
                const int32_t id = top_id[k];
                if (id < 0) continue;
                bool first = true; // the first entry of an id writes for all of them
                float p = 0.0f;
                for (int q = 0; q < A.top; ++q) {
                    if (top_id[q] != id) continue;
                    if (q < k) first = false;
                    p += top_p[q];
                }
                if (labelled && id == label) label_in_top = true;
                if (!first) continue;
                float g = dense(top_s[k]);
                g = fmaf(-share, p, g);
                if (id == label) g -= hit;
                dev::store1(ds + id, g);
            }
            if (!__syncthreads_or(label_in_top) && has_label && tid == 0)
                dev::store1(ds + label, dense(s_label) - hit);
        }
    }
}

// ------------------------------------------------ the row stays on the chip
// One cluster of `ranks` blocks per row; rank r holds the row's r-th part in
// shared memory, as the 16-byte pieces of memory that it lies in (a row may
// start at any element: the first and the last piece are then partly outside,
// read element by element, and hold -inf there).  A thread owns the same slots
// for all rows and is the only one that reads or fills them, so it asks for
// the next row's piece (cp.async) as soon as it has used this row's for the
// last time, and no barrier stands between a row's loads and the one before.
constexpr int kMaxRowWarps = 16;

// How many exponentials a logit takes.
//   kOne     one: temperature 1, or no labels
//   kSquare  temperature 2: e^(x/2), and its square
//   kFourth  temperature 4: e^(x/4), and its square's square
//   kTwo     two
enum Exps { kOne = 0, kSquare = 1, kFourth = 2, kTwo = 3 };

// e^x of e^(x/T), where a product gives it.
template <int kExps>
__device__ __forceinline__ float power_of(float e)
{
    return kExps == kSquare ? e * e : (e * e) * (e * e);
}

template <typename T>
struct Piece { // 16 bytes of a row
    static constexpr int kElems = 16 / sizeof(T), kPairs = kElems / 2;
};
__device__ __forceinline__ void unpack_piece(const uint4& w, float2 (&x)[4], Bf16)
{
    x[0] = make_float2(dev::bf16_lo(w.x), dev::bf16_hi(w.x));
    x[1] = make_float2(dev::bf16_lo(w.y), dev::bf16_hi(w.y));
    x[2] = make_float2(dev::bf16_lo(w.z), dev::bf16_hi(w.z));
    x[3] = make_float2(dev::bf16_lo(w.w), dev::bf16_hi(w.w));
}
__device__ __forceinline__ void unpack_piece(const uint4& w, float2 (&x)[2], float)
{
    x[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
    x[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
}
__device__ __forceinline__ uint4 pack_piece(const float2 (&x)[4], Bf16)
{
    return make_uint4(dev::cvt_bf16x2(x[0].x, x[0].y), dev::cvt_bf16x2(x[1].x, x[1].y),
                      dev::cvt_bf16x2(x[2].x, x[2].y), dev::cvt_bf16x2(x[3].x, x[3].y));
}
__device__ __forceinline__ uint4 pack_piece(const float2 (&x)[2], float)
{
    return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x),
                      __float_as_uint(x[1].y));
}
// The largest element (a NaN is passed over).
__device__ __forceinline__ float piece_max(const uint4& w, Bf16)
{
    uint32_t a, b;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(w.x), "r"(w.y));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(w.z), "r"(w.w));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
    return fmaxf(dev::bf16_lo(a), dev::bf16_hi(a));
}
__device__ __forceinline__ float piece_max(const uint4& w, float)
{
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)),
                 fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
}
__device__ __forceinline__ uint4 lowest_piece(Bf16)
{
    return make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
}
__device__ __forceinline__ uint4 lowest_piece(float)
{
    return make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
}
__device__ __forceinline__ float2 exp2_pair(float2 a)
{
    return make_float2(exp2_approx(a.x), exp2_approx(a.y));
}

__device__ __forceinline__ float warp_max(float x) // a NaN is passed over
{
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
// Sums of 4 values over the warp: lane 8 i (and the 7 that follow) get value
// i's.  A lane keeps half of the values at each of the first two steps.
__device__ __forceinline__ float warp_sum4(const float (&v)[4], int lane)
{
    constexpr uint32_t kAll = 0xFFFFFFFFu;
    const bool up = lane & 16, odd = lane & 8;
    const float a = (up ? v[2] : v[0]) + __shfl_xor_sync(kAll, up ? v[0] : v[2], 16);
    const float b = (up ? v[3] : v[1]) + __shfl_xor_sync(kAll, up ? v[1] : v[3], 16);
    float x = (odd ? b : a) + __shfl_xor_sync(kAll, odd ? a : b, 8);
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) x += __shfl_xor_sync(kAll, x, off);
    return x;
}

// A rank's part of a row: slots [0, n), of which [from, to) lie wholly inside
// the row; element i of slot j is column lo + j * kElems + i.
template <typename T>
struct Part {
    const T* row;
    int64_t lo;
    int n, from, to;

    __device__ __forceinline__ Part(const T* p, int64_t vocab, int64_t first_piece, int slots)
    {
        constexpr int kE = Piece<T>::kElems;
        const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
        row = p;
        lo = first_piece * kE - mis;
        const int64_t left = vocab - lo; // elements from slot 0 to the row's end
        const int64_t all = left <= 0 ? 0 : (left + kE - 1) / kE;
        n = static_cast<int>(all < slots ? all : slots);
        from = lo < 0 ? 1 : 0;
        const int64_t whole = left <= 0 ? 0 : left / kE;
        to = static_cast<int>(whole < n ? whole : n);
    }
};
__device__ __forceinline__ void fetch16(uint32_t to, const void* from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
// Asks for slot j where it lies inside the row.
template <typename T>
__device__ __forceinline__ void fetch_whole(uint32_t part, const Part<T>& p, int j)
{
    if (j >= p.from && j < p.to)
        fetch16(part + 16u * j, p.row + p.lo + static_cast<int64_t>(j) * Piece<T>::kElems);
}
// Fills the slots at the row's ends: at most one before `from`, one from `to`.
template <int kThreadsOf, typename T>
__device__ __forceinline__ void fetch_ends(uint4* part, const Part<T>& p, int64_t vocab)
{
    constexpr int kE = Piece<T>::kElems;
    auto fill = [&](int j) {
        if (j % kThreadsOf != static_cast<int>(threadIdx.x)) return; // its owner
        part[j] = lowest_piece(T());
        T* e = reinterpret_cast<T*>(part + j);
        const int64_t at = p.lo + static_cast<int64_t>(j) * kE;
        for (int i = 0; i < kE; ++i)
            if (at + i >= 0 && at + i < vocab) e[i] = p.row[at + i];
    };
    if (p.from == 1 && p.n > 0) fill(0);
    if (p.to < p.n && p.to >= p.from) fill(p.to);
}

struct RowShared {
    float most[2][kMaxRowWarps]; // maxima of the block's warps: logits, teacher
    float sum[4][kMaxRowWarps];  // sums of the block's warps
    dev::Words words;            // every rank's maximum and sums
};

// 2^(x c - m c) for a thread's maximum m so far.  The reference m c is rounded once
// and the product inside the fma is not, so the terms agree to rounding; what the
// reference was off by, at most 1, is taken out of the sum's logarithm.  Where |m c|
// is above 2^24 (a mask value, mostly; or m is -inf) it would be off by any amount, or
// out of range: there the terms are only kept finite, and count for nothing.  A
// thread's sum is used, times its factor, where the row's maximum is below half of
// that, and then each of those logits is at least 2^23 below it.
constexpr float kFar = 16777216.0f;
struct Scale {
    float c, ref;
    bool far;
    __device__ __forceinline__ Scale(float m, float factor)
    {
        far = fabsf(m) * factor > kFar;
        c = far ? 0x1p-126f : factor;
        ref = far ? 0.0f : m * factor;
    }
    __device__ __forceinline__ float2 exp2(float2 x) const
    {
        return exp2_pair(dev::fma2(x, dev::pair(c), dev::pair(-ref)));
    }
    // the factor that takes a sum relative to this to one relative to `ref`
    __device__ __forceinline__ float to(float ref_there) const
    {
        return far ? 0.0f : exp2_approx(ref - ref_there);
    }
};

// The same for the maximum of a block's part or of the row.  Where |m c| is above
// 2^23 (far) the terms are 2^((x - m) c), x - m exact wherever that is not 0: an
// operation more, in loops of their own, as in those that all rows go through it costs
// registers (5 x 50257 fp32 loss 5.80 us, so 5.65; 8192 x 32000 at temperature 1.5 220
// and 214).  A row without any logit that is not masked takes longer for it (8192 x
// 32000 bf16 279 us for 179, its loss 186 for 99); one with a masked part does not.
struct RowScale {
    float m, c, ref;
    bool far;
    __device__ __forceinline__ RowScale(float most, float factor)
    {
        m = most == -INFINITY ? 0.0f : most; // nothing above -inf: every term is 0
        c = factor;
        far = fabsf(m) * factor > kFar / 2;
        ref = far ? 0.0f : m * factor;
    }
    __device__ __forceinline__ float2 exp2(float2 x) const // where not far
    {
        return exp2_pair(dev::fma2(x, dev::pair(c), dev::pair(-ref)));
    }
    __device__ __forceinline__ float exp2_any(float x) const
    {
        return exp2_approx(fmaf(x - (far ? m : 0.0f), c, -ref));
    }
    __device__ __forceinline__ float off() const { return far ? 0.0f : fmaf(m, c, -ref); }
    // the factor that takes a sum relative to this to one relative to `there`
    __device__ __forceinline__ float to(const RowScale& there) const
    {
        return exp2_approx(fmaf(m - there.m, c, there.off() - off()));
    }
    // log of the sum of the terms, each to the power `power`, relative to m
    __device__ __forceinline__ float log_of(float sum, int power = 1) const
    {
        return fmaf(off(), -kLn2 * power, logf(sum));
    }
};

// The sums of a part of a row with a far maximum m, read again (from the L2, mostly):
// without a gradient, its place on the chip has been given to the next row.
template <typename T>
__device__ __noinline__ float2 far_sums(const Part<T> p, int64_t vocab, float m, float c1, float c2)
{
    constexpr int kE = Piece<T>::kElems, kBatch = 4;
    const T* at = p.row + p.lo;
    const int threads = static_cast<int>(blockDim.x), tid = static_cast<int>(threadIdx.x);
    float2 z = make_float2(0.0f, 0.0f);
    auto add = [&](float x) {
        z.x += exp2_approx((x - m) * c1);
        z.y += exp2_approx((x - m) * c2);
    };
    for (int j = p.from + tid; j < p.to; j += kBatch * threads) {
        uint4 raw[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            raw[u] = j + u * threads < p.to
                         ? *reinterpret_cast<const uint4*>(at + static_cast<int64_t>(j + u * threads) * kE)
                         : lowest_piece(T());
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            float2 x[Piece<T>::kPairs];
            unpack_piece(raw[u], x, T());
#pragma unroll
            for (int e = 0; e < Piece<T>::kPairs; ++e) {
                add(x[e].x);
                add(x[e].y);
            }
        }
    }
    // what lies in the pieces at the row's ends: one before `from`, one from `to`
    const int whole = p.to > p.from ? p.to : p.from;
    for (int i = tid; i < 2 * kE; i += threads) {
        const int64_t col = p.lo + (i < kE ? i : static_cast<int64_t>(whole) * kE + i - kE);
        const bool here = i < kE ? p.from == 1 && p.n > 0 && col >= 0 : whole < p.n;
        if (here && col < vocab) add(dev::load1(p.row + col));
    }
    return z;
}

template <typename T, bool kGrad, int kExps, int kThreadsOf>
__global__ void __launch_bounds__(kThreadsOf, kThreadsOf == 128 ? 5 : kThreadsOf == 160 ? 3 : 2)
row_kernel(const Args A, int ranks, int slots)
{
    constexpr int kE = Piece<T>::kElems, kP = Piece<T>::kPairs;
    constexpr int kBatch = 4; // pieces a thread has in registers at once
    constexpr int kStep = kThreadsOf * kBatch, kRowWarps = kThreadsOf / 32;
    extern __shared__ uint4 part[]; // [slots]; top_p, top_s, top_id; marks
    __shared__ RowShared sh;
    float* top_p = reinterpret_cast<float*>(part + slots);
    float* top_s = top_p + A.top;
    int32_t* top_id = reinterpret_cast<int32_t*>(top_s + A.top);
    // a bit for each of the part's columns: the teacher's entries
    uint32_t* marks = reinterpret_cast<uint32_t*>(top_id + A.top);
    const uint32_t part_at = static_cast<uint32_t>(__cvta_generic_to_shared(part));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = ranks > 1 ? static_cast<int>(blockIdx.x % ranks) : 0;
    const int64_t clusters = gridDim.x / ranks;
    const float inv_tau = 1.0f / A.tau;
    const float c2 = kLog2e * inv_tau; // kOne: the only one
    const int64_t vocab = A.vocab;
    const int64_t first_piece = static_cast<int64_t>(rank) * slots;

    auto part_of = [&](int64_t row) {
        return Part<T>(static_cast<const T*>(A.logits) + row * A.stride, vocab, first_piece, slots);
    };
    // A row's fetches are two groups: slots below half, which a row's first pass
    // waits for at its start, and the others (some below may wait with them).
    const int half = slots / 2;
    bool split = false;
    auto close_group = [&] { asm volatile("cp.async.commit_group;" ::: "memory"); };
    auto at_slot = [&](int j) {
        if (!split && j >= half) {
            close_group();
            split = true;
        }
    };
    auto close_row = [&] {
        if (!split) close_group();
        close_group();
        split = false;
    };
    auto fetch_from = [&](const Part<T>& p, int j) { // and the row's ends
        for (; j < p.to; j += kThreadsOf) {
            at_slot(j);
            fetch_whole(part_at, p, j);
        }
        fetch_ends<kThreadsOf>(part, p, vocab);
        close_row();
    };
    // What a row needs beside its logits is read a row ahead (the weight two, as
    // it decides whether the next row is fetched); rows past the last weigh 0.
    auto weight = [&](int64_t row) {
        return row >= A.rows ? 0.0f : A.row_weight ? A.row_weight[row] : 1.0f;
    };
    auto label_of = [&](int64_t row) {
        return A.labels && row < A.rows ? dev::load_index(A.labels, A.label_type, row) : int64_t(-1);
    };
    auto entry_of = [&](int64_t row, int k, int32_t& id, float& t) { // -1: not counted
        id = -1;
        t = -INFINITY;
        if (k >= A.top || row >= A.rows) return;
        const int64_t i = dev::load_index(A.ids, A.id_type, row * A.top + k);
        float x[1];
        dev::load_any<1>(A.teacher, A.teacher_type, row * A.top + k, x);
        if (i >= 0 && i < vocab) {
            id = static_cast<int32_t>(i);
            t = x[0];
        }
    };

    if (kGrad)
        for (int i = tid; i < (slots * kE + 31) / 32; i += kThreadsOf) marks[i] = 0;
    if (tid < kMaxRowWarps) { // places without a warp
        sh.most[0][tid] = sh.most[1][tid] = -INFINITY;
        for (int i = 0; i < 4; ++i) sh.sum[i][tid] = 0.0f;
    }
    if (tid == 0) dev::init_words(sh.words);
    __syncthreads();
    if (ranks > 1) dev::cluster_barrier(); // every block has begun before another writes to its shared memory
    int64_t row = blockIdx.x / ranks;
    if (row >= A.rows) row = A.rows;
    float w = weight(row), w_next = weight(row + clusters);
    int64_t label = label_of(row);
    int32_t my_id; // entry tid
    float my_t;
    entry_of(row, tid, my_id, my_t);
    Part<T> here = part_of(row < A.rows ? row : 0);
    if (w == 0.0f) here.n = here.from = here.to = 0;
    fetch_from(here, tid);
    here = part_of(row < A.rows ? row : 0);
    dev::Turns turns;
    while (row < A.rows) {
        const int64_t next = row + clusters;
        const int64_t this_row = row, this_label = label;
        const float this_w = w;
        const Part<T> now = here;
        const int32_t this_id = my_id;
        const float this_t = my_t;
        here = part_of(next < A.rows ? next : 0);
        Part<T> then = here;
        if (w_next == 0.0f) then.n = then.from = then.to = 0; // nothing to fetch
        w = w_next;
        row = next;
        const T* s = now.row;
        T* ds = kGrad ? static_cast<T*>(A.dlogits) + this_row * A.dstride : nullptr;
        const int n = now.n;
        const int64_t lo = now.lo, hi = lo + static_cast<int64_t>(n) * kE;
        // the student's logits at the label and at entry tid, then the next row's
        const bool labelled = this_label >= 0 && this_label < vocab;
        float s_label = 0.0f, my_s = -INFINITY; // -inf: not counted
        if (this_w != 0.0f) {
            if (labelled) s_label = dev::load1(s + this_label);
            if (this_id >= 0) my_s = dev::load1(s + this_id);
        }
        w_next = weight(next + clusters);
        label = label_of(next);
        entry_of(next, tid, my_id, my_t);
        if (this_w == 0.0f) { // a masked row: not read
            if (rank == 0 && tid == 0) {
                A.ce[this_row] = 0.0f;
                A.kl[this_row] = 0.0f;
            }
            if (kGrad)
                for (int64_t j = lo + tid; j < hi; j += kThreadsOf)
                    if (j >= 0 && j < vocab) dev::store1(ds + j, 0.0f);
            fetch_from(then, tid);
            continue; // the whole cluster does
        }

        // the next row comes to the L2 meanwhile
        if (kGrad && tid == 0 && then.to > then.from)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                             then.row + then.lo + static_cast<int64_t>(then.from) * kE),
                         "r"(16 * (then.to - then.from))
                         : "memory");
        // pass 1: the maximum, and the sums relative to it
        float m = -INFINITY;
        float2 z1 = dev::pair(0.0f), z2 = z1;
        auto take = [&](const uint4& w, const Scale& k1, const Scale& k2) {
            float2 x[kP];
            unpack_piece(w, x, T());
#pragma unroll
            for (int e = 0; e < kP; ++e) {
                const float2 e2 = k2.exp2(x[e]);
                z2 = dev::add2(z2, e2);
                if (kExps == kSquare) z1 = dev::fma2(e2, e2, z1);
                if (kExps == kFourth) {
                    const float2 q = dev::mul2(e2, e2);
                    z1 = dev::fma2(q, q, z1);
                }
                if (kExps == kTwo) z1 = dev::add2(z1, k1.exp2(x[e]));
            }
        };
        auto raise = [&](float mx) { // a larger maximum: the sums so far shrink
            if (mx > m) {
                const float f2 = Scale(m, c2).to(Scale(mx, c2).ref);
                z2 = dev::mul2(z2, dev::pair(f2));
                if (kExps == kSquare || kExps == kFourth)
                    z1 = dev::mul2(z1, dev::pair(power_of<kExps>(f2)));
                if (kExps == kTwo)
                    z1 = dev::mul2(z1, dev::pair(Scale(m, kLog2e).to(Scale(mx, kLog2e).ref)));
                m = mx;
            }
        };
        int j = tid;
        // the fetches of the first half have been under way for longer
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        bool rest = false; // whether the others have been waited for
        for (; j + kStep - kThreadsOf < n; j += kStep) {
            if (!rest && j + kStep - kThreadsOf >= half) {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
                rest = true;
            }
            uint4 raw[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) raw[u] = part[j + u * kThreadsOf];
            float mx = piece_max(raw[0], T());
#pragma unroll
            for (int u = 1; u < kBatch; ++u) mx = fmaxf(mx, piece_max(raw[u], T()));
            raise(mx);
            const Scale k1(m, kLog2e), k2(m, c2);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) take(raw[u], k1, k2);
            if (!kGrad) {
                at_slot(j);
#pragma unroll
                for (int u = 0; u < kBatch; ++u) fetch_whole(part_at, then, j + u * kThreadsOf);
            }
        }
        if (!rest) asm volatile("cp.async.wait_group 0;" ::: "memory");
        for (; j < n; j += kThreadsOf) {
            const uint4 raw = part[j];
            raise(piece_max(raw, T()));
            const Scale k1(m, kLog2e), k2(m, c2);
            take(raw, k1, k2);
            if (!kGrad) {
                at_slot(j);
                fetch_whole(part_at, then, j);
            }
        }
        if (!kGrad) fetch_from(then, j); // slots that the next row has beyond this one's

        // the teacher's entries; the student's logits there
        float tm = -INFINITY;
        bool twice = false; // an id of this part that an earlier entry has
        for (int k = tid; k < A.top; k += kThreadsOf) {
            int32_t id = this_id;
            float t = this_t, at = my_s;
            if (k != tid) {
                entry_of(this_row, k, id, t);
                at = id >= 0 ? dev::load1(s + id) : -INFINITY;
            }
            tm = fmaxf(tm, t);
            top_id[k] = id;
            top_p[k] = t;
            top_s[k] = at;
            if (kGrad && id >= 0 && id >= lo && id < hi) {
                const uint32_t place = static_cast<uint32_t>(id - lo), bit = 1u << (place & 31u);
                twice |= (atomicOr(&marks[place >> 5], bit) & bit) != 0;
            }
        }

        // the block's maxima
        float block_m = warp_max(m);
        tm = warp_max(tm);
        if (lane == 0) {
            sh.most[0][warp] = block_m;
            sh.most[1][warp] = tm;
        }
        twice = __syncthreads_or(twice);
        block_m = warp_max(sh.most[0][lane % kMaxRowWarps]);
        tm = warp_max(sh.most[1][lane % kMaxRowWarps]);
        const RowScale b1(block_m, kLog2e), b2(block_m, c2);
        float sbase = block_m;
        const bool far_part = b2.far || (kExps == kTwo && b1.far);
        bool nothing = false; // a masked part of a row that has a logit far above it
        if (ranks > 1) {
            sbase = -INFINITY;
            for (int k = lane; k < A.top; k += 32) sbase = fmaxf(sbase, top_s[k]);
            sbase = warp_max(sbase);
            nothing = far_part && (sbase - block_m) * (kExps == kTwo ? fminf(kLog2e, c2) : c2) > 512.0f;
        }
        if (sbase == -INFINITY) sbase = 0.0f;
        const float tbase = tm == -INFINITY ? 0.0f : tm;
        // its sums
        float v[4] = {z1.x + z1.y, z2.x + z2.y, 0.0f, 0.0f};
        if (far_part && !nothing) {
            float2 z = make_float2(0.0f, 0.0f);
            if (kGrad) {
                for (int j = tid; j < n; j += kThreadsOf) {
                    float2 x[kP];
                    unpack_piece(part[j], x, T());
#pragma unroll
                    for (int e = 0; e < kP; ++e) {
                        const float2 d = dev::add2(x[e], dev::pair(-b2.m));
                        const float2 e1 = exp2_pair(dev::mul2(d, dev::pair(kLog2e)));
                        const float2 e2 = exp2_pair(dev::mul2(d, dev::pair(c2)));
                        z.x += e1.x + e1.y;
                        z.y += e2.x + e2.y;
                    }
                }
            } else {
                z = far_sums(now, vocab, b2.m, kLog2e, c2);
            }
            v[0] = kExps == kTwo ? z.x * exp2_approx(b1.off()) : z.x;
            v[1] = z.y * exp2_approx(b2.off());
        } else { // a thread without anything above -inf has 0, or NaN
            const float f2 = nothing ? 0.0f : Scale(m, c2).to(b2.ref);
            v[1] *= f2;
            v[0] *= kExps == kOne || nothing ? 0.0f
                    : kExps == kTwo          ? Scale(m, kLog2e).to(b1.ref)
                                             : power_of<kExps>(f2);
        }
        for (int k = tid; k < A.top; k += kThreadsOf) {
            const float e = exp2_approx((top_p[k] - tbase) * c2); // 0 where not counted
            v[2] += e;
            if (e != 0.0f) v[3] = fmaf(e * kCrossUnit, (top_p[k] - tbase) - (top_s[k] - sbase), v[3]);
            top_p[k] = e;
        }
        const bool marked = kGrad && labelled && this_label >= lo && this_label < hi &&
                            (marks[(this_label - lo) >> 5] >> ((this_label - lo) & 31) & 1);
        const float sum = warp_sum4(v, lane);
        if (lane % 8 == 0) sh.sum[lane / 8][warp] = sum;
        __syncthreads();
        float all = sh.sum[lane / 8][lane % 8];
        if (kRowWarps > 8) all += sh.sum[lane / 8][lane % 8 + 8];
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, off);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, all, 8 * i);
        float row_m = block_m, zs1 = v[0], zs2 = v[1];
        const float zt = v[2], cross = v[3];
        if (ranks > 1) { // the cluster's
            const float4* words = turns.take(sh.words, rank, ranks, block_m, v[0], v[1]);
            for (int r = 0; r < ranks; ++r) row_m = fmaxf(row_m, words[r].x);
            const RowScale to1(row_m, kLog2e), to2(row_m, c2);
            zs1 = zs2 = 0.0f;
            for (int r = 0; r < ranks; ++r) {
                const float rm = words[r].x;
                // a part without anything above -inf holds 0, or NaN
                const float f2 = rm == -INFINITY ? 1.0f : RowScale(rm, c2).to(to2);
                const float f1 = kExps != kTwo     ? power_of<kExps>(f2)
                                 : rm != -INFINITY ? RowScale(rm, kLog2e).to(to1)
                                                   : 1.0f;
                zs1 = fmaf(words[r].y, f1, zs1);
                zs2 = fmaf(words[r].z, f2, zs2);
            }
            if (turns.lost) zs1 = zs2 = __int_as_float(0x7FC00000);
        }
        if (kExps == kOne) zs1 = zs2;
        const RowScale r1(row_m, kLog2e), r2(row_m, c2);
        // a row whose logits are all -inf has no distribution, a teacher whose
        // counted entries are all -inf (or none) has none either; a NaN is neither
        const bool empty = zs2 == 0.0f;
        const bool has_top = zt != 0.0f && !empty;
        const bool has_label = labelled && !empty;
        if (rank == 0 && tid == 0) {
            const float from = row_m == -INFINITY ? 0.0f : row_m;
            const float log1 = kExps == kTwo ? r1.log_of(zs1) : r2.log_of(zs1, 1 << kExps);
            A.ce[this_row] = has_label ? log1 - (s_label - from) : 0.0f;
            A.kl[this_row] = has_top ? kl_of(A.tau, cross, zt, from - sbase, r2.log_of(zs2)) : 0.0f;
        }
        if constexpr (kGrad) {
            for (int k = tid; k < A.top; k += kThreadsOf) { // the marks are read: clear them
                const int32_t id = top_id[k];
                if (id >= lo && id < hi && id >= 0) marks[(id - lo) >> 5] = 0;
            }
            const float hit = has_label ? this_w * A.ce_weight : 0.0f;
            const float pull = has_top ? this_w * A.kl_weight * A.tau : 0.0f;
            const float share = has_top ? __fdividef(pull, zt) : 0.0f;
            float a1 = has_label ? __fdividef(hit, zs1) : 0.0f;
            float a2 = has_top ? __fdividef(pull, zs2) : 0.0f;
            if (kExps == kOne) a2 += a1;
            const bool has_any = has_top || has_label; // else +0, whatever the logits are
            auto combine = [&](float2 e2, auto e1) {
                if (kExps == kSquare) // (a1 e2 + a2) e2
                    return dev::mul2(dev::fma2(dev::pair(a1), e2, dev::pair(a2)), e2);
                const float2 g = dev::mul2(e2, dev::pair(a2));
                if (kExps == kFourth) {
                    const float2 q = dev::mul2(e2, e2);
                    return dev::fma2(dev::mul2(q, dev::pair(a1)), q, g);
                }
                return kExps == kTwo ? dev::fma2(e1(), dev::pair(a1), g) : g;
            };
            auto dense = [&](float2 x) { // where the row is not far
                return combine(r2.exp2(x), [&] { return r1.exp2(x); });
            };
            auto dense1 = [&](float x) {
                return combine(dev::pair(r2.exp2_any(x)), [&] { return dev::pair(r1.exp2_any(x)); }).x;
            };
            const bool far = r2.far || (kExps == kTwo && r1.far);
            const bool alike = ((reinterpret_cast<uintptr_t>(ds) ^ reinterpret_cast<uintptr_t>(s)) & 15) == 0;
            // slots that are written 16 bytes at once
            const int wide_from = alike ? now.from : n, wide_to = alike ? now.to : n;
            T* out = ds + lo;
            auto write = [&](int j, const float2 (&x)[kP]) {
                if (j >= wide_from && j < wide_to) {
                    __stcs(reinterpret_cast<uint4*>(out + static_cast<int64_t>(j) * kE),
                           pack_piece(x, T()));
                    return;
                }
                const int64_t at = lo + static_cast<int64_t>(j) * kE;
#pragma unroll
                for (int e = 0; e < kE; ++e)
                    if (at + e >= 0 && at + e < vocab)
                        dev::store1(ds + at + e, e & 1 ? x[e / 2].y : x[e / 2].x);
            };
            int j = tid;
            if (!has_any) {
                const float2 zero[kP] = {};
                for (; j < n; j += kThreadsOf) {
                    write(j, zero);
                    at_slot(j);
                    fetch_whole(part_at, then, j);
                }
            }
            if (far) {
                const float f1 = kExps == kOne   ? 0.0f
                                 : kExps == kTwo ? a1 * exp2_approx(r1.off())
                                                 : a1;
                const float f2 = a2 * exp2_approx(r2.off());
                for (; j < n; j += kThreadsOf) {
                    float2 x[kP];
                    unpack_piece(part[j], x, T());
#pragma unroll
                    for (int e = 0; e < kP; ++e) {
                        const float2 d = dev::add2(x[e], dev::pair(-r2.m));
                        const float2 e1 = exp2_pair(dev::mul2(d, dev::pair(kLog2e)));
                        const float2 e2 = exp2_pair(dev::mul2(d, dev::pair(c2)));
                        x[e] = dev::fma2(e1, dev::pair(f1), dev::mul2(e2, dev::pair(f2)));
                    }
                    write(j, x);
                    at_slot(j);
                    fetch_whole(part_at, then, j);
                }
            }
            // whole batches: nothing of them at the ends, of this row or the next
            const int first = now.from > then.from ? now.from : then.from;
            int batches = wide_to < then.to || then.to == 0 ? wide_to : then.to;
            if (!alike) batches = 0;
            for (; j + kStep - kThreadsOf < batches; j += kStep) {
                at_slot(j);
                uint4 raw[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) raw[u] = part[j + u * kThreadsOf];
                T* to = out + static_cast<int64_t>(j) * kE;
                const T* from = then.row + then.lo + static_cast<int64_t>(j) * kE;
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    float2 x[kP];
                    unpack_piece(raw[u], x, T());
#pragma unroll
                    for (int e = 0; e < kP; ++e) x[e] = dense(x[e]);
                    if (u == 0 && j < first) {
                        write(j, x);
                        fetch_whole(part_at, then, j);
                    } else {
                        __stcs(reinterpret_cast<uint4*>(to + u * kThreadsOf * kE), pack_piece(x, T()));
                        if (then.to) fetch16(part_at + 16u * (j + u * kThreadsOf), from + u * kThreadsOf * kE);
                    }
                }
            }
            for (; j < n; j += kThreadsOf) {
                float2 x[kP];
                unpack_piece(part[j], x, T());
#pragma unroll
                for (int e = 0; e < kP; ++e) x[e] = dense(x[e]);
                write(j, x);
                at_slot(j);
                fetch_whole(part_at, then, j);
            }
            fetch_from(then, j);
            __syncthreads(); // before the teacher's entries are written over
            if (has_label && !marked && tid == 0 && this_label >= lo && this_label < hi)
                dev::store1(ds + this_label, dense1(s_label) - hit);
            for (int k = tid; k < A.top; k += kThreadsOf) {
                const int32_t id = top_id[k];
                if (id < lo || id >= hi || id < 0) continue; // not counted, or another rank's
                float p = top_p[k];
                if (twice) { // the first entry of an id writes for all of them
                    bool first_of = true;
                    p = 0.0f;
                    for (int q = 0; q < A.top; ++q) {
                        if (top_id[q] != id) continue;
                        if (q < k) first_of = false;
                        p += top_p[q];
                    }
                    if (!first_of) continue;
                }
                float g = has_any ? fmaf(-share, p, dense1(top_s[k])) : 0.0f;
                if (id == this_label) g -= hit;
                dev::store1(ds + id, g);
            }
            if (twice) __syncthreads(); // others' entries were read
        }
    }
    // no block ends while another may still write to its shared memory
    if (ranks > 1) dev::cluster_barrier();
}

// Bytes of a row that a block should hold, and may hold.  Larger parts leave one block
// to an SM, smaller ones hand round more sums: 4096 x 32000 fp32 takes 206, 166, 167, 174
// and 261 us on 1, 2, 3, 4 and 8 ranks, its loss alone 108, 91 and 101 on 1, 2 and 4;
// 8191 x 50257 bf16 308 and 337 on 1 and 2; 2000 x 50257 fp32 141, 146, 144 and 166 on
// 2, 3, 4 and 8; 2000 x 131072 bf16 263, 229, 194 and 224.  The number of ranks is a
// power of two; another is better by up to a tenth where the parts come to 74 KB (2000 x
// 151936 bf16 on 3, 4, 5 and 8 ranks 256, 265, 241 and 250; 1000 x 256000 on 4, 5, 6 and
// 8 273, 213, 238 and 214).
constexpr int64_t kPartBytes = 104 * 1024, kMostPartBytes = 192 * 1024;

// Five blocks with parts up to the first of these fit an SM, three up to the second,
// then two; the more threads they have.  Measured (8192 rows bf16, device time): 20000
// logits at temperature 2 with 128, 160 and 256 threads 120, 128 and 153 us; 32000 at
// temperature 1 with 128, 160 and 256 187, 175 and 179, at 1.5 223, 213 and 228; with
// 256, 320 and 384 threads 38000 at 2 262, 248 and 264, 48000 at 1 273, 267 and 281,
// 24000 fp32 245, 237 and 248.  The loss alone of 32000 at 1 with 128, 160 and 320: 101,
// 96 and 114, of 2000 x 131072 on 4 ranks 115, 112 and 142.
constexpr int64_t kSmallPartBytes = 43 * 1024, kWidePartBytes = 72 * 1024;
template <typename T, bool kGrad, int kExps, int kThreadsOf>
int launch_rows(const Args& A, int ranks, int64_t slots, cudaStream_t stream)
{
    auto smem_of = [](int64_t n_slots, int64_t top) {
        return static_cast<size_t>(n_slots * 16 + top * 12 + (kGrad ? (n_slots * Piece<T>::kElems + 31) / 32 * 4 : 0));
    };
    const size_t smem = smem_of(slots, A.top);
    auto* kernel = row_kernel<T, kGrad, kExps, kThreadsOf>;
    const void* k = reinterpret_cast<const void*>(kernel);
    if (smem > 32 * 1024 && !allow_shared(k, smem_of(kMostPartBytes / 16, kMaxTop))) return ZERO_ECUDA;
    const int resident = persistent_clusters(k, kThreadsOf, smem, ranks);
    if (resident < 1) return ZERO_ECUDA;
    const int64_t clusters = resident < A.rows ? resident : A.rows;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * ranks));
    cfg.blockDim = dim3(kThreadsOf);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(ranks);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, A, ranks, static_cast<int>(slots)));
}

template <typename T, bool kGrad, int kExps>
int launch_rows(const Args& A, cudaStream_t stream, bool& fits)
{
    const int64_t pieces = (A.vocab + 2 * (Piece<T>::kElems - 1)) / Piece<T>::kElems + 1;
    int ranks = 1;
    while (ranks < kMaxRanks &&
           ((pieces + ranks - 1) / ranks * 16 > kPartBytes || A.rows * ranks * 2 <= 152))
        ranks *= 2;
    const int64_t slots = (pieces + ranks - 1) / ranks;
    fits = slots * 16 <= kMostPartBytes;
    if (!fits) return ZERO_OK;
    if (slots * 16 > kWidePartBytes)
        return launch_rows<T, kGrad, kExps, 320>(A, ranks, slots, stream);
    return slots * 16 > kSmallPartBytes ? launch_rows<T, kGrad, kExps, 160>(A, ranks, slots, stream)
                                        : launch_rows<T, kGrad, kExps, 128>(A, ranks, slots, stream);
}

template <typename T, bool kGrad>
int launch(const Args& A, cudaStream_t stream)
{
    bool fits = false;
    const int rc = !A.labels || A.tau == 1.0f ? launch_rows<T, kGrad, kOne>(A, stream, fits)
                   : A.tau == 2.0f            ? launch_rows<T, kGrad, kSquare>(A, stream, fits)
                   : A.tau == 4.0f            ? launch_rows<T, kGrad, kFourth>(A, stream, fits)
                                              : launch_rows<T, kGrad, kTwo>(A, stream, fits);
    if (rc != ZERO_OK || fits) return rc;
    // a row that not even 8 blocks can hold is read twice
    const int resident =
        persistent_blocks(reinterpret_cast<const void*>(distill_kernel<T, kGrad>), kThreads, 0);
    if (resident < 1) return ZERO_ECUDA;
    const unsigned blocks = static_cast<unsigned>(A.rows < resident ? A.rows : resident);
    distill_kernel<T, kGrad><<<blocks, kThreads, 0, stream>>>(A);
    return cuda_status(cudaGetLastError());
}

int distill(const zero_distill_t* d, const void* logits, const void* teacher_logits,
            const void* teacher_ids, const void* labels, const float* row_weight, float* ce,
            float* kl, bool grad, void* dlogits, int64_t dlogits_stride, cudaStream_t stream)
{
    if (!d || d->n_rows < 0 || d->vocab < 1 || d->vocab > 0x7FFFFFFF ||
        d->logits_stride < d->vocab || d->top < 1 || d->top > kMaxTop ||
        !float_type(d->logits_type) || !float_type(d->teacher_type) || !index_type(d->id_type) ||
        !index_type(d->label_type))
        return ZERO_EINVAL;
    if (!std::isfinite(d->temperature) || d->temperature < 1e-3 || d->temperature > 1e3 ||
        !std::isfinite(d->ce_weight) || !std::isfinite(d->kl_weight))
        return ZERO_EINVAL;
    if (grad && dlogits_stride < d->vocab) return ZERO_EINVAL;
    if (d->n_rows == 0) return ZERO_OK;
    if (!logits || !teacher_logits || !teacher_ids || !ce || !kl || (grad && !dlogits))
        return ZERO_EINVAL;
    if (grad && dlogits == logits && dlogits_stride != d->logits_stride) return ZERO_EINVAL;
    if (!aligned_to(logits, type_bytes(d->logits_type)) ||
        !aligned_to(dlogits, type_bytes(d->logits_type)) ||
        !aligned_to(teacher_logits, type_bytes(d->teacher_type)) ||
        !aligned_to(teacher_ids, type_bytes(d->id_type)) ||
        !aligned_to(labels, type_bytes(d->label_type)) || !aligned_to(row_weight, 4) ||
        !aligned_to(ce, 4) || !aligned_to(kl, 4))
        return ZERO_EALIGN;
    Args A = {};
    A.logits = logits;
    A.teacher = teacher_logits;
    A.ids = teacher_ids;
    A.labels = labels;
    A.row_weight = row_weight;
    A.ce = ce;
    A.kl = kl;
    A.dlogits = dlogits;
    A.rows = d->n_rows;
    A.vocab = d->vocab;
    A.stride = d->logits_stride;
    A.dstride = dlogits_stride;
    A.top = d->top;
    A.teacher_type = d->teacher_type;
    A.id_type = d->id_type;
    A.label_type = d->label_type;
    A.tau = static_cast<float>(d->temperature);
    A.ce_weight = static_cast<float>(d->ce_weight);
    A.kl_weight = static_cast<float>(d->kl_weight);
    if (d->logits_type == ZERO_TYPE_BF16)
        return grad ? launch<Bf16, true>(A, stream) : launch<Bf16, false>(A, stream);
    return grad ? launch<float, true>(A, stream) : launch<float, false>(A, stream);
}

} // namespace
} // namespace zero

using namespace zero;

extern "C" int zero_distill_forward(const zero_distill_t* d, const void* logits,
                                    const void* teacher_logits, const void* teacher_ids,
                                    const void* labels, const float* row_weight, float* ce,
                                    float* kl, cudaStream_t stream)
{
    return distill(d, logits, teacher_logits, teacher_ids, labels, row_weight, ce, kl, false,
                   nullptr, 0, stream);
}

extern "C" int zero_distill_forward_backward(const zero_distill_t* d, const void* logits,
                                             const void* teacher_logits, const void* teacher_ids,
                                             const void* labels, const float* row_weight,
                                             float* ce, float* kl, void* dlogits,
                                             int64_t dlogits_stride, cudaStream_t stream)
{
    return distill(d, logits, teacher_logits, teacher_ids, labels, row_weight, ce, kl, true,
                   dlogits, dlogits_stride, stream);
}

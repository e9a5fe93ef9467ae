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
//   kl = tau^2 * ( sum_k p_k ((t_k - tm) - (s_ik - m)) / tau + log Z - log Zt )
// with Zt the teacher's sum: the large terms cancel before the products.
#include "typed.cuh"
#include "zero_internal.h"

namespace zero {
namespace {

using dev::Bf16;

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
            if (e != 0.0f)
                cross = fmaf(e, ((top_p[k] - tbase) - (top_s[k] - base)) * inv_tau, cross);
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
            A.kl[row] =
                has_top ? A.tau * A.tau * (cross / zt + (logf(z2) - logf(zt))) : 0.0f;
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

template <typename T>
int launch(const Args& A, bool grad, cudaStream_t stream)
{
    const void* kernel = grad ? reinterpret_cast<const void*>(distill_kernel<T, true>)
                              : reinterpret_cast<const void*>(distill_kernel<T, false>);
    const int resident = persistent_blocks(kernel, kThreads, 0);
    if (resident < 1) return ZERO_ECUDA;
    const unsigned blocks = static_cast<unsigned>(A.rows < resident ? A.rows : resident);
    if (grad)
        distill_kernel<T, true><<<blocks, kThreads, 0, stream>>>(A);
    else
        distill_kernel<T, false><<<blocks, kThreads, 0, stream>>>(A);
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
    return d->logits_type == ZERO_TYPE_BF16 ? launch<Bf16>(A, grad, stream)
                                            : launch<float>(A, grad, stream);
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

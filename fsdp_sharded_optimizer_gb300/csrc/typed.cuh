// typed.cuh -- element access by type for the training operators (embed.cu,
// block_norm.cu, distill.cu): bf16 or fp32 tensors, read as fp32 and rounded
// once (nearest-even) when written.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "device.cuh"
#include "zero.h"

namespace zero {

// Host-side checks shared by the operators.
inline bool float_type(int32_t t) { return t == ZERO_TYPE_BF16 || t == ZERO_TYPE_F32; }
inline bool index_type(int32_t t) { return t == ZERO_TYPE_I32 || t == ZERO_TYPE_I64; }
inline int type_bytes(int32_t t)
{
    return t == ZERO_TYPE_BF16 ? 2 : t == ZERO_TYPE_I64 ? 8 : 4;
}
// A tensor may start at any of its elements (a weight inside a flat unit), so
// only alignment to the element is required; wide accesses are chosen by the
// kernels' own checks.
inline bool aligned_to(const void* p, int bytes)
{
    return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(bytes - 1)) == 0;
}

namespace dev {

struct Bf16 { // one bf16 element
    uint16_t bits;
};

__device__ __forceinline__ float load1(const Bf16* p)
{
    return __uint_as_float(static_cast<uint32_t>(p->bits) << 16);
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(Bf16* p, float x)
{
    p->bits = static_cast<uint16_t>(bf16_rne(x));
}
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }

// 8 consecutive elements as loaded (16 or 32 bytes), from an address that is a
// multiple of 16 bytes.
template <typename T>
struct Raw8;
template <>
struct Raw8<Bf16> {
    uint4 a;
};
template <>
struct Raw8<float> {
    float4 a, b;
};

__device__ __forceinline__ void load_raw8(const Bf16* p, Raw8<Bf16>& r)
{
    r.a = *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ void load_raw8(const float* p, Raw8<float>& r)
{
    r.a = *reinterpret_cast<const float4*>(p);
    r.b = *reinterpret_cast<const float4*>(p + 4);
}
// The same for data that is read once.
__device__ __forceinline__ void stream_raw8(const Bf16* p, Raw8<Bf16>& r)
{
    r.a = __ldcs(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ void stream_raw8(const float* p, Raw8<float>& r)
{
    r.a = __ldcs(reinterpret_cast<const float4*>(p));
    r.b = __ldcs(reinterpret_cast<const float4*>(p + 4));
}
__device__ __forceinline__ void unpack8(const Raw8<Bf16>& r, float (&x)[8])
{
    x[0] = bf16_lo(r.a.x), x[1] = bf16_hi(r.a.x);
    x[2] = bf16_lo(r.a.y), x[3] = bf16_hi(r.a.y);
    x[4] = bf16_lo(r.a.z), x[5] = bf16_hi(r.a.z);
    x[6] = bf16_lo(r.a.w), x[7] = bf16_hi(r.a.w);
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&x)[8])
{
    x[0] = r.a.x, x[1] = r.a.y, x[2] = r.a.z, x[3] = r.a.w;
    x[4] = r.b.x, x[5] = r.b.y, x[6] = r.b.z, x[7] = r.b.w;
}

// Two fp32 values to a word of two bf16 (lo in the low half), nearest-even,
// NaN to a quiet NaN: one conversion instruction.
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi)
{
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(cvt_bf16x2(x[0], x[1]), cvt_bf16x2(x[2], x[3]), cvt_bf16x2(x[4], x[5]),
                      cvt_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(Bf16* p, const float (&x)[8])
{
    *reinterpret_cast<uint4*>(p) = pack8(x);
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8])
{
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
// The same for data that this call does not read again.
__device__ __forceinline__ void store8_stream(Bf16* p, const float (&x)[8])
{
    __stcs(reinterpret_cast<uint4*>(p), pack8(x));
}
__device__ __forceinline__ void store8_stream(float* p, const float (&x)[8])
{
    __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
}

// Two fp32 values in one register pair: one instruction works on both.
__device__ __forceinline__ unsigned long long as_pair(float2 a)
{
    return (static_cast<unsigned long long>(__float_as_uint(a.y)) << 32) | __float_as_uint(a.x);
}
__device__ __forceinline__ float2 from_pair(unsigned long long a)
{
    return make_float2(__uint_as_float(static_cast<uint32_t>(a)),
                       __uint_as_float(static_cast<uint32_t>(a >> 32)));
}
__device__ __forceinline__ float2 pair(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(as_pair(a)), "l"(as_pair(b)), "l"(as_pair(c)));
    return from_pair(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as_pair(a)), "l"(as_pair(b)));
    return from_pair(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as_pair(a)), "l"(as_pair(b)));
    return from_pair(d);
}
__device__ __forceinline__ void unpack8(const Raw8<Bf16>& r, float2 (&x)[4])
{
    x[0] = make_float2(bf16_lo(r.a.x), bf16_hi(r.a.x));
    x[1] = make_float2(bf16_lo(r.a.y), bf16_hi(r.a.y));
    x[2] = make_float2(bf16_lo(r.a.z), bf16_hi(r.a.z));
    x[3] = make_float2(bf16_lo(r.a.w), bf16_hi(r.a.w));
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float2 (&x)[4])
{
    x[0] = make_float2(r.a.x, r.a.y), x[1] = make_float2(r.a.z, r.a.w);
    x[2] = make_float2(r.b.x, r.b.y), x[3] = make_float2(r.b.z, r.b.w);
}
__device__ __forceinline__ void store8_stream(Bf16* p, const float2 (&x)[4])
{
    __stcs(reinterpret_cast<uint4*>(p),
           make_uint4(cvt_bf16x2(x[0].x, x[0].y), cvt_bf16x2(x[1].x, x[1].y),
                      cvt_bf16x2(x[2].x, x[2].y), cvt_bf16x2(x[3].x, x[3].y)));
}
__device__ __forceinline__ void store8_stream(float* p, const float2 (&x)[4])
{
    __stcs(reinterpret_cast<float4*>(p), make_float4(x[0].x, x[0].y, x[1].x, x[1].y));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[2].x, x[2].y, x[3].x, x[3].y));
}

// kVec (8 or 1) elements at once.
template <int kVec, typename T>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[kVec])
{
    if constexpr (kVec == 8) {
        Raw8<T> r;
        load_raw8(p, r);
        unpack8(r, x);
    } else {
        x[0] = load1(p);
    }
}
template <int kVec, typename T>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[kVec])
{
    if constexpr (kVec == 8)
        store8(p, x);
    else
        store1(p, x[0]);
}

// Tensors of a type known only at run time (small ones: weights, gates).
template <int kVec>
__device__ __forceinline__ void load_any(const void* p, int32_t type, int64_t i, float (&x)[kVec])
{
    if (type == ZERO_TYPE_BF16)
        load_vec<kVec>(static_cast<const Bf16*>(p) + i, x);
    else
        load_vec<kVec>(static_cast<const float*>(p) + i, x);
}
template <int kVec>
__device__ __forceinline__ void store_any(void* p, int32_t type, int64_t i, const float (&x)[kVec])
{
    if (type == ZERO_TYPE_BF16)
        store_vec<kVec>(static_cast<Bf16*>(p) + i, x);
    else
        store_vec<kVec>(static_cast<float*>(p) + i, x);
}

__device__ __forceinline__ int64_t load_index(const void* p, int32_t type, int64_t i)
{
    return type == ZERO_TYPE_I64 ? static_cast<const int64_t*>(p)[i]
                                 : static_cast<const int32_t*>(p)[i];
}

} // namespace dev
} // namespace zero

// Element types chosen at run time: 16-byte (or single-element) loads and
// stores of fp32, bf16 and fp16 rows, converted to and from fp32.  The type
// is the same for every thread of a launch, so each branch on it is uniform.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace moe {

enum ElemType : int { ELEM_F32 = 0, ELEM_BF16 = 1, ELEM_F16 = 2 };

__host__ __device__ __forceinline__ int elem_bytes(int dt) { return dt == ELEM_F32 ? 4 : 2; }

// V elements as loaded: V = 8 (one 16-byte word of a 16-bit type, two of
// fp32) or 1.  Loading and converting are separate, so that a kernel can have
// several loads in flight before it uses the first.
template <int V>
struct RawVec;

template <>
struct RawVec<8> {
    uint4 a, b;
};
template <>
struct RawVec<1> {
    float v;
};

__device__ __forceinline__ uint4 ld16(const void* p) { return *reinterpret_cast<const uint4*>(p); }

template <int V>
__device__ __forceinline__ RawVec<V> load_raw(const void* base, int64_t off, int dt);

template <>
__device__ __forceinline__ RawVec<8> load_raw<8>(const void* base, int64_t off, int dt) {
    RawVec<8> r;
    if (dt == ELEM_F32) {
        const uint8_t* p = static_cast<const uint8_t*>(base) + off * 4;
        r.a = ld16(p);
        r.b = ld16(p + 16);
    } else {
        r.a = ld16(static_cast<const uint8_t*>(base) + off * 2);
        r.b = make_uint4(0, 0, 0, 0);
    }
    return r;
}
template <>
__device__ __forceinline__ RawVec<1> load_raw<1>(const void* base, int64_t off, int dt) {
    RawVec<1> r;
    if (dt == ELEM_F32)
        r.v = static_cast<const float*>(base)[off];
    else if (dt == ELEM_BF16)
        r.v = __bfloat162float(static_cast<const __nv_bfloat16*>(base)[off]);
    else
        r.v = __half2float(static_cast<const __half*>(base)[off]);
    return r;
}

// Data that goes by once: loads and stores that leave L2 first.
template <int V, int DT>
__device__ __forceinline__ RawVec<V> load_stream(const void* base, int64_t off) {
    RawVec<V> r;
    if constexpr (V == 8) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + off * (DT == ELEM_F32 ? 4 : 2));
        r.a = __ldcs(p);
        if constexpr (DT == ELEM_F32) r.b = __ldcs(p + 1);
    } else {
        r = load_raw<1>(base, off, DT);
    }
    return r;
}

__device__ __forceinline__ void words_to_f32(const uint4& w, int dt, float* v) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (dt == ELEM_BF16) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        } else {
            __half2 h;
            memcpy(&h, &u[i], 4);
            const float2 f = __half22float2(h);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

__device__ __forceinline__ void raw_to_f32(const RawVec<8>& r, int dt, float (&v)[8]) {
    if (dt == ELEM_F32) {
        v[0] = __uint_as_float(r.a.x);
        v[1] = __uint_as_float(r.a.y);
        v[2] = __uint_as_float(r.a.z);
        v[3] = __uint_as_float(r.a.w);
        v[4] = __uint_as_float(r.b.x);
        v[5] = __uint_as_float(r.b.y);
        v[6] = __uint_as_float(r.b.z);
        v[7] = __uint_as_float(r.b.w);
    } else {
        words_to_f32(r.a, dt, v);
    }
}
__device__ __forceinline__ void raw_to_f32(const RawVec<1>& r, int, float (&v)[1]) { v[0] = r.v; }

// Two fp32 values rounded (nearest even) to a pair of 16-bit elements.
__device__ __forceinline__ uint32_t pack2(float lo, float hi, int dt) {
    uint32_t r;
    if (dt == ELEM_BF16) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
        memcpy(&r, &b, 4);
    } else {
        const __half2 h = __floats2half2_rn(lo, hi);
        memcpy(&r, &h, 4);
    }
    return r;
}

__device__ __forceinline__ void store_vec(void* base, int64_t off, int dt, const float (&v)[8]) {
    if (dt == ELEM_F32) {
        float* p = static_cast<float*>(base) + off;
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + off) =
            make_uint4(pack2(v[0], v[1], dt), pack2(v[2], v[3], dt), pack2(v[4], v[5], dt), pack2(v[6], v[7], dt));
    }
}
__device__ __forceinline__ void store_vec(void* base, int64_t off, int dt, const float (&v)[1]) {
    if (dt == ELEM_F32)
        static_cast<float*>(base)[off] = v[0];
    else if (dt == ELEM_BF16)
        static_cast<__nv_bfloat16*>(base)[off] = __float2bfloat16_rn(v[0]);
    else
        static_cast<__half*>(base)[off] = __float2half_rn(v[0]);
}

template <int V, int DT>
__device__ __forceinline__ void store_stream(void* base, int64_t off, const float (&v)[V]) {
    if constexpr (V == 8 && DT == ELEM_F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + off);
        __stcs(p, make_float4(v[0], v[1], v[2], v[3]));
        __stcs(p + 1, make_float4(v[4], v[5], v[6], v[7]));
    } else if constexpr (V == 8) {
        __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + off),
               make_uint4(pack2(v[0], v[1], DT), pack2(v[2], v[3], DT), pack2(v[4], v[5], DT), pack2(v[6], v[7], DT)));
    } else {
        store_vec(base, off, DT, v);
    }
}

// The value that a store in type dt keeps.
__device__ __forceinline__ float round_to(float v, int dt) {
    if (dt == ELEM_F32) return v;
    if (dt == ELEM_BF16) return __bfloat162float(__float2bfloat16_rn(v));
    return __half2float(__float2half_rn(v));
}

}  // namespace moe

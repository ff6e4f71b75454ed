// io.hpp -- reading and writing fp32 and bf16 elements as fp32 values, one or
// eight at a time.
#pragma once

#include "device_math.hpp"

namespace selscan {
namespace io {

template <typename T> __device__ __forceinline__ float ld(const T* p);
template <> __device__ __forceinline__ float ld<float>(const float* p) { return *p; }
template <> __device__ __forceinline__ float ld<uint16_t>(const uint16_t* p) { return bf16_to_f32(*p); }
template <typename T> __device__ __forceinline__ void st(T* p, float v);
template <> __device__ __forceinline__ void st<float>(float* p, float v) { *p = v; }
template <> __device__ __forceinline__ void st<uint16_t>(uint16_t* p, float v) { *p = f32_to_bf16(v); }

// Four (16-byte aligned for fp32, 8-byte for bf16) or eight (16-byte aligned)
// consecutive elements.
__device__ __forceinline__ void ld4(const float* p, float* v) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
}
__device__ __forceinline__ void ld4(const uint16_t* p, float* v) {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    v[0] = bf16lo(q.x); v[1] = bf16hi(q.x); v[2] = bf16lo(q.y); v[3] = bf16hi(q.y);
}
__device__ __forceinline__ void ld8(const float* p, float* v) {
    ld4(p, v);
    ld4(p + 4, v + 4);
}
__device__ __forceinline__ void ld8(const uint16_t* p, float* v) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16lo(w[i]);
        v[2 * i + 1] = bf16hi(w[i]);
    }
}
__device__ __forceinline__ void st4(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void st4(uint16_t* p, const float* v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
__device__ __forceinline__ void st8(float* p, const float* v) {
    st4(p, v);
    st4(p + 4, v + 4);
}
__device__ __forceinline__ void st8(uint16_t* p, const float* v) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// V consecutive elements wherever they start: as loaded, widened, stored.
// Global memory takes 16-byte accesses at any element's address on this GPU
// (only a whole piece has to be inside the tensor).
template <typename T, int V> struct Piece {
    typedef T Vec __attribute__((ext_vector_type(V)));
    struct __attribute__((packed, may_alias, aligned(sizeof(T)))) Loose { Vec v; };
    Vec v;
    __device__ __forceinline__ void get(const T* p) { v = reinterpret_cast<const Loose*>(p)->v; }
    __device__ __forceinline__ void zero() { v = Vec(0); }
    __device__ __forceinline__ void widen(float* f) const {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (sizeof(T) == 2) f[i] = bf16_to_f32((uint16_t)v[i]);
            else f[i] = v[i];
        }
    }
    __device__ __forceinline__ void narrow(const float* f) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (sizeof(T) == 2) v[i] = f32_to_bf16(f[i]);
            else v[i] = f[i];
        }
    }
    __device__ __forceinline__ void put(T* p) const { reinterpret_cast<Loose*>(p)->v = v; }
};
template <typename T> struct Piece<T, 1> {
    T v;
    __device__ __forceinline__ void get(const T* p) { v = *p; }
    __device__ __forceinline__ void zero() { v = T(0); }
    __device__ __forceinline__ void widen(float* f) const { f[0] = ld(&v); }
    __device__ __forceinline__ void narrow(const float* f) { st(&v, f[0]); }
    __device__ __forceinline__ void put(T* p) const { *p = v; }
};

// Workgroups 0 .. n - 1 over two dimensions (a dimension holds fewer than
// 2^32 threads): those past n are for the kernel to turn away.
inline dim3 groups(int64_t n) {
    const int64_t x = n < (1 << 20) ? n : 1 << 20;
    return dim3((unsigned)x, (unsigned)((n + x - 1) / x));
}
__device__ __forceinline__ int64_t group_id() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

}  // namespace io
}  // namespace selscan

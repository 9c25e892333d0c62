// elements.cuh -- fp32 and bf16 elements in memory: single ones, and vectors
// of 16 bytes taken apart into fp32 and put together again.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mr.h"

namespace mr {

__device__ __forceinline__ uint4 load16(const void* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}
// What is read once: not kept in L1.
__device__ __forceinline__ uint4 load16_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void store16(void* p, uint4 v) {
    asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// What nothing reads soon.
__device__ __forceinline__ void store16_once(void* p, uint4 v) {
    asm volatile("st.global.cs.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// A warp clears n bytes from p on (both multiples of B, the element's bytes).
template <int B>
__device__ __forceinline__ void clear_bytes(char* p, uint64_t n, uint32_t lane) {
    using Raw = typename std::conditional<B == 2, uint16_t, uint32_t>::type;
    const uint64_t head = min(n, (16 - (uintptr_t)p % 16) % 16), body = (n - head) / 16 * 16;
    for (uint64_t i = lane * B; i < head; i += 32 * B) *reinterpret_cast<Raw*>(p + i) = 0;
    for (uint64_t i = head + lane * 16; i < head + body; i += 512) store16(p + i, make_uint4(0, 0, 0, 0));
    for (uint64_t i = head + body + lane * B; i < n; i += 32 * B) *reinterpret_cast<Raw*>(p + i) = 0;
}

// Two fp32 values to packed bf16, each rounded to nearest even: a in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

template <int DT>
struct Element;
template <>
struct Element<MR_FP32> {
    static constexpr int kBytes = 4, kLanes = 4;    // kLanes: elements in 16 bytes
    static constexpr uint32_t kMinusInf = 0xff800000u;
    using Raw = uint32_t;
    static __device__ __forceinline__ float get(const void* p, uint64_t i) { return static_cast<const float*>(p)[i]; }
    static __device__ __forceinline__ void put(void* p, uint64_t i, float v) { static_cast<float*>(p)[i] = v; }
    static __device__ __forceinline__ void unpack(uint4 v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <>
struct Element<MR_BF16> {
    static constexpr int kBytes = 2, kLanes = 8;
    static constexpr uint32_t kMinusInf = 0xff80u;
    using Raw = uint16_t;
    static __device__ __forceinline__ float get(const void* p, uint64_t i) {
        return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
    }
    static __device__ __forceinline__ void put(void* p, uint64_t i, float v) {
        static_cast<uint16_t*>(p)[i] = (uint16_t)pack_bf16(v, 0.0f);
    }
    static __device__ __forceinline__ void unpack(uint4 v, float (&f)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
        return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
    }
};

}  // namespace mr

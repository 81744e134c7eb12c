// Two FP32 values in a 64-bit register: sm_103a adds, multiplies and fuses both
// in one instruction, each rounded as its scalar counterpart; the assembler may fuse
// a product with the sum that it goes into.  For kernels whose instructions, not their
// bytes, would bound them.
#pragma once

#include "token_internal.cuh"

namespace tbe {

struct Pair {
    unsigned long long v;
};
__device__ __forceinline__ Pair pair(float x, float y) {
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpair(Pair a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// Two neighbouring elements of a raw vector as floats, and back.
template <typename T, int VEC> __device__ __forceinline__ Pair widen_pair(const Raw<T, VEC> &r, int j) {
    if constexpr (sizeof(T) == 4) {
        return pair(__uint_as_float(r.w[2 * j]), __uint_as_float(r.w[2 * j + 1]));
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const float2 f = bf16x2_to_float2(r.w[j]);
        return pair(f.x, f.y);
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r.w[j]));
        return pair(f.x, f.y);
    }
}
template <typename T, int VEC> __device__ __forceinline__ void narrow_pair(Raw<T, VEC> &r, int j, Pair a) {
    const float2 f = unpair(a);
    const float two[2] = {f.x, f.y};
    const Raw<T, 2> n = narrow<T, 2>(two);
#pragma unroll
    for (int i = 0; i < Raw<T, 2>::WORDS; ++i) r.w[j * Raw<T, 2>::WORDS + i] = n.w[i];
}

}  // namespace tbe

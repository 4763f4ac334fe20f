// packed.cuh -- rows of 16-bit elements as pairs of floats: unpacking, packed arithmetic,
// and tables of floats that eight to a lane are read without bank conflicts.
#pragma once

#include "common.cuh"

namespace pkv {

// Pairs of floats: the packed multiply and fused multiply-add of this part (each
// half rounds as the scalar one does) halve the arithmetic's instructions.
using f2 = unsigned long long;

__device__ __forceinline__ f2 make_f2(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split_f2(f2 v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 neg2(f2 a) { return a ^ 0x8000000080000000ull; }

template <typename T>
__device__ __forceinline__ void unpack(const uint4& v, f2 (&f)[4]) {
    float x[8];
    Cvt<T>::unpack8(v, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = make_f2(x[2 * e], x[2 * e + 1]);
}

template <typename T>
__device__ __forceinline__ uint4 pack(const f2 (&f)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float a, b;
        split_f2(f[e], a, b);
        w[e] = Cvt<T>::pack2(a, b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Tables of N floats in shared memory, eight to a lane, are laid out as two halves
// of four floats a lane: a lane's two 16-byte reads then sit next to its
// neighbours'.  Place of float x:
template <int N>
__device__ __forceinline__ int place(int x) {
    return (x & 4) * (N / 8) + (x >> 3) * 4 + (x & 3);
}

// Floats 8 jl .. 8 jl + 7 of such a table.
template <int N>
__device__ __forceinline__ void load8(const float* p, int jl, f2 (&f)[4]) {
    const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(p + 4 * jl);
    const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(p + N / 2 + 4 * jl);
    f[0] = a.x;
    f[1] = a.y;
    f[2] = b.x;
    f[3] = b.y;
}

}  // namespace pkv

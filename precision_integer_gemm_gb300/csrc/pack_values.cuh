// The values of a matrix that is packed, as they are read: used by the packing kernels.
#pragma once
#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "ptx.cuh"

namespace igemm {

__device__ __forceinline__ float fp4_float(float v) { return v; }
__device__ __forceinline__ float fp4_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float fp4_float(__half v) { return __half2float(v); }

// The two values of a word of 16-bit ones.
template <class T>
__device__ __forceinline__ void fp4_floats(uint32_t w, float &lo, float &hi)
{
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        lo = __uint_as_float(w << 16);
        hi = __uint_as_float(w & 0xFFFF0000u);
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        lo = f.x;
        hi = f.y;
    }
}

// max(|a|, |b|) of each half, NaN where one is (the result's signs mean nothing).
template <class T>
__device__ __forceinline__ uint32_t fp4_absmax2(uint32_t a, uint32_t b)
{
    uint32_t r;
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// a *= f, b *= f as one pair (each rounded as a product of its own).
__device__ __forceinline__ void fp4_mul2(float &a, float &b, float f)
{
    asm("{\n\t.reg .b64 v, w;\n\t"
        "mov.b64 v, {%0, %1};\n\t"
        "mov.b64 w, {%2, %2};\n\t"
        "mul.rn.f32x2 v, v, w;\n\t"
        "mov.b64 {%0, %1}, v;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(f));
}

// 16 values of one row from k (zeros past K), as they lie in memory.  VEC: every row
// starts on 16 bytes.  Otherwise the 16-byte pieces that the values lie in are taken
// as they are, one more than there are words for, and moved into place when the
// values are wanted; the row's ends, where a piece would reach past it, go value by
// value.  (16384 x 8191: bfloat16 127 -> 80 us, float32 237 -> 100 us against values
// one by one.)
template <class T, bool VEC>
struct Fp4Raw {
    static constexpr int kWords = 4 * sizeof(T);
    static constexpr int kLoaded = kWords + (VEC ? 0 : 4);
    uint32_t w[kLoaded];
    uint32_t shift;  // (!VEC) bytes from the first piece to the values
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kLoaded; ++i) w[i] = 0;
        shift = 0;
    }
    __device__ __forceinline__ void load(const T *row, int k, int K)
    {
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + k);
        const uintptr_t first = VEC ? at : at & ~uintptr_t(15);
        constexpr int kPieces = kLoaded / 4;
        const bool whole = VEC ? k + 16 <= K
                               : first >= reinterpret_cast<uintptr_t>(row) &&
                                     first + 16 * kPieces <= reinterpret_cast<uintptr_t>(row + K);
        if (whole) {
            if constexpr (!VEC) shift = static_cast<uint32_t>(at - first);
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                // (!VEC: volatile, 16384 x 8191 float32 100 us against 105 with plain loads)
                const uint4 *piece = reinterpret_cast<const uint4 *>(first) + i;
                const uint4 q = VEC ? *piece : ld_v4(piece);
                w[4 * i] = q.x;
                w[4 * i + 1] = q.y;
                w[4 * i + 2] = q.z;
                w[4 * i + 3] = q.w;
            }
        } else {
            zero();
            const auto bits = [&](int i) -> uint32_t {
                if (k + i >= K) return 0;
                if constexpr (sizeof(T) == 4) return __float_as_uint(row[k + i]);
                else return reinterpret_cast<const uint16_t *>(row)[k + i];
            };
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                if constexpr (sizeof(T) == 4) w[i] = bits(i);
                else w[i] = bits(2 * i) | bits(2 * i + 1) << 16;
            }
        }
    }
    __device__ __forceinline__ void place()
    {
        if constexpr (!VEC) {
#pragma unroll
            for (int i = 0; i < kWords + 2; ++i) w[i] = shift & 8 ? w[i + 2] : w[i];
#pragma unroll
            for (int i = 0; i < kWords + 1; ++i) w[i] = shift & 4 ? w[i + 1] : w[i];
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int i = 0; i < kWords; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 8 * (shift & 2));
            }
        }
    }
    // Once the values are there: the bits of the largest magnitude, of 16-bit values as
    // pairs; then the values.
    __device__ __forceinline__ uint32_t largest()
    {
        uint32_t amax = 0;
        place();
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 16; ++i) amax = max(amax, w[i] & 0x7FFFFFFFu);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fp4_absmax2<T>(amax, w[i]);
            amax = max(amax & 0x7FFFu, amax >> 16 & 0x7FFFu);
            const uint16_t top = static_cast<uint16_t>(amax);
            amax = __float_as_uint(fp4_float(*reinterpret_cast<const T *>(&top)));
        }
        return amax;
    }
    __device__ __forceinline__ void values(float (&v)[16]) const
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) fp4_floats<T>(w[i], v[2 * i], v[2 * i + 1]);
        }
    }
    __device__ __forceinline__ uint32_t unpack(float (&v)[16])
    {
        const uint32_t amax = largest();
        values(v);
        return amax;
    }
};

}  // namespace igemm

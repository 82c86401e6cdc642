// Device building blocks of the token-generation operators (attention over
// shared prefixes and bounded caches, cache eviction, draft verification).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace df11serve {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// The two 16-bit element types: their matrix-core products, their rounding
// from float32 (to nearest, ties to even), the bits of a non-finite value, the
// greatest number (kMost), and the power of two that a row's greatest probability is held as (kLift):
// float16 loses bits below 2^-14 and all of them below 2^-25, so its
// probabilities stand 2^7 higher (with the 2^8 that the running maximum may
// lag behind, 2^15 of at most 65504).
struct Bf16 {
    static constexpr uint32_t kExpMask = 0x7f80u;
    static constexpr float kLift = 0.0f, kMost = 0x1.fep127f;
    static __device__ __forceinline__ float value(uint32_t x) { return __builtin_bit_cast(float, x << 16); }
    static __device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)lo, (__bf16)hi});
    }
};

struct Fp16 {
    static constexpr uint32_t kExpMask = 0x7c00u;
    static constexpr float kLift = 7.0f, kMost = 65504.0f;
    static __device__ __forceinline__ float value(uint32_t x) { return (float)__builtin_bit_cast(_Float16, (uint16_t)x); }
    static __device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                      0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                      0, 0, 0);
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        return __builtin_bit_cast(uint32_t, f16x2{(_Float16)lo, (_Float16)hi});
    }
};

// A float's order as an unsigned integer: NaN 0, then -infinity .. +infinity
// (at most 0xff800000); -0 and +0 are equal.
__device__ __forceinline__ uint32_t order_of(float w)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, w + 0.0f);
    const uint32_t flip = (uint32_t)((int32_t)u >> 31) | 0x80000000u;   // all bits of a negative number, else the sign
    return w != w ? 0 : u ^ flip;
}

// A barrier for what lies in LDS: loads from memory stay on their way.
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Keys and values of a step in LDS, in rows of K and rows of V^T, 16-byte chunks
// exchanged so that neighbouring rows lie in different banks.
template <int DP>
struct TileShape {
    static constexpr int kKeys = 8192 / DP;          // keys of a step: 16 KB of K and of V
    static constexpr int kChunks = DP / 8;           // 16-byte chunks of a K row
    static constexpr int kKeyChunks = kKeys / 8;     // of a V^T row
    static constexpr int kBuffer = 2 * kKeys * DP * 2;
    static __device__ __forceinline__ int k_at(int key, int chunk)
    {
        const int x = DP == 64 ? (key >> 1) & 7 : key & 15;
        return key * DP * 2 + (chunk ^ x) * 16;
    }
    static __device__ __forceinline__ int v_at(int d, int chunk)
    {
        const int x = DP == 64 ? (d ^ (d >> 4)) & 15 : DP == 128 ? ((d >> 1) ^ (d >> 4)) & 7 : ((d >> 2) ^ (d >> 4)) & 3;
        return kKeys * DP * 2 + d * kKeys * 2 + (chunk ^ x) * 16;
    }
    // The same places by exclusive or with one lane's first one: chunk + 2 i
    // of a K row (chunk < 2); dim d + i, i < 8, of V^T (d a multiple of 8);
    // dim d + 32 i and chunk + 2 j of V^T (d < 32, chunk < 2).
    static __device__ __forceinline__ int k_next(int first, int i) { return first ^ (2 * i * 16); }
    static __device__ __forceinline__ int v_next_dim(int first, int i)
    {
        return (first ^ ((DP == 64 ? i : DP == 128 ? i / 2 : i / 4) * 16)) + i * kKeys * 2;
    }
    static __device__ __forceinline__ int v_next(int first, int i, int j)
    {
        return (first ^ (((i ^ j) & (kKeyChunks / 2 - 1)) * 32)) + 32 * i * kKeys * 2;
    }
};

// A pointer for 16-byte loads and stores.
inline bool aligned16(const void *p) { return p && !((uintptr_t)p & 15); }

}  // namespace df11serve

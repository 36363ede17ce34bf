// paged_mma.cuh - pieces that the paged-attention kernels share: copies into shared
// memory, mma.sync with its operand loads, conversions.
#pragma once
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace moe {

// 16 bytes to shared memory without passing through registers, zeros if !valid
// (the source address is then not read).
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last N groups of this thread's copies have landed.
template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}

// d += a b, 16 x 8 x 16, in bf16 or (kHalf) fp16 with fp32 sums
template <bool kHalf>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (kHalf)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t bf16x2_of(float a, float b)
{
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&r);
}
// With a cache of codes p enters its product as fp16, whose smallest step is 2^-24.
// It is formed times 2^15 (its largest is 1) or 2^7 (2^8 where the maximum it is
// relative to may lag behind), and so is the sum of a row: the factor leaves with the
// quotient, and a weight may be 2^-32 of the largest before it is lost.  Plain, a
// quarter of a million keys of 2^-26 each, 2^-8 together, were.
constexpr float kF16Up = 15.0f, kF16UpLag = 7.0f;

// What a row's sums are divided by: 0 for a row that sees nothing.  A cache's scale is
// a factor of its own behind it, since their quotient may be too small for fp32 where
// neither the sum nor the result is.
__device__ __forceinline__ float row_inverse(float l) { return l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l; }

__device__ __forceinline__ uint32_t f16x2_of(float a, float b)
{
    const __half2 r = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ float lo_of(uint32_t bf16x2) { return __uint_as_float(bf16x2 << 16); }
__device__ __forceinline__ float hi_of(uint32_t bf16x2) { return __uint_as_float(bf16x2 & 0xFFFF0000u); }
// four E4M3 codes as fp16 values, exactly: codes 0 and 1 in lo, 2 and 3 in hi
__device__ __forceinline__ void f16x4_of_e4m3(uint32_t codes, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(codes));
}
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A query row meets an E4M3 cache as fp16 times a power of two that brings its
// largest magnitude to [2^14, 2^15): exact but for elements below 2^-28 of it.
// The power is 2^up (1 for a row with an infinity or NaN, which stay so).
__device__ __forceinline__ int row_power(float amax)
{
    // the exponent field of a normal amax; 0 and subnormals as 2^-126
    const int e = max(1, static_cast<int>(__float_as_uint(amax) >> 23)) - 127;
    return e == 128 ? 0 : min(126, 14 - e);
}
__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((127 + e) << 23); }

// 16-byte chunk c of row r of a tile with kChunks chunks a row, permuted so that
// the 8 rows an ldmatrix reads at one chunk lie in 8 different bank groups (the
// patterns of the 128- and 64-byte TMA swizzles)
template <int kChunks>
__device__ __forceinline__ int chunk_of(int r, int c)
{
    return kChunks >= 8 ? c ^ (r & 7) : c ^ ((r >> 1) & 3);
}

}  // namespace moe

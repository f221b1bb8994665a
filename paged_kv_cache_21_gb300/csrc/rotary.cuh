// Rotary positions, shared by the kernels that rotate queries and keys on their way
// into a cache or a query buffer (rotary_append.cu).
//
// Pair i of a vector is turned by the angle position * inv_freq[i].  At a position of
// a million the angle itself, in binary32, would be off by 0.03 radians; only its
// fraction of a turn matters, so that the frequency is held as a 64-bit fraction of a
// turn a position (2^64 = one turn) and the product with the position wraps: exact but
// for the frequency's rounding, less than 2^-63 of a turn a position.  Of the fraction,
// 32 bits go on to binary32's sine and cosine.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "device_common.cuh"

namespace pkv {

constexpr int kRotaryUnit = 16;          // elements, eight pairs, that a thread turns together

// Turns a position, of 2^64, for a frequency in radians: m 2^e of the float times
// 2^88 / (2 pi), with 32 bits behind the point, in integers (FP64 runs at 1/64 of FP32's rate
// here: in doubles the angles of 8192 tokens took 24 us of the kernel's 57).  Frequencies of 2^48
// and above, and what is not a number, count as zero.
__device__ __forceinline__ uint64_t rotary_step(float inv_freq)
{
    constexpr uint64_t kHi = 0x28be60ull, kLo = 0xdb9391054a7f09d5ull, kBehind = 0xf47d4d37ull;
    const uint32_t bits = __float_as_uint(inv_freq), ex = (bits >> 23) & 255u;
    const uint64_t m = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);
    const int shift = 174 - (int)(ex ? ex : 1u);         // 24 - e, e = ex - 150
    if (shift < 0 || shift >= 128) return 0ull;
    const uint64_t low = m * kLo, lo = low + (m * kBehind >> 32);
    const uint64_t hi = m * kHi + __umul64hi(m, kLo) + (lo < low ? 1u : 0u);
    const uint64_t step = shift >= 64 ? hi >> (shift - 64) : shift == 0 ? lo : (hi << (64 - shift)) | (lo >> shift);
    return bits >> 31 ? 0ull - step : step;
}

// magnitude * (cos, sin) of position * step.
__device__ __forceinline__ void rotary_angle(uint64_t step, int64_t position, float magnitude, float& c, float& s)
{
    const int32_t turn = (int32_t)((step * (uint64_t)position) >> 32);   // of 2^32
    sincospif((float)turn * 4.656612873077392578e-10f, &s, &c);          // 2^-31: half turns
    c *= magnitude;
    s *= magnitude;
}

// The two 16-byte pieces of unit u of a vector whose first `rot` elements are turned:
// element offsets.  Half layout: pair i is elements i and i + rot / 2, so the pieces
// are the pairs' two sides; interleaved, and behind `rot`: 16 elements in a row.
__device__ __forceinline__ void rotary_pieces(int u, int rot, bool interleaved, int& first, int& second)
{
    if (!interleaved && u * kRotaryUnit < rot) {
        first = u * 8;
        second = rot / 2 + u * 8;
    } else {
        first = u * kRotaryUnit;
        second = first + 8;
    }
}

// (cos, sin) of the n angles of a position, by a warp, for its lanes to take eights of.
__device__ __forceinline__ void rotary_table(const float* __restrict__ inv_freq, int n, int64_t position, float magnitude,
                                             float* cs, float* sn, int lane)
{
    for (int i = lane; i < n; i += 32) {
        float c, s;
        rotary_angle(rotary_step(__ldg(inv_freq + i)), position, magnitude, c, s);
        cs[i] = c;
        sn[i] = s;
    }
    __syncwarp();
}

__device__ __forceinline__ void rotary_take(const float* cs, const float* sn, int u, float (&c)[8], float (&s)[8])
{
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        const float4 a = *reinterpret_cast<const float4*>(cs + 8 * u + i), b = *reinterpret_cast<const float4*>(sn + 8 * u + i);
        c[i] = a.x; c[i + 1] = a.y; c[i + 2] = a.z; c[i + 3] = a.w;
        s[i] = b.x; s[i + 1] = b.y; s[i + 2] = b.z; s[i + 3] = b.w;
    }
}

// Turn a unit: x (16 elements as loaded from the two pieces) -> y in the same order.
__device__ __forceinline__ void rotary_turn(const float (&x)[16], const float (&c)[8], const float (&s)[8],
                                            bool interleaved, float (&y)[16])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = interleaved ? x[2 * i] : x[i], b = interleaved ? x[2 * i + 1] : x[8 + i];
        const float p = a * c[i] - b * s[i], q = b * c[i] + a * s[i];
        if (interleaved) {
            y[2 * i] = p;
            y[2 * i + 1] = q;
        } else {
            y[i] = p;
            y[8 + i] = q;
        }
    }
}

__device__ __forceinline__ void unpack8(uint4 v, float* x)
{
    x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x); x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
    x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z); x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint4 pack8(const float* x)
{
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

// Eight E4M3 codes of x / s (device_common.cuh's quantize8_e4m3, from binary32).
__device__ __forceinline__ uint2 quantize8_f32(const float* x, float s)
{
    uint32_t packed[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float2 a = make_float2(__fdiv_rn(x[4 * j], s), __fdiv_rn(x[4 * j + 1], s));
        const float2 b = make_float2(__fdiv_rn(x[4 * j + 2], s), __fdiv_rn(x[4 * j + 3], s));
        packed[j] = (uint32_t)__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3) |
                    ((uint32_t)__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3) << 16);
    }
    return make_uint2(packed[0], packed[1]);
}

}  // namespace pkv

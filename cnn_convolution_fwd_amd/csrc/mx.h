// Microscaled 4-bit floating point (MXFP4): host entry points behind the
// cfwd_mx_* calls of cfwd.h, and the device helpers that the kernels which
// read or write MXFP4 share.
//
// Mathematics.  32 consecutive values of a row share the scale 2^(e - 127).
// With E the biased fp32 exponent of the block's largest magnitude,
// e = max(E - 2, 0): E2M1's largest exponent is 2, so the scaled block lies
// in (-8, 8) and its largest magnitude in [4, 8), of which what is above 6
// saturates.  E = 255 (a NaN or an infinity in the block) gives e = 255, NaN,
// and codes of 0, so that the whole block, and every product with it, is NaN.
// A scaled value becomes the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (a tie to
// the even code), its sign kept (code bit 3).  gfx950's conversion instruction
// does exactly that: the tests hold it to the definition, bit for bit, over every
// bf16 value up to six binades below its block's largest, fp32 ties and their
// neighbours, and 2^20 random fp32 values.
#pragma once

#include "internal.h"

#include <atomic>
#include <type_traits>

namespace cfwd {

// A positive number that belongs to a device, asked for once on each.
class PerDevice {
    std::atomic<long long> known_[64] = {};

public:
    // of the current device; ask() gives it, or 0 where it cannot, and then `otherwise` stands
    template <typename Ask>
    long long get(Ask ask, long long otherwise) {
        int dev = 0;
        if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return otherwise;
        long long n = known_[dev].load(std::memory_order_relaxed);
        if (n == 0 && (n = ask(dev)) > 0) known_[dev].store(n, std::memory_order_relaxed);
        return n > 0 ? n : otherwise;
    }
};

int compute_units();  // of the current device

inline long long mx_blocks(long long k) { return (k + 31) / 32; }
// bytes of one row: codes (16 for each block), scales (a whole number of words)
inline long long mx_code_pitch(long long k) { return mx_blocks(k) * 16; }
inline long long mx_scale_pitch(long long k) { return (mx_blocks(k) + 3) / 4 * 4; }

// x [rows][k] of dtype (row pitch x_stride elements) -> codes and scales
cfwd_status mx_quantize(long long rows, int k, cfwd_dtype dtype, const void* x, long long x_stride, void* codes,
                        void* scales, hipStream_t st);
// codes and scales -> y [rows][k] of dtype
cfwd_status mx_dequantize(long long rows, int k, cfwd_dtype dtype, const void* codes, const void* scales, void* y,
                          hipStream_t st);

// Workspace of the product: the quantised x where x is not MXFP4, then partial sums.
size_t mx_matmul_workspace(const cfwd_mx_matmul_desc* d);
cfwd_status mx_matmul(const cfwd_mx_matmul_desc* d, const void* x, const void* x_scales, const void* w,
                      const void* w_scales, const float* bias, void* y, void* y_scales, void* workspace,
                      hipStream_t st);

#if defined(__HIPCC__)
namespace mx {

// Division of n < 2^31 by a fixed d as a multiply-high and a shift (the
// round-up reciprocal, exact for all such n).
struct Divisor {
    uint32_t mul, shift, d;
};

inline Divisor divisor(uint32_t d) {
    Divisor r{0, 0, d};
    while ((1ull << r.shift) < d) ++r.shift;
    r.mul = static_cast<uint32_t>(((1ull << (31 + r.shift)) + d - 1) / d);
    return r;
}

__device__ __forceinline__ uint32_t divide(uint32_t n, const Divisor& v) {
    return static_cast<uint32_t>((static_cast<uint64_t>(n) * v.mul) >> (31 + v.shift));
}

// 16 and 8 bytes at any address that suits the element type: the compiler
// uses whole loads and stores, which the hardware splits where it must.
struct __attribute__((packed, aligned(2))) Raw16 {
    uint32_t w[4];
};

// 8 consecutive values from p, of which the first `valid` (at most 8) exist;
// the others are 0.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int valid, float (&v)[8]);

template <>
__device__ __forceinline__ void load8<float>(const float* p, int valid, float (&v)[8]) {
    if (valid >= 8) {
        const Raw16 a = *reinterpret_cast<const Raw16*>(p), b = *reinterpret_cast<const Raw16*>(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = __uint_as_float(a.w[i]);
            v[i + 4] = __uint_as_float(b.w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < valid ? p[i] : 0.0f;
    }
}

template <>
__device__ __forceinline__ void load8<bf16_t>(const bf16_t* p, int valid, float (&v)[8]) {
    if (valid >= 8) {
        const Raw16 a = *reinterpret_cast<const Raw16*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(a.w[i] << 16);
            v[2 * i + 1] = __uint_as_float(a.w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < valid ? bf16_to_float(p[i].bits) : 0.0f;
    }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, int valid, const float (&v)[8]);

template <>
__device__ __forceinline__ void store8<float>(float* p, int valid, const float (&v)[8]) {
    if (valid >= 8) {
        Raw16 a, b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a.w[i] = __float_as_uint(v[i]);
            b.w[i] = __float_as_uint(v[i + 4]);
        }
        *reinterpret_cast<Raw16*>(p) = a;
        *reinterpret_cast<Raw16*>(p + 4) = b;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < valid) p[i] = v[i];
    }
}

template <>
__device__ __forceinline__ void store8<bf16_t>(bf16_t* p, int valid, const float (&v)[8]) {
    if (valid >= 8) {
        Raw16 a;
#pragma unroll
        for (int i = 0; i < 4; ++i) a.w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        *reinterpret_cast<Raw16*>(p) = a;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < valid) p[i].bits = float_to_bf16(v[i]);
    }
}

// Largest magnitude as its bit pattern: unlike fmaxf, integer maxima keep a
// NaN (whose pattern is above every number's).
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Exponent byte of a block from its largest magnitude's bit pattern.
__device__ __forceinline__ uint32_t exponent_byte(uint32_t amax_bits) {
    const int e = static_cast<int>(amax_bits >> 23);
    return e == 255 ? 255u : static_cast<uint32_t>(max(e - 2, 0));
}

// 2^(byte - 127); a NaN for 255.
__device__ __forceinline__ float scale_of(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23);
}

// Codes of 8 values under a block's exponent byte, the first in the lowest bits.
__device__ __forceinline__ uint32_t encode8(const float (&v)[8], uint32_t byte) {
    const float s = scale_of(byte);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
    return byte == 255 ? 0u : c;
}

// Largest of a value over the quad of lanes (4 i .. 4 i + 3), every lane of
// which must run this: two DPP moves.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xB1, 0xF, 0xF, false)));
    return max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x4E, 0xF, 0xF, false)));
}

// A thread's 8 values of a block that a quad of lanes holds -> their codes
// and the block's exponent byte.
__device__ __forceinline__ uint32_t quantize8(const float (&v)[8], uint32_t* byte) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
    *byte = exponent_byte(quad_max(m));
    return encode8(v, *byte);
}

// Activations in fp32.  NaN stays NaN.  silu(v) = v / (1 + e^-v); gelu is the
// form with tanh, 0.5 v (1 + tanh z) = v / (1 + e^-2z), z = sqrt(2 / pi) (v +
// 0.044715 v^3); the powers of 2 are taken directly, with log2(e) in the constants.
//
// The argument of a power of 2, rounded once, costs the power a relative error
// that grows with it: of silu 2.4 units of 2^-24 (rms) for v in [-8, -2], 6 in
// [-20, -8], 63 at most at -80.  A bf16 or 4-bit result, rounded to 2^-9 or
// 2^-3, does not show that.  An fp32 silu does, so it takes the argument apart
// into a whole number and what is left of it, under 1/2 and rounded there (under
// 6.4 units in all; six more instructions a value, 3 to 12% of a product with many rows).  An fp32 gelu stays as it
// is: below -2, where the power counts, the form with tanh loses more to 1 + tanh.
// Both are 0 from where 1 + e^.. passes 2^126 on (silu: v < -87.3, results under 2^-119).
__device__ __forceinline__ float silu_exponent(float v) { return -1.44269504f * v; }
__device__ __forceinline__ float gelu_exponent(float v) { return v * (-2.30220820f - 0.10294324f * (v * v)); }

// e^-v = 2^f 2^n.  n stays finite, so that v = inf gives f = -inf and not NaN.
__device__ __forceinline__ float silu_whole(float v) {
    return __builtin_amdgcn_fmed3f(__builtin_rintf(silu_exponent(v)), -1024.0f, 1024.0f);
}
__device__ __forceinline__ float silu_rest(float v, float n) {
    return __builtin_fmaf(v, -1.92596299e-8f, __builtin_fmaf(v, -1.44269504f, -n));  // log2(e) in two parts
}

// TY: float for a result that stays in fp32
template <typename TY>
__device__ __forceinline__ float activate(float v, int act) {
    if (act == CFWD_ACT_RELU) return v < 0.0f ? 0.0f : v;
    if (act == CFWD_ACT_SILU) {
        if constexpr (std::is_same<TY, float>::value) {
            const float n = silu_whole(v), e = __builtin_amdgcn_exp2f(silu_rest(v, n));
            return v * __builtin_amdgcn_rcpf(1.0f + __builtin_ldexpf(e, static_cast<int>(n)));
        }
        return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(silu_exponent(v)));
    }
    if (act == CFWD_ACT_GELU) return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(gelu_exponent(v)));
    return v;
}

}  // namespace mx
#endif

}  // namespace cfwd

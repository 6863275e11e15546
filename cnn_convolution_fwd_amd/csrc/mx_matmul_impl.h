// Device pieces that the kernels of the MXFP4 product share (k_mx_matmul.hip):
// addressing of the operands, and the output pass.
//
// The product runs on v_mfma_scale_f32_32x32x64_f8f6f4 with w as the A operand
// and x as B: a lane of half h = lane / 32 holds one block (32 values, 16
// bytes) of row lane % 32 of each, with the block's scale byte, and ends with
// 16 outputs of one row of y: columns 8 g + 4 h + i (g, i < 4) of 32.
//
// A K step ("stage") is 256 values, 8 blocks, as four such instructions.  The
// order of the sum is free as long as both operands agree, so half h takes
// the stage's blocks 4 h .. 4 h + 3, one an instruction: their four scale
// bytes are then one aligned word, and each instruction names its byte.
#pragma once

#include "mx.h"

#include <type_traits>

namespace cfwd {
namespace mx {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct MatmulParams {
    const uint8_t *x, *xs, *w, *ws;  // x: codes, or (stream kernel) values of x_stride elements a row
    long long x_stride;
    int k;
    const float* bias;
    void* y;
    uint8_t* ys;
    long long m;
    int n, kb;  // kb: blocks of a row
    int pitch, spitch;  // bytes of a row of codes / scales of x and w
    int act;
    int y_pitch, y_spitch;  // MXFP4 outputs
};

constexpr uint32_t kOutOfRange = 0x7ffffff0u;  // a buffer offset past every range: loads give 0

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, long long bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0,
                                             static_cast<int>(bytes < 0 ? 0 : bytes > 0x7fffffe0ll ? 0x7fffffe0ll : bytes),
                                             0x00020000);
}

template <int J>
__device__ __forceinline__ f32x16 mfma(const i32x4& a, const i32x4& b, const f32x16& c, int sa, int sb) {
    const i32x8 a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, b8 = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, J, sa, J, sb);
}

// The output pass of one wave's 32 rows of y x 32 FN columns: bias,
// activation, rounding, and a turn through the wave's own LDS area so that
// whole runs of columns are stored.  TY: float, bf16_t, or void for MXFP4.
template <int FN, typename TY>
constexpr int out_area() {  // bytes of the wave's LDS area
    return std::is_void<TY>::value ? 32 * (FN * 16 + 16) + 32 * FN
                                   : 32 * (FN * 32 * (std::is_same<TY, float>::value ? 4 : 2) + 16);
}

template <int FN, typename TY>
__device__ __forceinline__ void write_rows(const f32x16 (&acc)[FN], const MatmulParams& p, long long m0, int n0,
                                           uint8_t* area) {
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    const __amdgpu_buffer_rsrc_t bias = buffer(p.bias, p.bias ? p.n * 4ll : 0);
    if constexpr (!std::is_void<TY>::value) {
        constexpr int ES = sizeof(TY), PITCH = FN * 32 * ES + 16;
#pragma unroll
        for (int f = 0; f < FN; ++f)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int c = f * 32 + g * 8 + h * 4;
                const i32x4 q = __builtin_bit_cast(
                    i32x4, __builtin_amdgcn_raw_buffer_load_b128(bias, (n0 + c) * 4, 0, 0));
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = activate(acc[f][g * 4 + i] + __int_as_float(q[i]), p.act);
                if constexpr (ES == 4)
                    *reinterpret_cast<float4*>(area + r * PITCH + c * 4) = make_float4(v[0], v[1], v[2], v[3]);
                else
                    *reinterpret_cast<uint2*>(area + r * PITCH + c * 2) =
                        make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
            }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        constexpr int RUN = 16 / ES, RUNS = FN * 32 / RUN;  // 16-byte runs of a row
#pragma unroll
        for (int i = 0; i < RUNS / 2; ++i) {
            const int u = i * 64 + lane, row = u / RUNS, c = u % RUNS * RUN;
            const Raw16 t = *reinterpret_cast<const Raw16*>(__builtin_assume_aligned(area + row * PITCH + c * ES, 16));
            const long long m = m0 + row;
            const int valid = p.n - (n0 + c);
            if (m >= p.m || valid <= 0) continue;
            TY* dst = static_cast<TY*>(p.y) + m * p.n + n0 + c;
            if (valid >= RUN) {
                *reinterpret_cast<Raw16*>(dst) = t;
            } else {
#pragma unroll
                for (int j = 0; j < RUN; ++j)
                    if (j < valid) {
                        if constexpr (ES == 4)
                            dst[j] = __uint_as_float(t.w[j]);
                        else
                            dst[j].bits = static_cast<uint16_t>(t.w[j / 2] >> (j % 2 * 16));
                    }
            }
        }
    } else {
        constexpr int PITCH = FN * 16 + 16;
        uint8_t* sarea = area + 32 * PITCH;
#pragma unroll
        for (int f = 0; f < FN; ++f) {
            const int nb = n0 + f * 32;
            float v[16];
            uint32_t top = 0;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int n = nb + g * 8 + h * 4;
                const i32x4 q =
                    __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(bias, n * 4, 0, 0));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float t = activate(acc[f][g * 4 + i] + __int_as_float(q[i]), p.act);
                    v[g * 4 + i] = n + i < p.n ? t : 0.0f;  // a column past the row is no part of its block
                    top = max(top, abs_bits(v[g * 4 + i]));
                }
            }
            top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32)));
            const uint32_t byte = nb < p.n ? exponent_byte(top) : 127u;
            const float s = scale_of(byte);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                uint32_t c = 0;
                c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[g * 4], v[g * 4 + 1], s, 0);
                c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[g * 4 + 2], v[g * 4 + 3], s, 1);
                *reinterpret_cast<uint16_t*>(area + r * PITCH + f * 16 + g * 4 + h * 2) =
                    byte == 255 ? 0 : static_cast<uint16_t>(c);
            }
            if (h == 0) sarea[r * FN + f] = static_cast<uint8_t>(byte);
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < (FN + 1) / 2; ++i) {  // one block of one row a lane
            const int u = i * 64 + lane, row = u / FN, f = u % FN;
            const long long m = m0 + row;
            if (u < 32 * FN && m < p.m && n0 + f * 32 < p.n)
                *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.y) + m * p.y_pitch + (n0 / 32 + f) * 16) =
                    *reinterpret_cast<const uint4*>(area + row * PITCH + f * 16);
            if (u < 32 * FN && m < p.m && n0 / 32 + f < p.y_spitch)
                p.ys[m * p.y_spitch + n0 / 32 + f] = sarea[row * FN + f];
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();  // the area is written again only after every lane has read it
}

}  // namespace mx

// Few rows (k_mx_stream.hip).  `x`: MXFP4, or x's own type where mx_stream_takes_raw says so.
bool mx_stream_supported(long long m);
bool mx_stream_takes_raw(long long m, int k);
cfwd_status mx_stream(const mx::MatmulParams& p, cfwd_dtype x, cfwd_dtype y, hipStream_t st);

}  // namespace cfwd

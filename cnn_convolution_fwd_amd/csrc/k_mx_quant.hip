// Quantisation to MXFP4 and back (gfx950).
//
// Both directions are one pass: a thread owns 8 consecutive values of a row
// (16 bytes of bf16), four adjacent lanes a block of 32, whose largest
// magnitude they find with two cross-lane moves.  Bound by HBM traffic (100352 x
// 256 in bf16, 64 MB: 11.3 to 13.1 us one way, 11.2 to 11.7 back, 5 to 6 TB/s with part of
// it from the last-level cache); at small sizes by the launch (1.7 us).
#include "mx.h"

#include <algorithm>

namespace cfwd {
namespace mx {

// unit = (row, 8 values of it); `units` of them, quads of a row's padding included
template <typename T>
__global__ __launch_bounds__(256) void quantize_kernel(const T* __restrict__ x, long long x_stride, int k,
                                                       Divisor per_row, uint32_t units, int scale_pitch,
                                                       uint32_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    const uint32_t u = blockIdx.x * 256u + threadIdx.x;
    if (u >= units) return;  // units is a multiple of 4: whole quads leave
    const uint32_t row = divide(u, per_row), q = u - row * per_row.d;
    float v[8];
    load8(x + static_cast<long long>(row) * x_stride + q * 8, k - static_cast<int>(q * 8), v);
    uint32_t byte;
    codes[u] = quantize8(v, &byte);
    if ((q & 3) == 0) {
        uint8_t* s = scales + static_cast<long long>(row) * scale_pitch;
        s[q >> 2] = static_cast<uint8_t>(byte);
        if (q + 4 == per_row.d)  // the last block also writes what rounds the row up to whole words
            for (int i = per_row.d / 4; i < scale_pitch; ++i) s[i] = 127;
    }
}

template <typename T>
__global__ __launch_bounds__(256) void dequantize_kernel(const uint32_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales, int k, Divisor per_row,
                                                         uint32_t units, int scale_pitch, T* __restrict__ y) {
    const uint32_t u = blockIdx.x * 256u + threadIdx.x;
    if (u >= units) return;
    const uint32_t row = divide(u, per_row), q = u - row * per_row.d;
    const uint32_t c = codes[u];
    const float s = scale_of(scales[static_cast<long long>(row) * scale_pitch + (q >> 2)]);
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    const f32x2_t p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3)};
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[i / 2][i % 2] * s;  // exact: at most two significant bits
    const int valid = k - static_cast<int>(q * 8);
    if (valid > 0) store8(y + static_cast<long long>(row) * k + q * 8, valid, v);
}

// rows of one launch: fewer than 2^31 units
inline long long rows_per_launch(int k) { return ((1ll << 31) - 4) / (mx_blocks(k) * 4); }

}  // namespace mx

cfwd_status mx_quantize(long long rows, int k, cfwd_dtype dtype, const void* x, long long x_stride, void* codes,
                        void* scales, hipStream_t st) {
    const int per_row = static_cast<int>(mx_blocks(k) * 4), sp = static_cast<int>(mx_scale_pitch(k));
    const mx::Divisor dv = mx::divisor(per_row);
    for (long long r0 = 0; r0 < rows; r0 += mx::rows_per_launch(k)) {
        const long long r = std::min(rows - r0, mx::rows_per_launch(k));
        const uint32_t units = static_cast<uint32_t>(r * per_row), grid = (units + 255) / 256;
        uint32_t* c = static_cast<uint32_t*>(codes) + r0 * per_row;
        uint8_t* s = static_cast<uint8_t*>(scales) + r0 * sp;
        if (dtype == CFWD_F32)
            mx::quantize_kernel<float><<<grid, 256, 0, st>>>(static_cast<const float*>(x) + r0 * x_stride, x_stride, k,
                                                             dv, units, sp, c, s);
        else
            mx::quantize_kernel<bf16_t><<<grid, 256, 0, st>>>(static_cast<const bf16_t*>(x) + r0 * x_stride, x_stride,
                                                              k, dv, units, sp, c, s);
        const cfwd_status e = check_hip(hipGetLastError(), "MXFP4 quantisation launch");
        if (e != CFWD_OK) return e;
    }
    return CFWD_OK;
}

cfwd_status mx_dequantize(long long rows, int k, cfwd_dtype dtype, const void* codes, const void* scales, void* y,
                          hipStream_t st) {
    const int per_row = static_cast<int>(mx_blocks(k) * 4), sp = static_cast<int>(mx_scale_pitch(k));
    const mx::Divisor dv = mx::divisor(per_row);
    for (long long r0 = 0; r0 < rows; r0 += mx::rows_per_launch(k)) {
        const long long r = std::min(rows - r0, mx::rows_per_launch(k));
        const uint32_t units = static_cast<uint32_t>(r * per_row), grid = (units + 255) / 256;
        const uint32_t* c = static_cast<const uint32_t*>(codes) + r0 * per_row;
        const uint8_t* s = static_cast<const uint8_t*>(scales) + r0 * sp;
        if (dtype == CFWD_F32)
            mx::dequantize_kernel<float><<<grid, 256, 0, st>>>(c, s, k, dv, units, sp, static_cast<float*>(y) + r0 * k);
        else
            mx::dequantize_kernel<bf16_t><<<grid, 256, 0, st>>>(c, s, k, dv, units, sp,
                                                                static_cast<bf16_t*>(y) + r0 * k);
        const cfwd_status e = check_hip(hipGetLastError(), "MXFP4 dequantisation launch");
        if (e != CFWD_OK) return e;
    }
    return CFWD_OK;
}

}  // namespace cfwd

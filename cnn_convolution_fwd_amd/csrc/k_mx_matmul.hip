// Product of two MXFP4 matrices (gfx950): y = act(x w^T + bias).
#include "mx_matmul_impl.h"

#include <algorithm>
#include <type_traits>

namespace cfwd {
namespace mx {

// One workgroup: 128 rows of y x 128 columns, each of its four waves 64 x 64;
// the operands come straight from memory into registers.
template <typename TY>
__global__ __launch_bounds__(256) void tile_kernel(MatmulParams p) {
    __shared__ __attribute__((aligned(16))) uint8_t area[4 * out_area<2, TY>()];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 31, h = lane >> 5;
    const int tiles_n = (p.n + 127) / 128;
    const long long m0 = static_cast<long long>(blockIdx.x / tiles_n) * 128 + (wave >> 1) * 64;
    const int n0 = static_cast<int>(blockIdx.x % tiles_n) * 128 + (wave & 1) * 64;
    const long long rows_x = min(64ll, p.m - m0), rows_w = min(64, p.n - n0);
    const __amdgpu_buffer_rsrc_t x = buffer(p.x + m0 * p.pitch, rows_x * p.pitch),
                                 xs = buffer(p.xs + m0 * p.spitch, rows_x * p.spitch),
                                 w = buffer(p.w + static_cast<long long>(n0) * p.pitch, rows_w * p.pitch),
                                 ws = buffer(p.ws + static_cast<long long>(n0) * p.spitch, rows_w * p.spitch);
    f32x16 acc[2][2] = {};  // [32 rows of y][32 columns]
    for (int b0 = 0; b0 < p.kb; b0 += 8) {
        int sx[2], sw[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const int row = f * 32 + r, b = b0 + 4 * h;
            const int off = b < p.spitch ? row * p.spitch + b : kOutOfRange;
            sx[f] = __builtin_amdgcn_raw_buffer_load_b32(xs, off, 0, 0);
            sw[f] = __builtin_amdgcn_raw_buffer_load_b32(ws, off, 0, 0);
        }
        i32x4 ax[4][2], aw[4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const int row = f * 32 + r, b = b0 + 4 * h + j;
                const int off = b < p.kb ? row * p.pitch + b * 16 : kOutOfRange;
                ax[j][f] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(x, off, 0, 0));
                aw[j][f] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(w, off, 0, 0));
            }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                acc[i][f] = mfma<0>(aw[0][f], ax[0][i], acc[i][f], sw[f], sx[i]);
                acc[i][f] = mfma<1>(aw[1][f], ax[1][i], acc[i][f], sw[f], sx[i]);
                acc[i][f] = mfma<2>(aw[2][f], ax[2][i], acc[i][f], sw[f], sx[i]);
                acc[i][f] = mfma<3>(aw[3][f], ax[3][i], acc[i][f], sw[f], sx[i]);
            }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
        write_rows<2, TY>(acc[i], p, m0 + i * 32, n0, area + wave * out_area<2, TY>());
}

}  // namespace mx

namespace {
size_t round256(size_t v) { return (v + 255) / 256 * 256; }
}  // namespace

size_t mx_matmul_workspace(const cfwd_mx_matmul_desc* d) {
    if (d->x_dtype == CFWD_MXFP4) return 0;
    return round256(static_cast<size_t>(d->m) * mx_code_pitch(d->k)) + round256(static_cast<size_t>(d->m) * mx_scale_pitch(d->k));
}

cfwd_status mx_matmul(const cfwd_mx_matmul_desc* d, const void* x, const void* x_scales, const void* w,
                      const void* w_scales, const float* bias, void* y, void* y_scales, void* workspace,
                      hipStream_t st) {
    mx::MatmulParams p{};
    if (d->x_dtype != CFWD_MXFP4) {
        uint8_t* codes = static_cast<uint8_t*>(workspace);
        uint8_t* scales = codes + round256(static_cast<size_t>(d->m) * mx_code_pitch(d->k));
        const cfwd_status s = mx_quantize(d->m, d->k, d->x_dtype, x, d->x_stride, codes, scales, st);
        if (s != CFWD_OK) return s;
        x = codes;
        x_scales = scales;
    }
    p.x = static_cast<const uint8_t*>(x);
    p.xs = static_cast<const uint8_t*>(x_scales);
    p.w = static_cast<const uint8_t*>(w);
    p.ws = static_cast<const uint8_t*>(w_scales);
    p.bias = bias;
    p.y = y;
    p.ys = static_cast<uint8_t*>(y_scales);
    p.m = d->m;
    p.n = d->n;
    p.kb = static_cast<int>(mx_blocks(d->k));
    p.pitch = static_cast<int>(mx_code_pitch(d->k));
    p.spitch = static_cast<int>(mx_scale_pitch(d->k));
    p.act = d->act;
    p.y_pitch = static_cast<int>(mx_code_pitch(d->n));
    p.y_spitch = static_cast<int>(mx_scale_pitch(d->n));
    const long long tiles = (d->m + 127) / 128 * ((d->n + 127) / 128);
    const unsigned grid = static_cast<unsigned>(tiles);
    if (d->y_dtype == CFWD_F32)
        mx::tile_kernel<float><<<grid, 256, 0, st>>>(p);
    else if (d->y_dtype == CFWD_BF16)
        mx::tile_kernel<bf16_t><<<grid, 256, 0, st>>>(p);
    else
        mx::tile_kernel<void><<<grid, 256, 0, st>>>(p);
    return check_hip(hipGetLastError(), "MXFP4 product launch");
}

}  // namespace cfwd

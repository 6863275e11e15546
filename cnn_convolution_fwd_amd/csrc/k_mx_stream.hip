// Product of two MXFP4 matrices for few rows of y (gfx950): the weights are
// read once, straight into registers.
//
// With few rows the time is the weights' bytes, so what counts is how many of
// them are on their way at once.  A workgroup owns 16 NF columns of y (rows of
// w) and all of its rows; its eight waves share the sum over K among them and
// meet in LDS.  A wave requests all fragments of several K steps (up to 16 KB
// of w) before it uses the first.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 with w as A and x as B: lane l holds block
// l / 16 of the K step's four of row l % 16, of each operand, and ends with
// columns 4 (l / 16) .. + 3 of y's row l % 16.  An x in 16 or 32 bits is
// quantised on the way: a lane needs one whole block, so it reads the block's
// 32 values and finds their scale without any exchange.
#include "mx_matmul_impl.h"

#include <type_traits>

namespace cfwd {
namespace mx {

constexpr int kWaves = 8;

// An MXFP4 block's codes and scale byte from 32 values of x, the first at x[col].
template <typename T>
__device__ __forceinline__ i32x4 quantize32(const T* x, int valid, int* byte) {
    float v[4][8];
    uint32_t top = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        load8(x + q * 8, valid - q * 8, v[q]);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, abs_bits(v[q][i]));
    }
    const uint32_t e = exponent_byte(top);
    *byte = static_cast<int>(e);
    return i32x4{static_cast<int>(encode8(v[0], e)), static_cast<int>(encode8(v[1], e)),
                 static_cast<int>(encode8(v[2], e)), static_cast<int>(encode8(v[3], e))};
}

// MT: 16-row tiles of y.  TX: void for MXFP4, else x's type (p.x, p.x_stride
// elements a row).  TY as in write_rows.
template <int MT, int NF, typename TX, typename TY>
__global__ __launch_bounds__(64 * kWaves) void stream_kernel(MatmulParams p) {
    constexpr int STEPS = 20 / (NF + MT);  // K steps in flight: what 100 registers of operands and scales hold
    constexpr int ROW = NF * 16 + 4;       // floats of a row of partial sums, padded against bank conflicts
    __shared__ __attribute__((aligned(16))) float part[kWaves][MT * 16 * ROW];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = xcd_linear(blockIdx.x, gridDim.x) * (16 * NF);
    const long long rows_w = min(16 * NF, p.n - n0);
    const int m = static_cast<int>(p.m);
    const __amdgpu_buffer_rsrc_t w = buffer(p.w + static_cast<long long>(n0) * p.pitch, rows_w * p.pitch),
                                 ws = buffer(p.ws + static_cast<long long>(n0) * p.spitch, rows_w * p.spitch),
                                 x = buffer(p.x, static_cast<long long>(m) * p.pitch),
                                 xs = buffer(p.xs, static_cast<long long>(m) * p.spitch);
    f32x4 acc[MT][NF] = {};
    const int steps = (p.kb + 3) / 4;
    for (int s0 = wave; s0 < steps; s0 += kWaves * STEPS) {
        i32x4 a[STEPS][NF], cx[STEPS][MT];
        int sa[STEPS][NF], sx[STEPS][MT];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {  // steps past the end load nothing and multiply zeros
            const int b = (s0 + s * kWaves) * 4 + g;
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                const int row = f * 16 + r;
                a[s][f] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                        w, b < p.kb ? row * p.pitch + b * 16 : kOutOfRange, 0, 0));
                sa[s][f] = __builtin_amdgcn_raw_buffer_load_b8(ws, b < p.kb ? row * p.spitch + b : kOutOfRange, 0, 0);
            }
            if constexpr (std::is_void<TX>::value)
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const int row = t * 16 + r;
                    cx[s][t] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                             x, b < p.kb ? row * p.pitch + b * 16 : kOutOfRange, 0, 0));
                    sx[s][t] = __builtin_amdgcn_raw_buffer_load_b8(xs, b < p.kb ? row * p.spitch + b : kOutOfRange, 0, 0);
                }
        }
        __builtin_amdgcn_sched_barrier(0);  // all of them are on their way before the first is waited for
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int b = (s0 + s * kWaves) * 4 + g;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                i32x4 c = {};
                int sc = 0;
                if constexpr (std::is_void<TX>::value) {
                    c = cx[s][t];
                    sc = sx[s][t];
                } else if (r < m && b < p.kb) {
                    c = quantize32(reinterpret_cast<const TX*>(p.x) + r * p.x_stride + b * 32, p.k - b * 32, &sc);
                }
                const i32x8 c8 = {c[0], c[1], c[2], c[3], 0, 0, 0, 0};
#pragma unroll
                for (int f = 0; f < NF; ++f) {
                    const i32x8 a8 = {a[s][f][0], a[s][f][1], a[s][f][2], a[s][f][3], 0, 0, 0, 0};
                    acc[t][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, c8, acc[t][f], 4, 4, 0, sa[s][f],
                                                                                 0, sc);
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
        if (t * 16 + r < m)
#pragma unroll
            for (int f = 0; f < NF; ++f)
                *reinterpret_cast<float4*>(&part[wave][(t * 16 + r) * ROW + f * 16 + g * 4]) =
                    make_float4(acc[t][f][0], acc[t][f][1], acc[t][f][2], acc[t][f][3]);
    __syncthreads();

    // a thread joins the waves' sums of 8 columns of one row
    constexpr int RUNS = NF * 2;
    for (int u = threadIdx.x; u < m * RUNS; u += 64 * kWaves) {
        const int row = u / RUNS, c = u % RUNS * 8, n = n0 + c, valid = p.n - n;
        float v[8] = {};
#pragma unroll
        for (int q = 0; q < kWaves; ++q)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += part[q][row * ROW + c + i];
        if (p.bias) {
            float b[8];
            load8(p.bias + n, valid, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += b[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = activate(v[i], p.act);
        store_run<TY>(p, row, n, valid, v);  // RUNS is a multiple of 4 for MXFP4: a block's quad runs together
    }
}

template <int MT, int NF, typename TX>
void launch_stream_y(const MatmulParams& p, cfwd_dtype y, hipStream_t st) {
    const unsigned grid = static_cast<unsigned>((p.n + 16 * NF - 1) / (16 * NF));
    if (y == CFWD_F32)
        stream_kernel<MT, NF, TX, float><<<grid, 64 * kWaves, 0, st>>>(p);
    else if (y == CFWD_BF16)
        stream_kernel<MT, NF, TX, bf16_t><<<grid, 64 * kWaves, 0, st>>>(p);
    else if constexpr (NF > 1)  // a block of 32 outputs is one workgroup's
        stream_kernel<MT, NF, TX, void><<<grid, 64 * kWaves, 0, st>>>(p);
}

template <int MT, typename TX>
void launch_stream_n(const MatmulParams& p, cfwd_dtype y, hipStream_t st) {
    // the widest workgroups (fewest readings of x) that still reach every CU
    if (p.n >= 256 * 64)
        launch_stream_y<MT, 4, TX>(p, y, st);
    else if (p.n >= 256 * 32 || y == CFWD_MXFP4)
        launch_stream_y<MT, 2, TX>(p, y, st);
    else
        launch_stream_y<MT, 1, TX>(p, y, st);
}

}  // namespace mx

// An x that is not MXFP4 is quantised by every workgroup; beyond these sizes
// that costs more than one more launch.
bool mx_stream_takes_raw(long long m, int k) { return m <= 16 && mx_blocks(k) <= 4 * 4 * mx::kWaves; }

// Beyond 32 rows every workgroup's reading of x counts: the tile kernel then
// wins unless w is small (48 rows: 4096 x 4096 10.6 us here, 13.4 there; 11000 x
// 3000 13.8 and 13.1; 4096 x 16384 33 and 22).
bool mx_stream_supported(long long m, int n, int k) {
    return m <= 32 || (m <= 64 && static_cast<long long>(n) * k <= 1 << 24);
}

cfwd_status mx_stream(const mx::MatmulParams& p, cfwd_dtype x, cfwd_dtype y, hipStream_t st) {
    if (x == CFWD_F32)
        mx::launch_stream_n<1, float>(p, y, st);
    else if (x == CFWD_BF16)
        mx::launch_stream_n<1, bf16_t>(p, y, st);
    else if (p.m <= 16)
        mx::launch_stream_n<1, void>(p, y, st);
    else if (p.m <= 32)
        mx::launch_stream_n<2, void>(p, y, st);
    else
        mx::launch_stream_n<4, void>(p, y, st);
    return check_hip(hipGetLastError(), "MXFP4 product launch");
}

}  // namespace cfwd

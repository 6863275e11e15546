// Product of two MXFP4 matrices for few rows of y (gfx950): the weights are
// read once, straight into registers.
//
// With few rows the time is the weights' bytes, so what counts is how many of
// them are on their way at once, and in how few pieces.  A workgroup owns 16 NF
// columns of y (rows of w) and all of its rows; its waves share the sum over K
// in runs of several steps and meet in LDS.  A wave requests all fragments of a
// run (16 KB of w) before it uses the first.  A run's scales come as 16
// bytes, four steps, of each row: a byte a lane and step costs as many cache
// lines as the codes do, 11.1 us against 8.1 for 1 x 16384 x 4096 and 37 against 28
// for 1 x 65536 x 4096 (5.1 TB/s).
//
// v_mfma_scale_f32_16x16x128_f8f6f4 with w as A and x as B: lane l holds block
// l / 16 of the K step's four of row l % 16, of each operand, and ends with
// columns 4 (l / 16) .. + 3 of y's row l % 16.
//
// A small x in 16 or 32 bits is quantised on the way, by every workgroup for
// itself, into LDS: its values are requested before the first weights, and
// become codes while those are on their way (a quantisation by each lane of its
// own block at its use cost 3 us of 1 x 16384 x 4096).
#include "mx_matmul_impl.h"

#include <algorithm>
#include <type_traits>

namespace cfwd {
namespace mx {

constexpr int kWaves = 8;
constexpr int kRawBlocks = 1024;  // of an x that the kernel quantises: 8 runs of 8 values a thread

// K steps of a wave's run, which is what it has on its way; whole 16-byte runs of scales.
template <int MT, int NF>
constexpr int kSteps = MT * NF == 1 ? 8 : 4;

// MT: 16-row tiles of y.  TX: void for MXFP4, else x's type (p.x, p.x_stride
// elements a row).  TY as in write_tile.
template <int MT, int NF, typename TX, typename TY>
__global__ __launch_bounds__(64 * kWaves) void stream_kernel(MatmulParams p, Divisor per_row) {
    constexpr bool RAW = !std::is_void<TX>::value;
    constexpr int STEPS = kSteps<MT, NF>;
    constexpr int ROW = NF * 16 + 4;       // floats of a row of partial sums, padded against bank conflicts
    __shared__ __attribute__((aligned(16))) float part[kWaves][MT * 16 * ROW];
    __shared__ __attribute__((aligned(16))) uint32_t xcodes[RAW ? kRawBlocks * 4 : 4];
    __shared__ uint8_t xscales[RAW ? kRawBlocks : 4];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int n0 = xcd_linear(blockIdx.x, gridDim.x) * (16 * NF);
    const long long rows_w = min(16 * NF, p.n - n0);
    const int m = static_cast<int>(p.m);
    const __amdgpu_buffer_rsrc_t w = buffer(p.w + static_cast<long long>(n0) * p.pitch, rows_w * p.pitch),
                                 ws = buffer(p.ws + static_cast<long long>(n0) * p.spitch, rows_w * p.spitch),
                                 x = buffer(p.x, static_cast<long long>(m) * p.pitch),
                                 xs = buffer(p.xs, static_cast<long long>(m) * p.spitch);
    f32x4 acc[MT][NF] = {};
    const int steps = (p.kb + 3) / 4;
    i32x4 a[STEPS][NF], cx[STEPS][MT];
    i32x4 sa[STEPS / 4][NF], sx[STEPS / 4][MT];  // a step's four blocks in a word
    auto request = [&](int s0) {  // steps past the end load nothing and multiply zeros
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int b = (s0 + s) * 4 + g;
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                const int row = f * 16 + r;
                a[s][f] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                        w, b < p.kb ? row * p.pitch + b * 16 : kOutOfRange, 0, 0));
                if (s % 4 == 0)
                    sa[s / 4][f] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                                 ws, row * p.spitch + (s0 + s) * 4, 0, 0));
            }
            if constexpr (!RAW)
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const int row = t * 16 + r;
                    cx[s][t] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                             x, b < p.kb ? row * p.pitch + b * 16 : kOutOfRange, 0, 0));
                    if (s % 4 == 0)
                        sx[s / 4][t] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                                     xs, row * p.spitch + (s0 + s) * 4, 0, 0));
                }
        }
        __builtin_amdgcn_sched_barrier(0);  // all of them are on their way before the first is waited for
    };
    if constexpr (RAW) {
        // Runs of 8 values; one that crosses its row's end reads on into what follows, or zeros at x's end.
        constexpr int RUNS = kRawBlocks * 4 / (64 * kWaves), WORDS = sizeof(TX) / 2;
        const __amdgpu_buffer_rsrc_t gx = buffer(p.x, ((m - 1) * p.x_stride + p.k) * sizeof(TX));
        u32x4 v[RUNS][WORDS];
#pragma unroll
        for (int i = 0; i < RUNS; ++i) {
            const uint32_t u = threadIdx.x + i * 64 * kWaves, row = divide(u, per_row), q = u - row * per_row.d;
            const uint32_t off = static_cast<int>(row) < m
                                     ? static_cast<uint32_t>(row * p.x_stride + q * 8) * static_cast<uint32_t>(sizeof(TX))
                                     : kOutOfRange;
#pragma unroll
            for (int j = 0; j < WORDS; ++j) v[i][j] = __builtin_amdgcn_raw_buffer_load_b128(gx, off + j * 16, 0, 0);
        }
        request(wave * STEPS);
#pragma unroll
        for (int i = 0; i < RUNS; ++i) {
            const uint32_t u = threadIdx.x + i * 64 * kWaves, row = divide(u, per_row), q = u - row * per_row.d;
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float e;
                if constexpr (sizeof(TX) == 4) e = __uint_as_float(v[i][j / 4][j % 4]);
                else e = __uint_as_float(j % 2 ? v[i][0][j / 2] & 0xffff0000u : v[i][0][j / 2] << 16);
                f[j] = static_cast<int>(q * 8) + j < p.k ? e : 0.0f;
            }
            uint32_t byte;
            const uint32_t codes = quantize8(f, &byte);
            if (static_cast<int>(row) < m) {
                xcodes[u] = codes;
                if ((q & 3) == 0) xscales[u / 4] = static_cast<uint8_t>(byte);
            }
        }
        __syncthreads();
    } else {
        request(wave * STEPS);
    }
    for (int s0 = wave * STEPS; s0 < steps;) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int b = (s0 + s) * 4 + g;
            auto scale = [&](int word) { return b < p.kb ? word >> 8 * g : 0; };  // its lowest byte counts
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                i32x4 c = {};
                int sc = 0;
                if constexpr (RAW) {
                    if (r < m && b < p.kb) {
                        c = *reinterpret_cast<const i32x4*>(&xcodes[(r * p.kb + b) * 4]);
                        sc = xscales[r * p.kb + b];
                    }
                } else {
                    c = cx[s][t];
                    sc = scale(sx[s / 4][t][s % 4]);
                }
                const i32x8 c8 = {c[0], c[1], c[2], c[3], 0, 0, 0, 0};
#pragma unroll
                for (int f = 0; f < NF; ++f) {
                    const i32x8 a8 = {a[s][f][0], a[s][f][1], a[s][f][2], a[s][f][3], 0, 0, 0, 0};
                    acc[t][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, c8, acc[t][f], 4, 4, 0,
                                                                                 scale(sa[s / 4][f][s % 4]), 0, sc);
                }
            }
        }
        s0 += waves * STEPS;
        if (s0 < steps) request(s0);
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
    for (int u = threadIdx.x; u < m * RUNS; u += blockDim.x) {
        const int row = u / RUNS, c = u % RUNS * 8, n = n0 + c, valid = p.n - n;
        float v[8] = {};
        for (int q = 0; q < waves; ++q)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += part[q][row * ROW + c + i];
        if (p.bias) {
            float b[8];
            load8(p.bias + n, valid, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += b[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = activate<TY>(v[i], p.act);
        store_run<TY>(p, row, n, valid, v);  // RUNS is a multiple of 4 for MXFP4: a block's quad runs together
    }
}

template <int MT, int NF, typename TX>
void launch_stream_y(const MatmulParams& p, cfwd_dtype y, hipStream_t st) {
    const unsigned grid = static_cast<unsigned>((p.n + 16 * NF - 1) / (16 * NF));
    // no more waves than have a part of the sum; quantising x takes all
    constexpr int RUN = kSteps<MT, NF> * 4;
    const unsigned block = 64 * (std::is_void<TX>::value ? std::min(kWaves, (p.kb + RUN - 1) / RUN) : kWaves);
    if (y == CFWD_F32)
        stream_kernel<MT, NF, TX, float><<<grid, block, 0, st>>>(p, divisor(p.kb * 4));
    else if (y == CFWD_BF16)
        stream_kernel<MT, NF, TX, bf16_t><<<grid, block, 0, st>>>(p, divisor(p.kb * 4));
    else if constexpr (NF > 1)  // a block of 32 outputs is one workgroup's
        stream_kernel<MT, NF, TX, void><<<grid, block, 0, st>>>(p, divisor(p.kb * 4));
}

template <int MT, typename TX>
void launch_stream_n(const MatmulParams& p, cfwd_dtype y, int cus, hipStream_t st) {
    // the widest workgroups (fewest readings of x) that still reach every CU
    if (MT < 4 && p.n >= cus * 64)  // for 64 rows two sets of columns at most
        launch_stream_y<MT, MT < 4 ? 4 : 2, TX>(p, y, st);
    else if (p.n >= cus * 32 || y == CFWD_MXFP4)
        launch_stream_y<MT, 2, TX>(p, y, st);
    else
        launch_stream_y<MT, 1, TX>(p, y, st);
}

}  // namespace mx

// One tile of rows, small enough for every workgroup to quantise it, with rows of whole words
// (the last of a row is then in range as a whole) within a buffer's 31 bits.
bool mx_stream_takes_raw(const cfwd_mx_matmul_desc* d) {
    const long long es = d->x_dtype == CFWD_F32 ? 4 : 2;
    return d->m <= 16 && d->m * mx_blocks(d->k) <= mx::kRawBlocks && d->k * es % 4 == 0 && d->x_stride * es % 4 == 0 &&
           d->x_stride < (1 << 24);
}

// Beyond 16 rows every workgroup's reading of x counts, and tiles (64 rows high)
// win where w is large, wide for 64 rows, or long (here and there: 17 x 16384 x
// 4096 9.5 us and 10.6, 32 x 8192 x 8192 12.4 and 14.9, 32 x 16384 x 16384 34 and 29;
// 64 x 4096 x 4096 8.7 and 10.1, 64 x 8192 x 8192 17 and 16, 64 x 16384 x 1024 7.2 and
// 6.7, 64 x 512 x 16384 25 and 14).
bool mx_stream_supported(long long m, int n, int k) {
    const long long nk = static_cast<long long>(n) * k;
    return m <= 16 || (m <= 32 && nk <= 1 << 26) || (m <= 64 && nk <= 1 << 24 && k <= 8192 && n < 1 << 14);
}

cfwd_status mx_stream(const mx::MatmulParams& p, cfwd_dtype x, cfwd_dtype y, int cus, hipStream_t st) {
    if (x == CFWD_F32)
        mx::launch_stream_n<1, float>(p, y, cus, st);
    else if (x == CFWD_BF16)
        mx::launch_stream_n<1, bf16_t>(p, y, cus, st);
    else if (p.m <= 16)
        mx::launch_stream_n<1, void>(p, y, cus, st);
    else if (p.m <= 32)
        mx::launch_stream_n<2, void>(p, y, cus, st);
    else
        mx::launch_stream_n<4, void>(p, y, cus, st);
    return check_hip(hipGetLastError(), "MXFP4 product launch");
}

}  // namespace cfwd

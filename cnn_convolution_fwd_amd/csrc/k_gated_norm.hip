// Norms before and after a block, fused with its gate and residual scale (gfx950).
//
//   s = residual_scale * r + gate * post(b)      h = pre(s)
//   post, pre: v, v / rms(v) * w + bias, or (v - mean) / std(v) * w + bias
//
// Both norms need a sum over the whole row before any of its outputs, so a
// row stays in the registers of the T threads that own it: each tensor is read
// or written once and the kernel is bound by HBM traffic (by the launch and
// two to four row sums for single tokens).  T is 8 to 1024, a power of two,
// and a thread holds NV vectors of 8 values.  All statistics are fp32; the
// variance is summed from the centred values.  s and h are rounded once, h
// from the unrounded s.  Rows too long for registers run in a second kernel
// that reads them again for each sum.
#include "gated_norm.h"
#include "mx.h"

#include <algorithm>

namespace cfwd {
namespace gn {

struct Params {
    long long rows;
    int c;
    long long rows_per_gate;
    float residual_scale, eps, inv_c;
    int post, pre;
    int scale_pitch;
    long long code_pitch;
    GatedNormArgs a;
};

// Sum over the T threads of a row.  T <= 64: lanes of a wave.  Otherwise the
// waves' sums meet in LDS; two slots in turn, so that one barrier is enough.
template <int T>
struct RowSum {
    float* slots;  // [2][16], T > 64 only
    int turn = 0;

    __device__ __forceinline__ float operator()(float v) {
#pragma unroll
        for (int m = 1; m < (T < 64 ? T : 64); m *= 2) v += __shfl_xor(v, m);
        if constexpr (T > 64) {
            float* s = slots + 16 * turn;
            turn ^= 1;
            if ((threadIdx.x & 63) == 0) s[threadIdx.x / 64] = v;
            __syncthreads();
            v = 0.0f;
#pragma unroll
            for (int i = 0; i < T / 64; ++i) v += s[threadIdx.x / T * (T / 64) + i];
        }
        return v;
    }
};

// Factor and offset of a norm of f over the row: v -> (v - mean) * rstd.
template <int NV, typename Sum>
__device__ __forceinline__ void normalise(float (&f)[NV][8], int kind, const int (&valid)[NV], const Params& p,
                                          Sum& sum) {
    if (kind == CFWD_NORM_LAYER) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) t += f[i][j];  // values past the row are 0
        const float mean = sum(t) * p.inv_c;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) f[i][j] = j < valid[i] ? f[i][j] - mean : 0.0f;
    }
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) t += f[i][j] * f[i][j];
    const float rstd = 1.0f / sqrtf(sum(t) * p.inv_c + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) f[i][j] *= rstd;
}

// f * w + bias over a row's vectors (w, bias: fp32 [c] or null)
template <int NV>
__device__ __forceinline__ void affine(float (&f)[NV][8], const float* w, const float* bias, const int (&col)[NV],
                                       const int (&valid)[NV]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (valid[i] <= 0) continue;
        float t[8];
        if (w) {
            mx::load8(w + col[i], valid[i], t);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[i][j] *= t[j];
        }
        if (bias) {
            mx::load8(bias + col[i], valid[i], t);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[i][j] += t[j];
        }
    }
}

template <int T, int NV, typename TB, typename TS, bool MX>
__global__ __launch_bounds__(T < 256 ? 256 : T) void row_kernel(Params p) {
    constexpr int WG = T < 256 ? 256 : T, ROWS = WG / T;
    __shared__ float slots[T > 64 ? 32 : 1];
    RowSum<T> sum{slots};
    const int t = threadIdx.x % T;
    const long long row = static_cast<long long>(blockIdx.x) * ROWS + threadIdx.x / T;
    const bool live = row < p.rows;  // T > 64: the whole workgroup; else whole groups of lanes, which run on with zeros
    int col[NV], valid[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        col[i] = (i * T + t) * 8;
        valid[i] = live ? max(0, min(8, p.c - col[i])) : 0;
    }
    const long long base = row * p.c;
    float f[NV][8], r[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) f[i][j] = r[i][j] = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (valid[i] <= 0) continue;
        if (p.a.b) mx::load8(static_cast<const TB*>(p.a.b) + base + col[i], valid[i], f[i]);
        if (p.a.residual) mx::load8(static_cast<const TS*>(p.a.residual) + base + col[i], valid[i], r[i]);
    }
    if (p.post != CFWD_NORM_NONE) {
        normalise<NV>(f, p.post, valid, p, sum);
        affine<NV>(f, p.a.post_weight, p.a.post_bias, col, valid);
    }
    if (p.a.gate && live) {
        const TB* g = static_cast<const TB*>(p.a.gate) + row / p.rows_per_gate * p.c;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (valid[i] <= 0) continue;
            float q[8];
            mx::load8(g + col[i], valid[i], q);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[i][j] *= q[j];
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[i][j] = p.a.residual ? p.residual_scale * r[i][j] + f[i][j] : f[i][j];
        if (p.a.s && valid[i] > 0) mx::store8(static_cast<TS*>(p.a.s) + base + col[i], valid[i], f[i]);
    }
    if (!p.a.h) return;
    if (p.pre != CFWD_NORM_NONE) {
        normalise<NV>(f, p.pre, valid, p, sum);
        affine<NV>(f, p.a.pre_weight, p.a.pre_bias, col, valid);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if constexpr (MX) {
            uint32_t byte;
            const uint32_t codes = mx::quantize8(f[i], &byte);
            if (live && col[i] < static_cast<int>(p.code_pitch) * 2) {
                uint8_t* hc = static_cast<uint8_t*>(p.a.h) + row * p.code_pitch;
                *reinterpret_cast<uint32_t*>(hc + col[i] / 2) = codes;
            }
            if (live && (t & 3) == 0 && col[i] / 32 < p.scale_pitch)
                (static_cast<uint8_t*>(p.a.h_scales) + row * p.scale_pitch)[col[i] / 32] =
                    col[i] < p.c ? static_cast<uint8_t>(byte) : 127;
        } else {
            if (valid[i] > 0) mx::store8(static_cast<TB*>(p.a.h) + base + col[i], valid[i], f[i]);
        }
    }
    if constexpr (MX) {  // what rounds the row's scales up to whole words and lies past its last vector
        if (live && t == 0)
            for (int i = NV * T / 4; i < p.scale_pitch; ++i)
                (static_cast<uint8_t*>(p.a.h_scales) + row * p.scale_pitch)[i] = 127;
    }
}

// Rows of any length: 1024 threads walk the row once for each sum and once
// for the outputs.  s is formed anew in each walk, from b and r alone, so s
// may be written over either (the last walk reads a value before it writes it).
template <typename TB, typename TS, bool MX>
__global__ __launch_bounds__(1024) void long_row_kernel(Params p) {
    __shared__ float slots[32];
    RowSum<1024> sum{slots};
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const long long base = row * p.c;
        const TB* b = p.a.b ? static_cast<const TB*>(p.a.b) + base : nullptr;
        const TS* r = p.a.residual ? static_cast<const TS*>(p.a.residual) + base : nullptr;
        const TB* g = p.a.gate ? static_cast<const TB*>(p.a.gate) + row / p.rows_per_gate * p.c : nullptr;
        float mean_b = 0.0f, rstd_b = 1.0f, mean_s = 0.0f, rstd_s = 1.0f;
        auto get_b = [&](int col, float(&v)[8]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.0f;
            if (b) mx::load8(b + col, p.c - col, v);
        };
        auto get_s = [&](int col, float(&v)[8]) {
            const int valid = p.c - col;
            float t[8];
            get_b(col, v);
            if (p.post != CFWD_NORM_NONE) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = (v[j] - mean_b) * rstd_b;
                if (p.a.post_weight) {
                    mx::load8(p.a.post_weight + col, valid, t);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] *= t[j];
                }
                if (p.a.post_bias) {
                    mx::load8(p.a.post_bias + col, valid, t);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] += t[j];
                }
            }
            if (g) {
                mx::load8(g + col, valid, t);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] *= t[j];
            }
            if (r) {
                mx::load8(r + col, valid, t);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = p.residual_scale * t[j] + v[j];
            }
        };
        auto statistics = [&](int kind, auto get, float* mean, float* rstd) {
            if (kind == CFWD_NORM_NONE) return;
            float v[8], t = 0.0f;
            if (kind == CFWD_NORM_LAYER) {
                for (int col = threadIdx.x * 8; col < p.c; col += 8192) {
                    get(col, v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) t += j < p.c - col ? v[j] : 0.0f;
                }
                *mean = sum(t) * p.inv_c;
                t = 0.0f;
            }
            for (int col = threadIdx.x * 8; col < p.c; col += 8192) {
                get(col, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float d = j < p.c - col ? v[j] - *mean : 0.0f;
                    t += d * d;
                }
            }
            *rstd = 1.0f / sqrtf(sum(t) * p.inv_c + p.eps);
        };
        statistics(p.post, get_b, &mean_b, &rstd_b);
        if (p.a.h) statistics(p.pre, get_s, &mean_s, &rstd_s);
        // every lane of a quad walks whole blocks: up to the row's padding in MXFP4
        const int end = MX ? static_cast<int>(p.code_pitch) * 2 : p.c;
        for (int col = threadIdx.x * 8; col < end; col += 8192) {
            const int valid = p.c - col;
            float v[8], t[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.0f;
            if (valid > 0) {
                get_s(col, v);
                if (p.a.s) mx::store8(static_cast<TS*>(p.a.s) + base + col, valid, v);
            }
            if (!p.a.h) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = (v[j] - mean_s) * rstd_s;
            if (valid > 0 && p.pre != CFWD_NORM_NONE) {
                if (p.a.pre_weight) {
                    mx::load8(p.a.pre_weight + col, valid, t);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] *= t[j];
                }
                if (p.a.pre_bias) {
                    mx::load8(p.a.pre_bias + col, valid, t);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] += t[j];
                }
            }
            if constexpr (MX) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = j < valid ? v[j] : 0.0f;
                uint32_t byte;
                const uint32_t codes = mx::quantize8(v, &byte);
                uint8_t* hc = static_cast<uint8_t*>(p.a.h) + row * p.code_pitch;
                uint8_t* hs = static_cast<uint8_t*>(p.a.h_scales) + row * p.scale_pitch;
                *reinterpret_cast<uint32_t*>(hc + col / 2) = codes;
                if ((col & 31) == 0) {
                    hs[col / 32] = static_cast<uint8_t>(byte);
                    if (col + 32 == end)
                        for (int i = end / 32; i < p.scale_pitch; ++i) hs[i] = 127;
                }
            } else {
                mx::store8(static_cast<TB*>(p.a.h) + base + col, valid, v);
            }
        }
    }
}

template <int T, int NV, typename TB, typename TS>
void launch_rows(const Params& p, bool to_mx, hipStream_t st) {
    constexpr int WG = T < 256 ? 256 : T, ROWS = WG / T;
    const unsigned grid = static_cast<unsigned>((p.rows + ROWS - 1) / ROWS);
    if (to_mx)
        row_kernel<T, NV, TB, TS, true><<<grid, WG, 0, st>>>(p);
    else
        row_kernel<T, NV, TB, TS, false><<<grid, WG, 0, st>>>(p);
}

template <typename TB, typename TS>
void launch(const Params& p, bool to_mx, hipStream_t st) {
    // threads of a row: the least power of two whose vectors hold it
    if (p.c <= 64) launch_rows<8, 1, TB, TS>(p, to_mx, st);
    else if (p.c <= 128) launch_rows<16, 1, TB, TS>(p, to_mx, st);
    else if (p.c <= 256) launch_rows<32, 1, TB, TS>(p, to_mx, st);
    else if (p.c <= 512) launch_rows<64, 1, TB, TS>(p, to_mx, st);
    else if (p.c <= 1024) launch_rows<128, 1, TB, TS>(p, to_mx, st);
    else if (p.c <= 2048) launch_rows<256, 1, TB, TS>(p, to_mx, st);
    else if (p.c <= 4096) launch_rows<512, 1, TB, TS>(p, to_mx, st);
    else if (p.c <= 8192) launch_rows<1024, 1, TB, TS>(p, to_mx, st);
    else if (p.c <= 16384) launch_rows<1024, 2, TB, TS>(p, to_mx, st);
    else {
        const unsigned grid = static_cast<unsigned>(std::min<long long>(p.rows, 4096));
        if (to_mx)
            long_row_kernel<TB, TS, true><<<grid, 1024, 0, st>>>(p);
        else
            long_row_kernel<TB, TS, false><<<grid, 1024, 0, st>>>(p);
    }
}

}  // namespace gn

cfwd_status gated_norm(const cfwd_gated_norm_desc* d, const GatedNormArgs& a, hipStream_t st) {
    gn::Params p{};
    p.rows = d->rows;
    p.c = d->c;
    p.rows_per_gate = d->rows_per_gate > 0 ? d->rows_per_gate : d->rows;
    p.residual_scale = d->residual_scale;
    p.eps = d->eps;
    p.inv_c = 1.0f / static_cast<float>(d->c);
    p.post = d->post;
    p.pre = d->pre;
    p.scale_pitch = static_cast<int>(mx_scale_pitch(d->c));
    p.code_pitch = mx_code_pitch(d->c);
    p.a = a;
    const bool to_mx = d->out_dtype == CFWD_MXFP4;
    if (d->dtype == CFWD_F32)
        gn::launch<float, float>(p, to_mx, st);
    else if (d->stream_dtype == CFWD_F32)
        gn::launch<bf16_t, float>(p, to_mx, st);
    else
        gn::launch<bf16_t, bf16_t>(p, to_mx, st);
    return check_hip(hipGetLastError(), "gated norm launch");
}

}  // namespace cfwd

// Norms before and after a block, fused with its gate and residual scale (gfx950).
//
//   s = residual_scale * r + gate * post(b)      h = pre(s)
//   post, pre: v, v / rms(v) * w + bias, or (v - mean) / std(v) * w + bias
//
// Both norms need a sum over the whole row before any of its outputs, so a
// row stays in the registers of the T threads that own it: each tensor is read
// or written once and the kernel is bound by HBM traffic (by the launch and
// two to four row sums for single tokens).  T is 8 to 1024, a power of two,
// and a thread holds NV vectors of 8 values.  A workgroup walks a run of rows:
// weights and gate, which would otherwise cost as many bytes of L2 as the row
// of HBM, stay in registers, and a row's values are requested while the row
// before it is worked on.  That lasts only if a row's accesses are not behind a
// branch (a wait then has to cover the path with the fewest accesses after it),
// so absent tensors, rows past the end and columns past the row are accesses out
// of a buffer's range, which load zeros and store nothing.  Two loads are behind
// one: the gate's next row, once for each run of rows that shares it, and the
// weights of rows over 8192, which find no registers and are read for each row.
// All statistics are fp32; the variance is summed from the centred values.  s and
// h are rounded once, h from the unrounded s.  16384 x 8192 in bf16 with both
// norms: 200 to 217 us, 4.9 to 5.4 TB/s (a plain copy: 5.4); 25088 x 512 to MXFP4:
// 16.5; one row of 4096: 3.6.
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

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
constexpr uint32_t kOutOfRange = 0x7ffffff0u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, long long bytes) {  // none: nothing is in range
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, p ? static_cast<int>(bytes) : 0, 0x00020000);
}

// 8 values of a row as they lie in memory.  The last vector of a row whose
// length is no multiple of 8 is loaded from 8 values before the row's end; skip(d)
// then moves it down by the d values that are not its own, with zeros after them.
template <typename T>
struct Vec;
template <>
struct Vec<bf16_t> {
    u32x4 w;
    __device__ __forceinline__ void load(const __amdgpu_buffer_rsrc_t& p, uint32_t off) {
        w = __builtin_amdgcn_raw_buffer_load_b128(p, off, 0, 0);
    }
    __device__ __forceinline__ void skip(int d) {
        if (d & 4) w = u32x4{w[2], w[3], 0, 0};
        if (d & 2) w = u32x4{w[1], w[2], w[3], 0};
        const uint32_t s = d % 2 * 16;
        w = u32x4{__builtin_amdgcn_alignbit(w[1], w[0], s), __builtin_amdgcn_alignbit(w[2], w[1], s),
                  __builtin_amdgcn_alignbit(w[3], w[2], s), w[3] >> s};
    }
    __device__ __forceinline__ float at(int j) const { return __uint_as_float(j % 2 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16); }
};
template <>
struct Vec<float> {
    u32x4 w[2];
    __device__ __forceinline__ void load(const __amdgpu_buffer_rsrc_t& p, uint32_t off) {
        w[0] = __builtin_amdgcn_raw_buffer_load_b128(p, off, 0, 0);
        w[1] = __builtin_amdgcn_raw_buffer_load_b128(p, off + 16, 0, 0);
    }
    __device__ __forceinline__ void skip(int d) {
#pragma unroll
        for (int k = 4; k > 0; k /= 2)
            if (d & k)
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j / 4][j % 4] = j + k < 8 ? w[(j + k) / 4 % 2][(j + k) % 4] : 0;
    }
    __device__ __forceinline__ float at(int j) const { return __uint_as_float(w[j / 4][j % 4]); }
};

template <typename T>
__device__ __forceinline__ void store_vec(const __amdgpu_buffer_rsrc_t& p, uint32_t off, const float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                                     pack_bf16x2(v[6], v[7])}, p, off, 0, 0);
    } else {
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                                     __float_as_uint(v[3])}, p, off, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                                                     __float_as_uint(v[7])}, p, off + 16, 0, 0);
    }
}

// Rows of a workgroup: a run of `run` (a multiple of the rows that it holds at
// once), at most 2^30 bytes.  TAIL: the row's length is no multiple of 8.
template <int T, int NV, typename TB, typename TS, bool MX, bool TAIL>
__global__ __launch_bounds__(T < 256 ? 256 : T) void row_kernel(Params p, long long run) {
    constexpr int WG = T < 256 ? 256 : T, ROWS = WG / T;
    __shared__ float slots[T > 64 ? 32 : 1];
    RowSum<T> sum{slots};
    const int t = threadIdx.x % T, sub = threadIdx.x / T;
    const long long first = blockIdx.x * run;
    const int rows = static_cast<int>(min(run, p.rows - first));
    const long long count = static_cast<long long>(rows) * p.c, skipped = first * p.c;
    auto part = [&](const void* q, int es) {
        return buffer(q ? static_cast<const uint8_t*>(q) + skipped * es : nullptr, count * es);
    };
    const __amdgpu_buffer_rsrc_t gb = part(p.a.b, sizeof(TB)), gr = part(p.a.residual, sizeof(TS)), gs = part(p.a.s, sizeof(TS));
    int col[NV], valid[NV], from[NV];  // from: where the loaded vector starts
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        col[i] = (i * T + t) * 8;
        valid[i] = max(0, min(8, p.c - col[i]));
        from[i] = TAIL ? min(col[i], p.c - 8) : col[i];
    }
    // byte offset of a vector in a buffer of rows: at, or out of range
    auto offset = [&](int row, int i, int es, int at) {
        return valid[i] > 0 ? static_cast<uint32_t>(row * p.c + at) * es : kOutOfRange;
    };
    auto settle = [&](auto& v, int i) {  // a loaded vector's own values
        if constexpr (TAIL) v.skip(col[i] - from[i] > 7 ? 0 : col[i] - from[i]);
    };
    float post_w[NV][8], post_b[NV][8], pre_w[NV][8], pre_b[NV][8];
    auto parameters = [&](const float* q, float(&to)[NV][8], float absent) {
        const __amdgpu_buffer_rsrc_t g = buffer(q, p.c * 4ll);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Vec<float> v;
            v.load(g, offset(0, i, 4, from[i]));
            settle(v, i);
#pragma unroll
            for (int j = 0; j < 8; ++j) to[i][j] = q ? v.at(j) : absent;
        }
    };
    Vec<TB> b[NV], gate[NV];
    Vec<TS> r[NV];
    auto request = [&](int row) {  // rows past the run are out of range
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            b[i].load(gb, offset(row, i, sizeof(TB), from[i]));
            r[i].load(gr, offset(row, i, sizeof(TS), from[i]));
        }
    };
    auto store_row = [&](const __amdgpu_buffer_rsrc_t& g, int row, auto type, const float(&f)[NV][8]) {
        typedef decltype(type) TO;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t at = offset(row, i, sizeof(TO), col[i]);
            store_vec<TO>(g, TAIL && valid[i] < 8 ? kOutOfRange : at, f[i]);
            if constexpr (TAIL)
#pragma unroll
                for (int j = 0; j < 7; ++j) {
                    const uint32_t one = valid[i] < 8 && j < valid[i] ? at + j * static_cast<uint32_t>(sizeof(TO)) : kOutOfRange;
                    if constexpr (sizeof(TO) == 2)
                        __builtin_amdgcn_raw_buffer_store_b16(float_to_bf16(f[i][j]), g, one, 0, 0);
                    else
                        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(f[i][j]), g, one, 0, 0);
                }
        }
    };
    request(sub);
    // two vectors a thread leave no registers to hold them in: they are read for each row
    auto post_parameters = [&] {
        parameters(p.a.post_weight, post_w, 1.0f);
        parameters(p.a.post_bias, post_b, 0.0f);
    };
    auto pre_parameters = [&] {
        parameters(p.a.pre_weight, pre_w, 1.0f);
        parameters(p.a.pre_bias, pre_b, 0.0f);
    };
    if constexpr (NV == 1) {
        post_parameters();
        pre_parameters();
    }
    const __amdgpu_buffer_rsrc_t gh = part(MX ? nullptr : p.a.h, sizeof(TB)),
                                 gc = buffer(MX && p.a.h ? static_cast<uint8_t*>(p.a.h) + first * p.code_pitch : nullptr, rows * p.code_pitch),
                                 gcs = buffer(MX && p.a.h ? static_cast<uint8_t*>(p.a.h_scales) + first * p.scale_pitch : nullptr,
                                              static_cast<long long>(rows) * p.scale_pitch);
    long long next_gate = first + sub;  // the first row that needs another row of gate
    // A row past the end (T <= 128: one of several that the workgroup holds) runs on with zeros and stores nothing.
    for (int row = sub; row - sub < rows; row += ROWS) {
        float f[NV][8];
        Vec<TS> rr[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            settle(b[i], i);
            rr[i] = r[i];
            settle(rr[i], i);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[i][j] = b[i].at(j);
        }
        if (p.a.gate && first + row >= next_gate) {
            const long long g = min(first + row, p.rows - 1) / p.rows_per_gate;
            next_gate = (g + 1) * p.rows_per_gate;
            const TB* q = static_cast<const TB*>(p.a.gate) + g * p.c;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (valid[i] <= 0) continue;
                const mx::Raw16* raw = reinterpret_cast<const mx::Raw16*>(q + from[i]);
                if constexpr (sizeof(TB) == 2) gate[i].w = u32x4{raw->w[0], raw->w[1], raw->w[2], raw->w[3]};
                else {
                    gate[i].w[0] = u32x4{raw[0].w[0], raw[0].w[1], raw[0].w[2], raw[0].w[3]};
                    gate[i].w[1] = u32x4{raw[1].w[0], raw[1].w[1], raw[1].w[2], raw[1].w[3]};
                }
                settle(gate[i], i);
            }
        }
        request(row + ROWS);
        if (p.post != CFWD_NORM_NONE) {
            if (p.a.b) normalise<NV>(f, p.post, valid, p, sum);  // the norm of an absent b is 0, whatever eps is
            if constexpr (NV > 1) post_parameters();
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) f[i][j] = f[i][j] * post_w[i][j] + post_b[i][j];
        }
        if (p.a.gate) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) f[i][j] = j < valid[i] ? f[i][j] * gate[i].at(j) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (p.a.residual)
#pragma unroll
                for (int j = 0; j < 8; ++j) f[i][j] = p.residual_scale * rr[i].at(j) + f[i][j];
        store_row(gs, row, TS{}, f);
        if (!p.a.h) continue;
        if (p.pre != CFWD_NORM_NONE) {
            normalise<NV>(f, p.pre, valid, p, sum);
            if constexpr (NV > 1) pre_parameters();
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) f[i][j] = f[i][j] * pre_w[i][j] + pre_b[i][j];
        }
        if constexpr (!MX) {
            store_row(gh, row, TB{}, f);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
#pragma unroll
                for (int j = 0; j < 8; ++j) f[i][j] = j < valid[i] ? f[i][j] : 0.0f;
                uint32_t byte;
                const uint32_t codes = mx::quantize8(f[i], &byte);
                const uint32_t at = static_cast<uint32_t>(row) * static_cast<uint32_t>(p.code_pitch) + col[i] / 2;
                __builtin_amdgcn_raw_buffer_store_b32(codes, gc, col[i] < static_cast<int>(p.code_pitch) * 2 ? at : kOutOfRange, 0, 0);
                const bool own = (t & 3) == 0 && col[i] / 32 < p.scale_pitch;
                __builtin_amdgcn_raw_buffer_store_b8(col[i] < p.c ? static_cast<uint8_t>(byte) : 127, gcs,
                                                     own ? static_cast<uint32_t>(row * p.scale_pitch + col[i] / 32) : kOutOfRange, 0, 0);
            }
            if constexpr (NV * T < 16)  // the rest of the word of scales
#pragma unroll
                for (int i = NV * T / 4; i < 4; ++i)
                    __builtin_amdgcn_raw_buffer_store_b8(127, gcs, t == 0 ? static_cast<uint32_t>(row * p.scale_pitch + i) : kOutOfRange, 0, 0);
        }
    }
}

// Rows too long for registers, and those of less than a vector: 1024 threads walk
// the row once for each sum and once for the outputs.  s is formed anew in each
// walk, from b and r alone, so s may be written over either (the last walk reads a
// value before it writes it).  Both norms RMS in bf16: 4096 x 20000 235 us (121 for
// its bytes read once; b is read three times and r twice, which is 212), 4096 x
// 65536 to MXFP4 660 (324; 621), one row of 20000 8.5.  Rows under 8 values leave
// nearly all threads without work: 18 ns a row, 100352 x 4 1850 us.
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
        if (p.a.b) statistics(p.post, get_b, &mean_b, &rstd_b);
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

// Workgroups of a kernel that the current device holds at once (half of what its CUs' registers could where it cannot be asked).
template <typename Kernel>
long long resident(PerDevice& known, Kernel kernel, int threads) {
    return known.get(
        [&](int) {
            int per_cu = 0;
            if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&per_cu, kernel, threads, 0) != hipSuccess) return 0ll;
            return static_cast<long long>(compute_units()) * per_cu;
        },
        256ll * (2048 / threads) / 2);
}

template <int T, int NV, bool MX, bool TAIL, typename TB, typename TS>
void launch_rows(const Params& p, hipStream_t st) {
    constexpr int WG = T < 256 ? 256 : T, ROWS = WG / T;
    static PerDevice known;
    const long long most = resident(known, row_kernel<T, NV, TB, TS, MX, TAIL>, WG);
    const long long groups = (p.rows + ROWS - 1) / ROWS, longest = (1ll << 30) / (p.c * 4ll) / ROWS;
    const long long run = std::min((groups + most - 1) / most, longest) * ROWS;
    row_kernel<T, NV, TB, TS, MX, TAIL><<<static_cast<unsigned>((p.rows + run - 1) / run), WG, 0, st>>>(p, run);
}

// A stream narrower than b's type goes with an absent b, and h in that type alone.
template <typename TB, typename TS>
constexpr bool kToMx = sizeof(TB) <= sizeof(TS);

template <int T, int NV, typename TB, typename TS>
void launch_rows(const Params& p, bool to_mx, hipStream_t st) {
    const bool tail = p.c % 8 != 0;
    if constexpr (kToMx<TB, TS>)
        if (to_mx) {
            tail ? launch_rows<T, NV, true, true, TB, TS>(p, st) : launch_rows<T, NV, true, false, TB, TS>(p, st);
            return;
        }
    tail ? launch_rows<T, NV, false, true, TB, TS>(p, st) : launch_rows<T, NV, false, false, TB, TS>(p, st);
}

template <typename TB, typename TS>
void launch(const Params& p, bool to_mx, hipStream_t st) {
    // threads of a row: the least power of two whose vectors hold it
    const bool long_row = p.c < 8 || p.c > 16384;  // less than a vector: no place to load its end from
    if (long_row) {
        const unsigned grid = static_cast<unsigned>(std::min<long long>(p.rows, 4096));
        if constexpr (kToMx<TB, TS>)
            if (to_mx) {
                long_row_kernel<TB, TS, true><<<grid, 1024, 0, st>>>(p);
                return;
            }
        long_row_kernel<TB, TS, false><<<grid, 1024, 0, st>>>(p);
    } else if (p.c <= 64) launch_rows<8, 1, TB, TS>(p, to_mx, st);
    else if (p.c <= 128) launch_rows<16, 1, TB, TS>(p, to_mx, st);
    else if (p.c <= 256) launch_rows<32, 1, TB, TS>(p, to_mx, st);
    else if (p.c <= 512) launch_rows<64, 1, TB, TS>(p, to_mx, st);
    else if (p.c <= 1024) launch_rows<128, 1, TB, TS>(p, to_mx, st);
    else if (p.c <= 2048) launch_rows<256, 1, TB, TS>(p, to_mx, st);
    else if (p.c <= 4096) launch_rows<512, 1, TB, TS>(p, to_mx, st);
    else if (p.c <= 8192) launch_rows<1024, 1, TB, TS>(p, to_mx, st);
    else launch_rows<1024, 2, TB, TS>(p, to_mx, st);
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
    if (d->stream_dtype == CFWD_F32)
        d->dtype == CFWD_F32 ? gn::launch<float, float>(p, to_mx, st) : gn::launch<bf16_t, float>(p, to_mx, st);
    else if (d->dtype == CFWD_F32 && !to_mx)
        gn::launch<float, bf16_t>(p, false, st);  // no b, no gate: h alone is fp32
    else
        gn::launch<bf16_t, bf16_t>(p, to_mx, st);
    return check_hip(hipGetLastError(), "gated norm launch");
}

}  // namespace cfwd

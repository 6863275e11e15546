// Rotary positions with several axes (gfx950).
//
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t),  t = position[axis] * frequency
//
// Angles are whole turns and a fraction: a frequency is kept as the fraction of
// a turn that one position makes, in units of 2^-64, and its product with the
// position, taken modulo 2^64, is the fraction of the angle; its upper 32 bits
// are within 2^-32 of a turn (1.5e-9 radians) for any position.  The nearest quarter turn
// is split off those bits and sin and cos of the rest (up to pi / 4) come from
// their Taylor sums to x^9 and x^8, which end 2e-9 and 3e-8 off: fp32's own rounding.
//
// All heads of a token share its angles, so a workgroup takes a few tokens,
// puts their sines and cosines into LDS once, and then walks the heads, eight
// pairs a thread: bound by HBM traffic.  12544 tokens of 40 heads of 128 (bf16,
// 257 MB) take 46 us, 5.6 TB/s; one token 2.6 us, a launch.
#include "attention.h"
#include "mx.h"
#include "stream.h"

#include <algorithm>

namespace cfwd {
namespace rp {

struct Params {
    const void* in[2];
    void* out[2];
    long long stride[2], out_stride[2], head_stride[2], out_head_stride[2];
    long long tokens;
    int heads[2];
    int dim, pairs, axes;
    int copied;        // values from 2 * pairs on are copied
    int per_workgroup; // tokens
    int turn_units, padded_pairs;
    mx::Divisor per_token, per_head, per_angles;  // units
    const cfwd_rope_pair* table;
    const void* positions;
};

__device__ __forceinline__ void sin_cos(uint32_t turn, float* s, float* c) {
    const uint32_t quarter = (turn + 0x20000000u) >> 30;
    const float x = static_cast<float>(static_cast<int32_t>(turn - (quarter << 30))) * 1.46291807926715968e-9f;  // 2 pi / 2^32
    const float z = x * x;
    const float sn = __builtin_fmaf(
        x * z, __builtin_fmaf(z, __builtin_fmaf(z, __builtin_fmaf(z, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), x);
    const float cs = __builtin_fmaf(
        z, __builtin_fmaf(z, __builtin_fmaf(z, __builtin_fmaf(z, 1.0f / 40320, -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
    const float a = quarter & 1 ? cs : sn, b = quarter & 1 ? sn : cs;
    *s = quarter & 2 ? -a : a;
    *c = (quarter + 1) & 2 ? -b : b;
}

template <typename T, bool ADJACENT, bool WIDE, bool ONCE>
__global__ __launch_bounds__(256) void rope_kernel(Params p) {
    extern __shared__ float angles[];  // [token][cos, sin][pair]
    const long long t0 = static_cast<long long>(blockIdx.x) * p.per_workgroup;
    const int tokens = static_cast<int>(min(static_cast<long long>(p.per_workgroup), p.tokens - t0));
    for (uint32_t n = threadIdx.x; n < static_cast<uint32_t>(tokens * p.padded_pairs); n += 256) {
        const int t = mx::divide(n, p.per_angles), i = n - t * p.padded_pairs;
        float sn = 0.0f, c = 1.0f;
        if (i < p.pairs) {
            const cfwd_rope_pair e = p.table[i];
            if (e.axis >= 0 && e.axis < p.axes) {
                const long long at = (t0 + t) * p.axes + e.axis;
                const long long pos = WIDE ? static_cast<const long long*>(p.positions)[at]
                                           : static_cast<const int*>(p.positions)[at];
                const uint64_t turn = static_cast<uint64_t>(pos) * e.turns + 0x80000000ull;
                sin_cos(static_cast<uint32_t>(turn >> 32), &sn, &c);
            }
        }
        angles[2 * t * p.padded_pairs + i] = c;
        angles[(2 * t + 1) * p.padded_pairs + i] = sn;
    }
    __syncthreads();
    const uint32_t units = tokens * p.per_token.d;
    for (uint32_t u = blockIdx.y * 256u + threadIdx.x; u < units; u += gridDim.y * 256u) {
        const uint32_t t = mx::divide(u, p.per_token), r = u - t * p.per_token.d;
        uint32_t head = mx::divide(r, p.per_head);
        const int j = r - head * p.per_head.d;
        const int which = head >= static_cast<uint32_t>(p.heads[0]);
        if (which) head -= p.heads[0];
        const T* x = static_cast<const T*>(p.in[which]) + (t0 + t) * p.stride[which] + head * p.head_stride[which];
        T* y = static_cast<T*>(p.out[which]) + (t0 + t) * p.out_stride[which] + head * p.out_head_stride[which];
        float a[8], b[8];
        if (j >= p.turn_units) {
            const int at = 2 * p.pairs + (j - p.turn_units) * 8;
            mx::load8<ONCE>(x + at, p.dim - at, a);
            mx::store8(y + at, p.dim - at, a);
            continue;
        }
        const int first = ADJACENT ? 16 * j : 8 * j, second = ADJACENT ? first + 8 : p.pairs + 8 * j;
        const int n1 = ADJACENT ? 2 * p.pairs - first : p.pairs - first, n2 = ADJACENT ? n1 - 8 : n1;
        mx::load8<ONCE>(x + first, n1, a);
        mx::load8<ONCE>(x + second, n2, b);
        const float* cs = angles + 2 * t * p.padded_pairs + 8 * j;
        const float* sn = cs + p.padded_pairs;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float& u0 = ADJACENT ? (i < 4 ? a[2 * i] : b[2 * i - 8]) : a[i];
            float& u1 = ADJACENT ? (i < 4 ? a[2 * i + 1] : b[2 * i - 7]) : b[i];
            const float v0 = u0, v1 = u1;
            u0 = __builtin_fmaf(v0, cs[i], -(v1 * sn[i]));
            u1 = __builtin_fmaf(v0, sn[i], v1 * cs[i]);
        }
        mx::store8(y + first, n1, a);
        mx::store8(y + second, n2, b);
    }
}

template <typename T, bool ADJACENT, bool WIDE>
void launch(const Params& p, bool once, dim3 grid, size_t lds, hipStream_t st) {
    if (once) rope_kernel<T, ADJACENT, WIDE, true><<<grid, 256, lds, st>>>(p);
    else rope_kernel<T, ADJACENT, WIDE, false><<<grid, 256, lds, st>>>(p);
}

template <typename T>
void launch(const Params& p, const cfwd_rope_desc* d, bool once, dim3 grid, size_t lds, hipStream_t st) {
    if (d->adjacent) {
        if (d->wide_positions) launch<T, true, true>(p, once, grid, lds, st);
        else launch<T, true, false>(p, once, grid, lds, st);
    } else {
        if (d->wide_positions) launch<T, false, true>(p, once, grid, lds, st);
        else launch<T, false, false>(p, once, grid, lds, st);
    }
}

}  // namespace rp

cfwd_status rope(const cfwd_rope_desc* d, const void* q, const void* k, const void* positions,
                 const cfwd_rope_pair* table, void* q_out, void* k_out, hipStream_t st) {
    rp::Params p{};
    p.in[0] = q;
    p.in[1] = k;
    p.out[0] = q_out;
    p.out[1] = k_out;
    p.stride[0] = d->q_stride;
    p.stride[1] = d->k_stride;
    p.out_stride[0] = d->q_out_stride;
    p.out_stride[1] = d->k_out_stride;
    p.head_stride[0] = d->q_head_stride;
    p.head_stride[1] = d->k_head_stride;
    p.out_head_stride[0] = d->q_out_head_stride;
    p.out_head_stride[1] = d->k_out_head_stride;
    p.tokens = d->tokens;
    p.heads[0] = d->q_heads;
    p.heads[1] = d->k_heads;
    p.dim = d->head_dim;
    p.pairs = d->pairs;
    p.axes = d->axes;
    p.copied = (q != q_out || (d->k_heads && k != k_out)) && 2 * d->pairs < d->head_dim;
    p.turn_units = (d->pairs + 7) / 8;
    p.padded_pairs = p.turn_units * 8;
    const int per_head = p.turn_units + (p.copied ? (d->head_dim - 2 * d->pairs + 7) / 8 : 0);
    if (per_head == 0) return CFWD_OK;
    const int per_token = per_head * (d->q_heads + d->k_heads);
    p.per_head = mx::divisor(per_head);
    p.per_angles = mx::divisor(p.padded_pairs ? p.padded_pairs : 1);
    p.per_token = mx::divisor(per_token);
    // About 1024 units a workgroup (12544 tokens of 320 units: 48 us with 640 to 1280, 49 with 320, 53 with 2048); where that
    // leaves CUs idle, fewer, down to a part of one token's.
    const long long cus = compute_units();
    int n = std::max(1, std::min({1024 / per_token, 16, p.padded_pairs ? 4096 / p.padded_pairs : 16}));
    n = static_cast<int>(std::max(1ll, std::min<long long>(n, d->tokens / (4 * cus))));
    p.per_workgroup = n;
    p.table = table;
    p.positions = positions;
    const size_t lds = static_cast<size_t>(n) * 2 * p.padded_pairs * 4;
    const long long es = d->dtype == CFWD_F32 ? 4 : 2;
    const long long each = (p.copied ? d->head_dim : 2 * d->pairs) * static_cast<long long>(d->q_heads + d->k_heads);
    const bool once = d->tokens >= mx::kStreamBytes / (2 * es * each);
    // tokens behind what one grid holds go in further launches
    const long long most = static_cast<long long>(n) << 30;
    for (long long at = 0; at < d->tokens; at += most) {
        const long long tokens = std::min(most, d->tokens - at);
        rp::Params part = p;
        part.tokens = tokens;
        for (int i = 0; i < 2; ++i) {
            part.in[i] = static_cast<const char*>(p.in[i]) + at * p.stride[i] * es;
            part.out[i] = static_cast<char*>(p.out[i]) + at * p.out_stride[i] * es;
        }
        part.positions = static_cast<const char*>(positions) + at * d->axes * (d->wide_positions ? 8 : 4);
        const unsigned wgs = static_cast<unsigned>((tokens + n - 1) / n);
        const long long parts = (static_cast<long long>(n) * per_token + 255) / 256;
        const dim3 grid(wgs, static_cast<unsigned>(std::max(1ll, std::min(parts, 2 * cus / wgs))));
        if (d->dtype == CFWD_F32) rp::launch<float>(part, d, once, grid, lds, st);
        else rp::launch<bf16_t>(part, d, once, grid, lds, st);
        const cfwd_status e = check_hip(hipGetLastError(), "rotary positions launch");
        if (e != CFWD_OK) return e;
    }
    return CFWD_OK;
}

}  // namespace cfwd

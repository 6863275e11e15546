// Writing keys and values to the paged MXFP4 cache, and reading them back (gfx950).
//
// One pass each way, eight values a thread, four adjacent lanes a block of 32,
// as the plain quantisation (its formulas stand in mx.h); bound by HBM traffic.
#include "attention.h"
#include "mx.h"

#include <algorithm>

namespace cfwd {
namespace cache {

using namespace mx;

struct Params {
    uint32_t* codes[2];
    uint8_t* scales[2];
    int heads, dim, page_size, pages, sequences, table_pitch;
    int scale_pitch;                 // bytes of a row
    int per_workgroup;               // tokens (reading)
    long long tokens;                // reading
    Divisor per_row, per_side, per_token, page;  // units of a row, of a token's keys, of a token; tokens of a page
};

// unit = (token, keys or values, head, 8 values); whole quads share a token
template <typename T, bool WIDE>
__global__ __launch_bounds__(256) void write_kernel(Params p, const T* __restrict__ k, const T* __restrict__ v,
                                                    long long k_stride, long long k_head, long long v_stride,
                                                    long long v_head, const void* __restrict__ slots, uint32_t units) {
    const uint32_t u = blockIdx.x * 256u + threadIdx.x;
    if (u >= units) return;
    const uint32_t token = divide(u, p.per_token), r = u - token * p.per_token.d;
    const uint32_t side = divide(r, p.per_side), in_side = r - side * p.per_side.d;
    const uint32_t head = divide(in_side, p.per_row), q = in_side - head * p.per_row.d;
    const long long slot = WIDE ? static_cast<const long long*>(slots)[token] : static_cast<const int*>(slots)[token];
    if (slot < 0 || slot >= static_cast<long long>(p.pages) * p.page_size) return;
    const uint32_t page = divide(static_cast<uint32_t>(slot), p.page), offset = static_cast<uint32_t>(slot) - page * p.page.d;
    const long long row = (static_cast<long long>(page) * p.heads + head) * p.page_size + offset;
    const T* x = side ? v + token * v_stride + head * v_head : k + token * k_stride + head * k_head;
    float f[8];
    load8(x + q * 8, p.dim - static_cast<int>(q * 8), f);
    uint32_t byte;
    const uint32_t c = quantize8(f, &byte);
    (side ? p.codes[1] : p.codes[0])[row * p.per_row.d + q] = c;
    if ((q & 3) == 0) {
        uint8_t* s = (side ? p.scales[1] : p.scales[0]) + row * p.scale_pitch;
        s[q >> 2] = static_cast<uint8_t>(byte);
        if (q + 4 == p.per_row.d)  // the last block also writes what rounds the row up to whole words
            for (int i = p.per_row.d / 4; i < p.scale_pitch; ++i) s[i] = 127;
    }
}

constexpr int kMostTokens = 64;  // of a workgroup

template <typename T>
__global__ __launch_bounds__(256) void read_kernel(Params p, const int32_t* __restrict__ table,
                                                   const int32_t* __restrict__ starts, T* __restrict__ k,
                                                   T* __restrict__ v) {
    __shared__ long long first[kMostTokens];  // row of a token's head 0 in the cache, or -1
    const long long t0 = static_cast<long long>(blockIdx.x) * p.per_workgroup;
    const int tokens = static_cast<int>(min(static_cast<long long>(p.per_workgroup), p.tokens - t0));
    const int lane = threadIdx.x & 63;
    for (int i = threadIdx.x >> 6; i < tokens; i += 4) {
        const long long t = t0 + i;
        int seq = 0;  // sequences that end at or before t
        for (int s = 0; s < p.sequences; s += 64)
            seq += __popcll(__ballot(s + lane < p.sequences && starts[min(s + lane, p.sequences - 1) + 1] <= t));
        long long row = -1;
        if (seq < p.sequences) {
            const long long at = t - starts[seq];
            if (at >= 0) {
                const uint32_t page = divide(static_cast<uint32_t>(at), p.page);
                if (page < static_cast<uint32_t>(p.table_pitch)) {
                    const int id = table[static_cast<long long>(seq) * p.table_pitch + page];
                    if (id >= 0 && id < p.pages)
                        row = static_cast<long long>(id) * p.heads * p.page_size + (at - static_cast<long long>(page) * p.page_size);
                }
            }
        }
        if (lane == 0) first[i] = row;
    }
    __syncthreads();
    const uint32_t units = tokens * p.per_token.d;
    for (uint32_t u = threadIdx.x; u < units; u += 256) {
        const uint32_t token = divide(u, p.per_token), r = u - token * p.per_token.d;
        const uint32_t side = divide(r, p.per_side), in_side = r - side * p.per_side.d;
        const uint32_t head = divide(in_side, p.per_row), q = in_side - head * p.per_row.d;
        long long row = first[token];
        if (row < 0) continue;
        row += static_cast<long long>(head) * p.page_size;
        const uint32_t c = (side ? p.codes[1] : p.codes[0])[row * p.per_row.d + q];
        const float s = scale_of((side ? p.scales[1] : p.scales[0])[row * p.scale_pitch + (q >> 2)]);
        typedef float f32x2_t __attribute__((ext_vector_type(2)));
        const f32x2_t w[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0),
                              __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1),
                              __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2),
                              __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3)};
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = w[i / 2][i % 2] * s;  // exact: at most two significant bits
        const int valid = p.dim - static_cast<int>(q * 8);
        if (valid > 0) store8((side ? v : k) + ((t0 + token) * p.heads + head) * p.dim + q * 8, valid, f);
    }
}

Params params(const cfwd_mx_cache* c) {
    Params p{};
    p.codes[0] = static_cast<uint32_t*>(c->k_codes);
    p.codes[1] = static_cast<uint32_t*>(c->v_codes);
    p.scales[0] = static_cast<uint8_t*>(c->k_scales);
    p.scales[1] = static_cast<uint8_t*>(c->v_scales);
    p.heads = c->kv_heads;
    p.dim = c->head_dim;
    p.page_size = c->page_size;
    p.pages = c->pages;
    p.scale_pitch = static_cast<int>(mx_scale_pitch(c->head_dim));
    const int per_row = static_cast<int>(mx_blocks(c->head_dim)) * 4;
    p.per_row = divisor(per_row);
    p.per_side = divisor(per_row * c->kv_heads);
    p.per_token = divisor(2 * per_row * c->kv_heads);
    p.page = divisor(c->page_size);
    return p;
}

}  // namespace cache

cfwd_status mx_cache_write(const cfwd_mx_cache_write_desc* d, const cfwd_mx_cache* c, const void* k, const void* v,
                           const void* slots, hipStream_t st) {
    const cache::Params p = cache::params(c);
    const long long most = ((1ll << 31) - 4) / p.per_token.d;  // tokens of one launch: fewer than 2^31 units
    for (long long at = 0; at < d->tokens; at += most) {
        const long long n = std::min(most, d->tokens - at);
        const uint32_t units = static_cast<uint32_t>(n * p.per_token.d), grid = (units + 255) / 256;
        const void* s = static_cast<const char*>(slots) + at * (d->wide_slots ? 8 : 4);
        auto go = [&](auto kernel, auto type) {
            using T = decltype(type);
            kernel<<<grid, 256, 0, st>>>(p, static_cast<const T*>(k) + at * d->k_stride,
                                         static_cast<const T*>(v) + at * d->v_stride, d->k_stride, d->k_head_stride,
                                         d->v_stride, d->v_head_stride, s, units);
        };
        if (d->dtype == CFWD_F32) {
            if (d->wide_slots) go(cache::write_kernel<float, true>, float{});
            else go(cache::write_kernel<float, false>, float{});
        } else {
            if (d->wide_slots) go(cache::write_kernel<bf16_t, true>, bf16_t{});
            else go(cache::write_kernel<bf16_t, false>, bf16_t{});
        }
        const cfwd_status e = check_hip(hipGetLastError(), "cache write launch");
        if (e != CFWD_OK) return e;
    }
    return CFWD_OK;
}

cfwd_status mx_cache_read(const cfwd_mx_cache_read_desc* d, const cfwd_mx_cache* c, const int32_t* table,
                          const int32_t* starts, void* k, void* v, hipStream_t st) {
    cache::Params p = cache::params(c);
    p.sequences = d->sequences;
    p.table_pitch = d->table_pitch;
    p.tokens = d->tokens;  // below 2^31, as starts are 32 bits wide
    const long long cus = compute_units();
    p.per_workgroup = static_cast<int>(std::max<long long>(
        1, std::min<long long>({cache::kMostTokens, 2048 / p.per_token.d, d->tokens / (4 * cus)})));
    const unsigned grid = static_cast<unsigned>((d->tokens + p.per_workgroup - 1) / p.per_workgroup);
    if (d->dtype == CFWD_F32)
        cache::read_kernel<float><<<grid, 256, 0, st>>>(p, table, starts, static_cast<float*>(k), static_cast<float*>(v));
    else
        cache::read_kernel<bf16_t><<<grid, 256, 0, st>>>(p, table, starts, static_cast<bf16_t*>(k), static_cast<bf16_t*>(v));
    return check_hip(hipGetLastError(), "cache read launch");
}

}  // namespace cfwd

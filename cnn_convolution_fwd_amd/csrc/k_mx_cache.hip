// Writing keys and values to the paged MXFP4 cache, and reading them back (gfx950).
//
// One pass each way, eight values a thread, four adjacent lanes a block of 32,
// as the plain quantisation (its formulas stand in mx.h); bound by HBM traffic.
// 32768 tokens of 8 heads of 128 (bf16, 170 MB each way): written in 34 us, 5.0 TB/s,
// read in 29, 5.9 TB/s; 64 tokens: a launch each, 2.6 us.
#include "attention.h"
#include "mx.h"
#include "stream.h"

#include <algorithm>
#include <type_traits>

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
    int rows;                        // side by side in a workgroup (writing)
    Divisor per_row, per_side, per_token, page;  // units of a row, of a token's keys, of a token; tokens of a page
    Divisor lanes, sides;                        // threads of a row, rows of a token (writing)
};

// A workgroup writes one head, of keys or of values, of consecutive tokens: in pages filled in order their rows lie side by
// side, so that whole lines of codes and scales come from one workgroup (lines put together in two XCDs' caches cost
// 32768 tokens of 8 heads of 128 47 us instead of 38).  A row goes to `lanes` threads, 4, 8 or a multiple of 16 of
// them, so that the blocks of a word of scales lie within 16 lanes; ROUNDS rows to a thread, loaded before the first is written.
template <typename T, bool WIDE, int ROUNDS, bool ONCE>
__global__ __launch_bounds__(256) void write_kernel(Params p, const T* __restrict__ k, const T* __restrict__ v,
                                                    long long k_stride, long long k_head, long long v_stride,
                                                    long long v_head, const void* __restrict__ slots, uint32_t tokens) {
    const uint32_t block = divide(blockIdx.x, p.sides), pair = blockIdx.x - block * p.sides.d;
    const int side = pair >= static_cast<uint32_t>(p.heads), head = pair - side * p.heads;
    const uint32_t row = divide(threadIdx.x, p.lanes), q = threadIdx.x - row * p.lanes.d, per_round = p.rows;
    const bool has = row < per_round && q < p.per_row.d;
    const T* x = (side ? v + head * v_head : k + head * k_head) + q * 8;
    const long long stride = side ? v_stride : k_stride;
    const uint32_t first = block * per_round * ROUNDS + row;
    float f[ROUNDS][8];
    long long slot[ROUNDS];
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const uint32_t token = first + r * per_round;
        slot[r] = -1;
#pragma unroll
        for (int i = 0; i < 8; ++i) f[r][i] = 0.0f;
        if (has && token < tokens) {
            slot[r] = WIDE ? static_cast<const long long*>(slots)[token] : static_cast<const int*>(slots)[token];
            load8<ONCE>(x + token * stride, p.dim - static_cast<int>(q * 8), f[r]);
        }
    }
    uint32_t* codes = side ? p.codes[1] : p.codes[0];
    uint8_t* scales = side ? p.scales[1] : p.scales[0];
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        uint32_t byte;
        const uint32_t c = quantize8(f[r], &byte);
        // the bytes of this block and of the three behind it in the row; 127 where it has no more
        uint32_t word = byte;
        const uint32_t next[3] = {static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, byte, 0x104, 0xf, 0xf, false)),
                                  static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, byte, 0x108, 0xf, 0xf, false)),
                                  static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, byte, 0x10c, 0xf, 0xf, false))};
#pragma unroll
        for (int i = 0; i < 3; ++i) word |= (q + 4 * (i + 1) < p.per_row.d ? next[i] : 127u) << (8 * (i + 1));
        if (slot[r] < 0 || slot[r] >= static_cast<long long>(p.pages) * p.page_size) continue;
        const uint32_t page = divide(static_cast<uint32_t>(slot[r]), p.page), offset = static_cast<uint32_t>(slot[r]) - page * p.page.d;
        const long long to = (static_cast<long long>(page) * p.heads + head) * p.page_size + offset;
        codes[to * p.per_row.d + q] = c;
        if (q % 16 == 0) *reinterpret_cast<uint32_t*>(scales + to * p.scale_pitch + q / 4) = word;
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
        // sequences that end at or before t, by looking at 64 evenly spaced, and at 64 between two of those, ...
        int seq = 0;
        for (int step, left = p.sequences; left > 0; left = step == 1 ? 0 : min(step, p.sequences - seq)) {
            step = (left + 63) / 64;
            const int s = (lane + 1) * step;
            seq += __popcll(__ballot(s <= left && starts[seq + s] <= t)) * step;
        }
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
    cache::Params p = cache::params(c);
    const int units = static_cast<int>(p.per_row.d), lanes = units <= 4 ? 4 : units <= 8 ? 8 : (units + 15) / 16 * 16;
    p.lanes = mx::divisor(lanes);
    p.sides = mx::divisor(2 * c->kv_heads);
    p.rows = 256 / lanes;
    // two rows a thread where that leaves work for every CU (32768 tokens of 8 heads of 128, with one: 0.5 us more), else one
    const bool many = d->tokens * p.sides.d >= 4ll * p.rows * 2 * compute_units();
    const int per_block = p.rows * (many ? 2 : 1);
    const long long row_bytes = static_cast<long long>(d->dtype == CFWD_F32 ? 4 : 2) * c->head_dim + 4 * units + p.scale_pitch;
    const bool once = many && d->tokens >= mx::kStreamBytes / (p.sides.d * row_bytes);
    const long long most = std::min((1ll << 31) - 256 * 4, ((1ll << 31) / (2ll * c->kv_heads) - 1) * per_block);  // tokens of one launch
    for (long long at = 0; at < d->tokens; at += most) {
        const long long n = std::min(most, d->tokens - at);
        const unsigned grid = static_cast<unsigned>((n + per_block - 1) / per_block * p.sides.d);
        const void* s = static_cast<const char*>(slots) + at * (d->wide_slots ? 8 : 4);
        auto go = [&](auto kernel, auto type) {
            using T = decltype(type);
            kernel<<<grid, 256, 0, st>>>(p, static_cast<const T*>(k) + at * d->k_stride,
                                         static_cast<const T*>(v) + at * d->v_stride, d->k_stride, d->k_head_stride,
                                         d->v_stride, d->v_head_stride, s, static_cast<uint32_t>(n));
        };
        auto rounds = [&](auto type, auto wide) {
            using T = decltype(type);
            constexpr bool w = decltype(wide)::value;
            if (once) go(cache::write_kernel<T, w, 2, true>, type);
            else if (many) go(cache::write_kernel<T, w, 2, false>, type);
            else go(cache::write_kernel<T, w, 1, false>, type);
        };
        auto typed = [&](auto type) {
            if (d->wide_slots) rounds(type, std::true_type{});
            else rounds(type, std::false_type{});
        };
        if (d->dtype == CFWD_F32) typed(float{});
        else typed(bf16_t{});
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

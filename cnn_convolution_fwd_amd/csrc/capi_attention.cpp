// C ABI of the rotary positions, the paged MXFP4 cache and attention: checks
// of the arguments, then the launches (k_rope.hip, k_mx_cache.hip,
// k_mx_decode.hip, k_attention.hip).
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <string>

#include "attention.h"
#include "capi_checks.h"
#include "mx.h"

namespace cfwd {
namespace {

constexpr long long kMaxTokens = 1ll << 38, kMaxSpan = 1ll << 60;
constexpr int kMaxHeads = 1 << 16, kMaxDim = 1 << 10;

// [rows][heads][dim] at a row and a head stride, all in bytes
struct Heads {
    const void* p;
    long long rows, heads, row_stride, head_stride, width;
    unsigned long long in_row() const { return static_cast<unsigned long long>(heads - 1) * head_stride + width; }
    Span span() const {
        return {p, rows > 0 && heads > 0 ? static_cast<unsigned long long>(rows - 1) * row_stride + in_row() : 0};
    }
};

// Whether two of them share bytes.  Parts of one buffer (same strides, side by side within a row or a head) do not.
bool overlap(const Heads& a, const Heads& b) {
    if (!overlap(a.span(), b.span())) return false;
    auto beside = [&](unsigned long long stride, unsigned long long wa, unsigned long long wb) {
        if (!stride || wa > stride || wb > stride) return false;
        const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
        const unsigned long long d = y >= x ? (y - x) % stride : (stride - (x - y) % stride) % stride;
        return d >= wa && d + wb <= stride;
    };
    if (a.row_stride != b.row_stride) return true;
    if (beside(a.row_stride, a.in_row(), b.in_row())) return false;
    return !(a.head_stride == b.head_stride && a.head_stride && a.row_stride % a.head_stride == 0 &&
             beside(a.head_stride, a.width, b.width));
}

bool same(const Heads& a, const Heads& b) {
    return a.p == b.p && a.row_stride == b.row_stride && a.head_stride == b.head_stride && a.heads == b.heads;
}

// Strides, in elements, of a tensor that is only read: rows and heads may be one another's.
bool strides_ok(long long rows, long long heads, long long row_stride, long long head_stride) {
    return row_stride >= 0 && head_stride >= 0 && row_stride <= kMaxSpan / std::max(rows, 1ll) &&
           head_stride <= kMaxSpan / std::max(heads, 1ll);
}

// The same of one that is written: rows and heads do not run into each other.
bool strides_fit(long long rows, long long heads, int dim, long long row_stride, long long head_stride) {
    if (!strides_ok(rows, heads, row_stride, head_stride)) return false;
    if (heads > 1 && head_stride < dim) return false;
    if (rows <= 1) return true;
    // tokens outside heads (each row holds all heads), or heads outside tokens
    return row_stride >= (heads - 1) * head_stride + dim || (row_stride >= dim && (heads <= 1 || head_stride >= (rows - 1) * row_stride + dim));
}

cfwd_status check_cache(const cfwd_mx_cache* c) {
    if (!c) return invalid("cache is NULL");
    if (c->pages < 1 || c->page_size < 1) return invalid("pages and page_size must be at least 1");
    if (c->kv_heads < 1 || c->kv_heads > kMaxHeads) return invalid("kv_heads must be between 1 and 65536");
    if (c->head_dim < 1 || c->head_dim > kMaxDim) return invalid("head_dim must be between 1 and 1024");
    if (static_cast<long long>(c->pages) * c->page_size >= (1ll << 31)) return invalid("the cache must have fewer than 2^31 slots");
    return CFWD_OK;
}

struct CacheSpans {
    Span part[4];
};

CacheSpans spans(const cfwd_mx_cache* c) {
    const unsigned long long rows = static_cast<unsigned long long>(c->pages) * c->page_size * c->kv_heads;
    const unsigned long long codes = rows * mx_code_pitch(c->head_dim), scales = rows * mx_scale_pitch(c->head_dim);
    return {{{c->k_codes, codes}, {c->k_scales, scales}, {c->v_codes, codes}, {c->v_scales, scales}}};
}

cfwd_status check_cache_buffers(const cfwd_mx_cache* c, bool written) {
    if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales) return invalid("NULL buffer in the cache");
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 4) || !aligned(c->v_scales, 4))
        return invalid("codes must be aligned to 16 bytes, scales to 4");
    if (written) {
        const CacheSpans s = spans(c);
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < i; ++j)
                if (overlap(s.part[i], s.part[j])) return invalid("the cache's parts must not overlap");
    }
    return CFWD_OK;
}

cfwd_status check_cache_attention(const cfwd_mx_cache_attention_desc* d, const cfwd_mx_cache* c) {
    if (!d) return invalid("descriptor is NULL");
    const cfwd_status s = check_cache(c);
    if (s != CFWD_OK) return s;
    if (d->sequences < 0 || d->tokens < 0) return invalid("sequences and tokens must be >= 0");
    if (d->table_pitch < 1) return invalid("table_pitch must be at least 1");
    if (static_cast<long long>(d->table_pitch) * c->page_size >= (1ll << 31) - 4096)
        return invalid("a row of the page table must stand for fewer than 2^31 - 4096 tokens");
    if (!(d->scale > 0.0f) || std::isinf(d->scale)) return invalid("scale must be a number > 0");
    if (d->q_heads < 1 || d->q_heads > kMaxHeads || d->q_heads % c->kv_heads)
        return invalid("q_heads must be a multiple of kv_heads, at most 65536");
    if (d->dtype != CFWD_BF16) return set_error(CFWD_ERR_UNSUPPORTED, "attention runs in bf16 only");
    if (c->head_dim % 32 || c->head_dim > 256)
        return set_error(CFWD_ERR_UNSUPPORTED, "attention over the cache needs a head_dim that is a multiple of 32, at most 256");
    if (c->page_size % 16) return set_error(CFWD_ERR_UNSUPPORTED, "attention over the cache needs a page_size that is a multiple of 16");
    if (static_cast<long long>(c->page_size) * c->kv_heads * mx_code_pitch(c->head_dim) >= (1ll << 31))
        return set_error(CFWD_ERR_UNSUPPORTED, "attention over the cache needs pages of fewer than 2^31 bytes of codes");
    if (d->tokens > 1024) return set_error(CFWD_ERR_UNSUPPORTED, "attention over the cache takes at most 1024 tokens a sequence");
    if (static_cast<long long>(d->sequences) * d->q_heads * std::max(d->tokens, 1) >= (1ll << 31) / 16)
        return set_error(CFWD_ERR_UNSUPPORTED, "too many queries for one call");
    // units of work are counted in 32 bits: 128 tokens of a head for 16 queries at least, and some for each pair of these
    const long long units = (static_cast<long long>(d->table_pitch) * c->page_size / 128 + 8) * c->kv_heads *
                            ((static_cast<long long>(d->tokens) * (d->q_heads / c->kv_heads) + 15) / 16);
    if (d->sequences > 0 && units >= (1ll << 31) / d->sequences)
        return set_error(CFWD_ERR_UNSUPPORTED, "the page table stands for too many tokens for one call");
    return CFWD_OK;
}

cfwd_status check_attention(const cfwd_attention_desc* d) {
    if (!d) return invalid("descriptor is NULL");
    if (d->q_tokens < 0 || d->k_tokens < 0 || d->sequences < 0) return invalid("tokens and sequences must be >= 0");
    if (d->kv_heads < 1 || d->q_heads < 1 || d->q_heads > kMaxHeads || d->q_heads % d->kv_heads)
        return invalid("q_heads must be a multiple of kv_heads, at most 65536");
    if (d->head_dim < 1) return invalid("head_dim must be at least 1");
    if (!(d->scale > 0.0f) || std::isinf(d->scale)) return invalid("scale must be a number > 0");
    if (d->dtype != CFWD_BF16) return set_error(CFWD_ERR_UNSUPPORTED, "attention runs in bf16 only");
    if (d->head_dim % 8 || d->head_dim > 256)
        return set_error(CFWD_ERR_UNSUPPORTED, "attention needs a head_dim that is a multiple of 8, at most 256");
    if (d->q_tokens >= (1ll << 31) / d->q_heads || d->k_tokens >= (1ll << 31) - 4096)
        return set_error(CFWD_ERR_UNSUPPORTED, "q_tokens times q_heads, and k_tokens, must stay below 2^31");
    if ((d->q_tokens * (d->q_heads / d->kv_heads) / 128 + d->sequences + 1) * d->kv_heads >= (1ll << 31))
        return set_error(CFWD_ERR_UNSUPPORTED, "too many tiles for one launch");
    const struct { long long rows; int heads; long long stride, head; } t[] = {
        {d->q_tokens, d->q_heads, d->q_stride, d->q_head_stride}, {d->k_tokens, d->kv_heads, d->k_stride, d->k_head_stride},
        {d->k_tokens, d->kv_heads, d->v_stride, d->v_head_stride}};
    for (const auto& x : t) {
        if (!strides_ok(x.rows, x.heads, x.stride, x.head)) return invalid("strides are out of range");
        if (x.stride % 8 || x.head % 8) return invalid("strides must be multiples of 8 elements");
    }
    for (int i = 1; i < 3; ++i)
        if (t[i].rows > 0 && (t[i].stride < d->head_dim || t[i].stride > (1 << 24)))
            return set_error(CFWD_ERR_UNSUPPORTED, "strides between tokens of k and v must be at least head_dim, at most 2^24");
    return CFWD_OK;
}

}  // namespace
}  // namespace cfwd

using namespace cfwd;

extern "C" {

uint64_t cfwd_rope_turns(double frequency) {
    // in long double: a double's 53 bits would leave far positions 2^-22 off
    const long double turns = frequency / 6.283185307179586476925286766559L;
    if (!std::isfinite(turns)) return 0;
    long double part = turns - std::floor(turns);
    part = std::round(std::ldexp(part, 64));
    return part >= 18446744073709551616.0L ? 0 : static_cast<uint64_t>(part);
}

cfwd_status cfwd_rope(const cfwd_rope_desc* desc, const void* q, const void* k, const void* positions,
                      const cfwd_rope_pair* table, void* q_out, void* k_out, void* stream) {
    return guarded([&] {
        if (!desc) return invalid("descriptor is NULL");
        const cfwd_rope_desc& d = *desc;
        if (d.tokens < 0 || d.tokens > kMaxTokens) return invalid("tokens must be between 0 and 2^38");
        if (d.q_heads < 0 || d.k_heads < 0 || d.q_heads > kMaxHeads || d.k_heads > kMaxHeads || d.q_heads + d.k_heads < 1)
            return invalid("heads must be between 0 and 65536, and not all 0");
        if (d.head_dim < 1 || d.head_dim > kMaxDim) return invalid("head_dim must be between 1 and 1024");
        if (d.pairs < 0 || 2 * static_cast<long long>(d.pairs) > d.head_dim) return invalid("pairs must be between 0 and head_dim / 2");
        if (d.axes < 1 || d.axes > 1024) return invalid("axes must be between 1 and 1024");
        const size_t es = float_size(d.dtype);
        if (!es) return invalid("dtype must be fp32 or bf16");
        const int heads[] = {d.q_heads, d.k_heads};
        const long long strides[2][4] = {{d.q_stride, d.q_head_stride, d.q_out_stride, d.q_out_head_stride},
                                         {d.k_stride, d.k_head_stride, d.k_out_stride, d.k_out_head_stride}};
        for (int i = 0; i < 2; ++i)
            if (heads[i]) {
                if (!strides_ok(d.tokens, heads[i], strides[i][0], strides[i][1])) return invalid("strides are out of range");
                if (!strides_fit(d.tokens, heads[i], d.head_dim, strides[i][2], strides[i][3]))
                    return invalid("strides of outputs must keep heads and tokens apart");
            }
        if (d.tokens == 0) return CFWD_OK;
        const void* in[] = {q, k};
        void* out[] = {q_out, k_out};
        for (int i = 0; i < 2; ++i) {
            if (heads[i] && (!in[i] || !out[i])) return invalid("NULL buffer");
            if (heads[i] && (!aligned(in[i], es) || !aligned(out[i], es))) return invalid("tensors must be aligned to their elements");
        }
        if (d.pairs && (!positions || !table)) return invalid("NULL buffer");
        if (!aligned(positions, d.wide_positions ? 8 : 4) || !aligned(table, 16))
            return invalid("positions must be aligned to their elements, the table to 16 bytes");
        Heads x[2], y[2];
        for (int i = 0; i < 2; ++i) {
            const long long e = static_cast<long long>(es);
            x[i] = {in[i], d.tokens, heads[i], strides[i][0] * e, strides[i][1] * e, d.head_dim * e};
            y[i] = {out[i], d.tokens, heads[i], strides[i][2] * e, strides[i][3] * e, d.head_dim * e};
        }
        const Span others[] = {{positions, static_cast<unsigned long long>(d.tokens) * d.axes * (d.wide_positions ? 8 : 4)},
                               {table, static_cast<unsigned long long>(d.pairs) * sizeof(cfwd_rope_pair)}};
        for (int i = 0; i < 2; ++i) {
            if (!heads[i]) continue;
            for (const Span& o : others)
                if (overlap(y[i].span(), o)) return invalid("outputs must not overlap positions or table");
            for (int j = 0; j < 2; ++j)
                if (heads[j] && !(i == j && same(x[i], y[i])) && overlap(y[i], x[j]))
                    return invalid("an output may be its own input, and must not overlap an input otherwise");
        }
        if (heads[0] && heads[1] && overlap(y[0], y[1])) return invalid("outputs must not overlap");
        return rope(desc, q, k, positions, table, q_out, k_out, static_cast<hipStream_t>(stream));
    });
}

cfwd_status cfwd_mx_cache_write(const cfwd_mx_cache_write_desc* desc, const cfwd_mx_cache* cache, const void* k,
                                const void* v, const void* slots, void* stream) {
    return guarded([&] {
        if (!desc) return invalid("descriptor is NULL");
        const cfwd_status s = check_cache(cache);
        if (s != CFWD_OK) return s;
        if (desc->tokens < 0 || desc->tokens > kMaxTokens) return invalid("tokens must be between 0 and 2^38");
        const long long es = static_cast<long long>(float_size(desc->dtype));
        if (!es) return invalid("k and v must be fp32 or bf16");
        if (!strides_ok(desc->tokens, cache->kv_heads, desc->k_stride, desc->k_head_stride) ||
            !strides_ok(desc->tokens, cache->kv_heads, desc->v_stride, desc->v_head_stride))
            return invalid("strides are out of range");
        if (desc->tokens == 0) return CFWD_OK;
        if (!k || !v || !slots) return invalid("NULL buffer");
        const cfwd_status b = check_cache_buffers(cache, true);
        if (b != CFWD_OK) return b;
        if (!aligned(k, es) || !aligned(v, es) || !aligned(slots, desc->wide_slots ? 8 : 4))
            return invalid("k, v and slots must be aligned to their elements");
        const Heads in[] = {{k, desc->tokens, cache->kv_heads, desc->k_stride * es, desc->k_head_stride * es, cache->head_dim * es},
                            {v, desc->tokens, cache->kv_heads, desc->v_stride * es, desc->v_head_stride * es, cache->head_dim * es}};
        const Span list{slots, static_cast<unsigned long long>(desc->tokens) * (desc->wide_slots ? 8 : 4)};
        const CacheSpans c = spans(cache);
        for (const Span& o : c.part)
            if (overlap(o, in[0].span()) || overlap(o, in[1].span()) || overlap(o, list))
                return invalid("the cache must not overlap k, v or slots");
        return mx_cache_write(desc, cache, k, v, slots, static_cast<hipStream_t>(stream));
    });
}

cfwd_status cfwd_mx_cache_read(const cfwd_mx_cache_read_desc* desc, const cfwd_mx_cache* cache, const int32_t* page_table,
                               const int32_t* starts, void* k, void* v, void* stream) {
    return guarded([&] {
        if (!desc) return invalid("descriptor is NULL");
        const cfwd_status s = check_cache(cache);
        if (s != CFWD_OK) return s;
        if (desc->tokens < 0 || desc->tokens >= (1ll << 31)) return invalid("tokens must be between 0 and 2^31 - 1");
        if (desc->sequences < 0) return invalid("sequences must be >= 0");
        if (desc->table_pitch < 1) return invalid("table_pitch must be at least 1");
        const size_t es = float_size(desc->dtype);
        if (!es) return invalid("k and v must be fp32 or bf16");
        if (desc->tokens == 0 || desc->sequences == 0) return CFWD_OK;
        if (!k || !v || !page_table || !starts) return invalid("NULL buffer");
        const cfwd_status b = check_cache_buffers(cache, false);
        if (b != CFWD_OK) return b;
        if (!aligned(k, es) || !aligned(v, es) || !aligned(page_table, 4) || !aligned(starts, 4))
            return invalid("k, v, page_table and starts must be aligned to their elements");
        const unsigned long long bytes = static_cast<unsigned long long>(desc->tokens) * cache->kv_heads * cache->head_dim * es;
        const Span out[] = {{k, bytes}, {v, bytes}};
        if (overlap(out[0], out[1])) return invalid("k and v must not overlap");
        const CacheSpans c = spans(cache);
        for (const Span& o : out) {
            for (const Span& i : c.part)
                if (overlap(o, i)) return invalid("k and v must not overlap the cache");
            if (overlap(o, {page_table, static_cast<unsigned long long>(desc->sequences) * desc->table_pitch * 4}) ||
                overlap(o, {starts, (desc->sequences + 1ull) * 4}))
                return invalid("k and v must not overlap page_table or starts");
        }
        return mx_cache_read(desc, cache, page_table, starts, k, v, static_cast<hipStream_t>(stream));
    });
}

cfwd_status cfwd_mx_cache_attention_workspace_size(const cfwd_mx_cache_attention_desc* desc, const cfwd_mx_cache* cache,
                                                   size_t* bytes) {
    return guarded([&] {
        const cfwd_status s = check_cache_attention(desc, cache);
        if (s != CFWD_OK) return s;
        if (!bytes) return invalid("bytes must not be NULL");
        *bytes = desc->sequences && desc->tokens ? mx_cache_attention_workspace(desc, cache) : 0;
        return CFWD_OK;
    });
}

cfwd_status cfwd_mx_cache_attention(const cfwd_mx_cache_attention_desc* desc, const cfwd_mx_cache* cache, const void* q,
                                    const int32_t* page_table, const int32_t* lengths, void* o, void* workspace,
                                    size_t ws_bytes, void* stream) {
    return guarded([&] {
        const cfwd_status s = check_cache_attention(desc, cache);
        if (s != CFWD_OK) return s;
        const cfwd_mx_cache_attention_desc& d = *desc;
        const int dim = cache->head_dim;
        if (!strides_ok(d.tokens, d.q_heads, d.q_stride, d.q_head_stride)) return invalid("strides are out of range");
        if (d.q_seq_stride < 0 || d.q_seq_stride > kMaxSpan / std::max(d.sequences, 1)) return invalid("q_seq_stride is out of range");
        if (d.q_seq_stride % 8 || d.q_stride % 8 || d.q_head_stride % 8) return invalid("strides of q must be multiples of 8 elements");
        if (d.sequences == 0 || d.tokens == 0) return CFWD_OK;
        if (!q || !page_table || !lengths || !o) return invalid("NULL buffer");
        const cfwd_status b = check_cache_buffers(cache, false);
        if (b != CFWD_OK) return b;
        if (!aligned(q, 16) || !aligned(o, 16)) return invalid("q and o must be aligned to 16 bytes");
        if (!aligned(page_table, 4) || !aligned(lengths, 4)) return invalid("page_table and lengths must be 4-byte aligned");
        const size_t need = mx_cache_attention_workspace(desc, cache);
        if (need && (!workspace || ws_bytes < need))
            return set_error(CFWD_ERR_WORKSPACE, "attention over the cache needs a workspace of " + std::to_string(need) + " bytes");
        if (need && !aligned(workspace, 256)) return invalid("workspace must be 256-byte aligned");
        const unsigned long long rows = static_cast<unsigned long long>(d.sequences) * d.tokens;
        const CacheSpans c = spans(cache);
        const Span in[] = {c.part[0], c.part[1], c.part[2], c.part[3],
                           {q, ((d.sequences - 1ull) * d.q_seq_stride + (d.tokens - 1ull) * d.q_stride + (d.q_heads - 1ull) * d.q_head_stride + dim) * 2},
                           {page_table, static_cast<unsigned long long>(d.sequences) * d.table_pitch * 4},
                           {lengths, static_cast<unsigned long long>(d.sequences) * 4}};
        const Span out{o, rows * d.q_heads * dim * 2}, work{workspace, need};
        for (const Span& i : in)
            if (overlap(out, i) || overlap(work, i)) return invalid("o and workspace must not overlap an input");
        if (overlap(out, work)) return invalid("o and workspace must not overlap");
        return mx_cache_attention(desc, cache, q, page_table, lengths, o, workspace, static_cast<hipStream_t>(stream));
    });
}

cfwd_status cfwd_attention_workspace_size(const cfwd_attention_desc* desc, size_t* bytes) {
    return guarded([&] {
        const cfwd_status s = check_attention(desc);
        if (s != CFWD_OK) return s;
        if (!bytes) return invalid("bytes must not be NULL");
        *bytes = desc->sequences && desc->q_tokens ? attention_workspace(desc) : 0;
        return CFWD_OK;
    });
}

cfwd_status cfwd_attention(const cfwd_attention_desc* desc, const void* q, const void* k, const void* v,
                           const int32_t* q_starts, const int32_t* k_starts, void* o, void* workspace, size_t ws_bytes,
                           void* stream) {
    return guarded([&] {
        const cfwd_status s = check_attention(desc);
        if (s != CFWD_OK) return s;
        const cfwd_attention_desc& d = *desc;
        if (d.sequences == 0 || d.q_tokens == 0) return CFWD_OK;
        if (!q || (d.k_tokens && (!k || !v)) || !q_starts || !k_starts || !o) return invalid("NULL buffer");
        if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16)) return invalid("q, k, v and o must be aligned to 16 bytes");
        if (!aligned(q_starts, 4) || !aligned(k_starts, 4)) return invalid("starts must be 4-byte aligned");
        const size_t need = attention_workspace(desc);
        if (need && (!workspace || ws_bytes < need))
            return set_error(CFWD_ERR_WORKSPACE, "attention needs a workspace of " + std::to_string(need) + " bytes");
        if (need && !aligned(workspace, 256)) return invalid("workspace must be 256-byte aligned");
        const Heads t[] = {{q, d.q_tokens, d.q_heads, d.q_stride * 2, d.q_head_stride * 2, d.head_dim * 2},
                           {k, d.k_tokens, d.kv_heads, d.k_stride * 2, d.k_head_stride * 2, d.head_dim * 2},
                           {v, d.k_tokens, d.kv_heads, d.v_stride * 2, d.v_head_stride * 2, d.head_dim * 2}};
        const Heads y{o, d.q_tokens, d.q_heads, static_cast<long long>(d.q_heads) * d.head_dim * 2, d.head_dim * 2ll, d.head_dim * 2ll};
        const Span starts[] = {{q_starts, (d.sequences + 1ull) * 4}, {k_starts, (d.sequences + 1ull) * 4}}, work{workspace, need};
        for (const Heads& i : t)
            if (overlap(y, i) || overlap(work, i.span())) return invalid("o and workspace must not overlap an input");
        for (const Span& i : starts)
            if (overlap(y.span(), i) || overlap(work, i)) return invalid("o and workspace must not overlap an input");
        if (overlap(y.span(), work)) return invalid("o and workspace must not overlap");
        return attention(desc, q, k, v, q_starts, k_starts, o, workspace, static_cast<hipStream_t>(stream));
    });
}

}  // extern "C"

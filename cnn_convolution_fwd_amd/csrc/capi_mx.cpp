// C ABI of the 4-bit floating point operators and the gated norms: checks of
// the arguments, then the launches (k_mx_quant.hip, k_mx_matmul.hip,
// k_gated_norm.hip).
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <string>

#include "capi_checks.h"
#include "gated_norm.h"
#include "mx.h"

namespace cfwd {
namespace {

constexpr int kMaxK = 1 << 22;
// Both keep the byte counts below in 63 bits: rows of the longest row, and rows at a pitch (in elements).
constexpr long long kMaxRows = 1ll << 38, kMaxSpan = 1ll << 60;

unsigned long long code_bytes(long long rows, long long k) { return rows * mx_code_pitch(k); }
unsigned long long scale_bytes(long long rows, long long k) { return rows * mx_scale_pitch(k); }
// rows of k elements at a pitch
unsigned long long strided_bytes(long long rows, long long k, long long pitch, size_t es) {
    return rows > 0 ? ((rows - 1) * pitch + k) * es : 0;
}

cfwd_status check_rows(long long rows, int k) {
    if (rows < 0 || rows > kMaxRows) return invalid("rows must be between 0 and 2^38");
    if (k < 1 || k > kMaxK) return invalid("the row length must be between 1 and 2^22");
    return CFWD_OK;
}

cfwd_status check_stride(long long rows, int k, long long stride) {
    if (stride < k || stride > kMaxSpan / std::max(rows, 1ll))
        return invalid("x_stride must be at least k, and rows times x_stride at most 2^60");
    return CFWD_OK;
}

cfwd_status check_matmul(const cfwd_mx_matmul_desc* d) {
    if (!d) return invalid("descriptor is NULL");
    const cfwd_status s = check_rows(d->m, d->k);
    if (s != CFWD_OK) return s;
    if (d->n < 1 || d->n > kMaxK) return invalid("n must be between 1 and 2^22");
    if (d->x_dtype != CFWD_MXFP4 && !float_size(d->x_dtype)) return invalid("x must be fp32, bf16 or MXFP4");
    if (d->y_dtype != CFWD_MXFP4 && !float_size(d->y_dtype)) return invalid("y must be fp32, bf16 or MXFP4");
    if (d->act < CFWD_ACT_NONE || d->act > CFWD_ACT_GELU) return invalid("unknown activation");
    if (d->x_dtype != CFWD_MXFP4) {
        const cfwd_status st = check_stride(d->m, d->k, d->x_stride);
        if (st != CFWD_OK) return st;
    }
    if ((d->m + 31) / 32 * ((d->n + 31) / 32) >= (1ll << 31))
        return set_error(CFWD_ERR_UNSUPPORTED, "y has too many tiles for one launch");
    return CFWD_OK;
}

}  // namespace
}  // namespace cfwd

using namespace cfwd;

extern "C" {

cfwd_status cfwd_mx_size(long long rows, int k, size_t* code, size_t* scale) {
    return guarded([&] {
        const cfwd_status s = check_rows(rows, k);
        if (s != CFWD_OK) return s;
        if (!code || !scale) return invalid("code_bytes and scale_bytes must not be NULL");
        *code = code_bytes(rows, k);
        *scale = scale_bytes(rows, k);
        return CFWD_OK;
    });
}

cfwd_status cfwd_mx_quantize(long long rows, int k, cfwd_dtype dtype, const void* x, long long x_stride, void* codes,
                             void* scales, void* stream) {
    return guarded([&] {
        const cfwd_status s = check_rows(rows, k);
        if (s != CFWD_OK) return s;
        const size_t es = float_size(dtype);
        if (!es) return invalid("x must be fp32 or bf16");
        const cfwd_status st = check_stride(rows, k, x_stride);
        if (st != CFWD_OK) return st;
        if (rows == 0) return CFWD_OK;
        if (!x || !codes || !scales) return invalid("NULL buffer");
        if (!aligned(x, es) || !aligned(codes, 16) || !aligned(scales, 4))
            return invalid("x must be aligned to its elements, codes to 16 bytes, scales to 4");
        const Span in{x, strided_bytes(rows, k, x_stride, es)}, c{codes, code_bytes(rows, k)},
            sc{scales, scale_bytes(rows, k)};
        if (overlap(in, c) || overlap(in, sc) || overlap(c, sc)) return invalid("x, codes and scales must not overlap");
        return mx_quantize(rows, k, dtype, x, x_stride, codes, scales, static_cast<hipStream_t>(stream));
    });
}

cfwd_status cfwd_mx_dequantize(long long rows, int k, cfwd_dtype dtype, const void* codes, const void* scales, void* y,
                               void* stream) {
    return guarded([&] {
        const cfwd_status s = check_rows(rows, k);
        if (s != CFWD_OK) return s;
        const size_t es = float_size(dtype);
        if (!es) return invalid("y must be fp32 or bf16");
        if (rows == 0) return CFWD_OK;
        if (!y || !codes || !scales) return invalid("NULL buffer");
        if (!aligned(y, es) || !aligned(codes, 16) || !aligned(scales, 4))
            return invalid("y must be aligned to its elements, codes to 16 bytes, scales to 4");
        const Span out{y, static_cast<unsigned long long>(rows) * k * es};
        if (overlap(out, {codes, code_bytes(rows, k)}) || overlap(out, {scales, scale_bytes(rows, k)}))
            return invalid("y must not overlap codes or scales");
        return mx_dequantize(rows, k, dtype, codes, scales, y, static_cast<hipStream_t>(stream));
    });
}

cfwd_status cfwd_mx_matmul_workspace_size(const cfwd_mx_matmul_desc* desc, size_t* bytes) {
    return guarded([&] {
        const cfwd_status s = check_matmul(desc);
        if (s != CFWD_OK) return s;
        if (!bytes) return invalid("bytes must not be NULL");
        *bytes = desc->m ? mx_matmul_workspace(desc) : 0;
        return CFWD_OK;
    });
}

cfwd_status cfwd_mx_matmul(const cfwd_mx_matmul_desc* desc, const void* x, const void* x_scales, const void* w,
                           const void* w_scales, const float* bias, void* y, void* y_scales, void* workspace,
                           size_t ws_bytes, void* stream) {
    return guarded([&] {
        const cfwd_status st = check_matmul(desc);
        if (st != CFWD_OK) return st;
        const bool x_mx = desc->x_dtype == CFWD_MXFP4, y_mx = desc->y_dtype == CFWD_MXFP4;
        if (desc->m == 0) return CFWD_OK;
        if (!x || !w || !w_scales || !y) return invalid("NULL buffer");
        if (x_mx != (x_scales != nullptr)) return invalid("x_scales goes with an MXFP4 x, and only with one");
        if (y_mx != (y_scales != nullptr)) return invalid("y_scales goes with an MXFP4 y, and only with one");
        if (!aligned(w, 16) || !aligned(w_scales, 4) || (x_mx && (!aligned(x, 16) || !aligned(x_scales, 4))) ||
            (y_mx && (!aligned(y, 16) || !aligned(y_scales, 4))))
            return invalid("codes must be aligned to 16 bytes, scales to 4");
        if ((!x_mx && !aligned(x, float_size(desc->x_dtype))) || (!y_mx && !aligned(y, float_size(desc->y_dtype))))
            return invalid("x and y must be aligned to their elements");
        if (!aligned(bias, 4)) return invalid("bias must be 4-byte aligned");
        const long long m = desc->m;
        const int n = desc->n, k = desc->k;
        const Span in[] = {{x, x_mx ? code_bytes(m, k) : strided_bytes(m, k, desc->x_stride, float_size(desc->x_dtype))},
                           {x_scales, scale_bytes(m, k)}, {w, code_bytes(n, k)}, {w_scales, scale_bytes(n, k)},
                           {bias, n * 4ull}};
        const size_t need = mx_matmul_workspace(desc);
        if (need && (!workspace || ws_bytes < need))
            return set_error(CFWD_ERR_WORKSPACE, "the product needs a workspace of " + std::to_string(need) + " bytes");
        if (need && !aligned(workspace, 256)) return invalid("workspace must be 256-byte aligned");
        const Span out[] = {{y, y_mx ? code_bytes(m, n) : static_cast<unsigned long long>(m) * n * float_size(desc->y_dtype)},
                            {y_scales, scale_bytes(m, n)}, {workspace, need}};
        for (const Span& o : out)
            for (const Span& i : in)
                if (overlap(o, i)) return invalid("y, y_scales and workspace must not overlap an input");
        if (overlap(out[0], out[1]) || overlap(out[0], out[2]) || overlap(out[1], out[2]))
            return invalid("y, y_scales and workspace must not overlap");
        return mx_matmul(desc, x, x_scales, w, w_scales, bias, y, y_scales, workspace, static_cast<hipStream_t>(stream));
    });
}

cfwd_status cfwd_gated_norm(const cfwd_gated_norm_desc* desc, const void* b, const void* residual, const void* gate,
                            const float* post_weight, const float* post_bias, const float* pre_weight,
                            const float* pre_bias, void* s, void* h, void* h_scales, void* stream) {
    return guarded([&] {
        if (!desc) return invalid("descriptor is NULL");
        const cfwd_status st = check_rows(desc->rows, desc->c);
        if (st != CFWD_OK) return st;
        for (cfwd_norm_kind kind : {desc->post, desc->pre})
            if (kind < CFWD_NORM_NONE || kind > CFWD_NORM_LAYER) return invalid("unknown norm");
        const size_t es = float_size(desc->dtype), ss = float_size(desc->stream_dtype);
        if (!es || !ss || (ss < es && (b || gate)))
            return invalid("dtype must be fp32 or bf16, stream_dtype fp32 or dtype (either without b and gate)");
        const bool h_mx = desc->out_dtype == CFWD_MXFP4;
        if (!h_mx && desc->out_dtype != desc->dtype) return invalid("out_dtype must be dtype or MXFP4");
        if (!(desc->eps >= 0.0f) || std::isinf(desc->eps)) return invalid("eps must be a number >= 0");
        if (desc->rows_per_gate < 0) return invalid("rows_per_gate must be >= 0");
        if (desc->rows == 0) return CFWD_OK;
        if (!b && !residual) return invalid("b and residual must not both be NULL");
        if (!s && !h) return invalid("s and h must not both be NULL");
        if ((h && h_mx) != (h_scales != nullptr)) return invalid("h_scales goes with an MXFP4 h, and only with one");
        if (!aligned(b, es) || !aligned(gate, es) || !aligned(residual, ss) || !aligned(s, ss) || (!h_mx && !aligned(h, es)))
            return invalid("tensors must be aligned to their elements");
        if (h_mx && (!aligned(h, 16) || !aligned(h_scales, 4))) return invalid("codes must be aligned to 16 bytes, scales to 4");
        for (const float* p : {post_weight, post_bias, pre_weight, pre_bias})
            if (!aligned(p, 4)) return invalid("weights and biases must be 4-byte aligned");
        const unsigned long long count = static_cast<unsigned long long>(desc->rows) * desc->c;
        const long long gates = desc->rows_per_gate ? (desc->rows - 1) / desc->rows_per_gate + 1 : 1;
        const Span in[] = {{b, count * es}, {residual, count * ss}, {gate, static_cast<unsigned long long>(gates) * desc->c * es},
                           {post_weight, desc->c * 4ull}, {post_bias, desc->c * 4ull}, {pre_weight, desc->c * 4ull},
                           {pre_bias, desc->c * 4ull}};
        const Span sum{s, count * ss}, out{h, h_mx ? code_bytes(desc->rows, desc->c) : count * es},
            out_scales{h_scales, scale_bytes(desc->rows, desc->c)};
        for (const Span& i : in) {
            if (overlap(out, i) || overlap(out_scales, i)) return invalid("h must not overlap an input");
            const bool same = (&i == &in[0] || &i == &in[1]) && i.p == s && i.bytes == sum.bytes;
            if (!same && overlap(sum, i)) return invalid("s may be residual or b itself, and must not overlap an input otherwise");
        }
        if (overlap(sum, out) || overlap(sum, out_scales) || overlap(out, out_scales))
            return invalid("s, h and h_scales must not overlap");
        return gated_norm(desc, {b, residual, gate, post_weight, post_bias, pre_weight, pre_bias, s, h, h_scales},
                          static_cast<hipStream_t>(stream));
    });
}

}  // extern "C"

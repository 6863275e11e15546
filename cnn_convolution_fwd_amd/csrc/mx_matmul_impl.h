// Device pieces that the kernels of the MXFP4 product share (k_mx_matmul.hip):
// addressing of the operands, and the output pass.
//
// The product runs on v_mfma_scale_f32_32x32x64_f8f6f4 with w as the A operand
// and x as B: a lane of half h = lane / 32 holds one block (32 values, 16
// bytes) of row lane % 32 of each, with the block's scale byte, and ends with
// 16 outputs of one row of y: columns 8 g + 4 h + i (g, i < 4) of 32.
//
// A stage is 256 values of K, 8 blocks, as four such instructions, or half of
// that.  The order of the sum is free as long as both operands agree, so half h
// takes the stage's blocks 4 h .. 4 h + 3 (or 2 h and 2 h + 1), one an
// instruction: their scale bytes are then in one aligned word, and each
// instruction names its byte.
#pragma once

#include "mx.h"

#include <type_traits>

namespace cfwd {
namespace mx {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct MatmulParams {
    const uint8_t *x, *xs, *w, *ws;  // x: codes, or (stream kernel) values of x_stride elements a row
    long long x_stride;
    int k;
    const float* bias;
    void* y;
    uint8_t* ys;
    long long m;
    int n, kb;  // kb: blocks of a row
    int pitch, spitch;  // bytes of a row of codes / scales of x and w
    int act;
    int ldy;                // row pitch of an fp32 / bf16 y, in elements
    int y_pitch, y_spitch;  // MXFP4 outputs
};

constexpr uint32_t kOutOfRange = 0x7ffffff0u;  // a buffer offset past every range: loads give 0

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, long long bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0,
                                             static_cast<int>(bytes < 0 ? 0 : bytes > 0x7fffffe0ll ? 0x7fffffe0ll : bytes),
                                             0x00020000);
}

template <int J>
__device__ __forceinline__ f32x16 mfma(const i32x4& a, const i32x4& b, const f32x16& c, int sa, int sb) {
    const i32x8 a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, b8 = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, J, sa, J, sb);
}

// Bits of the scale bytes of two neighbouring blocks, of which `left` (2 or more: both) are blocks of the row:
// what the bytes past a row's blocks hold does not count.
__device__ __forceinline__ int scale_bits(int left) { return min(max(left, 0), 2) * 8; }

// 8 finished values of y's row from column n on, `valid` of them columns of y.
// An MXFP4 block's four runs belong to a quad of lanes, which all call this.
template <typename TY>
__device__ __forceinline__ void store_run(const MatmulParams& p, long long row, int n, int valid, float (&v)[8]) {
    if constexpr (!std::is_void<TY>::value) {
        if (valid > 0) store8(static_cast<TY*>(p.y) + row * p.n + n, valid, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < valid ? v[i] : 0.0f;
        uint32_t byte;
        const uint32_t codes = quantize8(v, &byte);
        const int block = n / 32;
        if (block * 16 >= p.y_pitch) return;
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.y) + row * p.y_pitch + n / 2) = codes;
        if (n % 32) return;
        uint8_t* s = p.ys + row * p.y_spitch;
        s[block] = static_cast<uint8_t>(byte);
        if ((block + 1) * 16 == p.y_pitch)  // the last block also writes what rounds the row up to whole words
            for (int i = block + 1; i < p.y_spitch; ++i) s[i] = 127;
    }
}

// The output pass of one wave: 32 FM rows of y x 32 FN columns from (m0, n0)
// on, with activation and the one rounding.
//
// fp32 and bf16 results take a turn through the wave's own LDS area (32 rows, of
// one or half a set of columns' fragments; 16-byte slots permuted by row instead
// of padded, and of bf16 their halves in rows 16 to 31, whose slots are those of
// rows 0 to 15), so that whole runs of columns are stored.  An MXFP4 block (32
// columns of a row) is spread over the two lanes r and r + 32, which exchange
// halves of two blocks, so that each then holds a block's 16 bytes.
//
// `fast`: rows of y are whole 16-byte runs, which leave as buffer stores,
// out-of-range ones dropped by the hardware: each wave then issues exactly
// stores<FM, FN, TY>() of them.  Otherwise stores follow the row's ends.
template <int FM, int FN, typename TY>
constexpr int stores() {
    return std::is_void<TY>::value ? FM * FN : FM * FN * (std::is_same<TY, float>::value ? 4 : 2);
}

// v / (1 + 2^power(v)), eight values at a time and step by step: a value's
// exponential and reciprocal, one right after the other, would each hold up the
// instruction that takes it.  WHOLE: the power in two parts, as an fp32 silu
// takes it (25088 x 2048 x 512 to fp32: 41.5 us without activation, 44.3 with the power
// in one part, 50 in two).
template <bool WHOLE, typename Power>
__device__ __forceinline__ void logistic16(float (&v)[16], Power power) {
#pragma unroll
    for (int g = 0; g < 16; g += 8) {
        float t[8], n[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            n[i] = WHOLE ? silu_whole(v[g + i]) : 0.0f;
            t[i] = power(v[g + i], n[i]);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = __builtin_amdgcn_exp2f(t[i]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = 1.0f + (WHOLE ? __builtin_ldexpf(t[i], static_cast<int>(n[i])) : t[i]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = __builtin_amdgcn_rcpf(t[i]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[g + i] *= t[i];
    }
}

template <typename TY>
__device__ __forceinline__ void activate16(float (&v)[16], int act) {
    if (act == CFWD_ACT_NONE) return;
    if (act == CFWD_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = activate<TY>(v[i], CFWD_ACT_RELU);
    } else if (act == CFWD_ACT_GELU) {
        logistic16<false>(v, [](float u, float) { return gelu_exponent(u); });
    } else if constexpr (std::is_same<TY, float>::value) {
        logistic16<true>(v, silu_rest);
    } else {
        logistic16<false>(v, [](float u, float) { return silu_exponent(u); });
    }
}

__device__ __forceinline__ void wave_sync() {  // a wave's LDS writes before its later reads, and the reverse
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_sched_barrier(0);  // and no register holds more than one turn's results
}

// bias of a lane's columns of the 32 F from n on; 0 if there is none
template <int F>
__device__ __forceinline__ void load_bias(const MatmulParams& p, int n, float (&v)[F][16]) {
    const __amdgpu_buffer_rsrc_t b = buffer(p.bias, p.bias ? p.n * 4ll : 0);
    const int h = (threadIdx.x >> 5) & 1;
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const u32x4 q = __builtin_amdgcn_raw_buffer_load_b128(b, (n + f * 32 + g * 8 + h * 4) * 4, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[f][g * 4 + i] = __uint_as_float(q[i]);
        }
}

template <int FM, int FN, typename TY>
__device__ __forceinline__ void write_tile(const f32x16 (&acc)[FM][FN], const MatmulParams& p, long long m0, int n0, bool fast,
                                           uint8_t* area) {
    uint32_t lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));  // keeps the pass's many addresses from being computed, and held, outside the caller's loop
    const uint32_t r = lane & 31, h = (lane >> 5) & 1;
    const long long rows = min(32ll * FM, p.m - m0);
    if constexpr (!std::is_void<TY>::value) {
        constexpr int ES = sizeof(TY), CF = ES == 4 ? FN / 2 : FN;  // columns' fragments of one turn
        constexpr int ROW = CF * 32 * ES, SLOTS = ROW / 16, RUN = 16 / ES;
        constexpr int RUNS = SLOTS / 2, STEP = 64 / SLOTS;  // of a lane in a turn; rows of one access of the wave
        const long long pitch = static_cast<long long>(p.ldy) * ES;
        uint8_t* y0 = static_cast<uint8_t*>(p.y) + m0 * pitch + static_cast<long long>(n0) * ES;
        const __amdgpu_buffer_rsrc_t y = buffer(y0, (rows - 1) * pitch + (static_cast<long long>(p.ldy) - n0) * ES);
        const uint32_t row0 = lane / SLOTS, slot = lane % SLOTS;
        static_assert(SLOTS == 8, "two rows span the banks");
        auto turned = [](uint32_t row) { return (row >> 1 & 7) * 16; };
        const uint32_t put = r * ROW + (turned(r) ^ (ES == 4 ? h * 16 : (h ^ r >> 4) * 8));
        auto store_turn = [&](int i, int f0, const u32x4(&t)[RUNS]) {
            const int c = f0 * 32 + static_cast<int>(slot) * RUN, valid = p.n - n0 - c;
            if (fast) {
                const uint32_t off = valid > 0 ? row0 * static_cast<uint32_t>(pitch) + c * ES : kOutOfRange;
#pragma unroll
                for (int u = 0; u < RUNS; ++u)
                    __builtin_amdgcn_raw_buffer_store_b128(t[u], y, off + (i * 32 + u * STEP) * static_cast<uint32_t>(pitch), 0, 0);
                return;
            }
#pragma unroll
            for (int u = 0; u < RUNS; ++u) {
                const int row = i * 32 + u * STEP + static_cast<int>(row0);
                if (row >= rows || valid <= 0) continue;
                TY* dst = reinterpret_cast<TY*>(y0 + row * pitch) + c;
                if (valid >= RUN) {
                    *reinterpret_cast<Raw16*>(dst) = Raw16{{t[u][0], t[u][1], t[u][2], t[u][3]}};
                    continue;
                }
#pragma unroll
                for (int j = 0; j < RUN; ++j)
                    if (j < valid) {
                        if constexpr (ES == 4)
                            dst[j] = __uint_as_float(t[u][j]);
                        else
                            dst[j].bits = static_cast<uint16_t>(t[u][j / 2] >> (j % 2 * 16));
                    }
            }
        };
        // a turn's results come back from LDS while the next turn's are computed
        constexpr int TURNS = FM * (FN / CF);
        u32x4 t[RUNS];
#pragma unroll
        for (int turn = 0; turn < TURNS; ++turn) {
            const int i = turn / (FN / CF), f0 = turn % (FN / CF) * CF;
#pragma unroll
            for (int f = 0; f < CF; ++f) {
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = acc[i][f0 + f][j];
                activate16<TY>(v, p.act);
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    uint8_t* at = area + (put ^ static_cast<uint32_t>((f * 32 + g * 8) * ES));
                    if constexpr (ES == 4)
                        *reinterpret_cast<float4*>(at) = make_float4(v[g * 4], v[g * 4 + 1], v[g * 4 + 2], v[g * 4 + 3]);
                    else
                        *reinterpret_cast<uint2*>(at) =
                            make_uint2(pack_bf16x2(v[g * 4], v[g * 4 + 1]), pack_bf16x2(v[g * 4 + 2], v[g * 4 + 3]));
                }
            }
            wave_sync();
            if (turn > 0) store_turn((turn - 1) / (FN / CF), (turn - 1) % (FN / CF) * CF, t);
#pragma unroll
            for (int u = 0; u < RUNS; ++u) {
                const uint32_t row = u * STEP + row0;
                t[u] = *reinterpret_cast<const u32x4*>(area + (row * ROW + (turned(row) ^ slot * 16)));
                if (ES == 2 && u * STEP >= 16) t[u] = u32x4{t[u][2], t[u][3], t[u][0], t[u][1]};
            }
            wave_sync();
        }
        store_turn(FM - 1, FN - CF, t);
    } else {
        const __amdgpu_buffer_rsrc_t y = buffer(static_cast<uint8_t*>(p.y) + m0 * p.y_pitch, rows * p.y_pitch),
                                     ys = buffer(p.ys + m0 * p.y_spitch, rows * p.y_spitch);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int f0 = 0; f0 < FN; f0 += 2) {
                uint32_t half[2][2], byte[2];  // this lane's halves of two blocks: codes of g = 0, 1 and of g = 2, 3
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int nb = n0 + (f0 + q) * 32;
                    float v[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = acc[i][f0 + q][j];
                    activate16<TY>(v, p.act);
                    if (nb + 32 > p.n) {  // columns past the row are no part of its last block
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = nb + j / 4 * 8 + static_cast<int>(h) * 4 + j % 4 < p.n ? v[j] : 0.0f;
                    }
                    // the largest |v|: the largest of v's bits as signed numbers is that of the positive values if there
                    // are any, as unsigned ones that of the negative values; without their signs the greater of the two
                    int most = static_cast<int>(__float_as_uint(v[0]));
                    uint32_t top = __float_as_uint(v[0]);
#pragma unroll
                    for (int j = 1; j < 16; ++j) {
                        most = max(most, static_cast<int>(__float_as_uint(v[j])));
                        top = max(top, __float_as_uint(v[j]));
                    }
                    top = max(top & 0x7fffffffu, static_cast<uint32_t>(most) & 0x7fffffffu);
                    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32)));
                    byte[q] = nb < p.n ? exponent_byte(top) : 127u;
                    const float s = scale_of(byte[q]);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        uint32_t c = 0;
                        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[t * 8], v[t * 8 + 1], s, 0);
                        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[t * 8 + 2], v[t * 8 + 3], s, 1);
                        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[t * 8 + 4], v[t * 8 + 5], s, 2);
                        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[t * 8 + 6], v[t * 8 + 7], s, 3);
                        half[q][t] = byte[q] == 255 ? 0u : c;
                    }
                }
                // lanes of half 0 take block f0, those of half 1 block f0 + 1
                u32x4 block;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const auto x = __builtin_amdgcn_permlane32_swap(half[0][t], half[1][t], false, false);
                    block[2 * t] = __builtin_amdgcn_perm(x[1], x[0], 0x05040100u);
                    block[2 * t + 1] = __builtin_amdgcn_perm(x[1], x[0], 0x07060302u);
                }
                __builtin_amdgcn_sched_barrier(0);  // no register holds more than one turn's results
                const int nb = n0 / 32 + f0 + static_cast<int>(h);    // rows past the end are out of the buffers' range
                const uint32_t off = nb * 16 < p.y_pitch ? r * p.y_pitch + nb * 16 : kOutOfRange;
                const uint32_t soff = nb < p.y_spitch ? r * p.y_spitch + nb : kOutOfRange;
                __builtin_amdgcn_raw_buffer_store_b128(block, y, off + i * 32 * p.y_pitch, 0, 0);
                __builtin_amdgcn_raw_buffer_store_b8(static_cast<uint8_t>(h ? byte[1] : byte[0]), ys,
                                                     soff + i * 32 * p.y_spitch, 0, 0);
            }
    }
}

}  // namespace mx

// Few rows (k_mx_stream.hip).  `x`: MXFP4, or x's own type where mx_stream_takes_raw says so.
bool mx_stream_supported(long long m, int n, int k);
bool mx_stream_takes_raw(const cfwd_mx_matmul_desc* d);
cfwd_status mx_stream(const mx::MatmulParams& p, cfwd_dtype x, cfwd_dtype y, int cus, hipStream_t st);

}  // namespace cfwd

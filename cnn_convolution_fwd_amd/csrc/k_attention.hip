// Attention over packed prompts (gfx950).
//
//   o = softmax(scale * q k^T) v
//
// A workgroup takes 128 RB rows of one head of keys and values, a row being a (token,
// query head) of the group that shares it: grouped heads read their keys once,
// and a tile of rows spans few tokens, which wastes little at the causal edge.
// Keys and values come 64 at a time through LDS, by copies that bypass the
// registers, STAGES deep.  S^T = k q^T has a query in each lane's column and 16 keys
// in its registers, which is how P^T enters O^T = v^T P^T: only the row's maximum
// and sum pass between lanes (two of them hold a row).  v^T comes out of LDS by transposing reads.
// With m the running maximum, O and l are multiplied by 2^(m - m') only
// where a score passes m by more than 2^8: until then weights up to 2^8 are as
// good.  A row goes by its own scores alone, so that its result does not depend on the others'.
//
// Few rows over many keys are split over the keys; a second launch joins the parts.
#include "attention.h"
#include "mx.h"

#include <algorithm>

namespace cfwd {
namespace fa {

using namespace mx;
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) u32x4_t lds_u32x4;

constexpr int BN = 64;          // keys of a tile
constexpr float kLow = -3.0e38f;  // m before any score: finite, so that differences are numbers
constexpr float kSlack = 8.0f;

struct Params {
    const bf16_t *q, *k, *v;
    bf16_t* o;
    const int32_t *q_starts, *k_starts;
    float *part, *part_ml;  // [split][row of q x heads][dim], [..][m, l]
    int sequences, heads, kv_heads, group, dim, causal, splits;
    int q_tokens, k_tokens;
    float scale2;  // scale * log2(e)
    long long q_stride, q_head_stride, k_stride, k_head_stride, v_stride, v_head_stride;
    Divisor per_group;
};

__device__ __forceinline__ void load_to_lds16(const __amdgpu_buffer_rsrc_t& b, uint32_t off, uint32_t lds) {
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" : : "{m0}"(lds), "v"(off), "s"(b) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads() {  // until at most N of this wave's loads are outstanding
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// All waves of the workgroup, each with its reads of LDS done: what they read may then be overwritten.
__device__ __forceinline__ void barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes), 0x00020000);
}

__device__ __forceinline__ f32x16 mma(const u32x4_t& a, const u32x4_t& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Rows of a tile in LDS are DP values; their 16-byte pieces are permuted so that
// the reads of 16 rows' same piece (keys), and of 4 rows' same 4 pieces (values), cover all of LDS's banks.
template <int DP>
__device__ __forceinline__ int k_swizzle(int row) { return DP == 64 ? (row >> 1) & 7 : row & 15; }
template <int DP>
__device__ __forceinline__ int v_swizzle(int row) { return DP == 64 ? ((row >> 1) & 1) * 4 : (row & 3) * 4; }

struct Range {
    int from, count;
};
__device__ __forceinline__ Range rows_of(const int32_t* starts, int seq, int tokens) {
    const int a = min(max(starts[seq], 0), tokens), b = min(max(starts[seq + 1], a), tokens);
    return {a, b - a};
}

// The sequence of the tile `tile`, counted from the last one back, and its tile; seq < 0: there is none.
struct Place {
    int seq, tile;
};
template <int BM>
__device__ Place find_tile(const Params& p, int tile, int lane) {
    int total = 0;
    for (int s = 0; s < p.sequences; s += 64) {
        int n = 0;
        if (s + lane < p.sequences) n = (rows_of(p.q_starts, s + lane, p.q_tokens).count * p.group + BM - 1) / BM;
        total += n;
    }
#pragma unroll
    for (int d = 32; d; d /= 2) total += __shfl_xor(total, d);
    const int x = total - 1 - tile;
    if (x < 0) return {-1, 0};
    int before = 0;
    for (int s = 0; s < p.sequences; s += 64) {
        int n = 0;
        if (s + lane < p.sequences) n = (rows_of(p.q_starts, s + lane, p.q_tokens).count * p.group + BM - 1) / BM;
        int upto = n;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(upto, d);
            if (lane >= d) upto += o;
        }
        upto += before;
        const unsigned long long past = __ballot(upto > x);
        if (past) {
            const int at = __ffsll(past) - 1;
            return {s + at, x - __shfl(upto - n, at)};
        }
        before = __shfl(upto, 63);
    }
    return {-1, 0};
}

template <int DP, int NK, int NV, int RB, int STAGES, int RESIDENT>
__global__ __launch_bounds__(256, RESIDENT) void kernel(Params p) {
    constexpr int BM = 128 * RB, PIECES = DP / 8, TILE = BN * DP * 2;
    constexpr int COPIES = BN * PIECES / 256;  // of 16 bytes, a thread and tile
    __shared__ __attribute__((aligned(1024))) uint8_t area[STAGES * 2 * TILE];
    const uint32_t lds = static_cast<uint32_t>(
        reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)area));
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 31, h = lane >> 5;
    const int head = blockIdx.x % p.kv_heads;
    const Place place = find_tile<BM>(p, blockIdx.x / p.kv_heads, lane);
    const int seq = __builtin_amdgcn_readfirstlane(place.seq);
    if (seq < 0) return;
    const int row0 = __builtin_amdgcn_readfirstlane(place.tile) * BM;
    const Range qs = rows_of(p.q_starts, seq, p.q_tokens), ks = rows_of(p.k_starts, seq, p.k_tokens);
    const int rows = qs.count * p.group;
    // row r sees the keys before offset + r / group + 1, and before ks.count
    const int offset = ks.count - qs.count;
    const int last_token = divide(min(row0 + BM, rows) - 1, p.per_group);
    const int keys = p.causal ? min(max(offset + last_token + 1, 0), ks.count) : ks.count;
    const int all_tiles = (keys + BN - 1) / BN;
    const int t0 = static_cast<int>(static_cast<long long>(blockIdx.y) * all_tiles / p.splits);
    const int t1 = static_cast<int>(static_cast<long long>(blockIdx.y + 1) * all_tiles / p.splits);

    // this wave's rows
    const int wave0 = row0 + wave * 32 * RB;
    int seen[RB];
    u32x4_t q[RB][NK];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
        const int row = min(wave0 + r * 32 + n, rows - 1);
        const int token = divide(row, p.per_group);
        seen[r] = p.causal ? min(offset + token + 1, ks.count) : ks.count;
        const bf16_t* x = p.q + (qs.from + token) * p.q_stride + (head * p.group + row - token * p.group) * p.q_head_stride;
#pragma unroll
        for (int c = 0; c < NK; ++c) {
            const int d = 16 * c + 8 * h;
            q[r][c] = d < p.dim ? *reinterpret_cast<const u32x4_t*>(x + d) : u32x4_t{0, 0, 0, 0};
        }
    }
    const int first_token = divide(min(wave0, rows - 1), p.per_group);
    const int least = p.causal ? min(offset + first_token + 1, ks.count) : ks.count;  // every row of the wave sees these
    const int wave_last = divide(min(wave0 + 32 * RB, rows) - 1, p.per_group);
    const int most = wave0 >= rows ? 0 : p.causal ? min(offset + wave_last + 1, ks.count) : ks.count;

    // copies: piece i * 256 + thread of a tile, from the place that the permutation puts there; outside dim: nothing
    uint32_t k_off[COPIES], v_off[COPIES];
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
        const int at = i * 256 + threadIdx.x, row = at / PIECES, piece = at % PIECES;
        const int kp = piece ^ k_swizzle<DP>(row), vp = piece ^ v_swizzle<DP>(row);
        k_off[i] = kp * 8 < p.dim ? static_cast<uint32_t>(row * p.k_stride + kp * 8) * 2 : 0xfffffff0u;
        v_off[i] = vp * 8 < p.dim ? static_cast<uint32_t>(row * p.v_stride + vp * 8) * 2 : 0xfffffff0u;
    }
    const bf16_t* kbase = p.k + ks.from * p.k_stride + head * p.k_head_stride;
    const bf16_t* vbase = p.v + ks.from * p.v_stride + head * p.v_head_stride;
    auto copy = [&](int t) __attribute__((always_inline)) {
        // rows from the sequence's end on are out of the buffer's range and become zeros
        const int left = t < t1 ? min(ks.count - t * BN, BN) : 0;
        const uint32_t to = lds + (t % STAGES) * 2 * TILE + wave * 1024;
        const auto kb = buffer(kbase + static_cast<long long>(t) * BN * p.k_stride, left * static_cast<uint32_t>(p.k_stride) * 2);
        const auto vb = buffer(vbase + static_cast<long long>(t) * BN * p.v_stride, left * static_cast<uint32_t>(p.v_stride) * 2);
#pragma unroll
        for (int i = 0; i < COPIES; ++i) load_to_lds16(kb, k_off[i], to + i * 4096);
#pragma unroll
        for (int i = 0; i < COPIES; ++i) load_to_lds16(vb, v_off[i], to + TILE + i * 4096);
    };

    f32x16 o[RB][NV];
    float m[RB], l[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
        m[r] = kLow;
        l[r] = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 16; ++j) o[r][i][j] = 0.0f;
    }

    for (int s = 0; s < STAGES - 1; ++s) copy(t0 + s);
    for (int t = t0; t < t1; ++t) {
        wait_loads<(STAGES - 2) * 2 * COPIES>();
        barrier();  // tile t is whole, and tile t - 1's stage is free
        copy(t + STAGES - 1);
        if (t * BN >= most) continue;
        const uint32_t kt = lds + (t % STAGES) * 2 * TILE, vt = kt + TILE;
        f32x16 score[RB][2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int j = 0; j < 16; ++j) score[r][b][j] = 0.0f;
            const int row = 32 * b + n;
#pragma unroll
            for (int c = 0; c < NK; ++c) {
                const u32x4_t f = *reinterpret_cast<lds_u32x4*>(kt + row * DP * 2 + ((2 * c + h) ^ k_swizzle<DP>(row)) * 16);
#pragma unroll
                for (int r = 0; r < RB; ++r) score[r][b] = mma(f, q[r][c], score[r][b]);
            }
        }
        if (t * BN + BN > least) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int key = t * BN + 32 * b + 8 * (j / 4) + 4 * h + j % 4;
#pragma unroll
                    for (int r = 0; r < RB; ++r)
                        if (key >= seen[r]) score[r][b][j] = -__builtin_inff();
                }
        }
        u32x4_t weight[RB][4];
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            float top = score[r][0][0];
#pragma unroll
            for (int j = 1; j < 32; ++j) top = fmaxf(top, score[r][j / 16][j % 16]);
            top *= p.scale2;
            if (__any(top > m[r] + kSlack)) {
                top = fmaxf(top, __shfl_xor(top, 32));
                const float to = top > m[r] + kSlack ? top : m[r], f = __builtin_amdgcn_exp2f(m[r] - to);
                m[r] = to;
                l[r] *= f;
#pragma unroll
                for (int i = 0; i < NV; ++i) o[r][i] *= f;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(score[r][i / 8][2 * i % 16], p.scale2, -m[r]));
                const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(score[r][i / 8][2 * i % 16 + 1], p.scale2, -m[r]));
                const uint32_t w = pack_bf16x2(e0, e1);
                weight[r][i / 4][i % 4] = w;
                // the sum takes the weights as they enter the product: rounded
                l[r] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, w),
                                                       __builtin_bit_cast(bf16x2_t, 0x3f803f80u), l[r], false);
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)  // 16 keys: 16 c + 4 h + (0 .. 3) and 8 on
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                u32x4_t f;
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    // four lanes point at 16 values of each of four keys; a lane gets one value of all four
                    const int in = lane & 15, row = 16 * c + 8 * part + 4 * h + (in >> 2);
                    const int d = 32 * i + 16 * ((lane >> 4) & 1) + 4 * (in & 3);
                    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4*>(
                        vt + row * DP * 2 + ((d >> 3) ^ v_swizzle<DP>(row)) * 16 + (d & 7) * 2));
                    const uint2 y = __builtin_bit_cast(uint2, x);
                    f[2 * part] = y.x;
                    f[2 * part + 1] = y.y;
                }
#pragma unroll
                for (int r = 0; r < RB; ++r) o[r][i] = mma(f, weight[r][c], o[r][i]);
            }
    }
    wait_loads<0>();  // none is left on its way to LDS that the next workgroup may own

#pragma unroll
    for (int r = 0; r < RB; ++r) {
        l[r] += __shfl_xor(l[r], 32);
        const int row = wave0 + r * 32 + n;
        if (row >= rows) continue;
        const int token = divide(row, p.per_group);
        const long long at = static_cast<long long>(qs.from + token) * p.heads + head * p.group + row - token * p.group;
        if (p.splits == 1) {
            const float inverse = l[r] == 0.0f ? 0.0f : 1.0f / l[r];
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int d = 32 * i + 8 * j + 4 * h;
                    if (d >= p.dim) continue;
                    uint2 y;
                    y.x = pack_bf16x2(o[r][i][4 * j] * inverse, o[r][i][4 * j + 1] * inverse);
                    y.y = pack_bf16x2(o[r][i][4 * j + 2] * inverse, o[r][i][4 * j + 3] * inverse);
                    *reinterpret_cast<uint2*>(p.o + at * p.dim + d) = y;
                }
        } else {
            const long long to = at * p.splits + blockIdx.y;
            if (h == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * to) = make_float2(m[r], l[r]);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int d = 32 * i + 8 * j + 4 * h;
                    if (d < p.dim)
                        *reinterpret_cast<f32x4*>(p.part + to * p.dim + d) =
                            f32x4{o[r][i][4 * j], o[r][i][4 * j + 1], o[r][i][4 * j + 2], o[r][i][4 * j + 3]};
                }
        }
    }
}

// Joins the splits of rows (token, head) of q: 4 values a thread.
__global__ __launch_bounds__(256) void join_kernel(Params p, Divisor across, uint32_t units) {
    const uint32_t u = blockIdx.x * 256u + threadIdx.x;
    if (u >= units) return;
    const uint32_t row = divide(u, across), d = (u - row * across.d) * 4;
    // rows before the first sequence and behind the last belong to none
    const int token = row / p.heads;
    if (token < p.q_starts[0] || token >= p.q_starts[p.sequences]) return;
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + static_cast<long long>(row) * p.splits;
    const float* part = p.part + static_cast<long long>(row) * p.splits * p.dim + d;
    float m = kLow;
    for (int s = 0; s < p.splits; ++s) m = fmaxf(m, ml[s].x);
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    float l = 0.0f;
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) {
        const float f = __builtin_amdgcn_exp2f(ml[s].x - m);
        l += ml[s].y * f;
        sum += *reinterpret_cast<const f32x4*>(part + static_cast<long long>(s) * p.dim) * f;
    }
    const float inverse = l == 0.0f ? 0.0f : 1.0f / l;
    uint2 y;
    y.x = pack_bf16x2(sum[0] * inverse, sum[1] * inverse);
    y.y = pack_bf16x2(sum[2] * inverse, sum[3] * inverse);
    *reinterpret_cast<uint2*>(p.o + static_cast<long long>(row) * p.dim + d) = y;
}

struct Plan {
    int rb, splits;
    long long tiles;  // upper bound
    size_t part_bytes, bytes;
};

Plan plan(const cfwd_attention_desc* d) {
    Plan r{};
    const long long group = d->q_heads / d->kv_heads, cus = compute_units();
    auto tiles = [&](int bm) { return std::max(1ll, d->q_tokens * group / bm + std::min<long long>(d->sequences, d->q_tokens)); };
    r.rb = d->head_dim <= 128 && tiles(256) * d->kv_heads >= cus ? 2 : 1;
    r.tiles = tiles(128 * r.rb);
    const long long keys = d->k_tokens / std::max(1, d->sequences);
    r.splits = static_cast<int>(std::max(1ll, std::min({2 * cus / (r.tiles * d->kv_heads), keys / 256, 64ll})));
    if (r.splits > 1) {
        const size_t n = static_cast<size_t>(d->q_tokens) * d->q_heads * r.splits;
        r.part_bytes = (n * d->head_dim * 4 + 255) / 256 * 256;
        r.bytes = r.part_bytes + n * 8;
    }
    return r;
}

}  // namespace fa

size_t attention_workspace(const cfwd_attention_desc* d) { return fa::plan(d).bytes; }

cfwd_status attention(const cfwd_attention_desc* d, const void* q, const void* k, const void* v, const int32_t* q_starts,
                      const int32_t* k_starts, void* o, void* workspace, hipStream_t st) {
    const fa::Plan plan = fa::plan(d);
    fa::Params p{};
    p.q = static_cast<const bf16_t*>(q);
    p.k = static_cast<const bf16_t*>(k);
    p.v = static_cast<const bf16_t*>(v);
    p.o = static_cast<bf16_t*>(o);
    p.q_starts = q_starts;
    p.k_starts = k_starts;
    p.part = static_cast<float*>(workspace);
    p.part_ml = plan.splits > 1 ? reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.part_bytes) : nullptr;
    p.sequences = d->sequences;
    p.heads = d->q_heads;
    p.kv_heads = d->kv_heads;
    p.group = d->q_heads / d->kv_heads;
    p.dim = d->head_dim;
    p.causal = d->causal;
    p.splits = plan.splits;
    p.q_tokens = static_cast<int>(d->q_tokens);
    p.k_tokens = static_cast<int>(d->k_tokens);
    p.scale2 = static_cast<float>(static_cast<double>(d->scale) * 1.4426950408889634);
    p.q_stride = d->q_stride;
    p.q_head_stride = d->q_head_stride;
    p.k_stride = d->k_stride;
    p.k_head_stride = d->k_head_stride;
    p.v_stride = d->v_stride;
    p.v_head_stride = d->v_head_stride;
    p.per_group = mx::divisor(p.group);
    const dim3 grid(static_cast<unsigned>(plan.tiles * p.kv_heads), plan.splits);
    auto go = [&](auto kernel) { kernel<<<grid, 256, 0, st>>>(p); };
    if (p.dim <= 64) {
        if (plan.rb == 1) go(fa::kernel<64, 4, 2, 1, 3, 2>);
        else go(fa::kernel<64, 4, 2, 2, 4, 1>);
    } else if (p.dim <= 96) {
        if (plan.rb == 1) go(fa::kernel<128, 6, 3, 1, 2, 2>);
        else go(fa::kernel<128, 6, 3, 2, 4, 1>);
    } else if (p.dim <= 128) {
        if (plan.rb == 1) go(fa::kernel<128, 8, 4, 1, 2, 2>);
        else go(fa::kernel<128, 8, 4, 2, 4, 1>);
    } else {
        go(fa::kernel<256, 16, 8, 1, 2, 1>);
    }
    const cfwd_status e = check_hip(hipGetLastError(), "attention launch");
    if (e != CFWD_OK || plan.splits == 1) return e;
    const long long units = d->q_tokens * d->q_heads * (d->head_dim / 4);  // split only where rows are few
    fa::join_kernel<<<static_cast<unsigned>((units + 255) / 256), 256, 0, st>>>(p, mx::divisor(d->head_dim / 4),
                                                                             static_cast<uint32_t>(units));
    return check_hip(hipGetLastError(), "attention's joining launch");
}

}  // namespace cfwd

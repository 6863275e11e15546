// Attention of a sequence's newest tokens over its paged MXFP4 cache (gfx950).
//
//   o = softmax(scale * q K^T) V,  K and V in blocks of 32 values with a scale
//
// Rows are the queries that share a head of the cache, (token, query head) of
// a group; 16 of them are one side of the matrix instruction, so that a head's
// cache is read once for all.  S^T = K q^T has a query in each lane's column and
// four keys in its registers, which is how P^T enters O^T = V^T P^T: nothing
// moves between lanes.  With m the running maximum and l the running sum,
// O and l are multiplied by 2^(m - m') only where a score passes m by more than
// 2^8: until then weights up to 2^8 are as good.  A row goes by its own scores
// alone, so that its result does not depend on the others'.
//
// One wave works on 32 tokens at a time.  The codes go from memory to registers:
// of K, a lane holds whole runs of one token's values; of V, the same columns of
// eight tokens, which after conversion (exact: a code has two significant bits)
// are paired token by token.
//
// Work is split by the lengths, which only the device knows: a unit is 128
// tokens of one sequence and head, every workgroup counts all units and takes an
// equal run of them, which may end within one head and begin within another.  What
// covers a head only in part leaves its sum, m and l in the workspace, and a
// second launch joins these in the order of the tokens.
#include "attention.h"
#include "mx.h"

#include <algorithm>

namespace cfwd {
namespace decode {

using namespace mx;

constexpr int kUnit = 128;      // tokens: a step of 32 for each of a workgroup's four waves
constexpr float kLow = -3.0e38f;  // m before any score: finite, so that differences are numbers
constexpr float kMost = 4096.0f;  // a lane's 8 weights sum up to this before m follows the scores

struct Params {
    const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
    const int32_t *table, *lengths;
    const bf16_t* q;
    bf16_t* o;
    float *part, *part_ml;  // [slot][row][dim], [slot][row][m, l]
    int sequences, tokens, heads, kv_heads, group, dim;
    int pages, page_size, table_pitch;
    int blocks, scale_pitch;  // of a row: code blocks, bytes of scales
    int rows, row_blocks, row_block;  // queries of a cache's head, in blocks of row_block
    int workgroups;
    float scale2;  // scale * log2(e)
    long long q_seq_stride, q_stride, q_head_stride;
    Divisor page, per_group;
};

__device__ __forceinline__ int length_of(const Params& p, int seq) {
    const long long most = static_cast<long long>(p.table_pitch) * p.page_size;
    return static_cast<int>(min(static_cast<long long>(max(p.lengths[seq], 0)), most));
}
__device__ __forceinline__ int units_of(int length) { return max(1, (length + kUnit - 1) / kUnit); }

// Units of one head, over all sequences: of those up to and with this lane's of the 64 from s on.
__device__ __forceinline__ int units_upto(const Params& p, int s, int lane, int* mine) {
    *mine = s + lane < p.sequences ? units_of(length_of(p, s + lane)) : 0;
    int v = *mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// The units of all pairs (head, block of rows) of all sequences, shared out: workgroup w takes `most` or one less of them,
// from start(w) on.
struct Shares {
    int units, workgroups, most, longer;  // the first `longer` workgroups take `most`
    __device__ __forceinline__ int start(int w) const { return w * (most - 1) + min(w, longer); }
    __device__ __forceinline__ int owner(int u) const {
        return u < longer * most ? u / most : longer + (u - longer * most) / (most - 1);
    }
};

__device__ __forceinline__ Shares shares_of(const Params& p, int units_of_a_head) {
    Shares r;
    r.units = units_of_a_head * p.kv_heads * p.row_blocks;
    r.workgroups = min(p.workgroups, r.units);
    r.most = r.units / r.workgroups + 1;
    r.longer = r.units - r.workgroups * (r.most - 1);
    return r;
}

__device__ __forceinline__ f32x4 mma(const u32x4_t& a, const u32x4_t& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Two values of a block as bf16.  The scale counts with its exponent alone: the byte where a float has it, 0 meaning 2^-127
// and 255 NaN.
template <int SEL>
__device__ __forceinline__ uint32_t two(uint32_t codes, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, SEL));
}

// Codes and scales of 32 tokens as a lane (n = lane % 16, g = lane / 16) needs them.
template <int DP>
struct Step {
    static constexpr int W = DP / 32;  // words of a token's K for each lane
    static constexpr int VW = DP >= 128 ? DP / 128 : 1;  // words of V's columns
    static constexpr int SW = DP == 256 ? 2 : 1;         // words of a token's scales
    uint32_t k[2][W], ks[2][SW];
    uint32_t v[8][VW], vs[8][SW];
    bool there[2];  // the tile's page is one of the cache's
};

// A lane's places in a tile of 16 tokens, in bytes.  Lanes past the row's values read its last block, which meets zeros of
// q (K) or is not stored (V).
template <int DP>
struct Places {
    uint32_t k[DP == 256 ? 2 : 1], ks[DP == 256 ? 2 : 1], v[4], vs;
    uint32_t turn[DP == 256 ? 2 : 1];  // of a token's word of scales, to bring the byte of the lane's columns to a float's exponent
    bool second;  // the byte is in the second word
};

template <int DP>
__device__ __forceinline__ Places<DP> places(const Params& p, int lane) {
    Places<DP> r;
    const int n = lane & 15, g = lane >> 4, pitch = p.blocks * 16;
    if constexpr (DP == 64) {
        const int b = min(g >> 1, p.blocks - 1);
        r.k[0] = n * pitch + b * 16 + (g & 1) * 8;
        r.ks[0] = n * p.scale_pitch + b;
    } else {
#pragma unroll
        for (int i = 0; i < DP / 128; ++i) {
            const int b = min(g * (DP / 128) + i, p.blocks - 1);
            r.k[i] = n * pitch + b * 16;
            r.ks[i] = n * p.scale_pitch + b;
        }
    }
    constexpr int E = DP / 16;  // values of a lane's columns
    const int b = min(n * E / 32, p.blocks - 1);
#pragma unroll
    for (int j = 0; j < 4; ++j) r.v[j] = (4 * g + j) * pitch + b * 16 + n * E / 2 - n * E / 32 * 16;
    r.vs = 4 * g * p.scale_pitch;
    r.turn[0] = (b % 4) * 8 + 9;
    r.second = b >= 4;
    return r;
}

// Page of the tile of 16 tokens from t on, or -1.  All in scalar registers.
__device__ __forceinline__ int page_of(const Params& p, int seq, int t, int length, int* offset) {
    *offset = 0;
    if (t >= length) return -1;
    const int page = divide(t, p.page);
    *offset = t - page * p.page_size;
    typedef const __attribute__((address_space(4))) int32_t* scalar;  // read only: a scalar load
    const int id = ((scalar)(p.table + static_cast<long long>(seq) * p.table_pitch))[page];
    return id < p.pages ? id : -1;
}

template <int DP>
__device__ __forceinline__ void load_step(const Params& p, const Places<DP>& at, int seq, int head, int length, int token, Step<DP>& s) {
#pragma unroll
    for (int a = 0; a < 2; ++a) {
        int offset;
        const int id = page_of(p, seq, token + 16 * a, length, &offset);
        s.there[a] = id >= 0;
        const long long row = (static_cast<long long>(max(id, 0)) * p.kv_heads + head) * p.page_size + offset;
        const uint8_t *kc = p.k_codes + row * (p.blocks * 16), *ks = p.k_scales + row * p.scale_pitch;
        const uint8_t *vc = p.v_codes + row * (p.blocks * 16), *vs = p.v_scales + row * p.scale_pitch;
        if constexpr (DP == 64) {
            const uint2 w = *reinterpret_cast<const uint2*>(kc + at.k[0]);
            s.k[a][0] = w.x;
            s.k[a][1] = w.y;
            s.ks[a][0] = ks[at.ks[0]];
        } else {
#pragma unroll
            for (int i = 0; i < DP / 128; ++i) {
                const uint4 w = *reinterpret_cast<const uint4*>(kc + at.k[i]);
                s.k[a][4 * i] = w.x;
                s.k[a][4 * i + 1] = w.y;
                s.k[a][4 * i + 2] = w.z;
                s.k[a][4 * i + 3] = w.w;
                s.ks[a][i] = ks[at.ks[i]];
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint8_t* c = vc + at.v[j];
            if constexpr (DP == 64) s.v[4 * a + j][0] = *reinterpret_cast<const uint16_t*>(c);
            if constexpr (DP == 128) s.v[4 * a + j][0] = *reinterpret_cast<const uint32_t*>(c);
            if constexpr (DP == 256) {
                const uint2 w = *reinterpret_cast<const uint2*>(c);
                s.v[4 * a + j][0] = w.x;
                s.v[4 * a + j][1] = w.y;
            }
        }
        // four tokens' words of scales lie side by side, of which a lane uses one byte each
        if constexpr (DP == 256) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t* w = reinterpret_cast<const uint32_t*>(vs + at.vs + j * p.scale_pitch);
                s.vs[4 * a + j][0] = w[0];
                s.vs[4 * a + j][1] = w[1];
            }
        } else {
            struct __attribute__((aligned(4))) Four {
                uint32_t w[4];
            };
            const Four w = *reinterpret_cast<const Four*>(vs + at.vs);
#pragma unroll
            for (int j = 0; j < 4; ++j) s.vs[4 * a + j][0] = w.w[j];
        }
    }
}

// A wave's state of RT * 16 queries: lane (n, g) holds, of query n, O at d = E (4 g + r) + i as o[][i][r].
template <int DP, int RT>
struct State {
    static constexpr int E = DP / 16;
    f32x4 o[RT][E];
    float m[RT], l[RT];
};

template <int DP, int RT>
__device__ __forceinline__ void attend(const Params& p, const Places<DP>& at, const Step<DP>& s, int seq, int head, int token,
                                       int length, const int (&seen)[RT], int least, const u32x4_t (&q)[RT][DP / 32],
                                       int lane, State<DP, RT>& st) {
    constexpr int E = DP / 16, W = DP / 32;
    const int g = lane >> 4;
    f32x4 score[RT][2];
#pragma unroll
    for (int a = 0; a < 2; ++a) {
#pragma unroll
        for (int r = 0; r < RT; ++r) score[r][a] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < W; ++c) {
            const float unit = __uint_as_float(s.ks[a][c / 4] << 23);
            const uint32_t w = s.k[a][c];
            const u32x4_t f = {two<0>(w, unit), two<1>(w, unit), two<2>(w, unit), two<3>(w, unit)};
#pragma unroll
            for (int r = 0; r < RT; ++r) score[r][a] = mma(f, q[r][c], score[r][a]);
        }
    }
    uint32_t v[8][Step<DP>::VW];
    float unit[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t w = DP == 256 && at.second ? s.vs[j][Step<DP>::SW - 1] : s.vs[j][0];
        unit[j] = __uint_as_float(__builtin_amdgcn_alignbit(w, w, at.turn[0]) & 0x7f800000u);
#pragma unroll
        for (int w = 0; w < Step<DP>::VW; ++w) v[j][w] = s.v[j][w];
    }
    bool odd = false;  // a value that is NaN, of a token that not all queries may see
    const bool masked = token + 32 > least || !s.there[0] || !s.there[1];
    if (masked) {
        asm volatile("");  // a branch around this stays one
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = token + 16 * a + 4 * g + j;
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    if (!s.there[a] || t >= seen[r]) score[r][a][j] = -__builtin_inff();
                // weights of 0 do not undo a NaN: it is taken out, and put back below where it is seen
                const bool absent = !s.there[a] || t >= length, nan = unit[4 * a + j] == __builtin_inff();
                odd |= !absent && nan;
                if (absent || nan) {
                    unit[4 * a + j] = 1.0f;
#pragma unroll
                    for (int w = 0; w < Step<DP>::VW; ++w) v[4 * a + j][w] = 0;
                }
            }
    }
    u32x4_t weight[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        float sum = 0.0f;
        auto weigh = [&]() __attribute__((always_inline)) {
            sum = 0.0f;
            float e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(score[r][i / 4][i % 4], p.scale2, -st.m[r]));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                weight[r][i] = pack_bf16x2(e[2 * i], e[2 * i + 1]);
                // the sum takes the weights as they enter the product: rounded
                sum = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, static_cast<uint32_t>(weight[r][i])),
                                                      __builtin_bit_cast(bf16x2_t, 0x3f803f80u), sum, false);
            }
        };
        weigh();
        if (__any(!(sum <= kMost))) {
            // scores far above m (or the first ones, or NaN): m moves up to the query's largest, and the weights are taken again
            float top = score[r][0][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) top = fmaxf(top, score[r][i / 4][i % 4]);
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32)) * p.scale2;
            int over = !(sum <= kMost);
            over |= __shfl_xor(over, 16);
            over |= __shfl_xor(over, 32);
            const float m = over && top > st.m[r] ? top : st.m[r], f = __builtin_amdgcn_exp2f(st.m[r] - m);
            st.m[r] = m;
            st.l[r] *= f;
#pragma unroll
            for (int i = 0; i < E; ++i) st.o[r][i] *= f;
            weigh();
        }
        st.l[r] += sum;
    }
#pragma unroll
    for (int b = 0; b < E / 2; ++b) {  // byte b of the columns: values 2 b and 2 b + 1
        uint32_t x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t w = v[j][b / 4];
            x[j] = b % 4 == 0   ? two<0>(w, unit[j])
                   : b % 4 == 1 ? two<1>(w, unit[j])
                   : b % 4 == 2 ? two<2>(w, unit[j])
                                : two<3>(w, unit[j]);
        }
        u32x4_t even, uneven;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            even[j] = __builtin_amdgcn_perm(x[2 * j + 1], x[2 * j], 0x05040100u);
            uneven[j] = __builtin_amdgcn_perm(x[2 * j + 1], x[2 * j], 0x07060302u);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            st.o[r][2 * b] = mma(even, weight[r], st.o[r][2 * b]);
            st.o[r][2 * b + 1] = mma(uneven, weight[r], st.o[r][2 * b + 1]);
        }
    }
    if (masked && __any(odd)) {
        // rare: the scales again, token by token, for the columns that this lane's outputs are of
        for (int t = token; t < min(token + 32, length); ++t) {
            const int page = divide(t, p.page), id = p.table[static_cast<long long>(seq) * p.table_pitch + page];
            if (id < 0 || id >= p.pages) continue;
            const uint8_t* sc = p.v_scales + ((static_cast<long long>(id) * p.kv_heads + head) * p.page_size + t -
                                              page * p.page_size) * p.scale_pitch;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int d = E * (4 * g + i);
                if (d / 32 >= p.blocks || sc[d / 32] != 255) continue;
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    if (t < seen[r])
#pragma unroll
                        for (int e = 0; e < E; ++e) st.o[r][e][i] = __builtin_nanf("");
            }
        }
    }
}

// Fewer registers than the widest forms need would spill them.
template <int DP, int RT>
__global__ __launch_bounds__(256, DP * RT <= 128 ? 3 : DP * RT <= 256 ? 2 : 1) void kernel(Params p) {
    constexpr int E = DP / 16, W = DP / 32;
    __shared__ f32x4 area[2][RT * E][64];
    __shared__ float area_m[4][RT * 16], area_l[4][RT * 16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int pairs = p.kv_heads * p.row_blocks;  // of a sequence: (head, block of rows)
    // the units of all sequences, then the sequence in which the first unit of this workgroup lies
    int mine, upto = units_upto(p, 0, lane, &mine), total = __shfl(upto, 63);
    for (int s = 64; s < p.sequences; s += 64) total += __shfl(units_upto(p, s, lane, &mine), 63);
    const Shares shares = shares_of(p, __builtin_amdgcn_readfirstlane(total));
    if (static_cast<int>(blockIdx.x) >= shares.workgroups) return;
    int u = shares.start(blockIdx.x);
    const int end = shares.start(blockIdx.x + 1);
    int seq = 0, before = 0;
    {
        const int x = u / pairs;
        if (p.sequences > 64) upto = units_upto(p, 0, lane, &mine);
        for (int s = 0; s < p.sequences; s += 64) {
            const unsigned long long past = __ballot(before + upto > x);
            if (past) {
                const int at = __ffsll(past) - 1;
                seq = s + at;
                before += __shfl(upto - mine, at);
                break;
            }
            before += __shfl(upto, 63);
            upto = units_upto(p, s + 64, lane, &mine);
        }
    }
    seq = __builtin_amdgcn_readfirstlane(seq);
    int length = __builtin_amdgcn_readfirstlane(length_of(p, seq));
    const int in_seq = __builtin_amdgcn_readfirstlane(u - before * pairs);
    int pair = min(__builtin_amdgcn_readfirstlane(in_seq / units_of(length)), pairs - 1);
    int first = __builtin_amdgcn_readfirstlane(in_seq - pair * units_of(length));
    const Places<DP> at = places<DP>(p, lane);
    int slot = 2 * blockIdx.x;
    while (u < end) {
        const int all = units_of(length);
        const int count = __builtin_amdgcn_readfirstlane(min(all - first, end - u));
        const int head = pair / p.row_blocks, row0 = (pair - head * p.row_blocks) * p.row_block;
        const int stop = min((first + count) * kUnit, length);
        State<DP, RT> st;
        u32x4_t q[RT][W];
        int seen[RT];
        const int least = length - p.tokens + 1;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int row = row0 + r * 16 + n;
            const int token = divide(min(row, p.rows - 1), p.per_group), h = head * p.group + min(row, p.rows - 1) - token * p.group;
            seen[r] = least + token;
            const bf16_t* x = p.q + seq * p.q_seq_stride + token * p.q_stride + h * p.q_head_stride;
#pragma unroll
            for (int c = 0; c < W; ++c) {
                const int d = 8 * W * g + 8 * c;
                q[r][c] = d < p.dim ? *reinterpret_cast<const u32x4_t*>(x + d) : u32x4_t{0, 0, 0, 0};
            }
            st.m[r] = kLow;
            st.l[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < E; ++i) st.o[r][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        {
            // two steps' codes in turn: while one is used, the other is on its way
            Step<DP> even, uneven;
            int token = first * kUnit + wave * 32;
            load_step<DP>(p, at, seq, head, token < stop ? length : 0, token, even);
            load_step<DP>(p, at, seq, head, token + kUnit < stop ? length : 0, token + kUnit, uneven);
            for (; token < stop; token += 2 * kUnit) {
                attend<DP, RT>(p, at, even, seq, head, token, length, seen, least, q, lane, st);
                load_step<DP>(p, at, seq, head, token + 2 * kUnit < stop ? length : 0, token + 2 * kUnit, even);
                if (token + kUnit >= stop) break;
                attend<DP, RT>(p, at, uneven, seq, head, token + kUnit, length, seen, least, q, lane, st);
                load_step<DP>(p, at, seq, head, token + 3 * kUnit < stop ? length : 0, token + 3 * kUnit, uneven);
            }
        }
        // join the four waves: m first, then the sums, 2 and 3 into 0 and 1, 1 into 0
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            st.l[r] += __shfl_xor(st.l[r], 16);
            st.l[r] += __shfl_xor(st.l[r], 32);
            if (g == 0) {
                area_m[wave][r * 16 + n] = st.m[r];
                area_l[wave][r * 16 + n] = st.l[r];
            }
        }
        __syncthreads();
        float l[RT], m[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            m[r] = kLow;
#pragma unroll
            for (int w = 0; w < 4; ++w) m[r] = fmaxf(m[r], area_m[w][r * 16 + n]);
            l[r] = 0.0f;
#pragma unroll
            for (int w = 0; w < 4; ++w)
                l[r] += area_l[w][r * 16 + n] * __builtin_amdgcn_exp2f(area_m[w][r * 16 + n] - m[r]);
            const float f = __builtin_amdgcn_exp2f(st.m[r] - m[r]);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                st.o[r][i] *= f;
                if (wave >= 2) area[wave - 2][r * E + i][lane] = st.o[r][i];
            }
        }
        __syncthreads();
        if (wave < 2) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    st.o[r][i] += area[wave][r * E + i][lane];
                    if (wave == 1) area[1][r * E + i][lane] = st.o[r][i];
                }
        }
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const int row = row0 + r * 16 + n;
#pragma unroll
                for (int i = 0; i < E; ++i) st.o[r][i] += area[1][r * E + i][lane];
                if (row >= p.rows) continue;
                if (count == all) {
                    const float inverse = l[r] == 0.0f ? 0.0f : 1.0f / l[r];
                    const int token_of = divide(row, p.per_group), h = head * p.group + row - token_of * p.group;
                    bf16_t* y = p.o + ((static_cast<long long>(seq) * p.tokens + token_of) * p.heads + h) * p.dim;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int d = E * (4 * g + j);
                        if (d >= p.dim) continue;
#pragma unroll
                        for (int i = 0; i < E; i += 2)
                            *reinterpret_cast<uint32_t*>(y + d + i) =
                                pack_bf16x2(st.o[r][i][j] * inverse, st.o[r][i + 1][j] * inverse);
                    }
                } else {
                    const long long to = static_cast<long long>(slot) * p.row_block + r * 16 + n;
                    if (g == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * to) = make_float2(m[r], l[r]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int d = E * (4 * g + j);
                        if (d >= p.dim) continue;
#pragma unroll
                        for (int i = 0; i < E; i += 4)
                            *reinterpret_cast<f32x4*>(p.part + to * p.dim + d + i) =
                                f32x4{st.o[r][i][j], st.o[r][i + 1][j], st.o[r][i + 2][j], st.o[r][i + 3][j]};
                    }
                }
            }
        }
        __syncthreads();
        slot = 2 * blockIdx.x + 1;
        u += count;
        first = 0;
        if (++pair == pairs && u < end) {
            pair = 0;
            seq = min(seq + 1, p.sequences - 1);
            length = __builtin_amdgcn_readfirstlane(length_of(p, seq));
        }
    }
}

// Joins the parts of one query: grid (sequence and pair, row of its block), 256 threads.
__global__ __launch_bounds__(256) void join_kernel(Params p) {
    __shared__ f32x4 area[256];
    __shared__ float area_m[4], area_l[256];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int pairs = p.kv_heads * p.row_blocks, seq = blockIdx.x / pairs, pair = blockIdx.x - seq * pairs;
    const int head = pair / p.row_blocks, in_block = blockIdx.y, row = (pair - head * p.row_blocks) * p.row_block + in_block;
    if (row >= p.rows) return;
    const int mine = units_of(length_of(p, seq));
    if (mine == 1) return;
    int n = 0, before = 0;
    for (int s = lane; s < p.sequences; s += 64) {
        const int c = units_of(length_of(p, s));
        n += c;
        before += s < seq ? c : 0;
    }
#pragma unroll
    for (int d = 32; d; d /= 2) {
        n += __shfl_xor(n, d);
        before += __shfl_xor(before, d);
    }
    const Shares shares = shares_of(p, n);
    const int u0 = before * pairs + pair * mine, w0 = shares.owner(u0), w1 = shares.owner(u0 + mine - 1);
    if (w0 == w1) return;
    auto place = [&](int w) {
        const int slot = 2 * w + (shares.start(w) >= u0 ? 0 : 1);
        return static_cast<long long>(slot) * p.row_block + in_block;
    };
    float m = kLow;
    for (int w = w0 + threadIdx.x; w <= w1; w += 256) m = fmaxf(m, p.part_ml[2 * place(w)]);
#pragma unroll
    for (int d = 32; d; d /= 2) m = fmaxf(m, __shfl_xor(m, d));
    if (lane == 0) area_m[wave] = m;
    __syncthreads();
    m = fmaxf(fmaxf(area_m[0], area_m[1]), fmaxf(area_m[2], area_m[3]));
    const int across = p.dim / 4, strands = 256 / across;  // threads of a row, rows at a time
    const int strand = threadIdx.x / across, d = (threadIdx.x - strand * across) * 4;
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    float l = 0.0f;
    if (strand < strands) {
#pragma unroll 4
        for (int w = w0 + strand; w <= w1; w += strands) {
            const long long at = place(w);
            const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * at);
            const float f = __builtin_amdgcn_exp2f(ml.x - m);
            l += ml.y * f;
            sum += *reinterpret_cast<const f32x4*>(p.part + at * p.dim + d) * f;
        }
    }
    area[threadIdx.x] = sum;
    area_l[threadIdx.x] = l;
    __syncthreads();
    if (strand != 0) return;
    for (int s = 1; s < strands; ++s) {
        sum += area[s * across + threadIdx.x];
        l += area_l[s * across + threadIdx.x];
    }
    const float inverse = l == 0.0f ? 0.0f : 1.0f / l;
    const int token = divide(row, p.per_group), h = head * p.group + row - token * p.group;
    uint2 y;
    y.x = pack_bf16x2(sum[0] * inverse, sum[1] * inverse);
    y.y = pack_bf16x2(sum[2] * inverse, sum[3] * inverse);
    *reinterpret_cast<uint2*>(p.o + ((static_cast<long long>(seq) * p.tokens + token) * p.heads + h) * p.dim + d) = y;
}

struct Plan {
    int dp, rt, row_blocks, workgroups;
    bool join;
    size_t part_bytes, bytes;
};

Plan plan(const cfwd_mx_cache_attention_desc* d, const cfwd_mx_cache* c) {
    Plan r{};
    const int rows = d->tokens * (d->q_heads / c->kv_heads);
    r.dp = c->head_dim <= 64 ? 64 : c->head_dim <= 128 ? 128 : 256;
    r.rt = rows <= 16 ? 1 : rows <= 32 || r.dp == 256 ? 2 : 4;
    r.row_blocks = (rows + r.rt * 16 - 1) / (r.rt * 16);
    const long long longest = static_cast<long long>(d->table_pitch) * c->page_size;
    const long long most = std::max(1ll, (longest + kUnit - 1) / kUnit);
    const long long units = most * d->sequences * c->kv_heads * r.row_blocks;
    const int resident = r.dp * r.rt <= 128 ? 3 : r.dp * r.rt <= 256 ? 2 : 1;
    r.workgroups = static_cast<int>(std::min<long long>(units, static_cast<long long>(compute_units()) * resident));
    r.join = most > 1;
    if (r.join) {
        const size_t slots = 2 * static_cast<size_t>(r.workgroups) * r.rt * 16;
        r.part_bytes = slots * c->head_dim * 4;
        r.bytes = r.part_bytes + slots * 8;
    }
    return r;
}

}  // namespace decode

size_t mx_cache_attention_workspace(const cfwd_mx_cache_attention_desc* d, const cfwd_mx_cache* c) {
    return decode::plan(d, c).bytes;
}

cfwd_status mx_cache_attention(const cfwd_mx_cache_attention_desc* d, const cfwd_mx_cache* c, const void* q,
                               const int32_t* table, const int32_t* lengths, void* o, void* workspace, hipStream_t st) {
    const decode::Plan plan = decode::plan(d, c);
    decode::Params p{};
    p.k_codes = static_cast<const uint8_t*>(c->k_codes);
    p.k_scales = static_cast<const uint8_t*>(c->k_scales);
    p.v_codes = static_cast<const uint8_t*>(c->v_codes);
    p.v_scales = static_cast<const uint8_t*>(c->v_scales);
    p.table = table;
    p.lengths = lengths;
    p.q = static_cast<const bf16_t*>(q);
    p.o = static_cast<bf16_t*>(o);
    p.part = static_cast<float*>(workspace);
    p.part_ml = plan.join ? reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.part_bytes) : nullptr;
    p.sequences = d->sequences;
    p.tokens = d->tokens;
    p.heads = d->q_heads;
    p.kv_heads = c->kv_heads;
    p.group = d->q_heads / c->kv_heads;
    p.dim = c->head_dim;
    p.pages = c->pages;
    p.page_size = c->page_size;
    p.table_pitch = d->table_pitch;
    p.blocks = static_cast<int>(mx_blocks(c->head_dim));
    p.scale_pitch = static_cast<int>(mx_scale_pitch(c->head_dim));
    p.rows = d->tokens * p.group;
    p.row_blocks = plan.row_blocks;
    p.row_block = plan.rt * 16;
    p.workgroups = plan.workgroups;
    p.scale2 = static_cast<float>(static_cast<double>(d->scale) * 1.4426950408889634);
    p.q_seq_stride = d->q_seq_stride;
    p.q_stride = d->q_stride;
    p.q_head_stride = d->q_head_stride;
    p.page = mx::divisor(c->page_size);
    p.per_group = mx::divisor(p.group);
    auto go = [&](auto kernel) { kernel<<<plan.workgroups, 256, 0, st>>>(p); };
    if (plan.dp == 64) {
        if (plan.rt == 1) go(decode::kernel<64, 1>);
        else if (plan.rt == 2) go(decode::kernel<64, 2>);
        else go(decode::kernel<64, 4>);
    } else if (plan.dp == 128) {
        if (plan.rt == 1) go(decode::kernel<128, 1>);
        else if (plan.rt == 2) go(decode::kernel<128, 2>);
        else go(decode::kernel<128, 4>);
    } else {
        if (plan.rt == 1) go(decode::kernel<256, 1>);
        else go(decode::kernel<256, 2>);
    }
    cfwd_status e = check_hip(hipGetLastError(), "cache attention launch");
    if (e != CFWD_OK || !plan.join) return e;
    decode::join_kernel<<<dim3(p.sequences * p.kv_heads * p.row_blocks, std::min(p.rows, p.row_block)), 256, 0, st>>>(p);
    return check_hip(hipGetLastError(), "cache attention's joining launch");
}

}  // namespace cfwd

// Attention of a sequence's newest tokens over its paged MXFP4 cache (gfx950).
//
//   o = softmax(scale * q K^T) V,  K and V in blocks of 32 values with a scale
//
// Rows are the queries that share a head of the cache, (token, query head) of
// a group; 16 of them are one side of the matrix instruction, so that a head's
// cache is read once for all.  S^T = K q^T has a query in each lane's column and
// four keys in its registers, which is how P^T enters O^T = V^T P^T: nothing
// moves between lanes.
//
// K goes into the matrix cores as it lies in the cache, codes and scale bytes; the
// queries beside it are two parts of 8 bits (Queries).  V's scales belong to
// tokens, over which the second product sums, so its codes become bf16 (exact: a
// code has two significant bits) and are paired token by token.
//
// Softmax.  Weights are 2^(s - m) with s in units of log2 and m no running maximum
// but any number that the scores have not passed by far: it moves only where a
// lane's 8 weights sum up to more than 2^12, then to the query's largest score, and
// O and l are multiplied by 2^(m - m').  Weights have bf16's 8 bits at any size, so
// nothing is lost.  A row goes by its own scores alone.
//
// One wave works on 32 tokens at a time, out of registers, while the codes of the
// next two such steps are on their way to its own part of LDS, by copies that
// bypass the registers: with the codes on their way to registers instead, only three
// workgroups fit a CU instead of four.
//
// Work is split by the lengths, which only the device knows: a unit is 128
// tokens of one sequence and head, or several times that, every workgroup counts all units and takes an
// equal run of them, which may end within one head and begin within another.  What
// covers a head only in part leaves its sum, m and l in the workspace, and a
// second launch joins these in the order of the tokens.  Where the page table has room for few tokens only,
// a workgroup takes a head as a whole, and one launch is all.
//
// Bound by memory: 64 sequences of up to 8192 tokens, 32 heads over 8 of 128, 296 MB in 62 us and 7 for the join (4.8 and 4.3
// TB/s; the loads alone 61.5); with 32 rows a head by vector instructions: 4 tokens over 131072, 64 heads over 8, 40 + 6 us.
#include "attention.h"
#include "mx.h"

#include <algorithm>
#include <type_traits>

namespace cfwd {
namespace decode {

using namespace mx;

constexpr int kRound = 128;  // tokens: a step of 32 for each of a workgroup's four waves
constexpr int kStart = 3;
constexpr int kLargest = 32;  // rounds of a unit
constexpr float kLow = -3.0e38f;  // m before any score: finite, so that differences are numbers
constexpr float kMost = 4096.0f;  // a lane's 8 weights sum up to this before m follows the scores

// Workgroups on a CU: what registers (and LDS) allow without spilling (but five of 64 x 64), for heads of dp values and rt * 16
// queries at once.
constexpr int resident(int dp, int rt) { return dp * rt > 256 ? 1 : dp * rt > 128 ? 2 : rt == 1 ? 4 : 3; }

struct Params {
    const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
    const int32_t *table, *lengths;
    const bf16_t* q;
    bf16_t* o;
    float *part, *part_ml;  // [slot][row][dim], [slot][row][m, l]
    int sequences, tokens, heads, kv_heads, group, dim;
    int pages, page_size, table_pitch;
    int blocks, scale_pitch;  // of a row: code blocks, bytes of scales
    uint32_t page_codes, page_scales;  // bytes of a page
    int rows, row_blocks, row_block;  // queries of a cache's head, in blocks of row_block
    int workgroups, whole, few;
    float scale2;  // scale * log2(e)
    long long q_seq_stride, q_stride, q_head_stride;
    Divisor page, per_group;
};

__device__ __forceinline__ int length_of(const Params& p, int seq) {
    const long long most = static_cast<long long>(p.table_pitch) * p.page_size;
    return static_cast<int>(min(static_cast<long long>(max(p.lengths[seq], 0)), most));
}
__device__ __forceinline__ int rounds_of(int length) { return max(1, (length + kRound - 1) / kRound); }

// Rounds of one head in the sequence of this lane, of the 64 from s on, and its length.
__device__ __forceinline__ int rounds_at(const Params& p, int s, int lane, int* length) {
    *length = length_of(p, min(s + lane, p.sequences - 1));
    return s + lane < p.sequences ? rounds_of(*length) : 0;
}

// Rounds of a unit, from those of one head in all sequences.  Where units of many rounds still give a part of the device's
// workgroups one each, there are fewer parts to begin and to join; where there is more to do, equal runs of the
// smallest units balance the workgroups (heads of 128, 8 of the cache; us: 1 sequence of 16000 tokens 18 by single rounds, 14 by 4,
// 8 of up to 8000 tokens 24 and 20 by 8; 64 of up to 8192 69 and 72 by 32).
__device__ __forceinline__ int unit_of(const Params& p, int rounds) {
    const long long all = static_cast<long long>(rounds) * (p.kv_heads * p.row_blocks);
    return all <= static_cast<long long>(p.few) * kLargest ? static_cast<int>((all + p.few - 1) / p.few) : 1;
}

// The units of all pairs (head, block of rows) of all sequences, shared out: workgroup w takes `most` or one less of them,
// from begin(w) on.  To begin a pair and to write its sums takes as long as several units of its tokens do, so where a
// workgroup has many, a pair counts as `start` units more, ahead of its own (64 sequences of up to 8192 tokens: the last workgroup ends after 68 us without, 54 with 3).
struct Shares {
    int units, workgroups, most, longer, start;  // the first `longer` workgroups take `most`
    __device__ __forceinline__ int begin(int w) const { return w * (most - 1) + min(w, longer); }
    __device__ __forceinline__ int owner(int u) const {
        return u < longer * most ? u / most : longer + (u - longer * most) / (most - 1);
    }
};

__device__ __forceinline__ Shares shares_of(const Params& p, int units_of_a_head) {
    Shares r;
    const int pairs = p.kv_heads * p.row_blocks;
    r.start = units_of_a_head * pairs >= 4 * p.workgroups ? kStart : 0;
    r.units = (units_of_a_head + r.start * p.sequences) * pairs;
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
    static constexpr int KB = DP == 256 ? 2 : 1;         // blocks of a token's K for each lane: 4 i + g
    static constexpr int VW = DP >= 128 ? DP / 128 : 1;  // words of V's columns
    static constexpr int SW = DP == 256 ? 2 : 1;         // words of a token's scales
    u32x4_t k[2][KB];
    uint32_t ks[2][KB];
    uint32_t v[8][VW], vs[8][SW];
};

// A lane's places in a tile of 16 tokens, in bytes.  Lanes past the row's values read its last block, which meets zeros of
// q (K) or is not stored (V).
template <int DP>
struct Places {
    uint32_t k[Step<DP>::KB], ks[Step<DP>::KB], v[4], vs;
    uint32_t turn;  // of a token's word of scales, to bring the byte of the lane's columns to a float's exponent
    bool second;  // the byte is in the second word
};

// To another stage.  Opaque, so that the reads hold what their own places differ by.
template <int DP>
__device__ __forceinline__ void move(Places<DP>& r, uint32_t by) {
#pragma unroll
    for (int i = 0; i < Step<DP>::KB; ++i) asm volatile("" : "+v"(r.k[i] += by), "+v"(r.ks[i] += by));
#pragma unroll
    for (int j = 0; j < 4; ++j) asm volatile("" : "+v"(r.v[j] += by));
    asm volatile("" : "+v"(r.vs += by));
}

template <int DP>
__device__ __forceinline__ Places<DP> places(const Params& p, int lane, uint32_t lds) {
    Places<DP> r;
    const int n = lane & 15, g = lane >> 4, pitch = p.blocks * 16;
#pragma unroll
    for (int i = 0; i < Step<DP>::KB; ++i) {
        const int b = min(4 * i + g, p.blocks - 1);
        r.k[i] = n * pitch + b * 16;
        r.ks[i] = n * p.scale_pitch + b;
    }
    constexpr int E = DP / 16;  // values of a lane's columns
    const int b = min(n * E / 32, p.blocks - 1);
#pragma unroll
    for (int j = 0; j < 4; ++j) r.v[j] = (4 * g + j) * pitch + b * 16 + n * E / 2 - n * E / 32 * 16;
    r.vs = 4 * g * p.scale_pitch;
    r.turn = (b % 4) * 8 + 9;
    r.second = b >= 4;
    move(r, lds);
    return r;
}

// Where the two tiles of 16 tokens of a step lie, in bytes of codes and scales, and whether their pages are the cache's.  All in
// scalar registers.  ONE: pages are whole steps, so that the tiles lie one behind the other.
template <bool ONE>
struct Where {
    static constexpr int N = ONE ? 1 : 2;
    uint64_t codes[N], scales[N];
    bool there[N];
    __device__ __forceinline__ bool has(int a) const { return there[ONE ? 0 : a]; }
};

template <bool ONE>
__device__ __forceinline__ Where<ONE> where_is(const Params& p, const int32_t* pages_of, int head, int token, int length) {
    Where<ONE> r;
#pragma unroll
    for (int a = 0; a < Where<ONE>::N; ++a) {
        const int t = token + 16 * a;
        int row = head * p.page_size, id = -1;
        if (t < length) {
            const int page = divide(t, p.page);
            row += t - page * p.page_size;
            typedef const __attribute__((address_space(4))) int32_t* scalar;  // read only: a scalar load
            id = ((scalar)pages_of)[page];
        }
        r.there[a] = static_cast<uint32_t>(id) < static_cast<uint32_t>(p.pages);
        const uint32_t of = r.there[a] ? id : 0;
        r.codes[a] = static_cast<uint64_t>(of) * p.page_codes + static_cast<uint32_t>(row * p.blocks * 16);
        r.scales[a] = static_cast<uint64_t>(of) * p.page_scales + static_cast<uint32_t>(row * p.scale_pitch);
    }
    return r;
}

// A step in LDS: the tiles' codes of K, of V, their scales; each wave has kStages of them, and waits for nobody.
template <int DP>
constexpr int kTile = DP * 8;  // bytes of 16 tokens' codes
template <int DP>
constexpr int kScales = DP == 256 ? 128 : 64;
template <int DP>
constexpr int kStage = 4 * kTile<DP> + 4 * kScales<DP>;
constexpr int kStages = 2;
template <int DP, bool ONE>
constexpr int kCopies = 4 * (DP == 256 ? 2 : 1) + (ONE ? 2 : 4);  // memory instructions of a step

// Copies a lane's 16 (or 4) bytes from a buffer straight to LDS, lane after lane from `lds` on (the same for the wave).  The
// compiler does not see these loads: wait_loads() comes before the data are read.  It may have moved the buffer's words to
// scalar registers with vector instructions, which a load must not follow closer than five wait states.
__device__ __forceinline__ void load_to_lds16(const __amdgpu_buffer_rsrc_t& b, uint32_t off, uint32_t lds) {
    asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" : : "{m0}"(lds), "v"(off), "s"(b) : "memory");
}
__device__ __forceinline__ void load_to_lds4(const __amdgpu_buffer_rsrc_t& b, uint32_t off, uint32_t lds) {
    asm volatile("s_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds" : : "{m0}"(lds), "v"(off), "s"(b) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads() {  // until at most N of this wave's loads are outstanding
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// All waves of the workgroup, each with what it wrote to LDS there; stores to memory go on.
__device__ __forceinline__ void barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Bytes from a scalar address on; beyond them a copy writes zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const uint8_t* base, uint64_t at, int bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(base) + at;
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(static_cast<uint64_t>(hi) << 32 | lo), 0,
                                             __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}

template <int DP, bool ONE>
__device__ __forceinline__ void copy_step(const Params& p, const Where<ONE>& where, int lane, uint32_t to) {
    const int tile = p.blocks * 256, tile_scales = p.scale_pitch * 16;  // bytes
#pragma unroll
    for (int w = 0; w < Where<ONE>::N; ++w) {
        const auto kc = buffer(p.k_codes, where.codes[w], ONE ? 2 * tile : tile);
        const auto vc = buffer(p.v_codes, where.codes[w], ONE ? 2 * tile : tile);
#pragma unroll
        for (int a = w; a < (ONE ? 2 : w + 1); ++a)
#pragma unroll
            for (int i = 0; i < (DP == 256 ? 2 : 1); ++i)
                if (DP >= 128 || lane < 32) {  // what lies past the tile's rows is not read
                    const uint32_t off = (ONE ? a * tile : 0) + lane * 16 + i * 1024;
                    load_to_lds16(kc, off, to + a * kTile<DP> + i * 1024);
                    load_to_lds16(vc, off, to + (2 + a) * kTile<DP> + i * 1024);
                }
        const auto ks = buffer(p.k_scales, where.scales[w], ONE ? 2 * tile_scales : tile_scales);
        const auto vs = buffer(p.v_scales, where.scales[w], ONE ? 2 * tile_scales : tile_scales);
        if (lane < kScales<DP> / 4 * (ONE ? 2 : 1)) {
            load_to_lds4(ks, lane * 4, to + 4 * kTile<DP> + w * kScales<DP>);
            load_to_lds4(vs, lane * 4, to + 4 * kTile<DP> + (2 + w) * kScales<DP>);
        }
    }
}

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
template <typename T>
__device__ __forceinline__ T lds_at(uint32_t at) {
    return *reinterpret_cast<const __attribute__((address_space(3))) T*>(at);
}

// A lane's places are addresses in LDS, and the reads hold the rest.
template <int DP>
__device__ __forceinline__ void read_step(const Places<DP>& at, Step<DP>& s) {
#pragma unroll
    for (int a = 0; a < 2; ++a) {
        constexpr int SCALES = 4 * kTile<DP>;
        const int kc = a * kTile<DP>, vc = kc + 2 * kTile<DP>, ks = SCALES + a * kScales<DP>, vs = ks + 2 * kScales<DP>;
#pragma unroll
        for (int i = 0; i < Step<DP>::KB; ++i) {
            s.k[a][i] = lds_at<u32x4_t>(kc + at.k[i]);
            s.ks[a][i] = lds_at<uint8_t>(ks + at.ks[i]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (DP == 64) s.v[4 * a + j][0] = lds_at<uint16_t>(vc + at.v[j]);
            if constexpr (DP == 128) s.v[4 * a + j][0] = lds_at<uint32_t>(vc + at.v[j]);
            if constexpr (DP == 256) {
                const auto w = lds_at<u32x2_t>(vc + at.v[j]);
                s.v[4 * a + j][0] = w[0];
                s.v[4 * a + j][1] = w[1];
            }
        }
        // four tokens' words of scales lie side by side, of which a lane uses one byte each
#pragma unroll
        for (int i = 0; i < Step<DP>::SW; ++i) {
            const auto w = lds_at<u32x4_t>(vs + at.vs + 16 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) s.vs[4 * a + (4 * i + j) / Step<DP>::SW][j % Step<DP>::SW] = w[j];
        }
    }
}

// 16 queries as the matrix instruction takes them beside codes of 4 bits: in two parts of 8 bits (e4m3), hi + lo / 16, of
// values with a common scale that brings the largest, of a query's 128, into [2^7, 2^8).  A bf16 has eight significant bits and
// an e4m3 four, of which the second part needs as many as the rounding of the first leaves: the sum is exact for
// values down to 2^-13 of the largest, and within 2^-21 of the largest below.  Lane (n, g) holds values 16 g .. 16 g + 15 and
// 64 on of query n.
template <int DP>
struct Queries {
    static constexpr int KB = Step<DP>::KB;
    i32x8_t hi[KB], lo[KB];
    int scale[KB];
};

template <int DP>
__device__ __forceinline__ void load_queries(const Params& p, const bf16_t* x, int g, Queries<DP>& q) {
#pragma unroll
    for (int i = 0; i < Queries<DP>::KB; ++i) {
        float v[32];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
            const int d = 128 * i + 64 * (j / 16) + 16 * g + j % 16;
            const u32x4_t w = d < p.dim ? *reinterpret_cast<const u32x4_t*>(x + d) : u32x4_t{0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                v[j + 2 * c] = __uint_as_float(w[c] << 16);
                v[j + 2 * c + 1] = __uint_as_float(w[c] & 0xffff0000u);
                top = max(top, max(abs_bits(v[j + 2 * c]), abs_bits(v[j + 2 * c + 1])));
            }
        }
        top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 16)));
        top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32)));
        const int e = max(static_cast<int>(top >> 23), 11);
        q.scale[i] = e == 255 ? 255 : e - 7;  // NaN or infinite: all is NaN
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
            float r[4];
            int hi = 0, lo = 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) r[c] = __builtin_amdgcn_ldexpf(v[j + c], 134 - e);
            hi = __builtin_amdgcn_cvt_pk_fp8_f32(r[0], r[1], hi, false);
            hi = __builtin_amdgcn_cvt_pk_fp8_f32(r[2], r[3], hi, true);
            const auto h0 = __builtin_amdgcn_cvt_pk_f32_fp8(hi, false), h1 = __builtin_amdgcn_cvt_pk_f32_fp8(hi, true);
            lo = __builtin_amdgcn_cvt_pk_fp8_f32((r[0] - h0[0]) * 16.0f, (r[1] - h0[1]) * 16.0f, lo, false);
            lo = __builtin_amdgcn_cvt_pk_fp8_f32((r[2] - h1[0]) * 16.0f, (r[3] - h1[1]) * 16.0f, lo, true);
            q.hi[i][j / 4] = hi;
            q.lo[i][j / 4] = lo;
        }
    }
}

// c + codes x queries: rows are the 16 tokens, columns the 16 queries.
template <int DP>
__device__ __forceinline__ f32x4 scores(const Step<DP>& s, int a, const Queries<DP>& q) {
    f32x4 c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < Step<DP>::KB; ++i) {
        const u32x4_t w = s.k[a][i];
        const i32x8_t k = {static_cast<int>(w[0]), static_cast<int>(w[1]), static_cast<int>(w[2]), static_cast<int>(w[3]), 0, 0, 0, 0};
        c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k, q.lo[i], c, 4, 0, 0, s.ks[a][i], 0, q.scale[i] == 255 ? 255 : q.scale[i] - 4);
        c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k, q.hi[i], c, 4, 0, 0, s.ks[a][i], 0, q.scale[i]);
    }
    return c;
}

// A wave's state of RT * 16 queries: lane (n, g) holds, of query n, O at d = E (4 g + r) + i as o[][i][r].
template <int DP, int RT>
struct State {
    static constexpr int E = DP / 16;
    f32x4 o[RT][E];
    float m[RT], l[RT];
};

template <int DP, int RT, bool ONE>
__device__ __forceinline__ void attend(const Params& p, const Places<DP>& at, const Step<DP>& s, const Where<ONE>& where, int seq,
                                       int head, int token, int length, const int (&seen)[RT], int least,
                                       const Queries<DP> (&q)[RT], int lane, State<DP, RT>& st) {
    constexpr int E = DP / 16;
    const int g = lane >> 4;
    f32x4 score[RT][2];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int r = 0; r < RT; ++r) score[r][a] = scores<DP>(s, a, q[r]);
    uint32_t v[8][Step<DP>::VW];
    float unit[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t w = DP == 256 && at.second ? s.vs[j][Step<DP>::SW - 1] : s.vs[j][0];
        unit[j] = __uint_as_float(__builtin_amdgcn_alignbit(w, w, at.turn) & 0x7f800000u);
#pragma unroll
        for (int w = 0; w < Step<DP>::VW; ++w) v[j][w] = s.v[j][w];
    }
    bool odd = false;  // a value that is NaN, of a token that not all queries may see
    const bool masked = token + 32 > least || !where.has(0) || !where.has(1);
    if (masked) {
        asm volatile("");  // a branch around this stays one
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = token + 16 * a + 4 * g + j;
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    if (!where.has(a) || t >= seen[r]) score[r][a][j] = -__builtin_inff();
                // weights of 0 do not undo a NaN: it is taken out, and put back below where it is seen
                const bool absent = !where.has(a) || t >= length, nan = unit[4 * a + j] == __builtin_inff();
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

template <int DP, int RT, bool ONE>
__global__ __launch_bounds__(256, resident(DP, RT)) void kernel(Params p) {
    constexpr int E = DP / 16;
    constexpr int STAGES = 4 * kStages * kStage<DP>, SUMS = 2 * RT * E * 64 * 16;  // of the waves' steps, then of their sums
    __shared__ __attribute__((aligned(16))) uint8_t shared[STAGES > SUMS ? STAGES : SUMS];
    const uint32_t lds = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)shared));
    f32x4(*area)[RT * E][64] = reinterpret_cast<f32x4(*)[RT * E][64]>(shared);
    __shared__ float area_m[4][RT * 16], area_l[4][RT * 16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int pairs = p.kv_heads * p.row_blocks;  // of a sequence: (head, block of rows)
    int u = blockIdx.x, end = u + 1;
    int seq = 0, length, unit = 0, pair, first;
    Shares shares{};
    if (p.whole) {  // a pair for each workgroup
        seq = u / pairs;
        pair = u - seq * pairs;
        first = 0;
        length = __builtin_amdgcn_readfirstlane(length_of(p, seq));
        unit = rounds_of(length);
    } else {
        // the units of all sequences, then the sequence in which the first unit of this workgroup lies
        int its, rounds = rounds_at(p, 0, lane, &its), sum = rounds;
#pragma unroll 4
        for (int s = 64; s < p.sequences; s += 64) {
            int unused;
            sum += rounds_at(p, s, lane, &unused);
        }
        unit = unit_of(p, __builtin_amdgcn_readlane(wave_scan(sum), 63));
        int mine = (rounds + unit - 1) / unit, upto = wave_scan(mine);
        sum = mine;
#pragma unroll 4
        for (int s = 64; s < p.sequences; s += 64) {
            int unused;
            sum += (rounds_at(p, s, lane, &unused) + unit - 1) / unit;
        }
        const int total = __builtin_amdgcn_readlane(wave_scan(sum), 63);
        shares = shares_of(p, total);
        if (u >= shares.workgroups) return;
        end = shares.begin(u + 1);
        u = shares.begin(u);
        int before = 0;
        length = 0;
        const int x = u / pairs;
        for (int s = 0; s < p.sequences; s += 64) {
            if (s > 0) {
                mine = (rounds_at(p, s, lane, &its) + unit - 1) / unit;
                upto = wave_scan(mine);
            }
            const int last = min(64, p.sequences - s) - 1, with = upto + shares.start * (min(lane, last) + 1);
            const unsigned long long past = __ballot(before + with > x);
            if (past) {
                const int at = __ffsll(past) - 1;
                seq = s + at;
                length = __builtin_amdgcn_readlane(its, at);
                before += __builtin_amdgcn_readlane(with - mine - shares.start, at);
                break;
            }
            before += __builtin_amdgcn_readlane(with, 63);
        }
        const int in_seq = u - before * pairs, each = shares.start + (rounds_of(length) + unit - 1) / unit;
        pair = min(in_seq / each, pairs - 1);
        first = in_seq - pair * each - shares.start;  // below 0: what only counts as units
    }
    const uint32_t own = lds + wave * (kStages * kStage<DP>);
    Places<DP> at = places<DP>(p, lane, own);
    uint32_t stage = own;
    int other = kStage<DP>;  // on from this stage to the other
    int slot = 2 * blockIdx.x;
    while (u < end) {
        const int all = (rounds_of(length) + unit - 1) / unit;
        int count = __builtin_amdgcn_readfirstlane(min(all - first, end - u));
        u += count;
        if (first < 0) {
            count = max(count + first, 0);
            first = 0;
        }
        if (count == 0) break;  // the last units of this workgroup, and none of tokens
        const int head = pair / p.row_blocks, row0 = (pair - head * p.row_blocks) * p.row_block;
        const int stop = min((first + count) * unit * kRound, length);
        // While a step is worked on, out of registers, the next two are on their way to LDS.
        int token = first * unit * kRound + wave * 32;
        const int32_t* pages_of = p.table + static_cast<long long>(seq) * p.table_pitch;
        auto place = [&](int t) __attribute__((always_inline)) { return where_is<ONE>(p, pages_of, head, t, t < stop ? length : 0); };
        Where<ONE> here = place(token), next = place(token + kRound);
        barrier();  // the sums of the pair before have been read
        copy_step<DP, ONE>(p, here, lane, stage);
        copy_step<DP, ONE>(p, next, lane, stage + other);
        State<DP, RT> st;
        Queries<DP> q[RT];
        int seen[RT];
        const int least = length - p.tokens + 1;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int row = row0 + r * 16 + n;
            const int of = divide(min(row, p.rows - 1), p.per_group), h = head * p.group + min(row, p.rows - 1) - of * p.group;
            seen[r] = least + of;
            load_queries<DP>(p, p.q + seq * p.q_seq_stride + of * p.q_stride + h * p.q_head_stride, g, q[r]);
            st.m[r] = kLow;
            st.l[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < E; ++i) st.o[r][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        for (; token < stop; token += kRound) {
            const Where<ONE> later = place(token + 2 * kRound);
            Step<DP> s;
            wait_loads<kCopies<DP, ONE>>();
            read_step<DP>(at, s);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the step has been read: its stage may be filled again
            copy_step<DP, ONE>(p, later, lane, stage);
            attend<DP, RT, ONE>(p, at, s, here, seq, head, token, length, seen, least, q, lane, st);
            here = next;
            next = later;
            stage += other;
            move(at, other);
            other = -other;
        }
        wait_loads<0>();  // none is left on its way to LDS, which the sums take over
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
        barrier();
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
        barrier();
        if (wave < 2) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    st.o[r][i] += area[wave][r * E + i][lane];
                    if (wave == 1) area[1][r * E + i][lane] = st.o[r][i];
                }
        }
        barrier();
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
        slot = 2 * blockIdx.x + 1;
        first = -shares.start;
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
    __shared__ float area_m[256], area_l[256];
    const int lane = threadIdx.x & 63;
    const int pairs = p.kv_heads * p.row_blocks, seq = blockIdx.x / pairs, pair = blockIdx.x - seq * pairs;
    const int head = pair / p.row_blocks, in_block = blockIdx.y, row = (pair - head * p.row_blocks) * p.row_block + in_block;
    if (row >= p.rows) return;
    const int rounds = rounds_of(length_of(p, seq));
    if (rounds == 1) return;
    auto count = [&](int unit, int* before) {  // units of a head in all sequences, and in those before this
        int n = 0, b = 0;
        for (int s = lane; s < p.sequences; s += 64) {
            const int c = (rounds_of(length_of(p, s)) + unit - 1) / unit;
            n += c;
            b += s < seq ? c : 0;
        }
        *before = __builtin_amdgcn_readlane(wave_scan(b), 63);
        return __builtin_amdgcn_readlane(wave_scan(n), 63);
    };
    int before;
    int n = count(1, &before);
    const int unit = unit_of(p, n), mine = (rounds + unit - 1) / unit;
    if (unit > 1) n = count(unit, &before);
    const Shares shares = shares_of(p, n);
    const int u0 = (before + shares.start * seq) * pairs + pair * (shares.start + mine) + shares.start;
    const int w0 = shares.owner(u0), w1 = shares.owner(u0 + mine - 1);
    if (w0 == w1) return;
    auto place = [&](int w) {
        const int slot = 2 * w + (shares.begin(w) >= u0 - shares.start ? 0 : 1);  // its first part, or its last
        return static_cast<long long>(slot) * p.row_block + in_block;
    };
    const int across = p.dim / 4, strands = 256 / across;  // threads of a row, rows at a time
    const int strand = threadIdx.x / across, d = (threadIdx.x - strand * across) * 4;
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    float l = 0.0f, m = kLow;
    if (strand < strands) {
#pragma unroll 4
        for (int w = w0 + strand; w <= w1; w += strands) {
            const long long at = place(w);
            const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * at);
            const f32x4 o = *reinterpret_cast<const f32x4*>(p.part + at * p.dim + d);
            const float to = fmaxf(m, ml.x), f = __builtin_amdgcn_exp2f(m - to), e = __builtin_amdgcn_exp2f(ml.x - to);
            m = to;
            l = l * f + ml.y * e;
            sum = sum * f + o * e;
        }
    }
    area[threadIdx.x] = sum;
    area_l[threadIdx.x] = l;
    area_m[threadIdx.x] = m;
    __syncthreads();
    if (strand != 0) return;
    for (int s = 1; s < strands; ++s) {
        const float ms = area_m[s * across + threadIdx.x], to = fmaxf(m, ms);
        const float f = __builtin_amdgcn_exp2f(m - to), e = __builtin_amdgcn_exp2f(ms - to);
        m = to;
        l = l * f + area_l[s * across + threadIdx.x] * e;
        sum = sum * f + area[s * across + threadIdx.x] * e;
    }
    const float inverse = l == 0.0f ? 0.0f : 1.0f / l;
    const int token = divide(row, p.per_group), h = head * p.group + row - token * p.group;
    uint2 y;
    y.x = pack_bf16x2(sum[0] * inverse, sum[1] * inverse);
    y.y = pack_bf16x2(sum[2] * inverse, sum[3] * inverse);
    *reinterpret_cast<uint2*>(p.o + ((static_cast<long long>(seq) * p.tokens + token) * p.heads + h) * p.dim + d) = y;
}

struct Plan {
    int dp, rt, row_blocks, workgroups, few;
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
    const long long pairs = static_cast<long long>(d->sequences) * c->kv_heads * r.row_blocks;
    const int resident = compute_units() * decode::resident(r.dp, r.rt);
    r.few = std::max(1, resident / 4);
    // Where the page table has little room for tokens, or there are pairs enough for the device, each goes to a workgroup as a
    // whole and nothing is joined (heads of 128, 8 of the cache; us by rounds and whole: 1 sequence of 250 tokens 10.3 and 7.6, of 500 10.4
    // and 9.2, of 1000 10.4 and 12; 32 sequences of 1000 20 and 15, of 2000 25 and 22; 64 of up to 4000 36 and 31, of up to 8192
    // 69 and 71; 128 of up to 8192 131 and 128).
    r.join = longest > std::max(512ll, std::min(8 * pairs, 8192ll));
    r.workgroups = static_cast<int>(r.join ? std::min<long long>((longest + kRound - 1) / kRound * pairs, resident) : pairs);
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
    p.page_codes = static_cast<uint32_t>(c->kv_heads) * c->page_size * p.blocks * 16;  // below 2^31, as checked
    p.page_scales = static_cast<uint32_t>(c->kv_heads) * c->page_size * p.scale_pitch;
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
    p.whole = !plan.join;
    p.few = plan.few;
    const bool one = c->page_size % 32 == 0;
    auto go = [&](auto whole, auto halves) {
        if (one) whole<<<plan.workgroups, 256, 0, st>>>(p);
        else halves<<<plan.workgroups, 256, 0, st>>>(p);
    };
    if (plan.dp == 64) {
        if (plan.rt == 1) go(decode::kernel<64, 1, true>, decode::kernel<64, 1, false>);
        else if (plan.rt == 2) go(decode::kernel<64, 2, true>, decode::kernel<64, 2, false>);
        else go(decode::kernel<64, 4, true>, decode::kernel<64, 4, false>);
    } else if (plan.dp == 128) {
        if (plan.rt == 1) go(decode::kernel<128, 1, true>, decode::kernel<128, 1, false>);
        else if (plan.rt == 2) go(decode::kernel<128, 2, true>, decode::kernel<128, 2, false>);
        else go(decode::kernel<128, 4, true>, decode::kernel<128, 4, false>);
    } else {
        if (plan.rt == 1) go(decode::kernel<256, 1, true>, decode::kernel<256, 1, false>);
        else go(decode::kernel<256, 2, true>, decode::kernel<256, 2, false>);
    }
    cfwd_status e = check_hip(hipGetLastError(), "cache attention launch");
    if (e != CFWD_OK || !plan.join) return e;
    decode::join_kernel<<<dim3(p.sequences * p.kv_heads * p.row_blocks, std::min(p.rows, p.row_block)), 256, 0, st>>>(p);
    return check_hip(hipGetLastError(), "cache attention's joining launch");
}

}  // namespace cfwd

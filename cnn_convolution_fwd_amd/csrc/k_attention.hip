// Attention over packed prompts (gfx950).
//
//   o = softmax(scale * q k^T) v
//
// A workgroup takes 128 rows of one head of keys and values, a row being a (token,
// query head) of the group that shares it: grouped heads read their keys once,
// and a tile of rows spans few tokens, which wastes little at the causal edge.
// Each of its four waves has 32 rows.  Keys and values come 64 at a time through
// LDS, by copies that bypass the registers.  S^T = k q^T has a query in each
// lane's column and 16 of 32 keys in its registers, which is how P^T enters
// O^T = v^T P^T: only the row's sum passes between lanes (two of them hold a row).
// v^T comes out of LDS by transposing reads.
//
// Softmax.  Weights are 2^(s - m) with s in units of log2 and m no running maximum
// but any number that the scores have not passed by far: it moves only where a
// lane's 16 weights sum up to more than 2^12, then to the row's largest score, and
// O and l are multiplied by 2^(m - m').  Weights have bf16's 8 bits at any size, so
// nothing is lost, and no maximum is taken otherwise: sixteen instructions for every 64 keys and a
// chain of latencies before the weights less (16384 tokens: 2010 us with the
// maxima, 1960 without).  A row goes by its own scores alone, so that its result
// does not depend on the others'.
//
// A wave issues a vector instruction at most every eight cycles or so, alone on its SIMD or not, and a
// matrix instruction takes 32.  So no phase is left without either: while the matrix cores take the scores of the next 32
// keys, half of this half's weights are computed, and the other half of the next ones' while they multiply by the values.
// Two waves a SIMD (three for heads of 64) fill what is left.
//
// Few rows over many keys are split over the keys; a second launch joins the parts.
//
// Bound by the matrix cores for heads of 128 (16384 tokens, 32 heads over 8, causal: 2.0 ms, 1.1 PFLOP/s, busy 63% of the cycles; the
// matrix instructions alone take 1.3 ms) and by vector instructions for heads of 64 (32 images of 784 tokens, 16 heads: 127 us).
#include "attention.h"
#include "mx.h"

#include <algorithm>
#include <type_traits>

namespace cfwd {
namespace fa {

using namespace mx;
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) u32x4_t lds_u32x4;

constexpr int BN = 64;          // keys of a tile
constexpr float kLow = -3.0e38f;  // m before any score: finite, so that differences are numbers
constexpr float kMost = 4096.0f;  // a lane's 16 weights sum up to this before m follows the scores

struct Params {
    const bf16_t *q, *k, *v;
    bf16_t* o;
    const int32_t *q_starts, *k_starts;
    float *part, *part_ml;  // [split][row of q x heads][dim], [..][m, l]
    int sequences, tiles, heads, kv_heads, group, dim, causal, splits;
    int q_tokens, k_tokens;
    float scale2;  // scale * log2(e)
    long long q_stride, q_head_stride, k_stride, k_head_stride, v_stride, v_head_stride;
    Divisor per_group;
};

// Copies 16 bytes a lane from a buffer straight to LDS, lane after lane from `lds` on (the same for the wave);
// out-of-range lanes write 0.  The compiler does not see these loads: wait_loads() and a barrier come before the data
// are read.  It may have moved the buffer's words to scalar registers with vector instructions, which a load must not
// follow closer than five wait states.
__device__ __forceinline__ void load_to_lds16(const __amdgpu_buffer_rsrc_t& b, uint32_t off, uint32_t lds) {
    asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" : : "{m0}"(lds), "v"(off), "s"(b) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads() {  // until at most N of this wave's loads are outstanding
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// All waves of the workgroup, each with its reads of LDS done: what they read may then be overwritten.
__device__ __forceinline__ void barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// A number that is the same for the whole wave, in scalar registers.
__device__ __forceinline__ uint64_t uniform(uint64_t a) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32));
    return static_cast<uint64_t>(hi) << 32 | lo;
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(uint64_t p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(uniform(p)), 0, __builtin_amdgcn_readfirstlane(bytes),
                                             0x00020000);
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

// Rows of a sequence.
struct Range {
    int from, count;
};
__device__ __forceinline__ Range rows_of(const int32_t* starts, int seq, int tokens) {
    const int a = min(max(starts[seq], 0), tokens);
    return {a, min(max(starts[seq + 1], a), tokens) - a};
}

// A tile of rows, counted from the last sequence's last one back: its number in its sequence (below 0: there is none), and the
// sequence's queries and keys.  The same for the whole wave; each lane looks at one sequence of 64.  Up to 64 sequences: tiles
// follow each other without gaps.  More: a sequence's tiles begin at its first row / BM + its number, which no other's reach, and it
// is found by looking at 64 sequences evenly spaced, and at 64 between two of those, ...; some tiles are empty (2000 sequences of 50
// tokens, 8 heads of 64: 440 us going through all, 170 so; 10000 7350 and 850).
struct Place {
    int tile;
    Range q, k;
};
template <int BM>
__device__ __forceinline__ Place find_tile(const Params& p, int tile, int lane) {
    Place r = {-1, {0, 0}, {0, 0}};
    int from = 0, x = p.tiles - 1 - tile;
    if (p.sequences > 64) {
        for (int step, left = p.sequences; left > 64; left = min(step, p.sequences - from)) {
            step = (left + 63) / 64;
            const int seq = from + lane * step;
            const bool before = lane * step < left && rows_of(p.q_starts, seq, p.q_tokens).from * p.group / BM + seq <= x;
            from += max(__popcll(__ballot(before)) - 1, 0) * step;
        }
    }
    const int seq = min(from + lane, p.sequences - 1);
    const Range q = rows_of(p.q_starts, seq, p.q_tokens), k = rows_of(p.k_starts, seq, p.k_tokens);
    const bool is = from + lane < p.sequences;
    const int n = is ? (q.count * p.group + BM - 1) / BM : 0;
    int first;  // of the sequence's tiles
    if (p.sequences > 64) {
        first = q.from * p.group / BM + seq;
    } else {
        const int upto = wave_scan(n);
        x -= p.tiles - __builtin_amdgcn_readlane(upto, 63);
        first = upto - n;
    }
    const unsigned long long here = __ballot(is && x >= first && x < first + n);
    if (here) {
        const int at = __ffsll(here) - 1;
        r.tile = x - __builtin_amdgcn_readlane(first, at);
        r.q = {__builtin_amdgcn_readlane(q.from, at), __builtin_amdgcn_readlane(q.count, at)};
        r.k = {__builtin_amdgcn_readlane(k.from, at), __builtin_amdgcn_readlane(k.count, at)};
    }
    return r;
}

template <int N>
using Int = std::integral_constant<int, N>;

template <int DP, int NK, int NV, int WAVES, int KS, int VS, int SIMD_WAVES>
__global__ __launch_bounds__(64 * WAVES, SIMD_WAVES) void kernel(Params p) {
    constexpr int BM = 32 * WAVES, PIECES = DP / 8, TILE = BN * DP * 2, HALF = TILE / 2;
    constexpr int COPIES = BN * PIECES / (64 * WAVES);  // of 16 bytes, a thread and tile
    __shared__ __attribute__((aligned(1024))) uint8_t area[(KS + VS) * TILE];  // KS tiles of keys, then VS of values
    const uint32_t lds = static_cast<uint32_t>(
        reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)area));
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 31, h = lane >> 5;
    const int head = blockIdx.x % p.kv_heads;
    const Place place = find_tile<BM>(p, blockIdx.x / p.kv_heads, lane);
    if (place.tile < 0) return;
    const int row0 = place.tile * BM;
    const Range qs = place.q, ks = place.k;
    const int rows = qs.count * p.group;
    // row r sees the keys before offset + r / group + 1, and before ks.count
    const int offset = ks.count - qs.count;
    const int last_token = divide(min(row0 + BM, rows) - 1, p.per_group);
    const int keys = p.causal ? min(max(offset + last_token + 1, 0), ks.count) : ks.count;
    const int all_tiles = (keys + BN - 1) / BN;
    const int t0 = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<long long>(blockIdx.y) * all_tiles / p.splits));
    const int t1 = __builtin_amdgcn_readfirstlane(static_cast<int>((blockIdx.y + 1ll) * all_tiles / p.splits));

    // this wave's rows
    const int wave0 = row0 + wave * 32;
    const int row = min(wave0 + n, rows - 1), token = divide(row, p.per_group);
    const int end = __builtin_amdgcn_readfirstlane(min(t1 * BN, ks.count));  // of this split's keys
    const int seen = p.causal ? min(offset + token + 1, end) : end;
    u32x4_t q[NK];
    {
        const bf16_t* x = p.q + (qs.from + token) * p.q_stride + (head * p.group + row - token * p.group) * p.q_head_stride;
#pragma unroll
        for (int c = 0; c < NK; ++c) {
            const int d = 16 * c + 8 * h;
            q[c] = d < p.dim ? *reinterpret_cast<const u32x4_t*>(x + d) : u32x4_t{0, 0, 0, 0};
        }
    }
    const int first_token = divide(min(wave0, rows - 1), p.per_group);
    const int least = p.causal ? min(offset + first_token + 1, end) : end;  // every row of the wave sees these
    const int wave_last = divide(min(wave0 + 32, rows) - 1, p.per_group);
    const int most = wave0 >= rows ? 0 : p.causal ? min(max(offset + wave_last + 1, 0), end) : end;
    const int wave_t1 = (most + BN - 1) / BN;

    // copies: piece i * threads + thread of a tile, from the place that the permutation puts there; outside dim: nothing
    uint32_t k_off[COPIES], v_off[COPIES];
    const uint32_t k_row = static_cast<uint32_t>(p.k_stride) * 2, v_row = static_cast<uint32_t>(p.v_stride) * 2;  // bytes
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
        const int at = i * 64 * WAVES + threadIdx.x, r = at / PIECES, piece = at % PIECES;
        const int kp = piece ^ k_swizzle<DP>(r), vp = piece ^ v_swizzle<DP>(r);
        k_off[i] = kp * 8 < p.dim ? r * k_row + kp * 16 : 0xfffffff0u;
        v_off[i] = vp * 8 < p.dim ? r * v_row + vp * 16 : 0xfffffff0u;
    }
    const uint64_t k_base = uniform(reinterpret_cast<uint64_t>(p.k + ks.from * p.k_stride + head * p.k_head_stride));
    const uint64_t v_base = uniform(reinterpret_cast<uint64_t>(p.v + ks.from * p.v_stride + head * p.v_head_stride));
    const uint32_t lds_wave = lds + wave * 1024;
    // rows from the end on are out of the buffer's range and become zeros
    auto copy = [&](uint64_t base, uint32_t row_bytes, const uint32_t(&off)[COPIES], int key, uint32_t to) __attribute__((always_inline)) {
        int left = end - key;
        left = left < 0 ? 0 : left;
        left = left > BN ? BN : left;
        const auto b = buffer(base + static_cast<uint64_t>(static_cast<uint32_t>(key)) * row_bytes, left * row_bytes);
#pragma unroll
        for (int i = 0; i < COPIES; ++i) load_to_lds16(b, off[i], lds_wave + to + i * WAVES * 1024);
    };
    auto copy_k = [&](int key, int slot) __attribute__((always_inline)) { copy(k_base, k_row, k_off, key, slot * TILE); };
    auto copy_v = [&](int key, int slot) __attribute__((always_inline)) { copy(v_base, v_row, v_off, key, (KS + slot) * TILE); };

    // places of a lane's reads in a tile; those of other tiles differ by constants, which the reads hold.  Of keys, piece
    // 2 c + h of row n; of values, four lanes point at 16 values of each of four keys (a lane then gets one value of all four).
    uint32_t k_at[NK], v_at[NV];
#pragma unroll
    for (int c = 0; c < NK; ++c) {
        k_at[c] = lds + n * DP * 2 + ((2 * c + h) ^ k_swizzle<DP>(n)) * 16;
        asm volatile("" : "+v"(k_at[c]));
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int in = lane & 15, r = 4 * h + (in >> 2), d = 32 * i + 16 * ((lane >> 4) & 1) + 4 * (in & 3);
        v_at[i] = lds + KS * TILE + r * DP * 2 + ((d >> 3) ^ v_swizzle<DP>(r)) * 16 + (d & 7) * 2;
        asm volatile("" : "+v"(v_at[i]));
    }

    f32x16 o[NV], score[2];
    u32x4_t kf[NK];
    float m = kLow, l = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;

    auto mask = [&](f32x16& s, int key) __attribute__((always_inline)) {
        asm volatile("");  // a branch around this stays one: selecting every score would cost half as much as the softmax
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (key + 8 * (j / 4) + 4 * h + j % 4 >= seen) s[j] = -__builtin_inff();
    };

    // The weights of pair w of a half's scores, and their sum.  It takes the weights as they enter the product: rounded.
    auto weigh = [&](const f32x16& s, int w, float(&e)[2]) __attribute__((always_inline)) {
        e[0] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * w], p.scale2, -m));
        e[1] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * w + 1], p.scale2, -m));
    };
    auto pack = [&](const float(&e)[2], uint32_t& weight, float& sum) __attribute__((always_inline)) {
        weight = pack_bf16x2(e[0], e[1]);
        sum = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, weight), __builtin_bit_cast(bf16x2_t, 0x3f803f80u), sum, false);
    };
    // One step: while the matrix cores take the scores of the half that follows (from key next_key on; its keys are in kf),
    // the later weights of half B of the tile in slot V; while they take the product of the weights and B's values, the
    // earlier weights of the half that follows.  The keys of the half after it are K bytes into the keys' area.
    uint32_t early[4];
    float early_sum = 0.0f;
    bool not_finite = false;  // a value that is NaN or infinite was taken out
    auto step = [&](auto which, auto v_slot, auto k_after, int next_key, auto between) __attribute__((always_inline)) {
        constexpr int B = decltype(which)::value, V = decltype(v_slot)::value * TILE, K = decltype(k_after)::value;
        f32x16& cur = score[B];
        f32x16& nxt = score[1 - B];
        u32x4_t vf[2][NV];
        uint32_t weight[8] = {early[0], early[1], early[2], early[3]};
        float e[4][2], sum = early_sum;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int c = 0; c < NK; ++c) {
            if (c == 0)
#pragma unroll
                for (int j = 0; j < 16; ++j) nxt[j] = 0.0f;
            nxt = mma(kf[c], q[c], nxt);
#pragma unroll
            for (int r = 2 * NV * c / NK; r < 2 * NV * (c + 1) / NK; ++r)
#pragma unroll
                for (int part = 0; part < 2; ++part) {  // 16 keys: 16 (r / NV) + 4 h + (0 .. 3) and 8 on
                    const uint2 x = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        reinterpret_cast<lds_s16x4*>(v_at[r % NV] + V + (32 * B + 16 * (r / NV) + 8 * part) * DP * 2)));
                    vf[r / NV][r % NV][2 * part] = x.x;
                    vf[r / NV][r % NV][2 * part + 1] = x.y;
                }
            // the last products have no weights beside them: they cover the way from the sum to the branch
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i * NK / 6 == c) weigh(cur, 4 + i, e[i]);
                if (i * NK / 6 + 1 == c) pack(e[i], weight[4 + i], sum);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        asm volatile("" : "+v"(weight[4]), "+v"(weight[5]), "+v"(weight[6]), "+v"(weight[7]), "+v"(sum));  // all before the branch
        if (__any(!(sum <= kMost))) {
            // scores far above m (or the first ones, or NaN): m moves up to the row's largest, and the weights are taken again
            float top = cur[0];
#pragma unroll
            for (int j = 1; j < 16; ++j) top = fmaxf(top, cur[j]);
            top = fmaxf(top, __shfl_xor(top, 32)) * p.scale2;
            const float other = __shfl_xor(sum, 32);
            const float to = (!(sum <= kMost) || !(other <= kMost)) && top > m ? top : m, f = __builtin_amdgcn_exp2f(m - to);
            m = to;
            l *= f;
#pragma unroll
            for (int i = 0; i < NV; ++i) o[i] *= f;
            sum = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                weigh(cur, w, e[0]);
                pack(e[0], weight[w], sum);
            }
        }
        l += sum;
        if (p.causal && next_key > least) {
            // Some rows see keys of this half that others do not, and a weight of 0 does not undo a NaN or an infinity among
            // the values: those are taken out, and added at the end where they are seen.
            asm volatile("");
            typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
            u16x2 largest = {0, 0};
#pragma unroll
            for (int r = 0; r < 2 * NV; ++r)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    largest = __builtin_elementwise_max(largest, __builtin_bit_cast(u16x2, vf[r / NV][r % NV][j] & 0x7fff7fffu));
            if (__any(largest[0] >= 0x7f80 || largest[1] >= 0x7f80)) {
                not_finite = true;
#pragma unroll
                for (int r = 0; r < 2 * NV; ++r)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t x = vf[r / NV][r % NV][j];
                        vf[r / NV][r % NV][j] = x & ((x & 0x7f80u) == 0x7f80u ? 0xffff0000u : ~0u) &
                                                ((x & 0x7f800000u) == 0x7f800000u ? 0x0000ffffu : ~0u);
                    }
            }
        }
        between();
        if (next_key + BN / 2 > least) mask(nxt, next_key);
        early_sum = 0.0f;
        constexpr int M = 2 * NV;
#pragma unroll
        for (int x = 0; x < M; ++x) {
            const u32x4_t w = {weight[x / NV * 4], weight[x / NV * 4 + 1], weight[x / NV * 4 + 2], weight[x / NV * 4 + 3]};
            o[x % NV] = mma(vf[x / NV][x % NV], w, o[x % NV]);
#pragma unroll
            for (int c = NK * x / M; c < NK * (x + 1) / M; ++c) kf[c] = *reinterpret_cast<lds_u32x4*>(k_at[c] + K);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (1 + i * M / 6 == x) weigh(nxt, i, e[i]);
                if (2 + i * M / 6 == x || (x == M - 1 && 2 + i * M / 6 == M)) pack(e[i], early[i], early_sum);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        asm volatile("" : "+v"(early[0]), "+v"(early[1]), "+v"(early[2]), "+v"(early[3]), "+v"(early_sum));
    };

    // Tiles of keys in LDS lie half a tile behind those of values: tile t's steps need the keys of its second half and of
    // the next tile's first.  The very first half comes in the slot of values that is filled last.
    copy(k_base, k_row, k_off, t0 * BN, (KS + VS - 1) * TILE);
#pragma unroll
    for (int s = 0; s < KS || s < VS - 1; ++s) {
        if (s < KS) copy_k((t0 + s) * BN + BN / 2, s);
        if (s < VS - 1) copy_v((t0 + s) * BN, s);
    }
    // here q has arrived: a wait inside the loop would also be one for the copies that are on their way
#pragma unroll
    for (int c = 0; c < NK; ++c) asm volatile("" : "+v"(q[c]));
    wait_loads<(KS + VS - 3) * COPIES>();
    barrier();
    if (t0 < wave_t1) {
#pragma unroll
        for (int c = 0; c < NK; ++c) kf[c] = *reinterpret_cast<lds_u32x4*>(k_at[c] + (KS + VS - 1) * TILE);
#pragma unroll
        for (int j = 0; j < 16; ++j) score[0][j] = 0.0f;
#pragma unroll
        for (int c = 0; c < NK; ++c) score[0] = mma(kf[c], q[c], score[0]);
        mask(score[0], t0 * BN);
#pragma unroll
        for (int c = 0; c < NK; ++c) kf[c] = *reinterpret_cast<lds_u32x4*>(k_at[c]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float e[2];
            weigh(score[0], i, e);
            pack(e, early[i], early_sum);
        }
    }
    // Tile t, the u-th of a round over all slots.  Its turn, between the last scores that its keys give and the product with
    // its last values: the next tile is whole, and the slots of its keys and of the values before it are free.
    auto tile = [&](int t, auto round) __attribute__((always_inline)) {
        constexpr int U = decltype(round)::value, TURNS = KS - 1 < VS - 2 ? KS - 1 : VS - 2;
        auto turn = [&]() __attribute__((always_inline)) {
            wait_loads<(TURNS - 1) * 2 * COPIES>();
            barrier();
            copy_k((t + KS) * BN + BN / 2, U % KS);
            copy_v((t + VS - 1) * BN, (U + VS - 1) % VS);
        };
        if (t >= wave_t1) {
            turn();
            return;
        }
        step(Int<0>{}, Int<U % VS>{}, Int<U % KS * TILE + HALF>{}, t * BN + BN / 2, [] {});
        step(Int<1>{}, Int<U % VS>{}, Int<(U + 1) % KS * TILE>{}, t * BN + BN, turn);
    };
    constexpr int ROUND = KS == VS ? KS : KS * VS;
    static_assert(KS == 2 || KS == 4, "the slots of a round");
    for (int t = t0; t < t1; t += ROUND) {
        tile(t, Int<0>{});
        if (t + 1 < t1) tile(t + 1, Int<1>{});
        if (ROUND > 2 && t + 2 < t1) tile(t + 2, Int<2 % ROUND>{});
        if (ROUND > 3 && t + 3 < t1) tile(t + 3, Int<3 % ROUND>{});
        if (ROUND > 4 && t + 4 < t1) tile(t + 4, Int<4 % ROUND>{});
        if (ROUND > 5 && t + 5 < t1) tile(t + 5, Int<5 % ROUND>{});
    }
    wait_loads<0>();  // none is left on its way to LDS that the next workgroup may own

    l += __shfl_xor(l, 32);
    if (not_finite) {
        const bf16_t* x = p.v + ks.from * p.v_stride + head * p.v_head_stride;
        for (int key = max(least & ~(BN / 2 - 1), t0 * BN); key < min(seen, end); ++key)
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int d = 32 * i + 8 * (j / 4) + 4 * h + j % 4;
                    const float y = d < p.dim ? bf16_to_float(x[key * p.v_stride + d].bits) : 0.0f;
                    if (!(__builtin_fabsf(y) < __builtin_inff())) o[i][j] += y;
                }
    }
    if (wave0 + n >= rows) return;
    const long long at = static_cast<long long>(qs.from + token) * p.heads + head * p.group + row - token * p.group;
    if (p.splits == 1) {
        const float inverse = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int d = 32 * i + 8 * j + 4 * h;
                if (d >= p.dim) continue;
                uint2 y;
                y.x = pack_bf16x2(o[i][4 * j] * inverse, o[i][4 * j + 1] * inverse);
                y.y = pack_bf16x2(o[i][4 * j + 2] * inverse, o[i][4 * j + 3] * inverse);
                *reinterpret_cast<uint2*>(p.o + at * p.dim + d) = y;
            }
    } else {
        const long long to = at * p.splits + blockIdx.y;
        if (h == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * to) = make_float2(m, l);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int d = 32 * i + 8 * j + 4 * h;
                if (d < p.dim)
                    *reinterpret_cast<f32x4*>(p.part + to * p.dim + d) =
                        f32x4{o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]};
            }
    }
}

// Joins the parts of rows (token, head) of q: 4 values a thread, eight parts or so, `strands` threads side by side for a row's
// (1 query of 8 heads over 131072 keys, 256 parts: 58 us with one strand, 24 so; 256 of 32 heads over 16640, 8 parts: 87 with eight, 83 with one).
__global__ __launch_bounds__(256) void join_kernel(Params p, int strands, int rows) {
    __shared__ f32x4 area[256];
    __shared__ float area_m[256], area_l[256];
    const int across = p.dim / 4, in_row = across * strands, mine = threadIdx.x / in_row;
    const int strand = threadIdx.x % in_row / across, d = threadIdx.x % across * 4;
    const int row = blockIdx.x * (256 / in_row) + mine, token = row / p.heads;
    // rows before the first sequence and behind the last belong to none
    const bool has = mine < 256 / in_row && row < rows && token >= p.q_starts[0] && token < p.q_starts[p.sequences];
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + static_cast<long long>(row) * p.splits;
    const float* part = p.part + static_cast<long long>(row) * p.splits * p.dim + d;
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    float l = 0.0f, m = kLow;
    auto add = [&](float m_of, float l_of, const f32x4& o) {
        const float to = fmaxf(m, m_of), f = __builtin_amdgcn_exp2f(m - to), e = __builtin_amdgcn_exp2f(m_of - to);
        m = to;
        l = l * f + l_of * e;
        sum = sum * f + o * e;
    };
    if (has) {
#pragma unroll 4
        for (int s = strand; s < p.splits; s += strands)
            add(ml[s].x, ml[s].y, *reinterpret_cast<const f32x4*>(part + static_cast<long long>(s) * p.dim));
        area[threadIdx.x] = sum;
        area_l[threadIdx.x] = l;
        area_m[threadIdx.x] = m;
    }
    __syncthreads();
    if (!has || strand != 0) return;
    for (int s = 1; s < strands; ++s) {
        const int at = threadIdx.x + s * across;
        add(area_m[at], area_l[at], area[at]);
    }
    const float inverse = l == 0.0f ? 0.0f : 1.0f / l;
    uint2 y;
    y.x = pack_bf16x2(sum[0] * inverse, sum[1] * inverse);
    y.y = pack_bf16x2(sum[2] * inverse, sum[3] * inverse);
    *reinterpret_cast<uint2*>(p.o + static_cast<long long>(row) * p.dim + d) = y;
}

struct Plan {
    int splits;
    long long tiles;  // of the grid, empty ones among them
    size_t part_bytes, bytes;
};

Plan plan(const cfwd_attention_desc* d) {
    Plan r{};
    const long long group = d->q_heads / d->kv_heads, cus = compute_units();
    // n sequences of x rows in all have at most (x + n (bm - 1)) / bm tiles
    const long long rows = d->q_tokens * group, tiles = (rows + std::min<long long>(d->sequences, d->q_tokens) * 127) / 128;
    r.tiles = d->sequences > 64 ? rows / 128 + d->sequences : tiles;
    // Two workgroups a CU from parts of 512 keys on, else one from parts of 256 on (32 heads over 8, us: 16 queries over 2000 keys
    // 20 by 512 and 15 by 256, over 16400 32 with 64 parts and 27 with 32; 512 over 8700 91 with one a CU and 85 with two; 1000 over
    // themselves 38 in two parts and 25 in one).
    const long long whole = tiles * d->kv_heads, n = std::max(1, d->sequences);
    const long long keys = std::max(0ll, d->k_tokens - (d->causal ? d->q_tokens / 2 : 0)) / n;  // that a query sees, on average
    r.splits = static_cast<int>(std::max({1ll, std::min(cus / whole, keys / 256), std::min(2 * cus / whole, keys / 512)}));
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
    p.tiles = static_cast<int>(plan.tiles);
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
    auto go = [&](auto kernel, int waves) { kernel<<<grid, 64 * waves, 0, st>>>(p); };
    if (p.dim <= 64) go(fa::kernel<64, 4, 2, 4, 2, 3, 3>, 4);
    else if (p.dim <= 96) go(fa::kernel<128, 6, 3, 4, 2, 3, 2>, 4);
    else if (p.dim <= 128) go(fa::kernel<128, 8, 4, 4, 2, 3, 2>, 4);
    else go(fa::kernel<256, 16, 8, 4, 2, 3, 1>, 4);
    const cfwd_status e = check_hip(hipGetLastError(), "attention launch");
    if (e != CFWD_OK || plan.splits == 1) return e;
    const int across = d->head_dim / 4, strands = std::min(256 / across, (plan.splits + 7) / 8), each = 256 / (across * strands);
    const int rows = static_cast<int>(d->q_tokens * d->q_heads);  // split only where they are few
    fa::join_kernel<<<(rows + each - 1) / each, 256, 0, st>>>(p, strands, rows);
    return check_hip(hipGetLastError(), "attention's joining launch");
}

}  // namespace cfwd

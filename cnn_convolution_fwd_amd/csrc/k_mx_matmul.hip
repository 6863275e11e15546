// Product of two MXFP4 matrices (gfx950): y = act(x w^T + bias).
#include "mx_matmul_impl.h"

#include <algorithm>
#include <type_traits>

namespace cfwd {
namespace mx {

// Copies 16 (or 4) bytes a lane from a buffer straight to LDS, lane after lane
// from `lds` on (wave-uniform); out-of-range lanes write 0.  The address in LDS
// travels in m0, which the compiler itself sets (one wait state before its use).  It does
// not see these loads: wait_loads() and a barrier come before the data are read.
__device__ __forceinline__ void load_to_lds16(const __amdgpu_buffer_rsrc_t& b, uint32_t off, uint32_t lds) {
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" : : "{m0}"(lds), "v"(off), "s"(b) : "memory");
}
__device__ __forceinline__ void load_to_lds4(const __amdgpu_buffer_rsrc_t& b, uint32_t off, uint32_t lds) {
    asm volatile("s_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" : : "{m0}"(lds), "v"(off), "s"(b) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads() {  // until at most N of this wave's loads are outstanding
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// All waves of the workgroup; what memory accesses the code has before and after stays there.
__device__ __forceinline__ void barrier() { asm volatile("s_barrier" ::: "memory"); }

struct Tiling {
    int tiles_m, tiles_n;
    int split_stages;  // of a part of the sum over K; each part has its own y (m x ldy) behind the last
    Divisor tiles;     // of one part
    Divisor group, height, last_height;  // of tiles in a group of 8 rows of tiles; of rows in a group, in the last one
};

// The u-th tile, of BM x BN: the order goes down columns of 8 tiles, part by part.
template <int BM, int BN>
__device__ __forceinline__ void tile_place(const Tiling& order, int u, long long* m0, int* n0, int* split) {
    *split = divide(u, order.tiles);
    const int t = u - *split * order.tiles.d;
    const int group = divide(t, order.group), in_group = t - group * order.group.d;
    const Divisor height = group == (order.tiles_m - 1) / 8 ? order.last_height : order.height;
    const int column = divide(in_group, height);
    *m0 = static_cast<long long>(group * 8 + in_group - column * height.d) * BM;
    *n0 = column * BN;
}

// Tiles through LDS: 128 rows of y x 128 columns; the four waves (2 x 2) of a
// workgroup take 64 x 64 each.  The grid is what fits the device at once, two
// workgroups on a CU, and each works through several tiles as one unbroken run of
// stages of 128 values of K, so that a tile's output pass finds the next tile's
// operands on their way.
//
// LDS holds four stages in turn.  While stage s is multiplied, s + 1 is whole,
// s + 2 is on its way and s + 3 is requested, so the operands of the next
// matrix instructions are always read from LDS ahead of their use, across
// stages and tiles too, and a memory latency has two stages to pass.  Requests
// past the last stage are made all the same (out of range: they load nothing),
// so that the count of outstanding loads is known.
//
// Scales come four stages ("a group") at a time, so that a 16-byte run of each
// row is read at once: a word at a time costs a cache line for every word
// (8192^3: 524 us so, 405 in groups).
//
// A stage's row is 64 bytes, four blocks, of which half h of a wave takes
// blocks 2 h and 2 h + 1.  LDS serves 16 lanes' 16 bytes at once if they cover
// its 64 banks, four rows, so block b of row i lies in slot b ^ ((i >> 2) & 3):
// 16 rows' reads of one block then do.  The copy to LDS is linear in lanes, so
// the permutation is made in the addresses that the lanes load from.
//
// The output pass of the tile uses the LDS of the stage multiplied last, which
// is filled again only after the next stage's barrier.

template <typename TY>
__global__ __launch_bounds__(256, 2) void tile_kernel(MatmulParams p, Tiling order, bool fast) {
    constexpr int F = 2, B = 64 * F, STAGE = 2 * B * 64, GROUP = 2 * B * 16;
    constexpr int CODE_LOADS = 2 * F, SCALE_LOADS = 2 * F;  // a wave's copies for a stage, for a group
    constexpr int STORES = stores<F, F, TY>();
    __shared__ __attribute__((aligned(128))) uint8_t lds[4 * STAGE + 4 * GROUP];
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;

    // The i-th tile of this workgroup.  A round of tiles is a run of their order, each XCD a run within it.
    const int tiles = order.tiles.d;
    const int rounds = (tiles - 1 - static_cast<int>(blockIdx.x)) / static_cast<int>(gridDim.x) + 1;
    auto tile_at = [&](int i, long long* m0, int* n0) {
        const int first = i * gridDim.x;
        int split;  // there is one part
        tile_place<B, B>(order, first + xcd_linear(blockIdx.x, min(static_cast<int>(gridDim.x), tiles - first)), m0, n0, &split);
    };

    const int stages = (p.kb + 3) / 4;
    const uint32_t lds0 = static_cast<uint32_t>(
        reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds));
    // copying: tile number, stage of K, stage and group of all
    int copy_tile = 0, copy_stage = 0, copy_count = 0, copy_group = 0;
    __amdgpu_buffer_rsrc_t gx, gxs, gw, gws;
    auto open_tile = [&] {
        long long m0 = 0, rows_x = 0, rows_w = 0;
        int n0 = 0;
        if (copy_tile < rounds) {
            tile_at(copy_tile, &m0, &n0);
            rows_x = min(static_cast<long long>(B), p.m - m0);
            rows_w = min(B, p.n - n0);
        }
        copy_stage = 0;
        gx = buffer(p.x + m0 * p.pitch, rows_x * p.pitch);
        gxs = buffer(p.xs + m0 * p.spitch, rows_x * p.spitch);
        gw = buffer(p.w + static_cast<long long>(n0) * p.pitch, rows_w * p.pitch);
        gws = buffer(p.ws + static_cast<long long>(n0) * p.spitch, rows_w * p.spitch);
    };
    // one copy: 16 rows' codes of a stage, or 16 rows' scales of a group
    const int copy_block = (lane & 3) ^ (lane >> 4);
    const uint32_t copy_off = (wave * 16 + (lane >> 2)) * p.pitch + copy_block * 16;
    const uint32_t copy_soff = (wave * 16 + (lane >> 2)) * p.spitch + (lane & 3) * 4;
    auto copy_codes = [&](int i) {  // i-th of each operand's F copies
        const uint32_t off = copy_stage * 4 + copy_block < p.kb ? copy_off + copy_stage * 64 : kOutOfRange;
        const uint32_t to = lds0 + (copy_count & 3) * STAGE + wave * 1024 + i * 4096;
        load_to_lds16(gw, off + i * 64 * p.pitch, to);
        load_to_lds16(gx, off + i * 64 * p.pitch, to + B * 64);
    };
    auto copy_scales = [&] {  // with a group's first stage
        const uint32_t off = copy_stage * 4 + (lane & 3) * 4 < p.spitch ? copy_soff + copy_stage * 4 : kOutOfRange;
        const uint32_t to = lds0 + 4 * STAGE + (copy_group & 3) * GROUP + wave * 256;
#pragma unroll
        for (int i = 0; i < F; ++i) {
            load_to_lds4(gws, off + i * 64 * p.spitch, to + i * 1024);
            load_to_lds4(gxs, off + i * 64 * p.spitch, to + B * 16 + i * 1024);
        }
    };
    auto next_copy = [&] {
        ++copy_count;
        if ((++copy_stage & 3) == 0 || copy_stage == stages) ++copy_group;
        if (copy_stage == stages) {
            ++copy_tile;
            open_tile();
        }
    };

    // fragments of one matrix instruction's depth, two sets in turn; scale words of a stage
    i32x4 a[2][F], b[2][F];
    int sw[2][F], sx[2][F];
    const int swz = (r >> 2) & 3;
    const uint8_t* lw = lds + (wn * 32 * F + r) * 64;
    const uint8_t* lx = lds + (B + wm * 32 * F + r) * 64;
    const uint8_t* lws = lds + 4 * STAGE + (wn * 32 * F + r) * 16;
    const uint8_t* lxs = lds + 4 * STAGE + (B + wm * 32 * F + r) * 16;
    auto read_pair = [&](int count, int j, int set, int f) {
        const int at = (count & 3) * STAGE + ((2 * h + j) ^ swz) * 16 + f * 2048;
        a[set][f] = *reinterpret_cast<const i32x4*>(lw + at);
        b[set][f] = *reinterpret_cast<const i32x4*>(lx + at);
    };
    auto read_scales = [&](int stage, int group, int set, int f) {
        const int at = (group & 3) * GROUP + (stage & 3) * 4 + f * 512;
        sw[set][f] = *reinterpret_cast<const int*>(lws + at);
        sx[set][f] = *reinterpret_cast<const int*>(lxs + at);
    };

    bool had_scales = false;  // whether the last copies were a group's first
    open_tile();
#pragma unroll
    for (int s = 0; s < 3; ++s) {
#pragma unroll
        for (int i = 0; i < F; ++i) copy_codes(i);
        had_scales = (copy_stage & 3) == 0;
        if (had_scales) copy_scales();
        next_copy();
    }
    wait_loads<2 * CODE_LOADS>();
    barrier();
#pragma unroll
    for (int f = 0; f < F; ++f) {
        read_scales(0, 0, 0, f);
        read_pair(0, 0, 0, f);
    }

    const int last_bits = scale_bits(p.kb - (stages - 1) * 4 - 2 * h);  // of this half's scales in a row's last stage
    f32x16 acc[F][F] = {};
    int count = 0, group = 0;  // of the stage that is multiplied, among all
    int since = 4;             // stages since the last output pass
    for (int tile = 0; tile < rounds; ++tile) {
        long long m0;
        int n0;
        tile_at(tile, &m0, &n0);
        m0 += wm * 32 * F;
        n0 += wn * 32 * F;
        float bias[F][16];
        load_bias(p, n0, bias);  // ahead of the output pass
        for (int stage = 0; stage < stages; ++stage, ++count, ++since) {
            // This wave's copies for the next stage: those for the one after it, and stores, may be outstanding.
            if (since < 2) {
                if (had_scales) wait_loads<(CODE_LOADS + SCALE_LOADS + STORES < 63 ? CODE_LOADS + SCALE_LOADS + STORES : 63)>();
                else wait_loads<(CODE_LOADS + STORES < 63 ? CODE_LOADS + STORES : 63)>();
            } else {
                if (had_scales) wait_loads<CODE_LOADS + SCALE_LOADS>();
                else wait_loads<CODE_LOADS>();
            }
            barrier();  // all waves' copies for it; and the stage before this one is no longer read
            const int bits = stage == stages - 1 ? last_bits : 16;
#pragma unroll
            for (int f = 0; f < F; ++f) {
                sw[0][f] = __builtin_amdgcn_ubfe(sw[0][f], 16 * h, bits);
                sx[0][f] = __builtin_amdgcn_ubfe(sx[0][f], 16 * h, bits);
            }
#pragma unroll
            for (int i = 0; i < F; ++i) {
                copy_codes(i);
                read_pair(count, 1, 1, i);
#pragma unroll
                for (int f = 0; f < F; ++f) acc[i][f] = mfma<0>(a[0][f], b[0][i], acc[i][f], sw[0][f], sx[0][i]);
                __builtin_amdgcn_sched_barrier(0);
            }
            had_scales = (copy_stage & 3) == 0;
            if (had_scales) copy_scales();
            next_copy();
            const int next_stage = stage + 1 == stages ? 0 : stage + 1;
            group += (next_stage & 3) == 0;
#pragma unroll
            for (int i = 0; i < F; ++i) {
                read_pair(count + 1, 0, 0, i);
                read_scales(next_stage, group, 1, i);
#pragma unroll
                for (int f = 0; f < F; ++f) acc[i][f] = mfma<1>(a[1][f], b[1][i], acc[i][f], sw[0][f], sx[0][i]);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int f = 0; f < F; ++f) {
                sw[0][f] = sw[1][f];
                sx[0][f] = sx[1][f];
            }
        }
        barrier();  // the last stage's LDS is no longer read
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int f = 0; f < F; ++f)
#pragma unroll
                for (int j = 0; j < 16; ++j) acc[i][f][j] += bias[f][j];
        write_tile<F, F, TY>(acc, p, m0, n0, fast, lds + ((count - 1) & 3) * STAGE + wave * (STAGE / 4));
        if (!fast) wait_loads<0>();  // an unknown number of stores
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int f = 0; f < F; ++f) acc[i][f] = f32x16{};
        since = 0;
    }
    wait_loads<0>();  // no copy may reach LDS after the workgroup has ended
}

// Short sums over many rows of y (a 1x1 convolution's shape): 128 x 128 of y as
// in the narrow kernel, but x is brought to LDS once for all columns of its 128
// rows, S stages = 128 S values of K, and only w streams through.  A workgroup
// has a run of tiles in the order of y, columns first.
//
// The output pass is most of such a product: its vector instructions (a gelu
// with its bias and rounding is 9 a value) bound it, and they want waves to
// change between.  So this kernel keeps its LDS and registers small enough for
// three workgroups a CU where it can, has no fragments on their way across the
// barrier, and begins sums with the bias, which travels to LDS with w's scale
// words (both by waves' own fourth of one copy).
//
// 100352 x 1024 x 256, gelu, bf16: 57 us (narrow tiles 76); x in MXFP4 to y in
// MXFP4, 25088 x 2048 x 512, gelu: 41 (47), without gelu 30 (37).  Quantising x
// on its way to LDS was slower than a launch of its own before (80 us
// against 73 with it, 53 against 46), because every workgroup then waits for memory.
template <int S, typename TY>
struct Resident {
    static constexpr int kStage = 128 * 64, kWords = 128 * 8;       // of w: a stage's codes; its scale words and the bias
    static constexpr bool kThree = S == 2 || std::is_void<TY>::value;  // workgroups a CU, by LDS
    static constexpr int kRing = S == 2 ? 3 : kThree ? 2 : 4;
    static constexpr int kW = S * (kStage + 128 * 4), kWS = kW + kRing * kStage, kArea = kWS + kRing * kWords;
    static constexpr int kBytes = kArea + (std::is_void<TY>::value ? 0 : 8192);
};

template <int S, typename TY>
__global__ __launch_bounds__(256, (Resident<S, TY>::kThree ? 3 : 2)) void rows_kernel(MatmulParams p, int tiles_n,
                                                                                    long long tiles, bool fast) {
    using L = Resident<S, TY>;
    constexpr int F = 2, B = 128, STAGE = L::kStage, R = L::kRing, XS = S * STAGE;
    constexpr int LOADS = 3;  // a wave's copies for a stage of w
    constexpr int STORES = stores<F, F, TY>();
    __shared__ __attribute__((aligned(128))) uint8_t lds[L::kBytes];
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int stages = (p.kb + 3) / 4;
    const long long begin = tiles * blockIdx.x / gridDim.x, end = tiles * (blockIdx.x + 1) / gridDim.x;
    const uint32_t lds0 = static_cast<uint32_t>(
        reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds));

    // copying w: tile's column, stage, place in the ring.  Past the last tile some column is copied that nobody reads.
    const __amdgpu_buffer_rsrc_t gw = buffer(p.w, static_cast<long long>(p.n) * p.pitch);
    const __amdgpu_buffer_rsrc_t gs =  // scales (waves 0 and 1) or bias
        wave < 2 ? buffer(p.ws, static_cast<long long>(p.n) * p.spitch) : buffer(p.bias, p.bias ? p.n * 4ll : 0);
    const uint32_t column_step = B * p.pitch, column_sstep = wave < 2 ? B * p.spitch : B * 4, stage_sstep = wave < 2 ? 4 : 0;
    int copy_column = static_cast<int>(begin % tiles_n), copy_stage = 0, copy_slot = 0;
    const int copy_block = (lane & 3) ^ (lane >> 4);
    const uint32_t copy_off = (wave * 16 + (lane >> 2)) * p.pitch + copy_block * 16;
    const uint32_t copy_soff = ((wave & 1) * 64 + lane) * (wave < 2 ? p.spitch : 4);
    auto copy_codes = [&](int i) {
        const uint32_t off = copy_off + (copy_column * column_step + copy_stage * 64 + i * 64 * p.pitch);
        load_to_lds16(gw, copy_stage * 4 + copy_block < p.kb ? off : kOutOfRange,
                      lds0 + L::kW + copy_slot * STAGE + wave * 1024 + i * 4096);
    };
    auto copy_scales = [&] {
        load_to_lds4(gs, copy_soff + (copy_column * column_sstep + copy_stage * stage_sstep),
                     lds0 + L::kWS + copy_slot * L::kWords + wave * 256);
    };
    auto next_copy = [&] {
        copy_slot = copy_slot == R - 1 ? 0 : copy_slot + 1;
        if (++copy_stage < stages) return;
        copy_stage = 0;
        copy_column = copy_column == tiles_n - 1 ? 0 : copy_column + 1;
    };

    // x's rows m0 .. m0 + 127 -> LDS; every wave is done with the rows before
    auto bring_x = [&](long long m0) {
        const long long rows = min(static_cast<long long>(B), p.m - m0);
        const __amdgpu_buffer_rsrc_t gx = buffer(p.x + m0 * p.pitch, rows * p.pitch),
                                     gxs = buffer(p.xs + m0 * p.spitch, rows * p.spitch);
#pragma unroll
        for (int t = 0; t < S; ++t) {
            const uint32_t off = t * 4 + copy_block < p.kb ? copy_off + t * 64 : kOutOfRange;
#pragma unroll
            for (int i = 0; i < 2; ++i) load_to_lds16(gx, off + i * 64 * p.pitch, lds0 + t * STAGE + wave * 1024 + i * 4096);
        }
        const int at = lane % S;
        const uint32_t off = at * 4 < p.spitch ? (wave * (64 / S) + lane / S) * p.spitch + at * 4 : kOutOfRange;
#pragma unroll
        for (int i = 0; i < S / 2; ++i)
            load_to_lds4(gxs, off + i * (256 / S) * p.spitch, lds0 + XS + wave * 256 + i * 1024);
    };

    const int swz = (r >> 2) & 3;
    const uint8_t* lw = lds + L::kW + (wn * 32 * F + r) * 64;
    const uint8_t* lx = lds + (wm * 32 * F + r) * 64;
    const uint8_t* lws = lds + L::kWS + (wn * 32 * F + r) * 4;
    const uint8_t* lxs = lds + XS + (wm * 32 * F + r) * (S * 4);
    const uint8_t* lb = lds + L::kWS + B * 4 + wn * 32 * F * 4 + h * 16;
    const int last_bits = scale_bits(p.kb - (stages - 1) * 4 - 2 * h);  // of this half's scales in a row's last stage

#pragma unroll
    for (int s = 0; s < R - 1; ++s) {
        copy_codes(0);
        copy_codes(1);
        copy_scales();
        next_copy();
    }
    int slot = 0, since = R, column = static_cast<int>(begin % tiles_n);
    long long m_tile = begin / tiles_n;
    bool fresh = true;  // rows of x to be brought
    for (long long tile = begin; tile < end; ++tile) {
        if (fresh) {
            barrier();
            bring_x(m_tile * B);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            wait_loads<0>();  // the first stage's barrier follows
            fresh = false;
        }
        f32x16 acc[F][F];
        for (int stage = 0; stage < stages; ++stage, ++since) {
            if (since < R - 1) wait_loads<(R - 2) * LOADS + STORES>();
            else wait_loads<(R - 2) * LOADS>();
            barrier();  // this stage of w is whole; the one before is no longer read
            copy_codes(0);
            copy_codes(1);
            copy_scales();
            next_copy();
            const uint8_t *w = lw + slot * STAGE, *x = lx + stage * STAGE;
            i32x4 a[2][F], b[2][F];
            int sw[F], sx[F];
            const int bits = stage == stages - 1 ? last_bits : 16;
#pragma unroll
            for (int f = 0; f < F; ++f) {
                sw[f] = __builtin_amdgcn_ubfe(*reinterpret_cast<const int*>(lws + slot * L::kWords + f * 128), 16 * h, bits);
                sx[f] = __builtin_amdgcn_ubfe(*reinterpret_cast<const int*>(lxs + stage * 4 + f * (S * 128)), 16 * h, bits);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int f = 0; f < F; ++f) {
                    a[j][f] = *reinterpret_cast<const i32x4*>(w + ((2 * h + j) ^ swz) * 16 + f * 2048);
                    b[j][f] = *reinterpret_cast<const i32x4*>(x + ((2 * h + j) ^ swz) * 16 + f * 2048);
                }
            if (stage == 0) {  // sums begin with the bias
#pragma unroll
                for (int f = 0; f < F; ++f)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const float4 v = *reinterpret_cast<const float4*>(lb + slot * L::kWords + f * 128 + g * 32);
#pragma unroll
                        for (int i = 0; i < F; ++i) {
                            acc[i][f][g * 4] = v.x;
                            acc[i][f][g * 4 + 1] = v.y;
                            acc[i][f][g * 4 + 2] = v.z;
                            acc[i][f][g * 4 + 3] = v.w;
                        }
                    }
            }
#pragma unroll
            for (int i = 0; i < F; ++i)
#pragma unroll
                for (int f = 0; f < F; ++f) acc[i][f] = mfma<0>(a[0][f], b[0][i], acc[i][f], sw[f], sx[i]);
#pragma unroll
            for (int i = 0; i < F; ++i)
#pragma unroll
                for (int f = 0; f < F; ++f) acc[i][f] = mfma<1>(a[1][f], b[1][i], acc[i][f], sw[f], sx[i]);
            slot = slot == R - 1 ? 0 : slot + 1;
        }
        uint8_t* area = nullptr;
        if constexpr (!std::is_void<TY>::value) {
            barrier();  // the last stage of w is no longer read
            area = lds + (wave < 2 ? L::kW + (slot == 0 ? R - 1 : slot - 1) * STAGE + wave * 4096 : L::kArea + (wave - 2) * 4096);
        }
        write_tile<F, F, TY>(acc, p, m_tile * B + wm * 32 * F, column * B + wn * 32 * F, fast, area);
        if (!fast) wait_loads<0>();  // an unknown number of stores
        since = 0;
        if (++column == tiles_n) {
            column = 0;
            ++m_tile;
            fresh = true;
        }
    }
    wait_loads<0>();  // no copy may reach LDS after the workgroup has ended
}

// Wide tiles, for long sums over many tiles: 256 rows of y x 256 columns, one
// tile a workgroup of eight waves, one workgroup a CU: half the copies of the
// narrow kernel for the same products.  A wave has 128 x 64 of y, so that every
// SIMD has two waves to alternate between: four waves of 128 x 128 read a third
// less from LDS but took longer (8192^3 263 us, 254 so; x 1024 70 and 60; 25088 x
// 512 x 2048 25 and 21).
//
// A stage is 256 values of K here, its rows 128 bytes: a copy costs by the cache
// line that it touches, whatever it takes of it (from L2 134 GB/s a CU in whole
// lines, 69 GB/s in halves).  LDS holds two stages.  A stage's matrix
// instructions are four steps, whose operands are read one step ahead; before
// the last of them all of the stage is in registers, and there the waves meet:
// the next stage is whole, and the copies of the one after it begin, over the one
// just read, spread over the matrix instructions of this step and the next
// (with four waves 281 us with all of them in one step, 269 so, 231 without copies;
// 305 with four stages of 128 values).
//
// Block b of row i lies in slot b ^ ((i >> 1) & 7), scale word q of a row's 8 (four
// stages', "a chunk") at q ^ (2 ((i >> 3) & 3)): 16 rows' reads of one block
// then cover the 64 banks (with i & 7, conflicts took 62% of LDS's cycles).
template <typename TY>
__global__ __launch_bounds__(512, 1) void wide_kernel(MatmulParams p, Tiling order, bool fast) {
    constexpr int FM = 4, FN = 2, B = 256, STAGE = 2 * B * 128, CHUNK = 2 * B * 32;
    __shared__ __attribute__((aligned(128))) uint8_t lds[2 * STAGE + 2 * CHUNK];
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    long long m0;
    int n0, split;
    tile_place<B, B>(order, xcd_linear(blockIdx.x, gridDim.x), &m0, &n0, &split);
    const int stages = (p.kb + 7) / 8;
    const long long rows_x = min(static_cast<long long>(B), p.m - m0), rows_w = min(B, p.n - n0);
    const __amdgpu_buffer_rsrc_t gx = buffer(p.x + m0 * p.pitch, rows_x * p.pitch),
                                 gxs = buffer(p.xs + m0 * p.spitch, rows_x * p.spitch),
                                 gw = buffer(p.w + static_cast<long long>(n0) * p.pitch, rows_w * p.pitch),
                                 gws = buffer(p.ws + static_cast<long long>(n0) * p.spitch, rows_w * p.spitch);
    const uint32_t lds0 = static_cast<uint32_t>(
        reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds));

    // one copy: 8 rows' codes of a stage, or 8 rows' scales of a chunk
    const int copy_row = wave * 8 + (lane >> 3);
    const int copy_block = (lane & 7) ^ ((copy_row >> 1) & 7), copy_word = (lane & 7) ^ (2 * (wave & 3));
    const uint32_t copy_off = copy_row * p.pitch + copy_block * 16, copy_soff = copy_row * p.spitch + copy_word * 4;
    auto copy_codes = [&](int stage, int i) {  // i-th of each operand's 4 copies
        const uint32_t off = stage * 8 + copy_block < p.kb ? copy_off + stage * 128 : kOutOfRange;
        const uint32_t to = lds0 + (stage & 1) * STAGE + wave * 1024 + i * 8192;
        load_to_lds16(gw, off + i * 64 * p.pitch, to);
        load_to_lds16(gx, off + i * 64 * p.pitch, to + B * 128);
    };
    auto copy_scales = [&](int part, int i) {  // i-th of 2 copies: quarter part % 4 of chunk part / 4, half the rows of w or of x
        const int chunk = part >> 2, half = (part & 1) * (B / 2);
        const uint32_t off = chunk * 32 + copy_word * 4 < p.spitch ? copy_soff + chunk * 32 : kOutOfRange;
        const uint32_t to = lds0 + 2 * STAGE + (chunk & 1) * CHUNK + (part & 2) / 2 * (B * 32) + half * 32 + wave * 256 + i * 2048;
        load_to_lds4(part & 2 ? gxs : gws, off + (half + i * 64) * p.spitch, to);
    };

    i32x4 a[2][FN], b[2][FM];  // operands of two steps in turn
    int sw[2][FN], sx[2][FM];  // scale words of a stage, and of the next
    const uint8_t* lw = lds + (wn * 32 * FN + r) * 128;
    const uint8_t* lx = lds + (B + wm * 32 * FM + r) * 128;
    const uint8_t* lws = lds + 2 * STAGE + (wn * 32 * FN + r) * 32;
    const uint8_t* lxs = lds + 2 * STAGE + (B + wm * 32 * FM + r) * 32;
    auto read_pair = [&](int stage, int j, int f) {
        const int at = (stage & 1) * STAGE + ((4 * h + j) ^ ((r >> 1) & 7)) * 16 + f * 4096;
        if (f < FN) a[j & 1][f] = *reinterpret_cast<const i32x4*>(lw + at);
        b[j & 1][f] = *reinterpret_cast<const i32x4*>(lx + at);
    };
    auto read_scales = [&](int stage, int set, int f) {
        const int at = (stage >> 2 & 1) * CHUNK + (((stage & 3) * 2 + h) ^ (2 * (r >> 3))) * 4 + f * 1024;
        if (f < FN) sw[set][f] = *reinterpret_cast<const int*>(lws + at);
        sx[set][f] = *reinterpret_cast<const int*>(lxs + at);
    };
    f32x16 acc[FM][FN];
    auto multiply = [&](auto j, int i) {
        constexpr int J = decltype(j)::value;
#pragma unroll
        for (int f = 0; f < FN; ++f) acc[i][f] = mfma<J>(a[J & 1][f], b[J & 1][i], acc[i][f], sw[0][f], sx[0][i]);
        __builtin_amdgcn_sched_barrier(0);
    };

#pragma unroll
    for (int i = 0; i < 4; ++i) copy_codes(0, i);
#pragma unroll
    for (int q = 0; q < 5; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) copy_scales(q, i);
    {  // sums begin with the bias
        float bias[FN][16];
        load_bias(p, n0 + wn * 32 * FN, bias);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int f = 0; f < FN; ++f)
#pragma unroll
                for (int j = 0; j < 16; ++j) acc[i][f][j] = bias[f][j];
    }
    wait_loads<0>();
#pragma unroll
    for (int i = 0; i < 2; ++i) copy_codes(1, i);
    barrier();
    // of this half's scale word in a row's last stage, the bytes of blocks
    const int last_left = p.kb - (stages - 1) * 8 - 4 * h;
    const int last_mask = last_left >= 4 ? -1 : (1 << scale_bits(last_left) << scale_bits(last_left - 2)) - 1;
#pragma unroll
    for (int f = 0; f < FM; ++f) {
        read_scales(0, 0, f);
        read_pair(0, 0, f);
        if (f < FN) sw[0][f] &= stages == 1 ? last_mask : -1;
        sx[0][f] &= stages == 1 ? last_mask : -1;
    }
    for (int s = 0; s < stages; ++s) {
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            if (i % 2 == 0) copy_codes(s + 1, 2 + i / 2);
            read_pair(s, 1, i);
            multiply(std::integral_constant<int, 0>{}, i);
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            read_pair(s, 2, i);
            multiply(std::integral_constant<int, 1>{}, i);
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            read_pair(s, 3, i);
            multiply(std::integral_constant<int, 2>{}, i);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // all of this stage is in registers
        wait_loads<0>();
        barrier();
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            if (i % 2 == 0) copy_codes(s + 2, i / 2);
            else copy_scales(s + 5, i / 2);  // a chunk's last quarter two stages before its first stage
            read_pair(s + 1, 0, i);
            read_scales(s + 1, 1, i);
            multiply(std::integral_constant<int, 3>{}, i);
        }
        const int mask = s + 2 == stages ? last_mask : -1;
#pragma unroll
        for (int f = 0; f < FM; ++f) {
            if (f < FN) sw[0][f] = sw[1][f] & mask;
            sx[0][f] = sx[1][f] & mask;
        }
    }
    wait_loads<0>();  // the copies past the last stage, which wrote zeros
    barrier();
    m0 += wm * 32 * FM;
    n0 += wn * 32 * FN;
    write_tile<FM, FN, TY>(acc, p, m0, n0, fast, lds + wave * (STAGE / 8));
}

// Few tiles, no more than CUs: 128 columns of y x 128 rows, or x 64 where those
// are still no more than CUs (of y, or of one part of a split sum), a workgroup,
// alone on its CU.  Two groups of four waves share each stage's products: group
// g takes steps 2 g and 2 g + 1, so every SIMD has two waves to alternate
// between, and the groups' sums meet in LDS at the end, each group finishing
// half of each wave's rows (2048 x 2048 x 8192: 26 us, 34 with the narrow kernel;
// 500 x 4096 x 4096 by 64 rows 12.0, by 128 13.5, narrow 17.6).  A fifth stage in
// LDS gained nothing: memory's latency is not what bounds it.  Nor are the two
// rates: of a stage's 0.45 us (64 rows) its products need 0.17 and its copies 0.24
// (24.5 KB of codes and 64 lines of scales at 134 GB/s a CU).  It is the chain
// from a stage's barrier over LDS reads, matrix instructions and the wait to the
// next, with two waves a SIMD to hide it.
//
// A stage is 256 values of K (whole cache lines, rows and slots as in the wide
// kernel); LDS holds four, used as by the narrow kernel: s is multiplied, s + 1
// is whole, s + 2 on its way, s + 3 requested.  Scales come in chunks of four
// stages, a quarter with each stage's copies, into three areas in turn.
template <int FM, typename TY>
__global__ __launch_bounds__(512, 1) void pair_kernel(MatmulParams p, Tiling order, bool fast) {
    constexpr int F = 2, B = 64 * F, BM = 64 * FM, STAGE = (B + BM) * 128, CHUNK = (B + BM) * 32;
    constexpr int LOADS = 3 + FM;  // a wave's copies in one stage
    __shared__ __attribute__((aligned(128))) uint8_t lds[4 * STAGE + 3 * CHUNK];
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = wave >> 2, wm = wave >> 1 & 1, wn = wave & 1;
    long long m0;
    int n0, split;
    tile_place<BM, B>(order, xcd_linear(blockIdx.x, gridDim.x), &m0, &n0, &split);
    const int first = split * order.split_stages / 2, stages = min(order.split_stages / 2, (p.kb + 7) / 8 - first);
    const long long rows_x = min(static_cast<long long>(BM), p.m - m0), rows_w = min(B, p.n - n0);
    const __amdgpu_buffer_rsrc_t gx = buffer(p.x + m0 * p.pitch, rows_x * p.pitch),
                                 gxs = buffer(p.xs + m0 * p.spitch, rows_x * p.spitch),
                                 gw = buffer(p.w + static_cast<long long>(n0) * p.pitch, rows_w * p.pitch),
                                 gws = buffer(p.ws + static_cast<long long>(n0) * p.spitch, rows_w * p.spitch);
    const uint32_t lds0 = static_cast<uint32_t>(
        reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds));

    // one copy: 8 rows' codes of a stage, or 8 rows' scales of a chunk
    const int copy_row = wave * 8 + (lane >> 3);
    const int copy_block = (lane & 7) ^ ((copy_row >> 1) & 7), copy_word = (lane & 7) ^ (2 * (wave & 3));
    const uint32_t copy_off = copy_row * p.pitch + copy_block * 16, copy_soff = copy_row * p.spitch + copy_word * 4;
    auto copy_stage = [&](int s, int i) {  // i-th of each operand's 2 copies of stage s
        const int stage = first + s;
        const uint32_t off = s < stages && stage * 8 + copy_block < p.kb ? copy_off + stage * 128 : kOutOfRange;
        const uint32_t to = lds0 + (s & 3) * STAGE + wave * 1024 + i * 8192;
        load_to_lds16(gw, off + i * 64 * p.pitch, to);
        if (i < FM) load_to_lds16(gx, off + i * 64 * p.pitch, to + B * 128);
    };
    auto copy_scales = [&](int part) {  // quarter part % 4 of chunk part / 4: 64 rows of w, or of x (64 rows in all: twice)
        const int chunk = part >> 2, of_x = part & 2, rows = of_x && FM == 1 ? 0 : (part & 1) * 64;
        const uint32_t off = (first * 2 + chunk * 8 + copy_word) * 4 < p.spitch ? copy_soff + (first * 2 + chunk * 8) * 4 : kOutOfRange;
        const uint32_t to = lds0 + 4 * STAGE + chunk % 3 * CHUNK + of_x / 2 * (B * 32) + rows * 32 + wave * 256;
        load_to_lds4(of_x ? gxs : gws, off + rows * p.spitch, to);
    };

    i32x4 a[2][F], b[2][FM];  // operands of two steps in turn
    int sw[2][F], sx[2][FM];  // scale words of a stage, and of the next
    const uint8_t* lw = lds + (wn * 32 * F + r) * 128;
    const uint8_t* lx = lds + (B + wm * 32 * FM + r) * 128;
    const uint8_t* lws = lds + 4 * STAGE + (wn * 32 * F + r) * 32;
    const uint8_t* lxs = lds + 4 * STAGE + (B + wm * 32 * FM + r) * 32;
    auto read_pair = [&](int s, int j, int f) {
        const int at = (s & 3) * STAGE + ((4 * h + 2 * half + j) ^ ((r >> 1) & 7)) * 16 + f * 4096;
        a[j][f] = *reinterpret_cast<const i32x4*>(lw + at);
        if (f < FM) b[j][f] = *reinterpret_cast<const i32x4*>(lx + at);
    };
    auto read_scales = [&](int s, int set, int f) {
        const int at = (s >> 2) % 3 * CHUNK + (((s & 3) * 2 + h) ^ (2 * (r >> 3))) * 4 + f * 1024;
        sw[set][f] = *reinterpret_cast<const int*>(lws + at);
        if (f < FM) sx[set][f] = *reinterpret_cast<const int*>(lxs + at);
    };
    float bias[F][16];
    load_bias(p, n0 + wn * 32 * F, bias);  // ahead of the output pass
    f32x16 acc[FM][F] = {};

#pragma unroll
    for (int q = 0; q < 4; ++q) copy_scales(q);
#pragma unroll
    for (int s = 0; s < 3; ++s) {
        copy_stage(s, 0);
        copy_stage(s, 1);
        if (s > 0) copy_scales(s + 3);
    }
    wait_loads<2 * LOADS>();
    barrier();
    // of this group's and half's scales in a row's last stage, which is in the last part
    const int row_stages = (p.kb + 7) / 8, last_bits = scale_bits(p.kb - (row_stages - 1) * 8 - 4 * h - 2 * half);
#pragma unroll
    for (int f = 0; f < F; ++f) {
        read_scales(0, 0, f);
        read_pair(0, 0, f);
    }
    for (int s = 0; s < stages; ++s) {
        wait_loads<LOADS>();  // this wave's copies for the next stage
        barrier();            // all waves'; and the stage before this one is no longer read
        const int bits = first + s == row_stages - 1 ? last_bits : 16;
#pragma unroll
        for (int f = 0; f < F; ++f) {
            sw[0][f] = __builtin_amdgcn_ubfe(sw[0][f], 16 * half, bits);
            if (f < FM) sx[0][f] = __builtin_amdgcn_ubfe(sx[0][f], 16 * half, bits);
        }
#pragma unroll
        for (int i = 0; i < F; ++i) {
            copy_stage(s + 3, i);
            read_pair(s, 1, i);
            if (i == F - 1) copy_scales(s + 6);
#pragma unroll
            for (int f = 0; f < (i < FM ? F : 0); ++f) acc[i][f] = mfma<0>(a[0][f], b[0][i], acc[i][f], sw[0][f], sx[0][i]);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < F; ++i) {
            read_pair(s + 1, 0, i);
            read_scales(s + 1, 1, i);
#pragma unroll
            for (int f = 0; f < (i < FM ? F : 0); ++f) acc[i][f] = mfma<1>(a[1][f], b[1][i], acc[i][f], sw[0][f], sx[0][i]);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int f = 0; f < F; ++f) {
            sw[0][f] = sw[1][f];
            if (f < FM) sx[0][f] = sx[1][f];
        }
    }
    wait_loads<0>();  // the copies past the last stage, which wrote zeros
    barrier();        // and no stage is read any more

    // this group keeps rows 32 half .. + 31 of its waves' 64 and hands the others over; of 32 rows group 0 keeps all
    float4* mine = reinterpret_cast<float4*>(lds + wave * 8192) + lane;
    const float4* theirs = reinterpret_cast<const float4*>(lds + (wave ^ 4) * 8192) + lane;
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const f32x16& v = half ? acc[0][f] : acc[FM - 1][f];
            mine[(f * 4 + g) * 64] = make_float4(v[g * 4], v[g * 4 + 1], v[g * 4 + 2], v[g * 4 + 3]);
        }
    __syncthreads();
    if (FM == 1 && half) return;
    f32x16 sum[1][F];
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const float4 t = theirs[(f * 4 + g) * 64];
            const f32x16& v = half ? acc[FM - 1][f] : acc[0][f];
            sum[0][f][g * 4] = v[g * 4] + t.x + bias[f][g * 4];
            sum[0][f][g * 4 + 1] = v[g * 4 + 1] + t.y + bias[f][g * 4 + 1];
            sum[0][f][g * 4 + 2] = v[g * 4 + 2] + t.z + bias[f][g * 4 + 2];
            sum[0][f][g * 4 + 3] = v[g * 4 + 3] + t.w + bias[f][g * 4 + 3];
        }
    m0 += wm * 32 * FM + half * 32;
    n0 += wn * 32 * F;
    MatmulParams out = p;
    if constexpr (std::is_same<TY, float>::value) out.y = static_cast<float*>(p.y) + split * p.m * p.ldy;
    write_tile<1, F, TY>(sum, out, m0, n0, fast, lds + 65536 + wave * 4096);
}

// The parts of a split sum, one behind the other -> y.  A thread owns 8 columns.
template <typename TY>
__global__ __launch_bounds__(256) void join_kernel(MatmulParams p, const float* __restrict__ parts, int splits,
                                                   Divisor per_row, uint32_t units) {
    const uint32_t u = blockIdx.x * 256u + threadIdx.x;
    if (u >= units) return;  // for MXFP4 units is a multiple of 4: whole blocks leave
    const uint32_t row = divide(u, per_row);
    const int n = static_cast<int>(u - row * per_row.d) * 8, valid = p.n - n;
    const float* at = parts + static_cast<long long>(row) * p.ldy + n;
    float v[8], t[8];
    load8(at, valid, v);
    for (int q = 1; q < splits; ++q) {
        load8(at + q * p.m * p.ldy, valid, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += t[i];
    }
    if (p.bias) {
        load8(p.bias + n, valid, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += t[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = activate<TY>(v[i], p.act);
    store_run<TY>(p, row, n, valid, v);
}

// rows of y are whole 16-byte runs, and a wave's rows within a buffer's 31 bits
template <typename TY>
bool whole_runs(const MatmulParams& p) {
    constexpr int ES = std::is_same<TY, float>::value ? 4 : 2;
    return std::is_void<TY>::value ||
           (p.ldy * ES % 16 == 0 && reinterpret_cast<uintptr_t>(p.y) % 16 == 0 && p.n <= (1 << 21));
}

template <typename TY>
void launch_tiles(const MatmulParams& p, bool wide, int splits, int cus, hipStream_t st) {
    const int side = wide ? 256 : 128;
    const bool low = !wide && (p.m + 63) / 64 * ((p.n + 127) / 128) * splits <= cus;  // tiles of 64 rows
    const int tiles_m = static_cast<int>(low ? (p.m + 63) / 64 : (p.m + side - 1) / side), tiles_n = (p.n + side - 1) / side;
    const int stages = (p.kb + 3) / 4;  // of 128 values; a part has a whole number of chunks of four of 256
    const int split_stages = splits > 1 ? (stages + 8 * splits - 1) / (8 * splits) * 8 : (stages + 1) / 2 * 2;
    const int parts = (stages + split_stages - 1) / split_stages;
    const Tiling order{tiles_m, tiles_n, split_stages, divisor(tiles_m * tiles_n), divisor(8u * tiles_n),
                       divisor(8), divisor((tiles_m - 1) % 8 + 1)};
    const int tiles = tiles_m * tiles_n * parts;
    const bool fast = whole_runs<TY>(p);
    if (wide)
        wide_kernel<TY><<<static_cast<unsigned>(tiles), 512, 0, st>>>(p, order, fast);
    else if (low)
        pair_kernel<1, TY><<<static_cast<unsigned>(tiles), 512, 0, st>>>(p, order, fast);
    else if (tiles <= cus)
        pair_kernel<2, TY><<<static_cast<unsigned>(tiles), 512, 0, st>>>(p, order, fast);
    else
        tile_kernel<TY><<<static_cast<unsigned>(tiles < 2 * cus ? tiles : 2 * cus), 256, 0, st>>>(p, order, fast);
}

template <int S, typename TY>
void launch_rows(const MatmulParams& p, int cus, hipStream_t st) {
    const int tiles_n = (p.n + 127) / 128;
    const long long tiles = (p.m + 127) / 128 * tiles_n;
    rows_kernel<S, TY><<<static_cast<unsigned>(std::min<long long>(tiles, (Resident<S, TY>::kThree ? 3 : 2) * cus)), 256, 0, st>>>(
        p, tiles_n, tiles, whole_runs<TY>(p));
}

// A split sum: parts in fp32 to `work`, then the joining pass.
void launch_split(const MatmulParams& p, cfwd_dtype y, int splits, int cus, float* work, hipStream_t st) {
    const int stages = (p.kb + 3) / 4, split_stages = (stages + 8 * splits - 1) / (8 * splits) * 8;
    const int parts = (stages + split_stages - 1) / split_stages;
    MatmulParams q = p;
    q.bias = nullptr;
    q.act = CFWD_ACT_NONE;
    q.y = work;
    q.ldy = (p.n + 3) / 4 * 4;
    launch_tiles<float>(q, false, splits, cus, st);
    q = p;
    q.ldy = (p.n + 3) / 4 * 4;
    const Divisor per_row = divisor(y == CFWD_MXFP4 ? p.y_pitch / 4 : (p.n + 7) / 8);
    const uint32_t units = static_cast<uint32_t>(p.m) * per_row.d, grid = (units + 255) / 256;
    if (y == CFWD_F32)
        join_kernel<float><<<grid, 256, 0, st>>>(q, work, parts, per_row, units);
    else if (y == CFWD_BF16)
        join_kernel<bf16_t><<<grid, 256, 0, st>>>(q, work, parts, per_row, units);
    else
        join_kernel<void><<<grid, 256, 0, st>>>(q, work, parts, per_row, units);
}

}  // namespace mx

int compute_units() {
    static PerDevice known;
    return static_cast<int>(known.get(
        [](int dev) {
            int n = 0;
            return hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess ? n : 0;
        },
        256));
}

namespace {

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

// How a product of more rows than the stream kernel takes is cut up: wide
// tiles or not, and parts of the sum over K.
struct Choice {
    bool wide;
    int splits;
    bool rows = false;  // x stays in LDS
};

// Sums of up to 512 values over more tiles than CUs go to the rows kernel, which
// was the fastest at every size (narrow, it and wide: 100352 x 128 x 256 13.3,
// 10.7 and 23 us; 2100 x 2048 x 512 8.7, 7.3 and 13; 8192 x 8192 x 512 48, 38 and
// 53).  Else the cheapest by a model of the time, in us, fitted to measurements
// over sums of 2 to 128 stages and 8 to 6000 tiles: a round of tiles takes its
// stages and an output pass; 128-wide tiles share a CU by twos, or have one to
// themselves (narrow and wide: 8192 x 8192 x 8192 420 and 254 us; x 1024: 76 and
// 60; 2500 x 2900 x 1024: 13 and 15).  A split sum pays for its parts' traffic and a second launch (128 x 1024 x
// 16384: 27 us whole, 16 in 8 parts; 500 x 4096 x 4096: 12 and 24 in 2).
Choice choose(const cfwd_mx_matmul_desc* d, int cus) {
    const double stages = static_cast<double>((mx_blocks(d->k) + 3) / 4);
    const long long t2 = (d->m + 127) / 128 * ((d->n + 127) / 128), t4 = (d->m + 255) / 256 * ((d->n + 255) / 256);
    if (stages <= 4 && t2 > cus) return {false, 1, true};
    auto rounds = [](long long tiles, long long slots) { return static_cast<double>((tiles + slots - 1) / slots); };
    const double alone = 0.22, shared = 0.9, wide = 0.86;  // us for 128 values of K
    double best = t2 <= cus ? stages * alone + 2 : rounds(t2, 2 * cus) * (stages * shared + 3.4);
    Choice c{false, 1};
    const double four = rounds(t4, cus) * (stages * wide + 8);
    if (four < best) {
        best = four;
        c = {true, 1};
    }
    for (int s = 2; s <= 8 && t2 * s <= cus && stages >= 8 * s; s *= 2) {
        const double split = stages / s * alone + 2 + 4 + static_cast<double>(d->m) * d->n * 8 * s / 4e6;
        if (split < best) {
            best = split;
            c = {false, s};
        }
    }
    return c;
}

size_t x_bytes(const cfwd_mx_matmul_desc* d) {  // of an x that the call quantises
    return round256(static_cast<size_t>(d->m) * mx_code_pitch(d->k)) + round256(static_cast<size_t>(d->m) * mx_scale_pitch(d->k));
}

}  // namespace

size_t mx_matmul_workspace(const cfwd_mx_matmul_desc* d) {
    if (mx_stream_supported(d->m, d->n, d->k)) return d->x_dtype == CFWD_MXFP4 || mx_stream_takes_raw(d) ? 0 : x_bytes(d);
    const Choice c = choose(d, compute_units());
    const size_t x = d->x_dtype == CFWD_MXFP4 ? 0 : x_bytes(d);
    return x + (c.splits > 1 ? static_cast<size_t>(c.splits) * d->m * ((d->n + 3) / 4 * 4) * 4 : 0);
}

cfwd_status mx_matmul(const cfwd_mx_matmul_desc* d, const void* x, const void* x_scales, const void* w,
                      const void* w_scales, const float* bias, void* y, void* y_scales, void* workspace,
                      hipStream_t st) {
    mx::MatmulParams p{};
    uint8_t* work = static_cast<uint8_t*>(workspace);
    const bool stream = mx_stream_supported(d->m, d->n, d->k);
    const int cus = compute_units();
    const Choice c = stream ? Choice{} : choose(d, cus);
    const bool raw = d->x_dtype != CFWD_MXFP4 && stream && mx_stream_takes_raw(d);
    if (d->x_dtype != CFWD_MXFP4 && !raw) {
        uint8_t* scales = work + round256(static_cast<size_t>(d->m) * mx_code_pitch(d->k));
        const cfwd_status s = mx_quantize(d->m, d->k, d->x_dtype, x, d->x_stride, work, scales, st);
        if (s != CFWD_OK) return s;
        x = work;
        x_scales = scales;
        work += x_bytes(d);
    }
    p.x = static_cast<const uint8_t*>(x);
    p.xs = static_cast<const uint8_t*>(x_scales);
    p.w = static_cast<const uint8_t*>(w);
    p.ws = static_cast<const uint8_t*>(w_scales);
    p.bias = bias;
    p.y = y;
    p.ys = static_cast<uint8_t*>(y_scales);
    p.m = d->m;
    p.n = d->n;
    p.ldy = d->n;
    p.kb = static_cast<int>(mx_blocks(d->k));
    p.pitch = static_cast<int>(mx_code_pitch(d->k));
    p.spitch = static_cast<int>(mx_scale_pitch(d->k));
    p.x_stride = d->x_stride;
    p.k = d->k;
    p.act = d->act;
    p.y_pitch = static_cast<int>(mx_code_pitch(d->n));
    p.y_spitch = static_cast<int>(mx_scale_pitch(d->n));
    if (stream) return mx_stream(p, raw ? d->x_dtype : CFWD_MXFP4, d->y_dtype, cus, st);
    const bool half = p.kb <= 8;  // of what the rows kernel can hold
    if (c.rows && d->y_dtype == CFWD_F32)
        half ? mx::launch_rows<2, float>(p, cus, st) : mx::launch_rows<4, float>(p, cus, st);
    else if (c.rows && d->y_dtype == CFWD_BF16)
        half ? mx::launch_rows<2, bf16_t>(p, cus, st) : mx::launch_rows<4, bf16_t>(p, cus, st);
    else if (c.rows)
        half ? mx::launch_rows<2, void>(p, cus, st) : mx::launch_rows<4, void>(p, cus, st);
    else if (c.splits > 1)
        mx::launch_split(p, d->y_dtype, c.splits, cus, reinterpret_cast<float*>(work), st);
    else if (d->y_dtype == CFWD_F32)
        mx::launch_tiles<float>(p, c.wide, 1, cus, st);
    else if (d->y_dtype == CFWD_BF16)
        mx::launch_tiles<bf16_t>(p, c.wide, 1, cus, st);
    else
        mx::launch_tiles<void>(p, c.wide, 1, cus, st);
    return check_hip(hipGetLastError(), "MXFP4 product launch");
}

}  // namespace cfwd

// Product of two MXFP4 matrices (gfx950): y = act(x w^T + bias).
#include "mx_matmul_impl.h"

#include <algorithm>
#include <cstdlib>
#include <type_traits>

namespace cfwd {
namespace mx {

// Copies 16 (or 4) bytes a lane from a buffer straight to LDS, lane after lane
// from `lds` on (wave-uniform); out-of-range lanes write 0.  The compiler does
// not see these loads: wait_loads() and a barrier come before the data are read.
__device__ __forceinline__ void load_to_lds16(const __amdgpu_buffer_rsrc_t& b, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(off), "s"(b)
                 : "memory");
}
__device__ __forceinline__ void load_to_lds4(const __amdgpu_buffer_rsrc_t& b, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(off), "s"(b)
                 : "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads() {  // until at most N of this wave's loads are outstanding
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// All waves of the workgroup; what memory accesses the code has before and after stays there.
__device__ __forceinline__ void barrier() { asm volatile("s_barrier" ::: "memory"); }

// Tiles through LDS.  A tile is 64 F rows of y x 64 F columns; the four waves
// (2 x 2) of a workgroup take 32 F x 32 F of it each.  With F = 2 the grid is
// what fits the device at once, and each workgroup works through several tiles
// as one unbroken run of stages of 128 values of K, so that a tile's output
// pass finds the next tile's operands on their way.  With F = 4, for long sums,
// a workgroup has one tile: its 256 accumulators leave no registers in which
// the next operands could outlast the output pass.
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
// (8192^3: 368 us so, 306 us without any scale copies).
//
// A stage's row is 64 bytes, four blocks, of which half h of a wave takes
// blocks 2 h and 2 h + 1; block b of row i lies in slot b ^ ((i >> 1) & 3), so
// that the 16-byte reads of consecutive rows spread over all banks.  The copy
// to LDS is linear in lanes, so the permutation is made in the addresses that
// the lanes load from.
//
// The output pass of the tile uses the LDS of the stage multiplied last, which
// is filled again only after the next stage's barrier.
template <int F, typename TY>
__global__ __launch_bounds__(256, F > 2 ? 1 : 2) void tile_kernel(MatmulParams p, int tiles_m, int tiles_n, bool fast) {
    static_assert(F == 2 || F == 4, "the copies below are laid out for these");
    constexpr int B = 64 * F, STAGE = 2 * B * 64, GROUP = 2 * B * 16;
    constexpr int CODE_LOADS = 2 * F, SCALE_LOADS = 2 * F;  // a wave's copies for a stage, for a group
    constexpr int STORES = stores<F, F, TY>();
    __shared__ __attribute__((aligned(128))) uint8_t lds[4 * STAGE + 4 * GROUP];
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;

    // The i-th tile of this workgroup.  A round of tiles is a run of the tiles'
    // order, each XCD a run within it; the order goes down columns of 8 tiles.
    const int tiles = tiles_m * tiles_n;
    const int rounds = F > 2 ? 1 : (tiles - 1 - static_cast<int>(blockIdx.x)) / static_cast<int>(gridDim.x) + 1;
    auto tile_at = [&](int i, long long* m0, int* n0) {
        const int first = i * gridDim.x;
        const int t = first + xcd_linear(blockIdx.x, min(static_cast<int>(gridDim.x), tiles - first));
        const int group = t / (8 * tiles_n), in_group = t % (8 * tiles_n), height = min(8, tiles_m - group * 8);
        *m0 = static_cast<long long>(group * 8 + in_group % height) * B;
        *n0 = in_group / height * B;
    };

    const int stages = (p.kb + 3) / 4;
    const uint32_t lds0 = static_cast<uint32_t>(
        reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds));
    // copying: tile number, stage of the tile, stage and group of all
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
        gx = buffer(p.x + m0 * p.pitch, rows_x * p.pitch);
        gxs = buffer(p.xs + m0 * p.spitch, rows_x * p.spitch);
        gw = buffer(p.w + static_cast<long long>(n0) * p.pitch, rows_w * p.pitch);
        gws = buffer(p.ws + static_cast<long long>(n0) * p.spitch, rows_w * p.spitch);
    };
    // one copy: 16 rows' codes of a stage, or 16 rows' scales of a group
    const int copy_block = (lane & 3) ^ ((lane >> 3) & 3);
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
            copy_stage = 0;
            ++copy_tile;
            open_tile();
        }
    };

    // fragments of one matrix instruction's depth, two sets in turn; scale words of a stage
    i32x4 a[2][F], b[2][F];
    int sw[2][F], sx[2][F];
    const int swz = (r >> 1) & 3;
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

    f32x16 acc[F][F] = {};
    int count = 0, group = 0;  // of the stage that is multiplied, among all
    int since = 2;             // stages since the last output pass
    for (int tile = 0; tile < rounds; ++tile) {
        long long m0;
        int n0;
        tile_at(tile, &m0, &n0);
        m0 += wm * 32 * F;
        n0 += wn * 32 * F;
        float bias[F > 2 ? 1 : F][16];
        if constexpr (F == 2)  // requested ahead of the output pass; wider tiles have no registers for that
            if (p.bias) {
#pragma unroll
                for (int f = 0; f < F; ++f) load_bias(p, n0 + f * 32, bias[f]);
            }
        for (int stage = 0; stage < stages; ++stage, ++count, ++since) {
            // This wave's copies for the next stage: later ones, and stores, may be outstanding.
            if (since < 2) {
                if (had_scales) wait_loads<(CODE_LOADS + SCALE_LOADS + STORES < 63 ? CODE_LOADS + SCALE_LOADS + STORES : 63)>();
                else wait_loads<(CODE_LOADS + STORES < 63 ? CODE_LOADS + STORES : 63)>();
            } else {
                if (had_scales) wait_loads<CODE_LOADS + SCALE_LOADS>();
                else wait_loads<CODE_LOADS>();
            }
            barrier();  // all waves' copies for it; and the stage before this one is no longer read
#pragma unroll
            for (int f = 0; f < F; ++f) {
                sw[0][f] >>= 16 * h;
                sx[0][f] >>= 16 * h;
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
        auto add_bias = [&](int f, float(&v)[16]) {
            if (!p.bias) return;
            if constexpr (F > 2) load_bias(p, n0 + f * 32, bias[0]);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] += bias[F > 2 ? 0 : f][j];
        };
        write_tile<F, F, TY>(acc, add_bias, p, m0, n0, fast, lds + ((count - 1) & 3) * STAGE + wave * (STAGE / 4));
        if (!fast) wait_loads<0>();  // an unknown number of stores
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int f = 0; f < F; ++f) acc[i][f] = f32x16{};
        since = 0;
    }
    wait_loads<0>();  // no copy may reach LDS after the workgroup has ended
}

template <int F>
void launch_tiles(const MatmulParams& p, cfwd_dtype y, int cus, hipStream_t st) {
    const int tiles_m = static_cast<int>((p.m + 64 * F - 1) / (64 * F)), tiles_n = (p.n + 64 * F - 1) / (64 * F);
    const unsigned grid = static_cast<unsigned>(F > 2 || tiles_m * tiles_n < 2 * cus ? tiles_m * tiles_n : 2 * cus);
    // whole 16-byte runs, and a wave's rows within a buffer's 31 bits
    const int es = y == CFWD_F32 ? 4 : 2;
    const bool fast = y == CFWD_MXFP4 || (p.n * es % 16 == 0 && reinterpret_cast<uintptr_t>(p.y) % 16 == 0 && p.n <= (1 << 21));
    if (y == CFWD_F32)
        tile_kernel<F, float><<<grid, 256, 0, st>>>(p, tiles_m, tiles_n, fast);
    else if (y == CFWD_BF16)
        tile_kernel<F, bf16_t><<<grid, 256, 0, st>>>(p, tiles_m, tiles_n, fast);
    else
        tile_kernel<F, void><<<grid, 256, 0, st>>>(p, tiles_m, tiles_n, fast);
}

}  // namespace mx

namespace {
size_t round256(size_t v) { return (v + 255) / 256 * 256; }
}  // namespace

size_t mx_matmul_workspace(const cfwd_mx_matmul_desc* d) {
    if (d->x_dtype == CFWD_MXFP4 || (mx_stream_supported(d->m) && mx_stream_takes_raw(d->m, d->k))) return 0;
    return round256(static_cast<size_t>(d->m) * mx_code_pitch(d->k)) + round256(static_cast<size_t>(d->m) * mx_scale_pitch(d->k));
}

cfwd_status mx_matmul(const cfwd_mx_matmul_desc* d, const void* x, const void* x_scales, const void* w,
                      const void* w_scales, const float* bias, void* y, void* y_scales, void* workspace,
                      hipStream_t st) {
    mx::MatmulParams p{};
    const bool stream = mx_stream_supported(d->m);
    const bool raw = d->x_dtype != CFWD_MXFP4 && stream && mx_stream_takes_raw(d->m, d->k);
    if (d->x_dtype != CFWD_MXFP4 && !raw) {
        uint8_t* codes = static_cast<uint8_t*>(workspace);
        uint8_t* scales = codes + round256(static_cast<size_t>(d->m) * mx_code_pitch(d->k));
        const cfwd_status s = mx_quantize(d->m, d->k, d->x_dtype, x, d->x_stride, codes, scales, st);
        if (s != CFWD_OK) return s;
        x = codes;
        x_scales = scales;
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
    p.kb = static_cast<int>(mx_blocks(d->k));
    p.pitch = static_cast<int>(mx_code_pitch(d->k));
    p.spitch = static_cast<int>(mx_scale_pitch(d->k));
    p.x_stride = d->x_stride;
    p.k = d->k;
    p.act = d->act;
    p.y_pitch = static_cast<int>(mx_code_pitch(d->n));
    p.y_spitch = static_cast<int>(mx_scale_pitch(d->n));
    if (stream) return mx_stream(p, raw ? d->x_dtype : CFWD_MXFP4, d->y_dtype, st);
    const int cus = 256;
    const char* force = getenv("MXT");
    if (force ? atoi(force) == 44 : ((d->m + 255) / 256 * ((d->n + 255) / 256) >= 256))
        mx::launch_tiles<4>(p, d->y_dtype, cus, st);
    else
        mx::launch_tiles<2>(p, d->y_dtype, cus, st);
    return check_hip(hipGetLastError(), "MXFP4 product launch");
}

}  // namespace cfwd

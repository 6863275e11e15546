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

// Tiles through LDS.  A workgroup owns 64 FM rows of y x 64 FN columns, its
// four waves (2 x 2) 32 FM x 32 FN each.
//
// LDS holds four stages of 128 values of K in turn.  While stage s is
// multiplied, s + 1 is whole, s + 2 is on its way and s + 3 is requested, so
// the operands of the next matrix instructions are always read from LDS ahead
// of their use, across stages too, and a memory latency has two stages to pass.
// Requests past the last stage are made all the same (they load nothing and
// write zeros), so that the count of outstanding loads is known.
//
// Scales come four stages ("a group") at a time, so that a 16-byte run of each
// row is read at once: a word at a time costs a cache line for every word
// (8192^3: 368 us so, 306 us without any scale copies).  A group's copies are
// spread over four stages, the last of them three stages before the group's
// first, into three areas in turn.
//
// A stage's row is 64 bytes, four blocks, of which half h of a wave takes
// blocks 2 h and 2 h + 1; block b of row i lies in slot b ^ ((i >> 1) & 3), so
// that the 16-byte reads of consecutive rows spread over all banks.  The copy
// to LDS is linear in lanes, so the permutation is made in the addresses that
// the lanes load from.
template <int FM, int FN, typename TY>
__global__ __launch_bounds__(256, FM * FN > 8 ? 1 : 2) void tile_kernel(MatmulParams p) {
    static_assert(FM == FN && (FM == 2 || FM == 4), "the copies below are laid out for square tiles");
    constexpr int BM = 64 * FM, BN = 64 * FN, STAGE = (BM + BN) * 64, GROUP = (BM + BN) * 16;
    constexpr int LOADS = 2 * FN + FN / 2;  // a wave's copies in one stage
    constexpr int OUT = out_area<FN, TY>();
    constexpr int LDS = 4 * STAGE + 3 * GROUP;
    static_assert(LDS >= 4 * OUT, "the output areas overlay the stages");
    __shared__ __attribute__((aligned(128))) uint8_t lds[LDS];
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;

    // order of tiles: each XCD a run of them; within a run, columns of 8 tiles of y's rows
    const int tiles_n = (p.n + BN - 1) / BN, tiles_m = static_cast<int>((p.m + BM - 1) / BM);
    const int t = xcd_linear(blockIdx.x, gridDim.x);
    const int group = t / (8 * tiles_n), in_group = t % (8 * tiles_n), height = min(8, tiles_m - group * 8);
    const long long m0 = static_cast<long long>(group * 8 + in_group % height) * BM;
    const int n0 = in_group / height * BN;

    const long long rows_x = min(static_cast<long long>(BM), p.m - m0);
    const int rows_w = min(BN, p.n - n0);
    const __amdgpu_buffer_rsrc_t gx = buffer(p.x + m0 * p.pitch, rows_x * p.pitch),
                                 gxs = buffer(p.xs + m0 * p.spitch, rows_x * p.spitch),
                                 gw = buffer(p.w + static_cast<long long>(n0) * p.pitch, static_cast<long long>(rows_w) * p.pitch),
                                 gws = buffer(p.ws + static_cast<long long>(n0) * p.spitch, static_cast<long long>(rows_w) * p.spitch);
    const uint32_t lds0 = static_cast<uint32_t>(
        reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds));

    // one copy: 16 rows' codes of a stage, or 16 rows' scales of a group
    const int copy_block = (lane & 3) ^ ((lane >> 3) & 3);
    const uint32_t copy_off = (wave * 16 + (lane >> 2)) * p.pitch + copy_block * 16;
    const uint32_t copy_soff = (wave * 16 + (lane >> 2)) * p.spitch + (lane & 3) * 4;
    auto codes_off = [&](int stage) { return stage * 4 + copy_block < p.kb ? copy_off + stage * 64 : kOutOfRange; };
    auto copy_codes = [&](int stage, uint32_t off, int i) {  // i-th of each operand's FN copies
        const uint32_t to = lds0 + (stage & 3) * STAGE + wave * 1024 + i * 4096;
        load_to_lds16(gw, off + i * 64 * p.pitch, to);
        load_to_lds16(gx, off + i * 64 * p.pitch, to + BN * 64);
    };
    auto copy_scales = [&](int part) {  // quarter part % 4 of group part / 4: half the rows of w, or of x
        const int group = part >> 2, word = group * 4 + (lane & 3), half = (part & 1) * 32 * FN;
        const uint32_t to = lds0 + 4 * STAGE + group % 3 * GROUP + ((part & 2 ? BN : 0) + half + wave * 16) * 16;
        const uint32_t off = word * 4 < p.spitch ? copy_soff + half * p.spitch + group * 16 : kOutOfRange;
#pragma unroll
        for (int i = 0; i < FN / 2; ++i) load_to_lds4(part & 2 ? gxs : gws, off + i * 64 * p.spitch, to + i * 1024);
    };

    // fragments of one matrix instruction's depth, two sets in turn; scale words of a stage, shifted to this half's bytes
    i32x4 a[2][FN], b[2][FM];
    int sw[2][FN], sx[2][FM];
    const int swz = (r >> 1) & 3;
    const uint8_t* lw = lds + (wn * 32 * FN + r) * 64;
    const uint8_t* lx = lds + BN * 64 + (wm * 32 * FM + r) * 64;
    const uint8_t* lws = lds + 4 * STAGE + (wn * 32 * FN + r) * 16;
    const uint8_t* lxs = lds + 4 * STAGE + (BN + wm * 32 * FM + r) * 16;
    auto read_pair = [&](int stage, int j, int set, int f) {
        const int at = (stage & 3) * STAGE + ((2 * h + j) ^ swz) * 16 + f * 2048;
        a[set][f] = *reinterpret_cast<const i32x4*>(lw + at);
        b[set][f] = *reinterpret_cast<const i32x4*>(lx + at);
    };
    auto read_scales = [&](int stage, int set, int f) {
        const int at = (stage >> 2) % 3 * GROUP + (stage & 3) * 4 + f * 512;
        sw[set][f] = *reinterpret_cast<const int*>(lws + at);
        sx[set][f] = *reinterpret_cast<const int*>(lxs + at);
    };

    f32x16 acc[FM][FN] = {};
    const int stages = (p.kb + 3) / 4;
#pragma unroll
    for (int q = 0; q < 4; ++q) copy_scales(q);
#pragma unroll
    for (int s = 0; s < 3; ++s) {
        const uint32_t off = codes_off(s);
#pragma unroll
        for (int i = 0; i < FN; ++i) copy_codes(s, off, i);
        if (s > 0) copy_scales(s + 3);
    }
    wait_loads<2 * LOADS>();
    barrier();
#pragma unroll
    for (int f = 0; f < FN; ++f) {
        read_scales(0, 0, f);
        read_pair(0, 0, 0, f);
    }
    for (int s = 0; s < stages; ++s) {
        wait_loads<LOADS>();           // stage s + 1 of this wave's copies
        barrier();  // of all waves'; and stage s - 1 is no longer read
        const uint32_t off = codes_off(s + 3);
#pragma unroll
        for (int f = 0; f < FN; ++f) {
            sw[0][f] >>= 16 * h;
            sx[0][f] >>= 16 * h;
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            copy_codes(s + 3, off, i);
            read_pair(s, 1, 1, i);
            if (i == FM - 1) copy_scales(s + 6);
#pragma unroll
            for (int f = 0; f < FN; ++f) acc[i][f] = mfma<0>(a[0][f], b[0][i], acc[i][f], sw[0][f], sx[0][i]);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            read_pair(s + 1, 0, 0, i);
            read_scales(s + 1, 1, i);
#pragma unroll
            for (int f = 0; f < FN; ++f) acc[i][f] = mfma<1>(a[1][f], b[1][i], acc[i][f], sw[0][f], sx[0][i]);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int f = 0; f < FN; ++f) {
            sw[0][f] = sw[1][f];
            sx[0][f] = sx[1][f];
        }
    }
    wait_loads<0>();
    __syncthreads();  // the output areas overlay the stages
#pragma unroll
    for (int i = 0; i < FM; ++i)
        write_rows<FN, TY>(acc[i], p, m0 + wm * 32 * FM + i * 32, n0 + wn * 32 * FN, lds + wave * OUT);
}

template <int FM, int FN>
void launch_tiles(const MatmulParams& p, cfwd_dtype y, hipStream_t st) {
    const unsigned grid = static_cast<unsigned>((p.m + 64 * FM - 1) / (64 * FM) * ((p.n + 64 * FN - 1) / (64 * FN)));
    if (y == CFWD_F32)
        tile_kernel<FM, FN, float><<<grid, 256, 0, st>>>(p);
    else if (y == CFWD_BF16)
        tile_kernel<FM, FN, bf16_t><<<grid, 256, 0, st>>>(p);
    else
        tile_kernel<FM, FN, void><<<grid, 256, 0, st>>>(p);
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
    const char* force = getenv("MXT");
    if (force ? atoi(force) == 44 : ((d->m + 255) / 256 * ((d->n + 255) / 256) >= 256))
        mx::launch_tiles<4, 4>(p, d->y_dtype, st);
    else
        mx::launch_tiles<2, 2>(p, d->y_dtype, st);
    return check_hip(hipGetLastError(), "MXFP4 product launch");
}

}  // namespace cfwd

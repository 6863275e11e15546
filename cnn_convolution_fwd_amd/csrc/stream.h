// Loads that leave the caches to other data.
//
// A pass that reads and writes more than the 256 MB Infinity Cache can keep does better when what it reads passes by and
// what it writes stays for the kernel after it.  Measured (bf16, heads of 128): rotary positions at 123 MB in all 26 us
// against 22 with plain loads, at 168 MB 32 against 31 and with attention over the result 86 against 91, at 257 MB 46
// against 54; writing the paged cache at 85 MB 20 against 19, at 170 MB and read back 65 against 76.
#pragma once

#include "mx.h"

namespace cfwd {
namespace mx {

constexpr long long kStreamBytes = 150000000;  // read and written

typedef uint32_t u32x4_once_t __attribute__((ext_vector_type(4), aligned(2)));

// load8 (mx.h); ONCE: of values that no one reads again.
template <bool ONCE, typename T>
__device__ __forceinline__ void load8(const T* p, int valid, float (&v)[8]) {
    if (!ONCE || valid < 8) return load8(p, valid, v);
    constexpr int n = sizeof(T) / 2;
    uint32_t w[4 * n];
#pragma unroll
    for (int i = 0; i < n; ++i) {
        const u32x4_once_t a = __builtin_nontemporal_load(reinterpret_cast<const u32x4_once_t*>(p) + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * i + j] = a[j];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = __uint_as_float(n == 2 ? w[i * n / 2] : i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
}

}  // namespace mx
}  // namespace cfwd

// Host entry points behind the attention section of cfwd.h (k_rope.hip,
// k_mx_cache.hip, k_mx_decode.hip, k_attention.hip).  Arguments are checked by the
// caller (capi_attention.cpp).
#pragma once

#include "internal.h"

namespace cfwd {

cfwd_status rope(const cfwd_rope_desc* d, const void* q, const void* k, const void* positions,
                 const cfwd_rope_pair* table, void* q_out, void* k_out, hipStream_t st);

cfwd_status mx_cache_write(const cfwd_mx_cache_write_desc* d, const cfwd_mx_cache* c, const void* k, const void* v,
                           const void* slots, hipStream_t st);
cfwd_status mx_cache_read(const cfwd_mx_cache_read_desc* d, const cfwd_mx_cache* c, const int32_t* table,
                          const int32_t* starts, void* k, void* v, hipStream_t st);

size_t mx_cache_attention_workspace(const cfwd_mx_cache_attention_desc* d, const cfwd_mx_cache* c);
cfwd_status mx_cache_attention(const cfwd_mx_cache_attention_desc* d, const cfwd_mx_cache* c, const void* q,
                               const int32_t* table, const int32_t* lengths, void* o, void* workspace, hipStream_t st);

size_t attention_workspace(const cfwd_attention_desc* d);
cfwd_status attention(const cfwd_attention_desc* d, const void* q, const void* k, const void* v, const int32_t* q_starts,
                      const int32_t* k_starts, void* o, void* workspace, hipStream_t st);

#if defined(__HIPCC__)
// Sum over the lanes of a wave up to and with this one, by moves within the vector unit (a shuffle goes through LDS).
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // from 1, 2, 4, 8 lanes before, in rows of 16
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // rows 1 and 3: the last lane of the row before
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // rows 2 and 3: the last lane of row 1
    return v;
}

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
#endif

}  // namespace cfwd

// Device helpers of the multi-adapter kernels (gfx950).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qn {

typedef short s16x4 __attribute__((ext_vector_type(4)));

// ds_read_b64_tr_b16: in each group of 16 lanes, lane 4 r + b gives the address of row r,
// columns 4 b .. 4 b + 3 of a 4 x 16 block of 16-bit entries; lane p of the group receives
// column p's 4 rows.
static __device__ __forceinline__ uint2 lds_tr4(const void* p) {
    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (__attribute__((address_space(3))) s16x4*)(const_cast<void*>(p))));
}

// The lane's MFMA fragment of 8 consecutive rows k .. k + 7 of one column: `p` is its address
// for the first 4 rows, `four` the bytes of 4 rows.
static __device__ __forceinline__ uint4 lds_tr8(const char* p, int four) {
    const uint2 a = lds_tr4(p), b = lds_tr4(p + four);
    return uint4{a.x, a.y, b.x, b.y};
}

}  // namespace qn

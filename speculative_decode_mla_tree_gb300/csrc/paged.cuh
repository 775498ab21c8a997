// What the paged decode kernels share.
#pragma once
#include "mt_common.cuh"
#include "paged.h"

namespace mt {

// Writes four heads of 32 dims: lane l holds dim l, v its heads. Two exchanges
// among four lanes turn that into four dims of one head a lane (8 bytes, 64 per
// head and warp), lane l taking head l % 4. out: element (first head, first
// dim), rows of 512; n: heads to write (1 to 4, or more).
__device__ __forceinline__ void store_heads4(uint16_t* out, int lane, const float (&v)[4], int n) {
  const __nv_bfloat162 a2 = __floats2bfloat162_rn(v[0], v[1]), b2 = __floats2bfloat162_rn(v[2], v[3]);
  const uint32_t a = *reinterpret_cast<const uint32_t*>(&a2), b = *reinterpret_cast<const uint32_t*>(&b2);
  const uint32_t oa = __shfl_xor_sync(0xffffffffu, a, 1), ob = __shfl_xor_sync(0xffffffffu, b, 1);
  // even lanes: heads 0 and 2 of dims (l, l + 1); odd lanes: heads 1 and 3 of dims (l - 1, l)
  const bool odd = lane & 1, upper = lane & 2;
  const uint32_t x = odd ? __byte_perm(oa, a, 0x7632) : __byte_perm(a, oa, 0x5410);
  const uint32_t y = odd ? __byte_perm(ob, b, 0x7632) : __byte_perm(b, ob, 0x5410);
  const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? x : y, 2);
  const uint2 w = upper ? make_uint2(got, y) : make_uint2(x, got);
  if ((lane & 3) < n) *reinterpret_cast<uint2*>(out + (lane & 3) * kDv + (lane & ~3)) = w;
}

}  // namespace mt

// Arithmetic shared by the tensor-core attention kernels: fp16 key operands and
// the softmax's 2^x on the FMA pipe.
#pragma once
#include <cuda_fp16.h>
#include <stdint.h>

#include "ptx.cuh"

namespace la {

using namespace ptx;

// bf16 pair + fp32 pair, rounded once to an fp16 pair (the K^a operand)
__device__ __forceinline__ uint32_t add_to_f16x2(uint32_t base_bf16x2, float2 d) {
  const float2 b = unpack_bf16(base_bf16x2);
  __half2 h = __floats2half2_rn(b.x + d.x, b.y + d.y);
  return *reinterpret_cast<uint32_t*>(&h);
}
// f16 pairs as 32-bit words and back, and a bf16 pair as an f16 pair (exact
// within f16's range)
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }
__device__ __forceinline__ __half2 bf16x2_h2(uint32_t v) {
  return __floats2half2_rn(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
// a bf16 pair as a packed fp32 pair (exact), and a packed fp32 pair rounded
// once to an fp16 pair
__device__ __forceinline__ uint64_t bf16x2_f2(uint32_t v) {
  return f2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ uint32_t f2_f16x2(uint64_t v) {
  const float2 f = f2_unpack(v);
  __half2 h = __floats2half2_rn(f.x, f.y);
  return *reinterpret_cast<uint32_t*>(&h);
}

// 2^x for a pair on the FMA pipe, beside the SFU's ex2 (the softmax's
// exponentials would otherwise queue on the SFU alone): x = n + f with n the
// nearest integer (the 1.5 * 2^23 rounding constant), f in [-1/2, 1/2]; 2^f by
// a degree-3 polynomial fitted here for least maximum relative error on that
// interval (Remez exchange: 7.5e-5, below the bf16 rounding P gets), and 2^n
// added to the exponent field.  x is clamped at -126, so a masked score gives
// about 1e-38 instead of 0 and the sum never leaves the normal range.
__device__ __forceinline__ uint64_t exp2_poly_f2(uint64_t x2) {
  constexpr float kRound = 12582912.f;   // 1.5 * 2^23
  const float2 xv = f2_unpack(x2);
  const uint64_t x = f2(fmaxf(xv.x, -126.f), fmaxf(xv.y, -126.f));
  const uint64_t t = add_f2(x, f2(kRound, kRound));
  const uint64_t fr = sub_f2(x, sub_f2(t, f2(kRound, kRound)));
  uint64_t p = fma_f2(f2(0.05517166853f, 0.05517166853f), fr, f2(0.24261112511f, 0.24261112511f));
  p = fma_f2(p, fr, f2(0.69326096773f, 0.69326096773f));
  p = fma_f2(p, fr, f2(0.99992805719f, 0.99992805719f));
  const float2 pv = f2_unpack(p), tv = f2_unpack(t);
  return f2(__uint_as_float(__float_as_uint(pv.x) + (__float_as_uint(tv.x) << 23)),
            __uint_as_float(__float_as_uint(pv.y) + (__float_as_uint(tv.y) << 23)));
}

}  // namespace la

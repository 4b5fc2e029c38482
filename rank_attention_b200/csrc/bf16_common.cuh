// Pieces shared by the bf16 tensor-core kernels: RoPE angles, host-side TMA
// descriptor encoding.
#pragma once
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

namespace la {

constexpr float kLog2e = 1.4426950408889634f;

constexpr int align1k(int x) { return (x + 1023) / 1024 * 1024; }

// Shared memory that keeps kernels with TMEM apart.  A CTA that has allocated TMEM and
// waits for its cluster holds its columns meanwhile.  If two such kernels (of two
// streams) shared SMs and one of them needs all 512 columns, a CTA of each could hold
// what the other's peer waits for, and neither tcgen05.alloc nor a cluster barrier gives
// up.  So a kernel that takes all columns asks for at least kSmemAllTmem and any other
// that allocates for at least kSmemSomeTmem (at most 256 columns): together they exceed
// an SM's 228 KB (1 KB of it reserved a CTA), and so do three of the second kind.
constexpr int kSmemSM = 228 * 1024, kSmemReserved = 1024;
constexpr int kSmemSomeTmem = 80 * 1024;
constexpr int kSmemAllTmem = kSmemSM - 2 * kSmemReserved - kSmemSomeTmem + 1024;
static_assert(3 * (kSmemSomeTmem + kSmemReserved) > kSmemSM, "two CTAs of at most 256 columns");

// RoPE frequencies theta_i = base^(-2i/d), formed in fp64 on the host
struct RopeTheta {
  double theta[64];
  float thetaf[64];   // the same, rounded to fp32 (small in-tile angles)
};

// theta_i = base^(-2i/d), i < d / 2, as powers of one root in extended precision
// (one pow instead of d / 2: the host's share of a short call)
inline void rope_thetas(double base, int d, RopeTheta* rt) {
  const long double root = std::pow((long double)base, -2.0L / d);
  long double t = 1.0L;
  for (int i = 0; i < d / 2; ++i, t *= root) {
    rt->theta[i] = (double)t;
    rt->thetaf[i] = (float)t;
  }
}

// (cos, sin) of t * theta, the angle formed and reduced modulo 2 pi in fp64
__device__ __forceinline__ float2 rope_cs_exact(int64_t t, double theta) {
  const double two_pi = 6.283185307179586476925286766559;
  const double ang = (double)t * theta;
  const float red = (float)fma(-two_pi, rint(ang * 0.15915494309189533577), ang);
  float s, c;
  sincosf(red, &s, &c);
  return make_float2(c, s);
}

// (cos, sin) of a small angle (|ang| < ~200 rad): Cody-Waite reduction with a
// two-constant split of 2 pi, then the SFU (about 2^-21 absolute on [-pi, pi])
__device__ __forceinline__ float2 sincos_small(float ang) {
  const float k = rintf(ang * 0.15915494309189535f);
  float red = fmaf(-k, 6.28318548202514648f, ang);
  red = fmaf(-k, -1.7484556000744083e-07f, red);
  float s, c;
  __sincosf(red, &s, &c);
  return make_float2(c, s);
}

// A driver function through the runtime's entry point (no -lcuda)
inline void* driver_fn(const char* name) {
  void* ptr = nullptr;
  cudaDriverEntryPointQueryResult q;
  const bool ok = cudaGetDriverEntryPoint(name, &ptr, cudaEnableDefault, &q) == cudaSuccess &&
                  q == cudaDriverEntryPointSuccess;
  return ok ? ptr : nullptr;
}

// cuTensorMapEncodeTiled, or null.  It wants a context, and a host thread whose first CUDA
// work is this call has none yet: the current device's primary one is bound then.
inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(driver_fn("cuTensorMapEncodeTiled"));
  static const auto current = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(driver_fn("cuCtxGetCurrent"));
  CUcontext ctx = nullptr;
  int dev = 0;
  if (!fn || !current || current(&ctx) != CUDA_SUCCESS) return nullptr;
  if (!ctx && (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess)) return nullptr;
  return fn;
}

// SMs of the current device (148 on B200; also the answer when no device is
// visible, so that workspace sizes can be planned on a host without a GPU)
inline int device_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return 148;
  }
  return n;
}

// the TMA swizzle whose span equals a box row of row_bytes (32, 64 or >= 128)
inline CUtensorMapSwizzle swizzle_for(int row_bytes) {
  return row_bytes >= 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                          : (row_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B);
}

}  // namespace la

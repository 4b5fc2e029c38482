// lora_grouped_delta: the entry point, and fp32 tokens on the CUDA cores (bf16:
// grouped_bf16.cu).
//
//   out = y + s (x A_a) B_a   over the rows of every segment of agent a
//
// A cluster of CS CTAs takes one tile of 16 rows of one segment: each CTA forms
// x A_a over its share of the hidden dimension, the shares are summed over
// distributed shared memory, and each CTA expands its share of the output
// columns, so the r-wide rows never reach memory and one short segment still
// spreads over CS SMs.
#include "grouped.cuh"
#include "la_internal.cuh"
#include "ptx.cuh"

namespace la {
namespace {

constexpr int TM = 16, NTH = 256, KC = 64;
constexpr int CS = 4;

__global__ void __launch_bounds__(NTH) grouped_simt_kernel(const GroupedParams p) {
  __shared__ __align__(16) float xs[TM][KC + 4];
  __shared__ __align__(16) float as[KC][64];
  __shared__ float part[TM][64];              // this CTA's share of x A
  __shared__ __align__(16) float ts[64][TM];  // x A, transposed
  __shared__ SegTile s_tile;
  const int tid = threadIdx.x, rank = blockIdx.x, R = p.r;
  if (tid < 32) {
    const SegTile t = find_seg_tile(p, blockIdx.y, TM);
    if (tid == 0) s_tile = t;
  }
  __syncthreads();
  const SegTile t = s_tile;
  if (t.bad) {
    if (tid == 0) atomicOr(p.err, kDevSegment);
    return;
  }
  if (t.rows == 0) return;   // the whole cluster: the same tile
  const float* y = reinterpret_cast<const float*>(p.y) + (int64_t)t.row0 * p.ldy;
  float* out = reinterpret_cast<float*>(p.out) + (int64_t)t.row0 * p.ldo;
  const int ns = (p.n_out + CS - 1) / CS, c0 = rank * ns, c1 = min(p.n_out, c0 + ns);
  if (t.agent < 0) {   // no adapter: out = y
    if (p.out != p.y)
      for (int i = tid; i < t.rows * (c1 - c0); i += NTH) {
        const int row = i / (c1 - c0), c = c0 + i % (c1 - c0);
        out[row * p.ldo + c] = y[row * p.ldy + c];
      }
    return;
  }
  const float* x = reinterpret_cast<const float*>(p.x) + (int64_t)t.row0 * p.ldx;
  const float* A = reinterpret_cast<const float*>(p.A) + t.agent * p.a_agent;
  const float* B = reinterpret_cast<const float*>(p.B) + (int64_t)t.agent * R * p.n_out;
  // hidden share: whole KC chunks
  const int chunks = (p.hidden + KC - 1) / KC;
  const int ch0 = chunks * rank / CS, ch1 = chunks * (rank + 1) / CS;
  // thread: row tid / 16, ranks tid % 16 + 16 i
  const int row = tid >> 4, col = tid & 15;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int ch = ch0; ch < ch1; ++ch) {
    const int k0 = ch * KC;
    __syncthreads();
    for (int i = tid; i < TM * KC; i += NTH) {
      const int rr = i / KC, k = k0 + i % KC;
      xs[rr][i % KC] = rr < t.rows && k < p.hidden ? x[rr * p.ldx + k] : 0.f;
    }
    for (int i = tid; i < KC * R; i += NTH) {
      const int k = k0 + i / R;
      as[i / R][i % R] = k < p.hidden ? A[(int64_t)k * R + i % R] : 0.f;
    }
    __syncthreads();
#pragma unroll 8
    for (int k = 0; k < KC; ++k) {
      const float xv = xs[row][k];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + 16 * i < R) acc[i] = fmaf(xv, as[k][col + 16 * i], acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (col + 16 * i < R) part[row][col + 16 * i] = acc[i];
  ptx::cluster_sync_all();
  const uint32_t pu = ptx::smem_u32(&part[0][0]);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (col + 16 * i < R) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < CS; ++k) v += ptx::dsmem_ld(ptx::dsmem_addr(pu + 4 * (row * 64 + col + 16 * i), k));
      ts[col + 16 * i][row] = v;
    }
  ptx::cluster_sync_all();   // every share is read (and ts is in place) before any CTA goes on or exits
  for (int c = c0 + tid; c < c1; c += NTH) {
    float z[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) z[i] = 0.f;
    for (int j = 0; j < R; ++j) {
      const float b = B[(int64_t)j * p.n_out + c];
#pragma unroll
      for (int i = 0; i < TM; i += 4) {
        const float4 tv = *reinterpret_cast<const float4*>(&ts[j][i]);
        z[i] = fmaf(tv.x, b, z[i]);
        z[i + 1] = fmaf(tv.y, b, z[i + 1]);
        z[i + 2] = fmaf(tv.z, b, z[i + 2]);
        z[i + 3] = fmaf(tv.w, b, z[i + 3]);
      }
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
      if (i < t.rows) out[i * p.ldo + c] = fmaf(p.s, z[i], y[i * p.ldy + c]);
  }
}

cudaError_t launch_grouped_simt(const GroupedParams& p, cudaStream_t st) {
  // every segment ends in at most one short tile
  const int64_t tiles = (int64_t)(p.n_tokens + TM - 1) / TM + p.n_segs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CS, (unsigned)tiles, 1);
  cfg.blockDim = dim3(NTH);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CS;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, grouped_simt_kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_grouped_bf16(const GroupedParams& p, cudaStream_t st);

}  // namespace la

extern "C" la_status lora_grouped_delta(const la_grouped_args* a, la_stream_t stream) {
  using namespace la;
  const auto aligned = [](const void* ptr, uintptr_t n) { return (reinterpret_cast<uintptr_t>(ptr) & (n - 1)) == 0; };
  if (!a || (a->dtype != LA_F32 && a->dtype != LA_BF16)) return LA_ERR_INVALID_ARG;
  if (a->n_segs < 0 || a->n_agents < 1 || a->n_tokens < 0 || a->hidden < 1 || a->n_out < 1)
    return LA_ERR_INVALID_ARG;
  if (!(a->r == 8 || a->r == 16 || a->r == 32 || a->r == 64)) return LA_ERR_UNSUPPORTED;
  const int64_t es = a->dtype == LA_F32 ? 4 : 2;
  if ((a->hidden * es) % 16 != 0 || (a->n_out * es) % 16 != 0) return LA_ERR_INVALID_ARG;
  if (!(a->lora_scale - a->lora_scale == 0.f)) return LA_ERR_INVALID_ARG;   // finite
  if (a->n_segs == 0 || a->n_tokens == 0) return LA_OK;   // nothing to read or write
  if (!a->x || !a->y || !a->out || !a->A || !a->B || !a->seg_start || !a->seg_agent) return LA_ERR_INVALID_ARG;
  if (!aligned(a->x, 16) || !aligned(a->y, 16) || !aligned(a->out, 16) || !aligned(a->A, 16) ||
      !aligned(a->B, 16) || !aligned(a->seg_start, 4) || !aligned(a->seg_agent, 4))
    return LA_ERR_INVALID_ARG;
  const auto ld_ok = [&](int64_t ld, int64_t n) { return ld >= n && (ld * es) % 16 == 0; };
  if (!ld_ok(a->ldx, a->hidden) || !ld_ok(a->ldy, a->n_out) || !ld_ok(a->ldo, a->n_out)) return LA_ERR_INVALID_ARG;
  if (a->out == a->y && a->ldo != a->ldy) return LA_ERR_INVALID_ARG;
  if (a->a_agent_stride != 0 &&
      (a->a_agent_stride < (int64_t)a->hidden * a->r || (a->a_agent_stride * es) % 16 != 0))
    return LA_ERR_INVALID_ARG;
  if ((int64_t)(a->n_tokens + 15) / 16 + a->n_segs > 65535) return LA_ERR_UNSUPPORTED;
  GroupedParams p = {};
  p.x = a->x; p.ldx = a->ldx;
  p.y = a->y; p.ldy = a->ldy;
  p.out = a->out; p.ldo = a->ldo;
  p.A = a->A; p.a_agent = a->a_agent_stride;
  p.B = a->B;
  p.seg_start = a->seg_start; p.seg_agent = a->seg_agent;
  p.n_segs = a->n_segs; p.n_agents = a->n_agents; p.n_tokens = a->n_tokens;
  p.hidden = a->hidden; p.n_out = a->n_out; p.r = a->r;
  p.s = a->lora_scale;
  p.err = error_word_ptr();
  if (!p.err) return LA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a->dtype == LA_BF16 ? launch_grouped_bf16(p, st) : launch_grouped_simt(p, st);
  return e == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

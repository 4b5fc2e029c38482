// lora_grouped_delta: the entry point, and fp32 tokens on the CUDA cores (bf16:
// grouped_bf16.cu).
//
//   out = y + s (x A_a) B_a   over the rows of every segment of agent a
//
// A cluster of CS CTAs takes one tile of 16 rows of one segment: each CTA forms
// x A_a over its share of the hidden dimension, the shares are summed over
// distributed shared memory, and each CTA expands its share of the output
// columns, so the r-wide rows never reach memory and one short segment still
// spreads over CS SMs (37 tokens, hidden and out 256, r 8: 9.6 us, latency).
#include "grouped.cuh"
#include "la_internal.cuh"
#include "ptx.cuh"

namespace la {
namespace {

constexpr int TM = kRowsNarrow, NTH = 256, KC = 64;
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

// The same over tiles of 64 rows, where segments are long enough to fill them: both
// products as register tiles of 4 x 4 (16 FMAs for two 16-byte shared-memory reads).
// 2048 tokens in 8 segments, hidden and out 4096, r 64: 120 us (18 TFLOP/s), with the
// 16-row tiles 320 us; r 16 (a quarter of the threads has ranks): 83 against 167 us.
constexpr int WM = kRowsWide, WK = 32, WN = 64;

// acc[4][4] += rows of a (4 ty ..) x columns of b (4 tx ..) over n steps
template <int LA, int LB>
__device__ __forceinline__ void tile_fma(float (&acc)[4][4], const float (*a)[LA], const float (*b)[LB], int ty, int tx,
                                         int n) {
#pragma unroll 8
  for (int k = 0; k < n; ++k) {
    const float4 u = *reinterpret_cast<const float4*>(&a[k][4 * ty]);
    const float4 v = *reinterpret_cast<const float4*>(&b[k][4 * tx]);
    const float av[4] = {u.x, u.y, u.z, u.w}, bv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
  }
}

__global__ void __launch_bounds__(NTH) grouped_wide_kernel(const GroupedParams p) {
  __shared__ __align__(16) float xs[WK][WM + 4];   // x, transposed
  __shared__ __align__(16) float ws[64][WN + 4];   // A_a's rows (WK), then B_a's (r)
  __shared__ __align__(16) float ts[64][WM + 4];   // x A_a, transposed: this CTA's share, then the sum
  __shared__ SegTile s_tile;
  const int tid = threadIdx.x, rank = blockIdx.x, R = p.r;
  if (tid < 32) {
    const SegTile t = find_seg_tile(p, blockIdx.y, WM);
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
  const int nb = (p.n_out + WN - 1) / WN, b0 = nb * rank / CS, b1 = nb * (rank + 1) / CS;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  // thread: rows 4 ty .. +3, ranks or columns 4 tx .. +3
  const int ty = tid >> 4, tx = tid & 15;
  const bool low = 4 * tx < R;   // this thread has ranks
  float acc[4][4] = {};
  if (t.agent >= 0) {
    const float* x = reinterpret_cast<const float*>(p.x) + (int64_t)t.row0 * p.ldx;
    const float* A = reinterpret_cast<const float*>(p.A) + t.agent * p.a_agent;
    const int chunks = (p.hidden + WK - 1) / WK, ch0 = chunks * rank / CS, ch1 = chunks * (rank + 1) / CS;
    // the next chunk's words travel while this one's are multiplied: x 64 rows x 8
    // float4, A_a 32 rows x 16, two of each a thread
    float4 xv[2], av[2];
    auto fetch = [&](int ch) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = tid + u * NTH, row = i >> 3, k = ch * WK + 4 * (i & 7);
        xv[u] = row < t.rows && k < p.hidden ? *reinterpret_cast<const float4*>(x + row * p.ldx + k) : zero;
        const int kk = ch * WK + (i >> 4), c = 4 * (i & 15);
        av[u] = kk < p.hidden && c < R ? *reinterpret_cast<const float4*>(A + (int64_t)kk * R + c) : zero;
      }
    };
    if (ch0 < ch1) fetch(ch0);
    for (int ch = ch0; ch < ch1; ++ch) {
      __syncthreads();
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = tid + u * NTH, row = i >> 3, k = 4 * (i & 7);
        xs[k][row] = xv[u].x;
        xs[k + 1][row] = xv[u].y;
        xs[k + 2][row] = xv[u].z;
        xs[k + 3][row] = xv[u].w;
        *reinterpret_cast<float4*>(&ws[i >> 4][4 * (i & 15)]) = av[u];
      }
      __syncthreads();
      if (ch + 1 < ch1) fetch(ch + 1);
      if (low) tile_fma(acc, xs, ws, ty, tx, WK);
    }
    if (low) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float4*>(&ts[4 * tx + j][4 * ty]) = make_float4(acc[0][j], acc[1][j], acc[2][j], acc[3][j]);
    }
    ptx::cluster_sync_all();   // (the agent is the whole cluster's)
    float4 sum[4];
    if (low) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sum[j] = zero;
        const uint32_t a = ptx::smem_u32(&ts[4 * tx + j][4 * ty]);
#pragma unroll
        for (int k = 0; k < CS; ++k) {
          const float4 v = ptx::dsmem_ld4(ptx::dsmem_addr(a, k));
          sum[j].x += v.x; sum[j].y += v.y; sum[j].z += v.z; sum[j].w += v.w;
        }
      }
    }
    ptx::cluster_sync_all();   // every share is read before the sum lies over it, or its CTA exits
    if (low) {
#pragma unroll
      for (int j = 0; j < 4; ++j) *reinterpret_cast<float4*>(&ts[4 * tx + j][4 * ty]) = sum[j];
    }
  } else if (p.out == p.y) {
    return;   // no adapter, in place
  }
  const float* B = reinterpret_cast<const float*>(p.B) + (int64_t)max(t.agent, 0) * R * p.n_out;
  for (int b = b0; b < b1; ++b) {
    const int col = b * WN + 4 * tx;
    const bool in = col < p.n_out;   // n_out is a multiple of 4
    float4 yv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      yv[i] = in && 4 * ty + i < t.rows ? *reinterpret_cast<const float4*>(y + (4 * ty + i) * p.ldy + col) : zero;
    if (t.agent >= 0) {
      __syncthreads();   // ts is in place, the last block's B_a has been read
      for (int i = tid; i < R * (WN / 4); i += NTH) {
        const int j = i >> 4, c = b * WN + 4 * (i & 15);
        *reinterpret_cast<float4*>(&ws[j][4 * (i & 15)]) =
            c < p.n_out ? *reinterpret_cast<const float4*>(B + (int64_t)j * p.n_out + c) : zero;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
      tile_fma(acc, ts, ws, ty, tx, R);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        yv[i] = make_float4(fmaf(p.s, acc[i][0], yv[i].x), fmaf(p.s, acc[i][1], yv[i].y),
                            fmaf(p.s, acc[i][2], yv[i].z), fmaf(p.s, acc[i][3], yv[i].w));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (in && 4 * ty + i < t.rows) *reinterpret_cast<float4*>(out + (4 * ty + i) * p.ldo + col) = yv[i];
  }
}

cudaError_t launch_grouped_simt(const GroupedParams& p, cudaStream_t st) {
  const int tm = grouped_tile_rows(false, p.n_tokens, p.n_segs);
  const bool wide = tm == WM;
  const int64_t tiles = grouped_tiles(p.n_tokens, p.n_segs, tm);
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, wide ? grouped_wide_kernel : grouped_simt_kernel, p);
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
  const int rows = grouped_tile_rows(a->dtype == LA_BF16, a->n_tokens, a->n_segs);
  if (grouped_tiles(a->n_tokens, a->n_segs, rows) > 65535) return LA_ERR_UNSUPPORTED;   // the grid's y
  if (a->out == a->x || a->out == a->A || a->out == a->B) return LA_ERR_INVALID_ARG;   // read to the end
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

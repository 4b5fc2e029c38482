// lora_grouped_delta on the tcgen05 tensor cores (bf16 storage, fp32
// accumulation in TMEM):  out = y + s (x A_a) B_a  over the rows of every
// segment of agent a.
//
// A cluster of CS CTAs takes one tile of up to 128 rows of one segment:
//   1. t = x A_a      M = 128 rows, N = r, over this CTA's share of the hidden
//                     dimension in chunks of 64 columns;
//   2. the shares of t are summed over distributed shared memory and split into
//      two bf16 terms, t = hi + lo (the remainder: 2^-18 of t), which go back to
//      TMEM as one operand of K = 2 r;
//   3. out = y + s t B_a   M = 128, N = 64, over this CTA's share of the columns.
// Where tiles are so few that clusters would leave SMs idle, several clusters form
// the same t (grid z) and share the columns.
// Both passes stream through one ring of stages (x and A_a, then y and B_a), so
// that y and B_a are on their way while t is reduced.  Loads come in boxes of 32
// rows, only those with rows of the tile; the other rows of a stage hold anything
// (rows do not mix).  Bound by memory for many rows (x, y and out once each; A_a
// and B_a come from L2), by latency for few: the cluster spreads a short segment
// over CS SMs.  Hidden and out 4096: 16384 tokens, r 64, 407 MB, 84 us with fresh inputs
// (4.9 TB/s, 74 % of the copy rate; 77 us where calls repeat their inputs, part of which
// is still in L2); 48 tokens, r 16, 9.1 us; on the CUDA cores 1604 and 76 us.
//
// Warps: four epilogue warps (a row a thread), one to issue the MMAs, one to load.
#include <cuda.h>

#include "bf16_common.cuh"
#include "grouped.cuh"
#include "la_internal.cuh"
#include "ptx.cuh"

namespace la {
namespace {

using namespace ptx;

constexpr int GM = kRowsTC;     // rows per tile
constexpr int GC = 64;          // columns per chunk (128-byte swizzled rows)
constexpr int GBOX = 32;        // rows per TMA box
constexpr int GNTH = 192;
constexpr int kMaxStages = 6;
constexpr int kGroupedPipeWait = 2;   // bit of the device error word
// TMEM columns: x A (R), its two terms (R), and two output blocks
constexpr int G_D1 = 0, G_A2 = 64, G_D2 = 128, G_COLS = 256;

template <int R>
struct GCfg {
  static constexpr int ROWB = R * 2;   // bytes of a row of A_a
  static constexpr uint32_t LAYOUT = ROWB == 128 ? 2u : (ROWB == 64 ? 4u : 6u);
  static constexpr int XB = GM * GC * 2;      // a stage's x or y
  static constexpr int WB = GC * R * 2;       // its A_a (64 rows of R) or B_a (R rows of 64)
  static constexpr int STAGE = XB + WB;
  static constexpr int RED = GM * R * 4;      // this CTA's share of t
  static constexpr int MISC = 16 * kMaxStages + 96;
};

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int R>
__global__ void __launch_bounds__(GNTH)
    grouped_tc_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmA,
                      const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmB,
                      const GroupedParams p, const int ns) {
  using C = GCfg<R>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int CS = gridDim.x, rank = blockIdx.x;
  const int part = rank + CS * blockIdx.z, parts = CS * gridDim.z;   // this CTA's share of the columns
  const uint32_t red = sb + ns * C::STAGE;                 // [GM][R] fp32, CS > 1 only
  const int off_bar = ns * C::STAGE + (CS > 1 ? C::RED : 0);
  const uint32_t b0 = sb + off_bar;
  auto full = [&](int s) { return b0 + 16 * s; };
  auto free_ = [&](int s) { return b0 + 16 * s + 8; };
  const uint32_t bx = b0 + 16 * kMaxStages;
  const uint32_t d1full = bx, a2ready = bx + 8;
  auto d2full = [&](int b) { return bx + 16 + 8 * b; };
  auto d2free = [&](int b) { return bx + 32 + 8 * b; };
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + off_bar + 16 * kMaxStages + 48);
  __shared__ SegTile s_tile;
  __shared__ int s_fail;

  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  if (w == 0) {
    const SegTile t = find_seg_tile(p, blockIdx.y, GM);
    if (lane == 0) s_tile = t;
  }
  if (w == 4 && lane == 0) {
    s_fail = 0;
    for (int s = 0; s < ns; ++s) {
      mbar_init(full(s), 1);
      mbar_init(free_(s), 4);
    }
    mbar_init(d1full, 1);
    mbar_init(a2ready, 4);
    for (int b = 0; b < 2; ++b) {
      mbar_init(d2full(b), 1);
      mbar_init(d2free(b), 4);
    }
    fence_mbar_init();
  }
  if (w == 3) tmem_alloc(smem_u32(tslot), G_COLS);
  if (w == 5 && lane == 0) {
    tma_prefetch(&tmX);
    tma_prefetch(&tmA);
    tma_prefetch(&tmY);
    tma_prefetch(&tmB);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const SegTile t = s_tile;
  const int nblk = (p.n_out + GC - 1) / GC;   // column blocks, and this CTA's share
  const int c0 = (int)((int64_t)nblk * part / parts), c1 = (int)((int64_t)nblk * (part + 1) / parts);
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out) + (int64_t)t.row0 * p.ldo;
  // the same verdict in every CTA of the cluster: a bad segment, no such tile, or no
  // adapter (out = y)
  if (t.bad || t.rows == 0 || t.agent < 0) {
    if (t.bad) {
      if (tid == 0) atomicOr(p.err, kDevSegment);
    } else if (t.rows > 0 && p.out != p.y) {
      const __nv_bfloat16* y = reinterpret_cast<const __nv_bfloat16*>(p.y) + (int64_t)t.row0 * p.ldy;
      const int lo = c0 * (GC / 8), n8 = min(c1 * (GC / 8), p.n_out / 8) - lo;   // 16-byte chunks
      for (int i = tid; i < t.rows * n8; i += GNTH) {
        const int row = i / n8, c = 8 * (lo + i % n8);
        *reinterpret_cast<uint4*>(out + row * p.ldo + c) = *reinterpret_cast<const uint4*>(y + row * p.ldy + c);
      }
    }
    if (w == 3) tmem_dealloc(tmem, G_COLS);
    return;
  }
  int fail = 0;

  const int chunks = (p.hidden + GC - 1) / GC;
  const int k0 = (int)((int64_t)chunks * rank / CS), n1 = (int)((int64_t)chunks * (rank + 1) / CS) - k0;
  const int n2 = c1 - c0;
  const int boxes = (t.rows + GBOX - 1) / GBOX;

  if (w == 5) {
    // ============================================================ loads
    if (CS > 1) cluster_arrive();   // nothing to publish at the first cluster barrier
    if (lane == 0) {
      const uint32_t bytes = (uint32_t)(boxes * GBOX * GC * 2 + C::WB);
      int s = 0, ph = 0;
      for (int i = 0; i < n1 + n2; ++i) {
        if (i >= ns && !mbar_wait(free_(s), ph ^ 1)) fail = 1;
        const uint32_t dst = sb + s * C::STAGE;
        mbar_expect_tx(full(s), bytes);
        const bool first = i < n1;
        const int col = GC * (first ? k0 + i : c0 + i - n1);
        for (int b = 0; b < boxes; ++b)
          tma_load_2d_(dst + b * (GBOX * GC * 2), first ? &tmX : &tmY, full(s), col, t.row0 + GBOX * b);
        if (first) {
          tma_load_3d(dst + C::XB, &tmA, full(s), 0, col, p.a_agent ? t.agent : 0);
        } else {
          tma_load_3d(dst + C::XB, &tmB, full(s), col, 0, t.agent);
          if (p.r < 16) tma_load_3d(dst + C::XB + 1024, &tmB, full(s), col, 0, t.agent);   // hi and lo share K = 16
        }
        if (++s == ns) { s = 0; ph ^= 1; }
      }
    }
    __syncwarp();
    if (CS > 1) {
      cluster_wait();
      cluster_sync_all();
    }
  } else if (w == 4) {
    // ============================================================ MMAs
    if (CS > 1) cluster_arrive();
    constexpr uint32_t ID1 = umma_idesc_bf16(GM, R, 0, 1), ID2 = umma_idesc_bf16(GM, GC, 0, 1);
    int s = 0, ph = 0;
    for (int i = 0; i < n1; ++i) {
      if (!mbar_wait(full(s), ph)) fail = 1;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t xd = umma_desc(sb + s * C::STAGE, 16, 1024, 2);
        const uint64_t ad = umma_desc(sb + s * C::STAGE + C::XB, GC * C::ROWB, 8 * C::ROWB, C::LAYOUT);
#pragma unroll
        for (int k = 0; k < GC / 16; ++k)
          umma_bf16(tmem + G_D1, umma_desc_add(xd, 32 * k), umma_desc_add(ad, 16 * C::ROWB * k), ID1,
                    i > 0 || k > 0 ? 1u : 0u);
        umma_commit(free_(s));
        for (int a = 0; a < 3; ++a) mbar_arrive(free_(s));   // of four arrivals; the commit's is the last
        if (i == n1 - 1) umma_commit(d1full);
      }
      __syncwarp();
      if (++s == ns) { s = 0; ph ^= 1; }
    }
    if (!mbar_wait(a2ready, 0)) fail = 1;
    for (int i = 0; i < n2; ++i) {
      const int b = i & 1;
      if (!mbar_wait(full(s), ph)) fail = 1;
      if (i >= 2 && !mbar_wait(d2free(b), ((i >> 1) - 1) & 1)) fail = 1;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t bd = umma_desc(sb + s * C::STAGE + C::XB, R * 128, 1024, 2);
        const uint32_t td = tmem + G_D2 + GC * b;
        umma_bf16_ts(td, tmem + G_A2, bd, ID2, 0u);
        if (p.r >= 16) {
#pragma unroll
          for (int k = 1; k < R / 8; ++k)   // R / 16 steps of hi, then of lo over the same B_a
            umma_bf16_ts(td, tmem + G_A2 + 8 * k, umma_desc_add(bd, (k % (R / 16)) * 16 * 128), ID2, 1u);
        }
        umma_commit(d2full(b));
      }
      __syncwarp();
      if (++s == ns) { s = 0; ph ^= 1; }
    }
    if (CS > 1) {
      cluster_wait();
      cluster_sync_all();
    }
  } else {
    // ============================================================ epilogue: thread = row (TMEM lane)
    const uint32_t tl = (uint32_t)(32 * w) << 16;
    const bool mine = tid < t.rows;
    const bool live = 32 * w < t.rows;   // this warp has rows
    float v[R];
    if (n1 > 0) {
      if (!mbar_wait(d1full, 0)) fail = 1;
      tc_fence_after();
#pragma unroll
      for (int h = 0; h < R / 16; ++h) {
        uint32_t u[16];
        tmem_ld32x32b_x16(u, tmem + G_D1 + 16 * h + tl);
        tmem_wait_ld_r16(u);
#pragma unroll
        for (int c = 0; c < 16; ++c) v[16 * h + c] = __uint_as_float(u[c]);
      }
    } else {
#pragma unroll
      for (int c = 0; c < R; ++c) v[c] = 0.f;
    }
    if (CS > 1) {
      // [R / 4][GM] float4: conflict-free by rows
      if (mine) {
#pragma unroll
        for (int c = 0; c < R; c += 4)
          sts128(red + (uint32_t)((c / 4) * GM + tid) * 16, __float_as_uint(v[c]), __float_as_uint(v[c + 1]),
                 __float_as_uint(v[c + 2]), __float_as_uint(v[c + 3]));
      }
      cluster_arrive();
      cluster_wait();
      if (mine) {
#pragma unroll
        for (int c = 0; c < R; ++c) v[c] = 0.f;
        for (int k = 0; k < CS; ++k) {   // in rank order: the same sum in every CTA
#pragma unroll
          for (int c = 0; c < R; c += 4) {
            const float4 o = dsmem_ld4(dsmem_addr(red + (uint32_t)((c / 4) * GM + tid) * 16, k));
            v[c] += o.x; v[c + 1] += o.y; v[c + 2] += o.z; v[c + 3] += o.w;
          }
        }
      }
    }
    // two bf16 terms, packed in pairs: hi in columns [0, r / 2), lo behind
    if (live) {
      if (R == 16 && p.r < 16) {   // r = 8: hi and lo fill one step of K = 16
        uint32_t a[16];
#pragma unroll
        for (int c = 0; c < 8; c += 2) {
          const uint32_t h = pack_bf16(v[c], v[c + 1]);
          const float2 hf = unpack_bf16(h);
          a[c / 2] = h;
          a[4 + c / 2] = pack_bf16(v[c] - hf.x, v[c + 1] - hf.y);
        }
#pragma unroll
        for (int c = 8; c < 16; ++c) a[c] = 0;
        tmem_st32x32b_x16(tmem + G_A2 + tl, a);
      } else {
#pragma unroll
        for (int q = 0; q < R / 16; ++q) {   // columns 16 q .. +15 of [hi | lo]
          uint32_t a[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const int e = 16 * q + c, j = 2 * (e % (R / 2));
            const uint32_t h = pack_bf16(v[j], v[j + 1]);
            const float2 hf = unpack_bf16(h);
            a[c] = e < R / 2 ? h : pack_bf16(v[j] - hf.x, v[j + 1] - hf.y);
          }
          tmem_st32x32b_x16(tmem + G_A2 + 16 * q + tl, a);
        }
      }
      tmem_wait_st();
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(a2ready);

    int s = n1 % ns, ph = (n1 / ns) & 1;
    for (int i = 0; i < n2; ++i) {
      const int b = i & 1;
      if (!mbar_wait(d2full(b), (i >> 1) & 1)) fail = 1;
      if (!mbar_wait(full(s), ph)) fail = 1;   // y, written by the loads
      tc_fence_after();
      const uint32_t st = sb + s * C::STAGE;
      if (live) {
        uint32_t d[2][32];
        tmem_ld32x32b_x32(d[0], tmem + G_D2 + GC * b + tl);
        tmem_ld32x32b_x32(d[1], tmem + G_D2 + GC * b + 32 + tl);
        tmem_wait_ld_r32(d[0]);
        tmem_wait_ld_r32(d[1]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(d2free(b));
        // out over y in its swizzled row, then row segments of 128 bytes to memory
        const uint32_t rowa = st + (uint32_t)tid * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint32_t a = rowa + (uint32_t)((c ^ (tid & 7)) << 4);
          const uint4 yv = lds128(a);
          const uint32_t yw[4] = {yv.x, yv.y, yv.z, yv.w};
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 yf = unpack_bf16(yw[e]);
            const int k = 8 * c + 2 * e;
            o[e] = pack_bf16(fmaf(p.s, __uint_as_float(d[k >> 5][k & 31]), yf.x),
                             fmaf(p.s, __uint_as_float(d[(k + 1) >> 5][(k + 1) & 31]), yf.y));
          }
          sts128(a, o[0], o[1], o[2], o[3]);
        }
        __syncwarp();
        const int col = GC * (c0 + i) + 8 * (lane & 7);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int row = 32 * w + 4 * u + (lane >> 3);
          const uint4 o = lds128(st + (uint32_t)row * 128 + (uint32_t)(((lane & 7) ^ (row & 7)) << 4));
          if (row < t.rows && col < p.n_out) *reinterpret_cast<uint4*>(out + (int64_t)row * p.ldo + col) = o;
        }
        fence_proxy_async_smem();   // these accesses before the next load into the stage
      } else {
        if (lane == 0) mbar_arrive(d2free(b));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(free_(s));
      if (++s == ns) { s = 0; ph ^= 1; }
    }
    if (CS > 1) cluster_sync_all();   // every share is read before any CTA of the cluster exits
  }
  if (fail) s_fail = 1;
  tc_fence_before();
  __syncthreads();
  if (w == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, G_COLS);
  }
  if (tid == 0 && s_fail) atomicOr(p.err, kGroupedPipeWait);
}

bool grouped_maps(const GroupedParams& p, int R, CUtensorMap* mx, CUtensorMap* ma, CUtensorMap* my, CUtensorMap* mb) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint32_t one[3] = {1, 1, 1};
  auto map = [&](CUtensorMap* m, const void* ptr, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                 const cuuint32_t* box) {
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(ptr), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle_for((int)box[0] * 2), CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const cuuint32_t rowbox[2] = {GC, GBOX};
  const cuuint64_t xd[2] = {(cuuint64_t)p.hidden, (cuuint64_t)p.n_tokens}, xs[1] = {(cuuint64_t)p.ldx * 2};
  const cuuint64_t yd[2] = {(cuuint64_t)p.n_out, (cuuint64_t)p.n_tokens}, ys[1] = {(cuuint64_t)p.ldy * 2};
  // A_a: 64 rows of R columns (at r = 8 columns 8..15 are the zero fill); one A: one agent
  const cuuint64_t ad[3] = {(cuuint64_t)p.r, (cuuint64_t)p.hidden, (cuuint64_t)(p.a_agent ? p.n_agents : 1)};
  const cuuint64_t as[2] = {(cuuint64_t)p.r * 2, (cuuint64_t)(p.a_agent ? p.a_agent : (int64_t)p.hidden * p.r) * 2};
  const cuuint32_t ab[3] = {(cuuint32_t)R, GC, 1};
  const cuuint64_t bd[3] = {(cuuint64_t)p.n_out, (cuuint64_t)p.r, (cuuint64_t)p.n_agents};
  const cuuint64_t bs[2] = {(cuuint64_t)p.n_out * 2, (cuuint64_t)p.r * p.n_out * 2};
  const cuuint32_t bb[3] = {GC, (cuuint32_t)p.r, 1};
  return map(mx, p.x, 2, xd, xs, rowbox) && map(my, p.y, 2, yd, ys, rowbox) && map(ma, p.A, 3, ad, as, ab) &&
         map(mb, p.B, 3, bd, bs, bb);
}

template <int R>
cudaError_t launch_gt(const GroupedParams& p, cudaStream_t st) {
  using C = GCfg<R>;
  CUtensorMap mx, ma, my, mb;
  if (!grouped_maps(p, R, &mx, &ma, &my, &mb)) return cudaErrorInvalidValue;
  const int64_t tiles = grouped_tiles(p.n_tokens, p.n_segs, GM);
  // CTAs a tile: eight or four while one CTA an SM covers the launch, two while two do.
  // The sum over distributed shared memory grows with CS: 16384 tokens, r 64, 132 tiles
  // at CS 1 / 2 / 4 / 8: 90 / 77 / 99 / 203 us; 1501 tokens, r 32, 21 tiles: 42 / 25 /
  // 17.8 / 18.9 us; 48 tokens, r 16, 4 tiles (one cluster a tile): 64 / 35 / 20 / 13 us.
  const int sms = device_sms();
  int CS = 8;
  while (CS > 2 && tiles * CS > sms) CS /= 2;
  if (tiles * CS > 2 * sms) CS = 1;
  // clusters a tile: those that would otherwise leave SMs idle form t again and share
  // the columns, down to two blocks of 64 a CTA
  int Z = 1;
  while (Z < 8 && tiles * CS * Z * 2 <= sms && (int64_t)CS * Z * 4 * GC <= p.n_out) Z *= 2;
  // as many stages as let two CTAs share an SM
  const int rest = 1024 + (CS > 1 ? C::RED : 0) + C::MISC;
  int ns = (113 * 1024 - rest) / C::STAGE;
  if (ns > kMaxStages) ns = kMaxStages;
  // never three CTAs an SM (their TMEM would not fit), and none beside a kernel with all of it
  static_assert(G_COLS <= 256, "TMEM of the kernels that take kSmemSomeTmem");
  const int smem = max(rest + ns * C::STAGE, kSmemSomeTmem);
  const auto kern = grouped_tc_kernel<R>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static bool allowed[64] = {};   // per device, once
  if (!allowed[dev & 63]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 114 * 1024);
    if (e != cudaSuccess) return e;
    allowed[dev & 63] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)CS, (unsigned)tiles, (unsigned)Z);
  cfg.blockDim = dim3(GNTH);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)CS;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, mx, ma, my, mb, p, ns);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_grouped_bf16(const GroupedParams& p, cudaStream_t st) {
  if (p.r <= 16) return launch_gt<16>(p, st);
  return p.r == 32 ? launch_gt<32>(p, st) : launch_gt<64>(p, st);
}

}  // namespace la

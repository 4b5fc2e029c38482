// Attention of drafted trees on the CUDA cores (fp32 arithmetic): fp32 inputs,
// whose accuracy bf16 or fp16 operands cannot meet (bf16: attn_tree_bf16.cu).
//
// One CTA = one (sequence, agent, KV head), a block of up to 64 query rows
// (tokens x the group's heads) and one split of the keys; the splits of a
// block form a thread-block cluster and merge over distributed shared memory,
// so the call needs no workspace.  Per tile of 32 keys:
//   K^a = K_base + RoPE_pos(s LRk B_k^a), pos = base + offset with the turn
//         R(base) R(offset): a context tile's base is its first row, a drafted
//         tile's base is C and its offsets are the nodes' depths
//   S   = Q K^a^T, masked; running maximum and sum; O += P V_base, O_lr += P LRv
// and once per row out = (O + s O_lr B_v^a) / l after the merge.
// Long contexts are bound by fp32 FMA issue: 4 rows x 2 keys of S and 4 rows x
// (d + r) / 16 of O a thread, operands as 16-byte shared-memory reads (2 agents, 8 / 2
// heads of 128, 16 nodes, 4096 keys: 176 us).  Short ones are bound by the chain of a
// tile (loads, delta, scores, values), so a split takes as little as one tile: 2 agents,
// 4 / 2 heads of 64, 8 nodes, 256 keys: 20 us, with four tiles a split at least 28 us.
#include <cmath>

#include "bf16_common.cuh"
#include "la_internal.cuh"
#include "ptx.cuh"
#include "tree.cuh"

namespace la {
namespace {

constexpr int TK = 32;     // keys per tile
constexpr int RB = 64;     // query rows per CTA
constexpr int NTH = 256;

template <int D>
struct TsCfg {
  static constexpr int LD = D + 4;
  int q, ka, v, lr, ps, cs, anc, mask, total;   // byte offsets
  __host__ __device__ explicit TsCfg(int R) {
    int off = 0;
    q = off; off += RB * LD * 4;
    ka = off; off += TK * LD * 4;
    v = off; off += TK * LD * 4;
    lr = off; off += TK * (2 * R + 4) * 4;
    // the partial [RB][D + R] and its (m, l) lie over q, ka, v and lr after the loop
    const int part = RB * (D + R) * 4 + RB * 8;
    if (off < part) off = part;
    ps = off; off += RB * (TK + 4) * 4;
    cs = off; off += TK * (D / 2) * 8;
    anc = off; off += (D / 2) * 8;
    mask = off; off += kTreeMaxNodes * 8;
    total = off;
  }
};

template <typename OUT, int D>
__global__ void __launch_bounds__(NTH)
    attn_tree_simt_kernel(const AttnParams p, const TreeParams tp, const __grid_constant__ RopeTheta rt) {
  constexpr int H2 = D / 2, LD = D + 4, NV = D / 64;
  extern __shared__ __align__(16) unsigned char smem[];
  const int R = p.r, g = p.g;
  const TsCfg<D> L(R);
  const int LDR = 2 * R + 4;
  float* Qs = reinterpret_cast<float*>(smem + L.q);
  float* Ka = reinterpret_cast<float*>(smem + L.ka);
  float* Vs = reinterpret_cast<float*>(smem + L.v);
  float* LRs = reinterpret_cast<float*>(smem + L.lr);
  float* Ps = reinterpret_cast<float*>(smem + L.ps);
  float2* CS = reinterpret_cast<float2*>(smem + L.cs);
  float2* Anc = reinterpret_cast<float2*>(smem + L.anc);
  uint64_t* Mk = reinterpret_cast<uint64_t*>(smem + L.mask);
  __shared__ int s_ok;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ty = tid >> 4, tx = tid & 15;
  const int S = p.n_splits, split = blockIdx.x;
  const int QB = RB / g, nblk = (p.n_q_tokens + QB - 1) / QB;
  const int blk = blockIdx.y % nblk, ua = blockIdx.y / nblk;
  const int agent = ua % p.n_agents, kvh = ua / p.n_agents;
  const int seq = blockIdx.z;
  const int tree = tp.n_trees > 1 ? agent : 0;
  const int tok0 = blk * QB;

  // the sequence's committed length and the tree; every CTA of the cluster
  // reads the same values and takes the same branch
  const int64_t C = p.kv_len[seq];
  const int m = tp.tree_len ? tp.tree_len[seq * tp.n_trees + tree] : tp.nodes;
  if (C < 0 || C + (int64_t)tp.n_trees * tp.nodes > p.max_kv_len) {
    if (tid == 0) atomicOr(p.err, kDevKvLen);
    return;
  }
  if (m < 0 || m > tp.nodes) {
    if (tid == 0) atomicOr(p.err, kDevTree);
    return;
  }
  if (warp == 0) {
    const bool ok = tree_masks_warp(
        tp.parent ? tp.parent + ((int64_t)seq * tp.n_trees + tree) * tp.nodes : nullptr, tp.nodes, m, Mk);
    if (lane == 0) s_ok = ok;
  }
  __syncthreads();
  if (!s_ok) {
    if (tid == 0) atomicOr(p.err, kDevTree);
    return;
  }
  const int ntok = min(QB, m - tok0);
  if (ntok <= 0) return;   // no live node in this block (the same in the whole cluster)
  const int rows = ntok * g;

  const float* kbase = reinterpret_cast<const float*>(p.k_base) + seq * p.kv_seq + kvh * p.kv_head;
  const float* vbase = reinterpret_cast<const float*>(p.v_base) + seq * p.kv_seq + kvh * p.kv_head;
  const float* lrp = reinterpret_cast<const float*>(p.lr) + seq * p.lr_seq + agent * p.lr_agent;
  const int64_t ldB = (int64_t)p.n_kv * D;
  const float* Bk = p.B_k ? reinterpret_cast<const float*>(p.B_k) + (int64_t)agent * R * ldB + kvh * D : nullptr;
  const float* Bv = reinterpret_cast<const float*>(p.B_v) + (int64_t)agent * R * ldB + kvh * D;
  const int64_t qrow0 = ((int64_t)seq * p.n_agents + agent) * p.n_q_tokens + tok0;

  for (int i = tid; i < RB * D / 4; i += NTH) {
    const int row = i / (D / 4), c = 4 * (i % (D / 4));
    float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < rows)
      q = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.q) +
                                           ((qrow0 + row / g) * p.n_q + kvh * g + row % g) * D + c);
    *reinterpret_cast<float4*>(Qs + row * LD + c) = q;
  }
  for (int i = tid; i < TK * H2; i += NTH) CS[i] = rope_cs_exact(i / H2, rt.theta[i % H2]);
  uint64_t vis[4];   // the drafted nodes this thread's rows see
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 4 * ty + i;
    vis[i] = row < rows ? Mk[tok0 + row / g] : 0;
  }

  const int Nc = (int)((C + TK - 1) / TK), Nt = (m + TK - 1) / TK, N = Nc + Nt;
  const int n0 = (int)((int64_t)N * split / S), n1 = (int)((int64_t)N * (split + 1) / S);

  float o[4][4 * NV], ol[4][4], mrow[4], lrow[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    mrow[i] = -INFINITY;
    lrow[i] = 0.f;
#pragma unroll
    for (int c = 0; c < 4 * NV; ++c) o[i][c] = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) ol[i][c] = 0.f;
  }

  for (int n = n0; n < n1; ++n) {
    const bool drafted = n >= Nc;
    const int64_t k0 = drafted ? (int64_t)(n - Nc) * TK : (int64_t)n * TK;   // first key of the tile
    const int cnt = (int)min((int64_t)TK, (drafted ? (int64_t)m : C) - k0);
    const int64_t row0 = drafted ? C + (int64_t)tree * tp.nodes + k0 : k0;
    __syncthreads();   // the last tile's reads are done
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int u = 0; u < TK * D / 4 / NTH; ++u) {
      const int i = tid + u * NTH, t = i / (D / 4), c = 4 * (i % (D / 4));
      float4 kv = zero, vv = zero;
      if (t < cnt) {
        kv = *reinterpret_cast<const float4*>(kbase + (row0 + t) * p.kv_tok + c);
        vv = *reinterpret_cast<const float4*>(vbase + (row0 + t) * p.kv_tok + c);
      }
      *reinterpret_cast<float4*>(Ka + t * LD + c) = kv;
      *reinterpret_cast<float4*>(Vs + t * LD + c) = vv;
    }
    for (int i = tid; i < TK * 2 * R / 4; i += NTH) {
      const int t = i / (R / 2), c = 4 * (i % (R / 2));
      *reinterpret_cast<float4*>(LRs + t * LDR + c) =
          t < cnt ? *reinterpret_cast<const float4*>(lrp + (row0 + t) * 2 * R + c) : zero;
    }
    if (Bk) {
      if (tid < H2) Anc[tid] = rope_cs_exact(drafted ? C : k0, rt.theta[tid]);
      if (drafted)
        for (int i = tid; i < TK * H2; i += NTH) {
          const int t = i / H2;
          CS[i] = rope_cs_exact(t < cnt ? __popcll(Mk[k0 + t]) - 1 : 0, rt.theta[i % H2]);
        }
    }
    __syncthreads();
    if (Bk) {   // K^a over K_base; this thread: one frequency, every G-th key
      constexpr int G = NTH / H2, U = TK / G;
      const int i = tid % H2, kq = tid / H2;
      float x1[U], x2[U];
#pragma unroll
      for (int u = 0; u < U; ++u) x1[u] = x2[u] = 0.f;
      for (int j = 0; j < R; ++j) {
        const float b1 = Bk[j * ldB + i], b2 = Bk[j * ldB + i + H2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float lv = LRs[(kq + G * u) * LDR + j];
          x1[u] = fmaf(lv, b1, x1[u]);
          x2[u] = fmaf(lv, b2, x2[u]);
        }
      }
      const float2 a = Anc[i];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = kq + G * u;
        const float2 b = CS[t * H2 + i];
        const float c = a.x * b.x - a.y * b.y, sn = a.y * b.x + a.x * b.y;
        const float y1 = p.s * x1[u], y2 = p.s * x2[u];
        Ka[t * LD + i] += y1 * c - y2 * sn;
        Ka[t * LD + i + H2] += y2 * c + y1 * sn;
      }
      __syncthreads();
    }
    // S: rows 4 ty .. +3, keys tx and tx + 16
    float s[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i][0] = s[i][1] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      const float4 ka = *reinterpret_cast<const float4*>(Ka + tx * LD + c);
      const float4 kb = *reinterpret_cast<const float4*>(Ka + (tx + 16) * LD + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 q = *reinterpret_cast<const float4*>(Qs + (4 * ty + i) * LD + c);
        s[i][0] = fmaf(q.x, ka.x, fmaf(q.y, ka.y, fmaf(q.z, ka.z, fmaf(q.w, ka.w, s[i][0]))));
        s[i][1] = fmaf(q.x, kb.x, fmaf(q.y, kb.y, fmaf(q.z, kb.z, fmaf(q.w, kb.w, s[i][1]))));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float z[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = tx + 16 * h;
        const bool see = t < cnt && (!drafted || ((vis[i] >> (k0 + t)) & 1));
        z[h] = see ? s[i][h] * p.scale : -INFINITY;
      }
      float mx = fmaxf(z[0], z[1]);
#pragma unroll
      for (int k = 8; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
      const float mn = fmaxf(mrow[i], mx);
      const float mu = mn == -INFINITY ? 0.f : mn;
      const float corr = mrow[i] == -INFINITY ? 0.f : expf(mrow[i] - mu);
      const float p0 = expf(z[0] - mu), p1 = expf(z[1] - mu);
      float ps = p0 + p1;
#pragma unroll
      for (int k = 8; k > 0; k >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, k);
      mrow[i] = mn;
      lrow[i] = lrow[i] * corr + ps;
      Ps[(4 * ty + i) * (TK + 4) + tx] = p0;
      Ps[(4 * ty + i) * (TK + 4) + tx + 16] = p1;
#pragma unroll
      for (int c = 0; c < 4 * NV; ++c) o[i][c] *= corr;
#pragma unroll
      for (int c = 0; c < 4; ++c) ol[i][c] *= corr;
    }
    __syncwarp();   // a row's P is written and read by the same half warp
    for (int t = 0; t < TK; t += 4) {
      float pr[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(Ps + (4 * ty + i) * (TK + 4) + t);
        pr[i][0] = v.x; pr[i][1] = v.y; pr[i][2] = v.z; pr[i][3] = v.w;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const float4 v = *reinterpret_cast<const float4*>(Vs + (t + u) * LD + 64 * k + 4 * tx);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o[i][4 * k] = fmaf(pr[i][u], v.x, o[i][4 * k]);
            o[i][4 * k + 1] = fmaf(pr[i][u], v.y, o[i][4 * k + 1]);
            o[i][4 * k + 2] = fmaf(pr[i][u], v.z, o[i][4 * k + 2]);
            o[i][4 * k + 3] = fmaf(pr[i][u], v.w, o[i][4 * k + 3]);
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (tx + 16 * k < R) {
            const float lv = LRs[(t + u) * LDR + R + tx + 16 * k];
#pragma unroll
            for (int i = 0; i < 4; ++i) ol[i][k] = fmaf(pr[i][u], lv, ol[i][k]);
          }
      }
    }
  }

  // ---- this split's partial: [RB][D + R], then (m, l) per row
  __syncthreads();
  float* part = reinterpret_cast<float*>(smem);
  const int W = D + R;
  float* pml = part + RB * W;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 4 * ty + i;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int c = 0; c < 4; ++c) part[row * W + 64 * k + 4 * tx + c] = o[i][4 * k + c];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (tx + 16 * k < R) part[row * W + D + tx + 16 * k] = ol[i][k];
    if (tx == 0) {
      pml[2 * row] = mrow[i];
      pml[2 * row + 1] = lrow[i];
    }
  }
  ptx::cluster_sync_all();
  // ---- merge: this CTA's share of the rows, a warp a row
  const uint32_t part_u = ptx::smem_u32(part), pml_u = ptx::smem_u32(pml);
  const int share = (rows + S - 1) / S;
  const int r1 = min(rows, (split + 1) * share);
  for (int row = split * share + warp; row < r1; row += NTH / 32) {
    const float mk = lane < S ? ptx::dsmem_ld(ptx::dsmem_addr(pml_u + 8 * row, lane)) : -INFINITY;
    const float lk = lane < S ? ptx::dsmem_ld(ptx::dsmem_addr(pml_u + 8 * row + 4, lane)) : 0.f;
    float mx = mk;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
    const float wk = mk == -INFINITY ? 0.f : expf(mk - mx);
    float lt = wk * lk;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, k);
    const float inv = lt > 0.f ? 1.f / lt : 0.f;
    float acc[2 * NV], lo[2];
#pragma unroll
    for (int c = 0; c < 2 * NV; ++c) acc[c] = 0.f;
    lo[0] = lo[1] = 0.f;
    for (int k = 0; k < S; ++k) {
      const float w = __shfl_sync(0xffffffffu, wk, k);
      if (w == 0.f) continue;
      const uint32_t rk = ptx::dsmem_addr(part_u + 4 * row * W, k);
#pragma unroll
      for (int c = 0; c < 2 * NV; ++c) acc[c] = fmaf(w, ptx::dsmem_ld(rk + 4 * (lane + 32 * c)), acc[c]);
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (lane + 32 * c < R) lo[c] = fmaf(w, ptx::dsmem_ld(rk + 4 * (D + lane + 32 * c)), lo[c]);
    }
    float z[2 * NV];
#pragma unroll
    for (int c = 0; c < 2 * NV; ++c) z[c] = 0.f;
    for (int j = 0; j < R; ++j) {
      const float lv = __shfl_sync(0xffffffffu, j < 32 ? lo[0] : lo[1], j & 31);
#pragma unroll
      for (int c = 0; c < 2 * NV; ++c) z[c] = fmaf(lv, Bv[j * ldB + lane + 32 * c], z[c]);
    }
    OUT* out = reinterpret_cast<OUT*>(p.out) + ((qrow0 + row / g) * p.n_q + kvh * g + row % g) * D;
#pragma unroll
    for (int c = 0; c < 2 * NV; ++c) out[lane + 32 * c] = from_f32<OUT>(fmaf(p.s, z[c], acc[c]) * inv);
  }
  ptx::cluster_sync_all();   // the partials are read before any CTA of the cluster exits
}

template <typename OUT, int D>
cudaError_t launch_ts(const AttnParams& pin, const TreeParams& tp, cudaStream_t st) {
  AttnParams p = pin;
  RopeTheta rt = {};
  rope_thetas(p.rope_base, D, &rt);
  const TsCfg<D> L(p.r);
  const auto kern = attn_tree_simt_kernel<OUT, D>;
  cudaError_t e = allow_smem(kern, L.total);
  if (e != cudaSuccess) return e;
  // splits: enough CTAs for two an SM, at least a tile a split, at most the
  // portable cluster size
  const int QB = RB / p.g, nblk = (p.n_q_tokens + QB - 1) / QB;
  const int64_t units = (int64_t)nblk * p.n_agents * p.n_kv * p.n_seqs;
  const int64_t tiles = (p.max_kv_len + TK - 1) / TK + 1;
  const int sms = device_sms();
  int S = 1;
  while (S < 8 && units * S < 2 * sms && tiles > S) S *= 2;
  p.n_splits = S;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)S, (unsigned)(nblk * p.n_agents * p.n_kv), (unsigned)p.n_seqs);
  cfg.blockDim = dim3(NTH);
  cfg.dynamicSmemBytes = L.total;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, p, tp, rt);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename OUT>
cudaError_t launch_ts_d(const AttnParams& p, const TreeParams& tp, cudaStream_t st) {
  return p.d == 128 ? launch_ts<OUT, 128>(p, tp, st) : launch_ts<OUT, 64>(p, tp, st);
}

}  // namespace

bool attn_tree_simt_supported(const AttnParams& p) {
  if (p.g > RB || p.n_seqs > 65535) return false;
  const int QB = RB / p.g;
  return (int64_t)((p.n_q_tokens + QB - 1) / QB) * p.n_agents * p.n_kv <= 65535;
}

cudaError_t launch_attn_tree_simt(const AttnParams& p, const TreeParams& tp, la_dtype out, cudaStream_t st) {
  return out == LA_F32 ? launch_ts_d<float>(p, tp, st) : launch_ts_d<__nv_bfloat16>(p, tp, st);
}

}  // namespace la

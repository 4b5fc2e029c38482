// lora_qk_norm_rope: per-head RMS norm of new queries and keys, the rotation
// at their positions and the cache rows, one pass.
//
//   q_out[s][a][j][h] = RoPE_pos( q / sqrt(mean(q^2) + eps) * w_q )
//   k_base row        = RoPE_pos( k / sqrt(mean(k^2) + eps) * w_k ),  v_base row = v
// pos = C + depth(j), row = C + t nodes + j (tree.cuh); without a norm weight
// the norm is left out.  Memory-bound: every value is read once and written
// once.  A head takes d / 16 lanes, 8 adjacent frequencies a lane (16-byte
// accesses at i and i + d/2 in bf16), so a pair is turned inside one thread and
// the sum of squares needs three shuffles.  (cos, sin) are formed once per token
// and CTA (angle reduced in fp64), shared by all its heads, and laid down with the norm
// weights folded in.  Two head rows in flight a thread, 64 registers and eight CTAs
// of 128 threads an SM measured best: 4096 tokens x (4 agents x 32 + 8) heads, 302 MB,
// 57.8 us (5.2 TB/s, 80 % of the copy rate); four CTAs of 256 threads 63.0 us, four
// rows at 80 registers 66.0 us, two sets of rows taking turns 75-82 us (they spill).
// A verification step's 16 tokens take 3.5 us, which is latency.
#include <cmath>

#include "bf16_common.cuh"
#include "la_internal.cuh"
#include "tree.cuh"

namespace la {
namespace {

constexpr int NTH = 128;
constexpr int kMaxTB = 2;   // tokens per CTA
constexpr int kUnr = 2;     // head rows a thread has in flight

struct QkParams {
  int n_seqs, n_agents, n_tok, n_q, n_kv;
  float eps;
  const void* q;
  int64_t q_seq, q_agent, q_tok;
  void* q_out;
  const void* k;
  const void* v;
  int64_t kv_in_seq, kv_in_tree, kv_in_tok;
  const void* w_q;
  const void* w_k;
  void* k_base;
  void* v_base;
  int64_t kv_seq, kv_head, kv_tok;
  const int32_t* kv_len;
  int64_t max_kv_len;
  int q_slots;   // n_agents, or 0 without queries
  int tb;        // tokens per CTA
  int* err;
};

template <typename IO>
struct Raw8;   // 8 adjacent elements as loaded
template <>
struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = u; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    u = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void store(float* p) const {
    *reinterpret_cast<float4*>(p) = a;
    *reinterpret_cast<float4*>(p + 4) = b;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
};

template <typename IO, int D>
__global__ void __launch_bounds__(NTH, 8)
    qk_norm_rope_kernel(const QkParams p, const TreeParams tp, const __grid_constant__ RopeTheta rt) {
  constexpr int LPH = D / 16, RPP = NTH / LPH;   // lanes per head row, head rows a pass
  // per token the turned pair's four factors: w1 cos, w2 sin, w2 cos, w1 sin
  // (a lane's 8 frequencies: 16-byte reads)
  __shared__ __align__(16) float tab[kMaxTB][4][D / 2];
  __shared__ uint64_t masks[kTreeMaxNodes];
  __shared__ int s_ok;
  const int tid = threadIdx.x, seq = blockIdx.z, slot = blockIdx.y;
  const bool isq = slot < p.q_slots;
  const int unit = isq ? slot : slot - p.q_slots;                   // agent, or tree
  const int tree = isq ? (tp.n_trees > 1 ? unit : 0) : unit;
  const int tok0 = blockIdx.x * p.tb;
  const int H = isq ? p.n_q : p.n_kv;
  const int sub = tid % LPH, slice = tid / LPH;
  const IO* src = isq ? reinterpret_cast<const IO*>(p.q) + seq * p.q_seq + unit * p.q_agent
                      : reinterpret_cast<const IO*>(p.k) + seq * p.kv_in_seq + unit * p.kv_in_tree;
  const int64_t src_tok = isq ? p.q_tok : p.kv_in_tok;
  const int slots = min(p.tb, p.n_tok - tok0) * H;   // head rows of the CTA's tokens, live or not
  auto token = [&](int idx) {   // idx / H for idx < kMaxTB H
    int t = 0;
#pragma unroll
    for (int k = 1; k < kMaxTB; ++k) t += idx >= k * H;
    return t;
  };
  Raw8<IO> lo[kUnr], hi[kUnr];
  auto fetch = [&](int base) {
#pragma unroll
    for (int u = 0; u < kUnr; ++u) {
      const int idx = base + u * RPP + slice;
      if (idx < slots) {
        const int t = token(idx);
        const IO* x = src + (tok0 + t) * src_tok + (idx - t * H) * D + 8 * sub;
        lo[u].load(x);
        hi[u].load(x + D / 2);
      }
    }
  };
  fetch(0);   // the first rows travel while the lengths are read
  const int64_t C = p.kv_len[seq];
  const int m = tp.tree_len ? tp.tree_len[seq * tp.n_trees + tree] : p.n_tok;
  if (C < 0 || C + (int64_t)tp.n_trees * p.n_tok > p.max_kv_len) {
    if (tid == 0) atomicOr(p.err, kDevKvLen);
    return;
  }
  if (m < 0 || m > p.n_tok) {
    if (tid == 0) atomicOr(p.err, kDevTree);
    return;
  }
  const int ntok = min(p.tb, m - tok0);
  if (ntok <= 0) return;
  const int total = ntok * H;
  const IO* wn = reinterpret_cast<const IO*>(isq ? p.w_q : p.w_k);
  if (tp.parent) {
    if (tid < 32) {
      const bool ok = tree_masks_warp(tp.parent + ((int64_t)seq * tp.n_trees + tree) * p.n_tok, p.n_tok, m, masks);
      if (tid == 0) s_ok = ok;
    }
    __syncthreads();
    if (!s_ok) {
      if (tid == 0) atomicOr(p.err, kDevTree);
      return;
    }
  }
  for (int i = tid; i < ntok * (D / 2); i += NTH) {
    const int t = i / (D / 2), f = i % (D / 2), j = tok0 + t;
    const float2 cs = rope_cs_exact(C + (tp.parent ? __popcll(masks[j]) - 1 : j), rt.theta[f]);
    const float a = wn ? to_f32(wn[f]) : 1.f, b = wn ? to_f32(wn[f + D / 2]) : 1.f;
    tab[t][0][f] = a * cs.x;
    tab[t][1][f] = b * cs.y;
    tab[t][2][f] = b * cs.x;
    tab[t][3][f] = a * cs.y;
  }
  __syncthreads();
  for (int base = 0; base < total; base += kUnr * RPP) {
    if (base > 0) fetch(base);
#pragma unroll
    for (int u = 0; u < kUnr; ++u) {
      const int idx = base + u * RPP + slice;
      float x1[8], x2[8];
      float ss = 0.f;
      if (idx < total) {
        lo[u].get(x1);
        hi[u].get(x2);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x1[i], x1[i], fmaf(x2[i], x2[i], ss));
      }
      float inv = 1.f;
      if (wn) {   // the same branch in every thread of the CTA
#pragma unroll
        for (int k = LPH / 2; k > 0; k >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, k);
        inv = rsqrtf(ss * (1.f / D) + p.eps);
      }
      if (idx >= total) continue;
      const int t = token(idx), h = idx - t * H;
      float y1[8], y2[8];
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        float f[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<float4*>(f[k]) = *reinterpret_cast<const float4*>(&tab[t][k][8 * sub + i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = x1[i + e] * inv, b = x2[i + e] * inv;
          y1[i + e] = a * f[0][e] - b * f[1][e];
          y2[i + e] = b * f[2][e] + a * f[3][e];
        }
      }
      IO* dst = isq ? reinterpret_cast<IO*>(p.q_out) +
                          ((((int64_t)seq * p.n_agents + unit) * p.n_tok + tok0 + t) * p.n_q + h) * D
                    : reinterpret_cast<IO*>(p.k_base) + seq * p.kv_seq + h * p.kv_head +
                          (C + (int64_t)tree * p.n_tok + tok0 + t) * p.kv_tok;
      lo[u].set(y1);
      hi[u].set(y2);
      lo[u].store(dst + 8 * sub);
      hi[u].store(dst + 8 * sub + D / 2);
    }
  }
  if (!isq && p.v) {   // the value rows, as they are
    const IO* vs = reinterpret_cast<const IO*>(p.v) + seq * p.kv_in_seq + unit * p.kv_in_tree;
    for (int idx = slice; idx < total; idx += RPP) {
      const int t = token(idx), h = idx - t * H;
      const IO* x = vs + (tok0 + t) * p.kv_in_tok + h * D + 8 * sub;
      IO* dst = reinterpret_cast<IO*>(p.v_base) + seq * p.kv_seq + h * p.kv_head +
                (C + (int64_t)tree * p.n_tok + tok0 + t) * p.kv_tok + 8 * sub;
      Raw8<IO> a, b;
      a.load(x);
      b.load(x + D / 2);
      a.store(dst);
      b.store(dst + D / 2);
    }
  }
}

template <typename IO, int D>
cudaError_t launch_qk(const QkParams& pin, const TreeParams& tp, double rope_base, cudaStream_t st) {
  QkParams p = pin;
  RopeTheta rt = {};
  rope_thetas(rope_base, D, &rt);
  const int slots = p.q_slots + (p.k ? tp.n_trees : 0);
  // two tokens a CTA (one angle a thread at d = 128), one where that would leave
  // SMs without a CTA
  p.tb = (int64_t)((p.n_tok + kMaxTB - 1) / kMaxTB) * slots * p.n_seqs >= device_sms() ? kMaxTB : 1;
  const dim3 grid((unsigned)((p.n_tok + p.tb - 1) / p.tb), (unsigned)slots, (unsigned)p.n_seqs);
  qk_norm_rope_kernel<IO, D><<<grid, NTH, 0, st>>>(p, tp, rt);
  return cudaGetLastError();
}

bool aligned(const void* ptr, uintptr_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) == 0; }

}  // namespace
}  // namespace la

extern "C" la_status lora_qk_norm_rope(const la_qk_args* a, const la_tree_args* tree, la_stream_t stream) {
  using namespace la;
  if (!a || (a->dtype != LA_F32 && a->dtype != LA_BF16)) return LA_ERR_INVALID_ARG;
  if (a->n_seqs < 0 || a->n_agents < 1 || a->n_tokens < 0 || a->n_q_heads < 1 || a->n_kv_heads < 1 ||
      a->L_max < 1 || a->max_kv_len < 1)
    return LA_ERR_INVALID_ARG;
  if (a->head_dim != 64 && a->head_dim != 128) return LA_ERR_UNSUPPORTED;
  if (!std::isfinite(a->rope_base) || !(a->rope_base > 1.0) || !std::isfinite(a->eps) || a->eps < 0.f)
    return LA_ERR_INVALID_ARG;
  const int32_t n_trees = tree ? tree->n_trees : 1;
  if (n_trees != 1 && n_trees != a->n_agents) return LA_ERR_INVALID_ARG;
  if (tree && tree->parent && a->n_tokens > kTreeMaxNodes) return LA_ERR_UNSUPPORTED;
  if (tree && (!aligned(tree->parent, 4) || !aligned(tree->tree_len, 4))) return LA_ERR_INVALID_ARG;
  if ((!a->q && !a->k) || !a->kv_len || !aligned(a->kv_len, 4)) return LA_ERR_INVALID_ARG;
  if ((a->q == nullptr) != (a->q_out == nullptr)) return LA_ERR_INVALID_ARG;
  if ((a->k == nullptr) != (a->k_base == nullptr) || (a->v == nullptr) != (a->v_base == nullptr) ||
      (a->v && !a->k))
    return LA_ERR_INVALID_ARG;
  const int64_t es = a->dtype == LA_F32 ? 4 : 2, d = a->head_dim;
  const auto stride_ok = [&](int64_t s) { return s >= 0 && (s * es) % 16 == 0; };
  if (a->q) {
    if (!aligned(a->q, 16) || !aligned(a->q_out, 16) || !aligned(a->w_q, 16)) return LA_ERR_INVALID_ARG;
    if (!stride_ok(a->q_seq_stride) || !stride_ok(a->q_agent_stride) || !stride_ok(a->q_tok_stride) ||
        a->q_tok_stride < a->n_q_heads * d)
      return LA_ERR_INVALID_ARG;
    // q_out is dense: over a strided q its rows would land on rows not read yet
    const int64_t tok = a->n_q_heads * d, agent = a->n_tokens * tok, seq = a->n_agents * agent;
    if (a->q == a->q_out && a->n_tokens > 0 &&
        ((a->n_tokens > 1 && a->q_tok_stride != tok) || (a->n_agents > 1 && a->q_agent_stride != agent) ||
         (a->n_seqs > 1 && a->q_seq_stride != seq)))
      return LA_ERR_INVALID_ARG;
  }
  if (a->k) {
    if (!aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->w_k, 16) || !aligned(a->k_base, 16) ||
        !aligned(a->v_base, 16))
      return LA_ERR_INVALID_ARG;
    if (!stride_ok(a->kv_in_seq_stride) || !stride_ok(a->kv_in_tree_stride) ||
        !stride_ok(a->kv_in_tok_stride) || a->kv_in_tok_stride < a->n_kv_heads * d)
      return LA_ERR_INVALID_ARG;
    if (!stride_ok(a->kv_seq_stride) || !stride_ok(a->kv_head_stride) || !stride_ok(a->kv_tok_stride) ||
        a->kv_tok_stride < d)
      return LA_ERR_INVALID_ARG;
  }
  if (a->max_kv_len > a->L_max || (int64_t)n_trees * a->n_tokens > a->max_kv_len) return LA_ERR_CAPACITY;
  if (a->n_seqs > 65535 || (int64_t)a->n_agents + n_trees > 65535 || a->n_q_heads > 65535 || a->n_kv_heads > 65535)
    return LA_ERR_UNSUPPORTED;
  if (a->n_seqs == 0 || a->n_tokens == 0) return LA_OK;
  QkParams p = {};
  p.n_seqs = a->n_seqs; p.n_agents = a->n_agents; p.n_tok = a->n_tokens;
  p.n_q = a->n_q_heads; p.n_kv = a->n_kv_heads;
  p.eps = a->eps;
  p.q = a->q; p.q_seq = a->q_seq_stride; p.q_agent = a->q_agent_stride; p.q_tok = a->q_tok_stride;
  p.q_out = a->q_out;
  p.k = a->k; p.v = a->v;
  p.kv_in_seq = a->kv_in_seq_stride; p.kv_in_tree = a->kv_in_tree_stride; p.kv_in_tok = a->kv_in_tok_stride;
  p.w_q = a->w_q; p.w_k = a->w_k;
  p.k_base = a->k_base; p.v_base = a->v_base;
  p.kv_seq = a->kv_seq_stride; p.kv_head = a->kv_head_stride; p.kv_tok = a->kv_tok_stride;
  p.kv_len = a->kv_len; p.max_kv_len = a->max_kv_len;
  p.q_slots = a->q ? a->n_agents : 0;
  p.err = error_word_ptr();
  if (!p.err) return LA_ERR_CUDA;
  TreeParams tp = {};
  if (tree) {
    tp.parent = tree->parent;
    tp.tree_len = tree->tree_len;
  }
  tp.n_trees = n_trees;
  tp.nodes = a->n_tokens;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a->dtype == LA_BF16)
    e = d == 128 ? launch_qk<__nv_bfloat16, 128>(p, tp, a->rope_base, st)
                 : launch_qk<__nv_bfloat16, 64>(p, tp, a->rope_base, st);
  else
    e = d == 128 ? launch_qk<float, 128>(p, tp, a->rope_base, st)
                 : launch_qk<float, 64>(p, tp, a->rope_base, st);
  return e == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

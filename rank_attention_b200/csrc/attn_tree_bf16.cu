// Attention of drafted trees on the tcgen05 tensor cores (bf16 storage, fp32
// accumulation in TMEM).
//
// One CTA = 128 query rows (nodes x the GQA group's heads, and without a key
// delta the agents too: their keys are the same then) of one (sequence, KV
// head), and one split of the keys; the splits of a block are a thread-block
// cluster and merge over distributed shared memory.  Keys stream in tiles of
// 128: the committed context, then one tile with the tree's own nodes.  Per tile
//   dK  = LRk B_k^a                     tcgen05, 32 frequencies at a time
//   K^a = K_base + s R(k0) R(j) dK      CUDA cores, in fp16 over K_base
//   S   = Q K^a^T                       tcgen05, Q (fp16) read from TMEM
//   P   = exp2(S log2e scale - m)       CUDA cores, bf16 to TMEM
//   [O | O_lr] += P [V_base | LRv]      tcgen05, P read from TMEM
// and once per row out = (O + s O_lr B_v^a) / l.  R(j) turns by the key's
// offset in its tile, or by a node's depth in the drafted tile (k0 = C there).
// Without a key delta (KEYS = false) K_base is the operand as it lies, in bf16,
// and the scores are double-buffered, P lying over the scores it came from.
//
// Warps: eight softmax warps (two per TMEM sub-partition, 64 keys each), eight
// build warps (16 keys each), and one warp each to issue S and P V, to load, to
// issue dK (a part's MMA runs while the build turns the part before), and to form the anchors
// s R(k0) in fp64.  The running maximum is rescaled lazily (O and l corrected
// only when a row's maximum grows by more than 2^8).
#include <cmath>

#include "attn_tc_common.cuh"
#include "bf16_common.cuh"
#include "la_internal.cuh"
#include "ptx.cuh"
#include "tree.cuh"

namespace la {
namespace {

constexpr int KT = 128;    // keys per tile
constexpr int QM = 128;    // query rows per CTA
constexpr int NSM = 8;     // softmax warps
constexpr int kMaxSplits = 8;   // the portable cluster size
constexpr int kPolyEvery = 4;   // every 4th pair of exponentials on the FMA pipe
constexpr int BAR_PAIR = 2;     // named barriers 2..5: the two warps of a row block

// TMEM columns.  With a key delta: Q, dK (64 columns: 32 frequencies), S, P, O
// and O_lr behind it; without: Q, S twice (P over each), O and O_lr.
constexpr int T_Q = 0, T_DK = 64, T_P = 256, T_O = 320, T_COLS = 512;

template <int D, int R, bool KEYS>
struct TCfg {
  static constexpr int NB = KEYS ? 8 : 0;                       // build warps
  static constexpr int NTHR = 32 * (NSM + NB + 4);
  static constexpr int NH = D / 64;                             // parts of 32 frequencies
  static constexpr int LR_ROWB = R * 2;
  static constexpr uint32_t LR_LAYOUT = LR_ROWB == 128 ? 2u : (LR_ROWB == 64 ? 4u : 6u);
  static constexpr int KV = KT * D * 2;                         // a K or V tile
  static constexpr int LRK = KEYS ? KT * R * 2 : 0;             // a tile's LRk columns
  // V_base and LRv: LRv as a third 64-column group of the same swizzled layout
  // (columns past LRv are the tensor map's zero fill), so that one MMA of N = D + R
  // covers P V and P LRv
  static constexpr int VST = KV + KT * 128;
  static constexpr int NK = 3, NL = 2;
  static constexpr int NV = KEYS && D == 128 && R == 64 ? 1 : 2;   // what 227 KB leave
  static constexpr int OFF_V = NK * KV;
  static constexpr int OFF_LRK = OFF_V + NV * VST;
  static constexpr int OFF_BK = OFF_LRK + NL * LRK;
  static constexpr int OFF_MISC = OFF_BK + (KEYS ? R * D * 2 : 0);
  // misc: anchors [3][64] float2, exchange [2][8][32] float, masks [64] u64, 32 mbarriers,
  // the TMEM slot, theta [64] float
  static constexpr int MISC = 1536 + 2048 + 512 + 256 + 16 + 256;
  // at least more than half an SM's, so that one CTA is resident: two would wait
  // for each other's TMEM across clusters
  static constexpr int NEED = 1024 + OFF_MISC + MISC;
  static constexpr int SMEM = NEED > 120 * 1024 ? NEED : 120 * 1024;
  // the partial (O, O_lr, m and l) over the drained stages
  static constexpr int P_OL = QM * D * 4, P_ML = P_OL + QM * R * 4;
  static_assert(P_ML + QM * 8 <= OFF_LRK, "the partial lies over the stages");
  static_assert(SMEM <= 227 * 1024, "shared memory of one CTA");
  // score buffers
  __host__ __device__ static constexpr int t_s(int b) { return KEYS ? 128 : 64 + 128 * b; }
  __host__ __device__ static constexpr int t_p(int b) { return KEYS ? T_P : 64 + 128 * b; }
};

// the split's registers: at 640 threads a CTA launches with 96 a thread
// (61,440); 2 x 112 (softmax) + 2 x 112 (build) + 32 = 480 x 128 threads uses all
constexpr int kLaunchRegs = 96;
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int D, int R, bool KEYS>
__global__ void __launch_bounds__(TCfg<D, R, KEYS>::NTHR, 1)
    attn_tree_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ CUtensorMap tmL, const __grid_constant__ CUtensorMap tmLk,
                        const AttnParams p, const TreeParams tp,
                        const __grid_constant__ RopeTheta rt, const int pooled, const int fold) {
  using C_ = TCfg<D, R, KEYS>;
  constexpr int NK = C_::NK, NV = C_::NV, NL = C_::NL, NH = C_::NH, H2 = D / 2, T_OL = T_O + D;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const uint32_t k_u = sb, v_u = sb + C_::OFF_V, lrk_u = sb + C_::OFF_LRK, bk_u = sb + C_::OFF_BK;
  unsigned char* misc = smem + C_::OFF_MISC;
  float2* anc = reinterpret_cast<float2*>(misc);
  float* xch = reinterpret_cast<float*>(misc + 1536);
  uint64_t* masks = reinterpret_cast<uint64_t*>(misc + 3584);
  const uint32_t b0 = smem_u32(misc + 4096);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(misc + 4096 + 256);
  float* thf = reinterpret_cast<float*>(misc + 4096 + 272);
  __shared__ int s_bad, s_fail;

  auto kfull = [&](int s) { return b0 + 8 * s; };
  auto kfree = [&](int s) { return b0 + 24 + 8 * s; };
  auto kaready = [&](int s) { return b0 + 48 + 8 * s; };
  auto vfull = [&](int s) { return b0 + 96 + 8 * s; };
  auto vfree = [&](int s) { return b0 + 112 + 8 * s; };
  auto lrfull = [&](int s) { return b0 + 128 + 8 * s; };
  auto lrfree = [&](int s) { return b0 + 144 + 8 * s; };
  auto sfull = [&](int s) { return b0 + 160 + 8 * s; };
  auto pfull = [&](int s) { return b0 + 176 + 8 * s; };
  const uint32_t staken = b0 + 192, pvdone = b0 + 200, qready = b0 + 208, dkfull = b0 + 216, dkfree = b0 + 224;

  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  constexpr int W0 = NSM + C_::NB;   // MMA, loads, dK, anchors
  const int g = p.g, n = tp.nodes;
  const int seq = blockIdx.z, split = blockIdx.x, S = p.n_splits;
  int y = blockIdx.y, agent0 = 0;
  if (!pooled) {
    agent0 = y % p.n_agents;
    y /= p.n_agents;
  }
  const int kvh = y % p.n_kv, blk = y / p.n_kv;
  const int tree = tp.n_trees > 1 ? agent0 : 0;
  const int lra = p.lr_agent ? agent0 : 0;

  pdl_wait();   // what the kernels before wrote is read from here on
  // the same values, so the same branches, in the whole cluster
  const int64_t C = p.kv_len[seq];
  const int m = tp.tree_len ? tp.tree_len[seq * tp.n_trees + tree] : n;
  constexpr int NBK = KEYS ? (R * D / 8 + C_::NTHR - 1) / C_::NTHR : 0;
  uint4 bkv[KEYS ? NBK : 1];
  if constexpr (KEYS) {   // B_k^a's rows, read behind the lengths (rows past r, at r = 8, are zero)
    const __nv_bfloat16* Bk = reinterpret_cast<const __nv_bfloat16*>(p.B_k) +
                              (int64_t)agent0 * p.r * p.n_kv * D + kvh * D;
#pragma unroll
    for (int u = 0; u < NBK; ++u) {
      const int i = tid + u * C_::NTHR, j = i / (D / 8);
      bkv[u] = make_uint4(0, 0, 0, 0);
      if (j < p.r) bkv[u] = *reinterpret_cast<const uint4*>(Bk + (int64_t)j * p.n_kv * D + 8 * (i % (D / 8)));
    }
  }
  const bool kv_ok = C >= 0 && C + (int64_t)tp.n_trees * n <= p.max_kv_len;
  const bool tree_ok = m >= 0 && m <= n;
  const int per = m * g;   // an agent's live rows, node by node
  const int rows = min(QM, (pooled ? p.n_agents * per : per) - QM * blk);
  if (!kv_ok || !tree_ok || rows <= 0) {
    if (tid == 0 && !(kv_ok && tree_ok)) atomicOr(p.err, kv_ok ? kDevTree : kDevKvLen);
    return;
  }
  const int Nc = (int)((C + KT - 1) / KT), N = Nc + 1;
  const int n0 = (int)((int64_t)N * split / S), NT = (int)((int64_t)N * (split + 1) / S) - n0;

  // loads: K_base, LRk and V_base with LRv of the CTA's tile i
  auto row0 = [&](int i) { return n0 + i == Nc ? (int)(C + (int64_t)tree * n) : (n0 + i) * KT; };
  auto load_k = [&](int i) {
    const uint32_t dst = k_u + (i % NK) * C_::KV, bar = kfull(i % NK);
    mbar_expect_tx(bar, (uint32_t)C_::KV);
#pragma unroll
    for (int b = 0; b < D / 64; ++b) tma_load_4d(dst + b * KT * 128, &tmK, bar, 64 * b, row0(i), kvh, seq);
  };
  auto load_lrk = [&](int i) {
    const uint32_t bar = lrfull(i % NL);
    mbar_expect_tx(bar, (uint32_t)C_::LRK);
    tma_load_4d(lrk_u + (i % NL) * C_::LRK, &tmLk, bar, 0, row0(i), seq, lra);
  };
  auto load_v = [&](int i) {
    const uint32_t dst = v_u + (i % NV) * C_::VST, bar = vfull(i % NV);
    mbar_expect_tx(bar, (uint32_t)C_::VST);
#pragma unroll
    for (int b = 0; b < D / 64; ++b) tma_load_4d(dst + b * KT * 128, &tmV, bar, 64 * b, row0(i), kvh, seq);
    tma_load_4d(dst + C_::KV, &tmL, bar, p.r < 16 ? 0 : R, row0(i), seq, lra);   // r = 8: one 16-wide row holds both
  };

  if (w == 0) {
    const bool ok = tree_masks_warp(
        tp.parent ? tp.parent + ((int64_t)seq * tp.n_trees + tree) * n : nullptr, n, m, masks);
    if (lane == 0) s_bad = !ok;
  }
  if (w == W0) tmem_alloc(smem_u32(tslot), T_COLS);
  if (KEYS && w == W0 + 3)
    for (int f = lane; f < H2; f += 32) thf[f] = rt.thetaf[f];
  if (w == W0 + 1 && lane == 0) {
    s_fail = 0;
    for (int s = 0; s < 3; ++s) {
      mbar_init(kfull(s), KEYS ? 2 : 1);   // the loads, and with a key delta the tile's anchors
      mbar_init(kfree(s), 1);
      mbar_init(kaready(s), 8);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(vfull(s), 1);
      mbar_init(vfree(s), 1);
      mbar_init(lrfull(s), 1);
      mbar_init(lrfree(s), 1);
      mbar_init(sfull(s), 1);
      mbar_init(pfull(s), NSM);
    }
    mbar_init(staken, NSM);
    mbar_init(pvdone, 1);
    mbar_init(qready, NSM);
    mbar_init(dkfull, 1);
    mbar_init(dkfree, 8);
    fence_mbar_init();
    for (int i = 0; i < min(NK, NT); ++i) {
      if (KEYS && i < NL) load_lrk(i);
      load_k(i);
      if (i < NV) load_v(i);
    }
  }
  if constexpr (KEYS) {
    // B_k^a as the dK MMA's operand: a part is R rows of 32 + 32 columns (a
    // frequency's two halves), 128-byte swizzle
#pragma unroll
    for (int u = 0; u < NBK; ++u) {
      const int i = tid + u * C_::NTHR, j = i / (D / 8), col = 8 * (i % (D / 8)), f = col % H2;
      if (i < R * D / 8)
        sts128(bk_u + (uint32_t)(f / 32) * (R * 128) + tile_off<64, R>(j, (col / H2) * 32 + f % 32), bkv[u].x,
               bkv[u].y, bkv[u].z, bkv[u].w);
    }
    fence_proxy_async_smem();
  }
  // offset of row r_ of the block in q and out
  const int64_t q_agent = (int64_t)n * p.n_q * D;
  auto locate = [&](int r_, int& node, int& ag) {
    int R_ = QM * blk + r_;
    ag = agent0;
    if (pooled) {
      ag = R_ / per;
      R_ -= ag * per;
    }
    node = R_ / g;
    return ((int64_t)seq * p.n_agents + ag) * q_agent + ((int64_t)node * p.n_q + kvh * g + R_ % g) * D;
  };
  // softmax warps: this thread's query row, in TMEM lane 32 sp + lane, and its half
  // of a tile's keys.  Folded (at most 64 rows): lanes 64.. repeat the rows and take
  // the keys 64.. of every tile for themselves, with a maximum, a sum and outputs of
  // their own that the merge joins like those of another split; one warp (ch = 0) a
  // sub-partition then works on scores.  Otherwise two warps share each row's keys.
  const int sp = w & 3, ch = w >> 2;
  const int tl = 32 * sp + lane;
  const int row = fold ? tl & 63 : tl;
  const int kh = fold ? tl >> 6 : ch;                     // half of the keys
  const bool has = (fold ? 32 * (sp & 1) : 32 * sp) < rows;   // these lanes have rows
  const bool live = has && !(fold && ch == 1);            // this warp has scores to weigh
  uint32_t qv[D / 4];
  int qnode = 0;
  if (w < NSM && has) {
    int ag;
    const int64_t off = locate(row < rows ? row : 0, qnode, ag);
    const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.q) + off + H2 * ch);
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      const uint4 v = row < rows ? src[c] : make_uint4(0, 0, 0, 0);
      qv[4 * c] = v.x; qv[4 * c + 1] = v.y; qv[4 * c + 2] = v.z; qv[4 * c + 3] = v.w;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  int fail = 0;

  if (!s_bad) {
    if (w >= W0) {
      if constexpr (KEYS) regs_dec<32>();
      if (w == W0 && NT > 0) {
        // ========================================================== S and P V
        // (the whole warp walks the loop and one elected lane issues: descriptors
        // stay in uniform registers, about 75 cycles an MMA instead of 95)
        constexpr uint32_t ID_S = KEYS ? umma_idesc_f16(QM, KT, 0, 0) : umma_idesc_bf16(QM, KT, 0, 0);
        constexpr uint32_t ID_PV = umma_idesc_bf16(QM, D + R, 0, 1);
        const uint64_t dK = umma_desc(k_u, 16, 1024, 2);
        const uint64_t dV = umma_desc(v_u, KT * 128, 1024, 2);
        auto mma_pv = [&](int i) {   // O, O_lr += P [V_base | LRv]
          const int vs = i % NV;
          if (!mbar_wait(pfull(i & 1), (i >> 1) & 1)) fail = 1;
          if (!mbar_wait(vfull(vs), (i / NV) & 1)) fail = 1;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t vd = umma_desc_add(dV, vs * C_::VST);
            const uint32_t tP = tmem + C_::t_p(i & 1), acc = i > 0 ? 1u : 0u;
#pragma unroll
            for (int ks = 0; ks < KT / 16; ++ks)
              umma_bf16_ts(tmem + T_O, tP + ks * 8, umma_desc_add(vd, ks * 16 * 128), ID_PV, ks > 0 ? 1u : acc);
            umma_commit(pvdone);
            umma_commit(vfree(vs));
          }
          __syncwarp();
        };
        if (!mbar_wait(qready, 0)) fail = 1;
        int ks_ = 0, kp = 0;
        for (int i = 0; i < NT; ++i) {
          if (KEYS) {
            if (!mbar_wait(kaready(ks_), kp)) fail = 1;
            if (i > 0 && !mbar_wait(staken, (i - 1) & 1)) fail = 1;
          } else {
            if (!mbar_wait(kfull(ks_), kp)) fail = 1;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t kd = umma_desc_add(dK, ks_ * C_::KV);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              umma_bf16_ts(tmem + C_::t_s(i & 1), tmem + T_Q + kk * 8,
                           umma_desc_add(kd, (kk >> 2) * (KT * 128) + (kk & 3) * 32), ID_S, kk > 0);
            umma_commit(sfull(i & 1));
            umma_commit(kfree(ks_));
          }
          __syncwarp();
          if (++ks_ == NK) { ks_ = 0; kp ^= 1; }
          if (i > 0) mma_pv(i - 1);
        }
        mma_pv(NT - 1);
      } else if (w == W0 + 1 && lane == 0) {
        // ========================================================== loads
        // refills in the order the MMAs free the stages: dK and S of tile i, then P V of tile i - 1
        for (int i = 0; i < NT; ++i) {
          if (KEYS && i + NL < NT) {
            if (!mbar_wait(lrfree(i % NL), (i / NL) & 1)) fail = 1;
            load_lrk(i + NL);
          }
          if (i + NK < NT) {
            if (!mbar_wait(kfree(i % NK), (i / NK) & 1)) fail = 1;
            load_k(i + NK);
          }
          if (i > 0 && i - 1 + NV < NT) {
            if (!mbar_wait(vfree((i - 1) % NV), ((i - 1) / NV) & 1)) fail = 1;
            load_v(i - 1 + NV);
          }
        }
      } else if (KEYS && w == W0 + 2) {
        // ========================================================== dK
        constexpr uint32_t ID_DK = umma_idesc_bf16(KT, 64, 0, 1);
        const uint64_t dLRk = umma_desc(lrk_u, 16, 8 * C_::LR_ROWB, C_::LR_LAYOUT);
        const uint64_t dBk = umma_desc(bk_u, R * 128, 1024, 2);
        for (int i = 0; i < NT; ++i) {
          if (!mbar_wait(lrfull(i % NL), (i / NL) & 1)) fail = 1;
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            const int c = i * NH + h;
            if (c > 0 && !mbar_wait(dkfree, (c - 1) & 1)) fail = 1;
            tc_fence_after();
            if (elect_one()) {
              const uint64_t lr = umma_desc_add(dLRk, (i % NL) * C_::LRK);
#pragma unroll
              for (int ks = 0; ks < R / 16; ++ks)
                umma_bf16(tmem + T_DK, umma_desc_add(lr, ks * 32),
                          umma_desc_add(dBk, h * (R * 128) + ks * 16 * 128), ID_DK, ks > 0);
              umma_commit(dkfull);
              if (h == NH - 1) umma_commit(lrfree(i % NL));
            }
            __syncwarp();
          }
        }
      } else if (KEYS && w == W0 + 3) {
        // ========================================================== anchors s R(k0)
        constexpr int NF = H2 / 32;   // frequencies a lane
        double th[NF];
#pragma unroll
        for (int u = 0; u < NF; ++u) th[u] = rt.theta[lane + 32 * u];
        int ks_ = 0, kp = 1;
        for (int i = 0; i < NT; ++i) {
          if (i >= 3 && !mbar_wait(kaready(ks_), kp)) fail = 1;   // build(i - 3) has read its slot
          const int64_t k0 = n0 + i == Nc ? C : (int64_t)(n0 + i) * KT;
#pragma unroll
          for (int u = 0; u < NF; ++u) {
            const float2 cs = rope_cs_exact(k0, th[u]);
            anc[ks_ * 64 + lane + 32 * u] = make_float2(cs.x * p.s, cs.y * p.s);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(kfull(ks_));
          if (++ks_ == 3) { ks_ = 0; kp ^= 1; }
        }
      }
      __syncwarp();
      cluster_sync_all();
      cluster_sync_all();
    } else {
      if constexpr (KEYS) regs_inc<112>();
      if (KEYS && w >= NSM) {
      // ============================================================ K^a build
      const int gq = lane >> 2, t4 = lane & 3;
      const int kb = 32 * sp + 16 * ((w - NSM) >> 2);   // this warp's 16 keys (its TMEM lanes)
      // R(j) of keys kb + gq (+ 8) as (cos, cos) and (sin, sin) f16 pairs over two
      // adjacent frequencies
      uint32_t RC[2 * NH][2][2], RS[2 * NH][2][2];
      int ks_ = 0, kp = 0;
      for (int i = 0; i < NT; ++i) {
        const bool drafted = n0 + i == Nc;
        if (i == 0 || drafted) {   // the drafted tile, a split's last: offsets are the nodes' depths
          int j0 = kb + gq, j1 = j0 + 8;
          if (drafted) {
            j0 = j0 < m ? __popcll(masks[j0]) - 1 : 0;
            j1 = j1 < m ? __popcll(masks[j1]) - 1 : 0;
          }
#pragma unroll
          for (int q = 0; q < 2 * NH; ++q)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int f = 16 * q + 8 * u + 2 * t4;
              const float th0 = thf[f], th1 = thf[f + 1];
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                const float j = (float)(hh ? j1 : j0);
                const float2 a = sincos_small(j * th0), b = sincos_small(j * th1);
                RC[q][hh][u] = h2_bits(__floats2half2_rn(a.x, b.x));
                RS[q][hh][u] = h2_bits(__floats2half2_rn(a.y, b.y));
              }
            }
        }
        if (!mbar_wait(kfull(ks_), kp)) fail = 1;
        const float2* an = anc + ks_ * 64;
        // this lane's pair of K elements in a 128-byte-swizzled row: key kb + gq
        // (+8), 16-byte chunk (2 q + u) ^ gq, word t4
        const uint32_t rowb = k_u + ks_ * C_::KV + (uint32_t)(kb + gq) * 128 + 4 * t4;
        constexpr uint32_t HI = KT * 128;   // columns + d/2: the next box, or (d = 64) 4 chunks on
        auto at = [&](int q, int u, int hh) { return rowb + hh * 1024 + (uint32_t)(((2 * q + u) ^ gq) << 4); };
        auto hi = [&](uint32_t o) { return D == 128 ? o + HI : o ^ 64; };
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          uint32_t w1[2][2], w2[2][2];   // a quarter's base words, read together
          auto base = [&](int q) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                w1[u][hh] = lds32(at(q, u, hh));
                w2[u][hh] = lds32(hi(at(q, u, hh)));
              }
          };
          if (!mbar_wait(dkfull, (i * NH + h) & 1)) fail = 1;
          tc_fence_after();
          uint32_t xa[2][8], xb[2][8];   // 32 frequencies' two halves
          const uint32_t tl = tmem + T_DK + ((uint32_t)kb << 16);
          tmem_ld16x256_x2(xa[0], tl);
          tmem_ld16x256_x2(xb[0], tl + 32);
          tmem_ld16x256_x2(xa[1], tl + 16);
          tmem_ld16x256_x2(xb[1], tl + 48);
          tmem_wait_ld_regs(xa[0], xb[0]);
          tmem_wait_ld_regs(xa[1], xb[1]);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(dkfree);   // the next part's MMA runs during this part's turn
#pragma unroll
          for (int qq = 0; qq < 2; ++qq) {
            const int q = 2 * h + qq;
            const uint32_t(&xl)[8] = xa[qq];
            const uint32_t(&xh)[8] = xb[qq];
            base(q);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int f = 16 * q + 8 * u + 2 * t4;
              const float4 a = *reinterpret_cast<const float4*>(an + f);   // two adjacent (cos, sin)
              const __half2 ac = __floats2half2_rn(a.x, a.z), as = __floats2half2_rn(a.y, a.w);
              const __half2 nas = __hneg2(as);
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                const __half2 x1 = __floats2half2_rn(__uint_as_float(xl[4 * u + 2 * hh]),
                                                     __uint_as_float(xl[4 * u + 2 * hh + 1]));
                const __half2 x2 = __floats2half2_rn(__uint_as_float(xh[4 * u + 2 * hh]),
                                                     __uint_as_float(xh[4 * u + 2 * hh + 1]));
                const __half2 c = bits_h2(RC[q][hh][u]), sn = bits_h2(RS[q][hh][u]);
                const __half2 y1 = __hfma2(x1, c, __hneg2(__hmul2(x2, sn)));   // R(j) dK
                const __half2 y2 = __hfma2(x2, c, __hmul2(x1, sn));
                // K_base + s R(k0) y, the base added inside the rotation's FMAs
                w1[u][hh] = h2_bits(__hfma2(ac, y1, __hfma2(nas, y2, bf16x2_h2(w1[u][hh]))));
                w2[u][hh] = h2_bits(__hfma2(ac, y2, __hfma2(as, y1, bf16x2_h2(w2[u][hh]))));
              }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                sts32(at(q, u, hh), w1[u][hh]);
                sts32(hi(at(q, u, hh)), w2[u][hh]);
              }
          }
        }
        fence_proxy_async_smem();   // the S MMA reads K^a through the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive(kaready(ks_));
        if (++ks_ == NK) { ks_ = 0; kp ^= 1; }
      }
      // B_v^a for the merge over B_k^a, which the last dK has read
      const __nv_bfloat16* Bv = reinterpret_cast<const __nv_bfloat16*>(p.B_v) +
                                (int64_t)agent0 * p.r * p.n_kv * D + kvh * D;
      for (int i = tid - 32 * NSM; i < p.r * D / 8; i += 256) {
        const uint4 v = *reinterpret_cast<const uint4*>(Bv + (int64_t)(i / (D / 8)) * p.n_kv * D + 8 * (i % (D / 8)));
        sts128(bk_u + 16 * i, v.x, v.y, v.z, v.w);
      }
      } else {
      // ============================================================ softmax
      const uint32_t tlane = (uint32_t)(32 * sp) << 16;
      const uint64_t vis = has && row < rows ? masks[qnode] : 0;   // the drafted nodes this row sees
      if (has) {
        if constexpr (KEYS) {   // fp16 beside the fp16 K^a (bf16 values convert exactly within its range)
#pragma unroll
          for (int c = 0; c < D / 4; ++c) qv[c] = h2_bits(bf16x2_h2(qv[c]));
        }
        if constexpr (D == 128) {
          tmem_st32x32b_x32(tmem + T_Q + (D / 4) * ch + tlane, qv);
        } else {
          tmem_st32x32b_x16(tmem + T_Q + (D / 4) * ch + tlane, qv);
        }
        if (KEYS && fold && ch == 0) {   // no weights for the other half's keys
          uint32_t z[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) z[c] = 0;
          tmem_st32x32b_x32(tmem + T_P + 32 * (1 - kh) + tlane, z);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(qready);

      const float sl2 = p.scale * kLog2e;
      float m_ref = -INFINITY, lsum = 0.f;
      for (int i = 0; i < NT; ++i) {
        const bool drafted = n0 + i == Nc;
        const int cnt = drafted ? m : (int)min((int64_t)KT, C - (int64_t)(n0 + i) * KT);
        const int buf = i & 1;
        if (!mbar_wait(sfull(buf), (i >> 1) & 1)) fail = 1;
        tc_fence_after();
        uint32_t sv[2][32];
        if (live) {
          const uint32_t ts = tmem + C_::t_s(buf) + 64 * kh + tlane;
          tmem_ld32x32b_x32(sv[0], ts);
          tmem_ld32x32b_x32(sv[1], ts + 32);
          tmem_wait_ld_r32(sv[0]);
          tmem_wait_ld_r32(sv[1]);
        }
        if constexpr (KEYS) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(staken);   // S may be overwritten by the next tile's MMA
        }
        if (cnt < KT) {
          // rows behind the last key may hold anything: their values become zero
          // (a weight of zero would not cover infinities)
          if (!mbar_wait(vfull(i % NV), (i / NV) & 1)) fail = 1;
          const uint32_t vst = v_u + (i % NV) * C_::VST;
          constexpr int CR = D / 8 + 8;   // 16-byte chunks a key
          for (int e = tid; e < (KT - cnt) * CR; e += 32 * NSM) {
            const int t = cnt + e / CR, c = e % CR;
            sts128(vst + (uint32_t)(c / 8) * (KT * 128) + t * 128 + (c % 8) * 16, 0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (live) {
          if (drafted) {
            // 64 nodes at most: this warp's half of the keys holds all of them or none
            const uint64_t vm = kh == 0 ? vis : 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t v32 = (uint32_t)(vm >> (32 * h));
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!((v32 >> c) & 1u)) sv[h][c] = __float_as_uint(-INFINITY);
            }
          } else if (cnt < KT) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (64 * kh + 32 * h + c >= cnt) sv[h][c] = __float_as_uint(-INFINITY);
          }
          float mr[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float mx = __uint_as_float(sv[h][0]);
#pragma unroll
            for (int c = 1; c < 31; c += 2) mx = max3f(mx, __uint_as_float(sv[h][c]), __uint_as_float(sv[h][c + 1]));
            mr[h] = fmaxf(mx, __uint_as_float(sv[h][31]));
          }
          float mt = fmaxf(mr[0], mr[1]) * sl2;   // the scale is positive
          if (!fold) {
            float* xb = xch + buf * 256;
            xb[w * 32 + lane] = mt;
            bar_sync(BAR_PAIR + sp, 64);
            mt = fmaxf(mt, xb[(w ^ 4) * 32 + lane]);
          }
          // lazy rescale: move the reference maximum only when a row's grew by > 8
          const bool need = mt > m_ref + 8.f || (m_ref == -INFINITY && mt != -INFINITY);
          if (__any_sync(0xffffffffu, need)) {
            const float m_new = fmaxf(m_ref, mt);
            const float corr = m_ref == -INFINITY ? 0.f : fast_exp2(m_ref - m_new);
            if (i > 0) {
              // O holds every tile before this one (S of this tile is done, so P V of tile i - 2 is)
              if (!mbar_wait(pvdone, (i - 1) & 1)) fail = 1;
              tc_fence_after();
              // O and O_lr behind it, 16 columns at a time: this warp's half, or folded all
#pragma unroll 1
              for (int h = fold ? 0 : ch; h < (D + R) / 16; h += fold ? 1 : 2) {
                const uint32_t ta = tmem + T_O + 16 * h + tlane;
                uint32_t ov[16];
                tmem_ld32x32b_x16(ov, ta);
                tmem_wait_ld_r16(ov);
#pragma unroll
                for (int c = 0; c < 16; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * corr);
                tmem_st32x32b_x16(ta, ov);
              }
              tmem_wait_st();
            }
            lsum *= corr;
            m_ref = m_new;
          }
          const float mu = m_ref == -INFINITY ? 0.f : m_ref;
          const uint64_t scl = f2(sl2, sl2), nmu = f2(-mu, -mu);
          uint64_t acc = f2(0.f, 0.f);
          uint32_t pk[32];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              const uint64_t xa2 = fma_f2(f2(__uint_as_float(sv[h][c]), __uint_as_float(sv[h][c + 1])), scl, nmu);
              float p0, p1;
              if (!KEYS && (c / 2) % kPolyEvery == 0) {
                const float2 pp = f2_unpack(exp2_poly_f2(xa2));
                p0 = pp.x;
                p1 = pp.y;
              } else {
                const float2 xa = f2_unpack(xa2);
                p0 = fast_exp2(xa.x);
                p1 = fast_exp2(xa.y);
              }
              acc = add_f2(acc, f2(p0, p1));
              pk[16 * h + c / 2] = pack_bf16(p0, p1);
            }
          const float2 accf = f2_unpack(acc);
          lsum += accf.x + accf.y;
          if (KEYS && i > 0) {   // P V of the last tile has read P
            if (!mbar_wait(pvdone, (i - 1) & 1)) fail = 1;
            tc_fence_after();
          }
          tmem_st32x32b_x32(tmem + C_::t_p(buf) + 32 * kh + tlane, pk);
          if (!KEYS && fold) {   // P lies over the scores: no weights for the other half's keys
#pragma unroll
            for (int c = 0; c < 32; ++c) pk[c] = 0;
            tmem_st32x32b_x32(tmem + C_::t_p(buf) + 32 * (1 - kh) + tlane, pk);
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull(buf));
      }

      // ---- this split's partial: O as 16-byte chunks, chunk c of a row at c ^ (row mod
      // D / 4) (no bank conflicts by rows or by columns), O_lr, then m and l
      constexpr int NCH = D / 4;
      const uint32_t pol = k_u + C_::P_OL, pml = k_u + C_::P_ML;
      if (NT > 0) {
        // a warp that did not wait for every P V: S of the last tile is done, so P V is at
        // tile NT - 2 or past it, and the parity of NT - 1 alone would be ambiguous
        if (NT > 1 && !mbar_wait(pvdone, (NT - 2) & 1)) fail = 1;
        if (!mbar_wait(pvdone, (NT - 1) & 1)) fail = 1;
        tc_fence_after();
        if (has) {
#pragma unroll 1
          for (int h = 0; h < H2 / 16; ++h) {
            uint32_t ov[16];
            tmem_ld32x32b_x16(ov, tmem + T_O + H2 * ch + 16 * h + tlane);
            tmem_wait_ld_r16(ov);
#pragma unroll
            for (int c = 0; c < 4; ++c)
              sts128(k_u + (uint32_t)tl * (D * 4) + (uint32_t)(((H2 * ch + 16 * h) / 4 + c) ^ (tl & (NCH - 1))) * 16,
                     ov[4 * c], ov[4 * c + 1], ov[4 * c + 2], ov[4 * c + 3]);
          }
#pragma unroll 1
          for (int h = ch; h < R / 16; h += 2) {
            uint32_t ov[16];
            tmem_ld32x32b_x16(ov, tmem + T_OL + 16 * h + tlane);
            tmem_wait_ld_r16(ov);
#pragma unroll
            for (int c = 0; c < 16; c += 4)
              sts128(pol + (uint32_t)(tl * R + 16 * h + c) * 4, ov[c], ov[c + 1], ov[c + 2], ov[c + 3]);
          }
        }
      }
      if (live) {
        if (!fold) {
          float* lx = xch + (NT & 1) * 256;   // the exchange buffer the last tile did not use
          lx[w * 32 + lane] = lsum;
          bar_sync(BAR_PAIR + sp, 64);
          lsum += lx[(w ^ 4) * 32 + lane];
        }
        if (ch == 0) {
          sts32(pml + tl * 8, __float_as_uint(m_ref));
          sts32(pml + tl * 8 + 4, __float_as_uint(lsum));
        }
      }
      }
      cluster_sync_all();
      // ---- merge: this CTA's share of the rows, a warp a row
      constexpr int NCH = D / 4, NW = NSM + C_::NB, NLO = R > 32 ? 2 : 1;
      const uint32_t pol = k_u + C_::P_OL, pml = k_u + C_::P_ML;
      const int share = (rows + S - 1) / S;
      const int r1 = min(rows, (split + 1) * share);
      const int c4 = lane & (NCH - 1);   // this lane's four columns
      const int lr0 = p.r < 16 ? 8 : 0;  // r = 8: the value half sits in columns 8..15
      // (kept short: it runs once, so every instruction of it is fetched cold)
      // partial i of a row: CTA i / F, lane row + 64 (i mod F) (F = 2 folded; 64 is a
      // multiple of the chunk swizzle's period)
      const int F = fold ? 2 : 1, np = S * F;
      for (int r_ = split * share + w; r_ < r1; r_ += NW) {
        const uint32_t ml = dsmem_addr(pml + 8 * (r_ + 64 * (lane & (F - 1))), lane < np ? lane / F : 0);
        const float mk = dsmem_ld(ml), lk = dsmem_ld(ml + 4);
        const uint32_t oa = k_u + (uint32_t)r_ * (D * 4) + (uint32_t)(c4 ^ (r_ & (NCH - 1))) * 16;
        const uint32_t la_ = pol + (uint32_t)(r_ * R + (lane & (R - 1))) * 4;
        float wk = lane < np ? mk : -INFINITY, inv = 0.f;   // the partials' weights, one a lane
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float lo[NLO] = {};
#pragma unroll 1
        for (int k0 = 0; k0 < np; k0 += 8) {
          float4 o[8];
          float l[8][NLO];
#pragma unroll
          for (int k = 0; k < 8; ++k) {   // requested before the weights are known
            if (k0 + k >= np) break;
            const uint32_t f = (k0 + k) & (F - 1), kc = (k0 + k) / F;
            o[k] = dsmem_ld4(dsmem_addr(oa + f * (64 * D * 4), kc));
#pragma unroll
            for (int h = 0; h < NLO; ++h) l[k][h] = dsmem_ld(dsmem_addr(la_ + f * (64 * R * 4) + 128 * h, kc));
          }
          if (k0 == 0) {
            float mx = wk;
#pragma unroll
            for (int k = kMaxSplits; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
            wk = wk == -INFINITY ? 0.f : fast_exp2(wk - mx);
            float lt = wk == 0.f ? 0.f : wk * lk;
#pragma unroll
            for (int k = kMaxSplits; k > 0; k >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, k);
            lt = __shfl_sync(0xffffffffu, lt, 0);
            inv = lt > 0.f ? 1.f / lt : 0.f;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float wv = __shfl_sync(0xffffffffu, wk, k0 + k);
            if (wv != 0.f) {   // a split without keys leaves nothing: its words are not read as numbers
              acc.x = fmaf(wv, o[k].x, acc.x);
              acc.y = fmaf(wv, o[k].y, acc.y);
              acc.z = fmaf(wv, o[k].z, acc.z);
              acc.w = fmaf(wv, o[k].w, acc.w);
#pragma unroll
              for (int h = 0; h < NLO; ++h) lo[h] = fmaf(wv, l[k][h], lo[h]);
            }
          }
        }
        // O_lr B_v^a (with a key delta all rows are one agent's, its B_v in shared memory)
        int node, ag;
        const int64_t off = locate(r_, node, ag) + 4 * c4;
        const int64_t ldB = KEYS ? D : (int64_t)p.n_kv * D;
        const __nv_bfloat16* B =
            KEYS ? reinterpret_cast<const __nv_bfloat16*>(smem + C_::OFF_BK) + 4 * c4
                 : reinterpret_cast<const __nv_bfloat16*>(p.B_v) + (int64_t)ag * p.r * ldB + kvh * D + 4 * c4;
        float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int j = 0; j < p.r; ++j) {
          const uint2 bw = *reinterpret_cast<const uint2*>(B + j * ldB);
          const float2 blo = unpack_bf16(bw.x), bhi = unpack_bf16(bw.y);
          const int jj = lr0 + j;
          const float lv = __shfl_sync(0xffffffffu, NLO > 1 && jj >= 32 ? lo[NLO - 1] : lo[0], jj & 31);
          z.x = fmaf(lv, blo.x, z.x);
          z.y = fmaf(lv, blo.y, z.y);
          z.z = fmaf(lv, bhi.x, z.z);
          z.w = fmaf(lv, bhi.y, z.w);
        }
        if (lane >= NCH) continue;
        const float4 o = make_float4(fmaf(p.s, z.x, acc.x) * inv, fmaf(p.s, z.y, acc.y) * inv,
                                     fmaf(p.s, z.z, acc.z) * inv, fmaf(p.s, z.w, acc.w) * inv);
        if (p.out_bf16)
          *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + off) =
              make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
        else
          *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + off) = o;
      }
      cluster_sync_all();   // the partials are read before any CTA of the cluster exits
    }
  } else {
    if (tid == 0) atomicOr(p.err, kDevTree);
    if (w == W0 + 1 && lane == 0)   // the first loads land before the CTA ends
      for (int i = 0; i < min(NK, NT); ++i) {
        if (KEYS && i < NL && !mbar_wait(lrfull(i), 0)) fail = 1;
        if (KEYS) mbar_arrive(kfull(i));   // in the anchors' place
        if (!mbar_wait(kfull(i), 0)) fail = 1;
        if (i < NV && !mbar_wait(vfull(i), 0)) fail = 1;
      }
  }
  if (fail) s_fail = 1;
  tc_fence_before();
  __syncthreads();
  if (w == W0) {
    tc_fence_after();
    tmem_dealloc(tmem, T_COLS);
  }
  if (tid == 0 && s_fail) atomicOr(p.err, kDevPipeWait);
}

// ------------------------------------------------------------------ host
bool tree_maps(const AttnParams& p, int D, int R, CUtensorMap* mk, CUtensorMap* mv, CUtensorMap* ml,
               CUtensorMap* mlk) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint32_t one[4] = {1, 1, 1, 1};
  cuuint64_t kd[4] = {(cuuint64_t)D, (cuuint64_t)p.L_max, (cuuint64_t)p.n_kv, (cuuint64_t)p.n_seqs};
  cuuint64_t ks[3] = {(cuuint64_t)p.kv_tok * 2, (cuuint64_t)p.kv_head * 2, (cuuint64_t)p.kv_seq * 2};
  cuuint32_t kb[4] = {64, (cuuint32_t)KT, 1, 1};
  for (int i = 0; i < 2; ++i)
    if (enc(i ? mv : mk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(i ? p.v_base : p.k_base), kd, ks, kb,
            one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  // LR rows [2r] in [n_lr][n_seqs][L_max][2r]: LRv as 64-column boxes from column
  // r (columns past 2r are filled with zeros), LRk as boxes of R columns from 0
  // (at r = 8 both take the whole 16-wide row)
  const int64_t n_lr = p.lr_agent ? p.n_agents : 1;
  const int64_t lr_agent_b = p.lr_agent ? p.lr_agent * 2 : p.lr_seq * 2 * p.n_seqs;
  cuuint64_t ld[4] = {(cuuint64_t)(2 * p.r), (cuuint64_t)p.L_max, (cuuint64_t)p.n_seqs, (cuuint64_t)n_lr};
  cuuint64_t ls[3] = {(cuuint64_t)(2 * p.r * 2), (cuuint64_t)p.lr_seq * 2, (cuuint64_t)lr_agent_b};
  for (int i = 0; i < 2; ++i) {
    const int cols = i ? R : 64;
    cuuint32_t lb[4] = {(cuuint32_t)cols, (cuuint32_t)KT, 1, 1};
    if (enc(i ? mlk : ml, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p.lr), ld, ls, lb, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle_for(cols * 2), CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  }
  return true;
}

bool tree_pooled(const AttnParams& p, const TreeParams& tp) {
  // agents share keys, masks and LR rows: their rows fill the blocks together
  return !p.B_k && tp.n_trees == 1 && !p.lr_agent;
}

int tree_blocks(const AttnParams& p, const TreeParams& tp) {
  const int64_t rows = (int64_t)tp.nodes * p.g * (tree_pooled(p, tp) ? p.n_agents : 1);
  return (int)((rows + QM - 1) / QM);
}

template <int D, int R, bool KEYS>
cudaError_t launch_tt(const AttnParams& pin, const TreeParams& tp, cudaStream_t st) {
  using C = TCfg<D, R, KEYS>;
  AttnParams p = pin;
  RopeTheta rt = {};
  rope_thetas(p.rope_base, D, &rt);
  CUtensorMap mk, mv, ml, mlk;
  if (!tree_maps(p, D, R, &mk, &mv, &ml, &mlk)) return cudaErrorInvalidValue;
  const auto kern = attn_tree_tc_kernel<D, R, KEYS>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  // resident clusters of 1..8 CTAs per device (0: not queried yet)
  static int resident[64][kMaxSplits + 1] = {};
  int* res = resident[dev & 63];
  const bool pooled = tree_pooled(p, tp);
  // at most 64 rows: folded
  const int fold = (int64_t)tp.nodes * p.g * (pooled ? p.n_agents : 1) <= QM / 2;
  const int ny = tree_blocks(p, tp) * p.n_kv * (pooled ? 1 : p.n_agents);
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(C::NTHR);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (res[1] == 0) {
    cudaFuncAttributes fa;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    if (KEYS && fa.numRegs != kLaunchRegs) return cudaErrorLaunchOutOfResources;   // setmaxnreg's split assumes it
    for (int k = kMaxSplits; k >= 1; --k) {
      attr[0].val.clusterDim.x = (unsigned)k;
      cfg.gridDim = dim3((unsigned)k, 1, 1);
      int c = 0;
      if (cudaOccupancyMaxActiveClusters(&c, kern, &cfg) != cudaSuccess) {
        cudaGetLastError();
        c = 0;
      }
      res[k] = c > 0 ? c : (k == 1 ? 1 : -1);
    }
  }
  // splits: the least waves x (tiles of a split + the tiles' worth of a CTA's
  // start and merge)
  const int64_t units = (int64_t)ny * p.n_seqs, tiles = (p.max_kv_len + KT - 1) / KT + 1;
  constexpr double kFixed = 5.0;
  int S = 1;
  double best = 0;
  for (int k = 1; k <= kMaxSplits; ++k) {
    if (res[k] < 1 || (k > 1 && k > tiles)) continue;
    const double t = (double)((units + res[k] - 1) / res[k]) * ((tiles + k - 1) / k + kFixed);
    if (k == 1 || t < best - 1e-9) {
      best = t;
      S = k;
    }
  }
  p.n_splits = S;
  cfg.numAttrs = 2;
  attr[0].val.clusterDim.x = (unsigned)S;
  cfg.gridDim = dim3((unsigned)S, (unsigned)ny, (unsigned)p.n_seqs);
  e = cudaLaunchKernelEx(&cfg, kern, mk, mv, ml, mlk, p, tp, rt, (int)pooled, fold);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D, bool KEYS>
cudaError_t launch_tt_r(const AttnParams& p, const TreeParams& tp, cudaStream_t st) {
  switch (p.r) {
    case 8:
    case 16: return launch_tt<D, 16, KEYS>(p, tp, st);
    case 32: return launch_tt<D, 32, KEYS>(p, tp, st);
    default: return launch_tt<D, 64, KEYS>(p, tp, st);
  }
}

}  // namespace

// bf16 caches whose rows a tensor map can count
bool attn_tree_bf16_supported(const AttnParams& p, const TreeParams& tp) {
  if (p.L_max >= (1ll << 31) || p.n_seqs > 65535 || p.g > 64) return false;
  const int64_t ny = (int64_t)tree_blocks(p, tp) * p.n_kv * (tree_pooled(p, tp) ? 1 : p.n_agents);
  return ny <= 65535;
}

cudaError_t launch_attn_tree_bf16(const AttnParams& pin, const TreeParams& tp, la_dtype out, cudaStream_t st) {
  AttnParams p = pin;
  p.out_bf16 = out == LA_BF16;
  if (p.d == 128) return p.B_k ? launch_tt_r<128, true>(p, tp, st) : launch_tt_r<128, false>(p, tp, st);
  return p.B_k ? launch_tt_r<64, true>(p, tp, st) : launch_tt_r<64, false>(p, tp, st);
}

}  // namespace la

// Attention of drafted trees on the tcgen05 tensor cores (bf16 storage, fp32
// accumulation in TMEM).
//
// One CTA = 128 query rows (nodes x the GQA group's heads, and without a key
// delta the agents too: their keys are the same then) of one (sequence, KV
// head), and one split of the keys; the splits of a block are a thread-block
// cluster and merge over distributed shared memory.  Keys stream in tiles of
// 128: the committed context, then one tile with the tree's own nodes.  Per tile
//   dK  = LRk B_k^a                     tcgen05, half the frequencies at a time
//   K^a = K_base + s R(k0) R(j) dK      CUDA cores, in fp16 over K_base (dK carries s's
//                                       power of two, through B_k^a)
//   S   = Q K^a^T                       tcgen05, Q (fp16) read from TMEM
//   P   = exp2(S log2e scale - m)       CUDA cores, bf16 to TMEM
//   [O | O_lr] += P [V_base | LRv]      tcgen05, P read from TMEM
// and once per row out = (O + s O_lr B_v^a) / l.  R(j) turns by the key's
// offset in its tile, or by a node's depth in the drafted tile (k0 = C there).
// Without a key delta (KEYS = false) K_base is the operand as it lies, in bf16,
// and the scores are double-buffered, P lying over the scores it came from.
//
// Warps: eight softmax warps (two per TMEM sub-partition), eight build warps (a
// thread: one key, half the frequencies), and one warp each to issue S and P V, to
// load, to issue dK (a part's MMA runs while the build turns the part before), and
// to form the anchors s R(k0) in fp64.  The reference maximum is moved lazily (O and
// l corrected only when a row's maximum grows by more than 2^8).
//
// Roundings.  Softmax weights go to bf16 (at most 2^-8 of each) because V_base
// is bf16 and one MMA takes one type; their sum stays fp32.  K^a, its delta and the
// delta's turns are fp16, the narrowest that keeps bf16 keys exact in its range.  Against
// fp64 the outputs are 1.4 times as far off as fp32 arithmetic rounded once to bf16
// (0.0024 against 0.0017 of the result's norm), nearly all of it the weights': a second
// bf16 term of P would halve P V's rate and need 64 more TMEM columns than r = 64 leaves.
//
// What bounds it (one B200).  16 nodes of 3 agents over 8192 keys (r 16, 32 / 8 heads,
// 24 x 5 CTAs): 34.6 us, of it 1.5 us a tile, 13 tiles a CTA, and about 15 us around
// them (launch, cold instructions, the first tile's way through the pipeline, the
// cluster's merge).  With the softmax's arithmetic left out a tile takes 1.3 us, with
// the build's too 0.97 us: three chains of dependent steps (load, dK, build, S;
// softmax; P V) share the SM's shared-memory bandwidth (212 KB a tile) and issue
// slots; the tensor pipe is active 23 %.  Without a key delta a tile takes 1.1 us.
// Measured and not kept: P over the scores with a key delta (dK's parts
// double-buffered in the columns won: folded tiles 2.0 us), dK in a ring of four
// parts (1.5 us), folded halves split over two warps (1.5 us), tiles prefetched into
// L2 ahead of the stages (no change), one lane polling for its warp (1.4x slower).
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
// named barriers: set-up (every thread), build warps, and the two warps of a row
// block (one id a sub-partition and direction)
constexpr int BAR_SETUP = 1, BAR_BUILD = 2, BAR_AB = 4, BAR_BA = 8;

// TMEM columns.  With a key delta: Q, dK (64 columns: 32 frequencies), S, P, O
// and O_lr behind it; without: Q, S twice (P over each), O and O_lr.
constexpr int T_Q = 0, T_DK = 64, T_P = 256, T_O = 320, T_COLS = 512;

template <int D, int R, bool KEYS>
struct TCfg {
  static constexpr int NB = KEYS ? 8 : 0;                       // build warps
  static constexpr int NTHR = 32 * (NSM + NB + 4);
  static constexpr int FP = D / 4;                              // frequencies of a part of dK (half of them)
  static constexpr int NDK = 32 / FP;                           // parts that fit dK's 64 TMEM columns: 1, or 2 at d = 64
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
  // misc: anchors [3][64] float2, references and sums of the rows [2][128] float, masks [64] u64, 64 mbarriers,
  // the TMEM slot, theta [64] float
  static constexpr int MISC = 1536 + 1024 + 512 + 512 + 16 + 256;
  // all of TMEM: one CTA an SM, and none of another kernel that holds some (at d = 64
  // the stages alone would leave room for one)
  static constexpr int NEED = 1024 + OFF_MISC + MISC;
  static constexpr int SMEM = NEED > kSmemAllTmem ? NEED : kSmemAllTmem;
  // the partial (O, O_lr, m and l) over the drained stages
  static constexpr int P_OL = QM * D * 4, P_ML = P_OL + QM * R * 4;
  static_assert(P_ML + QM * 8 <= OFF_LRK, "the partial lies over the stages");
  static_assert(SMEM <= 227 * 1024, "shared memory of one CTA");
  static_assert(T_COLS < 512 || SMEM >= kSmemAllTmem, "kept apart from other kernels with TMEM");
  // score buffers
  __host__ __device__ static constexpr int t_s(int b) { return KEYS ? 128 : 64 + 128 * b; }
  // weights of a tile's half h (64 keys, 32 columns); without a key delta over that half's scores
  __host__ __device__ static constexpr int t_p(int b, int h) { return KEYS ? T_P + 32 * h : 64 + 128 * b + 64 * h; }
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

// s as a power of two, which B_k^a carries (exactly, in bf16), and the rest, in [1, 2) or
// (-2, -1], for the anchors: so fp16 holds s LRk B_k^a to a factor of two and neither s nor
// LRk B_k^a alone.  An s below the normal numbers counts as (s 2^126) 2^-126.
__device__ __forceinline__ float scale_pow2(float s) {
  const uint32_t e = __float_as_uint(s) & 0x7f800000u;
  return __uint_as_float(e ? e : 0x00800000u);
}
__device__ __forceinline__ float scale_rest(float s) {
  const uint32_t b = __float_as_uint(s);
  return b & 0x7f800000u ? __uint_as_float((b & 0x807fffffu) | 0x3f800000u) : s * 0x1p126f;
}
__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t v, float f) {
  const __nv_bfloat162 h = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&v), __float2bfloat162_rn(f));
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int D, int R, bool KEYS>
__global__ void __launch_bounds__(TCfg<D, R, KEYS>::NTHR, 1)
    attn_tree_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ CUtensorMap tmL, const __grid_constant__ CUtensorMap tmLk,
                        const AttnParams p, const TreeParams tp,
                        const __grid_constant__ RopeTheta rt, const int pooled, const int fold) {
  using C_ = TCfg<D, R, KEYS>;
  constexpr int NK = C_::NK, NV = C_::NV, NL = C_::NL, FP = C_::FP, H2 = D / 2, T_OL = T_O + D;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const uint32_t k_u = sb, v_u = sb + C_::OFF_V, lrk_u = sb + C_::OFF_LRK, bk_u = sb + C_::OFF_BK;
  unsigned char* misc = smem + C_::OFF_MISC;
  uint2* anc = reinterpret_cast<uint2*>(misc);   // [3][32]: s (cos, cos) and s (sin, sin) of two frequencies at k0
                                                 // (s without its power of two), f16
  float* xref = reinterpret_cast<float*>(misc + 1536);   // a row's reference maximum, handed between its two warps
  float* xsum = xref + QM;
  uint64_t* masks = reinterpret_cast<uint64_t*>(misc + 2560);
  const uint32_t b0 = smem_u32(masks + kTreeMaxNodes);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(misc + 3584);
  float* thf = reinterpret_cast<float*>(misc + 3600);
  __shared__ int s_bad, s_fail;

  // mbarriers: K stages, V stages, LRk stages, then per half of a tile (h) and buffer
  auto kfull = [&](int s) { return b0 + 8 * s; };
  auto kfree = [&](int s) { return b0 + 24 + 8 * s; };
  auto kaready = [&](int s) { return b0 + 48 + 8 * s; };
  auto vfull = [&](int s) { return b0 + 72 + 8 * s; };
  auto vfree = [&](int s) { return b0 + 88 + 8 * s; };
  auto lrfull = [&](int s) { return b0 + 104 + 8 * s; };
  auto lrfree = [&](int s) { return b0 + 120 + 8 * s; };
  auto sfull = [&](int h, int b) { return b0 + 136 + 16 * h + 8 * b; };
  auto pfull = [&](int h, int b) { return b0 + 168 + 16 * h + 8 * b; };
  auto staken = [&](int h) { return b0 + 200 + 8 * h; };
  auto pvdone = [&](int h) { return b0 + 216 + 8 * h; };
  auto dkfull = [&](int h) { return b0 + 232 + 8 * h; };
  auto dkfree = [&](int h) { return b0 + 248 + 8 * h; };
  const uint32_t qready = b0 + 264, treeready = b0 + 272, alldone = b0 + 280;

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
  uint32_t tmem = 0;
  auto setup_sync = [&]() {   // barriers, TMEM, queries' and B_k's first reads: each role does its share before
    tc_fence_before();
    bar_sync(BAR_SETUP, C_::NTHR);
    tc_fence_after();
    tmem = *tslot;
  };
  int fail = 0;

  if (w >= W0) {
    if constexpr (KEYS) regs_dec<32>();
    if (w == W0) {
      // ========================================================== S and P V
      // (the whole warp walks the loop and one elected lane issues: descriptors
      // stay in uniform registers, about 75 cycles an MMA instead of 95)
      constexpr uint32_t ID_S = KEYS ? umma_idesc_f16(QM, KT / 2, 0, 0) : umma_idesc_bf16(QM, KT / 2, 0, 0);
      constexpr uint32_t ID_PV = umma_idesc_bf16(QM, D + R, 0, 1);
      tmem_alloc(smem_u32(tslot), T_COLS);
      setup_sync();
      const uint64_t dK = umma_desc(k_u, 16, 1024, 2);
      const uint64_t dV = umma_desc(v_u, KT * 128, 1024, 2);
      auto mma_pv = [&](int i, int h) {   // O, O_lr += P [V_base | LRv] over half h of tile i
        const int vs = i % NV;
        if (!mbar_wait(pfull(h, i & 1), (i >> 1) & 1)) fail = 1;
        if (h == 0 && !mbar_wait(vfull(vs), (i / NV) & 1)) fail = 1;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t vd = umma_desc_add(dV, vs * C_::VST + h * (KT / 2) * 128);
          const uint32_t tP = tmem + C_::t_p(i & 1, h), acc = i > 0 || h > 0 ? 1u : 0u;
#pragma unroll
          for (int ks = 0; ks < KT / 32; ++ks)
            umma_bf16_ts(tmem + T_O, tP + ks * 8, umma_desc_add(vd, ks * 16 * 128), ID_PV, ks > 0 ? 1u : acc);
          umma_commit(pvdone(h));
          if (h == 1) umma_commit(vfree(vs));
        }
        __syncwarp();
      };
      if (NT > 0 && !mbar_wait(qready, 0)) fail = 1;
      int ks_ = 0, kp = 0;
      if (fold) {
        // whole tiles: S of 128 keys, and P V once a row's both halves have their weights
        constexpr uint32_t ID_S2 = KEYS ? umma_idesc_f16(QM, KT, 0, 0) : umma_idesc_bf16(QM, KT, 0, 0);
#pragma unroll 1
        for (int i = 0; NT > 0 && i <= NT; ++i) {
          if (i < NT) {
            if (!mbar_wait(KEYS ? kaready(ks_) : kfull(ks_), kp)) fail = 1;
            if (KEYS && i > 0 && !(mbar_wait(staken(0), (i - 1) & 1) && mbar_wait(staken(1), (i - 1) & 1))) fail = 1;
            tc_fence_after();
            if (elect_one()) {
              const uint64_t kd = umma_desc_add(dK, ks_ * C_::KV);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                umma_bf16_ts(tmem + C_::t_s(i & 1), tmem + T_Q + kk * 8,
                             umma_desc_add(kd, (kk >> 2) * (KT * 128) + (kk & 3) * 32), ID_S2, kk > 0);
              umma_commit(sfull(0, i & 1));
              umma_commit(sfull(1, i & 1));
              umma_commit(kfree(ks_));
            }
            __syncwarp();
            if (++ks_ == NK) { ks_ = 0; kp ^= 1; }
          }
          if (i > 0) {
            const int j = i - 1, vs = j % NV;
            if (!(mbar_wait(pfull(0, j & 1), (j >> 1) & 1) && mbar_wait(pfull(1, j & 1), (j >> 1) & 1))) fail = 1;
            if (!mbar_wait(vfull(vs), (j / NV) & 1)) fail = 1;
            tc_fence_after();
            if (elect_one()) {
              const uint64_t vd = umma_desc_add(dV, vs * C_::VST);
#pragma unroll
              for (int ks = 0; ks < KT / 16; ++ks)
                umma_bf16_ts(tmem + T_O, tmem + C_::t_p(j & 1, ks / 4) + (ks % 4) * 8,
                             umma_desc_add(vd, ks * 16 * 128), ID_PV, ks > 0 || j > 0 ? 1u : 0u);
              umma_commit(pvdone(0));
              umma_commit(pvdone(1));
              umma_commit(vfree(vs));
            }
            __syncwarp();
          }
        }
      } else {
#pragma unroll 1
        for (int i = 0; NT > 0 && i <= NT; ++i) {
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            if (i < NT) {
              if (h == 0 && !mbar_wait(KEYS ? kaready(ks_) : kfull(ks_), kp)) fail = 1;
              if (KEYS && i > 0 && !mbar_wait(staken(h), (i - 1) & 1)) fail = 1;
              tc_fence_after();
              if (elect_one()) {
                const uint64_t kd = umma_desc_add(dK, ks_ * C_::KV + h * (KT / 2) * 128);   // keys 64 h ..
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                  umma_bf16_ts(tmem + C_::t_s(i & 1) + 64 * h, tmem + T_Q + kk * 8,
                               umma_desc_add(kd, (kk >> 2) * (KT * 128) + (kk & 3) * 32), ID_S, kk > 0);
                umma_commit(sfull(h, i & 1));
                if (h == 1) umma_commit(kfree(ks_));
              }
              __syncwarp();
            }
            if (i > 0) mma_pv(i - 1, h);
          }
          if (++ks_ == NK) { ks_ = 0; kp ^= 1; }
        }
      }
      if (NT > 0 && elect_one()) umma_commit(alldone);
      __syncwarp();
    } else if (w == W0 + 1) {
      // ========================================================== loads
      if (lane == 0) {
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
          for (int b = 0; b < 2; ++b) {
            mbar_init(sfull(s, b), 1);
            mbar_init(pfull(s, b), fold ? 2 : 4);
          }
          mbar_init(staken(s), fold ? 2 : 4);
          mbar_init(dkfull(s), 1);
          mbar_init(dkfree(s), 4);
          mbar_init(pvdone(s), 1);
        }
        mbar_init(qready, NSM);
        mbar_init(treeready, 1);
        mbar_init(alldone, 1);
        fence_mbar_init();
        for (int i = 0; i < min(NK, NT); ++i) {
          if (KEYS && i < NL) load_lrk(i);
          load_k(i);
          if (i < NV) load_v(i);
        }
      }
      __syncwarp();
      setup_sync();
      // the tree, while the first tiles are on their way; a bad one's outputs are left unwritten
      const bool ok = tree_masks_warp(
          tp.parent ? tp.parent + ((int64_t)seq * tp.n_trees + tree) * n : nullptr, n, m, masks);
      if (!ok) masks[lane] = masks[lane + 32] = 0;
      if (lane == 0) s_bad = !ok;
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(treeready);
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
      }
    } else if (KEYS && w == W0 + 2) {
      // ========================================================== dK
      constexpr uint32_t ID_DK = umma_idesc_bf16(KT, 2 * FP, 0, 1);
      constexpr uint32_t BROW = 4 * FP, BPART = R * BROW;   // bytes of a B_k row's part, and of the part
      setup_sync();
      const uint64_t dLRk = umma_desc(lrk_u, 16, 8 * C_::LR_ROWB, C_::LR_LAYOUT);
      const uint64_t dBk = umma_desc(bk_u, BPART, 8 * BROW, BROW == 128 ? 2 : 4);
      for (int i = 0; i < NT; ++i) {
        if (!mbar_wait(lrfull(i % NL), (i / NL) & 1)) fail = 1;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          // the buffer's last part has been read: the other part's, or (two buffers) this one's
          if (C_::NDK == 2 ? i > 0 : i + h > 0) {
            const int o = C_::NDK == 2 ? h : 1 - h;
            if (!mbar_wait(dkfree(o), (C_::NDK == 1 && h == 1 ? i : i - 1) & 1)) fail = 1;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t lr = umma_desc_add(dLRk, (i % NL) * C_::LRK);
#pragma unroll
            for (int ks = 0; ks < R / 16; ++ks)
              umma_bf16(tmem + T_DK + (C_::NDK == 2 ? 2 * FP * h : 0), umma_desc_add(lr, ks * 32),
                        umma_desc_add(dBk, h * BPART + ks * 16 * BROW), ID_DK, ks > 0);
            umma_commit(dkfull(h));
            if (h == 1) umma_commit(lrfree(i % NL));
          }
          __syncwarp();
        }
      }
    } else if (KEYS && w == W0 + 3) {
      // ========================================================== anchors s R(k0)
      // two adjacent frequencies a lane
      const int f = 2 * lane < H2 ? 2 * lane : 0;
      const double th0 = rt.theta[f], th1 = rt.theta[f + 1];
      setup_sync();
      const float sm = scale_rest(p.s);
      int ks_ = 0, kp = 1;
      for (int i = 0; i < NT; ++i) {
        if (i >= 3 && !mbar_wait(kaready(ks_), kp)) fail = 1;   // build(i - 3) has read its slot
        const int64_t k0 = n0 + i == Nc ? C : (int64_t)(n0 + i) * KT;
        const float2 a = rope_cs_exact(k0, th0), b = rope_cs_exact(k0, th1);
        if (2 * lane < H2)
          anc[ks_ * 32 + lane] = make_uint2(h2_bits(__floats2half2_rn(a.x * sm, b.x * sm)),
                                            h2_bits(__floats2half2_rn(a.y * sm, b.y * sm)));
        __syncwarp();
        if (lane == 0) mbar_arrive(kfull(ks_));
        if (++ks_ == 3) { ks_ = 0; kp ^= 1; }
      }
    } else {
      setup_sync();
    }
    __syncwarp();
    cluster_sync_all();
    cluster_sync_all();
  } else {
    if constexpr (KEYS) regs_inc<112>();
    if (KEYS && w >= NSM) {
      // ============================================================ K^a build
      // thread: key 32 sp + lane (its TMEM lane) and half h of the frequencies, in pairs
      const int key = 32 * (w & 3) + lane, h = (w - NSM) >> 2;
      uint32_t RC[FP / 2], RS[FP / 2];   // R(j): (cos, cos) and (sin, sin) of a pair, f16
      // B_k^a's rows (past r, at r = 8, zeros) travel while R(j) is formed
      constexpr int NBK = (R * D / 8 + 255) / 256;
      const int bt = tid - 32 * NSM;
      uint4 bkv[NBK];
      const __nv_bfloat16* Bk = reinterpret_cast<const __nv_bfloat16*>(p.B_k) +
                                (int64_t)agent0 * p.r * p.n_kv * D + kvh * D;
#pragma unroll
      for (int u = 0; u < NBK; ++u) {
        const int i = bt + u * 256, j = i / (D / 8);
        bkv[u] = make_uint4(0, 0, 0, 0);
        if (j < p.r) bkv[u] = *reinterpret_cast<const uint4*>(Bk + (int64_t)j * p.n_kv * D + 8 * (i % (D / 8)));
      }
      if (bt < H2) thf[bt] = rt.thetaf[bt];
      bar_sync(BAR_BUILD, 256);
      int ks_ = 0, kp = 0;
#pragma unroll 1
      for (int i = 0; i < max(NT, 1); ++i) {
        const bool drafted = n0 + i == Nc;
        // R(j) at the first tile and at the drafted one (a split's last: offsets are the
        // nodes' depths), before the set-up or, if it needs the tree, behind it
#pragma unroll 1
        for (int st = 0; (i == 0 || drafted) && st < 2; ++st) {
          if (st == (int)drafted) {
            int jo = key;
            if (drafted) {
              if (!mbar_wait(treeready, 0)) fail = 1;
              jo = jo < m ? __popcll(masks[jo]) - 1 : 0;
            }
            const float j = (float)jo;
#pragma unroll
            for (int k = 0; k < FP / 2; ++k) {
              const float2 th = *reinterpret_cast<const float2*>(thf + FP * h + 2 * k);
              const float2 a = sincos_small(j * th.x), b = sincos_small(j * th.y);
              RC[k] = h2_bits(__floats2half2_rn(a.x, b.x));
              RS[k] = h2_bits(__floats2half2_rn(a.y, b.y));
            }
          }
          if (st == 0 && i == 0) {
            // B_k^a as the dK MMA's operand: a part is R rows of FP + FP columns (its
            // frequencies' two sides), swizzled over the row's bytes
#pragma unroll
            for (int u = 0; u < NBK; ++u) {
              const int e = bt + u * 256, j = e / (D / 8), col = 8 * (e % (D / 8)), f = col % H2;
              const uint4 v = bkv[u];
              const float s2 = scale_pow2(p.s);
              if (e < R * D / 8)
                sts128(bk_u + (uint32_t)(f / FP) * (R * FP * 4) + tile_off<2 * FP, R>(j, (col / H2) * FP + f % FP),
                       scale_bf16x2(v.x, s2), scale_bf16x2(v.y, s2), scale_bf16x2(v.z, s2), scale_bf16x2(v.w, s2));
            }
            fence_proxy_async_smem();
            setup_sync();
          }
        }
        if (NT == 0) break;
        if (!mbar_wait(kfull(ks_), kp)) fail = 1;
        // dK's part as f16 pairs, x1 and x2 the two sides of the rotation
        uint32_t x1[FP / 2], x2[FP / 2];
        if (!mbar_wait(dkfull(h), i & 1)) fail = 1;
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < FP / 16; ++q) {
          uint32_t a[16], b[16];
          const uint32_t td = tmem + T_DK + (C_::NDK == 2 ? 2 * FP * h : 0) + 16 * q + ((uint32_t)(32 * (w & 3)) << 16);
          tmem_ld32x32b_x16(a, td);
          tmem_ld32x32b_x16(b, td + FP);
          tmem_wait_ld_r16(a);
          tmem_wait_ld_r16(b);
#pragma unroll
          for (int c = 0; c < 16; c += 2) {
            x1[8 * q + c / 2] = h2_bits(__floats2half2_rn(__uint_as_float(a[c]), __uint_as_float(a[c + 1])));
            x2[8 * q + c / 2] = h2_bits(__floats2half2_rn(__uint_as_float(b[c]), __uint_as_float(b[c + 1])));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(dkfree(h));   // the next part's MMA runs during this part's turn
        // eight frequencies at a time: a 16-byte chunk of each side of the key's swizzled
        // row.  Side 2 is the next box, or (d = 64) four chunks on.
        const uint32_t rowb = k_u + ks_ * C_::KV + (uint32_t)key * 128;
        const uint4* an = reinterpret_cast<const uint4*>(anc + ks_ * 32 + FP / 2 * h);
#pragma unroll
        for (int c = 0; c < FP / 8; ++c) {
          const uint32_t o1 = rowb + (uint32_t)(((FP / 8 * h + c) ^ (key & 7)) << 4);
          const uint32_t o2 = D == 128 ? o1 + KT * 128 : o1 ^ 64;
          const uint4 v1 = lds128(o1), v2 = lds128(o2);
          const uint4 a01 = an[2 * c], a23 = an[2 * c + 1];
          uint32_t w1[4] = {v1.x, v1.y, v1.z, v1.w}, w2[4] = {v2.x, v2.y, v2.z, v2.w};
          const uint32_t ac4[4] = {a01.x, a01.z, a23.x, a23.z}, as4[4] = {a01.y, a01.w, a23.y, a23.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __half2 u1 = bits_h2(x1[4 * c + e]), u2 = bits_h2(x2[4 * c + e]);
            const __half2 cj = bits_h2(RC[4 * c + e]), sj = bits_h2(RS[4 * c + e]);
            const __half2 ac = bits_h2(ac4[e]), as = bits_h2(as4[e]);
            const __half2 y1 = __hfma2(u1, cj, __hneg2(__hmul2(u2, sj)));   // R(j) dK
            const __half2 y2 = __hfma2(u2, cj, __hmul2(u1, sj));
            // K_base + s R(k0) y, the base added inside the rotation's FMAs
            w1[e] = h2_bits(__hfma2(ac, y1, __hfma2(__hneg2(as), y2, bf16x2_h2(w1[e]))));
            w2[e] = h2_bits(__hfma2(ac, y2, __hfma2(as, y1, bf16x2_h2(w2[e]))));
          }
          sts128(o1, w1[0], w1[1], w1[2], w1[3]);
          sts128(o2, w2[0], w2[1], w2[2], w2[3]);
        }
        fence_proxy_async_smem();   // the S MMA reads K^a through the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive(kaready(ks_));
        if (++ks_ == NK) { ks_ = 0; kp ^= 1; }
      }
      // B_v^a for the merge over B_k^a, once the last tile's dK has read it (both parts:
      // part 1 is issued last, and is at the last tile or behind it by now)
      if (NT > 0 && !mbar_wait(dkfull(1), (NT - 1) & 1)) fail = 1;
      const __nv_bfloat16* Bv = reinterpret_cast<const __nv_bfloat16*>(p.B_v) +
                                (int64_t)agent0 * p.r * p.n_kv * D + kvh * D;
      for (int i = tid - 32 * NSM; i < p.r * D / 8; i += 256) {
        const uint4 v = *reinterpret_cast<const uint4*>(Bv + (int64_t)(i / (D / 8)) * p.n_kv * D + 8 * (i % (D / 8)));
        sts128(bk_u + 16 * i, v.x, v.y, v.z, v.w);
      }
    } else {
      // ============================================================ softmax
      // This thread's query row, in TMEM lane 32 sp + lane, and its half h of a tile's
      // keys: two warps share a row block, h = 0 ahead of h = 1 by about half a tile's
      // time, so that one weighs scores (bound by the SFU) while the other reads and
      // stores.  A row's reference maximum is handed from one to the other, half after
      // half; sums stay with each until the end.
      // Folded (at most 64 rows): lanes 64.. repeat the rows and take the half h = 1 of
      // every tile for themselves, with a maximum, a sum and outputs of their own that
      // the merge joins like those of another split; the warps ch = 1 only help around
      // the loop.
      const int sp = w & 3, ch = w >> 2;
      const int tl = 32 * sp + lane;
      const int row = fold ? tl & 63 : tl;
      const int h = fold ? tl >> 6 : ch;
      const bool has = (fold ? 32 * (sp & 1) : 32 * sp) < rows;   // these lanes have rows
      const uint32_t tlane = (uint32_t)(32 * sp) << 16;
      int qnode = 0;
      uint32_t qv[D / 4];   // half a row's columns, packed
      if (has) {
        int ag;
        const int64_t off = locate(row < rows ? row : 0, qnode, ag);
        const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.q) + off + H2 * ch);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint4 v = row < rows ? src[c] : make_uint4(0, 0, 0, 0);
          qv[4 * c] = v.x; qv[4 * c + 1] = v.y; qv[4 * c + 2] = v.z; qv[4 * c + 3] = v.w;
        }
        if constexpr (KEYS) {   // fp16 beside the fp16 K^a (bf16 values convert exactly within its range)
#pragma unroll
          for (int c = 0; c < D / 4; ++c) qv[c] = h2_bits(bf16x2_h2(qv[c]));
        }
      }
      setup_sync();
      if (has) {
        if constexpr (D == 128) {
          tmem_st32x32b_x32(tmem + T_Q + (D / 4) * ch + tlane, qv);
        } else {
          tmem_st32x32b_x16(tmem + T_Q + (D / 4) * ch + tlane, qv);
        }
        if (KEYS && fold && ch == 0) {   // no weights for the other half's keys
          uint32_t z[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) z[c] = 0;
          tmem_st32x32b_x32(tmem + C_::t_p(0, 1 - h) + tlane, z);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(qready);

      const float sl2 = p.scale * kLog2e;
      float m_ref = -INFINITY, lsum = 0.f;   // m_ref: what this thread's sum refers to
      for (int i = 0; i < NT && !(fold && ch == 1); ++i) {
        const bool drafted = n0 + i == Nc;
        const int cnt = drafted ? m : (int)min((int64_t)KT, C - (int64_t)(n0 + i) * KT);
        const int buf = i & 1;
        if (!mbar_wait(sfull(h, buf), (i >> 1) & 1)) fail = 1;
        tc_fence_after();
        uint32_t sv[2][32];
        if (has) {
          const uint32_t ts = tmem + C_::t_s(buf) + 64 * h + tlane;
          tmem_ld32x32b_x32(sv[0], ts);
          tmem_ld32x32b_x32(sv[1], ts + 32);
          tmem_wait_ld_r32(sv[0]);
          tmem_wait_ld_r32(sv[1]);
        }
        if constexpr (KEYS) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(staken(h));   // these scores may be overwritten by the next tile's MMA
        }
        if (cnt < KT) {
          // rows behind the last key may hold anything: their values become zero
          // (a weight of zero would not cover infinities).  Each half's warps clear its rows.
          if (NV == 1 && i > 0) {
            // the one stage holds the last tile until its P V is done (two stages: the tile
            // before it, whose P V came before these scores).  Of half 0's at h = 1 that is
            // known, and its barrier may be a phase further.
            if (!mbar_wait(pvdone(1), (i - 1) & 1)) fail = 1;
            if ((fold || h == 0) && !mbar_wait(pvdone(0), (i - 1) & 1)) fail = 1;
          }
          if (!mbar_wait(vfull(i % NV), (i / NV) & 1)) fail = 1;
          const uint32_t vst = v_u + (i % NV) * C_::VST;
          constexpr int CR = D / 8 + 8;   // 16-byte chunks a key
          const int t0 = max(cnt, 64 * h), nt = 64 * h + 64 - t0;
          for (int e = fold ? tl & 63 : tl; e < nt * CR; e += fold ? 64 : 128) {
            const int t = t0 + e / CR, c = e % CR;
            sts128(vst + (uint32_t)(c / 8) * (KT * 128) + t * 128 + (c % 8) * 16, 0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (has) {
          if (cnt < KT) {
            // visible keys of this half: the drafted nodes this row sees (at most 64: in
            // half 0), or those in front of the context's end
            uint64_t vm = 0;
            if (drafted) {
              if (!mbar_wait(treeready, 0)) fail = 1;
              if (h == 0 && row < rows) vm = masks[qnode];
            } else {
              const int v = cnt - 64 * h;
              vm = v >= 64 ? ~0ull : (v > 0 ? (1ull << v) - 1 : 0);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t v32 = (uint32_t)(vm >> (32 * k));
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!((v32 >> c) & 1u)) sv[k][c] = __float_as_uint(-INFINITY);
            }
          }
          float mr[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float mx = __uint_as_float(sv[k][0]);
#pragma unroll
            for (int c = 1; c < 31; c += 2) mx = max3f(mx, __uint_as_float(sv[k][c]), __uint_as_float(sv[k][c + 1]));
            mr[k] = fmaxf(mx, __uint_as_float(sv[k][31]));
          }
          const float mt = fmaxf(mr[0], mr[1]) * sl2;   // the scale is positive
          float ref = m_ref;   // the row's reference before this half
          if (!fold && i + h > 0) {
            bar_sync((h ? BAR_AB : BAR_BA) + sp, 64);
            ref = xref[row];
          }
          // lazy rescale: move the reference only when a row's maximum grew by > 8
          const bool need = mt > ref + 8.f || (ref == -INFINITY && mt != -INFINITY);
          const float m_new = need ? mt : ref;
          if (__any_sync(0xffffffffu, need) && i + h > 0 && (i > 0 || !fold)) {
            const float corr = ref == -INFINITY ? 0.f : fast_exp2(ref - m_new);
            // O holds every half before this one, and no other is issued before this one's
            // weights (folded: neither half of this tile).  S of this half is done, so the P V
            // issued before it are, and the parities below are of the current phase or the last.
            if (fold) {
              if (!mbar_wait(pvdone(0), (i - 1) & 1)) fail = 1;
              if (!mbar_wait(pvdone(1), (i - 1) & 1)) fail = 1;
            } else if (!mbar_wait(pvdone(1 - h), (h ? i : i - 1) & 1)) {
              fail = 1;
            }
            tc_fence_after();
            // O and O_lr behind it, 16 columns at a time
#pragma unroll 1
            for (int k = 0; k < (D + R) / 16; ++k) {
              const uint32_t ta = tmem + T_O + 16 * k + tlane;
              uint32_t ov[16];
              tmem_ld32x32b_x16(ov, ta);
              tmem_wait_ld_r16(ov);
#pragma unroll
              for (int c = 0; c < 16; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * corr);
              tmem_st32x32b_x16(ta, ov);
            }
            tmem_wait_st();
            tc_fence_before();
          }
          if (!fold) {
            xref[row] = m_new;
            bar_arrive((h ? BAR_BA : BAR_AB) + sp, 64);
          }
          if (__any_sync(0xffffffffu, m_new != m_ref)) lsum *= m_ref == -INFINITY ? 0.f : fast_exp2(m_ref - m_new);
          m_ref = m_new;
          const float mu = m_ref == -INFINITY ? 0.f : m_ref;
          const uint64_t scl = f2(sl2, sl2), nmu = f2(-mu, -mu);
          uint64_t acc = f2(0.f, 0.f);
          uint32_t pk[32];
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
            const uint64_t xa2 = fma_f2(f2(__uint_as_float(sv[k][c]), __uint_as_float(sv[k][c + 1])), scl, nmu);
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
            pk[16 * k + c / 2] = pack_bf16(p0, p1);
          }
          const float2 accf = f2_unpack(acc);
          lsum += accf.x + accf.y;
          if (KEYS && i > 0) {   // P V of this half's last weights has read them
            if (!mbar_wait(pvdone(h), (i - 1) & 1)) fail = 1;
            tc_fence_after();
          }
          tmem_st32x32b_x32(tmem + C_::t_p(buf, h) + tlane, pk);
          if (!KEYS && fold) {   // P lies over the scores: no weights for the other half's keys
            if (!mbar_wait(sfull(1 - h, buf), (i >> 1) & 1)) fail = 1;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 32; ++c) pk[c] = 0;
            tmem_st32x32b_x32(tmem + C_::t_p(buf, 1 - h) + tlane, pk);
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull(h, buf));
      }

      // ---- this split's partial: O as 16-byte chunks, chunk c of a row at c ^ (row mod
      // D / 4) (no bank conflicts by rows or by columns), O_lr, then m and l
      constexpr int NCH = D / 4;
      const uint32_t pol = k_u + C_::P_OL, pml = k_u + C_::P_ML;
      if (NT > 0 && !mbar_wait(alldone, 0)) fail = 1;
      if (has && NT > 0 && !fold) {
        if (ch == 0) {   // the other half's last word on the reference
          bar_sync(BAR_BA + sp, 64);
          const float ref = xref[row];
          lsum *= m_ref == -INFINITY ? 0.f : fast_exp2(m_ref - ref);
          m_ref = ref;
        } else {
          xsum[row] = lsum;
        }
        bar_sync(BAR_AB + sp, 64);
        if (ch == 0) lsum += xsum[row];
      }
      if (has && ch == 0) {
        sts32(pml + tl * 8, __float_as_uint(m_ref));
        sts32(pml + tl * 8 + 4, __float_as_uint(lsum));
      }
      if (NT > 0) {
        tc_fence_after();
        if (has) {
#pragma unroll 1
          for (int k = 0; k < H2 / 16; ++k) {
            uint32_t ov[16];
            tmem_ld32x32b_x16(ov, tmem + T_O + H2 * ch + 16 * k + tlane);
            tmem_wait_ld_r16(ov);
#pragma unroll
            for (int c = 0; c < 4; ++c)
              sts128(k_u + (uint32_t)tl * (D * 4) + (uint32_t)(((H2 * ch + 16 * k) / 4 + c) ^ (tl & (NCH - 1))) * 16,
                     ov[4 * c], ov[4 * c + 1], ov[4 * c + 2], ov[4 * c + 3]);
          }
#pragma unroll 1
          for (int k = ch; k < R / 16; k += 2) {
            uint32_t ov[16];
            tmem_ld32x32b_x16(ov, tmem + T_OL + 16 * k + tlane);
            tmem_wait_ld_r16(ov);
#pragma unroll
            for (int c = 0; c < 16; c += 4)
              sts128(pol + (uint32_t)(tl * R + 16 * k + c) * 4, ov[c], ov[c + 1], ov[c + 2], ov[c + 3]);
          }
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
    if (!mbar_wait(treeready, 0)) fail = 1;
    for (int r_ = split * share + w; r_ < r1 && !s_bad; r_ += NW) {
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
  if (fail) s_fail = 1;
  tc_fence_before();
  __syncthreads();
  if (w == W0) {
    tc_fence_after();
    tmem_dealloc(tmem, T_COLS);
  }
  if (tid == 0 && (s_fail || s_bad)) atomicOr(p.err, (s_fail ? kDevPipeWait : 0) | (s_bad ? kDevTree : 0));
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
  // splits: the least waves x (tiles of a split + the tiles' worth of a CTA's start and
  // hand-over + that of merging its rows, a warp a row at a time).  Measured in tiles: a
  // row of a warp 1.4 without a key delta (1.5 us; 96 rows over 100 keys: 2 splits 17.9
  // us, 5 12.8 us, 8 11.7 us), about 1 with.  A split without keys still merges its share.
  const int64_t units = (int64_t)ny * p.n_seqs, tiles = (p.max_kv_len + KT - 1) / KT + 1;
  const int rows = (int)min((int64_t)QM, (int64_t)tp.nodes * p.g * (pooled ? p.n_agents : 1));
  constexpr double kFixed = 5.0, kRow = KEYS ? 1.0 : 1.4;
  constexpr int kMergeWarps = NSM + C::NB;
  int S = 1;
  double best = 0;
  for (int k = 1; k <= kMaxSplits; ++k) {
    if (res[k] < 1) continue;
    const int share = ((rows + k - 1) / k + kMergeWarps - 1) / kMergeWarps;
    const double t = (double)((units + res[k] - 1) / res[k]) * ((tiles + k - 1) / k + kFixed + kRow * share);
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

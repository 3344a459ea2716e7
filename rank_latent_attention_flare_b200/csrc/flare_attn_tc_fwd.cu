// Tensor-core softmax attention forward for sm_100a (bf16, D up to 128).
//
// Per CTA, for every tile of 128 keys:
//   S = Q K_tile^T           (tcgen05, 128 query rows x 128 keys x D)
//   P = 2^(c S - ref)        (one TMEM lane = one query row per thread)
//   O += P V_tile            (tcgen05, A = P from TMEM, B = V from smem)
// one pass with a running reference and sum per row; the reference moves (and
// O is rescaled) only when the row's maximum grows by more than 2^8, so the
// rescale leaves the critical path.  P is rounded to bf16 for the product;
// the row sum adds the unrounded weights in float32.
//
// Two query tiles per CTA (QT = 2): softmax warpgroup w owns query tile w,
// and the tensor core works on one tile while the other's softmax runs, so
// each key tile is read once for 256 query rows.  One query tile (QT = 1,
// calls with few query rows): the warpgroups take alternate key tiles with
// records of their own, joined through shared memory at the end.  When the
// query tiles do not fill the GPU, the key tiles are split over CTAs and the
// records joined by attn_join_kernel in a fixed order.
//
// TMEM: S of warpgroup w at columns 128 w, O at 256 + DP w.  P replaces the
// first half of S: its first 64 keys are handed to the tensor core while the
// others are computed.  All MMAs are issued by one thread, in the order in which
// they run, so that S of the next tile is issued behind the product that reads P
// from the same columns.  They come in batches whose length is a compile-time
// constant (KS steps over D): a first form with each MMA under a run-time
// condition of its own ended in illegal addresses, for a reason that reading did
// not show.  Whole batches under run-time conditions, as here, are in every form
// that has run since.  (P in columns of its own, where D <= 64 leaves room,
// lets S of the next tile start earlier, but takes one more barrier a tile: 2x8
// heads of 6000, D 64, 230 us against 223; of 1024, causal, 13.2 against 13.5.)
//
// Bound: per tile and SM the tensor core needs 4 D clocks for each of the two
// products and the MUFU 1024 clocks for the exponentials, so D = 128 is bound
// by both about equally and smaller D by the exponentials; single-token
// calls are bound by reading the keys and values once.  D is filled up with
// zeros: to 32, 64 or 128 columns in memory, and in the products to KS steps of 16
// (D 16 costs as much as 32, 40 to 56 as 64, 104 to 120 as 128).
#include <type_traits>

#include "flare_attn_tc.cuh"

namespace flare {
namespace attn {
namespace {

constexpr int kThreads = 384;        // warps 0-7 compute, 8 TMA, 9 MMA, 10 helper
constexpr int kWarpTma = 8;
constexpr int kWarpMma = 9;
constexpr int kWarpAux = 10;
constexpr int kRegsCompute = 216;    // 2 x 128 x 216 + 128 x 72 <= 384 x 168
constexpr int kRegsProducer = 72;
constexpr float kRescaleTau = 8.0f;  // log2 units

template <int DP, int QT>
struct FwdLayout {
  using T = Tile<DP>;
  static constexpr int STAGES = DP == 128 ? (QT == 2 ? 5 : 6) : DP == 64 ? 8 : 12;
  static constexpr int Q_OFF = 0;
  static constexpr int KV_OFF = QT * T::BYTES;
  static constexpr int BAR_OFF = KV_OFF + STAGES * T::BYTES;
  static constexpr int NBARS = 2 * STAGES + 1 + 2 + 2 + 2 + 2 + 1;
  static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;
  static constexpr int ML_OFF = MISC_OFF + 16;   // QT = 1: the second record's (ref, sum)
  static constexpr int BYTES = ML_OFF + 128 * 8;
  // QT = 1: the second warpgroup's O, column by column, over the drained K / V ring
  static_assert(STAGES * T::BYTES >= 128 * DP * 4, "exchange area");
};

// Every third pair of exponentials runs on the FMA pipe, off by 7.5e-5 at most
// (in P, and through the row's sum in lse; half a step of bf16 is 3.9e-3).  16
// heads of 4096 at D 32 / 64 / 128: 104 / 106 / 122 us; every second pair 115 / 123
// / 129, every fourth 105 / 107 / 122, every sixth 108 / 113 / 124, none 110 / 115
// / 125.
constexpr int kFwdPoly = 3;

// Ring order of the key and value tiles: the order in which the MMAs use
// them.  QT = 2: K0 V0 K1 V1 ...; QT = 1 runs two key tiles ahead: K0 K1 V0
// K2 V1 K3 ...
template <int QT>
__device__ __forceinline__ int item_k(int j) {
  return QT == 2 ? 2 * j : (j < 2 ? j : 2 * j - 1);
}
template <int QT>
__device__ __forceinline__ int item_v(int j) {
  return QT == 2 ? 2 * j + 1 : 2 * j + 2;
}

template <int KS, int QT>
__global__ void __launch_bounds__(kThreads, 1)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tmQ,
                    const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ AttnFwdArgs A) {
  pdl_wait();
  pdl_trigger();
  constexpr int DP = attn_dp(16 * KS);
  using L = FwdLayout<DP, QT>;
  using T = Tile<DP>;
  constexpr int NS = L::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* bars = (uint64_t*)(smem + L::BAR_OFF);
  uint64_t* kv_full = bars;
  uint64_t* kv_empty = bars + NS;
  uint64_t* q_full = bars + 2 * NS;
  uint64_t* s_full = q_full + 1;     // [w] S written by the MMA
  uint64_t* p_ready = s_full + 2;    // [w] P written by the softmax
  uint64_t* pv_done = p_ready + 2;   // [w] O holds the tile
  uint64_t* early = pv_done + 2;     // [w] the first half of P written
  uint64_t* drain = early + 2;
  uint32_t* tmem_slot = (uint32_t*)(smem + L::MISC_OFF);
  volatile int* abort_flag = (volatile int*)(smem + L::MISC_OFF + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- this CTA's work
  const int hgroups = A.Hq / A.hpt;              // head groups per batch element
  unsigned u = blockIdx.x;
  int split = 0;
  if (A.splits > 1) {
    u = blockIdx.x / (unsigned)A.splits;
    split = (int)(blockIdx.x - u * A.splits);
  }
  // causal: longest rows first; else the query blocks of a head together:
  // they share its keys in L2
  const unsigned inner = A.causal ? (unsigned)(A.B * hgroups) : (unsigned)A.qblocks;
  const unsigned uh = u / inner, ur = u - uh * inner;
  const int qb = A.causal ? A.qblocks - 1 - (int)uh : (int)ur;
  const int64_t bhg = A.causal ? ur : uh;
  const int b = (int)bhg / hgroups;
  const int h0 = ((int)bhg - b * hgroups) * A.hpt;
  const int hk = h0 / A.G;
  const int64_t rec = ((bhg * A.qblocks + qb) * A.splits + split) * (QT * 128);
  const AttnSeq sq(A.q_lens, A.k_lens, b, A.Nq, A.Nk, A.causal != 0);
  const bool packed = A.hpt > 1;
  const int q0 = qb * QT * 128;
  // key tiles per query tile w (QT = 2) or of the CTA
  int nt[2] = {0, 0};
#pragma unroll
  for (int w = 0; w < QT; ++w) {
    const int first = q0 + 128 * w;
    if (first < sq.ql) nt[w] = sq.key_tiles(packed ? A.Nq - 1 : first + 127, kAttnTile);
  }
  if (QT == 1) nt[1] = nt[0];
  const int nall = max(nt[0], nt[1]);
  const Part part(nall, split, A.splits);
  const int lo = part.lo, n = part.count, hi = lo + n;
  const int n0 = max(0, min(hi, nt[0]) - lo), n1 = max(0, min(hi, nt[1]) - lo);

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    mbar_init(q_full, 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(&s_full[w], 1);
      mbar_init(&p_ready[w], 4);
      mbar_init(&pv_done[w], 1);
      mbar_init(&early[w], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) tmem_alloc(tmem_slot, 512);
  if (warp == kWarpAux && blockIdx.x == 0)
    attn_check_lens(A.q_lens, A.k_lens, A.B, A.Nq, A.Nk, A.err);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 8) {
    regs_release<kRegsProducer>();
    if (warp == kWarpTma) {
      // ------------------------------------------------------------- TMA
      if (n > 0 && elect_one()) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        const int qb_ = (A.bcast & 1) ? 0 : b, qh_ = (A.bcast & 8) ? 0 : h0;
        const int kb_ = (A.bcast & 2) ? 0 : b, kh_ = (A.bcast & 16) ? 0 : hk;
        const int vb_ = (A.bcast & 4) ? 0 : b, vh_ = (A.bcast & 32) ? 0 : hk;
        const int box_rows = packed ? A.Nq * A.hpt : 128;
        mbar_arrive_expect_tx(q_full, QT * T::BLOCKS * box_rows * T::RB);
#pragma unroll
        for (int w = 0; w < QT; ++w)
          load_tile<DP>(smem + L::Q_OFF + w * T::BYTES, &tmQ, q_full, q0 + 128 * w, qh_, qb_);
        const int items = QT == 2 ? 2 * n : 2 * n + 1;
        int last = -1;   // the last item issued
        for (int it = 0; it < items; ++it) {
          // which tile this item is (QT = 1 has gaps where a key tile does not exist)
          int j;
          bool is_k;
          if (QT == 2) {
            j = it >> 1;
            is_k = (it & 1) == 0;
          } else if (it < 2) {
            j = it;
            is_k = true;
          } else {
            is_k = (it & 1) != 0;
            j = is_k ? (it + 1) / 2 : (it - 2) / 2;
          }
          if (j >= n) continue;
          const int s = it % NS, use = it / NS;
          if (use > 0 && !mbar_wait(&kv_empty[s], (uint32_t)((use - 1) & 1))) {
            record_error(A.err, kErrAttnFwdTmaWait);
            *abort_flag = 1;
            break;
          }
          if (*abort_flag) break;
          mbar_arrive_expect_tx(&kv_full[s], T::BYTES);
          const int row = tile_row0(lo + j, kAttnTile, sq.kl);
          uint8_t* dst = smem + L::KV_OFF + s * T::BYTES;
          if (is_k) load_tile<DP>(dst, &tmK, &kv_full[s], row, kh_, kb_);
          else load_tile<DP>(dst, &tmV, &kv_full[s], row, vh_, vb_);
          last = it;
        }
        // every load lands before the CTA can exit
        for (int it = max(0, last - NS + 1); it <= last; ++it)
          if (QT == 2 || it != 2 * n - 1)   // the gap before the last value tile
            mbar_wait_sleep(&kv_full[it % NS], (uint32_t)((it / NS) & 1));
        mbar_wait_sleep(q_full, 0);
      }
      __syncwarp();
    } else if (warp == kWarpMma) {
      // ------------------------------------------------------------- MMA
      if (n > 0 && elect_one()) {
        constexpr uint32_t idS = idesc_bf16_f32(128, 128, 0, 0);
        constexpr uint32_t idPV = idesc_bf16_f32(128, 16 * KS, 0, 1);
        const uint32_t kv0 = smem_u32(smem + L::KV_OFF);
        const uint64_t dQ = T::k_major(smem_u32(smem + L::Q_OFF));
        const uint64_t dK = T::k_major(kv0);
        const uint64_t dV = T::mn_major(kv0);
        bool ok = mbar_wait(q_full, 0);
        auto full = [&](int it) { return mbar_wait(&kv_full[it % NS], (uint32_t)((it / NS) & 1)); };
        auto issue_S = [&](int w, int j) {
          const uint32_t ko = (uint32_t)((item_k<QT>(j) % NS) * T::BYTES) >> 4;
          const uint32_t qo = QT == 2 ? (uint32_t)(w * T::BYTES) >> 4 : 0u;
#pragma unroll
          for (int kk = 0; kk < KS; ++kk)
            mma_ss(tmem + 128 * w, dQ + qo + T::kstep(kk), dK + ko + T::kstep(kk), idS, kk > 0);
          mma_commit(&s_full[w]);
        };
        // O += P V over the keys [64 half, 64 half + 64) of tile j
        auto issue_PV = [&](int w, int j, int half, bool first) {
          const uint32_t vo = (uint32_t)((item_v<QT>(j) % NS) * T::BYTES) >> 4;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int kk = 4 * half + k;
            mma_ts(tmem + 256 + DP * w, tmem + 128 * w + 8 * kk, dV + vo + kk * T::MN_STEP, idPV,
                   (!first || kk > 0) ? 1u : 0u);
          }
        };
        // waits for P of warpgroup w (its j-th use of the barriers) and multiplies
        auto do_PV = [&](int w, int j, int use) -> bool {
          if (!mbar_wait(&early[w], (uint32_t)(use & 1))) return false;
          tc_fence_after();
          issue_PV(w, j, 0, use == 0);
          if (!mbar_wait(&p_ready[w], (uint32_t)(use & 1))) return false;
          tc_fence_after();
          issue_PV(w, j, 1, use == 0);
          mma_commit(&pv_done[w]);
          return true;
        };
        if (QT == 2) {
          if (ok && (ok = full(item_k<QT>(0)))) {
            tc_fence_after();
            if (n0 > 0) issue_S(0, 0);
            if (n1 > 0) issue_S(1, 0);
            mma_commit(&kv_empty[item_k<QT>(0) % NS]);
          }
          for (int j = 0; ok && j < n; ++j) {
            ok = full(item_v<QT>(j)) && (j + 1 >= n || full(item_k<QT>(j + 1)));
            if (!ok) break;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const int nw = w ? n1 : n0;
              if (j >= nw) continue;
              if (!(ok = do_PV(w, j, j))) break;
              if (j + 1 < nw) issue_S(w, j + 1);
            }
            mma_commit(&kv_empty[item_v<QT>(j) % NS]);
            if (j + 1 < n) mma_commit(&kv_empty[item_k<QT>(j + 1) % NS]);
            if (*abort_flag) ok = false;
          }
        } else {
          for (int j = 0; ok && j < 2 && j < n; ++j) {
            if (!(ok = full(item_k<QT>(j)))) break;
            tc_fence_after();
            issue_S(j, j);
            mma_commit(&kv_empty[item_k<QT>(j) % NS]);
          }
          // S of tile j + 2 behind the product of tile j
          auto next_S = [&](int j) -> bool {
            if (j + 2 >= n) return true;
            if (!full(item_k<QT>(j + 2))) return false;
            tc_fence_after();
            issue_S(j & 1, j + 2);
            mma_commit(&kv_empty[item_k<QT>(j + 2) % NS]);
            return true;
          };
          auto next_PV = [&](int j) -> bool {
            if (!full(item_v<QT>(j)) || !do_PV(j & 1, j, j >> 1)) return false;
            mma_commit(&kv_empty[item_v<QT>(j) % NS]);
            return true;
          };
          for (int j = 0; ok && j < n; ++j) {
            ok = next_PV(j) && next_S(j);
            if (*abort_flag) ok = false;
          }
        }
        if (!ok) {
          record_error(A.err, kErrAttnFwdMmaWait);
          *abort_flag = 1;
        }
        mma_commit(drain);
        mbar_wait_sleep(drain, 0);
      }
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------- softmax
    regs_acquire<kRegsCompute>();
    const int w = warp >> 2;
    const int r = (warp & 3) * 32 + lane;               // TMEM lane
    const uint32_t lb = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lb + 128 * w;
    const uint32_t tO = tmem + lb + 256 + DP * w;
    // the row's query and head
    int i, h;
    bool live;
    if (packed) {
      h = h0 + min(r / A.Nq, A.hpt - 1);
      i = r % A.Nq;
      live = r < A.hpt * A.Nq;
    } else {
      h = h0;
      i = q0 + (QT == 2 ? 128 * w : 0) + r;
      live = i < A.Nq;
    }
    const bool warp_live = warp_any(live && i < sq.ql);
    const int nw = QT == 2 ? (w ? n1 : n0) : (n - w + 1) / 2;   // tiles of this warpgroup
    float mr = -INFINITY, l = 0.f;
    float top = -INFINITY;   // the largest logit so far; NaN once there was one
    bool ok = true;
    for (int j = 0; j < nw; ++j) {
      const int t = lo + (QT == 2 ? j : 2 * j + w);
      ok &= mbar_wait(&s_full[w], (uint32_t)(j & 1));
      if (!warp_live) {   // no row of this warp is stored
        warp_arrive(&early[w]);
        warp_arrive(&p_ready[w]);
        if (!(ok = warp_all(ok))) break;
        continue;
      }
      __syncwarp();
      tc_fence_after();
      const int row0 = tile_row0(t, kAttnTile, sq.kl);
      const int cl = t * kAttnTile - row0;
      const int ch = sq.causal ? i + sq.off - row0 : 127;
      const bool masked = warp_any(cl > 0 || ch < 127);
      uint32_t a[2][64];
      tmem_ld64(tS, a[0]);
      tmem_ld64(tS + 64, a[1]);
      tmem_wait_ld_dep128(a[0], a[1]);
      if (masked) {
        mask_cols(a[0], 0, cl, ch);
        mask_cols(a[1], 64, cl, ch);
      }
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      max_fold64(a[0], m4);
      max_fold64(a[1], m4);
      const float mx = max3_nan(max3_nan(m4[0], m4[1], m4[2]), m4[3], m4[3]);
      top = max3_nan(top, mx, mx);
      const bool move = (mx - mr) * A.c > kRescaleTau;   // not for NaN
      if (warp_any(move)) {
        const float nm = move ? mx : mr;
        const float f = move ? ex2((mr - nm) * A.c) : 1.f;
        l *= f;
        mr = nm;
        if (j > 0) {
          ok &= mbar_wait(&pv_done[w], (uint32_t)((j - 1) & 1));
          __syncwarp();
          tc_fence_after();
#pragma unroll 1
          for (int k = 0; k < DP / 32; ++k) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * k, o);
            tmem_wait_ld_dep(o);
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
            tmem_st32(tO + 32 * k, o);
          }
        }
      }
      const float neg = mr == -INFINITY ? 0.f : -mr * A.c;
      float s4[4] = {0.f, 0.f, 0.f, 0.f};
      // one block of straight code, so that the chunks' latencies overlap;
      // masked tiles: the MUFU's exponential maps -inf to exactly 0
      auto weights = [&](auto poly) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t pk[16];
          exp_pack_pairs<16, decltype(poly)::value>(a[k >> 1] + 32 * (k & 1), A.c, neg, pk, s4);
          tmem_st16(tS + 16 * k, pk);
          if (k == 1) {
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(&early[w]);
          }
        }
      };
      if (masked) weights(std::integral_constant<int, 0>());
      else weights(std::integral_constant<int, kFwdPoly>());
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(&p_ready[w]);
      l += (s4[0] + s4[1]) + (s4[2] + s4[3]);
      if (!(ok = warp_all(ok))) break;   // a wait ran out: one vote for all
    }
    if (ok && nw > 0 && !warp_all(mbar_wait(&pv_done[w], (uint32_t)((nw - 1) & 1)))) ok = false;
    if (!ok) {
      record_error(A.err, kErrAttnFwdRowWait);
      *abort_flag = 1;
      l = 0.f;
    }
    // The FMA pipe's exponentials clamp what they get to finite weights.  A NaN or
    // +inf among the logits makes the row NaN all the same, by its sum; a row with
    // nothing above -inf has no weight.
    if (!(top < INFINITY)) l = __uint_as_float(0x7fffffffu);
    else if (top == -INFINITY) l = 0.f;
    __syncwarp();
    tc_fence_after();
    float m2 = mr == -INFINITY ? -INFINITY : mr * A.c;   // reference, log2 units
    float own = 1.f, oth = 0.f;                          // weights of the two records (QT = 1)
    float* xo = (float*)(smem + L::KV_OFF);
    float2* xml = (float2*)(smem + L::ML_OFF);
    if (QT == 1 && n > 1) {
      // both warpgroups' products are complete: the ring is free
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (w == 1) {
        xml[r] = make_float2(m2, l);
        if (warp_live) {
#pragma unroll 1
          for (int k = 0; k < DP / 32; ++k) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * k, o);
            tmem_wait_ld_dep(o);
#pragma unroll
            for (int x = 0; x < 32; ++x) xo[(32 * k + x) * 128 + r] = __uint_as_float(o[x]);
          }
        }
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (w == 0) {
        const float2 other = xml[r];
        const float mm = fmaxf(m2, other.x);
        own = (l == 0.f) ? 0.f : ex2(m2 - mm);
        oth = (other.y == 0.f) ? 0.f : ex2(other.x - mm);
        l = l * own + other.y * oth;
        m2 = mm;
      }
    }
    // ------------------------------------------------------------ output
    const bool writer = (QT == 2 || w == 0) && warp_live;
    if ((QT == 2 || w == 0) && live && A.splits > 1)
      A.part_ml[rec + (QT == 2 ? 128 * w : 0) + r] = make_float2(m2, i < sq.ql ? l : 0.f);
    const bool some = live && i < sq.ql && l != 0.f;
    if (A.splits > 1) {
      if (writer && nw > 0) {
        float* po = A.part_o + (rec + (QT == 2 ? 128 * w : 0) + r) * (int64_t)DP;
#pragma unroll 1
        for (int k = 0; k < DP / 32; ++k) {
          uint32_t o[32];
          tmem_ld32(tO + 32 * k, o);
          tmem_wait_ld_dep(o);
          if (some) {
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
              float4 v = make_float4(__uint_as_float(o[x]), __uint_as_float(o[x + 1]),
                                     __uint_as_float(o[x + 2]), __uint_as_float(o[x + 3]));
              if (QT == 1) {
                v.x *= own, v.y *= own, v.z *= own, v.w *= own;
                if (oth != 0.f) {
                  const float* q = xo + (32 * k + x) * 128 + r;
                  v.x += oth * q[0], v.y += oth * q[128], v.z += oth * q[256], v.w += oth * q[384];
                }
              }
              *reinterpret_cast<float4*>(po + 32 * k + x) = v;
            }
          }
          __syncwarp();   // the warp's lanes load together
        }
      }
    } else if (QT == 2 || w == 0) {
      const float inv = some ? 1.f / l : 0.f;
      const int64_t at = b * A.y.sb + h * A.y.sh + i * A.y.sn;
      __nv_bfloat16* y = (__nv_bfloat16*)A.Y + at;
      __nv_bfloat16* low = A.Ylow ? (__nv_bfloat16*)A.Ylow + at : nullptr;
#pragma unroll 1
      for (int k = 0; k < DP / 32; ++k) {
        uint32_t o[32];
        tmem_ld32(tO + 32 * k, o);
        tmem_wait_ld_dep(o);
        if (live && 32 * k < A.D) {
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            float v = __uint_as_float(o[x]);
            if (QT == 1) {
              v *= own;
              if (oth != 0.f) v += oth * xo[(32 * k + x) * 128 + r];
            }
            o[x] = some ? __float_as_uint(v) : 0u;   // also clears rows never computed
          }
          store_bf16x32(y + 32 * k, o, inv, 32 * k, A.D, low ? low + 32 * k : nullptr);
        }
        __syncwarp();   // the warp's lanes load together
      }
      if (A.lse && live)
        A.lse[((int64_t)b * A.Hq + h) * A.Nq + i] = some ? (m2 + lg2(l)) * kLn2 : -INFINITY;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

template <int KS, int QT>
cudaError_t fwd_t(const void* Q, const void* K, const void* V, const AttnDims& d, const AttnPlan& p,
                  const AttnFwdArgs& a, cudaStream_t st) {
  constexpr int DP = attn_dp(16 * KS);
  CUtensorMap mq, mk, mv;
  cudaError_t e;
  const bool packed = p.hpt > 1;
  if ((e = attn_map(&mq, Q, d.q, d.B, d.Hq, d.Nq, d.D, DP, packed ? (int)d.Nq : 128,
                    packed ? p.hpt : 1)) != cudaSuccess)
    return e;
  if ((e = attn_map(&mk, K, d.k, d.B, d.Hk, d.Nk, d.D, DP, 128, 1)) != cudaSuccess) return e;
  if ((e = attn_map(&mv, V, d.v, d.B, d.Hk, d.Nk, d.D, DP, 128, 1)) != cudaSuccess) return e;
  const int need = FwdLayout<DP, QT>::BYTES + 1024;
  const int smem = need > kMinSmemBytes ? need : kMinSmemBytes;
  e = cudaFuncSetAttribute(attn_fwd_kernel<KS, QT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_fwd_kernel<KS, QT>, dim3((unsigned)(p.units * p.splits)), kThreads, smem, st,
                 mq, mk, mv, a);
  return e != cudaSuccess ? e : cudaPeekAtLastError();
}

template <int QT>
cudaError_t fwd_q(const void* Q, const void* K, const void* V, const AttnDims& d, const AttnPlan& p,
                  const AttnFwdArgs& a, cudaStream_t st) {
  switch (attn_ks(d.D)) {
    case 2: return fwd_t<2, QT>(Q, K, V, d, p, a, st);
    case 4: return fwd_t<4, QT>(Q, K, V, d, p, a, st);
    case 5: return fwd_t<5, QT>(Q, K, V, d, p, a, st);
    case 6: return fwd_t<6, QT>(Q, K, V, d, p, a, st);
    default: return fwd_t<8, QT>(Q, K, V, d, p, a, st);
  }
}

}  // namespace
}  // namespace attn

cudaError_t launch_attn_fwd_tc(const void* Q, const void* K, const void* V, const AttnDims& d,
                               const AttnPlan& p, const AttnFwdArgs& a, cudaStream_t st) {
  return p.qt == 2 ? attn::fwd_q<2>(Q, K, V, d, p, a, st) : attn::fwd_q<1>(Q, K, V, d, p, a, st);
}

}  // namespace flare

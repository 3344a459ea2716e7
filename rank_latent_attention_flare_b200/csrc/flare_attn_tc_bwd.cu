// Tensor-core backward of softmax attention for sm_100a (bf16, D up to 128):
// a kernel that recomputes the probabilities twice, in CTAs over key tiles (dK,
// dV) and CTAs over query tiles (dQ).  Each sum stays in one CTA's TMEM, so nothing is
// added by atomics and results repeat bit by bit; the price is computing the
// logits and dP twice, 7 products per tile pair instead of 5.
//
// dK, dV (attn_dkv): TMEM lanes are keys, columns queries.  Per tile
// of 128 queries of each head that shares the keys:
//   S^T = K Q^T,  P^T = 2^(c S^T + nl),   dV += P^T dY     (P^T from TMEM)
//   dP^T = V dY^T, dS^T = P^T (dP^T - delta), dK += dS^T Q
// nl = -lse and delta differ by column: they come from shared memory.
// Warpgroup w computes columns [32 w, 32 w + 32).  P^T and dS^T (bf16)
// replace the columns of S^T and dP^T that the same warp has read.  The
// MMAs alternate with the softmax so that the tensor core always has two
// products to run: {dV_j, S_j+1} while dS_j is computed, {dK_j, dP_j+1}
// while P_j+1 is.
//
// dQ (attn_dq): lanes are queries, columns keys, nl and delta one per
// lane:  S = Q K^T, dP = dY V^T, dS = P (dP - delta), dQ += dS K.  S has two
// buffers, so that P_j+1 is computed while {dQ_j, dP_j+1} run.
//
// Every batch of MMAs has a compile-time length (KS steps over D), as the
// forward's.  The tensor core runs the MMAs of the issuing thread in order, so
// S_j+1 may be issued behind the product that reads P_j from its columns.
//
// P in float32 enters dS; P and dS are rounded to bf16 for their products.
// Bound: per tile pair 4 D clocks for each product against 1024 clocks for
// the exponentials (a part of them on the FMA pipe): the tensor core for
// D = 128, the softmax warps for D <= 64.
#include "flare_attn_tc.cuh"

namespace flare {
namespace attn {
namespace {

// Every k-th pair of exponentials on the FMA pipe (tiles without a mask; 16 heads of
// 4096 at D 32 / 64 / 128: 236 / 251 / 376 us; second 244 / 258 / 382, fourth 238 /
// 253 / 383, none 241 / 258 / 386).
constexpr int kBwdPoly = 3;

// 16 softmax warps: warpgroup w of four takes 32 of a tile's 128 columns, so
// that four warps on each SM sub-partition hide each other's latencies (with
// eight warps of 64 columns the causal training step took 562 us, then 547).
constexpr int kBThreads = 640;
constexpr int kBWarpTma = 16, kBWarpMma = 17, kBWarpAux = 18;
constexpr int kCols = 32;
// 512 x 104 + 128 x 64 = 640 x 96; without the split the softmax's loop spills
// (2 x 8 heads of 6000, D 64: 567 against 540 us)
constexpr int kBRegsSoftmax = 104;
constexpr int kBRegsProducer = 64;

// 2^(c a + n) for a lane's columns, in place, n per column or one for all:
// probabilities in float32.
template <bool COLS, int POLY>
__device__ __forceinline__ void exp_cols(uint32_t (&a)[kCols], float c, float n,
                                         const float (&cols)[COLS ? kCols : 1]) {
  const uint64_t c2 = f32x2(c, c);
#pragma unroll
  for (int i = 0; i < kCols; i += 2) {
    const uint64_t x = fma_f32x2(f32x2(__uint_as_float(a[i]), __uint_as_float(a[i + 1])), c2,
                                 COLS ? f32x2(cols[COLS ? i : 0], cols[COLS ? i + 1 : 0])
                                      : f32x2(n, n));
    float p0, p1;
    if (POLY > 0 && (i / 2) % (POLY > 0 ? POLY : 1) == POLY - 1) {
      exp2_fma_pair(x, p0, p1);
    } else {
      split_f32x2(x, p0, p1);
      p0 = ex2(p0);
      p1 = ex2(p1);
    }
    a[i] = __float_as_uint(p0);
    a[i + 1] = __float_as_uint(p1);
  }
}

// A lane's columns as packed bf16 pairs to TMEM.
__device__ __forceinline__ void store_bf16_tmem(uint32_t taddr, const uint32_t (&a)[kCols]) {
  uint32_t pk[kCols / 2];
#pragma unroll
  for (int t = 0; t < kCols / 2; ++t)
    pk[t] = pack_bf16(__uint_as_float(a[2 * t]), __uint_as_float(a[2 * t + 1]));
  tmem_st16(taddr, pk);
}

// dS = P (dP - delta), in place in g (dP on entry).
template <bool COLS>
__device__ __forceinline__ void ds_cols(uint32_t (&g)[kCols], const uint32_t (&p)[kCols], float d,
                                     const float* cols) {
#pragma unroll
  for (int t = 0; t < kCols; t += 4) {
    float4 v;
    if (COLS) v = *reinterpret_cast<const float4*>(cols + t);
    else v = make_float4(d, d, d, d);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = t + 2 * h;
      const uint64_t x =
          mul_f32x2(f32x2(__uint_as_float(p[i]), __uint_as_float(p[i + 1])),
                    sub_f32x2(f32x2(__uint_as_float(g[i]), __uint_as_float(g[i + 1])),
                              h ? f32x2(v.z, v.w) : f32x2(v.x, v.y)));
      float x0, x1;
      split_f32x2(x, x0, x1);
      g[i] = __float_as_uint(x0);
      g[i + 1] = __float_as_uint(x1);
    }
  }
}

// TMEM column of K step kk (16 rows) of a bf16 operand stored by the
// warpgroups, each in the first half of its own columns.
__device__ __forceinline__ constexpr uint32_t a_step(int kk) {
  return kCols * (kk / (kCols / 16)) + 8 * (kk % (kCols / 16));
}

// One lane's row of an accumulator of DP columns, every step-th block of 32
// from the first: as bf16 times f to `out` (columns below D), or as float32
// to a record, or zeros.  Whole-warp call.
template <int DP>
__device__ __forceinline__ void put_row(uint32_t taddr, int first, int step, bool have, bool some,
                                        float f, __nv_bfloat16* out, float* rec, bool live, int D) {
#pragma unroll 1
  for (int k = first; k < DP / 32; k += step) {
    uint32_t o[32];
    if (have) {
      tmem_ld32(taddr + 32 * k, o);
      tmem_wait_ld_dep(o);
    }
    if (live) {
#pragma unroll
      for (int x = 0; x < 32; ++x) o[x] = some ? o[x] : 0u;
      if (rec) {
#pragma unroll
        for (int x = 0; x < 32; x += 4)
          *reinterpret_cast<uint4*>(rec + 32 * k + x) =
              make_uint4(o[x], o[x + 1], o[x + 2], o[x + 3]);
      } else if (32 * k < D) {
        store_bf16x32(out + 32 * k, o, f, 32 * k, D);
      }
    }
    __syncwarp();   // the warp's lanes load together
  }
}

// ---------------------------------------------------------------- dK, dV

template <int DP>
struct DkvLayout {
  using T = Tile<DP>;
  // ring of Q and dY tiles in the order Q0 dY0 Q1 dY1 ...
  static constexpr int SLOTS = DP == 128 ? 5 : 8;
  static constexpr int KB = DP == 128 ? 1 : 2;   // buffers of K and V
  static constexpr int NB = 2;                   // buffers of (nl, delta)
  static constexpr int K_OFF = 0;                // [KB][K, V]
  static constexpr int RING_OFF = 2 * KB * T::BYTES;
  static constexpr int NL_OFF = RING_OFF + SLOTS * T::BYTES;       // [NB][nl 128, delta 128]
  static constexpr int BAR_OFF = NL_OFF + NB * 1024;
  static constexpr int NBARS = 2 * SLOTS + 4 + 2 * NB + 6 + 2;
  static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;
  static constexpr int ITEM_OFF = MISC_OFF + 32;   // [4] pieces, for the softmax warps
  static constexpr int BYTES = ITEM_OFF + 4 * 64;
};

// One piece of the work: key tile kt of key head hk of batch b, and one part
// of the query tiles of the heads that share it (the tiles first ..
// first + per - 1 of each head; this part: n of them from number lo).
struct DkvItem {
  int b, hk, kt, split, k0, krow0, first, per, lo, n;
  unsigned bh;
  AttnSeq sq;
  __device__ __forceinline__ explicit DkvItem(const AttnBwdArgs& A) : n(0), sq(A.Nq, A.Nk) {}
  __device__ __forceinline__ DkvItem(const AttnBwdArgs& A, unsigned idx) : sq(A.Nq, A.Nk) {
    split = 0;
    unsigned u = idx;
    if (A.dkv_splits > 1) {
      u = idx / (unsigned)A.dkv_splits;
      split = (int)(idx - u * A.dkv_splits);
    }
    // causal: the keys that most queries see first
    const unsigned inner = A.causal ? (unsigned)(A.B * A.Hk) : (unsigned)A.ktiles;
    const unsigned hi = u / inner, rest = u - hi * inner;
    kt = (int)(A.causal ? hi : rest);
    bh = A.causal ? rest : hi;
    b = (int)(bh / (unsigned)A.Hk);
    hk = (int)bh - b * A.Hk;
    sq = AttnSeq(A.q_lens, A.k_lens, b, A.Nq, A.Nk, A.causal != 0);
    k0 = kt * kAttnTile;
    krow0 = tile_row0(kt, kAttnTile, sq.kl);
    first = sq.first_query_tile(k0, kAttnTile);
    per = k0 < sq.kl ? max(0, (sq.ql + kAttnTile - 1) / kAttnTile - first) : 0;
    const Part part(per * A.G, split, A.dkv_splits);
    lo = part.lo;
    n = part.count;
  }
};

static_assert(sizeof(DkvItem) <= 64, "a slot of the ring of pieces");

// The pieces of a CTA: one in each round of the grid, the order turned round
// every other time, so that sorted pieces add up to about the same.
struct Rounds {
  unsigned total, ctas, base;   // total < 2^31
  bool back;
  __device__ __forceinline__ Rounds(unsigned total_, unsigned ctas_)
      : total(total_), ctas(ctas_), base(0), back(false) {}
  __device__ __forceinline__ bool more() const { return base < total; }
  __device__ __forceinline__ unsigned index() const {
    return base + (back ? ctas - 1 - blockIdx.x : blockIdx.x);
  }
  __device__ __forceinline__ void next() {
    base += ctas;
    back = !back;
  }
};

// The query tiles of a piece in turn: head and tile number.
struct QueryTiles {
  int head, t, first, end;
  __device__ __forceinline__ explicit QueryTiles(const DkvItem& w)
      : head(w.lo > 0 ? w.lo / w.per : 0),
        t(w.first + (w.lo > 0 ? w.lo - head * w.per : 0)),
        first(w.first),
        end(w.first + w.per) {}
  __device__ __forceinline__ void next() {
    if (++t == end) t = first, ++head;
  }
};

// A place in the MMA thread's sequence of query tiles: tile j of n of piece c
// (those without a query tile left out), the J-th of all.  The first cursor to
// reach a piece finds its length, the others read it from ns[c % 4].
struct Cursor {
  int n = 0, j = 0, c = -1, J = 0;
  __device__ __forceinline__ void find(const AttnBwdArgs& A, Rounds& rd, volatile int* ns) {
    for (n = 0; rd.more() && n == 0; rd.next())
      if (rd.index() < rd.total) n = DkvItem(A, rd.index()).n;
    j = 0;
    ++c;
    ns[c & 3] = n;
  }
  __device__ __forceinline__ void follow(const volatile int* ns) {
    j = 0;
    ++c;
    n = ns[c & 3];
  }
  __device__ __forceinline__ bool on() const { return n > 0; }
  __device__ __forceinline__ bool last() const { return j + 1 == n; }
  // to the next tile; true at the end of the piece
  __device__ __forceinline__ bool step() {
    ++J;
    return ++j == n;
  }
};

// A CTA may stay for several pieces.  Barriers count on through them: J is the
// number of the query tile since the start, c that of the piece.  With two
// buffers of K and V the products of a piece follow those of the one before
// without a break, and its loads run ahead; the sums of a piece are stored
// between the tiles.  Long pieces are left to the hardware, one CTA each: it
// hands them out as SMs become free (attn_bwd_plan has the times of both).
template <int KS>
__device__ __forceinline__ void attn_dkv(const CUtensorMap& tmQ, const CUtensorMap& tmK,
                                         const CUtensorMap& tmV, const CUtensorMap& tmG,
                                         const AttnBwdArgs& A) {
  constexpr int DP = attn_dp(16 * KS);
  using L = DkvLayout<DP>;
  using T = Tile<DP>;
  constexpr int NS = L::SLOTS, NB = L::NB, KB = L::KB;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = (uint64_t*)(smem + L::BAR_OFF);
  uint64_t* full = bars;               // [slot] tile landed
  uint64_t* empty = bars + NS;         // [slot] its last product is done
  uint64_t* kv_full = bars + 2 * NS;   // [buffer of K and V]
  uint64_t* kv_empty = kv_full + 2;    // [buffer] K and V of the piece are read
  uint64_t* nl_full = kv_empty + 2;    // [NB]
  uint64_t* nl_empty = nl_full + NB;   // [NB]
  uint64_t* s_full = nl_empty + NB;    // [buffer of S]
  // [buffer of S]: with two of them a fast warp may be one tile ahead of a
  // slow one, and its arrival must not count for the tile before
  uint64_t* p_ready = s_full + 2;
  uint64_t* dp_full = s_full + 4;
  uint64_t* ds_ready = s_full + 5;
  uint64_t* done = s_full + 6;         // dK and dV of the piece are complete
  uint64_t* acc_free = s_full + 7;     // and stored
  uint32_t* tmem_slot = (uint32_t*)(smem + L::MISC_OFF);
  volatile int* abort_flag = (volatile int*)(smem + L::MISC_OFF + 4);
  volatile int* ns = (volatile int*)(smem + L::MISC_OFF + 16);   // [4]
  // S has two buffers where TMEM has room (SB = 2): S of tile j + 2 then
  // follows dV of tile j, and the softmax never waits for it
  constexpr int SB = DP <= 64 ? 2 : 1;
  constexpr uint32_t TP = 128 * SB, TK = TP + 128, TV = TK + DP;   // S at 0

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = A.G;
  unsigned total = (unsigned)(A.dkv_units * A.dkv_splits);
  if (smem_u32(smem) & 1023) {   // tiles and their descriptors need this alignment
    total = 0;
    if (threadIdx.x == 0) record_error(A.err, kErrAttnDkvTmaWait);
  }

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2 * NS + 4; ++s) mbar_init(&bars[s], 1);
    for (int s = 0; s < NB; ++s) {
      mbar_init(&nl_full[s], 1);
      mbar_init(&nl_empty[s], 16);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_ready[s], 16);
    }
    mbar_init(dp_full, 1);
    mbar_init(ds_ready, 16);
    mbar_init(done, 1);
    mbar_init(acc_free, 16);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kBWarpMma) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 16) {
    regs_release<kBRegsProducer>();
    if (warp == kBWarpTma) {
      // --------------------------------------------------------------- TMA
      if (elect_one()) {
        bool ok = true;
        int c = 0, it = 0;   // pieces and ring items so far
        for (Rounds rd(total, (unsigned)A.dkv_ctas); ok && rd.more(); rd.next()) {
          if (rd.index() >= total) continue;
          const DkvItem w(A, rd.index());
          if (w.n == 0) continue;
          const int kb = (A.bcast & 2) ? 0 : w.b, kh = (A.bcast & 16) ? 0 : w.hk;
          const int vb = (A.bcast & 4) ? 0 : w.b, vh = (A.bcast & 32) ? 0 : w.hk;
          const int qb = (A.bcast & 1) ? 0 : w.b, gb = (A.bcast & 64) ? 0 : w.b;
          const int kvb = c % KB, used = c / KB;
          if (used > 0 && !(ok = mbar_wait(&kv_empty[kvb], (uint32_t)((used - 1) & 1)))) break;
          uint8_t* kv = smem + L::K_OFF + kvb * 2 * T::BYTES;
          mbar_arrive_expect_tx(&kv_full[kvb], 2 * T::BYTES);
          load_tile<DP>(kv, &tmK, &kv_full[kvb], w.krow0, kh, kb);
          load_tile<DP>(kv + T::BYTES, &tmV, &kv_full[kvb], w.krow0, vh, vb);
          ++c;
          QueryTiles qt(w);
          for (int j = 0; ok && j < w.n; ++j, qt.next()) {
            const int h = w.hk * G + qt.head;
            const int row = tile_row0(qt.t, kAttnTile, w.sq.ql);
            for (int k = 0; k < 2; ++k, ++it) {
              const int s = it % NS, use = it / NS;
              if ((use > 0 && !mbar_wait(&empty[s], (uint32_t)((use - 1) & 1))) || *abort_flag) {
                ok = false;
                break;
              }
              uint8_t* dst = smem + L::RING_OFF + s * T::BYTES;
              mbar_arrive_expect_tx(&full[s], T::BYTES);
              if (k) load_tile<DP>(dst, &tmG, &full[s], row, (A.bcast & 128) ? 0 : h, gb);
              else load_tile<DP>(dst, &tmQ, &full[s], row, (A.bcast & 8) ? 0 : h, qb);
            }
          }
        }
        if (!ok) {
          record_error(A.err, kErrAttnDkvTmaWait);
          *abort_flag = 1;
        }
        // every load lands before the CTA can exit
        for (int x = max(0, it - NS); x < it; ++x)
          mbar_wait_sleep(&full[x % NS], (uint32_t)((x / NS) & 1));
        for (int x = max(0, c - KB); x < c; ++x)
          mbar_wait_sleep(&kv_full[x % KB], (uint32_t)((x / KB) & 1));
      }
      __syncwarp();
    } else if (warp == kBWarpMma) {
      // --------------------------------------------------------------- MMA
      if (elect_one()) {
        constexpr uint32_t idS = idesc_bf16_f32(128, 128, 0, 0);
        constexpr uint32_t idD = idesc_bf16_f32(128, 16 * KS, 0, 1);
        const uint64_t dK = T::k_major(smem_u32(smem + L::K_OFF));
        const uint32_t ring = smem_u32(smem + L::RING_OFF);
        const uint64_t rK = T::k_major(ring), rM = T::mn_major(ring);
        auto slot = [&](int it) { return (uint32_t)((it % NS) * T::BYTES) >> 4; };
        auto landed = [&](int it) { return mbar_wait(&full[it % NS], (uint32_t)((it / NS) & 1)); };
        // S^T or dP^T: A = keys' tile, B = ring tile
        auto issue_nt = [&](uint32_t d, uint64_t a, int it, uint64_t* bar) {
          const uint64_t bd = rK + slot(it);
#pragma unroll
          for (int kk = 0; kk < KS; ++kk)
            mma_ss(tmem + d, a + T::kstep(kk), bd + T::kstep(kk), idS, kk > 0);
          mma_commit(bar);
        };
        // dV or dK: A = P^T or dS^T in TMEM, B = ring tile, 128 queries deep
        auto issue_nn = [&](uint32_t d, uint32_t a, int it, bool start) {
          const uint64_t bd = rM + slot(it);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts(tmem + d, tmem + a + a_step(kk), bd + kk * T::MN_STEP, idD,
                   (!start || kk > 0) ? 1u : 0u);
          mma_commit(&empty[it % NS]);
        };
        auto kv = [&](int c) { return dK + ((uint32_t)((c % KB) * 2 * T::BYTES) >> 4); };
        // S or dP of the tile at a cursor; K and V of its piece have landed
        auto issue_S = [&](const Cursor& x) -> bool {
          if (x.j == 0 && !mbar_wait(&kv_full[x.c % KB], (uint32_t)((x.c / KB) & 1))) return false;
          if (!landed(2 * x.J)) return false;
          tc_fence_after();
          issue_nt(128 * (x.J % SB), kv(x.c), 2 * x.J, &s_full[x.J % SB]);
          return true;
        };
        auto issue_dP = [&](const Cursor& x) -> bool {
          if (!landed(2 * x.J + 1)) return false;
          tc_fence_after();
          issue_nt(TP, kv(x.c) + (T::BYTES >> 4), 2 * x.J + 1, dp_full);
          if (x.last()) mma_commit(&kv_empty[x.c % KB]);   // S was issued before
          return true;
        };
        // x: the tile whose dV and dK come next; xs, xp: the next S and dP
        Cursor x, xs, xp;
        Rounds rd(total, (unsigned)A.dkv_ctas);
        bool ok = true;
        auto next_S = [&]() {
          if (xs.step()) xs.find(A, rd, ns);
        };
        auto next_dP = [&]() {
          if (xp.step()) xp.follow(ns);
        };
        xs.find(A, rd, ns);
        xp.follow(ns);
        x.follow(ns);
        // S runs SB tiles ahead, dP one; into the next piece only where its K
        // and V have a buffer of their own
        auto may = [&](const Cursor& y) { return y.on() && (KB == 2 || y.c == x.c); };
        int c = 0;   // pieces complete
        while (x.on()) {
          if (x.j == 0 && (KB == 1 || x.J == 0)) {   // nothing of this piece is under way
            for (int k = 0; ok && k < SB && may(xs); ++k) {
              if ((ok = issue_S(xs))) next_S();
              if (k == 0 && ok && (ok = issue_dP(xp))) next_dP();
            }
            if (!ok) break;
          }
          const int J = x.J;
          if (!(ok = mbar_wait(&p_ready[J % SB], (uint32_t)((J / SB) & 1)))) break;
          if (x.j == 0 && c > 0 && !(ok = mbar_wait(acc_free, (uint32_t)((c - 1) & 1)))) break;
          tc_fence_after();
          issue_nn(TV, 128 * (J % SB), 2 * J + 1, x.j == 0);
          if (may(xs)) {
            if (!(ok = issue_S(xs))) break;
            next_S();
          }
          if (!(ok = mbar_wait(ds_ready, (uint32_t)(J & 1)))) break;
          tc_fence_after();
          issue_nn(TK, TP, 2 * J, x.j == 0);
          if (x.last()) {
            mma_commit(done);
            ++c;
          }
          if (may(xp)) {
            if (!(ok = issue_dP(xp))) break;
            next_dP();
          }
          if (*abort_flag) {
            ok = false;
            break;
          }
          if (x.step()) x.follow(ns);
        }
        if (!ok) {
          record_error(A.err, kErrAttnDkvMmaWait);
          *abort_flag = 1;
          mma_commit(done);
          ++c;
        }
        // every product is complete before the CTA can exit
        if (c > 0) mbar_wait_sleep(done, (uint32_t)((c - 1) & 1));
      }
      __syncwarp();
    } else if (warp == kBWarpAux) {
      // --------------------------- nl and delta of each tile's 128 columns
      // Columns before the tile's own queries (a last tile moved back) get
      // nl = -inf: weight 0.  With a piece's first tile goes the piece itself,
      // one without a tile at the end; pieces without a tile are zeros, written
      // here.
      bool ok = true;
      int J = 0, c = 0;
      auto slot_free = [&]() -> bool {
        const int use = J / NB;
        return use == 0 || warp_all(mbar_wait_sleep(&nl_empty[J % NB], (uint32_t)((use - 1) & 1)));
      };
      for (Rounds rd(total, (unsigned)A.dkv_ctas); ok && rd.more(); rd.next()) {
        if (rd.index() >= total) continue;
        const DkvItem w(A, rd.index());
        if (w.n == 0) {
          const int rows = min(kAttnTile, A.Nk - w.k0);
          const uint4 zero = make_uint4(0, 0, 0, 0);
          for (int v = 0; v < 2; ++v) {
            const Tok& to = v ? A.dv : A.dk;
            __nv_bfloat16* out = (__nv_bfloat16*)(v ? A.dV : A.dK) + w.b * to.sb + w.hk * to.sh;
            const int64_t part = ((int64_t)w.bh * A.ktiles + w.kt) * A.dkv_splits + w.split;
            float* rec = A.dkv_part + (part * 2 + v) * kAttnTile * DP;
            if (A.dkv_splits > 1) {
              for (int x = lane; x < kAttnTile * DP / 4; x += 32)
                reinterpret_cast<uint4*>(rec)[x] = zero;
            } else {
              const int per_row = A.D / 8;
              for (int x = lane; x < rows * per_row; x += 32) {
                const int row = x / per_row;
                *reinterpret_cast<uint4*>(out + (w.k0 + row) * to.sn + (x - row * per_row) * 8) =
                    zero;
              }
            }
          }
          continue;
        }
        QueryTiles qt(w);
        for (int j = 0; j < w.n; ++j, ++J, qt.next()) {
          const int s = J % NB;
          if (!(ok = slot_free())) break;
          if (j == 0) {
            if (lane == 0) *(DkvItem*)(smem + L::ITEM_OFF + (c & 3) * 64) = w;
            ++c;
          }
          const int row0 = tile_row0(qt.t, kAttnTile, w.sq.ql);
          const int64_t base = ((int64_t)w.b * A.Hq + w.hk * G + qt.head) * A.Nq;
          float* dst = (float*)(smem + L::NL_OFF + s * 1024);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int col = 32 * k + lane, q = row0 + col;
            const bool own = q >= qt.t * kAttnTile;
            dst[col] = own ? A.nl[base + q] : -INFINITY;
            dst[128 + col] = own ? A.delta[base + q] : 0.f;
          }
          warp_arrive(&nl_full[s]);
        }
      }
      if (ok && (ok = slot_free())) {
        if (lane == 0) *(DkvItem*)(smem + L::ITEM_OFF + (c & 3) * 64) = DkvItem(A);
        warp_arrive(&nl_full[J % NB]);
      }
      if (!ok) {
        record_error(A.err, kErrAttnDkvRowWait);
        *abort_flag = 1;
      }
    }
  } else {
    regs_acquire<kBRegsSoftmax>();
    // ----------------------------------------------------- softmax warps
    const int w = warp >> 2;
    const int r = (warp & 3) * 32 + lane;   // TMEM lane: key krow0 + r
    const uint32_t lb = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tP = tmem + lb + TP + kCols * w;
    bool ok = true;
    int J = 0;
    for (int c = 0;; ++c) {
      if (!(ok = warp_all(mbar_wait(&nl_full[J % NB], (uint32_t)((J / NB) & 1))))) break;
      // the piece stays in its slot until this warp has stored its sums: the
      // next two at most are published before that
      const DkvItem* item = (const DkvItem*)(smem + L::ITEM_OFF + (c & 3) * 64);
      const int n = item->n, krow0 = item->krow0, off = item->sq.off, ql = item->sq.ql;
      if (n == 0) break;
      QueryTiles qt(*item);
      for (int j = 0; j < n; ++j, ++J, qt.next()) {
        const int s = J % NB;
        const uint32_t tS = tmem + lb + 128 * (J % SB) + kCols * w;
        const int row0 = tile_row0(qt.t, kAttnTile, ql);
        // columns below cl do not see this lane's key
        const int cl = A.causal ? krow0 + r - off - row0 - kCols * w : -1;
        const float* nl = (const float*)(smem + L::NL_OFF + s * 1024) + kCols * w;
        ok &= mbar_wait(&nl_full[s], (uint32_t)((J / NB) & 1));
        float nv[kCols];   // read ahead of the wait for S
#pragma unroll
        for (int x = 0; x < kCols; x += 4) {
          const float4 v = *reinterpret_cast<const float4*>(nl + x);
          nv[x] = v.x, nv[x + 1] = v.y, nv[x + 2] = v.z, nv[x + 3] = v.w;
        }
        const bool odd = !(fabsf(nl[lane]) < INFINITY);
        ok &= mbar_wait(&s_full[J % SB], (uint32_t)((J / SB) & 1));
        __syncwarp();
        tc_fence_after();
        uint32_t p[kCols];
        tmem_ld32(tS, p);
        tmem_wait_ld_dep(p);
        // a tile with masked columns, or queries without weight or with a NaN
        // among their logits (and so in nl), keeps to the MUFU, whose exponential
        // of -inf is 0 and of NaN is NaN
        if (warp_any(cl > 0 || odd)) {
          mask_cols(p, 0, cl, kCols - 1);
          exp_cols<true, 0>(p, A.c, 0.f, nv);
        } else {
          exp_cols<true, kBwdPoly>(p, A.c, 0.f, nv);
        }
        store_bf16_tmem(tS, p);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&p_ready[J % SB]);
        ok &= mbar_wait(dp_full, (uint32_t)(J & 1));
        __syncwarp();
        tc_fence_after();
        uint32_t g[kCols];
        tmem_ld32(tP, g);
        tmem_wait_ld_dep(g);
        ds_cols<true>(g, p, 0.f, nl + 128);
        warp_arrive(&nl_empty[s]);
        store_bf16_tmem(tP, g);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(ds_ready);
        if (!(ok = warp_all(ok))) break;   // a wait ran out: one vote for the three
      }
      if (!ok || !(ok = warp_all(mbar_wait(done, (uint32_t)(c & 1))))) break;
      __syncwarp();
      tc_fence_after();
      const DkvItem it = *item;
      // warpgroups 0 and 1 store dK, 2 and 3 dV: this tile's own keys, then
      // zeros for the rows past the length
      const int key = it.krow0 + r, v = w >> 1;
      const Tok& to = v ? A.dv : A.dk;
      __nv_bfloat16* out = (__nv_bfloat16*)(v ? A.dV : A.dK) + it.b * to.sb + it.hk * to.sh;
      float* rec = nullptr;
      const int64_t part = ((int64_t)it.bh * A.ktiles + it.kt) * A.dkv_splits + it.split;
      if (A.dkv_splits > 1) rec = A.dkv_part + (part * 2 + v) * kAttnTile * DP;
      const bool own = key >= it.k0 && key < it.sq.kl;
      put_row<DP>(tmem + lb + (v ? TV : TK), w & 1, 2, true, true, v ? 1.f : A.scale,
                  out + key * to.sn, rec ? rec + (int64_t)(key - it.k0) * DP : nullptr, own, A.D);
      tc_fence_before();
      warp_arrive(acc_free);
      if ((w & 1) && !rec && it.k0 + r >= it.sq.kl && it.k0 + r < A.Nk)
        for (int d = 0; d < A.D; d += 8)
          *reinterpret_cast<uint4*>(out + (it.k0 + r) * to.sn + d) = make_uint4(0, 0, 0, 0);
      __syncwarp();
    }
    if (!ok) {
      record_error(A.err, kErrAttnDkvRowWait);
      *abort_flag = 1;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kBWarpMma) tmem_dealloc(tmem, 512);
}

// -------------------------------------------------------------------- dQ

template <int DP>
struct DqLayout {
  using T = Tile<DP>;
  // ring of K and V tiles in the order K0 V0 K1 V1 ...
  static constexpr int SLOTS = DP == 128 ? 5 : DP == 64 ? 9 : 8;
  static constexpr int Q_OFF = 0;
  static constexpr int G_OFF = T::BYTES;
  static constexpr int RING_OFF = 2 * T::BYTES;
  static constexpr int BAR_OFF = RING_OFF + SLOTS * T::BYTES;
  static constexpr int NBARS = 2 * SLOTS + 1 + 2 + 2 + 1;
  static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;
  static constexpr int BYTES = MISC_OFF + 16;
};

template <int KS>
__device__ __forceinline__ void attn_dq(const CUtensorMap& tmQ, const CUtensorMap& tmK,
                                        const CUtensorMap& tmV, const CUtensorMap& tmG,
                                        const AttnBwdArgs& A) {
  constexpr int DP = attn_dp(16 * KS);
  using L = DqLayout<DP>;
  using T = Tile<DP>;
  constexpr int NS = L::SLOTS;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = (uint64_t*)(smem + L::BAR_OFF);
  uint64_t* full = bars;
  uint64_t* empty = bars + NS;
  uint64_t* q_full = bars + 2 * NS;
  uint64_t* s_full = q_full + 1;   // [2]
  uint64_t* dp_full = s_full + 2;
  uint64_t* ds_ready = s_full + 3;
  uint64_t* done = s_full + 4;
  uint32_t* tmem_slot = (uint32_t*)(smem + L::MISC_OFF);
  volatile int* abort_flag = (volatile int*)(smem + L::MISC_OFF + 4);
  constexpr uint32_t TP = 256, TQ = 384;   // S: 0 and 128

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- this CTA's work
  const unsigned idx = blockIdx.x - (unsigned)A.dkv_ctas;
  unsigned u = idx;
  int split = 0;
  if (A.dq_splits > 1) {
    u = idx / (unsigned)A.dq_splits;
    split = (int)(idx - u * A.dq_splits);
  }
  // causal: longest rows first
  const unsigned inner = A.causal ? (unsigned)(A.B * A.Hq) : (unsigned)A.qtiles;
  const unsigned hi = u / inner, rest = u - hi * inner;
  const int qt = A.causal ? A.qtiles - 1 - (int)hi : (int)rest;
  const int64_t bh = A.causal ? rest : hi;
  const int b = (int)bh / A.Hq, h = (int)bh - b * A.Hq, hk = h / A.G;
  const AttnSeq sq(A.q_lens, A.k_lens, b, A.Nq, A.Nk, A.causal != 0);
  const int q0 = qt * kAttnTile;
  const Part part(q0 < sq.ql ? sq.key_tiles(q0 + kAttnTile - 1, kAttnTile) : 0, split, A.dq_splits);
  const int lo = part.lo;
  int n = part.count;
  if (smem_u32(smem) & 1023) {   // tiles and their descriptors need this alignment
    n = 0;
    if (threadIdx.x == 0) record_error(A.err, kErrAttnDqTmaWait);
  }

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2 * NS + 1; ++s) mbar_init(&bars[s], 1);
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(dp_full, 1);
    mbar_init(ds_ready, 16);
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kBWarpMma) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 16) {
    regs_release<kBRegsProducer>();
    if (warp == kBWarpTma) {
      // --------------------------------------------------------------- TMA
      if (n > 0 && elect_one()) {
        const int kb = (A.bcast & 2) ? 0 : b, kh = (A.bcast & 16) ? 0 : hk;
        const int vb = (A.bcast & 4) ? 0 : b, vh = (A.bcast & 32) ? 0 : hk;
        mbar_arrive_expect_tx(q_full, 2 * T::BYTES);
        load_tile<DP>(smem + L::Q_OFF, &tmQ, q_full, q0, (A.bcast & 8) ? 0 : h,
                      (A.bcast & 1) ? 0 : b);
        load_tile<DP>(smem + L::G_OFF, &tmG, q_full, q0, (A.bcast & 128) ? 0 : h,
                      (A.bcast & 64) ? 0 : b);
        int last = -1;
        for (int it = 0; it < 2 * n; ++it) {
          const int s = it % NS, use = it / NS;
          if (use > 0 && !mbar_wait(&empty[s], (uint32_t)((use - 1) & 1))) {
            record_error(A.err, kErrAttnDqTmaWait);
            *abort_flag = 1;
            break;
          }
          if (*abort_flag) break;
          const int row = tile_row0(lo + (it >> 1), kAttnTile, sq.kl);
          uint8_t* dst = smem + L::RING_OFF + s * T::BYTES;
          mbar_arrive_expect_tx(&full[s], T::BYTES);
          if (it & 1) load_tile<DP>(dst, &tmV, &full[s], row, vh, vb);
          else load_tile<DP>(dst, &tmK, &full[s], row, kh, kb);
          last = it;
        }
        for (int it = max(0, last - NS + 1); it <= last; ++it)
          mbar_wait_sleep(&full[it % NS], (uint32_t)((it / NS) & 1));
        mbar_wait_sleep(q_full, 0);
      }
      __syncwarp();
    } else if (warp == kBWarpMma) {
      // --------------------------------------------------------------- MMA
      if (n > 0 && elect_one()) {
        constexpr uint32_t idS = idesc_bf16_f32(128, 128, 0, 0);
        constexpr uint32_t idD = idesc_bf16_f32(128, 16 * KS, 0, 1);
        const uint64_t dQ = T::k_major(smem_u32(smem + L::Q_OFF));
        const uint64_t dG = T::k_major(smem_u32(smem + L::G_OFF));
        const uint32_t ring = smem_u32(smem + L::RING_OFF);
        const uint64_t rK = T::k_major(ring), rM = T::mn_major(ring);
        auto slot = [&](int it) { return (uint32_t)((it % NS) * T::BYTES) >> 4; };
        auto landed = [&](int it) { return mbar_wait(&full[it % NS], (uint32_t)((it / NS) & 1)); };
        auto issue_S = [&](int j) {
          const uint64_t bd = rK + slot(2 * j);
#pragma unroll
          for (int kk = 0; kk < KS; ++kk)
            mma_ss(tmem + 128 * (j & 1), dQ + T::kstep(kk), bd + T::kstep(kk), idS, kk > 0);
          mma_commit(&s_full[j & 1]);
        };
        auto issue_dP = [&](int j) {
          const uint64_t bd = rK + slot(2 * j + 1);
#pragma unroll
          for (int kk = 0; kk < KS; ++kk)
            mma_ss(tmem + TP, dG + T::kstep(kk), bd + T::kstep(kk), idS, kk > 0);
          mma_commit(dp_full);
          mma_commit(&empty[(2 * j + 1) % NS]);
        };
        auto issue_dQ = [&](int j) {
          const uint64_t bd = rM + slot(2 * j);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts(tmem + TQ, tmem + TP + a_step(kk), bd + kk * T::MN_STEP, idD,
                   (j > 0 || kk > 0) ? 1u : 0u);
          mma_commit(&empty[(2 * j) % NS]);
        };
        bool ok = mbar_wait(q_full, 0) && landed(0) && landed(1);
        if (ok) {
          tc_fence_after();
          issue_S(0);
          issue_dP(0);
        }
        if (ok && n > 1 && (ok = landed(2))) {
          tc_fence_after();
          issue_S(1);
        }
        for (int j = 0; ok && j < n; ++j) {
          if (!(ok = mbar_wait(ds_ready, (uint32_t)(j & 1)))) break;
          tc_fence_after();
          issue_dQ(j);
          if (j + 1 < n) {
            if (!(ok = landed(2 * j + 3))) break;
            tc_fence_after();
            issue_dP(j + 1);
          }
          if (j + 2 < n) {
            if (!(ok = landed(2 * j + 4))) break;
            tc_fence_after();
            issue_S(j + 2);
          }
          if (*abort_flag) ok = false;
        }
        if (!ok) {
          record_error(A.err, kErrAttnDqMmaWait);
          *abort_flag = 1;
        }
        mma_commit(done);
        mbar_wait_sleep(done, 0);
      }
      __syncwarp();
    }
  } else {
    regs_acquire<kBRegsSoftmax>();
    // ----------------------------------------------------- softmax warps
    const int w = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lb = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tP = tmem + lb + TP + kCols * w;
    const int i = q0 + r;
    const bool live = i < A.Nq;
    const int64_t row = bh * A.Nq + i;
    const float nl = live && i < sq.ql ? A.nl[row] : -INFINITY;
    const float delta = live && i < sq.ql ? A.delta[row] : 0.f;
    const bool gone = nl == -INFINITY, odd = !(fabsf(nl) < INFINITY);   // as for dK and dV
    const float none[1] = {0.f};
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int t = lo + j;
      const int row0 = tile_row0(t, kAttnTile, sq.kl);
      const int cl = t * kAttnTile - row0 - kCols * w;
      const int ch = (sq.causal ? i + sq.off - row0 : 127) - kCols * w;
      ok &= mbar_wait(&s_full[j & 1], (uint32_t)((j >> 1) & 1));
      __syncwarp();
      tc_fence_after();
      uint32_t p[kCols];
      tmem_ld32(tmem + lb + 128 * (j & 1) + kCols * w, p);
      tmem_wait_ld_dep(p);
      if (warp_any(cl > 0 || ch < kCols - 1 || odd)) {
        mask_cols(p, 0, cl, ch);
        exp_cols<false, 0>(p, A.c, nl, none);
      } else {
        exp_cols<false, kBwdPoly>(p, A.c, nl, none);
      }
      ok &= mbar_wait(dp_full, (uint32_t)(j & 1));
      __syncwarp();
      tc_fence_after();
      uint32_t g[kCols];
      tmem_ld32(tP, g);
      tmem_wait_ld_dep(g);
      ds_cols<false>(g, p, delta, nullptr);
      store_bf16_tmem(tP, g);
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(ds_ready);
      if (!(ok = warp_all(ok))) break;   // a wait ran out: one vote for both
    }
    if (ok && n > 0 && !warp_all(mbar_wait(done, 0))) ok = false;
    if (!ok) {
      record_error(A.err, kErrAttnDqRowWait);
      *abort_flag = 1;
    }
    __syncwarp();
    tc_fence_after();
    __nv_bfloat16* out = (__nv_bfloat16*)A.dQ + b * A.dq.sb + h * A.dq.sh + i * A.dq.sn;
    float* rec = nullptr;
    if (A.dq_splits > 1)
      rec = A.dq_part +
            (((bh * A.qtiles + qt) * A.dq_splits + split) * kAttnTile + r) * (int64_t)DP;
    put_row<DP>(tmem + lb + TQ, w, 4, n > 0, n > 0 && !gone, A.scale, out, rec, live, A.D);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kBWarpMma) tmem_dealloc(tmem, 512);
}

// Both in one launch, so that dQ's CTAs fill the SMs that the last of dK's and
// dV's leave idle (when it was made, the register split not yet: 2 x 8 heads of
// 6000, D 64, 5.1 waves each, 607 us as two launches and 567 as one; 16/4 heads of
// 4096, D 128, 385 and 364).
template <int KS>
__global__ void __launch_bounds__(kBThreads, 1)
    attn_bwd_kernel(const __grid_constant__ CUtensorMap tmQ,
                    const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ CUtensorMap tmG,
                    const __grid_constant__ AttnBwdArgs A) {
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x < (unsigned)A.dkv_ctas) attn_dkv<KS>(tmQ, tmK, tmV, tmG, A);
  else attn_dq<KS>(tmQ, tmK, tmV, tmG, A);
}

template <int KS>
cudaError_t bwd_t(const AttnDims& d, const AttnBwdPlan& p, AttnBwdArgs a, cudaStream_t st) {
  constexpr int DP = attn_dp(16 * KS);
  CUtensorMap mq, mk, mv, mg;
  cudaError_t e;
  if ((e = attn_map(&mq, a.Q, d.q, d.B, d.Hq, d.Nq, d.D, DP, 128, 1)) != cudaSuccess) return e;
  if ((e = attn_map(&mk, a.K, d.k, d.B, d.Hk, d.Nk, d.D, DP, 128, 1)) != cudaSuccess) return e;
  if ((e = attn_map(&mv, a.V, d.v, d.B, d.Hk, d.Nk, d.D, DP, 128, 1)) != cudaSuccess) return e;
  if ((e = attn_map(&mg, a.dY, d.dy, d.B, d.Hq, d.Nq, d.D, DP, 128, 1)) != cudaSuccess) return e;
  static_assert((DkvLayout<DP>::KB == 2) == (DP <= 64), "attn_bwd_plan's rule");
  const int64_t pieces = a.dK ? p.dkv_units * p.dkv_splits : 0;
  a.dkv_ctas = (int)(p.stay ? imin64(pieces, sm_count()) : pieces);
  const int64_t grid = a.dkv_ctas + (a.dQ ? p.dq_units * p.dq_splits : 0);
  constexpr int kBytes =
      DkvLayout<DP>::BYTES > DqLayout<DP>::BYTES ? DkvLayout<DP>::BYTES : DqLayout<DP>::BYTES;
  constexpr int kSmem = kBytes > kMinSmemBytes ? kBytes : kMinSmemBytes;
  if ((e = cudaFuncSetAttribute(attn_bwd_kernel<KS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSmem)) != cudaSuccess)
    return e;
  e = launch_pdl(attn_bwd_kernel<KS>, dim3((unsigned)grid), kBThreads, kSmem, st, mq, mk, mv, mg,
                 a);
  return e != cudaSuccess ? e : cudaPeekAtLastError();
}

}  // namespace
}  // namespace attn

cudaError_t launch_attn_bwd_tc(const AttnDims& d, const AttnBwdPlan& p, const AttnBwdArgs& a,
                               cudaStream_t st) {
  using namespace attn;
  switch (attn_ks(d.D)) {
    case 2: return bwd_t<2>(d, p, a, st);
    case 4: return bwd_t<4>(d, p, a, st);
    case 5: return bwd_t<5>(d, p, a, st);
    case 6: return bwd_t<6>(d, p, a, st);
    default: return bwd_t<8>(d, p, a, st);
  }
}

}  // namespace flare

// Attention: cutting a call into CTAs, the workspace, the kernels common to
// both paths (joining the forward's split records, the backward's per-query
// statistics and partial sums), and the C entry points.
#include "flare_attn.cuh"

namespace flare {

// ------------------------------------------------------------------ plans

namespace {

// The number of parts to cut each of `units` pieces of work into, on `slots`
// places: minimises an estimate of the time, in tiles, with `setup` for a
// CTA's start and end, `join` for one more launch and `part` for writing and
// reading back one part's sums.  Pieces of equal size run in waves.  With a
// causal mask their sizes spread evenly up to `tiles`, longest first: the
// places share the sum, and a piece at the end leaves some of them idle, for
// about kTail of the longest.
//
// kTail: with 0 the forward of 8/2 heads of 1024, D 64, would be cut in three (20.8
// us against 13.5) and the backward of 32/8 heads of 2048, D 128, in two (144
// against 125).  With 0.3 most of sixteen causal sizes keep their plan, the
// backward of 32/8 heads of 2048, D 64, would stay whole (85 us against 96).
constexpr double kTail = 0.15;

int choose_splits(int64_t units, int64_t tiles, int slots, bool causal, double setup, double join,
                  double part, double* estimate = nullptr) {
  int best = 1;
  double best_cost = 1e300;
  const int64_t hi = imin64(tiles, imax64(1, 4LL * slots / imax64(units, 1)));
  for (int64_t s = 1; s <= hi; ++s) {
    const double longest = (double)((tiles + s - 1) / s) + setup;
    double cost;
    if (causal) {
      const double sum = (double)units * (0.5 * (double)tiles + (double)s * setup) / slots;
      cost = fmax(longest, sum + kTail * longest);
    } else {
      cost = (double)((units * s + slots - 1) / slots) * longest;
    }
    if (s > 1) cost += join + part * (double)(units * s) / slots;
    if (cost < best_cost - 1e-9) {
      best_cost = cost;
      best = (int)s;
    }
  }
  if (estimate) *estimate = best_cost;
  return best;
}

// The backward's pieces on the tensor cores, one launch: those of dK and dV
// (n1 of cost c1), then those of dQ (n2 of cost c2), each to the place that is
// free first; sizes as in choose_splits.  The estimated end.
double bwd_end(double n1, double c1, double n2, double c2, double slots, bool causal) {
  if (causal) {   // pieces are half a tile row on average, the last ones short
    const double sum = 0.5 * (n1 * c1 + n2 * c2) / slots;
    return fmax(fmax(c1, c2), sum + kTail * c2);
  }
  const double q = floor(n1 / slots), late = n1 - q * slots, early = slots - late;
  // `late` places are free at t1, the others at t0
  const double t0 = q * c1, t1 = t0 + c1;
  double left = n2;
  // rounds of dQ's pieces: before t1, then on all places, the rest in order
  double k0 = late > 0 ? fmin(floor(left / early), floor(c1 / c2)) : 0.0;
  left -= k0 * early;
  double k1 = fmax(0.0, floor(left / slots) - 1);
  k0 += k1;
  left -= k1 * slots;
  while (left > 0) {
    if (late == 0 || t0 + (k0 + 1) * c2 <= t1 + (k1 + 1) * c2) ++k0, left -= early;
    else ++k1, left -= late;
  }
  double end = n1 > 0 ? (late > 0 ? t1 : t0) : 0.0;
  if (k0 > 0) end = fmax(end, t0 + k0 * c2);
  if (k1 > 0 && late > 0) end = fmax(end, t1 + k1 * c2);
  return end;
}

}  // namespace

AttnPlan attn_plan(const AttnDims& d, flare_dtype_t dt, int sms) {
  const bool tc = attn_tc(dt);
  const int64_t G = d.G(), tile = tc ? kAttnTile : 64;
  AttnPlan p;
  // the queries of several heads of a key head share a tile when that cuts
  // the number of tiles: their keys and values are then read once
  if (d.q.sh != 0 || d.Hq == 1)
    for (int64_t g = 2; g <= G; ++g)
      if (G % g == 0 && g * d.Nq <= tile) p.hpt = (int)g;
  const int64_t rows = p.hpt > 1 ? p.hpt * d.Nq : d.Nq;
  const int64_t ktiles = (d.Nk + tile - 1) / tile;
  // one or a few tokens see about all keys
  const bool triangle = d.causal && 2 * d.Nq > d.Nk;
  // One or two query tiles a CTA: two read each key tile once for both and run
  // faster (16 heads of 4096, one against two: 109 and 104 us at D 32, 117 and 106
  // at D 64, 131 and 125 at D 128); one leaves no half empty (2 x 16 heads of 333
  // queries over 5001 keys, D 64: 40 us against 45; D 128: 42 against 53).  Times
  // in microseconds: a tile 2.0 (two) or 1.06 (one), as rounds of whole CTAs show
  // them at D 128 (1.95 and 1.02; D 64: 1.66 and 0.91), or 8 (CUDA cores, two CTAs
  // an SM), a CTA's start and end about 4 (a call of one tile takes 6 to 8), a
  // join 3, a part's rows x DP floats at an SM's share of the memory bandwidth
  // (6551 GB/s over 148 SMs: 5500 written and read back in a microsecond).
  double best = 1e300;
  for (int qt = 1; qt <= (tc && rows > kAttnTile ? 2 : 1); ++qt) {
    AttnPlan c = p;
    c.qt = qt;
    c.rows = (int)(tile * qt);
    c.qblocks = (rows + c.rows - 1) / c.rows;
    c.units = d.B * (d.Hq / c.hpt) * c.qblocks;
    const double us = tc ? (qt == 2 ? 2.0 : 1.06) : 8.0;
    const double part = (double)imin64(rows, c.rows) * attn_dp(d.D) / 5500.0;
    double cost;
    c.splits = choose_splits(c.units, ktiles, tc ? sms : 2 * sms, triangle, 4.0 / us, 3.0 / us,
                             (tc ? part : 2 * part) / us, &cost);
    if (cost * us < best) {
      best = cost * us;
      p = c;
    }
  }
  return p;
}

AttnBwdPlan attn_bwd_plan(const AttnDims& d, flare_dtype_t dt, int sms) {
  const bool tc = attn_tc(dt);
  AttnBwdPlan p;
  p.tile = tc ? kAttnTile : 64;
  p.ktiles = (d.Nk + p.tile - 1) / p.tile;
  p.qtiles = (d.Nq + p.tile - 1) / p.tile;
  p.dkv_units = d.B * d.Hk * p.ktiles;
  p.dq_units = d.B * d.Hq * p.qtiles;
  const int slots = tc ? sms : 2 * sms;
  const double setup = tc ? 2.0 : 0.5, join = tc ? 4.0 : 0.5;
  const bool triangle = d.causal && d.Nq <= 2 * d.Nk && d.Nk <= 2 * d.Nq;
  // as the forward's, in tiles of dQ (1.0 us at D 64, 1.5 at D 128; CUDA cores 4)
  const double part = p.tile * attn_dp(d.D) / (tc ? 8000.0 : 22000.0);
  if (tc) {
    // In tiles of dQ, of which one of dK and dV costs 1.2 (four whole rounds of
    // each: 1.3; with 1.1 or 1.3 five of sixty sizes are cut otherwise); each
    // number of parts in turn, and only those that leave a piece fewer tiles than
    // the one before (choosing for each side alone: 32/8 heads of 2048, D 128,
    // causal 145 us against 126; 4 heads of 1000, D 64: 27 against 18.5).
    const auto cost = [&](int64_t s1, int64_t s2) {
      const double t1 = (double)((d.G() * p.qtiles + s1 - 1) / s1);
      const double t2 = (double)((p.ktiles + s2 - 1) / s2);
      const double n1 = (double)(p.dkv_units * s1), n2 = (double)(p.dq_units * s2);
      return bwd_end(n1, 1.2 * (t1 + setup), n2, t2 + setup, slots, triangle) +
             (s1 > 1 ? join + 2 * part * n1 / slots : 0) + (s2 > 1 ? join + part * n2 / slots : 0);
    };
    double best = cost(1, 1);
    for (int which = 0; which < 4; ++which) {
      int& at = which & 1 ? p.dkv_splits : p.dq_splits;
      const int64_t tiles = which & 1 ? d.G() * p.qtiles : p.ktiles;
      const int64_t units = which & 1 ? p.dkv_units : p.dq_units;
      const int64_t hi = imin64(tiles, imax64(1, 4LL * slots / units));
      int64_t last = 0;
      for (int64_t s = 1; s <= hi; ++s) {
        const int64_t each = (tiles + s - 1) / s;
        if (each == last) continue;
        last = each;
        const double c = which & 1 ? cost(s, p.dq_splits) : cost(p.dkv_splits, s);
        if (c < best - 1e-9) best = c, at = (int)s;
      }
    }
    // Where a piece is short, a CTA that stays saves its start and end and loads
    // the next piece's K and V ahead (2 x 8 heads, D 64, the whole backward by
    // query tiles a piece, one CTA a piece against staying: 1 tile 375 and 265 us,
    // 2 253 and 198, 4 190 and 165, 8 155 and 142).  The border is a cautious one:
    // 16 tiles, 275 and 262, would still gain, and so would D 128 with its one
    // buffer of K and V (8 tiles 240 and 228); lengths that leave some pieces
    // empty, which staying CTAs cannot share out, were not timed there.
    p.stay = attn_dp(d.D) <= 64 && d.G() * p.qtiles <= 8 * p.dkv_splits;
    return p;
  }
  p.dkv_splits =
      choose_splits(p.dkv_units, d.G() * p.qtiles, slots, triangle, setup, join, 2 * part);
  p.dq_splits = choose_splits(p.dq_units, p.ktiles, slots, triangle, setup, join, part);
  return p;
}

namespace {
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
}  // namespace

AttnWs attn_ws_fwd(const AttnDims& d, const AttnPlan& p) {
  AttnWs w;
  w.part_ml = 256;
  const size_t recs = p.splits > 1 ? (size_t)p.units * p.splits * p.rows : 0;
  w.part_o = up256(w.part_ml + recs * 8);
  w.total = up256(w.part_o + recs * attn_dp(d.D) * 4);
  return w;
}

AttnWs attn_ws_bwd(const AttnDims& d, const AttnBwdPlan& p) {
  AttnWs w;
  const size_t dp = attn_dp(d.D);
  w.stats = 256;
  w.dq_part = up256(w.stats + (size_t)d.B * d.Hq * d.Nq * 8);
  const size_t nq = p.dq_splits > 1 ? (size_t)p.dq_units * p.dq_splits * p.tile * dp * 4 : 0;
  w.dkv_part = up256(w.dq_part + nq);
  const size_t nk = p.dkv_splits > 1 ? (size_t)p.dkv_units * p.dkv_splits * p.tile * dp * 8 : 0;
  w.total = up256(w.dkv_part + nk);
  return w;
}

// ---------------------------------------------------------- common kernels

namespace {

template <typename T>
__device__ __forceinline__ void put(T* p, float v);
template <>
__device__ __forceinline__ void put<float>(float* p, float v) { *p = v; }
template <>
__device__ __forceinline__ void put<__nv_bfloat16>(__nv_bfloat16* p, float v) {
  *p = __float2bfloat16_rn(v);
}

// row = (b H + h) N + i.  32-bit divisions where they reach.
struct RowOf {
  int i, h;
  int64_t b, bh;
  __device__ __forceinline__ RowOf(int64_t row, int N, int H) {
    if (row <= 0x7fffffffLL) {
      const unsigned r = (unsigned)row, x = r / (unsigned)N;
      i = (int)(r - x * N);
      const unsigned y = x / (unsigned)H;
      h = (int)(x - y * H);
      b = y;
      bh = x;
    } else {
      bh = row / N;
      i = (int)(row - bh * N);
      b = bh / H;
      h = (int)(bh - b * H);
    }
  }
};

// Joins the records (ref, sum, O) of the splits of one query row: weights
// 2^(ref_s - max ref), added in split order (the result does not depend on
// timing).  One warp per row, DP / 32 columns per lane.  Bound by latency:
// the records were just written and sit in L2.
template <typename T, int DP>
__global__ void __launch_bounds__(128) attn_join_kernel(const __grid_constant__ AttnFwdArgs A,
                                                        int rows) {
  pdl_wait();
  pdl_trigger();
  constexpr int E = DP / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= (int64_t)A.B * A.Hq * A.Nq) return;
  const RowOf at(row, A.Nq, A.Hq);
  const int i = at.i, h = at.h;
  const int64_t b = at.b, bh = at.bh;
  // where the forward kernel put the row
  int64_t unit;
  int r;
  if (A.hpt > 1) {
    unit = b * (A.Hq / A.hpt) + h / A.hpt;
    r = (h % A.hpt) * A.Nq + i;
  } else {
    unit = bh * A.qblocks + i / rows;
    r = i % rows;
  }
  const int64_t rec0 = unit * A.splits * rows + r;   // + s * rows
  float m = -INFINITY;
  for (int s = lane; s < A.splits; s += 32) {
    const float2 ml = A.part_ml[rec0 + (int64_t)s * rows];
    if (ml.y != 0.f) m = fmaxf(m, ml.x);
  }
#pragma unroll
  for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
  float acc[E] = {};
  float l = 0.f;
  for (int s0 = 0; s0 < A.splits; s0 += 32) {
    float2 ml = make_float2(-INFINITY, 0.f);
    if (s0 + lane < A.splits) ml = A.part_ml[rec0 + (int64_t)(s0 + lane) * rows];
    const float wl = ml.y != 0.f ? exp2f(ml.x - m) : 0.f;
    const int cnt = min(32, A.splits - s0);
    for (int s = 0; s < cnt; ++s) {
      const float ls = __shfl_sync(0xffffffffu, ml.y, s);
      const float w = __shfl_sync(0xffffffffu, wl, s);
      if (ls == 0.f) continue;
      l += w * ls;
      const float* o = A.part_o + (rec0 + (int64_t)(s0 + s) * rows) * DP + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += w * o[e];
    }
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  const int64_t col = b * A.y.sb + h * A.y.sh + i * A.y.sn + lane * E;
  T* y = (T*)A.Y + col;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if (lane * E + e >= A.D) continue;
    const float v = l != 0.f ? acc[e] * inv : 0.f;
    put<T>(y + e, v);
    if (sizeof(T) == 2 && A.Ylow) put<T>((T*)A.Ylow + col + e, v - to_f(y[e]));
  }
  if (A.lse && lane == 0) A.lse[row] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

// Backward, before the products: per query row -lse in log2 units (-inf for
// a row without weight, so that its P is exactly 0) and
// delta = sum_d dY Y (= sum_j P dP, the softmax's Jacobian term).  Y rounded to
// bf16 would put an error of 2^-8 of its terms into every dS of the row; with
// the remainder of that rounding (Ylow) it is 2^-16.
// LP lanes per row of 16-byte loads; bound by reading Y and dY once.
template <typename T, int LP>
__global__ void __launch_bounds__(256) attn_bwd_prep_kernel(const __grid_constant__ AttnBwdArgs A) {
  pdl_wait();
  pdl_trigger();
  constexpr int V = 16 / sizeof(T);
  if (blockIdx.x == 0 && threadIdx.x < 32)
    attn_check_lens(A.q_lens, A.k_lens, A.B, A.Nq, A.Nk, A.err);
  const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LP;
  const int sub = threadIdx.x % LP;
  const bool in = row < (int64_t)A.B * A.Hq * A.Nq;
  const RowOf at(in ? row : 0, A.Nq, A.Hq);
  const int i = at.i, h = at.h;
  const int64_t b = at.b;
  bool live = in;
  if (in && A.q_lens) live = i < A.q_lens[b];
  float s = 0.f;
  if (live && sub * V < A.D) {
    const int64_t at_y = b * A.y.sb + h * A.y.sh + i * A.y.sn + sub * V;
    const uint4 y = *reinterpret_cast<const uint4*>((const T*)A.Y + at_y);
    uint4 low = make_uint4(0, 0, 0, 0);
    if (sizeof(T) == 2 && A.Ylow) low = *reinterpret_cast<const uint4*>((const T*)A.Ylow + at_y);
    const uint4 g = *reinterpret_cast<const uint4*>((const T*)A.dY + b * A.dy.sb + h * A.dy.sh +
                                                    i * A.dy.sn + sub * V);
    const uint32_t yy[4] = {y.x, y.y, y.z, y.w}, gg[4] = {g.x, g.y, g.z, g.w};
    const uint32_t ll[4] = {low.x, low.y, low.z, low.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (sizeof(T) == 4) {
        s += __uint_as_float(yy[k]) * __uint_as_float(gg[k]);
      } else {
        s += (__uint_as_float(yy[k] << 16) + __uint_as_float(ll[k] << 16)) *
             __uint_as_float(gg[k] << 16);
        s += (__uint_as_float(yy[k] & 0xffff0000u) + __uint_as_float(ll[k] & 0xffff0000u)) *
             __uint_as_float(gg[k] & 0xffff0000u);
      }
    }
  }
#pragma unroll
  for (int k = LP / 2; k; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
  if (in && sub == 0) {
    const float lse = live ? A.lse[row] : -INFINITY;
    A.nl[row] = lse == -INFINITY ? -INFINITY : -lse * kLog2e;
    A.delta[row] = lse == -INFINITY ? 0.f : s;
  }
}

// dQ (WHICH = 0) or dK and dV (1) as the sum of the splits' float32 partials
// in split order, scaled and rounded once.  Four columns per thread; bound by
// reading the partials, which sit in L2.  Rows past the lengths become zeros.
template <typename T, int DP, int WHICH>
__global__ void __launch_bounds__(256) attn_bwd_sum_kernel(const __grid_constant__ AttnBwdArgs A) {
  pdl_wait();
  pdl_trigger();
  constexpr int C = DP / 4;
  const int H = WHICH ? A.Hk : A.Hq, N = WHICH ? A.Nk : A.Nq;
  const int tiles = WHICH ? A.ktiles : A.qtiles, splits = WHICH ? A.dkv_splits : A.dq_splits;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int col = (int)(id % C) * 4;
  const int64_t row = id / C;
  if (row >= (int64_t)A.B * H * N || col >= A.D) return;
  const RowOf at(row, N, H);
  const int n = at.i, h = at.h;
  const int64_t b = at.b, bh = at.bh;
  const int32_t* lens = WHICH ? A.k_lens : A.q_lens;
  const bool own = lens == nullptr || n < lens[b];
  const int64_t unit = bh * tiles + n / A.tile;
  const int r = n % A.tile;
#pragma unroll
  for (int k = 0; k <= WHICH; ++k) {
    // partials [unit][split][dK, dV][row][DP]
    const float* p = (WHICH ? A.dkv_part : A.dq_part) +
                     ((unit * splits * (1 + WHICH) + k) * A.tile + r) * (int64_t)DP + col;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x = 0; own && x < splits; ++x) {
      const float4 v = *reinterpret_cast<const float4*>(p + (int64_t)x * (1 + WHICH) * A.tile * DP);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    const Tok& t = WHICH ? (k ? A.dv : A.dk) : A.dq;
    T* out = (T*)(WHICH ? (k ? A.dV : A.dK) : A.dQ) + b * t.sb + h * t.sh + n * t.sn + col;
    const float f = k ? 1.f : A.scale;
    put<T>(out, s.x * f), put<T>(out + 1, s.y * f), put<T>(out + 2, s.z * f),
        put<T>(out + 3, s.w * f);
  }
}

template <typename T>
cudaError_t join_t(const AttnPlan& p, const AttnFwdArgs& a, int dp, cudaStream_t st) {
  const dim3 grid((unsigned)(((int64_t)a.B * a.Hq * a.Nq + 3) / 4));
  if (dp == 32) return launch_pdl(attn_join_kernel<T, 32>, grid, 128, 0, st, a, p.rows);
  if (dp == 64) return launch_pdl(attn_join_kernel<T, 64>, grid, 128, 0, st, a, p.rows);
  return launch_pdl(attn_join_kernel<T, 128>, grid, 128, 0, st, a, p.rows);
}

template <typename T>
cudaError_t prep_t(const AttnBwdArgs& a, cudaStream_t st) {
  const int lanes = (int)((a.D * sizeof(T) + 15) / 16);
  const int64_t rows = (int64_t)a.B * a.Hq * a.Nq;
#define FLARE_PREP(LP) \
  launch_pdl(attn_bwd_prep_kernel<T, LP>, dim3((unsigned)((rows * LP + 255) / 256)), 256, 0, st, a)
  if (lanes <= 4) return FLARE_PREP(4);
  if (lanes <= 8) return FLARE_PREP(8);
  if (lanes <= 16) return FLARE_PREP(16);
  return FLARE_PREP(32);
#undef FLARE_PREP
}

template <typename T, int WHICH>
cudaError_t sum_t(const AttnBwdArgs& a, int dp, cudaStream_t st) {
  const int64_t rows = WHICH ? (int64_t)a.B * a.Hk * a.Nk : (int64_t)a.B * a.Hq * a.Nq;
  const dim3 grid((unsigned)((rows * (dp / 4) + 255) / 256));
  if (dp == 32) return launch_pdl(attn_bwd_sum_kernel<T, 32, WHICH>, grid, 256, 0, st, a);
  if (dp == 64) return launch_pdl(attn_bwd_sum_kernel<T, 64, WHICH>, grid, 256, 0, st, a);
  return launch_pdl(attn_bwd_sum_kernel<T, 128, WHICH>, grid, 256, 0, st, a);
}

}  // namespace

cudaError_t launch_attn_join(const AttnPlan& p, const AttnFwdArgs& a, int dp, flare_dtype_t dt,
                             cudaStream_t st) {
  return dt == FLARE_BF16 ? join_t<__nv_bfloat16>(p, a, dp, st) : join_t<float>(p, a, dp, st);
}

cudaError_t launch_attn_bwd_prep(const AttnBwdArgs& a, flare_dtype_t dt, cudaStream_t st) {
  return dt == FLARE_BF16 ? prep_t<__nv_bfloat16>(a, st) : prep_t<float>(a, st);
}

cudaError_t launch_attn_bwd_sum(const AttnBwdArgs& a, int dp, flare_dtype_t dt, int which,
                                cudaStream_t st) {
  if (dt == FLARE_BF16)
    return which ? sum_t<__nv_bfloat16, 1>(a, dp, st) : sum_t<__nv_bfloat16, 0>(a, dp, st);
  return which ? sum_t<float, 1>(a, dp, st) : sum_t<float, 0>(a, dp, st);
}

// ------------------------------------------------------------- validation

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    return 148;   // B200
  }
  return n;
}

namespace {

flare_status_t sizes(int64_t B, int64_t Hq, int64_t Hk, int64_t Nq, int64_t Nk, int64_t D,
                     flare_dtype_t dt) {
  if (B < 1 || Hq < 1 || Hk < 1 || Nq < 1 || Nk < 1 || D < 1) return FLARE_ERR_INVALID_ARG;
  if (dt != FLARE_F32 && dt != FLARE_BF16) return FLARE_ERR_INVALID_ARG;
  if (B > (1LL << 20) || Hq > (1LL << 16) || Hk > (1LL << 16)) return FLARE_ERR_INVALID_ARG;
  if (Hq % Hk != 0) return FLARE_ERR_INVALID_ARG;
  if (D % 8 != 0 || D > 128) return FLARE_ERR_UNSUPPORTED;
  // 32-bit token indices (with room for a tile before and after)
  if (Nq > (1LL << 30) || Nk > (1LL << 30)) return FLARE_ERR_UNSUPPORTED;
  if (B * Hq > (1LL << 24)) return FLARE_ERR_UNSUPPORTED;
  if ((double)B * Hq * Nq * D >= 1099511627776.0 || (double)B * Hk * Nk * D >= 1099511627776.0)
    return FLARE_ERR_INVALID_ARG;   // 2^40
  return FLARE_OK;
}

}  // namespace

flare_status_t check_ptr(const void* p) {
  return (p != nullptr && ((uintptr_t)p & 15u) == 0) ? FLARE_OK : FLARE_ERR_INVALID_ARG;
}

// The rows of an output do not overlap when, in order of stride, every
// dimension with more than one entry steps over all the rows of the
// dimensions inside it.
flare_status_t check_tok(const flare_strides_t* st, int64_t B, int64_t H, int64_t N, int64_t D,
                         flare_dtype_t dt, bool output, Tok* out) {
  const int64_t esz = dt == FLARE_F32 ? 4 : 2;
  int64_t s[3] = {H * N * D, N * D, D};
  if (st) s[0] = st->b_stride, s[1] = st->h_stride, s[2] = st->n_stride;
  int64_t e[3] = {B, H, N};
  for (int i = 0; i < 3; ++i) {
    if (e[i] == 1) {
      s[i] = i < 2 ? 0 : 16 / esz;   // not used
      continue;
    }
    const bool zero_ok = !output && i < 2;
    if (s[i] < (zero_ok ? 0 : 1) || s[i] >= (1LL << 40) / esz) return FLARE_ERR_INVALID_ARG;
    if ((s[i] * esz) % 16 != 0) return FLARE_ERR_UNSUPPORTED;
  }
  *out = Tok{s[0], s[1], s[2]};
  if (!output) return FLARE_OK;
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (s[j] < s[i]) {
        const int64_t ts = s[i], te = e[i];
        s[i] = s[j], e[i] = e[j];
        s[j] = ts, e[j] = te;
      }
  int64_t span = D;
  for (int i = 0; i < 3; ++i) {
    if (e[i] == 1) continue;
    if (s[i] < span) return FLARE_ERR_INVALID_ARG;
    span += s[i] * (e[i] - 1);
  }
  return FLARE_OK;
}

flare_status_t check_workspace(const void* ws, size_t bytes, size_t need) {
  if (ws == nullptr || ((uintptr_t)ws & 255u) != 0) return FLARE_ERR_WORKSPACE;
  return bytes >= need ? FLARE_OK : FLARE_ERR_WORKSPACE;
}

namespace {

flare_status_t lens(const int32_t* p) {
  return ((uintptr_t)p & 3u) == 0 ? FLARE_OK : FLARE_ERR_INVALID_ARG;
}

AttnDims dims(int64_t B, int64_t Hq, int64_t Hk, int64_t Nq, int64_t Nk, int64_t D, int causal) {
  AttnDims d;
  d.B = B, d.Hq = Hq, d.Hk = Hk, d.Nq = Nq, d.Nk = Nk, d.D = D;
  d.causal = causal != 0;
  return d;
}

// Zero strides (broadcast, or a dimension of one entry) -> one entry in the
// tensor map, coordinate 0.
int bcast_bits(const Tok& t, int k) {
  return (t.sb == 0 ? 1 << k : 0) | (t.sh == 0 ? 8 << k : 0);
}

}  // namespace
}  // namespace flare

using namespace flare;

extern "C" {

size_t flare_attn_workspace_size(int backward, int64_t B, int64_t Hq, int64_t Hk, int64_t Nq,
                                 int64_t Nk, int64_t D, flare_dtype_t dt) {
  if (sizes(B, Hq, Hk, Nq, Nk, D, dt) != FLARE_OK) return 0;
  const int sms = sm_count();
  size_t most = 0;
  // the plan of a call depends on its mask and on whether its queries are
  // broadcast over the heads: room for any
  for (int k = 0; k < 4; ++k) {
    AttnDims d = dims(B, Hq, Hk, Nq, Nk, D, k & 1);
    d.q.sh = k >> 1;
    const size_t need = backward ? attn_ws_bwd(d, attn_bwd_plan(d, dt, sms)).total
                                 : attn_ws_fwd(d, attn_plan(d, dt, sms)).total;
    most = need > most ? need : most;
  }
  return most;
}

flare_status_t flare_attn_plan(int backward, int64_t B, int64_t Hq, int64_t Hk, int64_t Nq,
                               int64_t Nk, int64_t D, flare_dtype_t dt, int causal,
                               int64_t* plan) {
  if (plan == nullptr) return FLARE_ERR_INVALID_ARG;
  FLARE_TRY(sizes(B, Hq, Hk, Nq, Nk, D, dt));
  AttnDims d = dims(B, Hq, Hk, Nq, Nk, D, causal);
  d.q.sh = 1;   // every head has queries of its own
  if (backward) {
    const AttnBwdPlan p = attn_bwd_plan(d, dt, sm_count());
    plan[0] = p.dkv_splits, plan[1] = p.dq_splits, plan[2] = p.stay;
  } else {
    const AttnPlan p = attn_plan(d, dt, sm_count());
    plan[0] = p.qt, plan[1] = p.hpt, plan[2] = p.splits;
  }
  return FLARE_OK;
}

flare_status_t flare_attn_fwd(const void* Q, const void* K, const void* V, void* Y,
                              const flare_strides_t* strides, const int32_t* q_lens,
                              const int32_t* k_lens, int64_t B, int64_t Hq, int64_t Hk, int64_t Nq,
                              int64_t Nk, int64_t D, flare_dtype_t dt, float scale, int causal,
                              float* lse_save, void* y_low_save, void* workspace,
                              size_t workspace_bytes, void* stream) {
  FLARE_TRY(sizes(B, Hq, Hk, Nq, Nk, D, dt));
  if (!std::isfinite(scale) || !(scale > 0.f)) return FLARE_ERR_INVALID_ARG;
  const void* must[4] = {Q, K, V, Y};
  for (const void* p : must) FLARE_TRY(check_ptr(p));
  if (lse_save) FLARE_TRY(check_ptr(lse_save));
  if (y_low_save) FLARE_TRY(check_ptr(y_low_save));
  FLARE_TRY(lens(q_lens));
  FLARE_TRY(lens(k_lens));
  AttnDims d = dims(B, Hq, Hk, Nq, Nk, D, causal);
  FLARE_TRY(check_tok(strides ? strides + 0 : nullptr, B, Hq, Nq, D, dt, false, &d.q));
  FLARE_TRY(check_tok(strides ? strides + 1 : nullptr, B, Hk, Nk, D, dt, false, &d.k));
  FLARE_TRY(check_tok(strides ? strides + 2 : nullptr, B, Hk, Nk, D, dt, false, &d.v));
  FLARE_TRY(check_tok(strides ? strides + 3 : nullptr, B, Hq, Nq, D, dt, true, &d.y));
  const AttnPlan p = attn_plan(d, dt, sm_count());
  const AttnWs w = attn_ws_fwd(d, p);
  FLARE_TRY(check_workspace(workspace, workspace_bytes, w.total));
  if (p.units * p.splits > 0x7fffffffLL || B * Hq * Nq > 0x7fffffffLL * 4)
    return FLARE_ERR_UNSUPPORTED;   // grid.x
  note_error("%s", "");
  char* ws = (char*)workspace;
  cudaStream_t st = (cudaStream_t)stream;
  AttnFwdArgs a = {};
  a.B = (int)B, a.Hq = (int)Hq, a.Hk = (int)Hk, a.G = (int)(Hq / Hk);
  a.Nq = (int)Nq, a.Nk = (int)Nk, a.D = (int)D;
  a.hpt = p.hpt, a.qblocks = (int)p.qblocks, a.splits = p.splits, a.causal = d.causal;
  a.c = scale * kLog2e;
  a.q_lens = q_lens, a.k_lens = k_lens;
  a.q = d.q, a.k = d.k, a.v = d.v, a.y = d.y;
  a.Y = Y;
  a.Ylow = dt == FLARE_BF16 ? y_low_save : nullptr;
  a.lse = lse_save;
  a.part_ml = (float2*)(ws + w.part_ml);
  a.part_o = (float*)(ws + w.part_o);
  a.err = (uint32_t*)ws;
  a.bcast = bcast_bits(d.q, 0) | bcast_bits(d.k, 1) | bcast_bits(d.v, 2);
  FLARE_CUDA(attn_tc(dt) ? launch_attn_fwd_tc(Q, K, V, d, p, a, st)
                         : launch_attn_fwd_simt(Q, K, V, p, a, st));
  if (p.splits > 1) FLARE_CUDA(launch_attn_join(p, a, attn_dp(D), dt, st));
  return FLARE_OK;
}

flare_status_t flare_attn_bwd(const void* Q, const void* K, const void* V, const void* Y,
                              const void* y_low, const void* dY, const float* lse, void* dQ,
                              void* dK, void* dV, const flare_strides_t* strides,
                              const int32_t* q_lens, const int32_t* k_lens, int64_t B, int64_t Hq,
                              int64_t Hk, int64_t Nq, int64_t Nk, int64_t D, flare_dtype_t dt,
                              float scale, int causal, void* workspace, size_t workspace_bytes,
                              void* stream) {
  FLARE_TRY(sizes(B, Hq, Hk, Nq, Nk, D, dt));
  if (!std::isfinite(scale) || !(scale > 0.f)) return FLARE_ERR_INVALID_ARG;
  // dQ, or dK and dV together, may be left out
  if ((dK == nullptr) != (dV == nullptr) || (dQ == nullptr && dK == nullptr))
    return FLARE_ERR_INVALID_ARG;
  const void* must[9] = {Q,   K, V, Y, dY, lse, dQ ? dQ : dK, dK ? dK : dQ, dV ? dV : dQ};
  for (const void* p : must) FLARE_TRY(check_ptr(p));
  if (y_low) FLARE_TRY(check_ptr(y_low));
  FLARE_TRY(lens(q_lens));
  FLARE_TRY(lens(k_lens));
  AttnDims d = dims(B, Hq, Hk, Nq, Nk, D, causal);
  Tok* where[8] = {&d.q, &d.k, &d.v, &d.y, &d.dy, &d.dq, &d.dk, &d.dv};
  for (int i = 0; i < 8; ++i) {
    const bool keys = i == 1 || i == 2 || i == 6 || i == 7;
    if ((i == 5 && !dQ) || (i > 5 && !dK)) continue;
    FLARE_TRY(check_tok(strides ? strides + i : nullptr, B, keys ? Hk : Hq, keys ? Nk : Nq, D, dt,
                        i >= 5, where[i]));
  }
  const AttnBwdPlan p = attn_bwd_plan(d, dt, sm_count());
  const AttnWs w = attn_ws_bwd(d, p);
  FLARE_TRY(check_workspace(workspace, workspace_bytes, w.total));
  const int64_t most = 0x7fffffffLL;
  if (p.dkv_units * p.dkv_splits + p.dq_units * p.dq_splits > most ||
      B * Hq * Nq > most * 8 || B * Hk * Nk > most * 8)
    return FLARE_ERR_UNSUPPORTED;   // grid.x
  note_error("%s", "");
  char* ws = (char*)workspace;
  cudaStream_t st = (cudaStream_t)stream;
  AttnBwdArgs a = {};
  a.B = (int)B, a.Hq = (int)Hq, a.Hk = (int)Hk, a.G = (int)(Hq / Hk);
  a.Nq = (int)Nq, a.Nk = (int)Nk, a.D = (int)D;
  a.tile = p.tile, a.ktiles = (int)p.ktiles, a.qtiles = (int)p.qtiles;
  a.dkv_splits = p.dkv_splits, a.dq_splits = p.dq_splits, a.causal = d.causal;
  a.dkv_units = p.dkv_units, a.dq_units = p.dq_units;
  a.scale = scale, a.c = scale * kLog2e;
  a.q_lens = q_lens, a.k_lens = k_lens;
  a.q = d.q, a.k = d.k, a.v = d.v, a.y = d.y, a.dy = d.dy, a.dq = d.dq, a.dk = d.dk, a.dv = d.dv;
  a.Q = Q, a.K = K, a.V = V, a.Y = Y, a.dY = dY, a.lse = lse;
  a.Ylow = dt == FLARE_BF16 ? y_low : nullptr;
  a.dQ = dQ, a.dK = dK, a.dV = dV;
  a.nl = (float*)(ws + w.stats);
  a.delta = a.nl + B * Hq * Nq;
  a.dq_part = (float*)(ws + w.dq_part);
  a.dkv_part = (float*)(ws + w.dkv_part);
  a.err = (uint32_t*)ws;
  a.bcast = bcast_bits(d.q, 0) | bcast_bits(d.k, 1) | bcast_bits(d.v, 2) |
            (d.dy.sb == 0 ? 64 : 0) | (d.dy.sh == 0 ? 128 : 0);
  FLARE_CUDA(launch_attn_bwd_prep(a, dt, st));
  FLARE_CUDA(attn_tc(dt) ? launch_attn_bwd_tc(d, p, a, st) : launch_attn_bwd_simt(p, a, st));
  if (dK && p.dkv_splits > 1) FLARE_CUDA(launch_attn_bwd_sum(a, attn_dp(D), dt, 1, st));
  if (dQ && p.dq_splits > 1) FLARE_CUDA(launch_attn_bwd_sum(a, attn_dp(D), dt, 0, st));
  return FLARE_OK;
}

}  // extern "C"

// Softmax attention forward and backward on the CUDA cores: float32 inputs,
// whose products the tensor cores' bf16 operands would round.
//
// Tiles of 64 queries x 64 keys, 128 threads, each with 8 x 4 logits: thread
// (ty, tx) = (tid / 16, tid % 16) owns rows 8 ty + i and columns tx + 16 c.
// Every product is one of two loops over shared memory:
//   nt: C[r][c] += sum_d A[r][d] B[c][d]      (logits, dP)
//   nn: C[r][e] += sum_k P[r][k] B[k][e]      (O, dV, dK, dQ)
// Rows are padded by 4 floats, so that both are free of bank conflicts.
// Bound: 128 FMAs per 12 (nt) or per 8 + E (nn, E columns a thread) 16-byte
// shared-memory reads, i.e. by shared memory and the FMA pipe about equally.
#include "flare_attn.cuh"

namespace flare {
namespace {

constexpr int kT = 64;             // queries and keys per tile
constexpr int kNT = 128;
constexpr int kR = 8;              // rows per thread
constexpr int kPS = kT + 4;        // row pitch of a 64 x 64 tile

// Rows [row0, row0 + 64) of p, the first n valid rows and D columns of it;
// zeros elsewhere.
template <int DP>
__device__ __forceinline__ void load_rows(float* dst, const float* p, int64_t sn, int row0, int n,
                                          int D) {
  constexpr int C = DP / 4;
#pragma unroll
  for (int x = threadIdx.x; x < kT * C; x += kNT) {
    const int r = x / C, c = (x % C) * 4;
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row0 + r < n && c < D) f = *reinterpret_cast<const float4*>(p + (row0 + r) * sn + c);
    *reinterpret_cast<float4*>(dst + r * (DP + 4) + c) = f;
  }
}

template <int DP>
__device__ __forceinline__ void prod_nt(const float* A, const float* B, int ty, int tx,
                                        float (&c)[kR][4]) {
#pragma unroll
  for (int i = 0; i < kR; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) c[i][j] = 0.f;
#pragma unroll 4
  for (int d = 0; d < DP; d += 4) {
    float4 a[kR], b[4];
#pragma unroll
    for (int i = 0; i < kR; ++i) a[i] = *(const float4*)(A + (kR * ty + i) * (DP + 4) + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = *(const float4*)(B + (tx + 16 * j) * (DP + 4) + d);
#pragma unroll
    for (int i = 0; i < kR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c[i][j] = fmaf(a[i].x, b[j].x, c[i][j]);
        c[i][j] = fmaf(a[i].y, b[j].y, c[i][j]);
        c[i][j] = fmaf(a[i].z, b[j].z, c[i][j]);
        c[i][j] = fmaf(a[i].w, b[j].w, c[i][j]);
      }
  }
}

// Columns of a thread in an nn product: DP / 16 of them, in groups of W
// consecutive ones starting at out_col(g).
template <int DP>
struct Cols {
  static constexpr int E = DP / 16, W = E < 4 ? E : 4, NG = E / W;
  static __device__ __forceinline__ int at(int tx, int g) { return tx * W + 64 * g; }
};

template <int DP>
__device__ __forceinline__ void prod_nn(const float* P, const float* B, int ty, int tx,
                                        float (&c)[kR][DP / 16]) {
  using C = Cols<DP>;
#pragma unroll 2
  for (int k = 0; k < kT; k += 4) {
    float p[kR][4];
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const float4 v = *(const float4*)(P + (kR * ty + i) * kPS + k);
      p[i][0] = v.x, p[i][1] = v.y, p[i][2] = v.z, p[i][3] = v.w;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int g = 0; g < C::NG; ++g) {
        float b[C::W];
        const float* src = B + (k + q) * (DP + 4) + C::at(tx, g);
        if constexpr (C::W == 4) {
          const float4 v = *(const float4*)src;
          b[0] = v.x, b[1] = v.y, b[2] = v.z, b[3] = v.w;
        } else {
          const float2 v = *(const float2*)src;
          b[0] = v.x, b[1] = v.y;
        }
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
          for (int w = 0; w < C::W; ++w)
            c[i][g * C::W + w] = fmaf(p[i][q], b[w], c[i][g * C::W + w]);
      }
  }
}

// Writes a thread's rows times f as rows [row0, n) of a token tensor.
template <int DP>
__device__ __forceinline__ void put_rows(float* p, int64_t sn, int row0, int n, int D, int ty,
                                         int tx, const float (&c)[kR][DP / 16], float f) {
  using C = Cols<DP>;
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int r = row0 + kR * ty + i;
    if (r >= n) continue;
#pragma unroll
    for (int g = 0; g < C::NG; ++g)
#pragma unroll
      for (int w = 0; w < C::W; ++w) {
        const int col = C::at(tx, g) + w;
        if (col < D) p[r * sn + col] = c[i][g * C::W + w] * f;
      }
  }
}

// Writes a thread's rows to a float32 record [64][DP].
template <int DP>
__device__ __forceinline__ void put_part(float* p, int ty, int tx, const float (&c)[kR][DP / 16]) {
  using C = Cols<DP>;
#pragma unroll
  for (int i = 0; i < kR; ++i)
#pragma unroll
    for (int e = 0; e < C::E; ++e)
      p[(kR * ty + i) * DP + C::at(tx, e / C::W) + e % C::W] = c[i][e];
}

__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int k = 8; k; k >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, k));
  return v;
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int k = 8; k; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
  return v;
}

template <int DP>
constexpr int tile_floats() { return kT * (DP + 4); }
constexpr int kPFloats = kT * kPS;

// Forward: one CTA = 64 query rows (of one head, or of hpt heads that share
// a key head) and one part of the key tiles.  The running maximum and sum of
// a row are held by the 16 threads that share it.  P overwrites the key tile.
template <int DP>
__global__ void __launch_bounds__(kNT)
    attn_fwd_simt_kernel(const float* __restrict__ Q, const float* __restrict__ K,
                         const float* __restrict__ V, const __grid_constant__ AttnFwdArgs A) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ float sm[];
  float* qs = sm;
  float* vs = qs + tile_floats<DP>();
  float* ks = vs + tile_floats<DP>();   // max(key tile, P)
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  if (blockIdx.x == 0 && threadIdx.x < 32)
    attn_check_lens(A.q_lens, A.k_lens, A.B, A.Nq, A.Nk, A.err);

  const int hgroups = A.Hq / A.hpt;
  const int split = (int)(blockIdx.x % A.splits);
  const int u = blockIdx.x / A.splits;
  // causal: the longest rows of all heads first
  const int BHG = A.B * hgroups;
  const int qb = A.causal ? A.qblocks - 1 - u / BHG : u % A.qblocks;
  const int bhg = A.causal ? u % BHG : u / A.qblocks;
  const int b = bhg / hgroups, h0 = (bhg % hgroups) * A.hpt, hk = h0 / (A.Hq / A.Hk);
  const int64_t rec = (((int64_t)bhg * A.qblocks + qb) * A.splits + split) * kT;
  const AttnSeq sq(A.q_lens, A.k_lens, b, A.Nq, A.Nk, A.causal != 0);
  const bool packed = A.hpt > 1;
  const int q0 = qb * kT;
  const int nall = q0 < sq.ql ? sq.key_tiles(packed ? A.Nq - 1 : q0 + kT - 1, kT) : 0;
  const Part part(nall, split, A.splits);
  const int lo = part.lo, hi = lo + part.count;

  int qi[kR], qh[kR];
  bool live[kR];
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int r = kR * ty + i;
    qh[i] = packed ? h0 + min(r / A.Nq, A.hpt - 1) : h0;
    qi[i] = packed ? r % A.Nq : q0 + r;
    live[i] = packed ? r < A.hpt * A.Nq : qi[i] < A.Nq;
  }
  if (packed) {
    for (int g = 0; g < A.hpt; ++g) {   // one head's queries at a time
      const float* p = Q + b * A.q.sb + (h0 + g) * A.q.sh;
      for (int x = threadIdx.x; x < A.Nq * DP; x += kNT) {
        const int i = x / DP, d = x % DP;
        float f = 0.f;
        if (i < sq.ql && d < A.D) f = p[i * A.q.sn + d];
        qs[(g * A.Nq + i) * (DP + 4) + d] = f;
      }
    }
    for (int x = threadIdx.x + A.hpt * A.Nq * DP; x < kT * DP; x += kNT)
      qs[x / DP * (DP + 4) + x % DP] = 0.f;
  } else {
    load_rows<DP>(qs, Q + b * A.q.sb + h0 * A.q.sh, A.q.sn, q0, sq.ql, A.D);
  }

  float m[kR], l[kR], o[kR][DP / 16];
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < DP / 16; ++e) o[i][e] = 0.f;
  }
  const float* kp = K + b * A.k.sb + hk * A.k.sh;
  const float* vp = V + b * A.v.sb + hk * A.v.sh;
  for (int t = lo; t < hi; ++t) {
    __syncthreads();
    load_rows<DP>(ks, kp, A.k.sn, t * kT, sq.kl, A.D);
    load_rows<DP>(vs, vp, A.v.sn, t * kT, sq.kl, A.D);
    __syncthreads();
    float s[kR][4];
    prod_nt<DP>(qs, ks, ty, tx, s);
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const int last = sq.causal ? min(sq.kl - 1, qi[i] + sq.off) : sq.kl - 1;
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = t * kT + tx + 16 * j <= last ? s[i][j] * A.c : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
      mx = fmaxf(m[i], row_max(mx));
      const float ref = mx == -INFINITY ? 0.f : mx;
      const float f = exp2f(m[i] - ref);
      m[i] = mx;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = exp2f(s[i][j] - ref);
        sum += s[i][j];
      }
      l[i] = l[i] * f + sum;
#pragma unroll
      for (int e = 0; e < DP / 16; ++e) o[i][e] *= f;
    }
    __syncthreads();   // the key tile is read
#pragma unroll
    for (int i = 0; i < kR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) ks[(kR * ty + i) * kPS + tx + 16 * j] = s[i][j];
    __syncthreads();
    prod_nn<DP>(ks, vs, ty, tx, o);
  }
#pragma unroll
  for (int i = 0; i < kR; ++i) l[i] = row_sum(l[i]);   // each thread held 4 columns of its rows
  if (A.splits > 1) {
#pragma unroll
    for (int i = 0; i < kR; ++i)
      if (tx == 0 && live[i])
        A.part_ml[rec + kR * ty + i] = make_float2(m[i], qi[i] < sq.ql ? l[i] : 0.f);
    put_part<DP>(A.part_o + rec * DP, ty, tx, o);
    return;
  }
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    if (!live[i]) continue;
    const bool some = qi[i] < sq.ql && l[i] != 0.f;
    float* y = (float*)A.Y + b * A.y.sb + qh[i] * A.y.sh + qi[i] * A.y.sn;
#pragma unroll
    for (int e = 0; e < DP / 16; ++e) {
      const int col = Cols<DP>::at(tx, e / Cols<DP>::W) + e % Cols<DP>::W;
      if (col < A.D) y[col] = some ? o[i][e] / l[i] : 0.f;
    }
    if (A.lse && tx == 0)
      A.lse[((int64_t)b * A.Hq + qh[i]) * A.Nq + qi[i]] =
          some ? (m[i] + log2f(l[i])) * kLn2 : -INFINITY;
  }
}

// dK and dV of 64 keys: over the query tiles of the heads that share them,
//   P^T = 2^(c K Q^T + nl),  dV += P^T dY,
//   dS^T = P^T (V dY^T - delta),  dK += dS^T Q.
template <int DP>
__global__ void __launch_bounds__(kNT) attn_dkv_simt_kernel(const __grid_constant__ AttnBwdArgs A) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ float sm[];
  float* ks = sm;
  float* vs = ks + tile_floats<DP>();
  float* qs = vs + tile_floats<DP>();
  float* gs = qs + tile_floats<DP>();
  float* ps = gs + tile_floats<DP>();
  float* nls = ps + kPFloats;
  float* dls = nls + kT;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const int split = (int)(blockIdx.x % A.dkv_splits);
  const int unit = blockIdx.x / A.dkv_splits;
  const int BH = A.B * A.Hk;
  const int kt = A.causal ? unit / BH : unit % A.ktiles;
  const int bh = A.causal ? unit % BH : unit / A.ktiles;
  const int b = bh / A.Hk, hk = bh % A.Hk, G = A.Hq / A.Hk;
  const AttnSeq sq(A.q_lens, A.k_lens, b, A.Nq, A.Nk, A.causal != 0);
  const int k0 = kt * kT;
  const int first = sq.first_query_tile(k0, kT);
  const int per = k0 < sq.kl ? max(0, (sq.ql + kT - 1) / kT - first) : 0;   // tiles of a head
  const Part part(per * G, split, A.dkv_splits);
  const int lo = part.lo, hi = lo + part.count;
  load_rows<DP>(ks, (const float*)A.K + b * A.k.sb + hk * A.k.sh, A.k.sn, k0, sq.kl, A.D);
  load_rows<DP>(vs, (const float*)A.V + b * A.v.sb + hk * A.v.sh, A.v.sn, k0, sq.kl, A.D);
  float dk[kR][DP / 16] = {}, dv[kR][DP / 16] = {};
  for (int it = lo; it < hi; ++it) {
    const int h = hk * G + it / per, q0 = (first + it % per) * kT;
    __syncthreads();
    load_rows<DP>(qs, (const float*)A.Q + b * A.q.sb + h * A.q.sh, A.q.sn, q0, sq.ql, A.D);
    load_rows<DP>(gs, (const float*)A.dY + b * A.dy.sb + h * A.dy.sh, A.dy.sn, q0, sq.ql, A.D);
    if (threadIdx.x < kT) {
      const int64_t row = ((int64_t)b * A.Hq + h) * A.Nq + q0 + threadIdx.x;
      const bool in = q0 + threadIdx.x < sq.ql;
      nls[threadIdx.x] = in ? A.nl[row] : -INFINITY;
      dls[threadIdx.x] = in ? A.delta[row] : 0.f;
    }
    __syncthreads();
    float s[kR][4], dp[kR][4];
    prod_nt<DP>(ks, qs, ty, tx, s);
    prod_nt<DP>(vs, gs, ty, tx, dp);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int q = tx + 16 * j;
      const float nl = nls[q], dl = dls[q];
      const int last = sq.causal ? min(sq.kl - 1, q0 + q + sq.off) : sq.kl - 1;
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        const bool seen = k0 + kR * ty + i <= last && nl != -INFINITY;
        s[i][j] = seen ? exp2f(fmaf(s[i][j], A.c, nl)) : 0.f;
        dp[i][j] = seen ? s[i][j] * (dp[i][j] - dl) : 0.f;
        ps[(kR * ty + i) * kPS + q] = s[i][j];
      }
    }
    __syncthreads();
    prod_nn<DP>(ps, gs, ty, tx, dv);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < kR; ++i) ps[(kR * ty + i) * kPS + tx + 16 * j] = dp[i][j];
    __syncthreads();
    prod_nn<DP>(ps, qs, ty, tx, dk);
  }
  if (A.dkv_splits > 1) {
    float* p = A.dkv_part + (((int64_t)bh * A.ktiles + kt) * A.dkv_splits + split) * 2 * kT * DP;
    put_part<DP>(p, ty, tx, dk);
    put_part<DP>(p + kT * DP, ty, tx, dv);
    return;
  }
  put_rows<DP>((float*)A.dK + b * A.dk.sb + hk * A.dk.sh, A.dk.sn, k0, A.Nk, A.D, ty, tx, dk,
               A.scale);
  put_rows<DP>((float*)A.dV + b * A.dv.sb + hk * A.dv.sh, A.dv.sn, k0, A.Nk, A.D, ty, tx, dv, 1.f);
}

// dQ of 64 queries: over the key tiles they see, dQ += (P (dY V^T - delta)) K.
template <int DP>
__global__ void __launch_bounds__(kNT) attn_dq_simt_kernel(const __grid_constant__ AttnBwdArgs A) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ float sm[];
  float* qs = sm;
  float* gs = qs + tile_floats<DP>();
  float* ks = gs + tile_floats<DP>();
  float* vs = ks + tile_floats<DP>();
  float* ps = vs + tile_floats<DP>();
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const int split = (int)(blockIdx.x % A.dq_splits);
  const int unit = blockIdx.x / A.dq_splits;
  const int BH = A.B * A.Hq;
  const int qt = A.causal ? A.qtiles - 1 - unit / BH : unit % A.qtiles;
  const int bh = A.causal ? unit % BH : unit / A.qtiles;
  const int b = bh / A.Hq, h = bh % A.Hq, hk = h / (A.Hq / A.Hk);
  const AttnSeq sq(A.q_lens, A.k_lens, b, A.Nq, A.Nk, A.causal != 0);
  const int q0 = qt * kT;
  const int nall = q0 < sq.ql ? sq.key_tiles(q0 + kT - 1, kT) : 0;
  const Part part(nall, split, A.dq_splits);
  const int lo = part.lo, hi = lo + part.count;
  load_rows<DP>(qs, (const float*)A.Q + b * A.q.sb + h * A.q.sh, A.q.sn, q0, sq.ql, A.D);
  load_rows<DP>(gs, (const float*)A.dY + b * A.dy.sb + h * A.dy.sh, A.dy.sn, q0, sq.ql, A.D);
  float nl[kR], dl[kR];
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int q = q0 + kR * ty + i;
    const int64_t row = ((int64_t)b * A.Hq + h) * A.Nq + q;
    nl[i] = q < sq.ql ? A.nl[row] : -INFINITY;
    dl[i] = q < sq.ql ? A.delta[row] : 0.f;
  }
  float dq[kR][DP / 16] = {};
  const float* kp = (const float*)A.K + b * A.k.sb + hk * A.k.sh;
  const float* vp = (const float*)A.V + b * A.v.sb + hk * A.v.sh;
  for (int t = lo; t < hi; ++t) {
    __syncthreads();
    load_rows<DP>(ks, kp, A.k.sn, t * kT, sq.kl, A.D);
    load_rows<DP>(vs, vp, A.v.sn, t * kT, sq.kl, A.D);
    __syncthreads();
    float s[kR][4], dp[kR][4];
    prod_nt<DP>(qs, ks, ty, tx, s);
    prod_nt<DP>(gs, vs, ty, tx, dp);
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const int last =
          sq.causal ? min(sq.kl - 1, q0 + kR * ty + i + sq.off) : sq.kl - 1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool seen = t * kT + tx + 16 * j <= last && nl[i] != -INFINITY;
        const float p = seen ? exp2f(fmaf(s[i][j], A.c, nl[i])) : 0.f;
        ps[(kR * ty + i) * kPS + tx + 16 * j] = seen ? p * (dp[i][j] - dl[i]) : 0.f;
      }
    }
    __syncthreads();
    prod_nn<DP>(ps, ks, ty, tx, dq);
  }
  if (A.dq_splits > 1) {
    // records by query tile, as the sum kernel counts them
    put_part<DP>(A.dq_part + (((int64_t)bh * A.qtiles + qt) * A.dq_splits + split) * kT * DP, ty,
                 tx, dq);
    return;
  }
  put_rows<DP>((float*)A.dQ + b * A.dq.sb + h * A.dq.sh, A.dq.sn, q0, A.Nq, A.D, ty, tx, dq,
               A.scale);
}

template <typename... KA, typename... As>
cudaError_t go(void (*kernel)(KA...), int64_t grid, int smem, cudaStream_t st, As... args) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, dim3((unsigned)grid), kNT, smem, st, args...);
  return e != cudaSuccess ? e : cudaPeekAtLastError();
}

template <int DP>
cudaError_t fwd_t(const void* Q, const void* K, const void* V, const AttnPlan& p,
                  const AttnFwdArgs& a, cudaStream_t st) {
  const int last = tile_floats<DP>() > kPFloats ? tile_floats<DP>() : kPFloats;
  return go(attn_fwd_simt_kernel<DP>, p.units * p.splits, (2 * tile_floats<DP>() + last) * 4, st,
            (const float*)Q, (const float*)K, (const float*)V, a);
}

template <int DP>
cudaError_t bwd_t(const AttnBwdPlan& p, const AttnBwdArgs& a, cudaStream_t st) {
  const int smem = (4 * tile_floats<DP>() + kPFloats + 2 * kT) * 4;
  cudaError_t e = cudaSuccess;
  if (a.dK) e = go(attn_dkv_simt_kernel<DP>, p.dkv_units * p.dkv_splits, smem, st, a);
  if (e == cudaSuccess && a.dQ)
    e = go(attn_dq_simt_kernel<DP>, p.dq_units * p.dq_splits, smem, st, a);
  return e;
}

}  // namespace

cudaError_t launch_attn_fwd_simt(const void* Q, const void* K, const void* V, const AttnPlan& p,
                                 const AttnFwdArgs& a, cudaStream_t st) {
  switch (attn_dp(a.D)) {
    case 32: return fwd_t<32>(Q, K, V, p, a, st);
    case 64: return fwd_t<64>(Q, K, V, p, a, st);
    default: return fwd_t<128>(Q, K, V, p, a, st);
  }
}

cudaError_t launch_attn_bwd_simt(const AttnBwdPlan& p, const AttnBwdArgs& a, cudaStream_t st) {
  switch (attn_dp(a.D)) {
    case 32: return bwd_t<32>(p, a, st);
    case 64: return bwd_t<64>(p, a, st);
    default: return bwd_t<128>(p, a, st);
  }
}

}  // namespace flare

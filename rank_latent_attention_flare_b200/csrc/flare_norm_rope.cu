// Norm of every query and key head with the rotation by position, forward and
// backward, and its C entry points.
//
// Per row x (one token of one head, D elements), weights w, angles t_p of the
// token's position for the first R elements in pairs (a, b):
//   r = 1 / sqrt(mean(x^2) + eps),  u = w x r,
//   y_a = u_a cos - u_b sin,  y_b = u_b cos + u_a sin   (the others: y = u).
// Backward (the rotation is orthogonal, so its gradient is its inverse):
//   du = rotation^-1(dy),  g = w du,
//   dx = r (g - x r^2 mean(g x)),  dw = sum over rows of du x r.
//
// Both kernels are bound by memory: one pass, a row held in the registers of
// LPG lanes (16 bytes each, so D = 128 in bf16 takes 16 lanes), all sums in
// float32, one rounding at the end.  A pair's other half sits in another lane
// when pairs are (i, i + R / 2): it comes by a shuffle.  A group of lanes
// takes one token and up to kHeads heads, so that the token's angles and the
// weights are loaded once for them and four rows are in flight per lane.
#include "flare_attn.cuh"

namespace flare {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;   // rows in flight per group

struct NormRopeArgs {
  int Hq, Hk, N, D, R, interleaved;
  int qchunks, kchunks, heads;   // units per token, heads per unit
  int h_inner;                   // units of a token are neighbours (else tokens of a chunk)
  int64_t tokens, units;         // tokens = B N
  int64_t tab_sb;                // batch stride of cos / sin
  float eps;
  const float *cos, *sin;
  const void *q, *k, *wq, *wk, *dqo, *dko;
  void *qo, *ko, *dq, *dk, *dwq, *dwk;
  Tok tq, tk, tqo, tko, tdq, tdk;   // tqo, tko: of the outputs or their gradients
  float* part;                      // backward: [blocks][2][128] weight gradients
};

template <typename T>
struct Vec {
  static constexpr int V = 16 / sizeof(T);
  static __device__ __forceinline__ void unpack(const uint4& u, float (&f)[V]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (sizeof(T) == 4) {
        f[k] = __uint_as_float(w[k]);
      } else {
        f[2 * k] = __uint_as_float(w[k] << 16);
        f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[V]) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (sizeof(T) == 4) {
        w[k] = __float_as_uint(f[k]);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// What a unit of work is: token (b, n) and heads [h0, h0 + cnt) of q or k.
struct Unit {
  int64_t b;
  int n, h0, cnt;
  bool k;
};
__device__ __forceinline__ Unit unit_of(const NormRopeArgs& A, int64_t u) {
  const int chunks = A.qchunks + A.kchunks;
  int64_t tok;
  int c;
  if (A.h_inner) {
    tok = u / chunks;
    c = (int)(u % chunks);
  } else {   // neighbouring groups: neighbouring tokens of one chunk
    const int64_t per = (int64_t)chunks * A.N;
    const int64_t b = u / per;
    const int64_t x = u % per;
    c = (int)(x / A.N);
    tok = b * A.N + x % A.N;
  }
  Unit r;
  r.b = tok / A.N;
  r.n = (int)(tok % A.N);
  r.k = c >= A.qchunks;
  r.h0 = (r.k ? c - A.qchunks : c) * A.heads;
  r.cnt = min(A.heads, (r.k ? A.Hk : A.Hq) - r.h0);
  return r;
}

// The angles of a lane's elements, and how it finds its pairs' other halves.
template <int V>
struct Angles {
  float c[V], s[V];   // s carries the sign of the other half's term
  int src;            // lane that holds the other halves
  __device__ __forceinline__ void load(const NormRopeArgs& A, const Unit& u, int sub, int lane) {
    const int d = sub * V;
    src = lane;
#pragma unroll
    for (int e = 0; e < V; ++e) c[e] = 1.f, s[e] = 0.f;
    if (d >= A.R) return;
    const int half = A.R / 2;
    const int64_t row = u.b * A.tab_sb + (int64_t)u.n * half;
    if (A.interleaved) {
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        const float cc = __ldg(A.cos + row + (d + e) / 2), ss = __ldg(A.sin + row + (d + e) / 2);
        c[e] = c[e + 1] = cc;
        s[e] = -ss;
        s[e + 1] = ss;
      }
    } else {
      const bool second = d >= half;
      const int64_t at = row + (second ? d - half : d);
      src = second ? lane - half / V : lane + half / V;
#pragma unroll
      for (int e = 0; e < V; e += 4) {
        const float4 cc = __ldg((const float4*)(A.cos + at + e));
        const float4 ss = __ldg((const float4*)(A.sin + at + e));
        c[e] = cc.x, c[e + 1] = cc.y, c[e + 2] = cc.z, c[e + 3] = cc.w;
        s[e] = ss.x, s[e + 1] = ss.y, s[e + 2] = ss.z, s[e + 3] = ss.w;
      }
      if (!second)
#pragma unroll
        for (int e = 0; e < V; ++e) s[e] = -s[e];
    }
  }
  // y = rotation(u), or its inverse (SIGN = -1).  Whole-warp call.
  template <int SIGN>
  __device__ __forceinline__ void rotate(const float (&u)[V], float (&y)[V], int interleaved) const {
    float o[V];
    if (interleaved) {
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = u[e ^ 1];
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = __shfl_sync(0xffffffffu, u[e], src);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) y[e] = fmaf(o[e], SIGN * s[e], u[e] * c[e]);
  }
};

template <int V, typename T>
__device__ __forceinline__ void load_w(const void* w, int sub, int D, float (&f)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] = 1.f;
  if (w != nullptr && sub * V < D)
    Vec<T>::unpack(__ldg((const uint4*)((const T*)w + sub * V)), f);
}

template <int LPG>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int k = LPG / 2; k; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
  return v;
}

template <typename T, int LPG>
__global__ void __launch_bounds__(kThreads)
    norm_rope_fwd_kernel(const __grid_constant__ NormRopeArgs A) {
  pdl_wait();
  pdl_trigger();
  constexpr int V = Vec<T>::V;
  const int lane = threadIdx.x & 31, sub = threadIdx.x % LPG;
  const int64_t id = (int64_t)blockIdx.x * (kThreads / LPG) + threadIdx.x / LPG;
  const bool on = id < A.units;            // every lane stays for the shuffles
  const Unit u = unit_of(A, on ? id : 0);
  const bool in = on && sub * V < A.D;
  Angles<V> ang;
  ang.load(A, u, sub, lane);
  float w[V];
  load_w<V, T>(u.k ? A.wk : A.wq, sub, A.D, w);
  const Tok ti = u.k ? A.tk : A.tq, to = u.k ? A.tko : A.tqo;
  const T* x = (const T*)(u.k ? A.k : A.q) + u.b * ti.sb + u.n * ti.sn + sub * V;
  T* y = (T*)(u.k ? A.ko : A.qo) + u.b * to.sb + u.n * to.sn + sub * V;
  const float inv = 1.f / A.D;
  for (int h = 0; h < A.heads; h += kUnroll) {
    uint4 raw[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      raw[j] = make_uint4(0, 0, 0, 0);
      if (in && h + j < u.cnt)
        raw[j] = *reinterpret_cast<const uint4*>(x + (u.h0 + h + j) * ti.sh);
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      float f[V], o[V], ss = 0.f;
      Vec<T>::unpack(raw[j], f);
#pragma unroll
      for (int e = 0; e < V; ++e) ss = fmaf(f[e], f[e], ss);
      const float r = rsqrtf(fmaf(group_sum<LPG>(ss), inv, A.eps));
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] *= w[e] * r;
      ang.template rotate<1>(f, o, A.interleaved);
      if (in && h + j < u.cnt)
        *reinterpret_cast<uint4*>(y + (u.h0 + h + j) * to.sh) = Vec<T>::pack(o);
    }
  }
}

// A fixed number of CTAs take the units in turn, so that the weight gradients
// stay in registers until the end; a CTA's groups are added in a fixed order.
template <typename T, int LPG>
__global__ void __launch_bounds__(kThreads)
    norm_rope_bwd_kernel(const __grid_constant__ NormRopeArgs A) {
  pdl_wait();
  pdl_trigger();
  constexpr int V = Vec<T>::V, GROUPS = kThreads / LPG;
  __shared__ float red[GROUPS][LPG * V + 4];
  const int lane = threadIdx.x & 31, sub = threadIdx.x % LPG, group = threadIdx.x / LPG;
  const float inv = 1.f / A.D;
  float dw[2][V] = {};
  for (int64_t base = (int64_t)blockIdx.x * GROUPS; base < A.units;
       base += (int64_t)gridDim.x * GROUPS) {
    const int64_t id = base + group;
    const bool on = id < A.units;
    const Unit u = unit_of(A, on ? id : 0);
    const bool in = on && sub * V < A.D;
    Angles<V> ang;
    ang.load(A, u, sub, lane);
    float w[V], acc[V] = {};
    load_w<V, T>(u.k ? A.wk : A.wq, sub, A.D, w);
    const Tok ti = u.k ? A.tk : A.tq, tg = u.k ? A.tko : A.tqo, to = u.k ? A.tdk : A.tdq;
    const T* x = (const T*)(u.k ? A.k : A.q) + u.b * ti.sb + u.n * ti.sn + sub * V;
    const T* g = (const T*)(u.k ? A.dko : A.dqo) + u.b * tg.sb + u.n * tg.sn + sub * V;
    T* dx = (T*)(u.k ? A.dk : A.dq) + u.b * to.sb + u.n * to.sn + sub * V;
    for (int h = 0; h < A.heads; h += kUnroll) {
      uint4 rx[kUnroll], rg[kUnroll];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        rx[j] = rg[j] = make_uint4(0, 0, 0, 0);
        if (in && h + j < u.cnt) {
          rx[j] = *reinterpret_cast<const uint4*>(x + (u.h0 + h + j) * ti.sh);
          rg[j] = *reinterpret_cast<const uint4*>(g + (u.h0 + h + j) * tg.sh);
        }
      }
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        float f[V], d[V], du[V], ss = 0.f, gx = 0.f;
        Vec<T>::unpack(rx[j], f);
        Vec<T>::unpack(rg[j], d);
        ang.template rotate<-1>(d, du, A.interleaved);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          d[e] = du[e] * w[e];
          ss = fmaf(f[e], f[e], ss);
          gx = fmaf(d[e], f[e], gx);
        }
        const float r = rsqrtf(fmaf(group_sum<LPG>(ss), inv, A.eps));
        const float m = group_sum<LPG>(gx) * inv * r * r;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          acc[e] = fmaf(du[e], f[e] * r, acc[e]);
          d[e] = r * fmaf(-f[e], m, d[e]);
        }
        if (in && h + j < u.cnt)
          *reinterpret_cast<uint4*>(dx + (u.h0 + h + j) * to.sh) = Vec<T>::pack(d);
      }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      dw[0][e] += u.k ? 0.f : acc[e];
      dw[1][e] += u.k ? acc[e] : 0.f;
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if ((k ? A.dwk : A.dwq) == nullptr) continue;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < V; ++e) red[group][sub * V + e] = dw[k][e];
    __syncthreads();
    if (threadIdx.x < A.D) {
      float s = 0.f;
      for (int gq = 0; gq < GROUPS; ++gq) s += red[gq][threadIdx.x];
      A.part[((int64_t)blockIdx.x * 2 + k) * 128 + threadIdx.x] = s;
    }
  }
}

// The CTAs' weight gradients, added in a fixed order: 32 columns per CTA, a
// warp per eighth of the records.
template <typename T>
__global__ void __launch_bounds__(256) norm_rope_dw_kernel(const float* part, int n, int D, T* dwq,
                                                           T* dwk) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int k = blockIdx.x / 4, col = (blockIdx.x % 4) * 32 + lane;
  T* out = k ? dwk : dwq;
  if (out == nullptr) return;
  float s = 0.f;
  if (col < D)
    for (int i = warp; i < n; i += 8) s += part[((int64_t)i * 2 + k) * 128 + col];
  red[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || col >= D) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += red[i][lane];
  if constexpr (sizeof(T) == 4) out[col] = s;
  else out[col] = __float2bfloat16_rn(s);
}

int lanes_per_row(int64_t D, flare_dtype_t dt) {
  const int64_t v = dt == FLARE_F32 ? 4 : 8, lanes = (D + v - 1) / v;
  return lanes <= 4 ? 4 : lanes <= 8 ? 8 : lanes <= 16 ? 16 : 32;
}

// CTAs of the backward: a multiple of the SMs, never more than the units.
int64_t bwd_blocks(int64_t units, int lpg) {
  const int64_t need = (units * lpg + kThreads - 1) / kThreads;
  return imin64(need, 4LL * sm_count());
}

constexpr int64_t kPartBytes = 2 * 128 * 4;

void cut(NormRopeArgs& a, int64_t B) {
  a.heads = kUnroll;
  a.qchunks = (a.Hq + a.heads - 1) / a.heads;
  a.kchunks = (a.Hk + a.heads - 1) / a.heads;
  a.tokens = B * a.N;
  a.units = a.tokens * (a.qchunks + a.kchunks);
  a.h_inner = a.tq.sh < a.tq.sn;
}

#define FLARE_LPG(kern, T, lpg, ...)                 \
  switch (lpg) {                                     \
    case 4: FLARE_CUDA(kern(T, 4, __VA_ARGS__)); break;   \
    case 8: FLARE_CUDA(kern(T, 8, __VA_ARGS__)); break;   \
    case 16: FLARE_CUDA(kern(T, 16, __VA_ARGS__)); break; \
    default: FLARE_CUDA(kern(T, 32, __VA_ARGS__));        \
  }
#define FLARE_FWD_KERNEL(T, L, a, grid, st) \
  launch_pdl(norm_rope_fwd_kernel<T, L>, grid, kThreads, 0, st, a)
#define FLARE_BWD_KERNEL(T, L, a, grid, st) \
  launch_pdl(norm_rope_bwd_kernel<T, L>, grid, kThreads, 0, st, a)

flare_status_t check(int64_t B, int64_t Hq, int64_t Hk, int64_t N, int64_t D, int64_t R,
                     flare_dtype_t dt, const void* cos, const void* sin, int64_t tab_sb,
                     float eps) {
  if (B < 1 || Hq < 1 || Hk < 1 || N < 1 || D < 1 || R < 0 || R > D) return FLARE_ERR_INVALID_ARG;
  if (dt != FLARE_F32 && dt != FLARE_BF16) return FLARE_ERR_INVALID_ARG;
  if (B > (1LL << 20) || Hq > (1LL << 16) || Hk > (1LL << 16)) return FLARE_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || !(eps > 0.f)) return FLARE_ERR_INVALID_ARG;
  if (D % 8 != 0 || D > 128 || R % 16 != 0) return FLARE_ERR_UNSUPPORTED;
  if (N > (1LL << 30)) return FLARE_ERR_UNSUPPORTED;
  if ((double)B * (Hq + Hk) * N * D >= 1099511627776.0) return FLARE_ERR_INVALID_ARG;   // 2^40
  // one group of lanes per unit, 31 bits of CTAs
  if ((double)B * N * (Hq + Hk) >= 8.0 * 2147483647.0) return FLARE_ERR_UNSUPPORTED;
  if (R > 0) {
    FLARE_TRY(check_ptr(cos));
    FLARE_TRY(check_ptr(sin));
    if (tab_sb != 0 && tab_sb < N * (R / 2)) return FLARE_ERR_INVALID_ARG;
    if (tab_sb % 4 != 0) return FLARE_ERR_UNSUPPORTED;
  }
  return FLARE_OK;
}

flare_status_t optional(const void* p) { return p ? check_ptr(p) : FLARE_OK; }

}  // namespace
}  // namespace flare

using namespace flare;

extern "C" {

flare_status_t flare_qk_norm_rope_fwd(const void* q, const void* k, const void* wq, const void* wk,
                                      const float* cos, const float* sin, int64_t tab_batch_stride,
                                      void* qo, void* ko, const flare_strides_t* strides, int64_t B,
                                      int64_t Hq, int64_t Hk, int64_t N, int64_t D, int64_t R,
                                      int interleaved, flare_dtype_t dt, float eps, void* stream) {
  FLARE_TRY(check(B, Hq, Hk, N, D, R, dt, cos, sin, tab_batch_stride, eps));
  const void* must[4] = {q, k, qo, ko};
  for (const void* p : must) FLARE_TRY(check_ptr(p));
  FLARE_TRY(optional(wq));
  FLARE_TRY(optional(wk));
  NormRopeArgs a = {};
  Tok* where[4] = {&a.tq, &a.tk, &a.tqo, &a.tko};
  for (int i = 0; i < 4; ++i)
    FLARE_TRY(check_tok(strides ? strides + i : nullptr, B, i % 2 ? Hk : Hq, N, D, dt, i >= 2,
                        where[i]));
  a.Hq = (int)Hq, a.Hk = (int)Hk, a.N = (int)N, a.D = (int)D, a.R = (int)R;
  a.interleaved = interleaved != 0;
  a.tab_sb = tab_batch_stride;
  a.eps = eps;
  a.cos = cos, a.sin = sin;
  a.q = q, a.k = k, a.wq = wq, a.wk = wk, a.qo = qo, a.ko = ko;
  cut(a, B);
  note_error("%s", "");
  const int lpg = lanes_per_row(D, dt);
  const int64_t per = kThreads / lpg;
  const dim3 grid((unsigned)((a.units + per - 1) / per));
  cudaStream_t st = (cudaStream_t)stream;
  if (dt == FLARE_BF16) {
    FLARE_LPG(FLARE_FWD_KERNEL, __nv_bfloat16, lpg, a, grid, st);
  } else {
    FLARE_LPG(FLARE_FWD_KERNEL, float, lpg, a, grid, st);
  }
  FLARE_CUDA(cudaPeekAtLastError());
  return FLARE_OK;
}

size_t flare_qk_norm_rope_workspace_size(int64_t B, int64_t Hq, int64_t Hk, int64_t N, int64_t D,
                                         flare_dtype_t dt) {
  alignas(16) static const float none[4] = {};
  if (check(B, Hq, Hk, N, D, 0, dt, none, none, 0, 1.f) != FLARE_OK) return 0;
  NormRopeArgs a = {};
  a.Hq = (int)Hq, a.Hk = (int)Hk, a.N = (int)N;
  cut(a, B);
  return (size_t)(bwd_blocks(a.units, lanes_per_row(D, dt)) * kPartBytes);
}

flare_status_t flare_qk_norm_rope_bwd(const void* q, const void* k, const void* wq, const void* wk,
                                      const float* cos, const float* sin, int64_t tab_batch_stride,
                                      const void* dqo, const void* dko, void* dq, void* dk,
                                      void* dwq, void* dwk, const flare_strides_t* strides,
                                      int64_t B, int64_t Hq, int64_t Hk, int64_t N, int64_t D,
                                      int64_t R, int interleaved, flare_dtype_t dt, float eps,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  FLARE_TRY(check(B, Hq, Hk, N, D, R, dt, cos, sin, tab_batch_stride, eps));
  const void* must[6] = {q, k, dqo, dko, dq, dk};
  for (const void* p : must) FLARE_TRY(check_ptr(p));
  const void* opt[4] = {wq, wk, dwq, dwk};
  for (const void* p : opt) FLARE_TRY(optional(p));
  NormRopeArgs a = {};
  Tok* where[6] = {&a.tq, &a.tk, &a.tqo, &a.tko, &a.tdq, &a.tdk};
  for (int i = 0; i < 6; ++i)
    FLARE_TRY(check_tok(strides ? strides + i : nullptr, B, i % 2 ? Hk : Hq, N, D, dt, i >= 4,
                        where[i]));
  FLARE_TRY(check_workspace(workspace, workspace_bytes,
                            flare_qk_norm_rope_workspace_size(B, Hq, Hk, N, D, dt)));
  a.Hq = (int)Hq, a.Hk = (int)Hk, a.N = (int)N, a.D = (int)D, a.R = (int)R;
  a.interleaved = interleaved != 0;
  a.tab_sb = tab_batch_stride;
  a.eps = eps;
  a.cos = cos, a.sin = sin;
  a.q = q, a.k = k, a.wq = wq, a.wk = wk, a.dqo = dqo, a.dko = dko, a.dq = dq, a.dk = dk;
  a.dwq = dwq, a.dwk = dwk;
  a.part = (float*)workspace;
  cut(a, B);
  note_error("%s", "");
  const int lpg = lanes_per_row(D, dt);
  const int64_t blocks = bwd_blocks(a.units, lpg);
  const dim3 grid((unsigned)blocks);
  cudaStream_t st = (cudaStream_t)stream;
  if (dt == FLARE_BF16) {
    FLARE_LPG(FLARE_BWD_KERNEL, __nv_bfloat16, lpg, a, grid, st);
  } else {
    FLARE_LPG(FLARE_BWD_KERNEL, float, lpg, a, grid, st);
  }
  if (dwq || dwk) {
    if (dt == FLARE_BF16)
      FLARE_CUDA(launch_pdl(norm_rope_dw_kernel<__nv_bfloat16>, dim3(8), dim3(256), 0, st,
                            (const float*)a.part, (int)blocks, (int)D, (__nv_bfloat16*)dwq,
                            (__nv_bfloat16*)dwk));
    else
      FLARE_CUDA(launch_pdl(norm_rope_dw_kernel<float>, dim3(8), dim3(256), 0, st,
                            (const float*)a.part, (int)blocks, (int)D, (float*)dwq, (float*)dwk));
  }
  FLARE_CUDA(cudaPeekAtLastError());
  return FLARE_OK;
}

}  // extern "C"

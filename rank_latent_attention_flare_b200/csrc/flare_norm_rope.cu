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
// when pairs are (i, i + R / 2): its raw 16 bytes come by a shuffle, and the
// weights are folded into the angles, y = r (x (w cos) + x' (w' sin)), so that
// a row costs about six instructions for every element pair (packed float32
// arithmetic); with more of them the kernel is bound by issue slots.  A group
// of lanes takes one token and up to 8 heads of it, so that the coefficients
// are built once for them.
#include "flare_attn.cuh"
#include "tc_primitives.cuh"

namespace flare {
namespace {

using tc::add_f32x2;
using tc::f32x2;
using tc::fma_f32x2;
using tc::mul_f32x2;
using tc::split_f32x2;

constexpr int kThreads = 256;
constexpr int kBwdPerSm = 3;   // resident CTAs of the backward

struct NormRopeArgs {
  int Hq, Hk, N, D, R, interleaved;
  int qchunks, kchunks, heads;   // units per token, heads per unit
  int h_inner;                   // units of a token are neighbours (else tokens of a chunk)
  int qblocks, kblocks;          // backward: CTAs for q and for k
  int64_t tokens, units;         // tokens = B N
  int64_t tab_sb;                // batch stride of cos / sin
  float eps;
  const float *cos, *sin;
  const void *q, *k, *wq, *wk, *dqo, *dko;
  void *qo, *ko, *dq, *dk, *dwq, *dwk;
  Tok tq, tk, tqo, tko, tdq, tdk;   // tqo, tko: of the outputs or their gradients
  float* part;                      // backward: [block][128] weight gradients
};

// The 16 bytes of a lane as pairs of float32.
template <typename T>
struct Vec {
  static constexpr int V = 16 / sizeof(T), P = V / 2;
  static __device__ __forceinline__ void unpack(const uint4& u, uint64_t (&f)[P]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < P; ++k) {
      if constexpr (sizeof(T) == 4)
        f[k] = f32x2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
      else
        f[k] = f32x2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
    }
  }
  static __device__ __forceinline__ uint4 pack(const uint64_t (&f)[P]) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < P; ++k) {
      float a, b;
      split_f32x2(f[k], a, b);
      if constexpr (sizeof(T) == 4) {
        w[2 * k] = __float_as_uint(a);
        w[2 * k + 1] = __float_as_uint(b);
      } else {
        w[k] = tc::pack_bf16(a, b);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // the elements at column d of a [D] vector (ones without one)
  static __device__ __forceinline__ void weights(const void* w, int d, int D, uint64_t (&f)[P]) {
#pragma unroll
    for (int k = 0; k < P; ++k) f[k] = f32x2(1.f, 1.f);
    if (w != nullptr && d < D) unpack(__ldg((const uint4*)((const T*)w + d)), f);
  }
};

__device__ __forceinline__ uint64_t swap_f32x2(uint64_t v) {
  float a, b;
  split_f32x2(v, a, b);
  return f32x2(b, a);
}
__device__ __forceinline__ float sum_f32x2(uint64_t v) {
  float a, b;
  split_f32x2(v, a, b);
  return a + b;
}

// unit u of `chunks` chunks per token (32-bit divisions where they reach)
__device__ __forceinline__ void unit_of(const NormRopeArgs& A, int64_t u, int chunks, int64_t& b,
                                        int& n, int& c) {
  if (A.units <= 0x7fffffffLL) {
    const unsigned v = (unsigned)u, N = (unsigned)A.N, C = (unsigned)chunks;
    if (A.h_inner) {
      c = (int)(v % C);
      b = (int64_t)(v / C / N);
      n = (int)(v / C % N);
    } else {   // neighbouring groups: neighbouring tokens of one chunk
      n = (int)(v % N);
      c = (int)(v / N % C);
      b = (int64_t)(v / N / C);
    }
  } else if (A.h_inner) {
    c = (int)(u % chunks);
    b = u / chunks / A.N;
    n = (int)(u / chunks % A.N);
  } else {
    n = (int)(u % A.N);
    c = (int)(u / A.N % chunks);
    b = u / A.N / chunks;
  }
}

// A lane's cosines, and sines with the sign of the other half's term in the
// rotation; where the other half is.
template <typename T>
struct Angles {
  static constexpr int P = Vec<T>::P;
  uint64_t c[P], s[P];
  int other;   // column of the other half (split pairs)
  __device__ __forceinline__ void load(const NormRopeArgs& A, int64_t b, int n, int d) {
    other = d;
#pragma unroll
    for (int k = 0; k < P; ++k) c[k] = f32x2(1.f, 1.f), s[k] = 0;
    if (d >= A.R) return;
    const int half = A.R / 2;
    const int64_t row = b * A.tab_sb + (int64_t)n * half;
    if (A.interleaved) {
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const float cc = __ldg(A.cos + row + d / 2 + k), ss = __ldg(A.sin + row + d / 2 + k);
        c[k] = f32x2(cc, cc);
        s[k] = f32x2(-ss, ss);
      }
      return;
    }
    const bool second = d >= half;
    other = second ? d - half : d + half;
    const float* pc = A.cos + row + (second ? d - half : d);
    const float* ps = A.sin + row + (second ? d - half : d);
    const float sign = second ? 1.f : -1.f;
#pragma unroll
    for (int k = 0; k < P; k += 2) {
      const float4 cc = __ldg((const float4*)(pc + 2 * k)), ss = __ldg((const float4*)(ps + 2 * k));
      c[k] = f32x2(cc.x, cc.y), c[k + 1] = f32x2(cc.z, cc.w);
      s[k] = f32x2(sign * ss.x, sign * ss.y), s[k + 1] = f32x2(sign * ss.z, sign * ss.w);
    }
  }
};

// The other halves of a lane's elements.  Whole-warp call.
template <typename T>
__device__ __forceinline__ void others(const uint4& raw, const uint64_t (&x)[Vec<T>::P],
                                       bool interleaved, int src, uint64_t (&o)[Vec<T>::P]) {
  if (interleaved) {
#pragma unroll
    for (int k = 0; k < Vec<T>::P; ++k) o[k] = swap_f32x2(x[k]);
  } else {
    uint4 t;
    t.x = __shfl_sync(0xffffffffu, raw.x, src);
    t.y = __shfl_sync(0xffffffffu, raw.y, src);
    t.z = __shfl_sync(0xffffffffu, raw.z, src);
    t.w = __shfl_sync(0xffffffffu, raw.w, src);
    Vec<T>::unpack(t, o);
  }
}

template <int LPG>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int k = LPG / 2; k; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
  return v;
}

template <typename T, int LPG>
__global__ void __launch_bounds__(kThreads, 3)
    norm_rope_fwd_kernel(const __grid_constant__ NormRopeArgs A) {
  pdl_wait();
  pdl_trigger();
  constexpr int V = Vec<T>::V, P = Vec<T>::P, U = 4;   // U rows in flight per lane
  const int lane = threadIdx.x & 31, sub = threadIdx.x % LPG, d = sub * V;
  const int64_t id = (int64_t)blockIdx.x * (kThreads / LPG) + threadIdx.x / LPG;
  const bool on = id < A.units;            // every lane stays for the shuffles
  int64_t b;
  int n, ch;
  unit_of(A, on ? id : 0, A.qchunks + A.kchunks, b, n, ch);
  const bool isk = ch >= A.qchunks;
  const int h0 = (isk ? ch - A.qchunks : ch) * A.heads;
  const int cnt = on && d < A.D ? min(A.heads, (isk ? A.Hk : A.Hq) - h0) : 0;
  const Tok ti = isk ? A.tk : A.tq, to = isk ? A.tko : A.tqo;
  const T* x = (const T*)(isk ? A.k : A.q) + b * ti.sb + n * ti.sn + h0 * ti.sh + d;
  T* y = (T*)(isk ? A.ko : A.qo) + b * to.sb + n * to.sn + h0 * to.sh + d;
  const void* w = isk ? A.wk : A.wq;
  uint4 raw[U];
  auto load = [&](int h) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      raw[j] = make_uint4(0, 0, 0, 0);
      if (h + j < cnt) raw[j] = *reinterpret_cast<const uint4*>(x + (h + j) * ti.sh);
    }
  };
  load(0);   // in flight while the coefficients are built
  // y = r (x ca + x' cb)
  uint64_t ca[P], cb[P];
  int src;
  {
    Angles<T> ang;
    ang.load(A, b, n, d);
    src = lane + (ang.other - d) / V;
    uint64_t wx[P], wo[P];
    Vec<T>::weights(w, d, A.D, wx);
    Vec<T>::weights(w, ang.other, A.D, wo);
#pragma unroll
    for (int k = 0; k < P; ++k) {
      ca[k] = mul_f32x2(ang.c[k], wx[k]);
      cb[k] = mul_f32x2(ang.s[k], A.interleaved ? swap_f32x2(wx[k]) : wo[k]);
    }
  }
  const float inv = 1.f / A.D;
  for (int h = 0; h < A.heads; h += U) {
    if (h > 0) load(h);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      uint64_t f[P], o[P], ss = 0;
      Vec<T>::unpack(raw[j], f);
#pragma unroll
      for (int k = 0; k < P; ++k) ss = fma_f32x2(f[k], f[k], ss);
      const float r = rsqrtf(fmaf(group_sum<LPG>(sum_f32x2(ss)), inv, A.eps));
      others<T>(raw[j], f, A.interleaved, src, o);
#pragma unroll
      for (int k = 0; k < P; ++k)
        f[k] = mul_f32x2(fma_f32x2(o[k], cb[k], mul_f32x2(f[k], ca[k])), f32x2(r, r));
      if (h + j < cnt) *reinterpret_cast<uint4*>(y + (h + j) * to.sh) = Vec<T>::pack(f);
    }
  }
}

// The CTAs that reside at once take the units in turn, those of q and those
// of k apart, so that the weight gradient stays in registers until the end; a
// CTA's groups are added in a fixed order.
template <typename T, int LPG>
__global__ void __launch_bounds__(kThreads, kBwdPerSm)
    norm_rope_bwd_kernel(const __grid_constant__ NormRopeArgs A) {
  pdl_wait();
  pdl_trigger();
  constexpr int V = Vec<T>::V, P = Vec<T>::P, U = 2, GROUPS = kThreads / LPG;
  __shared__ float red[GROUPS][LPG * V + 4];
  const int lane = threadIdx.x & 31, sub = threadIdx.x % LPG, group = threadIdx.x / LPG;
  const int d = sub * V;
  const bool isk = (int)blockIdx.x >= A.qblocks;
  const int block = (int)blockIdx.x - (isk ? A.qblocks : 0), blocks = isk ? A.kblocks : A.qblocks;
  const int chunks = isk ? A.kchunks : A.qchunks, H = isk ? A.Hk : A.Hq;
  const int64_t units = A.tokens * chunks;
  const Tok ti = isk ? A.tk : A.tq, tg = isk ? A.tko : A.tqo, to = isk ? A.tdk : A.tdq;
  uint64_t w[P], acc[P];
  Vec<T>::weights(isk ? A.wk : A.wq, d, A.D, w);
#pragma unroll
  for (int k = 0; k < P; ++k) acc[k] = 0;
  const float inv = 1.f / A.D;
  for (int64_t base = (int64_t)block * GROUPS; base < units; base += (int64_t)blocks * GROUPS) {
    const int64_t id = base + group;
    const bool on = id < units;
    int64_t b;
    int n, ch;
    unit_of(A, on ? id : 0, chunks, b, n, ch);
    const int h0 = ch * A.heads;
    const int cnt = on && d < A.D ? min(A.heads, H - h0) : 0;
    const T* x = (const T*)(isk ? A.k : A.q) + b * ti.sb + n * ti.sn + h0 * ti.sh + d;
    const T* g = (const T*)(isk ? A.dko : A.dqo) + b * tg.sb + n * tg.sn + h0 * tg.sh + d;
    T* dx = (T*)(isk ? A.dk : A.dq) + b * to.sb + n * to.sn + h0 * to.sh + d;
    Angles<T> ang;
    ang.load(A, b, n, d);
    const int src = lane + (ang.other - d) / V;
    for (int h = 0; h < A.heads; h += U) {
      uint4 rx[U], rg[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        rx[j] = rg[j] = make_uint4(0, 0, 0, 0);
        if (h + j < cnt) {
          rx[j] = *reinterpret_cast<const uint4*>(x + (h + j) * ti.sh);
          rg[j] = *reinterpret_cast<const uint4*>(g + (h + j) * tg.sh);
        }
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        uint64_t f[P], e[P], o[P], ss = 0, gx = 0;
        Vec<T>::unpack(rx[j], f);
        Vec<T>::unpack(rg[j], e);
        others<T>(rg[j], e, A.interleaved, src, o);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          // du: the inverse rotation has the other sign of the sine
          o[k] = fma_f32x2(o[k], ang.s[k] ^ 0x8000000080000000ull, mul_f32x2(e[k], ang.c[k]));
          e[k] = mul_f32x2(o[k], w[k]);
          ss = fma_f32x2(f[k], f[k], ss);
          gx = fma_f32x2(e[k], f[k], gx);
        }
        const float r = rsqrtf(fmaf(group_sum<LPG>(sum_f32x2(ss)), inv, A.eps));
        const float m = -group_sum<LPG>(sum_f32x2(gx)) * inv * r * r * r;
        const uint64_t r2 = f32x2(r, r), m2 = f32x2(m, m);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          acc[k] = fma_f32x2(o[k], mul_f32x2(f[k], r2), acc[k]);
          e[k] = fma_f32x2(f[k], m2, mul_f32x2(e[k], r2));
        }
        if (h + j < cnt) *reinterpret_cast<uint4*>(dx + (h + j) * to.sh) = Vec<T>::pack(e);
      }
    }
  }
  if ((isk ? A.dwk : A.dwq) == nullptr) return;
#pragma unroll
  for (int k = 0; k < P; ++k) {
    float a, c;
    split_f32x2(acc[k], a, c);
    red[group][d + 2 * k] = a;
    red[group][d + 2 * k + 1] = c;
  }
  __syncthreads();
  if (threadIdx.x < A.D) {
    float s = 0.f;
    for (int q = 0; q < GROUPS; ++q) s += red[q][threadIdx.x];
    A.part[(int64_t)blockIdx.x * 128 + threadIdx.x] = s;
  }
}

// The CTAs' weight gradients, added in a fixed order: 32 columns per CTA, a
// warp per eighth of the records.
template <typename T>
__global__ void __launch_bounds__(256) norm_rope_dw_kernel(const float* part, int nq, int nk, int D,
                                                           T* dwq, T* dwk) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int k = blockIdx.x / 4, col = (blockIdx.x % 4) * 32 + lane;
  T* out = k ? dwk : dwq;
  if (out == nullptr) return;
  const int lo = k ? nq : 0, hi = k ? nq + nk : nq;
  float s = 0.f;
  if (col < D) {
#pragma unroll 8
    for (int i = lo + warp; i < hi; i += 8) s += part[(int64_t)i * 128 + col];
  }
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

// Heads per unit: 8, or fewer where that leaves SMs without a CTA (a single
// token of 32 requests: 1).
void cut(NormRopeArgs& a, int64_t B, int lpg) {
  const int64_t per = kThreads / lpg, want = sm_count() * per;
  a.tokens = B * a.N;
  for (a.heads = 8;; a.heads /= 2) {
    a.qchunks = (a.Hq + a.heads - 1) / a.heads;
    a.kchunks = (a.Hk + a.heads - 1) / a.heads;
    a.units = a.tokens * (a.qchunks + a.kchunks);
    if (a.units >= want || a.heads == 1) break;
  }
  a.h_inner = a.tq.sh < a.tq.sn;
  // backward: the resident CTAs, shared by q and k as their units are
  const int64_t most = (int64_t)kBwdPerSm * sm_count();
  const int64_t q = (a.tokens * a.qchunks + per - 1) / per;
  const int64_t k = (a.tokens * a.kchunks + per - 1) / per;
  if (q + k <= most) {
    a.qblocks = (int)q;
    a.kblocks = (int)k;
  } else {
    const int64_t kb = most * a.kchunks / (a.qchunks + a.kchunks);
    a.kblocks = (int)imax64(1, imin64(kb, most - 1));
    a.qblocks = (int)most - a.kblocks;
  }
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
  const int lpg = lanes_per_row(D, dt);
  cut(a, B, lpg);
  note_error("%s", "");
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
  cut(a, B, lanes_per_row(D, dt));
  return (size_t)(a.qblocks + a.kblocks) * 128 * sizeof(float);
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
  const int lpg = lanes_per_row(D, dt);
  cut(a, B, lpg);
  note_error("%s", "");
  const dim3 grid((unsigned)(a.qblocks + a.kblocks));
  cudaStream_t st = (cudaStream_t)stream;
  if (dt == FLARE_BF16) {
    FLARE_LPG(FLARE_BWD_KERNEL, __nv_bfloat16, lpg, a, grid, st);
  } else {
    FLARE_LPG(FLARE_BWD_KERNEL, float, lpg, a, grid, st);
  }
  if (dwq || dwk) {
    if (dt == FLARE_BF16)
      FLARE_CUDA(launch_pdl(norm_rope_dw_kernel<__nv_bfloat16>, dim3(8), dim3(256), 0, st,
                            (const float*)a.part, a.qblocks, a.kblocks, (int)D, (__nv_bfloat16*)dwq,
                            (__nv_bfloat16*)dwk));
    else
      FLARE_CUDA(launch_pdl(norm_rope_dw_kernel<float>, dim3(8), dim3(256), 0, st,
                            (const float*)a.part, a.qblocks, a.kblocks, (int)D, (float*)dwq,
                            (float*)dwk));
  }
  FLARE_CUDA(cudaPeekAtLastError());
  return FLARE_OK;
}

}  // extern "C"

// Softmax attention Y = softmax(s Q K^T) V with its gradient: the sizes of a
// call, how it is cut into CTAs, its workspace, and the kernel launchers.
//
// Queries [B,Hq,Nq,D], keys and values [B,Hk,Nk,D], Hq = G Hk: the G query
// heads of a key head share its keys and values.  With per-batch lengths ql
// and kl only the first ql queries and kl keys count.  causal: query i sees
// keys j <= i + (kl - ql) (the last query sees the last key).  A query that
// sees no key has Y = 0, lse = -inf and gives and gets no gradient.
#pragma once

#include "flare_internal.cuh"

namespace flare {

struct AttnDims {
  int64_t B = 0, Hq = 0, Hk = 0, Nq = 0, Nk = 0, D = 0;
  bool causal = false;
  Tok q, k, v, y, dy, dq, dk, dv;   // inputs may have zero batch / head strides (broadcast)
  int64_t G() const { return Hq / Hk; }
};

// Per-batch view of the lengths and the mask, in the kernels' 32-bit indices.
struct AttnSeq {
  int ql, kl, off;   // valid queries, valid keys; causal: key j <= query i + off
  bool causal;
  __device__ __forceinline__ AttnSeq(int Nq, int Nk)
      : ql(Nq), kl(Nk), off(Nk - Nq), causal(false) {}
  __device__ __forceinline__ AttnSeq(const int32_t* q_lens, const int32_t* k_lens, int b, int Nq,
                                     int Nk, bool causal_)
      : ql(Nq), kl(Nk), causal(causal_) {
    if (q_lens) ql = min(max(q_lens[b], 0), Nq);
    if (k_lens) kl = min(max(k_lens[b], 0), Nk);
    off = kl - ql;
  }
  // tiles of T keys that some query up to i sees
  __device__ __forceinline__ int key_tiles(int i, int T) const {
    const int all = (kl + T - 1) / T;
    if (!causal) return all;
    const int last = min(i, ql - 1) + off;   // the last key seen (>= kl only past the end)
    return last < 0 ? 0 : min(all, last / T + 1);
  }
  // first tile of T queries of which some query sees key j
  __device__ __forceinline__ int first_query_tile(int j, int T) const {
    return causal ? max(0, j - off) / T : 0;
  }
};

// Part `split` of `splits` near-equal parts of n tiles: [lo, lo + count).
// (32-bit divisions here and in the kernels' indices: a 64-bit one costs as
// much as a hundred instructions.)
struct Part {
  int lo, count;
  __device__ __forceinline__ Part(int n, int split, int splits) : lo(0), count(n) {
    if (splits == 1) return;
    const int q = (int)((unsigned)n / (unsigned)splits), rem = n - q * splits;
    lo = q * split + min(split, rem);
    count = q + (split < rem);
  }
};

// Rows of tile t of T out of n valid rows: tile t covers [t T, t T + T), but
// the last one is moved back to end at row n, so that rows past n are never
// read (rows before 0 read as zeros); its first `lo` rows belong to the tile
// before.
__device__ __forceinline__ int tile_row0(int t, int T, int n) { return min(t * T, n - T); }

constexpr int kAttnTile = 128;   // query and key rows per tensor-core tile

// Head dimension of the kernels: D is padded with the TMA's zero fill.
__host__ __device__ constexpr int attn_dp(int64_t D) { return D <= 32 ? 32 : D <= 64 ? 64 : 128; }

// 16-element steps of the tensor cores' products over D, a compile-time
// constant of their kernels: the next of 2, 4, 5, 6, 8 (D = 80 and 96 are
// common; the zero fill makes a larger step count exact for the rest).
inline int attn_ks(int64_t D) { return D <= 32 ? 2 : D <= 64 ? 4 : D <= 80 ? 5 : D <= 96 ? 6 : 8; }

inline bool attn_tc(flare_dtype_t dt) { return dt == FLARE_BF16; }

// How the forward is cut.  A CTA takes `qt` tiles of query rows (tensor
// cores: one or two of 128 rows; CUDA cores: one of 64) of one head, or, when
// few queries leave a tile mostly empty, the queries of `hpt` heads that
// share a key head (row = head * Nq + query), and one of `splits` near-equal
// parts of the key tiles it sees.
struct AttnPlan {
  int qt = 1, hpt = 1, rows = 0, splits = 1;
  int64_t qblocks = 0, units = 0;   // units = CTAs without the split
};

struct AttnBwdPlan {
  int tile = 0;
  int64_t ktiles = 0, dkv_units = 0, qtiles = 0, dq_units = 0;
  int dkv_splits = 1, dq_splits = 1;
  bool stay = false;   // tensor cores: dK's and dV's CTAs take several pieces
};

AttnPlan attn_plan(const AttnDims& d, flare_dtype_t dt, int sms);
AttnBwdPlan attn_bwd_plan(const AttnDims& d, flare_dtype_t dt, int sms);

// Workspace offsets (bytes).  Header: the device error word.
struct AttnWs {
  size_t part_ml = 0, part_o = 0;              // forward: records of the splits
  size_t stats = 0;                            // backward: -lse (log2 units) and delta per query
  size_t dq_part = 0, dkv_part = 0;            // backward: partial sums of the splits
  size_t total = 0;
};
AttnWs attn_ws_fwd(const AttnDims& d, const AttnPlan& p);
AttnWs attn_ws_bwd(const AttnDims& d, const AttnBwdPlan& p);

// Zeroes the error word and reports lengths outside their range.  Called by
// thread 0..31 of the first CTA of the first kernel of a call: a bounded wait
// that runs out records its error a second later at the earliest.
__device__ __forceinline__ void attn_check_lens(const int32_t* q_lens, const int32_t* k_lens, int B,
                                                int Nq, int Nk, uint32_t* err) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  for (int b = lane; b < B; b += 32) {
    if (q_lens) bad |= q_lens[b] < 0 || q_lens[b] > Nq;
    if (k_lens) bad |= k_lens[b] < 0 || k_lens[b] > Nk;
  }
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) *err = bad ? (uint32_t)kErrSeqLen : 0u;
}

// Kernel arguments shared by the forward kernels.
struct AttnFwdArgs {
  int B, Hq, Hk, G, Nq, Nk, D;   // G = Hq / Hk
  int hpt, qblocks, splits, causal;
  float c;                 // scale * log2(e)
  const int32_t *q_lens, *k_lens;
  Tok q, k, v, y;
  void *Y, *Ylow;          // Ylow: what rounding Y left over, may be NULL
  float* lse;              // may be NULL
  float2* part_ml;         // [units * splits][rows] (reference, sum), log2 units
  float* part_o;           // [units * splits][rows][DP]
  uint32_t* err;
  // bits 0..5: q, k, v have one batch (1, 2, 4) or head (8, 16, 32) in memory
  int bcast;
};

struct AttnBwdArgs {
  int B, Hq, Hk, G, Nq, Nk, D;   // G = Hq / Hk
  int tile, ktiles, qtiles, dkv_splits, dq_splits, causal;
  int64_t dkv_units, dq_units;
  int dkv_ctas;            // tensor-core kernel: the first CTAs are dK's and dV's
  float scale, c;
  const int32_t *q_lens, *k_lens;
  Tok q, k, v, y, dy, dq, dk, dv;
  const void *Q, *K, *V, *Y, *Ylow, *dY;   // Ylow may be NULL
  const float* lse;
  void *dQ, *dK, *dV;
  float *nl, *delta;       // [B*Hq][Nq]: -lse in log2 units (-inf: no weight), sum(dY * Y)
  float *dq_part, *dkv_part;
  uint32_t* err;
  int bcast;               // as AttnFwdArgs, with dy: bits 6 (batch) and 7 (head)
};

cudaError_t launch_attn_fwd_tc(const void* Q, const void* K, const void* V, const AttnDims& d,
                               const AttnPlan& p, const AttnFwdArgs& a, cudaStream_t st);
cudaError_t launch_attn_fwd_simt(const void* Q, const void* K, const void* V, const AttnPlan& p,
                                 const AttnFwdArgs& a, cudaStream_t st);
// Joins the records of the splits into Y and lse.
cudaError_t launch_attn_join(const AttnPlan& p, const AttnFwdArgs& a, int dp, flare_dtype_t dt,
                             cudaStream_t st);
// Per query: -lse in log2 units and delta = sum(dY * Y).
cudaError_t launch_attn_bwd_prep(const AttnBwdArgs& a, flare_dtype_t dt, cudaStream_t st);
// The products; dQ, or dK and dV, may be NULL (not wanted).
cudaError_t launch_attn_bwd_tc(const AttnDims& d, const AttnBwdPlan& p, const AttnBwdArgs& a,
                               cudaStream_t st);
cudaError_t launch_attn_bwd_simt(const AttnBwdPlan& p, const AttnBwdArgs& a, cudaStream_t st);
// Sums the partials of the splits, in order, into dQ (which = 0) or dK and dV (1).
cudaError_t launch_attn_bwd_sum(const AttnBwdArgs& a, int dp, flare_dtype_t dt, int which,
                                cudaStream_t st);

// Argument checks shared by the entry points: a device pointer aligned to 16
// bytes; one tensor's strides (flare_strides_t, NULL = contiguous), reduced to
// Tok.  A dimension of one entry may have any stride.  Inputs may repeat a
// batch or a head (stride 0); the rows of an output may not overlap.
flare_status_t check_ptr(const void* p);
flare_status_t check_tok(const flare_strides_t* st, int64_t B, int64_t H, int64_t N, int64_t D,
                         flare_dtype_t dt, bool output, Tok* out);
flare_status_t check_workspace(const void* ws, size_t bytes, size_t need);
int sm_count();   // of the current device

#define FLARE_TRY(x)               \
  do {                             \
    flare_status_t s_ = (x);       \
    if (s_ != FLARE_OK) return s_; \
  } while (0)

// A failed launch: its description, unless the launcher left one.
#define FLARE_CUDA(x)                                                                \
  do {                                                                               \
    cudaError_t e_ = (x);                                                            \
    if (e_ != cudaSuccess) {                                                         \
      if (flare_last_error_detail()[0] == 0)                                         \
        note_error("%s: %s (%s)", #x, cudaGetErrorName(e_), cudaGetErrorString(e_)); \
      return FLARE_ERR_CUDA;                                                         \
    }                                                                                \
  } while (0)

}  // namespace flare

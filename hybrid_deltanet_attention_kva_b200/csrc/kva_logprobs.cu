// Scores of rows of logits (kva_op_token_logprobs): with m = max x, s = sum e^(x-m) and
// w = sum e^(x-m) (x-m),
//     lse = m + log s,   log p_j = (x_j - m) - log s,   entropy = log s - w / s,
// and the n_top largest logits (ties in token order).
#include "../../include/kva_ops.h"
#include "kva_common.cuh"

namespace kva {
namespace {

constexpr int LP_THREADS = 512;

template <typename T>
__device__ __forceinline__ float lp_load(const T* p) { return F16<T>::to(*p); }
template <>
__device__ __forceinline__ float lp_load<float>(const float* p) { return *p; }

struct LpArgs {
  const void* logits;
  int64_t ld;
  int V;
  const int32_t* tokens;
  float* logprob;
  float* lse;
  float* entropy;
  int n_top;
  int32_t* top_id;
  float* top_logprob;
};

// One block per row; one pass for the maximum, one for the sums, one per alternative.
template <typename T>
__global__ void __launch_bounds__(LP_THREADS) logprobs_kernel(const LpArgs p) {
  __shared__ float ra[LP_THREADS / 32], rb[LP_THREADS / 32];
  __shared__ int ri[LP_THREADS / 32];
  griddep_wait_and_release();
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(p.logits) + row * p.ld;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float kInf = __int_as_float(0x7f800000);
  const float kNan = __int_as_float(0x7fffffff);

  float m = -kInf, bad = 0.f;
  for (int i = tid; i < p.V; i += LP_THREADS) {
    const float v = lp_load(x + i);
    m = fmaxf(m, v);
    if (!(v < kInf)) bad = 1.f;  // NaN or +infinity
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    bad = fmaxf(bad, __shfl_xor_sync(0xffffffffu, bad, o));
  }
  if (lane == 0) {
    ra[warp] = m;
    rb[warp] = bad;
  }
  __syncthreads();
  for (int i = 0; i < LP_THREADS / 32; ++i) {
    m = fmaxf(m, ra[i]);
    bad = fmaxf(bad, rb[i]);
  }
  __syncthreads();
  const bool nan = bad != 0.f, empty = !nan && m == -kInf;

  float s = 0.f, w = 0.f;
  if (!nan && !empty)
    for (int i = tid; i < p.V; i += LP_THREADS) {
      const float d = lp_load(x + i) - m, e = expf(d);
      s += e;
      w += e > 0.f ? e * d : 0.f;
    }
  s = warp_sum(s);
  w = warp_sum(w);
  if (lane == 0) {
    ra[warp] = s;
    rb[warp] = w;
  }
  __syncthreads();
  s = w = 0.f;
  for (int i = 0; i < LP_THREADS / 32; ++i) {
    s += ra[i];
    w += rb[i];
  }
  __syncthreads();
  // a row with nothing left: with reference 0 and sum 1, x - m - log s is -infinity by itself
  if (empty) {
    m = w = 0.f;
    s = 1.f;
  }
  const float logs = logf(s);
  if (tid == 0) {
    if (p.lse) p.lse[row] = nan ? kNan : empty ? -kInf : m + logs;
    if (p.entropy) p.entropy[row] = nan ? kNan : logs - w / s;
    if (p.tokens) {
      const int t = p.tokens[row];
      if (nan || t < -1 || t >= p.V) p.logprob[row] = kNan;
      else if (t == -1) p.logprob[row] = 0.f;
      else p.logprob[row] = (lp_load(x + t) - m) - logs;
    }
  }

  // alternatives in order: the largest (value, then lowest id) behind the previous one
  float pv = kInf;
  int pi = -1;
  for (int j = 0; j < p.n_top; ++j) {
    float bv = -kInf;
    int bi = -1;
    if (!nan && !empty && (j == 0 || pi >= 0))
      for (int i = tid; i < p.V; i += LP_THREADS) {
        const float v = lp_load(x + i);
        if (v > bv && (v < pv || (v == pv && i > pi))) {
          bv = v;
          bi = i;
        }
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
      const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
      if (oi >= 0 && (bi < 0 || ov > bv || (ov == bv && oi < bi))) {
        bv = ov;
        bi = oi;
      }
    }
    if (lane == 0) {
      ra[warp] = bv;
      ri[warp] = bi;
    }
    __syncthreads();
    bv = ra[0];
    bi = ri[0];
    for (int i = 1; i < LP_THREADS / 32; ++i)
      if (ri[i] >= 0 && (bi < 0 || ra[i] > bv || (ra[i] == bv && ri[i] < bi))) {
        bv = ra[i];
        bi = ri[i];
      }
    __syncthreads();
    pv = bv;
    pi = bi;
    if (tid == 0) {
      p.top_id[row * p.n_top + j] = bi;
      p.top_logprob[row * p.n_top + j] = nan ? kNan : bi < 0 ? -kInf : (bv - m) - logs;
    }
  }
}

}  // namespace
}  // namespace kva

extern "C" int kva_op_token_logprobs(const void* logits, int32_t dtype, int64_t ld, int32_t rows, int32_t n_vocab,
                                     const int32_t* tokens, float* logprob, float* lse, float* entropy,
                                     int32_t n_top, int32_t* top_id, float* top_logprob, void* stream) {
  using namespace kva;
  if (rows < 0 || n_vocab <= 0 || n_top < 0) return KVA_ERR_INVALID_ARG;
  if (dtype != KVA_BF16 && dtype != KVA_F16 && dtype != KVA_F32) return KVA_ERR_INVALID_ARG;
  if (n_top > KVA_LOGPROB_MAX_TOP) return KVA_ERR_TOO_LARGE;
  if (rows == 0) return KVA_OK;
  if (!logits || ld < n_vocab || (tokens != nullptr) != (logprob != nullptr)) return KVA_ERR_INVALID_ARG;
  if (n_top > 0 && (!top_id || !top_logprob)) return KVA_ERR_INVALID_ARG;
  if (!tokens && !lse && !entropy && n_top == 0) return KVA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(logits) & (dtype == KVA_F32 ? 3u : 1u)) return KVA_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(tokens) | reinterpret_cast<uintptr_t>(logprob) | reinterpret_cast<uintptr_t>(lse) |
       reinterpret_cast<uintptr_t>(entropy) | reinterpret_cast<uintptr_t>(top_id) |
       reinterpret_cast<uintptr_t>(top_logprob)) & 3u)
    return KVA_ERR_ALIGNMENT;
  const LpArgs p{logits, ld, n_vocab, tokens, logprob, lse, entropy, n_top, top_id, top_logprob};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(rows), block(LP_THREADS);
  const cudaError_t r = dtype == KVA_F32   ? launch_pdl(logprobs_kernel<float>, grid, block, 0, s, p)
                        : dtype == KVA_F16 ? launch_pdl(logprobs_kernel<__half>, grid, block, 0, s, p)
                                           : launch_pdl(logprobs_kernel<__nv_bfloat16>, grid, block, 0, s, p);
  return r == cudaSuccess ? KVA_OK : KVA_ERR_CUDA;
}

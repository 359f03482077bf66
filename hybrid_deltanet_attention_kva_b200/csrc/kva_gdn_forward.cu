// Gated delta rule with its readout for every token (kva_op_gdn_forward):
//     u_t = beta_t (v_t - e^(g_t) S_(t-1) k_t)
//     S_t = e^(g_t) S_(t-1) + u_t k_t^T,   o_t = scale S_t q_t.
// Row v of S takes only v_t[v], k_t and the gates, so the d rows of a head are
// independent; the tokens are sequential.
#include "../../include/kva_ops.h"
#include "kva_common.cuh"

namespace kva {
namespace {

struct GdnFwd {
  const void* q;
  const void* k;
  const void* v;
  int64_t q_ld, q_seq, k_ld, k_seq, v_ld, v_seq;
  const float* gb;
  const float* state_in;
  float* state_out;
  void* out;
  int64_t out_ld, out_seq;
  int T, n_k, n_v, has_lens;
  float scale;
  int* err;
  int32_t lens[KVA_GDN_MAX_SEQ];
};

// 4 consecutive 16-bit values as floats
template <typename T>
__device__ __forceinline__ void load4(float (&f)[4], const T* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  const float2 a = F16<T>::unpack(u.x), b = F16<T>::unpack(u.y);
  f[0] = a.x;
  f[1] = a.y;
  f[2] = b.x;
  f[3] = b.y;
}
__device__ __forceinline__ float sum8(float v) {  // over the 8 lanes of a row
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v;
}

// Token by token.  8 lanes hold a state row in fp32 registers (lane l the columns
// 32 i + 4 l + j), a block of 256 threads 32 rows; grid (n_v * D / 32, n_seq).
template <typename T, int D>
__global__ void __launch_bounds__(256) gdn_recurrent_kernel(const __grid_constant__ GdnFwd p) {
  constexpr int NI = D / 32;
  griddep_wait_and_release();
  const int h = blockIdx.x / NI, seq = blockIdx.y;
  const int row = (blockIdx.x % NI) * 32 + (threadIdx.x >> 3), l = threadIdx.x & 7;
  const int kh = h / (p.n_v / p.n_k);
  const int len = p.has_lens ? p.lens[seq] : p.T;
  const int64_t srow = ((static_cast<int64_t>(seq) * p.n_v + h) * D + row) * D + 4 * l;
  const T* q = static_cast<const T*>(p.q) + seq * p.q_seq + kh * D + 4 * l;
  const T* k = static_cast<const T*>(p.k) + seq * p.k_seq + kh * D + 4 * l;
  const T* v = static_cast<const T*>(p.v) + seq * p.v_seq + h * D + row;
  T* out = static_cast<T*>(p.out) + seq * p.out_seq + h * D + row;
  const float* g = p.gb + (static_cast<int64_t>(seq) * 2 * p.n_v + h) * p.T;
  const float* b = g + static_cast<int64_t>(p.n_v) * p.T;

  float s[NI][4];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const float4 x = *reinterpret_cast<const float4*>(p.state_in + srow + 32 * i);
    s[i][0] = x.x;
    s[i][1] = x.y;
    s[i][2] = x.z;
    s[i][3] = x.w;
  }
  for (int t = 0; t < len; ++t) {
    const float dec = expf(g[t]);
    float kk[NI][4], sk = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      load4<T>(kk[i], k + t * p.k_ld + 32 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] *= dec;
        sk = fmaf(s[i][j], kk[i][j], sk);
      }
    }
    const float u = b[t] * (F16<T>::to(v[t * p.v_ld]) - sum8(sk));
    float o = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      float qq[4];
      load4<T>(qq, q + t * p.q_ld + 32 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = fmaf(u, kk[i][j], s[i][j]);
        o = fmaf(s[i][j], qq[j], o);
      }
    }
    o = sum8(o);
    if (l == 0) out[t * p.out_ld] = F16<T>::from(p.scale * o);
  }
#pragma unroll
  for (int i = 0; i < NI; ++i)
    *reinterpret_cast<float4*>(p.state_out + srow + 32 * i) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
}

template <typename T, int D>
cudaError_t launch(const GdnFwd& p, int n_seq, cudaStream_t s) {
  return launch_pdl(gdn_recurrent_kernel<T, D>, dim3(p.n_v * (D / 32), n_seq), dim3(256), 0, s, p);
}

bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace kva

extern "C" int kva_op_gdn_forward(const kva_gdn_forward_args* a, int32_t* err, void* stream) {
  using namespace kva;
  if (!a) return KVA_ERR_INVALID_ARG;
  if (a->dtype != KVA_BF16 && a->dtype != KVA_F16) return KVA_ERR_INVALID_ARG;
  if (a->n_seq < 0 || a->T < 0 || a->n_k <= 0 || a->n_v <= 0 || a->n_v % a->n_k) return KVA_ERR_INVALID_ARG;
  if (a->d != 64 && a->d != 128) return KVA_ERR_UNSUPPORTED;
  if (a->n_seq > KVA_GDN_MAX_SEQ || a->n_v > (1 << 20)) return KVA_ERR_TOO_LARGE;
  if (a->n_seq == 0) return KVA_OK;
  if (!a->state_in || !a->state_out) return KVA_ERR_INVALID_ARG;
  if (a->T > 0) {
    if (!a->q || !a->k || !a->v || !a->gb || !a->out) return KVA_ERR_INVALID_ARG;
    const int64_t wk = static_cast<int64_t>(a->n_k) * a->d, wv = static_cast<int64_t>(a->n_v) * a->d;
    if (a->q_ld < wk || a->k_ld < wk || a->v_ld < wv || a->out_ld < wv) return KVA_ERR_INVALID_ARG;
    if (a->q_seq < 0 || a->k_seq < 0 || a->v_seq < 0 || a->out_seq < 0) return KVA_ERR_INVALID_ARG;
    // the output rows are distinct: sequence after sequence, or token after token
    if (a->n_seq > 1 && a->out_seq < (a->T - 1) * a->out_ld + wv &&
        (a->out_seq < wv || a->out_ld < (a->n_seq - 1) * a->out_seq + wv))
      return KVA_ERR_INVALID_ARG;
    if ((a->q_ld | a->q_seq | a->k_ld | a->k_seq | a->v_ld | a->v_seq | a->out_ld | a->out_seq) & 7)
      return KVA_ERR_ALIGNMENT;
    if (!a16(a->q) || !a16(a->k) || !a16(a->v) || !a16(a->out) || (reinterpret_cast<uintptr_t>(a->gb) & 3u))
      return KVA_ERR_ALIGNMENT;
  }
  if (!a16(a->state_in) || !a16(a->state_out)) return KVA_ERR_ALIGNMENT;
  GdnFwd p;
  p.has_lens = a->lens != nullptr;
  if (a->lens)
    for (int i = 0; i < a->n_seq; ++i) {
      if (a->lens[i] < 0 || a->lens[i] > a->T) return KVA_ERR_INVALID_ARG;
      p.lens[i] = a->lens[i];
    }
  p.q = a->q;
  p.k = a->k;
  p.v = a->v;
  p.q_ld = a->q_ld;
  p.q_seq = a->q_seq;
  p.k_ld = a->k_ld;
  p.k_seq = a->k_seq;
  p.v_ld = a->v_ld;
  p.v_seq = a->v_seq;
  p.gb = a->gb;
  p.state_in = a->state_in;
  p.state_out = a->state_out;
  p.out = a->out;
  p.out_ld = a->out_ld;
  p.out_seq = a->out_seq;
  p.T = a->T;
  p.n_k = a->n_k;
  p.n_v = a->n_v;
  p.scale = a->scale;
  p.err = err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f16 = a->dtype == KVA_F16;
  const cudaError_t r = a->d == 128
                            ? (f16 ? launch<__half, 128>(p, a->n_seq, s) : launch<__nv_bfloat16, 128>(p, a->n_seq, s))
                            : (f16 ? launch<__half, 64>(p, a->n_seq, s) : launch<__nv_bfloat16, 64>(p, a->n_seq, s));
  return r == cudaSuccess ? KVA_OK : KVA_ERR_CUDA;
}

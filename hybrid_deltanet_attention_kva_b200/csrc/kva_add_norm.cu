// Residual addition and RMSNorm in one pass (kva_op_add_rmsnorm):
//     h' = h + x (rounded to the stream's type),  y = h' / sqrt(mean(h'^2) + eps) * g,
// y in 16 bits or as q8_0 blocks of 32 (int8 codes, fp16 scale max|y| / 127).
// The norm is taken of the stored row, so a later reader of the stream finds the row that was
// normalised.  The sum of squares is fp32.
#include "../../include/kva_ops.h"
#include "kva_common.cuh"

namespace kva {
namespace {

template <typename T>
struct Io;
template <>
struct Io<float> {
  __device__ static __forceinline__ float4 load(const float* p) { return *reinterpret_cast<const float4*>(p); }
  __device__ static __forceinline__ float4 store(float* p, float4 v) {
    *reinterpret_cast<float4*>(p) = v;
    return v;
  }
};
template <typename T>
struct Io16 {
  __device__ static __forceinline__ float4 load(const T* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const float2 a = F16<T>::unpack(u.x), b = F16<T>::unpack(u.y);
    return make_float4(a.x, a.y, b.x, b.y);
  }
  // stores v rounded to T and returns what was stored
  __device__ static __forceinline__ float4 store(T* p, float4 v) {
    uint2 u;
    u.x = F16<T>::pack(v.x, v.y);
    u.y = F16<T>::pack(v.z, v.w);
    *reinterpret_cast<uint2*>(p) = u;
    const float2 a = F16<T>::unpack(u.x), b = F16<T>::unpack(u.y);
    return make_float4(a.x, a.y, b.x, b.y);
  }
};
template <>
struct Io<__half> : Io16<__half> {};
template <>
struct Io<__nv_bfloat16> : Io16<__nv_bfloat16> {};

__device__ __forceinline__ float reciprocal(float x) {  // of the largest x too, which is subnormal
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// One q8_0 code in the low byte, y inv to the nearest integer, in one instruction and without the
// conversion unit: in the sum with 1.5 x 2^23 a last place is 1, and its low byte is the code in two's
// complement.
__device__ __forceinline__ uint32_t q8_code(float y, float inv) {
  return __float_as_uint(fmaf(y, inv, 12582912.f));
}
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {  // low bytes
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// TPR threads (a warp, or the block) take a row: NV groups of 4 values each, held in registers
// from the one read of x and h to the last write.  NV is the next of 4, 6 and 8 (fewer registers, more
// rows in flight).  HBM bounds the 16-bit forms: 8192 x 5120 bf16 50.5 us (6.6 TB/s, the measured copy rate);
// the q8_0 form also the conversion: 1024 x 5120 fp32 14.9 us (4.6 TB/s; 13.0 with a 16-bit output), 8192 x
// 5120 bf16 56.2 us (5.3 TB/s); the scattered scales cost nothing measurable.  One row 2.0 us.  Measured and
// not kept for q8_0: five or six blocks an SM (spills, 1.3 and 1.5 x the time); blocks as wide as a row needs
// with 8 values a thread (the same for fp32, 8192 x 5120 bf16 77 against 61 us); 8 values in a row a thread
// (14.5 against 14.8 us, bf16 68 against 56 us).
template <typename TX, typename TH, typename TO, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
    add_rmsnorm_kernel(const TX* __restrict__ x, int64_t ldx, const TH* h, TH* h_out, int64_t ldh,
                       const float* __restrict__ g, TO* __restrict__ out, int64_t ldo,
                       __half* __restrict__ scales, int rows, int n, float eps) {
  constexpr int THREADS = TPR < 256 ? 256 : TPR, RPB = THREADS / TPR;  // rows a block
  griddep_wait_and_release();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * RPB + threadIdx.x / TPR;
  const int col = threadIdx.x % TPR * 4;
  if (TPR == 32 && row >= rows) return;  // (whole warps)
  x += row * ldx;
  h += row * ldh;
  h_out += row * ldh;
  out += row * ldo;
  float4 v[NV], a[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = col + k * 4 * TPR;
    v[k] = a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < n) {
      a[k] = Io<TX>::load(x + i);
      v[k] = Io<TH>::load(h + i);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = col + k * 4 * TPR;
    if (i < n) {
      v[k] = Io<TH>::store(h_out + i, make_float4(a[k].x + v[k].x, a[k].y + v[k].y, a[k].z + v[k].z, a[k].w + v[k].w));
      ss += v[k].x * v[k].x + v[k].y * v[k].y + v[k].z * v[k].z + v[k].w * v[k].w;
    }
  }
  ss = warp_sum(ss);
  if (TPR > 32) {
    __shared__ float red[THREADS / 32];
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = ss;
    __syncthreads();
    ss = 0.f;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) ss += red[w];
  }
  const float sc = rsqrtf(ss / static_cast<float>(n) + eps);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = col + k * 4 * TPR;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < n) {
      const float4 gg = *reinterpret_cast<const float4*>(g + i);
      y = make_float4(v[k].x * sc * gg.x, v[k].y * sc * gg.y, v[k].z * sc * gg.z, v[k].w * sc * gg.w);
    }
    if constexpr (sizeof(TO) == 1) {
      if (k * 4 * TPR >= n) break;  // (the same for every thread)
      float amax = max_nan(max_nan(fabsf(y.x), fabsf(y.y)), max_nan(fabsf(y.z), fabsf(y.w)));
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (i < n) {
        const bool fine = amax < __int_as_float(0x7f800000);
        const float d = amax * (1.f / 127.f);
        // 127 / max to the last place by one Newton step (the residual 127 - max near, times the reciprocal), and
        // one up, so that a half goes away from zero; what is nearer to a half than 127 x 2^-22 may too.  (From
        // a subnormal d the reciprocal could overflow; such a d is 0 in fp16, whatever the codes.)
        const float r = reciprocal(amax), near = 127.f * r;
        const float up = __uint_as_float(__float_as_uint(fmaf(fmaf(-amax, near, 127.f), r, near)) + 1);
        const float inv = fine && d >= 1.1754944e-38f ? up : 0.f;
        uint32_t c = 0;
        if (fine) c = pack4(q8_code(y.x, inv), q8_code(y.y, inv), q8_code(y.z, inv), q8_code(y.w, inv));
        *reinterpret_cast<uint32_t*>(out + i) = c;
        if ((threadIdx.x & 7) == 0)
          scales[static_cast<int64_t>(i >> 5) * rows + row] = __float2half_rn(fine ? d : __int_as_float(0x7fffffff));
      }
    } else if (i < n) {
      Io<TO>::store(out + i, y);
    }
  }
}

struct Args {
  const void* x;
  int64_t ldx;
  const void* h;
  void* h_out;
  int64_t ldh;
  const float* g;
  void* out;
  int64_t ldo;
  void* scales;
  int rows, n;
  float eps;
  cudaStream_t s;
};

template <typename TX, typename TH, typename TO, int TPR, int NV>
cudaError_t launch(const Args& a) {
  constexpr int THREADS = TPR < 256 ? 256 : TPR, RPB = THREADS / TPR;
  return launch_pdl(add_rmsnorm_kernel<TX, TH, TO, TPR, NV>, dim3((static_cast<unsigned>(a.rows) + RPB - 1) / RPB), dim3(THREADS), 0, a.s,
                    static_cast<const TX*>(a.x), a.ldx, static_cast<const TH*>(a.h), static_cast<TH*>(a.h_out), a.ldh,
                    a.g, static_cast<TO*>(a.out), a.ldo, static_cast<__half*>(a.scales), a.rows, a.n, a.eps);
}
template <typename TX, typename TH, typename TO>
cudaError_t launch(const Args& a) {
  if (a.n <= 1024) return launch<TX, TH, TO, 32, 8>(a);
  if (a.n <= 4096) return launch<TX, TH, TO, 256, 4>(a);
  if (a.n <= 6144) return launch<TX, TH, TO, 256, 6>(a);
  return a.n <= 8192 ? launch<TX, TH, TO, 256, 8>(a) : launch<TX, TH, TO, 512, 8>(a);
}
template <typename TX, typename TH>
cudaError_t by_out(const Args& a, int out_dtype) {
  if (out_dtype == KVA_Q8_0) return launch<TX, TH, int8_t>(a);
  return out_dtype == KVA_F16 ? launch<TX, TH, __half>(a) : launch<TX, TH, __nv_bfloat16>(a);
}
template <typename TX>
cudaError_t by_h(const Args& a, int h_dtype, int out_dtype) {
  if (h_dtype == KVA_F32) return by_out<TX, float>(a, out_dtype);
  return h_dtype == KVA_F16 ? by_out<TX, __half>(a, out_dtype) : by_out<TX, __nv_bfloat16>(a, out_dtype);
}
bool is_float_dtype(int t) { return t == KVA_F32 || t == KVA_F16 || t == KVA_BF16; }

}  // namespace
}  // namespace kva

extern "C" int kva_op_add_rmsnorm(const void* x, int32_t x_dtype, int64_t ldx, const void* h, void* h_out,
                                  int32_t h_dtype, int64_t ldh, const float* g, void* out, int32_t out_dtype,
                                  int64_t ldo, void* scales, int32_t rows, int32_t n, float eps, void* stream) {
  using namespace kva;
  if (rows < 0 || n <= 0 || !(eps >= 0.f)) return KVA_ERR_INVALID_ARG;
  if (!is_float_dtype(x_dtype) || !is_float_dtype(h_dtype)) return KVA_ERR_INVALID_ARG;
  if (out_dtype != KVA_BF16 && out_dtype != KVA_F16 && out_dtype != KVA_Q8_0) return KVA_ERR_INVALID_ARG;
  if (n > 16 * 1024) return KVA_ERR_UNSUPPORTED;
  const bool q8 = out_dtype == KVA_Q8_0;
  if (q8 && n % 32) return KVA_ERR_UNSUPPORTED;
  if (rows == 0) return KVA_OK;
  if (!x || !h || !h_out || !g || !out || q8 != (scales != nullptr)) return KVA_ERR_INVALID_ARG;
  if (ldx < n || ldh < n || ldo < n) return KVA_ERR_INVALID_ARG;
  if (n % 4 || ldx % 4 || ldh % 4 || ldo % (q8 ? 16 : 4)) return KVA_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(h) | reinterpret_cast<uintptr_t>(h_out) |
       reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(out)) & 15u)
    return KVA_ERR_ALIGNMENT;
  if (reinterpret_cast<uintptr_t>(scales) & 1u) return KVA_ERR_ALIGNMENT;
  const Args a{x, ldx, h, h_out, ldh, g, out, ldo, scales, rows, n, eps, static_cast<cudaStream_t>(stream)};
  const cudaError_t r = x_dtype == KVA_F32   ? by_h<float>(a, h_dtype, out_dtype)
                        : x_dtype == KVA_F16 ? by_h<__half>(a, h_dtype, out_dtype)
                                             : by_h<__nv_bfloat16>(a, h_dtype, out_dtype);
  return r == cudaSuccess ? KVA_OK : KVA_ERR_CUDA;
}

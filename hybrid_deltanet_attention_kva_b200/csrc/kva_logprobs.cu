// Scores of rows of logits (kva_op_token_logprobs): with a reference m, s = sum 2^((x-m) log2 e)
// and w = sum 2^t t over t = (x-m) log2 e,
//     lse = m + log s,   log p_j = (x_j - m) - log s,   entropy = ln 2 (log2 s - w / s),
// and the n_top largest logits (ties in token order).
//
// One pass over the row: a thread keeps its own maximum, s and w.  The n_top largest come from a second
// look at a few threads' pieces only: the n_top-th largest of 64 thread groups' maxima is a lower bound
// of the n_top-th largest logit, and about n_top (1 + n_top / 128) logits reach it.  (A warp's sorted list, updated on the way, would issue more than the sums do.)
//
// 1024 rows of 131072 bf16 logits, 8 alternatives: 52.7 us, 5.1 TB/s.  A logit takes about 8
// instructions (conversion, half a maximum, half a multiply-add, clamp, exponential, half a sum and half a
// multiply-add), so the issue slots are busy too, and a row's joining and second look (10 k of 40 k
// cycles of its block) are hidden only by the SM's two other blocks.  One row in a cluster of 8: 5.5 us,
// four dependent memory and barrier latencies.
#include "../../include/kva_ops.h"
#include "kva_common.cuh"

namespace kva {
namespace {

constexpr int GROUPS = 64;      // thread groups whose maxima bound the alternatives
constexpr int CAP = 1024;       // logits at or above the bound that are kept for ranking
constexpr int MAX_CLUSTER = 8;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float T_MIN = -150.f; // 2^t is 0 from here on (and t times it: no 0 x infinity)

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

__device__ __forceinline__ float f_inf() { return __int_as_float(0x7f800000); }
__device__ __forceinline__ float f_nan() { return __int_as_float(0x7fffffff); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 bytes of logits
template <typename T>
struct Piece16 {
  static constexpr int N = 8;
  __device__ static __forceinline__ void unpack(const uint4& u, float (&f)[N]) {
    const float2 a = F16<T>::unpack(u.x), b = F16<T>::unpack(u.y), c = F16<T>::unpack(u.z), d = F16<T>::unpack(u.w);
    f[0] = a.x;
    f[1] = a.y;
    f[2] = b.x;
    f[3] = b.y;
    f[4] = c.x;
    f[5] = c.y;
    f[6] = d.x;
    f[7] = d.y;
  }
};
template <typename T>
struct Piece;
template <>
struct Piece<__half> : Piece16<__half> {
  static constexpr uint32_t NEG = 0xFC00FC00u;  // -infinity
  __device__ static __forceinline__ float one(const __half* p) { return __half2float(*p); }
  __device__ static __forceinline__ float largest(const uint4& u) {
    const __half2* h = reinterpret_cast<const __half2*>(&u);
    const __half2 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
    return max_nan(__low2float(m), __high2float(m));
  }
};
template <>
struct Piece<__nv_bfloat16> : Piece16<__nv_bfloat16> {
  static constexpr uint32_t NEG = 0xFF80FF80u;
  __device__ static __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  __device__ static __forceinline__ float largest(const uint4& u) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
    const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
    return max_nan(__low2float(m), __high2float(m));
  }
};
template <>
struct Piece<float> {
  static constexpr int N = 4;
  static constexpr uint32_t NEG = 0xFF800000u;
  __device__ static __forceinline__ float one(const float* p) { return *p; }
  __device__ static __forceinline__ void unpack(const uint4& u, float (&f)[N]) {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
  }
  __device__ static __forceinline__ float largest(const uint4& u) {
    return max_nan(max_nan(__uint_as_float(u.x), __uint_as_float(u.y)),
                   max_nan(__uint_as_float(u.z), __uint_as_float(u.w)));
  }
};

// Running sums of a thread relative to 2^r.  r follows the running maximum only when a logit comes
// 2^16 above it (so t keeps 20 bits behind the point), so it is set by the first batch and hardly
// ever again.  It is some logit times log2 e, rounded: r itself is the reference, so its rounding costs
// nothing.  From 1e38 on m log2 e would overflow; there no two different floats are near enough to
// weigh together: the factor is 1 and t = x - m is 0 or far below T_MIN.
constexpr float REBASE = 16.f;
struct Sums {
  float m, r, l;      // largest logit so far; the reference and its factor
  float2 s, w;        // two halves, for the packed fp32 instructions
  __device__ __forceinline__ void init() {
    m = r = -f_inf();
    l = LOG2E;
    s = w = make_float2(0.f, 0.f);
  }
  __device__ __forceinline__ void rebase(float to) {
    const float ln = fabsf(to) > 1e38f ? 1.f : LOG2E, rn = to * ln;
    const float d = l == LOG2E && ln == LOG2E ? fmaxf(r - rn, T_MIN) : T_MIN, f = ex2(d);
    // (nothing to move from the first reference, -infinity: s and w are 0)
    w = make_float2(f * fmaf(d, s.x, w.x), f * fmaf(d, s.y, w.y));
    s = make_float2(f * s.x, f * s.y);
    r = rn;
    l = ln;
  }
  // takes a batch whose largest logit is cm; false: NaN or infinity, the row has no distribution
  __device__ __forceinline__ bool take(float cm) {
    if (!(fmaf(cm, l, -r) <= REBASE)) {
      if (!(cm < f_inf())) return false;
      if (cm > -f_inf()) rebase(cm);
    }
    m = fmaxf(m, cm);
    return true;
  }
  // two logits; T_MIN keeps -infinity (0 x infinity) out of w
  __device__ __forceinline__ void add(float2 x) {
    float2 t = fma2(x, make_float2(l, l), make_float2(-r, -r));
    t = make_float2(fmaxf(t.x, T_MIN), fmaxf(t.y, T_MIN));
    const float2 e = make_float2(ex2(t.x), ex2(t.y));
    s = add2(s, e);
    w = fma2(e, t, w);
  }
};

// a row's results so far: of a warp, a block or the cluster; s and w relative to 2^r (factor l)
struct RowOut {
  float m, r, l, s, w;
  int bad;
};
// a joined with b, in place of a, relative to the reference of the larger maximum
__device__ __forceinline__ void join(RowOut& a, const RowOut& b) {
  const int bad = a.bad | b.bad;
  if (b.s > 0.f) {
    if (!(a.s > 0.f)) {
      a = b;
    } else {
      const RowOut hi = a.m >= b.m ? a : b, lo = a.m >= b.m ? b : a;
      const float d = lo.l == LOG2E && hi.l == LOG2E ? fmaxf(lo.r - hi.r, T_MIN)
                                                     : lo.l == hi.l && lo.r == hi.r ? 0.f : T_MIN;
      const float f = ex2(d);
      a.w = fmaf(f, fmaf(d, lo.s, lo.w), hi.w);
      a.s = fmaf(f, lo.s, hi.s);
      a.m = hi.m;
      a.r = hi.r;
      a.l = hi.l;
    }
  }
  a.bad = bad;
}

// over N lanes of every N-lane group
template <int N>
__device__ __forceinline__ void join_lanes(RowOut& a) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) {
    RowOut b;
    b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
    b.r = __shfl_xor_sync(0xffffffffu, a.r, o);
    b.l = __shfl_xor_sync(0xffffffffu, a.l, o);
    b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
    b.w = __shfl_xor_sync(0xffffffffu, a.w, o);
    b.bad = __shfl_xor_sync(0xffffffffu, a.bad, o);
    join(a, b);
  }
}

// A logit and its token as one number: larger logits first, of equal ones the lower token.  0: none.
__device__ __forceinline__ unsigned long long key_of(float v, int i) {
  const uint32_t u = __float_as_uint(v + 0.f);  // (-0 is 0)
  return static_cast<unsigned long long>(u & 0x80000000u ? ~u : u | 0x80000000u) << 32 | (0xffffffffu - i);
}
__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t u = static_cast<uint32_t>(k >> 32);
  return k ? __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u) : -f_inf();
}
__device__ __forceinline__ int key_token(unsigned long long k) {
  return k ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(k)) : -1;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// A cluster of CTAs per row, one contiguous range of 16-byte pieces each; block rank 0 joins them.
template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS, 1536 / THREADS) logprobs_kernel(const LpArgs p) {
  using P = Piece<T>;
  constexpr int WARPS = THREADS / 32, LANES = THREADS / GROUPS, BATCH = 4;
  using Key = unsigned long long;
  __shared__ RowOut part[WARPS], mine, all[MAX_CLUSTER];
  __shared__ float gmax[GROUPS], tau_s;
  __shared__ Key cand[CAP], top[KVA_LOGPROB_MAX_TOP], all_top[MAX_CLUSTER * KVA_LOGPROB_MAX_TOP];
  __shared__ int n_cand, n_again;
  __shared__ uint16_t again[THREADS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cl = static_cast<int>(gridDim.y), rank = blockIdx.y;
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(p.logits) + row * p.ld;
  // pieces: 16-byte aligned; piece j holds logits j N - off ..; the first and the last may be partial
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
  const int np = static_cast<int>((static_cast<int64_t>(p.V) + off + P::N - 1) / P::N);
  const int per = (np + cl - 1) / cl;
  const int j0 = min(rank * per, np), j1 = min(j0 + per, np);
  const int f0 = max(j0, off ? 1 : 0), f1 = min(j1, static_cast<int>((static_cast<int64_t>(p.V) + off) / P::N));
  const uint4* xp = reinterpret_cast<const uint4*>(x - off);
  if (tid == 0) {
    n_cand = n_again = 0;
    tau_s = -f_inf();
  }
  if (cl > 1) cluster_arrive();  // (waited for before the first write to another block)
  griddep_wait_and_release();

  Sums a;
  a.init();
  bool bad = false;
  float x_tok = 0.f;
  int tok = -1;
  if (tid == 0 && rank == 0 && p.tokens) {
    tok = p.tokens[row];
    if (tok >= 0 && tok < p.V) x_tok = P::one(x + tok);
  }
  for (int j = f0 + tid; j < f1; j += BATCH * THREADS) {
    uint4 u[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      u[i] = j + i * THREADS < f1 ? __ldg(xp + j + i * THREADS) : make_uint4(P::NEG, P::NEG, P::NEG, P::NEG);
    float cm = P::largest(u[0]);
#pragma unroll
    for (int i = 1; i < BATCH; ++i) cm = max_nan(cm, P::largest(u[i]));
    if (!a.take(cm)) {
      bad = true;
      break;
    }
    if (cm == -f_inf()) continue;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      float f[P::N];
      P::unpack(u[i], f);
#pragma unroll
      for (int e = 0; e < P::N; e += 2) a.add(make_float2(f[e], f[e + 1]));
    }
  }
  // the partial pieces, at most N - 1 logits before the first full one and behind the last: a thread
  // each.  e0 and e1 are the logits of this thread's
  int e0 = 0, e1 = 0;
  if (tid == 0 && rank == 0 && off) {
    e1 = min(P::N - off, p.V);
  } else if (tid == 1 && j1 == np && j0 < np) {
    const int last = static_cast<int>((static_cast<int64_t>(p.V) + off) / P::N * P::N) - off;  // behind the full pieces
    if (last >= (off ? P::N - off : 0)) {
      e0 = last;
      e1 = p.V;
    }
  }
  for (int i = e0; i < e1; ++i) {
    const float v = P::one(x + i);
    if (!a.take(v)) bad = true;
    else if (v > -f_inf()) a.add(make_float2(v, -f_inf()));
  }

  // join the block's threads
  float g = a.m;
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
  if (tid % LANES == 0) gmax[tid / LANES] = g;
  // a warp's sums, relative to its largest logit
  RowOut ro;
  {
    float m = a.m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float l = fabsf(m) > 1e38f ? 1.f : LOG2E, r = m * l;
    const float sa = a.s.x + a.s.y, wa = a.w.x + a.w.y;
    float d = a.l == LOG2E && l == LOG2E ? fmaxf(a.r - r, T_MIN) : a.l == l && a.r == r ? 0.f : T_MIN;
    if (!(sa > 0.f)) d = T_MIN;
    const float f = ex2(d);
    ro.m = m;
    ro.r = r;
    ro.l = l;
    ro.s = warp_sum(f * sa);
    ro.w = warp_sum(f * fmaf(d, sa, wa));
    ro.bad = __any_sync(0xffffffffu, bad);
  }
  if (lane == 0) part[warp] = ro;
  __syncthreads();
  const int k = p.n_top;
  float tau = 0.f;
  if (k > 0) {
    // the k-th largest of the groups' maxima: each of a group's threads compares with a share of them
    const int mg = tid / LANES, sub = tid % LANES;
    const float v = gmax[mg];
    int before_me = 0;
#pragma unroll
    for (int i = 0; i < GROUPS / LANES; ++i) {
      const float o = gmax[i * LANES + sub];
      before_me += o > v || (o == v && i * LANES + sub < mg);
    }
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) before_me += __shfl_xor_sync(0xffffffffu, before_me, o);
    if (sub == 0 && before_me == k - 1) tau_s = v;
    __syncthreads();
    tau = tau_s;
    if (tid < k) top[tid] = 0;
    // the threads that reach the bound are looked at again, a warp for each (its lanes take the
    // thread's pieces), so that one memory latency serves them all
    if (a.m >= tau && a.m > -f_inf()) again[atomicAdd(&n_again, 1)] = static_cast<uint16_t>(tid);
    __syncthreads();
  }
  if (warp == WARPS - 1) {
    RowOut r = part[lane % WARPS];
    join_lanes<WARPS>(r);
    if (lane == 0) mine = r;
  }
  if (k > 0) {
    auto take = [&](float v, int i) {
      if (v >= tau && v > -f_inf()) {
        const int at = atomicAdd(&n_cand, 1);  // (the order does not matter: candidates are ranked)
        if (at < CAP) cand[at] = key_of(v, i);
      }
    };
    const int n_look = n_again;
    for (int c = warp; c < n_look; c += WARPS)
      for (int j = f0 + again[c] + lane * THREADS; j < f1; j += 32 * THREADS) {
        const uint4 u = __ldg(xp + j);
        if (P::largest(u) >= tau) {
          float f[P::N];
          P::unpack(u, f);
#pragma unroll
          for (int e = 0; e < P::N; ++e) take(f[e], j * P::N - off + e);
        }
      }
    for (int i = e0; i < e1; ++i) take(P::one(x + i), i);
    __syncthreads();
    const int n = n_cand;
    if (n <= CAP) {
      for (int c = tid; c < n; c += THREADS) {
        const Key mk = cand[c];
        int before_me = 0;
#pragma unroll 8
        for (int i = 0; i < n; ++i) before_me += cand[i] > mk;
        if (before_me < k) top[before_me] = mk;
      }
    } else {
      // over CAP logits tie around the bound: one scan of the range per alternative, each for the
      // largest key below the one before
      const int s0 = max(j0 * P::N - off, 0), s1 = min(j1 * P::N - off, p.V);
      Key prev = ~0ull;
      for (int r = 0; r < k && prev; ++r) {  // (prev is the same for every thread)
        Key best = 0;
        for (int i = s0 + tid; i < s1; i += THREADS) {
          const float v = P::one(x + i);
          const Key c = v > -f_inf() ? key_of(v, i) : 0;
          if (c < prev && c > best) best = c;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const Key c = __shfl_xor_sync(0xffffffffu, best, o);
          best = c > best ? c : best;
        }
        if (lane == 0) cand[warp] = best;
        __syncthreads();
        best = cand[0];
        for (int i = 1; i < WARPS; ++i) best = cand[i] > best ? cand[i] : best;
        __syncthreads();
        prev = best;
        if (tid == 0) top[r] = best;
      }
    }
  }
  __syncthreads();
  if (cl > 1) {  // every block's results go to rank 0's shared memory
    cluster_wait();
    if (tid < k) st_cluster(mapa_shared(smem_u32(&all_top[rank * k + tid]), 0), top[tid]);
    if (tid >= THREADS - static_cast<int>(sizeof(RowOut) / 4)) {
      const int i = tid - (THREADS - static_cast<int>(sizeof(RowOut) / 4));
      st_cluster(mapa_shared(smem_u32(&all[rank]) + 4 * i, 0), reinterpret_cast<const uint32_t*>(&mine)[i]);
    }
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
    if (warp == WARPS - 1) {
      RowOut r{-f_inf(), 0.f, LOG2E, 0.f, 0.f, 0};
      if (lane < cl) r = all[lane];
      join_lanes<MAX_CLUSTER>(r);
      __syncwarp();
      if (lane == 0) mine = r;
    }
    const int n = cl * k;
    if (tid < k) top[tid] = 0;
    __syncthreads();
    for (int c = tid; c < n; c += THREADS) {
      const Key mk = all_top[c];
      int before_me = 0;
#pragma unroll 8
      for (int i = 0; i < n; ++i) before_me += all_top[i] > mk;
      if (mk && before_me < k) top[before_me] = mk;
    }
    __syncthreads();
  }
  // a row with nothing left: with reference 0 and sum 1, x - m - log s is -infinity by itself
  const bool nan = mine.bad != 0, empty = !nan && !(mine.s > 0.f);
  const float m = empty ? 0.f : mine.m, s = empty ? 1.f : mine.s, w = empty ? 0.f : mine.w;
  const float log2s = log2f(s);
  // log sum e^(x-m): the reference 2^r is 2^(m log2 e) but for r's rounding, which is added back
  const float logs = LN2 * (empty || mine.l != LOG2E ? log2s : log2s - fmaf(m, LOG2E, -mine.r));
  if (tid == 0) {
    if (p.lse) p.lse[row] = nan ? f_nan() : empty ? -f_inf() : m + logs;
    if (p.entropy) p.entropy[row] = nan ? f_nan() : LN2 * (log2s - w / s);
    if (p.tokens) p.logprob[row] = nan || tok < -1 || tok >= p.V ? f_nan() : tok == -1 ? 0.f : (x_tok - m) - logs;
  }
  for (int r = tid; r < k; r += THREADS) {
    p.top_id[row * k + r] = nan ? -1 : key_token(top[r]);
    p.top_logprob[row * k + r] = nan ? f_nan() : (key_value(top[r]) - m) - logs;
  }
}

// Blocks a row: as many as keep the GPU's SMs busy, at least one piece a thread and block, 8 at most
template <typename T, int THREADS>
cudaError_t launch(const LpArgs& p, int rows, cudaStream_t s) {
  const int np = (p.V + Piece<T>::N - 1) / Piece<T>::N, sms = num_sms();
  int cl = 1;
  while (cl < MAX_CLUSTER && static_cast<int64_t>(rows) * cl < sms && np / (2 * cl) >= THREADS) cl *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(rows, cl);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = cl;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cl > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, THREADS>, p);
}
template <typename T>
cudaError_t launch(const LpArgs& p, int rows, cudaStream_t s) {
  // Short rows take small blocks, so that a thread still has a batch of pieces.  So do many rows, where more
  // blocks an SM hide each other's joins and a thread has more pieces for its share of one: with 256 threads
  // against 512, 8192 x 32000 bf16 118 against 145 us, 8192 x 65536 195 against 222; but 512 x 32000 15.3
  // against 13.5, 1024 x 65536 34.1 against 32.5 (the last round of blocks), 4096 x 131072 192 against 190.
  const int np = (p.V + Piece<T>::N - 1) / Piece<T>::N, sms = num_sms();
  if (np <= 1024) return launch<T, 128>(p, rows, s);
  if (rows >= 6 * sms && np <= (rows >= 12 * sms ? 8192 : 4096)) return launch<T, 256>(p, rows, s);
  return launch<T, 512>(p, rows, s);
}

}  // namespace
}  // namespace kva

extern "C" int kva_op_token_logprobs(const void* logits, int32_t dtype, int64_t ld, int32_t rows, int32_t n_vocab,
                                     const int32_t* tokens, float* logprob, float* lse, float* entropy,
                                     int32_t n_top, int32_t* top_id, float* top_logprob, void* stream) {
  using namespace kva;
  if (rows < 0 || n_vocab <= 0 || n_top < 0) return KVA_ERR_INVALID_ARG;
  if (dtype != KVA_BF16 && dtype != KVA_F16 && dtype != KVA_F32) return KVA_ERR_INVALID_ARG;
  if (n_top > KVA_LOGPROB_MAX_TOP || n_vocab > (1 << 30)) return KVA_ERR_TOO_LARGE;
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
  const cudaError_t r = dtype == KVA_F32   ? launch<float>(p, rows, s)
                        : dtype == KVA_F16 ? launch<__half>(p, rows, s)
                                           : launch<__nv_bfloat16>(p, rows, s);
  return r == cudaSuccess ? KVA_OK : KVA_ERR_CUDA;
}

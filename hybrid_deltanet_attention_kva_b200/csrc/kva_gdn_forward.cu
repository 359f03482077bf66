// Gated delta rule with its readout for every token (kva_op_gdn_forward):
//     u_t = beta_t (v_t - e^(g_t) S_(t-1) k_t)
//     S_t = e^(g_t) S_(t-1) + u_t k_t^T,   o_t = scale S_t q_t.
// Row v of S takes only v_t[v], k_t and the gates, so the d rows of a head are
// independent; the tokens are sequential.
#include <algorithm>
#include <type_traits>

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
  int stall_run1;                  // test of the failure path: this run (from 1) is never handed over; 0: none
  int32_t lens[KVA_GDN_MAX_SEQ];
  uint8_t order[KVA_GDN_MAX_SEQ];  // with lens: the sequences, longest first
  int first;                       // with lens: of those, the launch's first
};
static_assert(KVA_GDN_MAX_SEQ <= 256, "a sequence's number takes a byte");

// Sequences of at most this many tokens go token by token, longer ones in runs of 16.  At 8 tokens of a
// 16/48-head layer (bf16) one sequence takes 6.0 us against 6.9 in a run, 16 take 33.5 against 50.6, 64 take 115
// against 171 (fp16: 5.9 against 5.9, one sequence); a token more costs 0.4 us, 3 us and 11 us, a run nothing until
// it is full.  One number, so that a sequence's result does not depend on its neighbours.
constexpr int kStepTokens = 8;

__device__ __forceinline__ float sum4(float v) {  // over the 4 lanes of a fragment's row
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v;
}
__device__ __forceinline__ float sum8(float v) {  // over the 8 lanes of a row
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v;
}

// Token by token, for at most kStepTokens tokens.  8 lanes hold a state row in fp32 registers (lane l
// the columns 32 i + 4 l + j); a block of 256 threads takes 32 RPT rows, RPT a thread, so its k, q, v and
// gates are read once, together with the state, into shared memory.  HBM bounds it (the state is read
// and written once): one token of 64 sequences, 16/48 heads of 128, 61.5 us, 6.6 TB/s; one of a single
// sequence 3.0 us, launch and two memory latencies.  grid (n_v * D / (32 RPT), n_seq)
template <typename T, int D, int RPT>
__global__ void __launch_bounds__(256) gdn_recurrent_kernel(const __grid_constant__ GdnFwd p) {
  constexpr int NI = D / 32, ROWS = 32 * RPT, PARTS = D / ROWS, PC = D / 8;
  __shared__ __align__(16) T ks[kStepTokens * D], qs[kStepTokens * D], vs[kStepTokens * ROWS];
  __shared__ float ds[kStepTokens], bs[kStepTokens];
  griddep_wait_and_release();
  const int tid = threadIdx.x, h = blockIdx.x / PARTS, r0 = (blockIdx.x % PARTS) * ROWS;
  const int seq = p.has_lens ? p.order[p.first + blockIdx.y] : blockIdx.y, row = tid >> 3, l = tid & 7;
  const int kh = h / (p.n_v / p.n_k);
  const int len = p.has_lens ? p.lens[seq] : p.T;
  const int64_t srow = ((static_cast<int64_t>(seq) * p.n_v + h) * D + r0 + row) * D + 4 * l;

  float2 s[RPT][NI][2];
#pragma unroll
  for (int a = 0; a < RPT; ++a)
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const float4 x = __ldcs(reinterpret_cast<const float4*>(p.state_in + srow + a * 32 * D + 32 * i));
      s[a][i][0] = make_float2(x.x, x.y);
      s[a][i][1] = make_float2(x.z, x.w);
    }
  for (int x = tid; x < len * PC; x += 256) {
    const int t = x / PC, c = x % PC * 8;
    *reinterpret_cast<uint4*>(ks + t * D + c) =
        *reinterpret_cast<const uint4*>(static_cast<const T*>(p.k) + seq * p.k_seq + t * p.k_ld + kh * D + c);
    *reinterpret_cast<uint4*>(qs + t * D + c) =
        *reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + seq * p.q_seq + t * p.q_ld + kh * D + c);
  }
  for (int x = tid; x < len * (ROWS / 8); x += 256) {
    const int t = x / (ROWS / 8), c = x % (ROWS / 8) * 8;
    *reinterpret_cast<uint4*>(vs + t * ROWS + c) =
        *reinterpret_cast<const uint4*>(static_cast<const T*>(p.v) + seq * p.v_seq + t * p.v_ld + h * D + r0 + c);
  }
  if (tid < len) {
    const float* g = p.gb + (static_cast<int64_t>(seq) * 2 * p.n_v + h) * p.T + tid;
    ds[tid] = expf(*g);
    bs[tid] = g[static_cast<int64_t>(p.n_v) * p.T];
  }
  __syncthreads();
  T* out = static_cast<T*>(p.out) + seq * p.out_seq + h * D + r0 + row;
  for (int t = 0; t < len; ++t) {
    const float2 dec = make_float2(ds[t], ds[t]);
    const float beta = bs[t];
    float2 kk[NI][2], sk[RPT];
#pragma unroll
    for (int a = 0; a < RPT; ++a) sk[a] = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const uint2 u = *reinterpret_cast<const uint2*>(ks + t * D + 32 * i + 4 * l);
      kk[i][0] = F16<T>::unpack(u.x);
      kk[i][1] = F16<T>::unpack(u.y);
#pragma unroll
      for (int a = 0; a < RPT; ++a)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[a][i][e] = mul2(s[a][i][e], dec);
          sk[a] = fma2(s[a][i][e], kk[i][e], sk[a]);
        }
    }
    float2 o[RPT], u2[RPT];
#pragma unroll
    for (int a = 0; a < RPT; ++a) {
      const float u = beta * (F16<T>::to(vs[t * ROWS + a * 32 + row]) - sum8(sk[a].x + sk[a].y));
      u2[a] = make_float2(u, u);
      o[a] = make_float2(0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const uint2 u = *reinterpret_cast<const uint2*>(qs + t * D + 32 * i + 4 * l);
      const float2 q0 = F16<T>::unpack(u.x), q1 = F16<T>::unpack(u.y);
#pragma unroll
      for (int a = 0; a < RPT; ++a) {
        s[a][i][0] = fma2(u2[a], kk[i][0], s[a][i][0]);
        s[a][i][1] = fma2(u2[a], kk[i][1], s[a][i][1]);
        o[a] = fma2(s[a][i][0], q0, o[a]);
        o[a] = fma2(s[a][i][1], q1, o[a]);
      }
    }
#pragma unroll
    for (int a = 0; a < RPT; ++a) {
      const float r = sum8(o[a].x + o[a].y);
      if (l == 0) out[t * p.out_ld + a * 32] = F16<T>::from(p.scale * r);
    }
  }
#pragma unroll
  for (int a = 0; a < RPT; ++a)
#pragma unroll
    for (int i = 0; i < NI; ++i)
      __stcs(reinterpret_cast<float4*>(p.state_out + srow + a * 32 * D + 32 * i),
             make_float4(s[a][i][0].x, s[a][i][0].y, s[a][i][1].x, s[a][i][1].y));
}

// ============================================================================
// Runs of 16 tokens on mma.sync.  With gam_t = sum_{s<=t} g_s inside a run and S the state at
// its start,
//     L[t,s] = e^(gam_t-gam_s) k_t.k_s beta_s (s < t),     Tm = (I + L)^-1,
//     U      = (V^T - S K^T diag(e^gam)) Tm^T diag(beta)   (column s: the update u_s),
//     O      = S Q^T diag(e^gam) + U M^T,                  M[t,s] = e^(gam_t-gam_s) q_t.k_s (s <= t),
//     S     <- e^gam_last S + U diag(e^(gam_last-gam)) K.
// Tm, M and the decays take no state: preparing warps form them ahead of the chain.  A chain warp
// owns 16 rows of S as fp32 accumulator fragments, which are also (packed) the A operand of the
// next product, so a run passes through registers alone: no barrier between the chain's warps, and
// no trip of S through shared or tensor memory.
//
// The state may not see a 16-bit rounding (it carries over thousands of tokens), so S, W, Tm and the
// updates enter as two fp16 terms: two products where the partner is K or Q, three where it has two terms
// itself.  So do S and M on the way to the readout, which sees one 16-bit rounding only, the output's.  That
// makes 108 MMAs a warp and run.  The terms are in units that follow the data, or small states and values would
// lose fp16's last bits (1e-3 of a state of 1e-4) and large ones leave its range; bf16 inputs take fp16 terms as
// well: two bf16 terms left states 3.4e-6 off after 1024 tokens (fp16 terms: 2e-7), three of them would cost
// 30 % of the time.
//
// What bounds it: a run's chain of dependent steps.  16/48 heads of 128, one sequence of 1024
// tokens (96 blocks, one chain warp a scheduler): fp16 84 us, 1.3 us a run, bf16 89 us; eight sequences, where
// two chain warps share a scheduler: fp16 385 us, bf16 400 us (tensor pipe 47 % and issue slots 51 % busy).
// Left out one at a time in a copy, the state's second term on the way to the readout costs 6 us of the 84
// (27 to 36 us of eight sequences), the second terms of M and of the updates there 2, the units 1.
// Measured and not kept (us for 1 / 8 sequences, against the state of that step): the state's update added to it
// behind the products, so that they do not cut its last bit (states after 1024 tokens without decay 4.8e-7 off
// instead of 1.1e-6; 84 / 435 against 84 / 385, fp16), keys in units of their own (84 / 439 against 84 / 396, bf16),
// runs of 32 tokens (100 / 399 against 82 / 362), the columns
// split over pairs of warps (76 / 450 against 68 / 349), the update fused with the next run's Y (75 / 380
// against 68 / 349), readouts by warps of their own (69 / 363 against 66 / 349), Tm diag(e^gam) K formed by the
// preparing warps, so that U is V^T Tm^T less a product with S (78 / 387 against 66 / 357: the second term's
// MMAs and loads cost more than the step they save), the next run's wait and first loads ahead of this one's
// stores (69 / 370 against 66 / 357), and chunks of 64 tokens on
// tcgen05 with the state in tensor memory (120 / 372 against 82 / 362): there every product makes a round
// trip through tensor memory, 8 conversions a chunk at 0.5-2 k cycles, and an MMA takes about 96 cycles to
// issue.
// ============================================================================
constexpr int CH = 16;          // tokens a run
constexpr int LOADED = 4;       // runs in flight behind those being prepared
constexpr int NST = 8;          // stages: the run of AHEAD + 1 own steps back is consumed when its place is needed

template <int D, int ROWS>       // ROWS state rows a block
struct Stage {
  static constexpr int K = 0;                      // [16][D], 16-byte pieces xor-swizzled by row
  static constexpr int Q = K + CH * D * 2;
  static constexpr int V = Q + CH * D * 2;         // [16][ROWS], this block's columns
  static constexpr int TH = V + CH * ROWS * 2;     // 2^10 Tm as two 16-bit terms, [s][t]
  static constexpr int TL = TH + CH * CH * 2;
  static constexpr int MH = TL + CH * CH * 2;      // M as two 16-bit terms in units of MU, [t][s]
  static constexpr int ML = MH + CH * CH * 2;
  static constexpr int EG = ML + CH * CH * 2;      // e^gam[16]
  static constexpr int DEC = EG + CH * 4;          // e^(gam_last - gam)[16]
  static constexpr int EZ = DEC + CH * 4;          // e^gam[16] in q's units
  static constexpr int MU = EZ + CH * 4;           // the units of M's rows
  static constexpr int BT = MU + CH * 4;           // 2^-10 beta
  static constexpr int GL = BT + CH * 4;          // e^gam_last, e^gam_first; 1: ordinary run; largest beta
  static constexpr int VM = GL + 64;               // the largest |v| of each column; NaN if it has one
  static constexpr int BYTES = (VM + ROWS * 2 + 127) / 128 * 128;
};
struct Prep {                                      // per preparing warp: L in fp32 (row stride 20)
  static constexpr int LDL = 20;
  static constexpr int BYTES = CH * LDL * 4;
};
template <int D, int ROWS, int PREP>
struct Chunk {
  static constexpr int L = NST * Stage<D, ROWS>::BYTES;
  static constexpr int BAR = L + PREP * Prep::BYTES;  // full[NST], empty[NST]
  static constexpr int MISC = BAR + 2 * NST * 8;      // abort flag
  static constexpr int BYTES = MISC + 16;
};

// 16-byte piece c of row r in a tile of W-byte rows (W = 128 or 256): eight rows of one piece
// index fall on different banks
template <int W>
__device__ __forceinline__ uint32_t piece(int r, int c) {
  return static_cast<uint32_t>(r * W + ((c ^ (r & 7)) << 4));
}
// the same in a [16][16] 16-bit tile (32-byte rows)
__device__ __forceinline__ uint32_t piece16(int r, int c) {
  return static_cast<uint32_t>(r * 32 + ((c ^ ((r >> 2) & 1)) << 4));
}

// x as two fp16 terms, hi + lo: hi is x cut to 11 bits, so that the remainder does not wait for a
// conversion and back (x to 2^-21)
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const float2 h = make_float2(__uint_as_float(__float_as_uint(x) & 0xffffe000u),
                               __uint_as_float(__float_as_uint(y) & 0xffffe000u));
  const float2 l = sub2(make_float2(x, y), h);
  hi = pack_f16(h.x, h.y);
  lo = pack_f16(l.x, l.y);
}
// The chain's products take fp16 terms whatever the inputs' type, each state row's in units of a power of two
// that follows its data.  What is at most m is below 2^8 in its units.  For S and U, m is the largest of the
// row's beta |v| of a run (as the product of both's largest) and of the decayed norms e^gam_t |S row| in which the
// run's tokens meet it (the row at the run's end may be far below those); for W, of |v| and those.  With keys of
// norm <= 1 and beta <= 1 all stay below 18 m: below fp16's 65504, and what fp16 drops is 2^-32 m (2^-35 of Tm,
// whose entries are at most 1).  A run that ends far below m (strong decay of a state with little
// written to it) would lose its own precision by that, and a tiny bf16 key its last bits in fp16; gates or
// keys out of their range could pass 18 m, and a value that is not finite would reach the run's tokens before
// it: such runs go token by token in fp32 (step_tokens).
constexpr float kFar = 256.f;  // m over the larger of beta |v| and the row's norm behind the run: 2^-24 of those
constexpr float kKeyNorm2 = 1.015625f;  // keys of norm 1, each entry rounded to bf16
constexpr float kTinyKey2 = 0x1p-12f;   // bf16 keys of norm 2^-6: few entries below fp16's normal range
constexpr float kMost = 1.7e38f;
template <typename T>
constexpr bool kBf16 = F16<T>::umma_fmt == 1;
struct Scale {
  float up, down;
  __device__ __forceinline__ explicit Scale(float m) {
    const uint32_t e = max(__float_as_uint(m) & 0x7f800000u, 8u << 23) - (7u << 23);  // the exponent, at least -126
    up = __uint_as_float(e);
    down = __uint_as_float((254u << 23) - e);
  }
};
// the largest |x| of a lane's two rows (those of its fragments' lower and upper half)
template <int N>
__device__ __forceinline__ float2 largest_of_rows(const float (&x)[N][4]) {
  float2 m = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    m.x = fmaxf(m.x, fmaxf(fabsf(x[i][0]), fabsf(x[i][1])));
    m.y = fmaxf(m.y, fmaxf(fabsf(x[i][2]), fabsf(x[i][3])));
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    m.x = fmaxf(m.x, __shfl_xor_sync(0xffffffffu, m.x, o));
    m.y = fmaxf(m.y, __shfl_xor_sync(0xffffffffu, m.y, o));
  }
  return m;
}
template <int N>
__device__ __forceinline__ void scale_all(float (&x)[N][4], float2 f) {  // f: the factors of a lane's two rows
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const float y01 = j ? f.y : f.x;
      const float2 y = mul2(make_float2(x[i][j], x[i][j + 1]), make_float2(y01, y01));
      x[i][j] = y.x;
      x[i][j + 1] = y.y;
    }
}
// accumulator fragments of two neighbouring 8-column tiles as an A operand (16 x 16)
__device__ __forceinline__ void split_a(const float (&c0)[4], const float (&c1)[4], uint32_t (&hi)[4],
                                        uint32_t (&lo)[4]) {
  split2(c0[0], c0[1], hi[0], lo[0]);
  split2(c0[2], c0[3], hi[1], lo[1]);
  split2(c1[0], c1[1], hi[2], lo[2]);
  split2(c1[2], c1[3], hi[3], lo[3]);
}
// D += A B on 16 x 8 x 16 tiles: registers to registers, free to be scheduled
__device__ __forceinline__ void mma_tile(__half, float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tile(__nv_bfloat16, float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <typename T = __half>
__device__ __forceinline__ void mma2(float (&d0)[4], float (&d1)[4], const uint32_t (&a)[4], const uint32_t (&b)[4],
                                     int i0, int i1, int i2, int i3) {
  mma_tile(T(), d0, a, b[i0], b[i1]);
  mma_tile(T(), d1, a, b[i2], b[i3]);
}

// The rows of a [16][D] bf16 tile in fp16, each in units of a power of two that puts its largest entry
// below 2^8 (exact but for entries below 2^-22 of that one); returns this lane's row's unit.  Two lanes take a
// row, eight of whose neighbours' pieces fall on different banks.
template <int D>
__device__ __forceinline__ Scale rows_to_f16(uint8_t* tile, int lane) {
  const int r = lane >> 1, h = lane & 1;
  uint4 x[D / 16];
  __nv_bfloat162 m = __float2bfloat162_rn(0.f);
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
    x[j] = *reinterpret_cast<const uint4*>(tile + piece<2 * D>(r, (j & 3) | h << 2 | (j >> 2) << 3));
    const __nv_bfloat162* x2 = reinterpret_cast<const __nv_bfloat162*>(&x[j]);
    m = __hmax2(m, __hmax2(__hmax2(__habs2(x2[0]), __habs2(x2[1])), __hmax2(__habs2(x2[2]), __habs2(x2[3]))));
  }
  float big = fmaxf(__low2float(m), __high2float(m));
  big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
  const Scale sc(big);
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&x[j]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = mul2(unpack_bf16(w[i]), make_float2(sc.down, sc.down));
      w[i] = pack_f16(f.x, f.y);
    }
    *reinterpret_cast<uint4*>(tile + piece<2 * D>(r, (j & 3) | h << 2 | (j >> 2) << 3)) = x[j];
  }
  return sc;
}

// A preparing warp: runs pw, pw + PREP, ...
template <typename T, int D, int ROWS, int PREP>
__device__ void prepare_runs(const GdnFwd& p, uint8_t* sm, int h, int half, int seq, int len, int pw, int lane,
                             volatile int* abort_flag) {
  using St = Stage<D, ROWS>;
  constexpr int AHEAD = LOADED / PREP;  // own runs in flight behind the one worked on
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + Chunk<D, ROWS, PREP>::BAR);
  uint64_t* empty = full + NST;
  const int kh = h / (p.n_v / p.n_k), n_runs = (len + CH - 1) / CH;
  const T* q = static_cast<const T*>(p.q) + seq * p.q_seq + kh * D;
  const T* k = static_cast<const T*>(p.k) + seq * p.k_seq + kh * D;
  const T* v = static_cast<const T*>(p.v) + seq * p.v_seq + h * D + half * ROWS;
  const float* g = p.gb + (static_cast<int64_t>(seq) * 2 * p.n_v + h) * p.T;
  const float* b = g + static_cast<int64_t>(p.n_v) * p.T;
  float* Ls = reinterpret_cast<float*>(sm + Chunk<D, ROWS, PREP>::L + pw * Prep::BYTES);
  const uint32_t base = smem_u32(sm);

  // a lane copies one 16-byte column of every RK-th (V: RV-th) row of a run
  constexpr int PK = D / 8, PV = ROWS / 8, RK = 32 / PK, RV = 32 / PV;
  const int xk = lane % PK, rk = lane / PK, xv = lane % PV, rv = lane / PV;
  auto load = [&](int c) {  // rows past the sequence's end are zero, never read
    const uint32_t st = base + (c % NST) * St::BYTES;
    const int64_t t0 = static_cast<int64_t>(c) * CH;
    const T* kp = k + (t0 + rk) * p.k_ld + 8 * xk;
    const T* qp = q + (t0 + rk) * p.q_ld + 8 * xk;
    const T* vp = v + (t0 + rv) * p.v_ld + 8 * xv;
    if (t0 + CH <= len) {
#pragma unroll
      for (int i = 0; i < CH / RK; ++i) {
        cp_async16(st + St::K + piece<2 * D>(i * RK + rk, xk), kp, 16);
        cp_async16(st + St::Q + piece<2 * D>(i * RK + rk, xk), qp, 16);
        kp += RK * p.k_ld;
        qp += RK * p.q_ld;
      }
#pragma unroll
      for (int i = 0; i < CH / RV; ++i) {
        cp_async16(st + St::V + piece<2 * ROWS>(i * RV + rv, xv), vp, 16);
        vp += RV * p.v_ld;
      }
    } else {
      for (int i = 0; i < CH / RK; ++i) {
        const bool on = t0 + i * RK + rk < len;
        cp_async16(st + St::K + piece<2 * D>(i * RK + rk, xk), on ? kp + i * RK * p.k_ld : k, on ? 16 : 0);
        cp_async16(st + St::Q + piece<2 * D>(i * RK + rk, xk), on ? qp + i * RK * p.q_ld : q, on ? 16 : 0);
      }
      for (int i = 0; i < CH / RV; ++i) {
        const bool on = t0 + i * RV + rv < len;
        cp_async16(st + St::V + piece<2 * ROWS>(i * RV + rv, xv), on ? vp + i * RV * p.v_ld : v, on ? 16 : 0);
      }
    }
  };
  float g_next = 0.f, b_next = 0.f;
  auto load_gates = [&](int c) {
    const int t = c * CH + lane;
    const bool on = lane < CH && t < len;
    g_next = on ? g[t] : 0.f;
    b_next = on ? b[t] : 0.f;
  };
  for (int j = 0; j < AHEAD; ++j) {
    if (pw + PREP * j < n_runs) load(pw + PREP * j);
    cp_async_commit();
  }
  load_gates(pw);
  const int mi = lane >> 3, lr = lane & 7, gr = lane >> 2, cq = lane & 3;

  for (int c = pw; c < n_runs; c += PREP) {
    const int cn = c + PREP * AHEAD;
    if (cn < n_runs) {
      if (cn >= NST && !mbar_wait_warp(&empty[cn % NST], (cn / NST - 1) & 1, abort_flag)) {
        *abort_flag = 1;
        set_device_error(p.err, KVA_DEV_WAIT_TIMEOUT);
        break;
      }
      load(cn);
    }
    cp_async_commit();
    float gt = g_next;
    const float bt = b_next;
    bool ordinary = gt <= 0.f && bt >= 0.f && bt <= 1.f;
    load_gates(c + PREP);  // (past the last run: zeros)
    // e^g is 0 in fp32 from -104 on; the clamp keeps -infinity out of the differences
    gt = gt < -1000.f ? -1000.f : gt;
    // cumulative decays as unevaluated sums of two floats: differences of neighbours keep fp32's
    // precision however far the sum has run (fp64 costs 3x the time here)
    float gam = gt, gaml = 0.f;
#pragma unroll
    for (int o = 1; o < CH; o <<= 1) {
      const float y = __shfl_up_sync(0xffffffffu, gam, o), yl = __shfl_up_sync(0xffffffffu, gaml, o);
      if (lane >= o) {
        const float s = gam + y, r = s - gam;
        gaml += yl + ((gam - (s - r)) + (y - r));  // the sum's rounding, exactly (Knuth's two-sum)
        gam = s;
      }
    }
    const float last = __shfl_sync(0xffffffffu, gam, CH - 1), lastl = __shfl_sync(0xffffffffu, gaml, CH - 1);
    uint8_t* st = sm + (c % NST) * St::BYTES;
    const uint32_t sst = base + (c % NST) * St::BYTES;
    if (lane < CH) {
      reinterpret_cast<float*>(st + St::EG)[lane] = expf(gam + gaml);
      reinterpret_cast<float*>(st + St::DEC)[lane] = expf((last - gam) + (lastl - gaml));
      reinterpret_cast<float*>(st + St::BT)[lane] = bt * 0x1p-10f;
      if (lane == 0) *reinterpret_cast<float2*>(st + St::GL) = make_float2(expf(last + lastl), expf(gam));
    }
    // pair decays of this thread's fragment elements (t = gr + 8 a, s = 8 i + 2 cq + e); the fast
    // exponential is off by 2^-22 + |x| 2^-24, and what is far has no weight
    float pd[2][4];
    {
      const float t0 = __shfl_sync(0xffffffffu, gam, gr), t0l = __shfl_sync(0xffffffffu, gaml, gr);
      const float t1 = __shfl_sync(0xffffffffu, gam, gr + 8), t1l = __shfl_sync(0xffffffffu, gaml, gr + 8);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int s = 8 * i + 2 * cq + e;
          const float gs = __shfl_sync(0xffffffffu, gam, s), gsl = __shfl_sync(0xffffffffu, gaml, s);
          pd[i][e] = s <= gr ? __expf((t0 - gs) + (t0l - gsl)) : 0.f;
          pd[i][2 + e] = s <= gr + 8 ? __expf((t1 - gs) + (t1l - gsl)) : 0.f;
        }
    }
    cp_async_wait<AHEAD>();
    __syncwarp();
    // K K^T and Q K^T: the K fragments serve as A and as B
    float kk[2][4] = {}, qk[2][4] = {};
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t a[4], x[4];
      ldmatrix_x4(a, sst + St::K + piece<2 * D>((mi & 1) * 8 + lr, 2 * ks + (mi >> 1)));
      ldmatrix_x4(x, sst + St::Q + piece<2 * D>((mi & 1) * 8 + lr, 2 * ks + (mi >> 1)));
      mma2<T>(kk[0], kk[1], a, a, 0, 2, 1, 3);
      mma2<T>(qk[0], qk[1], x, a, 0, 2, 1, 3);
    }
    {
      const float k0 = gr & 1 ? kk[0][1] : kk[0][0], k1 = gr & 1 ? kk[1][3] : kk[1][2];  // |k_t|^2, t = gr, gr + 8
      auto fits = [](float k2) { return k2 <= kKeyNorm2 && (!kBf16<T> || k2 >= kTinyKey2 || k2 == 0.f); };
      ordinary = __all_sync(0xffffffffu, ordinary && (cq != gr >> 1 || (fits(k0) && fits(k1))));
      const float most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(bt)));
      if (lane == 0) reinterpret_cast<float2*>(st + St::GL)[1] = make_float2(ordinary ? 1.f : 0.f, most);
    }
    {
      // V's columns: a lane's piece of every RV-th row, then its like among the lanes
      using V2 = std::conditional_t<kBf16<T>, __nv_bfloat162, __half2>;
      uint4 big = make_uint4(0, 0, 0, 0);
      V2* b2 = reinterpret_cast<V2*>(&big);
#pragma unroll
      for (int i = 0; i < CH / RV; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(st + St::V + piece<2 * ROWS>(i * RV + rv, xv));
#pragma unroll
        for (int j = 0; j < 4; ++j) b2[j] = __hmax2_nan(b2[j], __habs2(reinterpret_cast<const V2*>(&x)[j]));
      }
#pragma unroll
      for (int o = PV; o < 32; o <<= 1)
#pragma unroll
        for (int j = 0; j < 4; ++j) b2[j] = __hmax2_nan(b2[j], __shfl_xor_sync(0xffffffffu, b2[j], o));
      if (rv == 0) reinterpret_cast<uint4*>(st + St::VM)[xv] = big;
    }
    // M, and the units of its rows: bf16, those of the query, whose row the chain's products take in fp16 too;
    // fp16, from M's own largest entry
    float mm[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // (pd is 0 above the diagonal, but 0 times an infinite product would not be)
        const int s = 8 * i + 2 * cq + e;
        mm[i][e] = s <= gr ? pd[i][e] * qk[i][e] : 0.f;
        mm[i][2 + e] = s <= gr + 8 ? pd[i][2 + e] * qk[i][2 + e] : 0.f;
      }
    float ez = expf(gam + gaml), m0, m1;  // the factors that take M's rows to their units
    if constexpr (kBf16<T>) {
      __syncwarp();
      const Scale sq = rows_to_f16<D>(st + St::Q, lane);
      m0 = __shfl_sync(0xffffffffu, sq.down, 2 * gr);
      m1 = __shfl_sync(0xffffffffu, sq.down, 2 * gr + 16);
      const float up = __shfl_sync(0xffffffffu, sq.up, 2 * (lane & 15));
      if (lane < CH) reinterpret_cast<float*>(st + St::MU)[lane] = up;
      ez *= up;
    } else {
      float b0 = 0.f, b1 = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        b0 = fmaxf(b0, fmaxf(fabsf(mm[i][0]), fabsf(mm[i][1])));
        b1 = fmaxf(b1, fmaxf(fabsf(mm[i][2]), fabsf(mm[i][3])));
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        b0 = fmaxf(b0, __shfl_xor_sync(0xffffffffu, b0, o));
        b1 = fmaxf(b1, __shfl_xor_sync(0xffffffffu, b1, o));
      }
      const Scale s0(b0), s1(b1);
      m0 = s0.down;
      m1 = s1.down;
      if (cq == 0) {
        reinterpret_cast<float*>(st + St::MU)[gr] = s0.up;
        reinterpret_cast<float*>(st + St::MU)[gr + 8] = s1.up;
      }
    }
    if (lane < CH) reinterpret_cast<float*>(st + St::EZ)[lane] = ez;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int s = 8 * i + 2 * cq;
      const float b0 = __shfl_sync(0xffffffffu, bt, s), b1 = __shfl_sync(0xffffffffu, bt, s + 1);
      *reinterpret_cast<float2*>(Ls + gr * Prep::LDL + s) =
          make_float2(s < gr ? b0 * pd[i][0] * kk[i][0] : 0.f, s + 1 < gr ? b1 * pd[i][1] * kk[i][1] : 0.f);
      *reinterpret_cast<float2*>(Ls + (gr + 8) * Prep::LDL + s) =
          make_float2(s < gr + 8 ? b0 * pd[i][2] * kk[i][2] : 0.f, s + 1 < gr + 8 ? b1 * pd[i][3] * kk[i][3] : 0.f);
      uint32_t hi, lo;
      split2(mm[i][0] * m0, mm[i][1] * m0, hi, lo);
      *reinterpret_cast<uint32_t*>(st + St::MH + piece16(gr, i) + 4 * cq) = hi;
      *reinterpret_cast<uint32_t*>(st + St::ML + piece16(gr, i) + 4 * cq) = lo;
      split2(mm[i][2] * m1, mm[i][3] * m1, hi, lo);
      *reinterpret_cast<uint32_t*>(st + St::MH + piece16(gr + 8, i) + 4 * cq) = hi;
      *reinterpret_cast<uint32_t*>(st + St::ML + piece16(gr + 8, i) + 4 * cq) = lo;
    }
    __syncwarp();
    // (I + L)^-1 in fp32, row r = lane: x (I + L) = e_r from the last column down (x_s is final
    // when reached and leaves every earlier column)
    if (lane < CH) {
      float x[CH];
#pragma unroll
      for (int s = 0; s < CH; ++s) x[s] = s == lane ? 1.f : 0.f;
#pragma unroll
      for (int s = CH - 1; s >= 1; --s) {
        float l[CH];
#pragma unroll
        for (int i = 0; i < s; i += 4) {
          const float4 f = *reinterpret_cast<const float4*>(Ls + s * Prep::LDL + i);
          l[i] = f.x;
          l[i + 1] = f.y;
          l[i + 2] = f.z;
          l[i + 3] = f.w;
        }
#pragma unroll
        for (int i = 0; i < s; ++i) x[i] = fmaf(-x[s], l[i], x[i]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          split2(0x1p10f * x[8 * i + 2 * j], 0x1p10f * x[8 * i + 2 * j + 1], hi[j], lo[j]);
        *reinterpret_cast<uint4*>(st + St::TH + piece16(lane, i)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(st + St::TL + piece16(lane, i)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
    if constexpr (kBf16<T>) {  // the chain's products take K in fp16 too: exact but for what is below 2^-17
#pragma unroll 2
      for (int i = lane; i < CH * D / 8; i += 32) {
        uint4* k8 = reinterpret_cast<uint4*>(st + St::K) + i;
        uint4 x = *k8;
        uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = F16<T>::unpack(w[j]);
          w[j] = pack_f16(f.x, f.y);
        }
        *k8 = x;
      }
    }
    __syncwarp();
    if (lane == 0 && c + 1 != p.stall_run1) mbar_arrive(&full[c % NST]);
  }
  cp_async_wait<0>();
}

// n tokens from t0 on, one after the other in fp32, for the rows of a chain warp: a run that fp16 terms in one
// unit cannot hold.  `state`: a lane's fragments of S in true size; `row`: its first row of the head.  (Out of
// line, as between the runs' steps its instructions cost them 1 to 2 %: 16 sequences 814 against 799 us.)  A run
// takes about ten times as long this way: a sequence of 1024 tokens 0.93 ms, eight 3.6 ms.
template <typename T, int D>
__device__ __noinline__ void step_tokens(const GdnFwd& p, float* state, int h, int row, int seq, int t0, int n,
                                         int lane) {
  float S[D / 8][4];
#pragma unroll
  for (int j = 0; j < D / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) S[j][e] = state[4 * j + e];
  const int cq = lane & 3, kh = h / (p.n_v / p.n_k);
  const T* k = static_cast<const T*>(p.k) + seq * p.k_seq + t0 * p.k_ld + kh * D + 2 * cq;
  const T* q = static_cast<const T*>(p.q) + seq * p.q_seq + t0 * p.q_ld + kh * D + 2 * cq;
  const T* v = static_cast<const T*>(p.v) + seq * p.v_seq + t0 * p.v_ld + h * D + row;
  T* out = static_cast<T*>(p.out) + seq * p.out_seq + t0 * p.out_ld + h * D + row;
  const float* g = p.gb + (static_cast<int64_t>(seq) * 2 * p.n_v + h) * p.T + t0;
  for (int t = 0; t < n; ++t) {
    const float dec = expf(g[t]), beta = g[static_cast<int64_t>(p.n_v) * p.T + t];
    uint32_t kk[D / 8];
    float2 a0 = make_float2(0.f, 0.f), a1 = a0;
#pragma unroll
    for (int j = 0; j < D / 8; ++j) kk[j] = *reinterpret_cast<const uint32_t*>(k + 8 * j);
    scale_all(S, make_float2(dec, dec));
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
      const float2 f = F16<T>::unpack(kk[j]);
      a0 = fma2(make_float2(S[j][0], S[j][1]), f, a0);
      a1 = fma2(make_float2(S[j][2], S[j][3]), f, a1);
    }
    const float u0 = beta * (F16<T>::to(v[0]) - sum4(a0.x + a0.y));
    const float u1 = beta * (F16<T>::to(v[8]) - sum4(a1.x + a1.y));
    a0 = a1 = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
      const float2 f = F16<T>::unpack(kk[j]), qf = F16<T>::unpack(*reinterpret_cast<const uint32_t*>(q + 8 * j));
      const float2 s0 = fma2(make_float2(u0, u0), f, make_float2(S[j][0], S[j][1]));
      const float2 s1 = fma2(make_float2(u1, u1), f, make_float2(S[j][2], S[j][3]));
      a0 = fma2(s0, qf, a0);
      a1 = fma2(s1, qf, a1);
      S[j][0] = s0.x;
      S[j][1] = s0.y;
      S[j][2] = s1.x;
      S[j][3] = s1.y;
    }
    const float o0 = sum4(a0.x + a0.y), o1 = sum4(a1.x + a1.y);
    if (cq == 0) {
      out[0] = F16<T>::from(p.scale * o0);
      out[8] = F16<T>::from(p.scale * o1);
    }
    k += p.k_ld;
    q += p.q_ld;
    v += p.v_ld;
    out += p.out_ld;
  }
#pragma unroll
  for (int j = 0; j < D / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) state[4 * j + e] = S[j][e];
}

template <typename T, int D, int ROWS, int PREP>
__device__ void chain_runs(const GdnFwd& p, uint8_t* sm, int h, int half, int seq, int len, int warp, int lane,
                           volatile int* abort_flag) {
  using St = Stage<D, ROWS>;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + Chunk<D, ROWS, PREP>::BAR);
  uint64_t* empty = full + NST;
  const int n_runs = (len + CH - 1) / CH;
  const int mi = lane >> 3, lr = lane & 7, gr = lane >> 2, cq = lane & 3;
  const uint32_t base = smem_u32(sm);
  const int64_t srow = ((static_cast<int64_t>(seq) * p.n_v + h) * D + half * ROWS + warp * 16 + gr) * D + 2 * cq;
  float S[D / 8][4];
#pragma unroll
  for (int j = 0; j < D / 8; ++j) {
    const float2 a = *reinterpret_cast<const float2*>(p.state_in + srow + 8 * j);
    const float2 c = *reinterpret_cast<const float2*>(p.state_in + srow + 8 * D + 8 * j);
    S[j][0] = a.x;
    S[j][1] = a.y;
    S[j][2] = c.x;
    S[j][3] = c.y;
  }
  T* out = static_cast<T*>(p.out) + seq * p.out_seq + h * D + half * ROWS + warp * 16 + 2 * cq;
  // S is held in units of `up`; `norm` bounds the norm of a row.  (Of the lane's two rows.)
  const float root = D == 128 ? 11.32f : 8.f;  // sqrt(D): a row's norm is at most that times its largest entry
  float2 norm, up;
  auto measure = [&]() {  // S in true size
    const float2 m = largest_of_rows(S);
    norm = make_float2(fminf(root * m.x, kMost), fminf(root * m.y, kMost));
    const Scale s0(norm.x), s1(norm.y);
    up = make_float2(s0.up, s1.up);
    scale_all(S, make_float2(s0.down, s1.down));
  };
  if (n_runs) measure();
  else norm = up = make_float2(1.f, 1.f);  // (no tokens: the state goes out as it came)

  int c = 0;
  while (true) {
    for (; c < n_runs; ++c) {
      if (!mbar_wait_warp(&full[c % NST], (c / NST) & 1, abort_flag)) {
        *abort_flag = 1;
        set_device_error(p.err, KVA_DEV_WAIT_TIMEOUT);
        return;  // (the state at hand is of no token that the caller knows: state_out stays as it was)
      }
      const uint8_t* st = sm + (c % NST) * St::BYTES;
      const uint32_t sst = base + (c % NST) * St::BYTES;
      const float4 gv = *reinterpret_cast<const float4*>(st + St::GL);
      // Y = S K^T, Z = S Q^T, both terms of S
      float y[2][4] = {}, z[2][4] = {};
      uint32_t kf[2][4], qf[2][4];
      ldmatrix_x4(kf[0], sst + St::K + piece<2 * D>((mi & 1) * 8 + lr, mi >> 1));
      ldmatrix_x4(qf[0], sst + St::Q + piece<2 * D>((mi & 1) * 8 + lr, mi >> 1));
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        if (ks + 1 < D / 16) {
          ldmatrix_x4(kf[(ks + 1) & 1], sst + St::K + piece<2 * D>((mi & 1) * 8 + lr, 2 * ks + 2 + (mi >> 1)));
          ldmatrix_x4(qf[(ks + 1) & 1], sst + St::Q + piece<2 * D>((mi & 1) * 8 + lr, 2 * ks + 2 + (mi >> 1)));
        }
        uint32_t ah[4], al[4];
        split_a(S[2 * ks], S[2 * ks + 1], ah, al);
        mma2(y[0], y[1], ah, kf[ks & 1], 0, 2, 1, 3);
        mma2(y[0], y[1], al, kf[ks & 1], 0, 2, 1, 3);
        mma2(z[0], z[1], ah, qf[ks & 1], 0, 2, 1, 3);
        mma2(z[0], z[1], al, qf[ks & 1], 0, 2, 1, 3);
      }
      // Units for the run, from its values and the state's rows as its tokens meet them.  (The test comes after
      // the products, which hide what it waits for: fp16, 8 sequences, 385 against 392 us with it before them; bf16
      // 400 against 394.)
      const T* vm = reinterpret_cast<const T*>(st + St::VM) + warp * 16 + gr;
      const float2 mv = make_float2(F16<T>::to(vm[0]), F16<T>::to(vm[8]));
      const float most = fmaxf(gv.w, 0x1p-100f);  // (a smaller beta is written with fewer bits)
      const float2 bm = make_float2(most * mv.x, most * mv.y);
      const float2 met = make_float2(gv.y * norm.x, gv.y * norm.y), left = make_float2(gv.x * norm.x, gv.x * norm.y);
      const bool fits = gv.z != 0.f && mv.x <= kMost && mv.y <= kMost && met.x <= kFar * fmaxf(bm.x, left.x) &&
                        met.y <= kFar * fmaxf(bm.y, left.y);
      if (!__all_sync(0xffffffffu, fits)) break;
      // W = V^T - Y diag(e^gam)
      uint32_t vf[4], wh[4], wl[4];
      ldmatrix_x4_trans(vf, sst + St::V + piece<2 * ROWS>((mi >> 1) * 8 + lr, 2 * warp + (mi & 1)));
      const Scale now0(fmaxf(bm.x, met.x)), now1(fmaxf(bm.y, met.y));  // of S and U
      const Scale w0(fmaxf(mv.x, met.x)), w1(fmaxf(mv.y, met.y));      // of W
      const float2 into = make_float2(w0.up * now0.down, w1.up * now1.down);  // from these to those, at most 2^101
      // S into the run's units: what stays is below 18 x 2^8, but the units alone may be 2^250 apart, with nothing
      // left of S
      const float2 decay = make_float2(fminf(gv.x * up.x * now0.down, kMost), fminf(gv.x * up.y * now1.down, kMost));
      // S <- e^g S (I - beta k k^T) + beta v k^T, 16 times
      norm = make_float2(fminf(fmaf(16.25f, bm.x, left.x), kMost), fminf(fmaf(16.25f, bm.y, left.y), kMost));
      float w[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 e = *reinterpret_cast<const float2*>(st + St::EG + (8 * i + 2 * cq) * 4);
        const float2 ez = *reinterpret_cast<const float2*>(st + St::EZ + (8 * i + 2 * cq) * 4);
        const float2 e0 = mul2(e, make_float2(up.x, up.x)), e1 = mul2(e, make_float2(up.y, up.y));
        const float2 z0 = mul2(ez, make_float2(up.x, up.x)), z1 = mul2(ez, make_float2(up.y, up.y));
        const float2 v0 = F16<T>::unpack(vf[2 * i]), v1 = F16<T>::unpack(vf[2 * i + 1]);
        w[i][0] = v0.x - e0.x * y[i][0];
        w[i][1] = v0.y - e0.y * y[i][1];
        w[i][2] = v1.x - e1.x * y[i][2];
        w[i][3] = v1.y - e1.y * y[i][3];
        z[i][0] *= z0.x;
        z[i][1] *= z0.y;
        z[i][2] *= z1.x;
        z[i][3] *= z1.y;
      }
      scale_all(w, make_float2(w0.down, w1.down));
      up = make_float2(now0.up, now1.up);
      split_a(w[0], w[1], wh, wl);
      // U = W Tm^T diag(beta), from W's units to S's
      float u[2][4] = {};
      {
        uint32_t th[4], tl[4];
        ldmatrix_x4(th, sst + St::TH + piece16((mi & 1) * 8 + lr, mi >> 1));
        ldmatrix_x4(tl, sst + St::TL + piece16((mi & 1) * 8 + lr, mi >> 1));
        mma2(u[0], u[1], wh, th, 0, 2, 1, 3);
        mma2(u[0], u[1], wl, th, 0, 2, 1, 3);
        mma2(u[0], u[1], wh, tl, 0, 2, 1, 3);
      }
      uint32_t uh[4], uo[4], dh[4], dl[4];
      {
        float dd[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 e = *reinterpret_cast<const float2*>(st + St::DEC + (8 * i + 2 * cq) * 4);
          const float2 b = *reinterpret_cast<const float2*>(st + St::BT + (8 * i + 2 * cq) * 4);
          const float2 b0 = mul2(b, make_float2(into.x, into.x)), b1 = mul2(b, make_float2(into.y, into.y));
          u[i][0] *= b0.x;
          u[i][1] *= b0.y;
          u[i][2] *= b1.x;
          u[i][3] *= b1.y;
          dd[i][0] = u[i][0] * e.x;
          dd[i][1] = u[i][1] * e.y;
          dd[i][2] = u[i][2] * e.x;
          dd[i][3] = u[i][3] * e.y;
        }
        split_a(dd[0], dd[1], dh, dl);
        split_a(u[0], u[1], uh, uo);
      }
      // S <- e^gam_last S + U diag(dec) K
      scale_all(S, decay);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t kt[4];
        ldmatrix_x4_trans(kt, sst + St::K + piece<2 * D>((mi & 1) * 8 + lr, 2 * ks + (mi >> 1)));
        mma2(S[2 * ks], S[2 * ks + 1], dh, kt, 0, 1, 2, 3);
        mma2(S[2 * ks], S[2 * ks + 1], dl, kt, 0, 1, 2, 3);
      }
      if ((c & 7) == 7) {
        const float2 m = largest_of_rows(S);
        norm = make_float2(fminf(norm.x, root * up.x * m.x), fminf(norm.y, root * up.y * m.y));
      }
      // O = Z diag(e^gam) + U M^T, written token-major
      {
        uint32_t mh[4], ml[4];
        float o[2][4] = {};
        ldmatrix_x4(mh, sst + St::MH + piece16((mi & 1) * 8 + lr, mi >> 1));
        ldmatrix_x4(ml, sst + St::ML + piece16((mi & 1) * 8 + lr, mi >> 1));
        mma2(o[0], o[1], uh, mh, 0, 2, 1, 3);
        mma2(o[0], o[1], uo, mh, 0, 2, 1, 3);
        mma2(o[0], o[1], uh, ml, 0, 2, 1, 3);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 mu = *reinterpret_cast<const float2*>(st + St::MU + (8 * i + 2 * cq) * 4);
          const float2 mu0 = mul2(mu, make_float2(up.x, up.x)), mu1 = mul2(mu, make_float2(up.y, up.y));
          z[i][0] = fmaf(mu0.x, o[i][0], z[i][0]);
          z[i][1] = fmaf(mu0.y, o[i][1], z[i][1]);
          z[i][2] = fmaf(mu1.x, o[i][2], z[i][2]);
          z[i][3] = fmaf(mu1.y, o[i][3], z[i][3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[c % NST]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t o0 = movmatrix_trans(F16<T>::pack(p.scale * z[i][0], p.scale * z[i][1]));
        const uint32_t o1 = movmatrix_trans(F16<T>::pack(p.scale * z[i][2], p.scale * z[i][3]));
        const int64_t t = c * CH + 8 * i + gr;
        if (t < len) {
          *reinterpret_cast<uint32_t*>(out + t * p.out_ld) = o0;
          *reinterpret_cast<uint32_t*>(out + t * p.out_ld + 8) = o1;
        }
      }
    }
    if (c >= n_runs) break;
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[c % NST]);
    scale_all(S, up);
    float state[D / 2];
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) state[4 * j + e] = S[j][e];
    step_tokens<T, D>(p, state, h, half * ROWS + warp * 16 + gr, seq, c * CH, min(CH, len - c * CH), lane);
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[j][e] = state[4 * j + e];
    measure();
    ++c;
  }
  scale_all(S, up);
#pragma unroll
  for (int j = 0; j < D / 8; ++j) {
    *reinterpret_cast<float2*>(p.state_out + srow + 8 * j) = make_float2(S[j][0], S[j][1]);
    *reinterpret_cast<float2*>(p.state_out + srow + 8 * D + 8 * j) = make_float2(S[j][2], S[j][3]);
  }
}

// grid (n_v * D / ROWS, n_seq): ROWS state rows of one head, a chain warp for every 16 and PREP preparing ones
template <typename T, int D, int ROWS, int PREP, int BLOCKS>
__global__ void __launch_bounds__(32 * (ROWS / 16 + PREP), BLOCKS) gdn_chunk_kernel(const __grid_constant__ GdnFwd p) {
  extern __shared__ __align__(128) uint8_t sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Chunk<D, ROWS, PREP>::BAR);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + Chunk<D, ROWS, PREP>::MISC);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int HALVES = D / ROWS, CHAIN = ROWS / 16;
  const int h = blockIdx.x / HALVES, half = blockIdx.x % HALVES;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&bars[i], 1);
      mbar_init(&bars[NST + i], CHAIN);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  griddep_wait_and_release();
  const int seq = p.has_lens ? p.order[p.first + blockIdx.y] : blockIdx.y;
  const int len = p.has_lens ? p.lens[seq] : p.T;
  if (warp < CHAIN) chain_runs<T, D, ROWS, PREP>(p, sm, h, half, seq, len, warp, lane, abort_flag);
  else prepare_runs<T, D, ROWS, PREP>(p, sm, h, half, seq, len, warp - CHAIN, lane, abort_flag);
}

template <typename T, int D, int ROWS, int PREP, int BLOCKS>
cudaError_t launch_chunk(const GdnFwd& p, int n_seq, cudaStream_t s) {
  auto kern = gdn_chunk_kernel<T, D, ROWS, PREP, BLOCKS>;
  constexpr int bytes = Chunk<D, ROWS, PREP>::BYTES;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(p.n_v * (D / ROWS), n_seq), dim3(32 * (ROWS / 16 + PREP)), bytes, s, p);
}

template <typename T, int D>
cudaError_t launch_steps(const GdnFwd& p, int n_seq, cudaStream_t s) {
  // two rows a thread where that still leaves four blocks an SM (64 sequences, 8 tokens: 115 us against 139
  // with one row)
  if (static_cast<int64_t>(p.n_v) * (D / 64) * n_seq >= 4 * num_sms())
    return launch_pdl(gdn_recurrent_kernel<T, D, 2>, dim3(p.n_v * (D / 64), n_seq), dim3(256), 0, s, p);
  return launch_pdl(gdn_recurrent_kernel<T, D, 1>, dim3(p.n_v * (D / 32), n_seq), dim3(256), 0, s, p);
}
template <typename T, int D>
cudaError_t launch_runs(const GdnFwd& p, int n_seq, cudaStream_t s) {
  const int sms = num_sms();
  const int64_t blocks = static_cast<int64_t>(p.n_v) * (D / 64) * n_seq;  // of 64 state rows
  // A block that has its SM to itself takes a preparing warp on every scheduler (one sequence of 1024 tokens: fp16
  // 84 against 90 us, bf16 89 against 98).  With more work a head's 128 rows share one preparation (8 sequences:
  // fp16 385 against 407 us, bf16 400 against 442) but for a last round that fills less than half of the SMs: there
  // two blocks of 64 rows an SM end sooner (4 sequences: 240 against 267 us; 16: 799 against 794).
  if (blocks <= sms) return launch_chunk<T, D, 64, 4, 1>(p, n_seq, s);
  if constexpr (D == 128) {
    const int64_t last = blocks / 2 % sms;
    if (last == 0 || 2 * last >= sms) return launch_chunk<T, D, 128, 4, 1>(p, n_seq, s);
  }
  return launch_chunk<T, D, 64, 2, 2>(p, n_seq, s);
}
// A sequence goes by its own length, whatever the others': the first n_long of the order in runs, the n_short
// behind them token by token
template <typename T, int D>
cudaError_t launch(GdnFwd& p, int n_long, int n_short, cudaStream_t s) {
  p.first = 0;
  if (n_long > 0) {
    const cudaError_t e = launch_runs<T, D>(p, n_long, s);
    if (e != cudaSuccess || n_short == 0) return e;
    p.first = n_long;
  }
  return launch_steps<T, D>(p, n_short, s);
}

bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace kva

static int gdn_forward(const kva_gdn_forward_args* a, int32_t* err, void* stream, int stall_run1) {
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
  int n_long = a->T > kStepTokens ? a->n_seq : 0;
  if (a->lens) {
    n_long = 0;
    for (int i = 0; i < a->n_seq; ++i) {
      if (a->lens[i] < 0 || a->lens[i] > a->T) return KVA_ERR_INVALID_ARG;
      p.lens[i] = a->lens[i];
      p.order[i] = static_cast<uint8_t>(i);
      n_long += a->lens[i] > kStepTokens;
    }
    // the blocks of long sequences start first, so that the last ones to start are short (bf16, 16/48 heads:
    // 8 sequences of 1 to 1024 tokens 279 to 225 us, 16 of them 336 to 299, 32 of 1 to 512 505 to 482, 128 of 1 to 64
    // 426 to 411)
    if (n_long > 0)
      std::stable_sort(p.order, p.order + a->n_seq, [&](int x, int y) { return p.lens[x] > p.lens[y]; });
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
  p.stall_run1 = stall_run1;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f16 = a->dtype == KVA_F16;
  const cudaError_t r = a->d == 128
                            ? (f16 ? launch<__half, 128>(p, n_long, a->n_seq - n_long, s)
                                   : launch<__nv_bfloat16, 128>(p, n_long, a->n_seq - n_long, s))
                            : (f16 ? launch<__half, 64>(p, n_long, a->n_seq - n_long, s)
                                   : launch<__nv_bfloat16, 64>(p, n_long, a->n_seq - n_long, s));
  return r == cudaSuccess ? KVA_OK : KVA_ERR_CUDA;
}

extern "C" int kva_op_gdn_forward(const kva_gdn_forward_args* a, int32_t* err, void* stream) {
  return gdn_forward(a, err, stream, 0);
}

extern "C" int kva_test_gdn_forward_wait_timeout(const kva_gdn_forward_args* a, int32_t* err, void* stream) {
  if (!a || !err || a->T <= 32 || a->n_seq != 1 || a->lens) return KVA_ERR_INVALID_ARG;
  return gdn_forward(a, err, stream, 2);
}

// Dense products for blocks of tokens: Y = act(X WT + bias) + residual, the
// gate and up projections of a gated MLP with the activation and the product
// of the two in the epilogue, and the products of its backward pass.
//
//   dense_pair_kernel  persistent: CTA pairs walk tiles of 256 tokens x 256 (or
//                      128) columns with two accumulators in tensor memory, so
//                      the epilogue of a tile runs beside the mainloop of the
//                      next.  Bound by the tensor cores at the power limit: the
//                      weight gradients of 2048 tokens 4096/11008 bf16 in 357-375
//                      us on B200 (1.5 PFLOP/s, 0.9 of the measured burst rate; 85 %
//                      of the launch with the tensor pipe active at 1.52 GHz).  All
//                      weight gradients, and the shapes that its tiles fit better
//                      than the tall kernel's (shallow ones of many tokens).
//   dense_tall_kernel  persistent, with the weight as the MMA's M operand and the
//                      tokens as N: tiles of 256 columns x any multiple of 16
//                      tokens, the height chosen so that the tiles fill whole
//                      waves.  1300 x 4096 -> 11008 fp16 85 us (1.38 PFLOP/s; the
//                      tensor pipe active in 88 % of the SMs' active cycles).
//   dense_few_kernel   few tokens, bound by reading the weight: the weight is the
//                      MMA's M operand (128 of its columns, one a tensor-memory
//                      lane) and the tokens its N operand; one tile per cluster,
//                      whose CTAs each take a part of K and join their float32
//                      sums through distributed shared memory in a fixed order:
//                      no workspace, no atomics, the same bits in every run.
//                      16 tokens 4096 -> 11008: 18.4 us, 4.9 TB/s of weight
//                      (0.75 of the measured copy rate); 1 token 4096 -> 4096
//                      8.7 us, of which 5.1 are the weight at that rate.
#include "common.cuh"
#include "dense.h"
#include "internal.h"
#include "tc.cuh"

#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "../../include/sig.h"

namespace sig {

__device__ unsigned g_dense_error = 0u;
constexpr long long kDenseTimeout = 4000000000ll;   // ~2 s at 1.9 GHz
__device__ long long g_dense_wait_limit = kDenseTimeout;

namespace {

constexpr int kTile = 128;      // rows of one CTA's tile
constexpr int kSlab = 64;       // K of one stage: a 128-byte swizzle row of 16-bit values
constexpr uint32_t kBlock = kSlab * 128;   // 64 rows of 128 bytes

struct DenseMaps {
  CUtensorMap a[2], b[3], o[3], r[2];   // r: the residual, or g and u
};

struct DenseArgs {
  int rows, cols;      // rows (tokens) and columns of one output
  int kb0, kbt;        // K stages of the first segment, of both
  int tm, tn;          // tiles down, and across one weight
  int rows2, cols2, tm2, tn2;   // pair kernel: the second product of the launch (weight 2), if any
  int whole, items;    // pair kernel: tiles taken whole, and all items of the walk
  int group;           // tall kernel: token tiles walked together
  int mats;            // pair kernel: weights side by side
  int outs;            // outputs to store (DENSE_GATED: 1, or 3 with g and u)
  int act;
  bool plain;          // DENSE_LINEAR: no bias, activation or residual
  const uint16_t* bias;
  const uint16_t* residual;
  int64_t ldr;
  const uint16_t *g, *u;
  uint16_t* o[3];
  int64_t ldo;
};

// ---------------------------------------------------------------------------
// Waits (bounded, see nm_gemm.cu)
// ---------------------------------------------------------------------------
__device__ __forceinline__ bool try_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// The limit of this launch's waits, read once: a load in every wait that does
// not succeed at once would add its latency to the stage.
__device__ __forceinline__ long long wait_limit() { return *(volatile long long*)&g_dense_wait_limit; }

// The same without the hardware's own suspension, which may outlast a short limit.
__device__ __forceinline__ bool poll_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

constexpr long long kShortLimit = 1 << 20;   // cycles: shorter limits are polled

__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                             long long limit) {
  if (poll_cluster(bar, parity)) return true;
  const long long t0 = clock64();
  while (!(limit < kShortLimit ? poll_cluster(bar, parity) : try_cluster(bar, parity))) {
    if (*abort_flag) return false;
    if (clock64() - t0 > limit) {
      *abort_flag = 1;
      atomicOr(&g_dense_error, 1u);
      return false;
    }
  }
  return true;
}

// Not cut short by a give-up: lets issued copies and MMAs finish, so its limit is the
// default whatever the launch's is.
__device__ __forceinline__ bool wait_drain(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!try_cluster(bar, parity))
    if (clock64() - t0 > kDenseTimeout) return false;
  return true;
}

// The few-token kernel's wait for its sums, whose barrier completes once every issued
// MMA has finished, also when another wait has given up: tensor memory is kept until
// then.  It covers all stages of the part, so a limit for the waits of a single stage is
// too short for it: it lasts for the launch's limit rounded up to whole default limits,
// and has given up after that too.
__device__ __forceinline__ bool wait_sums(uint32_t bar, long long limit) {
  long long waited = 0;
  while (!wait_drain(bar, 0u))
    if ((waited += kDenseTimeout) >= limit) {
      atomicOr(&g_dense_error, 1u);
      return false;
    }
  return true;
}

// Hands an accumulator back: the tensor-memory loads are done and fenced, and no
// other memory is passed on, so the arrive needs no release, which waits for the
// warp's earlier stores (22016 x 4096 outputs of depth 16: 59.4 us with one, 39.1
// without).
__device__ __forceinline__ void arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

// Bring a tensor map (a kernel argument) into the descriptor cache.
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// ---------------------------------------------------------------------------
// Descriptors
// ---------------------------------------------------------------------------
// kind::f16, float32 accumulator; A and B both fp16 or both bf16, each K-major
// (K contiguous) or MN-major.
__host__ __device__ constexpr uint32_t dense_idesc(int M, int N, bool bf16, bool a_mn, bool b_k) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_k ? 0u : 1u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Shared-memory descriptor of an operand slab, in its two words (see
// smem_desc): the low one holds the address and the leading offset, the high
// one is constant.  K-major: rows of 128 bytes; MN-major: blocks of 64 columns
// x 64 k-rows, kBlock bytes apart.  A K step of 16 values is 32 bytes into the
// rows, or 16 k-rows down: slab_step in the address's 16-byte units.  The
// issuing thread only adds to the low word; building each descriptor in full
// took longer than the MMAs of the stage: 0.30 against 0.19 us a stage of 128
// columns at 256 x 8192 x 256 on B200.
template <bool MN>
__device__ __forceinline__ uint32_t slab_low(uint32_t addr) {
  // the address within the CTA: a cluster rank sits above it in the shared window
  return ((addr >> 4) & 0x3fffu) | ((MN ? kBlock >> 4 : 1u) << 16);
}
constexpr uint32_t kSlabHigh = (1024u >> 4) | (1u << 14) | (2u << 29);   // 8-row groups, version, swizzle
template <bool MN>
constexpr uint32_t slab_step = MN ? 2048u >> 4 : 32u >> 4;

__device__ __forceinline__ uint64_t slab_desc(uint32_t low) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(low), "r"(kSlabHigh));
  return d;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

template <int GROUP>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if constexpr (GROUP == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void commit_one(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}

// Start the load of 32 accumulator columns of this warp's 32 rows (one row a
// lane); the values are there after tmem_wait32.
__device__ __forceinline__ void tmem_start32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}

// Wait for the loads so far.  The registers pass through the wait, so that no
// use of them can move above it.
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                 "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]),
                 "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),
                 "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

__device__ __forceinline__ void as_floats(float (&v)[32], const uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// ---------------------------------------------------------------------------
// Epilogue arithmetic, float32 throughout
// ---------------------------------------------------------------------------
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (BF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <bool BF>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (BF)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

template <bool BF>
__device__ __forceinline__ void unpack8(float (&f)[8], const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = unpack2<BF>(w[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

template <bool BF>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2<BF>(f[0], f[1]), pack2<BF>(f[2], f[3]), pack2<BF>(f[4], f[5]),
                    pack2<BF>(f[6], f[7]));
}

// Phi(-x) exp(x^2 / 2) = t P(t), t = 1 / (1 + p x): P of degree 7, fitted by weighted
// least squares (Lawson's iteration) to the smallest largest relative error over
// 0 <= x <= 14, 1.1e-7 with these float32 coefficients.
constexpr float kTailP = 0.304f;
constexpr float kTailA[8] = {0.121236868f, 0.122136548f, 0.102640741f, 0.122816235f,
                             -0.0417008735f, 0.19059512f, -0.154348761f, 0.036624115f};
constexpr float kHalfLog2E = 0.72134752044448170f;   // log2(e) / 2
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kGeluC = 0.79788456080286536f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// 1 / (1 + exp(-v)) with the hardware's exponential and reciprocal: a relative
// error of about (3 + 1.2 |v|) 2^-23, and 0 where exp(-v) passes 2^126 (with
// the IEEE division 2048 x 1024 -> 2816 took 25.0 us with SiLU, now 15.1).
__device__ __forceinline__ float logistic(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// 1 / v for v >= 1, and exp(-z^2 / 2) as a power of two: the hardware's instructions
// without the steps for subnormal values, which the first has none of and the second
// gives as 0 (beyond |z| = 13.2).
__device__ __forceinline__ float reciprocal(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float bell(float z) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(z * (-kHalfLog2E * z)));
  return r;
}

// The normal distribution function.  Its lower tail has a small relative error, about
// (16 + z^2) 2^-23, which an error that is small against one (such as the five
// coefficients of Abramowitz and Stegun's 7.1.26, used before: 1.5e-7) is not: that is
// past half a step of bf16 below z = -6.2.  Its three more multiply-adds cost less than
// the two plain instructions save: 2048 x 1024 -> 2816 with GELU and residual 17.7 us,
// 18.9 with __fdividef and __expf, 18.5 with the five coefficients and these.  The
// exponential is the one that the slope of GELU needs too.
__device__ __forceinline__ float normal_cdf(float z) {
  const float t = reciprocal(fmaf(kTailP, fabsf(z), 1.f));
  const float high = fmaf(t, fmaf(t, fmaf(t, kTailA[7], kTailA[6]), kTailA[5]), kTailA[4]);
  const float poly = fmaf(t, fmaf(t, fmaf(t, fmaf(t, high, kTailA[3]), kTailA[2]), kTailA[1]), kTailA[0]);
  const float tail = t * poly * bell(z);
  return z >= 0.f ? 1.f - tail : tail;
}

// act(z) = z p(z); p is the share that passes (1, [z > 0], the logistic
// function, the normal distribution function, or the logistic of the tanh
// form: (1 + tanh v) / 2 = 1 / (1 + exp(-2 v))).
template <int ACT>
__device__ __forceinline__ float act_share(float z) {
  if constexpr (ACT == SIG_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  if constexpr (ACT == SIG_ACT_SILU) return logistic(z);
  if constexpr (ACT == SIG_ACT_GELU) return normal_cdf(z);
  if constexpr (ACT == SIG_ACT_GELU_TANH)
    return logistic(2.f * kGeluC * z * fmaf(kGeluA * z, z, 1.f));
  return 1.f;
}

// act(z), given p = act_share(z)
template <int ACT>
__device__ __forceinline__ float act_value(float z, float p) {
  if constexpr (ACT == SIG_ACT_NONE) return z;
  if constexpr (ACT == SIG_ACT_RELU) return z < 0.f ? 0.f : z;   // NaN stays, -inf gives 0
  return z * p;
}

// d act / dz, given p = act_share(z)
template <int ACT>
__device__ __forceinline__ float act_slope(float z, float p) {
  if constexpr (ACT == SIG_ACT_SILU) return p * fmaf(z, 1.f - p, 1.f);
  if constexpr (ACT == SIG_ACT_GELU) return fmaf(z * kInvSqrt2Pi, bell(z), p);
  if constexpr (ACT == SIG_ACT_GELU_TANH)   // beyond |z| = 20 p is 0 or 1 (and z^2 may overflow)
    return fabsf(z) > 20.f ? p : fmaf(z * p * (1.f - p), 2.f * kGeluC * fmaf(3.f * kGeluA * z, z, 1.f), p);
  return p;   // none, relu
}

// f(ACT) for the run-time activation, the branch outside the column loops
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case SIG_ACT_RELU: f(std::integral_constant<int, SIG_ACT_RELU>{}); break;
    case SIG_ACT_GELU: f(std::integral_constant<int, SIG_ACT_GELU>{}); break;
    case SIG_ACT_GELU_TANH: f(std::integral_constant<int, SIG_ACT_GELU_TANH>{}); break;
    case SIG_ACT_SILU: f(std::integral_constant<int, SIG_ACT_SILU>{}); break;
    default: f(std::integral_constant<int, SIG_ACT_NONE>{}); break;
  }
}

__device__ __forceinline__ uint4 ld16(const uint16_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// v[0 .. 8 G) = act(v + bias) for 8 G columns from `col` (columns from `cols` on
// are left without the bias)
template <bool BF, int G>
__device__ __forceinline__ void epi_bias_act(float* v, const DenseArgs& a, int col) {
  if (a.bias != nullptr) {
#pragma unroll
    for (int j = 0; j < G; ++j)
      if (col + 8 * j < a.cols) {
        float b[8];
        unpack8<BF>(b, ld16(a.bias + col + 8 * j));
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * j + i] += b[i];
      }
  }
  if (a.act != SIG_ACT_NONE)
    with_act(a.act, [&](auto A) {
#pragma unroll
      for (int i = 0; i < 8 * G; ++i)
        v[i] = act_value<decltype(A)::value>(v[i], act_share<decltype(A)::value>(v[i]));
    });
}

// g <- act(g) u over n columns
template <int n>
__device__ __forceinline__ void epi_gated(float* g, const float* u, int act) {
  with_act(act, [&](auto A) {
#pragma unroll
    for (int i = 0; i < n; ++i) g[i] = act_value<decltype(A)::value>(g[i], act_share<decltype(A)::value>(g[i])) * u[i];
  });
}

// dh -> (dg, du, h)
template <int ACT>
__device__ __forceinline__ void gate_grad(float dh, float g, float u, float& dg, float& du, float& h) {
  const float p = act_share<ACT>(g), v = act_value<ACT>(g, p);
  dg = dh * u * act_slope<ACT>(g, p);
  du = dh * v;
  h = v * u;
}

// the same over 8 columns
template <bool BF>
__device__ __forceinline__ void epi_grad8(const float* dh, const uint4& gv, const uint4& uv, int act,
                                          uint4& dg, uint4& du, uint4& h) {
  float g[8], u[8], a0[8], a1[8], a2[8];
  unpack8<BF>(g, gv);
  unpack8<BF>(u, uv);
  with_act(act, [&](auto A) {
#pragma unroll
    for (int i = 0; i < 8; ++i) gate_grad<decltype(A)::value>(dh[i], g[i], u[i], a0[i], a1[i], a2[i]);
  });
  dg = pack8<BF>(a0);
  du = pack8<BF>(a1);
  h = pack8<BF>(a2);
}

// What the few-token epilogue of 4 columns of a token reads besides the sums:
// the residual, or g and u.  Loaded ahead of the sums.
struct Extra {
  uint2 x, y;
};

template <int EPI>
__device__ __forceinline__ Extra load_extra(const DenseArgs& a, int row, int col) {
  Extra e = {make_uint2(0, 0), make_uint2(0, 0)};
  if constexpr (EPI == DENSE_LINEAR) {
    if (a.residual != nullptr)   // a plain load: Y may be the residual buffer itself
      e.x = *reinterpret_cast<const uint2*>(a.residual + (int64_t)row * a.ldr + col);
  } else if constexpr (EPI == DENSE_GRAD) {
    const int64_t at = (int64_t)row * a.cols + col;
    e.x = __ldg(reinterpret_cast<const uint2*>(a.g + at));
    e.y = __ldg(reinterpret_cast<const uint2*>(a.u + at));
  }
  return e;
}

__device__ __forceinline__ void prefetch_l2(const uint16_t* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

template <bool BF>
__device__ __forceinline__ float4 unpack4(const uint2& v) {
  const float2 a = unpack2<BF>(v.x), b = unpack2<BF>(v.y);
  return make_float4(a.x, a.y, b.x, b.y);
}

template <bool BF>
__device__ __forceinline__ uint2 pack4(const float4& v) {
  return make_uint2(pack2<BF>(v.x, v.y), pack2<BF>(v.z, v.w));
}

__device__ __forceinline__ float4 add4(const float4& a, const float4& b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

template <int ACT>
__device__ __forceinline__ float4 act4(const float4& z) {
  return make_float4(act_value<ACT>(z.x, act_share<ACT>(z.x)), act_value<ACT>(z.y, act_share<ACT>(z.y)),
                     act_value<ACT>(z.z, act_share<ACT>(z.z)), act_value<ACT>(z.w, act_share<ACT>(z.w)));
}

// The outputs of 4 columns of a token from its float32 sums v (DENSE_GATED: g
// in v and u in w, which are outputs 1 and 2).
template <int EPI, bool BF, int ACT>
__device__ __forceinline__ void finish4(const float4& v, const float4& w, const float4& bias, const Extra& e,
                                        uint2& o0, uint2& o1, uint2& o2) {
  if constexpr (EPI == DENSE_LINEAR) {
    o0 = pack4<BF>(add4(act4<ACT>(add4(v, bias)), unpack4<BF>(e.x)));
  } else if constexpr (EPI == DENSE_GATED) {
    const float4 h = act4<ACT>(v);
    o0 = pack4<BF>(make_float4(h.x * w.x, h.y * w.y, h.z * w.z, h.w * w.w));
    o1 = pack4<BF>(v);
    o2 = pack4<BF>(w);
  } else {
    const float4 g = unpack4<BF>(e.x), u = unpack4<BF>(e.y);
    float4 dg, du, h;
    gate_grad<ACT>(v.x, g.x, u.x, dg.x, du.x, h.x);
    gate_grad<ACT>(v.y, g.y, u.y, dg.y, du.y, h.y);
    gate_grad<ACT>(v.z, g.z, u.z, dg.z, du.z, h.z);
    gate_grad<ACT>(v.w, g.w, u.w, dg.w, du.w, h.w);
    o0 = pack4<BF>(dg);
    o1 = pack4<BF>(du);
    o2 = pack4<BF>(h);
  }
}

// The same for 16 columns (tokens)
__device__ __forceinline__ void tmem_start16(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}

__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                 "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void st_cluster_u8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void sts_b32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ float4 lds_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

// The join of `parts` CTAs that split K.  Part j joins tokens [j own, (j + 1)
// own) of the tile.  join_send: eight warps send this CTA's sums of every
// token to the part that joins it, at [part][token - j own][128 columns] of its
// buffer, beginning with the part after this one so that the parts do not all
// send to the same.  A warp's 32 lanes write 128 contiguous bytes, the two
// warps of a lane quarter take groups of 16 tokens in turn.  One lane a token
// works out where it goes, so that the stores follow one another without a
// branch: with the owner found token by token in every lane they took 4 us at
// 256 tokens, now 1.3.
__device__ __forceinline__ void join_send(uint32_t buf, uint32_t acc, int warp, int lane, int valid,
                                          int own, int part) {
  const int q = warp & 3;
  const uint32_t at = (uint32_t)((q * 32 + lane) * 4);
  const int groups = (valid + 15) / 16, turn = (part + 1) * own / 16 % groups;
#pragma unroll 1
  for (int g = warp >> 2; g < groups; g += 2) {
    const int c = (g + turn < groups ? g + turn : g + turn - groups) * 16;
    uint32_t r[16];
    tmem_start16(r, acc + ((uint32_t)(q * 32) << 16) + (uint32_t)c);
    const int token = min(c + (lane & 15), valid - 1), owner = token / own;
    const uint32_t to = map_to_rank(buf, (uint32_t)owner) + (uint32_t)((part * own + token - owner * own) * 512);
    tmem_wait16(r);
    if (c >= part * own && c + 16 <= (part + 1) * own && c + 16 <= valid) {   // all of them stay here
      const uint32_t dst = buf + (uint32_t)(c * 512) + at;
#pragma unroll
      for (int i = 0; i < 16; ++i) sts_b32(dst + i * 512u, r[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t dst = __shfl_sync(kFull, to, i) + at;
        if (c + i < valid) st_cluster(dst, r[i]);
      }
    }
  }
}

// The joining side: adds the parts in order and finishes this CTA's `mine`
// tokens (the tile's from `first`), 4 columns a lane, so that a warp reads a
// token's 512 bytes and writes its 256 in one piece each, and keeps the bias in
// registers.  kJoin tokens are under way in a warp, without a branch between
// them: 4 of a linear product (256 x 1024 -> 1024 with K whole 10.2 us, 11.0 with
// 2), fewer where a token's arithmetic is long, since code that runs once a launch
// costs what fetching it takes (a backward pass of 1024 / 2816 at one token 19.5 us
// with 4, 19.0 with 2).  What the first of them read from memory is asked for in
// the constructor, before the sums are there.
template <int EPI, bool BF>
struct Join {
  static constexpr int kJoin = EPI == DENSE_LINEAR ? 4 : EPI == DENSE_GRAD ? 2 : 1;
  static constexpr int kLanes = EPI == DENSE_GATED ? 16 : 32;   // lanes of a token
  static constexpr int kStep = 256 / kLanes;                    // tokens that the CTA takes at once
  const DenseArgs& args;
  int row0, col, mine, slot, ch;
  float4 bias;
  Extra e[kJoin];

  __device__ __forceinline__ Join(const DenseArgs& a, int n0, int first, int tokens)
      : args(a), row0(first), mine(tokens), bias(make_float4(0.f, 0.f, 0.f, 0.f)) {
    slot = (int)threadIdx.x / kLanes;
    ch = (int)threadIdx.x % kLanes * 4;
    col = n0 + ch;
    if (col >= a.cols) mine = 0;
    if (EPI == DENSE_LINEAR && a.bias != nullptr && slot < mine)
      bias = unpack4<BF>(__ldg(reinterpret_cast<const uint2*>(a.bias + col)));
#pragma unroll
    for (int t = 0; t < kJoin; ++t) e[t] = {make_uint2(0, 0), make_uint2(0, 0)};
    fetch(slot);
    // the later ones come from memory to the L2 cache meanwhile (dh and dX of 256
    // tokens 1024 / 2816: 19.2 us, 19.8 without)
    if (ch % 64 == 0 && (EPI == DENSE_GRAD || (EPI == DENSE_LINEAR && a.residual != nullptr)))
      for (int s = slot + kJoin * kStep; s < mine; s += kStep) {
        if constexpr (EPI == DENSE_GRAD) {
          prefetch_l2(a.g + (int64_t)(row0 + s) * a.cols + col);
          prefetch_l2(a.u + (int64_t)(row0 + s) * a.cols + col);
        } else {
          prefetch_l2(a.residual + (int64_t)(row0 + s) * a.ldr + col);
        }
      }
  }

  __device__ __forceinline__ void fetch(int s) {
    if (EPI == DENSE_GRAD || (EPI == DENSE_LINEAR && args.residual != nullptr))
#pragma unroll
      for (int t = 0; t < kJoin; ++t)
        if (s + t * kStep < mine) e[t] = load_extra<EPI>(args, row0 + s + t * kStep, col);
  }

  __device__ __forceinline__ void finish(uint32_t buf, int own, int parts) {
    if (slot >= mine) return;
    with_act(args.act, [&](auto A) {
#pragma unroll 1
      for (int s = slot; s < mine; s += kJoin * kStep) {
        uint32_t f[kJoin];
        float4 v[kJoin], w[kJoin];
#pragma unroll
        for (int t = 0; t < kJoin; ++t) {
          f[t] = buf + (uint32_t)((min(s + t * kStep, mine - 1) * 128 + ch) * 4);
          v[t] = w[t] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll 1
        for (int src = 0; src < parts; ++src)
#pragma unroll
          for (int t = 0; t < kJoin; ++t) {
            v[t] = add4(v[t], lds_f32x4(f[t]));
            if constexpr (EPI == DENSE_GATED) w[t] = add4(w[t], lds_f32x4(f[t] + 256u));
            f[t] += (uint32_t)own * 512u;
          }
        uint2 o[3][kJoin];
#pragma unroll
        for (int t = 0; t < kJoin; ++t)
          finish4<EPI, BF, decltype(A)::value>(v[t], w[t], bias, e[t], o[0][t], o[1][t], o[2][t]);
        const int64_t at = (int64_t)(row0 + s) * args.ldo + col, step = (int64_t)kStep * args.ldo;
        store(args.o[0] + at, step, s, o[0]);
        if (EPI == DENSE_GRAD || (EPI == DENSE_GATED && args.outs == 3)) {
          store(args.o[1] + at, step, s, o[1]);
          store(args.o[2] + at, step, s, o[2]);
        }
        fetch(s + kJoin * kStep);
      }
    });
  }

  __device__ __forceinline__ void store(uint16_t* to, int64_t step, int s, const uint2 (&o)[kJoin]) {
#pragma unroll
    for (int t = 0; t < kJoin; ++t)
      if (s + t * kStep < mine) *reinterpret_cast<uint2*>(to + t * step) = o[t];
  }
};

// The weight's boxes of K stage kb for a CTA's 128 accumulator lanes from
// output column n0: each(map, coordinates, byte offset in the operand).
template <bool B_K, int EPI, typename F>
__device__ __forceinline__ void weight_boxes(const DenseMaps& maps, const DenseArgs& args, int n0, int kb,
                                             F&& each) {
  const int seg = kb >= args.kb0 ? 1 : 0;
  const int k = (kb - (seg ? args.kb0 : 0)) * kSlab;
  if constexpr (B_K) {
    each(&maps.b[seg], k, n0, 0u);
  } else if constexpr (EPI == DENSE_GATED) {   // 64 columns of each weight: lanes 0 .. 63 g, 64 .. 127 u
    each(&maps.b[0], n0, k, 0u);
    each(&maps.b[1], n0, k, kBlock);
  } else {
    each(&maps.b[seg], n0, k, 0u);
    each(&maps.b[seg], n0 + 64, k, kBlock);
  }
}

// ---------------------------------------------------------------------------
// Persistent CTA pairs: tiles of 256 tokens x 256 (or 128) accumulator columns
//
// Tensor memory holds two accumulators of 256 columns, taken in turn, so the
// epilogue of a tile runs beside the mainloop of the next; it hands an
// accumulator back as soon as its last columns are in registers.  When the
// tiles left after the last whole wave of CTA pairs are at most half a wave,
// each is cut into two of 128 columns, so that the wave takes less time: a stage
// of 128 columns takes 0.19 us against 0.275 us (256 x 8192 x 256), and
// 512 x 4096 x 4096 19.2 against 25.3 us.
// ---------------------------------------------------------------------------
constexpr int kPairThreads = 320;                  // 8 epilogue warps, one loads, one issues MMAs
constexpr int kPairMaxStages = 5;
constexpr uint32_t kOperand = kTile * kSlab * 2;   // 16 KB: 128 rows (or columns) x 64 K
constexpr uint32_t kStoreBlock = 32 * 128;         // 32 rows x 64 columns; an epilogue warp has two
constexpr int kGroupRows = 8;                      // row tiles walked together (L2 reuse of B)
constexpr int kSmemPerCta = 227 * 1024, kSmemPerSm = 228 * 1024;   // a CTA costs 1 KB more than it asks for

// Shared memory: the ring (stage: 128 rows of A, then this CTA's half of the
// columns of B), the eight epilogue warps' blocks, the barriers.  A warp's
// blocks hold what it reads (residual; g and u), brought by TMA ahead of the
// accumulator, and in its place what it stores: two of 32 rows x 64 columns, or
// for DENSE_GRAD two sets of three of 32 x 32, at the price of a ring stage.
// Lanes reading 16 bytes of 32 different rows straight from global memory
// took 31.9 us instead of 27.4 in the gradient's first product, 2048 tokens
// 1024/2816.
template <int EPI>
struct PairCfg {
  static constexpr int kStages = EPI == DENSE_GRAD ? 4 : 5;
  static constexpr uint32_t kSet = EPI == DENSE_GRAD ? 3 * 2048 : kStoreBlock;   // bytes of one of the two
  static constexpr uint32_t kWarpBytes = 2 * kSet;
};

struct PairBars {
  unsigned long long full[kPairMaxStages];         // used in the leader
  unsigned long long empty[kPairMaxStages];
  unsigned long long acc_full[2], acc_empty[2];    // acc_empty used in the leader
  unsigned long long done;
  unsigned long long extra[8][2];                  // per epilogue warp: what it reads, per set
  uint32_t tmem_base;
  int abort_flag;
  int consumed;
  int brought[2];   // 0, or of a CTA that gave up 1 + the stages that it brought, see end_pair
};

// Item t of the walk: a tile of 256 accumulator columns, or, from `whole` on,
// one of the two halves of a tile.
struct TilePos {
  int m, mat, n;   // row tile, weight, accumulator column
  int bn;          // 256 or 128
  int rows, cols;  // of the output that the tile belongs to
};

// Row tiles are walked in groups, so that a group's tiles share their columns' B.
__device__ __forceinline__ TilePos tile_at(int t, const DenseArgs& a) {
  const int half = t < a.whole ? 0 : 1;
  int u = half ? a.whole + (t - a.whole) / 2 : t;
  const int first = a.tm * a.tn * a.mats;
  const bool also = u >= first;              // a tile of the second product
  if (also) u -= first;
  const int tm = also ? a.tm2 : a.tm, tn = also ? a.tn2 : a.tn;
  const int per = kGroupRows * (also ? tn : tn * a.mats);
  const int g0 = u / per * kGroupRows, r = u % per;
  const int gs = min(kGroupRows, tm - g0);
  const int n = r / gs, mat = n / tn;
  return {g0 + r % gs, also ? 2 : mat, (n - mat * tn) * 256 + (half ? (t - a.whole) % 2 * 128 : 0),
          half ? 128 : 256, also ? a.rows2 : a.rows, also ? a.cols2 : a.cols};
}

// Where lane's (row's) 16-byte chunk j lies in a block: 64 columns wide, in the
// 128-byte swizzled order of its tensor map, or 32 wide in the 64-byte one.
__device__ __forceinline__ uint32_t wide_at(uint32_t block, int lane, int j) {
  return block + (uint32_t)lane * 128u + (uint32_t)((j ^ (lane & 7)) << 4);
}
__device__ __forceinline__ uint32_t narrow_at(uint32_t block, int lane, int j) {
  return block + (uint32_t)lane * 64u + (uint32_t)((j ^ ((lane >> 1) & 3)) << 4);
}

__device__ __forceinline__ void sts16(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// A block is free once the stores from it have read it; `N` later ones may be on their way.
template <int N>
__device__ __forceinline__ void stage_wait(int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
  __syncwarp();
}

__device__ __forceinline__ void stage_store(uint32_t block, int lane, const CUtensorMap* map, int col,
                                            int row, const TilePos& p) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (lane == 0) {
    if (row < p.rows && col < p.cols) tma_store_2d(map, block, col, row);   // the map clips the rest
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}

// The end of a pair's walk, with the MMAs done and every warp of the CTA here.  After a
// give-up of either CTA, the copies that both issued land before shared memory goes.  A
// stage that only one of them brought never completes, so each says how far it came (a
// leader that waited for such a stage held the GPU for the default limit, 2 s, a stage);
// the copies of those stages were issued a wait's limit ago, and land in the last pause.
template <typename Bars>
__device__ __forceinline__ void end_pair(Bars& sm, int stages, uint32_t rank, int issued, uint32_t tmem, int warp,
                                         int lane) {
  if (warp == 8 && lane < 2 && *(volatile int*)&sm.abort_flag)
    st_cluster(map_to_rank(smem_u32(&sm.brought[rank]), (uint32_t)lane), (uint32_t)issued + 1u);
  __syncthreads();
  cluster_sync();
  if (warp == 8)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u)
                 : "memory");
  const int a = *(volatile int*)&sm.brought[0], b = *(volatile int*)&sm.brought[1];
  if ((a | b) == 0) return;
  if (warp == 8 && lane == 0) {
    // who did not give up has brought every stage
    const int both = min(a > 0 ? a - 1 : 0x7fffffff, b > 0 ? b - 1 : 0x7fffffff);
    if (rank == 0)
      for (int it = sm.consumed; it < both; ++it)
        wait_drain(smem_u32(&sm.full[it % stages]), (uint32_t)(it / stages) & 1u);
    const long long t0 = clock64();
    while (clock64() - t0 < 40000) {
    }
  }
  __syncthreads();
  cluster_sync();
}

template <bool A_MN, bool B_K, int EPI, bool BF>
__global__ void __launch_bounds__(kPairThreads, 1)
dense_pair_kernel(const __grid_constant__ DenseMaps maps, const __grid_constant__ DenseArgs args) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  using Cfg = PairCfg<EPI>;
  constexpr int S = Cfg::kStages;
  constexpr uint32_t stage_bytes = 2 * kOperand;   // 128 rows of A and up to 128 columns of B
  uint8_t* blocks = ring + (size_t)S * stage_bytes;
  PairBars& sm = *reinterpret_cast<PairBars*>(blocks + 8 * Cfg::kWarpBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  volatile int* abort_flag = &sm.abort_flag;

  if (warp == 9 && lane < 10)
    prefetch_map(lane < 2   ? &maps.a[lane]
                 : lane < 5 ? &maps.b[lane - 2]
                 : lane < 8 ? &maps.o[lane - 5]
                            : &maps.r[lane - 8]);
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&sm.full[s]), 1);
      mbar_init(smem_u32(&sm.empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&sm.acc_full[s]), 1);
      mbar_init(smem_u32(&sm.acc_empty[s]), 16);   // the epilogue warps of both CTAs
    }
    mbar_init(smem_u32(&sm.done), 1);
    for (int w = 0; w < 16; ++w) mbar_init(smem_u32(&sm.extra[w / 2][w % 2]), 1);
    sm.abort_flag = 0;
    sm.consumed = 0;
    sm.brought[0] = sm.brought[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  // All of tensor memory, at once: nothing else that uses it fits beside this
  // CTA's shared memory (see dense_few_kernel).
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sm.tmem_base)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  __syncwarp();
  cluster_sync();   // both CTAs' barriers exist before anything targets them
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = sm.tmem_base;
  pdl_wait();
  pdl_trigger();
  const long long limit = wait_limit();

  int issued = 0;   // stages whose copies this CTA's producer has issued
  if (warp == 8) {   // ---- TMA producer (both CTAs): the warp loops, one lane issues ----
    int s = 0;
    uint32_t ph = 1;
    bool go = true;
    const uint32_t full0 = map_to_rank(smem_u32(&sm.full[0]), 0);
    for (int t = pair; t < args.items && go; t += pairs) {
      const TilePos p = tile_at(t, args);
      const int m0 = p.m * 256 + (int)rank * 128;
      // DENSE_GATED: CTA 0 brings the gate's columns, CTA 1 the up's
      const int nb = EPI == DENSE_GATED ? p.n / 2 : p.n + (int)rank * (p.bn / 2);
      for (int kb = 0; kb < args.kbt; ++kb) {
        go = __all_sync(kFull, wait_bounded(smem_u32(&sm.empty[s]), ph, abort_flag, limit));
        if (!go) break;
        const int seg = kb >= args.kb0 ? 1 : 0;
        const int k = (kb - (seg ? args.kb0 : 0)) * kSlab;
        const CUtensorMap* ma = &maps.a[A_MN ? p.mat >> 1 : seg];   // A_MN: one segment, the second product's A
        const CUtensorMap* mb = &maps.b[EPI == DENSE_GATED ? (int)rank : seg | p.mat];
        const uint32_t fb = full0 + (uint32_t)s * 8u;
        const uint32_t a0 = smem_u32(ring) + (uint32_t)s * stage_bytes, b0 = a0 + kOperand;
        if (elect_one()) {
          if (leader) mbar_expect_tx(smem_u32(&sm.full[s]), 2 * (kOperand + (uint32_t)p.bn * 64u));
          if constexpr (A_MN) {
            tma_load_2d_pair(a0, ma, m0, k, fb);
            tma_load_2d_pair(a0 + kBlock, ma, m0 + 64, k, fb);
          } else {
            tma_load_2d_pair(a0, ma, k, m0, fb);
          }
          // 64 columns a box
          for (int j = 0; j < p.bn / 128; ++j) {
            if constexpr (B_K)
              tma_load_2d_pair(b0 + j * kBlock, mb, k, nb + j * 64, fb);
            else
              tma_load_2d_pair(b0 + j * kBlock, mb, nb + j * 64, k, fb);
          }
        }
        __syncwarp();
        ++issued;
        if (++s == S) { s = 0; ph ^= 1u; }
      }
    }
  } else if (warp == 9) {   // ---- MMA issuer (the leader's): the warp loops, one lane issues ----
    if (leader) {
      const uint32_t a_low = slab_low<A_MN>(smem_u32(ring)), b_low = slab_low<!B_K>(smem_u32(ring) + kOperand);
      int s = 0, count = 0, used = 0;
      uint32_t ph = 0, at = 0;   // at: the stage's offset in 16-byte units
      bool go = true;
      for (int t = pair; t < args.items && go; t += pairs, ++count) {
        const int slot = count & 1;
        const uint32_t idesc = dense_idesc(256, t < args.whole ? 256 : 128, BF, A_MN, B_K);
        go = __all_sync(kFull, wait_bounded(smem_u32(&sm.acc_empty[slot]),
                                            ((uint32_t)(count >> 1) & 1u) ^ 1u, abort_flag, limit));
        if (!go) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t d = tmem + (uint32_t)slot * 256u;
        for (int kb = 0; kb < args.kbt; ++kb) {
          go = __all_sync(kFull, wait_bounded(smem_u32(&sm.full[s]), ph, abort_flag, limit));
          if (!go) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          ++used;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kSlab / 16; ++k)
              mma_f16<2>(d, slab_desc(a_low + at + k * slab_step<A_MN>),
                         slab_desc(b_low + at + k * slab_step<!B_K>), idesc, (kb > 0 || k > 0) ? 1u : 0u);
            commit_pair(smem_u32(&sm.empty[s]));
            if (kb == args.kbt - 1) commit_pair(smem_u32(&sm.acc_full[slot]));
          }
          __syncwarp();
          at += stage_bytes >> 4;
          if (++s == S) { s = 0; at = 0; ph ^= 1u; }
        }
      }
      if (lane == 0) sm.consumed = used;
      if (elect_one()) commit_pair(smem_u32(&sm.done));   // completes once every issued MMA has finished
      __syncwarp();
    }
  } else {   // ---- epilogue: eight warps, each 32 rows x half of the columns ----
    const int q = warp & 3, half = warp >> 2;
    const uint32_t store = smem_u32(blocks) + (uint32_t)warp * Cfg::kWarpBytes;
    const uint32_t empty0 = map_to_rank(smem_u32(&sm.acc_empty[0]), 0);
    const uint32_t empty1 = map_to_rank(smem_u32(&sm.acc_empty[1]), 0);
    const bool reads = EPI == DENSE_GRAD || (EPI == DENSE_LINEAR && args.residual != nullptr);
    int count = 0;
    uint32_t set = 0;         // the set of blocks used next
    uint32_t extra_ph = 0;    // bit s: parity of extra[s]'s next phase
    uint32_t coming = 0;      // bit s: a read into set s is on its way
    // start the reads of a piece (64 columns; DENSE_GRAD 32) into set s; one lane
    auto fetch = [&](uint32_t s, int col, int row0) {
      if (row0 >= args.rows || col >= args.cols) return;
      coming |= 1u << s;
      if (lane == 0) {
        const uint32_t bar = smem_u32(&sm.extra[warp][s]), to = store + s * Cfg::kSet;
        mbar_expect_tx(bar, 4096u);
        tma_load_2d(to, &maps.r[0], col, row0, bar);
        if constexpr (EPI == DENSE_GRAD) tma_load_2d(to + 2048u, &maps.r[1], col, row0, bar);
      }
    };
    // wait for them; false when a wait gave up
    auto fetched = [&](uint32_t s) {
      const bool ok = __all_sync(kFull, wait_bounded(smem_u32(&sm.extra[warp][s]), (extra_ph >> s) & 1u,
                                                     abort_flag, limit));
      if (ok) {
        extra_ph ^= 1u << s;
        coming &= ~(1u << s);
      }
      return ok;
    };
    for (int t = pair; t < args.items; t += pairs, ++count) {
      const TilePos p = tile_at(t, args);
      const int row0 = p.m * 256 + (int)rank * 128 + q * 32;
      const int blocks_of_warp = p.bn / 128;   // pieces of 64 columns (DENSE_LINEAR, DENSE_GRAD)
      const int slot = count & 1, c_warp = half * (p.bn / 2), col_warp = p.n + c_warp;
      constexpr int kPiece = EPI == DENSE_GRAD ? 32 : 64;
      const int pieces = blocks_of_warp * 64 / kPiece;
      if (reads) {   // the first two pieces, before the accumulator is complete
        stage_wait<0>(lane);
        fetch(set, col_warp, row0);
        if (pieces > 1) fetch(set ^ 1u, col_warp + kPiece, row0);
      }
      // one verdict for the warp: the tensor-memory loads below need all its lanes
      if (!__all_sync(kFull, wait_bounded(smem_u32(&sm.acc_full[slot]), (uint32_t)(count >> 1) & 1u,
                                          abort_flag, limit)))
        break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t acc = tmem + (uint32_t)slot * 256u + ((uint32_t)(q * 32) << 16);
      auto release = [&] {   // this warp has read its part of the accumulator
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) arrive_remote(slot ? empty1 : empty0);
      };
      bool go = true;
      if constexpr (EPI == DENSE_LINEAR) {
#pragma unroll 1
        for (int blk = 0; blk < pieces; ++blk, set ^= 1u) {
          const int c = c_warp + blk * 64, col = p.n + c;
          const uint32_t to = store + set * Cfg::kSet;
          if (!reads)
            stage_wait<1>(lane);
          else if ((coming >> set) & 1u)
            go = fetched(set) && go;
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            uint32_t r[32];
            tmem_start32(r, acc + (uint32_t)(c + part * 32));
            tmem_wait32(r);
            if (blk == pieces - 1 && part == 1) release();
            float v[32];
            as_floats(v, r);
            if (!args.plain) {
              epi_bias_act<BF, 4>(v, args, col + part * 32);
              if (reads) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  float x[8];
                  unpack8<BF>(x, lds16(wide_at(to, lane, part * 4 + j)));
#pragma unroll
                  for (int i = 0; i < 8; ++i) v[8 * j + i] += x[i];
                }
              }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
              sts16(wide_at(to, lane, part * 4 + j), pack8<BF>(*reinterpret_cast<float(*)[8]>(&v[8 * j])));
          }
          if (go) stage_store(to, lane, &maps.o[p.mat], col, row0, p);
        }
      } else if constexpr (EPI == DENSE_GATED) {
        // accumulator columns [0, bn / 2) are g, the others u; 64 hidden columns a
        // warp (with bn 128 there is only work for the first of a quarter's two)
        const int c = half * 64, col = p.n / 2 + c;
        if (c >= p.bn / 2) {
          release();
          continue;
        }
#pragma unroll 1
        for (int out = 0; out < args.outs; ++out, set ^= 1u) {   // h, then g and u themselves
          const uint32_t to = store + set * Cfg::kSet;
          stage_wait<1>(lane);
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            uint32_t r[32];
            tmem_start32(r, acc + (uint32_t)(c + part * 32 + (out == 2 ? p.bn / 2 : 0)));
            float v[32];
            if (out == 0) {
              uint32_t ru[32];
              tmem_start32(ru, acc + (uint32_t)(p.bn / 2 + c + part * 32));
              tmem_wait32(r);
              tmem_wait32(ru);
              if (args.outs == 1 && part == 1) release();
              float u[32];
              as_floats(v, r);
              as_floats(u, ru);
              epi_gated<32>(v, u, args.act);
            } else {
              tmem_wait32(r);
              if (out == 2 && part == 1) release();
              as_floats(v, r);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
              sts16(wide_at(to, lane, part * 4 + j), pack8<BF>(*reinterpret_cast<float(*)[8]>(&v[8 * j])));
          }
          stage_store(to, lane, &maps.o[out], col, row0, p);
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < pieces; ++i, set ^= 1u) {
          const int c = c_warp + i * 32, col = p.n + c;
          const uint32_t to = store + set * Cfg::kSet;
          if ((coming >> set) & 1u) go = fetched(set) && go;
          uint32_t r[32];
          tmem_start32(r, acc + (uint32_t)c);
          tmem_wait32(r);
          if (i == pieces - 1) release();
          float v[32];
          as_floats(v, r);
#pragma unroll
          for (int j = 0; j < 4; ++j) {   // dg and du take the places of g and u, h the third
            const uint32_t at = narrow_at(to, lane, j);
            uint4 dg, du, h;
            epi_grad8<BF>(&v[8 * j], lds16(at), lds16(at + 2048u), args.act, dg, du, h);
            sts16(at, dg);
            sts16(at + 2048u, du);
            sts16(at + 4096u, h);
          }
          if (i > 0 && i + 1 < pieces) {   // the next piece goes where the last one was
            stage_wait<0>(lane);
            fetch(set ^ 1u, col + 32, row0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            if (go && row0 < p.rows && col < p.cols)
              for (int out = 0; out < 3; ++out) tma_store_2d(&maps.o[out], to + out * 2048u, col, row0);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        }
      }
      if (!go) break;
    }
    // after a give-up: reads on their way land before shared memory goes
    for (uint32_t s = 0; s < 2; ++s)
      if ((coming >> s) & 1u) wait_drain(smem_u32(&sm.extra[warp][s]), (extra_ph >> s) & 1u);
    __syncwarp();
    // the outputs are written before the CTA ends
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }

  __syncthreads();
  if (__builtin_expect(!wait_drain(smem_u32(&sm.done), 0u), 0) && tid == 0) atomicOr(&g_dense_error, 1u);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  end_pair(sm, S, rank, issued, tmem, warp, lane);
}

// ---------------------------------------------------------------------------
// Persistent CTA pairs with the tokens as N: tiles of 256 accumulator columns x
// any multiple of 16 tokens up to 256
//
// The same walk, two accumulators and warps' roles, but the weight is the MMA's M
// operand (128 of its columns a CTA) and the tokens, of which each CTA brings
// half, are N: 777 tokens cost 832 in four tiles, not 1024, and the height of the
// tiles can be chosen so that they fill whole waves.  A thread holds one output
// column of 16 tokens at a time; four warps turn them over in shared memory, from
// which each takes four tokens, 4 columns a lane.  Bound by the tensor cores (88 %
// of the SMs' active cycles at 1300 x 4096 -> 11008), below about 150 tokens a tile
// by a stage's bytes: 333 x 4096 -> 11008 in tiles of 112 35 us, 777 in tiles of 160
// 55 us.
// ---------------------------------------------------------------------------
constexpr uint32_t kTurn = 16 * 128 * 4;   // 16 tokens x 128 columns of float32; four warps have two
constexpr int kTallMaxStages = 8;

struct TallBars {
  unsigned long long full[kTallMaxStages];         // used in the leader
  unsigned long long empty[kTallMaxStages];
  unsigned long long acc_full[2], acc_empty[2];    // acc_empty used in the leader
  unsigned long long done;
  uint32_t tmem_base;
  int abort_flag;
  int consumed;
  int brought[2];   // 0, or of a CTA that gave up 1 + the stages that it brought, see end_pair
};

// Item t of the walk: token tile m, column tile n.  The token tiles of a group run
// side by side through all columns, so that a wave's pairs share their weight and
// the group's tokens stay in the L2 cache.
struct TallPos {
  int m, n;
};

__device__ __forceinline__ TallPos tall_at(int t, const DenseArgs& a) {
  const int per = a.group * a.tn, g0 = t / per * a.group, r = t % per;
  const int gs = min(a.group, a.tm - g0);
  return {g0 + r % gs, r / gs};
}

// Barrier `id` of 128 threads, which all learn whether every one said yes.
__device__ __forceinline__ bool all_of_128(int id, bool yes) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(yes ? 1u : 0u), "r"(id)
      : "memory");
  return r != 0;
}

template <bool B_K, int EPI, bool BF>
__global__ void __launch_bounds__(kPairThreads, 1)
dense_tall_kernel(const __grid_constant__ DenseMaps maps, const __grid_constant__ DenseArgs args, const int tn,
                  const int S) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t x_bytes = (uint32_t)tn * 64u, stage_bytes = kOperand + x_bytes;   // 1024-multiples
  uint8_t* turns = ring + (size_t)S * stage_bytes;
  TallBars& sm = *reinterpret_cast<TallBars*>(turns + 4 * kTurn);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  volatile int* abort_flag = &sm.abort_flag;
  constexpr int kOutCols = EPI == DENSE_GATED ? 64 : 128;   // output columns of a CTA

  if (warp == 9 && lane < 4) prefetch_map(lane < 2 ? &maps.a[lane] : &maps.b[lane - 2]);
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&sm.full[s]), 1);
      mbar_init(smem_u32(&sm.empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&sm.acc_full[s]), 1);
      mbar_init(smem_u32(&sm.acc_empty[s]), 16);   // the epilogue warps of both CTAs
    }
    mbar_init(smem_u32(&sm.done), 1);
    sm.abort_flag = 0;
    sm.consumed = 0;
    sm.brought[0] = sm.brought[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 8) {   // all of tensor memory, as in dense_pair_kernel
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sm.tmem_base)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  __syncwarp();
  cluster_sync();   // both CTAs' barriers exist before anything targets them
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = sm.tmem_base;
  pdl_wait();
  pdl_trigger();
  const long long limit = wait_limit();

  int issued = 0;   // stages whose copies this CTA's producer has issued
  if (warp == 8) {   // ---- TMA producer (both CTAs): the warp loops, one lane issues ----
    int s = 0;
    uint32_t ph = 1;
    bool go = true;
    const uint32_t full0 = map_to_rank(smem_u32(&sm.full[0]), 0);
    for (int t = pair; t < args.items && go; t += pairs) {
      const TallPos p = tall_at(t, args);
      const int t0 = p.m * tn + (int)rank * (tn / 2), n0 = (p.n * 2 + (int)rank) * kOutCols;
      for (int kb = 0; kb < args.kbt; ++kb) {
        go = __all_sync(kFull, wait_bounded(smem_u32(&sm.empty[s]), ph, abort_flag, limit));
        if (!go) break;
        const int seg = kb >= args.kb0 ? 1 : 0;
        const uint32_t fb = full0 + (uint32_t)s * 8u, w0 = smem_u32(ring) + (uint32_t)s * stage_bytes;
        if (elect_one()) {
          if (leader) mbar_expect_tx(smem_u32(&sm.full[s]), 2 * stage_bytes);
          weight_boxes<B_K, EPI>(maps, args, n0, kb, [&](const CUtensorMap* map, int c0, int c1, uint32_t at) {
            tma_load_2d_pair(w0 + at, map, c0, c1, fb);
          });
          tma_load_2d_pair(w0 + kOperand, &maps.a[seg], (kb - (seg ? args.kb0 : 0)) * kSlab, t0, fb);
        }
        __syncwarp();
        ++issued;
        if (++s == S) { s = 0; ph ^= 1u; }
      }
    }
  } else if (warp == 9) {   // ---- MMA issuer (the leader's): the warp loops, one lane issues ----
    if (leader) {
      const uint32_t idesc = dense_idesc(256, tn, BF, !B_K, true);
      const uint32_t w_low = slab_low<!B_K>(smem_u32(ring)), x_low = slab_low<false>(smem_u32(ring) + kOperand);
      int s = 0, count = 0, used = 0;
      uint32_t ph = 0, at = 0;   // at: the stage's offset in 16-byte units
      bool go = true;
      for (int t = pair; t < args.items && go; t += pairs, ++count) {
        const int slot = count & 1;
        go = __all_sync(kFull, wait_bounded(smem_u32(&sm.acc_empty[slot]),
                                            ((uint32_t)(count >> 1) & 1u) ^ 1u, abort_flag, limit));
        if (!go) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t d = tmem + (uint32_t)slot * 256u;
        for (int kb = 0; kb < args.kbt; ++kb) {
          go = __all_sync(kFull, wait_bounded(smem_u32(&sm.full[s]), ph, abort_flag, limit));
          if (!go) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          ++used;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kSlab / 16; ++k)
              mma_f16<2>(d, slab_desc(w_low + at + k * slab_step<!B_K>),
                         slab_desc(x_low + at + k * slab_step<false>), idesc, (kb > 0 || k > 0) ? 1u : 0u);
            commit_pair(smem_u32(&sm.empty[s]));
            if (kb == args.kbt - 1) commit_pair(smem_u32(&sm.acc_full[slot]));
          }
          __syncwarp();
          at += stage_bytes >> 4;
          if (++s == S) { s = 0; at = 0; ph ^= 1u; }
        }
      }
      if (lane == 0) sm.consumed = used;
      if (elect_one()) commit_pair(smem_u32(&sm.done));   // completes once every issued MMA has finished
      __syncwarp();
    }
  } else {   // ---- epilogue: two times four warps, groups of 16 tokens in turn ----
    constexpr int kLanes = kOutCols / 4, kSub = 32 / kLanes;   // lanes of a token, tokens of a warp's access
    constexpr int kTake = 4 / kSub;                            // accesses for a warp's four tokens
    const int q = warp & 3, half = warp >> 2;
    const uint32_t turn = smem_u32(turns) + (uint32_t)half * 2u * kTurn;
    const uint32_t empty0 = map_to_rank(smem_u32(&sm.acc_empty[0]), 0);
    const uint32_t empty1 = map_to_rank(smem_u32(&sm.acc_empty[1]), 0);
    const int mine = q * 4 + lane / kLanes, ch = lane % kLanes * 4;   // this lane's first token of 16, its columns
    uint32_t set = 0;   // the half of `turn` used next
    int count = 0;
    for (int t = pair; t < args.items; t += pairs, ++count) {
      const TallPos p = tall_at(t, args);
      const int t0 = p.m * tn, col = (p.n * 2 + (int)rank) * kOutCols + ch;
      const int groups = (min(tn, args.rows - t0) + 15) / 16;
      const int slot = count & 1;
      // what tokens [t0 + 16 g, ..) read besides the sums
      auto fetch = [&](Extra (&e)[kTake], int g) {
#pragma unroll
        for (int i = 0; i < kTake; ++i) {
          const int row = t0 + g * 16 + mine + i * kSub;
          e[i] = {make_uint2(0, 0), make_uint2(0, 0)};
          if (g < groups && row < args.rows && col < args.cols) e[i] = load_extra<EPI>(args, row, col);
        }
      };
      float4 bias = make_float4(0.f, 0.f, 0.f, 0.f);
      if (EPI == DENSE_LINEAR && args.bias != nullptr && col < args.cols)
        bias = unpack4<BF>(__ldg(reinterpret_cast<const uint2*>(args.bias + col)));
      Extra e[kTake];
      fetch(e, half);
      // one verdict for the four warps, whose barriers and tensor-memory loads need all of them
      if (!all_of_128(1 + half, wait_bounded(smem_u32(&sm.acc_full[slot]), (uint32_t)(count >> 1) & 1u,
                                             abort_flag, limit)))
        break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t acc = tmem + (uint32_t)slot * 256u + ((uint32_t)(q * 32) << 16);
      auto release = [&] {   // this warp has read its part of the accumulator
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) arrive_remote(slot ? empty1 : empty0);
      };
      if (half >= groups) release();
      with_act(args.act, [&](auto A) {
#pragma unroll 1
        for (int g = half; g < groups; g += 2, set ^= 1u) {
          uint32_t r[16];
          tmem_start16(r, acc + (uint32_t)(g * 16));
          Extra next[kTake];
          fetch(next, g + 2);
          tmem_wait16(r);
          if (g + 2 >= groups) release();
          const uint32_t buf = turn + set * kTurn, to = buf + (uint32_t)(q * 32 + lane) * 4u;
#pragma unroll
          for (int i = 0; i < 16; ++i) sts_b32(to + i * 512u, r[i]);
          // the other set is free again once every warp is here
          asm volatile("barrier.cta.sync.aligned %0, 128;" ::"r"(1 + half) : "memory");
          uint2 o[3][kTake];
#pragma unroll
          for (int i = 0; i < kTake; ++i) {
            const uint32_t f = buf + (uint32_t)((mine + i * kSub) * 128 + ch) * 4u;
            const float4 v = lds_f32x4(f);
            float4 w = {};
            if constexpr (EPI == DENSE_GATED) w = lds_f32x4(f + 256u);
            finish4<EPI, BF, decltype(A)::value>(v, w, bias, e[i], o[0][i], o[1][i], o[2][i]);
          }
#pragma unroll
          for (int i = 0; i < kTake; ++i) {
            const int row = t0 + g * 16 + mine + i * kSub;
            if (row < args.rows && col < args.cols) {
              const int64_t at = (int64_t)row * args.ldo + col;
              *reinterpret_cast<uint2*>(args.o[0] + at) = o[0][i];
              if (EPI == DENSE_GRAD || (EPI == DENSE_GATED && args.outs == 3)) {
                *reinterpret_cast<uint2*>(args.o[1] + at) = o[1][i];
                *reinterpret_cast<uint2*>(args.o[2] + at) = o[2][i];
              }
            }
            e[i] = next[i];
          }
        }
      });
    }
  }

  __syncthreads();
  if (__builtin_expect(!wait_drain(smem_u32(&sm.done), 0u), 0) && tid == 0) atomicOr(&g_dense_error, 1u);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  end_pair(sm, S, rank, issued, tmem, warp, lane);
}

// ---------------------------------------------------------------------------
// Few tokens: 128 output columns x up to 256 tokens a tile, K split over a cluster
//
// A stage carries 16 KB of weight and only 128 bytes a token, and a block of
// one token costs no more tensor work than one of sixteen.
// ---------------------------------------------------------------------------
constexpr int kFewThreads = 256;
constexpr int kFewMaxStages = 12;
constexpr int kFewCluster = 8;

struct FewBars {
  unsigned long long full[kFewMaxStages];
  unsigned long long empty[kFewMaxStages];
  unsigned long long accum;
  alignas(8) uint8_t gave_up[kFewCluster];   // each part's verdict, written by it in every CTA of the cluster
  uint32_t tmem_base;
  int abort_flag;
  int consumed;
};

struct FewShape {
  int tn;        // tokens of a tile: a multiple of 16, at most 256
  int stages;
  int tmem;      // tensor-memory columns: a power of two >= max(tn, 32)
  int join;      // bytes after the ring for the join, or 0: it takes the ring's place
};

template <bool B_K, int EPI, bool BF>
__global__ void __launch_bounds__(kFewThreads)
dense_few_kernel(const __grid_constant__ DenseMaps maps, const __grid_constant__ DenseArgs args,
                 const FewShape fs) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t x_bytes = (uint32_t)fs.tn * 128u, stage_bytes = kOperand + x_bytes;   // 1024-multiples
  const int S = fs.stages;
  FewBars& sm = *reinterpret_cast<FewBars*>(ring + (size_t)S * stage_bytes + fs.join);
  uint8_t* join = fs.join > 0 ? ring + (size_t)S * stage_bytes : ring;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)blockIdx.x, ranks = (int)gridDim.x;   // the cluster spans the grid's x
  constexpr int kOutCols = EPI == DENSE_GATED ? 64 : 128;     // output columns of the tile
  const int n0 = (int)blockIdx.y * kOutCols;
  const int t0 = (int)blockIdx.z * fs.tn;
  const int kb_lo = (int)((int64_t)args.kbt * rank / ranks);
  const int steps = (int)((int64_t)args.kbt * (rank + 1) / ranks) - kb_lo;
  volatile int* abort_flag = &sm.abort_flag;

  if (warp == 2 && lane < 4) prefetch_map(lane < 2 ? &maps.a[lane] : &maps.b[lane - 2]);
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&sm.full[s]), 1);
      mbar_init(smem_u32(&sm.empty[s]), 1);
    }
    mbar_init(smem_u32(&sm.accum), 1);
    sm.abort_flag = 0;
    sm.consumed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncthreads();
  // every CTA of the cluster runs once this barrier is passed (waited for
  // before the first access to another CTA's shared memory)
  if (ranks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait();
  const long long limit = wait_limit();

  int issued = 0;
  if (warp == 0) {   // ---- TMA producer: the warp loops, one lane issues ----
    int s = 0;
    uint32_t ph = 1;
    for (int i = 0; i < steps; ++i) {
      if (!__all_sync(kFull, wait_bounded(smem_u32(&sm.empty[s]), ph, abort_flag, limit))) break;
      const int kb = kb_lo + i, seg = kb >= args.kb0 ? 1 : 0;
      const int k = (kb - (seg ? args.kb0 : 0)) * kSlab;
      const uint32_t fb = smem_u32(&sm.full[s]), w0 = smem_u32(ring) + (uint32_t)s * stage_bytes;
      if (elect_one()) {
        mbar_expect_tx(fb, stage_bytes);
        weight_boxes<B_K, EPI>(maps, args, n0, kb, [&](const CUtensorMap* map, int c0, int c1, uint32_t at) {
          tma_load_2d(w0 + at, map, c0, c1, fb);
        });
        tma_load_2d(w0 + kOperand, &maps.a[seg], k, t0, fb);
      }
      __syncwarp();
      ++issued;
      if (++s == S) { s = 0; ph ^= 1u; }
    }
  } else if (warp == 1) {   // ---- MMA issuer: the warp loops, one lane issues ----
    // Tensor memory only now, with the launch before this one complete, and only
    // then may the next one start: CTAs of several launches fit an SM, and one
    // that waits for another must not hold what the other may still ask for.
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sm.tmem_base)),
                 "r"(fs.tmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    asm volatile("barrier.cta.sync.aligned 1, 32;" ::: "memory");   // this warp: the address is visible
    const uint32_t tmem = *(volatile uint32_t*)&sm.tmem_base;
    pdl_trigger();
    const uint32_t idesc = dense_idesc(kTile, fs.tn, BF, !B_K, true);
    const uint32_t w_low = slab_low<!B_K>(smem_u32(ring)), x_low = slab_low<false>(smem_u32(ring) + kOperand);
    int s = 0, used = 0;
    uint32_t ph = 0, at = 0;   // at: the stage's offset in 16-byte units
    for (int i = 0; i < steps; ++i) {
      if (!__all_sync(kFull, wait_bounded(smem_u32(&sm.full[s]), ph, abort_flag, limit))) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      ++used;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kSlab / 16; ++k)
          mma_f16<1>(tmem, slab_desc(w_low + at + k * slab_step<!B_K>),
                     slab_desc(x_low + at + k * slab_step<false>), idesc, (i > 0 || k > 0) ? 1u : 0u);
        commit_one(smem_u32(&sm.empty[s]));
      }
      __syncwarp();
      at += stage_bytes >> 4;
      if (++s == S) { s = 0; at = 0; ph ^= 1u; }
    }
    if (lane == 0) sm.consumed = used;
    if (elect_one()) commit_one(smem_u32(&sm.accum));   // completes once every issued MMA has finished
    __syncwarp();
  }

  const int valid = min(fs.tn, args.rows - t0);    // tokens of this tile
  const int own = (valid + ranks - 1) / ranks;     // rank r joins tokens [r own, (r + 1) own)
  Join<EPI, BF> last(args, n0, t0 + rank * own, min(own, valid - rank * own));

  // Every warp polls: with one of them, and the others at the barrier, 333 x 4096 ->
  // 4096 takes 16.9 us instead of 16.5.  One verdict for the CTA, since the
  // tensor-memory loads below need whole warps.
  const bool acc_done = wait_sums(smem_u32(&sm.accum), limit);
  const bool ok = __syncthreads_and(acc_done && !*abort_flag) != 0;
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *(volatile uint32_t*)&sm.tmem_base;
  if (ranks > 1) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (fs.join == 0) cluster_sync();   // the ring is free once every CTA's MMAs are done
    // and one for the cluster: a part that gave up is missing from every sum
    if (warp == 0 && lane < ranks)
      st_cluster_u8(map_to_rank(smem_u32(&sm.gave_up[rank]), (uint32_t)lane), ok ? 0u : 1u);
  }
  if (ok) join_send(smem_u32(join), tmem, warp, lane, valid, own, rank);
  bool whole = ok;
  if (ranks > 1) {
    cluster_sync();
    const unsigned long long parts = *reinterpret_cast<volatile unsigned long long*>(sm.gave_up);
    whole = whole && parts << (8 * (kFewCluster - ranks)) == 0ull;
  } else {
    __syncthreads();
  }
  if (whole) last.finish(smem_u32(join), own, ranks);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (tid == 0 && *abort_flag)
    for (int i = sm.consumed; i < issued; ++i)
      wait_drain(smem_u32(&sm.full[i % S]), (uint32_t)(i / S) & 1u);
  __syncthreads();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(fs.tmem)
                 : "memory");
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// 2-D map over 16-bit values: `inner` contiguous, `outer` rows `pitch` apart,
// box `width` (64, or 32) x `box` rows, swizzled by the box's row length of 128
// (or 64) bytes, zeros outside.
bool map16(CUtensorMap* map, const void* base, int64_t inner, int64_t outer, int64_t pitch, int box,
           int width = 64) {
  auto enc = get_encode();
  if (enc == nullptr) return false;
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  cuuint64_t strides[1] = {(cuuint64_t)pitch * 2};
  cuuint32_t boxes[2] = {(cuuint32_t)width, (cuuint32_t)box};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(base), dims, strides, boxes,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             width == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// K stages of a product, and of one of its segments
int segment_stages(const DenseGemm& d) { return ceil_div(d.K, kSlab); }
int all_stages(const DenseGemm& d) { return segment_stages(d) * (d.two_segments ? 2 : 1); }

// Clusters of 1 .. 8 CTAs are placed within a GPC, so fewer of the larger ones
// fit at once: what cudaOccupancyMaxActiveClusters gave on a B200 for the few-token
// kernel's shared memory with one and with two CTAs on an SM.  Where another card's
// GPCs differ, the choice below is off, never a result.
constexpr int kClusters1[kFewCluster + 1] = {0, 148, 74, 45, 33, 26, 22, 15, 15};
constexpr int kClusters2[kFewCluster + 1] = {0, 296, 148, 93, 71, 56, 45, 37, 33};

// Which kernel, and how a few-token launch is split.
//
// Up to 16 tokens the launch is bound by reading the weight and two CTAs share an
// SM.  K is split until there are 128 CTAs, and on while each keeps 32 stages and
// the clusters run at once.  Measured on B200 with 16 tokens: 4096 -> 4096 8.6 us
// with 4 parts against 9.3 with 3; 11008 -> 4096 17.2 with 5 against 17.6 with 8;
// 4096 -> 11008 17.2 with 2 or 3 against 18.5 with 1.
//
// Above, the estimates below, in us, pick the fastest of what is in play.
//
// The few-token kernel, to 4096 tokens (2048 x 4096 -> 512 12.8 us, the others 18.2),
// with blocks of 64 tokens or more (or two halves) and K split over the SMs.  A stage
// takes what its bytes take to arrive at an SM (about 136 KB/us, shared by the CTAs
// on it) or what the weight of all CTAs takes to arrive from memory and the L2 cache;
// two CTAs share an SM with blocks of at most 128 tokens and K whole (128 x 4096 ->
// 11008 in three parts 21.8 us, 20.0 alone with K whole), and several blocks run only
// within two waves, so that the second one finds the weight in the cache (400 x 8192
// -> 2 x 28672: 576 us in seven, 538 with the pair kernel).  Fitted to 321 shapes of
// 17 - 1024 tokens, K of 256 - 11008 and 512 - 32768 outputs, each timed with every
// split that fits: the choice costs 0.9 % over the fastest on average.  At 64 tokens:
// 4096 -> 4096 9.8 us with one CTA an SM against 11.2 with two, 2048 -> 20480 17.6
// with two against 23.7 with one.
//
// The tall kernel, with the tile height whose waves cost least, and the pair kernel
// with its whole and half tiles.  Fitted to 154 shapes of 128 - 4096 tokens, K of 512
// - 22016 and 1024 - 22016 outputs, the choice costs 0.6 % over the fastest.  At 256
// tokens: 4096 -> 4096 few 13.4 us, tall 17.8, pair 21.2; at 777: 4096 -> 11008 tall
// 56.1, pair 67.7; 4096 x 4096 -> 22016 tall 537, pair 568; 4096 x 1024 -> 1024 pair
// 11.1, tall 12.1.
constexpr int kGroupTiles = 16;   // token tiles the tall kernel walks together (4096 x 4096 -> 11008 in
                                  // tiles of 208: 276 us, 281 with 4; 16384 x 4096 -> 4096: 405, 413 with all)
}  // namespace

DensePlan plan_dense(const DenseGemm& d) {
  const int kbt = all_stages(d);
  const DensePlan pair = {DENSE_PAIR, 256, 1, 1};
  if (d.a_mn) return pair;
  const int shrink = d.epi == DENSE_GATED ? 2 : 1;   // accumulator columns of an output column
  const int cols = ceil_div(d.cols * shrink, 128);
  if (d.rows <= 16) {
    int parts = std::min({kFewCluster, kbt, std::max({1, kbt / 32, 128 / cols})});
    while (parts > 1 && cols > kClusters2[parts]) --parts;
    return {DENSE_FEW, 16, parts, 2};
  }
  const int tiles = ceil_div(d.rows, 256) * ceil_div(d.cols * shrink, 256);
  const int waves = tiles / (kNumSMs / 2), left = tiles % (kNumSMs / 2);
  double best = 4.1 + kbt * (0.36 * waves + (left == 0 ? 0.0 : left <= kNumSMs / 4 ? 0.25 : 0.33));
  DensePlan plan = pair;
  const int least = ceil_div(d.rows, 256);
  for (int blocks = least; blocks <= std::min(least + 16, ceil_div(d.rows, 64)); ++blocks) {
    const int tn = ceil_div(ceil_div(d.rows, blocks), 16) * 16;
    const double stage = std::max(0.00125 * tn, (16.0 + tn / 16.0) / 115.0);
    const int64_t items = (int64_t)ceil_div(d.rows, tn) * ceil_div(d.cols * shrink, 256);
    const double t = 3.6 + 0.005 * tn + ceil_div(items, kNumSMs / 2) * (kbt * stage + 0.5);
    if (t < best) {
      best = t;
      plan = {DENSE_TALL, tn, 1, 1};
    }
  }
  if (d.rows > 4096) return plan;
  for (int blocks = least; blocks <= std::max(2, ceil_div(d.rows, 64)); ++blocks) {
    if (blocks > 1 && blocks * cols > 2 * kClusters2[1]) break;   // more than two waves, each block reads the weight again
    const int tn = ceil_div(ceil_div(d.rows, blocks), 16) * 16, few = blocks * cols;
    for (int per_sm = 1; per_sm <= (tn <= 128 ? 2 : 1); ++per_sm)
      for (int parts = 1; parts <= (per_sm == 2 ? 1 : std::min(kFewCluster, kbt)); ++parts) {
        auto wave = [&](int clusters) {
          const int ctas = clusters * parts, sms = std::min(ctas, kNumSMs * per_sm);
          const double fill = (16.0 + tn / 8.0) / (ctas <= kNumSMs ? 136.0 : 68.0), read = 16.0 * sms / 10000.0;
          return 2.2 + 0.3 * (per_sm - 1) + ceil_div(kbt, parts) * std::max(fill, read) +
                 tn * (0.0095 + 0.02 * (parts - 1) / parts);
        };
        const int fit = per_sm == 2 ? kClusters2[parts] : kClusters1[parts], full = (few - 1) / fit;
        if (full > 1 && blocks > 1) break;
        const double t = full * wave(fit) + wave(few - full * fit);
        if (t < best) {
          best = t;
          plan = {DENSE_FEW, tn, parts, per_sm};
        }
      }
  }
  return plan;
}

DenseTiles tile_dense(const DenseGemm& d, const DensePlan& p) {
  DenseTiles t = {};
  t.tm = ceil_div(d.rows, p.tn);
  t.tn = ceil_div(d.cols, (p.kind == DENSE_FEW ? 128 : 256) / (d.epi == DENSE_GATED ? 2 : 1));
  t.whole = t.items = t.tm * t.tn;
  if (p.kind == DENSE_PAIR) {
    if (d.also != nullptr) {
      t.tm2 = ceil_div(d.also->rows, 256);
      t.tn2 = ceil_div(d.also->cols, 256);
    }
    const int tiles = t.tm * t.tn * d.mats + t.tm2 * t.tn2, left = tiles % (kNumSMs / 2);
    const bool cut = left <= kNumSMs / 4;   // a remainder of at most half a wave is cut in two
    t.whole = cut ? tiles - left : tiles;
    t.items = cut ? tiles + left : tiles;
  }
  return t;
}

namespace {

// `FN` may use all the shared memory of a CTA: asked for once per device.
template <auto FN>
cudaError_t allow_shared() {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(FN, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerCta);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <auto FN, typename... P>
cudaError_t launch_cluster(dim3 grid, int threads, int cluster, size_t smem, cudaStream_t stream,
                           const DenseMaps& maps, const DenseArgs& args, P... shape) {
  cudaError_t e = allow_shared<FN>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, FN, maps, args, shape...);
}

template <bool A_MN, bool B_K, int EPI, bool BF>
cudaError_t launch_pair_kernel(const DenseMaps& maps, const DenseArgs& args, cudaStream_t stream) {
  using Cfg = PairCfg<EPI>;
  constexpr int kSmem =
      Cfg::kStages * 2 * (int)kOperand + 8 * (int)Cfg::kWarpBytes + (int)sizeof(PairBars) + 1024;
  static_assert(kSmem <= kSmemPerCta, "ring, store blocks and barriers fit an SM");
  const int pairs = std::min(args.items, kNumSMs / 2);
  return launch_cluster<&dense_pair_kernel<A_MN, B_K, EPI, BF>>(dim3(2 * pairs), kPairThreads, 2, kSmem, stream,
                                                                maps, args);
}

template <bool B_K, int EPI, bool BF>
cudaError_t launch_few(const DensePlan& p, const DenseMaps& maps, const DenseArgs& args,
                       cudaStream_t stream) {
  FewShape fs;
  fs.tn = p.tn;
  fs.tmem = 32;
  // CTAs that wait for columns hold up their cluster, so those that an SM's shared
  // memory lets in, of one launch or several, need no more than its 512: 128 columns
  // come with at least 54 KB, 256 with 104 KB.
  while (fs.tmem < p.tn) fs.tmem *= 2;
  const int stage_bytes = (int)kOperand + p.tn * 128, extra = 1024 + (int)sizeof(FewBars);
  // shared memory of a CTA: half of the SM's 228 KB (less 1 KB a CTA), or what one CTA may have
  const int budget = (p.per_sm == 2 ? kSmemPerSm / 2 - 1024 : kSmemPerCta) - extra;
  // The join: tn tokens x 128 columns of float32, rounded up to whole ranks.
  // Up to 96 tokens (32 where two CTAs share an SM) it has a place of its own, which saves the cluster barrier
  // that says that every ring is free (96 x 4096 -> 4096: 10.6 against 11.1 us);
  // above, the ring would lose too many stages (256 x 4096 -> 4096 in two blocks:
  // 13.6 against 14.1 us; 80 x 4096 -> 22016 with two CTAs an SM: 32 against 44) and
  // it takes the ring's place.
  const int join = ceil_div(p.tn, p.parts) * p.parts * 512;
  fs.join = p.tn <= (p.per_sm == 2 ? 32 : 96) ? join : 0;
  const int fit = std::min(kFewMaxStages, (budget - fs.join) / stage_bytes);
  fs.stages = std::max({2, fs.join > 0 ? 0 : ceil_div(join, stage_bytes),
                        std::min(fit, ceil_div(args.kbt, p.parts))});
  const size_t smem = (size_t)fs.stages * stage_bytes + fs.join + extra;
  return launch_cluster<&dense_few_kernel<B_K, EPI, BF>>(
      dim3((unsigned)p.parts, (unsigned)args.tn, (unsigned)args.tm), kFewThreads, p.parts, smem,
      stream, maps, args, fs);
}

template <bool B_K, int EPI, bool BF>
cudaError_t launch_tall(const DensePlan& p, const DenseMaps& maps, const DenseArgs& args,
                        cudaStream_t stream) {
  const int stage_bytes = (int)kOperand + p.tn * 64, rest = 4 * (int)kTurn + (int)sizeof(TallBars) + 1024;
  const int stages = std::min(kTallMaxStages, (kSmemPerCta - rest) / stage_bytes);
  const int pairs = std::min(args.items, kNumSMs / 2);
  // all of an SM's shared memory, whatever the ring takes: nothing else that uses
  // tensor memory may run beside a CTA that holds all of it
  return launch_cluster<&dense_tall_kernel<B_K, EPI, BF>>(dim3(2 * pairs), kPairThreads, 2, kSmemPerCta, stream,
                                                          maps, args, p.tn, stages);
}

template <bool A_MN, bool B_K, int EPI, bool BF>
cudaError_t launch_as(const DensePlan& p, const DenseMaps& maps, const DenseArgs& args,
                      cudaStream_t stream) {
  if (p.kind == DENSE_PAIR) return launch_pair_kernel<A_MN, B_K, EPI, BF>(maps, args, stream);
  if constexpr (!A_MN)
    return p.kind == DENSE_TALL ? launch_tall<B_K, EPI, BF>(p, maps, args, stream)
                                : launch_few<B_K, EPI, BF>(p, maps, args, stream);
  return cudaErrorInvalidValue;
}

template <bool BF>
cudaError_t launch_typed(const DenseGemm& d, const DensePlan& p, const DenseMaps& maps,
                         const DenseArgs& args, cudaStream_t stream) {
  if (d.epi == DENSE_GATED) return launch_as<false, false, DENSE_GATED, BF>(p, maps, args, stream);
  if (d.epi == DENSE_GRAD) return launch_as<false, true, DENSE_GRAD, BF>(p, maps, args, stream);
  if (d.a_mn) return launch_as<true, false, DENSE_LINEAR, BF>(p, maps, args, stream);
  if (d.b_k) return launch_as<false, true, DENSE_LINEAR, BF>(p, maps, args, stream);
  return launch_as<false, false, DENSE_LINEAR, BF>(p, maps, args, stream);
}

}  // namespace

cudaError_t launch_dense(const DenseGemm& d, cudaStream_t stream) {
  if (!d.a_mn && (d.mats != 1 || d.also != nullptr)) return cudaErrorInvalidValue;   // one weight, one product
  const DensePlan p = plan_dense(d);
  const DenseTiles t = tile_dense(d, p);
  const bool dual = d.epi == DENSE_GATED;
  DenseMaps maps = {};
  DenseArgs a = {};
  a.rows = (int)d.rows;
  a.cols = (int)d.cols;
  a.kb0 = segment_stages(d);
  a.kbt = all_stages(d);
  const bool pair = p.kind == DENSE_PAIR;
  a.tm = t.tm;
  a.tn = t.tn;
  a.tm2 = t.tm2;
  a.tn2 = t.tn2;
  a.whole = t.whole;
  a.items = t.items;
  a.mats = d.mats;
  a.group = kGroupTiles;
  if (d.also != nullptr) {
    a.rows2 = (int)d.also->rows;
    a.cols2 = (int)d.also->cols;
  }
  a.outs = dual ? (d.o[1] != nullptr ? 3 : 1) : 1;
  a.act = d.act;
  a.plain = d.bias == nullptr && d.act == SIG_ACT_NONE && d.residual == nullptr;
  a.bias = d.bias;
  a.residual = d.residual;
  a.ldr = d.ldr;
  a.g = d.g;
  a.u = d.u;
  a.ldo = d.ldo;
  for (int i = 0; i < 3; ++i) a.o[i] = d.o[i];
  const int n_a = d.two_segments ? 2 : 1, n_b = (d.two_segments || d.mats == 2 || dual) ? 2 : 1;
  for (int i = 0; i < n_a; ++i)
    if (!(d.a_mn ? map16(&maps.a[i], d.a[i], d.rows, d.K, d.lda, kSlab)
                 : map16(&maps.a[i], d.a[i], d.K, d.rows, d.lda,
                          pair ? kTile : p.kind == DENSE_TALL ? p.tn / 2 : p.tn)))
      return cudaErrorInvalidValue;
  for (int i = 0; i < n_b; ++i)
    if (!(d.b_k ? map16(&maps.b[i], d.b[i], d.K, d.cols, d.ldb, pair ? 64 : kTile)
                : map16(&maps.b[i], d.b[i], d.cols, d.K, d.ldb, kSlab)))
      return cudaErrorInvalidValue;
  // the kernels prefetch every map: the unused ones repeat another
  if (n_a < 2) maps.a[1] = maps.a[0];
  if (n_b < 2) maps.b[1] = maps.b[0];
  maps.b[2] = maps.b[0];
  if (pair) {   // the pair kernel reads its other inputs and stores its outputs with TMA
    const int width = d.epi == DENSE_GRAD ? 32 : 64;
    const uint16_t* r[2] = {d.epi == DENSE_GRAD ? d.g : d.residual, d.epi == DENSE_GRAD ? d.u : nullptr};
    for (int i = 0; i < 3; ++i)
      if (d.o[i] == nullptr)
        maps.o[i] = maps.o[0];
      else if (!map16(&maps.o[i], d.o[i], d.cols, d.rows, d.ldo, 32, width))
        return cudaErrorInvalidValue;
    for (int i = 0; i < 2; ++i)
      if (r[i] == nullptr)
        maps.r[i] = maps.o[0];
      else if (!map16(&maps.r[i], r[i], d.cols, d.rows, d.epi == DENSE_GRAD ? d.cols : d.ldr, 32, width))
        return cudaErrorInvalidValue;
    if (const DenseGemm* e = d.also; e != nullptr) {
      if (!d.a_mn || !e->a_mn || d.b_k || e->b_k || d.K != e->K) return cudaErrorInvalidValue;
      if (!map16(&maps.a[1], e->a[0], e->rows, e->K, e->lda, kSlab) ||
          !map16(&maps.b[2], e->b[0], e->cols, e->K, e->ldb, kSlab) ||
          !map16(&maps.o[2], e->o[0], e->cols, e->rows, e->ldo, 32))
        return cudaErrorInvalidValue;
    }
  }
  return d.bf16 ? launch_typed<true>(d, p, maps, a, stream) : launch_typed<false>(d, p, maps, a, stream);
}

cudaError_t set_dense_wait_limit(long long cycles) {
  const long long v = cycles > 0 ? cycles : kDenseTimeout;
  return cudaMemcpyToSymbol(g_dense_wait_limit, &v, sizeof(v));
}

cudaError_t read_dense_error(unsigned* out, cudaStream_t stream) {
  cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_dense_error, sizeof(unsigned), 0,
                                            cudaMemcpyDeviceToHost, stream);
  if (e != cudaSuccess) return e;
  e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return e;
  const unsigned zero = 0;
  return cudaMemcpyToSymbolAsync(g_dense_error, &zero, sizeof(unsigned), 0, cudaMemcpyHostToDevice,
                                 stream);
}

}  // namespace sig

// Dense products for blocks of tokens: Y = act(X WT + bias) + residual, the
// gate and up projections of a gated MLP with the activation and the product
// of the two in the epilogue, and the products of its backward pass.
//
// Two kernels.  dense_pair_kernel is persistent: one CTA pair per SM pair
// walks 256 x 256 output tiles with two accumulators in tensor memory, so the
// epilogue of a tile runs beside the mainloop of the next.
// dense_split_kernel serves small blocks of tokens: one 128 x BN tile per
// cluster, the cluster's CTAs each taking a part of K and joining their
// sums through distributed shared memory in a fixed order.
#include "common.cuh"
#include "dense.h"
#include "internal.h"
#include "tc.cuh"

#include <cuda_bf16.h>

#include <algorithm>

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
  CUtensorMap a[2], b[2], o[3];
};

struct DenseArgs {
  int rows, cols;      // of one output
  int kb0, kbt;        // K stages of the first segment, of both
  int tm, tn;          // tiles down and across (of one weight)
  int mats;
  int outs;            // outputs to store (DENSE_GATED: 1, or 3 with g and u)
  int act;
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

__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (try_cluster(bar, parity)) return true;
  const long long t0 = clock64();
  const long long limit = *(volatile long long*)&g_dense_wait_limit;
  while (!try_cluster(bar, parity)) {
    if (*abort_flag) return false;
    if (clock64() - t0 > limit) {
      *abort_flag = 1;
      atomicOr(&g_dense_error, 1u);
      return false;
    }
  }
  return true;
}

// Not cut short by a give-up: lets issued copies and MMAs finish.
__device__ __forceinline__ bool wait_drain(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!try_cluster(bar, parity))
    if (clock64() - t0 > kDenseTimeout) return false;
  return true;
}

__device__ __forceinline__ void arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
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

// Shared-memory descriptor of K step k (16 values) of an operand slab.
// K-major: rows of 128 bytes, the step 32 bytes into each; MN-major: blocks of
// 64 columns x 64 k-rows (kBlock bytes apart), the step 16 k-rows down.
template <bool MN>
__device__ __forceinline__ uint64_t slab_desc(uint32_t base, int k) {
  return MN ? smem_desc(base + k * 2048, kBlock, 1024) : smem_desc(base + k * 32, 16, 1024);
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

// 32 accumulator columns of this warp's 32 rows (one row a lane).
__device__ __forceinline__ void tmem_ld32(float (&v)[32], uint32_t addr) {
  uint32_t r[32];
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
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
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

constexpr float kInvSqrt2 = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kGeluC = 0.79788456080286536f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// act(z) = z p(z); p is the share that passes (1, [z > 0], the logistic
// function, the normal distribution function, or the logistic of the tanh
// form: (1 + tanh v) / 2 = 1 / (1 + exp(-2 v))).
template <int ACT>
__device__ __forceinline__ float act_share(float z) {
  if constexpr (ACT == SIG_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  if constexpr (ACT == SIG_ACT_SILU) return 1.f / (1.f + __expf(-z));
  if constexpr (ACT == SIG_ACT_GELU) return 0.5f * erfcf(-z * kInvSqrt2);
  if constexpr (ACT == SIG_ACT_GELU_TANH)
    return 1.f / (1.f + __expf(-2.f * kGeluC * z * fmaf(kGeluA * z, z, 1.f)));
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
  if constexpr (ACT == SIG_ACT_GELU) return fmaf(z * kInvSqrt2Pi, __expf(-0.5f * z * z), p);
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

// v[0 .. 8 G) = act(v + bias) + residual for 8 G columns from `col` of `row`;
// columns from `cols` on and rows from `rows` on are left without the two.
template <bool BF, int G>
__device__ __forceinline__ void epi_linear(float* v, const DenseArgs& a, int row, int col) {
  uint4 res[G];
  const bool has_res = a.residual != nullptr && row < a.rows;
#pragma unroll
  for (int j = 0; j < G; ++j)
    res[j] = has_res && col + 8 * j < a.cols
                 // plain load: Y may be the residual buffer itself
                 ? *reinterpret_cast<const uint4*>(a.residual + (int64_t)row * a.ldr + col + 8 * j)
                 : make_uint4(0, 0, 0, 0);
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
      for (int i = 0; i < 8 * G; ++i) v[i] = act_value<decltype(A)::value>(v[i], act_share<decltype(A)::value>(v[i]));
    });
  if (a.residual != nullptr) {
#pragma unroll
    for (int j = 0; j < G; ++j) {
      float r[8];
      unpack8<BF>(r, res[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[8 * j + i] += r[i];
    }
  }
}

// g <- act(g) u over n columns
template <int n>
__device__ __forceinline__ void epi_gated(float* g, const float* u, int act) {
  with_act(act, [&](auto A) {
#pragma unroll
    for (int i = 0; i < n; ++i) g[i] = act_value<decltype(A)::value>(g[i], act_share<decltype(A)::value>(g[i])) * u[i];
  });
}

// dh -> (dg, du, h) over 8 columns
template <bool BF>
__device__ __forceinline__ void epi_grad8(const float* dh, const uint4& gv, const uint4& uv, int act,
                                          uint4& dg, uint4& du, uint4& h) {
  float g[8], u[8], a0[8], a1[8], a2[8];
  unpack8<BF>(g, gv);
  unpack8<BF>(u, uv);
  with_act(act, [&](auto A) {
    constexpr int ACT = decltype(A)::value;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float p = act_share<ACT>(g[i]), v = act_value<ACT>(g[i], p);
      a0[i] = dh[i] * u[i] * act_slope<ACT>(g[i], p);
      a1[i] = dh[i] * v;
      a2[i] = v * u[i];
    }
  });
  dg = pack8<BF>(a0);
  du = pack8<BF>(a1);
  h = pack8<BF>(a2);
}

// ---------------------------------------------------------------------------
// Persistent CTA-pair kernel, 256 x 256 tiles
// ---------------------------------------------------------------------------
constexpr int kPairStages = 6;
constexpr int kPairThreads = 320;                  // 8 epilogue warps, one loads, one issues MMAs
constexpr uint32_t kOperand = kTile * kSlab * 2;   // 16 KB: 128 rows (or columns) x 64 K
constexpr uint32_t kPairStageBytes = 2 * kOperand;
constexpr int kGroupRows = 8;                      // row tiles walked together (L2 reuse of B)

struct __align__(1024) PairShared {
  uint8_t A[kPairStages][kOperand];
  uint8_t B[kPairStages][kOperand];
  uint8_t stage[8][4096];                          // per epilogue warp: 32 rows x 64 columns
  unsigned long long full[kPairStages];            // used in the leader
  unsigned long long empty[kPairStages];
  unsigned long long acc_full[2], acc_empty[2];    // acc_empty used in the leader
  unsigned long long done;
  uint32_t tmem_base;
  int abort_flag;
  int consumed;
};

struct TilePos {
  int m, n;
};

__device__ __forceinline__ TilePos tile_at(int t, int tm, int tn_all) {
  const int per = kGroupRows * tn_all;
  const int g0 = t / per * kGroupRows, r = t % per;
  const int gs = min(kGroupRows, tm - g0);
  return {g0 + r % gs, r / gs};
}

// Write 32 rows x 32 columns (16 packed words a lane) into a warp's staging
// block at column 32 * part, in the 128-byte swizzled order of the store map.
__device__ __forceinline__ void stage_words(uint32_t stage, int lane, int part, const uint4 (&p)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t addr = stage + (uint32_t)lane * 128u + (uint32_t)(((part * 4 + j) ^ (lane & 7)) << 4);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(p[j].x), "r"(p[j].y),
                 "r"(p[j].z), "r"(p[j].w)
                 : "memory");
  }
}

// The staging block is free once the stores before have read it.
__device__ __forceinline__ void stage_wait(int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
}

__device__ __forceinline__ void stage_store(uint32_t stage, int lane, const CUtensorMap* map, int col,
                                            int row, const DenseArgs& a) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (lane == 0) {
    if (row < a.rows && col < a.cols) tma_store_2d(map, stage, col, row);   // the map clips the rest
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}

template <bool A_MN, bool B_K, int EPI, bool BF>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
dense_pair_kernel(const __grid_constant__ DenseMaps maps, const __grid_constant__ DenseArgs args) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  PairShared& sm = *reinterpret_cast<PairShared*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int tn_all = args.tn * args.mats, tiles = args.tm * tn_all;
  volatile int* abort_flag = &sm.abort_flag;
  pdl_trigger();

  if (tid == 0) {
    for (int s = 0; s < kPairStages; ++s) {
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
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sm.tmem_base)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  __syncwarp();
  cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = sm.tmem_base;
  pdl_wait();

  int issued = 0;   // stages whose copies this CTA's producer has issued
  if (warp == 8) {
    if (lane == 0) {   // ---- TMA producer (both CTAs) ----
      for (int t = pair; t < tiles && !*abort_flag; t += pairs) {
        const TilePos p = tile_at(t, args.tm, tn_all);
        const int m0 = p.m * 256 + (int)rank * 128;
        const int mat = p.n / args.tn, nt = p.n - mat * args.tn;
        const int nb = EPI == DENSE_GATED ? nt * 128 : nt * 256 + (int)rank * 128;
        for (int kb = 0; kb < args.kbt; ++kb) {
          const int s = issued % kPairStages;
          const uint32_t ph = (uint32_t)(issued / kPairStages) & 1u;
          if (!wait_bounded(smem_u32(&sm.empty[s]), ph ^ 1u, abort_flag)) break;
          const int seg = kb >= args.kb0 ? 1 : 0;
          const int k = (kb - (seg ? args.kb0 : 0)) * kSlab;
          const CUtensorMap* ma = &maps.a[seg];
          const CUtensorMap* mb = &maps.b[EPI == DENSE_GATED ? (int)rank : seg | mat];
          const uint32_t fb = map_to_rank(smem_u32(&sm.full[s]), 0);
          if (leader) mbar_expect_tx(smem_u32(&sm.full[s]), 2 * kPairStageBytes);
          if constexpr (A_MN) {
            tma_load_2d_pair(smem_u32(sm.A[s]), ma, m0, k, fb);
            tma_load_2d_pair(smem_u32(sm.A[s]) + kBlock, ma, m0 + 64, k, fb);
          } else {
            tma_load_2d_pair(smem_u32(sm.A[s]), ma, k, m0, fb);
          }
          if constexpr (B_K) {
            tma_load_2d_pair(smem_u32(sm.B[s]), mb, k, nb, fb);
          } else {
            tma_load_2d_pair(smem_u32(sm.B[s]), mb, nb, k, fb);
            tma_load_2d_pair(smem_u32(sm.B[s]) + kBlock, mb, nb + 64, k, fb);
          }
          ++issued;
        }
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    if (leader && lane == 0) {   // ---- MMA issuer ----
      constexpr uint32_t idesc = dense_idesc(256, 256, BF, A_MN, B_K);
      int it = 0, count = 0;
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs, ++count) {
        const int slot = count & 1;
        if (!wait_bounded(smem_u32(&sm.acc_empty[slot]), ((uint32_t)(count >> 1) & 1u) ^ 1u, abort_flag))
          break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t d = tmem + (uint32_t)slot * 256u;
        for (int kb = 0; kb < args.kbt; ++kb, ++it) {
          const int s = it % kPairStages;
          ok = wait_bounded(smem_u32(&sm.full[s]), (uint32_t)(it / kPairStages) & 1u, abort_flag);
          if (!ok) break;
          *(volatile int*)&sm.consumed = it + 1;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t a0 = smem_u32(sm.A[s]), b0 = smem_u32(sm.B[s]);
#pragma unroll
          for (int k = 0; k < kSlab / 16; ++k)
            mma_f16<2>(d, slab_desc<A_MN>(a0, k), slab_desc<!B_K>(b0, k), idesc,
                       (kb > 0 || k > 0) ? 1u : 0u);
          commit_pair(smem_u32(&sm.empty[s]));
        }
        if (ok) commit_pair(smem_u32(&sm.acc_full[slot]));
      }
      commit_pair(smem_u32(&sm.done));   // completes once every issued MMA has finished
    }
    __syncwarp();
  } else {   // ---- epilogue: eight warps, each 32 rows x half of the columns ----
    const int q = warp & 3, half = warp >> 2;
    const uint32_t stage = smem_u32(sm.stage[warp]);
    const uint32_t empty0 = map_to_rank(smem_u32(&sm.acc_empty[0]), 0);
    const uint32_t empty1 = map_to_rank(smem_u32(&sm.acc_empty[1]), 0);
    int count = 0;
    for (int t = pair; t < tiles; t += pairs, ++count) {
      const TilePos p = tile_at(t, args.tm, tn_all);
      const int row0 = p.m * 256 + (int)rank * 128 + q * 32, row = row0 + lane;
      const int mat = p.n / args.tn, nt = p.n - mat * args.tn;
      const int slot = count & 1;
      // one verdict for the warp: the tensor-memory loads below need all its lanes
      if (!__all_sync(kFull, wait_bounded(smem_u32(&sm.acc_full[slot]), (uint32_t)(count >> 1) & 1u,
                                          abort_flag)))
        break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t acc = tmem + (uint32_t)slot * 256u + ((uint32_t)(q * 32) << 16);
      auto release = [&] {   // this warp has read its part of the accumulator
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) arrive_remote(slot ? empty1 : empty0);
      };
      if constexpr (EPI == DENSE_LINEAR) {
#pragma unroll 1
        for (int blk = 0; blk < 2; ++blk) {
          const int c = half * 128 + blk * 64, col = nt * 256 + c;
          stage_wait(lane);
#pragma unroll 1
          for (int part = 0; part < 2; ++part) {
            float v[32];
            tmem_ld32(v, acc + (uint32_t)(c + part * 32));
            if (blk == 1 && part == 1) release();
            epi_linear<BF, 4>(v, args, row, col + part * 32);
            uint4 w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = pack8<BF>(*reinterpret_cast<float(*)[8]>(&v[8 * j]));
            stage_words(stage, lane, part, w);
          }
          stage_store(stage, lane, &maps.o[mat], col, row0, args);
        }
      } else if constexpr (EPI == DENSE_GATED) {
        // columns [0, 128) are g and [128, 256) are u of 128 hidden columns
        const int c = half * 64, col = nt * 128 + c;
#pragma unroll 1
        for (int out = 0; out < args.outs; ++out) {
          stage_wait(lane);
#pragma unroll 1
          for (int part = 0; part < 2; ++part) {
            float v[32];
            tmem_ld32(v, acc + (uint32_t)(c + part * 32 + (out == 2 ? 128 : 0)));
            if (out == 0) {
              float u[32];
              tmem_ld32(u, acc + (uint32_t)(128 + c + part * 32));
              if (args.outs == 1 && part == 1) release();
              epi_gated<32>(v, u, args.act);
            } else if (out == 2 && part == 1) {
              release();
            }
            uint4 w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = pack8<BF>(*reinterpret_cast<float(*)[8]>(&v[8 * j]));
            stage_words(stage, lane, part, w);
          }
          stage_store(stage, lane, &maps.o[out], col, row0, args);
        }
      } else {
#pragma unroll 1
        for (int blk = 0; blk < 2; ++blk) {
          const int c = half * 128 + blk * 64, col = nt * 256 + c;
          uint4 w[3][2][4];
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            uint4 gv[4], uv[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int cj = col + part * 32 + 8 * j;
              const bool in = row < args.rows && cj < args.cols;
              const int64_t at = (int64_t)row * args.cols + cj;
              gv[j] = in ? ld16(args.g + at) : make_uint4(0, 0, 0, 0);
              uv[j] = in ? ld16(args.u + at) : make_uint4(0, 0, 0, 0);
            }
            float v[32];
            tmem_ld32(v, acc + (uint32_t)(c + part * 32));
            if (blk == 1 && part == 1) release();
#pragma unroll
            for (int j = 0; j < 4; ++j)
              epi_grad8<BF>(&v[8 * j], gv[j], uv[j], args.act, w[0][part][j], w[1][part][j],
                            w[2][part][j]);
          }
#pragma unroll
          for (int out = 0; out < 3; ++out) {
            stage_wait(lane);
            stage_words(stage, lane, 0, w[out][0]);
            stage_words(stage, lane, 1, w[out][1]);
            stage_store(stage, lane, &maps.o[out], col, row0, args);
          }
        }
      }
    }
    // the outputs are written before the CTA ends
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }

  __syncthreads();
  wait_drain(smem_u32(&sm.done), 0u);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 8 && lane == 0 && *abort_flag) {
    // after a give-up: the copies that were issued land before shared memory goes
    if (leader)
      for (int it = *(volatile int*)&sm.consumed; it < issued; ++it)
        wait_drain(smem_u32(&sm.full[it % kPairStages]), (uint32_t)(it / kPairStages) & 1u);
    const long long t0 = clock64();
    while (clock64() - t0 < 40000) {
    }
  }
  __syncthreads();
  cluster_sync();
  if (warp == 8)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u)
                 : "memory");
}

// ---------------------------------------------------------------------------
// Split-K cluster kernel, one 128 x BN tile per cluster
// ---------------------------------------------------------------------------
constexpr int kSplitThreads = 256;

template <int BN>
struct SplitCfg {
  static constexpr int kStages = BN == 256 ? 4 : BN == 128 ? 3 : 4;
  static constexpr uint32_t kBBytes = BN * kSlab * 2;
  static constexpr uint32_t kStageBytes = kOperand + kBBytes;
};

template <int BN>
struct __align__(1024) SplitShared {
  using C = SplitCfg<BN>;
  uint8_t A[C::kStages][kOperand];
  uint8_t B[C::kStages][C::kBBytes];
  unsigned long long full[C::kStages];
  unsigned long long empty[C::kStages];
  unsigned long long accum;
  uint32_t tmem_base;
  int abort_flag;
  int consumed;
};

__device__ __forceinline__ void st_cluster_v4(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c),
               "f"(d)
               : "memory");
}

template <bool BF>
__device__ __forceinline__ void store8(uint16_t* o, int64_t at, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(o + at) = pack8<BF>(v);
}

template <bool B_K, int EPI, bool BF, int BN>
__global__ void __launch_bounds__(kSplitThreads)
dense_split_kernel(const __grid_constant__ DenseMaps maps, const __grid_constant__ DenseArgs args,
                   int log2c) {
  using C = SplitCfg<BN>;
  constexpr int S = C::kStages;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  SplitShared<BN>& sm = *reinterpret_cast<SplitShared<BN>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)blockIdx.x;          // the cluster spans the grid's x
  const int mat = (int)blockIdx.y / args.tn, nt = (int)blockIdx.y - mat * args.tn;
  const int m0 = (int)blockIdx.z * kTile;
  constexpr int kOutCols = EPI == DENSE_GATED ? BN / 2 : BN;   // output columns of the tile
  const int n0 = nt * kOutCols;
  // this CTA's part of the K stages
  const int kb_lo = (int)(((int64_t)args.kbt * rank) >> log2c);
  const int kb_hi = (int)(((int64_t)args.kbt * (rank + 1)) >> log2c);
  const int steps = kb_hi - kb_lo;
  volatile int* abort_flag = &sm.abort_flag;
  pdl_trigger();

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
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sm.tmem_base)),
                 "r"(BN)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = sm.tmem_base;
  pdl_wait();

  int issued = 0;
  if (warp == 0) {
    if (lane == 0) {   // ---- TMA producer ----
      for (int i = 0; i < steps; ++i) {
        const int s = i % S, kb = kb_lo + i;
        if (!wait_bounded(smem_u32(&sm.empty[s]), ((uint32_t)(i / S) & 1u) ^ 1u, abort_flag)) break;
        const int seg = kb >= args.kb0 ? 1 : 0;
        const int k = (kb - (seg ? args.kb0 : 0)) * kSlab;
        const uint32_t fb = smem_u32(&sm.full[s]), b0 = smem_u32(sm.B[s]);
        mbar_expect_tx(fb, C::kStageBytes);
        tma_load_2d(smem_u32(sm.A[s]), &maps.a[seg], k, m0, fb);
        if constexpr (EPI == DENSE_GATED) {
#pragma unroll
          for (int j = 0; j < BN / 64; ++j) {
            constexpr int kHalf = BN / 128;   // 64-column blocks of each weight
            tma_load_2d(b0 + j * kBlock, &maps.b[j / kHalf], n0 + (j % kHalf) * 64, k, fb);
          }
        } else if constexpr (B_K) {
          tma_load_2d(b0, &maps.b[seg | mat], k, n0, fb);
        } else {
#pragma unroll
          for (int j = 0; j < BN / 64; ++j)
            tma_load_2d(b0 + j * kBlock, &maps.b[seg | mat], n0 + j * 64, k, fb);
        }
        ++issued;
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {   // ---- MMA issuer ----
      constexpr uint32_t idesc = dense_idesc(kTile, BN, BF, false, B_K);
      for (int i = 0; i < steps; ++i) {
        const int s = i % S;
        if (!wait_bounded(smem_u32(&sm.full[s]), (uint32_t)(i / S) & 1u, abort_flag)) break;
        *(volatile int*)&sm.consumed = i + 1;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t a0 = smem_u32(sm.A[s]), b0 = smem_u32(sm.B[s]);
#pragma unroll
        for (int k = 0; k < kSlab / 16; ++k)
          mma_f16<1>(tmem, slab_desc<false>(a0, k), slab_desc<!B_K>(b0, k), idesc,
                     (i > 0 || k > 0) ? 1u : 0u);
        commit_one(smem_u32(&sm.empty[s]));
      }
      commit_one(smem_u32(&sm.accum));   // completes once every issued MMA has finished
    }
    __syncwarp();
  }

  const bool acc_done = wait_drain(smem_u32(&sm.accum), 0u);
  __syncwarp();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const int valid = min(kTile, args.rows - m0);    // rows of this tile
  const int q = warp & 3, half = warp >> 2;
  const int row = m0 + q * 32 + lane;
  const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16);
  // one verdict for the CTA: the tensor-memory loads below need whole warps
  const bool ok = __syncthreads_and(acc_done && !*abort_flag) != 0;

  if (log2c == 0) {
    // the tile's sums are complete: straight from tensor memory to the outputs
    if (ok && q * 32 < valid) {
#pragma unroll 1
      for (int cc = 0; cc < kOutCols / 2; cc += 32) {
        const int c = half * (kOutCols / 2) + cc, col = n0 + c;
        float v[32];
        if constexpr (EPI == DENSE_LINEAR) {
          tmem_ld32(v, acc + (uint32_t)c);
          epi_linear<BF, 4>(v, args, row, col);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (row < args.rows && col + 8 * j < args.cols)
              store8<BF>(args.o[mat], (int64_t)row * args.ldo + col + 8 * j,
                         *reinterpret_cast<float(*)[8]>(&v[8 * j]));
        } else if constexpr (EPI == DENSE_GATED) {
          float u[32];
          tmem_ld32(v, acc + (uint32_t)c);
          tmem_ld32(u, acc + (uint32_t)(BN / 2 + c));
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (row < args.rows && col + 8 * j < args.cols) {
              const int64_t at = (int64_t)row * args.ldo + col + 8 * j;
              if (args.outs == 3) {
                store8<BF>(args.o[1], at, *reinterpret_cast<float(*)[8]>(&v[8 * j]));
                store8<BF>(args.o[2], at, *reinterpret_cast<float(*)[8]>(&u[8 * j]));
              }
            }
          epi_gated<32>(v, u, args.act);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (row < args.rows && col + 8 * j < args.cols)
              store8<BF>(args.o[0], (int64_t)row * args.ldo + col + 8 * j,
                         *reinterpret_cast<float(*)[8]>(&v[8 * j]));
        } else {
          tmem_ld32(v, acc + (uint32_t)c);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (row < args.rows && col + 8 * j < args.cols) {
              const int64_t at = (int64_t)row * args.ldo + col + 8 * j;
              uint4 dg, du, h;
              epi_grad8<BF>(&v[8 * j], ld16(args.g + at), ld16(args.u + at), args.act, dg, du, h);
              *reinterpret_cast<uint4*>(args.o[0] + at) = dg;
              *reinterpret_cast<uint4*>(args.o[1] + at) = du;
              *reinterpret_cast<uint4*>(args.o[2] + at) = h;
            }
        }
      }
    }
  } else {
    // Join: rank r owns output columns [r W, (r + 1) W) of the tile.  Every
    // CTA sends its sums of those columns to r's shared memory (the ring, free
    // once every CTA's MMAs are done), and r adds them in rank order.
    const int lw = (EPI == DENSE_GATED ? 31 - __clz(BN / 2) : 31 - __clz(BN)) - log2c;   // log2 W
    const int W = 1 << lw;
    const int pitch = EPI == DENSE_GATED ? 2 * W : W;      // floats of a row in the join buffer
    const int swz = min(8, pitch / 4) - 1;
    const uint32_t buf = smem_u32(sm.A[0]);
    cluster_sync();
    if (ok && q * 32 < valid) {
#pragma unroll 1
      for (int cc = 0; cc < BN / 2; cc += 32) {
        const int c = half * (BN / 2) + cc;
        float v[32];
        tmem_ld32(v, acc + (uint32_t)c);
        if (row < args.rows) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int cj = (EPI == DENSE_GATED ? c - half * (BN / 2) : c) + 4 * j;
            const int owner = cj >> lw;
            const int lc = (cj & (W - 1)) + (EPI == DENSE_GATED && half ? W : 0);
            const int chunk = (lc >> 2) ^ (lane & swz);
            const uint32_t at = buf + (uint32_t)(((rank * kTile + q * 32 + lane) * pitch + chunk * 4) * 4);
            st_cluster_v4(map_to_rank(at, (uint32_t)owner), v[4 * j], v[4 * j + 1], v[4 * j + 2],
                          v[4 * j + 3]);
          }
        }
      }
    }
    cluster_sync();
    if (ok) {
      const int chunks = W >> 3;   // 8-column chunks of a row
      const int ranks = 1 << log2c;
      for (int i = tid; i < valid * chunks; i += kSplitThreads) {
        const int r = i / chunks, ch = i - r * chunks;
        const int col = n0 + rank * W + ch * 8;
        if (col >= args.cols) continue;
        auto gather = [&](float (&v)[8], int first) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = 0.f;
          for (int src = 0; src < ranks; ++src) {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const int chunk = ((first >> 2) + hh) ^ (r & swz);
              const float4 f = *reinterpret_cast<const float4*>(
                  &sm.A[0][0] + (size_t)((src * kTile + r) * pitch + chunk * 4) * 4);
              v[4 * hh] += f.x; v[4 * hh + 1] += f.y; v[4 * hh + 2] += f.z; v[4 * hh + 3] += f.w;
            }
          }
        };
        const int64_t at = (int64_t)(m0 + r) * args.ldo + col;
        float v[8];
        gather(v, ch * 8);
        if constexpr (EPI == DENSE_LINEAR) {
          epi_linear<BF, 1>(v, args, m0 + r, col);
          store8<BF>(args.o[mat], at, v);
        } else if constexpr (EPI == DENSE_GATED) {
          float u[8];
          gather(u, W + ch * 8);
          if (args.outs == 3) {
            store8<BF>(args.o[1], at, v);
            store8<BF>(args.o[2], at, u);
          }
          epi_gated<8>(v, u, args.act);
          store8<BF>(args.o[0], at, v);
        } else {
          uint4 dg, du, h;
          epi_grad8<BF>(v, ld16(args.g + at), ld16(args.u + at), args.act, dg, du, h);
          *reinterpret_cast<uint4*>(args.o[0] + at) = dg;
          *reinterpret_cast<uint4*>(args.o[1] + at) = du;
          *reinterpret_cast<uint4*>(args.o[2] + at) = h;
        }
      }
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (tid == 0 && *abort_flag)
    for (int i = *(volatile int*)&sm.consumed; i < issued; ++i)
      wait_drain(smem_u32(&sm.full[i % S]), (uint32_t)(i / S) & 1u);
  __syncthreads();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(BN)
                 : "memory");
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// 2-D map over 16-bit values: `inner` contiguous, `outer` rows `pitch` apart,
// box 64 x `box` rows, 128-byte swizzle, zeros outside.
bool map16(CUtensorMap* map, const void* base, int64_t inner, int64_t outer, int64_t pitch, int box) {
  auto enc = get_encode();
  if (enc == nullptr) return false;
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  cuuint64_t strides[1] = {(cuuint64_t)pitch * 2};
  cuuint32_t boxes[2] = {64, (cuuint32_t)box};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(base), dims, strides, boxes,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a product is run: the pair kernel, or the split kernel with tiles of bn
// columns and 2^log2c CTAs along K.
struct DensePlan {
  bool pair;
  int bn, log2c;
};

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

DensePlan plan_dense(const DenseGemm& d, int kbt) {
  if (d.a_mn) return {true, 256, 0};
  const int shrink = d.epi == DENSE_GATED ? 2 : 1;   // accumulator columns per output column
  const int64_t pair_tiles = (int64_t)ceil_div(d.rows, 256) * ceil_div(d.cols * shrink, 256) * d.mats;
  if (pair_tiles > kNumSMs / 4 && d.rows > 128) return {true, 256, 0};
  DensePlan best{true, 256, 0};
  double best_cost = 1e30;
  for (int bn : {128, 256}) {
    for (int l = 0; l <= 3; ++l) {
      if ((1 << l) > kbt) break;
      const int64_t ctas = (int64_t)ceil_div(d.rows, kTile) * ceil_div(d.cols * shrink, bn) * d.mats << l;
      const int slots = kNumSMs * (bn == 128 ? 2 : 1);
      const double waves = (double)ceil_div(ctas, slots);
      const double cost = waves * (((double)kbt / (1 << l)) * (bn + 128) + 2000.0) * (bn == 128 ? 2 : 1);
      if (cost < best_cost) {
        best_cost = cost;
        best = {false, bn, l};
      }
    }
  }
  return best;
}

template <bool A_MN, bool B_K, int EPI, bool BF>
cudaError_t launch_pair_kernel(const DenseMaps& maps, const DenseArgs& args, cudaStream_t stream) {
  auto fn = dense_pair_kernel<A_MN, B_K, EPI, BF>;
  const size_t smem = sizeof(PairShared) + 1024;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)args.tm * args.tn * args.mats;
  const int pairs = (int)std::min<int64_t>(tiles, kNumSMs / 2);
  e = launch_pdl(fn, dim3(2 * pairs), dim3(kPairThreads), smem, stream, maps, args);
  return e != cudaSuccess ? e : cudaPeekAtLastError();
}

template <bool B_K, int EPI, bool BF, int BN>
cudaError_t launch_split_bn(const DenseMaps& maps, const DenseArgs& args, int log2c,
                            cudaStream_t stream) {
  auto fn = dense_split_kernel<B_K, EPI, BF, BN>;
  const size_t smem = sizeof(SplitShared<BN>) + 1024;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1u << log2c, (unsigned)(args.tn * args.mats), (unsigned)args.tm);
  cfg.blockDim = dim3(kSplitThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1u << log2c;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, fn, maps, args, log2c);
  return e != cudaSuccess ? e : cudaPeekAtLastError();
}

template <bool A_MN, bool B_K, int EPI, bool BF>
cudaError_t launch_as(const DensePlan& p, const DenseMaps& maps, const DenseArgs& args,
                      cudaStream_t stream) {
  if (p.pair) return launch_pair_kernel<A_MN, B_K, EPI, BF>(maps, args, stream);
  if constexpr (!A_MN) {
    if (p.bn == 256) return launch_split_bn<B_K, EPI, BF, 256>(maps, args, p.log2c, stream);
    return launch_split_bn<B_K, EPI, BF, 128>(maps, args, p.log2c, stream);
  }
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
  const int kb = ceil_div(d.K, kSlab), kbt = d.two_segments ? 2 * kb : kb;
  const DensePlan p = plan_dense(d, kbt);
  const bool dual = d.epi == DENSE_GATED;
  DenseMaps maps = {};
  DenseArgs a = {};
  a.rows = (int)d.rows;
  a.cols = (int)d.cols;
  a.kb0 = kb;
  a.kbt = kbt;
  a.tm = ceil_div(d.rows, p.pair ? 256 : kTile);
  a.tn = ceil_div(d.cols, dual ? p.bn / 2 : p.bn);
  a.mats = d.mats;
  a.outs = dual ? (d.o[1] != nullptr ? 3 : 1) : 1;
  a.act = d.act;
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
                 : map16(&maps.a[i], d.a[i], d.K, d.rows, d.lda, kTile)))
      return cudaErrorInvalidValue;
  for (int i = 0; i < n_b; ++i)
    if (!(d.b_k ? map16(&maps.b[i], d.b[i], d.K, d.cols, d.ldb, p.pair ? 128 : p.bn)
                : map16(&maps.b[i], d.b[i], d.cols, d.K, d.ldb, kSlab)))
      return cudaErrorInvalidValue;
  if (p.pair)   // the pair kernel stores its outputs with TMA
    for (int i = 0; i < 3; ++i)
      if (d.o[i] != nullptr && !map16(&maps.o[i], d.o[i], d.cols, d.rows, d.ldo, 32))
        return cudaErrorInvalidValue;
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

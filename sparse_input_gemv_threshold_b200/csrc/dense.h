// Internal interface of the dense products for blocks of tokens (dense.cu):
// linear_act, gated_mlp and gated_mlp_backward call these launchers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace sig {

// What happens to the accumulators of a product.
enum DenseEpilogue : int {
  DENSE_LINEAR = 0,   // y = act(acc + bias) + residual
  DENSE_GATED = 1,    // two accumulators g, u: h = act(g) u (and g, u themselves on request)
  DENSE_GRAD = 2      // acc = dh, g and u given: dg = dh u act'(g), du = dh act(g), h = act(g) u
};

// One product of `rows` x `cols` outputs over K (two K segments with
// `two_segments`; with a_mn, two column blocks of `cols` when `mats` is 2).
struct DenseGemm {
  int epi = DENSE_LINEAR;
  bool bf16 = false;
  int64_t rows = 0, cols = 0, K = 0;
  // A: rows x K with K contiguous (a_mn false), or K x rows with rows contiguous
  bool a_mn = false;
  const uint16_t* a[2] = {};
  int64_t lda = 0;
  // B: K x cols with cols contiguous (b_k false), or cols x K with K contiguous
  bool b_k = false;
  const uint16_t* b[2] = {};
  int64_t ldb = 0;
  bool two_segments = false;   // acc = A0 B0 + A1 B1, both of depth K
  int mats = 1;                // 2 (with a_mn only): o[0] = A B0 and o[1] = A B1
  int act = 0;
  const uint16_t* bias = nullptr;
  const uint16_t* residual = nullptr;
  int64_t ldr = 0;
  const uint16_t *g = nullptr, *u = nullptr;   // DENSE_GRAD, rows x cols, contiguous
  uint16_t* o[3] = {};
  int64_t ldo = 0;
  // another product of the same depth with nothing in its epilogue, in the same
  // launch (both with a_mn, neither with b_k)
  const DenseGemm* also = nullptr;
};

// How a product is run: by the pair kernel, by the tall kernel with tiles of tn
// tokens, or by the few-token kernel with tiles of tn tokens, `parts` CTAs along K
// and per_sm CTAs resident on an SM.
enum DenseKind { DENSE_PAIR = 0, DENSE_TALL = 1, DENSE_FEW = 2 };

struct DensePlan {
  DenseKind kind;
  int tn, parts, per_sm;
};

// Its tiles: tm down and tn across one weight (pair kernel: tm2 and tn2 of the second
// product of the launch too), of which the first `whole` are taken whole and the
// others in two halves (pair kernel only); `items` steps of the walk in all.
struct DenseTiles {
  int tm, tn, tm2, tn2, whole, items;
};

DensePlan plan_dense(const DenseGemm& d);
DenseTiles tile_dense(const DenseGemm& d, const DensePlan& p);

cudaError_t launch_dense(const DenseGemm& d, cudaStream_t stream);
cudaError_t read_dense_error(unsigned* out, cudaStream_t stream);
cudaError_t set_dense_wait_limit(long long cycles);

}  // namespace sig

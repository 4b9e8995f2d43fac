// Dense attention around the compressed cache: whole packed prompts (causal) and trees of drafted
// tokens over a dense cache, and the rotary embedding both need. Argument blocks and host
// launchers; the C-ABI checks are in dense_api.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "iskv.h"

namespace iskv {

// Strides in elements; the head_dim elements of one (row, head) are contiguous.
struct DenseArgs {
  iskv_heads q, k, v;    // prompt: the packed rows; tree: the drafted nodes
  iskv_heads kc, vc;     // tree: the cache
  iskv_heads out;
  const int32_t *cu;        // prompt: [n_seqs + 1] first row of each sequence, or NULL
  const int32_t *n_cached;  // tree: [batch] cached rows in use, or NULL (all n_cap)
  const int32_t *parents;   // tree: [batch][nodes]
  int32_t tree;
  int32_t whole;            // tree: a CTA per unit, nothing to join
  int32_t batch;            // prompt: sequences; tree: batch entries
  int32_t nodes;            // tree: drafted nodes per entry
  int64_t rows;             // prompt: packed rows; tree: cache capacity n_cap
  int32_t n_q, n_kv, group, head_dim;
  float scale;
  int32_t dtype;
  int64_t *status;
  void *ws;                 // tree: partial results
};

constexpr int DENSE_MAX_NODES = 128;
// CTAs of a tree call: one per SM of a B200 (148) for the tensor-core kernel, two for the CUDA-core
// kernel. Fixed, so that the workspace size needs no device.
constexpr int DENSE_TC_GRID = 148;
constexpr int DENSE_CC_GRID = 296;

// Partial results of a tree call: a CTA's share of the key tiles is one contiguous range, so only
// its first and its last unit can be shared with other CTAs: two slots per CTA. A slot holds
// float4 O[hd_pad / 4][rows] (column-major, so that one row per lane writes whole lines), then
// m[rows] (log2 units) and l[rows].
__host__ __device__ inline size_t dense_slot_floats(int rows, int hd_pad) {
  return (size_t)rows * (hd_pad + 2);
}

// Head dimensions are padded with zeros to the kernel's compiled width.
inline int dense_hd_pad(int hd) { return hd <= 64 ? 64 : hd <= 128 ? 128 : 256; }

// CUDA-core kernel: float32 and whatever the tensor-core kernel does not take.
constexpr int DENSE_CC_ROWS = 64;
cudaError_t launch_dense_cc(const DenseArgs &a, cudaStream_t s);
// Tensor-core kernel: two-byte elements, head_dim a multiple of 8 up to 128, 16-byte aligned rows.
bool dense_tc_takes(const DenseArgs &a);
// false: a tensor map could not be encoded and nothing was launched.
bool launch_dense_tc(const DenseArgs &a, cudaStream_t s, cudaError_t &e);
// Joins the partial results of a tree call whose kernel ran `grid` CTAs over units of `rows` rows
// and tiles of `keys` keys.
cudaError_t launch_dense_join(const DenseArgs &a, int grid, int rows, int keys, cudaStream_t s);

// A kernel's dynamic shared-memory limit, raised once per device (the first 64 of a process).
struct SmemLimit {
  std::atomic<uint64_t> done{0};
  cudaError_t raise(const void *kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
  }
};

struct RopeArgs {
  const void *x;
  void *out;
  int64_t x_row, x_head, o_row, o_head;
  const int32_t *pos;
  int64_t n;
  int32_t heads, head_dim, inverse, dtype;
  double theta;
};
cudaError_t launch_rope(const RopeArgs &a, cudaStream_t s);

}  // namespace iskv

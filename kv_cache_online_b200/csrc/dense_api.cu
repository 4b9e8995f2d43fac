// C ABI of the rotary embedding and the dense attention (see include/iskv.h): argument checks, the
// choice between the tensor-core and the CUDA-core kernel, launches.
#include <cmath>

#include "api_error.h"
#include "dense.h"
#include "profiling.h"

using namespace iskv;

namespace {

// What calls without a status word of their own record, one word per device.
__device__ unsigned long long g_status;

__global__ void k_clear_status(unsigned long long bits) { atomicAnd(&g_status, ~bits); }

// `status`, or the current device's own word.
cudaError_t status_word(int64_t *status, int64_t **word) {
  void *p = status;
  const cudaError_t e = status ? cudaSuccess : cudaGetSymbolAddress(&p, g_status);
  *word = static_cast<int64_t *>(p);
  return e;
}

size_t elem_bytes(int32_t t) { return t == ISKV_F32 ? 4 : 2; }

iskv_status check_dtype(int32_t t, const char *who) {
  if (t != ISKV_F32 && t != ISKV_BF16 && t != ISKV_F16)
    return fail(ISKV_ERR_ARG, "%s: bad dtype", who);
  return ISKV_OK;
}

// `empty`: the block holds no element, its pointer is not used.
iskv_status check_heads(const iskv_heads *x, const char *name, int32_t dtype, bool empty,
                        bool entries, const char *who) {
  if (!x) return fail(ISKV_ERR_ARG, "%s: null %s", who, name);
  if (empty) return ISKV_OK;
  if (!x->data) return fail(ISKV_ERR_ARG, "%s: null %s data", who, name);
  if (reinterpret_cast<uintptr_t>(x->data) % elem_bytes(dtype))
    return fail(ISKV_ERR_ARG, "%s: misaligned %s", who, name);
  const int64_t lim = (int64_t)1 << 36;  // byte strides below 2^40, as a tensor map takes them
  if (x->row < 0 || x->head < 0 || x->row >= lim || x->head >= lim ||
      (entries && (x->batch < 0 || x->batch >= lim)))
    return fail(ISKV_ERR_SHAPE, "%s: bad strides of %s", who, name);
  return ISKV_OK;
}

// The stride of an axis of length one is never used; callers may leave anything there.
iskv_heads walked(const iskv_heads *x, int64_t entries, int64_t rows, int64_t heads) {
  iskv_heads y = *x;
  if (entries <= 1) y.batch = 0;
  if (rows <= 1) y.row = 0;
  if (heads <= 1) y.head = 0;
  return y;
}

iskv_status check_shape(int32_t n_q, int32_t n_kv, int32_t head_dim, float scale, const char *who) {
  if (n_kv < 1 || n_kv > 1024 || n_q < 1 || n_q % n_kv || n_q / n_kv > 64)
    return fail(ISKV_ERR_SHAPE, "%s: need n_q_heads a multiple of n_kv_heads (1..1024), at most 64 "
                "per key/value head (got %d, %d)", who, n_q, n_kv);
  if (head_dim < 1 || head_dim > 256)
    return fail(ISKV_ERR_SHAPE, "%s: need 1 <= head_dim <= 256 (got %d)", who, head_dim);
  // (scale log2(e) has to be finite too)
  if (!(std::fabs(scale) <= 0x1p127f))
    return fail(ISKV_ERR_ARG, "%s: scale must be finite, 2^127 at most in magnitude", who);
  return ISKV_OK;
}

iskv_status check_status_word(const int64_t *status, const char *who) {
  if (reinterpret_cast<uintptr_t>(status) % 8)
    return fail(ISKV_ERR_ARG, "%s: misaligned status", who);
  return ISKV_OK;
}

cudaError_t launch_dense(DenseArgs &a, cudaStream_t s) {
  cudaError_t e = status_word(a.status, &a.status);
  if (e != cudaSuccess) return e;
  if (dense_tc_takes(a) && launch_dense_tc(a, s, e)) return e;
  return launch_dense_cc(a, s);
}

}  // namespace

extern "C" {

iskv_status iskv_rope(const iskv_heads *x, const int32_t *pos, int64_t n, int32_t n_heads,
                      int32_t head_dim, double rope_theta, int32_t inverse, int32_t dtype,
                      const iskv_heads *out, void *stream) {
  const char *who = "iskv_rope";
  clear_last_error();
  iskv_status st = check_dtype(dtype, who);
  if (st != ISKV_OK) return st;
  if (n < 0 || n >= (int64_t)1 << 31) return fail(ISKV_ERR_SHAPE, "%s: n out of range", who);
  if (n_heads < 1 || n_heads > 1024 || head_dim < 2 || head_dim > 256 || head_dim % 2)
    return fail(ISKV_ERR_SHAPE, "%s: need 1 <= n_heads <= 1024, even head_dim <= 256", who);
  if (!(rope_theta > 0.0) || !std::isfinite(rope_theta))
    return fail(ISKV_ERR_ARG, "%s: rope_theta must be finite and > 0", who);
  st = check_heads(x, "x", dtype, n == 0, false, who);
  if (st == ISKV_OK) st = check_heads(out, "out", dtype, n == 0, false, who);
  if (st != ISKV_OK) return st;
  if (n == 0) return ISKV_OK;
  if (!pos || reinterpret_cast<uintptr_t>(pos) % 4)
    return fail(ISKV_ERR_ARG, "%s: null or misaligned pos", who);
  if (x->data == out->data && ((n > 1 && x->row != out->row) ||
                               (n_heads > 1 && x->head != out->head)))
    return fail(ISKV_ERR_ARG, "%s: in place needs equal strides", who);
  if ((n > 1 && out->row == 0) || (n_heads > 1 && out->head == 0))
    return fail(ISKV_ERR_SHAPE, "%s: out has a stride of 0", who);
  const iskv_heads xs = walked(x, 1, n, n_heads), os = walked(out, 1, n, n_heads);
  RopeArgs a;
  a.x = xs.data;
  a.out = os.data;
  a.x_row = xs.row;
  a.x_head = xs.head;
  a.o_row = os.row;
  a.o_head = os.head;
  a.pos = pos;
  a.n = n;
  a.heads = n_heads;
  a.head_dim = head_dim;
  a.inverse = inverse != 0;
  a.dtype = dtype;
  a.theta = rope_theta;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  stage_begin(s);
  cudaError_t e = launch_rope(a, s);
  if (e != cudaSuccess) return cuda_fail(e, who);
  stage_mark(s, ST_ROPE);
  return ISKV_OK;
}

iskv_status iskv_prompt_attention(const iskv_heads *q, const iskv_heads *k, const iskv_heads *v,
                                  const int32_t *cu_seqlens, int32_t n_seqs, int64_t n_rows,
                                  int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                  float scale, int32_t dtype, const iskv_heads *out,
                                  int64_t *status, void *stream) {
  const char *who = "iskv_prompt_attention";
  clear_last_error();
  iskv_status st = check_dtype(dtype, who);
  if (st == ISKV_OK) st = check_shape(n_q_heads, n_kv_heads, head_dim, scale, who);
  if (st != ISKV_OK) return st;
  if (n_rows < 0 || n_rows > (int64_t)1 << 24 || n_seqs < 0 || n_seqs > 4096)
    return fail(ISKV_ERR_SHAPE, "%s: need 0 <= n_rows <= 2^24, 0 <= n_seqs <= 4096", who);
  const bool empty = n_rows == 0 || n_seqs == 0;
  st = check_heads(q, "q", dtype, empty, false, who);
  if (st == ISKV_OK) st = check_heads(k, "k", dtype, empty, false, who);
  if (st == ISKV_OK) st = check_heads(v, "v", dtype, empty, false, who);
  if (st == ISKV_OK) st = check_heads(out, "out", dtype, empty, false, who);
  if (st == ISKV_OK) st = check_status_word(status, who);
  if (st != ISKV_OK) return st;
  if (empty) return ISKV_OK;
  if (reinterpret_cast<uintptr_t>(cu_seqlens) % 4)
    return fail(ISKV_ERR_ARG, "%s: misaligned cu_seqlens", who);
  // One block per 64 packed rows and key/value head at most.
  if ((n_rows * (n_q_heads / n_kv_heads) / 64 + n_seqs) * n_kv_heads >= (int64_t)1 << 31)
    return fail(ISKV_ERR_SHAPE, "%s: (n_rows * group / 64 + n_seqs) * n_kv_heads must stay below "
                "2^31", who);
  if (!cu_seqlens && n_seqs != 1)
    return fail(ISKV_ERR_ARG, "%s: cu_seqlens may be null for one sequence only", who);
  if ((n_rows > 1 && out->row == 0) || (n_q_heads > 1 && out->head == 0))
    return fail(ISKV_ERR_SHAPE, "%s: out has a stride of 0", who);
  DenseArgs a = {};
  a.q = walked(q, 1, n_rows, n_q_heads);
  a.k = walked(k, 1, n_rows, n_kv_heads);
  a.v = walked(v, 1, n_rows, n_kv_heads);
  a.out = walked(out, 1, n_rows, n_q_heads);
  a.cu = cu_seqlens;
  a.batch = n_seqs;
  a.rows = n_rows;
  a.n_q = n_q_heads;
  a.n_kv = n_kv_heads;
  a.group = n_q_heads / n_kv_heads;
  a.head_dim = head_dim;
  a.scale = scale;
  a.dtype = dtype;
  a.status = status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  stage_begin(s);
  cudaError_t e = launch_dense(a, s);
  if (e != cudaSuccess) return cuda_fail(e, who);
  stage_mark(s, ST_PROMPT_ATTN);
  return ISKV_OK;
}

size_t iskv_tree_attention_workspace_size(int32_t n_nodes, int32_t n_q_heads, int32_t n_kv_heads,
                                          int32_t head_dim) {
  if (n_nodes < 1 || n_nodes > DENSE_MAX_NODES || n_kv_heads < 1 || n_q_heads < 1 ||
      n_q_heads % n_kv_heads || n_q_heads / n_kv_heads > 64 || head_dim < 1 || head_dim > 256)
    return 0;
  const size_t cc = 2 * DENSE_CC_GRID * dense_slot_floats(DENSE_CC_ROWS, dense_hd_pad(head_dim));
  const int tc_rows = n_nodes * (n_q_heads / n_kv_heads) <= 128 ? 128 : 256;
  const size_t tc =
      head_dim <= 128 ? 2 * DENSE_TC_GRID * dense_slot_floats(tc_rows, dense_hd_pad(head_dim)) : 0;
  return (cc > tc ? cc : tc) * sizeof(float);
}

iskv_status iskv_tree_attention(const iskv_heads *q, const iskv_heads *k_draft,
                                const iskv_heads *v_draft, const int32_t *parents,
                                const iskv_heads *k_cache, const iskv_heads *v_cache,
                                const int32_t *n_cached, int32_t batch, int32_t n_nodes,
                                int64_t n_cap, int32_t n_q_heads, int32_t n_kv_heads,
                                int32_t head_dim, float scale, int32_t dtype,
                                const iskv_heads *out, int64_t *status, void *ws, size_t ws_bytes,
                                void *stream) {
  const char *who = "iskv_tree_attention";
  clear_last_error();
  iskv_status st = check_dtype(dtype, who);
  if (st == ISKV_OK) st = check_shape(n_q_heads, n_kv_heads, head_dim, scale, who);
  if (st != ISKV_OK) return st;
  if (batch < 0 || batch > 4096 || n_nodes < 0 || n_nodes > DENSE_MAX_NODES || n_cap < 0 ||
      n_cap >= (int64_t)1 << 31)
    return fail(ISKV_ERR_SHAPE, "%s: need 0 <= batch <= 4096, 0 <= n_nodes <= %d, 0 <= n_cap < "
                "2^31", who, DENSE_MAX_NODES);
  const bool empty = batch == 0 || n_nodes == 0, bare = empty || n_cap == 0;
  st = check_heads(q, "q", dtype, empty, true, who);
  if (st == ISKV_OK) st = check_heads(k_draft, "k_draft", dtype, empty, true, who);
  if (st == ISKV_OK) st = check_heads(v_draft, "v_draft", dtype, empty, true, who);
  if (st == ISKV_OK) st = check_heads(k_cache, "k_cache", dtype, bare, true, who);
  if (st == ISKV_OK) st = check_heads(v_cache, "v_cache", dtype, bare, true, who);
  if (st == ISKV_OK) st = check_heads(out, "out", dtype, empty, true, who);
  if (st == ISKV_OK) st = check_status_word(status, who);
  if (st != ISKV_OK) return st;
  if (empty) return ISKV_OK;
  // The line of key tiles is counted in 32 bits; no kernel's tiles or row blocks are smaller than
  // 64.
  const int64_t blocks = (n_nodes * (n_q_heads / n_kv_heads) + 63) / 64;
  if ((int64_t)batch * n_kv_heads * blocks >= ((int64_t)1 << 31) / (n_cap / 64 + 3))
    return fail(ISKV_ERR_SHAPE, "%s: batch * n_kv_heads * row blocks * key tiles must stay below "
                "2^31", who);
  if (!parents || reinterpret_cast<uintptr_t>(parents) % 4 ||
      reinterpret_cast<uintptr_t>(n_cached) % 4)
    return fail(ISKV_ERR_ARG, "%s: null or misaligned parents / n_cached", who);
  if ((n_nodes > 1 && out->row == 0) || (n_q_heads > 1 && out->head == 0) ||
      (batch > 1 && out->batch == 0))
    return fail(ISKV_ERR_SHAPE, "%s: out has a stride of 0", who);
  const size_t need =
      iskv_tree_attention_workspace_size(n_nodes, n_q_heads, n_kv_heads, head_dim);
  if (!ws) return fail(ISKV_ERR_WORKSPACE, "%s: null workspace", who);
  if (reinterpret_cast<uintptr_t>(ws) % 256)
    return fail(ISKV_ERR_WORKSPACE, "%s: workspace must be 256-byte aligned", who);
  if (ws_bytes < need)
    return fail(ISKV_ERR_WORKSPACE, "%s: workspace too small (%zu < %zu bytes)", who, ws_bytes,
                need);
  DenseArgs a = {};
  a.q = walked(q, batch, n_nodes, n_q_heads);
  a.k = walked(k_draft, batch, n_nodes, n_kv_heads);
  a.v = walked(v_draft, batch, n_nodes, n_kv_heads);
  a.kc = walked(k_cache, batch, n_cap, n_kv_heads);
  a.vc = walked(v_cache, batch, n_cap, n_kv_heads);
  a.out = walked(out, batch, n_nodes, n_q_heads);
  a.n_cached = n_cached;
  a.parents = parents;
  a.tree = 1;
  a.batch = batch;
  a.nodes = n_nodes;
  a.rows = n_cap;
  a.n_q = n_q_heads;
  a.n_kv = n_kv_heads;
  a.group = n_q_heads / n_kv_heads;
  a.head_dim = head_dim;
  a.scale = scale;
  a.dtype = dtype;
  a.status = status;
  a.ws = ws;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  stage_begin(s);
  cudaError_t e = launch_dense(a, s);
  if (e != cudaSuccess) return cuda_fail(e, who);
  stage_mark(s, ST_TREE_ATTN);
  return ISKV_OK;
}

iskv_status iskv_dense_status(int64_t *bits, int32_t reset) {
  const char *who = "iskv_dense_status";
  clear_last_error();
  if (!bits) return fail(ISKV_ERR_ARG, "%s: null output", who);
  // (The word's kernels may run on streams that the legacy default stream does not wait for.)
  cudaError_t e = cudaDeviceSynchronize();
  unsigned long long word = 0;
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&word, g_status, sizeof word);
  if (e == cudaSuccess && reset && word) {
    k_clear_status<<<1, 1>>>(word);
    count_launches(1);
    e = cudaGetLastError();
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
  }
  if (e != cudaSuccess) return cuda_fail(e, who);
  *bits = (int64_t)word;
  return ISKV_OK;
}

}  // extern "C"

// Dense attention on the CUDA cores: float32, and two-byte elements whose shape or alignment the
// tensor-core kernel does not take. Also the join of a tree call's partial results.
//
// One pass over the keys with a running maximum m and sum l per row (x = scale log2(e) q.k):
//   m' = max(m, max_j x_j);  p_j = 2^(x_j - m');  l' = l 2^(m - m') + sum p_j;
//   O' = O 2^(m - m') + sum_j p_j v_j;  out = O / l.
//
// FP32-FMA bound: 4 hd flops per visible pair on 128 lanes per SM. A block of 256 threads owns 64
// rows and walks tiles of 64 keys; thread (ty, tx) holds scores of rows 4 ty + i and keys tx + 16
// j, and output columns 4 tx + 64 c, so that a score step reads 8 float4 for 64 FMAs and a value
// step 4 + HD/16 float4 for HD FMAs, without bank conflicts (row strides of HD + 4 floats). All
// operands are float32 in shared memory, products and statistics float32. float32 rows whose
// 16-byte pieces are aligned (HD up to 128) arrive by asynchronous copies, the next tile's under
// this tile's arithmetic; other rows go through registers (a tile's loads are then waited for).
#include "dense.cuh"
#include "profiling.h"

namespace iskv {
namespace {

using namespace dense;

constexpr int ROWS = DENSE_CC_ROWS, KT = 64, NT = 256;

template <int HD, int BUF>
struct Smem {
  static constexpr int LD = HD + 4;
  float q[ROWS][LD], k[BUF][KT][LD], v[BUF][KT][LD];
  float p[ROWS][KT + 4];
  uint32_t mask[DENSE_MAX_NODES][4];
  Unit unit;
};

ISKV_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Element offset of (entry, row, head).
ISKV_DEV int64_t at(const iskv_heads &x, int64_t b, int64_t row, int64_t head) {
  return b * x.batch + row * x.row + head * x.head;
}

// `n` rows of one head as float32 rows of shared memory; rows from n on and columns from hd on are
// zero. VEC: 16-byte loads (hd and strides are multiples of a vector, the base is aligned).
template <typename T, int HD, bool VEC>
ISKV_DEV void load_rows(float (*dst)[HD + 4], const T *src, int64_t stride, int n, int hd) {
  if constexpr (VEC) {
    constexpr int V = 16 / sizeof(T), C = HD / V;
#pragma unroll 4
    for (int i = threadIdx.x; i < KT * C; i += NT) {
      const int r = i / C, c = i % C * V;
      alignas(16) T x[V];
      if (r < n && c < hd)
        *reinterpret_cast<uint4 *>(x) = *reinterpret_cast<const uint4 *>(src + r * stride + c);
      else
        *reinterpret_cast<uint4 *>(x) = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int e = 0; e < V; e += 4)
        *reinterpret_cast<float4 *>(&dst[r][c + e]) =
            make_float4(to_f(x[e]), to_f(x[e + 1]), to_f(x[e + 2]), to_f(x[e + 3]));
    }
  } else {
    for (int i = threadIdx.x; i < KT * HD; i += NT) {
      const int r = i / HD, c = i % HD;
      dst[r][c] = r < n && c < hd ? to_f(src[r * stride + c]) : 0.f;
    }
  }
}

// The same rows by asynchronous 16-byte copies (zero where there is nothing to read).
template <int HD>
ISKV_DEV void copy_rows(float (*dst)[HD + 4], const float *src, int64_t stride, int n, int hd) {
  constexpr int C = HD / 4;
#pragma unroll 4
  for (int i = threadIdx.x; i < KT * C; i += NT) {
    const int r = i / C, c = i % C * 4;
    const bool in = r < n && c < hd;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(&dst[r][c])),
                 "l"(in ? src + r * stride + c : src), "r"(in ? 16 : 0)
                 : "memory");
  }
}

template <typename T, int HD, bool VEC>
constexpr int BUFFERS = std::is_same<T, float>::value && VEC && HD <= 128 ? 2 : 1;

template <typename T, int HD, bool TREE, bool VEC>
ISKV_DEV void run_unit(const DenseArgs &a, Smem<HD, BUFFERS<T, HD, VEC>> &sm, const Unit &u) {
  constexpr int NC = HD / 64;
  constexpr bool ASYNC = BUFFERS<T, HD, VEC> == 2;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int hd = a.head_dim;
  // Non-negative factor on the scores; the scale's sign goes into the queries.
  const float c = score_factor(a);
  const int64_t row_base = TREE ? 0 : u.base;

  for (int i = threadIdx.x; i < ROWS * HD; i += NT) {
    const int r = i / HD, col = i % HD;
    float x = 0.f;
    if (r < u.n_rows && col < hd) {
      const int pr = u.row0 + r;
      x = to_f(static_cast<const T *>(a.q.data)[at(a.q, TREE ? u.b : 0, row_base + pr / a.group,
                                                   (int64_t)u.kvh * a.group + pr % a.group) + col]);
    }
    sm.q[r][col] = a.scale < 0.f ? -x : x;
  }
  if constexpr (TREE) {
    if (threadIdx.x < DENSE_MAX_NODES) {
      uint32_t m[4];
      node_mask(a, a.parents + (int64_t)u.b * a.nodes, min((int)threadIdx.x, a.nodes - 1), m);
#pragma unroll
      for (int w = 0; w < 4; ++w) sm.mask[threadIdx.x][w] = m[w];
    }
  }
  int tok[4];  // prompt: the row's token; tree: its node
  float raw[4], m[4], l[4];  // m = c max s (raw), l: sum of the weights
  alignas(8) float o[4][NC][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    tok[i] = (u.row0 + min(ty * 4 + i, u.n_rows - 1)) / a.group;
    raw[i] = m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][n][e] = 0.f;
  }

  // Keys and values of tile t into buffer `to`.
  auto fetch = [&](int t, int to) {
    const bool draft = TREE && t >= u.cache_tiles;
    const int k0 = (draft ? t - u.cache_tiles : t) * KT;
    const int n = min(KT, (draft ? a.nodes : u.len) - k0);
    const iskv_heads &K = TREE && !draft ? a.kc : a.k, &V = TREE && !draft ? a.vc : a.v;
    const T *k = static_cast<const T *>(K.data) + at(K, TREE ? u.b : 0, row_base + k0, u.kvh);
    const T *v = static_cast<const T *>(V.data) + at(V, TREE ? u.b : 0, row_base + k0, u.kvh);
    if constexpr (ASYNC) {
      copy_rows<HD>(sm.k[to], k, K.row, n, hd);
      copy_rows<HD>(sm.v[to], v, V.row, n, hd);
      asm volatile("cp.async.commit_group;" ::: "memory");
    } else {
      load_rows<T, HD, VEC>(sm.k[to], k, K.row, n, hd);
      load_rows<T, HD, VEC>(sm.v[to], v, V.row, n, hd);
    }
  };
  int buf = 0;
  if constexpr (ASYNC) fetch(u.t0, 0);
  for (int t = u.t0; t < u.t1; ++t) {
    const bool draft = TREE && t >= u.cache_tiles;
    const int k0 = (draft ? t - u.cache_tiles : t) * KT;  // first key of the tile
    const int n_keys = min(KT, (draft ? a.nodes : u.len) - k0);
    if constexpr (ASYNC) {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();  // this tile is there, and nobody reads the other buffer any more
      buf = (t - u.t0) & 1;
      if (t + 1 < u.t1) fetch(t + 1, buf ^ 1);
    } else {
      __syncthreads();  // the previous tile's keys, values and probabilities are no longer read
      fetch(t, 0);
      __syncthreads();
    }

    // Even and odd columns in the two halves of packed FMAs (half the instructions).
    float2 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int d = 0; d < HD; d += 4) {
      float4 qv[4], kv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) qv[i] = *reinterpret_cast<const float4 *>(&sm.q[ty * 4 + i][d]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        kv[j] = *reinterpret_cast<const float4 *>(&sm.k[buf][tx + 16 * j][d]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[i][j] = __ffma2_rn(make_float2(qv[i].x, qv[i].y), make_float2(kv[j].x, kv[j].y),
                                 acc[i][j]);
          acc[i][j] = __ffma2_rn(make_float2(qv[i].z, qv[i].w), make_float2(kv[j].z, kv[j].w),
                                 acc[i][j]);
        }
    }
    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = acc[i][j].x + acc[i][j].y;
    // Pairs the mask leaves out have p = -1 in shared memory: the value step skips them, so that
    // a value that is not finite cannot reach a row that does not see it.
    const bool masked = n_keys < KT || draft || (!TREE && k0 + KT > first_token(a, u) + 1);
    uint32_t seen = 0xffffu;
    if (masked) {
      seen = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = k0 + tx + 16 * j;
          bool see = tx + 16 * j < n_keys;
          if (draft) see = see && (sm.mask[tok[i]][(key >> 5) & 3] >> (key & 31) & 1);
          if (!TREE) see = see && key <= tok[i];
          if (see) seen |= 1u << (i * 4 + j);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float top = raw[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = seen >> (i * 4 + j) & 1 ? s[i][j] : -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
      // One rounding of s c - m (of s c alone it would be that of the larger number); m's own
      // rounding is common to the row's weights.
      raw[i] = top;
      const float mn = top == -INFINITY ? -INFINITY : top * c;
      const float ref = top == -INFINITY ? 0.f : mn;
      const float alpha = ex2(m[i] - ref);  // 0 while nothing was seen
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = ex2(fmaf(s[i][j], c, -ref));
        const bool see = seen >> (i * 4 + j) & 1;
        if (see) sum += p;
        sm.p[ty * 4 + i][tx + 16 * j] = see ? p : -1.f;
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      l[i] = l[i] * alpha + sum;
      m[i] = mn;
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][n][e] *= alpha;
    }
    __syncwarp();  // a row's probabilities are written and read by the same half-warp
    auto values = [&](auto guarded) {
#pragma unroll 2
      for (int k = 0; k < KT; k += 4) {
        float4 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4 *>(&sm.p[ty * 4 + i][k]);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            const float4 v = *reinterpret_cast<const float4 *>(&sm.v[buf][k + kk][tx * 4 + 64 * n]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float w = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
              if (decltype(guarded)::value && w < 0.f) continue;
              float2 *po = reinterpret_cast<float2 *>(o[i][n]);
              po[0] = __ffma2_rn(make_float2(w, w), make_float2(v.x, v.y), po[0]);
              po[1] = __ffma2_rn(make_float2(w, w), make_float2(v.z, v.w), po[1]);
            }
          }
        }
      }
    };
    if (masked) values(std::true_type{});
    else values(std::false_type{});
  }

  const bool whole = !TREE || (u.t0 == 0 && u.t1 == u.n_tiles);
  if (whole) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i;
      if (r >= u.n_rows) continue;
      bool live = true;  // padding nodes give zeros
      if constexpr (TREE)
        live = (sm.mask[tok[i]][0] | sm.mask[tok[i]][1] | sm.mask[tok[i]][2] | sm.mask[tok[i]][3]);
      const int pr = u.row0 + r;
      T *out = static_cast<T *>(a.out.data) + at(a.out, TREE ? u.b : 0, row_base + pr / a.group,
                                                 (int64_t)u.kvh * a.group + pr % a.group);
      const float inv = 1.f / l[i];
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = tx * 4 + 64 * n + e;
          if (col < hd) out[col] = from_f<T>(live && l[i] != 0.f ? o[i][n][e] * inv : 0.f);
        }
    }
  } else {
    const int slot = 2 * blockIdx.x + (u.t0 > 0 ? 0 : 1);
    float *ws = static_cast<float *>(a.ws) + slot * dense_slot_floats(ROWS, HD);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i;
      if (r >= u.n_rows) continue;
      const bool live =
          sm.mask[tok[i]][0] | sm.mask[tok[i]][1] | sm.mask[tok[i]][2] | sm.mask[tok[i]][3];
#pragma unroll
      for (int n = 0; n < NC; ++n)
        reinterpret_cast<float4 *>(ws)[(tx + 16 * n) * ROWS + r] =
            make_float4(o[i][n][0], o[i][n][1], o[i][n][2], o[i][n][3]);
      if (tx == 0) {
        ws[ROWS * HD + r] = live ? m[i] : -INFINITY;
        ws[ROWS * (HD + 1) + r] = live ? l[i] : 0.f;
      }
    }
  }
}

// Two blocks share an SM where their shared memory fits (HD = 64; 128 registers), else one block
// has all registers: four prompts of 600 tokens at head_dim 64, 95 against 107 us; 2,500 tokens at
// head_dim 128, 1,634 against 1,520 us.
template <typename T, int HD, bool TREE, bool VEC>
__global__ void __launch_bounds__(NT, HD == 64 ? 2 : 1)
    k_dense_cc(const __grid_constant__ DenseArgs a) {
  if constexpr (TREE) asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ __align__(16) char raw[];
  auto &sm = *reinterpret_cast<Smem<HD, BUFFERS<T, HD, VEC>> *>(raw);
  if constexpr (!TREE) {
    if (threadIdx.x < 32) {
      Unit u;
      if (find_prompt_unit<ROWS>(a, blockIdx.x / a.n_kv, u)) {
        u.kvh = blockIdx.x % a.n_kv;
        u.t0 = 0;
        u.t1 = u.n_tiles = last_token(a, u) / KT + 1;
      } else {
        u.b = -1;
      }
      if (threadIdx.x == 0) sm.unit = u;
    }
    __syncthreads();
    const Unit u = sm.unit;
    if (u.b >= 0) run_unit<T, HD, false, VEC>(a, sm, u);
  } else {
    TreeLine<ROWS, KT> line;
    if (threadIdx.x < 32) line.begin(a, gridDim.x, blockIdx.x);
    for (;;) {
      __syncthreads();  // the previous unit's place is no longer read
      if (threadIdx.x < 32) {
        Unit u;
        if (!line.next(a, u)) u.b = -1;
        if (threadIdx.x == 0) sm.unit = u;
      }
      __syncthreads();
      const Unit u = sm.unit;
      if (u.b < 0) break;
      run_unit<T, HD, true, VEC>(a, sm, u);
    }
  }
}

// A block: 32 rows (lanes) of one unit. SPLIT: its four warps take every fourth part of the unit
// for the same four columns, with a running maximum each, and add up in shared memory with weights
// 2^(m_i - max m) (few units of many parts each); otherwise every warp takes all parts for 32
// columns of its own (many units, a few parts each). Latency bound, a few KB per warp: all loads of
// four parts are in flight together.
template <typename T, int ROWS, int KT, bool SPLIT>
__global__ void __launch_bounds__(128) k_dense_join(const __grid_constant__ DenseArgs a, int grid,
                                                    int hd_pad) {
  constexpr int COLS = SPLIT ? 1 : 8;  // groups of four columns per warp
  __shared__ float part[4][2 + 4 * COLS][33], factor[5][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  TreeLine<ROWS, KT> line;
  line.begin(a, grid, 0);
  const int rows_all = a.nodes * a.group, unit = blockIdx.x;
  const int kvh = unit / line.blocks % a.n_kv, blk = unit % line.blocks;
  const int b = unit / line.blocks / a.n_kv;
  int before = 0;
  for (int e = lane; e < b; e += 32) before += line.entry_tiles(a, e);
  before = __reduce_add_sync(0xffffffffu, before);
  const int n = (cached_rows(a, b) + KT - 1) / KT + line.draft_tiles;
  const int u0 = before + (kvh * line.blocks + blk) * n;
  const int c0 = u0 / line.per, c1 = (u0 + n - 1) / line.per;
  const int n_rows = min(ROWS, rows_all - blk * ROWS);
  const int all_cols = (a.head_dim + 3) / 4;
  constexpr int BLOCK_COLS = SPLIT ? 1 : 4 * COLS;
  const int groups = (all_cols + BLOCK_COLS - 1) / BLOCK_COLS, chunk = blockIdx.y / groups;
  const int r = chunk * 32 + lane;
  const int rr = min(r, n_rows - 1);
  const int g0 = (blockIdx.y - chunk * groups) * BLOCK_COLS + (SPLIT ? 0 : warp * COLS);
  const size_t slot_floats = dense_slot_floats(ROWS, hd_pad);
  const int pr = blk * ROWS + rr, node = pr / a.group;
  T *const out = static_cast<T *>(a.out.data) +
                 at(a.out, b, node, (int64_t)kvh * a.group + (pr - node * a.group)) + g0 * 4;
  // Up to here only the call's inputs were read; the parts need the kernel before this one. Every
  // block waits, those without rows to join too: later work on the stream is ordered behind this
  // kernel alone, and this one behind the kernel before it only by the wait.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (c0 == c1) return;  // one CTA had all of the unit and wrote its rows itself
  if (chunk * 32 >= n_rows) return;
  constexpr int STEP = SPLIT ? 4 : 1;
  float m = -INFINITY, l = 0.f;
  float4 o[COLS];
#pragma unroll
  for (int g = 0; g < COLS; ++g) o[g] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = c0 + (SPLIT ? warp : 0); c <= c1; c += 4 * STEP) {
    float w[4], li[4];
    float4 v[4][COLS];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // The part with the unit's first tile is in its CTA's slot 1, the others open their CTA's
      // share: slot 0.
      const int ci = min(c + STEP * i, c1);
      const float *s =
          static_cast<const float *>(a.ws) + (ci == c0 ? 2 * ci + 1 : 2 * ci) * slot_floats;
      w[i] = s[(size_t)ROWS * hd_pad + rr];
      li[i] = s[(size_t)ROWS * (hd_pad + 1) + rr];
#pragma unroll
      for (int g = 0; g < COLS; ++g)
        v[i][g] = reinterpret_cast<const float4 *>(s)[min(g0 + g, all_cols - 1) * ROWS + rr];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + STEP * i > c1) {
        w[i] = -INFINITY;
        li[i] = 0.f;
      }
    float mn = m;
#pragma unroll
    for (int i = 0; i < 4; ++i) mn = fmaxf(mn, w[i]);
    const float ref = mn == -INFINITY ? 0.f : mn, f = ex2(m - ref);
    m = mn;
    l *= f;
#pragma unroll
    for (int g = 0; g < COLS; ++g)
      o[g] = make_float4(o[g].x * f, o[g].y * f, o[g].z * f, o[g].w * f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // A part that saw nothing has m = -inf and l = 0 (its O may be anything); with m = -inf and
      // another l, not-a-number scores alone were seen.
      if (w[i] == -INFINITY && li[i] == 0.f) continue;
      const float e = ex2(w[i] - ref);
      l = fmaf(li[i], e, l);
#pragma unroll
      for (int g = 0; g < COLS; ++g) {
        o[g].x = fmaf(v[i][g].x, e, o[g].x);
        o[g].y = fmaf(v[i][g].y, e, o[g].y);
        o[g].z = fmaf(v[i][g].z, e, o[g].z);
        o[g].w = fmaf(v[i][g].w, e, o[g].w);
      }
    }
  }
  // Rows leave through shared memory with neighbouring columns in neighbouring lanes. l = 0:
  // padding nodes, which came as parts that saw nothing.
#pragma unroll
  for (int g = 0; g < COLS; ++g) {
    part[warp][2 + 4 * g][lane] = o[g].x;
    part[warp][3 + 4 * g][lane] = o[g].y;
    part[warp][4 + 4 * g][lane] = o[g].z;
    part[warp][5 + 4 * g][lane] = o[g].w;
  }
  const int rows = min(32, n_rows - chunk * 32);
  if constexpr (!SPLIT) {
    part[warp][0][lane] = l;
    __syncwarp();
    const bool in = g0 * 4 + lane < a.head_dim;
#pragma unroll 4
    for (int row = 0; row < rows; ++row) {
      T *dst = reinterpret_cast<T *>(
          __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(out), row));
      const float sum = part[warp][0][row], v = part[warp][2 + lane][row];
      if (in) dst[lane] = from_f<T>(sum != 0.f ? v / sum : 0.f);
    }
  } else {
    part[warp][0][lane] = m;
    part[warp][1][lane] = l;
    __syncthreads();
    if (warp == 0) {
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) top = fmaxf(top, part[w][0][lane]);
      const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = ex2(part[w][0][lane] - ref);
        factor[w][lane] = f;
        sum += part[w][1][lane] * f;
      }
      factor[4][lane] = sum;
    }
    __syncthreads();
    // Eight rows of four columns per warp.
    const int row = warp * 8 + lane / 4, x = lane & 3;
    T *dst = reinterpret_cast<T *>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(out), row));
    const float sum = factor[4][row];
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) v += part[w][2 + x][row] * factor[w][row];
    if (row < rows && g0 * 4 + x < a.head_dim) dst[x] = from_f<T>(sum != 0.f ? v / sum : 0.f);
  }
}

template <typename T, int HD, bool TREE, bool VEC>
cudaError_t run(const DenseArgs &a, int grid, cudaStream_t s) {
  auto *kernel = k_dense_cc<T, HD, TREE, VEC>;
  const int smem = (int)sizeof(Smem<HD, BUFFERS<T, HD, VEC>>);
  static SmemLimit limit;
  cudaError_t e = limit.raise(reinterpret_cast<const void *>(kernel), smem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, NT, smem, s>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dense_join(const DenseArgs &a, int grid, int rows, int keys, cudaStream_t s) {
  const int all = a.nodes * a.group, blocks = (all + rows - 1) / rows;
  const int chunks = ((rows < all ? rows : all) + 31) / 32;
  cudaLaunchAttribute attr = {};
  // The launch overlaps the end of the kernel before it; the kernel itself waits for its results.
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const int cols = (a.head_dim + 3) / 4;
  const int64_t units = (int64_t)a.batch * a.n_kv * blocks;
  // `grid` shares over `units` units: up to about 40 units (four parts or more each) the parts of a
  // unit are split over warps, four columns per block; otherwise 128 columns per block.
  const bool split = units * 4 <= grid;
  const int block_cols = split ? 1 : 32;
  cfg.gridDim = dim3((unsigned)units, (unsigned)(chunks * ((cols + block_cols - 1) / block_cols)));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const int pad = dense_hd_pad(a.head_dim);
  cudaError_t e = cudaErrorInvalidValue;
  with_dtype(a.dtype, [&](auto tag) {
    using T = decltype(tag);
    auto go = [&](auto sp) {
      constexpr bool S = decltype(sp)::value;
      e = keys == 64    ? cudaLaunchKernelEx(&cfg, k_dense_join<T, 64, 64, S>, a, grid, pad)
          : rows == 128 ? cudaLaunchKernelEx(&cfg, k_dense_join<T, 128, 128, S>, a, grid, pad)
                        : cudaLaunchKernelEx(&cfg, k_dense_join<T, 256, 128, S>, a, grid, pad);
    };
    if (split) go(std::true_type{});
    else go(std::false_type{});
  });
  count_launches(1);
  return e;
}

cudaError_t launch_dense_cc(const DenseArgs &a, cudaStream_t s) {
  const int64_t v = a.dtype == ISKV_F32 ? 4 : 8;
  auto wide = [&](const iskv_heads &x) {
    return a.head_dim % v == 0 && reinterpret_cast<uintptr_t>(x.data) % 16 == 0 &&
           (!a.tree || x.batch % v == 0) && x.row % v == 0 && x.head % v == 0;
  };
  const bool vec = wide(a.k) && wide(a.v) && (!a.tree || (wide(a.kc) && wide(a.vc)));
  const int64_t grid = a.tree ? DENSE_CC_GRID
                              : (a.rows * a.group / ROWS + a.batch) * (int64_t)a.n_kv;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  with_dtype(a.dtype, [&](auto tag) {
    using T = decltype(tag);
    auto width = [&](auto hd) {
      constexpr int HD = decltype(hd)::value;
      auto mode = [&](auto tree) {
        constexpr bool TREE = decltype(tree)::value;
        e = vec ? run<T, HD, TREE, true>(a, (int)grid, s)
                : run<T, HD, TREE, false>(a, (int)grid, s);
      };
      if (a.tree) mode(std::true_type{});
      else mode(std::false_type{});
    };
    const int pad = dense_hd_pad(a.head_dim);
    if (pad == 64) width(std::integral_constant<int, 64>{});
    else if (pad == 128) width(std::integral_constant<int, 128>{});
    else width(std::integral_constant<int, 256>{});
  });
  if (e == cudaSuccess && a.tree) e = launch_dense_join(a, (int)grid, ROWS, KT, s);
  return e;
}

}  // namespace iskv

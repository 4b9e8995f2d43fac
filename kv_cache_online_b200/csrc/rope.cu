// Rotary embedding of row vectors (iskv_rope).
//
// x'[j]        = x[j] cos a - x[j + hd/2] sin a
// x'[j + hd/2] = x[j + hd/2] cos a + x[j] sin a,   a = +-pos * theta^(-2j/hd).
//
// Angles: w_j = theta^(-2j/hd) / 2 pi turns per position as a 0.64 fixed-point fraction; pos * w_j
// modulo 2^64 is the angle modulo one turn, exact but for w_j's own error (for theta >= 1 less than
// pos * 2^-63 turns: the truncation, and half of that again from its 64-bit logarithm and
// exponential).
// The two top bits after rounding pick the quadrant, the rest (|r| <= 1/8 turn) goes to the sine
// and cosine: CUDA's sincospif for float32, the hardware's for two-byte elements, whose own
// rounding (2^-12 and up) is far above the hardware's 2^-21.
//
// HBM bound: 2 * n * heads * hd elements. A thread owns 16 bytes at j and at j + hd/2 of one row,
// forms their angles once and walks the heads with four pairs of loads in flight; short calls
// spread the heads over more threads instead.
#include "common.cuh"
#include "dense.h"
#include "profiling.h"

#include <cmath>

namespace iskv {
namespace {

struct RopeTable {
  uint64_t w[128];
};

template <typename T>
ISKV_DEV void turn_sincos(uint64_t f, float &c, float &s) {
  const uint32_t quad = (uint32_t)((f + (1ull << 61)) >> 62);
  const int64_t r = (int64_t)(f - ((uint64_t)quad << 62));  // [-2^61, 2^61) / 2^64 turns
  const float half_turns = (float)(int32_t)(r >> 30) * 1.1641532182693481e-10f;  // 2^-33
  float c0, s0;
  if constexpr (sizeof(T) == 4) {
    sincospif(half_turns, &s0, &c0);
  } else {
    __sincosf(half_turns * 3.14159265358979f, &s0, &c0);
  }
  const float a = quad & 1 ? s0 : c0, b = quad & 1 ? c0 : s0;
  c = (quad == 1 || quad == 2) ? -a : a;
  s = quad >= 2 ? -b : b;
}

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

template <typename T, int V>
__global__ void __launch_bounds__(256) k_rope(RopeArgs a, const __grid_constant__ RopeTable tab,
                                              int lanes, int heads_per) {
  const int half = a.head_dim / 2;
  const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t row = idx / lanes;
  if (row >= a.n) return;
  const int j = (int)(idx - row * lanes) * V;
  const int64_t pos = a.inverse ? -(int64_t)a.pos[row] : (int64_t)a.pos[row];
  float c[V], s[V];
#pragma unroll
  for (int e = 0; e < V; ++e) turn_sincos<T>((uint64_t)pos * tab.w[j + e], c[e], s[e]);
  const T *x = static_cast<const T *>(a.x) + row * a.x_row + j;
  T *o = static_cast<T *>(a.out) + row * a.o_row + j;
  const int h0 = blockIdx.y * heads_per, h1 = min(h0 + heads_per, a.heads);
  constexpr int U = 4;
  using Q = Vec<T, V>;
  for (int h = h0; h < h1; h += U) {
    Q lo[U], hi[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h + u < h1) {
        lo[u] = *reinterpret_cast<const Q *>(x + (int64_t)(h + u) * a.x_head);
        hi[u] = *reinterpret_cast<const Q *>(x + (int64_t)(h + u) * a.x_head + half);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h + u < h1) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float p = to_f(lo[u].e[e]), q = to_f(hi[u].e[e]);
          lo[u].e[e] = from_f<T>(fmaf(p, c[e], -__fmul_rn(q, s[e])));
          hi[u].e[e] = from_f<T>(fmaf(q, c[e], __fmul_rn(p, s[e])));
        }
        *reinterpret_cast<Q *>(o + (int64_t)(h + u) * a.o_head) = lo[u];
        *reinterpret_cast<Q *>(o + (int64_t)(h + u) * a.o_head + half) = hi[u];
      }
  }
}

// theta^(-2j/hd) / 2 pi modulo 1 as 0.64 fixed point. The last table is kept per thread: a model
// uses one (theta, head_dim).
const RopeTable &rope_table(double theta, int hd) {
  thread_local RopeTable tab;
  thread_local double have_theta = 0.0;
  thread_local int have_hd = 0;
  if (have_theta != theta || have_hd != hd) {
    const long double two_pi = 6.283185307179586476925286766559005768L;
    const long double lt = logl((long double)theta);
    for (int j = 0; j < hd / 2; ++j) {
      long double w = expl(-2.0L * j / hd * lt) / two_pi;
      w -= floorl(w);
      tab.w[j] = (uint64_t)(w * 18446744073709551616.0L);
    }
    have_theta = theta;
    have_hd = hd;
  }
  return tab;
}

template <typename T, int V>
cudaError_t run(const RopeArgs &a, cudaStream_t s) {
  const int lanes = a.head_dim / 2 / V;
  const int64_t threads = a.n * lanes;
  // Heads per thread: as many as leave every SM (148) about 1,024 threads, at least one.
  int64_t per = threads * a.heads / (148 * 1024);
  per = per < 1 ? 1 : per > a.heads ? a.heads : per;
  const dim3 grid((unsigned)((threads + 255) / 256), (unsigned)((a.heads + per - 1) / per));
  k_rope<T, V><<<grid, 256, 0, s>>>(a, rope_table(a.theta, a.head_dim), lanes, (int)per);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  with_dtype(a.dtype, [&](auto tag) {
    using T = decltype(tag);
    constexpr int V = 16 / sizeof(T);
    // 16-byte accesses where every (row, head, half) starts on 16 bytes, else one element each.
    const bool wide = a.head_dim / 2 % V == 0 && a.x_row % V == 0 && a.x_head % V == 0 &&
                      a.o_row % V == 0 && a.o_head % V == 0 &&
                      reinterpret_cast<uintptr_t>(a.x) % 16 == 0 &&
                      reinterpret_cast<uintptr_t>(a.out) % 16 == 0;
    e = wide ? run<T, V>(a, s) : run<T, 1>(a, s);
  });
  return e;
}

}  // namespace iskv

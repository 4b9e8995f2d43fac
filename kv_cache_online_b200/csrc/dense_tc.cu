// Dense attention on the tensor cores (tcgen05): bf16 and fp16, head_dim up to 128.
//
// Mathematics: one pass over the keys in tiles of 128, half a tile at a time. Per row, with
// x = scale log2(e) q.k,
//   S = Q K^T;  m: reference maximum;  P = 2^(x - m + bias);  l += sum P;  O += P V;  out = O / l.
// (the online softmax of Milakov and Gimelshein, 2018). m only moves when a row's maximum exceeds
// it by more than 8 (a factor 2^8 in P, harmless in the float32 sums; published for attention on
// this chip in 2025 as conditional rescaling): then l and O are multiplied by 2^(m - m'). P enters
// the second product in the element type (half a step of relative rounding per weight, as the
// output's own); bias is 0 for bf16 and 6 for fp16, which moves fp16's subnormal range from 2^-14
// to 2^-20 of the largest weight. l sums the unrounded float32 values. S, m, l and O are float32.
//
// Streams: two per CTA, each with its own softmax warpgroup, MMA warp, two S and one O, so that one
// stream's exponentials run under the other's products. MODE_PROMPT and MODE_ROWS give each stream
// its own 128 rows over the same key tiles; MODE_KEYS (a tree of at most 128 packed rows) gives
// both the same rows and every other tile, and adds the two results up at the end.
//
// What bounds it: for 64 keys of both streams at head_dim 128 the products take 1,288 clocks of an
// SM (P V: 4 MMAs of 65; S: 8 MMAs of N = 64, which take 48 and not 32 because the A operand comes
// from shared memory), the exponentials 1,034 (a warp's 32 in 8). Measured 1,350 over a
// 32,768-token prompt: 7.4 ms = 1.19 PFLOP/s, call after call under the power cap. Short units pay
// about 5 us before the first S (unit lookup among eight sequences 1.5, queries 2.5) and 2.5 us
// after the last. Trees with few rows are bound by HBM instead (the cache crosses once).
//
// One S of 128 keys per stream left the softmax waiting for two products in a row (4,400 clocks for
// 128 keys; 2,700 now). Also measured and not kept: two threads per row (8 % slower: the exchange
// of the maxima), an eighth or a quarter of the exponentials as a polynomial on the FMA pipe (4 to
// 7 % slower at head_dim 128, no gain at 64), ex2.approx.f16x2 (the rate per element is the same).
//
// Warps: 0-3 and 4-7 softmax of stream 0 and 1 (thread = row; P goes back to tensor memory in S's
// place, as the A operand of the second product); 8 loads key and value tiles by TMA into a ring; 9
// and 10 issue the MMAs of stream 0 and 1; 11 looks through value tiles of which some row must not
// see some key, and replaces what is not finite by zero before the MMA reads it (0 * NaN would
// reach every row); if such a value is seen by some row, the epilogue adds it to exactly the rows
// that see it.
//
// Tensor memory (512 columns): two S of 128 x 64 per stream at 0 and 128 (P over the first half of
// each), O0, O1 at 256.
#include "dense.cuh"
#include "profiling.h"
#include "tc_sm100.cuh"

#include <cudaTypedefs.h>

#include <cstring>

namespace iskv {
namespace {

using namespace dense;
using namespace tc;

constexpr int KT = 128;
constexpr uint64_t WAIT_NS = 2000000000ull;
constexpr float LAZY = 8.f;  // log2 of the growth of a row's maximum that is left in P
enum { MODE_PROMPT = 0, MODE_ROWS = 1, MODE_KEYS = 2 };
constexpr int MAX_SLOTS = 8;

struct Maps {
  CUtensorMap k, v, kc, vc;  // kc, vc: tree
  // 0: the axis has stride 0 or length one, every index reads its one element
  int32_t k_head, v_head, kc_head, vc_head, k_batch, v_batch, kc_batch, vc_batch;
};

struct Ctl {
  uint64_t kv_full[MAX_SLOTS], kv_empty[MAX_SLOTS];
  // A value tile that needs the check: the loader has issued it (until then the parity of kv_full
  // says nothing about it), the check has passed it. A phase each per checked use of the slot,
  // which is not refilled before the MMA has read it.
  uint64_t v_req[MAX_SLOTS], v_ok[MAX_SLOTS];
  uint64_t q_full[2], s_full[2][2], p_full[2][2];  // [stream][half of the tile's keys]
  uint64_t o_full[2];      // a phase per product P V; read only where the one before is complete
  uint64_t o_last[2];      // a phase per unit: its last P V
  uint64_t both, drain;
  uint32_t tmem;
  int abort;
  int fix[8];              // unit number whose masked value tiles held something not finite
};

template <int HD, int MODE>
struct Cfg {
  static constexpr int SLABS = HD / 64;
  static constexpr int TILE = KT * HD * 2;                  // bytes of 128 rows
  static constexpr int NQ = MODE == MODE_KEYS ? 1 : 2;
  static constexpr int ROWS = 128 * NQ;                     // packed rows of a unit
  static constexpr int AHEAD = MODE == MODE_KEYS ? 2 : 1;   // key tiles ahead of the value tile
  // As many ring slots as fit beside the query tiles in 227 KB, at most 8.
  static constexpr int REST = (int)sizeof(Ctl) + (MODE == MODE_KEYS ? 2048 : 0);  // + m, l
  static constexpr int FIT = (232448 - REST - NQ * TILE) / TILE;
  static constexpr int SLOTS = FIT < MAX_SLOTS ? FIT : MAX_SLOTS;
  static constexpr int SMEM = NQ * TILE + SLOTS * TILE + REST;
};

ISKV_DEV void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w,
                          uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

ISKV_DEV void tmem_ld32(uint32_t taddr, float *v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

ISKV_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

ISKV_DEV float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <typename T>
ISKV_DEV uint32_t pack2(float a, float b) {
  if constexpr (std::is_same<T, __half>::value) {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
  } else {
    return pack_bf16(a, b);
  }
}

// The weights 2^(s c + off) of 32 scores as 16 packed pairs, added to sum.
template <typename T>
ISKV_DEV void weights(const float *s, float c, float off, float2 (&sum)[2], uint32_t (&p)[16]) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float2 x = __ffma2_rn(make_float2(s[2 * e], s[2 * e + 1]), make_float2(c, c),
                          make_float2(off, off));
    x.x = ex2(x.x);
    x.y = ex2(x.y);
    sum[e & 1] = __fadd2_rn(sum[e & 1], x);
    p[e] = pack2<T>(x.x, x.y);
  }
}

// Bits of the exponent of two packed elements; all set: not finite.
template <typename T>
constexpr uint32_t EXP_BITS = std::is_same<T, __half>::value ? 0x7C007C00u : 0x7F807F80u;

template <typename T>
ISKV_DEV bool finite_bits(T x) {
  const uint32_t e = EXP_BITS<T> & 0xffffu;
  return (*reinterpret_cast<const uint16_t *>(&x) & e) != e;
}

// kind::f16 instruction descriptor: float32 accumulator, A and B of type T, A K-major; b_mn: B is
// MN-major.
template <typename T>
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool b_mn) {
  return (1u << 4) | (std::is_same<T, __half>::value ? 0u : (1u << 7) | (1u << 10)) |
         (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

ISKV_DEV int64_t at(const iskv_heads &x, int64_t b, int64_t row, int64_t head) {
  return b * x.batch + row * x.row + head * x.head;
}

// The CTA's units in order, the same for every warp (whole-warp calls).
template <int MODE, int ROWS>
struct Walk {
  TreeLine<ROWS, KT> line;
  int count = 0;  // units handed out so far

  ISKV_DEV void begin(const DenseArgs &a) {
    if constexpr (MODE != MODE_PROMPT) line.begin(a, gridDim.x, blockIdx.x);
  }
  ISKV_DEV bool next(const DenseArgs &a, Unit &u) {
    if constexpr (MODE == MODE_PROMPT) {
      // One unit per CTA: the block scheduler hands the next one to the SM that is free first (148
      // resident CTAs with every 148th unit each took 4 % longer at 32,768 tokens).
      const int rank = blockIdx.x / a.n_kv;
      if (count || !find_prompt_unit<ROWS>(a, rank, u)) return false;
      u.kvh = blockIdx.x - rank * a.n_kv;
      u.t0 = 0;
      u.t1 = u.n_tiles = last_token(a, u) / KT + 1;
      u.cache_tiles = 0;
      u.open = first_token(a, u) + 1;
    } else {
      if (!line.next(a, u)) return false;
      u.open = u.len;
    }
    ++count;
    return true;
  }
};

// Half tiles (64 keys) that stream s takes of the unit.
template <int MODE>
ISKV_DEV int stream_halves(const DenseArgs &a, const Unit &u, int s) {
  if (MODE == MODE_PROMPT)
    return u.n_rows <= 128 * s
               ? 0
               : (u.row0 + min(u.n_rows, 128 * (s + 1)) - 1) / a.group / (KT / 2) + 1;
  const int n = u.t1 - u.t0;
  const int tiles = MODE == MODE_KEYS ? (n + 1 - s) / 2 : u.n_rows > 128 * s ? n : 0;
  if (tiles == 0) return 0;
  // The stream's last tile may have nothing in its second half.
  const int t = MODE == MODE_KEYS ? u.t0 + 2 * tiles - 2 + s : u.t1 - 1;
  const int keys = t < u.cache_tiles ? u.len - t * KT : a.nodes - (t - u.cache_tiles) * KT;
  return 2 * tiles - (keys <= KT / 2);
}

// First key row of tile t that some row of the unit must not see (>= KT: all rows see all keys).
template <int MODE>
ISKV_DEV int hidden_from(const Unit &u, int t) {
  return MODE == MODE_PROMPT || t < u.cache_tiles ? u.open - t * KT : 0;
}

// Whole warp: wait for the phase of the given parity; false after WAIT_NS or once another warp gave
// up (the same for all lanes). The clock is read every 64th try only.
ISKV_DEV bool warp_try(uint64_t *bar, uint32_t parity) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "vote.sync.all.pred p, p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return r != 0;
}
ISKV_DEV bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
  if (warp_try(bar, parity)) return true;
  uint64_t t0 = 0;
  for (int i = 1;; ++i) {
    if (warp_try(bar, parity)) return true;
    if (i % 64) continue;
    const uint64_t t = __shfl_sync(0xffffffffu, globaltimer(), 0);
    if (t0 == 0) t0 = t;
    if (__any_sync(0xffffffffu, *abort != 0 || t - t0 > WAIT_NS)) {
      *abort = 1;
      return false;
    }
  }
}

// One lane of the warp (all lanes ask): 1 for it, 0 for the others.
ISKV_DEV uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r;
}
// The tcgen05 instructions issued by the lane with `leader` set.
ISKV_DEV void mma_ss(uint32_t leader, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                     uint32_t id, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %5, 0;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(id), "r"(accumulate ? 1u : 0u), "r"(leader)
      : "memory");
}
ISKV_DEV void mma_ts(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                     uint32_t id, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %5, 0;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(id), "r"(accumulate ? 1u : 0u), "r"(leader)
      : "memory");
}
ISKV_DEV void commit(uint32_t leader, uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar)),
      "r"(leader)
      : "memory");
}

template <typename T, int HD, int MODE>
__global__ void __launch_bounds__(384, 1)
    k_dense_tc(const __grid_constant__ DenseArgs a, const __grid_constant__ Maps maps) {
  using C = Cfg<HD, MODE>;
  constexpr bool TREE = MODE != MODE_PROMPT;
  if constexpr (TREE) asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ __align__(1024) char base[];
  Ctl &ctl = *reinterpret_cast<Ctl *>(base + (C::NQ + C::SLOTS) * C::TILE);
  const uint32_t q_smem = smem_u32(base), ring_smem = q_smem + C::NQ * C::TILE;
  // (a shuffle, so that the compiler knows it uniform)
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x / 32, 0), lane = threadIdx.x & 31;
  volatile int *abort = &ctl.abort;

  // The swizzle needs tiles on 1,024 bytes, which the declaration asks for.
  if (q_smem & 1023) {
    if (threadIdx.x == 0) report(a.status, ISKV_ERR_ARG);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(&ctl.kv_full[i], 1);
      mbar_init(&ctl.kv_empty[i], 2);
      mbar_init(&ctl.v_req[i], 1);
      mbar_init(&ctl.v_ok[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.q_full[i], MODE == MODE_KEYS ? 8 : 4);
      mbar_init(&ctl.s_full[i][0], 1);
      mbar_init(&ctl.s_full[i][1], 1);
      mbar_init(&ctl.p_full[i][0], 4);
      mbar_init(&ctl.p_full[i][1], 4);
      mbar_init(&ctl.o_full[i], 1);
      mbar_init(&ctl.o_last[i], 1);
    }
    mbar_init(&ctl.both, 8);
    mbar_init(&ctl.drain, 2);
    ctl.abort = 0;
    for (int i = 0; i < 8; ++i) ctl.fix[i] = 0;
    fence_barrier_init();
  }
  if (warp == 9) tmem_alloc(&ctl.tmem, 512);
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  // All 512 columns are this CTA's: its tensor memory begins at address 0.
  constexpr uint32_t tmem = 0, O_COL = 256;

  Walk<MODE, C::ROWS> walk;
  Unit u;
  walk.begin(a);

  // Registers: 256 x 192 + 128 x 120 = 64,512, the launch's 384 x 168.
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    // ------------------------------------------------------------------------- softmax
    const int st = warp / 4, quad = warp & 3;     // stream; 32 rows
    const int row = quad * 32 + lane;             // row of the stream's tile
    const uint32_t lanes = (uint32_t)quad << 21;  // TMEM lane base of the warp
    const uint32_t o_tm = tmem + lanes + O_COL + HD * st;
    const float c = score_factor(a);
    constexpr float BIAS = std::is_same<T, __half>::value ? 6.f : 0.f;
    char *q_tile = base + (MODE == MODE_KEYS ? 0 : st) * C::TILE;
    const int row_off = MODE == MODE_KEYS ? 0 : 128 * st;  // first unit row of the tile
    // A warp's share of a row's columns, for queries and outputs, in 16-byte pieces: the same
    // bytes of the query tile in both.
    constexpr int CW = HD / 8 / (MODE == MODE_KEYS ? 2 : 1);
    const int ch0 = MODE == MODE_KEYS ? CW * st : 0;
    auto piece = [&](int r, int ch) {  // K-major, 128-byte swizzle
      return q_tile + (ch / 8) * 16384 + r * 128 + (((ch & 7) ^ (r & 7)) * 16);
    };
    uint32_t ph_s = 0, ph_o = 0, ph_both = 0;  // ph_s: a bit per half
    uint32_t n_pv = 0;               // products of the stream in earlier units: phases of o_full
    bool ok = true;
    // All softmax warps have come here.
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.both);
      ok = warp_wait(&ctl.both, ph_both, abort);
      ph_both ^= 1;
      return ok;
    };

    while (ok && walk.next(a, u)) {
      const int n_mine = stream_halves<MODE>(a, u, st);
      const int tile_rows = u.n_rows - row_off;  // rows of this stream's tile, may exceed 128
      const int64_t row_base = TREE ? 0 : u.base;
      const int entry = TREE ? u.b : 0;
      const int pr = u.row0 + row_off + row;  // packed row, its token (tree: node) and its head
      const int tok = pr / a.group;
      const int64_t head = (int64_t)u.kvh * a.group + (pr - tok * a.group);

      // Queries into shared memory, with the scale's sign: every warp its columns of its 32 rows,
      // all loads in flight at once; lane i holds row i's address. (A stream without tiles skips
      // the unit, so that it cannot run ahead of the MMA warp.)
      if (MODE == MODE_KEYS || n_mine > 0) {
        const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
        // (Rows beyond the tile read its last one and become zero: a load under a condition waits
        // for the one before it, 0.2 us each.)
        const int pq = u.row0 + row_off + min(row, max(tile_rows, 1) - 1), tq = pq / a.group;
        const uint64_t row_at = reinterpret_cast<uint64_t>(
            static_cast<const T *>(a.q.data) +
            at(a.q, entry, row_base + tq, (int64_t)u.kvh * a.group + (pq - tq * a.group)));
        const int ch = ch0 + lane % CW;
        const uint64_t col_off = (uint64_t)min(ch, a.head_dim / 8 - 1) * 16;
        const bool col_in = ch * 8 < a.head_dim;
        const uint4 *src[CW];
        uint4 x[CW];
#pragma unroll
        for (int i = 0; i < CW; ++i)
          src[i] = reinterpret_cast<const uint4 *>(
              __shfl_sync(0xffffffffu, row_at, (32 * i + lane) / CW) + col_off);
#pragma unroll
        for (int i = 0; i < CW; ++i) x[i] = *src[i];
#pragma unroll
        for (int i = 0; i < CW; ++i) {
          const int r = quad * 32 + (32 * i + lane) / CW;
          const uint32_t keep = col_in && r < tile_rows ? 0xffffffffu : 0u;
          *reinterpret_cast<uint4 *>(piece(r, ch)) =
              make_uint4((x[i].x ^ flip) & keep, (x[i].y ^ flip) & keep, (x[i].z ^ flip) & keep,
                         (x[i].w ^ flip) & keep);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.q_full[MODE == MODE_KEYS ? 0 : st]);
      }

      const bool busy = quad * 32 < tile_rows;  // the warp has a row
      uint32_t mask[4] = {0, 0, 0, 0};
      if constexpr (TREE) {
        if (busy) node_mask(a, a.parents + (int64_t)u.b * a.nodes, min(tok, a.nodes - 1), mask);
      }

      // m: the reference maximum; past top_lim it moves; off = BIAS - m c.
      float m = -INFINITY, l = 0.f, top_lim = -INFINITY, off = BIAS;
      auto step = [&](auto half, int i) {
        constexpr int h = decltype(half)::value;
        if (!warp_wait(&ctl.s_full[st][h], ph_s >> h & 1, abort)) return false;
        ph_s ^= 1u << h;
        fence_after_sync();
        if (busy) {
          const uint32_t s_tm = tmem + lanes + 128 * st + 64 * h;
          float s[64], top[4];
          tmem_ld32(s_tm, s);
          tmem_ld32(s_tm + 32, s + 32);
          tmem_ld_wait();
          const int t = u.t0 + (MODE == MODE_KEYS ? i - h + st : i / 2);
          if (hidden_from<MODE>(u, t) < 64 * h + 64) {
            uint32_t see[2];
            if (!TREE || t < u.cache_tiles) {
              const int n = (TREE ? u.len : tok + 1) - t * KT - 64 * h;  // visible keys
              see[0] = n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
              see[1] = n <= 32 ? 0u : n >= 64 ? 0xffffffffu : (1u << (n - 32)) - 1u;
            } else {
              see[0] = mask[2 * h];
              see[1] = mask[2 * h + 1];
            }
#pragma unroll
            for (int j = 0; j < 64; ++j) s[j] = see[j / 32] >> (j % 32) & 1 ? s[j] : -INFINITY;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) top[j] = fmaxf(s[j], s[j + 4]);
#pragma unroll
          for (int j = 8; j < 64; j += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) top[e] = max3(top[e], s[j + e], s[j + e + 4]);
          const float mn = max3(fmaxf(top[0], top[1]), top[2], top[3]);
          if (__any_sync(0xffffffffu, mn > top_lim)) {
            const float to = fmaxf(m, mn), f = to == -INFINITY ? 1.f : ex2((m - to) * c);
            l *= f;
            m = to;
            off = BIAS - (m == -INFINITY ? 0.f : m * c);
            top_lim = m + fminf(LAZY / c, 3e38f);  // (-inf while m is, whatever c)
            if (i > 0) {
              // The stream's previous product must have left O. (The one before it has: S(i) was
              // issued behind it. The next one waits for this warp.)
              if (!warp_wait(&ctl.o_full[st], (n_pv + i - 1) & 1, abort)) return false;
              fence_after_sync();
#pragma unroll 1
              for (int j = 0; j < HD / 16; ++j) {
                float o[16];
                tmem_ld16(o_tm + 16 * j, o);
                tmem_ld_wait();
                uint32_t r[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(o[e] * f);
                tmem_st16(o_tm + 16 * j, r);
              }
            }
          }
          float2 sum[2] = {make_float2(l, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t p[16];
            weights<T>(s + 32 * j, c, off, sum, p);
            tmem_st16(s_tm + 16 * j, p);
          }
          sum[0] = __fadd2_rn(sum[0], sum[1]);
          l = sum[0].x + sum[0].y;
          tmem_st_wait();
          fence_before_sync();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.p_full[st][h]);
        return true;
      };
      for (int i = 0; i < n_mine; i += 2) {
        ok = step(std::integral_constant<int, 0>{}, i);
        if (ok && i + 1 < n_mine) ok = step(std::integral_constant<int, 1>{}, i + 1);
        if (!ok) break;
      }
      if (!ok) break;

      // Epilogue. All products of the stream are complete, its query tile is idle.
      if (n_mine > 0) {
        n_pv += n_mine;
        ok = warp_wait(&ctl.o_last[st], ph_o, abort);
        ph_o ^= 1;
        if (!ok) break;
      }
      float w[2] = {0.f, 0.f};  // weights of the two streams' O
      float ml = m == -INFINITY ? -INFINITY : m * c;
      const bool two = MODE == MODE_KEYS && stream_halves<MODE>(a, u, 1) > 0;
      if constexpr (MODE == MODE_KEYS) {
        float *stat = reinterpret_cast<float *>(&ctl + 1);
        stat[2 * st * 128 + row] = ml;
        stat[(2 * st + 1) * 128 + row] = l;
        if (!meet()) break;
        const float m0 = stat[row], m1 = stat[256 + row];
        ml = fmaxf(m0, m1);
        const float ref = ml == -INFINITY ? 0.f : ml;
        w[0] = ex2(m0 - ref);
        w[1] = ex2(m1 - ref);
        l = stat[128 + row] * w[0] + (two ? stat[384 + row] * w[1] : 0.f);
      }
      fence_after_sync();
      const bool fix = *(volatile int *)&ctl.fix[walk.count & 7] == walk.count;
      const bool whole = !TREE || (u.t0 == 0 && u.t1 == u.n_tiles);
      const bool mine = row < tile_rows;
      if (busy) {
        const bool live = !TREE || (mask[0] | mask[1] | mask[2] | mask[3]);
        const uint32_t o0 = tmem + lanes + O_COL;
        const float inv = 1.f / l;
        const bool zero = l == 0.f || !live;
        float *slot = static_cast<float *>(a.ws) +
                      (2 * blockIdx.x + (u.t0 > 0 ? 0 : 1)) * dense_slot_floats(C::ROWS, HD);
#pragma unroll 1
        for (int ch = ch0; ch < ch0 + CW; ch += 2) {
          const int col = ch * 8;
          float o[16];
          if constexpr (MODE == MODE_KEYS) {
            float o1[16];
            tmem_ld16(o0 + col, o);
            tmem_ld16(o0 + HD + col, o1);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = two ? o[e] * w[0] + o1[e] * w[1] : o[e] * w[0];
          } else {
            tmem_ld16(o_tm + col, o);
            tmem_ld_wait();
          }
          if (fix && mine && (!TREE || u.t1 > u.cache_tiles)) {
            // Values that were replaced by zero, for the rows that see them.
            const int lo = TREE ? 0 : first_token(a, u) + 1, hi = TREE ? a.nodes : tok + 1;
            const T *v = static_cast<const T *>(a.v.data) + at(a.v, entry, row_base, u.kvh) + col;
            for (int j = lo; j < hi; ++j) {
              if (TREE && !((j < 64 ? j < 32 ? mask[0] : mask[1] : j < 96 ? mask[2] : mask[3]) >>
                            (j & 31) & 1))
                continue;
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                if (col + e >= a.head_dim) break;
                const T x = v[j * a.v.row + e];
                if (!finite_bits(x)) o[e] += to_f(x);
              }
            }
          }
          if (whole) {
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = zero ? 0.f : o[e] * inv;
#pragma unroll
            for (int h = 0; h < 2; ++h)
              *reinterpret_cast<uint4 *>(piece(row, ch + h)) = make_uint4(
                  pack2<T>(o[8 * h], o[8 * h + 1]), pack2<T>(o[8 * h + 2], o[8 * h + 3]),
                  pack2<T>(o[8 * h + 4], o[8 * h + 5]), pack2<T>(o[8 * h + 6], o[8 * h + 7]));
          } else if (mine) {
#pragma unroll
            for (int h = 0; h < 4; ++h)
              reinterpret_cast<float4 *>(slot)[(size_t)(col / 4 + h) * C::ROWS + row_off + row] =
                  make_float4(o[4 * h], o[4 * h + 1], o[4 * h + 2], o[4 * h + 3]);
          }
        }
        if (!whole) {
          if (mine && ch0 == 0) {  // padding nodes: a part that saw nothing
            slot[(size_t)C::ROWS * HD + row_off + row] = live ? ml : -INFINITY;
            slot[(size_t)C::ROWS * (HD + 1) + row_off + row] = live ? l : 0.f;
          }
        } else {
          // Whole rows leave in coalesced 16-byte pieces.
          __syncwarp();
          const uint64_t out = reinterpret_cast<uint64_t>(static_cast<T *>(a.out.data) +
                                                          at(a.out, entry, row_base + tok, head));
          const int ch = ch0 + lane % CW;
#pragma unroll
          for (int i = 0; i < CW; ++i) {
            const int r = (32 * i + lane) / CW;
            const uint64_t dst = __shfl_sync(0xffffffffu, out, r);
            if (quad * 32 + r < tile_rows && ch * 8 < a.head_dim)
              *reinterpret_cast<uint4 *>(dst + ch * 16) =
                  *reinterpret_cast<const uint4 *>(piece(quad * 32 + r, ch));
          }
          __syncwarp();
        }
      }
      fence_before_sync();
      // Both O and the statistics are read by both streams: neither goes on before the other.
      if constexpr (MODE == MODE_KEYS) {
        if (!meet()) break;
        fence_after_sync();
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
    if (warp == 8) {
      // ------------------------------------------------------------------------- loads
      RingPos pos;
      int issued = 0;
      bool ok = true;
      while (ok && walk.next(a, u)) {
        if (lane == 0) {
          const int n = u.t1 - u.t0;
          auto load = [&](int t, bool value) {
            if (!ok) return;
            if (!mbar_wait(&ctl.kv_empty[pos.slot], pos.phase ^ 1, abort, WAIT_NS)) {
              ok = false;
              ctl.abort = 1;
              return;
            }
            const bool cache = TREE && t < u.cache_tiles;
            const CUtensorMap *map =
                cache ? (value ? &maps.vc : &maps.kc) : (value ? &maps.v : &maps.k);
            const int head = u.kvh * (cache ? (value ? maps.vc_head : maps.kc_head)
                                            : (value ? maps.v_head : maps.k_head));
            const int entry = TREE ? u.b * (cache ? (value ? maps.vc_batch : maps.kc_batch)
                                                  : (value ? maps.v_batch : maps.k_batch))
                                   : 0;
            const int row = TREE ? (cache ? t : t - u.cache_tiles) * KT : (int)u.base + t * KT;
            const uint32_t dst = ring_smem + pos.slot * C::TILE;
            mbar_arrive_expect_tx(&ctl.kv_full[pos.slot], C::TILE);
            if (value && hidden_from<MODE>(u, t) < KT) mbar_arrive(&ctl.v_req[pos.slot]);
            for (int s = 0; s < C::SLABS; ++s)
              tma_load_4d(dst + s * 16384, map, s * 64, head, row, entry, &ctl.kv_full[pos.slot]);
            ++issued;
            pos.next(C::SLOTS);
          };
          for (int i = 0; i < C::AHEAD && i < n; ++i) load(u.t0 + i, false);
          for (int i = 0; i < n; ++i) {
            load(u.t0 + i, true);
            if (i + C::AHEAD < n) load(u.t0 + i + C::AHEAD, false);
          }
        }
        ok = __shfl_sync(0xffffffffu, (int)ok, 0);
      }
      if (lane == 0) {
        // Copies in flight land before the CTA ends (after a timeout nobody else waits for them):
        // the last use of every slot that was issued.
        RingPos p;
        for (int i = 0; i < issued; ++i) {
          if (i + C::SLOTS >= issued) {
            const uint64_t t0 = globaltimer();
            while (!mbar_try_wait(&ctl.kv_full[p.slot], p.phase) && globaltimer() - t0 < WAIT_NS) {
            }
          }
          p.next(C::SLOTS);
        }
      }
    } else if (warp < 11) {
      // ------------------------------------------------------------------------- MMAs A warp per
      // stream: what it takes to see that a P has come and to issue the next products is longer
      // than the products, and two warps overlap it (one warp for both: 1,740 clocks for 64 keys of
      // both streams at head_dim 128). The whole warp walks through the loops in step and one lane
      // issues: addresses and descriptors then stay in uniform registers, where the MMA takes them
      // from. Both warps follow every ring slot, used or not, so that neither loses a phase.
      constexpr uint32_t ID_S = idesc<T>(128, KT / 2, false), ID_O = idesc<T>(128, HD, true);
      const int st = warp - 9;
      const uint32_t leader = elect_one();
      RingPos pos;
      uint32_t ph_q = 0, ph_v = 0, ph_p = 0;  // ph_v: a bit per slot; ph_p: per half
      bool ok = true;
      const uint64_t qd = sw128_desc(q_smem + (MODE == MODE_KEYS ? 0 : st) * C::TILE);
      const uint32_t s_tm = 128 * st, o_tm = O_COL + HD * st;
      auto tile_at = [&](int slot) { return ring_smem + slot * C::TILE; };
      // S over half h of a key tile.
      auto scores = [&](int h, int slot) {
        const uint64_t kd = sw128_desc(tile_at(slot) + h * 8192);
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          const uint32_t off = (k / 4) * 16384 + (k % 4) * 32;
          mma_ss(leader, s_tm + 64 * h, desc_add(qd, off), desc_add(kd, off), ID_S, k > 0);
        }
        commit(leader, &ctl.s_full[st][h]);
      };
      // P V over half h of a value tile, once the softmax has written P.
      auto values = [&](int h, int slot, bool first, bool last) {
        if (!warp_wait(&ctl.p_full[st][h], ph_p >> h & 1, abort)) return false;
        ph_p ^= 1u << h;
        fence_after_sync();
        const uint64_t vd = sw128_mn_desc(tile_at(slot) + h * 8192, 16384);
#pragma unroll
        for (int k = 0; k < KT / 32; ++k)
          mma_ts(leader, o_tm, s_tm + 64 * h + 8 * k, desc_add(vd, k * 2048), ID_O,
                 !first || k > 0);
        commit(leader, &ctl.o_full[st]);
        if (last) commit(leader, &ctl.o_last[st]);
        return true;
      };
      // Two S per stream: the next half's scores are under way while the softmax works on this
      // half's. S(i + 2) goes where P(i) was, behind P(i) V(i) in the same pipe.
      while (ok && walk.next(a, u)) {
        const int n = __shfl_sync(0xffffffffu, u.t1 - u.t0, 0);
        const int n_mine = __shfl_sync(0xffffffffu, stream_halves<MODE>(a, u, st), 0);
        if (MODE == MODE_KEYS || n_mine > 0) {
          ok = warp_wait(&ctl.q_full[MODE == MODE_KEYS ? 0 : st], ph_q, abort);
          ph_q ^= 1;
          fence_after_sync();
        }
        for (int i = 0; ok && i < C::AHEAD && i < n; ++i) {
          ok = warp_wait(&ctl.kv_full[pos.slot], pos.phase, abort);
          if (!ok) break;
          if (MODE != MODE_KEYS || i == st) {
            if (n_mine > 0) scores(0, pos.slot);
            if (n_mine > 1) scores(1, pos.slot);
          }
          commit(leader, &ctl.kv_empty[pos.slot]);
          pos.next(C::SLOTS);
        }
        for (int i = 0; ok && i < n; ++i) {
          const int v_slot = pos.slot;
          ok = warp_wait(&ctl.kv_full[v_slot], pos.phase, abort);
          pos.next(C::SLOTS);
          if (ok && hidden_from<MODE>(u, u.t0 + i) < KT) {
            ok = warp_wait(&ctl.v_ok[v_slot], ph_v >> v_slot & 1, abort);
            ph_v ^= 1u << v_slot;
          }
          const bool more = i + C::AHEAD < n;
          const int k_slot = pos.slot;
          if (ok && more) {
            ok = warp_wait(&ctl.kv_full[k_slot], pos.phase, abort);
            pos.next(C::SLOTS);
          }
          if (!ok) break;
          if (MODE != MODE_KEYS || (i & 1) == st) {
            // the stream's first half of the tile
            const int b = MODE == MODE_KEYS ? i - st : 2 * i;
            if (b < n_mine) {
              ok = values(0, v_slot, b == 0, b + 1 == n_mine);
              if (ok && b + 2 < n_mine) scores(0, k_slot);
            }
            if (ok && b + 1 < n_mine) {
              ok = values(1, v_slot, false, b + 2 == n_mine);
              if (ok && b + 3 < n_mine) scores(1, k_slot);
            }
            if (!ok) break;
          }
          commit(leader, &ctl.kv_empty[v_slot]);
          if (more) commit(leader, &ctl.kv_empty[k_slot]);
        }
      }
      // Every MMA and commit has completed before the CTA gives its tensor memory back.
      commit(leader, &ctl.drain);
      if (lane == 0) {
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(&ctl.drain, 0) && globaltimer() - t0 < WAIT_NS) {
        }
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------------------- value check
      RingPos pos;
      uint32_t ph_req = 0;  // a bit per slot
      bool ok = true;
      while (ok && walk.next(a, u)) {
        const int n = u.t1 - u.t0;
        for (int i = 0; i < C::AHEAD && i < n; ++i) pos.next(C::SLOTS);
        for (int i = 0; i < n && ok; ++i) {
          const int t = u.t0 + i;
          const int r0 = max(0, hidden_from<MODE>(u, t));
          const int r1 = !TREE || t < u.cache_tiles ? KT : a.nodes;
          if (r0 < KT) {
            ok = warp_wait(&ctl.v_req[pos.slot], ph_req >> pos.slot & 1, abort) &&
                 warp_wait(&ctl.kv_full[pos.slot], pos.phase, abort);
            ph_req ^= 1u << pos.slot;
            if (!ok) {
              ctl.abort = 1;
              break;
            }
            // A row is 8 16-byte pieces of each 64-column slab, whatever their swizzled order.
            char *tile = base + (C::NQ + pos.slot) * C::TILE;
            const int p0 = r0 * 8, p1 = r1 * 8;
            uint32_t top = 0;
            for (int s = 0; s < C::SLABS; ++s)
#pragma unroll 4
              for (int p = p0 + lane; p < p1; p += 32) {
                const uint4 x = *reinterpret_cast<const uint4 *>(tile + s * 16384 + p * 16);
                top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                             __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
              }
            constexpr uint32_t E = EXP_BITS<T> & 0xffffu;
            if (__any_sync(0xffffffffu, (top & 0xffffu) >= E || (top >> 16) >= E)) {
              // Cache rows beyond the valid ones, and rows behind a sequence, are seen by nobody.
              const int seen_end = TREE ? (t < u.cache_tiles ? 0 : a.nodes) : u.len - t * KT;
              bool seen = false;
              for (int s = 0; s < C::SLABS; ++s)
                for (int p = p0 + lane; p < p1; p += 32) {
                  uint4 *at16 = reinterpret_cast<uint4 *>(tile + s * 16384 + p * 16);
                  uint4 x = *at16;
                  uint32_t *wd = reinterpret_cast<uint32_t *>(&x);
                  bool hit = false;
                  for (int e = 0; e < 4; ++e) {
                    if ((wd[e] & E) == E) {
                      wd[e] &= 0xffff0000u;
                      hit = true;
                    }
                    if ((wd[e] >> 16 & E) == E) {
                      wd[e] &= 0xffffu;
                      hit = true;
                    }
                  }
                  if (hit) {
                    *at16 = x;
                    seen |= p / 8 < seen_end;
                  }
                }
              if (__any_sync(0xffffffffu, seen) && lane == 0)
                *(volatile int *)&ctl.fix[walk.count & 7] = walk.count;
              fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.v_ok[pos.slot]);
          }
          pos.next(C::SLOTS);
          if (i + C::AHEAD < n) pos.next(C::SLOTS);
        }
      }
    }
  }

  __syncwarp();
  fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && ctl.abort) report(a.status, ISKV_ERR_TIMEOUT);
  if (warp == 9) {
    fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------------------------------------
// Host

// A driver entry point by name, looked up once.
template <typename F>
F driver_fn(const char *name) {
  void *f = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPoint(name, &f, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return nullptr;
  return reinterpret_cast<F>(f);
}
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const auto fn = driver_fn<PFN_cuTensorMapEncodeTiled_v12000>("cuTensorMapEncodeTiled");
  return fn;
}
PFN_cuTensorMapReplaceAddress_v12000 replace_fn() {
  static const auto fn =
      driver_fn<PFN_cuTensorMapReplaceAddress_v12000>("cuTensorMapReplaceAddress");
  return fn;
}

// Two-byte rows as a 4-D tensor {head_dim, heads, rows, entries}, box {64, 1, 128, 1}, 128-byte
// swizzle; what lies outside reads as zero. The thread's last maps are kept by their shape (a
// model's layers differ in addresses alone), which spares a short call an encoding of more than 1
// us each.
bool encode(CUtensorMap *m, int32_t &head_on, int32_t &batch_on, const iskv_heads &x, int hd,
            int heads, int64_t rows, int64_t entries, int dtype) {
  struct Shape {
    cuuint64_t dims[4], strides[3];
    int64_t dtype;
  };
  constexpr int KEEP = 8;
  thread_local Shape shapes[KEEP];
  thread_local CUtensorMap kept[KEEP];
  thread_local int used = 0, next = 0;
  head_on = heads > 1 && x.head > 0;
  batch_on = entries > 1 && x.batch > 0;
  // Axes that are not walked get length one and any legal stride.
  const cuuint64_t any = (cuuint64_t)(hd + 7) / 8 * 16;
  Shape s = {{(cuuint64_t)hd, head_on ? (cuuint64_t)heads : 1, (cuuint64_t)rows,
              batch_on ? (cuuint64_t)entries : 1},
             {head_on ? (cuuint64_t)x.head * 2 : any, x.row > 0 ? (cuuint64_t)x.row * 2 : any,
              batch_on ? (cuuint64_t)x.batch * 2 : any},
             dtype};
  if (replace_fn())
    for (int i = 0; i < used; ++i)
      if (!memcmp(&s, &shapes[i], sizeof s)) {
        *m = kept[i];
        return replace_fn()(m, x.data) == CUDA_SUCCESS;
      }
  cuuint32_t box[4] = {64, 1, KT, 1}, one[4] = {1, 1, 1, 1};
  if (encode_fn()(m, dtype == ISKV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                       : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                  4, x.data, s.dims, s.strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return false;
  shapes[next] = s;
  kept[next] = *m;
  next = (next + 1) % KEEP;
  if (used < KEEP) ++used;
  return true;
}

template <typename T, int HD, int MODE>
cudaError_t run(const DenseArgs &a, const Maps &maps, int grid, cudaStream_t s) {
  auto *kernel = k_dense_tc<T, HD, MODE>;
  constexpr int smem = Cfg<HD, MODE>::SMEM;
  static_assert(smem <= 232448 && Cfg<HD, MODE>::SLOTS >= 4, "ring does not fit");
  static SmemLimit limit;
  cudaError_t e = limit.raise(reinterpret_cast<const void *>(kernel), smem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, 384, smem, s>>>(a, maps);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

// The kernel's tiles are 64 or 128 columns of two bytes in 16-byte pieces, and its tensor memory is
// full at head_dim 128. What it does not take runs far slower: a 4,096-token bf16 prompt, 32 over 8
// heads, takes 135 us here at head_dim 120 and 128, and on the CUDA cores 5.6 ms at 100 and 7.2 ms
// at 256.
bool dense_tc_takes(const DenseArgs &a) {
  if (a.dtype == ISKV_F32 || a.head_dim % 8 || a.head_dim > 128 || !encode_fn()) return false;
  auto fits = [&](const iskv_heads &x, bool rows_walked) {
    return reinterpret_cast<uintptr_t>(x.data) % 16 == 0 && x.row % 8 == 0 && x.head % 8 == 0 &&
           (!a.tree || x.batch % 8 == 0) && (x.row > 0 || !rows_walked);
  };
  const int64_t n = a.tree ? a.nodes : a.rows;
  return fits(a.q, false) && fits(a.out, false) && fits(a.k, n > 1) && fits(a.v, n > 1) &&
         (!a.tree || a.rows == 0 || (fits(a.kc, a.rows > 1) && fits(a.vc, a.rows > 1)));
}

bool launch_dense_tc(const DenseArgs &args, cudaStream_t s, cudaError_t &e) {
  DenseArgs a = args;
  Maps maps = {};
  const int64_t n = a.tree ? a.nodes : a.rows, entries = a.tree ? a.batch : 1;
  bool ok =
      encode(&maps.k, maps.k_head, maps.k_batch, a.k, a.head_dim, a.n_kv, n, entries, a.dtype) &&
      encode(&maps.v, maps.v_head, maps.v_batch, a.v, a.head_dim, a.n_kv, n, entries, a.dtype);
  if (a.tree && a.rows > 0)
    ok = ok &&
         encode(&maps.kc, maps.kc_head, maps.kc_batch, a.kc, a.head_dim, a.n_kv, a.rows, entries,
                a.dtype) &&
         encode(&maps.vc, maps.vc_head, maps.vc_batch, a.vc, a.head_dim, a.n_kv, a.rows, entries,
                a.dtype);
  if (!ok) return false;
  const bool keys = a.tree && a.nodes * a.group <= 128;
  const int rows = keys ? 128 : 256;
  // A tree over a short cache (seven tiles at most and the drafts') is not cut: a unit takes about
  // 0.6 us a tile, the join 4 us and its launch 3.5 us of host time.
  const int64_t units = (int64_t)a.batch * a.n_kv * ((a.nodes * a.group + rows - 1) / rows);
  a.whole = a.tree && a.rows <= 7 * KT && units <= 0x7fffffff;
  const int64_t grid = a.whole  ? units
                       : a.tree ? DENSE_TC_GRID
                                : (a.rows * a.group / rows + a.batch) * (int64_t)a.n_kv;
  if (grid > 0x7fffffff) {
    e = cudaErrorInvalidValue;
    return true;
  }
  auto width = [&](auto tag, auto hd) {
    using T = decltype(tag);
    constexpr int HD = decltype(hd)::value;
    e = !a.tree ? run<T, HD, MODE_PROMPT>(a, maps, (int)grid, s)
        : keys  ? run<T, HD, MODE_KEYS>(a, maps, (int)grid, s)
                : run<T, HD, MODE_ROWS>(a, maps, (int)grid, s);
  };
  auto type = [&](auto tag) {
    if (a.head_dim <= 64) width(tag, std::integral_constant<int, 64>{});
    else width(tag, std::integral_constant<int, 128>{});
  };
  if (a.dtype == ISKV_F16) type(__half{});
  else type(__nv_bfloat16{});
  if (e == cudaSuccess && a.tree && !a.whole)
    e = launch_dense_join(a, (int)grid, rows, KT, s);
  return true;
}

}  // namespace iskv

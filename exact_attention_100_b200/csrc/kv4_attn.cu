// Attention of a few query rows over the 4-bit paged cache (decode, verification of drafted tokens).
//
// O = softmax(scale q K^T) V with K = u_k s_k + z_k and V = u_v s_v + z_v, codes u in 0 .. 15 and (s, z)
// per key and group of 64 dimensions.  Neither K nor V is formed: for a key,
//     q . K = sum_g  s_g (q_g . u_g) + z_g (sum q_g),
//     sum_j p_j V_j = sum_g  u_g^T (p s_g) + sum_j p_j z_jg,
// so the tensor core multiplies the codes themselves, and steps and minima meet them in the small
// products: once per (key, row, group) instead of once per element.
//
// Bound by memory: 1.125 d bytes per key and key/value head for at least 4 d G flops.  The arithmetic has to
// stay under the time the bytes take, about 100 cycles of an SM per 16 keys at d = 128; rows of q are few,
// so the products are the warp's m16n8k16 with keys (then dimensions) on the 16 side and rows on the
// 8 side: an operand register is then a pair of nibbles masked out of a word.  A nibble u masked in
// place is the float16 subnormal u 2^-24 (or, 4 bits up, 16 u 2^-24), which the tensor core
// multiplies exactly: no conversion, 5 logic operations per 8 codes; the factors 16 are taken out of q, and of
// O's rows at the end.  Pairs of V run over two tokens: two byte permutes bring their words together.
//
// One warp works on one tile of 16 keys at a time and keeps its own running maximum, sum and O.  Its tiles
// come through its own ring of shared-memory stages, each filled by one bulk copy (a tile with all its
// scales is contiguous) and watched by one mbarrier: no warp waits for another inside a request's keys.
// The maximum is lazy: it moves only when a score passes it by 2^8, found by one vote per tile.  p s is
// rounded to float16 (11 bits) under a running power-of-two reference of s, moved the same way, so that
// values of V of any size keep their bits.
//
// Work is the requests' tiles laid end to end, (request, kv head, chunk of rows) after another, cut into
// equal spans, one per block of threads.  A block that holds all tiles of a row chunk writes O; others
// leave partial (O, m, l) in the workspace, at most two per block (its first and its last row chunk),
// and the join kernel adds them in order.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_kernels.h"
#include "kv4_format.cuh"
#include "kv_kernels.h"
#include "sm100_ptx.cuh"

namespace ea {

namespace {

constexpr float kTau = 8.f;        // lazy maximum: p <= 2^kTau
constexpr float kNegBig = -1e30f;  // below any score, and finite
constexpr float kLn2f = 0.6931471805599453f;

// A block of threads gets at least this many tiles, two for each of its warps: fewer spans than
// blocks for short contexts, so that less is left to join
constexpr int kMinTiles = 16;

template <int D, int NT>
struct SplitCfg {
  static constexpr int kWarps = 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kRows = 8 * NT;
  static constexpr int kBlocksPerSm = D * NT <= 128 ? 2 : 1;
  static constexpr int kTile = Kv4Tile<D>::kBytes;
  // ring of a warp: about 9 KB, 4 tiles of d = 128 (150 KB in flight per SM; 45 KB cover the latency)
  static constexpr int kStages = D == 64 ? 8 : D == 128 ? 4 : 3;
  static constexpr int kRingOff = 0;
  static constexpr int kQOff = kRingOff + kWarps * kStages * kTile;  // [kRows][D] float
  static constexpr int kRedRow = D + 1;
  static constexpr int kRedOff = kQOff + kRows * D * 4;              // [kWarps][kRows][D + 1] float
  static constexpr int kMlOff = kRedOff + kWarps * kRows * kRedRow * 4;  // m, l: [2][kWarps][kRows]
  static constexpr int kRowFOff = kMlOff + 2 * kWarps * kRows * 4;       // [kRows] score factor
  static constexpr int kBarOff = (kRowFOff + kRows * 4 + 15) / 16 * 16;
  static constexpr int kScanOff = kBarOff + kWarps * kStages * 8;
  static constexpr int kSmem = kScanOff + 1024 * 8 / 4 + 64;
  static_assert(kSmem * kBlocksPerSm + 1024 * kBlocksPerSm <= 228 * 1024, "shared memory of an SM");
};

// Partial results in the workspace: per block of threads two slots of [kRows][D] float O, [kRows] m,
// [kRows] l, then int meta: {tail valid, request, kv head, chunk, head continues}.
template <int D, int NT>
__host__ __device__ constexpr int slot_floats() { return 8 * NT * (D + 2); }

struct Meta {
  int tail_valid;  // the block's last row chunk starts in it and goes on in the next block
  int b, h, chunk;
  int head_valid;  // the block's first row chunk started before it
  int head_ends;   // ... and ends in it
  int pad[2];
};

// A row chunk of one request and key/value head.
struct Item {
  int b, h, chunk;
  int nq, nk, q0;
  int tiles;
};

struct SeqLen {
  int nq, nk, q0;
  bool bad;
};

__device__ __forceinline__ SeqLen seq_len(const Kv4AttnParams& p, int b) {
  SeqLen s;
  int q0 = b, q1 = b + 1;
  if (p.cu_q != nullptr) {
    q0 = __ldg(p.cu_q + b);
    q1 = __ldg(p.cu_q + b + 1);
  }
  const int nk = __ldg(p.lens + b);
  s.bad = !(0 <= q0 && q0 <= q1 && q1 <= p.total_q && q1 - q0 <= p.max_q && nk >= 0 &&
            nk <= static_cast<long long>(p.width) * p.page);
  s.nq = s.bad ? 0 : q1 - q0;
  s.nk = s.bad ? 0 : nk;
  s.q0 = q0;
  // requests of the other launch
  const long long rows = static_cast<long long>(s.nq) * p.G;
  if (rows <= p.min_rows || rows > p.max_rows) s.nq = 0;
  return s;
}

// Tiles of one row chunk of a request (one, with every key masked, where it has no key).
__device__ __forceinline__ int chunk_tiles(int nk) { return nk > 0 ? (nk + 15) >> 4 : 1; }

template <int ROWS>
__device__ __forceinline__ long long seq_tiles(const Kv4AttnParams& p, const SeqLen& s) {
  const long long chunks = (static_cast<long long>(s.nq) * p.G + ROWS - 1) / ROWS;
  return chunks * p.Hk * chunk_tiles(s.nk);
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 2^e for -126 <= e <= 127
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
__device__ __forceinline__ int exponent_of(float x) { return static_cast<int>((__float_as_uint(x) >> 23) & 255u) - 127; }

// After a wait that ran out: waits for the stage's copy all the same (as long again), so that none
// lands after the block has ended.
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
  const unsigned long long t0 = global_timer_ns();
  while (!bar_try_wait(smem_addr(bar), parity))
    if (global_timer_ns() - t0 > kWaitLimitNs) return;
}

// Key of the tile that sits at index a of the products' key side: an order in which the rows that a
// quarter (K) or half (V) warp reads together fall into different banks.
__device__ __forceinline__ int key_at(int a) { return a ^ (((a >> 1) ^ (a >> 2)) & 1); }

template <int D, int NT>
__global__ void __launch_bounds__(SplitCfg<D, NT>::kThreads, SplitCfg<D, NT>::kBlocksPerSm)
    kv4_split_kernel(const Kv4AttnParams p) {
  using C = SplitCfg<D, NT>;
  using F = Kv4Tile<D>;
  constexpr int GR = D / 64;  // scale groups of a row
  constexpr int ROWS = C::kRows;
  extern __shared__ __align__(128) uint8_t smem[];
  float* sq = reinterpret_cast<float*>(smem + C::kQOff);
  float* red = reinterpret_cast<float*>(smem + C::kRedOff);
  float* sm_m = reinterpret_cast<float*>(smem + C::kMlOff);
  float* sm_l = sm_m + C::kWarps * ROWS;
  float* rowf = reinterpret_cast<float*>(smem + C::kRowFOff);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  long long* scan = reinterpret_cast<long long*>(smem + C::kScanOff);
  __shared__ int abort_flag;
  __shared__ long long s_first;  // tiles of the requests before s_b
  __shared__ int s_b;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  uint8_t* ring = smem + C::kRingOff + warp * C::kStages * C::kTile;
  uint64_t* bar = bars + warp * C::kStages;

  if (tid < C::kWarps * C::kStages) bar_init(&bars[tid], 1);
  if (tid == 0) {
    abort_flag = 0;
    s_b = p.B;
    s_first = 0;
  }
  fence_barrier_init();

  // ---- this block's span of the tiles: sums over the requests, a run of them per thread ----------
  const int per = (p.B + C::kThreads - 1) / C::kThreads;
  const int my0 = tid * per, my1 = min(p.B, my0 + per);
  long long mine = 0;
  bool bad = false;
  for (int b = my0; b < my1; ++b) {
    const SeqLen s = seq_len(p, b);
    bad |= s.bad;
    mine += seq_tiles<ROWS>(p, s);
  }
  if (bad && blockIdx.x == 0) atomicOr(p.status, kDevStatusBadSeqlens);
  long long incl = mine;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, incl, s);
    if (lane >= s) incl += o;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  long long total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < C::kWarps; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  const long long blocks = min(static_cast<long long>(gridDim.x), (total + kMinTiles - 1) / kMinTiles);
  Meta* meta = reinterpret_cast<Meta*>(p.ws) + blockIdx.x;
  float* slots = reinterpret_cast<float*>(p.ws + static_cast<size_t>(gridDim.x) * sizeof(Meta)) +
                 static_cast<size_t>(blockIdx.x) * 2 * slot_floats<D, NT>();
  if (blockIdx.x >= blocks) {
    if (tid == 0) *meta = Meta{};
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    return;
  }
  const long long span0 = total * blockIdx.x / blocks, span1 = total * (blockIdx.x + 1) / blocks;
  before += incl - mine;
  if (before <= span0 && span0 < before + mine) {  // one thread: the span starts in its run
    int b = my0;
    for (;; ++b) {
      const long long n = seq_tiles<ROWS>(p, seq_len(p, b));
      if (span0 < before + n) break;
      before += n;
    }
    s_b = b;
    s_first = before;
  }
  __syncthreads();

  const AbortState ab{&abort_flag, p.status};

  // the row chunk and tile at a position of the span: a cursor that only moves forward
  struct Cursor {
    long long first;  // position of the request's first tile
    int b;
    SeqLen s;
    long long n;      // tiles of the request
  };
  auto settle = [&](Cursor& cu, long long pos) {  // the request that holds pos (pos < total)
    while (pos >= cu.first + cu.n) {
      cu.first += cu.n;
      ++cu.b;
      cu.s = seq_len(p, cu.b);
      cu.n = seq_tiles<ROWS>(p, cu.s);
    }
  };
  auto item_at = [&](const Cursor& cu, long long pos, Item& it) -> int {  // returns the tile in the chunk
    it.b = cu.b;
    it.nq = cu.s.nq;
    it.nk = cu.s.nk;
    it.q0 = cu.s.q0;
    it.tiles = chunk_tiles(cu.s.nk);
    const long long rel = pos - cu.first;
    const long long idx = rel / it.tiles;
    const int chunks = (it.nq * p.G + ROWS - 1) / ROWS;
    it.h = static_cast<int>(idx / chunks);
    it.chunk = static_cast<int>(idx - static_cast<long long>(it.h) * chunks);
    return static_cast<int>(rel - idx * it.tiles);
  };

  // ---- producer side: the warp's tiles of the span, in order; lane 0 issues the copies ------------------
  Cursor pc{s_first, s_b, seq_len(p, s_b), 0};
  pc.n = seq_tiles<ROWS>(p, pc.s);
  long long ppos = span0;    // start of the row chunk (or its part) being loaded
  int p_end = 0;             // tiles [.., p_end) of it are in the span
  int p_next = 0;            // next tile of this warp
  int p_blk_base = 0;        // tile that lane 0's table entry belongs to
  int p_blk = -1;            // lane i: block of tile p_blk_base + kWarps * i
  Item pit{};
  bool p_more = true;
  uint32_t bad_stage = 0;    // stages whose tile was not loaded
  auto table_window = [&]() {
    p_blk_base = p_next;
    const int t = p_next + C::kWarps * lane;
    p_blk = -1;
    if (t < p_end && t * 16 < pit.nk) {
      const int e = __ldg(p.table + static_cast<long long>(pit.b) * p.width + (t * 16) / p.page);
      if (e >= 0 && e < p.num_blocks) p_blk = e;
      else atomicOr(p.status, kDevStatusBadSeqlens);
    }
  };
  auto open_chunk = [&]() {  // moves to the row chunk at ppos; p_more: there is one
    p_more = ppos < span1;
    if (!p_more) return;
    settle(pc, ppos);
    const int t0 = item_at(pc, ppos, pit);
    const long long left = span1 - ppos;
    p_end = left < pit.tiles - t0 ? t0 + static_cast<int>(left) : pit.tiles;
    ppos += p_end - t0;
    p_next = t0 + warp;
    table_window();
  };
  int p_stage = 0;
  int in_flight = 0;
  auto produce = [&]() {  // fills the next stage, if the warp has a tile left
    while (p_more && p_next >= p_end) open_chunk();
    if (!p_more) return;
    if (p_next - p_blk_base >= 32 * C::kWarps) table_window();
    const int blk = __shfl_sync(0xffffffffu, p_blk, (p_next - p_blk_base) / C::kWarps);
    const int off = (p_next * 16) % p.page;
    if (blk >= 0) {
      bad_stage &= ~(1u << p_stage);
      if (lane == 0) {
        bar_arrive_expect_tx(&bar[p_stage], C::kTile);
        bulk_load_g2s(ring + p_stage * C::kTile, p.cache + kv4_tile_offset<D>(blk, off, p.page, p.Hk, pit.h),
                      C::kTile, &bar[p_stage]);
      }
    } else {
      bad_stage |= 1u << p_stage;
      if (lane == 0) bar_arrive(&bar[p_stage]);
    }
    ++in_flight;
    p_next += C::kWarps;
    p_stage = p_stage + 1 == C::kStages ? 0 : p_stage + 1;
  };
  open_chunk();
#pragma unroll 1
  for (int i = 0; i < C::kStages; ++i) produce();

  // ---- consumer side --------------------------------------------------------------------------------------
  Cursor cc{s_first, s_b, seq_len(p, s_b), 0};
  cc.n = seq_tiles<ROWS>(p, cc.s);
  int stage = 0;
  uint32_t phase = 0;
  bool alive = true;  // false once a wait ran out: no more copies, and those in flight are waited for
  bool tail_valid = false, head_valid = false, head_ends = false;
  Item it{};
#pragma unroll 1
  for (long long pos = span0; pos < span1;) {
    settle(cc, pos);
    const int t0 = item_at(cc, pos, it);
    const long long left = span1 - pos;
    const int t1 = left < it.tiles - t0 ? t0 + static_cast<int>(left) : it.tiles;
    pos += t1 - t0;
    const int rows = min(ROWS, it.nq * p.G - it.chunk * ROWS);
    const int row0 = it.chunk * ROWS;

    // Q of the chunk: one warp per row, transformed in float32, scaled by a power of two
    for (int r = warp; r < ROWS; r += C::kWarps) {
      constexpr int E = D / 32;  // consecutive elements of a lane
      float x[E];
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = 0.f;
      if (r < rows) {
        const int i = (row0 + r) / p.G, hq = it.h * p.G + (row0 + r) - i * p.G;
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + (it.q0 + i) * p.q_sn + hq * p.q_sh + E * lane;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(src + e);
          x[e] = __uint_as_float(w << 16);
          x[e + 1] = __uint_as_float(w & 0xFFFF0000u);
        }
      }
      if (p.signs != nullptr) {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (p.signs[E * lane + e] == -1) x[e] = -x[e];
#pragma unroll
        for (int s = 1; s < E; s <<= 1)
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (!(e & s)) {
              const float u = x[e], v = x[e | s];
              x[e] = u + v;
              x[e | s] = u - v;
            }
#pragma unroll
        for (int s = 1; s < 32; s <<= 1)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float o = __shfl_xor_sync(0xffffffffu, x[e], s);
            x[e] = (lane & s) ? o - x[e] : x[e] + o;
          }
      }
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) top = fmaxf(top, fabsf(x[e]));
#pragma unroll
      for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
      // the largest entry at 2^13 .. 2^14; the factor of the scores takes it back, and the 2^-24
      // of the codes
      const int ex = top > 0.f ? min(max(exponent_of(top) - 13, -100), 100) : 0;
      const float f = exp2_int(-ex);
#pragma unroll
      for (int e = 0; e < E; ++e) sq[r * D + E * lane + e] = x[e] * f;
      if (lane == 0) rowf[r] = p.scale_log2 * exp2_int(ex) * 16777216.f;
    }
    __syncthreads();

    // operand of row n = g (one of 8 per NT): b0 pairs (r, r + 4), b1 pairs (r + 1, r + 5) / 16 of
    // 16 c + (0 | 2 | 8 | 10) in each group, and sums of the rounded entries per group
    uint32_t qf[NT][GR][4][2];
    float qs[NT][GR][2];  // rows 2c, 2c + 1
    float cf[NT][2];
    int lim[NT][2];       // keys that rows 2c, 2c + 1 see
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int gr = 0; gr < GR; ++gr) {
        float q16[16], sum = 0.f;
        const float4* src = reinterpret_cast<const float4*>(sq + (8 * nt + g) * D + 64 * gr + 16 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 v = src[i];
          q16[4 * i] = v.x, q16[4 * i + 1] = v.y, q16[4 * i + 2] = v.z, q16[4 * i + 3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float h = __half2float(__float2half_rn((i & 1) ? q16[i] * 0.0625f : q16[i]));
          q16[i] = h;
          sum += (i & 1) ? h * 16.f : h;
        }
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const int o = (ks >> 1) * 8 + (ks & 1) * 2;
          qf[nt][gr][ks][0] = pack_f16x2(q16[o], q16[o + 4]);
          qf[nt][gr][ks][1] = pack_f16x2(q16[o + 1], q16[o + 5]);
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum *= 1.f / 16777216.f;
        qs[nt][gr][0] = __shfl_sync(0xffffffffu, sum, 8 * c);
        qs[nt][gr][1] = __shfl_sync(0xffffffffu, sum, 8 * c + 4);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * nt + 2 * c + e;
        cf[nt][e] = rowf[r];
        lim[nt][e] = p.causal && r < rows ? min(it.nk, max(0, it.nk - it.nq + (row0 + r) / p.G + 1)) : it.nk;
      }
    }
    const int min_lim = p.causal ? min(it.nk, max(0, it.nk - it.nq + row0 / p.G + 1)) : it.nk;

    float m[NT][2], l[NT][2], zacc[NT][GR][2], o[NT][D / 16][4];
    float ef = exp2_int(100);  // 2^-E, E the reference exponent of V's steps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = kNegBig;
        l[nt][e] = 0.f;
#pragma unroll
        for (int gr = 0; gr < GR; ++gr) zacc[nt][gr][e] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
    }

#pragma unroll 1
    for (int t = t0 + warp; t < t1; t += C::kWarps) {
      if (alive) {
        if (!warp_all(wait_bar(&bar[stage], phase, ab))) {
          alive = p_more = false;
          drain(&bar[stage], phase);
        }
      } else if (in_flight > 0) {
        drain(&bar[stage], phase);
      }
      in_flight = max(in_flight - 1, 0);
      const uint8_t* tile = ring + stage * C::kTile;
      const int key0 = t * 16;
      const bool missing = (bad_stage >> stage) & 1u;
      const bool whole = !missing && key0 + 16 <= min_lim;
      const int ka = key0 + key_at(g), kb = ka + 8;  // this lane's keys of the scores

      // scores: y = sum_g s (q . u) + z (sum q)
      float y[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[nt][e] = 0.f;
#pragma unroll
      for (int pl = 0; pl < F::kPlanes; ++pl) {
        const uint8_t* ra = tile + pl * F::kPlaneBytes + key_at(g) * F::kRowBytes + c * 8 * F::kGroups;
        uint32_t wa[2 * F::kGroups], wb[2 * F::kGroups];
        if constexpr (F::kGroups == 2) {
          const uint4 u = *reinterpret_cast<const uint4*>(ra);
          const uint4 v = *reinterpret_cast<const uint4*>(ra + 8 * F::kRowBytes);
          wa[0] = u.x, wa[1] = u.y, wa[2] = u.z, wa[3] = u.w;
          wb[0] = v.x, wb[1] = v.y, wb[2] = v.z, wb[3] = v.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(ra);
          const uint2 v = *reinterpret_cast<const uint2*>(ra + 8 * F::kRowBytes);
          wa[0] = u.x, wa[1] = u.y;
          wb[0] = v.x, wb[1] = v.y;
        }
#pragma unroll
        for (int gp = 0; gp < F::kGroups; ++gp) {
          const int gr = pl * F::kGroups + gp;
          float acc[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint32_t a = wa[2 * gp + (ks >> 1)] >> (8 * (ks & 1));
            const uint32_t b = wb[2 * gp + (ks >> 1)] >> (8 * (ks & 1));
            const uint32_t fr[4] = {a & 0x000F000Fu, b & 0x000F000Fu, a & 0x00F000F0u, b & 0x00F000F0u};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(acc[nt], fr, qf[nt][gr][ks][0], qf[nt][gr][ks][1]);
          }
          const uint32_t za = *reinterpret_cast<const uint32_t*>(tile + F::kKszOff + key_at(g) * F::kSzRow + 4 * gr);
          const uint32_t zb = *reinterpret_cast<const uint32_t*>(tile + F::kKszOff + (key_at(g) + 8) * F::kSzRow + 4 * gr);
          const float s0 = __uint_as_float(za << 16), z0 = __uint_as_float(za & 0xFFFF0000u);
          const float s1 = __uint_as_float(zb << 16), z1 = __uint_as_float(zb & 0xFFFF0000u);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              y[nt][e] = fmaf(z0, qs[nt][gr][e], fmaf(s0, acc[nt][e], y[nt][e]));
              y[nt][2 + e] = fmaf(z1, qs[nt][gr][e], fmaf(s1, acc[nt][2 + e], y[nt][2 + e]));
            }
        }
      }
      bool over = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = y[nt][e] * cf[nt][e & 1];
          if (!whole && (missing || (e < 2 ? ka : kb) >= lim[nt][e & 1])) x = -INFINITY;
          y[nt][e] = x;
          over = over || x > m[nt][e & 1] + kTau;
        }
      // V's steps and minima of the lane's keys
      float vs[GR][2], vz[GR][2];
      float smax = 0.f;
#pragma unroll
      for (int gr = 0; gr < GR; ++gr)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(tile + F::kVszOff + (key_at(g) + 8 * e) * F::kSzRow + 4 * gr);
          vs[gr][e] = __uint_as_float(w << 16);
          vz[gr][e] = __uint_as_float(w & 0xFFFF0000u);
          if (!whole && (missing || (e ? kb : ka) >= it.nk)) vs[gr][e] = vz[gr][e] = 0.f;
          smax = fmaxf(smax, vs[gr][e]);
        }
      over = over || smax * ef > 32.f;
      if (__any_sync(0xffffffffu, over)) {  // rare: move the references, and what was summed under them
#pragma unroll
        for (int sft = 4; sft < 32; sft <<= 1) smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, sft));
        float fe = 1.f;
        if (smax * ef > 32.f) {
          const float nf = exp2_int(-min(exponent_of(smax), 120));
          fe = nf / ef;
          ef = nf;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(y[nt][e], y[nt][2 + e]);
#pragma unroll
            for (int sft = 4; sft < 32; sft <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sft));
            const float nm = fmaxf(m[nt][e], top);
            const float al = ex2_approx(m[nt][e] - nm);
            m[nt][e] = nm;
            l[nt][e] *= al;
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) zacc[nt][gr][e] *= al;
            const float oe = al * fe;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              o[nt][i][e] *= oe;
              o[nt][i][2 + e] *= oe;
            }
          }
      }
      // p, its sum, the minima's part, and p s as the operand of the second product
      uint32_t pf[NT][GR][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float pr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) pr[e] = ex2_approx(y[nt][e] - m[nt][e & 1]);
        l[nt][0] += pr[0] + pr[2];
        l[nt][1] += pr[1] + pr[3];
#pragma unroll
        for (int gr = 0; gr < GR; ++gr) {
          float t4[4], z4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            t4[e] = pr[e] * (vs[gr][e >> 1] * ef);
            z4[e] = pr[e] * vz[gr][e >> 1];
          }
          if (!whole) {  // a masked key adds nothing, whatever its scales are (NaN among them)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (missing || (e < 2 ? ka : kb) >= lim[nt][e & 1]) t4[e] = z4[e] = 0.f;
          }
          zacc[nt][gr][0] += z4[0] + z4[2];
          zacc[nt][gr][1] += z4[1] + z4[3];
          pf[nt][gr][0] = transpose8x8(pack_f16x2(t4[0], t4[1]));
          pf[nt][gr][1] = transpose8x8(pack_f16x2(t4[2], t4[3]));
        }
      }
      // O^T += u^T (p s): dimensions 8 g + 2 q (and + 1, times 16) of each group on the 16 side
#pragma unroll
      for (int pl = 0; pl < F::kPlanes; ++pl) {
        const uint8_t* rv = tile + F::kVOff + pl * F::kPlaneBytes + g * 4 * F::kGroups;
        uint32_t w[4][F::kGroups];  // tokens at indices 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint8_t* r = rv + (key_at(2 * c + (i & 1)) + 8 * (i >> 1)) * F::kRowBytes;
          if constexpr (F::kGroups == 2) {
            const uint2 u = *reinterpret_cast<const uint2*>(r);
            w[i][0] = u.x, w[i][1] = u.y;
          } else {
            w[i][0] = *reinterpret_cast<const uint32_t*>(r);
          }
        }
#pragma unroll
        for (int gp = 0; gp < F::kGroups; ++gp) {
          const int gr = pl * F::kGroups + gp;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t u = __byte_perm(w[0][gp], w[1][gp], hf ? 0x7632 : 0x5410);
            const uint32_t v = __byte_perm(w[2][gp], w[3][gp], hf ? 0x7632 : 0x5410);
#pragma unroll
            for (int q2 = 0; q2 < 2; ++q2) {
              const uint32_t a = u >> (8 * q2), b = v >> (8 * q2);
              const uint32_t fr[4] = {a & 0x000F000Fu, a & 0x00F000F0u, b & 0x000F000Fu, b & 0x00F000F0u};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][4 * gr + 2 * hf + q2], fr, pf[nt][gr][0], pf[nt][gr][1]);
            }
          }
        }
      }
      __syncwarp();
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
      produce();
    }

    // ---- join the warps -------------------------------------------------------------------------------
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float s = l[nt][e];
#pragma unroll
        for (int sft = 4; sft < 32; sft <<= 1) s += __shfl_xor_sync(0xffffffffu, s, sft);
        l[nt][e] = s;
#pragma unroll
        for (int gr = 0; gr < GR; ++gr) {
          float z = zacc[nt][gr][e];
#pragma unroll
          for (int sft = 4; sft < 32; sft <<= 1) z += __shfl_xor_sync(0xffffffffu, z, sft);
          zacc[nt][gr][e] = z;
        }
        if (g == 0) {
          sm_m[warp * ROWS + 8 * nt + 2 * c + e] = m[nt][e];
          sm_l[warp * ROWS + 8 * nt + 2 * c + e] = s;
        }
      }
    __syncthreads();
    const float back = 16777216.f / ef;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * nt + 2 * c + e;
        float top = kNegBig;
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) top = fmaxf(top, sm_m[w * ROWS + r]);
        const float f = ex2_approx(m[nt][e] - top);
        float* dst = red + (warp * ROWS + r) * C::kRedRow;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const int dim = 64 * (i >> 2) + 8 * g + 2 * (i & 3);
          dst[dim] = (o[nt][i][e] * back + zacc[nt][i >> 2][e]) * f;
          dst[dim + 1] = (o[nt][i][2 + e] * (back * 0.0625f) + zacc[nt][i >> 2][e]) * f;
        }
      }
    __syncthreads();
    const bool starts = t0 == 0, ends = t1 == it.tiles;
    float* slot = slots + (starts ? slot_floats<D, NT>() : 0);
    for (int i = tid; i < ROWS * (D / 2); i += C::kThreads) {
      const int r = i / (D / 2), x = 2 * (i - r * (D / 2));
      if (r >= rows) break;
      float a0 = 0.f, a1 = 0.f, top = kNegBig, sum = 0.f;
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) {
        a0 += red[(w * ROWS + r) * C::kRedRow + x];
        a1 += red[(w * ROWS + r) * C::kRedRow + x + 1];
        top = fmaxf(top, sm_m[w * ROWS + r]);
      }
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) sum += sm_l[w * ROWS + r] * ex2_approx(sm_m[w * ROWS + r] - top);
      if (starts && ends) {
        const int q = (row0 + r) / p.G, hq = it.h * p.G + (row0 + r) - q * p.G;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + (it.q0 + q) * p.o_sn + hq * p.o_sh + x) =
            pack_bf16x2(a0 * inv, a1 * inv);
        if (x == 0 && p.lse != nullptr)
          p.lse[static_cast<long long>(hq) * p.total_q + it.q0 + q] =
              sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2f;
      } else {
        *reinterpret_cast<float2*>(slot + r * D + x) = make_float2(a0, a1);
        if (x == 0) {
          slot[ROWS * D + r] = top;
          slot[ROWS * D + ROWS + r] = sum;
        }
      }
    }
    if (starts && !ends) tail_valid = true;
    if (!starts) {
      head_valid = true;
      head_ends = ends;
    }
    __syncthreads();
  }
  if (tid == 0)
    *meta = Meta{tail_valid, it.b, it.h, it.chunk, head_valid, head_ends, {0, 0}};
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Joins the parts of the row chunks that several blocks of threads share: block (i, r) does row r of
// the chunk that starts in block i's span and goes on, in the order of the spans.
template <int D, int NT>
__global__ void __launch_bounds__(D / 2) kv4_join_kernel(const Kv4AttnParams p) {
  constexpr int ROWS = 8 * NT;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Meta* metas = reinterpret_cast<const Meta*>(p.ws);
  const Meta mt = metas[blockIdx.x];
  if (!mt.tail_valid) return;
  const float* parts = reinterpret_cast<const float*>(p.ws + static_cast<size_t>(gridDim.x) * sizeof(Meta));
  const SeqLen s = seq_len(p, mt.b);
  const int row = mt.chunk * ROWS + blockIdx.y, r = blockIdx.y;
  if (row >= s.nq * p.G) return;
  int last = blockIdx.x + 1;
  while (last < static_cast<int>(gridDim.x) - 1 && !metas[last].head_ends) ++last;
  auto part = [&](int j) {
    return parts + (static_cast<size_t>(j) * 2 + (j == static_cast<int>(blockIdx.x) ? 1 : 0)) * slot_floats<D, NT>();
  };
  float top = kNegBig;
  for (int j = blockIdx.x; j <= last; ++j) top = fmaxf(top, part(j)[ROWS * D + r]);
  float a0 = 0.f, a1 = 0.f, sum = 0.f;
  for (int j = blockIdx.x; j <= last; ++j) {
    const float* q = part(j);
    const float f = ex2_approx(q[ROWS * D + r] - top);
    const float2 v = *reinterpret_cast<const float2*>(q + r * D + 2 * threadIdx.x);
    a0 += v.x * f;
    a1 += v.y * f;
    sum += q[ROWS * D + ROWS + r] * f;
  }
  const int q = row / p.G, hq = mt.h * p.G + row - q * p.G;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + (s.q0 + q) * p.o_sn + hq * p.o_sh + 2 * threadIdx.x) =
      pack_bf16x2(a0 * inv, a1 * inv);
  if (threadIdx.x == 0 && p.lse != nullptr)
    p.lse[static_cast<long long>(hq) * p.total_q + s.q0 + q] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2f;
}

template <int D, int NT>
unsigned long long ws_bytes(int num_sms) {
  const unsigned long long blocks = static_cast<unsigned long long>(num_sms) * SplitCfg<D, NT>::kBlocksPerSm;
  return blocks * (sizeof(Meta) + 2 * sizeof(float) * slot_floats<D, NT>());
}

template <int D, int NT>
cudaError_t setup() {
  return cudaFuncSetAttribute(kv4_split_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              SplitCfg<D, NT>::kSmem);
}

template <int D, int NT>
cudaError_t launch(const Kv4AttnParams& p, int num_sms, cudaStream_t stream) {
  using C = SplitCfg<D, NT>;
  const int grid = num_sms * C::kBlocksPerSm;
  kv4_split_kernel<D, NT><<<grid, C::kThreads, C::kSmem, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(grid, C::kRows);
  cfg.blockDim = dim3(D / 2);
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, NT>, p);
}

}  // namespace

unsigned long long kv4_attn_workspace_bytes(int d, int num_sms) {
  unsigned long long n = 0;
  auto most = [&](unsigned long long v) { n = v > n ? v : n; };
  if (d == 64) most(ws_bytes<64, 1>(num_sms)), most(ws_bytes<64, 2>(num_sms));
  if (d == 128) most(ws_bytes<128, 1>(num_sms)), most(ws_bytes<128, 2>(num_sms));
  if (d == 256) most(ws_bytes<256, 1>(num_sms));
  return n;
}

cudaError_t setup_kv4_attn_kernels() {
  cudaError_t e = setup<64, 1>();
  if (e == cudaSuccess) e = setup<64, 2>();
  if (e == cudaSuccess) e = setup<128, 1>();
  if (e == cudaSuccess) e = setup<128, 2>();
  if (e == cudaSuccess) e = setup<256, 1>();
  return e;
}

cudaError_t launch_kv4_attn(const Kv4AttnParams& p, int d, int num_sms, cudaStream_t stream, int* launches) {
  *launches = 2;
  // 8 rows on the small side of the products, or two sets of 8 for one pass over the keys where there
  // are more rows (not at d = 256, where O of 16 rows would fill the registers)
  const bool two = static_cast<long long>(p.max_q) * p.G > 8;
  if (d == 64) return two ? launch<64, 2>(p, num_sms, stream) : launch<64, 1>(p, num_sms, stream);
  if (d == 128) return two ? launch<128, 2>(p, num_sms, stream) : launch<128, 1>(p, num_sms, stream);
  return launch<256, 1>(p, num_sms, stream);
}

}  // namespace ea

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
// One warp works on two tiles of 16 keys at a time and keeps its own running maximum, sum and O.  They
// come through its own ring of shared-memory stages, filled by one bulk copy per tile (a tile with all its
// scales is contiguous), each stage watched by one mbarrier: no warp waits for another inside a request's
// keys.  The maximum is lazy: it moves only when a score passes it by 2^8, found by one vote per 32 keys.  p s is
// rounded to float16 (11 bits) under a running power-of-two reference of s, moved the same way, so that
// values of V of any size keep their bits.  The tensor core cuts its sums off (it does not round them), and codes
// are positive, so long sums would drift; every 512 keys the middle of the codes, 7.5 times the sum of p s, moves
// from the sums to the minima's part, which is small then too (0.5% of O over 10240 keys otherwise).
//
// Work is the requests' 32-key units laid end to end, (request, kv head, chunk of rows) after another, each
// chunk with the cost of its prologue and epilogue in front, cut into equal spans, one per warp.  Warps
// meet only twice, to find their spans and after their last unit.  (With a block's eight warps sharing every
// chunk, a chunk of one unit cost the block 6 us in barriers and in latencies that nothing covered.)  A warp
// that holds all of a chunk writes O; others leave (O, m, l) for the units they have.  A block then joins the
// parts of its warps, which follow one another, and leaves at most two parts itself, of a chunk that began
// before it and of one that goes on after it; the join kernel adds those, in order.

#include <type_traits>

#include "kv4_attn.cuh"

namespace ea {

namespace {

// Keys of a unit: two tiles, which share one wait, one vote and one round of copies (a tile at a time
// took 421 instructions per tile, a quarter of them for those)
constexpr int kKeys = 32;
// What a chunk costs besides its units (its Q, its O), in units
constexpr int kChunkCost = 3;
// A warp gets at least this much work: fewer spans than warps for short contexts, so that less is left to join
constexpr int kMinCost = 2;
// Requests of more rows per key/value head than this go to the chunk kernel (d = 64, 128)
constexpr int kChunkMinRows = 32;
// Units after which the sums of codes are centred
constexpr int kCentre = 16;

template <int D, int NT>
struct SplitCfg {
  static constexpr int kWarps = 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kRows = 8 * NT;
  static constexpr int kBlocksPerSm = D * NT <= 128 ? 2 : 1;
  static constexpr int kTile = Kv4Tile<D>::kBytes;
  // ring of a warp: 9 KB, 2 units of d = 128, where 16 warps share an SM (74 to 150 KB in flight; 45 KB cover
  // the latency), twice that where 8 do
  static constexpr int kStages = (D == 64 ? 4 : D == 128 ? 2 : 1) * (kBlocksPerSm == 1 ? 2 : 1);
  static constexpr int kStageBytes = 2 * kTile;
  static constexpr int kLoBytes = NT * (D / 64) * 1024;  // low parts of Q: [NT][D / 64][2][32] uint4
  static constexpr int kWarpBytes = kStages * kStageBytes + kLoBytes;
  static constexpr int kSmem = kWarps * kWarpBytes;
  static_assert((kSmem + 3072) * kBlocksPerSm <= 228 * 1024, "shared memory of an SM");
};

// Where a walk over a span's segments stands.
struct Walk {
  long long pos;    // next position of the span
  long long end;
  long long first;  // position of request b's first chunk
  long long cost;   // of request b, -1: not looked up yet
  int b;
};

// Units of one row chunk of a request (one, with every key masked, where it has no key).
__device__ __forceinline__ int chunk_units(int nk) { return nk > 0 ? (nk + kKeys - 1) / kKeys : 1; }

template <int ROWS>
__device__ __forceinline__ long long seq_cost(const Kv4AttnParams& p, const SeqLen& s) {
  const long long chunks = (static_cast<long long>(s.nq) * p.G + ROWS - 1) / ROWS;
  return chunks * p.Hk * (chunk_units(s.nk) + kChunkCost);
}

// The next segment of a walk (one lane): false when the span has ended.  A boundary inside the cost in front
// of a chunk counts as the chunk's start.
template <int ROWS>
__device__ __forceinline__ bool next_segment(const Kv4AttnParams& p, volatile Walk& w, volatile Segment& seg) {
  long long pos = w.pos, first = w.first, cost = w.cost;
  const long long end = w.end;
  int b = w.b;
  SeqLen s = seq_len(p, b);
  if (cost < 0) cost = seq_cost<ROWS>(p, s);
  while (pos < end) {
    while (pos >= first + cost) {
      first += cost;
      s = seq_len(p, ++b);
      cost = seq_cost<ROWS>(p, s);
    }
    const int units = chunk_units(s.nk), each = units + kChunkCost;
    const int chunks = static_cast<int>((static_cast<long long>(s.nq) * p.G + ROWS - 1) / ROWS);
    const long long rel = pos - first, idx = rel / each, start = first + idx * each;
    const long long stop = min(end, start + each);
    const int t0 = max(0, static_cast<int>(pos - start) - kChunkCost);
    const int t1 = max(0, static_cast<int>(stop - start) - kChunkCost);
    pos = stop;
    if (t1 > t0) {
      const int h = static_cast<int>(idx / chunks);
      seg.b = b, seg.h = h, seg.chunk = static_cast<int>(idx - static_cast<long long>(h) * chunks);
      seg.nq = s.nq, seg.nk = s.nk, seg.q0 = s.q0;
      seg.units = units, seg.t0 = t0, seg.t1 = t1;
      w.pos = pos, w.first = first, w.cost = cost, w.b = b;
      return true;
    }
  }
  w.pos = pos, w.first = first, w.cost = cost, w.b = b;
  return false;
}

// d = a b + c, the warp's m16n8k16
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                         const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// The codes of the low (high) byte of each half of w as float16 subnormals, code times 2^-24: n, the even
// one, and b, even + 16 odd.
__device__ __forceinline__ void low_codes(uint32_t w, uint32_t& n, uint32_t& b) {
  n = w & 0x000F000Fu;
  b = w & 0x00FF00FFu;
}
__device__ __forceinline__ void high_codes(uint32_t w, uint32_t& n, uint32_t& b) {
  b = __byte_perm(w, 0, 0x4341);
  n = b & 0x000F000Fu;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
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
  constexpr int kQueue = C::kStages + 2;  // segments from the one being loaded back to the one being summed
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[C::kWarps][C::kStages];
  __shared__ long long scan[C::kWarps];
  __shared__ int abort_flag;
  __shared__ Walk walks[C::kWarps];
  __shared__ Segment queues[C::kWarps][kQueue];
  __shared__ Meta metas[C::kWarps];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  uint8_t* ring = smem + warp * C::kWarpBytes;
  uint4* slo = reinterpret_cast<uint4*>(ring + C::kStages * C::kStageBytes);
  uint64_t* bar = bars[warp];

  if (tid < C::kWarps * C::kStages) bar_init(&bars[0][tid], 1);
  if (tid == 0) abort_flag = 0;
  fence_barrier_init();

  // ---- the warps' spans: sums over the requests, a run of them per thread -----------------------------
  const int per = (p.B + C::kThreads - 1) / C::kThreads;
  const int my0 = min(p.B, tid * per), my1 = min(p.B, my0 + per);
  long long mine = 0;
  bool bad = false;
  for (int b = my0; b < my1; ++b) {
    const SeqLen s = seq_len(p, b);
    bad |= s.bad;
    mine += seq_cost<ROWS>(p, s);
  }
  if (bad && blockIdx.x == 0) atomicOr(p.status, kDevStatusBadSeqlens);
  long long before = mine;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, before, s);
    if (lane >= s) before += o;
  }
  if (lane == 31) scan[warp] = before;
  before -= mine;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < C::kWarps; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  // blocks of threads in use, all their warps alike
  const long long blocks = min(static_cast<long long>(gridDim.x), (total + C::kWarps * kMinCost - 1) / (C::kWarps * kMinCost));
  Meta* meta = reinterpret_cast<Meta*>(p.ws) + blockIdx.x;
  if (blockIdx.x >= blocks) {
    if (tid == 0) *meta = Meta{};
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    return;
  }
  const long long spans = blocks * C::kWarps;
  for (int w = 0; w < C::kWarps; ++w) {
    const long long i = static_cast<long long>(blockIdx.x) * C::kWarps + w;
    const long long start = total * i / spans;
    if (before <= start && start < before + mine) {  // one thread: the span starts in its run
      int b = my0;
      long long at = before;
      for (;; ++b) {
        const long long n = seq_cost<ROWS>(p, seq_len(p, b));
        if (start < at + n) break;
        at += n;
      }
      walks[w] = Walk{start, total * (i + 1) / spans, at, -1, b};
    }
  }
  __syncthreads();

  const AbortState ab{&abort_flag, p.status};
  float* block_parts = reinterpret_cast<float*>(p.ws + static_cast<size_t>(gridDim.x) * sizeof(Meta));
  float* warp_parts = block_parts + static_cast<size_t>(gridDim.x) * 2 * part_floats<D, ROWS>() +
                      (static_cast<size_t>(blockIdx.x) * C::kWarps + warp) * 2 * part_floats<D, ROWS>();
  block_parts += static_cast<size_t>(blockIdx.x) * 2 * part_floats<D, ROWS>();

  // ---- producer side: the units of the span, in order; segments go into the warp's queue --------------
  int p_seg = -1;            // segments opened, less one
  int p_end = 0;             // units [.., p_end) of it are in the span
  int p_next = 0;            // next unit
  int p_base = 0;            // lane i keeps the address of tile i & 1 of unit p_base + i / 2 of the chunk, or
  const uint8_t* p_addr = nullptr;  // nullptr: past the keys, or no block of the cache
  bool p_more = true;
  uint32_t absent = 0;       // 2 bits per stage: its tiles that were not loaded
  int in_flight = 0;
  auto produce = [&](int at) {  // fills stage `at`, if there is a unit left
    if (p_more && p_next >= p_end) {
      volatile Segment& seg = queues[warp][(p_seg + 1) % kQueue];
      int more = 0;
      if (lane == 0) more = next_segment<ROWS>(p, walks[warp], seg);
      p_more = __shfl_sync(0xffffffffu, more, 0) != 0;
      __syncwarp();
      if (p_more) {
        ++p_seg;
        p_next = seg.t0;
        p_end = seg.t1;
        p_base = p_next - 16;  // no window yet
      }
    }
    if (!p_more) return;
    if (p_next - p_base >= 16) {
      volatile Segment& seg = queues[warp][p_seg % kQueue];
      p_base = p_next;
      const int u = p_next + (lane >> 1);
      const int key = u * kKeys + 16 * (lane & 1);
      p_addr = nullptr;
      if (u < p_end && key < seg.nk) {
        const int j = key / p.page;
        const int e = __ldg(p.table + static_cast<long long>(seg.b) * p.width + j);
        if (e >= 0 && e < p.num_blocks)
          p_addr = p.cache + kv4_tile_offset<D>(e, key - j * p.page, p.page, p.Hk, seg.h);
        else
          atomicOr(p.status, kDevStatusBadSeqlens);
      }
      __syncwarp();
    }
    const uint8_t* src = reinterpret_cast<const uint8_t*>(__shfl_sync(
        0xffffffffu, reinterpret_cast<unsigned long long>(p_addr), 2 * (p_next - p_base) + (lane & 1)));
    const uint32_t have = __ballot_sync(0xffffffffu, src != nullptr) & 3u;
    absent = (absent & ~(3u << (2 * at))) | ((have ^ 3u) << (2 * at));
    if (lane == 0) bar_arrive_expect_tx(&bar[at], __popc(have) * C::kTile);
    __syncwarp();
    if (lane < 2 && src != nullptr)
      bulk_load_g2s(ring + at * C::kStageBytes + lane * C::kTile, src, C::kTile, &bar[at]);
    ++in_flight;
    ++p_next;
  };
#pragma unroll 1
  for (int i = 0; i < C::kStages; ++i) produce(i);

  // ---- consumer side --------------------------------------------------------------------------------------
  int stage = 0;
  uint32_t phase = 0;
  bool alive = true;  // false once a wait ran out: no more copies, and those in flight are waited for
  if (lane == 0) metas[warp] = Meta{};
#pragma unroll 1
  for (int seg_no = 0; seg_no <= p_seg; ++seg_no) {
    volatile Segment& it = queues[warp][seg_no % kQueue];
    const int t0 = it.t0, t1 = it.t1;
    const int row0 = it.chunk * ROWS;
    const int rows = min(ROWS, it.nq * p.G - row0);

    // Q, as the operand of row n = g (one of 8 per NT): this lane has entries 16 c .. 16 c + 15 of every group.
    // Transformed in float32 (strides 16 and 32 lie between lanes), scaled by a power of two that puts the row's
    // largest entry at 2^13 .. 2^14 (cf takes it back, and the 2^-24 of the codes).
    // A byte of codes is b = even + 16 odd, so with cb = q_odd / 16 and cn = q_even - cb the products
    // cn even + cb b are q_even even + q_odd odd.  Both are kept as two float16, the rounded value and what its
    // rounding left (22 bits: bf16 rows are exact, transformed rows as near as float32 sums).  qs: sums of a
    // group's entries, times 2^-24.
    uint32_t qf[NT][GR][4][2];
    float qs[NT][GR][2];  // rows 2c, 2c + 1
    float cf[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[GR][16];
#pragma unroll
      for (int gr = 0; gr < GR; ++gr)
#pragma unroll
        for (int i = 0; i < 16; ++i) x[gr][i] = 0.f;
      if (8 * nt + g < rows) {
        const int r = row0 + 8 * nt + g, i = r / p.G, hq = it.h * p.G + r - i * p.G;
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + (it.q0 + i) * p.q_sn + hq * p.q_sh + 16 * c;
#pragma unroll
        for (int gr = 0; gr < GR; ++gr) {
          const uint4 u = *reinterpret_cast<const uint4*>(src + 64 * gr), v = *reinterpret_cast<const uint4*>(src + 64 * gr + 8);
          const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[gr][2 * j] = __uint_as_float(w[j] << 16);
            x[gr][2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
          }
        }
      }
      if (p.signs != nullptr) {
#pragma unroll
        for (int gr = 0; gr < GR; ++gr) {
          const int4 sg = *reinterpret_cast<const int4*>(p.signs + 64 * gr + 16 * c);
          const int sw[4] = {sg.x, sg.y, sg.z, sg.w};
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (static_cast<signed char>(sw[i >> 2] >> (8 * (i & 3))) == -1) x[gr][i] = -x[gr][i];
#pragma unroll
          for (int st = 1; st < 16; st <<= 1)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (!(i & st)) {
                const float a = x[gr][i], b = x[gr][i | st];
                x[gr][i] = a + b;
                x[gr][i | st] = a - b;
              }
#pragma unroll
          for (int st = 1; st < 4; st <<= 1)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float o2 = __shfl_xor_sync(0xffffffffu, x[gr][i], st);
              x[gr][i] = (c & st) ? o2 - x[gr][i] : x[gr][i] + o2;
            }
        }
#pragma unroll
        for (int st = 1; st < GR; st <<= 1)
#pragma unroll
          for (int gr = 0; gr < GR; ++gr)
            if (!(gr & st))
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float a = x[gr][i], b = x[gr | st][i];
                x[gr][i] = a + b;
                x[gr | st][i] = a - b;
              }
      }
      float top = 0.f;
#pragma unroll
      for (int gr = 0; gr < GR; ++gr)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[gr][i]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int ex = top > 0.f ? min(max(exponent_of(top) - 13, -100), 100) : 0;
      const float f = exp2_int(-ex), back = p.scale_log2 * exp2_int(ex) * 16777216.f;
      cf[nt][0] = __shfl_sync(0xffffffffu, back, 8 * c);
      cf[nt][1] = __shfl_sync(0xffffffffu, back, 8 * c + 4);
#pragma unroll
      for (int gr = 0; gr < GR; ++gr) {
        float hn[8], hb[8], ln[8], lb[8], sum = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float cb = x[gr][2 * k + 1] * f * 0.0625f, cn = x[gr][2 * k] * f - cb;
          hb[k] = __half2float(__float2half_rn(cb));
          lb[k] = __half2float(__float2half_rn(cb - hb[k]));
          hn[k] = __half2float(__float2half_rn(cn));
          ln[k] = __half2float(__float2half_rn(cn - hn[k]));
          sum += (hn[k] + ln[k]) + 17.f * (hb[k] + lb[k]);
        }
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const int k = 4 * (ks >> 1) + (ks & 1);
          qf[nt][gr][ks][0] = pack_f16x2(hn[k], hn[k + 2]);
          qf[nt][gr][ks][1] = pack_f16x2(hb[k], hb[k + 2]);
        }
#pragma unroll
        for (int k = 0; k < 8; k += 4)
          slo[((nt * GR + gr) * 2 + k / 4) * 32 + lane] =
              make_uint4(pack_f16x2(ln[k], ln[k + 2]), pack_f16x2(lb[k], lb[k + 2]),
                         pack_f16x2(ln[k + 1], ln[k + 3]), pack_f16x2(lb[k + 1], lb[k + 3]));
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum *= 1.f / 16777216.f;
        qs[nt][gr][0] = __shfl_sync(0xffffffffu, sum, 8 * c);
        qs[nt][gr][1] = __shfl_sync(0xffffffffu, sum, 8 * c + 4);
      }
    }
    __syncwarp();
    const int min_lim = p.causal ? min(it.nk, max(0, it.nk - it.nq + row0 / p.G + 1)) : it.nk;

    float m[NT][2], l[NT][2], zacc[NT][GR][2], o[NT][D / 16][4];
    float ps[NT][GR][2];       // sums of p s 2^-E of the lane's keys since the sums of codes were centred
    int uncentred = 0;
    float ef = exp2_int(100);  // 2^-E, E the reference exponent of V's steps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = kNegBig;
        l[nt][e] = 0.f;
#pragma unroll
        for (int gr = 0; gr < GR; ++gr) zacc[nt][gr][e] = ps[nt][gr][e] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
    }

#pragma unroll 1
    for (int t = t0; t < t1; ++t) {
      if (alive) {
        if (!warp_all(wait_bar(&bar[stage], phase, ab))) {
          alive = p_more = false;
          drain(&bar[stage], phase);
        }
      } else if (in_flight > 0) {
        drain(&bar[stage], phase);
      }
      in_flight = max(in_flight - 1, 0);
      const int key0 = t * kKeys;
      const uint32_t gone = (absent >> (2 * stage)) & 3u;
      auto step = [&](auto whole_unit) {
        constexpr bool whole = decltype(whole_unit)::value;
        // masks: whether this lane's key e (of two) of tile ti is one of the request's, and the number of keys
        // that row 2c + e2 of set nt sees
        const int ka = key0 + key_at(g);
        int nk = 0;
        if constexpr (!whole) nk = it.nk;
        auto held = [&](int ti, int e) { return !((gone >> ti) & 1u) && ka + 16 * ti + 8 * e < nk; };
        int lim[NT][2];
        if constexpr (!whole) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = 8 * nt + 2 * c + e;
              lim[nt][e] = p.causal && r < rows ? min(nk, nk - it.nq + (row0 + r) / p.G + 1) : nk;
            }
        }
        auto sees = [&](int ti, int e, int nt, int e2) {
          return !((gone >> ti) & 1u) && ka + 16 * ti + 8 * e < lim[nt][e2];
        };

        // scores: y = sum_g s (q . u) + z (sum q), in units of log2
        float y[2][NT][4];
        bool over = false;
#pragma unroll
        for (int pl = 0; pl < F::kPlanes; ++pl) {
          uint32_t wa[2][2 * F::kGroups], wb[2][2 * F::kGroups], sza[2][F::kGroups], szb[2][F::kGroups];
#pragma unroll
          for (int ti = 0; ti < 2; ++ti) {
            const uint8_t* tile = ring + stage * C::kStageBytes + ti * C::kTile;
            const uint8_t* ra = tile + pl * F::kPlaneBytes + key_at(g) * F::kRowBytes + c * 8 * F::kGroups;
            const uint8_t* rz = tile + F::kKszOff + key_at(g) * F::kSzRow + 4 * pl * F::kGroups;
            if constexpr (F::kGroups == 2) {
              const uint4 u = *reinterpret_cast<const uint4*>(ra);
              const uint4 v = *reinterpret_cast<const uint4*>(ra + 8 * F::kRowBytes);
              wa[ti][0] = u.x, wa[ti][1] = u.y, wa[ti][2] = u.z, wa[ti][3] = u.w;
              wb[ti][0] = v.x, wb[ti][1] = v.y, wb[ti][2] = v.z, wb[ti][3] = v.w;
              const uint2 x = *reinterpret_cast<const uint2*>(rz);
              const uint2 z = *reinterpret_cast<const uint2*>(rz + 8 * F::kSzRow);
              sza[ti][0] = x.x, sza[ti][1] = x.y, szb[ti][0] = z.x, szb[ti][1] = z.y;
            } else {
              const uint2 u = *reinterpret_cast<const uint2*>(ra);
              const uint2 v = *reinterpret_cast<const uint2*>(ra + 8 * F::kRowBytes);
              wa[ti][0] = u.x, wa[ti][1] = u.y;
              wb[ti][0] = v.x, wb[ti][1] = v.y;
              sza[ti][0] = *reinterpret_cast<const uint32_t*>(rz);
              szb[ti][0] = *reinterpret_cast<const uint32_t*>(rz + 8 * F::kSzRow);
            }
          }
#pragma unroll
          for (int gp = 0; gp < F::kGroups; ++gp) {
            const int gr = pl * F::kGroups + gp;
            float acc[2][NT][4];
#pragma unroll
            for (int kp = 0; kp < 2; ++kp) {
              uint4 lo[NT];
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) lo[nt] = slo[((nt * GR + gr) * 2 + kp) * 32 + lane];
#pragma unroll
              for (int ti = 0; ti < 2; ++ti) {
                uint32_t f0[4], f1[4];
                low_codes(wa[ti][2 * gp + kp], f0[0], f0[2]);
                low_codes(wb[ti][2 * gp + kp], f0[1], f0[3]);
                high_codes(wa[ti][2 * gp + kp], f1[0], f1[2]);
                high_codes(wb[ti][2 * gp + kp], f1[1], f1[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  float(&ac)[4] = acc[ti][nt];
                  constexpr float zero[4] = {0.f, 0.f, 0.f, 0.f};
                  if (kp == 0) mma16816(ac, f0, qf[nt][gr][0][0], qf[nt][gr][0][1], zero);
                  else mma16816(ac, f0, qf[nt][gr][2][0], qf[nt][gr][2][1], ac);
                  mma16816(ac, f0, lo[nt].x, lo[nt].y, ac);
                  mma16816(ac, f1, qf[nt][gr][2 * kp + 1][0], qf[nt][gr][2 * kp + 1][1], ac);
                  mma16816(ac, f1, lo[nt].z, lo[nt].w, ac);
                }
              }
            }
#pragma unroll
            for (int ti = 0; ti < 2; ++ti) {
              const float s0 = __uint_as_float(sza[ti][gp] << 16), z0 = __uint_as_float(sza[ti][gp] & 0xFFFF0000u);
              const float s1 = __uint_as_float(szb[ti][gp] << 16), z1 = __uint_as_float(szb[ti][gp] & 0xFFFF0000u);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const float a0 = s0 * acc[ti][nt][e], a1 = s1 * acc[ti][nt][2 + e];
                  const float b0 = gr == 0 ? a0 : fmaf(s0, acc[ti][nt][e], y[ti][nt][e]);
                  const float b1 = gr == 0 ? a1 : fmaf(s1, acc[ti][nt][2 + e], y[ti][nt][2 + e]);
                  y[ti][nt][e] = fmaf(z0, qs[nt][gr][e], b0);
                  y[ti][nt][2 + e] = fmaf(z1, qs[nt][gr][e], b1);
                }
            }
          }
        }
#pragma unroll
        for (int ti = 0; ti < 2; ++ti)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float x = y[ti][nt][e] * cf[nt][e & 1];
              if constexpr (!whole) x = sees(ti, e >> 1, nt, e & 1) ? x : -INFINITY;
              y[ti][nt][e] = x;
              over = over || x > m[nt][e & 1] + kTau;
            }
        // V's steps and minima of the lane's keys, as they are held
        float smax = 0.f;
        uint32_t vw[2][2][GR];
#pragma unroll
        for (int ti = 0; ti < 2; ++ti) {
          const uint8_t* tile = ring + stage * C::kStageBytes + ti * C::kTile;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint8_t* rz = tile + F::kVszOff + (key_at(g) + 8 * e) * F::kSzRow;
            if constexpr (GR == 1) {
              vw[ti][e][0] = *reinterpret_cast<const uint32_t*>(rz);
            } else {
#pragma unroll
              for (int gr = 0; gr < GR; gr += 2) {
                const uint2 v = *reinterpret_cast<const uint2*>(rz + 4 * gr);
                vw[ti][e][gr] = v.x, vw[ti][e][gr + 1] = v.y;
              }
            }
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) {
              if constexpr (!whole)
                if (!held(ti, e)) vw[ti][e][gr] = 0u;
              smax = fmaxf(smax, __uint_as_float(vw[ti][e][gr] << 16));
            }
          }
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
              float top = fmaxf(fmaxf(y[0][nt][e], y[0][nt][2 + e]), fmaxf(y[1][nt][e], y[1][nt][2 + e]));
#pragma unroll
              for (int sft = 4; sft < 32; sft <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sft));
              const float nm = fmaxf(m[nt][e], top);
              const float al = ex2_approx(m[nt][e] - nm);
              m[nt][e] = nm;
              l[nt][e] *= al;
              const float oe = al * fe;
#pragma unroll
              for (int gr = 0; gr < GR; ++gr) {
                zacc[nt][gr][e] *= al;
                ps[nt][gr][e] *= oe;
              }
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                o[nt][i][e] *= oe;
                o[nt][i][2 + e] *= oe;
              }
            }
        }
#pragma unroll
        for (int ti = 0; ti < 2; ++ti) {
          const uint8_t* tile = ring + stage * C::kStageBytes + ti * C::kTile;
          // p, its sum, the minima's part, and p s as the operand of the second product
          uint32_t pf[NT][GR][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float pr[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) pr[e] = ex2_approx(y[ti][nt][e] - m[nt][e & 1]);
            l[nt][0] += pr[0] + pr[2];
            l[nt][1] += pr[1] + pr[3];
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) {
              float t4[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t w = vw[ti][e >> 1][gr];
                const float z = __uint_as_float(w & 0xFFFF0000u);
                t4[e] = pr[e] * (__uint_as_float(w << 16) * ef);
                if constexpr (whole) {
                  zacc[nt][gr][e & 1] = fmaf(pr[e], z, zacc[nt][gr][e & 1]);
                } else if (sees(ti, e >> 1, nt, e & 1)) {
                  zacc[nt][gr][e & 1] = fmaf(pr[e], z, zacc[nt][gr][e & 1]);
                } else {  // a masked key adds nothing, whatever its scales are (NaN among them)
                  t4[e] = 0.f;
                }
              }
              ps[nt][gr][0] += t4[0] + t4[2];
              ps[nt][gr][1] += t4[1] + t4[3];
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
                uint32_t f0[4], f1[4];  // even codes on the first 8 rows, bytes on the others
                low_codes(u, f0[0], f0[1]);
                low_codes(v, f0[2], f0[3]);
                high_codes(u, f1[0], f1[1]);
                high_codes(v, f1[2], f1[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  float(&o0)[4] = o[nt][4 * gr + 2 * hf], (&o1)[4] = o[nt][4 * gr + 2 * hf + 1];
                  mma16816(o0, f0, pf[nt][gr][0], pf[nt][gr][1], o0);
                  mma16816(o1, f1, pf[nt][gr][0], pf[nt][gr][1], o1);
                }
              }
            }
          }
        }
      };
      // a unit that every row sees whole needs no masks
      if (gone == 0 && key0 + kKeys <= min_lim) step(std::true_type{});
      else step(std::false_type{});
      if (++uncentred == kCentre) {
        uncentred = 0;
        const float per_step = 7.5f / ef;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int gr = 0; gr < GR; ++gr)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float all = ps[nt][gr][e];
              zacc[nt][gr][e] = fmaf(per_step, all, zacc[nt][gr][e]);
              ps[nt][gr][e] = 0.f;
#pragma unroll
              for (int sft = 4; sft < 32; sft <<= 1) all += __shfl_xor_sync(0xffffffffu, all, sft);
              all *= 7.5f / 16777216.f;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                o[nt][4 * gr + k][e] -= all;
                o[nt][4 * gr + k][2 + e] -= 17.f * all;
              }
            }
      }
      __syncwarp();
      produce(stage);
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }

    // ---- O, or this segment's part of it: this lane has dimensions 8 g .. 8 g + 7 of every group of rows 2c, 2c + 1
    const bool starts = it.t0 == 0, ends = it.t1 == it.units;
    const float unscale = 16777216.f / ef;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * nt + 2 * c + e;
        float sum = l[nt][e];
#pragma unroll
        for (int sft = 4; sft < 32; sft <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, sft);
        const bool whole_chunk = starts && ends;
        const float inv = whole_chunk ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
        const int i = (row0 + r) / p.G, hq = it.h * p.G + (row0 + r) - i * p.G;
        float* part = warp_parts + (starts ? part_floats<D, ROWS>() : 0);
#pragma unroll
        for (int gr = 0; gr < GR; ++gr) {
          float z = zacc[nt][gr][e];
#pragma unroll
          for (int sft = 4; sft < 32; sft <<= 1) z += __shfl_xor_sync(0xffffffffu, z, sft);
          float v[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float n = o[nt][4 * gr + k][e], b = o[nt][4 * gr + k][2 + e];
            v[2 * k] = (n * unscale + z) * inv;
            v[2 * k + 1] = ((b - n) * (unscale * 0.0625f) + z) * inv;
          }
          if (r < rows) {
            if (whole_chunk) {
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + (it.q0 + i) * p.o_sn + hq * p.o_sh + 64 * gr + 8 * g) =
                  make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
            } else {
              float4* dst = reinterpret_cast<float4*>(part + r * D + 64 * gr + 8 * g);
              dst[0] = make_float4(v[0], v[1], v[2], v[3]);
              dst[1] = make_float4(v[4], v[5], v[6], v[7]);
            }
          }
        }
        if (g == 0 && r < rows) {
          if (!whole_chunk) {
            part[ROWS * D + r] = m[nt][e];
            part[ROWS * D + ROWS + r] = sum;
          } else if (p.lse != nullptr) {
            p.lse[static_cast<long long>(hq) * p.total_q + it.q0 + i] =
                sum == 0.f ? -INFINITY : (m[nt][e] + log2f(sum)) * kLn2f;
          }
        }
      }
    if (lane == 0) {
      Meta& mt = metas[warp];
      if (starts && !ends) {
        mt.tail_valid = 1;
        mt.b = it.b, mt.h = it.h, mt.chunk = it.chunk;
        mt.rows[0] = rows;
      } else if (!starts) {
        mt.head_valid = 1;
        mt.head_ends = ends;
        mt.rows[1] = rows;
      }
    }
    __syncwarp();
  }
  __syncthreads();

  // ---- join the parts of this block's warps, which follow one another ---------------------------------------
  float* first_part = warp_parts - static_cast<size_t>(warp) * 2 * part_floats<D, ROWS>();
  Meta mine_all{};
  for (int w = -1; w < C::kWarps;) {
    // a chunk from warp w's tail (w = -1: from the warps before this block) over the heads of the next ones
    if (w >= 0 && !metas[w].tail_valid) {
      ++w;
      continue;
    }
    int last = w;
    bool ended = false;
    while (last + 1 < C::kWarps && !ended && metas[last + 1].head_valid) ended = metas[++last].head_ends;
    if (last == w && w < 0) {  // no chunk from before
      ++w;
      continue;
    }
    const Meta& mt = metas[w < 0 ? 0 : w];
    const int rows = w < 0 ? mt.rows[1] : mt.rows[0];
    const bool done = w >= 0 && ended;  // the chunk lies in this block
    auto part = [&](int j) { return first_part + (static_cast<size_t>(j) * 2 + (j == w ? 1 : 0)) * part_floats<D, ROWS>(); };
    const int j0 = max(w, 0);
    for (int i = tid; i < rows * (D / 2); i += C::kThreads) {
      const int r = i / (D / 2), x = 2 * (i - r * (D / 2));
      float top = kNegBig, a0 = 0.f, a1 = 0.f, sum = 0.f;
      for (int j = j0; j <= last; ++j) top = fmaxf(top, part(j)[ROWS * D + r]);
      for (int j = j0; j <= last; ++j) {
        const float* q = part(j);
        const float f = ex2_approx(q[ROWS * D + r] - top);
        const float2 v = *reinterpret_cast<const float2*>(q + r * D + x);
        a0 += v.x * f;
        a1 += v.y * f;
        sum += q[ROWS * D + ROWS + r] * f;
      }
      if (done) {
        write_row_pair<D>(p, seq_len(p, mt.b).q0, mt.h, mt.chunk * ROWS + r, x, a0, a1, top, sum);
      } else {
        float* dst = block_parts + (w >= 0 ? part_floats<D, ROWS>() : 0);
        *reinterpret_cast<float2*>(dst + r * D + x) = make_float2(a0, a1);
        if (x == 0) {
          dst[ROWS * D + r] = top;
          dst[ROWS * D + ROWS + r] = sum;
        }
      }
    }
    if (w < 0) {
      mine_all.head_valid = 1;
      mine_all.head_ends = ended;
    } else if (!ended) {
      mine_all.tail_valid = 1;
      mine_all.b = mt.b;
      mine_all.h = mt.h;
      mine_all.chunk = mt.chunk;
    }
    w = w < 0 ? (ended ? last : C::kWarps) : ended ? last : C::kWarps;
    if (w < C::kWarps && !metas[w].tail_valid) ++w;
  }
  if (tid == 0) *meta = mine_all;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The workspace: the blocks' parts, then two parts per warp, likewise.
template <int D, int NT>
unsigned long long ws_bytes(int num_sms) {
  using C = SplitCfg<D, NT>;
  const unsigned long long blocks = static_cast<unsigned long long>(num_sms) * C::kBlocksPerSm;
  return part_bytes<D, C::kRows>(blocks) + blocks * C::kWarps * 2 * sizeof(float) * part_floats<D, C::kRows>();
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
  return launch_join<D, C::kRows>(p, grid, C::kRows, stream);
}

}  // namespace

// Whether some request may go to the chunk kernel.
bool may_chunk(long long max_q, int G, int d) { return d <= 128 && max_q * G > kChunkMinRows; }

unsigned long long kv4_attn_workspace_bytes(int B, int Hk, int G, long long total_q, int max_q, int d, int num_sms) {
  unsigned long long n = 0;
  auto most = [&](unsigned long long v) { n = v > n ? v : n; };
  if (d == 64) most(ws_bytes<64, 1>(num_sms)), most(ws_bytes<64, 2>(num_sms));
  if (d == 128) most(ws_bytes<128, 1>(num_sms)), most(ws_bytes<128, 2>(num_sms));
  if (d == 256) most(ws_bytes<256, 1>(num_sms));
  if (may_chunk(max_q, G, d)) most(kv4_chunk_workspace_bytes(B, Hk, G, total_q, d, num_sms));
  return n;
}

cudaError_t setup_kv4_attn_kernels() {
  cudaError_t e = setup<64, 1>();
  if (e == cudaSuccess) e = setup<64, 2>();
  if (e == cudaSuccess) e = setup<128, 1>();
  if (e == cudaSuccess) e = setup<128, 2>();
  if (e == cudaSuccess) e = setup<256, 1>();
  if (e == cudaSuccess) e = setup_kv4_chunk_kernels();
  return e;
}

cudaError_t launch_kv4_attn(const Kv4AttnParams& p, int d, int num_sms, cudaStream_t stream, int* launches) {
  Kv4AttnParams few = p;
  *launches = 2;
  if (may_chunk(p.max_q, p.G, d)) {
    // requests of many rows go to the chunk kernel, the others of the batch, if it has any, to this one; both
    // write their parts into the same workspace, one after the other
    Kv4AttnParams many = p;
    many.min_rows = few.max_rows = p.B == 1 ? 0 : kChunkMinRows;  // a request alone: one kernel, whatever its rows
    *launches = 3;
    const cudaError_t e = launch_kv4_chunk(many, d, num_sms, stream);
    if (e != cudaSuccess || p.B == 1) return e;
    *launches = 5;
  }
  // 8 rows on the small side of the products, or two sets of 8 for one pass over the keys where there
  // are more rows (not at d = 256, where O of 16 rows would fill the registers)
  const bool two = static_cast<long long>(p.max_q) * p.G > 8;
  if (d == 64) return two ? launch<64, 2>(few, num_sms, stream) : launch<64, 1>(few, num_sms, stream);
  if (d == 128) return two ? launch<128, 2>(few, num_sms, stream) : launch<128, 1>(few, num_sms, stream);
  return launch<256, 1>(few, num_sms, stream);
}

}  // namespace ea

// Attention of many query rows over the 4-bit paged cache: prompts taken in chunks (d = 64, 128).
//
// The rows of a request that share a key/value head (its queries times Hq / Hk heads) are cut into chunks of
// 256, two tiles of 128 rows; a chunk runs over the keys in blocks of 128 with tcgen05 products into tensor
// memory, S = Q K^T and O += P V, the two tiles taking turns at the tensor core while the other's softmax runs.
// Bound by arithmetic: 4 d flops per row and key for 1.125 d bytes per key, so the codes are brought to float16
// in shared memory once per block and used by both tiles.
//
//   warps 0-3, 4-7   softmax of tile 0, 1: one thread per row.  Loads and transforms Q, and writes O.
//   warps 8-11       codes to float16 K and V tiles (128-byte swizzle), 4 threads per key
//   warp 12          one thread issues every tcgen05.mma
//   warp 13          copies tiles of the cache (one bulk copy each) into a ring of shared memory
//
// Every operand is float16 (11 bits): Q, each row scaled by a power of two; K and V, u s + z in one fused
// multiply-add, scaled by a power of two of the block's largest value (K) or the largest so far (V, O moves with
// it as with the running maximum); P, at most 2^8.  A score is off by two roundings of 2^-11 per product (LSE
// by 5e-6 of itself at unit inputs); with bf16 operands it would be eight times that.
//
// A word of codes gives its nibbles in pairs (0, 4), (1, 5), (2, 6), (3, 7), so the 8 dimensions of a 16-byte chunk
// lie in that order, in K and Q alike, and the columns of O are put back on the way out.
//
// Work is (request, chunk, kv head) after another in blocks of keys (those that some row of the chunk sees), cut
// into equal spans, one per SM; parts are joined as for few rows (kv4_attn.cuh).

#include "kv4_attn.cuh"

namespace ea {

namespace {

constexpr int kRowsPerChunk = 256;
constexpr int kBlockKeys = 128;
// What a chunk costs besides its blocks (its Q, its O, no overlap at its ends), in blocks
constexpr int kChunkCost = 3;
// A span has at least this much work
constexpr int kMinCost = 2;

template <int D>
struct ChunkCfg {
  static constexpr int kThreads = 512;
  static constexpr int kBoxes = D / 64;                 // 64-dimension halves, rows of 128 bytes
  static constexpr int kBoxBytes = 128 * 128;
  static constexpr int kTileBytes = kBoxes * kBoxBytes;  // 128 rows x D float16
  static constexpr int kRawSlots = 6;                   // pairs of the cache's tiles
  static constexpr int kRawBytes = 2 * Kv4Tile<D>::kBytes;
  static constexpr int kQOff = 0;
  static constexpr int kKvOff = 2 * kTileBytes;         // K, V of block 0 mod 2, then of 1 mod 2
  static constexpr int kRawOff = kKvOff + 4 * kTileBytes;
  static constexpr int kSmem = kRawOff + kRawSlots * kRawBytes + 1024;  // room to align to 1024 bytes
  static constexpr int kOCol = 256;
  static constexpr int kTmemCols = 512;
  static_assert(kSmem + 2048 <= 227 * 1024, "shared memory");
  static constexpr uint32_t kRegSoftmax = 168, kRegCodes = 96, kRegOther = 80;
  static_assert((2 * kRegSoftmax + kRegCodes + kRegOther) * 128 == 65536, "register split");
};

// What the softmax needs to know of a block of keys
struct BlockInfo {
  float k_back;  // K was scaled by its inverse
  int v_exp;     // V was scaled by 2^-v_exp
  uint32_t gone;  // bit i: tile i of the block is not there (a table entry out of range)
};

struct ChunkWalk {
  long long pos, end;  // of the span
  long long first;     // position of the current chunk's first head
  int b, chunk, chunks;
  int more;
  Segment seg;
};

__device__ __forceinline__ int chunk_blocks(const Kv4AttnParams& p, const SeqLen& s, int chunk) {
  const int last = min(s.nq * p.G, (chunk + 1) * kRowsPerChunk) - 1;
  const int lim = p.causal ? min(s.nk, s.nk - s.nq + last / p.G + 1) : s.nk;
  return max(1, (lim + kBlockKeys - 1) / kBlockKeys);
}
__device__ __forceinline__ int chunk_count(const Kv4AttnParams& p, const SeqLen& s) {
  return static_cast<int>((static_cast<long long>(s.nq) * p.G + kRowsPerChunk - 1) / kRowsPerChunk);
}
__device__ __forceinline__ long long request_cost(const Kv4AttnParams& p, const SeqLen& s) {
  const int n = chunk_count(p, s);
  long long sum = 0;
  for (int i = 0; i < n; ++i) sum += chunk_blocks(p, s, i) + kChunkCost;
  return sum * p.Hk;
}

// The next segment of a walk (one lane): false when the span has ended.  A boundary inside the cost in front
// of a chunk counts as the chunk's start.
__device__ __forceinline__ bool next_segment(const Kv4AttnParams& p, volatile ChunkWalk& w) {
  long long pos = w.pos, first = w.first;
  const long long end = w.end;
  int b = w.b, chunk = w.chunk, chunks = w.chunks;
  SeqLen s = seq_len(p, b);
  if (chunks < 0) chunks = chunk_count(p, s);
  bool found = false;
  while (pos < end && !found) {
    while (chunk >= chunks) {
      s = seq_len(p, ++b);
      chunk = 0;
      chunks = chunk_count(p, s);
    }
    const int blocks = chunk_blocks(p, s, chunk), each = blocks + kChunkCost;
    const long long rel = pos - first;
    if (rel >= static_cast<long long>(each) * p.Hk) {
      first += static_cast<long long>(each) * p.Hk;
      ++chunk;
      continue;
    }
    const int h = static_cast<int>(rel / each);
    const long long start = first + static_cast<long long>(h) * each, stop = min(end, start + each);
    const int t0 = max(0, static_cast<int>(pos - start) - kChunkCost);
    const int t1 = max(0, static_cast<int>(stop - start) - kChunkCost);
    pos = stop;
    if (t1 > t0) {
      w.seg.b = b, w.seg.h = h, w.seg.chunk = chunk;
      w.seg.nq = s.nq, w.seg.nk = s.nk, w.seg.q0 = s.q0;
      w.seg.units = blocks, w.seg.t0 = t0, w.seg.t1 = t1;
      found = true;
    }
  }
  w.pos = pos, w.first = first, w.b = b, w.chunk = chunk, w.chunks = chunks;
  return found;
}

// One warp's look at the next segment.
__device__ __forceinline__ bool take_segment(const Kv4AttnParams& p, volatile ChunkWalk& w, int lane, Segment& seg) {
  __syncwarp();
  if (lane == 0) w.more = next_segment(p, w) ? 1 : 0;
  __syncwarp();
  if (!w.more) return false;
  seg.b = w.seg.b, seg.h = w.seg.h, seg.chunk = w.seg.chunk;
  seg.nq = w.seg.nq, seg.nk = w.seg.nk, seg.q0 = w.seg.q0;
  seg.units = w.seg.units, seg.t0 = w.seg.t0, seg.t1 = w.seg.t1;
  return true;
}

__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// The 8 codes of a word as float16 u s + z, in pairs (0, 4), (1, 5), (2, 6), (3, 7).  A nibble under the exponent of
// 1024 is 1024 + u (or 1024 + 16 u): one exact addition (or multiply-add by 1/16) gives u.
__device__ __forceinline__ uint4 expand(uint32_t w, uint32_t s2, uint32_t z2) {
  constexpr uint32_t kMagic = 0x64006400u, kMinus1024 = 0xE400E400u, kSixteenth = 0x2C002C00u, kMinus64 = 0xD400D400u;
  const uint32_t h = w >> 8;
  uint32_t a = (w & 0x000F000Fu) | kMagic, b = (w & 0x00F000F0u) | kMagic;
  uint32_t c = (h & 0x000F000Fu) | kMagic, d = (h & 0x00F000F0u) | kMagic;
  a = hadd2(a, kMinus1024);
  b = hfma2(b, kSixteenth, kMinus64);
  c = hadd2(c, kMinus1024);
  d = hfma2(d, kSixteenth, kMinus64);
  return make_uint4(hfma2(a, s2, z2), hfma2(b, s2, z2), hfma2(c, s2, z2), hfma2(d, s2, z2));
}

// (x0, x1) <- (s0 * c + nm, s1 * c + nm) and (a0, a1) += (b0, b1), packed
__device__ __forceinline__ void fma2_bcast(float& x0, float& x1, float s0, float s1, float c, float nm) {
  asm("{\n\t.reg .b64 ra, rc, rm, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rc, {%4, %4};\n\tmov.b64 rm, {%5, %5};\n\t"
      "fma.rn.f32x2 rd, ra, rc, rm;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(x0), "=f"(x1) : "f"(s0), "f"(s1), "f"(c), "f"(nm));
}
__device__ __forceinline__ void add2(float& a0, float& a1, float b0, float b1) {
  asm("{\n\t.reg .b64 ra, rb;\n\tmov.b64 ra, {%0, %1};\n\tmov.b64 rb, {%2, %3};\n\t"
      "add.rn.f32x2 ra, ra, rb;\n\tmov.b64 {%0, %1}, ra;\n\t}"
      : "+f"(a0), "+f"(a1) : "f"(b0), "f"(b1));
}

// A row of S (128 columns of this thread's lane)
__device__ __forceinline__ void load_row(uint32_t taddr, uint32_t (&r)[128]) {
  tmem_ld_32cols(taddr, *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
  tmem_ld_32cols(taddr + 32, *reinterpret_cast<uint32_t(*)[32]>(&r[32]));
  tmem_ld_32cols(taddr + 64, *reinterpret_cast<uint32_t(*)[32]>(&r[64]));
  tmem_ld_32cols(taddr + 96, *reinterpret_cast<uint32_t(*)[32]>(&r[96]));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 128; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                 "+r"(r[i + 6]), "+r"(r[i + 7]));
}

// p = 2^(s c + nm) of a row: packed float16 in pk, their sum returned.  A quarter of the exponentials of a block
// that every row sees whole run on the FMA pipe, as in the bf16 forward.
template <bool kMasked>
__device__ __forceinline__ float softmax_row(uint32_t (&r)[128], uint32_t (&pk)[64], float c, float nm) {
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    float x0, x1, p0, p1;
    fma2_bcast(x0, x1, __uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]), c, nm);
    if (!kMasked && (i & 3) == 3) {
      exp2_fma_pair(p0, p1, x0, x1);
    } else {
      p0 = ex2_approx(x0);
      p1 = ex2_approx(x1);
    }
    add2(acc[2 * (i & 3)], acc[2 * (i & 3) + 1], p0, p1);
    pk[i] = pack_f16x2(p0, p1);
  }
  add2(acc[0], acc[1], acc[2], acc[3]);
  add2(acc[4], acc[5], acc[6], acc[7]);
  add2(acc[0], acc[1], acc[4], acc[5]);
  return acc[0] + acc[1];
}

// A barrier of the four warps 8-11: whether all of them say yes.
__device__ __forceinline__ bool codes_all(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r) : "r"(v ? 1u : 0u) : "memory");
  return r != 0;
}

template <int D>
__global__ void __launch_bounds__(ChunkCfg<D>::kThreads, 1) kv4_chunk_kernel(const Kv4AttnParams p) {
  using C = ChunkCfg<D>;
  using F = Kv4Tile<D>;
  constexpr int ROWS = kRowsPerChunk;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t raw_full[C::kRawSlots], raw_empty[C::kRawSlots];
  __shared__ uint64_t kv_full[2], kv_empty[2], q_full[2], s_full[2], p_full[2], o_done[2], drained;
  __shared__ uint32_t raw_gone[C::kRawSlots];
  __shared__ BlockInfo info[2];
  __shared__ float wmax[2][2][4];
  __shared__ long long scan[C::kThreads / 32];
  __shared__ ChunkWalk walks[14];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < C::kRawSlots; ++i) {
      bar_init(&raw_full[i], 1);
      bar_init(&raw_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&kv_full[i], 4);
      bar_init(&kv_empty[i], 1);
      bar_init(&q_full[i], 4);
      bar_init(&s_full[i], 1);
      bar_init(&p_full[i], 4);
      bar_init(&o_done[i], 1);
    }
    bar_init(&drained, 1);
    abort_flag = 0;
    fence_barrier_init();
  }

  // ---- this block's span ------------------------------------------------------------------------------------
  const int per = (p.B + C::kThreads - 1) / C::kThreads;
  const int my0 = min(p.B, tid * per), my1 = min(p.B, my0 + per);
  long long mine = 0;
  bool bad = false;
  for (int b = my0; b < my1; ++b) {
    const SeqLen s = seq_len(p, b);
    bad |= s.bad;
    mine += request_cost(p, s);
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
  for (int w = 0; w < C::kThreads / 32; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  Meta* meta = reinterpret_cast<Meta*>(p.ws) + blockIdx.x;
  // blocks of threads in use: none of their spans is empty, so the parts of a chunk lie in neighbours
  const long long blocks = min(static_cast<long long>(gridDim.x), (total + kMinCost - 1) / kMinCost);
  if (blockIdx.x >= blocks) {
    if (tid == 0) *meta = Meta{};
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    return;
  }
  const long long span0 = total * blockIdx.x / blocks, span1 = total * (blockIdx.x + 1) / blocks;
  if (before <= span0 && span0 < before + mine) {  // one thread: the span starts in its run
    int b = my0;
    for (;; ++b) {
      const long long n = request_cost(p, seq_len(p, b));
      if (span0 < before + n) break;
      before += n;
    }
    for (int w = 0; w < 14; ++w) {
      walks[w].pos = span0;
      walks[w].end = span1;
      walks[w].first = before;
      walks[w].b = b;
      walks[w].chunk = 0;
      walks[w].chunks = -1;
    }
  }
  if (warp == 0) {
    tmem_alloc(&tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const AbortState ab{&abort_flag, p.status};
  float* parts = reinterpret_cast<float*>(p.ws + static_cast<size_t>(gridDim.x) * sizeof(Meta)) +
                 static_cast<size_t>(blockIdx.x) * 2 * part_floats<D, ROWS>();

  if (warp < 8) {
    // ================================================================ softmax, Q and O of tile q
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegSoftmax));
    const int q = warp >> 2;
    const int row = (warp & 3) * 32 + lane;  // of the tile, and lane of tensor memory
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t tS = lane_base + q * 128, tO = lane_base + C::kOCol + q * D;
    uint8_t* sq = smem + C::kQOff + q * C::kTileBytes;
    uint32_t blk = 0;   // blocks of keys so far
    uint32_t sit = 0;   // of them, blocks of this tile
    uint32_t uit = 0;   // segments of this tile
    Meta found{};
    bool ok = true;
    Segment S;
    while (ok && take_segment(p, walks[warp], lane, S)) {
      const int row0 = S.chunk * ROWS, rows = min(ROWS, S.nq * p.G - row0);
      const bool starts = S.t0 == 0, ends = S.t1 == S.units;
      if (starts && !ends) {
        found.tail_valid = 1;
        found.b = S.b, found.h = S.h, found.chunk = S.chunk;
      } else if (!starts) {
        found.head_valid = 1;
        found.head_ends = ends;
      }
      if (q * 128 >= rows) {  // no row of this tile
        blk += S.t1 - S.t0;
        continue;
      }
      const int rr = row0 + q * 128 + row;  // row of the request
      const bool valid = q * 128 + row < rows;
      const int tok = rr / p.G, hq = S.h * p.G + rr - tok * p.G;

      // Q: one row per thread, transformed in float32, largest entry at 2^13 .. 2^14
      float c_row;
      {
        float x[D];
        if (valid) {
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                            (S.q0 + tok) * p.q_sn + hq * p.q_sh);
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            const uint4 u = src[i];
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
              x[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < D; ++i) x[i] = 0.f;
        }
        if (p.signs != nullptr) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const int4 sg = reinterpret_cast<const int4*>(p.signs)[i];
            const int sw[4] = {sg.x, sg.y, sg.z, sg.w};
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (static_cast<signed char>(sw[k >> 2] >> (8 * (k & 3))) == -1) x[16 * i + k] = -x[16 * i + k];
          }
#pragma unroll
          for (int st = 1; st < D; st <<= 1)
#pragma unroll
            for (int i = 0; i < D; ++i)
              if (!(i & st)) {
                const float a = x[i], b = x[i | st];
                x[i] = a + b;
                x[i | st] = a - b;
              }
        }
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < D; ++i) top = fmaxf(top, fabsf(x[i]));
        const int ex = top > 0.f ? min(max(exponent_of(top) - 13, -100), 100) : 0;
        const float f = exp2_int(-ex);
        c_row = p.scale_log2 * exp2_int(ex);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const float* v = x + 8 * i;
          *reinterpret_cast<uint4*>(sq + (i / 8) * C::kBoxBytes + row * 128 + (((i & 7) ^ (row & 7)) << 4)) =
              make_uint4(pack_f16x2(v[0] * f, v[4] * f), pack_f16x2(v[1] * f, v[5] * f), pack_f16x2(v[2] * f, v[6] * f),
                         pack_f16x2(v[3] * f, v[7] * f));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive(&q_full[q]);

      const int off = S.nk - S.nq;
      const int lim_row = !valid ? S.nk : p.causal ? min(S.nk, off + tok + 1) : S.nk;  // keys [0, lim_row) are seen
      const int lim_first = p.causal ? min(S.nk, off + (row0 + q * 128) / p.G + 1) : S.nk;  // by the tile's first row
      float m = kNegBig, l = 0.f;
      int v_exp = 0;
      for (int t = S.t0; t < S.t1; ++t, ++blk, ++sit) {
        ok = warp_all(wait_bar(&s_full[q], sit & 1u, ab));
        if (!ok) break;
        tc_fence_after();
        const BlockInfo bi = info[blk & 1u];
        const float c = c_row * bi.k_back;
        uint32_t r[128];
        load_row(tS, r);
        const int key0 = t * kBlockKeys;
        const bool need_mask = key0 + kBlockKeys > lim_first || bi.gone != 0;
        if (need_mask) {
          const int lim = lim_row - key0;
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i >= lim || ((bi.gone >> (i >> 4)) & 1u)) r[i] = __float_as_uint(-INFINITY);
        }
        float mx[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) mx[i] = __uint_as_float(r[i]);
#pragma unroll
        for (int i = 8; i < 128; i += 8)
#pragma unroll
          for (int k = 0; k < 8; ++k) mx[k] = fmaxf(mx[k], __uint_as_float(r[i + k]));
        const float mb = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                               fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * c;
        float alpha = 1.f;
        if (mb > m + kTau) {
          alpha = ex2_approx(m - mb);
          m = mb;
          l *= alpha;
        }
        uint32_t pk[64];
        l += need_mask ? softmax_row<true>(r, pk, c, -m) : softmax_row<false>(r, pk, c, -m);
        tmem_st_32cols(tS, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
        tmem_st_32cols(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
        tmem_st_wait();
        if (t > S.t0 && bi.v_exp != v_exp) alpha *= exp2_int(max(v_exp - bi.v_exp, -126));
        v_exp = bi.v_exp;
        if (__any_sync(0xffffffffu, alpha != 1.f) && t > S.t0) {
          // O *= alpha: the P.V of the block before has completed (it was issued before this block's S)
          tc_fence_after();
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];
            tmem_ld_32cols(tO + 32 * cc, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st_32cols(tO + 32 * cc, o);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&p_full[q]);
      }
      if (!ok) break;

      // O, or this segment's part of it
      ok = warp_all(wait_bar(&o_done[q], uit & 1u, ab));
      ++uit;
      if (!ok) break;
      tc_fence_after();
      const bool whole = starts && ends;
      const float back = exp2_int(v_exp) * (!whole ? 1.f : l == 0.f ? 0.f : 1.f / l);
      const int pr = q * 128 + row;
      float* part = parts + (starts ? part_floats<D, ROWS>() : 0);
#pragma unroll 1
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t o[32];
        tmem_ld_32cols(tO + 32 * cc, o);
        tmem_ld_wait(o);
        if (!valid) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // columns hold dimensions 0 4 1 5 2 6 3 7
            v[k] = __uint_as_float(o[8 * i + 2 * k]) * back;
            v[4 + k] = __uint_as_float(o[8 * i + 2 * k + 1]) * back;
          }
          if (whole) {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + (S.q0 + tok) * p.o_sn + hq * p.o_sh + 32 * cc + 8 * i) =
                make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
          } else {
            float4* dst = reinterpret_cast<float4*>(part + pr * D + 32 * cc + 8 * i);
            dst[0] = make_float4(v[0], v[1], v[2], v[3]);
            dst[1] = make_float4(v[4], v[5], v[6], v[7]);
          }
        }
      }
      if (valid) {
        if (!whole) {
          part[ROWS * D + pr] = m;
          part[ROWS * D + ROWS + pr] = l;
        } else if (p.lse != nullptr) {
          p.lse[static_cast<long long>(hq) * p.total_q + S.q0 + tok] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2f;
        }
      }
      tc_fence_before();  // the next segment's first P.V comes after its q_full
    }
    if (tid == 0) *meta = found;
  } else if (warp < 12) {
    // ================================================================ codes to float16
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegCodes));
    const int ct = tid - 256;
    const int c = ct & 3;
    uint32_t blk = 0, pair = 0;
    int v_exp = -200;  // reference exponent of V in this segment
    bool ok = true;
    Segment S;
    while (ok && take_segment(p, walks[warp], lane, S)) {
      v_exp = -200;
      for (int t = S.t0; t < S.t1 && ok; ++t, ++blk) {
        for (int i = 0; i < 4 && ok; ++i)
          ok = warp_all(wait_bar(&raw_full[(pair + i) % C::kRawSlots], ((pair + i) / C::kRawSlots) & 1u, ab));
        ok = ok && warp_all(wait_bar(&kv_empty[blk & 1u], ((blk >> 1) & 1u) ^ 1u, ab));
        // largest values of the block, one key per thread; a key that is not there, or not finite, counts as zero
        float mk = 0.f, mv = 0.f;
        if (ok) {
          const uint32_t slot = (pair + (ct >> 5)) % C::kRawSlots;
          const int ti = (ct >> 4) & 1, r = ct & 15;
          const uint8_t* tile = smem + C::kRawOff + slot * C::kRawBytes + ti * F::kBytes;
          if (!((raw_gone[slot] >> ti) & 1u) && t * kBlockKeys + ct < S.nk) {
#pragma unroll
            for (int g = 0; g < D / 64; ++g) {
              const uint32_t k = *reinterpret_cast<const uint32_t*>(tile + F::kKszOff + r * F::kSzRow + 4 * g);
              const uint32_t v = *reinterpret_cast<const uint32_t*>(tile + F::kVszOff + r * F::kSzRow + 4 * g);
              const float ks = __uint_as_float(k << 16), kz = __uint_as_float(k & 0xFFFF0000u);
              const float vs = __uint_as_float(v << 16), vz = __uint_as_float(v & 0xFFFF0000u);
              mk = fmaxf(mk, fmaxf(fabsf(kz), fabsf(fmaf(15.f, ks, kz))));
              mv = fmaxf(mv, fmaxf(fabsf(vz), fabsf(fmaf(15.f, vs, vz))));
            }
          }
        }
        mk = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mk)));
        mv = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mv)));
        if (lane == 0) {
          wmax[blk & 1u][0][warp - 8] = mk;
          wmax[blk & 1u][1][warp - 8] = mv;
        }
        // the four warps meet here once per block, whatever came of their waits, and go on or stop together
        ok = codes_all(ok);
        if (!ok) break;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          mk = fmaxf(mk, wmax[blk & 1u][0][w]);
          mv = fmaxf(mv, wmax[blk & 1u][1][w]);
        }
        // K's largest value of the block at 2^10 .. 2^11, V's of the segment so far at most there
        const int ke = mk > 0.f ? min(max(exponent_of(mk) - 10, -110), 110) : 0;
        const int ve = mv > 0.f ? min(max(exponent_of(mv) - 10, -110), 110) : -110;
        v_exp = max(v_exp, ve);
        const float kf = exp2_int(-ke), vf = exp2_int(-v_exp);
        uint8_t* sk = smem + C::kKvOff + (blk & 1u) * 2 * C::kTileBytes;
        uint8_t* sv = sk + C::kTileBytes;
        uint32_t gone = 0;
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          const uint32_t slot = (pair + i) % C::kRawSlots;
          gone |= raw_gone[slot] << (2 * i);
          const int key = 32 * i + (ct >> 2), ti = ct >> 6, r = (ct >> 2) & 15;
          const uint8_t* tile = smem + C::kRawOff + slot * C::kRawBytes + ti * F::kBytes;
          const bool there = !((raw_gone[slot] >> ti) & 1u) && t * kBlockKeys + key < S.nk;
          uint32_t kw[2 * (D / 64)], vw[2 * (D / 64)];  // K: [group][8 dimensions]; V: [8 dimensions][group]
          if constexpr (D == 128) {
            const uint4 a = *reinterpret_cast<const uint4*>(tile + r * F::kRowBytes + 16 * c);
            const uint4 b = *reinterpret_cast<const uint4*>(tile + F::kVOff + r * F::kRowBytes + 16 * c);
            kw[0] = a.x, kw[1] = a.y, kw[2] = a.z, kw[3] = a.w;
            vw[0] = b.x, vw[1] = b.y, vw[2] = b.z, vw[3] = b.w;
          } else {
            const uint2 a = *reinterpret_cast<const uint2*>(tile + r * F::kRowBytes + 8 * c);
            const uint2 b = *reinterpret_cast<const uint2*>(tile + F::kVOff + r * F::kRowBytes + 8 * c);
            kw[0] = a.x, kw[1] = a.y;
            vw[0] = b.x, vw[1] = b.y;
          }
          uint32_t ksz[D / 64], vsz[D / 64];
          bool odd = false;  // a V that is not finite
#pragma unroll
          for (int g = 0; g < D / 64; ++g) {
            ksz[g] = *reinterpret_cast<const uint32_t*>(tile + F::kKszOff + r * F::kSzRow + 4 * g);
            vsz[g] = *reinterpret_cast<const uint32_t*>(tile + F::kVszOff + r * F::kSzRow + 4 * g);
            if (!there) ksz[g] = vsz[g] = 0u;
            const float vz = __uint_as_float(vsz[g] & 0xFFFF0000u);
            odd = odd || !(fabsf(vz) < INFINITY) || !(__uint_as_float(vsz[g] << 16) < INFINITY);
          }
#pragma unroll
          for (int g = 0; g < D / 64; ++g) {
            // rows that do not see a key must not see its NaN either: V of such a key is zero, and its scores, which
            // the mask replaces, are NaN
            if (odd) ksz[g] = 0x7FC07FC0u, vsz[g] = 0u;
            const float ks = __uint_as_float(ksz[g] << 16) * kf, kz = __uint_as_float(ksz[g] & 0xFFFF0000u) * kf;
            const float vs = __uint_as_float(vsz[g] << 16) * vf, vz = __uint_as_float(vsz[g] & 0xFFFF0000u) * vf;
            const uint32_t ks2 = pack_f16x2(ks, ks), kz2 = pack_f16x2(kz, kz);
            const uint32_t vs2 = pack_f16x2(vs, vs), vz2 = pack_f16x2(vz, vz);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t at = g * C::kBoxBytes + key * 128 + (((2 * c + h) ^ (key & 7)) << 4);
              *reinterpret_cast<uint4*>(sk + at) = expand(kw[2 * g + h], ks2, kz2);
              *reinterpret_cast<uint4*>(sv + at) = expand(vw[(D / 64) * h + g], vs2, vz2);
            }
          }
          __syncwarp();
          if (lane == 0) bar_arrive(&raw_empty[slot]);
        }
        pair += 4;
        if (ct == 0) info[blk & 1u] = BlockInfo{exp2_int(ke), v_exp, gone};
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(&kv_full[blk & 1u]);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegOther));
    if (warp == 12) {
      // ============================================================== MMA issuer
      constexpr uint32_t kIdS = make_idesc(128, 128, 0, false);  // float16, both K-major
      constexpr uint32_t kIdPV = make_idesc(128, D, 0, true);    // V MN-major
      const uint32_t q_base = smem_addr(smem + C::kQOff), kv_base = smem_addr(smem + C::kKvOff);
      uint32_t blk = 0, n_p[2] = {0, 0}, n_q[2] = {0, 0};
      auto issue_s = [&](int q, uint32_t buf) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk / 4) * C::kBoxBytes + (kk % 4) * 32;
          mma_f16_ss(tmem + q * 128, make_sdesc_sw128(q_base + q * C::kTileBytes + off, 16, 1024),
                     make_sdesc_sw128(kv_base + buf * 2 * C::kTileBytes + off, 16, 1024), kIdS, kk > 0 ? 1u : 0u);
        }
        tc_commit(&s_full[q]);
      };
      auto issue_pv = [&](int q, uint32_t buf, bool acc) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_f16_ts(tmem + C::kOCol + q * D, tmem + q * 128 + kk * 8,
                     make_sdesc_sw128(kv_base + (2 * buf + 1) * C::kTileBytes + kk * 16 * 128, C::kBoxBytes, 1024), kIdPV,
                     (acc || kk > 0) ? 1u : 0u);
      };
      bool ok = true;
      Segment S;
      while (ok && take_segment(p, walks[warp], lane, S)) {
        const int tiles = min(ROWS, S.nq * p.G - S.chunk * ROWS) > 128 ? 2 : 1;
        if (lane == 0) {
          const int n = S.t1 - S.t0;
          ok = wait_bar(&kv_full[blk & 1u], (blk >> 1) & 1u, ab);
          for (int q = 0; q < tiles && ok; ++q) {
            ok = wait_bar(&q_full[q], n_q[q]++ & 1u, ab);
            if (!ok) break;
            tc_fence_after();
            issue_s(q, blk & 1u);
          }
          for (int j = 0; j < n && ok; ++j, ++blk) {
            const bool more = j + 1 < n;
            for (int q = 0; q < tiles && ok; ++q) {
              ok = wait_bar(&p_full[q], n_p[q]++ & 1u, ab);
              if (!ok) break;
              tc_fence_after();
              issue_pv(q, blk & 1u, j > 0);
              if (q == tiles - 1) tc_commit(&kv_empty[blk & 1u]);
              if (more) {
                if (q == 0) ok = wait_bar(&kv_full[(blk + 1) & 1u], ((blk + 1) >> 1) & 1u, ab);
                if (!ok) break;
                tc_fence_after();
                issue_s(q, (blk + 1) & 1u);
              } else {
                tc_commit(&o_done[q]);
              }
            }
          }
        }
        ok = warp_all(ok);
      }
      if (lane == 0) {  // every product has completed before tensor memory is given back
        tc_commit(&drained);
        drain(&drained, 0);
      }
      __syncwarp();
    } else if (warp == 13) {
      // ============================================================== copies of the cache's tiles
      uint32_t pair = 0;
      bool ok = true;
      Segment S;
      while (ok && take_segment(p, walks[warp], lane, S)) {
        const uint8_t* next = nullptr;
        int state = 0;  // of this lane's tile of the block: 0 past the keys, 1 there, 2 no block of the cache
        auto look = [&](int t) {
          const int key = t * kBlockKeys + 16 * lane;
          state = 0;
          if (lane < 8 && t < S.t1 && key < S.nk) {
            const int j = key / p.page;
            const int e = __ldg(p.table + static_cast<long long>(S.b) * p.width + j);
            state = e >= 0 && e < p.num_blocks ? 1 : 2;
            if (state == 1) next = p.cache + kv4_tile_offset<D>(e, key - j * p.page, p.page, p.Hk, S.h);
            else atomicOr(p.status, kDevStatusBadSeqlens);
          }
        };
        look(S.t0);
        for (int t = S.t0; t < S.t1 && ok; ++t) {
          const uint8_t* src = next;
          const uint32_t there = __ballot_sync(0xffffffffu, state == 1), gone = __ballot_sync(0xffffffffu, state == 2);
          look(t + 1);  // one block ahead of its copies
          for (int i = 0; i < 4 && ok; ++i, ++pair) {
            const uint32_t slot = pair % C::kRawSlots;
            ok = warp_all(wait_bar(&raw_empty[slot], ((pair / C::kRawSlots) & 1u) ^ 1u, ab));
            if (!ok) break;
            const uint32_t have = (there >> (2 * i)) & 3u;
            if (lane == 0) {
              raw_gone[slot] = (gone >> (2 * i)) & 3u;
              bar_arrive_expect_tx(&raw_full[slot], __popc(have) * F::kBytes);
            }
            __syncwarp();
            if ((lane >> 1) == i && ((have >> (lane & 1)) & 1u))
              bulk_load_g2s(smem + C::kRawOff + slot * C::kRawBytes + (lane & 1) * F::kBytes, src, F::kBytes, &raw_full[slot]);
          }
        }
      }
      // after a wait that ran out, the copies in flight still land in this block's memory: wait for them
      if (!ok && lane == 0)
        for (uint32_t i = pair > C::kRawSlots ? pair - C::kRawSlots : 0; i < pair; ++i)
          drain(&raw_full[i % C::kRawSlots], (i / C::kRawSlots) & 1u);
      __syncwarp();
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D>
cudaError_t launch(const Kv4AttnParams& p, int num_sms, cudaStream_t stream) {
  using C = ChunkCfg<D>;
  kv4_chunk_kernel<D><<<num_sms, C::kThreads, C::kSmem, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_join<D, kRowsPerChunk>(p, num_sms, 16, stream);
}

}  // namespace

cudaError_t setup_kv4_chunk_kernels() {
  cudaError_t e = cudaFuncSetAttribute(kv4_chunk_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, ChunkCfg<64>::kSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kv4_chunk_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, ChunkCfg<128>::kSmem);
  return e;
}

unsigned long long kv4_chunk_workspace_bytes(int d, int num_sms) {
  return d == 64 ? part_bytes<64, kRowsPerChunk>(num_sms) : d == 128 ? part_bytes<128, kRowsPerChunk>(num_sms) : 0;
}

cudaError_t launch_kv4_chunk(const Kv4AttnParams& p, int d, int num_sms, cudaStream_t stream) {
  return d == 64 ? launch<64>(p, num_sms, stream) : launch<128>(p, num_sms, stream);
}

}  // namespace ea

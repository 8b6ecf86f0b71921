// Writer and reader of the 4-bit key/value cache.
//
// Append: y = x, or for K with signs y = (1/sqrt d) H_d (D x) ("FlashAttention-3", section "FP8
// 路径与低精度误差": the transform spreads outliers over the row before it is quantised; Q is given the
// same one, and scores do not change).  Per group of 64: z = the largest bf16 <= min y, s = the smallest
// bf16 >= (max y - z) / 15, u = rint((y - z) / s).  Rounding z down and s up keeps every value within
// z .. z + 15 s, so no code is cut off by the rounding of its own scale.
//
// Append has 4 bytes to read and 1.125 to write per value pair (13 us for 16,384 tokens of 8 heads of 128), and is bound
// by its instructions, 28.6 us: a lane holds 16 consecutive values of a row (two 16-byte loads, d / 16 lanes per
// row, several rows per warp), so four of the transform's stages and most of the minimum and maximum stay in the
// lane, and a group is four adjacent lanes.  K and V rows go to different blocks of threads.  The quotients come from the
// group's one reciprocal, corrected to the rounded quotient (three operations instead of a division each: 54 us
// before), each row's addresses from one lane instead of its d / 16, and a round's values are asked for while the
// one before is worked on.
//
// Read: a thread has four dimensions of a row, so that each store of a warp is contiguous.

#include <cuda_bf16.h>

#include "attn_kernels.h"
#include "kv4_format.cuh"
#include "kv_kernels.h"

namespace ea {

namespace {

constexpr int kThreads = 256;

// Largest bf16 not above x, smallest not below, as float bits (infinities and NaN stay what they are
// or become infinite; the caller has looked for them).
__device__ __forceinline__ float bf16_down(float x) {
  const uint32_t b = __float_as_uint(x);
  return __uint_as_float(((b >> 31) ? b + 0xFFFFu : b) & 0xFFFF0000u);
}
__device__ __forceinline__ float bf16_up(float x) {  // x >= 0
  return __uint_as_float((__float_as_uint(x) + 0xFFFFu) & 0xFFFF0000u);
}

// minimum and maximum that a NaN goes through
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Rounds of a warp of the writer, up to 4 where there are enough rows for 4 blocks of threads on each of 148 processors
// all the same (16,384 tokens of 8 heads of 128: 39.6, 32.1 and 28.6 us with 1, 2 and 4).
constexpr int kAppendRounds = 4;
constexpr long long kAppendBlocks = 4 * 148;

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const Kv4CacheParams p, const int rounds) {
  using F = Kv4Tile<D>;
  constexpr int kLanes = D / 16;         // lanes per row
  constexpr int kAtOnce = 32 / kLanes;   // rows of a warp
  const int lane = threadIdx.x & 31;
  const int j = lane % kLanes;
  const bool is_v = blockIdx.y != 0;
  const bool transform = !is_v && p.signs != nullptr;
  // Lane i finds where row first + i comes from and goes to, for the whole warp (fewer than 2^31 rows, the caller's bound,
  // and a block's rows past them at most).  `to`: its row in the tile in the upper 8 bits, all ones: nowhere.
  const unsigned rows = static_cast<unsigned>(p.T) * static_cast<unsigned>(p.Hk);
  const unsigned first = (blockIdx.x * (kThreads / 32) + threadIdx.x / 32) * (rounds * kAtOnce);
  long long from = 0;
  unsigned long long to = ~0ull;
  if (lane < rounds * kAtOnce && first + lane < rows) {
    const unsigned row = first + lane;
    const int t = static_cast<int>(row / static_cast<unsigned>(p.Hk)), h = static_cast<int>(row) - t * p.Hk;
    const int slot = p.slots[t];
    from = t * (is_v ? p.v_sn : p.k_sn) + h * (is_v ? p.v_sh : p.k_sh);
    const int block = slot < 0 ? 0 : slot / p.page, off = slot - block * p.page;
    if (slot < -1 || block >= p.num_blocks) atomicOr(p.status, kDevStatusBadSeqlens);
    else if (slot >= 0)
      to = static_cast<unsigned long long>(kv4_tile_offset<D>(block, off, p.page, p.Hk, h)) |
           (static_cast<unsigned long long>(off & 15) << 56);
  }
  uint32_t flip[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};  // the sign bits of this lane's pairs
  if (transform) {
    const int4 sg = *reinterpret_cast<const int4*>(p.signs + 16 * j);
    const int sw[4] = {sg.x, sg.y, sg.z, sg.w};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (static_cast<signed char>(sw[i >> 2] >> (8 * (i & 3))) == -1) flip[i >> 1] |= i & 1 ? 0x80000000u : 0x8000u;
  }
  const __nv_bfloat16* const src = static_cast<const __nv_bfloat16*>(is_v ? p.v : p.k) + 16 * j;
  uint4 na = make_uint4(0u, 0u, 0u, 0u), nb = na;
  auto ask = [&](int k) {  // for the values of round k
    const int of = k * kAtOnce + lane / kLanes;
    const long long at = __shfl_sync(0xffffffffu, from, of);
    if (first + of < rows) {
      na = reinterpret_cast<const uint4*>(src + at)[0];
      nb = reinterpret_cast<const uint4*>(src + at)[1];
    }
  };
  ask(0);
#pragma unroll 1
  for (int k = 0; k < rounds; ++k) {
    const unsigned long long dst = __shfl_sync(0xffffffffu, to, k * kAtOnce + lane / kLanes);
    float x[16];
    {
      const uint32_t w[8] = {na.x, na.y, na.z, na.w, nb.x, nb.y, nb.z, nb.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t u = w[i] ^ flip[i];
        x[2 * i] = __uint_as_float(u << 16);
        x[2 * i + 1] = __uint_as_float(u & 0xFFFF0000u);
      }
    }
    if (k + 1 < rounds) ask(k + 1);
    if (transform) {  // uniform over the block
#pragma unroll
      for (int s = 1; s < 16; s <<= 1)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (!(i & s)) {
            const float a = x[i], b = x[i | s];
            x[i] = a + b;
            x[i | s] = a - b;
          }
#pragma unroll
      for (int s = 1; s < kLanes; s <<= 1) {
        const float sign = (j & s) ? -1.f : 1.f;
#pragma unroll
        for (int i = 0; i < 16; ++i)  // other + x, or other - x: the product is exact
          x[i] = fmaf(sign, x[i], __shfl_xor_sync(0xffffffffu, x[i], s));
      }
      constexpr float kNorm = D == 64 ? 0.125f : D == 128 ? 0.08838834764831845f : 0.0625f;
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(x[i], kNorm);
    }
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) {
      lo = min_nan(lo, x[i]);
      hi = max_nan(hi, x[i]);
    }
#pragma unroll
    for (int s = 1; s < 4; s <<= 1) {
      lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, s));
      hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, s));
    }
    float z = bf16_down(lo);
    const float range = __fsub_rn(hi, z);
    // a NaN goes through the minimum and the maximum, an infinity makes the range infinite or NaN
    const unsigned odds = __ballot_sync(0xffffffffu, !isfinite(range));
    // range / 15 rounded, likewise
    float s;
    if (range > 1e-28f && range < 1e30f) {
      constexpr float kY = 1.f / 15.f;
      const float q = __fmul_rn(range, kY);
      s = bf16_up(fmaf(fmaf(-q, 15.f, range), kY, q));
    } else {
      s = bf16_up(__fdiv_rn(range, 15.f));
    }
    uint32_t code[2] = {0u, 0u};
    if ((odds >> (lane & ~3)) & 15u) {
      s = z = __uint_as_float(0x7FC00000u);
    } else if (s > 1e-30f && s < 1e30f) {
      // With y = 1 / s rounded, q = t y and the exact remainder t - q s, q + remainder y is the rounded quotient (Markstein).
      // It is at least 0 and rounds to 15 at most; 1.5 2^23 added rounds it to the nearest integer, in the low bits.
      const float y = __frcp_rn(s);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        uint32_t c = 0u;
#pragma unroll
        for (int i = 7; i >= 0; --i) {
          const float u = __fsub_rn(x[8 * w + i], z);
          const float q = __fmul_rn(u, y);
          const float n = __fadd_rn(fmaf(fmaf(-q, s, u), y, q), 12582912.f);
          c = c * 16u + __float_as_uint(n);
        }
        code[w] = c - 0x11111111u * 0x4B400000u;  // what the shift's own bits add up to
      }
    } else if (s > 0.f) {
#pragma unroll 1
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float u = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(w ? x[8 + i] : x[i], z), s)), 0.f), 15.f);
          code[w] |= static_cast<uint32_t>(u) << (4 * i);
        }
    }
    if (dst == ~0ull) continue;
    uint8_t* tile = p.cache + (dst & ((1ull << 56) - 1));
    const int r = static_cast<int>(dst >> 56);
    const int plane = j / (F::kPlaneDims / 16), g = (j / 4) % F::kGroups, c = j & 3;  // dims 64 g + 16 c .. of the plane
    if (!is_v) {
      *reinterpret_cast<uint2*>(tile + plane * F::kPlaneBytes + r * F::kRowBytes + c * 8 * F::kGroups + 8 * g) =
          make_uint2(code[0], code[1]);
    } else {
      uint8_t* d = tile + F::kVOff + plane * F::kPlaneBytes + r * F::kRowBytes + 2 * c * 4 * F::kGroups + 4 * g;
      *reinterpret_cast<uint32_t*>(d) = code[0];
      *reinterpret_cast<uint32_t*>(d + 4 * F::kGroups) = code[1];
    }
    if (c == 0)
      *reinterpret_cast<uint32_t*>(tile + (is_v ? F::kVszOff : F::kKszOff) + r * F::kSzRow + 4 * (j / 4)) =
          (__float_as_uint(s) >> 16) | (__float_as_uint(z) & 0xFFFF0000u);
  }
}

// One store of a warp: half a row of d = 256, a row of 128, two of 64.  A warp has kReadRows such rows (or pairs), whose
// loads are in flight together; each of its lanes finds one of them in the cache (every lane for itself, the divisions
// took longer than the memory).
constexpr int kReadRows = 8;

template <int D>
struct ReadCfg {
  static constexpr int kLanes = D / 4;                              // of a row, four dimensions each
  static constexpr int kAtOnce = kLanes < 32 ? 32 / kLanes : 1;     // rows of one store
  static constexpr int kWarpsPerRow = kLanes > 32 ? kLanes / 32 : 1;
  static constexpr int kRowsPerWarp = kAtOnce * kReadRows;
  static constexpr int kRowsPerBlock = kThreads / 32 / kWarpsPerRow * kRowsPerWarp;
};

template <int D, bool F32>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const Kv4CacheParams p) {
  using F = Kv4Tile<D>;
  using C = ReadCfg<D>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int x = 4 * (threadIdx.x % C::kLanes);  // this thread's dimensions x .. x + 3
  const bool is_v = blockIdx.y != 0;
  const int xp = x % F::kPlaneDims, g = xp / 64, rr = xp % 64;
  const int code_at = (is_v ? F::kVOff + (rr / 8) * 4 * F::kGroups + 4 * g + (rr % 8) / 2
                            : (rr / 16) * 8 * F::kGroups + 8 * g + (rr % 16) / 2) + (x / F::kPlaneDims) * F::kPlaneBytes;
  const int sz_at = (is_v ? F::kVszOff : F::kKszOff) + 4 * (x / 64);
  const unsigned rows = static_cast<unsigned>(p.T) * static_cast<unsigned>(p.Hk);
  const unsigned first = blockIdx.x * C::kRowsPerBlock + (warp / C::kWarpsPerRow) * C::kRowsPerWarp;
  // lane i: where row first + i lies, its row in the tile in the upper 8 bits; all ones: nowhere
  unsigned long long at = ~0ull;
  if (lane < C::kRowsPerWarp && first + lane < rows) {
    const unsigned row = first + lane;
    const int t = static_cast<int>(row / static_cast<unsigned>(p.Hk)), h = static_cast<int>(row) - t * p.Hk;
    const int slot = p.slots[t];
    const int block = slot < 0 ? 0 : slot / p.page, off = slot - block * p.page;
    if (slot < -1 || block >= p.num_blocks) atomicOr(p.status, kDevStatusBadSeqlens);
    else if (slot >= 0)
      at = static_cast<unsigned long long>(kv4_tile_offset<D>(block, off, p.page, p.Hk, h)) |
           (static_cast<unsigned long long>(off & 15) << 56);
  }
  const int sub = lane / C::kLanes;  // 0, or which of two rows
  uint32_t code[kReadRows], sz[kReadRows];
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    const unsigned long long a = __shfl_sync(0xffffffffu, at, i * C::kAtOnce + sub);
    code[i] = sz[i] = 0u;
    if (a != ~0ull) {
      const uint8_t* tile = p.cache + (a & ((1ull << 56) - 1));
      const int r = static_cast<int>(a >> 56);
      code[i] = *reinterpret_cast<const uint16_t*>(tile + code_at + r * F::kRowBytes);
      sz[i] = *reinterpret_cast<const uint32_t*>(tile + sz_at + r * F::kSzRow);
    }
  }
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    const unsigned row = first + i * C::kAtOnce + sub;
    if (row >= rows) break;
    const float s = __uint_as_float(sz[i] << 16), z = __uint_as_float(sz[i] & 0xFFFF0000u);
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = fmaf(static_cast<float>((code[i] >> (4 * k)) & 15u), s, z);
    const long long to = static_cast<long long>(row) * D + x;
    if constexpr (F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(is_v ? p.v_out : p.k_out) + to) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      uint32_t w[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[k]) : "f"(v[2 * k + 1]), "f"(v[2 * k]));
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(is_v ? p.v_out : p.k_out) + to) = make_uint2(w[0], w[1]);
    }
  }
}

dim3 grid_of(const Kv4CacheParams& p, int rows_per_block) {
  const long long rows = static_cast<long long>(p.T) * p.Hk;
  return dim3(static_cast<unsigned>((rows + rows_per_block - 1) / rows_per_block), 2);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4CacheParams& p, int d, cudaStream_t stream) {
  const int step = kThreads / (d / 16);
  const long long full = static_cast<long long>(p.T) * p.Hk / (kAppendBlocks * step);
  const int rounds = full < 1 ? 1 : full > kAppendRounds ? kAppendRounds : static_cast<int>(full);
  const dim3 grid = grid_of(p, rounds * step);
  if (d == 64) kv4_append_kernel<64><<<grid, kThreads, 0, stream>>>(p, rounds);
  else if (d == 128) kv4_append_kernel<128><<<grid, kThreads, 0, stream>>>(p, rounds);
  else kv4_append_kernel<256><<<grid, kThreads, 0, stream>>>(p, rounds);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4CacheParams& p, int d, bool out_f32, cudaStream_t stream) {
  const dim3 grid = grid_of(p, d == 64 ? ReadCfg<64>::kRowsPerBlock : d == 128 ? ReadCfg<128>::kRowsPerBlock
                                                                              : ReadCfg<256>::kRowsPerBlock);
  if (out_f32) {
    if (d == 64) kv4_read_kernel<64, true><<<grid, kThreads, 0, stream>>>(p);
    else if (d == 128) kv4_read_kernel<128, true><<<grid, kThreads, 0, stream>>>(p);
    else kv4_read_kernel<256, true><<<grid, kThreads, 0, stream>>>(p);
  } else {
    if (d == 64) kv4_read_kernel<64, false><<<grid, kThreads, 0, stream>>>(p);
    else if (d == 128) kv4_read_kernel<128, false><<<grid, kThreads, 0, stream>>>(p);
    else kv4_read_kernel<256, false><<<grid, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace ea

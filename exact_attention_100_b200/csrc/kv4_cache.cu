// Writer and reader of the 4-bit key/value cache.
//
// Append: y = x, or for K with signs y = (1/sqrt d) H_d (D x) ("FlashAttention-3", section "FP8
// 路径与低精度误差": the transform spreads outliers over the row before it is quantised; Q is given the
// same one, and scores do not change).  Per group of 64: z = the largest bf16 <= min y, s = the smallest
// bf16 >= (max y - z) / 15, u = rint((y - z) / s).  Rounding z down and s up keeps every value within
// z .. z + 15 s, so no code is cut off by the rounding of its own scale.
//
// Bound by memory: 4 bytes of K and V read and 1.125 written per value pair.  A lane holds 16
// consecutive values of a row (two 16-byte loads, d / 16 lanes per row, several rows per warp), so four of
// the transform's stages and most of the minimum and maximum stay in the lane, and a group is four
// adjacent lanes.  K and V rows go to different blocks of threads.

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

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const Kv4CacheParams p) {
  using F = Kv4Tile<D>;
  constexpr int kLanes = D / 16;  // lanes per row
  const int lane = threadIdx.x & 31;
  const int j = lane % kLanes;
  const bool is_v = blockIdx.y != 0;
  const bool transform = !is_v && p.signs != nullptr;
  const long long rows = static_cast<long long>(p.T) * p.Hk;
  const long long row = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) / kLanes;
  const bool live = row < rows;
  int t = 0, h = 0, slot = -1;
  if (live) {
    t = static_cast<int>(row / p.Hk);
    h = static_cast<int>(row - static_cast<long long>(t) * p.Hk);
    slot = p.slots[t];
  }
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.f;
  if (slot >= 0) {
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_v ? p.v : p.k) +
                               t * (is_v ? p.v_sn : p.k_sn) + h * (is_v ? p.v_sh : p.k_sh) + 16 * j;
    const uint4 a = reinterpret_cast<const uint4*>(src)[0], b = reinterpret_cast<const uint4*>(src)[1];
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  if (transform) {  // uniform over the block
    const int4 sg = *reinterpret_cast<const int4*>(p.signs + 16 * j);
    const int sw[4] = {sg.x, sg.y, sg.z, sg.w};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (static_cast<signed char>(sw[i >> 2] >> (8 * (i & 3))) == -1) x[i] = -x[i];
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
      const bool hi = (j & s) != 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float o = __shfl_xor_sync(0xffffffffu, x[i], s);
        x[i] = hi ? o - x[i] : x[i] + o;
      }
    }
    constexpr float kNorm = D == 64 ? 0.125f : D == 128 ? 0.08838834764831845f : 0.0625f;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(x[i], kNorm);
  }
  float lo = x[0], hi = x[0];
  bool odd = false;  // a value that is not finite
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
    odd = odd || !isfinite(x[i]);
  }
#pragma unroll
  for (int s = 1; s < 4; s <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, s));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, s));
  }
  float z = bf16_down(lo);
  const float range = __fsub_rn(hi, z);
  const unsigned odds = __ballot_sync(0xffffffffu, odd || !isfinite(range));
  float s = bf16_up(__fdiv_rn(range, 15.f));
  uint32_t code[2] = {0u, 0u};
  if ((odds >> (lane & ~3)) & 15u) {
    s = z = __uint_as_float(0x7FC00000u);
  } else if (s > 0.f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float u = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x[i], z), s)), 0.f), 15.f);
      code[i >> 3] |= static_cast<uint32_t>(u) << (4 * (i & 7));
    }
  }
  if (slot == -1) return;
  const int block = slot / p.page, off = slot - block * p.page;
  if (slot < 0 || block >= p.num_blocks) {
    atomicOr(p.status, kDevStatusBadSeqlens);
    return;
  }
  uint8_t* tile = p.cache + kv4_tile_offset<D>(block, off, p.page, p.Hk, h);
  const int r = off & 15;
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

template <int D, bool F32>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const Kv4CacheParams p) {
  using F = Kv4Tile<D>;
  constexpr int kLanes = D / 16;
  const long long id = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const int j = static_cast<int>(id % kLanes);
  const long long row = id / kLanes;
  if (row >= static_cast<long long>(p.T) * p.Hk) return;
  const bool is_v = blockIdx.y != 0;
  const int t = static_cast<int>(row / p.Hk), h = static_cast<int>(row - static_cast<long long>(t) * p.Hk);
  const int slot = p.slots[t];
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.f;
  const int block = slot < 0 ? 0 : slot / p.page, off = slot - block * p.page;
  if (slot < -1 || block >= p.num_blocks) atomicOr(p.status, kDevStatusBadSeqlens);
  if (slot >= 0 && block < p.num_blocks) {
    const uint8_t* tile = p.cache + kv4_tile_offset<D>(block, off, p.page, p.Hk, h);
    const int r = off & 15;
    const int plane = j / (F::kPlaneDims / 16), g = (j / 4) % F::kGroups, c = j & 3;
    uint32_t code[2];
    if (!is_v) {
      const uint2 w = *reinterpret_cast<const uint2*>(tile + plane * F::kPlaneBytes + r * F::kRowBytes +
                                                      c * 8 * F::kGroups + 8 * g);
      code[0] = w.x, code[1] = w.y;
    } else {
      const uint8_t* d = tile + F::kVOff + plane * F::kPlaneBytes + r * F::kRowBytes + 2 * c * 4 * F::kGroups + 4 * g;
      code[0] = *reinterpret_cast<const uint32_t*>(d);
      code[1] = *reinterpret_cast<const uint32_t*>(d + 4 * F::kGroups);
    }
    const uint32_t sz = *reinterpret_cast<const uint32_t*>(tile + (is_v ? F::kVszOff : F::kKszOff) + r * F::kSzRow +
                                                           4 * (j / 4));
    const float s = __uint_as_float(sz << 16), z = __uint_as_float(sz & 0xFFFF0000u);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = fmaf(static_cast<float>((code[i >> 3] >> (4 * (i & 7))) & 15u), s, z);
  }
  const long long at = row * D + 16 * j;
  if constexpr (F32) {
    float4* out = reinterpret_cast<float4*>(static_cast<float*>(is_v ? p.v_out : p.k_out) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  } else {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_v ? p.v_out : p.k_out) + at);
    out[0] = make_uint4(w[0], w[1], w[2], w[3]);
    out[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

dim3 grid_of(const Kv4CacheParams& p, int d) {
  const long long threads = static_cast<long long>(p.T) * p.Hk * (d / 16);
  return dim3(static_cast<unsigned>((threads + kThreads - 1) / kThreads), 2);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4CacheParams& p, int d, cudaStream_t stream) {
  const dim3 grid = grid_of(p, d);
  if (d == 64) kv4_append_kernel<64><<<grid, kThreads, 0, stream>>>(p);
  else if (d == 128) kv4_append_kernel<128><<<grid, kThreads, 0, stream>>>(p);
  else kv4_append_kernel<256><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4CacheParams& p, int d, bool out_f32, cudaStream_t stream) {
  const dim3 grid = grid_of(p, d);
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

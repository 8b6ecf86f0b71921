// Rotary position embedding with several position axes, and its transpose (the backward pass).
//
// Pair i of a row (coordinates i and i + half) turns by the angle whose cosine and sine the caller's
// tables hold at [position of the row on the pair's axis, i].  The rotation is orthogonal, so the
// gradient of x is the same rotation of the gradient of y with the sine negated.  float32, each product
// and the sum rounded separately, so that results do not depend on how the compiler contracts them.
//
// Bound by memory: every element of Q and K is read once and written once; the tables come from L2 (one
// row of `half` cosines and sines per token and axis, for all heads).  A thread keeps the angles of VEC
// pairs in registers and applies them to up to kHeads heads of one token, so each table load serves that
// many heads, and their loads are all in flight together.

#include <cuda_bf16.h>

#include <type_traits>

#include "attn_kernels.h"
#include "kv_kernels.h"

namespace ea {

namespace {

constexpr int kHeads = 4;
constexpr int kThreads = 256;

// VEC values as they lie in memory (kept so until they are used: half the registers of their floats), and as floats
template <typename T, int VEC>
struct Raw {
  static constexpr int kWords = VEC * sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWords == 4) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      w[0] = u.x, w[1] = u.y;
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return __uint_as_float((i & 1) ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
  }
};

template <int VEC>
__device__ __forceinline__ void load_table(const float* p, float (&v)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; i += 4) {
    const float4 u = __ldg(reinterpret_cast<const float4*>(p + i));
    v[i] = u.x, v[i + 1] = u.y, v[i + 2] = u.z, v[i + 3] = u.w;
  }
}
template <int VEC>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&v)[VEC]) {
  uint32_t w[VEC / 2];
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
  if constexpr (VEC == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}

// Work is numbered ((token * chunks + head chunk) * lanes + lane): lanes 0 .. half / VEC - 1 rotate VEC
// pairs each, the lanes behind them copy VEC of the coordinates past 2 * half (none if 2 * half = d).
// I numbers the work: 32 bits wherever it has fewer than 2^31 pieces (three divisions of 64 bits per piece took as
// long as the memory: 54 us for 8,192 tokens of 40 heads of 128).
template <typename TI, typename TO, int VEC, typename I>
__global__ void __launch_bounds__(kThreads, 3) rope_axes_kernel(const RopeParams p) {
  const int rot_lanes = p.half / VEC;
  const int lanes = rot_lanes + (p.d - 2 * p.half) / VEC;
  const int heads = p.H[0] + p.H[1];
  const int chunks = (heads + kHeads - 1) / kHeads;
  const long long tokens = static_cast<long long>(p.B) * p.N;
  const I total = static_cast<I>(tokens) * chunks * lanes;
  const I step = static_cast<I>(gridDim.x) * kThreads;
  for (I id = static_cast<I>(blockIdx.x) * kThreads + threadIdx.x; id < total; id += step) {
    const I rest = id / lanes;
    const int lane = static_cast<int>(id - rest * lanes);
    const I tok = rest / chunks;
    const int h0 = static_cast<int>(rest - tok * chunks) * kHeads;
    const int b = p.B == 1 ? 0 : static_cast<int>(tok / p.N), n = static_cast<int>(tok - static_cast<I>(b) * p.N);
    const bool rot = lane < rot_lanes;
    float c[VEC], s[VEC];
    bool ok[VEC];
    bool all = true;
    if (rot) {
      const int i0 = lane * VEC;
      int ax0 = 0;
      while (ax0 < p.naxes - 1 && i0 >= p.sec_end[ax0]) ++ax0;
      const int pos0 = p.positions[ax0 * tokens + tok];
      if (i0 + VEC <= p.sec_end[ax0]) {  // all VEC pairs turn with one axis
        all = pos0 >= 0 && pos0 < p.n_pos;
        const long long at = static_cast<long long>(all ? pos0 : 0) * p.half + i0;
        load_table<VEC>(p.cos + at, c);
        load_table<VEC>(p.sin + at, s);
#pragma unroll
        for (int i = 0; i < VEC; ++i) ok[i] = all;
      } else {
        int ax = ax0;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          while (ax < p.naxes - 1 && i0 + i >= p.sec_end[ax]) ++ax;
          const int pos = p.positions[ax * tokens + tok];
          ok[i] = pos >= 0 && pos < p.n_pos;
          all = all && ok[i];
          const long long at = static_cast<long long>(ok[i] ? pos : 0) * p.half + i0 + i;
          c[i] = p.cos[at];
          s[i] = p.sin[at];
        }
      }
      if (p.inverse) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[i] = -s[i];
      }
      if (!all) atomicOr(p.status, kDevStatusBadSeqlens);
    }
    // first and second coordinate of the lane's vectors (a copying lane has one)
    const int ca = rot ? lane * VEC : 2 * p.half + (lane - rot_lanes) * VEC;
    const int cb = rot ? p.half + lane * VEC : ca;
    Raw<TI, VEC> a[kHeads], d[kHeads];
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const int h = h0 + j;
      if (h < heads) {
        const int t = h < p.H[0] ? 0 : 1;
        const TI* x = static_cast<const TI*>(p.x[t]) + b * p.xs[t][0] + (t ? h - p.H[0] : h) * p.xs[t][1] + n * p.xs[t][2];
        a[j].load(x + ca);
        if (rot) d[j].load(x + cb);
      }
    }
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const int h = h0 + j;
      if (h < heads) {
        const int t = h < p.H[0] ? 0 : 1;
        TO* y = static_cast<TO*>(p.y[t]) + b * p.ys[t][0] + (t ? h - p.H[0] : h) * p.ys[t][1] + n * p.ys[t][2];
        if (!rot) {
          float u[VEC];
#pragma unroll
          for (int i = 0; i < VEC; ++i) u[i] = a[j].at(i);
          store_vec<VEC>(y + ca, u);
          continue;
        }
        float u[VEC], v[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float xa = a[j].at(i), xb = d[j].at(i);
          u[i] = __fsub_rn(__fmul_rn(xa, c[i]), __fmul_rn(xb, s[i]));
          v[i] = __fadd_rn(__fmul_rn(xb, c[i]), __fmul_rn(xa, s[i]));
        }
        if (all) {
          store_vec<VEC>(y + ca, u);
          store_vec<VEC>(y + cb, v);
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i)
            if (ok[i]) {
              y[ca + i] = static_cast<TO>(u[i]);
              y[cb + i] = static_cast<TO>(v[i]);
            }
        }
      }
    }
  }
}

template <typename TI, typename TO, int VEC>
cudaError_t launch(const RopeParams& p, int num_sms, cudaStream_t stream) {
  const long long lanes = p.half / VEC + (p.d - 2 * p.half) / VEC;
  const long long chunks = (p.H[0] + p.H[1] + kHeads - 1) / kHeads;
  const long long total = static_cast<long long>(p.B) * p.N * chunks * lanes;
  const long long want = (total + kThreads - 1) / kThreads;
  const long long cap = static_cast<long long>(num_sms) * 32;
  const int grid = static_cast<int>(want < cap ? want : cap);
  // below 2^31 pieces plus a round of the grid, the unsigned counter does not wrap
  if (total < (1ll << 31)) rope_axes_kernel<TI, TO, VEC, unsigned><<<grid, kThreads, 0, stream>>>(p);
  else rope_axes_kernel<TI, TO, VEC, unsigned long long><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_axes(const RopeParams& p, bool in_f32, bool out_f32, int num_sms, cudaStream_t stream) {
  // 8 pairs per lane are one 16-byte load of bf16; 4 where half is not a multiple of 8, and for
  // float32, where they are 16 bytes already
  const bool v8 = p.half % 8 == 0 && !in_f32 && !out_f32;
  if (v8) return launch<__nv_bfloat16, __nv_bfloat16, 8>(p, num_sms, stream);
  if (!in_f32 && !out_f32) return launch<__nv_bfloat16, __nv_bfloat16, 4>(p, num_sms, stream);
  if (!in_f32) return launch<__nv_bfloat16, float, 4>(p, num_sms, stream);
  if (!out_f32) return launch<float, __nv_bfloat16, 4>(p, num_sms, stream);
  return launch<float, float, 4>(p, num_sms, stream);
}

}  // namespace ea

// Pieces shared by the two kernels that attend over the 4-bit cache: the requests' lengths, the partial results
// and their join.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_kernels.h"
#include "kv4_format.cuh"
#include "kv_kernels.h"
#include "sm100_ptx.cuh"

namespace ea {

constexpr float kTau = 8.f;        // lazy maximum: p <= 2^kTau
constexpr float kNegBig = -1e30f;  // below any score, and finite
constexpr float kLn2f = 0.6931471805599453f;

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

// A part of a row chunk of one request and key/value head: its units [t0, t1) of `units`.
struct Segment {
  int b, h, chunk;
  int nq, nk, q0;
  int units, t0, t1;
};

// A part of a chunk: [ROWS][D] float O, [ROWS] m, [ROWS] l.  The workspace holds a Meta per block of
// threads, then two parts per block: of the chunk that began before it, and of the one that goes on after it.
template <int D, int ROWS>
__host__ __device__ constexpr int part_floats() { return ROWS * (D + 2); }

struct Meta {
  int tail_valid;  // the last chunk starts here and goes on behind
  int b, h, chunk;
  int head_valid;  // the first chunk started before
  int head_ends;   // ... and ends here
  int rows[2];     // of the tail, of the head (a warp's)
};

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

// Writes dimensions x, x + 1 of O (a0, a1 over sum) of a request's row, and with x = 0 its LSE.
template <int D>
__device__ __forceinline__ void write_row_pair(const Kv4AttnParams& p, int q0, int h, int row, int x, float a0, float a1,
                                               float top, float sum) {
  const int i = row / p.G, hq = h * p.G + row - i * p.G;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + (q0 + i) * p.o_sn + hq * p.o_sh + x) =
      pack_bf16x2(a0 * inv, a1 * inv);
  if (x == 0 && p.lse != nullptr)
    p.lse[static_cast<long long>(hq) * p.total_q + q0 + i] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2f;
}

// Joins the parts of the row chunks that several blocks of threads share: block (i, r) does row r of
// the chunk that starts in block i's span and goes on (and every gridDim.y-th row after it), in the order of
// the spans.  Its threads first look
// together for the span where the chunk ends and for the largest m; then each adds two dimensions over
// its share of the parts, whose loads do not wait for one another.
constexpr int kJoinThreads = 128;

template <int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(const Kv4AttnParams p) {
  constexpr int kShares = kJoinThreads / (D / 2);
  __shared__ int s_last;
  __shared__ float s_top[kJoinThreads / 32];
  __shared__ float s_part[kShares][D / 2][3];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Meta* metas = reinterpret_cast<const Meta*>(p.ws);
  const int first = blockIdx.x, tid = threadIdx.x;
  const Meta mt = metas[first];
  if (!mt.tail_valid) return;
  const SeqLen s = seq_len(p, mt.b);
  const int rows = min(ROWS, s.nq * p.G - mt.chunk * ROWS);
  if (static_cast<int>(blockIdx.y) >= rows) return;
  if (tid == 0) s_last = gridDim.x - 1;
  for (int base = first + 1;; base += kJoinThreads) {
    const int j = base + tid;
    const bool end = j >= static_cast<int>(gridDim.x) || metas[j].head_ends;
    if (__syncthreads_or(end)) {
      if (end) atomicMin(&s_last, j);
      break;
    }
  }
  __syncthreads();
  const int last = s_last;
  const float* parts = reinterpret_cast<const float*>(p.ws + static_cast<size_t>(gridDim.x) * sizeof(Meta));
  auto part = [&](int j) {  // the first span holds the chunk in its second slot, the others in their first
    return parts + (static_cast<size_t>(j) * 2 + (j == first ? 1 : 0)) * part_floats<D, ROWS>();
  };
  for (int r = blockIdx.y; r < rows; r += gridDim.y) {
    float top = kNegBig;
    for (int j = first + tid; j <= last; j += kJoinThreads) top = fmaxf(top, part(j)[ROWS * D + r]);
#pragma unroll
    for (int sft = 16; sft; sft >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sft));
    if ((tid & 31) == 0) s_top[tid >> 5] = top;
    __syncthreads();
    top = s_top[0];
#pragma unroll
    for (int w = 1; w < kJoinThreads / 32; ++w) top = fmaxf(top, s_top[w]);
    const int x = tid % (D / 2), share = tid / (D / 2);
    float a0 = 0.f, a1 = 0.f, sum = 0.f;
#pragma unroll 4
    for (int j = first + share; j <= last; j += kShares) {
      const float* q = part(j);
      const float f = ex2_approx(q[ROWS * D + r] - top);
      const float2 v = *reinterpret_cast<const float2*>(q + r * D + 2 * x);
      a0 += v.x * f;
      a1 += v.y * f;
      sum += q[ROWS * D + ROWS + r] * f;
    }
    if constexpr (kShares > 1) {
      s_part[share][x][0] = a0;
      s_part[share][x][1] = a1;
      s_part[share][x][2] = sum;
      __syncthreads();
      if (share == 0) {
#pragma unroll
        for (int i = 1; i < kShares; ++i) {
          a0 += s_part[i][x][0];
          a1 += s_part[i][x][1];
          sum += s_part[i][x][2];
        }
      }
    }
    if (share == 0) write_row_pair<D>(p, s.q0, mt.h, mt.chunk * ROWS + r, 2 * x, a0, a1, top, sum);
    __syncthreads();
  }
}

template <int D, int ROWS>
unsigned long long part_bytes(unsigned long long blocks) {
  return blocks * (sizeof(Meta) + 2 * sizeof(float) * part_floats<D, ROWS>());
}

// The join, started while the kernel that leaves the parts still runs (it waits for its end).
template <int D, int ROWS>
cudaError_t launch_join(const Kv4AttnParams& p, int blocks, int rows_at_once, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(blocks, rows_at_once);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, ROWS>, p);
}

}  // namespace ea

// What the softmax cross entropy of a linear head needs beside its products: the
// rows' statistics joined over the vocabulary, dx's sums added and rounded, and x twice.
//
//   lse = M + log sum over tiles of s_t e^(m_t - M),  M = max over tiles of m_t
//   loss = lse - (the target's logit), 0 for a row without a target
#include <algorithm>

#include "bf16_tile.h"

namespace fg8 {

namespace {

// Sixteen waves to 64 rows, a lane a row: a wave reads every sixteenth tile's
// pieces, and the waves join in LDS in a fixed order.
__global__ __launch_bounds__(1024) void loss_finish_kernel(BfLoss s, int tiles, int64_t m, float* __restrict__ loss,
                                                           float* __restrict__ lse) {
  __shared__ float2 part[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t r0 = (int64_t)blockIdx.x * 64; r0 < m; r0 += (int64_t)gridDim.x * 64) {
    const int64_t row = r0 + lane;
    int target = -1;
    float picked = 0.f;                  // (read before the pieces are waited for)
    if (wave == 0 && row < m) {
      target = target_of(s, row);
      if (target >= 0) picked = s.picked[row];
    }
    float top = kLowest, sum = 0.f;
    auto add = [&](const float2 (&v)[8]) {
      float t = top;
#pragma unroll
      for (int u = 0; u < 8; ++u) t = fmaxf(t, v[u].x);
      sum *= __builtin_amdgcn_exp2f((top - t) * kLog2e);
#pragma unroll
      for (int u = 0; u < 8; ++u) sum += v[u].y * __builtin_amdgcn_exp2f((v[u].x - t) * kLog2e);
      top = t;
    };
    if (row < m) {
      for (int t0 = wave; t0 < tiles; t0 += 16 * 8) {      // (eight loads before the first is used)
        float2 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = t0 + 16 * u < tiles ? s.pieces[(int64_t)(t0 + 16 * u) * m + row] : make_float2(kLowest, 0.f);
        add(v);
      }
    }
    part[wave][lane] = make_float2(top, sum);
    __syncthreads();
    if (wave == 0 && row < m) {
      top = kLowest;
      sum = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float2 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = part[8 * h + u][lane];
        add(v);
      }
      const float l = logf(sum);
      lse[row] = top + l;
      // (the maximum and the target's logit first: where the target dominates
      // they cancel exactly)
      loss[row] = target < 0 ? 0.f : (top - picked) + l;
    }
    __syncthreads();
  }
}

// (n is a multiple of 8)
__global__ __launch_bounds__(256) void sum_kernel(const float* __restrict__ x, int parts, int64_t n, uint16_t* __restrict__ y) {
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (int64_t)gridDim.x * 2048) {
    v4f a = {0.f, 0.f, 0.f, 0.f}, b = a;
    for (int p = 0; p < parts; ++p) {
      a += *reinterpret_cast<const v4f*>(x + p * n + i);
      b += *reinterpret_cast<const v4f*>(x + p * n + i + 4);
    }
    *reinterpret_cast<uint4*>(y + i) = make_uint4(bf16x2(a[0], a[1]), bf16x2(a[2], a[3]), bf16x2(b[0], b[1]), bf16x2(b[2], b[3]));
  }
}

// x [m][ldx] twice, one under the other (k a multiple of 8), for the two parts of
// dlogits that a float weight gradient takes.  A launch's latency at few rows.
__global__ __launch_bounds__(256) void twice_kernel(const uint16_t* __restrict__ x, int64_t ldx, int64_t m, int64_t k,
                                                    uint16_t* __restrict__ y) {
  const int64_t c = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 8;
  if (c >= k) return;
  for (int64_t r = blockIdx.x; r < m; r += gridDim.x) {
    const uint4 v = *reinterpret_cast<const uint4*>(x + r * ldx + c);
    *reinterpret_cast<uint4*>(y + r * k + c) = v;
    *reinterpret_cast<uint4*>(y + (m + r) * k + c) = v;
  }
}

constexpr int64_t kMostBlocks = 1 << 16;

}  // namespace

hipError_t launch_loss_finish(const BfLoss& s, int64_t tiles, int64_t m, float* loss, float* lse, hipStream_t stream) {
  hipLaunchKernelGGL(loss_finish_kernel, dim3((unsigned)std::min((m + 63) / 64, kMostBlocks)), dim3(1024), 0, stream, s, (int)tiles, m, loss, lse);
  return hipGetLastError();
}

hipError_t launch_sum_bf16(const float* x, int parts, int64_t n, uint16_t* y, hipStream_t stream) {
  hipLaunchKernelGGL(sum_kernel, dim3((unsigned)std::min((n + 2047) / 2048, kMostBlocks)), dim3(256), 0, stream, x, parts, n, y);
  return hipGetLastError();
}

hipError_t launch_twice(const uint16_t* x, int64_t ldx, int64_t m, int64_t k, uint16_t* y, hipStream_t stream) {
  const dim3 grid((unsigned)std::min(m, kMostBlocks), (unsigned)((k + 2047) / 2048));
  hipLaunchKernelGGL(twice_kernel, grid, dim3(256), 0, stream, x, ldx, m, k, y);
  return hipGetLastError();
}

}  // namespace fg8

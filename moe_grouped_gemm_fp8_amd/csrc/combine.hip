// The step after the second expert product: each token's rows weighted and
// summed, and the gradients of that.
//
//   out[t] = sum_j p[t][j] y[token_row[t][j]]  (+ residual[t])
//   dy[token_row[t][j]] = p[t][j] dout[t]
//   dp[t][j] = sum_c dout[t][c] y[token_row[t][j]][c]
//
// A position whose token_row lies outside [0, rows) adds nothing (its dp is
// 0).  HBM bounds both: every row of y is read once.  A wave takes 16-byte
// pieces of a token and has the pieces of up to kAhead of its rows in flight
// together; a token's indices and weights sit in its lanes and are handed out
// with readlane.  8192 tokens x 7168, top-8 of 32: forward with a residual
// 0.212 ms (5.5 TB/s), backward 0.398 ms (5.0 TB/s); in FP32 0.44 and 0.83 ms
// (5.4 and 5.0); a plain copy moves 4.8-4.9.
#include "fg8_device.h"
#include "fg8_internal.h"

namespace fg8 {

namespace {

constexpr int kAhead = 8;   // rows of a token in flight

template <class T>
__device__ __forceinline__ uint4 load16(const T* p) { return *reinterpret_cast<const uint4*>(p); }

template <class T>
__device__ __forceinline__ void store16(T* p, const float* f) {
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  u4 v;
  if constexpr (sizeof(T) == 4)
    v = u4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
  else
    v = u4{bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]), bf16x2(f[6], f[7])};
  __builtin_nontemporal_store(v, reinterpret_cast<u4*>(p));
}

// A wave's item: one span of 64 pieces of one token.
template <class T>
__global__ __launch_bounds__(kCombineThreads) void combine_kernel(
    const T* __restrict__ y, int64_t rows, const int32_t* __restrict__ token_row,
    const float* __restrict__ weights, const T* __restrict__ residual, int64_t tokens, int topk,
    int64_t hidden, int spans, T* __restrict__ out) {
  constexpr int N = RowVec<T>::kElems;
  const int lane = threadIdx.x & 63;
  const int64_t item = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = item / spans, c = ((item - t * spans) * 64 + lane) * N;
  if (t >= tokens) return;
  const bool mine = c < hidden;
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;
  uint4 res = make_uint4(0, 0, 0, 0);
  if (residual && mine) res = load16(residual + t * hidden + c);
  for (int j0 = 0; j0 < topk; j0 += 64) {
    int row = -1;
    float p = 0.f;
    if (j0 + lane < topk) {
      row = token_row[t * topk + j0 + lane];
      p = weights[t * topk + j0 + lane];
      if (row >= rows) row = -1;
    }
    const int nj = min(topk - j0, 64);
    for (int j = 0; j < nj; j += kAhead) {
      uint4 raw[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int r = j + a < nj ? __builtin_amdgcn_readlane(row, j + a) : -1;
        raw[a] = r >= 0 && mine ? load16(y + r * hidden + c) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int r = j + a < nj ? __builtin_amdgcn_readlane(row, j + a) : -1;
        if (r < 0) continue;   // (an infinite weight of a dead position adds nothing)
        const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(p), j + a));
        float f[N];
        RowVec<T>::widen(raw[a], f);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = fmaf(w, f[i], acc[i]);
      }
    }
  }
  if (!mine) return;
  if (residual) {
    float f[N];
    RowVec<T>::widen(res, f);
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] += f[i];
  }
  store16(out + t * hidden + c, acc);
}

// Workgroups [0, tokens): one token each, its pieces dealt to four waves; the
// others clear the rows that hold no token, four rows each.
template <class T>
__global__ __launch_bounds__(kCombineThreads) void combine_backward_kernel(
    const T* __restrict__ dout, const T* __restrict__ y, int64_t rows,
    const int32_t* __restrict__ token_row, const int32_t* __restrict__ row_token,
    const float* __restrict__ weights, int64_t tokens, int topk, int64_t hidden,
    T* __restrict__ dy, float* __restrict__ dweights) {
  constexpr int N = RowVec<T>::kElems;
  __shared__ float part[4][kAhead];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.x;
  if (t >= tokens) {
    const int64_t r = (t - tokens) * 4 + wave;
    if (r >= rows) return;
    const int owner = row_token[r];
    if (owner >= 0 && owner < tokens) return;
    float zero[N];
#pragma unroll
    for (int i = 0; i < N; ++i) zero[i] = 0.f;
    for (int64_t c = (int64_t)lane * N; c < hidden; c += 64 * N) store16(dy + r * hidden + c, zero);
    return;
  }
  for (int j0 = 0; j0 < topk; j0 += kAhead) {
    int row = -1;
    float p = 0.f;
    if (lane < kAhead && j0 + lane < topk) {
      row = token_row[t * topk + j0 + lane];
      p = weights[t * topk + j0 + lane];
      if (row >= rows) row = -1;
    }
    int r[kAhead];
    float w[kAhead], dot[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      r[a] = __builtin_amdgcn_readlane(row, a);
      w[a] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(p), a));
      dot[a] = 0.f;
    }
    for (int64_t c = (int64_t)threadIdx.x * N; c < hidden; c += 256 * N) {
      uint4 raw[kAhead];
      const uint4 rd = load16(dout + t * hidden + c);
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
        raw[a] = r[a] >= 0 ? load16(y + r[a] * hidden + c) : make_uint4(0, 0, 0, 0);
      float d[N];
      RowVec<T>::widen(rd, d);
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        if (r[a] < 0) continue;
        float f[N], o[N];
        RowVec<T>::widen(raw[a], f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          dot[a] = fmaf(d[i], f[i], dot[a]);
          o[i] = w[a] * d[i];
        }
        store16(dy + r[a] * hidden + c, o);
      }
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) dot[a] += __shfl_xor(dot[a], o, 64);
      if (lane == 0) part[wave][a] = dot[a];
    }
    __syncthreads();
    if (threadIdx.x < kAhead && j0 + (int)threadIdx.x < topk) {
      const int a = threadIdx.x;
      dweights[t * topk + j0 + a] = (part[0][a] + part[1][a]) + (part[2][a] + part[3][a]);
    }
    __syncthreads();
  }
}

int combine_spans(bool bf16, int64_t hidden) {
  const int64_t span = 64 * (bf16 ? 8 : 4);
  return (int)((hidden + span - 1) / span);
}

}  // namespace

int64_t combine_workgroups(bool bf16, int64_t tokens, int64_t hidden) {
  return (tokens * combine_spans(bf16, hidden) + 3) / 4;
}
int64_t combine_backward_workgroups(int64_t rows, int64_t tokens) { return tokens + (rows + 3) / 4; }

hipError_t launch_combine(const void* y, bool bf16, int64_t rows, const int32_t* token_row,
                          const float* weights, const void* residual, int64_t tokens, int topk,
                          int64_t hidden, void* out, hipStream_t stream) {
  const int spans = combine_spans(bf16, hidden);
  const dim3 grid((unsigned)combine_workgroups(bf16, tokens, hidden));
  if (bf16)
    hipLaunchKernelGGL(combine_kernel<uint16_t>, grid, dim3(kCombineThreads), 0, stream, (const uint16_t*)y, rows,
                       token_row, weights, (const uint16_t*)residual, tokens, topk, hidden, spans,
                       (uint16_t*)out);
  else
    hipLaunchKernelGGL(combine_kernel<float>, grid, dim3(kCombineThreads), 0, stream, (const float*)y, rows,
                       token_row, weights, (const float*)residual, tokens, topk, hidden, spans,
                       (float*)out);
  return hipGetLastError();
}

hipError_t launch_combine_backward(const void* dout, const void* y, bool bf16, int64_t rows,
                                   const int32_t* token_row, const int32_t* row_token,
                                   const float* weights, int64_t tokens, int topk, int64_t hidden,
                                   void* dy, float* dweights, hipStream_t stream) {
  const dim3 grid((unsigned)combine_backward_workgroups(rows, tokens));
  if (bf16)
    hipLaunchKernelGGL(combine_backward_kernel<uint16_t>, grid, dim3(kCombineThreads), 0, stream,
                       (const uint16_t*)dout, (const uint16_t*)y, rows, token_row, row_token, weights,
                       tokens, topk, hidden, (uint16_t*)dy, dweights);
  else
    hipLaunchKernelGGL(combine_backward_kernel<float>, grid, dim3(kCombineThreads), 0, stream, (const float*)dout,
                       (const float*)y, rows, token_row, row_token, weights, tokens, topk, hidden,
                       (float*)dy, dweights);
  return hipGetLastError();
}

}  // namespace fg8

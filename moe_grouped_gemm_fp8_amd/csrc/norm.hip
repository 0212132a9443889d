// Layer norm over the last axis and its gradient, and the column sums that
// bias and weight gradients need.
//
//   y = (x - mean) * rstd * weight + bias,   rstd = 1 / sqrt(var + eps)
//   g = dy * weight,  h = (x - mean) * rstd
//   dx = rstd * (g - mean(g) - h * mean(g h))
//   dweight = sum over rows of dy h,   dbias = sum over rows of dy
//
// All arithmetic is FP32.  A row is read once (x, and dy) and written once.
// HBM bounds the forward pass of many rows: 32768 x 7168 BF16 0.19-0.20 ms
// (4.7-5.0 TB/s), 16383 x 7168 FP32 0.178 (5.3), rows of odd length the same
// (20000 x 2051 FP32 0.060, 5.5); 16000 x 12000 and 4000 x 32768 BF16 run at 3.8.
// A plain copy moves 4.8-4.9 TB/s here.  The backward pass by size:
//   many rows of up to 8192 columns: HBM.  32768 x 7168 BF16 0.295-0.305 ms (4.6
//     to 4.8 TB/s), 16383 x 7168 FP32 0.27 (5.2), 20000 x 2051 FP32 0.100 (4.9).
//   above 8192 columns: registers.  Both parameters' running sums leave no room
//     for a row ahead, and from there on spill: 16000 x 12000 BF16 0.45 ms and
//     8000 x 16384 FP32 0.615 (2.6 TB/s), 4000 x 32768 BF16 1.3-1.4 (0.6).
//   up to a few thousand rows: the partial sums, 8 bytes a column from every team
//     and read again.  512 x 7168 BF16 22 us, 2048 x 7168 31 (2.8 TB/s), 4096 x
//     7168 44 (4.0); 65536 x 256 38 (2.7), whose sums are added by 8 workgroups.
//
// A team of WAVES waves owns a row at a time and holds it in registers, so the
// variance is taken around the mean (two passes over registers, not the sum of
// squares); a thread owns the same columns of every row its team takes, which
// keeps the weight and, backward, both parameters' running sums in registers
// too.  Teams leave one partial sum each; a second kernel adds them in team
// order, so the result is the same on every call.
#include <type_traits>

#include "fg8_device.h"
#include "fg8_internal.h"

namespace fg8 {

namespace {

// Sixteen bytes of a row: rows need no alignment beyond their element's.
template <class T>
struct Piece {
  static constexpr int N = 16 / sizeof(T);
  // elements c .. c + N - 1, those at or past `cols` zeros
  __device__ static uint4 load(const T* row, int64_t c, int64_t cols) {
    if (c + N <= cols) return whole(row + c);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c + i < cols) {
        if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(row[c + i]);
        else w[i / 2] |= (uint32_t)row[c + i] << (16 * (i & 1));
      }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ static uint4 whole(const T* p) {
    uint4 v;   // (one 16-byte load at any element's address)
    __builtin_memcpy(&v, p, 16);
    return v;
  }
  __device__ static void store(T* row, int64_t c, int64_t cols, const float* f) { store(row, c, c, cols, f); }
  // elements max(c, from) .. of c .. c + N - 1 that lie before `cols`
  __device__ static void store(T* row, int64_t c, int64_t from, int64_t cols, const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(f[i]);
      else w[i] = bf16x2(f[2 * i], f[2 * i + 1]);
    }
    if (c + N <= cols && from <= c) {
      __builtin_memcpy(row + c, w, 16);
      return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c + i < cols && c + i >= from) {
        if constexpr (sizeof(T) == 4) row[c + i] = f[i];
        else row[c + i] = (T)(w[i / 2] >> (16 * (i & 1)));
      }
  }
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Sum over the team of `K` values at once; `at` alternates between the two
// halves of the exchange buffer, so one barrier a call is enough.
template <int WAVES, int K>
__device__ __forceinline__ void team_sum(float (&v)[K], float (*buf)[16][2], int& at, int wave, int lane) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
  if constexpr (WAVES > 1) {
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) buf[at][wave][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) s += buf[at][w][k];
      v[k] = s;
    }
    at ^= 1;
  }
}

// Threads of a workgroup: one team of WAVES waves, or four teams of one wave.
template <int WAVES>
constexpr int threads_of() { return WAVES == 1 ? 256 : 64 * WAVES; }
template <int WAVES>
constexpr int teams_of() { return WAVES == 1 ? 4 : 1; }

// What a thread of a team holds: NV pieces of N columns each.  A row is loaded
// without branches, so that all its loads are in flight together: a piece that
// would cross the row's end starts at the row's last N elements instead, and
// what lies before its own first column (another thread's) is masked to zero.
// (Rows shorter than a piece are loaded by element: TINY.)  LEAN, where a
// lane's registers do not suffice (more than 16 columns a thread; backward,
// teams of sixteen waves, which have 128 a lane): no row ahead in flight, and
// the parameters are read again for every row.
template <class T, int WAVES, int NV, bool TINY, bool BACKWARD>
struct Team {
  static constexpr int N = Piece<T>::N;
  static constexpr bool LEAN = NV * N > 16 || (BACKWARD && WAVES > 8);
  int lane, wave, me, cols;
  int64_t team, teams;
  __device__ Team(int cols_) : cols(cols_) {
    lane = threadIdx.x & 63;
    wave = threadIdx.x >> 6;
    me = WAVES == 1 ? lane : threadIdx.x;
    team = WAVES == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
    teams = (int64_t)gridDim.x * teams_of<WAVES>();
  }
  __device__ int own(int i) const { return (i * 64 * WAVES + me) * N; }              // its own first column
  __device__ int column(int i) const { return TINY ? own(i) : min(own(i), cols - N); }   // where its piece starts
  __device__ bool mine(int i, int j) const { return TINY ? own(i) + j < cols : column(i) + j >= own(i); }
  // are all lanes' pieces i whole?  (the same answer in every lane)
  __device__ bool whole(int i) const { return (i + 1) * 64 * WAVES * N <= cols; }
  __device__ uint4 masked(int i, uint4 v) const {
    if (TINY || whole(i)) return v;
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (N == 4) w[k] = mine(i, k) ? w[k] : 0u;
      else w[k] &= (mine(i, 2 * k) ? 0xffffu : 0u) | (mine(i, 2 * k + 1) ? 0xffff0000u : 0u);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  template <class U>
  __device__ uint4 fetch(const U* row, int c) const {
    return TINY ? Piece<U>::load(row, c, cols) : Piece<U>::whole(row + c);
  }
  __device__ void load(const T* row, uint4 (&raw)[NV]) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) raw[i] = fetch(row, column(i));
  }
  // N parameter values of piece i, FP32 or BF16
  __device__ void parameters(const void* p, bool bf16, int i, float* f) const {
    if (bf16) {
      const uint16_t* q = (const uint16_t*)p;
      if constexpr (N == 8) {
        RowVec<uint16_t>::widen(fetch(q, column(i)), f);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
          f[j] = !TINY || column(i) + j < cols ? __uint_as_float((uint32_t)q[column(i) + j] << 16) : 0.f;
      }
    } else {
#pragma unroll
      for (int h = 0; h < N; h += 4) {
        if (TINY && own(i) + h >= cols) f[h] = f[h + 1] = f[h + 2] = f[h + 3] = 0.f;
        else RowVec<float>::widen(fetch((const float*)p, column(i) + h), f + h);
      }
    }
  }
};

template <class T, int WAVES, int NV, bool TINY>
__global__ __launch_bounds__(threads_of<WAVES>()) void norm_kernel(
    const T* __restrict__ x, int64_t ldx, const void* __restrict__ weight,
    const void* __restrict__ bias, bool w_bf16, float eps, int64_t rows, int cols,
    T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd) {
  typedef Team<T, WAVES, NV, TINY, false> Me;
  constexpr int N = Me::N;
  __shared__ float buf[2][16][2];
  const Me t(cols);
  int at = 0;
  uint4 raw[NV], ahead[NV];
  float w[NV][N], b[NV][N];
  auto parameters = [&](int i) {
    t.parameters(weight, w_bf16, i, w[i]);
    if (bias) {
      t.parameters(bias, w_bf16, i, b[i]);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) b[i][j] = 0.f;
    }
  };
  if (t.team < rows) t.load(x + t.team * ldx, raw);
  if constexpr (!Me::LEAN) {
#pragma unroll
    for (int i = 0; i < NV; ++i) parameters(i);
  }
  for (int64_t r = t.team; r < rows; r += t.teams) {
    const bool more = r + t.teams < rows;
    if (!Me::LEAN && more) t.load(x + (r + t.teams) * ldx, ahead);   // in flight under this row's sums
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[N];
      RowVec<T>::widen(t.masked(i, raw[i]), f);
#pragma unroll
      for (int j = 0; j < N; ++j) s[0] += f[j];
    }
    team_sum<WAVES, 1>(s, buf, at, t.wave, t.lane);
    const float m = s[0] / (float)cols;   // (a row of one value has that mean)
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[N];
      RowVec<T>::widen(raw[i], f);
      if (t.whole(i)) {
#pragma unroll
        for (int j = 0; j < N; ++j) q[0] = fmaf(f[j] - m, f[j] - m, q[0]);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float d = t.mine(i, j) ? f[j] - m : 0.f;
          q[0] = fmaf(d, d, q[0]);
        }
      }
    }
    team_sum<WAVES, 1>(q, buf, at, t.wave, t.lane);
    const float rs = 1.f / sqrtf(q[0] / (float)cols + eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[N], o[N];
      if constexpr (Me::LEAN) parameters(i);
      RowVec<T>::widen(raw[i], f);
#pragma unroll
      for (int j = 0; j < N; ++j) o[j] = fmaf((f[j] - m) * rs, w[i][j], b[i][j]);
      if (t.own(i) < cols) Piece<T>::store(y + r * cols, t.column(i), t.own(i), cols, o);
    }
    if (t.me == 0) {
      mean[r] = m;
      rstd[r] = rs;
    }
    if (Me::LEAN && more) t.load(x + (r + t.teams) * ldx, raw);
    if constexpr (!Me::LEAN) {
#pragma unroll
      for (int i = 0; i < NV; ++i) raw[i] = ahead[i];
    }
  }
}

template <class T, int WAVES, int NV, bool TINY>
__global__ __launch_bounds__(threads_of<WAVES>()) void norm_backward_kernel(
    const T* __restrict__ dy, int64_t lddy, const T* __restrict__ x, int64_t ldx,
    const void* __restrict__ weight, bool w_bf16, const float* __restrict__ mean,
    const float* __restrict__ rstd, int64_t rows, int cols, T* __restrict__ dx,
    float* __restrict__ partial) {
  typedef Team<T, WAVES, NV, TINY, true> Me;
  constexpr int N = Me::N;
  __shared__ float buf[2][16][2];
  const Me t(cols);
  const float inv = 1.f / (float)cols;
  int at = 0;
  uint4 rx[NV], rd[NV], nx[NV], nd[NV];
  float w[NV][N], dw[NV][N], db[NV][N], m = 0.f, rs = 0.f, nm = 0.f, nrs = 0.f;
  auto fetch = [&](int64_t r, uint4 (&fx)[NV], uint4 (&fd)[NV], float& fm, float& fr) {
    t.load(x + r * ldx, fx);
    t.load(dy + r * lddy, fd);
    fm = mean[r];
    fr = rstd[r];
  };
  if (t.team < rows) fetch(t.team, rx, rd, m, rs);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if constexpr (!Me::LEAN) t.parameters(weight, w_bf16, i, w[i]);
#pragma unroll
    for (int j = 0; j < N; ++j) dw[i][j] = db[i][j] = 0.f;
  }
  // h, and g times the weight, of piece i; what is not this thread's is zero
  // in g (and may be anything in h, whose columns nobody stores from here)
  float h[NV][N], g[NV][N];
  auto widen = [&](int i) {
    RowVec<T>::widen(rx[i], h[i]);
    RowVec<T>::widen(t.masked(i, rd[i]), g[i]);
    if constexpr (Me::LEAN) t.parameters(weight, w_bf16, i, w[i]);
#pragma unroll
    for (int j = 0; j < N; ++j) h[i][j] = (h[i][j] - m) * rs;
  };
  for (int64_t r = t.team; r < rows; r += t.teams) {
    const bool more = r + t.teams < rows;
    if (!Me::LEAN && more) fetch(r + t.teams, nx, nd, nm, nrs);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      widen(i);
      if (!t.whole(i)) {     // (another thread's column may hold NaN: it must not meet these sums)
#pragma unroll
        for (int j = 0; j < N; ++j) h[i][j] = t.mine(i, j) ? h[i][j] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < N; ++j) {
        dw[i][j] = fmaf(g[i][j], h[i][j], dw[i][j]);
        db[i][j] += g[i][j];
        g[i][j] *= w[i][j];
        s[0] += g[i][j];
        s[1] = fmaf(g[i][j], h[i][j], s[1]);
      }
    }
    team_sum<WAVES, 2>(s, buf, at, t.wave, t.lane);
    const float c1 = s[0] * inv, c2 = s[1] * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[N];
      if constexpr (Me::LEAN) {          // again from the packed row: half the registers
        widen(i);
#pragma unroll
        for (int j = 0; j < N; ++j) g[i][j] *= w[i][j];
      }
#pragma unroll
      for (int j = 0; j < N; ++j) o[j] = rs * (g[i][j] - c1 - h[i][j] * c2);
      if (t.own(i) < cols) Piece<T>::store(dx + r * cols, t.column(i), t.own(i), cols, o);
    }
    if (Me::LEAN && more) fetch(r + t.teams, rx, rd, m, rs);
    if constexpr (!Me::LEAN) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        rx[i] = nx[i];
        rd[i] = nd[i];
      }
      m = nm;
      rs = nrs;
    }
  }
  float* sums = partial + t.team * 2 * cols;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      const int c = t.column(i) + j;
      if (t.own(i) < cols) {
        Piece<float>::store(sums, c, t.own(i), cols, dw[i] + j);
        Piece<float>::store(sums + cols, c, t.own(i), cols, db[i] + j);
      }
    }
}

// Column sums of partial [parts][cols]: each column's parts are added in a
// fixed order (16 waves take every sixteenth, then meet in LDS).  Columns from
// `split` on go to the second output.
__global__ __launch_bounds__(1024) void column_sum_kernel(const float* __restrict__ partial,
                                                          int parts, int64_t cols, int64_t split,
                                                          float* __restrict__ out,
                                                          float* __restrict__ out2) {
  __shared__ float buf[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int p = wave; p < parts; p += 16) s += partial[p * cols + c];
  }
  buf[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < cols) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) t += buf[k][lane];
    (c < split ? out + c : out2 + (c - split))[0] = t;
  }
}

// The team shape for a row length: waves a row and 16-byte pieces a thread.
// Sixteen columns a thread are the rule (registers for a row ahead and,
// backward, both running sums); the longest rows take 32.  (Backward, 16000 x
// 12000 BF16: 0.45 ms in eight waves of 32 columns, 0.76 in sixteen of 16; FP32
// 8000 x 16384 0.79 and 0.62.)
template <class T, bool BACKWARD, class F>
hipError_t with_shape(int64_t cols, F f) {
  constexpr int P = sizeof(T) == 4 ? 2 : 1;        // pieces of eight columns
  constexpr std::integral_constant<int, P> p1{};
  constexpr std::integral_constant<int, 2 * P> p2{};
  constexpr std::integral_constant<int, 4 * P> p4{};
  constexpr std::integral_constant<int, 1> w1{};
  constexpr std::integral_constant<int, 4> w4{};
  constexpr std::integral_constant<int, 8> w8{};
  constexpr std::integral_constant<int, 16> w16{};
  if (cols < Piece<T>::N) return f(w1, p1, std::true_type{});
  if (cols <= 512) return f(w1, p1, std::false_type{});
  if (cols <= 1024) return f(w1, p2, std::false_type{});
  if (cols <= 2048) return f(w4, p1, std::false_type{});
  if (cols <= 4096) return f(w4, p2, std::false_type{});
  if (cols <= 8192) return f(w8, p2, std::false_type{});
  if constexpr (BACKWARD && sizeof(T) == 2) {
    if (cols <= 16384) return f(w8, p4, std::false_type{});
  }
  if (cols <= 16384) return f(w16, p2, std::false_type{});
  return f(w16, p4, std::false_type{});
}

// Workgroups: enough for two or more a SIMD, and no more than there are rows.
int64_t groups_of(int waves, int64_t rows, int cus) {
  const int64_t most = (int64_t)cus * (waves <= 4 ? 4 : waves == 8 ? 2 : 1);
  const int64_t need = waves == 1 ? (rows + 3) / 4 : rows;
  return need < most ? need : most;
}

}  // namespace

namespace {

template <class T>
int64_t teams_as(int64_t rows, int64_t cols, int cus) {
  int64_t teams = 0;
  (void)with_shape<T, true>(cols, [&](auto waves, auto, auto) {
    teams = groups_of(waves, rows, cus) * teams_of<decltype(waves)::value>();
    return hipSuccess;
  });
  return teams;
}

template <class T>
hipError_t norm_as(const void* x, int64_t ldx, const void* weight, const void* bias, bool w_bf16,
                   float eps, int64_t rows, int64_t cols, void* y, float* mean, float* rstd, int cus,
                   hipStream_t stream) {
  return with_shape<T, false>(cols, [&](auto waves, auto nv, auto tiny) {
    constexpr int W = decltype(waves)::value, NV = decltype(nv)::value;
    hipLaunchKernelGGL((norm_kernel<T, W, NV, decltype(tiny)::value>), dim3((unsigned)groups_of(W, rows, cus)),
                       dim3(threads_of<W>()), 0, stream, (const T*)x, ldx, weight, bias, w_bf16, eps,
                       rows, (int)cols, (T*)y, mean, rstd);
    return hipGetLastError();
  });
}

template <class T>
hipError_t norm_backward_as(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                            const void* weight, bool w_bf16, const float* mean, const float* rstd,
                            int64_t rows, int64_t cols, void* dx, float* partial, int cus,
                            hipStream_t stream) {
  return with_shape<T, true>(cols, [&](auto waves, auto nv, auto tiny) {
    constexpr int W = decltype(waves)::value, NV = decltype(nv)::value;
    hipLaunchKernelGGL((norm_backward_kernel<T, W, NV, decltype(tiny)::value>), dim3((unsigned)groups_of(W, rows, cus)),
                       dim3(threads_of<W>()), 0, stream, (const T*)dy, lddy, (const T*)x, ldx, weight,
                       w_bf16, mean, rstd, rows, (int)cols, (T*)dx, partial);
    return hipGetLastError();
  });
}

}  // namespace

int64_t layer_norm_teams(int64_t rows, int64_t cols, bool bf16, int cus) {
  return bf16 ? teams_as<uint16_t>(rows, cols, cus) : teams_as<float>(rows, cols, cus);
}

hipError_t launch_layer_norm(const void* x, int64_t ldx, bool bf16, const void* weight,
                             const void* bias, bool w_bf16, float eps, int64_t rows, int64_t cols,
                             void* y, float* mean, float* rstd, int cus, hipStream_t stream) {
  return bf16 ? norm_as<uint16_t>(x, ldx, weight, bias, w_bf16, eps, rows, cols, y, mean, rstd, cus, stream)
              : norm_as<float>(x, ldx, weight, bias, w_bf16, eps, rows, cols, y, mean, rstd, cus, stream);
}

hipError_t launch_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                      bool bf16, const void* weight, bool w_bf16,
                                      const float* mean, const float* rstd, int64_t rows,
                                      int64_t cols, void* dx, float* dweight, float* dbias,
                                      float* partial, int cus, hipStream_t stream) {
  const int64_t teams = rows > 0 ? layer_norm_teams(rows, cols, bf16, cus) : 0;
  if (rows > 0) {
    const hipError_t e =
        bf16 ? norm_backward_as<uint16_t>(dy, lddy, x, ldx, weight, w_bf16, mean, rstd, rows, cols, dx, partial, cus, stream)
             : norm_backward_as<float>(dy, lddy, x, ldx, weight, w_bf16, mean, rstd, rows, cols, dx, partial, cus, stream);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((2 * cols + 63) / 64)), dim3(1024), 0, stream, partial,
                     (int)teams, 2 * cols, cols, dweight, dbias);
  return hipGetLastError();
}

// ------------------------------------------- the activation's backward pass
namespace {

// dy act'(z).  Under ReLU nothing passes where z <= 0, an infinite dy either.
__device__ __forceinline__ float act_gradient(int act, float z, float dy) {
  if (act == kActRelu) return z > 0.f ? dy : (z != z ? z : 0.f);
  if (act == kActSilu) {
    const float p = 1.f / (1.f + __expf(-z));
    return dy * (p * (1.f + z * (1.f - p)));
  }
  if (act == kActGelu) {
    float bell;
    const float cdf = normal_cdf(z, &bell);
    return dy * fmaf(z, bell * 0.39894228040143268f, cdf);
  }
  return dy;
}

// What rounding d to BF16 leaves (exact in FP32); 0 beside an infinity or NaN.
__device__ __forceinline__ float bf16_rest(float d) {
  const uint32_t hi = bf16x2(d, 0.f) << 16;
  return (hi & 0x7f800000u) == 0x7f800000u ? 0.f : d - __uint_as_float(hi);
}

constexpr int kActCols = 512;   // columns of a workgroup: eight a lane

// Bound by HBM: dy and z read, dz written once (4096 x 7168 0.036 ms, 4.9 TB/s).
// Workgroup (column block, row chunk): its four waves take the chunk's rows in
// turn and meet in LDS for the column sums, taken before dz is rounded.  REST:
// what that rounding left, in dz's place (an instance of its own: as a run-time
// choice it cost every dz 20 us of these 36).
template <bool REST>
__global__ __launch_bounds__(256) void act_backward_kernel(
    const uint16_t* __restrict__ dy, int64_t lddy, const uint16_t* __restrict__ z, int64_t ldzin,
    int act, int64_t m, int64_t n, int64_t per, uint16_t* __restrict__ dz, int64_t ldz,
    float* __restrict__ partial) {
  __shared__ float buf[4][kActCols];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * kActCols + lane * 8;
  const int64_t r1 = min((int64_t)(blockIdx.y + 1) * per, m);
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (c < n) {
#pragma unroll 4
    for (int64_t r = blockIdx.y * per + wave; r < r1; r += 4) {
      float d[8];
      RowVec<uint16_t>::widen(Piece<uint16_t>::load(dy + r * lddy, c, n), d);
      if (act != kActNone) {
        float v[8];
        RowVec<uint16_t>::widen(Piece<uint16_t>::load(z + r * ldzin, c, n), v);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = act_gradient(act, v[i], d[i]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // (a slope of NaN past the last column would not reach dz's padding)
        if (c + i >= n) d[i] = 0.f;
        s[i] += d[i];
        if constexpr (REST) d[i] = bf16_rest(d[i]);
      }
      if (dz) Piece<uint16_t>::store(dz + r * ldz, c, ldz, d);
    }
  }
  if (!partial) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) buf[wave][lane * 8 + i] = s[i];
  __syncthreads();
  for (int i = threadIdx.x; i < kActCols; i += 256) {
    const int64_t col = (int64_t)blockIdx.x * kActCols + i;
    if (col < n) partial[blockIdx.y * n + col] = (buf[0][i] + buf[1][i]) + (buf[2][i] + buf[3][i]);
  }
}

}  // namespace

int act_backward_chunks(int64_t m, int64_t n) {
  // about 2048 workgroups, of 16 rows at least
  const int64_t blocks = (n + kActCols - 1) / kActCols;
  int64_t chunks = (2048 + blocks - 1) / blocks;
  if (chunks > (m + 15) / 16) chunks = (m + 15) / 16;
  return (int)(chunks < 1 ? 1 : chunks);
}

hipError_t launch_act_backward(const uint16_t* dy, int64_t lddy, const uint16_t* z, int64_t ldzin,
                               int act, int64_t m, int64_t n, bool rest, uint16_t* dz, int64_t ldz,
                               float* partial, float* dbias, hipStream_t stream) {
  const int chunks = act_backward_chunks(m, n);
  const int64_t per = (m + chunks - 1) / chunks;
  hipLaunchKernelGGL(rest ? act_backward_kernel<true> : act_backward_kernel<false>,
                     dim3((unsigned)((n + kActCols - 1) / kActCols), (unsigned)chunks), dim3(256), 0, stream, dy,
                     lddy, z, ldzin, act, m, n, per, dz, ldz, dbias ? partial : nullptr);
  if (dbias)
    hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((n + 63) / 64)), dim3(1024), 0, stream,
                       partial, chunks, n, n, dbias, dbias);
  return hipGetLastError();
}

}  // namespace fg8

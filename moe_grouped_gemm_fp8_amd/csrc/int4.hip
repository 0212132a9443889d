// Weights in 4 bits with group scales: quantize, dequantize, and products with
// few rows of BF16, dense or over ragged row runs.
//
//   s = fl32(amax / 7) of GROUP consecutive k of a row (1 where that is 0),
//   rounded to the scales' type;  code = rne(fl32(w / s)) + 8;  value (code - 8) s
//   codes [n][k / 2], element 2 j in the low half of byte j; scales [k / GROUP][n]
//
//   D[m][n] = sum over groups of s[group][n] * sum over its k of (code - 8) x[m][k]
//
// The product reads half a byte a weight and little else: it is bound by HBM,
// and where few weights are read by the launch and one round trip.
#include "bf16_tile.h"

namespace fg8 {

namespace {

// ------------------------------------------------------- few-row products
// A workgroup owns 16 TM rows and 16 TN weight rows; its waves take chunks of
// 128 k in turn and load both operands straight into registers, the next chunk
// ahead of the one being multiplied; their sums meet in LDS at the end.
//
// A lane loads 16 bytes of codes, 32 k of one weight row; four swaps between the
// four groups of sixteen lanes turn that into the layout of four MFMAs of 32 k
// each (lane i + 16 g: row i, k = 8 g .. 8 g + 7), so a group of 32 k or more is
// whole MFMAs.  A code goes into the upper four mantissa bits of a BF16 whose
// exponent is 16's: 16 + code, one shift and one bit operation for two weights.
// Pairs come out as k, k + 4 of a lane's eight; x's pairs are put in that order.
// The 24 that every weight is too large is taken off with an MFMA against a
// constant -24, once for all the tiles that share x: the group's sum then starts
// from -24 sum(x).  Every value and product is exact; what the detour adds is
// FP32 rounding of partial sums at the size of 24 |x| for 8 |x|.
struct Int4Problem {
  BfProblem p;             // a: x; N: weight rows; d, epilogue, runs
  const uint8_t* codes;
  const void* scales;
};

template <bool BF16>
__device__ __forceinline__ v4i load_scales(const void* s, int64_t at, int left, bool four) {
  // four: rows of scales are whole fours of columns
  v4i v = {0, 0, 0, 0};
  if constexpr (BF16) {
    const uint16_t* q = (const uint16_t*)s + at;
    if (four) {
      if (left > 0) {
        const uint2 u = *reinterpret_cast<const uint2*>(q);
        v[0] = (int)u.x;
        v[1] = (int)u.y;
      }
    } else {
      uint32_t e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = i < left ? q[i] : 0;
      v[0] = (int)(e[0] | e[1] << 16);
      v[1] = (int)(e[2] | e[3] << 16);
    }
  } else {
    const int* q = (const int*)s + at;
    if (four) {
      if (left > 0) v = *reinterpret_cast<const v4i*>(q);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) v[i] = q[i];
    }
  }
  return v;
}
template <bool BF16>
__device__ __forceinline__ v4f scale_values(v4i v) {
  if constexpr (BF16)
    return v4f{__uint_as_float((uint32_t)v[0] << 16), __uint_as_float((uint32_t)v[0] & 0xffff0000u),
               __uint_as_float((uint32_t)v[1] << 16), __uint_as_float((uint32_t)v[1] & 0xffff0000u)};
  else
    return __builtin_bit_cast(v4f, v);
}

// Word 4 g + j of sixteen, held by lane group g as its word j, to word 4 j + g.
__device__ __forceinline__ void transpose_words(v4i& w) {
  typedef unsigned u2 __attribute__((ext_vector_type(2)));
  const u2 a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  const u2 b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  const u2 lo = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const u2 hi = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  w = v4i{(int)lo[0], (int)lo[1], (int)hi[0], (int)hi[1]};
}

// Eight codes as BF16 16 + code: elements 0, 4, 1, 5, 2, 6, 3, 7.
__device__ __forceinline__ v8bf codes_plus_16(uint32_t w) {
  constexpr uint32_t kCode = 0x00780078u, k16 = 0x41804180u;
  const v4i v = {(int)((w << 3 & kCode) | k16), (int)((w >> 1 & kCode) | k16), (int)((w >> 5 & kCode) | k16),
                 (int)((w >> 9 & kCode) | k16)};
  return __builtin_bit_cast(v8bf, v);
}
// x's elements in that order
__device__ __forceinline__ v8bf paired(v4i x) {
  const v4i v = {(int)__builtin_amdgcn_perm(x[2], x[0], 0x05040100u), (int)__builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
                 (int)__builtin_amdgcn_perm(x[3], x[1], 0x05040100u), (int)__builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
  return __builtin_bit_cast(v8bf, v);
}

template <int TM, int TN, int GROUP, bool SBF16>
__global__ __launch_bounds__(512, 2) void int4_kernel(Int4Problem q) {
  constexpr int NG = 128 / GROUP, GJ = GROUP / 32;      // groups of a chunk, MFMAs of a group
  __shared__ v4f sums[8][TM * TN][64];
  const BfProblem& p = q.p;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int waves = blockDim.x >> 6, i = lane & 15, g = lane >> 4;
  BfUnit w;
  if (!(p.mode == kBfRowRuns ? find_unit<16 * TM, 16 * TN, kBfRowRuns>(p, lane, w)
                             : find_unit<16 * TM, 16 * TN, kBfDense>(p, lane, w)))
    return;
  const int N = p.N, K = p.K, half = N / 2;
  const int64_t expert = max(w.g, 0);
  const int64_t row_bytes = K / 2, per_group = N;
  const uint8_t* codes = q.codes + expert * N * row_bytes;
  const int64_t scales0 = expert * per_group * (K / GROUP);

  // weight row that tile t starts at (gated: the first half of the tiles are
  // gate rows, the others the up rows of the same columns)
  auto row_of = [&](int t) {
    if (p.kind != kKindGated) return w.n0 + 16 * t;
    return t < TN / 2 ? w.n0 / 2 + 16 * t : half + w.n0 / 2 + 16 * (t - TN / 2);
  };
  __amdgpu_buffer_rsrc_t wr[TN];
  int col[TN], left[TN];             // this lane's four columns of scales, and how many there are from them on
#pragma unroll
  for (int t = 0; t < TN; ++t) {
    const int r = uniform(row_of(t));
    const int64_t bytes = r < N ? (N - r) * row_bytes : 0;
    wr[t] = buffer_rsrc(uniform((const void*)(codes + (r < N ? r : 0) * row_bytes)),
                        (uint32_t)(bytes > 0x7fffffff ? 0x7fffffff : bytes));
    col[t] = r + 4 * g;
    left[t] = N - col[t];
  }
  const bool four = N % 4 == 0;
  const uint32_t wo = (uint32_t)(i * (int)row_bytes + 16 * g);
  const __amdgpu_buffer_rsrc_t xr = buffer_rsrc(uniform((const void*)(p.a + w.m0 * p.lda)), 0x7fffffff);
  uint32_t xo[TM];
#pragma unroll
  for (int m = 0; m < TM; ++m)
    xo[m] = 16 * m + i < w.rows ? (uint32_t)((16 * m + i) * (int)p.lda + 8 * g) * 2 : kNowhere;

  struct Batch {
    v4i w[TN], x[TM][4], s[TN][NG];
  };
  auto fetch = [&](Batch& f, int c) {
    const int rem = uniform(w.ks - c * 128);      // k from this chunk on, a multiple of 32 (0 or less: no chunk)
    const uint32_t at = 32 * g < rem ? wo : kNowhere;
#pragma unroll
    for (int t = 0; t < TN; ++t)
      f.w[t] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(wr[t], at, uniform(c * 64), kStream));
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        f.x[m][j] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(xr, 32 * j < rem ? xo[m] : kNowhere,
                                                                                  uniform(c * 256 + 64 * j), 0));
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
      for (int e = 0; e < NG; ++e)
        f.s[t][e] = load_scales<SBF16>(q.scales, scales0 + (int64_t)(c * NG + e) * per_group + col[t],
                                       e * GROUP < rem ? left[t] : 0, four);
  };

  v4f acc[TM][TN];
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int t = 0; t < TN; ++t) acc[m][t] = v4f{0.f, 0.f, 0.f, 0.f};
  const v8bf minus24 = __builtin_bit_cast(v8bf, v4i{(int)0xC1C0C1C0u, (int)0xC1C0C1C0u, (int)0xC1C0C1C0u, (int)0xC1C0C1C0u});
  auto multiply = [&](Batch& f) {
#pragma unroll
    for (int t = 0; t < TN; ++t) transpose_words(f.w[t]);
#pragma unroll
    for (int e = 0; e < NG; ++e) {
      v8bf x[TM][GJ];
      v4f start[TM], part[TM][TN];
#pragma unroll
      for (int m = 0; m < TM; ++m) {
        start[m] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < GJ; ++j) {
          x[m][j] = paired(f.x[m][e * GJ + j]);
          start[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(minus24, x[m][j], start[m], 0, 0, 0);
        }
      }
#pragma unroll
      for (int j = 0; j < GJ; ++j)
#pragma unroll
        for (int t = 0; t < TN; ++t) {
          const v8bf v = codes_plus_16((uint32_t)f.w[t][e * GJ + j]);
#pragma unroll
          for (int m = 0; m < TM; ++m)
            part[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, x[m][j], j ? part[m][t] : start[m], 0, 0, 0);
        }
#pragma unroll
      for (int t = 0; t < TN; ++t) {
        const v4f s = scale_values<SBF16>(f.s[t][e]);
#pragma unroll
        for (int m = 0; m < TM; ++m)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[m][t][v] = fmaf(s[v], part[m][t][v], acc[m][t][v]);
      }
    }
  };
  const int chunks = (w.ks + 127) / 128;
  if (wave < chunks) {
    Batch f0, f1;
    fetch(f0, wave);
    for (int c = wave; c < chunks; c += 2 * waves) {
      fetch(f1, c + waves);
      multiply(f0);
      if (c + waves >= chunks) break;
      fetch(f0, c + 2 * waves);
      multiply(f1);
    }
  }

#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int t = 0; t < TN; ++t) sums[wave][m * TN + t][lane] = acc[m][t];
  __syncthreads();
  auto sum_of = [&](int at) {
    v4f v = sums[0][at][lane];
    for (int u = 1; u < waves; ++u) v += sums[u][at][lane];
    return v;
  };
  if (p.kind == kKindGated) {
    if constexpr (TN > 1) {
      for (int u = wave; u < TM * (TN / 2); u += waves) {
        const int m = u / (TN / 2), t = u % (TN / 2);
        v4f gate[1] = {sum_of(m * TN + t)}, up[1] = {sum_of(m * TN + TN / 2 + t)};
        GatedOut<1>(p, w, 16 * TM, 16 * TN, 32 * t, nullptr, lane).rows16(16 * m, gate, up);
      }
    }
  } else {
    const BfOut out(p, w.g);
    for (int u = wave; u < TM * TN; u += waves) {
      const int r = 16 * (u / TN) + i;
      const v4f v = sum_of(u);
      if (r < w.rows) out.four(w.m0 + r, w.n0 + 16 * (u % TN) + 4 * g, v);
    }
  }
}

template <int TM, int TN>
hipError_t start(const Int4Problem& q, int group, bool sbf16, unsigned grid, int threads, hipStream_t stream) {
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(threads), 0, stream, q);
    return hipGetLastError();
  };
  if (group == 32) return sbf16 ? go(int4_kernel<TM, TN, 32, true>) : go(int4_kernel<TM, TN, 32, false>);
  if (group == 64) return sbf16 ? go(int4_kernel<TM, TN, 64, true>) : go(int4_kernel<TM, TN, 64, false>);
  return sbf16 ? go(int4_kernel<TM, TN, 128, true>) : go(int4_kernel<TM, TN, 128, false>);
}

}  // namespace

Int4Tile int4_tile(const BfProblem& p, int cus) {
  Int4Tile t{};
  const int64_t rows = p.mode == kBfRowRuns ? (p.M + p.groups - 1) / p.groups : p.M;
  t.tm = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  t.tn = 2;
  if (p.kind != kKindGated && t.tm == 1 && p.mode == kBfDense) {
    if ((int64_t)p.N < 16 * 2 * cus) t.tn = 1;
    else if ((int64_t)p.N >= 16 * 4 * cus) t.tn = 4;
  }
  t.threads = p.K >= 16 * 128 ? 512 : 256;
  const int64_t bm = 16 * t.tm, bn = 16 * t.tn;
  t.units = ((p.M + bm - 1) / bm + (p.mode == kBfRowRuns ? p.groups + 1 : 0)) * ((p.N + bn - 1) / bn);
  return t;
}

hipError_t launch_int4(const BfProblem& p, const Int4Tile& t, const uint8_t* codes, const void* scales, bool scales_bf16,
                       int group, hipStream_t stream) {
  const Int4Problem q{p, codes, scales};
  const unsigned grid = (unsigned)((t.units + 7) / 8 * 8);
  if (t.tm == 1 && t.tn == 1) return start<1, 1>(q, group, scales_bf16, grid, t.threads, stream);
  if (t.tm == 1 && t.tn == 2) return start<1, 2>(q, group, scales_bf16, grid, t.threads, stream);
  if (t.tm == 1) return start<1, 4>(q, group, scales_bf16, grid, t.threads, stream);
  if (t.tm == 2) return start<2, 2>(q, group, scales_bf16, grid, t.threads, stream);
  return start<4, 2>(q, group, scales_bf16, grid, t.threads, stream);
}

// ------------------------------------------------- quantize and dequantize
namespace {

// A workgroup owns 32 rows x 512 k: a wave reads 512 k of a row, eight a lane,
// eight rows in all.  Scales lie [group][row] in memory and cross in LDS, so that
// they are written and read as runs of 32 rows.
constexpr int kQuantRows = 32, kQuantCols = 512;

template <class T>
__device__ __forceinline__ void load_eight(const T* p, float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    RowVec<T>::widen(load_nt16(p), f);
  } else {
    RowVec<T>::widen(load_nt16(p), f);
    RowVec<T>::widen(load_nt16(p + 4), f + 4);
  }
}

template <class T, class S, int GROUP>
__global__ __launch_bounds__(256) void int4_quantize_kernel(const T* __restrict__ w, int64_t rows, int64_t cols,
                                                            uint8_t* __restrict__ q, S* __restrict__ scales) {
  constexpr int G = kQuantCols / GROUP, LANES = GROUP / 8;     // groups of a row's piece, lanes of a group
  __shared__ float kept[G][kQuantRows + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t r0 = (int64_t)blockIdx.x * kQuantRows, c0 = (int64_t)blockIdx.y * kQuantCols, c = c0 + lane * 8;
  w += (int64_t)blockIdx.z * rows * cols;
  q += (int64_t)blockIdx.z * rows * (cols / 2);
  scales += (int64_t)blockIdx.z * rows * (cols / GROUP);
  constexpr int PER = kQuantRows / 4;
  float f[PER][8];
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int64_t r = r0 + wave * PER + u;
    if (r < rows && c < cols) {
      load_eight(w + r * cols + c, f[u]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[u][e] = 0.f;
    }
  }
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    // the largest absolute value by its bits: a NaN or infinity wins, and the
    // scale, and with it the whole group, is NaN
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(f[u][e]) & 0x7fffffffu);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o, 64));
    float s = __fdiv_rn(__uint_as_float(top >= 0x7f800000u ? 0x7fc00000u : top), 7.f);
    if constexpr (sizeof(S) == 2) s = __uint_as_float(bf16x2(s, 0.f) << 16);
    if (s == 0.f) s = 1.f;
    if (lane % LANES == 0) kept[lane / LANES][wave * PER + u] = s;
    // w / s rounded correctly from the correctly rounded reciprocal (Markstein:
    // t = w r, then t + r (w - t s)), where nothing leaves the range of normal
    // numbers; one addition then rounds it to the code, 8 on top
    const float r = __fdiv_rn(1.f, s);
    uint32_t code = 0;
    const bool plain = s > 0x1p-100f && s < 0x1p100f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float t = f[u][e] * r;
      t = fmaf(fmaf(-t, s, f[u][e]), r, t);
      if (!plain) t = __fdiv_rn(f[u][e], s);
      const uint32_t v = __float_as_uint(t + (12582912.f + 8.f)) & 15u;
      code |= v << (4 * e);
    }
    const int64_t row = r0 + wave * PER + u;
    if (row < rows && c < cols) store_nt(q + row * (cols / 2) + c / 2, code);
  }
  __syncthreads();
  for (int at = threadIdx.x; at < G * kQuantRows; at += 256) {
    const int grp = at / kQuantRows, r = at % kQuantRows;
    if (r0 + r < rows && c0 + grp * GROUP < cols) {
      S* to = scales + (c0 / GROUP + grp) * rows + r0 + r;
      if constexpr (sizeof(S) == 2) *to = (S)(__float_as_uint(kept[grp][r]) >> 16);
      else *to = kept[grp][r];
    }
  }
}

template <class T, class S, int GROUP>
__global__ __launch_bounds__(256) void int4_dequantize_kernel(const uint8_t* __restrict__ q, const S* __restrict__ scales,
                                                              int64_t rows, int64_t cols, T* __restrict__ w) {
  constexpr int G = kQuantCols / GROUP, LANES = GROUP / 8;
  __shared__ float kept[G][kQuantRows + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t r0 = (int64_t)blockIdx.x * kQuantRows, c0 = (int64_t)blockIdx.y * kQuantCols, c = c0 + lane * 8;
  w += (int64_t)blockIdx.z * rows * cols;
  q += (int64_t)blockIdx.z * rows * (cols / 2);
  scales += (int64_t)blockIdx.z * rows * (cols / GROUP);
  constexpr int PER = kQuantRows / 4;
  uint32_t code[PER];
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int64_t r = r0 + wave * PER + u;
    code[u] = r < rows && c < cols
                  ? __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(q + r * (cols / 2) + c / 2)) : 0;
  }
  for (int at = threadIdx.x; at < G * kQuantRows; at += 256) {
    const int grp = at / kQuantRows, r = at % kQuantRows;
    if (r0 + r < rows && c0 + grp * GROUP < cols) {
      const S v = scales[(c0 / GROUP + grp) * rows + r0 + r];
      if constexpr (sizeof(S) == 2) kept[grp][r] = __uint_as_float((uint32_t)v << 16);
      else kept[grp][r] = v;
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int64_t r = r0 + wave * PER + u;
    if (r >= rows || c >= cols) continue;
    const float s = kept[lane / LANES][wave * PER + u];
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (float)((int)(code[u] >> (4 * e) & 15u) - 8) * s;
    T* to = w + r * cols + c;
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    if constexpr (sizeof(T) == 2) {
      __builtin_nontemporal_store(u4{bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]), bf16x2(f[6], f[7])},
                                  reinterpret_cast<u4*>(to));
    } else {
      __builtin_nontemporal_store(v4f{f[0], f[1], f[2], f[3]}, reinterpret_cast<v4f*>(to));
      __builtin_nontemporal_store(v4f{f[4], f[5], f[6], f[7]}, reinterpret_cast<v4f*>(to + 4));
    }
  }
}

dim3 quant_grid(int64_t batch, int64_t rows, int64_t cols) {
  return dim3((unsigned)((rows + kQuantRows - 1) / kQuantRows), (unsigned)((cols + kQuantCols - 1) / kQuantCols), (unsigned)batch);
}

template <class T, class S>
hipError_t quantize_as(const void* w, int64_t batch, int64_t rows, int64_t cols, int group, uint8_t* q, void* scales,
                       hipStream_t stream) {
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, quant_grid(batch, rows, cols), dim3(256), 0, stream, (const T*)w, rows, cols, q, (S*)scales);
    return hipGetLastError();
  };
  return group == 32 ? go(int4_quantize_kernel<T, S, 32>) : group == 64 ? go(int4_quantize_kernel<T, S, 64>)
                                                                        : go(int4_quantize_kernel<T, S, 128>);
}
template <class T, class S>
hipError_t dequantize_as(const uint8_t* q, const void* scales, int64_t batch, int64_t rows, int64_t cols, int group, void* w,
                         hipStream_t stream) {
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, quant_grid(batch, rows, cols), dim3(256), 0, stream, q, (const S*)scales, rows, cols, (T*)w);
    return hipGetLastError();
  };
  return group == 32 ? go(int4_dequantize_kernel<T, S, 32>) : group == 64 ? go(int4_dequantize_kernel<T, S, 64>)
                                                                          : go(int4_dequantize_kernel<T, S, 128>);
}

}  // namespace

int64_t int4_workgroups(int64_t batch, int64_t rows, int64_t cols) {
  return batch * ((rows + kQuantRows - 1) / kQuantRows) * ((cols + kQuantCols - 1) / kQuantCols);
}

hipError_t launch_int4_quantize(const void* w, bool bf16, int64_t batch, int64_t rows, int64_t cols, int group, uint8_t* q,
                                void* scales, bool scales_bf16, hipStream_t stream) {
  if (bf16)
    return scales_bf16 ? quantize_as<uint16_t, uint16_t>(w, batch, rows, cols, group, q, scales, stream)
                       : quantize_as<uint16_t, float>(w, batch, rows, cols, group, q, scales, stream);
  return scales_bf16 ? quantize_as<float, uint16_t>(w, batch, rows, cols, group, q, scales, stream)
                     : quantize_as<float, float>(w, batch, rows, cols, group, q, scales, stream);
}
hipError_t launch_int4_dequantize(const uint8_t* q, const void* scales, bool scales_bf16, int64_t batch, int64_t rows,
                                  int64_t cols, int group, void* w, bool bf16, hipStream_t stream) {
  if (bf16)
    return scales_bf16 ? dequantize_as<uint16_t, uint16_t>(q, scales, batch, rows, cols, group, w, stream)
                       : dequantize_as<uint16_t, float>(q, scales, batch, rows, cols, group, w, stream);
  return scales_bf16 ? dequantize_as<float, uint16_t>(q, scales, batch, rows, cols, group, w, stream)
                     : dequantize_as<float, float>(q, scales, batch, rows, cols, group, w, stream);
}

}  // namespace fg8

// What the BF16-output products share: the work unit of a workgroup (which rows
// and columns, looked up among the ragged runs) and the epilogue.
#pragma once

#include <type_traits>

#include "fg8_device.h"
#include "fg8_internal.h"

namespace fg8 {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kLdsBytes = 160 * 1024;          // of a CU
constexpr int kBK = 64;                       // k depth of one step
constexpr uint32_t kNowhere = 0x80000000u;    // an offset past every buffer resource

// A copy of 16 bytes a lane into LDS at `lds` + 16 * lane.  The instruction
// writes no VGPR; the wait state between the write of m0 and its use is ours
// to keep inside an asm block.
__device__ __forceinline__ void copy16(v4i rsrc, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :
               : "v"(off), "s"(rsrc), "s"(lds)
               : "memory", "m0");
}

__device__ __forceinline__ v4i resource(const void* base, int64_t bytes) {
  const uint64_t a = uniform((uint64_t)base);
  const int n = uniform((int)(bytes < 0 ? 0 : bytes > 0x7fffffff ? 0x7fffffff : bytes));
  return v4i{(int)(uint32_t)a, (int)((uint32_t)(a >> 32) & 0xffffu), n, kBufferDword3};
}

// ------------------------------------------------------------ work units
struct BfUnit {
  int g;                 // expert (0 for dense), -1: rows of no run, written as zeros
  int64_t m0, k0;        // first row of D / first k
  int n0, rows, ks;      // first column; rows of D from m0 on; k length
  int split, tile;
};

__device__ __forceinline__ int clamp_off(int v, int most) { return min(max(v, 0), most); }

// The row tiles of the runs of `groups` experts: tiles of a run are its rows in
// pieces of BM; the rows before the first run and after the last one are two
// more runs (g = -1), whose output is zeros.  A wave looks at 64 runs at a
// time, one a lane; `incl` counts the tiles of the 64 up to and with this one.
template <int BM>
struct Runs {
  int a, b, tiles, incl;
  __device__ Runs(const int32_t* off, int groups, int rows, int c, int lane) {
    const int e = c + lane;
    a = b = 0;
    if (e < groups) {
      a = clamp_off(off[e], rows);
      b = clamp_off(off[e + 1], rows);
    } else if (e == groups) {
      a = clamp_off(off[groups], rows);
      b = rows;
    } else if (e == groups + 1) {
      b = clamp_off(off[0], rows);
    }
    tiles = b > a ? (b - a + BM - 1) / BM : 0;
    incl = scan(tiles);
  }
  // Running sum over the lanes: within rows of sixteen (row_shr by 1, 2, 4, 8),
  // then each row's last lane into the row after it (rows 1 and 3, then the
  // upper two).  Register moves, where shuffles go through LDS.
  __device__ static int scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
    return v;
  }
  __device__ int all() const { return __builtin_amdgcn_readlane(incl, 63); }
  // looks row tile u of these 64 runs up (u < all()); c: the first run
  __device__ void find(int u, int c, int groups, int& g, int& m0, int& end) const {
    const int l = __builtin_ctzll(__ballot(incl > u));
    const int first = __builtin_amdgcn_readlane(incl - tiles, l);
    g = c + l < groups ? c + l : -1;
    m0 = __builtin_amdgcn_readlane(a, l) + (u - first) * BM;
    end = __builtin_amdgcn_readlane(b, l);
  }
};

// The same for a persistent workgroup that looks up many units: the runs'
// tile counts as a running sum in LDS, with each run's start and end.
constexpr int kMaxRuns = 1024 + 2;
struct RunTable {
  int sum[kMaxRuns], start[kMaxRuns], end[kMaxRuns];   // sum: tiles of the runs up to and with this one
};
// Filled by one wave (the caller's barrier makes it visible).
template <int BM>
__device__ __forceinline__ void fill_runs(RunTable& t, const int32_t* off, int groups, int rows, int lane) {
  int base = 0;
  for (int c = 0; c < groups + 2; c += 64) {
    const Runs<BM> r(off, groups, rows, c, lane);
    if (c + lane < groups + 2) {
      t.sum[c + lane] = base + r.incl;
      t.start[c + lane] = r.a;
      t.end[c + lane] = r.b;
    }
    base += r.all();
  }
}
template <int BM>
__device__ __forceinline__ void look_up_run(const RunTable& t, int groups, int m, int& g, int& m0, int& rows) {
  int lo = 0, hi = groups + 1;      // the first run whose sum exceeds m
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (uniform(t.sum[mid]) > m) hi = mid; else lo = mid + 1;
  }
  const int first = lo > 0 ? uniform(t.sum[lo - 1]) : 0;
  g = lo < groups ? lo : -1;
  m0 = uniform(t.start[lo]) + (m - first) * BM;
  rows = uniform(t.end[lo]) - m0;
}

// Tile order: XCD x runs the workgroups of index x mod 8.  In every round of G
// units (a CU's worth each) it takes a contiguous run of ids, and ids walk
// kRaster row tiles before the next column, so the tiles an XCD runs together
// share operand rows in its L2.
constexpr int kRaster = 8;
constexpr int kCus = 256;     // of the device; only the tile order goes by it
__device__ __forceinline__ int xcd_round(int u, int total, int G) {
  const int base = u / G * G;
  if (G % 8 || base + G > total) return u;
  const int b = u - base;
  return base + (b % 8) * (G / 8) + b / 8;
}
__device__ __forceinline__ void raster(int id, int mt, int nt, int& m, int& n) {
  const int per = kRaster * nt, grp = id / per, first = grp * kRaster;
  const int rows = min(mt - first, kRaster), r = id - grp * per;
  m = first + r % rows;
  n = r / rows;
}

// The unit of this workgroup; false where it has none (the grid is an upper
// bound: how the rows fall into runs is known on the device only).
template <int BM, int BN, int MODE>
__device__ __forceinline__ bool find_unit(const BfProblem& p, int lane, BfUnit& w) {
  const int nt = (p.N + BN - 1) / BN;
  w = BfUnit{};
  if constexpr (MODE == kBfRowRuns) {
    // (every wave for itself; up to 62 experts are one look at the offsets)
    const Runs<BM> head(p.offsets, p.groups, p.M, 0, lane);
    int mt = head.all();
    for (int c = 64; c < p.groups + 2; c += 64) mt += Runs<BM>(p.offsets, p.groups, p.M, c, lane).all();
    if ((int)blockIdx.x >= mt * nt) return false;
    const int id = xcd_round(blockIdx.x, mt * nt, kCus);
    int m, n, g, m0, end;
    raster(id, mt, nt, m, n);
    if (m < head.all()) {
      head.find(m, 0, p.groups, g, m0, end);
    } else {
      int before = head.all();
      for (int c = 64;; c += 64) {     // (m < mt, so one of the pieces holds it)
        const Runs<BM> r(p.offsets, p.groups, p.M, c, lane);
        if (m < before + r.all()) {
          r.find(m - before, c, p.groups, g, m0, end);
          break;
        }
        before += r.all();
      }
    }
    w.g = uniform(g);
    w.m0 = uniform(m0);
    w.n0 = uniform(n) * BN;
    w.rows = uniform(end - m0);
    w.ks = w.g < 0 ? 0 : p.K;
  } else {
    const int mt = (p.M + BM - 1) / BM, tiles = mt * nt;
    const int total = tiles * (MODE == kBfKRuns ? p.groups : p.splits);
    if ((int)blockIdx.x >= total) return false;
    int id = xcd_round(blockIdx.x, total, kCus);
    int m, n;
    const int part = id / tiles;
    id -= part * tiles;
    raster(id, mt, nt, m, n);
    w.m0 = (int64_t)m * BM;
    w.n0 = n * BN;
    w.rows = p.M - (int)w.m0;
    if constexpr (MODE == kBfKRuns) {
      const int a = clamp_off(p.offsets[part], p.K), b = clamp_off(p.offsets[part + 1], p.K);
      w.g = part;
      w.k0 = uniform(a);
      w.ks = uniform(max(b - a, 0));
    } else {
      const int steps = (p.K + kBK - 1) / kBK;
      const int s0 = (int)((int64_t)part * steps / p.splits), s1 = (int)((int64_t)(part + 1) * steps / p.splits);
      w.split = part;
      w.tile = id;
      w.k0 = (int64_t)s0 * kBK;
      w.ks = min(p.K, s1 * kBK) - s0 * kBK;
    }
  }
  return true;
}

// ---------------------------------------------------------------- epilogue
template <class F, int N>
__device__ __forceinline__ void each(v4f (&v)[N], F f) {
#pragma unroll
  for (int e = 0; e < 4 * N; ++e) v[e / 4][e % 4] = f(v[e / 4][e % 4]);
}
// act(v) in place; the branch is taken once for all the values
template <int N>
__device__ __forceinline__ void activate(int act, v4f (&v)[N]) {
  if (act == kActRelu) {
    each(v, [](float z) { return z < 0.f ? 0.f : z; });      // (NaN stays)
  } else if (act == kActSilu) {
    // -0 for very negative z: exp2 gives inf, its reciprocal 0
    each(v, [](float z) {
      return z * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
    });
  } else if (act == kActGelu) {
    each(v, [](float z) {
      float bell;
      return z * normal_cdf(z, &bell);
    });
  }
}

// bias[n .. n + 3] (0 past N, or without a bias)
__device__ __forceinline__ v4f bias4(const BfProblem& p, int n) {
  v4f v = {0.f, 0.f, 0.f, 0.f};
  if (p.bias) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < p.N)
        v[i] = p.bias_bf16 ? __uint_as_float((uint32_t)((const uint16_t*)p.bias)[n + i] << 16)
                           : ((const float*)p.bias)[n + i];
  }
  return v;
}
// residual[m][n .. n + 3] as BF16 bits (0 past N)
__device__ __forceinline__ uint2 residual4(const BfProblem& p, int64_t m, int n) {
  const uint16_t* r = p.residual + m * p.ldr + n;
  if (p.ldr % 4 == 0 && n + 4 <= p.N) return *reinterpret_cast<const uint2*>(r);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < p.N) w[i / 2] |= (uint32_t)r[i] << (16 * (i & 1));
  return make_uint2(w[0], w[1]);
}

// The four columns n .. n + 3 of row m that a lane holds: bias, activation,
// residual, and the stores.
struct BfOut {
  const BfProblem& p;
  char* d;               // the unit's D (first row of the tensor or expert)
  __device__ BfOut(const BfProblem& q, int g) : p(q) {
    d = (char*)p.d + (int64_t)(p.mode == kBfKRuns ? g : 0) * p.d_stride * (p.out_bf16 ? 2 : 4);
  }
  __device__ void four(int64_t m, int n, v4f v) const {
    if (p.bias) v += bias4(p, n);
    if (p.z) store(p.z, p.ldz, true, m, n, v);
    v4f t[1] = {v};
    activate(p.act, t);
    v = t[0];
    if (p.residual) {
      const uint2 w = residual4(p, m, n);
      v += v4f{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
               __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u)};
    }
    store(d, p.ldd, p.out_bf16, m, n, v);
  }
  __device__ void store(void* to, int64_t ld, bool bf16, int64_t m, int n, v4f v) const {
    const int N = p.N;
    if (bf16) {
      uint16_t* q = (uint16_t*)to + m * ld + n;
      const uint32_t lo = bf16x2(v[0], v[1]), hi = bf16x2(v[2], v[3]);
      if (ld % 4 == 0 && n + 4 <= N) {
        *reinterpret_cast<uint2*>(q) = make_uint2(lo, hi);
      } else {
        if (n < N) q[0] = (uint16_t)lo;
        if (n + 1 < N) q[1] = (uint16_t)(lo >> 16);
        if (n + 2 < N) q[2] = (uint16_t)hi;
        if (n + 3 < N) q[3] = (uint16_t)(hi >> 16);
      }
    } else {
      float* q = (float*)to + m * ld + n;
      if (ld % 4 == 0 && n + 4 <= N) {
        *reinterpret_cast<v4f*>(q) = v;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < N) q[i] = v[i];
      }
    }
  }
};

// The epilogue of waves that own 64 columns.  In registers a lane holds four
// columns of one row, and neighbouring lanes hold neighbouring rows; memory
// wants neighbouring lanes on neighbouring columns (256 KB tiles written
// straight from the registers leave a CU at 36 GB/s, as whole rows at 120
// GB/s; non-temporal stores of such 16-byte pieces reach 3 TB/s over the chip,
// whole rows 5.2).  So each wave turns sixteen rows of its columns at a time
// in a piece of LDS of its own, without a barrier.  In the staged rows the
// 16-byte chunk index is XORed with a function of the row, which keeps writes
// and reads free of bank conflicts.
__device__ __forceinline__ void stream16(void* to, uint4 v) {
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  __builtin_nontemporal_store(u4{v.x, v.y, v.z, v.w}, reinterpret_cast<u4*>(to));
}

// Eight BF16 or four FP32 columns from c on of the row at q, those below N.
__device__ __forceinline__ void store_eight(uint16_t* q, int64_t ld, int c, int N, bool full, uint4 v) {
  if (full) {
    stream16(q + c, v);
  } else if (ld % 8 == 0 && c + 8 <= N) {
    *reinterpret_cast<uint4*>(q + c) = v;
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < N) q[c + i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
  }
}
__device__ __forceinline__ void store_four(float* q, int64_t ld, int c, int N, bool full, v4f v) {
  if (full) {
    __builtin_nontemporal_store(v, reinterpret_cast<v4f*>(q + c));
  } else if (ld % 4 == 0 && c + 4 <= N) {
    *reinterpret_cast<v4f*>(q + c) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < N) q[c + i] = v[i];
  }
}

// The four columns from c on of the row at q as they lie there (0 past N).
__device__ __forceinline__ v4f load_four(const float* q, int64_t ld, int c, int N) {
  if (ld % 4 == 0 && c + 4 <= N) return *reinterpret_cast<const v4f*>(q + c);
  v4f v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (c + i < N) v[i] = q[c + i];
  return v;
}

// Sixteen rows x 64 columns as BF16 (2 KB of LDS) -> rows m + l / 8 (+ 8),
// columns n + 8 (l % 8) ..: eight lanes a row, 128 bytes.
__device__ __forceinline__ void store_bf16_rows(uint8_t* turn, const v4f (&v)[4], uint16_t* to, int64_t ld,
                                                int rows, int n, int N, int lane, bool full) {
  const int i = lane & 15, g = lane >> 4;
#pragma unroll
  for (int t = 0; t < 4; ++t)
    *reinterpret_cast<uint2*>(turn + i * 128 + (((2 * t + (g >> 1)) ^ swz(i)) << 4) + (g & 1) * 8) =
        make_uint2(bf16x2(v[t][0], v[t][1]), bf16x2(v[t][2], v[t][3]));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = 8 * h + (lane >> 3), c = lane & 7;
    const uint4 u = *reinterpret_cast<const uint4*>(turn + r * 128 + ((c ^ swz(r)) << 4));
    if (full || r < rows) store_eight(to + r * ld, ld, n + 8 * c, N, full, u);
  }
}
// Sixteen rows x 32 columns as FP32 (2 KB): eight lanes a row, 128 bytes.  ADD:
// on top of what lies there.
template <bool ADD>
__device__ __forceinline__ void store_f32_rows(uint8_t* turn, v4f a, v4f b, float* to, int64_t ld, int rows,
                                               int n, int N, int lane, bool full) {
  const int i = lane & 15, g = lane >> 4;
  *reinterpret_cast<v4f*>(turn + i * 128 + ((g ^ swz(i)) << 4)) = a;
  *reinterpret_cast<v4f*>(turn + i * 128 + (((4 + g) ^ swz(i)) << 4)) = b;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = 8 * h + (lane >> 3), c = lane & 7;
    v4f u = *reinterpret_cast<const v4f*>(turn + r * 128 + ((c ^ swz(r)) << 4));
    if (full || r < rows) {
      if constexpr (ADD) u += load_four(to + r * ld, ld, n + 4 * c, N);
      store_four(to + r * ld, ld, n + 4 * c, N, full, u);
    }
  }
}
// Sixteen rows x 64 columns staged as FP32 (4 KB), the residual's piece (res)
// added on the way out.
__device__ __forceinline__ void store_rows_plus(uint8_t* turn, const v4f (&v)[4], const uint4 (&res)[2],
                                                void* to, int64_t ld, bool bf16, int rows, int n, int N,
                                                int lane, bool full) {
  const int i = lane & 15, g = lane >> 4;
#pragma unroll
  for (int t = 0; t < 4; ++t) *reinterpret_cast<v4f*>(turn + i * 256 + (((4 * t + g) ^ i) << 4)) = v[t];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = 8 * h + (lane >> 3), c = lane & 7;
    v4f a = *reinterpret_cast<const v4f*>(turn + r * 256 + (((2 * c) ^ r) << 4));
    v4f b = *reinterpret_cast<const v4f*>(turn + r * 256 + (((2 * c + 1) ^ r) << 4));
    float f[8];
    RowVec<uint16_t>::widen(res[h], f);
    a += v4f{f[0], f[1], f[2], f[3]};
    b += v4f{f[4], f[5], f[6], f[7]};
    if (full || r < rows) {
      if (bf16) {
        store_eight((uint16_t*)to + r * ld, ld, n + 8 * c, N, full,
                    make_uint4(bf16x2(a[0], a[1]), bf16x2(a[2], a[3]), bf16x2(b[0], b[1]), bf16x2(b[2], b[3])));
      } else {
        store_four((float*)to + r * ld, ld, n + 8 * c, N, full, a);
        store_four((float*)to + r * ld, ld, n + 8 * c + 4, N, full, b);
      }
    }
  }
}
// residual[m][c .. c + 7] (0 past N)
__device__ __forceinline__ uint4 residual8(const BfProblem& p, int64_t m, int c) {
  const uint16_t* r = p.residual + m * p.ldr;
  if (p.ldr % 8 == 0 && c + 8 <= p.N) return *reinterpret_cast<const uint4*>(r + c);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < p.N) w[i / 2] |= (uint32_t)r[c + i] << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One unit's output: what rows16() needs beside the values.  ADD: on top of an
// FP32 output that is there (instances of their own, the others stay as they are).
template <bool EPI, bool ADD>
struct TileOut {
  static constexpr int kTurn = EPI ? 4096 : 2048;    // LDS of a wave
  const BfProblem& p;
  char* d;             // the unit's D
  uint8_t* turn;
  int64_t m0;
  int rows, n, lane;   // rows of D from m0 on; the wave's first column
  bool whole, full;    // the tile exists whole; and rows are whole 16-byte pieces
  v4f bias[EPI ? 4 : 1];
  __device__ TileOut(const BfProblem& q, const BfUnit& w, int bm, int bn, int wave_n, uint8_t* t, int l)
      : p(q), turn(t), m0(w.m0), rows(w.rows), n(w.n0 + wave_n), lane(l) {
    d = (char*)p.d + w.g * p.d_stride * (p.out_bf16 ? 2 : 4);     // (row runs: d_stride is 0)
    whole = w.rows >= bm && w.n0 + bn <= p.N;
    full = whole && p.ldd % (p.out_bf16 ? 8 : 4) == 0;
    if constexpr (EPI) {
#pragma unroll
      for (int i = 0; i < 4; ++i) bias[i] = bias4(p, n + 16 * i + 4 * (lane >> 4));
    }
  }
  // the residual of rows r .. r + 15, as rows16() takes it
  __device__ void residual(int r, uint4 (&res)[2]) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = r + 8 * h + (lane >> 3);
      res[h] = p.residual && at < rows ? residual8(p, m0 + at, n + 8 * (lane & 7)) : make_uint4(0, 0, 0, 0);
    }
  }
  // rows r .. r + 15 of the tile, the wave's 64 columns
  __device__ void rows16(int r, v4f (&v)[4], const uint4 (&res)[2]) const {
    const int64_t m = m0 + r;
    const int left = rows - r;
    if constexpr (EPI) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += bias[i];
      if (p.z) store_bf16_rows(turn, v, p.z + m * p.ldz, p.ldz, left, n, p.N, lane, whole && p.ldz % 8 == 0);
      activate(p.act, v);
      if (p.residual) {
        store_rows_plus(turn, v, res, d + m * p.ldd * (p.out_bf16 ? 2 : 4), p.ldd, p.out_bf16, left, n, p.N, lane, full);
        return;
      }
    }
    if (p.out_bf16) {
      store_bf16_rows(turn, v, (uint16_t*)d + m * p.ldd, p.ldd, left, n, p.N, lane, full);
    } else {
      store_f32_rows<ADD>(turn, v[0], v[1], (float*)d + m * p.ldd, p.ldd, left, n, p.N, lane, full);
      store_f32_rows<ADD>(turn, v[2], v[3], (float*)d + m * p.ldd, p.ldd, left, n + 32, p.N, lane, full);
    }
  }
};

// Sixteen rows x 32 columns as BF16 (1 KB of LDS) -> four lanes a row, 64 bytes.
// ld8: to and ld are whole 16-byte pieces.  Half lines, which meet their other
// halves in the L2: ordinary stores (29,319 ragged rows, k = 360, with z of 2 x 1520
// columns 120 us for 165 with the non-temporal hint).
__device__ __forceinline__ void store_bf16_half_rows(uint8_t* turn, v4f a, v4f b, uint16_t* to, int64_t ld, bool ld8,
                                                     int rows, int n, int N, int lane, bool whole) {
  const int i = lane & 15, g = lane >> 4;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const v4f v = t ? b : a;
    *reinterpret_cast<uint2*>(turn + i * 64 + (((2 * t + (g >> 1)) ^ (i >> 2)) << 4) + (g & 1) * 8) =
        make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
  }
  const int r = lane >> 2, c = lane & 3;
  const uint4 u = *reinterpret_cast<const uint4*>(turn + r * 64 + ((c ^ (r >> 2)) << 4));
  if (whole || r < rows) store_eight(to + r * ld, ld8 ? 8 : 1, n + 8 * c, N, false, u);
}

// One unit's output of a gated product: a wave holds the gate and the up sums of
// the same 16 COLS columns of h.  z is taken before the activation, h from the
// FP32 sums.
template <int COLS>
struct GatedOut {
  static constexpr int kTurn = 2048;                 // LDS of a wave
  const BfProblem& p;
  uint8_t* turn;
  int64_t m0;
  int rows, j, n, lane;      // rows of D from m0 on; the wave's first column, of n
  bool whole, z8, h8;
  __device__ GatedOut(const BfProblem& q, const BfUnit& w, int bm, int bn, int wave_n, uint8_t* t, int l)
      : p(q), turn(t), m0(w.m0), rows(w.rows), j((w.n0 + wave_n) / 2), n(p.N / 2), lane(l) {
    whole = w.rows >= bm && w.n0 + bn <= p.N;
    z8 = n % 8 == 0 && p.ldz % 8 == 0;               // (the up half of z starts at column n)
    h8 = p.ldd % (p.out_bf16 ? 8 : 4) == 0;
  }
  // rows r .. r + 15 of the tile
  __device__ void rows16(int r, v4f (&gate)[COLS], v4f (&up)[COLS]) const {
    const int64_t m = m0 + r;
    if (p.z) {
      put(true, p.z + m * p.ldz, p.ldz, z8, r, gate);
      put(true, p.z + m * p.ldz + n, p.ldz, z8, r, up);
    }
    activate(p.act, gate);
#pragma unroll
    for (int t = 0; t < COLS; ++t) gate[t] *= up[t];
    put(p.out_bf16, (char*)p.d + m * p.ldd * (p.out_bf16 ? 2 : 4), p.ldd, h8, r, gate);
  }
  __device__ void put(bool bf16, void* to, int64_t ld, bool pieces, int r, const v4f (&v)[COLS]) const {
    if constexpr (COLS == 2) {
      if (bf16) store_bf16_half_rows(turn, v[0], v[1], (uint16_t*)to, ld, pieces, rows - r, j, n, lane, whole);
      else store_f32_rows<false>(turn, v[0], v[1], (float*)to, ld, rows - r, j, n, lane, whole && pieces);
    } else if (r + (lane & 15) < rows) {
      // (sixteen columns: four a lane, straight from the registers)
      const int c = j + 4 * (lane >> 4), row = lane & 15;
      const bool four = pieces && c + 4 <= n;
      if (bf16) {
        uint16_t* q = (uint16_t*)to + row * ld + c;
        const uint32_t w[2] = {bf16x2(v[0][0], v[0][1]), bf16x2(v[0][2], v[0][3])};
        if (four) {
          *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c + i < n) q[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
        }
      } else {
        float* q = (float*)to + row * ld + c;
        if (four) {
          *reinterpret_cast<v4f*>(q) = v[0];
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c + i < n) q[i] = v[0][i];
        }
      }
    }
  }
};

// ----------------------------------------------------- loss of a linear head
// The target of a row as a class, -1 for none.
__device__ __forceinline__ int target_of(const BfLoss& s, int64_t row) {
  const int64_t t = s.targets64 ? ((const int64_t*)s.targets)[row] : ((const int32_t*)s.targets)[row];
  return t >= 0 && t < s.classes ? (int)t : -1;
}
// v of the four lanes that hold a row's columns, combined
template <class F>
__device__ __forceinline__ float over_row(float v, F f) {
  typedef unsigned u2 __attribute__((ext_vector_type(2)));
  u2 a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = f(__uint_as_float(a[0]), __uint_as_float(a[1]));
  a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return f(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
constexpr float kLog2e = 1.4426950408889634f;
// From here on down an exponential adds nothing, and where every logit of a piece
// is -inf or past the last class the piece has a maximum to subtract.
constexpr float kLowest = -3.4028235e38f;

// A wave's 64 columns of a tile of logits, GROUPS times sixteen rows: kKindLse
// leaves each row's maximum and sum in LDS (merge() below joins the waves'; one pair
// a row and tile goes to memory, 33 MB for the 4 GB of logits of 8192 x 128000),
// kKindDlogits stores dlogits.  The logits are the FP32 sums, never rounded.
template <int KIND, int GROUPS>
struct LossOut {
  static constexpr int kTurn = 2048;    // LDS of a wave
  const BfProblem& p;
  uint8_t* turn;
  int64_t m0;
  int rows, n, lane;
  bool whole;
  static constexpr int kNone = -0x7fffffff - 1;
  int target[GROUPS];                   // of this lane's row, counted from this product's first class
  float lse[GROUPS], dloss[GROUPS];
  __device__ LossOut(const BfProblem& q, const BfUnit& w, int bm, int bn, int wave_n, uint8_t* t, int l)
      : p(q), turn(t), m0(w.m0), rows(w.rows), n(w.n0 + wave_n), lane(l) {
    whole = w.rows >= bm && w.n0 + bn <= p.N;
  }
  // what the rows from r0 of the tile on need
  __device__ void fetch(int r0) {
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      const int64_t row = m0 + min(r0 + 16 * g + (lane & 15), rows - 1);
      const int t = target_of(p.loss, row);
      target[g] = t < 0 ? kNone : t - p.loss.first;
      if constexpr (KIND == kKindDlogits) {
        lse[g] = p.loss.lse[row];
        dloss[g] = p.loss.dloss[row];
      }
    }
  }
  // rows r .. r + 15 of the tile, the g-th sixteen of this wave
  __device__ void rows16(int g, int r, v4f (&v)[4]) {
    const int64_t m = m0 + r;
    const int c0 = n + 4 * (lane >> 4);         // v[t][e] is column c0 + 16 t + e
    if constexpr (KIND == kKindLse) {
      float top = kLowest, sum = 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = c0 + 16 * t + e;
          if (c == target[g] && r + (lane & 15) < rows) p.loss.picked[m + (lane & 15)] = v[t][e];
          if (!whole && c >= p.N) v[t][e] = -__builtin_inff();
          top = fmaxf(top, v[t][e]);
        }
      top = over_row(top, [](float a, float b) { return fmaxf(a, b); });
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += __builtin_amdgcn_exp2f((v[t][e] - top) * kLog2e);
      sum = over_row(sum, [](float a, float b) { return a + b; });
      if (lane < 16) reinterpret_cast<float2*>(turn)[16 * g + lane] = make_float2(top, sum);
    } else {
      v4f rest[4];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = c0 + 16 * t + e;
          float d = __builtin_amdgcn_exp2f((v[t][e] - lse[g]) * kLog2e);
          if (c == target[g]) d -= 1.f;
          d = target[g] == kNone || (!whole && c >= p.N) ? 0.f : d * dloss[g];
          v[t][e] = d;
          rest[t][e] = bf16_rest(d);
        }
      const int N = (p.N + 7) & ~7;             // (zeros up to whole pieces)
      store_bf16_rows(turn, v, (uint16_t*)p.d + m * p.ldd, p.ldd, rows - r, n, N, lane, whole);
      if (p.loss.rest) store_bf16_rows(turn, rest, p.loss.rest + m * p.ldd, p.ldd, rows - r, n, N, lane, whole);
    }
  }
  // After a barrier: the maxima and sums of WAVES waves side by side, whose pieces
  // of LDS lie `apart`, joined and stored; row: this lane's of 16 GROUPS.
  template <int WAVES>
  __device__ static void merge(const BfProblem& p, const BfUnit& w, const uint8_t* turns, int apart, int row, int r0, int bn) {
    if (r0 + row >= w.rows) return;
    float2 v[WAVES];
    float top = kLowest, sum = 0.f;
#pragma unroll
    for (int q = 0; q < WAVES; ++q) {
      v[q] = reinterpret_cast<const float2*>(turns + q * apart)[row];
      top = fmaxf(top, v[q].x);
    }
#pragma unroll
    for (int q = 0; q < WAVES; ++q) sum += v[q].y * __builtin_amdgcn_exp2f((v[q].x - top) * kLog2e);
    p.loss.pieces[(int64_t)(w.n0 / bn) * p.M + w.m0 + r0 + row] = make_float2(top, sum);
  }
};

}  // namespace fg8

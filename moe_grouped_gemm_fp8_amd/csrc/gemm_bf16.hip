// BF16 products for gfx950: the expert products over ragged row runs
// (forward, input gradient, weight gradient) and the dense product with bias,
// activation and residual in its epilogue.
//
// Every one is D[m][n] = sum_k A(m, k) B(n, k) with BF16 operands, FP32
// accumulators and one rounding at the end; they differ in how the operands
// lie in memory and in where a tile's rows, columns and k range come from:
//   dense           A [M][K], B [N][K]            y  = x W^T
//   dense, B by k   A [M][K], B [K][N]            dx = dz W
//   dense, both     A [K][M], B [K][N]            dW = dz^T x
//   row runs        the same first two, rows off[e] .. off[e + 1] - 1 of A and
//                   D belonging to expert e, whose B is b + e * b_stride
//   k runs          the third, k (a token row) off[e] .. off[e + 1] - 1
//                   belonging to expert e, whose D is d + e * d_stride
//
// An operand tile of one 64-deep k step is copied from global memory straight
// into LDS (16 bytes a lane, no staging registers).  The copies go through a
// buffer resource that ends where the operand's run ends, so rows past a
// ragged end arrive as zeros: for the k runs that is what keeps one expert's
// rows (whatever they hold, NaN included) out of another expert's sum.
//   k-contiguous operand: LDS [row][64 k], 128-byte rows, 16-byte chunk index
//     XOR (row >> 1) & 7; a fragment is one ds_read_b128 a lane.
//   k-major operand: LDS [64 k][cols], 32-byte granule index XOR a function of
//     k; a fragment is two ds_read_b64_tr_b16, which hand lane i of a 16-lane
//     group column i of a 4 x 16 block.  Eight rows of a half wave's read fall
//     on eight granules, so neither read has bank conflicts.
// MFMA 16x16x32: lane i + 16 g holds row i, k = 8 g .. 8 g + 7 of either
// operand; result register v of that lane is row 4 g + v, column i.  B goes in
// as the first operand, so a lane holds four consecutive columns n of one row.
//
// What bounds them (one MI355X; a library product of 8192^3 in BF16 runs at
// 1480-1620 TFLOP/s there, 1.4 to 1.6 GHz under that load):
//   compute: 8192^3 0.72-0.76 ms, 1440-1530 TFLOP/s, with B k-major 0.75-0.81,
//     with both 0.78-0.83 (the library 0.79-0.84 and 0.91-0.96); MFMA busy 73% on ragged
//     runs of 1563 rows, K = 7168.  Short runs and few tiles lose to tiles that
//     a run ends in and to the last round of the CUs.
//   stores: the weight gradient of short runs, whose FP32 tiles take as long as
//     their sums and do not overlap them (kernel below).
//   weights: few rows, where the time is that of reading them once.
#include <type_traits>

#include "fg8_device.h"
#include "fg8_internal.h"

namespace fg8 {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

constexpr int kLdsBytes = 160 * 1024;          // of a CU
constexpr int kBK = 64;                       // k depth of one step
constexpr uint32_t kNowhere = 0x80000000u;    // an offset past every buffer resource

template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int STAGES_, int OCC_, int DEPTH_ = kBK>
struct BfCfg {
  static constexpr int DEPTH = DEPTH_;     // k of a stage
  static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_;
  static constexpr int STAGES = STAGES_, OCC = OCC_;
  static constexpr int WAVES = WAVES_M * WAVES_N, THREADS = 64 * WAVES;
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N, TM = WM / 16, TN = WN / 16;
  static constexpr int A_BYTES = BM * DEPTH * 2, B_BYTES = BN * DEPTH * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static_assert(WM % 16 == 0 && WN % 16 == 0 && STAGES >= 2, "whole MFMA tiles, two stages");
  // (the stages, and bf16_kernel's flag beside them)
  static_assert(OCC * (STAGES * STAGE_BYTES + 16) <= kLdsBytes, "OCC workgroups share the LDS of a CU");
};

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

// One operand's tile: BX rows (m or n) by 64 k.  KMAJOR: memory is [k][x].
template <bool KMAJOR, int BX, int WAVES, int DEPTH = kBK>
struct Operand {
  static constexpr int BYTES = BX * DEPTH * 2;
  static constexpr int COPIES = BYTES / 1024;                     // of a wave's 1 KB
  static constexpr int PER = (COPIES + WAVES - 1) / WAVES;        // per wave (the last may be short)
  static constexpr bool EVEN = COPIES % WAVES == 0;
  static constexpr int PITCH = KMAJOR ? BX * 2 : DEPTH * 2;       // bytes of an LDS row
  static_assert(!KMAJOR || BX >= 64, "a k-major tile is 64 columns at least");

  const char* base;      // the tile's first element at the first k of the run
  int64_t ld;            // bytes between memory rows
  int64_t left;          // k-contiguous: bytes of the rows before the last one; k-major: bytes of a row
  uint32_t off[PER];     // this lane's source of each copy, from base
  int rem_k;             // k elements of the run

  // XOR of the 16-byte chunks of k-contiguous row r: with 64-byte rows two rows
  // share the 128 bytes that the 64-deep layout gives one
  __device__ static int chunk_xor(int r) { return DEPTH == 64 ? swz(r) : r >> 2 & 3; }
  // XOR of the 32-byte granules of k-major row k
  __device__ static int gran(int k) {
    return BX >= 128 ? (k & 3) | ((k >> 3 & 1) << 2) : (k >> 1 & 1) | ((k >> 3 & 1) << 1);
  }

  // A memory row is whole 16-byte chunks: dz's rows end in zeros up to one, the
  // row length of every other operand is a multiple of 8.
  // x0: the tile's first row (m or n); xs: rows of the operand from there
  // (>= 1); k0, ks: the run's first k and its length
  __device__ void init(const uint16_t* p, int64_t ld_elems, int64_t x0, int xs, int64_t k0, int ks,
                       int wave, int lane) {
    ld = ld_elems * 2;
    rem_k = ks;
    if constexpr (KMAJOR) {
      base = (const char*)(p + k0 * ld_elems + x0);
      left = (int64_t)((xs < BX ? xs + 7 : BX) & ~7) * 2;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int at = (wave + i * WAVES) * 1024 + lane * 16;      // byte of the LDS tile
        const int k = at / PITCH, c = (at % PITCH / 16) ^ (gran(k) << 1);
        off[i] = c * 8 < xs ? (uint32_t)(k * ld) + c * 16 : kNowhere;
      }
    } else {
      base = (const char*)(p + x0 * ld_elems + k0);
      left = (int64_t)((xs < BX ? xs : BX) - 1) * ld;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int at = (wave + i * WAVES) * 1024 + lane * 16;
        const int r = at / PITCH, c = (at % PITCH / 16) ^ chunk_xor(r);
        off[i] = (uint32_t)(r * ld) + c * 16;
      }
    }
  }

  // the copies of k step kt into the LDS tile at `lds`
  __device__ void issue(int kt, uint32_t lds, int wave, int lane) const {
    const int rem = rem_k - kt * DEPTH;   // k elements from this step on (> 0)
    if constexpr (KMAJOR) {
      const v4i rs = resource(base + (int64_t)kt * DEPTH * ld, (int64_t)(rem - 1) * ld + left);
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (EVEN || wave + i * WAVES < COPIES)
          copy16(rs, off[i], uniform(lds + (uint32_t)(wave + i * WAVES) * 1024));
    } else {
      const v4i rs = resource(base + (int64_t)kt * (DEPTH * 2), left + (int64_t)((rem + 7) & ~7) * 2);
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (EVEN || wave + i * WAVES < COPIES) {
          // chunks at or past the end of k are zeros (K is a multiple of 8)
          const int at = (wave + i * WAVES) * 1024 + lane * 16;
          const int c = (at % PITCH / 16) ^ chunk_xor(at / PITCH);
          copy16(rs, c * 8 < rem ? off[i] : kNowhere, uniform(lds + (uint32_t)(wave + i * WAVES) * 1024));
        }
    }
  }

  // fragment of rows x .. x + 15, k = 32 kk .. 32 kk + 31
  __device__ static v8bf frag(const uint8_t* tile, int x, int kk, int lane) {
    const int i = lane & 15, g = lane >> 4;
    if constexpr (KMAJOR) {
      const int k = kk * 32 + 8 * g + (i >> 2);
      const uint8_t* p = tile + k * PITCH + (((x >> 4) ^ gran(k)) << 5) + (i & 3) * 8;
      const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p));
      const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 4 * PITCH));
      return __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const int r = x + i;
      return *reinterpret_cast<const v8bf*>(tile + r * PITCH + (((g + 4 * kk) ^ chunk_xor(r)) << 4));
    }
  }
};

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
    d = (char*)p.d + (int64_t)(p.mode == kBfKRuns ? w.g : 0) * p.d_stride * (p.out_bf16 ? 2 : 4);
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

// ---------------------------------------------------------------- split k
// Every split publishes its FP32 tile past the caches of its XCD and counts
// itself in; the last one to arrive adds them up in the order of the splits
// (the same bits on every call) and leaves the counter at zero.  False: this
// workgroup is not the last.
__device__ __forceinline__ bool last_of_splits(const BfProblem& p, const BfUnit& w, int tid, int* last) {
  wait_all_memory();        // this thread's part has reached the point of coherence
  __syncthreads();          // ... and every other thread's
  if (tid == 0) {
    *last = __hip_atomic_fetch_add(p.counters + w.tile, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == p.splits - 1;
    if (*last) __hip_atomic_store(p.counters + w.tile, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  return *last;
}
// ------------------------------------------------------------------ kernel
template <class C, bool AK, bool BK, int MODE, bool ADD = false>
__global__ __launch_bounds__(C::THREADS, C::OCC) void bf16_kernel(BfProblem p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::STAGES * C::STAGE_BYTES];
  __shared__ int last;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm0 = wave % C::WAVES_M * C::WM, wn0 = wave / C::WAVES_M * C::WN;
  BfUnit w;
  if (!find_unit<C::BM, C::BN, MODE>(p, lane, w)) return;

  v4f acc[C::TM][C::TN];
#pragma unroll
  for (int i = 0; i < C::TM; ++i)
#pragma unroll
    for (int j = 0; j < C::TN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  const int steps = (w.ks + C::DEPTH - 1) / C::DEPTH;
  if (steps > 0) {
    typedef Operand<AK, C::BM, C::WAVES, C::DEPTH> OpA;
    typedef Operand<BK, C::BN, C::WAVES, C::DEPTH> OpB;
    OpA a;
    OpB b;
    a.init(p.a, p.lda, w.m0, w.rows, w.k0, w.ks, wave, lane);
    b.init(p.b + (MODE == kBfRowRuns ? w.g * p.b_stride : 0), p.ldb, w.n0, p.N - w.n0, w.k0, w.ks, wave, lane);
    const uint32_t lds0 = lds_addr(smem);
    auto issue = [&](int kt) {
      const uint32_t st = uniform(lds0 + (uint32_t)(kt % C::STAGES * C::STAGE_BYTES));
      a.issue(kt, st, wave, lane);
      b.issue(kt, st + C::A_BYTES, wave, lane);
    };
    // copies a wave has in flight for one step (uneven tiles: some waves have
    // fewer, and then wait for a little more than they need)
    constexpr int LEAST = OpA::COPIES / C::WAVES + OpB::COPIES / C::WAVES;
    for (int s = 0; s < C::STAGES - 1; ++s)
      if (s < steps) issue(s);
    for (int kt = 0; kt < steps; ++kt) {
      if (steps - 1 - kt >= C::STAGES - 2) wait_vmcnt<(C::STAGES - 2) * LEAST>();
      else wait_vmcnt<0>();
      __syncthreads();
      if (kt + C::STAGES - 1 < steps) issue(kt + C::STAGES - 1);
      const uint8_t* As = smem + kt % C::STAGES * C::STAGE_BYTES;
      const uint8_t* Bs = As + C::A_BYTES;
#pragma unroll
      for (int kk = 0; kk < C::DEPTH / 32; ++kk) {
        v8bf fa[C::TM], fb[C::TN];
#pragma unroll
        for (int i = 0; i < C::TM; ++i) fa[i] = OpA::frag(As, wm0 + 16 * i, kk, lane);
#pragma unroll
        for (int j = 0; j < C::TN; ++j) fb[j] = OpB::frag(Bs, wn0 + 16 * j, kk, lane);
#pragma unroll
        for (int j = 0; j < C::TN; ++j)
#pragma unroll
          for (int i = 0; i < C::TM; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
      }
    }
  }

  if (MODE == kBfDense && p.splits > 1) {
    constexpr uint32_t kTile = C::BM * C::BN * 4;
    const __amdgpu_buffer_rsrc_t ws =
        buffer_rsrc(p.partial + (int64_t)w.tile * p.splits * (C::BM * C::BN), kTile * p.splits);
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
      for (int j = 0; j < C::TN; ++j)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i, acc[i][j]), ws,
                                               w.split * kTile + (((wave * C::TM + i) * C::TN + j) * 64 + lane) * 16,
                                               0, kCoherent);
    if (!last_of_splits(p, w, tid, &last)) return;
    // as many splits' tiles at a time as registers hold, all their loads
    // before the first addition
    constexpr int TILES = C::TM * C::TN, AT_ONCE = TILES >= 16 ? 2 : 32 / TILES;
    for (int s0 = 0; s0 < p.splits; s0 += AT_ONCE) {
      v4f part[AT_ONCE][TILES];
#pragma unroll
      for (int s = 0; s < AT_ONCE; ++s)
#pragma unroll
        for (int t = 0; t < TILES; ++t)
          if (s0 + s < p.splits)
            part[s][t] = __builtin_bit_cast(
                v4f, __builtin_amdgcn_raw_buffer_load_b128(
                         ws, (s0 + s) * kTile + ((wave * TILES + t) * 64 + lane) * 16, 0, kCoherent));
#pragma unroll
      for (int s = 0; s < AT_ONCE; ++s)
#pragma unroll
        for (int t = 0; t < TILES; ++t)
          if (s0 + s < p.splits) {
            v4f& a = acc[t / C::TN][t % C::TN];
            a = s0 + s == 0 ? part[s][t] : a + part[s][t];
          }
    }
  }

  if constexpr (C::WN == 64) {
    constexpr bool EPI = MODE == kBfDense && !AK && !BK;
    typedef TileOut<EPI, ADD> Out;
    static_assert(C::WAVES * Out::kTurn <= C::STAGES * C::STAGE_BYTES, "rows turn in the stages");
    __syncthreads();      // every wave is done with the stages
    const Out out(p, w, C::BM, C::BN, wn0, smem + wave * Out::kTurn, lane);
#pragma unroll
    for (int i = 0; i < C::TM; ++i) {
      uint4 res[2];
      if constexpr (EPI) out.residual(wm0 + 16 * i, res);
      v4f v[4] = {acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
      out.rows16(wm0 + 16 * i, v, res);
    }
  } else {
    const BfOut out(p, w.g);
#pragma unroll
    for (int i = 0; i < C::TM; ++i) {
      const int r = wm0 + 16 * i + (lane & 15);
      if (r < w.rows) {
#pragma unroll
        for (int j = 0; j < C::TN; ++j) out.four(w.m0 + r, w.n0 + wn0 + 16 * j + 4 * (lane >> 4), acc[i][j]);
      }
    }
  }
}

// ------------------------------------------------------------ few rows
// A few rows a run, both operands k-contiguous, a short k: the call's latency
// counts.  A workgroup owns 16 rows x 16 columns; its eight waves split k among
// themselves, 64 at a time in turn, and load their fragments of both operands
// straight into registers (16 bytes a lane, a lane's k are contiguous): no LDS
// and no barrier stands between a wave and its loads, and eight steps of them
// are in flight.  The waves' sums meet in LDS at the end.  (1 x 1024 x 2048:
// 5.5 us for the 6.6 of the thin tile.  A load of this shape touches 16 lines
// for 1 KB where a copy into LDS touches 8, so longer k go the other way:
// 16 x 2112 x 7168 19 us for 11.)
template <int MODE>
__global__ __launch_bounds__(512, 2) void bf16_few_kernel(BfProblem p) {
  constexpr int U = 4;       // steps of a batch; two batches in flight
  __shared__ v4f sums[8][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  BfUnit w;
  if (!find_unit<16, 16, MODE>(p, lane, w)) return;
  const int i = lane & 15, g = lane >> 4;

  // Offsets of a lane's row in either tile; rows and columns past the end read
  // the last one and are not stored.  k goes into the scalar offset, and a
  // lane whose k lies past the end loads zeros.
  const uint16_t* xp = p.a + w.m0 * p.lda;
  const uint16_t* wp = p.b + (MODE == kBfRowRuns ? max(w.g, 0) * p.b_stride : 0) + (int64_t)w.n0 * p.ldb;
  const __amdgpu_buffer_rsrc_t xr = buffer_rsrc(uniform((const void*)xp), 0x7fffffff);
  const __amdgpu_buffer_rsrc_t wr = buffer_rsrc(uniform((const void*)wp), 0x7fffffff);
  const uint32_t xo = (uint32_t)(min(i, w.rows - 1) * (int)p.lda + 8 * g) * 2;
  const uint32_t wo = (uint32_t)(min(i, p.N - 1 - w.n0) * (int)p.ldb + 8 * g) * 2;
  struct Batch {
    v4i x[U][2], w[U][2];
  };
  auto fetch = [&](Batch& f, int s0) {     // steps s0, s0 + 8, ..
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const int k = uniform((s0 + 8 * u) * kBK + 32 * kk);
        const bool in = 8 * g < w.ks - k;
        f.w[u][kk] = __builtin_bit_cast(
            v4i, __builtin_amdgcn_raw_buffer_load_b128(wr, in ? wo : kNowhere, k * 2, kStream));
        f.x[u][kk] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(xr, in ? xo : kNowhere, k * 2, 0));
      }
  };
  v4f acc = {0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const Batch& f) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, f.w[u][kk]),
                                                      __builtin_bit_cast(v8bf, f.x[u][kk]), acc, 0, 0, 0);
  };
  const int steps = (w.ks + kBK - 1) / kBK;
  if (wave < steps) {
    Batch f0, f1;
    fetch(f0, wave);
    for (int s = wave; s < steps; s += 16 * U) {
      fetch(f1, s + 8 * U);
      multiply(f0);
      if (s + 8 * U >= steps) break;
      fetch(f0, s + 16 * U);
      multiply(f1);
    }
  }
  sums[wave][lane] = acc;
  __syncthreads();
  if (wave == 0 && i < w.rows) {
    v4f sum = sums[0][lane];
#pragma unroll
    for (int v = 1; v < 8; ++v) sum += sums[v][lane];
    BfOut(p, w.g).four(w.m0 + i, w.n0 + 4 * g, sum);
  }
}

// ------------------------------------------------------- the 256 x 256 tile
// Half of an operand's 256 x 64 tile: the 128 rows (m or n) that the waves
// multiply together in one phase.  Row x of half h is tile row
// (x / RUN) * 2 RUN + h * RUN + x % RUN, RUN being the rows of a wave's half.
// A half is sixteen 1 KB copies, two a wave.
template <bool KMAJOR, int RUN>
struct HalfTile {
  static constexpr int ROWS = 128, BYTES = ROWS * kBK * 2;
  static constexpr int COPIES = BYTES / 1024 / 8;     // a wave's
  static constexpr int PITCH = KMAJOR ? ROWS * 2 : kBK * 2;
  typedef Operand<KMAJOR, ROWS, 8> Frag;    // the layout inside a half

  const char* base;
  int64_t ld;
  int64_t left;
  uint32_t off[2][COPIES];     // [half][copy]
  int rem_k;

  __device__ static int tile_row(int x, int h) { return x / RUN * (2 * RUN) + h * RUN + x % RUN; }

  __device__ void init(const uint16_t* p, int64_t ld_elems, int64_t x0, int xs, int64_t k0, int ks,
                       int wave, int lane) {
    ld = ld_elems * 2;
    rem_k = ks;
    base = KMAJOR ? (const char*)(p + k0 * ld_elems + x0) : (const char*)(p + x0 * ld_elems + k0);
    left = KMAJOR ? (int64_t)((xs < 256 ? xs + 7 : 256) & ~7) * 2 : (int64_t)((xs < 256 ? xs : 256) - 1) * ld;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < COPIES; ++i) {
        const int at = (wave * COPIES + i) * 1024 + lane * 16;
        if constexpr (KMAJOR) {
          const int k = at / PITCH, c = tile_row(((at % PITCH / 16) ^ (Frag::gran(k) << 1)) * 8, h);
          off[h][i] = c < xs ? (uint32_t)(k * ld) + c * 2 : kNowhere;
        } else {
          const int r = at / PITCH;
          off[h][i] = (uint32_t)(tile_row(r, h) * ld) + (((at % PITCH / 16) ^ swz(r)) << 4);
        }
      }
  }

  // this wave's copies of half h of k step kt into LDS; past the last step
  // they copy zeros, so the count of copies in flight stays what the waits
  // assume
  __device__ void issue(int kt, int h, uint32_t lds, int wave, int lane) const {
    const int rem = rem_k - kt * kBK;
    const int64_t bytes = KMAJOR ? (int64_t)(rem - 1) * ld + left : left + (int64_t)((rem + 7) & ~7) * 2;
    const v4i rs = resource(base + (int64_t)kt * (KMAJOR ? kBK * ld : kBK * 2), rem > 0 ? bytes : 0);
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
      uint32_t o = off[h][i];
      if constexpr (!KMAJOR) {
        const int c = (lane & 7) ^ (4 * i + (lane >> 4));     // the chunk of k, swz(row) undone
        o = c * 8 < rem ? o : kNowhere;
      }
      copy16(rs, o, uniform(lds + (uint32_t)(wave * COPIES + i) * 1024));
    }
  }
};

// A copy of a per-lane value that the compiler cannot trace: what is computed
// from it is computed here, not before the loop over units, where it would
// take registers through the main loop.
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Between the phases of the big tile: neither the compiler's memory accesses
// nor its instruction scheduling move across.
__device__ __forceinline__ void phase_fence() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void phase_barrier() {
  phase_fence();
  __builtin_amdgcn_s_barrier();
  phase_fence();
}

// Eight waves, two a SIMD, in two groups of four: group 0 owns the upper 128
// rows, group 1 the lower, wave q of a group columns 64 q .. 64 q + 63.  A k
// step is two phases, half of the wave's rows each: 32 MFMAs on fragments that
// are read once.  A phase is a memory part (fragment reads, four copies of a
// later step) and an MFMA part, with a workgroup barrier after each; group 1
// runs one part behind group 0, so on every SIMD one wave feeds the matrix
// unit while the other one waits for memory.  (Four phases of 16 MFMAs ran
// 8% slower: every change of the wave that feeds the unit costs a barrier.)
//
//   phase   reads of step t             copies                   MFMAs on
//   0       B half 1, A half 0          A0 and B1 of t + 1       A0 B0, A0 B1
//   1       B half 0 of t + 1, A half 1 A1 of t + 1, B0 of t + 2 A1 B1, A1 B0
//
// Number the parts of group 0 from 4 t (phase 0 of step t, memory), those of
// group 1 one later.  A wave has its reads of a memory part by the end of the
// MFMA part after it (LDS reads return in order, and each part's last ones are
// used there), so what was read in part s by group 0 is read by everybody
// before part s + 3.  A0 and B1 of t (s = 4 t) are overwritten from part 4 t + 4
// on, A1 of t and B0 of t + 1 (s = 4 t + 2) from part 4 t + 6.  A wave waits
// for its own copies in the memory part before the first read of them, and the
// barrier after that makes it everybody's: a copy has a whole step to land.
//
// The grid is one workgroup a CU, each walking the units; a unit's first
// copies are issued before the last unit's epilogue, which they run under.
//
// What a unit costs beside its steps (1.4-1.6 us each at full load): finding
// the next one and its first copies 1.3 us, and an epilogue of 4 to 9 us where
// every CU stores FP32 tiles.  The weight gradient of 32 runs, 16383 rows,
// 7168 x 2048, takes 0.72 ms, 0.43 without its 1.88 GB of stores, which alone
// take 0.31: the two add up whatever the order of the tiles (experts mixed over
// the XCDs, other numbers of tiles together on one, staggered starts and two
// workgroups a CU measured within 2% or slower).
template <bool AK, bool BK, int MODE, bool EPI, bool ADD = false>
__global__ __launch_bounds__(512, 2) void bf16_big_kernel(BfProblem p) {
  typedef HalfTile<AK, 64> HalfA;
  typedef HalfTile<BK, 32> HalfB;
  typedef TileOut<EPI, ADD> Out;
  constexpr uint32_t kHalf = HalfA::BYTES;         // LDS: per stage A0, A1, B0, B1
  constexpr uint32_t kTurns = 8 * kHalf, kTable = kTurns + 8 * Out::kTurn;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kTable + (MODE == kBfRowRuns ? sizeof(RunTable) : 0)];
  static_assert(sizeof(smem) <= kLdsBytes, "all the LDS of the kernel: the stages, the waves' turns, the runs");
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grp = wave >> 2, q = wave & 3;
  const int nt = (p.N + 255) / 256;
  int mt = (p.M + 255) / 256;
  if constexpr (MODE == kBfRowRuns) {
    RunTable& runs = *reinterpret_cast<RunTable*>(smem + kTable);
    if (wave == 0) fill_runs<256>(runs, p.offsets, p.groups, p.M, lane);
    __syncthreads();
    mt = uniform(runs.sum[p.groups + 1]);
  }
  const int total = mt * nt * (MODE == kBfKRuns ? p.groups : 1), G = p.grid;

  auto find = [&](int u, BfUnit& w) {
    int id = xcd_round(u, total, G), m, n;
    w = BfUnit{};
    if constexpr (MODE == kBfRowRuns) {
      raster(id, mt, nt, m, n);
      int m0;
      look_up_run<256>(*reinterpret_cast<const RunTable*>(smem + kTable), p.groups, m, w.g, m0, w.rows);
      w.m0 = m0;
      w.ks = w.g < 0 ? 0 : p.K;
    } else {
      const int part = MODE == kBfKRuns ? id / (mt * nt) : 0;
      raster(id - part * (mt * nt), mt, nt, m, n);
      w.m0 = (int64_t)m * 256;
      w.rows = p.M - (int)w.m0;
      w.ks = p.K;
      w.g = part;
      if constexpr (MODE == kBfKRuns) {
        const int a = clamp_off(p.offsets[part], p.K), b = clamp_off(p.offsets[part + 1], p.K);
        w.k0 = uniform(a);
        w.ks = uniform(max(b - a, 0));
      }
    }
    w.n0 = n * 256;
  };

  HalfA a;
  HalfB b;
  const uint32_t lds0 = lds_addr(smem);
  auto copy_a = [&](int t, int h) { a.issue(t, h, lds0 + ((t & 1) * 4 + h) * kHalf, wave, lane); };
  auto copy_b = [&](int t, int h) { b.issue(t, h, lds0 + ((t & 1) * 4 + 2 + h) * kHalf, wave, lane); };
  // Copies of two halves may be in flight wherever a wave waits for its own.
  static_assert(HalfA::COPIES == HalfB::COPIES);
  constexpr int kTwoHalves = 2 * HalfA::COPIES;
  auto start = [&](const BfUnit& w) {     // a unit's first five halves
    const int here = opaque(lane);
    a.init(p.a, p.lda, w.m0, w.rows, w.k0, w.ks, wave, here);
    b.init(p.b + (MODE == kBfRowRuns ? w.g * p.b_stride : 0), p.ldb, w.n0, p.N - w.n0, w.k0, w.ks, wave, here);
    copy_a(0, 0);
    copy_b(0, 0);
    copy_b(0, 1);
    copy_a(0, 1);
    copy_b(1, 0);
  };

  BfUnit w;
  int u = blockIdx.x;
  if (u >= total) return;
  find(u, w);
  if (w.ks > 0) start(w);
  while (true) {
    v4f acc[2][4][2][2];    // [A half][row tile][B half][column tile]
#pragma unroll
    for (int i = 0; i < 32; ++i) (&acc[0][0][0][0])[i] = v4f{0.f, 0.f, 0.f, 0.f};
    const int steps = (w.ks + kBK - 1) / kBK;
    if (steps > 0) {
      v8bf fa[4][2], fb[2][2][2], fb1[2][2];       // A half in use; B half 0 of two steps; B half 1
      auto read_a = [&](int st, int h) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            fa[i][kk] = HalfA::Frag::frag(smem + (st * 4 + h) * kHalf, grp * 64 + 16 * i, kk, lane);
      };
      auto read_b = [&](v8bf (&f)[2][2], int st, int h) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            f[j][kk] = HalfB::Frag::frag(smem + (st * 4 + 2 + h) * kHalf, q * 32 + 16 * j, kk, lane);
      };
      // 32 MFMAs: row half ha against column halves hb, then the other one
      auto multiply = [&](auto ha, v8bf (&f)[2][2], auto hb, v8bf (&f2)[2][2]) {
        phase_barrier();
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              acc[ha][i][hb][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[j][kk], fa[i][kk], acc[ha][i][hb][j], 0, 0, 0);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              acc[ha][i][1 - hb][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f2[j][kk], fa[i][kk], acc[ha][i][1 - hb][j], 0, 0, 0);
        __builtin_amdgcn_s_setprio(0);
        phase_barrier();
      };
      constexpr std::integral_constant<int, 0> c0{};
      constexpr std::integral_constant<int, 1> c1{};
      wait_vmcnt<kTwoHalves>();     // step 0 but for A1 (the last of start()'s five is B0 of step 1)
      phase_barrier();
      read_b(fb[0], 0, 0);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (grp == 1) phase_barrier();
      auto step = [&](auto par, int t) {
        constexpr int P = decltype(par)::value;
        read_b(fb1, P, 1);
        read_a(P, 0);
        copy_a(t + 1, 0);
        copy_b(t + 1, 1);
        wait_vmcnt<kTwoHalves>();   // A1 of step t, B0 of step t + 1
        multiply(c0, fb[P], c0, fb1);
        read_b(fb[P ^ 1], P ^ 1, 0);
        read_a(P, 1);
        copy_a(t + 1, 1);
        copy_b(t + 2, 0);
        wait_vmcnt<kTwoHalves>();   // A0 and B1 of step t + 1
        multiply(c1, fb1, c1, fb[P]);
      };
      for (int t = 0; t < steps; t += 2) {
        step(c0, t);
        if (t + 1 < steps) step(c1, t + 1);
      }
      if (grp == 0) phase_barrier();
      wait_vmcnt<0>();              // (the copies of zeros past the last step)
      __syncthreads();              // every wave's, and its reads
    }

    const int here = opaque(lane);
    Out out(p, w, 256, 256, q * 64, smem + kTurns + wave * Out::kTurn, here);
    if constexpr (EPI) {       // the bias has arrived before the copies below queue up
#pragma unroll
      for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(out.bias[i]));
    }
    // the next unit's first copies, under this one's epilogue
    BfUnit next{};
    u += G;
    if (u < total) {
      find(u, next);
      if (next.ks > 0) start(next);
    }

    // (the residual one group of sixteen rows ahead: before the stores, which
    // its loads would have to wait for)
    uint4 res[2], ahead[2];
    if constexpr (EPI) out.residual(grp * 128, res);
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      if constexpr (EPI) {
        if (g < 7) out.residual(grp * 128 + 16 * (g + 1), ahead);
      }
      const int ha = g / 4, i = g % 4;
      v4f v[4] = {acc[ha][i][0][0], acc[ha][i][0][1], acc[ha][i][1][0], acc[ha][i][1][1]};
      out.rows16(grp * 128 + 16 * g, v, res);
      if constexpr (EPI) {
        res[0] = ahead[0];
        res[1] = ahead[1];
      }
    }
    if (u >= total) return;
    w = next;
  }
}

// ------------------------------------------------------------------- host
// Tile configurations.  kBig: bf16_big_kernel; kFew: bf16_few_kernel; the
// others: bf16_kernel with two workgroups a CU.
enum { kBig = 0, kDuo, kMid, kHigh, kLow, kFlat, kThin, kFew, kConfigs };
using BfDuo = BfCfg<128, 256, 1, 4, 3, 2, 32>;
using BfMid = BfCfg<128, 128, 2, 2, 2, 2>;
using BfHigh = BfCfg<128, 64, 2, 2, 3, 2>;
using BfLow = BfCfg<64, 64, 2, 2, 4, 2>;
using BfFlat = BfCfg<32, 64, 2, 2, 5, 2>;
using BfThin = BfCfg<16, 64, 1, 4, 6, 2>;
constexpr int kBm[kConfigs] = {256, 128, 128, 128, 64, 32, 16, 16};
constexpr int kBn[kConfigs] = {256, 256, 128, 64, 64, 64, 64, 16};
constexpr int kThreads[kConfigs] = {512, BfDuo::THREADS, BfMid::THREADS, BfHigh::THREADS,
                                    BfLow::THREADS, BfFlat::THREADS, BfThin::THREADS, 512};

namespace {

// Workgroups for tiles of bm x bn, a multiple of the eight XCDs.
unsigned grid_of(const BfProblem& p, int bm, int bn) {
  const int64_t nt = ((int64_t)p.N + bn - 1) / bn;
  int64_t units = ((int64_t)p.M + bm - 1) / bm * nt;
  // row runs: a run may end inside a tile, so one more tile a run at most
  if (p.mode == kBfRowRuns) units += (int64_t)(p.groups + 1) * nt;
  if (p.mode == kBfKRuns) units *= p.groups;
  if (p.mode == kBfDense) units *= p.splits;
  return (unsigned)((units + 7) / 8 * 8);
}

template <class K>
hipError_t start(K kernel, const BfProblem& p, unsigned grid, int threads, hipStream_t stream) {
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(threads), 0, stream, p);
  return hipGetLastError();
}

template <bool AK, bool BK, int MODE>
hipError_t launch_tile(BfProblem p, const BfTile& t, hipStream_t stream) {
  const unsigned units = grid_of(p, t.bm, t.bn);
  if constexpr (!AK && !BK) {
    if (t.cfg == kFew) return start(bf16_few_kernel<MODE>, p, units, 512, stream);
  }
  if constexpr (!AK) {
    if (t.cfg == kThin) return start(bf16_kernel<BfThin, AK, BK, MODE>, p, units, BfThin::THREADS, stream);
    if (t.cfg == kFlat) return start(bf16_kernel<BfFlat, AK, BK, MODE>, p, units, BfFlat::THREADS, stream);
    if (t.cfg == kLow) return start(bf16_kernel<BfLow, AK, BK, MODE>, p, units, BfLow::THREADS, stream);
    if (t.cfg == kHigh) return start(bf16_kernel<BfHigh, AK, BK, MODE>, p, units, BfHigh::THREADS, stream);
  }
  if constexpr (MODE == kBfKRuns) {
    if (t.cfg == kDuo) return start(bf16_kernel<BfDuo, AK, BK, MODE>, p, units, BfDuo::THREADS, stream);
  }
  const unsigned cus = (unsigned)device_cu_count();
  p.grid = (int)(units < cus ? units : cus);
  if constexpr (MODE == kBfDense && AK && BK) {
    if (p.add)
      return t.cfg == kMid ? start(bf16_kernel<BfMid, AK, BK, MODE, true>, p, units, BfMid::THREADS, stream)
                           : start(bf16_big_kernel<AK, BK, MODE, false, true>, p, p.grid, 512, stream);
  }
  if (t.cfg == kMid) return start(bf16_kernel<BfMid, AK, BK, MODE>, p, units, BfMid::THREADS, stream);
  if constexpr (MODE == kBfDense && !AK && !BK) {
    if (p.bias || p.act != kActNone || p.residual || p.z)
      return start(bf16_big_kernel<AK, BK, MODE, true>, p, p.grid, 512, stream);
  }
  return start(bf16_big_kernel<AK, BK, MODE, false>, p, p.grid, 512, stream);
}

}  // namespace

BfTile bf16_tile(const BfProblem& p, int cus) {
  BfTile t{};
  // rows of one tile column: a run's average for the row runs
  const int64_t rows = p.mode == kBfRowRuns ? (p.M + p.groups - 1) / p.groups : p.M;
  const int64_t runs = p.mode == kBfDense ? 1 : p.groups;
  auto units = [&](int c) { return runs * ((rows + kBm[c] - 1) / kBm[c]) * (((int64_t)p.N + kBn[c] - 1) / kBn[c]); };
  // (times in us, the choice first; 256 CUs)
  //
  // One product: 128 x 128 tiles while all of them run at once, two a CU, and
  // the big tile beyond, where they would take a second round.  At 512 of them
  // (128 big ones): 2048 x 4096 x 7168 111 for 118, with GELU, residual and z
  // 122 for 135, dx of 4096 x 7168 x 2048 148 for 159 alone and 250 for 266
  // within its backward pass, dW of 4096 x 4096 x 2048 169 for 182 within its.
  // At 560 to 640: 1280 x 7168 x 2048 42 for 56, 4096 x 2560 x 7168 129 for 182,
  // dW of 4000 x 5000 x 2048 207 for 239.
  const bool dense = p.mode == kBfDense;
  const bool second_round = units(kMid) > 2 * cus;
  if (p.a_kmajor) {
    // Weight gradients of runs: the big tile from two tiles and 64 of its steps
    // a CU on (8 runs of 4096 rows, 4096 x 2048: 461-482 for 520-529 and
    // 562-578; 8 of 1024 144-152 for 149-155 and 158-165; 16 of 512 175-200 for
    // 178-187 and 200-209; below: 8 of 512 96-98 for 90-92, 16 of 1024,
    // 2048 x 1024, 129 for 106).  Short runs of many tiles are bound by their
    // stores, which two workgroups a CU interleave with sums (32 runs of 64
    // rows, 7168 x 2048: 288 for 312).  Few tiles: small ones (16 runs of 250
    // rows, 2048 x 1024: 39 for 43 and 47).
    const bool deep = units(kBig) >= 2 * cus && units(kBig) * (p.K / runs) >= (int64_t)4096 * cus;
    if (dense ? second_round : deep) t.cfg = kBig;
    else t.cfg = !dense && units(kBig) >= 6 * cus ? kDuo : kMid;
  } else if (rows > 128 && (dense ? second_round : 2 * units(kBig) >= cus)) {
    // Row runs, whose ends inside tiles are not known here: the big tile from
    // half the CUs on, by the runs' average.  8 ragged runs of 512 rows on
    // average, 2048 x 2048 (128 big tiles by it, 168 in fact): 43 for 54, of
    // 1024 rows (256, 296) 89 for 82, of 1024 rows, 4096 x 2048 (512, 592) 136
    // for 145.  Runs of whole tiles: 41 for 34, 56 for 65, 104 for 137.
    t.cfg = kBig;
  } else if (rows <= 8 && !p.b_kmajor && p.K <= 4096 && units(kFew) <= 2 * cus) {
    t.cfg = kFew;      // 1 x 1024 x 2048 5.5 for 6.6; 1 x 2112 x 7168 12.8 for 11.2
  } else if (rows <= (dense ? 16 : 8)) {
    t.cfg = kThin;     // 16 x 2112 x 7168 11.3 for 12.2; 32 runs of 16 rows on average 366 for 345
  } else if (rows <= 32) {
    t.cfg = kFlat;     // 32 x 2112 x 7168 12.3 for 13.7
  } else if (units(kMid) >= (dense ? 3 * cus / 2 : cus)) {
    t.cfg = kMid;      // 1024 x 7168 x 2048 36 for 47; 512 x 7168 x 2048 35 for 29
  } else {
    // 192 x 2112 x 7168 20.8 for 24.2; 384 x 2112 x 7168 28.9 for 33.9
    t.cfg = rows <= 256 ? kLow : kHigh;
  }
  t.bm = kBm[t.cfg];
  t.bn = kBn[t.cfg];
  t.threads = kThreads[t.cfg];
  t.persistent = t.cfg == kBig;
  t.splits = 1;
  if (dense && t.cfg != kBig && t.cfg != kFew) {
    // One workgroup a CU; two where several row tiles read the same weights
    // (64 x 2112 x 7168 14.1 in 6 splits, 16.2 in 12; 128 x 2112 x 7168 18.9
    // in 6, 19.8 in 3), and five steps a split at least.
    const int64_t u = units(t.cfg), steps = (p.K + kBK - 1) / kBK;
    if (4 * u < 3 * cus && u <= kSplitKMaxTiles) {
      int64_t s = (rows > t.bm ? 2 * cus : cus) / u;
      if (s > steps / 5) s = steps / 5;
      if (s > kBfMaxSplits) s = kBfMaxSplits;
      if (s > 1) t.splits = (int)s;
    }
  }
  return t;
}

size_t bf16_workspace_bytes(const BfProblem& p, int cus) {
  const BfTile t = bf16_tile(p, cus);
  if (t.splits <= 1) return 0;
  const size_t tiles = (size_t)((p.M + t.bm - 1) / t.bm) * ((p.N + t.bn - 1) / t.bn);
  return kSplitKCounterBytes + tiles * t.splits * t.bm * t.bn * 4;
}

hipError_t launch_bf16(BfProblem p, const BfTile& t, hipStream_t stream) {
  p.splits = t.splits;
  if (p.mode == kBfRowRuns)
    return p.b_kmajor ? launch_tile<false, true, kBfRowRuns>(p, t, stream)
                      : launch_tile<false, false, kBfRowRuns>(p, t, stream);
  if (p.mode == kBfKRuns) return launch_tile<true, true, kBfKRuns>(p, t, stream);
  if (p.a_kmajor) return launch_tile<true, true, kBfDense>(p, t, stream);
  return p.b_kmajor ? launch_tile<false, true, kBfDense>(p, t, stream)
                    : launch_tile<false, false, kBfDense>(p, t, stream);
}

}  // namespace fg8

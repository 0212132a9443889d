// Weights in 4 bits with group scales: quantize, dequantize, and products with
// few rows of BF16, dense or over ragged row runs.
//
//   s = fl32(amax / 7) of GROUP consecutive k of a row (1 where that is 0),
//   rounded to the scales' type;  code = rne(fl32(w / s) within -7 .. 7) + 8;  value (code - 8) s
//   codes [n][k / 2], element 2 j in the low half of byte j; scales [k / GROUP][n]
//
//   D[m][n] = sum over groups of s[group][n] * sum over its k of (code - 8) x[m][k]
//
// The product reads half a byte a weight and little else: HBM bounds it (1 x 16384 x
// 16384 27 us, 5.1 TB/s of codes and scales), the launch and one round trip a
// step where the weights are few (1 x 2112 x 7168, four steps, 7 us; 1 x 24576 x 1536,
// two, 8.5 for 3.9 us of bytes), and with more rows the copies of x that
// every workgroup makes (13 x 7168 x 16384 26 us, 2.9 TB/s: 24.9 without the
// arithmetic, 16 without the copies; 512 rows over 32 experts, gated, 2 x 2048 x 7168
// 116-124, 3.9 TB/s).
#include "bf16_tile.h"

namespace fg8 {

namespace {

// ------------------------------------------------------- few-row products
// A workgroup is WK x WN waves.  A wave owns 16 TM rows by 16 TN weight rows (its
// place among the WN) and every WK-th chunk of 256 k, a 128-byte line of codes a
// row; the WK waves' sums meet in LDS at the end.  Codes, scales and x of a chunk
// are copied from global memory straight into LDS, a chunk ahead: what is in flight
// takes no registers, and nothing waits for it but one counter.  (A second chunk
// ahead takes the LDS of another workgroup: 4 x 24576 x 2048 16.4 us for 12.0.)
// Codes and scales are the wave's own; x is shared by the WN waves of a chunk (a
// barrier a chunk, none where WN is 1).
//
// A lane reads 16 bytes of codes, 32 k of one weight row; four swaps between the
// four groups of sixteen lanes turn that into the layout of four MFMAs of 32 k
// each (lane i + 16 g: row i, k = 8 g .. 8 g + 7), so a group of 32 k or more is
// whole MFMAs.  A code goes into the upper four mantissa bits of a BF16 whose
// exponent is 16's: 16 + code, one product and one bit operation for two weights.
// The 24 that every weight is too large is taken off with an MFMA against a
// constant -24, once for all the tiles that share x: the group's sum then starts
// from -24 sum(x).  Every value and product is exact; what the detour adds is
// FP32 rounding of partial sums at the size of 24 |x| for 8 |x|.  x goes in as the
// first operand, so a lane holds rows of one weight column and needs one scale.
struct Int4Problem {
  BfProblem p;             // a: x; N: weight rows; d, epilogue, runs
  const uint8_t* codes;
  const void* scales;
};

// The copies of bf16_tile.h with the non-temporal hint (weights are read once),
// and of four bytes a lane.
__device__ __forceinline__ void copy16_nt(v4i rsrc, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen nt lds"
               :
               : "v"(off), "s"(rsrc), "s"(lds)
               : "memory", "m0");
}
__device__ __forceinline__ void copy4(v4i rsrc, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
               :
               : "v"(off), "s"(rsrc), "s"(lds)
               : "memory", "m0");
}

// A lane holds column i's scale of group g of four, or of group g / 2 of two; this
// hands every lane all of them.
template <int NG>
__device__ __forceinline__ void spread_scales(uint32_t v, float* s) {
  typedef unsigned u2 __attribute__((ext_vector_type(2)));
  const u2 a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  if constexpr (NG == 2) {
    s[0] = __uint_as_float(a[0]);
    s[1] = __uint_as_float(a[1]);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u2 b = __builtin_amdgcn_permlane16_swap(a[h], a[h], false, false);
      s[2 * h] = __uint_as_float(b[0]);
      s[2 * h + 1] = __uint_as_float(b[1]);
    }
  }
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

// Eight codes as BF16 16 + code, two a byte: a byte times 2^15 + 2^3 has its low
// half in bits 3 .. 6 and its high half in bits 19 .. 22.  The constants come from
// registers: as literals they keep the two bit operations apart.
struct CodeBits {
  uint32_t mask = 0x00780078u, sixteen = 0x41804180u, twice = 0x8008u;
  __device__ CodeBits() { asm("" : "+s"(mask), "+v"(sixteen), "+v"(twice)); }
  __device__ v8bf plus_16(uint32_t w) const {
    v4i v;
#pragma unroll
    for (int p = 0; p < 4; ++p) v[p] = (int)((__umul24(w >> (8 * p) & 255u, twice) & mask) | sixteen);
    return __builtin_bit_cast(v8bf, v);
  }
};

// XR: rows of x that are copied (the least that hold the tile's rows).
constexpr int kChunk = 256, kStages = 2;
template <int TM_, int XR_, int TN_, int WK_, int WN_>
struct I4Cfg {
  static constexpr int TM = TM_, XR = XR_, TN = TN_, WK = WK_, WN = WN_;
  static constexpr int WAVES = WK * WN, THREADS = 64 * WAVES, BM = 16 * TM, BN = 16 * TN * WN;
  static constexpr int CODES = WAVES * TN * 2048, X = WK * XR * 512;
  static constexpr int XCOPIES = XR / 2 / WN;          // of 1 KB, a wave's of a chunk
  static constexpr int scale_copies(int group) { return kChunk / group > 4 ? 2 : 1; }
  static constexpr int stage(int group) { return CODES + WAVES * TN * 256 * scale_copies(group) + X; }
  static_assert(XR / 2 % WN == 0 && XR >= 2 && (XR == 16 * TM || (TM == 1 && XR < 16)), "every wave copies the same number");
};

template <class C, int GROUP, bool SBF16>
__global__ __launch_bounds__(C::THREADS) void int4_kernel(Int4Problem q) {
  constexpr int TM = C::TM, TN = C::TN, WK = C::WK, WN = C::WN;
  constexpr int NG = 128 / GROUP, GJ = GROUP / 32;      // groups of 128 k, MFMAs of a group
  constexpr int GC = 2 * NG, SC = C::scale_copies(GROUP);     // groups of a chunk, copies of their scales
  constexpr int STAGE = C::stage(GROUP), SCALES = C::WAVES * TN * 256 * SC;
  static_assert(C::WAVES * TM * TN * 1024 <= kStages * STAGE && kStages * STAGE <= kLdsBytes, "sums in the stages, stages in the LDS");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kStages * STAGE];
  const BfProblem& p = q.p;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kg = wave / WN, wn = wave % WN, i = lane & 15, g = lane >> 4;
  BfUnit w;
  if (!(p.mode == kBfRowRuns ? find_unit<C::BM, C::BN, kBfRowRuns>(p, lane, w) : find_unit<C::BM, C::BN, kBfDense>(p, lane, w)))
    return;
  const bool gated = p.kind == kKindGated;
  const int N = p.N, K = p.K, half = N / 2;
  const int64_t expert = max(w.g, 0), row_bytes = K / 2;

  // Weight row that tile t of this wave starts at (gated: the first half of the
  // tiles are gate rows, the others the up rows of the same columns).
  auto row_of = [&](int t) {
    if (!gated) return w.n0 + 16 * (wn * TN + t);
    const int j = w.n0 / 2 + 16 * (wn * (TN / 2) + (t < TN / 2 ? t : t - TN / 2));
    return t < TN / 2 ? j : half + j;
  };
  // Sources of the copies.  A row of codes is eight pieces of 16 bytes, a row of x 32;
  // a copy of 1 KB is whole rows, piece l of it lane l's.  In LDS the pieces of a row
  // are XORed with a function of it, which keeps the reads free of bank conflicts.
  // Rows that do not exist, and k past the end, are no address.
  const char* cfrom[TN];               // at this wave's chunk of the step to copy next
  uint32_t coff[TN][2];
  int cpart[2], col[TN];              // first k of a lane's piece in the chunk; its column of scales
#pragma unroll
  for (int h = 0; h < 2; ++h) cpart[h] = ((lane & 7) ^ swz(8 * h + (lane >> 3))) * 32;
#pragma unroll
  for (int t = 0; t < TN; ++t) {
    const int r = uniform(row_of(t));
    cfrom[t] = (const char*)q.codes + (expert * N + (r < N ? r : 0)) * row_bytes + kg * (kChunk / 2);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = 8 * h + (lane >> 3);
      coff[t][h] = row < N - r ? (uint32_t)(row * (int)row_bytes + cpart[h] / 2) : kNowhere;
    }
    col[t] = r + i;
  }
  const char* xfrom = (const char*)(p.a + w.m0 * p.lda) + kg * (kChunk * 2);
  uint32_t xoff[C::XCOPIES];
  int xpart[C::XCOPIES];
#pragma unroll
  for (int u = 0; u < C::XCOPIES; ++u) {
    const int r = (wn * C::XCOPIES + u) * 2 + (lane >> 5), piece = (lane & 31) ^ (r & 15);
    xoff[u] = r < w.rows ? (uint32_t)(r * (int)p.lda + piece * 8) * 2 : kNowhere;
    xpart[u] = piece * 8;
  }
  // Scales: elements from the expert's first on, copied as the dwords that hold them
  // (two BF16 ones each).  The very last of an odd number of BF16 ones is in no whole
  // dword and is kept aside.  A lane's copy u holds column i's of group 4 u + g of the
  // chunk, or of group g / 2 where a chunk has two.
  constexpr int SIZE = SBF16 ? 2 : 4;
  const int64_t per_expert = (int64_t)N * (K / GROUP), all = per_expert * (p.mode == kBfRowRuns ? p.groups : 1);
  const int group0 = GC == 2 ? g >> 1 : g, last_group = K / GROUP - 1;
  const bool odd_end = SBF16 && (all & 1) && (expert + 1) * per_expert == all;
  uint32_t slast = 0;
  if (odd_end) slast = (uint32_t)((const uint16_t*)q.scales)[all - 1] << 16;
  int64_t sfrom = expert * per_expert + (int64_t)kg * GC * N;      // of the step to copy next
  const int odd = SBF16 ? (int)(sfrom & 1) : 0;                    // (a chunk has an even number of groups)
  int cnext = kg, next_slot = 0, rem_next = w.ks - kg * kChunk;

  const int chunks = (w.ks + kChunk - 1) / kChunk, steps = (chunks + WK - 1) / WK;
  const uint32_t lds0 = lds_addr(smem);
  auto all_of = [](const char* from) { return resource(from, 0x7fffffff); };
  auto issue_as = [&](auto whole) {
    constexpr bool WHOLE = decltype(whole)::value;      // all of the chunk's k exist
    const uint32_t st = uniform(lds0 + (uint32_t)(next_slot * STAGE));
    const int rem = rem_next;          // k from this chunk on
#pragma unroll
    for (int t = 0; t < TN; ++t) {
      const v4i rs = all_of(cfrom[t]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        copy16_nt(rs, WHOLE || cpart[h] < rem ? coff[t][h] : kNowhere, uniform(st + (uint32_t)((wave * TN + t) * 2 + h) * 1024));
      cfrom[t] += WK * (kChunk / 2);
    }
    const v4i srs = all_of((const char*)q.scales + (sfrom - odd) * SIZE);
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
      for (int u = 0; u < SC; ++u) {
        const int grp = 4 * u + group0;
        uint32_t o = (uint32_t)((odd + grp * N + col[t]) * SIZE) & ~3u;
        if (odd_end && cnext * GC + grp == last_group && col[t] == N - 1) o = kNowhere;
        copy4(srs, (WHOLE || grp * GROUP < rem) && col[t] < N ? o : kNowhere,
              uniform(st + C::CODES + (uint32_t)((wave * TN + t) * SC + u) * 256));
      }
    sfrom += (int64_t)(WK * GC) * N;
    const v4i xrs = all_of(xfrom);
#pragma unroll
    for (int u = 0; u < C::XCOPIES; ++u)
      copy16(xrs, WHOLE || xpart[u] < rem ? xoff[u] : kNowhere,
             uniform(st + C::CODES + SCALES + (uint32_t)(kg * C::XR * 512 + (wn * C::XCOPIES + u) * 1024)));
    xfrom += WK * (kChunk * 2);
    rem_next -= WK * kChunk;
    cnext += WK;
    next_slot ^= 1;
  };
  auto issue = [&] {
    if (rem_next >= kChunk) issue_as(std::true_type{});
    else issue_as(std::false_type{});
  };

  v4f acc[TM][TN];
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int t = 0; t < TN; ++t) acc[m][t] = v4f{0.f, 0.f, 0.f, 0.f};
  const v8bf minus24 = __builtin_bit_cast(v8bf, v4i{(int)0xC1C0C1C0u, (int)0xC1C0C1C0u, (int)0xC1C0C1C0u, (int)0xC1C0C1C0u});
  const CodeBits bits;
  int slot = 0, cnow = kg;
  auto multiply = [&] {
    const uint8_t* st = smem + slot * STAGE;
    const uint8_t* xs = st + C::CODES + SCALES + kg * C::XR * 512;
    uint32_t sraw[TN][SC];
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
      for (int u = 0; u < SC; ++u)
        sraw[t][u] = *reinterpret_cast<const uint32_t*>(st + C::CODES + ((wave * TN + t) * SC + u) * 256 + lane * 4);
    // all the codes and x out of LDS before any of them is used
    v4i codes[2][TN], raw[2][TM][4];
    auto read = [&](int h) {
#pragma unroll
      for (int t = 0; t < TN; ++t)
        codes[h][t] = *reinterpret_cast<const v4i*>(st + (wave * TN + t) * 2048 + i * 128 + (((4 * h + g) ^ swz(i)) << 4));
#pragma unroll
      for (int m = 0; m < TM; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = (16 * m + i) & (C::XR - 1);
          raw[h][m][j] = *reinterpret_cast<const v4i*>(xs + r * 512 + (((16 * h + 4 * j + g) ^ (r & 15)) << 4));
        }
    };
    read(0);
    read(1);
    __builtin_amdgcn_sched_barrier(0);
    float s[TN][GC];
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
      for (int u = 0; u < SC; ++u) {
        uint32_t v = sraw[t][u];
        const int grp = 4 * u + group0;
        if constexpr (SBF16) {
          v = (odd + grp * N + col[t]) & 1 ? v & 0xffff0000u : v << 16;
          if (odd_end && cnow * GC + grp == last_group && col[t] == N - 1) v = slast;
        }
        spread_scales<GC == 2 ? 2 : 4>(v, s[t] + 4 * u);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int t = 0; t < TN; ++t) transpose_words(codes[h][t]);
#pragma unroll
      for (int e = 0; e < NG; ++e) {
        v8bf x[TM][GJ];
        v4f start[TM], part[TM][TN];
#pragma unroll
        for (int m = 0; m < TM; ++m) {
          start[m] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < GJ; ++j) {
            x[m][j] = __builtin_bit_cast(v8bf, raw[h][m][e * GJ + j]);
            start[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[m][j], minus24, start[m], 0, 0, 0);
          }
        }
#pragma unroll
        for (int j = 0; j < GJ; ++j)
#pragma unroll
          for (int t = 0; t < TN; ++t) {
            const v8bf v = bits.plus_16((uint32_t)codes[h][t][e * GJ + j]);
#pragma unroll
            for (int m = 0; m < TM; ++m)
              part[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[m][j], v, j ? part[m][t] : start[m], 0, 0, 0);
          }
#pragma unroll
        for (int t = 0; t < TN; ++t)
#pragma unroll
          for (int m = 0; m < TM; ++m)
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[m][t][v] = fmaf(s[t][h * NG + e], part[m][t][v], acc[m][t][v]);
      }
    }
    slot ^= 1;
    cnow += WK;
  };
  if (steps > 0) {
    issue();
    for (int step = 0; step < steps; ++step) {
      wait_vmcnt<0>();                        // this step's copies
      if constexpr (WN > 1) __syncthreads();
      else asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      issue();                                // over the last step's, which everybody has read
      multiply();
    }
  }
  wait_vmcnt<0>();
  __syncthreads();

  // The sums over the WK waves.  Lane i + 16 g has column i of rows 4 g .. 4 g + 3;
  // here it takes columns 4 g .. 4 g + 3 of row i.
  v4f* sums = reinterpret_cast<v4f*>(smem);     // [wave][tile][lane]
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int t = 0; t < TN; ++t) sums[(wave * TM * TN + m * TN + t) * 64 + lane] = acc[m][t];
  __syncthreads();
  auto sum_of = [&](int n, int m, int t) {      // of the n-th of the WN waves
    const int from = (4 * g + 16 * (i >> 2)) * 4 + (i & 3);
    v4f v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < WK; ++u) {
      const float* f = reinterpret_cast<const float*>(sums + ((u * WN + n) * TM * TN + m * TN + t) * 64) + from;
      v += v4f{f[0], f[4], f[8], f[12]};
    }
    return v;
  };
  if (gated) {
    if constexpr (TN > 1) {
      for (int u = wave; u < TM * WN * (TN / 2); u += C::WAVES) {
        const int m = u / (WN * (TN / 2)), pair = u % (WN * (TN / 2)), n = pair / (TN / 2), t = pair % (TN / 2);
        v4f gate[1] = {sum_of(n, m, t)}, up[1] = {sum_of(n, m, TN / 2 + t)};
        GatedOut<1>(p, w, C::BM, C::BN, 32 * pair, nullptr, lane).rows16(16 * m, gate, up);
      }
    }
  } else {
    const BfOut out(p, w.g);
    for (int u = wave; u < TM * WN * TN; u += C::WAVES) {
      const int m = u / (WN * TN), t = u % (WN * TN), r = 16 * m + i;
      const v4f v = sum_of(t / TN, m, t % TN);
      if (r < w.rows) out.four(w.m0 + r, w.n0 + 16 * t + 4 * g, v);
    }
  }
}

// TM, XR, TN, WK, WN
enum { kI4One = 0, kI4OneWide, kI4Four, kI4FourWide, kI4Row, kI4RowWide, kI4Runs, kI4Many };
using I4One = I4Cfg<1, 2, 1, 8, 1>;
using I4OneWide = I4Cfg<1, 2, 2, 4, 1>;
using I4Four = I4Cfg<1, 4, 1, 8, 1>;
using I4FourWide = I4Cfg<1, 4, 2, 4, 1>;
using I4Row = I4Cfg<1, 16, 1, 4, 2>;
using I4RowWide = I4Cfg<1, 16, 2, 2, 2>;
using I4Runs = I4Cfg<1, 16, 2, 1, 4>;
using I4Many = I4Cfg<2, 32, 2, 1, 4>;

template <class C>
hipError_t start(const Int4Problem& q, int group, bool sbf16, unsigned grid, hipStream_t stream) {
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(C::THREADS), 0, stream, q);
    return hipGetLastError();
  };
  if (group == 32) return sbf16 ? go(int4_kernel<C, 32, true>) : go(int4_kernel<C, 32, false>);
  if (group == 64) return sbf16 ? go(int4_kernel<C, 64, true>) : go(int4_kernel<C, 64, false>);
  return sbf16 ? go(int4_kernel<C, 128, true>) : go(int4_kernel<C, 128, false>);
}

template <class F>
auto with_config(int cfg, F f) {
  switch (cfg) {
    case kI4One: return f(I4One{});
    case kI4OneWide: return f(I4OneWide{});
    case kI4Four: return f(I4Four{});
    case kI4FourWide: return f(I4FourWide{});
    case kI4Row: return f(I4Row{});
    case kI4RowWide: return f(I4RowWide{});
    case kI4Runs: return f(I4Runs{});
    default: return f(I4Many{});
  }
}

}  // namespace

// (times in us, the choice first; 256 CUs)
Int4Tile int4_tile(const BfProblem& p, int cus) {
  Int4Tile t{};
  const bool runs = p.mode == kBfRowRuns, pairs = p.kind == kKindGated;     // (gate and up: two tiles a wave at least)
  const int64_t rows = runs ? (p.M + p.groups - 1) / p.groups : p.M;
  // 64 columns a workgroup fill the device
  const bool wide = (rows + 15) / 16 * ((int64_t)p.N + 63) / 64 >= cus;
  if (runs) {
    // One row tile a run while most runs fit it: 512 rows over 32 experts of 4096 x
    // 7168 (gated) 124 for 129, 128 rows 87 for 104, 1280 rows 234 for 189.
    t.cfg = rows <= 24 ? kI4Runs : kI4Many;
  } else if (rows <= 4) {
    // One tile a wave and eight waves on k where columns are few, two tiles and four
    // waves where they are many or k is short: 1 x 7168 x 16384 15.3 for 19.2, 1 x
    // 2112 x 7168 7.0 for 9.2, 1 x 4096 x 2048 4.6 for 5.1; 1 x 16384 x 16384 28.5 for
    // 26.3, 1 x 7168 x 2048 6.2 for 5.8, 1 x 24576 x 1536 14.4 for 8.7.  Copying two
    // rows of x, not four, leaves room for another workgroup.
    const bool narrow = !pairs && !wide && (p.K > 4096 || p.N <= 16 * cus);
    t.cfg = rows <= 2 ? (narrow ? kI4One : kI4OneWide) : (narrow ? kI4Four : kI4FourWide);
  } else if (rows <= 64) {
    // 16 x 16384 x 8192 22.4 for 25.4, 32 x 8192 x 8192 19.1 for 23.4, 48 x 16384 x
    // 4096 24 for 41; 24 x 4096 x 7168 17.5 for 11.7, 13 x 7168 x 16384 35 for 25
    t.cfg = pairs || wide ? kI4RowWide : kI4Row;
  } else {
    t.cfg = kI4Many;
  }
  with_config(t.cfg, [&](auto c) {
    typedef decltype(c) C;
    t.threads = C::THREADS;
    t.units = (((int64_t)p.M + C::BM - 1) / C::BM + (runs ? p.groups + 1 : 0)) * (((int64_t)p.N + C::BN - 1) / C::BN);
    return 0;
  });
  return t;
}

hipError_t launch_int4(const BfProblem& p, const Int4Tile& t, const uint8_t* codes, const void* scales, bool scales_bf16,
                       int group, hipStream_t stream) {
  const Int4Problem q{p, codes, scales};
  const unsigned grid = (unsigned)((t.units + 7) / 8 * 8);
  return with_config(t.cfg, [&](auto c) { return start<decltype(c)>(q, group, scales_bf16, grid, stream); });
}

// ------------------------------------------------- quantize and dequantize
namespace {

// Bound by HBM: 32 x 4096 x 7168 BF16 weights 400 us (5.9 TB/s) and back 455 (5.3);
// 2112 x 7168 10 and 8 us.
// A workgroup owns 16 rows x 512 k: a wave reads 512 k of a row, eight a lane, four
// rows in all (eight rows a wave: 13 us for 11).  Scales lie [group][row] in memory
// and cross in LDS, so that they are written and read as runs of 16 rows.
constexpr int kQuantRows = 16, kQuantCols = 512;

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
  const int here = (int)min(rows - r0 - wave * PER, (int64_t)PER);     // this wave's rows
  w += (r0 + wave * PER) * cols + c;
  q += ((r0 + wave * PER) * cols + c) / 2;
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    if (u < here && c < cols) {
      load_eight(w + u * cols, f[u]);
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
    // numbers; one addition then rounds it to the code, 8 on top.  A scale that is a
    // normal number is 2^-8 below amax / 7 at most, and no quotient rounds past 7; one
    // of few bits may be far below it (amax of 10 smallest steps: a scale of 1), so
    // there the quotient is limited (a NaN, beside a NaN for the scale, to -7).
    uint32_t code = 0;
    auto put = [&](int e, float t) { code |= (__float_as_uint(t + (12582912.f + 8.f)) & 15u) << (4 * e); };
    if (__all(s > 0x1p-100f && s < 0x1p100f)) {
      const float r = __fdiv_rn(1.f, s);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float t = f[u][e] * r;
        put(e, fmaf(fmaf(-t, s, f[u][e]), r, t));
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) put(e, fminf(fmaxf(__fdiv_rn(f[u][e], s), -7.f), 7.f));
    }
    if (u < here && c < cols) store_nt(q + u * (cols / 2), code);
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

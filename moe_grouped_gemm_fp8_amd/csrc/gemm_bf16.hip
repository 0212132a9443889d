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
// and the gated form of the first one, dense or over row runs: B is 2 n rows,
// gate rows over up rows, D[m][j] = act(sum of gate row j) * (sum of up row j).
// A tile's columns are then half gate rows, half the up rows of the same j, laid
// so that one wave holds both sums of its columns.
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
// A gated product runs at the rate of the plain one of 2 n columns (8192 x 4096 x
// 7168: 312 us for 311, with z 323 for 311), and so do a head's logits with
// their statistics (8192 x 128000 x 7168: 10.3 to 10.9 ms, 1380 to
// 1460 TFLOP/s).
#include "bf16_tile.h"

namespace fg8 {

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;


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

// B's tile of a gated product (k-contiguous): the columns that a wave owns, WN of
// the tile's BX, are WN / 2 gate rows and then the up rows of the same columns of
// h.  A copy of 1 KB lies in one of the two.
template <int BX, int WN, int WAVES, int DEPTH>
struct GatedOperand {
  typedef Operand<false, BX, WAVES, DEPTH> Plain;
  static constexpr int COPIES = Plain::COPIES, PER = Plain::PER, PITCH = Plain::PITCH, HALF = WN / 2;
  static constexpr bool EVEN = Plain::EVEN;
  static_assert(HALF % (1024 / PITCH) == 0, "a copy's rows are all gate or all up");

  const char* base;      // gate row j0 at the first k
  int64_t up;            // bytes from there to up row j0
  int64_t left;          // bytes of either's rows before the last one
  uint32_t off[PER];
  int rem_k;

  __device__ static bool is_up(int copy) { return copy * (1024 / PITCH) % WN >= HALF; }

  // j0: the tile's first column of h; js: columns from there (>= 1) of n
  __device__ void init(const uint16_t* p, int64_t ld_elems, int64_t j0, int js, int64_t n, int64_t k0, int ks,
                       int wave, int lane) {
    const int64_t ld = ld_elems * 2;
    rem_k = ks;
    base = (const char*)(p + j0 * ld_elems + k0);
    up = n * ld;
    left = (int64_t)((js < BX / 2 ? js : BX / 2) - 1) * ld;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = (wave + i * WAVES) * 1024 + lane * 16;
      const int r = at / PITCH, c = (at % PITCH / 16) ^ Plain::chunk_xor(r);
      off[i] = (uint32_t)((r / WN * HALF + r % HALF) * ld) + c * 16;
    }
  }
  __device__ void issue(int kt, uint32_t lds, int wave, int lane) const {
    const int rem = rem_k - kt * DEPTH;
    const char* from = base + (int64_t)kt * (DEPTH * 2);
    const int64_t bytes = left + (int64_t)((rem + 7) & ~7) * 2;
    const v4i gate = resource(from, bytes), above = resource(from + up, bytes);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (EVEN || wave + i * WAVES < COPIES) {
        const int at = (wave + i * WAVES) * 1024 + lane * 16;
        const int c = (at % PITCH / 16) ^ Plain::chunk_xor(at / PITCH);
        copy16(is_up(wave + i * WAVES) ? above : gate, c * 8 < rem ? off[i] : kNowhere,
               uniform(lds + (uint32_t)(wave + i * WAVES) * 1024));
      }
  }
  __device__ static v8bf frag(const uint8_t* tile, int x, int kk, int lane) { return Plain::frag(tile, x, kk, lane); }
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
template <class C, bool AK, bool BK, int MODE, bool ADD = false, int KIND = kKindTile>
__global__ __launch_bounds__(C::THREADS, C::OCC) void bf16_kernel(BfProblem p) {
  constexpr bool GATED = KIND == kKindGated;
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
    typedef std::conditional_t<GATED, GatedOperand<C::BN, C::WN, C::WAVES, C::DEPTH>,
                               Operand<BK, C::BN, C::WAVES, C::DEPTH>> OpB;
    OpA a;
    OpB b;
    a.init(p.a, p.lda, w.m0, w.rows, w.k0, w.ks, wave, lane);
    const uint16_t* pb = p.b + (MODE == kBfRowRuns ? w.g * p.b_stride : 0);
    if constexpr (GATED) b.init(pb, p.ldb, w.n0 / 2, (p.N - w.n0) / 2, p.N / 2, w.k0, w.ks, wave, lane);
    else b.init(pb, p.ldb, w.n0, p.N - w.n0, w.k0, w.ks, wave, lane);
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

  if constexpr (GATED) {
    constexpr int COLS = C::TN / 2;
    typedef GatedOut<COLS> Out;
    static_assert(C::WAVES * Out::kTurn <= C::STAGES * C::STAGE_BYTES, "rows turn in the stages");
    __syncthreads();      // every wave is done with the stages
    const Out out(p, w, C::BM, C::BN, wn0, smem + wave * Out::kTurn, lane);
#pragma unroll
    for (int i = 0; i < C::TM; ++i) {
      v4f gate[COLS], up[COLS];
#pragma unroll
      for (int t = 0; t < COLS; ++t) {
        gate[t] = acc[i][t];
        up[t] = acc[i][COLS + t];
      }
      out.rows16(wm0 + 16 * i, gate, up);
    }
  } else if constexpr (KIND != kKindTile) {
    typedef LossOut<KIND, C::TM> Out;
    static_assert(C::WN == 64 && C::WAVES * Out::kTurn <= C::STAGES * C::STAGE_BYTES && C::WM * 8 <= Out::kTurn);
    Out out(p, w, C::BM, C::BN, wn0, smem + wave * Out::kTurn, lane);
    out.fetch(wm0);
    __syncthreads();      // every wave is done with the stages
#pragma unroll
    for (int i = 0; i < C::TM; ++i) out.rows16(i, wm0 + 16 * i, acc[i]);
    if constexpr (KIND == kKindLse) {
      __syncthreads();
      // (waves w and w + WAVES_M hold the same rows; the first WAVES_M join them)
      if (wave < C::WAVES_M)
        for (int r = lane; r < C::WM; r += 64)
          Out::template merge<C::WAVES_N>(p, w, smem + wave * Out::kTurn, C::WAVES_M * Out::kTurn, r, wm0, C::BN);
    }
  } else if constexpr (C::WN == 64) {
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
template <int MODE, bool GATED = false>
__global__ __launch_bounds__(512, 2) void bf16_few_kernel(BfProblem p) {
  constexpr int U = GATED ? 3 : 4;       // steps of a batch; two batches in flight
  constexpr int SETS = GATED ? 2 : 1;    // rows of B for a column: gate and up
  __shared__ v4f sums[8][SETS][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  BfUnit w;
  if (!find_unit<16, 16 * SETS, MODE>(p, lane, w)) return;
  const int i = lane & 15, g = lane >> 4;
  const int n0 = w.n0 / SETS, N = p.N / SETS;

  // Offsets of a lane's row in either tile; rows and columns past the end read
  // the last one and are not stored.  k goes into the scalar offset, and a
  // lane whose k lies past the end loads zeros.
  const uint16_t* xp = p.a + w.m0 * p.lda;
  const uint16_t* wp = p.b + (MODE == kBfRowRuns ? max(w.g, 0) * p.b_stride : 0) + (int64_t)n0 * p.ldb;
  const __amdgpu_buffer_rsrc_t xr = buffer_rsrc(uniform((const void*)xp), 0x7fffffff);
  const __amdgpu_buffer_rsrc_t wr = buffer_rsrc(uniform((const void*)wp), 0x7fffffff);
  const uint32_t xo = (uint32_t)(min(i, w.rows - 1) * (int)p.lda + 8 * g) * 2;
  const __amdgpu_buffer_rsrc_t ur = buffer_rsrc(uniform((const void*)(wp + (int64_t)N * p.ldb)), 0x7fffffff);
  const uint32_t wo = (uint32_t)(min(i, N - 1 - n0) * (int)p.ldb + 8 * g) * 2;
  struct Batch {
    v4i x[U][2], w[SETS][U][2];
  };
  auto fetch = [&](Batch& f, int s0) {     // steps s0, s0 + 8, ..
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const int k = uniform((s0 + 8 * u) * kBK + 32 * kk);
        const bool in = 8 * g < w.ks - k;
#pragma unroll
        for (int s = 0; s < SETS; ++s)
          f.w[s][u][kk] = __builtin_bit_cast(
              v4i, __builtin_amdgcn_raw_buffer_load_b128(s ? ur : wr, in ? wo : kNowhere, k * 2, kStream));
        f.x[u][kk] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(xr, in ? xo : kNowhere, k * 2, 0));
      }
  };
  v4f acc[SETS];
#pragma unroll
  for (int s = 0; s < SETS; ++s) acc[s] = v4f{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const Batch& f) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int s = 0; s < SETS; ++s)
          acc[s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, f.w[s][u][kk]),
                                                           __builtin_bit_cast(v8bf, f.x[u][kk]), acc[s], 0, 0, 0);
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
#pragma unroll
  for (int s = 0; s < SETS; ++s) sums[wave][s][lane] = acc[s];
  __syncthreads();
  if (wave == 0) {
    v4f sum[SETS][1];
#pragma unroll
    for (int s = 0; s < SETS; ++s) {
      sum[s][0] = sums[0][s][lane];
#pragma unroll
      for (int v = 1; v < 8; ++v) sum[s][0] += sums[v][s][lane];
    }
    if constexpr (GATED) GatedOut<1>(p, w, 16, 32, 0, nullptr, lane).rows16(0, sum[0], sum[1]);
    else if (i < w.rows) BfOut(p, w.g).four(w.m0 + i, w.n0 + 4 * g, sum[0][0]);
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

// B's halves of a gated product: half 0 is 128 gate rows, half 1 the up rows of
// the same columns of h, so that a wave's two halves are both sums of its columns.
struct GatedHalf {
  typedef HalfTile<false, 32> Plain;
  typedef Plain::Frag Frag;
  static constexpr int BYTES = Plain::BYTES, COPIES = Plain::COPIES, PITCH = Plain::PITCH;

  const char* base;            // gate row j0 at the first k
  int64_t up, left;            // bytes to up row j0; of either's rows before the last one
  uint32_t off[COPIES];
  int rem_k;

  __device__ void init(const uint16_t* p, int64_t ld_elems, int64_t j0, int js, int64_t n, int64_t k0, int ks,
                       int wave, int lane) {
    const int64_t ld = ld_elems * 2;
    rem_k = ks;
    base = (const char*)(p + j0 * ld_elems + k0);
    up = n * ld;
    left = (int64_t)((js < 128 ? js : 128) - 1) * ld;
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
      const int at = (wave * COPIES + i) * 1024 + lane * 16, r = at / PITCH;
      off[i] = (uint32_t)(r * ld) + (((at % PITCH / 16) ^ swz(r)) << 4);
    }
  }
  __device__ void issue(int kt, int h, uint32_t lds, int wave, int lane) const {
    const int rem = rem_k - kt * kBK;
    const int64_t bytes = left + (int64_t)((rem + 7) & ~7) * 2;
    const v4i rs = resource(base + (h ? up : 0) + (int64_t)kt * (kBK * 2), rem > 0 ? bytes : 0);
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
      const int c = (lane & 7) ^ (4 * i + (lane >> 4));
      copy16(rs, c * 8 < rem ? off[i] : kNowhere, uniform(lds + (uint32_t)(wave * COPIES + i) * 1024));
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
template <bool AK, bool BK, int MODE, bool EPI, bool ADD = false, int KIND = kKindTile>
__global__ __launch_bounds__(512, 2) void bf16_big_kernel(BfProblem p) {
  constexpr bool GATED = KIND == kKindGated, LOSS = KIND == kKindLse || KIND == kKindDlogits;
  typedef HalfTile<AK, 64> HalfA;
  typedef std::conditional_t<GATED, GatedHalf, HalfTile<BK, 32>> HalfB;
  typedef std::conditional_t<GATED, GatedOut<2>, std::conditional_t<LOSS, LossOut<KIND, 8>, TileOut<EPI, ADD>>> Out;
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
  // dx of a head in parts of its classes: each part's sums are an output of their own
  constexpr bool PARTS = MODE == kBfDense && !AK && BK;
  const int total = mt * nt * (MODE == kBfKRuns ? p.groups : PARTS ? p.splits : 1), G = p.grid;

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
      const int part = MODE == kBfKRuns || PARTS ? id / (mt * nt) : 0;
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
      if constexpr (PARTS) {
        const int steps = (p.K + kBK - 1) / kBK;
        const int s0 = (int)((int64_t)part * steps / p.splits), s1 = (int)((int64_t)(part + 1) * steps / p.splits);
        w.k0 = s0 * kBK;
        w.ks = min(p.K, s1 * kBK) - s0 * kBK;
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
    const uint16_t* pb = p.b + (MODE == kBfRowRuns ? w.g * p.b_stride : 0);
    if constexpr (GATED) b.init(pb, p.ldb, w.n0 / 2, (p.N - w.n0) / 2, p.N / 2, w.k0, w.ks, wave, here);
    else b.init(pb, p.ldb, w.n0, p.N - w.n0, w.k0, w.ks, wave, here);
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
    if constexpr (LOSS) {
      out.fetch(grp * 128);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        asm volatile("" : "+v"(out.target[i]));
        if constexpr (KIND == kKindDlogits) asm volatile("" : "+v"(out.lse[i]), "+v"(out.dloss[i]));
      }
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
      if constexpr (GATED) {
        v4f gate[2] = {acc[ha][i][0][0], acc[ha][i][0][1]}, up[2] = {acc[ha][i][1][0], acc[ha][i][1][1]};
        out.rows16(grp * 128 + 16 * g, gate, up);
      } else if constexpr (LOSS) {
        v4f v[4] = {acc[ha][i][0][0], acc[ha][i][0][1], acc[ha][i][1][0], acc[ha][i][1][1]};
        out.rows16(g, grp * 128 + 16 * g, v);
      } else {
        v4f v[4] = {acc[ha][i][0][0], acc[ha][i][0][1], acc[ha][i][1][0], acc[ha][i][1][1]};
        out.rows16(grp * 128 + 16 * g, v, res);
      }
      if constexpr (EPI) {
        res[0] = ahead[0];
        res[1] = ahead[1];
      }
    }
    if constexpr (KIND == kKindLse) {
      __syncthreads();
      // (waves 4 grp .. 4 grp + 3 hold the same 128 rows; the first two of them join them)
      if (q < 2) Out::template merge<4>(p, w, smem + kTurns + 4 * grp * Out::kTurn, Out::kTurn, 64 * q + here, 128 * grp, 256);
    }
    if (u >= total) return;
    w = next;
  }
}

// ------------------------------------------------------------------- host
// Tile configurations.  kBig: bf16_big_kernel; kFew: bf16_few_kernel; the
// others: bf16_kernel with two workgroups a CU.
enum { kBig = 0, kDuo, kMid, kHigh, kLow, kFlat, kThin, kFew, kSlab, kDeep, kConfigs };
using BfDuo = BfCfg<128, 256, 1, 4, 3, 2, 32>;
using BfMid = BfCfg<128, 128, 2, 2, 2, 2>;
using BfHigh = BfCfg<128, 64, 2, 2, 3, 2>;
using BfLow = BfCfg<64, 64, 2, 2, 4, 2>;
using BfFlat = BfCfg<32, 64, 2, 2, 5, 2>;
using BfThin = BfCfg<16, 64, 1, 4, 6, 2>;
using BfSlab = BfCfg<64, 128, 2, 2, 3, 2>;    // (this and the next for a head's logits only)
using BfDeep = BfCfg<128, 128, 2, 2, 3, 1>;
constexpr int kBm[kConfigs] = {256, 128, 128, 128, 64, 32, 16, 16, 64, 128};
constexpr int kBn[kConfigs] = {256, 256, 128, 64, 64, 64, 64, 16, 128, 128};
constexpr int kThreads[kConfigs] = {512, BfDuo::THREADS, BfMid::THREADS, BfHigh::THREADS,
                                    BfLow::THREADS, BfFlat::THREADS, BfThin::THREADS, 512, BfSlab::THREADS, BfDeep::THREADS};

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

// The gated products.
template <int MODE>
hipError_t launch_gated(BfProblem p, const BfTile& t, hipStream_t stream) {
  const unsigned units = grid_of(p, t.bm, t.bn);
  if (t.cfg == kFew) return start(bf16_few_kernel<MODE, true>, p, units, 512, stream);
  if (t.cfg == kFlat) return start(bf16_kernel<BfFlat, false, false, MODE, false, kKindGated>, p, units, BfFlat::THREADS, stream);
  if (t.cfg == kLow) return start(bf16_kernel<BfLow, false, false, MODE, false, kKindGated>, p, units, BfLow::THREADS, stream);
  if (t.cfg == kHigh) return start(bf16_kernel<BfHigh, false, false, MODE, false, kKindGated>, p, units, BfHigh::THREADS, stream);
  if (t.cfg == kMid) return start(bf16_kernel<BfMid, false, false, MODE, false, kKindGated>, p, units, BfMid::THREADS, stream);
  const unsigned cus = (unsigned)device_cu_count();
  p.grid = (int)(units < cus ? units : cus);
  return start(bf16_big_kernel<false, false, MODE, false, false, kKindGated>, p, p.grid, 512, stream);
}

// A linear head's logits.
template <int KIND>
hipError_t launch_loss(BfProblem p, const BfTile& t, hipStream_t stream) {
  const unsigned units = grid_of(p, t.bm, t.bn);
  if (t.cfg == kSlab) return start(bf16_kernel<BfSlab, false, false, kBfDense, false, KIND>, p, units, BfSlab::THREADS, stream);
  if (t.cfg == kDeep) return start(bf16_kernel<BfDeep, false, false, kBfDense, false, KIND>, p, units, BfDeep::THREADS, stream);
  if (t.cfg == kMid) return start(bf16_kernel<BfMid, false, false, kBfDense, false, KIND>, p, units, BfMid::THREADS, stream);
  const unsigned cus = (unsigned)device_cu_count();
  p.grid = (int)(units < cus ? units : cus);
  return start(bf16_big_kernel<false, false, kBfDense, false, false, KIND>, p, p.grid, 512, stream);
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
    if (t.cfg == kDuo)
      return p.add ? start(bf16_kernel<BfDuo, AK, BK, MODE, true>, p, units, BfDuo::THREADS, stream)
                   : start(bf16_kernel<BfDuo, AK, BK, MODE>, p, units, BfDuo::THREADS, stream);
  }
  const unsigned cus = (unsigned)device_cu_count();
  p.grid = (int)(units < cus ? units : cus);
  if constexpr (BK && MODE != kBfRowRuns) {
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
  // (a gated product's N counts gate and up rows)
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
  const bool dense = p.mode == kBfDense, gated = p.kind == kKindGated;
  const bool loss = p.kind == kKindLse || p.kind == kKindDlogits;
  const bool second_round = units(kMid) > 2 * cus;
  if (loss) {
    // Few rows: the weights' one way through, 64-row tiles for less work (64 x 128000
    // x 7168 341).  128 x 128 tiles with a third stage while one a CU holds them all:
    // 128 x 32000 x 4096 74 for 87, 200 x 16000 x 7168 90 for 122, beyond, two a CU:
    // 256 x 32000 x 4096 99 for 109.
    t.cfg = rows <= 64 ? kSlab : second_round ? kBig : units(kMid) <= cus ? kDeep : kMid;
  } else if (p.parts) {
    t.cfg = kBig;
  } else if (p.add && !p.a_kmajor) {      // (the tiles that add)
    t.cfg = second_round ? kBig : kMid;
  } else if (p.a_kmajor) {
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
  } else if (rows <= 8 && !p.b_kmajor && p.K <= 4096 && units(kFew) <= (gated ? 4 : 2) * cus) {
    t.cfg = kFew;      // 1 x 1024 x 2048 5.5 for 6.6; 1 x 2112 x 7168 12.8 for 11.2
  } else if (rows <= (dense ? 16 : 8) && !gated) {   // (its waves own too few columns for both sums)
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
  t.bn = kBn[t.cfg] * (gated && t.cfg == kFew ? 2 : 1);   // (16 gate and 16 up rows)
  t.threads = kThreads[t.cfg];
  t.persistent = t.cfg == kBig;
  t.splits = p.parts ? p.parts : 1;
  if (dense && t.cfg != kBig && t.cfg != kFew) {
    // One workgroup a CU; two where several row tiles read the same weights
    // (64 x 2112 x 7168 14.1 in 6 splits, 16.2 in 12; 128 x 2112 x 7168 18.9
    // in 6, 19.8 in 3), and five steps a split at least.  A head's loss: 40 x 5000
    // x 7168 28 for 64 unsplit, 200 x 8000 x 4096 40 for 51 (in tiles of kDeep, of
    // which a CU holds one; 46 at two a CU).
    const int64_t u = units(t.cfg), steps = (p.K + kBK - 1) / kBK;
    if (4 * u < 3 * cus && u <= kSplitKMaxTiles) {
      int64_t s = (rows > t.bm && t.cfg != kDeep ? 2 * cus : cus) / u;
      if (s > steps / 5) s = steps / 5;
      if (s > kBfMaxSplits) s = kBfMaxSplits;
      if (s > 1) t.splits = (int)s;
    }
  }
  return t;
}

size_t bf16_workspace_bytes(const BfProblem& p, int cus) {
  const BfTile t = bf16_tile(p, cus);
  if (t.splits <= 1 || p.parts) return 0;
  const size_t tiles = (size_t)((p.M + t.bm - 1) / t.bm) * ((p.N + t.bn - 1) / t.bn);
  return kSplitKCounterBytes + tiles * t.splits * t.bm * t.bn * 4;
}

hipError_t launch_bf16(BfProblem p, const BfTile& t, hipStream_t stream) {
  p.splits = t.splits;
  if (p.kind == kKindLse) return launch_loss<kKindLse>(p, t, stream);
  if (p.kind == kKindDlogits) return launch_loss<kKindDlogits>(p, t, stream);
  if (p.kind == kKindGated) return p.mode == kBfRowRuns ? launch_gated<kBfRowRuns>(p, t, stream) : launch_gated<kBfDense>(p, t, stream);
  if (p.mode == kBfRowRuns)
    return p.b_kmajor ? launch_tile<false, true, kBfRowRuns>(p, t, stream)
                      : launch_tile<false, false, kBfRowRuns>(p, t, stream);
  if (p.mode == kBfKRuns) return launch_tile<true, true, kBfKRuns>(p, t, stream);
  if (p.a_kmajor) return launch_tile<true, true, kBfDense>(p, t, stream);
  return p.b_kmajor ? launch_tile<false, true, kBfDense>(p, t, stream)
                    : launch_tile<false, false, kBfDense>(p, t, stream);
}

}  // namespace fg8

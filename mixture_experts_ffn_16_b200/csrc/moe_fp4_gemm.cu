// moe_fp4_gemm.cu - the experts' products in MXFP4 on the 5th-generation
// tensor cores (kind::mxf4, block scales applied by the MMA):
//
//   product : out[r, n] = a[r,:] . W[e(r), n, :]
//   swiglu  : h[r, j]   = SiLU(a[r,:] . Wg[e(r), j, :]) * (a[r,:] . Wu[e(r), j, :]),
//             written as MXFP4 (a block = 32 consecutive j)
//
// for rows r sorted by expert, e(r) given by offsets[E+1] on the device.
//
// The weights are the MMA's M side and the tokens its N side: a unit of work
// is 2 x 128 weight rows (product: 256 consecutive output features; swiglu:
// 128 gate rows and the 128 up rows of the same features) times a run of up
// to 96 rows of one expert, cut evenly and rounded up to 16, so that an expert
// with few rows costs few MMA columns and no row is padded in memory.  Experts
// of more than 96 rows on average run on CTA pairs (below).
//
//   warp 0      TMA: 256 elements of K a stage (128-byte swizzled rows) of both
//               weight tiles and the token rows.
//   warp 1      tensor-memory owner and MMA issuer: copies the stage's scales
//               to tensor memory, where the MMA reads them, then 4 x 64
//               elements of K.
//   warps 2, 3  scales, one chunk of 128 elements of K each: 4-byte
//               asynchronous copies (the first row of a token run may be any)
//               that land word (row 32 c + l) of 128 rows at 16 l + 4 c, the
//               order in which tc_cp_scales reads them.  One warp for both
//               chunks took 640-720 cycles a stage, more than the MMAs; loads
//               to registers two stages ahead and 16-byte shared stores in
//               their place made the products of large experts 13-20% slower.
//   warps 4-11  epilogue: two warps per lane quarter.  A lane of tensor memory
//               is a feature, a warp's 32 lanes are one block of h, turned in
//               shared memory to 8 features of a token a lane.  16 warps were
//               slower (product 284 -> 315 us at 384 experts of 165 rows).
//
// What bounds them, on a B200 under its 1 kW limit: experts of few rows stream
// their weights (512 experts, 640 rows, N = 4096, K = 1024: 115 us on the same
// tensors again, 124-127 us on others each time, 7.1 and 6.5-6.6 TB/s; a pass
// that only reads 4 GiB reaches 7.26, a copy 6.56).  With many rows the power
// limit binds: 64 experts x about 512 rows, N = K = 4096, takes 286 us from a
// cool start and 333 us in a loop of seconds (3.3 PFLOP/s, 992 W, 1327 MHz).  Of
// its 340 us at an earlier step the MMAs alone, on operands that are already
// there, took 175, the tensor loads alone 184, loads and epilogue 245, all but
// the scales' copies to shared memory 331, all but those to tensor memory 323;
// the clock took what was saved, up to 1.9 GHz.  DRAM reads are the operands once
// (164 MB of 160 at 16 experts x 512 rows).
//
// K need not be a multiple of 256: loads past its end read zeros, and the MMAs
// past it are not issued.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_fp4.cuh"
#include "moe_internal.h"
#include "moe_ptx.cuh"

namespace moe {

namespace {

constexpr int kNA = 2;                                    // weight tiles per unit
constexpr int kStageK = 256;                              // elements of K per stage
constexpr uint32_t kTile = kTileRows * 128u;              // 128 rows x 256 codes
constexpr uint32_t kChunkScales = kTileRows * 4u;         // scale words of 128 rows x 128 elements
constexpr int kEpiWarps = 8;
constexpr int kEpiPer = kEpiWarps / 4;                    // epilogue warps per lane quarter
constexpr int kFirstEpi = 4;
constexpr int kScaleLanes = 64;
constexpr int kThreads = 32 * (kFirstEpi + kEpiWarps);
constexpr int kBufs = 2;                                  // accumulators
constexpr uint32_t kTmemCols = 512;
constexpr int kStgRow = 80;                               // 64 bytes of features + 16: distinct banks
constexpr uint32_t kXchTile = 16 * 32 * 4;                // 16 tokens x 32 features in fp32
constexpr uint32_t kStgBytes = kXchTile;                  // per epilogue warp
static_assert(16 * kStgRow <= kStgBytes, "staging of 16 tokens");
constexpr int kSmemAlign = 1024;
constexpr int kSmemTail = 512;                            // barriers, TMEM slot, abort flag
constexpr int64_t kMaxUnits = 1 << 30;

enum OutKind { kOutBf16 = 0, kOutFp16 = 1, kOutFp32 = 2, kOutSwiglu = 3 };

struct Params {
  CUtensorMap mapW[kNA];     // codes: product: [0] both tiles; swiglu: gate, up
  CUtensorMap mapA[4];       // token codes, boxes of 16 / 32 / 64 / 128 rows
  const uint32_t* w_scales[kNA];   // words [E][KC][N]
  const uint32_t* a_scales;  // [KC][rows]
  const int32_t* offsets;
  void* out;
  uint8_t* out_scales;
  uint32_t* err;
  int rows, E, N, K;
  int64_t timeout_cycles;
};

struct Unit {
  int e, wb, row0, rows, n;
};

// Layout of a kernel: NA weight tiles of 128 rows and TOK token rows a stage,
// S stages, runs of up to NMAX tokens.
template <int NA_, int NMAX_, int TOK_, int S_, uint32_t STG_>
struct Form {
  static constexpr int NA = NA_, NMAX = NMAX_, S = S_;
  static constexpr int NB = (NMAX + kTileRows - 1) / kTileRows;    // 128s of tokens
  // Scales of one stage: 2 chunks of 128 elements for each 128 rows of the
  // weight tiles, then of the run; 4 columns of tensor memory each.
  static constexpr int kChunks = 2 * (NA + NB);
  static constexpr uint32_t kTokOff = NA * kTile, kScaleOff = kTokOff + TOK_ * 128u;
  static constexpr uint32_t kStage = kScaleOff + kChunks * kChunkScales;
  static constexpr uint32_t kStg = STG_;                             // epilogue staging
  static constexpr uint32_t kSfBase = kTmemCols - S * 4 * kChunks;   // its columns behind the accumulators
  static constexpr int kPool = kSfBase & ~31u;                       // columns for accumulators
  static constexpr uint32_t kFixed = kSmemAlign + S * kStage + kStg + kSmemTail;
  static_assert(kStage % 1024 == 0 && kTokOff % 1024 == 0, "swizzled tiles start at multiples of 1024");
  static_assert(NA * NMAX <= kPool, "tensor memory");
  static_assert(kFixed + 2 * 4 * (kMaxE + 1) <= 232448, "shared memory, with the tables of kMaxE experts");
};

// Columns of an accumulator of n tokens, and where the one in place 0 or 1
// starts: at either end of the pool.  Two neighbouring units that do not fit
// beside each other take turns.
__device__ __forceinline__ int acc_cols(int n) { return (n + 31) & ~31; }
template <class F>
__device__ __forceinline__ uint32_t acc_at(int buf, int n) {
  return buf ? static_cast<uint32_t>(F::kPool - acc_cols(n)) : 0u;
}

template <class F>
__device__ __forceinline__ int runs_of(int rows) {
  return (rows + F::NMAX - 1) / F::NMAX;
}

// Units of each expert: first[e] = number of units before expert e's (nwb
// weight blocks times its runs), first[E] their number.  Offsets are clamped
// to the rows there are, an expert whose end lies before its start gets none,
// and the count saturates (valid offsets stay below kMaxUnits), so nothing is
// read or written out of bounds whatever the offsets say.  All threads; a
// barrier must follow.
template <class F>
__device__ __forceinline__ void unit_table(const Params& p, int nwb, int* off, int* first, int64_t* wsum) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, threads = blockDim.x;
  for (int e = tid; e <= p.E; e += threads) off[e] = min(max(__ldg(p.offsets + e), 0), p.rows);
  __syncthreads();
  const int per = (p.E + threads - 1) / threads;
  const int e0 = tid * per, e1 = min(e0 + per, p.E);
  int64_t sum = 0;
  for (int e = e0; e < e1; ++e) sum += static_cast<int64_t>(runs_of<F>(max(off[e + 1] - off[e], 0))) * nwb;
  int64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  int64_t at = inc - sum;
  for (int w = 0; w < warp; ++w) at += wsum[w];
  for (int e = e0; e < e1; ++e) {
    first[e] = static_cast<int>(min(at, kMaxUnits));
    at += static_cast<int64_t>(runs_of<F>(max(off[e + 1] - off[e], 0))) * nwb;
  }
  // threads past the experts carry the total
  if (tid == threads - 1) first[p.E] = static_cast<int>(min(at, kMaxUnits));
}

// The expert that owns unit u: the last e with first[e] <= u.  The whole warp
// searches: 32 probes spread over the experts, then 32 at a time between two.
template <class F>
__device__ __forceinline__ Unit find_unit(const int* first, const int* off, int E, int u, int lane) {
  const int step = (E + 31) / 32;
  const int i = lane * step;
  const uint32_t m = __ballot_sync(0xffffffffu, i < E && first[i] <= u);
  const int b = (__popc(m) - 1) * step;
  int cnt = 0;
  for (int j = 0; j < step; j += 32) {
    const int q = b + j + lane;
    cnt += __popc(__ballot_sync(0xffffffffu, j + lane < step && q < E && first[q] <= u));
  }
  Unit un;
  un.e = b + cnt - 1;
  const int c = off[un.e + 1] - off[un.e];
  const int nr = runs_of<F>(c);
  const int per = ((c + nr - 1) / nr + 15) & ~15;
  const int v = u - first[un.e];
  un.wb = v / nr;
  const int run = v - un.wb * nr;
  un.row0 = off[un.e] + run * per;
  un.rows = min(per, c - run * per);
  un.n = (un.rows + 15) & ~15;
  return un;
}

// Bounded wait for a barrier phase: the thread sleeps in the hardware, up to
// 20 us an attempt.  The clock is read every 8 attempts only.  CLUSTER: the
// peer CTA's threads arrive too, with a release at cluster scope.
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                           const Params& p) {
  const uint32_t a = smem_u32(bar);
  const auto arrived = [&] {
    return CLUSTER ? mbar_try_wait_sleep_cluster(a, parity, 20000u) : mbar_try_wait_sleep(a, parity, 20000u);
  };
  if (CLUSTER ? arrived() : mbar_try_wait(a, parity)) return true;
  int64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (arrived()) return true;
    if ((it & 7u) == 0) {
      if (*abort_flag) return false;
      const int64_t now = clock64();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > p.timeout_cycles) {
        *abort_flag = 1;
        atomicOr(p.err, kDevErrTimeout);
        return false;
      }
    }
  }
}

// The same for work this block itself put in flight, before it leaves: does
// not give up for another role's sake.
__device__ __forceinline__ void wait_drain(uint64_t* bar, uint32_t parity, const Params& p) {
  const uint32_t a = smem_u32(bar);
  const int64_t t0 = clock64();
  while (!mbar_try_wait(a, parity) && clock64() - t0 <= p.timeout_cycles) {
  }
}

// Every lane waits, since each goes on to touch what the barrier guards (a
// shuffle from one that waits would not order the others' accesses); all or
// none go on.  Also faster than one lane and a shuffle: 64 experts x about 512
// rows 346 -> 315 us.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, const Params& p) {
  return __all_sync(0xffffffffu, wait_phase(bar, parity, abort_flag, p));
}

template <int KIND>
__device__ __forceinline__ uint32_t pack16(uint32_t lo, uint32_t hi) {
  if constexpr (KIND == kOutFp16) {
    const __half2 v = __floats2half2_rn(__uint_as_float(lo), __uint_as_float(hi));
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

// SiLU(g) u, for a result that is rounded to 3 bits next, where a value beside a
// border moves by a whole step: fp32 operations each to their last ulps, as
// elementary fp32 arithmetic gives them.  (__expf and __fdividef are faster, 146
// against 150 us for a prefill of 4096 tokens on 256 experts, but off by an ulp
// for every unit of |g|, and 0 for g below -87.3.)
// The division has no branch for its extremes, which cost 10%: an approximate
// reciprocal and one correction of the quotient by its remainder (Markstein,
// IBM J. Res. Dev. 34, 1990), numerator and denominator scaled down together
// where the reciprocal could be subnormal.  Compared with g / (1 + expf(-g)) at
// every fp32 g: the same bits but for -0 (gives +0) and +inf (gives NaN; either
// way the block of h is NaN).  Where expf(-g) overflows, g below -88.7, both are
// -0 (SiLU itself is above -2.6e-37).
__device__ __forceinline__ float swiglu(float g, float u) {
  const float s = g < -64.0f ? 0x1p-4f : 1.0f;
  const float d = fmaf(expf(-g), s, s), n = g * s, r = rcp_approx(d), q = n * r;
  return fmaf(fmaf(-fminf(d, 0x1.fffffep127f), q, n), r, q) * u;
}

// Words [16 tokens][32 features] of a warp's block in shared memory: written
// by lane = feature, read 4 at a time by lane = (token, 8 features).  The xor
// keeps the 8 lanes of such a read, 2 tokens, on distinct banks.
__device__ __forceinline__ int xch_at(int tok, int feat) { return 32 * tok + (feat ^ (4 * (tok & 1))); }
__device__ __forceinline__ void xch_get8(const float* x, int tok, int feat, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(x + xch_at(tok, feat));
  const float4 b = *reinterpret_cast<const float4*>(x + xch_at(tok, feat + 4));
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// h of token `tok` of the run and features feat0 + 8 (lane & 3) .. + 7 as
// MXFP4: the block's four lanes are neighbours.  (Gate/up of 256 experts x 128
// rows 76.0 us; with a lane a feature and the block's maximum by shuffles over
// 32 lanes 77.6 us.)
__device__ __forceinline__ void emit_h8(const Params& p, const Unit& un, int feat0, int tok, const float (&h)[8],
                                        int lane) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(h[j]) & 0x7FFFFFFFu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const uint32_t byte = fp4_scale_byte(m);
  const float inv = fp4_inv_scale(byte);
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = h[j] * inv;
  const uint32_t word = byte == kFp4NanScale ? 0u : e2m1x8(v);
  if (tok >= un.rows) return;
  const size_t row = static_cast<size_t>(un.row0) + tok;
  uint8_t* codes = static_cast<uint8_t*>(p.out) + row * (p.N >> 1) + (feat0 >> 1);
  *reinterpret_cast<uint32_t*>(codes + 4 * (lane & 3)) = word;
  if ((lane & 3) == 0) {
    uint8_t* scale = p.out_scales + (static_cast<size_t>(feat0 >> 7) * p.rows + row) * 4 + ((feat0 >> 5) & 3);
    *scale = static_cast<uint8_t>(byte);
    // f a multiple of 64 only: the last word's two spare bytes
    if (feat0 + 32 == p.N && (p.N & 127)) *reinterpret_cast<uint16_t*>(scale + 1) = 0;
  }
}

// 16 tokens (c ..) of the accumulator at `taddr` (this warp's lane quarter,
// features feat0 .. + 31) to the output.
template <int KIND>
__device__ __forceinline__ void emit_out16(const Params& p, const Unit& un, int feat0, int c, uint32_t taddr,
                                           uint8_t* stg, int lane) {
  if constexpr (KIND == kOutFp32) {
    uint32_t v[16];
    tmem_ld_32x32b_x16(taddr, v);
    tmem_ld_wait();
    float* out = static_cast<float*>(p.out) + static_cast<size_t>(un.row0 + c) * p.N + feat0 + lane;
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (c + j < un.rows) out[static_cast<size_t>(j) * p.N] = __uint_as_float(v[j]);
  } else {
    uint32_t v[2][8];
    tmem_ld_16x256b_x2(taddr, v[0]);
    tmem_ld_16x256b_x2(taddr + (16u << 16), v[1]);
    tmem_ld_wait();
    // matrices: 0 = features 16h + 0..7 x tokens 0..7, 1 = features
    // 16h + 8..15 x tokens 0..7, 2 and 3 = the same for tokens 8..15
    const uint32_t stg_s = smem_u32(stg);
    const int mi = lane >> 3, mj = lane & 7;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      stmatrix_x4_trans(stg_s + static_cast<uint32_t>((8 * (mi >> 1) + mj) * kStgRow + (16 * h + 8 * (mi & 1)) * 2),
                        pack16<KIND>(v[h][0], v[h][1]), pack16<KIND>(v[h][2], v[h][3]),
                        pack16<KIND>(v[h][4], v[h][5]), pack16<KIND>(v[h][6], v[h][7]));
    __syncwarp();
#pragma unroll
    for (int rep = 0; rep < 2; ++rep) {
      const int cc = lane + 32 * rep;
      const int tok = cc >> 2, part = cc & 3;
      if (c + tok < un.rows)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + static_cast<size_t>(un.row0 + c + tok) * p.N +
                                  feat0 + part * 8) = *reinterpret_cast<const uint4*>(stg + tok * kStgRow + part * 16);
    }
    __syncwarp();
  }
}

// The MMAs of one stage: scales to tensor memory, then `steps` x 64 elements
// of K for each of the unit's NA weight tiles.
template <class F, int NA, bool PAIR>
__device__ __forceinline__ void issue_stage(uint32_t a_lo, uint32_t b_lo, uint64_t s_desc, uint32_t sf, uint32_t dcol,
                                            uint32_t id0, uint32_t id1, int kb, int steps) {
#pragma unroll
  for (int i = 0; i < F::kChunks; ++i)
    if (i < 2 * NA || i >= 2 * F::NA)
      tc_cp_scales<PAIR>(sf + 4u * i, s_desc + static_cast<uint64_t>(i * (kChunkScales >> 4)));
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    if (ks < steps) {
#pragma unroll
      for (int a = 0; a < NA; ++a)
        tc_mma_mxf4<PAIR>(dcol + static_cast<uint32_t>(a * F::NMAX), a_lo + a * (kTile >> 4) + 2u * ks,
                          b_lo + 2u * ks, (ks & 1) ? id1 : id0, sf + 4u * (2 * a + (ks >> 1)),
                          sf + 4u * (2 * F::NA + F::NB * (ks >> 1)), (kb | ks) != 0);
    }
  }
}

// Experts of up to 96 rows on average: 256 weight rows x 96 tokens a unit.
// Shorter runs did not help the smallest experts (1 to 12 rows, 16 to 96
// columns: within 3%), and at 64 rows 64-token runs cost 15% (two runs for
// every second expert).
using Single = Form<2, 96, 96, 4, kEpiWarps * kStgBytes>;
static_assert(kBufs * Single::NA * Single::NMAX <= Single::kPool, "both accumulators");

template <int KIND>
__global__ void __launch_bounds__(kThreads, 1) fp4_gemm_kernel(const __grid_constant__ Params p) {
  using F = Single;
  constexpr bool SWIGLU = KIND == kOutSwiglu;
  constexpr int kRowsPerWb = SWIGLU ? kTileRows : kNA * kTileRows;   // weight rows between units
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + (kSmemAlign - 1)) & ~static_cast<uintptr_t>(kSmemAlign - 1));
  constexpr int S = F::S;
  uint8_t* stg_all = smem + S * F::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(stg_all + F::kStg);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + kBufs;
  uint64_t* drain = tempty + kBufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int64_t* wsum = reinterpret_cast<int64_t*>(tmem_slot + 2);   // one per warp
  int* off = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(full) + kSmemTail);   // [E + 1] row offsets, clamped
  int* first = off + p.E + 1;                                  // [E + 1] first unit of each expert

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full + s, 1 + kScaleLanes);     // the TMA warp and the lanes of the scale warps
      mbar_init(empty + s, 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(tfull + b, 1);
      mbar_init(tempty + b, kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    for (int i = 0; i < kNA; ++i) prefetch_tensormap(&p.mapW[i]);
    for (int i = 0; i < 4; ++i) prefetch_tensormap(&p.mapA[i]);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  chain_wait();

  unit_table<F>(p, (p.N + kRowsPerWb - 1) / kRowsPerWb, off, first, wsum);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int num_units = first[p.E];
  const int KB = (p.K + kStageK - 1) / kStageK;
  const int grid = gridDim.x;

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    const uint64_t pol_w = policy_evict_first(), pol_a = policy_evict_last();
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < num_units; u += grid) {
      const Unit un = find_unit<F>(first, off, p.E, u, lane);
      const int f0 = un.wb * kRowsPerWb;
      const int na = (!SWIGLU && f0 + kTileRows >= p.N) ? 1 : kNA;      // the second tile may lie past the weight
      const uint32_t tx = static_cast<uint32_t>(na) * kTile + static_cast<uint32_t>(un.n) * 128u;
      if (elect_one()) {
        for (int kb = 0; kb < KB; ++kb) {
          if (!wait_phase(&empty[stage], phase ^ 1u, abort_flag, p)) {
            ok = false;
            break;
          }
          const uint32_t sbase = smem_u32(smem + stage * F::kStage);
          const uint32_t fb = smem_u32(&full[stage]);
          mbar_arrive_expect_tx(&full[stage], tx);
          for (int a = 0; a < na; ++a)
            tma_load_3d_hint(sbase + a * kTile, &p.mapW[SWIGLU ? a : 0], fb, kb * 128,
                             f0 + (SWIGLU ? 0 : a * kTileRows), un.e, pol_w);
          tma_load_rows<false>(sbase + F::kTokOff, p.mapA, fb, kb * 128, un.row0, un.n, pol_a);
          ++issued;
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    if (elect_one()) {
      // leave no copy in flight
      const uint32_t outstanding = issued < static_cast<uint32_t>(S) ? issued : static_cast<uint32_t>(S);
      for (uint32_t i = 1; i <= outstanding; ++i) {
        const uint32_t I = issued - i;
        wait_drain(&full[I % S], (I / S) & 1u, p);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    int stage = 0;
    uint32_t phase = 0, count = 0;
    bool any = false, ok = true;
    const uint32_t a_lo = sw128_desc_lo(smem_u32(smem)), b_lo = sw128_desc_lo(smem_u32(smem) + F::kTokOff);
    const uint64_t s_lo = rows16_desc(smem_u32(smem) + F::kScaleOff);
    for (int u = blockIdx.x; ok && u < num_units; u += grid) {
      const Unit un = find_unit<F>(first, off, p.E, u, lane);
      if (elect_one()) {
        const int na = (!SWIGLU && un.wb * kRowsPerWb + kTileRows >= p.N) ? 1 : kNA;
        const int buf = static_cast<int>(count % kBufs);
        const uint32_t bpar = (count / kBufs) & 1u;
        ok = wait_phase(&tempty[buf], bpar ^ 1u, abort_flag, p);
        tc_fence_after();
        const uint32_t id0 = idesc_mxf4(kTileRows, un.n, 0), id1 = idesc_mxf4(kTileRows, un.n, 1);
        const uint32_t dcol = tmem_base + static_cast<uint32_t>(buf * F::NA * F::NMAX);
        for (int kb = 0; ok && kb < KB; ++kb) {
          ok = wait_phase(&full[stage], phase, abort_flag, p);
          if (!ok) break;
          tc_fence_after();
          fence_proxy_async_smem();      // scales written by cp.async are read by the tensor core
          const uint32_t off_s = static_cast<uint32_t>(stage) * (F::kStage >> 4);
          const uint32_t sf = tmem_base + F::kSfBase + static_cast<uint32_t>(stage * 4 * F::kChunks);
          const int steps = min(4, (p.K - kb * kStageK) / 64);
          if (na == kNA)
            issue_stage<F, kNA, false>(a_lo + off_s, b_lo + off_s, s_lo + off_s, sf, dcol, id0, id1, kb, steps);
          else
            issue_stage<F, 1, false>(a_lo + off_s, b_lo + off_s, s_lo + off_s, sf, dcol, id0, id1, kb, steps);
          any = true;
          tc_commit(&empty[stage]);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) tc_commit(&tfull[buf]);
        ++count;
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    if (elect_one() && any) {
      // leave no MMA in flight
      tc_commit(drain);
      wait_drain(drain, 0, p);
    }
    __syncwarp();
  } else if (warp < kFirstEpi) {
    // ------------------------------------------------------------ scales
    const int KC = (p.K + 127) / 128, h = warp - 2;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < num_units; u += grid) {
      const Unit un = find_unit<F>(first, off, p.E, u, lane);
      const int f0 = un.wb * kRowsPerWb;
      // Rows past the weight or the run repeat the last one there is; their
      // results are never stored.
      uint32_t wrow[kNA][4], trow[4 * F::NB];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int a = 0; a < kNA; ++a)
          wrow[a][c] = static_cast<uint32_t>(min(f0 + (SWIGLU ? 0 : a * kTileRows) + 32 * c + lane, p.N - 1));
      }
#pragma unroll
      for (int c = 0; c < 4 * F::NB; ++c) trow[c] = static_cast<uint32_t>(min(un.row0 + 32 * c + lane, p.rows - 1));
      for (int kb = 0; kb < KB; ++kb) {
        ok = warp_wait(&empty[stage], phase ^ 1u, abort_flag, p);
        if (!ok) break;
        const uint32_t dst = smem_u32(smem + stage * F::kStage) + F::kScaleOff + 16u * lane;
        const int kc = min(2 * kb + h, KC - 1);
        const size_t wchunk = (static_cast<size_t>(un.e) * KC + kc) * p.N;
        const uint32_t* tsrc = p.a_scales + static_cast<size_t>(kc) * p.rows;
#pragma unroll
        for (int a = 0; a < kNA; ++a) {
          const uint32_t* wsrc = p.w_scales[a] + wchunk;
#pragma unroll
          for (int c = 0; c < 4; ++c) cp_async_4(dst + (2 * a + h) * kChunkScales + 4 * c, wsrc + wrow[a][c]);
        }
#pragma unroll
        for (int c = 0; c < 4 * F::NB; ++c)
          if (32 * c < un.n)
            cp_async_4(dst + (2 * F::NA + F::NB * h + c / 4) * kChunkScales + 4 * (c & 3), tsrc + trow[c]);
        cp_async_mbar_arrive_noinc(&full[stage]);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    cp_async_wait_all();
  } else if (warp >= kFirstEpi) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, part = (warp - kFirstEpi) >> 2;
    uint8_t* stg = stg_all + (warp - kFirstEpi) * kStgBytes;
    uint32_t count = 0;
    for (int u = blockIdx.x; u < num_units; u += grid, ++count) {
      const Unit un = find_unit<F>(first, off, p.E, u, lane);
      const int buf = static_cast<int>(count % kBufs);
      const uint32_t bpar = (count / kBufs) & 1u;
      if (!warp_wait(&tfull[buf], bpar, abort_flag, p)) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(32 * q) << 16) +
                          static_cast<uint32_t>(buf * F::NA * F::NMAX);
      // column blocks of 16 tokens, every kEpiPer-th one
      if constexpr (SWIGLU) {
        const int feat0 = un.wb * kTileRows + 32 * q;
        if (feat0 < p.N) {
          for (int c = 16 * part; c < un.n; c += 16 * kEpiPer) {
            uint32_t g[16], v[16];
            tmem_ld_32x32b_x16(tb + static_cast<uint32_t>(c), g);
            tmem_ld_32x32b_x16(tb + static_cast<uint32_t>(F::NMAX + c), v);
            tmem_ld_wait();
            float* x = reinterpret_cast<float*>(stg);
#pragma unroll
            for (int j = 0; j < 16; ++j)
              x[xch_at(j, lane)] = swiglu(__uint_as_float(g[j]), __uint_as_float(v[j]));
            __syncwarp();
#pragma unroll
            for (int o = 0; o < 16; o += 8) {
              float h[8];
              xch_get8(x, o + (lane >> 2), 8 * (lane & 3), h);
              emit_h8(p, un, feat0, c + o + (lane >> 2), h, lane);
            }
            __syncwarp();
          }
        }
      } else {
#pragma unroll 1
        for (int a = 0; a < kNA; ++a) {
          const int feat0 = un.wb * kRowsPerWb + a * kTileRows + 32 * q;
          if (feat0 >= p.N) break;
          for (int c = 16 * part; c < un.n; c += 16 * kEpiPer)
            emit_out16<KIND>(p, un, feat0, c, tb + static_cast<uint32_t>(a * F::NMAX + c), stg, lane);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[buf]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

// The form for large experts, on CTA pairs (cta_group::2): 256 weight rows, 128
// per CTA, times runs of up to 256 tokens, of which each CTA loads half.  Per
// multiply-add that moves half of the bytes of the single CTA's 256 x 96 units
// into shared memory, with a quarter of the MMAs.  The scales leave 384
// columns of tensor memory for two accumulators: of 192 each they lie side by
// side and the epilogue overlaps the next unit; a longer one and its neighbour
// share columns, which the epilogue reads first and reports before the rest.
// Against runs of up to 192 in two fixed places, 32 experts of 160 / 256 / 320
// / 512 / 2048 rows, N = 2048, K = 4096: 36.7 / 55.9 / 61.7 / 93.0 / 311 us
// there, 36.4 / 46.9 / 62.2 / 84.0 / 285 us this way (without the early report
// longer runs gained nothing at 512 rows; all of it at an earlier step).
//   product: CTA r has output features 128 r .. of the unit's 256.
//   swiglu:  CTA r has features 64 r .. of the unit's 128, their gate rows in
//            lanes 0..63 and their up rows in lanes 64..127.  A gate warp and
//            the up warp of the same features put 16 tokens of both into shared
//            memory, then each finishes 8 of them.
// Roles as above, in both CTAs; the MMAs are issued by the leader (rank 0)
// for both.  cp.async can only arrive on a barrier of its own CTA, so the
// peer's scale copies complete a barrier there, and the peer's warp 1, which
// has no MMAs to issue, reports it to the leader's, with a release restricted to
// shared memory.  (With a full release at cluster scope 64 experts x about 512
// rows, N = K = 4096, took 838 us in place of 304, a prefill of 4096 tokens on
// 256 experts 266 in place of 149.)
constexpr uint32_t kXchBytes = 2 * 2 * kXchTile;          // per warp pair: 2 buffers of gate and up

using Pair = Form<1, 256, 128, 5, kEpiWarps / 2 * kXchBytes>;

template <int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    fp4_gemm_pair_kernel(const __grid_constant__ Params p) {
  using F = Pair;
  constexpr bool SWIGLU = KIND == kOutSwiglu;
  constexpr int kCtaFeats = SWIGLU ? kTileRows / 2 : kTileRows;      // output features per CTA
  constexpr int kRowsPerWb = 2 * kCtaFeats;
  constexpr int kTwoFit = F::kPool / 2;      // columns of which two accumulators fit side by side
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + (kSmemAlign - 1)) & ~static_cast<uintptr_t>(kSmemAlign - 1));
  constexpr int S = F::S;
  uint8_t* stg_all = smem + S * F::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(stg_all + F::kStg);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + kBufs;
  uint64_t* tpart = tempty + kBufs;
  uint64_t* drain = tpart + kBufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int64_t* wsum = reinterpret_cast<int64_t*>(tmem_slot + 2);
  int* off = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(full) + kSmemTail);
  int* first = off + p.E + 1;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      // leader: TMA warps of both CTAs, its scale lanes, the peer's report;
      // peer: its scale lanes
      mbar_init(full + s, rank == 0 ? 2 + kScaleLanes + 1 : kScaleLanes);
      mbar_init(empty + s, 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(tfull + b, 1);
      mbar_init(tempty + b, 2 * kEpiWarps);
      mbar_init(tpart + b, 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    for (int i = 0; i < kNA; ++i) prefetch_tensormap(&p.mapW[i]);
    for (int i = 0; i < 4; ++i) prefetch_tensormap(&p.mapA[i]);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  chain_wait();
  unit_table<F>(p, (p.N + kRowsPerWb - 1) / kRowsPerWb, off, first, wsum);
  tc_fence_before();
  __syncthreads();
  cluster_sync();                        // the peer's barriers are initialised
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int num_units = first[p.E];
  const int KB = (p.K + kStageK - 1) / kStageK;
  const uint32_t full_leader = mapa_shared(smem_u32(full), 0);       // + 8 * stage
  const uint32_t tempty_leader = mapa_shared(smem_u32(tempty), 0);   // + 8 * buffer
  const uint32_t tpart_leader = mapa_shared(smem_u32(tpart), 0);

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    const uint64_t pol_w = policy_evict_first(), pol_a = policy_evict_last();
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    for (int u = pair; ok && u < num_units; u += npairs) {
      const Unit un = find_unit<F>(first, off, p.E, u, lane);
      const int f0 = un.wb * kRowsPerWb + static_cast<int>(rank) * kCtaFeats;
      // Half of the run, a multiple of 8 rows; loaded as a multiple of 16.
      const int half = un.n >> 1, row0 = un.row0 + static_cast<int>(rank) * half, load = (half + 15) & ~15;
      const uint32_t tx = kTile + static_cast<uint32_t>(load) * 128u;
      if (elect_one()) {
        for (int kb = 0; kb < KB; ++kb) {
          if (!wait_phase(&empty[stage], phase ^ 1u, abort_flag, p)) {
            ok = false;
            break;
          }
          const uint32_t sbase = smem_u32(smem + stage * F::kStage);
          const uint32_t fb = full_leader + 8u * stage;
          mbar_arrive_expect_tx_cluster(fb, tx);
          tma_load_3d_pair_hint(sbase, &p.mapW[0], fb, kb * 128, f0, un.e, pol_w);
          if (SWIGLU) tma_load_3d_pair_hint(sbase + kTile / 2, &p.mapW[1], fb, kb * 128, f0, un.e, pol_w);
          tma_load_rows<true>(sbase + F::kTokOff, p.mapA, fb, kb * 128, row0, load, pol_a);
          ++issued;
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    if (rank == 0 && elect_one()) {
      // leave no copy in flight: the leader's barriers count both CTAs'
      const uint32_t outstanding = issued < static_cast<uint32_t>(S) ? issued : static_cast<uint32_t>(S);
      for (uint32_t i = 1; i <= outstanding; ++i) {
        const uint32_t I = issued - i;
        wait_drain(&full[I % S], (I / S) & 1u, p);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs (leader)
    if (rank == 0) {
      int stage = 0, before = 0;         // columns of the unit before
      uint32_t phase = 0, count = 0, part_phase = 3;     // bit: parity of the last early report of a place
      bool any = false, ok = true;
      const uint32_t a_lo = sw128_desc_lo(smem_u32(smem)), b_lo = sw128_desc_lo(smem_u32(smem) + F::kTokOff);
      const uint64_t s_lo = rows16_desc(smem_u32(smem) + F::kScaleOff);
      for (int u = pair; ok && u < num_units; u += npairs) {
        const Unit un = find_unit<F>(first, off, p.E, u, lane);
        if (elect_one()) {
          const int buf = static_cast<int>(count % kBufs);
          const uint32_t bpar = (count / kBufs) & 1u;
          ok = wait_phase<true>(&tempty[buf], bpar ^ 1u, abort_flag, p);
          const int cols = acc_cols(un.n);
          if (ok && cols + before > F::kPool) {
            // the unit before still holds columns of this one
            ok = before > kTwoFit ? wait_phase<true>(&tpart[buf ^ 1], (part_phase >> (buf ^ 1)) & 1u, abort_flag, p)
                                  : wait_phase<true>(&tempty[buf ^ 1], ((count - 1) / kBufs) & 1u, abort_flag, p);
          }
          if (cols > kTwoFit) part_phase ^= 1u << buf;
          before = cols;
          tc_fence_after();
          const uint32_t id0 = idesc_mxf4(2 * kTileRows, un.n, 0), id1 = idesc_mxf4(2 * kTileRows, un.n, 1);
          const uint32_t dcol = tmem_base + acc_at<F>(buf, un.n);
          for (int kb = 0; ok && kb < KB; ++kb) {
            ok = wait_phase<true>(&full[stage], phase, abort_flag, p);
            if (!ok) break;
            tc_fence_after();
            fence_proxy_async_smem();
            const uint32_t off_s = static_cast<uint32_t>(stage) * (F::kStage >> 4);
            issue_stage<F, 1, true>(a_lo + off_s, b_lo + off_s, s_lo + off_s,
                                    tmem_base + F::kSfBase + static_cast<uint32_t>(stage * 4 * F::kChunks), dcol, id0,
                                    id1, kb, min(4, (p.K - kb * kStageK) / 64));
            any = true;
            tc_commit_pair(&empty[stage], 0x3);
            if (++stage == S) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (ok) tc_commit_pair(&tfull[buf], 0x3);
          ++count;
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      if (elect_one() && any) {
        // leave no MMA in flight
        tc_commit_pair(drain, 0x1);
        wait_drain(drain, 0, p);
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------- report of the peer's scales
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int u = pair; ok && u < num_units; u += npairs) {
        if (elect_one()) {
          for (int kb = 0; kb < KB; ++kb) {
            ok = wait_phase(&full[stage], phase, abort_flag, p);
            if (!ok) break;
            // The scales, written by asynchronous copies to this CTA's shared
            // memory, are read by its tensor core at the leader's request:
            // proxy fence, then release at cluster scope, which the leader's
            // wait acquires.
            fence_proxy_async_smem();
            mbar_arrive_cluster_release_smem(full_leader + 8u * stage);
            if (++stage == S) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
    }
  } else if (warp < kFirstEpi) {
    // ------------------------------------------------------------ scales
    const int KC = (p.K + 127) / 128, h = warp - 2;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = pair; ok && u < num_units; u += npairs) {
      const Unit un = find_unit<F>(first, off, p.E, u, lane);
      const int f0 = un.wb * kRowsPerWb + static_cast<int>(rank) * kCtaFeats;
      // Rows past the weight or the run repeat the last one there is; their
      // results are never stored.
      const uint32_t* wsrc[4];
      uint32_t trow[4 * F::NB];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int r = SWIGLU ? f0 + 32 * (c & 1) + lane : f0 + 32 * c + lane;
        wsrc[c] = p.w_scales[SWIGLU ? c >> 1 : 0] + static_cast<size_t>(un.e) * KC * p.N + min(r, p.N - 1);
      }
#pragma unroll
      for (int c = 0; c < 4 * F::NB; ++c) trow[c] = static_cast<uint32_t>(min(un.row0 + 32 * c + lane, p.rows - 1));
      for (int kb = 0; kb < KB; ++kb) {
        ok = warp_wait(&empty[stage], phase ^ 1u, abort_flag, p);
        if (!ok) break;
        const uint32_t dst = smem_u32(smem + stage * F::kStage) + F::kScaleOff + 16u * lane;
        const int kc = min(2 * kb + h, KC - 1);
        const uint32_t* tsrc = p.a_scales + static_cast<size_t>(kc) * p.rows;
#pragma unroll
        for (int c = 0; c < 4; ++c) cp_async_4(dst + h * kChunkScales + 4 * c, wsrc[c] + static_cast<size_t>(kc) * p.N);
#pragma unroll
        for (int c = 0; c < 4 * F::NB; ++c)
          if (32 * c < un.n)
            cp_async_4(dst + (2 * F::NA + F::NB * h + c / 4) * kChunkScales + 4 * (c & 3), tsrc + trow[c]);
        cp_async_mbar_arrive_noinc(&full[stage]);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    cp_async_wait_all();
  } else if (warp >= kFirstEpi) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, part = (warp - kFirstEpi) >> 2;
    uint8_t* stg = stg_all + (warp - kFirstEpi) * kStgBytes;
    // swiglu: lane quarters q and q ^ 2 hold gate and up of the same features
    const int wp = 2 * part + (q & 1);
    float* xch = reinterpret_cast<float*>(stg_all + wp * kXchBytes);
    volatile int* vote = reinterpret_cast<volatile int*>(wsum + kThreads / 32) + 2 * wp;
    uint32_t count = 0;
    int turn = 0;
    for (int u = pair; u < num_units; u += npairs, ++count) {
      const Unit un = find_unit<F>(first, off, p.E, u, lane);
      const int buf = static_cast<int>(count % kBufs);
      const uint32_t bpar = (count / kBufs) & 1u;
      bool got_acc = warp_wait(&tfull[buf], bpar, abort_flag, p);
      if constexpr (SWIGLU) {
        // Both warps of an exchange go on, or neither does: they meet at its
        // barriers.  The slots of a unit are written again two units later.
        volatile int* v = vote + kEpiWarps * (count & 1);
        if (lane == 0) v[q >> 1] = got_acc;
        named_barrier(1 + wp, 64);
        got_acc = got_acc && v[1 - (q >> 1)] != 0;
      }
      if (!got_acc) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + acc_at<F>(buf, un.n);
      const int f0 = un.wb * kRowsPerWb + static_cast<int>(rank) * kCtaFeats;
      const int feat0 = f0 + 32 * (SWIGLU ? q & 1 : q);
      // Blocks of kBlock tokens.  An accumulator of more than kTwoFit columns
      // is read in the order in which the next unit may need them, which takes
      // up to NMAX from the pool's other end: from its last column down in
      // place 0, from its first up in place 1; those that it may need are
      // reported early.
      constexpr int kBlock = 16;
      const int cols = acc_cols(un.n);
      int c = kBlock * part, step = kBlock * kEpiPer, left = (un.n - c + step - 1) / step, late = 0;
      if (cols > kTwoFit) {
        // blocks i < early of the order are reported early; this warp has every kEpiPer-th
        const int early = (cols - (F::kPool - F::NMAX)) / kBlock;
        late = left - (early - part + kEpiPer - 1) / kEpiPer;
        if (buf == 0) {
          c = (un.n - 1) / kBlock * kBlock - c;
          step = -step;
        }
      }
#pragma unroll 1
      for (;;) {
        if (feat0 < p.N) {
          for (; left > late; --left, c += step) {
            if constexpr (SWIGLU) {
              // gate and up of 16 tokens meet in shared memory, each warp
              // finishes 8 of them
              uint32_t v[16];
              tmem_ld_32x32b_x16(tb + static_cast<uint32_t>(c), v);
              tmem_ld_wait();
              float* x = xch + turn * (kXchTile / 2);
              float* mine = x + (q >> 1) * (kXchTile / 4);
#pragma unroll
              for (int j = 0; j < 16; ++j) mine[xch_at(j, lane)] = __uint_as_float(v[j]);
              named_barrier(1 + wp, 64);
              turn ^= 1;                   // the other buffer next: one barrier a block suffices
              const int tok = 8 * (q >> 1) + (lane >> 2);
              float g[8], h[8];
              xch_get8(x, tok, 8 * (lane & 3), g);
              xch_get8(x + kXchTile / 4, tok, 8 * (lane & 3), h);
#pragma unroll
              for (int j = 0; j < 8; ++j) h[j] = swiglu(g[j], h[j]);
              emit_h8(p, un, feat0, c + tok, h, lane);
            } else {
              emit_out16<KIND>(p, un, feat0, c, tb + static_cast<uint32_t>(c), stg, lane);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed((late ? tpart_leader : tempty_leader) + 8u * buf);
        if (late == 0) break;
        late = 0;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();                        // no CTA leaves while its peer may still touch it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

bool encode(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* ptr, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
  const cuuint32_t one[3] = {1, 1, 1};
  EncodeTiledFn fn = encode_fn();
  return fn && fn(m, type, rank, const_cast<void*>(ptr), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Weight codes uint8 [E, N, K/2]: tiles of `rows` x 128 bytes, swizzled.
bool map_weight(CUtensorMap* m, const void* codes, int E, int N, int K, int rows) {
  const cuuint64_t n = N, half = K / 2;
  const cuuint64_t d[3] = {half, n, static_cast<cuuint64_t>(E)}, s[2] = {half, half * n};
  const cuuint32_t b[3] = {128, static_cast<cuuint32_t>(rows), 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, codes, d, s, b, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Both forms of one kind: the function launched, its grid and shared memory.
template <int KIND>
int launch_kind(const Params& prm, bool pair, int sms, cudaStream_t st) {
  static std::atomic<int> single_limit[64], pair_limit[64];
  const auto kern = pair ? fp4_gemm_pair_kernel<KIND> : fp4_gemm_kernel<KIND>;
  const uint32_t fixed = pair ? Pair::kFixed : Single::kFixed, tables = 2u * 4u * (kMaxE + 1);
  const int rc = raise_smem_limit(kern, pair ? pair_limit : single_limit, static_cast<int>(fixed + tables));
  if (rc != MOE_OK) return rc;
  const size_t smem = fixed + 2 * 4 * (static_cast<size_t>(prm.E) + 1);
  return launch_chained(kern, dim3(pair ? sms & ~1 : sms), dim3(kThreads), smem, st, prm) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

}  // namespace

int launch_fp4_product(const Fp4Product& q, const DeviceInfo& di, uint32_t* err, cudaStream_t st) {
  const bool swiglu = q.w1_codes != nullptr;
  // CTA pairs above 96 rows an expert on average, what a single CTA's unit
  // takes in one run.  64 experts of 80 / 96 / 104 / 128 / 512 rows, pairs
  // against single CTAs: N = 4096, K = 1024 product 33 / 35 / 35 / 40 / 114 us
  // against 28 / 30 / 43 / 46 / 149; f = 1024, K = 4096 gate/up 55 / 59 / 57 / 62 /
  // 174 against 51 / 55 / 63 / 72 / 219.  256 experts of 96 rows on average, the
  // largest 48 times the smallest: gate/up 266 against 245.
  const int64_t avg = (static_cast<int64_t>(q.rows) + q.E - 1) / q.E;
  const bool pair = avg > Single::NMAX && di.sms >= 2;
  Params p;
  const int wrows = pair && swiglu ? kTileRows / 2 : kTileRows;
  for (int a = 0; a < kNA; ++a) {
    const bool second = swiglu && a == 1;
    if (!map_weight(&p.mapW[a], second ? q.w1_codes : q.w0_codes, q.E, q.N, q.K, wrows)) return MOE_ERR_CUDA;
    p.w_scales[a] = static_cast<const uint32_t*>(second ? q.w1_scales : q.w0_scales);
  }
  for (int b = 0; b < 4; ++b) {
    const cuuint64_t d[2] = {static_cast<cuuint64_t>(q.K / 2), static_cast<cuuint64_t>(q.rows)};
    const cuuint64_t s[1] = {static_cast<cuuint64_t>(q.K / 2)};
    const cuuint32_t box[2] = {128, 16u << b};
    if (!encode(&p.mapA[b], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, q.a_codes, d, s, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return MOE_ERR_CUDA;
  }
  p.a_scales = static_cast<const uint32_t*>(q.a_scales);
  p.offsets = q.offsets;
  p.out = q.out;
  p.out_scales = static_cast<uint8_t*>(q.out_scales);
  p.err = err;
  p.rows = q.rows;
  p.E = q.E;
  p.N = q.N;
  p.K = q.K;
  p.timeout_cycles = 2 * static_cast<int64_t>(kWaitTimeoutNs);   // at up to 2 GHz: 2 s or more
  if (swiglu) return launch_kind<kOutSwiglu>(p, pair, di.sms, st);
  switch (q.dtype) {
    case MOE_BF16: return launch_kind<kOutBf16>(p, pair, di.sms, st);
    case MOE_FP16: return launch_kind<kOutFp16>(p, pair, di.sms, st);
    default: return launch_kind<kOutFp32>(p, pair, di.sms, st);
  }
}

}  // namespace moe

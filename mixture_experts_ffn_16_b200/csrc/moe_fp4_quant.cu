// moe_fp4_quant.cu - rows to MXFP4 and back, and quantisation fused with the
// dispatch of tokens to their expert-sorted rows.
//
// A warp takes 1024 consecutive elements as 4 x 32 groups of 8: four lanes
// share a block of 32, so the loads of 16-bit types are 16 bytes a lane and
// coalesced, and a block's largest magnitude takes two shuffles.  Each lane
// then holds 4 bytes of codes of four groups; a 4 x 4 exchange between the
// lanes of a block gives each lane one whole block, stored as 16 bytes.  Two
// more shuffles a group collect the four scale bytes of 128 elements in one
// word of scales[g][K/128][row][4]: the words of consecutive rows are
// neighbours, which is what a product's row tile loads.  Rows count as padded
// to 128 elements, so a word's 16 lanes and a block's 4 stay together.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_fp4.cuh"
#include "moe_internal.h"
#include "moe_ptx.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;

// Eight elements as they lie in memory: their largest magnitude as float bits
// (NaN above infinity above every number) and their multiples by a power of
// two.  16-bit types stay packed for the first, bf16 for both: the scaled
// value is exact in bf16, or so small (below 2^-126) that it rounds to 0.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  float4 a, b;
  // 32 bytes a lane in one access where the tensor allows it: two of 16 bytes
  // each touch every sector (4097 x 7168 rows: 23.7 us to MXFP4 and 25.0 back,
  // 21.8 and 22.9 this way).
  template <bool STREAM>
  __device__ __forceinline__ void load(const float* p, bool wide) {
    const float4* v = reinterpret_cast<const float4*>(p);
    if (wide) {
      asm volatile("ld.global.nc.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=f"(a.x), "=f"(a.y), "=f"(a.z), "=f"(a.w), "=f"(b.x), "=f"(b.y), "=f"(b.z), "=f"(b.w)
                   : "l"(p));        // volatile: stays behind the wait for the kernel before
    } else {
      a = STREAM ? __ldcs(v) : __ldg(v);
      b = STREAM ? __ldcs(v + 1) : __ldg(v + 1);
    }
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ uint32_t amax_bits() const {
    const uint32_t k = 0x7FFFFFFFu;
    return max(max(max(__float_as_uint(a.x) & k, __float_as_uint(a.y) & k),
                   max(__float_as_uint(a.z) & k, __float_as_uint(a.w) & k)),
               max(max(__float_as_uint(b.x) & k, __float_as_uint(b.y) & k),
                   max(__float_as_uint(b.z) & k, __float_as_uint(b.w) & k)));
  }
  __device__ __forceinline__ void times(float s, float (&f)[8]) const {
    f[0] = a.x * s; f[1] = a.y * s; f[2] = a.z * s; f[3] = a.w * s;
    f[4] = b.x * s; f[5] = b.y * s; f[6] = b.z * s; f[7] = b.w * s;
  }
};
template <>
struct Eight<__nv_bfloat16> {
  __nv_bfloat162 h[4];
  template <bool STREAM>
  __device__ __forceinline__ void load(const __nv_bfloat16* p, bool) {
    const uint4* v = reinterpret_cast<const uint4*>(p);
    *reinterpret_cast<uint4*>(h) = STREAM ? __ldcs(v) : __ldg(v);
  }
  __device__ __forceinline__ void zero() { *reinterpret_cast<uint4*>(h) = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ uint32_t amax_bits() const {
    const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])),
                                         __hmax2_nan(__habs2(h[2]), __habs2(h[3])));
    const uint32_t w = *reinterpret_cast<const uint32_t*>(&m);
    return max(w << 16, w & 0xFFFF0000u);
  }
  __device__ __forceinline__ void times(float s, float (&f)[8]) const {
    const __nv_bfloat162 s2 = __float2bfloat162_rn(s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 q = __bfloat1622float2(__hmul2(h[i], s2));
      f[2 * i] = q.x;
      f[2 * i + 1] = q.y;
    }
  }
};
template <>
struct Eight<__half> {
  __half2 h[4];
  template <bool STREAM>
  __device__ __forceinline__ void load(const __half* p, bool) {
    const uint4* v = reinterpret_cast<const uint4*>(p);
    *reinterpret_cast<uint4*>(h) = STREAM ? __ldcs(v) : __ldg(v);
  }
  __device__ __forceinline__ void zero() { *reinterpret_cast<uint4*>(h) = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ uint32_t amax_bits() const {
    const float2 m = __half22float2(__hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])),
                                                __hmax2_nan(__habs2(h[2]), __habs2(h[3]))));
    return max(__float_as_uint(m.x), __float_as_uint(m.y));
  }
  __device__ __forceinline__ void times(float s, float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 q = __half22float2(h[i]);
      f[2 * i] = q.x * s;
      f[2 * i + 1] = q.y * s;
    }
  }
};
__device__ __forceinline__ void store8(float* p, const float (&f)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.f32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};"
                 ::"f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]), "l"(p)
                 : "memory");
    return;
  }
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8], bool) {
  uint4 v;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = v;
}
__device__ __forceinline__ void store8(__half* p, const float (&f)[8], bool) {
  uint4 v;
  __half2* h = reinterpret_cast<__half2*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = v;
}

constexpr int kUnits = 4;                        // groups of 8 per lane
constexpr int kWarpGroups = 32 * kUnits;

// This lane's 8 elements to a word of codes; `word`: the four scale bytes of
// the 16 lanes' 128 elements (every lane of the 16 gets it).  All lanes of the
// warp take part; a lane behind the row's end passes zeros, and its byte of
// the word is 0.
template <typename T>
__device__ __forceinline__ uint32_t quantize8(const Eight<T>& x, uint32_t* word) {
  uint32_t m = x.amax_bits();
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const uint32_t byte = fp4_scale_byte(m);
  uint32_t w = byte << (8 * ((threadIdx.x >> 2) & 3));
  w |= __shfl_xor_sync(0xffffffffu, w, 4);
  w |= __shfl_xor_sync(0xffffffffu, w, 8);
  *word = w;
  float f[8];
  x.times(fp4_inv_scale(byte), f);
  return byte == kFp4NanScale ? 0u : e2m1x8(f);
}

// 4 x 4 words between the four lanes of a block: lane i gets word i of lanes
// 0..3, in order.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
  const bool hi1 = threadIdx.x & 1, hi2 = threadIdx.x & 2;
  uint32_t a = __shfl_xor_sync(0xffffffffu, hi1 ? w[0] : w[1], 1);
  uint32_t b = __shfl_xor_sync(0xffffffffu, hi1 ? w[2] : w[3], 1);
  if (hi1) {
    w[0] = a;
    w[2] = b;
  } else {
    w[1] = a;
    w[3] = b;
  }
  a = __shfl_xor_sync(0xffffffffu, hi2 ? w[0] : w[2], 2);
  b = __shfl_xor_sync(0xffffffffu, hi2 ? w[1] : w[3], 2);
  if (hi2) {
    w[0] = a;
    w[1] = b;
  } else {
    w[2] = a;
    w[3] = b;
  }
}

// Rows of K elements as a flat sequence of groups of 8, each row padded to P
// groups.  Divisions by multiplication: by P with m64 = ceil(2^64 / P), exact
// for the first group of a warp (below 2^41, P at most 2^13), and with m32 =
// ceil(2^32 / P) for offsets below P + 128; by the rows of a matrix with g64 =
// ceil(2^64 / per_matrix) for rows below 2^28 (0 stands for 2^64, one matrix
// a row).
struct Layout {
  int64_t rows;
  uint64_t m64, g64;
  uint32_t m32;
  int P, groups, chunks, per_matrix;     // groups = K / 8; rows per matrix
  bool wide;                             // x starts at a multiple of 32 bytes
};

// The groups of one warp: they start at group rem0 of row row0.  WHOLE: K is a
// multiple of 1024, so the warp's 128 groups lie in one row and all exist.
struct Span {
  int64_t row0;
  uint32_t rem0;
  int left;          // rows from row0 on (capped)
};
__device__ __forceinline__ Span warp_span(const Layout& l) {
  const uint64_t first =
      (static_cast<uint64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * kWarpGroups;
  Span s;
  s.row0 = static_cast<int64_t>(__umul64hi(first, l.m64));
  s.rem0 = static_cast<uint32_t>(first - static_cast<uint64_t>(s.row0) * l.P);
  s.left = static_cast<int>(min(max(l.rows - s.row0, static_cast<int64_t>(0)), static_cast<int64_t>(kWarpGroups)));
  return s;
}
// Group `o` of the warp's: its row, counted from row0, and its place in the
// row; false behind the row's end or the last row.
template <bool WHOLE>
__device__ __forceinline__ bool locate(const Layout& l, const Span& s, int o, int* dr, int* u) {
  if constexpr (WHOLE) {
    *dr = 0;
    *u = static_cast<int>(s.rem0) + o;
    return s.left > 0;
  }
  const uint32_t t = s.rem0 + static_cast<uint32_t>(o);
  *dr = static_cast<int>(__umulhi(t, l.m32));
  *u = static_cast<int>(t) - *dr * l.P;
  return *dr < s.left && *u < l.groups;
}
// Word index of chunk c of row r in the scales.
__device__ __forceinline__ int64_t scale_at(const Layout& l, int64_t row, int chunk) {
  if (l.rows == l.per_matrix) return chunk * l.rows + row;
  const int64_t g = l.g64 ? static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(row), l.g64)) : row;
  return (g * l.chunks + chunk) * l.per_matrix + (row - g * l.per_matrix);
}

// SLOTS: row = token; the codes and scales go to the rows that its k slots
// have (slot_row), the token being read and quantised once.  Tokens and codes
// then pass through the L2 as streams, so that the scale words, 4 bytes here
// and there, can be gathered in it (360k rows of 7168: 470 -> 381 us).
template <typename T, bool SLOTS, bool WHOLE>
__global__ void __launch_bounds__(kThreads)
quantize_kernel(const T* __restrict__ x, uint4* __restrict__ codes, uint32_t* __restrict__ scales,
                const __grid_constant__ Layout l, const int32_t* __restrict__ slot_row, int k) {
  chain_wait();
  const int lane = threadIdx.x & 31;
  const Span s = warp_span(l);
  const T* x0 = x + s.row0 * l.groups * 8;
  Eight<T> f[kUnits];
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    int dr, u;
    if (locate<WHOLE>(l, s, 32 * j + lane, &dr, &u))
      f[j].template load<SLOTS>(x0 + (dr * l.groups + u) * 8, l.wide);
    else
      f[j].zero();
  }
  uint32_t w[kUnits], word = 0;       // word: lanes 0..7, the scales of the warp's chunk `lane`
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    uint32_t mine;
    w[j] = quantize8(f[j], &mine);
    const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 16);
    if (lane == 2 * j) word = mine;            // lanes below 16: the first chunk of the unit
    if (lane == 2 * j + 1) word = other;
  }
  transpose4(w);
  const uint4 block = make_uint4(w[0], w[1], w[2], w[3]);
  int bdr, bu, sdr, su;
  const bool bin = locate<WHOLE>(l, s, 32 * (lane & 3) + (lane & ~3), &bdr, &bu);   // this lane's block of 32
  const bool sin = locate<WHOLE>(l, s, 16 * (lane & 7), &sdr, &su) && lane < 8;             // lanes 0..7: chunk of 128
  const int64_t brow = s.row0 + bdr, srow = s.row0 + sdr;
  if constexpr (SLOTS) {
    const uint32_t R = static_cast<uint32_t>(l.rows) * static_cast<uint32_t>(k);
    const int32_t* bto = slot_row + brow * k;
    const int32_t* sto = slot_row + srow * k;
    uint4* const c0 = codes + (bu >> 2);
    uint32_t* const s0 = scales + static_cast<size_t>(su >> 4) * R;
    if constexpr (WHOLE) {
      // one token a warp: a lane a slot
      const uint32_t mine = (lane < k && s.left > 0) ? static_cast<uint32_t>(__ldg(bto + lane)) : R;
#pragma unroll 4
      for (int j = 0; j < k; ++j) {
        const uint32_t r = __shfl_sync(0xffffffffu, mine, j);
        if (r >= R) continue;
        __stcs(c0 + static_cast<size_t>(r) * (l.groups >> 2), block);
        if (lane < 8) s0[r] = word;
      }
      return;
    }
#pragma unroll 4
    for (int j = 0; j < k; ++j) {
      if (bin) {
        const uint32_t r = static_cast<uint32_t>(__ldg(bto + j));
        if (r < R) __stcs(c0 + static_cast<size_t>(r) * (l.groups >> 2), block);
      }
      if (sin) {
        const uint32_t r = static_cast<uint32_t>(__ldg(sto + j));
        if (r < R) s0[r] = word;
      }
    }
  } else {
    if (bin) codes[(brow * l.groups + bu) >> 2] = block;
    if (sin) scales[scale_at(l, srow, su >> 4)] = word;
  }
}

template <typename T, bool WHOLE>
__global__ void __launch_bounds__(kThreads)
dequantize_kernel(const uint4* __restrict__ codes, const uint32_t* __restrict__ scales, T* __restrict__ x,
                  const __grid_constant__ Layout l) {
  chain_wait();
  const int lane = threadIdx.x & 31;
  const Span s = warp_span(l);
  int bdr, bu;                                                  // the block of 32 this lane loads
  const bool bin = locate<WHOLE>(l, s, 32 * (lane & 3) + (lane & ~3), &bdr, &bu);
  uint32_t w[kUnits] = {0, 0, 0, 0}, byte = 0;
  if (bin) {
    const int64_t brow = s.row0 + bdr;
    const uint4 v = __ldg(codes + ((brow * l.groups + bu) >> 2));
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    byte = (__ldg(scales + scale_at(l, brow, bu >> 4)) >> (8 * ((bu >> 2) & 3))) & 255u;
  }
  transpose4(w);                                                // unit j: group 32 j + lane
  T* x0 = x + s.row0 * l.groups * 8;
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    // unit j of this lane lies in the block that lane (lane & ~3) + j loaded
    const float sc = fp4_scale(__shfl_sync(0xffffffffu, byte, (lane & ~3) + j));
    int dr, u;
    if (locate<WHOLE>(l, s, 32 * j + lane, &dr, &u)) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t h = e2m1x2_to_half2((w[j] >> (8 * i)) & 255u);
        const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&h));
        f[2 * i] = q.x * sc;
        f[2 * i + 1] = q.y * sc;
      }
      store8(x0 + (dr * l.groups + u) * 8, f, l.wide);
    }
  }
}

Layout make_layout(int64_t rows, int per_matrix, int K, const void* x) {
  Layout l;
  l.rows = rows;
  l.wide = (reinterpret_cast<uintptr_t>(x) & 31u) == 0;
  l.per_matrix = per_matrix;
  l.chunks = (K + 127) / 128;
  l.groups = K / 8;
  l.P = 16 * l.chunks;
  l.m64 = ~0ull / l.P + 1;          // ceil(2^64 / P), P being at least 16 (a power of two: exactly 2^64 / P)
  l.m32 = static_cast<uint32_t>(((1ull << 32) + l.P - 1) / l.P);
  l.g64 = per_matrix > 1 ? ~0ull / per_matrix + 1 : 0;
  return l;
}
dim3 layout_grid(const Layout& l) {
  const int64_t per_block = static_cast<int64_t>(kThreads / 32) * kWarpGroups;
  return dim3(static_cast<unsigned>((l.rows * l.P + per_block - 1) / per_block));
}

template <typename T, bool SLOTS>
int quantize_t(int64_t rows, int per_matrix, int K, const void* x, const int32_t* slot_row, int k, void* codes,
               void* scales, cudaStream_t st) {
  const Layout l = make_layout(rows, per_matrix, K, x);
  const auto kern = K % 1024 ? quantize_kernel<T, SLOTS, false> : quantize_kernel<T, SLOTS, true>;
  return launch_chained(kern, layout_grid(l), dim3(kThreads), 0, st, static_cast<const T*>(x),
                        static_cast<uint4*>(codes), static_cast<uint32_t*>(scales), l, slot_row, k) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

template <typename T>
int dequantize_t(int64_t rows, int per_matrix, int K, const void* codes, const void* scales, void* x,
                 cudaStream_t st) {
  const Layout l = make_layout(rows, per_matrix, K, x);
  const auto kern = K % 1024 ? dequantize_kernel<T, false> : dequantize_kernel<T, true>;
  return launch_chained(kern, layout_grid(l), dim3(kThreads), 0, st,
                        static_cast<const uint4*>(codes), static_cast<const uint32_t*>(scales), static_cast<T*>(x),
                        l) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

}  // namespace

int launch_quantize_fp4(int G, int rows, int K, int dtype, const void* x, void* codes, void* scales,
                        cudaStream_t st) {
  const int64_t all = static_cast<int64_t>(G) * rows;
  switch (dtype) {
    case MOE_BF16: return quantize_t<__nv_bfloat16, false>(all, rows, K, x, nullptr, 0, codes, scales, st);
    case MOE_FP16: return quantize_t<__half, false>(all, rows, K, x, nullptr, 0, codes, scales, st);
    default: return quantize_t<float, false>(all, rows, K, x, nullptr, 0, codes, scales, st);
  }
}

int launch_dispatch_fp4(int T, int k, int d, int dtype, const void* x, const int32_t* slot_row, void* codes,
                        void* scales, cudaStream_t st) {
  switch (dtype) {
    case MOE_BF16: return quantize_t<__nv_bfloat16, true>(T, T, d, x, slot_row, k, codes, scales, st);
    case MOE_FP16: return quantize_t<__half, true>(T, T, d, x, slot_row, k, codes, scales, st);
    default: return quantize_t<float, true>(T, T, d, x, slot_row, k, codes, scales, st);
  }
}

int launch_dequantize_fp4(int G, int rows, int K, int dtype, const void* codes, const void* scales, void* x,
                          cudaStream_t st) {
  const int64_t all = static_cast<int64_t>(G) * rows;
  switch (dtype) {
    case MOE_BF16: return dequantize_t<__nv_bfloat16>(all, rows, K, codes, scales, x, st);
    case MOE_FP16: return dequantize_t<__half>(all, rows, K, codes, scales, x, st);
    default: return dequantize_t<float>(all, rows, K, codes, scales, x, st);
  }
}

}  // namespace moe

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

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[8]) {
  const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 q = __bfloat1622float2(h[i]);
    f[2 * i] = q.x;
    f[2 * i + 1] = q.y;
  }
}
__device__ __forceinline__ void load8(const __half* p, float (&f)[8]) {
  const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
  const __half2* h = reinterpret_cast<const __half2*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 q = __half22float2(h[i]);
    f[2 * i] = q.x;
    f[2 * i + 1] = q.y;
  }
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
  uint4 v;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = v;
}
__device__ __forceinline__ void store8(__half* p, const float (&f)[8]) {
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
__device__ __forceinline__ uint32_t quantize8(float (&f)[8], uint32_t* word) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const uint32_t byte = fp4_scale_byte(m);
  uint32_t w = byte << (8 * ((threadIdx.x >> 2) & 3));
  w |= __shfl_xor_sync(0xffffffffu, w, 4);
  w |= __shfl_xor_sync(0xffffffffu, w, 8);
  *word = w;
  if (byte == kFp4NanScale) return 0u;
  const float inv = fp4_inv_scale(byte);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] *= inv;
  return e2m1x8(f);
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
// groups.  Division by P by multiplication: m64 = ceil(2^64 / P) is exact for
// the first group of a warp (below 2^41, P at most 2^13), m32 = ceil(2^32 / P)
// for offsets below P + 128.
struct Layout {
  int64_t rows;
  uint64_t m64;
  uint32_t m32;
  int P, groups, chunks, per_matrix;     // groups = K / 8; rows per matrix
};

struct Span {
  int64_t row0;
  uint32_t rem0;
};
__device__ __forceinline__ Span warp_span(const Layout& l) {
  const uint64_t first =
      (static_cast<uint64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * kWarpGroups;
  Span s;
  s.row0 = static_cast<int64_t>(__umul64hi(first, l.m64));
  s.rem0 = static_cast<uint32_t>(first - static_cast<uint64_t>(s.row0) * l.P);
  return s;
}
// Group `o` of the warp's: its row and its place in the row.
__device__ __forceinline__ void locate(const Layout& l, const Span& s, int o, int64_t* row, int* u) {
  const uint32_t t = s.rem0 + static_cast<uint32_t>(o);
  const uint32_t dr = __umulhi(t, l.m32);
  *row = s.row0 + dr;
  *u = static_cast<int>(t - dr * static_cast<uint32_t>(l.P));
}
// Word index of chunk c of row r in the scales.
__device__ __forceinline__ int64_t scale_at(const Layout& l, int64_t row, int chunk) {
  if (l.rows == l.per_matrix) return chunk * l.rows + row;
  const int64_t g = row / l.per_matrix;
  return (g * l.chunks + chunk) * l.per_matrix + (row - g * l.per_matrix);
}

// SLOTS: row = token; the codes and scales go to the rows that its k slots
// have (slot_row), the token being read and quantised once.
template <typename T, bool SLOTS>
__global__ void __launch_bounds__(kThreads)
quantize_kernel(const T* __restrict__ x, uint4* __restrict__ codes, uint32_t* __restrict__ scales,
                const __grid_constant__ Layout l, const int32_t* __restrict__ slot_row, int k) {
  chain_wait();
  const int lane = threadIdx.x & 31;
  const Span s = warp_span(l);
  float f[kUnits][8];
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    int64_t row;
    int u;
    locate(l, s, 32 * j + lane, &row, &u);
    if (row < l.rows && u < l.groups) {
      load8(x + (row * l.groups + u) * 8, f[j]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[j][i] = 0.0f;
    }
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
  int64_t brow, srow;
  int bu, su;
  locate(l, s, 32 * (lane & 3) + (lane & ~3), &brow, &bu);      // this lane's block of 32
  locate(l, s, 16 * (lane & 7), &srow, &su);                    // and, lanes 0..7, chunk of 128
  const bool bin = brow < l.rows && bu < l.groups, sin = lane < 8 && srow < l.rows;
  if constexpr (SLOTS) {
    const uint32_t R = static_cast<uint32_t>(l.rows) * static_cast<uint32_t>(k);
    const int32_t* bto = slot_row + brow * k;
    const int32_t* sto = slot_row + srow * k;
#pragma unroll 4
    for (int j = 0; j < k; ++j) {
      if (bin) {
        const uint32_t r = static_cast<uint32_t>(__ldg(bto + j));
        if (r < R) codes[(static_cast<size_t>(r) * l.groups + bu) >> 2] = block;
      }
      if (sin) {
        const uint32_t r = static_cast<uint32_t>(__ldg(sto + j));
        if (r < R) scales[static_cast<size_t>(su >> 4) * R + r] = word;
      }
    }
  } else {
    if (bin) codes[(brow * l.groups + bu) >> 2] = block;
    if (sin) scales[scale_at(l, srow, su >> 4)] = word;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
dequantize_kernel(const uint4* __restrict__ codes, const uint32_t* __restrict__ scales, T* __restrict__ x,
                  const __grid_constant__ Layout l) {
  chain_wait();
  const int lane = threadIdx.x & 31;
  const Span s = warp_span(l);
  int64_t brow;
  int bu;
  locate(l, s, 32 * (lane & 3) + (lane & ~3), &brow, &bu);      // the block of 32 this lane loads
  uint32_t w[kUnits] = {0, 0, 0, 0}, byte = 0;
  if (brow < l.rows && bu < l.groups) {
    const uint4 v = __ldg(codes + ((brow * l.groups + bu) >> 2));
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    byte = (__ldg(scales + scale_at(l, brow, bu >> 4)) >> (8 * ((bu >> 2) & 3))) & 255u;
  }
  transpose4(w);                                                // unit j: group 32 j + lane
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    // unit j of this lane lies in the block that lane (lane & ~3) + j loaded
    const float sc = fp4_scale(__shfl_sync(0xffffffffu, byte, (lane & ~3) + j));
    int64_t row;
    int u;
    locate(l, s, 32 * j + lane, &row, &u);
    if (row < l.rows && u < l.groups) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t h = e2m1x2_to_half2((w[j] >> (8 * i)) & 255u);
        const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&h));
        f[2 * i] = q.x * sc;
        f[2 * i + 1] = q.y * sc;
      }
      store8(x + (row * l.groups + u) * 8, f);
    }
  }
}

Layout make_layout(int64_t rows, int per_matrix, int K) {
  Layout l;
  l.rows = rows;
  l.per_matrix = per_matrix;
  l.chunks = (K + 127) / 128;
  l.groups = K / 8;
  l.P = 16 * l.chunks;
  l.m64 = ~0ull / l.P + 1;          // ceil(2^64 / P), P being at least 16 (a power of two: exactly 2^64 / P)
  l.m32 = static_cast<uint32_t>(((1ull << 32) + l.P - 1) / l.P);
  return l;
}
dim3 layout_grid(const Layout& l) {
  const int64_t per_block = static_cast<int64_t>(kThreads / 32) * kWarpGroups;
  return dim3(static_cast<unsigned>((l.rows * l.P + per_block - 1) / per_block));
}

template <typename T, bool SLOTS>
int quantize_t(int64_t rows, int per_matrix, int K, const void* x, const int32_t* slot_row, int k, void* codes,
               void* scales, cudaStream_t st) {
  const Layout l = make_layout(rows, per_matrix, K);
  return launch_chained(quantize_kernel<T, SLOTS>, layout_grid(l), dim3(kThreads), 0, st, static_cast<const T*>(x),
                        static_cast<uint4*>(codes), static_cast<uint32_t*>(scales), l, slot_row, k) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

template <typename T>
int dequantize_t(int64_t rows, int per_matrix, int K, const void* codes, const void* scales, void* x,
                 cudaStream_t st) {
  const Layout l = make_layout(rows, per_matrix, K);
  return launch_chained(dequantize_kernel<T>, layout_grid(l), dim3(kThreads), 0, st,
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

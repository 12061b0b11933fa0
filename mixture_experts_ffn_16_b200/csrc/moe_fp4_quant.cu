// moe_fp4_quant.cu - rows to MXFP4 and back, and quantisation fused with the
// dispatch of tokens to their expert-sorted rows.
//
// Four lanes share a block of 32 elements, 8 each: 16-byte loads of 16-bit
// types, two shuffles for the block's largest magnitude, four bytes of codes
// a lane.  Two more shuffles collect the four scale bytes of 128 elements in
// one word, stored as scales[g][K/128][row][4]: the words of consecutive rows
// are neighbours, which is what a product's row tile loads.
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

// Thread -> (row, group of 8 elements), rows padded to whole 128-element
// chunks so that the 16 lanes of a chunk stay together.
struct Where {
  int64_t row;
  int u;          // group of 8 in the row
  bool row_in;
};
__device__ __forceinline__ Where place(int64_t rows, int padded) {
  Where p;
  if (padded >= kThreads) {
    p.row = blockIdx.x;
    p.u = blockIdx.y * kThreads + threadIdx.x;
    p.row_in = p.u < padded;
  } else {
    const int lr = threadIdx.x / padded, per = kThreads / padded;
    p.row = static_cast<int64_t>(blockIdx.x) * per + lr;
    p.u = threadIdx.x - lr * padded;
    p.row_in = lr < per && p.row < rows;
  }
  return p;
}
dim3 place_grid(int64_t rows, int padded) {
  if (padded >= kThreads) return dim3(static_cast<unsigned>(rows), (padded + kThreads - 1) / kThreads);
  const int per = kThreads / padded;
  return dim3(static_cast<unsigned>((rows + per - 1) / per));
}

// SLOTS: row = token; the codes and scales go to the rows that its k slots
// have (slot_row), the token being read and quantised once.
template <typename T, bool SLOTS>
__global__ void __launch_bounds__(kThreads)
quantize_kernel(const T* __restrict__ x, uint32_t* __restrict__ codes, uint32_t* __restrict__ scales, int64_t rows,
                int per_matrix, int K, const int32_t* __restrict__ slot_row, int k) {
  chain_wait();
  const int chunks = (K + 127) / 128, padded = 16 * chunks, groups = K / 8;
  const Where p = place(rows, padded);
  float f[8];
  const bool in = p.row_in && p.u < groups;
  if (in) {
    load8(x + p.row * K + 8 * p.u, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 0.0f;
  }
  uint32_t word;
  const uint32_t code = quantize8(f, &word);
  const bool first = p.row_in && (threadIdx.x & 15) == 0;     // writes the chunk's scale word
  const int chunk = p.u >> 4;
  if constexpr (SLOTS) {
    if (!p.row_in) return;
    const uint32_t R = static_cast<uint32_t>(rows) * static_cast<uint32_t>(k);
    const int32_t* to = slot_row + p.row * k;
#pragma unroll 4
    for (int j = 0; j < k; ++j) {
      const uint32_t r = static_cast<uint32_t>(__ldg(to + j));
      if (r >= R) continue;
      if (in) codes[static_cast<size_t>(r) * groups + p.u] = code;
      if (first) scales[static_cast<size_t>(chunk) * R + r] = word;
    }
  } else {
    if (in) codes[p.row * groups + p.u] = code;
    if (first) {
      const int64_t g = p.row / per_matrix, r = p.row - g * per_matrix;
      scales[(g * chunks + chunk) * per_matrix + r] = word;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
dequantize_kernel(const uint32_t* __restrict__ codes, const uint32_t* __restrict__ scales, T* __restrict__ x,
                  int64_t rows, int per_matrix, int K) {
  chain_wait();
  const int chunks = (K + 127) / 128, groups = K / 8;
  const Where p = place(rows, 16 * chunks);
  if (!p.row_in || p.u >= groups) return;
  const int64_t g = p.row / per_matrix, r = p.row - g * per_matrix;
  const uint32_t word = __ldg(scales + (g * chunks + (p.u >> 4)) * per_matrix + r);
  const float sc = fp4_scale((word >> (8 * ((p.u >> 2) & 3))) & 255u);
  const uint32_t c = __ldg(codes + p.row * groups + p.u);
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = e2m1x2_to_half2((c >> (8 * i)) & 255u);
    const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&h));
    f[2 * i] = q.x * sc;
    f[2 * i + 1] = q.y * sc;
  }
  store8(x + p.row * K + 8 * p.u, f);
}

template <typename T, bool SLOTS>
int quantize_t(int64_t rows, int per_matrix, int K, const void* x, const int32_t* slot_row, int k, void* codes,
               void* scales, cudaStream_t st) {
  const int padded = (K + 127) / 128 * 16;
  return launch_chained(quantize_kernel<T, SLOTS>, place_grid(rows, padded), dim3(kThreads), 0, st,
                        static_cast<const T*>(x), static_cast<uint32_t*>(codes), static_cast<uint32_t*>(scales), rows,
                        per_matrix, K, slot_row, k) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

template <typename T>
int dequantize_t(int64_t rows, int per_matrix, int K, const void* codes, const void* scales, void* x,
                 cudaStream_t st) {
  const int padded = (K + 127) / 128 * 16;
  return launch_chained(dequantize_kernel<T>, place_grid(rows, padded), dim3(kThreads), 0, st,
                        static_cast<const uint32_t*>(codes), static_cast<const uint32_t*>(scales),
                        static_cast<T*>(x), rows, per_matrix, K) == cudaSuccess
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

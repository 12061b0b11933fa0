// moe_dispatch.cu - tokens to expert order and back, with the gradients:
//
//   sort        : (token, slot) pairs sorted stably by expert; row of each slot
//   dispatch    : x_sorted[row(t,j)] = x[t]
//   undispatch  : out[t] = sum_j w[t,j] y[row(t,j)]          (w = 1: the gradient of dispatch)
//   its gradient: dy[row(t,j)] = w[t,j] dout[t],  dw[t,j] = <dout[t], y[row(t,j)]>
//
// A slot without an expert (row -1) adds nothing, gets dw = 0, and no row is
// read or written for it.  Every kernel walks the tokens, not the rows: a
// token's row is read once for all of its copies, and sums over slots are
// taken by one thread in slot order, in fp32, so no atomics are needed and
// results do not depend on scheduling.
//
// Rows are bound by HBM: every sorted row is read or written once, as a stream
// (evict-first), which leaves the L2 to what is used again.  8191 tokens, 8
// slots, d = 2048, bf16: dispatch 44 us, undispatch 46 us (6.2-6.5 TB/s; 48 and
// 49 us without the hints), the weights' gradient 93 us (5.8 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_internal.h"
#include "moe_ptx.cuh"

namespace moe {

namespace {

// ---------------------------------------------------------------- sort

constexpr int kSortMaxCluster = 8;                       // the portable cluster size
constexpr int kSortBatch = 8;                            // groups of 32 slots a warp has in flight

// Warps of a CTA: 16 up to 1024 experts, above that 8, whose counters and lane
// masks (one of each per warp and expert) still fit in shared memory.
constexpr int sort_experts(int warps) { return warps == 16 ? 1024 : kMaxE; }

__device__ __forceinline__ uint32_t cluster_nctas() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ int ld_cluster(uint32_t cluster_addr) {
  int v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// One cluster sorts all slots.  Warp w < active of CTA c owns the c * active +
// w-th run of consecutive slots.  Pass 1 counts each warp's slots per expert in
// shared memory; prefix sums over warps, then (through distributed shared
// memory) over CTAs, then over experts give each (warp, expert) its first
// row; pass 2 walks the slots again and places them, 32 at a time, each
// behind the lower lanes with the same expert (each lane sets its bit in the
// expert's mask): the order of slots inside an expert is kept.  One launch
// instead of the count / scan / scatter of three.  Bound by the instructions
// of pass 2 on the cluster's SMs: 65k slots of 256 experts 7.7 us (15.1 us with
// a warp match for the lanes of one expert, 11.0 us with a vote per bit), 360k
// of 896 experts 29 us; 640 slots of 512 experts 3.1 us.
template <int WARPS>
__global__ void __launch_bounds__(32 * WARPS)
sort_kernel(const int32_t* __restrict__ topk_idx, int n, int E, int run, int active, int32_t* __restrict__ offsets,
            int32_t* __restrict__ slot_row, uint32_t* __restrict__ err) {
  constexpr int kThreads = 32 * WARPS, kPer = sort_experts(WARPS) / kThreads;   // kPer: experts per thread
  extern __shared__ int32_t sm[];
  int32_t* hist = sm;                       // [WARPS][E]
  int32_t* total = sm + WARPS * E;          // [E] this CTA's counts
  uint32_t* masks = reinterpret_cast<uint32_t*>(total + E);   // [WARPS][E]
  __shared__ int32_t wsum[WARPS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank(), ctas = cluster_nctas();
  for (int i = tid; i < active * E; i += kThreads) {
    hist[i] = 0;
    masks[i] = 0;
  }
  chain_wait();
  if (rank == 0 && tid == 0) *err = 0;
  __syncthreads();

  int32_t* mine = hist + warp * E;
  const int64_t lo = warp < active ? static_cast<int64_t>(rank * active + warp) * run : n;
  const int begin = static_cast<int>(min(lo, static_cast<int64_t>(n)));
  const int end = static_cast<int>(min(lo + run, static_cast<int64_t>(n)));
  // The loads of a batch are issued before any is used.
  auto load = [&](int (&e)[kSortBatch], int i0) {
#pragma unroll
    for (int q = 0; q < kSortBatch; ++q) {
      const int i = i0 + 32 * q + lane;
      e[q] = (i < end) ? __ldg(topk_idx + i) : -1;
    }
  };
  for (int i0 = begin; i0 < end; i0 += 32 * kSortBatch) {
    int e[kSortBatch];
    load(e, i0);
#pragma unroll
    for (int q = 0; q < kSortBatch; ++q)
      if (e[q] >= 0 && e[q] < E) atomicAdd(mine + e[q], 1);
  }
  __syncthreads();
  for (int e = tid; e < E; e += kThreads) {
    int s = 0;
#pragma unroll 4
    for (int w = 0; w < active; ++w) {
      const int c = hist[w * E + e];
      hist[w * E + e] = s;
      s += c;
    }
    total[e] = s;
  }
  const bool alone = ctas == 1;
  if (alone)
    __syncthreads();
  else
    cluster_sync();

  // thread t: experts t * per .. + per - 1
  const int per = (E + kThreads - 1) / kThreads;
  int below[kPer], all[kPer];
  int sum = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    below[q] = all[q] = 0;
    const int e = tid * per + q;
    if (q < per && e < E) {
      if (alone) {
        all[q] = total[e];
      } else {
#pragma unroll
        for (uint32_t c = 0; c < kSortMaxCluster; ++c) {
          const int v = c < ctas ? ld_cluster(mapa_shared(smem_u32(total + e), c)) : 0;
          if (c < rank) below[q] += v;
          all[q] += v;
        }
      }
      sum += all[q];
    }
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) wsum[warp] = inc;
  if (alone)
    __syncthreads();
  else
    cluster_sync();    // every CTA's reads of `total` are done; wsum is written
  int base = inc - sum;
  for (int w = 0; w < warp; ++w) base += wsum[w];
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int e = tid * per + q;
    if (q < per && e < E) {
      if (rank == 0) offsets[e] = base;
#pragma unroll 4
      for (int w = 0; w < active; ++w) hist[w * E + e] += base + below[q];    // first row of each warp's
      base += all[q];
      if (rank == 0 && e == E - 1) offsets[E] = base;
    }
  }
  __syncthreads();

  uint32_t lt;
  asm volatile("mov.u32 %0, %%lanemask_lt;" : "=r"(lt));
  uint32_t* mask = masks + warp * E;
  bool bad = false;
  for (int i0 = begin; i0 < end; i0 += 32 * kSortBatch) {
    int e[kSortBatch];
    load(e, i0);
#pragma unroll
    for (int q = 0; q < kSortBatch; ++q) {
      if (i0 + 32 * q >= end) break;
      const int x = e[q];
      const bool has = x >= 0 && x < E;
      bad |= !has && x != -1;
      if (has) atomicOr(mask + x, 1u << lane);
      __syncwarp();
      int row = -1;
      uint32_t peers = 0;
      if (has) {
        peers = mask[x];
        row = mine[x] + __popc(peers & lt);
      }
      __syncwarp();
      if (has && (peers & lt) == 0) {        // the first of them
        mask[x] = 0;
        mine[x] += __popc(peers);
      }
      __syncwarp();
      const int i = i0 + 32 * q + lane;
      if (i < end) slot_row[i] = row;
    }
  }
  if (bad) atomicOr(err, kDevErrBadRouting);
}

// ---------------------------------------------------------------- rows

constexpr int kRowThreads = 256;
constexpr int kBatch = 8;              // rows a thread has in flight

template <typename T>
struct Vec;                            // 16 bytes of T as floats
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(const uint4 v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4 v, float (&f)[8]) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = __bfloat1622float2(h[i]);
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[8]) {
    uint4 v;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    return v;
  }
};
template <>
struct Vec<__half> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4 v, float (&f)[8]) {
    const __half2* h = reinterpret_cast<const __half2*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = __half22float2(h[i]);
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[8]) {
    uint4 v;
    __half2* h = reinterpret_cast<__half2*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    return v;
  }
};

// Thread -> (token, 16-byte unit of its row).  Rows of kRowThreads units or
// more: blockIdx.y picks the piece of the row; shorter rows: a block takes
// several tokens.
struct Where {
  int t, u;
  bool in;
};
__device__ __forceinline__ Where place(int T, int units) {
  Where p;
  if (units >= kRowThreads) {
    p.t = blockIdx.x;
    p.u = blockIdx.y * kRowThreads + threadIdx.x;
    p.in = p.u < units;
  } else {
    const int lt = threadIdx.x / units, per = kRowThreads / units;
    p.t = blockIdx.x * per + lt;
    p.u = threadIdx.x - lt * units;
    p.in = lt < per && p.t < T;
  }
  return p;
}
dim3 place_grid(int T, int units) {
  if (units >= kRowThreads) return dim3(T, (units + kRowThreads - 1) / kRowThreads);
  const int per = kRowThreads / units;
  return dim3((T + per - 1) / per);
}

__global__ void __launch_bounds__(kRowThreads)
dispatch_kernel(const uint4* __restrict__ x, const int32_t* __restrict__ slot_row, uint4* __restrict__ xs, int T,
                int k, int units) {
  chain_wait();
  const Where p = place(T, units);
  if (!p.in) return;
  const int32_t* rows = slot_row + static_cast<size_t>(p.t) * k;
  const uint32_t R = static_cast<uint32_t>(T) * static_cast<uint32_t>(k);
  const uint4 v = __ldg(x + static_cast<size_t>(p.t) * units + p.u);
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const uint32_t r = static_cast<uint32_t>(__ldg(rows + j));
    if (r < R) __stcs(xs + static_cast<size_t>(r) * units + p.u, v);
  }
}

template <typename T, bool WEIGHTED>
__global__ void __launch_bounds__(kRowThreads)
undispatch_kernel(const uint4* __restrict__ y, const int32_t* __restrict__ slot_row, const float* __restrict__ w,
                  uint4* __restrict__ out, int tokens, int k, int units) {
  constexpr int N = Vec<T>::N;
  chain_wait();
  const Where p = place(tokens, units);
  if (!p.in) return;
  const size_t s0 = static_cast<size_t>(p.t) * k;
  const uint32_t R = static_cast<uint32_t>(tokens) * static_cast<uint32_t>(k);
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.0f;
  for (int j0 = 0; j0 < k; j0 += kBatch) {
    uint4 v[kBatch];
    bool has[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      has[q] = false;
      if (j0 + q < k) {
        const uint32_t r = static_cast<uint32_t>(__ldg(slot_row + s0 + j0 + q));
        has[q] = r < R;
        if (has[q]) v[q] = __ldcs(y + static_cast<size_t>(r) * units + p.u);
      }
    }
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      if (has[q]) {
        float f[N];
        Vec<T>::get(v[q], f);
        const float g = WEIGHTED ? __ldg(w + s0 + j0 + q) : 1.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = fmaf(g, f[i], acc[i]);
      }
    }
  }
  out[static_cast<size_t>(p.t) * units + p.u] = Vec<T>::put(acc);
}

// One CTA per token: the token's dout is read once; for every slot its row of
// y is read (dot product) and its row of dy written.  KM: an upper bound of k
// that keeps the k partial dots in registers.
template <typename T, int KM>
__global__ void __launch_bounds__(kRowThreads, KM <= 8 ? 3 : 1)
undispatch_backward_kernel(const uint4* __restrict__ dout, const uint4* __restrict__ y,
                           const int32_t* __restrict__ slot_row, const float* __restrict__ w, uint4* __restrict__ dy,
                           float* __restrict__ dw, int tokens, int k, int units) {
  constexpr int N = Vec<T>::N;
  __shared__ float red[kRowThreads / 32][KM];
  chain_wait();
  const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t s0 = static_cast<size_t>(t) * k;
  const uint32_t R = static_cast<uint32_t>(tokens) * static_cast<uint32_t>(k);
  float dot[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j) dot[j] = 0.0f;
  for (int u = threadIdx.x; u < units; u += blockDim.x) {
    float g[N];
    Vec<T>::get(__ldg(dout + static_cast<size_t>(t) * units + u), g);
#pragma unroll
    for (int j0 = 0; j0 < KM; j0 += kBatch) {
      if (j0 >= k) break;
      uint4 v[kBatch];
      uint32_t r[kBatch];
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        r[q] = (j0 + q < k) ? static_cast<uint32_t>(__ldg(slot_row + s0 + j0 + q)) : R;
        if (r[q] < R) v[q] = __ldcs(y + static_cast<size_t>(r[q]) * units + u);
      }
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        if (r[q] < R) {
          const float wj = __ldg(w + s0 + j0 + q);
          float f[N], o[N];
          Vec<T>::get(v[q], f);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            dot[j0 + q] = fmaf(g[i], f[i], dot[j0 + q]);
            o[i] = wj * g[i];
          }
          __stcs(dy + static_cast<size_t>(r[q]) * units + u, Vec<T>::put(o));
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < KM; ++j) {
    if (j >= k) break;
    float v = dot[j];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) red[warp][j] = v;
  }
  __syncthreads();
  if (threadIdx.x < static_cast<unsigned>(k)) {
    float v = 0.0f;
    for (unsigned i = 0; i < blockDim.x / 32; ++i) v += red[i][threadIdx.x];
    dw[s0 + threadIdx.x] = v;
  }
}

int ok_or_cuda(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

template <typename T>
int undispatch_t(int tokens, int k, int d, const void* y, const int32_t* slot_row, const float* w, void* out,
                 cudaStream_t st) {
  const int units = d / Vec<T>::N;
  const auto kern = w ? undispatch_kernel<T, true> : undispatch_kernel<T, false>;
  return ok_or_cuda(launch_chained(kern, place_grid(tokens, units), dim3(kRowThreads), 0, st,
                                   static_cast<const uint4*>(y), slot_row, w, static_cast<uint4*>(out), tokens, k,
                                   units));
}

template <typename T>
int undispatch_backward_t(int tokens, int k, int d, const void* dout, const void* y, const int32_t* slot_row,
                          const float* w, void* dy, float* dw, cudaStream_t st) {
  const int units = d / Vec<T>::N;
  const int threads = units >= kRowThreads ? kRowThreads : (units + 31) / 32 * 32;
  const auto kern = k <= 8    ? undispatch_backward_kernel<T, 8>
                    : k <= 16 ? undispatch_backward_kernel<T, 16>
                              : undispatch_backward_kernel<T, 32>;
  return ok_or_cuda(launch_chained(kern, dim3(tokens), dim3(threads), 0, st, static_cast<const uint4*>(dout),
                                   static_cast<const uint4*>(y), slot_row, w, static_cast<uint4*>(dy), dw, tokens, k,
                                   units));
}

}  // namespace

template <int WARPS>
static int launch_sort(int n, int E, const int32_t* topk_idx, int32_t* offsets, int32_t* slot_row, uint32_t* err,
                       cudaStream_t st) {
  // CTAs: enough that a warp walks one batch of slots, up to the portable
  // cluster size.
  int ctas = 1;
  while (ctas < kSortMaxCluster && static_cast<int64_t>(ctas) * 32 * WARPS * kSortBatch < n) ctas *= 2;
  // Of one CTA, as many warps as have half a batch each: the counters of every
  // warp are cleared and summed, which is most of the work of a small sort.
  int active = WARPS;
  if (ctas == 1) active = (n + 32 * kSortBatch / 2 - 1) / (32 * kSortBatch / 2);
  active = active < WARPS ? active : WARPS;
  const int warps = ctas * active;
  const int run = static_cast<int>((static_cast<int64_t>(n) + warps * 32 - 1) / (warps * 32)) * 32;
  static std::atomic<int> limit[64];
  const int rc = raise_smem_limit(sort_kernel<WARPS>, limit,
                                  (2 * WARPS + 1) * sort_experts(WARPS) * static_cast<int>(sizeof(int32_t)));
  if (rc != MOE_OK) return rc;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(32 * WARPS);
  cfg.dynamicSmemBytes = static_cast<size_t>(2 * WARPS + 1) * E * sizeof(int32_t);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return ok_or_cuda(cudaLaunchKernelEx(&cfg, sort_kernel<WARPS>, topk_idx, n, E, run, active, offsets, slot_row, err));
}

int launch_sort_tokens(int T, int k, int E, const int32_t* topk_idx, int32_t* offsets, int32_t* slot_row,
                       uint32_t* err, cudaStream_t st) {
  return E <= sort_experts(16) ? launch_sort<16>(T * k, E, topk_idx, offsets, slot_row, err, st)
                               : launch_sort<8>(T * k, E, topk_idx, offsets, slot_row, err, st);
}

int launch_dispatch(int T, int k, size_t row_bytes, const void* x, const int32_t* slot_row, void* x_sorted,
                    cudaStream_t st) {
  const int units = static_cast<int>(row_bytes / 16);
  return ok_or_cuda(launch_chained(dispatch_kernel, place_grid(T, units), dim3(kRowThreads), 0, st,
                                   static_cast<const uint4*>(x), slot_row, static_cast<uint4*>(x_sorted), T, k,
                                   units));
}

int launch_undispatch(int T, int k, int d, int dtype, const void* y, const int32_t* slot_row, const float* topk_w,
                      void* out, cudaStream_t st) {
  switch (dtype) {
    case MOE_BF16: return undispatch_t<__nv_bfloat16>(T, k, d, y, slot_row, topk_w, out, st);
    case MOE_FP16: return undispatch_t<__half>(T, k, d, y, slot_row, topk_w, out, st);
    default: return undispatch_t<float>(T, k, d, y, slot_row, topk_w, out, st);
  }
}

int launch_undispatch_backward(int T, int k, int d, int dtype, const void* dout, const void* y,
                               const int32_t* slot_row, const float* topk_w, void* dy, float* dw, cudaStream_t st) {
  switch (dtype) {
    case MOE_BF16: return undispatch_backward_t<__nv_bfloat16>(T, k, d, dout, y, slot_row, topk_w, dy, dw, st);
    case MOE_FP16: return undispatch_backward_t<__half>(T, k, d, dout, y, slot_row, topk_w, dy, dw, st);
    default: return undispatch_backward_t<float>(T, k, d, dout, y, slot_row, topk_w, dy, dw, st);
  }
}

}  // namespace moe

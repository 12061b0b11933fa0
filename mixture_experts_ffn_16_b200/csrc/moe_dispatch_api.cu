// moe_dispatch_api.cu - the C ABI of the token dispatch, its gradients and the
// MXFP4 operators (declared in include/moe.h): argument checks and launches.
#include "moe_internal.h"

namespace moe {

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Any null pointer: MOE_ERR_INVALID_ARG; any misaligned: MOE_ERR_UNSUPPORTED.
template <typename... P>
int check_ptrs(P... ptrs) {
  const void* all[] = {static_cast<const void*>(ptrs)...};
  for (const void* p : all)
    if (!p) return MOE_ERR_INVALID_ARG;
  for (const void* p : all)
    if (!aligned16(p)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_fp4(const moe_fp4_tensor* t) { return t ? check_ptrs(t->codes, t->scales) : MOE_ERR_INVALID_ARG; }

int check_tokens(int T, int k) {
  if (T < 1 || k < 1) return MOE_ERR_INVALID_ARG;
  return (T > (1 << 22) || k > kMaxK) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}
int check_width(int d) {
  if (d < 1) return MOE_ERR_INVALID_ARG;
  return (d % 64 || d > (1 << 16)) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}
int check_dtype(int dtype) { return dtype < MOE_BF16 || dtype > MOE_FP32 ? MOE_ERR_INVALID_ARG : MOE_OK; }
int check_rows(int64_t rows) {
  if (rows < 1) return MOE_ERR_INVALID_ARG;
  return rows > (static_cast<int64_t>(kMaxK) << 22) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}
int check_experts(int E) {
  if (E < 1) return MOE_ERR_INVALID_ARG;
  return E > kMaxE ? MOE_ERR_UNSUPPORTED : MOE_OK;
}
int check_workspace(const void* ws, size_t bytes) {
  return !ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || bytes < MOE_DISPATCH_WORKSPACE_BYTES
             ? MOE_ERR_WORKSPACE
             : MOE_OK;
}

// The first code of a list that is not MOE_OK.
template <typename... R>
int first_of(R... rcs) {
  int rc = MOE_OK;
  ((rc = rc == MOE_OK ? rcs : rc), ...);
  return rc;
}

int device(DeviceInfo* di) { return device_info(di) != MOE_OK || !di->ok ? MOE_ERR_UNSUPPORTED : MOE_OK; }
cudaStream_t as_stream(moe_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }
size_t size_of(int dtype) { return dtype == MOE_FP32 ? 4 : 2; }

int convert(bool quantize, int G, int rows, int K, int dtype, const void* x, const moe_fp4_tensor* q,
            moe_stream_t stream) {
  if (G < 1 || rows < 1) return MOE_ERR_INVALID_ARG;
  int rc = first_of(check_dtype(dtype), check_width(K), check_rows(static_cast<int64_t>(G) * rows), check_ptrs(x),
                    check_fp4(q));
  if (rc != MOE_OK) return rc;
  DeviceInfo di;
  if ((rc = device(&di)) != MOE_OK) return rc;
  return quantize ? launch_quantize_fp4(G, rows, K, dtype, x, q->codes, q->scales, as_stream(stream))
                  : launch_dequantize_fp4(G, rows, K, dtype, q->codes, q->scales, const_cast<void*>(x),
                                          as_stream(stream));
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

int moe_sort_tokens(int32_t T, int32_t k, int32_t E, const int32_t* topk_idx, int32_t* offsets, int32_t* slot_row,
                    void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  int rc = first_of(check_tokens(T, k), check_experts(E), check_ptrs(topk_idx, offsets, slot_row),
                    check_workspace(workspace, workspace_bytes));
  if (rc != MOE_OK) return rc;
  DeviceInfo di;
  if ((rc = device(&di)) != MOE_OK) return rc;
  return launch_sort_tokens(T, k, E, topk_idx, offsets, slot_row, static_cast<uint32_t*>(workspace),
                            as_stream(stream));
}

int moe_dispatch(int32_t T, int32_t k, int32_t d, int dtype, const void* x, const int32_t* slot_row, void* x_sorted,
                 moe_stream_t stream) {
  int rc = first_of(check_tokens(T, k), check_width(d), check_dtype(dtype), check_ptrs(x, slot_row, x_sorted));
  if (rc != MOE_OK) return rc;
  DeviceInfo di;
  if ((rc = device(&di)) != MOE_OK) return rc;
  return launch_dispatch(T, k, static_cast<size_t>(d) * size_of(dtype), x, slot_row, x_sorted, as_stream(stream));
}

int moe_dispatch_backward(int32_t T, int32_t k, int32_t d, int dtype, const void* dx_sorted, const int32_t* slot_row,
                          void* dx, moe_stream_t stream) {
  int rc = first_of(check_tokens(T, k), check_width(d), check_dtype(dtype), check_ptrs(dx_sorted, slot_row, dx));
  if (rc != MOE_OK) return rc;
  DeviceInfo di;
  if ((rc = device(&di)) != MOE_OK) return rc;
  return launch_undispatch(T, k, d, dtype, dx_sorted, slot_row, nullptr, dx, as_stream(stream));
}

int moe_undispatch(int32_t T, int32_t k, int32_t d, int dtype, const void* y, const int32_t* slot_row,
                   const float* topk_w, void* out, moe_stream_t stream) {
  int rc = first_of(check_tokens(T, k), check_width(d), check_dtype(dtype), check_ptrs(y, slot_row, topk_w, out));
  if (rc != MOE_OK) return rc;
  DeviceInfo di;
  if ((rc = device(&di)) != MOE_OK) return rc;
  return launch_undispatch(T, k, d, dtype, y, slot_row, topk_w, out, as_stream(stream));
}

int moe_undispatch_backward(int32_t T, int32_t k, int32_t d, int dtype, const void* dout, const void* y,
                            const int32_t* slot_row, const float* topk_w, void* dy, float* dw, moe_stream_t stream) {
  int rc = first_of(check_tokens(T, k), check_width(d), check_dtype(dtype),
                    check_ptrs(dout, y, slot_row, topk_w, dy, dw));
  if (rc != MOE_OK) return rc;
  DeviceInfo di;
  if ((rc = device(&di)) != MOE_OK) return rc;
  return launch_undispatch_backward(T, k, d, dtype, dout, y, slot_row, topk_w, dy, dw, as_stream(stream));
}

int moe_quantize_fp4(int32_t G, int32_t rows, int32_t K, int dtype, const void* x, const moe_fp4_tensor* q,
                     moe_stream_t stream) {
  return convert(true, G, rows, K, dtype, x, q, stream);
}

int moe_dequantize_fp4(int32_t G, int32_t rows, int32_t K, int dtype, const moe_fp4_tensor* q, void* x,
                       moe_stream_t stream) {
  return convert(false, G, rows, K, dtype, x, q, stream);
}

int moe_dispatch_fp4(int32_t T, int32_t k, int32_t d, int dtype, const void* x, const int32_t* slot_row,
                     const moe_fp4_tensor* x_sorted, moe_stream_t stream) {
  int rc = first_of(check_tokens(T, k), check_width(d), check_dtype(dtype), check_ptrs(x, slot_row),
                    check_fp4(x_sorted));
  if (rc != MOE_OK) return rc;
  DeviceInfo di;
  if ((rc = device(&di)) != MOE_OK) return rc;
  return launch_dispatch_fp4(T, k, d, dtype, x, slot_row, x_sorted->codes, x_sorted->scales, as_stream(stream));
}

int moe_matmul_fp4(int32_t rows, int32_t E, int32_t N, int32_t K, const moe_fp4_tensor* a, const int32_t* offsets,
                   const moe_fp4_tensor* W, int dtype, void* out, void* workspace, size_t workspace_bytes,
                   moe_stream_t stream) {
  int rc = first_of(check_rows(rows), check_experts(E), check_width(N), check_width(K), check_dtype(dtype),
                    check_fp4(a), check_fp4(W), check_ptrs(offsets, out),
                    check_workspace(workspace, workspace_bytes));
  if (rc != MOE_OK) return rc;
  DeviceInfo di;
  if ((rc = device(&di)) != MOE_OK) return rc;
  const Fp4Product q = {rows,      E,        N,       K,       dtype, a->codes, a->scales, offsets,
                        W->codes, W->scales, nullptr, nullptr, out,   nullptr};
  return launch_fp4_product(q, di, static_cast<uint32_t*>(workspace), as_stream(stream));
}

int moe_swiglu_fp4(int32_t rows, int32_t E, int32_t f, int32_t K, const moe_fp4_tensor* a, const int32_t* offsets,
                   const moe_fp4_tensor* W_gate, const moe_fp4_tensor* W_up, const moe_fp4_tensor* h, void* workspace,
                   size_t workspace_bytes, moe_stream_t stream) {
  int rc = first_of(check_rows(rows), check_experts(E), check_width(f), check_width(K), check_fp4(a),
                    check_fp4(W_gate), check_fp4(W_up), check_fp4(h), check_ptrs(offsets),
                    check_workspace(workspace, workspace_bytes));
  if (rc != MOE_OK) return rc;
  DeviceInfo di;
  if ((rc = device(&di)) != MOE_OK) return rc;
  const Fp4Product q = {rows,          E,              f,           K,            MOE_BF16, a->codes, a->scales, offsets,
                        W_gate->codes, W_gate->scales, W_up->codes, W_up->scales, h->codes, h->scales};
  return launch_fp4_product(q, di, static_cast<uint32_t*>(workspace), as_stream(stream));
}

}  // extern "C"

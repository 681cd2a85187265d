// sq_w4_api.cu -- the C ABI of the 4-bit weight operators (include/sq_w8a8.h): argument checks on
// the host, before any CUDA call, then the launches on the caller's stream.
#include <climits>
#include <mutex>
#include <set>
#include <utility>

#include "sq_w4.cuh"

namespace sqh {
cudaError_t launch_w4_fold(const void* W, bool bf16, int64_t K, int64_t N, int64_t ldw, const float* s,
                           const float* gamma, const float* beta, int group, uint8_t* wq, uint16_t* sg, uint8_t* zp,
                           float* gamma_f, float* beta_f, cudaStream_t st);
cudaError_t launch_w4_dequant(const uint8_t* wq, const uint16_t* sg, const uint8_t* zp, int64_t K, int64_t N, int group,
                              void* y, bool y_bf16, int64_t ldy, cudaStream_t st);
cudaError_t launch_w4_gemm(const void* x, bool bf16, int64_t M, int64_t K, int64_t ldx, const uint8_t* wq,
                           const uint16_t* sg, const uint8_t* zp, int64_t N, int group, void* y, bool y_bf16,
                           int64_t ldy, cudaStream_t st);
size_t moe_workspace_size(int64_t T, int64_t D, int64_t F, int64_t E, int64_t top_k);
cudaError_t launch_moe_w4(const void* x, bool bf16, int64_t T, int64_t D, int64_t ldx, const void* wr, bool wr_bf16,
                          int64_t E, int64_t top_k, bool renorm, int* ids, float* wts, const int* ids_in,
                          const float* wts_in, const uint8_t* w13, const uint16_t* s13, const uint8_t* z13,
                          const uint8_t* w2, const uint16_t* s2, const uint8_t* z2, int64_t F, int group, void* y,
                          bool y_bf16, int64_t ldy, void* workspace, cudaStream_t st);

cudaError_t allow_shared_memory(const void* kern, int64_t bytes) {
  static std::mutex mu;
  static std::set<std::pair<int, const void*>> done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  try {
    std::lock_guard<std::mutex> lock(mu);
    const auto key = std::make_pair(dev, kern);
    if (done.count(key)) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.insert(key);
  } catch (...) {  // out of host memory, or a lock that cannot be taken: no exception leaves a C entry
    return cudaErrorMemoryAllocation;
  }
  return e;
}
}  // namespace sqh

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int elt_size(sq_dtype dt) { return dt == SQ_BF16 ? 2 : 4; }
bool float_dtype(sq_dtype dt) { return dt == SQ_BF16 || dt == SQ_F32; }
sq_status cuda_status(cudaError_t e) { return e == cudaSuccess ? SQ_OK : SQ_ERR_CUDA; }

sq_status check_group(int group) {
  if (group <= 0) return SQ_ERR_INVALID_ARG;
  return group == 32 || group == 64 || group == 128 ? SQ_OK : SQ_ERR_UNSUPPORTED;
}

// A row-major matrix that is read or written in 16-byte vectors.
sq_status check_rows(const void* x, sq_dtype dt, int64_t rows, int64_t cols, int64_t ld) {
  if (!float_dtype(dt) || rows < 0 || cols < 0 || ld < cols) return SQ_ERR_INVALID_ARG;
  if (rows > 0 && cols > 0 && x == nullptr) return SQ_ERR_INVALID_ARG;
  const int e = elt_size(dt);
  if (!aligned(x, 16) || (cols * e) % 16 != 0 || (ld * e) % 16 != 0) return SQ_ERR_ALIGNMENT;
  return SQ_OK;
}

// A packed weight: codes 16-byte aligned, scales 2-byte aligned.
sq_status check_packed(const void* wq, const void* sg) {
  if (wq == nullptr || sg == nullptr) return SQ_ERR_INVALID_ARG;
  return aligned(wq, 16) && aligned(sg, 2) ? SQ_OK : SQ_ERR_ALIGNMENT;
}

// An output with a leading dimension, stored element by element.
sq_status check_out(const void* y, sq_dtype ydt, int64_t cols, int64_t ldy) {
  if (!float_dtype(ydt) || ldy < cols) return SQ_ERR_INVALID_ARG;
  return SQ_OK;
}

struct MoeArgs {
  const void* x;
  sq_dtype dt;
  int64_t T, D, ldx;
  const void* wr;
  sq_dtype rdt;
  int64_t E;
  int top_k, renorm;
  int* ids;
  float* wts;
  const int* ids_in;
  const float* wts_in;
  const uint8_t* w13;
  const uint16_t* s13;
  const uint8_t* z13;
  const uint8_t* w2;
  const uint16_t* s2;
  const uint8_t* z2;
  int64_t F;
  int group;
  void* y;
  sq_dtype ydt;
  int64_t ldy;
  void* workspace;
  size_t ws_bytes;
};

bool moe_sizes_ok(int64_t T, int64_t D, int64_t F, int64_t E, int64_t top_k) {
  return T >= 0 && D > 0 && F > 0 && E > 0 && top_k > 0 && top_k <= E;
}
bool moe_sizes_supported(int64_t T, int64_t D, int64_t F, int64_t E, int64_t top_k) {
  if (T > SQ_MOE_MAX_TOKENS || E > SQ_MOE_MAX_EXPERTS || top_k > SQ_MOE_MAX_TOP_K || D > SQ_MAX_K || F > SQ_MAX_K)
    return false;
  // an expert's codes are reached by 32-bit offsets
  return 2 * F * sq_w4_row_bytes(D) <= (int64_t)UINT_MAX && D * sq_w4_row_bytes(F) <= (int64_t)UINT_MAX;
}

sq_status run_moe(const MoeArgs& a, bool routed, void* stream) {
  if (!moe_sizes_ok(a.T, a.D, a.F, a.E, a.top_k)) return SQ_ERR_INVALID_ARG;
  if (a.renorm != 0 && a.renorm != 1) return SQ_ERR_INVALID_ARG;
  sq_status st = check_group(a.group);
  if (st != SQ_OK) return st;
  st = check_rows(a.x, a.dt, a.T, a.D, a.ldx);
  if (st != SQ_OK) return st;
  st = check_out(a.y, a.ydt, a.D, a.ldy);
  if (st != SQ_OK) return st;
  if (!routed && !float_dtype(a.rdt)) return SQ_ERR_INVALID_ARG;
  if (a.T == 0) return SQ_OK;
  if (a.y == nullptr || (a.z13 == nullptr) != (a.z2 == nullptr)) return SQ_ERR_INVALID_ARG;
  if (routed ? (!a.ids_in || !a.wts_in) : (!a.wr || !a.ids || !a.wts)) return SQ_ERR_INVALID_ARG;
  st = check_packed(a.w13, a.s13);
  if (st != SQ_OK) return st;
  st = check_packed(a.w2, a.s2);
  if (st != SQ_OK) return st;
  if (!aligned(a.s13, 16) || !aligned(a.s2, 16) || !aligned(a.z13, 16) || !aligned(a.z2, 16)) return SQ_ERR_ALIGNMENT;
  if (a.D % 16 != 0 || a.F % 16 != 0 || !aligned(a.y, elt_size(a.ydt))) return SQ_ERR_ALIGNMENT;
  if (!aligned(a.wr, 16) || !aligned(a.ids, 4) || !aligned(a.wts, 4) || !aligned(a.ids_in, 4) || !aligned(a.wts_in, 4))
    return SQ_ERR_ALIGNMENT;
  if (!moe_sizes_supported(a.T, a.D, a.F, a.E, a.top_k)) return SQ_ERR_UNSUPPORTED;
  if (a.workspace == nullptr || a.ws_bytes < sqh::moe_workspace_size(a.T, a.D, a.F, a.E, a.top_k)) return SQ_ERR_WORKSPACE;
  if (!aligned(a.workspace, 256)) return SQ_ERR_ALIGNMENT;
  return cuda_status(sqh::launch_moe_w4(a.x, a.dt == SQ_BF16, a.T, a.D, a.ldx, a.wr, a.rdt == SQ_BF16, a.E, a.top_k,
                                        a.renorm != 0, a.ids, a.wts, a.ids_in, a.wts_in, a.w13, a.s13, a.z13, a.w2,
                                        a.s2, a.z2, a.F, a.group, a.y, a.ydt == SQ_BF16, a.ldy, a.workspace,
                                        static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int64_t sq_w4_row_bytes(int64_t K) { return K < 0 ? -1 : (K + 127) / 128 * 64; }

sq_status sq_fold_quant_weights_w4(const void* W, sq_dtype dt, int64_t K, int64_t N, int64_t ldw, const float* s,
                                   const float* gamma, const float* beta, int group, uint8_t* Wq, uint16_t* scales,
                                   uint8_t* zeros, float* gamma_f, float* beta_f, void* stream) {
  if (K < 0 || N < 0) return SQ_ERR_INVALID_ARG;
  sq_status st = check_group(group);
  if (st != SQ_OK) return st;
  st = check_rows(W, dt, K, N, ldw);
  if (st != SQ_OK) return st;
  if (K == 0 || N == 0) return SQ_OK;
  st = check_packed(Wq, scales);
  if (st != SQ_OK) return st;
  if (!aligned(s, 4) || !aligned(gamma, 4) || !aligned(beta, 4) || !aligned(gamma_f, 4) || !aligned(beta_f, 4))
    return SQ_ERR_INVALID_ARG;
  if (K % 16 != 0) return SQ_ERR_ALIGNMENT;
  if (K > SQ_MAX_K || N > (int64_t)INT_MAX) return SQ_ERR_UNSUPPORTED;
  return cuda_status(sqh::launch_w4_fold(W, dt == SQ_BF16, K, N, ldw, s, gamma, beta, group, Wq, scales, zeros,
                                         gamma_f, beta_f, static_cast<cudaStream_t>(stream)));
}

sq_status sq_w4_dequant(const uint8_t* Wq, const uint16_t* scales, const uint8_t* zeros, int64_t K, int64_t N,
                        int group, void* y, sq_dtype ydt, int64_t ldy, void* stream) {
  if (K < 0 || N < 0) return SQ_ERR_INVALID_ARG;
  sq_status st = check_group(group);
  if (st != SQ_OK) return st;
  st = check_rows(y, ydt, N, K, ldy);
  if (st != SQ_OK) return st;
  if (K == 0 || N == 0) return SQ_OK;
  st = check_packed(Wq, scales);
  if (st != SQ_OK) return st;
  if (K % 16 != 0) return SQ_ERR_ALIGNMENT;
  if (K > SQ_MAX_K || N > (int64_t)INT_MAX) return SQ_ERR_UNSUPPORTED;
  return cuda_status(sqh::launch_w4_dequant(Wq, scales, zeros, K, N, group, y, ydt == SQ_BF16, ldy,
                                            static_cast<cudaStream_t>(stream)));
}

sq_status sq_w4_gemm(const void* x, sq_dtype dt, int64_t M, int64_t K, int64_t ldx, const uint8_t* Wq,
                     const uint16_t* scales, const uint8_t* zeros, int64_t N, int group, void* y, sq_dtype ydt,
                     int64_t ldy, void* stream) {
  if (M < 0 || N < 0 || K <= 0) return SQ_ERR_INVALID_ARG;
  sq_status st = check_group(group);
  if (st != SQ_OK) return st;
  st = check_rows(x, dt, M, K, ldx);
  if (st != SQ_OK) return st;
  st = check_out(y, ydt, N, ldy);
  if (st != SQ_OK) return st;
  if (M == 0 || N == 0) return SQ_OK;
  if (y == nullptr) return SQ_ERR_INVALID_ARG;
  st = check_packed(Wq, scales);
  if (st != SQ_OK) return st;
  if (K % 16 != 0 || !aligned(y, elt_size(ydt))) return SQ_ERR_ALIGNMENT;
  if (K > SQ_MAX_K || N > (int64_t)INT_MAX || M > SQ_W4_MAX_M) return SQ_ERR_UNSUPPORTED;
  if ((K + group - 1) / group * N > (int64_t)UINT_MAX) return SQ_ERR_UNSUPPORTED;  // 32-bit offsets of scales
  return cuda_status(sqh::launch_w4_gemm(x, dt == SQ_BF16, M, K, ldx, Wq, scales, zeros, N, group, y, ydt == SQ_BF16,
                                         ldy, static_cast<cudaStream_t>(stream)));
}

size_t sq_moe_w4_workspace_size(int64_t T, int64_t D, int64_t F, int64_t E, int top_k) {
  if (!moe_sizes_ok(T, D, F, E, top_k) || !moe_sizes_supported(T, D, F, E, top_k)) return (size_t)-1;
  return sqh::moe_workspace_size(T, D, F, E, top_k);
}

sq_status sq_moe_w4(const void* x, sq_dtype dt, int64_t T, int64_t D, int64_t ldx, const void* Wr, sq_dtype rdt,
                    int64_t E, int top_k, int renorm, int32_t* ids, float* weights, const uint8_t* W13,
                    const uint16_t* s13, const uint8_t* z13, const uint8_t* W2, const uint16_t* s2, const uint8_t* z2,
                    int64_t F, int group, void* y, sq_dtype ydt, int64_t ldy, void* workspace, size_t ws_bytes,
                    void* stream) {
  MoeArgs a{x, dt, T, D, ldx, Wr, rdt, E, top_k, renorm, ids, weights, nullptr, nullptr, W13, s13, z13,
            W2, s2, z2, F, group, y, ydt, ldy, workspace, ws_bytes};
  return run_moe(a, false, stream);
}

sq_status sq_moe_w4_routed(const void* x, sq_dtype dt, int64_t T, int64_t D, int64_t ldx, const int32_t* ids,
                           const float* weights, int64_t E, int top_k, const uint8_t* W13, const uint16_t* s13,
                           const uint8_t* z13, const uint8_t* W2, const uint16_t* s2, const uint8_t* z2, int64_t F,
                           int group, void* y, sq_dtype ydt, int64_t ldy, void* workspace, size_t ws_bytes,
                           void* stream) {
  MoeArgs a{x, dt, T, D, ldx, nullptr, SQ_BF16, E, top_k, 0, nullptr, nullptr, ids, weights, W13, s13, z13,
            W2, s2, z2, F, group, y, ydt, ldy, workspace, ws_bytes};
  return run_moe(a, true, stream);
}

}  // extern "C"

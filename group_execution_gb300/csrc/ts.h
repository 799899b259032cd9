// Training-step operators: what the C ABI (ts_api.cpp) hands to the kernel
// files.  Every matrix is row major with a row pitch in elements; nothing
// here is checked again below the ABI.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

// The handle behind ts_create.  The workspace holds what one call leaves for
// its own later kernels; calls of one handle are ordered by the caller.
struct ts_ops {
  int device = 0;
  int nsm = 0;
  uint8_t* ws = nullptr;
  int64_t ws_bytes = 0;
  int32_t* err = nullptr;   // latched by a bounded wait that expired
  int64_t wait_limit_ns = 2000000000LL;
  int inject = 0;           // failure injection for tests: no copies are issued
};

namespace fg {

struct TsMat {
  const void* p = nullptr;
  int bf16 = 0;
  int64_t ld = 0;
  int elem() const { return bf16 ? 2 : 4; }
};
struct TsOut {
  void* p = nullptr;
  int bf16 = 0;
  int64_t ld = 0;
  int elem() const { return bf16 ? 2 : 4; }
};

// Whether every row starts on 16 bytes (the pitch of a single row counts too).
inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
template <class M>
inline bool rows_aligned(const M& m) {
  return aligned16(m.p) && m.ld * m.elem() % 16 == 0;
}

// An 8-bit checkpoint of rows x cols values: int8 values, `pitch` a row (the
// columns rounded up to 128), then pitch / 32 scale bytes a row.
constexpr int kCkptBlock = 32;
inline int64_t ckpt_pitch(int64_t cols) { return (cols + 127) / 128 * 128; }
struct TsCkpt {
  int8_t* q = nullptr;
  uint8_t* scale = nullptr;
  int64_t pitch = 0;
};
inline TsCkpt ckpt_view(void* buf, int64_t rows, int64_t cols) {
  TsCkpt c;
  c.pitch = ckpt_pitch(cols);
  c.q = static_cast<int8_t*>(buf);
  c.scale = buf ? static_cast<uint8_t*>(buf) + rows * c.pitch : nullptr;
  return c;
}

struct NormArgs {
  TsMat x, dy;
  TsOut y, dx;
  TsCkpt ckpt;
  int64_t rows = 0;
  int cols = 0;
  const float* gamma = nullptr;
  const float* beta = nullptr;
  float eps = 0.f;
  float* mean = nullptr;
  float* rstd = nullptr;
  float* dgamma = nullptr;
  float* dbeta = nullptr;
  int accumulate = 0;
};
cudaError_t launch_layer_norm(const ts_ops& h, const NormArgs& a, cudaStream_t st);
cudaError_t launch_layer_norm_backward(const ts_ops& h, const NormArgs& a, cudaStream_t st);

cudaError_t launch_checkpoint_save(const ts_ops& h, const TsMat& x, int64_t rows, int cols, const TsCkpt& c,
                                   cudaStream_t st);
cudaError_t launch_checkpoint_load(const ts_ops& h, const TsCkpt& c, int64_t rows, int cols, const TsOut& y,
                                   cudaStream_t st);
// act: 0 relu, 1 sigmoid, 2 tanh
cudaError_t launch_activation_backward(const ts_ops& h, int act, const TsMat& dy, const TsCkpt& c, int64_t rows,
                                       int cols, const TsOut& dx, cudaStream_t st);

struct WgradArgs {
  TsCkpt x;
  int64_t rows = 0;
  int cols = 0, n = 0;
  const float* gamma = nullptr;
  const float* beta = nullptr;
  TsMat dy;
  float* dw = nullptr;
  int64_t lddw = 0;
  float* db = nullptr;
  int accumulate = 0;
};
cudaError_t launch_weight_grad(const ts_ops& h, const WgradArgs& a, cudaStream_t st);

// Sums of dy's columns over its rows into db, if not null (added to what it
// holds when accumulate is set), and by themselves into fresh, if not null.
cudaError_t launch_column_sums(const ts_ops& h, const TsMat& dy, int64_t rows, int cols, float* fresh, float* db,
                               int accumulate, cudaStream_t st);

struct LogprobArgs {
  TsMat logits;
  int64_t rows = 0;
  int vocab = 0;
  const int64_t* tokens = nullptr;
  float* logprob = nullptr;
  float* entropy = nullptr;
  float* lse = nullptr;
  int k = 0;
  float* top_logprob = nullptr;
  int32_t* top_id = nullptr;
  const float* g_logprob = nullptr;
  const float* g_entropy = nullptr;
  TsOut dlogits;
};
cudaError_t launch_token_logprobs(const ts_ops& h, const LogprobArgs& a, cudaStream_t st);
cudaError_t launch_token_logprobs_backward(const ts_ops& h, const LogprobArgs& a, cudaStream_t st);

}  // namespace fg

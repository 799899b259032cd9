// The C ABI of the training-step operators (include/groupexec.h): argument
// checks, the handle with its workspace and error word, and the launches.
#include <cuda_runtime.h>

#include <initializer_list>
#include <memory>
#include <new>
#include <string>

#include "groupexec.h"
#include "host.h"
#include "launch.h"
#include "ts.h"

using namespace fg;

#define TS_TRY(x) \
  if (fg_status s_ = (x)) return s_

namespace {

fg_status err(fg_status st, const std::string& msg) { return (fg_status)set_last_error(st, msg.c_str()); }
fg_status cuda_err(cudaError_t e, const char* what) {
  return err(FG_ECUDA, std::string(what) + ": " + cudaGetErrorString(e));
}
fg_status done(cudaError_t e, const char* what) { return e == cudaSuccess ? FG_OK : cuda_err(e, what); }

// Rows and columns index with 32 bits inside a kernel, some rows past the last
// one among them (offsets are 64-bit).
constexpr int64_t kMaxExtent = (int64_t(1) << 31) - 65536;

fg_status check_handle(const ts_ops* h) {
  if (!h) return err(FG_EINVAL, "null handle");
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return err(FG_ECUDA, "no CUDA device");
  }
  if (dev != h->device) return err(FG_EINVAL, "the handle was created on another device than the current one");
  return FG_OK;
}
fg_status check_extent(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1) return err(FG_ESHAPE, "rows must be at least 0 and columns at least 1");
  if (rows > kMaxExtent || cols > kMaxExtent) return err(FG_ESHAPE, "an extent is too large");
  return FG_OK;
}
fg_status check_matrix(const char* name, const void* p, int dtype, int64_t ld, int64_t rows, int64_t cols) {
  if (dtype != FG_F32 && dtype != FG_BF16) return err(FG_EINVAL, std::string(name) + ": unknown dtype");
  if (rows > 0 && !p) return err(FG_EINVAL, std::string(name) + ": null pointer");
  if (ld < cols) return err(FG_ESHAPE, std::string(name) + ": the row pitch is smaller than the columns");
  if (reinterpret_cast<uintptr_t>(p) % (dtype == FG_BF16 ? 2 : 4))
    return err(FG_EINVAL, std::string(name) + ": not aligned to its element");
  return FG_OK;
}
// A dense array of 4- or 8-byte elements; `needed` = null is an error.
fg_status check_array(const char* name, const void* p, bool needed, size_t elem = 4) {
  if (needed && !p) return err(FG_EINVAL, std::string(name) + ": null pointer");
  if (reinterpret_cast<uintptr_t>(p) % elem) return err(FG_EINVAL, std::string(name) + ": not aligned to its element");
  return FG_OK;
}
fg_status check_checkpoint(const void* p, bool needed) {
  if (needed && !p) return err(FG_EINVAL, "checkpoint: null pointer");
  if (reinterpret_cast<uintptr_t>(p) % 16) return err(FG_EINVAL, "checkpoint: must be 16-byte aligned");
  return FG_OK;
}
// An output that is an input too: rows have to lie alike, or one row's output
// is another row's input (one row's pitch says nothing).
fg_status check_in_place(const char* names, const void* out_p, int out_dtype, int64_t out_ld, const void* in_p,
                         int in_dtype, int64_t in_ld, int64_t rows) {
  if (out_p && out_p == in_p && (out_dtype != in_dtype || (rows > 1 && out_ld != in_ld)))
    return err(FG_EINVAL, std::string(names) + " needs the same dtype and row pitch");
  return FG_OK;
}
// An output that may not lie on any of these.
fg_status check_apart(const char* name, const void* out_p, std::initializer_list<const void*> others) {
  for (const void* p : others)
    if (out_p && out_p == p) return err(FG_EINVAL, std::string(name) + " starts where another argument does");
  return FG_OK;
}
fg_status check_vocab(int64_t vocab) {
  if (vocab < 1) return err(FG_ESHAPE, "the vocabulary must hold at least 1");
  if (vocab > kMaxExtent) return err(FG_ESHAPE, "an extent is too large");
  return FG_OK;
}
fg_status check_loss_extent(int64_t rows, int64_t cols, int64_t vocab) {
  TS_TRY(check_extent(rows, cols));
  TS_TRY(check_vocab(vocab));
  constexpr int64_t most = int64_t(1) << 20;
  if (rows > most || cols > most || vocab > most)
    return err(FG_EUNSUPPORTED, "more than 2^20 rows, columns or vocabulary");
  return FG_OK;
}
fg_status check_workspace(const ts_ops* h, int64_t needed) {
  if (needed > h->ws_bytes)
    return err(FG_EUNSUPPORTED, "the workspace holds " + std::to_string(h->ws_bytes) + " bytes, the call needs " +
                                    std::to_string(needed));
  return FG_OK;
}
TsMat mat(const void* p, int dtype, int64_t ld) { return TsMat{p, dtype == FG_BF16, ld}; }
TsOut out(void* p, int dtype, int64_t ld) { return TsOut{p, dtype == FG_BF16, ld}; }

}  // namespace

extern "C" {

fg_status ts_create(int64_t workspace_bytes, ts_ops** out_h) {
  if (!out_h) return err(FG_EINVAL, "null argument");
  *out_h = nullptr;
  if (workspace_bytes < 0) return err(FG_EINVAL, "negative workspace size");
  if (workspace_bytes == 0) workspace_bytes = int64_t(64) << 20;
  workspace_bytes = (workspace_bytes + 255) / 256 * 256;
  if (workspace_bytes < (int64_t(1) << 20)) return err(FG_EINVAL, "the workspace must hold at least 1 MiB");
  std::unique_ptr<ts_ops> h(new (std::nothrow) ts_ops());
  if (!h) return err(FG_ENOMEM, "out of host memory");
  int n = 0;
  if (cudaGetDeviceCount(&n) != cudaSuccess || n == 0) {
    cudaGetLastError();
    return err(FG_ECUDA, "no CUDA device");
  }
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->nsm, cudaDevAttrMultiProcessorCount, h->device);
  if (e != cudaSuccess) return cuda_err(e, "device query");
  e = cudaMalloc(&h->ws, (size_t)workspace_bytes + 256);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return err(FG_ENOMEM, std::string("cudaMalloc(workspace): ") + cudaGetErrorString(e));
  }
  h->ws_bytes = workspace_bytes;
  h->err = reinterpret_cast<int32_t*>(h->ws + workspace_bytes);
  e = cudaMemset(h->err, 0, 256);
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
  if (e != cudaSuccess) {
    cudaFree(h->ws);
    return cuda_err(e, "cudaMemset(error word)");
  }
  *out_h = h.release();
  return FG_OK;
}

fg_status ts_set_wait_limit(ts_ops* h, int64_t wait_limit_ns, int32_t flags) {
  if (!h) return err(FG_EINVAL, "null handle");
  if (wait_limit_ns <= 0) return err(FG_EINVAL, "wait_limit_ns must be positive");
  if (flags & ~FG_FLAG_INJECT_NO_LOADS) return err(FG_EINVAL, "unknown flag");
  h->wait_limit_ns = wait_limit_ns;
  h->inject = (flags & FG_FLAG_INJECT_NO_LOADS) != 0;
  return FG_OK;
}

fg_status ts_sync_status(ts_ops* h, void* stream) {
  TS_TRY(check_handle(h));
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_err(e, "cudaStreamSynchronize");
  int32_t flag = 0;
  e = cudaMemcpy(&flag, h->err, sizeof(flag), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_err(e, "reading the device error word");
  if (flag == 0) return FG_OK;
  e = cudaMemset(h->err, 0, sizeof(int32_t));
  if (e != cudaSuccess) return cuda_err(e, "clearing the device error word");
  if (flag == DEVERR_TIMEOUT)
    return err(FG_ETIMEOUT, "a device-side wait of ts_weight_grad or ts_linear_cross_entropy expired");
  return err(FG_EDEVICE, "device error word " + std::to_string(flag));
}

void ts_destroy(ts_ops* h) {
  if (!h) return;
  if (h->ws) cudaFree(h->ws);
  delete h;
}

fg_status ts_layer_norm(ts_ops* h, const void* x, fg_dtype x_dtype, int64_t ldx, int64_t rows, int64_t cols,
                        const float* gamma, const float* beta, float eps, void* y, fg_dtype y_dtype, int64_t ldy,
                        float* mean, float* rstd, void* checkpoint, void* stream) {
  TS_TRY(check_handle(h));
  TS_TRY(check_extent(rows, cols));
  TS_TRY(check_matrix("x", x, x_dtype, ldx, rows, cols));
  TS_TRY(check_matrix("y", y, y_dtype, ldy, rows, cols));
  TS_TRY(check_array("gamma", gamma, false));
  TS_TRY(check_array("beta", beta, false));
  TS_TRY(check_array("mean", mean, false));
  TS_TRY(check_array("rstd", rstd, false));
  TS_TRY(check_checkpoint(checkpoint, false));
  TS_TRY(check_in_place("y in place of x", y, y_dtype, ldy, x, x_dtype, ldx, rows));
  if (!(eps >= 0.f)) return err(FG_EINVAL, "eps must not be negative");
  if (rows == 0) return FG_OK;
  NormArgs a;
  a.x = mat(x, x_dtype, ldx);
  a.y = out(y, y_dtype, ldy);
  a.ckpt = ckpt_view(checkpoint, rows, cols);
  a.rows = rows;
  a.cols = (int)cols;
  a.gamma = gamma;
  a.beta = beta;
  a.eps = eps;
  a.mean = mean;
  a.rstd = rstd;
  return done(launch_layer_norm(*h, a, static_cast<cudaStream_t>(stream)), "ts_layer_norm launch");
}

fg_status ts_layer_norm_backward(ts_ops* h, const void* dy, fg_dtype dy_dtype, int64_t lddy, const void* x,
                                 fg_dtype x_dtype, int64_t ldx, const void* checkpoint, int64_t rows, int64_t cols,
                                 const float* gamma, const float* mean, const float* rstd, void* dx,
                                 fg_dtype dx_dtype, int64_t lddx, float* dgamma, float* dbeta, int32_t accumulate,
                                 void* stream) {
  TS_TRY(check_handle(h));
  TS_TRY(check_extent(rows, cols));
  if (x && checkpoint) return err(FG_EINVAL, "give x or its checkpoint, not both");
  TS_TRY(check_matrix("dy", dy, dy_dtype, lddy, rows, cols));
  TS_TRY(check_matrix("dx", dx, dx_dtype, lddx, rows, cols));
  TS_TRY(check_in_place("dx in place of dy", dx, dx_dtype, lddx, dy, dy_dtype, lddy, rows));
  if (!checkpoint && (x || rows > 0)) {   // (no rows: either buffer may be null)
    TS_TRY(check_matrix("x", x, x_dtype, ldx, rows, cols));
    if (x_dtype != dx_dtype) return err(FG_EINVAL, "dx has the dtype of x");
    TS_TRY(check_array("mean", mean, rows > 0));
  }
  TS_TRY(check_checkpoint(checkpoint, false));
  TS_TRY(check_array("rstd", rstd, rows > 0));
  TS_TRY(check_array("gamma", gamma, false));
  TS_TRY(check_array("dgamma", dgamma, false));
  TS_TRY(check_array("dbeta", dbeta, false));
  if (16 * cols > h->ws_bytes) return err(FG_EUNSUPPORTED, "the workspace is smaller than one row of partial sums");
  NormArgs a;
  a.dy = mat(dy, dy_dtype, lddy);
  if (!checkpoint) a.x = mat(x, x_dtype, ldx);
  a.dx = out(dx, dx_dtype, lddx);
  a.ckpt = ckpt_view(const_cast<void*>(checkpoint), rows, cols);
  a.rows = rows;
  a.cols = (int)cols;
  a.gamma = gamma;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.accumulate = accumulate != 0;
  return done(launch_layer_norm_backward(*h, a, static_cast<cudaStream_t>(stream)), "ts_layer_norm_backward launch");
}

fg_status ts_checkpoint_layout(int64_t rows, int64_t cols, int64_t* pitch, int64_t* scale_offset, int64_t* bytes) {
  TS_TRY(check_extent(rows, cols));
  const int64_t p = ckpt_pitch(cols);
  if (pitch) *pitch = p;
  if (scale_offset) *scale_offset = rows * p;
  if (bytes) *bytes = rows * p + rows * (p / kCkptBlock);
  return FG_OK;
}

fg_status ts_checkpoint_save(ts_ops* h, const void* x, fg_dtype x_dtype, int64_t ldx, int64_t rows, int64_t cols,
                             void* checkpoint, void* stream) {
  TS_TRY(check_handle(h));
  TS_TRY(check_extent(rows, cols));
  TS_TRY(check_matrix("x", x, x_dtype, ldx, rows, cols));
  TS_TRY(check_checkpoint(checkpoint, rows > 0));
  if (rows == 0) return FG_OK;
  return done(launch_checkpoint_save(*h, mat(x, x_dtype, ldx), rows, (int)cols, ckpt_view(checkpoint, rows, cols),
                                     static_cast<cudaStream_t>(stream)),
              "ts_checkpoint_save launch");
}

fg_status ts_checkpoint_load(ts_ops* h, const void* checkpoint, int64_t rows, int64_t cols, void* y, fg_dtype y_dtype,
                             int64_t ldy, void* stream) {
  TS_TRY(check_handle(h));
  TS_TRY(check_extent(rows, cols));
  TS_TRY(check_matrix("y", y, y_dtype, ldy, rows, cols));
  TS_TRY(check_checkpoint(checkpoint, rows > 0));
  if (rows == 0) return FG_OK;
  return done(launch_checkpoint_load(*h, ckpt_view(const_cast<void*>(checkpoint), rows, cols), rows, (int)cols,
                                     out(y, y_dtype, ldy), static_cast<cudaStream_t>(stream)),
              "ts_checkpoint_load launch");
}

fg_status ts_activation_backward(ts_ops* h, int32_t opcode, const void* dy, fg_dtype dy_dtype, int64_t lddy,
                                 const void* checkpoint, int64_t rows, int64_t cols, void* dx, fg_dtype dx_dtype,
                                 int64_t lddx, void* stream) {
  TS_TRY(check_handle(h));
  const int act = opcode == FG_OP_RELU ? 0 : opcode == FG_OP_SIGMOID ? 1 : opcode == FG_OP_TANH ? 2 : -1;
  if (act < 0) return err(FG_EINVAL, "opcode must be FG_OP_RELU, FG_OP_SIGMOID or FG_OP_TANH");
  TS_TRY(check_extent(rows, cols));
  TS_TRY(check_matrix("dy", dy, dy_dtype, lddy, rows, cols));
  TS_TRY(check_matrix("dx", dx, dx_dtype, lddx, rows, cols));
  TS_TRY(check_in_place("dx in place of dy", dx, dx_dtype, lddx, dy, dy_dtype, lddy, rows));
  TS_TRY(check_checkpoint(checkpoint, rows > 0));
  if (rows == 0) return FG_OK;
  return done(launch_activation_backward(*h, act, mat(dy, dy_dtype, lddy),
                                         ckpt_view(const_cast<void*>(checkpoint), rows, cols), rows, (int)cols,
                                         out(dx, dx_dtype, lddx), static_cast<cudaStream_t>(stream)),
              "ts_activation_backward launch");
}

fg_status ts_weight_grad(ts_ops* h, const void* checkpoint, int64_t rows, int64_t cols, const float* gamma,
                         const float* beta, const void* dy, fg_dtype dy_dtype, int64_t lddy, int64_t n, float* dw,
                         int64_t lddw, float* db, int32_t accumulate, void* stream) {
  TS_TRY(check_handle(h));
  TS_TRY(check_extent(rows, cols));
  TS_TRY(check_extent(rows, n));
  if (dy_dtype != FG_BF16) return err(FG_EINVAL, "dy must be bf16 (the tensor cores' operand)");
  TS_TRY(check_matrix("dy", dy, dy_dtype, lddy, rows, n));
  TS_TRY(check_matrix("dw", dw, FG_F32, lddw, cols, n));
  TS_TRY(check_checkpoint(checkpoint, rows > 0));
  TS_TRY(check_array("gamma", gamma, false));
  TS_TRY(check_array("beta", beta, false));
  TS_TRY(check_array("db", db, false));
  if (16 * n > h->ws_bytes) return err(FG_EUNSUPPORTED, "the workspace is smaller than one row of partial sums");
  if (cols > (int64_t(1) << 20) || n > (int64_t(1) << 20))
    return err(FG_EUNSUPPORTED, "weights of more than 2^20 rows or columns");
  WgradArgs a;
  a.x = ckpt_view(const_cast<void*>(checkpoint), rows, cols);
  a.rows = rows;
  a.cols = (int)cols;
  a.n = (int)n;
  a.gamma = gamma;
  a.beta = beta;
  a.dy = mat(dy, dy_dtype, lddy);
  a.dw = dw;
  a.lddw = lddw;
  a.db = db;
  a.accumulate = accumulate != 0;
  return done(launch_weight_grad(*h, a, static_cast<cudaStream_t>(stream)), "ts_weight_grad launch");
}

fg_status ts_token_logprobs(ts_ops* h, const void* logits, fg_dtype dtype, int64_t ld, int64_t rows, int64_t vocab,
                            const int64_t* tokens, float* logprob, float* entropy, float* lse, int32_t k,
                            float* top_logprob, int32_t* top_id, void* stream) {
  TS_TRY(check_handle(h));
  TS_TRY(check_extent(rows, vocab));
  TS_TRY(check_matrix("logits", logits, dtype, ld, rows, vocab));
  TS_TRY(check_array("tokens", tokens, rows > 0 && logprob, 8));
  TS_TRY(check_array("logprob", logprob, false));
  TS_TRY(check_array("entropy", entropy, false));
  TS_TRY(check_array("lse", lse, false));
  if (k < 0 || k > 32 || k > vocab) return err(FG_EINVAL, "k must be 0 to 32 and at most the vocabulary");
  TS_TRY(check_array("top_logprob", top_logprob, rows > 0 && k > 0));
  TS_TRY(check_array("top_id", top_id, rows > 0 && k > 0));
  if (rows == 0) return FG_OK;
  LogprobArgs a;
  a.logits = mat(logits, dtype, ld);
  a.rows = rows;
  a.vocab = (int)vocab;
  a.tokens = tokens;
  a.logprob = logprob;
  a.entropy = entropy;
  a.lse = lse;
  a.k = k;
  a.top_logprob = top_logprob;
  a.top_id = top_id;
  return done(launch_token_logprobs(*h, a, static_cast<cudaStream_t>(stream)), "ts_token_logprobs launch");
}

fg_status ts_token_logprobs_backward(ts_ops* h, const void* logits, fg_dtype dtype, int64_t ld, int64_t rows,
                                     int64_t vocab, const int64_t* tokens, const float* lse, const float* entropy,
                                     const float* g_logprob, const float* g_entropy, void* dlogits, fg_dtype d_dtype,
                                     int64_t ldd, void* stream) {
  TS_TRY(check_handle(h));
  TS_TRY(check_extent(rows, vocab));
  TS_TRY(check_matrix("logits", logits, dtype, ld, rows, vocab));
  TS_TRY(check_matrix("dlogits", dlogits, d_dtype, ldd, rows, vocab));
  TS_TRY(check_array("tokens", tokens, rows > 0, 8));
  TS_TRY(check_array("lse", lse, rows > 0));
  TS_TRY(check_array("g_logprob", g_logprob, rows > 0));
  TS_TRY(check_array("g_entropy", g_entropy, false));
  TS_TRY(check_array("entropy", entropy, rows > 0 && g_entropy));
  TS_TRY(check_in_place("dlogits in place of logits", dlogits, d_dtype, ldd, logits, dtype, ld, rows));
  if (rows == 0) return FG_OK;
  LogprobArgs a;
  a.logits = mat(logits, dtype, ld);
  a.rows = rows;
  a.vocab = (int)vocab;
  a.tokens = tokens;
  a.lse = const_cast<float*>(lse);
  a.entropy = const_cast<float*>(entropy);
  a.g_logprob = g_logprob;
  a.g_entropy = g_entropy;
  a.dlogits = out(dlogits, d_dtype, ldd);
  return done(launch_token_logprobs_backward(*h, a, static_cast<cudaStream_t>(stream)),
              "ts_token_logprobs_backward launch");
}

fg_status ts_embedding(ts_ops* h, const int64_t* ids, int64_t rows, const void* table, fg_dtype table_dtype,
                       int64_t ld_table, int64_t vocab, int64_t cols, float scale, void* y, fg_dtype y_dtype,
                       int64_t ldy, void* stream) {
  TS_TRY(check_handle(h));
  TS_TRY(check_extent(rows, cols));
  TS_TRY(check_vocab(vocab));
  TS_TRY(check_array("ids", ids, rows > 0, 8));
  TS_TRY(check_matrix("table", table, table_dtype, ld_table, rows > 0 ? vocab : 0, cols));
  TS_TRY(check_matrix("y", y, y_dtype, ldy, rows, cols));
  if (rows == 0) return FG_OK;
  TS_TRY(check_apart("y", y, {ids, table}));
  EmbedArgs a;
  a.ids = ids;
  a.rows = rows;
  a.vocab = vocab;
  a.cols = (int)cols;
  a.table = mat(table, table_dtype, ld_table);
  a.y = out(y, y_dtype, ldy);
  a.scale = scale;
  return done(launch_embedding(*h, a, static_cast<cudaStream_t>(stream)), "ts_embedding launch");
}

fg_status ts_embedding_backward(ts_ops* h, const int64_t* ids, const void* dy, fg_dtype dy_dtype, int64_t lddy,
                                int64_t rows, int64_t vocab, int64_t cols, float scale, void* dtable,
                                fg_dtype d_dtype, int64_t ldd, int32_t accumulate, void* stream) {
  TS_TRY(check_handle(h));
  TS_TRY(check_extent(rows, cols));
  TS_TRY(check_vocab(vocab));
  TS_TRY(check_array("ids", ids, rows > 0, 8));
  TS_TRY(check_matrix("dy", dy, dy_dtype, lddy, rows, cols));
  TS_TRY(check_matrix("dtable", dtable, d_dtype, ldd, vocab, cols));
  if (rows > 0) TS_TRY(check_apart("dtable", dtable, {ids, dy}));
  TS_TRY(check_workspace(h, embedding_backward_workspace(rows, vocab)));
  EmbedArgs a;
  a.ids = ids;
  a.rows = rows;
  a.vocab = vocab;
  a.cols = (int)cols;
  a.dy = mat(dy, dy_dtype, lddy);
  a.d = out(dtable, d_dtype, ldd);
  a.scale = scale;
  a.accumulate = accumulate != 0;
  return done(launch_embedding_backward(*h, a, static_cast<cudaStream_t>(stream)), "ts_embedding_backward launch");
}

fg_status ts_linear_cross_entropy_workspace(int64_t rows, int64_t cols, int64_t vocab, int64_t* least, int64_t* most) {
  TS_TRY(check_loss_extent(rows, cols, vocab));
  auto larger = [&](bool whole) {
    const int64_t f = vocab_loss_workspace(rows, cols, vocab, true, true, false, whole),
                  b = vocab_loss_workspace(rows, cols, vocab, true, true, true, whole);
    return f > b ? f : b;
  };
  if (least) *least = larger(false);
  if (most) *most = larger(true);
  return FG_OK;
}

fg_status ts_linear_cross_entropy(ts_ops* h, const void* x, int64_t ldx, const void* w, int64_t ldw, fg_dtype dtype,
                                  int64_t rows, int64_t cols, int64_t vocab, const int64_t* targets, float* loss,
                                  float* lse, void* stream) {
  TS_TRY(check_handle(h));
  TS_TRY(check_loss_extent(rows, cols, vocab));
  if (dtype != FG_BF16) return err(FG_EINVAL, "x and w must be bf16 (the tensor cores' operands)");
  TS_TRY(check_matrix("x", x, dtype, ldx, rows, cols));
  TS_TRY(check_matrix("w", w, dtype, ldw, rows > 0 ? vocab : 0, cols));
  TS_TRY(check_array("targets", targets, rows > 0 && loss, 8));
  TS_TRY(check_array("loss", loss, false));
  TS_TRY(check_array("lse", lse, false));
  if (rows == 0) return FG_OK;
  TS_TRY(check_apart("loss", loss, {x, w, targets, lse}));
  TS_TRY(check_apart("lse", lse, {x, w, targets}));
  VocabLossArgs a;
  a.x = mat(x, dtype, ldx);
  a.w = mat(w, dtype, ldw);
  a.rows = rows;
  a.cols = (int)cols;
  a.vocab = vocab;
  a.targets = targets;
  a.loss = loss;
  a.lse = lse;
  TS_TRY(check_workspace(h, vocab_loss_workspace(rows, cols, vocab, !rows_aligned(a.x), !rows_aligned(a.w), false,
                                                 false)));
  return done(launch_vocab_loss(*h, a, static_cast<cudaStream_t>(stream)), "ts_linear_cross_entropy launch");
}

fg_status ts_linear_cross_entropy_backward(ts_ops* h, const void* x, int64_t ldx, const void* w, int64_t ldw,
                                           fg_dtype dtype, int64_t rows, int64_t cols, int64_t vocab,
                                           const int64_t* targets, const float* lse, const float* g_loss,
                                           const float* g_lse, void* dx, fg_dtype dx_dtype, int64_t lddx, void* dw,
                                           fg_dtype dw_dtype, int64_t lddw, int32_t accumulate, void* stream) {
  TS_TRY(check_handle(h));
  TS_TRY(check_loss_extent(rows, cols, vocab));
  if (dtype != FG_BF16) return err(FG_EINVAL, "x and w must be bf16 (the tensor cores' operands)");
  TS_TRY(check_matrix("x", x, dtype, ldx, rows, cols));
  TS_TRY(check_matrix("w", w, dtype, ldw, rows > 0 ? vocab : 0, cols));
  TS_TRY(check_array("targets", targets, rows > 0, 8));
  TS_TRY(check_array("lse", lse, rows > 0));
  TS_TRY(check_array("g_loss", g_loss, rows > 0));
  TS_TRY(check_array("g_lse", g_lse, false));
  if (dx) TS_TRY(check_matrix("dx", dx, dx_dtype, lddx, rows, cols));
  if (dw) TS_TRY(check_matrix("dw", dw, dw_dtype, lddw, vocab, cols));
  if (rows > 0) {
    TS_TRY(check_in_place("dx in place of x", dx, dx_dtype, lddx, x, dtype, ldx, rows));
    TS_TRY(check_apart("dx", dx, {w, targets, lse, g_loss, g_lse, dw}));
    TS_TRY(check_apart("dw", dw, {x, w, targets, lse, g_loss, g_lse}));
  }
  VocabLossArgs a;
  a.x = mat(x, dtype, ldx);
  a.w = mat(w, dtype, ldw);
  a.rows = rows;
  a.cols = (int)cols;
  a.vocab = vocab;
  a.targets = targets;
  a.lse = const_cast<float*>(lse);
  a.g_loss = g_loss;
  a.g_lse = g_lse;
  a.dx = out(dx, dx_dtype, lddx);
  a.dw = out(dw, dw_dtype, lddw);
  a.accumulate = accumulate != 0;
  TS_TRY(check_workspace(h, vocab_loss_workspace(rows, cols, vocab, true, !rows_aligned(a.w), true, false)));
  return done(launch_vocab_loss_backward(*h, a, static_cast<cudaStream_t>(stream)),
              "ts_linear_cross_entropy_backward launch");
}

}  // extern "C"

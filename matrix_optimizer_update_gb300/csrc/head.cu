// head.cu - host side of the head's losses (include/dmuon.h, "The
// language-model head"): checks of arguments, workspace layout and the launch
// sequence of each call.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>

#include "head.h"
#include "internal.h"

using namespace dmuon;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 20;
constexpr int64_t kMaxVocab = int64_t(1) << 22;
constexpr int64_t kMaxDim = int64_t(1) << 16;
constexpr size_t kAlign = 1024;
// dz exists for one piece of the vocabulary at a time: as many entries as keep it within these bytes.
constexpr int64_t kPieceBytes = int64_t(512) << 20;
constexpr int64_t kPieceStep = 256;
constexpr int64_t kMaxPairs = 128;
constexpr int64_t kFewTokens = 128;
constexpr int64_t kMaxSlices = 2 * kMaxPairs;
constexpr int64_t kSliceBytes = kMaxSlices * 256 * 256 * 4;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

dmuon_status refuse(dmuon_status st, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return set_last_error(st, buf);
}

dmuon_status cuda_refuse(cudaError_t e, const char* what) {
  return refuse(DMUON_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

dmuon_status ok() { return set_last_error(DMUON_OK, ""); }

bool misaligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

}  // namespace

struct dmuon_head_s {
  int64_t max_tokens = 0, vocab = 0, dim = 0;
  int32_t max_top = 0;
  int64_t piece = 0;   // vocabulary entries per piece of the backward pass, a multiple of kPieceStep
  size_t off_status = 0, off_parts = 0, off_picked = 0, off_ids = 0, off_q = 0, off_count = 0, off_entropy = 0,
         off_dz = 0, off_acc = 0, bytes = 0;
  char* ws = nullptr;
  int device = -1, pairs = 0;

  head::Pipe pipe() const {
    unsigned* words = reinterpret_cast<unsigned*>(ws + off_status);
    return {words, words + 32, reinterpret_cast<float*>(words + 48), pairs};
  }
};

namespace {

// One side of a call: tensors with a row pitch.
dmuon_status check_matrix(const void* p, int64_t ld, int64_t dim, const char* name) {
  if (p == nullptr) return refuse(DMUON_ERR_INVALID_ARG, "%s is NULL", name);
  if (misaligned(p, 16)) return refuse(DMUON_ERR_INVALID_ARG, "%s does not start on 16 bytes", name);
  if (ld < dim || ld % 8 != 0)
    return refuse(DMUON_ERR_INVALID_ARG, "the row pitch of %s (%lld) must be a multiple of 8 and at least dim (%lld)",
                  name, (long long)ld, (long long)dim);
  if (ld > (int64_t(1) << 32)) return refuse(DMUON_ERR_INVALID_ARG, "the row pitch of %s is too large", name);
  return DMUON_OK;
}

dmuon_status check_call(dmuon_head_t H, const void* hidden, int64_t ld_hidden, const void* weight, int64_t ld_weight,
                        int64_t tokens) {
  if (H == nullptr) return refuse(DMUON_ERR_INVALID_ARG, "head is NULL");
  if (tokens < 0 || tokens > H->max_tokens)
    return refuse(DMUON_ERR_INVALID_ARG, "tokens (%lld) must be between 0 and max_tokens (%lld)", (long long)tokens,
                  (long long)H->max_tokens);
  if (H->ws == nullptr) return refuse(DMUON_ERR_NOT_BOUND, "head is not bound");
  int device = -1;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return cuda_refuse(e, "cudaGetDevice");
  if (device != H->device)
    return refuse(DMUON_ERR_INVALID_ARG, "head is bound on device %d, the current device is %d", H->device, device);
  if (tokens == 0) return DMUON_OK;
  dmuon_status st = check_matrix(hidden, ld_hidden, H->dim, "hidden");
  if (st == DMUON_OK) st = check_matrix(weight, ld_weight, H->dim, "weight");
  return st;
}

// The loss of a call: targets (cross entropy) or a teacher's lists (distillation).
struct Loss {
  const int64_t* targets = nullptr;
  const int64_t* top_ids = nullptr;
  const float* top_logits = nullptr;
  int32_t top = 0;
  float temperature = 1.f;
};

dmuon_status check_loss(dmuon_head_t H, const Loss& L, int64_t tokens, bool distill) {
  if (!distill) {
    if (tokens > 0 && (L.targets == nullptr || misaligned(L.targets, 8)))
      return refuse(DMUON_ERR_INVALID_ARG, "targets is NULL or not 8-byte aligned");
    return DMUON_OK;
  }
  if (L.top < 1 || L.top > H->max_top)
    return refuse(DMUON_ERR_INVALID_ARG, "top (%d) must be between 1 and max_top (%d)", L.top, H->max_top);
  if (!(L.temperature > 0.f) || !std::isfinite(L.temperature) || !std::isfinite(1.f / L.temperature))
    return refuse(DMUON_ERR_INVALID_ARG, "temperature must be positive and finite");
  if (tokens > 0 && (L.top_ids == nullptr || L.top_logits == nullptr || misaligned(L.top_ids, 8) ||
                     misaligned(L.top_logits, 4)))
    return refuse(DMUON_ERR_INVALID_ARG, "top_ids or top_logits is NULL or not aligned to its elements");
  return DMUON_OK;
}

// What the kernels are told of the loss; for distillation the lists are sorted into the workspace first.
dmuon_status prepare_wanted(dmuon_head_t H, const Loss& L, int64_t tokens, const head::DotParams& in,
                            head::Wanted* w, cudaStream_t s) {
  *w = head::Wanted{};
  w->vocab = static_cast<int32_t>(H->vocab);
  if (L.targets != nullptr) {
    w->targets = L.targets;
    w->top = 1;
    return DMUON_OK;
  }
  head::TeacherParams p{};
  p.ids = L.top_ids;
  p.logits = L.top_logits;
  p.tokens = tokens;
  p.top = L.top;
  p.vocab = static_cast<int32_t>(H->vocab);
  p.scale = 1.f / L.temperature;
  p.out_ids = reinterpret_cast<int32_t*>(H->ws + H->off_ids);
  p.out_q = reinterpret_cast<float*>(H->ws + H->off_q);
  p.out_count = reinterpret_cast<int32_t*>(H->ws + H->off_count);
  p.out_entropy = reinterpret_cast<float*>(H->ws + H->off_entropy);
  p.dot = in;
  p.picked = reinterpret_cast<float*>(H->ws + H->off_picked);
  cudaError_t e = head::launch_teacher(p, s);
  if (e != cudaSuccess) return cuda_refuse(e, "teacher kernel");
  w->ids = p.out_ids;
  w->q = p.out_q;
  w->count = p.out_count;
  w->top = L.top;
  return DMUON_OK;
}

head::LogitParams logit_params(dmuon_head_t H, const void* hidden, int64_t ld_hidden, const void* weight,
                               int64_t ld_weight, int64_t tokens, const Loss& L) {
  head::LogitParams p{};
  p.in = {static_cast<const head::bf16*>(hidden), static_cast<const head::bf16*>(weight), ld_hidden, ld_weight,
          static_cast<int32_t>(H->dim), 1.f / L.temperature};
  p.tokens = tokens;
  p.vocab = static_cast<int32_t>(H->vocab);
  p.width = p.vocab;
  p.picked = reinterpret_cast<float*>(H->ws + H->off_picked);
  return p;
}

dmuon_status forward(dmuon_head_t H, const void* hidden, int64_t ld_hidden, const void* weight, int64_t ld_weight,
                     const Loss& L, bool distill, int64_t tokens, float* loss, float* lse, void* stream) {
  dmuon_status st = check_call(H, hidden, ld_hidden, weight, ld_weight, tokens);
  if (st == DMUON_OK) st = check_loss(H, L, tokens, distill);
  if (st != DMUON_OK) return st;
  if (tokens == 0) return ok();
  if (loss == nullptr || lse == nullptr || misaligned(loss, 4) || misaligned(lse, 4))
    return refuse(DMUON_ERR_INVALID_ARG, "loss or lse is NULL or not 4-byte aligned");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  head::LogitParams p = logit_params(H, hidden, ld_hidden, weight, ld_weight, tokens, L);
  if ((st = prepare_wanted(H, L, tokens, p.in, &p.want, s)) != DMUON_OK) return st;
  p.parts = reinterpret_cast<head::Part*>(H->ws + H->off_parts);
  p.after_lists = distill;
  cudaError_t e = head::launch_logits(p, H->pipe(), s);
  if (e != cudaSuccess) return cuda_refuse(e, "logits kernel");
  head::RowParams r{};
  r.tokens = tokens;
  r.vocab = p.vocab;
  r.want = p.want;
  r.dot = p.in;
  r.parts = p.parts;
  r.groups = head::logit_groups(tokens, H->vocab, H->pairs);
  r.token_step = head::thin_tokens(tokens) ? r.groups : 1;
  r.group_step = head::thin_tokens(tokens) ? 1 : tokens;
  r.picked = p.picked;
  r.entropy = reinterpret_cast<const float*>(H->ws + H->off_entropy);
  r.temperature = L.temperature;
  r.loss = loss;
  r.lse = lse;
  if ((e = head::launch_rows(r, s)) != cudaSuccess) return cuda_refuse(e, "rows kernel");
  return ok();
}

dmuon_status backward(dmuon_head_t H, const void* hidden, int64_t ld_hidden, const void* weight, int64_t ld_weight,
                      const Loss& L, bool distill, int64_t tokens, const float* lse, const float* losses,
                      const float* grad_loss, void* dhidden, int64_t ld_dhidden, void* dweight, int64_t ld_dweight,
                      void* stream) {
  dmuon_status st = check_call(H, hidden, ld_hidden, weight, ld_weight, tokens);
  if (st == DMUON_OK) st = check_loss(H, L, tokens, distill);
  if (st == DMUON_OK && dhidden != nullptr && tokens > 0) st = check_matrix(dhidden, ld_dhidden, H->dim, "dhidden");
  if (st == DMUON_OK && dweight != nullptr) st = check_matrix(dweight, ld_dweight, H->dim, "dweight");
  if (st != DMUON_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (tokens == 0) {
    if (dweight != nullptr &&
        (e = cudaMemset2DAsync(dweight, ld_dweight * 2, 0, H->dim * 2, H->vocab, s)) != cudaSuccess)
      return cuda_refuse(e, "clearing dweight");
    return ok();
  }
  if (lse == nullptr || grad_loss == nullptr || misaligned(lse, 4) || misaligned(grad_loss, 4))
    return refuse(DMUON_ERR_INVALID_ARG, "lse or grad_loss is NULL or not 4-byte aligned");
  if (dhidden == nullptr && dweight == nullptr) return ok();
  head::LogitParams p = logit_params(H, hidden, ld_hidden, weight, ld_weight, tokens, L);
  if ((st = prepare_wanted(H, L, tokens, p.in, &p.want, s)) != DMUON_OK) return st;
  p.lse = lse;
  p.loss = losses;
  p.grad = grad_loss;
  p.dz = reinterpret_cast<head::bf16*>(H->ws + H->off_dz);
  p.ld_dz = H->piece;
  head::GradParams g{};
  g.hidden = p.in.hidden;
  g.weight = p.in.weight;
  g.ld_hidden = ld_hidden;
  g.ld_weight = ld_weight;
  g.tokens = tokens;
  g.vocab = p.vocab;
  g.dim = p.in.dim;
  g.dz = p.dz;
  g.ld_dz = p.ld_dz;
  g.gscale = L.temperature;
  g.slices = head::dh_slices(tokens, H->dim, std::min(H->piece, H->vocab), dweight != nullptr, H->pairs);
  const bool direct = H->vocab <= H->piece && g.slices.count == 1 && !head::thin_tokens(tokens);
  if (dhidden != nullptr && direct) {
    g.dhidden = static_cast<head::bf16*>(dhidden);
    g.ld_dhidden = ld_dhidden;
  } else if (dhidden != nullptr) {
    g.dh_acc = reinterpret_cast<float*>(H->ws + H->off_acc);
  }
  g.dweight = static_cast<head::bf16*>(dweight);
  g.ld_dweight = ld_dweight;
  for (int64_t v0 = 0; v0 < H->vocab; v0 += H->piece) {
    p.v0 = g.v0 = static_cast<int32_t>(v0);
    p.width = g.width = static_cast<int32_t>(std::min(H->piece, H->vocab - v0));
    g.first = v0 == 0;
    p.after_lists = distill && v0 == 0;  // a later piece's dz has to wait for the one before to be read
    if ((e = head::launch_dz(p, H->pipe(), s)) != cudaSuccess) return cuda_refuse(e, "dz kernel");
    if ((e = head::launch_grads(g, H->pipe(), s)) != cudaSuccess) return cuda_refuse(e, "gradient kernel");
  }
  if (g.dh_acc != nullptr &&
      (e = head::launch_round(g.dh_acc, g.slices.count, tokens, g.dim, g.gscale, H->pipe().gmax,
                              static_cast<head::bf16*>(dhidden), ld_dhidden, s)) != cudaSuccess)
    return cuda_refuse(e, "rounding kernel");
  return ok();
}

}  // namespace

extern "C" dmuon_status dmuon_head_create(int64_t max_tokens, int64_t vocab, int64_t dim, int32_t max_top,
                                          dmuon_head_t* out) {
  if (out == nullptr) return refuse(DMUON_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (max_tokens < 1 || max_tokens > kMaxTokens || vocab < 1 || vocab > kMaxVocab || dim < 1 || dim > kMaxDim)
    return refuse(DMUON_ERR_INVALID_ARG, "max_tokens must be 1..2^20, vocab 1..2^22 and dim 1..2^16");
  if (max_top < 0 || max_top > head::kMaxTop)
    return refuse(DMUON_ERR_INVALID_ARG, "max_top must be between 0 and %d", head::kMaxTop);
  dmuon_head_s* H = new (std::nothrow) dmuon_head_s;
  if (H == nullptr) return refuse(DMUON_ERR_INVALID_ARG, "out of host memory");
  H->max_tokens = max_tokens;
  H->vocab = vocab;
  H->dim = dim;
  H->max_top = max_top;
  const int64_t fit = std::max<int64_t>(kPieceStep, kPieceBytes / 2 / max_tokens / kPieceStep * kPieceStep);
  H->piece = std::min(fit, cdiv(vocab, kPieceStep) * kPieceStep);
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t o = at;
    at += cdiv(bytes, kAlign) * kAlign;
    return o;
  };
  H->off_status = take(256);
  // a call with few tokens has up to 8 groups for each 256 entries and for each pair of SMs
  H->off_parts = take(sizeof(head::Part) * std::max(cdiv(vocab, head::kGroup) * max_tokens,
                                                    (cdiv(vocab, 32) + 8 * kMaxPairs) *
                                                        std::min<int64_t>(max_tokens, kFewTokens)));
  H->off_picked = take(4 * max_tokens * std::max(1, max_top));
  H->off_ids = take(4 * max_tokens * max_top);
  H->off_q = take(4 * max_tokens * max_top);
  H->off_count = take(max_top > 0 ? 4 * max_tokens : 0);
  H->off_entropy = take(max_top > 0 ? 4 * max_tokens : 0);
  H->off_dz = take(2 * std::max(max_tokens, std::min<int64_t>(2 * max_tokens, 2 * head::kTwofold)) * H->piece);
  // dH's sums: one set where tokens are many; where K is cut into slices, up to 2 tiles of 256 x 256 per pair
  const int64_t row = 4 * head::acc_pitch(dim);
  H->off_acc = take(std::max(row * max_tokens, std::min(row * max_tokens * kMaxSlices, kSliceBytes)));
  H->bytes = at;
  *out = H;
  return ok();
}

extern "C" dmuon_status dmuon_head_workspace_bytes(dmuon_head_t H, size_t* bytes) {
  if (H == nullptr || bytes == nullptr) return refuse(DMUON_ERR_INVALID_ARG, "NULL argument");
  *bytes = H->bytes;
  return ok();
}

extern "C" dmuon_status dmuon_head_bind(dmuon_head_t H, void* d_workspace, size_t bytes, void* stream) {
  if (H == nullptr) return refuse(DMUON_ERR_INVALID_ARG, "head is NULL");
  H->ws = nullptr;
  if (d_workspace == nullptr || misaligned(d_workspace, kAlign) || bytes < H->bytes)
    return refuse(DMUON_ERR_WORKSPACE, "workspace is NULL, not 1024-byte aligned or smaller than %zu bytes", H->bytes);
  int device = -1, major = 0, minor = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return cuda_refuse(e, "cudaGetDevice");
  cudaPointerAttributes pa;
  if (cudaPointerGetAttributes(&pa, d_workspace) != cudaSuccess || pa.type != cudaMemoryTypeDevice ||
      pa.device != device) {
    cudaGetLastError();
    return refuse(DMUON_ERR_WORKSPACE, "workspace is not device memory of the current device %d", device);
  }
  if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device)) != cudaSuccess ||
      (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device)) != cudaSuccess ||
      (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device)) != cudaSuccess)
    return cuda_refuse(e, "cudaDeviceGetAttribute");
  if (major != 10 || minor != 3)
    return refuse(DMUON_ERR_UNSUPPORTED, "the head's losses need an sm_103 GPU (found sm_%d%d)", major, minor);
  if ((e = cudaMemsetAsync(static_cast<char*>(d_workspace) + H->off_status, 0, 256,
                           reinterpret_cast<cudaStream_t>(stream))) != cudaSuccess)
    return cuda_refuse(e, "clearing the status word");
  H->ws = static_cast<char*>(d_workspace);
  H->device = device;
  H->pairs = std::min<int>(sms / 2, kMaxPairs);
  return ok();
}

extern "C" dmuon_status dmuon_head_xent(dmuon_head_t H, const void* hidden, int64_t ld_hidden, const void* weight,
                                        int64_t ld_weight, const int64_t* targets, int64_t tokens, float* loss,
                                        float* lse, void* stream) {
  Loss L;
  L.targets = targets;
  return forward(H, hidden, ld_hidden, weight, ld_weight, L, false, tokens, loss, lse, stream);
}

extern "C" dmuon_status dmuon_head_xent_backward(dmuon_head_t H, const void* hidden, int64_t ld_hidden,
                                                 const void* weight, int64_t ld_weight, const int64_t* targets,
                                                 int64_t tokens, const float* lse, const float* grad_loss,
                                                 void* dhidden, int64_t ld_dhidden, void* dweight, int64_t ld_dweight,
                                                 void* stream) {
  Loss L;
  L.targets = targets;
  return backward(H, hidden, ld_hidden, weight, ld_weight, L, false, tokens, lse, nullptr, grad_loss, dhidden,
                  ld_dhidden, dweight, ld_dweight, stream);
}

extern "C" dmuon_status dmuon_head_xent_backward_loss(dmuon_head_t H, const void* hidden, int64_t ld_hidden,
                                                      const void* weight, int64_t ld_weight, const int64_t* targets,
                                                      int64_t tokens, const float* lse, const float* loss,
                                                      const float* grad_loss, void* dhidden, int64_t ld_dhidden,
                                                      void* dweight, int64_t ld_dweight, void* stream) {
  if (tokens > 0 && (loss == nullptr || misaligned(loss, 4)))
    return refuse(DMUON_ERR_INVALID_ARG, "loss is NULL or not 4-byte aligned");
  Loss L;
  L.targets = targets;
  return backward(H, hidden, ld_hidden, weight, ld_weight, L, false, tokens, lse, loss, grad_loss, dhidden, ld_dhidden,
                  dweight, ld_dweight, stream);
}

extern "C" dmuon_status dmuon_head_distill(dmuon_head_t H, const void* hidden, int64_t ld_hidden, const void* weight,
                                           int64_t ld_weight, const int64_t* top_ids, const float* top_logits,
                                           int32_t top, float temperature, int64_t tokens, float* loss, float* lse,
                                           void* stream) {
  Loss L;
  L.top_ids = top_ids;
  L.top_logits = top_logits;
  L.top = top;
  L.temperature = temperature;
  return forward(H, hidden, ld_hidden, weight, ld_weight, L, true, tokens, loss, lse, stream);
}

extern "C" dmuon_status dmuon_head_distill_backward(dmuon_head_t H, const void* hidden, int64_t ld_hidden,
                                                    const void* weight, int64_t ld_weight, const int64_t* top_ids,
                                                    const float* top_logits, int32_t top, float temperature,
                                                    int64_t tokens, const float* lse, const float* grad_loss,
                                                    void* dhidden, int64_t ld_dhidden, void* dweight,
                                                    int64_t ld_dweight, void* stream) {
  Loss L;
  L.top_ids = top_ids;
  L.top_logits = top_logits;
  L.top = top;
  L.temperature = temperature;
  return backward(H, hidden, ld_hidden, weight, ld_weight, L, true, tokens, lse, nullptr, grad_loss, dhidden,
                  ld_dhidden, dweight, ld_dweight, stream);
}

extern "C" dmuon_status dmuon_head_read_device_status(dmuon_head_t H, void* stream, uint32_t* bits) {
  if (H == nullptr || bits == nullptr) return refuse(DMUON_ERR_INVALID_ARG, "NULL argument");
  if (H->ws == nullptr) return refuse(DMUON_ERR_NOT_BOUND, "head is not bound");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint32_t word = 0;
  cudaError_t e = cudaMemcpyAsync(&word, H->ws + H->off_status, 4, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(H->ws + H->off_status, 0, 4, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_refuse(e, "reading the status word");
  *bits = word;
  return ok();
}

extern "C" void dmuon_head_destroy(dmuon_head_t H) { delete H; }

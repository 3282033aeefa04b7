// head.h - structures shared by the host side of the head's losses (head.cu) and their kernels.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dmuon.h"

namespace dmuon {
namespace head {

using bf16 = __nv_bfloat16;

// The forward pass reduces each token's logits over groups of 128 vocabulary entries (of up to 32 when the
// tokens are few: logit_groups).
constexpr int kGroup = 128;
constexpr int kMaxTop = 256;

// What the loss wants of a token's logits. Cross entropy: one entry, targets[t]. Distillation: a
// list per token, sorted by id and padded with ids >= vocab, and its probabilities.
struct Wanted {
  const int64_t* targets;  // cross entropy (then ids, q, count are nullptr)
  const int32_t* ids;      // [tokens][top], ascending
  const float* q;          // [tokens][top]
  const int32_t* count;    // [tokens]: entries in the list
  int32_t top;             // row pitch of ids, q and picked
  int32_t vocab;
};

// Logits formed in fp32 FMAs.
struct DotParams {
  const bf16* hidden;
  const bf16* weight;
  int64_t ld_hidden, ld_weight;
  int32_t dim;
  float scale;
};

// Tensor cores truncate what they accumulate, always towards zero: a logit z whose terms are spread evenly along the
// sum is off by about 1.0e-9 * dim * z (-6.6e-5 at z = 16, dim = 4096, where fp32 FMAs are off by 8e-7). Measured at
// 1024 to 65536 dims: 0.74e-9 to 1.05e-9 for normal and planted states, 1.25e-9 with one common state of 100, 1.8e-9
// where a sixteenth of the terms at the start makes the logit, 0.05e-9 to 0.25e-9 where it lies at the end or nothing
// comes after it (at 256 dims up to 2.2e-9 and down to 0.2e-9; more only where partial sums far above z cancel). Their
// scale puts 1.0e-9 back, the middle of that range: log sums are off by 4e-8 in place of 4.1e-7 (3912 dims, normal
// states), 3.7e-7 in place of 3.8e-6 (one logit of 12), and by up to 1.0e-9 * dim * z either way, where it was up to
// twice that one way, for logits made at one end of the sum (3.5e-6 of lse at 4096 dims). Below about 60 dims the
// scale rounds to 1 / temperature alone, and up to 180 by up to half a unit in the last place too much or too little.
constexpr double kTruncated = 1.0e-9;

// What remains is a few percent of it, in a loss still too much: that of a token predicted with near certainty is
// 1 - p of its target, and its relative error the absolute one of the target's logit. So the logits of wanted
// entries with at least this probability (at most 8 per token, for cross entropy the target) are formed apart, in
// fp32 FMAs, in both passes.
constexpr float kSure = 0.125f;

// Up to so many tokens, dz is held as the sum of two bf16, `tokens` rows apart: a gradient's row is then often
// one token's product with one dz, whose rounding nothing averages (2.1e-3 to 2.6e-3 in norm over 16 tokens, of
// which 1.7e-3 are the result's own rounding; with two parts 1.7e-3). The second parts' products fit beside the
// first's: dH^T's N is 128 at most, dW's K two stages. Both passes over 16 tokens x 128000 x 4096 take 676 us
// against 664 with one part, over 64 tokens 701 against 677; with more tokens the second parts would take time
// of the tensor cores.
constexpr int kTwofold = 64;

// One group's share of a token's softmax sum: sum of exp(z - peak), over the entries that are not wanted.
struct alignas(8) Part {
  float peak;
  float sum;
};

struct LogitParams {
  DotParams in;            // H, W and their pitches, dim, 1 / temperature
  int64_t tokens;
  int32_t vocab;
  Wanted want;
  // forward
  Part* parts;             // [groups][tokens]; few tokens: [tokens][groups]
  int32_t after_lists;     // the launch before this one on the stream is launch_teacher's
  float* picked;           // [tokens][want.top]: scaled logits of the wanted entries
  int32_t v0, width;       // entries v0 .. v0 + width - 1 (forward: all)
  // backward
  const float* lse;
  const float* grad;
  const float* loss;       // cross entropy: the losses, or nullptr: the targets' logits are formed again
  bf16* dz;                // [tokens][ld_dz]; up to kTwofold tokens: [2][tokens][ld_dz]
  int64_t ld_dz;
};

// What the tensor-core launches share: words in the workspace, and the SM pairs they run on.
struct Pipe {
  unsigned* status;
  unsigned* sched;         // two words, zero between launches
  float* gmax;             // the largest finite |grad| of a backward call; dz is relative to it
  int pairs;
};

// The cut of dH's K (a piece's entries) into slices of nk stages.
struct Slices {
  int32_t nk, count;
};

struct GradParams {
  const bf16* hidden;
  const bf16* weight;
  int64_t ld_hidden, ld_weight;
  int64_t tokens;
  int32_t vocab, dim;
  int32_t v0, width;
  const bf16* dz;
  int64_t ld_dz;
  float gscale;            // gradients = gscale * gmax * (products of dz)
  // dH: straight into dhidden (one piece, one slice), or into sums of fp32, or neither
  bf16* dhidden;
  int64_t ld_dhidden;
  float* dh_acc;           // [slices.count][tokens][acc_pitch(dim)]
  Slices slices;           // as the call's first (widest) piece has them
  int32_t first;           // this piece starts the sums
  bf16* dweight;           // or nullptr
  int64_t ld_dweight;
};

inline int64_t acc_pitch(int64_t dim) { return (dim + 7) / 8 * 8; }

struct RowParams {
  int64_t tokens;
  int32_t vocab;
  DotParams dot;           // cross entropy: the target's logit
  Wanted want;
  const Part* parts;       // of token t and group g at t * token_step + g * group_step
  int64_t token_step, group_step;
  int32_t groups;
  const float* picked;
  const float* entropy;    // [tokens]: sum_k q log q (distillation)
  float temperature;
  float* loss;
  float* lse;
};

struct TeacherParams {
  const int64_t* ids;
  const float* logits;
  int64_t tokens;
  int32_t top, vocab;
  float scale;
  int32_t* out_ids;
  float* out_q;
  int32_t* out_count;
  float* out_entropy;
  DotParams dot;
  float* picked;           // the logits of entries of at least kSure
};

// Tiles of a launch over so many vocabulary entries when the tokens are few.
struct Thin {
  int32_t height, tiles;
};
bool thin_tokens(int64_t tokens);
Thin thin_tiles(int64_t entries, int pairs);
int logit_groups(int64_t tokens, int64_t vocab, int pairs);

cudaError_t launch_logits(const LogitParams& p, const Pipe& pipe, cudaStream_t s);
cudaError_t launch_dz(const LogitParams& p, const Pipe& pipe, cudaStream_t s);
Slices dh_slices(int64_t tokens, int64_t dim, int64_t width, bool dweight, int pairs);
cudaError_t launch_grads(const GradParams& p, const Pipe& pipe, cudaStream_t s);
cudaError_t launch_teacher(const TeacherParams& p, cudaStream_t s);
cudaError_t launch_rows(const RowParams& p, cudaStream_t s);
// out = bf16(gscale * *gmax * the sum of the slices of acc)
cudaError_t launch_round(const float* acc, int slices, int64_t tokens, int32_t dim, float gscale, const float* gmax,
                         bf16* out, int64_t ld_out, cudaStream_t s);

}  // namespace head
}  // namespace dmuon

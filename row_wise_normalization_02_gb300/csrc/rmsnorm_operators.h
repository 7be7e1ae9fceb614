// Parameters and kernel lookup of the rotary positions and the token losses, shared
// by their translation units and the C ABI.
#pragma once

#include <stdint.h>

namespace rmsn {

// ---------------------------------------------------------------- rotary positions

constexpr int kRopeMaxAxes = 4;
constexpr int64_t kRopeMaxD = 8192;
// One [T, H, D] view of rows: element (t, h, d) at t * st + h * sh + d.
struct RopeView {
  const void* x;     // forward: input; backward: the forward's input
  const void* dy;    // backward with the norm: gradient of the output
  void* y;           // output, or gradient of the input
  const void* gamma; // null: rotation alone
  int64_t x_st, x_sh, dy_st, dy_sh, y_st, y_sh;
  int heads;
};
struct RopeParams {
  RopeView v[2];             // q, k (heads 0: absent)
  const int64_t* positions;  // [axes][pos_st]
  int64_t pos_st;
  const float* inv_freq;     // R / 2
  int axes;
  int order;                 // 0: frequencies in blocks per axis, 1: interleaved over the axes
  int sections[kRopeMaxAxes];
  int64_t T;
  int D, R;
  float sign;                // +1, or -1 to rotate back
  float eps, inv_d;
  int chunks[2];             // work items per token: chunks of heads_per_chunk heads (forward:
  int heads_per_chunk[2];    //   [0] covers the rows of q and k together)
  int block;                 // or, where rows are few, tokens per work item (one chunk)
  int split;                 // backward with the norm: the CTAs before this one take q, the
                             // others k (0: all take both)
  float* partial;            // backward with the norm: [gridDim.x][2 * ld_half], or null
  int ld_half;
};
using RopeKernel = void (*)(RopeParams);
struct RopeKey {
  int xd, wd;
  bool bwd;        // backward with the norm
  bool norm;
  bool adjacent;   // pairs (2i, 2i + 1); else (i, i + R / 2)
  int e;           // elements per vector, 0: the scalar kernel
  int g;           // lanes per row
  int l;           // units (pairs of vectors) per lane
  bool block;      // items of several tokens
};
RopeKernel get_rope_kernel_f32_f32(const RopeKey& k);
RopeKernel get_rope_kernel_bf16_bf16(const RopeKey& k);
RopeKernel get_rope_kernel_bf16_f32(const RopeKey& k);
constexpr int kRopeThreads = 256;
constexpr int kRopeFwdSteps = 4;   // steps of rows in a thread's ring
constexpr int kRopeBwdSteps = 3;
constexpr int kRopeMaxBlock = 8;   // tokens of one work item

// ---------------------------------------------------------------- token losses

struct LossParams {
  const void* logits;        // M rows of V, row stride ld elements
  int64_t ld;
  const int64_t* targets;    // negative: the row takes no part
  int64_t M;
  int V;
  float inv_tf, inv_tlo;     // 1 / temperature in two parts
  float c_hi, c_lo;          // times log2(e), in two parts: c_hi rounded down, c_lo > 0
  float* logp;
  float* lse;                // the row's log-sum-exp seen from its target: -logp
  float* dlogp;              // policy, preference: d loss / d logp of each row
  // policy
  const float* old_logp;
  const float* ref_logp;     // null: no KL term (preference: no reference)
  const float* advantages;
  const float* weights;      // null: 1
  float ratio_lo, ratio_hi, kl;
  float* token_loss;
  // preference: rows of sequence s are [cu[s], cu[s + 1]); s < pairs chosen, then rejected
  const int64_t* cu;
  int64_t pairs;
  float beta, smoothing;
  float* margins;
  float* loss;
  // gradient: the backward, and the policy loss in one pass with it
  const float* scale;        // backward: device scalar that multiplies dlogp, or null
  const float* dlogp_in;     // backward
  bool whole_rows;           // backward: a CTA takes whole rows (dlogits is logits)
  void* dlogits;
  int64_t ld_out;
  long long wait_limit;      // clock cycles before a wait for a cluster's peers gives up
  unsigned* status;          // device status word (kStatus* bits)
};
enum LossMode : int { kLossLogprob = 0, kLossPolicy = 1, kLossPolicyGrad = 2, kLossPreference = 3 };
using LossKernel = void (*)(LossParams);
// Kernel of a mode for clusters of `cluster` CTAs per row (with the gradient: for
// CTAs of `threads` threads with rings of `stages` batches).
LossKernel get_loss_rows_f32(int mode, int cluster, int threads, int stages);
LossKernel get_loss_rows_bf16(int mode, int cluster, int threads, int stages);
LossKernel get_loss_bwd_f32(int threads);
LossKernel get_loss_bwd_bf16(int threads);
LossKernel get_loss_sum();        // loss = sum of token_loss, one CTA
LossKernel get_loss_pairs();      // one CTA per pair: margins, dlogp
LossKernel get_loss_pairs_all();  // one CTA: margins, dlogp and loss
LossKernel get_loss_pairs_mean(); // loss = mean over the pairs, one CTA
constexpr int kLossThreads = 256;  // at most: eight warps
constexpr int kLossBatch = 4;     // 16-byte vectors a thread takes at a time
constexpr int kLossStages = 4;    // batches in a thread's ring (loss with gradient)
constexpr int loss_stages(int threads) { return threads == 32 ? 2 : kLossStages; }

}  // namespace rmsn

// Launchers of the scored router (score.hip) and its gradients (score_grad.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr int kScoreMaxExperts = 256;

// Sums of sigmoid scores under 2^-126, fp32's normal range, count as that: its reciprocal is
// finite and a score over it at most about 1.
constexpr float kLeastSum = 0x1p-126f;

struct ScoreShape {
  bool bf16;
  int T, d, E, k;
};

// Parts the d-long dot products are cut into (partial logits [parts][T][E]).
int score_parts(const ScoreShape& s);

struct ScoreArgs {
  ScoreShape sh;
  const void* x;
  const void* w;
  const float* b_router;   // or null
  const float* b_select;   // or null
  bool sigmoid;
  int groups, top_groups, group_top;
  bool renorm;
  float scale;
  int32_t* topk_idx;
  float* topk_w;
  float* logits;           // or null
  int32_t* load;           // the rest or null
  float* prob_mean;
  float* aux;
  float* z_loss;
  float* part;             // workspace [parts][T][E]
  double* psum;            // workspace [E][blocks], blocks <= 256
  int32_t* pload;          // workspace [E][blocks]
  double* pz;              // workspace [blocks]
  double* share;           // workspace [E]
  uint32_t* done;          // workspace [1]
};
hipError_t launch_score(const ScoreArgs& a, hipStream_t s);

// Slices of the token range that d_w_router is summed in.
int score_grad_slices(const ScoreShape& s);
// Bytes of the logit gradients in the workspace, and blocks that sum them for d_b.
size_t score_dl_bytes(const ScoreShape& s);
int score_grad_sum_blocks(int T);

struct ScoreGradArgs {
  ScoreShape sh;
  bool sigmoid, renorm;
  float scale;
  const void* x;
  const void* w;
  const int32_t* topk_idx;
  const float* logits;
  const int32_t* load;     // with d_aux
  const float* d_topk_w;   // or null, as the next two
  const float* d_aux;
  const float* d_z;
  void* d_x;               // or null, as the next three
  float* d_w;
  float* d_b;
  float* d_logits;
  float* dl;               // workspace of score_dl_bytes
  double* pb;              // workspace [E][score_grad_sum_blocks]
  float* pw;               // workspace [slices][E][d]
};
hipError_t launch_score_grad(const ScoreGradArgs& a, hipStream_t s);

}  // namespace moe

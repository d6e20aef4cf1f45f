// Launchers of the balance loss by sequence and its gradient (balance.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr int kBalanceMaxExperts = 256;

struct BalanceShape {
  int T, E, k, S;
  bool sigmoid;
};

int balance_chunks(const BalanceShape& s);   // runs of tokens that a block sums
int balance_blocks(int E);                   // blocks of experts a sequence is finished in

struct BalanceArgs {
  BalanceShape sh;
  const float* logits;       // [T][E]
  const int32_t* topk_idx;   // [T][k]
  const int32_t* offsets;    // [S + 1]
  const uint8_t* mask;       // [T] or null
  int32_t* load;             // [S][E]
  int32_t* valid;            // [S + 1]
  float* prob_mean;          // [S][E] or null, as the rest
  float* seq_loss;           // [S]
  float* loss;               // [1]
  int32_t* total_load;       // [E]
  float* pq;                 // workspace [chunks + S][E]
  int32_t* pload;            // workspace [chunks + S][E]
  int32_t* pvalid;           // workspace [chunks + S]
  double* part;              // workspace [S][balance_blocks(E)]
};
hipError_t launch_balance(const BalanceArgs& a, hipStream_t s);

struct BalanceGradArgs {
  BalanceShape sh;
  const float* logits;
  const int32_t* offsets;
  const uint8_t* mask;       // or null
  const int32_t* load;
  const int32_t* valid;
  const float* d_loss;       // [1] or null
  const float* d_seq_loss;   // [S] or null
  float* d_logits;           // [T][E]
};
hipError_t launch_balance_grad(const BalanceGradArgs& a, hipStream_t s);

}  // namespace moe

// Parameters and host launchers of the row operators: filtered sampling, top logits, distillation (internal to the
// library).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace specv {

// filtered sampling: a cluster of CTAs per row
struct FilterParams {
  const void* logits;          // [R, V]
  const float* uniforms;       // [R]
  const float* temperature;    // [R] or nullptr: temperature0 for every row, and so on
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  float temperature0, top_p0, min_p0;
  int top_k0;
  int R, V;
  int sms;                     // streaming multiprocessors of the device (0 if unknown)
  int32_t* tokens;             // [R]
  float* thr;                  // [R] or nullptr
  float* logp;                 // [R] or nullptr
  uint32_t* err;               // the workspace's error word
};
cudaError_t sample_filtered_launch(const FilterParams& p, int dtype, cudaStream_t stream);

// the K largest logits of each row and its log-sum-exp
struct TopParams {
  const void* logits;          // [R, V]
  float temperature;
  int R, V, K;
  int sms;                     // streaming multiprocessors of the device (0 if unknown)
  float* values;               // [R, K]
  int32_t* ids;                // [R, K]
  float* lse;                  // [R] or nullptr
};
cudaError_t top_logits_launch(const TopParams& p, int dtype, cudaStream_t stream);

// distillation from a teacher's top logits
struct DistillParams {
  const void* student;         // [N, V]
  const float* values;         // [N, K]
  const int32_t* ids;          // [N, K]
  const float* teacher_lse;    // [N] or nullptr: the record's probabilities are renormalised
  const float* grad_loss;      // [N] or nullptr: ones
  float temperature;
  float inv_t, inv_t_rest;     // 1 / T as a float32 and the rest
  float c;                     // log2(e) / T
  int N, V, K;
  int vec;                     // the gradient's rows lie as the student's do relative to 16 bytes
  int sms;                     // streaming multiprocessors of the device (0 if unknown)
  float* loss;                 // [N]
  float* stats;                // [N, 2]
  void* grad;                  // [N, V]
};
cudaError_t distill_forward_launch(const DistillParams& p, int dtype, cudaStream_t stream);
cudaError_t distill_backward_launch(const DistillParams& p, int dtype, cudaStream_t stream);
cudaError_t distill_loss_grad_launch(const DistillParams& p, int dtype, cudaStream_t stream);

#ifdef SPEC_DEBUG_BOUNDS
// what the kernels' index checks recorded (0: nothing), which is cleared
cudaError_t filtered_bounds(uint32_t* word);
cudaError_t distill_bounds(uint32_t* word);
#endif

}  // namespace specv

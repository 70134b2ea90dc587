// loss.cuh -- a cross entropy's sizes, between the C entry points and the kernels.
#pragma once

#include <cstddef>
#include <cstdint>

#include "internal.h"

namespace msim {

struct LossShape {
  int64_t V;
  int T, d, is_bf16;
  float scale;
};

size_t loss_workspace_bytes(const LossShape& s);
maxsim_status launch_loss(const LossShape& s, const maxsim_rows& x, const maxsim_rows& w, const int64_t* targets,
                          float* loss, float* lse, void* workspace, cudaStream_t stream);
size_t loss_bwd_workspace_bytes(const LossShape& s);
maxsim_status launch_loss_bwd(const LossShape& s, const float* dloss, const maxsim_rows& x, const maxsim_rows& w,
                              const int64_t* targets, const float* lse, const maxsim_rows* dx, const maxsim_rows* dw,
                              void* workspace, cudaStream_t stream);

}  // namespace msim

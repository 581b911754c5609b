// The optimizer step's table as the kernel reads it (gfx950).  Internal header.
#pragma once

#include <stdint.h>

#include "../../include/mbok.h"

namespace mbok {

// One tensor.  groups > 0: the scales of a layer ([kernels][rows][groups]), out
// the scales of its packed buffer; else out (may be null) is a flat copy.
struct AdamTensor {
  float* param;
  const void* grad;
  void *m, *v;
  float *m_scale, *v_scale;
  void* out;
  double decay;
  uint32_t salt;
  int32_t grad_dtype, state_dtype, out_dtype;
  int32_t groups, kernels, rows, pad;
};

// What one workgroup takes: len values from start of a tensor.
struct AdamPart {
  int64_t start;
  int32_t tensor, len;
};

// The step's numbers (the kernel's argument)
struct AdamStep {
  double lr, log_b1, log_b2, correct1, correct2;
  float b1, c1, b2, c2, eps, grad_scale;
  uint32_t key;
};

int adamw_part(int64_t values);
int adamw_layer_lds(int G, int part);
uint32_t adamw_salt(int tensor);

}  // namespace mbok

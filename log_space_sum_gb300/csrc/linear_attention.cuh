// What the linear attention's kernels share: a pass, and the powers of a decay.
#pragma once

#include "pc_device.cuh"
#include "pc_host.h"

namespace pc {

// One pass, in the terms of linear_attention.cu.
struct LaPass {
  const void *q, *k, *v;
  void* o;
  long long qs[3], ks[3], vs[3], os[3];  // strides of batch, token, head (elements)
  int dk, dv;
  const float* s_in;  // [B][H][dk][dv], or transposed; NULL: zeros
  float* s_out;       // [B][H][dk][dv]; NULL: not wanted
  int s_in_transposed, reverse;
  float c_intra, c_inter, c_up;  // factors of P, of Q S, and of the outer products
};

struct LaArgs {
  LaPass pass[3];
  int B, T, H;
  const float* log_decay;
  const int* lengths;
};

// l^n, with l^0 = 1 also for l = 0 (log_decay = -inf)
__device__ __forceinline__ float decay_pow(float g, int n) { return n == 0 ? 1.f : expf(g * static_cast<float>(n)); }

// Tokens of sequence b.
__device__ __forceinline__ int la_length(const LaArgs& a, int b) {
  return a.lengths ? min(max(a.lengths[b], 0), a.T) : a.T;
}

// A pass ends after the launch of its states, whether or not a segment read them: a later
// dependent launch (of another host thread's call, between this one's) waits for the pass alone.
__device__ __forceinline__ void la_end_after_states() {
  if ((blockIdx.x | blockIdx.y | blockIdx.z) == 0) grid_dependency_wait();
}

}  // namespace pc

// Launchers of linear attention and of its queries' and keys' norm and rotation.
// The argument blocks are the public ones of m3ssm.h, validated and with every
// `*_ld` filled in.
#pragma once
#include "layer_internal.hpp"

namespace m3 {

size_t attention_workspace(const m3_linear_attention_args& a);
bool attention_fits(const m3_linear_attention_args& a);
hipError_t launch_attention(const m3_linear_attention_args& a, hipStream_t s);
bool attention_step_fits(const m3_linear_attention_step_args& a);
hipError_t launch_attention_step(const m3_linear_attention_step_args& a, hipStream_t s);
bool attention_backward_fits(const m3_linear_attention_backward_args& a);
size_t attention_backward_workspace(const m3_linear_attention_backward_args& a);
hipError_t launch_attention_backward(const m3_linear_attention_backward_args& a, hipStream_t s);

hipError_t launch_rope(const m3_qk_norm_rope_args& a, hipStream_t s);
size_t rope_backward_workspace(const m3_qk_norm_rope_backward_args& a);
hipError_t launch_rope_backward(const m3_qk_norm_rope_backward_args& a, hipStream_t s);

// ---------------------------------------------------------------- the walk of linear attention
// Every output of linear attention and of its gradients is one walk over the tokens
// with other operands.  With p the position in the order of the walk,
//   out_p = s sum_{j <= p} l^(p-j) (a_p . b_j) c_j + w l^(p+e) a_p E,
//   E' = l^n E + u sum_j l^(n-e-j) b_j c_j^T   (E: the state in front of position 0).
// A chunk of 64 tokens is a triangle of scores and two products with the state.
struct WalkSide {
  const void* p;
  int64_t ld;  // elements from one token to the next
  int heads;   // of the tensor; head h of the walk takes head h / (H / heads)
  int cols;    // elements of a head
  int words;   // rows and heads are whole, aligned 16-byte words
};
struct WalkJob {
  WalkSide a, b, c;
  void* out;  // [Bt, L, H, c.cols]
  int out_f32, zero_tail;
  int out_words;  // 1: four columns are an aligned word, 2: 16 bytes are
  const float* init;  // [Bt, H, .] or null
  float* fin;         // likewise
  int64_t sn, sv;     // a state's element (n of b, v of c) is at n sn + v sv
  float* states;      // [Bt, H, segments, .] laid out likewise, or null: the state in front of each
  int rev, e;
  float s, u, w;
  int blocks;  // of one segment, item and head: tiles of c's columns
};
struct WalkPlan {
  WalkJob job[3];
  int jobs;
  int Bt, L, H, seg_len, segs;
  const float* log_decay;
  const int32_t* lengths;
};
// Launches the walk of all jobs, one block per (job, item, head, segment, column tile),
// or, with states_only, the segments' own states (all but each item's last) into the place
// of the next segment's in `states`.
// `kb`: blocks of 32 that a's and b's elements take, `nct`: 64 nct columns of c per block.
hipError_t launch_walk_bf16(const WalkPlan& p, int kb, int nct, bool states_only, hipStream_t s);
hipError_t launch_walk_f32(const WalkPlan& p, int kb, int nct, bool states_only, hipStream_t s);

}  // namespace m3

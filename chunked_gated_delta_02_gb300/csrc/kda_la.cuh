// Linear attention with one decay per head, chunked form: what the kernels and the host share.
#pragma once

#include "kda_common.cuh"

namespace kda {

constexpr int kLaChunk = 128;   // tokens per chunk: one 128-row tensor-core tile

// A run of chunks of one sequence that one CTA takes for one head.
struct LaItem {
  int seq;
  int t0, len;        // tokens [t0, t0 + len) of batch row b
  int b;
  int slot;           // index of its segment among those of sequences of more than one
  int seg, n_seg;     // segment of the sequence, number of them
  int part;           // while a CTA has it: kLaFromOther, kLaToOther
};
// The CTA before does the item's first chunks; the CTA after this, its last ones.
constexpr int kLaFromOther = 1, kLaToOther = 2;

struct LaProblem {
  const float *decay;            // log decay, [H] or per token (kLaTokenDecay)
  long long ds[3];               // strides of the per-token log decay: batch row, token, head
  const void *init;              // [N,H,V,K] or [N,H,K,V], fp32 or bf16, or null
  void *final_state;             // the same, or null
  const int32_t *cu;             // [N+1] or null
  __nv_bfloat16 *o;              // [B,T,H,V]
  // Segments (n_seg > 1): slot s of head h holds at seg_state + (s H + h) K V first the state that
  // the segment adds when started from zero, after the combine the start state of segment s + 1; the
  // slot of a sequence's last segment that of its first. seg_decay[s H + h] is the product of its decays.
  float *seg_state;
  float *seg_decay;
  // Varlen, by the schedule kernel: the work list, the segments formed ahead first; how many items, how
  // many of them are formed ahead, and how many sequences have such; the first slot of each sequence that
  // has more than one segment [N + 1]; those sequences.
  LaItem *items;
  int32_t *counts;
  int32_t *slot0;
  int32_t *multi;
  // Items that two CTAs share (fixed length): the state at the end of CTA c's part at hand + c K V, and for
  // each of its state warps whether it is there; how many CTAs have started. Null where none are shared.
  float *hand;
  int32_t *hand_there;           // [CTAs][8]
  int32_t *started;
  int32_t *flag;                 // per-call data-error flag (varlen) or null
  int *dev_status;
  float scale;
  int B, T, Hk, H, N;
  int seg_chunks, n_seg;         // chunks per segment; segments per sequence (fixed length)
  uint32_t flags;
};

struct LaMaps {
  CUtensorMap q, k, v, o;
};

}  // namespace kda

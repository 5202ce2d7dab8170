// Launch parameters of the operators beside kda_prefill: linear attention with one decay
// per head, the state pool's slot operations and the gated norm.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda.h"

namespace kda {

// Keeps `text` as the calling thread's kda_last_error() and returns s.
kda_status set_error(kda_status s, const char* text) noexcept;

constexpr int kLinChunk = 64;       // tokens per chunk
constexpr int kLinRows = 64;        // state rows (values) per workgroup of the chunked form
constexpr int kLinDecodeMaxT = 8;   // longest fixed-layout call of the token loop

struct LinParams {
  const void* q;
  const void* k;
  const void* v;
  const void* g;             // null: 0
  const float* log_decay;    // null: 0
  const void* state_in;      // null: zeros
  const int64_t* cu_seqlens; // null: fixed layout
  void* o;
  void* state_out;           // null: not written
  int64_t T, N;
  int32_t H, Hk, V;
  int64_t qs[3], ks[3], vs[3];  // strides in elements: batch, token, head
  float scale;
  double log2_scale;
  int32_t g_bf16, st_bf16;
  int32_t split;             // FP32 states of BF16 inputs: the decayed values in three parts
  const int32_t* in_idx;     // pool slots read and written (null: sequence n at n)
  const int32_t* out_idx;
  int64_t pool_slots, slot_pitch;
  // Segments: seg_len tokens each (a multiple of 64; serial form: at least T). Slot w of
  // the scan area belongs to segment p of sequence n: w = n * segs_per_seq + p (fixed
  // layout) or cu[n] / seg_len + n + p (varlen).
  int64_t seg_len;
  int64_t segs_per_seq;      // fixed layout
  int64_t slots;             // bound on w; the serial form has one per sequence
  int32_t segmented;
  int32_t longest_first;     // serial varlen form: workgroups by decreasing sequence length
  float* scan_s;             // FP32 [H][slots][V][K]
  float* scan_d;             // FP32 [H][slots]: the segment's total decay
  int32_t vblocks;           // workgroups (value blocks) of one head of a slot
};

// Workgroups of a chunk launch (see find_task).
inline int64_t linear_grid(const LinParams& p) { return (p.slots * p.H + 7) / 8 * 8 * p.vblocks; }

hipError_t launch_linear_chunks(const LinParams& p, int k_dim, bool io_bf16, int rows,
                                hipStream_t stream);
hipError_t launch_linear_states(const LinParams& p, int k_dim, bool io_bf16, hipStream_t stream);
hipError_t launch_linear_scan(const LinParams& p, int k_dim, hipStream_t stream);
// rows: state rows per workgroup (16, 32 or 64; 32 or 64 with K = 64)
hipError_t launch_linear_tokens(const LinParams& p, int k_dim, bool io_bf16, int rows,
                                hipStream_t stream);

constexpr int kCopyUnits = 4;                          // pieces of eight elements per thread
constexpr int kCopyGroup = 256 * kCopyUnits * 8;       // elements of a slot per workgroup

struct PoolCopy {
  const void* src;
  void* dst;
  int64_t src_slots, src_pitch, src_layer;  // elements
  int64_t dst_slots, dst_pitch, dst_layer;
  int64_t slot_elems, layers, pairs;
  const int32_t* src_idx;
  const int32_t* dst_idx;
  const int32_t* count;  // null, or the number of pairs (at most `pairs`) on the device
  int32_t src_bf16, dst_bf16;
};
hipError_t launch_pool_copy(const PoolCopy& p, hipStream_t stream);
// Writes new_idx, count, and the moves (src, dst, their number) into the workspace.
hipError_t launch_pool_plan(const int32_t* idx, int32_t* new_idx, int32_t* count, int64_t n,
                            int64_t slots, int32_t* move_src, int32_t* move_dst,
                            int32_t* moves, hipStream_t stream);

constexpr int kNormMax = 16384;  // longest row

// Threads of a row of D elements: part of a wave up to D = 512, a workgroup beyond.
inline int norm_threads(int64_t D) {
  if (D > 6144) return 512;
  int t = 8;
  while (t < 256 && 8 * t < D) t *= 2;
  return t;
}

struct NormParams {
  const void* x;
  const void* gate;
  const void* residual;
  const float* weight;
  const float* next_weight;
  void* out;
  void* next_out;
  int64_t M, G;
  int32_t D;
  int64_t xs[2], gs[2], rs[2];
  int32_t silu;
  float eps, scale;
};
hipError_t launch_gated_norm(const NormParams& p, bool io_bf16, hipStream_t stream);

}  // namespace kda

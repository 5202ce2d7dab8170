// Launch parameters of the short causal convolution and the selective state space scan.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda.h"

namespace kda {

// Where sequences keep their states: dense by sequence, or in slots of a pool.
struct StateSlots {
  const void* in;          // null: zeros
  void* out;               // null: not written
  const int32_t* in_idx;   // slots read and written (null: sequence n at n)
  const int32_t* out_idx;
  int64_t slots, pitch;    // slots that exist, elements between them
  int32_t bf16;
};

constexpr int kConvRows = 4;  // tokens that a thread of the convolution has in flight

struct ConvParams {
  const void* x;
  const float* weight;
  const float* bias;         // null: 0
  const int64_t* cu_seqlens; // null: fixed layout
  void* out;
  int64_t T, N, C;
  int64_t xs[2];             // strides in elements: batch, token
  // A thread takes eight channels of `run` tokens of one sequence. Slot w of the runs
  // belongs to run r of sequence n: w = n * runs_per_seq + r (fixed layout) or
  // cu[n] / run + n + r (varlen).
  int64_t run, runs_per_seq, slots;
  int32_t lanes;             // octets of channels of a workgroup: 64, 32 or 8
  int32_t silu;
  StateSlots state;
};
hipError_t launch_short_conv(const ConvParams& p, int width, bool io_bf16, hipStream_t stream);

constexpr int kScanTile = 32;      // tokens of a tile
constexpr int kScanChannels = 32;  // channels of a workgroup
constexpr int kScanTokensMaxT = 8; // longest fixed-layout call of the token form

struct ScanParams {
  const void* u;
  const void* delta;
  const void* z;             // null: no gate
  const void* B;
  const void* C;
  const float* A;
  const float* skip;         // null: 0
  const float* bias;         // null: 0
  const int64_t* cu_seqlens; // null: fixed layout
  void* out;
  int64_t T, N, D;
  int64_t per_group;         // channels that share one row of B and C
  int64_t us[2], ds[2], zs[2];  // strides in elements: batch, token
  int64_t bs[3], cs[3];         // batch, token, group
  int32_t softplus;
  StateSlots state;
  // Segments: seg_len tokens each (serial form: at least T). Slot w belongs to segment r of
  // sequence n: w = n * segs_per_seq + r (fixed layout) or cu[n] / seg_len + n + r (varlen).
  int64_t seg_len, segs_per_seq, slots;
  int64_t cblocks;           // workgroups (channel blocks) of a slot
  int32_t segmented;
  int32_t longest_first;     // serial varlen form: workgroups by decreasing sequence length
  float* ends;               // FP32 [slots][D][n]: a segment's end state
  float* sums;               // FP32 [slots][D]: the sum of its step sizes
  float* starts;             // FP32 [N][D][n]: the sequences' start states
};
// Both launches take states of n = 8, 16, 32 or 64 entries per channel.
hipError_t launch_scan_ends(const ScanParams& p, int n, bool io_bf16, hipStream_t stream);
hipError_t launch_scan_outputs(const ScanParams& p, int n, bool io_bf16, hipStream_t stream);
hipError_t launch_scan_tokens(const ScanParams& p, int n, bool io_bf16, hipStream_t stream);

// Workgroups of a chunk launch: a multiple of 16, see scan_task.
inline int64_t scan_grid(const ScanParams& p) { return (p.slots * p.cblocks + 15) / 16 * 16; }

}  // namespace kda

// Slots of a state pool: copies (with forks, restores from the other dtype and clears)
// and compaction.

#include "kda_device.h"
#include "kda_ops_internal.h"

namespace kda {

namespace {

// A workgroup copies kCopyGroup consecutive elements of one slot of one layer, all
// loads before the first store. Bound by its bytes: 48 slots of 24 heads in four layers from
// FP32 to BF16, 434 MB, 90 us (4.8 TB/s); 120 slots x 24 heads x two layers of FP32,
// 755 MB, 149 us (5.1 TB/s). Pairs are known on the device only, so a compaction launches a
// grid for the most moves there can be; a workgroup without one ends at once.
template <bool SRC_BF16, bool DST_BF16>
__global__ __launch_bounds__(256) void pool_copy_kernel(PoolCopy p, int64_t blocks) {
  const int64_t b = blockIdx.x;
  const int64_t row = b / blocks;
  const int64_t pair = row / p.layers;
  const int64_t layer = row - pair * p.layers;
  if (p.count && pair >= *p.count) return;
  const int64_t si = p.src_idx[pair], di = p.dst_idx[pair];
  if (di < 0 || di >= p.dst_slots) return;
  const bool held = si >= 0 && si < p.src_slots;
  const int64_t first = (b - row * blocks) * kCopyGroup + 8 * threadIdx.x;
  constexpr int kSrc = SRC_BF16 ? 2 : 4, kDst = DST_BF16 ? 2 : 4;
  const char* from = static_cast<const char*>(p.src) + (si * p.src_pitch + layer * p.src_layer) * kSrc;
  char* to = static_cast<char*>(p.dst) + (di * p.dst_pitch + layer * p.dst_layer) * kDst;
  if (SRC_BF16 == DST_BF16 && held && from == to) return;  // a slot onto itself
  u32x4 x[kCopyUnits][SRC_BF16 ? 1 : 2];
#pragma unroll
  for (int u = 0; u < kCopyUnits; ++u) {
    const int64_t e = first + u * 2048;
#pragma unroll
    for (int w = 0; w < (SRC_BF16 ? 1 : 2); ++w) {
      x[u][w] = u32x4{0u, 0u, 0u, 0u};
      if (held && e < p.slot_elems) x[u][w] = *reinterpret_cast<const u32x4*>(from + e * kSrc + 16 * w);
    }
  }
#pragma unroll
  for (int u = 0; u < kCopyUnits; ++u) {
    const int64_t e = first + u * 2048;
    if (e >= p.slot_elems) continue;
    u32x4* w = reinterpret_cast<u32x4*>(to + e * kDst);
    if constexpr (SRC_BF16 == DST_BF16) {
#pragma unroll
      for (int i = 0; i < (SRC_BF16 ? 1 : 2); ++i) w[i] = x[u][i];
    } else if constexpr (SRC_BF16) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        w[i] = u32x4{x[u][0][2 * i] << 16, x[u][0][2 * i] & 0xffff0000u, x[u][0][2 * i + 1] << 16,
                     x[u][0][2 * i + 1] & 0xffff0000u};
    } else {
      *reinterpret_cast<bf16x8*>(w) = pack8(__builtin_bit_cast(f32x4, x[u][0]),
                                            __builtin_bit_cast(f32x4, x[u][SRC_BF16 ? 0 : 1]));
    }
  }
}

constexpr int kWords = KDA_POOL_COMPACT_SLOTS / 32;

// One workgroup: a bitmap of the live slots and its running counts in LDS. rank(s) is the
// number of live slots below s; with L live ones in all, the free slot s < L is hole
// number s - rank(s), and the live slot s >= L is move number rank(s) - rank(L). Bound by
// the latency of its few passes: 2.8 us for 64 slots, 4.8 for 512.
__global__ __launch_bounds__(1024) void pool_plan_kernel(const int32_t* idx, int32_t* new_idx,
                                                         int32_t* count, int64_t n, int slots,
                                                         int32_t* move_src, int32_t* move_dst,
                                                         int32_t* moves) {
  __shared__ uint32_t bits[kWords];
  __shared__ int before[kWords];
  __shared__ int wave_sum[16];
  const int tid = threadIdx.x;
  const int words = (slots + 31) / 32;
  for (int w = tid; w < words; w += 1024) bits[w] = 0u;
  __syncthreads();
  for (int64_t i = tid; i < n; i += 1024) {
    const int s = idx[i];
    if (s >= 0 && s < slots) atomicOr(&bits[s >> 5], 1u << (s & 31));
  }
  __syncthreads();
  const int per = (words + 1023) / 1024;  // consecutive words of each thread
  int sum = 0;
  for (int w = tid * per; w < (tid + 1) * per && w < words; ++w) sum += __popc(bits[w]);
  int incl = sum;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const int y = __shfl_up(incl, s);
    if ((tid & 63) >= s) incl += y;
  }
  if ((tid & 63) == 63) wave_sum[tid >> 6] = incl;
  __syncthreads();
  int live = 0, base = 0;
  for (int w = 0; w < 16; ++w) {
    if (w < (tid >> 6)) base += wave_sum[w];
    live += wave_sum[w];
  }
  int run = base + incl - sum;
  for (int w = tid * per; w < (tid + 1) * per && w < words; ++w) {
    before[w] = run;
    run += __popc(bits[w]);
  }
  __syncthreads();
  auto rank = [&](int s) { return before[s >> 5] + __popc(bits[s >> 5] & ((1u << (s & 31)) - 1u)); };
  const int below = live < slots ? rank(live) : live;  // live slots that stay
  for (int s = tid; s < slots; s += 1024) {
    const bool in_use = (bits[s >> 5] >> (s & 31)) & 1u;
    if (s < live && !in_use) move_dst[s - rank(s)] = s;
    if (s >= live && in_use) move_src[rank(s) - below] = s;
  }
  if (tid == 0) {
    *count = live;
    *moves = live - below;
  }
  __syncthreads();
  for (int64_t i = tid; i < n; i += 1024) {
    const int s = idx[i];
    new_idx[i] = s >= live && s < slots ? move_dst[rank(s) - below] : s;
  }
}

}  // namespace

hipError_t launch_pool_copy(const PoolCopy& p, hipStream_t stream) {
  const int64_t blocks = (p.slot_elems + kCopyGroup - 1) / kCopyGroup;
  const int64_t wgs = blocks * p.layers * p.pairs;
  if (wgs <= 0) return hipSuccess;
  const dim3 grid(static_cast<unsigned>(wgs));
  if (p.src_bf16 && p.dst_bf16)
    hipLaunchKernelGGL((pool_copy_kernel<true, true>), grid, dim3(256), 0, stream, p, blocks);
  else if (p.src_bf16)
    hipLaunchKernelGGL((pool_copy_kernel<true, false>), grid, dim3(256), 0, stream, p, blocks);
  else if (p.dst_bf16)
    hipLaunchKernelGGL((pool_copy_kernel<false, true>), grid, dim3(256), 0, stream, p, blocks);
  else
    hipLaunchKernelGGL((pool_copy_kernel<false, false>), grid, dim3(256), 0, stream, p, blocks);
  return hipGetLastError();
}

hipError_t launch_pool_plan(const int32_t* idx, int32_t* new_idx, int32_t* count, int64_t n,
                            int64_t slots, int32_t* move_src, int32_t* move_dst, int32_t* moves,
                            hipStream_t stream) {
  hipLaunchKernelGGL(pool_plan_kernel, dim3(1), dim3(1024), 0, stream, idx, new_idx, count, n,
                     static_cast<int>(slots), move_src, move_dst, moves);
  return hipGetLastError();
}

}  // namespace kda

// The selective state space scan for a few tokens per sequence (fixed layout, T <=
// kScanTokensMaxT): each state is read once, takes the T steps in FP32 registers and is
// written once, so the launch is bound by the states' bytes. A channel is n / 4 lanes of four
// states each.

#include "kda_ssm_device.h"

namespace kda {

namespace {

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                           0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}

// Sum over the LANES lanes (2 to 16) of a channel, in each of them.
template <int LANES>
__device__ __forceinline__ float lane_sum(float x) {
  x = dpp_add<0xB1>(x);                               // quad_perm [1, 0, 3, 2]
  if constexpr (LANES >= 4) x = dpp_add<0x4E>(x);     // quad_perm [2, 3, 0, 1]
  if constexpr (LANES >= 8) x = dpp_add<0x141>(x);    // row_half_mirror
  if constexpr (LANES == 16) x = dpp_add<0x128>(x);   // row_ror 8
  return x;
}

template <bool BF16, int N>
__global__ __launch_bounds__(256) void scan_tokens_kernel(ScanParams p, int64_t blocks) {
  constexpr int kLanes = N / 4, kChannels = 256 / kLanes;
  const int64_t b = blockIdx.x;
  const int64_t n = b / blocks;
  const int64_t c = (b - n * blocks) * kChannels + threadIdx.x / kLanes;
  const int q = threadIdx.x % kLanes;
  if (c >= p.D) return;  // whole channels
  const int64_t mine = c * N + 4 * q;
  const int64_t in = slot_in(p.state, n);
  f32x4 h = {0.f, 0.f, 0.f, 0.f};
  if (in >= 0) h = p.state.bf16 ? load4<true>(p.state.in, in + mine) : load4<false>(p.state.in, in + mine);
  f32x4 A = load4<false>(p.A, mine);
#pragma unroll
  for (int e = 0; e < 4; ++e) A[e] *= kLog2e;
  const float bias = p.bias ? p.bias[c] : 0.f, skip = p.skip ? p.skip[c] : 0.f;
  const int64_t group = c / p.per_group;
  const int T = static_cast<int>(p.T);
  for (int t = 0; t < T; ++t) {
    const float u = load1<BF16>(p.u, n * p.us[0] + t * p.us[1] + c);
    float d = load1<BF16>(p.delta, n * p.ds[0] + t * p.ds[1] + c) + bias;
    const f32x4 B = load4<BF16>(p.B, n * p.bs[0] + t * p.bs[1] + group * p.bs[2] + 4 * q);
    const f32x4 C = load4<BF16>(p.C, n * p.cs[0] + t * p.cs[1] + group * p.cs[2] + 4 * q);
    const float z = p.z ? load1<BF16>(p.z, n * p.zs[0] + t * p.zs[1] + c) : 0.f;
    if (p.softplus) d = softplusf_(d);
    const float x = d * u;
    float y = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      h[e] = __builtin_fmaf(__builtin_amdgcn_exp2f(d * A[e]), h[e], x * B[e]);
      y = __builtin_fmaf(h[e], C[e], y);
    }
    y = lane_sum<kLanes>(y);
    if (p.skip) y = __builtin_fmaf(skip, u, y);
    if (p.z) y *= siluf_(z);
    if (q == 0) {
      const int64_t at = (n * T + t) * p.D + c;
      if constexpr (BF16) static_cast<unsigned short*>(p.out)[at] = float_to_bf16_bits(y);
      else static_cast<float*>(p.out)[at] = y;
    }
  }
  const int64_t out = slot_out(p.state, n);
  if (out >= 0) {
    if (p.state.bf16) store4<true>(p.state.out, out + mine, h);
    else store4<false>(p.state.out, out + mine, h);
  }
}

template <bool BF16, int N>
hipError_t go(const ScanParams& p, hipStream_t stream) {
  constexpr int kChannels = 1024 / N;
  const int64_t blocks = (p.D + kChannels - 1) / kChannels;
  hipLaunchKernelGGL((scan_tokens_kernel<BF16, N>), dim3(static_cast<unsigned>(p.N * blocks)), dim3(256), 0,
                     stream, p, blocks);
  return hipGetLastError();
}

template <bool BF16>
hipError_t go_n(const ScanParams& p, int n, hipStream_t stream) {
  switch (n) {
    case 8: return go<BF16, 8>(p, stream);
    case 16: return go<BF16, 16>(p, stream);
    case 32: return go<BF16, 32>(p, stream);
    default: return go<BF16, 64>(p, stream);
  }
}

}  // namespace

hipError_t launch_scan_tokens(const ScanParams& p, int n, bool io_bf16, hipStream_t stream) {
  return io_bf16 ? go_n<true>(p, n, stream) : go_n<false>(p, n, stream);
}

}  // namespace kda

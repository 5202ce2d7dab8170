// The selective state space scan for a few tokens per sequence (fixed layout, T <=
// kScanTokensMaxT): each state is read once, takes the T steps in FP32 registers and is
// written once, so the launch is bound by the states' bytes: 128 sequences of 8192 channels x 16
// FP32 states between slots of a pool, 143 MB in 29 us (4.9 TB/s, a copy of as much 28). A channel
// is n / 4 lanes of four states each.

#include <type_traits>

#include "kda_ssm_device.h"

namespace kda {

namespace {

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// v of lane J of each quad (of each pair of lanes where there are two to a channel).
template <int PAIR, int J>
__device__ __forceinline__ float of_lane(float v) {
  if constexpr (PAIR) return dpp<J == 0 ? 0xA0 : 0xF5>(v);
  else return dpp<0x55 * J>(v);
}

// LANES lanes of four states each hold NC channels: the sums of y[j] over them, channel j's in
// the lanes j of each quad (or pair).
template <int LANES, int NC>
__device__ __forceinline__ float lane_sums(const float (&y)[NC]) {
  const bool two = threadIdx.x & 2, odd = threadIdx.x & 1;
  float x;
  if constexpr (NC == 1) {
    x = y[0] + dpp<0xB1>(y[0]);                    // quad_perm [1, 0, 3, 2]
    if constexpr (LANES >= 4) x += dpp<0x4E>(x);   // quad_perm [2, 3, 0, 1]
  } else {
    float b[2] = {y[0], y[1]};
    if constexpr (NC == 4) {
#pragma unroll
      for (int i = 0; i < 2; ++i) b[i] = (two ? y[i + 2] : y[i]) + dpp<0x4E>(two ? y[i] : y[i + 2]);
    }
    x = (odd ? b[1] : b[0]) + dpp<0xB1>(odd ? b[0] : b[1]);
  }
  if constexpr (LANES >= 8) x += __shfl_xor(x, 4);
  if constexpr (LANES == 16) x += __shfl_xor(x, 8);
  return x;
}

// NC channels for the lanes of a channel (four, or two of eight states; one in small calls):
// lane j brings channel j's input and step size and finishes its output. The channels of
// lanes side by side are neighbours, so a wave's load of states is 1 KB without gaps (with
// NC neighbouring channels in a lane, 64 bytes of every 256: 128 tokens of 8192 channels, FP32
// states in a pool, 39.6 us, 32.1 so; one channel a lane 37.5).
template <bool BF16, int N, int NC>
__global__ __launch_bounds__(256) void scan_tokens_kernel(ScanParams p, uint32_t blocks) {
  constexpr int kLanes = N / 4, kSide = 64 / kLanes, kChannels = 4 * kSide * NC;
  const uint32_t seq = blockIdx.x / blocks;
  const int64_t n = seq;
  const int q = threadIdx.x % kLanes;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x - seq * blocks) * kChannels + threadIdx.x / 64 * (kSide * NC) + threadIdx.x % 64 / kLanes;
  const int64_t own = c0 + q % NC * kSide;
  const int64_t c = own < p.D ? own : p.D - 1;
  const int64_t in = slot_in(p.state, n), out = slot_out(p.state, n);
  const int64_t mine = c0 * N + 4 * q;
  f32x4 h[NC], A[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int64_t at = mine + j * (kSide * N);
    h[j] = A[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (c0 + j * kSide >= p.D) continue;
    if (in >= 0) h[j] = p.state.bf16 ? load_once4<true>(p.state.in, in + at) : load_once4<false>(p.state.in, in + at);
    A[j] = load4<false>(p.A, at);
  }
  const float bias = p.bias ? p.bias[c] : 0.f, skip = p.skip ? p.skip[c] : 0.f;
  const int64_t group = divide(c0 < p.D ? c0 : p.D - 1, p.per_group);
  const int T = static_cast<int>(p.T);
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) A[j][e] *= kLog2e;
  for (int t = 0; t < T; ++t) {
    const float u = load1<BF16>(p.u, n * p.us[0] + t * p.us[1] + c);
    float d = load1<BF16>(p.delta, n * p.ds[0] + t * p.ds[1] + c) + bias;
    const f32x4 B = load4<BF16>(p.B, n * p.bs[0] + t * p.bs[1] + group * p.bs[2] + 4 * q);
    const f32x4 C = load4<BF16>(p.C, n * p.cs[0] + t * p.cs[1] + group * p.cs[2] + 4 * q);
    const float z = p.z ? load1<BF16>(p.z, n * p.zs[0] + t * p.zs[1] + c) : 0.f;
    if (p.softplus) d = softplusf_(d);
    const float x = d * u;
    float y[NC];
    auto step = [&](auto index) {
      constexpr int j = decltype(index)::value;
      const float dj = NC == 1 ? d : of_lane<NC == 2, j>(d), xj = NC == 1 ? x : of_lane<NC == 2, j>(x);
      y[j] = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[j][e] = __builtin_fmaf(__builtin_amdgcn_exp2f(dj * A[j][e]), h[j][e], xj * B[e]);
        y[j] = __builtin_fmaf(h[j][e], C[e], y[j]);
      }
    };
    step(std::integral_constant<int, 0>{});
    if constexpr (NC >= 2) step(std::integral_constant<int, 1>{});
    if constexpr (NC == 4) {
      step(std::integral_constant<int, 2>{});
      step(std::integral_constant<int, 3>{});
    }
    float o = lane_sums<kLanes, NC>(y);
    if (p.skip) o = __builtin_fmaf(skip, u, o);
    if (p.z) o *= siluf_(z);
    if (q < NC && own < p.D) {
      const int64_t at = (n * T + t) * p.D + own;
      if constexpr (BF16) static_cast<unsigned short*>(p.out)[at] = float_to_bf16_bits(o);
      else static_cast<float*>(p.out)[at] = o;
    }
  }
  if (out < 0) return;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int64_t at = out + mine + j * (kSide * N);
    if (c0 + j * kSide >= p.D) continue;
    if (p.state.bf16) store_once4<true>(p.state.out, at, h[j]);
    else store_once4<false>(p.state.out, at, h[j]);
  }
}

template <bool BF16, int N, int NC>
hipError_t go_channels(const ScanParams& p, hipStream_t stream) {
  constexpr int kChannels = 1024 / N * NC;
  const int64_t blocks = (p.D + kChannels - 1) / kChannels;
  hipLaunchKernelGGL((scan_tokens_kernel<BF16, N, NC>), dim3(static_cast<unsigned>(p.N * blocks)), dim3(256), 0,
                     stream, p, static_cast<uint32_t>(blocks));
  return hipGetLastError();
}

template <bool BF16, int N>
hipError_t go(const ScanParams& p, hipStream_t stream) {
  // several channels where that still leaves two workgroups for each of 256 compute units, and
  // a wave's channels (at most 64) share their rows of B and C
  constexpr int kMost = N == 8 ? 2 : 4;
  const bool many = p.N * p.D * (N / 4) >= int64_t(512) * 256 * kMost &&
                    (p.per_group == p.D || p.per_group % 64 == 0);
  return many ? go_channels<BF16, N, kMost>(p, stream) : go_channels<BF16, N, 1>(p, stream);
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

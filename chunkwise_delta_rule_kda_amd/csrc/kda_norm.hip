// The gated norm,
//   y = residual + scale * act(gate) * weight * x / sqrt(mean(x^2) + eps)
//   z = next_weight * y / sqrt(mean(y^2) + eps)
// A row is held in registers between its two reductions, so every tensor is read or
// written once; the launch is bound by those bytes: 8192 x 12288 BF16 with gate, residual
// and the next norm, 1007 MB in 182 to 190 us by the run (5.3 to 5.5 TB/s); 8192 x 96 heads of 128 with a gate
// 111 us (5.4 TB/s). Rows of at most 512 elements share a wave; wider ones are a workgroup
// of as many threads as keep at most three or four pieces of eight each (2048 x 16384: 37 us
// by 512 threads, 50 by 256 with twice the registers).

#include "kda_device.h"
#include "kda_ops_internal.h"

namespace kda {

namespace {

// Eight values of a row as loaded.
template <bool BF16>
struct Raw8 {
  u32x4 x[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    const u32x4* w = reinterpret_cast<const u32x4*>(static_cast<const char*>(base) + at * (BF16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) x[i] = w[i];
  }
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (BF16) {
      const uint32_t w = x[0][e / 2];
      return __uint_as_float(e % 2 ? w & 0xffff0000u : w << 16);
    } else {
      return __uint_as_float(x[e / 4][e % 4]);
    }
  }
};

template <bool BF16>
__device__ __forceinline__ void store8(void* base, int64_t at, const float (&y)[8]) {
  const f32x4 lo = {y[0], y[1], y[2], y[3]}, hi = {y[4], y[5], y[6], y[7]};
  if constexpr (BF16) {
    *reinterpret_cast<bf16x8*>(static_cast<unsigned short*>(base) + at) = pack8(lo, hi);
  } else {
    f32x4* w = reinterpret_cast<f32x4*>(static_cast<float*>(base) + at);
    w[0] = lo;
    w[1] = hi;
  }
}

// One row: threads t of kThreads with NV pieces of eight, piece t + kThreads i.
// sum(x) must return the sum over the row's threads in each of them.
template <bool BF16, int THREADS, int NV, typename Sum>
__device__ __forceinline__ void norm_row(const NormParams& p, int64_t row, int t, Sum sum) {
  const int64_t mm = row / p.G, gg = row - mm * p.G;
  const int64_t xb = mm * p.xs[0] + gg * p.xs[1], gb = mm * p.gs[0] + gg * p.gs[1],
                rb = mm * p.rs[0] + gg * p.rs[1], ob = row * p.D;
  Raw8<BF16> x[NV], gate[NV], res[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = 8 * (t + THREADS * i);
    if (e < p.D) x[i].load(p.x, xb + e);
  }
  if (p.gate) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = 8 * (t + THREADS * i);
      if (e < p.D) gate[i].load(p.gate, gb + e);
    }
  }
  if (p.residual) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = 8 * (t + THREADS * i);
      if (e < p.D) res[i].load(p.residual, rb + e);
    }
  }
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (8 * (t + THREADS * i) >= p.D) continue;
#pragma unroll
    for (int k = 0; k < 8; ++k) sq += x[i][k] * x[i][k];
  }
  const float inv_d = 1.f / static_cast<float>(p.D);
  const float r = rsqrtf(sum(sq) * inv_d + p.eps);
  float y[NV][8];
  sq = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = 8 * (t + THREADS * i);
    if (e >= p.D) continue;
    float w[8];
    if (p.weight) load8<false>(p.weight, e, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float v = x[i][k] * r;
      if (p.weight) v *= w[k];
      if (p.gate) {
        const float a = gate[i][k];
        v *= p.silu ? a * sigmoidf_(a) : sigmoidf_(a);
      }
      v *= p.scale;
      if (p.residual) v += res[i][k];
      y[i][k] = v;
      sq += v * v;
    }
    store8<BF16>(p.out, ob + e, y[i]);
  }
  if (!p.next_out) return;
  const float rn = rsqrtf(sum(sq) * inv_d + p.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = 8 * (t + THREADS * i);
    if (e >= p.D) continue;
    float w[8];
    if (p.next_weight) load8<false>(p.next_weight, e, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      y[i][k] *= rn;
      if (p.next_weight) y[i][k] *= w[k];
    }
    store8<BF16>(p.next_out, ob + e, y[i]);
  }
}

// D <= 8 LANES <= 512: a row is LANES lanes of a wave.
template <bool BF16, int LANES>
__global__ __launch_bounds__(256) void norm_narrow_kernel(NormParams p) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / LANES) + threadIdx.x / LANES;
  if (row >= p.M * p.G) return;  // whole groups of LANES lanes
  norm_row<BF16, LANES, 1>(p, row, threadIdx.x % LANES, [](float x) {
#pragma unroll
    for (int s = 1; s < LANES; s <<= 1) x += __shfl_xor(x, s);
    return x;
  });
}

// D <= 8 THREADS NV: a row is a workgroup.
template <bool BF16, int THREADS, int NV>
__global__ __launch_bounds__(THREADS) void norm_wide_kernel(NormParams p) {
  constexpr int kWaves = THREADS / 64;
  __shared__ float part[2][kWaves];
  int turn = 0;
  norm_row<BF16, THREADS, NV>(p, blockIdx.x, threadIdx.x, [&](float x) {
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) x += __shfl_xor(x, s);
    float* w = part[turn++];  // the second sum has words of its own
    if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = x;
    __syncthreads();
    float all = 0.f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) all += w[i];
    return all;
  });
}

template <bool BF16, int LANES>
hipError_t narrow(const NormParams& p, hipStream_t stream) {
  const int64_t rows = p.M * p.G, per = 256 / LANES;
  hipLaunchKernelGGL((norm_narrow_kernel<BF16, LANES>), dim3(static_cast<unsigned>((rows + per - 1) / per)),
                     dim3(256), 0, stream, p);
  return hipGetLastError();
}

template <bool BF16, int THREADS, int NV>
hipError_t wide(const NormParams& p, hipStream_t stream) {
  hipLaunchKernelGGL((norm_wide_kernel<BF16, THREADS, NV>), dim3(static_cast<unsigned>(p.M * p.G)),
                     dim3(THREADS), 0, stream, p);
  return hipGetLastError();
}

template <bool BF16>
hipError_t go(const NormParams& p, hipStream_t stream) {
  const int threads = norm_threads(p.D);
  const int pieces = (p.D / 8 + threads - 1) / threads;  // of eight elements, per thread
  switch (threads) {
    case 8: return narrow<BF16, 8>(p, stream);
    case 16: return narrow<BF16, 16>(p, stream);
    case 32: return narrow<BF16, 32>(p, stream);
    case 64: return narrow<BF16, 64>(p, stream);
    case 128: return wide<BF16, 128, 1>(p, stream);
    case 256:
      return pieces == 1 ? wide<BF16, 256, 1>(p, stream)
             : pieces == 2 ? wide<BF16, 256, 2>(p, stream) : wide<BF16, 256, 3>(p, stream);
    default:
      return pieces == 2 ? wide<BF16, 512, 2>(p, stream)
             : pieces == 3 ? wide<BF16, 512, 3>(p, stream) : wide<BF16, 512, 4>(p, stream);
  }
}
static_assert(kNormMax == 8 * 512 * 4, "the widest row is four pieces of 512 threads");

}  // namespace

hipError_t launch_gated_norm(const NormParams& p, bool io_bf16, hipStream_t stream) {
  if (p.M * p.G <= 0) return hipSuccess;
  return io_bf16 ? go<true>(p, stream) : go<false>(p, stream);
}

}  // namespace kda

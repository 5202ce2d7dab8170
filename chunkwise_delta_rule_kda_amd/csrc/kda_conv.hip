// The short causal convolution of each channel with its own W taps,
//   y_t = act(bias + sum_i w_i x_{t - (W-1) + i})
// whose rows before the sequence are its state, and the state behind it: the last W - 1 rows.
// A thread takes eight channels (one 16-byte piece of a BF16 row) of a run of tokens of one
// sequence and keeps the last W - 1 rows in registers, so a row is read once, and W - 1 rows
// a second time where a run begins. Bound by its bytes, inputs and outputs in turn: 8192 x 36864
// BF16, 1209 MB in 216 us (5.6 TB/s, a copy of as much 227); FP32 packed, 221 MB in 52 us (4.3
// TB/s, the copy 42; 45 where each call writes the memory that the last one wrote, which the
// last-level cache then holds); 8192 x 2304 BF16, 76 MB in 18.3 us (the copy 16).

#include "kda_ssm_device.h"

namespace kda {

namespace {

template <bool BF16>
struct Row8 {
  u32x4 x[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    const u32x4* w = reinterpret_cast<const u32x4*>(static_cast<const char*>(base) + at * (BF16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) x[i] = w[i];
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) x[i] = u32x4{0u, 0u, 0u, 0u};
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

// LANES octets of channels and 256 / LANES runs for a workgroup; ROWS tokens in flight, one
// for calls of one token each. The taps come through LDS: read by each thread from memory they
// would be 64 cache lines a load.
template <bool BF16, int W, int ROWS, int LANES>
__global__ __launch_bounds__(256) void conv_kernel(ConvParams p, uint32_t blocks) {
  constexpr int kPitch = 8 * W + 4;  // floats of an octet's taps: sixteen lanes meet all banks
  __shared__ float taps[LANES * kPitch];
  const uint32_t row = blockIdx.x / blocks;
  const int64_t octet0 = static_cast<int64_t>(blockIdx.x - row * blocks) * LANES;
  const int lane = threadIdx.x % LANES;
  const int64_t octets = p.C / 8;
  const bool held = octet0 + lane < octets;
  const int64_t c = 8 * (held ? octet0 + lane : octets - 1);
  const int64_t w = static_cast<int64_t>(row) * (256 / LANES) + threadIdx.x / LANES;

  // All loads are on their way before the first wait: the taps', the first rows' and, of BF16, the
  // rows before those (8192 x 36864: 216 us, 223 with these behind the taps; FP32, whose rows
  // take twice the registers, packed 45.0 and 44.8).
  constexpr int kTaps = (LANES * 8 * W + 1023) / 1024;  // pieces of four of this thread
  const int count = static_cast<int>(octets - octet0 < LANES ? octets - octet0 : LANES) * 8 * W;
  f32x4 piece[kTaps];
#pragma unroll
  for (int k = 0; k < kTaps; ++k) {
    const int i = 4 * threadIdx.x + 1024 * k;
    if (i < count) piece[k] = *reinterpret_cast<const f32x4*>(&p.weight[octet0 * 8 * W + i]);
  }

  int64_t n, begin = 0, total = p.T, r;
  if (p.cu_seqlens) {
    // the wave's first lane's sequence, from which the others' are a few further
    n = find_sequence(p.cu_seqlens, p.N, p.run, __shfl(w, 0));
    while (n + 1 < p.N && divide(p.cu_seqlens[n + 1], p.run) + n + 1 <= w) ++n;
    begin = p.cu_seqlens[n];
    total = p.cu_seqlens[n + 1] - begin;
    r = w - (divide(begin, p.run) + n);
  } else if (ROWS == 1) {
    n = w;
    r = 0;
  } else {
    n = divide(w, p.runs_per_seq);
    r = w - n * p.runs_per_seq;
  }
  const int64_t t0 = r * p.run;
  const bool active = held && w < p.slots && r >= 0 && (r == 0 || t0 < total);
  const int64_t len = !active ? 0 : total - t0 < p.run ? total - t0 : p.run;
  const int64_t xb = (p.cu_seqlens ? 0 : n * p.xs[0]) + begin * p.xs[1] + c;
  const int64_t ob = ((p.cu_seqlens ? 0 : n * p.T) + begin) * p.C + c;
  const int64_t in = active ? slot_in(p.state, n) : -1;

  Row8<BF16> next[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
    if (i < len) next[i].load(p.x, xb + (t0 + i) * p.xs[1]);

  // Row `pos` of the sequence (pos < total), before its begin the state's.
  auto row_at = [&](int64_t pos, float (&v)[8]) {
    if (pos >= 0) {
      Row8<BF16> raw;
      raw.load(p.x, xb + pos * p.xs[1]);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = raw[e];
    } else if (in >= 0) {
      const int64_t at = in + (W - 1 + pos) * p.C + c;
      if (p.state.bf16) load8<true>(p.state.in, at, v);
      else load8<false>(p.state.in, at, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.f;
    }
  };
  float win[W - 1][8];  // the rows before the next token, the oldest first
  auto rows_before = [&] {
#pragma unroll
    for (int i = 0; i < W - 1; ++i) row_at(t0 - (W - 1) + i, win[i]);
  };
  if (BF16 && active) rows_before();

#pragma unroll
  for (int k = 0; k < kTaps; ++k) {
    const int i = 4 * threadIdx.x + 1024 * k;
    if (i < count) *reinterpret_cast<f32x4*>(&taps[i / (8 * W) * kPitch + i % (8 * W)]) = piece[k];
  }
  meet();
  if (!active) return;
  if (!BF16) rows_before();

  float wt[W][8], bias[8];
#pragma unroll
  for (int i = 0; i < 8 * W; i += 4) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(&taps[lane * kPitch + i]);
#pragma unroll
    for (int k = 0; k < 4; ++k) wt[(i + k) % W][(i + k) / W] = v[k];
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) bias[e] = 0.f;
  if (p.bias) load8<false>(p.bias, c, bias);

  // The first run's thread writes the final state too: nobody else reads these channels of
  // the initial one, which may be the same memory.
  const int64_t out = r == 0 ? slot_out(p.state, n) : -1;
  if (out >= 0) {
    float last[W - 1][8];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) row_at(total - (W - 1) + i, last[i]);
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      const int64_t at = out + i * p.C + c;
      if (p.state.bf16) store8<true>(p.state.out, at, last[i]);
      else store8<false>(p.state.out, at, last[i]);
    }
  }

  for (int64_t t = 0; t < len; t += ROWS) {
    Row8<BF16> now[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) now[i] = next[i];
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
      if (t + ROWS + i < len) next[i].load(p.x, xb + (t0 + t + ROWS + i) * p.xs[1]);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (t + i >= len) break;
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = now[i][e];
        float a = bias[e];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) a = __builtin_fmaf(wt[k][e], win[k][e], a);
        a = __builtin_fmaf(wt[W - 1][e], x, a);
        y[e] = p.silu ? siluf_(a) : a;
#pragma unroll
        for (int k = 0; k + 1 < W - 1; ++k) win[k][e] = win[k + 1][e];
        win[W - 2][e] = x;
      }
      store8<BF16>(p.out, ob + (t0 + t + i) * p.C, y);
    }
  }
}

template <bool BF16, int W, int LANES>
hipError_t go_lanes(const ConvParams& p, hipStream_t stream) {
  const int64_t blocks = (p.C / 8 + LANES - 1) / LANES, rows = (p.slots * LANES + 255) / 256;
  const dim3 grid(static_cast<unsigned>(blocks * rows));
  if (p.T == 1 && !p.cu_seqlens)
    hipLaunchKernelGGL((conv_kernel<BF16, W, 1, LANES>), grid, dim3(256), 0, stream, p,
                       static_cast<uint32_t>(blocks));
  else
    hipLaunchKernelGGL((conv_kernel<BF16, W, kConvRows, LANES>), grid, dim3(256), 0, stream, p,
                       static_cast<uint32_t>(blocks));
  return hipGetLastError();
}

template <bool BF16, int W>
hipError_t go(const ConvParams& p, hipStream_t stream) {
  return p.lanes == 64 ? go_lanes<BF16, W, 64>(p, stream)
         : p.lanes == 32 ? go_lanes<BF16, W, 32>(p, stream) : go_lanes<BF16, W, 8>(p, stream);
}

template <bool BF16>
hipError_t go_width(const ConvParams& p, int width, hipStream_t stream) {
  return width == 4 ? go<BF16, 4>(p, stream) : width == 3 ? go<BF16, 3>(p, stream) : go<BF16, 2>(p, stream);
}

}  // namespace

hipError_t launch_short_conv(const ConvParams& p, int width, bool io_bf16, hipStream_t stream) {
  if (p.slots * p.C <= 0) return hipSuccess;
  return io_bf16 ? go_width<true>(p, width, stream) : go_width<false>(p, width, stream);
}

}  // namespace kda

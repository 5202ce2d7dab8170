// Linear attention with one decay per head for a few tokens per sequence (fixed layout,
// T <= kLinDecodeMaxT): the token step itself,
//   S <- exp(g) S + v k^T ; o = s S q
// Each state is read once, takes the T steps in FP32 registers and is written once, so
// the launch is bound by the state traffic: 128 sequences x 24 heads of FP32 states, 404 MB
// in 73 us (5.5 TB/s, as a copy of 256 MB), 78 between scattered slots of a pool. A row of the state is K / 8 lanes of eight
// keys each; rows never meet, so a (sequence, head) is split over workgroups of `rows`
// value rows where there are few of them (one sequence of 6 heads: 3.4 us by 16 rows, 4.3
// by 64).

#include "kda_device.h"
#include "kda_ops_internal.h"

namespace kda {

namespace {

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                           0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}

// Sum over the LANES lanes (8 or 16) that hold one state row, in each of them.
template <int LANES>
__device__ __forceinline__ float lane_sum(float x) {
  x = dpp_add<0xB1>(x);   // quad_perm [1, 0, 3, 2]
  x = dpp_add<0x4E>(x);   // quad_perm [2, 3, 0, 1]
  x = dpp_add<0x141>(x);  // row_half_mirror: the other quad of eight lanes
  if constexpr (LANES == 16) x = dpp_add<0x128>(x);  // row_ror 8
  return x;
}

template <bool BF16, int KD, int NI>
__global__ __launch_bounds__(256) void linear_tokens_kernel(LinParams p, int blocks) {
  constexpr int kLanes = KD / 8, kPass = 256 / kLanes;  // rows per pass of the workgroup
  constexpr int kRows = kPass * NI;
  const int64_t b = blockIdx.x;
  const int64_t pair = b / blocks;
  const int64_t n = pair / p.H;
  const int h = static_cast<int>(pair - n * p.H);
  const int row0 = static_cast<int>(b - pair * blocks) * kRows + threadIdx.x / kLanes;
  const int cb = threadIdx.x % kLanes;
  const int hk = h / (p.H / p.Hk);

  const int64_t in = p.in_idx ? p.in_idx[n] : n;
  const int64_t head = static_cast<int64_t>(h) * p.V * KD + static_cast<int64_t>(row0) * KD + 8 * cb;
  float s[NI][8];
  if (p.state_in && in >= 0 && in < p.pool_slots) {
    const int64_t at = in * p.slot_pitch + head;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (p.st_bf16) load8<true>(p.state_in, at + i * kPass * KD, s[i]);
      else load8<false>(p.state_in, at + i * kPass * KD, s[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[i][e] = 0.f;
  }

  const float fixed = p.log_decay ? p.log_decay[h] : 0.f;
  const int64_t qb = n * p.qs[0] + hk * p.qs[2] + 8 * cb;
  const int64_t kb = n * p.ks[0] + hk * p.ks[2] + 8 * cb;
  const int64_t vb = n * p.vs[0] + h * p.vs[2] + row0;
  const int T = static_cast<int>(p.T);
  for (int t = 0; t < T; ++t) {
    const int64_t tok = (n * T + t) * p.H + h;
    float q[8], k[8], v[NI];
    load8<BF16>(p.q, qb + t * p.qs[1], q);
    load8<BF16>(p.k, kb + t * p.ks[1], k);
#pragma unroll
    for (int i = 0; i < NI; ++i) v[i] = load1<BF16>(p.v, vb + t * p.vs[1] + i * kPass);
    float x = fixed;
    if (p.g) x += p.g_bf16 ? load1<true>(p.g, tok) : load1<false>(p.g, tok);
    const float d = expf(x);
    float o[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s[i][e] = s[i][e] * d + v[i] * k[e];
        dot += s[i][e] * q[e];
      }
      o[i] = p.scale * lane_sum<kLanes>(dot);
    }
    // lane cb of a row's lanes stores the row of pass cb
    float mine = o[0];
#pragma unroll
    for (int i = 1; i < NI; ++i) mine = cb == i ? o[i] : mine;
    if (cb < NI) {
      const int64_t at = tok * p.V + row0 + cb * kPass;
      if constexpr (BF16) static_cast<unsigned short*>(p.o)[at] = float_to_bf16_bits(mine);
      else static_cast<float*>(p.o)[at] = mine;
    }
  }

  const int64_t out = p.out_idx ? p.out_idx[n] : n;
  if (p.state_out && out >= 0 && out < p.pool_slots) {
    const int64_t at = out * p.slot_pitch + head;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const f32x4 lo = {s[i][0], s[i][1], s[i][2], s[i][3]}, hi = {s[i][4], s[i][5], s[i][6], s[i][7]};
      if (p.st_bf16) {
        *reinterpret_cast<bf16x8*>(static_cast<unsigned short*>(p.state_out) + at + i * kPass * KD) = pack8(lo, hi);
      } else {
        f32x4* w = reinterpret_cast<f32x4*>(static_cast<float*>(p.state_out) + at + i * kPass * KD);
        w[0] = lo;
        w[1] = hi;
      }
    }
  }
}

template <bool BF16, int KD, int NI>
hipError_t go(const LinParams& p, hipStream_t stream) {
  const int rows = 256 / (KD / 8) * NI;
  const int blocks = p.V / rows;
  const int64_t wgs = p.N * p.H * blocks;
  hipLaunchKernelGGL((linear_tokens_kernel<BF16, KD, NI>), dim3(static_cast<unsigned>(wgs)), dim3(256),
                     0, stream, p, blocks);
  return hipGetLastError();
}

template <bool BF16>
hipError_t go_io(const LinParams& p, int k_dim, int rows, hipStream_t stream) {
  if (k_dim == 128) {
    switch (rows) {
      case 64: return go<BF16, 128, 4>(p, stream);
      case 32: return go<BF16, 128, 2>(p, stream);
      default: return go<BF16, 128, 1>(p, stream);
    }
  }
  return rows == 64 ? go<BF16, 64, 2>(p, stream) : go<BF16, 64, 1>(p, stream);
}

}  // namespace

hipError_t launch_linear_tokens(const LinParams& p, int k_dim, bool io_bf16, int rows,
                                hipStream_t stream) {
  return io_bf16 ? go_io<true>(p, k_dim, rows, stream) : go_io<false>(p, k_dim, rows, stream);
}

}  // namespace kda

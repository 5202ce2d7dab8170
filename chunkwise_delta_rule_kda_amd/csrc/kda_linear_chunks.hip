// Linear attention with one decay per head, chunk by chunk: outputs and final states of a
// segment (or a whole sequence) from its start state. The layout and the equations are in
// kda_linear_core.h.

#include "kda_linear_core.h"

namespace kda {

namespace {

// P^T tile (J, I): rows are tokens j of block J, columns tokens i of block I; this lane
// holds j = 16 J + 4 grp + 0..3 of token i = 16 I + m, scaled by s and the decay from j
// to i, and writes them as row i of P in operand order.
template <bool BF16, int KD, int PPR_P, int J, int I>
__device__ __forceinline__ void score_tile(const unsigned char* q_tile, const unsigned char* k_tile,
                                           unsigned char* p_tile, const Gates& gt, float scale,
                                           int grp, int m) {
  typedef typename FragOf<BF16>::type Frag;
  constexpr int kPpr = KD * (BF16 ? 2 : 4) / 16;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int kb = 0; kb < KD / 32; ++kb) {
    Frag kf, qf;
    row_frag<kPpr>(k_tile, 16 * J + m, kb, grp, kf);
    row_frag<kPpr>(q_tile, 16 * I + m, kb, grp, qf);
    acc = mma(kf, qf, acc);
  }
  const int i = 16 * I + m;
  if constexpr (I == J) {
    const double Gi = gt.G[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float f = __builtin_amdgcn_exp2f(static_cast<float>(Gi - gt.G[16 * J + 4 * grp + j]));
      acc[j] = 4 * grp + j <= m ? acc[j] * (scale * f) : 0.f;
    }
  } else {
    float a = gt.a[i];
#pragma unroll
    for (int b = J + 1; b < I; ++b) a *= gt.E[b];
    acc *= a * *reinterpret_cast<const f32x4*>(&gt.b[16 * J + 4 * grp]);
  }
  if constexpr (BF16) {
    *reinterpret_cast<i16x4*>(p_tile + 16 * piece_at<PPR_P>(i, 4 * (J / 2) + grp) + 8 * (J % 2)) = pack4(acc);
  } else {
    *reinterpret_cast<f32x4*>(p_tile + 16 * piece_at<PPR_P>(i, 4 * J + grp)) = acc;
  }
}

// Operand of token row i of P over the 32 tokens kappa(kb, grp, e).
template <int PPR>
__device__ __forceinline__ void p_frag(const unsigned char* tile, int i, int kb, int grp, bf16x8& f) {
  f = *reinterpret_cast<const bf16x8*>(tile + 16 * piece_at<PPR>(i, 4 * kb + grp));
}
template <int PPR>
__device__ __forceinline__ void p_frag(const unsigned char* tile, int i, int kb, int grp, F32x8& f) {
  f.lo = *reinterpret_cast<const f32x4*>(tile + 16 * piece_at<PPR>(i, 8 * kb + grp));
  f.hi = *reinterpret_cast<const f32x4*>(tile + 16 * piece_at<PPR>(i, 8 * kb + 4 + grp));
}

template <bool BF16, int KD, int NC, bool LOW>
__global__ __launch_bounds__(256) void linear_chunks_kernel(LinParams p) {
  typedef typename FragOf<BF16>::type Frag;
  constexpr int kEs = BF16 ? 2 : 4;
  constexpr int R = 64 * NC;
  constexpr int KB = KD / 32;
  constexpr int kPprK = KD * kEs / 16, kPprV = R * kEs / 16, kPprP = 64 * kEs / 16;
  __shared__ __align__(16) unsigned char q_tile[64 * KD * kEs];
  __shared__ __align__(16) unsigned char k_tile[64 * KD * kEs];
  __shared__ __align__(16) unsigned char v_tile[64 * R * kEs];
  __shared__ __align__(16) unsigned char p_tile[64 * 64 * kEs];
  __shared__ Gates gates;

  LinTask task;
  if (!find_task(p, task)) return;  // uniform
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int grp = lane >> 4, m = lane & 15;
  const int hk = task.h / (p.H / p.Hk);
  const int row0 = task.vblk * R + wave * 16 * NC;  // the wave's first value row
  const unsigned char* qp = static_cast<const unsigned char*>(p.q) +
                            (row_offset(p, p.qs, task.n, task.tok0) + hk * p.qs[2]) * kEs;
  const unsigned char* kp = static_cast<const unsigned char*>(p.k) +
                            (row_offset(p, p.ks, task.n, task.tok0) + hk * p.ks[2]) * kEs;
  const unsigned char* vp = static_cast<const unsigned char*>(p.v) +
                            (row_offset(p, p.vs, task.n, task.tok0) + task.h * p.vs[2] + task.vblk * R) * kEs;
  const uint32_t qpitch = static_cast<uint32_t>(p.qs[1] * kEs);
  const uint32_t kpitch = static_cast<uint32_t>(p.ks[1] * kEs);
  const uint32_t vpitch = static_cast<uint32_t>(p.vs[1] * kEs);

  Tile<kPprK> qt, kt;
  Tile<kPprV> vt;
  double x = 0.0;
  auto fetch = [&](int64_t at) {
    const int left = static_cast<int>(task.len - at < 64 ? task.len - at : 64);
    qt.load(qp + at * qpitch, qpitch, left, tid);
    kt.load(kp + at * kpitch, kpitch, left, tid);
    vt.load(vp + at * vpitch, vpitch, left, tid);
    if (wave == 0) x = load_log_decay(p, task.tok0 + at, lane, left, task.h);
  };
  if (task.len > 0) fetch(0);

  // Start state: the scan's, or the sequence's own.
  f32x4 S[KD / 16][NC];
  const int64_t head_state = static_cast<int64_t>(task.h) * p.V * KD;
  if (p.segmented && !(task.first && task.last)) {
    load_state(S, p.scan_s, (static_cast<int64_t>(task.h) * p.slots + task.slot) * p.V * KD, false, KD,
               row0, grp, m);
  } else {
    const int64_t slot = p.in_idx ? p.in_idx[task.n] : task.n;
    if (p.state_in && slot >= 0 && slot < p.pool_slots) {
      load_state(S, p.state_in, slot * p.slot_pitch + head_state, p.st_bf16, KD, row0, grp, m);
    } else {
#pragma unroll
      for (int t = 0; t < KD / 16; ++t)
#pragma unroll
        for (int c = 0; c < NC; ++c) S[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }
  // The tiles of P above the diagonal that an operand read covers are zero throughout.
#pragma unroll
  for (int i = tid; i < 64 * kPprP; i += 256) {
    const u32x4 zero = {0u, 0u, 0u, 0u};
    *reinterpret_cast<u32x4*>(p_tile + 16 * i) = zero;
  }

  for (int64_t at = 0; at < task.len; at += 64) {
    const int left = static_cast<int>(task.len - at < 64 ? task.len - at : 64);
    __syncthreads();  // the previous chunk's operands have been read
    qt.store(q_tile, tid);
    kt.store(k_tile, tid);
    vt.store(v_tile, tid);
    if (wave == 0) make_gates(gates, x, lane, left, p.scale);
    __syncthreads();
    if (at + 64 < task.len) fetch(at + 64);

    // The ten score tiles on and below the diagonal, two or three per wave.
    switch (wave) {
      case 0:
        score_tile<BF16, KD, kPprP, 0, 0>(q_tile, k_tile, p_tile, gates, p.scale, grp, m);
        score_tile<BF16, KD, kPprP, 0, 2>(q_tile, k_tile, p_tile, gates, p.scale, grp, m);
        score_tile<BF16, KD, kPprP, 1, 2>(q_tile, k_tile, p_tile, gates, p.scale, grp, m);
        break;
      case 1:
        score_tile<BF16, KD, kPprP, 0, 1>(q_tile, k_tile, p_tile, gates, p.scale, grp, m);
        score_tile<BF16, KD, kPprP, 1, 1>(q_tile, k_tile, p_tile, gates, p.scale, grp, m);
        score_tile<BF16, KD, kPprP, 2, 2>(q_tile, k_tile, p_tile, gates, p.scale, grp, m);
        break;
      case 2:
        score_tile<BF16, KD, kPprP, 0, 3>(q_tile, k_tile, p_tile, gates, p.scale, grp, m);
        score_tile<BF16, KD, kPprP, 1, 3>(q_tile, k_tile, p_tile, gates, p.scale, grp, m);
        break;
      default:
        score_tile<BF16, KD, kPprP, 2, 3>(q_tile, k_tile, p_tile, gates, p.scale, grp, m);
        score_tile<BF16, KD, kPprP, 3, 3>(q_tile, k_tile, p_tile, gates, p.scale, grp, m);
        break;
    }

    // O^T from the entering state.
    f32x4 O[4][NC];
    {
      Frag sf[NC][KB];
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) to_frag(S[2 * kb][c], S[2 * kb + 1][c], sf[c][kb]);
#pragma unroll
      for (int it = 0; it < 4; ++it) {
#pragma unroll
        for (int c = 0; c < NC; ++c) O[it][c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          Frag qf;
          row_frag<kPprK>(q_tile, 16 * it + m, kb, grp, qf);
#pragma unroll
          for (int c = 0; c < NC; ++c) O[it][c] = mma(sf[c][kb], qf, O[it][c]);
        }
        const float d = gates.d[16 * it + m];
#pragma unroll
        for (int c = 0; c < NC; ++c) O[it][c] *= d;
      }
    }
    Frag vf[NC][2];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
        col_frag<kPprV>(v_tile, wave * 16 * NC + 4 * c, 4 * NC, kb, grp, m, vf[c][kb]);
    update_state<BF16, KD, NC, LOW>(S, vf, k_tile, gates, grp, m);
    __syncthreads();  // P is whole

#pragma unroll
    for (int it = 0; it < 4; ++it) {
#pragma unroll
      for (int kb = 0; kb <= it / 2; ++kb) {
        Frag pf;
        p_frag<kPprP>(p_tile, 16 * it + m, kb, grp, pf);
#pragma unroll
        for (int c = 0; c < NC; ++c) O[it][c] = mma(vf[c][kb], pf, O[it][c]);
      }
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int i = 16 * it + m;
      if (i >= left) continue;
      const int64_t e = ((task.tok0 + at + i) * p.H + task.h) * p.V + row0 + 4 * NC * grp;
      if constexpr (BF16 && NC == 2) {
        *reinterpret_cast<bf16x8*>(static_cast<unsigned short*>(p.o) + e) = pack8(O[it][0], O[it][1]);
      } else {
#pragma unroll
        for (int c = 0; c < NC; ++c) store4<BF16>(p.o, e + 4 * c, O[it][c]);
      }
    }
  }

  if (task.last && p.state_out) {
    const int64_t slot = p.out_idx ? p.out_idx[task.n] : task.n;
    if (slot >= 0 && slot < p.pool_slots)
      store_state(S, p.state_out, slot * p.slot_pitch + head_state, p.st_bf16, KD, row0, grp, m);
  }
}

template <bool BF16, int KD, int NC, bool LOW>
hipError_t go(const LinParams& p, hipStream_t stream) {
  const int64_t sub = static_cast<int64_t>(p.heads_per_task) * p.vblocks;
  const int64_t wgs = (p.tasks + 7) / 8 * 8 * sub;
  hipLaunchKernelGGL((linear_chunks_kernel<BF16, KD, NC, LOW>), dim3(static_cast<unsigned>(wgs)),
                     dim3(256), 0, stream, p);
  return hipGetLastError();
}

template <int KD>
hipError_t go_k(const LinParams& p, bool bf16, int rows, hipStream_t stream) {
  if (!bf16) return go<false, KD, 1, false>(p, stream);
  if (rows == 128) {
    if (p.hi_lo) return go<true, KD, 2, true>(p, stream);
    return go<true, KD, 2, false>(p, stream);
  }
  if (p.hi_lo) return go<true, KD, 1, true>(p, stream);
  return go<true, KD, 1, false>(p, stream);
}

}  // namespace

hipError_t launch_linear_chunks(const LinParams& p, int k_dim, bool io_bf16, int value_block,
                                hipStream_t stream) {
  return k_dim == 128 ? go_k<128>(p, io_bf16, value_block, stream)
                      : go_k<64>(p, io_bf16, value_block, stream);
}

}  // namespace kda

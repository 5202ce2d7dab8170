// Segments of linear attention with one decay per head: the end state from zero of every
// segment that has a later one in its sequence, and the scan over a sequence's segments.

#include "kda_linear_core.h"

namespace kda {

namespace {

// 64 value rows of one (segment, head) by eight waves, as in the output launch
// (kda_linear_chunks.hip): four load the tiles of chunk c + 2 into a ring of three and make
// the decay factors of chunk c + 1, four update the state. Z_p goes to the segment's scan
// slot, the segment's total decay to scan_d. A segment is a chain of chunks, so the launch
// is as long as one: 8192 tokens x 6 heads in 19 segments of seven chunks 12.5 us (1.5 us a
// chunk and the launch); FP32 I/O, bound by its matrix products, 2 x 1999 tokens x 12 heads
// 25.2 us (28.8 by four waves that also loaded the tiles).
constexpr int kStages = 3;

template <bool BF16, int KD, int PARTS>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 4))) void linear_states_kernel(LinParams p) {
  constexpr int R = kLinRows;
  constexpr int kElem = BF16 ? 2 : 4;
  constexpr int kPprK = KD * kElem / 16, kPprV = R * kElem / 16;
  constexpr int kTileK = 64 * KD * kElem, kStage = kTileK + 64 * R * kElem;
  constexpr int kLoads = AsyncTile<kPprK>::kLoads + AsyncTile<kPprV>::kLoads;
  extern __shared__ __align__(1024) unsigned char lds[];
  Gates* const gates = reinterpret_cast<Gates*>(lds + kStages * kStage);

  LinTask task;
  if (!find_task(p, task) || task.last) return;  // uniform
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) & 3;
  const int grp = lane >> 4, m = lane & 15;
  const int chunks = static_cast<int>((task.len + 63) >> 6);  // a segment with a later one is whole
  const int64_t slot = static_cast<int64_t>(task.h) * p.slots + task.slot;

  if (__builtin_amdgcn_readfirstlane(tid >> 8) != 0) {
    __builtin_amdgcn_s_setprio(2);
    const int hk = task.h / (p.H / p.Hk);
    const unsigned char* kp = static_cast<const unsigned char*>(p.k) +
                              (row_offset(p, p.ks, task.n, task.tok0) + hk * p.ks[2]) * kElem;
    const unsigned char* vp = static_cast<const unsigned char*>(p.v) +
                              (row_offset(p, p.vs, task.n, task.tok0) + task.h * p.vs[2] + task.vblk * R) * kElem;
    const uint32_t kpitch = static_cast<uint32_t>(p.ks[1] * kElem);
    const uint32_t vpitch = static_cast<uint32_t>(p.vs[1] * kElem);
    AsyncTile<kPprK> kt;
    AsyncTile<kPprV> vt;
    kt.init(wave, lane, kpitch);
    vt.init(wave, lane, vpitch);
    auto fetch = [&](int stage) {
      unsigned char* st = lds + stage * kStage;
      kt.load(kp, kpitch, 64, st, wave, lane);
      vt.load(vp, vpitch, 64, st + kTileK, wave, lane);
      kp += static_cast<uint64_t>(kpitch) * 64;
      vp += static_cast<uint64_t>(vpitch) * 64;
    };
    const float fixed = p.log_decay ? p.log_decay[task.h] : 0.f;
    auto log_decay = [&](int chunk) {
      return load_log_decay(p, task.tok0 + 64 * static_cast<int64_t>(chunk) + 16 * wave + m, task.h);
    };
    float x0 = log_decay(0), x1 = 0.f;
    fetch(0);
    if (chunks > 1) {
      x1 = log_decay(1);
      fetch(1);
    }
    make_gates(gates[0], x0, fixed, wave, lane, true, 1.f);
    int stage = 0;
    auto step = [&](int chunk, float x_next, float& x_load) {
      if (chunk + 1 < chunks) wait_and_meet<kLoads>();
      else wait_and_meet<0>();
      if (chunk + 2 < chunks) {
        x_load = log_decay(chunk + 2);
        fetch(stage >= 1 ? stage - 1 : kStages - 1);
      }
      make_gates(gates[(chunk + 1) & 1], x_next, fixed, wave, lane, chunk + 1 < chunks, 1.f);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    };
    for (int chunk = 0; chunk < chunks; chunk += 2) {
      step(chunk, x1, x0);
      if (chunk + 1 < chunks) step(chunk + 1, x0, x1);
    }
    return;
  }

  float total = 1.f;
  int stage = 0;
  auto chunk_loop = [&](auto update) {
    for (int chunk = 0; chunk < chunks; ++chunk) {
      meet();
      const unsigned char* k_tile = lds + stage * kStage;
      const Gates& gt = gates[chunk & 1];
      const BlockDecays bd = block_decays(gt);
      update(k_tile, k_tile + kTileK, gt, bd);
      total *= bd.all;
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
  };
  const int row0 = task.vblk * R + wave * 16;
  if constexpr (BF16) {
    f32x4 S[KD / 16][1];
#pragma unroll
    for (int t = 0; t < KD / 16; ++t) S[t][0] = f32x4{0.f, 0.f, 0.f, 0.f};
    chunk_loop([&](const unsigned char* k_tile, const unsigned char* v_tile, const Gates& gt, const BlockDecays& bd) {
      bf16x8 vf[2], kf[KD / 16][2];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) col_frag<kPprV>(v_tile, wave * 16, 4, kb, grp, m, vf[kb]);
      KeyDecays kd;
      kd.read(gt, bd, grp);
      // all reads before the products: left alone, each is read right before its use
#pragma unroll
      for (int t = 0; t < KD / 16; ++t)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) col_frag<kPprK>(k_tile, 32 * (t / 2) + 4 * (t % 2), 8, kb, grp, m, kf[t][kb]);
      __builtin_amdgcn_sched_barrier(0);
      bf16x8 vw[2][PARTS];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) scale_frag<PARTS>(vf[kb], kd.w[kb][0], kd.w[kb][1], vw[kb]);
#pragma unroll
      for (int t = 0; t < KD / 16; ++t) S[t][0] *= bd.all;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int part = 0; part < PARTS; ++part)
#pragma unroll
          for (int t = 0; t < KD / 16; ++t) S[t][0] = mma(kf[t][kb], vw[kb][part], S[t][0]);
    });
    store_state(S, p.scan_s, slot * p.V * KD, false, KD, row0, grp, m);
  } else {
    f32x4 S[KD / 16];
#pragma unroll
    for (int t = 0; t < KD / 16; ++t) S[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    chunk_loop([&](const unsigned char* k_tile, const unsigned char* v_tile, const Gates& gt, const BlockDecays& bd) {
      F32x8 vf[2];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) col_frag<kPprV>(v_tile, wave * 16, 4, kb, grp, m, vf[kb]);
      update_state_f32<KD>(S, vf, k_tile, gt, bd, grp, m);
    });
    store_state_f32(S, p.scan_s, slot * p.V * KD, false, row0 + m, grp);
  }
  if (tid == 0 && task.vblk == 0) p.scan_d[slot] = total;
}

// S_{p+1} = D_p S_p + Z_p over the segments of one (sequence, head), elementwise and bound
// by the latency of its loads (19 segments x 6 heads, 15 MB: 5.5 us): a
// thread carries four elements of the state and leaves every segment's start state in its
// slot. The first segment's slot gets the sequence's initial state, so that the launch
// that follows reads no state another workgroup of it writes (in-place updates).
__global__ __launch_bounds__(256) void linear_scan_kernel(LinParams p, int K) {
  const int64_t per = static_cast<int64_t>(p.V) * K / 4;
  const int64_t blocks = (per + 255) / 256;
  const int64_t pair = blockIdx.x / blocks;
  const int64_t e = (blockIdx.x - pair * blocks) * 256 + threadIdx.x;
  const int64_t n = pair / p.H;
  const int h = static_cast<int>(pair - n * p.H);
  if (e >= per) return;
  int64_t first = n * p.segs_per_seq, segs = p.segs_per_seq;
  if (p.cu_seqlens) {
    const int64_t a = p.cu_seqlens[n], b = p.cu_seqlens[n + 1];
    first = a / p.seg_len + n;
    segs = (b - a + p.seg_len - 1) / p.seg_len;
  }
  if (segs <= 1) return;  // the output launch reads state_in itself
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (p.state_in) {
    const int64_t slot = p.in_idx ? p.in_idx[n] : n;
    if (slot >= 0 && slot < p.pool_slots) {
      const int64_t at = slot * p.slot_pitch + h * static_cast<int64_t>(p.V) * K + 4 * e;
      s = p.st_bf16 ? load4<true>(p.state_in, at) : load4<false>(p.state_in, at);
    }
  }
  const int64_t base = static_cast<int64_t>(h) * p.slots + first;
  f32x4* z = reinterpret_cast<f32x4*>(p.scan_s) + base * per + e;
  const float* d = p.scan_d + base;
  // Eight segments' loads before their stores: a chain of dependent loads would be a trip
  // through the memory for each segment.
  int64_t i = 0;
  for (; i + 8 < segs; i += 8) {
    f32x4 zi[8];
    float di[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      zi[j] = z[(i + j) * per];
      di[j] = d[i + j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      z[(i + j) * per] = s;
      s = s * di[j] + zi[j];
    }
  }
  f32x4 zi[8];
  float di[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bool has = i + j + 1 < segs;
    zi[j] = has ? z[(i + j) * per] : f32x4{0.f, 0.f, 0.f, 0.f};
    di[j] = has ? d[i + j] : 0.f;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (i + j >= segs) break;
    z[(i + j) * per] = s;
    s = s * di[j] + zi[j];
  }
}

template <bool BF16, int KD, int PARTS>
hipError_t go(const LinParams& p, hipStream_t stream) {
  constexpr int kLds = kStages * 64 * (BF16 ? 2 : 4) * (KD + kLinRows) + 2 * sizeof(Gates);
  static_assert(kLds <= (BF16 ? 80 : 160) * 1024, "two workgroups (FP32: one) per compute unit");
  hipLaunchKernelGGL((linear_states_kernel<BF16, KD, PARTS>), dim3(static_cast<unsigned>(linear_grid(p))),
                     dim3(512), kLds, stream, p);
  return hipGetLastError();
}

template <int KD>
hipError_t go_k(const LinParams& p, bool bf16, hipStream_t stream) {
  if (!bf16) return go<false, KD, 1>(p, stream);
  return p.split ? go<true, KD, 3>(p, stream) : go<true, KD, 1>(p, stream);
}

}  // namespace

hipError_t launch_linear_states(const LinParams& p, int k_dim, bool io_bf16, hipStream_t stream) {
  return k_dim == 128 ? go_k<128>(p, io_bf16, stream) : go_k<64>(p, io_bf16, stream);
}

hipError_t launch_linear_scan(const LinParams& p, int k_dim, hipStream_t stream) {
  const int64_t per = static_cast<int64_t>(p.V) * k_dim / 4;
  const int64_t wgs = (per + 255) / 256 * p.N * p.H;
  hipLaunchKernelGGL(linear_scan_kernel, dim3(static_cast<unsigned>(wgs)), dim3(256), 0, stream, p,
                     k_dim);
  return hipGetLastError();
}

}  // namespace kda

// Linear attention with one decay per head, chunk by chunk: outputs and final states of a
// segment (or a whole sequence) from its start state. The layout and the equations are in
// kda_linear_core.h.

#include "kda_linear_core.h"

namespace kda {

namespace {

// P in LDS: operand (I, kb), tokens 16 I + m over the 32 tokens kappa(kb, grp, e), is a
// 16-byte piece of each lane in turn (FP32: two such halves). The operands on and below the
// diagonal are six.
template <bool BF16>
__device__ __forceinline__ constexpr int p_block(int I, int kb) {
  return (I < 2 ? I : 2 * I - 2 + kb) * (BF16 ? 1024 : 2048);
}
template <bool BF16>
constexpr int kScoreBytes = 6 * (BF16 ? 1024 : 2048);

__device__ __forceinline__ void p_frag(const unsigned char* tile, int I, int kb, int lane_piece, F32x8& f) {
  f.lo = *reinterpret_cast<const f32x4*>(tile + p_block<false>(I, kb) + lane_piece);
  f.hi = *reinterpret_cast<const f32x4*>(tile + p_block<false>(I, kb) + 1024 + lane_piece);
}

// The scores of a chunk are the ten 16 x 16 tiles P^T (J, I), J <= I, shared out so that wave
// W of four has its diagonal one and one or two others. Rows are tokens j of block J,
// columns tokens i of block I; a lane holds j = 16 J + 4 grp + 0..3 of token i = 16 I + m,
// scaled by s and the decay from j to i, and writes them as row i of P in operand order.
// read() has all LDS reads (reads are not moved before a write), make() none.
template <bool BF16, int KD, int W>
struct Scores {
  typedef typename FragOf<BF16>::type Frag;
  static constexpr int KB = KD / 32, kPpr = KD * (BF16 ? 2 : 4) / 16;
  static constexpr int J1 = W == 0 ? 0 : W - 1, I1 = W == 0 ? 3 : W;  // the second tile
  static constexpr bool kThird = W < 2;
  static constexpr int J2 = W == 0 ? 1 : 0, I2 = W == 0 ? 3 : 2;
  Frag k0[KB], q0[KB], other[KB], third[KB];
  double Li, Lj[4];
  float a1, a2;
  f32x4 b1, b2, x, y, z;

  static __device__ __forceinline__ void rows(const unsigned char* tile, int block, int grp, int m,
                                              Frag (&f)[KB]) {
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) row_frag<kPpr>(tile, 16 * block + m, kb, grp, f[kb]);
  }
  template <int J, int I>
  static __device__ __forceinline__ void factors(const Gates& gt, int grp, int m, float& a, f32x4& b) {
    a = gt.a[16 * I + m];
#pragma unroll
    for (int e = J + 1; e < I; ++e) a *= gt.E[e];
    b = *reinterpret_cast<const f32x4*>(&gt.b[16 * J + 4 * grp]);
  }
  static __device__ __forceinline__ f32x4 product(const Frag (&kf)[KB], const Frag (&qf)[KB]) {
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) acc = mma(kf[kb], qf[kb], acc);
    return acc;
  }
  __device__ __forceinline__ void read(const unsigned char* q_tile, const unsigned char* k_tile,
                                       const Gates& gt, int grp, int m) {
    rows(k_tile, W, grp, m, k0);
    rows(q_tile, W, grp, m, q0);
    if constexpr (W == 0) rows(q_tile, I1, grp, m, other);
    else rows(k_tile, J1, grp, m, other);
    if constexpr (W == 0) rows(k_tile, J2, grp, m, third);
    if constexpr (W == 1) rows(q_tile, I2, grp, m, third);
    Li = gt.L[16 * W + m];
#pragma unroll
    for (int j = 0; j < 4; ++j) Lj[j] = gt.L[16 * W + 4 * grp + j];
    factors<J1, I1>(gt, grp, m, a1, b1);
    if constexpr (kThird) factors<J2, I2>(gt, grp, m, a2, b2);
  }
  __device__ __forceinline__ void make(double log2_scale, int grp, int m) {
    x = product(k0, q0);
    if constexpr (W == 0) y = product(k0, other), z = product(third, other);
    else y = product(other, q0);
    if constexpr (W == 1) z = product(other, third);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float f = exp2_of((Li + log2_scale) - Lj[j]);
      x[j] = 4 * grp + j <= m ? x[j] * f : 0.f;
    }
    y *= a1 * b1;
    if constexpr (kThird) z *= a2 * b2;
  }
  template <int J, int I>
  static __device__ __forceinline__ void put(unsigned char* p_tile, int lane, f32x4 v) {
    unsigned char* at = p_tile + p_block<BF16>(I, J / 2) + 16 * lane;
    if constexpr (BF16) *reinterpret_cast<i16x4*>(at + 8 * (J % 2)) = pack4(v);
    else *reinterpret_cast<f32x4*>(at + 1024 * (J % 2)) = v;
  }
  __device__ __forceinline__ void write(unsigned char* p_tile, int lane) const {
    put<W, W>(p_tile, lane, x);
    put<J1, I1>(p_tile, lane, y);
    if constexpr (kThird) put<J2, I2>(p_tile, lane, z);
  }
};

template <int W>
struct WaveNumber {
  static constexpr int value = W;
};
// f(WaveNumber<wave>()) for one of four waves.
template <typename F>
__device__ __forceinline__ void by_wave(int wave, F f) {
  switch (wave) {
    case 0: f(WaveNumber<0>()); break;
    case 1: f(WaveNumber<1>()); break;
    case 2: f(WaveNumber<2>()); break;
    default: f(WaveNumber<3>()); break;
  }
}

// FP32 I/O, FP32 MFMA (a sixteenth of the BF16 rate), which bounds it: 12288 clocks of
// products per SIMD and chunk of about 17000. Four waves hold the next chunk's tiles in
// registers, write them to LDS, and form the scores beside the other four's products with
// the state; those add P V while the next tiles are written. Two tiles of each kind do not
// fit the LDS (a stage is 80 KB). 2 x 1999 tokens x 12 heads (240 workgroups of at most seven
// chunks): 59 us, the matrix pipes busy 65 % of it; operands read one group ahead of their
// products spilled (86 us).
template <int KD>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void linear_f32_kernel(LinParams p) {
  constexpr int R = kLinRows;
  constexpr int kPprK = KD / 4, kPprV = R / 4;
  extern __shared__ __align__(1024) unsigned char lds[];
  unsigned char* const q_tile = lds;
  unsigned char* const k_tile = q_tile + 64 * KD * 4;
  unsigned char* const v_tile = k_tile + 64 * KD * 4;
  unsigned char* const p_tile = v_tile + 64 * R * 4;
  Gates& gates = *reinterpret_cast<Gates*>(p_tile + kScoreBytes<false>);

  LinTask task;
  if (!find_task(p, task)) return;  // uniform
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) & 3;
  const int grp = lane >> 4, m = lane & 15;
  const int chunks = static_cast<int>((task.len + 63) >> 6);
  const int tail = static_cast<int>(task.len - 64 * static_cast<int64_t>(chunks - 1));
  // The tiles of P above the diagonal that an operand read covers are zero throughout.
  for (int i = tid; i < kScoreBytes<false> / 16; i += 512)
    *reinterpret_cast<u32x4*>(p_tile + 16 * i) = u32x4{0u, 0u, 0u, 0u};

  if (__builtin_amdgcn_readfirstlane(tid >> 8) != 0) {
    __builtin_amdgcn_s_setprio(2);
    const int hk = task.h / (p.H / p.Hk), t = tid & 255;
    const unsigned char* qp = static_cast<const unsigned char*>(p.q) +
                              (row_offset(p, p.qs, task.n, task.tok0) + hk * p.qs[2]) * 4;
    const unsigned char* kp = static_cast<const unsigned char*>(p.k) +
                              (row_offset(p, p.ks, task.n, task.tok0) + hk * p.ks[2]) * 4;
    const unsigned char* vp = static_cast<const unsigned char*>(p.v) +
                              (row_offset(p, p.vs, task.n, task.tok0) + task.h * p.vs[2] + task.vblk * R) * 4;
    const uint32_t qpitch = static_cast<uint32_t>(p.qs[1] * 4);
    const uint32_t kpitch = static_cast<uint32_t>(p.ks[1] * 4);
    const uint32_t vpitch = static_cast<uint32_t>(p.vs[1] * 4);
    Tile<kPprK> qt, kt;
    Tile<kPprV> vt;
    const float fixed = p.log_decay ? p.log_decay[task.h] : 0.f;
    float x = 0.f;
    auto fetch = [&](int chunk) {
      const int rows = chunk + 1 < chunks ? 64 : tail, i = 16 * wave + m;
      const int64_t at = 64 * static_cast<int64_t>(chunk);
      qt.load(qp + at * qpitch, qpitch, rows, t);
      kt.load(kp + at * kpitch, kpitch, rows, t);
      vt.load(vp + at * vpitch, vpitch, rows, t);
      x = load_log_decay(p, task.tok0 + at + (i < rows ? i : rows - 1), task.h);
    };
    if (chunks > 0) fetch(0);
    for (int chunk = 0; chunk < chunks; ++chunk) {
      qt.store(q_tile, t);
      kt.store(k_tile, t);
      vt.store(v_tile, t);
      make_gates(gates, x, fixed, wave, lane, 16 * wave + m < (chunk + 1 < chunks ? 64 : tail), p.scale);
      meet();  // the tiles are whole
      if (chunk + 1 < chunks) fetch(chunk + 1);
      by_wave(wave, [&](auto w) {
        Scores<false, KD, decltype(w)::value> scores;
        scores.read(q_tile, k_tile, gates, grp, m);
        scores.make(p.log2_scale, grp, m);
        scores.write(p_tile, lane);
      });
      meet();  // the tiles have been read, P is whole
    }
    return;
  }

  const int row0 = task.vblk * R + wave * 16;  // the wave's first value row
  f32x4 S[KD / 16];
#pragma unroll
  for (int t = 0; t < KD / 16; ++t) S[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const StateAt from = start_state(p, task, KD), to = end_state(p, task, KD);
  if (from.base) load_state_f32(S, from.base, from.at, from.bf16, row0 + m, grp);
  for (int chunk = 0; chunk < chunks; ++chunk) {
    meet();
    // O^T from the entering state.
    const BlockDecays bd = block_decays(gates);
    f32x4 O[4];
#pragma unroll
    for (int it = 0; it < 4; ++it) O[it] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int h = 0; h < KD / 64; ++h) {
      f32x4 q[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int it = 0; it < 4; ++it)
          q[j][it] = *reinterpret_cast<const f32x4*>(q_tile + 16 * piece_at<kPprK>(16 * it + m, 16 * h + 4 * grp + j));
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int it = 0; it < 4; ++it)
            O[it] = __builtin_amdgcn_mfma_f32_16x16x4f32(S[4 * h + t][j], q[j][it][t], O[it], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) O[it] *= bd.before[it] * gates.a[16 * it + m];
    F32x8 vf[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) col_frag<kPprV>(v_tile, wave * 16, 4, kb, grp, m, vf[kb]);
    update_state_f32<KD>(S, vf, k_tile, gates, bd, grp, m);
    meet();

#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int it = 2 * kb; it < 4; it += 2) {
        F32x8 pf[2];
        p_frag(p_tile, it, kb, 16 * lane, pf[0]);
        p_frag(p_tile, it + 1, kb, 16 * lane, pf[1]);
        mma_pair(vf[kb], pf, O[it], O[it + 1]);
      }
    const int rows = chunk + 1 < chunks ? 64 : tail;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int i = 16 * it + m;
      if (i < rows)
        store4<false>(p.o, ((task.tok0 + 64 * static_cast<int64_t>(chunk) + i) * p.H + task.h) * p.V + row0 + 4 * grp, O[it]);
    }
  }
  if (to.base) store_state_f32(S, const_cast<void*>(to.base), to.at, to.bf16, row0 + m, grp);
}

// BF16 I/O: eight waves and one barrier per chunk. Behind the barrier of chunk c its tiles
// and factors are whole, and the scores of chunk c - 1.
// * Four score waves load the tiles of chunk c + 2 into an LDS ring of three, form the
//   scores of chunk c and the decay factors of chunk c + 1.
// * Four state waves add P V of chunk c - 1 to its outputs and store them, form the
//   outputs of chunk c from the entering state, and update the state.
// The chain through a chunk bounds it, no unit alone: of the 3000 clocks (1.33 us) that a chunk
// of 64 rows takes within the last-level cache the LDS is active for 1405 (362 instructions,
// each state wave reads all of Q and K), the vector units for 1430, the matrix pipes for 770.
// With one wave of each kind per SIMD there is little to fill the gaps: over 8192 tokens x 96
// heads (3920 clocks a chunk, from memory) the waves wait for data or the barrier 30 % of
// their time and to be issued 39 %. 128 rows per workgroup read Q and K once for twice the
// rows, 4400 clocks a chunk, but are half as many workgroups: the geometry's model chooses
// (kda_ops_api.cpp). 8192 tokens x 96 heads: 247 us (815 MB, 3.3 TB/s); four waves with two
// barriers per chunk and tiles through registers took 377.
constexpr int kStages = 3;

template <int KD, int NC, int PARTS>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void linear_ring_kernel(LinParams p) {
  constexpr int R = 64 * NC;
  constexpr int KB = KD / 32;
  constexpr int kPprK = KD / 8, kPprV = R / 8;
  constexpr int kTileK = 128 * KD, kTileV = 128 * R, kStage = 2 * kTileK + kTileV;
  constexpr int kLoads = 2 * AsyncTile<kPprK>::kLoads + AsyncTile<kPprV>::kLoads;
  extern __shared__ __align__(1024) unsigned char lds[];
  unsigned char* const p_tile = lds + kStages * kStage;
  Gates* const gates = reinterpret_cast<Gates*>(p_tile + 2 * kScoreBytes<true>);

  LinTask task;
  if (!find_task(p, task)) return;  // uniform
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) & 3;
  const bool score_wave = __builtin_amdgcn_readfirstlane(tid >> 8) != 0;
  const int grp = lane >> 4, m = lane & 15;
  const int chunks = static_cast<int>((task.len + 63) >> 6);
  const int tail = static_cast<int>(task.len - 64 * static_cast<int64_t>(chunks - 1));  // of the last chunk

  // The tiles of P above the diagonal that an operand read covers are zero throughout.
  for (int i = tid; i < 2 * kScoreBytes<true> / 16; i += 512)
    *reinterpret_cast<u32x4*>(p_tile + 16 * i) = u32x4{0u, 0u, 0u, 0u};

  if (score_wave) {
    __builtin_amdgcn_s_setprio(2);  // short, and the state waves wait for it
    const int hk = task.h / (p.H / p.Hk);
    const unsigned char* qp = static_cast<const unsigned char*>(p.q) +
                              (row_offset(p, p.qs, task.n, task.tok0) + hk * p.qs[2]) * 2;
    const unsigned char* kp = static_cast<const unsigned char*>(p.k) +
                              (row_offset(p, p.ks, task.n, task.tok0) + hk * p.ks[2]) * 2;
    const unsigned char* vp = static_cast<const unsigned char*>(p.v) +
                              (row_offset(p, p.vs, task.n, task.tok0) + task.h * p.vs[2] + task.vblk * R) * 2;
    const uint32_t qpitch = static_cast<uint32_t>(p.qs[1] * 2);
    const uint32_t kpitch = static_cast<uint32_t>(p.ks[1] * 2);
    const uint32_t vpitch = static_cast<uint32_t>(p.vs[1] * 2);
    AsyncTile<kPprK> qt, kt;
    AsyncTile<kPprV> vt;
    qt.init(wave, lane, qpitch);
    kt.init(wave, lane, kpitch);
    vt.init(wave, lane, vpitch);
    auto fetch = [&](int chunk, int stage) {
      const int rows = chunk + 1 < chunks ? 64 : tail;
      unsigned char* st = lds + stage * kStage;
      qt.load(qp, qpitch, rows, st, wave, lane);
      kt.load(kp, kpitch, rows, st + kTileK, wave, lane);
      vt.load(vp, vpitch, rows, st + 2 * kTileK, wave, lane);
      qp += static_cast<uint64_t>(qpitch) * 64;
      kp += static_cast<uint64_t>(kpitch) * 64;
      vp += static_cast<uint64_t>(vpitch) * 64;
    };
    const float fixed = p.log_decay ? p.log_decay[task.h] : 0.f;
    auto log_decay = [&](int chunk) {  // of the wave's 16-token block
      const int rows = chunk + 1 < chunks ? 64 : tail, i = 16 * wave + m;
      return load_log_decay(p, task.tok0 + 64 * static_cast<int64_t>(chunk) + (i < rows ? i : rows - 1), task.h);
    };
    // The log decays of chunk c are loaded right before its tiles (operations complete in
    // issue order: behind them they would wait for them), and kept in x0 or x1 by parity.
    float x0 = 0.f, x1 = 0.f;
    if (chunks > 0) {
      x0 = log_decay(0);
      fetch(0, 0);
      if (chunks > 1) {
        x1 = log_decay(1);
        fetch(1, 1);
      }
      make_gates(gates[0], x0, fixed, wave, lane, 16 * wave + m < (chunks > 1 ? 64 : tail), p.scale);
    }
    int stage = 0;
    auto step = [&](int chunk, float x_next, float& x_load) {
      const bool more = chunk + 1 < chunks;
      // This chunk's loads are done; the next chunk's may be outstanding.
      if (more) wait_and_meet<kLoads>();
      else wait_and_meet<0>();
      const unsigned char* q_tile = lds + stage * kStage;
      const unsigned char* k_tile = q_tile + kTileK;
      const Gates& gt = gates[chunk & 1];
      const int next_rows = !more ? 0 : chunk + 2 < chunks ? 64 : tail;
      by_wave(wave, [&](auto w) {
        Scores<true, KD, decltype(w)::value> scores;
        scores.read(q_tile, k_tile, gt, grp, m);
        if (chunk + 2 < chunks) {
          x_load = log_decay(chunk + 2);
          fetch(chunk + 2, stage >= 1 ? stage - 1 : kStages - 1);
        }
        BlockGates next;
        next.make(x_next, fixed, 16 * wave + m < next_rows, p.scale);
        scores.make(p.log2_scale, grp, m);
        scores.write(p_tile + (chunk & 1) * kScoreBytes<true>, lane);
        next.write(gates[(chunk + 1) & 1], wave, lane);
      });
      stage = stage + 1 == kStages ? 0 : stage + 1;
    };
    for (int chunk = 0; chunk < chunks; chunk += 2) {
      step(chunk, x1, x0);
      if (chunk + 1 < chunks) step(chunk + 1, x0, x1);
    }
    if (chunks > 0) meet();
    return;
  }

  const int row0 = task.vblk * R + wave * 16 * NC;  // the wave's first value row
  f32x4 S[KD / 16][NC];
#pragma unroll
  for (int t = 0; t < KD / 16; ++t)
#pragma unroll
    for (int c = 0; c < NC; ++c) S[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  const StateAt from = start_state(p, task, KD);
  if (from.base) load_state(S, from.base, from.at, from.bf16, KD, row0, grp, m);
  // Output rows: stores past a chunk's last token are dropped by the bounds (of the chunk
  // before the first one all are).
  const uint32_t opitch = static_cast<uint32_t>(p.H) * p.V * 2;
  unsigned char* op = static_cast<unsigned char*>(p.o) +
                      (task.tok0 * p.H + task.h) * static_cast<int64_t>(p.V) * 2 -
                      static_cast<int64_t>(opitch) * 64;
  const int col = 2 * (row0 + 4 * NC * grp), lane_piece = 16 * lane;
  f32x4 O[4][NC];      // of the chunk before: from the state that entered it
  bf16x8 vf[NC][2];    // its V operands
#pragma unroll
  for (int c = 0; c < NC; ++c) {
#pragma unroll
    for (int it = 0; it < 4; ++it) O[it][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    vf[c][0] = vf[c][1] = bf16x8{};
  }
  u32x2 done[4][NC];
  // O + P V of a chunk, rounded.
  bf16x8 pf[6];
  auto read_scores = [&](int chunk) {
    const unsigned char* scores = p_tile + (chunk & 1) * kScoreBytes<true>;
#pragma unroll
    for (int i = 0; i < 6; ++i) pf[i] = *reinterpret_cast<const bf16x8*>(scores + 1024 * i + lane_piece);
  };
  auto with_scores = [&]() {
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int it = 2 * kb; it < 4; ++it)
#pragma unroll
        for (int c = 0; c < NC; ++c) O[it][c] = mma(vf[c][kb], pf[p_block<true>(it, kb) / 1024], O[it][c]);
  };
  auto round = [&]() {
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
      for (int c = 0; c < NC; ++c) done[it][c] = __builtin_bit_cast(u32x2, pack4(O[it][c]));
  };
  auto store = [&](int rows) {
    const uint32_t bytes = rows > 0 ? static_cast<uint32_t>(rows - 1) * opitch + p.V * 2 : 0;
    __amdgpu_buffer_rsrc_t out = __builtin_amdgcn_make_buffer_rsrc(op, 0, bytes, 0x00020000);
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int e = (16 * it + m) * static_cast<int>(opitch) + col;
      if constexpr (NC == 2)
        __builtin_amdgcn_raw_buffer_store_b128(
            u32x4{done[it][0][0], done[it][0][1], done[it][1][0], done[it][1][1]}, out, e, 0, 0);
      else
        __builtin_amdgcn_raw_buffer_store_b64(done[it][0], out, e, 0, 0);
    }
    op += static_cast<uint64_t>(opitch) * 64;
  };

  // The chunk's work in an order that keeps LDS reads one group ahead of the products that
  // need them (left alone, the compiler reads each operand right before its use).
  int stage = 0;
  for (int chunk = 0; chunk < chunks; ++chunk) {
    meet();
    const unsigned char* q_tile = lds + stage * kStage;
    const unsigned char* k_tile = q_tile + kTileK;
    const unsigned char* v_tile = k_tile + kTileK;
    const Gates& gt = gates[chunk & 1];
    bf16x8 qf[4][KB];
    auto read_queries = [&](int it) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) row_frag<kPprK>(q_tile, 16 * it + m, kb, grp, qf[it][kb]);
    };
    read_scores(chunk + 1);  // of the chunk before
    read_queries(0);
    read_queries(1);
    const BlockDecays bd = block_decays(gt);
    float a[4];
#pragma unroll
    for (int it = 0; it < 4; ++it) a[it] = gt.a[16 * it + m];
    __builtin_amdgcn_sched_barrier(0);
    bf16x8 sf[NC][KB];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) sf[c][kb] = pack8(S[2 * kb][c], S[2 * kb + 1][c]);
    with_scores();
    read_queries(2);
    __builtin_amdgcn_sched_barrier(0);
    round();
    // O^T from the entering state.
    auto inter = [&](int it) {  // blocks it and it + 1: products in turn are independent
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int i = it; i < it + 2; ++i)
#pragma unroll
          for (int c = 0; c < NC; ++c)
            O[i][c] = mma(sf[c][kb], qf[i][kb], kb == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : O[i][c]);
    };
    auto scale = [&](int it) {
      const float d = bd.before[it] * a[it];
#pragma unroll
      for (int c = 0; c < NC; ++c) O[it][c] *= d;
    };
    read_queries(3);
    inter(0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
        col_frag<kPprV>(v_tile, wave * 16 * NC + 4 * c, 4 * NC, kb, grp, m, vf[c][kb]);
    KeyDecays kd;
    kd.read(gt, bd, grp);
    bf16x8 kf[KD / 16][2];
    auto read_keys = [&](int t) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) col_frag<kPprK>(k_tile, 32 * (t / 2) + 4 * (t % 2), 8, kb, grp, m, kf[t][kb]);
    };
    read_keys(0);
    read_keys(1);
    inter(2);
    __builtin_amdgcn_sched_barrier(0);
    scale(0), scale(1);
    bf16x8 vw[NC][2][PARTS];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int c = 0; c < NC; ++c) scale_frag<PARTS>(vf[c][kb], kd.w[kb][0], kd.w[kb][1], vw[c][kb]);
    read_keys(2);
    read_keys(3);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < KD / 16; t += 2) {
      if (t + 4 < KD / 16) {
        read_keys(t + 4);
        read_keys(t + 5);
      }
#pragma unroll
      for (int u = t; u < t + 2; ++u)
#pragma unroll
        for (int c = 0; c < NC; ++c) S[u][c] *= bd.all;
#pragma unroll
      for (int part = 0; part < PARTS; ++part)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int u = t; u < t + 2; ++u)
#pragma unroll
            for (int c = 0; c < NC; ++c)
              S[u][c] = mma(kf[u][kb], vw[c][kb][part], S[u][c]);
      __builtin_amdgcn_sched_barrier(0);
    }
    scale(2), scale(3);
    store(chunk > 0 ? 64 : 0);
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  if (chunks > 0) {
    meet();
    read_scores(chunks + 1);
    with_scores();
    round();
    store(tail);
  }

  const StateAt to = end_state(p, task, KD);
  if (to.base) store_state(S, const_cast<void*>(to.base), to.at, to.bf16, KD, row0, grp, m);
}

template <int KD, int NC, int PARTS>
hipError_t go_ring(const LinParams& p, hipStream_t stream) {
  constexpr int kLds = kStages * (256 * KD + 128 * 64 * NC) + 2 * kScoreBytes<true> + 2 * sizeof(Gates);
  static_assert(kLds <= 160 * 1024, "LDS of a compute unit");
  const int64_t wgs = linear_grid(p);
  hipLaunchKernelGGL((linear_ring_kernel<KD, NC, PARTS>), dim3(static_cast<unsigned>(wgs)), dim3(512), kLds,
                     stream, p);
  return hipGetLastError();
}

template <int KD>
hipError_t go_f32(const LinParams& p, hipStream_t stream) {
  constexpr int kLds = 64 * 4 * (2 * KD + kLinRows) + kScoreBytes<false> + sizeof(Gates);
  static_assert(kLds <= 160 * 1024, "LDS of a compute unit");
  const int64_t wgs = linear_grid(p);
  hipLaunchKernelGGL((linear_f32_kernel<KD>), dim3(static_cast<unsigned>(wgs)), dim3(512), kLds, stream, p);
  return hipGetLastError();
}

template <int KD>
hipError_t go_k(const LinParams& p, bool bf16, int rows, hipStream_t stream) {
  if (!bf16) return go_f32<KD>(p, stream);
  if (rows == 128) return go_ring<KD, 2, 1>(p, stream);
  return p.split ? go_ring<KD, 1, 3>(p, stream) : go_ring<KD, 1, 1>(p, stream);
}

}  // namespace

hipError_t launch_linear_chunks(const LinParams& p, int k_dim, bool io_bf16, int rows,
                                hipStream_t stream) {
  return k_dim == 128 ? go_k<128>(p, io_bf16, rows, stream) : go_k<64>(p, io_bf16, rows, stream);
}

}  // namespace kda

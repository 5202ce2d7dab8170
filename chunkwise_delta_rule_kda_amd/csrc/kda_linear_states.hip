// Segments of linear attention with one decay per head: the end state from zero of every
// segment that has a later one in its sequence, and the scan over a sequence's segments.

#include "kda_linear_core.h"

namespace kda {

namespace {

// Workgroup: R = 64 NC value rows of one (segment, head); Z_p to the segment's scan slot,
// the segment's total decay to scan_d.
template <bool BF16, int KD, int NC, bool LOW>
__global__ __launch_bounds__(256) void linear_states_kernel(LinParams p) {
  typedef typename FragOf<BF16>::type Frag;
  constexpr int kEs = BF16 ? 2 : 4;
  constexpr int R = 64 * NC;
  constexpr int kPprK = KD * kEs / 16, kPprV = R * kEs / 16;
  __shared__ __align__(16) unsigned char k_tile[64 * KD * kEs];
  __shared__ __align__(16) unsigned char v_tile[64 * R * kEs];
  __shared__ Gates gates;

  LinTask task;
  if (!find_task(p, task) || task.last) return;  // uniform
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int grp = lane >> 4, m = lane & 15;
  const int hk = task.h / (p.H / p.Hk);
  const int row0 = task.vblk * R + wave * 16 * NC;
  const unsigned char* kp = static_cast<const unsigned char*>(p.k) +
                            (row_offset(p, p.ks, task.n, task.tok0) + hk * p.ks[2]) * kEs;
  const unsigned char* vp = static_cast<const unsigned char*>(p.v) +
                            (row_offset(p, p.vs, task.n, task.tok0) + task.h * p.vs[2] + task.vblk * R) * kEs;
  const uint32_t kpitch = static_cast<uint32_t>(p.ks[1] * kEs);
  const uint32_t vpitch = static_cast<uint32_t>(p.vs[1] * kEs);

  f32x4 S[KD / 16][NC];
#pragma unroll
  for (int t = 0; t < KD / 16; ++t)
#pragma unroll
    for (int c = 0; c < NC; ++c) S[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  float total = 1.f;

  Tile<kPprK> kt;
  Tile<kPprV> vt;
  double x = 0.0;
  auto fetch = [&](int64_t at) {
    const int left = static_cast<int>(task.len - at < 64 ? task.len - at : 64);
    kt.load(kp + at * kpitch, kpitch, left, tid);
    vt.load(vp + at * vpitch, vpitch, left, tid);
    if (wave == 0) x = load_log_decay(p, task.tok0 + at, lane, left, task.h);
  };
  if (task.len > 0) fetch(0);
  for (int64_t at = 0; at < task.len; at += 64) {
    const int left = static_cast<int>(task.len - at < 64 ? task.len - at : 64);
    __syncthreads();
    kt.store(k_tile, tid);
    vt.store(v_tile, tid);
    if (wave == 0) make_gates(gates, x, lane, left, 1.f);
    __syncthreads();
    if (at + 64 < task.len) fetch(at + 64);
    Frag vf[NC][2];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
        col_frag<kPprV>(v_tile, wave * 16 * NC + 4 * c, 4 * NC, kb, grp, m, vf[c][kb]);
    total *= gates.D;
    update_state<BF16, KD, NC, LOW>(S, vf, k_tile, gates, grp, m);
  }
  const int64_t slot = static_cast<int64_t>(task.h) * p.slots + task.slot;
  store_state(S, p.scan_s, slot * p.V * KD, false, KD, row0, grp, m);
  if (tid == 0 && task.vblk == 0) p.scan_d[slot] = total;
}

// S_{p+1} = D_p S_p + Z_p over the segments of one (sequence, head), elementwise: a
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
  for (int64_t i = 0; i + 1 < segs; ++i) {
    const f32x4 zi = z[i * per];
    z[i * per] = s;
    s = s * d[i] + zi;
  }
  z[(segs - 1) * per] = s;
}

template <bool BF16, int KD, int NC, bool LOW>
hipError_t go(const LinParams& p, hipStream_t stream) {
  const int64_t sub = static_cast<int64_t>(p.heads_per_task) * p.vblocks;
  const int64_t wgs = (p.tasks + 7) / 8 * 8 * sub;
  hipLaunchKernelGGL((linear_states_kernel<BF16, KD, NC, LOW>), dim3(static_cast<unsigned>(wgs)),
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

hipError_t launch_linear_states(const LinParams& p, int k_dim, bool io_bf16, int value_block,
                                hipStream_t stream) {
  return k_dim == 128 ? go_k<128>(p, io_bf16, value_block, stream)
                      : go_k<64>(p, io_bf16, value_block, stream);
}

hipError_t launch_linear_scan(const LinParams& p, int k_dim, hipStream_t stream) {
  const int64_t per = static_cast<int64_t>(p.V) * k_dim / 4;
  const int64_t wgs = (per + 255) / 256 * p.N * p.H;
  hipLaunchKernelGGL(linear_scan_kernel, dim3(static_cast<unsigned>(wgs)), dim3(256), 0, stream, p,
                     k_dim);
  return hipGetLastError();
}

}  // namespace kda

// The selective state space scan over prompts. For channel c and its n states,
//   h <- exp(d A) h + d u B ; y = sum C h + D u ; out = y z sigmoid(z)
// with d = softplus(delta + bias). The decay differs by channel and state and its sums over
// time by channel, so nothing of it is a matrix product: per (token, channel, state) it is two
// multiplications, an exponential and two fused multiply-adds of the vector units.
//
// A workgroup holds 32 channels of one sequence (or of one time segment of it), a wave eight
// of them: lane L has channel L % 8 and the n / 8 states of group L / 8, in registers for the
// whole run. Tiles of 32 tokens go through LDS twice buffered, with one barrier each: all
// threads bring u, delta and B, C from memory two tiles ahead and turn delta into d and d u,
// and finish the outputs of the tile before.

#include "kda_ssm_device.h"

namespace kda {

namespace {

// LDS operations are complete and all waves here; loads from memory stay in flight.
__device__ __forceinline__ void meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

struct ScanTask {
  int64_t n, slot, row0, len, seg;  // row0: token row of the segment's begin in its sequence's strides
  int64_t begin;                    // first row of the sequence (0 in the fixed layout)
  int cblk;
  bool first, last;
};

// Workgroups b and b + 8 run on the same XCD one after the other: they get neighbouring
// channel blocks, whose 64-byte parts of a BF16 row share a cache line.
__device__ __forceinline__ bool scan_task(const ScanParams& p, ScanTask& t) {
  const int64_t b = blockIdx.x;
  const int64_t i = b >> 3;
  const int64_t task = ((i >> 1) * 8 + (b & 7)) * 2 + (i & 1);
  const int64_t w = task / p.cblocks;
  if (w >= p.slots) return false;
  t.cblk = static_cast<int>(task - w * p.cblocks);
  t.slot = w;
  int64_t total = p.T;
  if (p.cu_seqlens) {
    t.n = find_sequence(p.cu_seqlens, p.N, p.seg_len, w);
    t.begin = p.cu_seqlens[t.n];
    total = p.cu_seqlens[t.n + 1] - t.begin;
    t.seg = w - (t.begin / p.seg_len + t.n);
  } else {
    t.n = w / p.segs_per_seq;
    t.begin = 0;
    t.seg = w - t.n * p.segs_per_seq;
  }
  const int64_t at = t.seg * p.seg_len;
  t.first = t.seg == 0;
  if (t.seg < 0 || (t.seg > 0 && at >= total)) return false;
  t.row0 = t.begin + at;
  t.len = total - at < p.seg_len ? total - at : p.seg_len;
  t.last = at + t.len >= total;
  return true;
}

// Four consecutive elements as loaded.
template <bool BF16>
struct Raw4 {
  uint32_t x[BF16 ? 2 : 4];
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    if constexpr (BF16) {
      const u32x2 w = *reinterpret_cast<const u32x2*>(static_cast<const unsigned short*>(base) + at);
      x[0] = w[0];
      x[1] = w[1];
    } else {
      const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const float*>(base) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = w[i];
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (BF16 ? 2 : 4); ++i) x[i] = 0u;
  }
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (BF16) return __uint_as_float(e % 2 ? x[e / 2] & 0xffff0000u : x[e / 2] << 16);
    else return __uint_as_float(x[e]);
  }
};

// Sums of eight tokens' values over the lane groups L / 8: lane L gets token L / 8's.
__device__ __forceinline__ float reduce8(const float (&v)[8]) {
  float a[4], b[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // lanes from 32 on: token i + 4
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[i]), __float_as_uint(v[i + 4]), false, false);
    a[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // odd rows of 16 lanes: token i + 2
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(a[i]), __float_as_uint(a[i + 2]), false, false);
    b[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  const bool odd = threadIdx.x & 8;
  const float keep = odd ? b[1] : b[0], give = odd ? b[0] : b[1];
  return keep + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                              0, __builtin_bit_cast(int, give), 0x128, 0xF, 0xF, false));  // row_ror 8
}

constexpr int kYRow = kScanChannels + 8;  // floats of an LDS row of y: no two rows' banks meet

// OUT: outputs from the true start state; otherwise a segment's end state from zero (the
// first segment's from the sequence's start) and the sum of its step sizes.
template <bool BF16, int N, bool OUT>
__global__ __launch_bounds__(256) void scan_kernel(ScanParams p) {
  constexpr int NS = N / 8;                // states of a lane
  constexpr int kBC = OUT ? 2 * NS : NS;   // of B and C, for a lane and token
  constexpr int kQuads = N / 4 * (OUT ? 2 : 1) * kScanTile;  // pieces of four of a tile's B and C
  constexpr int kPer = (kQuads + 255) / 256;
  __shared__ float dx[2][kScanTile / 2][kScanChannels][4];  // d, d u of two tokens
  __shared__ float bc[2][kScanTile][8][kBC];
  __shared__ float ys[OUT ? 2 : 1][OUT ? kScanTile : 1][kYRow];

  ScanTask task;
  if (!scan_task(p, task)) return;
  if (!OUT && task.last && !task.first) return;  // nobody starts from its end
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int ch = lane & 7, g = lane >> 3;
  const int64_t c0 = static_cast<int64_t>(task.cblk) * kScanChannels;

  // ---- this lane's channel and states
  const int64_t c = c0 + 8 * wave + ch;
  const bool held = c < p.D;
  float A[NS], h[NS];
  float sum = 0.f;
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    A[s] = held ? p.A[c * N + g * NS + s] * kLog2e : 0.f;
    h[s] = 0.f;
  }
  const int64_t mine = c * N + g * NS;  // in a slot
  if (held) {
    if (p.segmented && OUT) {
      // the start state, through the ends of the segments before
      const int64_t base = task.slot - task.seg, all = p.D * N;
      if (task.first) {
#pragma unroll
        for (int s = 0; s < NS; ++s) h[s] = p.starts[task.n * all + mine + s];
      }
      for (int64_t q = 0; q < task.seg; ++q) {
        const float d = p.sums[(base + q) * p.D + c];
#pragma unroll
        for (int s = 0; s < NS; ++s)
          h[s] = __builtin_fmaf(__builtin_amdgcn_exp2f(d * A[s]), h[s], p.ends[(base + q) * all + mine + s]);
      }
    } else if (task.first) {
      const int64_t in = slot_in(p.state, task.n);
      if (in >= 0) {
#pragma unroll
        for (int s = 0; s < NS; ++s) h[s] = load_state(p.state, in + mine + s);
      }
      if (!OUT) {
#pragma unroll
        for (int s = 0; s < NS; ++s) p.starts[task.n * p.D * N + mine + s] = h[s];
        if (task.last) return;
      }
    }
  }
  if (!OUT && task.last) return;

  // ---- what this thread brings of each tile: four channels of a token, pieces of B and C
  const int tok = tid >> 3, quad = 4 * (tid & 7);
  const bool loads = c0 + quad < p.D;
  const int64_t nb = p.cu_seqlens ? 0 : task.n;
  const int64_t ub = nb * p.us[0] + task.row0 * p.us[1] + c0 + quad;
  const int64_t db = nb * p.ds[0] + task.row0 * p.ds[1] + c0 + quad;
  const int64_t zb = nb * p.zs[0] + task.row0 * p.zs[1] + c0 + quad;
  const int64_t group = c0 / p.per_group;
  const int64_t bb = nb * p.bs[0] + task.row0 * p.bs[1] + group * p.bs[2];
  const int64_t cb = nb * p.cs[0] + task.row0 * p.cs[1] + group * p.cs[2];
  const int64_t ob = (nb * p.T + task.row0) * p.D + c0 + quad;
  float bias[4], skip[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    bias[e] = loads && p.bias ? p.bias[c0 + quad + e] : 0.f;
    skip[e] = OUT && loads && p.skip ? p.skip[c0 + quad + e] : 0.f;
  }

  struct Raw {
    Raw4<BF16> u, d, z, b[kPer];
  };
  auto fetch = [&](int64_t t0, Raw& r) {
    const int64_t t = t0 + tok;
    if (loads && t < task.len) {
      r.u.load(p.u, ub + t * p.us[1]);
      r.d.load(p.delta, db + t * p.ds[1]);
      if (OUT && p.z) r.z.load(p.z, zb + t * p.zs[1]);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int j = tid + 256 * i;
      // piece j: the token's quads of B, then those of C
      const int row = j / (kQuads / kScanTile), q = j % (kQuads / kScanTile);
      const int64_t tt = t0 + row;
      if (j < kQuads && tt < task.len) {
        if (q < N / 4) r.b[i].load(p.B, bb + tt * p.bs[1] + 4 * q);
        else r.b[i].load(p.C, cb + tt * p.cs[1] + 4 * (q - N / 4));
      } else {
        r.b[i].clear();
      }
    }
  };
  auto prepare = [&](int64_t t0, const Raw& r, int buf) {
    const bool here = loads && t0 + tok < task.len;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float d = r.d[e] + bias[e];
      if (p.softplus) d = softplusf_(d);
      float x = d * r.u[e];
      if (!here) d = x = 0.f;
      f32x2 pair = {d, x};
      *reinterpret_cast<f32x2*>(&dx[buf][tok >> 1][quad + e][2 * (tok & 1)]) = pair;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int j = tid + 256 * i;
      const int row = j / (kQuads / kScanTile), q = j % (kQuads / kScanTile);
      if (j >= kQuads) continue;
      const int at = q < N / 4 ? 0 : NS, n0 = q < N / 4 ? 4 * q : 4 * q - N;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = r.b[i][e];
#pragma unroll
      for (int e = 0; e < 4; ++e) bc[buf][row][(n0 + e) / NS][at + (n0 + e) % NS] = v[e];
    }
  };
  // Eight tokens of a tile from t8 on (the last ones of a segment may be fewer).
  auto eight = [&](int buf, int t8, int count) {
    float y[8];
#pragma unroll
    for (int tp = 0; tp < 4; ++tp) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(&dx[buf][t8 / 2 + tp][8 * wave + ch][0]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = 2 * tp + j;
        const float d = v[2 * j], x = v[2 * j + 1];
        float r[kBC];
#pragma unroll
        for (int e = 0; e < kBC; ++e) r[e] = bc[buf][t8 + t][g][e];
        float acc = 0.f;
        if (t < count) {  // a token behind the end must not touch the state: 0 A may be NaN
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            const float a = __builtin_amdgcn_exp2f(d * A[s]);
            h[s] = __builtin_fmaf(a, h[s], x * r[s]);
            if constexpr (OUT) acc = s == 0 ? h[s] * r[NS] : __builtin_fmaf(h[s], r[NS + s], acc);
          }
          if constexpr (!OUT) sum += d;
        }
        y[t] = acc;
      }
    }
    if constexpr (OUT) ys[buf][t8 + g][8 * wave + ch] = reduce8(y);
  };
  auto finish = [&](int64_t t0, const Raw4<BF16>& u, const Raw4<BF16>& z, int buf) {
    if (!loads || t0 + tok >= task.len) return;
    const f32x4 y = *reinterpret_cast<const f32x4*>(&ys[buf][tok][quad]);
    f32x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[e] = p.skip ? __builtin_fmaf(skip[e], u[e], y[e]) : y[e];
      if (p.z) o[e] *= siluf_(z[e]);
    }
    store4<BF16>(p.out, ob + (t0 + tok) * p.D, o);
  };

  Raw raw[2];
  fetch(0, raw[0]);
  fetch(kScanTile, raw[1]);
  prepare(0, raw[0], 0);
  meet();
  auto tile = [&](int64_t t0, int buf) {
    Raw& r = raw[buf];
    const Raw4<BF16> u = r.u, z = r.z;
    fetch(t0 + 2 * kScanTile, r);
    const int64_t left = task.len - t0;
    if (left >= kScanTile) {
#pragma unroll
      for (int t8 = 0; t8 < kScanTile; t8 += 8) eight(buf, t8, 8);
    } else {
      for (int t8 = 0; t8 < left; t8 += 8) eight(buf, t8, left - t8 < 8 ? static_cast<int>(left) - t8 : 8);
    }
    prepare(t0 + kScanTile, raw[buf ^ 1], buf ^ 1);
    meet();
    if constexpr (OUT) finish(t0, u, z, buf);
  };
  for (int64_t t0 = 0; t0 < task.len; t0 += 2 * kScanTile) {
    tile(t0, 0);
    if (t0 + kScanTile < task.len) tile(t0 + kScanTile, 1);
  }

  if (!held) return;
  if constexpr (OUT) {
    const int64_t out = task.last ? slot_out(p.state, task.n) : -1;
    if (out >= 0) {
#pragma unroll
      for (int s = 0; s < NS; ++s) store_state(p.state, out + mine + s, h[s]);
    }
  } else {
#pragma unroll
    for (int s = 0; s < NS; ++s) p.ends[task.slot * p.D * N + mine + s] = h[s];
    if (g == 0) p.sums[task.slot * p.D + c] = sum;
  }
}

template <bool OUT, bool BF16>
hipError_t go(const ScanParams& p, int n, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(scan_grid(p))), block(256);
  switch (n) {
    case 8: hipLaunchKernelGGL((scan_kernel<BF16, 8, OUT>), grid, block, 0, stream, p); break;
    case 16: hipLaunchKernelGGL((scan_kernel<BF16, 16, OUT>), grid, block, 0, stream, p); break;
    case 32: hipLaunchKernelGGL((scan_kernel<BF16, 32, OUT>), grid, block, 0, stream, p); break;
    default: hipLaunchKernelGGL((scan_kernel<BF16, 64, OUT>), grid, block, 0, stream, p); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_scan_ends(const ScanParams& p, int n, bool io_bf16, hipStream_t stream) {
  return io_bf16 ? go<false, true>(p, n, stream) : go<false, false>(p, n, stream);
}

hipError_t launch_scan_outputs(const ScanParams& p, int n, bool io_bf16, hipStream_t stream) {
  return io_bf16 ? go<true, true>(p, n, stream) : go<true, false>(p, n, stream);
}

}  // namespace kda

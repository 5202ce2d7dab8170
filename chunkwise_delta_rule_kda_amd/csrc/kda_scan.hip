// The selective state space scan over prompts. For channel c and its n states,
//   h <- exp(d A) h + d u B ; y = sum C h + D u ; out = y z sigmoid(z)
// with d = softplus(delta + bias). The decay differs by channel and state and its sums over
// time by channel, so nothing of it is a matrix product: per (token, channel, state) it is two
// multiplications, an exponential and two fused multiply-adds of the vector units.
//
// A workgroup has 32 channels of one sequence (or of one time segment of it). Four waves hold
// the states of eight channels each: lane L has channel L % 8 and the n / 8 states of group
// L / 8, in registers for the whole run. Four others bring tiles of 32 tokens through LDS,
// twice buffered, with one barrier each: u, delta, z, B and C come from memory two tiles ahead,
// delta becomes d and d u, and the outputs of the tile before are finished.

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

constexpr int kYRow = kScanChannels + 8;      // floats of an LDS row of y, and of a pair of
constexpr int kDxRow = 4 * kScanChannels + 4; // tokens' step sizes: no two rows' banks meet

// A tile in LDS.
template <int N, bool OUT>
struct ScanTile {
  static constexpr int kBC = OUT ? N / 4 : N / 8;  // of B and C, for a lane and token
  float dx[kScanTile / 2][kDxRow];  // [channel][4]: d, d u of two tokens
  float bc[kScanTile][8][kBC];      // [group]: its B, then its C
  float y[OUT ? kScanTile : 1][kYRow];
};

// A lane's states, in the waves that hold them.
template <int N, bool OUT>
struct ScanStates {
  static constexpr int NS = N / 8;
  float A[NS], h[NS], sum;

  // What two tokens need from LDS.
  struct Pair {
    f32x4 dx;
    float bc[2][ScanTile<N, OUT>::kBC];
  };
  static __device__ __forceinline__ void load(const ScanTile<N, OUT>& tile, int column, int g, int pair, Pair& o) {
    o.dx = *reinterpret_cast<const f32x4*>(&tile.dx[pair][4 * column]);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < ScanTile<N, OUT>::kBC; ++e) o.bc[j][e] = tile.bc[2 * pair + j][g][e];
  }
  __device__ __forceinline__ float token(const Pair& o, int j) {
    const float d = o.dx[2 * j], x = o.dx[2 * j + 1];
    const float* r = o.bc[j];
    float y = 0.f;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const float a = __builtin_amdgcn_exp2f(d * A[s]);
      h[s] = __builtin_fmaf(a, h[s], x * r[s]);
      if constexpr (OUT) y = s == 0 ? h[s] * r[NS] : __builtin_fmaf(h[s], r[NS + s], y);
    }
    if constexpr (!OUT) sum += d;
    return y;
  }

  __device__ __forceinline__ void run(ScanTile<N, OUT>& tile, int column, int g, int64_t left) {
    constexpr int kPairs = kScanTile / 2;
    if (left >= kScanTile) {
      // LDS is read some tokens ahead; the compiler by itself would read just before the use
      constexpr int kAhead = NS <= 2 ? 4 : NS == 4 ? 2 : 1;
      Pair o[kPairs];
      float y[8];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) load(tile, column, g, i, o[i]);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        if (i + kAhead < kPairs) load(tile, column, g, i + kAhead, o[i + kAhead]);
        __builtin_amdgcn_sched_barrier(0x407);  // arithmetic may pass
        y[2 * i % 8] = token(o[i], 0);
        y[2 * i % 8 + 1] = token(o[i], 1);
        if constexpr (OUT) {
          if (i % 4 == 3) tile.y[2 * i - 6 + g][column] = reduce8(y);
        }
      }
      return;
    }
    // the last tokens of a segment: what is behind the end must not touch the state
    for (int t8 = 0; t8 < left; t8 += 8) {
      float y[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        Pair o;
        if (t8 + t < left) {
          load(tile, column, g, (t8 + t) / 2, o);
          y[t] = token(o, t & 1);
        } else {
          y[t] = 0.f;
        }
      }
      if constexpr (OUT) tile.y[t8 + g][column] = reduce8(y);
    }
  }
};

// The waves that bring the tiles and finish the outputs: a thread has four channels of a
// token, and pieces of four of B and C. Rows and channels behind the end are read as the last
// ones there are.
template <bool BF16, int N, bool OUT>
struct ScanLoader {
  static constexpr int kRow = N / 4 * (OUT ? 2 : 1);  // pieces of a token's B and C
  static constexpr int kPieces = kRow * kScanTile, kPer = (kPieces + 255) / 256;
  static constexpr int kElem = BF16 ? 2 : 4;
  const ScanParams& p;
  const int64_t len;
  const int tok, quad;
  const char *u, *delta, *z;  // the segment's first row and this workgroup's first channel
  char* out;
  const char* piece[kPer];
  int64_t piece_stride[kPer];
  int channel;                // of this thread's four, inside D
  bool held;
  float bias[4], skip[4];

  struct Raw {
    Raw4<BF16> u, d, z, b[kPer];
  };

  __device__ __forceinline__ ScanLoader(const ScanParams& params, const ScanTask& t, int tid)
      : p(params), len(t.len), tok(tid >> 3), quad(4 * (tid & 7)) {
    const int64_t c0 = static_cast<int64_t>(t.cblk) * kScanChannels;
    const int64_t n = p.cu_seqlens ? 0 : t.n;
    held = c0 + quad < p.D;
    channel = held ? quad : static_cast<int>(p.D - 4 - c0);
    u = static_cast<const char*>(p.u) + (n * p.us[0] + t.row0 * p.us[1] + c0) * kElem;
    delta = static_cast<const char*>(p.delta) + (n * p.ds[0] + t.row0 * p.ds[1] + c0) * kElem;
    z = static_cast<const char*>(p.z) + (n * p.zs[0] + t.row0 * p.zs[1] + c0) * kElem;
    out = static_cast<char*>(p.out) + ((n * p.T + t.row0) * p.D + c0) * kElem;
    const int64_t group = c0 / p.per_group;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int q = (tid + 256 * i) % kRow;
      const bool is_b = q < N / 4;
      const int64_t(&st)[3] = is_b ? p.bs : p.cs;
      piece_stride[i] = st[1] * kElem;
      piece[i] = static_cast<const char*>(is_b ? p.B : p.C) +
                 (n * st[0] + t.row0 * st[1] + group * st[2] + 4 * (is_b ? q : q - N / 4)) * kElem;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      bias[e] = p.bias ? p.bias[c0 + channel + e] : 0.f;
      skip[e] = OUT && p.skip ? p.skip[c0 + channel + e] : 0.f;
    }
  }

  // Tile from t0 on, where it has a token.
  __device__ __forceinline__ void fetch(int64_t t0, int tid, Raw& r) {
    if (t0 >= len) return;
    const int last = len - t0 < kScanTile ? static_cast<int>(len - t0) - 1 : kScanTile - 1;
    const uint32_t row = tok < last ? tok : last;
    r.u.load(u + t0 * p.us[1] * kElem, row * static_cast<uint32_t>(p.us[1]) + channel);
    r.d.load(delta + t0 * p.ds[1] * kElem, row * static_cast<uint32_t>(p.ds[1]) + channel);
    if (OUT && p.z) r.z.load(z + t0 * p.zs[1] * kElem, row * static_cast<uint32_t>(p.zs[1]) + channel);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int j = tid + 256 * i;
      if (kPieces % 256 && j >= kPieces) continue;
      const int of = j / kRow < last ? j / kRow : last;
      r.b[i].load(piece[i] + (t0 + of) * piece_stride[i], 0);
    }
  }

  __device__ __forceinline__ void prepare(int tid, const Raw& r, ScanTile<N, OUT>& tile) {
    constexpr int NS = N / 8;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float d = r.d[e] + bias[e];
      if (p.softplus) d = softplusf_(d);
      const f32x2 pair = {d, d * r.u[e]};
      *reinterpret_cast<f32x2*>(&tile.dx[tok >> 1][4 * (quad + e) + 2 * (tok & 1)]) = pair;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int j = tid + 256 * i;
      if (kPieces % 256 && j >= kPieces) continue;
      const int q = j % kRow;
      const int at = q < N / 4 ? 0 : NS, n0 = q < N / 4 ? 4 * q : 4 * q - N;
#pragma unroll
      for (int e = 0; e < 4; ++e) tile.bc[j / kRow][(n0 + e) / NS][at + (n0 + e) % NS] = r.b[i][e];
    }
  }

  __device__ __forceinline__ void finish(int64_t t0, const Raw4<BF16>& ru, const Raw4<BF16>& rz,
                                         const ScanTile<N, OUT>& tile) {
    const f32x4 y = *reinterpret_cast<const f32x4*>(&tile.y[OUT ? tok : 0][quad]);
    f32x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[e] = p.skip ? __builtin_fmaf(skip[e], ru[e], y[e]) : y[e];
      if (p.z) o[e] *= siluf_(rz[e]);
    }
    if (held && t0 + tok < len)
      store4<BF16>(out + t0 * p.D * kElem, static_cast<uint32_t>(tok) * static_cast<uint32_t>(p.D) + quad, o);
  }
};

// OUT: outputs from the true start state; otherwise a segment's end state from zero (the
// first segment's from the sequence's start) and the sum of its step sizes.
template <bool BF16, int N, bool OUT>
__global__ __launch_bounds__(512) void scan_kernel(ScanParams p) {
  constexpr int NS = N / 8;  // states of a lane
  __shared__ ScanTile<N, OUT> tiles[2];

  ScanTask task;
  if (!scan_task(p, task)) return;
  if (!OUT && task.last && !task.first) return;  // nobody starts from its end
  const int tid = threadIdx.x & 255;

  if (threadIdx.x >= 256) {
    // ---- the waves that load and finish
    using Loader = ScanLoader<BF16, N, OUT>;
    if (!OUT && task.last) return;
    Loader load(p, task, tid);
    typename Loader::Raw raw[2];
    load.fetch(0, tid, raw[0]);
    load.fetch(kScanTile, tid, raw[1]);
    Raw4<BF16> u[2], z[2];  // of the tile being scanned and of the one before
    u[0] = u[1] = raw[0].u;
    z[0] = z[1] = raw[0].z;
    load.prepare(tid, raw[0], tiles[0]);
    load.fetch(2 * kScanTile, tid, raw[0]);
    meet();
    auto step = [&](int64_t t0, int buf) {  // while the tile at t0 is scanned
      if (OUT && t0 > 0) load.finish(t0 - kScanTile, u[1], z[1], tiles[buf ^ 1]);
      u[1] = u[0];
      z[1] = z[0];
      if (t0 + kScanTile < task.len) {
        u[0] = raw[buf ^ 1].u;
        z[0] = raw[buf ^ 1].z;
        load.prepare(tid, raw[buf ^ 1], tiles[buf ^ 1]);
        load.fetch(t0 + 3 * kScanTile, tid, raw[buf ^ 1]);
      }
      meet();
    };
    int64_t t0 = 0;
    for (; t0 < task.len; t0 += 2 * kScanTile) {
      step(t0, 0);
      if (t0 + kScanTile < task.len) step(t0 + kScanTile, 1);
    }
    if (OUT && task.len > 0) {
      const int64_t tiles_done = (task.len + kScanTile - 1) / kScanTile;
      load.finish((tiles_done - 1) * kScanTile, u[1], z[1], tiles[(tiles_done - 1) & 1]);
    }
    return;
  }

  // ---- the waves that hold the states
  const int lane = tid & 63, ch = lane & 7, g = lane >> 3;
  const int column = 8 * (tid >> 6) + ch;
  const int64_t c = static_cast<int64_t>(task.cblk) * kScanChannels + column;
  const bool held = c < p.D;
  const int64_t mine = c * N + g * NS;  // in a slot
  ScanStates<N, OUT> st;
  st.sum = 0.f;
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    st.A[s] = held ? p.A[mine + s] * kLog2e : 0.f;
    st.h[s] = 0.f;
  }
  if (held && p.segmented && OUT) {
    // the start state, through the ends of the segments before
    const int64_t base = task.slot - task.seg, all = p.D * N;
    if (task.first) {
#pragma unroll
      for (int s = 0; s < NS; ++s) st.h[s] = p.starts[task.n * all + mine + s];
    }
    for (int64_t q = 0; q < task.seg; ++q) {
      const float d = p.sums[(base + q) * p.D + c];
#pragma unroll
      for (int s = 0; s < NS; ++s)
        st.h[s] = __builtin_fmaf(__builtin_amdgcn_exp2f(d * st.A[s]), st.h[s], p.ends[(base + q) * all + mine + s]);
    }
  } else if (held && task.first) {
    const int64_t in = slot_in(p.state, task.n);
    if (in >= 0) {
#pragma unroll
      for (int s = 0; s < NS; ++s) st.h[s] = load_state(p.state, in + mine + s);
    }
    if (!OUT) {
#pragma unroll
      for (int s = 0; s < NS; ++s) p.starts[task.n * p.D * N + mine + s] = st.h[s];
    }
  }
  if (!OUT && task.last) return;

  meet();
  for (int64_t t0 = 0; t0 < task.len; t0 += 2 * kScanTile) {
    st.run(tiles[0], column, g, task.len - t0);
    meet();
    if (t0 + kScanTile < task.len) {
      st.run(tiles[1], column, g, task.len - t0 - kScanTile);
      meet();
    }
  }

  if (!held) return;
  if constexpr (OUT) {
    const int64_t out = task.last ? slot_out(p.state, task.n) : -1;
    if (out >= 0) {
#pragma unroll
      for (int s = 0; s < NS; ++s) store_state(p.state, out + mine + s, st.h[s]);
    }
  } else {
#pragma unroll
    for (int s = 0; s < NS; ++s) p.ends[task.slot * p.D * N + mine + s] = st.h[s];
    if (g == 0) p.sums[task.slot * p.D + c] = st.sum;
  }
}

template <bool OUT, bool BF16>
hipError_t go(const ScanParams& p, int n, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(scan_grid(p))), block(512);
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

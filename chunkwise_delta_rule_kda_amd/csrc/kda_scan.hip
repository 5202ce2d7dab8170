// The selective state space scan over prompts. For channel c and its n states,
//   h <- exp(d A) h + d u B ; y = sum C h + D u ; out = y z sigmoid(z)
// with d = softplus(delta + bias). The decay differs by channel and state and its sums over
// time by channel, so nothing of it is a matrix product: per (token, channel, state) it is two
// multiplications, an exponential and two fused multiply-adds of the vector units.
//
// A workgroup has 32 channels of one sequence (or of one time segment of it). Four waves hold
// the states of eight channels each: lane L has channel L / 4 % 8 and the n / 8 states of
// group L % 4 + 4 (L / 32), in registers for the whole run. Four others bring tiles of 32 tokens through LDS,
// twice buffered, with one barrier each: u, delta, z, B and C come from memory two tiles ahead,
// delta becomes d and d u, and the outputs of the tile before are finished.
//
// Bound by the vector units: of 612 issue slots that a SIMD spends on a tile (N = 16) 397 are the
// recurrence, 68 the sums over the lanes, 146 the loaders'; 8 x 1024 x 4096 BF16 in 132 us, with
// the units busy all the time. 8192 x 8192 in one run, a workgroup on each compute unit: 318 us,
// 80 % busy. All waves in turn at loading and scanning took 542 there, LDS reads just before their
// use 364.

#include "kda_ssm_device.h"

namespace kda {

namespace {

struct ScanTask {
  int64_t n, slot, row0, len, seg;  // row0: token row of the segment's begin in its sequence's strides
  int64_t begin;                    // first row of the sequence (0 in the fixed layout)
  int cblk;
  bool first, last;
};

// The sequence of rank `rank` by decreasing length (in tiles); n at most 64, one for each lane.
__device__ __forceinline__ int by_length(const int64_t* cu, int n, int rank) {
  const int lane = threadIdx.x & 63;
  int64_t len = -1;
  if (lane < n) len = cu[lane + 1] - cu[lane];
  const int tiles = static_cast<int>((len + kScanTile - 1) / kScanTile);
  int mine = 0;
  for (int j = 0; j < n; ++j) {
    const int other = __builtin_amdgcn_readlane(tiles, j);
    mine += other > tiles || (other == tiles && j < lane);
  }
  return __builtin_ctzll(__ballot(lane < n && mine == rank));
}

// Workgroups b and b + 8 run on the same XCD one after the other: they get neighbouring
// channel blocks, whose 64-byte parts of a BF16 row share a cache line.
__device__ __forceinline__ bool scan_task(const ScanParams& p, ScanTask& t) {
  const uint32_t b = blockIdx.x;
  const uint32_t i = b >> 3;
  const uint32_t task = ((i >> 1) * 8 + (b & 7)) * 2 + (i & 1);
  const uint32_t w = task / static_cast<uint32_t>(p.cblocks);
  if (w >= p.slots) return false;
  t.cblk = static_cast<int>(task - w * static_cast<uint32_t>(p.cblocks));
  t.slot = w;
  int64_t total = p.T;
  if (p.cu_seqlens) {
    t.n = p.longest_first ? by_length(p.cu_seqlens, static_cast<int>(p.N), static_cast<int>(w))
                          : find_sequence(p.cu_seqlens, p.N, p.seg_len, w);
    t.begin = p.cu_seqlens[t.n];
    total = p.cu_seqlens[t.n + 1] - t.begin;
    t.seg = p.longest_first ? 0 : w - (divide(t.begin, p.seg_len) + t.n);
  } else {
    t.n = divide(w, p.segs_per_seq);
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

// Four consecutive elements as loaded, `at` bytes from base.
template <bool BF16>
struct Raw4 {
  uint32_t x[BF16 ? 2 : 4];
  __device__ __forceinline__ void load(const char* base, uint32_t at) {
    if constexpr (BF16) {
      const u32x2 w = *reinterpret_cast<const u32x2*>(base + at);
      x[0] = w[0];
      x[1] = w[1];
    } else {
      const u32x4 w = *reinterpret_cast<const u32x4*>(base + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = w[i];
    }
  }
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (BF16) return __uint_as_float(e % 2 ? x[e / 2] & 0xffff0000u : x[e / 2] << 16);
    else return __uint_as_float(x[e]);
  }
};

// x of the lanes of a quad that CTRL names, two bits for each of the four.
template <int CTRL>
__device__ __forceinline__ float quad_lanes(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true));
}

// Sums of eight tokens' values over the eight lanes of a channel, which differ in L % 4 and
// L / 32: lane L gets token L % 4 + 4 (L / 32)'s.
__device__ __forceinline__ float reduce8(const float (&v)[8]) {
  float a[4], b[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // lanes from 32 on: token i + 4
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[i]), __float_as_uint(v[i + 4]), false, false);
    a[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  const bool two = threadIdx.x & 2, odd = threadIdx.x & 1;
#pragma unroll
  for (int i = 0; i < 2; ++i)  // lanes 2 and 3 of the quad: token i + 2
    b[i] = (two ? a[i + 2] : a[i]) + quad_lanes<0x4E>(two ? a[i] : a[i + 2]);
  return (odd ? b[1] : b[0]) + quad_lanes<0xB1>(odd ? b[0] : b[1]);
}

// Floats of an LDS row of y, and of a pair of tokens' step sizes. What a wave writes is spread
// evenly over the banks. The two rows of step sizes that its quads read share 28 of their 32
// banks; rows of 164 floats, which share none, take the same time (8 x 1024 x 4096 131.7 us and
// 131.9, 8192 x 8192 317.8 and 317.7).
constexpr int kYRow = kScanChannels + 8;
constexpr int kDxRow = 4 * kScanChannels + 4;

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

  // LDS operands: of a token its row of B and C, of four tokens the step sizes and inputs. The
  // four lanes of a quad share their channel: each reads one of the four tokens', and the
  // products take them from their quad.
  static __device__ __forceinline__ void load_bc(const ScanTile<N, OUT>& tile, int g, int t, float (&r)[ScanTile<N, OUT>::kBC]) {
#pragma unroll
    for (int e = 0; e < ScanTile<N, OUT>::kBC; ++e) r[e] = tile.bc[t][g][e];
  }
  static __device__ __forceinline__ f32x2 load_dx(const ScanTile<N, OUT>& tile, int column, int t4) {
    const int t = t4 + (threadIdx.x & 3);
    return *reinterpret_cast<const f32x2*>(&tile.dx[t / 2][4 * column + 2 * (t & 1)]);
  }
  template <int J>
  __device__ __forceinline__ float token(f32x2 dx, const float (&r)[ScanTile<N, OUT>::kBC]) {
    float y = 0.f;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const float a = __builtin_amdgcn_exp2f(quad_lanes<0x55 * J>(dx[0]) * A[s]);
      h[s] = __builtin_fmaf(a, h[s], quad_lanes<0x55 * J>(dx[1]) * r[s]);
      if constexpr (OUT) y = s == 0 ? h[s] * r[NS] : __builtin_fmaf(h[s], r[NS + s], y);
    }
    if constexpr (!OUT) sum += quad_lanes<0x55 * J>(dx[0]);
    return y;
  }

  __device__ __forceinline__ void run(ScanTile<N, OUT>& tile, int column, int g, int64_t left) {
    if (left >= kScanTile) {
      // LDS is read ahead; the compiler by itself would read just before the use. 8192 x 8192:
      // four tokens ahead 324 us, two 318
      constexpr int kAhead = NS <= 4 ? 2 : 1;  // tokens
      float r[kScanTile][ScanTile<N, OUT>::kBC], y[8];
      f32x2 dx[kScanTile / 4];
      dx[0] = load_dx(tile, column, 0);
#pragma unroll
      for (int t = 0; t < kAhead; ++t) load_bc(tile, g, t, r[t]);
#pragma unroll
      for (int t4 = 0; t4 < kScanTile; t4 += 4) {
        if (t4 + 4 < kScanTile) dx[t4 / 4 + 1] = load_dx(tile, column, t4 + 4);
#pragma unroll
        for (int j = 0; j < 4; j += kAhead) {
          const int t = t4 + j;
#pragma unroll
          for (int i = t + kAhead; i < t + 2 * kAhead && i < kScanTile; ++i) load_bc(tile, g, i, r[i]);
          __builtin_amdgcn_sched_barrier(0);
          float* out = &y[t % 8];
          const f32x2 v = dx[t4 / 4];
          if constexpr (kAhead == 2) {
            out[0] = j == 0 ? token<0>(v, r[t]) : token<2>(v, r[t]);
            out[1] = j == 0 ? token<1>(v, r[t + 1]) : token<3>(v, r[t + 1]);
          } else {
            out[0] = j == 0 ? token<0>(v, r[t]) : j == 1 ? token<1>(v, r[t]) : j == 2 ? token<2>(v, r[t]) : token<3>(v, r[t]);
          }
        }
        if constexpr (OUT) {
          if (t4 % 8) tile.y[t4 - 4 + g][column] = reduce8(y);
        }
      }
      return;
    }
    // the last tokens of a segment: what is behind the end must not touch the state
    for (int t8 = 0; t8 < left; t8 += 8) {
      float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const int64_t more = left - t8 - i;
        float r[4][ScanTile<N, OUT>::kBC];
#pragma unroll
        for (int j = 0; j < 4; ++j) load_bc(tile, g, t8 + i + j, r[j]);
        const f32x2 dx = load_dx(tile, column, t8 + i);
        if (more > 0) y[i] = token<0>(dx, r[0]);
        if (more > 1) y[i + 1] = token<1>(dx, r[1]);
        if (more > 2) y[i + 2] = token<2>(dx, r[2]);
        if (more > 3) y[i + 3] = token<3>(dx, r[3]);
      }
      if constexpr (OUT) tile.y[t8 + g][column] = reduce8(y);
    }
  }
};

// The waves that bring the tiles and finish the outputs: a thread has four channels of a
// token, and pieces of four of B and C, those of B in the first waves. Rows and channels
// behind the end are read as the last ones there are: every tile then has the same number of
// loads, and the wait for one tile's leaves the next one's in flight.
template <bool BF16, int N, bool OUT>
struct ScanLoader {
  static constexpr int kOne = N / 4 * kScanTile;             // pieces of a tile's B
  static constexpr int kPieces = kOne * (OUT ? 2 : 1), kPer = (kPieces + 255) / 256;
  static constexpr uint32_t kElem = BF16 ? 2 : 4;
  const ScanParams& p;
  const int64_t len;
  const int tid, tok, quad;
  int64_t left;                // tokens from the next tile on, of the last tile at the end
  int64_t done = -kScanTile;   // the tile to finish: none is when the first one is scanned
  const char *u, *delta, *z;   // the next tile's first row and this workgroup's first channel
  char* out;                   // of the tile to finish
  const char* piece[kPer];
  int64_t piece_stride[kPer];  // bytes
  uint32_t u_at, delta_at, z_at, out_at, piece_at[kPer];  // this thread's part of a whole tile
  int64_t z_stride;
  int channel;                 // the first of this thread's four, inside D
  bool held;
  float bias[4], skip[4];

  struct Raw {
    Raw4<BF16> u, d, z, b[kPer];
  };

  __device__ __forceinline__ ScanLoader(const ScanParams& params, const ScanTask& t, int thread)
      : p(params), len(t.len), tid(thread), tok(thread >> 3), quad(4 * (thread & 7)), left(t.len) {
    const int64_t c0 = static_cast<int64_t>(t.cblk) * kScanChannels;
    const int64_t n = p.cu_seqlens ? 0 : t.n;
    held = c0 + quad < p.D;
    channel = held ? quad : static_cast<int>(p.D - 4 - c0);
    u = static_cast<const char*>(p.u) + (n * p.us[0] + t.row0 * p.us[1] + c0) * kElem;
    delta = static_cast<const char*>(p.delta) + (n * p.ds[0] + t.row0 * p.ds[1] + c0) * kElem;
    z = p.z ? static_cast<const char*>(p.z) + (n * p.zs[0] + t.row0 * p.zs[1] + c0) * kElem : u;
    z_stride = p.z ? p.zs[1] : p.us[1];
    out = static_cast<char*>(p.out) + ((n * p.T + t.row0 - kScanTile) * p.D + c0) * kElem;
    out_at = (static_cast<uint32_t>(tok) * static_cast<uint32_t>(p.D) + quad) * kElem;
    const int64_t group = divide(c0, p.per_group);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const bool is_b = !OUT || 256 * i + 64 * wave < kOne;
      const int64_t(&st)[3] = is_b ? p.bs : p.cs;
      piece_stride[i] = st[1] * kElem;
      piece[i] = static_cast<const char*>(is_b ? p.B : p.C) + (n * st[0] + t.row0 * st[1] + group * st[2]) * kElem;
    }
    places(kScanTile - 1);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      bias[e] = p.bias ? p.bias[c0 + channel + e] : 0.f;
      skip[e] = OUT && p.skip ? p.skip[c0 + channel + e] : 0.f;
    }
  }

  // Where this thread's parts of a tile are whose last row is `last`.
  __device__ __forceinline__ void places(int last) {
    const uint32_t row = tok < last ? tok : last;
    u_at = (row * static_cast<uint32_t>(p.us[1]) + channel) * kElem;
    delta_at = (row * static_cast<uint32_t>(p.ds[1]) + channel) * kElem;
    z_at = (row * static_cast<uint32_t>(z_stride) + channel) * kElem;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int j = (tid + 256 * i) % kOne;
      const uint32_t of = j / (N / 4) < last ? j / (N / 4) : last;
      piece_at[i] = of * static_cast<uint32_t>(piece_stride[i]) + 4 * (j % (N / 4)) * kElem;
    }
  }

  // The next tile, or the last one again.
  __device__ __forceinline__ void fetch(Raw& r) {
    if (left < kScanTile) places(static_cast<int>(left) - 1);
    r.u.load(u, u_at);
    r.d.load(delta, delta_at);
    if (OUT) r.z.load(z, z_at);
#pragma unroll
    for (int i = 0; i < kPer; ++i) r.b[i].load(piece[i], piece_at[i]);
    const int64_t rows = left > kScanTile ? kScanTile : 0;
    left -= rows;
    u += p.us[1] * rows * kElem;
    delta += p.ds[1] * rows * kElem;
    z += z_stride * rows * kElem;
#pragma unroll
    for (int i = 0; i < kPer; ++i) piece[i] += piece_stride[i] * rows;
  }

  __device__ __forceinline__ void prepare(const Raw& r, ScanTile<N, OUT>& tile) {
    constexpr int NS = N / 8;
    float d[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = r.d[e] + bias[e];
    if (p.softplus) {
#pragma unroll
      for (int e = 0; e < 4; ++e) d[e] = softplusf_(d[e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const f32x2 pair = {d[e], d[e] * r.u[e]};
      *reinterpret_cast<f32x2*>(&tile.dx[tok >> 1][4 * (quad + e) + 2 * (tok & 1)]) = pair;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (kPieces % 256 && tid + 256 * i >= kPieces) continue;
      const int j = (tid + 256 * i) % kOne, row = j / (N / 4), n0 = 4 * (j % (N / 4));
      const int at = tid + 256 * i < kOne ? 0 : NS;
      const Raw4<BF16>& v = r.b[i];
      if constexpr (NS == 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) tile.bc[row][n0 + e][at] = v[e];
      } else if constexpr (NS == 2) {
#pragma unroll
        for (int e = 0; e < 4; e += 2)
          *reinterpret_cast<f32x2*>(&tile.bc[row][(n0 + e) / 2][at]) = f32x2{v[e], v[e + 1]};
      } else {
        *reinterpret_cast<f32x4*>(&tile.bc[row][n0 / NS][at + n0 % NS]) = f32x4{v[0], v[1], v[2], v[3]};
      }
    }
  }

  // The outputs of the tile behind the one finished before.
  __device__ __forceinline__ void finish(const Raw4<BF16>& ru, const Raw4<BF16>& rz,
                                         const ScanTile<N, OUT>& tile) {
    f32x4 o = *reinterpret_cast<const f32x4*>(&tile.y[OUT ? tok : 0][quad]);
    if (p.skip) {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(skip[e], ru[e], o[e]);
    }
    if (p.z) {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] *= siluf_(rz[e]);
    }
    if (held && done >= 0 && done + tok < len) store4<BF16>(out + out_at, 0, o);
    done += kScanTile;
    out += p.D * (kScanTile * kElem);
  }
};

// OUT: outputs from the true start state; otherwise a segment's end state from zero (the
// first segment's from the sequence's start) and the sum of its step sizes.
template <bool BF16, int N, bool OUT>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(BF16 && N <= 16 ? 6 : 4))) void
scan_kernel(ScanParams p) {
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
    if (task.len == 0) {
      meet();
      return;
    }
    Loader load(p, task, tid);
    typename Loader::Raw raw[2];
    load.fetch(raw[0]);
    load.fetch(raw[1]);
    Raw4<BF16> u[2], z[2];  // of the tile to be scanned next and of the one before
    u[0] = u[1] = raw[0].u;
    z[0] = z[1] = raw[0].z;
    load.prepare(raw[0], tiles[0]);
    load.fetch(raw[0]);
    meet();
    auto step = [&](int buf) {  // while tiles[buf] is scanned
      if (OUT) load.finish(u[1], z[1], tiles[buf ^ 1]);
      u[1] = u[0];
      z[1] = z[0];
      u[0] = raw[buf ^ 1].u;
      z[0] = raw[buf ^ 1].z;
      load.prepare(raw[buf ^ 1], tiles[buf ^ 1]);
      load.fetch(raw[buf ^ 1]);
      meet();
    };
    for (int64_t t0 = 0; t0 < task.len; t0 += 2 * kScanTile) {
      step(0);
      if (t0 + kScanTile >= task.len) break;
      step(1);
    }
    if (OUT) load.finish(u[1], z[1], tiles[(task.len - 1) / kScanTile & 1]);
    return;
  }

  // ---- the waves that hold the states
  const int lane = tid & 63, ch = lane >> 2 & 7, g = (lane & 3) + 4 * (lane >> 5);
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
    constexpr int kBatch = NS <= 2 ? 8 : 2;  // read together: the chain through them is short
    for (int64_t q0 = 0; q0 < task.seg; q0 += kBatch) {
      float d[kBatch], e[kBatch][NS];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int64_t q = base + (q0 + i < task.seg ? q0 + i : task.seg - 1);
        d[i] = p.sums[q * p.D + c];
#pragma unroll
        for (int s = 0; s < NS; ++s) e[i][s] = p.ends[q * all + mine + s];
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (q0 + i >= task.seg) break;
#pragma unroll
        for (int s = 0; s < NS; ++s)
          st.h[s] = __builtin_fmaf(__builtin_amdgcn_exp2f(d[i] * st.A[s]), st.h[s], e[i][s]);
      }
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

// The chunked form of linear attention with one decay per head (device code).
//
// A chunk of C = 64 tokens that enters with the state S (V x K), with G_i the inclusive
// prefix sum of its log decays:
//   o_i = s exp(G_i) S q_i + s sum_{j <= i} exp(G_i - G_j) (q_i . k_j) v_j
//   S'  = exp(G_C) S + sum_j exp(G_C - G_j) v_j k_j^T
// Every exponent is a sum of log decays over some of the chunk's tokens, so no factor
// passes 1 where the decays do not. The prefix sums are kept in FP64: their differences
// are then exact to FP32 also behind a token that empties the state (-inf).
//
// One workgroup owns R = 64 NC value rows of one (segment, head) and walks its chunks with
// eight waves: four that load tiles and form the scores P, and four "state waves" that each
// own 16 NC of the rows with all keys, as MFMA accumulators S[key][value] in registers,
// FP32. Everything is computed transposed (values or keys as MFMA rows, tokens as columns),
// which lets the accumulators serve as operands without any exchange between lanes:
//   P^T tile (j, i)     = K . Q^T, scaled by its decays, through LDS to all waves
//   O^T tile (value, i) = S^T Q^T (scaled by s exp(G_i)) + V^T P^T
//   S tile (key, value) = exp(G_C) S + K^T (V exp(G_C - G_j))
// Two 16-key accumulator tiles hold keys 8 grp .. 8 grp + 7 of 32 in each lane (the K^T
// operand's rows are permuted so), which are those of a plain 16-byte read of Q. For the
// contractions over tokens both sides use the order
// kappa(kb, grp, e) = 32 kb + 16 (e / 4) + 4 grp + e % 4.
//
// LDS tiles are rows of 16-byte pieces, permuted within a row by an exclusive or with a
// number of the row's: one that differs over the 16 rows of a plain operand read, and in
// its upper bits over the four rows from which 16 lanes of a transposing read take 32 or
// 64 bytes each, so that both touch every bank alike. BF16 operands that need eight tokens
// of one column come from the transposing LDS read; FP32 ones (FP32 I/O) from 4-byte reads.
// Roundings to BF16 of BF16 calls: the state as the operand of S^T Q^T, the scores P and the
// decayed values (see scale_frag), each by at most 2^-8 of a term; sums stay in FP32.
#pragma once

#include "kda_device.h"
#include "kda_ops_internal.h"

namespace kda {

struct F32x8 {
  f32x4 lo, hi;
};

template <bool BF16>
struct FragOf {
  typedef bf16x8 type;
};
template <>
struct FragOf<false> {
  typedef F32x8 type;
};

// C += A B over 32 contraction indices, eight per lane on each side in the same order.
__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c) { return mfma32(a, b, c); }
__device__ __forceinline__ f32x4 mma(const F32x8& a, const F32x8& b, f32x4 c) {
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.lo[e], b.lo[e], c, 0, 0, 0);
#pragma unroll
  for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.hi[e], b.hi[e], c, 0, 0, 0);
  return c;
}

// Two products with one FP32 operand in common, a and b[0] / b[1]: their FP32 MFMAs in turn,
// since each waits for the one before it on the same accumulator.
__device__ __forceinline__ void mma_pair(const F32x8& a, const F32x8 (&b)[2], f32x4& c0, f32x4& c1) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    c0 = __builtin_amdgcn_mfma_f32_16x16x4f32(a.lo[e], b[0].lo[e], c0, 0, 0, 0);
    c1 = __builtin_amdgcn_mfma_f32_16x16x4f32(a.lo[e], b[1].lo[e], c1, 0, 0, 0);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    c0 = __builtin_amdgcn_mfma_f32_16x16x4f32(a.hi[e], b[0].hi[e], c0, 0, 0, 0);
    c1 = __builtin_amdgcn_mfma_f32_16x16x4f32(a.hi[e], b[1].hi[e], c1, 0, 0, 0);
  }
}

// Piece p of row r of a tile is stored at p ^ piece_swap(r).
template <int PPR>
__device__ __forceinline__ int piece_swap(int r) {
  static_assert(PPR == 8 || PPR == 16 || PPR == 32, "row sizes of 128, 256 or 512 bytes");
  const int q = (r >> 2) & 3, low = (((q ^ (q >> 1)) & 1) << 1) | (q >> 1);  // 0, 2, 3, 1
  return (PPR >= 16 ? (r & 3) << 2 : (r & 2) << 1) | low;
}
// Index (in 16-byte pieces) of piece p of row r in a tile of PPR pieces per row.
template <int PPR>
__device__ __forceinline__ int piece_at(int r, int p) {
  return r * PPR + (p ^ piece_swap<PPR>(r));
}

// Operand of row `row` (this lane's token) and its eight keys 32 kb + 8 grp ...
template <int PPR>
__device__ __forceinline__ void row_frag(const unsigned char* tile, int row, int kb, int grp,
                                         bf16x8& f) {
  f = *reinterpret_cast<const bf16x8*>(tile + 16 * piece_at<PPR>(row, 4 * kb + grp));
}
template <int PPR>
__device__ __forceinline__ void row_frag(const unsigned char* tile, int row, int kb, int grp,
                                         F32x8& f) {
  f.lo = *reinterpret_cast<const f32x4*>(tile + 16 * piece_at<PPR>(row, 8 * kb + 2 * grp));
  f.hi = *reinterpret_cast<const f32x4*>(tile + 16 * piece_at<PPR>(row, 8 * kb + 2 * grp + 1));
}

// Operand of one column and the eight tokens kappa(kb, grp, e). Lane m of 16 gets column
// base + step * (m / 4) + m % 4: the transposing read takes four consecutive elements
// from each of 16 lanes (lane i: row i / 4, column quad i % 4) and gives lane i element
// i % 4 of quad i / 4 in all four rows.
template <int PPR>
__device__ __forceinline__ void col_frag(const unsigned char* tile, int base, int step, int kb,
                                         int grp, int m, bf16x8& f) {
  typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
  const int row = 32 * kb + 4 * grp + (m >> 2);
  const int col = base + step * (m & 3);
  const unsigned char* a = tile + 16 * piece_at<PPR>(row, col >> 3) + 2 * (col & 7);
  const unsigned char* b = tile + 16 * piece_at<PPR>(row + 16, col >> 3) + 2 * (col & 7);
  i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)a);
  i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)b);
  f = __builtin_shufflevector(__builtin_bit_cast(bf16x4, lo), __builtin_bit_cast(bf16x4, hi),
                              0, 1, 2, 3, 4, 5, 6, 7);
}
template <int PPR>
__device__ __forceinline__ void col_frag(const unsigned char* tile, int base, int step, int kb,
                                         int grp, int m, F32x8& f) {
  const int col = base + step * (m >> 2) + (m & 3);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int row = 32 * kb + 4 * grp + e;
    f.lo[e] = *reinterpret_cast<const float*>(tile + 16 * piece_at<PPR>(row, col >> 2) + 4 * (col & 3));
    f.hi[e] = *reinterpret_cast<const float*>(tile + 16 * piece_at<PPR>(row + 16, col >> 2) + 4 * (col & 3));
  }
}

// x scaled by one factor per token, as PARTS BF16 numbers: the product rounded, then twice
// what the rounding left. One part (off by at most 2^-8 of a term) goes into BF16 states, whose
// own rounding is as large; three (2^-24, FP32's own) into FP32 states, whose updates are then
// products of BF16 keys and FP32 numbers. Two parts left FP32 states 2.2e-6 off over 2000
// tokens, three 1.1e-7 (as FP32 arithmetic does), for 6 % of the call's time.
template <int PARTS>
__device__ __forceinline__ void scale_frag(bf16x8 x, f32x4 wlo, f32x4 whi, bf16x8 (&f)[PARTS]) {
  f32x4 lo, hi;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    lo[e] = static_cast<float>(x[e]) * wlo[e];
    hi[e] = static_cast<float>(x[4 + e]) * whi[e];
  }
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    f[i] = pack8(lo, hi);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      lo[e] -= static_cast<float>(f[i][e]);
      hi[e] -= static_cast<float>(f[i][4 + e]);
    }
  }
}

// The decay factors of one chunk, in LDS, by its four 16-token blocks.
struct Gates {
  double L[kLinChunk];  // sums of the log2 decays from the start of the token's block to it
  float a[kLinChunk];   // s * decay from the start of the block to the token
  float b[kLinChunk];   // decay from the token to the end of the block; 0 behind the end
  float E[4];           // total decay of each block
};

constexpr double kLog2e = 1.4426950408889634074;

template <int CTRL>
__device__ __forceinline__ double dpp_shift(double x) {
  const u32x2 w = __builtin_bit_cast(u32x2, x);
  u32x2 r;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    r[i] = static_cast<unsigned>(__builtin_amdgcn_update_dpp(0, static_cast<int>(w[i]), CTRL, 0xF, 0xF, true));
  return __builtin_bit_cast(double, r);
}

__device__ __forceinline__ double read_lane(double x, int lane) {
  const u32x2 w = __builtin_bit_cast(u32x2, x);
  u32x2 r;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    r[i] = static_cast<unsigned>(__builtin_amdgcn_readlane(static_cast<int>(w[i]), lane));
  return __builtin_bit_cast(double, r);
}

__device__ __forceinline__ float exp2_of(double x) {
  return __builtin_amdgcn_exp2f(static_cast<float>(x));
}

// The log decay of a token as it is in memory: the g of head h at token row `row`.
__device__ __forceinline__ float load_log_decay(const LinParams& p, int64_t row, int h) {
  if (!p.g) return 0.f;
  const int64_t at = row * p.H + h;
  return p.g_bf16 ? load1<true>(p.g, at) : load1<false>(p.g, at);
}

// One wave makes the factors of block `blk`: every row of 16 lanes holds its 16 tokens, x
// their log decays, `held` whether the token exists. The prefix sums are FP64, so that
// their differences are exact to FP32 whatever the decays before the two tokens are.
struct BlockGates {
  double L;
  float a, b, e;
  __device__ __forceinline__ void make(float x, float fixed, bool held, float scale) {
    double y = static_cast<double>(x) + static_cast<double>(fixed);
    // -inf (an emptied state) as a finite number whose factor is 0; NaN stays
    y = (y < -1000.0 ? -1000.0 : y) * kLog2e;
    y = held ? y : 0.0;
    y += dpp_shift<0x111>(y);  // row_shr 1, 2, 4, 8
    y += dpp_shift<0x112>(y);
    y += dpp_shift<0x114>(y);
    y += dpp_shift<0x118>(y);
    const double total = read_lane(y, 15);
    L = y;
    a = scale * exp2_of(y);
    b = held ? exp2_of(total - y) : 0.f;
    e = exp2_of(total);
  }
  __device__ __forceinline__ void write(Gates& gt, int blk, int lane) const {
    if (lane < 16) {
      gt.L[16 * blk + lane] = L;
      gt.a[16 * blk + lane] = a;
      gt.b[16 * blk + lane] = b;
      if (lane == 0) gt.E[blk] = e;
    }
  }
};
__device__ __forceinline__ void make_gates(Gates& gt, float x, float fixed, int blk, int lane, bool held,
                                           float scale) {
  BlockGates g;
  g.make(x, fixed, held, scale);
  g.write(gt, blk, lane);
}

// Decays of whole blocks of a chunk: before a block, behind it, and of all four.
struct BlockDecays {
  float before[4], behind[4], all;
};
__device__ __forceinline__ BlockDecays block_decays(const Gates& gt) {
  const f32x4 E = *reinterpret_cast<const f32x4*>(gt.E);
  BlockDecays r;
  r.before[0] = 1.f;
  r.before[1] = E[0];
  r.before[2] = E[0] * E[1];
  r.before[3] = r.before[2] * E[2];
  r.behind[3] = 1.f;
  r.behind[2] = E[3];
  r.behind[1] = E[3] * E[2];
  r.behind[0] = r.behind[1] * E[1];
  r.all = r.before[3] * E[3];
  return r;
}

// A tile of 64 rows x PPR pieces between memory and LDS, held in registers in between:
// rows behind the sequence's end read as zeros (buffer loads past num_records).
template <int PPR>
struct Tile {
  static constexpr int kPieces = 64 * PPR / 256;
  u32x4 x[kPieces];
  // base: the chunk's first row; pitch: bytes between rows; left: rows of the sequence
  __device__ __forceinline__ void load(const unsigned char* base, uint32_t pitch, int left, int tid) {
    const int rows = left < 64 ? left : 64;
    const uint32_t bytes = static_cast<uint32_t>(rows - 1) * pitch + PPR * 16;
    __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<unsigned char*>(base), 0, bytes, 0x00020000);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int at = tid + 256 * i;
      const int off = static_cast<int>(static_cast<uint32_t>(at / PPR) * pitch + (at % PPR) * 16);
      x[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
    }
  }
  __device__ __forceinline__ void store(unsigned char* tile, int tid) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int at = tid + 256 * i;
      *reinterpret_cast<u32x4*>(tile + 16 * piece_at<PPR>(at / PPR, at % PPR)) = x[i];
    }
  }
};

// A tile of 64 rows x PPR pieces from memory straight into LDS (asynchronous 16-byte loads,
// one KB of consecutive LDS for each instruction of a wave), 64 PPR / 256 instructions per
// wave. The lanes fetch the pieces in the order in which the tile stores them. Rows behind
// the sequence's end repeat its last row: their keys and values meet a zero factor, their
// queries' outputs are not stored.
template <int PPR>
struct AsyncTile {
  static constexpr int kLoads = PPR / 4;  // instructions per wave
  int off[kLoads];
  static __device__ __forceinline__ int offset(int wave, int lane, int j, uint32_t pitch, int last) {
    const int at = (wave * kLoads + j) * 64 + lane;
    const int r = at / PPR;
    const int piece = (at % PPR) ^ piece_swap<PPR>(r);
    return static_cast<int>(static_cast<uint32_t>(r < last ? r : last) * pitch) + 16 * piece;
  }
  __device__ __forceinline__ void init(int wave, int lane, uint32_t pitch) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) off[j] = offset(wave, lane, j, pitch, 63);
  }
  // base: the chunk's first row; left: rows of the sequence from there on
  __device__ __forceinline__ void load(const unsigned char* base, uint32_t pitch, int left,
                                       unsigned char* tile, int wave, int lane) const {
    typedef __attribute__((address_space(3))) void lds_void;
    const int rows = left < 64 ? left : 64;
    const uint32_t bytes = static_cast<uint32_t>(rows - 1) * pitch + PPR * 16;
    __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<unsigned char*>(base), 0, bytes, 0x00020000);
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int o = rows == 64 ? off[j] : offset(wave, lane, j, pitch, rows - 1);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(tile + (wave * kLoads + j) * 1024), 16, o,
                                               0, 0, 0);
    }
  }
};

// All but the `N` newest of the wave's memory operations are done (operations complete in
// issue order), its LDS accesses too; then the workgroup's barrier. The tiles that every
// wave has waited for are whole behind it.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// The workgroup's barrier alone: the wave's LDS accesses are done, its memory operations may
// be outstanding.
__device__ __forceinline__ void meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// What a workgroup works on: false where it has nothing to do.
struct LinTask {
  int64_t tok0;     // first token row of the segment
  int64_t len;      // tokens of the segment
  int64_t n;        // sequence
  int64_t slot;     // scan slot
  int h, vblk;
  bool first, last; // segment of its sequence
};

__device__ __forceinline__ bool find_task(const LinParams& p, LinTask& t) {
  // Workgroup b runs on XCD b % 8. A task, one head of one slot, has its value blocks on one
  // XCD, whose L2 then reads q and k once.
  const int64_t b = blockIdx.x;
  const int xcd = static_cast<int>(b & 7);
  int64_t i = b >> 3;
  t.vblk = static_cast<int>(i % p.vblocks);
  i /= p.vblocks;
  const int64_t task = i * 8 + xcd;
  const int64_t w = task / p.H;
  if (w >= p.slots) return false;
  t.h = static_cast<int>(task % p.H);
  t.slot = w;
  int64_t begin, end, seg;
  if (p.longest_first) {
    // one lane per sequence (at most 64): w is its rank by decreasing length
    const int lane = threadIdx.x & 63, N = static_cast<int>(p.N);
    int64_t from = 0, len = -1;
    if (lane < N) {
      from = p.cu_seqlens[lane];
      len = p.cu_seqlens[lane + 1] - from;
    }
    const int chunks = static_cast<int>((len + 63) >> 6);
    int rank = 0;
    for (int j = 0; j < N; ++j) {
      const int other = __builtin_amdgcn_readlane(chunks, j);
      rank += other > chunks || (other == chunks && j < lane);
    }
    const uint64_t mine = __ballot(lane < N && rank == static_cast<int>(w));
    const int n = __builtin_ctzll(mine);
    t.n = n;
    begin = p.cu_seqlens[n];
    end = p.cu_seqlens[n + 1];
    seg = 0;
  } else if (p.cu_seqlens) {
    // the last n with cu[n] / seg_len + n <= w, 64 candidates at a time
    const int lane = threadIdx.x & 63;
    int64_t lo = 0, size = p.N;
    while (size > 1) {
      const int64_t step = (size + 63) / 64;
      const int64_t at = lo + lane * step;
      const bool ok = lane * step < size && p.cu_seqlens[at] / p.seg_len + at <= w;
      const int c = __popcll(__ballot(ok));
      const int64_t skip = (c > 0 ? c - 1 : 0) * step;
      lo += skip;
      size = size - skip < step ? size - skip : step;
    }
    t.n = lo;
    begin = p.cu_seqlens[lo];
    end = p.cu_seqlens[lo + 1];
    seg = w - (begin / p.seg_len + lo);
  } else {
    t.n = w / p.segs_per_seq;
    seg = w - t.n * p.segs_per_seq;
    begin = t.n * p.T;
    end = begin + p.T;
  }
  const int64_t total = end - begin;
  const int64_t at = seg * p.seg_len;
  t.first = seg == 0;
  if (seg < 0 || (seg > 0 && at >= total)) return false;
  t.tok0 = begin + at;
  t.len = total - at < p.seg_len ? total - at : p.seg_len;
  t.last = at + t.len >= total;
  return true;
}

// Element offset of token row r (n * T + t, or a packed row) in a strided input.
__device__ __forceinline__ int64_t row_offset(const LinParams& p, const int64_t (&st)[3], int64_t n,
                                              int64_t row) {
  if (p.cu_seqlens) return row * st[1];
  return n * st[0] + (row - n * p.T) * st[1];
}

// S[t][c]: keys 32 (t / 2) + 8 grp + 4 (t % 2) + j of the value row of column m.
template <int KT, int NC>
__device__ __forceinline__ void load_state(f32x4 (&S)[KT][NC], const void* base, int64_t at, bool bf16,
                                           int K, int row0, int grp, int m) {
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t row = at + static_cast<int64_t>(row0 + 4 * NC * (m >> 2) + 4 * c + (m & 3)) * K;
#pragma unroll
    for (int t = 0; t < KT; t += 2) {
      float x[8];
      if (bf16) load8<true>(base, row + 16 * t + 8 * grp, x);
      else load8<false>(base, row + 16 * t + 8 * grp, x);
      S[t][c] = f32x4{x[0], x[1], x[2], x[3]};
      S[t + 1][c] = f32x4{x[4], x[5], x[6], x[7]};
    }
  }
}

template <int KT, int NC>
__device__ __forceinline__ void store_state(const f32x4 (&S)[KT][NC], void* base, int64_t at, bool bf16,
                                            int K, int row0, int grp, int m) {
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t row = at + static_cast<int64_t>(row0 + 4 * NC * (m >> 2) + 4 * c + (m & 3)) * K;
#pragma unroll
    for (int t = 0; t < KT; t += 2) {
      const int64_t idx = row + 16 * t + 8 * grp;
      const f32x4 x = S[t][c], y = S[t + 1][c];
      if (bf16) {
        *reinterpret_cast<bf16x8*>(static_cast<unsigned short*>(base) + idx) = pack8(x, y);
      } else {
        f32x4* q = reinterpret_cast<f32x4*>(static_cast<float*>(base) + idx);
        q[0] = x;
        q[1] = y;
      }
    }
  }
}

// The state a workgroup starts from: the scan's, or the sequence's own; and where the last
// segment's goes.
struct StateAt {
  const void* base;  // null: zeros (nothing is written)
  int64_t at;        // element of the head's first value row
  bool bf16;
};
__device__ __forceinline__ StateAt start_state(const LinParams& p, const LinTask& task, int K) {
  if (p.segmented && !(task.first && task.last))
    return {p.scan_s, (static_cast<int64_t>(task.h) * p.slots + task.slot) * p.V * K, false};
  const int64_t slot = p.in_idx ? p.in_idx[task.n] : task.n;
  const bool held = p.state_in && slot >= 0 && slot < p.pool_slots;
  return {held ? p.state_in : nullptr, slot * p.slot_pitch + static_cast<int64_t>(task.h) * p.V * K,
          p.st_bf16 != 0};
}
__device__ __forceinline__ StateAt end_state(const LinParams& p, const LinTask& task, int K) {
  if (!task.last || !p.state_out) return {nullptr, 0, false};
  const int64_t slot = p.out_idx ? p.out_idx[task.n] : task.n;
  const bool held = slot >= 0 && slot < p.pool_slots;
  return {held ? p.state_out : nullptr, slot * p.slot_pitch + static_cast<int64_t>(task.h) * p.V * K,
          p.st_bf16 != 0};
}

// The decays of a lane's tokens kappa(kb, grp, e) to the end of the chunk.
struct KeyDecays {
  f32x4 w[2][2];
  __device__ __forceinline__ void read(const Gates& gt, const BlockDecays& bd, int grp) {
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        w[kb][i] = bd.behind[2 * kb + i] * *reinterpret_cast<const f32x4*>(&gt.b[32 * kb + 16 * i + 4 * grp]);
  }
};

// FP32 I/O. Key tile t of the state, rows r: key 64 (t / 4) + 4 r + t % 4, so that a 16-byte
// read of four keys of a token is an operand of four tiles (4-byte reads of single keys were
// four times as many). A lane's S[t][j] is key 64 (t / 4) + 16 grp + 4 j + t % 4.
template <int KT>
__device__ __forceinline__ f32x4 keys_of(const f32x4 (&S)[KT], int h, int j) {
  return f32x4{S[4 * h][j], S[4 * h + 1][j], S[4 * h + 2][j], S[4 * h + 3][j]};
}
template <int KT>
__device__ __forceinline__ void load_state_f32(f32x4 (&S)[KT], const void* base, int64_t at, bool bf16,
                                               int row, int grp) {
#pragma unroll
  for (int h = 0; h < KT / 4; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t idx = at + static_cast<int64_t>(row) * 16 * KT + 64 * h + 16 * grp + 4 * j;
      const f32x4 x = bf16 ? load4<true>(base, idx) : load4<false>(base, idx);
#pragma unroll
      for (int t = 0; t < 4; ++t) S[4 * h + t][j] = x[t];
    }
}
template <int KT>
__device__ __forceinline__ void store_state_f32(const f32x4 (&S)[KT], void* base, int64_t at, bool bf16,
                                                int row, int grp) {
#pragma unroll
  for (int h = 0; h < KT / 4; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t idx = at + static_cast<int64_t>(row) * 16 * KT + 64 * h + 16 * grp + 4 * j;
      if (bf16) store4<true>(base, idx, keys_of(S, h, j));
      else store4<false>(base, idx, keys_of(S, h, j));
    }
}

// S <- D S + K^T (V w) for one chunk; vf: the wave's V operands, w a token's decay to the end
// of the chunk.
template <int KD>
__device__ __forceinline__ void update_state_f32(f32x4 (&S)[KD / 16], const F32x8 (&vf)[2],
                                                 const unsigned char* k_tile, const Gates& gt,
                                                 const BlockDecays& bd, int grp, int m) {
  constexpr int kPpr = KD / 4, KH = KD / 64;
  KeyDecays kd;
  kd.read(gt, bd, grp);
#pragma unroll
  for (int t = 0; t < KD / 16; ++t) S[t] *= bd.all;
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // 16 tokens: a lane's 16 i + 4 grp + e
    const f32x4 v = i % 2 ? vf[i / 2].hi : vf[i / 2].lo;
    const f32x4 vw = v * kd.w[i / 2][i % 2];
    f32x4 k[4][KH];
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int h = 0; h < KH; ++h)
        k[e][h] = *reinterpret_cast<const f32x4*>(k_tile + 16 * piece_at<kPpr>(16 * i + 4 * grp + e, 16 * h + m));
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int t = 0; t < KD / 16; ++t)
        S[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(k[e][t / 4][t % 4], vw[e], S[t], 0, 0, 0);
    // reads of the next tokens beside these products, not of all
    if (i % 2) __builtin_amdgcn_sched_barrier(0);
  }
}

}  // namespace kda

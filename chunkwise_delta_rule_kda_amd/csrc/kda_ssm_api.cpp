// Host side of the short causal convolution and the selective state space scan
// (include/kda.h): argument checks, launch geometry and the extern "C" entry points. No
// allocation, no device synchronisation, no state kept between calls.

#include <hip/hip_runtime.h>

#include <cmath>

#include "kda.h"
#include "kda_checks.h"
#include "kda_ssm_internal.h"

namespace {

// ------------------------------------------------------------ sequences and their states

kda_status sequences_shape(int64_t B, int64_t T, int64_t N, const int64_t* cu_seqlens) {
  if (B < 1 || B > (int64_t(1) << 31) || T < 0 || T > (int64_t(1) << 36) || N < 0 ||
      N > (int64_t(1) << 31))
    return fail(KDA_ERR_SHAPE, "bad B=%lld T=%lld N=%lld", (long long)B, (long long)T, (long long)N);
  if (cu_seqlens) {
    if (B != 1) return fail(KDA_ERR_SHAPE, "packed varlen needs B=1 (got %lld)", (long long)B);
    if (N < 1) return fail(KDA_ERR_SHAPE, "packed varlen needs N>=1");
  } else if (N != B) {
    return fail(KDA_ERR_SHAPE, "fixed layout needs N == B (N=%lld, B=%lld)", (long long)N, (long long)B);
  }
  return KDA_OK;
}

// Strides of `name`: `n` of them, the second one the token's.
kda_status strides_shape(const int64_t* st, int n, const char* name) {
  for (int d = 0; d < n; ++d)
    if (st[d] < 0 || st[d] > kBig || st[d] % 8)
      return fail(KDA_ERR_SHAPE, "%s stride %lld is negative or not a multiple of 8", name, (long long)st[d]);
  if (st[1] > (int64_t(1) << 22))  // a tile's rows stay within 2^31 bytes
    return fail(KDA_ERR_SHAPE, "%s token stride %lld exceeds 2^22", name, (long long)st[1]);
  return KDA_OK;
}

// The state arguments that both operators have; dense: elements of a sequence's state.
template <typename Args>
kda_status state_shape(const Args* a, int64_t dense) {
  if (!known_dtype(a->io_dtype)) return fail(KDA_ERR_DTYPE, "io_dtype %d", a->io_dtype);
  if (!known_dtype(a->state_dtype)) return fail(KDA_ERR_DTYPE, "state_dtype %d", a->state_dtype);
  if (a->ssm_state_indices) {
    if (!a->state_in) return fail(KDA_ERR_CONFIG, "a state pool needs state_in");
    if (a->state_pool_slots < 1 || a->state_pool_slots > (int64_t(1) << 31))
      return fail(KDA_ERR_CONFIG, "state_pool_slots %lld", (long long)a->state_pool_slots);
    if (a->state_slot_pitch != 0 &&
        (a->state_slot_pitch < dense || a->state_slot_pitch % 8 || a->state_slot_pitch > kBig))
      return fail(KDA_ERR_CONFIG, "state_slot_pitch %lld", (long long)a->state_slot_pitch);
    if (a->state_out && a->state_out != a->state_in)
      return fail(KDA_ERR_ALIAS, "with a state pool, state_out must be NULL or state_in");
  } else if (a->state_out_indices) {
    return fail(KDA_ERR_CONFIG, "state_out_indices needs ssm_state_indices");
  }
  return KDA_OK;
}

template <typename Args>
Wide state_bytes(const Args* a, int64_t dense) {
  const Wide es = elem_size(a->state_dtype);
  if (!a->ssm_state_indices) return static_cast<Wide>(a->N) * dense * es;
  const int64_t pitch = a->state_slot_pitch ? a->state_slot_pitch : dense;
  return (static_cast<Wide>(a->state_pool_slots - 1) * pitch + dense) * es;
}

template <typename Args>
kda::StateSlots state_slots(const Args* a, int64_t dense) {
  kda::StateSlots s{};
  s.in = a->state_in;
  s.out = a->state_out;
  s.slots = a->N;
  s.pitch = dense;
  s.bf16 = a->state_dtype == KDA_BF16;
  if (a->ssm_state_indices) {
    s.in_idx = a->ssm_state_indices;
    s.out_idx = a->state_out_indices ? a->state_out_indices : a->ssm_state_indices;
    s.slots = a->state_pool_slots;
    if (a->state_slot_pitch) s.pitch = a->state_slot_pitch;
    s.out = const_cast<void*>(a->state_in);  // the pool is updated in place
  }
  return s;
}

// Bytes from the first to behind the last element of [B, T, heads, dim] by its strides.
Wide strided_bytes(int64_t B, int64_t T, const int64_t* st, int64_t heads, int64_t head_stride,
                   int64_t dim, int64_t es) {
  if (T == 0) return 0;
  return (static_cast<Wide>(B - 1) * st[0] + static_cast<Wide>(T - 1) * st[1] +
          static_cast<Wide>(heads - 1) * head_stride + dim) * es;
}

// outs[1] is the written state, ins[state] the read one: those two may be the same memory.
template <int OUTS, int INS>
kda_status no_overlap(const Range (&outs)[OUTS], const Range (&ins)[INS], int state) {
  for (int i = 0; i < OUTS; ++i) {
    for (int j = 0; j < INS; ++j) {
      const bool same_state = i == 1 && j == state && outs[1].lo == ins[j].lo;
      if (!same_state && overlap(outs[i], ins[j]))
        return fail(KDA_ERR_ALIAS, "%s overlaps %s", outs[i].name, ins[j].name);
    }
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j]))
        return fail(KDA_ERR_ALIAS, "%s overlaps %s", outs[i].name, outs[j].name);
  }
  return KDA_OK;
}

// ------------------------------------------------------------ short convolution

struct ConvPlan {
  int64_t run, runs_per_seq, slots;
  int lanes;
};

ConvPlan conv_plan(const kda_short_conv_args* a) {
  ConvPlan pl{};
  // Tokens of a thread: longer runs read fewer rows twice, shorter ones keep what is in flight
  // closer together. BF16, 8192 rows, 8 and 16 tokens: 2304 channels 21.4 and 20.0 us, 9216 59.9
  // and 60.7, 36864 216 and 225 (32 tokens: 239); FP32, 2304 channels: 32.3 and 35.5.
  const bool few = a->io_dtype == KDA_BF16 && static_cast<Wide>(a->B) * a->T * a->C <= 64000000;
  pl.run = a->T <= 1 && !a->cu_seqlens ? 1 : few ? 16 : 8;
  pl.runs_per_seq = a->T > 0 ? ceil_div(a->T, pl.run) : 1;
  pl.slots = a->cu_seqlens ? a->T / pl.run + a->N : a->N * pl.runs_per_seq;
  // as many octets side by side as leave at most an eighth of the lanes idle
  const int64_t octets = a->C / 8;
  pl.lanes = 64;
  while (pl.lanes > 8 && ceil_div(octets, pl.lanes) * pl.lanes * 8 > octets * 9) pl.lanes = pl.lanes == 64 ? 32 : 8;
  return pl;
}

// Workgroups of the launch.
Wide conv_grid(const kda_short_conv_args* a, const ConvPlan& pl) {
  return static_cast<Wide>(ceil_div(a->C / 8, pl.lanes)) * ceil_div(pl.slots, 256 / pl.lanes);
}

kda_status conv_check(const kda_short_conv_args* a, ConvPlan* pl) {
  if (!a) return fail(KDA_ERR_NULL, "args is NULL");
  kda_status s = sequences_shape(a->B, a->T, a->N, a->cu_seqlens);
  if (s != KDA_OK) return s;
  if (a->C < 8 || a->C > (1 << 22) || a->C % 8)
    return fail(KDA_ERR_SHAPE, "C=%lld is not a multiple of 8 up to 2^22", (long long)a->C);
  if (a->W < 2 || a->W > 4) return fail(KDA_ERR_SHAPE, "W=%lld, 2 to 4 taps are supported", (long long)a->W);
  if (a->flags & ~KDA_CONV_SILU) return fail(KDA_ERR_FLAGS, "unknown flags 0x%x", a->flags);
  const int64_t dense = (a->W - 1) * a->C;
  s = state_shape(a, dense);
  if (s == KDA_OK) s = strides_shape(a->x_stride, 2, "x");
  if (s != KDA_OK) return s;
  const Wide rows = static_cast<Wide>(a->B) * a->T;
  if (rows * a->C > (Wide(1) << 50) || static_cast<Wide>(a->N) * dense > (Wide(1) << 50))
    return fail(KDA_ERR_SHAPE, "B*T*C or N*C is out of range");
  *pl = conv_plan(a);
  if (conv_grid(a, *pl) * 256 > kMaxThreads)
    return fail(KDA_ERR_SHAPE, "too much for one launch (B*T*C)");
  if (!a->weight) return fail(KDA_ERR_NULL, "weight is NULL");
  if (a->T > 0 && (!a->x || !a->out)) return fail(KDA_ERR_NULL, "%s is NULL", !a->x ? "x" : "out");
  const void* vec[] = {a->x, a->weight, a->bias, a->out, a->state_in, a->state_out};
  for (const void* p : vec)
    if (!aligned(p, 16)) return fail(KDA_ERR_SHAPE, "a tensor is not 16-byte aligned");
  if (!aligned(a->cu_seqlens, 8) || !aligned(a->ssm_state_indices, 4) || !aligned(a->state_out_indices, 4))
    return fail(KDA_ERR_SHAPE, "cu_seqlens or an index array is misaligned");
  const int64_t es = elem_size(a->io_dtype);
  const bool pool = a->ssm_state_indices != nullptr;
  const Wide st = state_bytes(a, dense);
  const Range in[] = {
      range_of(a->state_in, st, "state_in"),
      range_of(a->x, strided_bytes(a->B, a->T, a->x_stride, 1, 0, a->C, es), "x"),
      range_of(a->weight, Wide(4) * a->C * a->W, "weight"),
      range_of(a->bias, Wide(4) * a->C, "bias"),
      range_of(a->cu_seqlens, Wide(8) * (a->N + 1), "cu_seqlens"),
      range_of(a->ssm_state_indices, Wide(4) * a->N, "ssm_state_indices"),
      range_of(a->state_out_indices, Wide(4) * a->N, "state_out_indices"),
  };
  const Range out[] = {
      range_of(a->out, rows * a->C * es, "out"),
      range_of(pool ? a->state_in : a->state_out, st, pool ? "the pool" : "state_out"),
  };
  return no_overlap(out, in, 0);
}

// ------------------------------------------------------------ selective scan

struct ScanPlan {
  bool tokens;           // the token form
  int64_t seg;           // tokens per segment; 0: serial
  int64_t slots, segs;   // sequences (serial) or the bound on the segments; segments per sequence
  int64_t cblocks;
  size_t sums, starts, bytes;  // workspace: ends, sums, starts
};

ScanPlan scan_plan(const kda_selective_scan_args* a) {
  ScanPlan pl{};
  pl.cblocks = ceil_div(a->D, kda::kScanChannels);
  pl.slots = a->N;
  pl.segs = 1;
  if (!a->cu_seqlens && a->T >= 1 && a->T <= kda::kScanTokensMaxT && a->segment_tokens == 0) {
    pl.tokens = true;
    return pl;
  }
  // The geometry: the cheapest by a model of the time, in microseconds, fitted to one MI355X,
  // where a step is a tile of 32 tokens. S = 16, BF16: a workgroup alone on its compute unit
  // takes 1.25 a step, several 1.04 each; with S it is 0.5 + 0.047 S and 0.4 + 0.04 S, FP32
  // 0.15 more. The end states take 0.7 of the outputs' time. Serial: the longest sequence's
  // steps, or all workgroups' over 256 compute units. Segments: two launches of all of them
  // (8, and 0.2 for each segment whose end a start state has to come through).
  // One sequence of 8192 tokens, S = 16: D = 768 314 serial, 56 by segments of 256 or 384, 64
  // by 832; D = 1536 316, 97 (384, 512), 104 (832); D = 4096 320, 227 (512), 242 (1664); D =
  // 8192 318, 394 by two segments. T = 512, D = 1536: 23.5 serial, 17.8 by segments of 64.
  // A packed batch of 64 sequences, 8063 tokens, D = 1536: even lengths 74 serial, 79 by segments
  // of 1024; one of 8000 tokens 312 serial, which is what the guess of its longest one gives,
  // 119 by segments of 512.
  const bool bf16 = a->io_dtype == KDA_BF16;
  const double states = static_cast<double>(a->S);
  const double alone = 0.5 + 0.047 * states + (bf16 ? 0 : 0.15), shared = 0.4 + 0.04 * states + (bf16 ? 0 : 0.15);
  const int64_t wgs = a->N * pl.cblocks;
  // a launch of n workgroups, per step of theirs
  auto launch = [&](double n) {
    const double each = n / 256;
    return each <= 1 ? alone : std::fmax(alone, shared * (each < 4 ? std::ceil(each) : each));
  };
  const double steps = static_cast<double>(a->T) / kda::kScanTile;
  double best;
  if (a->cu_seqlens && a->N > 1) {
    // the lengths are not known here: the longest one is taken for 1.75 times the mean
    const double longest = steps * std::fmin(1.0, 1.75 / static_cast<double>(a->N));
    best = std::fmax(longest * alone, steps * static_cast<double>(pl.cblocks) / 256 * shared);
  } else {
    best = steps * launch(static_cast<double>(wgs));
  }
  int64_t seg = 0;
  for (int64_t parts = 2; a->segment_tokens == 0 && parts <= 64; ++parts) {
    const int64_t len = ceil_div(ceil_div(a->T, parts), 64) * 64;
    if (len >= a->T) continue;
    const double n = a->cu_seqlens ? static_cast<double>(ceil_div(a->T, len) + a->N / 2) * static_cast<double>(pl.cblocks)
                                   : static_cast<double>(ceil_div(a->T, len) * wgs);
    const double mean = a->cu_seqlens ? static_cast<double>(a->T / a->N) : static_cast<double>(a->T);
    const double chain = std::fmin(static_cast<double>(parts), 1.75 * mean / static_cast<double>(len));
    const double time = 8 + 0.2 * chain + static_cast<double>(len / kda::kScanTile) *
                                              (0.7 * launch(n - static_cast<double>(wgs)) + launch(n));
    if (1.05 * time < best) {  // two launches and a workspace have to save 5 %
      best = 1.05 * time;
      seg = len;
    }
  }
  if (a->segment_tokens > 0) seg = a->segment_tokens;
  if (seg >= a->T) seg = 0;
  pl.seg = seg;
  if (seg == 0) return pl;
  pl.segs = ceil_div(a->T, seg);
  pl.slots = a->cu_seqlens ? a->T / seg + a->N : a->N * pl.segs;
  const size_t state = static_cast<size_t>(a->D * a->S) * 4;
  pl.sums = static_cast<size_t>(pl.slots) * state;
  pl.starts = pl.sums + round_up(static_cast<size_t>(pl.slots * a->D) * 4, 256);
  pl.bytes = round_up(pl.starts + static_cast<size_t>(a->N) * state, 256);
  return pl;
}

kda_status scan_sizes(const kda_selective_scan_args* a, ScanPlan* pl) {
  if (!a) return fail(KDA_ERR_NULL, "args is NULL");
  kda_status s = sequences_shape(a->B, a->T, a->N, a->cu_seqlens);
  if (s != KDA_OK) return s;
  if (a->D < 8 || a->D > (1 << 22) || a->D % 8)
    return fail(KDA_ERR_SHAPE, "D=%lld is not a multiple of 8 up to 2^22", (long long)a->D);
  if (a->S != 8 && a->S != 16 && a->S != 32 && a->S != 64)
    return fail(KDA_ERR_SHAPE, "S=%lld states per channel, 8, 16, 32 and 64 are supported", (long long)a->S);
  if (a->G < 1 || a->G > a->D || a->D % a->G || (a->G > 1 && a->D / a->G % kda::kScanChannels))
    return fail(KDA_ERR_SHAPE, "G=%lld does not divide D=%lld into groups of a multiple of 32 channels",
                (long long)a->G, (long long)a->D);
  if (a->flags & ~KDA_SCAN_SOFTPLUS) return fail(KDA_ERR_FLAGS, "unknown flags 0x%x", a->flags);
  const int64_t dense = a->D * a->S;
  s = state_shape(a, dense);
  if (s == KDA_OK) s = strides_shape(a->u_stride, 2, "u");
  if (s == KDA_OK) s = strides_shape(a->delta_stride, 2, "delta");
  if (s == KDA_OK && a->z) s = strides_shape(a->z_stride, 2, "z");
  if (s == KDA_OK) s = strides_shape(a->B_stride, 3, "B");
  if (s == KDA_OK) s = strides_shape(a->C_stride, 3, "C");
  if (s != KDA_OK) return s;
  if (a->segment_tokens > 0 && (a->segment_tokens % 64 || a->segment_tokens > kBig))
    return fail(KDA_ERR_CONFIG, "segment_tokens %lld is not a multiple of 64", (long long)a->segment_tokens);
  const Wide rows = static_cast<Wide>(a->B) * a->T;
  // bound on the segments before any is counted: one per 64 tokens
  if (rows * a->D > (Wide(1) << 50) || (rows / 64 + a->N) * dense > (Wide(1) << 50))
    return fail(KDA_ERR_SHAPE, "B*T*D or N*D*S is out of range");
  *pl = scan_plan(a);
  const Wide threads = pl->tokens ? static_cast<Wide>(a->N) * ceil_div(a->D, 1024 / a->S) * 256
                                  : (static_cast<Wide>(pl->slots) * pl->cblocks + 16) * 512;
  if (threads > kMaxThreads) return fail(KDA_ERR_SHAPE, "too much for one launch (N*D, or segments*D)");
  return KDA_OK;
}

kda_status scan_check(const kda_selective_scan_args* a, ScanPlan* pl) {
  kda_status s = scan_sizes(a, pl);
  if (s != KDA_OK) return s;
  if (!a->A) return fail(KDA_ERR_NULL, "A is NULL");
  if (a->T > 0) {
    const void* need[] = {a->u, a->delta, a->B_in, a->C_in, a->out};
    const char* name[] = {"u", "delta", "B", "C", "out"};
    for (int i = 0; i < 5; ++i)
      if (!need[i]) return fail(KDA_ERR_NULL, "%s is NULL", name[i]);
  }
  const void* vec[] = {a->u, a->delta, a->z, a->B_in, a->C_in, a->A, a->out, a->state_in, a->state_out};
  for (const void* p : vec)
    if (!aligned(p, 16)) return fail(KDA_ERR_SHAPE, "a tensor is not 16-byte aligned");
  if (!aligned(a->D_skip, 4) || !aligned(a->delta_bias, 4) || !aligned(a->cu_seqlens, 8) ||
      !aligned(a->ssm_state_indices, 4) || !aligned(a->state_out_indices, 4))
    return fail(KDA_ERR_SHAPE, "D_skip, delta_bias, cu_seqlens or an index array is misaligned");
  if (pl->bytes > 0) {
    if (!a->workspace || a->workspace_bytes < pl->bytes)
      return fail(KDA_ERR_WORKSPACE, "workspace of %zu bytes, %zu are needed",
                  a->workspace ? a->workspace_bytes : size_t(0), pl->bytes);
    if (!aligned(a->workspace, 256)) return fail(KDA_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  }
  const int64_t es = elem_size(a->io_dtype), dense = a->D * a->S;
  const bool pool = a->ssm_state_indices != nullptr;
  const Wide st = state_bytes(a, dense);
  const Range in[] = {
      range_of(a->state_in, st, "state_in"),
      range_of(a->u, strided_bytes(a->B, a->T, a->u_stride, 1, 0, a->D, es), "u"),
      range_of(a->delta, strided_bytes(a->B, a->T, a->delta_stride, 1, 0, a->D, es), "delta"),
      range_of(a->z, strided_bytes(a->B, a->T, a->z_stride, 1, 0, a->D, es), "z"),
      range_of(a->B_in, strided_bytes(a->B, a->T, a->B_stride, a->G, a->B_stride[2], a->S, es), "B"),
      range_of(a->C_in, strided_bytes(a->B, a->T, a->C_stride, a->G, a->C_stride[2], a->S, es), "C"),
      range_of(a->A, Wide(4) * dense, "A"),
      range_of(a->D_skip, Wide(4) * a->D, "D_skip"),
      range_of(a->delta_bias, Wide(4) * a->D, "delta_bias"),
      range_of(a->cu_seqlens, Wide(8) * (a->N + 1), "cu_seqlens"),
      range_of(a->ssm_state_indices, Wide(4) * a->N, "ssm_state_indices"),
      range_of(a->state_out_indices, Wide(4) * a->N, "state_out_indices"),
  };
  const Range out[] = {
      range_of(a->out, static_cast<Wide>(a->B) * a->T * a->D * es, "out"),
      range_of(pool ? a->state_in : a->state_out, st, pool ? "the pool" : "state_out"),
      range_of(pl->bytes ? a->workspace : nullptr, static_cast<Wide>(pl->bytes), "workspace"),
  };
  return no_overlap(out, in, 0);
}

}  // namespace

extern "C" {

kda_status kda_short_conv_check(const kda_short_conv_args* a) {
  clear();
  ConvPlan pl;
  return conv_check(a, &pl);
}

kda_status kda_short_conv(const kda_short_conv_args* a, void* stream) {
  clear();
  ConvPlan pl;
  kda_status s = conv_check(a, &pl);
  if (s != KDA_OK) return s;
  kda::ConvParams p{};
  p.x = a->x;
  p.weight = a->weight;
  p.bias = a->bias;
  p.cu_seqlens = a->cu_seqlens;
  p.out = a->out;
  p.T = a->T;
  p.N = a->N;
  p.C = a->C;
  p.xs[0] = a->x_stride[0];
  p.xs[1] = a->x_stride[1];
  p.run = pl.run;
  p.runs_per_seq = pl.runs_per_seq;
  p.slots = pl.slots;
  p.lanes = pl.lanes;
  p.silu = (a->flags & KDA_CONV_SILU) != 0;
  p.state = state_slots(a, (a->W - 1) * a->C);
  return done(kda::launch_short_conv(p, static_cast<int>(a->W), a->io_dtype == KDA_BF16,
                                     static_cast<hipStream_t>(stream)));
}

kda_status kda_selective_scan_workspace_bytes(const kda_selective_scan_args* a, size_t* bytes) {
  clear();
  if (!bytes) return fail(KDA_ERR_NULL, "bytes is NULL");
  ScanPlan pl;
  kda_status s = scan_sizes(a, &pl);
  if (s == KDA_OK) *bytes = pl.bytes;
  return s;
}

kda_status kda_selective_scan_check(const kda_selective_scan_args* a) {
  clear();
  ScanPlan pl;
  return scan_check(a, &pl);
}

kda_status kda_selective_scan_plan(const kda_selective_scan_args* a, kda_selective_scan_plan_info* out) {
  clear();
  if (!out) return fail(KDA_ERR_NULL, "out is NULL");
  ScanPlan pl;
  kda_status s = scan_sizes(a, &pl);
  if (s != KDA_OK) return s;
  *out = kda_selective_scan_plan_info{};
  out->decode = pl.tokens ? 1 : 0;
  out->segment_tokens = pl.seg;
  out->segments_bound = pl.seg ? pl.slots : 0;
  out->workgroups = pl.tokens ? a->N * ceil_div(a->D, 1024 / a->S) : pl.slots * pl.cblocks;
  out->workspace_bytes = pl.bytes;
  return KDA_OK;
}

kda_status kda_selective_scan(const kda_selective_scan_args* a, void* stream_) {
  clear();
  ScanPlan pl;
  kda_status s = scan_check(a, &pl);
  if (s != KDA_OK) return s;
  hipStream_t stream = static_cast<hipStream_t>(stream_);
  const bool bf16 = a->io_dtype == KDA_BF16;
  const int n = static_cast<int>(a->S);
  kda::ScanParams p{};
  p.u = a->u;
  p.delta = a->delta;
  p.z = a->z;
  p.B = a->B_in;
  p.C = a->C_in;
  p.A = a->A;
  p.skip = a->D_skip;
  p.bias = a->delta_bias;
  p.cu_seqlens = a->cu_seqlens;
  p.out = a->out;
  p.T = a->T;
  p.N = a->N;
  p.D = a->D;
  p.per_group = a->D / a->G;
  for (int d = 0; d < 2; ++d) {
    p.us[d] = a->u_stride[d];
    p.ds[d] = a->delta_stride[d];
    p.zs[d] = a->z_stride[d];
  }
  for (int d = 0; d < 3; ++d) {
    p.bs[d] = a->B_stride[d];
    p.cs[d] = a->C_stride[d];
  }
  p.softplus = (a->flags & KDA_SCAN_SOFTPLUS) != 0;
  p.state = state_slots(a, a->D * a->S);
  if (pl.tokens) return done(kda::launch_scan_tokens(p, n, bf16, stream));
  p.seg_len = pl.seg ? pl.seg : a->T + 1;  // longer than any sequence: a slot for each
  p.segs_per_seq = pl.segs;
  p.slots = pl.slots;
  p.cblocks = pl.cblocks;
  p.segmented = pl.seg ? 1 : 0;
  p.longest_first = a->cu_seqlens && !pl.seg && a->N > 1 && a->N <= 64;
  unsigned char* ws = static_cast<unsigned char*>(a->workspace);
  p.ends = reinterpret_cast<float*>(ws);
  p.sums = reinterpret_cast<float*>(ws + pl.sums);
  p.starts = reinterpret_cast<float*>(ws + pl.starts);
  hipError_t e = hipSuccess;
  if (pl.seg) e = kda::launch_scan_ends(p, n, bf16, stream);
  if (e == hipSuccess) e = kda::launch_scan_outputs(p, n, bf16, stream);
  return done(e);
}

}  // extern "C"

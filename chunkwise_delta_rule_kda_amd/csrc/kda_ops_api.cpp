// Host side of the operators beside kda_prefill (include/kda.h): argument checks, launch
// geometry and the extern "C" entry points of linear attention with one decay per head,
// the state pool's slot operations and the gated norm. No allocation, no device
// synchronisation, no state kept between calls.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "kda.h"
#include "kda_ops_internal.h"

namespace {

kda_status fail(kda_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
kda_status fail(kda_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return kda::set_error(s, buf);
}

kda_status clear() { return kda::set_error(KDA_OK, ""); }

constexpr int64_t kBig = int64_t(1) << 40;  // bound on sizes, strides and pitches
constexpr int64_t kMaxThreads = 0xffffffffLL;  // of one launch: HIP refuses more

bool known_dtype(int32_t d) { return d == KDA_BF16 || d == KDA_FP32; }
int64_t elem_size(int32_t d) { return d == KDA_BF16 ? 2 : 4; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

typedef __int128 Wide;

struct Range {
  Wide lo, hi;
  const char* name;
};
Range range_of(const void* p, Wide bytes, const char* name) {
  const Wide lo = static_cast<Wide>(reinterpret_cast<uintptr_t>(p));
  return Range{lo, p ? lo + bytes : lo, name};
}
bool overlap(const Range& a, const Range& b) {
  return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

// ------------------------------------------------------------ linear attention

bool linear_token_form(const kda_linear_args* a) {
  return !a->cu_seqlens && a->T >= 1 && a->T <= kda::kLinDecodeMaxT && a->segment_tokens == 0;
}

kda_status linear_shape(const kda_linear_args* a) {
  if (!a) return fail(KDA_ERR_NULL, "args is NULL");
  if (a->K != 64 && a->K != 128)
    return fail(KDA_ERR_SHAPE, "K=%lld, only 64 and 128 are supported", (long long)a->K);
  if (a->V < 64 || a->V > 512 || a->V % 64)
    return fail(KDA_ERR_SHAPE, "V=%lld is not a multiple of 64 up to 512", (long long)a->V);
  if (a->B < 1 || a->B > (int64_t(1) << 31) || a->T < 0 || a->T > (int64_t(1) << 36) || a->N < 0 ||
      a->N > (int64_t(1) << 31))
    return fail(KDA_ERR_SHAPE, "bad B=%lld T=%lld N=%lld", (long long)a->B, (long long)a->T,
                (long long)a->N);
  if (a->H < 1 || a->H > (1 << 22) || a->H * a->V > (1 << 22))  // a chunk's rows of o stay within 2^31 bytes
    return fail(KDA_ERR_SHAPE, "H=%lld is not positive, or H*V exceeds 2^22", (long long)a->H);
  if (a->Hk < 1 || a->Hk > a->H || a->H % a->Hk)
    return fail(KDA_ERR_SHAPE, "Hk=%lld does not divide H=%lld", (long long)a->Hk, (long long)a->H);
  if (a->cu_seqlens) {
    if (a->B != 1) return fail(KDA_ERR_SHAPE, "packed varlen needs B=1 (got %lld)", (long long)a->B);
    if (a->N < 1) return fail(KDA_ERR_SHAPE, "packed varlen needs N>=1");
  } else if (a->N != a->B) {
    return fail(KDA_ERR_SHAPE, "fixed layout needs N == B (N=%lld, B=%lld)", (long long)a->N,
                (long long)a->B);
  }
  if (!known_dtype(a->io_dtype)) return fail(KDA_ERR_DTYPE, "io_dtype %d", a->io_dtype);
  if (!known_dtype(a->state_dtype)) return fail(KDA_ERR_DTYPE, "state_dtype %d", a->state_dtype);
  if (a->g && !known_dtype(a->g_dtype)) return fail(KDA_ERR_DTYPE, "g_dtype %d", a->g_dtype);
  if (!std::isfinite(a->scale) || a->scale < 0.0f)
    return fail(KDA_ERR_BOUND, "scale %g", (double)a->scale);
  if (a->segment_tokens > 0 && (a->segment_tokens % kda::kLinChunk || a->segment_tokens > kBig))
    return fail(KDA_ERR_CONFIG, "segment_tokens %lld is not a multiple of 64",
                (long long)a->segment_tokens);
  const int64_t* strides[3] = {a->q_stride, a->k_stride, a->v_stride};
  for (int i = 0; i < 3; ++i) {
    for (int d = 0; d < 3; ++d)
      if (strides[i][d] < 0 || strides[i][d] > kBig || strides[i][d] % 8)
        return fail(KDA_ERR_SHAPE, "%c stride %lld is negative or not a multiple of 8", "qkv"[i],
                    (long long)strides[i][d]);
    if (strides[i][1] > (int64_t(1) << 22))
      return fail(KDA_ERR_SHAPE, "%c token stride %lld exceeds 2^22", "qkv"[i],
                  (long long)strides[i][1]);
  }
  if (a->ssm_state_indices) {
    if (!a->state_in) return fail(KDA_ERR_CONFIG, "a state pool needs state_in");
    if (a->state_pool_slots < 1 || a->state_pool_slots > (int64_t(1) << 31))
      return fail(KDA_ERR_CONFIG, "state_pool_slots %lld", (long long)a->state_pool_slots);
    const int64_t dense = a->H * a->V * a->K;
    if (a->state_slot_pitch != 0 &&
        (a->state_slot_pitch < dense || a->state_slot_pitch % 8 || a->state_slot_pitch > kBig))
      return fail(KDA_ERR_CONFIG, "state_slot_pitch %lld", (long long)a->state_slot_pitch);
  } else if (a->state_out_indices) {
    return fail(KDA_ERR_CONFIG, "state_out_indices needs ssm_state_indices");
  }
  return KDA_OK;
}

struct LinPlan {
  bool tokens;         // the token loop
  int rows;            // value rows per workgroup
  int64_t seg;         // tokens per segment; 0: serial
  int64_t slots;       // sequences (serial) or the bound on the segments of one head
  int64_t segs;        // fixed layout: segments per sequence
  size_t scan_d, bytes;
};

LinPlan linear_plan(const kda_linear_args* a) {
  LinPlan pl{};
  if (linear_token_form(a)) {
    pl.tokens = true;
    // 64 rows per workgroup where that gives 512 of them (N H = 384, BF16 states, one token:
    // 6.9 us, 9.3 with 16 rows; 24 heads of 128: 34 and 46), fewer rows below (N H = 6: 3.4 us with
    // 16, 4.3 with 64); FP32 states of one token stream best in the smallest pieces (24 heads of
    // 128 sequences: 73.0 us with 16 rows, 74.4 with 32, 76.4 with 64; 96 of 64: 142, 147, 150)
    const int least = a->K == 128 ? 16 : 32;
    int rows = a->T == 1 && a->state_dtype == KDA_FP32 ? least : 64;
    while (rows > least && a->N * a->H * (a->V / rows) < 512) rows /= 2;
    pl.rows = rows;
    pl.slots = a->N;
    pl.segs = 1;
    return pl;
  }
  // The chunked form's geometry: the cheapest by a model of the time, in microseconds, fitted
  // to one MI355X (K = V = 128), where a compute unit takes one workgroup at a time and a step
  // is 64 tokens. BF16 I/O, by 64 or 128 value rows, W workgroups (at most 256):
  //   serial    5 + steps x 1.27 or 1.85 x rounds of 256 workgroups; a step takes 0.3 more
  //             where q, k, v and o are more than the 256 MB of the last-level cache
  //   segments  14.3 + 0.028 W + steps of a segment x 1.8, or 18 + 0.028 W + 3.5 x steps, both
  //             passes and the scan; 2.7 and 4.5 a step past the last-level cache, from which
  //             the second pass else reads k and v
  // T = 8192: H = 6 32 us by 64-row segments, 168 serial; H = 12 44 by 64-row segments, 49 by
  // 128-row ones; H = 40 (past the cache) 132 and 113, 220 serial; H = 96 239 to 248 serial, 283
  // by 128 rows, 243 by two 128-row segments and a workspace. T = 1024: H = 6 21 us by segments,
  // 24 serial; H = 20 27 and 25.
  // FP32 I/O: serial 6 + 7 x steps x rounds, segments 10 + rounds x (6 + 10.2 x steps), bound
  // by its products, so segments over several rounds gain as well: T = 1999, H = 48: 152 us
  // over two rounds, 177 over one, 228 serial.
  constexpr int64_t kUnits = 256;  // compute units
  const bool bf16 = a->io_dtype == KDA_BF16;
  const double bytes = static_cast<double>(elem_size(a->io_dtype)) * static_cast<double>(a->B) *
                       static_cast<double>(a->T) * 2.0 * static_cast<double>(a->Hk * a->K + a->H * a->V);
  const bool cached = bytes <= 256e6;
  // 128 rows of an FP32 state (its updates in three parts) do not fit the registers
  const int most = bf16 && a->state_dtype == KDA_BF16 && a->V % 128 == 0 ? 128 : 64;
  // The host does not know a packed batch's lengths. Its longest sequence is taken for 1.75
  // times the mean, not for the mean, since a wrong choice costs more where lengths are
  // uneven: two sequences, T = 2386, H = 20, are cut and take 35 to 37 us whatever their
  // lengths; serial 31 at 1 : 1, 38 at 2 : 1, 48 at 7 : 1 (T = 6678, H = 38: 87 to 103 cut; 75,
  // 97 and 124 serial). One long prompt among many short ones is a longer chain than this.
  const double steps = a->cu_seqlens && a->N > 1
                           ? std::fmin(1.0, 1.75 / static_cast<double>(a->N)) * static_cast<double>(a->T) / 64
                           : static_cast<double>(a->T) / 64;
  double best = 1e300;
  int64_t seg = 0;
  for (int rows = 64; rows <= most; rows *= 2) {
    const int64_t blocks = a->H * (a->V / rows), wgs = a->N * blocks;
    const double step = !bf16 ? 7.0 : (rows == 64 ? 1.27 : 1.85) + (cached ? 0.0 : 0.3);
    const double serial = (bf16 ? 5 : 6) + steps * step * static_cast<double>(ceil_div(wgs, kUnits));
    if (serial < best) {
      best = serial;
      pl.rows = rows;
      seg = 0;
    }
    for (int64_t rounds = 1; a->segment_tokens == 0 && rounds <= (bf16 ? 1 : 3); ++rounds) {
      const int64_t units = kUnits * rounds;
      if (wgs > units / 2) continue;
      int64_t len = a->cu_seqlens ? ceil_div(a->T * blocks, units - wgs) : ceil_div(a->T, units / wgs);
      len = ceil_div(len < 128 ? 128 : len, kda::kLinChunk) * kda::kLinChunk;
      const double chunks = static_cast<double>(len / 64);
      const double filled = std::fmin(256.0, static_cast<double>(ceil_div(a->T, len) * wgs));
      // three launches and a workspace have to save 5 %
      const double cut = 1.05 * (!bf16 ? 10 + static_cast<double>(rounds) * (6 + 10.2 * chunks)
                                 : rows == 64 ? 14.3 + 0.028 * filled + (cached ? 1.8 : 2.7) * chunks
                                              : 18 + 0.028 * filled + (cached ? 3.5 : 4.5) * chunks);
      if (len < a->T && cut < best) {
        best = cut;
        pl.rows = rows;
        seg = len;
      }
    }
  }
  if (a->segment_tokens > 0) seg = a->segment_tokens;
  if (seg >= a->T) seg = 0;
  pl.seg = seg;
  if (seg == 0) {
    pl.slots = a->N;
    pl.segs = 1;
    return pl;
  }
  pl.segs = ceil_div(a->T, seg);
  pl.slots = a->cu_seqlens ? a->T / seg + a->N : a->N * pl.segs;
  const size_t state = static_cast<size_t>(a->V * a->K) * 4;
  pl.scan_d = static_cast<size_t>(a->H * pl.slots) * state;
  pl.bytes = round_up(pl.scan_d + static_cast<size_t>(a->H * pl.slots) * 4, 256);
  return pl;
}

// Every size below stays far from overflow: slots <= 2^40, H <= 2^16, checked here.
kda_status linear_sizes(const kda_linear_args* a, LinPlan* out) {
  kda_status s = linear_shape(a);
  if (s != KDA_OK) return s;
  const Wide states = static_cast<Wide>(a->N) * a->H * a->V * a->K;
  const Wide tokens = static_cast<Wide>(a->cu_seqlens ? 1 : a->B) * a->T;
  if (states > (Wide(1) << 50) || tokens * a->H * a->V > (Wide(1) << 50))
    return fail(KDA_ERR_SHAPE, "N*H*V*K or B*T*H*V is out of range");
  // bound on the segments before any is counted: one per chunk
  if ((tokens / kda::kLinChunk + a->N) * a->H * a->V * a->K > (Wide(1) << 56))
    return fail(KDA_ERR_SHAPE, "too many chunks");
  const LinPlan pl = linear_plan(a);
  // the token loop's launch, or the scan's and the larger one of the states' (always by
  // kLinRows) and the outputs'
  const Wide pairs = static_cast<Wide>(a->N) * a->H;
  const Wide threads = pl.tokens ? pairs * (a->V / pl.rows) * 256
                                 : (static_cast<Wide>(pl.slots) * a->H + 8) *
                                       (a->V / (pl.seg ? kda::kLinRows : pl.rows)) * 512;
  if (threads > kMaxThreads || (pl.seg && pairs * ceil_div(a->V * a->K, 1024) * 256 > kMaxThreads))
    return fail(KDA_ERR_SHAPE, "too much for one launch (N*H, or segments*H)");
  *out = pl;
  return KDA_OK;
}

Wide strided_bytes(const kda_linear_args* a, const int64_t* st, int64_t heads, int64_t dim) {
  if (a->T == 0) return 0;
  const Wide e = static_cast<Wide>(a->B - 1) * st[0] + static_cast<Wide>(a->T - 1) * st[1] +
                 static_cast<Wide>(heads - 1) * st[2] + dim;
  return e * elem_size(a->io_dtype);
}

kda_status linear_check(const kda_linear_args* a, LinPlan* pl) {
  kda_status s = linear_sizes(a, pl);
  if (s != KDA_OK) return s;
  if (a->T > 0 && (!a->q || !a->k || !a->v || !a->o))
    return fail(KDA_ERR_NULL, "%s is NULL", !a->q ? "q" : !a->k ? "k" : !a->v ? "v" : "o");
  const int64_t dense = a->H * a->V * a->K;
  const int64_t pitch = a->state_slot_pitch ? a->state_slot_pitch : dense;
  const bool pool = a->ssm_state_indices != nullptr;
  if (pool && a->state_out && a->state_out != a->state_in)
    return fail(KDA_ERR_ALIAS, "with a state pool, state_out must be NULL or state_in");
  const void* vec[] = {a->q, a->k, a->v, a->o, a->state_in, a->state_out};
  for (const void* p : vec)
    if (!aligned(p, 16)) return fail(KDA_ERR_SHAPE, "a tensor is not 16-byte aligned");
  if (!aligned(a->g, 4) || !aligned(a->log_decay, 4) || !aligned(a->cu_seqlens, 8) ||
      !aligned(a->ssm_state_indices, 4) || !aligned(a->state_out_indices, 4))
    return fail(KDA_ERR_SHAPE, "g, log_decay, cu_seqlens or an index array is misaligned");
  if (pl->bytes > 0) {
    if (!a->workspace || a->workspace_bytes < pl->bytes)
      return fail(KDA_ERR_WORKSPACE, "workspace of %zu bytes, %zu are needed",
                  a->workspace ? a->workspace_bytes : size_t(0), pl->bytes);
    if (!aligned(a->workspace, 256)) return fail(KDA_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  }
  const Wide st = elem_size(a->state_dtype);
  const Wide rows = static_cast<Wide>(a->B) * a->T * a->H;
  const Wide in_state = pool ? (static_cast<Wide>(a->state_pool_slots - 1) * pitch + dense) * st
                             : static_cast<Wide>(a->N) * dense * st;
  const Range in[] = {
      range_of(a->q, strided_bytes(a, a->q_stride, a->Hk, a->K), "q"),
      range_of(a->k, strided_bytes(a, a->k_stride, a->Hk, a->K), "k"),
      range_of(a->v, strided_bytes(a, a->v_stride, a->H, a->V), "v"),
      range_of(a->g, rows * elem_size(a->g_dtype), "g"),
      range_of(a->log_decay, Wide(4) * a->H, "log_decay"),
      range_of(a->cu_seqlens, Wide(8) * (a->N + 1), "cu_seqlens"),
      range_of(a->ssm_state_indices, Wide(4) * a->N, "ssm_state_indices"),
      range_of(a->state_out_indices, Wide(4) * a->N, "state_out_indices"),
      range_of(a->state_in, in_state, "state_in"),
  };
  const Range out[] = {
      range_of(a->o, rows * a->V * elem_size(a->io_dtype), "o"),
      range_of(pool ? a->state_in : a->state_out, in_state, pool ? "the pool" : "state_out"),
      range_of(pl->bytes ? a->workspace : nullptr, static_cast<Wide>(pl->bytes), "workspace"),
  };
  for (int i = 0; i < 3; ++i) {
    for (const Range& r : in) {
      const bool same_state = i == 1 && r.lo == out[1].lo && r.name == in[8].name;
      if (!same_state && overlap(out[i], r))
        return fail(KDA_ERR_ALIAS, "%s overlaps %s", out[i].name, r.name);
    }
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j]))
        return fail(KDA_ERR_ALIAS, "%s overlaps %s", out[i].name, out[j].name);
  }
  return KDA_OK;
}

// ------------------------------------------------------------ pools

kda_status pool_shape(const kda_pool* p, const char* name) {
  if (!known_dtype(p->dtype)) return fail(KDA_ERR_DTYPE, "%s dtype %d", name, p->dtype);
  if (p->slots < 1 || p->slots > (int64_t(1) << 31) || p->layers < 1 || p->layers > (1 << 20) ||
      p->slot_elems < 8 || p->slot_elems > kBig || p->slot_elems % 8)
    return fail(KDA_ERR_SHAPE, "%s: slots=%lld layers=%lld slot_elems=%lld", name,
                (long long)p->slots, (long long)p->layers, (long long)p->slot_elems);
  if (p->slot_pitch < p->slot_elems || p->slot_pitch > kBig || p->slot_pitch % 8 ||
      p->layer_pitch < 0 || p->layer_pitch > (int64_t(1) << 50) || p->layer_pitch % 8)
    return fail(KDA_ERR_CONFIG, "%s: slot_pitch=%lld layer_pitch=%lld", name,
                (long long)p->slot_pitch, (long long)p->layer_pitch);
  const Wide all = static_cast<Wide>(p->slots - 1) * p->slot_pitch + p->slot_elems;
  // layers one behind another, or interleaved inside the slots' pitch
  if (p->layers > 1 && p->layer_pitch < all &&
      (p->layer_pitch < p->slot_elems ||
       static_cast<Wide>(p->layers - 1) * p->layer_pitch + p->slot_elems > p->slot_pitch))
    return fail(KDA_ERR_CONFIG, "%s: layers overlap (layer_pitch=%lld)", name,
                (long long)p->layer_pitch);
  if (!p->base) return fail(KDA_ERR_NULL, "%s is NULL", name);
  if (!aligned(p->base, 16)) return fail(KDA_ERR_SHAPE, "%s is not 16-byte aligned", name);
  return KDA_OK;
}

Range pool_range(const kda_pool* p, const char* name) {
  const Wide e = static_cast<Wide>(p->slots - 1) * p->slot_pitch +
                 static_cast<Wide>(p->layers - 1) * p->layer_pitch + p->slot_elems;
  return range_of(p->base, e * elem_size(p->dtype), name);
}

bool same_pool(const kda_pool* a, const kda_pool* b) {
  return a->base == b->base && a->dtype == b->dtype && a->slots == b->slots &&
         a->slot_pitch == b->slot_pitch && (a->layers == 1 || a->layer_pitch == b->layer_pitch);
}

kda_status grid_of(const kda_pool* p, int64_t pairs) {
  if (static_cast<Wide>(ceil_div(p->slot_elems, kda::kCopyGroup)) * p->layers * pairs * 256 > kMaxThreads)
    return fail(KDA_ERR_SHAPE, "pairs x layers x slot_elems are too many for one launch");
  return KDA_OK;
}

kda_status copy_check(const kda_pool_copy_args* a) {
  if (!a) return fail(KDA_ERR_NULL, "args is NULL");
  kda_status s = pool_shape(&a->src, "src");
  if (s == KDA_OK) s = pool_shape(&a->dst, "dst");
  if (s != KDA_OK) return s;
  if (a->src.layers != a->dst.layers || a->src.slot_elems != a->dst.slot_elems)
    return fail(KDA_ERR_SHAPE, "src and dst differ in layers or slot_elems");
  if (a->pairs < 0 || a->pairs > (int64_t(1) << 31))
    return fail(KDA_ERR_SHAPE, "pairs=%lld", (long long)a->pairs);
  s = grid_of(&a->dst, a->pairs);
  if (s != KDA_OK) return s;
  if (a->pairs > 0 && (!a->src_idx || !a->dst_idx)) return fail(KDA_ERR_NULL, "an index array is NULL");
  if (!aligned(a->src_idx, 4) || !aligned(a->dst_idx, 4))
    return fail(KDA_ERR_SHAPE, "an index array is misaligned");
  const Range dst = pool_range(&a->dst, "dst");
  if (!same_pool(&a->src, &a->dst) && overlap(pool_range(&a->src, "src"), dst))
    return fail(KDA_ERR_ALIAS, "src and dst overlap and are not the same pool");
  if (overlap(range_of(a->src_idx, Wide(4) * a->pairs, ""), dst) ||
      overlap(range_of(a->dst_idx, Wide(4) * a->pairs, ""), dst))
    return fail(KDA_ERR_ALIAS, "dst overlaps an index array");
  return KDA_OK;
}

// Workspace of the compaction: the moves' sources and destinations, and their number.
int64_t most_moves(const kda_pool_compact_args* a) {
  return a->n < a->pool.slots ? a->n : a->pool.slots;
}
size_t compact_bytes(const kda_pool_compact_args* a) {
  return round_up(static_cast<size_t>(2 * most_moves(a) + 1) * 4, 256);
}

kda_status compact_shape(const kda_pool_compact_args* a) {
  if (!a) return fail(KDA_ERR_NULL, "args is NULL");
  kda_status s = pool_shape(&a->pool, "pool");
  if (s != KDA_OK) return s;
  if (a->pool.slots > KDA_POOL_COMPACT_SLOTS)
    return fail(KDA_ERR_SHAPE, "slots=%lld exceeds %d", (long long)a->pool.slots, KDA_POOL_COMPACT_SLOTS);
  if (a->n < 0 || a->n > (int64_t(1) << 31)) return fail(KDA_ERR_SHAPE, "n=%lld", (long long)a->n);
  return grid_of(&a->pool, most_moves(a));
}

kda_status compact_check(const kda_pool_compact_args* a) {
  kda_status s = compact_shape(a);
  if (s != KDA_OK) return s;
  if (a->n > 0 && (!a->idx || !a->new_idx)) return fail(KDA_ERR_NULL, "idx or new_idx is NULL");
  if (!a->count) return fail(KDA_ERR_NULL, "count is NULL");
  if (!aligned(a->idx, 4) || !aligned(a->new_idx, 4) || !aligned(a->count, 4))
    return fail(KDA_ERR_SHAPE, "idx, new_idx or count is misaligned");
  if (!a->workspace || a->workspace_bytes < compact_bytes(a))
    return fail(KDA_ERR_WORKSPACE, "workspace of %zu bytes, %zu are needed",
                a->workspace ? a->workspace_bytes : size_t(0), compact_bytes(a));
  if (!aligned(a->workspace, 256)) return fail(KDA_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  const Range r[] = {
      range_of(a->idx, Wide(4) * a->n, "idx"), range_of(a->new_idx, Wide(4) * a->n, "new_idx"),
      range_of(a->count, 4, "count"), pool_range(&a->pool, "pool"),
      range_of(a->workspace, static_cast<Wide>(compact_bytes(a)), "workspace")};
  for (int i = 0; i < 5; ++i)
    for (int j = 0; j < i; ++j)
      if (!(i == 1 && j == 0 && a->idx == a->new_idx) && overlap(r[i], r[j]))
        return fail(KDA_ERR_ALIAS, "%s overlaps %s", r[i].name, r[j].name);
  return KDA_OK;
}

// ------------------------------------------------------------ gated norm

kda_status norm_check(const kda_gated_norm_args* a) {
  if (!a) return fail(KDA_ERR_NULL, "args is NULL");
  if (a->D < 8 || a->D > kda::kNormMax || a->D % 8)
    return fail(KDA_ERR_SHAPE, "D=%lld is not a multiple of 8 up to %d", (long long)a->D,
                kda::kNormMax);
  if (a->M < 0 || a->M > kBig || a->G < 1 || a->G > kBig ||
      static_cast<Wide>(a->M) * a->G * kda::norm_threads(a->D) > kMaxThreads - 256)
    return fail(KDA_ERR_SHAPE, "M=%lld G=%lld D=%lld", (long long)a->M, (long long)a->G, (long long)a->D);
  if (!known_dtype(a->io_dtype)) return fail(KDA_ERR_DTYPE, "io_dtype %d", a->io_dtype);
  if (a->act != KDA_ACT_SIGMOID && a->act != KDA_ACT_SILU)
    return fail(KDA_ERR_FLAGS, "act %d", a->act);
  if (!(a->eps >= 0.0f) || !std::isfinite(a->eps) || !std::isfinite(a->scale))
    return fail(KDA_ERR_BOUND, "eps %g, scale %g", (double)a->eps, (double)a->scale);
  if (a->next_weight && !a->next_out) return fail(KDA_ERR_NULL, "next_weight needs next_out");
  if (a->M > 0 && (!a->x || !a->out)) return fail(KDA_ERR_NULL, "x or out is NULL");
  const void* vec[] = {a->x, a->gate, a->residual, a->weight, a->next_weight, a->out, a->next_out};
  for (const void* p : vec)
    if (!aligned(p, 16)) return fail(KDA_ERR_SHAPE, "a tensor is not 16-byte aligned");
  const void* in[] = {a->x, a->gate, a->residual};
  const int64_t* st[] = {a->x_stride, a->gate_stride, a->residual_stride};
  const char* name[] = {"x", "gate", "residual"};
  const Wide es = elem_size(a->io_dtype);
  const Wide all = static_cast<Wide>(a->M) * a->G * a->D * es;
  const Range out = range_of(a->out, all, "out"), next = range_of(a->next_out, all, "next_out");
  if (overlap(out, next)) return fail(KDA_ERR_ALIAS, "out overlaps next_out");
  for (int i = 0; i < 3; ++i) {
    if (!in[i]) continue;
    for (int d = 0; d < 2; ++d)
      if (st[i][d] < 0 || st[i][d] > kBig || st[i][d] % 8)
        return fail(KDA_ERR_SHAPE, "%s stride %lld is negative or not a multiple of 8", name[i],
                    (long long)st[i][d]);
    if (a->M == 0) continue;
    const Wide e = static_cast<Wide>(a->M - 1) * st[i][0] + static_cast<Wide>(a->G - 1) * st[i][1] + a->D;
    const Range r = range_of(in[i], e * es, name[i]);
    const bool dense = (a->G == 1 || st[i][1] == a->D) && (a->M == 1 || st[i][0] == a->G * a->D);
    if (overlap(out, r) && !(in[i] == a->out && dense))
      return fail(KDA_ERR_ALIAS, "out overlaps %s", name[i]);
    if (overlap(next, r)) return fail(KDA_ERR_ALIAS, "next_out overlaps %s", name[i]);
  }
  const Range w = range_of(a->weight, Wide(4) * a->D, "weight"),
              nw = range_of(a->next_weight, Wide(4) * a->D, "next_weight");
  if (overlap(out, w) || overlap(next, w) || overlap(out, nw) || overlap(next, nw))
    return fail(KDA_ERR_ALIAS, "an output overlaps a weight");
  return KDA_OK;
}

kda_status done(hipError_t e) {
  return e == hipSuccess ? KDA_OK : fail(KDA_ERR_HIP, "%s", hipGetErrorString(e));
}

}  // namespace

extern "C" {

kda_status kda_linear_workspace_bytes(const kda_linear_args* a, size_t* bytes) {
  clear();
  if (!bytes) return fail(KDA_ERR_NULL, "bytes is NULL");
  LinPlan pl;
  kda_status s = linear_sizes(a, &pl);
  if (s == KDA_OK) *bytes = pl.bytes;
  return s;
}

kda_status kda_linear_check(const kda_linear_args* a) {
  clear();
  LinPlan pl;
  return linear_check(a, &pl);
}

kda_status kda_linear_plan(const kda_linear_args* a, kda_linear_plan_info* out) {
  clear();
  if (!out) return fail(KDA_ERR_NULL, "out is NULL");
  LinPlan pl;
  kda_status s = linear_sizes(a, &pl);
  if (s != KDA_OK) return s;
  *out = kda_linear_plan_info{};
  out->decode = pl.tokens ? 1 : 0;
  out->value_block = pl.rows;
  out->segment_tokens = pl.seg;
  out->segments_bound = pl.seg ? pl.slots : 0;
  out->workgroups = pl.slots * a->H * (a->V / pl.rows);
  out->state_workgroups = pl.seg ? pl.slots * a->H * (a->V / kda::kLinRows) : 0;
  out->workspace_bytes = pl.bytes;
  return KDA_OK;
}

kda_status kda_linear(const kda_linear_args* a, void* stream_) {
  clear();
  LinPlan pl;
  kda_status s = linear_check(a, &pl);
  if (s != KDA_OK) return s;
  hipStream_t stream = static_cast<hipStream_t>(stream_);
  const bool bf16 = a->io_dtype == KDA_BF16;
  kda::LinParams p{};
  p.q = a->q;
  p.k = a->k;
  p.v = a->v;
  p.g = a->g;
  p.log_decay = a->log_decay;
  p.state_in = a->state_in;
  p.cu_seqlens = a->cu_seqlens;
  p.o = a->o;
  p.state_out = a->state_out;
  p.T = a->T;
  p.N = a->N;
  p.H = static_cast<int32_t>(a->H);
  p.Hk = static_cast<int32_t>(a->Hk);
  p.V = static_cast<int32_t>(a->V);
  for (int d = 0; d < 3; ++d) {
    p.qs[d] = a->q_stride[d];
    p.ks[d] = a->k_stride[d];
    p.vs[d] = a->v_stride[d];
  }
  p.scale = a->scale > 0.0f ? a->scale : 1.0f / std::sqrt(static_cast<float>(a->K));
  p.log2_scale = std::log2(static_cast<double>(p.scale));
  p.g_bf16 = a->g_dtype == KDA_BF16;
  p.st_bf16 = a->state_dtype == KDA_BF16;
  p.split = bf16 && !p.st_bf16;
  p.pool_slots = a->N;
  p.slot_pitch = a->H * a->V * a->K;
  if (a->ssm_state_indices) {
    p.in_idx = a->ssm_state_indices;
    p.out_idx = a->state_out_indices ? a->state_out_indices : a->ssm_state_indices;
    p.pool_slots = a->state_pool_slots;
    if (a->state_slot_pitch) p.slot_pitch = a->state_slot_pitch;
    p.state_out = const_cast<void*>(a->state_in);  // the pool is updated in place
  }
  const int k_dim = static_cast<int>(a->K);
  if (pl.tokens) return done(kda::launch_linear_tokens(p, k_dim, bf16, pl.rows, stream));
  p.seg_len = pl.seg ? pl.seg : (a->T > 0 ? ceil_div(a->T, kda::kLinChunk) * kda::kLinChunk + kda::kLinChunk : kda::kLinChunk);
  p.segs_per_seq = pl.segs;
  p.slots = pl.slots;
  p.segmented = pl.seg ? 1 : 0;
  p.longest_first = a->cu_seqlens && !pl.seg && a->N > 1 && a->N <= 64;
  p.scan_s = static_cast<float*>(a->workspace);
  p.scan_d = reinterpret_cast<float*>(static_cast<unsigned char*>(a->workspace) + pl.scan_d);
  p.vblocks = static_cast<int32_t>(a->V / pl.rows);
  hipError_t e = hipSuccess;
  if (pl.seg) {
    kda::LinParams ps = p;
    ps.vblocks = static_cast<int32_t>(a->V / kda::kLinRows);
    e = kda::launch_linear_states(ps, k_dim, bf16, stream);
    if (e == hipSuccess) e = kda::launch_linear_scan(p, k_dim, stream);
  }
  if (e == hipSuccess) e = kda::launch_linear_chunks(p, k_dim, bf16, pl.rows, stream);
  return done(e);
}

kda_status kda_pool_copy_check(const kda_pool_copy_args* a) {
  clear();
  return copy_check(a);
}

kda_status kda_pool_copy(const kda_pool_copy_args* a, void* stream) {
  clear();
  kda_status s = copy_check(a);
  if (s != KDA_OK) return s;
  kda::PoolCopy p{};
  p.src = a->src.base;
  p.dst = a->dst.base;
  p.src_slots = a->src.slots;
  p.src_pitch = a->src.slot_pitch;
  p.src_layer = a->src.layer_pitch;
  p.dst_slots = a->dst.slots;
  p.dst_pitch = a->dst.slot_pitch;
  p.dst_layer = a->dst.layer_pitch;
  p.slot_elems = a->dst.slot_elems;
  p.layers = a->dst.layers;
  p.pairs = a->pairs;
  p.src_idx = a->src_idx;
  p.dst_idx = a->dst_idx;
  p.src_bf16 = a->src.dtype == KDA_BF16;
  p.dst_bf16 = a->dst.dtype == KDA_BF16;
  return done(kda::launch_pool_copy(p, static_cast<hipStream_t>(stream)));
}

kda_status kda_pool_compact_workspace_bytes(const kda_pool_compact_args* a, size_t* bytes) {
  clear();
  if (!bytes) return fail(KDA_ERR_NULL, "bytes is NULL");
  kda_status s = compact_shape(a);
  if (s == KDA_OK) *bytes = compact_bytes(a);
  return s;
}

kda_status kda_pool_compact_check(const kda_pool_compact_args* a) {
  clear();
  return compact_check(a);
}

kda_status kda_pool_compact(const kda_pool_compact_args* a, void* stream_) {
  clear();
  kda_status s = compact_check(a);
  if (s != KDA_OK) return s;
  hipStream_t stream = static_cast<hipStream_t>(stream_);
  const int64_t most = most_moves(a);
  int32_t* ws = static_cast<int32_t*>(a->workspace);
  int32_t* moves = ws + 2 * most;
  hipError_t e = kda::launch_pool_plan(a->idx, a->new_idx, a->count, a->n, a->pool.slots, ws,
                                       ws + most, moves, stream);
  if (e != hipSuccess) return done(e);
  kda::PoolCopy p{};
  p.src = p.dst = a->pool.base;
  p.src_slots = p.dst_slots = a->pool.slots;
  p.src_pitch = p.dst_pitch = a->pool.slot_pitch;
  p.src_layer = p.dst_layer = a->pool.layer_pitch;
  p.slot_elems = a->pool.slot_elems;
  p.layers = a->pool.layers;
  p.pairs = most;
  p.src_idx = ws;
  p.dst_idx = ws + most;
  p.count = moves;
  p.src_bf16 = p.dst_bf16 = a->pool.dtype == KDA_BF16;
  return done(kda::launch_pool_copy(p, stream));
}

kda_status kda_gated_norm_check(const kda_gated_norm_args* a) {
  clear();
  return norm_check(a);
}

kda_status kda_gated_norm(const kda_gated_norm_args* a, void* stream) {
  clear();
  kda_status s = norm_check(a);
  if (s != KDA_OK) return s;
  kda::NormParams p{};
  p.x = a->x;
  p.gate = a->gate;
  p.residual = a->residual;
  p.weight = a->weight;
  p.next_weight = a->next_weight;
  p.out = a->out;
  p.next_out = a->next_out;
  p.M = a->M;
  p.G = a->G;
  p.D = static_cast<int32_t>(a->D);
  for (int d = 0; d < 2; ++d) {
    p.xs[d] = a->x_stride[d];
    p.gs[d] = a->gate_stride[d];
    p.rs[d] = a->residual_stride[d];
  }
  p.silu = a->act == KDA_ACT_SILU;
  p.eps = a->eps;
  p.scale = a->scale;
  return done(kda::launch_gated_norm(p, a->io_dtype == KDA_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

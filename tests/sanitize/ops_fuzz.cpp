// Host-side fuzz driver for the operators beside kda_prefill (kda_ops_api.cpp and
// kda_ssm_api.cpp), built with AddressSanitizer and UndefinedBehaviorSanitizer on the host
// pass: argument sets, a third of them well formed, a third with an extreme size, stride or
// pitch here and there, a third with null, misaligned or overlapping pointers and unknown
// dtypes or flags as well, go through the checks, plans, workspace sizes and launches of
// kda_linear, kda_pool_copy, kda_pool_compact, kda_gated_norm, kda_short_conv and
// kda_selective_scan. The device launches are stubs that check what the kernels assume of
// their geometry and then fail (no GPU is touched); pointers are only compared. A sanitizer
// report or a broken assumption ends the run with a non-zero status.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>

#include "kda.h"
#include "kda_ops_internal.h"
#include "kda_ssm_internal.h"

namespace {

constexpr int64_t kThreads = 0xffffffffLL;  // of one launch

uintptr_t g_workspace = 0;  // of the call that launches
size_t g_bytes = 0;
int g_launches = 0;

void need(bool ok, const char* what) {
  if (ok) return;
  std::printf("broken assumption: %s\n", what);
  std::exit(3);
}

void in_workspace(const void* p, __int128 bytes, const char* what) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  need(at >= g_workspace && static_cast<__int128>(at) - g_workspace + bytes <= static_cast<__int128>(g_bytes), what);
}

}  // namespace

namespace kda {
kda_status set_error(kda_status s, const char* text) noexcept {
  static char last[512];
  std::snprintf(last, sizeof last, "%s", text);
  return s;
}
hipError_t launch_linear_chunks(const LinParams& p, int, bool, int rows, hipStream_t) {
  ++g_launches;
  need(rows == 64 || rows == 128, "rows of a chunk launch");
  need(static_cast<__int128>(linear_grid(p)) * 512 <= kThreads, "threads of a chunk launch");
  return hipErrorInvalidValue;
}
hipError_t launch_linear_states(const LinParams& p, int k, bool, hipStream_t) {
  ++g_launches;
  need(p.segmented && p.seg_len > 0 && p.seg_len % 64 == 0, "segments of the states");
  in_workspace(p.scan_s, static_cast<__int128>(p.H) * p.slots * p.V * k * 4, "scan_s");
  in_workspace(p.scan_d, static_cast<__int128>(p.H) * p.slots * 4, "scan_d");
  return hipSuccess;
}
hipError_t launch_linear_scan(const LinParams&, int, hipStream_t) { return hipSuccess; }
hipError_t launch_linear_tokens(const LinParams& p, int, bool, int rows, hipStream_t) {
  ++g_launches;
  need(p.T >= 1 && p.T <= kLinDecodeMaxT && rows >= 16 && rows <= 64, "the token loop's geometry");
  return hipErrorInvalidValue;
}
hipError_t launch_pool_copy(const PoolCopy& p, hipStream_t) {
  ++g_launches;
  need((static_cast<__int128>(p.slot_elems) + kCopyGroup - 1) / kCopyGroup * p.layers * p.pairs * 256 <= kThreads,
       "threads of a copy");
  return hipErrorInvalidValue;
}
hipError_t launch_pool_plan(const int32_t*, int32_t*, int32_t*, int64_t n, int64_t slots,
                            int32_t* src, int32_t* dst, int32_t* moves, hipStream_t) {
  const __int128 most = n < slots ? n : slots;
  in_workspace(src, 4 * most, "moves' sources");
  in_workspace(dst, 4 * most, "moves' destinations");
  in_workspace(moves, 4, "number of moves");
  return hipSuccess;
}
hipError_t launch_gated_norm(const NormParams& p, bool, hipStream_t) {
  ++g_launches;
  need(p.D >= 8 && p.D <= kNormMax && p.D % 8 == 0, "rows of the norm");
  return hipErrorInvalidValue;
}
hipError_t launch_short_conv(const ConvParams& p, int width, bool, hipStream_t) {
  ++g_launches;
  need(width >= 2 && width <= 4 && p.C % 8 == 0, "taps and channels");
  need(p.lanes == 64 || p.lanes == 32 || p.lanes == 8, "octets of a workgroup");
  // the first run's state is read by its own thread only
  need(p.run >= (p.T <= 1 && !p.cu_seqlens ? 1 : width - 1), "run");
  const __int128 blocks = (p.C / 8 + p.lanes - 1) / p.lanes;
  need(blocks * ((static_cast<__int128>(p.slots) * p.lanes + 255) / 256) * 256 <= kThreads, "threads of a convolution");
  need(p.cu_seqlens ? p.slots == p.T / p.run + p.N
                    : p.slots == p.N * p.runs_per_seq && p.runs_per_seq * p.run >= p.T, "runs");
  return hipErrorInvalidValue;
}
namespace {
void scan_geometry(const ScanParams& p, int n) {
  need(n == 8 || n == 16 || n == 32 || n == 64, "states of a channel");
  need(p.D % 8 == 0 && p.per_group > 0 && p.D % p.per_group == 0, "channels of a group");
  need(p.per_group == p.D || p.per_group % kScanChannels == 0, "groups across workgroups");
}
void scan_chunks(const ScanParams& p, int n) {
  scan_geometry(p, n);
  need(p.cblocks * kScanChannels >= p.D && static_cast<__int128>(scan_grid(p)) * 512 <= kThreads, "threads of a scan");
  need(!p.longest_first || (p.cu_seqlens && !p.segmented && p.N >= 2 && p.N <= 64 && p.slots == p.N), "order by length");
  if (p.segmented) {
    need(p.seg_len > 0 && p.seg_len % 64 == 0 && p.seg_len < p.T, "segments");
    need(p.cu_seqlens ? p.slots == p.T / p.seg_len + p.N
                      : p.slots == p.N * p.segs_per_seq && p.segs_per_seq * p.seg_len >= p.T, "segments of a call");
    const __int128 states = static_cast<__int128>(p.D) * n * 4;
    in_workspace(p.ends, p.slots * states, "ends");
    in_workspace(p.sums, static_cast<__int128>(p.slots) * p.D * 4, "sums");
    in_workspace(p.starts, p.N * states, "starts");
    need(reinterpret_cast<uintptr_t>(p.ends) + p.slots * states <= reinterpret_cast<uintptr_t>(p.sums) &&
             reinterpret_cast<uintptr_t>(p.sums) + static_cast<__int128>(p.slots) * p.D * 4 <= reinterpret_cast<uintptr_t>(p.starts),
         "parts of the workspace");
  } else {
    need(p.seg_len > p.T && p.slots == p.N, "a slot for each sequence");
  }
}
}  // namespace
hipError_t launch_scan_ends(const ScanParams& p, int n, bool, hipStream_t) {
  need(p.segmented, "ends without segments");
  scan_chunks(p, n);
  return hipSuccess;
}
hipError_t launch_scan_outputs(const ScanParams& p, int n, bool, hipStream_t) {
  ++g_launches;
  scan_chunks(p, n);
  return hipErrorInvalidValue;
}
hipError_t launch_scan_tokens(const ScanParams& p, int n, bool, hipStream_t) {
  ++g_launches;
  scan_geometry(p, n);
  need(p.T >= 1 && p.T <= kScanTokensMaxT && !p.cu_seqlens, "tokens of a call");
  need(static_cast<__int128>(p.N) * ((p.D + 1024 / n - 1) / (1024 / n)) * 256 <= kThreads, "threads of a token call");
  return hipErrorInvalidValue;
}
}  // namespace kda

namespace {

std::mt19937_64 rng(24680);
bool g_sane = false;  // this argument set: well formed
bool g_wild = false;  // pointers as well

int64_t pick(std::initializer_list<int64_t> v) {
  return *(v.begin() + static_cast<size_t>(rng() % v.size()));
}
// `good` in a well-formed set, otherwise mostly that and sometimes one of `bad`.
int64_t size(std::initializer_list<int64_t> good, std::initializer_list<int64_t> bad) {
  return g_sane || rng() % (g_wild ? 4 : 12) ? pick(good) : pick(bad);
}

// A device address that is never read: regions 1 TiB apart.
void* fake(int i) {
  const uintptr_t at = uintptr_t(i + 1) << 40;
  if (!g_wild) return reinterpret_cast<void*>(at);
  switch (rng() % 24) {
    case 0: return nullptr;
    case 1: return reinterpret_cast<void*>(at + 8);
    case 2: return reinterpret_cast<void*>(uintptr_t(1) << 40);
    case 3: return reinterpret_cast<void*>(uintptr_t(0x7fffffffff00));
    default: return reinterpret_cast<void*>(at);
  }
}
template <typename T>
const T* fake_of(int i) { return static_cast<const T*>(fake(i)); }

int32_t dtype() { return static_cast<int32_t>(size({0, 1}, {2, -1})); }
int64_t stride(int64_t dense) { return size({0, dense, dense + 8, 3 * dense}, {-8, 4, 1 << 22, (1 << 22) + 8, INT64_MAX, INT64_MIN}); }

template <typename Args>
void sequences(Args* a) {
  const bool varlen = rng() % 3 == 0;
  a->B = varlen ? size({1}, {2, 0}) : size({1, 2, 3, 16, 256}, {0, -1, int64_t(1) << 31, int64_t(1) << 40, INT64_MAX});
  a->T = size({0, 1, 4, 8, 9, 17, 100, 256, 8192, 65536, 1000003}, {-1, int64_t(1) << 36, (int64_t(1) << 36) + 1, INT64_MAX, INT64_MIN});
  a->N = varlen ? size({1, 2, 8, 64, 65, 300}, {0, -1, int64_t(1) << 31, INT64_MAX}) : g_sane || rng() % 8 ? a->B : pick({0, 5, INT64_MAX});
  a->cu_seqlens = varlen ? fake_of<int64_t>(9) : nullptr;
}
template <typename Args>
void states(Args* a, int64_t dense) {
  a->io_dtype = dtype();
  a->state_dtype = dtype();
  a->state_in = rng() % 3 ? fake(6) : nullptr;
  a->state_out = rng() % 4 == 0 ? const_cast<void*>(a->state_in) : rng() % 3 ? fake(7) : nullptr;
  if (rng() % 4 == 0) {
    a->ssm_state_indices = fake_of<int32_t>(10);
    a->state_out_indices = rng() % 2 ? fake_of<int32_t>(11) : nullptr;
    a->state_pool_slots = size({1, 4, 1000}, {0, -1, int64_t(1) << 31, INT64_MAX});
    a->state_slot_pitch = size({0, dense, dense + 8}, {8, dense + 4, INT64_MAX, INT64_MIN});
    if (!g_wild) a->state_in = fake(6);
    if (rng() % 2) a->state_out = nullptr;
    if (!g_wild && a->state_out) a->state_out = const_cast<void*>(a->state_in);
  }
}
// Often exactly as many bytes as are needed, at an address of its own.
template <typename Args>
void workspace(Args* a, size_t bytes) {
  a->workspace = fake(8);
  a->workspace_bytes = !g_wild || rng() % 2 ? bytes : static_cast<size_t>(pick({0, 256, 1 << 20, INT64_MAX, -1}));
  g_workspace = reinterpret_cast<uintptr_t>(a->workspace);
  g_bytes = a->workspace_bytes;
}

int g_ok[6], g_no[6];
void count(int op, kda_status checked, kda_status ran) {
  need(checked == KDA_OK ? ran == KDA_ERR_HIP || ran == KDA_OK : ran == checked, "a launch refuses what its check refuses");
  ++(checked == KDA_OK ? g_ok : g_no)[op];
}

void linear() {
  kda_linear_args a;
  std::memset(&a, 0, sizeof a);
  sequences(&a);
  a.Hk = size({1, 2, 6, 24}, {0, -3, 5, INT64_MAX});
  a.H = g_sane || rng() % 4 ? a.Hk > 0 && a.Hk < 100 ? a.Hk * pick({1, 2, 4}) : 6 : pick({0, 7, 65536, INT64_MAX});
  a.K = size({64, 128}, {0, 96, INT64_MAX});
  a.V = size({64, 128, 512}, {0, 65, 1024, INT64_MAX});
  const bool whole = a.K > 0 && a.K <= 128 && a.V > 0 && a.V <= 1024 && a.H > 0 && a.H <= 65536;
  states(&a, whole ? a.H * a.V * a.K : 128);
  a.q = fake(0); a.k = fake(1); a.v = fake(2); a.o = fake(5);
  a.g = rng() % 2 ? fake(3) : nullptr;
  a.log_decay = rng() % 2 ? fake_of<float>(4) : nullptr;
  for (int d = 0; d < 3; ++d) a.q_stride[d] = stride(128), a.k_stride[d] = stride(256), a.v_stride[d] = stride(512);
  a.g_dtype = dtype();
  a.scale = static_cast<float>(size({0, 1}, {-1}));
  a.segment_tokens = size({0, 0, -1, 64, 192}, {1, 1 << 30, int64_t(1) << 40, INT64_MAX, INT64_MIN});
  size_t bytes = 0;
  (void)kda_linear_workspace_bytes(&a, &bytes);
  workspace(&a, bytes);
  kda_linear_plan_info info;
  (void)kda_linear_plan(&a, &info);
  const kda_status s = kda_linear_check(&a);
  count(0, s, kda_linear(&a, nullptr));
}

kda_pool pool(int i) {
  kda_pool p;
  std::memset(&p, 0, sizeof p);
  p.base = fake(i);
  p.slots = size({1, 8, 512}, {0, -1, 1 << 18, (1 << 18) + 1, int64_t(1) << 31, INT64_MAX});
  p.layers = size({1, 2, 48}, {0, 1 << 20, INT64_MAX});
  p.slot_elems = size({8, 16384, 98304}, {0, 12, int64_t(1) << 40, INT64_MAX});
  const int64_t e = p.slot_elems > 0 && p.slot_elems < (int64_t(1) << 40) ? p.slot_elems : 8;
  p.slot_pitch = size({e, e + 8, 48 * e}, {0, e - 8, int64_t(1) << 40, INT64_MAX, INT64_MIN});
  const int64_t all = p.slots > 0 && p.slots < 1000 && p.slot_pitch > 0 && p.slot_pitch < (1 << 30) ? p.slots * p.slot_pitch : 8;
  p.layer_pitch = size({all, all + 64}, {e, 0, 8, INT64_MAX, INT64_MIN, int64_t(1) << 50});
  p.dtype = dtype();
  return p;
}
void copy() {
  kda_pool_copy_args a;
  std::memset(&a, 0, sizeof a);
  a.src = pool(0);
  a.dst = rng() % 3 ? pool(1) : a.src;
  if (g_sane) {
    a.dst.layers = a.src.layers;
    a.dst.slot_elems = a.src.slot_elems;
    a.dst.slot_pitch = a.src.slot_pitch;
    a.dst.layer_pitch = a.dst.slots * a.dst.slot_pitch;
  }
  a.src_idx = fake_of<int32_t>(10);
  a.dst_idx = fake_of<int32_t>(11);
  a.pairs = size({0, 1, 48}, {-1, 1 << 24, int64_t(1) << 31, INT64_MAX});
  const kda_status s = kda_pool_copy_check(&a);
  count(1, s, kda_pool_copy(&a, nullptr));
}
void compact() {
  kda_pool_compact_args a;
  std::memset(&a, 0, sizeof a);
  a.pool = pool(0);
  a.idx = fake_of<int32_t>(10);
  a.new_idx = rng() % 3 ? static_cast<int32_t*>(fake(11)) : const_cast<int32_t*>(a.idx);
  a.count = static_cast<int32_t*>(fake(12));
  a.n = size({0, 1, 64, 700}, {-1, 1 << 30, int64_t(1) << 31, INT64_MAX});
  size_t bytes = 0;
  (void)kda_pool_compact_workspace_bytes(&a, &bytes);
  workspace(&a, bytes);
  const kda_status s = kda_pool_compact_check(&a);
  count(2, s, kda_pool_compact(&a, nullptr));
}
void norm() {
  kda_gated_norm_args a;
  std::memset(&a, 0, sizeof a);
  a.M = size({0, 1, 64, 8192}, {-1, int64_t(1) << 40, INT64_MAX});
  a.G = size({1, 24}, {0, int64_t(1) << 40, INT64_MAX});
  a.D = size({8, 128, 12288, 16384}, {0, 12, 16392, INT64_MAX});
  a.x = fake(0);
  a.gate = rng() % 2 ? fake(1) : nullptr;
  a.residual = rng() % 2 ? fake(2) : nullptr;
  a.weight = rng() % 2 ? fake_of<float>(3) : nullptr;
  a.out = rng() % 4 ? fake(5) : const_cast<void*>(a.x);
  a.next_out = rng() % 2 ? fake(7) : nullptr;
  a.next_weight = a.next_out && rng() % 2 ? fake_of<float>(4) : nullptr;
  const int64_t d = a.D > 0 && a.D < 20000 ? a.D : 8, g = a.G > 0 && a.G < 100 ? a.G : 1;
  for (int64_t* st : {a.x_stride, a.gate_stride, a.residual_stride}) st[0] = stride(d * g), st[1] = stride(d);
  a.io_dtype = dtype();
  a.act = static_cast<int32_t>(size({0, 1}, {2}));
  a.eps = 1e-6f;
  a.scale = 1.f;
  const kda_status s = kda_gated_norm_check(&a);
  count(3, s, kda_gated_norm(&a, nullptr));
}

void conv() {
  kda_short_conv_args a;
  std::memset(&a, 0, sizeof a);
  sequences(&a);
  a.C = size({8, 72, 2304, 36864, 1 << 22}, {0, 12, -8, (1 << 22) + 8, INT64_MAX});
  a.W = size({2, 3, 4}, {0, 1, 5, INT64_MAX});
  states(&a, a.C > 0 && a.C <= (1 << 22) && a.W > 0 && a.W < 8 ? (a.W - 1) * a.C : 8);
  a.x = fake(0); a.out = fake(5);
  a.weight = fake_of<float>(1);
  a.bias = rng() % 2 ? fake_of<float>(2) : nullptr;
  a.x_stride[0] = stride(4096);
  a.x_stride[1] = stride(2304);
  a.flags = static_cast<int32_t>(size({0, 1}, {2, -1}));
  const kda_status s = kda_short_conv_check(&a);
  count(4, s, kda_short_conv(&a, nullptr));
}
void scan() {
  kda_selective_scan_args a;
  std::memset(&a, 0, sizeof a);
  sequences(&a);
  a.S = size({8, 16, 32, 64}, {0, 1, 24, 128, INT64_MAX, INT64_MIN});
  a.G = size({1, 1, 2, 3}, {0, -1, 7, 1 << 22, INT64_MAX});
  a.D = size({192, 384, 1536, 8256}, {0, 8, 100, 1 << 22, (1 << 22) + 8, INT64_MAX});
  states(&a, a.D > 0 && a.D <= (1 << 22) && a.S > 0 && a.S <= 128 ? a.D * a.S : 8);
  a.u = fake(0); a.delta = fake(1); a.B_in = fake(2); a.C_in = fake(3); a.out = fake(5);
  a.z = rng() % 2 ? fake(4) : nullptr;
  a.A = fake_of<float>(12);
  a.D_skip = rng() % 2 ? fake_of<float>(13) : nullptr;
  a.delta_bias = rng() % 2 ? fake_of<float>(14) : nullptr;
  for (int64_t* st : {a.u_stride, a.delta_stride, a.z_stride}) st[0] = stride(4096), st[1] = stride(1536);
  for (int64_t* st : {a.B_stride, a.C_stride}) st[0] = stride(4096), st[1] = stride(64), st[2] = stride(16);
  a.flags = static_cast<int32_t>(size({0, 1}, {2, -1}));
  a.segment_tokens = size({0, 0, -1, 64, 192}, {1, 1 << 30, int64_t(1) << 40, INT64_MAX, INT64_MIN});
  size_t bytes = 0;
  const kda_status sized = kda_selective_scan_workspace_bytes(&a, &bytes);
  workspace(&a, bytes);
  kda_selective_scan_plan_info info;
  const kda_status planned = kda_selective_scan_plan(&a, &info);
  need(sized == planned && (sized != KDA_OK || info.workspace_bytes == bytes), "plan and workspace size agree");
  const kda_status s = kda_selective_scan_check(&a);
  need(s != KDA_OK || sized == KDA_OK, "a call that passes has a workspace size");
  count(5, s, kda_selective_scan(&a, nullptr));
}

}  // namespace

int main(int argc, char** argv) {
  const int iters = argc > 1 ? std::atoi(argv[1]) : 20000;
  void (*const ops[])() = {linear, copy, compact, norm, conv, scan};
  const char* const names[] = {"linear", "copy", "compact", "norm", "conv", "scan"};
  for (int it = 0; it < iters; ++it) {
    for (auto* op : ops) {
      g_sane = rng() % 3 == 0;
      g_wild = !g_sane && rng() % 2;
      g_workspace = 0;
      g_bytes = 0;
      op();
    }
  }
  bool both = g_launches > 0;
  for (int i = 0; i < 6; ++i) {
    std::printf("fuzz %s: %d argument sets accepted, %d rejected\n", names[i], g_ok[i], g_no[i]);
    both = both && g_ok[i] > iters / 8 && g_no[i] > iters / 16;
  }
  return both ? 0 : 2;
}

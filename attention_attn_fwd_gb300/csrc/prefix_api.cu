// C ABI of the attention behind a shared prefix: argument checks, the choice
// of kernels and launches.  No device memory is allocated here.
#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/attn.h"
#include "attn_host.h"
#include "prefix_common.cuh"

namespace {

using attn::prefix::PrefixParams;

constexpr size_t kWorkspaceAlign = 256;

size_t round_up(size_t x) {
  return (x + kWorkspaceAlign - 1) / kWorkspaceAlign * kWorkspaceAlign;
}

bool misaligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) != 0;
}

struct Range {
  const void* p;
  size_t n;
};

bool any_overlap(const Range& a, const Range* others, int count) {
  for (int i = 0; i < count; ++i)
    if (attn::ranges_overlap(a.p, a.n, others[i].p, others[i].n)) return true;
  return false;
}

struct Sizes {
  int B, Hq, Hkv, Sq, prefix_capacity, capacity, D;
};

attn_status_t check_sizes(const Sizes& z) {
  if (z.B < 0 || z.Hkv <= 0 || z.Hq <= 0 || z.Hq % z.Hkv != 0 || z.Sq < 0 ||
      z.prefix_capacity < 1 || z.capacity < 1 || z.D <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (z.D != 64 && z.D != 128) return ATTN_ERR_UNSUPPORTED;
  if (z.Hq / z.Hkv > attn::prefix::kTM) return ATTN_ERR_UNSUPPORTED;
  // Counts of tokens, tiles and rows stay within int32 with a tile behind.
  constexpr long long kMost = 0x7fffffffLL - (1 << 16);
  if (z.prefix_capacity >= kMost || z.capacity >= kMost ||
      static_cast<long long>(z.B) * z.Hkv >= (1 << 24))
    return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

// How the rows of a K/V head meet the keys; see Mode.  Rows of a sequence that
// fill a tile are not packed with others': packed, their results over the
// prefix and over their own keys have to meet in memory.
struct Plan {
  int mode;
  long long rows;        // R
  int tile_seqs, tile_rows;
  long long pack_blocks, row_blocks;
  int grid;
};

long long units_of(long long tiles) { return (tiles + 1) / 2; }

Plan make_plan(const Sizes& z, int sms) {
  constexpr int kTM = attn::prefix::kTM;
  Plan p;
  const int group = z.Hq / z.Hkv;
  p.rows = static_cast<long long>(group) * z.Sq;
  const long long few =
      4LL * z.B * z.Hkv > sms || z.B == 1 ? 16 : 8;  // see Mode
  p.mode = p.rows <= few              ? attn::prefix::kFew
           : p.rows > kTM || z.B == 1 ? attn::prefix::kJoint
                                      : attn::prefix::kPacked;
  p.tile_seqs =
      p.mode == attn::prefix::kJoint ? 1 : static_cast<int>(kTM / p.rows);
  p.tile_rows = kTM / group * group;
  if (p.tile_rows > p.rows) p.tile_rows = static_cast<int>(p.rows);
  p.pack_blocks = p.mode == attn::prefix::kJoint
                      ? 0
                      : units_of((z.B + p.tile_seqs - 1) / p.tile_seqs);
  p.row_blocks = p.mode == attn::prefix::kFew
                     ? 0
                     : units_of((p.rows + p.tile_rows - 1) / p.tile_rows);
  // (One for the prefix, one for own keys; the merge counts on 224 at most.)
  p.grid = std::min(std::max(sms, 2), 224);
  return p;
}

// Whether the kernels' counts of rows and list places fit 32 bits.
bool counts_fit(const Sizes& z, const Plan& p) {
  const long long kMost = 0x7fffffffLL - 4096;
  if (p.rows > kMost || z.B * p.rows > kMost) return false;
  const double tiles = z.prefix_capacity / 128.0 + z.capacity / 128.0 + 16;
  const double units =
      static_cast<double>(z.Hkv) * (p.pack_blocks + z.B * p.row_blocks);
  if (units * tiles > kMost) return false;
  const double few = static_cast<double>(z.B) * z.Hkv *
                     (z.capacity / (2048.0 / z.D) + 16);
  return p.mode != attn::prefix::kFew || few <= kMost;
}

struct Workspace {
  size_t base_o, base_lse2, slot_o, slot_lse2, info, split;
  size_t few_o, few_lse2, own_info;
  size_t total;
};

Workspace workspace_layout(const Sizes& z, const Plan& p) {
  const bool joint = p.mode == attn::prefix::kJoint;
  const size_t row = static_cast<size_t>(z.D) * 4;
  const size_t all = static_cast<size_t>(z.B) * z.Hkv * p.rows;
  const size_t base = joint ? 0 : p.mode == attn::prefix::kFew ? all : 2 * all;
  const size_t slots = static_cast<size_t>(p.grid) * (joint ? 2 : 1) *
                       attn::prefix::kUnitRows;
  const size_t units =
      joint ? 0
            : static_cast<size_t>(p.pack_blocks + z.B * p.row_blocks) * z.Hkv;
  const size_t few =
      p.mode == attn::prefix::kFew
          ? (static_cast<size_t>(p.grid) * attn::prefix::kFewWarps +
             static_cast<size_t>(z.B) * z.Hkv) *
                attn::prefix::few_rows(static_cast<int>(p.rows))
          : 0;
  Workspace w;
  w.base_o = 0;
  w.base_lse2 = w.base_o + round_up(base * row);
  w.slot_o = w.base_lse2 + round_up(base * 4);
  w.slot_lse2 = w.slot_o + round_up(slots * row);
  w.info = w.slot_lse2 + round_up(slots * 4);
  w.split = w.info + round_up(units * 8);
  w.few_o = w.split + (joint ? round_up(p.grid * size_t(16)) : 0);
  w.few_lse2 = w.few_o + round_up(few * row);
  w.own_info = w.few_lse2 + round_up(few * 4);
  w.total = w.own_info +
            (few ? round_up(static_cast<size_t>(z.B) * z.Hkv * 8) : 0);
  return w;
}

int current_sms() {
  int dev = -1, sms = 0;
  if (cudaGetDevice(&dev) == cudaSuccess) sms = attn::device_sms(dev);
  cudaGetLastError();  // no device: not an error of the caller's
  return sms > 0 ? sms : 152;  // a GB300's without a device
}

attn_status_t fwd_impl(const attn_prefix_cache_t* c, const void* Q, void* O,
                       float* LSE, int Hq, int Sq, const int* new_lens,
                       float scale, int causal, attn_dtype_t dtype,
                       void* workspace, size_t workspace_bytes,
                       cudaStream_t stream, unsigned long long timeout_ns = 0,
                       int hold_keys = -1, int hold_rows = -1) {
  if (c == nullptr) return ATTN_ERR_INVALID_ARG;
  const Sizes z{c->B, Hq, c->Hkv, Sq, c->prefix_capacity, c->capacity, c->D};
  attn_status_t st = check_sizes(z);
  if (st != ATTN_OK) return st;
  if (!std::isfinite(scale) || (dtype != ATTN_F16 && dtype != ATTN_BF16))
    return ATTN_ERR_INVALID_ARG;
  if (z.B == 0 || Sq == 0) return ATTN_OK;
  const void* need[] = {c->prefix_k, c->prefix_v, c->prefix_len, c->k,
                        c->v,        c->lens,     Q,             O};
  for (const void* x : need)
    if (x == nullptr) return ATTN_ERR_INVALID_ARG;
  if (misaligned(c->prefix_k, 16) || misaligned(c->prefix_v, 16) ||
      misaligned(c->k, 16) || misaligned(c->v, 16) || misaligned(Q, 16) ||
      misaligned(O, 16) || misaligned(c->prefix_len, 4) ||
      misaligned(c->lens, 4) || misaligned(LSE, 4) || misaligned(new_lens, 4))
    return ATTN_ERR_ALIGNMENT;
  if (workspace == nullptr || misaligned(workspace, kWorkspaceAlign))
    return ATTN_ERR_ALIGNMENT;
  const Plan plan = make_plan(z, current_sms());
  if (!counts_fit(z, plan)) return ATTN_ERR_INVALID_ARG;
  const Workspace w = workspace_layout(z, plan);
  if (workspace_bytes < w.total) return ATTN_ERR_INVALID_ARG;
  const size_t rows = static_cast<size_t>(z.B) * Hq * Sq;
  const size_t head = static_cast<size_t>(z.D) * 2;
  const size_t pre = static_cast<size_t>(z.Hkv) * z.prefix_capacity * head;
  const size_t own = static_cast<size_t>(z.B) * z.Hkv * z.capacity * head;
  const size_t len_bytes = static_cast<size_t>(z.B) * 4;
  const Range in[] = {{c->prefix_k, pre}, {c->prefix_v, pre},
                      {c->prefix_len, 4}, {c->k, own},
                      {c->v, own},        {c->lens, len_bytes},
                      {Q, rows * head},
                      {new_lens, new_lens ? len_bytes : 0}};
  const Range out[] = {{O, rows * head},
                       {LSE, LSE ? rows * 4 : 0},
                       {workspace, w.total}};
  for (int i = 0; i < 3; ++i)
    if (any_overlap(out[i], in, 8) || any_overlap(out[i], out + i + 1, 2 - i))
      return ATTN_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_CUDA;
  const void* more[] = {LSE, new_lens, workspace};
  for (const void* x : need)
    if (!attn::on_device(x, dev)) return ATTN_ERR_INVALID_ARG;
  for (const void* x : more)
    if (x != nullptr && !attn::on_device(x, dev)) return ATTN_ERR_INVALID_ARG;
  PrefixParams p{};
  p.k = static_cast<const uint16_t*>(c->k);
  p.v = static_cast<const uint16_t*>(c->v);
  p.plen = c->prefix_len;
  p.lens = c->lens;
  p.new_lens = new_lens;
  p.q = static_cast<const uint16_t*>(Q);
  p.o = static_cast<uint16_t*>(O);
  p.lse = LSE;
  p.B = z.B;
  p.Hq = Hq;
  p.Hkv = z.Hkv;
  p.Sq = Sq;
  p.prefix_capacity = z.prefix_capacity;
  p.capacity = z.capacity;
  p.group = Hq / z.Hkv;
  p.rows = static_cast<int>(plan.rows);
  p.mode = plan.mode;
  p.causal = causal != 0;
  p.pack_blocks = static_cast<int>(plan.pack_blocks);
  p.row_blocks = static_cast<int>(plan.row_blocks);
  p.tile_seqs = plan.tile_seqs;
  p.tile_rows = plan.tile_rows;
  p.scale_log2 = std::fabs(scale) * 1.4426950408889634f;
  p.negate = scale < 0.f;
  char* ws = static_cast<char*>(workspace);
  p.base_o = reinterpret_cast<float*>(ws + w.base_o);
  p.base_lse2 = reinterpret_cast<float*>(ws + w.base_lse2);
  p.slot_o = reinterpret_cast<float*>(ws + w.slot_o);
  p.slot_lse2 = reinterpret_cast<float*>(ws + w.slot_lse2);
  p.info = reinterpret_cast<int2*>(ws + w.info);
  p.split = reinterpret_cast<int4*>(ws + w.split);
  p.few_o = reinterpret_cast<float*>(ws + w.few_o);
  p.few_lse2 = reinterpret_cast<float*>(ws + w.few_lse2);
  p.own_info = reinterpret_cast<int2*>(ws + w.own_info);
  p.grid = plan.grid;
  p.fd_group = attn::make_fast_div(p.group);
  p.fd_rows = attn::make_fast_div(p.rows);
  p.fd_blocks = attn::make_fast_div(p.row_blocks > 0 ? p.row_blocks : 1);
  p.fd_hkv = attn::make_fast_div(p.Hkv);
  p.fd_tile_seqs = attn::make_fast_div(p.tile_seqs);
  p.hold_keys = hold_keys;
  p.hold_rows = hold_rows;
  p.timeout_ns = timeout_ns != 0 ? timeout_ns : attn::wait_timeout_ns();
  p.status = attn::device_status_word(dev);
  if (p.status == nullptr) return ATTN_ERR_CUDA;
  const bool bf16 = dtype == ATTN_BF16;
  // (The many-row kernel reads a sequence's own keys only where it works on
  // them.)
  CUtensorMap maps[9];
  const bool joint = plan.mode == attn::prefix::kJoint;
  if (!attn::make_rows_map(&maps[8], Q, bf16, z.D, Sq, Hq, z.B, p.group,
                           joint ? p.tile_rows / p.group : Sq, p.tile_seqs))
    return ATTN_ERR_CUDA;
  const void* bases[] = {c->prefix_k, c->prefix_v, c->k, c->v};
  for (int i = 0; i < 4; ++i) {
    const bool is_own = i >= 2;
    for (int tail = 0; tail < 2; ++tail) {
      CUtensorMap* m = &maps[(is_own ? 4 : 0) + 2 * tail + i % 2];
      if (is_own && plan.mode == attn::prefix::kFew)
        *m = maps[2 * tail + i % 2];
      else if (!attn::make_tile_map(
                   m, bases[i], bf16, z.D,
                   is_own ? z.capacity : z.prefix_capacity,
                   is_own ? static_cast<long long>(z.B) * z.Hkv : z.Hkv,
                   tail ? attn::prefix::kTailRows : attn::prefix::kTN))
        return ATTN_ERR_CUDA;
    }
  }
  cudaError_t err = attn::prefix::launch_many(z.D, bf16, p, maps, stream);
  if (err == cudaSuccess)
    err = attn::prefix::launch_merge(z.D, bf16, p, stream);
  return err == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

extern "C" {

attn_status_t attn_prefix_fwd(const attn_prefix_cache_t* cache, const void* Q,
                              void* O, float* LSE, int Hq, int Sq,
                              const int* new_lens, float scale, int causal,
                              attn_dtype_t dtype, void* workspace,
                              size_t workspace_bytes, attn_stream_t stream) {
  return fwd_impl(cache, Q, O, LSE, Hq, Sq, new_lens, scale, causal, dtype,
                  workspace, workspace_bytes,
                  reinterpret_cast<cudaStream_t>(stream));
}

attn_status_t attn_selftest_prefix_timeout(
    const attn_prefix_cache_t* cache, const void* Q, void* O, float* LSE,
    int Hq, int Sq, const int* new_lens, float scale, int causal,
    attn_dtype_t dtype, void* workspace, size_t workspace_bytes,
    int block, int query_rows, unsigned long long timeout_ns,
    attn_stream_t stream) {
  if (timeout_ns == 0 || block < 0) return ATTN_ERR_INVALID_ARG;
  return fwd_impl(cache, Q, O, LSE, Hq, Sq, new_lens, scale, causal, dtype,
                  workspace, workspace_bytes,
                  reinterpret_cast<cudaStream_t>(stream), timeout_ns,
                  query_rows != 0 ? -1 : block, query_rows != 0 ? block : -1);
}

size_t attn_prefix_workspace_bytes(int B, int Hq, int Hkv, int Sq,
                                   int prefix_capacity, int capacity, int D) {
  const Sizes z{B, Hq, Hkv, Sq, prefix_capacity, capacity, D};
  if (check_sizes(z) != ATTN_OK || B == 0 || Sq == 0) return 0;
  const Plan plan = make_plan(z, current_sms());
  if (!counts_fit(z, plan)) return 0;
  return workspace_layout(z, plan).total;
}

}  // extern "C"

// C ABI of the 8-bit KV cache: argument checks and launches of append,
// attention and eviction.  No device memory is allocated here.
#include <cmath>
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/attn.h"
#include "kv8_common.cuh"

namespace {

constexpr size_t kWorkspaceAlign = 256;
constexpr int kKeyTile = 128;  // keys of the many-row kernels' tiles

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

int block_shift(int block) {
  return block == 16 ? 4 : block == 32 ? 5 : block == 64 ? 6 : 7;
}

size_t heads(const attn_kv8_t& c) {
  return static_cast<size_t>(c.B) * c.Hkv;
}
int blocks(const attn_kv8_t& c) {
  return (c.capacity - 1) / c.block + 1;
}
size_t code_bytes(const attn_kv8_t& c) {
  return heads(c) * c.capacity * c.D;
}
size_t scale_bytes(const attn_kv8_t& c) {
  return heads(c) * blocks(c) * 4;
}

// Sizes of a cache.
attn_status_t check_cache_sizes(const attn_kv8_t* c) {
  if (c == nullptr) return ATTN_ERR_INVALID_ARG;
  if (c->B < 0 || c->Hkv <= 0 || c->capacity <= 0 || c->D <= 0 ||
      c->block <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(c->B) * c->Hkv >= (1 << 24))
    return ATTN_ERR_INVALID_ARG;
  // Places that the kernels count to behind a length (a turn of the select
  // kernel or an in-place round of moved weights, 16384 tokens each, at most)
  // must stay within int32.  Sums of two token counts are not among them: they
  // are taken by kv8_index.h.
  if (c->capacity >= 0x7fffffff - (1 << 16)) return ATTN_ERR_INVALID_ARG;
  if (c->D != 64 && c->D != 128) return ATTN_ERR_UNSUPPORTED;
  if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128)
    return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

// NULL and misaligned pointers (found without a device).
attn_status_t check_cache_pointers(const attn_kv8_t& c) {
  const void* p[] = {c.k, c.v, c.k_scale, c.v_scale, c.lens};
  for (const void* x : p)
    if (x == nullptr) return ATTN_ERR_INVALID_ARG;
  if (misaligned(c.k, 16) || misaligned(c.v, 16) || misaligned(c.k_scale, 4) ||
      misaligned(c.v_scale, 4) || misaligned(c.lens, 4))
    return ATTN_ERR_ALIGNMENT;
  return ATTN_OK;
}

// Every non-NULL pointer is memory of the current device.
bool all_on_device(const attn_kv8_t& c, const void* const* more, int count,
                   int dev) {
  const void* p[] = {c.k, c.v, c.k_scale, c.v_scale, c.lens};
  for (const void* x : p)
    if (!attn::on_device(x, dev)) return false;
  for (int i = 0; i < count; ++i)
    if (more[i] != nullptr && !attn::on_device(more[i], dev)) return false;
  return true;
}

// How the query rows of a K/V head are worked on: up to 16 by the decode
// kernels (8 or 16 a CTA; bound by the codes' bytes), more by the tcgen05
// kernel in units of 256.  At 16 rows decode against tcgen05: 26 / 37 us on
// 8 x 4096 tokens of 8 heads, 54 / 99 on 131072 of 8, 10 / 14 on 2000 of 2
// (D = 128), 20 / 36 on 16 x 1024 of 16 (D = 64).  At 20 to 32 rows, where
// decode would take two passes of that, tcgen05 takes the same 37 to 38, 99,
// 14 and 36.
struct RowPlan {
  long long rows;   // query rows per (batch, K/V head)
  int tile;         // rows a CTA holds: 8, 16 or 256
  long long blocks; // units of 256 rows (1 for few rows)
  int grid;         // CTAs of the forward launch
};

constexpr int kFewRows = 16;

RowPlan plan_rows(int Hq, int Hkv, int Sq, int D, int sms) {
  RowPlan r;
  r.rows = static_cast<long long>(Hq / Hkv) * Sq;
  r.tile = r.rows <= 8 ? 8 : r.rows <= kFewRows ? kFewRows : 256;
  r.blocks = r.tile == 256 ? (r.rows + 255) / 256 : 1;
  r.grid = sms * (r.tile <= kFewRows ? attn::kv8::decode_ctas(D, r.tile) : 1);
  return r;
}

struct Workspace {
  size_t part_o, part_ml, scores, split, lse2, total;
};

// log2 of the scores kept per key: the rows, padded to a power of two.
int score_shift(const RowPlan& r) {
  int s = 0;
  while ((1 << s) < r.rows) ++s;
  return s;
}

Workspace workspace_layout(int B, int Hkv, int capacity, int D,
                           const RowPlan& r, bool weights) {
  const size_t bh = static_cast<size_t>(B) * Hkv;
  const bool few = r.tile <= kFewRows;
  const size_t slots = few ? r.grid + bh : 2 * static_cast<size_t>(r.grid);
  Workspace w;
  w.part_o = 0;
  w.part_ml = w.part_o + round_up(slots * r.tile * D * 4);
  w.scores = w.part_ml + round_up(slots * r.tile * (few ? 4 : 8));
  w.split = w.scores +
            (few && weights ? round_up(bh * capacity * 4 << score_shift(r))
                              : 0);
  w.lse2 = w.split + (few ? 0 : round_up(static_cast<size_t>(r.grid) * 16));
  w.total = w.lse2 +
            (!few && weights ? round_up(bh * r.blocks * r.tile * 4) : 0);
  return w;
}

int current_sms() {
  int dev = -1, sms = 0;
  if (cudaGetDevice(&dev) == cudaSuccess) sms = attn::device_sms(dev);
  cudaGetLastError();  // no device: not an error of the caller's
  return sms > 0 ? sms : 152;  // a GB300's without a device
}

attn_status_t append_impl(const attn_kv8_t* c, const void* K, const void* V,
                          int Sq, const int* new_lens, attn_dtype_t dtype,
                          attn_stream_t stream) {
  attn_status_t st = check_cache_sizes(c);
  if (st != ATTN_OK) return st;
  if (Sq < 0 || (dtype != ATTN_F16 && dtype != ATTN_BF16))
    return ATTN_ERR_INVALID_ARG;
  if (c->B == 0 || Sq == 0) return ATTN_OK;
  if (Sq > c->capacity) return ATTN_ERR_INVALID_ARG;
  st = check_cache_pointers(*c);
  if (st != ATTN_OK) return st;
  if (K == nullptr || V == nullptr) return ATTN_ERR_INVALID_ARG;
  if (misaligned(K, 16) || misaligned(V, 16) || misaligned(new_lens, 4))
    return ATTN_ERR_ALIGNMENT;
  const size_t x_bytes = heads(*c) * Sq * c->D * 2;
  const Range in[] = {{K, x_bytes},
                      {V, x_bytes},
                      {c->lens, static_cast<size_t>(c->B) * 4},
                      {new_lens, new_lens ? static_cast<size_t>(c->B) * 4 : 0}};
  const Range out[] = {{c->k, code_bytes(*c)},
                       {c->v, code_bytes(*c)},
                       {c->k_scale, scale_bytes(*c)},
                       {c->v_scale, scale_bytes(*c)}};
  for (int i = 0; i < 4; ++i)
    if (any_overlap(out[i], in, 4) || any_overlap(out[i], out + i + 1, 3 - i))
      return ATTN_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_CUDA;
  const void* mem[] = {K, V, new_lens};
  if (!all_on_device(*c, mem, 3, dev)) return ATTN_ERR_INVALID_ARG;
  attn::kv8::AppendParams p{};
  p.code[0] = static_cast<uint8_t*>(c->k);
  p.code[1] = static_cast<uint8_t*>(c->v);
  p.scale[0] = c->k_scale;
  p.scale[1] = c->v_scale;
  p.x[0] = K;
  p.x[1] = V;
  p.lens = c->lens;
  p.new_lens = new_lens;
  p.Hkv = c->Hkv;
  p.Sq = Sq;
  p.capacity = c->capacity;
  p.nblk = blocks(*c);
  // Sq tokens that start anywhere in a block touch so many blocks at most.
  const long long units = (static_cast<long long>(Sq) + c->block - 2) / c->block + 1;
  p.units_per_seq = static_cast<int>(units);
  if (static_cast<long long>(heads(*c)) * units > 0x7fffffffLL / 2)
    return ATTN_ERR_INVALID_ARG;
  p.status = attn::device_status_word(dev);
  if (p.status == nullptr) return ATTN_ERR_CUDA;
  const cudaError_t err = attn::kv8::launch_append(
      c->D, c->block, dtype == ATTN_BF16, p, c->B,
      reinterpret_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t fwd_impl(const attn_kv8_t* c, const void* Q, void* O, float* LSE,
                       float* weights, int Hq, int Sq, const int* new_lens,
                       float scale, int causal, attn_dtype_t dtype,
                       void* workspace, size_t workspace_bytes,
                       attn_stream_t stream) {
  attn_status_t st = check_cache_sizes(c);
  if (st != ATTN_OK) return st;
  if (Hq <= 0 || Hq % c->Hkv != 0 || Sq < 0 || !std::isfinite(scale) ||
      (dtype != ATTN_F16 && dtype != ATTN_BF16))
    return ATTN_ERR_INVALID_ARG;
  if (c->B == 0 || Sq == 0) return ATTN_OK;
  st = check_cache_pointers(*c);
  if (st != ATTN_OK) return st;
  if (Q == nullptr || O == nullptr) return ATTN_ERR_INVALID_ARG;
  if (misaligned(Q, 16) || misaligned(O, 16) || misaligned(LSE, 4) ||
      misaligned(weights, 4) || misaligned(new_lens, 4))
    return ATTN_ERR_ALIGNMENT;
  if (workspace == nullptr || misaligned(workspace, kWorkspaceAlign))
    return ATTN_ERR_ALIGNMENT;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_CUDA;
  const int sms = attn::device_sms(dev);
  if (sms <= 0) return ATTN_ERR_CUDA;
  const RowPlan rp = plan_rows(Hq, c->Hkv, Sq, c->D, sms);
  // Rows, CTAs of every launch, and steps (unit, key tile) fit 32 bits.
  const long long segs = static_cast<long long>(heads(*c)) * rp.blocks;
  const long long tiles = (c->capacity - 1LL) / kKeyTile + 1;
  if (rp.rows > 0x7fffffffLL - 1024 || segs > 0x7fffffffLL / (16 + tiles))
    return ATTN_ERR_INVALID_ARG;
  const Workspace w = workspace_layout(c->B, c->Hkv, c->capacity, c->D, rp,
                                       weights != nullptr);
  if (workspace_bytes < w.total) return ATTN_ERR_INVALID_ARG;
  const size_t rows = static_cast<size_t>(c->B) * Hq * Sq;
  const size_t len_bytes = static_cast<size_t>(c->B) * 4;
  const Range in[] = {{c->k, code_bytes(*c)},      {c->v, code_bytes(*c)},
                      {c->k_scale, scale_bytes(*c)}, {c->v_scale, scale_bytes(*c)},
                      {c->lens, len_bytes},        {Q, rows * c->D * 2},
                      {new_lens, new_lens ? len_bytes : 0}};
  const Range out[] = {{O, rows * c->D * 2},
                       {LSE, LSE ? rows * 4 : 0},
                       {weights, weights ? heads(*c) * c->capacity * 4 : 0},
                       {workspace, w.total}};
  for (int i = 0; i < 4; ++i)
    if (any_overlap(out[i], in, 7) || any_overlap(out[i], out + i + 1, 3 - i))
      return ATTN_ERR_INVALID_ARG;
  const void* mem[] = {Q, O, LSE, weights, workspace, new_lens};
  if (!all_on_device(*c, mem, 6, dev)) return ATTN_ERR_INVALID_ARG;
  attn::kv8::FwdParams p{};
  p.k = static_cast<const uint8_t*>(c->k);
  p.v = static_cast<const uint8_t*>(c->v);
  p.k_scale = c->k_scale;
  p.v_scale = c->v_scale;
  p.lens = c->lens;
  p.new_lens = new_lens;
  p.q = Q;
  p.o = O;
  p.lse = LSE;
  p.weights = weights;
  p.B = c->B;
  p.Hq = Hq;
  p.Hkv = c->Hkv;
  p.Sq = Sq;
  p.capacity = c->capacity;
  p.nblk = blocks(*c);
  p.block_shift = block_shift(c->block);
  p.group = Hq / c->Hkv;
  p.row_blocks = static_cast<int>(rp.blocks);
  p.causal = causal != 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  char* ws = static_cast<char*>(workspace);
  p.part_o = reinterpret_cast<float*>(ws + w.part_o);
  const bool few = rp.tile <= kFewRows;
  if (few)
    p.part_lse2 = reinterpret_cast<float*>(ws + w.part_ml);
  else
    p.part_ml = reinterpret_cast<float2*>(ws + w.part_ml);
  if (weights != nullptr && few) {
    p.scores = reinterpret_cast<float*>(ws + w.scores);
    p.score_shift = score_shift(rp);
  }
  if (weights != nullptr && !few)
    p.lse2 = reinterpret_cast<float*>(ws + w.lse2);
  p.split = reinterpret_cast<int4*>(ws + w.split);
  p.grid = rp.grid;
  p.timeout_ns = attn::wait_timeout_ns();
  p.status = attn::device_status_word(dev);
  if (p.status == nullptr) return ATTN_ERR_CUDA;
  const bool bf16 = dtype == ATTN_BF16;
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t err;
  if (few) {
    err = attn::kv8::launch_decode(c->D, bf16, rp.tile, p, cs);
  } else {
    err = attn::kv8::launch_prefill(c->D, bf16, p, cs);
    if (err == cudaSuccess && weights != nullptr)
      err = attn::kv8::launch_weights(c->D, bf16,
                                      static_cast<int>(rp.blocks * rp.tile),
                                      p, cs);
  }
  return err == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t evict_impl(const attn_kv8_t* src, const attn_kv8_t* dst,
                         const float* weights, float* dst_weights, int keep,
                         int recent, int* indices, attn_stream_t stream) {
  attn_status_t st = check_cache_sizes(src);
  if (st != ATTN_OK) return st;
  st = check_cache_sizes(dst);
  if (st != ATTN_OK) return st;
  if (src->B != dst->B || src->Hkv != dst->Hkv || src->D != dst->D ||
      src->block != dst->block)
    return ATTN_ERR_INVALID_ARG;
  if (keep < 1 || keep > dst->capacity || recent < 0 || recent > keep)
    return ATTN_ERR_INVALID_ARG;
  if (src->B == 0) return ATTN_OK;
  // CTAs of the move launch: K and V by blocks of a head, weights by 128.
  if (2LL * src->B * src->Hkv *
          ((keep - 1) / src->block + dst->capacity / 128 + 16) > 0x7fffffffLL)
    return ATTN_ERR_INVALID_ARG;
  st = check_cache_pointers(*src);
  if (st != ATTN_OK) return st;
  st = check_cache_pointers(*dst);
  if (st != ATTN_OK) return st;
  if (weights == nullptr || dst_weights == nullptr || indices == nullptr)
    return ATTN_ERR_INVALID_ARG;
  if (misaligned(weights, 4) || misaligned(dst_weights, 4) ||
      misaligned(indices, 4))
    return ATTN_ERR_ALIGNMENT;
  const bool in_place = src->k == dst->k && src->v == dst->v &&
                        src->k_scale == dst->k_scale &&
                        src->v_scale == dst->v_scale;
  if (in_place && src->capacity != dst->capacity) return ATTN_ERR_INVALID_ARG;
  const size_t len_bytes = static_cast<size_t>(src->B) * 4;
  const Range in[] = {{src->lens, len_bytes},
                      {src->k, code_bytes(*src)},
                      {src->v, code_bytes(*src)},
                      {src->k_scale, scale_bytes(*src)},
                      {src->v_scale, scale_bytes(*src)},
                      {weights, heads(*src) * src->capacity * 4}};
  const Range out[] = {{dst->k, code_bytes(*dst)},
                       {dst->v, code_bytes(*dst)},
                       {dst->k_scale, scale_bytes(*dst)},
                       {dst->v_scale, scale_bytes(*dst)},
                       {dst_weights, heads(*dst) * dst->capacity * 4},
                       {dst->lens, len_bytes},
                       {indices, heads(*src) * keep * 4}};
  for (int i = 0; i < 7; ++i) {
    if (any_overlap(out[i], out + i + 1, 6 - i)) return ATTN_ERR_INVALID_ARG;
    for (int j = 0; j < 6; ++j) {
      // In place a buffer may be its own source.
      if (in_place && ((i < 4 && j == i + 1) ||
                       (i == 4 && j == 5 && dst_weights == weights)))
        continue;
      if (attn::ranges_overlap(out[i].p, out[i].n, in[j].p, in[j].n))
        return ATTN_ERR_INVALID_ARG;
    }
  }
  // Distinct sources, too: K must not be V.
  for (int j = 0; j < 6; ++j)
    if (any_overlap(in[j], in + j + 1, 5 - j)) return ATTN_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_CUDA;
  const void* mem[] = {dst->k,       dst->v, dst->k_scale, dst->v_scale,
                       dst->lens, weights, dst_weights,  indices};
  if (!all_on_device(*src, mem, 8, dev)) return ATTN_ERR_INVALID_ARG;
  attn::kv8::EvictParams p{};
  p.src_code[0] = static_cast<const uint8_t*>(src->k);
  p.src_code[1] = static_cast<const uint8_t*>(src->v);
  p.src_scale[0] = src->k_scale;
  p.src_scale[1] = src->v_scale;
  p.dst_code[0] = static_cast<uint8_t*>(dst->k);
  p.dst_code[1] = static_cast<uint8_t*>(dst->v);
  p.dst_scale[0] = dst->k_scale;
  p.dst_scale[1] = dst->v_scale;
  p.src_lens = src->lens;
  p.dst_lens = dst->lens;
  p.weights = weights;
  p.dst_weights = dst_weights;
  p.indices = indices;
  p.B = src->B;
  p.Hkv = src->Hkv;
  p.src_capacity = src->capacity;
  p.dst_capacity = dst->capacity;
  p.src_nblk = blocks(*src);
  p.dst_nblk = blocks(*dst);
  p.block_shift = block_shift(src->block);
  p.keep = keep;
  p.recent = recent;
  p.in_place = in_place;
  p.status = attn::device_status_word(dev);
  if (p.status == nullptr) return ATTN_ERR_CUDA;
  const cudaError_t err = attn::kv8::launch_evict(
      src->D, p, reinterpret_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

extern "C" {

attn_status_t attn_kv8_append(const attn_kv8_t* cache, const void* K,
                              const void* V, int Sq, const int* new_lens,
                              attn_dtype_t dtype, attn_stream_t stream) {
  return append_impl(cache, K, V, Sq, new_lens, dtype, stream);
}

attn_status_t attn_kv8_fwd(const attn_kv8_t* cache, const void* Q, void* O,
                           float* LSE, float* weights, int Hq, int Sq,
                           const int* new_lens, float scale, int causal,
                           attn_dtype_t dtype, void* workspace,
                           size_t workspace_bytes, attn_stream_t stream) {
  return fwd_impl(cache, Q, O, LSE, weights, Hq, Sq, new_lens, scale, causal,
                  dtype, workspace, workspace_bytes, stream);
}

size_t attn_kv8_workspace_bytes(int B, int Hq, int Hkv, int Sq, int capacity,
                                int D, int weights) {
  if (B < 0 || Hkv <= 0 || Hq <= 0 || Hq % Hkv != 0 || Sq < 0 ||
      capacity <= 0 || (D != 64 && D != 128))
    return 0;
  if (B == 0 || Sq == 0) return 0;
  const RowPlan rp = plan_rows(Hq, Hkv, Sq, D, current_sms());
  return workspace_layout(B, Hkv, capacity, D, rp, weights != 0).total;
}

attn_status_t attn_kv8_evict(const attn_kv8_t* src, const attn_kv8_t* dst,
                             const float* weights, float* dst_weights,
                             int keep, int recent, int* indices,
                             attn_stream_t stream) {
  return evict_impl(src, dst, weights, dst_weights, keep, recent, indices,
                    stream);
}

}  // extern "C"

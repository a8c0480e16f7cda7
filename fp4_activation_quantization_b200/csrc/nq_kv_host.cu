// nq_kv_host.cu — the C ABI of the 4-bit key/value cache: argument checks and
// launches.  Contracts are in include/nq.h.  Nothing here allocates,
// synchronizes or reads device memory.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "nq.h"
#include "nq_host.h"
#include "nq_kv.h"

namespace {

using nq::host::error;

#define NQ_REQUIRE(cond, ...)                                              \
  do {                                                                     \
    if (!(cond)) return error(NQ_ERR_INVALID_ARGUMENT, __VA_ARGS__);       \
  } while (0)

constexpr int64_t kInt32Max = 0x7fffffff;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int log2_of_page(int32_t page) {
  for (int l = 4; l <= 7; ++l)
    if (page == (1 << l)) return l;
  return -1;
}

nq_status check_cache(const char* fn, const void* cache, int64_t page_stride, int64_t pages, int32_t heads, int32_t d,
                      int32_t page, nq::KvCache* c) {
  if (d != 64 && d != 128 && d != 256) return error(NQ_ERR_UNSUPPORTED, "%s: head dimension %d not in {64, 128, 256}", fn, d);
  const int l = log2_of_page(page);
  if (l < 0) return error(NQ_ERR_UNSUPPORTED, "%s: page of %d tokens not in {16, 32, 64, 128}", fn, page);
  NQ_REQUIRE(heads >= 1 && heads <= 65535, "%s: kv_heads = %d not in 1..65535", fn, heads);
  NQ_REQUIRE(pages >= 0 && pages <= kInt32Max, "%s: num_pages = %lld out of range", fn, (long long)pages);
  const int64_t need = int64_t(heads) * page * d * 9 / 8;
  NQ_REQUIRE(page_stride >= need && page_stride % 16 == 0,
             "%s: page_stride = %lld must be a multiple of 16 and at least %lld", fn, (long long)page_stride, (long long)need);
  NQ_REQUIRE(aligned(cache, 16), "%s: the cache must be 16-byte aligned", fn);
  c->base = static_cast<uint8_t*>(const_cast<void*>(cache));
  c->page_stride = page_stride;
  c->pages = pages;
  c->heads = heads;
  c->log_page = l;
  c->d = d;
  return NQ_OK;
}

// Either order of tokens and heads; rows of d elements that do not overlap.
bool strides_ok(int64_t token, int64_t head, int64_t T, int64_t heads, int64_t d) {
  if ((heads > 1 && head < d) || (T > 1 && token < d)) return false;
  return heads <= 1 || T <= 1 || token >= (heads - 1) * head + d || head >= (T - 1) * token + d;
}

nq_status kv_copy(const char* fn, bool gather, const void* k, int64_t ld_kt, int64_t ld_kh, const void* v, int64_t ld_vt,
                  int64_t ld_vh, const int64_t* slots, const float* k_scale, const float* v_scale, const void* cache,
                  int64_t page_stride, int64_t pages, int64_t T, int32_t heads, int32_t d, int32_t page, uint32_t flags,
                  nq_stream_t stream) {
  nq::KvCopyArgs a{};
  const nq_status st = check_cache(fn, cache, page_stride, pages, heads, d, page, &a.cache);
  if (st != NQ_OK) return st;
  NQ_REQUIRE((flags & ~uint32_t(NQ_FLAG_PDL)) == 0, "%s: only NQ_FLAG_PDL applies", fn);
  NQ_REQUIRE(T >= 0, "%s: T = %lld < 0", fn, (long long)T);
  if (T > kInt32Max) return error(NQ_ERR_UNSUPPORTED, "%s: T = %lld too large", fn, (long long)T);
  NQ_REQUIRE(strides_ok(ld_kt, ld_kh, T, heads, d) && strides_ok(ld_vt, ld_vh, T, heads, d),
             "%s: token and head strides must keep rows of %d elements apart", fn, d);
  if (T == 0) return NQ_OK;
  NQ_REQUIRE(k && v && slots && k_scale && v_scale && (cache || pages == 0), "%s: null pointer", fn);
  a.k = static_cast<uint16_t*>(const_cast<void*>(k));
  a.v = static_cast<uint16_t*>(const_cast<void*>(v));
  a.ld_kt = ld_kt, a.ld_kh = ld_kh, a.ld_vt = ld_vt, a.ld_vh = ld_vh;
  a.slots = slots;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.T = int32_t(T);
  const bool vec = aligned(k, 32) && aligned(v, 32) && (ld_kt | ld_vt) % 16 == 0 && (heads == 1 || (ld_kh | ld_vh) % 16 == 0);
  const int per_warp = 512 / d;  // tokens of a warp
  const int64_t warps = (T + per_warp - 1) / per_warp * ((heads + 1) / 2);  // two heads a warp
  const int64_t grid = (warps + nq::kKvCopyThreads / 32 - 1) / (nq::kKvCopyThreads / 32);
  if (grid > kInt32Max) return error(NQ_ERR_UNSUPPORTED, "%s: too many tokens", fn);
  a.err = nq::host::error_word();
  if (a.err == nullptr) return error(NQ_ERR_CUDA, "%s: no CUDA device", fn);
  void* args[] = {&a};
  return nq::host::launch(fn, gather ? nq::kv_gather_kernel(d, vec) : nq::kv_append_kernel(d, vec), unsigned(grid),
                          nq::kKvCopyThreads, 0, args, (flags & NQ_FLAG_PDL) != 0, static_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

int64_t nq_kv_page_bytes(int32_t kv_heads, int32_t d, int32_t page_size) {
  return int64_t(kv_heads) * page_size * d * 9 / 8;
}

nq_status nq_kv_plan(const int32_t* cached_lens, const int32_t* new_lens, int32_t* block_table, int64_t ld_table,
                     int32_t table_width, const int32_t* free_pages, int64_t n_free, const int32_t* free_head,
                     int32_t* free_head_out, int32_t* cu_q, int32_t* kv_lens, int32_t* positions, int64_t* slots,
                     int64_t B, int64_t T, int32_t page_size, uint32_t flags, nq_stream_t stream) {
  const char* fn = "nq_kv_plan";
  const int l = log2_of_page(page_size);
  if (l < 0) return error(NQ_ERR_UNSUPPORTED, "%s: page of %d tokens not in {16, 32, 64, 128}", fn, page_size);
  NQ_REQUIRE((flags & ~uint32_t(NQ_FLAG_PDL)) == 0, "%s: only NQ_FLAG_PDL applies", fn);
  NQ_REQUIRE(B >= 0 && T >= 0 && n_free >= 0, "%s: negative size", fn);
  if (B > NQ_KV_MAX_REQUESTS)
    return error(NQ_ERR_UNSUPPORTED, "%s: %lld requests > NQ_KV_MAX_REQUESTS (%d)", fn, (long long)B, NQ_KV_MAX_REQUESTS);
  if (T > kInt32Max || n_free > kInt32Max) return error(NQ_ERR_UNSUPPORTED, "%s: sizes beyond 32 bits", fn);
  NQ_REQUIRE(table_width >= 0 && ld_table >= table_width, "%s: ld_table must be >= table_width", fn);
  if (int64_t(table_width) * page_size > (int64_t(1) << 30))
    return error(NQ_ERR_UNSUPPORTED, "%s: a table row addresses more than 2^30 tokens", fn);
  NQ_REQUIRE(free_head && free_head_out && cu_q && (B == 0 || (cached_lens && new_lens && kv_lens)) &&
                 (B == 0 || table_width == 0 || block_table) && (n_free == 0 || free_pages) &&
                 (T == 0 || (positions && slots)),
             "%s: null pointer", fn);
  const auto overlap = [](const void* p, int64_t n, const void* q, int64_t m) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
    return n > 0 && m > 0 && x < y + uintptr_t(m) && y < x + uintptr_t(n);
  };
  NQ_REQUIRE(!overlap(kv_lens, 4 * B, cached_lens, 4 * B) && !overlap(kv_lens, 4 * B, new_lens, 4 * B) &&
                 !overlap(cu_q, 4 * B + 4, cached_lens, 4 * B) && !overlap(cu_q, 4 * B + 4, new_lens, 4 * B),
             "%s: kv_lens and cu_q must not overlap cached_lens or new_lens", fn);
  nq::KvPlanArgs a{};
  a.cached = cached_lens;
  a.added = new_lens;
  a.table = block_table;
  a.ld_table = ld_table;
  a.free_pages = free_pages;
  a.free_head = free_head;
  a.free_head_out = free_head_out;
  a.cu_q = cu_q;
  a.kv_lens = kv_lens;
  a.positions = positions;
  a.slots = slots;
  a.B = int32_t(B);
  a.T = int32_t(T);
  a.width = table_width;
  a.n_free = int32_t(n_free);
  a.log_page = l;
  a.err = nq::host::error_word();
  if (a.err == nullptr) return error(NQ_ERR_CUDA, "%s: no CUDA device", fn);
  const void* k = nq::kv_plan_kernel();
  const size_t smem = size_t(3 * B + 2) * sizeof(int32_t);
  if (!nq::host::allow_smem(k, smem)) return error(NQ_ERR_UNSUPPORTED, "%s: %zu bytes of shared memory not available", fn, smem);
  // Every CTA repeats the scan; one token a thread as far as the SMs go (B = 2048, T = 95647: 8.0 us with four).
  int64_t grid = (T + nq::kKvPlanThreads - 1) / nq::kKvPlanThreads;
  grid = grid < 1 ? 1 : (grid > 148 ? 148 : grid);
  if (free_head_out == free_head) grid = 1;  // every CTA reads the head: only a lone one may overwrite it
  void* args[] = {&a};
  return nq::host::launch(fn, k, unsigned(grid), nq::kKvPlanThreads, smem, args, (flags & NQ_FLAG_PDL) != 0,
                          static_cast<cudaStream_t>(stream));
}

nq_status nq_kv_append_nvfp4(const void* k, int64_t ld_k_token, int64_t ld_k_head, const void* v, int64_t ld_v_token,
                             int64_t ld_v_head, const int64_t* slots, const float* k_scale, const float* v_scale,
                             void* cache, int64_t page_stride, int64_t num_pages, int64_t T, int32_t kv_heads, int32_t d,
                             int32_t page_size, uint32_t flags, nq_stream_t stream) {
  return kv_copy("nq_kv_append_nvfp4", false, k, ld_k_token, ld_k_head, v, ld_v_token, ld_v_head, slots, k_scale, v_scale,
                 cache, page_stride, num_pages, T, kv_heads, d, page_size, flags, stream);
}

nq_status nq_kv_gather_nvfp4(const void* cache, int64_t page_stride, int64_t num_pages, const int64_t* slots,
                             const float* k_scale, const float* v_scale, void* k_out, int64_t ld_k_token,
                             int64_t ld_k_head, void* v_out, int64_t ld_v_token, int64_t ld_v_head, int64_t T,
                             int32_t kv_heads, int32_t d, int32_t page_size, uint32_t flags, nq_stream_t stream) {
  return kv_copy("nq_kv_gather_nvfp4", true, k_out, ld_k_token, ld_k_head, v_out, ld_v_token, ld_v_head, slots, k_scale,
                 v_scale, cache, page_stride, num_pages, T, kv_heads, d, page_size, flags, stream);
}

nq_status nq_attention_nvfp4_kv(const void* q, int64_t ld_q_token, int64_t ld_q_head, const void* cache,
                                int64_t page_stride, int64_t num_pages, const int32_t* block_table, int64_t ld_table,
                                int32_t table_width, const int32_t* kv_lens, const int32_t* cu_q, const float* k_scale,
                                const float* v_scale, void* out, int64_t ld_out_token, int64_t ld_out_head, float* lse,
                                int64_t ld_lse, void* workspace, int64_t workspace_bytes, int64_t T, int64_t B,
                                int32_t heads, int32_t kv_heads, int32_t d, int32_t page_size, float softmax_scale,
                                int32_t window, uint32_t flags, nq_stream_t stream) {
  const char* fn = "nq_attention_nvfp4_kv";
  nq::AttnArgs a{};
  const nq_status st = check_cache(fn, cache, page_stride, num_pages, kv_heads, d, page_size, &a.cache);
  if (st != NQ_OK) return st;
  NQ_REQUIRE((flags & ~uint32_t(NQ_FLAG_PDL | NQ_FLAG_NONCAUSAL)) == 0, "%s: only NQ_FLAG_PDL and NQ_FLAG_NONCAUSAL apply", fn);
  NQ_REQUIRE(heads >= kv_heads && heads % kv_heads == 0, "%s: heads = %d is not a multiple of kv_heads = %d", fn, heads,
             kv_heads);
  NQ_REQUIRE(T >= 0 && B >= 0, "%s: negative size", fn);
  if (heads / kv_heads > 1024) return error(NQ_ERR_UNSUPPORTED, "%s: more than 1024 query heads per kv head", fn);
  if (T > (1 << 30) / heads || B > (1 << 24)) return error(NQ_ERR_UNSUPPORTED, "%s: T or B too large", fn);
  NQ_REQUIRE(std::isfinite(softmax_scale), "%s: softmax_scale must be finite", fn);
  NQ_REQUIRE(window >= 0, "%s: window = %d < 0", fn, window);
  NQ_REQUIRE(table_width >= 0 && ld_table >= table_width, "%s: ld_table must be >= table_width", fn);
  if (int64_t(table_width) * page_size > (int64_t(1) << 30))
    return error(NQ_ERR_UNSUPPORTED, "%s: a table row addresses more than 2^30 tokens", fn);
  NQ_REQUIRE(strides_ok(ld_q_token, ld_q_head, T, heads, d) && strides_ok(ld_out_token, ld_out_head, T, heads, d),
             "%s: token and head strides must keep rows of %d elements apart", fn, d);
  NQ_REQUIRE(lse == nullptr || ld_lse >= heads, "%s: ld_lse must be >= heads", fn);
  if (T == 0 || B == 0) return NQ_OK;
  NQ_REQUIRE(q && out && kv_lens && cu_q && k_scale && v_scale && (cache || num_pages == 0) && (block_table || table_width == 0),
             "%s: null pointer", fn);
  NQ_REQUIRE(workspace && aligned(workspace, 16) && workspace_bytes >= NQ_ATTENTION_WORKSPACE_BYTES,
             "%s: a 16-byte aligned workspace of NQ_ATTENTION_WORKSPACE_BYTES (%d) is required", fn,
             NQ_ATTENTION_WORKSPACE_BYTES);
  a.q = static_cast<const uint16_t*>(q);
  a.ld_qt = ld_q_token, a.ld_qh = ld_q_head;
  a.table = block_table;
  a.ld_table = ld_table;
  a.width = table_width;
  a.kv_lens = kv_lens;
  a.cu_q = cu_q;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.out = static_cast<uint16_t*>(out);
  a.ld_ot = ld_out_token, a.ld_oh = ld_out_head;
  a.lse = lse;
  a.ld_lse = ld_lse;
  a.workspace = static_cast<uint8_t*>(workspace);
  a.T = int32_t(T);
  a.B = int32_t(B);
  a.heads = heads;
  a.group = heads / kv_heads;
  a.window = window < (1 << 30) ? window : 1 << 30;  // no key is further away
  a.group_magic = uint32_t(((uint64_t(1) << 32) + a.group - 1) / a.group);
  a.causal = (flags & NQ_FLAG_NONCAUSAL) ? 0 : 1;
  a.scale_log2 = softmax_scale * 1.44269504088896340736f;
  a.err = nq::host::error_word();
  if (a.err == nullptr) return error(NQ_ERR_CUDA, "%s: no CUDA device", fn);

  // Rows of an average request and kv head: few of them go to the rows kernel,
  // in 8-row tiles of which a warp takes n_tiles.  Segments (request, row tile, kv
  // head) fewer than half the CTAs that the GPU holds: a chunk a CTA and one
  // launch; else a share a warp and a second launch.
  const int64_t rows = (T * a.group + B - 1) / B;
  const int n_tiles = rows <= 8 ? 1 : (d > 64 || rows <= 16 || (rows > 32 && rows <= 48) ? 2 : 4);
  nq::AttnRows k = nq::attn_rows(d, n_tiles, false);
  if (!nq::host::allow_smem(k.kernel, k.smem))
    return error(NQ_ERR_UNSUPPORTED, "%s: %zu bytes of shared memory not available", fn, k.smem);
  int64_t grid = nq::host::resident_ctas(k.kernel, k.threads, k.smem);
  if (grid <= 0) return error(NQ_ERR_CUDA, "%s: no CUDA device", fn);
  const int64_t segments = (T * a.group / (8 * n_tiles) + B) * kv_heads;
  const bool few = segments <= grid / 2;
  // Rows kernel / 128-row tiles, 8 kv heads, us:
  //                             d = 64            d = 128                          d = 256
  //   24 requests of 4096 keys  64 rows  84/115   48 rows 123/132, 64 rows 150/133   24 rows 152/166, 32 rows 190/168
  //   200 requests of 700 keys  64 rows 143/164   48 rows 174/199, 64 rows 221/201   24 rows 211/231, 32 rows 272/238
  //   2 requests of 8192 (few)  32 rows  23/31    32 rows  29/39                     16 rows  35/43,  24 rows  45/43
  //   1 request of 65536 (few)  32 rows  39/66    32 rows  61/78,  48 rows  86/78    16 rows  66/92,  24 rows 111/96
  const int64_t most = d == 256 ? (few ? 16 : 24) : (few ? 32 : (d == 128 ? 48 : 64));
  if (rows > most) {
    const nq::AttnTiles t = nq::attn_tiles(d);
    if (!nq::host::allow_smem(t.kernel, t.smem))
      return error(NQ_ERR_UNSUPPORTED, "%s: %zu bytes of shared memory not available", fn, t.smem);
    const int64_t tiles = T * a.group / t.rows + B, items = tiles * kv_heads;
    const int64_t sms = nq::host::resident_ctas(t.kernel, nq::kAttnTilesThreads, t.smem);
    if (sms <= 0) return error(NQ_ERR_CUDA, "%s: no CUDA device", fn);
    const int64_t room = (workspace_bytes - nq::kAttnHeader) / (int64_t(t.rows) * (d + 2) * int64_t(sizeof(float)));
    int64_t splits = (sms < room ? sms : room) / items;
    const int64_t blocks = (int64_t(table_width) * page_size + 511) / 512;  // at least four blocks of keys each
    splits = splits < blocks ? splits : blocks;
    splits = splits < 1 ? 1 : splits;
    const int64_t ctas = items * splits, join_grid = items * (t.rows / 8);
    if (ctas > kInt32Max - 2 * sms || join_grid > kInt32Max) return error(NQ_ERR_UNSUPPORTED, "%s: T or B too large", fn);
    a.tiles = int32_t(tiles);
    a.splits = int32_t(splits);
    void* args[] = {&a};
    nq_status s = nq::host::launch(fn, t.kernel, unsigned(ctas < sms ? ctas : sms), nq::kAttnTilesThreads, t.smem, args,
                                   (flags & NQ_FLAG_PDL) != 0, static_cast<cudaStream_t>(stream));
    if (s == NQ_OK && splits > 1)
      s = nq::host::launch(fn, t.join, unsigned(join_grid), 256, 0, args, (flags & NQ_FLAG_PDL) != 0,
                           static_cast<cudaStream_t>(stream));
    return s;
  }
  const int64_t atoms = (int64_t(table_width) * page_size + 15) / 16;
  const auto slot = [&](int tiles) { return int64_t(8 * tiles) * (d + 2) * int64_t(sizeof(float)); };
  void* args[] = {&a};
  if (few) {
    const int64_t room = (workspace_bytes - nq::kAttnHeader) / slot(n_tiles), counters = nq::kAttnCounterBytes / 4 - 3;
    grid = grid < room ? grid : room;
    grid = grid < counters ? grid : counters;
    if (segments * (atoms / 32 + 1) < grid) grid = segments * (atoms / 32 + 1);
    return nq::host::launch(fn, k.kernel, unsigned(grid), k.threads, k.smem, args, (flags & NQ_FLAG_PDL) != 0,
                            static_cast<cudaStream_t>(stream));
  }
  // 256 x 16 rows do not fit a thread's registers beside the walk (24 requests: 108 us, twice 8 rows 103).
  const int walk_tiles = d == 256 ? 1 : n_tiles;
  k = nq::attn_rows(d, walk_tiles, true);
  if (!nq::host::allow_smem(k.kernel, k.smem))
    return error(NQ_ERR_UNSUPPORTED, "%s: %zu bytes of shared memory not available", fn, k.smem);
  grid = nq::host::resident_ctas(k.kernel, k.threads, k.smem);
  const int warps = k.threads / 32;
  if (grid <= 0) return error(NQ_ERR_CUDA, "%s: no CUDA device", fn);
  int64_t room = (workspace_bytes - nq::kAttnHeader) / (2 * slot(walk_tiles)) / 2;  // two parts a warp, two slots each
  room = room < nq::kAttnMaxParts / 2 ? room : nq::kAttnMaxParts / 2;
  grid = grid < room / warps ? grid : room / warps;
  nq_status s = nq::host::launch(fn, k.kernel, unsigned(grid), k.threads, k.smem, args,
                                 (flags & NQ_FLAG_PDL) != 0, static_cast<cudaStream_t>(stream));
  if (s == NQ_OK)  // may start while the first launch ends; it waits for its results
    s = nq::host::launch(fn, k.join, unsigned(4 * grid), nq::kAttnJoinThreads, 0, args, true,
                         static_cast<cudaStream_t>(stream));
  return s;
}

}  // extern "C"

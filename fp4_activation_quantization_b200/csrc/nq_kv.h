// nq_kv.h — argument blocks of the 4-bit key/value cache calls, shared by their
// host launcher (nq_kv_host.cu) and their kernels.  Not installed.
#pragma once

#include <cstddef>
#include <cstdint>

#include "nq.h"

namespace nq {

// Bits of the device error word that these kernels set (read and cleared by
// nq_check_device_errors).
constexpr uint32_t kErrSlot = 4u;  // a slot or page outside the cache: skipped
constexpr uint32_t kErrWait = 16u;  // a bounded wait inside a kernel ran out: its output is not valid
constexpr uint32_t kErrPlan = 8u;  // a plan ran out of free pages, table columns or token rows

// The cache: [pages, kv_heads, page / 16] atoms of 16 tokens (18 * D bytes each,
// keys and values of one kv head; the byte order is in nq.h).  Pages lie
// page_stride bytes apart.
struct KvCache {
  uint8_t* base;
  int64_t page_stride;
  int64_t pages;
  int32_t heads;
  int32_t log_page;  // log2(tokens per page), 4 .. 7
  int32_t d;
};

struct KvPlanArgs {
  const int32_t* cached;   // [B] tokens each request holds already
  const int32_t* added;    // [B] tokens it gains
  int32_t* table;          // [B, ld_table] page numbers, `width` columns used
  int64_t ld_table;
  const int32_t* free_pages;  // [n_free]
  const int32_t* free_head;   // [1] first entry of the list not yet taken
  int32_t* free_head_out;     // [1]
  int32_t* cu_q;       // [B + 1]
  int32_t* kv_lens;    // [B]
  int32_t* positions;  // [T]
  int64_t* slots;      // [T]
  int32_t B, T, width, n_free, log_page;
  uint32_t* err;
};

struct KvCopyArgs {  // append (bf16 -> cache) and gather (cache -> bf16)
  uint16_t* k;       // bf16 [T, heads, d] with token and head strides (elements)
  uint16_t* v;
  int64_t ld_kt, ld_kh, ld_vt, ld_vh;
  const int64_t* slots;  // [T], < 0: a padding token
  const float* k_scale;
  const float* v_scale;
  KvCache cache;
  int32_t T;
  uint32_t* err;
};

struct AttnArgs {
  const uint16_t* q;  // bf16 [T, heads, d]
  int64_t ld_qt, ld_qh;
  KvCache cache;
  const int32_t* table;
  int64_t ld_table;
  int32_t width;  // columns of the table
  const int32_t* kv_lens;
  const int32_t* cu_q;
  const float* k_scale;
  const float* v_scale;
  uint16_t* out;  // bf16 [T, heads, d]
  int64_t ld_ot, ld_oh;
  float* lse;  // [T, ld_lse] or null
  int64_t ld_lse;
  uint8_t* workspace;  // parts of rows whose keys were split
  int32_t T, B, heads, group;  // group: query heads per kv head
  uint32_t group_magic;        // ceil(2^32 / group)
  int32_t window;              // 0: none
  int32_t causal;
  float scale_log2;  // softmax scale * log2(e)
  int32_t tiles;       // tiles kernel: row tiles counted over the batch
  int32_t splits;      // tiles kernel: parts of an item's keys
  uint32_t* err;
};

// The head of the attention workspace: counters, zero between calls, then what
// describes the parts; their values follow.
constexpr int kAttnCounterBytes = 1 << 14;
constexpr int kAttnHeader = 1 << 19;
constexpr int kAttnMaxParts = (kAttnHeader - kAttnCounterBytes) / 32;

// Kernels (nullptr: not built).
const void* kv_plan_kernel();
const void* kv_append_kernel(int d, bool vec);
const void* kv_gather_kernel(int d, bool vec);
constexpr int kKvPlanThreads = 512;
constexpr int kKvCopyThreads = 256;

constexpr int kAttnJoinThreads = 128;
struct AttnRows {
  const void* kernel;
  const void* join;  // walk: after it
  size_t smem;
  int threads;
};
AttnRows attn_rows(int d, int n_tiles, bool walk);  // n_tiles: 8-row tiles of a warp

constexpr int kAttnTilesThreads = 512;
struct AttnTiles {
  const void* kernel;
  const void* join;  // 256 threads, 8 rows a CTA; only after a kernel with splits > 1
  int rows;          // of an item
  size_t smem;
};
AttnTiles attn_tiles(int d);

}  // namespace nq

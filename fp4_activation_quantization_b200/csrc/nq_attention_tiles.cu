// nq_attention_tiles.cu — attention over the 4-bit cache for prompts and chunks
// of prompts: 128-row tiles on the fifth-generation tensor cores.
//
// The mathematics and the numerics are those of nq_attention_rows.cu: k' and v'
// exact in f16, query rows scaled by a power of two, float32 accumulation, f16
// weights that reach up to 2^15, the running maximum raised only by more than 2^8.
//
// One CTA an SM takes items in turn: NS tiles of 128 (token, head of the group)
// rows of one request and kv head.  It walks an item's keys in blocks of 128:
//   producer warps   4-bit atoms -> f16 K or V block in shared memory (128-byte
//                    rows, 128-byte swizzle; the next item's bytes are already
//                    in registers while one is converted);
//   one thread       S = Q K^T (both from shared memory) and O += P V (P from
//                    tensor memory, V read with its dimensions contiguous);
//   NS x 128 threads a row each: S from tensor memory, maximum, exponentials,
//                    P back over S as f16, sums; O rescaled in place when a
//                    row's maximum is raised; the output at the end.
// D <= 128: two tiles in turn (NS = 2), so that one tile's exponentials run
// under the other's products.  D = 256: O alone takes 256 of the 512 tensor
// memory columns, so one tile with two S buffers, the next block's S being
// computed under this block's exponentials.
//
// A warp finds the next item while this one is worked on, the producers go on to
// its keys while the last blocks are multiplied, and the barriers count on, so that
// between items only the output and the queries stand still.  Measured with 16 chunks
// of 512 behind 1536 tokens, 8 kv heads of 128 / 256 / 64: a CTA per item 332 / 385 /
// 506 us, items in turn 315 / 358 / 465, query rows loaded in one go 274 / 287 / 430,
// rows loaded and stored side by side 274 / 279 / 436.  A prompt of 8192, 32/8 heads
// of 128, alone: 510 us, 1078 TFLOP/s, 0.67 of the measured product rate; a block of 128
// keys takes the CTA about 4100 cycles; products and exponentials are about 2100 each
// (tensor pipe 53 %, exponential unit 51 % busy), and a tile's own chain, S to maximum
// to exponentials to P V to the next S, is what the step waits for.
// An item of at most 128 rows takes almost as long; with its keys shared out between
// two tiles of the same rows, 24 x 64 rows over 4096 keys gained 6 %, but items of
// two tiles lost 3 to 7 %.  Items are claimed when
// five blocks of the item before are left: earlier, the last items went to CTAs
// that were not the first to be free (256 items of 33 blocks: 252 us, now 168).
//
// Every wait on an mbarrier is bounded; a CTA whose wait runs out records it in
// the device error word, frees its tensor memory and leaves.
#include "nq_kv_layout.cuh"

namespace nq {

namespace {

constexpr int kThreads = kAttnTilesThreads;
constexpr int kBlock = 128;  // keys of a block
constexpr int kAtoms = kBlock / 16;
constexpr int kBad = 8;  // ring of the blocks' missing-atom masks

template <int D>
struct Cfg {
  static constexpr int kTiles = D == 256 ? 1 : 2;              // tiles of a CTA
  static constexpr int kRows = 128 * kTiles;
  static constexpr int kProducerWarps = 4 * (3 - kTiles);      // warps 4 kTiles ... 11
  static constexpr int kChunks = D / 64;                       // 64-dimension chunks of a block
  static constexpr int kSlotBytes = kChunks * 16384;           // K or V block in f16
  static constexpr int kSlots = 131072 / kSlotBytes;
  static constexpr int kQBytes = 128 * D * 2;                  // of a tile
  static constexpr int kOCol = 256;                            // first tensor memory column of O
  static constexpr int kSmem = 131072 + kTiles * kQBytes + 1024;  // 1024: alignment
  // Registers of a thread after the split; the launch holds 512 x 128, so a
  // role above 128 asks for more and one below 128 gives some up.
  static constexpr int kRegsSoftmax = D == 256 ? 224 : 192;
  static constexpr int kRegsProducer = D == 256 ? 128 : 96;
  static constexpr int kRegsMma = 32;
  static_assert(kRegsSoftmax > 128 && kRegsProducer <= 128 && kRegsMma < 128, "direction of the split");
  static_assert(kTiles * kRegsSoftmax + (3 - kTiles) * kRegsProducer + kRegsMma <= 4 * 128, "register split");
};

// ---------------------------------------------------------------- PTX ----
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return uint32_t(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(ok)
               : "r"(bar), "r"(parity)
               : "memory");
  return ok != 0;
}
// Waits for the phase of the given parity to complete; false when the limit
// runs out (no wait of a sound run comes near it) or another role gave up.  NAP:
// a wait that may take as long as an item, so it leaves the issue slots to others.
template <bool NAP>
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* gave_up) {
  for (int i = 0; i < (NAP ? 1 << 26 : 1 << 22); ++i) {
    if (mbar_try(bar, parity)) return true;
    if ((i & 1023) == 1023 && *gave_up) return false;
    if (NAP && i > 8) __nanosleep(200);
  }
  *gave_up = 1;
  return false;
}
// The same for a whole warp, which stays together.
template <bool NAP = false>
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, volatile int* gave_up) {
  return __all_sync(kFull, mbar_wait<NAP>(bar, parity, gave_up));
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_smem_to_mma() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
               ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate))
               : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
               ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate))
               : "memory");
}
#define NQ_R8(v, o) "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), "=r"(v[o + 5]), "=r"(v[o + 6]), "=r"(v[o + 7])
#define NQ_W8(v, o) "r"(v[o]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), "r"(v[o + 5]), "r"(v[o + 6]), "r"(v[o + 7])
// 32 columns of this thread's row (lane) of tensor memory.
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : NQ_R8(v, 0), NQ_R8(v, 8), NQ_R8(v, 16), NQ_R8(v, 24)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      NQ_W8(v, 0), NQ_W8(v, 8), NQ_W8(v, 16), NQ_W8(v, 24)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Shared memory descriptor of a matrix of 128-byte rows in 1024-byte groups of
// eight with the 128-byte swizzle.  Contraction along the row (Q, K): groups
// 1024 bytes apart.  Contraction across rows (V): 64-dimension chunks 16384
// bytes apart, groups of eight keys 1024 bytes apart.
__device__ __forceinline__ uint64_t matrix(uint32_t addr) {
  return uint64_t((addr & 0x3FFFF) >> 4) | (uint64_t(16384 >> 4) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
         (uint64_t(2) << 61);
}
// f16 x f16 -> f32, 128 rows, N columns; b_across: B's rows run along the contraction.
constexpr uint32_t instruction(int n, bool b_across) {
  return (1u << 4) | (b_across ? 1u << 16 : 0u) | (uint32_t(n / 8) << 17) | (uint32_t(128 / 16) << 24);
}

// A piece of work: up to kRows rows of a request and kv head, and a part of their keys.
struct Item {
  int b, head, row0;  // request, kv head, first row (token * group + head of the group)
  int rows;           // rows, 0: none
  int q0, q_len, kv_len;
  int first, blocks;  // first key (a multiple of 16), blocks of this split
  int index, split;   // number of the item among tiles and heads, of the split
  int before;         // blocks of the CTA's items before
};

__device__ __forceinline__ float* partials_of(const AttnArgs& a) { return reinterpret_cast<float*>(a.workspace + kAttnHeader); }
// Of the workspace's counters, zero between calls: items claimed beyond each CTA's first, CTAs that are done.
__device__ __forceinline__ uint32_t* claims_of(const AttnArgs& a) {
  return reinterpret_cast<uint32_t*>(a.workspace + kAttnCounterBytes) - 1;
}
__device__ __forceinline__ uint32_t* done_of(const AttnArgs& a) { return claims_of(a) - 1; }

// Tiles of request b are numbered from floor(cu_q[b] * group / R) + b on: as
// many numbers as it has tiles at least, without a sum over the requests.
template <int R>
__device__ __forceinline__ int64_t tile_start(const AttnArgs& a, int b, int c0) {
  return int64_t(c0) * a.group / R + b;
}
__device__ __forceinline__ int first_row_of(const AttnArgs& a, int b) { return min(max(a.cu_q[b], 0), a.T); }

// Item number `block`, by a whole warp; later tiles of a request, which see more
// keys, come first.
template <int R>
__device__ __forceinline__ Item find_item(const AttnArgs& a, int block, int lane) {
  const int heads = a.cache.heads;
  Item it{};
  it.index = block / a.splits;
  it.split = block - it.index * a.splits;
  const int tg = a.tiles - 1 - it.index / heads;
  it.head = it.index % heads;
  // The last request that starts at tg or before, 32 places at a time.
  int from_b = 0, to_b = a.B;
  do {
    const int step = (to_b - from_b + 31) / 32, at = from_b + lane * step;
    const uint32_t reached = __ballot_sync(kFull, at < to_b && tile_start<R>(a, at, first_row_of(a, at)) <= tg);
    if (reached == 0) return it;
    from_b += (31 - __clz(int(reached))) * step;
    to_b = min(to_b, from_b + step);
  } while (to_b - from_b > 1);
  it.b = from_b;
  const int c0 = first_row_of(a, it.b), c1 = min(max(a.cu_q[it.b + 1], c0), a.T);
  it.q0 = c0;
  it.q_len = c1 - c0;
  const int64_t row0 = (tg - tile_start<R>(a, it.b, c0)) * R, all = int64_t(it.q_len) * a.group;
  if (row0 >= all) return it;
  it.row0 = int(row0);
  it.rows = int(min(int64_t(R), all - row0));
  it.kv_len = int(min(int64_t(max(a.kv_lens[it.b], 0)), int64_t(a.width) << a.cache.log_page));
  // Keys that some row of the item sees.
  const int64_t pos0 = int64_t(it.kv_len) - it.q_len + it.row0 / a.group;
  const int64_t pos1 = int64_t(it.kv_len) - it.q_len + (it.row0 + it.rows - 1) / a.group;
  const int lo = a.window > 0 ? int(max(int64_t(0), pos0 + 1 - a.window)) & ~15 : 0;
  const int hi = a.causal ? int(min(int64_t(it.kv_len), max(int64_t(0), pos1 + 1))) : it.kv_len;
  const int all_blocks = hi > lo ? (hi - lo + kBlock - 1) / kBlock : 0;
  const int from = int(int64_t(all_blocks) * it.split / a.splits), to = int(int64_t(all_blocks) * (it.split + 1) / a.splits);
  it.first = lo + from * kBlock;
  it.blocks = to - from;
  return it;
}

// ------------------------------------------------------------ producers ----
// One item of a producer warp's stream: its atoms of a K or a V block.
template <int D>
struct RawAtom {
  uint4 codes[D / 64];
  uint32_t sf[D >= 128 ? D / 128 : 1];
};

template <int D>
__device__ __forceinline__ void load_atom(RawAtom<D>& x, const uint8_t* atom, bool value, int lane) {
  constexpr int kN = KvAtom<D>::kN, kW = KvAtom<D>::kW;
  if (atom == nullptr) {
#pragma unroll
    for (int p = 0; p < kN; ++p) x.codes[p] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < (D >= 128 ? D / 128 : 1); ++i) x.sf[i] = 0u;
    return;
  }
  if (!value) {  // lanes count rows fastest: eight lanes store eight rows
    const int at = 4 * (lane & 7) + (lane >> 3);
#pragma unroll
    for (int p = 0; p < kN; ++p) x.codes[p] = __ldg(reinterpret_cast<const uint4*>(atom + p * 512 + at * 16));
    const uint8_t* s = atom + KvAtom<D>::kKScales + at * 2 * kN;
    if constexpr (D == 64) x.sf[0] = __ldg(reinterpret_cast<const uint16_t*>(s));
    else
#pragma unroll
      for (int i = 0; i < D / 128; ++i) x.sf[i] = __ldg(reinterpret_cast<const uint32_t*>(s) + i);
  } else {
    const int r = lane >> 2, j = lane & 3;
#pragma unroll
    for (int p = 0; p < kN; ++p)
      x.codes[p] = __ldg(reinterpret_cast<const uint4*>(atom + KvAtom<D>::kVCodes + p * 512 + lane * 16));
    const uint8_t* s = atom + KvAtom<D>::kVScales + ((D == 64 ? r >> 1 : r) * 4 + j) * (4 * kW);
#pragma unroll
    for (int i = 0; i < kW; ++i) x.sf[i] = __ldg(reinterpret_cast<const uint32_t*>(s) + i);
  }
}

// Eight codes times their scale (both halves of s) into 16 bytes of a swizzled row.
__device__ __forceinline__ void store8(uint32_t slot, int token, int chunk, int g, uint32_t codes, uint32_t s) {
  uint32_t h[4];
  e2m1x8_to_f16x2(codes, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = mul_f16x2(h[i], s);
  const uint32_t at = slot + chunk * 16384 + token * 128 + ((g ^ (token & 7)) << 4);
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
}
__device__ __forceinline__ uint32_t both_halves(uint32_t pair, int i) { return __byte_perm(pair, pair, i ? 0x3232 : 0x1010); }

// keys: how many of the atom's 16 tokens exist (values behind them count as zero).
template <int D>
__device__ __forceinline__ void convert_atom(const RawAtom<D>& x, uint32_t slot, int token0, bool value, int keys, int lane) {
  constexpr int kN = KvAtom<D>::kN, kW = KvAtom<D>::kW;
  if (!value) {
    const int r = lane & 7, j = lane >> 3;
    uint32_t s2[2 * kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const uint32_t h = e4m3x2_to_f16x2(x.sf[i / 2] >> (16 * (i % 2)));
      s2[2 * i] = both_halves(h, 0);
      s2[2 * i + 1] = both_halves(h, 1);
    }
#pragma unroll
    for (int p = 0; p < kN; ++p) {
      const uint32_t w[4] = {x.codes[p].x, x.codes[p].y, x.codes[p].z, x.codes[p].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int s = 2 * p + i / 2;                       // block of the lane's sequence
        const int dim8 = (j * kN + s % kN) * 2 + (i & 1);  // 8-dimension group of the row
        store8(slot, token0 + r + 8 * (s / kN), dim8 >> 3, dim8 & 7, w[i], s2[s]);
      }
    }
  } else {
    const int r = lane >> 2, j = lane & 3, odd = r & 1;
    constexpr int kVW = D / 64;  // words of 8 dimensions per token
    uint32_t s2[4][kW];
    {
      uint32_t sf[kW];
#pragma unroll
      for (int i = 0; i < kW; ++i) sf[i] = x.sf[i];
      if (keys < 16) {
#pragma unroll
        for (int i = 0; i < 4 * kW; ++i) {
          const int t = i / kW;
          if (8 * (t >> 1) + 2 * j + (t & 1) >= keys) sf[i >> 2] &= ~(0xFFu << (8 * (i & 3)));
        }
      }
#pragma unroll
      for (int i = 0; i < 2 * kW; ++i) {  // bytes: token, block
        const uint32_t h = e4m3x2_to_f16x2(sf[i / 2] >> (16 * (i % 2)));
        s2[(2 * i) / kW][(2 * i) % kW] = both_halves(h, 0);
        s2[(2 * i + 1) / kW][(2 * i + 1) % kW] = both_halves(h, 1);
      }
    }
#pragma unroll
    for (int p = 0; p < kN; ++p) {
      const uint32_t w[4] = {x.codes[p].x, x.codes[p].y, x.codes[p].z, x.codes[p].w};
      // Odd lanes take a pair's words the other way round, so that eight lanes
      // (two r, four j) store to eight different 16-byte columns.
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int q = 4 * p + i, t = q / kVW;  // word of the lane's sequence, its token
        const int token = token0 + 8 * (t >> 1) + 2 * j + (t & 1);
        if constexpr (D == 64) {
          store8(slot, token, 0, r, w[i], s2[t][0]);
        } else {
          const int dim8 = r * kVW + ((q % kVW) ^ odd);
          store8(slot, token, dim8 >> 3, dim8 & 7, odd ? w[i ^ 1] : w[i], s2[t][(q % kVW) / 2]);
        }
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) tiles_kernel(const AttnArgs a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[33];
  __shared__ uint32_t s_tmem, s_bad[kBad];
  __shared__ int s_gave_up;
  __shared__ Item s_item[2];  // this item and the next

  const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t ring = smem, qs = smem + 131072;
  const uint32_t bars = smem_u32(s_bar);
  // All of these count on through the CTA's items.
  auto full = [&](int s) { return bars + 8 * s; };          // a slot holds its block
  auto empty = [&](int s) { return bars + 64 + 8 * s; };    // products that read a slot are done
  auto s_full = [&](int t) { return bars + 128 + 8 * t; };  // S of a tile (or buffer)
  auto p_full = [&](int t, int half) { return bars + 144 + 16 * t + 8 * half; };  // 64 keys of P of a tile (or buffer)
  auto q_full = [&](int t) { return bars + 176 + 8 * t; };   // Q of a tile
  auto o_last = [&](int t) { return bars + 192 + 8 * t; };   // the last P V of a tile
  auto item_full = [&](int s) { return bars + 208 + 8 * s; };
  auto item_empty = [&](int s) { return bars + 224 + 8 * s; };
  const uint32_t o_done = bars + 240;
  const uint32_t drained = bars + 248;  // after a wait ran out
  const uint32_t item_due = bars + 256;  // the producers are near an item's end

  if (tid == 0) {
    for (int s = 0; s < 8; ++s) {
      mbar_init(full(s), C::kProducerWarps);
      mbar_init(empty(s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(s_full(t), 1);
      mbar_init(p_full(t, 0), 4);
      mbar_init(p_full(t, 1), 4);
      mbar_init(q_full(t), 4);
      mbar_init(o_last(t), 1);
      mbar_init(item_full(t), 1);
      mbar_init(item_empty(t), 13);  // every warp that takes items
    }
    mbar_init(o_done, 1);
    mbar_init(drained, 1);
    mbar_init(item_due, 1);
    s_gave_up = 0;
    for (int i = 0; i < kBad; ++i) s_bad[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    fence_before();
  }
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();
  fence_after();
  const uint32_t tmem = s_tmem;
  volatile int* gave_up = &s_gave_up;
  // Waits for the CTA's k-th item; false: there is none.
  auto take = [&](int k) { return mbar_wait_warp<true>(item_full(k & 1), (k >> 1) & 1, gave_up) && s_item[k & 1].rows > 0; };
  auto leave = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(item_empty(k & 1));
  };

  if (warp < 4 * C::kTiles) {
    // ------------------------------------------------------------ softmax ----
    regs_inc<C::kRegsSoftmax>();
    const int t = warp >> 2, row = tid;  // row of the item; tile t's thread holds lane row % 128
    const uint32_t lanes = uint32_t(warp & 3) << 21;  // tensor memory: lane in the upper half
    const uint32_t o_addr = tmem + lanes + C::kOCol + t * D;
    uint32_t done = 0;  // blocks of this tile so far; bit 31: parity of o_last
    bool ok = true;
#pragma unroll 1
    for (int k = 0; ok && take(k); leave(k++)) {
      const Item& it = s_item[k & 1];  // read again where it is used: the block loop needs the registers
      const int n = it.blocks;
      if (it.rows <= 128 * t) continue;
      float c = 0.0f;
      // Without keys no queries are laid out and q_full does not count: nothing but o_last holds these warps to the
      // products' pace, so they could pass two of its phases, which one parity cannot tell apart.
      if (n > 0) {
        // The row, scaled by a power of two (and the score factor's sign), as f16.
        const bool live = row < it.rows;
        const int x = it.row0 + row, token = x / a.group;
        const uint16_t* qp = a.q + int64_t(it.q0 + token) * a.ld_qt + int64_t(it.head * a.group + x - token * a.group) * a.ld_qh;
        // A warp's 32 rows, D / 8 lanes to a row, 16 loads on their way at once (a
        // thread's own row in turns of four: 8 us an item).
        constexpr int kLanes = D / 8, kPer = 32 / kLanes, kBatch = kLanes < 16 ? kLanes : 16;
        const uint64_t own = live ? reinterpret_cast<uint64_t>(qp) : 0;
        const float factor = a.scale_log2 * __ldg(a.k_scale);
        auto power = [](float amax) {  // of two, to which the row's largest is scaled
          const int e = int(__float_as_uint(amax) >> 23) - 127;
          return amax == 0.0f || e > 127 ? 0 : min(14 - e, kMostPower);
        };
        const uint32_t q_tile = qs + t * C::kQBytes;
        float mine = 0.0f;  // this thread's row's largest
        auto put = [&](const uint4& raw, int i) {  // rows i kPer ... of the warp
          float v[8], amax = 0.0f;
          unpack_bf16x8(raw, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
          const float row_max = __shfl_sync(kFull, amax, (lane % kPer) * kLanes);
          if (lane / kPer == i) mine = row_max;
          const float up = copysignf(__uint_as_float(uint32_t(power(amax) + 127) << 23), factor);
          uint32_t h[4];
#pragma unroll
          for (int e2 = 0; e2 < 4; ++e2) h[e2] = pack_f16x2(v[2 * e2] * up, v[2 * e2 + 1] * up);
          const int at = (warp & 3) * 32 + i * kPer + lane / kLanes, piece = lane % kLanes;
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(q_tile + (piece >> 3) * 16384 + at * 128 +
                                                                       (((piece & 7) ^ (at & 7)) << 4)),
                       "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                       : "memory");
        };
        auto from = [&](int i) {
          const uint64_t row_p = __shfl_sync(kFull, own, i * kPer + lane / kLanes);
          return row_p ? reinterpret_cast<const uint16_t*>(row_p) + 8 * (lane % kLanes) : nullptr;
        };
        if (__all_sync(kFull, (own & 15) == 0)) {
#pragma unroll 1
          for (int b = 0; b < kLanes; b += kBatch) {
            uint4 raw[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const uint16_t* p = from(b + i);
              raw[i] = p ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) put(raw[i], b + i);
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < kLanes; ++i) {
            const uint16_t* p = from(i);
            uint32_t w[4] = {0u, 0u, 0u, 0u};
            if (p)
#pragma unroll
              for (int e = 0; e < 4; ++e) w[e] = uint32_t(p[2 * e]) | (uint32_t(p[2 * e + 1]) << 16);
            put(make_uint4(w[0], w[1], w[2], w[3]), i);
          }
        }
        // At least the smallest normal number: 0 would make NaN of a masked key's -inf.
        c = fmaxf(fabsf(factor) * __uint_as_float(uint32_t(127 - power(mine)) << 23), 1.17549435e-38f);
        fence_smem_to_mma();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full(t));
      }
      int lo = 0, hi = 0;  // keys in sight, relative to the first block
      const bool live = row < it.rows;
      if (live) {
        const int64_t pos = int64_t(it.kv_len) - it.q_len + (it.row0 + row) / a.group;
        hi = (a.causal ? int(min(int64_t(it.kv_len), max(int64_t(0), pos + 1))) : it.kv_len) - it.first;
        lo = (a.window > 0 ? int(max(int64_t(0), pos + 1 - a.window)) : 0) - it.first;
      }
      // Blocks that every row of the warp sees whole need no mask.
      int lo_all = live ? lo : -0x7fffffff, hi_all = live ? hi : 0x7fffffff;
#pragma unroll
      for (int w = 1; w < 32; w <<= 1) {
        lo_all = max(lo_all, __shfl_xor_sync(kFull, lo_all, w));
        hi_all = min(hi_all, __shfl_xor_sync(kFull, hi_all, w));
      }
      float m = -INFINITY;
      float2 l2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
      for (int i = 0; i < n; ++i, ++done) {
        const int buf = C::kTiles == 2 ? t : (done & 1);
        const uint32_t par = (C::kTiles == 2 ? done : done >> 1) & 1;
        const uint32_t s_addr = tmem + lanes + buf * 128;
        if (!(ok = mbar_wait_warp(s_full(buf), par, gave_up))) break;
        fence_after();
        uint32_t sv[128];
#pragma unroll
        for (int p = 0; p < 4; ++p) tmem_load32(s_addr + 32 * p, sv + 32 * p);
        tmem_wait_load();
        const uint32_t bad = s_bad[(it.before + i) % kBad];
        const int k0 = i * kBlock;
        const bool masked = k0 < lo_all || k0 + kBlock > hi_all || bad != 0;
        if (masked) {
#pragma unroll
          for (int e = 0; e < 128; ++e)
            if (k0 + e < lo || k0 + e >= hi || ((bad >> (e / 16)) & 1u)) sv[e] = 0xFF800000u;  // -inf
        }
        float tops[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          tops[y] = fmaxf(__uint_as_float(sv[32 * y]), __uint_as_float(sv[32 * y + 1]));
#pragma unroll
          for (int e = 2; e < 32; e += 2)
            tops[y] = fmax3(tops[y], __uint_as_float(sv[32 * y + e]), __uint_as_float(sv[32 * y + e + 1]));
        }
        const float top = __fmaf_rn(fmaxf(fmax3(tops[0], tops[1], tops[2]), tops[3]), c, -kHeadroom);
        const bool raise = top > m + kRaise;
        if (__any_sync(kFull, raise)) {
          const float f = raise ? ex2(m - top) : 1.0f;
          if (raise) m = top;
#pragma unroll
          for (int y = 0; y < 2; ++y) l2[y] = make_float2(l2[y].x * f, l2[y].y * f);
          if (i > 0) {
            // Tiles in turn: S of block i was issued after P V of block i - 1, so O
            // is at rest.  Two S buffers: S of block i was issued after P V of block
            // i - 2, so o_done has completed done - 1 or done times and the parity
            // tells which; wait for the last.
            if (C::kTiles == 1) {
              if (!(ok = mbar_wait_warp(o_done, (done - 1) & 1, gave_up))) break;
              fence_after();
            }
#pragma unroll 1
            for (int p = 0; p < D / 32; ++p) {
              uint32_t ov[32];
              tmem_load32(o_addr + 32 * p, ov);
              tmem_wait_load();
#pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f);
              tmem_store32(o_addr + 32 * p, ov);
            }
            tmem_wait_store();
          }
        }
        const float2 c2 = make_float2(c, c);
        const float nm = m == -INFINITY ? 0.0f : -m;
        const float2 nm2 = make_float2(nm, nm);
        // Two halves of 64 keys, each handed over on its own, so that P V starts
        // under the second half's exponentials.
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          uint32_t pv[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float2 v = __ffma2_rn(
                make_float2(__uint_as_float(sv[64 * p + 2 * e]), __uint_as_float(sv[64 * p + 2 * e + 1])), c2, nm2);
            const float2 w = make_float2(ex2(v.x), ex2(v.y));
            l2[e & 1] = __fadd2_rn(l2[e & 1], w);
            pv[e] = pack_f16x2(w.x, w.y);
          }
          tmem_store32(s_addr + 32 * p, pv);
          tmem_wait_store();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(buf, p));
        }
      }
      // ---- output: this thread's row
      if (ok && n > 0) {
        ok = mbar_wait_warp(o_last(t), done >> 31, gave_up);
        done ^= 1u << 31;
        fence_after();
      }
      float l = (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
      if (l > 0.0f) l += nan_of(a.scale_log2 * __ldg(a.k_scale));
      const int x = it.row0 + row, token = x / a.group, head = it.head * a.group + x - token * a.group;
      const int64_t at = it.q0 + token;
      float* part = nullptr;
      if (a.splits > 1) part = partials_of(a) + (int64_t(it.index) * a.splits + it.split) * (C::kRows * (D + 2)) + row * D;
      const float f = l > 0.0f || l != l ? __ldg(a.v_scale) / l : 0.0f;
      uint16_t* orow = a.out + at * a.ld_ot + int64_t(head) * a.ld_oh;
      const uint64_t own = live ? reinterpret_cast<uint64_t>(orow) : 0;
      const bool wide = part == nullptr && __all_sync(kFull, (own & 15) == 0);
      if (ok) {
#pragma unroll 1
        for (int p = 0; p < D / 32; ++p) {
          uint32_t ov[32];
          if (n > 0) {
            tmem_load32(o_addr + 32 * p, ov);
            tmem_wait_load();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = 0u;
          }
          if (wide) {  // over the tile's queries, whose products are done
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              w[e] = pack_bf16x2(__uint_as_float(ov[2 * e]) * f, __uint_as_float(ov[2 * e + 1]) * f);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int piece = 4 * p + e;
              asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(qs + t * C::kQBytes + (piece >> 3) * 16384 + (row & 127) * 128 +
                                                                           (((piece & 7) ^ (row & 7)) << 4)),
                           "r"(w[4 * e]), "r"(w[4 * e + 1]), "r"(w[4 * e + 2]), "r"(w[4 * e + 3])
                           : "memory");
            }
            continue;
          }
          if (!live) continue;
          if (part != nullptr) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(part + 32 * p + e) = make_uint4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
            continue;
          }
          uint16_t* op = orow + 32 * p;
#pragma unroll
          for (int e = 0; e < 32; ++e) op[e] = f32_to_bf16(__uint_as_float(ov[e]) * f);
        }
        if (wide) {
          __syncwarp();
          constexpr int kLanes = D / 8, kPer = 32 / kLanes;
#pragma unroll 8
          for (int i = 0; i < kLanes; ++i) {
            const int in = i * kPer + lane / kLanes, at_row = (warp & 3) * 32 + in, piece = lane % kLanes;
            const uint64_t to = __shfl_sync(kFull, own, in);
            uint4 w;
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                         : "r"(qs + t * C::kQBytes + (piece >> 3) * 16384 + at_row * 128 + (((piece & 7) ^ (at_row & 7)) << 4))
                         : "memory");
            if (to) *(reinterpret_cast<uint4*>(to) + piece) = w;
          }
        }
        if (live) {
          if (part != nullptr)
            *reinterpret_cast<float2*>(part - row * D + C::kRows * D + 2 * row) = make_float2(m, l);
          else if (a.lse != nullptr)
            a.lse[at * a.ld_lse + head] = lse_of(m, l);
        }
      }
    }
  } else if (warp < 12) {
    // ---------------------------------------------------------- producers ----
    if constexpr (C::kRegsProducer < 128) regs_dec<C::kRegsProducer>();
    constexpr int kMine = kAtoms / C::kProducerWarps;  // atoms of a block per warp
    const int pw = warp - 4 * C::kTiles;
    int q = 0;  // blocks of K and V filled
    bool ok = true;
#pragma unroll 1
    for (int k = 0; ok && take(k); ++k) {
      const Item it = s_item[k & 1];
      leave(k);
      const int n = it.blocks;
      const int32_t* table = a.table + int64_t(it.b) * a.ld_table;
      const int64_t head_off = int64_t(it.head) * (int64_t(KvAtom<D>::kBytes) << (a.cache.log_page - 4));
      auto token_of = [&](int block, int i) { return it.first + block * kBlock + 16 * (pw + C::kProducerWarps * i); };
      // Pages of this warp's atoms of a block; -1: none (out of the cache), -2: behind the last key.
      struct Pages {
        int32_t of[kMine];
      };
      auto pages_of = [&](int block) {
        Pages p;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const int t = token_of(block, i);
          p.of[i] = -2;
          if (block < n && t < it.kv_len) {
            const int32_t page = __ldg(table + (t >> a.cache.log_page));
            p.of[i] = page < 0 || page >= a.cache.pages ? -1 : page;
          }
        }
        return p;
      };
      struct Raw {
        RawAtom<D> atom[kMine];
      };
      auto fetch = [&](Raw& raw, int block, const Pages& p, bool value) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const int t = token_of(block, i);
          const uint8_t* atom = p.of[i] < 0 ? nullptr
                                            : a.cache.base + p.of[i] * a.cache.page_stride + head_off +
                                                  ((t & ((1 << a.cache.log_page) - 1)) >> 4) * KvAtom<D>::kBytes;
          load_atom<D>(raw.atom[i], atom, value, lane);
        }
      };
      // A block's bytes on their way to L2, as from HBM they take longer than a block: 32 chunks of 64 tokens over
      // 4096 keys 172 -> 168 us.  (With heads of 256 a prompt of 8192 lost, 576 -> 594: off there.)
      auto warm = [&](int block, const Pages& p) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const int t = token_of(block, i);
          const uint8_t* atom = a.cache.base + p.of[i] * a.cache.page_stride + head_off +
                                ((t & ((1 << a.cache.log_page) - 1)) >> 4) * KvAtom<D>::kBytes;
#pragma unroll
          for (int at = 0; at < KvAtom<D>::kBytes; at += 4096)
            if (p.of[i] >= 0 && at + 128 * lane < KvAtom<D>::kBytes)
              asm volatile("prefetch.global.L2 [%0];" ::"l"(atom + at + 128 * lane));
        }
      };
      auto convert = [&](const Raw& raw, int block, bool value) {
        const int slot = q % C::kSlots, round = q / C::kSlots;
        ++q;
        if (round > 0 && !(ok = mbar_wait_warp(empty(slot), (round - 1) & 1, gave_up))) return;
#pragma unroll
        for (int i = 0; i < kMine; ++i)
          convert_atom<D>(raw.atom[i], ring + slot * C::kSlotBytes, 16 * (pw + C::kProducerWarps * i), value,
                          it.kv_len - token_of(block, i), lane);
        fence_smem_to_mma();
        __syncwarp();
        if (lane == 0) mbar_arrive(full(slot));
      };
      // Atoms without a page: their keys count as out of sight.  Written before
      // the block's K slot is filled.
      auto note_missing = [&](int block, const Pages& p) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const uint32_t bit = 1u << (pw + C::kProducerWarps * i);
          if (lane == 0) {
            if (p.of[i] == -1) {
              atomicOr(&s_bad[(it.before + block) % kBad], bit);
              atomicOr(a.err, kErrSlot);
            } else {
              atomicAnd(&s_bad[(it.before + block) % kBad], ~bit);
            }
          }
        }
      };
      // The stream: tiles in turn K0 V0 K1 V1 ..., two S buffers K0 K1 V0 K2 V1 ...
      // The bytes of the next block's keys (values) are on their way while this
      // block's are converted, and the pages of the block after that.
      Raw raw_k, raw_v;
      Pages now = pages_of(0), next = pages_of(1), later = pages_of(2);
      fetch(raw_k, 0, now, false);
      fetch(raw_v, 0, now, true);
      if (C::kTiles == 2) warm(1, next);
      // Near the end, and not before, the CTA claims its next item: whoever is free first gets it.
      const int due = max(0, n - 5);
      if (n == 0 && pw == 0 && lane == 0) mbar_arrive(item_due);
      if (C::kTiles == 1 && n > 0) {
        note_missing(0, now);
        convert(raw_k, 0, false);
        fetch(raw_k, 1, next, false);
      }
      for (int i = 0; i < n && ok; ++i) {
        const int kb = C::kTiles == 2 ? i : i + 1;
        if (C::kTiles == 2) warm(i + 2, later);
        if (i == due && pw == 0 && lane == 0) mbar_arrive(item_due);
        if (kb < n) {
          const Pages& kp = C::kTiles == 2 ? now : next;
          note_missing(kb, kp);
          convert(raw_k, kb, false);
          if (!ok) break;
          fetch(raw_k, kb + 1, C::kTiles == 2 ? next : later, false);
        }
        convert(raw_v, i, true);
        if (!ok) break;
        fetch(raw_v, i + 1, next, true);
        now = next;
        next = later;
        later = pages_of(i + 3);
      }
    }
  } else {
    regs_dec<C::kRegsMma>();
    if (warp == 13) {
      // ------------------------------------------------------------- items ----
      // The next item is found while this one is worked on.  The first is the
      // CTA's own number, further ones are claimed.
      const int total = a.tiles * a.cache.heads * a.splits;
      int next = int(blockIdx.x), before = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        Item it{};
        if (k > 0 && !(ok = mbar_wait_warp<true>(item_due, (k - 1) & 1, gave_up))) break;
        while (true) {
          if (next < 0) {
            if (lane == 0) next = int(gridDim.x + atomicAdd(claims_of(a), 1u));
            next = __shfl_sync(kFull, next, 0);
          }
          if (next >= total) break;
          it = find_item<C::kRows>(a, next, lane);
          next = -1;
          if (it.rows > 0) break;
        }
        if (k > 1 && !(ok = mbar_wait_warp<true>(item_empty(k & 1), ((k >> 1) - 1) & 1, gave_up))) break;
        it.before = before;
        before += it.blocks;
        if (lane == 0) {
          s_item[k & 1] = it;
          mbar_arrive(item_full(k & 1));
        }
        if (it.rows == 0) break;
      }
    } else if (warp == 12) {
      // ---------------------------------------------------------- products ----
      // The whole warp walks the loop, so that descriptors and counters stay in
      // uniform registers; one elected lane issues.  Rolled loops: this code runs
      // for a moment between long waits, and unrolled it was slowed to 100 cycles
      // per product by instruction fetches (a prompt of 8192: 757 us).
      const bool leader = elect_one();
      const uint32_t tm = __shfl_sync(kFull, tmem, 0);
      constexpr uint32_t kIdQK = instruction(kBlock, false), kIdPV = instruction(D, true);
      bool ok = true;
      auto wait_slot = [&](int q) {
        ok = ok && mbar_wait_warp(full(q % C::kSlots), (q / C::kSlots) & 1, gave_up);
        fence_after();
      };
      auto arrive = [&](uint32_t bar) {
        if (leader) commit(bar);
        __syncwarp();
      };
      auto qk = [&](int t, int s_col, int q) {
        uint64_t qd = matrix(qs + t * C::kQBytes), kd = matrix(ring + (q % C::kSlots) * C::kSlotBytes);
#pragma unroll 1
        for (int k = 0; k < C::kChunks; ++k) {
          if (leader) {
#pragma unroll
            for (int x = 0; x < 4; ++x) mma_ss(tm + s_col, qd + 2 * x, kd + 2 * x, kIdQK, k > 0 || x > 0);
          }
          __syncwarp();
          qd += 16384 >> 4;
          kd += 16384 >> 4;
        }
      };
      auto pv = [&](int t, int buf, uint32_t parity, int q, bool first) {
        uint64_t vd = matrix(ring + (q % C::kSlots) * C::kSlotBytes);
        const uint32_t o = tm + C::kOCol + t * D;
        uint32_t p = tm + 128 * buf;
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          if (!(ok = mbar_wait_warp(p_full(buf, k), parity, gave_up))) return;
          fence_after();
          if (leader) {
#pragma unroll
            for (int x = 0; x < 4; ++x) mma_ts(o, p + 8 * x, vd + x * (2048 >> 4), kIdPV, k > 0 || x > 0 || !first);
          }
          __syncwarp();
          p += 32;
          vd += 8192 >> 4;
        }
      };
      int q = 0, done = 0;                // blocks of K and V used; S buffers filled (two buffers)
      uint32_t p_par = 0, q_par = 0;      // bit t: parity of p_full (tiles in turn) and q_full of tile t
#pragma unroll 1
      for (int item = 0; ok && take(item); ++item) {
        const int n = s_item[item & 1].blocks, tiles = s_item[item & 1].rows > 128 ? 2 : 1;
        leave(item);
        const uint32_t both = uint32_t(tiles) | 1u;  // bit t: tile t has rows
        if (n == 0) continue;  // no barrier but the item's own takes part in it
        const uint32_t q_now = q_par;
        q_par ^= both;
        auto wait_q = [&](int t) {
          ok = ok && mbar_wait_warp(q_full(t), (q_now >> t) & 1, gave_up);
          fence_after();
        };
        wait_slot(q);
        if constexpr (C::kTiles == 2) {
          for (int t = 0; t < tiles && ok; ++t) {
            wait_q(t);
            if (!ok) break;
            qk(t, 128 * t, q);
            arrive(s_full(t));
          }
          if (ok) arrive(empty(q % C::kSlots));
#pragma unroll 1
          for (int i = 0; i < n && ok; ++i) {
            // The producers fill V(i) before K(i + 1): one wait covers both.
            const int qv = q + 2 * i + 1, qn = qv + 1;
            wait_slot(i + 1 < n ? qn : qv);
#pragma unroll 1
            for (int t = 0; t < tiles && ok; ++t) {
              pv(t, t, ((p_par >> t) ^ uint32_t(i)) & 1, qv, i == 0);
              if (!ok) break;
              if (i + 1 < n) qk(t, 128 * t, qn);
              arrive(i + 1 < n ? s_full(t) : o_last(t));
            }
            if (!ok) break;
            arrive(empty(qv % C::kSlots));
            if (i + 1 < n) arrive(empty(qn % C::kSlots));
          }
          if (n & 1) p_par ^= both;
        } else {
          // K0 K1 V0 K2 V1 ... K(n-1) V(n-2) V(n-1)
          wait_q(0);
          if (!ok) break;
          int at = q;
          qk(0, 128 * (done & 1), at);
          arrive(s_full(done & 1));
          arrive(empty(at % C::kSlots));
          ++at;
#pragma unroll 1
          for (int i = 0; i < n && ok; ++i) {
            const int buf = (done + i) & 1;
            if (i + 1 < n) {
              wait_slot(at);
              if (!ok) break;
              qk(0, 128 * (buf ^ 1), at);
              arrive(s_full(buf ^ 1));
              arrive(empty(at % C::kSlots));
              ++at;
            }
            wait_slot(at);
            if (!ok) break;
            pv(0, buf, ((done + i) >> 1) & 1, at, i == 0);
            if (!ok) break;
            arrive(empty(at % C::kSlots));
            arrive(o_done);
            ++at;
          }
          done += n;
          if (ok) arrive(o_last(0));
        }
        q += 2 * n;
      }
      if (__any_sync(kFull, !ok || *gave_up)) {
        // Products in flight end before their tensor memory is freed.
        arrive(drained);
        for (int i = 0; i < (1 << 20) && !mbar_try(drained, 0); ++i) {
        }
      }
    }
    __syncwarp();
  }
  fence_before();
  __syncthreads();
  if (tid == 0) {
    if (s_gave_up) atomicOr(a.err, kErrWait);
    // The last CTA leaves the counters at zero (its own wraps around).
    if (atomicInc(done_of(a), gridDim.x - 1) == gridDim.x - 1) *claims_of(a) = 0;
  }
  if (warp == 12) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// Joins the splits of a CTA's rows: a warp per row.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const AttnArgs a) {
  constexpr int R = Cfg<D>::kRows, kSlot = R * (D + 2);
  griddep_wait();
  griddep_launch_dependents();
  const int part = int(blockIdx.x) % (R / 8);
  const int row = part * 8 + int(threadIdx.x >> 5), lane = int(threadIdx.x) & 31;
  const Item it = find_item<R>(a, int(blockIdx.x) / (R / 8) * a.splits, lane);
  if (row >= it.rows) return;
  const int x = it.row0 + row, token = x / a.group, head = it.head * a.group + x - token * a.group;
  const float* base = partials_of(a) + int64_t(it.index) * a.splits * kSlot;
  float top = -INFINITY, l = 0.0f;
  float o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = 0.0f;
  for (int s = 0; s < a.splits; ++s) {
    const float2 st = __ldcg(reinterpret_cast<const float2*>(base + int64_t(s) * kSlot + R * D + 2 * row));
    const float up = fmaxf(top, st.x);
    const float f0 = top == up ? 1.0f : ex2(top - up), f1 = st.x == up ? 1.0f : ex2(st.x - up);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = o[i] * f0 + __ldcg(base + int64_t(s) * kSlot + row * D + 32 * i + lane) * f1;
    l = l * f0 + st.y * f1;
    top = up;
  }
  const float f = l > 0.0f || l != l ? __ldg(a.v_scale) / l : 0.0f;
  const int64_t at = it.q0 + token;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
    a.out[at * a.ld_ot + int64_t(head) * a.ld_oh + 32 * i + lane] = f32_to_bf16(o[i] * f);
  if (lane == 0 && a.lse != nullptr)
    a.lse[at * a.ld_lse + head] = lse_of(top, l);
}

}  // namespace

AttnTiles attn_tiles(int d) {
#define NQ_TILES(D) \
  if (d == D)       \
    return {reinterpret_cast<const void*>(&tiles_kernel<D>), reinterpret_cast<const void*>(&join_kernel<D>), Cfg<D>::kRows, size_t(Cfg<D>::kSmem)};
  NQ_TILES(64) NQ_TILES(128) NQ_TILES(256)
#undef NQ_TILES
  return {nullptr, nullptr, 0, 0};
}

}  // namespace nq

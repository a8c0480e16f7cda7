// nq_attention_rows.cu — attention over the 4-bit cache for few rows per request
// (single tokens, draft verification): each warp streams atoms of 16 tokens
// through matrix products whose fragments are the cache's own byte order.
//
//   s_j = c <q, k'_j>,  m = max s_j - 7,  p_j = 2^(s_j - m),  l = sum p_j,
//   o = g_v / l * sum p_j v'_j,  lse = ln 2 (m + log2 l),
// with k', v' = e2m1 * e4m3 and c = scale * log2(e) * g_k.
//
// Numerics.  k' and v' have at most six significant bits and lie in [2^-10,
// 2688], so they are exact in f16.  A query row is scaled by a power of two to
// a largest magnitude in [2^14, 2^15): its bf16 values are then exact in f16
// down to 2^-28 of the row's largest (a row whose largest lies below 2^-112, to
// one below 2^14, and exact down to 2^-126 * 2^-24).  Products accumulate in float32.  p is
// rounded to f16: half a step is 2^-11 of it, an eighth of the bf16 output's,
// and 2^-32 of the row's largest where that is more (f16's subnormal numbers),
// which n keys can lose of a sum of p once each, less than the 2^-24 of the
// sum that each of n additions in float32 may lose.  l sums the float32
// values.  m lies 2^7 below the running maximum, and that is only raised when
// a score exceeds it by more than 2^8: p stays at or below 2^15, and the
// accumulators are rescaled once or twice per row instead of at every atom.
//
// Work.  S^T = K' q^T and O^T = V'^T P^T put the 16 tokens (or dimensions) on
// the 16-row side of the product and up to 8 rows of a (request, kv head) on
// its 8-column side.  An atom of D = 128 (2304 bytes) costs a warp scheduler about
// 405 cycles: the conversion of its codes and the products share the issue slots
// (61 % of them used), and each warp's chain of scores, vote, weights and values,
// with 3.5 warps a scheduler to cover it, binds before HBM does (128 ragged requests
// to 8192 keys, 8 kv heads: 154 us, 0.66 of copy bandwidth; 2 requests of 131071
// keys 72 us, 0.64).
//
// Split.  The atoms of all (request, row tile, kv head) segments form one axis,
// which is shared out equally whatever the lengths, in one of two ways:
//  - many segments (WALK): every warp takes a contiguous share and walks the
//    segments in it on its own, without a barrier, so that one warp's change of
//    segment (five dependent loads) passes under the others' work.  A segment
//    inside one share is written out by its warp; the parts of one that is cut
//    go to the workspace, and a second launch, which starts under the first
//    one's end, joins them.
//  - few segments: every CTA takes one chunk of one segment, of 32 atoms or more,
//    its warps an eighth each; they are joined in shared memory, and the CTA
//    that arrives last at a segment's counter joins its chunks.  One launch: a
//    second one costs as much as a short context takes.
// Parts are joined in the order of the tokens, so results do not depend on
// timing.  No CTA waits for another.
// (The first way by CTAs instead of warps: every segment cost 5 us of loads,
// barriers and fences; 128 ragged requests 172 us.)
#include "nq_kv_layout.cuh"

namespace nq {

namespace {

constexpr int kWalkWarps = 4, kChunkWarps = 8;
constexpr float kLowest = -3.0e38f; // the maximum of no scores: below every finite one, and 0 * 2^(kLowest - kLowest) is 0

constexpr int stages_of(int d) { return d == 64 ? 3 : 2; }  // pairs of atoms
constexpr size_t ring_bytes(int d, int warps) { return size_t(warps) * stages_of(d) * 36 * d; }
constexpr int row_pitch(int d) { return d + 4; }  // floats between rows of a warp's result in shared memory
constexpr size_t merge_bytes(int d, int rows) { return size_t(kChunkWarps) * rows * (row_pitch(d) + 2) * 4; }

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Waits for the phase of the given parity; false when the limit runs out (no wait of a sound run comes near it).
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
  for (int i = 0; i < (1 << 22); ++i) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    if (ok) return true;
  }
  return false;
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}
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
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// first: the accumulator starts from zero.
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1, bool first = false) {
  if (first)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int N>
struct IntTag {
  static constexpr int value = N;
};

// One request's share of the axis.
struct Span {
  int q0, q_len, kv_len;  // first query row, rows, keys
  int first;              // first key any row sees, rounded down to an atom
  int tiles, units;       // row tiles; atoms of keys per tile and kv head
};
// A quotient that mostly fits 32 bits (a 64-bit division is 100 instructions).
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t d) {
  return (uint64_t(x | d) >> 32) == 0 ? int64_t(uint32_t(x) / uint32_t(d)) : x / d;
}
template <int R>
__device__ __forceinline__ Span span_of(const AttnArgs& a, int b) {
  Span s;
  const int room = a.width << a.cache.log_page;  // at most 2^30, as the window; rows stay below 2^30 too
  const int c0 = min(max(__ldg(a.cu_q + b), 0), a.T), c1 = min(max(__ldg(a.cu_q + b + 1), c0), a.T);
  s.q0 = c0;
  s.q_len = c1 - c0;
  s.kv_len = min(max(__ldg(a.kv_lens + b), 0), room);
  s.first = 0;
  if (a.window > 0) s.first = max(0, s.kv_len - s.q_len + 1 - a.window) & ~15;
  s.tiles = (s.q_len * a.group + R - 1) / R;
  s.units = max(1, (s.kv_len - s.first + 15) >> 4);
  return s;
}

// What the joining launch needs to know of a segment that was cut.
struct __align__(16) Cut {
  int32_t first, last, head, q0;  // parts, kv head, first query row of the request
  int32_t row0, rows, pad0, pad1;  // first row and rows of the tile
};
// The workspace: counters, zero between calls: of the chunked segments and, the
// last three of them, of the walk's claimed parts, its cuts and the joining CTAs
// that are done; then the cuts, in any order, and the parts' slots, each of R rows
// of D floats and R pairs (maximum, sum).
__device__ __forceinline__ uint32_t* counters_of(const AttnArgs& a) { return reinterpret_cast<uint32_t*>(a.workspace); }
enum WalkCounter { kClaims = 1, kCuts, kDone };
__device__ __forceinline__ uint32_t* counter_of(const AttnArgs& a, WalkCounter c) {
  return counters_of(a) + kAttnCounterBytes / 4 - c;
}
__device__ __forceinline__ Cut* cuts_of(const AttnArgs& a) { return reinterpret_cast<Cut*>(a.workspace + kAttnCounterBytes); }
template <int D, int R>
__device__ __forceinline__ float* slot_of(const AttnArgs& a, int64_t i) {
  return reinterpret_cast<float*>(a.workspace + kAttnHeader) + i * (R * (D + 2));
}

__device__ __forceinline__ void store_pair(uint16_t* op, float x0, float x1) {
  const uint32_t v = pack_bf16x2(x0, x1);
  if ((reinterpret_cast<uintptr_t>(op) & 3) == 0) {
    *reinterpret_cast<uint32_t*>(op) = v;
  } else {
    op[0] = uint16_t(v);
    op[1] = uint16_t(v >> 16);
  }
}
__device__ __forceinline__ float out_factor(float sum, float gv) { return sum > 0.0f || sum != sum ? gv / sum : 0.0f; }

// Joins n parts of a tile (part p at slot(p)), in order, with THREADS threads of a
// CTA, and writes the rows out.  Weights first, then the rows in independent
// loads: one dependent load a part would cost 0.7 us each.
template <int D, int R, int THREADS>
struct Join {
  static constexpr int kMax = 64;  // parts at a time
  float weight[kMax * R], sum[kMax * R], top[R], l[R], f[R];

  template <typename Slot>
  __device__ __forceinline__ void run(const AttnArgs& a, int n, Slot&& slot, const Cut& cut, float gv) {
    constexpr int kE = (R * D / 4 + THREADS - 1) / THREADS;
    constexpr int kBatch = kE >= 16 ? 1 : 16 / kE;  // parts whose rows are on their way together
    const int tid = int(threadIdx.x);
    float4 x[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) x[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    __syncthreads();  // a tile joined before has been written out
    if (tid < R) top[tid] = kLowest, l[tid] = 0.0f;
    for (int p0 = 0; p0 < n; p0 += kMax) {
      const int here = min(kMax, n - p0);
      __syncthreads();
      for (int i = tid; i < here * R; i += THREADS) {
        const int row = i % R;
        const float2 st = row < cut.rows ? __ldcg(reinterpret_cast<const float2*>(slot(p0 + i / R) + R * D + 2 * row))
                                         : make_float2(kLowest, 0.0f);
        weight[i] = st.x;
        sum[i] = st.y;
      }
      __syncthreads();
      if (tid < R) {
        float m = top[tid];
#pragma unroll 8
        for (int p = 0; p < here; ++p) m = fmaxf(m, weight[p * R + tid]);
        const float g = ex2(top[tid] - m);
        float s = l[tid] * g;
#pragma unroll 8
        for (int p = 0; p < here; ++p) {
          const float w = ex2(weight[p * R + tid] - m);
          weight[p * R + tid] = w;
          s += w * sum[p * R + tid];
        }
        top[tid] = m;
        l[tid] = s;
        f[tid] = g;
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const int row = (e * THREADS + tid) / (D / 4);
        const float g = row < R ? f[row] : 0.0f;
        x[e] = make_float4(x[e].x * g, x[e].y * g, x[e].z * g, x[e].w * g);
      }
      for (int p = 0; p < here; p += kBatch) {
        float4 v[kBatch][kE];
#pragma unroll
        for (int q = 0; q < kBatch; ++q)
#pragma unroll
          for (int e = 0; e < kE; ++e) {
            const int i = e * THREADS + tid, row = i / (D / 4);
            v[q][e] = p + q < here && row < cut.rows
                          ? __ldcg(reinterpret_cast<const float4*>(slot(p0 + p + q) + row * D + 4 * (i % (D / 4))))
                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          }
#pragma unroll
        for (int q = 0; q < kBatch; ++q)
#pragma unroll
          for (int e = 0; e < kE; ++e) {
            const int row = (e * THREADS + tid) / (D / 4);
            if (p + q < here && row < cut.rows) {
              const float w = weight[(p + q) * R + row];
              x[e] = make_float4(x[e].x + w * v[q][e].x, x[e].y + w * v[q][e].y, x[e].z + w * v[q][e].z,
                                 x[e].w + w * v[q][e].w);
            }
          }
      }
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const int i = e * THREADS + tid, row = i / (D / 4), d = 4 * (i % (D / 4));
      if (row >= cut.rows) continue;
      const int y = cut.row0 + row, token = y / a.group, h = cut.head * a.group + y - token * a.group;
      const int64_t at = cut.q0 + token;
      const float g = out_factor(l[row], gv);
      uint16_t* op = a.out + at * a.ld_ot + h * a.ld_oh + d;
      store_pair(op, x[e].x * g, x[e].y * g);
      store_pair(op + 2, x[e].z * g, x[e].w * g);
      if (a.lse != nullptr && d == 0) a.lse[at * a.ld_lse + h] = lse_of(top[row], l[row]);
    }
  }
};

// CTAs of an SM (of 4 warps; of the chunks' 8, half as many).  128 x 16 rows at
// three instead of two spilled 500 bytes a thread: 24 x 16 rows over 4096 keys 71
// us, was 58.  (Chunks of 256 x 16 rows spill 534 bytes; as twice 8 rows each key
// is converted twice: 4 requests 42 us, with the spills 28.7.)
template <int D, int NT, bool WALK>
__global__ void __launch_bounds__((WALK ? kWalkWarps : kChunkWarps) * 32,
                                  (NT == 1 && D < 256 ? 4 : (NT == 2 && D == 64 ? 3 : 2)) * kWalkWarps / (WALK ? kWalkWarps : kChunkWarps))
    rows_kernel(const AttnArgs a) {
  constexpr int kWarps = WALK ? kWalkWarps : kChunkWarps, kThreads = kWarps * 32;
  constexpr int R = 8 * NT;  // rows of a tile: (token, head of the group), token-major
  constexpr int kStages = stages_of(D);
  constexpr int kN = KvAtom<D>::kN, kW = KvAtom<D>::kW;
  constexpr int kAtom = KvAtom<D>::kBytes;
  constexpr int kPitch = row_pitch(D);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t s_scan[kWarps], s_before[kThreads];
  __shared__ int s_last;
  __shared__ __align__(8) uint64_t s_bar[kWarps][kStages];  // a pair of atoms has landed

  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, j = lane & 3;
  const int heads = a.cache.heads;

  const uint32_t bars = uint32_t(__cvta_generic_to_shared(s_bar[warp]));
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(bars + 8 * i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  griddep_wait();
  griddep_launch_dependents();

  // ---- the axis: atoms of all requests (each thread counts a run of them)
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b_lo = min(a.B, tid * per), b_hi = min(a.B, b_lo + per);
  // Sum of `mine` over the CTA's threads, and over those before this one.
  auto scan = [&](int64_t mine, int64_t* before) {
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += up;
    }
    __syncthreads();
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    int64_t total = 0;
    *before = incl - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) *before += s_scan[w];
      total += s_scan[w];
    }
    return total;
  };
  int64_t mine = 0, segments = 0, before;
  for (int b = b_lo; b < b_hi; ++b) {
    const Span s = span_of<R>(a, b);
    mine += int64_t(s.tiles) * heads * s.units;
    segments += int64_t(s.tiles) * heads;
  }
  int64_t total = scan(mine, &before);

  // WALK: parts of the axis.  The first four fifths are one part a warp (of two
  // atoms or more); the rest, as many small ones, go to whoever is free:
  // the warps of an SM do not advance alike, and with equal shares alone the last
  // one was done a seventh after the average.  Else: chunks of `chunk` atoms that
  // no segment shares, one a CTA.
  int fixed = 0, parts = 0, chunk = 0;
  int64_t fixed_end = 0;
  auto start_of = [&](int p) {
    return p <= fixed ? quotient(fixed_end * p, fixed) : fixed_end + quotient((total - fixed_end) * (p - fixed), parts - fixed);
  };
  auto owner_of = [&](int64_t u) {
    return u < fixed_end ? int(quotient((u + 1) * fixed - 1, fixed_end))
                         : fixed + int(quotient((u - fixed_end + 1) * (parts - fixed) - 1, total - fixed_end));
  };
  if constexpr (WALK) {
    const int64_t warps = int64_t(gridDim.x) * kWarps;
    fixed = int(min(warps, (total + 1) >> 1));
    fixed_end = total;
    parts = fixed;
    if (fixed == warps && total >= 96 * warps) {  // small parts of 20 atoms or more: shorter ones cost more than they save
      fixed_end = total / 5 * 4;
      parts = 2 * fixed;
    }
  } else {
    int64_t unused;
    const int64_t all = scan(segments, &unused);
    // Sum over the segments of ceil(atoms / chunk) stays within the grid.
    const int64_t free = int64_t(gridDim.x) - all;
    chunk = int(max(int64_t(32), free > 0 ? (total + free - 1) / free : total));
    mine = 0;
    for (int b = b_lo; b < b_hi; ++b) {
      const Span s = span_of<R>(a, b);
      mine += int64_t(s.tiles) * heads * ((s.units + chunk - 1) / chunk);
    }
    total = scan(mine, &before);
  }
  auto units_of = [&](const Span& s) { return WALK ? s.units : (s.units + chunk - 1) / chunk; };  // of the axis, per segment
  s_before[tid] = before;
  __syncthreads();
  int part = int(blockIdx.x) + (WALK ? warp * int(gridDim.x) : 0);
  if (WALK ? part >= fixed : part >= total) return;
  int b;
  int64_t base;  // where request b begins on the axis
  // The first request of the run of requests in which position u lies.
  auto locate = [&](int64_t u) {
    int i = -1;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) i += __popc(__ballot_sync(kFull, s_before[q * 32 + lane] <= u));
    b = i * per;
    base = s_before[i];
  };

  const uint32_t ring = uint32_t(__cvta_generic_to_shared(smem)) + warp * (2 * kStages * kAtom);
  const uint8_t* ring_p = smem + warp * (2 * kStages * kAtom);
  const float gk = __ldg(a.k_scale), gv = __ldg(a.v_scale);
  const int64_t head_bytes = int64_t(kAtom) << (a.cache.log_page - 4);
  // The ring: slots in turn, their parity changes with every turn; all is read at a segment's end.
  int wr_slot = 0, rd_slot = 0;
  uint32_t rd_parity = 0;

  int64_t u0, u1;  // this part
  if constexpr (WALK) u0 = start_of(part), u1 = start_of(part + 1);
  else u0 = part, u1 = part + 1;
  int64_t u = u0;
  locate(u);
  while (true) {
    if constexpr (WALK) {
      if (u >= u1) {  // the part's end
        if (parts == fixed) return;
        if (lane == 0) part = fixed + int(atomicAdd(counter_of(a, kClaims), 1u));
        part = __shfl_sync(kFull, part, 0);
        if (part >= parts) return;
        u0 = u = start_of(part), u1 = start_of(part + 1);
        locate(u);
      }
    }
    Span s = span_of<R>(a, b);
    while (base + int64_t(s.tiles) * heads * units_of(s) <= u) {  // the next request that has rows
      base += int64_t(s.tiles) * heads * units_of(s);
      s = span_of<R>(a, ++b);
    }
    // ---- segment (request b, row tile, kv head): atoms [ua, ub) of it are this warp's
    const int units = units_of(s);
    const int seg = int(quotient(u - base, units));
    const int64_t seg0 = base + int64_t(seg) * units;
    const int tile = seg / heads, head = seg - tile * heads;
    const int rows = min(R, s.q_len * a.group - tile * R);
    // Row y of the tile is head g of token: one division here, then of numbers
    // below group + R by a multiplication (exact: their product stays below 2^32).
    const int token0 = tile * R / a.group, rest0 = tile * R - token0 * a.group;
    auto token_of = [&](int y, int* g) {
      const uint32_t x = uint32_t(rest0 + y), q = a.group == 1 ? x : __umulhi(x, a.group_magic);
      *g = int(x) - int(q) * a.group;
      return token0 + int(q);
    };
    int ua, ub;
    if constexpr (WALK) {
      ua = int(u - seg0);
      ub = int(min(u1 - seg0, int64_t(units)));
    } else {
      const int c0 = int(u - seg0) * chunk, n = min(chunk, s.units - c0);
      ua = c0 + n * warp / kWarps;
      ub = c0 + n * (warp + 1) / kWarps;
    }

    // Keys in sight of columns 2j and 2j + 1 of each 8-row tile.
    int lo[NT][2], hi[NT][2];
    int lo_all = 0x7fffffff, hi_all = 0;    // union and ...
    int lo_full = 0, hi_full = 0x7fffffff;  // ... intersection over the tile's rows
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = nt * 8 + 2 * j + i;
        lo[nt][i] = 0;
        hi[nt][i] = 0;
        if (row < rows) {
          int g;
          const int pos = s.kv_len - s.q_len + token_of(row, &g);
          hi[nt][i] = a.causal ? min(s.kv_len, max(0, pos + 1)) : s.kv_len;
          lo[nt][i] = a.window > 0 ? max(0, pos + 1 - a.window) : 0;
          lo_all = min(lo_all, lo[nt][i]);
          hi_all = max(hi_all, hi[nt][i]);
          lo_full = max(lo_full, lo[nt][i]);
          hi_full = min(hi_full, hi[nt][i]);
        }
      }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      lo_all = min(lo_all, __shfl_xor_sync(kFull, lo_all, o));
      hi_all = max(hi_all, __shfl_xor_sync(kFull, hi_all, o));
      lo_full = max(lo_full, __shfl_xor_sync(kFull, lo_full, o));
      hi_full = min(hi_full, __shfl_xor_sync(kFull, hi_full, o));
    }

    // ---- the atoms of the share that some row sees; the first ones are on their way from here
    const int t0 = max(s.first + 16 * ua, lo_all & ~15), t1 = min(s.first + 16 * ub, hi_all);
    const int n_atoms = t0 < t1 ? (t1 - t0 + 15) >> 4 : 0;
    const int32_t* table = a.table + int64_t(b) * a.ld_table;
    const uint8_t* const base_head = a.cache.base + head * head_bytes;
    const int page_atoms = 1 << (a.cache.log_page - 4);
    // Atoms are issued in order, a pair to a slot: within a page the source only
    // moves on and a pair is one copy.
    int page_i = t0 >> a.cache.log_page;
    const int page_end = n_atoms > 0 ? (t1 - 1) >> a.cache.log_page : -1;
    auto page_at = [&](int i) { return i <= page_end ? __ldg(table + i) : 0; };
    int page = page_at(page_i), next_page = page_at(page_i + 1);
    int skip = (t0 >> 4) & (page_atoms - 1);  // atoms of the first page before the share
    int left = page_atoms - skip, to_issue = n_atoms;
    bool gone = uint32_t(page) >= uint32_t(a.cache.pages);
    const uint8_t* src = base_head + int64_t(page) * a.cache.page_stride + skip * kAtom;
    uint32_t missing = 0;  // bit i: the atom issued i + 1 calls ago has no page
    auto turn_page = [&]() {
      page = next_page;
      ++page_i;
      next_page = page_at(page_i + 1);
      left = page_atoms;
      gone = uint32_t(page) >= uint32_t(a.cache.pages);
      src = base_head + int64_t(page) * a.cache.page_stride;
    };
    auto issue_pair = [&]() {
      missing <<= 2;
      if (to_issue <= 0) return;
      const uint32_t bar = bars + 8 * wr_slot, dst = ring + wr_slot * (2 * kAtom);
      if (left >= 2 && to_issue >= 2 && !gone) {
        if (lane == 0) {
          mbar_expect(bar, 2 * kAtom);
          bulk_copy(dst, src, 2 * kAtom, bar);
        }
        src += 2 * kAtom;
        left -= 2;
      } else {
        uint32_t bytes = 0;
        const uint8_t* from[2] = {nullptr, nullptr};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h >= to_issue) break;
          if (left == 0) turn_page();
          if (!gone) from[h] = src, bytes += kAtom;
          else missing |= 2u >> h;
          src += kAtom;
          --left;
        }
        if (lane == 0) {
          mbar_expect(bar, bytes);
          if (from[0]) bulk_copy(dst, from[0], kAtom, bar);
          if (from[1]) bulk_copy(dst + kAtom, from[1], kAtom, bar);
        }
      }
      if (left == 0) turn_page();
      to_issue -= 2;
      if (++wr_slot == kStages) wr_slot = 0;
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) issue_pair();

    // Query fragments: lane (n = r, j) holds row n's dimensions [j D/4, (j+1) D/4) of each 8-row tile.
    uint32_t qf[NT][D / 16][2];
    float c_row[NT];  // this lane's row: score = c_row * accumulator
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = nt * 8 + r;
      uint4 raw[D / 32];
      float amax = 0.0f;
      if (row < rows) {
        int g;
        const int token = token_of(row, &g);
        const uint16_t* qp = a.q + int64_t(s.q0 + token) * a.ld_qt + int64_t(head * a.group + g) * a.ld_qh + j * (D / 4);
        if ((reinterpret_cast<uintptr_t>(qp) & 15) == 0) {
#pragma unroll
          for (int i = 0; i < D / 32; ++i) raw[i] = __ldg(reinterpret_cast<const uint4*>(qp) + i);
        } else {
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = uint32_t(qp[8 * i + 2 * e]) | (uint32_t(qp[8 * i + 2 * e + 1]) << 16);
            raw[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) raw[i] = make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        float v[8];
        unpack_bf16x8(raw[i], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
      }
      amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
      const int e = int(__float_as_uint(amax) >> 23) - 127;
      const int k = (amax == 0.0f || e > 127) ? 0 : min(14 - e, kMostPower);
      const float factor = a.scale_log2 * gk;
      const float up = copysignf(__uint_as_float(uint32_t(k + 127) << 23), factor);
      // At least the smallest normal number: 0 would make NaN of a masked key's -inf.
      c_row[nt] = fmaxf(fabsf(factor) * __uint_as_float(uint32_t(127 - k) << 23), 1.17549435e-38f);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        float v[8];
        unpack_bf16x8(raw[i], v);
#pragma unroll
        for (int e2 = 0; e2 < 4; ++e2) qf[nt][2 * i + (e2 >> 1)][e2 & 1] = pack_f16x2(v[2 * e2] * up, v[2 * e2 + 1] * up);
      }
    }
    float cs[NT][2], m[NT][2], l[NT][2];  // columns 2j and 2j + 1: score factor, maximum, sum of this lane's weights
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        cs[nt][i] = __shfl_sync(kFull, c_row[nt], 4 * (2 * j + i));
        m[nt][i] = kLowest;
        l[nt][i] = 0.0f;
      }
    float o[D / 16][NT][4];
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[mt][nt][i] = 0.0f;

    // ---- S^T = K' q^T of N atoms, their products taking turns
    auto scores = [&](auto n_tag, const uint8_t* atom, float (*sc)[NT][4]) {
      constexpr int N = decltype(n_tag)::value;
      uint32_t kw[N][2][kN][2];  // codes of rows r and r + 8
      uint32_t ks2[N][2 * kN];   // each scale in both halves of an f16 pair
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const uint8_t* at = atom + n * kAtom;
        uint32_t ksw[(2 * kN + 3) / 4];  // the lane's 2 kN key scales
        if constexpr (kN == 1) {
          ksw[0] = *reinterpret_cast<const uint16_t*>(at + KvAtom<D>::kKScales + lane * 2);
        } else {
#pragma unroll
          for (int x = 0; x < kN / 2; ++x)
            ksw[x] = *reinterpret_cast<const uint32_t*>(at + KvAtom<D>::kKScales + lane * 2 * kN + 4 * x);
        }
#pragma unroll
        for (int pl = 0; pl < kN; ++pl) {
          const uint4 w = *reinterpret_cast<const uint4*>(at + pl * 512 + lane * 16);
          kw[n][(2 * pl) / kN][(2 * pl) % kN][0] = w.x;
          kw[n][(2 * pl) / kN][(2 * pl) % kN][1] = w.y;
          kw[n][(2 * pl + 1) / kN][(2 * pl + 1) % kN][0] = w.z;
          kw[n][(2 * pl + 1) / kN][(2 * pl + 1) % kN][1] = w.w;
        }
#pragma unroll
        for (int x = 0; x < kN; ++x) {
          const uint32_t h = e4m3x2_to_f16x2(ksw[x / 2] >> (16 * (x % 2)));
          ks2[n][2 * x] = __byte_perm(h, h, 0x1010);
          ks2[n][2 * x + 1] = __byte_perm(h, h, 0x3232);
        }
      }
#pragma unroll
      for (int c = 0; c < kN; ++c)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t ha[N][4], hb[N][4];
#pragma unroll
          for (int n = 0; n < N; ++n) {
            e2m1x8_to_f16x2(kw[n][0][c][x], ha[n]);
            e2m1x8_to_f16x2(kw[n][1][c][x], hb[n]);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              ha[n][y] = mul_f16x2(ha[n][y], ks2[n][c]);
              hb[n][y] = mul_f16x2(hb[n][y], ks2[n][kN + c]);
            }
          }
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma(sc[n][nt], ha[n][2 * y], hb[n][2 * y], ha[n][2 * y + 1], hb[n][2 * y + 1],
                    qf[nt][4 * c + 2 * x + y][0], qf[nt][4 * c + 2 * x + y][1], c + x + y == 0);
        }
    };
    // ---- softmax over N atoms' tokens t + r (x = 0, 1) and t + r + 8 (x = 2, 3): scores to weights
    auto weights = [&](auto n_tag, float (*sc)[NT][4], uint32_t (*pf)[NT][2]) {
      constexpr int N = decltype(n_tag)::value;
      bool raise = false;
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 4; ++x) raise |= __fmaf_rn(sc[n][nt][x], cs[nt][x & 1], -m[nt][x & 1]) > kHeadroom + kRaise;
      if (__any_sync(kFull, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float top = fmaxf(sc[0][nt][y], sc[0][nt][y + 2]);
            if (N == 2) top = fmaxf(top, fmaxf(sc[N - 1][nt][y], sc[N - 1][nt][y + 2]));
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, w));
            if (__fmaf_rn(top, cs[nt][y], -m[nt][y]) > kHeadroom + kRaise) {  // a row's results do not depend on its neighbours'
              top = __fmaf_rn(top, cs[nt][y], -kHeadroom);
              const float f = ex2(m[nt][y] - top);
              m[nt][y] = top;
              l[nt][y] *= f;
#pragma unroll
              for (int mt = 0; mt < D / 16; ++mt) o[mt][nt][y] *= f, o[mt][nt][y + 2] *= f;
            }
          }
      }
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            p[x] = ex2(__fmaf_rn(sc[n][nt][x], cs[nt][x & 1], -m[nt][x & 1]));
            l[nt][x & 1] += p[x];
          }
          pf[n][nt][0] = transpose8x8(pack_f16x2(p[0], p[1]));
          pf[n][nt][1] = transpose8x8(pack_f16x2(p[2], p[3]));
        }
    };
    // ---- one atom's O^T += V'^T P^T: tokens 2j, 2j+1 (pair 0) and 2j+8, 2j+9 (pair 1), dimensions
    // [r D/8, (r+1) D/8); keys: tokens of the atom that exist
    auto values = [&](const uint8_t* atom, const uint32_t (&pf)[NT][2], int keys) {
      uint32_t vs2[2][kW];  // scale pairs (token, next token) of each block
      {
        uint32_t w[kW];
#pragma unroll
        for (int x = 0; x < kW; ++x)
          w[x] = *reinterpret_cast<const uint32_t*>(atom + KvAtom<D>::kVScales +
                                                    ((D == 64 ? r >> 1 : r) * 4 + j) * (4 * kW) + 4 * x);
        if (keys < 16) {
          // Bytes behind the last key are whatever the page held: their scales
          // become zero, so that 0 * NaN cannot reach the sum.
#pragma unroll
          for (int x = 0; x < 4 * kW; ++x) {
            const int i4 = x / kW;
            if (8 * (i4 >> 1) + 2 * j + (i4 & 1) >= keys) w[x >> 2] &= ~(0xFFu << (8 * (x & 3)));
          }
        }
        if constexpr (kW == 1) {
          vs2[0][0] = e4m3x2_to_f16x2(w[0]);
          vs2[1][0] = e4m3x2_to_f16x2(w[0] >> 16);
        } else {  // bytes: token, block
#pragma unroll
          for (int pr = 0; pr < 2; ++pr) {
            vs2[pr][0] = e4m3x2_to_f16x2(__byte_perm(w[pr], 0u, 0x4420));
            vs2[pr][1] = e4m3x2_to_f16x2(__byte_perm(w[pr], 0u, 0x4431));
          }
        }
      }
      constexpr int kVW = D / 64;  // 32-bit words of a lane's dimensions per token
      uint32_t vw[4][kVW];
#pragma unroll
      for (int pl = 0; pl < kN; ++pl) {
        const uint4 w = *reinterpret_cast<const uint4*>(atom + KvAtom<D>::kVCodes + pl * 512 + lane * 16);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int x = 0; x < 4; ++x) vw[(4 * pl + x) / kVW][(4 * pl + x) % kVW] = ww[x];
      }
#pragma unroll
      for (int x = 0; x < kVW; ++x) {
        uint32_t ev[2][4], od[2][4];  // even and odd dimensions of token pairs
#pragma unroll
        for (int pr = 0; pr < 2; ++pr) {
          const uint32_t w0 = vw[2 * pr][x], w1 = vw[2 * pr + 1][x];
          e2m1x8_to_f16x2((w0 & 0x0F0F0F0Fu) | ((w1 << 4) & 0xF0F0F0F0u), ev[pr]);
          e2m1x8_to_f16x2(((w0 >> 4) & 0x0F0F0F0Fu) | (w1 & 0xF0F0F0F0u), od[pr]);
          const uint32_t sf = vs2[pr][kW == 1 ? 0 : x / 2];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            ev[pr][y] = mul_f16x2(ev[pr][y], sf);
            od[pr][y] = mul_f16x2(od[pr][y], sf);
          }
        }
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma(o[4 * x + y][nt], ev[0][y], od[0][y], ev[1][y], od[1][y], pf[nt][0], pf[nt][1]);
      }
    };

    // Atoms [i_lo, i_hi) are seen whole by every row.
    const int i_lo = lo_full > t0 ? (lo_full - t0 + 15) >> 4 : 0;
    const int i_hi = hi_full > t0 ? min(n_atoms, (hi_full - t0) >> 4) : 0;
    bool lost = false;
#pragma unroll 1
    for (int i = 0; i < n_atoms; i += 2) {
      __syncwarp();  // all lanes have read the pair before
      issue_pair();
      const uint8_t* atom = ring_p + rd_slot * (2 * kAtom);
      lost = __any_sync(kFull, !mbar_wait(bars + 8 * rd_slot, rd_parity));
      if (lost) break;
      if (++rd_slot == kStages) rd_slot = 0, rd_parity ^= 1;
      const uint32_t absent = (missing >> (2 * kStages - 2)) & 3u;  // bit 1: the first atom
      if (i >= i_lo && i + 2 <= i_hi && absent == 0) {
        // Two atoms at a time: two independent chains of products, one vote.
        float sc[2][NT][4];
        uint32_t pf[2][NT][2];
        scores(IntTag<2>{}, atom, sc);
        weights(IntTag<2>{}, sc, pf);
        values(atom, pf[0], 16);
        values(atom + kAtom, pf[1], 16);
      } else {
#pragma unroll 1
        for (int h = 0; h < 2 && i + h < n_atoms; ++h) {
          const int t = t0 + 16 * (i + h);
          if ((absent >> (1 - h)) & 1u) {
            if (lane == 0) atomicOr(a.err, kErrSlot);
            continue;
          }
          float sc[1][NT][4];
          uint32_t pf[1][NT][2];
          scores(IntTag<1>{}, atom + h * kAtom, sc);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int key = t + r + (x >> 1) * 8;
              if (key < lo[nt][x & 1] || key >= hi[nt][x & 1]) sc[0][nt][x] = -INFINITY;
            }
          weights(IntTag<1>{}, sc, pf);
          values(atom + h * kAtom, pf[0], s.kv_len - t);
        }
      }
    }
    __syncwarp();
    if (lost) {
      // Never in a sound run: the results of this call are not valid.  Waits, as long, for the copies behind the one
      // that did not come, and takes no further part.
      if (lane == 0) atomicOr(a.err, kErrWait);
      if (++rd_slot == kStages) rd_slot = 0, rd_parity ^= 1;
      while (rd_slot != wr_slot) {
        mbar_wait(bars + 8 * rd_slot, rd_parity);
        if (++rd_slot == kStages) rd_slot = 0, rd_parity ^= 1;
      }
      if constexpr (WALK) return;
    }

    // ---- the segment's end: sums over the lanes of a column
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[nt][y] += __shfl_xor_sync(kFull, l[nt][y], w);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int y = 0; y < 2; ++y)
        if (l[nt][y] > 0.0f) l[nt][y] += nan_of(a.scale_log2 * gk);
    if constexpr (WALK) {
      if (seg0 >= u0 && seg0 + units <= u1) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int row = nt * 8 + 2 * j + y;
            if (row >= rows) continue;
            int g;
            const int64_t at = s.q0 + token_of(row, &g);
            const int h = head * a.group + g;
            const float f = out_factor(l[nt][y], gv);
            uint16_t* op = a.out + at * a.ld_ot + h * a.ld_oh + r * (D / 8);
            if ((reinterpret_cast<uintptr_t>(op) & 15) == 0) {
#pragma unroll
              for (int mt = 0; mt < D / 16; mt += 4) {
                uint4 w;
                w.x = pack_bf16x2(o[mt][nt][y] * f, o[mt][nt][y + 2] * f);
                w.y = pack_bf16x2(o[mt + 1][nt][y] * f, o[mt + 1][nt][y + 2] * f);
                w.z = pack_bf16x2(o[mt + 2][nt][y] * f, o[mt + 2][nt][y + 2] * f);
                w.w = pack_bf16x2(o[mt + 3][nt][y] * f, o[mt + 3][nt][y + 2] * f);
                *reinterpret_cast<uint4*>(op + 2 * mt) = w;
              }
            } else {
#pragma unroll
              for (int mt = 0; mt < D / 16; ++mt) store_pair(op + 2 * mt, o[mt][nt][y] * f, o[mt][nt][y + 2] * f);
            }
            if (a.lse != nullptr && r == 0) a.lse[at * a.ld_lse + h] = lse_of(m[nt][y], l[nt][y]);
          }
      } else {
        // A part: of a segment that began earlier, or of one that begins here.
        const bool begins = seg0 >= u0;
        float* slot = slot_of<D, R>(a, 2 * int64_t(part) + (begins ? 1 : 0));
        if (begins && lane == 0)
          cuts_of(a)[atomicAdd(counter_of(a, kCuts), 1u)] = {part, owner_of(seg0 + units - 1), head, s.q0, tile * R, rows, 0, 0};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int row = nt * 8 + 2 * j + y;
            if (row >= rows) continue;
            float* rp = slot + row * D + r * (D / 8);
#pragma unroll
            for (int mt = 0; mt < D / 16; mt += 2)
              *reinterpret_cast<float4*>(rp + 2 * mt) =
                  make_float4(o[mt][nt][y], o[mt][nt][y + 2], o[mt + 1][nt][y], o[mt + 1][nt][y + 2]);
            if (r == 0) *reinterpret_cast<float2*>(slot + R * D + 2 * row) = make_float2(m[nt][y], l[nt][y]);
          }
      }
      u = seg0 + ub;
    } else {
      // The warps' shares of the chunk, through shared memory (over the rings).
      float* res = reinterpret_cast<float*>(smem);  // [kWarps][R][kPitch]
      float* stat = res + kWarps * R * kPitch;      // [kWarps][R][2]
      __syncthreads();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int row = nt * 8 + 2 * j + y;
          float* rp = res + (warp * R + row) * kPitch + r * (D / 8);
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt)
            *reinterpret_cast<float2*>(rp + 2 * mt) = make_float2(o[mt][nt][y], o[mt][nt][y + 2]);
          if (r == 0) *reinterpret_cast<float2*>(stat + (warp * R + row) * 2) = make_float2(m[nt][y], l[nt][y]);
        }
      __syncthreads();
      float* slot = slot_of<D, R>(a, part);
      for (int i = tid; i < rows * (D / 2); i += kThreads) {
        const int row = i / (D / 2), d = 2 * (i % (D / 2));
        float top = kLowest;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stat[(w * R + row) * 2]);
        float x0 = 0.0f, x1 = 0.0f, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = ex2(stat[(w * R + row) * 2] - top);
          const float2 v = *reinterpret_cast<const float2*>(res + (w * R + row) * kPitch + d);
          x0 += f * v.x;
          x1 += f * v.y;
          sum += f * stat[(w * R + row) * 2 + 1];
        }
        if (units == 1) {
          int g;
          const int64_t at = s.q0 + token_of(row, &g);
          const int h = head * a.group + g;
          const float f = out_factor(sum, gv);
          store_pair(a.out + at * a.ld_ot + h * a.ld_oh + d, x0 * f, x1 * f);
          if (a.lse != nullptr && d == 0) a.lse[at * a.ld_lse + h] = lse_of(top, sum);
        } else {
          *reinterpret_cast<float2*>(slot + row * D + d) = make_float2(x0, x1);
          if (d == 0) *reinterpret_cast<float2*>(slot + R * D + 2 * row) = make_float2(top, sum);
        }
      }
      if (units > 1) {
        __threadfence();
        __syncthreads();
        if (tid == 0) s_last = atomicAdd(counters_of(a) + seg0, 1u) == uint32_t(units - 1) ? 1 : 0;
        __syncthreads();
        if (s_last) {
          __threadfence();
          const Cut cut = {0, 0, head, s.q0, tile * R, rows, 0, 0};
          reinterpret_cast<Join<D, R, kThreads>*>(smem)->run(
              a, units, [&](int p) { return slot_of<D, R>(a, seg0 + p); }, cut, gv);
          if (tid == 0) counters_of(a)[seg0] = 0;
        }
      }
      return;
    }
  }
}

// Joins the parts of the segments that the walk has cut, a CTA each in turn.
template <int D, int R>
__global__ void __launch_bounds__(kAttnJoinThreads) rows_join_kernel(const AttnArgs a) {
  __shared__ Join<D, R, kAttnJoinThreads> join;
  griddep_wait();
  griddep_launch_dependents();
  const int n = int(__ldcg(counter_of(a, kCuts)));
  const float gv = __ldg(a.v_scale);
  for (int i = int(blockIdx.x); i < n; i += int(gridDim.x)) {
    const int4 c0 = __ldcg(reinterpret_cast<const int4*>(cuts_of(a) + i));
    const int4 c1 = __ldcg(reinterpret_cast<const int4*>(cuts_of(a) + i) + 1);
    const Cut cut = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, 0, 0};
    join.run(a, cut.last - cut.first + 1,
             [&](int p) { return slot_of<D, R>(a, 2 * int64_t(cut.first + p) + (p == 0 ? 1 : 0)); }, cut, gv);
  }
  // The last CTA leaves the counters at zero (its own wraps around).
  __syncthreads();
  if (threadIdx.x == 0 && atomicInc(counter_of(a, kDone), gridDim.x - 1) == gridDim.x - 1) {
    *counter_of(a, kClaims) = 0;
    *counter_of(a, kCuts) = 0;
  }
}

}  // namespace

AttnRows attn_rows(int d, int n_tiles, bool walk) {
#define NQ_WALK(D, NT)                               \
  if (walk && d == D && n_tiles == NT)               \
    return {reinterpret_cast<const void*>(&rows_kernel<D, NT, true>), \
            reinterpret_cast<const void*>(&rows_join_kernel<D, 8 * NT>), ring_bytes(D, kWalkWarps), kWalkWarps * 32};
#define NQ_CHUNK(D, NT)                                                                            \
  if (!walk && d == D && n_tiles == NT) {                                                          \
    const size_t merge = merge_bytes(D, 8 * NT), join = sizeof(Join<D, 8 * NT, kChunkWarps * 32>); \
    const size_t ring = ring_bytes(D, kChunkWarps), need = merge > join ? merge : join;            \
    return {reinterpret_cast<const void*>(&rows_kernel<D, NT, false>), nullptr, need > ring ? need : ring, kChunkWarps * 32}; \
  }
  NQ_WALK(64, 1) NQ_WALK(64, 2) NQ_WALK(64, 4) NQ_WALK(128, 1) NQ_WALK(128, 2) NQ_WALK(256, 1)
  NQ_CHUNK(64, 1) NQ_CHUNK(64, 2) NQ_CHUNK(64, 4) NQ_CHUNK(128, 1) NQ_CHUNK(128, 2) NQ_CHUNK(256, 1) NQ_CHUNK(256, 2)
#undef NQ_WALK
#undef NQ_CHUNK
  return {nullptr, nullptr, 0, 0};
}

}  // namespace nq

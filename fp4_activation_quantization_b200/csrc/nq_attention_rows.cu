// nq_attention_rows.cu — attention over the 4-bit cache for few rows per request
// (single tokens, draft verification): each warp streams atoms of 16 tokens
// through matrix products whose fragments are the cache's own byte order.
//
//   s_j = c <q, k'_j>,  m = max s_j,  p_j = 2^(s_j - m),  l = sum p_j,
//   o = g_v / l * sum p_j v'_j,  lse = ln 2 (m + log2 l),
// with k', v' = e2m1 * e4m3 and c = scale * log2(e) * g_k.
//
// Numerics.  k' and v' have at most six significant bits and lie in [2^-10,
// 2688], so they are exact in f16.  A query row is scaled by a power of two to
// a largest magnitude in [2^14, 2^15): its bf16 values are then exact in f16
// down to 2^-28 of the row's largest.  Products accumulate in float32.  p is
// rounded to f16 (half a step is 2^-11 of it, an eighth of the bf16 output's);
// l sums the float32 values.  The running maximum is only raised when a score
// exceeds it by more than 2^8: p stays below 2^9, far inside f16's range, and
// the accumulators are rescaled once or twice per row instead of at every atom.
//
// Work.  S^T = K' q^T and O^T = V'^T P^T put the 16 tokens (or dimensions) on
// the 16-row side of the product and up to 8 rows of a (request, kv head) on
// its 8-column side.  Bound by HBM in the limit: an atom of D = 128 is 2304
// bytes and costs a warp about 250 instructions.
//
// Split.  The tokens of all (request, kv head) pairs form one axis of units of
// 64 tokens; every CTA takes an equal share of it, whatever the lengths.  A
// segment cut by a CTA's boundary leaves its unnormalised result in the
// workspace, and the CTA that arrives last joins them in the order of the
// tokens, so results do not depend on timing.  No CTA waits for another.
#include "nq_kv_layout.cuh"

namespace nq {

namespace {

constexpr int kWarps = kAttnRowsThreads / 32;
constexpr int kUnit = 16 * kWarps;  // tokens of a unit: one atom per warp
constexpr float kRaise = 8.0f;      // log2 by which a score may exceed the running maximum

constexpr int stages_of(int d) { return d == 256 ? 3 : 4; }
constexpr size_t ring_bytes(int d) { return size_t(kWarps) * stages_of(d) * 18 * d; }
constexpr int row_pitch(int d) { return d + 4; }  // floats between rows of a warp's result in shared memory
constexpr size_t merge_bytes(int d, int rows) { return size_t(kWarps) * rows * (row_pitch(d) + 2) * 4; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One request's share of the axis.
struct Span {
  int q0, q_len, kv_len;  // first query row, rows, keys
  int first;              // first key any row sees, rounded down to an atom
  int tiles, units;       // row tiles; units of keys per tile and kv head
};
template <int R>
__device__ __forceinline__ Span span_of(const AttnArgs& a, int b) {
  Span s;
  const int64_t room = int64_t(a.width) << a.cache.log_page;
  const int c0 = min(max(a.cu_q[b], 0), a.T), c1 = min(max(a.cu_q[b + 1], c0), a.T);
  s.q0 = c0;
  s.q_len = c1 - c0;
  s.kv_len = int(min(int64_t(max(a.kv_lens[b], 0)), room));
  s.first = 0;
  if (a.window > 0) s.first = int(max(int64_t(0), int64_t(s.kv_len) - s.q_len + 1 - a.window)) & ~15;
  s.tiles = int((int64_t(s.q_len) * a.group + R - 1) / R);
  s.units = max(1, (s.kv_len - s.first + kUnit - 1) / kUnit);
  return s;
}

template <int D, int NT>
__global__ void __launch_bounds__(kAttnRowsThreads, D == 256 ? 2 : (NT == 1 ? 4 : 3)) rows_kernel(const AttnArgs a) {
  constexpr int R = 8 * NT;  // rows of a tile: (token, head of the group), token-major
  constexpr int kStages = stages_of(D);
  constexpr int kN = KvAtom<D>::kN, kW = KvAtom<D>::kW;
  constexpr int kAtom = KvAtom<D>::kBytes;
  constexpr int kPitch = row_pitch(D);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t s_scan[2][kWarps];
  __shared__ int64_t s_found[3];
  __shared__ int s_last;

  const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, j = lane & 3;
  const int heads = a.cache.heads;

  griddep_wait();
  griddep_launch_dependents();

  // ---- the axis: units and segments of all requests, and the request of this CTA's first unit
  const int per = (a.B + kAttnRowsThreads - 1) / kAttnRowsThreads;
  const int b_lo = min(a.B, tid * per), b_hi = min(a.B, b_lo + per);
  int64_t mine = 0, segs = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const Span s = span_of<R>(a, b);
    mine += int64_t(s.tiles) * heads * s.units;
    segs += int64_t(s.tiles) * heads;
  }
  int64_t incl = mine, segs_all = segs;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += up;
    segs_all += __shfl_xor_sync(kFull, segs_all, o);
  }
  if (lane == 31) s_scan[0][warp] = incl, s_scan[1][warp] = segs_all;
  __syncthreads();
  int64_t total = 0, before = incl - mine;
  segs_all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_scan[0][w];
    total += s_scan[0][w];
    segs_all += s_scan[1][w];
  }
  if (total == 0) return;
  // CTAs that take part: at most one per unit, and at most max_splits per segment on average.
  const int64_t parts = min(int64_t(gridDim.x), min(total, segs_all * a.max_splits));
  if (int64_t(blockIdx.x) >= parts) return;
  const int64_t u0 = total * blockIdx.x / parts, u1 = total * (blockIdx.x + 1) / parts;
  auto part_of = [&](int64_t u) { return int(((u + 1) * parts - 1) / total); };  // the CTA that owns unit u
  if (mine > 0 && u0 >= before && u0 < before + mine) {
    int64_t at = before;
    int b = b_lo;
    for (; b < b_hi; ++b) {
      const Span s = span_of<R>(a, b);
      const int64_t n = int64_t(s.tiles) * heads * s.units;
      if (u0 < at + n) break;
      at += n;
    }
    s_found[0] = b;
    s_found[1] = at;
  }
  __syncthreads();
  int b = int(s_found[0]);
  int64_t base = s_found[1];  // first unit of request b

  const uint32_t ring = uint32_t(__cvta_generic_to_shared(smem)) + warp * (kStages * kAtom);
  const uint8_t* ring_p = smem + warp * (kStages * kAtom);
  const float gk = __ldg(a.k_scale), gv = __ldg(a.v_scale);
  const int64_t head_bytes = int64_t(kAtom) << (a.cache.log_page - 4);

  int64_t u = u0;
  while (u < u1) {
    Span s = span_of<R>(a, b);
    while (base + int64_t(s.tiles) * heads * s.units <= u) {  // the next request that has rows
      base += int64_t(s.tiles) * heads * s.units;
      s = span_of<R>(a, ++b);
    }
    // ---- segment (request b, row tile, kv head): units [ua, ub) of it are ours
    const int64_t seg = (u - base) / s.units;
    const int64_t seg0 = base + seg * s.units;
    const int head = int(seg % heads), tile = int(seg / heads);
    const int ua = int(u - seg0), ub = int(min(u1 - seg0, int64_t(s.units)));
    const int rows = min(R, s.q_len * a.group - tile * R);

    // Query fragments: lane (n = r, j) holds row n's dimensions [j D/4, (j+1) D/4) of each 8-row tile.
    uint32_t qf[NT][D / 16][2];
    float c_row[NT];  // this lane's row: score = c_row * accumulator
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = nt * 8 + r;
      uint4 raw[D / 32];
      float amax = 0.0f;
      if (row < rows) {
        const int x = tile * R + row, token = x / a.group, g = x - token * a.group;
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
      const int k = (amax == 0.0f || e > 127) ? 0 : min(14 - e, 100);
      const float up = __uint_as_float(uint32_t(k + 127) << 23), down = __uint_as_float(uint32_t(127 - k) << 23);
      c_row[nt] = a.scale_log2 * gk * down;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        float v[8];
        unpack_bf16x8(raw[i], v);
#pragma unroll
        for (int e2 = 0; e2 < 4; ++e2) qf[nt][2 * i + (e2 >> 1)][e2 & 1] = pack_f16x2(v[2 * e2] * up, v[2 * e2 + 1] * up);
      }
    }
    // Columns 2j and 2j + 1 of each tile: score factor, keys in sight.
    float cs[NT][2], m[NT][2], l[NT][2];
    int lo[NT][2], hi[NT][2];
    int lo_all = 0x7fffffff, hi_all = 0;    // union and ...
    int lo_full = 0, hi_full = 0x7fffffff;  // ... intersection over the tile's rows
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = nt * 8 + 2 * j + i;
        cs[nt][i] = __shfl_sync(kFull, c_row[nt], 4 * (2 * j + i));
        m[nt][i] = -INFINITY;
        l[nt][i] = 0.0f;
        lo[nt][i] = 0;
        hi[nt][i] = 0;
        if (row < rows) {
          const int64_t pos = int64_t(s.kv_len) - s.q_len + (tile * R + row) / a.group;
          hi[nt][i] = a.causal ? int(min(int64_t(s.kv_len), max(int64_t(0), pos + 1))) : s.kv_len;
          lo[nt][i] = a.window > 0 ? int(max(int64_t(0), pos + 1 - a.window)) : 0;
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
    float o[D / 16][NT][4];
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[mt][nt][i] = 0.0f;

    // ---- this warp's atoms: first + 16 * (kWarps * unit + warp), those in sight of some row
    int t0 = s.first + kUnit * ua + 16 * warp;
    int t1 = s.first + kUnit * ub;
    {
      const int lo_atom = lo_all & ~15;
      if (t0 < lo_atom) t0 += (lo_atom - t0 + kUnit - 1) / kUnit * kUnit;
      t1 = min(t1, hi_all);
    }
    const int n_atoms = t0 < t1 ? (t1 - t0 + kUnit - 1) / kUnit : 0;
    const int32_t* table = a.table + int64_t(b) * a.ld_table;
    uint32_t missing = 0;  // bit i: the atom issued i + 1 calls ago has no page
    auto issue = [&](int i) {
      bool gone = false;
      if (i < n_atoms) {
        const int t = t0 + i * kUnit;
        const int page = __ldg(table + (t >> a.cache.log_page));
        gone = page < 0 || page >= a.cache.pages;
        if (!gone) {
          const uint8_t* src = a.cache.base + page * a.cache.page_stride + head * head_bytes +
                               ((t & ((1 << a.cache.log_page) - 1)) >> 4) * kAtom;
          const uint32_t dst = ring + (i % kStages) * kAtom;
#pragma unroll
          for (int x = 0; x < (kAtom / 16 + 31) / 32; ++x) {
            const int c = x * 32 + lane;
            if (kAtom / 16 % 32 == 0 || c < kAtom / 16) cp_async16(dst + 16 * c, src + 16 * c);
          }
        }
      }
      missing = (missing << 1) | (gone ? 1u : 0u);
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i);

    for (int i = 0; i < n_atoms; ++i) {
      cp_async_wait<kStages - 2>();
      __syncwarp();  // all lanes' copies of atom i have landed, and all have read atom i - 1
      const bool gone = (missing >> (kStages - 2)) & 1u;
      issue(i + kStages - 1);
      if (gone) {
        if (lane == 0) atomicOr(a.err, kErrSlot);
        continue;
      }
      const uint8_t* atom = ring_p + (i % kStages) * kAtom;
      const int t = t0 + i * kUnit;

      // ---- S^T = K' q^T
      float sc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 4; ++x) sc[nt][x] = 0.0f;
      uint32_t ksw[(2 * kN + 3) / 4];  // the lane's 2 kN key scales
      if constexpr (kN == 1) ksw[0] = *reinterpret_cast<const uint16_t*>(atom + KvAtom<D>::kKScales + lane * 2);
      else
#pragma unroll
        for (int x = 0; x < kN / 2; ++x)
          ksw[x] = *reinterpret_cast<const uint32_t*>(atom + KvAtom<D>::kKScales + lane * 2 * kN + 4 * x);
      uint32_t kw[2][kN][2];  // codes of rows r and r + 8
#pragma unroll
      for (int pl = 0; pl < kN; ++pl) {
        const uint4 w = *reinterpret_cast<const uint4*>(atom + pl * 512 + lane * 16);
        kw[(2 * pl) / kN][(2 * pl) % kN][0] = w.x;
        kw[(2 * pl) / kN][(2 * pl) % kN][1] = w.y;
        kw[(2 * pl + 1) / kN][(2 * pl + 1) % kN][0] = w.z;
        kw[(2 * pl + 1) / kN][(2 * pl + 1) % kN][1] = w.w;
      }
      uint32_t ks2[2 * kN];  // each scale in both halves of an f16 pair
#pragma unroll
      for (int x = 0; x < kN; ++x) {
        const uint32_t h = e4m3x2_to_f16x2(ksw[x / 2] >> (16 * (x % 2)));
        ks2[2 * x] = __byte_perm(h, h, 0x1010);
        ks2[2 * x + 1] = __byte_perm(h, h, 0x3232);
      }
#pragma unroll
      for (int c = 0; c < kN; ++c)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t ha[4], hb[4];
          e2m1x8_to_f16x2(kw[0][c][x], ha);
          e2m1x8_to_f16x2(kw[1][c][x], hb);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            ha[y] = mul_f16x2(ha[y], ks2[c]);
            hb[y] = mul_f16x2(hb[y], ks2[kN + c]);
          }
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma(sc[nt], ha[2 * y], hb[2 * y], ha[2 * y + 1], hb[2 * y + 1], qf[nt][4 * c + 2 * x + y][0],
                  qf[nt][4 * c + 2 * x + y][1]);
        }

      // ---- softmax over the atom's tokens t + r (x = 0, 1) and t + r + 8 (x = 2, 3)
      const bool masked = t < lo_full || t + 16 > hi_full;
      bool raise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          float v = sc[nt][x] * cs[nt][x & 1];
          if (masked) {
            const int key = t + r + (x >> 1) * 8;
            if (key < lo[nt][x & 1] || key >= hi[nt][x & 1]) v = -INFINITY;
          }
          sc[nt][x] = v;
          raise |= v > m[nt][x & 1] + kRaise;
        }
      if (__any_sync(kFull, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float top = fmaxf(m[nt][y], fmaxf(sc[nt][y], sc[nt][y + 2]));
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, w));
            if (!(top > m[nt][y] + kRaise)) top = m[nt][y];  // a row's results do not depend on its neighbours'
            const float f = top == m[nt][y] ? 1.0f : ex2(m[nt][y] - top);  // (-inf: both empty)
            m[nt][y] = top;
            l[nt][y] *= f;
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) o[mt][nt][y] *= f, o[mt][nt][y + 2] *= f;
          }
      }
      uint32_t pf[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float p[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float top = m[nt][x & 1];
          p[x] = ex2(sc[nt][x] - (top == -INFINITY ? 0.0f : top));
          l[nt][x & 1] += p[x];
        }
        pf[nt][0] = transpose8x8(pack_f16x2(p[0], p[1]));
        pf[nt][1] = transpose8x8(pack_f16x2(p[2], p[3]));
      }

      // ---- O^T += V'^T P^T: tokens 2j, 2j+1 (pair 0) and 2j+8, 2j+9 (pair 1), dimensions [r D/8, (r+1) D/8)
      uint32_t vs2[2][kW];  // scale pairs (token, next token) of each block
      {
        uint32_t w[kW];
#pragma unroll
        for (int x = 0; x < kW; ++x)
          w[x] = *reinterpret_cast<const uint32_t*>(atom + KvAtom<D>::kVScales +
                                                    ((D == 64 ? r >> 1 : r) * 4 + j) * (4 * kW) + 4 * x);
        if (masked && t + 16 > s.kv_len) {
          // Bytes behind the last key are whatever the page held: their scales
          // become zero, so that 0 * NaN cannot reach the sum.
#pragma unroll
          for (int x = 0; x < 4 * kW; ++x) {
            const int i4 = x / kW;
            if (t + 8 * (i4 >> 1) + 2 * j + (i4 & 1) >= s.kv_len) w[x >> 2] &= ~(0xFFu << (8 * (x & 3)));
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
      // The lane's D/4 value bytes: words of 8 dimensions, D/64 * ... per token.
      constexpr int kVW = D / 64;  // 32-bit words per token
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
    }
    cp_async_wait<0>();

    // ---- join the warps: results per row in shared memory (over the ring)
    __syncthreads();
    float* res = reinterpret_cast<float*>(smem);                 // [kWarps][R][kPitch]
    float* stat = res + kWarps * R * kPitch;                     // [kWarps][R][2]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float sum = l[nt][y];
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) sum += __shfl_xor_sync(kFull, sum, w);
        const int row = nt * 8 + 2 * j + y;
        float* rp = res + (warp * R + row) * kPitch + r * (D / 8);
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt)
          *reinterpret_cast<float2*>(rp + 2 * mt) = make_float2(o[mt][nt][y], o[mt][nt][y + 2]);
        if (r == 0) {
          stat[(warp * R + row) * 2] = m[nt][y];
          stat[(warp * R + row) * 2 + 1] = sum;
        }
      }
    __syncthreads();
    const int p_first = part_of(seg0), p_last = part_of(seg0 + s.units - 1);
    const bool whole = p_first == p_last;
    constexpr int kSlot = R * (D + 2);  // floats of a partial result: R rows of D, then R pairs (m, l)
    float* slot = a.partials + (2 * int64_t(blockIdx.x) + (seg0 >= u0 ? 1 : 0)) * kSlot;
    auto store_row = [&](int row, int d, float x0, float x1, float top, float sum) {
      const int x = tile * R + row, token = x / a.group, g = x - token * a.group;
      const int64_t at = s.q0 + token;
      const int h = head * a.group + g;
      const float f = sum > 0.0f || sum != sum ? gv / sum : 0.0f;
      uint16_t* op = a.out + at * a.ld_ot + h * a.ld_oh + d;
      const uint32_t v = pack_bf16x2(x0 * f, x1 * f);
      if ((reinterpret_cast<uintptr_t>(op) & 3) == 0) {
        *reinterpret_cast<uint32_t*>(op) = v;
      } else {
        op[0] = uint16_t(v);
        op[1] = uint16_t(v >> 16);
      }
      if (a.lse != nullptr && d == 0)
        a.lse[at * a.ld_lse + h] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    };
    for (int i = tid; i < rows * (D / 2); i += kAttnRowsThreads) {
      const int row = i / (D / 2), d = 2 * (i % (D / 2));
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stat[(w * R + row) * 2]);
      float x0 = 0.0f, x1 = 0.0f, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = stat[(w * R + row) * 2];
        const float f = mw == -INFINITY ? (stat[(w * R + row) * 2 + 1] == 0.0f ? 0.0f : 1.0f) : ex2(mw - top);
        const float2 v = *reinterpret_cast<const float2*>(res + (w * R + row) * kPitch + d);
        x0 += f * v.x;
        x1 += f * v.y;
        sum += f * stat[(w * R + row) * 2 + 1];
      }
      if (whole) {
        store_row(row, d, x0, x1, top, sum);
      } else {
        *reinterpret_cast<float2*>(slot + row * D + d) = make_float2(x0, x1);
        if (d == 0) *reinterpret_cast<float2*>(slot + R * D + 2 * row) = make_float2(top, sum);
      }
    }
    if (!whole) {
      // The last of the segment's CTAs to arrive joins the parts, in the order of their tokens.
      __threadfence();
      __syncthreads();
      if (tid == 0) s_last = atomicAdd(a.counters + p_first, 1u) == uint32_t(p_last - p_first) ? 1 : 0;
      __syncthreads();
      if (s_last) {
        __threadfence();
        auto part = [&](int p) { return a.partials + (2 * int64_t(p) + (p == p_first ? 1 : 0)) * kSlot; };
        for (int i = tid; i < rows * (D / 2); i += kAttnRowsThreads) {
          const int row = i / (D / 2), d = 2 * (i % (D / 2));
          float top = -INFINITY, x0 = 0.0f, x1 = 0.0f, sum = 0.0f;
          for (int p = p_first; p <= p_last; ++p) {
            const float2 st = __ldcg(reinterpret_cast<const float2*>(part(p) + R * D + 2 * row));
            const float2 v = __ldcg(reinterpret_cast<const float2*>(part(p) + row * D + d));
            const float up = fmaxf(top, st.x);
            const float f0 = top == up ? 1.0f : ex2(top - up);
            const float f1 = st.x == up ? 1.0f : ex2(st.x - up);
            x0 = x0 * f0 + v.x * f1;
            x1 = x1 * f0 + v.y * f1;
            sum = sum * f0 + st.y * f1;
            top = up;
          }
          store_row(row, d, x0, x1, top, sum);
        }
        if (tid == 0) a.counters[p_first] = 0;
      }
    }
    __syncthreads();  // shared memory is free for the next segment
    u = seg0 + ub;
  }
}

}  // namespace

const void* attn_rows_kernel(int d, int n_tiles) {
#define NQ_ROWS(D, NT) \
  if (d == D && n_tiles == NT) return reinterpret_cast<const void*>(&rows_kernel<D, NT>);
  NQ_ROWS(64, 1) NQ_ROWS(64, 2) NQ_ROWS(128, 1) NQ_ROWS(128, 2) NQ_ROWS(256, 1) NQ_ROWS(256, 2)
#undef NQ_ROWS
  return nullptr;
}

size_t attn_rows_smem(int d, int n_tiles) {
  const size_t m = merge_bytes(d, 8 * n_tiles);
  return m > ring_bytes(d) ? m : ring_bytes(d);
}

}  // namespace nq

// nq_kv_cache.cu — tokens into the 4-bit key/value cache and back.
//
// A block is 16 elements of one token's key or value of one kv head.  Append:
// sf = e4m3(RN(RN(absmax / 6) / g)), codes e2m1(RN(x * RN(1 / RN(sf * g)))),
// the block quantizer of nq_rmsnorm_quant_nvfp4 on raw activations.  Gather:
// RN_bf16(RN((e2m1 * sf) * g)); the product e2m1 * sf has at most six
// significant bits, so it is exact in float32.
//
// Both are bound by memory: a pair of key and value elements moves 4 bytes of
// bf16 and 1.125 bytes of cache.  A thread owns one block of the key and the
// same block of the value (32 contiguous bf16 bytes each, one 32-byte access) of
// two heads, whose loads all wait for the slot once, and a warp covers 512 / D
// consecutive tokens of a head, so that the 8-byte pieces into which the atom's
// order cuts a value row (16 bytes hold a pair of tokens, 32 bytes two pairs) leave
// the warp as whole 32-byte sectors when the tokens are consecutive.
// 65536 tokens, 8 heads of 128: append 60.4 us (5.7 TB/s; 69 with one head a
// thread), gather 55 us (6.2 TB/s, 0.95 of copy bandwidth; 64).
#include "nq_kv_layout.cuh"
#include "nq_row_kernel.cuh"

namespace nq {

namespace {

struct Raw {
  uint32_t w[8];  // 16 bf16
};

template <bool VEC>
__device__ __forceinline__ Raw load16(const uint16_t* p) {
  Raw r;
  if constexpr (VEC) {
    asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]),
                   "=r"(r.w[7])
                 : "l"(p));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = uint32_t(p[2 * i]) | (uint32_t(p[2 * i + 1]) << 16);
  }
  return r;
}

template <bool VEC>
__device__ __forceinline__ void store16(uint16_t* p, const Raw& r) {
  if constexpr (VEC) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r.w[0]), "r"(r.w[1]), "r"(r.w[2]),
                 "r"(r.w[3]), "r"(r.w[4]), "r"(r.w[5]), "r"(r.w[6]), "r"(r.w[7])
                 : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[2 * i] = uint16_t(r.w[i]);
      p[2 * i + 1] = uint16_t(r.w[i] >> 16);
    }
  }
}

struct Place {
  int token, head, block;
  bool live;         // a token of the batch
  bool second;       // a second head, head + 1
  int64_t slot;      // -1: nothing to do
  uint8_t* atom;     // of the slot, first head
  int64_t per_head;  // bytes between the heads' atoms
};

// The blocks that this thread owns, of two heads: warps count pairs of heads
// fastest, then groups of 512 / D tokens.
template <int D>
__device__ __forceinline__ Place place_of(const KvCopyArgs& a) {
  constexpr int kBlocks = D / 16, kTokens = 32 / kBlocks;
  const int64_t warp = (int64_t(blockIdx.x) * kKvCopyThreads + threadIdx.x) >> 5;
  const int lane = int(threadIdx.x) & 31;
  Place p;
  const int pairs = (a.cache.heads + 1) >> 1;
  const int64_t group = warp / pairs;
  p.head = 2 * int(warp - group * pairs);
  p.second = p.head + 1 < a.cache.heads;
  p.per_head = int64_t(18 * D) << (a.cache.log_page - 4);
  const int64_t token = group * kTokens + lane / kBlocks;
  p.block = lane % kBlocks;
  p.live = token < a.T;
  p.token = p.live ? int(token) : 0;
  p.slot = p.live ? a.slots[token] : -1;
  p.atom = nullptr;
  if (p.slot >= 0) {
    const int64_t page = p.slot >> a.cache.log_page;
    if (page >= a.cache.pages) {
      atomicOr(a.err, kErrSlot);
      p.slot = -1;
    } else {
      const int in = int(p.slot) & ((1 << a.cache.log_page) - 1);
      p.atom = a.cache.base + page * a.cache.page_stride + p.head * p.per_head + (in >> 4) * (18 * D);
    }
  }
  return p;
}

// Codes and scale of one block; every lane of the warp calls this together.
__device__ __forceinline__ void quantize_block(const Raw& r, float g, float ngr, bool g_fast, uint2* codes,
                                               uint32_t* sf) {
  float2 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = make_float2(bf16_lo(r.w[i]), bf16_hi(r.w[i]));
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmax3(amax, fabsf(v[i].x), fabsf(v[i].y));
  const Nvfp4Scale s = nvfp4_block_scale<false>(amax, g, ngr, g_fast);
  float t[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 q = mul2(v[i], f2(s.mult));
    t[i / 4][2 * (i % 4)] = q.x;
    t[i / 4][2 * (i % 4) + 1] = q.y;
  }
  *codes = make_uint2(pack_e2m1x8(t[0]), pack_e2m1x8(t[1]));
  *sf = s.code;
}

template <int D, bool VEC>
__global__ void __launch_bounds__(kKvCopyThreads, 4) append_kernel(const KvCopyArgs a) {
  griddep_wait();
  const Place p = place_of<D>(a);
  Raw k[2] = {}, v[2] = {};
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (p.slot >= 0 && (h == 0 || p.second)) {
      k[h] = load16<VEC>(a.k + p.token * a.ld_kt + (p.head + h) * a.ld_kh + 16 * p.block);
      v[h] = load16<VEC>(a.v + p.token * a.ld_vt + (p.head + h) * a.ld_vh + 16 * p.block);
    }
  griddep_launch_dependents();
  const float gk = __ldg(a.k_scale), gv = __ldg(a.v_scale);
  const float nrk = -__frcp_rn(gk), nrv = -__frcp_rn(gv);
  const bool fast_k = fast_div_ok(gk), fast_v = fast_div_ok(gv);
  const int t = int(p.slot) & 15;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint2 kc, vc;
    uint32_t ks, vs;
    quantize_block(k[h], gk, nrk, fast_k, &kc, &ks);
    quantize_block(v[h], gv, nrv, fast_v, &vc, &vs);
    if (p.slot < 0 || (h == 1 && !p.second)) continue;
    uint8_t* atom = p.atom + h * p.per_head;
    *reinterpret_cast<uint2*>(atom + KvAtom<D>::k_codes(t, p.block)) = kc;
    uint8_t* vp = atom + KvAtom<D>::v_codes(t, p.block);
    if constexpr (D == 64) {  // the block's halves belong to two lanes, 64 bytes apart
      *reinterpret_cast<uint32_t*>(vp) = vc.x;
      *reinterpret_cast<uint32_t*>(vp + 64) = vc.y;
    } else {
      *reinterpret_cast<uint2*>(vp) = vc;
    }
    atom[KvAtom<D>::k_scale(t, p.block)] = uint8_t(ks);
    atom[KvAtom<D>::v_scale(t, p.block)] = uint8_t(vs);
  }
}

__device__ __forceinline__ Raw dequantize_block(uint2 codes, uint32_t sf, float g) {
  const float s = e4m3_to_f32(sf);
  Raw r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h[4];
    e2m1x8_to_f16x2(i ? codes.y : codes.x, h);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
      const float2 y = mul2(mul2(x, f2(s)), f2(g));
      r.w[4 * i + j] = pack_bf16x2(y.x, y.y);
    }
  }
  return r;
}

template <int D, bool VEC>
__global__ void __launch_bounds__(kKvCopyThreads) gather_kernel(const KvCopyArgs a) {
  griddep_wait();
  const Place p = place_of<D>(a);
  uint2 kc[2] = {}, vc[2] = {};
  uint32_t ks[2] = {}, vs[2] = {};
  const int t = int(p.slot) & 15;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (p.slot >= 0 && (h == 0 || p.second)) {
      const uint8_t* atom = p.atom + h * p.per_head;
      kc[h] = *reinterpret_cast<const uint2*>(atom + KvAtom<D>::k_codes(t, p.block));
      const uint8_t* vp = atom + KvAtom<D>::v_codes(t, p.block);
      if constexpr (D == 64)
        vc[h] = make_uint2(*reinterpret_cast<const uint32_t*>(vp), *reinterpret_cast<const uint32_t*>(vp + 64));
      else
        vc[h] = *reinterpret_cast<const uint2*>(vp);
      ks[h] = atom[KvAtom<D>::k_scale(t, p.block)];
      vs[h] = atom[KvAtom<D>::v_scale(t, p.block)];
    }
  griddep_launch_dependents();
  if (!p.live) return;
  // A padding token reads as zeros whatever the global scales hold.
  const float gk = p.slot >= 0 ? __ldg(a.k_scale) : 0.0f, gv = p.slot >= 0 ? __ldg(a.v_scale) : 0.0f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (h == 1 && !p.second) continue;
    store16<VEC>(a.k + p.token * a.ld_kt + (p.head + h) * a.ld_kh + 16 * p.block, dequantize_block(kc[h], ks[h], gk));
    store16<VEC>(a.v + p.token * a.ld_vt + (p.head + h) * a.ld_vh + 16 * p.block, dequantize_block(vc[h], vs[h], gv));
  }
}

}  // namespace

const void* kv_append_kernel(int d, bool vec) {
#define NQ_KV(D) \
  if (d == D)    \
    return vec ? reinterpret_cast<const void*>(&append_kernel<D, true>) : reinterpret_cast<const void*>(&append_kernel<D, false>);
  NQ_KV(64) NQ_KV(128) NQ_KV(256)
#undef NQ_KV
  return nullptr;
}

const void* kv_gather_kernel(int d, bool vec) {
#define NQ_KV(D) \
  if (d == D)    \
    return vec ? reinterpret_cast<const void*>(&gather_kernel<D, true>) : reinterpret_cast<const void*>(&gather_kernel<D, false>);
  NQ_KV(64) NQ_KV(128) NQ_KV(256)
#undef NQ_KV
  return nullptr;
}

}  // namespace nq

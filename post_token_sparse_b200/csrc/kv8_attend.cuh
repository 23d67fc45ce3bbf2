// Decode attention over the paged 8-bit cache.
//
//   l_t = scale * sK(t) * (q . kcode_t),  p = softmax(l),
//   O = sum_t p_t sV(t) vcode_t,  lse = log sum_t exp(l_t)
// over every token of a sequence (dense) or over a list of kept tokens.
//
// HBM-bound: 256 B a token and KV head, read once for all query heads of the
// head's group.  A query head needs 256 multiply-adds a row and the codes have
// to be widened first, which at HBM rate is more than the CUDA cores issue
// next to the copies, so both products run as small matrix products on the
// tensor cores (mma.sync m16n8k16, f16 in, fp32 accumulate).  tcgen05 takes the
// rows from shared or tensor memory, so that every widened row would have to be
// written there first; here it goes on from registers, 8 columns (the heads of
// a list) are all there is to multiply by, and the copies are the bound:
//   S^T[16 rows x 8 heads]  = K[16 rows x 128] . Q^T[128 x 8 heads]
//   O^T[128 x 8 heads]     += V^T[128 x 16 rows] . W^T[16 rows x 8 heads]
// A tile is 32 rows, two such products side by side: what a tile costs beside
// them (addresses, the softmax's shuffles) is shared by more rows.
// An 8-bit code is exact in f16.  Q (bf16, 8 significant bits) is brought to a
// largest value of 2^13..2^14 by a power of two per head, after which f16
// holds it exactly (below 2^-28 of the largest to 2^-39 of it).
//
// Softmax: a warp keeps a reference r per head, the running maximum of
// y_t = x_t + e_t, x the logit in the log2 domain and 2^(e+29) just above sV,
//   p_t = 2^(x_t - r),  L = sum p_t,  w_t = p_t sV(t) 2^-29 <= 1.
// So w fits f16 whatever the pages' scales (r takes the place of the maximum
// logit), and w 2^14 is split into an f16 and the f16 of its remainder: 22
// bits, or 2^-39 of the largest w.  e is at least -93 and, for finite V, at
// most 93, which keeps p away from both ends of fp32.  Logits far from zero
// would swallow e: once a maximum is beyond 2^20 the head's base b moves there,
// and x is the logit less b (one fused multiply-add).
//
// Work split: the tiles of all lists (a list: the rows that up to 8 query heads
// attend over) form one sequence, sequence after sequence; a CTA takes an equal
// run of it, and its warps equal parts of that.  The lengths are on the GPU, so
// every CTA sums them itself (lens are a few KB in L2) and finds where its warps
// begin.  A list within one warp's range is written directly; otherwise the
// warps' partials (r, L, b, unnormalised O) meet after the CTA's last tile (a
// warp's last list in its idle ring, the one it began inside, whose partial is
// done while the ring is full, in a place beside), all its warps merge them, and
// what crosses CTAs goes to global memory, where the CTA that arrives last (a
// counter per CTA in which a list begins) merges the CTAs' partials in order.
// Where all lists have as many tiles a CTA may take whole lists instead.
//
// Measured on B200 (bytes it cannot do without by device time, a copy makes
// 6553 GB/s): dense, 8 sequences of 4096 tokens, 32 KV heads 49 us, 5490 GB/s;
// 16 of 5000 to 16384, 64 heads over 8, 66 us, 5310 GB/s; one of 1000, 32
// heads, 10.3 us; per-head lists of 16384 of 262144 tokens, 32 heads, 32 us, 4340
// GB/s; group lists of 1024, 16 sequences, 64 heads over 8, 13.8 us.  The loop
// over tiles runs at the copy's rate (41 of the 49 us of the first); the rest
// is the chain lengths -> page ids -> rows before it (3 us), and after it the
// slower CTAs (3 us) and the merges (3 us).
//
// Shared memory: per warp a ring of tiles of 32 rows x 256 B (K row, V row)
// filled by cp.async; chunk c (16 B) of row r sits at c ^ (r & 7), so that the
// 8 rows an ldmatrix reads fall in 8 bank groups.  V goes through
// ldmatrix.trans, which moves pairs of bytes: a lane gets two dims of two
// rows, and the even and odd bytes are the operands of two dims.
#pragma once

#include "attend_group.cuh"
#include "common.cuh"
#include "kv8_append.cuh"

namespace ds {

constexpr int kKv8Ctas = kAttnCtas;
constexpr int kKv8Rows = 32;                        // rows per tile
constexpr int kKv8TileBytes = kKv8Rows * 2 * kHeadDim;
constexpr int kKv8SideBytes = kKv8Rows * 8 + 16;    // the rows' scales, the tile's info
constexpr int kKv8MinTiles = 8;                     // of a CTA, where there are as many
// Query heads of a list: an mma's columns.  More heads of a KV head are several
// lists, each of which reads and widens the rows again: 57 and 62 us (e4m3, int8)
// for 16 ragged sequences of up to 16384, 64 heads over 4, whose bytes need 27.
// Lists of up to 16, whose accumulators leave 8 warps, took 55 and 57 us where
// two of 8 took 54 and 60, and 25 where they took 18 (kept lists of 2048 over the
// same heads).
constexpr int kKv8MaxHeads = 8;

struct Kv8Cfg {
  static constexpr int kWarps = 12;  // by the registers of the accumulators
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kStages = 2;
  static constexpr int kPart = kKv8MaxHeads * kPartialStride;  // floats of a partial at most
  static constexpr int kRing = kStages * kKv8TileBytes;
  static constexpr int kSideAt = kWarps * kRing;
  static constexpr int kPlaceAt = kSideAt + kWarps * kStages * kKv8SideBytes;
  // Places for the partial of the list a warp's range began inside: as many as
  // fit, which is one for every warp up to 4 heads.  Beyond these the partial
  // waits in global memory for the warp's ring to be idle.
  static constexpr int kPlaceBytes = 6 * kPart * 4;
  static constexpr size_t kSmem = kPlaceAt + kPlaceBytes;
  static_assert(2 * kPart * 4 <= kRing, "two partials fit a ring");
  static_assert(kSmem <= 225 * 1024, "one CTA per SM, with the static part");
  static_assert(2 * kWarps <= 32, "a lane for each partial slot");
};

// Workspace: a counter for each CTA, then two partials for each CTA and one for
// each warp.
constexpr size_t kKv8CounterBytes = 1024;
static_assert(kKv8Ctas * 4 <= kKv8CounterBytes, "");
inline size_t kv8_workspace_bytes(int heads) {
  return kKv8CounterBytes +
         (size_t)(2 + Kv8Cfg::kWarps) * kKv8Ctas * heads * kPartialStride * sizeof(float);
}

struct Kv8Params {
  const uint16_t* Q;     // [B, Hq, 128]
  const uint8_t* KV;     // [P, Hkv, p, 2, 128]
  const float* scales;   // [P, Hkv, 2]
  const int32_t* table;  // [B, W]
  const int32_t* lens;   // [B]
  const int32_t* idx;    // kept tokens, null: dense
  float* O;              // [B, Hq, 128]
  float* lse;            // [B, Hq] or null
  uint32_t* arrivals;    // [kKv8Ctas], zero between calls
  float* partial;        // [2 * kKv8Ctas, heads, kPartialStride]
  float* warp_partial;   // [kKv8Ctas * warps, heads, kPartialStride]
  int B, Hq, Hkv, P, W, shift;
  int k;
  int G;                 // query heads of a KV head
  int parts;             // lists of a KV head
  int heads;             // query heads of a list (the last of a KV head may have fewer)
  int lists;             // lists of a sequence: Hkv * parts
  int idx_shared;        // idx [B * Hkv, k] rather than [B * Hq, k]
  float scale_log2;      // softmax scale * log2(e)
};

struct Kv8Shared {
  static constexpr int kWarps = Kv8Cfg::kWarps;
  int sum[kWarps];
  int seq[kWarps];  // the sequence a warp's range begins in
  int lo[kWarps];   // that sequence's first tile
  // partials: slot 2w the list that warp w's range began inside, 2w+1 its last
  int gs[2 * kWarps], ge[2 * kWarps];  // the list's tiles
  int list[2 * kWarps];                // -1: none
  int places;                          // taken
  float* place[kWarps];                // of slot 2w
  int last[2], cf[2], cl[2], gi[2];
};

__device__ __forceinline__ void cp_async8_zfill(uint32_t smem, const void* gmem, bool v) {
  const uint32_t n = v ? 8u : 0u;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem), "l"(gmem), "r"(n)
               : "memory");
}
// +1 on a counter in global memory, in order with this thread's accesses
// before and after
__device__ __forceinline__ uint32_t arrive_acq_rel(uint32_t* p) {
  uint32_t old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(p) : "memory");
  return old;
}
// 2^x to 2 ulp, results below 2^-126 as 0
__device__ __forceinline__ float exp2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// d += a . b for one m16n8k16 tile, f16 operands, fp32 accumulators
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// {lo, hi} -> f16x2 (lo in the low half), round to nearest even
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ void unpack_f16(uint32_t w, float& lo, float& hi) {
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}"
      : "=f"(lo), "=f"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  return h;
}

// Bytes 0 and 2 of a word of codes as f16x2 in `even`, 1 and 3 in `odd`.  int8:
// the byte of x + 128 under 0x64 is the f16 of 1152 + x, and the subtraction
// is exact.
template <bool kE4m3>
__device__ __forceinline__ void kv8_widen(uint32_t w, uint32_t& even, uint32_t& odd) {
  if constexpr (kE4m3) {
    const uint32_t s = __byte_perm(w, 0, 0x3120);
    even = e4m3x2_f16x2(s & 0xffffu);
    odd = e4m3x2_f16x2(s >> 16);
  } else {
    const uint32_t s = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(s, 0x64646464u, 0x4240), b = __byte_perm(s, 0x64646464u, 0x4341);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(even) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(odd) : "r"(b), "r"(0x64806480u));
  }
}

// Bytes {0, 1} and {2, 3} of e4m3 codes (K, whose dims may be taken in any
// order: one step less than by parity); int8 as above.
template <bool kE4m3>
__device__ __forceinline__ void kv8_widen_k(uint32_t w, uint32_t& a, uint32_t& b) {
  if constexpr (kE4m3) {
    a = e4m3x2_f16x2(w & 0xffffu);
    b = e4m3x2_f16x2(w >> 16);
  } else {
    kv8_widen<false>(w, a, b);
  }
}

// e with |s| < 2^(e + 29), at least -93
__device__ __forceinline__ float scale_exponent(float s) {
  return (float)max((int)((__float_as_uint(s) >> 23) & 255u) - 155, -93);
}

// Reference, sum and base of a partial.
struct Kv8Ends {
  float r, l, b;
};
__device__ __forceinline__ Kv8Ends kv8_no_ends() { return {-INFINITY, 0.f, 0.f}; }

// Brings the references of n partials a lane of a warp to their largest base,
// which is returned.
template <int n>
__device__ __forceinline__ float kv8_common_base(Kv8Ends (&h)[n]) {
  bool any = false;
#pragma unroll
  for (int q = 0; q < n; ++q) any |= h[q].b != 0.f;
  if (!__any_sync(0xffffffffu, any)) return 0.f;
  float b = -INFINITY;
#pragma unroll
  for (int q = 0; q < n; ++q) b = fmaxf(b, h[q].r == -INFINITY ? -INFINITY : h[q].b);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, d));
#pragma unroll
  for (int q = 0; q < n; ++q)
    if (h[q].r != -INFINITY) h[q].r += h[q].b - b;
  return b;
}

// The common reference M of a warp's partials, lane i holding the reference r
// and sum l of one (-inf, 0: none), their merged sum L, and in return the
// lane's weight.
__device__ __forceinline__ float kv8_weights(float r, float l, float& M, float& L) {
  M = r;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  const float w = rescale(r, M);
  L = l * w;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
  return w;
}
__device__ __forceinline__ void kv8_add(float4& acc, float w, const float4& v) {
  acc.x = fmaf(v.x, w, acc.x);
  acc.y = fmaf(v.y, w, acc.y);
  acc.z = fmaf(v.z, w, acc.z);
  acc.w = fmaf(v.w, w, acc.w);
}

// Merge of n partials of a head (r, L, b, -, o[128]; the first at `at0`, the
// others at at + i * stride, written by other CTAs and read around L1) by a
// warp.  acc: dims 4*lane.. of the merged o over the partials first, first +
// step, ..
__device__ __forceinline__ void kv8_merge(const float* at0, const float* at, size_t stride, int n,
                                          int first, int step, int lane, Kv8Ends& all,
                                          float4& acc) {
  auto part = [&](int i) { return i == 0 ? at0 : at + min(i, n - 1) * stride; };
  auto ends = [&](int i) {
    if (i >= n) return kv8_no_ends();
    const float4 v = __ldcg(reinterpret_cast<const float4*>(part(i)));
    return Kv8Ends{v.x, v.y, v.z};
  };
  auto row = [&](int i) { return __ldcg(reinterpret_cast<const float4*>(part(i) + 4) + lane); };
  // everything that up to 4 partials a warp need is loaded at once
  constexpr int kF = 4, kQ = (kKv8Ctas + 31) / 32;
  float4 v[kF];
#pragma unroll
  for (int e = 0; e < kF; ++e) v[e] = row(first + e * step);
  Kv8Ends h[kQ];  // partials lane, lane + 32, ..
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    h[q] = kv8_no_ends();
    if (q * 32 < n) h[q] = ends(lane + q * 32);
  }
  all.b = kv8_common_base(h);
  float r = -INFINITY, l = 0.f;
#pragma unroll
  for (int q = 0; q < kQ; ++q) r = fmaxf(r, h[q].r);
#pragma unroll
  for (int q = 0; q < kQ; ++q) l = fmaf(h[q].l, rescale(h[q].r, r), l);
  kv8_weights(r, l, all.r, all.l);
  float w0[kQ];  // weights
#pragma unroll
  for (int q = 0; q < kQ; ++q) w0[q] = rescale(h[q].r, all.r);
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = first; i0 < n; i0 += kF * step) {
    float4 next[kF];
    if (i0 + kF * step < n) {
#pragma unroll
      for (int e = 0; e < kF; ++e) next[e] = row(i0 + (kF + e) * step);
    }
#pragma unroll
    for (int e = 0; e < kF; ++e) {
      const int i = i0 + e * step;
      float w = __shfl_sync(0xffffffffu, w0[0], i & 31);
      if (n > 32) {
#pragma unroll
        for (int q = 1; q < kQ; ++q) {
          const float x = __shfl_sync(0xffffffffu, w0[q], i & 31);
          if (i >> 5 == q) w = x;
        }
      }
      if (i < n) kv8_add(acc, w, v[e]);
      v[e] = next[e];
    }
  }
}

constexpr float kKv8Unit = 32768.f;  // the accumulators hold w 2^14 = p sV 2^-15

// 1 / L, or 0 for a list with nothing in it
__device__ __forceinline__ float kv8_inverse(float L) { return L == 0.f ? 0.f : 1.f / L; }
__device__ __forceinline__ float kv8_lse(const Kv8Ends& h) {
  return h.l == 0.f ? -INFINITY : (h.b + (h.r + log2f(h.l))) * 0.69314718055994530942f;
}

// O and lse of one query head by a warp: lane i has dims 4i..4i+3.
__device__ __forceinline__ void kv8_write(const Kv8Params& p, size_t head, int lane,
                                          const Kv8Ends& h, const float4& a) {
  const float inv = kv8_inverse(h.l);
  reinterpret_cast<float4*>(p.O + head * kHeadDim)[lane] =
      make_float4(a.x * kKv8Unit * inv, a.y * kKv8Unit * inv, a.z * kKv8Unit * inv,
                  a.w * kKv8Unit * inv);
  if (p.lse && lane == 0) p.lse[head] = kv8_lse(h);
}

// A merged partial of one head by a warp.
__device__ __forceinline__ void kv8_keep(float* at, int lane, const Kv8Ends& h, const float4& a) {
  if (lane == 0) *reinterpret_cast<float4*>(at) = make_float4(h.r, h.l, h.b, 0.f);
  *reinterpret_cast<float4*>(at + 4 + 4 * lane) = a;
}

// First query head (of all B * Hq) and number of heads of list gi.
__device__ __forceinline__ void kv8_heads(const Kv8Params& p, int gi, size_t& head, int& n) {
  n = p.heads;
  head = (size_t)gi * p.heads;
  if (p.heads * p.parts == p.G) return;
  const int b = gi / p.lists, c = gi - b * p.lists;
  const int g = c / p.parts, part = c - g * p.parts;
  head = (size_t)b * p.Hq + (size_t)g * p.G + (size_t)part * p.heads;
  n = min(p.heads, p.G - part * p.heads);
}

// grid: at most kKv8Ctas CTAs
template <bool kE4m3, bool kSparse>
__global__ void __launch_bounds__(Kv8Cfg::kThreads, 1)
k_kv8_attend(const Kv8Params p) {
  using C = Kv8Cfg;
  constexpr int W = C::kWarps, S = C::kStages;
  extern __shared__ __align__(128) unsigned char kv8_smem[];
  __shared__ Kv8Shared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, tq = lane & 3;  // fragment coordinates

  // ---- the plan: this CTA's tiles and where its warps begin
  const int row_cap = p.W << p.shift;  // at most 2^30
  auto rows_of = [&](int b) {
    const int n = __ldg(p.lens + b);
    if (kSparse && (n < 0 || n > row_cap)) flag_status(16u);
    return min(max(n, 0), row_cap);
  };
  const int sparse_tiles = (p.k + kKv8Rows - 1) / kKv8Rows;
  constexpr int kChunk = C::kThreads * 4;
  // tiles of sequences base .. base + kChunk-1: four a thread (t), the sum of
  // those before the thread's (ex), the sum of all (returned)
  auto scan = [&](int base, int (&t)[4], int& ex, bool& empty) -> int {
    int own = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int b = base + (int)threadIdx.x * 4 + j;
      t[j] = 0;
      if (b < p.B) {
        const int n = __ldg(p.lens + b);
        if (n < 0 || n > row_cap) flag_status(16u);
        if (n <= 0) empty = true;
        t[j] = (min(max(n, 0), row_cap) + kKv8Rows - 1) / kKv8Rows;
      }
      own += t[j];
    }
    int in = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, in, d);
      if (lane >= d) in += y;
    }
    __syncthreads();  // readers of the chunk before are done
    if (lane == 31) sh.sum[warp] = in;
    __syncthreads();
    int all = 0;
    ex = in - own;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < warp) ex += sh.sum[w];
      all += sh.sum[w];
    }
    return all;
  };
  // up to 128 sequences: every warp finds its place by itself, without a barrier
  // (10.0 and 9.85 us for one sequence, 11.1 and 10.6 for 64)
  const bool small = !kSparse && p.B <= 128;
  int t4[4], ex = 0, total = 0;
  int even = kSparse ? sparse_tiles : 0;  // tiles of every list, 0: they differ
  if constexpr (kSparse) {
    total = p.B * p.lists * sparse_tiles;
  } else {
    bool empty = false;
    if (small) {
      int own = 0, most = 0, least = INT32_MAX;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int b = lane * 4 + j;
        const int n = b < p.B ? __ldg(p.lens + b) : 1;
        if (n <= 0) empty = true;
        if (n < 0 || n > row_cap) flag_status(16u);
        t4[j] = b < p.B ? (min(max(n, 0), row_cap) + kKv8Rows - 1) / kKv8Rows : 0;
        own += t4[j];
        most = max(most, t4[j]);
        if (b < p.B) least = min(least, t4[j]);
      }
      most = __reduce_max_sync(0xffffffffu, most);
      least = __reduce_min_sync(0xffffffffu, least);
      if (most == least) even = most;
      ex = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, ex, d);
        if (lane >= d) ex += y;
      }
      total = __shfl_sync(0xffffffffu, ex, 31);
      ex -= own;
      empty = __any_sync(0xffffffffu, empty);
    } else {
      for (int base = 0; base < p.B; base += kChunk) total += scan(base, t4, ex, empty);
      empty = __syncthreads_or(empty);
    }
    total *= p.lists;
    if (empty) {
      // sequences of no tokens
      for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (__ldg(p.lens + b) > 0) continue;
        for (int i = threadIdx.x; i < p.Hq * kHeadDim; i += C::kThreads)
          p.O[(size_t)b * p.Hq * kHeadDim + i] = 0.f;
        if (p.lse)
          for (int i = threadIdx.x; i < p.Hq; i += C::kThreads)
            p.lse[(size_t)b * p.Hq + i] = -INFINITY;
      }
    }
  }
  int per = max((total + (int)gridDim.x - 1) / (int)gridDim.x, kKv8MinTiles);
  if (even > 0) {
    // Whole lists, where that costs few tiles more, leave nothing to merge
    // between CTAs.  For dense calls this holds up to 128 sequences, beyond which
    // `even` is not known.  Whole and cut, by more tiles on those of a cut:
    // group lists of 8 heads 13.6 and 18.4 us (4 on 28), 18.2 and 21.6 (13 on 35),
    // 21.8 and 24.5 (21 on 51), 25.0 and 27.7 (23 on 61), 42.1 and 43.3 (23 on
    // 153); beyond the limit 16.8 and 17.9 (22 on 26), 27.0 and 28.0 (25 on 65),
    // 44.7 and 45.7 (25 on 167), 29.7 and 29.9 (30 on 78).  One head a list, whose
    // merges are shorter: 9.9 and 12.1 (11 on 13), 12.1 and 11.9 (14 on 18), 22.7
    // and 22.7 (23 on 57), beyond the limit 14.0 and 12.8 (18 on 22), 17.6 and
    // 15.9 (26 on 32).
    const int whole = (p.B * p.lists + (int)gridDim.x - 1) / (int)gridDim.x * even;
    if (whole - per <= min(12 + per / 4, 24)) per = max(whole, 1);
  }
  const int xc = (int)min((long long)blockIdx.x * per, (long long)total);
  const int nc = min(per, total - xc);
  if (nc == 0) return;
  // warps without a tile, if any, are the last
  auto from = [&](int w) { return xc + nc / W * w + min(w, nc % W); };
  const int x0 = from(warp), cnt = from(warp + 1) - x0;
  if (lane < 2) sh.list[2 * warp + lane] = -1;
  if (threadIdx.x == 0) sh.places = 0;
  __syncthreads();
  int seq0 = 0, lo0 = 0;  // the sequence this warp's range begins in and its first tile
  if constexpr (!kSparse) {
    if (small) {
      int lo = ex * p.lists;
      bool mine = false;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int hi = lo + t4[j] * p.lists;
        if (x0 >= lo && x0 < hi) {
          mine = true;
          seq0 = lane * 4 + j;
          lo0 = lo;
        }
        lo = hi;
      }
      const uint32_t who = __ballot_sync(0xffffffffu, mine);
      const int from_lane = who ? __ffs(who) - 1 : 0;  // none: an idle warp at the end
      seq0 = __shfl_sync(0xffffffffu, seq0, from_lane);
      lo0 = __shfl_sync(0xffffffffu, lo0, from_lane);
    } else {
      int before = 0;
      bool empty = false;
      for (int base = 0; base < p.B; base += kChunk) {
        const int n = p.B <= kChunk ? total : scan(base, t4, ex, empty);
        int lo = (before + ex) * p.lists;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int hi = lo + t4[j] * p.lists;
          if (hi > xc && lo < xc + nc)
            for (int w = 0; w < W; ++w)
              if (from(w) >= lo && from(w) < hi) {
                sh.seq[w] = base + (int)threadIdx.x * 4 + j;
                sh.lo[w] = lo;
              }
          lo = hi;
        }
        before += n;
      }
      __syncthreads();
      seq0 = sh.seq[warp];
      lo0 = sh.lo[warp];
    }
  }

  // ---- tiles
  unsigned char* const ring = kv8_smem + warp * C::kRing;
  unsigned char* const side = kv8_smem + C::kSideAt + warp * S * kKv8SideBytes;
  const uint32_t ring_s = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  const uint32_t side_s = static_cast<uint32_t>(__cvta_generic_to_shared(side));
  auto ring_part = [&](int w) { return reinterpret_cast<float*>(kv8_smem + w * C::kRing); };
  // a place for this warp's slot 2w, taken when it is needed
  float* const away = p.warp_partial + (size_t)(blockIdx.x * W + warp) * p.heads * kPartialStride;
  bool is_away = false;
  const int part_floats = p.heads * kPartialStride;
  auto take_place = [&]() -> float* {
    int i = 0;
    if (lane == 0) i = atomicAdd(&sh.places, 1);
    i = __shfl_sync(0xffffffffu, i, 0);
    if ((i + 1) * part_floats * 4 > C::kPlaceBytes) return away;
    float* at = reinterpret_cast<float*>(kv8_smem + C::kPlaceAt) + i * part_floats;
    if (lane == 0) sh.place[warp] = at;
    return at;
  };

  // a tile on its way to being copied
  struct Tile {
    int b, g, gi;   // sequence, KV head, list
    int tile, nt;   // of the list
    int rows;       // the sequence's length
    int t, pg;      // the token of row `lane` (-1: none) and its page
  };
  Tile cur = {};  // the next tile to describe
  int part = 0;   // its list among the KV head's
  if (cnt > 0) {
    if constexpr (kSparse) {
      cur.nt = sparse_tiles;
      cur.gi = x0 / sparse_tiles;
      cur.tile = x0 - cur.gi * sparse_tiles;
      cur.b = cur.gi / p.lists;
      cur.rows = rows_of(cur.b);
    } else {
      cur.b = seq0;
      cur.rows = rows_of(cur.b);
      cur.nt = (cur.rows + kKv8Rows - 1) / kKv8Rows;
      const int rel = x0 - lo0, c = rel / cur.nt;
      cur.tile = rel - c * cur.nt;
      cur.gi = cur.b * p.lists + c;
    }
    const int c = cur.gi - cur.b * p.lists;
    cur.g = c / p.parts;
    part = c - cur.g * p.parts;
  }
  int described = 0;

  // the next tile and its tokens (sparse: being loaded)
  auto describe = [&](Tile& d) {
    d = cur;
    d.t = -1;
    d.pg = -1;
    if (described == cnt) {
      d.nt = 0;  // none
      return;
    }
    ++described;
    if constexpr (kSparse) {
      const int r = d.tile * kKv8Rows + lane;
      const size_t row = p.idx_shared ? (size_t)d.b * p.Hkv + d.g : (size_t)d.gi;
      if (r < p.k) d.t = __ldg(p.idx + row * p.k + r);
    } else {
      const int r = d.tile * kKv8Rows + lane;
      if (r < d.rows) d.t = r;
    }
    if (described == cnt) return;
    if (++cur.tile < cur.nt) return;
    cur.tile = 0;
    ++cur.gi;
    if (++part < p.parts) return;
    part = 0;
    if (++cur.g < p.Hkv) return;
    cur.g = 0;
    do {
      cur.rows = rows_of(++cur.b);
      if constexpr (!kSparse) cur.nt = (cur.rows + kKv8Rows - 1) / kKv8Rows;
    } while (!kSparse && cur.nt == 0);  // a later tile exists, so a later sequence has rows
    cur.gi = cur.b * p.lists;
  };
  // the pages of a described tile's tokens
  auto look_up = [&](Tile& d) {
    if (kSparse && d.t >= d.rows) {
      flag_status(2u);
      d.t = -1;
    }
    if (d.t >= 0) {
      d.pg = __ldg(p.table + (size_t)d.b * p.W + (d.t >> p.shift));
    } else if (kSparse && d.t != -1) {
      flag_status(2u);
    }
  };

  // raw query fragments of a list: lane (gq, tq) holds head column gq's values
  // at dims 16c + 4tq .. +3
  uint2 qnext[8];
  auto load_q = [&](int gi) {
    size_t head;
    int n;
    kv8_heads(p, gi, head, n);
    const uint2* q = reinterpret_cast<const uint2*>(p.Q + (head + (gq < n ? gq : 0)) * kHeadDim);
#pragma unroll
    for (int c = 0; c < 8; ++c)
      qnext[c] = gq < n ? __ldg(q + c * 4 + tq) : make_uint2(0u, 0u);
  };

  // copy i: rows 2i + crow, 16-byte chunk cch of a row; four swizzles
  const int crow = lane >> 4, cch = lane & 15;
  int swz[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) swz[i] = crow * 256 + ((cch ^ ((2 * i + crow) & 7)) << 4);
  auto copy = [&](const Tile& d, int st) {
    if (d.nt == 0) return;
    unsigned char* const to = ring + st * kKv8TileBytes;
    bool ok = d.t >= 0;
    if (ok && (d.pg < 0 || d.pg >= p.P)) {
      flag_status(8u);
      ok = false;
    }
    const int tile = ok ? d.pg * p.Hkv + d.g : 0;
    const int at = (tile << p.shift) + (ok ? d.t & ((1 << p.shift) - 1) : 0);
    const uint32_t mask = __ballot_sync(0xffffffffu, ok);
    cp_async8_zfill(side_s + st * kKv8SideBytes + lane * 8, p.scales + (size_t)tile * 2, ok);
    const bool all = mask == 0xffffffffu;
    if (!kSparse && all) {
      // 16 rows of a page are one run
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int src = __shfl_sync(0xffffffffu, at, 16 * h);
        const uint8_t* from = p.KV + (size_t)src * (2 * kHeadDim) + lane * 16;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          cp_async16(to + (8 * h + i) * 512 + swz[i & 3], from + i * 512);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int row = 2 * i + crow;
        const int src = __shfl_sync(0xffffffffu, at, row);
        cp_async16_zfill(to + i * 512 + swz[i & 3],
                         p.KV + (size_t)src * (2 * kHeadDim) + cch * 16, (mask >> row) & 1u);
      }
    }
    if (lane == 0)
      *reinterpret_cast<int4*>(side + st * kKv8SideBytes + kKv8Rows * 8) =
          make_int4((int)mask, d.gi, d.tile, d.nt);
  };

  // d0: the tile copied next, its pages loaded; d1: the one after, its tokens loaded
  Tile d0, d1;
  {
    Tile first;
    describe(first);
    if constexpr (kSparse) {
      describe(d0);
      if (cnt > 0) load_q(first.gi);
      look_up(first);
      look_up(d0);
    } else {
      look_up(first);
      describe(d0);
      look_up(d0);
      if (cnt > 0) load_q(first.gi);
    }
    describe(d1);
    copy(first, 0);
    cp_async_commit();
  }

  const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8, lch = lane >> 4;  // ldmatrix rows
  uint32_t q[16];
  float qs[2];  // logit of a product of codes, per column: times sK
  float o[8][4];
  // references, sums and bases of columns 2tq, 2tq+1
  float r2[2], l2[2], b2[2];

  bool fresh = true;
  for (int n = 0; n < cnt; ++n) {
    __syncwarp();  // every lane's reads of the slot about to be refilled are done
    copy(d0, (n + 1) % S);
    cp_async_commit();
    d0 = d1;
    look_up(d0);
    describe(d1);
    if (fresh) {  // a list begins: its queries as fragments
      // the head's largest exponent, over its four lanes
      uint32_t mx = 0;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint2 w = qnext[c];
        mx = max(max(mx, max(w.x & 0x7fff0000u, (w.x << 16) & 0x7fffffffu)),
                 max(w.y & 0x7fff0000u, (w.y << 16) & 0x7fffffffu));
      }
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const uint32_t e = max(mx >> 23, 14u);                       // q < 2^(e - 126)
      const float up = __uint_as_float((267u - e) << 23);          // 2^(140 - e)
      const float down = __uint_as_float((e - 13u) << 23) * p.scale_log2;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint2 w = qnext[c];
        const float a = bf_lo(w.x) * up, b = bf_hi(w.x) * up, x = bf_lo(w.y) * up,
                    y = bf_hi(w.y) * up;
        // the order in which kv8_widen_k gives K's dims
        q[2 * c] = kE4m3 ? pack_f16(a, b) : pack_f16(a, x);
        q[2 * c + 1] = kE4m3 ? pack_f16(x, y) : pack_f16(b, y);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        qs[i] = __shfl_sync(0xffffffffu, down, (2 * tq + i) * 4);
        r2[i] = -INFINITY;
        l2[i] = 0.f;
        b2[i] = 0.f;
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.f;
    }
    cp_async_wait<1>();
    __syncwarp();
    const int st = n % S;
    const unsigned char* sd = side + st * kKv8SideBytes;
    const int4 info = *reinterpret_cast<const int4*>(sd + kKv8Rows * 8);
    const bool ends = info.z == info.w - 1, done = n == cnt - 1;
    fresh = ends;

    if (ends && !done)  // the next list's queries on their way
      load_q(reinterpret_cast<const int*>(side + ((n + 1) % S) * kKv8SideBytes + kKv8Rows * 8)[1]);

    const uint32_t ld = ring_s + st * kKv8TileBytes + lrow * 256;
    // S^T = K . Q^T
    float s4[2][4] = {};
#pragma unroll
    for (int c = 0; c < 8; c += 2) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t w[4];
        ldsm_x4(ld + u * 4096 + (((c + lch) ^ (lrow & 7)) << 4), w);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t a[4];
          kv8_widen_k<kE4m3>(w[2 * i], a[0], a[2]);
          kv8_widen_k<kE4m3>(w[2 * i + 1], a[1], a[3]);
          mma_f16(s4[u], a, q[2 * (c + i)], q[2 * (c + i) + 1]);
        }
      }
    }

    // rows gq + 8i: scales, exponents, whether the row counts
    float sk[4], sv[4], ev[4];
    bool in[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 sc = *reinterpret_cast<const float2*>(sd + (gq + 8 * i) * 8);
      sk[i] = sc.x;
      sv[i] = sc.y * (1.f / 32768.f);
      ev[i] = scale_exponent(sc.y);
      in[i] = (info.x >> (gq + 8 * i)) & 1;
    }
    // W^T: for 16 rows parts of rows 0-7 and 8-15 (, remainders)
    uint32_t bw[2][4];
    float x[2][4], y[2];  // column 2tq + i, row gq + 8e; their maximum
    // rows that do not count are selected away, not added to: their zero codes
    // times an infinite or NaN query are NaN
    auto logits = [&](int i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = fmaf(s4[e >> 1][2 * (e & 1) + i], qs[i] * sk[e], -b2[i]);
        x[i][e] = in[e] ? v : -INFINITY;
      }
      y[i] = fmaxf(fmaxf(x[i][0] + ev[0], x[i][1] + ev[1]),
                   fmaxf(x[i][2] + ev[2], x[i][3] + ev[3]));
#pragma unroll
      for (int d = 4; d <= 16; d <<= 1) y[i] = fmaxf(y[i], __shfl_xor_sync(0xffffffffu, y[i], d));
    };
    logits(0);
    logits(1);
    bool g0 = y[0] > r2[0], g1 = y[1] > r2[1];
    if (__any_sync(0xffffffffu, g0 || g1)) {
      auto far = [&](float v) { return fabsf(v) > 0x1p20f && fabsf(v) < INFINITY; };
      if (__any_sync(0xffffffffu, (g0 && far(y[0])) || (g1 && far(y[1])))) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if ((i ? g1 : g0) && far(y[i])) {
            const float b = b2[i] + y[i];
            r2[i] += b2[i] - b;
            b2[i] = b;
          }
          logits(i);
        }
        g0 = y[0] > r2[0];
        g1 = y[1] > r2[1];
      }
      const float f0 = g0 ? exp2_ftz(r2[0] - y[0]) : 1.f;  // 0 while r is -inf
      const float f1 = g1 ? exp2_ftz(r2[1] - y[1]) : 1.f;
      if (g0) r2[0] = y[0];
      if (g1) r2[1] = y[1];
      l2[0] *= f0;
      l2[1] *= f1;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        o[c][0] *= f0;
        o[c][1] *= f1;
        o[c][2] *= f0;
        o[c][3] *= f1;
      }
    }
    float w[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float r = r2[i] == -INFINITY ? 0.f : r2[i];
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float pe = exp2_ftz(x[i][e] - r);
        sum += pe;
        w[i][e] = pe * sv[e];
      }
      l2[i] += sum;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t ha = pack_f16(w[0][2 * u], w[1][2 * u]);
      const uint32_t hb = pack_f16(w[0][2 * u + 1], w[1][2 * u + 1]);
      float f[4];
      unpack_f16(ha, f[0], f[1]);
      unpack_f16(hb, f[2], f[3]);
      const uint32_t ra = pack_f16(w[0][2 * u] - f[0], w[1][2 * u] - f[1]);
      const uint32_t rb = pack_f16(w[0][2 * u + 1] - f[2], w[1][2 * u + 1] - f[3]);
      bw[u][0] = movm_t(ha);
      bw[u][1] = movm_t(hb);
      bw[u][2] = movm_t(ra);
      bw[u][3] = movm_t(rb);
    }

    // O^T += V^T . W^T
#pragma unroll
    for (int c = 0; c < 8; c += 2) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t w[4];
        ldsm_x4_t(ld + u * 4096 + (((8 + c + lch) ^ (lrow & 7)) << 4), w);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t a[4];
          kv8_widen<kE4m3>(w[2 * i], a[0], a[1]);
          kv8_widen<kE4m3>(w[2 * i + 1], a[2], a[3]);
          mma_f16(o[c + i], a, bw[u][0], bw[u][1]);
          mma_f16(o[c + i], a, bw[u][2], bw[u][3]);
        }
      }
    }

    if (ends || done) {
      // the warp's rows of the list are done: sums over the 8 lanes of a column
      const int gs = x0 + n - info.z, ge = gs + info.w;
      const bool whole = gs >= x0 && ends;
      size_t head;
      int nh;
      kv8_heads(p, info.y, head, nh);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1)
          l2[i] += __shfl_xor_sync(0xffffffffu, l2[i], d);
      }
      const int slot = 2 * warp + (done ? 1 : 0);
      float* pt = ring_part(warp);
      if (!whole) {
        if (!done) {
          pt = take_place();
          is_away = pt == away;
        } else {
          // the ring is idle: nothing is left to copy
          cp_async_wait<0>();
          __syncwarp();
        }
        if (lane == 0) {
          sh.list[slot] = info.y;
          sh.gs[slot] = gs;
          sh.ge[slot] = ge;
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int h = 2 * tq + i;
        if (h >= nh) continue;
        if (whole) {
          const float inv = kv8_inverse(l2[i]);
          float2* out = reinterpret_cast<float2*>(p.O + (head + h) * kHeadDim) + gq;
#pragma unroll
          for (int c = 0; c < 8; ++c)
            out[c * 8] = make_float2(o[c][i] * kKv8Unit * inv, o[c][2 + i] * kKv8Unit * inv);
          if (p.lse && gq == 0)
            p.lse[head + h] = kv8_lse({r2[i], l2[i], b2[i]});
        } else {
          float* w = pt + h * kPartialStride;
          if (gq == 0)
            *reinterpret_cast<float4*>(w) = make_float4(r2[i], l2[i], b2[i], 0.f);
#pragma unroll
          for (int c = 0; c < 8; ++c)
            *reinterpret_cast<float2*>(w + 4 + 16 * c + 2 * gq) =
                make_float2(o[c][i], o[c][2 + i]);
        }
      }
    }
  }
  cp_async_wait<0>();
  if (is_away) {
    // back beside the last list's partial, in the idle ring
    __syncwarp();
    float4* to = reinterpret_cast<float4*>(ring_part(warp) + C::kPart);
    const float4* from4 = reinterpret_cast<const float4*>(away);
    constexpr int kN = (C::kPart / 4 + 31) / 32;
    const int words = part_floats / 4;
    float4 v[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (lane + 32 * i < words) v[i] = from4[lane + 32 * i];
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (lane + 32 * i < words) to[lane + 32 * i] = v[i];
    if (lane == 0) sh.place[warp] = reinterpret_cast<float*>(to);
  }

  // ---- lists shared by warps: the CTA's partials in the order of their tiles
  __syncthreads();
  const int mine = lane < 2 * W ? sh.list[lane] : -1;
  const int gs = mine >= 0 ? sh.gs[lane] : xc, ge = mine >= 0 ? sh.ge[lane] : xc;
  const uint32_t held = __ballot_sync(0xffffffffu, mine >= 0);
  if (held == 0) return;
  const uint32_t below = held & lanemask_lt();
  const int prev = __shfl_sync(0xffffffffu, mine, below ? 31 - __clz(below) : lane);
  const bool first = mine >= 0 && (below == 0 || prev != mine);  // of its list
  const bool enters = gs < xc, leaves = ge > xc + nc;            // from or to another CTA
  const uint32_t across = __ballot_sync(0xffffffffu, first && (enters || leaves));
  int item = 0;
  for (uint32_t starts = __ballot_sync(0xffffffffu, first); starts;) {
    const int s = __ffs(starts) - 1;
    starts &= starts - 1;
    const uint32_t members =
        held & (0xffffffffu << s) & (starts ? (1u << (__ffs(starts) - 1)) - 1u : 0xffffffffu);
    size_t head;
    int nh;
    kv8_heads(p, __shfl_sync(0xffffffffu, mine, s), head, nh);
    // a partial each of warps s/2, s/2 + 1, ..: that of a warp's last list in
    // its ring, after them one in a place beside if the list ends inside a range
    const int e = 31 - __clz(members);
    const bool extra = !(e & 1);
    const int nr = __popc(members) - (extra ? 1 : 0);
    // items (list, head) go round the warps
    const int item0 = item;
    item = (item + nh) % W;
    for (int j = (warp + W - item0) % W; j < nh; j += W) {
      const unsigned char* at = kv8_smem + (s >> 1) * C::kRing + j * (kPartialStride * 4);
      const float* xt = extra ? sh.place[e >> 1] + j * kPartialStride : nullptr;
      const unsigned char* row = at + 16 + 16 * lane;
      Kv8Ends h[1] = {kv8_no_ends()};
      auto ends = [](const void* q) {
        const float4 v = *static_cast<const float4*>(q);
        return Kv8Ends{v.x, v.y, v.z};
      };
      if (lane < nr) h[0] = ends(at + lane * C::kRing);
      float4 vx = make_float4(0.f, 0.f, 0.f, 0.f);
      if (extra) {
        vx = *reinterpret_cast<const float4*>(xt + 4 + 4 * lane);
        if (lane == nr) h[0] = ends(xt);
      }
      Kv8Ends all;
      all.b = kv8_common_base(h);
      const float wl = kv8_weights(h[0].r, h[0].l, all.r, all.l);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int i = 0; i < nr; ++i)
        kv8_add(acc, __shfl_sync(0xffffffffu, wl, i),
                *reinterpret_cast<const float4*>(row + i * C::kRing));
      if (extra) kv8_add(acc, __shfl_sync(0xffffffffu, wl, nr), vx);
      if (!((across >> s) & 1u)) {
        kv8_write(p, head + j, lane, all, acc);
      } else {
        const int slot = 2 * blockIdx.x + (__shfl_sync(0xffffffffu, (int)enters, s) ? 0 : 1);
        kv8_keep(p.partial + ((size_t)slot * p.heads + j) * kPartialStride, lane, all, acc);
      }
    }
  }
  if (across == 0) return;

  // ---- lists shared by CTAs: the last to arrive merges.  0: the list that
  // began before this CTA, 1: the one that begins here and goes on
  if (threadIdx.x < 2) sh.last[threadIdx.x] = 0;
  __syncthreads();
  if (warp == 0 && ((across >> lane) & 1u)) {
    const int which = enters ? 0 : 1, cf = gs / per, cl = (ge - 1) / per;
    // releases the CTA's partials (ordered before by the barrier), acquires the others'
    if (arrive_acq_rel(p.arrivals + cf) == (uint32_t)(cl - cf)) {
      p.arrivals[cf] = 0u;  // zero again for the next call
      sh.cf[which] = cf;
      sh.cl[which] = cl;
      sh.gi[which] = mine;
      sh.last[which] = 1;
    }
  }
  __syncthreads();
  // Both lists side by side.  With few heads and many partials each, several
  // warps share a head's partials: how many depends on the list alone, not on
  // which CTA is last, so that a result's bits do not.
  size_t head[2] = {0, 0};
  int nh[2] = {0, 0}, n[2] = {0, 0}, cf[2] = {0, 0}, split[2] = {1, 1};
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (!sh.last[which]) continue;
    kv8_heads(p, sh.gi[which], head[which], nh[which]);
    cf[which] = sh.cf[which];
    n[which] = sh.cl[which] - cf[which] + 1;
    if (n[which] > 8 && nh[which] < W) split[which] = W / nh[which];
  }
  const int items0 = nh[0] * split[0], items = items0 + nh[1] * split[1];
  const size_t stride = (size_t)2 * p.heads * kPartialStride;
  // item i's share of a head: in the rings, at most two a warp
  auto share = [&](int i) {
    return reinterpret_cast<float*>(kv8_smem + i % W * C::kRing) + i / W * kPartialStride;
  };
  for (int item = warp; item < items; item += W) {
    const bool second = item >= items0;
    const int sp = second ? split[1] : split[0], it = second ? item - items0 : item;
    const int h = it / sp, c0 = second ? cf[1] : cf[0];
    // the CTA in which the list begins has it in its second slot, the next in their first
    const float* first = p.partial + ((size_t)(2 * c0 + 1) * p.heads + h) * kPartialStride;
    const float* rest = p.partial + ((size_t)(2 * c0) * p.heads + h) * kPartialStride;
    Kv8Ends all;
    float4 acc;
    kv8_merge(first, rest, stride, second ? n[1] : n[0], it - h * sp, sp, lane, all, acc);
    if (sp == 1)
      kv8_write(p, (second ? head[1] : head[0]) + h, lane, all, acc);
    else
      kv8_keep(share(item), lane, all, acc);
  }
  if (split[0] == 1 && split[1] == 1) return;
  __syncthreads();
  for (int hh = warp; hh < nh[0] + nh[1]; hh += W) {
    const bool second = hh >= nh[0];
    const int h = second ? hh - nh[0] : hh, sp = second ? split[1] : split[0];
    if (sp == 1) continue;
    const int i0 = (second ? items0 : 0) + h * sp;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = i0; i < i0 + sp; ++i)
      kv8_add(acc, 1.f, *reinterpret_cast<const float4*>(share(i) + 4 + 4 * lane));
    const float4 e = *reinterpret_cast<const float4*>(share(i0));
    kv8_write(p, (second ? head[1] : head[0]) + h, lane, {e.x, e.y, e.z}, acc);
  }
}

}  // namespace ds

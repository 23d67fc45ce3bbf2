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
// tensor cores (mma.sync m16n8k16, f16 in, fp32 accumulate: at most 16 columns
// are useful, below the smallest tcgen05 tile, and the copies are the bound):
//   S^T[16 rows x 8 heads]  = K[16 rows x 128] . Q^T[128 x 8 heads]
//   O^T[128 x 8 heads]     += V^T[128 x 16 rows] . W^T[16 rows x 8 heads]
// An 8-bit code is exact in f16.  Q (bf16, 8 significant bits) is brought to a
// largest value of 2^13..2^14 by a power of two per head, after which f16
// holds it exactly (below 2^-28 of the largest to 2^-39 of it).
//
// Softmax: a warp keeps a reference r per head, the running maximum of
// y_t = x_t + e_t, x the logit in the log2 domain and 2^e just above sV, with
//   p_t = 2^(x_t - r),  L = sum p_t,  w_t = p_t sV(t) <= 1.
// So w fits f16 whatever the pages' scales (r takes the place of the maximum
// logit), and w 2^14 is split into an f16 and the f16 of its remainder: 22
// bits, or 2^-39 of the largest w.  With up to 4 heads the two parts share one
// product (columns 0-3 and 4-7), with more they take two.
//
// Work split: the 16-row tiles of all lists (a list: the rows one set of query
// heads attends over) form one sequence, sequence after sequence, and warp u
// of the grid takes tiles [T u/U, T (u+1)/U).  The lengths are on the GPU, so
// every CTA sums them itself (lens are a few KB in L2) and finds where its
// warps begin.  A list within one warp's range is written directly; otherwise
// the warps' partials (r, L, unnormalised O) meet in shared memory after the
// CTA's last tile, all its warps merge them, and what crosses CTAs goes to
// global memory, where the CTA that arrives last (a counter per CTA in which a
// list begins) merges the CTAs' partials in order.
//
// Shared memory: per warp a ring of tiles of 16 rows x 256 B (K row, V row)
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
constexpr int kKv8Rows = 16;                        // rows per tile
constexpr int kKv8TileBytes = kKv8Rows * 2 * kHeadDim;
constexpr int kKv8SideBytes = kKv8Rows * 8 + 16;    // the rows' scales, the tile's info
constexpr int kKv8MaxHeads = 16;                    // query heads of a list

// kHeads: query heads of a list at most.
template <int kHeads>
struct Kv8Cfg {
  static constexpr int kWarps = kHeads == 16 ? 8 : 12;  // by the registers of the accumulators
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kStages = kHeads == 8 ? 3 : 4;
  static constexpr int kNt = kHeads == 16 ? 2 : 1;      // 8-column products
  static constexpr bool kPack = kHeads == 4;            // both parts of w in one product
  static constexpr int kPart = kHeads * kPartialStride; // floats of a partial
  static constexpr int kRing = kStages * kKv8TileBytes;
  static constexpr int kSideAt = kWarps * kRing;
  static constexpr int kPartAt = kSideAt + kWarps * kStages * kKv8SideBytes;
  static constexpr size_t kSmem = kPartAt + (size_t)kWarps * kPart * 4;
  static_assert(kPart * 4 <= kRing, "a partial fits a ring");
  static_assert(kSmem <= 225 * 1024, "one CTA per SM, with the static part");
  static_assert(2 * kWarps <= 32, "a lane for each partial slot");
};

// Workspace: a counter for each CTA, then two partials for each CTA.
constexpr size_t kKv8CounterBytes = 1024;
static_assert(kKv8Ctas * 4 <= kKv8CounterBytes, "");
inline size_t kv8_workspace_bytes(int heads) {
  return kKv8CounterBytes + (size_t)2 * kKv8Ctas * heads * kPartialStride * 4;
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
  int B, Hq, Hkv, P, W, shift;
  int k;
  int G;                 // query heads of a KV head
  int parts;             // lists of a KV head
  int heads;             // query heads of a list (the last of a KV head may have fewer)
  int lists;             // lists of a sequence: Hkv * parts
  int idx_shared;        // idx [B * Hkv, k] rather than [B * Hq, k]
  float scale_log2;      // softmax scale * log2(e)
};

template <int kWarps>
struct Kv8Shared {
  long long sum[kWarps];
  long long from[kWarps + 1];  // first tile of each warp's range, and the end
  long long lo[kWarps];        // first tile of the sequence it begins in
  int seq[kWarps];
  // partials: slot 2w the list that warp w's range began inside, 2w+1 its last
  long long gs[2 * kWarps], ge[2 * kWarps];  // the list's tiles
  int list[2 * kWarps];                      // -1: none
  int flags[2 * kWarps];                     // 1: begins before the CTA, 2: ends after it
  int cf[2], cl[2], gi[2], last[2];
};

__device__ __forceinline__ void cp_async8(uint32_t smem, const void* gmem) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem), "l"(gmem) : "memory");
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

// e with |s| < 2^e, at least -64
__device__ __forceinline__ float scale_exponent(float s) {
  return (float)max((int)((__float_as_uint(s) >> 23) & 255u) - 126, -64);
}

// A partial's share of a merge: (M, L, acc) takes in (m, l, o), in fp32.
__device__ __forceinline__ void kv8_take(float& M, float& L, float4& acc, float m, float l,
                                         const float4& o) {
  const float mn = fmaxf(M, m);
  const float a = rescale(M, mn), c = rescale(m, mn);
  M = mn;
  L = L * a + l * c;
  acc.x = acc.x * a + o.x * c;
  acc.y = acc.y * a + o.y * c;
  acc.z = acc.z * a + o.z * c;
  acc.w = acc.w * a + o.w * c;
}

constexpr float kKv8Unit = 1.f / 16384.f;  // the accumulators hold w 2^14

// 1 / L, or 0 for a list with nothing in it
__device__ __forceinline__ float kv8_inverse(float L) { return L == 0.f ? 0.f : 1.f / L; }
__device__ __forceinline__ float kv8_lse(float M, float L) {
  return L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
}

// O and lse of one query head by a warp: lane i has dims 4i..4i+3.
__device__ __forceinline__ void kv8_write(const Kv8Params& p, size_t head, int lane, float M,
                                          float L, const float4& a) {
  const float inv = kv8_inverse(L);
  reinterpret_cast<float4*>(p.O + head * kHeadDim)[lane] =
      make_float4(a.x * kKv8Unit * inv, a.y * kKv8Unit * inv, a.z * kKv8Unit * inv,
                  a.w * kKv8Unit * inv);
  if (p.lse && lane == 0) p.lse[head] = kv8_lse(M, L);
}

// First query head (of all B * Hq) and number of heads of list gi.
__device__ __forceinline__ void kv8_heads(const Kv8Params& p, int gi, size_t& head, int& n) {
  const int b = gi / p.lists, c = gi - b * p.lists;
  const int g = c / p.parts, part = c - g * p.parts;
  head = (size_t)b * p.Hq + (size_t)g * p.G + (size_t)part * p.heads;
  n = min(p.heads, p.G - part * p.heads);
}

// grid: at most kKv8Ctas CTAs
template <bool kE4m3, bool kSparse, int kHeads>
__global__ void __launch_bounds__(Kv8Cfg<kHeads>::kThreads, 1)
k_kv8_attend(const Kv8Params p) {
  using C = Kv8Cfg<kHeads>;
  constexpr int W = C::kWarps, S = C::kStages;
  extern __shared__ __align__(128) unsigned char kv8_smem[];
  __shared__ Kv8Shared<W> sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, tq = lane & 3;  // fragment coordinates

  // ---- the plan: T tiles, this CTA's ranges and where they begin
  auto rows_of = [&](int b) {
    const int n = __ldg(p.lens + b);
    return n < 0 ? 0 : (int)min((long long)n, (long long)p.W << p.shift);
  };
  const int sparse_tiles = (p.k + kKv8Rows - 1) / kKv8Rows;
  constexpr int kChunk = C::kThreads * 4;
  // tiles of sequences base .. base + kChunk-1: four a thread (t), the sum of
  // those before the thread's (ex), the sum of all (returned)
  auto scan = [&](int base, int (&t)[4], long long& ex, bool flag) -> long long {
    long long own = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int b = base + (int)threadIdx.x * 4 + j;
      t[j] = 0;
      if (b < p.B) {
        const int n = __ldg(p.lens + b);
        if (flag && (n < 0 || n > (long long)p.W << p.shift)) flag_status(16u);
        t[j] = (int)((n < 0 ? 0 : min((long long)n, (long long)p.W << p.shift)) + kKv8Rows - 1) /
               kKv8Rows;
      }
      own += t[j];
    }
    long long in = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, in, d);
      if (lane >= d) in += y;
    }
    __syncthreads();  // readers of the chunk before are done
    if (lane == 31) sh.sum[warp] = in;
    __syncthreads();
    long long all = 0;
    ex = in - own;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < warp) ex += sh.sum[w];
      all += sh.sum[w];
    }
    return all;
  };
  int t4[4];
  long long ex = 0, total;
  if constexpr (kSparse) {
    total = (long long)p.B * p.lists * sparse_tiles;
  } else {
    total = 0;
    for (int base = 0; base < p.B; base += kChunk) total += scan(base, t4, ex, blockIdx.x == 0);
    total *= p.lists;
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
  const long long units = min((long long)gridDim.x * W, total);
  if ((long long)blockIdx.x * W >= units) return;
  if (threadIdx.x <= W) {
    const long long u = (long long)blockIdx.x * W + threadIdx.x;
    sh.from[threadIdx.x] = u >= units ? total : total * u / units;
  }
  if (threadIdx.x < 2 * W) sh.list[threadIdx.x] = -1;
  __syncthreads();
  const long long x0 = sh.from[warp];
  const int cnt = (int)(sh.from[warp + 1] - x0);
  if constexpr (!kSparse) {
    long long before = 0;
    for (int base = 0; base < p.B; base += kChunk) {
      const long long n = p.B <= kChunk ? total : scan(base, t4, ex, false);
      long long lo = (before + ex) * p.lists;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const long long hi = lo + (long long)t4[j] * p.lists;
        if (hi > sh.from[0] && lo < sh.from[W])
          for (int w = 0; w < W; ++w)
            if (sh.from[w] >= lo && sh.from[w] < hi) {
              sh.seq[w] = base + (int)threadIdx.x * 4 + j;
              sh.lo[w] = lo;
            }
        lo = hi;
      }
      before += n;
    }
    __syncthreads();
  }

  // ---- tiles
  unsigned char* const ring = kv8_smem + warp * C::kRing;
  unsigned char* const side = kv8_smem + C::kSideAt + warp * S * kKv8SideBytes;
  const uint32_t ring_s = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  const uint32_t side_s = static_cast<uint32_t>(__cvta_generic_to_shared(side));
  auto part_at = [&](int slot) -> float* {
    return slot & 1 ? reinterpret_cast<float*>(kv8_smem + (slot >> 1) * C::kRing)
                    : reinterpret_cast<float*>(kv8_smem + C::kPartAt) + (slot >> 1) * C::kPart;
  };

  // a tile on its way to being copied
  struct Tile {
    int b, g, gi;   // sequence, KV head, list
    int tile, nt;   // of the list
    int rows;       // dense: the sequence's rows; sparse: its length
    int t, pg;      // this lane's token (sparse: of row lane & 15) and page
  };
  Tile cur = {};  // the next tile to describe
  int part = 0;   // its list among the KV head's
  if (cnt > 0) {
    if constexpr (kSparse) {
      cur.nt = sparse_tiles;
      const long long l = x0 / sparse_tiles;
      cur.tile = (int)(x0 - l * sparse_tiles);
      cur.b = (int)(l / p.lists);
      cur.gi = (int)l;
      cur.rows = rows_of(cur.b);
    } else {
      cur.b = sh.seq[warp];
      cur.rows = rows_of(cur.b);
      cur.nt = (cur.rows + kKv8Rows - 1) / kKv8Rows;
      const long long rel = x0 - sh.lo[warp];
      const int c = (int)(rel / cur.nt);
      cur.tile = (int)(rel - (long long)c * cur.nt);
      cur.gi = cur.b * p.lists + c;
    }
    const int c = cur.gi - cur.b * p.lists;
    cur.g = c / p.parts;
    part = c - cur.g * p.parts;
  }
  int described = 0, issued = 0;

  // the next tile, its token ids (sparse) or page (dense) being loaded
  auto describe = [&](Tile& d) {
    d = cur;
    d.t = -1;
    d.pg = -1;
    if (described >= cnt) return;
    ++described;
    if constexpr (kSparse) {
      const int r = d.tile * kKv8Rows + (lane & 15);
      const size_t row = p.idx_shared ? (size_t)d.b * p.Hkv + d.g : (size_t)d.gi;
      if (r < p.k) d.t = __ldg(p.idx + row * p.k + r);
    } else {
      d.pg = __ldg(p.table + (size_t)d.b * p.W + ((d.tile * kKv8Rows) >> p.shift));
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
  // sparse: the pages of a described tile's tokens
  auto look_up = [&](Tile& d) {
    if constexpr (kSparse) {
      if (d.t >= 0 && d.t < d.rows) {
        d.pg = __ldg(p.table + (size_t)d.b * p.W + (d.t >> p.shift));
      } else {
        if (d.t != -1) flag_status(2u);
        d.t = -1;
      }
    }
  };

  // raw query fragments of a list: lane (gq, tq) holds head column gq's values
  // at dims 16c + 4tq .. +3
  uint2 qnext[C::kNt][8];
  int qn_list = -1;
  auto load_q = [&](int gi) {
    size_t head;
    int n;
    kv8_heads(p, gi, head, n);
#pragma unroll
    for (int j = 0; j < C::kNt; ++j) {
      const int h = C::kPack ? gq & 3 : gq + 8 * j;
      const uint2* q = reinterpret_cast<const uint2*>(p.Q + (head + (h < n ? h : 0)) * kHeadDim);
#pragma unroll
      for (int c = 0; c < 8; ++c)
        qnext[j][c] = h < n ? __ldg(q + c * 4 + tq) : make_uint2(0u, 0u);
    }
    qn_list = gi;
  };

  Tile d0, d1, d2;
  describe(d0);
  describe(d1);
  if (cnt > 0) load_q(d0.gi);
  describe(d2);
  look_up(d0);
  look_up(d1);

  const int crow = lane >> 4, cch = lane & 15;  // copy i: rows 2i + crow, 16-byte chunk cch
  auto issue = [&]() {
    if (issued >= cnt) return;
    const int st = issued % S;
    ++issued;
    const Tile d = d0;
    d0 = d1;
    d1 = d2;
    look_up(d1);
    describe(d2);
    if (d.tile == 0 && qn_list < 0) load_q(d.gi);

    unsigned char* const to = ring + st * kKv8TileBytes;
    const uint32_t sd = side_s + st * kKv8SideBytes;
    uint32_t mask;
    const int in_page = (1 << p.shift) - 1;
    if constexpr (kSparse) {
      bool ok = d.t >= 0;
      if (ok && (d.pg < 0 || d.pg >= p.P)) {
        flag_status(8u);
        ok = false;
      }
      const int tile = ok ? d.pg * p.Hkv + d.g : 0;
      const int at = (tile << p.shift) + (ok ? d.t & in_page : 0);
      mask = __ballot_sync(0xffffffffu, ok) & 0xffffu;
      if (lane < 16) cp_async8(sd + lane * 8, p.scales + (size_t)tile * 2);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = 2 * i + crow;
        const int src = __shfl_sync(0xffffffffu, at, row);
        cp_async16_zfill(to + row * 256 + ((cch ^ (row & 7)) << 4),
                         p.KV + (size_t)src * (2 * kHeadDim) + cch * 16, (mask >> row) & 1u);
      }
    } else {
      const int r = d.tile * kKv8Rows;
      bool ok = true;
      if (d.pg < 0 || d.pg >= p.P) {
        if (lane == 0) flag_status(8u);
        ok = false;
      }
      const int tile = ok ? d.pg * p.Hkv + d.g : 0;
      const int n = ok ? min(kKv8Rows, d.rows - r) : 0;
      mask = (1u << n) - 1u;
      if (lane < 16) cp_async8(sd + lane * 8, p.scales + (size_t)tile * 2);
      const uint8_t* src =
          p.KV + ((size_t)((tile << p.shift) + (r & in_page))) * (2 * kHeadDim) + lane * 16;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = 2 * i + crow;
        cp_async16_zfill(to + row * 256 + ((cch ^ (row & 7)) << 4), src + i * 512, row < n);
      }
    }
    if (lane == 0)
      *reinterpret_cast<int4*>(side + st * kKv8SideBytes + kKv8Rows * 8) =
          make_int4((int)mask, d.gi, d.tile, d.nt);
  };

#pragma unroll
  for (int s = 0; s < S - 1; ++s) {
    issue();
    cp_async_commit();
  }

  const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8, lch = lane >> 4;  // ldmatrix rows
  uint32_t q[C::kNt][16];
  float qs[C::kNt][2];  // logit of a product of codes, per column: times sK
  float o[C::kNt][8][4];
  float r2[C::kNt][2], l2[C::kNt][2];  // references and sums of columns 2tq, 2tq+1

  for (int n = 0; n < cnt; ++n) {
    __syncwarp();  // every lane's reads of the slot about to be refilled are done
    issue();
    cp_async_commit();
    cp_async_wait<S - 1>();
    __syncwarp();
    const int st = n % S;
    const unsigned char* sd = side + st * kKv8SideBytes;
    const int4 info = *reinterpret_cast<const int4*>(sd + kKv8Rows * 8);

    if (n == 0 || info.z == 0) {
      if (qn_list != info.y) load_q(info.y);
      qn_list = -1;
#pragma unroll
      for (int j = 0; j < C::kNt; ++j) {
        // the head's largest exponent, over its four lanes
        uint32_t mx = 0;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint2 w = qnext[j][c];
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
          const uint2 w = qnext[j][c];
          const float a = bf_lo(w.x) * up, b = bf_hi(w.x) * up, x = bf_lo(w.y) * up,
                      y = bf_hi(w.y) * up;
          // the order in which kv8_widen_k gives K's dims
          q[j][2 * c] = kE4m3 ? pack_f16(a, b) : pack_f16(a, x);
          q[j][2 * c + 1] = kE4m3 ? pack_f16(x, y) : pack_f16(b, y);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          qs[j][i] = __shfl_sync(0xffffffffu, down, (2 * tq + i) * 4);
          r2[j][i] = -INFINITY;
          l2[j][i] = 0.f;
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) o[j][c][0] = o[j][c][1] = o[j][c][2] = o[j][c][3] = 0.f;
      }
    }

    const uint32_t ld = ring_s + st * kKv8TileBytes + lrow * 256;
    // S^T = K . Q^T; with one product of columns, two sums side by side
    float s4[2][4] = {};
#pragma unroll
    for (int c = 0; c < 8; c += 2) {
      uint32_t w[4];
      ldsm_x4(ld + (((c + lch) ^ (lrow & 7)) << 4), w);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t a[4];
        kv8_widen_k<kE4m3>(w[2 * i], a[0], a[2]);
        kv8_widen_k<kE4m3>(w[2 * i + 1], a[1], a[3]);
#pragma unroll
        for (int j = 0; j < C::kNt; ++j)
          mma_f16(s4[C::kNt == 2 ? j : i], a, q[j][2 * (c + i)], q[j][2 * (c + i) + 1]);
      }
    }
    if constexpr (C::kNt == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s4[0][i] += s4[1][i];
    }

    float2 sa = *reinterpret_cast<const float2*>(sd + gq * 8);
    float2 sb = *reinterpret_cast<const float2*>(sd + (gq + 8) * 8);
    const bool va = (info.x >> gq) & 1, vb = (info.x >> (gq + 8)) & 1;
    if (!va) sa.y = 0.f;  // a row left out has the scale of any page, NaN perhaps
    if (!vb) sb.y = 0.f;
    const float ea = scale_exponent(sa.y), eb = scale_exponent(sb.y);
    uint32_t bw[C::kNt][C::kPack ? 2 : 4];  // W^T: parts of rows 0-7 and 8-15 (, remainders)
#pragma unroll
    for (int j = 0; j < C::kNt; ++j) {
      float x[4], y[2], pw[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[i] = va ? s4[j][i] * (qs[j][i] * sa.x) : -INFINITY;
        x[2 + i] = vb ? s4[j][2 + i] * (qs[j][i] * sb.x) : -INFINITY;
        y[i] = fmaxf(x[i] + ea, x[2 + i] + eb);
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) y[i] = fmaxf(y[i], __shfl_xor_sync(0xffffffffu, y[i], d));
      }
      const bool g0 = y[0] > r2[j][0], g1 = y[1] > r2[j][1];
      if (__any_sync(0xffffffffu, g0 || g1)) {
        const float f0 = g0 ? exp2f(r2[j][0] - y[0]) : 1.f;  // 0 while r is -inf
        const float f1 = g1 ? exp2f(r2[j][1] - y[1]) : 1.f;
        if (g0) r2[j][0] = y[0];
        if (g1) r2[j][1] = y[1];
        l2[j][0] *= f0;
        l2[j][1] *= f1;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          o[j][c][0] *= f0;
          o[j][c][1] *= f1;
          o[j][c][2] *= f0;
          o[j][c][3] *= f1;
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float r = r2[j][i] == -INFINITY ? 0.f : r2[j][i];
        const float pa = exp2f(x[i] - r), pb = exp2f(x[2 + i] - r);
        l2[j][i] += pa + pb;
        pw[i] = pa * 16384.f * sa.y;
        pw[2 + i] = pb * 16384.f * sb.y;
      }
      const uint32_t ha = pack_f16(pw[0], pw[1]), hb = pack_f16(pw[2], pw[3]);
      float f[4];
      unpack_f16(ha, f[0], f[1]);
      unpack_f16(hb, f[2], f[3]);
      const uint32_t ra = pack_f16(pw[0] - f[0], pw[1] - f[1]);
      const uint32_t rb = pack_f16(pw[2] - f[2], pw[3] - f[3]);
      if constexpr (C::kPack) {
        bw[j][0] = movm_t(tq < 2 ? ha : ra);
        bw[j][1] = movm_t(tq < 2 ? hb : rb);
      } else {
        bw[j][0] = movm_t(ha);
        bw[j][1] = movm_t(hb);
        bw[j][2] = movm_t(ra);
        bw[j][3] = movm_t(rb);
      }
    }

    // O^T += V^T . W^T
#pragma unroll
    for (int c = 0; c < 8; c += 2) {
      uint32_t w[4];
      ldsm_x4_t(ld + (((8 + c + lch) ^ (lrow & 7)) << 4), w);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t a[4];
        kv8_widen<kE4m3>(w[2 * i], a[0], a[1]);
        kv8_widen<kE4m3>(w[2 * i + 1], a[2], a[3]);
#pragma unroll
        for (int j = 0; j < C::kNt; ++j) {
          mma_f16(o[j][c + i], a, bw[j][0], bw[j][1]);
          if constexpr (!C::kPack) mma_f16(o[j][c + i], a, bw[j][2], bw[j][3]);
        }
      }
    }

    const bool ends = info.z == info.w - 1, done = n == cnt - 1;
    if (ends || done) {
      // the warp's rows of the list are done: sums over the 8 lanes of a column
      const long long gs = x0 + n - info.z, ge = gs + info.w;
      const bool whole = gs >= x0 && ends;
      size_t head;
      int nh;
      kv8_heads(p, info.y, head, nh);
#pragma unroll
      for (int j = 0; j < C::kNt; ++j) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int d = 4; d <= 16; d <<= 1)
            l2[j][i] += __shfl_xor_sync(0xffffffffu, l2[j][i], d);
        }
        if constexpr (C::kPack) {
          // a head's two parts of w: columns h and h + 4
#pragma unroll
          for (int c = 0; c < 8; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[j][c][i] += __shfl_xor_sync(0xffffffffu, o[j][c][i], 2);
        }
      }
      const int slot = 2 * warp + (done ? 1 : 0);
      float* const pt = part_at(slot);
      if (!whole) {
        if (done) {
          // the ring is idle: nothing is left to copy
          cp_async_wait<0>();
          __syncwarp();
        }
        if (lane == 0) {
          sh.list[slot] = info.y;
          sh.gs[slot] = gs;
          sh.ge[slot] = ge;
          sh.flags[slot] = (gs < sh.from[0] ? 1 : 0) | (ge > sh.from[W] ? 2 : 0);
        }
      }
#pragma unroll
      for (int j = 0; j < C::kNt; ++j) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int h = 8 * j + 2 * tq + i;
          if (h >= nh || (C::kPack && tq >= 2)) continue;
          if (whole) {
            const float inv = kv8_inverse(l2[j][i]);
            float2* out = reinterpret_cast<float2*>(p.O + (head + h) * kHeadDim) + gq;
#pragma unroll
            for (int c = 0; c < 8; ++c)
              out[c * 8] = make_float2(o[j][c][i] * kKv8Unit * inv, o[j][c][2 + i] * kKv8Unit * inv);
            if (p.lse && gq == 0) p.lse[head + h] = kv8_lse(r2[j][i], l2[j][i]);
          } else {
            float* w = pt + h * kPartialStride;
            if (gq == 0) *reinterpret_cast<float2*>(w) = make_float2(r2[j][i], l2[j][i]);
#pragma unroll
            for (int c = 0; c < 8; ++c)
              *reinterpret_cast<float2*>(w + 4 + 16 * c + 2 * gq) =
                  make_float2(o[j][c][i], o[j][c][2 + i]);
          }
        }
      }
    }
  }
  cp_async_wait<0>();

  // ---- lists shared by warps: the CTA's partials in the order of their tiles
  __syncthreads();
  const int mine = lane < 2 * W ? sh.list[lane] : -1;
  const int flags = lane < 2 * W && mine >= 0 ? sh.flags[lane] : 0;
  const uint32_t held = __ballot_sync(0xffffffffu, mine >= 0);
  if (held == 0) return;
  const uint32_t below = held & lanemask_lt();
  const int prev = __shfl_sync(0xffffffffu, mine, below ? 31 - __clz(below) : lane);
  uint32_t starts = __ballot_sync(0xffffffffu, mine >= 0 && (below == 0 || prev != mine));
  const uint32_t crossing = __ballot_sync(0xffffffffu, flags != 0);
  for (int item = 0; starts;) {
    const int s = __ffs(starts) - 1;
    starts &= starts - 1;
    const uint32_t members =
        held & (0xffffffffu << s) & (starts ? (1u << (__ffs(starts) - 1)) - 1u : 0xffffffffu);
    const int gi = sh.list[s], fl = sh.flags[s];
    size_t head;
    int nh;
    kv8_heads(p, gi, head, nh);
    for (int j = 0; j < nh; ++j, ++item) {
      if (item % W != warp) continue;
      float M = -INFINITY, L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (uint32_t m = members; m; m &= m - 1) {
        const float* pt = part_at(__ffs(m) - 1) + j * kPartialStride;
        kv8_take(M, L, acc, pt[0], pt[1], *reinterpret_cast<const float4*>(pt + 4 + 4 * lane));
      }
      if (fl == 0) {
        kv8_write(p, head + j, lane, M, L, acc);
      } else {
        float* w = p.partial + ((size_t)(2 * blockIdx.x + (fl & 1 ? 0 : 1)) * p.heads + j) *
                                   kPartialStride;
        if (lane == 0) *reinterpret_cast<float2*>(w) = make_float2(M, L);
        *reinterpret_cast<float4*>(w + 4 + 4 * lane) = acc;
      }
    }
  }
  if (crossing == 0) return;

  // ---- lists shared by CTAs: the last to arrive merges
  __threadfence();
  __syncthreads();
  if (threadIdx.x < 2) {
    // 0: the list that began before this CTA, 1: the one that begins here and goes on
    sh.last[threadIdx.x] = 0;
    const int want = threadIdx.x;
    for (int s = 0; s < 2 * W; ++s) {
      if (sh.list[s] < 0 || sh.flags[s] == 0 || (sh.flags[s] & 1 ? 0 : 1) != want) continue;
      auto cta_of = [&](long long x) { return (int)((((x + 1) * units - 1) / total) / W); };
      const int cf = cta_of(sh.gs[s]), cl = cta_of(sh.ge[s] - 1);
      sh.cf[want] = cf;
      sh.cl[want] = cl;
      sh.gi[want] = sh.list[s];
      if (atomicAdd(p.arrivals + cf, 1u) == (uint32_t)(cl - cf)) {
        p.arrivals[cf] = 0u;  // zero again for the next call
        sh.last[want] = 1;
      }
      break;
    }
    __threadfence();
  }
  __syncthreads();
#pragma unroll 1
  for (int want = 0; want < 2; ++want) {
    if (!sh.last[want]) continue;
    const int cf = sh.cf[want], n = sh.cl[want] - cf + 1;
    size_t head;
    int nh;
    kv8_heads(p, sh.gi[want], head, nh);
    // each warp takes every W-th CTA, then a warp takes a head
    if (warp < n) {
      for (int j = 0; j < nh; ++j) {
        float M = -INFINITY, L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = warp; i < n; i += W) {
          const float* pt =
              p.partial + ((size_t)(2 * (cf + i) + (i == 0 ? 1 : 0)) * p.heads + j) * kPartialStride;
          const float2 ml = __ldcg(reinterpret_cast<const float2*>(pt));
          kv8_take(M, L, acc, ml.x, ml.y, __ldcg(reinterpret_cast<const float4*>(pt + 4) + lane));
        }
        float* w = part_at(2 * warp + 1) + j * kPartialStride;
        if (lane == 0) *reinterpret_cast<float2*>(w) = make_float2(M, L);
        *reinterpret_cast<float4*>(w + 4 + 4 * lane) = acc;
      }
    }
    __syncthreads();
    for (int j = warp; j < nh; j += W) {
      float M = -INFINITY, L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < min(W, n); ++w) {
        const float* pt = part_at(2 * w + 1) + j * kPartialStride;
        kv8_take(M, L, acc, pt[0], pt[1], *reinterpret_cast<const float4*>(pt + 4 + 4 * lane));
      }
      kv8_write(p, head + j, lane, M, L, acc);
    }
    __syncthreads();
  }
}

}  // namespace ds

// Quantising append: new K and V rows into their pages of the 8-bit cache.
//
// Per page, KV head and K or V: a = max |x| over the new rows, s = max(a/qmax,
// 2^-64, the page's old scale when it holds earlier rows), code = round(x/s);
// where s grew, the earlier rows are rounded again by s0/s.  1/s, the products
// and the scales are fp32 (a bf16 value has 8 significant bits, so the product
// decides the code to 2^-23 of it; a code's own rounding is 2^-8 (int8 at full
// scale) or 2^-4 (e4m3)).
//
// A run: the call's tokens that follow one another in one page.  It begins
// where a slot does not follow the one before it, or at a page's first slot,
// so the slots alone tell the runs.
//
// HBM-bound: 256 B read and 128 B written a row of long runs, a chain of
// dependent loads for single tokens; the two have a kernel each.  Measured on
// B200: 20480 prompt tokens of 32 KV heads with 16 label channels 101 us, 5190
// GB/s of the bytes it cannot do without (79% of a copy's rate; 50 M
// instructions at half the issue rate, rows waited for the rest); one token
// of 256 sequences, 8 KV heads, 4.5 us.  max_new chooses one kernel for all runs
// of a call: 255 single tokens beside a prompt of 512 (8 KV heads) take 70 us by
// the kernel of long runs, whose CTAs take a block's short runs in series, and 19
// by the other; 31 beside one of 4096 take 23 by either, 32 KV heads 40 and 61.
#pragma once

#include "attend_group.cuh"
#include "common.cuh"

namespace ds {

constexpr float kKv8MinScale = 5.421010862427522e-20f;  // 2^-64
// New tokens of a sequence up to which every run is a warp's.  A warp a run and
// a CTA a block took 5.0 and 28.7 us for 64 sequences of 16 new tokens (8 KV
// heads, pages of 64), 10.1 and 18.3 for 32 tokens, 15.5 and 10.4 for 16
// sequences of 64.
constexpr int kKv8ShortRun = 32;
constexpr int kKv8WarpRows = 4;  // rows of a run that a warp takes beside longer ones

struct Kv8AppendParams {
  const uint16_t* K;  // [N, Hkv, 128], `stride` elements a token
  const uint16_t* V;
  long long stride;
  uint8_t* KV;        // [P, Hkv, p, 2, 128]
  float* scales;      // [P, Hkv, 2]
  const int32_t* slots;
  const int32_t* cu;
  const int32_t* C;   // label channels [Hq, r], null: no labels
  uint16_t* label;    // [B, Hq, T_cap, r]
  const int32_t* lens;
  int N, B, Hq, Hkv, P, shift, T_cap, r;
};

// Four products to four codes.  kClamp: int8 products may be beyond +-127.
template <bool kE4m3, bool kClamp>
__device__ __forceinline__ uint32_t kv8_round(const float (&y)[4]) {
  if constexpr (kE4m3) {
    uint16_t c[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
          : "=h"(c[j])
          : "f"(y[2 * j + 1]), "f"(y[2 * j]));
    return c[0] | (uint32_t)c[1] << 16;
  } else {
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = kClamp ? fminf(fmaxf(y[j], -127.f), 127.f) : y[j];
      c[j] = __float_as_uint(__fadd_rn(v, 12582912.f));
    }
    return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
  }
}

// Eight bf16 values (packed in d) to eight codes.  int8: the product is at most
// 127 (1 + 2^-22), as inv is the reciprocal of a scale >= a/127, so adding 1.5
// * 2^23 rounds it to a whole number whose low byte is the code.  kOdd: there
// may be infinities and NaN.
template <bool kE4m3, bool kOdd>
__device__ __forceinline__ uint2 kv8_codes(const uint4& d, float inv) {
  const uint32_t in[4] = {d.x, d.y, d.z, d.w};
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float y[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float a = bf_lo(in[2 * h + j]), b = bf_hi(in[2 * h + j]);
      if (kOdd) {
        a = a != a ? 0.f : a;
        b = b != b ? 0.f : b;
      }
      y[2 * j] = __fmul_rn(a, inv);
      y[2 * j + 1] = __fmul_rn(b, inv);
    }
    w[h] = kv8_round<kE4m3, kOdd>(y);
  }
  return make_uint2(w[0], w[1]);
}

// The value of a code.
template <bool kE4m3>
__device__ __forceinline__ float kv8_value(uint32_t c) {
  if constexpr (kE4m3) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
    float f;
    asm("{.reg .b16 l, u; mov.b32 {l, u}, %1; cvt.f32.f16 %0, l;}" : "=f"(f) : "r"(h));
    return f;
  } else {
    return (float)(int8_t)c;
  }
}

// Four codes rounded again by f < 1 (an infinity or NaN of a foreign code included).
template <bool kE4m3>
__device__ __forceinline__ uint32_t kv8_again(uint32_t c, float f) {
  float y[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) y[j] = __fmul_rn(kv8_value<kE4m3>((c >> (8 * j)) & 255u), f);
  return kv8_round<kE4m3, true>(y);
}

// Largest magnitude of bf16 pairs so far and of 8 more values, as bf16 bits:
// 0x7f80 an infinity, above it NaN (signs are left over).
__device__ __forceinline__ uint32_t kv8_max8(uint32_t m, const uint4& d) {
  const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[j]));
  return m;
}
__device__ __forceinline__ uint32_t kv8_max_half(uint32_t m) {
  return max(m & 0x7fffu, (m >> 16) & 0x7fffu);
}
// The same without infinities and NaN.
__device__ __forceinline__ uint32_t kv8_max8_finite(uint32_t m, const uint4& d) {
  const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = w[j] & 0x7fffu, hi = (w[j] >> 16) & 0x7fffu;
    m = max(m, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
  }
  return m;
}

// The scale a page needs for values up to mx (bf16 bits).
template <bool kE4m3>
__device__ __forceinline__ float kv8_scale(uint32_t mx) {
  constexpr float kQmax = kE4m3 ? 448.f : 127.f;
  return fmaxf(__fdiv_rn(__uint_as_float(mx << 16), kQmax), kKv8MinScale);
}

// Sequence of token i: the last whose first token is not behind i.  By a whole
// warp: 32 places of cu at a time.
__device__ __forceinline__ int kv8_sequence(const Kv8AppendParams& p, int i) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5, at = lo + (lane + 1) * step;
    const uint32_t le = __ballot_sync(0xffffffffu, at < hi && __ldg(p.cu + at) <= i);
    lo += __popc(le) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// Its position in sequence b, -1: it is not one of its tokens.  Reads lens, which
// is there with labels alone.
__device__ __forceinline__ int kv8_position(const Kv8AppendParams& p, int i, int b) {
  const int first = __ldg(p.cu + b);
  return first <= i && i < __ldg(p.cu + b + 1) ? __ldg(p.lens + b) + (i - first) : -1;
}

// Whether the run of token i at `slot` is refused, since another run of the same
// page may be on its way: its page is that of the token before, or it begins
// inside a page and is no sequence's first.  So the runs of a sequence are the
// first and others at the starts of pages.  begins: known to be a sequence's
// first.  By a whole warp.
__device__ __forceinline__ bool kv8_stray(const Kv8AppendParams& p, int i, int slot, bool begins) {
  if (i == 0) return false;
  const int prev = __ldg(p.slots + i - 1);
  if (prev < 0 || (prev >> p.shift) != (slot >> p.shift)) {
    if (begins || (slot & ((1 << p.shift) - 1)) == 0) return false;
    if (__ldg(p.cu + kv8_sequence(p, i)) == i) return false;
  }
  if ((threadIdx.x & 31) == 0) flag_status(8u);
  return true;
}

// Label rows of a run's K rows (value(row, channel)) from position t0 of
// sequence b on, by `threads` threads.
template <class Value>
__device__ __forceinline__ void kv8_labels(const Kv8AppendParams& p, int b, int t0, int n, int g,
                                           int thread, int threads, Value value) {
  if (t0 < 0) {
    if (thread == 0) flag_status(16u);
    return;
  }
  const int G = p.Hq / p.Hkv, rows = min(n, p.T_cap - t0);
  if (rows < n && thread == 0) flag_status(16u);
  auto channel = [&](int h, int j) {
    int ch = __ldg(p.C + h * p.r + j);
    if (ch < 0 || ch >= kHeadDim) {
      flag_status(1u);
      ch &= kHeadDim - 1;
    }
    return ch;
  };
  const int row1 = threads / p.r, j1 = threads - row1 * p.r;  // a thread's step
  const int row0 = thread / p.r, j0 = thread - row0 * p.r;
  for (int h = g * G; h < (g + 1) * G; ++h) {
    uint16_t* out = p.label + (((size_t)b * p.Hq + h) * p.T_cap + t0) * p.r;
    if (j1 == 0) {  // a thread's channel stays
      if (row0 >= rows) continue;
      const int ch = channel(h, j0);
#pragma unroll 4
      for (int row = row0; row < rows; row += row1) out[row * p.r + j0] = value(row, ch);
      continue;
    }
    for (int row = row0, j = j0; row < rows;) {
      out[row * p.r + j] = value(row, channel(h, j));
      row += row1;
      j += j1;
      if (j >= p.r) j -= p.r, ++row;
    }
  }
}

// A run by one warp: n rows of token i on, at `slot`.  kHeld: pairs of rows
// held between the maximum and the codes (more are read twice); kF: loads of
// 4 earlier rows on their way at a time.  refused() is looked up while the rows
// are on their way.
template <bool kE4m3, int kHeld, int kF, class Refused>
__device__ __forceinline__ void kv8_run_warp(const Kv8AppendParams& p, int i, int n, int slot,
                                             int g, int kv, Refused refused) {
  const int lane = threadIdx.x & 31, half = lane >> 4, ch = lane & 15;
  const int pg = slot >> p.shift, off = slot & ((1 << p.shift) - 1);
  if (pg >= p.P) {
    if (lane == 0) flag_status(8u);
    return;
  }
  const uint16_t* src = (kv ? p.V : p.K) + (size_t)i * p.stride + (size_t)g * kHeadDim;
  const size_t tile = (size_t)pg * p.Hkv + g;
  uint8_t* rows = p.KV + (tile << p.shift) * (2 * kHeadDim) + kv * kHeadDim;
  float* sc = p.scales + tile * 2 + kv;
  const float s0 = off > 0 ? *sc : 0.f;
  auto load = [&](int r) {
    return r < n ? ldg_stream(src + (size_t)r * p.stride + ch * 8) : make_uint4(0, 0, 0, 0);
  };
  uint4 d[kHeld];
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < kHeld; ++e) d[e] = load(2 * e + half);
  if (refused()) return;
#pragma unroll
  for (int e = 0; e < kHeld; ++e) m = kv8_max8(m, d[e]);
  for (int r = 2 * kHeld; r < n; r += 2) m = kv8_max8(m, load(r + half));
  uint32_t mx = __reduce_max_sync(0xffffffffu, kv8_max_half(m));
  const bool odd = mx >= 0x7f80u;
  if (odd) {
    if (lane == 0) flag_status(64u);
    m = 0;
    for (int r = 0; r < n; r += 2) m = kv8_max8_finite(m, load(r + half));
    mx = __reduce_max_sync(0xffffffffu, m);
  }
  float s = kv8_scale<kE4m3>(mx);
  if (s0 >= s) {
    s = s0;
  } else if (off > 0) {
    // the scale grew: the earlier rows are rounded again
    const float f = __fdiv_rn(s0, s);
    const int sub = lane >> 3;
    for (int r0 = 0; r0 < off; r0 += 4 * kF) {
      uint4 c[kF];
#pragma unroll
      for (int e = 0; e < kF; ++e) {
        const int r = r0 + 4 * e + sub;
        if (r < off)
          c[e] = *reinterpret_cast<const uint4*>(rows + (size_t)r * 256 + (lane & 7) * 16);
      }
#pragma unroll
      for (int e = 0; e < kF; ++e) {
        const int r = r0 + 4 * e + sub;
        if (r < off)
          *reinterpret_cast<uint4*>(rows + (size_t)r * 256 + (lane & 7) * 16) =
              make_uint4(kv8_again<kE4m3>(c[e].x, f), kv8_again<kE4m3>(c[e].y, f),
                         kv8_again<kE4m3>(c[e].z, f), kv8_again<kE4m3>(c[e].w, f));
      }
    }
  }
  if (lane == 0) *sc = s;
  const float inv = __fdiv_rn(1.f, s);
  auto store = [&](int r, const uint4& v) {
    if (r < n)
      *reinterpret_cast<uint2*>(rows + (size_t)(off + r) * 256 + ch * 8) =
          odd ? kv8_codes<kE4m3, true>(v, inv) : kv8_codes<kE4m3, false>(v, inv);
  };
#pragma unroll
  for (int e = 0; e < kHeld; ++e) store(2 * e + half, d[e]);
  for (int r = 2 * kHeld; r < n; r += 2) store(r + half, load(r + half));
  if (p.label != nullptr && kv == 0) {
    const int b = kv8_sequence(p, i);
    kv8_labels(p, b, kv8_position(p, i, b), n, g, lane, 32,
               [&](int r, int c) { return __ldg(src + (size_t)r * p.stride + c); });
  }
}

// Counts that are not an ascending sequence within [0, N], by the first CTA.
__device__ __forceinline__ void kv8_check_counts(const Kv8AppendParams& p, int threads) {
  if (blockIdx.x != 0) return;
  for (int b = threadIdx.x; b < p.B; b += threads) {
    const int a = __ldg(p.cu + b), z = __ldg(p.cu + b + 1);
    if (a < 0 || z < a || z > p.N) flag_status(16u);
  }
}

// Short runs: a warp for each (window of tokens, KV head, K or V), and the runs
// that begin in its window.  What a step of single tokens costs is the chain
// slot -> scale and row -> codes, so there a window is one token; where
// sequences have more the window is as long (up to 8), so that few warps find
// nothing to do (256 sequences of 9: 13.6 us with windows of 1, 8.3 of 8).
// kHeld: pairs of rows a warp holds, 4 where no run has more than 8 rows (single
// tokens of 256 sequences: 4.5 us, with 8 pairs 5.2), else 8 (64 sequences of
// 32: 10.1 us, with 4 pairs 12.4).
// grid: ceil(ceil(N / window) * Hkv * 2 / 4) CTAs of 128 threads
template <bool kE4m3, int kHeld>
__global__ void __launch_bounds__(128) k_kv8_append_short(const Kv8AppendParams p, int window) {
  kv8_check_counts(p, 128);
  const int item = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int kv = item & 1, u = item >> 1, w = u / p.Hkv, g = u - w * p.Hkv;
  const long long i64 = (long long)w * window;
  if (i64 >= p.N) return;
  const int i0 = (int)i64;
  const int page = 1 << p.shift;
  // token t goes on with the run of the one before
  auto goes_on = [&](long long t, int& slot) {
    slot = t < p.N ? __ldg(p.slots + t) : -1;
    const int prev = t > 0 && t < p.N ? __ldg(p.slots + t - 1) : -1;
    return slot >= 0 && prev >= 0 && slot == prev + 1 && (slot & (page - 1)) != 0;
  };
  // In a step of single tokens cu[i] = i, which tells that a token is a sequence's
  // first without a search after its slot (256 sequences: 4.3 us, by search 4.8).
  const int single = i0 + lane < p.B ? __ldg(p.cu + i0 + lane) : -1;
  int slot;
  const bool go = goes_on((long long)i0 + lane, slot);
  const uint32_t on = __ballot_sync(0xffffffffu, go);
  const uint32_t singles = __ballot_sync(0xffffffffu, single == i0 + lane);
  uint32_t starts = __ballot_sync(0xffffffffu, slot >= 0 && !go && lane < window);
  while (starts) {
    const int s = __ffs(starts) - 1;  // below 8
    starts &= starts - 1;
    int n = __ffs(~(on >> (s + 1)));
    if (n > 31 - s) {  // to the end of the 32 tokens seen
      n = 32 - s;
      for (long long t = (long long)i0 + 32;; t += 32) {
        int other;
        const uint32_t m = __ballot_sync(0xffffffffu, goes_on(t + lane, other));
        n += m == 0xffffffffu ? 32 : __ffs(~m) - 1;
        if (m != 0xffffffffu) break;
      }
    }
    const int first = __shfl_sync(0xffffffffu, slot, s);
    kv8_run_warp<kE4m3, kHeld, 8>(p, i0 + s, n, first, g, kv, [&] {
      return kv8_stray(p, i0 + s, first, (singles >> s & 1u) != 0);
    });
  }
}

// Long runs.  An item is a block of a page's number of tokens, a KV head and K
// or V, with the runs that begin in the block: one, but where sequences meet.
// A CTA takes groups of kGroup items, which share a block for the most part, so
// that the block's slots are looked at once a group, and the rows of the next
// two items are on their way (cp.async) while one is rounded.  Runs of up to
// kKv8WarpRows rows beside others are a warp's.  The groups go round the CTAs:
// a block with many runs takes longer, and its items are not one CTA's.
template <int kPage>
struct Kv8Append {
  static constexpr int kThreads = kPage < 64 ? 64 : 2 * kPage;
  static constexpr int kChunks = kPage * 16 / kThreads;  // 16-byte pieces a thread holds
  static constexpr int kStages = 3;
  static constexpr int kTile = kPage * kHeadDim * 2;
  static constexpr int kSmem = kStages * kTile;
  static constexpr int kCtas = kPage < 64 ? 8 : 256 / kPage;  // an SM's: 16 warps
  static constexpr int kGroup = 4;
};

template <bool kE4m3, int kPage>
__global__ void __launch_bounds__(Kv8Append<kPage>::kThreads, Kv8Append<kPage>::kCtas)
k_kv8_append(const Kv8AppendParams p, int items) {
  using C = Kv8Append<kPage>;
  constexpr int T = C::kThreads, kWarps = T / 32, kStep = T / 16;
  extern __shared__ __align__(128) unsigned char kv8_stage[];
  __shared__ uint32_t on[2 * kPage / 32];  // token goes on with the run of the one before
  __shared__ int first[kPage];             // tokens of the block that begin a run
  __shared__ int runs;
  __shared__ uint32_t red[2][kWarps];
  kv8_check_counts(p, T);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = threadIdx.x >> 4, ch = threadIdx.x & 15;  // pieces of rows row0 + m * kStep
  const int per_block = p.Hkv * 2;
  for (int group = blockIdx.x; group * C::kGroup < items; group += gridDim.x) {
    for (int it = group * C::kGroup, z = min(items, it + C::kGroup); it < z;) {
      // ---- the block and its runs
      const int blk = it / per_block, base = blk * kPage;
      const int end = min(z, (blk + 1) * per_block);
      __syncthreads();  // the block before is done with
      if (threadIdx.x == 0) runs = 0;
      __syncthreads();
      for (int t = threadIdx.x; t < 2 * kPage; t += T) {
        const int i = base + t;
        const int slot = i < p.N ? __ldg(p.slots + i) : -1;
        const int prev = i > 0 && i < p.N ? __ldg(p.slots + i - 1) : -1;
        const bool go = slot >= 0 && prev >= 0 && slot == prev + 1 && (slot & (kPage - 1)) != 0;
        const uint32_t m = __ballot_sync(0xffffffffu, go);
        if ((t & 31) == 0) on[t >> 5] = m;
        if (t < kPage && slot >= 0 && !go) first[atomicAdd(&runs, 1)] = i;
      }
      __syncthreads();
      // rows of the run that begins with token i
      auto length = [&](int i) {
        int t = i - base + 1, n = 1;
        for (;;) {  // ends within kPage tokens, at a page's end at the latest
          if (t >= 2 * kPage) return n;
          const uint32_t w = ~(on[t >> 5] >> (t & 31));
          const int k = min(w ? __ffs(w) - 1 : 32, 32 - (t & 31));
          n += k;
          t += k;
          if ((t & 31) != 0 || k == 0) return n;
        }
      };
      const int nruns = runs;
      if (nruns > 1) {
        for (int e = warp; e < nruns; e += kWarps) {
          const int i = first[e], n = length(i);
          if (n > kKv8WarpRows) continue;
          const int slot = __ldg(p.slots + i);
          if (kv8_stray(p, i, slot, false)) continue;
          for (int x = it; x < end; ++x)
            kv8_run_warp<kE4m3, kKv8WarpRows / 2, 2>(p, i, n, slot, (x - blk * per_block) >> 1,
                                                     x & 1, [] { return false; });
        }
      }
      for (int run = 0; run < nruns; ++run) {
        const int i = first[run], n = length(i), slot = __ldg(p.slots + i);
        if (nruns > 1 && n <= kKv8WarpRows) continue;
        const int pg = slot >> p.shift, off = slot & (kPage - 1);
        if (pg >= p.P || kv8_stray(p, i, slot, false)) {
          if (pg >= p.P && threadIdx.x == 0) flag_status(8u);
          continue;
        }
        __syncthreads();  // the stages and maxima of the run before are read
        int seq = 0, t0 = -1;
        if (p.label != nullptr) {
          seq = kv8_sequence(p, i);
          t0 = kv8_position(p, i, seq);
        }

        // ---- its items
        auto scale_at = [&](int x) {
          const int g = (x - blk * per_block) >> 1;
          return p.scales + ((size_t)pg * p.Hkv + g) * 2 + (x & 1);
        };
        auto issue = [&](int x) {
          if (x < end) {
            const int g = (x - blk * per_block) >> 1;
            const uint16_t* q = ((x & 1) ? p.V : p.K) + (size_t)(i + row0) * p.stride +
                                (size_t)g * kHeadDim + ch * 8;
            const size_t step = (size_t)kStep * p.stride;
            unsigned char* to = kv8_stage + (x - it) % C::kStages * C::kTile + threadIdx.x * 16;
#pragma unroll
            for (int m = 0; m < C::kChunks; ++m, q += step)
              cp_async16_zfill(to + m * (T * 16), q, row0 + m * kStep < n);
          }
          cp_async_commit();
        };
        issue(it);
        issue(it + 1);
        float s_old = off > 0 ? *scale_at(it) : 0.f;
        for (int x = it; x < end; ++x) {
          const int g = (x - blk * per_block) >> 1, kv = x & 1;
          cp_async_wait<1>();
          const unsigned char* from = kv8_stage + (x - it) % C::kStages * C::kTile;
          uint4 d[C::kChunks];
          uint32_t m2 = 0;
#pragma unroll
          for (int m = 0; m < C::kChunks; ++m)
            d[m] = *reinterpret_cast<const uint4*>(from + threadIdx.x * 16 + m * (T * 16));
#pragma unroll
          for (int m = 0; m < C::kChunks; ++m) m2 = kv8_max8(m2, d[m]);
          auto block_max = [&](uint32_t v) {
            v = __reduce_max_sync(0xffffffffu, v);
            if (lane == 0) red[x & 1][warp] = v;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v = max(v, red[x & 1][w]);
            return v;
          };
          uint32_t mx = block_max(kv8_max_half(m2));
          // every thread is done with the item before, so its stage may be filled
          issue(x + 2);
          const float s0 = s_old;
          if (off > 0 && x + 1 < end) s_old = *scale_at(x + 1);
          const bool odd = mx >= 0x7f80u;
          if (odd) {
            if (threadIdx.x == 0) flag_status(64u);
            m2 = 0;
#pragma unroll
            for (int m = 0; m < C::kChunks; ++m) m2 = kv8_max8_finite(m2, d[m]);
            __syncthreads();  // red is read
            mx = block_max(m2);
          }
          const size_t tile = (size_t)pg * p.Hkv + g;
          uint8_t* rows = p.KV + (tile << p.shift) * (2 * kHeadDim) + kv * kHeadDim;
          float s = kv8_scale<kE4m3>(mx);
          if (s0 >= s) {
            s = s0;
          } else if (off > 0) {
            // the scale grew: the earlier rows are rounded again
            const float f = __fdiv_rn(s0, s);
            constexpr int kF = 4;
            for (int c0 = threadIdx.x; c0 < off * 8; c0 += kF * T) {
              uint4 c[kF];
#pragma unroll
              for (int e = 0; e < kF; ++e) {
                const int y = c0 + e * T;
                if (y < off * 8)
                  c[e] = *reinterpret_cast<const uint4*>(rows + (size_t)(y >> 3) * 256 +
                                                         (y & 7) * 16);
              }
#pragma unroll
              for (int e = 0; e < kF; ++e) {
                const int y = c0 + e * T;
                if (y < off * 8)
                  *reinterpret_cast<uint4*>(rows + (size_t)(y >> 3) * 256 + (y & 7) * 16) =
                      make_uint4(kv8_again<kE4m3>(c[e].x, f), kv8_again<kE4m3>(c[e].y, f),
                                 kv8_again<kE4m3>(c[e].z, f), kv8_again<kE4m3>(c[e].w, f));
              }
            }
          }
          if (threadIdx.x == 0) *scale_at(x) = s;
          const float inv = __fdiv_rn(1.f, s);
          uint8_t* to = rows + (size_t)(off + row0) * 256 + ch * 8;
          if (odd) {
#pragma unroll
            for (int m = 0; m < C::kChunks; ++m)
              if (row0 + m * kStep < n)
                *reinterpret_cast<uint2*>(to + m * (kStep * 256)) =
                    kv8_codes<kE4m3, true>(d[m], inv);
          } else if (n == kPage) {
#pragma unroll
            for (int m = 0; m < C::kChunks; ++m)
              *reinterpret_cast<uint2*>(to + m * (kStep * 256)) =
                  kv8_codes<kE4m3, false>(d[m], inv);
          } else {
#pragma unroll
            for (int m = 0; m < C::kChunks; ++m)
              if (row0 + m * kStep < n)
                *reinterpret_cast<uint2*>(to + m * (kStep * 256)) =
                    kv8_codes<kE4m3, false>(d[m], inv);
          }
          if (p.label != nullptr && kv == 0)
            kv8_labels(p, seq, t0, n, g, threadIdx.x, T, [&](int r, int c) {
              return reinterpret_cast<const uint16_t*>(from)[r * kHeadDim + c];
            });
        }
        cp_async_wait<0>();
      }
      it = end;
    }
  }
}

}  // namespace ds

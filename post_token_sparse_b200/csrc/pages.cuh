// Page tables and slot maps of the paged cache, from request lengths.
//
//   cu[b] = sum n_new,  e[b] = sum need,  need = ceil((len+n)/p) - ceil(len/p)
// over the sequences before b; token i of sequence b sits at pos = len + i -
// cu[b], on a page it already holds or on free_pages[n_free-1-e-j].
//
// What it has to move is a few bytes a sequence and four a token, so the time
// is the launch, two dependent loads and the prefix sums.  The sums are
// therefore recomputed by every CTA (no second launch, no waiting between
// CTAs): tiles of kPageTile sequences, four a thread, one block scan; a CTA
// then writes its kPageTok slots, each token finding its sequence by a binary
// search of the tile's sums in shared memory.  The first token on a page
// writes the table entry, so pages need no work list of their own.
//
// Measured (B200, device time of a launch): 3.3 us for one token of 192
// sequences, 6.5 us for 590K slots of 48 prompts, 4.5 us for the pages of 10
// of 192 requests, 6.3 us for 470K pages of 1024 requests.
#pragma once

#include "common.cuh"

namespace ds {

constexpr int kPageThreads = 256;
constexpr int kPageTile = 4 * kPageThreads;  // sequences per scan
constexpr int kPageTok = 2048;               // slots (or released pages) per CTA

struct PageParams {
  const int32_t* lens;
  const int32_t* n_new;   // assign
  const int32_t* done;    // release
  int32_t* table;         // [B, W]
  int32_t* free_pages;    // [P]
  const int32_t* n_free;
  int32_t* lens_out;
  int32_t* n_free_out;
  int32_t* cu_new;
  int32_t* slots;
  int B, W, P, N;
  int shift;              // log2 of the tokens a page
};

struct PageShared {
  unsigned long long wsum[2][kPageThreads / 32];
  int32_t cu[kPageTile];   // first token (assign) or page (release) of a sequence
  int32_t e[kPageTile];    // its first new page
  int32_t len[kPageTile];  // its length, -1: refused
};

// Exclusive prefix of two counts over the CTA's threads, and the totals.
__device__ __forceinline__ void page_scan(PageShared& sh, unsigned long long& a,
                                          unsigned long long& b, unsigned long long& ta,
                                          unsigned long long& tb) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long xa = a, xb = b;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned long long ya = __shfl_up_sync(0xffffffffu, xa, d);
    const unsigned long long yb = __shfl_up_sync(0xffffffffu, xb, d);
    if (lane >= d) xa += ya, xb += yb;
  }
  __syncthreads();  // the previous tile's readers are done
  if (lane == 31) sh.wsum[0][warp] = xa, sh.wsum[1][warp] = xb;
  __syncthreads();
  unsigned long long pa = 0, pb = 0;
  ta = tb = 0;
#pragma unroll
  for (int w = 0; w < kPageThreads / 32; ++w) {
    if (w == warp) pa = ta, pb = tb;
    ta += sh.wsum[0][w];
    tb += sh.wsum[1][w];
  }
  a = pa + xa - a;
  b = pb + xb - b;
}

// Largest s in [0, n) with first[s] <= i[e] (first[0] <= i[e]), for kIlp places
// side by side: a search is log2(n) dependent shared-memory loads, ten for a full
// tile of sequences.
constexpr int kPageIlp = 4;  // 590K slots: 6.9 us, one at a time 8.3
template <int kIlp>
__device__ __forceinline__ void page_find(const int32_t* first, int n, const int (&i)[kIlp],
                                          int (&s)[kIlp]) {
#pragma unroll
  for (int e = 0; e < kIlp; ++e) s[e] = 0;
  for (int step = kPageTile / 2; step > 0; step >>= 1) {
    if (step >= n) continue;
#pragma unroll
    for (int e = 0; e < kIlp; ++e)
      if (s[e] + step < n && first[s[e] + step] <= i[e]) s[e] += step;
  }
}

// n_free as stored, cut to [0, P].
__device__ __forceinline__ int page_free_count(const PageParams& p) {
  const int f = __ldg(p.n_free);
  if (f >= 0 && f <= p.P) return f;
  if (blockIdx.x == 0 && threadIdx.x == 0) flag_status(16u);
  return f < 0 ? 0 : p.P;
}

// Slots [a, z) of the nb sequences from `base` on that sh describes.
template <int kIlp>
__device__ __forceinline__ void page_slots(const PageParams& p, const PageShared& sh, int base,
                                           int nb, int nf, int a, int z) {
  const int mask = (1 << p.shift) - 1;
  for (int i0 = a + threadIdx.x; i0 < z; i0 += kIlp * kPageThreads) {
    int i[kIlp], s[kIlp], pos[kIlp], id[kIlp];
    bool fresh[kIlp];
#pragma unroll
    for (int e = 0; e < kIlp; ++e) i[e] = min(i0 + e * kPageThreads, z - 1);
    page_find(sh.cu, nb, i, s);
#pragma unroll
    for (int e = 0; e < kIlp; ++e) {
      const int l = sh.len[s[e]];
      pos[e] = l < 0 ? -1 : l + i[e] - sh.cu[s[e]];
      id[e] = -1;
      fresh[e] = false;
      if (pos[e] >= 0) {
        const int j = pos[e] >> p.shift, have = (l + mask) >> p.shift;
        fresh[e] = j >= have;
        id[e] = fresh[e] ? __ldg(p.free_pages + (nf - 1 - sh.e[s[e]] - (j - have)))
                         : p.table[(size_t)(base + s[e]) * p.W + j];
      }
    }
#pragma unroll
    for (int e = 0; e < kIlp; ++e) {
      if (i0 + e * kPageThreads >= z) break;
      if (pos[e] >= 0 && (id[e] < 0 || id[e] >= p.P)) {
        flag_status(8u);
        id[e] = -1;
      }
      if (fresh[e] && (pos[e] & mask) == 0)
        p.table[(size_t)(base + s[e]) * p.W + (pos[e] >> p.shift)] = id[e];
      p.slots[i[e]] = id[e] >= 0 ? (id[e] << p.shift) + (pos[e] & mask) : -1;
    }
  }
}

// grid: max(1, ceil(N / kPageTok)) CTAs of kPageThreads
__global__ void __launch_bounds__(kPageThreads) k_page_assign(const PageParams p) {
  __shared__ PageShared sh;
  const int mask = (1 << p.shift) - 1;
  const int nf = page_free_count(p);
  const int i0 = blockIdx.x * kPageTok, i1 = min(i0 + kPageTok, p.N);
  const bool lead = blockIdx.x == 0;
  unsigned long long c_tok = 0, c_pg = 0;  // totals of the tiles before
  int used = 0;                            // pages given so far, by this thread's sequences
  for (int base = 0; base < p.B; base += kPageTile) {
    int len[4], n[4], need[4];
    bool fits[4];
    unsigned long long tok = 0, pg = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int b = base + threadIdx.x * 4 + j;
      len[j] = b < p.B ? __ldg(p.lens + b) : 0;
      n[j] = b < p.B ? __ldg(p.n_new + b) : 0;
      const long long end = (long long)len[j] + n[j];
      fits[j] = len[j] >= 0 && n[j] >= 0 && end <= (long long)p.W << p.shift;
      need[j] = fits[j] ? (int)((end + mask) >> p.shift) - ((len[j] + mask) >> p.shift) : 0;
      tok += n[j] > 0 ? n[j] : 0;
      pg += need[j];
    }
    unsigned long long t_tok, t_pg;
    page_scan(sh, tok, pg, t_tok, t_pg);
    tok += c_tok;
    pg += c_pg;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int s = threadIdx.x * 4 + j, b = base + s;
      const unsigned long long end = tok + (n[j] > 0 ? n[j] : 0);
      const bool roomy = fits[j] && end <= (unsigned long long)p.N;
      const bool paged = need[j] == 0 || pg + need[j] <= (unsigned long long)nf;
      const bool ok = roomy && paged;
      sh.cu[s] = (int)min(tok, (unsigned long long)p.N);
      sh.e[s] = (int)min(pg, (unsigned long long)nf);
      sh.len[s] = ok ? len[j] : -1;
      if (lead && b < p.B) {
        if (!roomy) flag_status(16u);
        else if (!paged) flag_status(32u);
        p.lens_out[b] = ok ? len[j] + n[j] : len[j];
        p.cu_new[b] = (int)min(tok, 0x7fffffffull);
        if (ok && need[j] > 0) used = max(used, (int)(pg + need[j]));
      }
      tok = end;
      pg += need[j];
    }
    __syncthreads();
    // this CTA's tokens among the tile's
    const int nb = min(kPageTile, p.B - base);
    const unsigned long long hi = c_tok + t_tok;
    const int a = (int)max((unsigned long long)i0, min(c_tok, (unsigned long long)p.N));
    const int z = (int)min((unsigned long long)i1, hi);
    if (z - a <= kPageThreads)
      page_slots<1>(p, sh, base, nb, nf, a, z);
    else
      page_slots<kPageIlp>(p, sh, base, nb, nf, a, z);
    c_tok = hi;
    c_pg += t_pg;
    if (!lead && c_tok >= (unsigned long long)i1) break;
  }
  // slots past the last token
  const int a = (int)max((unsigned long long)i0, min(c_tok, (unsigned long long)p.N));
  for (int i = a + threadIdx.x; i < i1; i += kPageThreads) p.slots[i] = -1;
  if (lead) {
    __syncthreads();
    used = __reduce_max_sync(0xffffffffu, used);
    if ((threadIdx.x & 31) == 0) sh.cu[threadIdx.x >> 5] = used;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kPageThreads / 32; ++w) used = max(used, sh.cu[w]);
      p.n_free_out[0] = nf - used;
      p.cu_new[p.B] = (int)min(c_tok, 0x7fffffffull);
    }
  }
}

// grid: max(1, ceil(min(P, B*W) / kPageTok)) CTAs of kPageThreads
__global__ void __launch_bounds__(kPageThreads) k_page_release(const PageParams p) {
  __shared__ PageShared sh;
  const int mask = (1 << p.shift) - 1;
  const int nf = page_free_count(p);
  const int i0 = blockIdx.x * kPageTok;
  const int room = p.P - nf;  // pages that may come back
  const int i1 = min(i0 + kPageTok, room);
  const bool lead = blockIdx.x == 0;
  unsigned long long c_pg = 0;
  for (int base = 0; base < p.B; base += kPageTile) {
    int cnt[4];
    unsigned long long pg = 0, zero = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int b = base + threadIdx.x * 4 + j;
      cnt[j] = 0;
      if (b < p.B) {
        const int len = __ldg(p.lens + b);
        const bool over = __ldg(p.done + b) != 0;
        if (over) {
          const bool fits = len >= 0 && len <= (long long)p.W << p.shift;
          if (!fits && lead) flag_status(16u);
          cnt[j] = fits ? (len + mask) >> p.shift : len < 0 ? 0 : p.W;
        }
        if (lead) p.lens_out[b] = over ? 0 : len;
      }
      pg += cnt[j];
    }
    unsigned long long t_pg, t_zero;
    page_scan(sh, pg, zero, t_pg, t_zero);
    pg += c_pg;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sh.cu[threadIdx.x * 4 + j] = (int)min(pg, 0x7fffffffull);
      pg += cnt[j];
    }
    __syncthreads();
    const int nb = min(kPageTile, p.B - base);
    const unsigned long long hi = c_pg + t_pg;
    const int a = (int)max((unsigned long long)i0, min(c_pg, (unsigned long long)p.P));
    const int z = (int)min((unsigned long long)max(i1, 0), hi);
    for (int i0 = a + threadIdx.x; i0 < z; i0 += kPageIlp * kPageThreads) {
      int i[kPageIlp], s[kPageIlp], id[kPageIlp];
#pragma unroll
      for (int e = 0; e < kPageIlp; ++e) i[e] = min(i0 + e * kPageThreads, z - 1);
      page_find(sh.cu, nb, i, s);
#pragma unroll
      for (int e = 0; e < kPageIlp; ++e)
        id[e] = __ldg(p.table + (size_t)(base + s[e]) * p.W + (i[e] - sh.cu[s[e]]));
#pragma unroll
      for (int e = 0; e < kPageIlp; ++e) {
        if (i0 + e * kPageThreads >= z) break;
        if (id[e] < 0 || id[e] >= p.P) {
          flag_status(8u);
          id[e] = -1;
        }
        p.free_pages[nf + i[e]] = id[e];
      }
    }
    c_pg = hi;
    if (!lead && c_pg >= (unsigned long long)max(i1, 0)) break;
  }
  if (lead && threadIdx.x == 0) {
    if (c_pg > (unsigned long long)room) flag_status(16u);  // more pages than the pool has
    p.n_free_out[0] = nf + (int)min(c_pg, (unsigned long long)room);
  }
}

}  // namespace ds

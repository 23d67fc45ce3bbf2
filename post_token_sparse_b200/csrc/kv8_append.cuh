// Quantising append: new K and V rows into their pages of the 8-bit cache.
//
// Per page, KV head and K or V: a = max |x| over the new rows, s = max(a/qmax,
// 2^-64, the page's old scale when it holds earlier rows), code = round(x/s);
// where s grew, the earlier rows are rounded again by s0/s.  1/s, the products
// and the scales are fp32 (a bf16 value has 8 significant bits, so the product
// decides the code to 2^-23 of it; a code's own rounding is 2^-8 (int8 at full
// scale) or 2^-4 (e4m3)).
//
// HBM-bound: 256 B read and 128 B written a row.  One CTA per (page of a
// sequence, KV head, K or V) holds the rows in registers between the maximum
// and the quantisation, so that they are read once.
#pragma once

#include "common.cuh"

namespace ds {

constexpr float kKv8MinScale = 5.421010862427522e-20f;  // 2^-64
constexpr int kAppThreads = 128;

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
  int N, B, Hq, Hkv, P, shift, J, T_cap, r;
};

// Eight values to eight codes.
template <bool kE4m3>
__device__ __forceinline__ uint2 kv8_codes(const float (&x)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (kE4m3) {
      uint16_t c[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float lo = __fmul_rn(x[4 * h + 2 * j], inv), hi = __fmul_rn(x[4 * h + 2 * j + 1], inv);
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c[j]) : "f"(hi), "f"(lo));
      }
      w[h] = c[0] | (uint32_t)c[1] << 16;
    } else {
      uint32_t c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float q = fminf(fmaxf(__fmul_rn(x[4 * h + j], inv), -127.f), 127.f);
        c[j] = (uint32_t)__float2int_rn(q);
      }
      w[h] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    }
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

// grid: B * J * Hkv * 2 CTAs (K or V fastest, then head, page, sequence); kChunks: 16-byte pieces a thread holds
template <bool kE4m3, int kChunks>
__global__ void __launch_bounds__(kAppThreads) k_kv8_append(const Kv8AppendParams p) {
  __shared__ uint32_t red[kAppThreads / 32];
  const int kv = blockIdx.x & 1;
  int u = blockIdx.x >> 1;
  const int g = u % p.Hkv;
  u /= p.Hkv;
  const int jp = u % p.J, b = u / p.J;
  const int page = 1 << p.shift;
  const bool lead = kv == 0 && g == 0 && threadIdx.x == 0;

  int i0 = __ldg(p.cu + b), i1 = __ldg(p.cu + b + 1);
  if (i0 < 0 || i1 < i0 || i1 > p.N) {
    if (lead && jp == 0) flag_status(16u);
    i0 = min(max(i0, 0), p.N);
    i1 = min(i1, p.N);
  }
  if (i0 >= i1) return;
  const int first = __ldg(p.slots + i0);
  if (first < 0) return;
  const int off0 = first & (page - 1);
  if (lead && jp == 0 && (long long)(i1 - i0) + off0 > (long long)p.J << p.shift) flag_status(16u);
  // this page's tokens [a, z)
  const long long a64 = jp == 0 ? i0 : (long long)i0 - off0 + ((long long)jp << p.shift);
  if (a64 >= i1) return;
  const int a = (int)a64;
  const int z = (int)min((long long)i1, (long long)i0 - off0 + ((long long)(jp + 1) << p.shift));
  const int slot = jp == 0 ? first : __ldg(p.slots + a);
  const int pg = slot >> p.shift, off = slot & (page - 1);
  if (slot < 0 || pg >= p.P || off != (jp == 0 ? off0 : 0)) {
    if (lead) flag_status(8u);
    return;
  }
  const int n = z - a;

  const uint16_t* src = (kv ? p.V : p.K) + (size_t)a * p.stride + (size_t)g * kHeadDim;
  uint4 d[kChunks];
#pragma unroll
  for (int m = 0; m < kChunks; ++m) {
    const int c = threadIdx.x + m * kAppThreads, row = c >> 4;
    d[m] = row < n ? ldg_stream(src + (size_t)row * p.stride + (c & 15) * 8) : make_uint4(0, 0, 0, 0);
  }
  uint32_t mx = 0;
  bool odd = false;  // an infinity or NaN among the values
#pragma unroll
  for (int m = 0; m < kChunks; ++m) {
    const uint32_t w[4] = {d[m].x, d[m].y, d[m].z, d[m].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = (w[j] << 16) & 0x7fffffffu, hi = w[j] & 0x7fff0000u;
      odd |= lo >= 0x7f800000u || hi >= 0x7f800000u;
      mx = max(mx, max(lo >= 0x7f800000u ? 0u : lo, hi >= 0x7f800000u ? 0u : hi));
    }
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = mx;
  odd = __syncthreads_or(odd);
  if (odd && threadIdx.x == 0) flag_status(64u);
#pragma unroll
  for (int w = 0; w < kAppThreads / 32; ++w) mx = max(mx, red[w]);

  constexpr float kQmax = kE4m3 ? 448.f : 127.f;
  float s = fmaxf(__fdiv_rn(__uint_as_float(mx), kQmax), kKv8MinScale);
  const size_t tile = (size_t)pg * p.Hkv + g;
  uint8_t* rows = p.KV + (tile << p.shift) * (2 * kHeadDim) + kv * kHeadDim;
  float* sc = p.scales + tile * 2 + kv;
  if (off > 0) {
    const float s0 = *sc;
    if (s0 >= s) {
      s = s0;
    } else {
      // the scale grew: the earlier rows are rounded again
      const float f = __fdiv_rn(s0, s);
      for (int c = threadIdx.x; c < off * 16; c += kAppThreads) {
        uint2* q = reinterpret_cast<uint2*>(rows + (size_t)(c >> 4) * (2 * kHeadDim) + (c & 15) * 8);
        const uint2 o = *q;
        float x[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[j] = kv8_value<kE4m3>((o.x >> (8 * j)) & 255u);
          x[4 + j] = kv8_value<kE4m3>((o.y >> (8 * j)) & 255u);
        }
        *q = kv8_codes<kE4m3>(x, f);
      }
    }
    __syncthreads();  // every thread has read the old scale
  }
  if (threadIdx.x == 0) *sc = s;
  const float inv = __fdiv_rn(1.f, s);
#pragma unroll
  for (int m = 0; m < kChunks; ++m) {
    const int c = threadIdx.x + m * kAppThreads, row = c >> 4;
    if (row >= n) break;
    const uint32_t w[4] = {d[m].x, d[m].y, d[m].z, d[m].w};
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = bf_lo(w[j]);
      x[2 * j + 1] = bf_hi(w[j]);
    }
    if (odd) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (x[j] != x[j]) x[j] = 0.f;
    }
    *reinterpret_cast<uint2*>(rows + (size_t)(off + row) * (2 * kHeadDim) + (c & 15) * 8) =
        kv8_codes<kE4m3>(x, inv);
  }

  if (p.label != nullptr && kv == 0) {
    const int G = p.Hq / p.Hkv, t0 = __ldg(p.lens + b) + (a - i0);
    const int per = n * p.r;
    for (int e = threadIdx.x; e < G * per; e += kAppThreads) {
      const int h = g * G + e / per, w = e % per, row = w / p.r, j = w - row * p.r;
      const int t = t0 + row;
      int ch = __ldg(p.C + h * p.r + j);
      if (ch < 0 || ch >= kHeadDim) {
        flag_status(1u);
        ch &= kHeadDim - 1;
      }
      if (t < 0 || t >= p.T_cap) {
        flag_status(16u);
        continue;
      }
      p.label[(((size_t)b * p.Hq + h) * p.T_cap + t) * p.r + j] =
          __ldg(src + (size_t)row * p.stride + ch);
    }
  }
}

}  // namespace ds

// Decode attention over the paged 8-bit cache.
//
//   l_t = scale * sK(t) * (q . kcode_t),  w = softmax(l),
//   O = sum_t w_t sV(t) vcode_t,  lse = log sum_t exp(l_t)
// over every token of a sequence (dense) or over a list of kept tokens.
//
// One CTA per query head; a warp takes every eighth row, a lane four channels
// (one word of K codes, one of V codes), with an online softmax per warp and
// one merge of the warps in shared memory.
#pragma once

#include "common.cuh"
#include "kv8_append.cuh"

namespace ds {

constexpr int kKv8Threads = 256;
constexpr int kKv8Warps = kKv8Threads / 32;

struct Kv8Params {
  const uint16_t* Q;     // [B, Hq, 128]
  const uint8_t* KV;     // [P, Hkv, p, 2, 128]
  const float* scales;   // [P, Hkv, 2]
  const int32_t* table;  // [B, W]
  const int32_t* lens;   // [B]
  const int32_t* idx;    // [B * lists, k] kept tokens, null: dense
  float* O;              // [B, Hq, 128]
  float* lse;            // [B, Hq] or null
  int B, Hq, Hkv, P, W, shift;
  int k;
  int per_list;          // query heads that share a list
  float scale_log2;
};

// grid: B * Hq
template <bool kE4m3>
__global__ void __launch_bounds__(kKv8Threads) k_kv8_attend(const Kv8Params p) {
  __shared__ float sm[kKv8Warps][132];
  const int h = blockIdx.x % p.Hq, b = blockIdx.x / p.Hq, g = h / (p.Hq / p.Hkv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int page = 1 << p.shift;
  int len = __ldg(p.lens + b);
  if (len < 0 || len > (long long)p.W << p.shift) {
    if (threadIdx.x == 0) flag_status(16u);
    len = len < 0 ? 0 : p.W << p.shift;
  }
  const uint2 qw = *reinterpret_cast<const uint2*>(p.Q + (size_t)blockIdx.x * kHeadDim + lane * 4);
  const float q[4] = {bf_lo(qw.x), bf_hi(qw.x), bf_lo(qw.y), bf_hi(qw.y)};
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  const int rows = p.idx ? p.k : len;
  const int32_t* list = p.idx ? p.idx + (size_t)(blockIdx.x / p.per_list) * p.k : nullptr;
  for (int r = warp; r < rows; r += kKv8Warps) {
    int t = r;
    if (list) {
      t = __ldg(list + r);
      if (t < 0 || t >= len) {
        if (t != -1 && lane == 0) flag_status(2u);
        continue;
      }
    }
    const int pg = __ldg(p.table + (size_t)b * p.W + (t >> p.shift));
    if (pg < 0 || pg >= p.P) {
      if (lane == 0) flag_status(8u);
      continue;
    }
    const size_t tile = (size_t)pg * p.Hkv + g;
    const uint32_t* row = reinterpret_cast<const uint32_t*>(
        p.KV + ((tile << p.shift) + (t & (page - 1))) * (2 * kHeadDim));
    const uint32_t kw = __ldg(row + lane), vw = __ldg(row + 32 + lane);
    float x = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) x = fmaf(q[j], kv8_value<kE4m3>((kw >> (8 * j)) & 255u), x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    x *= p.scale_log2 * __ldg(p.scales + tile * 2);
    const float sv = __ldg(p.scales + tile * 2 + 1);
    const float mn = fmaxf(m, x), a = exp2f(m - mn), w = exp2f(x - mn);
    m = mn;
    l = l * a + w;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = o[j] * a + w * sv * kv8_value<kE4m3>((vw >> (8 * j)) & 255u);
  }
  if (lane == 0) sm[warp][0] = m, sm[warp][1] = l;
#pragma unroll
  for (int j = 0; j < 4; ++j) sm[warp][4 + lane * 4 + j] = o[j];
  __syncthreads();
  if (threadIdx.x < kHeadDim) {
    float M = -INFINITY, L = 0.f, acc = 0.f;
    for (int w = 0; w < kKv8Warps; ++w) M = fmaxf(M, sm[w][0]);
    for (int w = 0; w < kKv8Warps; ++w) {
      const float f = sm[w][1] == 0.f ? 0.f : exp2f(sm[w][0] - M);
      L += sm[w][1] * f;
      acc += sm[w][4 + threadIdx.x] * f;
    }
    p.O[(size_t)blockIdx.x * kHeadDim + threadIdx.x] = L == 0.f ? 0.f : acc / L;
    if (p.lse && threadIdx.x == 0)
      p.lse[blockIdx.x] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
  }
}

}  // namespace ds

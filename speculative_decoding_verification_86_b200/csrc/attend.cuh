// Attention of a request's block over its 4-bit cache.
#pragma once
#include "cache.cuh"

namespace sv {

struct AttendParams {
  CacheView c;
  CacheRows q, out;
  const int32_t* cache_len;
  const int32_t* block_len;  // nullptr: T
  int B, T, heads_q, group;  // group: query heads per key/value head
  float scale;
  int causal, window;
  float* lse;  // [B, T, heads_q] or nullptr
  uint32_t* status;
};

// One CTA per query row; thread = token of a tile of 128 for the scores, then
// thread = channel for the values.
template <int D, typename T>
__global__ void __launch_bounds__(128) k_attend(AttendParams p) {
  __shared__ float q[D], pr[128], red[4];
  const int hq = blockIdx.x, j = blockIdx.y, i = blockIdx.z, t = threadIdx.x;
  const int64_t n = __ldg(p.cache_len + i);
  const int L = p.block_len ? min(max(__ldg(p.block_len + i), 0), p.T) : p.T;
  if (n < 0 || n + L > p.c.capacity) {
    if (p.status && hq == 0 && j == 0 && t == 0) atomicOr(p.status + i, kDevBadLength);
    return;
  }
  if (j >= L) return;
  const int h = hq / p.group;
  const T* src = static_cast<const T*>(p.q.data) + i * p.q.sb + j * p.q.st + hq * p.q.sh;
  for (int c = t; c < D; c += 128) q[c] = static_cast<float>(src[c]);
  const int64_t end = p.causal ? n + j + 1 : n + L;
  const int64_t first = p.window ? max(n + j + 1 - p.window, int64_t(0)) : 0;
  const float kx = p.scale * (p.c.k_scale ? __ldg(p.c.k_scale + h) : 1.0f);
  float m = -INFINITY, l = 0.0f, acc[(D + 127) / 128] = {};
  for (int64_t t0 = first & ~int64_t(15); t0 < end; t0 += 128) {
    __syncthreads();
    const int64_t pos = t0 + t;
    float s = -INFINITY;
    bool see = pos >= first && pos < end;
    if (see) {
      const uint8_t* r = cache_run<D>(p.c, i, h, pos >> 4);
      const int tok = static_cast<int>(pos & 15);
      if (!r) {
        if (p.status) atomicOr(p.status + i, kDevBadPage);
      } else {
        float dot = 0.0f;
        for (int g = 0; g < D / 16; ++g) {
          const uint32_t sc = r[run_k_scales(D) + tok * (D / 16) + g];
          const uint32_t s2 = e4m3x2_to_f16x2(sc | (sc << 8));
          for (int u = 0; u < 2; ++u) {
            uint32_t hh[4];
            e2m1x8_to_f16(*reinterpret_cast<const uint32_t*>(r + (g >> 1) * 256 + tok * 16 + (g & 1) * 8 + 4 * u), hh);
            for (int e = 0; e < 4; ++e) {
              const float2 f = h2_to_f2(h2_mul(hh[e], s2));
              dot = fmaf(q[g * 16 + u * 8 + 2 * e], f.x, dot);
              dot = fmaf(q[g * 16 + u * 8 + 2 * e + 1], f.y, dot);
            }
          }
        }
        s = dot * kx;
      }
    }
    float mx = s;
    bool nan = s != s;
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if ((t & 31) == 0) red[t >> 5] = mx;
    nan = __syncthreads_or(nan);
    mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float mn = fmaxf(m, mx), ref = mn == -INFINITY ? 0.0f : mn;
    const float f = expf(m - ref);
    float pe = expf(s - ref);
    pr[t] = pe;
    for (int o = 16; o; o >>= 1) pe += __shfl_xor_sync(0xffffffffu, pe, o);
    __syncthreads();
    if ((t & 31) == 0) red[t >> 5] = pe;
    __syncthreads();
    l = l * f + red[0] + red[1] + red[2] + red[3];
    if (nan) l = NAN;
    m = mn;
    for (int u = 0; u < (D + 127) / 128; ++u) {
      const int c = t + 128 * u;
      if (c >= D) continue;
      float a = acc[u] * f;
      for (int e = 0; e < 128; ++e) {
        const int64_t pe2 = t0 + e;
        if (pe2 < first || pe2 >= end) continue;
        const uint8_t* r = cache_run<D>(p.c, i, h, pe2 >> 4);
        if (!r) continue;
        const int tok = static_cast<int>(pe2 & 15);
        uint32_t b = r[run_v_codes(D) + c * 8 + (tok >> 1)];
        b = tok & 1 ? b >> 4 : b & 15u;
        uint32_t hh[4];
        e2m1x8_to_f16(b, hh);
        const uint32_t sc = r[run_v_scales(D) + (c >> 4) * 16 + tok];
        a = fmaf(pr[e], h2_to_f2(h2_mul(hh[0], e4m3x2_to_f16x2(sc))).x, a);
      }
      acc[u] = a;
    }
  }
  const float vx = p.c.v_scale ? __ldg(p.c.v_scale + h) : 1.0f;
  T* dst = static_cast<T*>(p.out.data) + i * p.out.sb + j * p.out.st + hq * p.out.sh;
  for (int u = 0; u < (D + 127) / 128; ++u) {
    const int c = t + 128 * u;
    if (c < D) dst[c] = static_cast<T>(l == 0.0f ? 0.0f : acc[u] * vx / l);
  }
  if (p.lse && t == 0)
    p.lse[(static_cast<int64_t>(i) * p.T + j) * p.heads_q + hq] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace sv

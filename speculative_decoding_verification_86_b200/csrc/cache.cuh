// The 4-bit block cache: its layout, and the kernels that quantise keys and
// values into it and read them back.
//
// A page holds, per key/value head, runs of 16 tokens.  A run is 18 D bytes
// (D = head_dim): key codes [D/32][16][16 B], key scales [16][D/16], value codes
// [D][8 B], value scales [D/16][16].  The attention gives one thread a token of
// the keys and a channel of the values; in this order its threads read their
// 16 and 8 bytes next to one another, and one copy of 18 D contiguous bytes
// brings a run into shared memory whatever the page size.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

namespace sv {

constexpr uint32_t kDevBadPage = 8u;
constexpr uint32_t kDevInternal = 16u;
constexpr uint32_t kDevBadLength = 32u;
constexpr int kRun = 16;    // tokens of a run
constexpr int kGroup = 16;  // channels that share a scale
constexpr uint32_t kScaleNaN = 0x7fu;  // e4m3

__host__ __device__ constexpr int run_bytes(int D) { return 18 * D; }
__host__ __device__ constexpr int run_k_scales(int D) { return 8 * D; }
__host__ __device__ constexpr int run_v_codes(int D) { return 9 * D; }
__host__ __device__ constexpr int run_v_scales(int D) { return 17 * D; }

// n / d for 0 <= n < 2^31 by a multiplication: with 2^shift >= d and
// mul = floor(2^32 (2^shift - d) / d) + 1 the error of (2^32 + mul) n / 2^32 stays
// below 2^shift / d for such n.  A division by a number that the compiler does not
// know is some 100 cycles.
struct Quotient {
  uint32_t mul = 0;
  int shift = 0;
  Quotient() = default;
  explicit Quotient(uint32_t d) {
    while ((1u << shift) < d) ++shift;
    mul = static_cast<uint32_t>((((uint64_t{1} << shift) - d) << 32) / d + 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
#endif
};

struct CacheView {
  uint8_t* pages;
  int64_t num_pages;
  const int32_t* table;
  int64_t table_stride;
  int64_t capacity;  // positions the table reaches: table_width * page_size
  int heads;         // key/value heads
  int page_shift;    // log2(page_size)
  const float* k_scale;
  const float* v_scale;
};

struct CacheRows {
  void* data;
  int64_t sb, st, sh;  // elements
  bool wide;           // rows start on 32 bytes
};

// The run `run` (position / 16) of request i, head h; nullptr where the table
// names no page of the pool.
template <int D>
__device__ __forceinline__ uint8_t* cache_run(const CacheView& c, int i, int h, int64_t run) {
  const int per_page = c.page_shift - 4;  // log2(runs of a page)
  const int64_t page = c.table[i * c.table_stride + (run >> per_page)];
  if (page < 0 || page >= c.num_pages) return nullptr;
  const int64_t r = ((page * c.heads + h) << per_page) + (run & ((1 << per_page) - 1));
  return c.pages + r * run_bytes(D);
}

// Two e4m3 scales (low byte first) -> two fp16; exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<unsigned short>(two)));
  return r;
}
// Eight e2m1 codes (low four bits first) -> four fp16 pairs; exact.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
// Eight values -> eight e2m1 codes, the first in the low four bits: to nearest,
// ties to even, saturating.
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float (&q)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}\n"
      : "=r"(r)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return r;
}
// (a, b) * (c, c) and (a, b) * (c, c) + (d, e), two at a time.
__device__ __forceinline__ float2 mul_pair(float2 a, float c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(c));
  return r;
}
__device__ __forceinline__ float2 fma_pair(float2 a, float c, float2 d) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tmov.b64 z, {%5, %6};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(c), "f"(d.x), "f"(d.y));
  return r;
}
// e4m3 of a value in [0, 448], to nearest, ties to even.
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(x));
  return r & 0xffu;
}
__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float2 h2_to_f2(uint32_t a) {
  return __half22float2(*reinterpret_cast<const __half2*>(&a));
}

// 32 bytes at once where the rows allow it (`wide`: 32-byte aligned), else in two
// halves: a sector that two instructions write by halves costs twice the requests.
__device__ __forceinline__ void load32(const void* p, bool wide, uint32_t (&v)[8]) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
        : "l"(p)
        : "memory");
  } else {
    const uint4 a = static_cast<const uint4*>(p)[0], b = static_cast<const uint4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}
__device__ __forceinline__ void store32(void* p, bool wide, const uint32_t (&v)[8]) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    static_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// 16 neighbouring channels of a row, as they are (half the registers of fp32, so
// more warps are resident), and as fp32.
template <typename T>
struct Group {
  static constexpr int kWords = 4 * sizeof(T);
  uint32_t v[kWords];

  __device__ __forceinline__ void load(const T* p, bool wide) {
#pragma unroll
    for (int u = 0; u < kWords / 8; ++u) load32(p + 8 * u, wide, *reinterpret_cast<uint32_t(*)[8]>(v + 8 * u));
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int e = 0; e < kWords; ++e) v[e] = 0;
  }
  __device__ __forceinline__ float2 pair(uint32_t w) const {
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
      return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else return h2_to_f2(w);
  }
  // elements 2 e and 2 e + 1
  __device__ __forceinline__ float2 at(int e) const {
    if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
    else return pair(v[e]);
  }
  // the largest magnitude, NaN where there is a NaN
  __device__ __forceinline__ float top() const {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < kWords; ++e) {
      if constexpr (sizeof(T) == 4) m = max(m, v[e] & 0x7fffffffu);  // NaN above all
      else if constexpr (std::is_same<T, __nv_bfloat16>::value)
        asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(v[e] & 0x7fff7fffu));
      else asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(m) : "r"(v[e] & 0x7fff7fffu));
    }
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(m);
    } else {
      const float2 t = pair(m);
      return t.x != t.x || t.x > t.y ? t.x : t.y;
    }
  }
};
template <typename T>
__device__ __forceinline__ void store_group(T* p, bool wide, const float (&x)[16]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __float_as_uint(x[8 * u + e]);
      store32(p + 8 * u, wide, v);
    }
  } else {
    uint32_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
        v[e] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __half2 h = __floats2half2_rn(x[2 * e], x[2 * e + 1]);
        v[e] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    store32(p, wide, v);
  }
}

// Quantise one group.  `code` gets the sixteen codes, channel c in bits 4c;
// returns the scale's byte.  rg = RN(1/g); the largest |x| bounds y, |y| <= RN(top rg),
// since rounding is monotone; where that is not finite (some y is not), the group is NaN.
// The quotient y / s is formed as q0 = y r, q = q0 - (q0 s - y) r with r = RN(1/s):
// the correctly rounded quotient (Markstein, IBM J. Res. Dev. 34, 1990), and -0
// for y = -0.  A correctly rounded quotient lies on a midpoint of two codes only if
// the exact one does (the midpoints have three significant bits), so the
// conversion's ties-to-even decides exactly the ties of y / s.
template <typename T>
__device__ __forceinline__ uint32_t quantise_group(const Group<T>& x, float rg, uint64_t& code) {
  const float top = __fmul_rn(x.top(), rg);
  const bool bad = !(top < INFINITY);
  // top / 6 in the same way (where it is not a normal number, or overflows on its
  // way, the scale is the smallest, or the largest or NaN, all the same)
  const float sixth = 1.0f / 6.0f, t0 = __fmul_rn(top, sixth);
  uint32_t sb = f32_to_e4m3(fminf(__fmaf_rn(__fmaf_rn(-6.0f, t0, top), sixth, t0), 448.0f));
  sb = sb ? sb : 1u;  // 2^-9, the smallest scale
  const float s = h2_to_f2(e4m3x2_to_f16x2(sb)).x;
  const float r = __frcp_rn(s);
  uint32_t w[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float2 yn = mul_pair(x.at(4 * u + e / 2), -rg);  // -y
      const float2 q0 = mul_pair(yn, -r);
      const float2 v = fma_pair(fma_pair(q0, s, yn), -r, q0);
      q[e] = v.x;
      q[e + 1] = v.y;
    }
    w[u] = f32x8_to_e2m1(q);
  }
  code = bad ? 0ull : (static_cast<uint64_t>(w[1]) << 32) | w[0];
  return bad ? kScaleNaN : sb;
}

// Exchange between the eight lanes that share a scale group (lane bits 0-2 = b):
// halfword c of lane b becomes halfword b of lane c.  Its own inverse.
__device__ __forceinline__ void transpose_lanes8(uint32_t (&w)[4], int b) {
  // 4 x 4 words between lanes that differ in bits 1 and 2, then the halfwords
  // between neighbours
#pragma unroll
  for (int bit = 4; bit >= 2; bit >>= 1) {
    const bool up = b & bit;
    const int step = bit >> 1;  // words apart: 2, then 1
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      if (a & step) continue;
      const uint32_t send = up ? w[a] : w[a + step];
      const uint32_t got = __shfl_xor_sync(0xffffffffu, send, bit);
      if (up) w[a] = got;
      else w[a + step] = got;
    }
  }
  const bool odd = b & 1;
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, w[a], 1);
    w[a] = odd ? __byte_perm(got, w[a], 0x7632) : __byte_perm(w[a], got, 0x5410);
  }
}

struct CacheMove {
  CacheView c;
  CacheRows k, v;
  const int32_t* start;  // first position per request (nullptr: 0)
  const int32_t* count;  // tokens per request, clamped to [0, T] (nullptr: T)
  int B, T;
  uint32_t warps;        // of one request: runs its tokens can touch x heads x 2 (x chunks)
  Quotient by_heads;
  uint32_t* status;
};

// The request's span of positions, or false where it is skipped.
__device__ __forceinline__ bool cache_span(const CacheMove& p, int i, int64_t& n, int& L) {
  n = p.start ? p.start[i] : 0;
  L = p.count ? min(max(p.count[i], 0), p.T) : p.T;
  return n >= 0 && n + L <= p.c.capacity;
}

// One warp moves a run of one (request, head), keys or values (the write: 64
// channels of it): lane = token pair b (tokens 2b, 2b+1) + 8 * scale group.  A pair
// of tokens fills one byte of a value's row, so a warp holds whole rows of codes, and
// no two warps touch the same bytes.  Blocks (x, request); neighbouring warps have
// the chunks, keys and values, and heads of one run.
struct CacheTask {
  int i, h, chunk, is_v;
  int64_t run;
};
template <int C>
__device__ __forceinline__ bool cache_task(const CacheMove& p, CacheTask& t) {
  const uint32_t w = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  t.i = static_cast<int>(blockIdx.y);
  t.chunk = static_cast<int>(w % C);
  t.is_v = static_cast<int>(w / C & 1);
  const uint32_t run = p.by_heads(w / (2 * C));
  t.run = run;
  t.h = static_cast<int>(w / (2 * C) - run * static_cast<uint32_t>(p.c.heads));
  return w < p.warps;
}

constexpr int kMoveThreads = 128;

// These kernels and the attention start while what is before them in the stream
// drains, let what is behind them do the same, and touch memory only after this.
// So their inputs may change within their lifetime: none is read by a
// non-coherent load.
__device__ __forceinline__ void wait_for_stream() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Nearest to a limit is issue: 70 % of the slots, the ALU pipe 55 %, some 400 instructions
// for a warp's 2 KB (12 or 14 blocks a SM instead of 10 change nothing).  4 x 8191 tokens,
// 8 heads of 128, fp16: 43 us, 4.0 TB/s (0.61 of the copy bandwidth); a block of 6
// tokens 8 us from cold memory, four dependent reads.  Back to back in a graph (part
// of the rows in the L2) 36 us at any width, 46 us from fp32; 256 blocks of 6: 8.5 us.
template <int D, typename T>
__global__ void __launch_bounds__(kMoveThreads) k_cache_write(CacheMove p) {
  wait_for_stream();
  CacheTask t;
  if (!cache_task<D / 64>(p, t)) return;
  const int lane = threadIdx.x & 31;
  int64_t n;
  int L;
  const bool fits = cache_span(p, t.i, n, L);
  if (!fits) {
    if (p.status && t.run == 0 && t.h == 0 && t.chunk == 0 && !t.is_v && lane == 0)
      atomicOr(p.status + t.i, kDevBadLength);
    return;
  }
  const int64_t run = (n >> 4) + t.run;
  // the request's tokens of this run: [lo, hi)
  const int lo = static_cast<int>(max(n - run * kRun, int64_t(0)));
  const int hi = static_cast<int>(min(n + L - run * kRun, int64_t(kRun)));
  if (lo >= hi) return;
  uint8_t* dst = cache_run<D>(p.c, t.i, t.h, run);
  const int b = lane & 7, g = t.chunk * 4 + (lane >> 3);
  const CacheRows& rows = t.is_v ? p.v : p.k;
  const float* gs = t.is_v ? p.c.v_scale : p.c.k_scale;
  const float rg = gs ? __frcp_rn(gs[t.h]) : 1.0f;
  const T* src = static_cast<const T*>(rows.data) + t.i * rows.sb + t.h * rows.sh + g * kGroup;
  Group<T> x[2];
  bool in[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int tok = 2 * b + u;
    in[u] = tok >= lo && tok < hi;
    if (in[u]) x[u].load(src + (run * kRun + tok - n) * rows.st, rows.wide);
    else x[u].clear();
  }
  if (!dst) {
    if (p.status && t.h == 0 && t.chunk == 0 && !t.is_v && lane == 0)
      atomicOr(p.status + t.i, kDevBadPage);
    return;
  }
  uint64_t code[2];
  uint32_t sc[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) sc[u] = quantise_group(x[u], rg, code[u]);
  if (!t.is_v) {
    // The lanes of neighbouring groups (lane ^ 8) trade halves, so that each stores
    // the 16 bytes of one token's chunk: the even group token 2b, the odd one 2b + 1;
    // and four lanes' scale bytes come together in the first two (lane ^ 8, ^ 16).
    const bool u = g & 1;
    const uint64_t got = __shfl_xor_sync(0xffffffffu, u ? code[0] : code[1], 8);
    const uint64_t first = u ? got : code[0], second = u ? code[1] : got;
    uint32_t four[2];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      uint32_t x = sc[v] << (8 * (g & 3));
      x |= __shfl_xor_sync(0xffffffffu, x, 8);
      four[v] = x | __shfl_xor_sync(0xffffffffu, x, 16);
    }
    const int tok = 2 * b + u;
    if (!(u ? in[1] : in[0])) return;
    *reinterpret_cast<uint4*>(dst + (g >> 1) * 256 + tok * 16) =
        make_uint4(static_cast<uint32_t>(first), static_cast<uint32_t>(first >> 32), static_cast<uint32_t>(second),
                   static_cast<uint32_t>(second >> 32));
    if ((g & 2) == 0)
      *reinterpret_cast<uint32_t*>(dst + run_k_scales(D) + tok * (D / kGroup) + (g & ~3)) = u ? four[1] : four[0];
    return;
  }
  // bytes of channel pairs: channel c of tokens (2b, 2b+1) in byte c
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t a = static_cast<uint32_t>(code[0] >> (16 * q)) & 0xffffu;
    const uint32_t c = static_cast<uint32_t>(code[1] >> (16 * q)) & 0xffffu;
    // spread the four codes of each token over four bytes
    const uint32_t sa = (a | (a << 8)) & 0x00ff00ffu, sc2 = (c | (c << 8)) & 0x00ff00ffu;
    const uint32_t ea = (sa | (sa << 4)) & 0x0f0f0f0fu, ec = (sc2 | (sc2 << 4)) & 0x0f0f0f0fu;
    w[q] = ea | (ec << 4);
  }
  transpose_lanes8(w, b);
  // now the channels 2b, 2b+1 of the group, interleaved: part them into rows of
  // eight bytes, one for each token pair
  {
    const uint32_t a0 = __byte_perm(w[0], w[1], 0x6420), a1 = __byte_perm(w[2], w[3], 0x6420);
    const uint32_t b0 = __byte_perm(w[0], w[1], 0x7531), b1 = __byte_perm(w[2], w[3], 0x7531);
    w[0] = a0, w[1] = a1, w[2] = b0, w[3] = b1;
  }
  uint4* row = reinterpret_cast<uint4*>(dst + run_v_codes(D) + (g * kGroup + 2 * b) * 8);
  if (hi - lo == kRun) {
    *row = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    const uint64_t mask = ((1ull << (4 * (hi - lo))) - 1) << (4 * lo);
    const uint32_t ml = static_cast<uint32_t>(mask), mh = static_cast<uint32_t>(mask >> 32);
    const uint4 o = *row;
    *row = make_uint4((o.x & ~ml) | (w[0] & ml), (o.y & ~mh) | (w[1] & mh),
                      (o.z & ~ml) | (w[2] & ml), (o.w & ~mh) | (w[3] & mh));
  }
  uint8_t* vs = dst + run_v_scales(D) + g * kRun + 2 * b;
  if (in[0] && in[1]) {
    *reinterpret_cast<uint16_t*>(vs) = static_cast<uint16_t>(sc[0] | (sc[1] << 8));
  } else if (in[0]) {
    vs[0] = static_cast<uint8_t>(sc[0]);
  } else if (in[1]) {
    vs[1] = static_cast<uint8_t>(sc[1]);
  }
}

// Bound by the memory it writes: 12 requests of 1000..16384 positions, 8 heads of 128,
// to fp16: 113 us, 5.2 TB/s (0.80 of the copy bandwidth), 101 us back to back in a
// graph (0.90); to fp32 180 us (0.90).
template <int D, typename T>
__global__ void __launch_bounds__(kMoveThreads) k_cache_read(CacheMove p) {
  wait_for_stream();
  CacheTask t;
  if (!cache_task<1>(p, t)) return;  // the whole run: all its bytes in flight
  const int lane = threadIdx.x & 31;
  int64_t n;
  int L;
  if (!cache_span(p, t.i, n, L)) {
    if (p.status && t.run == 0 && t.h == 0 && t.chunk == 0 && !t.is_v && lane == 0)
      atomicOr(p.status + t.i, kDevBadLength);
    return;
  }
  const int64_t run = (n >> 4) + t.run;
  const int lo = static_cast<int>(max(n - run * kRun, int64_t(0)));
  const int hi = static_cast<int>(min(n + L - run * kRun, int64_t(kRun)));
  if (lo >= hi) return;
  const uint8_t* src = cache_run<D>(p.c, t.i, t.h, run);
  if (!src) {
    if (p.status && t.h == 0 && t.chunk == 0 && !t.is_v && lane == 0)
      atomicOr(p.status + t.i, kDevBadPage);
    return;
  }
  const int b = lane & 7;
  const float* gs = t.is_v ? p.c.v_scale : p.c.k_scale;
  const float gv = gs ? gs[t.h] : 1.0f;
  constexpr int C = D / 64;
  uint4 raw[C];  // keys: token 2b's codes, token 2b + 1's; values: channel 2b's, channel 2b + 1's
  uint32_t sc[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int g = c * 4 + (lane >> 3);
    if (!t.is_v) {
      const uint8_t* at = src + (g >> 1) * 256 + 2 * b * 16 + (g & 1) * 8;
      const uint2 k0 = *reinterpret_cast<const uint2*>(at), k1 = *reinterpret_cast<const uint2*>(at + 16);
      raw[c] = make_uint4(k0.x, k0.y, k1.x, k1.y);
      const uint8_t* s = src + run_k_scales(D) + 2 * b * (D / kGroup) + g;
      sc[c] = s[0] | (static_cast<uint32_t>(s[D / kGroup]) << 8);
    } else {
      raw[c] = *reinterpret_cast<const uint4*>(src + run_v_codes(D) + (g * kGroup + 2 * b) * 8);
      sc[c] = *reinterpret_cast<const uint16_t*>(src + run_v_scales(D) + g * kRun + 2 * b);
    }
  }
  const CacheRows& rows = t.is_v ? p.v : p.k;
  T* out = static_cast<T*>(rows.data) + t.i * rows.sb + t.h * rows.sh;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int g = c * 4 + (lane >> 3);
    uint32_t code[2][2] = {{raw[c].x, raw[c].y}, {raw[c].z, raw[c].w}};
    if (t.is_v) {
      const uint4 o = raw[c];
      uint32_t w[4] = {__byte_perm(o.x, o.z, 0x5140), __byte_perm(o.x, o.z, 0x7362),
                       __byte_perm(o.y, o.w, 0x5140), __byte_perm(o.y, o.w, 0x7362)};
      transpose_lanes8(w, b);  // byte: a channel of the tokens 2b (low four bits), 2b + 1
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        // eight channels' bytes to the eight codes of each token
        const uint32_t l0 = w[2 * q] & 0x0f0f0f0fu, l1 = w[2 * q + 1] & 0x0f0f0f0fu;
        const uint32_t h0 = (w[2 * q] >> 4) & 0x0f0f0f0fu, h1 = (w[2 * q + 1] >> 4) & 0x0f0f0f0fu;
        code[0][q] = __byte_perm(l0 | (l0 >> 4), l1 | (l1 >> 4), 0x6420);
        code[1][q] = __byte_perm(h0 | (h0 >> 4), h1 | (h1 >> 4), 0x6420);
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int tok = 2 * b + u;
      if (tok < lo || tok >= hi) continue;
      const uint32_t one = u ? sc[c] >> 8 : sc[c] & 0xffu;
      const uint32_t s2 = e4m3x2_to_f16x2(one | (one << 8));
      float x[16];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t h[4];
        e2m1x8_to_f16(code[u][q], h);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = mul_pair(h2_to_f2(h2_mul(h[e], s2)), gv);
          x[8 * q + 2 * e] = f.x;
          x[8 * q + 2 * e + 1] = f.y;
        }
      }
      store_group(out + (run * kRun + tok - n) * rows.st + g * kGroup, rows.wide, x);
    }
  }
}

}  // namespace sv

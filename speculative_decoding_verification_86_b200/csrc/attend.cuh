// Attention of a request's block over its 4-bit cache.
//
// For one key/value head, the R = block tokens x query heads of the group rows
// that share its keys are one problem: S^T = K Q^T and O^T = V^T P^T, with the
// cache's tokens (for S) and channels (for O) on the 128 rows of a tcgen05 tile
// and the few query rows on its N.  So every 4-bit code is decoded once for all
// R rows, and is decoded where the tensor core reads it: a thread owns one token
// of the keys (or one channel of the values), converts its codes to fp16 times
// the group's scale -- exact, six significant bits -- and stores them as its
// lane of the A operand in tensor memory.  Shared memory carries the packed
// bytes and the small B operands (Q, P) only; the decoded tile, 3.6 times the
// bytes, never passes through it.
//
// One persistent CTA per SM walks an equal share of all (request, head, tile of
// 128 tokens) units in order, so a long context is split over many CTAs and
// short ones share one.  Roles (warps):
//   plan          writes the share's segments (one request, head, row tile each)
//                 into a ring that the other roles read;
//   producer      bulk copies of the runs of a tile into a ring of stages;
//   K 0-3, V 4-7  decode into tensor memory, lane = token / channel;
//   MMA           one thread issues S(t+1) before O(t), so the softmax of one
//                 tile overlaps the products of its neighbours;
//   softmax       lane = token, registers = query rows: S from tensor memory,
//                 P (fp16) to shared memory, sums in registers.  The reference
//                 maximum of a row is raised only when a P passes 2^15 (a vote of
//                 the warps); then, and only then, O is rescaled in tensor memory;
//   epilogue      loads and converts the next segment's Q, and writes O of the
//                 finished one: final rows, or (a segment cut by a CTA's share)
//                 unnormalised fp32 partials, which k_attend_join adds in the
//                 order of the CTAs.
// Every wait is bounded (warp_wait): a role whose wait runs out leaves, those that
// wait for it follow, copies and products in flight are awaited and tensor memory is
// freed.  The error word and SPEC_DEV_INTERNAL of the batch's requests are raised,
// and rows that such a CTA has a part of are not joined.
//
// What bounds it: no unit (24 rows: 63 % of the issue slots, ALU 49 %, tensor 16 %,
// half of the copy bandwidth) but the roles' own serial paths, which share the issue
// slots.  A tile of 128 tokens takes 1270 cycles at 8 query rows, 1570 at 24, 2450 at
// 48 (D = 128) and costs 3000 to 4000 warp instructions, about half of them to decode
// the codes.  With clocks around one role's waits at a time: above 32 rows the softmax
// works 2250 of the 2450 cycles and waits for nothing; up to 32 rows the warp that
// issues the products sets the pace (clocks around its five waits a tile lengthen the
// call by half, around the two of a decoder by a tenth), and K and V decoders, some
// 1000 and 1100 cycles a tile, follow closely; at D = 256 and 8 rows the decoders do
// (1700 and 1800 of 2300; one K buffer).
// Measured: 256 requests of 64..4096 positions, 24 rows each (32 / 8 heads of 128):
// 216 us (225 on another B200), 2.9 TB/s, 0.45 of the copy bandwidth; 64 requests of
// 500..8192 positions, 8 rows: 93 us, 3.3 TB/s; one of 100,003 positions: 46 us; one
// of 700: 12.3 us, of which 3 us are the plan, 3 us the join and the rest the chain of
// memory round trips and one cold pass through every role's code.
#pragma once
#include <climits>

#include "cache.cuh"
#include "ptx.cuh"

namespace sv {

constexpr int kTile = 128;          // tokens of a tile: the rows of S^T
constexpr int kTileRuns = kTile / kRun;
constexpr float kLift = 8.0f;       // P = 2^(x - max + kLift): keeps small P out of fp16's subnormals
constexpr uint32_t kRaise = 0x7800u;  // fp16 2^15: a larger P raises the row's reference

struct AttendParams {
  CacheView c;
  CacheRows q, out;
  const int32_t* cache_len;
  const int32_t* block_len;  // nullptr: T
  int B, T, heads_q, group;  // group: query heads per key/value head
  int rp;                    // query rows of a row tile
  Quotient by_group;
  int seg_units;             // what a segment costs beside its tiles, in tiles
  int bf16;                  // q and out are bf16 (else fp16)
  float scale;
  float one;  // 1.0f (mul_add_2)
  int causal, window;
  float* lse;  // [B, T, heads_q] or nullptr
  uint32_t* status;
  // workspace
  float* part_o;   // [2 grid][NP][D]: unnormalised rows of a CTA's cut segments
  float2* part_l;  // [2 grid][NP]: (reference exponent, sum)
  struct AttendCut* cuts;  // [grid]
  unsigned* error;
  int* lost;  // [grid]: this CTA gave up
};

// A segment that is cut at the start of a CTA's share: which rows, and which
// CTAs hold its parts (first: slot 1, the others: slot 0).
struct AttendCut {
  int i, h, row0, rows;
  int first, last;  // last < 0: nothing to join here
  int pad[2];
};

constexpr int kSegs = 8;  // ring of planned segments
constexpr int kSharedBytes = 18432;

// NP: rows a row tile may have, a multiple of 8.
template <int D, int NP>
struct AttendGeo {
  static constexpr int kN = (NP + 15) / 16 * 16;  // N of the products: columns of S, O, P
  static constexpr int kMT = (D + 127) / 128;   // tiles of 128 channels of O^T
  // Softmax: two sets of one warpgroup that take the tiles in turn, each with its
  // own references and its own O (a tile's path through wait, scores, vote is longer
  // than the other roles'), where tensor memory holds both; else one set of two
  // warpgroups by columns.
  static constexpr int kSets = NP <= 32 && kMT * kN <= 32 ? 2 : 1;
  static constexpr int kSoftGroups = NP > 32 ? 2 : 1;
  static constexpr int kCW = NP / kSoftGroups;  // query rows per softmax thread
  static constexpr int kSoftWarps = 4 * kSoftGroups * kSets;
  // buffers in tensor memory (512 columns)
  static constexpr int kKB = D > 128 ? 1 : 2;
  static constexpr int kOB = D > 128 ? 1 : 2;
  static constexpr int kKCols = D / 2;          // 32-bit columns of one K buffer
  static constexpr int kVCols = 64 * kMT;
  static constexpr int kOCols = kSets * kMT * kN;
  static constexpr int kTmemK = 0;
  static constexpr int kTmemV = kTmemK + kKB * kKCols;
  static constexpr int kTmemS = kTmemV + 2 * kVCols;
  static constexpr int kTmemO = kTmemS + 2 * kN;
  static constexpr int kTmemUsed = kTmemO + kOB * kOCols;
  static constexpr int kTmemCols = kTmemUsed <= 256 ? 256 : 512;
  static_assert(kTmemUsed <= 512, "tensor memory");
  static constexpr int kWarpEpi = 8;
  static constexpr int kWarpSoft = 12;
  static constexpr int kWarpLoad = kWarpSoft + kSoftWarps;
  static constexpr int kWarpMma = kWarpLoad + 1;
  static constexpr int kWarpPlan = kWarpMma + 1;
  static constexpr int kThreads = 32 * (kWarpPlan + 1);
  static constexpr int kSegReaders = 1 + 1 + 4 + 4 + kSoftWarps + 4;  // warps that read a segment
  static constexpr int kGroups = D / kGroup;
  static constexpr uint32_t kStageBytes = kTileRuns * run_bytes(D);
  static constexpr uint32_t kQBytes = kN * D * 2;
  static constexpr uint32_t kPBytes = kN * kTile * 2;
  static constexpr uint32_t kFixed = 2 * kQBytes + 2 * kPBytes + 4 * 512 * kMT + kSharedBytes;
  static constexpr int kStages = static_cast<int>((227 * 1024 - 1024 - kFixed) / kStageBytes) < 8
                                     ? static_cast<int>((227 * 1024 - 1024 - kFixed) / kStageBytes)
                                     : 8;
  static_assert(kStages >= 3, "stages");
  static constexpr size_t kSmemBytes = 1024 + kFixed + kStages * kStageBytes;
  // fp32 accumulator, fp16 operands, M = 128, N = kN; B of O is N-major
  static constexpr uint32_t kIdescS = (1u << 4) | (static_cast<uint32_t>(kN >> 3) << 17) | (8u << 24);
  static constexpr uint32_t kIdescO = kIdescS | (1u << 16);
};

// One row tile of one request and head: its rows, the positions it reads, and
// the token tiles that cover them from its first position's run on.
struct AttendSeg {
  int i, h, row0, rows;  // rows = 0: the share's end
  int64_t run0;          // first run
  int64_t n;
  int L;
  int tiles;             // token tiles of the whole segment
  int t0, t1;            // this CTA's
  int lo, hi;            // visible to any row, in tokens from run0
  int full_lo, full_hi;  // visible to every row
};

template <int D, int NP>
struct alignas(16) AttendShared {
  using G = AttendGeo<D, NP>;
  uint64_t full[8], empty[8];
  // By tile, two of each: K and V decoded; S complete (K's buffer is free too);
  // P stored (S has been read too); O complete (V's and P's buffers are free too).
  uint64_t kready[2], vready[2], sdone[2], pready[2], odone[2];
  // By segment: Q loaded; O's last product complete, O read; sums stored.
  uint64_t qready[2], oready[2], ofree[2], lready[2];
  uint64_t segfull[kSegs], segfree[kSegs];
  uint64_t drain;
  AttendSeg seg[kSegs];
  uint32_t row[kSegs][NP];  // block token << 16 | query head of the group
  int2 lim[kSegs][NP];      // visible tokens of a row, counted from the segment's first run
  int nan_seen[kSegs];  // the value decoder took NaN scales out of the segment
  uint32_t valid[8];   // per stage: runs that were copied
  uint32_t kvalid[4];  // the same by tile, for the softmax (which lags the stages)
  alignas(16) float cs[2][NP];  // log2 units of one unit of S, per query row
  // by softmax set
  alignas(16) float nmr[G::kSets][NP];  // minus the subtracted exponent: kLift - mref, 0 while nothing was seen
  alignas(16) float fac[G::kSets][NP];
  float mref[G::kSets][NP];     // running maximum (log2 units)
  float red[G::kSets][4][NP];
  float mout[2][G::kSets][NP];  // references and sums (by warp) of a finished segment
  float lsum[2][G::kSets][4][NP];
  float weight[4][G::kSets][NP];  // epilogue, by warp: factors of the sets' O
  long long to[4][NP];    // and where its rows go
  long long scan[32];
  long long units;      // this CTA's share: number of units, and where it starts
  int start_i;
  long long start_off, start_units;
  uint32_t tmem;
};

// ---------------------------------------------------------------- helpers --
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
// (without the compiler's memory barrier: a fence follows before anyone reads)
__device__ __forceinline__ void sts128_free(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w));
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
// 8 or 16 columns of this thread's lane, and the wait for them: one statement, so
// that nothing uses the registers in between.
template <int N>
__device__ __forceinline__ void tmem_get(uint32_t t, float* r) {
  if constexpr (N == 8) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
        : "r"(t));
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
          "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(t));
  }
}
__device__ __forceinline__ void tmem_st8(uint32_t t, const float* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t),
               "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
  return r;
}
// D[tmem] (+)= A[tmem] B[smem] over 64 values of K, fp16 operands, fp32
// accumulator: four instructions of K = 16 (A 8 columns apart, B `step` units of
// 16 bytes).  The whole warp runs this and one lane's predicate
// issues: in a branch that only one lane takes, an instruction needs 50 cycles
// (operands move to uniform registers one by one), so it takes 18 at N = 32.
__device__ __forceinline__ void umma_ts64(uint32_t d, uint32_t a, uint64_t b, uint64_t step, uint32_t idesc,
                                          uint32_t accumulate, uint32_t elected) {
  asm volatile(
      "{\n\t.reg .pred e, p, t;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 e, %6, 0;\n\t"
      "setp.eq.b32 t, %4, %4;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %4, p;\n\t"
      "add.u32 a, %1, 8;\n\tadd.s64 b, %2, %3;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %4, t;\n\t"
      "add.u32 a, %1, 16;\n\tadd.s64 b, b, %3;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %4, t;\n\t"
      "add.u32 a, %1, 24;\n\tadd.s64 b, b, %3;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %4, t;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "l"(step), "r"(idesc), "r"(accumulate), "r"(elected)
      : "memory");
}
// Matrix descriptor of P^T, N-major with the 32-byte swizzle: rows of 16 query
// rows (32 bytes) per token, eight tokens 256 bytes apart (stride byte offset),
// blocks of 16 query rows `block` bytes apart (leading byte offset).
__device__ __forceinline__ uint64_t sw32_n_desc(uint32_t saddr, uint32_t block) {
  uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(block >> 4) << 16;
  d |= static_cast<uint64_t>(256 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(6) << 61;
  return d;
}
__device__ __forceinline__ void umma_commit_if(uint64_t* bar, uint32_t elected) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(smem_addr(bar)),
      "r"(elected)
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// (a, b) = (a, b) * (fa, fb), rounded, + (ma, mb).  A packed product and a packed
// sum get joined into one rounding (measured), so the sum is a multiply-add by
// `one`, a 1.0f that the compiler does not know.
__device__ __forceinline__ void mul_add_2(float& a, float& b, float fa, float fb, float ma, float mb, float one) {
  asm("{\n\t.reg .b64 x, f, m, one;\n\t"
      "mov.b64 x, {%0, %1};\n\t"
      "mov.b64 f, {%2, %3};\n\t"
      "mov.b64 m, {%4, %5};\n\t"
      "mov.b64 one, {%6, %6};\n\t"
      "mul.rn.f32x2 x, x, f;\n\t"
      "fma.rn.f32x2 x, x, one, m;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}\n"
      : "+f"(a), "+f"(b)
      : "f"(fa), "f"(fb), "f"(ma), "f"(mb), "f"(one));
}
__device__ __forceinline__ void add_2(float& a, float& b, float x, float y) {
  asm("{\n\t.reg .b64 s, t;\n\t"
      "mov.b64 s, {%0, %1};\n\t"
      "mov.b64 t, {%2, %3};\n\t"
      "add.rn.f32x2 s, s, t;\n\t"
      "mov.b64 {%0, %1}, s;\n\t}\n"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}
// Sum of v[c] over the warp's lanes, in lane c (< N): the lanes trade halves of
// the columns.
template <int N>
__device__ __forceinline__ float warp_column_sums(const float (&v)[N]) {
  constexpr int W = N > 16 ? 32 : (N > 8 ? 16 : 8);
  const int lane = threadIdx.x & 31;
  float x[W];
#pragma unroll
  for (int c = 0; c < W; ++c) x[c] = c < N ? v[c] : 0.0f;
#pragma unroll
  for (int o = 16; o >= W; o >>= 1) {
#pragma unroll
    for (int c = 0; c < W; ++c) x[c] += __shfl_xor_sync(0xffffffffu, x[c], o);
  }
#pragma unroll
  for (int o = W / 2; o; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int c = 0; c < o; ++c) {
      const float send = up ? x[c] : x[c + o];
      const float got = __shfl_xor_sync(0xffffffffu, send, o);
      x[c] = (up ? x[c + o] : x[c]) + got;
    }
  }
  return x[0];
}
__device__ __forceinline__ uint32_t h2_max(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
// Barrier `id` of 128 threads; true if `pred` holds in any of them.
__device__ __forceinline__ bool group_any(int id, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(id), "r"(static_cast<uint32_t>(pred))
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int id) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory");
}

// ------------------------------------------------------------- work shares --
// A request's units, in order: head, row tile, token tile.  A segment (one row
// tile of one head) counts p.seg_units more than its tiles: what its first
// references, its Q and its output cost beside them (chosen in cache.cu).  Equal shares of bare tiles
// left the CTAs with many short segments 29% behind the mean (256 requests of
// 64..4096 positions).
__device__ __forceinline__ bool attend_len(const AttendParams& p, int i, int64_t& n, int& L) {
  n = p.cache_len[i];
  L = p.block_len ? min(max(p.block_len[i], 0), p.T) : p.T;
  return n >= 0 && n + L <= p.c.capacity;
}

__device__ __forceinline__ int of_group(const AttendParams& p, int row) {
  return static_cast<int>(p.by_group(static_cast<uint32_t>(row)));
}
__device__ __forceinline__ int row_tiles(const AttendParams& p, int L) {
  const int rows = L * p.group;
  return rows <= p.rp ? (rows > 0) : (rows + p.rp - 1) / p.rp;
}

__device__ __forceinline__ void attend_rows(const AttendParams& p, int64_t n, int L, int rt, AttendSeg& s) {
  s.row0 = rt * p.rp;
  s.rows = min(p.rp, L * p.group - s.row0);
  const int j0 = of_group(p, s.row0), j1 = of_group(p, s.row0 + s.rows - 1);
  const int64_t hi = p.causal ? n + j1 + 1 : n + L;
  const int64_t lo = p.window ? max(n + j0 + 1 - p.window, int64_t(0)) : 0;
  s.run0 = lo >> 4;
  const int64_t base = s.run0 << 4;
  s.lo = static_cast<int>(lo - base);
  s.hi = static_cast<int>(hi - base);
  s.full_lo = p.window ? static_cast<int>(max(n + j1 + 1 - p.window, lo) - base) : s.lo;
  s.full_hi = p.causal ? static_cast<int>(n + j0 + 1 - base) : s.hi;
  s.tiles = (s.hi + kTile - 1) / kTile;
  s.n = n;
  s.L = L;
}

// Units of one head of request i; -1 where the request is skipped.
__device__ __forceinline__ long long attend_units(const AttendParams& p, int i) {
  int64_t n;
  int L;
  if (!attend_len(p, i, n, L)) return -1;
  const int nrt = row_tiles(p, L);
  long long u = 0;
  AttendSeg s;
#pragma unroll 1
  for (int rt = 0; rt < nrt; ++rt) {
    attend_rows(p, n, L, rt, s);
    u += s.tiles + p.seg_units;
  }
  return u;
}

static __device__ __noinline__ long long div64(long long a, long long b) { return a / b; }
// a / b for a >= 0, b > 0; small numbers in a few instructions
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 31) == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : div64(a, b);
}
// Of n CTAs each takes `base` units, the first `more` of them one more.
struct AttendShares {
  long long base;
  int more;
  __device__ __forceinline__ AttendShares(long long total, int n) : base(quotient(total, n)) {
    more = static_cast<int>(total - base * n);
  }
  __device__ __forceinline__ long long start(int c) const { return base * c + min(c, more); }
  __device__ __forceinline__ int of(long long unit) const {
    const long long t = (base + 1) * more;
    return static_cast<int>(unit < t ? quotient(unit, base + 1) : more + quotient(unit - t, base));
  }
};

// All lanes of a warp leave a wait together; false where the phase did not complete
// within kWaitTries tries.  A try sleeps for up to 2700 cycles (measured) but may
// return at once, some 30 cycles with the loop, so this is 60 ms at least and 6 s at
// most; a healthy launch waits 40 ms at most, for a share of all the tokens that fit
// 180 GB.  Looking at the clock here, or a limit that the compiler does not know, cost
// a sixth to a third of the kernel's time (256 requests 215 -> 250..290 us): this
// stands at some thirty places.  A role that gives up returns false, and the roles
// that wait for it give up in their turn.  The tests build with 1 and run that.
#ifndef SV_WAIT_TRIES
#define SV_WAIT_TRIES (1u << 22)
#endif
constexpr uint32_t kWaitTries = SV_WAIT_TRIES;
constexpr uint32_t kDrainTries = 1u << 22;  // what is in flight lands whatever the roles do
template <uint32_t TRIES = kWaitTries>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (uint32_t left = TRIES; left; --left)
    if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
  return false;
}

// ------------------------------------------------------------------- roles --
// One warp.  Also leaves the cut at the start of the share for k_attend_join.
template <int D, int NP>
__device__ __forceinline__ bool attend_plan(const AttendParams& p, AttendShared<D, NP>& sh, long long u0,
                                            const AttendShares& shares) {
  const int lane = threadIdx.x & 31;
  long long left = sh.units, off = sh.start_off;
  int i = sh.start_i, h = 0, rt = 0;
  AttendSeg s;
  uint32_t ns = 0;
  int64_t n = 0;
  int L = 0, nrt = 0;
  long long per_head = sh.start_units;
  bool known = true;  // per_head is request i's
  bool open = false;  // request i is under way at (h, rt, off tiles into it)
  AttendCut cut;
  cut.last = -1;
  while (left > 0) {
    if (!open) {
      if (!known) {
        while ((per_head = attend_units(p, i)) <= 0) ++i;  // requests without units
      }
      known = false;
      attend_len(p, i, n, L);
      nrt = row_tiles(p, L);
      h = off ? static_cast<int>(quotient(off, per_head)) : 0;
      off -= h * per_head;
      rt = 0;
      open = true;
    }
    attend_rows(p, n, L, rt, s);
    const int all = s.tiles + p.seg_units;
    if (off >= all) {  // only where the share starts behind a row tile
      off -= all;
      ++rt;
      continue;
    }
    s.i = i;
    s.h = h;
    s.t0 = static_cast<int>(max(off - p.seg_units, 0ll));
    s.t1 = static_cast<int>(max(min(static_cast<long long>(all), off + left) - p.seg_units, 0ll));
    const long long here = min(static_cast<long long>(all) - off, left);
    off = 0;
    if (s.t1 > s.t0) {
      const int slot = static_cast<int>(ns % kSegs);
      if (!warp_wait(&sh.segfree[slot], ((ns / kSegs) & 1u) ^ 1u)) break;
      for (int r = lane; r < NP; r += 32) {
        const int row = s.row0 + r, j = of_group(p, row);
        sh.row[slot][r] = static_cast<uint32_t>(j) << 16 | static_cast<uint32_t>(row - j * p.group);
        int2 v = make_int2(0, INT_MAX);
        if (r < s.rows) {
          const int64_t base = s.run0 << 4, pos = n + j;
          v.x = p.window ? static_cast<int>(max(pos + 1 - p.window - base, int64_t(0))) : 0;
          v.y = static_cast<int>((p.causal ? pos + 1 : n + L) - base);
        }
        sh.lim[slot][r] = v;
      }
      if (lane == 0) {
        sh.seg[slot] = s;
        sh.nan_seen[slot] = 0;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.segfull[slot]);
      if (ns == 0 && s.t0 > 0) {  // behind the first segment, which the roles wait for
        const long long first = u0 - s.t0;  // the segment's first tile
        if (shares.of(first) == static_cast<int>(blockIdx.x) - 1) {
          cut.i = s.i;
          cut.h = s.h;
          cut.row0 = s.row0;
          cut.rows = s.rows;
          cut.first = static_cast<int>(blockIdx.x) - 1;
          cut.last = shares.of(first + s.tiles - 1);
        }
      }
      ++ns;
    }
    left -= here;
    if (++rt == nrt) {
      rt = 0;
      if (++h == p.c.heads) {
        open = false;
        ++i;
      }
    }
  }
  const int slot = static_cast<int>(ns % kSegs);
  const bool ok = left == 0 && warp_wait(&sh.segfree[slot], ((ns / kSegs) & 1u) ^ 1u);
  if (lane == 0) {
    if (ok) {
      sh.seg[slot].rows = 0;
      mbar_arrive(&sh.segfull[slot]);
    }
    p.cuts[blockIdx.x] = cut;
  }
  return ok;
}

// The roles' view of the ring: the segment, or nullptr at the share's end and where
// the wait for it ran out (seg_ended tells which).
template <class SH>
__device__ __forceinline__ const AttendSeg* seg_wait(SH& sh, uint32_t ns) {
  const int slot = static_cast<int>(ns % kSegs);
  if (!warp_wait(&sh.segfull[slot], (ns / kSegs) & 1u)) return nullptr;
  return sh.seg[slot].rows > 0 ? &sh.seg[slot] : nullptr;
}
template <class SH>
__device__ __forceinline__ bool seg_ended(SH& sh, uint32_t ns) {
  const int slot = static_cast<int>(ns % kSegs);
  return __all_sync(0xffffffffu, mbar_test(&sh.segfull[slot], (ns / kSegs) & 1u)) && sh.seg[slot].rows == 0;
}
template <class SH>
__device__ __forceinline__ void seg_done(SH& sh, uint32_t ns) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.segfree[ns % kSegs]);
}

template <int D, int NP>
__device__ __forceinline__ bool attend_producer(const AttendParams& p, AttendShared<D, NP>& sh, uint32_t stages) {
  using G = AttendGeo<D, NP>;
  const int lane = threadIdx.x & 31;
  uint32_t g = 0;
  bool ok = true;
  const AttendSeg* sp;
  uint32_t ns = 0;
  for (; ok && (sp = seg_wait(sh, ns)) != nullptr; ++ns) {
    const int i = sp->i, h = sp->h, t1 = sp->t1, hi = sp->hi;
    const int64_t run0 = sp->run0;
    // a lane looks up one run; 32 runs are four tiles
    auto look_up = [&](int t) -> const uint8_t* {
      const int run = t * kTileRuns + lane;
      if (run * kRun >= hi || run >= t1 * kTileRuns) return nullptr;
      const uint8_t* a = cache_run<D>(p.c, i, h, run0 + run);
      if (!a && p.status) atomicOr(p.status + i, kDevBadPage);
      return a;
    };
    const uint8_t* next = look_up(sp->t0);
#pragma unroll 1
    for (int t = sp->t0; ok && t < t1; t += 4) {
      const uint8_t* src = next;
      if (t + 4 < t1) next = look_up(t + 4);
      const uint32_t have = __ballot_sync(0xffffffffu, src != nullptr);
#pragma unroll 1
      for (int u = 0; u < 4 && t + u < t1; ++u, ++g) {
        const int st = static_cast<int>(g % G::kStages);
        if (!warp_wait(&sh.empty[st], ((g / G::kStages) & 1u) ^ 1u)) {
          ok = false;
          break;
        }
        const uint32_t v = (have >> (8 * u)) & 0xffu;
        if (lane == 0) {
          sh.valid[st] = v;
          mbar_expect_tx(&sh.full[st], __popc(v) * run_bytes(D));
        }
        __syncwarp();
        if ((lane >> 3) == u && src)
          bulk_load(stages + st * G::kStageBytes + (lane & 7) * run_bytes(D), src, run_bytes(D), &sh.full[st]);
      }
    }
    seg_done(sh, ns);
  }
  ok = ok && seg_ended(sh, ns);
  // the copies this warp issued land before the CTA's memory goes away
#pragma unroll 1
  for (uint32_t e = g > G::kStages ? g - G::kStages : 0; e < g; ++e)
    ok = warp_wait<kDrainTries>(&sh.full[e % G::kStages], (e / G::kStages) & 1u) && ok;
  return ok;
}

template <int D, int NP>
__device__ __forceinline__ bool attend_keys(const AttendParams& p, AttendShared<D, NP>& sh, uint32_t stages) {
  using G = AttendGeo<D, NP>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tok = warp * 32 + lane;
  const uint32_t row = (tok >> 4) * run_bytes(D) + (tok & 15) * 16;
  const uint32_t scales = (tok >> 4) * run_bytes(D) + run_k_scales(D) + (tok & 15) * G::kGroups;
  const uint32_t tmem = sh.tmem + (static_cast<uint32_t>(warp * 32) << 16) + G::kTmemK;
  uint32_t g = 0;
  const AttendSeg* sp;
  uint32_t ns = 0;
  for (; (sp = seg_wait(sh, ns)) != nullptr; ++ns) {
    const uint32_t end = g + static_cast<uint32_t>(sp->t1 - sp->t0);
#pragma unroll 1
    for (; g != end; ++g) {
      const int st = static_cast<int>(g % G::kStages);
      const uint32_t kb = g % G::kKB;
      if (!warp_wait(&sh.full[st], (g / G::kStages) & 1u)) return false;
      const uint32_t base = stages + st * G::kStageBytes;
      // the buffer's last reader: S of tile g - kKB
      if (g >= G::kKB &&
          !warp_wait(&sh.sdone[(g - G::kKB) & 1u], ((g - G::kKB) >> 1) & 1u))
        return false;
      tc_fence_after();
      // K of tile g follows S of tile g - kKB, so the softmax has read S of tile
      // g - 4 and its mask
      if (tok == 0) sh.kvalid[g & 3] = sh.valid[st];
#pragma unroll 1
      for (int c = 0; c < D / 32; c += 2) {
        uint32_t four;  // the scales of two chunks' groups
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(four) : "r"(base + scales + 2 * c));
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint4 w = lds128(base + row + (c + u) * 256);
          const uint32_t sc = e4m3x2_to_f16x2(u ? four >> 16 : four & 0xffffu);
          const uint32_t s0 = __byte_perm(sc, 0, 0x1010), s1 = __byte_perm(sc, 0, 0x3232);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
          uint32_t v[16];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t h[4];
            e2m1x8_to_f16(ww[x], h);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * x + e] = h2_mul(h[e], x < 2 ? s0 : s1);
          }
          tmem_st16(tmem + kb * G::kKCols + (c + u) * 16, v);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh.kready[g & 1u]);
        mbar_arrive(&sh.empty[st]);
      }
    }
    seg_done(sh, ns);
  }
  return seg_ended(sh, ns);
}

// 0xff in the bytes that are NaN as e4m3.
static __device__ __noinline__ uint32_t nan_bytes(uint32_t w) { return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); }

// Rows of a segment that see a NaN value of scale group `group` in the tiles of
// this CTA, one warp: the rare second look at scales that the decoder took out.
template <int D>
static __device__ __noinline__ unsigned long long attend_nan_rows(const AttendParams& p, const AttendSeg& s, int group) {
  const int lane = threadIdx.x & 31;
  unsigned long long m = 0;
  const int64_t base = s.run0 << 4;
  for (int t = s.t0 * kTile + lane; t < min(s.t1 * kTile, s.hi); t += 32) {
    if (t < s.lo) continue;
    const uint8_t* run = cache_run<D>(p.c, s.i, s.h, s.run0 + (t >> 4));
    if (!run || (run[run_v_scales(D) + group * 16 + (t & 15)] & 0x7fu) != kScaleNaN) continue;
    for (int r = 0; r < s.rows; ++r) {
      const int64_t q = s.n + of_group(p, s.row0 + r), pos = base + t;
      if ((p.causal ? pos <= q : pos < s.n + s.L) && (!p.window || pos > q - p.window)) m |= 1ull << r;
    }
  }
  for (int o = 16; o; o >>= 1) m |= __shfl_xor_sync(0xffffffffu, m, o);
  return m;
}

template <int D, int NP>
__device__ __forceinline__ bool attend_values(const AttendParams& p, AttendShared<D, NP>& sh, uint32_t stages,
                                              uint32_t scratch) {
  using G = AttendGeo<D, NP>;
  const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const uint32_t tmem = sh.tmem + (static_cast<uint32_t>(warp * 32) << 16) + G::kTmemV;
  const bool mine = warp * 32 < D;  // D = 64 fills half of the tile's rows
  scratch += warp * 512 * G::kMT;
  uint32_t g = 0;
  const AttendSeg* sp;
  uint32_t ns = 0;
  for (; (sp = seg_wait(sh, ns)) != nullptr; ++ns) {
    const int t1 = sp->t1, lo = sp->lo, hi = sp->hi;
#pragma unroll 1
    for (int t = sp->t0; t < t1; ++t, ++g) {
      const int st = static_cast<int>(g % G::kStages);
      const uint32_t vb = g & 1u;
      if (!warp_wait(&sh.full[st], (g / G::kStages) & 1u)) return false;
      const uint32_t base = stages + st * G::kStageBytes;
      const int tb = t * kTile;
      const uint32_t valid = sh.valid[st];
      const bool whole = valid == 0xffu && tb >= lo && tb + kTile <= hi;
      if (mine) {
        // this warp's scales (two groups of every 128 channels) to fp16, eight tokens a lane
        const int sub = lane >> 2, grp = (lane >> 1) & 1, half = lane & 1;
#pragma unroll
        for (int mt = 0; mt < G::kMT; ++mt) {
          const int group = mt * 8 + warp * 2 + grp;
          uint2 w = lds64(base + sub * run_bytes(D) + run_v_scales(D) + group * 16 + half * 8);
          if (!whole) {  // tokens that no row sees weigh nothing, whatever their bytes
            const int first = tb + sub * 16 + half * 8;
            uint32_t keep[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const bool in = ((valid >> sub) & 1u) && first + e >= lo && first + e < hi;
              if (in) keep[e >> 2] |= 0xffu << (8 * (e & 3));
            }
            w.x &= keep[0];
            w.y &= keep[1];
          }
          // scales are 0..0x7e; 0x7f (NaN) plus one, or a sign, sets a byte's top bit
          const uint32_t odd = ((w.x + 0x01010101u) | w.x | (w.y + 0x01010101u) | w.y) & 0x80808080u;
          if (__any_sync(0xffffffffu, odd != 0)) {
            // A NaN scale must not meet the zeros of P (0 NaN = NaN): it is taken out
            // here, and the epilogue looks for the rows that see it.
            w.x &= ~nan_bytes(w.x);
            w.y &= ~nan_bytes(w.y);
            sh.nan_seen[ns % kSegs] = 1;
          }
          sts128(scratch + mt * 512 + (sub * 2 + grp) * 32 + half * 16,
                 make_uint4(e4m3x2_to_f16x2(w.x & 0xffffu), e4m3x2_to_f16x2(w.x >> 16),
                            e4m3x2_to_f16x2(w.y & 0xffffu), e4m3x2_to_f16x2(w.y >> 16)));
        }
        __syncwarp();
      }
      // the buffer's last reader: O of tile g - 2
      if (!warp_wait(&sh.odone[vb], ((g >> 1) & 1u) ^ 1u)) return false;
      tc_fence_after();
      if (mine) {
#pragma unroll
        for (int mt = 0; mt < G::kMT; ++mt) {
          const uint32_t codes = base + run_v_codes(D) + (mt * 128 + warp * 32 + lane) * 8;
          const uint32_t sc = scratch + mt * 512 + (lane >> 4) * 32;
#pragma unroll 1
          for (int half = 0; half < kTileRuns; half += 4)
#pragma unroll
          for (int sub = half; sub < half + 4; sub += 2) {
            uint32_t v[16];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint2 w = lds64(codes + (sub + x) * run_bytes(D));
              const uint4 sa = lds128(sc + (sub + x) * 64), sb = lds128(sc + (sub + x) * 64 + 16);
              uint32_t h[4];
              e2m1x8_to_f16(w.x, h);
              v[8 * x] = h2_mul(h[0], sa.x);
              v[8 * x + 1] = h2_mul(h[1], sa.y);
              v[8 * x + 2] = h2_mul(h[2], sa.z);
              v[8 * x + 3] = h2_mul(h[3], sa.w);
              e2m1x8_to_f16(w.y, h);
              v[8 * x + 4] = h2_mul(h[0], sb.x);
              v[8 * x + 5] = h2_mul(h[1], sb.y);
              v[8 * x + 6] = h2_mul(h[2], sb.z);
              v[8 * x + 7] = h2_mul(h[3], sb.w);
            }
            tmem_st16(tmem + vb * G::kVCols + mt * 64 + sub * 8, v);
          }
        }
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh.vready[vb]);
        mbar_arrive(&sh.empty[st]);
      }
    }
    seg_done(sh, ns);
  }
  return seg_ended(sh, ns);
}

// One lane issues; the warp stays together.  S of tile g goes before O of tile
// g - 1.  This warp's own path is on the critical cycle (three waits, two commits
// and the products of a tile), so it waits for nothing that another wait implies:
// P of tile g - 2 stored (awaited for its O) means that S of that tile was read.
template <int D, int NP>
__device__ __forceinline__ bool attend_mma(const AttendParams& p, AttendShared<D, NP>& sh, uint32_t q_smem,
                                           uint32_t p_smem) {
  using G = AttendGeo<D, NP>;
  uint32_t g = 0, ns = 0;
  bool ok = true;
  const uint32_t tm = sh.tmem, el = elect_one();
  const uint64_t q_desc = sw128_desc(q_smem), p_desc = sw32_n_desc(p_smem, kTile * 32);
  // O of the tile before: 1 there is one, 2 the first of its segment, 4 the last,
  // 8 the first of its set in the segment
  int pend = 0;
  const AttendSeg* sp = seg_wait(sh, ns);
  bool more = sp != nullptr;
  int left = more ? sp->t1 - sp->t0 : 0;
  int idx = 0;  // of the tile in its segment
#pragma unroll 1
  while (more || pend) {
    const uint32_t b = g & 1u, use = (g >> 1) & 1u;
    if (more) {
      if (idx == 0) ok = warp_wait(&sh.qready[ns & 1u], (ns >> 1) & 1u);
      ok = ok && warp_wait(&sh.kready[b], use);
      if (!ok) break;
      tc_fence_after();
      const uint64_t q = q_desc + (ns & 1u) * (G::kQBytes >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 64; ++kk)
        umma_ts64(tm + G::kTmemS + b * G::kN, tm + G::kTmemK + (G::kKB == 2 ? b * G::kKCols : 0) + 32 * kk,
                  q + kk * (G::kN * 128 >> 4), 2, G::kIdescS, kk > 0 ? 1u : 0u, el);
      umma_commit_if(&sh.sdone[b], el);
    }
    if (pend) {
      const uint32_t pb = b ^ 1u, puse = ((g - 1) >> 1) & 1u;
      // the segment whose tile it is: this one, or the one before where this tile is its first
      const uint32_t pns = idx == 0 || !more ? ns - 1 : ns, ob = pns % G::kOB;
      ok = warp_wait(&sh.vready[pb], puse) &&
           warp_wait(&sh.pready[pb], puse) &&
           (!(pend & 2) || warp_wait(&sh.ofree[ob], ((pns / G::kOB) & 1u) ^ 1u));
      if (!ok) break;
      tc_fence_after();
      // a step is 16 tokens: 512 bytes of P
      const uint64_t pd = p_desc + pb * (G::kPBytes >> 4);
      const uint32_t d = tm + G::kTmemO + ob * G::kOCols + (G::kSets == 2 ? pb * (G::kMT * G::kN) : 0);
      const uint32_t a = tm + G::kTmemV + pb * G::kVCols;
#pragma unroll
      for (int mt = 0; mt < G::kMT; ++mt) {
        umma_ts64(d + mt * G::kN, a + mt * 64, pd, 32, G::kIdescO, (pend & 8) ? 0u : 1u, el);
        umma_ts64(d + mt * G::kN, a + mt * 64 + 32, pd + 128, 32, G::kIdescO, 1u, el);
      }
      umma_commit_if(&sh.odone[pb], el);
      if (pend & 4) umma_commit_if(&sh.oready[ob], el);
    }
    if (!more) break;
    pend = 1 | (idx == 0 ? 2 : 0) | (left == 1 ? 4 : 0) | (idx < G::kSets ? 8 : 0);
    ++idx;
    ++g;
    if (--left == 0) {
      seg_done(sh, ns);
      sp = seg_wait(sh, ++ns);
      more = sp != nullptr;
      left = more ? sp->t1 - sp->t0 : 0;
      idx = 0;
    }
  }
  ok = ok && seg_ended(sh, ns);
  // what was issued completes before tensor memory is released
  umma_commit_if(&sh.drain, el);
  return warp_wait<kDrainTries>(&sh.drain, 0) && ok;
}

// Which of a thread's N rows see the token `at` (counted from the segment's first run).
template <int N>
static __device__ __noinline__ uint32_t attend_see(const int2* lim, int at, uint32_t have) {
  uint32_t m = 0;
#pragma unroll 1
  for (int c = 0; c < N; ++c) {
    const int2 v = lim[c];
    if (at >= v.x && at < v.y) m |= 1u << c;
  }
  return have ? m : 0u;
}

// W (8 or 16) scores of a token to P: x - reference, with x = S cs rounded (the
// maximum is taken of the same rounded x, so P stays in range at any size of the
// scores), its power of two, and that in fp16.
template <int W>
__device__ __forceinline__ void attend_p(uint32_t s_tmem, const float* cs, const float* nmr, float one, bool whole,
                                         uint32_t see, float (&e)[W], uint32_t (&w)[W / 2]) {
  tmem_get<W>(s_tmem, e);
#pragma unroll
  for (int c = 0; c < W; c += 4) {
    const float4 f = *reinterpret_cast<const float4*>(cs + c);
    const float4 m = *reinterpret_cast<const float4*>(nmr + c);
    mul_add_2(e[c], e[c + 1], f.x, f.y, m.x, m.y, one);
    mul_add_2(e[c + 2], e[c + 3], f.z, f.w, m.z, m.w, one);
  }
  if (!whole) {
#pragma unroll
    for (int c = 0; c < W; ++c)
      if (!((see >> c) & 1u)) e[c] = -INFINITY;
  }
#pragma unroll
  for (int c = 0; c < W / 2; ++c) {
    e[2 * c] = ex2(e[2 * c]);
    e[2 * c + 1] = ex2(e[2 * c + 1]);
    const __half2 h = __floats2half2_rn(e[2 * c], e[2 * c + 1]);
    w[c] = *reinterpret_cast<const uint32_t*>(&h);
  }
}

// The same for columns [C, C + W) of a softmax thread: P to shared memory, its
// largest value, and the sums.
template <int C, int W, int CW>
__device__ __forceinline__ void attend_columns(uint32_t s_tmem, const float* cs, const float* nmr, float one,
                                               bool whole, uint32_t see, uint32_t p_tile, int c0, uint32_t pflip,
                                               bool again, uint32_t redo, float (&l)[CW], uint32_t& top) {
  float e[W];
  uint32_t w[W / 2];
  attend_p<W>(s_tmem + C, cs + C, nmr + C, one, whole, see >> C, e, w);
#pragma unroll
  for (int x = 0; x < W / 2; x += 4) {
    const int col = c0 + C + 2 * x;
    top = h2_max(top, h2_max(h2_max(w[x], w[x + 1]), h2_max(w[x + 2], w[x + 3])));
    sts128_free(p_tile + (col >> 4) * (kTile * 32) + (((col & 8) * 2) ^ pflip),
                make_uint4(w[x], w[x + 1], w[x + 2], w[x + 3]));
  }
  if (!again) {
#pragma unroll
    for (int x = 0; x < W; x += 2) add_2(l[C + x], l[C + x + 1], e[x], e[x + 1]);
  } else {
#pragma unroll
    for (int x = 0; x < W; ++x)
      if ((redo >> (C + x)) & 1u) l[C + x] += e[x];
  }
}

template <int D, int NP>
__device__ __forceinline__ bool attend_softmax(const AttendParams& p, AttendShared<D, NP>& sh, uint32_t p_smem) {
  using G = AttendGeo<D, NP>;
  constexpr int CW = G::kCW;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, wg = ((warp - G::kWarpSoft) >> 2) % G::kSoftGroups;
  const uint32_t set = ((warp - G::kWarpSoft) >> 2) / G::kSoftGroups;
  const int c0 = wg * CW, id = 1 + ((warp - G::kWarpSoft) >> 2);
  float* const nmr = sh.nmr[set];
  const int tok = quarter * 32 + lane;
  const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
  // this token's 32 bytes of a block of the P tile (sw32_n_desc)
  const uint32_t prow = p_smem + tok * 32, pflip = (tok & 4) << 2;
  uint32_t g = 0;
  bool ok = true;
  for (uint32_t ns = 0;; ++ns) {
    const AttendSeg* sp = seg_wait(sh, ns);
    // together: the group's barriers wait for all of it
    if (group_any(id, sp == nullptr)) return ok && seg_ended(sh, ns);
    const int rows = sp->rows, t1 = sp->t1, full_lo = sp->full_lo, full_hi = sp->full_hi;
    const uint32_t qb = ns & 1u, ob = ns % G::kOB;
    const int slot = static_cast<int>(ns % kSegs);
    bool unset = true;  // some row has seen nothing yet (uniform over the warpgroup)
    ok = ok && warp_wait(&sh.qready[qb], (ns >> 1) & 1u);
    float l[CW];
#pragma unroll
    for (int c = 0; c < CW; ++c) l[c] = 0.0f;
    bool fresh = true;  // this set's first tile of the segment
#pragma unroll 1
    for (int t = sp->t0; t < t1; ++t, ++g) {
      const uint32_t b = g & 1u;
      if (G::kSets == 2 && b != set) continue;
      const uint32_t s_tmem = sh.tmem + lanes + G::kTmemS + b * G::kN + c0;
      // S of tile g was issued behind O of tile g - 2, so P's buffer is free too
      ok = ok && warp_wait(&sh.sdone[b], (g >> 1) & 1u);
      tc_fence_after();
      const int at = t * kTile + tok;
      const uint32_t valid = sh.kvalid[g & 3];
      const bool whole = t * kTile >= full_lo && t * kTile + kTile <= full_hi && valid == 0xffu;
      uint32_t see = 0xffffffffu;  // rows that see this token
      if (!whole) see = attend_see<CW>(&sh.lim[slot][c0], at, (valid >> (tok >> 4)) & 1u);
      uint32_t redo = 0;   // second pass: rows whose sums lack this tile
      bool again = false;  // a second pass follows a raised reference
#pragma unroll 1
      for (;; again = true) {
        uint32_t top = 0;
        if (!unset || again) {
          const uint32_t pt = prow + b * G::kPBytes;
          const float* cs = &sh.cs[qb][c0];
          const float* nm = &nmr[c0];
          if constexpr (CW == 8) {
            attend_columns<0, 8>(s_tmem, cs, nm, p.one, whole, see, pt, c0, pflip, again, redo, l, top);
          } else {
            attend_columns<0, 16>(s_tmem, cs, nm, p.one, whole, see, pt, c0, pflip, again, redo, l, top);
            // columns behind the segment's rows: whatever their P holds stays in
            // columns of O that nobody reads
            if constexpr (CW > 16) {
              if (rows > c0 + 16)
                attend_columns<16, CW - 16>(s_tmem, cs, nm, p.one, whole, see, pt, c0, pflip, again, redo, l, top);
            }
          }
          fence_async_shared();
        }
        tc_fence_before();
        const bool raise = !again && (unset || !ok || (top & 0xffffu) > kRaise || (top >> 16) > kRaise);
        if (!group_any(id, raise)) break;
        if (group_any(id, !ok)) return false;
        const bool unset_before = unset;
        // new references: the maximum over the tile's tokens of every row
#pragma unroll 1
        for (int c = 0; c < CW; c += 8) {
          float x[8], keep = 0.0f;
          tmem_get<8>(s_tmem + c, x);
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const float m = warp_max(((see >> (c + u)) & 1u) ? __fmul_rn(x[u], sh.cs[qb][c0 + c + u]) : -INFINITY);
            if (lane == u) keep = m;
          }
          if (lane < 8) sh.red[set][quarter][c0 + c + lane] = keep;
        }
        group_sync(id);
        bool none = false;
        if (tok < CW) {
          const int c = c0 + tok;
          const float was = fresh ? -INFINITY : sh.mref[set][c];
          const float m = fmaxf(fmaxf(fmaxf(sh.red[set][0][c], sh.red[set][1][c]), fmaxf(sh.red[set][2][c], sh.red[set][3][c])), was);
          // rounded up, so that x - reference is at most kLift; +inf gives NaN
          const float mr = m == -INFINITY ? 0.0f : (m == INFINITY ? NAN : __fsub_ru(m, kLift));
          sh.fac[set][c] = was == -INFINITY ? 0.0f : ex2(-nmr[c] - mr);
          sh.mref[set][c] = m;
          nmr[c] = -mr;
          none = c < rows && m == -INFINITY;
        }
        unset = group_any(id, none);
        if (!fresh) {
          // O of the set's previous tile has to be complete before it is scaled;
          // with two sets that is tile g - 2, which S of tile g came after
          if (G::kSets == 1) ok = warp_wait(&sh.odone[b ^ 1u], ((g - 1) >> 1) & 1u);
          tc_fence_after();
          if (ok) {
#pragma unroll 1
            for (int mt = 0; mt < G::kMT; ++mt) {
              const uint32_t o = sh.tmem + lanes + G::kTmemO + ob * G::kOCols + (set * G::kMT + mt) * G::kN + c0;
#pragma unroll 1
              for (int c = 0; c < CW; c += 8) {
                float v[8];
                tmem_get<8>(o + c, v);
#pragma unroll
                for (int x = 0; x < 8; ++x) v[x] *= sh.fac[set][c0 + c + x];
                tmem_st8(o + c, v);
              }
            }
            tmem_st_wait();
          }
        }
        // The sums to the new references.  Where they hold this tile's P already,
        // scaling is all they need, unless they overflowed: what came before the
        // tile is then less than 2^-100 of it, and they start anew.
        redo = unset_before ? 0xffffffffu : 0u;
#pragma unroll
        for (int c = 0; c < CW; ++c) {
          const bool over = l[c] == INFINITY;
          l[c] = over ? 0.0f : l[c] * sh.fac[set][c0 + c];
          redo |= static_cast<uint32_t>(over) << c;
        }
      }
      // behind the vote: every thread of the group has read S and stored P
      if (tok == 0 && ok) mbar_arrive(&sh.pready[b]);
      fresh = false;
    }
    // the references and sums: over the warp's tokens here, over the warps in the epilogue
    ok = ok && warp_wait(&sh.ofree[ob], ((ns / G::kOB) & 1u) ^ 1u);
    const float sum = warp_column_sums<CW>(l);
    if (ok) {
      if (lane < CW) {
        sh.lsum[ob][set][quarter][c0 + lane] = sum;
        if (quarter == 0) sh.mout[ob][set][c0 + lane] = -nmr[c0 + lane];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.lready[ob]);
    }
    seg_done(sh, ns);
  }
}

// Q of a segment: rows to fp16 times a power of two that brings the row's
// largest element into [2^14, 2^15), where bf16 and fp16 values are exact down to
// 2^-39 of it; the power goes into the row's factor cs.
template <int D, int NP>
__device__ __forceinline__ void attend_load_q(const AttendParams& p, AttendShared<D, NP>& sh, const AttendSeg& s,
                                              uint32_t ns, uint32_t q_smem) {
  using G = AttendGeo<D, NP>;
  constexpr int E = D / 32;  // elements of a lane
  const int warp = (threadIdx.x >> 5) - G::kWarpEpi, lane = threadIdx.x & 31;
  const uint32_t qb = ns & 1u;
  const int ch = lane * E;
  const uint16_t* q = static_cast<const uint16_t*>(p.q.data) + s.i * p.q.sb +
                      static_cast<int64_t>(s.h * p.group) * p.q.sh;
  const float gk = p.c.k_scale ? p.c.k_scale[s.h] : 1.0f;
  const float unit = p.scale * 1.4426950408889634f * gk;
  struct alignas(E * 2) Raw {
    uint32_t w[E / 2];
  };
  // A warp's rows (every fourth; zeros behind the last) come into the tile as they
  // are, all in flight, and are converted where they lie.
  const uint32_t tile = q_smem + qb * G::kQBytes;
#pragma unroll 1
  for (int e = lane; e < NP / 4 * (D / 8); e += 32) {
    const int r = 4 * (e / (D / 8)) + warp, c = e % (D / 8);
    const uint32_t at = sh.row[ns % kSegs][r];
    const uint16_t* src = q + (at >> 16) * p.q.st + (at & 0xffffu) * p.q.sh + 8 * c;
    const uint32_t dst = tile + (c >> 3) * (G::kN * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(r < s.rows ? src : q),
                 "r"(r < s.rows ? 16 : 0)
                 : "memory");
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
#pragma unroll 1
  for (int r = warp; r < NP; r += 4) {
    const uint32_t a = tile + (ch >> 6) * (G::kN * 128) + r * 128 + (((ch & 63) * 2) ^ ((r & 7) << 4));
    Raw raw;
    if constexpr (E == 2) {
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(raw.w[0]) : "r"(a) : "memory");
    } else if constexpr (E == 4) {
      const uint2 v = lds64(a);
      raw.w[0] = v.x, raw.w[1] = v.y;
    } else {
      const uint4 v = lds128(a);
      raw.w[0] = v.x, raw.w[1] = v.y, raw.w[2] = v.z, raw.w[3] = v.w;
    }
    float x[E];
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      float2 f;
      if (p.bf16) f = make_float2(__uint_as_float(raw.w[e] << 16), __uint_as_float(raw.w[e] & 0xffff0000u));
      else f = h2_to_f2(raw.w[e]);
      x[2 * e] = f.x;
      x[2 * e + 1] = f.y;
      top = max(top, max(__float_as_uint(f.x) & 0x7fffffffu, __float_as_uint(f.y) & 0x7fffffffu));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    const bool bad = top >= 0x7f800000u;  // NaN or infinity: the whole row is NaN
    const int k = bad ? 0 : 14 + 127 - static_cast<int>(top >> 23);
    // 2^k in two factors: k reaches 141
    const float f1 = __uint_as_float(static_cast<uint32_t>(127 + (k >> 1)) << 23);
    const float f2 = __uint_as_float(static_cast<uint32_t>(127 + (k - (k >> 1))) << 23);
    Raw w;
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      const __half2 h = __floats2half2_rn(bad ? 0.0f : x[2 * e] * f1 * f2, bad ? 0.0f : x[2 * e + 1] * f1 * f2);
      w.w[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if constexpr (E == 2) asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(w.w[0]) : "memory");
    else if constexpr (E == 4)
      asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(a), "r"(w.w[0]), "r"(w.w[1]) : "memory");
    else sts128(a, make_uint4(w.w[0], w.w[1], w.w[2], w.w[3]));
    if (lane == 0) {
      const float b1 = __uint_as_float(static_cast<uint32_t>(127 - (k >> 1)) << 23);
      const float b2 = __uint_as_float(static_cast<uint32_t>(127 - (k - (k >> 1))) << 23);
      sh.cs[qb][r] = r >= s.rows ? 0.0f : (bad ? NAN : unit * b1 * b2);
    }
  }
  fence_async_shared();
  __syncwarp();
  if (lane == 0) mbar_arrive(&sh.qready[qb]);
}

template <int D, int NP>
__device__ __forceinline__ bool attend_epilogue(const AttendParams& p, AttendShared<D, NP>& sh, uint32_t q_smem) {
  using G = AttendGeo<D, NP>;
  const int warp = (threadIdx.x >> 5) - G::kWarpEpi, lane = threadIdx.x & 31;
  const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
  AttendSeg s, ahead;
  bool more = true;
  // Q of segment na goes before O of segment na - 1: the two Q buffers are then
  // free in turn, since O of segment na - 2 was the last that used its own
#pragma unroll 1
  for (uint32_t na = 0; more; ++na) {
    const AttendSeg* sp = seg_wait(sh, na);
    more = sp != nullptr;
    if (!more && !seg_ended(sh, na)) return false;
    if (more) {
      ahead = *sp;
      attend_load_q<D, NP>(p, sh, ahead, na, q_smem);
    }
    if (na == 0) {
      s = ahead;
      continue;
    }
    const uint32_t ns = na - 1, ob = ns % G::kOB, par = (ns / G::kOB) & 1u;
    const float gv = p.c.v_scale ? p.c.v_scale[s.h] : 1.0f;
    if (!warp_wait(&sh.lready[ob], par)) return false;
    if (!warp_wait(&sh.oready[ob], par)) return false;
    tc_fence_after();
    const bool cut = s.t0 > 0 || s.t1 < s.tiles;
    const int slot = 2 * static_cast<int>(blockIdx.x) + (s.t0 > 0 ? 0 : 1);
    const uint32_t* row = sh.row[ns % kSegs];
    for (int r = lane; r < s.rows; r += 32) {
      // join the sets: a set that saw nothing of the row (or had no tile) has l = 0
      float l[G::kSets], mr = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int u = 0; u < G::kSets; ++u) {
        const float* x = &sh.lsum[ob][u][0][r];
        l[u] = (x[0] + x[NP]) + (x[2 * NP] + x[3 * NP]);
        if (l[u] != 0.0f) mr = fmaxf(mr, sh.mout[ob][u][r]);
      }
      if (mr == -INFINITY) mr = 0.0f;
#pragma unroll
      for (int u = 0; u < G::kSets; ++u) {
        float w = l[u] != 0.0f ? ex2(sh.mout[ob][u][r] - mr) : 0.0f;
        if (l[u] != l[u]) w = l[u];  // NaN counts, however far below the other set's maximum
        sh.weight[warp][u][r] = w;
        if (w != 0.0f) sum += w * l[u];
      }
      if (!cut) {
        const float inv = sum == 0.0f ? 0.0f : rcp(sum);
#pragma unroll
        for (int u = 0; u < G::kSets; ++u) sh.weight[warp][u][r] *= inv;
      }
      const uint32_t at = row[r];
      const int hq = s.h * p.group + static_cast<int>(at & 0xffffu), j = static_cast<int>(at >> 16);
      sh.to[warp][r] = cut ? (static_cast<long long>(slot) * NP + r) * D
                           : s.i * p.out.sb + j * p.out.st + hq * p.out.sh;
      if (warp == 0) {
        if (cut) {
          p.part_l[slot * NP + r] = make_float2(mr, sum);
        } else if (p.lse) {
          p.lse[(static_cast<int64_t>(s.i) * p.T + j) * p.heads_q + hq] =
              sum == 0.0f ? -INFINITY : (mr + lg2(sum)) * 0.6931471805599453f;
        }
      }
    }
    __syncwarp();
#pragma unroll 1
    for (int mt = 0; mt < G::kMT; ++mt) {
      const int ch = mt * 128 + warp * 32 + lane;
      const bool mine = ch < D;
      unsigned long long nan = 0;
      if (sh.nan_seen[ns % kSegs] && mine) {  // a warp's channels are two groups
        const unsigned long long n0 = attend_nan_rows<D>(p, sh.seg[ns % kSegs], (mt * 128 + warp * 32) / kGroup);
        const unsigned long long n1 = attend_nan_rows<D>(p, sh.seg[ns % kSegs], (mt * 128 + warp * 32) / kGroup + 1);
        nan = lane < 16 ? n0 : n1;
      }
#pragma unroll 1
      for (int c = 0; c < s.rows; c += 8) {
        float v[8], u[8];
        const uint32_t o = sh.tmem + lanes + G::kTmemO + ob * G::kOCols + mt * G::kN + c;
        tmem_get<8>(o, v);
        if (G::kSets == 2) tmem_get<8>(o + G::kMT * G::kN, u);
#pragma unroll
        for (int x = 0; x < 8; ++x) {  // a set without weight may hold anything
          const float f = sh.weight[warp][0][min(c + x, NP - 1)];
          v[x] = f != 0.0f ? v[x] * f : 0.0f;
          if (G::kSets == 2) {
            const float w = sh.weight[warp][G::kSets - 1][min(c + x, NP - 1)];
            if (w != 0.0f) v[x] = fmaf(u[x], w, v[x]);
          }
        }
        if (!mine) continue;
        if (nan >> c) {
#pragma unroll
          for (int x = 0; x < 8; ++x)
            if ((nan >> (c + x)) & 1ull) v[x] = NAN;
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          if (c + x < s.rows) {
            const long long to = sh.to[warp][c + x] + ch;
            if (cut) {
              p.part_o[to] = v[x];
            } else {
              const float f = v[x] * gv;
              static_cast<uint16_t*>(p.out.data)[to] = p.bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(f))
                                                              : __half_as_ushort(__float2half_rn(f));
            }
          }
        }
      }
      __syncwarp();
    }
    tc_fence_before();
    seg_done(sh, ns);
    if (lane == 0) mbar_arrive(&sh.ofree[ob]);
    s = ahead;
  }
  return true;
}

// Exclusive prefix of v over the first `warps` warps of the CTA, and the total; the
// value of the others' threads is not looked at.
template <class SH>
__device__ __forceinline__ long long block_scan(SH& sh, long long v, int warps, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
  if (warp < warps) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sh.scan[warp] = x;
  }
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll 4
  for (int w = 0; w < warps; ++w) {
    const long long y = sh.scan[w];
    if (w < warp) before += y;
    total += y;
  }
  return before + x - v;
}

template <int D, int NP>
__global__ void __launch_bounds__(AttendGeo<D, NP>::kThreads, 1) k_attend(const __grid_constant__ AttendParams p) {
  using G = AttendGeo<D, NP>;
  extern __shared__ uint8_t attend_smem[];
  static_assert(sizeof(AttendShared<D, NP>) <= kSharedBytes, "shared block");
  const uint32_t pad = (1024u - (smem_addr(attend_smem) & 1023u)) & 1023u;
  uint8_t* base = attend_smem + pad;
  const uint32_t q_smem = smem_addr(base), p_smem = q_smem + 2 * G::kQBytes;
  const uint32_t stages = p_smem + 2 * G::kPBytes;
  const uint32_t scratch = stages + G::kStages * G::kStageBytes;
  AttendShared<D, NP>& sh = *reinterpret_cast<AttendShared<D, NP>*>(
      base + 2 * G::kQBytes + 2 * G::kPBytes + G::kStages * G::kStageBytes + 4 * 512 * G::kMT);
  const int warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int u = 0; u < G::kStages; ++u) {
      mbar_init(&sh.full[u], 1);
      mbar_init(&sh.empty[u], 8);
    }
    for (int u = 0; u < 2; ++u) {
      mbar_init(&sh.kready[u], 4);
      mbar_init(&sh.vready[u], 4);
      mbar_init(&sh.sdone[u], 1);
      mbar_init(&sh.pready[u], G::kSoftGroups);
      mbar_init(&sh.odone[u], 1);
      mbar_init(&sh.qready[u], 4);
      mbar_init(&sh.oready[u], 1);
      mbar_init(&sh.ofree[u], 4);
      mbar_init(&sh.lready[u], G::kSoftWarps);
    }
    for (int u = 0; u < kSegs; ++u) {
      mbar_init(&sh.segfull[u], 1);
      mbar_init(&sh.segfree[u], G::kSegReaders);
    }
    mbar_init(&sh.drain, 1);
    sh.start_i = 0;
    sh.start_off = 0;
    sh.start_units = 0;
    mbar_init_fence();
  }
  if (threadIdx.x < kSegs) sh.nan_seen[threadIdx.x] = 0;
  if (warp == G::kWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)),
                 "r"(G::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // what came before in the stream is complete: from here on memory is read
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x == 0) p.lost[blockIdx.x] = 0;
  // this CTA's share of the units
  long long per_head = 0, mine = 0, total = 0, before = 0;
  auto scan = [&](int i0, bool tell) {
    const int i = i0 + static_cast<int>(threadIdx.x);
    per_head = i < p.B ? attend_units(p, i) : 0;
    if (per_head < 0) {
      per_head = 0;
      if (tell && p.status && blockIdx.x == 0) atomicOr(p.status + i, kDevBadLength);
    }
    mine = per_head * p.c.heads;
    long long sum;
    before = total + block_scan(sh, mine, (min(p.B - i0, G::kThreads) + 31) >> 5, sum);
    total += sum;
  };
#pragma unroll 1
  for (int i0 = 0; i0 < p.B; i0 += G::kThreads) {
    if (i0) __syncthreads();
    scan(i0, true);
  }
  const int n = static_cast<int>(min(static_cast<long long>(gridDim.x), total));
  const int c = static_cast<int>(blockIdx.x);
  const AttendShares shares(total, max(n, 1));
  const long long u0 = c < n ? shares.start(c) : 0, u1 = c < n ? shares.start(c + 1) : 0;
  // whose request holds unit u0: known from the scan, or from a second one where
  // the batch is larger than the CTA
  const bool once = p.B <= G::kThreads;
  if (!once) total = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < p.B; i0 += G::kThreads) {
    if (!once) {
      __syncthreads();
      scan(i0, false);
    }
    if (u0 >= before && u0 < before + mine) {
      sh.start_i = i0 + static_cast<int>(threadIdx.x);
      sh.start_off = u0 - before;
      sh.start_units = per_head;
    }
  }
  if (threadIdx.x == 0) sh.units = u1 - u0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  bool ok;
  if (warp == G::kWarpLoad) {
    ok = attend_producer<D, NP>(p, sh, stages);
  } else if (warp == G::kWarpMma) {
    ok = attend_mma<D, NP>(p, sh, q_smem, p_smem);
  } else if (warp == G::kWarpPlan) {
    ok = attend_plan<D, NP>(p, sh, u0, shares);
  } else if (warp < 4) {
    ok = attend_keys<D, NP>(p, sh, stages);
  } else if (warp < 8) {
    ok = attend_values<D, NP>(p, sh, stages, scratch);
  } else if (warp < G::kWarpSoft) {
    ok = attend_epilogue<D, NP>(p, sh, q_smem);
  } else {
    ok = attend_softmax<D, NP>(p, sh, p_smem);
  }
  if (!ok) {
    atomicOr(p.error, 1u);
    p.lost[blockIdx.x] = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == G::kWarpMma) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem), "r"(G::kTmemCols)
                 : "memory");
  }
}

// Joins: a block small enough to be resident beside the attention's, whose end it
// waits for, and two rows a block.
__host__ __device__ constexpr int join_threads(int D) { return D > 128 ? D : 128; }
constexpr int kJoinRows = 2;
constexpr int kJoinMaxParts = 256;

// Memory latency bounds it, three dependent reads of the L2: some 3 us behind the
// attention.  Joining in the CTA that finishes last would save a launch, but one
// CTA would then read all the parts of a long context (19 x 24 rows x 128 channels
// for one of 100,003 positions).
// Join the parts of the segments that were cut: block (x, y), x > 0, takes the rows
// [2 y, 2 y + 2) of the segment that CTA x's share starts inside of, where
// that is the segment's first cut; block (0, 0) looks for CTAs that gave up.  Parts
// are added in the order of the CTAs (at D = 64 in two interleaved halves, then their
// sum), so the result does not depend on timing.
template <int D, int NP>
__global__ void __launch_bounds__(join_threads(D)) k_attend_join(const __grid_constant__ AttendParams p) {
  constexpr int kThreads = join_threads(D);
  constexpr int S = kThreads / D;  // threads of a channel
  __shared__ float weight[kJoinRows][kJoinMaxParts];
  __shared__ float inv[kJoinRows];
  __shared__ float sum[kJoinRows][kThreads];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0) {
    if (blockIdx.y > 0 || !p.status) return;
    bool gone = false;
    for (int c = threadIdx.x; c < static_cast<int>(gridDim.x); c += kThreads) gone |= __ldcg(p.lost + c) != 0;
    if (__syncthreads_or(gone))
      for (int i = threadIdx.x; i < p.B; i += kThreads) atomicOr(p.status + i, kDevInternal);
    return;
  }
  const AttendCut& cut = p.cuts[blockIdx.x];
  const int last = __ldcg(&cut.last);
  if (last < 0) return;
  const int i = __ldcg(&cut.i), h = __ldcg(&cut.h), row0 = __ldcg(&cut.row0), rows = __ldcg(&cut.rows),
            first = __ldcg(&cut.first);
  const int r0 = static_cast<int>(blockIdx.y) * kJoinRows;
  if (r0 >= rows) return;
  const int parts = last - first + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto slot = [&](int e) { return 2 * (first + e) + (e == 0 ? 1 : 0); };
  const int nr = min(kJoinRows, rows - r0);
  const float gv = p.c.v_scale ? p.c.v_scale[h] : 1.0f;
  int gone = 0;  // a part's CTA gave up
  if (warp < nr) {
    const int r = r0 + warp;
    constexpr int kPer = kJoinMaxParts / 32;
    float2 v[kPer];
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int e = lane + 32 * u;
      v[u] = e < parts ? __ldcg(p.part_l + slot(e) * NP + r) : make_float2(0.0f, 0.0f);
      gone |= e < parts ? __ldcg(p.lost + first + e) : 0;
    }
    gone = __any_sync(0xffffffffu, gone);
#pragma unroll
    for (int u = 0; u < kPer; ++u)
      if (v[u].y != 0.0f) m = fmaxf(m, v[u].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.0f;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int e = lane + 32 * u;
      const float w = v[u].y == 0.0f ? 0.0f : ex2(v[u].x - m);
      if (e < parts) weight[warp][e] = w;
      l += w * v[u].y;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) {
      // the functions of the rows that are not cut (attend_epilogue), to the bit
      inv[warp] = l == 0.0f ? 0.0f : rcp(l);
      if (p.lse && !gone) {
        const int row = row0 + r, j = of_group(p, row), hq = h * p.group + row - j * p.group;
        p.lse[(static_cast<int64_t>(i) * p.T + j) * p.heads_q + hq] =
            l == 0.0f ? -INFINITY : (m + lg2(l)) * 0.6931471805599453f;
      }
    }
  }
  if (__syncthreads_or(gone)) return;
  const int ch = threadIdx.x % D, part = threadIdx.x / D;
  float acc[kJoinRows] = {};
#pragma unroll 8
  for (int e = part; e < parts; e += S) {
    const float* src = p.part_o + (static_cast<int64_t>(slot(e)) * NP + r0) * D + ch;
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r)
      if (r < nr) acc[r] = fmaf(weight[r][e], __ldcg(src + r * D), acc[r]);
  }
#pragma unroll
  for (int r = 0; r < kJoinRows; ++r) sum[r][threadIdx.x] = acc[r];
  __syncthreads();
  for (int e = threadIdx.x; e < nr * D; e += kThreads) {
    const int r = e / D, cc = e % D;
    float o = 0.0f;
#pragma unroll
    for (int u = 0; u < S; ++u) o += sum[r][u * D + cc];
    o = o * inv[r] * gv;
    const int row = row0 + r0 + r, j = of_group(p, row), hq = h * p.group + row - j * p.group;
    const int64_t to = i * p.out.sb + j * p.out.st + hq * p.out.sh + cc;
    if (p.bf16) static_cast<__nv_bfloat16*>(p.out.data)[to] = __float2bfloat16_rn(o);
    else static_cast<__half*>(p.out.data)[to] = __float2half_rn(o);
  }
}

}  // namespace sv

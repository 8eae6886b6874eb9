// Host side of the 4-bit block cache (spec_cache_* in include/spec_verify.h):
// argument checks, the context's workspace and the launches.
#include "spec_verify.h"

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>

#include "attend_launch.cuh"
#include "cache.cuh"
#include "host.cuh"

struct spec_cache_ctx {
  int device = 0;
  int num_sms = 0;
  int max_batch = 0;
  int heads_q = 0, heads_kv = 0, head_dim = 0, page_size = 0;
  void* ws = nullptr;
  float* part_o = nullptr;
  float2* part_l = nullptr;
  sv::AttendCut* cuts = nullptr;
  unsigned* error = nullptr;
  int* lost = nullptr;
};

namespace {

constexpr int64_t kMaxPositions = 2147483392;  // 2^31 - 256

bool geometry_ok(int heads_kv, int head_dim, int page_size) {
  return heads_kv >= 1 && heads_kv <= 1024 && (head_dim == 64 || head_dim == 128 || head_dim == 256) &&
         page_size >= 16 && page_size <= 256 && (page_size & (page_size - 1)) == 0;
}

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

size_t dtype_bytes(spec_dtype t) { return t == SPEC_F32 ? 4 : 2; }

// The pages of a call.  `requests` is false for a batch of no requests, whose
// table is not looked at.
spec_status check_pages(const spec_cache_ctx* c, const spec_cache_pages* p, sv::CacheView* out) {
  if (!p || !p->pages || !p->table || p->num_pages < 0 || p->table_width < 0 ||
      p->table_stride < p->table_width)
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(p->pages, 16) || !aligned(p->table, 4) || (p->k_scale && !aligned(p->k_scale, 4)) ||
      (p->v_scale && !aligned(p->v_scale, 4)))
    return SPEC_ERR_UNSUPPORTED;
  out->pages = static_cast<uint8_t*>(p->pages);
  out->num_pages = p->num_pages;
  out->table = p->table;
  out->table_stride = p->table_stride;
  // positions are counted in 32 bits from a segment's first run
  out->capacity = std::min(static_cast<int64_t>(p->table_width) * c->page_size, kMaxPositions);
  out->heads = c->heads_kv;
  out->page_shift = log2_of(c->page_size);
  out->k_scale = p->k_scale;
  out->v_scale = p->v_scale;
  return SPEC_OK;
}

spec_status check_rows(const spec_cache_rows* r, spec_dtype dtype, sv::CacheRows* out) {
  if (!r || !r->data) return SPEC_ERR_INVALID_ARG;
  const int64_t unit = static_cast<int64_t>(16 / dtype_bytes(dtype));
  if (!aligned(r->data, 16) || r->stride_b % unit || r->stride_t % unit || r->stride_h % unit)
    return SPEC_ERR_UNSUPPORTED;
  const bool wide = aligned(r->data, 32) && r->stride_b % (2 * unit) == 0 && r->stride_t % (2 * unit) == 0 &&
                    r->stride_h % (2 * unit) == 0;
  *out = sv::CacheRows{r->data, r->stride_b, r->stride_t, r->stride_h, wide};
  return SPEC_OK;
}

// Launch the write (a warp per 64 channels of a run, keys or values) or the read
// (a warp per run).
template <bool WRITE, int D>
spec_status launch_move(sv::CacheMove& p, int64_t runs, spec_dtype dtype, cudaStream_t stream) {
  const int64_t warps = runs * p.c.heads * 2 * (WRITE ? D / 64 : 1);
  if (warps >= (int64_t{1} << 27)) return SPEC_ERR_INVALID_ARG;  // threads in 32 bits
  p.warps = static_cast<uint32_t>(warps);
  p.by_heads = sv::Quotient(static_cast<uint32_t>(p.c.heads));
  const dim3 grid(static_cast<unsigned>((warps * 32 + sv::kMoveThreads - 1) / sv::kMoveThreads), p.B);
  auto launch = [&](auto kernel) {
    return launch_waiting(kernel, grid, sv::kMoveThreads, 0, stream, p);
  };
  bool ok;
  if constexpr (WRITE)
    ok = dtype == SPEC_F32    ? launch(sv::k_cache_write<D, float>)
         : dtype == SPEC_BF16 ? launch(sv::k_cache_write<D, __nv_bfloat16>)
                              : launch(sv::k_cache_write<D, __half>);
  else
    ok = dtype == SPEC_F32    ? launch(sv::k_cache_read<D, float>)
         : dtype == SPEC_BF16 ? launch(sv::k_cache_read<D, __nv_bfloat16>)
                              : launch(sv::k_cache_read<D, __half>);
  return ok ? SPEC_OK : SPEC_ERR_CUDA;
}

template <bool WRITE>
spec_status move(spec_cache_ctx* c, const spec_cache_pages* cache, const spec_cache_rows* k,
                 const spec_cache_rows* v, spec_dtype dtype, const int32_t* start,
                 const int32_t* count, int B, int T, uint32_t* out_status, cudaStream_t stream) {
  if (!c || B < 0 || B > c->max_batch || T < 0) return SPEC_ERR_INVALID_ARG;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return SPEC_OK;
  if (WRITE && !start) return SPEC_ERR_INVALID_ARG;
  sv::CacheMove p{};
  if (spec_status st = check_pages(c, cache, &p.c); st != SPEC_OK) return st;
  if (spec_status st = check_rows(k, dtype, &p.k); st != SPEC_OK) return st;
  if (spec_status st = check_rows(v, dtype, &p.v); st != SPEC_OK) return st;
  if ((start && !aligned(start, 4)) || (count && !aligned(count, 4)) ||
      (out_status && !aligned(out_status, 4)))
    return SPEC_ERR_UNSUPPORTED;
  p.start = start;
  p.count = count;
  p.B = B;
  p.T = T;
  const int64_t runs = (static_cast<int64_t>(T) + 2 * (sv::kRun - 1)) / sv::kRun;  // a span may start anywhere in a run
  p.status = out_status;
  DeviceGuard g(c->device);
  if (!g.ok) return SPEC_ERR_CUDA;
  cudaGetLastError();
  if (c->head_dim == 64) return launch_move<WRITE, 64>(p, runs, dtype, stream);
  if (c->head_dim == 128) return launch_move<WRITE, 128>(p, runs, dtype, stream);
  return launch_move<WRITE, 256>(p, runs, dtype, stream);
}

// Query rows of a row tile at most: the accumulators of 128 (256) channels
// share 512 columns of tensor memory with the decoded tiles.
int max_rows(int head_dim) { return head_dim == 256 ? 32 : 64; }

bool prepare_attend(int head_dim) {
  return head_dim == 64    ? sv::attend_prepare<64>()
         : head_dim == 128 ? sv::attend_prepare<128>()
                           : sv::attend_prepare<256>();
}

}  // namespace

extern "C" {

spec_status spec_cache_page_bytes(int heads_kv, int head_dim, int page_size, size_t* bytes) {
  if (!bytes) return SPEC_ERR_INVALID_ARG;
  *bytes = 0;
  if (!geometry_ok(heads_kv, head_dim, page_size)) return SPEC_ERR_UNSUPPORTED;
  *bytes = static_cast<size_t>(heads_kv) * (page_size / sv::kRun) * sv::run_bytes(head_dim);
  return SPEC_OK;
}

spec_status spec_cache_init(spec_cache_ctx** out, int device, int max_batch, int heads_q,
                            int heads_kv, int head_dim, int page_size) {
  if (!out) return SPEC_ERR_INVALID_ARG;
  *out = nullptr;
  if (max_batch < 1 || max_batch > 65535 || heads_kv < 1 || heads_q < heads_kv || heads_q > 65535 ||
      heads_q % heads_kv != 0)
    return SPEC_ERR_INVALID_ARG;
  if (!geometry_ok(heads_kv, head_dim, page_size)) return SPEC_ERR_UNSUPPORTED;
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess) {
    cudaGetLastError();
    return SPEC_ERR_CUDA;
  }
  if (device < 0 || device >= ndev) return SPEC_ERR_INVALID_ARG;
  DeviceGuard g(device);
  if (!g.ok) return SPEC_ERR_CUDA;
  spec_cache_ctx* c = new (std::nothrow) spec_cache_ctx();
  if (!c) return SPEC_ERR_NOMEM;
  c->device = device;
  c->max_batch = max_batch;
  c->heads_q = heads_q;
  c->heads_kv = heads_kv;
  c->head_dim = head_dim;
  c->page_size = page_size;
  if (cudaDeviceGetAttribute(&c->num_sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) {
    delete c;
    return SPEC_ERR_CUDA;
  }
  // two cut segments per CTA (one CTA per SM): fp32 rows, their sums, the list of cuts
  const size_t rows = 2 * static_cast<size_t>(c->num_sms) * max_rows(head_dim);
  const size_t o_l = align_up(rows * head_dim * sizeof(float), 256);
  const size_t o_cuts = align_up(o_l + rows * sizeof(float2), 256);
  const size_t o_lost = align_up(o_cuts + c->num_sms * sizeof(sv::AttendCut), 256);
  const size_t o_err = align_up(o_lost + c->num_sms * sizeof(int), 256);
  if (c->num_sms > sv::kJoinMaxParts || cudaMalloc(&c->ws, o_err + 256) != cudaSuccess) {
    cudaGetLastError();
    delete c;
    return SPEC_ERR_NOMEM;
  }
  char* b = static_cast<char*>(c->ws);
  c->part_o = reinterpret_cast<float*>(b);
  c->part_l = reinterpret_cast<float2*>(b + o_l);
  c->cuts = reinterpret_cast<sv::AttendCut*>(b + o_cuts);
  c->lost = reinterpret_cast<int*>(b + o_lost);
  c->error = reinterpret_cast<unsigned*>(b + o_err);
  if (cudaMemset(c->error, 0, 256) != cudaSuccess || !prepare_attend(head_dim)) {
    cudaFree(c->ws);
    delete c;
    return SPEC_ERR_CUDA;
  }
  *out = c;
  return SPEC_OK;
}

spec_status spec_cache_destroy(spec_cache_ctx* c) {
  if (!c) return SPEC_OK;
  DeviceGuard g(c->device);
  cudaDeviceSynchronize();
  cudaFree(c->ws);
  delete c;
  return SPEC_OK;
}

spec_status spec_cache_write(spec_cache_ctx* c, const spec_cache_pages* cache,
                             const spec_cache_rows* k, const spec_cache_rows* v, spec_dtype dtype,
                             const int32_t* cache_len, const int32_t* block_len, int B, int T,
                             uint32_t* out_status, cudaStream_t stream) {
  return move<true>(c, cache, k, v, dtype, cache_len, block_len, B, T, out_status, stream);
}

spec_status spec_cache_read(spec_cache_ctx* c, const spec_cache_pages* cache,
                            const int32_t* start, const int32_t* count, int B, int T,
                            spec_dtype dtype, const spec_cache_rows* out_k,
                            const spec_cache_rows* out_v, uint32_t* out_status,
                            cudaStream_t stream) {
  return move<false>(c, cache, out_k, out_v, dtype, start, count, B, T, out_status, stream);
}

spec_status spec_cache_attend(spec_cache_ctx* c, const spec_cache_pages* cache,
                              const spec_cache_rows* q, spec_dtype dtype,
                              const int32_t* cache_len, const int32_t* block_len, int B, int T,
                              float scale, int causal, int window, const spec_cache_rows* out,
                              float* out_lse, uint32_t* out_status, cudaStream_t stream) {
  if (!c || B < 0 || B > c->max_batch || T < 0 || T > 65535 || window < 0 || !std::isfinite(scale))
    return SPEC_ERR_INVALID_ARG;
  if (dtype != SPEC_BF16 && dtype != SPEC_F16)
    return dtype == SPEC_F32 ? SPEC_ERR_UNSUPPORTED : SPEC_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return SPEC_OK;
  if (!cache_len) return SPEC_ERR_INVALID_ARG;
  sv::AttendParams p{};
  if (spec_status st = check_pages(c, cache, &p.c); st != SPEC_OK) return st;
  if (spec_status st = check_rows(q, dtype, &p.q); st != SPEC_OK) return st;
  if (spec_status st = check_rows(out, dtype, &p.out); st != SPEC_OK) return st;
  if (!aligned(cache_len, 4) || (block_len && !aligned(block_len, 4)) ||
      (out_lse && !aligned(out_lse, 4)) || (out_status && !aligned(out_status, 4)))
    return SPEC_ERR_UNSUPPORTED;
  p.cache_len = cache_len;
  p.block_len = block_len;
  p.B = B;
  p.T = T;
  p.heads_q = c->heads_q;
  p.group = c->heads_q / c->heads_kv;
  p.scale = scale;
  p.one = 1.0f;
  p.causal = causal != 0;
  p.window = window;
  p.lse = out_lse;
  p.status = out_status;
  p.bf16 = dtype == SPEC_BF16;
  p.by_group = sv::Quotient(static_cast<uint32_t>(p.group));
  // row tiles of equal size
  const int64_t rows = static_cast<int64_t>(T) * p.group;
  const int64_t tiles = (rows + max_rows(c->head_dim) - 1) / max_rows(c->head_dim);
  p.rp = static_cast<int>((rows + tiles - 1) / tiles);
  if (rows > INT_MAX - 64) return SPEC_ERR_INVALID_ARG;
  // One softmax thread has 8 or at least 16 rows.  3 against 6 tiles, 96 requests of
  // 64..4096 positions (width 256: ..2048), us, width 64 / 128 / 256:
  //    8 rows   74.9 : 78.4   74.1 : 76.7   40.3 : 44.1
  //   12 rows   91.7 : 84.5   89.3 : 82.9   51.6 : 48.7
  //   16 rows   97.5 : 85.7   89.4 : 83.3   52.8 : 49.2
  //   24 rows    115 : 93.1    106 : 91.3   62.3 : 53.4
  //   32 rows    141 : 115     128 : 114    72.6 : 60.4
  //   64 rows    205 : 168     191 : 167
  // 2, 4 and 8 are no better, but for contexts of 16..1000: 6 gains 2 us at 8 rows
  // too (37.8 : 35.3), and 8 some at 48 rows and more (width 128, 6 : 8, 72.7 : 65.4).
  p.seg_units = p.rp <= 8 ? 3 : 6;
  p.part_o = c->part_o;
  p.part_l = c->part_l;
  p.cuts = c->cuts;
  p.error = c->error;
  p.lost = c->lost;
  DeviceGuard g(c->device);
  if (!g.ok) return SPEC_ERR_CUDA;
  cudaGetLastError();
  const bool done = c->head_dim == 64    ? sv::attend_launch<64>(p, c->num_sms, stream)
                    : c->head_dim == 128 ? sv::attend_launch<128>(p, c->num_sms, stream)
                                         : sv::attend_launch<256>(p, c->num_sms, stream);
  return done && cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

spec_status spec_cache_errors(spec_cache_ctx* c, uint32_t* out) {
  if (!c || !out) return SPEC_ERR_INVALID_ARG;
  DeviceGuard g(c->device);
  if (cudaDeviceSynchronize() != cudaSuccess) return SPEC_ERR_CUDA;
  unsigned h = 0;
  if (cudaMemcpy(&h, c->error, sizeof h, cudaMemcpyDeviceToHost) != cudaSuccess) return SPEC_ERR_CUDA;
  *out = h;
  return SPEC_OK;
}

}  // extern "C"

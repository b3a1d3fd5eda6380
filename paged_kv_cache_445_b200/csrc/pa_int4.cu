// pa_int4.cu -- attention over the 4-bit paged KV cache.
//
// out[t, h] = sum_j softmax_j(scale q[t, h] . K_j) V_j over the keys the row
// sees, K and V read as (u - 8) s (pa_int4.cuh), gathered through the block
// table.  One pass over the keys with the running maximum and sum of the
// softmax ("Inference optimization", "Build it -- Step 2").
//
// Simple form: one CTA per (query row, query head), its warps taking every
// fourth key, a lane D / 32 dims.
#include "pa_device.cuh"
#include "pa_int4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int I4_WARPS = 4;

struct Int4Params {
  __nv_bfloat16* out;
  const __nv_bfloat16* q;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;  // nullptr: one row per sequence
  int num_seqs, num_rows, max_blocks, num_q_heads, num_kv_heads, group, block_shift, num_blocks;
  float scale_log2;
  int* status;
};

template <int D>
__device__ __forceinline__ float int4_value(const uint8_t* rec, int bs, int r, int dim) {
  const int c = dim >> 5, i = dim & 31;
  const uint8_t b = rec[int4_code_offset<D>(r, c) + 2 * (i & 7) + (i >> 4)];
  const float s = __half2float(*reinterpret_cast<const __half*>(rec + int4_scale_offset<D>(bs, r, c)));
  return static_cast<float>(((b >> (4 * ((i >> 3) & 1))) & 15) - 8) * s;
}

template <int D>
__global__ void __launch_bounds__(32 * I4_WARPS) int4_simple_kernel(const Int4Params p) {
  constexpr int N = D / 32;
  __shared__ float sm[I4_WARPS], sl[I4_WARPS], so[I4_WARPS][D];
  const int row = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int kh = h / p.group, bs = 1 << p.block_shift;
  int s = row, keys;
  if (p.query_start) {
    int lo = 0, hi = p.num_seqs - 1;  // the sequence that owns the row
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.query_start[mid] <= row) lo = mid; else hi = mid - 1;
    }
    s = lo;
    const int first = p.query_start[s], end = p.query_start[s + 1];
    if (row == 0 && h == 0) {
      for (int i = threadIdx.x; i < p.num_seqs; i += 32 * I4_WARPS)
        if (p.query_start[i] < 0 || p.query_start[i + 1] < p.query_start[i] || p.query_start[i + 1] > p.num_rows)
          set_status(p.status, PA_STATUS_BIT(PA_ERR_RANGE));
    }
    if (first < 0 || end > p.num_rows) return;
    if (row < first || row >= end) return;  // behind the last sequence: left alone
    keys = p.context_lens[s] - (p.query_start[s + 1] - row) + 1;
  } else {
    keys = p.context_lens[s];
  }
  if (keys > p.max_blocks << p.block_shift) {
    if (threadIdx.x == 0) set_status(p.status, PA_STATUS_BIT(PA_ERR_RANGE));
    keys = 0;
  }
  float q[N], o[N] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i)
    q[i] = __bfloat162float(p.q[(static_cast<long long>(row) * p.num_q_heads + h) * D + i * 32 + lane]);
  for (int j = warp; j < keys; j += I4_WARPS) {
    const int blk = p.block_tables[static_cast<long long>(s) * p.max_blocks + (j >> p.block_shift)];
    if (blk < 0 || blk >= p.num_blocks) {
      if (lane == 0) set_status(p.status, PA_STATUS_BIT(PA_ERR_RANGE));
      continue;
    }
    const long long rec = (static_cast<long long>(blk) * p.num_kv_heads + kh) * int4_record_bytes(bs, D);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) dot += q[i] * int4_value<D>(p.k_cache + rec, bs, j & (bs - 1), i * 32 + lane);
#pragma unroll
    for (int x = 16; x; x >>= 1) dot += __shfl_xor_sync(FULL_MASK, dot, x);
    dot *= p.scale_log2;
    const float mn = fmaxf(m, dot), a = exp2f(m - mn), w = exp2f(dot - mn);
    m = mn;
    l = l * a + w;
#pragma unroll
    for (int i = 0; i < N; ++i)
      o[i] = o[i] * a + w * int4_value<D>(p.v_cache + rec, bs, j & (bs - 1), i * 32 + lane);
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int i = 0; i < N; ++i) so[warp][i * 32 + lane] = o[i];
  __syncthreads();
  float mm = -INFINITY, ll = 0.f;
  for (int w = 0; w < I4_WARPS; ++w) mm = fmaxf(mm, sm[w]);
  for (int w = 0; w < I4_WARPS; ++w) ll += sl[w] != 0.f ? sl[w] * exp2f(sm[w] - mm) : 0.f;
  for (int d = threadIdx.x; d < D; d += 32 * I4_WARPS) {
    float x = 0.f;
    for (int w = 0; w < I4_WARPS; ++w) x += sl[w] != 0.f ? so[w][d] * exp2f(sm[w] - mm) : 0.f;
    p.out[(static_cast<long long>(row) * p.num_q_heads + h) * D + d] = __float2bfloat16(ll != 0.f ? x / ll : 0.f);
  }
}

int run_int4(void* out, const void* q, const int32_t* query_start, const void* k_cache, const void* v_cache,
             const int32_t* block_tables, int max_blocks, const int32_t* context_lens, int num_seqs, int total_rows,
             int num_q_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
             void* workspace, size_t workspace_bytes, int* dev_status, void* stream) {
  if (num_seqs < 0 || total_rows < 0 || max_blocks <= 0 || num_blocks <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
      num_q_heads % num_kv_heads)
    return PA_ERR_SHAPE;
  const int group = num_q_heads / num_kv_heads;
  if (block_size != 16 && block_size != 32) return PA_ERR_UNSUPPORTED;
  if (!rows_supported(group, head_dim)) return PA_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_blocks) * block_size > INT32_MAX) return PA_ERR_SHAPE;
  if (num_seqs == 0 || total_rows == 0) return PA_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !workspace) return PA_ERR_NULL;
  const auto ok = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; };
  if (!ok(out) || !ok(q) || !ok(k_cache) || !ok(v_cache) || !ok(workspace)) return PA_ERR_SHAPE;
  DeviceInfo di;
  const int rc = device_info(&di);
  if (rc != PA_OK) return rc;
  if (workspace_bytes < pa_int4_workspace_bytes(num_q_heads, num_kv_heads, head_dim)) return PA_ERR_WORKSPACE;
  Int4Params p{static_cast<__nv_bfloat16*>(out), static_cast<const __nv_bfloat16*>(q),
               static_cast<const uint8_t*>(k_cache), static_cast<const uint8_t*>(v_cache), block_tables, context_lens,
               query_start, num_seqs, total_rows, max_blocks, num_q_heads, num_kv_heads, group,
               block_size == 16 ? 4 : 5, num_blocks, scale * 1.4426950408889634f, dev_status};
  const dim3 grid(total_rows, num_q_heads);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (head_dim == 64) int4_simple_kernel<64><<<grid, 32 * I4_WARPS, 0, st>>>(p);
  else if (head_dim == 128) int4_simple_kernel<128><<<grid, 32 * I4_WARPS, 0, st>>>(p);
  else int4_simple_kernel<256><<<grid, 32 * I4_WARPS, 0, st>>>(p);
  return check_launch(cudaSuccess, "int4_simple_kernel launch");
}

}  // namespace

}  // namespace pa

extern "C" {

size_t pa_int4_workspace_bytes(int num_q_heads, int num_kv_heads, int head_dim) {
  if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads) return 0;
  if (!pa::rows_supported(num_q_heads / num_kv_heads, head_dim)) return 0;
  return 256;
}

int pa_decode_int4(void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                   int max_blocks_per_seq, const int32_t* context_lens, int num_seqs, int num_q_heads,
                   int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale, void* workspace,
                   size_t workspace_bytes, int* dev_status, void* stream) {
  return pa::run_int4(out, q, nullptr, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs,
                      num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, scale, workspace,
                      workspace_bytes, dev_status, stream);
}

int pa_prefill_chunk_int4(void* out, const void* q, const int32_t* query_start, const void* k_cache,
                          const void* v_cache, const int32_t* block_tables, int max_blocks_per_seq,
                          const int32_t* context_lens, int num_seqs, int total_q_tokens, int num_q_heads,
                          int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
                          void* workspace, size_t workspace_bytes, int* dev_status, void* stream) {
  if (!query_start && num_seqs > 0) return PA_ERR_NULL;
  return pa::run_int4(out, q, query_start, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs,
                      total_q_tokens, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, scale, workspace,
                      workspace_bytes, dev_status, stream);
}

}  // extern "C"

// pa_accept.cu -- verification of drafted tokens against the target's
// probabilities from given random numbers.
//
// "Inference optimization" (AI Engineering from Scratch, Phase 10 / 12),
// "Speculative decoding": draft token d of row r is kept with probability
// min(1, p_r(d) / q_r(d)); the first one refused is replaced by a draw from
// max(p_r - q_r, 0), normalised; if all are kept one more token is drawn from
// the last row's p.  With the uniform u given, the test is u q(d) < p(d) (both
// products exact in binary64) and the draw is the first index whose running
// sum of weights passes u times their total.
//
// Only the rows that decide a draw are read whole: one target row and, after a
// refusal, one draft row per sequence, V values each, so HBM bounds a full
// batch and latency a single chat.  One cluster of 2 to 8 CTAs per sequence: its
// warps take contiguous slices of the vocabulary, their sums meet in
// distributed shared memory, and the CTA whose slice holds the draw scans it
// again (from L1/L2).  128 sequences of 128,000 float values take 28 us (90 MB
// read, 14 us at the copy rate; the rest is the chain of loads before and after the
// sweep), one chat of 32,000 values 6 us.  No workspace, no atomics; sums are binary64, so the
// index does not depend on how they are split, short of rounding at 2^-53.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

namespace cg = cooperative_groups;

constexpr int ACC_THREADS = 512;
constexpr int ACC_WARPS = ACC_THREADS / 32;

struct AcceptParams {
  int32_t* out_tokens;
  int32_t* num_accepted;
  const void* target;
  const void* draft;  // nullptr: point masses
  long long target_stride, draft_stride;
  const int32_t* tokens;
  const int32_t* query_start;
  const float* uniforms;
  const int32_t* context_lens;  // may be nullptr
  int32_t* context_lens_out;
  int total_rows, vocab;
  int* status;
};

__device__ __forceinline__ float prob(const float* p) { return __ldg(p); }
__device__ __forceinline__ float prob(const __nv_bfloat16* p) { return __bfloat162float(*p); }

__device__ __forceinline__ float value_of(float x) { return x; }
__device__ __forceinline__ float value_of(__nv_bfloat16 x) { return __bfloat162float(x); }

// Which weights a draw uses.
enum Mode { FROM_TARGET, FROM_DIFFERENCE, FROM_OTHERS };

// A weight from the target's value and what is taken off it; negative, infinite and NaN ones weigh nothing.  Signs
// and ranges are told in binary32, where they are exact, the difference is taken in binary64, where it is.
__device__ __forceinline__ double weight_of(float t, float d) {
  const bool ok = t > d && t < INFINITY && d > -INFINITY;
  return static_cast<double>(ok ? t : 0.f) - static_cast<double>(ok ? d : 0.f);
}
template <class T>
__device__ __forceinline__ double weight(Mode mode, const T* t, const T* d, int refused, int v) {
  if (mode == FROM_OTHERS && v == refused) return 0.0;
  return weight_of(prob(t + v), mode == FROM_DIFFERENCE ? prob(d + v) : 0.f);
}

// Sum of the weights of [lo, hi) over the warp's lanes: max(t, d) - d, five instructions a value (binary64
// conversions bound the loop otherwise).  What may not weigh (NaN, infinities) shows in the sum, and the slice is then
// taken again with weight().  VEC values (16 bytes) per load.
template <class T, int VEC, bool DIFF>
__device__ __forceinline__ double slice_sum(const T* t, const T* d, int lo, int hi, int lane) {
  constexpr int STEP = 32 * VEC, UNROLL = 4;
  double sum = 0.0;
  const auto add = [&](T x, T y) {
    const float a = value_of(x), b = DIFF ? value_of(y) : 0.f;
    sum += DIFF ? static_cast<double>(fmaxf(a, b)) - static_cast<double>(b) : static_cast<double>(fmaxf(a, 0.f));
  };
  int v0 = lo + lane * VEC;
  for (; v0 - lane * VEC + STEP * UNROLL <= hi; v0 += STEP * UNROLL) {
    uint4 a[UNROLL], b[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if constexpr (VEC > 1) {
        a[u] = __ldg(reinterpret_cast<const uint4*>(t + v0 + u * STEP));
        if (DIFF) b[u] = __ldg(reinterpret_cast<const uint4*>(d + v0 + u * STEP));
      } else {
        *reinterpret_cast<T*>(&a[u]) = t[v0 + u * STEP];
        if (DIFF) *reinterpret_cast<T*>(&b[u]) = d[v0 + u * STEP];
      }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
#pragma unroll
      for (int k = 0; k < VEC; ++k) add(reinterpret_cast<const T*>(&a[u])[k], reinterpret_cast<const T*>(&b[u])[k]);
  }
  for (int v = v0 - lane * VEC + lane; v < hi; v += 32) add(t[v], DIFF ? d[v] : T(0.f));
  return sum;
}

// CTAS: CTAs per sequence, one cluster.
template <class T, int CTAS>
__global__ void __launch_bounds__(ACC_THREADS, 2) accept_kernel(const AcceptParams p) {
  constexpr int ACC_CTAS = CTAS, ACC_SLICES = CTAS * ACC_WARPS;
  __shared__ double sums[2][ACC_SLICES];  // double-buffered over the two passes a draw may take
  __shared__ int lasts[ACC_SLICES];       // last index with a weight in each slice, -1: none
  __shared__ double parts[ACC_WARPS];
  __shared__ int sh_acc, sh_mode, sh_refused;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int s = blockIdx.x / ACC_CTAS;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int start = p.query_start[s], end = p.query_start[s + 1];
  const int rows = end - start;
  if (start < 0 || end < start || end > p.total_rows) {  // uniform over the cluster: all its CTAs leave
    if (rank == 0 && tid == 0) {
      set_status(p.status, PA_STATUS_BIT(PA_ERR_RANGE));
      p.num_accepted[s] = 0;
      if (p.context_lens) p.context_lens_out[s] = p.context_lens[s];
      __threadfence();  // an attention kernel launched behind this one reads the lengths in its prologue
    }
    return;
  }
  if (rows == 0) {
    if (rank == 0 && tid == 0) {
      p.num_accepted[s] = 0;
      if (p.context_lens) p.context_lens_out[s] = p.context_lens[s];
      __threadfence();  // (as above)
    }
    return;
  }
  cluster.barrier_arrive();  // met before the first store into another CTA: that CTA has started then
  const T* target = static_cast<const T*>(p.target);
  const T* draft = static_cast<const T*>(p.draft);
  if (warp == 0) {
    int acc = rows - 1, refused = -1;
    bool found = false;
    for (int i0 = 0; i0 < rows - 1 && !found; i0 += 32) {
      const int i = i0 + lane;
      bool stop = false, ends = false;
      int d = 0;
      if (i < rows - 1) {
        const long long r = start + i;
        d = p.tokens[r + 1];
        if (d < 0 || d >= p.vocab) {  // negative: the drafts end here
          ends = stop = true;
          if (d >= 0 && rank == 0) set_status(p.status, PA_STATUS_BIT(PA_ERR_RANGE));
        } else {
          const double pt = prob(target + r * p.target_stride + d);
          const double qd = draft ? static_cast<double>(prob(draft + r * p.draft_stride + d)) : 1.0;
          stop = !(static_cast<double>(p.uniforms[r]) * qd < pt);
        }
      }
      const unsigned m = __ballot_sync(FULL_MASK, stop);
      if (m) {
        const int first = __ffs(m) - 1;
        acc = i0 + first;
        const int tok = __shfl_sync(FULL_MASK, d, first);
        const int e = __shfl_sync(FULL_MASK, ends ? 1 : 0, first);
        refused = e ? -1 : tok;
        found = true;
      }
    }
    if (lane == 0) {
      sh_acc = acc;
      sh_refused = refused;
      sh_mode = refused < 0 ? FROM_TARGET : draft ? FROM_DIFFERENCE : FROM_OTHERS;
    }
  }
  __syncthreads();
  const int acc = sh_acc, refused = sh_refused;
  Mode mode = static_cast<Mode>(sh_mode);
  const T* t = target + (start + static_cast<long long>(acc)) * p.target_stride;
  const T* d = draft ? draft + (start + static_cast<long long>(acc)) * p.draft_stride : nullptr;
  // slices: whole groups of 128 values per warp
  const int per = (p.vocab + ACC_SLICES * 128 - 1) / (ACC_SLICES * 128) * 128;
  const int mine = rank * ACC_WARPS + warp;
  const long long lo64 = static_cast<long long>(mine) * per;
  const int lo = static_cast<int>(lo64 < p.vocab ? lo64 : p.vocab);
  const int hi = static_cast<int>(lo64 + per < p.vocab ? lo64 + per : p.vocab);
  cluster.barrier_wait();
  double total = 0.0, before = 0.0, u = 0.0;
  int owner = -1;
  for (int pass = 0; pass < 2; ++pass) {
    double sum = 0.0;
    // (slices start at multiples of 128)
    const uintptr_t at = reinterpret_cast<uintptr_t>(t) | (mode == FROM_DIFFERENCE ? reinterpret_cast<uintptr_t>(d) : 0);
    constexpr int VEC = 16 / sizeof(T);
    if (mode == FROM_DIFFERENCE)
      sum = at % 16 == 0 ? slice_sum<T, VEC, true>(t, d, lo, hi, lane) : slice_sum<T, 1, true>(t, d, lo, hi, lane);
    else
      sum = at % 16 == 0 ? slice_sum<T, VEC, false>(t, d, lo, hi, lane) : slice_sum<T, 1, false>(t, d, lo, hi, lane);
    const bool odd = !(sum < INFINITY) || (mode == FROM_OTHERS && refused >= lo && refused < hi);
    if (__any_sync(FULL_MASK, odd)) {
      sum = 0.0;
      for (int v = lo + lane; v < hi; v += 32) sum += weight(mode, t, d, refused, v);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, o);
    if (lane < ACC_CTAS) *cluster.map_shared_rank(&sums[pass][mine], lane) = sum;  // to every CTA of the cluster
    cluster.sync();
    // every warp finds the slice that holds the draw
    double c[ACC_SLICES / 32], run = 0.0;
#pragma unroll
    for (int k = 0; k < ACC_SLICES / 32; ++k) {
      const int j = lane * (ACC_SLICES / 32) + k;
      run += sums[pass][j];
      c[k] = run;
    }
    double pre = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double x = __shfl_up_sync(FULL_MASK, pre, o);
      if (lane >= o) pre += x;
    }
    total = __shfl_sync(FULL_MASK, pre, 31);
    u = static_cast<double>(p.uniforms[end - 1]) * total;
    pre = __shfl_up_sync(FULL_MASK, pre, 1);  // sum before this lane's slices
    if (lane == 0) pre = 0.0;
    int hit = -1;
    double hit_before = 0.0;
#pragma unroll
    for (int k = ACC_SLICES / 32 - 1; k >= 0; --k)
      if (pre + c[k] > u && sums[pass][lane * (ACC_SLICES / 32) + k] > 0.0) {
        hit = lane * (ACC_SLICES / 32) + k;
        hit_before = pre + (k > 0 ? c[k - 1] : 0.0);
      }
    const unsigned m = __ballot_sync(FULL_MASK, hit >= 0);
    const int src = m ? __ffs(m) - 1 : 0;
    owner = m ? __shfl_sync(FULL_MASK, hit, src) : -1;
    before = __shfl_sync(FULL_MASK, hit_before, src);
    if (total > 0.0 || mode == FROM_TARGET) break;
    mode = FROM_TARGET;  // the draft leaves nothing of the target: draw from the target
  }
  // rows after the draw, the counts; the draw itself comes from one warp
  if (rank == 0) {
    for (int i = tid; i < rows; i += ACC_THREADS)
      if (i != acc) p.out_tokens[start + i] = i < acc ? p.tokens[start + i + 1] : -1;
    if (tid == 0) {
      p.num_accepted[s] = acc;
      if (p.context_lens) p.context_lens_out[s] = p.context_lens[s] - (rows - 1 - acc);
      __threadfence();  // (as above)
    }
  }
  if (owner < 0) {  // u times the total is not passed (rounding, u >= 1): the last token with a weight
    int last = -1;
    for (int v = lo + lane; v < hi; v += 32)
      if (weight(mode, t, d, refused, v) > 0.0) last = v;
#pragma unroll
    for (int o = 16; o; o >>= 1) last = max(last, __shfl_xor_sync(FULL_MASK, last, o));
    if (lane == 0) *cluster.map_shared_rank(&lasts[mine], 0) = last;
    cluster.sync();
    if (rank == 0 && warp == 0) {
      last = -1;
      for (int j = lane; j < ACC_SLICES; j += 32) last = max(last, lasts[j]);
#pragma unroll
      for (int o = 16; o; o >>= 1) last = max(last, __shfl_xor_sync(FULL_MASK, last, o));
      if (lane == 0) {
        p.out_tokens[start + acc] = last;
        if (last < 0) set_status(p.status, PA_STATUS_BIT(PA_ERR_RANGE));
      }
    }
  } else if (owner / ACC_WARPS == rank) {
    // The slice that holds the draw, again: its CTA's warps take a part each, the one whose part passes u scans it.
    const long long from = static_cast<long long>(owner) * per;
    const int to = static_cast<int>(from + per < p.vocab ? from + per : p.vocab);
    const int part = (to - static_cast<int>(from) + ACC_WARPS * 128 - 1) / (ACC_WARPS * 128) * 128;
    const int a = min(static_cast<int>(from) + warp * part, to), b = min(a + part, to);
    double sum = 0.0;
    for (int v = a + lane; v < b; v += 32) sum += weight(mode, t, d, refused, v);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(FULL_MASK, sum, o);
    if (lane == 0) parts[warp] = sum;
    __syncthreads();
    int win = -1;  // rounding may leave no part past u: then the last one with a weight
    double run = before, at = before;
    for (int w = 0; w < ACC_WARPS; ++w) {
      if (parts[w] > 0.0 && (win < 0 || !(at + parts[win] > u))) win = w, at = run;
      run += parts[w];
    }
    if (win == warp) {
      int token = -1, last = -1;
      for (int v0 = a; v0 < b && token < 0; v0 += 128) {
        double w[4], mine4 = 0.0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int v = v0 + lane * 4 + k;
          w[k] = v < b ? weight(mode, t, d, refused, v) : 0.0;
          mine4 += w[k];
        }
        double pre = mine4;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double x = __shfl_up_sync(FULL_MASK, pre, o);
          if (lane >= o) pre += x;
        }
        const double all = __shfl_sync(FULL_MASK, pre, 31);
        double c = __shfl_up_sync(FULL_MASK, pre, 1);
        c = at + (lane == 0 ? 0.0 : c);
        int hit = -1;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          c += w[k];
          if (w[k] > 0.0) last = v0 + lane * 4 + k;
          if (hit < 0 && w[k] > 0.0 && c > u) hit = v0 + lane * 4 + k;
        }
        const unsigned m = __ballot_sync(FULL_MASK, hit >= 0);
        if (m) token = __shfl_sync(FULL_MASK, hit, __ffs(m) - 1);
        at += all;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) last = max(last, __shfl_xor_sync(FULL_MASK, last, o));
      if (lane == 0) p.out_tokens[start + acc] = token >= 0 ? token : last;
    }
  }
}

template <class T, int ACC_CTAS>
int launch_accept(const AcceptParams& p, int num_seqs, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(num_seqs) * ACC_CTAS);
  cfg.blockDim = dim3(ACC_THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ACC_CTAS;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return check_launch(cudaLaunchKernelEx(&cfg, accept_kernel<T, ACC_CTAS>, p), "accept_kernel launch");
}

}  // namespace

}  // namespace pa

extern "C" int pa_accept_drafts(int32_t* out_tokens, int32_t* num_accepted, const void* target_probs,
                                long long target_stride, const void* draft_probs, long long draft_stride,
                                int probs_bf16, const int32_t* tokens, const int32_t* query_start,
                                const float* uniforms, int num_seqs, int total_rows, int vocab,
                                const int32_t* context_lens, int32_t* context_lens_out, int* dev_status,
                                void* stream) {
  if (num_seqs < 0 || total_rows < 0 || vocab <= 0 || target_stride < vocab) return PA_ERR_SHAPE;
  if (draft_probs && draft_stride < vocab) return PA_ERR_SHAPE;
  if (num_seqs > INT32_MAX / 8 || vocab > pa::PA_MAX_COUNT) return PA_ERR_SHAPE;
  if ((context_lens == nullptr) != (context_lens_out == nullptr)) return PA_ERR_NULL;
  if (num_seqs == 0) return PA_OK;
  if (!num_accepted || !query_start) return PA_ERR_NULL;
  if (total_rows > 0 && (!out_tokens || !target_probs || !tokens || !uniforms)) return PA_ERR_NULL;
  pa::DeviceInfo di;
  const int rc = pa::device_info(&di);
  if (rc != PA_OK) return rc;
  pa::AcceptParams p{out_tokens, num_accepted, target_probs, draft_probs, target_stride, draft_stride, tokens,
                     query_start, uniforms, context_lens, context_lens_out, total_rows, vocab, dev_status};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // As many CTAs a sequence as keep the batch in one wave (two CTAs fit an SM), 8 at most.  With 2, 4 and 8 of them 128
  // sequences of 128,000 values take 28.1, 28.7 and 35.5 us, 64 20.5, 17.0 and 22.0, 37 16.5, 14.4 and 14.9, 16 15.4,
  // 11.7 and 10.4; 128 of 32,000 values 12.2, 16.5 and 26.2.
  const int room = 2 * di.num_sms / num_seqs;
  const auto launch = room >= 8   ? probs_bf16 ? pa::launch_accept<__nv_bfloat16, 8> : pa::launch_accept<float, 8>
                      : room >= 4 ? probs_bf16 ? pa::launch_accept<__nv_bfloat16, 4> : pa::launch_accept<float, 4>
                                  : probs_bf16 ? pa::launch_accept<__nv_bfloat16, 2> : pa::launch_accept<float, 2>;
  return launch(p, num_seqs, st);
}

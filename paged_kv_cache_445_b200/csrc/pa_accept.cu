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
// batch and latency a single chat.  One cluster of 8 CTAs per sequence: 128
// warps take contiguous slices of the vocabulary, their sums meet in
// distributed shared memory, and the warp whose slice holds the draw scans it
// again (from L1/L2).  No workspace, no atomics; sums are binary64, so the
// index does not depend on how they are split, short of rounding at 2^-53.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

namespace cg = cooperative_groups;

constexpr int ACC_CTAS = 8;      // per sequence (one cluster)
constexpr int ACC_THREADS = 512;
constexpr int ACC_WARPS = ACC_THREADS / 32;
constexpr int ACC_SLICES = ACC_CTAS * ACC_WARPS;

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

// Which weights a draw uses.
enum Mode { FROM_TARGET, FROM_DIFFERENCE, FROM_OTHERS };

// Weight of token v: the target's probability, what the draft leaves of it, or
// zero for the refused token.  Negative, infinite and NaN values weigh nothing.
template <class T>
__device__ __forceinline__ double weight(Mode mode, const T* t, const T* d, int refused, int v) {
  double w = prob(t + v);
  if (mode == FROM_DIFFERENCE) w -= static_cast<double>(prob(d + v));
  if (mode == FROM_OTHERS && v == refused) w = 0.0;
  return w > 0.0 && w < INFINITY ? w : 0.0;
}

template <class T>
__global__ void __launch_bounds__(ACC_THREADS) accept_kernel(const AcceptParams p) {
  __shared__ double sums[2][ACC_SLICES];  // double-buffered over the two passes a draw may take
  __shared__ int lasts[2][ACC_SLICES];    // last index with a weight in each slice, -1: none
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
    }
    return;
  }
  if (rows == 0) {
    if (rank == 0 && tid == 0) {
      p.num_accepted[s] = 0;
      if (p.context_lens) p.context_lens_out[s] = p.context_lens[s];
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
  int owner = -1, last = -1;
  for (int pass = 0; pass < 2; ++pass) {
    double sum = 0.0;
    int at = -1;
    for (int v = lo + lane; v < hi; v += 32) {
      const double w = weight(mode, t, d, refused, v);
      sum += w;
      if (w > 0.0) at = v;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      sum += __shfl_xor_sync(FULL_MASK, sum, o);
      at = max(at, __shfl_xor_sync(FULL_MASK, at, o));
    }
    if (lane < ACC_CTAS) {  // to every CTA of the cluster
      cluster.map_shared_rank(&sums[pass][mine], lane)[0] = sum;
      cluster.map_shared_rank(&lasts[pass][mine], lane)[0] = at;
    }
    cluster.sync();
    // every warp finds the slice that holds the draw
    double c[ACC_SLICES / 32], run = 0.0;
    int l = -1;
#pragma unroll
    for (int k = 0; k < ACC_SLICES / 32; ++k) {
      const int j = lane * (ACC_SLICES / 32) + k;
      run += sums[pass][j];
      c[k] = run;
      l = max(l, lasts[pass][j]);
    }
    double pre = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double x = __shfl_up_sync(FULL_MASK, pre, o);
      if (lane >= o) pre += x;
      l = max(l, __shfl_xor_sync(FULL_MASK, l, o));
    }
    total = __shfl_sync(FULL_MASK, pre, 31);
    last = l;
    u = static_cast<double>(p.uniforms[end - 1]) * total;
    pre = __shfl_up_sync(FULL_MASK, pre, 1);  // sum before this lane's slices
    if (lane == 0) pre = 0.0;
    int hit = -1;
    double hit_before = 0.0;
#pragma unroll
    for (int k = ACC_SLICES / 32 - 1; k >= 0; --k)
      if (pre + c[k] > u && lasts[pass][lane * (ACC_SLICES / 32) + k] >= 0) {
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
      __threadfence();  // an attention kernel launched behind this one reads the lengths in its prologue
    }
  }
  if (owner < 0) {  // u times the total is not passed (rounding, u >= 1): the last token with a weight
    if (rank == 0 && tid == 0) {
      p.out_tokens[start + acc] = last;
      if (last < 0) set_status(p.status, PA_STATUS_BIT(PA_ERR_RANGE));
    }
  } else if (owner == mine) {
    int token = -1;
    double sum = before;
    for (int v0 = lo; v0 < hi && token < 0; v0 += 128) {
      double w[4], run = 0.0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int v = v0 + lane * 4 + k;
        w[k] = v < hi ? weight(mode, t, d, refused, v) : 0.0;
        run += w[k];
      }
      double pre = run;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double x = __shfl_up_sync(FULL_MASK, pre, o);
        if (lane >= o) pre += x;
      }
      const double all = __shfl_sync(FULL_MASK, pre, 31);
      double at = __shfl_up_sync(FULL_MASK, pre, 1);
      at = sum + (lane == 0 ? 0.0 : at);
      int hit = -1;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        at += w[k];
        if (hit < 0 && w[k] > 0.0 && at > u) hit = v0 + lane * 4 + k;
      }
      const unsigned m = __ballot_sync(FULL_MASK, hit >= 0);
      if (m) token = __shfl_sync(FULL_MASK, hit, __ffs(m) - 1);
      sum += all;
    }
    if (lane == 0) {
      const int slice_last = lasts[mode == static_cast<Mode>(sh_mode) ? 0 : 1][mine];
      p.out_tokens[start + acc] = token >= 0 ? token : slice_last;
    }
  }
}

template <class T>
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
  return check_launch(cudaLaunchKernelEx(&cfg, accept_kernel<T>, p), "accept_kernel launch");
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
  if (num_seqs > INT32_MAX / pa::ACC_CTAS) return PA_ERR_SHAPE;
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
  return probs_bf16 ? pa::launch_accept<__nv_bfloat16>(p, num_seqs, st) : pa::launch_accept<float>(p, num_seqs, st);
}

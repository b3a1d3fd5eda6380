// pa_slots.cu -- block tables, positions and slot mapping of a step, built on
// the GPU from request lengths.
//
// The host allocator's bookkeeping ("vLLM serving internals", AI Engineering
// from Scratch, Phase 17 / 04, "PagedAttention as a virtual memory system": a
// sequence takes a block when its last one is full, a finished one returns
// its blocks) as three prefix sums over the batch:
//   rows(s)  = max(n_s, 0)                        -> query_start
//   need(s)  = max(0, ceil((ctx + n) / bs) - held) -> place in the free queue
//   back(s)  = blocks past the new end, n_s < 0    -> place at the queue's tail
// Row t of sequence s then has position ctx + i and slot table[pos / bs] * bs
// + pos % bs, where a new block's ID is read straight from the queue.
//
// A few bytes per row: bound by launch and dependent-load latency (4.2 us for 128
// decodes, 16 us for 2000 requests and a buffer of 264,000 rows).  Every CTA
// scans the whole batch (tiles of one sequence per thread) and writes its share
// of the rows, found by binary search in the tile's row ends.  The lengths and
// the queue state may be updated in place, so they are written only when every
// CTA has read them: after the barrier of one cluster of up to 8 CTAs, or, for
// row buffers that keep more CTAs busy, by a second launch.  Written elsewhere,
// they need neither.
#include <cooperative_groups.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

namespace cg = cooperative_groups;

constexpr int SLOT_MAX_CTAS = 8;        // of a cluster
constexpr int SLOT_ROWS_PER_CTA = 2048;  // below that a second CTA only repeats the scan

// What a launch writes; APART: the lengths and the queue state go elsewhere than they came from, so nothing is waited
// for before they are written.
enum SlotsPart { SLOTS_ROWS = 1, SLOTS_STATE = 2, SLOTS_APART = 4 };

struct SlotsParams {
  const int32_t* new_tokens;
  const int32_t* context_lens;
  const int32_t* blocks_held;
  int32_t* context_lens_out;
  int32_t* blocks_held_out;
  int32_t* block_tables;
  int32_t* free_blocks;
  const int32_t* free_state;
  int32_t* free_state_out;
  int32_t* query_start;
  int32_t* positions;
  int32_t* slots;
  int num_seqs, max_blocks, num_blocks, block_shift, max_tokens;
  int* status;
};

// What a sequence asks for, and its prefix sums over the batch.
struct Seq {
  long long rows_end, need_end, back_end;  // inclusive
  int n, ctx, held, need, back;
  bool served;  // n >= 0 and it gets what it needs
  bool drops;   // n < 0 and valid
};

struct Carry {
  long long rows, need, back;
};

template <int THREADS>
struct SlotsShared {
  long long warp[3][THREADS / 32];
  long long rows_end[THREADS];  // inclusive prefix of the rows
  int ctx[THREADS];
  int held[THREADS];            // -1: the sequence is refused
  int first[THREADS];           // queue place of its first new block
  int taken;                    // blocks taken so far
};

__device__ __forceinline__ long long warp_inclusive(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(FULL_MASK, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Sum of the totals of the warps before this one, and of all WARPS: every warp scans them itself.
template <int WARPS>
__device__ __forceinline__ long long before_warp(const long long* totals, int warp, int lane, long long& all) {
  const long long incl = warp_inclusive(lane < WARPS ? totals[lane] : 0, lane);
  all = __shfl_sync(FULL_MASK, incl, 31);
  const long long x = __shfl_sync(FULL_MASK, incl, warp > 0 ? warp - 1 : 0);
  return warp > 0 ? x : 0;
}

// Load sequence s of the tile and scan the tile; `carry` moves to its end.
template <int THREADS>
__device__ Seq scan_tile(const SlotsParams& p, SlotsShared<THREADS>& sh, int s, int count, bool bad_queue, Carry& carry) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Seq q{};
  int bits = 0;
  bool fits = false;
  if (s < p.num_seqs) {
    q.n = p.new_tokens[s];
    q.ctx = p.context_lens[s];
    q.held = p.blocks_held[s];
    const long long after = static_cast<long long>(q.ctx) + q.n;
    const long long round = (1ll << p.block_shift) - 1;
    const long long now_blocks = (static_cast<long long>(q.ctx) + round) >> p.block_shift;
    const long long blocks = (after + round) >> p.block_shift;
    if (q.ctx < 0 || q.held < now_blocks || q.held > p.max_blocks || after < 0) {
      bits |= PA_STATUS_BIT(PA_ERR_RANGE);
    } else if (q.n < 0) {
      q.drops = !bad_queue;
      q.back = q.drops ? static_cast<int>(q.held - blocks) : 0;
    } else if (blocks > p.max_blocks) {
      bits |= PA_STATUS_BIT(PA_ERR_RANGE);
    } else {
      fits = true;
      q.need = blocks > q.held ? static_cast<int>(blocks - q.held) : 0;
    }
  }
  // rows first: a sequence whose rows pass the row buffer is refused and needs no block
  long long v = warp_inclusive(q.n > 0 ? q.n : 0, lane);
  if (lane == 31) sh.warp[0][warp] = v;
  __syncthreads();
  long long total;
  const long long base = carry.rows + before_warp<THREADS / 32>(sh.warp[0], warp, lane, total);
  q.rows_end = base + v;
  carry.rows += total;
  if (fits && q.rows_end > p.max_tokens) {
    fits = false;
    q.need = 0;
    bits |= PA_STATUS_BIT(PA_ERR_RANGE);
  }
  const long long nv = warp_inclusive(q.need, lane);
  const long long bv = warp_inclusive(q.back, lane);
  if (lane == 31) {
    sh.warp[1][warp] = nv;
    sh.warp[2][warp] = bv;
  }
  __syncthreads();
  long long nt, bt;
  const long long nb = carry.need + before_warp<THREADS / 32>(sh.warp[1], warp, lane, nt);
  const long long bb = carry.back + before_warp<THREADS / 32>(sh.warp[2], warp, lane, bt);
  q.need_end = nb + nv;
  q.back_end = bb + bv;
  carry.need += nt;
  carry.back += bt;
  q.served = fits && (q.need == 0 || q.need_end <= count);
  if (fits && !q.served) bits |= PA_STATUS_BIT(PA_ERR_NO_BLOCKS);
  if (bits) set_status(p.status, bits);
  if (q.served && q.need > 0) atomicMax(&sh.taken, static_cast<int>(q.need_end));
  return q;
}

__device__ __forceinline__ void write_seq(const SlotsParams& p, int s, const Seq& q) {
  if (s >= p.num_seqs) return;
  p.context_lens_out[s] = q.served || q.drops ? q.ctx + q.n : q.ctx;
  p.blocks_held_out[s] = q.held + (q.served ? q.need : 0) - q.back;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) slots_kernel(const SlotsParams p, int parts) {
  constexpr int SLOT_THREADS = THREADS;
  __shared__ SlotsShared<THREADS> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x, ctas = gridDim.x;
  int head = p.free_state[0], count = p.free_state[1];
  const bool bad_queue = head < 0 || head >= p.num_blocks || count < 0 || count > p.num_blocks;
  if (bad_queue) {
    if (tid == 0 && (parts & SLOTS_ROWS)) set_status(p.status, PA_STATUS_BIT(PA_ERR_RANGE));
    head = count = 0;
  }
  if (tid == 0) sh.taken = 0;
  __syncthreads();
  Carry carry{0, 0, 0};
  const int tiles = (p.num_seqs + SLOT_THREADS - 1) / SLOT_THREADS;
  const int bs = 1 << p.block_shift;
  Seq q{};
  if (rank == 0 && tid == 0) p.query_start[0] = 0;
  for (int tile = 0; tile < tiles && (parts & SLOTS_ROWS); ++tile) {
    const int s = tile * SLOT_THREADS + tid;
    const long long first_row = carry.rows;
    q = scan_tile(p, sh, s, count, bad_queue, carry);
    sh.rows_end[tid] = q.rows_end;
    sh.ctx[tid] = q.ctx;
    sh.held[tid] = q.served ? q.held : -1;
    sh.first[tid] = static_cast<int>(q.need_end - q.need);
    if (rank == tile % ctas && s < p.num_seqs)
      p.query_start[s + 1] = static_cast<int>(q.rows_end < INT32_MAX ? q.rows_end : INT32_MAX);
    __syncthreads();
    // rows of this tile's sequences
    const long long last_row = carry.rows < p.max_tokens ? carry.rows : p.max_tokens;
    for (long long t = first_row + rank * SLOT_THREADS + tid; t < last_row; t += ctas * SLOT_THREADS) {
      int lo = 0, hi = SLOT_THREADS - 1;  // first sequence whose rows end after t
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (sh.rows_end[mid] > t) hi = mid; else lo = mid + 1;
      }
      const int held = sh.held[lo];
      int pos = -1, slot = -1;
      if (held >= 0) {
        const long long start = lo > 0 ? sh.rows_end[lo - 1] : first_row;
        pos = sh.ctx[lo] + static_cast<int>(t - start);
        const int blk = pos >> p.block_shift;
        int32_t* entry = p.block_tables + static_cast<long long>(tile * SLOT_THREADS + lo) * p.max_blocks + blk;
        int id;
        if (blk >= held) {
          long long at = static_cast<long long>(head) + sh.first[lo] + (blk - held);
          if (at >= p.num_blocks) at -= p.num_blocks;
          id = p.free_blocks[at];
          if ((pos & (bs - 1)) == 0) *entry = id;  // a new block's first position is always one of the rows
        } else {
          id = *entry;
        }
        if (id >= 0 && id < p.num_blocks)
          slot = (id << p.block_shift) + (pos & (bs - 1));
        else
          set_status(p.status, PA_STATUS_BIT(PA_ERR_RANGE));
      }
      p.positions[t] = pos;
      p.slots[t] = slot;
    }
    __syncthreads();
    // released blocks: one warp per sequence
    sh.held[tid] = q.held;
    sh.first[tid] = q.back;
    sh.rows_end[tid] = q.back_end - q.back;
    const int any = __syncthreads_or(q.back > 0);
    if (any) {
      for (int i = warp * ctas + rank; i < SLOT_THREADS; i += ctas * (SLOT_THREADS / 32)) {
        const int back = sh.first[i];
        const int32_t* row = p.block_tables + static_cast<long long>(tile * SLOT_THREADS + i) * p.max_blocks;
        for (int k = lane; k < back; k += 32) {
          const long long place = count + sh.rows_end[i] + k;
          if (place >= p.num_blocks) {  // more blocks than the pool has: the caller's state is wrong
            set_status(p.status, PA_STATUS_BIT(PA_ERR_RANGE));
            continue;
          }
          long long at = head + place;
          if (at >= p.num_blocks) at -= p.num_blocks;
          const int id = row[sh.held[i] - back + k];
          if (id < 0 || id >= p.num_blocks) set_status(p.status, PA_STATUS_BIT(PA_ERR_RANGE));  // queued all the same
          p.free_blocks[at] = id;
        }
      }
    }
    __syncthreads();
  }
  // rows behind the last sequence are padding
  if (parts & SLOTS_ROWS) {
    for (long long t = carry.rows + rank * SLOT_THREADS + tid; t < p.max_tokens; t += ctas * SLOT_THREADS) {
      p.positions[t] = -1;
      p.slots[t] = -1;
    }
  }
  // An attention kernel launched behind this one reads offsets and lengths in its prologue, once every CTA here has
  // ended but before it waits for their stores: every path fences what it wrote (CTA 0 with outputs apart at its end).
  if (rank != 0 || (parts & SLOTS_STATE) == 0 || (parts & SLOTS_APART) == 0) __threadfence();
  if (!(parts & SLOTS_STATE)) return;
  // every CTA has read the lengths and the queue state: now they may change
  if (parts & SLOTS_ROWS) {
    if (!(parts & SLOTS_APART)) cg::this_cluster().sync();
    if (rank != 0) return;
  }
  if (tiles == 1 && (parts & SLOTS_ROWS)) {
    write_seq(p, tid, q);
  } else {
    carry = Carry{0, 0, 0};
    SlotsParams quiet = p;
    quiet.status = nullptr;
    for (int tile = 0; tile < tiles; ++tile) {
      const int s = tile * SLOT_THREADS + tid;
      q = scan_tile(quiet, sh, s, count, bad_queue, carry);
      write_seq(p, s, q);
      __syncthreads();
    }
  }
  __syncthreads();
  if (tid == 0) {
    const int taken = sh.taken;
    const long long left = count - taken + carry.back;
    int at = head + taken;
    if (at >= p.num_blocks) at -= p.num_blocks;
    if (!bad_queue) {
      p.free_state_out[0] = at;
      p.free_state_out[1] = static_cast<int>(left < p.num_blocks ? left : p.num_blocks);
    } else {
      p.free_state_out[0] = p.free_state[0];
      p.free_state_out[1] = p.free_state[1];
    }
  }
  __threadfence();  // (as above)
}

}  // namespace

}  // namespace pa

extern "C" int pa_step_slots(const int32_t* new_tokens, const int32_t* context_lens, int32_t* context_lens_out,
                             const int32_t* blocks_held, int32_t* blocks_held_out, int32_t* block_tables,
                             int max_blocks_per_seq, int32_t* free_blocks, const int32_t* free_state,
                             int32_t* free_state_out, int num_seqs, int num_blocks, int block_size,
                             int32_t* query_start, int32_t* positions, int32_t* slot_mapping, int max_tokens,
                             int* dev_status, void* stream) {
  if (num_seqs < 0 || num_blocks <= 0 || max_blocks_per_seq <= 0 || max_tokens < 0) return PA_ERR_SHAPE;
  if (num_seqs > pa::PA_MAX_COUNT) return PA_ERR_SHAPE;
  if (block_size != 16 && block_size != 32) return PA_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_blocks) * block_size > INT32_MAX) return PA_ERR_SHAPE;  // slots are int32
  if (static_cast<long long>(max_blocks_per_seq) * block_size > INT32_MAX) return PA_ERR_SHAPE;
  if (num_seqs > 0 && (!new_tokens || !context_lens || !context_lens_out || !blocks_held || !blocks_held_out ||
                       !block_tables))
    return PA_ERR_NULL;
  if (!free_blocks || !free_state || !free_state_out || !query_start) return PA_ERR_NULL;
  if (max_tokens > 0 && (!positions || !slot_mapping)) return PA_ERR_NULL;
  pa::DeviceInfo di;
  const int rc = pa::device_info(&di);
  if (rc != PA_OK) return rc;
  pa::SlotsParams p{new_tokens,     context_lens, blocks_held, context_lens_out, blocks_held_out, block_tables,
                    free_blocks,    free_state,   free_state_out, query_start,   positions,       slot_mapping,
                    num_seqs,       max_blocks_per_seq, num_blocks, block_size == 16 ? 4 : 5, max_tokens, dev_status};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int ctas = static_cast<int>((static_cast<long long>(max_tokens) + pa::SLOT_ROWS_PER_CTA - 1) / pa::SLOT_ROWS_PER_CTA);
  const bool apart = context_lens_out != context_lens && blocks_held_out != blocks_held && free_state_out != free_state;
  if (ctas > pa::SLOT_MAX_CTAS) {  // 264,000 rows: 55 us as one cluster, 18 as two launches over the GPU, 16 as one
    ctas = max_tokens / 1024 < di.num_sms ? max_tokens / 1024 : di.num_sms;
    const int rows = pa::SLOTS_ROWS | (apart ? pa::SLOTS_STATE | pa::SLOTS_APART : 0);
    pa::slots_kernel<1024><<<ctas, 1024, 0, st>>>(p, rows);
    const int r = pa::check_launch(cudaSuccess, "slots_kernel launch");
    if (r != PA_OK || apart) return r;
    pa::slots_kernel<1024><<<1, 1024, 0, st>>>(p, pa::SLOTS_STATE);
    return pa::check_launch(cudaSuccess, "slots_kernel launch");
  }
  if (ctas < 1) ctas = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int parts = pa::SLOTS_ROWS | pa::SLOTS_STATE | (apart ? pa::SLOTS_APART : 0);
  // a small batch: fewer warps to wait for at each of the scan's barriers
  const bool small = num_seqs <= 256 && max_tokens <= 1024;
  cfg.blockDim = dim3(small ? 256 : 1024);
  return pa::check_launch(cudaLaunchKernelEx(&cfg, small ? pa::slots_kernel<256> : pa::slots_kernel<1024>, p, parts),
                          "slots_kernel launch");
}

// pa_int4.cu -- attention over the 4-bit paged KV cache.
//
// out[t, h] = sum_j softmax_j(scale q[t, h] . K_j) V_j over the keys the row
// sees, K and V read as (u - 8) s (pa_int4.cuh), gathered through the block
// table.  One pass over the keys with the running maximum and sum of the
// softmax ("Inference optimization", "Build it -- Step 2").
//
// The cache is read once: 2 D * 9/16 bytes per token and KV head, so HBM is the
// floor.  Unpacking sets the pace beside it: every code passes the integer pipe,
// which takes half an instruction a cycle, so what counts below is instructions
// per code.  On 128 sequences (lognormal lengths, 64 query and 8 KV heads, 263,000
// tokens, 304 MB) the kernel takes 78 us, 3.9 TB/s of codes and scales; a copy of
// it that only streams takes 62, one that only computes 72.
//
// Work: an item is (sequence, group of query rows, KV head); its columns are the
// rows times the G query heads, 8 or 16 (NT n-tiles of 8).  Its keys are cut
// into units of 64 (32 where O takes the registers).  All units of the batch, in
// order, are cut into equal contiguous ranges, one per CTA, and a CTA's range
// into one per warp; each warp streams its own units through a ring of record
// copies (a record is one contiguous run of bytes, so plain bulk copies bring it).
// Eight warps of up to 255 registers a CTA, one CTA an SM: 64 keys a turn give a
// warp enough independent instructions, where 12 or 16 warps of 32-key units took
// 79 and 85 us.
//
// Math, on fp16 warp MMAs with fp32 accumulators, keys or head dims in M and
// the columns in N:
//  - a nibble masked out of its word is an fp16 subnormal, u 2^-24 or u 2^-20 by
//    its place, and an MMA takes it as it is: five integer instructions per 8
//    codes, no conversion (masking in an exponent and subtracting its constant
//    took 9).  The powers of two go into q and into the output's scale.
//    (The tensor core adds a step's products on one grid that the exponent fields
//    give, and a subnormal's field stands for 2^-14: in units of P s the grid is 2^-15
//    of the step's largest one for the even nibbles, 2^-19 for the odd ones, as
//    measured; bf16 keeps 2^-8.)
//  - S = K q: a chunk's 32 dims share a scale, S += s S_chunk.  The codes' 8 too
//    many are one more product, of the chunks' scales with -8 sum(q) (split in a
//    high and a low fp16 part: 22 bits).
//  - q enters as fp16 scaled by a power of two per column (exact but for dims
//    2^24 below the column's largest); the power is folded into the softmax scale.
//  - the weights P = 2^(x - m) use a reference m that only moves when a score
//    passes it by 13, so a unit needs one vote and no lane exchange.  It moves to
//    12 below the largest score seen: P <= 2^13, in the upper half of fp16's range.
//  - O += V^T (P s), s the chunk's scale of the key.  P is rounded to fp16 and P s
//    again (2^-11 of the value each, below bf16's 2^-8; a product in binary32
//    would be rounded once, at six instructions a chunk and tile more).  So that
//    neither leaves fp16's range, a chunk's scales enter times a power of two that
//    puts the largest one the warp met in the item between 1/2 and 1: it moves when
//    a unit holds one past 2 (the vote that m needs tells it), O with it.  A unit's
//    scales are multiplied in place, by one lane each.  Scales down to 2^-13 of the
//    chunk's largest and products down to 2^-26 of the largest keep all of fp16's
//    bits; less ones lose them gradually, a scale at 2^-24 or a product at 2^-37
//    the last.  (Scales taken as they are: 74 us in place of 78 on the batch
//    above, and outputs past their bound where |V| is below 1e-3.)
//  - the 8 too many are one product of constants with P s per chunk, taken off O
//    every 8 units, before they outgrow what O's last bits can tell.
// Pieces of an item cut between warps go to the workspace as (O, m, l).  The warp
// that brings an item's last piece merges them, in order, where few share it or
// all are in one CTA; else the CTAs merge theirs and the last CTA the CTAs'.  No
// thread waits for another CTA.
#include <type_traits>

#include "pa_device.cuh"
#include "pa_int4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

// Pieces of an item across CTAs that one warp merges: 128 decodes take 81.6, 77.9 and 77.6 us with 2, 6 and 12,
// 64 sequences of up to 5 rows 103.0, 97.5 and 97.3, 16 sequences of 2000 keys 26.9, 27.0 and 28.6.
constexpr int I4_FEW = 6;
constexpr int I4_MAX_CTAS = 256;      // the counters, one word per CTA, then four bits for each of its warps, fill the
                                      // 2048 bytes that the other attention kernels keep at zero between calls too
constexpr int I4_FOLD = 8;             // units between two corrections of O
constexpr float I4_NO_MAX = -3e38f; // maximum over no pieces
constexpr float I4_TOP = 13.f;        // a weight's largest power of two; beside it a scale may be below 4
// What V's scales enter with, and the largest that may enter so (it then stays below 2), per chunk, fp16 in two halves:
// each is this constant minus the other (the sign bit of the limit is set).  2^15 is the largest power, for subnormal
// scales.
constexpr uint32_t I4_POWERS = 0xfbfffbffu, I4_FIRST_LIMIT = I4_POWERS - 0x78007800u;

template <int D, int NT>
struct I4 {
  static constexpr int NC = D / 32;                         // chunks of a row
  static constexpr int COLS = 8 * NT;
  static constexpr int WARPS = 8;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int PER = 2;                             // prefix sums of the batch's units, per thread
  static constexpr int BUCKETS = THREADS * PER;            // of runs of sequences
  static constexpr int MT = D * NT >= 256 ? 2 : 4;          // 16-key m-tiles of a unit: what the registers hold
  static constexpr int UNIT = 16 * MT;
  static constexpr int HALF_BYTES = UNIT * (D * 9 / 16);    // K (or V) of a unit
  static constexpr int STAGE_BYTES = 2 * HALF_BYTES;
  static constexpr int STAGES = 221184 / WARPS / STAGE_BYTES;
  // a piece, in floats, as the lanes hold it: O [2 NC][NT] and (m, m, l, l) [NT] of 32 lanes x 4
  static constexpr int PIECE = (2 * NC + 1) * NT * 128;
  static constexpr int RING_BYTES = WARPS * STAGES * STAGE_BYTES;
  static constexpr int SMEM = RING_BYTES + 8 * BUCKETS + 8 * WARPS * STAGES + 512;
};

struct Int4Params {
  __nv_bfloat16* out;
  const __nv_bfloat16* q;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;  // nullptr: one row per sequence
  int pad;                     // units that an item's start and end are counted for in the split
  int num_seqs, num_rows, max_blocks, num_q_heads, num_kv_heads, group, rows_per_item, block_shift, num_blocks;
  float scale_log2;
  int* status;
  unsigned* counters;   // workspace: pieces brought per CTA or warp that an item starts in; zero between calls
  float* warp_pieces;   // workspace: [CTA][warp][2]
  float* cta_pieces;    // workspace: [CTA][2]
};

struct SeqInfo {
  int q0, qlen, ctx, units;  // units of one item (0: no work), from the whole context
};

__device__ __forceinline__ SeqInfo i4_seq(const Int4Params& p, int s, int unit, int* bits = nullptr) {
  SeqInfo i;
  i.ctx = p.context_lens[s];
  i.q0 = s;
  i.qlen = 1;
  int bad = 0;
  if (p.query_start) {
    i.q0 = p.query_start[s];
    const int end = p.query_start[s + 1];
    if (i.q0 < 0 || end < i.q0 || end > p.num_rows) {
      bad = PA_STATUS_BIT(PA_ERR_RANGE);
      i.q0 = 0;
      i.qlen = 0;
    } else {
      i.qlen = end - i.q0;
    }
  }
  if (i.ctx > p.max_blocks << p.block_shift) {
    bad = PA_STATUS_BIT(PA_ERR_RANGE);
    i.ctx = 0;
  }
  i.units = i.ctx > 0 && i.qlen > 0 ? (i.ctx + unit - 1) / unit + p.pad : 0;
  if (bits) *bits |= bad;
  return i;
}

__device__ __forceinline__ int i4_groups(const Int4Params& p, int qlen) {
  return p.query_start ? (qlen + p.rows_per_item - 1) / p.rows_per_item : 1;
}

// A place in the batch's order of items: sequence, row group, KV head.
struct Walk {
  SeqInfo seq;
  int s, rg, h;
  int groups;
  int live;  // units of the item that some row sees
};

__device__ __forceinline__ void i4_enter(const Int4Params& p, Walk& w, int unit) {
  const int last = min((w.rg + 1) * p.rows_per_item, w.seq.qlen);  // rows of the item end here
  const int keys = w.seq.ctx - w.seq.qlen + last;
  w.live = keys > 0 ? (keys + unit - 1) / unit : 0;
}

__device__ __forceinline__ void i4_next(const Int4Params& p, Walk& w, int unit) {
  if (++w.h == p.num_kv_heads) {
    w.h = 0;
    if (++w.rg == w.groups) {
      w.rg = 0;
      do {
        if (++w.s >= p.num_seqs) return;  // the range ends before this is used
        w.seq = i4_seq(p, w.s, unit);
      } while (w.seq.units == 0);
      w.groups = i4_groups(p, w.seq.qlen);
    }
    i4_enter(p, w, unit);
  }
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// 8 codes (nibbles of the two halves of w) -> 4 fp16 pairs.  A nibble left alone in the mantissa is the subnormal
// number u 2^-24 (0 and 2) or u 2^-20 (1 and 3): nothing to convert, five operations.
__device__ __forceinline__ void i4_expand(uint32_t w, uint32_t (&h)[4]) {
  const uint32_t b = w >> 8;
  h[0] = w & 0x000f000fu;
  h[1] = w & 0x00f000f0u;
  h[2] = b & 0x000f000fu;
  h[3] = b & 0x00f000f0u;
}
constexpr uint32_t I4_NEG8_EVEN = 0x80088008u, I4_NEG8_ODD = 0x80808080u;  // -8 in the two places
// D[16x8] += A[16x8] B[8x8]
__device__ __forceinline__ void mma_f16_1688(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(b0));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// The power of two that a chunk's scales enter with, from the largest of them (fp16 bits, finite): what makes it 1/2 to 1,
// 2^-14 at least (scales from 2^15 on enter below 4).
__device__ __forceinline__ uint32_t i4_power(uint32_t top) { return (30 - min((top >> 10) + 1, 29u)) << 10; }
__device__ __forceinline__ float half_of(uint32_t w, int hi) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(hi ? w >> 16 : w & 0xffff)));
}
template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  } else {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr));
  }
}

template <int N>
__device__ __forceinline__ void sts_words(uint32_t addr, const uint32_t (&w)[N]) {
  if constexpr (N == 2)
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(w[0]), "r"(w[1]) : "memory");
  else
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                 : "memory");
}

// Merge the k-th pair of O tiles of n pieces (piece(i): the i-th record, or nullptr): a warp takes a pair, each lane
// the elements and the columns it would hold in the main loop.  One pass with a running maximum; a few pieces' loads
// are in flight together.
template <int D, int NT, class Piece>
__device__ __forceinline__ void merge_pair(Piece piece, int n, int k, int lane, float (&o)[2][NT][4], float (&m)[NT][2],
                                           float (&l)[NT][2]) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt][0] = m[nt][1] = I4_NO_MAX;
    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[0][nt][i] = o[1][nt][i] = 0.f;
  }
  constexpr int BATCH = 8 / NT;  // pieces whose loads are in flight together
  for (int i0 = 0; i0 < n; i0 += BATCH) {
    float4 ml[BATCH][NT], x[BATCH][NT], y[BATCH][NT];
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      const float4* r = i0 + b < n ? reinterpret_cast<const float4*>(piece(i0 + b)) : nullptr;
      const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        ml[b][nt] = r ? __ldcg(r + (D / 16 * NT + nt) * 32 + lane) : none;
        x[b][nt] = r ? __ldcg(r + (2 * k * NT + nt) * 32 + lane) : none;
        y[b][nt] = r ? __ldcg(r + ((2 * k + 1) * NT + nt) * 32 + lane) : none;
      }
    }
#pragma unroll
    for (int b = 0; b < BATCH; ++b)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float4 q = ml[b][nt], u = x[b][nt], v = y[b][nt];
        const float lk[2] = {q.z, q.w};
        const float mk[2] = {lk[0] != 0.f ? q.x : I4_NO_MAX, lk[1] != 0.f ? q.y : I4_NO_MAX};  // no key: no maximum
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float mn = fmaxf(m[nt][j], mk[j]);
          const float a = fast_exp2(m[nt][j] - mn), w = fast_exp2(mk[j] - mn);
          m[nt][j] = mn;
          l[nt][j] = l[nt][j] * a + lk[j] * w;
          o[0][nt][j] = o[0][nt][j] * a + (j ? u.y : u.x) * w;
          o[0][nt][j + 2] = o[0][nt][j + 2] * a + (j ? u.w : u.z) * w;
          o[1][nt][j] = o[1][nt][j] * a + (j ? v.y : v.x) * w;
          o[1][nt][j + 2] = o[1][nt][j + 2] * a + (j ? v.w : v.z) * w;
        }
      }
  }
}

// Store one 16-dim tile of O, scaled, to the column's row (dst: its place for this lane, dims 2 qd of the tile).
__device__ __forceinline__ void store_tile(__nv_bfloat16* dst, const float (&o)[4], float i0, float i1, bool on) {
  const uint32_t a = movmatrix_trans(pack_bf16x2(o[0] * i0, o[1] * i1));
  const uint32_t b = movmatrix_trans(pack_bf16x2(o[2] * i0, o[3] * i1));
  if (on) {
    *reinterpret_cast<uint32_t*>(dst) = a;
    *reinterpret_cast<uint32_t*>(dst + 8) = b;
  }
}

// The pieces of one CTA's warps (2 slots each, from `first`; bit i of `there`: the i-th warp left one; bit 31: `first` is
// a slot 1) into the CTA's piece.  Calls of their own: the main loop's registers are not theirs to press.
template <int D, int NT>
__device__ __noinline__ void merge_warps(const float* first, uint32_t there, int n, int k, float* dst_piece) {
  constexpr int PIECE = I4<D, NT>::PIECE;
  const int lane = threadIdx.x & 31;
  float o[2][NT][4], m[NT][2], l[NT][2];
  const int back = there >> 31 ? PIECE : 0;  // `first` is a slot 1, the others are slots 0
  merge_pair<D, NT>(
      [&](int i) -> const float* {
        return there >> i & 1 ? first + static_cast<long long>(i) * 2 * PIECE - (i > 0 ? back : 0) : nullptr;
      },
      n, k, lane, o, m, l);
  float4* dst = reinterpret_cast<float4*>(dst_piece) + lane;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    dst[(2 * k * NT + nt) * 32] = make_float4(o[0][nt][0], o[0][nt][1], o[0][nt][2], o[0][nt][3]);
    dst[((2 * k + 1) * NT + nt) * 32] = make_float4(o[1][nt][0], o[1][nt][1], o[1][nt][2], o[1][nt][3]);
    if (k == 0) dst[(D / 16 * NT + nt) * 32] = make_float4(m[nt][0], m[nt][1], l[nt][0], l[nt][1]);
  }
}

// The pieces of n CTAs (2 slots each; `first`: the first CTA's slot 1, the others' slot 0 follow) into the output rows.
template <int D, int NT>
__device__ __noinline__ void merge_ctas(const float* first, int n, int k, __nv_bfloat16* out, int num_q_heads, int group,
                                        int rows) {
  constexpr int PIECE = I4<D, NT>::PIECE;
  const int lane = threadIdx.x & 31, g = lane >> 2, qd = lane & 3;
  float o[2][NT][4], m[NT][2], l[NT][2];
  merge_pair<D, NT>(
      [&](int i) -> const float* { return first + static_cast<long long>(i) * 2 * PIECE - (i > 0 ? PIECE : 0); }, n, k,
      lane, o, m, l);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float i0 = l[nt][0] != 0.f ? 1.f / l[nt][0] : 0.f, i1 = l[nt][1] != 0.f ? 1.f / l[nt][1] : 0.f;
    const int r = (nt * 8 + g) / group, head = nt * 8 + g - r * group;
    __nv_bfloat16* dst = out + (static_cast<long long>(r) * num_q_heads + head) * D + k * 32 + 2 * qd;
    store_tile(dst, o[0][nt], i0, i1, r < rows);
    store_tile(dst + 16, o[1][nt], i0, i1, r < rows);
  }
}

// What a warp left behind, for the CTA's merge.
struct WarpEnd {
  // the item its range starts inside of (slot 0), and the one that starts in it and goes on (slot 1)
  int has0, on0, has1;  // on0: slot 0's item goes on past the range
  int row[2], rows[2], h[2];  // its first query row, its rows, its KV head
  long long first[2];   // first unit of the item
  int units[2];
};

// State of a warp's walk over its items that only item changes touch.
struct WarpState {
  Walk c, p;               // consumer's and producer's place
  long long cbase, pbase;  // first units of their items
  long long u0, u1;        // the warp's range
  unsigned lost[8];        // per stage: m-tiles of its unit that were not loaded
};

// VARLEN: several query rows per sequence (columns see different numbers of keys).
template <int D, int NT, bool VARLEN>
__global__ void __launch_bounds__(I4<D, NT>::THREADS, 1) int4_kernel(const __grid_constant__ Int4Params p) {
  using C = I4<D, NT>;
  constexpr int NC = C::NC, WARPS = C::WARPS, STAGES = C::STAGES, MT = C::MT, UNIT = C::UNIT;
  extern __shared__ __align__(128) uint8_t smem[];
  long long* prefix = reinterpret_cast<long long*>(smem + C::RING_BYTES);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::RING_BYTES + 8 * C::BUCKETS);
  __shared__ long long scan[WARPS];
  __shared__ WarpEnd ends[WARPS];
  __shared__ WarpState walks[WARPS];
  __shared__ int sh_merge[2];
  __shared__ int arrived[WARPS];  // pieces of the item inside the CTA that starts in each warp
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(FULL_MASK, tid >> 5, 0);  // (one value to the compiler)
  const int g = lane >> 2, qd = lane & 3;
  const int bs = 1 << p.block_shift;

  if (lane == 0) {
    arrived[warp] = 0;
    ends[warp].has0 = ends[warp].on0 = ends[warp].has1 = 0;
    for (int i = 0; i < STAGES; ++i) mbar_init(&bars[warp * STAGES + i], 1);
    fence_mbar_init();
  }

  grid_dependency_wait();
  grid_launch_dependents();  // the next kernel's launch overlaps this one; it waits for this one's end itself

  // ---- units of the batch: prefix sums over runs of sequences
  const int run = (p.num_seqs + C::BUCKETS - 1) / C::BUCKETS;
  constexpr int PER = C::PER;
  long long mine[PER], sum = 0;
  int bits = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = tid * PER + i;
    for (int s = b * run; s < min((b + 1) * run, p.num_seqs); ++s) {
      const SeqInfo q = i4_seq(p, s, UNIT, &bits);
      sum += static_cast<long long>(q.units) * i4_groups(p, q.qlen) * p.num_kv_heads;
    }
    mine[i] = sum;
  }
  if (bits && blockIdx.x == 0) set_status(p.status, bits);
  long long incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(FULL_MASK, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  long long before = incl - sum, total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    before += w < warp ? scan[w] : 0;
    total += scan[w];
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) prefix[tid * PER + i] = before + mine[i];  // inclusive
  __syncthreads();

  // rows without a key
  const int row_vecs = p.num_q_heads * D / 8;
  for (int s = blockIdx.x; s < p.num_seqs; s += gridDim.x) {
    const SeqInfo q = i4_seq(p, s, UNIT);
    if (q.units == 0 && q.qlen > 0) {
      uint4* o = reinterpret_cast<uint4*>(p.out + static_cast<long long>(q.q0) * p.num_q_heads * D);
      for (long long i = tid; i < static_cast<long long>(q.qlen) * row_vecs; i += C::THREADS)
        o[i] = make_uint4(0, 0, 0, 0);
    }
  }

  // ---- this CTA's and this warp's range: as few CTAs as give every warp a unit
  const long long want = (total + WARPS - 1) / WARPS;
  const int ctas = static_cast<int>(want < gridDim.x ? want : gridDim.x);
  if (static_cast<int>(blockIdx.x) >= ctas) return;
  const auto cta_first = [&](long long c) { return c * (total / ctas) + (c < total % ctas ? c : total % ctas); };
  const bool dense = total / ctas >= WARPS;  // every warp has a unit (else none has two)
  const auto cta_of = [&](long long u) {
    const long long q = total / ctas, r = total % ctas;
    return static_cast<int>(u < r * (q + 1) ? u / (q + 1) : r + (u - r * (q + 1)) / q);
  };
  const auto warp_of = [&](long long u) {  // of all the grid's warps
    const int c = cta_of(u);
    const long long f = cta_first(c);
    return c * WARPS + static_cast<int>((u - f) * WARPS / (cta_first(c + 1) - f));
  };
  const long long c0 = cta_first(blockIdx.x), cn = cta_first(blockIdx.x + 1) - c0;
  // (rounded up: warp 0 always has a unit)
  const long long u0 = c0 + (warp * cn + WARPS - 1) / WARPS, u1 = c0 + ((warp + 1) * cn + WARPS - 1) / WARPS;
  float* piece0 = p.warp_pieces + (static_cast<long long>(blockIdx.x) * WARPS + warp) * 2 * C::PIECE;

  // column constants: rows of column g + 8 nt of the B operand and of columns 2 qd, 2 qd + 1 of the accumulators
  int colrow[NT];  // three bytes
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
    colrow[nt] = (nt * 8 + g) / p.group | (nt * 8 + 2 * qd) / p.group << 8 | (nt * 8 + 2 * qd + 1) / p.group << 16;
  const auto rowB = [&](int nt) { return colrow[nt] & 0xff; };
  const auto rowA = [&](int nt, int j) { return colrow[nt] >> (8 + 8 * j) & 0xff; };
  // where column g + 8 nt of an item's output starts for this lane
  const auto out_place = [&](int row, int h, int nt) {
    const int r = rowB(nt), head = nt * 8 + g - r * p.group;
    return p.out + (static_cast<long long>(row + r) * p.num_q_heads + h * p.group + head) * D + 2 * qd;
  };
  const auto write_out = [&](const float (&o)[2 * NC][NT][4], const float (&l)[NT][2], int row, int rows, int h) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float i0 = l[nt][0] != 0.f ? 1.f / l[nt][0] : 0.f, i1 = l[nt][1] != 0.f ? 1.f / l[nt][1] : 0.f;
      __nv_bfloat16* dst = out_place(row, h, nt);
#pragma unroll
      for (int k = 0; k < 2 * NC; ++k) store_tile(dst + k * 16, o[k][nt], i0, i1, rowB(nt) < rows);
    }
  };
  // ldmatrix: lane i gives row (i & 7) + 8 ((i >> 3) & 1) of chunk i >> 4 (+ 2 per step)
  const uint32_t code_at = int4_code_offset<D>((lane & 7) + (lane & 8), lane >> 4);
  const uint32_t ring_at = smem_u32(smem) + warp * STAGES * C::STAGE_BYTES;
  uint64_t* bar = bars + warp * STAGES;
  const int rec = int4_record_bytes(bs, D);
  const int half_unit = p.block_shift - 4;  // 1: a block holds two m-tiles
  const int blocks = MT >> half_unit;       // of a unit
  WarpState& ws = walks[warp];
  // the scales of m-tile mt's rows stand here (within K or V)
  const auto scales_at = [&](int mt) {
    return half_unit ? (mt >> 1) * rec + 32 * (D / 2) + (mt & 1) * 16 * 2 * NC : mt * rec + 16 * (D / 2);
  };
  // V's scales of a unit are looked over by the whole warp, those of SK keys a lane (SW words of two chunks)
  constexpr int SK = MT / 2, SW = SK * NC / 2;
  const int scale_mt = lane / (32 / MT);
  const uint32_t lane_scales = C::HALF_BYTES + scales_at(scale_mt) + lane % (32 / MT) * SW * 4;

  if (u0 < u1) {
    // ---- find the item of u0
    {
      int lo = 0, hi = C::BUCKETS - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] > u0) hi = mid; else lo = mid + 1;
      }
      long long at = lo > 0 ? prefix[lo - 1] : 0;
      Walk w;
      int s = lo * run;
      for (;; ++s) {
        w.seq = i4_seq(p, s, UNIT);
        w.groups = i4_groups(p, w.seq.qlen);
        const long long n = static_cast<long long>(w.seq.units) * w.groups * p.num_kv_heads;
        if (at + n > u0) break;
        at += n;
      }
      const long long item = (u0 - at) / w.seq.units;
      w.s = s;
      w.rg = static_cast<int>(item / p.num_kv_heads);
      w.h = static_cast<int>(item - static_cast<long long>(w.rg) * p.num_kv_heads);
      i4_enter(p, w, UNIT);
      if (lane == 0) {
        ws.c = ws.p = w;
        ws.cbase = ws.pbase = at + item * w.seq.units;
        ws.u0 = u0;
        ws.u1 = u1;
      }
      __syncwarp();
    }
    // ---- producer: the same walk, ahead by up to STAGES units
    int pu = static_cast<int>(u0 - ws.pbase), pend = static_cast<int>(min(static_cast<long long>(ws.p.live), u1 - ws.pbase));
    int entries = (ws.p.seq.ctx + bs - 1) >> p.block_shift, head_off = ws.p.h * rec;
    unsigned odd = 0;                   // stages whose unit lacks a block
    int ids = 0, ids_from = INT32_MAX;  // block IDs of 32 table entries from ids_from on, one per lane; -1: no such block
    const uint32_t stride = p.num_kv_heads * rec;
    const long long k_to_v = p.v_cache - p.k_cache;

    const auto produce = [&](int to) {
      if (pu >= pend) {
        do {
          const long long next = ws.pbase + ws.p.seq.units;
          if (next >= ws.u1) {
            pend = 0;
            return;
          }
          __syncwarp();
          if (lane == 0) {
            ws.pbase = next;
            i4_next(p, ws.p, UNIT);
          }
          __syncwarp();
          pu = 0;
          pend = static_cast<int>(min(static_cast<long long>(ws.p.live), ws.u1 - next));
        } while (pend <= 0);
        entries = (ws.p.seq.ctx + bs - 1) >> p.block_shift;
        head_off = ws.p.h * rec;
        ids_from = INT32_MAX;
      }
      const int entry = pu * blocks;
      if (static_cast<unsigned>(entry - ids_from) >= 32u) {
        ids_from = entry;
        ids = entry + lane < entries
                  ? __ldg(p.block_tables + static_cast<long long>(ws.p.s) * p.max_blocks + entry + lane)
                  : -1;
        if (ids >= p.num_blocks) ids = -1;
      }
      int id[MT], all = 0;  // (blocks of 32: every other one)
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        id[i] = __shfl_sync(FULL_MASK, ids, entry - ids_from + (i >> half_unit));
        all |= id[i];
      }
      const uint32_t dst = ring_at + to * C::STAGE_BYTES;
      uint64_t* fb = bar + to;
      odd &= ~(1u << to);
      if (all >= 0) {
        if (lane == 0) {
          mbar_arrive_expect_tx(fb, C::STAGE_BYTES);
#pragma unroll
          for (int i = 0; i < MT; ++i)
            if (!(half_unit && (i & 1))) {
              const uint8_t* k = p.k_cache + static_cast<unsigned long long>(id[i]) * stride + head_off;
              bulk_load(dst + (i >> half_unit) * rec, k, rec, fb);
              bulk_load(dst + C::HALF_BYTES + (i >> half_unit) * rec, k + k_to_v, rec, fb);
            }
        }
      } else {  // the last blocks of a context, or a bad ID
        unsigned lost = 0;  // by m-tile
        int there = 0;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          if (id[i] < 0 && entry + (i >> half_unit) < entries) lost |= 1u << i;
          if (id[i] >= 0 && !(half_unit && (i & 1))) ++there;
        }
        odd |= (lost ? 1u : 0u) << to;
        if (lane == 0) {
          ws.lost[to] = lost;
          if (lost) set_status(p.status, PA_STATUS_BIT(PA_ERR_RANGE));
          mbar_arrive_expect_tx(fb, 2 * rec * there);
#pragma unroll
          for (int i = 0; i < MT; ++i)
            if (id[i] >= 0 && !(half_unit && (i & 1))) {
              const uint8_t* k = p.k_cache + static_cast<unsigned long long>(id[i]) * stride + head_off;
              bulk_load(dst + (i >> half_unit) * rec, k, rec, fb);
              bulk_load(dst + C::HALF_BYTES + (i >> half_unit) * rec, k + k_to_v, rec, fb);
            }
        }
      }
      ++pu;
    };
#pragma unroll 1
    for (int i = 0; i < STAGES; ++i) produce(i);

    int stage = 0;
    uint32_t phase = 0;
    bool dead = false, more = true;
    // ---- items of the range
    while (more) {
      const Walk w = ws.c;
      const int first = static_cast<int>(max(ws.u0 - ws.cbase, 0ll));
      const int last = static_cast<int>(min(static_cast<long long>(w.live), ws.u1 - ws.cbase));
      const int row0 = w.rg * p.rows_per_item;
      const int rows = min(p.rows_per_item, w.seq.qlen - row0);
      const int see0 = w.seq.ctx - w.seq.qlen + row0 + 1;  // keys the item's first row sees
      // q, scaled to fp16 by a power of two per column
      uint32_t qf[2 * NC][NT][2];
      float fac[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const bool on = rowB(nt) < rows;
        const int row = on ? rowB(nt) : 0, head = nt * 8 + g - row * p.group;
        const __nv_bfloat16* src =
            p.q + (static_cast<long long>(w.seq.q0 + row0 + row) * p.num_q_heads + w.h * p.group + head) * D + 2 * qd;
        uint32_t raw[2 * NC][2];
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < 2 * NC; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            raw[k][i] = on ? *reinterpret_cast<const uint32_t*>(src + k * 16 + i * 8) : 0u;
            const uint32_t a = raw[k][i] & 0x7fff7fffu;
            top = fmaxf(top, fmaxf(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u)));
          }
        top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, 1));
        top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, 2));
        int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;  // top in [2^e, 2^(e+1))
        if (e < -126) e = top > 0.f ? -126 : 0;
        if (e > 126) e = 126;
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int k = 0; k < 2 * NC; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qf[k][nt][i] = pack_f16x2(__uint_as_float(raw[k][i] << 16) * down * (i ? 1024.f : 16384.f),
                                      __uint_as_float(raw[k][i] & 0xffff0000u) * down * (i ? 1024.f : 16384.f));
        const float f = ldexpf(p.scale_log2, e + 10);
        fac[nt][0] = __shfl_sync(FULL_MASK, f, 8 * qd);  // column 2 qd lives in lanes 4 (2 qd) ..
        fac[nt][1] = __shfl_sync(FULL_MASK, f, 8 * qd + 4);
      }
      // The codes carry 8 too many: -8 sum(q) of every chunk, as the B operand of one more product with the chunks'
      // scales (k: the chunks' high parts, then their low parts).
      uint32_t qc[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint32_t hi[NC / 2], lo[NC / 2];
#pragma unroll
        for (int c = 0; c < NC; c += 2) {
          float x[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 2 * (c + i); k < 2 * (c + i) + 2; ++k)
              mma_f16_16816(d, I4_NEG8_EVEN, I4_NEG8_EVEN, I4_NEG8_ODD, I4_NEG8_ODD, qf[k][nt][0], qf[k][nt][1]);
            const float e0 = __shfl_sync(FULL_MASK, d[0], g >> 1), e1 = __shfl_sync(FULL_MASK, d[1], g >> 1);
            x[i] = g & 1 ? e1 : e0;  // of column g
          }
          hi[c / 2] = pack_f16x2(x[0], x[1]);
          lo[c / 2] = pack_f16x2(x[0] - half_of(hi[c / 2], 0), x[1] - half_of(hi[c / 2], 1));
        }
        if constexpr (NC == 2) {
          qc[nt][0] = qd == 0 ? hi[0] : qd == 1 ? lo[0] : 0u;
        } else if constexpr (NC == 4) {
          qc[nt][0] = qd == 0 ? hi[0] : qd == 1 ? hi[1] : qd == 2 ? lo[0] : lo[1];
        } else {
          qc[nt][0] = qd == 0 ? hi[0] : qd == 1 ? hi[1] : qd == 2 ? hi[2] : hi[3];
          qc[nt][1] = qd == 0 ? lo[0] : qd == 1 ? lo[1] : qd == 2 ? lo[2] : lo[3];
        }
      }
      float o[2 * NC][NT][4];
      float over[NC][NT][4];  // -8 times the weights' sum, per chunk: what the codes' 8 adds to O
      float l[NT][2], m[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int k = 0; k < 2 * NC; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[k][nt][i] = over[k / 2][nt][i] = 0.f;
        l[nt][0] = l[nt][1] = 0.f;
        m[nt][0] = m[nt][1] = 0.f;
      }
      unsigned fresh = (1u << 2 * NT) - 1;  // columns without a score so far: their reference is not one yet
      uint32_t limit[NC / 2];               // of V's scales, two chunks a word
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) limit[i] = I4_FIRST_LIMIT;

      const auto unit = [&](auto partial, int u, uint32_t ka, unsigned lost) {
        constexpr bool PARTIAL = decltype(partial)::value;

        // where m-tile mt's codes stand (within K or V)
        const auto codes_at = [&](int mt) {
          return half_unit ? (mt >> 1) * rec + (mt & 1) * 16 * (D / 2) : mt * rec;
        };
        const int seen = see0 + rows - 1 - u * UNIT;  // keys of the unit that some column sees
        // ---- scores
        float y[MT][NT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          if (PARTIAL && mt * 16 >= seen) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) y[mt][nt][0] = y[mt][nt][1] = y[mt][nt][2] = y[mt][nt][3] = 0.f;
            continue;
          }
          const uint32_t rb = ka + codes_at(mt), sb = ka + scales_at(mt);
          uint32_t sc0[NC / 2], sc1[NC / 2];
          lds_words(sb + g * 2 * NC, sc0);
          lds_words(sb + (g + 8) * 2 * NC, sc1);
          uint32_t wa[1], wb[1];
          lds_words(sb + g * 2 * NC + (qd * 4 & (2 * NC - 1)), wa);
          lds_words(sb + (g + 8) * 2 * NC + (qd * 4 & (2 * NC - 1)), wb);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            y[mt][nt][0] = y[mt][nt][1] = y[mt][nt][2] = y[mt][nt][3] = 0.f;
            if constexpr (NC == 8)
              mma_f16_16816(y[mt][nt], wa[0], wb[0], wa[0], wb[0], qc[nt][0], qc[nt][1]);
            else
              mma_f16_1688(y[mt][nt], wa[0], wb[0], qc[nt][0]);
          }
#pragma unroll
          for (int cp = 0; cp < NC / 2; ++cp) {
            uint32_t r[4];
            ldsm_x4(rb + (code_at ^ (cp * 32)), r[0], r[1], r[2], r[3]);
#pragma unroll
            for (int x = 0; x < 2; ++x) {  // chunk 2 cp + x: rows 0-7 in r[2 x], rows 8-15 in r[2 x + 1]
              const int c = 2 * cp + x;
              uint32_t a[4], b[4];
              i4_expand(r[2 * x], a);
              i4_expand(r[2 * x + 1], b);
              const float f0 = half_of(sc0[cp], x), f1 = half_of(sc1[cp], x);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float d[4] = {0.f, 0.f, 0.f, 0.f};
                mma_f16_16816(d, a[0], b[0], a[1], b[1], qf[2 * c][nt][0], qf[2 * c][nt][1]);
                mma_f16_16816(d, a[2], b[2], a[3], b[3], qf[2 * c + 1][nt][0], qf[2 * c + 1][nt][1]);
#pragma unroll
                for (int i = 0; i < 4; ++i) y[mt][nt][i] = fmaf(d[i], i < 2 ? f0 : f1, y[mt][nt][i]);
              }
            }
          }
        }
        // ---- softmax: y = score - m
        float top = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              y[mt][nt][i] = fmaf(y[mt][nt][i], fac[nt][i & 1], -m[nt][i & 1]);
              if (!PARTIAL) top = fmaxf(top, y[mt][nt][i]);
            }
        if (PARTIAL) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int row = rowA(nt, i & 1);
                if (u * UNIT + mt * 16 + (i >> 1) * 8 + g >= (row < rows ? see0 + row : 0) || (lost >> mt & 1))
                  y[mt][nt][i] = -INFINITY;
                top = fmaxf(top, y[mt][nt][i]);
              }
        }
        // does one of V's scales pass its chunk's limit?  (It borrows the bit above the limit then.)
        const auto scales = [&](uint32_t (&vs)[SW]) {
          lds_words(ka + lane_scales, vs);
          if (PARTIAL) {  // the scale of a key that no column sees may be anything: zero times it must stay zero
            const int keys = (lost >> scale_mt & 1) ? 0 : seen - lane * SK;
#pragma unroll
            for (int i = 0; i < SW; ++i)
              if (i / (NC / 2) >= keys) vs[i] = 0;
          }
        };
        uint32_t within = 0x80008000u;
        {
          uint32_t vs[SW];
          scales(vs);
#pragma unroll
          for (int i = 0; i < SW; ++i) within &= limit[i % (NC / 2)] - vs[i];
        }
        const bool rise = within != 0x80008000u;
        if (__any_sync(FULL_MASK, top > I4_TOP || fresh || rise)) {  // a score or a scale passes its reference: move it
          float fall[NC];  // of a chunk's sums, with its scales
#pragma unroll
          for (int c = 0; c < NC; ++c) fall[c] = 1.f;
          if (__any_sync(FULL_MASK, rise)) {
            uint32_t vs[SW];
            scales(vs);
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) {
              uint32_t big = 0;  // of the lane's keys; NaN moves nothing
#pragma unroll
              for (int k = i; k < SW; k += NC / 2)
                big = __vmaxu2(big, ((vs[k] & 0x7fffu) < 0x7c00u ? vs[k] & 0x7fffu : 0u) |
                                        ((vs[k] & 0x7fff0000u) < 0x7c000000u ? vs[k] & 0x7fff0000u : 0u));
#pragma unroll
              for (int x = 16; x; x >>= 1) big = __vmaxu2(big, __shfl_xor_sync(FULL_MASK, big, x));
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t old = (I4_POWERS - limit[i]) >> (16 * x) & 0xffffu;
                const uint32_t now = min(old, i4_power(big >> (16 * x) & 0xffffu));
                limit[i] += (old - now) << (16 * x);
                fall[2 * i + x] = __uint_as_float((127 + (now >> 10) - (old >> 10)) << 23);
              }
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float mx = fmaxf(y[0][nt][j], y[0][nt][j + 2]);
#pragma unroll
              for (int mt = 1; mt < MT; ++mt) mx = fmaxf(mx, fmaxf(y[mt][nt][j], y[mt][nt][j + 2]));
              mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, 16));
              const bool first_one = fresh >> (2 * nt + j) & 1;
              const float up = mx > I4_TOP || (first_one && mx > -INFINITY) ? mx - (I4_TOP - 1.f) : 0.f;
              const float a = first_one ? 0.f : fast_exp2(-up);
              if (mx > -INFINITY) fresh &= ~(1u << (2 * nt + j));
              m[nt][j] = m[nt][j] + up;
              l[nt][j] *= a;
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                y[mt][nt][j] -= up;
                y[mt][nt][j + 2] -= up;
              }
#pragma unroll
              for (int k = 0; k < 2 * NC; ++k) {
                o[k][nt][j] *= a * fall[k / 2];
                o[k][nt][j + 2] *= a * fall[k / 2];
              }
#pragma unroll
              for (int c = 0; c < NC; ++c) {
                over[c][nt][j] *= a * fall[c];
                over[c][nt][j + 2] *= a * fall[c];
              }
            }
        }
        {  // the scales go back as they enter
          uint32_t vs[SW];
          scales(vs);
#pragma unroll
          for (int i = 0; i < SW; ++i) vs[i] = hmul2(vs[i], I4_POWERS - limit[i % (NC / 2)]);
          sts_words(ka + lane_scales, vs);
          fence_proxy_async_smem();  // (ordered before the copy that overwrites them)
          __syncwarp();
        }
        uint32_t pf[MT][NT][2];  // B operand: keys 2 qd, 2 qd + 1 (and + 8) of column g
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            float e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              e[i] = fast_exp2(y[mt][nt][i]);
              l[nt][i & 1] += e[i];
            }
            pf[mt][nt][0] = movmatrix_trans(pack_f16x2(e[0], e[1]));
            pf[mt][nt][1] = movmatrix_trans(pack_f16x2(e[2], e[3]));
          }
        // ---- values
        const uint32_t va = ka + C::HALF_BYTES;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          if (PARTIAL && mt * 16 >= seen) continue;
          const uint32_t rb = va + codes_at(mt), sb = va + scales_at(mt);
          uint32_t w0[NC / 2], w1[NC / 2], w2[NC / 2], w3[NC / 2];
          lds_words(sb + (2 * qd) * 2 * NC, w0);
          lds_words(sb + (2 * qd + 1) * 2 * NC, w1);
          lds_words(sb + (2 * qd + 8) * 2 * NC, w2);
          lds_words(sb + (2 * qd + 9) * 2 * NC, w3);
#pragma unroll
          for (int cp = 0; cp < NC / 2; ++cp) {
            uint32_t r[4];
            ldsm_x4_trans(rb + (code_at ^ (cp * 32)), r[0], r[1], r[2], r[3]);
#pragma unroll
            for (int x = 0; x < 2; ++x) {  // chunk 2 cp + x: keys 0-7 in r[2 x], keys 8-15 in r[2 x + 1]
              const int c = 2 * cp + x;
              uint32_t a[4], b[4];
              i4_expand(r[2 * x], a);
              i4_expand(r[2 * x + 1], b);
              const uint32_t s01 = __byte_perm(w0[cp], w1[cp], x ? 0x7632 : 0x5410);
              const uint32_t s89 = __byte_perm(w2[cp], w3[cp], x ? 0x7632 : 0x5410);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                uint32_t b0 = hmul2(pf[mt][nt][0], s01), b1 = hmul2(pf[mt][nt][1], s89);
                if (VARLEN && PARTIAL) {  // likewise the scale of a key that only other columns see
                  const int k0 = u * UNIT + mt * 16 + 2 * qd;
                  const int lim = (lost >> mt) & 1 ? 0 : see0 + rowB(nt);
                  b0 &= (k0 < lim ? 0xffffu : 0u) | (k0 + 1 < lim ? 0xffff0000u : 0u);
                  b1 &= (k0 + 8 < lim ? 0xffffu : 0u) | (k0 + 9 < lim ? 0xffff0000u : 0u);
                }
                mma_f16_16816(over[c][nt], I4_NEG8_EVEN, I4_NEG8_ODD, I4_NEG8_EVEN, I4_NEG8_ODD, b0, b1);
                mma_f16_16816(o[2 * c][nt], a[0], a[1], b[0], b[1], b0, b1);
                mma_f16_16816(o[2 * c + 1][nt], a[2], a[3], b[2], b[3], b0, b1);
              }
            }
          }
        }
      };

      const auto settle = [&]() {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              o[2 * c][nt][i] += over[c][nt][i];
              o[2 * c + 1][nt][i] += over[c][nt][i];
              over[c][nt][i] = 0.f;
            }
      };
#pragma unroll 1
      for (int u = first; u < last; ++u) {
        const uint32_t ka = ring_at + stage * C::STAGE_BYTES;
        if (!__all_sync(FULL_MASK, !dead && mbar_wait(bar + stage, phase))) {
          dead = true;
          break;
        }
        // (some key is masked for some column, or none is: two copies of the body)
        if (u * UNIT + UNIT > see0 || (odd >> stage & 1))
          unit(std::true_type{}, u, ka, odd >> stage & 1 ? ws.lost[stage] : 0u);
        else
          unit(std::false_type{}, u, ka, 0u);
        __syncwarp();  // every lane has read the stage
        produce(stage);
        // O holds sums of u, not of u - 8: taken off before they grow past what their last bits can tell
        if ((u & (I4_FOLD - 1)) == I4_FOLD - 1) settle();
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      settle();
#pragma unroll
      for (int k = 0; k < 2 * NC; ++k) {  // the codes' 2^-24 and 2^-20, the scales' powers
        const uint32_t e = (I4_POWERS - limit[k / 4]) >> (16 * (k / 2 & 1) + 10) & 31;  // 2^(e - 15)
        const float even = __uint_as_float((127 + 24 + 15 - e) << 23), odd_half = __uint_as_float((127 + 20 + 15 - e) << 23);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[k][nt][i] *= i < 2 ? even : odd_half;
      }
      // ---- the item's end, or the range's
      const long long base = ws.cbase, item_end = base + ws.c.seq.units, end = ws.u1;
      const bool starts = base >= ws.u0, finishes = item_end <= end;
      const int row = ws.c.seq.q0 + ws.c.rg * p.rows_per_item, h = ws.c.h;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int x = 4; x <= 16; x <<= 1) l[nt][j] += __shfl_xor_sync(FULL_MASK, l[nt][j], x);
      if (starts && finishes) {
        write_out(o, l, row, rows, h);
      } else {
        const int slot = starts ? 1 : 0;
        float4* rec_out = reinterpret_cast<float4*>(piece0 + slot * C::PIECE) + lane;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int k = 0; k < 2 * NC; ++k)
            rec_out[(k * NT + nt) * 32] = make_float4(o[k][nt][0], o[k][nt][1], o[k][nt][2], o[k][nt][3]);
          rec_out[(2 * NC * NT + nt) * 32] = make_float4(m[nt][0], m[nt][1], l[nt][0], l[nt][1]);
        }
        // Merged at once, by the warp that brings the last piece: an item inside the CTA, and one that few warps of
        // several CTAs share.  Where not every warp has a unit, none has more than one: a piece per unit.
        const bool local = base >= c0 && item_end <= c0 + cn;
        const int w0 = warp_of(base);
        const int n = dense ? warp_of(item_end - 1) - w0 + 1 : static_cast<int>(item_end - base);
        const int self = dense ? static_cast<int>(blockIdx.x) * WARPS + warp - w0 : static_cast<int>(ws.u0 - base);
        if (local || n <= I4_FEW) {
          int got = 0;
          if (local) {
            __threadfence_block();
            __syncwarp();
            if (lane == 0) got = atomicAdd(&arrived[w0 - blockIdx.x * WARPS], 1);
            got = __shfl_sync(FULL_MASK, got, 0);
            __threadfence_block();
          } else {
            __threadfence();
            __syncwarp();
            if (lane == 0) {
              static_assert(WARPS == 8 && I4_FEW < 16, "four bits a warp");
              unsigned* const word = p.counters + I4_MAX_CTAS + w0 / WARPS;
              const int at = w0 % WARPS * 4;
              got = atomicAdd(word, 1u << at) >> at & 15;
              if (got == n - 1) atomicSub(word, static_cast<unsigned>(n) << at);
            }
            got = __shfl_sync(FULL_MASK, got, 0);
            __threadfence();
          }
          if (got == n - 1) {
            const auto piece = [&](int i) {
              const int at = dense ? w0 + i : warp_of(base + i);
              return reinterpret_cast<const float4*>(p.warp_pieces +
                                                     (static_cast<long long>(at) * 2 + (i == 0 ? 1 : 0)) * C::PIECE) + lane;
            };
            float top[NT][2], sum[NT][2], acc[2 * NC][NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              top[nt][0] = top[nt][1] = I4_NO_MAX;
              sum[nt][0] = sum[nt][1] = 0.f;
#pragma unroll
              for (int k = 0; k < 2 * NC; ++k)
#pragma unroll
                for (int x = 0; x < 4; ++x) acc[k][nt][x] = 0.f;
            }
            for (int i = 0; i < n; ++i) {  // in the pieces' order, whoever merges
              const float4* r = piece(i);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float4 ml = make_float4(m[nt][0], m[nt][1], l[nt][0], l[nt][1]);
                if (i != self) ml = __ldcg(r + (2 * NC * NT + nt) * 32);
                constexpr int K = D * NT < 256 ? 2 * NC : 4;  // tiles loaded at a time: what the registers hold
                float a0, a1, b0, b1;
#pragma unroll
                for (int k0 = 0; k0 < 2 * NC; k0 += K) {
                  float4 x[K];
#pragma unroll
                  for (int k = 0; k < K; ++k) {
                    const float (&own)[4] = o[k0 + k][nt];
                    x[k] = i == self ? make_float4(own[0], own[1], own[2], own[3]) : __ldcg(r + ((k0 + k) * NT + nt) * 32);
                  }
                  if (k0 == 0) {
                    const float m0 = ml.z != 0.f ? ml.x : I4_NO_MAX, m1 = ml.w != 0.f ? ml.y : I4_NO_MAX;
                    const float t0 = fmaxf(top[nt][0], m0), t1 = fmaxf(top[nt][1], m1);
                    a0 = fast_exp2(top[nt][0] - t0), a1 = fast_exp2(top[nt][1] - t1);
                    b0 = fast_exp2(m0 - t0), b1 = fast_exp2(m1 - t1);
                    top[nt][0] = t0;
                    top[nt][1] = t1;
                    sum[nt][0] = sum[nt][0] * a0 + ml.z * b0;
                    sum[nt][1] = sum[nt][1] * a1 + ml.w * b1;
                  }
#pragma unroll
                  for (int k = 0; k < K; ++k) {
                    float (&to)[4] = acc[k0 + k][nt];
                    to[0] = to[0] * a0 + x[k].x * b0;
                    to[1] = to[1] * a1 + x[k].y * b1;
                    to[2] = to[2] * a0 + x[k].z * b0;
                    to[3] = to[3] * a1 + x[k].w * b1;
                  }
                }
              }
            }
            write_out(acc, sum, row, rows, h);
          }
        } else if (lane == 0) {
          WarpEnd& we = ends[warp];
          we.row[slot] = row;
          we.rows[slot] = rows;
          we.h[slot] = h;
          we.first[slot] = base;
          we.units[slot] = ws.c.seq.units;
          if (slot == 0) {
            we.has0 = 1;
            we.on0 = !finishes;
          } else {
            we.has1 = 1;
          }
        }
      }
      more = item_end < end;
      if (more) {
        __syncwarp();
        if (lane == 0) {
          ws.cbase = item_end;
          i4_next(p, ws.c, UNIT);
        }
        __syncwarp();
      }
    }
    if (dead) {  // a copy did not land in time: report it, and give those in flight as long again
      if (lane == 0) set_status(p.status, PA_STATUS_BIT(PA_ERR_TIMEOUT));
      for (int i = 0; i < STAGES; ++i) {
        (void)mbar_wait(bar + stage, phase);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
  }
  __syncthreads();

  // ---- what is left: items that many warps of several CTAs share
  bool any = false;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) any |= ends[w].has0 || ends[w].has1;
  if (!any) return;

  // ---- merge the CTA's pieces of each.  Chain e: the item the CTA's range starts inside of (0), or the one that
  // starts in it and goes on past it (1).
  float* cta_piece = p.cta_pieces + static_cast<long long>(blockIdx.x) * 2 * C::PIECE;
  const float* pieces = p.warp_pieces + static_cast<long long>(blockIdx.x) * WARPS * 2 * C::PIECE;
  int chain[2] = {ends[0].has0 ? 0 : -1, -1};  // first warps
  for (int w = 0; w < WARPS; ++w)
    if (ends[w].has1) chain[1] = w;
  for (int e = 0; e <= 1; ++e) {
    const int w0 = chain[e];
    if (w0 < 0) continue;
    uint32_t there = 1;
    int n = 1;
    if (e == 1 || ends[0].on0)
      for (int w = w0 + 1; w < WARPS; ++w) {
        if (!ends[w].has0) continue;  // (a warp without units)
        n = w - w0 + 1;
        there |= 1u << (w - w0);
        if (!ends[w].on0) break;
      }
    for (int k = (warp + e * NC) % WARPS; k < NC; k += WARPS)
      merge_warps<D, NT>(pieces + (static_cast<long long>(w0) * 2 + e) * C::PIECE, there | (e ? 1u << 31 : 0u), n, k,
                         cta_piece + e * C::PIECE);
  }
  // ---- pieces of items that cross CTAs: count them in; the last CTA merges
  __threadfence();
  __syncthreads();
  int from[2], count[2];
#pragma unroll
  for (int e = 0; e <= 1; ++e) {
    from[e] = count[e] = 0;
    if (chain[e] < 0) continue;
    const WarpEnd& we = ends[chain[e]];
    from[e] = cta_of(we.first[e]);
    count[e] = cta_of(we.first[e] + we.units[e] - 1) - from[e] + 1;
  }
  if (tid < 2) {  // both at once: neither item waits for the other's merge
    const int f = tid ? from[1] : from[0], n = tid ? count[1] : count[0];
    bool last = false;
    if (n > 0) {
      last = atomicAdd(p.counters + f, 1u) == static_cast<unsigned>(n - 1);
      if (last) p.counters[f] = 0;
    }
    sh_merge[tid] = last;
    __threadfence();
  }
  __syncthreads();
  for (int job = warp; job < 2 * NC; job += WARPS) {
    const int e = job >= NC, k = job - e * NC;
    if (!sh_merge[e]) continue;
    const WarpEnd& we = ends[e ? chain[1] : chain[0]];
    merge_ctas<D, NT>(p.cta_pieces + (static_cast<long long>(e ? from[1] : from[0]) * 2 + 1) * C::PIECE,
                      e ? count[1] : count[0], k,
                      p.out + (static_cast<long long>(we.row[e]) * p.num_q_heads + we.h[e] * p.group) * D, p.num_q_heads,
                      p.group, we.rows[e]);
  }
}

template <int D, int NT>
size_t workspace_of(int num_sms) {
  using C = I4<D, NT>;
  return attention_counter_bytes(num_sms) + sizeof(float) * static_cast<size_t>(num_sms) * 2 * C::PIECE * (C::WARPS + 1);
}

size_t int4_workspace(int head_dim, int num_sms) {
  size_t n = 0;
  const auto most = [&](size_t x) { n = x > n ? x : n; };
  if (head_dim == 64) most(workspace_of<64, 1>(num_sms)), most(workspace_of<64, 2>(num_sms));
  if (head_dim == 128) most(workspace_of<128, 1>(num_sms)), most(workspace_of<128, 2>(num_sms));
  if (head_dim == 256) most(workspace_of<256, 1>(num_sms));
  return (n + 255) / 256 * 256;
}

template <int D, int NT, bool VARLEN>
int launch_int4(Int4Params& p, void* workspace, cudaStream_t stream, int num_sms) {
  using C = I4<D, NT>;
  p.rows_per_item = p.query_start ? C::COLS / p.group : 1;
  // An item's start and end cost about a unit: counted where items are many (80.8 -> 79.6 us on 128 sequences), not
  // where a unit more would only cut short items in two.
  p.pad = 4ll * p.num_seqs * p.num_kv_heads >= static_cast<long long>(num_sms) * C::WARPS ? 1 : 0;
  p.counters = static_cast<unsigned*>(workspace);
  // The pieces take what the bf16 and FP8 kernels use for theirs (fewer bytes than those on every shape), so that one
  // workspace may serve all three caches.
  p.warp_pieces = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + attention_counter_bytes(num_sms));
  p.cta_pieces = p.warp_pieces + static_cast<size_t>(num_sms) * 2 * C::PIECE * C::WARPS;
  static PerDevice ready;
  int done = 0;
  const int rc = per_device(
      ready,
      [](int) {
        const cudaError_t e =
            cudaFuncSetAttribute(int4_kernel<D, NT, VARLEN>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        return e == cudaSuccess ? 1 : cuda_fail(e, "cudaFuncSetAttribute");
      },
      &done);
  if (rc != PA_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return check_launch(cudaLaunchKernelEx(&cfg, int4_kernel<D, NT, VARLEN>, p), "int4_kernel launch");
}

int run_int4(void* out, const void* q, const int32_t* query_start, const void* k_cache, const void* v_cache,
             const int32_t* block_tables, int max_blocks, const int32_t* context_lens, int num_seqs, int total_rows,
             int num_q_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
             void* workspace, size_t workspace_bytes, int* dev_status, void* stream) {
  if (num_seqs < 0 || total_rows < 0 || max_blocks <= 0 || num_blocks <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
      num_q_heads % num_kv_heads)
    return PA_ERR_SHAPE;
  if (num_seqs > PA_MAX_COUNT) return PA_ERR_SHAPE;
  const int group = num_q_heads / num_kv_heads;
  if (block_size != 16 && block_size != 32) return PA_ERR_UNSUPPORTED;
  if (!rows_supported(group, head_dim)) return PA_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_blocks) * block_size > INT32_MAX - 256) return PA_ERR_SHAPE;
  if (num_seqs == 0 || total_rows == 0) return PA_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !workspace) return PA_ERR_NULL;
  const auto ok = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; };
  if (!ok(out) || !ok(q) || !ok(k_cache) || !ok(v_cache) || !ok(workspace)) return PA_ERR_SHAPE;
  DeviceInfo di;
  const int rc = device_info(&di);
  if (rc != PA_OK) return rc;
  if (di.num_sms > I4_MAX_CTAS) return PA_ERR_UNSUPPORTED;
  if (workspace_bytes < int4_workspace(head_dim, di.num_sms)) return PA_ERR_WORKSPACE;
  Int4Params p{};
  p.out = static_cast<__nv_bfloat16*>(out);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.query_start = query_start;
  p.num_seqs = num_seqs;
  p.num_rows = total_rows;
  p.max_blocks = max_blocks;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = group;
  p.block_shift = block_size == 16 ? 4 : 5;
  p.num_blocks = num_blocks;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.status = dev_status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // One n-tile of columns where 8 hold a row's heads and the call has one row per sequence; two for wider groups,
  // and for several rows, which then share each unpacked key.
  const auto launch = [&](auto kernel) { return kernel(p, workspace, st, di.num_sms); };
  if (query_start)
    return launch(head_dim == 64 ? launch_int4<64, 2, true>
                                 : head_dim == 128 ? launch_int4<128, 2, true> : launch_int4<256, 1, true>);
  if (group > 8) return launch(head_dim == 64 ? launch_int4<64, 2, false> : launch_int4<128, 2, false>);
  return launch(head_dim == 64 ? launch_int4<64, 1, false>
                               : head_dim == 128 ? launch_int4<128, 1, false> : launch_int4<256, 1, false>);
}

}  // namespace

}  // namespace pa

extern "C" {

size_t pa_int4_workspace_bytes(int num_q_heads, int num_kv_heads, int head_dim) {
  if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads) return 0;
  if (!pa::rows_supported(num_q_heads / num_kv_heads, head_dim)) return 0;
  pa::DeviceInfo di;
  if (pa::device_info(&di) != PA_OK) return 0;
  return pa::int4_workspace(head_dim, di.num_sms);
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

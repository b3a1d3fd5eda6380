// pa_rope.cu -- rotary positions of a step's q and k, written where attention
// reads them: q to its rows, k (and v unrotated) to their cache slots, in the
// cache's own format (bf16, E4M3, 4 bits).  Also the 4-bit cache's plain
// append and its read-back, and the table of cosines and sines.
//
// A pair (x, y) of a head's first rot_dim dims turns by the angle of its
// position: x' = x c - y s, y' = y c + x s, with (c, s) a binary32 table row.
// Pairs are (i, i + rot_dim / 2) or, interleaved, (2 i, 2 i + 1); the dims
// past rot_dim pass.  The result is the exact x c - y s rounded once to bf16,
// whatever the order of operations: codes of a quantised cache taken from it
// then do not depend on rounding noise.
//
// HBM-bound: q is read and written, k and v are read, their cache rows
// written.  One thread per 16-byte vector (8 dims) of a head; a thread keeps
// its vector's place in the head and walks over heads, so that a position's
// table row is read once per thread and not once per head.  The partner vector
// of a half-split pair is loaded too (an L1 hit); both lie in one warp, which
// loads before it stores, so q may be rotated in place.
#include <cmath>

#include "pa_device.cuh"
#include "pa_int4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int ROPE_THREADS = 256;

struct RopeParams {
  __nv_bfloat16* q_out;        // [T, Hq, D]; heads counted first: 0 .. Hq-1 are q, then k, then v
  const __nv_bfloat16* q;
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  void* k_cache;
  void* v_cache;
  const float* table;          // [table_len, rot_dim]: cosines, then sines
  const int32_t* positions;
  const int32_t* slots;
  long long q_stride, k_stride, v_stride;  // elements from one token's rows to the next's
  long long num_slots;
  int num_tokens, num_q_heads, num_kv_heads, rot_dim, table_len, block_shift;
  float k_inv, v_inv;
  int* status;
};

enum Cache { CACHE_BF16, CACHE_E4M3, CACHE_INT4 };
enum Pairs { PAIRS_NONE, PAIRS_HALF, PAIRS_INTERLEAVED };

// a c - b s (b's term added for the second half of a pair), rounded once to
// bf16.  Two fused operations leave an error of at most 2 ulp of binary32; only
// a value that close to a bf16 tie is taken again in binary64, where both
// products are exact.
__device__ __noinline__ uint32_t turn_exact(float a, float c, float b, float s) {
  const double d = static_cast<double>(a) * c + static_cast<double>(b) * s;
  const float z = __double2float_rz(d);  // round to odd: then one more rounding is right
  uint32_t u = __float_as_uint(z);
  if (static_cast<double>(z) != d) u |= 1;
  return u;
}
__device__ __forceinline__ uint32_t turn(float a, float c, float b, float s) {
  const float p = b * s;
  const float e = fmaf(b, s, -p);
  float r = fmaf(a, c, p) + e;
  if (r != r) r = fmaf(a, c, p);  // an infinite product has no rest to add
  uint32_t u = __float_as_uint(r);
  if (((u + 4u) & 0xffffu) - 0x8000u <= 8u) u = turn_exact(a, c, b, s);
  return __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(u)));
}

__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w, float inv) {
  return f32x2_to_e4m3x2(lo_f32(w) * inv, hi_f32(w) * inv);
}

// Quantise 32 dims held as 8 by each of 4 adjacent lanes (j = lane & 3) and
// store them: lane j writes the chunk's j-th 4 bytes, lane 0 its scale.
template <int D>
__device__ __forceinline__ void store_int4(uint8_t* record, int block_size, int row, int chunk, int j, uint4 x,
                                           unsigned group) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float f[8], m = 0.f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = lo_f32(w[i]);
    f[2 * i + 1] = hi_f32(w[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m = fmaxf(m, fabsf(f[i]));
    nan |= f[i] != f[i];
  }
  if (nan) m = __uint_as_float(0x7fffffffu);
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {  // a NaN wins: the chunk then reads as NaN
    const float y = __shfl_xor_sync(group, m, o);
    m = (m != m || y != y) ? __uint_as_float(0x7fffffffu) : fmaxf(m, y);
  }
  const float top = __fdiv_rn(m, 7.0f);
  const __half h = __float2half_rn(top > 65504.f ? 65504.f : top);
  const float s = __half2float(h);
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t v = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float n = s > 0.f ? rintf(__fdiv_rn(f[2 * i + k], s)) : 0.f;
      n = fminf(fmaxf(n, -7.f), 7.f);
      v |= static_cast<uint32_t>(static_cast<int>(n) + 8) << (16 * k + 4 * j);
    }
    out[i] = v;
  }
  // unit 2 i + k has this lane's nibble j of dim 8 j + 2 i + k: gather the four lanes' nibbles
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    out[i] |= __shfl_xor_sync(group, out[i], 1);
    out[i] |= __shfl_xor_sync(group, out[i], 2);
  }
  const uint32_t mine = j == 0 ? out[0] : j == 1 ? out[1] : j == 2 ? out[2] : out[3];
  *reinterpret_cast<uint32_t*>(record + int4_code_offset<D>(row, chunk) + 4 * j) = mine;
  if (j == 0) *reinterpret_cast<__half*>(record + int4_scale_offset<D>(block_size, row, chunk)) = h;
}

template <int D, Cache CACHE, Pairs PAIRS>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(const RopeParams p) {
  constexpr int VECS = D / 8;                       // 8 .. 32: a head's vectors lie in one warp
  constexpr int HEADS = ROPE_THREADS / VECS;        // heads a CTA takes at a time
  grid_launch_dependents();
  const int vec = threadIdx.x % VECS;
  const int h0 = blockIdx.y * HEADS + threadIdx.x / VECS;
  const int heads = p.num_q_heads + 2 * p.num_kv_heads;
  const int bs = 1 << p.block_shift;
  const unsigned group = 0xfu << (threadIdx.x & 28);
  const unsigned head_lanes = VECS == 32 ? FULL_MASK : ((1u << (VECS & 31)) - 1) << (threadIdx.x & 31 & ~(VECS - 1));
  const int half_vecs = p.rot_dim / 16;
  const bool turns = PAIRS != PAIRS_NONE && vec * 8 < p.rot_dim;
  for (int t = blockIdx.x; t < p.num_tokens; t += gridDim.x) {
    long long slot = p.slots[t];
    if (slot >= p.num_slots) {
      if (threadIdx.x == 0 && blockIdx.y == 0) set_status(p.status, PA_STATUS_BIT(PA_ERR_RANGE));
      slot = -1;
    }
    float c[8], s[8];
    if (PAIRS != PAIRS_NONE) {
      const int pos = p.positions[t];
      if (pos < 0) continue;  // padding: nothing of this row is written
      if (pos >= p.table_len) {
        if (threadIdx.x == 0 && blockIdx.y == 0) set_status(p.status, PA_STATUS_BIT(PA_ERR_RANGE));
        continue;
      }
      if (turns) {
        const float* row = p.table + static_cast<long long>(pos) * p.rot_dim;
        if (PAIRS == PAIRS_HALF) {
          const bool second = vec >= half_vecs;
          const int i = (second ? vec - half_vecs : vec) * 8;
#pragma unroll
          for (int k = 0; k < 8; k += 4) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(row + i + k));
            const float4 b = __ldg(reinterpret_cast<const float4*>(row + p.rot_dim / 2 + i + k));
            c[k] = a.x, c[k + 1] = a.y, c[k + 2] = a.z, c[k + 3] = a.w;
            s[k] = b.x, s[k + 1] = b.y, s[k + 2] = b.z, s[k + 3] = b.w;
          }
          if (!second) {
#pragma unroll
            for (int k = 0; k < 8; ++k) s[k] = -s[k];
          }
        } else {
          const float4 a = __ldg(reinterpret_cast<const float4*>(row + vec * 4));
          const float4 b = __ldg(reinterpret_cast<const float4*>(row + p.rot_dim / 2 + vec * 4));
          c[0] = c[1] = a.x, c[2] = c[3] = a.y, c[4] = c[5] = a.z, c[6] = c[7] = a.w;
          s[0] = -b.x, s[1] = b.x, s[2] = -b.y, s[3] = b.y, s[4] = -b.z, s[5] = b.z, s[6] = -b.w, s[7] = b.w;
        }
      }
    }
    const long long blk = slot >> p.block_shift;
    const int off = static_cast<int>(slot & (bs - 1));
    for (int h = h0; h < heads; h += gridDim.y * HEADS) {
      const bool is_q = h < p.num_q_heads;
      const bool is_v = h >= p.num_q_heads + p.num_kv_heads;
      const int kh = is_q ? 0 : is_v ? h - p.num_q_heads - p.num_kv_heads : h - p.num_q_heads;
      const __nv_bfloat16* src = is_q   ? p.q + t * p.q_stride + static_cast<long long>(h) * D
                                 : is_v ? p.v_new + t * p.v_stride + static_cast<long long>(kh) * D
                                        : p.k_new + t * p.k_stride + static_cast<long long>(kh) * D;
      uint4 x = make_uint4(0, 0, 0, 0);
      const bool live = is_q || slot >= 0;
      if (live) x = *reinterpret_cast<const uint4*>(src + vec * 8);
      if (PAIRS != PAIRS_NONE) {
        uint4 y = x;
        const bool rotate = turns && !is_v && live;
        if (PAIRS == PAIRS_HALF && rotate) {
          const int other = vec >= half_vecs ? vec - half_vecs : vec + half_vecs;
          y = *reinterpret_cast<const uint4*>(src + other * 8);
        }
        __syncwarp(head_lanes);  // both vectors of every pair are loaded before any is stored (q in place)
        if (rotate) {
          const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float al = lo_f32(a[i]), ah = hi_f32(a[i]);
            const float bl = PAIRS == PAIRS_HALF ? lo_f32(b[i]) : ah, bh = PAIRS == PAIRS_HALF ? hi_f32(b[i]) : al;
            o[i] = turn(al, c[2 * i], bl, s[2 * i]) | (turn(ah, c[2 * i + 1], bh, s[2 * i + 1]) << 16);
          }
          x = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      if (is_q) {
        *reinterpret_cast<uint4*>(p.q_out + (static_cast<long long>(t) * p.num_q_heads + h) * D + vec * 8) = x;
      } else if (slot >= 0) {
        void* cache = is_v ? p.v_cache : p.k_cache;
        const long long head = blk * p.num_kv_heads + kh;
        if (CACHE == CACHE_BF16) {
          static_cast<uint4*>(cache)[(head * bs + off) * VECS + vec] = x;
        } else if (CACHE == CACHE_E4M3) {
          const float inv = is_v ? p.v_inv : p.k_inv;
          static_cast<uint2*>(cache)[(head * bs + off) * VECS + vec] =
              make_uint2(e4m3_pair(x.x, inv) | (e4m3_pair(x.y, inv) << 16),
                         e4m3_pair(x.z, inv) | (e4m3_pair(x.w, inv) << 16));
        } else {
          store_int4<D>(static_cast<uint8_t*>(cache) + head * int4_record_bytes(bs, D), bs, off, vec >> 2, vec & 3, x,
                        group);
        }
      }
    }
  }
}

// Rows of the 4-bit cache as values: one thread per 8 dims (k, then v).
template <int D>
__global__ void __launch_bounds__(ROPE_THREADS)
    read_int4_kernel(float* k_out, float* v_out, const uint8_t* k_cache, const uint8_t* v_cache, const int32_t* slots,
                     int num_tokens, int num_kv_heads, int block_shift, long long num_slots, int* status) {
  constexpr int VECS = D / 8, HEADS = ROPE_THREADS / VECS;
  const int vec = threadIdx.x % VECS, chunk = vec >> 2, j = vec & 3, bs = 1 << block_shift;
  for (int t = blockIdx.x; t < num_tokens; t += gridDim.x) {
    const long long slot = slots[t];
    if (slot < 0) continue;
    if (slot >= num_slots) {
      if (threadIdx.x == 0 && blockIdx.y == 0) set_status(status, PA_STATUS_BIT(PA_ERR_RANGE));
      continue;
    }
    const long long blk = slot >> block_shift;
    const int off = static_cast<int>(slot & (bs - 1));
    for (int h = blockIdx.y * HEADS + threadIdx.x / VECS; h < 2 * num_kv_heads; h += gridDim.y * HEADS) {
      const bool is_v = h >= num_kv_heads;
      const int kh = is_v ? h - num_kv_heads : h;
      const uint8_t* rec = (is_v ? v_cache : k_cache) + (blk * num_kv_heads + kh) * int4_record_bytes(bs, D);
      const uint4 w = *reinterpret_cast<const uint4*>(rec + int4_code_offset<D>(off, chunk));
      const float s = __half2float(*reinterpret_cast<const __half*>(rec + int4_scale_offset<D>(bs, off, chunk)));
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)  // unit i, nibble j: dim 8 j + i
        f[i] = static_cast<float>(static_cast<int>((u[i >> 1] >> (16 * (i & 1) + 4 * j)) & 15) - 8) * s;
      float4* dst = reinterpret_cast<float4*>((is_v ? v_out : k_out) +
                                              (static_cast<long long>(t) * num_kv_heads + kh) * D + vec * 8);
      dst[0] = make_float4(f[0], f[1], f[2], f[3]);
      dst[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
  }
}

// Table row of position p: m cos(p w_i), then m sin(p w_i); angles in binary64
// (positions reach 2^20, where a binary32 angle is off by a tenth of a turn).
// A thread takes one pair over ROPE_RUN positions: cosine and sine of the first,
// then one rotation by w_i per position (four binary64 operations in place of a
// sincos; the error grows by 2^-52 a step, 2^-47 in all against the 2^-24 kept).
constexpr int ROPE_MAX_PAIRS = 128;
constexpr int ROPE_RUN = 16;
struct Frequencies {
  double w[ROPE_MAX_PAIRS], cos_w[ROPE_MAX_PAIRS], sin_w[ROPE_MAX_PAIRS];
};
__global__ void __launch_bounds__(256)
    rope_table_kernel(float* table, int table_len, int half, double factor, const __grid_constant__ Frequencies f) {
  const long long runs = (table_len + ROPE_RUN - 1) / ROPE_RUN;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < runs * half; i += gridDim.x * 256ll) {
    const long long r = i / half;
    const int k = static_cast<int>(i - r * half);
    const int first = static_cast<int>(r) * ROPE_RUN;
    const int n = min(ROPE_RUN, table_len - first);
    const double cw = f.cos_w[k], sw = f.sin_w[k];
    double sn, cs;
    sincos(first * f.w[k], &sn, &cs);
    sn *= factor;
    cs *= factor;
    float* row = table + static_cast<long long>(first) * 2 * half;
    for (int j = 0; j < n; ++j, row += 2 * half) {
      row[k] = static_cast<float>(cs);
      row[half + k] = static_cast<float>(sn);
      const double c = cs * cw - sn * sw;
      sn = sn * cw + cs * sw;
      cs = c;
    }
  }
}

// CTAs in x walk over tokens, in y over heads: enough of both to fill the GPU, no more passes than needed.
dim3 row_grid(int num_tokens, int heads, int heads_per_cta, int num_sms) {
  const int passes = (heads + heads_per_cta - 1) / heads_per_cta;
  const long long want = static_cast<long long>(num_sms) * 8;
  long long y = (want + num_tokens - 1) / num_tokens;
  if (y > passes) y = passes;
  long long x = num_tokens < 65535ll * 16 ? num_tokens : 65535ll * 16;
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>(y));
}

template <int D, Cache CACHE, Pairs PAIRS>
int launch_rope(const RopeParams& p, cudaStream_t stream, int num_sms) {
  const int heads = p.num_q_heads + 2 * p.num_kv_heads;
  rope_kernel<D, CACHE, PAIRS><<<row_grid(p.num_tokens, heads, ROPE_THREADS / (D / 8), num_sms), ROPE_THREADS, 0,
                                stream>>>(p);
  return check_launch(cudaSuccess, "rope_kernel launch");
}

template <Cache CACHE, Pairs PAIRS>
int launch_rope_d(const RopeParams& p, int head_dim, cudaStream_t stream, int num_sms) {
  if (head_dim == 64) return launch_rope<64, CACHE, PAIRS>(p, stream, num_sms);
  if (head_dim == 128) return launch_rope<128, CACHE, PAIRS>(p, stream, num_sms);
  return launch_rope<256, CACHE, PAIRS>(p, stream, num_sms);
}

bool ok16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <Cache CACHE>
int rope_append(void* q_out, const void* q, long long q_stride, const void* k_new, long long k_stride,
                const void* v_new, long long v_stride, void* k_cache, void* v_cache, const float* table, int table_len,
                int rot_dim, int interleaved, const int32_t* positions, const int32_t* slot_mapping, int num_tokens,
                int num_blocks, int num_q_heads, int num_kv_heads, int head_dim, int block_size, float k_inv,
                float v_inv, int* dev_status, void* stream) {
  if (num_tokens < 0 || num_blocks <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || table_len <= 0)
    return PA_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (block_size != 16 && block_size != 32) return PA_ERR_UNSUPPORTED;
  if (rot_dim <= 0 || rot_dim > head_dim || rot_dim % 16) return PA_ERR_UNSUPPORTED;
  const long long qw = static_cast<long long>(num_q_heads) * head_dim, kw = static_cast<long long>(num_kv_heads) * head_dim;
  if (q_stride < qw || k_stride < kw || v_stride < kw || q_stride % 8 || k_stride % 8 || v_stride % 8)
    return PA_ERR_SHAPE;
  if (num_tokens == 0) return PA_OK;
  if (!q_out || !q || !k_new || !v_new || !k_cache || !v_cache || !table || !positions || !slot_mapping)
    return PA_ERR_NULL;
  if (!ok16(q_out) || !ok16(q) || !ok16(k_new) || !ok16(v_new) || !ok16(k_cache) || !ok16(v_cache) || !ok16(table))
    return PA_ERR_SHAPE;
  if (q_out == q && q_stride != qw) return PA_ERR_SHAPE;  // in place: the same rows
  DeviceInfo di;
  const int rc = device_info(&di);
  if (rc != PA_OK) return rc;
  RopeParams p{};
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.table = table;
  p.positions = positions;
  p.slots = slot_mapping;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.num_slots = static_cast<long long>(num_blocks) * block_size;
  p.num_tokens = num_tokens;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.rot_dim = rot_dim;
  p.table_len = table_len;
  p.block_shift = block_size == 16 ? 4 : 5;
  p.k_inv = k_inv;
  p.v_inv = v_inv;
  p.status = dev_status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return interleaved ? launch_rope_d<CACHE, PAIRS_INTERLEAVED>(p, head_dim, st, di.num_sms)
                     : launch_rope_d<CACHE, PAIRS_HALF>(p, head_dim, st, di.num_sms);
}

}  // namespace

}  // namespace pa

extern "C" {

int pa_rope_table(float* table, int table_len, int rot_dim, double base, const pa_rope_scaling* scaling,
                  void* stream) {
  if (table_len < 0 || !(base > 0.0) || !(base < INFINITY)) return PA_ERR_SHAPE;
  if (rot_dim <= 0 || rot_dim % 16 || rot_dim > 2 * pa::ROPE_MAX_PAIRS) return PA_ERR_UNSUPPORTED;
  pa_rope_scaling sc = {};
  sc.type = PA_ROPE_PLAIN;
  if (scaling) sc = *scaling;
  if (sc.type < PA_ROPE_PLAIN || sc.type > PA_ROPE_BANDS) return PA_ERR_UNSUPPORTED;
  if (sc.type != PA_ROPE_PLAIN && (!(sc.factor > 0.0) || !(sc.factor < INFINITY))) return PA_ERR_SHAPE;
  if ((sc.type == PA_ROPE_YARN || sc.type == PA_ROPE_BANDS) &&
      (sc.original_positions <= 0 || !(sc.low > 0.0) || !(sc.high > sc.low)))
    return PA_ERR_SHAPE;
  if (!(sc.attention_factor >= 0.0) || !(sc.attention_factor < INFINITY)) return PA_ERR_SHAPE;
  if (sc.type == PA_ROPE_YARN && !(base > 1.0)) return PA_ERR_SHAPE;  // the ramp divides by log(base)
  if (table_len == 0) return PA_OK;
  if (!table) return PA_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(table) & 15) return PA_ERR_SHAPE;
  pa::DeviceInfo di;
  const int rc = pa::device_info(&di);
  if (rc != PA_OK) return rc;

  const double two_pi = 6.283185307179586476925286766559;
  const int half = rot_dim / 2;
  double m = 1.0, b = base;
  if (sc.type == PA_ROPE_NTK) b = base * std::pow(sc.factor, rot_dim / (rot_dim - 2.0));
  double first = 0.0, last = 0.0;  // YaRN: the pairs that turn sc.high and sc.low times within the trained context
  if (sc.type == PA_ROPE_YARN) {
    const auto at = [&](double turns) {
      return rot_dim * std::log(sc.original_positions / (turns * two_pi)) / (2.0 * std::log(base));
    };
    first = std::fmax(std::floor(at(sc.high)), 0.0);
    last = std::fmin(std::ceil(at(sc.low)), rot_dim - 1.0);
    m = sc.factor > 1.0 ? 0.1 * std::log(sc.factor) + 1.0 : 1.0;
  }
  if (sc.attention_factor > 0.0) m = sc.attention_factor;
  pa::Frequencies f;
  for (int i = 0; i < half; ++i) {
    const double w = std::pow(b, -2.0 * i / rot_dim);
    double keep = 1.0;  // share of the unscaled frequency
    if (sc.type == PA_ROPE_LINEAR) {
      keep = 0.0;
    } else if (sc.type == PA_ROPE_YARN) {
      keep = 1.0 - std::fmin(std::fmax((i - first) / std::fmax(last - first, 0.001), 0.0), 1.0);
    } else if (sc.type == PA_ROPE_BANDS) {
      const double turns = sc.original_positions * w / two_pi;
      keep = std::fmin(std::fmax((turns - sc.low) / (sc.high - sc.low), 0.0), 1.0);
    }
    f.w[i] = keep == 1.0 ? w : w / sc.factor * (1.0 - keep) + w * keep;
    f.cos_w[i] = std::cos(f.w[i]);
    f.sin_w[i] = std::sin(f.w[i]);
  }
  const long long total = (static_cast<long long>(table_len) + pa::ROPE_RUN - 1) / pa::ROPE_RUN * half;
  const long long blocks = (total + 255) / 256, cap = di.num_sms * 8ll;
  pa::rope_table_kernel<<<static_cast<unsigned>(blocks < cap ? blocks : cap), 256, 0,
                          static_cast<cudaStream_t>(stream)>>>(table, table_len, half, m, f);
  return pa::check_launch(cudaSuccess, "rope_table_kernel launch");
}

int pa_rope_append(void* q_out, const void* q, long long q_stride, const void* k_new, long long k_stride,
                   const void* v_new, long long v_stride, void* k_cache, void* v_cache, const float* table,
                   int table_len, int rot_dim, int interleaved, const int32_t* positions, const int32_t* slot_mapping,
                   int num_tokens, int num_blocks, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                   int* dev_status, void* stream) {
  return pa::rope_append<pa::CACHE_BF16>(q_out, q, q_stride, k_new, k_stride, v_new, v_stride, k_cache, v_cache, table,
                                         table_len, rot_dim, interleaved, positions, slot_mapping, num_tokens,
                                         num_blocks, num_q_heads, num_kv_heads, head_dim, block_size, 1.f, 1.f,
                                         dev_status, stream);
}

int pa_rope_append_fp8(void* q_out, const void* q, long long q_stride, const void* k_new, long long k_stride,
                       const void* v_new, long long v_stride, void* k_cache, void* v_cache, const float* table,
                       int table_len, int rot_dim, int interleaved, const int32_t* positions,
                       const int32_t* slot_mapping, int num_tokens, int num_blocks, int num_q_heads, int num_kv_heads,
                       int head_dim, int block_size, float k_scale, float v_scale, int* dev_status, void* stream) {
  if (!(k_scale > 0.f) || !(v_scale > 0.f) || !(k_scale < INFINITY) || !(v_scale < INFINITY)) return PA_ERR_SHAPE;
  return pa::rope_append<pa::CACHE_E4M3>(q_out, q, q_stride, k_new, k_stride, v_new, v_stride, k_cache, v_cache, table,
                                         table_len, rot_dim, interleaved, positions, slot_mapping, num_tokens,
                                         num_blocks, num_q_heads, num_kv_heads, head_dim, block_size, 1.f / k_scale,
                                         1.f / v_scale, dev_status, stream);
}

int pa_rope_append_int4(void* q_out, const void* q, long long q_stride, const void* k_new, long long k_stride,
                        const void* v_new, long long v_stride, void* k_cache, void* v_cache, const float* table,
                        int table_len, int rot_dim, int interleaved, const int32_t* positions,
                        const int32_t* slot_mapping, int num_tokens, int num_blocks, int num_q_heads, int num_kv_heads,
                        int head_dim, int block_size, int* dev_status, void* stream) {
  return pa::rope_append<pa::CACHE_INT4>(q_out, q, q_stride, k_new, k_stride, v_new, v_stride, k_cache, v_cache, table,
                                         table_len, rot_dim, interleaved, positions, slot_mapping, num_tokens,
                                         num_blocks, num_q_heads, num_kv_heads, head_dim, block_size, 1.f, 1.f,
                                         dev_status, stream);
}

int pa_cache_append_int4(const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                         const int32_t* slot_mapping, int num_tokens, int num_blocks, int num_kv_heads, int head_dim,
                         int block_size, int* dev_status, void* stream) {
  if (num_tokens < 0 || num_blocks <= 0 || num_kv_heads <= 0) return PA_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (block_size != 16 && block_size != 32) return PA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PA_OK;
  if (!k_new || !v_new || !k_cache || !v_cache || !slot_mapping) return PA_ERR_NULL;
  if (!pa::ok16(k_new) || !pa::ok16(v_new) || !pa::ok16(k_cache) || !pa::ok16(v_cache)) return PA_ERR_SHAPE;
  pa::DeviceInfo di;
  const int rc = pa::device_info(&di);
  if (rc != PA_OK) return rc;
  pa::RopeParams p{};
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.slots = slot_mapping;
  p.k_stride = p.v_stride = static_cast<long long>(num_kv_heads) * head_dim;
  p.num_slots = static_cast<long long>(num_blocks) * block_size;
  p.num_tokens = num_tokens;
  p.num_kv_heads = num_kv_heads;
  p.block_shift = block_size == 16 ? 4 : 5;
  p.status = dev_status;
  return pa::launch_rope_d<pa::CACHE_INT4, pa::PAIRS_NONE>(p, head_dim, static_cast<cudaStream_t>(stream), di.num_sms);
}

int pa_cache_read_int4(float* k_out, float* v_out, const void* k_cache, const void* v_cache,
                       const int32_t* slot_mapping, int num_tokens, int num_blocks, int num_kv_heads, int head_dim,
                       int block_size, int* dev_status, void* stream) {
  if (num_tokens < 0 || num_blocks <= 0 || num_kv_heads <= 0) return PA_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return PA_ERR_UNSUPPORTED;
  if (block_size != 16 && block_size != 32) return PA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PA_OK;
  if (!k_out || !v_out || !k_cache || !v_cache || !slot_mapping) return PA_ERR_NULL;
  if (!pa::ok16(k_out) || !pa::ok16(v_out) || !pa::ok16(k_cache) || !pa::ok16(v_cache)) return PA_ERR_SHAPE;
  pa::DeviceInfo di;
  const int rc = pa::device_info(&di);
  if (rc != PA_OK) return rc;
  const long long slots = static_cast<long long>(num_blocks) * block_size;
  const int shift = block_size == 16 ? 4 : 5;
  const dim3 grid = pa::row_grid(num_tokens, 2 * num_kv_heads, pa::ROPE_THREADS / (head_dim / 8), di.num_sms);
  const auto kernel = head_dim == 64    ? pa::read_int4_kernel<64>
                      : head_dim == 128 ? pa::read_int4_kernel<128>
                                        : pa::read_int4_kernel<256>;
  kernel<<<grid, pa::ROPE_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(
      k_out, v_out, static_cast<const uint8_t*>(k_cache), static_cast<const uint8_t*>(v_cache), slot_mapping,
      num_tokens, num_kv_heads, shift, slots, dev_status);
  return pa::check_launch(cudaSuccess, "read_int4_kernel launch");
}

}  // extern "C"

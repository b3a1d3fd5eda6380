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
// Floor: q is read and written, k and v are read, their cache rows written (177 MB
// for 8192 tokens of 32 + 8 + 8 heads into 4 bits, 27 us).  Instructions bound it:
// 64 us there, at some 200 a warp and 16-byte vector, most of them the two products
// rounded once; 4.3 us for 128 decode rows, one chain of dependent loads.
// One thread takes one 16-byte vector (8 dims) of one head over a run of tokens:
// its addresses grow by constants, the next two tokens' vectors are in flight, and
// the tokens' slots, positions and table rows are fetched once per CTA into shared
// memory.  The other vector of a half-split pair comes from its lane (both lie in
// one warp, loaded before either is stored, so q may be rotated in place).
#include <cmath>

#include "pa_device.cuh"
#include "pa_int4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_MAX_TOKENS = 8;  // a CTA's

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

// Eight values a c + b s, each rounded once to bf16.  Two fused operations (the product's error added to the sum) leave
// an error of at most 1.5 ulp of binary32, which decides the rounding only within 2 ulp of a tie; such a value, and an
// infinity or NaN, is taken again in binary64, where both products are exact; their sum is not where one lies 2^-21
// below the other, so it is rounded to odd from there on (the last bit kept tells that something follows): then one more
// rounding is right.  One vector in 1600 holds one.
__device__ __noinline__ float turn_exact(float a, float c, float b, float s) {
  const double x = static_cast<double>(a) * c, y = static_cast<double>(b) * s;
  const double d = __dadd_rz(x, y);
  const float z = __double2float_rz(d);
  const bool exact = static_cast<double>(z) == d && __dadd_rd(x, y) == __dadd_ru(x, y);
  return exact ? z : __uint_as_float(__float_as_uint(z) | 1);
}
__device__ __forceinline__ uint4 turn(const float (&a)[8], const float (&b)[8], const float (&c)[8],
                                      const float (&s)[8]) {
  float r[8], finite = 0.f;
  uint32_t tie = 0xffffffffu;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float p = b[i] * s[i];
    const float e = fmaf(b[i], s[i], -p);
    r[i] = fmaf(a[i], c[i], p) + e;
    finite = fmaf(r[i], 0.f, finite);                                   // NaN if r is not finite
    tie = min(tie, __float_as_uint(r[i]) * 65536u + 0x80020000u);       // the low half, with ties moved to 0 .. 4
  }
  if (tie < 0x00050000u || finite != 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (__float_as_uint(r[i]) * 65536u + 0x80020000u < 0x00050000u || r[i] * 0.f != 0.f)
        r[i] = turn_exact(a[i], c[i], b[i], s[i]);
  }
  return make_uint4(pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3]), pack_bf16x2(r[4], r[5]), pack_bf16x2(r[6], r[7]));
}

__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w, float inv) {
  return f32x2_to_e4m3x2(lo_f32(w) * inv, hi_f32(w) * inv);
}

// Quantise 32 dims held as 8 by each of 4 adjacent lanes (j = lane & 3) and
// store them (all lanes of the warp call): lane j writes the chunk's j-th 4 bytes, lane 0 its scale.  Codes
// come from x * (1 / s), which tells every rounding but those next to a tie;
// those are told by the exact rest x - n s.  A chunk with an odd scale (zero,
// subnormal, clamped, NaN) is divided.
template <int D>
__device__ __forceinline__ void store_int4(uint8_t* record, int block_size, int row, int chunk, int j, uint4 x,
                                           bool store) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  // bf16 magnitudes order as integers, NaN above infinity above all
  uint32_t m2 = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu), __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
  m2 = __vmaxu2(m2, __shfl_xor_sync(FULL_MASK, m2, 1));
  m2 = __vmaxu2(m2, __shfl_xor_sync(FULL_MASK, m2, 2));
  const uint32_t top_bits = max(m2 & 0xffffu, m2 >> 16);
  const float m = fminf(__uint_as_float(top_bits << 16), 458528.f);  // 7 * 65504, the largest scale's
  // m / 7 rounded to nearest: the quotient by the rounded reciprocal, corrected by its exact residual
  float top = m * 0.142857149243354797f;
  top = fmaf(fmaf(-7.f, top, m), 0.142857149243354797f, top);
  const __half h = top_bits > 0x7f80u ? __ushort_as_half(0x7fff) : __float2half_rn(top);
  const float s = __half2float(h);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  float f[8], n[8], far = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = lo_f32(w[i]);
    f[2 * i + 1] = hi_f32(w[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    n[i] = fmaf(f[i], inv, 12582912.f);  // 1.5 2^23: the nearest integer, ties to even, in the low bits
    far = fmaxf(far, fabsf(fmaf(f[i], inv, 12582912.f - n[i])));
  }
  if (!(s >= 6.2e-5f) || top_bits > 0x48e0u) {  // (0x48e0: 458752, where the scale is clamped)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = s > 0.f ? rintf(__fdiv_rn(f[i], s)) : 0.f;
      n[i] = fminf(fmaxf(t, -7.f), 7.f) + 12582912.f;
    }
  } else if (far > 0.49999f) {  // next to a tie (one chunk in 35: bf16 values over a scale of few bits): by the exact rest
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float k = n[i] - 12582912.f;
      const float rest = fmaf(-k, s, f[i]), twice = fabsf(rest + rest);
      if (twice > s || (twice == s && (__float_as_uint(n[i]) & 1))) n[i] += copysignf(1.f, rest);
    }
  }
  uint32_t out[4];
  const uint32_t place = 1u << (4 * j);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t pair = __byte_perm(__float_as_uint(n[2 * i]), __float_as_uint(n[2 * i + 1]), 0x5410);
    out[i] = ((pair & 0x000f000fu) ^ 0x00080008u) * place;  // n + 8
  }
  // unit 2 i + k has this lane's nibble j of dim 8 j + 2 i + k: gather the four lanes' nibbles
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    out[i] |= __shfl_xor_sync(FULL_MASK, out[i], 1);
    out[i] |= __shfl_xor_sync(FULL_MASK, out[i], 2);
  }
  const uint32_t mine = j == 0 ? out[0] : j == 1 ? out[1] : j == 2 ? out[2] : out[3];
  if (!store) return;
  *reinterpret_cast<uint32_t*>(record + int4_code_offset<D>(row, chunk) + 4 * j) = mine;
  if (j == 0) *reinterpret_cast<__half*>(record + int4_scale_offset<D>(block_size, row, chunk)) = h;
}

template <int D, Cache CACHE, Pairs PAIRS>
__global__ void __launch_bounds__(ROPE_THREADS, 4) rope_kernel(const RopeParams p, int tokens) {
  constexpr int VECS = D / 8;                       // 8 .. 32: a head's vectors lie in one warp
  constexpr int HEADS = ROPE_THREADS / VECS;        // heads a CTA takes at a time
  __shared__ int sh_pos[ROPE_MAX_TOKENS];           // -1: nothing of the row is written
  __shared__ long long sh_slot[ROPE_MAX_TOKENS];    // -1: not stored
  __shared__ float4 sh_row[PAIRS == PAIRS_NONE ? 1 : ROPE_MAX_TOKENS * D / 4];
  grid_launch_dependents();
  const int vec = threadIdx.x % VECS;
  const int h = blockIdx.y * HEADS + threadIdx.x / VECS;  // this thread's head: of q, then of k, then of v
  const bool some = h < p.num_q_heads + 2 * p.num_kv_heads;
  const bool is_q = h < p.num_q_heads, is_v = h >= p.num_q_heads + p.num_kv_heads;
  const int kh = is_q ? 0 : is_v ? h - p.num_q_heads - p.num_kv_heads : h - p.num_q_heads;
  const int bs = 1 << p.block_shift;
  const int half_vecs = p.rot_dim / 16;
  const bool turns = PAIRS != PAIRS_NONE && vec * 8 < p.rot_dim;
  const bool second = vec >= half_vecs;
  const int other = second ? vec - half_vecs : vec + half_vecs;
  const int partner = (threadIdx.x & 31) - vec % 32 + other;  // lane of the pair's other vector
  const int pair = second ? vec - half_vecs : vec;            // the vector's place in the table's half row
  const int t0 = blockIdx.x * tokens;
  const int n = min(tokens, p.num_tokens - t0);

  // The thread walks over the tokens; the vectors of the next two are on their way.
  const long long stride = is_q ? p.q_stride : is_v ? p.v_stride : p.k_stride;
  const __nv_bfloat16* src = (is_q ? p.q + static_cast<long long>(h) * D
                              : is_v ? p.v_new + static_cast<long long>(kh) * D
                                     : p.k_new + static_cast<long long>(kh) * D) + t0 * stride + vec * 8;
  const auto fetch = [&](int i) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (some && i < n) v = *reinterpret_cast<const uint4*>(src);
    src += stride;
    return v;
  };
  uint4 x0 = fetch(0), x1 = fetch(1);
  __nv_bfloat16* dst = p.q_out + (static_cast<long long>(t0) * p.num_q_heads + h) * D + vec * 8;
  const long long dst_step = static_cast<long long>(p.num_q_heads) * D;
  void* cache = is_v ? p.v_cache : p.k_cache;

  // the tokens' slots, positions and table rows
  if (threadIdx.x < n) {
    const int t = t0 + threadIdx.x;
    long long slot = p.slots[t];
    int pos = PAIRS == PAIRS_NONE ? 0 : p.positions[t], bits = 0;
    if (PAIRS != PAIRS_NONE && pos >= p.table_len) {
      bits = PA_STATUS_BIT(PA_ERR_RANGE);
      pos = -1;
    }
    if (pos >= 0 && slot >= p.num_slots) {
      bits = PA_STATUS_BIT(PA_ERR_RANGE);
      slot = -1;
    }
    if (bits && blockIdx.y == 0) set_status(p.status, bits);
    sh_pos[threadIdx.x] = pos < 0 ? -1 : pos;
    sh_slot[threadIdx.x] = slot < 0 ? -1 : slot;
  }
  __syncthreads();
  if (PAIRS != PAIRS_NONE) {
    const int words = p.rot_dim / 4;  // of a table row, by 16 bytes
    for (int t = threadIdx.x / 32; t < n; t += ROPE_THREADS / 32) {
      const int pos = sh_pos[t];
      if (pos < 0) continue;
      const float4* row = reinterpret_cast<const float4*>(p.table + static_cast<long long>(pos) * p.rot_dim);
      for (int w = threadIdx.x & 31; w < words; w += 32) sh_row[t * (D / 4) + w] = __ldg(row + w);
    }
    __syncthreads();
  }

  for (int i = 0; i < n; ++i, dst += dst_step) {
    const bool mine = some && sh_pos[i] >= 0;
    uint4 out = x0, y = x0;
    if (PAIRS == PAIRS_HALF) {
      y.x = __shfl_sync(FULL_MASK, x0.x, partner);
      y.y = __shfl_sync(FULL_MASK, x0.y, partner);
      y.z = __shfl_sync(FULL_MASK, x0.z, partner);
      y.w = __shfl_sync(FULL_MASK, x0.w, partner);
    }
    if (PAIRS != PAIRS_NONE && turns && !is_v && mine) {
      const uint32_t wa[4] = {x0.x, x0.y, x0.z, x0.w}, wb[4] = {y.x, y.y, y.z, y.w};
      float a[8], b[8], c[8], s[8];
#pragma unroll
      for (int m = 0; m < 4; ++m) {  // b: the partner, its sign turned for the first of a pair
        const uint32_t w = PAIRS == PAIRS_HALF ? wb[m] ^ (second ? 0u : 0x80008000u)
                                               : __byte_perm(wa[m], wa[m], 0x1032) ^ 0x00008000u;
        a[2 * m] = lo_f32(wa[m]);
        a[2 * m + 1] = hi_f32(wa[m]);
        b[2 * m] = lo_f32(w);
        b[2 * m + 1] = hi_f32(w);
      }
      const float4* row = sh_row + i * (D / 4);
      if (PAIRS == PAIRS_HALF) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float4 cc = row[pair * 2 + k], ss = row[p.rot_dim / 8 + pair * 2 + k];
          c[4 * k] = cc.x, c[4 * k + 1] = cc.y, c[4 * k + 2] = cc.z, c[4 * k + 3] = cc.w;
          s[4 * k] = ss.x, s[4 * k + 1] = ss.y, s[4 * k + 2] = ss.z, s[4 * k + 3] = ss.w;
        }
      } else {
        const float4 cc = row[vec], ss = row[p.rot_dim / 8 + vec];
        c[0] = c[1] = cc.x, c[2] = c[3] = cc.y, c[4] = c[5] = cc.z, c[6] = c[7] = cc.w;
        s[0] = s[1] = ss.x, s[2] = s[3] = ss.y, s[4] = s[5] = ss.z, s[6] = s[7] = ss.w;
      }
      out = turn(a, b, c, s);
    }
    x0 = x1;
    x1 = fetch(i + 2);  // (q in place: a vector is fetched and stored by its own thread, its pair's came by the exchange)
    if (mine && is_q) *reinterpret_cast<uint4*>(dst) = out;
    const long long slot = sh_slot[i];
    const bool store = mine && !is_q && slot >= 0;
    const long long head = (slot >> p.block_shift) * p.num_kv_heads + kh;
    const int off = static_cast<int>(slot & (bs - 1));
    if (CACHE == CACHE_BF16) {
      if (store) static_cast<uint4*>(cache)[(head * bs + off) * VECS + vec] = out;
    } else if (CACHE == CACHE_E4M3) {
      const float inv = is_v ? p.v_inv : p.k_inv;
      if (store)
        static_cast<uint2*>(cache)[(head * bs + off) * VECS + vec] =
            make_uint2(e4m3_pair(out.x, inv) | (e4m3_pair(out.y, inv) << 16),
                       e4m3_pair(out.z, inv) | (e4m3_pair(out.w, inv) << 16));
    } else if (__any_sync(FULL_MASK, store)) {  // whole warps: their lanes exchange codes
      store_int4<D>(static_cast<uint8_t*>(cache) + head * int4_record_bytes(bs, D), bs, off, vec >> 2, vec & 3, out,
                    store);
    }
  }
}

// Rows of the 4-bit cache as values: one thread per 4 dims (k, then v), so that a warp stores whole lines.
template <int D>
__global__ void __launch_bounds__(ROPE_THREADS)
    read_int4_kernel(float* k_out, float* v_out, const uint8_t* k_cache, const uint8_t* v_cache, const int32_t* slots,
                     int num_tokens, int num_kv_heads, int block_shift, long long num_slots, int tokens, int* status) {
  constexpr int VECS = D / 4, HEADS = ROPE_THREADS / VECS;
  const int vec = threadIdx.x % VECS, chunk = vec >> 3, bs = 1 << block_shift;
  const int j = vec >> 1 & 3;    // dims 8 j + 4 half .. + 3 of the chunk: nibble j of four units
  const int half = vec & 1;
  __shared__ long long sh_slot[ROPE_MAX_TOKENS];
  const int t0 = blockIdx.x * tokens, n = min(tokens, num_tokens - t0);
  if (threadIdx.x < n) {
    const long long slot = slots[t0 + threadIdx.x];
    if (slot >= num_slots && blockIdx.y == 0) set_status(status, PA_STATUS_BIT(PA_ERR_RANGE));
    sh_slot[threadIdx.x] = slot < num_slots ? slot : -1;
  }
  __syncthreads();
  const int h = blockIdx.y * HEADS + threadIdx.x / VECS;
  if (h >= 2 * num_kv_heads) return;
  const bool is_v = h >= num_kv_heads;
  const int kh = is_v ? h - num_kv_heads : h;
  const uint8_t* cache = is_v ? v_cache : k_cache;
  float4* dst = reinterpret_cast<float4*>((is_v ? v_out : k_out) + (static_cast<long long>(t0) * num_kv_heads + kh) * D) + vec;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const long long slot = sh_slot[i];
    if (slot < 0) continue;
    const int off = static_cast<int>(slot & (bs - 1));
    const uint8_t* rec = cache + ((slot >> block_shift) * num_kv_heads + kh) * int4_record_bytes(bs, D);
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(rec + int4_code_offset<D>(off, chunk) + 8 * half));
    const float s = __half2float(__ldg(reinterpret_cast<const __half*>(rec + int4_scale_offset<D>(bs, off, chunk))));
    const uint32_t u[2] = {w.x >> (4 * j), w.y >> (4 * j)};
    float f[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      f[k] = static_cast<float>(static_cast<int>(u[k >> 1] >> (16 * (k & 1)) & 15) - 8) * s;
    dst[static_cast<long long>(i) * num_kv_heads * VECS] = make_float4(f[0], f[1], f[2], f[3]);
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
  const long long runs = (static_cast<long long>(table_len) + ROPE_RUN - 1) / ROPE_RUN;
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

// x: runs of tokens, y: heads.  A CTA's slots, positions and table rows are fetched once, then its tokens stream: as
// many as leave the GPU four CTAs an SM.
dim3 row_grid(int num_tokens, int heads, int heads_per_cta, int num_sms, int* tokens) {
  const int y = (heads + heads_per_cta - 1) / heads_per_cta;
  const long long n = static_cast<long long>(num_tokens) * y / (num_sms * 4ll);
  *tokens = static_cast<int>(n < 1 ? 1 : n > ROPE_MAX_TOKENS ? ROPE_MAX_TOKENS : n);
  return dim3(static_cast<unsigned>((num_tokens + *tokens - 1) / *tokens), static_cast<unsigned>(y));
}

template <int D, Cache CACHE, Pairs PAIRS>
int launch_rope(const RopeParams& p, cudaStream_t stream, int num_sms) {
  int tokens;
  const dim3 grid = row_grid(p.num_tokens, p.num_q_heads + 2 * p.num_kv_heads, ROPE_THREADS / (D / 8), num_sms, &tokens);
  rope_kernel<D, CACHE, PAIRS><<<grid, ROPE_THREADS, 0, stream>>>(p, tokens);
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
      (sc.original_positions <= 0 || !(sc.low > 0.0) || !(sc.high > sc.low) || !(sc.high < INFINITY)))
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
  int tokens;
  const dim3 grid = pa::row_grid(num_tokens, 2 * num_kv_heads, pa::ROPE_THREADS / (head_dim / 4), di.num_sms, &tokens);
  const auto kernel = head_dim == 64    ? pa::read_int4_kernel<64>
                      : head_dim == 128 ? pa::read_int4_kernel<128>
                                        : pa::read_int4_kernel<256>;
  kernel<<<grid, pa::ROPE_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(
      k_out, v_out, static_cast<const uint8_t*>(k_cache), static_cast<const uint8_t*>(v_cache), slot_mapping,
      num_tokens, num_kv_heads, shift, slots, tokens, dev_status);
  return pa::check_launch(cudaSuccess, "read_int4_kernel launch");
}

}  // extern "C"

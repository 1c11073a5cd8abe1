// Shared pieces of the rotated key/value cache kernels: where a token lives,
// rotary angles, and the head rotation H_d diag(s) / sqrt(d) of a vector held
// by a few lanes.
#pragma once
#include "device.cuh"
#include "kv.h"
#include "kv_turn.h"

namespace hit {

// A token's sequence, position and place.
struct KvToken {
  int seq;       // -1: the token belongs to no sequence
  int64_t pos;   // position in the sequence (may be negative)
  int64_t slot;  // page * kv_heads * page_size + offset of head 0, or -1
};

// Number of i in [0, seqs] with cu[i] <= t, found by the whole warp: every
// step probes 32 evenly spaced entries at once, so that the chain of dependent
// loads is log32(seqs) long.  For an ascending cu this is the token's sequence
// plus one; for any other contents it is some value in [0, seqs + 1].
__device__ __forceinline__ int kv_count_le(const int32_t* __restrict__ cu, int seqs, int64_t t, int lane) {
  int lo = 0, n = seqs + 1;  // the count is in [lo, lo + n]
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int i = lane * step;  // probes lo + i, the first of its piece
    const bool le = i < n && __ldg(cu + lo + i) <= t;
    const int k = __popc(__ballot_sync(0xffffffffu, le));
    if (k == 0) return lo;
    lo += (k - 1) * step + 1;
    const int left = n - ((k - 1) * step + 1);
    n = left < step - 1 ? left : step - 1;
  }
  return lo;
}

// Slot of position p of sequence s, or -1 where it does not exist.
__device__ __forceinline__ int64_t kv_slot(const KvArgs& a, int s, int64_t p) {
  if (p < 0) return -1;
  const int64_t c = p >> a.log_page;
  if (c >= a.max_pages) return -1;
  const int64_t page = __ldg(a.table + int64_t(s) * a.ld_table + c);
  if (page < 0 || page >= a.pages) return -1;
  return ((page * a.hk) << a.log_page) + (p & ((int64_t(1) << a.log_page) - 1));
}

// Token t of the call (whole warp, same t).
__device__ __forceinline__ KvToken kv_token(const KvArgs& a, int64_t t, int lane) {
  KvToken k{-1, 0, -1};
  int64_t b, e, len;
  int s;
  if (a.seqs < 32) {  // every boundary and length is some lane's: one round of loads
    const int cu = lane <= a.seqs ? __ldg(a.cu + lane) : 0;
    const int ln = lane < a.seqs ? __ldg(a.lens + lane) : 0;
    const int c = __popc(__ballot_sync(0xffffffffu, lane <= a.seqs && cu <= t));
    if (c < 1 || c > a.seqs) return k;
    s = c - 1;
    b = __shfl_sync(0xffffffffu, cu, s);
    e = __shfl_sync(0xffffffffu, cu, c);
    len = __shfl_sync(0xffffffffu, ln, s);
  } else {
    const int c = kv_count_le(a.cu, a.seqs, t, lane);
    if (c < 1 || c > a.seqs) return k;
    s = c - 1;
    b = __ldg(a.cu + s), e = __ldg(a.cu + s + 1), len = __ldg(a.lens + s);
  }
  if (t < b || t >= e) return k;
  k.seq = s;
  k.pos = len - (e - b) + (t - b);
  k.slot = kv_slot(a, s, k.pos);
  return k;
}

// Tokens t0 + lane of the call, one to a lane (lanes from n on: none).
__device__ __forceinline__ KvToken kv_tokens(const KvArgs& a, int64_t t0, int n, int lane) {
  KvToken k{-1, 0, -1};
  const int64_t t = t0 + lane;
  int64_t b = 0, e = 0, len = 0;
  int s = -1;
  if (a.seqs < 32) {  // every boundary and length is some lane's: one round of loads
    const int cu = lane <= a.seqs ? __ldg(a.cu + lane) : 0;
    const int ln = lane < a.seqs ? __ldg(a.lens + lane) : 0;
    int c = 0;
    for (int i = 0; i <= a.seqs; ++i) c += __shfl_sync(0xffffffffu, cu, i) <= t;
    s = c - 1;
    b = __shfl_sync(0xffffffffu, cu, max(s, 0));
    e = __shfl_sync(0xffffffffu, cu, min(c, 31));
    len = __shfl_sync(0xffffffffu, ln, max(s, 0));
    if (s >= a.seqs) s = -1;
  } else {
    s = kv_count_le(a.cu, a.seqs, t0, lane) - 1;  // of the first token; the others are a few sequences on
    while (s < a.seqs && __ldg(a.cu + s + 1) <= t) ++s;
    if (s >= a.seqs) s = -1;
    if (s >= 0) b = __ldg(a.cu + s), e = __ldg(a.cu + s + 1), len = __ldg(a.lens + s);
  }
  if (lane >= n || s < 0 || t < b || t >= e) return k;
  k.seq = s;
  k.pos = len - (e - b) + (t - b);
  k.slot = kv_slot(a, s, k.pos);
  return k;
}

// Rotary angles.  A frequency is held as the fraction of a turn that one
// position makes, in units of 2^-64: a position times it, modulo 2^64, is the
// angle's fraction of a turn, exactly, in one integer product (in fp32 a
// position of 10^6 would leave no correct digits).  kv_turn gives the units of
// a frequency, found in fp64 once per CTA and pair.
__device__ __forceinline__ uint64_t kv_turn(const KvArgs& a, int j) {
  const double f = double(__ldg(a.inv_freq + j)) * 0.15915494309189533577;
  return __double2ull_rz((f - floor(f)) * 18446744073709551616.0);
}
// The table of all pairs; followed by a barrier of the caller's.
__device__ __forceinline__ void kv_turns(const KvArgs& a, uint64_t* turns, int thread, int threads) {
  for (int j = thread; j < a.n_freq; j += threads) turns[j] = kv_turn(a, j);
}
// Position that pair j of token t (at sequence position pos) turns by.
__device__ __forceinline__ int kv_turn_pos(const KvArgs& a, int64_t t, int pos, int j) {
  if (a.positions == nullptr) return pos;
  const int ax = a.rope_axis != nullptr ? __ldg(a.rope_axis + j) : 0;
  // a pair without an axis is not turned
  return ax < 0 || ax >= a.rope_axes ? 0 : __ldg(a.positions + int64_t(ax) * a.ld_pos + t);
}
// Twice the angle's fraction of a turn, in [-1, 1].
__device__ __forceinline__ float kv_halfturns(int pos, uint64_t turn) {
  return float(kv_fraction(pos, turn)) * 4.656612873077393e-10f;
}
// (cos, sin) to fp32's precision, for keys.
__device__ __forceinline__ float2 kv_angle(const KvArgs& a, const uint64_t* turns, int64_t t, int pos, int j) {
  float s, c;
  sincospif(kv_halfturns(kv_turn_pos(a, t, pos, j), turns[j]), &s, &c);
  return make_float2(c, s);
}
// The same to an absolute error below 2^-19 by the hardware's functions (2^-21.2 on this
// range, the argument's roundings as much again), for queries, which are rounded to
// 2^-11 after their turn.
__device__ __forceinline__ float2 kv_angle_fast(const KvArgs& a, const uint64_t* turns, int64_t t, int pos, int j) {
  const float x = kv_halfturns(kv_turn_pos(a, t, pos, j), turns[j]) * 3.14159265358979f;
  return make_float2(__cosf(x), __sinf(x));
}

// ---------------------------------------------------------------------------
// A head vector of D elements on LPV = D / 32 neighbouring lanes: lane l of
// them holds the four 8-element chunks l, l + LPV, l + 2 LPV, l + 3 LPV
// (x[8 c + e] = element 8 (c LPV + l) + e), so that loads of a chunk are
// coalesced over the lanes and five of the log2 D Hadamard stages are
// register stages.
// ---------------------------------------------------------------------------
template <int D>
struct KvLanes {
  static constexpr int LPV = D / 32;
  static constexpr int LOG = LPV == 2 ? 1 : LPV == 4 ? 2 : 3;
};

// Unnormalised Hadamard transform of the vector.
template <int D>
__device__ __forceinline__ void kv_hadamard(float (&x)[32], int l) {
  reg_stages<32, 0, 5>(x);
#pragma unroll
  for (int b = 0; b < KvLanes<D>::LOG; ++b) shfl_stage<32>(x, b, (l >> b) & 1);
}

// Table of signs times `norm` for the elements of a head, by the whole CTA, with
// PAD floats between its quarters.
template <int D, int PAD>
__device__ __forceinline__ void kv_factors(float* f, const int8_t* __restrict__ signs, float norm) {
  for (int i = threadIdx.x; i < D; i += blockDim.x)
    f[i + i / (D / 4) * PAD] = signs != nullptr && __ldg(signs + i) < 0 ? -norm : norm;
}
// x <- x * f elementwise, f a table of the head's elements.
template <int D>
__device__ __forceinline__ void kv_times(float (&x)[32], const float* f, int l) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float4* q = reinterpret_cast<const float4*>(f + 8 * (c * KvLanes<D>::LPV + l));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 g = q[h];
      float* y = x + 8 * c + 4 * h;
      mul_x2(y[0], y[1], g.x, g.y);
      mul_x2(y[2], y[3], g.z, g.w);
    }
  }
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// max that keeps a NaN
__device__ __forceinline__ float kv_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The power of two of a row whose largest absolute element has the bits m, and
// its reciprocal; 1 for an infinity or a NaN, which are left to spread.
__device__ __forceinline__ void kv_row_power(uint32_t m, float& up, float& down) {
  const uint32_t ex = max(1u, m >> 23);
  const bool odd = ex == 255;
  up = odd ? 1.0f : __uint_as_float(ex << 23);
  down = odd ? 1.0f : __uint_as_float(ex == 254 ? 0x00400000u : (254 - ex) << 23);
}
// The same of a whole vector: x * down is in [-2, 2), where fp16 keeps it to half
// a step of 2^-10 of its largest element or better.
template <int D>
__device__ __forceinline__ void kv_row_power(const float (&x)[32], float& up, float& down) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
  for (int b = 0; b < KvLanes<D>::LOG; ++b) m = max(m, __shfl_xor_sync(0xffffffffu, m, 1 << b));
  kv_row_power(m, up, down);
}

// Eight consecutive elements as fp32.
template <bool F32>
__device__ __forceinline__ void kv_load8(const void* p, int64_t at, float* x) {
  if constexpr (F32) {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 a = __ldg(s), b = __ldg(s + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at));
    bf16x2_to_f32(w.x, x[0], x[1]);
    bf16x2_to_f32(w.y, x[2], x[3]);
    bf16x2_to_f32(w.z, x[4], x[5]);
    bf16x2_to_f32(w.w, x[6], x[7]);
  }
}
template <bool F32>
__device__ __forceinline__ void kv_store8(void* p, int64_t at, const float* x) {
  if constexpr (F32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
    d[0] = make_float4(x[0], x[1], x[2], x[3]);
    d[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + at) =
        make_uint4(f32_to_bf16x2(x[0], x[1]), f32_to_bf16x2(x[2], x[3]), f32_to_bf16x2(x[4], x[5]),
                   f32_to_bf16x2(x[6], x[7]));
  }
}

// Zeros in the rows of tokens [0, lo) and [hi, tokens) of out, 16 bytes a thread;
// thread: this one's number among `threads`.
__device__ __forceinline__ void kv_zero_rows(void* out, int64_t lo, int64_t hi, int64_t tokens, int heads, int row_bytes,
                                             int64_t token_bytes, int64_t head_bytes, int64_t thread, int64_t threads) {
  lo = max(int64_t(0), min(lo, tokens));
  hi = max(lo, min(hi, tokens));
  const int pieces = row_bytes / 16;
  const int64_t of_token = int64_t(heads) * pieces, n = (lo + tokens - hi) * of_token;
  for (int64_t i = thread; i < n; i += threads) {
    const int64_t r = i / of_token, t = r < lo ? r : r - lo + hi;
    const int in = int(i - r * of_token), h = in / pieces;
    uint8_t* const p = static_cast<uint8_t*>(out) + t * token_bytes + h * head_bytes + (in - h * pieces) * 16;
    *reinterpret_cast<uint4*>(p) = make_uint4(0, 0, 0, 0);
  }
}

// The rotary turn of a vector whose elements start at p + at; cs holds the
// token's (cos, sin) pairs.
template <int D, bool F32>
__device__ __forceinline__ void kv_rope(float (&x)[32], const void* p, int64_t at, const float2* cs, int n_freq,
                                        bool interleaved, int l) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int i0 = 8 * (c * KvLanes<D>::LPV + l);
    if (i0 >= 2 * n_freq) continue;
    float* v = x + 8 * c;
    if (interleaved) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 t = cs[(i0 + e) / 2];
        const float u = v[e], w = v[e + 1];
        v[e] = u * t.x - w * t.y;
        v[e + 1] = u * t.y + w * t.x;
      }
    } else if (2 * n_freq == D) {  // both chunks of a pair are the lane's own
      if (c >= 2) continue;
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float4 t = *reinterpret_cast<const float4*>(cs + i0 + e);
        const float u0 = v[e], u1 = v[e + 1], w0 = v[16 + e], w1 = v[17 + e];
        v[e] = u0 * t.x - w0 * t.y;
        v[16 + e] = u0 * t.y + w0 * t.x;
        v[e + 1] = u1 * t.z - w1 * t.w;
        v[17 + e] = u1 * t.w + w1 * t.z;
      }
    } else {
      // the partner chunk lies n_freq elements on or back (n_freq % 8 == 0)
      const bool low = i0 < n_freq;
      float o[8];
      kv_load8<F32>(p, at + (low ? i0 + n_freq : i0 - n_freq), o);
      const int j0 = low ? i0 : i0 - n_freq;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 t = cs[j0 + e];
        v[e] = low ? v[e] * t.x - o[e] * t.y : o[e] * t.y + v[e] * t.x;
      }
    }
  }
}

}  // namespace hit

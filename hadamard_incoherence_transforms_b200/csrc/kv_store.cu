// Appending to and reading from the rotated key/value cache.
//
// Append: per (token, head) vector u = H diag(s) rope(x) / sqrt(d), absmax
// RTN with one scale per vector, codes and scale to the token's slot.  Read:
// R^-1 (q s) = diag(s) H (q s) / sqrt(d).  Both touch every byte once and do
// log2 d + a few operations per element, so memory bounds them for long calls
// and latency for short ones.  A vector sits on d / 32 lanes (32 elements
// each), which leaves only 1 to 3 of the 6 to 8 Hadamard stages to shuffles.
#include "kv.cuh"

#include <algorithm>

namespace hit {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTile = 64;  // tokens per CTA
constexpr int kAppendCtas = 2, kReadCtas = 4;  // CTAs on an SM

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Stored codes of the vector x and its scale.  All LPV lanes of the vector call it
// together.  The usual case takes t = y / s by the correctly rounded quotient:
// q0 = y r with r = RN(1/s), one correction step (exact remainder), and the code in
// the low byte of t + 1.5 * 2^23 + 2^(b-1) (ties to even), on pairs.
template <int D, int BITS>
__device__ __forceinline__ float kv_quantize(float (&x)[32], uint32_t (&w)[BITS]) {
  constexpr int QMAX = (1 << (BITS - 1)) - 1;
  constexpr float MAGIC = 12582912.0f + float(1 << (BITS - 1));
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) a = max_nan(a, fabsf(x[i]));
#pragma unroll
  for (int b = 0; b < KvLanes<D>::LOG; ++b) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, 1 << b));
  float s = __fdiv_rn(a, float(QMAX));
  if (!(a < INFINITY)) s = __uint_as_float(0x7fc00000u);
  uint32_t u[32];
  if (a > 7.9e-31f && a < 1.2e30f) {  // quotient, remainder and reciprocal stay normal
    const float r = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      float q0 = x[i], q1 = x[i + 1], e0, e1;
      mul_x2(q0, q1, r, r);
      fma_x2(q0, q1, -s, -s, x[i], x[i + 1], e0, e1);
      fma_x2(e0, e1, r, r, q0, q1, q0, q1);
      fma_x2(q0, q1, 1.0f, 1.0f, MAGIC, MAGIC, q0, q1);
      u[i] = __float_as_uint(q0);
      u[i + 1] = __float_as_uint(q1);
    }
  } else {
    const bool live = s > 0.0f;  // false for s = 0 and for NaN
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float t = live ? fminf(fmaxf(__fdiv_rn(x[i], s), -float(QMAX)), float(QMAX)) : 0.0f;
      u[i] = __float_as_uint(t + MAGIC);
    }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if constexpr (BITS == 4) {
      w[c] = pack4x8(u + 8 * c);
    } else {
      w[2 * c] = low_bytes4(u[8 * c], u[8 * c + 1], u[8 * c + 2], u[8 * c + 3]);
      w[2 * c + 1] = low_bytes4(u[8 * c + 4], u[8 * c + 5], u[8 * c + 6], u[8 * c + 7]);
    }
  }
  return s;
}

// Codes of eight elements (4 or 8 bytes) as fp32: the byte under 2^23's exponent,
// minus 2^23 and the offset, exact.
template <int BITS>
__device__ __forceinline__ void kv_dequantize(const uint32_t* w, float* z) {
  constexpr float OFF = -(8388608.0f + float(1 << (BITS - 1)));
  const uint32_t a = BITS == 4 ? w[0] & 0x0f0f0f0fu : w[0], b = BITS == 4 ? (w[0] >> 4) & 0x0f0f0f0fu : w[1];
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    // 4 bits: a holds the even elements, b the odd ones; 8 bits: a the first four
    const uint32_t w0 = BITS == 4 ? a : e < 4 ? a : b, w1 = BITS == 4 ? b : w0;
    const int i0 = BITS == 4 ? e / 2 : e % 4, i1 = BITS == 4 ? e / 2 : e % 4 + 1;
    float x0 = __uint_as_float(__byte_perm(w0, 0x4b000000u, 0x7650 | i0));
    float x1 = __uint_as_float(__byte_perm(w1, 0x4b000000u, 0x7650 | i1));
    fma_x2(x0, x1, 1.0f, 1.0f, OFF, OFF, z[e], z[e + 1]);
  }
}

struct Tile {
  KvToken tok[kMaxTile];
};

// A CTA's tile of tokens; vector v of it is token v / (2 hk), keys of all heads
// before values.
template <int D, int BITS, bool F32>
__global__ void __launch_bounds__(kThreads, kAppendCtas) k_kv_append(const KvArgs a, const KvDense x, int tile, float norm) {
  constexpr int LPV = KvLanes<D>::LPV;
  extern __shared__ __align__(16) float2 cs[];  // [tile][n_freq]
  __shared__ Tile tl;
  __shared__ uint64_t turns[D / 2];
  __shared__ __align__(16) float factors[2][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  const int64_t t0 = int64_t(blockIdx.x) * tile;
  const int nt = int(min(int64_t(tile), a.tokens - t0));
  const int l = threadIdx.x % LPV;
  const int vectors = nt * 2 * a.hk, per = blockDim.x / LPV;
  struct Place {
    int j, h;
    bool in, is_v;
  };
  auto place = [&](int v) {
    Place p;
    p.in = v < vectors;
    p.j = p.in ? v / (2 * a.hk) : 0;
    const int r = p.in ? v - p.j * 2 * a.hk : 0;
    p.is_v = r >= a.hk;
    p.h = p.is_v ? r - a.hk : r;
    return p;
  };
  // a vector's pieces as they lie in memory, 16 bytes each
  constexpr int RAW = F32 ? 8 : 4;
  uint4 raw[RAW];
  auto load = [&](const Place& p) {
    const void* src = p.is_v ? x.v : x.k;
    const int64_t at = (t0 + p.j) * (p.is_v ? x.v_ts : x.k_ts) + p.h * (p.is_v ? x.v_hs : x.k_hs);
#pragma unroll
    for (int c = 0; c < RAW; ++c) {
      raw[c] = make_uint4(0, 0, 0, 0);
      const int64_t e = at + (F32 ? 8 * ((c >> 1) * LPV + l) + 4 * (c & 1) : 8 * (c * LPV + l));
      if (p.in) raw[c] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(src) + e * (F32 ? 4 : 2)));
    }
  };
  Place p = place(threadIdx.x / LPV);
  load(p);  // the first vectors are on their way while their places are found
  for (int j = 32 * warp; j < nt; j += 32 * nw) {
    const KvToken k = kv_tokens(a, t0 + j, nt - j, lane);
    if (j + lane < nt) tl.tok[j + lane] = k;
  }
  kv_turns(a, turns, threadIdx.x, blockDim.x);
  kv_factors<D>(factors[0], a.k_signs, norm);
  kv_factors<D>(factors[1], a.v_signs, norm);
  __syncthreads();
  for (int i = threadIdx.x; i < nt * a.n_freq; i += blockDim.x) {
    const int j = i / a.n_freq, f = i - j * a.n_freq;
    if (tl.tok[j].slot >= 0) cs[i] = kv_angle(a, turns, t0 + j, int(tl.tok[j].pos), f);
  }
  __syncthreads();
  for (int v0 = 0; v0 < vectors; v0 += per) {  // every lane stays in the loop for the shuffles
    float y[32];
#pragma unroll
    for (int c = 0; c < RAW; ++c) {
      if constexpr (F32) {
        y[4 * c] = __uint_as_float(raw[c].x), y[4 * c + 1] = __uint_as_float(raw[c].y);
        y[4 * c + 2] = __uint_as_float(raw[c].z), y[4 * c + 3] = __uint_as_float(raw[c].w);
      } else {
        bf16x2_to_f32(raw[c].x, y[8 * c], y[8 * c + 1]);
        bf16x2_to_f32(raw[c].y, y[8 * c + 2], y[8 * c + 3]);
        bf16x2_to_f32(raw[c].z, y[8 * c + 4], y[8 * c + 5]);
        bf16x2_to_f32(raw[c].w, y[8 * c + 6], y[8 * c + 7]);
      }
    }
    const Place p = place(v0 + int(threadIdx.x) / LPV);
    if (v0 + per < vectors) load(place(v0 + per + int(threadIdx.x) / LPV));  // the next vectors
    const int64_t slot = tl.tok[p.j].slot;
    const bool live = p.in && slot >= 0;
    if (live && !p.is_v && a.n_freq > 0)
      kv_rope<D, F32>(y, x.k, (t0 + p.j) * x.k_ts + p.h * x.k_hs, cs + p.j * a.n_freq, a.n_freq, a.interleaved, l);
    kv_times<D>(y, factors[p.is_v], l);
    kv_hadamard<D>(y, l);
    uint32_t w[BITS];
    const float s = kv_quantize<D, BITS>(y, w);
    if (live) {
      const int64_t vec = slot + (int64_t(p.h) << a.log_page);
      uint8_t* dst = (p.is_v ? a.v_codes : a.k_codes) + vec * (D * BITS / 8);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if constexpr (BITS == 4)
          reinterpret_cast<uint32_t*>(dst)[c * LPV + l] = w[c];
        else
          reinterpret_cast<uint2*>(dst)[c * LPV + l] = make_uint2(w[2 * c], w[2 * c + 1]);
      }
      if (l == 0) (p.is_v ? a.v_scales : a.k_scales)[vec] = s;
    }
  }
}

template <int D, int BITS, bool F32>
__global__ void __launch_bounds__(kThreads, kReadCtas) k_kv_read(const KvArgs a, const KvDense y, int tile, float norm) {
  constexpr int LPV = KvLanes<D>::LPV;
  __shared__ Tile tl;
  __shared__ __align__(16) float factors[2][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  const int64_t t0 = int64_t(blockIdx.x) * tile;
  const int nt = int(min(int64_t(tile), a.tokens - t0));
  for (int j = 32 * warp; j < nt; j += 32 * nw) {
    const KvToken k = kv_tokens(a, t0 + j, nt - j, lane);
    if (j + lane < nt) tl.tok[j + lane] = k;
  }
  kv_factors<D>(factors[0], a.k_signs, norm);
  kv_factors<D>(factors[1], a.v_signs, norm);
  __syncthreads();
  const int l = threadIdx.x % LPV;
  const int vectors = nt * 2 * a.hk;
  const int per = blockDim.x / LPV;
  struct Row {
    int64_t at;
    void* dst;  // NULL: not to be written
    bool is_v, there;
  };
  uint32_t w[BITS];  // the lane's codes
  float s = 0.0f;
  auto load = [&](int v) {
    Row r{0, nullptr, false, false};
    s = 0.0f;
    if (v >= vectors) return r;
    const int j = v / (2 * a.hk), i = v - j * 2 * a.hk;
    r.is_v = i >= a.hk;
    const int h = r.is_v ? i - a.hk : i;
    void* const dst = const_cast<void*>(r.is_v ? y.v : y.k);
    if (tl.tok[j].seq < 0 || dst == nullptr) return r;
    r.dst = dst;
    r.at = (t0 + j) * (r.is_v ? y.v_ts : y.k_ts) + h * (r.is_v ? y.v_hs : y.k_hs);
    const int64_t slot = tl.tok[j].slot;
    if (slot < 0) return r;
    r.there = true;
    const int64_t vec = slot + (int64_t(h) << a.log_page);
    const uint8_t* src = (r.is_v ? a.v_codes : a.k_codes) + vec * (D * BITS / 8);
    s = __ldg((r.is_v ? a.v_scales : a.k_scales) + vec);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if constexpr (BITS == 4) {
        w[c] = __ldg(reinterpret_cast<const uint32_t*>(src) + c * LPV + l);
      } else {
        const uint2 t = __ldg(reinterpret_cast<const uint2*>(src) + c * LPV + l);
        w[2 * c] = t.x, w[2 * c + 1] = t.y;
      }
    }
    return r;
  };
  Row next = load(threadIdx.x / LPV);
  for (int v0 = 0; v0 < vectors; v0 += per) {
    const Row row = next;
    const float scale = s;
    float z[32];
#pragma unroll
    for (int c = 0; c < 4; ++c) kv_dequantize<BITS>(w + c * (BITS / 4), z + 8 * c);
    if (!row.there) {
#pragma unroll
      for (int i = 0; i < 32; ++i) z[i] = 0.0f;
    }
    if (v0 + per < vectors) next = load(v0 + per + int(threadIdx.x) / LPV);  // the next codes
    kv_hadamard<D>(z, l);  // of whole numbers: exact
    if (row.dst != nullptr) {
#pragma unroll
      for (int i = 0; i < 32; i += 2) mul_x2(z[i], z[i + 1], scale, scale);
      kv_times<D>(z, factors[row.is_v], l);
#pragma unroll
      for (int c = 0; c < 4; ++c) kv_store8<F32>(row.dst, row.at + 8 * (c * LPV + l), z + 8 * c);
    }
  }
}

// Tokens per CTA such that the CTAs that fit the GPU at once (`ctas` on an SM)
// share them evenly: a CTA finds its tokens' places once and then has the next
// vectors on their way while it works on these.
int pick_tile(int64_t tokens, int ctas, int most) {
  const int64_t at_once = 148 * ctas;
  return int(std::max<int64_t>(1, std::min<int64_t>(most, (tokens + at_once - 1) / at_once)));
}
int pick_threads(int tile, int hk, int lpv) {
  const int64_t want = int64_t(tile) * 2 * hk * lpv;
  return int(std::min<int64_t>(kThreads, (want + 31) / 32 * 32));
}
float norm_of(int d) { return d == 64 ? 0.125f : d == 256 ? 0.0625f : 0.08838834764831845f; }

template <typename F>
cudaError_t by_format(const KvArgs& a, int dt, F f) {
  const bool f32 = dt == 0;
  if (a.head_dim == 64)
    return a.bits == 4 ? (f32 ? f.template go<64, 4, true>() : f.template go<64, 4, false>())
                       : (f32 ? f.template go<64, 8, true>() : f.template go<64, 8, false>());
  if (a.head_dim == 128)
    return a.bits == 4 ? (f32 ? f.template go<128, 4, true>() : f.template go<128, 4, false>())
                       : (f32 ? f.template go<128, 8, true>() : f.template go<128, 8, false>());
  return a.bits == 4 ? (f32 ? f.template go<256, 4, true>() : f.template go<256, 4, false>())
                     : (f32 ? f.template go<256, 8, true>() : f.template go<256, 8, false>());
}

struct Append {
  const KvArgs& a;
  const KvDense& x;
  cudaStream_t st;
  template <int D, int BITS, bool F32>
  cudaError_t go() {
    const int tile = pick_tile(a.tokens, kAppendCtas, D == 256 ? 32 : kMaxTile);  // at most 32 KB of angles
    const unsigned grid = unsigned((a.tokens + tile - 1) / tile);
    const int threads = pick_threads(tile, a.hk, D / 32);
    k_kv_append<D, BITS, F32><<<grid, threads, size_t(tile) * a.n_freq * sizeof(float2), st>>>(a, x, tile, norm_of(D));
    return cudaGetLastError();
  }
};
struct Read {
  const KvArgs& a;
  const KvDense& y;
  cudaStream_t st;
  template <int D, int BITS, bool F32>
  cudaError_t go() {
    const int tile = pick_tile(a.tokens, kReadCtas, kMaxTile);
    const unsigned grid = unsigned((a.tokens + tile - 1) / tile);
    k_kv_read<D, BITS, F32><<<grid, pick_threads(tile, a.hk, D / 32), 0, st>>>(a, y, tile, norm_of(D));
    return cudaGetLastError();
  }
};

}  // namespace

cudaError_t launch_kv_append(const KvArgs& a, const KvDense& x, int dt, cudaStream_t st) {
  return by_format(a, dt, Append{a, x, st});
}
cudaError_t launch_kv_read(const KvArgs& a, const KvDense& y, int dt, cudaStream_t st) {
  return by_format(a, dt, Read{a, y, st});
}

}  // namespace hit

// Appending to and reading from the rotated key/value cache.
//
// Append: per (token, head) vector u = H diag(s) rope(x) / sqrt(d), absmax
// RTN with one scale per vector, codes and scale to the token's slot.  Read:
// R^-1 (q s) = diag(s) H (q s) / sqrt(d).  Both touch every byte once and do
// log2 d + a few operations per element, so memory bounds them for long calls
// and latency for short ones.  A vector sits on d / 32 lanes (32 elements
// each), which leaves only 1 to 3 of the 6 to 8 Hadamard stages to shuffles.
#include "kv.cuh"
#include "internal.h"
#include "kv_codes.cuh"

#include <algorithm>

namespace hit {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTile = 64;  // tokens per CTA
constexpr int kAppendCtas = 2, kReadCtas = 2;  // CTAs on an SM

// Stored codes of the vector x and its scale.  All LPV lanes of the vector call it
// together.  The usual case takes t = y / s by Markstein's correctly rounded
// quotient, as rows_ops.cuh does: q0 = y r with r = RN(1/s), one correction step (exact
// remainder), and the code in the low byte of t + 1.5 * 2^23 + 2^(b-1) (ties to even), on pairs.
template <int D, int BITS>
__device__ __forceinline__ float kv_quantize(float (&x)[32], uint32_t (&w)[BITS]) {
  constexpr int QMAX = (1 << (BITS - 1)) - 1;
  constexpr float MAGIC = 12582912.0f + float(1 << (BITS - 1));
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) a = kv_max(a, fabsf(x[i]));
#pragma unroll
  for (int b = 0; b < KvLanes<D>::LOG; ++b) a = kv_max(a, __shfl_xor_sync(0xffffffffu, a, 1 << b));
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

// Places of a tile's tokens: slots (kv.cuh), kNone for a token of no sequence.
constexpr int64_t kNone = -2;
struct Tile {
  int64_t slot[kMaxTile];
  int pos[kMaxTile];
  __device__ __forceinline__ void find(const KvArgs& a, int64_t t0, int nt) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int j = 32 * warp; j < nt; j += 32 * int(blockDim.x >> 5)) {
      const KvToken k = kv_tokens(a, t0 + j, nt - j, lane);
      if (j + lane < nt) {
        slot[j + lane] = k.seq < 0 ? kNone : k.slot;
        pos[j + lane] = int(k.pos);
      }
    }
  }
};
// n / d for n < 2^31 (make_fastdiv)
__device__ __forceinline__ int div_by(int n, const FastDiv& f) { return int((__umulhi(uint32_t(n), f.mul) + uint32_t(n)) >> f.shr); }

// A CTA's tile of tokens; vector v of it is token v / (2 hk), keys of all heads
// before values.
template <int D, int BITS, bool F32>
__global__ void __launch_bounds__(kThreads, kAppendCtas) k_kv_append(const KvArgs a, const KvDense x, int tile, float norm,
                                                                     FastDiv by_token) {
  constexpr int LPV = KvLanes<D>::LPV;
  extern __shared__ __align__(16) float2 cs[];  // [tile][n_freq]
  __shared__ Tile tl;
  __shared__ uint64_t turns[D / 2];
  __shared__ __align__(16) float factors[2][D];
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
    p.j = p.in ? div_by(v, by_token) : 0;
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
  tl.find(a, t0, nt);
  kv_turns(a, turns, threadIdx.x, blockDim.x);
  kv_factors<D, 0>(factors[0], a.k_signs, norm);
  kv_factors<D, 0>(factors[1], a.v_signs, norm);
  __syncthreads();
  for (int i = threadIdx.x; i < nt * a.n_freq; i += blockDim.x) {
    const int j = i / a.n_freq, f = i - j * a.n_freq;
    if (tl.slot[j] >= 0) cs[i] = kv_angle(a, turns, t0 + j, tl.pos[j], f);
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
    const int64_t slot = tl.slot[p.j];
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

// Read.  The transform of stored codes is a sum of whole numbers, exact in fp16
// and on the tensor cores, so that it takes no shuffles: a warp takes 16 vectors,
// lane (r, c) the codes of quarter c of vectors r and r + 8.  Of the log2 D element
// bits the quarter's own ones but two are butterflies on fp16 pairs in registers;
// the other two and the quarter's number are the 16 of m16n8k16's inner
// dimension, against a +-1 matrix that lies in four registers.  Its columns are
// numbered such that a lane ends with D / 4 neighbouring elements of its rows.
template <int D, int BITS, bool F32>
__global__ void __launch_bounds__(kThreads, kReadCtas) k_kv_read(const KvArgs a, const KvDense y, int tile, float norm,
                                                                 int wide, int zero, FastDiv by_heads) {
  constexpr int VB = D * BITS / 8, NW = VB / 16;  // a lane's words of a vector's codes
  constexpr int NP = D / 8;                       // ... and its fp16 pairs
  __shared__ Tile tl;
  __shared__ __align__(16) float factors[2][D + 16];  // quarters in different banks
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r8 = lane >> 2, c4 = lane & 3;
  const int64_t t0 = int64_t(blockIdx.x) * tile;
  const int nt = int(min(int64_t(tile), a.tokens - t0));
  tl.find(a, t0, nt);
  kv_factors<D, 4>(factors[0], a.k_signs, norm);
  kv_factors<D, 4>(factors[1], a.v_signs, norm);
  // the +-1 matrix: inner index (quarter c, then the pair's half and which of two
  // pairs), column 2 c' + u of tile t: c' is the output's quarter, u and t its bits
  // for the pair's number and half (4 bits), or the other way around (8 bits)
  uint32_t hm[2][2];
  {
    const int n = lane >> 2, s0 = __popc(c4 & (n >> 1)) & 1, u = n & 1;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int half = BITS == 4 ? t : u, pair = BITS == 4 ? u : t;
      auto one = [&](int h, int p) { return 0x3c00u | (uint32_t((s0 + (h & half) + (p & pair)) & 1) << 15); };
      hm[t][0] = one(0, 0) | (one(1, 0) << 16);
      hm[t][1] = one(0, 1) | (one(1, 1) << 16);
    }
  }
  __syncthreads();
  const int vectors = nt * a.hk, groups = (vectors + 15) / 16;  // of keys; as many of values
  struct Row {
    int64_t at;
    bool owned;
  };
  uint32_t code[2][NW];
  float scale[2];  // 0 for a position that does not exist: zeros, whatever the last codes were
  auto load = [&](int g, Row (&row)[2]) {
    const bool is_v = g >= groups;
    const bool wanted = (is_v ? y.v : y.k) != nullptr;
    const int64_t ts = is_v ? y.v_ts : y.k_ts, hs = is_v ? y.v_hs : y.k_hs;
    const uint8_t* const codes = (is_v ? a.v_codes : a.k_codes) + c4 * (VB / 4);
    const float* const scales = is_v ? a.v_scales : a.k_scales;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int v = (g - (is_v ? groups : 0)) * 16 + r8 + 8 * k;
      row[k] = Row{0, false};
      scale[k] = 0.0f;
      if (v >= vectors || !wanted) continue;
      const int j = div_by(v, by_heads), h = v - j * a.hk;
      const int64_t slot = tl.slot[j];
      row[k].owned = slot != kNone || zero;
      row[k].at = (t0 + j) * ts + h * hs + c4 * (D / 4);
      if (slot < 0) continue;
      const int64_t vec = slot + (int64_t(h) << a.log_page);
      const uint8_t* src = codes + vec * VB;
      scale[k] = __ldg(scales + vec);
      if constexpr (NW == 2) {
        const uint2 q = __ldg(reinterpret_cast<const uint2*>(src));
        code[k][0] = q.x, code[k][1] = q.y;
      } else {
#pragma unroll
        for (int i = 0; i < NW; i += 4) {
          const uint4 q = __ldg(reinterpret_cast<const uint4*>(src) + i / 4);
          code[k][i] = q.x, code[k][i + 1] = q.y, code[k][i + 2] = q.z, code[k][i + 3] = q.w;
        }
      }
    }
  };
  const int step = int(blockDim.x >> 5);
  Row next[2];
#pragma unroll
  for (int i = 0; i < NW; ++i) code[0][i] = code[1][i] = 0;
  if (warp < 2 * groups) load(warp, next);
  for (int g = warp; g < 2 * groups; g += step) {
    const Row row[2] = {next[0], next[1]};
    const float s[2] = {scale[0], scale[1]};
    uint32_t p[2][NP];  // pairs: 4 bits (e, e + 4), e = 0 .. 3 of each eight; 8 bits (e, e + 1)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        if constexpr (BITS == 4) {
          uint32_t h[4];
          half_of4(code[k][i], h);
#pragma unroll
          for (int e = 0; e < 4; ++e) p[k][4 * i + e] = h[e];
        } else {
          half_of8(code[k][i], p[k][2 * i], p[k][2 * i + 1]);
        }
      }
#pragma unroll
      for (int b = 2; b < NP; b <<= 1) {  // butterflies on every bit of the pair's number but the lowest
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          if (i & b) continue;
          const uint32_t u = p[k][i], w = p[k][i | b];
          p[k][i] = hadd2(u, w);
          p[k][i | b] = hadd2(u, w ^ 0x80008000u);
        }
      }
    }
    if (g + step < 2 * groups) load(g + step, next);  // the next codes
    const bool is_v = g >= groups;
    void* const dst = const_cast<void*>(is_v ? y.v : y.k);
    const float* f = factors[is_v] + c4 * (D / 4 + 4);
#pragma unroll
    for (int e0 = 0; e0 < D / 4; e0 += 16) {  // sixteen elements of both rows
      float z[2][16];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int i = e0 / 2 + 2 * m;  // pairs i, i + 1
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma_f16(d, p[0][i], p[1][i], p[0][i + 1], p[1][i + 1], hm[t][0], hm[t][1]);
          // element of (pair number without its lowest bit, tile, column's low bit)
          const int e = BITS == 4 ? 8 * (m >> 1) + 2 * (m & 1) + 4 * t : 4 * m + 2 * t;
          z[0][e] = d[0], z[0][e + 1] = d[1];
          z[1][e] = d[2], z[1][e + 1] = d[3];
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (!row[k].owned) continue;
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const float4 q = *reinterpret_cast<const float4*>(f + e0 + e);
          float* w = z[k] + e;
          mul_x2(w[0], w[1], s[k], s[k]);
          mul_x2(w[2], w[3], s[k], s[k]);
          mul_x2(w[0], w[1], q.x, q.y);
          mul_x2(w[2], w[3], q.z, q.w);
        }
        const float* w = z[k];
        if (wide) {  // whole 32-byte sectors
          if constexpr (F32) {
            float* o = static_cast<float*>(dst) + row[k].at + e0;
#pragma unroll
            for (int e = 0; e < 16; e += 8)
              st_stream_v8(o + e, __float_as_uint(w[e]), __float_as_uint(w[e + 1]), __float_as_uint(w[e + 2]),
                           __float_as_uint(w[e + 3]), __float_as_uint(w[e + 4]), __float_as_uint(w[e + 5]),
                           __float_as_uint(w[e + 6]), __float_as_uint(w[e + 7]));
          } else {
            st_stream_v8(static_cast<__nv_bfloat16*>(dst) + row[k].at + e0, f32_to_bf16x2(w[0], w[1]),
                         f32_to_bf16x2(w[2], w[3]), f32_to_bf16x2(w[4], w[5]), f32_to_bf16x2(w[6], w[7]),
                         f32_to_bf16x2(w[8], w[9]), f32_to_bf16x2(w[10], w[11]), f32_to_bf16x2(w[12], w[13]),
                         f32_to_bf16x2(w[14], w[15]));
          }
        } else {
          kv_store8<F32>(dst, row[k].at + e0, w);
          kv_store8<F32>(dst, row[k].at + e0 + 8, w + 8);
        }
      }
    }
  }
}

// A call without sequences whose rows are to be zero.
__global__ void __launch_bounds__(kThreads) k_kv_zero(void* out, int64_t tokens, int heads, int row_bytes,
                                                      int64_t token_bytes, int64_t head_bytes) {
  kv_zero_rows(out, 0, 0, tokens, heads, row_bytes, token_bytes, head_bytes,
               int64_t(blockIdx.x) * blockDim.x + threadIdx.x, int64_t(gridDim.x) * blockDim.x);
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
    k_kv_append<D, BITS, F32><<<grid, threads, size_t(tile) * a.n_freq * sizeof(float2), st>>>(a, x, tile, norm_of(D),
                                                                                                 make_fastdiv(2 * a.hk));
    return cudaGetLastError();
  }
};
struct Read {
  const KvArgs& a;
  const KvDense& y;
  bool zero;
  cudaStream_t st;
  template <int D, int BITS, bool F32>
  cudaError_t go() {
    const int tile = pick_tile(a.tokens, kReadCtas, kMaxTile);
    const unsigned grid = unsigned((a.tokens + tile - 1) / tile);
    // a warp for each 16 vectors of either kind, eight at most
    const int64_t groups = 2 * ((int64_t(tile) * a.hk + 15) / 16);
    const int threads = 32 * int(std::min<int64_t>(kThreads / 32, groups));
    const int es = F32 ? 4 : 2;
    const bool wide = (reinterpret_cast<uintptr_t>(y.k) | reinterpret_cast<uintptr_t>(y.v) | uintptr_t(y.k_ts * es) |
                       uintptr_t(y.k_hs * es) | uintptr_t(y.v_ts * es) | uintptr_t(y.v_hs * es)) % 32 == 0;
    k_kv_read<D, BITS, F32><<<grid, threads, 0, st>>>(a, y, tile, norm_of(D), wide, zero, make_fastdiv(a.hk));
    return cudaGetLastError();
  }
};

}  // namespace

cudaError_t launch_kv_append(const KvArgs& a, const KvDense& x, int dt, cudaStream_t st) {
  return by_format(a, dt, Append{a, x, st});
}
cudaError_t launch_kv_read(const KvArgs& a, const KvDense& y, int dt, bool zero, cudaStream_t st) {
  return by_format(a, dt, Read{a, y, zero, st});
}
cudaError_t launch_kv_zero(void* out, int64_t tokens, int heads, int head_dim, int64_t ts, int64_t hs, int dt,
                           cudaStream_t st) {
  const int es = dt == 0 ? 4 : 2;
  const int64_t pieces = tokens * heads * (head_dim * es / 16);
  const unsigned grid = unsigned(std::min<int64_t>(148 * 8, (pieces + kThreads - 1) / kThreads));
  k_kv_zero<<<grid, kThreads, 0, st>>>(out, tokens, heads, head_dim * es, ts * es, hs * es);
  return cudaGetLastError();
}

}  // namespace hit

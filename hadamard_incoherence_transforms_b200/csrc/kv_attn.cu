// Attention of new tokens over the rotated key/value cache.
//
// One CTA per (token, query head): its warps walk the visible keys, a warp a
// key at a time with the head spread over the lanes, each warp with its own
// running maximum and sum; the warps' parts are joined at the end and rotated
// back.
#include "kv.cuh"

namespace hit {
namespace {

constexpr int kWarps = 4;

// In-place unnormalised Hadamard transform of D floats in shared memory.
template <int D>
__device__ __forceinline__ void smem_hadamard(float* x) {
  for (int h = 1; h < D; h *= 2) {
    __syncthreads();
    for (int i = threadIdx.x; i < D / 2; i += blockDim.x) {
      const int p = (i / h) * 2 * h + i % h;
      const float u = x[p], w = x[p + h];
      x[p] = u + w;
      x[p + h] = u - w;
    }
  }
  __syncthreads();
}

template <int D, int BITS>
__global__ void __launch_bounds__(kWarps * 32) k_kv_attn(const KvArgs a, const KvAttn t, float norm) {
  constexpr int E = D / 32;
  constexpr int VB = D * BITS / 8;
  __shared__ KvToken tok;
  __shared__ float2 cs[D / 2];
  __shared__ float raw[D], qv[D], acc[kWarps][D], mx[kWarps], sm[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tt = blockIdx.x / t.heads;
  const int head = blockIdx.x % t.heads, h = head / (t.heads / a.hk);
  if (warp == 0) {
    const KvToken k = kv_token(a, tt, lane);
    if (lane == 0) tok = k;
  }
  __syncthreads();
  if (tok.seq < 0) return;
  const int64_t pos = tok.pos, len = __ldg(a.lens + tok.seq);
  for (int f = threadIdx.x; f < a.n_freq; f += blockDim.x) cs[f] = kv_angle(a, tt, pos, f);
  for (int i = threadIdx.x; i < D; i += blockDim.x) {
    const int64_t at = tt * t.q_ts + head * t.q_hs + i;
    raw[i] = t.q_f32 ? static_cast<const float*>(t.q)[at] : __bfloat162float(static_cast<const __nv_bfloat16*>(t.q)[at]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += blockDim.x) {
    float v = raw[i];
    if (i < 2 * a.n_freq) {
      if (a.interleaved) {
        const float2 c = cs[i / 2];
        v = i & 1 ? raw[i - 1] * c.y + v * c.x : v * c.x - raw[i + 1] * c.y;
      } else {
        const float2 c = cs[i % a.n_freq];
        v = i >= a.n_freq ? raw[i - a.n_freq] * c.y + v * c.x : v * c.x - raw[i + a.n_freq] * c.y;
      }
    }
    if (a.k_signs != nullptr && a.k_signs[i] < 0) v = -v;
    qv[i] = v * (norm * t.scale * 1.4426950408889634f);
  }
  smem_hadamard<D>(qv);
  float q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) q[e] = qv[E * lane + e], o[e] = 0.0f;
  float m = -INFINITY, l = 0.0f;
  int64_t j1 = len, j0 = 0;
  if (t.causal) j1 = min(j1, pos + 1);
  if (t.window > 0) j0 = max(j0, pos - t.window + 1);
  for (int64_t j = j0 + warp; j < j1; j += kWarps) {
    const int64_t slot = kv_slot(a, tok.seq, j);
    if (slot < 0) continue;
    const int64_t vec = slot + (int64_t(h) << a.log_page);
    float kq[E], vq[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = E * lane + e;
      if (BITS == 8) {
        kq[e] = float(int(a.k_codes[vec * VB + i]) - 128);
        vq[e] = float(int(a.v_codes[vec * VB + i]) - 128);
      } else {
        kq[e] = float(int(a.k_codes[vec * VB + i / 2] >> (4 * (i & 1)) & 15) - 8);
        vq[e] = float(int(a.v_codes[vec * VB + i / 2] >> (4 * (i & 1)) & 15) - 8);
      }
    }
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], kq[e], s);
#pragma unroll
    for (int b = 16; b; b >>= 1) s += __shfl_xor_sync(0xffffffffu, s, b);
    s *= a.k_scales[vec];
    const float mn = s > m || s != s ? s : m;
    const float f = m == -INFINITY ? 0.0f : exp2f(m - mn), p = exp2f(s - mn);
    m = mn;
    l = l * f + p;
    const float pv = p * a.v_scales[vec];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(pv, vq[e], o[e] * f);
  }
  if (lane == 0) mx[warp] = m, sm[warp] = l;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[warp][E * lane + e] = o[e];
  __syncthreads();
  float top = -INFINITY;
  bool nan = false;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, mx[w]), nan |= mx[w] != mx[w];
  float total = 0.0f, f[kWarps];
  for (int w = 0; w < kWarps; ++w) {
    f[w] = mx[w] == -INFINITY ? 0.0f : exp2f(mx[w] - top);
    total += f[w] * sm[w];
  }
  const float inv = nan ? NAN : total > 0.0f ? norm / total : total != total ? NAN : 0.0f;
  for (int i = threadIdx.x; i < D; i += blockDim.x) {
    float v = 0.0f;
    for (int w = 0; w < kWarps; ++w) v = f[w] == 0.0f ? v : fmaf(f[w], acc[w][i], v);
    qv[i] = v * inv;
  }
  smem_hadamard<D>(qv);
  for (int i = threadIdx.x; i < D; i += blockDim.x) {
    const float v = a.v_signs != nullptr && a.v_signs[i] < 0 ? -qv[i] : qv[i];
    const int64_t at = tt * t.o_ts + head * t.o_hs + i;
    if (t.o_f32) static_cast<float*>(t.out)[at] = v;
    else static_cast<__nv_bfloat16*>(t.out)[at] = __float2bfloat16_rn(v);
  }
}

template <int D, int BITS>
cudaError_t go(const KvArgs& a, const KvAttn& t, cudaStream_t st) {
  const float norm = D == 64 ? 0.125f : D == 256 ? 0.0625f : 0.08838834764831845f;
  k_kv_attn<D, BITS><<<unsigned(a.tokens * t.heads), kWarps * 32, 0, st>>>(a, t, norm);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_attention(const KvArgs& a, const KvAttn& t, cudaStream_t st) {
  if (a.head_dim == 64) return a.bits == 4 ? go<64, 4>(a, t, st) : go<64, 8>(a, t, st);
  if (a.head_dim == 128) return a.bits == 4 ? go<128, 4>(a, t, st) : go<128, 8>(a, t, st);
  return a.bits == 4 ? go<256, 4>(a, t, st) : go<256, 8>(a, t, st);
}

}  // namespace hit

// Attention over the rotated cache as a list of equal units of work, split
// evenly over the CTAs of a grid wherever sequences begin and end, and the
// joining of the parts (shared by the attention kernels).
//
// A pair is one (sequence, key/value head, tile of query rows); query rows of
// a sequence and key/value head are numbered token * G + (head within the
// group).  A unit is TK consecutive positions of a pair's keys.  All pairs of a
// sequence have the same number of units, so the list needs only one number
// per sequence, and every CTA finds its own part of it from cu and lens.
#pragma once
#include "kv.cuh"

namespace hit {

struct KvSeq {
  int64_t t0;       // first token of the call
  int n;            // tokens
  int64_t pos0;     // position of the first token
  int64_t hi;       // positions that can exist: [0, hi)
  int64_t unit0;    // first unit any row sees
  int64_t units;    // units of a pair: `lead` empty ones, then those of its keys (at least
                    // one, so that every row is written)
  int row_tiles;
};

// ROWS query rows to a tile, TK positions to a unit, LEAD empty units ahead of a
// pair's: what beginning a pair costs, so that CTAs with many short pairs get
// fewer positions.
template <int ROWS, int TK, int LEAD>
__device__ __forceinline__ KvSeq kv_seq(const KvArgs& a, const KvAttn& t, int s) {
  KvSeq q;
  const int64_t b = __ldg(a.cu + s), e = __ldg(a.cu + s + 1), len = __ldg(a.lens + s);
  q.t0 = b;
  const int64_t n = min(e, a.tokens) - b;
  q.n = b < 0 || n < 0 ? 0 : int(n);
  q.pos0 = len - (e - b);
  q.hi = max(int64_t(0), min(len, int64_t(a.max_pages) << a.log_page));
  int64_t lo = 0;
  if (t.window > 0) lo = min(q.hi, max(int64_t(0), q.pos0 - t.window + 1));
  q.unit0 = lo / TK;
  q.units = LEAD + max(int64_t(1), (q.hi + TK - 1) / TK - q.unit0);
  const int64_t rows = int64_t(q.n) * t.group;
  q.row_tiles = int((rows + ROWS - 1) / ROWS);
  return q;
}
// Whether a sequence belongs to this launch (KvAttn::rows_lo, rows_hi).
__device__ __forceinline__ bool kv_mine(const KvAttn& t, const KvSeq& q) {
  const int64_t rows = int64_t(q.n) * t.group;
  return rows >= t.rows_lo && rows <= t.rows_hi;
}
__device__ __forceinline__ int64_t kv_work(const KvArgs& a, const KvAttn& t, const KvSeq& q) {
  return kv_mine(t, q) ? int64_t(a.hk) * q.row_tiles * q.units : 0;
}

// The CTA's part [u0, u1) of the list, and where it begins.
struct KvPlan {
  int64_t total;    // units in the list
  int64_t u0, u1;
  int seq;          // sequence that holds unit u0
  int64_t base;     // first unit of that sequence
  int ctas;         // CTAs that have work
};

// All `THREADS` threads of the CTA.  least: units that a CTA has at least.
template <int ROWS, int TK, int LEAD, int THREADS>
__device__ __forceinline__ KvPlan kv_plan(const KvArgs& a, const KvAttn& t, int least) {
  __shared__ int64_t sums[THREADS / 32];
  __shared__ int64_t found_base;
  __shared__ int found_seq;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  KvPlan p;
  int64_t mine = 0;
  for (int s = threadIdx.x; s < a.seqs; s += THREADS) mine += kv_work(a, t, kv_seq<ROWS, TK, LEAD>(a, t, s));
  int64_t w = mine;
#pragma unroll
  for (int b = 16; b; b >>= 1) w += __shfl_xor_sync(0xffffffffu, w, b);
  if (lane == 0) sums[warp] = w;
  __syncthreads();
  p.total = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) p.total += sums[i];
  __syncthreads();
  p.ctas = int(max(int64_t(1), min(int64_t(gridDim.x), (p.total + least - 1) / least)));
  const int64_t c = blockIdx.x;
  p.u0 = c < p.ctas ? c * p.total / p.ctas : p.total;
  p.u1 = c < p.ctas ? (c + 1) * p.total / p.ctas : p.total;
  if (threadIdx.x == 0) found_seq = a.seqs, found_base = p.total;
  int64_t before = 0;
  for (int s0 = 0; s0 < a.seqs; s0 += THREADS) {
    const int s = s0 + int(threadIdx.x);
    const int64_t v = a.seqs <= THREADS ? mine : s < a.seqs ? kv_work(a, t, kv_seq<ROWS, TK, LEAD>(a, t, s)) : 0;
    int64_t x = v;
#pragma unroll
    for (int b = 1; b < 32; b <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, b);
      if (lane >= b) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int64_t ahead = before, all = before;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i < warp) ahead += sums[i];
      all += sums[i];
    }
    const int64_t first = ahead + x - v;
    if (v > 0 && first <= p.u0 && p.u0 < first + v) found_seq = s, found_base = first;
    before = all;
    __syncthreads();
    if (before > p.u0) break;
  }
  __syncthreads();
  p.seq = found_seq;
  p.base = found_base;
  return p;
}

// CTA that holds unit u of a list of `total` units over `ctas` CTAs.
__device__ __forceinline__ int kv_cta_of(int64_t u, int64_t total, int ctas) { return int(((u + 1) * ctas - 1) / total); }

// What a CTA left unfinished: slot 2 c holds the end (or middle) of a pair that
// began in an earlier CTA, slot 2 c + 1 the beginning of one that goes on.
struct KvPart {
  int first, last;  // CTAs of the pair; first = -1: nothing here
  int rows;         // query rows of the tile
  int row0;         // first of them (token * G + g)
  int64_t t0;       // first token of the sequence
  int h;            // key/value head
  int pad;
};

// Workspace: KvPart of every slot, then (max, sum) of every row, then the rows.
struct KvWork {
  KvPart* part;
  float2* ms;
  float* rows;
};
template <int D, int ROWS>
__host__ __device__ __forceinline__ KvWork kv_work_of(void* ws, int ctas) {
  KvWork w;
  uint8_t* p = static_cast<uint8_t*>(ws);
  w.part = reinterpret_cast<KvPart*>(p);
  p += size_t(ctas) * 2 * sizeof(KvPart);
  w.ms = reinterpret_cast<float2*>(p);
  p += size_t(ctas) * 2 * ROWS * sizeof(float2);
  w.rows = reinterpret_cast<float*>(p);
  return w;
}
template <int D, int ROWS>
constexpr size_t kv_work_bytes(int ctas) {
  return size_t(ctas) * 2 * (sizeof(KvPart) + ROWS * (sizeof(float2) + D * sizeof(float)));
}
static_assert(sizeof(KvPart) == 32, "parts keep the rows 16-byte aligned");

// A finished row (the sum of its values over the sum of its probabilities, still
// rotated): lane holds elements (D / 32) lane ...  Rotates back and stores.
template <int D>
__device__ __forceinline__ void kv_finish(float (&x)[D / 32], const KvArgs& a, const KvAttn& t, int64_t token, int head,
                                          int lane) {
  constexpr int E = D / 32;
  constexpr int LOGE = E == 2 ? 1 : E == 4 ? 2 : 3;
  const float norm = D == 64 ? 0.125f : D == 256 ? 0.0625f : 0.08838834764831845f;
  reg_stages<E, 0, LOGE>(x);
#pragma unroll
  for (int b = 0; b < 5; ++b) shfl_stage<E>(x, b, (lane >> b) & 1);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    x[e] *= norm;
    if (a.v_signs != nullptr && __ldg(a.v_signs + E * lane + e) < 0) x[e] = -x[e];
  }
  const int64_t at = token * t.o_ts + head * t.o_hs + E * lane;
  if (t.o_f32) {
    float* o = static_cast<float*>(t.out) + at;
    if constexpr (E == 2) {
      *reinterpret_cast<float2*>(o) = make_float2(x[0], x[1]);
    } else {
#pragma unroll
      for (int e = 0; e < E; e += 4) *reinterpret_cast<float4*>(o + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
    }
  } else {
    uint32_t w[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) w[e / 2] = f32_to_bf16x2(x[e], x[e + 1]);
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(t.out) + at;
    if constexpr (E == 2) *reinterpret_cast<uint32_t*>(o) = w[0];
    if constexpr (E == 4) *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
    if constexpr (E == 8) *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Square root of the weight of a part with reference m below the joint one, top (base 2); a NaN
// reference or sum stays NaN.  Taken twice, so that a part's sum outlives a weight below
// 2^-126: references follow the values' sizes too.
__device__ __forceinline__ float kv_weight(float m, float top) { return m == -INFINITY ? 0.0f : exp2f(0.5f * (m - top)); }

// Joins the parts of the pairs that several CTAs share: block c handles the
// pair that CTA c began and did not end (slot 2 c + 1), rows PER y ... of it.  A
// row's parts are dealt to the warps left over by the number of rows.
constexpr int kJoinWarps = 4;
template <int D, int ROWS, int PER>
__global__ void __launch_bounds__(kJoinWarps * 32) k_kv_join(const KvArgs a, const KvAttn t, int ctas) {
  constexpr int E = D / 32;
  __shared__ float sx[kJoinWarps][D];
  __shared__ float sm[kJoinWarps], sl[kJoinWarps];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const KvWork w = kv_work_of<D, ROWS>(t.ws, ctas);
  const int c = blockIdx.x, first_row = blockIdx.y * PER;
  const KvPart p = w.part[2 * c + 1];
  if (t.zero) {
    const int es = t.o_f32 ? 4 : 2;
    kv_zero_rows(t.out, __ldg(a.cu), __ldg(a.cu + a.seqs), a.tokens, t.heads, D * es, t.o_ts * es, t.o_hs * es,
                 (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x,
                 int64_t(gridDim.x) * gridDim.y * blockDim.x);
  }
  if (p.first < 0 || first_row >= p.rows) return;
  const int rows = min(PER, p.rows - first_row);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int per = 1;  // rows handled at once, a power of two
  while (per < kJoinWarps && per < rows) per *= 2;
  const int teams = kJoinWarps / per, team = warp / per;
  const int parts = p.last - p.first + 1;
  for (int r0 = 0; r0 < rows; r0 += per) {
    const int in = r0 + warp % per, r = first_row + in;
    float m = -INFINITY, l = 0.0f, x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = 0.0f;
    if (in < rows) {
      // this team's parts are team + j teams; their (max, sum) first, a lane a part,
      // then the rows, whose loads wait for nothing
      const int count = (parts - team + teams - 1) / teams;
      auto place = [&](int j) {
        const int i = team + j * teams;
        return size_t(i == 0 ? 2 * c + 1 : 2 * (c + i)) * ROWS + r;
      };
      for (int j = lane; j < count; j += 32) m = kv_max(m, w.ms[place(j)].x);
#pragma unroll
      for (int b = 16; b; b >>= 1) m = kv_max(m, __shfl_xor_sync(0xffffffffu, m, b));
      for (int j0 = 0; j0 < count; j0 += 32) {
        const float2 q = j0 + lane < count ? w.ms[place(j0 + lane)] : make_float2(-INFINITY, 0.0f);
        const float mine = kv_weight(q.x, m);
        l = fmaf(q.y * mine, mine, l);
        const int n = min(32, count - j0);
#pragma unroll 8
        for (int j = 0; j < n; ++j) {
          const float half = __shfl_sync(0xffffffffu, mine, j), f = half * half;
          const float* src = w.rows + place(j0 + j) * D + E * lane;
          float v[E];
          if constexpr (E == 2) {
            const float2 u = __ldcs(reinterpret_cast<const float2*>(src));
            v[0] = u.x, v[1] = u.y;
          } else {
#pragma unroll
            for (int e = 0; e < E; e += 4) {
              const float4 u = __ldcs(reinterpret_cast<const float4*>(src + e));
              v[e] = u.x, v[e + 1] = u.y, v[e + 2] = u.z, v[e + 3] = u.w;
            }
          }
#pragma unroll
          for (int e = 0; e < E; ++e) x[e] = fmaf(f, v[e], x[e]);
        }
      }
#pragma unroll
      for (int b = 16; b; b >>= 1) l += __shfl_xor_sync(0xffffffffu, l, b);
    }
    if (teams > 1) {
#pragma unroll
      for (int e = 0; e < E; ++e) sx[warp][E * lane + e] = x[e];
      if (lane == 0) sm[warp] = m, sl[warp] = l;
      __syncthreads();
      if (team == 0) {
        float top = m;
        for (int i = 1; i < teams; ++i) top = kv_max(top, sm[warp + i * per]);
        const float half0 = kv_weight(m, top), f0 = half0 * half0;
        l = l * half0 * half0;
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] *= f0;
        for (int i = 1; i < teams; ++i) {
          const float half = kv_weight(sm[warp + i * per], top), f = half * half;
          l = fmaf(sl[warp + i * per] * half, half, l);
#pragma unroll
          for (int e = 0; e < E; ++e) x[e] = fmaf(f, sx[warp + i * per][E * lane + e], x[e]);
        }
      }
      __syncthreads();
    }
    if (team == 0 && in < rows) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] *= inv;
      const int row = p.row0 + r;
      kv_finish<D>(x, a, t, p.t0 + row / t.group, p.h * t.group + row % t.group, lane);
    }
  }
}

template <int D, int ROWS, int PER>
cudaError_t launch_kv_join(const KvArgs& a, const KvAttn& t, int ctas, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(ctas), (ROWS + PER - 1) / PER);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_kv_join<D, ROWS, PER>, a, t, ctas);
}

}  // namespace hit

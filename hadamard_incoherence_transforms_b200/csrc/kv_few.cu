// Attention over the rotated cache for few query rows (single tokens, drafted
// tokens): bound by reading the codes once.
//
// A CTA of four warps takes an equal share of the list of units (kv_split.cuh);
// each warp streams its units through a private ring of shared-memory stages
// with 16-byte asynchronous copies, so that the warps never wait for one
// another inside a pair.  Scores are computed transposed, S^T = K Q^T: the 16
// rows of m16n8k16 are positions and the 8 columns query rows, so eight query
// heads of one key head cost one instruction.  The order of the head's
// elements is free inside a product; it is chosen such that a lane's operands
// are the codes of one 16-byte piece, unpacked in registers:
//   K to fp16: a code under the exponent of 1024 (one logic operation), minus
//     the offset -- exact; the query is scaled to [-2, 2) by a power of two of
//     its own row, so that fp16 holds it to 2^-11 whatever its size;
//   V to bf16, as the other operand (probability times the value's scale)
//     spans more than fp16's range.
// O^T += V^T P^T takes P^T from the score accumulators with one 8x8 transpose
// per 8 positions.  Scales never touch the codes: the key's multiplies its
// score, the value's its probability.
#include "kv_codes.cuh"
#include "kv_split.cuh"

#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

namespace hit {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 3;

// Positions of a unit: stages of about 4 KB (8 KB for heads of 256), which is
// 16 warps x 2 stages = 140 KB in flight on an SM.
template <int D, int BITS>
struct Few {
  static constexpr int VB = D * BITS / 8;  // bytes of a vector's codes
  static constexpr int CH = VB / 16;
  static constexpr int TK = VB == 32 ? 64 : VB == 64 ? 32 : VB == 128 ? (D == 256 ? 32 : 16) : 16;
  static constexpr int MT = TK / 16;
  static constexpr int STAGE = TK * (2 * VB + 8) + 16;
  static constexpr int KS = D / 16;
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_b16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t p) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(p));
  return r;
}
__device__ __forceinline__ void lds64(uint32_t p, uint32_t* r) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(p));
}
__device__ __forceinline__ void lds128(uint32_t p, uint32_t* r) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(p));
}

// Places of 16-byte piece q of position t in a stage.  Score rows r and r + 1
// are positions that differ in bit 2 (position = r / 2 + 4 (r % 2)), output
// columns c are positions c, c + 4, ...; the pieces are moved such that the
// lanes of one shared-memory read touch every bank once.
template <int CH>
__device__ __forceinline__ int k_place(int t, int q) {
  if constexpr (CH == 2) return ((t & ~6) | ((t & 2) << 1) | ((t & 4) >> 1)) * CH + q;
  if constexpr (CH == 4) return (t ^ ((t >> 2) & 1)) * CH + q;
  return t * CH + (q ^ (t & 4));
}
template <int CH>
__device__ __forceinline__ int v_place(int t, int q) {
  if constexpr (CH == 2) return t * CH + q;
  if constexpr (CH == 4) return t * CH + (q ^ (t & 2));
  if constexpr (CH == 8) return t * CH + (q ^ (2 * (t & 3)));
  return t * CH + (q ^ ((t & 1) | ((t & 2) << 1)));
}

template <int D, int BITS, int NT, int MINB>
__global__ void __launch_bounds__(kThreads, MINB) k_kv_few(const KvArgs a, const KvAttn t) {
  using F = Few<D, BITS>;
  constexpr int ROWS = 8 * NT, TK = F::TK, MT = F::MT, CH = F::CH, VB = F::VB, KS = F::KS;
  constexpr int OM = D / 16;   // 16-element tiles of the output's head dimension
  constexpr int QP = D + 8;    // padded row of the query in shared memory
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t turns[D / 2];
  kv_turns(a, turns, threadIdx.x, kThreads);  // kv_plan's barriers follow
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r8 = lane >> 2, c4 = lane & 3;
  const KvPlan plan = kv_plan<ROWS, TK, kThreads>(a, t, kWarps);
  const KvWork work = kv_work_of<D, ROWS>(t.ws, gridDim.x);
  KvPart open;
  open.first = -1;

  int s = plan.seq;
  int64_t base = plan.base;
  KvSeq q{};
  if (s < a.seqs) q = kv_seq<ROWS, TK>(a, t, s);
  for (int64_t u = plan.u0; u < plan.u1;) {
    const int64_t rel = u - base;
    const int64_t pair = rel / q.units;
    const int64_t x0 = rel - pair * q.units;
    const int64_t x1 = min(q.units, x0 + plan.u1 - u);
    const int h = int(pair / q.row_tiles), rt = int(pair - int64_t(h) * q.row_tiles);
    const int row0 = rt * ROWS;
    const int nr = int(min(int64_t(ROWS), int64_t(q.n) * t.group - row0));
    const int i0 = row0 / t.group, i1 = (row0 + nr - 1) / t.group;  // first and last token of the tile
    // what the tile's rows see, first and last
    const int64_t hi_min = t.causal ? min(q.hi, q.pos0 + i0 + 1) : q.hi;
    const int64_t hi_max = t.causal ? min(q.hi, q.pos0 + i1 + 1) : q.hi;
    const int64_t lo_min = t.window > 0 ? max(int64_t(0), q.pos0 + i0 - t.window + 1) : 0;
    const int64_t lo_max = t.window > 0 ? max(int64_t(0), q.pos0 + i1 - t.window + 1) : 0;
    const int64_t b0 = max(x0, lo_min / TK - q.unit0);
    const int64_t b1 = min(x1, (hi_max + TK - 1) / TK - q.unit0);
    const int nu = b0 + warp < b1 ? int((b1 - b0 - warp + kWarps - 1) / kWarps) : 0;

    // Unit i of this warp into its stage i % kStages.
    auto issue = [&](int i) {
      if (i < nu) {
        const uint32_t st = smem_u32(smem) + uint32_t(((i % kStages) * kWarps + warp) * F::STAGE);
        const int64_t p0 = (q.unit0 + b0 + warp + int64_t(kWarps) * i) * TK;
        int64_t at[(TK + 31) / 32];
        uint64_t there = 0;
#pragma unroll
        for (int k = 0; k < (TK + 31) / 32; ++k) {
          const int64_t p = p0 + lane + 32 * k;
          at[k] = lane + 32 * k < TK && p < q.hi ? kv_slot(a, s, p) : -1;
          there |= uint64_t(__ballot_sync(0xffffffffu, at[k] >= 0)) << (32 * k);
          const bool in = at[k] >= 0;
          at[k] = in ? at[k] + (int64_t(h) << a.log_page) : 0;
          if (lane + 32 * k < TK) {
            copy4(st + 2 * TK * VB + 4 * (lane + 32 * k), a.k_scales + at[k], in);
            copy4(st + 2 * TK * VB + 4 * (TK + lane + 32 * k), a.v_scales + at[k], in);
          }
        }
#pragma unroll
        for (int k = 0; k < TK * CH / 32; ++k) {
          const int tk = (32 * k) / CH + lane / CH, piece = lane % CH;
          const int64_t vec = __shfl_sync(0xffffffffu, at[(32 * k) / CH / 32], tk & 31);
          const bool in = (there >> tk) & 1;
          copy16(st + 16 * k_place<CH>(tk, piece), a.k_codes + vec * VB + 16 * piece, in);
          copy16(st + TK * VB + 16 * v_place<CH>(tk, piece), a.v_codes + vec * VB + 16 * piece, in);
        }
        if (lane == 0) {
          *reinterpret_cast<uint64_t*>(smem + ((i % kStages) * kWarps + warp) * F::STAGE + TK * (2 * VB + 8)) = there;
        }
      }
      copies_commit();
    };
    issue(0);

    // The tile's queries: turned, rotated, scaled (into base-2 scores), and
    // brought to [-2, 2) by a power of two; scratch in the stages behind the first.
    uint32_t qf[KS][NT][2];
    float qe[NT][2];
    int lo[NT][2], hi[NT][2];
    {
      uint8_t* scratch = smem + kWarps * F::STAGE;
      float2* cs = reinterpret_cast<float2*>(scratch);
      __half* qs = reinterpret_cast<__half*>(scratch + sizeof(float2) * ROWS * (D / 2));
      float* es = reinterpret_cast<float*>(qs + ROWS * QP);
      static_assert(sizeof(float2) * ROWS * (D / 2) + 2 * ROWS * QP + 4 * ROWS <= 2 * kWarps * F::STAGE, "scratch");
      for (int i = threadIdx.x; i < (i1 - i0 + 1) * a.n_freq; i += kThreads) {
        const int j = i / a.n_freq;
        cs[i] = kv_angle_fast(a, turns, q.t0 + i0 + j, int(q.pos0) + i0 + j, i - j * a.n_freq);
      }
      __syncthreads();
      constexpr int LPV = KvLanes<D>::LPV;
      const int l = threadIdx.x % LPV;
      for (int r0 = 0; r0 < ROWS; r0 += kThreads / LPV) {
        const int r = r0 + int(threadIdx.x) / LPV;
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = 0.0f;
        if (r < nr) {
          const int row = row0 + r, tok = row / t.group;
          const int64_t src = (q.t0 + tok) * t.q_ts + (int64_t(h) * t.group + row - tok * t.group) * t.q_hs;
          if (t.q_f32) {
#pragma unroll
            for (int c = 0; c < 4; ++c) kv_load8<true>(t.q, src + 8 * (c * LPV + l), x + 8 * c);
            if (a.n_freq > 0) kv_rope<D, true>(x, t.q, src, cs + (tok - i0) * a.n_freq, a.n_freq, a.interleaved, l);
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) kv_load8<false>(t.q, src + 8 * (c * LPV + l), x + 8 * c);
            if (a.n_freq > 0) kv_rope<D, false>(x, t.q, src, cs + (tok - i0) * a.n_freq, a.n_freq, a.interleaved, l);
          }
          kv_signs<D>(x, a.k_signs, l);
        }
        kv_hadamard<D>(x, l);
        float up, down;
        kv_query_scale<D>(x, t.scale, up, down);
        if (r < ROWS) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __half2 p = __floats2half2_rn(x[8 * c + 2 * e] * down, x[8 * c + 2 * e + 1] * down);
              w[e] = *reinterpret_cast<const uint32_t*>(&p);
            }
            *reinterpret_cast<uint4*>(qs + r * QP + 8 * (c * LPV + l)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          if (l == 0) es[r] = up;
        }
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint16_t* row = reinterpret_cast<const uint16_t*>(qs + (8 * n + r8) * QP);
        auto two = [&](int i, int j) { return uint32_t(row[i]) | (uint32_t(row[j]) << 16); };
#pragma unroll
        for (int w = 0; w < VB / 16; ++w) {  // the lane's words of a vector's codes
          const int byte = CH == 2 ? 8 * c4 + 4 * w : 16 * (4 * (w / 4) + c4) + 4 * (w % 4);
          if constexpr (BITS == 4) {
            const int d = 2 * byte;
            qf[2 * w][n][0] = two(d, d + 4);
            qf[2 * w][n][1] = two(d + 1, d + 5);
            qf[2 * w + 1][n][0] = two(d + 2, d + 6);
            qf[2 * w + 1][n][1] = two(d + 3, d + 7);
          } else {
            qf[w][n][0] = two(byte, byte + 1);
            qf[w][n][1] = two(byte + 2, byte + 3);
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int r = 8 * n + 2 * c4 + k;
          qe[n][k] = es[r];
          const int64_t pos = q.pos0 + (row0 + r) / t.group;
          hi[n][k] = r < nr ? int(max(int64_t(0), t.causal ? min(q.hi, pos + 1) : q.hi)) : 0;
          lo[n][k] = t.window > 0 ? int(max(int64_t(0), min(q.hi, pos - t.window + 1))) : 0;
        }
      }
      __syncthreads();
    }

    float o[OM][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < OM; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.0f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
    }
    issue(1);
    for (int i = 0; i < nu; ++i) {
      issue(i + 2);
      copies_wait<2>();
      __syncwarp();
      uint8_t* stp = smem + ((i % kStages) * kWarps + warp) * F::STAGE;
      const uint32_t st = smem_u32(stp);
      const uint64_t there = *reinterpret_cast<const uint64_t*>(stp + TK * (2 * VB + 8));
      const float* ks = reinterpret_cast<const float*>(stp + 2 * TK * VB);
      const float* vs = ks + TK;
      const int64_t p0 = (q.unit0 + b0 + warp + int64_t(kWarps) * i) * TK;
      const bool full = p0 >= lo_max && p0 + TK <= hi_min && there == (TK == 64 ? ~uint64_t(0) : (uint64_t(1) << (TK & 63)) - 1);
      const int own = (r8 >> 1) + 4 * (r8 & 1);  // position of score row r8 within its 16

      float sc[MT][NT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int n = 0; n < NT; ++n) sc[mt][n][0] = sc[mt][n][1] = sc[mt][n][2] = sc[mt][n][3] = 0.0f;
        const int tk = 16 * mt + own;
#pragma unroll
        for (int j = 0; j < (CH == 2 ? 1 : CH / 4); ++j) {
          uint32_t wa[4], wb[4];
          constexpr int NW = CH == 2 ? 2 : 4;
          if constexpr (CH == 2) {
            lds64(st + 16 * k_place<CH>(tk, 0) + 8 * c4, wa);
            lds64(st + 16 * k_place<CH>(tk + 8, 0) + 8 * c4, wb);
          } else {
            lds128(st + 16 * k_place<CH>(tk, 4 * j + c4), wa);
            lds128(st + 16 * k_place<CH>(tk + 8, 4 * j + c4), wb);
          }
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            if constexpr (BITS == 4) {
              uint32_t ha[4], hb[4];
              half_of4(wa[w], ha);
              half_of4(wb[w], hb);
              const int k = 2 * (4 * j + w);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                mma_f16(sc[mt][n], ha[0], hb[0], ha[1], hb[1], qf[k][n][0], qf[k][n][1]);
                mma_f16(sc[mt][n], ha[2], hb[2], ha[3], hb[3], qf[k + 1][n][0], qf[k + 1][n][1]);
              }
            } else {
              uint32_t a0, a2, b0_, b2_;
              half_of8(wa[w], a0, a2);
              half_of8(wb[w], b0_, b2_);
              const int k = 4 * j + w;
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_f16(sc[mt][n], a0, b0_, a2, b2_, qf[k][n][0], qf[k][n][1]);
            }
          }
        }
        const float k0 = ks[tk], k1 = ks[tk + 8];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sc[mt][n][e] *= (e < 2 ? k0 : k1) * qe[n][e & 1];
            if (!full) {
              const int w = tk + (e < 2 ? 0 : 8);
              const int64_t p = p0 + w;
              if (!((there >> w) & 1) || p < lo[n][e & 1] || p >= hi[n][e & 1]) sc[mt][n][e] = -INFINITY;
            }
          }
        }
      }

      // running maximum and sum of each column
      bool moved = false;
      float f[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float v = m[n][k];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) v = fmaxf(v, fmaxf(sc[mt][n][k], sc[mt][n][k + 2]));
#pragma unroll
          for (int b = 4; b < 32; b <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, b));
          moved |= v > m[n][k];
          const float top = v == -INFINITY ? 0.0f : v;
          f[n][k] = exp2f(m[n][k] - top);
          m[n][k] = v;
          float sum = 0.0f;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int e = k; e < 4; e += 2) {
              const bool hidden = !full && sc[mt][n][e] == -INFINITY;
              const float p = exp2f(sc[mt][n][e] - top);
              sum += p;
              const float v_scale = vs[16 * mt + own + (e < 2 ? 0 : 8)];
              sc[mt][n][e] = hidden ? 0.0f : p * v_scale;
            }
          }
          l[n][k] = l[n][k] * f[n][k] + sum;
        }
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int d = 0; d < OM; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][n][e] *= f[n][e & 1];
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        uint32_t pb[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          pb[n][0] = transpose8x8(f32_to_bf16x2(sc[mt][n][0], sc[mt][n][1]));
          pb[n][1] = transpose8x8(f32_to_bf16x2(sc[mt][n][2], sc[mt][n][3]));
        }
        // the lane's D / 8 elements of four positions
        constexpr int NW = VB / 32;
        uint32_t v[4][NW];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int tk = 16 * mt + c4 + 4 * g;
          const uint32_t vb = st + TK * VB;
          if constexpr (NW == 1) v[g][0] = lds32(vb + 16 * v_place<CH>(tk, r8 >> 2) + 4 * (r8 & 3));
          if constexpr (NW == 2) lds64(vb + 16 * v_place<CH>(tk, r8 >> 1) + 8 * (r8 & 1), v[g]);
          if constexpr (NW == 4) lds128(vb + 16 * v_place<CH>(tk, r8), v[g]);
          if constexpr (NW == 8) {
            lds128(vb + 16 * v_place<CH>(tk, 2 * r8), v[g]);
            lds128(vb + 16 * v_place<CH>(tk, 2 * r8 + 1), v[g] + 4);
          }
        }
#pragma unroll
        for (int w = 0; w < NW; ++w) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t ab = __byte_perm(v[0][w], v[1][w], half ? 0x7632 : 0x5410);
            const uint32_t cd = __byte_perm(v[2][w], v[3][w], half ? 0x7632 : 0x5410);
            if constexpr (BITS == 4) {
              uint32_t x[4], y[4];
              bf_of4(ab, x);
              bf_of4(cd, y);
              const int d = 4 * w + 2 * half;
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                mma_b16(o[d][n], x[0], x[1], y[0], y[1], pb[n][0], pb[n][1]);
                mma_b16(o[d + 1][n], x[2], x[3], y[2], y[3], pb[n][0], pb[n][1]);
              }
            } else {
              uint32_t x0, x1_, y0, y1;
              bf_of8(ab, x0, x1_);
              bf_of8(cd, y0, y1);
              const int d = 2 * w + half;
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_b16(o[d][n], x0, x1_, y0, y1, pb[n][0], pb[n][1]);
            }
          }
        }
      }
      __syncwarp();
    }
    copies_wait<0>();
    __syncthreads();

    // join the warps; shared memory is free now
    float* mo = reinterpret_cast<float*>(smem);                       // [kWarps][ROWS][D]
    float2* ms = reinterpret_cast<float2*>(mo + kWarps * ROWS * D);   // [kWarps][ROWS]
    static_assert(kWarps * ROWS * (D * 4 + 8) <= kStages * kWarps * F::STAGE, "join buffer");
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int b = 4; b < 32; b <<= 1) l[n][k] += __shfl_xor_sync(0xffffffffu, l[n][k], b);
        const int r = 8 * n + 2 * c4 + k;
        if (r8 == 0) ms[warp * ROWS + r] = make_float2(m[n][k], l[n][k]);
        float* dst = mo + (warp * ROWS + r) * D + r8 * (D / 8);
#pragma unroll
        for (int i = 0; i < OM; i += 2)
          *reinterpret_cast<float4*>(dst + 2 * i) =
              make_float4(o[i][n][k], o[i][n][k + 2], o[i + 1][n][k], o[i + 1][n][k + 2]);
      }
    }
    __syncthreads();
    const bool whole = x0 == 0 && x1 == q.units;
    const size_t slot = x0 == 0 ? 2 * blockIdx.x + 1 : 2 * blockIdx.x;
    constexpr int E = D / 32;
    for (int r = warp; r < nr; r += kWarps) {
      float top = ms[r].x;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = kv_max(top, ms[w * ROWS + r].x);
      float sum = 0.0f, x[E];
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 v = ms[w * ROWS + r];
        const float g = kv_weight(v.x, top);
        sum = fmaf(g, v.y, sum);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = fmaf(g, mo[(w * ROWS + r) * D + E * lane + e], x[e]);
      }
      if (whole) {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] *= inv;
        const int row = row0 + r;
        kv_finish<D>(x, a, t, q.t0 + row / t.group, h * t.group + row % t.group, lane);
      } else {
        float* dst = work.rows + (slot * ROWS + r) * D + E * lane;
#pragma unroll
        for (int e = 0; e < E; e += 2) *reinterpret_cast<float2*>(dst + e) = make_float2(x[e], x[e + 1]);
        if (lane == 0) work.ms[slot * ROWS + r] = make_float2(top, sum);
      }
    }
    if (!whole && x0 == 0) {
      open.first = blockIdx.x;
      open.last = kv_cta_of(base + (pair + 1) * q.units - 1, plan.total, plan.ctas);
      open.rows = nr;
      open.row0 = row0;
      open.t0 = q.t0;
      open.h = h;
      open.pad = 0;
    }
    __syncthreads();
    u += x1 - x0;
    if (u < plan.u1 && u >= base + kv_work(a, t, q)) {
      base += kv_work(a, t, q);
      do {
        q = kv_seq<ROWS, TK>(a, t, ++s);
      } while (kv_work(a, t, q) == 0);
    }
  }
  if (threadIdx.x == 0) work.part[2 * blockIdx.x + 1] = open;
}

template <int D, int BITS, int NT>
cudaError_t go(const KvArgs& a, const KvAttn& t, cudaStream_t st) {
  constexpr int MINB = D <= 128 && NT == 1 ? 4 : 2;
  constexpr int bytes = kStages * kWarps * Few<D, BITS>::STAGE;
  auto* kernel = k_kv_few<D, BITS, NT, MINB>;
  static std::atomic<uint64_t> ready{0};  // devices on which the kernel may use its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (!(ready.load() & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit);
  }
  constexpr int ctas = 148 * MINB;
  kernel<<<ctas, kThreads, bytes, st>>>(a, t);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_kv_join<D, 8 * NT, 8 * NT>(a, t, ctas, st);
}

}  // namespace

size_t kv_few_bytes(int head_dim) {
  if (head_dim == 64) return std::max(kv_work_bytes<64, 8>(592), kv_work_bytes<64, 16>(296));
  if (head_dim == 128) return std::max(kv_work_bytes<128, 8>(592), kv_work_bytes<128, 16>(296));
  return kv_work_bytes<256, 8>(296);
}

cudaError_t launch_kv_few(const KvArgs& a, const KvAttn& t, cudaStream_t st) {
  // Eight query rows to a tile while no sequence has more; else sixteen, which
  // reads the codes half as often (heads of 256 keep eight: the accumulators of
  // sixteen rows do not fit the registers).
  const bool wide = t.max_new * t.group > 8;
  if (a.head_dim == 64) {
    if (a.bits == 4) return wide ? go<64, 4, 2>(a, t, st) : go<64, 4, 1>(a, t, st);
    return wide ? go<64, 8, 2>(a, t, st) : go<64, 8, 1>(a, t, st);
  }
  if (a.head_dim == 128) {
    if (a.bits == 4) return wide ? go<128, 4, 2>(a, t, st) : go<128, 4, 1>(a, t, st);
    return wide ? go<128, 8, 2>(a, t, st) : go<128, 8, 1>(a, t, st);
  }
  return a.bits == 4 ? go<256, 4, 1>(a, t, st) : go<256, 8, 1>(a, t, st);
}

}  // namespace hit

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
//   V to fp16 likewise; the other operand, probability times the value's scale, is
//     rounded to fp16.
// What a row's sums are relative to follows that product (the base-2 score plus the logarithm
// of the value's scale), so that fp16 holds the ones that make up the result, whatever
// the scales of positions that the row does not see or gives no weight.
// O^T += V^T P^T takes P^T from the score accumulators with one 8x8 transpose
// per 8 positions.  Scales never touch the codes: the key's multiplies its
// score, the value's its probability.
//
// 64 sequences of 300 to 8,000 positions (32 heads on 8, head 128, 4 bits) take
// 85 us, two of 125,000 (8 bits) 69 us: 3.0 and 4.0 TB/s, where the loop over the
// units alone runs at 5.3 to 5.9 TB/s.  The rest is finding the share, preparing
// the queries and the first loads (about 10 us), uneven ends, and the joining
// launch (8 us).
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
constexpr float kGrow = 32768.0f;  // bound of a column's products above which it gets a new reference
constexpr float kRoom = 4.0f;      // the largest product is 2^kRoom with a new reference
// A reference stays within 2^kFar of the largest probability, and a lane's share of a column's
// sum below kFull, so that fp32 holds the sum where the values are next to nothing.
constexpr float kFar = 90.0f, kFull = 1.2676506e30f;  // 2^100
constexpr int kLead = 16;  // beginning a pair takes a CTA about as long as 16 units

// Positions of a unit: stages of 2 to 4 KB (8 KB for heads of 256); three of
// them for each of 16 warps on an SM (8 with more than eight query rows or heads of 256),
// two on their way while one is worked on.
template <int D, int BITS>
struct Few {
  static constexpr int VB = D * BITS / 8;  // bytes of a vector's codes
  static constexpr int CH = VB / 16;
  static constexpr int TK = VB <= 64 ? 32 : VB == 128 ? (D == 256 ? 32 : 16) : 16;
  static constexpr int MT = TK / 16;
  static constexpr int STAGE = TK * (2 * VB + 8) + 16;
  static constexpr int KS = D / 16;
};

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void lds64(uint32_t p, uint32_t* r) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(p));
}
__device__ __forceinline__ void lds128(uint32_t p, uint32_t* r) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(p));
}

// Places of 16-byte piece q of position t in a stage, such that the lanes of one
// shared-memory read touch every bank once.  Keys are read as 8 positions x 4
// pieces (16 bytes a lane; 8 bytes where a position has only two pieces), values
// by 8x8 transposing loads of one piece of 8 positions.
template <int CH>
__device__ __forceinline__ int k_place(int t, int q) {
  return CH <= 4 ? t * CH + q : t * CH + (q ^ ((t & 1) << 2));
}
template <int CH>
__device__ __forceinline__ int v_place(int t, int q) {
  if constexpr (CH == 2) return t * CH + (q ^ ((t >> 2) & 1));
  if constexpr (CH == 4) return t * CH + (q ^ ((t >> 1) & 3));
  return t * CH + (q ^ (t & 7));
}
// Four 8x8 transposing loads of 16-bit units (`at`: this lane's row of matrix lane / 8).
__device__ __forceinline__ void load_transposed(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}

template <int D, int BITS, int NT, int MINB>
__global__ void __launch_bounds__(kThreads, MINB) k_kv_few(const KvArgs a, const KvAttn t) {
  using F = Few<D, BITS>;
  constexpr int ROWS = 8 * NT, TK = F::TK, MT = F::MT, CH = F::CH, VB = F::VB, KS = F::KS;
  constexpr int OM = D / 16;   // 16-element tiles of the output's head dimension
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t turns[D / 2];
  __shared__ uint4 qs[ROWS * (D / 8)];  // [rows / 8][D / 32][8 rows][4 lanes]: a lane's operands of eight elements
  __shared__ float es[ROWS];
  __shared__ uint32_t k_neg[D / 32];  // a bit for each element whose sign is flipped
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r8 = lane >> 2, c4 = lane & 3;
  kv_turns(a, turns, threadIdx.x, kThreads);  // kv_plan's barriers follow
  for (int i = warp; i < D / 32; i += kWarps) {
    const uint32_t b = __ballot_sync(0xffffffffu, a.k_signs != nullptr && __ldg(a.k_signs + 32 * i + lane) < 0);
    if (lane == 0) k_neg[i] = b;
  }
  const KvPlan plan = kv_plan<ROWS, TK, kLead, kThreads>(a, t, kWarps);
  const KvWork work = kv_work_of<D, ROWS>(t.ws, gridDim.x);
  KvPart open;
  open.first = -1;
  const bool one_page = (1 << a.log_page) >= TK;
  const uint32_t in_page = (1u << a.log_page) - 1;
  uint8_t* const ring = smem + warp * F::STAGE;  // of this warp, a stage every kWarps * STAGE
  auto page_at = [&](int s, int64_t p) {  // p >= 0 lies in the table: units end at KvSeq::hi
    return __ldg(a.table + int64_t(s) * a.ld_table + (p >> a.log_page));
  };
  constexpr uint64_t kAll = TK == 64 ? ~uint64_t(0) : (uint64_t(1) << (TK & 63)) - 1;

  int s = plan.seq;
  int64_t base = plan.base;
  KvSeq q{};
  if (s < a.seqs) q = kv_seq<ROWS, TK, kLead>(a, t, s);
  for (int64_t u = plan.u0; u < plan.u1;) {
    const int64_t rel = u - base;
    const int64_t pair = rel / q.units;
    const int64_t x0 = rel - pair * q.units;
    const int64_t x1 = min(q.units, x0 + plan.u1 - u);
    const bool begins = x0 <= kLead;  // no unit of the pair's keys lies in an earlier CTA's share
    if (x1 <= kLead) {                // and none in this one's
      u += x1 - x0;
      continue;
    }
    const int h = int(pair / q.row_tiles), rt = int(pair - int64_t(h) * q.row_tiles);
    const int row0 = rt * ROWS;
    const int nr = int(min(int64_t(ROWS), int64_t(q.n) * t.group - row0));
    const int i0 = row0 / t.group, i1 = (row0 + nr - 1) / t.group;  // first and last token of the tile
    // what the tile's rows see, first and last
    const int64_t hi_min = t.causal ? min(q.hi, q.pos0 + i0 + 1) : q.hi;
    const int64_t hi_max = t.causal ? min(q.hi, q.pos0 + i1 + 1) : q.hi;
    const int64_t lo_min = t.window > 0 ? max(int64_t(0), q.pos0 + i0 - t.window + 1) : 0;
    const int64_t lo_max = t.window > 0 ? max(int64_t(0), q.pos0 + i1 - t.window + 1) : 0;
    const int64_t b0 = max(max(x0 - kLead, int64_t(0)), lo_min / TK - q.unit0);
    const int64_t b1 = min(x1 - kLead, (hi_max + TK - 1) / TK - q.unit0);
    const int nu = b0 + warp < b1 ? int((b1 - b0 - warp + kWarps - 1) / kWarps) : 0;

    // The warp's next unit into its next stage.  Where a unit lies inside a page
    // (pages of at least TK positions) its vectors are one run of memory and the
    // lane's pieces have fixed offsets; positions behind the sequence's end are
    // then copied too (they are the page's) and hidden from every row later.  A
    // missing page leaves the stage as it is: nothing of it is seen.
    const int64_t head = int64_t(h) << a.log_page;
    int next = 0, next_stage = 0;
    int64_t next_p = (q.unit0 + b0 + warp) * TK;
    int next_page = one_page && nu > 0 ? page_at(s, next_p) : -1;
    auto issue = [&]() {
      if (next < nu) {
        uint8_t* const stp = ring + next_stage * (kWarps * F::STAGE);
        const uint32_t st = smem_u32(stp);
        uint64_t there = 0;
        if (one_page) {
          const int page = next_page;
          if (next + 1 < nu) next_page = page_at(s, next_p + kWarps * TK);
          if (page >= 0 && page < a.pages) {
            there = kAll;
            const int64_t vec = ((int64_t(page) * a.hk) << a.log_page) + head + (uint32_t(next_p) & in_page);
            const uint8_t* const kc = a.k_codes + vec * VB + 16 * lane;
            const uint8_t* const vc = a.v_codes + vec * VB + 16 * lane;
#pragma unroll
            for (int k = 0; k < TK * CH / 32; ++k) {
              const int tk = (32 * k) / CH + lane / CH;
              copy16(st + 16 * k_place<CH>(tk, lane % CH), kc + 512 * k);
              copy16(st + TK * VB + 16 * v_place<CH>(tk, lane % CH), vc + 512 * k);
            }
            if (lane < TK / 4) {
              copy16(st + 2 * TK * VB + 16 * lane, a.k_scales + vec + 4 * lane);
              copy16(st + 2 * TK * VB + 4 * TK + 16 * lane, a.v_scales + vec + 4 * lane);
            }
          }
        } else {
          int64_t at[(TK + 31) / 32];
#pragma unroll
          for (int k = 0; k < (TK + 31) / 32; ++k) {
            const int64_t p = next_p + lane + 32 * k;
            at[k] = lane + 32 * k < TK && p < q.hi ? kv_slot(a, s, p) : -1;
            there |= uint64_t(__ballot_sync(0xffffffffu, at[k] >= 0)) << (32 * k);
            if (at[k] >= 0) {
              at[k] += head;
              copy4(st + 2 * TK * VB + 4 * (lane + 32 * k), a.k_scales + at[k]);
              copy4(st + 2 * TK * VB + 4 * (TK + lane + 32 * k), a.v_scales + at[k]);
            }
          }
#pragma unroll
          for (int k = 0; k < TK * CH / 32; ++k) {
            const int tk = (32 * k) / CH + lane / CH, piece = lane % CH;
            const int64_t vec = __shfl_sync(0xffffffffu, at[(32 * k) / CH / 32], tk & 31);
            if (vec >= 0) {
              copy16(st + 16 * k_place<CH>(tk, piece), a.k_codes + vec * VB + 16 * piece);
              copy16(st + TK * VB + 16 * v_place<CH>(tk, piece), a.v_codes + vec * VB + 16 * piece);
            }
          }
        }
        if (lane == 0) *reinterpret_cast<uint64_t*>(stp + TK * (2 * VB + 8)) = there;
        ++next;
        next_p += kWarps * TK;
        next_stage = next_stage == kStages - 1 ? 0 : next_stage + 1;
      }
      copies_commit();
    };
    // The tile's queries: turned, rotated, scaled (into base-2 scores), and
    // brought to [-2, 2) by a power of two.  D / 8 threads a row, eight elements
    // each; the first units are on their way meanwhile.
    uint32_t qf[KS][NT][2];
    float qe[NT][2];
    int lo[NT][2], hi[NT][2];
    {
      constexpr int TPR = D / 8, PER = kThreads / TPR;
      const int ch = threadIdx.x % TPR, i0e = 8 * ch;
      float x[(ROWS + PER - 1) / PER][8];
#pragma unroll
      for (int p = 0; p * PER < ROWS; ++p) {
        const int r = p * PER + int(threadIdx.x) / TPR;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[p][e] = 0.0f;
        if (r < nr) {
          const int row = row0 + r, tok = row / t.group;
          const int64_t src = (q.t0 + tok) * t.q_ts + (int64_t(h) * t.group + row - tok * t.group) * t.q_hs + i0e;
          if (t.q_f32) kv_load8<true>(t.q, src, x[p]);
          else kv_load8<false>(t.q, src, x[p]);
        }
      }
      issue();
      issue();
#pragma unroll
      for (int p = 0; p * PER < ROWS; ++p) {
        const int r = p * PER + int(threadIdx.x) / TPR;
        float(&y)[8] = x[p];
        if (a.n_freq > 0) {
          const int tok = r < nr ? (row0 + r) / t.group : 0;
          const int pos = int(q.pos0) + tok;
          const bool low = i0e < a.n_freq, turned = i0e < 2 * a.n_freq;
          if (a.interleaved) {
            if (turned) {
#pragma unroll
              for (int e = 0; e < 8; e += 2) {
                const float2 cs = kv_angle_fast(a, turns, q.t0 + tok, pos, (i0e + e) / 2);
                const float u = y[e], w = y[e + 1];
                y[e] = u * cs.x - w * cs.y;
                y[e + 1] = u * cs.y + w * cs.x;
              }
            }
          } else {
            // the partner chunk is n_freq elements on or back (n_freq % 8 == 0), with another lane of the row
            const int shift = turned ? (low ? a.n_freq / 8 : -(a.n_freq / 8)) : 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float w = __shfl_sync(0xffffffffu, y[e], lane + shift);
              if (turned) {
                const float2 cs = kv_angle_fast(a, turns, q.t0 + tok, pos, (low ? i0e : i0e - a.n_freq) + e);
                y[e] = low ? y[e] * cs.x - w * cs.y : w * cs.y + y[e] * cs.x;
              }
            }
          }
        }
        const uint32_t neg = k_neg[ch >> 2] >> (8 * (ch & 3));
#pragma unroll
        for (int e = 0; e < 8; ++e)
          y[e] = __uint_as_float(__float_as_uint(y[e]) ^ ((neg << (31 - e)) & 0x80000000u));
        reg_stages<8, 0, 3>(y);
#pragma unroll
        for (int b = 1; b < TPR; b <<= 1) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float w = __shfl_xor_sync(0xffffffffu, y[e], b);
            y[e] = ch & b ? w - y[e] : y[e] + w;
          }
        }
        const float f = (D == 64 ? 0.125f : D == 256 ? 0.0625f : 0.08838834764831845f) * 1.4426950408889634f * t.scale;
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          y[e] *= f;
          top = max(top, __float_as_uint(y[e]) & 0x7fffffffu);
        }
#pragma unroll
        for (int b = 1; b < TPR; b <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, b));
        float up, down;
        kv_row_power(top, up, down);
        if (r < ROWS) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = BITS == 4 ? e : 2 * e, j = BITS == 4 ? e + 4 : 2 * e + 1;
            const __half2 v = __floats2half2_rn(y[i] * down, y[j] * down);
            w[e] = *reinterpret_cast<const uint32_t*>(&v);
          }
          // the chunk goes to the lane (of four) that holds its codes, as its how manieth
          const int owner = CH == 2 ? ch >> 1 : BITS == 4 ? (ch >> 2) & 3 : (ch >> 1) & 3;
          const int at = CH == 2 ? ch & 1 : BITS == 4 ? 4 * (ch >> 4) + (ch & 3) : 2 * (ch >> 3) + (ch & 1);
          qs[(((r >> 3) * (D / 32) + at) * 8 + (r & 7)) * 4 + owner] = make_uint4(w[0], w[1], w[2], w[3]);
          if (ch == 0) es[r] = up;
        }
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          const uint4 v = qs[((n * (D / 32) + w) * 8 + r8) * 4 + c4];
          qf[2 * w][n][0] = v.x;
          qf[2 * w][n][1] = v.y;
          qf[2 * w + 1][n][0] = v.z;
          qf[2 * w + 1][n][1] = v.w;
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
    }

    float o[OM][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < OM; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.0f;
      // columns behind the tile's rows need no reference
      m[n][0] = 8 * n + 2 * c4 < nr ? -INFINITY : 0.0f;
      m[n][1] = 8 * n + 2 * c4 + 1 < nr ? -INFINITY : 0.0f;
      l[n][0] = l[n][1] = 0.0f;
    }
    int stage = 0;
    for (int i = 0; i < nu; ++i) {
      issue();
      copies_wait<2>();
      __syncwarp();
      uint8_t* const stp = ring + stage * (kWarps * F::STAGE);
      stage = stage == kStages - 1 ? 0 : stage + 1;
      const uint32_t st = smem_u32(stp);
      const uint64_t there = *reinterpret_cast<const uint64_t*>(stp + TK * (2 * VB + 8));
      const float* ks = reinterpret_cast<const float*>(stp + 2 * TK * VB);
      const float* vs = ks + TK;
      const int64_t p0 = (q.unit0 + b0 + warp + int64_t(kWarps) * i) * TK;
      const bool full = p0 >= lo_max && p0 + TK <= hi_min && there == kAll;

      float sc[MT][NT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int n = 0; n < NT; ++n) sc[mt][n][0] = sc[mt][n][1] = sc[mt][n][2] = sc[mt][n][3] = 0.0f;
        const int tk = 16 * mt + r8;
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
            sc[mt][n][e] *= e < 2 ? k0 : k1;
          }
        }
      }
      if (!full) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int w = 16 * mt + r8 + (e < 2 ? 0 : 8);
            const int p = int(p0) + w;
            const bool in = (there >> w) & 1;
#pragma unroll
            for (int n = 0; n < NT; ++n)
              if (!in || p < lo[n][e & 1] || p >= hi[n][e & 1]) sc[mt][n][e] = -INFINITY;
          }
      }

      // Probabilities against the columns' references so far, and a bound of their products
      // with the values' scales.  A reference is a maximum of products seen before (as
      // logarithms), less kRoom, and is only raised where the bound exceeds kGrow.
      float pr[MT][NT][4], add[NT][2];
      auto powers = [&]() {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float b0_ = m[n][0] == -INFINITY ? 0.0f : -m[n][0], b1_ = m[n][1] == -INFINITY ? 0.0f : -m[n][1];
          add[n][0] = add[n][1] = 0.0f;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              pr[mt][n][e] = ex2(fmaf(sc[mt][n][e], qe[n][e & 1], e & 1 ? b1_ : b0_));
              add[n][e & 1] += pr[mt][n][e];
            }
        }
      };
      powers();
      uint32_t big = __float_as_uint(vs[lane & (TK - 1)]) & 0x7fffffffu;
      if (!full) {  // of positions that a row of the tile sees: others hold anything
        const int64_t p = p0 + (lane & (TK - 1));
        if (!((there >> (lane & (TK - 1))) & 1) || p < lo_min || p >= hi_max) big = 0;
      }
      if (big >= 0x7f800000u) big = 0;
      const float largest = __uint_as_float(__reduce_max_sync(0xffffffffu, big));
      bool grow = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) grow |= m[n][k] == -INFINITY || add[n][k] * largest > kGrow || add[n][k] > kFull;
      if (__any_sync(0xffffffffu, grow)) {
        float lv[MT][2];  // the values' scales as logarithms
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          lv[mt][0] = __log2f(vs[16 * mt + r8]);
          lv[mt][1] = __log2f(vs[16 * mt + r8 + 8]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float f[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float v = -INFINITY, w = -INFINITY;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const float x0 = sc[mt][n][k] * qe[n][k], x1 = sc[mt][n][k + 2] * qe[n][k];
              v = fmaxf(v, fmaxf(x0, x1));
              w = fmaxf(w, fmaxf(x0 == -INFINITY ? x0 : x0 + lv[mt][0], x1 == -INFINITY ? x1 : x1 + lv[mt][1]));
            }
            v = fmaxf(w, v - kFar);
#pragma unroll
            for (int b = 4; b < 32; b <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, b));
            // a column's lanes agree on v, and so on its new reference
            v -= kRoom;
            // in two halves: the sum of probabilities outlives a step of more than 2^126
            const float half = v > m[n][k] ? ex2(0.5f * (m[n][k] - v)) : 1.0f;
            m[n][k] = fmaxf(m[n][k], v);
            f[k] = half * half;
            l[n][k] = l[n][k] * half * half;
          }
#pragma unroll
          for (int d = 0; d < OM; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][n][e] *= f[e & 1];
        }
        powers();
      }
      // fp16 keeps 11 bits of a product down to 2^-18 of the largest (bf16 kept 8: an error
      // of 0.0024 of the result in place of 0.0017).
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        l[n][0] += add[n][0];
        l[n][1] += add[n][1];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const float v0 = vs[16 * mt + r8], v1 = vs[16 * mt + r8 + 8];
#pragma unroll
          for (int e = 0; e < 4; ++e) pr[mt][n][e] *= e < 2 ? v0 : v1;
        }
      }
      if (!full) {  // the scale of a hidden position may be anything
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) pr[mt][n][e] = sc[mt][n][e] == -INFINITY ? 0.0f : pr[mt][n][e];
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        uint32_t pb[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const __half2 lo2 = __floats2half2_rn(pr[mt][n][0], pr[mt][n][1]), hi2 = __floats2half2_rn(pr[mt][n][2], pr[mt][n][3]);
          pb[n][0] = transpose8x8(*reinterpret_cast<const uint32_t*>(&lo2));
          pb[n][1] = transpose8x8(*reinterpret_cast<const uint32_t*>(&hi2));
        }
        // 16-bit units of codes, of two neighbouring positions a register: matrix
        // lane / 8 of a load is positions 8 (lane / 8 % 2) ... of piece x or x + 1
#pragma unroll
        for (int x = 0; x < CH; x += 2) {
          const int tk = 16 * mt + (lane & 15), piece = x + (lane >> 4);
          uint32_t v[4];
          load_transposed(st + TK * VB + 16 * v_place<CH>(tk, piece), v);
#pragma unroll
          for (int y = 0; y < 2; ++y) {  // positions 0-7 and 8-15 of piece x + y
            if constexpr (BITS == 4) {
              uint32_t ab[4], cd[4];
              half_runs4(v[2 * y], ab);
              half_runs4(v[2 * y + 1], cd);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                mma_f16(o[2 * (x + y)][n], ab[0], ab[1], cd[0], cd[1], pb[n][0], pb[n][1]);
                mma_f16(o[2 * (x + y) + 1][n], ab[2], ab[3], cd[2], cd[3], pb[n][0], pb[n][1]);
              }
            } else {
              uint32_t a0, a1, c0, c1;
              half_runs8(v[2 * y], a0, a1);
              half_runs8(v[2 * y + 1], c0, c1);
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_f16(o[x + y][n], a0, a1, c0, c1, pb[n][0], pb[n][1]);
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
        float* dst = mo + (warp * ROWS + r) * D;
        if constexpr (BITS == 4) {  // tiles 2 x and 2 x + 1: elements 32 x + 4 r8 ...
#pragma unroll
          for (int x = 0; x < CH; ++x)
            *reinterpret_cast<float4*>(dst + 32 * x + 4 * r8) =
                make_float4(o[2 * x][n][k], o[2 * x][n][k + 2], o[2 * x + 1][n][k], o[2 * x + 1][n][k + 2]);
        } else {  // tile x: elements 16 x + 2 r8, + 1
#pragma unroll
          for (int x = 0; x < CH; ++x)
            *reinterpret_cast<float2*>(dst + 16 * x + 2 * r8) = make_float2(o[x][n][k], o[x][n][k + 2]);
        }
      }
    }
    __syncthreads();
    const bool whole = begins && x1 == q.units;
    const size_t slot = begins ? 2 * blockIdx.x + 1 : 2 * blockIdx.x;
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
        const float half = kv_weight(v.x, top), g = half * half;
        sum = fmaf(v.y * half, half, sum);
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
    if (!whole && begins) {
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
        q = kv_seq<ROWS, TK, kLead>(a, t, ++s);
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
  return launch_kv_join<D, 8 * NT, 1>(a, t, ctas, st);
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

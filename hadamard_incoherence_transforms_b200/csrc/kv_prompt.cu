// Attention over the rotated cache for many query rows (chunks of prompts):
// bound by the matrix products.
//
// A CTA (one per SM) takes an equal share of the list of (sequence, key/value
// head, 256 query rows) x 128 positions units.  Roles:
//   warps 0-3, 4-7  softmax of the upper and of the lower 128 query rows, a
//                   thread a row, its scores in tensor memory;
//   warps 8-11      codes to fp16 keys and values in shared memory (128-byte
//                   swizzle), a two-stage ring each, the next unit's codes on
//                   their way in registers;
//   warp 13         finds the CTA's segments and hands them to the others;
//   warp 12         one thread issues the products: S = Q K^T, O += P V (fp16, P
//                   read from tensor memory where it replaced S).
// The two halves alternate: while one half's softmax runs, the tensor cores
// work on the other's products.  Key and value units are converted once for
// both, their scales folded in with one rounding of 2^-11 (half the work of the
// softmax roles went into scales otherwise, see UnitSoftmax for what is left) wherever a
// block's scales lie within 2^kSpread of one another.
//
// 4,096 tokens on 12,000 cached ones (32 heads on 8, head 128, 4 bits) take 1.27 ms,
// 742 TFLOP/s or 44 % of a measured library product; 8 bits 1.44 ms.  Before positions could
// have powers of two of their own it was 1.23 ms; of the 0.04 the unpacking warps'
// tests of each scale are 0.03.  A unit took 5,600 cycles then: a half's softmax 3,400 of
// them (1,500 were it alone on the SM; both halves share the exponential units, 2,048 a
// unit), and 2,200 until its next scores are there (products of both halves, 2,050 a
// unit at the pipe's rate).  Scores in two parts of 64 positions, the next one's product
// under way during the softmax, took 1.30 ms against 1.24: products of 64 columns read the
// queries from shared memory twice.  Heads of 64 and 128 spill 300 to 440 bytes a thread
// (-Xptxas -v; heads of 256 none to speak of); what that costs is not known.
#include "internal.h"
#include "kv_codes.cuh"
#include "kv_split.cuh"

#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

namespace hit {

__device__ unsigned int g_wait_timeouts_kv = 0;

namespace {

constexpr int kKeys = 128;      // positions of a unit
constexpr int kThreads = 16 * 32;  // warps 14 and 15 are idle: registers are dealt out to groups of four warps
constexpr int kCtas = 148;
constexpr float kGrow = 32768.0f;  // sum of 32 probabilities above which a row gets a new reference
constexpr float kRoom = 4.0f;      // a reference's own probability is 2^kRoom
constexpr int kKeyBits = 7;        // the largest key scale of a unit becomes 2^kKeyBits or more
constexpr int kValueBits = 4;      // the largest value scale of the unit that a power of two was taken from, 2^kValueBits
// Scales down to 2^-kSpread of the largest share its power of two: the second part of a scale
// is 2^-16 (keys) and 2^-12 (values) of it there, or more.  A block with a scale below that
// takes nine times as long (UnitSoftmax::run_apart): values' scales drawn over 2^10 from
// position to position, beside their usual spread, take 1.28 ms with 16 and 10.6 with 12.
constexpr int kSpread = 16;

template <int D>
struct Prompt {
  // Heads of 256 have room for one half of 128 rows (256 columns of O, 64 KB tiles),
  // and for one stage of keys and of values.
  static constexpr int HALVES = D == 256 ? 1 : 2;
  static constexpr int ROWS = 128 * HALVES;      // query rows of a unit
  static constexpr uint32_t STAGES = HALVES;
  static constexpr int TILE = D * 2 * 128;       // 128 vectors of D 16-bit elements
  static constexpr int Q = 0, K = HALVES * TILE, V = K + STAGES * TILE, SC = V + STAGES * TILE;
  // registers of a thread of the four groups of warps; the launch has 4 x 128
  static constexpr int SOFTMAX = D == 256 ? 208 : 160, UNPACK = 112, OTHER = 80;
  static_assert(SOFTMAX + (HALVES == 2 ? SOFTMAX : UNPACK) + UNPACK + OTHER <= 512, "registers");
  static constexpr float NORM = D == 64 ? 0.125f : D == 256 ? 0.0625f : 0.08838834764831845f;
  // ring of four units: which positions exist (128 bits), the powers of two of keys and of
  // values, and whether any position of each unpacking warp has its own (4 + 4 bytes)
  static constexpr int SC_STAGE = 32;
  static constexpr int TS = SC + 4 * SC_STAGE;   // the largest scales of each unpacking warp, two units
  // ring of four units: the exponents of the keys' and of the values' own powers of two, a
  // byte a position.  (Shared memory of more than 196 KB leaves a third of the L1 cache, and
  // registers live there: 1.31 ms in place of 1.23 with 4 KB more.)
  static constexpr int OWN = TS + 64, OWN_STAGE = 2 * kKeys;
  static constexpr int BARS = OWN + 4 * OWN_STAGE;
  static constexpr int BYTES = BARS + 240 + 1008;  // the last for the alignment of the tiles
  static constexpr int S_COL = 0, O_COL = 2 * 128;  // tensor memory columns
  static constexpr int COLS = 512;
};

struct Bars {
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2], sc[4];
  uint64_t q[2], s[2], p[2], o[2], done;
  uint32_t tmem;
  int abort;
  // the CTA's share
  int64_t total, units;
  int ctas, seq, h, rt, x0;
};
static_assert(sizeof(Bars) <= 240, "barrier block");

// ---------------------------------------------------------------------------
// The list of units.
// ---------------------------------------------------------------------------
// Every row tile counts kLead units ahead of its keys' ones: what its queries and
// its result take, so that CTAs with many short tiles get fewer positions. 16
// prompts of 16 to 512 tokens on up to 8,000 (32 heads on 8): 360 us without, 311
// with 3; one prompt of 1,024 tokens 93 and 82; 2 and 5 lie within 2 %.
constexpr int kLead = 3;
// Units of row tile rt of a sequence: [first, first + count).
template <int ROWS>
__device__ __forceinline__ void tile_units(const KvAttn& t, const KvSeq& q, int rt, int& first, int& count) {
  const int64_t rows = int64_t(q.n) * t.group;
  const int64_t r0 = int64_t(rt) * ROWS, r1 = min(rows, r0 + ROWS);
  const int64_t i0 = r0 / t.group, i1 = (r1 - 1) / t.group;
  const int64_t hi = t.causal ? max(int64_t(0), min(q.hi, q.pos0 + i1 + 1)) : q.hi;
  const int64_t lo = t.window > 0 ? min(hi, max(int64_t(0), q.pos0 + i0 - t.window + 1)) : 0;
  first = int(lo / kKeys);
  count = max(1, int((hi + kKeys - 1) / kKeys) - first);
}

// Units of a sequence for one key/value head, found by a warp.
template <int ROWS>
__device__ __forceinline__ int64_t head_units_warp(const KvAttn& t, const KvSeq& q, int lane) {
  int64_t sum = 0;
  for (int rt = lane; rt < q.row_tiles; rt += 32) {
    int f, c;
    tile_units<ROWS>(t, q, rt, f, c);
    sum += c + kLead;
  }
#pragma unroll
  for (int b = 16; b; b >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, b);
  return sum;
}

// Units of sequences s0 .. s0 + 31, one to a lane.
template <int ROWS>
__device__ __forceinline__ int64_t chunk_units(const KvArgs& a, const KvAttn& t, int s0, int lane) {
  int64_t w = 0;
  bool big = false;
  if (s0 + lane < a.seqs) {
    const KvSeq q = kv_seq<ROWS, kKeys, 0>(a, t, s0 + lane);
    if (kv_mine(t, q)) {
      big = q.row_tiles > 4;
      for (int rt = 0; rt < q.row_tiles && !big; ++rt) {
        int f, c;
        tile_units<ROWS>(t, q, rt, f, c);
        w += c + kLead;
      }
    }
  }
  for (uint32_t m = __ballot_sync(0xffffffffu, big); m; m &= m - 1) {
    const int k = __ffs(m) - 1;
    const int64_t v = head_units_warp<ROWS>(t, kv_seq<ROWS, kKeys, 0>(a, t, s0 + k), lane);
    if (lane == k) w = v;
  }
  return w * a.hk;
}

// One warp finds the CTA's share and where it begins.
template <int ROWS>
__device__ __forceinline__ void plan_warp(const KvArgs& a, const KvAttn& t, Bars* b, int lane) {
  int64_t total = 0;
  for (int s0 = 0; s0 < a.seqs; s0 += 32) total += chunk_units<ROWS>(a, t, s0, lane);
#pragma unroll
  for (int i = 16; i; i >>= 1) total += __shfl_xor_sync(0xffffffffu, total, i);
  const int64_t ctas = max(int64_t(1), min(int64_t(gridDim.x), (total + 1) / 2));
  const int64_t c = blockIdx.x;
  const int64_t u0 = c < ctas ? c * total / ctas : total, u1 = c < ctas ? (c + 1) * total / ctas : total;
  int seq = a.seqs;
  int64_t base = 0;
  if (u0 < u1) {
    for (int s0 = 0; s0 < a.seqs; s0 += 32) {
      const int64_t v = chunk_units<ROWS>(a, t, s0, lane);
      int64_t x = v;
#pragma unroll
      for (int i = 1; i < 32; i <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, i);
        if (lane >= i) x += y;
      }
      const uint32_t in = __ballot_sync(0xffffffffu, base + x > u0);
      if (in) {
        const int k = __ffs(in) - 1;
        seq = s0 + k;
        base += __shfl_sync(0xffffffffu, x - v, k);
        break;
      }
      base += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  int h = 0, rt = 0, x0 = 0;
  if (seq < a.seqs) {
    const KvSeq q = kv_seq<ROWS, kKeys, 0>(a, t, seq);
    const int64_t per = head_units_warp<ROWS>(t, q, lane);
    h = int((u0 - base) / per);
    int64_t r = u0 - base - h * per;
    for (int r0 = 0; r0 < q.row_tiles; r0 += 32) {
      int f, v = 0;
      if (r0 + lane < q.row_tiles) {
        tile_units<ROWS>(t, q, r0 + lane, f, v);
        v += kLead;
      }
      int64_t x = v;
#pragma unroll
      for (int i = 1; i < 32; i <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, i);
        if (lane >= i) x += y;
      }
      const uint32_t in = __ballot_sync(0xffffffffu, x > r);
      if (in) {
        const int k = __ffs(in) - 1;
        rt = r0 + k;
        x0 = int(r - __shfl_sync(0xffffffffu, x - v, k));
        break;
      }
      r -= __shfl_sync(0xffffffffu, x, 31);
    }
  }
  if (lane == 0) {
    b->total = total;
    b->units = u1 - u0;
    b->ctas = int(ctas);
    b->seq = seq;
    b->h = h;
    b->rt = rt;
    b->x0 = x0;
  }
}

// Half of a segment's rows: the units [js, je) that its rows may see there, and
// the positions [lo_max, hi_min) that all of them see.
struct Half {
  int rows, js, je, pad;
  int64_t lo_max, hi_min;
};
// A CTA's part of one (sequence, head, row tile).  One warp walks the CTA's
// share and hands the segments to the other roles through shared memory.
struct Segment {
  int64_t t0, pos0, hi;  // of the sequence: first token, its position, positions that can exist
  int s, h, row0, nr;
  int ub, ue;            // units that either half needs
  int begins, whole;     // the row tile begins here; it begins and ends here
  int last;              // last CTA of the row tile
  int valid;             // 0: no more segments
  Half half[2];
};
constexpr int kSegments = 4;
struct SegmentRing {
  Segment seg[kSegments];
  uint64_t full[kSegments], empty[kSegments];
};

// The walk over the share: segments into the ring, then one that ends it.
// True unless a wait ran out.
template <int ROWS>
__device__ __forceinline__ bool walk(const KvArgs& a, const KvAttn& t, const Bars* b, SegmentRing* ring,
                                     volatile int* abort) {
  int s = b->seq, h = b->h, rt = b->rt, x0 = b->x0;
  int64_t left = b->units, at = int64_t(blockIdx.x) * b->total / b->ctas;
  KvSeq q{};
  if (left > 0) q = kv_seq<ROWS, kKeys, 0>(a, t, s);
  // the next row tile
  auto step = [&]() {
    x0 = 0;
    if (++rt == q.row_tiles) {
      rt = 0;
      if (++h == a.hk) {
        h = 0;
        do {
          q = kv_seq<ROWS, kKeys, 0>(a, t, ++s);
        } while (q.n == 0 || !kv_mine(t, q));
      }
    }
  };
  for (int n = 0;; ++n) {
    int first = 0, count = 0, x1 = 0;
    while (left > 0) {
      tile_units<ROWS>(t, q, rt, first, count);
      x1 = int(min(int64_t(count + kLead), x0 + left));
      if (x1 > kLead) break;
      // no unit of keys: what is left begins in the next CTA
      at += x1 - x0;
      left -= x1 - x0;
      if (left > 0) step();
    }
    if (n >= kSegments && !mbar_wait(&ring->empty[n % kSegments], uint32_t(n / kSegments - 1) & 1u)) return false;
    if (*abort) return true;
    Segment& g = ring->seg[n % kSegments];
    g.valid = left > 0;
    if (left > 0) {
      g.t0 = q.t0;
      g.pos0 = q.pos0;
      g.hi = q.hi;
      g.s = s;
      g.h = h;
      g.row0 = rt * ROWS;
      g.nr = int(min(int64_t(ROWS), int64_t(q.n) * t.group - g.row0));
      int ub = INT32_MAX, ue = 0;
      for (int k = 0; k < 2; ++k) {
        Half f{min(128, max(0, g.nr - 128 * k)), 0, 0, 0, 0, 0};
        if (f.rows > 0) {
          const int64_t i0 = (g.row0 + 128 * k) / t.group, i1 = (g.row0 + 128 * k + f.rows - 1) / t.group;
          const int64_t hi = t.causal ? max(int64_t(0), min(q.hi, q.pos0 + i1 + 1)) : q.hi;
          const int64_t lo = t.window > 0 ? min(hi, max(int64_t(0), q.pos0 + i0 - t.window + 1)) : 0;
          f.hi_min = t.causal ? min(q.hi, q.pos0 + i0 + 1) : q.hi;
          f.lo_max = t.window > 0 ? q.pos0 + i1 - t.window + 1 : 0;
          f.js = max(first + max(0, x0 - kLead), int(lo / kKeys));
          f.je = min(first + x1 - kLead, int((hi + kKeys - 1) / kKeys));
          if (f.js < f.je) {
            ub = min(ub, f.js);
            ue = max(ue, f.je);
          } else {
            f.je = f.js;
          }
        }
        g.half[k] = f;
      }
      g.ub = ub < ue ? ub : 0;
      g.ue = ub < ue ? ue : 0;
      g.begins = x0 <= kLead;
      g.whole = x0 <= kLead && x1 == count + kLead;
      g.last = kv_cta_of(at - x0 + count + kLead - 1, b->total, b->ctas);
      at += x1 - x0;
      left -= x1 - x0;
      if (left > 0) step();
    }
    mbar_arrive(&ring->full[n % kSegments]);
    if (!g.valid) return true;
  }
}

// A role's view of the ring; next() is called by whole warps.
struct Follow {
  SegmentRing* ring;
  int n = -1;
  __device__ __forceinline__ const Segment& seg() const { return ring->seg[n % kSegments]; }
  // 1: a segment, 0: no more, -1: a wait ran out
  __device__ __forceinline__ int next(int lane) {
    if (n >= 0) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring->empty[n % kSegments]);
    }
    ++n;
    const bool ok = mbar_wait(&ring->full[n % kSegments], uint32_t(n / kSegments) & 1u);
    if (!__all_sync(0xffffffffu, ok)) return -1;
    return seg().valid ? 1 : 0;
  }
};

// ---------------------------------------------------------------------------
// tcgen05
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return uint64_t((addr >> 4) & 0x3fff) | (uint64_t((lbo >> 4) & 0x3fff) << 16) | (uint64_t((sbo >> 4) & 0x3fff) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// fp32 accumulator; A and B fp16; A K-major, M = 128
__host__ __device__ constexpr uint32_t instr_desc(int n, bool b_mn_major) {
  return (1u << 4) | (uint32_t(b_mn_major) << 16) | (uint32_t(n >> 3) << 17) | (uint32_t(128 >> 4) << 24);
}
// Shared-memory descriptors as their two words.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t id, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(id), "r"(uint32_t(add))
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t id, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(hi), "r"(id), "r"(uint32_t(add))
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void tmem_load32(uint32_t at, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
// Waits for the thread's loads; v: what must not be used before.
__device__ __forceinline__ void tmem_load_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_load32_now(uint32_t at, uint32_t (&r)[32]) {
  tmem_load32(at, r);
  tmem_load_wait(r);
}
__device__ __forceinline__ void tmem_load16_now(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_store8(uint32_t at, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Loads that stay where they are written.
__device__ __forceinline__ void load16(uint4& x, const void* p) {
  asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p));
}
__device__ __forceinline__ void load4(int& x, const int* p) {
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(x) : "l"(p));
}
__device__ __forceinline__ void load4(float& x, const float* p) {
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(x) : "l"(p));
}
// Registers of a group of four warps (all four run it).  The kernel starts with
// 128 a thread; 2 x 160 + 112 + 80 are the same 512.
template <int N>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_less() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// One row's softmax of a unit: its 128 scores in tensor memory become
// probabilities (fp16, in the same place).  m: the reference they are relative
// to, a maximum of scores seen before; l: the sum of probabilities; fix: what
// sums from before have to be multiplied with.
//
// 32 columns at a time, stored as soon as they are done (holding all of them
// costs more registers than the roles leave).  No maximum is taken as long as a
// row's probabilities add up to less than kGrow, which fp16 holds.  Above it, or
// while a row has no reference yet, the largest score, less kRoom, becomes the
// reference of the rows concerned, and the columns already stored (and, through
// `fix`, l and O) are brought to it.  fp16 then keeps 11 bits of a probability down
// to 2^-18 of the largest one, and the rest to 2^-29 of it.
struct UnitSoftmax {
  uint32_t s_at, p_at;  // tensor memory of the scores and of the probabilities
  uint4 there;          // positions that exist
  int c_lo, c_hi;       // columns [c_lo, c_hi) are this row's
  float qu;             // the row's and the unit's power of two

  // The softmax of a unit some of whose scales lie so far below the largest that their
  // keys or values are held by powers of two of their own (own: their exponents, keys' ahead
  // of values'; 0 where it is the unit's).  Scores are multiplied by the keys',
  // and probabilities (not their sum) by the values', relative to a power of two
  // 2^(ve - 127) that the row takes for O so that its largest product is 2^kRoom or more:
  // what a row does not see, or gives no weight to, costs it no digits.  Two
  // passes, as the largest product is wanted first; a function of its own, so that the
  // usual case keeps its registers.
  struct Row {
    float m, l, fix;
    uint32_t ve;
  };
  static __device__ __noinline__ Row run_apart(const UnitSoftmax u, const uint8_t* own, float qe, uint4 unit, float m, float l,
                                               uint32_t ve) {
    // unit: as in shared memory; only the runs of 32 positions that it names have bytes
    auto score = [&](uint32_t v, int j) {
      const uint32_t k = (unit.z >> (j / 32 * 8)) & 255 ? own[j] : 0;
      return __uint_as_float(v) * __uint_as_float(k == 0 ? unit.x : k << 23) * qe;
    };
    auto exponent = [&](int j) {
      const uint32_t v = (unit.w >> (j / 32 * 8)) & 255 ? own[kKeys + j] : 0;
      return float(int(v == 0 ? unit.y : v) - 127);
    };
    float top = -INFINITY, heavy = -INFINITY, fix = 1.0f;
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
      const uint32_t see = u.seen(c >> 1) >> (16 * (c & 1));
      if (!__any_sync(0xffffffffu, (see & 0xffffu) != 0)) continue;
      uint32_t v[16];
      tmem_load16_now(u.s_at + 16 * c, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (!((see >> i) & 1)) continue;
        const float x = score(v[i], 16 * c + i);
        top = fmaxf(top, x);
        heavy = fmaxf(heavy, x + exponent(16 * c + i));
      }
    }
    if (m == -INFINITY ? top > m : top - m > 11.0f) {  // probabilities stay below 2^11
      fix = ex2(m - (top - kRoom));                    // 0 for a first reference
      m = top - kRoom;
      l *= fix;
    }
    const float base = m == -INFINITY ? 0.0f : -m;
    float shift = 0.0f;  // what the values' exponents are relative to
    if (heavy > -INFINITY) {
      shift = fminf(fmaxf(floorf(heavy + base) - kRoom, -126.0f), 127.0f);
      ve = uint32_t(127 + int(shift));
    }
    // 16 columns at a time: their probabilities go where scores have been read before
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
      const uint32_t see = u.seen(c >> 1) >> (16 * (c & 1));
      uint32_t v[16], p[8];
      tmem_load16_now(u.s_at + 16 * c, v);
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        float y[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int j = 16 * c + i + k;
          const float x = (see >> (i + k)) & 1 ? score(v[i + k], j) + base : -INFINITY;
          l += ex2(x);
          y[k] = ex2(x + (exponent(j) - shift));
        }
        const __half2 h = __floats2half2_rn(y[0], y[1]);
        p[i / 2] = *reinterpret_cast<const uint32_t*>(&h);
      }
      tmem_store8(u.p_at + 8 * c, p);
    }
    return Row{m, l, fix, ve};
  }

  // O (times f) is to be brought to a power of two 2^d times as fine, the row's new ve.  Where
  // it would leave fp32's range ve is raised, and the unit's probabilities, which are
  // nothing beside it then, are lowered.  The factor for O, in Row::fix.
  template <int D>
  static __device__ __noinline__ Row fit(uint32_t o_at, uint32_t p_at, float f, int d, uint32_t ve) {
    tmem_store_wait();
    float top = 0.0f;
#pragma unroll 1
    for (int c = 0; c < D / 16; ++c) {
      uint32_t v[16];
      tmem_load16_now(o_at + 16 * c, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(__uint_as_float(v[i])));
    }
    top *= f;
    const int delta = top > 0.0f ? max(0, max(int(__float_as_uint(top) >> 23) - 127 + d - 100, d - 126)) : 0;
    if (__any_sync(0xffffffffu, delta > 0)) {
      const float less = delta > 126 ? 0.0f : __uint_as_float(uint32_t(127 - delta) << 23);
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t p[16];
        tmem_load16_now(p_at + 16 * c, p);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&p[i]));
          const __half2 z = __floats2half2_rn(y.x * less, y.y * less);
          p[i] = *reinterpret_cast<const uint32_t*>(&z);
        }
        tmem_store16(p_at + 16 * c, p);
      }
    }
    return Row{0.0f, 0.0f, f * __uint_as_float(uint32_t(127 + min(126, max(-126, d - delta))) << 23), ve + uint32_t(delta)};
  }

  __device__ __forceinline__ uint32_t seen(int c) const {  // of columns 32 c .. 32 c + 31
    const uint32_t e = c == 0 ? there.x : c == 1 ? there.y : c == 2 ? there.z : there.w;
    const int x0 = max(0, min(32, c_lo - 32 * c)), x1 = max(0, min(32, c_hi - 32 * c));
    const uint32_t below = x1 == 32 ? ~0u : (1u << x1) - 1, under = x0 == 32 ? ~0u : (1u << x0) - 1;
    return e & below & ~under;
  }
  // Probabilities of 32 columns, packed, and their sum.  The exponential unit
  // takes a warp's instruction every 8 cycles, and a warp issues in order: the
  // other work of the neighbouring columns is placed between two exponentials
  // (volatile, so that it stays there), else its time adds to theirs.
  template <bool FULL>
  __device__ __forceinline__ float probabilities(const uint32_t (&v)[32], uint32_t see, unsigned long long qu2,
                                                 unsigned long long base2, uint32_t (&p)[16]) const {
    unsigned long long sum[2] = {0, 0};
    float x[2][4];  // exponents of these and the next four columns
    float e[2][4];  // probabilities of these and the four before
    auto exponents = [&](int g, int h, float (&y)[4]) {  // columns 4 g + 2 h, + 1
      const int i = 4 * g + 2 * h;
      unsigned long long r;
      asm volatile("fma.rn.f32x2 %0, %1, %2, %3;"
                   : "=l"(r)
                   : "l"(pk2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]))), "l"(qu2), "l"(base2));
      upk2(r, y[2 * h], y[2 * h + 1]);
      if constexpr (!FULL) {
        y[2 * h] = (see >> i) & 1 ? y[2 * h] : -INFINITY;
        y[2 * h + 1] = (see >> i) & 2 ? y[2 * h + 1] : -INFINITY;
      }
    };
    auto finish = [&](int g, int h, const float (&y)[4]) {
      asm volatile("add.rn.f32x2 %0, %0, %1;" : "+l"(sum[h]) : "l"(pk2(y[2 * h], y[2 * h + 1])));
      asm volatile("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(p[2 * g + h]) : "f"(y[2 * h + 1]), "f"(y[2 * h]));
    };
    auto power = [](float y) {
      float r;
      asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
      return r;
    };
    exponents(0, 0, x[0]);
    exponents(0, 1, x[0]);
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      float(&now)[4] = x[g & 1];
      float(&next)[4] = x[(g + 1) & 1];
      float(&made)[4] = e[g & 1];
      float(&before)[4] = e[(g + 1) & 1];
      made[0] = power(now[0]);
      if (g < 7) exponents(g + 1, 0, next);
      made[1] = power(now[1]);
      if (g < 7) exponents(g + 1, 1, next);
      made[2] = power(now[2]);
      if (g > 0) finish(g - 1, 0, before);
      made[3] = power(now[3]);
      if (g > 0) finish(g - 1, 1, before);
    }
    finish(7, 0, e[1]);
    finish(7, 1, e[1]);
    float s0, s1, s2, s3;
    upk2(sum[0], s0, s1);
    upk2(sum[1], s2, s3);
    return (s0 + s1) + (s2 + s3);
  }
  // Brings the row to a larger reference where its sum asks for one (or it has
  // none); c: columns already stored, in units of 32.
  __device__ __forceinline__ void raise(const uint32_t (&w)[32], uint32_t see, int c, float sum, float& m, float& l,
                                        float& fix, unsigned long long& base2) const {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 32; ++i) top = (see >> i) & 1 ? fmaxf(top, __uint_as_float(w[i])) : top;
    top *= qu;
    const bool grow = m == -INFINITY ? top > m : sum > kGrow;
    const float f = grow ? ex2(m - (top - kRoom)) : 1.0f;  // 0 for a first reference
    if (grow) m = top - kRoom;
    const float base = m == -INFINITY ? 0.0f : -m;
    base2 = pk2(base, base);
    fix *= f;
    l *= f;
    tmem_store_wait();
#pragma unroll 1
    for (int k = 0; k < c; ++k) {
      uint32_t p[16];
      tmem_load16_now(p_at + 16 * k, p);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&p[i]));
        const __half2 z = __floats2half2_rn(y.x * f, y.y * f);
        p[i] = *reinterpret_cast<const uint32_t*>(&z);
      }
      tmem_store16(p_at + 16 * k, p);
    }
  }
  // FULL: every row of the warp sees every column.  Else 32 columns that no row sees
  // cost nothing, and those that every row sees nothing more.
  template <bool FULL>
  __device__ __forceinline__ void run(float& m, float& l, float& fix) const {
    const unsigned long long qu2 = pk2(qu, qu);
    const float base = m == -INFINITY ? 0.0f : -m;
    unsigned long long base2 = pk2(base, base);
    uint32_t v[2][32];
    tmem_load32(s_at, v[0]);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t(&w)[32] = v[c & 1];
      tmem_load_wait(v[c & 1]);
      if (c < 3) tmem_load32(s_at + 32 * c + 32, v[(c + 1) & 1]);
      uint32_t p[16];
      float sum = 0.0f;
      if constexpr (FULL) {
#pragma unroll 1
        for (bool again = false;; again = true) {
          sum = probabilities<true>(w, ~0u, qu2, base2, p);
          if (again || !__any_sync(0xffffffffu, sum > kGrow || m == -INFINITY)) break;
          raise(w, ~0u, c, sum, m, l, fix, base2);
        }
      } else {
        const uint32_t see = seen(c);
        const bool all = __all_sync(0xffffffffu, see == ~0u);
        if (!__any_sync(0xffffffffu, see != 0)) {
#pragma unroll
          for (int i = 0; i < 16; ++i) p[i] = 0;
        } else {
          bool rise = __any_sync(0xffffffffu, m == -INFINITY);
#pragma unroll 1
          for (bool again = false;; again = true) {
            if (rise) raise(w, see, c, sum, m, l, fix, base2);
            sum = all ? probabilities<true>(w, see, qu2, base2, p) : probabilities<false>(w, see, qu2, base2, p);
            rise = __any_sync(0xffffffffu, sum > kGrow);
            if (again || !rise) break;
          }
        }
      }
      l += sum;
      tmem_store16(p_at + 16 * c, p);
    }
  }
};

// Element of the head that column c of an 8-column chunk of K, Q and V holds:
// the order in which the codes fall out of a word.
template <int BITS>
__host__ __device__ constexpr int v_elem(int c) {
  return BITS == 4 ? (c >> 1) + 4 * (c & 1) : c;
}

// ---------------------------------------------------------------------------
// Queries of the sequences that belong to the launch: turned, rotated, scaled
// into base-2 scores, each row brought to [-2, 2) by its power of two and rounded
// to fp16, in the order of the keys' elements.  A launch of its own: done inside
// the attention kernel, whose warps then had nothing else to do, it took 30,000
// cycles for every 256 rows.
// ---------------------------------------------------------------------------
constexpr int kQueryTile = 8;  // tokens
template <int D>
struct QueryWork {
  __half* rows;    // [tokens, heads, D]
  float* factors;  // [tokens, heads]
};
template <int D>
__host__ __device__ __forceinline__ QueryWork<D> query_work_of(void* ws, int64_t tokens, int heads) {
  uint8_t* p = static_cast<uint8_t*>(ws) + kv_work_bytes<D, Prompt<D>::ROWS>(kCtas);
  QueryWork<D> w;
  w.rows = reinterpret_cast<__half*>(p);
  w.factors = reinterpret_cast<float*>(p + size_t(tokens) * heads * D * 2);
  return w;
}

template <int D, int BITS>
__global__ void __launch_bounds__(256) k_kv_query(const KvArgs a, const KvAttn t, FastDiv by_heads) {
  constexpr int LPV = KvLanes<D>::LPV;
  __shared__ __align__(16) float2 cs[kQueryTile * (D / 2)];
  __shared__ __align__(16) float factors[D];
  __shared__ uint64_t turns[D / 2];
  __shared__ int pos[kQueryTile], mine[kQueryTile];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t0 = int64_t(blockIdx.x) * kQueryTile;
  const int nt = int(min(int64_t(kQueryTile), a.tokens - t0));
  if (warp < nt) {
    const KvToken k = kv_token(a, t0 + warp, lane);
    if (lane == 0) {
      pos[warp] = int(k.pos);
      const int64_t rows = k.seq < 0 ? 0 : (min(int64_t(a.cu[k.seq + 1]), a.tokens) - a.cu[k.seq]) * t.group;
      mine[warp] = k.seq >= 0 && rows >= t.rows_lo && rows <= t.rows_hi;
    }
  }
  kv_turns(a, turns, threadIdx.x, blockDim.x);
  kv_factors<D, 0>(factors, a.k_signs, Prompt<D>::NORM * 1.4426950408889634f * t.scale);
  __syncthreads();
  for (int i = threadIdx.x; i < nt * a.n_freq; i += blockDim.x) {
    const int j = i / a.n_freq, f = i - j * a.n_freq;
    if (mine[j]) cs[i] = kv_angle_fast(a, turns, t0 + j, pos[j], f);
  }
  __syncthreads();
  const QueryWork<D> w = query_work_of<D>(t.ws, a.tokens, t.heads);
  const int l = threadIdx.x % LPV;
  const int vectors = nt * t.heads, per = blockDim.x / LPV;
  for (int v0 = blockIdx.y * per; v0 < vectors; v0 += gridDim.y * per) {
    const int v = v0 + int(threadIdx.x) / LPV;
    const int j = v < vectors ? int((__umulhi(uint32_t(v), by_heads.mul) + uint32_t(v)) >> by_heads.shr) : 0;
    const int head = v - j * t.heads;
    const bool live = v < vectors && mine[j];
    if (!__any_sync(0xffffffffu, live)) continue;
    float x[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = 0.0f;
    if (live) {
      const int64_t at = (t0 + j) * t.q_ts + head * t.q_hs;
      if (t.q_f32) {
#pragma unroll
        for (int c = 0; c < 4; ++c) kv_load8<true>(t.q, at + 8 * (c * LPV + l), x + 8 * c);
        if (a.n_freq > 0) kv_rope<D, true>(x, t.q, at, cs + j * a.n_freq, a.n_freq, a.interleaved, l);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) kv_load8<false>(t.q, at + 8 * (c * LPV + l), x + 8 * c);
        if (a.n_freq > 0) kv_rope<D, false>(x, t.q, at, cs + j * a.n_freq, a.n_freq, a.interleaved, l);
      }
      kv_times<D>(x, factors, l);
    }
    kv_hadamard<D>(x, l);
    float up, down;
    kv_row_power<D>(x, up, down);
    if (live) {
      const int64_t row = (t0 + j) * t.heads + head;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i0 = BITS == 4 ? e : 2 * e, i1 = BITS == 4 ? e + 4 : 2 * e + 1;
          const __half2 p = __floats2half2_rn(x[8 * c + i0] * down, x[8 * c + i1] * down);
          y[e] = *reinterpret_cast<const uint32_t*>(&p);
        }
        *reinterpret_cast<uint4*>(w.rows + row * D + 8 * (c * LPV + l)) = make_uint4(y[0], y[1], y[2], y[3]);
      }
      if (l == 0) w.factors[row] = up;
    }
  }
}

template <int D, int BITS>
__global__ void __launch_bounds__(kThreads, 1) k_kv_prompt(const KvArgs a, const KvAttn t, const FastDiv by_group) {
  using F = Prompt<D>;
  constexpr int VB = D * BITS / 8, CH = VB / 16;  // bytes and 16-byte pieces of a vector's codes
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + F::BARS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &bars->abort;
  __shared__ SegmentRing ring;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->kfull[i], 128);
      mbar_init(&bars->kempty[i], 1);
      mbar_init(&bars->vfull[i], 128);
      mbar_init(&bars->vempty[i], 1);
      mbar_init(&bars->q[i], 128);
      mbar_init(&bars->s[i], 1);
      mbar_init(&bars->p[i], 128);
      mbar_init(&bars->o[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&bars->sc[i], F::HALVES == 2 ? 128 : 256);
    for (int i = 0; i < kSegments; ++i) {
      mbar_init(&ring.full[i], 1);
      mbar_init(&ring.empty[i], 13);  // softmax and unpacking warps, and the issuing one
    }
    mbar_init(&bars->done, 1);
    bars->abort = 0;
    mbar_init_fence();
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars->tmem)),
                 "r"(uint32_t(F::COLS))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  __shared__ uint32_t v_neg[D / 32];  // a bit for each element of the result whose sign is flipped
  if (warp >= 4 && warp < 4 + D / 32) {
    const uint32_t b = __ballot_sync(0xffffffffu, a.v_signs != nullptr && __ldg(a.v_signs + 32 * (warp - 4) + lane) < 0);
    if (lane == 0) v_neg[warp - 4] = b;
  }
  if (warp == 0) plan_warp<F::ROWS>(a, t, bars, lane);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = bars->tmem;
  auto give_up = [&]() {
    atomicAdd(&g_wait_timeouts_kv, 1u);
    *abort = 1;
  };

  Follow w{&ring};
  int more = 1;
  if (warp < 4 * F::HALVES) {
    regs_more<F::SOFTMAX>();
    // the launch begins before the one ahead of it has ended: the queries, and
    // the workspace that is written here, are its
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // ---------------- softmax of half `hf`, a thread a row ----------------
    const int hf = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lane_at = tmem + (uint32_t(32 * (warp & 3)) << 16);
    const uint32_t s_at = lane_at + F::S_COL + 128 * hf, o_at = lane_at + F::O_COL + D * hf;
    const QueryWork<D> queries = query_work_of<D>(t.ws, a.tokens, t.heads);
    const KvWork work = kv_work_of<D, Prompt<D>::ROWS>(t.ws, gridDim.x);
    uint32_t ns = 0, no = 0;  // score units and outputs seen so far
    uint32_t kv0 = 0;         // units converted before this segment
    KvPart open;
    open.first = -1;
    while (!__any_sync(0xffffffffu, *abort) && (more = w.next(lane)) > 0) {
      const Segment& g = w.seg();
      const Half f = g.half[hf];
      const int ub = g.ub, row = g.row0 + 128 * hf + r;
      const bool mine = r < f.rows;
      const int tok = mine ? row / t.group : 0;
      const int head = g.h * t.group + (mine ? row - tok * t.group : 0);
      float m = -INFINITY, l = 0.0f;
      uint32_t ve = 0;  // exponent of the power of two that O is relative to; 0: none yet
      bool ok = true;
      if (f.js < f.je) {
        // the half's queries, a row's 16-byte pieces to their swizzled places
        constexpr int PIECES = D / 8;
#pragma unroll 4
        for (int k = 0; k < PIECES; ++k) {
          const int qr = (k * 128 + r) / PIECES, c = r % PIECES;
          const int row_q = g.row0 + 128 * hf + qr;
          const int tk = int((__umulhi(uint32_t(row_q), by_group.mul) + uint32_t(row_q)) >> by_group.shr);
          const bool there = qr < f.rows;
          const int64_t src = there ? (g.t0 + tk) * t.heads + g.h * t.group + (row_q - tk * t.group) : 0;
          const uint32_t dst = smem_u32(smem) + F::Q + hf * F::TILE + (c / 8) * 16384 + qr * 128 + ((c % 8) ^ (qr & 7)) * 16;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(queries.rows + src * D + 8 * c),
                       "r"(there ? 16 : 0)
                       : "memory");
        }
        const float qe = mine ? queries.factors[(g.t0 + tok) * t.heads + head] : 1.0f;
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        mbar_arrive(&bars->q[hf]);
        const int64_t pos = g.pos0 + tok;
        const int64_t hi = mine ? (t.causal ? min(g.hi, pos + 1) : g.hi) : 0;
        const int64_t lo = t.window > 0 ? pos - t.window + 1 : 0;

        for (int j = f.js; j < f.je && ok; ++j) {
          const uint32_t kv = kv0 + uint32_t(j - ub);
          const uint8_t* scp = smem + F::SC + (kv & 3) * F::SC_STAGE;
          ok = mbar_wait(&bars->sc[kv & 3], (kv >> 2) & 1u) && mbar_wait(&bars->s[hf], ns & 1u);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          ++ns;
          fence_after();
          const uint4 there = *reinterpret_cast<const uint4*>(scp);
          const uint32_t ve_before = ve;
          uint4 power = *reinterpret_cast<const uint4*>(scp + 16);  // of keys and of values; whether a position has its own
          if (F::HALVES == 2) power.w = power.z;                    // the same warps unpack both
          const float qu = qe * __uint_as_float(power.x);
          const bool apart = (power.z | power.w) != 0;
          const int64_t p0 = int64_t(j) * kKeys;
          const bool full = !apart && p0 >= f.lo_max && p0 + kKeys <= f.hi_min && (there.x & there.y & there.z & there.w) == ~0u;
          // columns [c_lo, c_hi) are this row's
          const int c_lo = int(max(int64_t(0), min(int64_t(128), lo - p0)));
          const int c_hi = int(max(int64_t(0), min(int64_t(128), hi - p0)));
          float fix = 1.0f;
          const UnitSoftmax unit{s_at, s_at, there, c_lo, c_hi, qu};
          if (full) {
            ve = power.y;
            unit.run<true>(m, l, fix);
          } else if (!apart) {
            if (c_lo < c_hi) ve = power.y;  // a row that sees nothing here keeps its own
            unit.run<false>(m, l, fix);
          } else {
            const UnitSoftmax::Row row = UnitSoftmax::run_apart(unit, smem + F::OWN + (kv & 3) * F::OWN_STAGE, qe,
                                                                power, m, l, ve);
            m = row.m, l = row.l, fix = row.fix, ve = row.ve;
          }
          const int finer = ve_before != 0 ? int(ve_before) - int(ve) : 0;
          if (j > f.js && __any_sync(0xffffffffu, fix != 1.0f || finer != 0)) {
            // the product of the unit before has to be in O
            ok = mbar_wait(&bars->o[hf], (no - 1) & 1u);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            fence_after();
            if (__any_sync(0xffffffffu, abs(finer) > 24)) {
              const UnitSoftmax::Row row = UnitSoftmax::fit<D>(o_at, s_at, fix, finer, ve);
              fix = row.fix, ve = row.ve;
            } else {
              fix *= __uint_as_float(uint32_t(127 + finer) << 23);
            }
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t v[32], x[16];
              tmem_load32_now(o_at + 32 * c, v);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(v[16 * k + i]) * fix);
                tmem_store16(o_at + 32 * c + 16 * k, x);
              }
            }
          }
          ++no;
          tmem_store_wait();
          fence_before();
          mbar_arrive(&bars->p[hf]);
        }
        if (ok) ok = mbar_wait(&bars->o[hf], (no - 1) & 1u);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          if (lane == 0) give_up();
          break;
        }
        fence_after();
      }
      // ---------------- the half's result ----------------
      const bool any = f.js < f.je;
      const size_t slot_row = (2 * size_t(blockIdx.x) + (g.begins ? 1 : 0)) * Prompt<D>::ROWS + 128 * hf + r;
      const float up = __uint_as_float(ve << 23);
      const float inv = l == 0.0f ? 0.0f : F::NORM / l * up;
      if (f.rows > 0) {  // by the whole warp: tensor memory is read together
        if (g.whole) {
          constexpr int N = D / 64;  // the transform's last stages join the runs of 64 elements
#pragma unroll 1
          for (int b = 0; b < N; ++b) {
            float x[64];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t u[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) x[32 * c + i] = 0.0f;
              if (any) {
#pragma unroll
                for (int e = 0; e < N; ++e) {
                  const float f = __popc(b & e) & 1 ? -inv : inv;
                  tmem_load32_now(o_at + 64 * e + 32 * c, u);
#pragma unroll
                  for (int i = 0; i < 32; ++i) {
                    float& y = x[32 * c + 8 * (i / 8) + v_elem<BITS>(i % 8)];
                    y = fmaf(__uint_as_float(u[i]), f, y);
                  }
                }
              }
            }
            reg_stages<64, 0, 6>(x);
            if (mine) {
#pragma unroll
              for (int i = 0; i < 64; ++i)
                x[i] = __uint_as_float(__float_as_uint(x[i]) ^ ((v_neg[2 * b + i / 32] << (31 - i % 32)) & 0x80000000u));
              const int64_t at = (g.t0 + tok) * t.o_ts + head * t.o_hs + 64 * b;
              if (t.o_f32) {
#pragma unroll
                for (int i = 0; i < 64; i += 8) kv_store8<true>(t.out, at + i, x + i);
              } else if (t.wide) {  // whole 32-byte sectors
#pragma unroll
                for (int i = 0; i < 64; i += 16)
                  st_stream_v8(static_cast<__nv_bfloat16*>(t.out) + at + i, f32_to_bf16x2(x[i], x[i + 1]),
                               f32_to_bf16x2(x[i + 2], x[i + 3]), f32_to_bf16x2(x[i + 4], x[i + 5]),
                               f32_to_bf16x2(x[i + 6], x[i + 7]), f32_to_bf16x2(x[i + 8], x[i + 9]),
                               f32_to_bf16x2(x[i + 10], x[i + 11]), f32_to_bf16x2(x[i + 12], x[i + 13]),
                               f32_to_bf16x2(x[i + 14], x[i + 15]));
              } else {
#pragma unroll
                for (int i = 0; i < 64; i += 8) kv_store8<false>(t.out, at + i, x + i);
              }
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t u[32];
            if (any) tmem_load32_now(o_at + 32 * c, u);
            float x[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) x[8 * (i / 8) + v_elem<BITS>(i % 8)] = any ? __uint_as_float(u[i]) * up : 0.0f;
            if (mine) {
#pragma unroll
              for (int i = 0; i < 32; i += 8) kv_store8<true>(work.rows, slot_row * D + 32 * c + i, x + i);
            }
          }
          if (mine) work.ms[slot_row] = make_float2(m, l);
        }
      }
      if (g.begins && !g.whole) {
        open.first = blockIdx.x;
        open.last = g.last;
        open.rows = g.nr;
        open.row0 = g.row0;
        open.t0 = g.t0;
        open.h = g.h;
        open.pad = 0;
      }
      fence_before();
      kv0 += uint32_t(g.ue - g.ub);
    }
    if (more < 0 && lane == 0) give_up();
    if (threadIdx.x == 0) work.part[2 * blockIdx.x + 1] = open;
  } else if (warp < 12) {
    // ---------------- codes to operands, a thread a position ----------------
    regs_less<F::UNPACK>();
    const int i = threadIdx.x & 127;
    // keys and values by the same threads, or (heads of 256) the values by warps 4-7:
    // 1,024 tokens on 12,000 (32 heads on 8) take 730 us with 8 bits and 695 with 4 (706 and
    // 660, with one group 1,010 and 674, before positions had powers of two of their own)
    auto unpack = [&](auto keys_too, auto values_too) {
      constexpr bool KEYS = decltype(keys_too)::value, VALUES = decltype(values_too)::value;
      uint32_t kv = 0;
      bool ok = true;
      // The group's four warps meet once a unit.  The barrier has no limit of its own, so
      // a warp one of whose waits (which have a limit) has run out comes to the next meeting
      // all the same, says so there, and all of them leave.
      auto meet = [&]() { asm volatile("bar.sync %0, 128;" ::"n"(KEYS ? 3 : 4) : "memory"); };
      constexpr uint32_t kFailed = ~0u;  // in the place of a warp's largest scale
      bool told = false;                 // one of them leaves
      while (ok && !told && (more = w.next(lane)) > 0) {
        const int ub = w.seg().ub, ue = w.seg().ue, h = w.seg().h;
        const int64_t hi = w.seg().hi;
        const int32_t* const pages = a.table + int64_t(w.seg().s) * a.ld_table;
        uint4 kr[CH], vr[CH];
        float ksc = 0.0f, vsc = 0.0f;
        int vex = 0;  // exponent of the largest value scale that the unit's values are relative to
        bool in = false;
        // the page of this thread's position in unit j (-1: there is none), and its vector in that page
        auto page_of = [&](int j) {
          const int64_t p = int64_t(j) * kKeys + i;
          int page = -1;
          if (j < ue && p < hi) load4(page, pages + (p >> a.log_page));
          return page;
        };
        auto vector_of = [&](int j, int page) {
          const int64_t p = int64_t(j) * kKeys + i;
          in = page >= 0 && page < a.pages;
          return (((int64_t(page) * a.hk + h) << a.log_page) + (p & ((int64_t(1) << a.log_page) - 1)));
        };
        auto load = [&](const uint8_t* codes, int64_t vec, uint4 (&x)[CH]) {
#pragma unroll
          for (int k = 0; k < CH; ++k) {
            x[k] = make_uint4(0, 0, 0, 0);
            if (in) load16(x[k], codes + vec * VB + 16 * k);
          }
        };
        auto load_scales = [&](int64_t vec) {
          ksc = vsc = 0.0f;
          if (in) {
            if constexpr (KEYS) load4(ksc, a.k_scales + vec);
            load4(vsc, a.v_scales + vec);
          }
        };
        int64_t vec = 0;
        if (ub < ue) {
          vec = vector_of(ub, page_of(ub));
          load_scales(vec);
          if constexpr (KEYS) load(a.k_codes, vec, kr);
          if constexpr (VALUES) load(a.v_codes, vec, vr);
        }
        for (int j = ub; j < ue; ++j, ++kv) {
          const uint32_t st = kv % F::STAGES, round = kv / F::STAGES;
          const int page = page_of(j + 1);
          // The scales are folded into the operands, with one rounding: a product
          // with a scale in two parts, hi and the rest.  Keys are relative to a
          // power of two of the unit's largest scale, so that fp16 holds them, values
          // to one of the largest scale of a unit before while that of this one is at most
          // 2^3 times as large and no less than 2^-6 of it (else its own, and O is brought to
          // it).  Codes times scales then stay below 2^15 and keep 11 bits (bf16 values cost
          // the result 2^-8 of each, 0.0029 in place of 0.0017 in all).  A position whose
          // scale is smaller by more than 2^kSpread takes its own power of two, which the
          // softmax multiplies in (UnitSoftmax::run_apart): else one large scale, hidden or
          // not, would leave the others no digits.  A position whose scale is not finite
          // becomes NaN in its scores, and only there.
          uint32_t* const tops = reinterpret_cast<uint32_t*>(smem + F::TS + (kv & 1) * 32);
          uint8_t* const scp = smem + F::SC + (kv & 3) * F::SC_STAGE;
          uint8_t* const apart = scp + (KEYS ? 24 : 28) + (warp & 3);  // whether a position of this warp's is
          const bool k_fine = (__float_as_uint(ksc) & 0x7f800000u) != 0x7f800000u;
          const bool v_fine = (__float_as_uint(vsc) & 0x7f800000u) != 0x7f800000u;
          {
            const uint32_t top = KEYS ? __reduce_max_sync(0xffffffffu, k_fine ? __float_as_uint(ksc) & 0x7fffffffu : 0u) : 0u;
            const uint32_t vtop = VALUES ? __reduce_max_sync(0xffffffffu, v_fine ? __float_as_uint(vsc) & 0x7fffffffu : 0u) : 0u;
            const uint32_t b = __ballot_sync(0xffffffffu, in);
            if (lane == 0) {
              *apart = 0;
              if (KEYS) tops[warp & 3] = ok ? top : kFailed, reinterpret_cast<uint32_t*>(scp)[warp & 3] = b;
              if (VALUES) tops[4 + (warp & 3)] = ok ? vtop : kFailed;
            }
          }
          meet();
          int kex = 0;  // exponent of the unit's largest key scale
          if constexpr (KEYS) {
            const uint4 all = *reinterpret_cast<const uint4*>(tops);
            kex = int(max(8u, max(max(all.x, all.y), max(all.z, all.w)) >> 23));
            told = kex > 255;
            if (i == 0) *reinterpret_cast<uint32_t*>(scp + 16) = uint32_t(kex - kKeyBits) << 23;
          }
          if constexpr (VALUES) {
            const uint4 all = *reinterpret_cast<const uint4*>(tops + 4);
            const uint32_t vtop = max(max(all.x, all.y), max(all.z, all.w)) >> 23;
            told = vtop > 255;
            const int vx = max(8, int(vtop));
            if (j == ub || vx > vex + 3 || (vtop != 0 && vx < vex - 6)) vex = vx;
            if (i == 0) *reinterpret_cast<uint32_t*>(scp + 20) = uint32_t(vex - kValueBits);
          }
          if (told) break;
          const int k_own = int(__float_as_uint(ksc) >> 23) & 255, v_own = int(__float_as_uint(vsc) >> 23) & 255;
          const bool k_apart = KEYS && k_own + kSpread < kex && ksc != 0.0f;
          const bool v_apart = VALUES && v_own + kSpread < vex && vsc != 0.0f;
          const int ke = k_apart ? max(1, k_own) : kex - kKeyBits, ve = v_apart ? max(1, v_own) : vex - kValueBits;
          uint32_t k_hi, k_lo, v_hi, v_lo;
          {
            auto inverse = [](int e) { return __uint_as_float(e == 254 ? 0x00400000u : uint32_t(254 - e) << 23); };
            const float sc = v_fine ? ksc * inverse(ke) : __uint_as_float(0x7fc00000u);
            const __half hi = __float2half_rn(sc), lo = __float2half_rn(sc - __half2float(hi));
            k_hi = uint32_t(__half_as_ushort(hi)) * 0x10001u;
            k_lo = uint32_t(__half_as_ushort(lo)) * 0x10001u;
            const float vz = v_fine ? vsc * inverse(ve) : 0.0f;
            const __half vh = __float2half_rn(vz), vl = __float2half_rn(vz - __half2float(vh));
            v_hi = uint32_t(__half_as_ushort(vh)) * 0x10001u;
            v_lo = uint32_t(__half_as_ushort(vl)) * 0x10001u;
          }
          // tells the softmax; the rings of four units are free here, as it is done with the unit
          // before the one that the last wait was for
          auto tell = [&]() {
            if (__any_sync(0xffffffffu, k_apart || v_apart)) {
              uint8_t* const own = smem + F::OWN + (kv & 3) * F::OWN_STAGE + i;
              if (KEYS) own[0] = k_apart ? uint8_t(ke) : 0;
              if (VALUES) own[kKeys] = v_apart ? uint8_t(ve) : 0;
              if (lane == 0) *apart = 1;
            }
            mbar_arrive(&bars->sc[kv & 3]);
          };
          if constexpr (!KEYS) tell();
          ok = ok && !*abort && (round == 0 || mbar_wait(KEYS ? &bars->kempty[st] : &bars->vempty[st], (round - 1) & 1u));
          ok = __all_sync(0xffffffffu, ok);
          auto store = [&](uint8_t* tile, const uint4 (&x)[CH], uint32_t s_hi, uint32_t s_lo) {
            uint8_t* row = tile + i * 128;
            const int turn = i & 7;
#pragma unroll
            for (int k = 0; k < CH; ++k) {
              const uint32_t wd[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
              constexpr int OUT = 128 / (8 * BITS);  // 16-byte chunks of operand from 16 bytes of codes
#pragma unroll
              for (int e = 0; e < OUT; ++e) {
                uint32_t o[4];
                if constexpr (BITS == 4) {
                  half_of4(wd[e], o);
                } else {
                  half_of8(wd[2 * e], o[0], o[1]);
                  half_of8(wd[2 * e + 1], o[2], o[3]);
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) o[y] = hfma2(o[y], s_hi, hfma2(o[y], s_lo, 0x80008000u));
                const int c = OUT * k + e;  // chunk of the position's row
                *reinterpret_cast<uint4*>(row + (c / 8) * 16384 + ((c % 8) ^ turn) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
              }
            }
          };
          if constexpr (KEYS) {
            store(smem + F::K + st * F::TILE, kr, k_hi, k_lo);
            tell();
            fence_proxy_async_smem();
            mbar_arrive(&bars->kfull[st]);
          }
          // the next unit's codes are on their way while this one's are waited for and unpacked
          vec = vector_of(j + 1, page);
          load_scales(vec);
          if constexpr (KEYS) load(a.k_codes, vec, kr);
          if constexpr (VALUES) {
            if constexpr (KEYS) {
              ok = round == 0 || mbar_wait(&bars->vempty[st], (round - 1) & 1u);
              ok = __all_sync(0xffffffffu, ok);
            }
            store(smem + F::V + st * F::TILE, vr, v_hi, v_lo);
            fence_proxy_async_smem();
            mbar_arrive(&bars->vfull[st]);
            load(a.v_codes, vec, vr);
          }
        }
      }
      if ((!ok || more < 0) && !*abort) give_up();
      if (!told) {  // no unit is left for this warp: the others may be at the meeting of one
        if (lane == 0 && (!ok || more < 0))
          reinterpret_cast<uint32_t*>(smem + F::TS + (kv & 1) * 32)[(KEYS ? 0 : 4) + (warp & 3)] = kFailed;
        meet();
      }
    };
    if constexpr (F::HALVES == 2) unpack(std::true_type{}, std::true_type{});
    else if (warp < 8) unpack(std::false_type{}, std::true_type{});
    else unpack(std::true_type{}, std::false_type{});
  } else {
    regs_less<F::OTHER>();
    if (warp == 12) {
      // ---------------- products: the warp waits, one thread issues ----------------
      constexpr uint32_t id_s = instr_desc(128, false), id_o = instr_desc(D, true);
      const uint32_t base = smem_u32(smem);
      // descriptors of the tiles: the upper word is the same for all, the lower one holds the address
      const uint64_t dk = desc_sw128(base, 16, 1024), dv = desc_sw128(base + F::V, 16384, 1024);
      const uint32_t k_hi = uint32_t(dk >> 32), v_hi = uint32_t(dv >> 32);
      const uint32_t q_lo = uint32_t(dk), k_lo = q_lo + (F::K >> 4), v_lo = uint32_t(dv);
      uint32_t nq[2] = {0, 0}, np[2] = {0, 0};
      uint32_t kv0 = 0;
      bool ok = true;
      while (ok && (more = w.next(lane)) > 0) {
        const int ub = w.seg().ub, ue = w.seg().ue;
        const int js[2] = {w.seg().half[0].js, w.seg().half[1].js}, je[2] = {w.seg().half[0].je, w.seg().half[1].je};
        for (int j = ub - 1; j < ue && ok && ub < ue; ++j) {
          const uint32_t kv = kv0 + uint32_t(j - ub);  // unit j (j = ub - 1: none)
          const uint32_t kn = kv + 1;
          bool have_v = false, have_k = false;
#pragma unroll
          for (int hf = 0; hf < F::HALVES; ++hf) {
            if (ok && j >= js[hf] && j < je[hf]) {
              if (!have_v) ok = mbar_wait(&bars->vfull[kv % F::STAGES], (kv / F::STAGES) & 1u);
              have_v = true;
              ok = ok && !*abort && mbar_wait(&bars->p[hf], np[hf] & 1u);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              ++np[hf];
              fence_after();
              if (elect_one()) {
                const uint32_t lo = v_lo + (kv % F::STAGES) * (F::TILE >> 4);
                const bool add = j > js[hf];
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                  mma_ts(tmem + F::O_COL + D * hf, tmem + F::S_COL + 128 * hf + 8 * k, lo + k * 128, v_hi, id_o, k > 0 || add);
                commit(&bars->o[hf]);
                if (F::HALVES == 1) commit(&bars->vempty[0]);  // ahead of the next scores: it is the only stage
              }
            }
            if (ok && j + 1 >= js[hf] && j + 1 < je[hf]) {
              if (!have_k) ok = mbar_wait(&bars->kfull[kn % F::STAGES], (kn / F::STAGES) & 1u);
              have_k = true;
              if (ok && j + 1 == js[hf]) ok = mbar_wait(&bars->q[hf], nq[hf]++ & 1u);
              ok = __all_sync(0xffffffffu, ok && !*abort);
              if (!ok) break;
              fence_after();
              if (elect_one()) {
                const uint32_t lo_q = q_lo + hf * (F::TILE >> 4), lo_k = k_lo + (kn % F::STAGES) * (F::TILE >> 4);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                  mma_ss(tmem + F::S_COL + 128 * hf, lo_q + (k / 4) * 1024 + 2 * (k % 4), lo_k + (k / 4) * 1024 + 2 * (k % 4),
                         k_hi, id_s, k > 0);
                commit(&bars->s[hf]);
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          if (elect_one()) {
            if (F::HALVES == 2 && j >= ub) commit(&bars->vempty[kv % F::STAGES]);
            if (j + 1 < ue) commit(&bars->kempty[kn % F::STAGES]);
          }
          __syncwarp();
        }
        kv0 += uint32_t(ue - ub);
      }
      if ((!ok || more < 0) && !*abort) give_up();
      // every product has ended before tensor memory is given back
      if (elect_one()) commit(&bars->done);
      if (!mbar_wait(&bars->done, 0u)) atomicAdd(&g_wait_timeouts_kv, 1u);
    } else if (warp == 13 && lane == 0) {
      if (!walk<F::ROWS>(a, t, bars, &ring, abort)) give_up();
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == 12) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(uint32_t(F::COLS)) : "memory");
  }
}

template <int D, int BITS>
cudaError_t prepare(const KvArgs& a, const KvAttn& t, cudaStream_t st) {
  const int64_t tiles = (a.tokens + kQueryTile - 1) / kQueryTile;
  const int64_t passes = (int64_t(kQueryTile) * t.heads * (D / 32) + 255) / 256;
  // heads are dealt to several CTAs while the tokens alone do not fill the GPU four times
  const unsigned y = unsigned(std::max<int64_t>(1, std::min(passes, 4 * 148 * 4 / tiles)));
  k_kv_query<D, BITS><<<dim3(unsigned(tiles), y), 256, 0, st>>>(a, t, make_fastdiv(uint32_t(t.heads)));
  return cudaGetLastError();
}

template <int D, int BITS>
cudaError_t go(const KvArgs& a, const KvAttn& t, cudaStream_t st) {
  constexpr int bytes = Prompt<D>::BYTES;
  auto* kernel = k_kv_prompt<D, BITS>;
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
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, a, t, make_fastdiv(uint32_t(t.group)));
  if (e != cudaSuccess) return e;
  return launch_kv_join<D, Prompt<D>::ROWS, 8>(a, t, kCtas, st);
}

}  // namespace

size_t kv_prompt_bytes(int64_t tokens, int heads, int head_dim) {
  const size_t queries = size_t(tokens) * heads * (size_t(head_dim) * 2 + 4);
  const size_t parts = head_dim == 64    ? kv_work_bytes<64, Prompt<64>::ROWS>(kCtas)
                       : head_dim == 128 ? kv_work_bytes<128, Prompt<128>::ROWS>(kCtas)
                                         : kv_work_bytes<256, Prompt<256>::ROWS>(kCtas);
  return parts + queries;
}

// Two launches; nothing else may write the workspace's part for queries between them.
cudaError_t launch_kv_prompt_queries(const KvArgs& a, const KvAttn& t, cudaStream_t st) {
  if (a.head_dim == 64) return a.bits == 4 ? prepare<64, 4>(a, t, st) : prepare<64, 8>(a, t, st);
  if (a.head_dim == 128) return a.bits == 4 ? prepare<128, 4>(a, t, st) : prepare<128, 8>(a, t, st);
  return a.bits == 4 ? prepare<256, 4>(a, t, st) : prepare<256, 8>(a, t, st);
}
cudaError_t launch_kv_prompt(const KvArgs& a, const KvAttn& t, cudaStream_t st) {
  if (a.head_dim == 64) return a.bits == 4 ? go<64, 4>(a, t, st) : go<64, 8>(a, t, st);
  if (a.head_dim == 128) return a.bits == 4 ? go<128, 4>(a, t, st) : go<128, 8>(a, t, st);
  return a.bits == 4 ? go<256, 4>(a, t, st) : go<256, 8>(a, t, st);
}

cudaError_t wait_timeouts_kv(unsigned long long* count, bool reset) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_wait_timeouts_kv, sizeof v);
  if (e != cudaSuccess) return e;
  *count += v;
  if (reset && v != 0) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_wait_timeouts_kv, &zero, sizeof zero);
  }
  return e;
}

}  // namespace hit

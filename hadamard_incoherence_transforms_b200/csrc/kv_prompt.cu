// Attention over the rotated cache for many query rows (chunks of prompts):
// bound by the matrix products.
//
// A CTA (one per SM) takes an equal share of the list of (sequence, key/value
// head, 256 query rows) x 128 positions units.  Roles:
//   warps 0-3, 4-7  softmax of the upper and of the lower 128 query rows, a
//                   thread a row, its scores in tensor memory;
//   warps 8-11      codes to fp16 keys and bf16 values in shared memory (128-byte
//                   swizzle), a two-stage ring each, the next unit's codes on
//                   their way in registers;
//   warp 12         one thread issues the products: S = Q K^T (fp16), O += P V
//                   (bf16, P read from tensor memory where it replaced S).
// The two halves alternate: while one half's softmax runs, the tensor cores
// work on the other's products.  Key and value units are converted once for
// both, their scales folded in with one rounding (2^-11 of a key, 2^-8 of a
// value: half the work of the softmax roles went into scales otherwise, see
// UnitSoftmax for what is left of it).
#include "kv_codes.cuh"
#include "kv_split.cuh"

#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

namespace hit {

__device__ unsigned int g_wait_timeouts_kv = 0;

namespace {

constexpr int kRows = 256;      // query rows of a unit
constexpr int kKeys = 128;      // positions of a unit
constexpr int kThreads = 16 * 32;  // warps 13-15 are idle: registers are dealt out to groups of four warps
constexpr int kCtas = 148;
constexpr float kGrow = 65536.0f;  // sum of 32 probabilities above which a row gets a new reference

template <int D>
struct Prompt {
  static constexpr int BLK = D / 64;             // 64-element column blocks of an operand
  static constexpr int TILE = BLK * 128 * 128;   // 128 vectors of D 16-bit elements
  static constexpr int Q = 0, K = 2 * TILE, V = 4 * TILE, SC = 6 * TILE;
  // ring of four units: which positions exist (128 bits), the power of two of the key scales
  static constexpr int SC_STAGE = 32;
  static constexpr int ES = SC + 4 * SC_STAGE;   // 256 row factors
  static constexpr int TS = ES + kRows * 4;      // two units' scales, and the largest key scale of each warp
  static constexpr int TS_STAGE = 2 * 128 * 4 + 16;
  static constexpr int BARS = TS + 2 * TS_STAGE;
  static constexpr int BYTES = BARS + 512 + 1024;
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
static_assert(sizeof(Bars) <= 512, "barrier block");

// ---------------------------------------------------------------------------
// The list of units.
// ---------------------------------------------------------------------------
// Units of row tile rt of a sequence: [first, first + count).
__device__ __forceinline__ void tile_units(const KvAttn& t, const KvSeq& q, int rt, int& first, int& count) {
  const int64_t rows = int64_t(q.n) * t.group;
  const int64_t r0 = int64_t(rt) * kRows, r1 = min(rows, r0 + kRows);
  const int64_t i0 = r0 / t.group, i1 = (r1 - 1) / t.group;
  const int64_t hi = t.causal ? max(int64_t(0), min(q.hi, q.pos0 + i1 + 1)) : q.hi;
  const int64_t lo = t.window > 0 ? min(hi, max(int64_t(0), q.pos0 + i0 - t.window + 1)) : 0;
  first = int(lo / kKeys);
  count = max(1, int((hi + kKeys - 1) / kKeys) - first);
}

// Units of a sequence for one key/value head, found by a warp.
__device__ __forceinline__ int64_t head_units_warp(const KvAttn& t, const KvSeq& q, int lane) {
  int64_t sum = 0;
  for (int rt = lane; rt < q.row_tiles; rt += 32) {
    int f, c;
    tile_units(t, q, rt, f, c);
    sum += c;
  }
#pragma unroll
  for (int b = 16; b; b >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, b);
  return sum;
}

// Units of sequences s0 .. s0 + 31, one to a lane.
__device__ __forceinline__ int64_t chunk_units(const KvArgs& a, const KvAttn& t, int s0, int lane) {
  int64_t w = 0;
  bool big = false;
  if (s0 + lane < a.seqs) {
    const KvSeq q = kv_seq<kRows, kKeys>(a, t, s0 + lane);
    if (kv_mine(t, q)) {
      big = q.row_tiles > 4;
      for (int rt = 0; rt < q.row_tiles && !big; ++rt) {
        int f, c;
        tile_units(t, q, rt, f, c);
        w += c;
      }
    }
  }
  for (uint32_t m = __ballot_sync(0xffffffffu, big); m; m &= m - 1) {
    const int k = __ffs(m) - 1;
    const int64_t v = head_units_warp(t, kv_seq<kRows, kKeys>(a, t, s0 + k), lane);
    if (lane == k) w = v;
  }
  return w * a.hk;
}

// One warp finds the CTA's share and where it begins.
__device__ __forceinline__ void plan_warp(const KvArgs& a, const KvAttn& t, Bars* b, int lane) {
  int64_t total = 0;
  for (int s0 = 0; s0 < a.seqs; s0 += 32) total += chunk_units(a, t, s0, lane);
#pragma unroll
  for (int i = 16; i; i >>= 1) total += __shfl_xor_sync(0xffffffffu, total, i);
  const int64_t ctas = max(int64_t(1), min(int64_t(gridDim.x), (total + 1) / 2));
  const int64_t c = blockIdx.x;
  const int64_t u0 = c < ctas ? c * total / ctas : total, u1 = c < ctas ? (c + 1) * total / ctas : total;
  int seq = a.seqs;
  int64_t base = 0;
  if (u0 < u1) {
    for (int s0 = 0; s0 < a.seqs; s0 += 32) {
      const int64_t v = chunk_units(a, t, s0, lane);
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
    const KvSeq q = kv_seq<kRows, kKeys>(a, t, seq);
    const int64_t per = head_units_warp(t, q, lane);
    h = int((u0 - base) / per);
    int64_t r = u0 - base - h * per;
    for (int r0 = 0; r0 < q.row_tiles; r0 += 32) {
      int f, v = 0;
      if (r0 + lane < q.row_tiles) tile_units(t, q, r0 + lane, f, v);
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
// the bounds inside which every row sees everything.
struct Half {
  int rows, js, je;
  int64_t lo_max, hi_min;
};
// A CTA's part of one (sequence, head, row tile); every role walks the same ones.
struct Segment {
  KvSeq q;
  int s, h, rt;
  int row0, nr;
  int first, count;      // units of the row tile
  int x0, x1;            // of them, this CTA's
  int ub, ue;            // units that either half needs
  Half half[2];
};
struct Walk {
  Segment g;
  int64_t left;
  __device__ __forceinline__ void start(const Bars* b) {
    left = b->units;
    g.s = b->seq;
    g.h = b->h;
    g.rt = b->rt;
    g.x0 = b->x0;
  }
  __device__ __forceinline__ void fill(const KvArgs& a, const KvAttn& t) {
    tile_units(t, g.q, g.rt, g.first, g.count);
    g.x1 = int(min(int64_t(g.count), g.x0 + left));
    g.row0 = g.rt * kRows;
    g.nr = int(min(int64_t(kRows), int64_t(g.q.n) * t.group - g.row0));
    g.ub = INT32_MAX;
    g.ue = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      Half& f = g.half[k];
      f.rows = min(128, max(0, g.nr - 128 * k));
      f.js = f.je = 0;
      f.lo_max = f.hi_min = 0;
      if (f.rows > 0) {
        const int64_t i0 = (g.row0 + 128 * k) / t.group, i1 = (g.row0 + 128 * k + f.rows - 1) / t.group;
        const int64_t hi = t.causal ? max(int64_t(0), min(g.q.hi, g.q.pos0 + i1 + 1)) : g.q.hi;
        const int64_t lo = t.window > 0 ? min(hi, max(int64_t(0), g.q.pos0 + i0 - t.window + 1)) : 0;
        f.hi_min = t.causal ? min(g.q.hi, g.q.pos0 + i0 + 1) : g.q.hi;
        f.lo_max = t.window > 0 ? g.q.pos0 + i1 - t.window + 1 : 0;
        f.js = max(g.first + g.x0, int(lo / kKeys));
        f.je = min(g.first + g.x1, int((hi + kKeys - 1) / kKeys));
        if (f.js < f.je) {
          g.ub = min(g.ub, f.js);
          g.ue = max(g.ue, f.je);
        } else {
          f.je = f.js;
        }
      }
    }
    if (g.ub > g.ue) g.ub = g.ue = 0;
  }
  __device__ __forceinline__ bool begin(const KvArgs& a, const KvAttn& t) {
    if (left <= 0) return false;
    g.q = kv_seq<kRows, kKeys>(a, t, g.s);
    fill(a, t);
    return true;
  }
  __device__ __forceinline__ bool next(const KvArgs& a, const KvAttn& t) {
    left -= g.x1 - g.x0;
    if (left <= 0) return false;
    g.x0 = 0;
    if (++g.rt == g.q.row_tiles) {
      g.rt = 0;
      if (++g.h == a.hk) {
        g.h = 0;
        do {
          g.q = kv_seq<kRows, kKeys>(a, t, ++g.s);
        } while (g.q.n == 0 || !kv_mine(t, g.q));
      }
    }
    fill(a, t);
    return true;
  }
};

// ---------------------------------------------------------------------------
// tcgen05
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return uint64_t((addr >> 4) & 0x3fff) | (uint64_t((lbo >> 4) & 0x3fff) << 16) | (uint64_t((sbo >> 4) & 0x3fff) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// fp32 accumulator; A and B both fp16 or both bf16; A K-major, M = 128
__host__ __device__ constexpr uint32_t instr_desc(bool bf16, int n, bool b_mn_major) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (uint32_t(b_mn_major) << 16) | (uint32_t(n >> 3) << 17) |
         (uint32_t(128 >> 4) << 24);
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
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Loads that stay where they are written.
__device__ __forceinline__ void load16(uint4& x, const void* p) {
  asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p));
}
__device__ __forceinline__ void load4(float& x, const float* p) {
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(x) : "l"(p));
}
// Registers of a group of four warps (all four run it).  The kernel starts with
// 128 a thread; 2 x 176 + 112 + 48 are the same 512.
template <int N>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_less() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// {a0, a1} += {b0, b1}
__device__ __forceinline__ void add_x2(float& a0, float& a1, float b0, float b1) {
  unsigned long long A = pk2(a0, a1), B = pk2(b0, b1), R;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(R) : "l"(A), "l"(B));
  upk2(R, a0, a1);
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// One row's softmax of a unit: its 128 scores in tensor memory become
// probabilities (bf16, in the same place).  m: the reference they are relative
// to, a maximum of scores seen before; l: the sum of probabilities; fix: what
// sums from before have to be multiplied with.  FULL: every column is seen.
//
// 32 columns at a time.  No maximum is taken as long as their probabilities add
// up to less than kGrow: bf16 and fp32 hold a probability of 2^16 as well as one
// of 1.  Above it, or while a row has no reference yet, the warp takes the
// largest score as the reference of the rows concerned and brings the columns
// already done (and, through `fix`, l and O) to it.  The loop is not unrolled:
// the roles share the instruction cache.
template <bool FULL>
struct UnitSoftmax {
  uint32_t s_at;
  uint4 there;
  int c_lo, c_hi;
  float qu;  // the row's and the unit's power of two

  __device__ __forceinline__ uint32_t seen(int c) const {  // of columns 32 c .. 32 c + 31
    const uint32_t e = c == 0 ? there.x : c == 1 ? there.y : c == 2 ? there.z : there.w;
    const int x0 = max(0, min(32, c_lo - 32 * c)), x1 = max(0, min(32, c_hi - 32 * c));
    const uint32_t below = x1 == 32 ? ~0u : (1u << x1) - 1, under = x0 == 32 ? ~0u : (1u << x0) - 1;
    return e & below & ~under;
  }
  // Probabilities of 32 columns; their sum.
  __device__ __forceinline__ float probabilities(const uint32_t (&v)[32], uint32_t see, float base, uint32_t (&p)[16]) const {
    float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      float x[4];
      fma_x2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]), qu, qu, base, base, x[0], x[1]);
      fma_x2(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]), qu, qu, base, base, x[2], x[3]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (!FULL) x[e] = (see >> (i + e)) & 1 ? x[e] : -INFINITY;
        x[e] = ex2(x[e]);
      }
      add_x2(s0, s1, x[0], x[1]);
      add_x2(s2, s3, x[2], x[3]);
      p[i / 2] = f32_to_bf16x2(x[0], x[1]);
      p[i / 2 + 1] = f32_to_bf16x2(x[2], x[3]);
    }
    add_x2(s0, s1, s2, s3);
    return s0 + s1;
  }
  __device__ __forceinline__ void run(float& m, float& l, float& fix) const {
    float base = m == -INFINITY ? 0.0f : -m;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint32_t v[32], p[16];
      tmem_load32_now(s_at + 32 * c, v);
      const uint32_t see = FULL ? ~0u : seen(c);
      float sum = probabilities(v, see, base, p);
      if (__any_sync(0xffffffffu, sum > kGrow || m == -INFINITY)) {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; ++i) top = (see >> i) & 1 ? fmaxf(top, fmaf(__uint_as_float(v[i]), qu, base)) : top;
        const bool grow = (m == -INFINITY || sum > kGrow) && top > -INFINITY;
        const float f = grow ? (m == -INFINITY ? 0.0f : ex2(-top)) : 1.0f;
        if (grow) {
          base -= top;
          m = -base;
        }
        fix *= f;
        l *= f;
        tmem_store_wait();
#pragma unroll 1
        for (int k = 0; k < c; ++k) {
          tmem_load16_now(s_at + 16 * k, p);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float u, w;
            bf16x2_to_f32(p[i], u, w);
            p[i] = f32_to_bf16x2(u * f, w * f);
          }
          tmem_store16(s_at + 16 * k, p);
        }
        sum = probabilities(v, see, base, p);
      }
      l += sum;
      tmem_store16(s_at + 16 * c, p);
    }
  }
};

// Element of the head that column c of an 8-column chunk of K, Q and V holds:
// the order in which the codes fall out of a word.
template <int BITS>
__host__ __device__ constexpr int v_elem(int c) {
  return BITS == 4 ? (c >> 1) + 4 * (c & 1) : (c & 4) + 2 * (c & 1) + ((c >> 1) & 1);
}

template <int D, int BITS>
__global__ void __launch_bounds__(kThreads, 1) k_kv_prompt(const KvArgs a, const KvAttn t) {
  using F = Prompt<D>;
  constexpr int VB = D * BITS / 8, CH = VB / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + F::BARS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &bars->abort;

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
    for (int i = 0; i < 4; ++i) mbar_init(&bars->sc[i], 128);
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
  __shared__ uint64_t turns[D / 2];
  __shared__ uint32_t k_neg[D / 32], v_neg[D / 32];  // a bit for each element whose sign is flipped
  kv_turns(a, turns, threadIdx.x, kThreads);
  if (warp >= 4 && warp < 4 + D / 32) {
    const int i = 32 * (warp - 4) + lane;
    const uint32_t kb = __ballot_sync(0xffffffffu, a.k_signs != nullptr && __ldg(a.k_signs + i) < 0);
    const uint32_t vb = __ballot_sync(0xffffffffu, a.v_signs != nullptr && __ldg(a.v_signs + i) < 0);
    if (lane == 0) k_neg[warp - 4] = kb, v_neg[warp - 4] = vb;
  }
  if (warp == 0) plan_warp(a, t, bars, lane);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = bars->tmem;
  auto give_up = [&]() {
    atomicAdd(&g_wait_timeouts_kv, 1u);
    *abort = 1;
  };

  Walk w;
  if (warp < 8) {
    regs_more<176>();
    w.start(bars);
    // ---------------- softmax of half `hf`, a thread a row ----------------
    const int hf = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lane_at = tmem + (uint32_t(32 * (warp & 3)) << 16);
    const uint32_t s_at = lane_at + F::S_COL + 128 * hf, o_at = lane_at + F::O_COL + D * hf;
    float* es = reinterpret_cast<float*>(smem + F::ES) + 128 * hf;
    const KvWork work = kv_work_of<D, kRows>(t.ws, gridDim.x);
    uint32_t ns = 0, no = 0;  // score units and outputs seen so far
    uint32_t kv0 = 0;         // units converted before this segment
    KvPart open;
    open.first = -1;
    int64_t unit = w.left;    // of the CTA's share, what is left before this segment
    for (bool more = w.begin(a, t); more && !*abort; more = w.next(a, t)) {
      const Segment& g = w.g;
      const Half& f = g.half[hf];
      const int row = g.row0 + 128 * hf + r;
      const bool mine = r < f.rows;
      const int tok = mine ? row / t.group : 0;
      const int head = g.h * t.group + (mine ? row - tok * t.group : 0);
      float m = -INFINITY, l = 0.0f;
      bool ok = true;
      if (f.js < f.je) {
        // the half's queries: turned, rotated, scaled into base-2 scores, brought to [-2, 2)
        constexpr int LPV = KvLanes<D>::LPV;
        const int ln = r % LPV;
#pragma unroll 1
        for (int q0 = 0; q0 < 128; q0 += 128 / LPV) {
          const int qr = q0 + r / LPV;
          float x[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = 0.0f;
          if (qr < f.rows) {
            const int row_q = g.row0 + 128 * hf + qr, tk = row_q / t.group;
            const int64_t src = (g.q.t0 + tk) * t.q_ts + (int64_t(g.h) * t.group + row_q - tk * t.group) * t.q_hs;
            if (t.q_f32) {
#pragma unroll
              for (int c = 0; c < 4; ++c) kv_load8<true>(t.q, src + 8 * (c * LPV + ln), x + 8 * c);
              if (a.n_freq > 0) kv_rope_direct<D, true>(x, t.q, src, a, turns, g.q.t0 + tk, int(g.q.pos0) + tk, ln);
            } else {
#pragma unroll
              for (int c = 0; c < 4; ++c) kv_load8<false>(t.q, src + 8 * (c * LPV + ln), x + 8 * c);
              if (a.n_freq > 0) kv_rope_direct<D, false>(x, t.q, src, a, turns, g.q.t0 + tk, int(g.q.pos0) + tk, ln);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int ch = c * LPV + ln;
              const uint32_t neg = k_neg[ch >> 2] >> (8 * (ch & 3));
#pragma unroll
              for (int e = 0; e < 8; ++e)
                x[8 * c + e] = __uint_as_float(__float_as_uint(x[8 * c + e]) ^ ((neg << (31 - e)) & 0x80000000u));
            }
          }
          kv_hadamard<D>(x, ln);
          float up, down;
          kv_query_scale<D>(x, t.scale, up, down);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int d0 = 8 * (c * LPV + ln);
            uint32_t v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int i = BITS == 4 ? e : 2 * e, j = BITS == 4 ? e + 4 : 2 * e + 1;
              const __half2 p = __floats2half2_rn(x[8 * c + i] * down, x[8 * c + j] * down);
              v[e] = *reinterpret_cast<const uint32_t*>(&p);
            }
            *reinterpret_cast<uint4*>(smem + F::Q + hf * F::TILE + (d0 / 64) * 16384 + qr * 128 +
                                      (((d0 % 64) / 8) ^ (qr & 7)) * 16) = make_uint4(v[0], v[1], v[2], v[3]);
          }
          if (ln == 0) es[qr] = up;
        }
        fence_proxy_async_smem();
        mbar_arrive(&bars->q[hf]);
        asm volatile("bar.sync %0, 128;" ::"r"(1 + hf) : "memory");
        const float qe = es[r];
        const int64_t pos = g.q.pos0 + tok;
        const int64_t hi = mine ? (t.causal ? min(g.q.hi, pos + 1) : g.q.hi) : 0;
        const int64_t lo = t.window > 0 ? pos - t.window + 1 : 0;

        for (int j = f.js; j < f.je && ok; ++j) {
          const uint32_t kv = kv0 + uint32_t(j - g.ub);
          const uint8_t* scp = smem + F::SC + (kv & 3) * F::SC_STAGE;
          ok = mbar_wait(&bars->sc[kv & 3], (kv >> 2) & 1u) && mbar_wait(&bars->s[hf], ns & 1u);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          ++ns;
          fence_after();
          const uint4 there = *reinterpret_cast<const uint4*>(scp);
          const float qu = qe * *reinterpret_cast<const float*>(scp + 16);
          const int64_t p0 = int64_t(j) * kKeys;
          const bool full = p0 >= f.lo_max && p0 + kKeys <= f.hi_min && (there.x & there.y & there.z & there.w) == ~0u;
          // columns [c_lo, c_hi) are this row's
          const int c_lo = int(max(int64_t(0), min(int64_t(128), lo - p0)));
          const int c_hi = int(max(int64_t(0), min(int64_t(128), hi - p0)));
          float fix = 1.0f;
          if (full) UnitSoftmax<true>{s_at, there, 0, kKeys, qu}.run(m, l, fix);
          else UnitSoftmax<false>{s_at, there, c_lo, c_hi, qu}.run(m, l, fix);
          if (j > f.js && __any_sync(0xffffffffu, fix != 1.0f)) {
            // the product of the unit before has to be in O
            ok = mbar_wait(&bars->o[hf], (no - 1) & 1u);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            fence_after();
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
      const bool whole = g.x0 == 0 && g.x1 == g.count;
      const bool any = f.js < f.je;
      const size_t slot_row = (g.x0 == 0 ? 2 * size_t(blockIdx.x) + 1 : 2 * size_t(blockIdx.x)) * kRows + 128 * hf + r;
      const float inv = l == 0.0f ? 0.0f : (D == 64 ? 0.125f : 0.08838834764831845f) / l;
      if (f.rows > 0) {  // by the whole warp: tensor memory is read together
        if (whole) {
          constexpr int N = D / 64;  // the transform's last stage joins the halves of 128 elements
#pragma unroll 1
          for (int b = 0; b < N; ++b) {
            float x[64];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t u[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) x[32 * c + i] = 0.0f;
              if (any) {
                tmem_load32_now(o_at + 32 * c, u);
#pragma unroll
                for (int i = 0; i < 32; ++i) x[32 * c + 8 * (i / 8) + v_elem<BITS>(i % 8)] = __uint_as_float(u[i]) * inv;
                if constexpr (N == 2) {
                  tmem_load32_now(o_at + 64 + 32 * c, u);
#pragma unroll
                  for (int i = 0; i < 32; ++i)
                    x[32 * c + 8 * (i / 8) + v_elem<BITS>(i % 8)] += __uint_as_float(u[i]) * (b == 0 ? inv : -inv);
                }
              }
            }
            reg_stages<64, 0, 6>(x);
            if (mine) {
#pragma unroll
              for (int i = 0; i < 64; ++i)
                x[i] = __uint_as_float(__float_as_uint(x[i]) ^ ((v_neg[2 * b + i / 32] << (31 - i % 32)) & 0x80000000u));
              const int64_t at = (g.q.t0 + tok) * t.o_ts + head * t.o_hs + 64 * b;
#pragma unroll
              for (int i = 0; i < 64; i += 8) {
                if (t.o_f32) kv_store8<true>(t.out, at + i, x + i);
                else kv_store8<false>(t.out, at + i, x + i);
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
            for (int i = 0; i < 32; ++i) x[8 * (i / 8) + v_elem<BITS>(i % 8)] = any ? __uint_as_float(u[i]) : 0.0f;
            if (mine) {
#pragma unroll
              for (int i = 0; i < 32; i += 8) kv_store8<true>(work.rows, slot_row * D + 32 * c + i, x + i);
            }
          }
          if (mine) work.ms[slot_row] = make_float2(m, l);
        }
      }
      if (!whole && g.x0 == 0) {
        const int64_t at = int64_t(blockIdx.x) * bars->total / bars->ctas + (unit - w.left);
        open.first = blockIdx.x;
        open.last = kv_cta_of(at + g.count - 1, bars->total, bars->ctas);
        open.rows = g.nr;
        open.row0 = g.row0;
        open.t0 = g.q.t0;
        open.h = g.h;
        open.pad = 0;
      }
      fence_before();
      kv0 += uint32_t(g.ue - g.ub);
    }
    if (threadIdx.x == 0) work.part[2 * blockIdx.x + 1] = open;
  } else if (warp < 12) {
    // ---------------- codes to operands ----------------
    regs_less<112>();
    w.start(bars);
    const int i = threadIdx.x - 256;
    const int piece = i % CH;
    uint32_t kv = 0;
    bool ok = true;
    for (bool more = w.begin(a, t); more && ok; more = w.next(a, t)) {
      const Segment& g = w.g;
      uint4 kr[CH], vr[CH];
      float ksc = 0.0f, vsc = 0.0f;
      bool in = false;
      // this thread's vectors of unit j (-1: no such position), and the one whose scales it brings
      int64_t vec[CH], own;
      auto find = [&](int j) {
#pragma unroll
        for (int k = 0; k <= CH; ++k) {
          const int64_t p = int64_t(j) * kKeys + (k < CH ? i / CH + (128 / CH) * k : i);
          const int64_t slot = p < g.q.hi ? kv_slot(a, g.s, p) : -1;
          const int64_t v = slot < 0 ? slot : slot + (int64_t(g.h) << a.log_page);
          if (k < CH) vec[k] = v;
          else own = v;
        }
      };
      auto load = [&](const uint8_t* codes, uint4 (&x)[CH]) {
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          x[k] = make_uint4(0, 0, 0, 0);
          if (vec[k] >= 0) load16(x[k], codes + vec[k] * VB + 16 * piece);
        }
      };
      auto load_scales = [&]() {
        in = own >= 0;
        ksc = vsc = 0.0f;
        if (in) {
          load4(ksc, a.k_scales + own);
          load4(vsc, a.v_scales + own);
        }
      };
      if (g.ub < g.ue) {
        find(g.ub);
        load(a.k_codes, kr);
        load_scales();
        load(a.v_codes, vr);
      }
      for (int j = g.ub; j < g.ue; ++j, ++kv) {
        const int st = kv & 1;
        const uint32_t round = kv >> 1;
        ok = !*abort && (round == 0 || mbar_wait(&bars->kempty[st], (round - 1) & 1u));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        // The scales are folded into the operands, with one rounding: a product
        // with a scale in two parts, hi and the rest.  Keys are relative to a
        // power of two of the unit's largest scale, so that fp16 holds them.  A
        // position whose scale is not finite becomes NaN in its scores, and only there.
        uint8_t* tsp = smem + F::TS + (kv & 1) * F::TS_STAGE;
        {
          const bool k_fine = (__float_as_uint(ksc) & 0x7f800000u) != 0x7f800000u;
          const bool v_fine = (__float_as_uint(vsc) & 0x7f800000u) != 0x7f800000u;
          reinterpret_cast<float*>(tsp)[i] = v_fine ? ksc : __uint_as_float(0x7fc00000u);
          reinterpret_cast<float*>(tsp)[128 + i] = v_fine ? vsc : 0.0f;
          const uint32_t top = __reduce_max_sync(0xffffffffu, k_fine ? __float_as_uint(ksc) & 0x7fffffffu : 0u);
          const uint32_t b = __ballot_sync(0xffffffffu, in);
          if (lane == 0) {
            reinterpret_cast<uint32_t*>(tsp + 1024)[warp - 8] = top;
            reinterpret_cast<uint32_t*>(smem + F::SC + (kv & 3) * F::SC_STAGE)[warp - 8] = b;
          }
        }
        asm volatile("bar.sync 3, 128;" ::: "memory");
        const uint4 tops = *reinterpret_cast<const uint4*>(tsp + 1024);
        const uint32_t ex = max(1u, max(max(tops.x, tops.y), max(tops.z, tops.w)) >> 23);
        const float down = __uint_as_float(ex == 254 ? 0x00400000u : (254 - ex) << 23);
        if (i == 0) *reinterpret_cast<uint32_t*>(smem + F::SC + (kv & 3) * F::SC_STAGE + 16) = ex << 23;
        mbar_arrive(&bars->sc[kv & 3]);
        auto store = [&](uint8_t* tile, const uint4 (&x)[CH], bool value) {
#pragma unroll
          for (int k = 0; k < CH; ++k) {
            const int tk = i / CH + (128 / CH) * k;
            uint32_t s_hi, s_lo;
            if (value) {
              const float sc = reinterpret_cast<const float*>(tsp)[128 + tk];
              const float hi = __bfloat162float(__float2bfloat16_rn(sc));
              s_hi = f32_to_bf16x2(hi, hi);
              s_lo = f32_to_bf16x2(sc - hi, sc - hi);
            } else {
              const float sc = reinterpret_cast<const float*>(tsp)[tk] * down;
              const __half hi = __float2half_rn(sc), lo = __float2half_rn(sc - __half2float(hi));
              s_hi = uint32_t(__half_as_ushort(hi)) * 0x10001u;
              s_lo = uint32_t(__half_as_ushort(lo)) * 0x10001u;
            }
            const uint32_t wd[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
            constexpr int OUT = 128 / (8 * BITS);  // 16-byte chunks of operand from 16 bytes of codes
            const int c0 = OUT * piece;
            uint8_t* row = tile + (c0 / 8) * 16384 + tk * 128;
            // lanes of different column blocks store their chunks in another order (bank conflicts)
            const int turn = D == 128 ? (BITS == 4 ? 2 * (c0 / 8) : c0 / 8) : 0;
#pragma unroll
            for (int e0 = 0; e0 < OUT; ++e0) {
              uint32_t o[4];
              const int e = e0 ^ turn;
              if constexpr (BITS == 4) {
                const uint32_t u = e == 0 ? wd[0] : e == 1 ? wd[1] : e == 2 ? wd[2] : wd[3];
                if (value) bf_of4(u, o);
                else half_of4(u, o);
              } else {
                const uint32_t u0 = e == 0 ? wd[0] : wd[2], u1 = e == 0 ? wd[1] : wd[3];
                if (value) {
                  bf_of8(u0, o[0], o[1]);
                  bf_of8(u1, o[2], o[3]);
                } else {
                  half_of8(u0, o[0], o[1]);
                  half_of8(u1, o[2], o[3]);
                }
              }
#pragma unroll
              for (int y = 0; y < 4; ++y)
                o[y] = value ? bfma2(o[y], s_hi, bfma2(o[y], s_lo, 0x80008000u)) : hfma2(o[y], s_hi, hfma2(o[y], s_lo, 0x80008000u));
              *reinterpret_cast<uint4*>(row + (((c0 % 8) + e) ^ (tk & 7)) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
        };
        store(smem + F::K + st * F::TILE, kr, false);
        fence_proxy_async_smem();
        mbar_arrive(&bars->kfull[st]);
        // the next unit's codes are on their way while this one's are waited for and unpacked
        if (j + 1 < g.ue) {
          find(j + 1);
          load(a.k_codes, kr);
          load_scales();
        }
        ok = round == 0 || mbar_wait(&bars->vempty[st], (round - 1) & 1u);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        store(smem + F::V + st * F::TILE, vr, true);
        fence_proxy_async_smem();
        mbar_arrive(&bars->vfull[st]);
        if (j + 1 < g.ue) load(a.v_codes, vr);
      }
    }
    if (!ok && !*abort) give_up();
  } else {
    regs_less<48>();
    if (warp == 12) {
      // ---------------- products: the warp waits, one thread issues ----------------
      w.start(bars);
      constexpr uint32_t id_s = instr_desc(false, 128, false), id_o = instr_desc(true, D, true);
      const uint32_t base = smem_u32(smem);
      // descriptors of the tiles: the upper word is the same for all, the lower one holds the address
      const uint64_t dk = desc_sw128(base, 16, 1024), dv = desc_sw128(base + F::V, 16384, 1024);
      const uint32_t k_hi = uint32_t(dk >> 32), v_hi = uint32_t(dv >> 32);
      const uint32_t q_lo = uint32_t(dk), k_lo = q_lo + (F::K >> 4), v_lo = uint32_t(dv);
      uint32_t nq[2] = {0, 0}, np[2] = {0, 0};
      uint32_t kv0 = 0;
      bool ok = true;
      for (bool more = w.begin(a, t); more && ok; more = w.next(a, t)) {
        const Segment& g = w.g;
        for (int j = g.ub - 1; j < g.ue && ok; ++j) {
          if (g.ub == g.ue) break;
          const uint32_t kv = kv0 + uint32_t(j - g.ub);  // unit j (j = ub - 1: none)
          const uint32_t kn = kv + 1;
          bool have_v = false, have_k = false;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const Half& f = g.half[hf];
            if (ok && j >= f.js && j < f.je) {
              if (!have_v) ok = mbar_wait(&bars->vfull[kv & 1], (kv >> 1) & 1u);
              have_v = true;
              ok = ok && !*abort && mbar_wait(&bars->p[hf], np[hf] & 1u);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              ++np[hf];
              fence_after();
              if (elect_one()) {
                const uint32_t lo = v_lo + (kv & 1) * (F::TILE >> 4);
                const bool add = j > f.js;
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                  mma_ts(tmem + F::O_COL + D * hf, tmem + F::S_COL + 128 * hf + 8 * k, lo + k * 128, v_hi, id_o, k > 0 || add);
                commit(&bars->o[hf]);
              }
            }
            if (ok && j + 1 >= f.js && j + 1 < f.je) {
              if (!have_k) ok = mbar_wait(&bars->kfull[kn & 1], (kn >> 1) & 1u);
              have_k = true;
              if (ok && j + 1 == f.js) ok = mbar_wait(&bars->q[hf], nq[hf]++ & 1u);
              ok = __all_sync(0xffffffffu, ok && !*abort);
              if (!ok) break;
              fence_after();
              if (elect_one()) {
                const uint32_t lo_q = q_lo + hf * (F::TILE >> 4), lo_k = k_lo + (kn & 1) * (F::TILE >> 4);
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
            if (j >= g.ub) commit(&bars->vempty[kv & 1]);
            if (j + 1 < g.ue) commit(&bars->kempty[kn & 1]);
          }
          __syncwarp();
        }
        kv0 += uint32_t(g.ue - g.ub);
      }
      if (!ok && !*abort) give_up();
      // every product has ended before tensor memory is given back
      if (elect_one()) commit(&bars->done);
      if (!mbar_wait(&bars->done, 0u)) atomicAdd(&g_wait_timeouts_kv, 1u);
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
  kernel<<<kCtas, kThreads, bytes, st>>>(a, t);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_kv_join<D, kRows>(a, t, kCtas, st);
}

}  // namespace

size_t kv_prompt_bytes(int head_dim) {
  return head_dim == 64 ? kv_work_bytes<64, kRows>(kCtas) : head_dim == 128 ? kv_work_bytes<128, kRows>(kCtas) : 0;
}

cudaError_t launch_kv_prompt(const KvArgs& a, const KvAttn& t, cudaStream_t st) {
  if (a.head_dim == 64) return a.bits == 4 ? go<64, 4>(a, t, st) : go<64, 8>(a, t, st);
  return a.bits == 4 ? go<128, 4>(a, t, st) : go<128, 8>(a, t, st);
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

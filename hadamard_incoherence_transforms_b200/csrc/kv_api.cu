// C ABI of the rotated key/value cache (declared in include/hit.h): host-side
// argument checks and dispatch.  Every check runs before the first CUDA call.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>

#include "hit.h"
#include "internal.h"
#include "kv.h"

namespace {

int fail(int status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  hit::set_last_error(buf);
  return status;
}

int cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return HIT_OK;
  return fail(HIT_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxTokens = int64_t(1) << 31;

// Sequences with up to kFewRows query rows for a key/value head go to the kernel
// that streams the codes once for 16 rows (an SM takes 7 cycles for a position and
// 16 rows), the others to the one that works on 256 rows at a time (40 cycles for a
// position, whatever the rows).  64 sequences of up to 4,000 positions take 216 us and
// 277 with 32 rows, 414 and 283 with 64, 849 and 324 with 128; a call of few sequences
// gains more from the first kind's one launch.  Heads of 256 go 8 and 128 rows at a time:
// 233 and 345 us with 16 rows, 425 and 348 with 32, 848 and 359 with 64; two sequences of
// 25 rows 32 and 50.  Each launch leaves the other's sequences alone, so that max_new
// decides only whether the second kind is needed.
constexpr int64_t kFewRows = 64, kFewRows256 = 32;
int64_t few_rows(int head_dim) { return head_dim == 256 ? kFewRows256 : kFewRows; }
bool few_only(int64_t max_new, int64_t group, int head_dim) { return max_new * group <= few_rows(head_dim); }

// Checks what the three calls share and fills `a`.  `rope`: whether the call
// uses the rotary fields.
int check_kv(const char* fn, const hit_kv* c, int64_t tokens, bool rope, hit::KvArgs& a) {
  if (c == nullptr) return fail(HIT_EINVAL, "%s: kv is NULL", fn);
  if (tokens < 0 || tokens >= kMaxTokens) return fail(HIT_EINVAL, "%s: tokens outside [0, 2^31)", fn);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(HIT_EUNSUPPORTED, "%s: head_dim must be 64, 128 or 256", fn);
  if (c->bits != 4 && c->bits != 8) return fail(HIT_EUNSUPPORTED, "%s: bits must be 4 or 8", fn);
  if (c->kv_heads < 1 || c->kv_heads > 65535) return fail(HIT_EINVAL, "%s: kv_heads outside [1, 65535]", fn);
  if (c->page_size < 1 || c->page_size > 65536 || (c->page_size & (c->page_size - 1)) != 0)
    return fail(HIT_EUNSUPPORTED, "%s: page_size must be a power of two <= 65536", fn);
  if (c->pages < 0 || c->pages >= kMaxTokens) return fail(HIT_EINVAL, "%s: pages outside [0, 2^31)", fn);
  if (c->seqs < 0 || c->seqs == INT32_MAX || c->max_pages < 0)
    return fail(HIT_EINVAL, "%s: negative or too large seqs or max_pages", fn);
  if (c->ld_table < c->max_pages) return fail(HIT_EINVAL, "%s: ld_table < max_pages", fn);
  if (tokens > 0 && c->seqs > 0) {
    if (c->cu == nullptr || c->lens == nullptr || (c->page_table == nullptr && c->max_pages > 0))
      return fail(HIT_EINVAL, "%s: page_table, lens and cu are required", fn);
    if (c->pages > 0 && (c->k_codes == nullptr || c->v_codes == nullptr || c->k_scales == nullptr || c->v_scales == nullptr))
      return fail(HIT_EINVAL, "%s: the cache's codes and scales are required", fn);
  }
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_scales, 16))
    return fail(HIT_EALIGN, "%s: codes and scales must be 16-byte aligned", fn);
  if (!aligned(c->page_table, 4) || !aligned(c->lens, 4) || !aligned(c->cu, 4) || !aligned(c->positions, 4) ||
      !aligned(c->inv_freq, 4))
    return fail(HIT_EALIGN, "%s: page_table, lens, cu, positions and inv_freq must be 4-byte aligned", fn);
  if (rope && c->inv_freq != nullptr) {
    if (c->n_freq < 0 || 2 * int64_t(c->n_freq) > c->head_dim)
      return fail(HIT_EINVAL, "%s: n_freq must be in [0, head_dim / 2]", fn);
    if (c->n_freq % (c->interleaved ? 4 : 8) != 0)
      return fail(HIT_EUNSUPPORTED, "%s: n_freq must be a multiple of %d for %s pairs", fn, c->interleaved ? 4 : 8,
                  c->interleaved ? "interleaved" : "half-split");
    if (c->n_freq > 0 && c->positions != nullptr) {
      if (c->rope_axes < 1 || c->rope_axes > 127) return fail(HIT_EINVAL, "%s: rope_axes outside [1, 127]", fn);
      if (c->ld_positions < tokens) return fail(HIT_EINVAL, "%s: ld_positions < tokens", fn);
      if (c->rope_axes > 1 && c->rope_axis == nullptr)
        return fail(HIT_EINVAL, "%s: several position axes need rope_axis", fn);
    }
  }
  a.k_codes = c->k_codes;
  a.v_codes = c->v_codes;
  a.k_scales = c->k_scales;
  a.v_scales = c->v_scales;
  a.table = c->page_table;
  a.lens = c->lens;
  a.cu = c->cu;
  a.k_signs = c->k_signs;
  a.v_signs = c->v_signs;
  if (rope && c->inv_freq != nullptr && c->n_freq > 0) {
    a.inv_freq = c->inv_freq;
    a.n_freq = c->n_freq;
    a.interleaved = c->interleaved ? 1 : 0;
    a.positions = c->positions;
    a.rope_axis = c->rope_axis;
    a.rope_axes = c->rope_axes;
    a.ld_pos = c->ld_positions;
  }
  a.pages = c->pages;
  a.ld_table = c->ld_table;
  a.tokens = tokens;
  a.hk = c->kv_heads;
  while ((int64_t(1) << a.log_page) < c->page_size) ++a.log_page;
  a.seqs = c->seqs;
  a.max_pages = c->max_pages;
  a.head_dim = c->head_dim;
  a.bits = c->bits;
  return HIT_OK;
}

// A [tokens, heads, head_dim] operand: 16-byte pieces of a head are read or written whole.
int check_dense(const char* fn, const char* name, const void* p, int64_t ts, int64_t hs, int dt) {
  if (p == nullptr) return fail(HIT_EINVAL, "%s: %s is NULL", fn, name);
  const int64_t per = dt == HIT_F32 ? 4 : 8;
  if (ts < 0 || hs < 0) return fail(HIT_EINVAL, "%s: %s has a negative stride", fn, name);
  if (!aligned(p, 16) || ts % per != 0 || hs % per != 0)
    return fail(HIT_EALIGN, "%s: %s and its strides must be 16-byte aligned", fn, name);
  return HIT_OK;
}

// Whether two rows of n elements of a [tokens, heads, n] tensor share an element.
bool rows_overlap(int64_t tokens, int64_t heads, int64_t n, int64_t ts, int64_t hs) {
  if ((heads > 1 && hs < n) || (tokens > 1 && ts < n)) return true;
  // a token's heads end before the next token, or a head's tokens before the next head
  if (heads < 2 || tokens < 2 || (ts - n) / hs >= heads - 1 || (hs - n) / ts >= tokens - 1) return false;
  for (int64_t h = 1; h < heads; ++h)  // rows (t + a, 0) and (t, h) for the a on both sides of h hs / ts
    for (int64_t a = h * hs / ts; a <= h * hs / ts + 1 && a < tokens; ++a)
      if (std::abs(h * hs - a * ts) < n) return true;
  return false;
}

// An operand that is written.
int check_out(const char* fn, const char* name, const void* p, int64_t tokens, int64_t heads, int64_t n, int64_t ts,
              int64_t hs, int dt) {
  const int r = check_dense(fn, name, p, ts, hs, dt);
  if (r == HIT_OK && rows_overlap(tokens, heads, n, ts, hs)) return fail(HIT_EINVAL, "%s: rows of %s overlap", fn, name);
  return r;
}

}  // namespace

extern "C" {

int rht_kv_append(const hit_kv* kv, const void* k, const void* v, int64_t tokens, int64_t k_ts, int64_t k_hs,
                  int64_t v_ts, int64_t v_hs, int dtype, void* stream) {
  const char* fn = "rht_kv_append";
  if (dtype != HIT_F32 && dtype != HIT_BF16) return fail(HIT_EUNSUPPORTED, "%s: unknown dtype", fn);
  hit::KvArgs a;
  int r = check_kv(fn, kv, tokens, true, a);
  if (r) return r;
  if (tokens == 0 || a.seqs == 0 || a.pages == 0) return HIT_OK;
  r = check_dense(fn, "k", k, k_ts, k_hs, dtype);
  if (r) return r;
  r = check_dense(fn, "v", v, v_ts, v_hs, dtype);
  if (r) return r;
  hit::KvDense x;
  x.k = k;
  x.v = v;
  x.k_ts = k_ts;
  x.k_hs = k_hs;
  x.v_ts = v_ts;
  x.v_hs = v_hs;
  return cuda_status(hit::launch_kv_append(a, x, dtype, static_cast<cudaStream_t>(stream)), fn);
}

int rht_kv_read(const hit_kv* kv, void* k, void* v, int64_t rows, int64_t k_ts, int64_t k_hs, int64_t v_ts, int64_t v_hs,
                int dtype, void* stream) {
  const char* fn = "rht_kv_read";
  const bool zero = (dtype & HIT_KV_ZERO) != 0;
  dtype &= ~HIT_KV_ZERO;
  if (dtype != HIT_F32 && dtype != HIT_BF16) return fail(HIT_EUNSUPPORTED, "%s: unknown dtype", fn);
  hit::KvArgs a;
  int r = check_kv(fn, kv, rows, false, a);
  if (r) return r;
  if (rows == 0 || (a.seqs == 0 && !zero) || (k == nullptr && v == nullptr)) return HIT_OK;
  if (k != nullptr && (r = check_out(fn, "k", k, rows, a.hk, a.head_dim, k_ts, k_hs, dtype)) != 0) return r;
  if (v != nullptr && (r = check_out(fn, "v", v, rows, a.hk, a.head_dim, v_ts, v_hs, dtype)) != 0) return r;
  hit::KvDense y;
  y.k = k;
  y.v = v;
  y.k_ts = k_ts;
  y.k_hs = k_hs;
  y.v_ts = v_ts;
  y.v_hs = v_hs;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a.seqs == 0) {
    cudaError_t e = cudaSuccess;
    if (k != nullptr) e = hit::launch_kv_zero(k, rows, a.hk, a.head_dim, k_ts, k_hs, dtype, st);
    if (v != nullptr && e == cudaSuccess) e = hit::launch_kv_zero(v, rows, a.hk, a.head_dim, v_ts, v_hs, dtype, st);
    return cuda_status(e, fn);
  }
  return cuda_status(hit::launch_kv_read(a, y, dtype, zero, st), fn);
}

size_t rht_kv_workspace_bytes(int64_t tokens, int heads, int kv_heads, int head_dim, int64_t max_new) {
  if (tokens < 1 || tokens >= kMaxTokens || heads < 1 || kv_heads < 1 || heads % kv_heads != 0 || max_new < 1 ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return 0;
  const size_t few = hit::kv_few_bytes(head_dim);
  if (few_only(std::min(tokens, max_new), heads / kv_heads, head_dim)) return few;
  return std::max(few, hit::kv_prompt_bytes(tokens, heads, head_dim));
}

int rht_kv_attention(const hit_kv* kv, const void* q, void* out, int64_t tokens, int heads, int64_t q_ts, int64_t q_hs,
                     int64_t o_ts, int64_t o_hs, int dtype_q, int dtype_out, float sm_scale, int causal, int64_t window,
                     int64_t max_new, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "rht_kv_attention";
  const bool zero = (dtype_out & HIT_KV_ZERO) != 0;
  dtype_out &= ~HIT_KV_ZERO;
  if ((dtype_q != HIT_F32 && dtype_q != HIT_BF16) || (dtype_out != HIT_F32 && dtype_out != HIT_BF16))
    return fail(HIT_EUNSUPPORTED, "%s: unknown dtype", fn);
  hit::KvArgs a;
  int r = check_kv(fn, kv, tokens, true, a);
  if (r) return r;
  if (heads < 1 || heads % a.hk != 0) return fail(HIT_EINVAL, "%s: heads must be a multiple of kv_heads", fn);
  if (heads > 65536) return fail(HIT_EUNSUPPORTED, "%s: more than 65536 heads", fn);
  if (!std::isfinite(sm_scale)) return fail(HIT_EINVAL, "%s: sm_scale must be finite", fn);
  if (window < 0 || (window > 0 && !causal)) return fail(HIT_EINVAL, "%s: a window must be positive and causal", fn);
  if (max_new < 1) return fail(HIT_EINVAL, "%s: max_new must be positive", fn);
  if (tokens == 0 || (a.seqs == 0 && !zero)) return HIT_OK;
  if (tokens * heads >= kMaxTokens) return fail(HIT_EUNSUPPORTED, "%s: tokens * heads must stay below 2^31", fn);
  r = check_dense(fn, "q", q, q_ts, q_hs, dtype_q);
  if (r) return r;
  r = check_out(fn, "out", out, tokens, heads, a.head_dim, o_ts, o_hs, dtype_out);
  if (r) return r;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a.seqs == 0) return cuda_status(hit::launch_kv_zero(out, tokens, heads, a.head_dim, o_ts, o_hs, dtype_out, st), fn);
  const size_t need = rht_kv_workspace_bytes(tokens, heads, a.hk, a.head_dim, max_new);
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need)
      return fail(HIT_EWORKSPACE, "%s: needs %zu workspace bytes", fn, need);
    if (!aligned(workspace, 16)) return fail(HIT_EALIGN, "%s: workspace must be 16-byte aligned", fn);
  }
  hit::KvAttn t;
  t.q = q;
  t.out = out;
  t.q_ts = q_ts;
  t.q_hs = q_hs;
  t.o_ts = o_ts;
  t.o_hs = o_hs;
  t.heads = heads;
  t.group = heads / a.hk;
  t.q_f32 = dtype_q == HIT_F32;
  t.o_f32 = dtype_out == HIT_F32;
  const int64_t out_bytes = t.o_f32 ? 4 : 2;
  t.wide = aligned(out, 32) && o_ts * out_bytes % 32 == 0 && o_hs * out_bytes % 32 == 0;
  t.zero = zero ? 1 : 0;
  t.causal = causal ? 1 : 0;
  t.scale = sm_scale;
  t.window = std::min<int64_t>(window, kMaxTokens * 4);  // as good as any longer one, and positions less it stay in 64 bits
  t.max_new = max_new < tokens ? max_new : tokens;
  t.ws = workspace;
  if (few_only(t.max_new, t.group, a.head_dim)) return cuda_status(hit::launch_kv_few(a, t, st), fn);
  hit::KvAttn few = t;
  few.rows_hi = few.max_new = few_rows(a.head_dim);
  t.rows_lo = few.rows_hi + 1;
  t.zero = 0;  // few's part
  r = cuda_status(hit::launch_kv_prompt_queries(a, t, st), fn);
  if (r == HIT_OK) r = cuda_status(hit::launch_kv_few(a, few, st), fn);
  return r ? r : cuda_status(hit::launch_kv_prompt(a, t, st), fn);
}

}  // extern "C"

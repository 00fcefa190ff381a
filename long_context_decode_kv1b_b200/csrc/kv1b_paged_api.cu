// kv1b_paged_api.cu -- the paged-cache entry points of include/kv1b.h: argument checks on the host,
// then launches on the caller's stream.  Nothing here allocates device memory or synchronises.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "kv1b.h"
#include "kv1b_launch.h"
#include "kv1b_paged.h"

namespace {

constexpr int64_t kMaxBlocks = 1LL << 30;  // blocks of one kv-head that a call's page tables may name; 64 times as many in all

bool aligned(const void* ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }
bool dtype_ok(int32_t dt) { return dt == KV1B_DTYPE_F32 || dt == KV1B_DTYPE_BF16 || dt == KV1B_DTYPE_F16; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? KV1B_OK : KV1B_ERR_CUDA; }

int log2_exact(int32_t x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

bool page_tokens_ok(int32_t n) {
  return n >= KV1B_PAGED_BLOCK_TOKENS && n <= KV1B_PAGED_MAX_PAGE_TOKENS && (n & (n - 1)) == 0;
}

bool paged_ok(const kv1b_paged_t* c) {
  return c && c->pages && c->signs && c->num_pages >= 1 && c->num_kv_heads >= 1 && c->num_kv_heads <= KV1B_PAGED_MAX_HEADS &&
         page_tokens_ok(c->page_tokens) && aligned(c->pages, 128) && aligned(c->signs, 16);
}

kv1b::PagedView view(const kv1b_paged_t* c) {
  kv1b::PagedView v;
  v.pages = static_cast<uint8_t*>(c->pages);
  v.signs = c->signs;
  v.status = c->d_status;
  v.num_pages = c->num_pages;
  v.Hkv = c->num_kv_heads;
  v.bpp_shift = log2_exact(c->page_tokens / KV1B_PAGED_BLOCK_TOKENS);
  return v;
}

int num_sms() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if (cached[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    cached[dev] = n < kv1b::kMaxCtas ? n : kv1b::kMaxCtas;
  }
  return cached[dev];
}

int heads_check(const kv1b_paged_t* c, int32_t num_q_heads) {
  if (num_q_heads < 1 || num_q_heads % c->num_kv_heads != 0) return KV1B_ERR_INVALID_ARG;
  if (num_q_heads / c->num_kv_heads > KV1B_MAX_GROUP) return KV1B_ERR_UNSUPPORTED;
  return KV1B_OK;
}

// `one_for_all`: whether every sequence may have the same pages (a stride of 0).
int table_check(const kv1b_paged_t* c, int32_t num_seqs, int64_t table_stride, int32_t max_pages, int32_t prefix_pages,
                bool one_for_all) {
  if (num_seqs < 1 || max_pages < 1 || table_stride < 0 || prefix_pages < 0) return KV1B_ERR_INVALID_ARG;
  if (num_seqs > 1 && table_stride < max_pages && !(one_for_all && table_stride == 0)) return KV1B_ERR_INVALID_ARG;
  if (num_seqs > KV1B_PAGED_MAX_SEQS) return KV1B_ERR_UNSUPPORTED;
  const int64_t bpp = c->page_tokens / KV1B_PAGED_BLOCK_TOKENS;
  const int64_t blocks = num_seqs * bpp * (static_cast<int64_t>(max_pages) + prefix_pages);
  if (blocks > kMaxBlocks || blocks * c->num_kv_heads > kMaxBlocks * 64) return KV1B_ERR_UNSUPPORTED;
  if (bpp * max_pages * KV1B_PAGED_BLOCK_TOKENS > 0x7fffffff || bpp * prefix_pages * KV1B_PAGED_BLOCK_TOKENS > 0x7fffffff)
    return KV1B_ERR_UNSUPPORTED;
  return KV1B_OK;
}

// The rows of a tensor [T][H][128]: element strides of a token and a head.
struct Rows {
  uintptr_t base;
  int64_t T, st, H, sh;
};
typedef __int128 Wide;
constexpr Wide kRowElems = KV1B_HEAD_DIM;

Wide span(int64_t n, int64_t stride) { return Wide(n - 1) * stride + kRowElems; }  // of n rows

// No two rows share an element: one stride steps over all rows along the other.
bool rows_apart(const Rows& r) {
  if ((r.T > 1 && r.st < kRowElems) || (r.H > 1 && r.sh < kRowElems)) return false;
  return r.T == 1 || r.H == 1 || r.st >= span(r.H, r.sh) || r.sh >= span(r.T, r.st);
}

// About the d of lo .. hi for which x + d step is nearest to 0 (one of its neighbours may be nearer).
Wide nearest(Wide x, Wide step, Wide lo, Wide hi) {
  const Wide d = -x / step;
  return d < lo ? lo : (d > hi ? hi : d);
}

// Whether rows 0, a, 2 a, .. (na of them) and x, x + b, .. (nb) share an element; true also where they only may.
bool lines_meet(int64_t na, int64_t a, Wide x, int64_t nb, int64_t b) {
  if (x >= span(na, a) || x + span(nb, b) <= 0) return false;
  if (na > 1 && nb > 1 && a != b) return true;
  const Wide step = na > 1 ? a : b, lo = -Wide(na - 1), hi = nb - 1;  // x + d step for d = lo .. hi against one row at 0
  if (step == 0) return true;
  const Wide at = nearest(x, step, lo, hi);
  for (Wide d = at - 1; d <= at + 1; ++d)
    if (d >= lo && d <= hi && x + d * step > -kRowElems && x + d * step < kRowElems) return true;
  return false;
}

// Whether rows that are apart and those of another tensor of as many tokens share an element: exactly where their
// strides of tokens, or of heads, agree and step over the other dimension; else where their ranges meet.
bool rows_meet(const Rows& o, const Rows& r, int64_t es) {
  if (o.base == r.base) return true;
  const Wide delta = r.base > o.base ? Wide((r.base - o.base) / es) : -Wide((o.base - r.base) / es);
  if (delta >= Wide(o.T - 1) * o.st + span(o.H, o.sh) || delta + Wide(r.T - 1) * r.st + span(r.H, r.sh) <= 0) return false;
  auto outer = [&](int64_t no, int64_t nr, int64_t so, int64_t sr, int64_t mo, int64_t a, int64_t mr, int64_t b) {
    if (no == 1 && nr == 1) return lines_meet(mo, a, delta, mr, b);
    if (so != sr || so < span(mo, a) || so < span(mr, b)) return true;
    const Wide lo = -Wide(no - 1), hi = nr - 1, at = nearest(delta, so, lo, hi);
    for (Wide d = at - 1; d <= at + 1; ++d)  // so steps over both: no other d comes near
      if (d >= lo && d <= hi && lines_meet(mo, a, delta + d * so, mr, b)) return true;
    return false;
  };
  return outer(o.T, r.T, o.st, r.st, o.H, o.sh, r.H, r.sh) && outer(o.H, r.H, o.sh, r.sh, o.T, o.st, r.T, r.st);
}

}  // namespace

extern "C" {

size_t kv1b_paged_bytes(int32_t num_pages, int32_t num_kv_heads, int32_t head_dim, int32_t page_tokens) {
  if (num_pages < 1 || num_kv_heads < 1 || num_kv_heads > KV1B_PAGED_MAX_HEADS || head_dim != KV1B_HEAD_DIM ||
      !page_tokens_ok(page_tokens))
    return 0;
  return static_cast<size_t>(num_pages) * num_kv_heads * (page_tokens / KV1B_PAGED_BLOCK_TOKENS) * KV1B_PAGED_BLOCK_BYTES;
}

int kv1b_paged_signs(float* signs, uint64_t seed, int32_t rounds, int32_t* d_status, void* stream) {
  if (!signs || !d_status || rounds < 1 || rounds > KV1B_MAX_ROUNDS) return KV1B_ERR_INVALID_ARG;
  if (!aligned(signs, 16) || !aligned(d_status, 4)) return KV1B_ERR_MISALIGNED;
  return cuda_status(kv1b_launch_init(seed, rounds, signs, nullptr, 0, d_status, static_cast<cudaStream_t>(stream)));
}

int kv1b_paged_append(const kv1b_paged_t* cache, const void* k, const void* v, int32_t dtype, int32_t num_tokens,
                      int64_t k_stride_t, int64_t k_stride_h, int64_t v_stride_t, int64_t v_stride_h, int32_t num_seqs,
                      const int32_t* cu_new, const int32_t* start, const int32_t* page_table, int64_t table_stride,
                      int32_t max_pages, const kv1b_rope_t* rope, const int32_t* positions, int64_t pos_stride,
                      const void* q, void* q_out, int32_t num_q_heads, int64_t q_stride_t, int64_t q_stride_h,
                      int64_t qo_stride_t, int64_t qo_stride_h, void* stream) {
  if (!paged_ok(cache) || !k || !v || !dtype_ok(dtype) || num_tokens < 0 || !cu_new || !start || !page_table)
    return KV1B_ERR_INVALID_ARG;
  const int tc = table_check(cache, num_seqs, table_stride, max_pages, 0, false);
  if (tc != KV1B_OK) return tc;
  if (k_stride_t < 0 || k_stride_h < 0 || v_stride_t < 0 || v_stride_h < 0) return KV1B_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || k_stride_t % 4 || k_stride_h % 4 || v_stride_t % 4 || v_stride_h % 4)
    return KV1B_ERR_MISALIGNED;
  if (!aligned(cu_new, 4) || !aligned(start, 4) || !aligned(page_table, 4)) return KV1B_ERR_MISALIGNED;
  // rows of one launch
  if (num_tokens > (1 << 28) || static_cast<int64_t>(num_tokens) * (cache->num_kv_heads + (q ? num_q_heads : 0)) > (1LL << 33))
    return KV1B_ERR_UNSUPPORTED;
  kv1b::PagedAppendParams p;
  memset(&p, 0, sizeof(p));
  if (rope) {
    if (!rope->cos_sin || !positions || rope->num_positions < 1 || rope->rot_dim < 8 || rope->rot_dim > KV1B_HEAD_DIM ||
        rope->axes < 1 || rope->axes > KV1B_ROPE_MAX_AXES || pos_stride < 0 || (rope->axes > 1 && pos_stride > 0 && pos_stride < num_tokens))
      return KV1B_ERR_INVALID_ARG;
    if (rope->rot_dim % 8) return KV1B_ERR_UNSUPPORTED;
    int sum = 0;
    for (int a = 0; a < rope->axes; ++a) {
      if (rope->sections[a] < 0) return KV1B_ERR_INVALID_ARG;
      sum += rope->sections[a];
    }
    if (sum != rope->rot_dim / 2) return KV1B_ERR_INVALID_ARG;
    if (!aligned(rope->cos_sin, 16) || !aligned(positions, 4)) return KV1B_ERR_MISALIGNED;
    p.cos_sin = rope->cos_sin;
    p.cs_rows = rope->num_positions;
    p.rot = rope->rot_dim;
    p.interleaved = rope->interleaved ? 1 : 0;
    p.sec0 = rope->sections[0];
    p.sec01 = p.sec0 + (rope->axes > 1 ? rope->sections[1] : 0);
    p.pos = positions;
    p.pos_stride = pos_stride;
  }
  if (q || q_out) {
    if (!q || !q_out || q_stride_t < 0 || q_stride_h < 0 || qo_stride_t < 0 || qo_stride_h < 0) return KV1B_ERR_INVALID_ARG;
    if (num_q_heads < 1 || num_q_heads > KV1B_PAGED_MAX_HEADS) return KV1B_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(q_out, 16) || q_stride_t % 4 || q_stride_h % 4 || qo_stride_t % 4 || qo_stride_h % 4)
      return KV1B_ERR_MISALIGNED;
    if (num_tokens > 0) {
      // rows are written while others are read: a result row is no other's, nor an input's but its own
      auto rows = [&](const void* ptr, int64_t st, int64_t H, int64_t sh) {
        return Rows{reinterpret_cast<uintptr_t>(ptr), num_tokens, st, H, sh};
      };
      const Rows out = rows(q_out, qo_stride_t, num_q_heads, qo_stride_h);
      const bool in_place = q == q_out && (num_tokens == 1 || q_stride_t == qo_stride_t) && (num_q_heads == 1 || q_stride_h == qo_stride_h);
      const int64_t es = dtype == KV1B_DTYPE_F32 ? 4 : 2;
      if (!rows_apart(out) || (!in_place && rows_meet(out, rows(q, q_stride_t, num_q_heads, q_stride_h), es)) ||
          rows_meet(out, rows(k, k_stride_t, cache->num_kv_heads, k_stride_h), es) ||
          rows_meet(out, rows(v, v_stride_t, cache->num_kv_heads, v_stride_h), es))
        return KV1B_ERR_INVALID_ARG;
    }
    p.q = q;
    p.q_out = q_out;
    p.Hq = num_q_heads;
    p.q_st = q_stride_t;
    p.q_sh = q_stride_h;
    p.qo_st = qo_stride_t;
    p.qo_sh = qo_stride_h;
  }
  if (num_tokens == 0) return KV1B_OK;
  p.c = view(cache);
  p.k = k;
  p.v = v;
  p.k_st = k_stride_t;
  p.k_sh = k_stride_h;
  p.v_st = v_stride_t;
  p.v_sh = v_stride_h;
  p.dtype = dtype;
  p.T = num_tokens;
  p.B = num_seqs;
  p.cu = cu_new;
  p.start = start;
  p.table = page_table;
  p.table_stride = table_stride;
  p.max_pages = max_pages;
  p.groups = num_tokens / 8 + 2 * num_seqs;
  p.sms = num_sms();
  return cuda_status(kv1b_launch_paged_append(p, static_cast<cudaStream_t>(stream)));
}

size_t kv1b_paged_attend_workspace_bytes(const kv1b_paged_t* cache, int32_t num_q_heads) {
  if (!paged_ok(cache) || heads_check(cache, num_q_heads) != KV1B_OK) return 0;
  const size_t G = num_q_heads / cache->num_kv_heads;
  const size_t n = static_cast<size_t>(num_sms()) * ((2 + kv1b::kAttendWarps) * G * kv1b::kPartStride * 4 + 8);  // part, first, spread
  return (n + 255) / 256 * 256;
}

namespace {

// How the batch's queries and the prefix are split over CTAs: the number of token ranges whose waves of
// CTAs take the fewest tile times, a range counted kFixed more for its start and its merge.
kv1b::PagedSharedParams shared_plan(int32_t Hkv, int32_t G, int32_t num_seqs, int64_t max_tokens) {
  constexpr int64_t kFixed = 4;
  kv1b::PagedSharedParams s;
  memset(&s, 0, sizeof(s));
  s.R = num_seqs * G;
  s.two = s.R > 128;
  const int rows = s.two ? 256 : 128;
  s.row_tiles = (s.R + rows - 1) / rows;
  const int64_t tiles = (max_tokens + 127) / 128, units = static_cast<int64_t>(Hkv) * s.row_tiles, sms = num_sms();
  int64_t best = -1;
  for (int64_t n = 1; n <= tiles && n <= kv1b::kMaxSplits; ++n) {
    const int64_t cost = (units * n + sms - 1) / sms * ((tiles + n - 1) / n + kFixed);
    if (best < 0 || cost < best) {
      best = cost;
      s.splits = static_cast<int32_t>(n);
    }
  }
  return s;
}

// Fewer ranges where the SMs that they leave can do the sequences' own tokens meanwhile, as far as the tables'
// widths tell (the lengths are the device's to know: it looks again): 170 against 179 us for 64 sequences of 512
// tokens behind 131,072 (8 kv-heads, 4 heads each), 65 against 77 for 100 tokens behind 30,000.
void side_by_side(kv1b::PagedSharedParams* s, kv1b::PagedAttendParams* p, int32_t Hkv, int64_t max_tokens, int64_t own_units) {
  const int64_t tiles = (max_tokens + 127) / 128, units = static_cast<int64_t>(Hkv) * s->row_tiles, sms = num_sms();
  p->tile_ns = s->two ? kv1b::kTile256Ns : kv1b::kTile128Ns;
  const int64_t after = kv1b::kCtaNs + own_units * kv1b::kUnitNs / sms;
  int64_t best = -1;
  const int32_t most = s->splits;
  for (int32_t n = most; n >= 1; --n) {
    const int64_t left = sms - units * n, waves = (units * n + sms - 1) / sms;
    const int64_t prefix = waves * ((tiles + n - 1) / n * p->tile_ns + kv1b::kPrefixNs);
    const bool beside = left > 0 && kv1b::kCtaNs + own_units * kv1b::kUnitNs / left <= prefix;
    const int64_t cost = beside ? prefix : prefix + after;
    if (best < 0 || cost < best) {
      best = cost;
      s->splits = n;
      p->beside = beside ? static_cast<int32_t>(left) : 0;
    }
  }
  p->splits = s->splits;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Whether the attend's kernel takes the prefix, eight rows of a kv-head at a time and the prefix once for each
// eight, and in how many groups (0: the matrix kernel does).  It starts sooner and costs rows x tiles; measured
// over 8 kv-heads, it against the other, us:
//   rows   64 tiles       504            1,880          6,256 (of all kv-heads)
//   16                                   26 against 35  57 against 73
//   32     14 against 20  22 against 24  35 against 36  102 against 76
//   64     17 against 22  27 against 27  62 against 41  194 against 83
//   128    20 against 25  40 against 33  118 against 49
//   256    30 against 30  74 against 39
// and 47 against 60 for 32 rows of 32 kv-heads, 2,048 tiles, with 300 tokens of each sequence's own.  The prefix's
// length is the device's to know; its table's width stands for it.
int packed_groups(int32_t rows, int32_t Hkv, int64_t max_tokens) {
  const int64_t tiles = Hkv * ((max_tokens + 127) / 128);
  const int64_t most = rows <= 16 ? INT64_MAX : (rows <= 32 ? 65536 : (rows <= 128 ? 32768 : 0));
  return rows * tiles <= most ? (rows + 7) / 8 : 0;
}

// The buffers of a shared call in its workspace; bytes in all.
size_t shared_carve(kv1b::PagedSharedParams* s, kv1b::PagedAttendParams* p, int32_t Hkv, int32_t G, int64_t max_tokens,
                    uint8_t* ws) {
  const size_t rows = static_cast<size_t>(Hkv) * s->R, row = kv1b::kPartStride * 4;
  const size_t packed = packed_groups(s->R, Hkv, max_tokens), n = packed ? 8 : G;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* const here = ws + at;
    at += up256(bytes);
    return here;
  };
  uint8_t* const part = take(static_cast<size_t>(num_sms()) * 2 * n * row);
  uint8_t* const first = take(static_cast<size_t>(num_sms()) * kv1b::kAttendWarps * n * row);
  uint8_t* const whole = take((packed ? 2 : 1) * rows * row);
  uint8_t* const spread = take(static_cast<size_t>(Hkv) * (packed + s->R / G) * 8);
  uint8_t* const pieces = take(packed ? 0 : static_cast<size_t>(Hkv) * s->row_tiles * s->splits * 256 * row);
  uint8_t* const codes = take(packed ? 0 : rows * KV1B_HEAD_DIM);
  uint8_t* const factors = take(packed ? 0 : rows * 8);
  if (p) {
    p->packed = static_cast<int32_t>(packed);
    // Behind the prefix's CTAs, which take nearly every SM, few CTAs do better than short ones: 56 against 66 us
    // for 64 rows a kv-head over 30,000 tokens; with the SMs to themselves, 20 against 26 us the other way.
    if (!packed) p->min_units = 64;
    p->part = reinterpret_cast<float*>(part);
    p->first = reinterpret_cast<float*>(first);
    p->rows = reinterpret_cast<float*>(whole);
    p->spread = reinterpret_cast<int2*>(spread);
    s->pieces = reinterpret_cast<float*>(pieces);
    s->codes = codes;
    s->factors = reinterpret_cast<float2*>(factors);
  }
  return at;
}

}  // namespace

size_t kv1b_paged_shared_workspace_bytes(const kv1b_paged_t* cache, int32_t num_seqs, int32_t num_q_heads,
                                         int32_t max_prefix_pages) {
  if (num_seqs < 1 || num_seqs > KV1B_PAGED_MAX_SEQS || max_prefix_pages < 1) return 0;
  if (!paged_ok(cache) || heads_check(cache, num_q_heads) != KV1B_OK || table_check(cache, 1, 0, 1, max_prefix_pages, true) != KV1B_OK) return 0;
  const int32_t G = num_q_heads / cache->num_kv_heads;
  const int64_t max_tokens = static_cast<int64_t>(max_prefix_pages) * cache->page_tokens;
  kv1b::PagedSharedParams s = shared_plan(cache->num_kv_heads, G, num_seqs, max_tokens);
  return shared_carve(&s, nullptr, cache->num_kv_heads, G, max_tokens, nullptr);
}

static int attend(const kv1b_paged_t* cache, const void* q, int32_t q_dtype, int32_t num_q_heads, float scale,
                  int32_t num_seqs, const int32_t* prefix_pages, int32_t max_prefix_pages, const int32_t* prefix_length,
                  const int32_t* page_table, int64_t table_stride, int32_t max_pages, const int32_t* lengths,
                  int32_t window, int32_t sinks, void* out, void* ws, size_t ws_bytes, void* stream) {
  if (!paged_ok(cache) || !q || !out || !ws || !page_table || !lengths || !dtype_ok(q_dtype)) return KV1B_ERR_INVALID_ARG;
  if (q_dtype == KV1B_DTYPE_F32) return KV1B_ERR_UNSUPPORTED;
  const int hc = heads_check(cache, num_q_heads);
  if (hc != KV1B_OK) return hc;
  const int tc = table_check(cache, num_seqs, table_stride, max_pages, max_prefix_pages, true);
  if (tc != KV1B_OK) return tc;
  if (!(scale == scale) || window < 0 || sinks < 0) return KV1B_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(ws, 256) || !aligned(page_table, 4) || !aligned(lengths, 4) ||
      !aligned(prefix_pages, 4) || !aligned(prefix_length, 4))
    return KV1B_ERR_MISALIGNED;
  // results over the queries, or clear of them: rows are written while others' queries are still read
  const Wide rows = Wide(num_seqs) * num_q_heads * KV1B_HEAD_DIM * 2;
  const Wide apart = Wide(reinterpret_cast<uintptr_t>(out)) - Wide(reinterpret_cast<uintptr_t>(q));
  if (apart != 0 && apart < rows && -apart < rows) return KV1B_ERR_INVALID_ARG;
  if (ws_bytes < (prefix_pages ? kv1b_paged_shared_workspace_bytes(cache, num_seqs, num_q_heads, max_prefix_pages)
                               : kv1b_paged_attend_workspace_bytes(cache, num_q_heads)))
    return KV1B_ERR_WORKSPACE;
  kv1b::PagedAttendParams p;
  memset(&p, 0, sizeof(p));
  p.c = view(cache);
  p.q = q;
  p.q_dtype = q_dtype;
  p.Hq = num_q_heads;
  p.B = num_seqs;
  p.scale = scale;
  p.table = page_table;
  p.table_stride = table_stride;
  p.max_pages = max_pages;
  p.lengths = lengths;
  p.window = window;
  p.sinks = sinks;
  p.prefix_pages = prefix_pages;
  p.prefix_len = prefix_length;
  p.max_prefix_pages = max_prefix_pages;
  p.out = out;
  p.ncta = num_sms();
  // 12, 16, 24 units a CTA: 11.6, 12.2, 12.9 us for 397 tokens of 8 kv-heads; 13.4, 14.0, 16.4 for 16 rows and 15.6,
  // 14.2, 16.7 for 32 rows of each behind a prefix of 1,000.  Where there is more work every SM has a CTA anyway.
  p.min_units = 16;
  p.part = static_cast<float*>(ws);
  p.first = p.part + static_cast<size_t>(p.ncta) * 2 * (num_q_heads / cache->num_kv_heads) * kv1b::kPartStride;
  p.spread = reinterpret_cast<int2*>(p.first + static_cast<size_t>(p.ncta) * kv1b::kAttendWarps * (num_q_heads / cache->num_kv_heads) * kv1b::kPartStride);
  const int32_t G = num_q_heads / cache->num_kv_heads;
  if (!prefix_pages) return cuda_status(kv1b_launch_paged_attend(p, G, static_cast<cudaStream_t>(stream)));
  const int64_t max_tokens = static_cast<int64_t>(max_prefix_pages) * cache->page_tokens;
  kv1b::PagedSharedParams s = shared_plan(cache->num_kv_heads, G, num_seqs, max_tokens);
  shared_carve(&s, &p, cache->num_kv_heads, G, max_tokens, static_cast<uint8_t*>(ws));
  if (!p.packed) {
    const int64_t blocks = static_cast<int64_t>(max_pages) * (cache->page_tokens / KV1B_PAGED_BLOCK_TOKENS);
    side_by_side(&s, &p, cache->num_kv_heads, max_tokens, num_seqs * (blocks + kv1b::kSegUnits) * cache->num_kv_heads);
  }
  return cuda_status(kv1b_launch_paged_shared(p, s, G, static_cast<cudaStream_t>(stream)));
}

int kv1b_paged_attend(const kv1b_paged_t* cache, const void* q, int32_t q_dtype, int32_t num_q_heads, float scale,
                      int32_t num_seqs, const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                      const int32_t* lengths, int32_t window, int32_t sinks, void* out, void* ws, size_t ws_bytes,
                      void* stream) {
  return attend(cache, q, q_dtype, num_q_heads, scale, num_seqs, nullptr, 0, nullptr, page_table, table_stride, max_pages,
                lengths, window, sinks, out, ws, ws_bytes, stream);
}

int kv1b_paged_attend_shared(const kv1b_paged_t* cache, const void* q, int32_t q_dtype, int32_t num_q_heads, float scale,
                             int32_t num_seqs, const int32_t* prefix_pages, int32_t max_prefix_pages,
                             const int32_t* prefix_length, const int32_t* page_table, int64_t table_stride,
                             int32_t max_pages, const int32_t* lengths, void* out, void* ws, size_t ws_bytes,
                             void* stream) {
  if (!prefix_pages || !prefix_length || max_prefix_pages < 1) return KV1B_ERR_INVALID_ARG;
  return attend(cache, q, q_dtype, num_q_heads, scale, num_seqs, prefix_pages, max_prefix_pages, prefix_length, page_table,
                table_stride, max_pages, lengths, 0, 0, out, ws, ws_bytes, stream);
}

}  // extern "C"

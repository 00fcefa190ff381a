// kv1b_paged_append.cu -- encode new tokens into a paged cache, with the rotary position applied to
// the key on the way in and, in the same call, to the queries.
//
// Rotary embedding, pair i of a row: a' = fl(fl(a cos) - fl(b sin)), b' = fl(fl(b cos) + fl(a sin)) in
// fp32, cos and sin from the caller's table at the position of the pair's axis.  The turned key goes to
// the encoder in fp32 without a rounding in between.  Encoder: as kv1b_encode.cu (rotation, sign bits,
// N and 1/C kept as their product, 4-bit values), in the same fixed orders, so every stored bit is
// reproducible; values are first limited to the finite binary16 range and a group's scale is lowered
// by one step where min + 15 scale would leave it, so that a reader may expand values to binary16.
//
// Work is split in groups of 8 aligned tokens of one sequence and kv-head: the tokens that share a
// 32-bit word of every channel's codes, so one warp owns every word it rewrites.
#include "kv1b_device.cuh"
#include "kv1b_encode_q4.cuh"
#include "kv1b_paged.h"
#include "kv1b_paged_device.cuh"

namespace kv1b {
namespace paged {

constexpr float kF16Max = 65504.0f;

__device__ __forceinline__ float limit_value(float v) {
  return v == v ? fminf(fmaxf(v, -kF16Max), kF16Max) : 0.0f;
}

// Sequence, first position and positions of the group with index `gi`.  Sequence b owns the indices
// from cu[b] / 8 + 2 b on: its n tokens touch at most floor(n / 8) + 2 groups, so the ranges never
// overlap, and both the sequence and the group follow from cu without a prefix sum.
struct Group {
  int b;
  int row0;          // row of the sequence's first new token
  int64_t L0, L1;    // positions [L0, L1) are new
  int64_t g0;        // first position of the group
  bool any;
};

__device__ __forceinline__ Group find_group(const PagedAppendParams& p, int gi) {
  const int lane = threadIdx.x & 31;
  // the last sequence whose first index is <= gi: two rounds of 32 probes (B <= 1024)
  int lo = 0;
  if (p.B > 32) {
    const int step = (p.B + 31) / 32;
    const int b = lane * step;
    const bool le = b < p.B && (__ldg(p.cu + b) >> 3) + 2 * b <= gi;
    const unsigned m = __ballot_sync(kFull, le);
    lo = m ? (31 - __clz(m)) * step : 0;
  }
  const int bb = lo + lane;
  const int mine = bb < p.B ? __ldg(p.cu + bb) : 0x7fffffff;
  const bool le2 = bb < p.B && (mine >> 3) + 2 * bb <= gi;
  const unsigned m2 = __ballot_sync(kFull, le2);
  const int off = m2 ? 31 - __clz(m2) : 0;
  Group g;
  g.b = lo + off;
  g.row0 = __shfl_sync(kFull, mine, off);
  const int row1 = __ldg(p.cu + g.b + 1);
  const int first = __ldg(p.start + g.b);
  const bool ok = g.row0 >= 0 && row1 >= g.row0 && row1 <= p.T && first >= 0;
  if (!ok && lane == 0 && p.c.status) atomicOr(p.c.status, KV1B_STATUS_BAD_INDEX);
  g.L0 = first;
  g.L1 = g.L0 + (ok ? row1 - g.row0 : 0);
  g.g0 = ((g.L0 >> 3) + (gi - ((g.row0 >> 3) + 2 * g.b))) << 3;
  g.any = ok && g.g0 < g.L1 && g.g0 + 8 > g.L0;
  return g;
}

// Whether the sequences' rows ascend, by a warp that has nothing else to do.  Where they do not, find_group may pass by a
// sequence, the one at fault among them, so nobody else would report it.
__device__ __forceinline__ void check_rows(const PagedAppendParams& p) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  for (int b = lane; b < p.B; b += 32) {
    const int row0 = __ldg(p.cu + b), row1 = __ldg(p.cu + b + 1);
    bad |= row0 < 0 || row1 < row0 || row1 > p.T;
  }
  if (__any_sync(kFull, bad) && lane == 0 && p.c.status) atomicOr(p.c.status, KV1B_STATUS_BAD_INDEX);
}

// The block of position `pos` of sequence b and kv-head h, or null (flagged) if its page is not there.
__device__ __forceinline__ uint8_t* block_of(const PagedAppendParams& p, int b, int h, int64_t pos) {
  const int64_t blk = pos >> 5;
  const int64_t lp = blk >> p.c.bpp_shift;
  const int page = lp < p.max_pages ? __ldg(p.table + b * p.table_stride + lp) : -1;
  if (page < 0 || page >= p.c.num_pages) return nullptr;
  const int64_t in = blk & ((1 << p.c.bpp_shift) - 1);
  return p.c.pages + ((((static_cast<int64_t>(page) * p.c.Hkv + h) << p.c.bpp_shift) + in) * kBlkBytes);
}

// The rotary table's row of a pair: the position on the pair's axis.
__device__ __forceinline__ const float* factor_row(const PagedAppendParams& p, const int (&ps)[3], int pair) {
  return p.cos_sin + static_cast<int64_t>(pair < p.sec0 ? ps[0] : (pair < p.sec01 ? ps[1] : ps[2])) * p.rot;
}

// Positions of row t on the three axes (the same for unused ones); false if one is outside the table.
__device__ __forceinline__ bool positions(const PagedAppendParams& p, int64_t t, int (&ps)[3]) {
  const int half = p.rot >> 1;
  ps[0] = __ldg(p.pos + t);
  ps[1] = p.sec0 < half ? __ldg(p.pos + p.pos_stride + t) : ps[0];
  ps[2] = p.sec01 < half ? __ldg(p.pos + 2 * p.pos_stride + t) : ps[0];
  const int n = p.cs_rows;
  return ps[0] >= 0 && ps[0] < n && ps[1] >= 0 && ps[1] < n && ps[2] >= 0 && ps[2] < n;
}

__device__ __forceinline__ void store4(void* base, int64_t off, int dtype, const float x[4]) {
  if (dtype == KV1B_DTYPE_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(base) + off) = make_float4(x[0], x[1], x[2], x[3]);
    return;
  }
  uint32_t h[4];
  #pragma unroll
  for (int r = 0; r < 4; ++r)
    h[r] = dtype == KV1B_DTYPE_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x[r])) : __half_as_ushort(__float2half_rn(x[r]));
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + off) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// Rotary turn of one row held by a warp (lane l: channels 4l .. 4l + 3).  rot is a multiple of 8, so in
// the half-split form the partner of a lane's channels are another lane's four.
__device__ __forceinline__ void rope_warp(const PagedAppendParams& p, const int (&ps)[3], float (&x)[4]) {
  const int lane = threadIdx.x & 31, half = p.rot >> 1;
  const int c0 = 4 * lane;
  const bool in = c0 < p.rot;
  if (p.interleaved) {
    if (!in) return;
    #pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = 2 * lane + u;
      const float* row = factor_row(p, ps, i);
      const float c = __ldg(row + i), s = __ldg(row + half + i);
      const float a = x[2 * u], b = x[2 * u + 1];
      x[2 * u] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
      x[2 * u + 1] = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    }
    return;
  }
  const bool upper = c0 >= half;
  const int src = in ? (upper ? lane - (half >> 2) : lane + (half >> 2)) : lane;
  #pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float o = __shfl_sync(kFull, x[r], src);
    if (in) {
      const int i = c0 + r - (upper ? half : 0);
      const float* row = factor_row(p, ps, i);
      const float c = __ldg(row + i), s = __ldg(row + half + i);
      x[r] = upper ? __fadd_rn(__fmul_rn(x[r], c), __fmul_rn(o, s)) : __fsub_rn(__fmul_rn(x[r], c), __fmul_rn(o, s));
    }
  }
}

// Channels of a row as they lie in memory, as fp32, and back: two from a word, four from a Four.
__device__ __forceinline__ float2 as_floats(uint32_t raw, int dtype) {
  if (dtype == KV1B_DTYPE_BF16) return make_float2(__uint_as_float(raw << 16), __uint_as_float(raw & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&raw));
}
__device__ __forceinline__ uint32_t as_word(float a, float b, int dtype) {
  if (dtype == KV1B_DTYPE_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <int DT> struct Four {
  typedef uint2 Raw;
  static __device__ __forceinline__ void get(Raw w, float* x) {
    const float2 a = as_floats(w.x, DT), b = as_floats(w.y, DT);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
  }
  static __device__ __forceinline__ Raw put(const float* x) { return make_uint2(as_word(x[0], x[1], DT), as_word(x[2], x[3], DT)); }
};
template <> struct Four<KV1B_DTYPE_F32> {
  typedef float4 Raw;
  static __device__ __forceinline__ void get(Raw w, float* x) { x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w; }
  static __device__ __forceinline__ Raw put(const float* x) { return make_float4(x[0], x[1], x[2], x[3]); }
};

// a b for two pairs, each product rounded by itself.  (The assembler joins a product of pairs with a sum of
// pairs behind it into one fma, also where both say .rn; it leaves single products alone.)
__device__ __forceinline__ uint64_t products(uint64_t a, uint64_t b) {
  float a0, a1, b0, b1;
  unpair(a, a0, a1);
  unpair(b, b0, b1);
  return pair(__fmul_rn(a0, b0), __fmul_rn(a1, b1));
}

// Query rows [h0, h1) of token t by the calling warp, a row by 16 lanes.  A lane holds four pairs of each of
// its rows, so that nothing is exchanged (channels a .. a + 3 and b .. b + 3: a row's pairs in order, then what
// is not turned); the token's factors are read once for all rows, sixteen of which are in flight.
template <int DT, bool INTERLEAVED>
__device__ __forceinline__ void query_rows(const PagedAppendParams& p, int64_t t, int h0, int h1) {
  typedef typename Elem<DT>::T E;
  typedef typename Four<DT>::Raw Raw;
  const int lane = threadIdx.x & 31, half = p.rot >> 1, first = 4 * (lane & 15);  // pairs first .. first + 3
  const bool in = p.cos_sin && first < half;
  int a = 2 * first, b = a + 4;
  float cs[4] = {1.0f, 1.0f, 1.0f, 1.0f}, sn[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (p.cos_sin) {
    int ps[3];
    if (!positions(p, t, ps)) {
      if (lane == 0 && p.c.status) atomicOr(p.c.status, KV1B_STATUS_BAD_INDEX);
      return;
    }
    if (in) {
      if (!INTERLEAVED) a = first, b = first + half;
      #pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* row = factor_row(p, ps, first + i) + first + i;
        cs[i] = __ldg(row);
        sn[i] = __ldg(row + half);
      }
    }
  }
  const E* q = static_cast<const E*>(p.q) + t * p.q_st;
  E* out = static_cast<E*>(p.q_out) + t * p.qo_st;
  constexpr int kSteps = 8;  // two rows each
  #pragma unroll 1
  for (int left = h1 - h0, h = h0 + (lane >> 4); left > 0; left -= 2 * kSteps, h += 2 * kSteps) {  // alike for both rows' lanes
    Raw ra[kSteps], rb[kSteps];
    #pragma unroll
    for (int k = 0; k < kSteps; ++k) {  // behind the last row: it again
      const E* row = q + min(h + 2 * k, h1 - 1) * p.q_sh;
      ra[k] = *reinterpret_cast<const Raw*>(row + a);
      rb[k] = *reinterpret_cast<const Raw*>(row + b);
    }
    #pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      float x[8];
      Four<DT>::get(ra[k], x);
      Four<DT>::get(rb[k], x + 4);
      #pragma unroll
      for (int i = 0; i < 4; ++i) {  // pair i: its members in x
        float& u = x[INTERLEAVED ? 2 * i : i];
        float& v = x[INTERLEAVED ? 2 * i + 1 : 4 + i];
        const float un = __fsub_rn(__fmul_rn(u, cs[i]), __fmul_rn(v, sn[i]));
        v = __fadd_rn(__fmul_rn(v, cs[i]), __fmul_rn(u, sn[i]));
        u = un;
      }
      const Raw ta = Four<DT>::put(x), tb = Four<DT>::put(x + 4);
      if (h + 2 * k < h1) {  // what is not turned goes through as it is
        E* row = out + (h + 2 * k) * p.qo_sh;
        *reinterpret_cast<Raw*>(row + a) = in ? ta : ra[k];
        *reinterpret_cast<Raw*>(row + b) = in ? tb : rb[k];
      }
    }
  }
}

// One query row by the calling warp.
__device__ __forceinline__ void query_row(const PagedAppendParams& p, int64_t t, int h) {
  const int lane = threadIdx.x & 31;
  float x[4];
  load_query(p.q, t * p.q_st + h * p.q_sh + 4 * lane, p.dtype, x);
  if (p.cos_sin) {
    int ps[3];
    if (!positions(p, t, ps)) {
      if (lane == 0 && p.c.status) atomicOr(p.c.status, KV1B_STATUS_BAD_INDEX);
      return;
    }
    rope_warp(p, ps, x);
  }
  store4(p.q_out, t * p.qo_st + h * p.qo_sh + 4 * lane, p.dtype, x);
}

// Scale and min of a value group from its limited extremes.
__device__ __forceinline__ void group_scale(float mn, float mx, uint32_t* scale_bits, uint32_t* min_bits, bool walk) {
  int sat = 0;
  *min_bits = half_round_down(mn, &sat);
  const float mf = __half2float(__ushort_as_half(static_cast<unsigned short>(*min_bits)));
  uint32_t s = walk ? half_scale_up(mx, mf, &sat) : half_scale_up_fast(mx, mf, &sat);
  // one step down where the top code would leave the binary16 range: exact in fp64
  if (static_cast<double>(mf) + 15.0 * half_bits_to_double(s) > 65504.0) --s;
  *scale_bits = s;
}

// ---------------------------------------------------------------------------------------------
// Decode form: one warp per (group, kv-head) and half (key or value), 32 lanes x 4 channels, the
// group's new tokens one after another (one, in a decode step); then one warp per query row, and one more.  The
// chain of dependent loads (cu, start, page, old words) is what a step waits for.
__global__ void __launch_bounds__(128) paged_append_token_kernel(const PagedAppendParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int64_t kv_units = 2LL * p.groups * p.c.Hkv;
  if (unit >= kv_units) {
    const int64_t r = unit - kv_units, query_rows = p.q ? static_cast<int64_t>(p.T) * p.Hq : 0;
    if (r == query_rows) check_rows(p);
    if (r >= query_rows) return;
    const int64_t t = r / p.Hq;
    if (t >= __ldg(p.cu + p.B)) return;  // rows behind the last sequence
    query_row(p, t, static_cast<int>(r - t * p.Hq));
    return;
  }
  const int h = static_cast<int>(unit % p.c.Hkv);
  const int64_t gv = unit / p.c.Hkv;
  const bool value = (gv & 1) != 0;
  const Group g = find_group(p, static_cast<int>(gv >> 1));
  if (!g.any) return;
  int flags = 0;
  uint8_t* blk = block_of(p, g.b, h, g.g0);
  const int w = static_cast<int>(g.g0 & 31) >> 3;  // the group's code word of each row
  uint32_t* words = reinterpret_cast<uint32_t*>(blk + kBlkOffCodes) + w;
  uint32_t cw[4];
  if (blk && value) {
    #pragma unroll
    for (int r = 0; r < 4; ++r) cw[r] = words[(4 * lane + r) * 4];
  }
  bool wrote = false;
  #pragma unroll 1
  for (int64_t pos = g.g0 < g.L0 ? g.L0 : g.g0; pos < g.L1 && pos < g.g0 + 8; ++pos) {
    const int64_t t = g.row0 + (pos - g.L0);
    const int tok = static_cast<int>(pos & 31);
    int ps[3] = {0, 0, 0};
    const bool ok = (!p.cos_sin || positions(p, t, ps)) && blk;
    if (!ok) {
      flags |= KV1B_STATUS_BAD_INDEX;
      continue;
    }
    float x[4];
    if (!value) {
      load4(p.k, t * p.k_st + h * p.k_sh + 4 * lane, p.dtype, x);
      if (p.cos_sin) rope_warp(p, ps, x);
      float sq[4], ab[4];
      #pragma unroll
      for (int r = 0; r < 4; ++r) {
        sq[r] = __fmul_rn(x[r], x[r]);
        if (!isfinite(x[r])) flags |= KV1B_STATUS_NONFINITE;
      }
      const float nrm = __fsqrt_rn(tree_sum128(sq));
      rotate_rounds(x, p.c.signs);
      uint32_t nib = 0;
      #pragma unroll
      for (int r = 0; r < 4; ++r) {
        nib |= static_cast<uint32_t>(x[r] >= 0.0f) << r;
        ab[r] = fabsf(x[r]);
      }
      const uint32_t word = pack_word(nib);
      const float sabs = tree_sum128(ab);
      const float cinv = (sabs > 0.0f) ? __fdiv_rn(__fmul_rn(static_cast<float>(kD), nrm), sabs) : 1.0f;
      const int row = 8 * ((tok >> 1) & 3) + 2 * (tok >> 3) + (tok & 1);
      if ((lane & 7) == 0) reinterpret_cast<uint32_t*>(blk)[row * 4 + (lane >> 3)] = word;
      if (lane == 0) reinterpret_cast<float*>(blk + kBlkOffNc)[tok] = __fmul_rn(nrm, cinv);
    } else {
      load4(p.v, t * p.v_st + h * p.v_sh + 4 * lane, p.dtype, x);
      #pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (!isfinite(x[r])) flags |= KV1B_STATUS_NONFINITE;
        else if (fabsf(x[r]) > kF16Max) flags |= KV1B_STATUS_FP16_SATURATED;
        x[r] = limit_value(x[r]);
      }
      float mn = fminf(fminf(x[0], x[1]), fminf(x[2], x[3]));
      float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      #pragma unroll
      for (int m = 1; m <= 4; m <<= 1) {
        mn = fminf(mn, __shfl_xor_sync(kFull, mn, m));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, m));
      }
      uint32_t sb, mb;
      group_scale(mn, mx, &sb, &mb, true);
      const float sf = __half2float(__ushort_as_half(static_cast<unsigned short>(sb)));
      const float mf = __half2float(__ushort_as_half(static_cast<unsigned short>(mb)));
      const int j = tok & 7;
      const int sh = 4 * ((j >> 1) + 4 * (j & 1));
      #pragma unroll
      for (int r = 0; r < 4; ++r) {
        uint32_t c = 0;
        if (sf > 0.0f) {
          const float fl = floorf(__fadd_rn(__fdiv_rn(__fsub_rn(x[r], mf), sf), 0.5f));
          c = !(fl > 0.0f) ? 0u : (fl >= 15.0f ? 15u : static_cast<uint32_t>(fl));
        }
        cw[r] = (cw[r] & ~(0xfu << sh)) | (c << sh);
      }
      if ((lane & 7) == 0) {
        reinterpret_cast<uint16_t*>(blk + kBlkOffScale)[32 * (lane >> 3) + tok] = static_cast<uint16_t>(sb);
        reinterpret_cast<uint16_t*>(blk + kBlkOffMin)[32 * (lane >> 3) + tok] = static_cast<uint16_t>(mb);
      }
      wrote = true;
    }
  }
  if (wrote) {
    #pragma unroll
    for (int r = 0; r < 4; ++r) words[(4 * lane + r) * 4] = cw[r];
  }
  flags = static_cast<int>(__reduce_or_sync(kFull, static_cast<unsigned>(flags)));
  if (lane == 0 && flags && p.c.status) atomicOr(p.c.status, flags);
}

// ---------------------------------------------------------------------------------------------
// Prefill form: one warp per group and a few kv-heads, one after another, 4 lanes per token
// (kv1b_encode_q4.cuh).  The rows of the next head are copied to shared memory while this one's are worked on:
// the key's as soon as its values are in registers, the value's likewise (loads into registers instead, with
// 20 warps an SM and nothing ahead of them, left the issue slots idle for a third of the time).  The group's
// rotary factors are staged too, a row per token (cos, then sin).
// Rows lie so far apart that lanes (token, part) read 32 banks: keys one element at a time, values 8
// channels at a time, part j beginning with its j-th eight.
constexpr int kFactorRow = kD + 4;
constexpr int kQueryHeads = 32;  // query rows of a token that a warp turns
template <int DT> struct Prefill {
  static constexpr int kEs = DT == KV1B_DTYPE_F32 ? 4 : 2;
  static constexpr int kWarps = DT == KV1B_DTYPE_F32 ? 2 : 4;
  static constexpr int kKeyRow = kD * kEs + (DT == KV1B_DTYPE_F32 ? 16 : 8);
  static constexpr int kValueRow = kD * kEs + 16;
  static constexpr int kStage = 8 * (kKeyRow + kValueRow);  // bytes per warp
};

// Rows of a group's eight tokens (row i where bit i of `on` is set, zeros elsewhere) to shared memory; `first`:
// the first of them that is set.
template <int BYTES>
__device__ __forceinline__ void copy_rows(uint32_t dst, int row_bytes, const uint8_t* first, int64_t stride, uint32_t on) {
  const int lane = threadIdx.x & 31, skip = __ffs(on) - 1;
  #pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t d = dst + i * row_bytes + lane * BYTES;
    const bool is = (on >> i) & 1u;
    const uint8_t* s = first + (is ? (i - skip) * stride : 0) + lane * BYTES;
    if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(s), "r"(is ? 16 : 0) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(d), "l"(s), "r"(is ? 8 : 0) : "memory");
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// Half-split pairs (c, c + 4 HQ) both sit in the lane: x[r] and x[r + HQ].
template <int HQ>
__device__ __forceinline__ void rope_in_lane(float (&x)[32], const float* cs, const float* sn, int j) {
  #pragma unroll
  for (int r = 0; r < HQ; ++r) {
    const float c = cs[j + 4 * r], s = sn[j + 4 * r], a = x[r], b = x[r + HQ];
    x[r] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    x[r + HQ] = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  }
}

// rotate_q4 (kv1b_encode_q4.cuh) with the butterflies that join two registers done for two of them at once:
// the same sums and differences, a - c as fma(-1, c, a).
__device__ __forceinline__ void rotate_pairs(float (&x)[32], uint32_t smask, int j) {
  #pragma unroll
  for (int r = 0; r < 32; ++r)  // D: flip the sign bit where the mask has a 1
    x[r] = __int_as_float(__float_as_int(x[r]) ^ static_cast<int>((smask << (31 - r)) & 0x80000000u));
  #pragma unroll
  for (int h = 1; h <= 2; h <<= 1) {
    const float sgn = (j & h) ? -1.0f : 1.0f;  // the lane of the pair's upper element forms a - c
    const uint64_t s2 = pair(sgn, sgn);
    #pragma unroll
    for (int r = 0; r < 32; r += 2)
      unpair(fma2(s2, pair(x[r], x[r + 1]), pair(__shfl_xor_sync(kFull, x[r], h), __shfl_xor_sync(kFull, x[r + 1], h))), x[r], x[r + 1]);
  }
  #pragma unroll
  for (int r = 0; r < 32; r += 2) {
    const float a = x[r], c = x[r + 1];
    x[r] = __fadd_rn(a, c);
    x[r + 1] = __fsub_rn(a, c);
  }
  const uint64_t minus = pair(-1.0f, -1.0f);
  #pragma unroll
  for (int hr = 2; hr <= 16; hr <<= 1) {
    #pragma unroll
    for (int r = 0; r < 32; r += 2) {
      if (r & hr) continue;
      const uint64_t a = pair(x[r], x[r + 1]), c = pair(x[r + hr], x[r + hr + 1]);
      unpair(add2(a, c), x[r], x[r + 1]);
      unpair(fma2(minus, c, a), x[r + hr], x[r + hr + 1]);
    }
  }
}

// tree_sum_q4 of the squares.
__device__ __forceinline__ float square_sum_pairs(const float (&x)[32]) {
  uint64_t a[16];
  #pragma unroll
  for (int i = 0; i < 16; ++i) a[i] = products(pair(x[2 * i], x[2 * i + 1]), pair(x[2 * i], x[2 * i + 1]));
  #pragma unroll
  for (int n = 8; n >= 1; n >>= 1)
    #pragma unroll
    for (int i = 0; i < n; ++i) a[i] = add2(a[i], a[i + n]);
  float s0, s1;
  unpair(a[0], s0, s1);
  float s = __fadd_rn(s0, s1);
  s = __fadd_rn(s, __shfl_xor_sync(kFull, s, 2));  // h = 2: lanes j < 2 add lane j + 2
  s = __fadd_rn(s, __shfl_xor_sync(kFull, s, 1));  // h = 1: lane 0 adds lane 1
  return __shfl_sync(kFull, s, (threadIdx.x & 31) & ~3);
}

// The token's word j of bits x >= 0 from its four lanes: each lane shifts its 32 sign bits into a mask, spreads
// a byte of it (channels j, j + 4, .. of a word) to every fourth bit, and the four lanes swap.
__device__ __forceinline__ uint32_t sign_word(const float (&x)[32], int j) {
  uint32_t m = 0u;  // bit r: x[r] negative
  #pragma unroll
  for (int r = 30; r >= 0; r -= 2) {
    float a, b;
    unpair(add2(pair(x[r], x[r + 1]), pair(0.0f, 0.0f)), a, b);  // -0 counts as >= 0
    m = __funnelshift_l(__float_as_uint(b), m, 1);
    m = __funnelshift_l(__float_as_uint(a), m, 1);
  }
  m = ~m;
  uint32_t w[4];  // this lane's bits of the token's words
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t v = (m >> (8 * i)) & 0xFFu;
    v = (v | (v << 12)) & 0x000F000Fu;
    v = (v | (v << 6)) & 0x03030303u;
    v = (v | (v << 3)) & 0x11111111u;
    w[i] = v << j;
  }
  // lanes j and j ^ 2 share words 0, 1 against 2, 3; then j and j ^ 1
  const bool up = (j & 2) != 0, odd = (j & 1) != 0;
  const uint32_t k0 = (up ? w[2] : w[0]) | __shfl_xor_sync(kFull, up ? w[0] : w[2], 2);
  const uint32_t k1 = (up ? w[3] : w[1]) | __shfl_xor_sync(kFull, up ? w[1] : w[3], 2);
  return (odd ? k1 : k0) | __shfl_xor_sync(kFull, odd ? k0 : k1, 1);
}

__device__ __forceinline__ float min3_nan(float a, float b, float c) {
  float d;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <int DT>
__global__ void __launch_bounds__(32 * Prefill<DT>::kWarps, 20 / Prefill<DT>::kWarps) paged_append_prefill_kernel(const PagedAppendParams p, const uint32_t kv_share,
                                                                                       const int heads_per_warp) {
  typedef typename Elem<DT>::T T;
  typedef Prefill<DT> F;
  __shared__ __align__(16) uint8_t s_rows[F::kWarps][F::kStage];
  __shared__ __align__(16) float s_factors[F::kWarps][8 * kFactorRow];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tau = lane >> 2, j = lane & 3;
  // A block behind the others, which costs 32,768 tokens 155.2 against 154.5 us.  (The check by a warp behind the groups
  // took 159.4 against 150.6, as a call 181.7 against 154.4.)
  if (blockIdx.x == gridDim.x - 1) {
    if (warp == 0) check_rows(p);
    return;
  }
  // Blocks of keys and values, which are bound by their instructions, and blocks of queries, by memory,
  // are spread evenly among one another: both kinds run on every SM at all times.  kv_share is the keys' share
  // of the blocks in units of 2^-32, rounded up (0: all), and block u theirs where its multiple passes a whole.
  const uint32_t u = blockIdx.x, kv0 = kv_share ? __umulhi(u, kv_share) : u;
  if (kv_share && __umulhi(u + 1, kv_share) == kv0) {
    const uint32_t chunks = (p.Hq + kQueryHeads - 1) / kQueryHeads;
    const uint32_t unit = (u - kv0) * F::kWarps + warp, t = unit / chunks;
    if (t >= static_cast<uint32_t>(p.T) || static_cast<int>(t) >= __ldg(p.cu + p.B)) return;
    const int h0 = static_cast<int>(unit - t * chunks) * kQueryHeads;
    if (p.interleaved) query_rows<DT, true>(p, t, h0, min(h0 + kQueryHeads, p.Hq));
    else query_rows<DT, false>(p, t, h0, min(h0 + kQueryHeads, p.Hq));
    return;
  }
  const uint32_t head_chunks = (p.c.Hkv + heads_per_warp - 1) / heads_per_warp;
  const int gi = static_cast<int>(kv0 / head_chunks) * F::kWarps + warp;
  if (gi >= p.groups) return;
  int h = static_cast<int>(kv0 % head_chunks) * heads_per_warp;
  const int h_end = min(h + heads_per_warp, p.c.Hkv);
  const Group g = find_group(p, gi);
  if (!g.any) return;
  const int64_t pos = g.g0 + tau;
  const bool is_new = pos >= g.L0 && pos < g.L1;
  const int64_t t = g.row0 + (pos - g.L0);
  uint8_t* blk = block_of(p, g.b, h, g.g0);
  int flags = 0;
  int ps[3] = {0, 0, 0};
  bool on = is_new && blk;
  if (on && p.cos_sin) on = positions(p, t, ps);
  if (is_new && !on) flags |= KV1B_STATUS_BAD_INDEX;
  const int tok = static_cast<int>(pos & 31);
  const uint32_t onb = __ballot_sync(kFull, on && j == 0);  // bit 4 tau
  if (onb == 0u) {
    flags = static_cast<int>(__reduce_or_sync(kFull, static_cast<unsigned>(flags)));
    if (lane == 0 && flags && p.c.status) atomicOr(p.c.status, flags);
    return;
  }
  uint32_t on8 = 0u, keep = 0xFFFFFFFFu;  // bit per token; nibbles of a code word whose tokens are not written
  #pragma unroll
  for (int i = 0; i < 8; ++i)
    if (onb & (1u << (4 * i))) {
      on8 |= 1u << i;
      keep &= ~(0xFu << (4 * ((i >> 1) + 4 * (i & 1))));
    }

  const uint32_t rows = smem_u32(s_rows[warp]);
  const int64_t t0 = g.row0 + (g.g0 - g.L0) + (__ffs(on8) - 1);  // the first written token
  auto copy_keys = [&](int hh) {
    copy_rows<4 * F::kEs>(rows, F::kKeyRow, static_cast<const uint8_t*>(p.k) + (t0 * p.k_st + hh * p.k_sh) * F::kEs, p.k_st * F::kEs, on8);
  };
  auto copy_values = [&](int hh) {
    copy_rows<4 * F::kEs>(rows + 8 * F::kKeyRow, F::kValueRow, static_cast<const uint8_t*>(p.v) + (t0 * p.v_st + hh * p.v_sh) * F::kEs,
                          p.v_st * F::kEs, on8);
  };
  copy_keys(h);
  copy_values(h);
  const int half = p.rot >> 1;
  float* const cs = s_factors[warp] + tau * kFactorRow;  // of token tau, brought by its four lanes
  float* const sn = cs + half;
  if (p.cos_sin && on) {
    if (((p.sec0 | p.sec01) & 3) == 0) {  // four pairs behind one another are of one axis
      #pragma unroll 4
      for (int i = 4 * j; i < half; i += 16) {
        const float* row = factor_row(p, ps, i) + i;
        *reinterpret_cast<float4*>(cs + i) = __ldg(reinterpret_cast<const float4*>(row));
        *reinterpret_cast<float4*>(sn + i) = __ldg(reinterpret_cast<const float4*>(row + half));
      }
    } else {
      #pragma unroll 1
      for (int i = j; i < half; i += 4) {
        const float* row = factor_row(p, ps, i) + i;
        cs[i] = __ldg(row);
        sn[i] = __ldg(row + half);
      }
    }
  }
  const float f0 = p.c.signs[0], f1 = p.c.signs[kD], f2 = p.c.signs[2 * kD];
  const int rounds = f0 == 0.0f ? 0 : (f1 == 0.0f ? 1 : (f2 == 0.0f ? 2 : 3));
  const uint32_t smask0 = sign_mask(p.c.signs, 0, j);

  #pragma unroll 1
  for (; h < h_end; ++h, blk += static_cast<int64_t>(kBlkBytes) << p.c.bpp_shift) {
  {  // ---- key: lane j holds channels j + 4 r
    const T* krow = reinterpret_cast<const T*>(s_rows[warp] + tau * F::kKeyRow);
    asm volatile("cp.async.wait_group 1;" ::: "memory");  // the value's rows may still be under way
    __syncwarp();
    float x[32];
    #pragma unroll
    for (int r = 0; r < 32; ++r) x[r] = Elem<DT>::get(krow[j + 4 * r]);
    if (p.cos_sin) {
      if (p.interleaved) {  // the partner of channel c is c ^ 1, lane j ^ 1
        #pragma unroll
        for (int r = 0; r < 32; ++r) {
          if (4 * r >= p.rot) break;  // rot is a multiple of 8
          const float o = __shfl_xor_sync(kFull, x[r], 1);
          const int i = (j >> 1) + 2 * r;
          const float a = __fmul_rn(x[r], cs[i]), b = __fmul_rn(o, sn[i]);
          x[r] = (j & 1) ? __fadd_rn(a, b) : __fsub_rn(a, b);
        }
      } else if (half == 64) {
        rope_in_lane<16>(x, cs, sn, j);
      } else if (half == 32) {
        rope_in_lane<8>(x, cs, sn, j);
      } else if (half == 16) {
        rope_in_lane<4>(x, cs, sn, j);
      } else if (half == 48) {
        rope_in_lane<12>(x, cs, sn, j);
      } else if (on) {  // other widths: the partner is read again
        #pragma unroll
        for (int r = 0; r < 32; ++r) {
          const int c = j + 4 * r;
          if (c < p.rot) {
            const bool upper = c >= half;
            const int i = upper ? c - half : c;
            const float o = Elem<DT>::get(krow[upper ? c - half : c + half]);
            const float a = __fmul_rn(x[r], cs[i]), b = __fmul_rn(o, sn[i]);
            x[r] = upper ? __fadd_rn(a, b) : __fsub_rn(a, b);
          }
        }
      }
      if (!on) {  // a place without a token: nothing of it is kept, but it takes part in the exchanges
        #pragma unroll
        for (int r = 0; r < 32; ++r) x[r] = 0.0f;
      }
    }
    __syncwarp();
    if (h + 1 < h_end) copy_keys(h + 1);
    else asm volatile("cp.async.commit_group;" ::: "memory");
    const float squares = square_sum_pairs(x);
    const float nrm = __fsqrt_rn(squares);
    bool fin = true;
    if (!isfinite(squares)) {  // an entry is not finite, or its square is not
      #pragma unroll
      for (int r = 0; r < 32; ++r) fin &= isfinite(x[r]);
      flags |= fin ? 0 : KV1B_STATUS_NONFINITE;
    }
    #pragma unroll 1
    for (int rd = 0; rd < rounds; ++rd) rotate_pairs(x, rd == 0 ? smask0 : sign_mask(p.c.signs, rd, j), j);
    uint32_t word = sign_word(x, j);
    if (__any_sync(kFull, !isfinite(squares))) {  // NaN is not >= 0, whatever its sign bit
      word = 0u;
      #pragma unroll
      for (int r = 0; r < 32; ++r) {
        const uint32_t bal = __ballot_sync(kFull, x[r] >= 0.0f);
        if ((r >> 3) == j) word |= ((bal >> (4 * tau)) & 0xFu) << (4 * (r & 7));
      }
    }
    float a[32];
    #pragma unroll
    for (int r = 0; r < 32; ++r) a[r] = fabsf(x[r]);
    const float sabs = tree_sum_q4(a);
    const float cinv = (sabs > 0.0f) ? __fdiv_rn(__fmul_rn(static_cast<float>(kD), nrm), sabs) : 1.0f;
    if (on) {
      const int row = 8 * ((tok >> 1) & 3) + 2 * (tok >> 3) + (tok & 1);
      reinterpret_cast<uint32_t*>(blk)[row * 4 + j] = word;
      if (j == 0) reinterpret_cast<float*>(blk + kBlkOffNc)[tok] = __fmul_rn(nrm, cinv);
    }
  }

  // ---- value: lane j holds group j, its eights i ^ j
  float v[32];
  asm volatile("cp.async.wait_group 1;" ::: "memory");  // the next key's rows may still be under way
  __syncwarp();
  {
    const uint8_t* vrow = s_rows[warp] + 8 * F::kKeyRow + tau * F::kValueRow + 32 * j * F::kEs;
    #pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint4* at = reinterpret_cast<const uint4*>(vrow + (q ^ j) * 8 * F::kEs);
      const uint4 w0 = at[0];
      if (DT == KV1B_DTYPE_F32) {
        const uint4 w1 = at[1];
        const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
        #pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * q + i] = __uint_as_float(w[i]);
      } else {
        const uint32_t w[4] = {w0.x, w0.y, w0.z, w0.w};
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = as_floats(w[i], DT);
          v[8 * q + 2 * i] = f.x;
          v[8 * q + 2 * i + 1] = f.y;
        }
      }
    }
  }
  __syncwarp();
  if (h + 1 < h_end) copy_values(h + 1);
  else asm volatile("cp.async.commit_group;" ::: "memory");
  float mn = v[0], mx = v[0];  // NaN if one of them is
  #pragma unroll
  for (int i = 0; i < 32; i += 2) {
    mn = min3_nan(mn, v[i], v[i + 1]);
    mx = max3_nan(mx, v[i], v[i + 1]);
  }
  if (!(mn >= -kF16Max && mx <= kF16Max)) {  // rare: limit the values
    bool fin = true, big = false;
    mn = INFINITY;
    mx = -INFINITY;
    #pragma unroll
    for (int i = 0; i < 32; ++i) {
      fin &= isfinite(v[i]);
      big |= fabsf(v[i]) > kF16Max;
      v[i] = limit_value(v[i]);
      mn = fminf(mn, v[i]);
      mx = fmaxf(mx, v[i]);
    }
    flags |= fin ? (big ? KV1B_STATUS_FP16_SATURATED : 0) : KV1B_STATUS_NONFINITE;
  }
  uint32_t sb, mb;
  group_scale(mn, mx, &sb, &mb, false);
  const float sf = __half2float(__ushort_as_half(static_cast<unsigned short>(sb)));
  const float mf = __half2float(__ushort_as_half(static_cast<unsigned short>(mb)));
  const float rs = __frcp_rn(sf);
  const uint64_t sf2 = pair(-sf, -sf), rs2 = pair(rs, rs), mf2 = pair(-mf, -mf), half2 = pair(0.5f, 0.5f);
  uint32_t cw[4];  // token-major: nibble i of word k = channel 32 j + 8 (k ^ j) + i of this token
  #pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t w = 0u - kMagicPacked;
    #pragma unroll
    for (int i = 0; i < 8; i += 2) {
      // div_markstein for two: q0 + (x - s q0) / s; x >= 0, the group's least value rounded down
      const uint64_t x = add2(pair(v[8 * k + i], v[8 * k + i + 1]), mf2);
      const uint64_t q0 = mul2(x, rs2);
      float y0, y1;
      unpair(add2(fma2(fma2(sf2, q0, x), rs2, q0), half2), y0, y1);
      w += __float_as_uint(__fadd_rd(fminf(y0, 15.5f), 8388608.0f)) << (4 * i);
      w += __float_as_uint(__fadd_rd(fminf(y1, 15.5f), 8388608.0f)) << (4 * i + 4);
    }
    cw[k] = (on && sf > 0.0f) ? w : 0u;
  }
  if (on) {
    reinterpret_cast<uint16_t*>(blk + kBlkOffScale)[32 * j + tok] = static_cast<uint16_t>(sb);
    reinterpret_cast<uint16_t*>(blk + kBlkOffMin)[32 * j + tok] = static_cast<uint16_t>(mb);
  }
  // transpose the 8 x 8 nibbles of each word across the 8 token lanes of group j (nibble = token), then
  // move the even tokens to nibbles 0 .. 3 and the odd ones to 4 .. 7
  #pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t x = cw[k];
    uint32_t y = __shfl_xor_sync(kFull, x, 16);
    x = (tau & 4) ? ((x & 0xFFFF0000u) | (y >> 16)) : ((x & 0x0000FFFFu) | (y << 16));
    y = __shfl_xor_sync(kFull, x, 8);
    x = (tau & 2) ? ((x & 0xFF00FF00u) | ((y >> 8) & 0x00FF00FFu)) : ((x & 0x00FF00FFu) | ((y & 0x00FF00FFu) << 8));
    y = __shfl_xor_sync(kFull, x, 4);
    x = (tau & 1) ? ((x & 0xF0F0F0F0u) | ((y >> 4) & 0x0F0F0F0Fu)) : ((x & 0x0F0F0F0Fu) | ((y & 0x0F0F0F0Fu) << 4));
    uint32_t s1 = (x ^ (x >> 4)) & 0x00F000F0u;   // swap nibbles 1 and 2 of each half word
    x ^= s1 ^ (s1 << 4);
    s1 = (x ^ (x >> 8)) & 0x0000FF00u;            // swap bytes 1 and 2
    x ^= s1 ^ (s1 << 8);
    cw[k] = x;
  }
  {
    uint32_t* dst = reinterpret_cast<uint32_t*>(blk + kBlkOffCodes) + (32 * j + tau) * 4 + (static_cast<int>(g.g0 & 31) >> 3);
    #pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t* at = dst + 8 * 4 * (k ^ j);
      *at = keep ? ((*at & keep) | (cw[k] & ~keep)) : cw[k];
    }
  }
  }
  flags = static_cast<int>(__reduce_or_sync(kFull, static_cast<unsigned>(flags)));
  if (lane == 0 && flags && p.c.status) atomicOr(p.c.status, flags);
}

}  // namespace paged
}  // namespace kv1b

using namespace kv1b;

template <int DT>
static cudaError_t launch_prefill(const PagedAppendParams& p, int heads, cudaStream_t stream) {
  constexpr int kWarps = paged::Prefill<DT>::kWarps;
  const int64_t kv_blocks = static_cast<int64_t>((p.groups + kWarps - 1) / kWarps) * ((p.c.Hkv + heads - 1) / heads);
  const int64_t rows = p.q ? static_cast<int64_t>(p.T) * ((p.Hq + paged::kQueryHeads - 1) / paged::kQueryHeads) : 0;
  const int64_t blocks = kv_blocks + (rows + kWarps - 1) / kWarps;  // below 2^30: the API limits the rows
  const uint32_t kv_share = blocks == kv_blocks ? 0u : static_cast<uint32_t>(((kv_blocks << 32) + blocks - 1) / blocks);
  return launch_pdl(paged::paged_append_prefill_kernel<DT>, dim3(static_cast<unsigned>(blocks + 1)), dim3(32 * kWarps), 0, stream, p, kv_share, heads);
}

cudaError_t kv1b_launch_paged_append(const PagedAppendParams& p, cudaStream_t stream) {
  // The decode form where hardly a sequence can bring a second token: 3.7 against 6.8 us for one token of each of 4
  // sequences, 5.4 against 7.6 for 64, 8.5 against 15.4 for 256, but 15.4 against 8.0 for two of each of 64 (8 kv-heads,
  // 32 query heads).  Which sequences bring them is the device's to know: where one of many slots brings all, its warps
  // take eight in turn, and the prompts' form would do better: 14.1 against 7.1 us for 64 tokens of one of 64 slots, 15.9
  // against 8.6 for 256, 30.1 against 21.5 for 1,023.
  if (p.T <= p.B + 1) {
    const int64_t units = 2LL * p.groups * p.c.Hkv + (p.q ? static_cast<int64_t>(p.T) * p.Hq : 0);
    return launch_pdl(paged::paged_append_token_kernel, dim3(static_cast<unsigned>(units / 4 + 1)), dim3(128), 0, stream, p);
  }
  // Heads a warp takes in turn, so that their rows can be copied ahead, while every SM still gets its 20 warps more
  // than once: 1, 2, 4 heads take 13.1, 15.1, 21.2 us for 2,048 tokens x 8 heads, 47.1, 45.2, 47.5 for 8,192 and
  // 175.9, 163.4, 156.8 for 32,768.
  const int64_t share = static_cast<int64_t>(p.groups) * p.c.Hkv / (p.sms * 28);
  const int heads = share < 1 ? 1 : (share > 4 ? 4 : static_cast<int>(share));
  switch (p.dtype) {
    case KV1B_DTYPE_F32: return launch_prefill<KV1B_DTYPE_F32>(p, heads, stream);
    case KV1B_DTYPE_BF16: return launch_prefill<KV1B_DTYPE_BF16>(p, heads, stream);
    default: return launch_prefill<KV1B_DTYPE_F16>(p, heads, stream);
  }
}

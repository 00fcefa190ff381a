// kv1b_paged_device.cuh -- device-side pieces shared by the paged attention kernels: bulk copies and
// bounded waits, code expansion, and the split of the visible blocks over CTAs.
#pragma once
#include "kv1b_device.cuh"
#include "kv1b_paged.h"

namespace kv1b {
namespace paged {

constexpr float kTau = 8.0f;    // a logit may pass the reference by 2^8 before it is raised
constexpr float kBase = 7.0f;   // weights are 2^7 at the reference: at most 2^15 < 65504
constexpr float kNoRef = -1e30f;
constexpr int kRow = 2 + kD;    // partial row: m (log2 units), l, o[128]
constexpr int kMaxSeqs = KV1B_PAGED_MAX_SEQS;
constexpr int kWaitTries = 4096;

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void mbar_init(uint64_t* bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count));
}
__device__ __forceinline__ bool mbar_try(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(ok)
               : "r"(smem_u32(bar)), "r"(parity)
               : "memory");
  return ok != 0;
}
// Bounded wait: at most `tries` suspended tries of up to 0.5 ms (the first, which finds nearly every barrier
// complete, without a time: 82 against 118 clocks); false when they ran out.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, int tries) {
  if (mbar_try(bar, parity)) return true;
  #pragma unroll 1
  for (int i = 0; i < tries; ++i) {
    uint32_t ok;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(500000u)
        : "memory");
    if (ok) return true;
  }
  return false;
}
__device__ __forceinline__ void block_g2s(uint32_t dst, const void* src, uint64_t* bar) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(kBlkBytes) : "memory");
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(kBlkBytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t r[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void lds128(uint32_t r[4], uint32_t addr) {
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void imma(int d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same with every sum starting at c
__device__ __forceinline__ void imma_from(int d[4], int c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(c));
}
__device__ __forceinline__ void hmma(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// ---- pairs of fp32
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ uint64_t pair(uint32_t a, uint32_t b) { return pair(__uint_as_float(a), __uint_as_float(b)); }
__device__ __forceinline__ void unpair(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// The four token pairs of a code word as exact binary16 integers 0 .. 15: a nibble in the mantissa of
// 1024 (low nibble of a byte: 1024 + c; high nibble: 1024 + 16 c), the offset taken off exactly.
__device__ __forceinline__ void expand_codes(uint32_t w, uint32_t (&c)[4]) {
  const uint32_t w8 = w >> 8;
  c[0] = hadd2((w & 0x000F000Fu) | 0x64006400u, 0xE400E400u);               // - 1024
  c[1] = hfma2((w & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD400D400u);  // / 16 - 64
  c[2] = hadd2((w8 & 0x000F000Fu) | 0x64006400u, 0xE400E400u);
  c[3] = hfma2((w8 & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD400D400u);
}

// A lane's four channels of a query row.  The append turns queries, in place if the caller likes, and a kernel
// behind it may start before it ends: coherent loads, where load4's are for data that nothing writes meanwhile.
__device__ __forceinline__ void load_query(const void* q, int64_t at, int dtype, float (&x)[4]) {
  if (dtype == KV1B_DTYPE_F32) {
    const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(q) + at);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    return;
  }
  const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(q) + at);
  const uint32_t h[4] = {u.x & 0xffffu, u.x >> 16, u.y & 0xffffu, u.y >> 16};
  #pragma unroll
  for (int r = 0; r < 4; ++r)
    x[r] = dtype == KV1B_DTYPE_BF16 ? __uint_as_float(h[r] << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(h[r])));
}

// Results as binary16.  They are means of values within +-65504, whose roundings (a weight's 2^-11 against the
// unrounded normaliser in the shared prefix) may pass that by more than half a step: limited to it.  NaN stays.
__device__ __forceinline__ uint32_t pack_result_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ void store_out(void* out, int dtype, int64_t i, float x) {
  if (dtype == KV1B_DTYPE_BF16) static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(x);
  else static_cast<uint16_t*>(out)[i] = static_cast<uint16_t>(pack_result_f16(x, 0.0f));
}

// ---------------------------------------------------------------------------------------------
// The work plan, computed alike by every CTA from the device lengths.
struct Visible {
  int blocks;       // blocks seen
  int skip_from;    // blocks [0, skip_from) and from skip_to on are seen
  int skip_to;
};
__device__ __forceinline__ Visible visible(int len, int window, int sinks) {
  Visible v;
  const int nb = (len + kBlkTok - 1) / kBlkTok;
  v.skip_from = v.skip_to = 0;
  if (window > 0 && len > window) {
    const int wb = (len - window) / kBlkTok;
    const int s = sinks < len ? sinks : len;
    const int sb = (s + kBlkTok - 1) / kBlkTok;
    v.skip_from = sb < wb ? sb : wb;
    v.skip_to = wb;
  }
  v.blocks = nb - (v.skip_to - v.skip_from);
  return v;
}

// a / b for a >= 0, b > 0: a 32-bit division where both fit (the 64-bit one is a long subroutine)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// The segments in order, each of as many units as it has blocks and kSegUnits more for its start and end
// (queries, a piece or a result), cut into n equal ranges of units.
struct Plan {
  const uint32_t* pre;   // [B + 1] blocks of one kv-head before each sequence
  const int* len;
  const uint16_t* some;  // [nsome] the sequences that see a block, in order
  int nsome;
  int B, Hkv, n;         // n: CTAs with work
  int64_t S;             // blocks in all
  int64_t q;             // units / n: the first `rem` ranges are one unit longer
  int rem;
  __device__ __forceinline__ int blocks(int k) const { return static_cast<int>(pre[some[k] + 1] - pre[some[k]]); }
  __device__ __forceinline__ int64_t first_block(int k) const { return static_cast<int64_t>(pre[some[k]]) * Hkv; }
  __device__ __forceinline__ int64_t first_unit(int k) const { return (pre[some[k]] + static_cast<int64_t>(kSegUnits) * k) * Hkv; }
  // first block of range c: a segment's kSegUnits come before its blocks
  __device__ __forceinline__ int64_t begin(int c) const {
    if (c >= n) return S;
    const int64_t u = c * q + (c < rem ? c : rem);
    int lo = 0, hi = nsome;  // largest lo with first_unit(lo) <= u
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first_unit(mid) <= u) lo = mid;
      else hi = mid;
    }
    const int nb = blocks(lo);
    const int64_t in = u - first_unit(lo), h = quotient(in, nb + kSegUnits);
    const int64_t i = in - h * (nb + kSegUnits) - kSegUnits;
    return first_block(lo) + h * nb + (i > 0 ? i : 0);
  }
  // the range that holds block i of head h of sequence some[k]
  __device__ __forceinline__ int owner(int k, int h, int i) const {
    const int64_t u = first_unit(k) + static_cast<int64_t>(h) * (blocks(k) + kSegUnits) + kSegUnits + i, longer = rem * (q + 1);
    return u < longer ? static_cast<int>(quotient(u, q + 1)) : rem + static_cast<int>(quotient(u - longer, q));
  }
};

// A sequence's length, limited to what its page table can hold.
__device__ __forceinline__ int plan_length(const PagedAttendParams& p, int b, bool* bad) {
  const bool own = b >= p.packed;
  const int64_t top = static_cast<int64_t>(own ? p.max_pages : p.max_prefix_pages) << (p.c.bpp_shift + 5);
  const int n = own ? __ldg(p.lengths + b - p.packed) : __ldg(p.prefix_len);
  *bad |= n < 0 || n > top;
  return n < 0 ? 0 : static_cast<int>(n > top ? top : n);
}

// All threads of the CTA.  pre, len and some are in shared memory and, as the plan, the same for every warp: each
// warp may use them at once.
// BESIDE: the plan of a shared call's own tokens beside the matrix kernel's CTAs.
template <int THREADS, bool BESIDE>
__device__ __forceinline__ Plan make_plan(const PagedAttendParams& p, uint32_t* pre, int* len, uint16_t* some, int ncta, bool report) {
  const int nseq = p.packed + p.B;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  bool bad = false;
  uint64_t total = 0;  // blocks, and sequences with some << 40
  if (nseq <= 32) {  // by every warp for itself: a barrier less, and shorter chains
    const int n = lane < nseq ? plan_length(p, lane, &bad) : 0;
    const uint32_t blocks = visible(n, p.window, p.sinks).blocks;
    const unsigned with = __ballot_sync(kFull, blocks > 0);
    uint32_t x = blocks;
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    if (lane < nseq) {
      len[lane] = n;
      pre[lane + 1] = x;
      if (blocks > 0) some[__popc(with & ((1u << lane) - 1u))] = static_cast<uint16_t>(lane);
    }
    if (lane == 0) pre[0] = 0;
    total = __shfl_sync(kFull, x, 31) | static_cast<uint64_t>(__popc(with)) << 40;
    __syncwarp();
  } else {
    __shared__ uint64_t s_tot[THREADS / 32];
    const int per = (nseq + THREADS - 1) / THREADS;
    const int b0 = threadIdx.x * per, b1 = min(b0 + per, nseq);
    uint64_t mine = 0;
    for (int b = b0; b < b1; ++b) {
      const int n = plan_length(p, b, &bad);
      len[b] = n;
      const int blocks = visible(n, p.window, p.sinks).blocks;
      mine += static_cast<uint64_t>(blocks) | (blocks > 0 ? 1ull << 40 : 0ull);
    }
    uint64_t x = mine;
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_tot[warp] = x;
    __syncthreads();
    uint64_t at = x - mine;
    for (int w = 0; w < THREADS / 32; ++w) {
      at += w < warp ? s_tot[w] : 0ull;
      total += s_tot[w];
    }
    for (int b = b0; b < b1; ++b) {
      pre[b] = static_cast<uint32_t>(at);
      const int blocks = visible(len[b], p.window, p.sinks).blocks;
      if (blocks > 0) some[at >> 40] = static_cast<uint16_t>(b);
      at += static_cast<uint64_t>(blocks) | (blocks > 0 ? 1ull << 40 : 0ull);
    }
    if (threadIdx.x == 0) pre[nseq] = static_cast<uint32_t>(total);
    __syncthreads();
  }
  if (bad && report && p.c.status) atomicOr(p.c.status, KV1B_STATUS_BAD_INDEX);
  Plan pl;
  pl.pre = pre;
  pl.len = len;
  pl.some = some;
  pl.nsome = static_cast<int>(total >> 40);
  pl.B = nseq;
  pl.Hkv = p.c.Hkv;
  pl.S = static_cast<int64_t>(static_cast<uint32_t>(total)) * p.c.Hkv;
  const int64_t units = pl.S + static_cast<int64_t>(kSegUnits) * pl.nsome * pl.Hkv;
  const int64_t want = quotient(units + p.min_units - 1, p.min_units);
  pl.n = static_cast<int>(want < 1 ? 1 : (want < ncta ? want : ncta));
  if (BESIDE && p.beside > 0) {
    const int64_t tiles = (static_cast<int64_t>(max(__ldg(p.prefix_len), 0)) + 127) / 128;
    const int64_t prefix_ns = kPrefixNs + quotient(tiles + p.splits - 1, p.splits) * p.tile_ns;
    if (kCtaNs + quotient(units * kUnitNs, p.beside) <= prefix_ns) pl.n = p.beside;
  }
  pl.q = quotient(units, pl.n);
  pl.rem = static_cast<int>(units - pl.q * pl.n);
  return pl;
}

constexpr int kMaxPieces = 512;  // a row's pieces: CTAs of the split, and the token ranges of two lanes or the CTAs once more
static_assert(kMaxCtas + 2 * kMaxSplits <= kMaxPieces && 2 * kMaxCtas <= kMaxPieces, "pieces of a merge");

// Log-sum-exp merge of n <= kMaxPieces partial rows by a block of 128 threads.  Warp w takes pieces w, w + 4, ..,
// kAtOnce of them in flight, two pairs of channels a lane; then the four sums meet.  (A channel a thread and one piece
// behind another took 23 us for 512 rows of 69 pieces, and 10 for 2,048 rows of 19.)
template <typename Piece>
__device__ __forceinline__ void merge_pieces(int n, Piece piece, float2* s_head, float* s_max, void* out, int dtype, int64_t at) {
  constexpr int kAtOnce = 8;
  __shared__ float2 s_num[4][kD / 2];
  __shared__ float s_den[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float M = kNoRef;
  for (int i = threadIdx.x; i < n; i += 128) {
    const float2 h = *reinterpret_cast<const float2*>(piece(i));
    s_head[i] = h;
    M = fmaxf(M, h.x);
  }
  #pragma unroll
  for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
  if (lane == 0) s_max[warp] = M;
  __syncthreads();
  M = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
  float2 lo = make_float2(0.0f, 0.0f), hi = lo;
  float den = 0.0f;
  #pragma unroll 1
  for (int i0 = warp; i0 < n; i0 += 4 * kAtOnce) {
    float2 a[kAtOnce], b[kAtOnce];
    #pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      a[u] = b[u] = make_float2(0.0f, 0.0f);
      if (i0 + 4 * u < n) {
        const float2* o = reinterpret_cast<const float2*>(piece(i0 + 4 * u) + 2);
        a[u] = o[lane];
        b[u] = o[32 + lane];
      }
    }
    #pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      if (i0 + 4 * u < n) {
        const float2 h = s_head[i0 + 4 * u];
        const float f = ex2(h.x - M);
        lo.x = __fmaf_rn(f, a[u].x, lo.x), lo.y = __fmaf_rn(f, a[u].y, lo.y);
        hi.x = __fmaf_rn(f, b[u].x, hi.x), hi.y = __fmaf_rn(f, b[u].y, hi.y);
        den = __fmaf_rn(f, h.y, den);
      }
    }
  }
  s_num[warp][lane] = lo;
  s_num[warp][32 + lane] = hi;
  if (lane == 0) s_den[warp] = den;
  __syncthreads();
  float num = 0.0f;
  den = 0.0f;
  #pragma unroll
  for (int w = 0; w < 4; ++w) {
    num = __fadd_rn(num, reinterpret_cast<const float*>(s_num[w])[threadIdx.x]);
    den = __fadd_rn(den, s_den[w]);
  }
  store_out(out, dtype, at + threadIdx.x, den != 0.0f ? __fdiv_rn(num, den) : 0.0f);
}

}  // namespace paged
}  // namespace kv1b

// kv1b_paged_shared.cu -- attention of a whole batch over one shared prefix: every query of a kv-head
// against each prefix token once, as products of a matrix of queries on the 5th-generation tensor cores.
//
// For kv-head h the batch's queries are R = sequences x G rows.  A CTA takes up to 256 rows (two lanes
// of 128) and a range of 128-token tiles; the ranges' partial rows (m, l, o) are merged afterwards with
// the sequences' own tokens.  With at most 128 rows both lanes hold the same rows, one takes the first
// half of each tile and one the second.
//
// A job is 64 tokens of a tile on a lane: S = Q K^T (f8, exact: codes 0 .. 15 times signs +-1, sums below
// 2^11) into tensor memory; each softmax thread owns one row, x = nc (delta I2 + vl I1) with I2 = S and I1
// the token's sum of signs, and leaves 2^(x - m + kBase) as binary16; O += P V (f16, fp32 sums in tensor
// memory).  A softmax thread takes its 64 sums into registers at once and gives S back, so the next job's
// scores are made while it works, and P has two places, so it never waits for the products: per lane 64
// columns of S, 2 x 32 of P and 128 of O, for two lanes all 512.  (One S of 128 columns with P written
// over it, so that each job went round softmax, P V and Q K: 201 us instead of 123 us at 256 rows x
// 131,072 tokens x 8 kv-heads.)
//
// Warps: 0 - 3 and 4 - 7 the lanes' softmax, 8 - 11 the values' expansion (codes to f16, one rounding), 12
// and 13 issue a lane's products each, 14 and 15 expand the signs to f8, 14 also copies the blocks.  Each wait
// is bounded; one that runs out ends the CTA with KV1B_STATUS_TIMEOUT.
//
// Roundings: a weight 2^(x - m + kBase) is a binary16 in the products, while the normaliser sums the unrounded weights:
// they may differ by 2^-11.  A value min + scale code is rounded to binary16 once; as a multiple of 2^-24 it is exact
// below 2^-13, so small values lose nothing.
//
// A tile of 128 tokens x 256 rows costs 512 + 1,024 clocks of products and 32,768 exponentials, 2,048
// clocks at 16 a clock: the exponentials are its floor.  What bounds it are the waits between the parts of a job (2,050
// clocks against 1,142 of exponentials), the longest for the scores to come out of tensor memory.
#include "kv1b_paged_attend.cuh"

namespace kv1b {
namespace paged {

constexpr int kTile = 128;                 // tokens
constexpr int kTileBlocks = kTile / kBlkTok;
constexpr int kSoftWarps = 8, kValueWarps = 4, kSignWarps = 2;
constexpr int kMmaWarp = kSoftWarps + kValueWarps, kSignWarp = kMmaWarp + 2;
constexpr int kHalf = 64;                  // tokens of a job
constexpr float kMostSum = 32768.0f;       // 2^(kBase + kTau): a sum up to it holds no larger weight
constexpr int kShThreads = 512;            // four warpgroups
// 512 x 128 registers at launch; the softmax groups take what the others give back: 2 (168 + 88) = 4 x 128
constexpr int kSoftRegs = 168, kOtherRegs = 88;
constexpr int kRaw = 3;                    // tiles of blocks in flight
constexpr int kBuf = 3;                    // expanded tiles
constexpr int kQBytes = 128 * 128;         // one lane's codes
constexpr int kKBytes = kTile * 128;       // signs as f8
constexpr int kVBytes = kTile * kD * 2;    // values as f16: two halves of 64 tokens
constexpr int kRawBytes = kTileBlocks * kBlkBytes;

constexpr int kShQ = 0;
constexpr int kShK = kShQ + 2 * kQBytes;
constexpr int kShV = kShK + kBuf * kKBytes;
constexpr int kShRaw = kShV + kBuf * kVBytes;
constexpr int kShNc = kShRaw + kRaw * kRawBytes;     // f32 [kBuf][2][128]: nc, nc I1
constexpr int kShMask = kShNc + kBuf * 2 * kTile * 4;  // u32 [kBuf][4]: tokens seen
constexpr int kShSmem = kShMask + kBuf * 16 + 1024;    // and the alignment of the base
static_assert(kRawBytes % 128 == 0 && kShSmem <= 226 * 1024, "shared memory");

// ---- tensor memory and products
__device__ __forceinline__ void tmem_alloc(uint32_t* dst) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(dst)) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t base) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(base) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// One lane of a converged warp.  (The compiler then knows that the branch has one thread and keeps the
// products' descriptors in uniform registers.)
__device__ __forceinline__ bool elect() {
  uint32_t one;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(one));
  return one != 0;
}
// K-major operand in 128-byte swizzled rows (8-row groups of 1,024 bytes)
__device__ __forceinline__ uint64_t operand(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (1ull << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) |
         (2ull << 61);
}
// M 128, fp32 sums; operand types 0 (e4m3, f16)
constexpr uint32_t kScoreShape = (1u << 4) | ((kHalf / 8) << 17) | ((128u / 16) << 24);
constexpr uint32_t kValueShape = (1u << 4) | ((kD / 8) << 17) | ((128u / 16) << 24);
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, bool add) {
  asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a),
               "l"(b), "r"(kScoreShape), "r"(static_cast<uint32_t>(add))
               : "memory");
}
__device__ __forceinline__ void mma_f16_ta(uint32_t d, uint32_t a, uint64_t b, bool add) {
  asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d), "r"(a),
               "l"(b), "r"(kValueShape), "r"(static_cast<uint32_t>(add))
               : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
// the registers of a load are valid from here on: the dependency keeps their uses behind the wait
template <int N>
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  #pragma unroll
  for (int i = 0; i < N; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7]));
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------------------------------------------
// Query rows as f8 codes in the order of the expanded signs (channel 32 w + 8 j + r at byte 32 w + 4 r + j),
// and each row's two factors of the logit.  One warp per row, every row once: the CTAs of the prefix's token
// ranges preparing their 256 rows each took 24 us before their first product.
__global__ void __launch_bounds__(256) paged_query_codes_kernel(const PagedAttendParams p, const PagedSharedParams s, const int G) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);  // [sequence][q head]
  if (row >= static_cast<int64_t>(p.B) * p.Hq) return;
  float x[4];
  load_query(p.q, row * kD + 4 * lane, p.q_dtype, x);
  int code[4];
  float vl, dl;
  query_quantise(x, p.c.signs, code, &vl, &dl);
  const int b = static_cast<int>(row / p.Hq), hq = static_cast<int>(row - static_cast<int64_t>(b) * p.Hq);
  const int h = hq / G, g = hq - h * G;
  const int64_t at = static_cast<int64_t>(h) * s.R + static_cast<int64_t>(b) * G + g;
  uint8_t* bytes = s.codes + at * kD + 32 * (lane >> 3) + 16 * (lane & 1) + ((lane & 7) >> 1);  // channel 4 (lane & 7) of word lane / 8
  #pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint32_t v = static_cast<uint32_t>(code[r]);
    const int e = 31 - __clz(v | 1u);
    bytes[4 * r] = static_cast<uint8_t>(v == 0 ? 0u : static_cast<uint32_t>((7 + e) << 3) | ((v << (3 - e)) & 7u));
  }
  if (lane == 0) {
    const float qs = __fmul_rn(__fmul_rn(p.scale, 1.4426950408889634f), 1.0f / kD);
    s.factors[at] = make_float2(__fmul_rn(dl, qs), __fmul_rn(vl, qs));
  }
}

__device__ __forceinline__ int prefix_tokens(const PagedAttendParams& p, bool report) {
  const int64_t top = static_cast<int64_t>(p.max_prefix_pages) << (p.c.bpp_shift + 5);
  const int n = __ldg(p.prefix_len);
  if (report && (n < 0 || n > top) && p.c.status) atomicOr(p.c.status, KV1B_STATUS_BAD_INDEX);
  return n < 0 ? 0 : static_cast<int>(n > top ? top : n);
}

// Exponents of four of a row's weights: logit - m + kBase, -infinity where MASKED and not seen.
template <bool MASKED>
__device__ __forceinline__ void exponents(const uint32_t (&x)[2][32], const float4* nc, int q, uint64_t fa, uint64_t fb, uint64_t off,
                                          uint2 seen, float (&y)[4]) {
  const float4 a = nc[q], i1 = nc[kTile / 4 + q];
  const uint32_t* xq = &x[q >> 3][4 * (q & 7)];
  unpair(fma2(mul2(pair(xq[0], xq[1]), pair(a.x, a.y)), fa, fma2(pair(i1.x, i1.y), fb, off)), y[0], y[1]);
  unpair(fma2(mul2(pair(xq[2], xq[3]), pair(a.z, a.w)), fa, fma2(pair(i1.z, i1.w), fb, off)), y[2], y[3]);
  if (MASKED) {
    const uint32_t bits = (q < 8 ? seen.x : seen.y) >> (4 * (q & 7));
    #pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = (bits >> e) & 1u ? y[e] : -INFINITY;
  }
}

// A row's 64 weights as pairs of binary16, and their sum in fp32.
template <bool MASKED>
__device__ __forceinline__ float row_weights(const uint32_t (&x)[2][32], const float4* nc, uint64_t fa, uint64_t fb, float offset, uint2 seen,
                                             uint32_t (&pw)[32]) {
  const uint64_t off = pair(offset, offset);
  uint64_t acc0 = pair(0.0f, 0.0f), acc1 = acc0;
  #pragma unroll
  for (int q = 0; q < kHalf / 4; ++q) {
    float y[4];
    exponents<MASKED>(x, nc, q, fa, fb, off, seen, y);
    const float e0 = ex2(y[0]), e1 = ex2(y[1]), e2 = ex2(y[2]), e3 = ex2(y[3]);
    pw[2 * q] = pack_f16(e0, e1);
    pw[2 * q + 1] = pack_f16(e2, e3);
    acc0 = add2(acc0, pair(e0, e1));
    acc1 = add2(acc1, pair(e2, e3));
  }
  float s0, s1;
  unpair(add2(acc0, acc1), s0, s1);
  return __fadd_rn(s0, s1);
}

// Unit u of the prefix's part.
__device__ __forceinline__ void prefix_cta(const PagedAttendParams& p, const PagedSharedParams& s, const int u, uint8_t* smem) {
  __shared__ __align__(8) uint64_t raw_full[kRaw], raw_empty[kRaw], kv_full[kBuf], kv_empty[kBuf];
  __shared__ __align__(8) uint64_t s_full[2], turn[2], pv_done[2][2];
  __shared__ uint32_t s_tmem, s_absent[kRaw];
  const uint32_t sb = smem_u32(smem);
  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // the warp as a uniform value

  if (threadIdx.x == 0) {
    for (int i = 0; i < kRaw; ++i) mbar_init(&raw_full[i], 1), mbar_init(&raw_empty[i], kValueWarps + kSignWarps);
    for (int i = 0; i < kBuf; ++i) mbar_init(&kv_full[i], kValueWarps + kSignWarps), mbar_init(&kv_empty[i], 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1), mbar_init(&turn[i], 4);
      mbar_init(&pv_done[i][0], 1), mbar_init(&pv_done[i][1], 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  pdl_launch_dependents();

  // unit: kv-head, row tile, split
  const int split = u % s.splits, hr = u / s.splits;
  const int rt = hr % s.row_tiles, h = hr / s.row_tiles;
  const int n = prefix_tokens(p, u == 0 && threadIdx.x == 0);
  const int64_t nt = (static_cast<int64_t>(n) + kTile - 1) / kTile;
  const int t0 = static_cast<int>(nt * split / s.splits), tiles = static_cast<int>(nt * (split + 1) / s.splits) - t0;
  const bool two = s.two != 0;
  if (tiles == 0) {  // the whole CTA: empty pieces (the merge reads none where the prefix is empty)
    if (nt > 0)
      for (int e = threadIdx.x; e < 256 * kRow; e += kShThreads)
        s.pieces[static_cast<int64_t>(u) * 256 * kRow + e] = e % kRow == 0 ? kNoRef : 0.0f;
    return;
  }
  // job j of lane w: half j & 1 of tile j / 2, or half w of tile j where the lanes hold the same rows
  const int jobs = two ? 2 * tiles : tiles;
  auto tile_of = [&](int j) { return two ? j >> 1 : j; };
  auto half_of = [&](int w, int j) { return two ? j & 1 : w; };

  if (warp == 0) tmem_alloc(&s_tmem);
  {  // the rows' codes, swizzled; zeros behind the last row
    const int rows = two ? 256 : 128;
    for (int e = threadIdx.x; e < rows * 8; e += kShThreads) {
      const int r = e >> 3, c = e & 7, row = rt * rows + r;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (row < s.R) v = *reinterpret_cast<const uint4*>(s.codes + (static_cast<int64_t>(h) * s.R + row) * kD + 16 * c);
      *reinterpret_cast<uint4*>(smem + kShQ + r * 128 + ((c ^ (r & 7)) << 4)) = v;
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = __shfl_sync(kFull, s_tmem, 0);
  if (warp >= kSoftWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  bool ok = true;  // false once a wait ran out
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!__all_sync(kFull, mbar_wait(bar, parity, kWaitTries))) ok = false;
    return ok;
  };

  if (warp < kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ------------------------------------------------------------------ softmax: a thread per row
    const int w = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const int row = rt * (two ? 256 : 128) + (two ? w * 128 : 0) + r;
    const bool warp_rows = row - lane < s.R;  // a warp without rows only keeps the barriers going
    const uint32_t tS = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + w * 256, tO = tS + 128;
    const float2 f = row < s.R ? s.factors[static_cast<int64_t>(h) * s.R + row] : make_float2(0.0f, 0.0f);
    const uint64_t fa = pair(f.x, f.x), fb = pair(f.y, f.y);
    float m = 0.0f, l = 0.0f;
    bool have = false;  // a finite logit has set m
    bool cold = true;   // not in all of the warp's rows
    for (int j = 0; j < jobs; ++j) {
      const int k = tile_of(j), buf = k % kBuf, half = half_of(w, j), slot = j & 1;
      // The commit of the job's scores covers the products issued before them, P V of job j - 2 among them, so
      // P's place is free; and the tile's factors and masks were written before the products' warp waited for
      // the tile.
      if (!wait(&s_full[w], j & 1)) break;
      tc_after();
      // (The wait for a load follows it in a straight line: nothing may copy the registers of a load in
      // flight.  Warps without rows load and store along, in rows that nobody reads.)
      uint32_t x[2][32];
      tmem_ld32(x[0], tS);
      tmem_ld32(x[1], tS + 32);
      const uint2 seen = *(reinterpret_cast<const uint2*>(smem + kShMask) + buf * 2 + half);  // the job's tokens
      tmem_ld_wait(x[0]);
      tmem_ld_wait(x[1]);
      tmem_st_wait();
      tc_before();
      __syncwarp();
      if (elect()) mbar_arrive(&turn[w]);  // S of job j has been read, P of job j - 1 written
      uint32_t pw[32];
      if (!warp_rows) {
        #pragma unroll
        for (int i = 0; i < 32; ++i) pw[i] = 0;
      } else {
        const float4* nc = reinterpret_cast<const float4*>(smem + kShNc + buf * 2 * kTile * 4) + half * (kHalf / 4);
        float sum = 0.0f;
        bool slow = cold || (seen.x & seen.y) != 0xFFFFFFFFu;
        if (!slow) {
          sum = row_weights<false>(x, nc, fa, fb, kBase - m, seen, pw);
          slow = __any_sync(kFull, sum > kMostSum);  // perhaps a weight past the bound
        }
        if (slow) {  // the first job, a tile with unseen tokens, or a reference to raise
          float top = -INFINITY;
          #pragma unroll
          for (int q = 0; q < kHalf / 4; ++q) {
            float y[4];
            exponents<true>(x, nc, q, fa, fb, pair(-m, -m), seen, y);
            top = max3(max3(top, y[0], y[1]), y[2], y[3]);
          }
          // also where many tokens above the reference, none by 2^kTau, pass the bound together: left there, such a row
          // would send its warp through here job after job (369 against 163 us for 64 x 4 rows behind 131,072 tokens of 8
          // heads where each token range's first 64 score low)
          const bool up = top > kTau || (sum > kMostSum && top > 0.0f) || (!have && top > -INFINITY);
          if (__any_sync(kFull, up)) {
            // the row's sums so far come down by 2^(m - m')
            const float alpha = up && have ? ex2(-top) : 1.0f;
            m = up ? m + top : m;
            have |= up;
            l = __fmul_rn(l, alpha);
            if (j >= 1) {
              if (!wait(&pv_done[w][slot ^ 1], ((j - 1) >> 1) & 1)) break;
              tc_after();
              #pragma unroll 1
              for (int c = 0; c < 8; ++c) {
                uint32_t o[16];
                tmem_ld16(o, tO + 16 * c);
                tmem_ld_wait(o);
                #pragma unroll
                for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__fmul_rn(__uint_as_float(o[q]), alpha));
                tmem_st16(tO + 16 * c, o);
              }
            }
          }
          cold = __any_sync(kFull, !have);
          sum = row_weights<true>(x, nc, fa, fb, kBase - m, seen, pw);
        }
        l = __fadd_rn(l, sum);
      }
      if (!ok) break;
      tmem_st16(tS + kHalf + 32 * slot, pw);
      tmem_st16(tS + kHalf + 32 * slot + 16, pw + 16);
    }
    // the last P, not before all four warps' last turn
    if (ok && wait(&turn[w], (jobs - 1) & 1)) {
      tmem_st_wait();
      tc_before();
      __syncwarp();
      if (elect()) mbar_arrive(&turn[w]);
    }
    // the lane's sums
    if (ok && wait(&pv_done[w][(jobs - 1) & 1], ((jobs - 1) >> 1) & 1)) {
      tc_after();
      float* out = s.pieces + ((static_cast<int64_t>(u) * 2 + w) * 128 + r) * kRow;
      if (warp_rows) {
        if (row < s.R) *reinterpret_cast<float2*>(out) = make_float2(have ? m : kNoRef, l);
        #pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          uint32_t o[16];
          tmem_ld16(o, tO + 16 * c);
          tmem_ld_wait(o);
          if (row < s.R) {
            #pragma unroll
            for (int q = 0; q < 16; q += 2)
              *reinterpret_cast<uint2*>(out + 2 + 16 * c + q) = make_uint2(o[q], o[q + 1]);
          }
        }
      }
    }
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------------------------ values: 32 channels of all tokens
    const int g = warp - kSoftWarps;
    const int ch = 32 * g + lane;
    for (int k = 0; k < tiles; ++k) {
      const int raw = k % kRaw, buf = k % kBuf;
      if (!wait(&raw_full[raw], (k / kRaw) & 1)) break;
      if (k >= kBuf && !wait(&kv_empty[buf], (k / kBuf - 1) & 1)) break;
      const uint32_t absent = s_absent[raw];
      uint8_t* blk = smem + kShRaw + raw * kRawBytes;
      const int left = n - (t0 + k) * kTile;
      if (left < kTile || absent) {  // unseen tokens' values are zeros, whatever their places hold
        #pragma unroll 1
        for (int b = 0; b < kTileBlocks; ++b)
          if (((absent >> b) & 1u) || 32 * b + lane >= left) {
            reinterpret_cast<uint16_t*>(blk + b * kBlkBytes + kBlkOffScale)[32 * g + lane] = 0;
            reinterpret_cast<uint16_t*>(blk + b * kBlkBytes + kBlkOffMin)[32 * g + lane] = 0;
          }
        __syncwarp();
      }
      #pragma unroll 2
      for (int b = 0; b < kTileBlocks; ++b) {
        const uint8_t* base = blk + b * kBlkBytes;
        const uint4 cw4 = *reinterpret_cast<const uint4*>(base + kBlkOffCodes + ch * 16);
        const uint32_t cw[4] = {cw4.x, cw4.y, cw4.z, cw4.w};
        uint8_t* vrow = smem + kShV + buf * kVBytes + (b >> 1) * (kVBytes / 2) + ch * 128;
        #pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint4 sc = *reinterpret_cast<const uint4*>(base + kBlkOffScale + g * 64 + q * 16);
          const uint4 mn = *reinterpret_cast<const uint4*>(base + kBlkOffMin + g * 64 + q * 16);
          uint32_t c[4];
          expand_codes(cw[q], c);
          *reinterpret_cast<uint4*>(vrow + (((4 * (b & 1) + q) ^ (lane & 7)) << 4)) =
              make_uint4(hfma2(c[0], sc.x, mn.x), hfma2(c[1], sc.y, mn.y), hfma2(c[2], sc.z, mn.z), hfma2(c[3], sc.w, mn.w));
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&kv_full[buf]);
        mbar_arrive(&raw_empty[raw]);
      }
    }
  } else if (warp >= kSignWarp) {
    // ------------------------------------------------------------------ signs as +-1 in f8 and the tokens' factors
    // and, by the first of the two warps, the copies of the blocks (lane b < 4 block b of a tile)
    const int bit_row = 8 * ((lane >> 1) & 3) + 2 * (lane >> 3) + (lane & 1);
    const bool copies = warp == kSignWarp;
    const int nblk = (n + kBlkTok - 1) / kBlkTok;
    int copied = 0;  // tiles
    auto entry = [&](int k) {
      const int blk = (t0 + k) * kTileBlocks + lane;
      return lane < kTileBlocks && blk < nblk ? __ldg(p.prefix_pages + (blk >> p.c.bpp_shift)) : -1;
    };
    int page = copies ? entry(0) : -1;
    auto copy_next = [&]() {
      const int raw = copied % kRaw, blk = (t0 + copied) * kTileBlocks + lane;
      const bool want = lane < kTileBlocks && blk < nblk;
      const bool here = want && page >= 0 && page < p.c.num_pages;
      const uint32_t have = __ballot_sync(kFull, here);
      if (want && !here && p.c.status) atomicOr(p.c.status, KV1B_STATUS_BAD_INDEX);
      if (lane == 0) {
        s_absent[raw] = ~have & 0xFu;
        asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(&raw_full[raw])),
                     "r"(__popc(have) * kBlkBytes)
                     : "memory");
      }
      __syncwarp();
      if (here) {
        const int in = blk & ((1 << p.c.bpp_shift) - 1);
        const uint8_t* src = p.c.pages + ((((static_cast<int64_t>(page) * p.c.Hkv + h) << p.c.bpp_shift) + in) * kBlkBytes);
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                         sb + kShRaw + raw * kRawBytes + lane * kBlkBytes),
                     "l"(src), "r"(kBlkBytes), "r"(smem_u32(&raw_full[raw]))
                     : "memory");
      }
      ++copied;
      if (copied < tiles) page = entry(copied);
    };
    if (copies)
      while (copied < kRaw && copied < tiles) copy_next();
    for (int k = 0; k < tiles; ++k) {
      const int raw = k % kRaw, buf = k % kBuf;
      if (!wait(&raw_full[raw], (k / kRaw) & 1)) break;
      if (k >= kBuf && !wait(&kv_empty[buf], (k / kBuf - 1) & 1)) break;
      const uint32_t absent = s_absent[raw];
      const int left = n - (t0 + k) * kTile;
      #pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int b = 2 * (warp - kSignWarp) + i, tok = 32 * b + lane;
        const uint8_t* blk = smem + kShRaw + raw * kRawBytes + b * kBlkBytes;
        const bool on = tok < left && !((absent >> b) & 1u);
        const uint4 w4 = *reinterpret_cast<const uint4*>(blk + bit_row * 16);
        const uint32_t bits[4] = {w4.x, w4.y, w4.z, w4.w};
        const float ncv = on ? reinterpret_cast<const float*>(blk + kBlkOffNc)[lane] : 0.0f;
        const int i1 = 2 * (__popc(bits[0]) + __popc(bits[1]) + __popc(bits[2]) + __popc(bits[3])) - kD;
        float* ncp = reinterpret_cast<float*>(smem + kShNc) + buf * 2 * kTile + tok;
        ncp[0] = ncv;
        ncp[kTile] = __fmul_rn(ncv, static_cast<float>(i1));
        const uint32_t seen = __ballot_sync(kFull, on);
        if (lane == 0) reinterpret_cast<uint32_t*>(smem + kShMask)[buf * 4 + b] = seen;
        uint8_t* krow = smem + kShK + buf * kKBytes + tok * 128;
        #pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t v[4];
          #pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = ((~bits[c >> 1] << (7 - (4 * (c & 1) + e))) & 0x80808080u) | 0x38383838u;
          *reinterpret_cast<uint4*>(krow + ((c ^ (lane & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&kv_full[buf]);
        mbar_arrive(&raw_empty[raw]);
      }
      if (copies && copied < tiles) {
        if (!wait(&raw_empty[raw], (k / kRaw) & 1)) break;
        copy_next();
      }
    }
    if (copies)  // no copy may outlive the CTA, also where the expansion gave up
      for (int i = copied > kRaw ? copied - kRaw : 0; i < copied; ++i) mbar_wait(&raw_full[i % kRaw], (i / kRaw) & 1, kWaitTries);
  } else {
    // ------------------------------------------------------------------ products of one lane
    const int w = warp - kMmaWarp;
    auto scores = [&](int j) {
      const int k = tile_of(j), buf = k % kBuf;
      if ((!two || (j & 1) == 0) && !wait(&kv_full[buf], (k / kBuf) & 1)) return;
      tc_after();
      if (elect()) {
        const uint64_t a = operand(sb + kShQ + (two ? w * kQBytes : 0));
        const uint64_t b = operand(sb + kShK + buf * kKBytes + half_of(w, j) * (kKBytes / 2));
        #pragma unroll
        for (int i = 0; i < 4; ++i) mma_f8(tmem + w * 256, a + 2 * i, b + 2 * i, i > 0);  // 32 channels each
        tc_commit(&s_full[w]);
      }
      __syncwarp();
    };
    scores(0);
    for (int j = 0; ok && j <= jobs; ++j) {  // S of job j has been read and P of job j - 1 written
      if (!wait(&turn[w], j & 1)) break;
      if (j > 0) {
        const int i = j - 1, half = half_of(w, i), slot = i & 1, buf = tile_of(i) % kBuf;
        tc_after();
        if (elect()) {
          const uint64_t b = operand(sb + kShV + buf * kVBytes + half * (kVBytes / 2));
          #pragma unroll
          for (int c = 0; c < 4; ++c)  // 16 tokens each
            mma_f16_ta(tmem + w * 256 + 128, tmem + w * 256 + kHalf + 32 * slot + 8 * c, b + 2 * c, i > 0 || c > 0);
          tc_commit(&pv_done[w][slot]);
          if (!two || half == 1) tc_commit(&kv_empty[buf]);
        }
        __syncwarp();
      }
      if (j + 1 < jobs) scores(j + 1);
    }
  }
  if (!ok && lane == 0 && p.c.status) atomicOr(p.c.status, KV1B_STATUS_TIMEOUT);
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 0) tmem_free(tmem);
}

// The prefix's units, then the CTAs of the sequences' own tokens: where the prefix leaves SMs idle the two
// parts run side by side.
template <bool kFine>
__global__ void __launch_bounds__(kShThreads, 1) paged_shared_kernel(const PagedAttendParams p, const PagedSharedParams s, const int G,
                                                                      const int units) {
  static_assert(kThreads == 384 && kShThreads == 512 && kSmem <= kShSmem, "one launch for both parts");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  if (static_cast<int>(blockIdx.x) < units) prefix_cta(p, s, blockIdx.x, smem);
  else if (threadIdx.x < kThreads) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(160));  // 3 x 160 + 32 = 4 x 128
    attend_cta<kFine, true>(p, G, blockIdx.x - units, smem);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(32));
  }
}

// One (sequence, kv-head, query head) per block: the sequence's own pieces and the prefix's.
__global__ void __launch_bounds__(128) paged_shared_merge_kernel(const PagedAttendParams p, const PagedSharedParams s, const int G) {
  __shared__ float2 s_head[kMaxPieces];
  __shared__ float s_max[4];
  pdl_wait();
  const int b = blockIdx.x / p.c.Hkv, h = blockIdx.x - b * p.c.Hkv, g = blockIdx.y;
  const int64_t out_row = static_cast<int64_t>(b) * p.Hq + static_cast<int64_t>(h) * G + g;
  const int stride = p.packed ? 8 : G;  // rows of a piece
  // pieces of a segment of the plan: one row of p.rows, or slot 1 of its first CTA and slot 0 of the others
  struct Seg {
    const float *first, *rest;
    int n;
  };
  auto segment = [&](int seq, int64_t row, int i) {
    const int2 at = p.spread[static_cast<int64_t>(seq) * p.c.Hkv + h];
    Seg s;
    s.n = at.y;
    s.first = at.y == 1 ? p.rows + row * kRow : p.part + ((static_cast<int64_t>(at.x) * 2 + 1) * stride + i) * kRow;
    s.rest = p.part + (static_cast<int64_t>(at.x) * 2 * stride + i) * kRow;
    return s;
  };
  const int64_t step = 2LL * stride * kRow;
  const Seg own = segment(p.packed + b, out_row, g);
  const int r = b * G + g;
  auto own_piece = [&](int i) { return i == 0 ? own.first : own.rest + i * step; };
  if (p.packed) {
    const Seg pre = segment(r >> 3, static_cast<int64_t>(p.B) * p.Hq + static_cast<int64_t>(h) * p.B * G + r, r & 7);
    merge_pieces(own.n + pre.n,
                 [&](int i) { return i < own.n ? own_piece(i) : (i == own.n ? pre.first : pre.rest + (i - own.n) * step); }, s_head, s_max,
                 p.out, p.q_dtype, out_row * kD);
    return;
  }
  const int rows = s.two ? 256 : 128, rt = r / rows, in = r - rt * rows;
  // each token range has the same number of pieces; those without a tile are empty
  const bool any = prefix_tokens(p, false) > 0;
  const float* base = s.pieces + ((static_cast<int64_t>(h) * s.row_tiles + rt) * s.splits * 256 + in) * kRow;
  const int per = s.two ? 1 : 2;
  auto piece = [&](int i) -> const float* {
    if (i < own.n) return own_piece(i);
    i -= own.n;
    return base + (per == 1 ? static_cast<int64_t>(i) * 256 : static_cast<int64_t>(i >> 1) * 256 + (i & 1) * 128) * kRow;
  };
  merge_pieces(own.n + (any ? s.splits * per : 0), piece, s_head, s_max, p.out, p.q_dtype, out_row * kD);
}

}  // namespace paged
}  // namespace kv1b

using namespace kv1b;

static cudaError_t launch_prefix(const PagedAttendParams& p, const PagedSharedParams& s, int32_t G, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0}, configured_fine{0};
  const bool fine = p.q_dtype == KV1B_DTYPE_F16;
  const auto kernel = fine ? paged::paged_shared_kernel<true> : paged::paged_shared_kernel<false>;
  cudaError_t e = configure_smem(reinterpret_cast<const void*>(kernel), paged::kShSmem, fine ? &configured_fine : &configured);
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(p.B) * p.Hq;
  e = launch_pdl(paged::paged_query_codes_kernel, dim3(static_cast<unsigned>((rows + 7) / 8)), dim3(256), 0, stream, p, s, G);
  if (e != cudaSuccess) return e;
  const int units = p.c.Hkv * s.row_tiles * s.splits;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(units + p.ncta)), dim3(paged::kShThreads), paged::kShSmem, stream, p, s, G, units);
}

cudaError_t kv1b_launch_paged_shared(const PagedAttendParams& p, const PagedSharedParams& s, int32_t G, cudaStream_t stream) {
  const cudaError_t e = p.packed ? kv1b_launch_paged_pieces(p, G, stream) : launch_prefix(p, s, G, stream);
  if (e != cudaSuccess) return e;
  return launch_pdl(paged::paged_shared_merge_kernel, dim3(static_cast<unsigned>(p.B) * p.c.Hkv, G), dim3(128), 0, stream, p, s, G);
}

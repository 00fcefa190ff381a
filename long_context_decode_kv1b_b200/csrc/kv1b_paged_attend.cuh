// kv1b_paged_attend.cuh -- decode attention over a paged cache, one query token per sequence, uneven
// lengths read on the device: one CTA's part.
//
// Split.  The visible 32-token blocks of all (sequence, kv-head) segments are laid end to end and cut
// into one equal contiguous range per CTA (one CTA per SM), whatever the lengths, and a CTA's range into
// one equal run per warp.  Each warp streams its run through its own ring of kStages shared-memory
// buffers (one 3,200-byte bulk copy per block, an mbarrier each), so nothing waits on another warp until
// the end.  A segment inside one run is finished by its warp; the warps' pieces of a longer one meet in
// shared memory; one that a range boundary cuts leaves a partial row per CTA, which a second kernel
// merges.  (One segment at a time for the whole CTA, every 16th block a warp's, cost 5 us a segment in
// barriers and restarts: 53 us for 32 segments of 61 tokens on 4 CTAs.)
//
// Per block and warp (lane (g, t) = (lane / 4, lane % 4)), for up to 8 query heads g:
//   scores   s8 m16n8k32 products: rows 0 - 7 of A are the heads' 4-bit codes, rows 8 - 15 ones, columns
//            of B eight tokens' sign bits, one AND per register (the bit stays in place and the code
//            carries 2^(3 - place)).  Lane (g, t) gets 8 A and 8 Bc of head g, tokens 8 t + 2 i + {0, 1}:
//            with the row order of the block, all eight tokens of its code words, so probabilities are
//            formed where the next product wants them and nothing is shuffled;
//   softmax  log2 units against a reference that a warp raises only when a logit passes it by kTau;
//   P.V      v = min + scale code, so sum p v = sum p min + sum (p scale) code.  f16 m16n8k16 products with
//            fp32 sums: A = 16 channels x 16 tokens of codes, one AND per register (a nibble in the low
//            mantissa bits is a binary16 subnormal, code 2^-24, or 2^-20 where the nibble is the byte's
//            upper one: those tokens' weights are 2^-4 lower), B = p scale, one multiplication per pair of
//            tokens and value group.  A last pair of products with the four groups' mins and a row of ones
//            gives sum p min and the normaliser from the same binary16 p, so p's rounding cancels in the
//            quotient.
// Roundings: p scale is rounded to 11 bits for bf16 results, which have 8; for fp16 results its remainder
// (exact: the product of two 11-bit numbers has 22) goes through a second set of products.  What is left is
// the subnormal codes' own loss: the tensor cores line a product up by its operands' exponents, so the sums
// of scale code keep some ten bits fewer than fp32's 24 (2^-14.6 of them seen).
// Range: p = 2^(x - m + kBase) <= 2^15 and scale < 2 keep p scale finite.  The sums of scale code have a unit, a
// power of two: 1 for ordinary blocks, whose largest scale is in [2^-7, 2), and else such that a block's scales, as
// multiples of it, are below 2 and reach 2^-3.  Those blocks' scales are divided by it in place, and the sums are
// rescaled where a block needs another unit, up or down (exactly: fp32 by a power of two).  Small values held to
// unit 1 lost their codes where p scale is below 2^-25: errors of 5.6e-7 for 4,096 tokens of 1e-5 behind one 6 nats
// above them, a result of 1e-6.  The test for them costs 1 to 3 % (1M tokens x 8 heads: 190.6 and 193.1 us over other
// pages each time, 174 and 179 over the same); where every block is divided, 212 us instead of 180.
// p keeps 11 bits down to 2^-21 of the reference (2^7), and to 2^-17 for the weights that are 2^-4 lower; p scale, in
// units, keeps 11 bits while it is 2^-14 or more.  Below, each loses 2^-25 at most: of a token's code part no more than
// 2^-24 units, relative to a reference of weight 1.
//
// 12 warps: their 168 registers hold the loop's sums, operands and addresses (the fp16 instance, which keeps the
// weights' remainders too, spills 32 bytes), where 16 warps' 128 spilled; 8 warps of 255 hid less of the products'
// latency (178, 190 and 222 us for 1M tokens x 8 heads).
// 609 warp instructions a block (values expanded to binary16 by fma, a page entry and an address per
// block) became 389 and 243 us for 1M tokens x 8 heads 174; with the units 395 and 179, the issue slots 55 % and the ALU
// 53 % busy: dependencies of fixed latency bound it.
#pragma once
#include "kv1b_paged_device.cuh"

namespace kv1b {
namespace paged {

constexpr int kWarps = kAttendWarps;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 4;

constexpr int kQuerySlots = 256;  // prepared query rows a round holds
constexpr int kMaxSegs = 64;      // segments a round holds

// a segment of a round, in blocks from the round's start
struct Seg {
  int base, nb;  // first block (below 0 where the CTA's range begins inside the segment), blocks
  int b, h;
  int k;         // place of b among the sequences that see a block
  int skip_from, skip_to, pad;  // Visible
};

constexpr int kOffPre = kWarps * kStages * kBlkBytes;            // u32 [kMaxSeqs + 1] blocks before each sequence
constexpr int kOffLen = kOffPre + (kMaxSeqs + 4) * 4;            // i32 [kMaxSeqs]
constexpr int kOffSome = kOffLen + kMaxSeqs * 4;                 // u16 [kMaxSeqs]
constexpr int kOffSeg = kOffSome + kMaxSeqs * 2;                 // Seg [kMaxSegs]
constexpr int kOffPlane = kOffSeg + kMaxSegs * 32;               // u32 [kQuerySlots][4 planes][4]
constexpr int kOffConst = kOffPlane + kQuerySlots * 64;          // f32 [kQuerySlots][4]: c1, c2, c0
constexpr int kOffRows = kOffConst + kQuerySlots * 16;           // f16 [2][8]: ones, zeros
constexpr int kOffSigns = kOffRows + 32;                         // f32 [3][128]
constexpr int kSmem = kOffSigns + 3 * kD * 4;
constexpr int kOffRed = 0;                                       // f32 [kWarps][G][kRow], over the ring once it is drained
static_assert(kOffPre % 16 == 0 && kOffRows % 16 == 0 && kWarps * KV1B_MAX_GROUP * kRow * 4 <= kOffPre && kSmem + 2048 <= 227 * 1024, "shared memory");

// Block i of a segment: its place in the sequence.
__device__ __forceinline__ int own_block(const Seg& g, int i) { return i < g.skip_from ? i : i + (g.skip_to - g.skip_from); }

// The copy side's place in a round's blocks.  Stretches of blocks that lie behind one another in a page
// are walked by a pointer; the page entry of the next stretch is loaded when one begins.  What follows from
// the segment is read from shared memory when it is needed: registers are what the loop is short of.
struct Ahead {
  const uint8_t* ptr;  // next block, null where the page is not there
  int in;              // blocks of the stretch that are left
  int left;            // blocks of the warp's run behind the stretch
  int s, i;            // segment and block behind the stretch
  int page;            // page entry there
  __device__ __forceinline__ void look_up(const Seg& g, const PagedAttendParams& p) {
    const int32_t* list = g.b < p.packed ? p.prefix_pages : p.table + (g.b - p.packed) * p.table_stride;
    page = __ldg(list + (own_block(g, i) >> p.c.bpp_shift));
  }
  __device__ __forceinline__ void next_stretch(const Seg* seg, const PagedAttendParams& p) {
    const Seg g = seg[s];
    const int off = own_block(g, i) & ((1 << p.c.bpp_shift) - 1);
    const bool ok = page >= 0 && page < p.c.num_pages;
    ptr = ok ? p.c.pages + ((((static_cast<int64_t>(page) * p.c.Hkv + g.h) << p.c.bpp_shift) + off) * kBlkBytes) : nullptr;
    if (!ok && (threadIdx.x & 31) == 0 && p.c.status) atomicOr(p.c.status, KV1B_STATUS_BAD_INDEX);
    in = min(min((1 << p.c.bpp_shift) - off, g.nb - i), left);
    if (i < g.skip_from) in = min(in, g.skip_from - i);
    left -= in;
    i += in;
    if (left > 0) {
      if (i == g.nb) {
        ++s;
        i = 0;
        look_up(seg[s], p);
      } else {
        look_up(g, p);
      }
    }
  }
};

// The first block from i on of which the query may see only a part: where the sinks end, where the window
// begins (the first block of all where there is none), the last one.
__device__ __forceinline__ int next_edge(const Seg& g, int i) {
  return i < g.skip_from ? g.skip_from - 1 : (i == g.skip_from ? i : g.nb - 1);
}

constexpr int kCodeBits = 24;  // codes enter the products as binary16 subnormals, units of 2^-24
__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((127 + e) << 23); }

// The query heads of kv-head h that sequence b of the plan serves: G, or up to 8 rows b G' + g of the batch.
struct Heads {
  int V, G, Hq, B;
  __device__ __forceinline__ int count(int b) const { return b < V ? min(8, B * G - 8 * b) : G; }
  // row of q and out of head i
  __device__ __forceinline__ int64_t query(int b, int h, int i) const {
    const int r = 8 * b + i;
    return b < V ? static_cast<int64_t>(r / G) * Hq + h * G + r % G : static_cast<int64_t>(b - V) * Hq + h * G + i;
  }
  // row of p.rows of head 0
  __device__ __forceinline__ int64_t row(int b, int h) const {
    return b < V ? static_cast<int64_t>(B) * Hq + static_cast<int64_t>(h) * B * G + 8 * b : static_cast<int64_t>(b - V) * Hq + h * G;
  }
};

// kFine: the weights of the codes in two binary16 parts (fp16 results); one part is enough for bf16.
// `cta` of p.ncta, kThreads threads, kSmem bytes at `smem` (128-byte aligned).
template <bool kFine, bool kBeside>
__device__ __forceinline__ void attend_cta(const PagedAttendParams& p, const int G_, const int cta, uint8_t* smem) {
  const Heads heads = {p.packed, G_, p.Hq, p.B};
  const int G = p.packed ? 8 : G_;  // rows that a segment may have
  __shared__ __align__(8) uint64_t bars[kWarps][kStages];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint32_t* pre = reinterpret_cast<uint32_t*>(smem + kOffPre);
  int* slen = reinterpret_cast<int*>(smem + kOffLen);
  Seg* seg = reinterpret_cast<Seg*>(smem + kOffSeg);
  uint32_t* planes = reinterpret_cast<uint32_t*>(smem + kOffPlane);
  float4* consts = reinterpret_cast<float4*>(smem + kOffConst);
  float* red = reinterpret_cast<float*>(smem + kOffRed);

  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&bars[warp][s], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  pdl_launch_dependents();
  float* signs = reinterpret_cast<float*>(smem + kOffSigns);
  for (int i = threadIdx.x; i < KV1B_MAX_ROUNDS * kD; i += kThreads) signs[i] = __ldg(p.c.signs + i);
  __shared__ Plan pl;
  {
    const Plan mine = make_plan<kThreads, kBeside>(p, pre, slen, reinterpret_cast<uint16_t*>(smem + kOffSome), p.ncta, cta == 0);
    if (lane == 0) pl = mine;  // every warp writes the same
    __syncwarp();
  }

  // sequences that see nothing: zeros
  for (int b = p.rows ? p.B : cta; b < p.B; b += p.ncta)  // (none are packed here)
    if (pre[b + 1] == pre[b])
      for (int e = threadIdx.x; e < p.Hq * kD; e += kThreads) store_out(p.out, p.q_dtype, static_cast<int64_t>(b) * p.Hq * kD + e, 0.0f);
  if (p.rows)
    for (int64_t i = static_cast<int64_t>(cta) * kThreads + threadIdx.x; i < static_cast<int64_t>(pl.B) * pl.Hkv;
         i += static_cast<int64_t>(p.ncta) * kThreads) {
      const int b = static_cast<int>(i / pl.Hkv);
      if (pre[b + 1] == pre[b]) p.spread[i] = make_int2(0, 0);
    }
  if (cta >= pl.n || pl.S == 0) {
    if (threadIdx.x == 0 && !p.rows) p.spread[cta] = make_int2(0, 0);
    return;
  }

  const int64_t border = pl.begin(cta + (lane & 1));  // both ends in one go
  const int64_t r0 = __shfl_sync(kFull, border, 0);
  __shared__ int64_t r1;  // every warp writes the same; kept out of the loop's registers
  if (lane == 1) r1 = border;
  __syncwarp();
  if (r0 == r1) {  // within what a segment counts besides its blocks
    if (threadIdx.x == 0 && !p.rows) p.spread[cta] = make_int2(0, 0);
    return;
  }
  const uint32_t ring = smem_u32(smem) + warp * kStages * kBlkBytes;
  const int max_segs = min(kMaxSegs, kQuerySlots / G);
  if (threadIdx.x < 8) reinterpret_cast<uint32_t*>(smem + kOffRows)[threadIdx.x] = threadIdx.x < 4 ? 0x3C003C00u : 0u;
  const uint32_t side_row = smem_u32(smem) + kOffRows + (g == 4 ? 0 : 16);  // rows 4 and 5 .. 7 of the side product
  uint32_t phases = 0;  // bit s: parity of stage s's next completion
  bool gave_up = false;

  // ---- rounds of up to max_segs segments; nearly always one
  for (int64_t a = r0; a < r1;) {
    // the round's segments
    int nseg;
    {
      int lo = 0, hi = pl.nsome;  // the sequence of block a: largest lo with Hkv pre[some[lo]] <= a
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pl.first_block(mid) <= a) lo = mid;
        else hi = mid;
      }
      const int h0 = static_cast<int>(quotient(a - pl.first_block(lo), pl.blocks(lo)));
      bool valid = false;
      if (static_cast<int>(threadIdx.x) < max_segs) {
        const int id = h0 + threadIdx.x, k = lo + id / pl.Hkv, h = id % pl.Hkv;
        if (k < pl.nsome) {
          const int nb = pl.blocks(k);
          const int64_t base = pl.first_block(k) + static_cast<int64_t>(h) * nb;
          valid = base < r1;
          if (valid) {
            const int b = pl.some[k];
            const Visible v = visible(pl.len[b], p.window, p.sinks);
            seg[threadIdx.x] = {static_cast<int>(base - a), nb, b, h, k, v.skip_from, v.skip_to, 0};
          }
        }
      }
      nseg = __syncthreads_count(valid);
    }
    const int n = static_cast<int>(min(r1 - a, static_cast<int64_t>(seg[nseg - 1].base) + seg[nseg - 1].nb));
    const int run_q = n / kWarps, run_r = n % kWarps;  // the first run_r runs are one longer
    auto run_begin = [&](int w) { return w * run_q + min(w, run_r); };
    auto run_owner = [&](int x) {
      const int longer = run_r * (run_q + 1);
      return x < longer ? x / (run_q + 1) : run_r + (x - longer) / run_q;
    };
    const int w0 = run_begin(warp), w1 = run_begin(warp + 1);

    // the round's rows: those of the packed segments, which come first, then the others'
    int npacked = 0;
    if (p.packed)
      while (npacked < nseg && seg[npacked].b < p.packed) ++npacked;
    const int nrow = npacked * G + (nseg - npacked) * heads.G;
    auto slot_of = [&](int r) {  // its segment G + head
      if (r < npacked * G) return r;
      const int x = (r - npacked * G) / heads.G;
      return (npacked + x) * G + r - npacked * G - x * heads.G;
    };
    // a warp's first two are loaded before the copies fill the memory's queues
    auto load_row = [&](int r, float (&x)[4]) {
      const int s = slot_of(r);
      const Seg sg = seg[s / G];
      const int i = min(s % G, heads.count(sg.b) - 1);  // a row that is not there: the last one again, unused
      load_query(p.q, heads.query(sg.b, sg.h, i) * kD + 4 * lane, p.q_dtype, x);
    };
    float q0[4], q1[4];
    if (warp < nrow) load_row(warp, q0);
    if (warp + kWarps < nrow) load_row(warp + kWarps, q1);

    // ---- copy side: `ahead` walks kStages blocks in front of the compute
    Ahead ahead;
    ahead.in = 0;
    ahead.left = w1 - w0;
    uint32_t absent = 0;  // bit s: stage s holds no block (its page is outside the cache)
    auto issue = [&](int s) {
      if (ahead.in == 0) ahead.next_stretch(seg, p);
      absent = ahead.ptr ? absent & ~(1u << s) : absent | (1u << s);
      if (ahead.ptr) {
        if (lane == 0) block_g2s(ring + s * kBlkBytes, ahead.ptr, &bars[warp][s]);
        ahead.ptr += kBlkBytes;
      }
      --ahead.in;
    };
    struct { int s, i, left; } cur = {0, 0, w1 - w0};
    if (cur.left > 0) {
      int k = 0;  // the segment of block w0
      for (int x = lane; x < nseg; x += 32)
        if (seg[x].base <= w0) k = x;
      k = __reduce_max_sync(kFull, k);
      ahead.s = k;
      ahead.i = w0 - seg[k].base;
      ahead.look_up(seg[k], p);
      cur.s = k;
      cur.i = ahead.i;
      for (int s = 0; s < kStages && ahead.in + ahead.left > 0 && !gave_up; ++s) issue(s);
    }

    // ---- the round's queries
    const float qs = __fmul_rn(__fmul_rn(p.scale, 1.4426950408889634f), 1.0f / kD);
    for (int r0 = warp; r0 < nrow; r0 += kWarps) {
      if (r0 >= 2 * kWarps) load_row(r0, q0);
      const QueryPrep qp = query_prep_values(q0, signs);
      #pragma unroll
      for (int j = 0; j < 4; ++j) q0[j] = q1[j];
      const int r = slot_of(r0);
      if (lane == 0) {
        #pragma unroll
        for (int j = 0; j < 4; ++j)
          reinterpret_cast<uint4*>(planes)[r * 4 + j] = make_uint4(qp.planes[j][0], qp.planes[j][1], qp.planes[j][2], qp.planes[j][3]);
        // log2 logit = (c1 8A + c2 8Bc + c0) (N/C):  delta (2A - Sq) + vl (2 Bc - 128), times scale log2(e) / 128
        consts[r] = make_float4(__fmul_rn(0.25f * qp.delta, qs), __fmul_rn(0.25f * qp.vl, qs),
                                -__fmul_rn(__fadd_rn(__fmul_rn(qp.delta, static_cast<float>(qp.sq)), 128.0f * qp.vl), qs), 0.0f);
      }
    }
    __syncthreads();

    // acc: sums of weight scale code (units of 2^-24); side: rows 0 .. 3 sums of weight min per group, row 4 of weight
    float acc[8][4], side[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    #pragma unroll
    for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
    float m = kNoRef;  // reference of head g
    int unit = 0;      // acc is in units of 2^(unit - 24)
    // element (i, e, hi) of the weighted value sum of head 2 t + e, channel 16 i + g + 8 hi
    auto value = [&](int i, int e, int hi) {
      return __fmaf_rn(acc[i][2 * hi + e], power_of_two(kCodeBits + unit), __shfl_sync(kFull, side[e], 4 * (i >> 1) + t));
    };
    // the warp's sums of a segment to a piece [head][kRow]
    auto put_piece = [&](float* w) {
      const int n_heads = heads.count(seg[cur.s].b);
      if (t == 0 && g < n_heads) w[g * kRow] = m;
      #pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int hd = 2 * t + e;
        if (g == 4 && hd < n_heads) w[hd * kRow + 1] = side[e];
        #pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float lo = value(i, e, 0), hi = value(i, e, 1);
          if (hd < n_heads) {
            w[hd * kRow + 2 + 16 * i + g] = lo;
            w[hd * kRow + 2 + 16 * i + g + 8] = hi;
          }
        }
      }
    };
    int stage = 0;
    bool last = w0 == w1;  // the sums in registers are a piece that the CTA merges (an empty run's: nothing)
    while (cur.left > 0) {
      // A operand: k-row 4 t + j of product kb, half hi is channel 32 t + 8 j + r, r = 2 kb + hi, its code
      // times 2^(3 - (r & 3)) (the sign bit stays at place r & 3 of its byte)
      uint32_t aq[4][2];
      float4 cc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      {
        uint32_t pw[4] = {0u, 0u, 0u, 0u};
        if (g < heads.count(seg[cur.s].b)) {
          #pragma unroll
          for (int j = 0; j < 4; ++j) pw[j] = planes[((cur.s * G + g) * 4 + j) * 4 + t];
          cc = consts[cur.s * G + g];
        }
        #pragma unroll
        for (int kb = 0; kb < 4; ++kb)
          #pragma unroll
          for (int hi = 0; hi < 2; ++hi) {
            const int r = 2 * kb + hi;
            uint32_t code = 0u;
            #pragma unroll
            for (int j = 0; j < 4; ++j) code |= ((pw[j] >> r) & 0x01010101u) << j;
            aq[kb][hi] = code << (3 - (r & 3));
          }
      }
      const float c1 = cc.x, c2 = cc.y, c0 = cc.z;
      #pragma unroll
      for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
      side[0] = side[1] = side[2] = side[3] = 0.0f;
      m = 0.0f;
      bool fresh = true;   // no block has set m
      unit = 0;
      uint32_t ordinary = 0x20002000u;  // the bit that a scale of [2^-7, 2) has; none where every block is looked at
      const bool starts = cur.i == 0;
      const int count = min(cur.left, seg[cur.s].nb - cur.i);  // blocks of the segment in the warp's run
      const bool ends = cur.i + count == seg[cur.s].nb;
      int edge_at = next_edge(seg[cur.s], cur.i);

      for (int x = cur.i; x < cur.i + count; ++x) {
        const uint32_t st = ring + stage * kBlkBytes;
        if (!((absent >> stage) & 1u)) {
          if (!__all_sync(kFull, mbar_wait(&bars[warp][stage], (phases >> stage) & 1u, gave_up ? 1 : kWaitTries)))
            gave_up = true;  // every lane alike
          phases ^= 1u << stage;
          uint32_t seen = 0xFFFFFFFFu;
          if (x == edge_at) {
            // which of the block's tokens the query sees.  Unseen ones: what their places hold (another
            // sequence's remains, infinities) must not reach a product, so their scale, min and norm
            // become zeros and their weights are zero
            const Seg& sg = seg[cur.s];
            const int len = pl.len[sg.b], tk = own_block(sg, x) * kBlkTok + lane;
            const int wstart = (p.window > 0 && len > p.window) ? len - p.window : 0;
            const bool on = tk < len && (tk >= wstart || tk < p.sinks);
            seen = __ballot_sync(kFull, on);
            if (!on) {
              uint8_t* bp = smem + (warp * kStages + stage) * kBlkBytes;
              reinterpret_cast<float*>(bp + kBlkOffNc)[lane] = 0.0f;
              #pragma unroll
              for (int q = 0; q < 4; ++q) {
                reinterpret_cast<uint16_t*>(bp + kBlkOffScale)[32 * q + lane] = 0;
                reinterpret_cast<uint16_t*>(bp + kBlkOffMin)[32 * q + lane] = 0;
              }
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the next copy to the stage
            }
            __syncwarp();
            edge_at = next_edge(sg, x + 1);
          }
          // ---- scores
          // (Where loads stand matters: the mins' right before their products made 191 of 176 us for 1M tokens, the
          // norms' behind the scores 182.)
          float dot[8];
          uint32_t ncr[8], mn[4];
          {
            uint32_t kw[4];
            ldsm_x4(kw, st + lane * 16);
            lds128(ncr, st + kBlkOffNc + 32 * t);
            lds128(ncr + 4, st + kBlkOffNc + 32 * t + 16);
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
              // the sums start at the bits of 1.5 2^23: as a float, an entry is that plus its integer
              int d[4];
              const uint32_t w[2] = {kw[i], kw[i] >> 4};
              imma_from(d, 0x4B400000, aq[0][0], 0x08080808u, aq[0][1], 0x04040404u, w[0] & 0x01010101u, w[0] & 0x02020202u);
              imma(d, aq[1][0], 0x02020202u, aq[1][1], 0x01010101u, w[0] & 0x04040404u, w[0] & 0x08080808u);
              imma(d, aq[2][0], 0x08080808u, aq[2][1], 0x04040404u, w[1] & 0x01010101u, w[1] & 0x02020202u);
              imma(d, aq[3][0], 0x02020202u, aq[3][1], 0x01010101u, w[1] & 0x04040404u, w[1] & 0x08080808u);
              #pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float a8 = __fadd_rn(__int_as_float(d[e]), -12582912.0f);
                const float b8 = __fadd_rn(__int_as_float(d[2 + e]), -12582912.0f);
                dot[2 * i + e] = __fmaf_rn(c1, a8, __fmaf_rn(c2, b8, c0));
              }
            }
          }
          lds128(mn, g < 4 ? st + kBlkOffMin + g * 64 + 16 * t : side_row);
          {
            // the block's 128 scales, four a lane: whether one is 2 or more, or a lane has none of 2^-7
            const uint32_t at = st + kBlkOffScale + 8 * lane;
            uint32_t w0, w1;
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w0), "=r"(w1) : "r"(at) : "memory");
            if (__any_sync(kFull, ((w0 | w1) & 0x40004000u) != 0 || ((w0 | w1) & ordinary) == 0)) {
              uint32_t top = max(max(w0 & 0xFFFFu, w0 >> 16), max(w1 & 0xFFFFu, w1 >> 16));
              top = __reduce_max_sync(kFull, top);  // the largest, as its bits
              if (top != 0) {
                const int k = top >= 0x400u ? static_cast<int>(top >> 10) - 15 : 7 - __clz(top);  // 2^k <= it < 2^(k + 1)
                if (k > unit || k < unit - (unit == 0 ? 7 : 3)) {
                  const int to = k <= 0 && k >= -7 ? 0 : k;
                  const float f = power_of_two(unit - to);
                  unit = to;
                  ordinary = to == 0 ? 0x20002000u : 0u;
                  #pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    #pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][e] = __fmul_rn(acc[i][e], f);
                  }
                }
                if (unit != 0) {  // by 2^-unit, in two factors: neither 2^24 nor 2^-15 is a normal binary16
                  const int up = max(min(-unit, 12), -14);
                  const uint32_t f0 = static_cast<uint32_t>(15 + up) * 0x04000400u, f1 = static_cast<uint32_t>(15 - unit - up) * 0x04000400u;
                  w0 = hmul2(hmul2(w0, f0), f1);
                  w1 = hmul2(hmul2(w1, f0), f1);
                  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(w0), "r"(w1) : "memory");
                  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the next copy to the stage
                  __syncwarp();
                }
              }
            }
          }
          // exponents of the weights: logit - m + kBase
          float y[8];
          {
            const float off = kBase - m;
            #pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = __fmaf_rn(dot[j], __uint_as_float(ncr[j]), off);
          }
          if (seen != 0xFFFFFFFFu) {
            const uint32_t mine = seen >> (8 * t);
            #pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = (mine >> j) & 1u ? y[j] : -INFINITY;
          }
          float mx = fmaxf(max3(max3(y[0], y[1], y[2]), y[3], y[4]), max3(y[5], y[6], y[7]));
          if (__any_sync(kFull, mx > kBase + kTau) || fresh) {  // rare: raise references
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
            const float rise = fresh || mx > kBase + kTau ? mx - kBase : 0.0f;
            const float alpha = fresh ? 0.0f : ex2(-rise);
            m += rise;
            #pragma unroll
            for (int j = 0; j < 8; ++j) y[j] -= rise;
            const float a0 = __shfl_sync(kFull, alpha, 8 * t), a1 = __shfl_sync(kFull, alpha, 8 * t + 4);
            #pragma unroll
            for (int i = 0; i < 8; ++i) {
              acc[i][0] = __fmul_rn(acc[i][0], a0);
              acc[i][1] = __fmul_rn(acc[i][1], a1);
              acc[i][2] = __fmul_rn(acc[i][2], a0);
              acc[i][3] = __fmul_rn(acc[i][3], a1);
            }
            side[0] = __fmul_rn(side[0], a0);
            side[1] = __fmul_rn(side[1], a1);
            fresh = false;
          }
          uint32_t pw[4];
          #pragma unroll
          for (int i = 0; i < 4; ++i) pw[i] = pack_f16(ex2(y[2 * i]), ex2(y[2 * i + 1]));
          {
            hmma(side, mn[0], 0u, mn[1], 0u, pw[0], pw[1]);
            hmma(side, mn[2], 0u, mn[3], 0u, pw[2], pw[3]);
          }
          // the codes of pairs 1 and 3 sit four bits higher
          pw[1] = hmul2(pw[1], 0x2C002C00u);
          pw[3] = hmul2(pw[3], 0x2C002C00u);
          // ---- P.V, value group by value group (32 channels: rows of two products)
          #pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t cw[4], sc[4], wt[4], rest[4];
            lds128(sc, st + kBlkOffScale + q * 64 + 16 * t);
            ldsm_x4(cw, st + kBlkOffCodes + (32 * q + lane) * 16);  // rows g, g + 8, g + 16, g + 24; word t
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
              wt[i] = hmul2(pw[i], sc[i]);
              if (kFine) rest[i] = hfma2(pw[i], sc[i], wt[i] ^ 0x80008000u);
            }
            #pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t lo = cw[2 * u], hi = cw[2 * u + 1], lo8 = lo >> 8, hi8 = hi >> 8;
              const uint32_t a0 = lo & 0x000F000Fu, a1 = hi & 0x000F000Fu, a2 = lo & 0x00F000F0u, a3 = hi & 0x00F000F0u;
              const uint32_t b0 = lo8 & 0x000F000Fu, b1 = hi8 & 0x000F000Fu, b2 = lo8 & 0x00F000F0u, b3 = hi8 & 0x00F000F0u;
              hmma(acc[2 * q + u], a0, a1, a2, a3, wt[0], wt[1]);
              hmma(acc[2 * q + u], b0, b1, b2, b3, wt[2], wt[3]);
              if (kFine) {
                hmma(acc[2 * q + u], a0, a1, a2, a3, rest[0], rest[1]);
                hmma(acc[2 * q + u], b0, b1, b2, b3, rest[2], rest[3]);
              }
            }
          }
        } else if (x == edge_at) {  // a block that is not there: the edges behind it still count
          edge_at = next_edge(seg[cur.s], x + 1);
        }
        __syncwarp();
        // ---- the stage's next block
        if (ahead.in + ahead.left > 0 && !gave_up) issue(stage);
        else if (gave_up) absent |= 1u << stage;
        stage = stage + 1 == kStages ? 0 : stage + 1;
      }
      if (fresh) m = kNoRef;
      cur.left -= count;

      if (starts && ends) {  // all of it: finished here
        const Seg& sg = seg[cur.s];
        const int64_t qrow = heads.query(sg.b, sg.h, 0);
        if (p.rows) {
          put_piece(p.rows + heads.row(sg.b, sg.h) * kRow);
        } else {
          #pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int hd = 2 * t + e;
            // (one reciprocal: 32 divisions were 2.6 of 18.3 us for 64 sequences of 40 tokens)
            const float den = __shfl_sync(kFull, side[e], 16 + t), r = den != 0.0f ? __frcp_rn(den) : 0.0f;
            uint16_t* const row = static_cast<uint16_t*>(p.out) + (qrow + hd) * kD + g;
            #pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float lo = __fmul_rn(value(i, e, 0), r), hi = __fmul_rn(value(i, e, 1), r);
              const uint32_t w = kFine ? pack_result_f16(lo, hi) : pack_bf16(lo, hi);
              if (hd < G) {
                row[16 * i] = static_cast<uint16_t>(w);
                row[16 * i + 8] = static_cast<uint16_t>(w >> 16);
              }
            }
          }
        }
      } else if (cur.left > 0) {  // its end: the run goes on with another segment
        put_piece(p.first + (static_cast<int64_t>(cta) * kWarps + warp) * G * kRow);
      } else {
        last = true;
      }
      if (cur.left > 0) {
        ++cur.s;
        cur.i = 0;
      }
    }

    // ---- the warps' pieces meet: of segment x, warps wf .. wl have one each, in `red` or (an end inside the
    // warp's run) in `first`
    __syncthreads();  // the ring is drained, the pieces in `first` are written
    if (last) put_piece(red + warp * G * kRow);
    __syncthreads();
    // for the merge: pieces of the segment that goes on past the range, or of every segment (rows)
    for (int x = threadIdx.x; x < nseg; x += kThreads) {
      const Seg sg = seg[x];
      const bool starts = sg.base >= 0, ends = sg.base + sg.nb <= n;
      const int pieces = ends ? 1 : pl.owner(sg.k, sg.h, sg.nb - 1) - cta + 1;
      if (p.rows) {
        if (starts) p.spread[static_cast<int64_t>(sg.b) * pl.Hkv + sg.h] = make_int2(cta, pieces);
      } else if (x == nseg - 1 && a + n == r1) {
        p.spread[cta] = make_int2(static_cast<int>(heads.query(sg.b, sg.h, 0)), starts && !ends ? pieces : 0);
      }
    }
    for (int r = warp; r < nrow; r += kWarps) {  // a row (segment, head) per warp, four channels per lane
      const int x = slot_of(r) / G, hd = slot_of(r) - x * G;
      const Seg sg = seg[x];
      if (hd >= heads.count(sg.b)) continue;
      const int s = max(sg.base, 0), e = min(sg.base + sg.nb, n);
      const int wf = run_owner(s), wl = run_owner(e - 1);
      const bool starts = sg.base >= 0, ends = sg.base + sg.nb <= n;
      if (wf == wl && starts && ends) continue;  // finished by its warp
      const bool inside = e < run_begin(wl + 1);  // the last piece is in `first`
      const float* tail = p.first + ((static_cast<int64_t>(cta) * kWarps + wl) * G + hd) * kRow;
      float2 head = make_float2(kNoRef, 0.0f);  // lane w: piece w's m and l
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (lane >= wf && lane <= wl) head = *reinterpret_cast<const float2*>(red + (lane * G + hd) * kRow);
      if (inside) {
        if (lane == wl) head = *reinterpret_cast<const float2*>(tail);
        #pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = tail[2 + lane + 32 * i];
      }
      float M = head.x;
      #pragma unroll
      for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
      const float f = ex2(head.x - M);
      float num[4] = {0.0f, 0.0f, 0.0f, 0.0f}, den = 0.0f;
      #pragma unroll 4
      for (int w = wf; w <= wl; ++w) {
        const float fw = __shfl_sync(kFull, f, w), lw = __shfl_sync(kFull, head.y, w);
        const float* o = red + (w * G + hd) * kRow + 2 + lane;
        const bool in_first = inside && w == wl;
        #pragma unroll
        for (int i = 0; i < 4; ++i) num[i] = __fmaf_rn(fw, in_first ? v[i] : o[32 * i], num[i]);
        den = __fmaf_rn(fw, lw, den);
      }
      const int64_t qrow = heads.query(sg.b, sg.h, hd);
      if (starts && ends && !p.rows) {
        const float r = den != 0.0f ? __frcp_rn(den) : 0.0f;
        #pragma unroll
        for (int i = 0; i < 4; ++i) store_out(p.out, p.q_dtype, qrow * kD + lane + 32 * i, __fmul_rn(num[i], r));
      } else {
        float* row = starts && ends ? p.rows + (heads.row(sg.b, sg.h) + hd) * kRow
                                    : p.part + ((static_cast<int64_t>(cta) * 2 + (starts ? 1 : 0)) * G + hd) * kRow;
        if (lane == 0) *reinterpret_cast<float2*>(row) = make_float2(M, den);
        #pragma unroll
        for (int i = 0; i < 4; ++i) row[2 + lane + 32 * i] = num[i];
      }
    }
    a += n;
    if (a < r1) {  // the next round's copies land where the pieces were
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncthreads();
    }
  }
  if (gave_up) {
    if (lane == 0 && p.c.status) atomicOr(p.c.status, KV1B_STATUS_TIMEOUT);
    for (int s = 0; s < kStages; ++s) mbar_wait(&bars[warp][s], (phases >> s) & 1u, 64);  // a copy that is still under way
  }
}

}  // namespace paged
}  // namespace kv1b

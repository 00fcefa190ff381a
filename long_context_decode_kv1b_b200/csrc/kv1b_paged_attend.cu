// kv1b_paged_attend.cu -- decode attention over a paged cache, one query token per sequence, uneven
// lengths read on the device.
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
//   P.V      f16 m16n8k16 products: A = 16 channels x 16 tokens expanded from the codes in registers
//            (v = min + scale code by one fma per pair of tokens, a single rounding to binary16), B = the
//            probabilities as binary16, fp32 sums.  The normaliser is summed by the same product with a
//            row of ones, so the roundings of the weights cancel in the quotient.
// Values and weights are rounded to 11 bits because the result is: out has the query's 16-bit type.
// Weights are 2^(x - m + kBase) <= 2^15, so a weight keeps its 11 bits down to 2^-21 of the reference.
#include "kv1b_paged_device.cuh"

namespace kv1b {
namespace paged {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 3;

constexpr int kQuerySlots = 128;  // prepared query rows a round holds
constexpr int kMaxSegs = 64;      // segments a round holds

// a segment of a round, in blocks from the round's start
struct Seg {
  int base, nb;  // first block (below 0 where the CTA's range begins inside the segment), blocks
  int b, h;
};

constexpr int kOffPre = kWarps * kStages * kBlkBytes;            // u32 [kMaxSeqs + 1] blocks before each sequence
constexpr int kOffLen = kOffPre + (kMaxSeqs + 4) * 4;            // i32 [kMaxSeqs]
constexpr int kOffSome = kOffLen + kMaxSeqs * 4;                 // u16 [kMaxSeqs]
constexpr int kOffSeg = kOffSome + kMaxSeqs * 2;                 // Seg [kMaxSegs]
constexpr int kOffPlane = kOffSeg + kMaxSegs * 16;               // u32 [kQuerySlots][4 planes][4]
constexpr int kOffConst = kOffPlane + kQuerySlots * 64;          // f32 [kQuerySlots][4]: c1, c2, c0
constexpr int kSmem = kOffConst + kQuerySlots * 16;
constexpr int kOffRed = 0;                                       // f32 [kWarps][G][kRow], over the ring once it is drained
static_assert(kOffPre % 16 == 0 && kWarps * KV1B_MAX_GROUP * kRow * 4 <= kOffPre && kSmem + 2048 <= 227 * 1024, "shared memory");

// Block i of a segment: its place in the sequence.
__device__ __forceinline__ int own_block(const Visible& v, int j) { return j < v.skip_from ? j : j + (v.skip_to - v.skip_from); }

// A place in a round's blocks: segment and block within it.
struct Walk {
  int s, i, left;  // segment, block of it, blocks of the warp's run that are left
  int b, h, nb;
  Visible vis;
  __device__ __forceinline__ void enter(const Seg* seg, const Plan& pl, const PagedAttendParams& p) {
    const Seg g = seg[s];
    b = g.b;
    h = g.h;
    nb = g.nb;
    vis = visible(pl.len[b], p.window, p.sinks);
  }
  __device__ __forceinline__ void step(const Seg* seg, const Plan& pl, const PagedAttendParams& p) {
    --left;
    if (++i == nb && left > 0) {
      ++s;
      i = 0;
      enter(seg, pl, p);
    }
  }
};

__device__ __forceinline__ int page_entry(const PagedAttendParams& p, const Walk& w) {
  return __ldg(p.table + w.b * p.table_stride + (own_block(w.vis, w.i) >> p.c.bpp_shift));
}

__global__ void __launch_bounds__(kThreads, 1) paged_attend_kernel(const PagedAttendParams p, const int G) {
  extern __shared__ __align__(128) uint8_t smem[];
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
  const Plan pl = make_plan<kThreads>(p, pre, slen, reinterpret_cast<uint16_t*>(smem + kOffSome), gridDim.x, blockIdx.x == 0);

  // sequences that see nothing: zeros
  for (int b = p.rows ? p.B : blockIdx.x; b < p.B; b += gridDim.x)
    if (pre[b + 1] == pre[b])
      for (int e = threadIdx.x; e < p.Hq * kD; e += kThreads) store_out(p.out, p.q_dtype, static_cast<int64_t>(b) * p.Hq * kD + e, 0.0f);
  if (static_cast<int>(blockIdx.x) >= pl.n || pl.S == 0) return;

  const int64_t r0 = pl.begin(blockIdx.x), r1 = pl.begin(blockIdx.x + 1);
  if (r0 >= r1) return;
  const uint32_t ring = smem_u32(smem) + warp * kStages * kBlkBytes;
  const int max_segs = min(kMaxSegs, kQuerySlots / G);
  const float qs = __fmul_rn(__fmul_rn(p.scale, 1.4426950408889634f), 1.0f / kD);
  float* first = p.first + (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * G * kRow;
  uint32_t phases = 0;  // bit s: parity of stage s's next completion
  bool gave_up = false;

  // ---- rounds of up to max_segs segments; nearly always one
  for (int64_t a = r0; a < r1;) {
    // the round's segments
    {
      int lo = 0, hi = pl.nsome;  // the sequence of block a: largest lo with Hkv pre[some[lo]] <= a
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (static_cast<int64_t>(pre[pl.some[mid]]) * pl.Hkv <= a) lo = mid;
        else hi = mid;
      }
      const int b0 = pl.some[lo];
      const int h0 = static_cast<int>((a - static_cast<int64_t>(pre[b0]) * pl.Hkv) / (pre[b0 + 1] - pre[b0]));
      if (static_cast<int>(threadIdx.x) < max_segs) {
        const int id = h0 + threadIdx.x, k = lo + id / pl.Hkv, h = id % pl.Hkv;
        Seg sg = {0x7fffffff, 0, 0, 0};
        if (k < pl.nsome) {
          const int b = pl.some[k], nb = static_cast<int>(pre[b + 1] - pre[b]);
          const int64_t base = static_cast<int64_t>(pre[b]) * pl.Hkv + static_cast<int64_t>(h) * nb;
          if (base < r1) sg = {static_cast<int>(base - a), nb, b, h};
        }
        seg[threadIdx.x] = sg;
      }
    }
    __syncthreads();
    int nseg = max_segs, n;  // segments and blocks of the round
    while (seg[nseg - 1].nb == 0) --nseg;
    n = static_cast<int>(min(r1 - a, static_cast<int64_t>(seg[nseg - 1].base) + seg[nseg - 1].nb));
    auto run_begin = [&](int w) { return static_cast<int>(static_cast<int64_t>(n) * w / kWarps); };
    auto run_owner = [&](int x) { return static_cast<int>(((x + 1LL) * kWarps - 1) / n); };
    const int w0 = run_begin(warp), w1 = run_begin(warp + 1);

    // ---- copy side: `ahead` walks kStages blocks in front of the compute
    Walk ahead, cur;
    ahead.left = w1 - w0;
    uint32_t absent = 0;  // bit s: stage s holds no block (its page is outside the cache)
    int pend = 0;         // page entry of the block `ahead` stands at
    auto issue = [&](int s, int page) {
      const bool ok = page >= 0 && page < p.c.num_pages;
      absent = ok ? absent & ~(1u << s) : absent | (1u << s);
      if (lane == 0) {
        if (ok) {
          const int in = own_block(ahead.vis, ahead.i) & ((1 << p.c.bpp_shift) - 1);
          const uint8_t* src = p.c.pages + ((((static_cast<int64_t>(page) * p.c.Hkv + ahead.h) << p.c.bpp_shift) + in) * kBlkBytes);
          block_g2s(ring + s * kBlkBytes, src, &bars[warp][s]);
        } else if (p.c.status) {
          atomicOr(p.c.status, KV1B_STATUS_BAD_INDEX);
        }
      }
      ahead.step(seg, pl, p);
    };
    if (ahead.left > 0) {
      int k = 0;  // the segment of block w0
      for (int x = lane; x < nseg; x += 32)
        if (seg[x].base <= w0) k = x;
      k = __reduce_max_sync(kFull, k);
      ahead.s = k;
      ahead.i = w0 - seg[k].base;
      ahead.enter(seg, pl, p);
      cur = ahead;
      for (int s = 0; s < kStages && ahead.left > 0 && !gave_up; ++s) issue(s, page_entry(p, ahead));
      if (ahead.left > 0) pend = page_entry(p, ahead);
    } else {
      cur = Walk();
      cur.left = 0;
    }

    // ---- the round's queries
    for (int r = warp; r < nseg * G; r += kWarps) {
      const Seg sg = seg[r / G];
      const QueryPrep qp = query_prep_warp(p.q, (static_cast<int64_t>(sg.b) * p.Hq + static_cast<int64_t>(sg.h) * G + r % G) * kD,
                                           p.q_dtype, p.c.signs);
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

    float acc[8][4], lsum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    #pragma unroll
    for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
    float m = kNoRef;  // reference of head g
    // the warp's sums of a segment to a piece [head][kRow]
    auto put_piece = [&](float* w) {
      if (t == 0 && g < G) w[g * kRow] = m;
      #pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int hd = 2 * t + e;
        if (hd < G) {
          if (g == 0) w[hd * kRow + 1] = lsum[e];
          #pragma unroll
          for (int i = 0; i < 8; ++i) {
            w[hd * kRow + 2 + 16 * i + g] = acc[i][e];
            w[hd * kRow + 2 + 16 * i + g + 8] = acc[i][2 + e];
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
        if (g < G) {
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
      lsum[0] = lsum[1] = lsum[2] = lsum[3] = 0.0f;
      m = kNoRef;
      const bool starts = cur.i == 0;
      const int count = min(cur.left, cur.nb - cur.i);  // blocks of the segment in the warp's run
      const bool ends = cur.i + count == cur.nb;
      const int len = pl.len[cur.b];
      const int wstart = (p.window > 0 && len > p.window) ? len - p.window : 0;

      for (int e = 0; e < count; ++e) {
        const uint32_t st = ring + stage * kBlkBytes;
        if (!((absent >> stage) & 1u)) {
          if (!__all_sync(kFull, mbar_wait(&bars[warp][stage], (phases >> stage) & 1u, gave_up ? 1 : kWaitTries)))
            gave_up = true;  // every lane alike
          phases ^= 1u << stage;
          // which of the block's tokens the query sees
          const int tok0 = own_block(cur.vis, cur.i + e) * kBlkTok;
          const bool edge = tok0 + kBlkTok > len || (tok0 < wstart && tok0 + kBlkTok > p.sinks);
          uint32_t seen = 0xFFFFFFFFu;
          if (edge) {
            // unseen tokens: what their places hold (another sequence's remains, infinities) must not
            // reach a product, so their scale, min and norm become zeros and their weights are zero
            const int tk = tok0 + lane;
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
            }
            __syncwarp();
          }
          // ---- scores
          float x[8];
          {
            uint32_t kw[4];
            ldsm_x4(kw, st + lane * 16);
            int d[4][4];
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
              // the sums start at the bits of 1.5 2^23: as a float, an entry is that plus its integer
              d[i][0] = d[i][1] = d[i][2] = d[i][3] = 0x4B400000;
              const uint32_t w[2] = {kw[i], kw[i] >> 4};
              #pragma unroll
              for (int kb = 0; kb < 4; ++kb) {
                const int pl0 = 2 * (kb & 1);
                const uint32_t lo = 0x01010101u << pl0, hi = lo << 1;
                imma(d[i], aq[kb][0], 0x01010101u << (3 - pl0), aq[kb][1], 0x01010101u << (2 - pl0), w[kb >> 1] & lo, w[kb >> 1] & hi);
              }
            }
            uint32_t ncr[8];
            lds128(ncr, st + kBlkOffNc + 32 * t);
            lds128(ncr + 4, st + kBlkOffNc + 32 * t + 16);
            #pragma unroll
            for (int i = 0; i < 4; ++i)
              #pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float a8 = __fadd_rn(__int_as_float(d[i][e]), -12582912.0f);
                const float b8 = __fadd_rn(__int_as_float(d[i][2 + e]), -12582912.0f);
                const float dot = __fmaf_rn(c1, a8, __fmaf_rn(c2, b8, c0));
                x[2 * i + e] = __fmul_rn(dot, __uint_as_float(ncr[2 * i + e]));
              }
          }
          if (edge) {
            const uint32_t mine = seen >> (8 * t);
            #pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = (mine >> j) & 1u ? x[j] : -INFINITY;
          }
          float mx = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
          if (__any_sync(kFull, mx > m + kTau)) {  // rare: raise references
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
            const bool up = mx > m + kTau;
            const float alpha = up ? ex2(m - mx) : 1.0f;  // 0 from kNoRef
            m = up ? mx : m;
            const float a0 = __shfl_sync(kFull, alpha, 8 * t), a1 = __shfl_sync(kFull, alpha, 8 * t + 4);
            #pragma unroll
            for (int i = 0; i < 8; ++i) {
              acc[i][0] = __fmul_rn(acc[i][0], a0);
              acc[i][1] = __fmul_rn(acc[i][1], a1);
              acc[i][2] = __fmul_rn(acc[i][2], a0);
              acc[i][3] = __fmul_rn(acc[i][3], a1);
            }
            lsum[0] = __fmul_rn(lsum[0], a0);
            lsum[1] = __fmul_rn(lsum[1], a1);
            lsum[2] = __fmul_rn(lsum[2], a0);
            lsum[3] = __fmul_rn(lsum[3], a1);
          }
          const float mb = m - kBase;
          uint32_t pw[4];
          #pragma unroll
          for (int i = 0; i < 4; ++i) pw[i] = pack_f16(ex2(x[2 * i] - mb), ex2(x[2 * i + 1] - mb));
          hmma(lsum, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, pw[0], pw[1]);
          hmma(lsum, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, pw[2], pw[3]);
          // ---- P.V, value group by value group (32 channels: rows of two products)
          #pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t sc[4], mn[4], cw[4];
            lds128(sc, st + kBlkOffScale + q * 64 + 16 * t);
            lds128(mn, st + kBlkOffMin + q * 64 + 16 * t);
            ldsm_x4(cw, st + kBlkOffCodes + (32 * q + lane) * 16);  // rows g, g + 8, g + 16, g + 24; word t
            #pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t lo[4], hi[4];
              expand_codes(cw[2 * u], lo);
              expand_codes(cw[2 * u + 1], hi);
              #pragma unroll
              for (int i = 0; i < 4; ++i) {
                lo[i] = hfma2(lo[i], sc[i], mn[i]);
                hi[i] = hfma2(hi[i], sc[i], mn[i]);
              }
              hmma(acc[2 * q + u], lo[0], hi[0], lo[1], hi[1], pw[0], pw[1]);
              hmma(acc[2 * q + u], lo[2], hi[2], lo[3], hi[3], pw[2], pw[3]);
            }
          }
          if (edge) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // own writes before the next copy
        }
        __syncwarp();
        // ---- the stage's next block
        if (ahead.left > 0 && !gave_up) {
          issue(stage, pend);
          if (ahead.left > 0) pend = page_entry(p, ahead);
        } else if (gave_up) {
          absent |= 1u << stage;
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
      }
      cur.left -= count;

      if (starts && ends) {  // all of it: finished here
        const int64_t qrow = static_cast<int64_t>(cur.b) * p.Hq + static_cast<int64_t>(cur.h) * G;
        if (p.rows) {
          put_piece(p.rows + qrow * kRow);
        } else {
          #pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int hd = 2 * t + e;
            if (hd < G) {
              const float den = lsum[e];
              #pragma unroll
              for (int i = 0; i < 8; ++i) {
                store_out(p.out, p.q_dtype, (qrow + hd) * kD + 16 * i + g, den != 0.0f ? __fdiv_rn(acc[i][e], den) : 0.0f);
                store_out(p.out, p.q_dtype, (qrow + hd) * kD + 16 * i + g + 8, den != 0.0f ? __fdiv_rn(acc[i][2 + e], den) : 0.0f);
              }
            }
          }
        }
      } else if (cur.left > 0) {  // its end: the run goes on with another segment
        put_piece(first);
      } else {
        last = true;
      }
      if (cur.left > 0) {
        ++cur.s;
        cur.i = 0;
        cur.enter(seg, pl, p);
      }
    }

    // ---- the warps' pieces meet: of segment x, warps wf .. wl have one each, in `red` or (an end inside the
    // warp's run) in `first`
    __syncthreads();  // the ring is drained, the pieces in `first` are written
    if (last) put_piece(red + warp * G * kRow);
    __syncthreads();
    for (int x = 0; x < nseg; ++x) {
      const Seg sg = seg[x];
      const int s = max(sg.base, 0), e = min(sg.base + sg.nb, n);
      const int wf = run_owner(s), wl = run_owner(e - 1);
      const bool starts = sg.base >= 0, ends = sg.base + sg.nb <= n;
      if (wf == wl && starts && ends) continue;  // finished by its warp
      const float* tail = e < run_begin(wl + 1) ? p.first + (static_cast<int64_t>(blockIdx.x) * kWarps + wl) * G * kRow : red + wl * G * kRow;
      const int64_t qrow = static_cast<int64_t>(sg.b) * p.Hq + static_cast<int64_t>(sg.h) * G;
      for (int i = threadIdx.x; i < G * kD; i += kThreads) {
        const int hd = i / kD, ch = i - hd * kD;
        auto piece = [&](int w) { return (w == wl ? tail : red + w * G * kRow) + hd * kRow; };
        float M = kNoRef;
        for (int w = wf; w <= wl; ++w) M = fmaxf(M, piece(w)[0]);
        float num = 0.0f, den = 0.0f;
        #pragma unroll 4
        for (int w = wf; w <= wl; ++w) {
          const float* r = piece(w);
          const float f = ex2(r[0] - M);
          num = __fmaf_rn(f, r[2 + ch], num);
          den = __fmaf_rn(f, r[1], den);
        }
        if (starts && ends && !p.rows) {
          store_out(p.out, p.q_dtype, (qrow + hd) * kD + ch, den != 0.0f ? __fdiv_rn(num, den) : 0.0f);
        } else {
          float* row = starts && ends ? p.rows + (qrow + hd) * kRow
                                      : p.part + ((static_cast<int64_t>(blockIdx.x) * 2 + (starts ? 1 : 0)) * G + hd) * kRow;
          if (ch == 0) {
            row[0] = M;
            row[1] = den;
          }
          row[2 + ch] = num;
        }
      }
    }
    a += n;
    if (a < r1) {  // the next round's copies land where the pieces were
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncthreads();
    }
  }
  if (gave_up && lane == 0 && p.c.status) atomicOr(p.c.status, KV1B_STATUS_TIMEOUT);
}

// Segments cut by a range boundary: block (c, head) merges the one that starts in CTA c's range and goes
// on past it -- slot 1 of c, then slot 0 of the CTAs after it.
__global__ void __launch_bounds__(128) paged_merge_kernel(const PagedAttendParams p, const int G) {
  __shared__ uint32_t pre[kMaxSeqs + 1];
  __shared__ int slen[kMaxSeqs];
  pdl_wait();
  const Plan pl = make_plan<128>(p, pre, slen, nullptr, p.ncta, false);
  const int c = blockIdx.x, hd = blockIdx.y;
  if (c + 1 >= pl.n || pl.S == 0) return;
  const int64_t r0 = pl.begin(c), r1 = pl.begin(c + 1);
  if (r0 >= r1) return;
  int b, h;
  int64_t base;
  pl.locate(r1 - 1, &b, &h, &base);
  const int64_t end = base + (pre[b + 1] - pre[b]);
  if (base < r0 || end <= r1) return;
  int last = c + 1;
  while (last + 1 < pl.n && pl.begin(last + 1) < end) ++last;
  const int n = last - c + 1;  // pieces
  const int64_t step = 2LL * G * kRow;
  const float* first = p.part + ((static_cast<int64_t>(c) * 2 + 1) * G + hd) * kRow;
  const float* rest = p.part + ((static_cast<int64_t>(c) * 2) * G + hd) * kRow;
  auto piece = [&](int i) { return i == 0 ? first : rest + i * step; };
  float M = kNoRef;
  for (int i = 0; i < n; ++i) M = fmaxf(M, piece(i)[0]);
  float num = 0.0f, den = 0.0f;
  #pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float* r = piece(i);
    const float f = ex2(r[0] - M);
    num = __fmaf_rn(f, r[2 + threadIdx.x], num);
    den = __fmaf_rn(f, r[1], den);
  }
  const int64_t row = static_cast<int64_t>(b) * p.Hq + static_cast<int64_t>(h) * G + hd;
  store_out(p.out, p.q_dtype, row * kD + threadIdx.x, den != 0.0f ? __fdiv_rn(num, den) : 0.0f);
}

}  // namespace paged
}  // namespace kv1b

using namespace kv1b;

cudaError_t kv1b_launch_paged_attend(const PagedAttendParams& p, int32_t G, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = configure_smem(reinterpret_cast<const void*>(paged::paged_attend_kernel),
                                 paged::kSmem, &configured);
  if (e != cudaSuccess) return e;
  e = launch_pdl(paged::paged_attend_kernel, dim3(p.ncta), dim3(paged::kThreads), paged::kSmem, stream, p, G);
  if (e != cudaSuccess || p.ncta < 2 || p.rows) return e;
  return launch_pdl(paged::paged_merge_kernel, dim3(p.ncta - 1, G), dim3(128), 0, stream, p, G);
}

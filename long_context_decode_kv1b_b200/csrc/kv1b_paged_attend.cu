// kv1b_paged_attend.cu -- decode attention over a paged cache, one query token per sequence, uneven
// lengths read on the device.
//
// Split.  The visible 32-token blocks of all (sequence, kv-head) segments are laid end to end and cut
// into one equal contiguous range per CTA (one CTA per SM), whatever the lengths.  Each of a CTA's 16
// warps takes every 16th block of the range's current segment and streams its blocks through its own
// ring of kStages shared-memory buffers (one 3,200-byte bulk copy per block, an mbarrier each), so the
// main loop has no barrier between warps.  At a segment's end the warps' sums meet in shared memory; a
// segment that a range boundary cuts leaves a partial row per CTA, which a second kernel merges.
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

constexpr int kOffPre = kWarps * kStages * kBlkBytes;            // u32 [kMaxSeqs + 1] blocks before each sequence
constexpr int kOffLen = kOffPre + (kMaxSeqs + 4) * 4;            // i32 [kMaxSeqs]
constexpr int kOffRed = kOffLen + kMaxSeqs * 4;                  // f32 [kWarps][G][kRow]
constexpr int smem_bytes(int G) { return kOffRed + kWarps * G * kRow * 4; }
static_assert(kOffPre % 16 == 0 && kOffRed % 16 == 0, "alignment");
static_assert(smem_bytes(KV1B_MAX_GROUP) + 2048 <= 227 * 1024, "shared memory");

// A walk over one warp's blocks of the CTA's range [r0, r1).
struct Walk {
  int b, h, i, iend, nb;  // segment, next block, end within the range, blocks of the segment
  int64_t rnext, r1;      // first block after the segment's part
  Visible vis;
  __device__ __forceinline__ void segment(const Plan& pl, const PagedAttendParams& p, int64_t r, int first) {
    int64_t base;
    pl.locate(r, &b, &h, &base);
    vis = visible(pl.len[b], p.window, p.sinks);
    nb = vis.blocks;
    const int64_t e = base + nb;
    rnext = e < r1 ? e : r1;
    i = static_cast<int>(r - base) + first;
    iend = static_cast<int>(rnext - base);
  }
  __device__ __forceinline__ bool next_segment(const Plan& pl, const PagedAttendParams& p, int first) {
    if (rnext >= r1) return false;
    segment(pl, p, rnext, first);
    return true;
  }
};

// Block i of a segment: its place in the sequence, and its page's entry.
__device__ __forceinline__ int own_block(const Visible& v, int j) { return j < v.skip_from ? j : j + (v.skip_to - v.skip_from); }

template <typename W>
__device__ __forceinline__ int page_entry(const PagedAttendParams& p, const W& w) {
  const int blk = own_block(w.vis, w.i);
  return __ldg(p.table + w.b * p.table_stride + (blk >> p.c.bpp_shift));
}

__global__ void __launch_bounds__(kThreads, 1) paged_attend_kernel(const PagedAttendParams p, const int G) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kWarps][kStages];
  __shared__ __align__(16) uint4 s_planes[KV1B_MAX_GROUP][4];
  __shared__ float s_vl[KV1B_MAX_GROUP], s_dl[KV1B_MAX_GROUP];
  __shared__ int s_sq[KV1B_MAX_GROUP];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint32_t* pre = reinterpret_cast<uint32_t*>(smem + kOffPre);
  int* slen = reinterpret_cast<int*>(smem + kOffLen);
  float* red = reinterpret_cast<float*>(smem + kOffRed);

  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&bars[warp][s], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  pdl_launch_dependents();
  const Plan pl = make_plan<kThreads>(p, pre, slen, gridDim.x, blockIdx.x == 0);

  // sequences that see nothing: zeros
  for (int b = p.rows ? p.B : blockIdx.x; b < p.B; b += gridDim.x)
    if (pre[b + 1] == pre[b])
      for (int e = threadIdx.x; e < p.Hq * kD; e += kThreads) store_out(p.out, p.q_dtype, static_cast<int64_t>(b) * p.Hq * kD + e, 0.0f);
  if (static_cast<int>(blockIdx.x) >= pl.n || pl.S == 0) return;

  const int64_t r0 = pl.begin(blockIdx.x), r1 = pl.begin(blockIdx.x + 1);
  if (r0 >= r1) return;
  const uint32_t ring = smem_u32(smem) + warp * kStages * kBlkBytes;

  // ---- copy side: `ahead` walks kStages blocks in front of the compute
  Walk ahead;
  ahead.r1 = r1;
  ahead.segment(pl, p, r0, warp);
  auto settle = [&](Walk& w) {  // to the warp's next block; false at the end
    while (w.i >= w.iend)
      if (!w.next_segment(pl, p, warp)) return false;
    return true;
  };
  uint32_t absent = 0;  // bit s: stage s holds no block (its page is outside the cache)
  auto issue = [&](int s, int page) {
    const bool ok = page >= 0 && page < p.c.num_pages;
    const int blk = own_block(ahead.vis, ahead.i);
    absent = ok ? absent & ~(1u << s) : absent | (1u << s);
    if (lane == 0) {
      if (ok) {
        const int in = blk & ((1 << p.c.bpp_shift) - 1);
        const uint8_t* src = p.c.pages + ((((static_cast<int64_t>(page) * p.c.Hkv + ahead.h) << p.c.bpp_shift) + in) * kBlkBytes);
        block_g2s(ring + s * kBlkBytes, src, &bars[warp][s]);
      } else if (p.c.status) {
        atomicOr(p.c.status, KV1B_STATUS_BAD_INDEX);
      }
    }
    ahead.i += kWarps;
  };
  bool more = true;
  int pend = 0;  // page entry of the block `ahead` stands at
  {
    // the first kStages entries
    for (int s = 0; s < kStages && more; ++s) {
      more = settle(ahead);
      if (more) issue(s, page_entry(p, ahead));
    }
    if (more) more = settle(ahead);
    if (more) pend = page_entry(p, ahead);
  }

  Walk cur;
  cur.r1 = r1;
  cur.segment(pl, p, r0, warp);
  int stage = 0;
  uint32_t phases = 0;  // bit s: parity of stage s's next completion
  bool gave_up = false;

  for (;;) {
    // ---- queries of the segment
    const int64_t qrow = static_cast<int64_t>(cur.b) * p.Hq + static_cast<int64_t>(cur.h) * G;
    if (warp < G) {
      const QueryPrep qp = query_prep_warp(p.q, (qrow + warp) * kD, p.q_dtype, p.c.signs);
      if (lane == 0) {
        #pragma unroll
        for (int j = 0; j < 4; ++j) s_planes[warp][j] = make_uint4(qp.planes[j][0], qp.planes[j][1], qp.planes[j][2], qp.planes[j][3]);
        s_vl[warp] = qp.vl;
        s_dl[warp] = qp.delta;
        s_sq[warp] = qp.sq;
      }
    }
    __syncthreads();
    // A operand: k-row 4 t + j of product kb, half hi is channel 32 t + 8 j + r, r = 2 kb + hi, its code
    // times 2^(3 - (r & 3)) (the sign bit stays at place r & 3 of its byte)
    uint32_t aq[4][2];
    {
      uint32_t pw[4] = {0u, 0u, 0u, 0u};
      if (g < G) {
        #pragma unroll
        for (int j = 0; j < 4; ++j) pw[j] = reinterpret_cast<const uint32_t*>(&s_planes[g][j])[t];
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
    // log2 logit = (c1 8A + c2 8Bc + c0) (N/C):  delta (2A - Sq) + vl (2 Bc - 128), times scale log2(e) / 128
    const float qs = __fmul_rn(__fmul_rn(p.scale, 1.4426950408889634f), 1.0f / kD);
    const float dl = g < G ? s_dl[g] : 0.0f, vl = g < G ? s_vl[g] : 0.0f;
    const float sq = g < G ? static_cast<float>(s_sq[g]) : 0.0f;
    const float c1 = __fmul_rn(0.25f * dl, qs), c2 = __fmul_rn(0.25f * vl, qs);
    const float c0 = -__fmul_rn(__fadd_rn(__fmul_rn(dl, sq), 128.0f * vl), qs);

    float acc[8][4], lsum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    #pragma unroll
    for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
    float m = kNoRef;  // reference of head g

    for (; cur.i < cur.iend; cur.i += kWarps) {
      const uint32_t st = ring + stage * kBlkBytes;
      const bool here = !((absent >> stage) & 1u);
      bool edge = false;
      if (here) {
        if (!__all_sync(kFull, mbar_wait(&bars[warp][stage], (phases >> stage) & 1u, gave_up ? 1 : kWaitTries)))
          gave_up = true;  // every lane alike
        phases ^= 1u << stage;
        // which of the block's tokens the query sees
        const int tok0 = own_block(cur.vis, cur.i) * kBlkTok;
        const int len = pl.len[cur.b];
        const int wstart = (p.window > 0 && len > p.window) ? len - p.window : 0;
        edge = tok0 + kBlkTok > len || (tok0 < wstart && tok0 + kBlkTok > p.sinks);
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
      if (more && !gave_up) {
        issue(stage, pend);
        more = settle(ahead);
        if (more) pend = page_entry(p, ahead);
      } else if (gave_up) {
        absent |= 1u << stage;
      }
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }

    // ---- the warps' sums meet: red[warp][head] = m, l, o[128]
    {
      float* w0 = red + warp * G * kRow;
      if (t == 0 && g < G) w0[g * kRow] = m;
      #pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int hd = 2 * t + e;
        if (hd < G) {
          if (g == 0) w0[hd * kRow + 1] = lsum[e];
          #pragma unroll
          for (int i = 0; i < 8; ++i) {
            w0[hd * kRow + 2 + 16 * i + g] = acc[i][e];
            w0[hd * kRow + 2 + 16 * i + g + 8] = acc[i][2 + e];
          }
        }
      }
    }
    __syncthreads();
    {
      int64_t base;
      int b, h;
      const int64_t rfirst = cur.rnext - 1;
      pl.locate(rfirst, &b, &h, &base);
      const bool starts = base >= r0, ends = base + cur.nb <= r1;
      for (int e = threadIdx.x; e < G * kD; e += kThreads) {
        const int hd = e / kD, ch = e - hd * kD;
        float M = kNoRef;
        #pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red[(w * G + hd) * kRow]);
        float num = 0.0f, den = 0.0f;
        #pragma unroll 4
        for (int w = 0; w < kWarps; ++w) {
          const float* r = red + (w * G + hd) * kRow;
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
    if (cur.rnext >= r1) break;
    cur.next_segment(pl, p, warp);
    __syncthreads();  // red and the planes are rewritten
  }
  if (gave_up && lane == 0 && p.c.status) atomicOr(p.c.status, KV1B_STATUS_TIMEOUT);
}

// Segments cut by a range boundary: block (c, head) merges the one that starts in CTA c's range and goes
// on past it -- slot 1 of c, then slot 0 of the CTAs after it.
__global__ void __launch_bounds__(128) paged_merge_kernel(const PagedAttendParams p, const int G) {
  __shared__ uint32_t pre[kMaxSeqs + 1];
  __shared__ int slen[kMaxSeqs];
  pdl_wait();
  const Plan pl = make_plan<128>(p, pre, slen, p.ncta, false);
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
                                 paged::smem_bytes(KV1B_MAX_GROUP), &configured);
  if (e != cudaSuccess) return e;
  e = launch_pdl(paged::paged_attend_kernel, dim3(p.ncta), dim3(paged::kThreads), paged::smem_bytes(G), stream, p, G);
  if (e != cudaSuccess || p.ncta < 2 || p.rows) return e;
  return launch_pdl(paged::paged_merge_kernel, dim3(p.ncta - 1, G), dim3(128), 0, stream, p, G);
}

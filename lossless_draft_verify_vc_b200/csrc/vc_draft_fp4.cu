// vc_draft_fp4.cu -- single-token draft attention over the 4-bit
// floating-point cache (vc_fp4.cuh), with an optional sliding window and
// first tokens that stay visible.
//
// Drafting decodes one token per step from the compressed cache in HBM
// ("VeriCache: Turning Lossy KV Cache into Lossless LLM Inference",
// menfem.com, "Key Contributions"); the pages give no kernel.
//
// Arithmetic, per (request, KV head) and record of 16 tokens, on mma.sync
// m16n8k16 (fp16 x fp16 -> fp32); the query rows of a GQA group (at most 8)
// are far too few for a tcgen05 tile, and the call is bound by HBM:
//   scores  S[token][head] = K_hat[token][chan] x q[chan][head]
//   values  O[chan][head] += V_hat^T[chan][token] x P[token][head]
// A code times its scale (2 + 4 significant bits, between 2^-10 and 2688) is
// exact in fp16, and so is a query row once it is scaled by a power of two
// that brings its largest element to 2^14 .. 2^15 (bf16 has 8 significant
// bits).  P is split into an fp16 high and an fp16 low part (22 significant
// bits): with at most 4 query heads they are two columns of one tile (heads
// 0..3 | 0..3, the score tile computes both copies), else two products into
// the same accumulators.  A column's reference m is an integer (in log2
// units) about 11 below its running maximum and P = 2^(s - m), so that small
// weights keep their bits in fp16 (P <= 2^15) and every rescale and merge
// weight is a power of two; m moves only when a score exceeds it by more
// than 15.
// Contractions may take their terms in any order, so a lane reads its codes
// as contiguous runs of a record (the record layout of include/vc.h).
//
// The split of the work, its merges and their reasons are in vc_stream.cuh;
// every warp reads its stages through its own ring of bulk copies, which runs
// ahead across units.  Bound by HBM: 8 x 32K tokens (302 MB) take 59 us, of
// which the stage loops run at 6.2 TB/s and starting, merging and uneven ends
// take 10 us; below that instruction issue is next (about 285 instructions a
// record, 64 of them e2m1 conversions and 64 scalings).
#include <algorithm>

#include "vc_fp4.cuh"
#include "vc_stream.cuh"

namespace vc {
namespace {

using stream::Span;

constexpr float kFBelow = 11.f;  // m is set this far below the largest score
constexpr float kFMost = 15.f;   // a score this far above m moves it: P <= 2^15

struct FArgs {
  stream::Args s;
  const uint8_t* records;
  const __nv_bfloat16* q;
  const int32_t* k_exp;
  float scale_log2;
  // failure-path test only (vc_debug_draft_fp4_abort): the warp of every block
  // whose first stage never counts as landed (-1: none), and the limit of the
  // stages' waits
  int stuck_warp;
  uint64_t wait_ns;
};

// mma_f16 into zeros
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// (a & m) | (b & ~m)
__device__ __forceinline__ uint32_t blend(uint32_t a, uint32_t b, uint32_t m) { return (a & m) | (b & ~m); }

// One half of an f16x2 in both, and a product with it: as intrinsics, which
// the compiler folds into the multiplication's operand.
template <int HIGH>
__device__ __forceinline__ __half2 both(uint32_t p) {
  const __half2 v = *reinterpret_cast<__half2*>(&p);
  return HIGH ? __high2half2(v) : __low2half2(v);
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, __half2 b) {
  const __half2 v = __hmul2(*reinterpret_cast<__half2*>(&a), b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <int D_, bool HALF>
struct FTile {
  static constexpr int D = D_;
  static constexpr int REC = fp4::Rec<D>::BYTES;
  static constexpr int NR = 256 / D;      // records per stage: 32 (D = 128) or 64 tokens
  static constexpr int STAGE = NR * REC;  // 4608 bytes
  static constexpr int NST = 2;           // ring depth of a warp (3 were slower: 68.6 against 67.0 us at 8 x 32K)
  static constexpr int RING = NST * STAGE;
  static constexpr int BAR_OFF = stream::kWarps * RING;
  static constexpr int STATE_OFF = BAR_OFF + (stream::kWarps * NST * 8 + 15) / 16 * 16;
  static constexpr int COLS = HALF ? 4 : 8;
  static constexpr int SMEM_B = STATE_OFF + stream::kWarps * stream::State<D>::bytes(COLS);
  static_assert(2 * stream::kMergeB <= BAR_OFF, "the final merges' buffers take the rings' place");
  // A unit's begin -- query load, state, partial -- costs a block about as much
  // as 32 stages; counted as nothing the blocks that hold parts of two units
  // finish last.  Measured on B200, us of device time per call at 8 requests x
  // 32K and 1 x 262K: 8 stages 62.5, 62.4; 24 59.7, 58.1; 32 59.2, 57.7; 40
  // 58.9, 57.7 (but one unit of 65K 19.6 against 18.4).  D = 64 takes the same
  // numbers: its stages have the same bytes and products.
  static constexpr int PAD = 32;
  static constexpr int MIN = 48;  // padding and a short unit (16 stages)
  static constexpr int GAIN = 40;  // see stream::choose
  static constexpr int KT = D / 16;  // k-steps of a score tile, m-tiles of the values
  using R = fp4::Rec<D>;

  const FArgs& a;
  const int warp, lane, row, i4;
  unsigned char* ring;
  uint64_t* bars;
  // the next copy: stage is of unit (ib, ih), at isrc if it is below ifast
  // (stages of NR records, one after the other)
  int ib, ih, istart, is, ifast, islot, share;
  const uint8_t* isrc;
  uint64_t policy;
  int slot;
  uint32_t phase;  // parity of the slot's next completion
  uint32_t qf[2 * KT];
  float kup, sc0, sc1, m0, m1, l0, l1;
  float acc[KT][4];

  __device__ __forceinline__ FTile(const FArgs& a_, unsigned char* smem)
      : a(a_), warp(threadIdx.x >> 5), lane(threadIdx.x & 31), row(lane >> 2), i4(lane & 3), slot(0), phase(0) {
    ring = smem + warp * RING;
    bars = reinterpret_cast<uint64_t*>(smem + BAR_OFF) + warp * NST;
    if (lane == 0) {
      for (int i = 0; i < NST; ++i) mbar_init(&bars[i], i == 0 && warp == a.stuck_warp ? 2 : 1);
      fence_mbar_init();
      fence_proxy_async_smem();
    }
    __syncwarp();  // the other lanes wait on them
  }

  // bf16 query words of this lane: its tile column's head, D / 4 channels from
  // i4 * D / 4 (requested before the copies, which fill the memory's queues)
  __device__ __forceinline__ void query(int b, int h) {
    const int head = HALF ? (row & 3) : row;
    const uint4* src = reinterpret_cast<const uint4*>(
        a.q + (static_cast<int64_t>(b) * a.s.Hq + h * a.s.g + head) * D + i4 * (D / 4));
#pragma unroll
    for (int x = 0; x < D / 32; ++x) {
      const uint4 v = head < a.s.g ? stream::load_16(src + x) : make_uint4(0, 0, 0, 0);
      qf[4 * x] = v.x, qf[4 * x + 1] = v.y, qf[4 * x + 2] = v.z, qf[4 * x + 3] = v.w;
    }
    kup = two_to(a.k_exp, h, 1);
  }

  __device__ __forceinline__ void begin(int b, int h, int start, int share_) {
    ib = b, ih = h, istart = start, share = share_;
    is = max(0, -start) + warp;
    ifast = islot = 0;
    isrc = nullptr;
    policy = l2_evict_first();  // the records are read once per call
#pragma unroll 1
    for (int i = 0; i < NST; ++i) issue_next();
  }

  // The warp's next stage with records into the next slot.
  __device__ __forceinline__ void issue_next() {
    uint32_t bytes = STAGE;
    if (is >= ifast) {  // look for it
      for (;;) {
        if (istart >= share) return;
        const Span ip = stream::request_span<NR>(a.s, ib);
        const int end = min(ip.n, share - istart);
        if (is < end) {
          const int n = stream::stage_records<NR>(ip, is);
          if (n > 0) {
            bytes = static_cast<uint32_t>(n) * REC;
            isrc = a.records + ((static_cast<int64_t>(ib) * a.s.Hkv + ih) * (a.s.T_cap / fp4::kTok) +
                                stream::stage_record<NR>(ip, is)) * REC;
            ifast = is < ip.ns ? 0 : min(end, ip.ns + (ip.r1 - ip.r0) / NR);
            break;
          }
          is += stream::kWarps;
        } else {
          istart += ip.n + PAD;
          is = warp;
          ifast = 0;
          if (++ih == a.s.Hkv) ih = 0, ++ib;
        }
      }
    }
    if (lane == 0) {
      mbar_arrive_expect_tx(&bars[islot], bytes);
      bulk_g2s_hint(ring + islot * STAGE, isrc, bytes, &bars[islot], policy);
    }
    islot = islot + 1 == NST ? 0 : islot + 1;
    is += stream::kWarps;
    isrc += stream::kWarps * STAGE;
  }

  // Query fragments: lane's head = its tile column, channels 4 s .. of each k-step s.
  __device__ __forceinline__ void unit(const Span&, int, int, int, int) {
    float big = 0.f;
#pragma unroll
    for (int x = 0; x < D / 8; ++x) {
      const float2 f = unpack_bf2(qf[x]);
      big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
    // a row of zeros (and a column without a head) keeps the factor 1
    const int e = big > 0.f ? max(-100, (__float_as_int(big) >> 23) - 127) - 14 : 0;
    const float up = __int_as_float((127 - e) << 23);
#pragma unroll
    for (int x = 0; x < D / 8; ++x) {
      const float2 f = unpack_bf2(qf[x]);
      qf[x] = pack_h2(f.x * up, f.y * up);
    }
    // floor: -inf (a masked score) times the factor stays -inf
    const float sc = fmaxf(a.scale_log2 * kup * __int_as_float((127 + e) << 23), 1e-37f);
    sc0 = __shfl_sync(0xffffffffu, sc, 8 * i4);
    sc1 = __shfl_sync(0xffffffffu, sc, 8 * i4 + 4);
#pragma unroll
    for (int x = 0; x < KT; ++x) acc[x][0] = acc[x][1] = acc[x][2] = acc[x][3] = 0.f;
    m0 = m1 = stream::kNone;
    l0 = l1 = 0.f;
  }

  __device__ __forceinline__ bool stage(const Span& p, int x, int) {
    const bool full = x >= p.f0 && x < p.f1;
    if (!__all_sync(0xffffffffu, mbar_try_wait_hint(&bars[slot], phase, 20000u)) &&
        __any_sync(0xffffffffu, !mbar_wait_bounded(&bars[slot], phase, a.s.flags, a.wait_ns)))
      return false;
    const unsigned char* st = ring + slot * STAGE;
    if (++slot == NST) slot = 0, phase ^= 1;
    // two copies of the body: the masks cost the whole stages nothing (9 of 298 instructions a record)
    if (full)
      body<true>(p, x, st);
    else
      body<false>(p, x, st);
    __syncwarp();
    issue_next();
    return true;
  }

  template <bool full>
  __device__ __forceinline__ void body(const Span& p, int x, const unsigned char* st) {
    // hi lanes keep a weight's first 11 bits, lo lanes the rest: v = p * lo_f + ((p & mask) ^ lo_s)
    const float lo_f = i4 < 2 ? 0.f : 1.f;
    const uint32_t lo_s = i4 < 2 ? 0u : 0x80000000u;
    // ---- scores
    float c[NR][4];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const unsigned char* rec = st + r * REC;
      uint32_t ka[D / 32], kb[D / 32];
      __half2 sa[D / 64], sb[D / 64];  // token row, row + 8: codes, scales (both halves)
      if constexpr (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(rec + lane * 16);
        const uint4 y = *reinterpret_cast<const uint4*>(rec + 512 + lane * 16);
        ka[0] = x.x, ka[1] = x.y, ka[2] = x.z, ka[3] = x.w;
        kb[0] = y.x, kb[1] = y.y, kb[2] = y.z, kb[3] = y.w;
        const uint32_t w = *reinterpret_cast<const uint32_t*>(rec + R::KS + lane * 4);
        const uint32_t p = fp4::scales_to_h2(w & 0xffffu), q = fp4::scales_to_h2(w >> 16);
        sa[0] = both<0>(p), sa[1] = both<1>(p);
        sb[0] = both<0>(q), sb[1] = both<1>(q);
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(rec + lane * 8);
        const uint2 y = *reinterpret_cast<const uint2*>(rec + 256 + lane * 8);
        ka[0] = x.x, ka[1] = x.y;
        kb[0] = y.x, kb[1] = y.y;
        const uint32_t p = fp4::scales_to_h2(*reinterpret_cast<const uint16_t*>(rec + R::KS + lane * 2));
        sa[0] = both<0>(p);
        sb[0] = both<1>(p);
      }
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        uint32_t oa[4], ob[4];
        fp4::codes_to_h2(ka[w], oa);
        fp4::codes_to_h2(kb[w], ob);
#pragma unroll
        for (int x = 0; x < 4; ++x) oa[x] = mul_h2(oa[x], sa[w / 2]), ob[x] = mul_h2(ob[x], sb[w / 2]);
        const uint32_t f0[4] = {oa[0], ob[0], oa[1], ob[1]}, f1[4] = {oa[2], ob[2], oa[3], ob[3]};
        if (w == 0)
          mma_f16_zero(c[r], f0, qf[0], qf[1]);
        else
          mma_f16(c[r], f0, qf[4 * w], qf[4 * w + 1]);
        mma_f16(c[r], f1, qf[4 * w + 2], qf[4 * w + 3]);
      }
    }
    uint32_t t0 = 0;
    int nrec = NR;
    if (!full) {
      t0 = static_cast<uint32_t>(stream::stage_record<NR>(p, x)) * fp4::kTok;
      nrec = stream::stage_records<NR>(p, x);
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const uint32_t t = t0 + r * fp4::kTok + row;
        if (r >= nrec || !stream::seen(a.s, p, t)) c[r][0] = c[r][1] = -INFINITY;
        if (r >= nrec || !stream::seen(a.s, p, t + 8)) c[r][2] = c[r][3] = -INFINITY;
      }
    }

    // ---- online softmax
    float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      x0 = fmaxf(x0, fmaxf(c[r][0], c[r][2]));
      x1 = fmaxf(x1, fmaxf(c[r][1], c[r][3]));
    }
    x0 *= sc0;
    x1 *= sc1;
    if (__any_sync(0xffffffffu, x0 - m0 > kFMost || x1 - m1 > kFMost)) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        x0 = warp_max_xor(x0, d);
        x1 = warp_max_xor(x1, d);
      }
      x0 = ceilf(x0), x1 = ceilf(x1);
      // (past 2^22 the subtraction would round: m = the maximum itself)
      const float n0 = fmaxf(m0, fabsf(x0) < 4194304.f ? x0 - kFBelow : x0);
      const float n1 = fmaxf(m1, fabsf(x1) < 4194304.f ? x1 - kFBelow : x1);
      const float al0 = ex2(m0 - n0), al1 = ex2(m1 - n1);
      m0 = n0, m1 = n1;
      l0 *= al0, l1 *= al1;
#pragma unroll
      for (int x = 0; x < KT; ++x) acc[x][0] *= al0, acc[x][2] *= al0, acc[x][1] *= al1, acc[x][3] *= al1;
    }

    // ---- values
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      uint32_t bh[2], bl[2];  // P of tokens 2 i4 (+ 1) and 8 more, column = row of the lane
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float p0 = ex2(fmaf(c[r][2 * x], sc0, -m0)), p1 = ex2(fmaf(c[r][2 * x + 1], sc1, -m1));
        l0 += p0;
        l1 += p1;
        const uint32_t h0 = __float_as_uint(p0) & 0xffffe000u, h1 = __float_as_uint(p1) & 0xffffe000u;
        if constexpr (HALF) {
          bh[x] = stream::movm_t(pack_h2(fmaf(p0, lo_f, __uint_as_float(h0 ^ lo_s)), fmaf(p1, lo_f, __uint_as_float(h1 ^ lo_s))));
        } else {
          bh[x] = stream::movm_t(pack_h2(__uint_as_float(h0), __uint_as_float(h1)));
          bl[x] = stream::movm_t(pack_h2(p0 - __uint_as_float(h0), p1 - __uint_as_float(h1)));
        }
      }
      const unsigned char* rec = st + r * REC;
      uint32_t u[2][D / 32];  // [half][words of the token pair]: D = 128: 2 words of each token, else 1
      uint32_t sw;            // scales of tokens 2 i4, + 1, + 8, + 9
      if constexpr (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(rec + R::V + lane * 16);
        const uint4 y = *reinterpret_cast<const uint4*>(rec + R::V + 512 + lane * 16);
        u[0][0] = x.x, u[0][1] = x.y, u[0][2] = x.z, u[0][3] = x.w;
        u[1][0] = y.x, u[1][1] = y.y, u[1][2] = y.z, u[1][3] = y.w;
        sw = *reinterpret_cast<const uint32_t*>(rec + R::VS + lane * 4);
      } else {
        const uint4 x = *reinterpret_cast<const uint4*>(rec + R::V + lane * 16);
        u[0][0] = x.x, u[0][1] = x.y, u[1][0] = x.z, u[1][1] = x.w;
        sw = *reinterpret_cast<const uint32_t*>(rec + R::VS + (lane >> 3) * 16 + i4 * 4);
      }
      if (!full) {  // a hidden token's scale may be a NaN: 0 instead
        const uint32_t t = t0 + r * fp4::kTok + 2 * i4;
        uint32_t keep = 0;
        if (r < nrec) {
          if (stream::seen(a.s, p, t)) keep |= 0xffu;
          if (stream::seen(a.s, p, t + 1)) keep |= 0xff00u;
          if (stream::seen(a.s, p, t + 8)) keep |= 0xff0000u;
          if (stream::seen(a.s, p, t + 9)) keep |= 0xff000000u;
        }
        sw &= keep;
      }
      const uint32_t sv[2] = {fp4::scales_to_h2(sw & 0xffffu), fp4::scales_to_h2(sw >> 16)};
#pragma unroll
      for (int w = 0; w < D / 64; ++w) {
        // bytes of a token's word (channel pairs) -> bytes (token, token + 1) of even and of odd channels
        uint32_t fr[2][2][4];  // [half][odd][channel pair]
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint32_t wa = u[hf][w], wb = u[hf][D / 64 + w];
          fp4::codes_to_h2(blend(wa, wb << 4, 0x0f0f0f0fu), fr[hf][0]);
          fp4::codes_to_h2(blend(wa >> 4, wb, 0x0f0f0f0fu), fr[hf][1]);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t f[4] = {hmul2(fr[0][0][x], sv[0]), hmul2(fr[0][1][x], sv[0]), hmul2(fr[1][0][x], sv[1]),
                                 hmul2(fr[1][1][x], sv[1])};
          mma_f16(acc[4 * w + x], f, bh[0], bh[1]);
          if constexpr (!HALF) mma_f16(acc[4 * w + x], f, bl[0], bl[1]);
        }
      }
    }
  }

  __device__ __forceinline__ void finish(float* o, float (*ml)[2], bool failed) {
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    if (failed || m0 == stream::kNone) m0 = -INFINITY;
    if (failed || m1 == stream::kNone) m1 = -INFINITY;
    constexpr int OS = stream::State<D>::OS;
    o += 2 * i4 * OS + row * 2;
#pragma unroll
    for (int x = 0; x < KT; ++x) {
      if constexpr (HALF) {  // high + low part
#pragma unroll
        for (int y = 0; y < 4; ++y) acc[x][y] += __shfl_xor_sync(0xffffffffu, acc[x][y], 2);
      }
      if (!HALF || i4 < 2) {
        *reinterpret_cast<float2*>(o + x * 16) = make_float2(acc[x][0], acc[x][2]);
        *reinterpret_cast<float2*>(o + OS + x * 16) = make_float2(acc[x][1], acc[x][3]);
      }
    }
    if (row == 0 && (!HALF || i4 < 2)) {
      ml[2 * i4][0] = m0, ml[2 * i4][1] = l0;
      ml[2 * i4 + 1][0] = m1, ml[2 * i4 + 1][1] = l1;
    }
  }

  __device__ __forceinline__ void drain() {
    for (int i = 0; i < NST; ++i) mbar_wait_bounded(&bars[i], i < slot ? phase ^ 1 : phase, nullptr, 100000000ull);
  }
};

template <int D, bool HALF>
__global__ void __launch_bounds__(stream::kThreads, 1) draft_fp4_kernel(FArgs a) {
  using Tile = FTile<D, HALF>;
  extern __shared__ __align__(128) unsigned char smem[];
  Tile tile(a, smem);
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  stream::run(a.s, tile, smem + Tile::STATE_OFF, smem);
}

vc_status check_draft(const vc_attn_shape* sh, const vc_fp4_cache* c, const char* who) {
  VC_REQUIRE(sh && c, "%s: null shape or cache", who);
  VC_REQUIRE(sh->B >= 1 && sh->Hkv >= 1 && sh->Hq >= 1 && sh->Hq % sh->Hkv == 0 && sh->Hq / sh->Hkv <= 8,
             "%s: need B >= 1, Hq a multiple of Hkv, Hq/Hkv <= 8", who);
  VC_REQUIRE(sh->D == 64 || sh->D == 128, "%s: head dim must be 64 or 128 (got %d)", who, sh->D);
  VC_REQUIRE(static_cast<int64_t>(sh->B) * sh->Hkv <= 65535, "%s: too many (request, head) pairs", who);
  VC_REQUIRE(c->T_cap >= fp4::kTok && c->T_cap % fp4::kTok == 0 && c->T_cap < (int64_t(1) << 31),
             "%s: T_cap must be a multiple of 16 in [16, 2^31) (got %lld)", who, static_cast<long long>(c->T_cap));
  VC_REQUIRE(c->lens || (c->T >= 0 && c->T <= c->T_cap), "%s: need 0 <= T <= T_cap", who);
  return VC_OK;
}

template <int D, bool HALF>
void launch_draft(FArgs& a, const stream::Plan& p, uint32_t L, cudaStream_t s) {
  using Tile = FTile<D, HALF>;
  static stream::Launcher<FArgs> k(draft_fp4_kernel<D, HALF>, Tile::SMEM_B);
  const int n = stream::choose(a.s, p, L, Tile::NR, Tile::PAD, Tile::MIN, Tile::GAIN, [&](int C) { return k.active(C); });
  k.launch(a, n, a.s.cluster, s);
}

vc_status draft_call(const char* who, const vc_attn_shape* shape, const vc_fp4_cache* cache, int64_t window,
                     int64_t n_sink, const void* q, float* out, float* lse, void* ws, size_t ws_bytes, int stuck_warp,
                     uint64_t wait_ns, void* stream_) {
  vc_status st = check_draft(shape, cache, who);
  if (st != VC_OK) return st;
  VC_REQUIRE(window >= 0 && n_sink >= 0, "%s: window and n_sink must be >= 0", who);
  VC_REQUIRE(cache->records && q && out && ws, "%s: null pointer argument", who);
  VC_REQUIRE(aligned16(cache->records) && aligned16(q) && aligned16(out) && aligned16(ws),
             "%s: records, q, out and workspace must be 16-byte aligned", who);
  const int g = shape->Hq / shape->Hkv;
  const stream::Plan p = stream::plan(g, shape->D);
  VC_REQUIRE(ws_bytes >= p.total, "%s: workspace too small (%zu < %zu)", who, ws_bytes, p.total);
  FArgs a{};
  a.records = static_cast<const uint8_t*>(cache->records);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k_exp = cache->k_exp;
  const float sm = shape->sm_scale > 0.f ? shape->sm_scale : 1.0f / sqrtf(static_cast<float>(shape->D));
  a.scale_log2 = sm * 1.4426950408889634f;
  a.stuck_warp = stuck_warp;
  a.wait_ns = wait_ns;
  a.s.out = out;
  a.s.lse = lse;
  a.s.lens = cache->lens;
  a.s.v_exp = cache->v_exp;
  a.s.T_cap = cache->T_cap;
  a.s.T = static_cast<uint32_t>(cache->lens ? 0 : cache->T);
  // a window as long as the cache hides nothing; no position reaches 2^31 - 1
  a.s.window = window >= cache->T_cap ? 0u : static_cast<uint32_t>(window);
  a.s.n_sink = static_cast<uint32_t>(std::min<int64_t>(n_sink, INT32_MAX));
  a.s.B = shape->B;
  a.s.Hq = shape->Hq;
  a.s.Hkv = shape->Hkv;
  a.s.g = g;
  a.s.nq = 1;
  stream::bind_workspace(a.s, p, ws);
  const uint32_t L = static_cast<uint32_t>(cache->lens ? cache->T_cap : cache->T);
  cudaStream_t s = static_cast<cudaStream_t>(stream_);
  if (shape->D == 128)
    g <= 4 ? launch_draft<128, true>(a, p, L, s) : launch_draft<128, false>(a, p, L, s);
  else
    g <= 4 ? launch_draft<64, true>(a, p, L, s) : launch_draft<64, false>(a, p, L, s);
  return launch_status(who);
}

}  // namespace
}  // namespace vc

extern "C" {

size_t vc_draft_attn_fp4_workspace_size(const vc_attn_shape* shape, const vc_fp4_cache* cache) {
  if (vc::check_draft(shape, cache, "vc_draft_attn_fp4_workspace_size") != VC_OK) return 0;
  return vc::stream::plan(shape->Hq / shape->Hkv, shape->D).total;
}

vc_status vc_draft_attn_fp4(const vc_attn_shape* shape, const vc_fp4_cache* cache, int64_t window, int64_t n_sink,
                            const void* q, float* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  return vc::draft_call("vc_draft_attn_fp4", shape, cache, window, n_sink, q, out, lse, ws, ws_bytes, -1, 2000000000ull,
                        stream);
}

vc_status vc_debug_draft_fp4_abort(const vc_attn_shape* shape, const vc_fp4_cache* cache, int64_t window,
                                   int64_t n_sink, const void* q, float* out, float* lse, void* ws, size_t ws_bytes,
                                   int stuck_warp, int64_t limit_ns, void* stream) {
  VC_REQUIRE(stuck_warp >= 0 && stuck_warp < vc::stream::kWarps,
             "vc_debug_draft_fp4_abort: stuck_warp must be 0 .. 15 (got %d)", stuck_warp);
  VC_REQUIRE(limit_ns >= 1000 && limit_ns <= 100000000,
             "vc_debug_draft_fp4_abort: limit must be 1 us .. 100 ms (got %lld ns)", static_cast<long long>(limit_ns));
  return vc::draft_call("vc_debug_draft_fp4_abort", shape, cache, window, n_sink, q, out, lse, ws, ws_bytes, stuck_warp,
                        static_cast<uint64_t>(limit_ns), stream);
}

}  // extern "C"

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
// Work layout.  The visible tokens of every unit (request, KV head) are a
// list of stages (STAGE bytes of consecutive records: those of the first
// n_sink tokens, then those of the window).  The stages of all units form
// one axis that the blocks cut into equal shares, whatever the requests'
// lengths (read on the device): a share holds part of one unit, whole units,
// and part of another.  The 4 warps of a block take a segment's stages
// round-robin, each through its own ring of bulk copies that runs ahead
// across units.  A unit inside one share is written out at once; the others
// leave one partial per block, merged by the block that finishes last.
#include <algorithm>

#include "vc_fp4.cuh"
#include "vc_splitk.cuh"

namespace vc {
namespace {

constexpr int kFWarps = 4;
constexpr int kFThreads = kFWarps * 32;
constexpr int kFBlocksPerSm = 4;
constexpr int kFMinStages = 4;   // stages a block takes at least (one per warp)
constexpr float kFBelow = 11.f;  // m is set this far below the largest score
constexpr float kFMost = 15.f;   // a score this far above m moves it: P <= 2^15

template <int D>
struct FCfg {
  static constexpr int REC = fp4::Rec<D>::BYTES;
  static constexpr int NR = 256 / D;        // records per stage: 32 (D = 128) or 64 tokens
  static constexpr int STAGE = NR * REC;    // 4608 bytes
  static constexpr int NST = 3;             // ring depth of a warp
  static constexpr int RING = NST * STAGE;
  static constexpr int BAR_OFF = kFWarps * RING;
  static constexpr int SMEM_B = BAR_OFF + kFWarps * NST * 8;
  static_assert(8 * D * 4 <= STAGE, "a consumed stage holds a warp's state");
};

struct FArgs {
  const uint8_t* records;
  const __nv_bfloat16* q;
  float* out;
  float* lse;
  const int32_t* lens;
  const int32_t* k_exp;
  const int32_t* v_exp;
  int64_t T_cap, T, window, n_sink;
  int B, Hq, Hkv, g;
  float scale_log2;
  uint32_t* flags;
  uint32_t* tickets;  // [B * Hkv] partials of a unit written so far (back to 0 after the call)
  float* part_ml;     // [2 * blocks][g][2]
  float* part_o;      // [2 * blocks][g][D]
};

// One request's visible records as stages: [0, ns) cover records [0, rs),
// the others records [r0, r1).  A request without tokens has one stage
// without records, so that every unit is in some block's share.
struct Span {
  int64_t L, lo;  // length; first token of the window
  int rs, r0, r1, ns, n;
};

__host__ __device__ inline Span make_span(int64_t L, int64_t window, int64_t n_sink, int NR) {
  Span p;
  p.L = L;
  p.lo = window > 0 && L > window ? L - window : 0;
  const int64_t sinks = n_sink < p.lo ? n_sink : p.lo;
  p.rs = static_cast<int>((sinks + fp4::kTok - 1) / fp4::kTok);
  p.r0 = static_cast<int>(p.lo / fp4::kTok);
  p.r1 = static_cast<int>((L + fp4::kTok - 1) / fp4::kTok);
  if (p.rs >= p.r0) p.rs = p.r0 = 0;  // the two meet: one list from record 0
  p.ns = (p.rs + NR - 1) / NR;
  p.n = p.ns + (p.r1 - p.r0 + NR - 1) / NR;
  if (p.n == 0) p.n = 1;
  return p;
}

template <int D>
__device__ __forceinline__ Span request_span(const FArgs& a, int b) {
  int64_t L = a.T;
  if (a.lens) {
    L = __ldg(a.lens + b);
    if (L < 0 || L > a.T_cap) L = 0;
  }
  return make_span(L, a.window, a.n_sink, FCfg<D>::NR);
}

// A warp's place on the stage axis: stage s of unit (b, h), whose first stage
// is `start` stages after the block's first one; the block's part of the unit
// ends at stage `end`.
template <int D>
struct Cursor {
  Span p;
  int b, h, start, s, end;

  __device__ __forceinline__ int begin() const { return start < 0 ? -start : 0; }
  __device__ __forceinline__ void clip(int share) { end = min(p.n, share - start); }
  __device__ __forceinline__ bool valid(int share) const { return start < share; }
  __device__ __forceinline__ void next_unit(const FArgs& a, int share) {
    start += p.n;
    if (++h == a.Hkv) {
      h = 0;
      ++b;
      if (start < share) p = request_span<D>(a, b);
    }
    clip(share);
  }
  __device__ __forceinline__ int record() const { return s < p.ns ? s * FCfg<D>::NR : p.r0 + (s - p.ns) * FCfg<D>::NR; }
  __device__ __forceinline__ int records() const {
    return min(FCfg<D>::NR, (s < p.ns ? p.rs : p.r1) - record());
  }
};

__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}

// (a & m) | (b & ~m)
__device__ __forceinline__ uint32_t blend(uint32_t a, uint32_t b, uint32_t m) { return (a & m) | (b & ~m); }

template <int D, bool HALF>
__global__ void __launch_bounds__(kFThreads, kFBlocksPerSm) draft_fp4_kernel(FArgs a) {
  using C = FCfg<D>;
  using R = fp4::Rec<D>;
  constexpr int NR = C::NR;
  constexpr int KT = D / 16;  // k-steps of a score tile, m-tiles of the values
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int s_pre[kFThreads + 1];   // stages before each group of requests
  __shared__ int s_wsum[kFWarps];
  __shared__ float s_ml[kFWarps][8][2];  // (m, l) of each warp
  __shared__ int s_at[kFWarps];          // where each warp's o is (-1: no stage)
  __shared__ float s_fin[8][2];          // (M, L) of the merge
  __shared__ int s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = lane >> 2, i4 = lane & 3;
  unsigned char* ring = smem + warp * C::RING;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF) + warp * C::NST;
  if (lane == 0) {
    for (int i = 0; i < C::NST; ++i) mbar_init(&bars[i], 1);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");

  // ---- this block's share of the stage axis
  int64_t W;
  const int per = (a.B + kFThreads - 1) / kFThreads;  // requests per group
  int n_same = 0;
  if (a.lens) {
    int mine = 0;
    for (int b = tid * per; b < min(a.B, (tid + 1) * per); ++b) {
      const int64_t L = __ldg(a.lens + b);
      if ((L < 0 || L > a.T_cap) && blockIdx.x == 0) atomicOr(a.flags, VC_FLAG_BAD_LENGTH);
      mine += request_span<D>(a, b).n * a.Hkv;
    }
    int x = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) s_wsum[warp] = x;
    __syncthreads();
    for (int w = 0; w < warp; ++w) x += s_wsum[w];
    s_pre[tid + 1] = x;
    if (tid == 0) s_pre[0] = 0;
    __syncthreads();
    W = s_pre[kFThreads];
  } else {
    n_same = request_span<D>(a, 0).n;
    W = static_cast<int64_t>(n_same) * a.B * a.Hkv;
  }
  int64_t nb = (W + kFMinStages - 1) / kFMinStages;
  if (nb > gridDim.x) nb = gridDim.x;
  const int64_t k = blockIdx.x;
  if (k >= nb) return;
  const int64_t w0 = k * W / nb;
  const int share = static_cast<int>((k + 1) * W / nb - w0);
  Cursor<D> cc;
  {
    int64_t first;  // stage that unit (cc.b, 0) starts at
    if (a.lens) {
      int lo = 0, hi = kFThreads;  // group with s_pre[lo] <= w0 < s_pre[lo + 1]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_pre[mid] <= w0) lo = mid; else hi = mid;
      }
      cc.b = lo * per;
      first = s_pre[lo];
      cc.p = request_span<D>(a, cc.b);
      while (first + static_cast<int64_t>(cc.p.n) * a.Hkv <= w0) {
        first += static_cast<int64_t>(cc.p.n) * a.Hkv;
        cc.p = request_span<D>(a, ++cc.b);
      }
    } else {
      cc.b = static_cast<int>(w0 / (static_cast<int64_t>(n_same) * a.Hkv));
      first = static_cast<int64_t>(cc.b) * n_same * a.Hkv;
      cc.p = request_span<D>(a, cc.b);
    }
    cc.h = static_cast<int>((w0 - first) / cc.p.n);
    cc.start = static_cast<int>(first + static_cast<int64_t>(cc.h) * cc.p.n - w0);
    cc.clip(share);
  }

  // ---- the warp's copies: next stage with records of this warp into the next slot
  Cursor<D> ic = cc;
  ic.s = ic.begin() + warp;
  const int64_t unit_bytes = a.T_cap / fp4::kTok * R::BYTES;
  int islot = 0;
  auto issue_next = [&]() {
    for (;;) {
      if (!ic.valid(share)) return;
      if (ic.s < ic.end) {
        const int n = ic.records();
        if (n > 0) {
          if (lane == 0) {
            const uint32_t bytes = static_cast<uint32_t>(n) * C::REC;
            mbar_arrive_expect_tx(&bars[islot], bytes);
            bulk_g2s_once(ring + islot * C::STAGE,
                          a.records + (static_cast<int64_t>(ic.b) * a.Hkv + ic.h) * unit_bytes +
                              static_cast<int64_t>(ic.record()) * C::REC,
                          bytes, &bars[islot]);
          }
          islot = islot + 1 == C::NST ? 0 : islot + 1;
          ic.s += kFWarps;
          return;
        }
        ic.s += kFWarps;
      } else {
        ic.next_unit(a, share);
        ic.s = warp;  // later units start inside the share
      }
    }
  };
#pragma unroll
  for (int i = 0; i < C::NST; ++i) issue_next();

  int slot = 0;
  uint32_t phase = 0;  // bit i: parity of slot i's next completion
  bool fail = false;
  for (; cc.valid(share); cc.next_unit(a, share)) {
    const int s0 = cc.begin();
    const int unit = cc.b * a.Hkv + cc.h;
    // ---- query fragments: lane's head = its tile column, channels 4 i4 .. of each k-step
    uint32_t qf[2 * KT];
    float sc0, sc1;
    {
      const int head = HALF ? (row & 3) : row;
      const uint4* src = reinterpret_cast<const uint4*>(a.q + (static_cast<int64_t>(cc.b) * a.Hq + cc.h * a.g + head) * D + i4 * (D / 4));
      uint32_t w[D / 8];
      float big = 0.f;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        const uint4 v = head < a.g ? __ldg(src + x) : make_uint4(0, 0, 0, 0);
        w[4 * x] = v.x, w[4 * x + 1] = v.y, w[4 * x + 2] = v.z, w[4 * x + 3] = v.w;
      }
#pragma unroll
      for (int x = 0; x < D / 8; ++x) {
        const float2 f = unpack_bf2(w[x]);
        big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // a row of zeros (and a column without a head) keeps the factor 1
      const int e = big > 0.f ? max(-100, (__float_as_int(big) >> 23) - 127) - 14 : 0;
      const float up = __int_as_float((127 - e) << 23);
#pragma unroll
      for (int x = 0; x < D / 8; ++x) {
        const float2 f = unpack_bf2(w[x]);
        qf[x] = pack_h2(f.x * up, f.y * up);
      }
      // floor: -inf (a masked score) times the factor stays -inf
      const float sc = fmaxf(a.scale_log2 * fp4::two_to(a.k_exp, cc.h, 1) * __int_as_float((127 + e) << 23), 1e-37f);
      sc0 = __shfl_sync(0xffffffffu, sc, 8 * i4);
      sc1 = __shfl_sync(0xffffffffu, sc, 8 * i4 + 4);
    }
    float acc[KT][4];
#pragma unroll
    for (int x = 0; x < KT; ++x) acc[x][0] = acc[x][1] = acc[x][2] = acc[x][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    int state = -1;

    for (cc.s = s0 + warp; cc.s < cc.end; cc.s += kFWarps) {
      const int nrec = cc.records();
      if (nrec <= 0) continue;
      if (!fail && !mbar_wait_bounded(&bars[slot], (phase >> slot) & 1, a.flags)) fail = true;
      if (__any_sync(0xffffffffu, fail)) {
        fail = true;
        break;
      }
      phase ^= 1u << slot;
      const unsigned char* st = ring + slot * C::STAGE;
      state = slot;
      slot = slot + 1 == C::NST ? 0 : slot + 1;
      const int64_t t0 = static_cast<int64_t>(cc.record()) * fp4::kTok;
      const int64_t t1 = t0 + NR * fp4::kTok;
      const bool full = t1 <= cc.p.L && nrec == NR && (t0 >= cc.p.lo || t1 <= a.n_sink);

      // ---- scores
      float c[NR][4];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const unsigned char* rec = st + r * C::REC;
        c[r][0] = c[r][1] = c[r][2] = c[r][3] = 0.f;
        uint32_t ka[D / 32], kb[D / 32], sa[D / 64], sb[D / 64];  // token row, row + 8: codes, scales (both halves)
        if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(rec + lane * 16);
          const uint4 y = *reinterpret_cast<const uint4*>(rec + 512 + lane * 16);
          ka[0] = x.x, ka[1] = x.y, ka[2] = x.z, ka[3] = x.w;
          kb[0] = y.x, kb[1] = y.y, kb[2] = y.z, kb[3] = y.w;
          const uint32_t w = *reinterpret_cast<const uint32_t*>(rec + R::KS + lane * 4);
          const uint32_t p = fp4::scales_to_h2(w & 0xffffu), q = fp4::scales_to_h2(w >> 16);
          sa[0] = prmt(p, p, 0x1010), sa[1] = prmt(p, p, 0x3232);
          sb[0] = prmt(q, q, 0x1010), sb[1] = prmt(q, q, 0x3232);
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(rec + lane * 8);
          const uint2 y = *reinterpret_cast<const uint2*>(rec + 256 + lane * 8);
          ka[0] = x.x, ka[1] = x.y;
          kb[0] = y.x, kb[1] = y.y;
          const uint32_t p = fp4::scales_to_h2(*reinterpret_cast<const uint16_t*>(rec + R::KS + lane * 2));
          sa[0] = prmt(p, p, 0x1010);
          sb[0] = prmt(p, p, 0x3232);
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          uint32_t oa[4], ob[4];
          fp4::codes_to_h2(ka[w], oa);
          fp4::codes_to_h2(kb[w], ob);
#pragma unroll
          for (int x = 0; x < 4; ++x) oa[x] = hmul2(oa[x], sa[w / 2]), ob[x] = hmul2(ob[x], sb[w / 2]);
          const uint32_t f0[4] = {oa[0], ob[0], oa[1], ob[1]}, f1[4] = {oa[2], ob[2], oa[3], ob[3]};
          mma_f16(c[r], f0, qf[4 * w], qf[4 * w + 1]);
          mma_f16(c[r], f1, qf[4 * w + 2], qf[4 * w + 3]);
        }
      }
      auto seen = [&](int64_t t) { return t < cc.p.L && (t >= cc.p.lo || t < a.n_sink); };
      if (!full) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const int64_t t = t0 + r * fp4::kTok + row;
          if (r >= nrec || !seen(t)) c[r][0] = c[r][1] = -INFINITY;
          if (r >= nrec || !seen(t + 8)) c[r][2] = c[r][3] = -INFINITY;
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
        const float al0 = m0 == -INFINITY ? 0.f : ex2(m0 - n0), al1 = m1 == -INFINITY ? 0.f : ex2(m1 - n1);
        m0 = n0, m1 = n1;
        l0 *= al0, l1 *= al1;
#pragma unroll
        for (int x = 0; x < KT; ++x) acc[x][0] *= al0, acc[x][2] *= al0, acc[x][1] *= al1, acc[x][3] *= al1;
      }
      const float off0 = m0 == -INFINITY ? 0.f : -m0, off1 = m1 == -INFINITY ? 0.f : -m1;

      // ---- values
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        uint32_t bh[2], bl[2];  // P of tokens 2 i4 (+ 1) and 8 more, column = row of the lane
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float p0 = ex2(fmaf(c[r][2 * x], sc0, off0)), p1 = ex2(fmaf(c[r][2 * x + 1], sc1, off1));
          l0 += p0;
          l1 += p1;
          const uint32_t hi = pack_h2(p0, p1);
          const float2 f = unpack_h2(hi);
          const uint32_t lo = pack_h2(p0 - f.x, p1 - f.y);
          if constexpr (HALF) {
            bh[x] = movm_t(i4 < 2 ? hi : lo);
          } else {
            bh[x] = movm_t(hi);
            bl[x] = movm_t(lo);
          }
        }
        const unsigned char* rec = st + r * C::REC;
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
          const int64_t t = t0 + r * fp4::kTok + 2 * i4;
          uint32_t keep = 0;
          if (r < nrec) {
            if (seen(t)) keep |= 0xffu;
            if (seen(t + 1)) keep |= 0xff00u;
            if (seen(t + 8)) keep |= 0xff0000u;
            if (seen(t + 9)) keep |= 0xff000000u;
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
      __syncwarp();
      if (cc.s + kFWarps < cc.end) issue_next();  // the segment's last slot takes the warp's state first
    }

    // ---- the warp's state into its last consumed slot: o [head][chan]
    if (fail) {  // no result: flagged
      state = -1;
      m0 = m1 = -INFINITY;
    }
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    if (state >= 0) {
      float* o = reinterpret_cast<float*>(ring + state * C::STAGE);
#pragma unroll
      for (int x = 0; x < KT; ++x) {
        if constexpr (HALF) {  // high + low part
#pragma unroll
          for (int y = 0; y < 4; ++y) acc[x][y] += __shfl_xor_sync(0xffffffffu, acc[x][y], 2);
        }
        const int ch = row * (D / 8) + 2 * x;
        if (!HALF || i4 < 2) {
          *reinterpret_cast<float2*>(o + 2 * i4 * D + ch) = make_float2(acc[x][0], acc[x][2]);
          *reinterpret_cast<float2*>(o + (2 * i4 + 1) * D + ch) = make_float2(acc[x][1], acc[x][3]);
        }
      }
    }
    if (row == 0 && (!HALF || i4 < 2)) {
      s_ml[warp][2 * i4][0] = m0, s_ml[warp][2 * i4][1] = l0;
      s_ml[warp][2 * i4 + 1][0] = m1, s_ml[warp][2 * i4 + 1][1] = l1;
    }
    if (lane == 0) s_at[warp] = state < 0 ? -1 : warp * C::RING + state * C::STAGE;
    __syncthreads();

    // ---- the block's result for this unit: final, or a partial
    const bool whole = cc.start >= 0 && cc.end == cc.p.n;
    const int64_t my_slot = 2 * k + (cc.start > 0 ? 1 : 0);
    const float vup = fp4::two_to(a.v_exp, cc.h, 1);
    const int64_t row0 = static_cast<int64_t>(cc.b) * a.Hq + cc.h * a.g;
    for (int e = tid; e < a.g * (D / 4); e += kFThreads) {
      const int hd = e / (D / 4), ch = (e - hd * (D / 4)) * 4;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kFWarps; ++w) M = fmaxf(M, s_ml[w][hd][0]);
      float L = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kFWarps; ++w) {
        const float mw = s_ml[w][hd][0];
        if (mw == -INFINITY) continue;
        const float f = ex2(mw - M);
        L += f * s_ml[w][hd][1];
        const float4 x = *reinterpret_cast<const float4*>(smem + s_at[w] + (hd * D + ch) * 4);
        v.x += f * x.x, v.y += f * x.y, v.z += f * x.z, v.w += f * x.w;
      }
      if (whole) {
        const float n = L > 0.f ? vup / L : 0.f;
        *reinterpret_cast<float4*>(a.out + (row0 + hd) * D + ch) = make_float4(v.x * n, v.y * n, v.z * n, v.w * n);
        if (a.lse && ch == 0) a.lse[row0 + hd] = lse_from(M, L);
      } else {
        *reinterpret_cast<float4*>(a.part_o + (my_slot * a.g + hd) * D + ch) = v;
        if (ch == 0) *reinterpret_cast<float2*>(a.part_ml + (my_slot * a.g + hd) * 2) = make_float2(M, L);
      }
    }
    if (!whole) __threadfence();
    __syncthreads();
    if (state >= 0) {  // the state's slot is free again
      if (lane == 0) fence_proxy_async_smem();
      __syncwarp();
      if (!fail) issue_next();
    }
    if (whole) continue;

    // ---- the block that finishes a unit's last partial merges them
    const int64_t p0 = w0 + cc.start, p1 = p0 + cc.p.n;  // the unit's stages
    const int64_t kf = ((p0 + 1) * nb - 1) / W, kl = (p1 * nb - 1) / W;  // blocks that hold the first and the last one
    if (tid == 0) s_last = atomicAdd(a.tickets + unit, 1u) == static_cast<uint32_t>(kl - kf);
    __syncthreads();
    if (!s_last) continue;
    __threadfence();
    const int64_t first = 2 * kf + (p0 > kf * W / nb ? 1 : 0);  // then 2 k of the others
    const int np = static_cast<int>(kl - kf + 1);
    auto at = [&](int p) { return p == 0 ? first : 2 * (kf + p); };
    for (int hd = warp; hd < a.g; hd += kFWarps) {
      float M = -INFINITY, L = 0.f;
      for (int p = lane; p < np; p += 32) M = fmaxf(M, __ldcg(a.part_ml + (at(p) * a.g + hd) * 2));
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) M = warp_max_xor(M, d);
      for (int p = lane; p < np; p += 32) {
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml + (at(p) * a.g + hd) * 2));
        if (ml.x != -INFINITY) L += ex2(ml.x - M) * ml.y;
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
      if (lane == 0) s_fin[hd][0] = M, s_fin[hd][1] = L;
    }
    if (tid == 0) a.tickets[unit] = 0;
    __syncthreads();
    for (int e = tid; e < a.g * (D / 4); e += kFThreads) {
      const int hd = e / (D / 4), ch = (e - hd * (D / 4)) * 4;
      const float M = s_fin[hd][0], L = s_fin[hd][1];
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
      for (int p = 0; p < np; ++p) {
        const int64_t sl = at(p) * a.g + hd;
        const float mp = __ldcg(a.part_ml + sl * 2);
        const float4 x = __ldcg(reinterpret_cast<const float4*>(a.part_o + sl * D + ch));
        const float f = mp == -INFINITY ? 0.f : ex2(mp - M);
        v.x += f * x.x, v.y += f * x.y, v.z += f * x.z, v.w += f * x.w;
      }
      const float n = L > 0.f ? vup / L : 0.f;
      *reinterpret_cast<float4*>(a.out + (row0 + hd) * D + ch) = make_float4(v.x * n, v.y * n, v.z * n, v.w * n);
      if (a.lse && ch == 0) a.lse[row0 + hd] = lse_from(M, L);
    }
    __syncthreads();  // s_fin and s_last are the next unit's
  }
  // after a wait that gave up, copies may still be in flight
  if (fail)
    for (int i = 0; i < C::NST; ++i) mbar_wait_bounded(&bars[i], (phase >> i) & 1, nullptr, 100000000ull);
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

struct FPlan {
  int max_blocks;  // a full wave
  size_t off_ml, off_o, total;
};

FPlan plan_draft(const vc_attn_shape& sh) {
  FPlan p;
  const int g = sh.Hq / sh.Hkv;
  p.max_blocks = sm_count() * kFBlocksPerSm;
  const size_t slots = 2 * static_cast<size_t>(p.max_blocks) * g;
  p.off_ml = align_up(sizeof(WsHeader) + static_cast<size_t>(sh.B) * sh.Hkv * 4, 256);
  p.off_o = align_up(p.off_ml + slots * 2 * 4, 256);
  p.total = align_up(p.off_o + slots * sh.D * 4, 256);
  return p;
}

template <int D, bool HALF>
void launch_draft(const FArgs& a, int blocks, cudaStream_t s) {
  static bool set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !set[dev]) {
    cudaFuncSetAttribute(draft_fp4_kernel<D, HALF>, cudaFuncAttributeMaxDynamicSharedMemorySize, FCfg<D>::SMEM_B);
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kFThreads);
  cfg.dynamicSmemBytes = FCfg<D>::SMEM_B;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, draft_fp4_kernel<D, HALF>, a);
}

}  // namespace
}  // namespace vc

extern "C" {

size_t vc_draft_attn_fp4_workspace_size(const vc_attn_shape* shape, const vc_fp4_cache* cache) {
  if (vc::check_draft(shape, cache, "vc_draft_attn_fp4_workspace_size") != VC_OK) return 0;
  return vc::plan_draft(*shape).total;
}

vc_status vc_draft_attn_fp4(const vc_attn_shape* shape, const vc_fp4_cache* cache, int64_t window, int64_t n_sink,
                            const void* q, float* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  vc_status st = vc::check_draft(shape, cache, "vc_draft_attn_fp4");
  if (st != VC_OK) return st;
  VC_REQUIRE(window >= 0 && n_sink >= 0, "vc_draft_attn_fp4: window and n_sink must be >= 0");
  VC_REQUIRE(cache->records && q && out && ws, "vc_draft_attn_fp4: null pointer argument");
  VC_REQUIRE(vc::aligned16(cache->records) && vc::aligned16(q) && vc::aligned16(out) && vc::aligned16(ws),
             "vc_draft_attn_fp4: records, q, out and workspace must be 16-byte aligned");
  const vc::FPlan p = vc::plan_draft(*shape);
  VC_REQUIRE(ws_bytes >= p.total, "vc_draft_attn_fp4: workspace too small (%zu < %zu)", ws_bytes, p.total);
  char* w = static_cast<char*>(ws);
  vc::FArgs a{};
  a.records = static_cast<const uint8_t*>(cache->records);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.out = out;
  a.lse = lse;
  a.lens = cache->lens;
  a.k_exp = cache->k_exp;
  a.v_exp = cache->v_exp;
  a.T_cap = cache->T_cap;
  a.T = cache->T;
  // no position reaches 2^31: larger values mean the same and would overflow
  a.window = std::min<int64_t>(window, int64_t(1) << 31);
  a.n_sink = std::min<int64_t>(n_sink, int64_t(1) << 31);
  a.B = shape->B;
  a.Hq = shape->Hq;
  a.Hkv = shape->Hkv;
  a.g = shape->Hq / shape->Hkv;
  const float sm = shape->sm_scale > 0.f ? shape->sm_scale : 1.0f / sqrtf(static_cast<float>(shape->D));
  a.scale_log2 = sm * 1.4426950408889634f;
  a.flags = reinterpret_cast<uint32_t*>(w);
  a.tickets = reinterpret_cast<uint32_t*>(w + sizeof(vc::WsHeader));
  a.part_ml = reinterpret_cast<float*>(w + p.off_ml);
  a.part_o = reinterpret_cast<float*>(w + p.off_o);
  // blocks for the most stages that the requests can have; the kernel leaves
  // out those that their real lengths do not fill
  const vc::Span sp = vc::make_span(cache->lens ? cache->T_cap : cache->T, a.window, a.n_sink, 256 / shape->D);
  const int64_t stages = (static_cast<int64_t>(sp.n) + 1) * shape->B * shape->Hkv;
  const int blocks = static_cast<int>(
      std::min<int64_t>(p.max_blocks, (stages + vc::kFMinStages - 1) / vc::kFMinStages));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (shape->D == 128)
    a.g <= 4 ? vc::launch_draft<128, true>(a, blocks, s) : vc::launch_draft<128, false>(a, blocks, s);
  else
    a.g <= 4 ? vc::launch_draft<64, true>(a, blocks, s) : vc::launch_draft<64, false>(a, blocks, s);
  return vc::launch_status("vc_draft_attn_fp4");
}

}  // extern "C"

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
// and part of another.  The 16 warps of a block take a segment's stages
// round-robin, each through its own ring of bulk copies that runs ahead
// across units.  A unit inside one share is written out at once; the others
// leave one partial per block, merged by the block that finishes last.
#include <algorithm>

#include "vc_fp4.cuh"
#include "vc_splitk.cuh"

namespace vc {
namespace {

constexpr int kFWarps = 16;
constexpr int kFThreads = kFWarps * 32;
constexpr int kFMaxBlocks = 160;  // one per SM; partials of one unit that a merge takes
// Measured on B200 (us of device time per call at 8 requests x 32K, 1 x 262K,
// 4 x window 4096): a unit's begin -- query load, state, partial -- costs a
// block about as much as 24 stages; counted as nothing the blocks that hold
// parts of two units finish last: 66.0, 66.4, 22.5 against 61.5, 60.4, 15.7.
constexpr int kFPad = 24;
constexpr int kFMinStages = 40;  // padding and stages a block takes at least: a short unit (16 stages) stays whole
constexpr float kFBelow = 11.f;  // m is set this far below the largest score
constexpr float kFNone = -3e38f; // m before any score (finite: -inf + -m stays -inf)
constexpr float kFMost = 15.f;   // a score this far above m moves it: P <= 2^15

template <int D, bool HALF>
struct FCfg {
  static constexpr int REC = fp4::Rec<D>::BYTES;
  static constexpr int NR = 256 / D;        // records per stage: 32 (D = 128) or 64 tokens
  static constexpr int STAGE = NR * REC;    // 4608 bytes
  static constexpr int NST = 2;             // ring depth of a warp
  static constexpr int RING = NST * STAGE;
  static constexpr int BAR_OFF = kFWarps * RING;
  // a warp's state, fp32 [heads][OS] in the order of store_out's positions (the
  // padding keeps its stores free of bank conflicts)
  static constexpr int OS = D + 4;
  static constexpr int STATE = (HALF ? 4 : 8) * OS * 4;
  static constexpr int STATE_OFF = BAR_OFF + (kFWarps * NST * 8 + 15) / 16 * 16;
  static constexpr int SMEM_B = STATE_OFF + kFWarps * STATE;
  // the final merges' buffers take the ring's place
  static_assert(2 * (kFMaxBlocks * 8 * 8 + kFThreads / 2 * 16) <= BAR_OFF, "merge buffers");
};

struct FArgs {
  const uint8_t* records;
  const __nv_bfloat16* q;
  float* out;
  float* lse;
  const int32_t* lens;
  const int32_t* k_exp;
  const int32_t* v_exp;
  int64_t T_cap;
  uint32_t T, window, n_sink;  // below 2^31
  int B, Hq, Hkv, g;
  float scale_log2;
  uint32_t* flags;
  uint32_t* tickets;  // [B * Hkv] partials of a unit written so far (back to 0 after the call)
  float* part_ml;     // [2 * blocks][g][2]
  float* part_o;      // [2 * blocks][g][D]
};

// One request's visible records as stages: [0, ns) cover records [0, rs),
// the others records [r0, r1).  All tokens of stages [f0, f1) are visible.  A
// request without tokens has one stage without records, so that every unit is
// in some block's share.
struct Span {
  uint32_t L, lo;  // length; first token of the window
  int rs, r0, r1, ns, n, f0, f1;
};

__host__ __device__ inline Span make_span(uint32_t L, uint32_t window, uint32_t n_sink, int NR) {
  Span p;
  p.L = L;
  p.lo = window > 0 && L > window ? L - window : 0;
  const uint32_t sinks = n_sink < p.lo ? n_sink : p.lo;
  p.rs = static_cast<int>((sinks + fp4::kTok - 1) / fp4::kTok);
  p.r0 = static_cast<int>(p.lo / fp4::kTok);
  p.r1 = static_cast<int>((L + fp4::kTok - 1) / fp4::kTok);
  if (p.rs >= p.r0) p.rs = p.r0 = 0;  // the two meet: one list from record 0
  p.ns = (p.rs + NR - 1) / NR;
  p.n = p.ns + (p.r1 - p.r0 + NR - 1) / NR;
  p.f0 = p.ns + static_cast<int>((p.lo - p.r0 * fp4::kTok + NR * fp4::kTok - 1) / (NR * fp4::kTok));
  p.f1 = p.ns + (static_cast<int>(L / fp4::kTok) - p.r0) / NR;
  if (p.n == 0) p.n = 1;
  return p;
}

template <int D>
__device__ __forceinline__ Span request_span(const FArgs& a, int b) {
  uint32_t L = a.T;
  if (a.lens) {
    L = static_cast<uint32_t>(__ldg(a.lens + b));
    if (L > a.T_cap) L = 0;  // (a negative length too)
  }
  return make_span(L, a.window, a.n_sink, 256 / D);
}

template <int D>
__device__ __forceinline__ int stage_record(const Span& p, int s) {
  return s < p.ns ? s * 256 / D : p.r0 + (s - p.ns) * 256 / D;
}
template <int D>
__device__ __forceinline__ int stage_records(const Span& p, int s) {
  return min(256 / D, (s < p.ns ? p.rs : p.r1) - stage_record<D>(p, s));
}

// The cut of W stages into nb shares: share k starts at stage first(k).
struct Cut {
  uint32_t q, r;
  __device__ Cut(uint32_t W, uint32_t nb) : q(W / nb), r(W - W / nb * nb) {}
  __device__ uint32_t first(uint32_t k) const { return k * q + min(k, r); }
  __device__ uint32_t share_of(uint32_t x) const {  // that holds stage x
    const uint32_t big = r * (q + 1);
    return x < big ? x / (q + 1) : r + (x - big) / q;
  }
};

// mma_f16 into zeros
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}

// (a & m) | (b & ~m)
__device__ __forceinline__ uint32_t blend(uint32_t a, uint32_t b, uint32_t m) { return (a & m) | (b & ~m); }

// A warp's accumulators hold channel row * (D / 8) + 2 x + c at position
// x * 16 + row * 2 + c (m-tile x, the lane's row, c = 0, 1); states and
// partials stay in that order.  Stores positions pos .. pos + 3 of head hd of
// unit (b, h), sum v with total (M, L).
template <int D>
__device__ __forceinline__ void store_row(const FArgs& a, int b, int h, int hd, int pos, const float4& v,
                                          const float (&tot)[2]) {
  const int64_t r = static_cast<int64_t>(b) * a.Hq + h * a.g + hd;
  float* dst = a.out + r * D + (pos % 16) / 2 * (D / 8) + pos / 16 * 2;
  const float f = tot[1] > 0.f ? fp4::two_to(a.v_exp, h, 1) / tot[1] : 0.f;
  *reinterpret_cast<float2*>(dst) = make_float2(v.x * f, v.y * f);
  *reinterpret_cast<float2*>(dst + D / 8) = make_float2(v.z * f, v.w * f);
  if (a.lse && pos == 0) a.lse[r] = lse_from(tot[0], tot[1]);
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x = warp_max_xor(x, d);
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

// Merges the partials of one unit (first stage u0, n stages) into its output
// rows, by one half of the block (t: thread of the half; buf, tot: shared
// memory of the half).  Written for few instructions rather than few cycles:
// this code, like the rest of the prologue and epilogue, runs once per block,
// out of an empty instruction cache.
constexpr int kFHalf = kFThreads / 2;
constexpr int kFMergeB = kFMaxBlocks * 8 * 8 + kFHalf * 16;

template <int D>
__device__ __forceinline__ void merge_unit(const FArgs& a, const Cut cut, int unit, uint32_t u0, int n, int half, int t,
                                           unsigned char* buf, float (*tot)[2]) {
  const int warp = t >> 5, lane = t & 31;
  const int g = a.g;
  const uint32_t kf = cut.share_of(u0);
  const int np = static_cast<int>(cut.share_of(u0 + n - 1) - kf) + 1;
  // slot of partial 0 (the unit is the first or the last one of its block), then 2 k of block k
  const int first = 2 * kf + (u0 - kFPad > cut.first(kf) ? 1 : 0);
  float2* ml = reinterpret_cast<float2*>(buf);  // [np][g] (m, l), then (weight, -)
  float4* sum = reinterpret_cast<float4*>(buf + kFMaxBlocks * 8 * 8);
  auto at = [&](int i) { return i == 0 ? first : 2 * (static_cast<int>(kf) + i); };
  auto sync = [&]() { asm volatile("bar.sync %0, %1;\n" ::"r"(1 + half), "n"(kFHalf) : "memory"); };
  // thread groups take partials in turn, 4 positions a thread, 8 loads in flight
  const int items = g * D / 4, groups = kFHalf / items;
  const int grp = t / items, it = t - grp * items, hd = it * 4 / D;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int base = 0; base < np; base += 8 * groups) {
    float4 x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = base + j * groups + grp;
      x[j] = grp < groups && i < np
                 ? __ldcg(reinterpret_cast<const float4*>(a.part_o + static_cast<int64_t>(at(i)) * g * D) + it)
                 : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (base == 0) {  // meanwhile the weights
#pragma unroll 1
      for (int e = t; e < np * g; e += kFHalf) {
        const int i = e / g;
        ml[e] = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + at(i) * g + (e - i * g));
      }
      sync();
      if (warp < g) {
        float M = -INFINITY, L = 0.f;
#pragma unroll 1
        for (int i = lane; i < np; i += 32) M = fmaxf(M, ml[i * g + warp].x);
        M = warp_max(M);
#pragma unroll 1
        for (int i = lane; i < np; i += 32) {
          const float2 y = ml[i * g + warp];
          const float w = y.x == -INFINITY ? 0.f : ex2(y.x - M);
          L += w * y.y;
          ml[i * g + warp].x = w;
        }
        L = warp_sum(L);
        if (lane == 0) tot[warp][0] = M, tot[warp][1] = L;
      }
      sync();
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = base + j * groups + grp;
      const float w = i < np && grp < groups ? ml[i * g + hd].x : 0.f;
      v.x += w * x[j].x, v.y += w * x[j].y, v.z += w * x[j].z, v.w += w * x[j].w;
    }
  }
  sum[t] = v;
  sync();
  if (grp == 0) {
#pragma unroll 1
    for (int i = 1; i < min(groups, np); ++i) {
      const float4 x = sum[i * items + it];
      v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
    }
    const int b = unit / a.Hkv, h = unit - b * a.Hkv;
    store_row<D>(a, b, h, hd, it * 4 % D, v, tot[hd]);
  }
}

template <int D, bool HALF>
__global__ void __launch_bounds__(kFThreads, 1) draft_fp4_kernel(FArgs a) {
  using C = FCfg<D, HALF>;
  using R = fp4::Rec<D>;
  constexpr int NR = C::NR;
  constexpr int KT = D / 16;  // k-steps of a score tile, m-tiles of the values
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int s_pre[kFThreads + 1];   // stages before each group of requests
  __shared__ int s_wsum[kFWarps];
  __shared__ float s_ml[kFWarps][8][2];  // (m, l) of each warp
  __shared__ float s_f[kFWarps][8];      // its weight in the block's sum
  __shared__ float s_tot[2][8][2];       // (M, L) of the sum
  __shared__ int s_last[2];
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

  // ---- this block's share of the stage axis (below 2^31 stages: they all have bytes in memory)
  uint32_t W;
  const int per = (a.B + kFThreads - 1) / kFThreads;  // requests per group
  uint32_t n_same = 0;
  if (a.lens) {
    int mine = 0;
    for (int b = tid * per; b < min(a.B, (tid + 1) * per); ++b) {
      if (blockIdx.x == 0 && static_cast<uint32_t>(__ldg(a.lens + b)) > a.T_cap) atomicOr(a.flags, VC_FLAG_BAD_LENGTH);
      mine += (request_span<D>(a, b).n + kFPad) * a.Hkv;
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
    n_same = request_span<D>(a, 0).n + kFPad;
    W = n_same * a.B * a.Hkv;
  }
  const uint32_t nb = min((W + kFMinStages - 1) / kFMinStages, gridDim.x);
  const uint32_t k = blockIdx.x;
  if (k >= nb) return;
  const Cut cut(W, nb);
  const uint32_t w0 = cut.first(k);
  const int share = static_cast<int>(cut.first(k + 1) - w0);
  // the place on the axis: unit (b, h), whose first stage (past its padding)
  // is `start` stages after the share's first one
  int b, h, start;
  Span p;
  {
    uint32_t first;  // stage that unit (b, 0) starts at
    if (a.lens) {
      int lo = 0, hi = kFThreads;  // group with s_pre[lo] <= w0 < s_pre[lo + 1]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_pre[mid] <= w0) lo = mid; else hi = mid;
      }
      b = lo * per;
      first = s_pre[lo];
      p = request_span<D>(a, b);
      while (first + (p.n + kFPad) * a.Hkv <= w0) {
        first += (p.n + kFPad) * a.Hkv;
        p = request_span<D>(a, ++b);
      }
    } else {
      b = w0 / (n_same * a.Hkv);
      first = b * n_same * a.Hkv;
      p = request_span<D>(a, b);
    }
    h = (w0 - first) / (p.n + kFPad);
    start = static_cast<int>(first + h * (p.n + kFPad)) - static_cast<int>(w0) + kFPad;
  }

  // ---- the warp's copies run ahead of its work: stage is of unit (ib, ih),
  //      at isrc if it is below ifast (stages of NR records, one after the
  //      other)
  // bf16 query words of this lane: its tile column's head, D / 4 channels from
  // i4 * D / 4 (requested before the copies, which fill the memory's queues)
  uint32_t qf[2 * KT];
  float kup;
  auto load_q = [&](int b, int h) {
    const int head = HALF ? (row & 3) : row;
    const uint4* src = reinterpret_cast<const uint4*>(a.q + (static_cast<int64_t>(b) * a.Hq + h * a.g + head) * D + i4 * (D / 4));
#pragma unroll
    for (int x = 0; x < D / 32; ++x) {
      const uint4 v = head < a.g ? __ldg(src + x) : make_uint4(0, 0, 0, 0);
      qf[4 * x] = v.x, qf[4 * x + 1] = v.y, qf[4 * x + 2] = v.z, qf[4 * x + 3] = v.w;
    }
    kup = fp4::two_to(a.k_exp, h, 1);
  };
  load_q(b, h);
  const int64_t unit_bytes = a.T_cap / fp4::kTok * R::BYTES;
  int ib = b, ih = h, istart = start, is = max(0, -start) + warp, ifast = 0, islot = 0;
  const uint8_t* isrc = nullptr;
  const uint64_t policy = l2_evict_first();  // the records are read once per call
  auto issue_next = [&]() {
    uint32_t bytes = C::STAGE;
    if (is >= ifast) {  // look for the next stage with records
      for (;;) {
        if (istart >= share) return;
        const Span ip = request_span<D>(a, ib);
        const int end = min(ip.n, share - istart);
        if (is < end) {
          const int n = stage_records<D>(ip, is);
          if (n > 0) {
            bytes = static_cast<uint32_t>(n) * C::REC;
            isrc = a.records + (static_cast<int64_t>(ib) * a.Hkv + ih) * unit_bytes +
                   static_cast<int64_t>(stage_record<D>(ip, is)) * C::REC;
            ifast = is < ip.ns ? 0 : min(end, ip.ns + (ip.r1 - ip.r0) / NR);
            break;
          }
          is += kFWarps;
        } else {
          istart += ip.n + kFPad;
          is = warp;
          ifast = 0;
          if (++ih == a.Hkv) ih = 0, ++ib;
        }
      }
    }
    if (lane == 0) {
      mbar_arrive_expect_tx(&bars[islot], bytes);
      bulk_g2s_hint(ring + islot * C::STAGE, isrc, bytes, &bars[islot], policy);
    }
    islot = islot + 1 == C::NST ? 0 : islot + 1;
    is += kFWarps;
    isrc += kFWarps * C::STAGE;
  };
#pragma unroll 1
  for (int i = 0; i < C::NST; ++i) issue_next();

  // hi lanes keep a weight's first 11 bits, lo lanes the rest: v = p * lo_f + ((p & mask) ^ lo_s)
  const float lo_f = i4 < 2 ? 0.f : 1.f;
  const uint32_t lo_s = i4 < 2 ? 0u : 0x80000000u;
  int slot = 0;
  uint32_t phase = 0;  // parity of the slot's next completion
  // the share's first and last unit when other blocks hold parts of them
  int open[2] = {-1, -1}, open_n[2] = {0, 0};
  uint32_t open_u0[2] = {0, 0};  // their first stage
  bool fail = false;
#pragma unroll 1
  while (start < share) {
    const int s0 = max(0, -start), end = min(p.n, share - start);
    const int unit = b * a.Hkv + h;
    // ---- query fragments: lane's head = its tile column, channels 4 i4 .. of each k-step
    float sc0, sc1;
    {
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
    }
    float acc[KT][4];
#pragma unroll
    for (int x = 0; x < KT; ++x) acc[x][0] = acc[x][1] = acc[x][2] = acc[x][3] = 0.f;
    float m0 = kFNone, m1 = kFNone, l0 = 0.f, l1 = 0.f;

    for (int x = s0 + warp; x < end && !fail; x += kFWarps) {
      const bool full = x >= p.f0 && x < p.f1;
      if (!full && stage_records<D>(p, x) <= 0) break;  // a request without tokens
      if (!__all_sync(0xffffffffu, mbar_try_wait_hint(&bars[slot], phase, 20000u)) &&
          __any_sync(0xffffffffu, !mbar_wait_bounded(&bars[slot], phase, a.flags))) {
        fail = true;
        break;
      }
      const unsigned char* st = ring + slot * C::STAGE;
      if (++slot == C::NST) slot = 0, phase ^= 1;

      // ---- scores
      float c[NR][4];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const unsigned char* rec = st + r * C::REC;
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
          if (w == 0)
            mma_f16_zero(c[r], f0, qf[0], qf[1]);
          else
            mma_f16(c[r], f0, qf[4 * w], qf[4 * w + 1]);
          mma_f16(c[r], f1, qf[4 * w + 2], qf[4 * w + 3]);
        }
      }
      auto seen = [&](uint32_t t) { return t < p.L && (t >= p.lo || t < a.n_sink); };
      uint32_t t0 = 0;
      int nrec = NR;
      if (!full) {
        t0 = static_cast<uint32_t>(stage_record<D>(p, x)) * fp4::kTok;
        nrec = stage_records<D>(p, x);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const uint32_t t = t0 + r * fp4::kTok + row;
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
            bh[x] = movm_t(pack_h2(fmaf(p0, lo_f, __uint_as_float(h0 ^ lo_s)), fmaf(p1, lo_f, __uint_as_float(h1 ^ lo_s))));
          } else {
            bh[x] = movm_t(pack_h2(__uint_as_float(h0), __uint_as_float(h1)));
            bl[x] = movm_t(pack_h2(p0 - __uint_as_float(h0), p1 - __uint_as_float(h1)));
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
          const uint32_t t = t0 + r * fp4::kTok + 2 * i4;
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
      issue_next();
    }

    if (start + p.n + kFPad < share) load_q(h + 1 < a.Hkv ? b : b + 1, h + 1 < a.Hkv ? h + 1 : 0);

    // ---- the warp's state, then the block's result for this unit: output
    //      rows, or a partial
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    if (fail || m0 == kFNone) m0 = -INFINITY;
    if (fail || m1 == kFNone) m1 = -INFINITY;
    float* o = reinterpret_cast<float*>(smem + C::STATE_OFF + warp * C::STATE) + 2 * i4 * C::OS + row * 2;
#pragma unroll
    for (int x = 0; x < KT; ++x) {
      if constexpr (HALF) {  // high + low part
#pragma unroll
        for (int y = 0; y < 4; ++y) acc[x][y] += __shfl_xor_sync(0xffffffffu, acc[x][y], 2);
      }
      if (!HALF || i4 < 2) {
        *reinterpret_cast<float2*>(o + x * 16) = make_float2(acc[x][0], acc[x][2]);
        *reinterpret_cast<float2*>(o + C::OS + x * 16) = make_float2(acc[x][1], acc[x][3]);
      }
    }
    if (row == 0 && (!HALF || i4 < 2)) {
      s_ml[warp][2 * i4][0] = m0, s_ml[warp][2 * i4][1] = l0;
      s_ml[warp][2 * i4 + 1][0] = m1, s_ml[warp][2 * i4 + 1][1] = l1;
    }
    __syncthreads();
    if (warp < a.g) {
      const float m = lane < kFWarps ? s_ml[lane][warp][0] : -INFINITY;
      const float M = warp_max(m);
      const float f = m == -INFINITY ? 0.f : ex2(m - M);
      const float L = warp_sum(lane < kFWarps ? f * s_ml[lane][warp][1] : 0.f);
      if (lane < kFWarps) s_f[lane][warp] = f;
      if (lane == 0) s_tot[0][warp][0] = M, s_tot[0][warp][1] = L;
    }
    __syncthreads();
    const bool whole = start >= 0 && end == p.n;
    if (tid < a.g * (D / 4)) {
      const int hd = tid / (D / 4), pos = (tid - hd * (D / 4)) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int w = 0; w < kFWarps; ++w) {
        const float f = s_f[w][hd];
        const float4 x = *reinterpret_cast<const float4*>(smem + C::STATE_OFF + w * C::STATE + (hd * C::OS + pos) * 4);
        v.x += f * x.x, v.y += f * x.y, v.z += f * x.z, v.w += f * x.w;
      }
      if (whole) {
        store_row<D>(a, b, h, hd, pos, v, s_tot[0][hd]);
      } else {
        const int64_t at = (2 * static_cast<int64_t>(k) + (start > kFPad ? 1 : 0)) * a.g + hd;
        *reinterpret_cast<float4*>(a.part_o + at * D + pos) = v;
        if (pos == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(s_tot[0][hd][0], s_tot[0][hd][1]);
      }
    }
    __syncthreads();
    if (!whole) {
      if (start > kFPad)
        open[1] = unit, open_u0[1] = w0 + start, open_n[1] = p.n;
      else
        open[0] = unit, open_u0[0] = w0 + start, open_n[0] = p.n;
    }
    start += p.n + kFPad;
    if (++h == a.Hkv) {
      h = 0;
      if (start < share) p = request_span<D>(a, ++b);
    }
  }
  // after a wait that gave up, copies may still be in flight
  if (fail)
    for (int i = 0; i < C::NST; ++i) mbar_wait_bounded(&bars[i], i < slot ? phase ^ 1 : phase, nullptr, 100000000ull);

  // ---- the block that finishes a unit's last partial merges them
  if (open[0] < 0 && open[1] < 0) return;
  if (tid < 2) {  // (the barrier above ordered the other threads' stores before the fence)
    const int u = tid ? open[1] : open[0];
    bool last = false;
    if (u >= 0) {
      const uint32_t u0 = tid ? open_u0[1] : open_u0[0];
      const uint32_t others = cut.share_of(u0 + (tid ? open_n[1] : open_n[0]) - 1) - cut.share_of(u0);
      __threadfence();
      last = atomicAdd(a.tickets + u, 1u) == others;
      if (last) {
        a.tickets[u] = 0;
        __threadfence();
      }
    }
    s_last[tid] = last;
  }
  __syncthreads();
  const int half = tid / kFHalf;
  if (s_last[half])
    merge_unit<D>(a, cut, half ? open[1] : open[0], half ? open_u0[1] : open_u0[0], half ? open_n[1] : open_n[0], half,
                  tid - half * kFHalf, smem + half * kFMergeB, s_tot[half]);
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
  p.max_blocks = std::min(sm_count(), kFMaxBlocks);
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
    cudaFuncSetAttribute(draft_fp4_kernel<D, HALF>, cudaFuncAttributeMaxDynamicSharedMemorySize, FCfg<D, HALF>::SMEM_B);
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kFThreads);
  cfg.dynamicSmemBytes = FCfg<D, HALF>::SMEM_B;
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
  a.T = static_cast<uint32_t>(cache->lens ? 0 : cache->T);
  // no position reaches 2^31 - 1: larger values mean the same
  a.window = static_cast<uint32_t>(std::min<int64_t>(window, INT32_MAX));
  a.n_sink = static_cast<uint32_t>(std::min<int64_t>(n_sink, INT32_MAX));
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
  const vc::Span sp = vc::make_span(static_cast<uint32_t>(cache->lens ? cache->T_cap : cache->T), a.window, a.n_sink, 256 / shape->D);
  const int64_t stages = (static_cast<int64_t>(sp.n) + 1 + vc::kFPad) * shape->B * shape->Hkv;
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

// vc_stream.cuh -- attention of a few query rows per (request, KV head) over
// its whole cache: the work split and the merges shared by the 4-bit draft
// (vc_draft_fp4.cu) and the one-token form of windowed verification
// (vc_verify_rows.cu).
//
// A unit is one (request, KV head); its query rows (nq positions x g heads, at
// most 8) are the columns of every tile.  The visible tokens of a unit are a
// list of stages (NR records of 16 tokens: those of the first n_sink tokens,
// then those of the windows).  The stages of all units form one axis that the
// blocks -- one of 16 warps per SM -- cut into equal shares, whatever the
// requests' lengths (read on the device): a share holds part of one unit,
// whole units, and part of another.  A unit's begin counts as PAD stages, what
// its fixed costs take.  The warps of a block take a segment's stages
// round-robin; at its end their states meet in shared memory.  A unit inside
// one share is written out at once; the others leave one partial per block,
// merged (in a fixed order) by the block that finishes last.
//
// Short contexts (Args::cluster): the blocks of one thread-block cluster take
// one unit's stages and merge through each other's shared memory, without the
// axis, partials in memory and tickets.  See choose() for the rule.
//
// Both kernels are programmatic dependents, resident while the call before
// them still writes: nothing is read before griddepcontrol.wait, and nothing
// through the read-only path.  The wait comes before launch_dependents, so a
// grid that is scheduled early finds only its direct predecessor unfinished,
// which is what a caller promises about with VC_CACHE_STATIC.
//
// Code outside the stage loop is kept short rather than fast: it runs once or
// twice per block out of an empty instruction cache (unrolled merges and one
// block of 4 warps more per SM cost 5 us of 66 at 8 x 32K tokens).
#pragma once

#include "vc_once.h"
#include "vc_splitk.cuh"

namespace vc {
namespace stream {

constexpr int kTok = 16;  // tokens per record
constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxBlocks = 160;    // one per SM; partials of one unit that a merge takes
constexpr float kNone = -3e38f;    // a column's m before any score (finite: -inf + -m stays -inf)

struct Args {
  float* out;
  float* lse;
  const int32_t* lens;
  const int32_t* v_exp;
  int64_t T_cap;               // lengths above are invalid
  uint32_t T, window, n_sink;  // below 2^31
  int B, Hq, Hkv, g, nq;
  int cluster;  // blocks per unit, one cluster; 0: the shared axis
  uint32_t* flags;
  uint32_t* tickets;  // [B * Hkv] partials of a unit written so far (back to 0 after the call)
  float* part_ml;     // [2 * blocks][nq * g][2]
  float* part_o;      // [2 * blocks][nq * g][D]
};

// Row i of a request of L tokens sits at p = L - nq + i and sees t <= p with
// window == 0, t > p - window or t < n_sink.
//
// One request's visible records as stages: [0, ns) cover records [0, rs),
// the others records [r0, r1).  Every row sees all tokens of stages [f0, f1).
// A request without tokens has one stage without records, so that every unit
// is in some block's share.
struct Span {
  uint32_t L, lo;  // length; first token of the first row's window
  int rs, r0, r1, ns, n, f0, f1;
};

__host__ __device__ inline Span make_span(uint32_t L, uint32_t nq, uint32_t window, uint32_t n_sink, int NR) {
  Span p;
  p.L = L;
  p.lo = window > 0 && L + 1 > window + nq ? L + 1 - nq - window : 0;
  const uint32_t sinks = n_sink < p.lo ? n_sink : p.lo;
  p.rs = static_cast<int>((sinks + kTok - 1) / kTok);
  p.r0 = static_cast<int>(p.lo / kTok);
  p.r1 = static_cast<int>((L + kTok - 1) / kTok);
  if (p.rs >= p.r0) p.rs = p.r0 = 0;  // the two meet: one list from record 0
  p.ns = (p.rs + NR - 1) / NR;
  p.n = p.ns + (p.r1 - p.r0 + NR - 1) / NR;
  const uint32_t last = window > 0 && L > window ? L - window : 0;  // first token of the last row's window
  const uint32_t below = L + 1 > nq ? L + 1 - nq : 0;               // tokens that the first row sees
  p.f0 = p.ns + static_cast<int>((last - p.r0 * kTok + NR * kTok - 1) / (NR * kTok));
  p.f1 = p.ns + (static_cast<int>(below / kTok) - p.r0) / NR;
  if (p.n == 0) p.n = 1;
  return p;
}

// Loads of what the call before may have written (see above), through L1 but
// never the read-only path, whatever the compiler can prove.
__device__ __forceinline__ uint32_t load_word(const void* p) {
  uint32_t v;
  asm volatile("ld.global.b32 %0, [%1];\n" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 load_16(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Request b's length as stored (a negative one is above every T_cap).
__device__ __forceinline__ uint32_t stored_length(const Args& a, int b) { return load_word(a.lens + b); }

template <int NR>
__device__ __forceinline__ Span request_span(const Args& a, int b) {
  uint32_t L = a.T;
  if (a.lens) {
    L = stored_length(a, b);
    if (L > a.T_cap) L = 0;
  }
  return make_span(L, a.nq, a.window, a.n_sink, NR);
}

template <int NR>
__device__ __forceinline__ int stage_record(const Span& p, int s) {
  return s < p.ns ? s * NR : p.r0 + (s - p.ns) * NR;
}
template <int NR>
__device__ __forceinline__ int stage_records(const Span& p, int s) {
  return min(NR, (s < p.ns ? p.rs : p.r1) - stage_record<NR>(p, s));
}

// Whether row i sees token t.
__device__ __forceinline__ bool row_sees(const Args& a, const Span& p, int i, uint32_t t) {
  const uint32_t up = p.L + i;  // position + nq
  return t + a.nq <= up && (a.window == 0 || t + a.nq + a.window > up || t < a.n_sink);
}
// Whether any row does.
__device__ __forceinline__ bool seen(const Args& a, const Span& p, uint32_t t) {
  return t < p.L && (t >= p.lo || t < a.n_sink);
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

__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
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

// A warp's accumulators hold channel row * (D / 8) + 2 x + c at position
// x * 16 + row * 2 + c (m-tile x, the lane's row, c = 0, 1); states and
// partials stay in that order.  A state is fp32 [columns][OS] (the padding
// keeps its stores free of bank conflicts).
template <int D>
struct State {
  static constexpr int OS = D + 4;
  static constexpr int bytes(int cols) { return cols * OS * 4; }
};

// Stores positions pos .. pos + 3 of column col of unit (b, h), sum v with total (M, L).
template <int D>
__device__ __forceinline__ void store_row(const Args& a, int b, int h, int col, int pos, const float4& v,
                                          const float (&tot)[2]) {
  const int i = col / a.g;
  const int64_t r = (static_cast<int64_t>(b) * a.nq + i) * a.Hq + h * a.g + col - i * a.g;
  float* dst = a.out + r * D + (pos % 16) / 2 * (D / 8) + pos / 16 * 2;
  const float f = tot[1] > 0.f ? two_to(a.v_exp, h, 1) / tot[1] : 0.f;
  *reinterpret_cast<float2*>(dst) = make_float2(v.x * f, v.y * f);
  *reinterpret_cast<float2*>(dst + D / 8) = make_float2(v.z * f, v.w * f);
  if (a.lse && pos == 0) a.lse[r] = lse_from(tot[0], tot[1]);
}

// Merges the partials of one unit (first stage u0, n stages) into its output
// rows, by one half of the block: the other half may have the block's other
// open unit to merge.  (Never by all threads: the order of the sum must not
// depend on which block finishes last.)  t: thread of the half; bar: its
// barrier; buf, tot: its shared memory.
constexpr int kHalf = kThreads / 2;
constexpr int kMergeB = kMaxBlocks * 8 * 8 + kHalf * 16;

template <int D, int PAD>
__device__ __forceinline__ void merge_unit(const Args& a, const Cut cut, int unit, uint32_t u0, int n, int bar, int t,
                                           unsigned char* buf, float (*tot)[2]) {
  const int warp = t >> 5, lane = t & 31;
  const int g = a.nq * a.g;  // columns
  const uint32_t kf = cut.share_of(u0);
  const int np = static_cast<int>(cut.share_of(u0 + n - 1) - kf) + 1;
  // slot of partial 0 (the unit is the first or the last one of its block), then 2 k of block k
  const int first = 2 * kf + (u0 - PAD > cut.first(kf) ? 1 : 0);
  float2* ml = reinterpret_cast<float2*>(buf);  // [np][g] (m, l), then (weight, -)
  float4* sum = reinterpret_cast<float4*>(buf + kMaxBlocks * 8 * 8);
  auto at = [&](int i) { return i == 0 ? first : 2 * (static_cast<int>(kf) + i); };
  auto sync = [&]() { asm volatile("bar.sync %0, %1;\n" ::"r"(bar), "n"(kHalf) : "memory"); };
  // thread groups take partials in turn, 4 positions a thread, 16 loads in flight
  const int items = g * D / 4, groups = kHalf / items;
  const int grp = t / items, it = t - grp * items, hd = it * 4 / D;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int base = 0; base < np; base += 16 * groups) {
    float4 x[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int i = base + j * groups + grp;
      x[j] = grp < groups && i < np
                 ? __ldcg(reinterpret_cast<const float4*>(a.part_o + static_cast<int64_t>(at(i)) * g * D) + it)
                 : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (base == 0) {  // meanwhile the weights
#pragma unroll 1
      for (int e = t; e < np * g; e += kHalf) {
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
    for (int j = 0; j < 16; ++j) {
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

// One block's work.  Tile: the cache format's part --
//   D, NR, COLS (columns of a state, 4 or 8), PAD, MIN (least share) constants;
//   query(b, h)                   requests a unit's query rows
//   begin(b, h, start, share)     starts the warp's copies
//   unit(p, b, h, x, end)         a unit's first stage of this warp is x
//   stage(p, x, end)              one stage; false when a wait gave up
//   finish(o, ml)                 the warp's state, ml [COLS][2]
//   drain()                       after a wait that gave up: copies in flight
// smem: kWarps states; merge: 2 kMergeB bytes (free after the last unit).
template <class Tile>
__device__ __forceinline__ void run(const Args& a, Tile& tile, unsigned char* states, unsigned char* merge) {
  constexpr int D = Tile::D, NR = Tile::NR, PAD = Tile::PAD;
  constexpr int STATE = State<D>::bytes(Tile::COLS), OS = State<D>::OS;
  __shared__ int s_pre[kThreads + 1];  // stages before each group of requests
  __shared__ int s_wsum[kWarps];
  __shared__ float s_ml[kWarps][8][2];  // (m, l) of each warp
  __shared__ float s_f[kWarps][8];      // its weight in the block's sum
  __shared__ __align__(16) float s_tot[2][8][2];  // (M, L) of the sum
  __shared__ int s_last[2];
  __shared__ __align__(16) float s_part[8 * D];  // cluster: the block's sum, [columns][D]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cols = a.nq * a.g;

  // the place on the axis: unit (b, h), whose first stage (past its padding)
  // is `start` stages after the first one of the block's `share`
  int b, h, start, share;
  Span p;
  const uint32_t k = blockIdx.x;
  Cut cut(0, 1);
  uint32_t w0 = 0;
  if (a.cluster) {  // rank r of a unit's C blocks: stages from ceil(r n / C)
    const int unit = k / a.cluster, rank = k - unit * a.cluster;
    b = unit / a.Hkv, h = unit - b * a.Hkv;
    if (a.lens && tid == 0 && stored_length(a, b) > a.T_cap) atomicOr(a.flags, VC_FLAG_BAD_LENGTH);
    p = request_span<NR>(a, b);
    const uint32_t n = p.n, C = a.cluster;  // (the product stays below 2^31: at most 8 blocks)
    const int s0 = (rank * n + C - 1) / C;
    start = -s0;
    share = static_cast<int>(((rank + 1) * n + C - 1) / C) - s0;
  } else {
    // ---- this block's share of the stage axis (below 2^31 stages: they all have bytes in memory)
    uint32_t W;
    const int per = (a.B + kThreads - 1) / kThreads;  // requests per group
    uint32_t n_same = 0;
    if (a.lens) {
      int mine = 0;
      for (int b = tid * per; b < min(a.B, (tid + 1) * per); ++b) {
        if (blockIdx.x == 0 && stored_length(a, b) > a.T_cap) atomicOr(a.flags, VC_FLAG_BAD_LENGTH);
        mine += (request_span<NR>(a, b).n + PAD) * a.Hkv;
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
      W = s_pre[kThreads];
    } else {
      n_same = request_span<NR>(a, 0).n + PAD;
      W = n_same * a.B * a.Hkv;
    }
    const uint32_t nb = min((W + Tile::MIN - 1) / Tile::MIN, gridDim.x);
    if (k >= nb) return;
    cut = Cut(W, nb);
    w0 = cut.first(k);
    share = static_cast<int>(cut.first(k + 1) - w0);
    {
      uint32_t first;  // stage that unit (b, 0) starts at
      if (a.lens) {
        int lo = 0, hi = kThreads;  // group with s_pre[lo] <= w0 < s_pre[lo + 1]
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (s_pre[mid] <= w0) lo = mid; else hi = mid;
        }
        b = lo * per;
        first = s_pre[lo];
        p = request_span<NR>(a, b);
        while (first + (p.n + PAD) * a.Hkv <= w0) {
          first += (p.n + PAD) * a.Hkv;
          p = request_span<NR>(a, ++b);
        }
      } else {
        b = w0 / (n_same * a.Hkv);
        first = b * n_same * a.Hkv;
        p = request_span<NR>(a, b);
      }
      h = (w0 - first) / (p.n + PAD);
      start = static_cast<int>(first + h * (p.n + PAD)) - static_cast<int>(w0) + PAD;
    }
  }
  tile.query(b, h);
  tile.begin(b, h, start, share);

  // the share's first and last unit when other blocks hold parts of them
  int open[2] = {-1, -1}, open_n[2] = {0, 0};
  uint32_t open_u0[2] = {0, 0};  // their first stage
  bool fail = false;
#pragma unroll 1
  while (start < share) {
    const int s0 = max(0, -start), end = min(p.n, share - start);
    tile.unit(p, b, h, s0 + warp, end);
    for (int x = s0 + warp; x < end && !fail; x += kWarps) {
      if (x >= p.f1 && stage_records<NR>(p, x) <= 0) break;  // a request without tokens
      fail = !tile.stage(p, x, end);
    }
    if (start + p.n + PAD < share) tile.query(h + 1 < a.Hkv ? b : b + 1, h + 1 < a.Hkv ? h + 1 : 0);

    // ---- the warps' states, then the block's result for this unit: output
    //      rows, or a partial
    tile.finish(reinterpret_cast<float*>(states + warp * STATE), s_ml[warp], fail);
    __syncthreads();
    if (warp < cols) {
      const float m = lane < kWarps ? s_ml[lane][warp][0] : -INFINITY;
      const float M = warp_max(m);
      const float f = m == -INFINITY ? 0.f : ex2(m - M);
      const float L = warp_sum(lane < kWarps ? f * s_ml[lane][warp][1] : 0.f);
      if (lane < kWarps) s_f[lane][warp] = f;
      if (lane == 0) s_tot[0][warp][0] = M, s_tot[0][warp][1] = L;
    }
    __syncthreads();
    const bool whole = start >= 0 && end == p.n;
    if (tid < cols * (D / 4)) {
      const int col = tid / (D / 4), pos = (tid - col * (D / 4)) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int w = 0; w < kWarps; ++w) {
        const float f = s_f[w][col];
        const float4 x = *reinterpret_cast<const float4*>(states + w * STATE + (col * OS + pos) * 4);
        v.x += f * x.x, v.y += f * x.y, v.z += f * x.z, v.w += f * x.w;
      }
      if (a.cluster > 1) {
        *reinterpret_cast<float4*>(s_part + col * D + pos) = v;
      } else if (whole) {
        store_row<D>(a, b, h, col, pos, v, s_tot[0][col]);
      } else {
        const int64_t at = (2 * static_cast<int64_t>(k) + (start > PAD ? 1 : 0)) * cols + col;
        *reinterpret_cast<float4*>(a.part_o + at * D + pos) = v;
        if (pos == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(s_tot[0][col][0], s_tot[0][col][1]);
      }
    }
    __syncthreads();
    if (!whole && !a.cluster) {
      const int unit = b * a.Hkv + h;
      if (start > PAD)
        open[1] = unit, open_u0[1] = w0 + start, open_n[1] = p.n;
      else
        open[0] = unit, open_u0[0] = w0 + start, open_n[0] = p.n;
    }
    start += p.n + PAD;
    if (++h == a.Hkv) {
      h = 0;
      if (start < share) p = request_span<NR>(a, ++b);
    }
  }
  if (fail) tile.drain();
  __syncwarp();

  // ---- cluster: every block sums its share of the unit's rows from all of them
  if (a.cluster > 1) {
    cluster_sync();
    const int C = a.cluster, unit = k / C, rank = k - unit * C;
    const int items = cols * (D / 4), each = (items + C - 1) / C;
    const int it = rank * each + tid;
    if (tid < each && it < items) {
      const int col = it / (D / 4), pos = (it - col * (D / 4)) * 4;
      float2 ml[8];
      float4 x[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        ml[r] = make_float2(-INFINITY, 0.f);
        x[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < C) {
          ml[r] = cluster_ld2(cluster_addr(smem_addr(&s_tot[0][col][0]), r));
          x[r] = cluster_ld4(cluster_addr(smem_addr(s_part + it * 4), r));
        }
      }
      float tot[2] = {-INFINITY, 0.f};
#pragma unroll
      for (int r = 0; r < 8; ++r) tot[0] = fmaxf(tot[0], ml[r].x);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const float f = ml[r].x == -INFINITY ? 0.f : ex2(ml[r].x - tot[0]);
        tot[1] += f * ml[r].y;
        v.x += f * x[r].x, v.y += f * x[r].y, v.z += f * x[r].z, v.w += f * x[r].w;
      }
      const int cb = unit / a.Hkv;
      store_row<D>(a, cb, unit - cb * a.Hkv, col, pos, v, tot);
    }
    __syncwarp();
    cluster_sync();  // the others may still read this block's sum
    return;
  }

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
  const int u = tid / kHalf;
  if (s_last[u])
    merge_unit<D, PAD>(a, cut, u ? open[1] : open[0], u ? open_u0[1] : open_u0[0], u ? open_n[1] : open_n[0], 1 + u,
                       tid - u * kHalf, merge + u * kMergeB, s_tot[u]);
}

// ------------------------------------------------------------------ host side
struct Plan {
  int max_blocks;  // a full wave
  size_t off_ml, off_o, total;
};

// Workspace: header, tickets, partials of every block's first and last unit.
inline Plan plan(int cols, int D) {
  Plan p;
  p.max_blocks = sm_count() < kMaxBlocks ? sm_count() : kMaxBlocks;
  const size_t slots = 2 * static_cast<size_t>(p.max_blocks) * cols;
  p.off_ml = kWsTickets;
  p.off_o = align_up(p.off_ml + slots * 2 * 4, 256);
  p.total = align_up(p.off_o + slots * D * 4, 256);
  return p;
}

inline void bind_workspace(Args& a, const Plan& p, void* ws) {
  char* w = static_cast<char*>(ws);
  a.flags = reinterpret_cast<uint32_t*>(w);
  a.tickets = reinterpret_cast<uint32_t*>(w + sizeof(WsHeader));
  a.part_ml = reinterpret_cast<float*>(w + p.off_ml);
  a.part_o = reinterpret_cast<float*>(w + p.off_o);
}

// Blocks of a call whose requests have up to L tokens, and whether the blocks
// of a unit form a cluster.
//
// Axis: blocks for the most stages that the requests can have; the kernel
// leaves out those that the real lengths do not fill.
// Cluster: C = 1, 2, 4 or 8 blocks per unit, all of them resident at once
// (active: clusters of C that the device holds) and with a stage for every
// warp.  Its fixed cost is lower by about what `gain` stages of a block take;
// it is chosen when sharing the units out unevenly costs less.  Measured on
// B200 in the 4-bit draft (D = 128, us of device time per call, axis against
// cluster): 8 units of 2K tokens 14.5 : 8.2, of 16K 14.4 : 13.7; 32 units,
// window 4096, g = 8 15.4 : 12.0; 64 units of 4K 18.5 : 14.0; 128 units of 1K
// 16.3 : 8.8.  Longer contexts take the axis (64 units of 32K: 61).
template <class Active>
int choose(Args& a, const Plan& p, uint32_t L, int NR, int pad, int least, int gain, const Active& active) {
  const Span sp = make_span(L, a.nq, a.window, a.n_sink, NR);
  const int64_t units = static_cast<int64_t>(a.B) * a.Hkv;
  const int64_t even = units * (sp.n + pad) / p.max_blocks;  // an axis block's stages
  for (int C = 8; C >= 1; C /= 2) {
    if (units * C > p.max_blocks || (C > 1 && sp.n <= kWarps * (C / 2))) continue;
    if ((sp.n + C - 1) / C > even + gain) break;
    if (C > 1 && units > active(C)) continue;
    a.cluster = C;
    return static_cast<int>(units * C);
  }
  a.cluster = 0;
  const int64_t n = ((static_cast<int64_t>(sp.n) + 1 + pad) * units + least - 1) / least;
  return static_cast<int>(n < p.max_blocks ? n : p.max_blocks);
}

// One kernel's launches: programmatic dependents, one block per SM.  Its
// attribute and its cluster capacities are looked up once per device.
template <class Params>
struct Launcher {
  void (*kernel)(Params);
  int smem;
  Launcher(void (*k)(Params), int bytes) : kernel(k), smem(bytes) {}
  struct Device {
    int active[4];  // clusters of 1, 2, 4, 8 blocks that the device holds
  };
  PerDevice<Device> devices;

  void fill(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, int n, int cluster, cudaStream_t s) const {
    cfg.gridDim = dim3(static_cast<unsigned>(n));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster > 0 ? cluster : 1;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
  const Device& device() {
    int d = 0;
    if (cudaGetDevice(&d) != cudaSuccess) d = 0;
    return devices.get(d, [&](Device& dev) {
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      for (int i = 0, C = 1; i < 4; ++i, C *= 2) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[2];
        fill(cfg, attr, C, C, nullptr);
        attr[0] = attr[1];
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
          cudaGetLastError();
          n = 0;
        }
        dev.active[i] = n;
      }
    });
  }
  int active(int C) { return device().active[C == 8 ? 3 : C == 4 ? 2 : C == 2 ? 1 : 0]; }
  void launch(const Params& a, int n, int cluster, cudaStream_t s) {
    device();
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    fill(cfg, attr, n, cluster, s);
    cudaLaunchKernelEx(&cfg, kernel, a);
  }
};

}  // namespace stream
}  // namespace vc

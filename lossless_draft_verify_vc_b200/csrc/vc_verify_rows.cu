// vc_verify_rows.cu -- windowed verification (vc_verify_attn_window) of at
// most 8 query rows per (request, KV head): single-token decoding and short
// blocks.  A tcgen05 tile would carry 4 to 8 live rows of 128 and its set-up,
// so these calls take the split of vc_stream.cuh instead, with K and V read
// straight into the fragments of mma.sync m16n8k16 (bf16 x bf16 -> fp32):
//   scores  S[token][col] = K[token][chan] x q[chan][col]
//   values  O[chan][col] += V^T[chan][token] x P[token][col]
// A lane reads runs of a row -- a quarter of a key row, an eighth of a value
// row -- and contractions take their channels in that order; value pairs of
// neighbouring tokens are put together with byte permutes.  P is split into
// three bf16 parts, which hold all 24 bits of a weight.  The next stage's keys
// are requested as soon as a stage's scores are done, its values after the
// products, so a warp always has loads in flight.
//
// Bound by HBM for long contexts and by the chain of a block (launch, loads,
// merge) for short ones.  Measured on B200, us of device time per call, the
// tcgen05 form against this one: 1 row, g = 4, 8 KV heads, window 1024 10.4 :
// 7.2, window 8192 16.0 : 13.6, 8 requests with window 4096 33.1 : 27.8; 16
// requests with window 512 16.5 : 10.0; 2 rows, 2 KV heads, window 4096 10.5 :
// 10.5; but one KV head of 200K keys 31.2 : 34.0 (148 partials of one unit,
// merged by half a block), which keeps this form for its exact weights.
#include <algorithm>

#include "vc_stream.cuh"
#include "vc_verify_rows.h"

namespace vc {
namespace {

using stream::Span;

struct RArgs {
  stream::Args s;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t T;  // rows allocated per KV head
  float scale_log2;
};

// 32 or 16 bytes of a row, zeros unless `live`; 32 in one access when the
// rows are 32-byte aligned.
__device__ __forceinline__ void load_16(uint32_t* w, const void* p, bool live) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}\n"
      : "=&r"(w[0]), "=&r"(w[1]), "=&r"(w[2]), "=&r"(w[3])
      : "l"(p), "r"(static_cast<uint32_t>(live)));
}
__device__ __forceinline__ void load_32(uint32_t* w, const void* p, bool live, bool wide) {
  if (wide) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %9, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "mov.b32 %4, 0;\n\tmov.b32 %5, 0;\n\tmov.b32 %6, 0;\n\tmov.b32 %7, 0;\n\t"
        "@p ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t}\n"
        : "=&r"(w[0]), "=&r"(w[1]), "=&r"(w[2]), "=&r"(w[3]), "=&r"(w[4]), "=&r"(w[5]), "=&r"(w[6]), "=&r"(w[7])
        : "l"(p), "r"(static_cast<uint32_t>(live)));
  } else {
    load_16(w, p, live);
    load_16(w + 4, static_cast<const char*>(p) + 16, live);
  }
}

template <int D_>
struct RTile {
  static constexpr int D = D_;
  static constexpr int NR = 1;  // records of 16 tokens per stage
  static constexpr int COLS = 8;
  // every warp's query fragments, in the order its lanes read them
  static constexpr int Q_OFF = stream::kWarps * stream::State<D>::bytes(COLS);
  static constexpr int SMEM_B = Q_OFF + stream::kWarps * (D / 32) * 512;
  static_assert(2 * stream::kMergeB <= SMEM_B, "the final merges' buffers take this place");
  // a unit's begin in stages (8 KB, D = 128) and the least share, as in the
  // 4-bit draft; measured at D = 128, used for D = 64 too
  static constexpr int PAD = 8;
  static constexpr int MIN = 24;
  static constexpr int GAIN = 64;
  static constexpr int KT = D / 16;
  static constexpr int KW = D / 8;   // words of a lane's key run (D / 4 channels)
  static constexpr int VW = D / 16;  // words of a lane's value run (D / 8 channels)

  const RArgs& a;
  const int warp, lane, row, i4;
  const bool wide;
  const __nv_bfloat16 *kp, *vp;  // the unit's rows, at the lane's run
  uint4* qs;
  uint32_t kw[2][KW], vw[4][VW];
  float m0, m1, l0, l1;
  float acc[KT][4];

  __device__ __forceinline__ RTile(const RArgs& a_, unsigned char* smem)
      : a(a_),
        warp(threadIdx.x >> 5),
        lane(threadIdx.x & 31),
        row(lane >> 2),
        i4(lane & 3),
        wide(((reinterpret_cast<uintptr_t>(a_.k) | reinterpret_cast<uintptr_t>(a_.v)) & 31) == 0),
        qs(reinterpret_cast<uint4*>(smem + Q_OFF) + warp * (D / 32) * 32 + lane) {}

  // query words of this lane: its tile column's row and head, D / 4 channels from i4 * D / 4
  __device__ __forceinline__ void query(int b, int h) {
    const int i = row / a.s.g, head = row - i * a.s.g;
    const uint4* src = reinterpret_cast<const uint4*>(
        a.q + ((static_cast<int64_t>(b) * a.s.nq + i) * a.s.Hq + h * a.s.g + head) * D + i4 * (D / 4));
#pragma unroll
    for (int x = 0; x < D / 32; ++x) {
      qs[32 * x] = i < a.s.nq ? stream::load_16(src + x) : make_uint4(0, 0, 0, 0);  // read by this lane alone
    }
  }

  __device__ __forceinline__ void begin(int, int, int, int) {}

  // Tokens past the request's length are not read: zeros.
  __device__ __forceinline__ void load_k(const Span& p, int x) {
    const uint32_t t = static_cast<uint32_t>(stream::stage_record<NR>(p, x)) * stream::kTok + row;
    const __nv_bfloat16* src = kp + static_cast<int64_t>(t) * D;
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int w = 0; w < KW; w += 8) load_32(kw[y] + w, src + 8 * y * D + 2 * w, t + 8 * y < p.L, wide);
  }
  __device__ __forceinline__ void load_v(const Span& p, int x) {
    const uint32_t t = static_cast<uint32_t>(stream::stage_record<NR>(p, x)) * stream::kTok + 2 * i4;
    const __nv_bfloat16* src = vp + static_cast<int64_t>(t) * D;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int o = (y & 1) + 8 * (y >> 1);
      if constexpr (VW == 8)
        load_32(vw[y], src + o * D, t + o < p.L, wide);
      else
        load_16(vw[y], src + o * D, t + o < p.L);
    }
  }

  __device__ __forceinline__ void unit(const Span& p, int b, int h, int x, int end) {
    const int64_t at = (static_cast<int64_t>(b) * a.s.Hkv + h) * a.T * D;
    kp = a.k + at + i4 * (D / 4);
    vp = a.v + at + row * (D / 8);
    if (x < end) {
      load_k(p, x);
      load_v(p, x);
    }
#pragma unroll
    for (int y = 0; y < KT; ++y) acc[y][0] = acc[y][1] = acc[y][2] = acc[y][3] = 0.f;
    m0 = m1 = stream::kNone;
    l0 = l1 = 0.f;
  }

  __device__ __forceinline__ bool stage(const Span& p, int x, int end) {
    const bool full = x >= p.f0 && x < p.f1;
    const uint32_t t0 = static_cast<uint32_t>(stream::stage_record<NR>(p, x)) * stream::kTok;
    // ---- scores
    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < KT; s += 2) {
      const uint4 qw = qs[16 * s];
      const uint32_t f0[4] = {kw[0][2 * s], kw[1][2 * s], kw[0][2 * s + 1], kw[1][2 * s + 1]};
      const uint32_t f1[4] = {kw[0][2 * s + 2], kw[1][2 * s + 2], kw[0][2 * s + 3], kw[1][2 * s + 3]};
      mma_bf16(c, f0, qw.x, qw.y);
      mma_bf16(c, f1, qw.z, qw.w);
    }
    if (x + stream::kWarps < end) load_k(p, x + stream::kWarps);
    if (!full) {
      const int r0 = 2 * i4 / a.s.g, r1 = (2 * i4 + 1) / a.s.g;  // rows of the lane's columns
      const uint32_t t = t0 + row;
      if (!stream::row_sees(a.s, p, r0, t)) c[0] = -INFINITY;
      if (!stream::row_sees(a.s, p, r1, t)) c[1] = -INFINITY;
      if (!stream::row_sees(a.s, p, r0, t + 8)) c[2] = -INFINITY;
      if (!stream::row_sees(a.s, p, r1, t + 8)) c[3] = -INFINITY;
      // values that no row sees may hold anything
#pragma unroll
      for (int y = 0; y < 4; ++y)
        if (!stream::seen(a.s, p, t0 + 2 * i4 + (y & 1) + 8 * (y >> 1)))
#pragma unroll
          for (int w = 0; w < VW; ++w) vw[y][w] = 0;
    }
    // ---- online softmax; m moves only when a score exceeds it by more than
    //      15 (base 2), by whole units, so that rescales are powers of two
    const float sc = a.scale_log2;
    float x0 = fmaxf(c[0], c[2]) * sc, x1 = fmaxf(c[1], c[3]) * sc;
    if (__any_sync(0xffffffffu, x0 - m0 > 15.f || x1 - m1 > 15.f)) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        x0 = warp_max_xor(x0, d);
        x1 = warp_max_xor(x1, d);
      }
      const float n0 = fmaxf(m0, ceilf(x0)), n1 = fmaxf(m1, ceilf(x1));
      const float al0 = ex2(m0 - n0), al1 = ex2(m1 - n1);
      m0 = n0, m1 = n1;
      l0 *= al0, l1 *= al1;
#pragma unroll
      for (int y = 0; y < KT; ++y) acc[y][0] *= al0, acc[y][2] *= al0, acc[y][1] *= al1, acc[y][3] *= al1;
    }
    // ---- P = h + m + l, each the next 8 bits of a weight, as value operands
    uint32_t pf[3][2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      float q0 = ex2(fmaf(c[2 * y], sc, -m0)), q1 = ex2(fmaf(c[2 * y + 1], sc, -m1));
      l0 += q0;
      l1 += q1;
#pragma unroll
      for (int z = 0; z < 3; ++z) {
        const uint32_t b0 = __float_as_uint(q0) & 0xffff0000u, b1 = __float_as_uint(q1) & 0xffff0000u;
        pf[z][y] = stream::movm_t(prmt(b0, b1, 0x7632));
        q0 -= __uint_as_float(b0);
        q1 -= __uint_as_float(b1);
      }
    }
    // ---- values
#pragma unroll
    for (int s = 0; s < KT; ++s) {
      const uint32_t f[4] = {prmt(vw[0][s], vw[1][s], 0x5410), prmt(vw[0][s], vw[1][s], 0x7632),
                             prmt(vw[2][s], vw[3][s], 0x5410), prmt(vw[2][s], vw[3][s], 0x7632)};
#pragma unroll
      for (int z = 0; z < 3; ++z) mma_bf16(acc[s], f, pf[z][0], pf[z][1]);
    }
    if (x + stream::kWarps < end) load_v(p, x + stream::kWarps);
    return true;
  }

  __device__ __forceinline__ void finish(float* o, float (*ml)[2], bool) {
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    constexpr int OS = stream::State<D>::OS;
    o += 2 * i4 * OS + row * 2;
#pragma unroll
    for (int x = 0; x < KT; ++x) {
      *reinterpret_cast<float2*>(o + x * 16) = make_float2(acc[x][0], acc[x][2]);
      *reinterpret_cast<float2*>(o + OS + x * 16) = make_float2(acc[x][1], acc[x][3]);
    }
    if (row == 0) {
      ml[2 * i4][0] = m0 == stream::kNone ? -INFINITY : m0, ml[2 * i4][1] = l0;
      ml[2 * i4 + 1][0] = m1 == stream::kNone ? -INFINITY : m1, ml[2 * i4 + 1][1] = l1;
    }
  }

  __device__ __forceinline__ void drain() {}
};

template <int D>
__global__ void __launch_bounds__(stream::kThreads, 1) verify_rows_kernel(RArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  RTile<D> tile(a, smem);
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  stream::run(a.s, tile, smem, smem);
}

template <int D>
void launch_rows(RArgs& a, const stream::Plan& p, cudaStream_t s) {
  using Tile = RTile<D>;
  static stream::Launcher<RArgs> k(verify_rows_kernel<D>, Tile::SMEM_B);
  const int n = stream::choose(a.s, p, static_cast<uint32_t>(a.T), Tile::NR, Tile::PAD, Tile::MIN, Tile::GAIN,
                               [&](int C) { return k.active(C); });
  k.launch(a, n, a.s.cluster, s);
}

}  // namespace

size_t verify_rows_workspace(const vc_attn_shape& sh, int nq) {
  return stream::plan(nq * (sh.Hq / sh.Hkv), sh.D).total;
}

vc_status verify_rows_launch(const vc_attn_shape& sh, const void* q, const void* k, const void* v, int64_t T,
                             const int32_t* lens, int nq, int64_t window, int64_t n_sink, float* out, float* lse,
                             void* ws, void* stream_) {
  const int g = sh.Hq / sh.Hkv;
  const stream::Plan p = stream::plan(nq * g, sh.D);
  RArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.T = T;
  const float sm = sh.sm_scale > 0.f ? sh.sm_scale : 1.0f / sqrtf(static_cast<float>(sh.D));
  a.scale_log2 = std::max(sm * 1.4426950408889634f, 1e-37f);  // (-inf times it stays -inf)
  a.s.out = out;
  a.s.lse = lse;
  a.s.lens = lens;
  a.s.T_cap = T;
  a.s.T = static_cast<uint32_t>(T);
  // a window as long as the cache hides nothing; no position reaches 2^31 - 1
  a.s.window = window >= T ? 0u : static_cast<uint32_t>(window);
  a.s.n_sink = static_cast<uint32_t>(std::min<int64_t>(n_sink, INT32_MAX));
  a.s.B = sh.B;
  a.s.Hq = sh.Hq;
  a.s.Hkv = sh.Hkv;
  a.s.g = g;
  a.s.nq = nq;
  stream::bind_workspace(a.s, p, ws);
  cudaStream_t s = static_cast<cudaStream_t>(stream_);
  if (sh.D == 128)
    launch_rows<128>(a, p, s);
  else
    launch_rows<64>(a, p, s);
  return launch_status("vc_verify_attn_window");
}

}  // namespace vc

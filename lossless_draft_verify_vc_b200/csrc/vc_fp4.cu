// vc_fp4.cu -- the 4-bit floating-point draft cache: rows quantised as they
// are written, and read back (format and layout: vc_fp4.cuh).
//
// A drafted token's key and value rows have to enter the compressed cache
// before the next draft step ("VeriCache: Turning Lossy KV Cache into
// Lossless LLM Inference", menfem.com, "Key Contributions": drafting decodes
// one token at a time from the compressed cache); the pages give no format.
#include <algorithm>

#include "vc_fp4.cuh"

namespace vc {
namespace {

__device__ __forceinline__ bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; }

// Where request b's rows go: false (and a flag) when they do not fit.
__device__ __forceinline__ bool fp4_span(const int32_t* pos, int64_t pos0, const int32_t* counts, int b, int64_t n,
                                         int64_t T_cap, uint32_t* flags, bool report, int64_t& p, int64_t& c) {
  p = pos ? static_cast<int64_t>(__ldcg(pos + b)) : pos0;
  c = counts ? static_cast<int64_t>(__ldcg(counts + b)) : n;
  if (p >= 0 && c >= 0 && c <= n && p + c <= T_cap) return true;
  if (report) atomicOr(flags, VC_FLAG_BAD_LENGTH);
  return false;
}

// Loads in this file avoid the read-only path: a programmatic dependent is
// resident while the call before it still writes what it will read.
//
// 32 bytes of a row: one access (whole sectors) when the rows are 32-byte
// aligned (`wide`), else two of 16.
struct W8 {
  uint32_t w[8];
};
__device__ __forceinline__ W8 load32(const void* p, bool wide) {
  W8 x;
  if (wide) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
                 : "=r"(x.w[0]), "=r"(x.w[1]), "=r"(x.w[2]), "=r"(x.w[3]), "=r"(x.w[4]), "=r"(x.w[5]), "=r"(x.w[6]),
                   "=r"(x.w[7])
                 : "l"(p));
  } else {
    const uint4 a = __ldcg(static_cast<const uint4*>(p)), b = __ldcg(static_cast<const uint4*>(p) + 1);
    x.w[0] = a.x, x.w[1] = a.y, x.w[2] = a.z, x.w[3] = a.w;
    x.w[4] = b.x, x.w[5] = b.y, x.w[6] = b.z, x.w[7] = b.w;
  }
  return x;
}
__device__ __forceinline__ void store32(void* p, const uint32_t* w, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (std::is_same<T, __half>::value)
    return unpack_h2(w);
  else
    return unpack_bf2(w);
}

// max(|a|, |b|) of both halves, NaN if one is NaN.
template <typename T>
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
  const T2 m = __hmax2_nan(__habs2(*reinterpret_cast<T2*>(&a)), __habs2(*reinterpret_cast<T2*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// Values of NW words and their largest |x| * down.  Patterns of |x| are
// ordered as integers, NaN above infinity above the rest; a run with NaN (0
// instead) or values past the scales' range (clamped to it) is flagged.
template <typename T, int NW>
__device__ __forceinline__ float take(const uint32_t* w, float (&x)[2 * NW], float down, bool& odd) {
  uint32_t m = w[0];
#pragma unroll
  for (int i = 1; i < NW; ++i) m = max_abs2<T>(m, w[i]);
  m = max(m & 0xffffu, m >> 16);
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    const float2 f = unpack2<T>(w[i]);
    x[2 * i] = f.x, x[2 * i + 1] = f.y;
  }
  float amax = unpack2<T>(m).x * down;
  if (!(amax <= fp4::kMaxAbs)) {
    odd = true;
    amax = 0.f;
    const float lim = fp4::kMaxAbs / down;
#pragma unroll
    for (int i = 0; i < 2 * NW; ++i) {
      x[i] = x[i] != x[i] ? 0.f : fminf(fmaxf(x[i], -lim), lim);
      amax = fmaxf(amax, fabsf(x[i]));
    }
    amax *= down;
  }
  return amax;
}

constexpr int kRowWarps = 4;  // warps per block of the two kernels below

// The tokens of a warp, half a record (tokens 8 half .. 8 half + 7): token t
// of the half is row row0 + t of the call if t0 <= t < t1.
constexpr int kHalfTok = fp4::kTok / 2;
struct HalfRows {
  int64_t row0;
  int t0, t1, half;
};

__device__ __forceinline__ HalfRows half_rows(int64_t hr, int64_t p, int64_t c) {
  HalfRows r;
  r.row0 = hr * kHalfTok - p;
  r.t0 = r.row0 < 0 ? static_cast<int>(-r.row0) : 0;
  r.t1 = static_cast<int>(min(static_cast<int64_t>(kHalfTok), c - r.row0));
  r.half = static_cast<int>(hr & 1);
  return r;
}

// Rows into the cache, one warp per half record at a time.  A lane takes the
// runs of the rows whose codes are contiguous in the record (the draft
// kernel's order): of K, token lane / 4, a quarter of the channels; of V,
// two tokens and an eighth of the channels (8 channels, D = 64: two lanes
// share a block of 16).  Bytes of tokens that the call does not write stay.
//
// Bound by HBM (4 D bytes in, 18 D / 16 out per token).
template <int D, typename T>
__global__ void __launch_bounds__(kRowWarps * 32) fp4_write_kernel(
    uint8_t* __restrict__ records, int64_t T_cap, const T* __restrict__ k, const T* __restrict__ v, int64_t n,
    const int32_t* __restrict__ pos, int64_t pos0, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ k_exp, const int32_t* __restrict__ v_exp, int Hkv, uint32_t* flags) {
  using R = fp4::Rec<D>;
  constexpr int KB = D / 64;  // 16-channel blocks of a lane's K run
  constexpr int VW = D / 16;  // words of a lane's V run (16 or 8 channels)
  const int unit = blockIdx.y, lane = threadIdx.x & 31;
  const int b = unit / Hkv, h = unit - b * Hkv;
  // (in this order: the next call's blocks may be scheduled as this grid's
  // retire, but not while the grid before it still writes)
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const float kdown = two_to(k_exp, h, -1), vdown = two_to(v_exp, h, -1);
  int64_t p, c;
  if (!fp4_span(pos, pos0, counts, b, n, T_cap, flags, threadIdx.x == 0, p, c) || c == 0) return;
  const bool kwide = aligned32(k), vwide = aligned32(v);
  const int64_t last = (p + c - 1) / kHalfTok;
  const int kt = lane >> 2, vt = 2 * (lane & 3);
  bool odd = false;
#pragma unroll 1
  for (int64_t hr = p / kHalfTok + blockIdx.x * kRowWarps + threadIdx.x / 32; hr <= last;
       hr += static_cast<int64_t>(gridDim.x) * kRowWarps) {
    const HalfRows rr = half_rows(hr, p, c);
    const int64_t base = (static_cast<int64_t>(unit) * n + rr.row0) * D;
    uint8_t* dst = records + (static_cast<int64_t>(unit) * (T_cap / fp4::kTok) + hr / 2) * R::BYTES;
    const bool klive = kt >= rr.t0 && kt < rr.t1;
    W8 kw[KB];
    uint32_t vw[2][VW];
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      kw[j] = W8{};
      if (klive) kw[j] = load32(k + base + kt * D + (lane & 3) * (16 * KB) + 16 * j, kwide);
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int j = 0; j < VW; ++j) vw[x][j] = 0;
      if (vt + x >= rr.t0 && vt + x < rr.t1) {
        const T* src = v + base + (vt + x) * D + (lane >> 2) * (D / 8);
        if constexpr (D == 128) {
          const W8 w = load32(src, vwide);
#pragma unroll
          for (int j = 0; j < 8; ++j) vw[x][j] = w.w[j];
        } else {
          const uint4 w = __ldcg(reinterpret_cast<const uint4*>(src));
          vw[x][0] = w.x, vw[x][1] = w.y, vw[x][2] = w.z, vw[x][3] = w.w;
        }
      }
    }
    // ---- K
    uint32_t kc[2 * KB], ks = 0;
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      float f[16];
      uint32_t cd[2];
      const float amax = take<T, 8>(kw[j].w, f, kdown, odd);
      const uint8_t s8 = fp4::block_scale(amax);
      fp4::quantise_codes<16>(f, s8, kdown, cd);
      kc[2 * j] = cd[0], kc[2 * j + 1] = cd[1];
      ks |= static_cast<uint32_t>(s8) << (8 * j);
    }
    if (klive) {
      uint8_t* at = dst + rr.half * (kHalfTok * D / 2) + lane * (8 * KB);
      uint8_t* sc = dst + R::KS + lane * (2 * KB) + rr.half * KB;
      if constexpr (KB == 2) {
        *reinterpret_cast<uint4*>(at) = make_uint4(kc[0], kc[1], kc[2], kc[3]);
        *reinterpret_cast<uint16_t*>(sc) = static_cast<uint16_t>(ks);
      } else {
        *reinterpret_cast<uint2*>(at) = make_uint2(kc[0], kc[1]);
        *sc = static_cast<uint8_t>(ks);
      }
    }
    // ---- V
    uint32_t vc[2][VW / 4], vs = 0;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float f[2 * VW];
      float amax = take<T, VW>(vw[x], f, vdown, odd);
      if constexpr (D == 64) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
      const uint8_t s8 = fp4::block_scale(amax);
      fp4::quantise_codes<2 * VW>(f, s8, vdown, vc[x]);
      vs |= static_cast<uint32_t>(s8) << (8 * x);
    }
    uint8_t* at = dst + R::V + lane * 16 + rr.half * (D == 128 ? 512 : 8);
    uint8_t* sc = dst + R::VS + (D == 128 ? lane * 4 : (lane >> 3) * 16 + (lane & 3) * 4) + rr.half * 2;
    const bool put = D == 128 || (lane & 4) == 0;  // of the two lanes that share a scale
    if (vt >= rr.t0 && vt + 1 < rr.t1) {
      if constexpr (D == 128)
        *reinterpret_cast<uint4*>(at) = make_uint4(vc[0][0], vc[0][1], vc[1][0], vc[1][1]);
      else
        *reinterpret_cast<uint2*>(at) = make_uint2(vc[0][0], vc[1][0]);
      if (put) *reinterpret_cast<uint16_t*>(sc) = static_cast<uint16_t>(vs);
    } else {
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (vt + x >= rr.t0 && vt + x < rr.t1) {
          if constexpr (D == 128)
            *reinterpret_cast<uint2*>(at + x * 8) = make_uint2(vc[x][0], vc[x][1]);
          else
            *reinterpret_cast<uint32_t*>(at + x * 4) = vc[x][0];
          if (put) sc[x] = static_cast<uint8_t>(vs >> (8 * x));
        }
    }
  }
  if (odd) atomicOr(flags, VC_FLAG_RANGE);
}

// N values (codes of N / 8 words times `up`) to dst.
template <int N, typename T>
__device__ __forceinline__ void put_values(T* dst, const uint32_t* codes, float up, bool wide) {
  float x[N];
#pragma unroll
  for (int m = 0; m < N / 8; ++m) {
    uint32_t o[4];
    fp4::codes_to_h2(codes[m], o);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 f = unpack_h2(o[q]);
      x[8 * m + 2 * q] = f.x * up;
      x[8 * m + 2 * q + 1] = f.y * up;
    }
  }
  if constexpr (std::is_same<T, float>::value) {
#pragma unroll
    for (int i = 0; i < N; i += 8) store32(dst + i, reinterpret_cast<const uint32_t*>(x + i), wide);
  } else {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      w[i] = std::is_same<T, __half>::value ? pack_h2(x[2 * i], x[2 * i + 1]) : pack_bf2(x[2 * i], x[2 * i + 1]);
    if constexpr (N == 16)
      store32(dst, w, wide);
    else
      *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The way back, in the same order.  Bound by HBM.
template <int D, typename T>
__global__ void __launch_bounds__(kRowWarps * 32) fp4_read_kernel(
    const uint8_t* __restrict__ records, int64_t T_cap, T* __restrict__ k, T* __restrict__ v, int64_t n,
    const int32_t* __restrict__ pos, int64_t pos0, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ k_exp, const int32_t* __restrict__ v_exp, int Hkv, uint32_t* flags) {
  using R = fp4::Rec<D>;
  constexpr int KB = D / 64;
  constexpr int VN = D / 8;  // channels of a lane's V run
  const int unit = blockIdx.y, lane = threadIdx.x & 31;
  const int b = unit / Hkv, h = unit - b * Hkv;
  // (in this order: the next call's blocks may be scheduled as this grid's
  // retire, but not while the grid before it still writes)
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const float kup = two_to(k_exp, h, 1), vup = two_to(v_exp, h, 1);
  int64_t p, c;
  if (!fp4_span(pos, pos0, counts, b, n, T_cap, flags, threadIdx.x == 0, p, c) || c == 0) return;
  const bool kwide = aligned32(k), vwide = aligned32(v);
  const int64_t last = (p + c - 1) / kHalfTok;
  const int kt = lane >> 2, vt = 2 * (lane & 3);
#pragma unroll 1
  for (int64_t hr = p / kHalfTok + blockIdx.x * kRowWarps + threadIdx.x / 32; hr <= last;
       hr += static_cast<int64_t>(gridDim.x) * kRowWarps) {
    const HalfRows rr = half_rows(hr, p, c);
    const int64_t base = (static_cast<int64_t>(unit) * n + rr.row0) * D;
    const uint8_t* src = records + (static_cast<int64_t>(unit) * (T_cap / fp4::kTok) + hr / 2) * R::BYTES;
    uint32_t kc[2 * KB], vc[2][VN / 8];
    const uint8_t* kat = src + rr.half * (kHalfTok * D / 2) + lane * (8 * KB);
    const uint8_t* vat = src + R::V + lane * 16 + rr.half * (D == 128 ? 512 : 8);
    const uint8_t* ksat = src + R::KS + lane * (2 * KB) + rr.half * KB;
    const uint32_t vs = __ldcg(reinterpret_cast<const uint16_t*>(
        src + R::VS + (D == 128 ? lane * 4 : (lane >> 3) * 16 + (lane & 3) * 4) + rr.half * 2));
    uint32_t ks;
    if constexpr (D == 128) {
      const uint4 a = __ldcg(reinterpret_cast<const uint4*>(kat)), e = __ldcg(reinterpret_cast<const uint4*>(vat));
      ks = __ldcg(reinterpret_cast<const uint16_t*>(ksat));
      kc[0] = a.x, kc[1] = a.y, kc[2] = a.z, kc[3] = a.w;
      vc[0][0] = e.x, vc[0][1] = e.y, vc[1][0] = e.z, vc[1][1] = e.w;
    } else {
      const uint2 a = __ldcg(reinterpret_cast<const uint2*>(kat)), e = __ldcg(reinterpret_cast<const uint2*>(vat));
      ks = __ldcg(ksat);
      kc[0] = a.x, kc[1] = a.y;
      vc[0][0] = e.x, vc[1][0] = e.y;
    }
    if (kt >= rr.t0 && kt < rr.t1)
#pragma unroll
      for (int j = 0; j < KB; ++j)
        put_values<16>(k + base + kt * D + (lane & 3) * (16 * KB) + 16 * j, kc + 2 * j,
                       fp4::scale_to_float(static_cast<uint8_t>(ks >> (8 * j))) * kup, kwide);
#pragma unroll
    for (int x = 0; x < 2; ++x)
      if (vt + x >= rr.t0 && vt + x < rr.t1)
        put_values<VN>(v + base + (vt + x) * D + (lane >> 2) * VN, vc[x],
                       fp4::scale_to_float(static_cast<uint8_t>(vs >> (8 * x))) * vup, vwide);
  }
}

vc_status check_rows(const vc_attn_shape* shape, const vc_fp4_cache* cache, const void* k, const void* v, int dtype,
                     bool f32_ok, int64_t n, const int32_t* pos, int64_t pos0, const void* ws, size_t ws_bytes,
                     const char* who) {
  VC_REQUIRE(shape && cache, "%s: null shape or cache", who);
  VC_REQUIRE(shape->B >= 1 && shape->Hkv >= 1 && static_cast<int64_t>(shape->B) * shape->Hkv <= 65535,
             "%s: need 1 <= B * Hkv <= 65535", who);
  VC_REQUIRE(shape->D == 64 || shape->D == 128, "%s: head dim must be 64 or 128 (got %d)", who, shape->D);
  VC_REQUIRE(cache->T_cap >= fp4::kTok && cache->T_cap % fp4::kTok == 0 && cache->T_cap < (int64_t(1) << 31),
             "%s: T_cap must be a multiple of 16 in [16, 2^31) (got %lld)", who, static_cast<long long>(cache->T_cap));
  VC_REQUIRE(dtype == VC_BF16 || dtype == VC_F16 || (f32_ok && dtype == VC_F32), "%s: unsupported dtype %d", who,
             dtype);
  VC_REQUIRE(n >= 0 && n < (int64_t(1) << 31), "%s: need 0 <= n < 2^31 (got %lld)", who, static_cast<long long>(n));
  VC_REQUIRE(pos || (pos0 >= 0 && pos0 <= cache->T_cap), "%s: pos0 outside [0, T_cap]", who);
  VC_REQUIRE(cache->records && ws, "%s: null records or workspace", who);
  VC_REQUIRE(n == 0 || (k && v), "%s: null k or v", who);
  VC_REQUIRE(aligned16(cache->records) && aligned16(k) && aligned16(v) && aligned16(ws),
             "%s: records, k, v and workspace must be 16-byte aligned", who);
  VC_REQUIRE(ws_bytes >= vc_compress_workspace_size(), "%s: workspace too small", who);
  return VC_OK;
}

// Blocks per (request, KV head): a warp for each half record that n rows can
// touch, at most about 8 waves of the card.
unsigned row_blocks(int64_t n, int64_t units) {
  const int64_t halves = (n + kHalfTok - 2) / kHalfTok + 1;
  const int64_t want = (halves + kRowWarps - 1) / kRowWarps;
  const int64_t most = std::max<int64_t>(1, static_cast<int64_t>(sm_count()) * 8 * 16 / units);
  return static_cast<unsigned>(std::min(want, most));
}

// Launch as a programmatic dependent.
template <class... Params, class... Args>
void launch_rows(void (*kernel)(Params...), dim3 grid, void* stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kRowWarps * 32);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

}  // namespace
}  // namespace vc

extern "C" {

vc_status vc_fp4_cache_write(const vc_attn_shape* shape, const vc_fp4_cache* cache, const void* k, const void* v,
                             int dtype, int64_t n, const int32_t* pos, int64_t pos0, const int32_t* counts, void* ws,
                             size_t ws_bytes, void* stream) {
  vc_status st = vc::check_rows(shape, cache, k, v, dtype, false, n, pos, pos0, ws, ws_bytes, "vc_fp4_cache_write");
  if (st != VC_OK) return st;
  if (n == 0) {
    vc::clear_error();
    return VC_OK;
  }
  const int units = shape->B * shape->Hkv;
  const dim3 grid(vc::row_blocks(n, units), units);
  auto go = [&](auto DD, auto tag) {
    using T = decltype(tag);
    vc::launch_rows(vc::fp4_write_kernel<decltype(DD)::value, T>, grid, stream,
        static_cast<uint8_t*>(cache->records), cache->T_cap, static_cast<const T*>(k), static_cast<const T*>(v), n,
        pos, pos0, counts, cache->k_exp, cache->v_exp, shape->Hkv, static_cast<uint32_t*>(ws));
  };
  auto by_type = [&](auto DD) { dtype == VC_F16 ? go(DD, __half{}) : go(DD, __nv_bfloat16{}); };
  if (shape->D == 128)
    by_type(std::integral_constant<int, 128>{});
  else
    by_type(std::integral_constant<int, 64>{});
  return vc::launch_status("vc_fp4_cache_write");
}

vc_status vc_fp4_cache_read(const vc_attn_shape* shape, const vc_fp4_cache* cache, void* k_out, void* v_out, int dtype,
                            int64_t n, const int32_t* pos, int64_t pos0, const int32_t* counts, void* ws,
                            size_t ws_bytes, void* stream) {
  vc_status st =
      vc::check_rows(shape, cache, k_out, v_out, dtype, true, n, pos, pos0, ws, ws_bytes, "vc_fp4_cache_read");
  if (st != VC_OK) return st;
  if (n == 0) {
    vc::clear_error();
    return VC_OK;
  }
  const int units = shape->B * shape->Hkv;
  const dim3 grid(vc::row_blocks(n, units), units);
  auto go = [&](auto DD, auto tag) {
    using T = decltype(tag);
    vc::launch_rows(vc::fp4_read_kernel<decltype(DD)::value, T>, grid, stream,
        static_cast<const uint8_t*>(cache->records), cache->T_cap, static_cast<T*>(k_out), static_cast<T*>(v_out), n,
        pos, pos0, counts, cache->k_exp, cache->v_exp, shape->Hkv, static_cast<uint32_t*>(ws));
  };
  auto by_type = [&](auto DD) {
    if (dtype == VC_F32)
      go(DD, float{});
    else if (dtype == VC_F16)
      go(DD, __half{});
    else
      go(DD, __nv_bfloat16{});
  };
  if (shape->D == 128)
    by_type(std::integral_constant<int, 128>{});
  else
    by_type(std::integral_constant<int, 64>{});
  return vc::launch_status("vc_fp4_cache_read");
}

}  // extern "C"

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

// Where request b's rows go: false (and a flag) when they do not fit.
__device__ __forceinline__ bool fp4_span(const int32_t* pos, int64_t pos0, const int32_t* counts, int b, int64_t n,
                                         int64_t T_cap, uint32_t* flags, bool report, int64_t& p, int64_t& c) {
  p = pos ? static_cast<int64_t>(__ldg(pos + b)) : pos0;
  c = counts ? static_cast<int64_t>(__ldg(counts + b)) : n;
  if (p >= 0 && c >= 0 && c <= n && p + c <= T_cap) return true;
  if (report) atomicOr(flags, VC_FLAG_BAD_LENGTH);
  return false;
}

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (std::is_same<T, __half>::value)
    return unpack_h2(w);
  else
    return unpack_bf2(w);
}

// One thread per (row, K or V, block of 16 channels).
template <int D, typename T>
__global__ void __launch_bounds__(256) fp4_write_kernel(uint8_t* __restrict__ records, int64_t T_cap,
                                                        const T* __restrict__ k, const T* __restrict__ v, int64_t n,
                                                        const int32_t* __restrict__ pos, int64_t pos0,
                                                        const int32_t* __restrict__ counts,
                                                        const int32_t* __restrict__ k_exp,
                                                        const int32_t* __restrict__ v_exp, int Hkv, uint32_t* flags) {
  using R = fp4::Rec<D>;
  const int unit = blockIdx.y;
  const int b = unit / Hkv, h = unit - b * Hkv;
  int64_t p, c;
  if (!fp4_span(pos, pos0, counts, b, n, T_cap, flags, threadIdx.x == 0, p, c)) return;
  const int64_t work = c * 2 * R::BLKS;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; e < work;
       e += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int j = static_cast<int>(e % R::BLKS);
    const bool val = (e / R::BLKS) & 1;
    const int64_t i = e / (2 * R::BLKS);
    const uint4* src = reinterpret_cast<const uint4*>((val ? v : k) + (static_cast<int64_t>(unit) * n + i) * D + j * 16);
    const uint4 w0 = src[0], w1 = src[1];
    const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    const float down = fp4::two_to(val ? v_exp : k_exp, h, -1);
    float x[16];
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      const float2 f = unpack2<T>(w[m]);
      x[2 * m] = f.x * down;
      x[2 * m + 1] = f.y * down;
    }
    uint32_t codes[2];
    uint8_t s8;
    if (fp4::quantise_block(x, codes, s8)) atomicOr(flags, VC_FLAG_RANGE);
    const int64_t at = p + i;
    const int t = static_cast<int>(at & (fp4::kTok - 1));
    uint8_t* rec = records + (static_cast<int64_t>(unit) * (T_cap / fp4::kTok) + at / fp4::kTok) * R::BYTES;
    if (val) {
      *reinterpret_cast<uint32_t*>(rec + R::v_word(t, j, 0)) = codes[0];
      *reinterpret_cast<uint32_t*>(rec + R::v_word(t, j, 1)) = codes[1];
      rec[R::v_scale(t, j)] = s8;
    } else {
      *reinterpret_cast<uint2*>(rec + R::k_codes(t, j)) = make_uint2(codes[0], codes[1]);
      rec[R::k_scale(t, j)] = s8;
    }
  }
}

template <typename T>
__device__ __forceinline__ void store16(T* dst, const float (&x)[16]) {
  if constexpr (std::is_same<T, float>::value) {
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *reinterpret_cast<float4*>(dst + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  } else {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i] = std::is_same<T, __half>::value ? pack_h2(x[2 * i], x[2 * i + 1]) : pack_bf2(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(dst + 8) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <int D, typename T>
__global__ void __launch_bounds__(256) fp4_read_kernel(const uint8_t* __restrict__ records, int64_t T_cap,
                                                       T* __restrict__ k, T* __restrict__ v, int64_t n,
                                                       const int32_t* __restrict__ pos, int64_t pos0,
                                                       const int32_t* __restrict__ counts,
                                                       const int32_t* __restrict__ k_exp,
                                                       const int32_t* __restrict__ v_exp, int Hkv, uint32_t* flags) {
  using R = fp4::Rec<D>;
  const int unit = blockIdx.y;
  const int b = unit / Hkv, h = unit - b * Hkv;
  int64_t p, c;
  if (!fp4_span(pos, pos0, counts, b, n, T_cap, flags, threadIdx.x == 0, p, c)) return;
  const int64_t work = c * 2 * R::BLKS;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; e < work;
       e += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int j = static_cast<int>(e % R::BLKS);
    const bool val = (e / R::BLKS) & 1;
    const int64_t i = e / (2 * R::BLKS);
    const int64_t at = p + i;
    const int t = static_cast<int>(at & (fp4::kTok - 1));
    const uint8_t* rec = records + (static_cast<int64_t>(unit) * (T_cap / fp4::kTok) + at / fp4::kTok) * R::BYTES;
    uint32_t w[2];
    uint8_t s8;
    if (val) {
      w[0] = *reinterpret_cast<const uint32_t*>(rec + R::v_word(t, j, 0));
      w[1] = *reinterpret_cast<const uint32_t*>(rec + R::v_word(t, j, 1));
      s8 = rec[R::v_scale(t, j)];
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(rec + R::k_codes(t, j));
      w[0] = u.x, w[1] = u.y;
      s8 = rec[R::k_scale(t, j)];
    }
    const float up = fp4::scale_to_float(s8) * fp4::two_to(val ? v_exp : k_exp, h, 1);
    float x[16];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      uint32_t o[4];
      fp4::codes_to_h2(w[m], o);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 f = unpack_h2(o[q]);
        x[8 * m + 2 * q] = f.x * up;
        x[8 * m + 2 * q + 1] = f.y * up;
      }
    }
    store16((val ? v : k) + (static_cast<int64_t>(unit) * n + i) * D + j * 16, x);
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

// Blocks of 256 threads per (request, KV head): all of the rows' blocks, at
// most about 16 waves of the card.
unsigned row_blocks(int64_t n, int D, int64_t units) {
  const int64_t want = (n * 2 * (D / fp4::kBlk) + 255) / 256;
  const int64_t most = std::max<int64_t>(1, static_cast<int64_t>(sm_count()) * 8 * 16 / units);
  return static_cast<unsigned>(std::min(want, most));
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
  const dim3 grid(vc::row_blocks(n, shape->D, units), units);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto go = [&](auto DD, auto tag) {
    using T = decltype(tag);
    vc::fp4_write_kernel<decltype(DD)::value, T><<<grid, 256, 0, s>>>(
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
  const dim3 grid(vc::row_blocks(n, shape->D, units), units);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto go = [&](auto DD, auto tag) {
    using T = decltype(tag);
    vc::fp4_read_kernel<decltype(DD)::value, T><<<grid, 256, 0, s>>>(
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

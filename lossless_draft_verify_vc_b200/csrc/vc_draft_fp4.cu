// vc_draft_fp4.cu -- single-token draft attention over the 4-bit
// floating-point cache (vc_fp4.cuh), with an optional sliding window and
// first tokens that stay visible.
//
// Drafting decodes one token per step from the compressed cache in HBM
// ("VeriCache: Turning Lossy KV Cache into Lossless LLM Inference",
// menfem.com, "Key Contributions"); the pages give no kernel.
#include <algorithm>

#include "vc_fp4.cuh"
#include "vc_splitk.cuh"

namespace vc {
namespace {

constexpr int kFThreads = 256;

struct FArgs {
  const uint8_t* records;
  const __nv_bfloat16* q;
  float* out;
  float* lse;
  const int32_t* lens;
  const int32_t* k_exp;
  const int32_t* v_exp;
  int64_t T_cap, T, window, n_sink;
  int Hq, Hkv, g;
  float scale_log2;
  uint32_t* flags;
};

// One block per (request, KV head); a warp takes every 8th visible token,
// its lanes the channels.
template <int D>
__global__ void __launch_bounds__(kFThreads) draft_fp4_kernel(FArgs a) {
  using R = fp4::Rec<D>;
  constexpr int PER = D / 32;  // channels of a lane
  __shared__ float s_o[8][8][D];
  __shared__ float s_ml[8][8][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x;
  const int b = unit / a.Hkv, h = unit - b * a.Hkv;
  int64_t L = a.lens ? static_cast<int64_t>(__ldg(a.lens + b)) : a.T;
  if (L < 0 || L > a.T_cap) {
    if (threadIdx.x == 0) atomicOr(a.flags, VC_FLAG_BAD_LENGTH);
    L = 0;
  }
  int64_t lo = a.window > 0 ? L - a.window : 0;
  if (lo < 0) lo = 0;
  const int64_t sinks = min(a.n_sink, lo);
  const int64_t nvis = sinks + (L - lo);
  const float kup = fp4::two_to(a.k_exp, h, 1) * a.scale_log2, vup = fp4::two_to(a.v_exp, h, 1);
  float q[8][PER], o[8][PER], m[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < PER; ++c) {
      o[i][c] = 0.f;
      q[i][c] = i < a.g ? __bfloat162float(a.q[(static_cast<size_t>(b) * a.Hq + h * a.g + i) * D + lane * PER + c]) : 0.f;
    }
  }
  const uint8_t* base = a.records + static_cast<int64_t>(unit) * (a.T_cap / fp4::kTok) * R::BYTES;
  const int c0 = lane * PER, j = c0 / 16;
  for (int64_t x = warp; x < nvis; x += 8) {
    const int64_t at = x < sinks ? x : lo + (x - sinks);
    const int t = static_cast<int>(at & 15);
    const uint8_t* rec = base + at / fp4::kTok * R::BYTES;
    const float ks = fp4::scale_to_float(rec[R::k_scale(t, j)]), vs = fp4::scale_to_float(rec[R::v_scale(t, j)]);
    float kk[PER], vv[PER];
    const int in_blk = c0 % 16;  // this lane's channels lie in one word of 8
    uint32_t k4[4], v4[4];
    fp4::codes_to_h2(*reinterpret_cast<const uint32_t*>(rec + R::k_codes(t, j) + in_blk / 8 * 4), k4);
    fp4::codes_to_h2(*reinterpret_cast<const uint32_t*>(rec + R::v_word(t, j, in_blk / 8)), v4);
#pragma unroll
    for (int c = 0; c < PER; c += 2) {
      const float2 fk = unpack_h2(k4[in_blk % 8 / 2 + c / 2]), fv = unpack_h2(v4[in_blk % 8 / 2 + c / 2]);
      kk[c] = fk.x * ks, kk[c + 1] = fk.y * ks;
      vv[c] = fv.x * vs, vv[c + 1] = fv.y * vs;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= a.g) break;
      float d = 0.f;
#pragma unroll
      for (int c = 0; c < PER; ++c) d += q[i][c] * kk[c];
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) d += __shfl_xor_sync(0xffffffffu, d, w);
      d *= kup;
      const float mn = fmaxf(m[i], d), al = ex2(m[i] - mn), p = ex2(d - mn);
      l[i] = l[i] * al + p;
      m[i] = mn;
#pragma unroll
      for (int c = 0; c < PER; ++c) o[i][c] = o[i][c] * al + p * vv[c];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int c = 0; c < PER; ++c) s_o[warp][i][c0 + c] = o[i][c];
    if (lane == 0) s_ml[warp][i][0] = m[i], s_ml[warp][i][1] = l[i];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.g * D; e += kFThreads) {
    const int i = e / D, c = e - i * D;
    float M = -INFINITY, Ls = 0.f, acc = 0.f;
    for (int w = 0; w < 8; ++w) M = fmaxf(M, s_ml[w][i][0]);
    for (int w = 0; w < 8; ++w) {
      const float sc = s_ml[w][i][0] == -INFINITY ? 0.f : ex2(s_ml[w][i][0] - M);
      Ls += sc * s_ml[w][i][1];
      acc += sc * s_o[w][i][c];
    }
    const size_t row = static_cast<size_t>(b) * a.Hq + h * a.g + i;
    a.out[row * D + c] = Ls > 0.f ? acc / Ls * vup : 0.f;
    if (a.lse && c == 0) a.lse[row] = lse_from(M, Ls);
  }
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

}  // namespace
}  // namespace vc

extern "C" {

size_t vc_draft_attn_fp4_workspace_size(const vc_attn_shape* shape, const vc_fp4_cache* cache) {
  if (vc::check_draft(shape, cache, "vc_draft_attn_fp4_workspace_size") != VC_OK) return 0;
  return vc::align_up(sizeof(vc::WsHeader), 256);
}

vc_status vc_draft_attn_fp4(const vc_attn_shape* shape, const vc_fp4_cache* cache, int64_t window, int64_t n_sink,
                            const void* q, float* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  vc_status st = vc::check_draft(shape, cache, "vc_draft_attn_fp4");
  if (st != VC_OK) return st;
  VC_REQUIRE(window >= 0 && n_sink >= 0, "vc_draft_attn_fp4: window and n_sink must be >= 0");
  VC_REQUIRE(cache->records && q && out && ws, "vc_draft_attn_fp4: null pointer argument");
  VC_REQUIRE(vc::aligned16(cache->records) && vc::aligned16(q) && vc::aligned16(out) && vc::aligned16(ws),
             "vc_draft_attn_fp4: records, q, out and workspace must be 16-byte aligned");
  const size_t need = vc_draft_attn_fp4_workspace_size(shape, cache);
  VC_REQUIRE(ws_bytes >= need, "vc_draft_attn_fp4: workspace too small (%zu < %zu)", ws_bytes, need);
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
  a.Hq = shape->Hq;
  a.Hkv = shape->Hkv;
  a.g = shape->Hq / shape->Hkv;
  const float sm = shape->sm_scale > 0.f ? shape->sm_scale : 1.0f / sqrtf(static_cast<float>(shape->D));
  a.scale_log2 = sm * 1.4426950408889634f;
  a.flags = static_cast<uint32_t*>(ws);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int units = shape->B * shape->Hkv;
  if (shape->D == 128)
    vc::draft_fp4_kernel<128><<<units, vc::kFThreads, 0, s>>>(a);
  else
    vc::draft_fp4_kernel<64><<<units, vc::kFThreads, 0, s>>>(a);
  return vc::launch_status("vc_draft_attn_fp4");
}

}  // extern "C"

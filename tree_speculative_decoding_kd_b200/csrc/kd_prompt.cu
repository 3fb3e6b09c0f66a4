// Causal attention of packed prompts with grouped heads, one warp per query row and
// head: the keys one at a time under an online softmax.
#include <math.h>

#include "kd_common.cuh"
#include "kd_ptx.cuh"

namespace kd {
namespace pr {

struct Params {
  const uint16_t *qn, *qr, *kn, *kr, *v;
  int64_t qnt, qnh, qrt, qrh, knt, knh, krt, krh, vt, vh;
  const int32_t *cu_q, *cu_k;
  uint16_t* out;
  float* lse;
  int32_t* err;
  int B, T, Tk, H, group;
  float scale;
};

__device__ __forceinline__ float bf(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

// blockIdx.y: sequence; warps over (row, head)
__global__ void __launch_bounds__(256) prompt_kernel(const Params p) {
  const int lane = threadIdx.x & 31, b = blockIdx.y;
  const int64_t q0 = p.cu_q[b], q1 = p.cu_q[b + 1];
  const int64_t k0 = p.cu_k ? p.cu_k[b] : q0, k1 = p.cu_k ? p.cu_k[b + 1] : q1;
  if (q0 < 0 || q1 < q0 || q1 > p.T || k0 < 0 || k1 < k0 || k1 > p.Tk) {
    if (threadIdx.x == 0 && blockIdx.x == 0) raise_dev_error(p.err, KD_DEV_BAD_SEQLENS);
    return;
  }
  const int64_t nq = q1 - q0, nk = k1 - k0;
  for (int64_t w = blockIdx.x * 8 + (threadIdx.x >> 5); w < nq * p.H; w += (int64_t)gridDim.x * 8) {
    const int64_t i = w / p.H;
    const int h = (int)(w % p.H), g = h / p.group;
    float q[4], r[2] = {0.f, 0.f}, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int e = 0; e < 4; ++e) q[e] = bf(p.qn[(q0 + i) * p.qnt + h * p.qnh + e * 32 + lane]);
    if (p.qr)
      for (int e = 0; e < 2; ++e) r[e] = bf(p.qr[(q0 + i) * p.qrt + h * p.qrh + e * 32 + lane]);
    float m = -INFINITY, l = 0.f;
    const int64_t end = min(nk, i + nk - nq + 1);
    for (int64_t j = 0; j < end; ++j) {
      float s = 0.f;
      for (int e = 0; e < 4; ++e) s += q[e] * bf(p.kn[(k0 + j) * p.knt + g * p.knh + e * 32 + lane]);
      if (p.qr)
        for (int e = 0; e < 2; ++e) s += r[e] * bf(p.kr[(k0 + j) * p.krt + g * p.krh + e * 32 + lane]);
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      s *= p.scale;
      const float mn = fmaxf(m, s), c = m == mn ? 1.f : expf(m - mn), x = expf(s - mn);
      l = l * c + x;
      m = mn;
      for (int e = 0; e < 4; ++e) o[e] = o[e] * c + x * bf(p.v[(k0 + j) * p.vt + g * p.vh + e * 32 + lane]);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    for (int e = 0; e < 4; ++e)
      p.out[((q0 + i) * p.H + h) * 128 + e * 32 + lane] = (uint16_t)ptx::pack_bf16x2(o[e] * inv, 0.f);
    if (lane == 0) p.lse[(q0 + i) * p.H + h] = l > 0.f ? m + logf(l) : -INFINITY;
  }
}

}  // namespace pr
}  // namespace kd

using namespace kd;

static bool view_ok(const void* p, int64_t tok, int64_t head) {
  return p && aligned16(p) && tok >= 0 && head >= 0 && tok % 8 == 0 && head % 8 == 0;
}

extern "C" int kd_prompt_attn(const kd_bf16_t* q_nope, int64_t qnt, int64_t qnh, const kd_bf16_t* q_rope, int64_t qrt,
                              int64_t qrh, const kd_bf16_t* k_nope, int64_t knt, int64_t knh, const kd_bf16_t* k_rope,
                              int64_t krt, int64_t krh, const kd_bf16_t* v, int64_t vt, int64_t vh,
                              const int32_t* cu_q, const int32_t* cu_k, int B, int T, int Tk, int H, int Hk,
                              float scale, kd_bf16_t* out, float* lse, int32_t* dev_error, cudaStream_t stream) {
  if (B < 1 || B > 65535 || T < 0 || Tk < 0 || H < 1 || H > KD_MAX_HEADS || Hk < 1 || H % Hk || !(scale > 0.f && isfinite(scale)) ||
      (int64_t)T * H > INT32_MAX || (int64_t)Tk * Hk > INT32_MAX || (q_rope != nullptr) != (k_rope != nullptr))
    return KD_EINVAL;
  if (T == 0) return KD_OK;
  if (!view_ok(q_nope, qnt, qnh) || !out || !aligned16(out) || !lse || !cu_q ||
      (Tk && (!view_ok(k_nope, knt, knh) || !view_ok(v, vt, vh))) ||
      (q_rope && (!view_ok(q_rope, qrt, qrh) || (Tk && !view_ok(k_rope, krt, krh)))))
    return KD_EINVAL;
  int st = device_sms(nullptr);
  if (st) return st;
  pr::Params p{q_nope, q_rope, k_nope, k_rope, v, qnt, qnh, qrt, qrh, knt, knh, krt, krh, vt, vh,
               cu_q, cu_k, out, lse, dev_error, B, T, Tk, H, H / Hk, scale};
  int64_t blocks = ((int64_t)T * H + 7) / 8;
  if (blocks > 4096) blocks = 4096;
  pr::prompt_kernel<<<dim3((unsigned)blocks, B), 256, 0, stream>>>(p);
  return launch_status("prompt_kernel");
}

// Attention weight that each cache slot receives from the counted nodes, one warp per
// slot: every counted node and head in turn, the dot product split over the lanes.
#include <math.h>

#include "kd_common.cuh"
#include "kd_ptx.cuh"
#include "kd_slots.cuh"

namespace kd {
namespace aw {

struct Params {
  const uint16_t *qa, *qr, *c, *r;
  int64_t sc, sr;
  SlotMap map;
  const int32_t *lens, *path, *len;
  const uint32_t* vis;
  const float *lse, *w_in;
  float* w_out;
  int64_t wi, wo;
  int32_t* err;
  int B, n, H, W;
  float scale;
};

__device__ __forceinline__ float bf(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

__global__ void __launch_bounds__(256) weights_kernel(const Params p) {
  __shared__ int nodes[KD_MAX_NODES];
  __shared__ int bad;
  const int b = blockIdx.y, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int64_t L = p.lens[b];
  const int count = p.path ? p.len[b] : p.n;
  if (tid == 0) bad = L < 0 || L + p.n > p.map.cap ? KD_DEV_CACHE_FULL : (count < 1 || count > p.n) ? KD_DEV_BAD_PATH : 0;
  __syncthreads();
  if (!bad) {
    if (tid < count) {
      const int k = p.path ? p.path[(size_t)b * p.n + tid] : tid;
      nodes[tid] = k;
      if (k < 0 || k >= p.n) atomicOr(&bad, KD_DEV_BAD_PATH);
    }
    if (p.map.pt)
      for (int64_t q = tid; q * p.map.P < L + p.n; q += 256)
        if (!p.map.pages_ok(b, q * p.map.P, q * p.map.P + 1)) atomicOr(&bad, KD_DEV_BAD_PAGE);
  }
  __syncthreads();
  if (bad) {
    if (tid == 0 && blockIdx.x == 0) raise_dev_error(p.err, bad);
    return;
  }
  // slots [0, L), then the counted nodes' slots in path order
  for (int64_t w = blockIdx.x * 8 + (tid >> 5); w < L + count; w += (int64_t)gridDim.x * 8) {
    const int node = w < L ? -1 : nodes[w - L];
    const int64_t row = p.map.row(b, w < L ? w : L + node);
    float c[16], r[2], sum = 0.f;
    for (int e = 0; e < 16; ++e) c[e] = bf(p.c[row * p.sc + e * 32 + lane]);
    for (int e = 0; e < 2; ++e) r[e] = bf(p.r[row * p.sr + e * 32 + lane]);
    for (int m = 0; m < count; ++m) {
      const int64_t i = (int64_t)b * p.n + nodes[m];
      if (node >= 0 && !(p.vis[i * p.W + (node >> 5)] >> (node & 31) & 1u)) continue;
      for (int h = 0; h < p.H; ++h) {
        const float z = p.lse[i * p.H + h];
        float s = 0.f;
        for (int e = 0; e < 16; ++e) s += c[e] * bf(p.qa[(i * p.H + h) * KD_D_C + e * 32 + lane]);
        for (int e = 0; e < 2; ++e) s += r[e] * bf(p.qr[(i * p.H + h) * KD_D_R + e * 32 + lane]);
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        if (z != -INFINITY) sum += expf(s * p.scale - z);
      }
    }
    if (lane == 0) p.w_out[b * p.wo + w] = sum + (w < L && p.w_in ? p.w_in[b * p.wi + w] : 0.f);
  }
}

}  // namespace aw
}  // namespace kd

using namespace kd;

static int weights_impl(const kd_bf16_t* qa, const kd_bf16_t* qr, const kd_bf16_t* c, const kd_bf16_t* r, int64_t sc,
                        int64_t sr, const SlotMap& map, int64_t cache_rows, const int32_t* lens, const uint32_t* vis,
                        const float* lse, const int32_t* path, const int32_t* len, int B, int n, int H, float scale,
                        const float* w_in, int64_t wi, float* w_out, int64_t wo, int32_t* dev_error,
                        cudaStream_t stream) {
  if (!qa || !qr || !lens || !vis || !lse || !w_out || !shapes_ok(B, n) || B > 65535 || H < 1 || H > KD_MAX_HEADS ||
      !cache_ok(c, r, sc, sr, map.cap) || !aligned16(qa) || !aligned16(qr) || !(scale > 0.f && isfinite(scale)) ||
      (path != nullptr) != (len != nullptr) || wo < map.cap || (w_in && wi < map.cap) || (w_in == w_out && wi != wo) ||
      (int64_t)B * n * H > INT32_MAX || cache_rows > INT32_MAX)
    return KD_EINVAL;
  int st = device_sms(nullptr);
  if (st) return st;
  aw::Params p{qa, qr, c, r, sc, sr, map, lens, path, len, vis, lse, w_in, w_out, wi, wo, dev_error, B, n, H, (n + 31) / 32, scale};
  int64_t blocks = (map.cap + 7) / 8;
  if (blocks > 4096) blocks = 4096;
  aw::weights_kernel<<<dim3((unsigned)blocks, B), 256, 0, stream>>>(p);
  return launch_status("weights_kernel");
}

extern "C" int kd_kv_attn_weights(const kd_bf16_t* q_nope_absorbed, const kd_bf16_t* q_rope, const kd_bf16_t* c_kv,
                                  const kd_bf16_t* k_rope, int64_t sc, int64_t sr, int64_t cap,
                                  const int32_t* cache_lens, const uint32_t* vis, const float* lse,
                                  const int32_t* path, const int32_t* len, int B, int n, int H, float scale,
                                  const float* weights_in, int64_t w_in_stride, float* weights_out,
                                  int64_t w_out_stride, int32_t* dev_error, cudaStream_t stream) {
  return weights_impl(q_nope_absorbed, q_rope, c_kv, k_rope, sc, sr, SlotMap{nullptr, cap, 0, 1, 0}, B * cap,
                      cache_lens, vis, lse, path, len, B, n, H, scale, weights_in, w_in_stride, weights_out,
                      w_out_stride, dev_error, stream);
}

extern "C" int kd_kv_attn_weights_paged(const kd_bf16_t* q_nope_absorbed, const kd_bf16_t* q_rope,
                                        const kd_bf16_t* c_pages, const kd_bf16_t* r_pages, int64_t sc, int64_t sr,
                                        int page_size, const int32_t* page_table, int64_t pages_per_req,
                                        int64_t num_pages, const int32_t* cache_lens, const uint32_t* vis,
                                        const float* lse, const int32_t* path, const int32_t* len, int B, int n, int H,
                                        float scale, const float* weights_in, int64_t w_in_stride, float* weights_out,
                                        int64_t w_out_stride, int32_t* dev_error, cudaStream_t stream) {
  if (!paged_ok(page_table, page_size, pages_per_req, num_pages) ||
      (page_size != 64 && page_size != 128 && page_size != 256))
    return KD_EINVAL;
  return weights_impl(q_nope_absorbed, q_rope, c_pages, r_pages, sc, sr,
                      SlotMap{page_table, pages_per_req * page_size, num_pages, page_size, (int)pages_per_req},
                      num_pages * page_size, cache_lens, vis, lse, path, len, B, n, H, scale, weights_in, w_in_stride,
                      weights_out, w_out_stride, dev_error, stream);
}

// RMS norm and position rotation in one pass: over packed query and key heads
// (kd_qk_norm_rope), and over a down-projection's output on its way into the latent
// cache (kd_kv_norm_rope_write).
//
//   y = x / sqrt(mean(x^2) + eps) * w,   (a, b) -> (a cos - b sin, a sin + b cos)
//
// Both are bound by memory (about 7 operations per 4 bytes moved), so every element is
// read once and written once, 16 bytes at a time.  A head's D <= 256 elements lie in one
// group of 8, 16 or 32 lanes, eight neighbouring elements per lane: the sum of squares
// is a few shuffles inside the group, and the partner of a pair (i, i + rot/2) sits at
// the same place of another lane, rot/16 lanes away.  A group takes four heads of one
// token: four loads in flight per lane, and the token's cosines and sines, which cost
// more loads than the data they turn, are read once for the four.  Sums, norm and
// rotation are in fp32; the one rounding is the store's.

#include "kd_common.cuh"
#include "kd_ptx.cuh"
#include "kd_slots.cuh"

namespace kd {
namespace nr {

constexpr int U = 4;                       // heads a group works on at once
constexpr int THREADS = 256;

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]), ptx::pack_bf16x2(x[4], x[5]),
                    ptx::pack_bf16x2(x[6], x[7]));
}

// One lane's part of a rotation: its eight elements start at element e of the rotated
// range (or lie outside it: on == false).
struct Turn {
  float c[8], s[8];     // interleaved pairs use the first four
  int partner;          // lane of the group that holds the pairs' other halves
  bool on, inter;
  // lane: this lane's index in its group; e: first element relative to the range
  __device__ __forceinline__ void load(const float* row, int e, int rot, bool interleaved, int lane) {
    on = e >= 0 && e < rot;
    inter = interleaved;
    partner = lane;
    if (!on) return;
    const int half = rot >> 1;
    if (inter) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(row + (e >> 1)));
      const float4 b = __ldg(reinterpret_cast<const float4*>(row + half + (e >> 1)));
      c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w;
      s[0] = b.x, s[1] = b.y, s[2] = b.z, s[3] = b.w;
      return;
    }
    const bool first = e < half;
    const int i = first ? e : e - half;
    partner = first ? lane + (half >> 3) : lane - (half >> 3);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(row + i + 4 * q));
      const float4 b = __ldg(reinterpret_cast<const float4*>(row + half + i + 4 * q));
      c[4 * q] = a.x, c[4 * q + 1] = a.y, c[4 * q + 2] = a.z, c[4 * q + 3] = a.w;
      const float sg = first ? -1.f : 1.f;
      s[4 * q] = sg * b.x, s[4 * q + 1] = sg * b.y, s[4 * q + 2] = sg * b.z, s[4 * q + 3] = sg * b.w;
    }
  }
  // All lanes of the warp call it; WIDTH: lanes of a group.
  template <int WIDTH>
  __device__ __forceinline__ void apply(float (&x)[8]) const {
    if (inter) {                                   // the same in every lane of the warp
      if (!on) return;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = a * c[i] - b * s[i];
        x[2 * i + 1] = a * s[i] + b * c[i];
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float p = __shfl_sync(0xffffffffu, x[i], partner, WIDTH);
      if (on) x[i] = x[i] * c[i] + p * s[i];
    }
  }
};

// ------------------------------------------------------------------ query and key heads
struct QkSide {
  const uint16_t* in;
  const uint16_t* w;
  uint16_t* out;
  int64_t it, ih, ot, oh;      // token and head strides, in and out
  int heads, items;            // items = ceil(heads / U) groups per token
};
struct QkParams {
  QkSide q, k;
  const float* table;
  const int32_t* pos;
  int32_t* err;
  int64_t max_pos;
  float eps, inv_d;
  int T, D, rot, off, inter;
};

// G lanes per head (the least power of two that holds D / 8).
template <int G>
__global__ void __launch_bounds__(THREADS) qk_norm_rope_kernel(const QkParams p) {
  const int lane = threadIdx.x & (G - 1);
  const unsigned items = (unsigned)(p.q.items + p.k.items);
  const unsigned g = blockIdx.x * (THREADS / G) + threadIdx.x / G;
  unsigned t = g / items, item = g - t * items;
  bool live = t < (unsigned)p.T;                   // no early exit: the shuffles take whole warps
  int64_t at = 0;
  if (live) {
    at = p.pos[t];
    if (at < 0 || at >= p.max_pos) {
      if (lane == 0) raise_dev_error(p.err, KD_DEV_BAD_POSITION);
      live = false;
    }
  }
  const bool is_k = item >= (unsigned)p.q.items;
  const QkSide& s = is_k ? p.k : p.q;
  const int h0 = (int)(is_k ? item - p.q.items : item) * U, e = lane * 8;
  const bool mine = live && e < p.D;

  uint4 raw[U];
  const uint16_t* in = s.in + (int64_t)t * s.it + e;
#pragma unroll
  for (int u = 0; u < U; ++u)
    raw[u] = mine && h0 + u < s.heads ? *reinterpret_cast<const uint4*>(in + (h0 + u) * s.ih) : make_uint4(0, 0, 0, 0);
  float w[8];
  const bool norm = s.w != nullptr;
  if (norm && mine) unpack8(__ldg(reinterpret_cast<const uint4*>(s.w + e)), w);
  Turn turn;
  turn.load(p.table + (live ? at : 0) * p.rot, mine ? e - p.off : -1, p.rot, p.inter != 0, lane);

#pragma unroll
  for (int u = 0; u < U; ++u) {
    float x[8];
    unpack8(raw[u], x);
    // the group's lanes agree on `norm`, a warp's groups may not: the shuffles are for all
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
    for (int m = G / 2; m; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    if (norm) {
      const float r = rsqrtf(ss * p.inv_d + p.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * r * (mine ? w[i] : 0.f);
    }
    turn.template apply<G>(x);
    if (mine && h0 + u < s.heads)
      *reinterpret_cast<uint4*>(s.out + (int64_t)t * s.ot + (h0 + u) * s.oh + e) = pack8(x);
  }
}

// ------------------------------------------------------------------ into the cache
struct WriteParams {
  uint16_t *c_kv, *k_rope, *q_out;
  const uint16_t *kv, *w, *q_in;
  const float* table;
  const int32_t *lens, *pos, *cu;
  int32_t* err;
  SlotMap map;
  int64_t sc, sr, kv_stride, qt, qh, max_pos;
  float eps;
  int B, T, n, H, items, inter;      // items = 1 + ceil(H / 16) warps per token
};

// Sequence of token t: the last b with cu[b] <= t (B when t lies past the last one).
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, int t) {
  int lo = 0, hi = B;                  // cu[lo] <= t < cu[hi + 1], were cu[B + 1] infinite
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// One warp per item of a token: item 0 its latent and rope key, item 1 + i the rope parts
// of query heads 16 i .. 16 i + 15 (eight lanes a head, four heads at a time).
__global__ void __launch_bounds__(THREADS) kv_norm_rope_write_kernel(const WriteParams p) {
  const int lane = threadIdx.x & 31;
  const unsigned wi = blockIdx.x * (THREADS / 32) + threadIdx.x / 32;
  const unsigned t = wi / (unsigned)p.items, item = wi - t * (unsigned)p.items;
  if (t >= (unsigned)p.T) return;
  int b, first, count;
  if (p.cu) {
    b = sequence_of(p.cu, p.B, (int)t);
    if (b == p.B) return;                                    // behind the last sequence
    first = p.cu[b];
    count = p.cu[b + 1] - first;
    if (first < 0 || (int)t < first || (int)t - first >= count || p.cu[b + 1] > p.T) {
      if (lane == 0) raise_dev_error(p.err, KD_DEV_BAD_SEQLENS);
      return;
    }
  } else {
    b = (int)(t / (unsigned)p.n);
    first = b * p.n;
    count = p.n;
  }
  const int64_t L = p.lens[b], slot = L + ((int)t - first);
  const int64_t at = p.pos ? (int64_t)p.pos[t] : slot;
  if (at < 0 || at >= p.max_pos) {
    if (lane == 0) raise_dev_error(p.err, KD_DEV_BAD_POSITION);
    return;
  }
  const float* row = p.table + at * KD_D_R;

  if (item == 0) {
    if (L < 0 || L + count > p.map.cap) {
      if (lane == 0) raise_dev_error(p.err, KD_DEV_CACHE_FULL);
      return;
    }
    if (!p.map.pages_ok(b, slot, slot + 1)) {
      if (lane == 0) raise_dev_error(p.err, KD_DEV_BAD_PAGE);
      return;
    }
    const uint16_t* src = p.kv + (int64_t)t * p.kv_stride;
    uint4 raw[2], rr = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int q = 0; q < 2; ++q) raw[q] = *reinterpret_cast<const uint4*>(src + (lane + 32 * q) * 8);
    if (lane < 8) rr = *reinterpret_cast<const uint4*>(src + KD_D_C + lane * 8);
    Turn turn;
    turn.load(row, lane < 8 ? lane * 8 : -1, KD_D_R, p.inter != 0, lane & 7);
    float x[2][8], ss = 0.f;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      unpack8(raw[q], x[q]);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += x[q][i] * x[q][i];
    }
    const int64_t r = p.map.row(b, slot);
    if (p.w) {
#pragma unroll
      for (int m = 16; m; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
      const float rs = rsqrtf(ss * (1.f / KD_D_C) + p.eps);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float w[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(p.w + (lane + 32 * q) * 8)), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[q][i] = x[q][i] * rs * w[i];
      }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q)
      *reinterpret_cast<uint4*>(p.c_kv + r * p.sc + (lane + 32 * q) * 8) = pack8(x[q]);
    float y[8];
    unpack8(rr, y);
    turn.template apply<8>(y);
    if (lane < 8) *reinterpret_cast<uint4*>(p.k_rope + r * p.sr + lane * 8) = pack8(y);
    return;
  }

  const int h0 = (int)(item - 1) * 16 + (lane >> 3), e = (lane & 7) * 8;
  uint4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    raw[u] = h0 + 4 * u < p.H ? *reinterpret_cast<const uint4*>(p.q_in + (int64_t)t * p.qt + (h0 + 4 * u) * p.qh + e)
                              : make_uint4(0, 0, 0, 0);
  Turn turn;
  turn.load(row, e, KD_D_R, p.inter != 0, lane & 7);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float x[8];
    unpack8(raw[u], x);
    turn.template apply<8>(x);
    if (h0 + 4 * u < p.H)
      *reinterpret_cast<uint4*>(p.q_out + ((int64_t)t * p.H + h0 + 4 * u) * KD_D_R + e) = pack8(x);
  }
}

}  // namespace nr
}  // namespace kd

using namespace kd;

// ================================================================== C ABI
static bool strides_ok(int64_t a, int64_t b) { return a % 8 == 0 && b % 8 == 0 && a >= 0 && b >= 0; }

extern "C" int kd_qk_norm_rope(const kd_bf16_t* q, int64_t qt, int64_t qh, const kd_bf16_t* k, int64_t kt,
                               int64_t kh, const kd_bf16_t* q_weight, const kd_bf16_t* k_weight, float eps,
                               const float* rope_table, int64_t max_pos, const int32_t* positions, int T, int H,
                               int Hk, int D, int rot, int rot_offset, int interleaved, kd_bf16_t* q_out,
                               int64_t qot, int64_t qoh, kd_bf16_t* k_out, int64_t kot, int64_t koh,
                               int32_t* dev_error, cudaStream_t stream) {
  if (T < 0 || H < 1 || Hk < 0 || D < 16 || D > 256 || D % 8 || rot < 16 || rot % 16 || rot_offset < 0 ||
      rot_offset % 8 || rot_offset + rot > D || !(eps >= 0.f) || max_pos < 1 ||
      (int64_t)T * ((int64_t)H + Hk) > INT32_MAX)
    return KD_EINVAL;
  if (T == 0) return KD_OK;
  if (!q || !q_out || !rope_table || !positions || !aligned16(q) || !aligned16(q_out) || !aligned16(q_weight) ||
      !aligned16(k_weight) || !aligned16(rope_table) || !strides_ok(qt, qh) || !strides_ok(qot, qoh))
    return KD_EINVAL;
  if (Hk && (!k || !k_out || !aligned16(k) || !aligned16(k_out) || !strides_ok(kt, kh) || !strides_ok(kot, koh)))
    return KD_EINVAL;
  int st = device_sms(nullptr);
  if (st) return st;
  nr::QkParams p;
  p.q = {q, q_weight, q_out, qt, qh, qot, qoh, H, (H + nr::U - 1) / nr::U};
  p.k = {k, k_weight, k_out, kt, kh, kot, koh, Hk, (Hk + nr::U - 1) / nr::U};
  p.table = rope_table;
  p.pos = positions;
  p.err = dev_error;
  p.max_pos = max_pos;
  p.eps = eps;
  p.inv_d = 1.f / (float)D;
  p.T = T;
  p.D = D;
  p.rot = rot;
  p.off = rot_offset;
  p.inter = interleaved;
  const int G = D <= 64 ? 8 : D <= 128 ? 16 : 32;
  const int64_t groups = (int64_t)T * (p.q.items + p.k.items);
  const unsigned grid = (unsigned)((groups * G + nr::THREADS - 1) / nr::THREADS);
  if (G == 8) nr::qk_norm_rope_kernel<8><<<grid, nr::THREADS, 0, stream>>>(p);
  else if (G == 16) nr::qk_norm_rope_kernel<16><<<grid, nr::THREADS, 0, stream>>>(p);
  else nr::qk_norm_rope_kernel<32><<<grid, nr::THREADS, 0, stream>>>(p);
  return launch_status("qk_norm_rope_kernel");
}

static int write_impl(kd_bf16_t* c_kv, kd_bf16_t* k_rope, int64_t sc, int64_t sr, const SlotMap& map,
                      const int32_t* cache_lens, const kd_bf16_t* kv, int64_t kv_stride, const kd_bf16_t* kv_weight,
                      float eps, const float* rope_table, int64_t max_pos, const int32_t* positions,
                      int interleaved, const int32_t* cu, int B, int T, const kd_bf16_t* q_in, int64_t qt,
                      int64_t qh, int H, kd_bf16_t* q_out, int32_t* dev_error, cudaStream_t stream) {
  if (B < 1 || T < 0 || T > (1 << 27) || H < 0 || H > KD_MAX_HEADS || !(eps >= 0.f) || max_pos < 1 ||
      (!cu && T % B) || !cache_ok(c_kv, k_rope, sc, sr, map.cap))
    return KD_EINVAL;
  if (T == 0) return KD_OK;
  if (!cache_lens || !kv || !aligned16(kv) || kv_stride < KD_D_C + KD_D_R || kv_stride % 8 || !aligned16(kv_weight) ||
      !rope_table || !aligned16(rope_table))
    return KD_EINVAL;
  if (H && (!q_in || !q_out || !aligned16(q_in) || !aligned16(q_out) || !strides_ok(qt, qh))) return KD_EINVAL;
  int st = device_sms(nullptr);
  if (st) return st;
  nr::WriteParams p;
  p.c_kv = c_kv;
  p.k_rope = k_rope;
  p.q_out = q_out;
  p.kv = kv;
  p.w = kv_weight;
  p.q_in = q_in;
  p.table = rope_table;
  p.lens = cache_lens;
  p.pos = positions;
  p.cu = cu;
  p.err = dev_error;
  p.map = map;
  p.sc = sc;
  p.sr = sr;
  p.kv_stride = kv_stride;
  p.qt = qt;
  p.qh = qh;
  p.max_pos = max_pos;
  p.eps = eps;
  p.B = B;
  p.T = T;
  p.n = cu ? 0 : T / B;
  p.H = H;
  p.items = 1 + (H + 15) / 16;
  p.inter = interleaved;
  const unsigned grid = (unsigned)(((int64_t)T * p.items + nr::THREADS / 32 - 1) / (nr::THREADS / 32));
  nr::kv_norm_rope_write_kernel<<<grid, nr::THREADS, 0, stream>>>(p);
  return launch_status("kv_norm_rope_write_kernel");
}

extern "C" int kd_kv_norm_rope_write(kd_bf16_t* c_kv, kd_bf16_t* k_rope, int64_t sc, int64_t sr, int64_t cap,
                                     const int32_t* cache_lens, const kd_bf16_t* kv, int64_t kv_row_stride,
                                     const kd_bf16_t* kv_weight, float eps, const float* rope_table,
                                     int64_t max_pos, const int32_t* positions, int interleaved,
                                     const int32_t* cu_seqlens, int B, int T, const kd_bf16_t* q_rope_in,
                                     int64_t q_tok_stride, int64_t q_head_stride, int H, kd_bf16_t* q_rope_out,
                                     int32_t* dev_error, cudaStream_t stream) {
  return write_impl(c_kv, k_rope, sc, sr, SlotMap{nullptr, cap, 0, 1, 0}, cache_lens, kv, kv_row_stride, kv_weight,
                    eps, rope_table, max_pos, positions, interleaved, cu_seqlens, B, T, q_rope_in, q_tok_stride,
                    q_head_stride, H, q_rope_out, dev_error, stream);
}

extern "C" int kd_kv_norm_rope_write_paged(kd_bf16_t* c_pages, kd_bf16_t* r_pages, int64_t sc, int64_t sr,
                                           int page_size, const int32_t* page_table, int64_t pages_per_req,
                                           int64_t num_pages, const int32_t* cache_lens, const kd_bf16_t* kv,
                                           int64_t kv_row_stride, const kd_bf16_t* kv_weight, float eps,
                                           const float* rope_table, int64_t max_pos, const int32_t* positions,
                                           int interleaved, const int32_t* cu_seqlens, int B, int T,
                                           const kd_bf16_t* q_rope_in, int64_t q_tok_stride, int64_t q_head_stride,
                                           int H, kd_bf16_t* q_rope_out, int32_t* dev_error, cudaStream_t stream) {
  if (!paged_ok(page_table, page_size, pages_per_req, num_pages)) return KD_EINVAL;
  return write_impl(c_pages, r_pages, sc, sr,
                    SlotMap{page_table, pages_per_req * page_size, num_pages, page_size, (int)pages_per_req},
                    cache_lens, kv, kv_row_stride, kv_weight, eps, rope_table, max_pos, positions, interleaved,
                    cu_seqlens, B, T, q_rope_in, q_tok_stride, q_head_stride, H, q_rope_out, dev_error, stream);
}

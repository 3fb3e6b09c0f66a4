// RMS norm and position rotation in one pass: over packed query and key heads
// (kd_qk_norm_rope), and over a down-projection's output on its way into the latent
// cache (kd_kv_norm_rope_write).
//
//   y = x / sqrt(mean(x^2) + eps) * w,   (a, b) -> (a cos - b sin, a sin + b cos)
//
// Both are bound by memory (about 7 operations per 4 bytes moved), so every element is
// read once and written once, 16 bytes at a time.  A lane holds two pieces of eight
// neighbouring elements of a head, chosen so that the rotation needs no other lane: with
// pairs (i, i + rot/2) the two pieces are rot/2 apart.  A head's D <= 256 elements lie in a group of 4, 8 or 16 lanes; the sum
// of squares is a few shuffles inside the group.  A group walks over up to eight heads, of
// one token where that fills it, so that the token's cosines and sines and the weights are
// read once for them; the heads ahead are on their way into shared memory meanwhile (each
// lane copies and reads only its own pieces: no barrier).  Sums, norm and rotation are in fp32; the one rounding is the
// store's.
//
// Measured (one B200): 16385 tokens of 40 heads of 128, 344 MB: 57 us, 5.9 TB/s, nine tenths of
// what a plain copy reaches; 14.3 K tokens of 64 heads into a paged cache, 271 MB: 48 us.  One
// piece per lane and four heads a group, loaded into registers, took 78 and 62 us: the
// rotation's shuffles and the instructions spent once per group left too few loads under way.
// Two or eight heads on their way instead of four: 61 and 61 us.

#include "kd_common.cuh"
#include "kd_ptx.cuh"
#include "kd_slots.cuh"

namespace kd {
namespace nr {

constexpr int THREADS = 128;
constexpr int DEPTH = 4;                   // heads on their way per group

// A lane's ring of DEPTH heads, two 16-byte pieces each, in shared memory.
struct Ring {
  uint32_t at;                             // this lane's first piece; pieces of a block lie side by side
  __device__ __forceinline__ explicit Ring(const uint4* smem) : at(ptx::smem_u32(smem + threadIdx.x)) {}
  __device__ __forceinline__ uint32_t piece(int slot, int i) const { return at + (slot * 2 + i) * THREADS * 16; }
  // Copies a piece (zeros when !on).
  __device__ __forceinline__ void copy(int slot, int i, const void* src, bool on) const {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(piece(slot, i)), "l"(src), "r"(on ? 16 : 0)
                 : "memory");
  }
  __device__ __forceinline__ static void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // The oldest of the DEPTH groups on their way has landed.
  __device__ __forceinline__ static void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory"); }
};

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

// One lane's part of a rotation: two pieces of eight elements, a and b.
struct Turn {
  float c[8], s[8];     // of the eight pairs (a_i, b_i); interleaved: four pairs of a, four of b
  bool on, inter;
  // ea, eb: first elements of the pieces relative to the rotated range, if both are in it
  __device__ __forceinline__ void load(const float* row, int ea, int eb, int rot, bool rotated, bool interleaved) {
    on = rotated;
    inter = interleaved;
    if (!on) return;
    const float* sn = row + (rot >> 1);
    const int i0 = inter ? ea >> 1 : ea, i1 = inter ? eb >> 1 : ea + 4;
    const float4 c0 = __ldg(reinterpret_cast<const float4*>(row + i0)), c1 = __ldg(reinterpret_cast<const float4*>(row + i1));
    const float4 s0 = __ldg(reinterpret_cast<const float4*>(sn + i0)), s1 = __ldg(reinterpret_cast<const float4*>(sn + i1));
    c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w, c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
    s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w, s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
  }
  __device__ __forceinline__ static void pair(float& x, float& y, float c, float s) {
    const float a = x, b = y;
    x = a * c - b * s;
    y = a * s + b * c;
  }
  __device__ __forceinline__ void apply(float (&a)[8], float (&b)[8]) const {
    if (!on) return;
    if (inter) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pair(a[2 * i], a[2 * i + 1], c[i], s[i]);
        pair(b[2 * i], b[2 * i + 1], c[4 + i], s[4 + i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) pair(a[i], b[i], c[i], s[i]);
    }
  }
};

// ------------------------------------------------------------------ query and key heads
struct QkSide {
  const uint16_t* in;
  const uint16_t* w;
  uint16_t* out;
  int64_t it, ih, ot, oh;      // token and head strides, in and out
  int heads;
  unsigned groups;             // of `per` heads in a row, counted over all tokens
};
struct QkParams {
  QkSide q, k;
  const float* table;
  const int32_t* pos;
  int32_t* err;
  int64_t max_pos;
  float eps, inv_d;
  int T, D, rot, off, inter, per;      // per: heads of a group
};

// G lanes per head (the least power of two that holds D / 16).  Lane l of a group has
//   l < rot / 16: elements off + 8 l and off + rot / 2 + 8 l, eight each: both halves of pairs;
//   else: one piece of each half of those outside the rotated range (neighbouring lanes have
//         neighbouring pieces: two pieces in a row per lane, half of each 32-byte sector at a time,
//         took 70 us where this takes 60, 20000 tokens of 32 heads of 128, half of each rotated).
//
// A group has `per` heads in a row, counted over all tokens.  SPAN: they may be of several tokens,
// whose angles are then loaded as the group comes to them.
template <int G, bool SPAN>
__global__ void __launch_bounds__(THREADS) qk_norm_rope_kernel(const QkParams p) {
  __shared__ uint4 pieces[DEPTH * 2 * THREADS];
  const Ring ring(pieces);
  const int lane = threadIdx.x & (G - 1);
  const unsigned g = blockIdx.x * (THREADS / G) + threadIdx.x / G;
  const bool is_k = g >= p.q.groups;
  const QkSide& s = is_k ? p.k : p.q;
  // the group's heads: n, from head h of token t on
  const unsigned heads = (unsigned)s.heads, f0 = (is_k ? g - p.q.groups : g) * (unsigned)p.per;
  const unsigned all = (unsigned)p.T * heads;
  const int n = f0 < all ? (int)min((unsigned)p.per, all - f0) : 0;    // no early exit: the shuffles take whole warps
  unsigned t = n ? f0 / heads : 0u;
  const unsigned h = n ? f0 - t * heads : 0u;
  const int rest = (p.D - p.rot) >> 3;               // pieces outside the range; this lane's:
  const int r0 = lane - (p.rot >> 4), r1 = r0 + ((rest + 1) >> 1);
  const bool rotated = r0 < 0;
  int ea, eb;
  if (rotated) {
    ea = p.off + 8 * lane;
    eb = ea + (p.rot >> 1);
  } else {
    ea = 8 * r0 < p.off ? 8 * r0 : 8 * r0 + p.rot;
    eb = 8 * r1 < p.off ? 8 * r1 : 8 * r1 + p.rot;
  }
  const bool has_a = rotated || 2 * r0 < rest, has_b = rotated || (has_a && r1 < rest);
  const uint16_t* in = s.in + (int64_t)t * s.it + h * s.ih;
  uint16_t* out = s.out + (int64_t)t * s.ot + h * s.oh;
  int left = (int)(heads - h), left_in = left;       // heads of the token that are left, to store and to ask for
  const int64_t wrap_in = s.it - (heads - 1) * s.ih, wrap_out = s.ot - (heads - 1) * s.oh;
  auto ask = [&](int i) {
    if (i < n) {
      ring.copy(i & (DEPTH - 1), 0, in + (has_a ? ea : 0), has_a);
      ring.copy(i & (DEPTH - 1), 1, in + (has_b ? eb : 0), has_b);
      if (SPAN && --left_in == 0) {
        in += wrap_in;
        left_in = (int)heads;
      } else {
        in += s.ih;
      }
    }
    Ring::commit();
  };
  const int pos = n ? p.pos[t] : 0;
  int next = SPAN && left < n ? p.pos[t + 1] : 0;    // position of the token after this one
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) ask(i);
  const bool norm = s.w != nullptr;
  float wa[8], wb[8];
  if (norm && n) {
    unpack8(has_a ? __ldg(reinterpret_cast<const uint4*>(s.w + ea)) : make_uint4(0, 0, 0, 0), wa);
    unpack8(has_b ? __ldg(reinterpret_cast<const uint4*>(s.w + eb)) : make_uint4(0, 0, 0, 0), wb);
  }
  // a token's angles; false when its position is bad
  auto turn_of = [&](Turn& turn, int64_t at) -> bool {
    const bool good = at >= 0 && at < p.max_pos;
    if (!good && lane == 0) raise_dev_error(p.err, KD_DEV_BAD_POSITION);
    turn.load(p.table + at * p.rot, ea - p.off, eb - p.off, p.rot, good && rotated, p.inter != 0);
    return good;
  };
  Turn turn;
  bool live = n && turn_of(turn, pos);

  // the groups of a warp may have fewer heads or none: the shuffles are for all
  const int most = __reduce_max_sync(0xffffffffu, n);
#pragma unroll 1
  for (int i = 0; i < most; ++i) {
    Ring::wait();
    float a[8], b[8];
    unpack8(ptx::ld_shared_v4(ring.piece(i & (DEPTH - 1), 0)), a);
    unpack8(ptx::ld_shared_v4(ring.piece(i & (DEPTH - 1), 1)), b);
    ask(i + DEPTH);
    float ss = 0.f, sb = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      ss += a[e] * a[e];
      sb += b[e] * b[e];
    }
    ss += sb;
#pragma unroll
    for (int m = G / 2; m; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    if (norm) {
      const float r = rsqrtf(ss * p.inv_d + p.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] = a[e] * r * wa[e];
        b[e] = b[e] * r * wb[e];
      }
    }
    turn.apply(a, b);
    if (i < n && live) {
      if (has_a) *reinterpret_cast<uint4*>(out + ea) = pack8(a);
      if (has_b) *reinterpret_cast<uint4*>(out + eb) = pack8(b);
    }
    if (SPAN && --left == 0) {                       // the next token
      out += wrap_out;
      left = (int)heads;
      ++t;
      if (i + 1 < n) {
        live = turn_of(turn, next);
        if (i + 1 + (int)heads < n) next = p.pos[t + 1];
      }
    } else {
      out += s.oh;
    }
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
  int B, T, n, H, items, inter, per;   // items = max(1, ceil(H / per)) warps per token
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

// A warp's work: item i of a token is the rope parts of `per` query heads from per i on (four
// lanes a head, eight heads at a time), item 0 the token's latent and rope key too, whose
// loads are on their way with the queries' first ones.
__device__ __forceinline__ void write_item(const WriteParams& p, const Ring& ring, unsigned t, unsigned item) {
  const int lane = threadIdx.x & 31;
  int b, first, count;
  if (p.cu) {
    b = sequence_of(p.cu, p.B, (int)t);
    if (b == p.B) return;                                    // behind the last sequence
    first = p.cu[b];
    count = p.cu[b + 1] - first;
  } else {
    b = (int)(t / (unsigned)p.n);
    first = b * p.n;
    count = p.n;
  }
  const int64_t L = p.lens[b], slot = L + ((int)t - first);
  const bool full = L < 0 || L + count > p.map.cap;          // reported whatever the position is
  if (full && item == 0 && lane == 0) raise_dev_error(p.err, KD_DEV_CACHE_FULL);
  const int64_t at = p.pos ? (int64_t)p.pos[t] : slot;
  if (at < 0 || at >= p.max_pos) {
    if (lane == 0) raise_dev_error(p.err, KD_DEV_BAD_POSITION);
    return;
  }
  const float* row = p.table + at * KD_D_R;

  const int h0 = (int)item * p.per + (lane >> 2), end = min(p.H, (int)(item + 1) * p.per);
  const int ea = (lane & 3) * 8, eb = ea + KD_D_R / 2;
  const uint16_t* in = p.q_in + (int64_t)t * p.qt;
  auto ask = [&](int i) {
    const int h = h0 + 8 * i;
    if (h < end) {
      ring.copy(i & (DEPTH - 1), 0, in + h * p.qh + ea, true);
      ring.copy(i & (DEPTH - 1), 1, in + h * p.qh + eb, true);
    }
    Ring::commit();
  };
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) ask(i);

  Turn turn;                                         // of the lane's two pieces of any head
  if (item == 0) {
    const uint16_t* src = p.kv + (int64_t)t * p.kv_stride;
    uint4 raw[2], rr[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) raw[q] = *reinterpret_cast<const uint4*>(src + (lane + 32 * q) * 8);
    if (lane < 4) {
      rr[0] = *reinterpret_cast<const uint4*>(src + KD_D_C + ea);
      rr[1] = *reinterpret_cast<const uint4*>(src + KD_D_C + eb);
    }
    turn.load(row, ea, eb, KD_D_R, true, p.inter != 0);
    const bool stored = !full && p.map.pages_ok(b, slot, slot + 1);
    if (!full && !stored && lane == 0) raise_dev_error(p.err, KD_DEV_BAD_PAGE);
    if (stored) {
      const int64_t r = p.map.row(b, slot);
      float x[2][8], ss = 0.f;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        unpack8(raw[q], x[q]);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += x[q][i] * x[q][i];
      }
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
      if (lane < 4) {
        unpack8(rr[0], x[0]);
        unpack8(rr[1], x[1]);
        turn.apply(x[0], x[1]);
        *reinterpret_cast<uint4*>(p.k_rope + r * p.sr + ea) = pack8(x[0]);
        *reinterpret_cast<uint4*>(p.k_rope + r * p.sr + eb) = pack8(x[1]);
      }
    }
  } else {
    turn.load(row, ea, eb, KD_D_R, true, p.inter != 0);
  }

  uint16_t* out = p.q_out + ((int64_t)t * p.H + h0) * KD_D_R;
#pragma unroll 1
  for (int i = 0; h0 + 8 * i < end; ++i, out += 8 * KD_D_R) {
    Ring::wait();
    float a[8], b[8];
    unpack8(ptx::ld_shared_v4(ring.piece(i & (DEPTH - 1), 0)), a);
    unpack8(ptx::ld_shared_v4(ring.piece(i & (DEPTH - 1), 1)), b);
    ask(i + DEPTH);
    turn.apply(a, b);
    *reinterpret_cast<uint4*>(out + ea) = pack8(a);
    *reinterpret_cast<uint4*>(out + eb) = pack8(b);
  }
}

__global__ void __launch_bounds__(THREADS) kv_norm_rope_write_kernel(const WriteParams p) {
  __shared__ uint4 pieces[DEPTH * 2 * THREADS];
  const Ring ring(pieces);
  if (p.cu) {
    // cumulative lengths: all of them, by every block; a bad one ends the call (a token's search
    // over an unsorted array can end on an interval that looks right)
    bool bad = false;
    for (int i = threadIdx.x; i < p.B; i += THREADS) {
      const int a = p.cu[i], z = p.cu[i + 1];
      bad |= (i == 0 && a != 0) || a < 0 || z < a || z > p.T;
    }
    if (__syncthreads_or(bad)) {
      if (threadIdx.x == 0 && blockIdx.x == 0) raise_dev_error(p.err, KD_DEV_BAD_SEQLENS);
      return;
    }
  }
  const unsigned all = (unsigned)p.T * (unsigned)p.items, step = gridDim.x * (THREADS / 32);
  for (unsigned i = blockIdx.x * (THREADS / 32) + threadIdx.x / 32; i < all; i += step) {
    const unsigned t = i / (unsigned)p.items;
    write_item(p, ring, t, i - t * (unsigned)p.items);
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
  int sms = 0, st = device_sms(&sms);
  if (st) return st;
  const int G = D <= 64 ? 4 : D <= 128 ? 8 : 16;
  // heads of a group: as many as leave every SM about 512 lanes of work, at most 8 (1088 tokens of 32 +
  // 8 heads of 128 5.3 us; with 256, 1024 or 2048 lanes 6.2, 5.9 and 7.5)
  int per = 8;
  while (per > 1 && (int64_t)T * (H + Hk) / per * G < (int64_t)sms * 512) per /= 2;
  nr::QkParams p;
  p.per = per;
  p.q = {q, q_weight, q_out, qt, qh, qot, qoh, H, (unsigned)(((int64_t)T * H + per - 1) / per)};
  p.k = {k, k_weight, k_out, kt, kh, kot, koh, Hk, (unsigned)(((int64_t)T * Hk + per - 1) / per)};
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
  const int64_t groups = (int64_t)p.q.groups + p.k.groups;
  const unsigned grid = (unsigned)((groups * G + nr::THREADS - 1) / nr::THREADS);
  // Groups stay inside a token where that leaves none of them short, else they span tokens:
  // 116186 tokens of 1 + 1 heads of 192 56 us against 78 inside, 30000 of 14 + 2 heads of 128 50
  // against 53; 16385 tokens of 32 + 8 heads 60 against 57, 20000 of 16 + 16 of 192 107 against 92.
  const bool span = H % per || Hk % per;
  const auto go = [&](auto inside, auto spanning) { (span ? spanning : inside)<<<grid, nr::THREADS, 0, stream>>>(p); };
  if (G == 4) go(nr::qk_norm_rope_kernel<4, false>, nr::qk_norm_rope_kernel<4, true>);
  else if (G == 8) go(nr::qk_norm_rope_kernel<8, false>, nr::qk_norm_rope_kernel<8, true>);
  else go(nr::qk_norm_rope_kernel<16, false>, nr::qk_norm_rope_kernel<16, true>);
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
  int sms = 0, st = device_sms(&sms);
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
  // query heads of a warp: as many as leave every SM about 8 warps of work, 8 to 64 (1088 tokens of
  // 64 heads 4.2 us; with 4, 16 or 32 warps 4.6, 5.8 and 6.0)
  p.per = 64;
  while (p.per > 8 && (int64_t)T * ((H + p.per - 1) / p.per) < (int64_t)sms * 8) p.per /= 2;
  p.items = H > p.per ? (H + p.per - 1) / p.per : 1;
  p.inter = interleaved;
  unsigned grid = (unsigned)(((int64_t)T * p.items + nr::THREADS / 32 - 1) / (nr::THREADS / 32));
  // Every block reads all cumulative lengths: of thousands of requests, so many that it pays to have
  // no more blocks than fit at once and several tokens for each (8192 requests of a token 15 us
  // against 19 with a block for every four tokens, 65536 104 against 402; 4096 10 and 10).
  if (cu && B >= 4096 && grid > (unsigned)sms * 7) grid = (unsigned)sms * 7;
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

// Eviction by accumulated attention weight: a request's cache cut down to its first
// `sink` slots, its last `recent` slots and the slots of the largest weights between.
//
// Two launches.  select_kernel (a cluster of up to 8 CTAs per request) finds the weight of
// the last slot that is kept, by a radix selection over order-preserving 32-bit keys (11 +
// 11 + 10 bits, a histogram in shared memory each, added up across the cluster through
// distributed shared memory; where at most 4096 keys share the first digit, every CTA fetches
// those and goes on by itself), and then walks the slots in order once, numbering the kept
// ones: equal weights are taken from the lowest slot.  It is bound by latency: about 15 us, 4 for
// a pass of the cluster (histogram 0.8, cluster barrier 0.9, 57 KB of the others' histograms 1
// to 2, scan 0.3), 5 for the other two by itself and 4 for the numbering; where a pass ends on a
// digit whose keys are all kept, the rest is left out.  Measured: three passes of the cluster 1 to
// 2 us more; 1024 threads of 32 registers and four slots each another 2; one CTA per request 66
// us for 32 K slots; rows already known to be kept prefetched into L2 during the passes 4 to 20
// more.
// The move copies the kept rows: bound by memory, 2 x 1152 bytes a row, 16 bytes per lane: 302
// MB in 46 us, 6.6 TB/s.  It is launched with the selection still running (programmatic
// dependent launch) and waits for it on the device.

#include "kd_common.cuh"
#include "kd_ptx.cuh"
#include "kd_slots.cuh"

namespace kd {
namespace ev {

constexpr int THREADS = 512, WARPS = THREADS / 32;
constexpr int BINS = 2048;
constexpr int PER = 8;                       // neighbouring slots a thread numbers per step
constexpr int CHUNK = THREADS * PER;         // slots a CTA works on per step
constexpr int MAXC = 8;                      // CTAs of a cluster
constexpr int MOST = 1 << 30;                // slots of a request: 32-bit numbers have room for a step more
constexpr int FEW = 4096;                    // keys of one first digit that every CTA goes on with by itself

// Unsigned key in the order of the weights: NaN lowest, -0 equal to +0.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);        // -0 + 0 = +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct SelectParams {
  const int32_t* lens;
  const float* w_in;
  float* w_out;
  int32_t *lens_out, *kept, *err;
  SlotMap src, dst;
  int64_t wi, wo;
  int keep, sink, recent;
};

// Inclusive sum over the block of one value per thread; `warp_sums` [WARPS].
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warp_sums, uint32_t& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  if (lane == 31) warp_sums[w] = v;
  __syncthreads();
  uint32_t s = lane < WARPS ? warp_sums[lane] : 0u;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += o;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  const uint32_t before = __shfl_sync(0xffffffffu, s, w ? w - 1 : 0);
  __syncthreads();                                    // warp_sums may be written again
  return v + (w ? before : 0u);
}

// A word of another CTA's shared memory.
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_cluster_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// CTA r of a cluster of cs takes the chunks r, r + cs, ... of its request's slots.
__global__ void __launch_bounds__(THREADS, 2) select_kernel(const SelectParams p, const int cs) {
  __shared__ __align__(16) uint32_t hist[3][BINS];
  __shared__ uint32_t warp_sums[WARPS];
  __shared__ uint32_t found[3], totals[2], counts[MAXC];
  __shared__ uint32_t list[FEW], listed;
  asm volatile("griddepcontrol.launch_dependents;");      // the move may come up and wait
  const int b = blockIdx.x / cs, tid = threadIdx.x;
  const int rank = cs > 1 ? (int)ptx::cluster_ctarank() : 0;
  const int64_t L64 = p.lens[b];
  int32_t* kept = p.kept + (size_t)b * p.keep;
  const int64_t fit = L64 < p.keep ? L64 : p.keep;
  int bad = 0;
  if (L64 < 0 || L64 > p.src.cap || fit > p.dst.cap) bad = KD_DEV_CACHE_FULL;
  if (!bad && p.src.pt) {                              // pages of every slot read or written
    bool out = false;
    for (int64_t q = tid; q * p.src.P < L64; q += THREADS)
      out |= !p.src.pages_ok(b, q * p.src.P, q * p.src.P + 1);
    for (int64_t q = tid; q * p.dst.P < fit; q += THREADS)
      out |= !p.dst.pages_ok(b, q * p.dst.P, q * p.dst.P + 1);
    if (__syncthreads_or(out)) bad = KD_DEV_BAD_PAGE;
  }
  if (bad) {                                           // the same in every CTA of the cluster
    if (rank == 0) {
      if (tid == 0) raise_dev_error(p.err, bad);
      for (int m = tid; m < p.keep; m += THREADS) kept[m] = -1;
    }
    return;
  }
  const int L = (int)L64, first = p.sink, last = L - p.recent;
  const float* w = p.w_in + (int64_t)b * p.wi;
  // a thread's PER neighbouring slots of a step; read once when one step covers the request
  const int span = cs * CHUNK, j0 = rank * CHUNK + tid * PER, steps = (L + span - 1) / span;
  float v[PER];
  auto load = [&](int step) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int j = step * span + j0 + i;
      v[i] = j < L ? w[j] : 0.f;
    }
  };
  load(0);
  uint32_t thr = 0, need = 0, mask = 0;                // keys whose bits of mask are above thr are kept, `need` equal to it
  if (L > p.keep && p.keep > p.sink + p.recent) {
    need = (uint32_t)(p.keep - p.sink - p.recent);
    for (int i = tid; i < 3 * BINS; i += THREADS) (&hist[0][0])[i] = 0u;
    if (tid == 0) listed = 0u;
    __syncthreads();
    // The next digit, from its histogram: thread t has the bins 2047 - 4t to 2044 - 4t, `h` their
    // counts, the largest digit's first: sums run from that.  True when every key of the digit is
    // kept: the rest does not matter.
    auto pick = [&](int pass, const uint32_t (&h)[4]) -> bool {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      uint32_t total;
      const uint32_t mine = (h[0] + h[1]) + (h[2] + h[3]);
      uint32_t above = block_scan(mine, warp_sums, total) - mine;
      if (above < need && above + mine >= need) {
        int i = 0;
#pragma unroll
        for (int k = 0; k < 3; ++k)
          if (i == k && above + h[k] < need) above += h[k], i = k + 1;
        found[0] = (uint32_t)(BINS - 1 - 4 * tid - i);
        found[1] = need - above;
        found[2] = i == 0 ? h[0] : i == 1 ? h[1] : i == 2 ? h[2] : h[3];
      }
      __syncthreads();
      thr |= found[0] << shift;
      need = found[1];
      mask |= (pass == 2 ? 1023u : 2047u) << shift;
      return found[2] == need;
    };
    auto counted = [&](int pass, uint32_t (&h)[4]) {   // the bins of this CTA
      const uint4 o = *reinterpret_cast<const uint4*>(&hist[pass][BINS - 4 - 4 * tid]);
      h[0] = o.w, h[1] = o.z, h[2] = o.y, h[3] = o.x;
    };
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t digits = pass == 2 ? 1023u : 2047u;
#pragma unroll 1
      for (int step = 0; step < steps; ++step) {
        if (steps > 1) load(step);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int j = step * span + j0 + i;
          const uint32_t key = order_key(v[i]);
          if (j >= first && j < last && (key & mask) == thr) atomicAdd(&hist[pass][(key >> shift) & digits], 1u);
        }
      }
      __syncthreads();
      if (cs > 1) ptx::cluster_sync();
      uint32_t h[4];
      counted(pass, h);
      const uint32_t at = ptx::smem_u32(&hist[pass][BINS - 4 - 4 * tid]);
      for (int r = 1; r < cs; ++r) {                   // the others', from the next one on
        const int q = rank + r < cs ? rank + r : rank + r - cs;
        const uint4 o = ld_cluster_v4(ptx::map_to_rank(at, (uint32_t)q));
        h[0] += o.w, h[1] += o.z, h[2] += o.y, h[3] += o.x;
      }
      if (pick(pass, h)) break;
      if (pass > 0 || cs == 1 || found[2] > (uint32_t)FEW) continue;

      // Few keys have that digit: every CTA looks at all of them and goes on without the others.
      const uint32_t few = found[2];
#pragma unroll 1
      for (int step = 0; step < steps; ++step) {
        if (steps > 1) load(step);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int j = step * span + j0 + i;
          const uint32_t key = order_key(v[i]);
          if (j >= first && j < last && (key & mask) == thr) list[atomicAdd(&listed, 1u)] = key;
        }
      }
      __syncthreads();
      ptx::cluster_sync();
      if (tid < cs) counts[tid] = ld_cluster_u32(ptx::map_to_rank(ptx::smem_u32(&listed), (uint32_t)tid));
      __syncthreads();
      uint32_t key[FEW / THREADS];
#pragma unroll
      for (int i = 0; i < FEW / THREADS; ++i) {
        uint32_t n = tid + i * THREADS;
        if (n < few) {
          int r = 0;
          while (r < cs - 1 && n >= counts[r]) n -= counts[r++];
          key[i] = ld_cluster_u32(ptx::map_to_rank(ptx::smem_u32(&list[min(n, FEW - 1u)]), (uint32_t)r));
        }
      }
#pragma unroll 1
      for (int next = 1; next < 3; ++next) {
        const int low = next == 1 ? 10 : 0;
#pragma unroll
        for (int i = 0; i < FEW / THREADS; ++i)
          if (tid + i * THREADS < (int)few && (key[i] & mask) == thr)
            atomicAdd(&hist[next][(key[i] >> low) & (next == 1 ? 2047u : 1023u)], 1u);
        __syncthreads();
        counted(next, h);
        if (pick(next, h)) break;
      }
      break;
    }
  }
  const bool all = L <= p.keep, none = !all && p.keep == p.sink + p.recent;
  float* wo = p.w_out + (int64_t)b * p.wo;
  uint32_t taken = 0, equal = 0;                       // before this step: above or forced, and equal
#pragma unroll 1
  for (int step = 0; step < steps; ++step) {
    if (steps > 1) load(step);
    const int at0 = step * span + j0;
    uint32_t kind[PER], mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int j = at0 + i;
      kind[i] = 0;
      if (j < L) {
        const uint32_t key = order_key(v[i]) & mask;
        if (all || j < first || j >= last || (!none && key > thr)) kind[i] = 1u << 16;
        else if (!none && key == thr) kind[i] = 1u;
      }
      mine += kind[i];
    }
    uint32_t total;
    uint32_t at = block_scan(mine, warp_sums, total) - mine;
    // every CTA has read its slots of this step before any weight is written (weights_out may
    // be weights_in), and the ones before it say where its own numbers start
    uint32_t before_t = 0, before_e = 0, all_t = total >> 16, all_e = total & 0xFFFFu;
    if (cs > 1) {
      if (tid == 0) totals[step & 1] = total;
      __syncthreads();
      ptx::cluster_sync();
      for (int r = 0; r < cs; ++r) {
        if (r == rank) continue;
        const uint32_t o = ld_cluster_u32(ptx::map_to_rank(ptx::smem_u32(&totals[step & 1]), (uint32_t)r));
        all_t += o >> 16;
        all_e += o & 0xFFFFu;
        if (r < rank) {
          before_t += o >> 16;
          before_e += o & 0xFFFFu;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t a = taken + before_t + (at >> 16), e = equal + before_e + (at & 0xFFFFu);
      if (kind[i] == 1u << 16 || (kind[i] == 1u && e < need)) {
        const uint32_t m = a + (e < need ? e : need);
        kept[m] = at0 + i;
        wo[m] = v[i];
      }
      at += kind[i];
    }
    taken += all_t;
    equal += all_e;
  }
  for (int m = (int)fit + rank * THREADS + tid; m < p.keep; m += cs * THREADS) kept[m] = -1;
  if (cs > 1) {
    __syncthreads();
    ptx::cluster_sync();                               // nobody leaves while its memory is read
  }
  if (tid == 0 && rank == 0) p.lens_out[b] = (int32_t)fit;   // (lens_out may be cache_lens)
}

struct MoveParams {
  const uint4 *c, *r;
  uint4 *cd, *rd;
  const int32_t* kept;
  SlotMap src, dst;
  int64_t sc, sr, dc, dr;          // row strides in 16-byte units
  int keep;
};
constexpr int CC = KD_D_C / 8, CR = KD_D_R / 8;    // 16-byte pieces of a row

// Another destination: a warp a row.  (Two, four and eight rows, their loads in flight together,
// took 2, 9 and 17 us more for 302 MB: so many rows are on their way anyway that the memory does
// better with them close together; stores that stay in the L2 cost another 2.)
constexpr int ROWS = 8;                              // of a CTA
__global__ void __launch_bounds__(32 * ROWS) move_kernel(const MoveParams p) {
  const int b = blockIdx.y, lane = threadIdx.x & 31, m = blockIdx.x * ROWS + (threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the selection is complete
  const int s = m < p.keep ? p.kept[(size_t)b * p.keep + m] : -1;
  if (s < 0) return;
  const int64_t from = p.src.row(b, s), to = p.dst.row(b, m);
  const uint4 v0 = __ldcs(p.c + from * p.sc + lane), v1 = __ldcs(p.c + from * p.sc + lane + 32);
  uint4 x = {};
  if (lane < CR) x = __ldcs(p.r + from * p.sr + lane);
  __stcs(p.cd + to * p.dc + lane, v0);
  __stcs(p.cd + to * p.dc + lane + 32, v1);
  if (lane < CR) __stcs(p.rd + to * p.dr + lane, x);
}

// In place: a CTA takes one 64-byte column slice of every row (four 16-byte pieces; 16
// slices of the latent, 2 of the rope key), so that rows of one slice move in order while
// the slices need no order between them.  Rows move down (kept[m] >= m, ascending): once
// the sources of rows [m0, m1) are read, nothing that is still to be read lies below row
// m1, so each step reads its rows, waits for the whole CTA to have read, and writes.  The next
// step's reads, all from m1 on, are on their way meanwhile, as are the numbers of the one after.
constexpr int PIECES = 4, SLICES = (CC + CR) / PIECES;
template <int SIZE, int STEP>                          // threads, rows of a thread and step
__global__ void __launch_bounds__(SIZE) move_inplace_kernel(const MoveParams p) {
  constexpr int AT_ONCE = SIZE / PIECES;
  const int b = blockIdx.y, sl = blockIdx.x, piece = threadIdx.x % PIECES, r = threadIdx.x / PIECES;
  const int32_t* kept = p.kept + (size_t)b * p.keep;
  const bool lat = sl < CC / PIECES;
  uint4* base = lat ? p.cd + sl * PIECES + piece : p.rd + (sl - CC / PIECES) * PIECES + piece;
  const int64_t stride = lat ? p.dc : p.dr;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the selection is complete
  // sources of the step at m0, -1 where nothing moves
  auto look = [&](int m0, int (&s)[STEP]) {
#pragma unroll
    for (int i = 0; i < STEP; ++i) {
      const int m = m0 + i * AT_ONCE + r;
      s[i] = m < p.keep ? kept[m] : -1;
      if (s[i] == m) s[i] = -1;                        // already in place
    }
  };
  auto read = [&](const int (&s)[STEP], uint4 (&v)[STEP]) {
#pragma unroll
    for (int i = 0; i < STEP; ++i)
      if (s[i] >= 0) v[i] = base[p.src.row(b, s[i]) * stride];
  };
  int s[STEP], s1[STEP], s2[STEP];
  uint4 v[STEP], v1[STEP];
  look(0, s);
  look(STEP * AT_ONCE, s1);
  read(s, v);
  for (int m0 = 0; m0 < p.keep; m0 += STEP * AT_ONCE) {
    look(m0 + 2 * STEP * AT_ONCE, s2);
    read(s1, v1);                                      // lies behind every row written so far, and in this step
    __syncthreads();
#pragma unroll
    for (int i = 0; i < STEP; ++i) {
      if (s[i] >= 0) base[p.dst.row(b, m0 + i * AT_ONCE + r) * stride] = v[i];
      s[i] = s1[i];
      s1[i] = s2[i];
      v[i] = v1[i];
    }
  }
}

}  // namespace ev
}  // namespace kd

using namespace kd;

// ================================================================== C ABI
static int evict_impl(const kd_bf16_t* c_kv, const kd_bf16_t* k_rope, int64_t sc, int64_t sr, const SlotMap& src,
                      const int32_t* cache_lens, const float* w_in, int64_t wi, int keep, int sink, int recent, int B,
                      kd_bf16_t* c_dst, kd_bf16_t* r_dst, int64_t dc, int64_t dr, const SlotMap& dst, bool inplace,
                      float* w_out, int64_t wo, int32_t* lens_out, int32_t* kept, int32_t* dev_error,
                      cudaStream_t stream) {
  if (!cache_ok(c_kv, k_rope, sc, sr, src.cap) || !cache_ok(c_dst, r_dst, dc, dr, dst.cap) || !cache_lens || !w_in ||
      !w_out || !lens_out || !kept || B < 1 || B > 65535 || keep < 1 || sink < 0 || recent < 0 ||
      (int64_t)sink + recent > keep || keep > ev::MOST || src.cap > ev::MOST || dst.cap > ev::MOST || wi < src.cap ||
      wo < (dst.cap < keep ? dst.cap : keep) || (w_out == w_in && wi != wo))
    return KD_EINVAL;
  int sms = 0, st = device_sms(&sms);
  if (st) return st;
  ev::SelectParams s;
  s.lens = cache_lens;
  s.w_in = w_in;
  s.w_out = w_out;
  s.lens_out = lens_out;
  s.kept = kept;
  s.err = dev_error;
  s.src = src;
  s.dst = dst;
  s.wi = wi;
  s.wo = wo;
  s.keep = keep;
  s.sink = sink;
  s.recent = recent;
  // CTAs for the longest request there can be, but no more than two per SM over all requests
  int cs = 1;
  while (cs < ev::MAXC && cs * (int64_t)ev::CHUNK < src.cap && 2 * cs * B <= 2 * sms) cs *= 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at;
  cfg.gridDim = dim3((unsigned)(B * cs));
  cfg.blockDim = dim3(ev::THREADS);
  cfg.stream = stream;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)cs;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if ((st = cuda_status(cudaLaunchKernelEx(&cfg, ev::select_kernel, s, cs), "select_kernel"))) return st;
  ev::MoveParams m;
  m.c = reinterpret_cast<const uint4*>(c_kv);
  m.r = reinterpret_cast<const uint4*>(k_rope);
  m.cd = reinterpret_cast<uint4*>(c_dst);
  m.rd = reinterpret_cast<uint4*>(r_dst);
  m.kept = kept;
  m.src = src;
  m.dst = dst;
  m.sc = sc / 8;
  m.sr = sr / 8;
  m.dc = dc / 8;
  m.dr = dr / 8;
  m.keep = keep;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  if (!inplace) {
    cfg.gridDim = dim3((unsigned)((keep + ev::ROWS - 1) / ev::ROWS), B);
    cfg.blockDim = dim3(32 * ev::ROWS);
    return cuda_status(cudaLaunchKernelEx(&cfg, ev::move_kernel, m), "move_kernel");
  }
  // Small CTAs where there are enough of them, else large ones that have more rows on their way: 64
  // caches of 9000 slots to 2048 take 76 and 87 us, 8 of 32768 to 16384 102 and 80 (140 and 137
  // by 512 threads of eight rows without reading ahead).
  const bool many = (int64_t)ev::SLICES * B >= 4 * (int64_t)sms;
  cfg.gridDim = dim3(ev::SLICES, B);
  cfg.blockDim = dim3(many ? 256 : 1024);
  return cuda_status(cudaLaunchKernelEx(&cfg, many ? ev::move_inplace_kernel<256, 4> : ev::move_inplace_kernel<1024, 2>, m),
                     "move_inplace_kernel");
}

// Whether the memory of two sets of rows (width elements each) meets.
static bool overlap(const kd_bf16_t* a, int64_t sa, const kd_bf16_t* b, int64_t sb, int width, int64_t na, int64_t nb) {
  if (na < 1 || nb < 1) return false;
  const kd_bf16_t *ea = a + (na - 1) * sa + width, *eb = b + (nb - 1) * sb + width;
  return a < eb && b < ea;
}

extern "C" int kd_kv_evict(const kd_bf16_t* c_kv, const kd_bf16_t* k_rope, int64_t sc, int64_t sr, int64_t cap,
                           const int32_t* cache_lens, const float* weights_in, int64_t w_in_stride, int keep, int sink,
                           int recent, int B, kd_bf16_t* c_dst, kd_bf16_t* r_dst, int64_t dst_row_stride_c,
                           int64_t dst_row_stride_r, int64_t dst_cap, float* weights_out, int64_t w_out_stride,
                           int32_t* lens_out, int32_t* kept, int32_t* dev_error, cudaStream_t stream) {
  const bool c_same = c_dst == c_kv, r_same = r_dst == k_rope;
  if (c_same != r_same || (c_same && (dst_row_stride_c != sc || dst_row_stride_r != sr || dst_cap != cap)))
    return KD_EINVAL;
  if (!c_same && B >= 1 && (overlap(c_kv, sc, c_dst, dst_row_stride_c, KD_D_C, B * cap, B * dst_cap) ||
                            overlap(k_rope, sr, r_dst, dst_row_stride_r, KD_D_R, B * cap, B * dst_cap)))
    return KD_EINVAL;
  return evict_impl(c_kv, k_rope, sc, sr, SlotMap{nullptr, cap, 0, 1, 0}, cache_lens, weights_in, w_in_stride, keep,
                    sink, recent, B, c_dst, r_dst, dst_row_stride_c, dst_row_stride_r,
                    SlotMap{nullptr, dst_cap, 0, 1, 0}, c_same, weights_out, w_out_stride, lens_out, kept, dev_error,
                    stream);
}

extern "C" int kd_kv_evict_paged(const kd_bf16_t* c_pages, const kd_bf16_t* r_pages, int64_t sc, int64_t sr,
                                 int page_size, const int32_t* page_table, int64_t pages_per_req, int64_t num_pages,
                                 const int32_t* cache_lens, const float* weights_in, int64_t w_in_stride, int keep,
                                 int sink, int recent, int B, kd_bf16_t* c_dst, kd_bf16_t* r_dst,
                                 int64_t dst_row_stride_c, int64_t dst_row_stride_r, const int32_t* dst_page_table,
                                 int64_t dst_pages_per_req, int64_t dst_num_pages, float* weights_out,
                                 int64_t w_out_stride, int32_t* lens_out, int32_t* kept, int32_t* dev_error,
                                 cudaStream_t stream) {
  if (!paged_ok(page_table, page_size, pages_per_req, num_pages) ||
      !paged_ok(dst_page_table, page_size, dst_pages_per_req, dst_num_pages))
    return KD_EINVAL;
  const bool c_same = c_dst == c_pages, r_same = r_dst == r_pages;
  const bool table_same = dst_page_table == page_table;
  if (c_same != r_same || (c_same && (dst_row_stride_c != sc || dst_row_stride_r != sr)) ||
      (c_same && table_same && (dst_pages_per_req != pages_per_req || dst_num_pages != num_pages)))
    return KD_EINVAL;
  return evict_impl(c_pages, r_pages, sc, sr,
                    SlotMap{page_table, pages_per_req * page_size, num_pages, page_size, (int)pages_per_req},
                    cache_lens, weights_in, w_in_stride, keep, sink, recent, B, c_dst, r_dst, dst_row_stride_c,
                    dst_row_stride_r,
                    SlotMap{dst_page_table, dst_pages_per_req * page_size, dst_num_pages, page_size,
                            (int)dst_pages_per_req},
                    c_same && table_same, weights_out, w_out_stride, lens_out, kept, dev_error, stream);
}

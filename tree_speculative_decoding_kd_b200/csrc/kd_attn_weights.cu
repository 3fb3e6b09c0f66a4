// Attention weight that each cache slot receives from the counted nodes (tcgen05 + TMEM +
// TMA):
//   col_j = sum over counted rows (node i, head h) that see slot j of exp(s_ihj - lse_ih).
//
// The scores are computed transposed, S^T = K Q^T: keys are the M rows of the MMA (the TMEM
// lanes), up to 256 query rows its N columns.  A thread of the epilogue then owns one key
// and adds up along its own columns: no reduction between threads, no second product, a
// fixed order.  With the rows' lse known, one pass is enough: nothing runs a maximum.
// Scores are summed up in fp32 by the tensor core, in 36 steps, whose roundings make the weights
// off by 4e-8 to 3.9e-6 of their 2-norm (fp32 products throughout: 3e-8 to 7e-7), most where
// scores reach 20; scale and lse held as two floats each did not change that.
//
// Two CTAs work as a pair (cta_group::2): M = 256 keys, 128 in each CTA's shared memory,
// while each CTA holds only half of the query rows.  The query rows then stream from L2 at
// 32 bytes a cycle and SM, half of what one CTA alone would need for the tensor pipe's rate.
// Shared memory is thirteen 16 KB stages of 64 columns: the unit's keys stay in nine of them,
// the query rows pass through four.  A chunk of keys is refilled for the next unit as soon as
// the last query tile has used it, so that with few rows (one query tile, as for an accepted
// path) the next unit's keys stream in behind this one's products.
// Measured (one B200): 4 x 16384 keys against 8192 rows 455 to 481 us (1.3 to 1.37 PFLOP/s at the
// power cap, 1.5 cold); the accepted paths of 64 requests 147 to 185 us (3.7 to 4.6 TB/s of keys;
// 178 with the next tile's path looked up only when its turn came).
// One CTA alone, with two 32 KB stages for the query rows, took 588 and 195 us.  Letting the
// keys pass through 6, 8, 10 or 11 of the stages instead of keeping them cost 3 to 20% for the
// accepted paths: fewer bytes of keys on their way, or too few query stages.
//
// A unit is (request, 256 keys); a cluster of 1, 2 or 4 pairs shares a unit by dealing the
// query tiles out among its pairs, whose sums meet in the first pair's shared memory.
//
// Query tiles hold whole nodes: rows of one node are contiguous in memory, nodes on an
// accepted path are not, so a stage is filled by one box per node, 16-row aligned.  When every
// node counts and H is a multiple of 16, one box fills the stage.
//
// Roles in each CTA: warp 0 loads K, warp 1 loads Q, warp 2 (one thread, even CTA) issues the
// MMAs, warp 3 stages the rows' lse and masks, warps 4 to 11 are the epilogue (two groups of
// four warps, taking the S tile's 32-column chunks in turn).  Two S tiles of 256 TMEM columns
// alternate.  Every wait is bounded (kd_pipe.cuh).  No TMA multicast.

#include <math.h>

#include <atomic>

#include "kd_pipe.cuh"
#include "kd_slots.cuh"
#include "kd_tmap.cuh"

namespace kd {
namespace aw {

using namespace ptx;

constexpr int THREADS = 384;
constexpr int BK = 128;                       // keys per CTA
constexpr int UK = 2 * BK;                    // keys per unit
constexpr int BN = 256;                       // query rows per tile
constexpr int NCH = 9;                        // 64-column chunks: 8 latent, 1 rope
constexpr int STAGE = BK * 128;               // bytes: 128 keys, or a CTA's half of the query rows
constexpr int NQ = 4;                         // stages of the query rows
constexpr int NS = 2;                         // S tiles in TMEM
constexpr int MAXP = 4;                       // pairs of a cluster

enum Bar {
  K_FULL = 0,                   // even CTA: both CTAs' chunk landed (TMA)
  K_FREE = K_FULL + NCH,        // chunk used for the last time (MMA commit, both CTAs)
  Q_FULL = K_FREE + NCH,        // even CTA: both halves landed
  Q_FREE = Q_FULL + NQ,         // stage used (both CTAs)
  Z_FULL = Q_FREE + NQ,         // lse and masks of the tile staged (32 arrivals)
  Z_FREE = Z_FULL + NS,         // the epilogue has read them (8 arrivals: a lane of each warp)
  S_FULL = Z_FREE + NS,         // S tile ready (both CTAs)
  S_FREE = S_FULL + NS,         // even CTA: S tile read in both CTAs (16 arrivals)
  P_FULL = S_FREE + NS,         // first pair: the others' sums of a unit arrived
  P_FREE = P_FULL + 2,          // other pairs: the first has read them
  DRAIN = P_FREE + 2,           // all MMAs done
  NBAR = DRAIN + 1
};
constexpr int OFF_ABORT = 512, OFF_TMEM = 516;
constexpr int OFF_Z = 1024;                             // f32 [NS][256]: -lse log2(e), -inf for a row that adds nothing
constexpr int OFF_NODE = OFF_Z + NS * BN * 4;           // u8 [NS][16]: node of each 16 columns
constexpr int OFF_VIS = OFF_NODE + 64;                 // u32 [NS][128][4]: masks of the tile's nodes, by place in the tile
constexpr int OFF_X = OFF_VIS + NS * 128 * 16;          // f32 [2][128]: sums of the second group
constexpr int OFF_PART = OFF_X + 2 * BK * 4;            // f32 [2][MAXP - 1][128]: sums of the other pairs
constexpr int OFF_STAGE = ((OFF_PART + 2 * (MAXP - 1) * BK * 4 + 1023) / 1024) * 1024;
constexpr int SMEM = OFF_STAGE + (NCH + NQ) * STAGE + 1024;
static_assert(NBAR * 8 <= OFF_ABORT && SMEM <= 232448, "shared memory");

struct Params {
  const int32_t *lens, *path, *len, *pt;
  const uint32_t* vis;
  const float *lse, *w_in;
  float* w_out;
  int32_t* err;
  int64_t cap, wi, wo, pages;
  int B, n, H, W, P, M;         // page size (0: contiguous) and pages per request
  int Hp, per_tile;             // rows a node takes in a tile, nodes per tile (even)
  int linear;                   // one box per stage: `linear` rows (0: a box per node)
  int kbox;                     // rows of a K box
  float scale_log2;
};

// Cursor over the units of this cluster: units are numbered request by request, cluster c
// takes c, c + clusters, ...  A warp looks at 32 requests at once.
struct Cursor {
  int b, kt;                    // current unit
  int64_t L;
  int count, tiles;             // counted nodes, query tiles
  int base, b0, incl, step, u;  // window of 32 requests: first request, units before it, inclusive sums
  int len_l, count_l;           // lane i: committed length and counted nodes of request b0 + i
  __device__ __forceinline__ static int bad_of(const Params& p, int64_t L, int count) {
    return L < 0 || L + p.n > p.cap ? KD_DEV_CACHE_FULL : count < 1 || count > p.n ? KD_DEV_BAD_PATH : 0;
  }
  __device__ __forceinline__ void window(const Params& p, int first) {
    b0 = first;
    const int i = b0 + (threadIdx.x & 31);
    len_l = i < p.B ? p.lens[i] : 0;
    count_l = i < p.B && p.path ? p.len[i] : p.n;
    // a request without work has one unit, which reports it
    incl = i >= p.B ? 0 : bad_of(p, len_l, count_l) ? 1 : (int)(((int64_t)len_l + p.n + UK - 1) / UK);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, d);
      if ((int)(threadIdx.x & 31) >= d) incl += o;
    }
  }
  __device__ __forceinline__ void start(const Params& p, int cluster, int clusters) {
    base = 0;
    u = cluster - clusters;
    step = clusters;
    window(p, 0);
  }
  // The next unit; false when there is none.  `bad`: KD_DEV_* bits of a request that has no work.
  __device__ __forceinline__ bool next(const Params& p, int& bad) {
    u += step;
    int total = __shfl_sync(0xffffffffu, incl, 31);
    while (u - base >= total) {
      base += total;
      if (b0 + 32 >= p.B) return false;
      window(p, b0 + 32);
      total = __shfl_sync(0xffffffffu, incl, 31);
    }
    const int at = u - base;
    const int i = __popc(__ballot_sync(0xffffffffu, incl <= at));
    b = b0 + i;
    const int before = __shfl_sync(0xffffffffu, incl, i ? i - 1 : 0);
    kt = at - (i ? before : 0);
    b = __shfl_sync(0xffffffffu, b, 0);                 // (uniform to the compiler too)
    L = __shfl_sync(0xffffffffu, len_l, i);
    count = __shfl_sync(0xffffffffu, count_l, i);
    bad = bad_of(p, L, count);
    tiles = bad ? 0 : (count + p.per_tile - 1) / p.per_tile;
    return true;
  }
};

// Node of place m on the path, kept inside [0, n) (a bad path is reported by the epilogue).
__device__ __forceinline__ int node_at(const Params& p, int b, int m) {
  if (!p.path) return m;
  const int k = p.path[(size_t)b * p.n + m];
  return k < 0 || k >= p.n ? 0 : k;
}

__device__ __forceinline__ uint64_t desc_of(uint32_t saddr) { return smem_desc_sw128(saddr, 16, 1024); }

// Adds exp2(s * scale + z) of four columns.
__device__ __forceinline__ void add4(float (&acc)[4], const uint32_t* s, const float4& z, float scale) {
  float a, b, c, d;
  ffma2v(a, b, __uint_as_float(s[0]), __uint_as_float(s[1]), scale, z.x, z.y);
  ffma2v(c, d, __uint_as_float(s[2]), __uint_as_float(s[3]), scale, z.z, z.w);
  fadd2(acc[0], acc[1], ex2(a), ex2(b));
  fadd2(acc[2], acc[3], ex2(c), ex2(d));
}

__global__ void __launch_bounds__(THREADS, 1)
weights_kernel(const __grid_constant__ CUtensorMap tm_qa, const __grid_constant__ CUtensorMap tm_qr,
               const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_r, const Params p,
               const int pairs) {
  extern __shared__ uint8_t dyn[];
  uint8_t* gbase = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
  const uint32_t base = smem_u32(gbase);
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank(), half = rank & 1, pr = rank >> 1;
  const int cluster = blockIdx.x / (2 * pairs), clusters = gridDim.x / (2 * pairs);
  const uint32_t k_at = base + OFF_STAGE, q_at = k_at + NCH * STAGE;
  const uint16_t both = (uint16_t)(3u << (rank & ~1));
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(gbase + OFF_ABORT);
  const Pipe pipe{base, abort_flag, p.err};
  auto even = [&](int bar) { return map_to_rank(pipe.bar(bar), (uint32_t)(rank & ~1)); };

  if (threadIdx.x == 0) *abort_flag = 0u;
  if (threadIdx.x < NBAR) {                             // a thread each: by one, 1600 cycles
    const int i = threadIdx.x;
    const int n = i >= Z_FULL && i < Z_FULL + NS ? 32 : i >= Z_FREE && i < Z_FREE + NS ? 8
                  : i >= S_FREE && i < S_FREE + NS ? 16 : i >= P_FULL && i < P_FULL + 2 && pairs > 1 ? 128 * (pairs - 1) : 1;
    mbar_init(base + 8 * i, n);
    fence_mbar_init();
  }
  if (warp == 3) {
    tmem_alloc_pair(base + OFF_TMEM, 512);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_qa);
    tma_prefetch_desc(&tm_qr);
    tma_prefetch_desc(&tm_c);
    tma_prefetch_desc(&tm_r);
  }
  Cursor cur;
  int bad;
  cur.start(p, cluster, clusters);
  tc_fence_before();
  __syncthreads();
  cluster_sync();                                       // barriers of all CTAs are ready
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(gbase + OFF_TMEM), 0);

  if (warp == 0) {
    // ------------------------------------------------------------ K
    uint32_t it = 0;                                    // units loaded
    bool ok = true;
    while (ok && cur.next(p, bad)) {
      if (bad || pr >= cur.tiles) continue;
      int64_t row[2];
      const int boxes = BK / p.kbox;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t key = (int64_t)cur.kt * UK + half * BK + i * p.kbox;
        if (!p.P) row[i] = (int64_t)cur.b * p.cap + key;
        else {
          const int64_t q = key / p.P;                  // pages past the last one, or bad ones: page 0
          const int32_t id = q < p.M ? p.pt[(size_t)cur.b * p.M + q] : 0;
          row[i] = (id < 0 || id >= p.pages ? 0 : (int64_t)id * p.P) + key % p.P;
        }
      }
      int c = 0;
      for (; c < NCH; ++c) {
        if (!(ok = pipe.wait_warp(K_FREE + c, (it & 1u) ^ 1u))) break;
        if (lane == 0) {
          const uint32_t bar = even(K_FULL + c);
          if (half == 0) mbar_arrive_expect_tx(pipe.bar(K_FULL + c), 2 * STAGE);
          for (int i = 0; i < boxes; ++i)
            tma_load_3d_pair(k_at + c * STAGE + i * p.kbox * 128, c < 8 ? &tm_c : &tm_r, c < 8 ? c * 64 : 0,
                             (int32_t)row[i], 0, bar);
        }
        __syncwarp();
      }
      if (ok) ++it;
      else if (half == 0)
        while (c-- > 0) pipe.drain(K_FULL + c, it & 1u);  // chunks of this unit that were asked for
    }
    // (the odd CTA's copies land on the even CTA's barriers; neither leaves before the other)
    if (it > 0 && half == 0)
      for (int c = 0; c < NCH; ++c) pipe.drain(K_FULL + c, (it - 1) & 1u);
  } else if (warp == 1) {
    // ------------------------------------------------------------ Q
    uint32_t it = 0;
    // The next tile of this pair, and what its stages take: looked up while the ring is full,
    // for the path costs a trip to memory.
    int t = 0, row = 0, bytes = 0;
    bool issue = false;
    cur.tiles = 0;
    auto advance = [&]() -> bool {
      t += pairs;
      while (t >= cur.tiles) {
        if (!cur.next(p, bad)) return false;
        t = pr;                                         // (a request without work has no tiles)
      }
      const int m0 = t * p.per_tile, nodes = min(p.per_tile, cur.count - m0), first = half * ((nodes + 1) >> 1);
      // This CTA's nodes: its half of the columns.  The odd CTA always has one, the last one
      // again where there is none for it: were a stage filled without it, the even CTA could
      // go round the stage's barriers once more before the odd one looked at them.
      const int mine = half ? max(1, nodes >> 1) : (nodes + 1) >> 1, boxes = ((nodes + 1) >> 1) + max(1, nodes >> 1);
      bytes = (p.linear ? 2 * p.linear : boxes * p.H) * 128;
      // lane i has the box of this CTA's node i (8 at most): first row of the flat [B n H] query
      row = p.linear ? (cur.b * p.n + m0 + first) * p.H
                     : (cur.b * p.n + node_at(p, cur.b, m0 + min(first + lane, nodes - 1))) * p.H;
      issue = p.linear ? lane == 0 : lane < mine;
      return true;
    };
    int row_now = 0, bytes_now = 0, c = NQ;
    bool issue_now = false, live = false, more = false;
    for (;;) {
      if (c == NQ) more = advance();                    // (first of all, too: no tile is live yet)
      if (!live || c == NCH) {
        if (!more) break;
        row_now = row, bytes_now = bytes, issue_now = issue;
        live = true;
        c = 0;
      }
      const uint32_t st = it % NQ;
      if (!pipe.wait_warp(Q_FREE + st, ((it / NQ) & 1u) ^ 1u)) break;
      const uint32_t bar = even(Q_FULL + st);
      if (lane == 0 && half == 0) mbar_arrive_expect_tx(pipe.bar(Q_FULL + st), bytes_now);
      __syncwarp();
      if (issue_now)
        tma_load_3d_pair(q_at + st * STAGE + lane * p.Hp * 128, c < 8 ? &tm_qa : &tm_qr, c < 8 ? c * 64 : 0, row_now, 0,
                         bar);
      __syncwarp();
      ++c;
      ++it;
    }
    if (half == 0)
      for (uint32_t j = it > NQ ? it - NQ : 0; j < it; ++j) pipe.drain(Q_FULL + j % NQ, (j / NQ) & 1u);
  } else if (warp == 2 && half == 0) {
    // ------------------------------------------------------------ MMA (one thread of the even CTA)
    uint32_t un = 0, qc = 0, ts = 0, ok = 1;            // units, chunks of query rows, tiles
    while (ok && cur.next(p, bad)) {
      if (bad || pr >= cur.tiles) continue;
      const int todo = (cur.tiles - pr + pairs - 1) / pairs;
      if (elect_one()) {
        uint32_t q = qc, s = ts;
        for (int t = 0; t < todo && ok; ++t, ++s) {
          const int nodes = min(p.per_tile, cur.count - (pr + t * pairs) * p.per_tile);
          const uint32_t idesc = idesc_bf16(UK, 2 * ((nodes + 1) >> 1) * p.Hp, 0, 0);
          const uint32_t sb = s % NS, d = tmem + sb * BN;
          if (!(ok = pipe.wait(S_FREE + sb, ((s / NS) & 1u) ^ 1u))) break;
          tc_fence_after();
          for (int c = 0; c < NCH; ++c, ++q) {
            const uint32_t st = q % NQ;
            if (t == 0 && !(ok = pipe.wait(K_FULL + c, un & 1u))) break;
            if (!(ok = pipe.wait(Q_FULL + st, (q / NQ) & 1u))) break;
            tc_fence_after();
            const uint64_t a = desc_of(k_at + c * STAGE), b = desc_of(q_at + st * STAGE);
#pragma unroll
            for (int i = 0; i < 4; ++i) mma_bf16_ss_pair(d, a + 2 * i, b + 2 * i, idesc, c + i > 0);
            tc_commit_pair(pipe.bar(Q_FREE + st), both);
            if (t + 1 == todo) tc_commit_pair(pipe.bar(K_FREE + c), both);
          }
          if (ok) tc_commit_pair(pipe.bar(S_FULL + sb), both);
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      ++un;
      qc += todo * NCH;
      ts += todo;
    }
    if (elect_one()) tc_commit_pair(pipe.bar(DRAIN), (uint16_t)(1u << rank));
    __syncwarp();
    pipe.drain(DRAIN, 0);                               // no MMA in flight when TMEM is released
  } else if (warp == 3) {
    // ------------------------------------------------------------ lse and masks
    uint32_t ts = 0;
    bool ok = true;
    while (ok && cur.next(p, bad)) {
      if (bad) continue;
      const bool tail = (int64_t)cur.kt * UK + half * BK + BK > cur.L;
      for (int t = pr; t < cur.tiles; t += pairs, ++ts) {
        const uint32_t sb = ts % NS;
        if (!(ok = pipe.wait_warp(Z_FREE + sb, ((ts / NS) & 1u) ^ 1u))) break;
        float* z = reinterpret_cast<float*>(gbase + OFF_Z) + sb * BN;
        uint8_t* node16 = gbase + OFF_NODE + sb * (BN / 16);
        uint32_t* vis = reinterpret_cast<uint32_t*>(gbase + OFF_VIS) + sb * 128 * 4;
        const int m0 = t * p.per_tile, nodes = min(p.per_tile, cur.count - m0);
#pragma unroll
        for (int j = lane; j < BN; j += 32) {
          const int i = j / p.Hp, h = j - i * p.Hp;
          float v = -INFINITY;
          if (i < nodes && h < p.H) {
            const float l = p.lse[((int64_t)cur.b * p.n + node_at(p, cur.b, m0 + i)) * p.H + h];
            v = l == -INFINITY ? -INFINITY : l * -1.4426950408889634f;
          }
          z[j] = v;
          if (tail && (j & 15) == 0) node16[j >> 4] = (uint8_t)(i < nodes ? i : 0);
        }
        if (tail)
          for (int i = lane; i < nodes; i += 32) {
            const uint32_t* row = p.vis + ((size_t)cur.b * p.n + node_at(p, cur.b, m0 + i)) * p.W;
            for (int w = 0; w < 4; ++w) vis[i * 4 + w] = w < p.W ? row[w] : 0u;
          }
        mbar_arrive(pipe.bar(Z_FULL + sb));
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int tid = threadIdx.x - 128, g = tid >> 7, r = tid & 127;       // group, key of the CTA
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    uint32_t ts = 0, un = 0;
    bool ok = true;
    while (cur.next(p, bad)) {
      if (bad) {
        if (tid == 0 && rank == 0) raise_dev_error(p.err, bad);
        continue;
      }
      // a group that gave up at the end of the last unit takes the other one with it
      if (pairs > 1 && named_bar_red_or(1, 256, !ok)) break;
      const int64_t key0 = (int64_t)cur.kt * UK + half * BK, key = key0 + r;
      const int k = key < cur.L ? -1 : (int)(key - cur.L);                // node of a tree slot
      const bool tail = key0 + BK > cur.L;
      // asked for before the scores are ready, looked at when they are summed up: what was
      // there, and every CTA's own look at the request's path and pages
      const float was = k < 0 && p.w_in && g == 0 ? p.w_in[(int64_t)cur.b * p.wi + key] : 0.f;
      const int node = p.path && r < cur.count ? p.path[(size_t)cur.b * p.n + r] : 0;
      bool bad_page = false;
      if (p.P)
        for (int64_t q = tid; q * p.P < cur.L + p.n; q += 256) {
          const int32_t id = p.pt[(size_t)cur.b * p.M + q];
          bad_page |= id < 0 || id >= p.pages;
        }
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      for (int t = pr; t < cur.tiles; t += pairs, ++ts) {
        const uint32_t sb = ts % NS, par = (ts / NS) & 1u;
        const int rows = min(p.per_tile, cur.count - t * p.per_tile) * p.Hp;
        ok = pipe.wait(Z_FULL + sb, par) && pipe.wait(S_FULL + sb, par);
        if (named_bar_red_or(1, 256, !ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float* z = reinterpret_cast<const float*>(gbase + OFF_Z) + sb * BN;
        const uint32_t src = tmem + lanes + sb * BN;
        if (!tail && p.Hp == p.H) {
          int j = g * 32;
          for (; j + 32 <= rows; j += 64) {
            uint32_t s[32];
            tmem_ld32(src + j, s);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; i += 4) add4(acc, s + i, *reinterpret_cast<const float4*>(z + j + i), p.scale_log2);
          }
          if (j < rows) {                               // 16 columns are left
            uint32_t s[16];
            tmem_ld16(src + j, s);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; i += 4) add4(acc, s + i, *reinterpret_cast<const float4*>(z + j + i), p.scale_log2);
          }
        } else {
          // sixteen columns are of one node: seen or not together
          const uint8_t* node16 = gbase + OFF_NODE + sb * (BN / 16);
          const uint32_t* vis = reinterpret_cast<const uint32_t*>(gbase + OFF_VIS) + sb * 128 * 4;
          for (int j = g * 32; j < rows; j += 64)
            for (int q = j; q < j + 32 && q < rows; q += 16) {
              uint32_t s[16];
              tmem_ld16(src + q, s);
              const bool see = k < 0 || (k < p.n && (vis[node16[q >> 4] * 4 + (k >> 5)] >> (k & 31) & 1u));
              tmem_wait_ld();
              float part[4] = {0.f, 0.f, 0.f, 0.f};
              if (p.Hp == p.H) {
#pragma unroll
                for (int i = 0; i < 16; i += 4) add4(part, s + i, *reinterpret_cast<const float4*>(z + q + i), p.scale_log2);
              } else {                                  // rows that pad a node hold whatever was there before
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  part[i & 3] += z[q + i] != -INFINITY ? ex2(__uint_as_float(s[i]) * p.scale_log2 + z[q + i]) : 0.f;
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[i] += see ? part[i] : 0.f;
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(pipe.bar(Z_FREE + sb));
          mbar_arrive_remote_tmem(even(S_FREE + sb));
        }
      }
      if (!ok) break;
      // the two groups' sums, then the other pairs' in order
      float sum = (acc[0] + acc[1]) + (acc[2] + acc[3]);
      float* x = reinterpret_cast<float*>(gbase + OFF_X) + (un & 1) * BK;
      if (g == 1) x[r] = sum;
      const bool bad_node = node < 0 || node >= p.n;
      if (bad_node) raise_dev_error(p.err, KD_DEV_BAD_PATH);
      if (bad_page) raise_dev_error(p.err, KD_DEV_BAD_PAGE);
      const bool out = named_bar_red_or(1, 256, bad_node || bad_page);
      const uint32_t slot = un & 1, turn = (un >> 1) & 1u;
      ++un;
      if (g == 0) {
        sum += x[r];
        if (pr > 0) {
          if (!(ok = __all_sync(0xffffffffu, pipe.wait_remote(P_FREE + slot, turn ^ 1u)))) continue;
          const uint32_t to = map_to_rank(base + OFF_PART + ((slot * (MAXP - 1) + pr - 1) * BK + r) * 4, (uint32_t)half);
          st_cluster_u32(to, __float_as_uint(sum));
          mbar_arrive_remote(map_to_rank(pipe.bar(P_FULL + slot), (uint32_t)half));
        } else {
          if (pairs > 1) {
            ok = pipe.wait_remote(P_FULL + slot, turn);
            const float* part = reinterpret_cast<const float*>(gbase + OFF_PART) + slot * (MAXP - 1) * BK;
            for (int i = 0; i < pairs - 1; ++i) sum += part[i * BK + r];
            if (named_bar_red_or(2, 128, !ok)) {        // everyone has read the parts, or gives up
              ok = false;
              continue;
            }
            // (before the weights are stored: the arrival would wait for that)
            if (r < pairs - 1) mbar_arrive_remote(map_to_rank(pipe.bar(P_FREE + slot), (uint32_t)(2 * (r + 1) + half)));
          }
          if (!out) {
            float* wo = p.w_out + (int64_t)cur.b * p.wo;
            if (k < 0) wo[key] = sum + was;
            else if (k < p.n) {
              if (!p.path) wo[key] = sum;
              else
                for (int m = 0; m < cur.count; ++m)
                  if (p.path[(size_t)cur.b * p.n + m] == k) wo[cur.L + m] = sum;
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                       // no CTA leaves, or frees its TMEM, while another works on it
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
  __syncwarp();
  cluster_sync();
}

}  // namespace aw
}  // namespace kd

using namespace kd;

// Clusters of `c` CTAs (2, 4 or 8) that fit on the device at once (cached per device).
static int active_clusters(int c, int sms) {
  static std::atomic<int> cached[64][3];
  int dev = 0;
  const int slot = c == 2 ? 0 : c == 4 ? 1 : 2;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return sms / c;
  int v = cached[dev][slot].load(std::memory_order_relaxed);
  if (v > 0) return v;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(sms / c * c));
  cfg.blockDim = dim3(aw::THREADS);
  cfg.dynamicSmemBytes = aw::SMEM;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)c;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  int nc = 0;
  v = sms / c;
  if (cudaOccupancyMaxActiveClusters(&nc, aw::weights_kernel, &cfg) == cudaSuccess && nc > 0) v = nc;
  cudaGetLastError();
  cached[dev][slot].store(v, std::memory_order_relaxed);
  return v;
}

static int weights_impl(const kd_bf16_t* qa, const kd_bf16_t* qr, const kd_bf16_t* c, const kd_bf16_t* r, int64_t sc,
                        int64_t sr, int64_t cap, int64_t cache_rows, const int32_t* pt, int page, int64_t M,
                        int64_t pages, const int32_t* lens, const uint32_t* vis, const float* lse, const int32_t* path,
                        const int32_t* len, int B, int n, int H, float scale, const float* w_in, int64_t wi,
                        float* w_out, int64_t wo, int32_t* dev_error, cudaStream_t stream) {
  if (!qa || !qr || !lens || !vis || !lse || !w_out || !shapes_ok(B, n) || B > 65535 || H < 1 || H > KD_MAX_HEADS ||
      !cache_ok(c, r, sc, sr, cap) || !aligned16(qa) || !aligned16(qr) || !(scale > 0.f && isfinite(scale)) ||
      (path != nullptr) != (len != nullptr) || wo < cap || (w_in && wi < cap) || (w_in == w_out && wi != wo) ||
      (int64_t)B * n * H > INT32_MAX || cache_rows > INT32_MAX)
    return KD_EINVAL;
  int sms = 0, st = device_sms(&sms);
  if (st) return st;
  int dev = 0;
  if ((st = cuda_status(cudaGetDevice(&dev), "cudaGetDevice"))) return st;
  static std::once_flag once[64];
  static std::atomic<int> attr[64];
  std::call_once(once[dev], [&] {
    attr[dev].store(cuda_status(cudaFuncSetAttribute(aw::weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     aw::SMEM),
                                "cudaFuncSetAttribute(weights_kernel)"));
  });
  if ((st = attr[dev].load())) return st;

  aw::Params p;
  p.lens = lens;
  p.path = path;
  p.len = len;
  p.pt = pt;
  p.vis = vis;
  p.lse = lse;
  p.w_in = w_in;
  p.w_out = w_out;
  p.err = dev_error;
  p.cap = cap;
  p.wi = wi;
  p.wo = wo;
  p.pages = pages;
  p.B = B;
  p.n = n;
  p.H = H;
  p.W = (n + 31) / 32;
  p.P = pt ? page : 0;
  p.M = (int)M;
  p.Hp = (H + 15) / 16 * 16;
  p.per_tile = aw::BN / p.Hp & ~1;
  const int64_t rows = (int64_t)B * n * H;
  p.linear = !path && H % 16 == 0 ? ((p.per_tile < n ? p.per_tile : n) + 1) / 2 * H : 0;
  p.kbox = pt && page < aw::BK ? page : aw::BK;
  p.scale_log2 = scale * 1.4426950408889634f;
  const uint32_t qbox = (uint32_t)(p.linear ? p.linear : H);
  CUtensorMap tqa, tqr, tc, tr;
  if ((st = make_tmap3(&tqa, qa, KD_D_C, (uint64_t)rows, 1, KD_D_C, 0, qbox, 1))) return st;
  if ((st = make_tmap3(&tqr, qr, KD_D_R, (uint64_t)rows, 1, KD_D_R, 0, qbox, 1))) return st;
  if ((st = make_tmap3(&tc, c, KD_D_C, (uint64_t)cache_rows, 1, sc, 0, (uint32_t)p.kbox, 1))) return st;
  if ((st = make_tmap3(&tr, r, KD_D_R, (uint64_t)cache_rows, 1, sr, 0, (uint32_t)p.kbox, 1))) return st;

  // Pairs of a cluster: the number with the shortest longest run of query tiles, were every
  // request of length cap.  A path is short as a rule (acceptance ends within a few nodes), so
  // it counts as at most four nodes: a guess, not measured against paths that are long.
  const int64_t units = B * ((cap + aw::UK - 1) / aw::UK);
  const int nodes = path && n > 4 ? 4 : n;
  const int64_t qt = (nodes + p.per_tile - 1) / p.per_tile;
  int best = 1, fit = 0;
  double cost = 1e300;
  for (int c = 1; c <= aw::MAXP; c *= 2) {
    if (c > 1 && c > qt) break;
    const int nc = active_clusters(2 * c, sms);
    const double t = (double)((units + nc - 1) / nc) * ((double)((qt + c - 1) / c) + 0.3);
    if (t < 0.95 * cost) cost = t, best = c, fit = nc;
  }
  if (units > INT32_MAX) return KD_EINVAL;
  const int64_t clusters = units < fit ? units : fit;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * 2 * best));
  cfg.blockDim = dim3(aw::THREADS);
  cfg.dynamicSmemBytes = aw::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)(2 * best);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, aw::weights_kernel, tqa, tqr, tc, tr, p, best), "weights_kernel");
}

extern "C" int kd_kv_attn_weights(const kd_bf16_t* q_nope_absorbed, const kd_bf16_t* q_rope, const kd_bf16_t* c_kv,
                                  const kd_bf16_t* k_rope, int64_t sc, int64_t sr, int64_t cap,
                                  const int32_t* cache_lens, const uint32_t* vis, const float* lse,
                                  const int32_t* path, const int32_t* len, int B, int n, int H, float scale,
                                  const float* weights_in, int64_t w_in_stride, float* weights_out,
                                  int64_t w_out_stride, int32_t* dev_error, cudaStream_t stream) {
  return weights_impl(q_nope_absorbed, q_rope, c_kv, k_rope, sc, sr, cap, B * cap, nullptr, 0, 0, 0, cache_lens, vis,
                      lse, path, len, B, n, H, scale, weights_in, w_in_stride, weights_out, w_out_stride, dev_error,
                      stream);
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
  return weights_impl(q_nope_absorbed, q_rope, c_pages, r_pages, sc, sr, pages_per_req * page_size,
                      num_pages * page_size, page_table, page_size, pages_per_req, num_pages, cache_lens, vis, lse,
                      path, len, B, n, H, scale, weights_in, w_in_stride, weights_out, w_out_stride, dev_error, stream);
}

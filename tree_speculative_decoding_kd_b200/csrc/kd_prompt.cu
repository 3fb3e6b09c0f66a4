// Causal attention of packed prompts with grouped heads (tcgen05 + TMEM + TMA).
//
//   s_ij = scale (q_i . k_j), j <= i + nk - nq;  out_i = softmax(s_i) . v;  lse_i = ln sum exp s_ij
//
// A unit is (sequence, 256 query rows, head): two 128-row tiles that share every key and
// value tile of 128 keys.  PACK: a tile's rows are 128 / G tokens, each with the G heads
// of one key head.  Each tile has its own score tile S (128 TMEM columns) and output
// O (128 columns), 512 columns in all, and its own four softmax warps (a thread per row), so
// that one tile's products run while the other's exponentials do.
//
// One thread issues all products, in the order PV0 QK0 PV1 QK1.  At N = 128 its own scalar
// work is what can keep the tensor pipe waiting (an MMA takes 64 cycles, its issue 72): no
// votes, no divisions, a wait per hand-over, operands in uniform registers.  (Two issuing
// threads, one per tile, reach the pipe's full rate but share it MMA by MMA, which brings the
// two tiles into step, both in their products and then both in their exponentials: 1520 us
// where one thread takes 1000.)
//
// Per key tile the softmax warps take the row maximum from S and write P = exp2(s - m) in
// bf16 over S's own columns, where it is the second product's A operand from TMEM; the first
// half of the keys is handed over while the second is still being computed.  S is read twice:
// held in registers from the maximum to the exponentials, it would leave no room to keep more
// than a few of those in flight (4%).  The running maximum m only moves when it would rise by
// more than 8 (log2): P stays below 2^8 and O is rescaled rarely, by the softmax warps
// themselves, between two products (the commit that announced S also covers every earlier
// product into O).  The sum is kept in fp32 from the unrounded exponentials; the rounding of P
// to bf16 is the type of the MMA's operand: outputs are off by 2.0e-3 of their 2-norm where fp32
// products throughout give 1.6e-3, the output's own rounding to bf16.
//
// Shared memory: Q (two tiles of 128 rows), then a ring of 16 KB chunks through which keys
// (128 keys x 64 columns) and values (64 keys x 128 columns) stream in the order they are
// used.  Values past a sequence's last key are cleared before they meet P = 0: what lies there
// belongs to another sequence.
//
// The grid has a block per possible unit, longest first inside a sequence; a block that is
// done takes over the next one that has not started (cluster launch control), late, so that
// no block holds units it has not begun while others are idle (6%), and early enough that the
// next unit's queries load and its scores begin while the last one's output is written.
//
// Measured (one B200, calls behind each other; the longer two at the 1000 W cap, 1.4 to 1.6
// GHz): one prompt of 16384 tokens, 16 query heads on 2 key heads of 128: 980 to 1040 us (1.06 to
// 1.12 PFLOP/s, 1.29 in a call by itself); 4 prompts of 2000 to 3070 tokens, 64 heads of 192/128:
// 585 to 632 us (0.87 to 0.94, 1.11); 32 prompts of 1 to 300 tokens, 64 heads of 192/128: 86 to
// 101 us, where its inputs and outputs are 352 MB, 54 us.  What bounds it: the chain of one tile (scores, maximum,
// exponentials, the two products' hand-overs, about 2900 cycles a key tile where the products
// of both tiles take 2050 to 2560), and the power cap.
//
// Every wait is bounded (kd_pipe.cuh).  No TMA multicast.

#include <math.h>

#include <atomic>

#include "kd_pipe.cuh"
#include "kd_tmap.cuh"

namespace kd {
namespace pr {

using namespace ptx;

constexpr int THREADS = 384;        // warps 0-3 softmax of tile 0, 4-7 of tile 1, 8 TMA, 9 MMA, 10 clears, 11 units
constexpr int BM = 128, BN = 128;
constexpr int CHUNK = 16384;
constexpr int NS = 2;               // unit slots
constexpr int NO = 4;               // barriers of key (value) tiles in flight: a power of two, at least what the ring holds

enum Bar {
  K_FULL = 0,                       // [NO] a key tile's keys landed (TMA)
  K_FREE = K_FULL + NO,             // [NO] both query tiles' scores are done
  V_FULL = K_FREE + NO,             // [NO] its values
  V_FREE = V_FULL + NO,             // [NO]
  V_CLEAN = V_FREE + NO,            // the rows past a sequence's last key are cleared
  V_GO = V_CLEAN + 1,               // that tile is the next its barrier will announce
  Q_FULL = V_GO + 1,                // [2]
  Q_FREE = Q_FULL + 2,              // [2] the unit's last QK MMA of the tile is done
  S_FULL = Q_FREE + 2,              // [2]
  P_FULL = S_FULL + 2,              // [2][2] half of P written (128 arrivals)
  O_DONE = P_FULL + 4,              // [2] the unit's last PV MMA of the tile is done
  U_FULL = O_DONE + 2,              // [NS] unit published
  U_FREE = U_FULL + NS,             // [NS] unit read (11 arrivals: a lane of each other warp)
  GO = U_FREE + NS,                    // the unit's last loads are near: time to claim the next one
  CLC = GO + 1,                     // the next block's answer arrived
  DRAIN = CLC + 1,
  NBAR = DRAIN + 1
};
constexpr int OFF_ABORT = 512, OFF_TMEM = 516, OFF_CLC = 528, OFF_UNIT = 544;
constexpr int CTRL = 1024;
constexpr int SMEM = CTRL + 1024 + 14 * CHUNK;      // Q and ring: 6 + 8 or 4 + 10 chunks
static_assert(NBAR * 8 <= OFF_ABORT && OFF_UNIT + NS * 32 <= CTRL && SMEM <= 232448, "shared memory");

struct Params {
  const int32_t *cu_q, *cu_k;
  uint16_t* out;
  float* lse;
  int32_t* err;
  int B, T, Tk, H, slots;
  int packed, tokens;                 // a tile's rows are `tokens` (128 / packed) tokens of `packed` heads each
  int heads, group;                   // units beside each other (H / packed), of which `group` share a key head
  int k_heads, r_heads, v_heads;      // 0: one head for all (head coordinate 0)
  float scale, scale_log2;
};

// What a unit is; n[i]: key tiles of query tile i.
struct Unit {
  int q0, nq, k0, nk, row, head;      // row: first token of the unit inside its sequence; head: among p.heads
  int n0, n1;
  __device__ __forceinline__ int tiles(int i) const { return i ? n1 : n0; }
};

// Chunk index inside a ring of N.
template <int N>
__device__ __forceinline__ uint32_t wrap(uint32_t x) { return x >= N ? x - N : x; }

// Key tiles that the `rows` tokens from `row` on see.
__device__ __forceinline__ int tiles_of(int nq, int nk, int row, int rows) {
  if (row >= nq) return 0;
  const int last = min(row + rows, nq) - 1;
  const int keys = min((int64_t)nk, (int64_t)last + nk - nq + 1);
  return keys > 0 ? (keys + BN - 1) / BN : 0;
}

__device__ __forceinline__ uint64_t desc_k(uint32_t a) { return smem_desc_sw128(a, 16, 1024); }
__device__ __forceinline__ uint64_t desc_v(uint32_t a) { return smem_desc_sw128(a, 8192, 1024); }

// A value all lanes hold, as one the compiler knows to be the same in all of them: what the
// MMAs' operands and the loops around them are made of then stays in uniform registers.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

__device__ __forceinline__ Unit read_unit(const uint8_t* gbase, int k) {
  const int4* s = reinterpret_cast<const int4*>(gbase + OFF_UNIT + (k % NS) * 32);
  const int4 a = s[0], b = s[1];
  return Unit{uniform(a.x), uniform(a.y), uniform(a.z), uniform(a.w),
              uniform(b.x), uniform(b.y), uniform(b.z), uniform(b.w)};
}

// The first `n` of 32 columns stay, the others become -inf.
__device__ __forceinline__ void mask32(uint32_t (&s)[32], int n) {
#pragma unroll
  for (int c = 0; c < 32; ++c) s[c] = c < n ? s[c] : 0xff800000u;
}

// P of N columns: exponentials of s, rounded to bf16 in pk, summed up in (l0, l1).
template <int N>
__device__ __forceinline__ void exp_columns(const uint32_t (&s)[N], uint32_t (&pk)[N / 2], float scale, float nm,
                                            float& l0, float& l1) {
#pragma unroll
  for (int c = 0; c < N / 2; ++c) {
    float a, b;
    ffma2(a, b, __uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1]), scale, nm);
    a = ex2(a);
    b = ex2(b);
    fadd2(l0, l1, a, b);
    pk[c] = pack_bf16x2(a, b);
  }
}

// Maximum of N columns, in four chains (the latency of one would show).
template <int N>
__device__ __forceinline__ float max_columns(const uint32_t* s) {
  float mv[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) mv[q] = fmaxf(__uint_as_float(s[2 * q]), __uint_as_float(s[2 * q + 1]));
#pragma unroll
  for (int c = 8; c < N; c += 8)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      mv[q] = fmax3(mv[q], __uint_as_float(s[c + 2 * q]), __uint_as_float(s[c + 2 * q + 1]));
  return fmaxf(fmaxf(mv[0], mv[1]), fmaxf(mv[2], mv[3]));
}

// Asks the hardware for a block that has not started; the answer lands at `dst` and completes 16 bytes on `bar`.
__device__ __forceinline__ void try_cancel(uint32_t dst, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(dst),
               "r"(bar)
               : "memory");
}
// Block index in the answer, -1 when none was left.
__device__ __forceinline__ int cancelled_block(uint32_t src) {
  uint32_t ok, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\t.reg .b32 y, z, w;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\tmov.b32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, h;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(src)
      : "memory");
  return ok ? (int)x : -1;
}

template <bool ROPE, bool PACK>
__global__ void __launch_bounds__(THREADS, 1)
prompt_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_qr,
              const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_kr,
              const __grid_constant__ CUtensorMap tm_v, const Params p) {
  constexpr int KC = ROPE ? 3 : 2;            // 64-column chunks of a key
  constexpr int RING = ROPE ? 8 : 10;
  const int packed = PACK ? p.packed : 1, tokens = PACK ? p.tokens : BM;
  extern __shared__ uint8_t dyn[];
  uint8_t* gbase = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
  const uint32_t base = smem_u32(gbase);
  const uint32_t q_smem = base + CTRL, ring = q_smem + 2 * KC * CHUNK;
  const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(gbase + OFF_ABORT);
  const Pipe pipe{base, abort_flag, p.err};

  // cumulative lengths: all of them, by every block; a bad one ends the call
  bool bad = false;
  for (int b = threadIdx.x; b < p.B; b += THREADS) {
    const int a = p.cu_q[b], z = p.cu_q[b + 1];
    bad |= (b == 0 && a != 0) || a < 0 || z < a || z > p.T;
    if (p.cu_k) {
      const int ka = p.cu_k[b], kz = p.cu_k[b + 1];
      bad |= (b == 0 && ka != 0) || ka < 0 || kz < ka || kz > p.Tk;
    } else {
      bad |= z > p.Tk;
    }
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0 && blockIdx.x == 0) raise_dev_error(p.err, KD_DEV_BAD_SEQLENS);
    return;
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0u;
    for (int i = 0; i < NBAR; ++i) {
      const int n = i >= P_FULL && i < P_FULL + 4 ? 128
                    : i >= U_FREE && i < U_FREE + NS ? 11 : 1;
      mbar_init(base + 8 * i, n);
    }
    fence_mbar_init();
  }
  if (warp == 11) {
    tmem_alloc(base + OFF_TMEM, 512);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    if (ROPE) {
      tma_prefetch_desc(&tm_qr);
      tma_prefetch_desc(&tm_kr);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*reinterpret_cast<volatile uint32_t*>(gbase + OFF_TMEM));
  const uint32_t t_s = tmem, t_o = tmem + 2 * BN;

  if (warp == 11) {
    // ------------------------------------------------------------ units
    int u = (int)blockIdx.x, k = 0, asks = 0;
    bool ok = true;
    while (true) {
      // unit u: slot (two tiles' tokens) and head; sequence b has the slots from
      // cu[b] / (2 tokens) + b on
      const int slot = p.slots - 1 - u / p.heads, head = u % p.heads;
      int lo = 0, hi = p.B - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.cu_q[mid] / (2 * tokens) + mid <= slot) lo = mid;
        else hi = mid - 1;
      }
      Unit w;
      w.q0 = p.cu_q[lo];
      w.nq = p.cu_q[lo + 1] - w.q0;
      w.k0 = p.cu_k ? p.cu_k[lo] : w.q0;
      w.nk = p.cu_k ? p.cu_k[lo + 1] - w.k0 : w.nq;
      const int64_t row = (int64_t)(slot - w.q0 / (2 * tokens) - lo) * (2 * tokens);
      if (row >= 0 && row < w.nq) {
        w.row = (int)row;
        if (!(ok = pipe.wait_warp(U_FREE + k % NS, ((k / NS) & 1) ^ 1))) break;
        if (lane == 0) {
          int4* s = reinterpret_cast<int4*>(gbase + OFF_UNIT + (k % NS) * 32);
          s[0] = make_int4(w.q0, w.nq, w.k0, w.nk);
          s[1] = make_int4(w.row, head, tiles_of(w.nq, w.nk, w.row, tokens),
                           tiles_of(w.nq, w.nk, w.row + tokens, tokens));
          mbar_arrive(pipe.bar(U_FULL + k % NS));
        }
        __syncwarp();
        // claimed late: a block that holds units it has not begun leaves the others idle at the end
        if (!(ok = pipe.wait_warp(GO, k & 1))) break;
        ++k;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(pipe.bar(CLC), 16);
        try_cancel(base + OFF_CLC, pipe.bar(CLC));
      }
      __syncwarp();
      if (!(ok = pipe.wait_warp(CLC, asks & 1))) {
        pipe.drain(CLC, asks & 1);
        break;
      }
      ++asks;
      u = cancelled_block(base + OFF_CLC);
      fence_proxy_async_cta();                          // read before the next answer is written
      __syncwarp();
      if (u < 0) break;
    }
    if (ok && pipe.wait_warp(U_FREE + k % NS, ((k / NS) & 1) ^ 1)) {
      if (lane == 0) {
        reinterpret_cast<int4*>(gbase + OFF_UNIT + (k % NS) * 32)[0] = make_int4(-1, 0, 0, 0);
        mbar_arrive(pipe.bar(U_FULL + k % NS));
      }
      __syncwarp();
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ loads
    uint32_t kt = 0, nk = 0, nv = 0, nq[2] = {0, 0};    // key tiles; keys, values and queries asked for
    uint32_t pos = 0, used = 0, fk = 0, fv = 0;         // ring: next chunk, chunks held; keys and values freed
    bool ok = true;
    // makes room for `chunks` more; what is freed is freed in the order it was loaded
    auto room = [&](uint32_t chunks) -> bool {
      while (used + chunks > RING) {
        if (fk == fv) {
          if (!pipe.wait_warp(K_FREE + fk % NO, (fk / NO) & 1u)) return false;
          ++fk;
          used -= KC;
        } else {
          if (!pipe.wait_warp(V_FREE + fv % NO, (fv / NO) & 1u)) return false;
          ++fv;
          used -= 2;
        }
      }
      used += chunks;
      return true;
    };
    for (int k = 0; ok; ++k) {
      if (!(ok = pipe.wait_warp(U_FULL + k % NS, (k / NS) & 1))) break;
      const Unit u = read_unit(gbase, k);
      __syncwarp();
      if (lane == 0) mbar_arrive(pipe.bar(U_FREE + k % NS));
      if (u.q0 < 0) break;
      const int g = u.head / p.group, n = max(u.n0, u.n1);
      if (n == 0 && lane == 0) mbar_arrive(pipe.bar(GO));
      auto load_q = [&](int i) -> bool {
        if (u.tiles(i) == 0) return true;
        if (!pipe.wait_warp(Q_FREE + i, (nq[i] & 1u) ^ 1u)) return false;
        if (lane == 0) {
          const uint32_t bar = pipe.bar(Q_FULL + i), dst = q_smem + i * KC * CHUNK;
          const int row = u.q0 + u.row + i * tokens, head = u.head * packed;
          mbar_arrive_expect_tx(bar, PACK ? KC * tokens * packed * 128 : KC * CHUNK);
          tma_load_3d(dst, &tm_q, 0, head, row, bar);
          tma_load_3d(dst + CHUNK, &tm_q, 64, head, row, bar);
          if (ROPE) tma_load_3d(dst + 2 * CHUNK, &tm_qr, 0, head, row, bar);
        }
        __syncwarp();
        ++nq[i];
        return true;
      };
      for (int j = 0; j < n; ++j, ++kt) {
        const int key = u.k0 + j * BN;
        const uint32_t o = kt % NO;
        if (j == max(n - 2, 0) && lane == 0) mbar_arrive(pipe.bar(GO));
        if (j == 0 && !(ok = load_q(0))) break;
        if (!(ok = room(KC))) break;
        if (lane == 0) {
          const uint32_t bar = pipe.bar(K_FULL + o);
          mbar_arrive_expect_tx(bar, KC * CHUNK);
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            const uint32_t dst = ring + wrap<RING>(pos + c) * CHUNK;
            if (c < 2) tma_load_3d(dst, &tm_k, c * 64, p.k_heads ? g : 0, key, bar);
            else tma_load_3d(dst, &tm_kr, 0, p.r_heads ? g : 0, key, bar);
          }
        }
        __syncwarp();
        pos = wrap<RING>(pos + KC);
        ++nk;
        if (j == 0 && !(ok = load_q(1))) break;
        if (!(ok = room(2))) break;
        if (lane == 0) {
          const uint32_t bar = pipe.bar(V_FULL + o);
          mbar_arrive_expect_tx(bar, 2 * CHUNK);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t dst = ring + wrap<RING>(pos + h) * CHUNK;
            tma_load_3d(dst, &tm_v, 0, p.v_heads ? g : 0, key + h * 64, bar);
            tma_load_3d(dst + CHUNK / 2, &tm_v, 64, p.v_heads ? g : 0, key + h * 64, bar);
          }
        }
        __syncwarp();
        pos = wrap<RING>(pos + 2);
        ++nv;
      }
    }
    // every copy asked for lands before the block may leave
    for (uint32_t o = nk > NO ? nk - NO : 0; o < nk; ++o) pipe.drain(K_FULL + o % NO, (o / NO) & 1u);
    for (uint32_t o = nv > NO ? nv - NO : 0; o < nv; ++o) pipe.drain(V_FULL + o % NO, (o / NO) & 1u);
    for (int i = 0; i < 2; ++i)
      if (nq[i]) pipe.drain(Q_FULL + i, (nq[i] - 1) & 1u);
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA (one thread)
    // Its scalar work is what keeps the tensor pipe waiting: no votes, no divisions, a wait
    // per hand-over.
    if (elect_one()) {
      constexpr uint32_t IDESC_QK = idesc_bf16(BM, BN, 0, 0), IDESC_PV = idesc_bf16(BM, 128, 0, 1);
      uint32_t kt = 0, pos = 0, nc = 0, nu[2] = {0, 0}, np[2] = {0, 0};  // key tiles, ring, cleared, units, P tiles
      bool ok = true;
      // S = Q K^T of one tile; `at`: chunk where the keys begin
      auto qk = [&](int i, uint32_t at, bool last) {
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          const uint64_t a = desc_k(q_smem + (i * KC + c) * CHUNK), b = desc_k(ring + wrap<RING>(at + c) * CHUNK);
#pragma unroll
          for (int s = 0; s < 4; ++s) mma_bf16_ss(t_s + i * BN, a + 2 * s, b + 2 * s, IDESC_QK, c + s > 0);
        }
        tc_commit(pipe.bar(S_FULL + i));
        if (last) tc_commit(pipe.bar(Q_FREE + i));
      };
      // O += P V of one tile; keys: the sequence's keys from this key tile on
      auto pv = [&](int i, uint32_t at, int j, int keys) -> bool {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint64_t b = desc_v(ring + wrap<RING>(at + h) * CHUNK);
          if (!pipe.wait(P_FULL + 2 * i + h, np[i] & 1u)) return false;
          if (keys <= h * 64) continue;
          tc_fence_after();
#pragma unroll
          for (int s = 0; s < 4; ++s)
            mma_bf16_ts(t_o + i * BN, t_s + i * BN + h * 32 + s * 8, b + s * 128, IDESC_PV, j + h + s > 0);
        }
        ++np[i];
        return true;
      };
      for (int k = 0; ok; ++k) {
        if (!(ok = pipe.wait(U_FULL + k % NS, (k / NS) & 1))) break;
        const int4* w = reinterpret_cast<const int4*>(gbase + OFF_UNIT + (k % NS) * 32);
        const int q0 = w[0].x, nk = w[0].w, n0 = w[1].z, n1 = w[1].w;
        mbar_arrive(pipe.bar(U_FREE + k % NS));
        if (q0 < 0) break;
        const int all = max(n0, n1);
        if (all == 0) continue;
        // the last value tile may be cleared once the one NO before it, whose barrier it has, is used
        if (all <= NO && nk < all * BN) mbar_arrive(pipe.bar(V_GO));
        if (!(ok = pipe.wait(K_FULL + kt % NO, (kt / NO) & 1u))) break;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int n = i ? n1 : n0;
          if (ok && n > 0) {
            if (!(ok = pipe.wait(Q_FULL + i, nu[i] & 1u))) continue;
            tc_fence_after();
            qk(i, pos, n == 1);
            ++nu[i];
          }
        }
        if (!ok) break;
        tc_commit(pipe.bar(K_FREE + kt % NO));
        for (int j = 0; j < all; ++j, ++kt) {
          const uint32_t v_at = wrap<RING>(pos + KC), next = wrap<RING>(v_at + 2), o = kt % NO, o1 = (kt + 1) % NO;
          const int keys = nk - j * BN;
          if (j > 0 && j == all - NO && nk < all * BN) mbar_arrive(pipe.bar(V_GO));
          if (!(ok = pipe.wait(V_FULL + o, (kt / NO) & 1u))) break;
          if (keys < BN) {                                // its tail is being cleared
            if (!(ok = pipe.wait(V_CLEAN, nc & 1u))) break;
            ++nc;
          }
          if (j < n0 && !(ok = pv(0, v_at, j, keys))) break;
          if (j + 1 < all && !(ok = pipe.wait(K_FULL + o1, ((kt + 1) / NO) & 1u))) break;
          if (j + 1 < n0) qk(0, next, j + 2 == n0);
          else if (j + 1 == n0) tc_commit(pipe.bar(O_DONE));
          if (j < n1 && !(ok = pv(1, v_at, j, keys))) break;
          tc_commit(pipe.bar(V_FREE + o));                // both tiles are past these values
          if (j + 1 < n1) qk(1, next, j + 2 == n1);
          else if (j + 1 == n1) tc_commit(pipe.bar(O_DONE + 1));
          if (j + 1 < all) tc_commit(pipe.bar(K_FREE + o1));
          pos = next;
        }
      }
      tc_commit(pipe.bar(DRAIN));
      pipe.drain(DRAIN, 0);                               // nothing in flight when TMEM is released
    }
    __syncwarp();
  } else if (warp == 10) {
    // ------------------------------------------------------------ values past a sequence's last key
    // They meet P = 0, but belong to another sequence or to nobody, and 0 x NaN is not 0.
    uint32_t kt = 0, pos = 0, nc = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!(ok = pipe.wait_warp(U_FULL + k % NS, (k / NS) & 1))) break;
      const Unit u = read_unit(gbase, k);
      __syncwarp();
      if (lane == 0) mbar_arrive(pipe.bar(U_FREE + k % NS));
      if (u.q0 < 0) break;
      const int all = max(u.n0, u.n1);
      if (all == 0) continue;
      const uint32_t last = kt + all - 1;
      const int keys = u.nk - (all - 1) * BN;
      if (keys < BN) {
        const uint32_t at = (pos + (uint32_t)(all - 1) * (KC + 2) + KC) % RING;
        // (not before the MMAs are close: the barrier's phases alternate)
        if (!(ok = pipe.wait_warp(V_GO, nc & 1u))) break;
        ++nc;
        if (!(ok = pipe.wait_warp(V_FULL + last % NO, (last / NO) & 1u))) break;
        // a row is 128 bytes of each 64-column box; the swizzle stays inside it
        for (int h = 0; h < 2; ++h) {
          uint4* z = reinterpret_cast<uint4*>(gbase + (ring - base) + wrap<RING>(at + h) * CHUNK);
          const int from = max(keys - h * 64, 0);
          if (keys <= h * 64) continue;                   // not multiplied at all
          for (int e = from * 8 + lane; e < 512; e += 32) z[e] = z[512 + e] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_cta();
        __syncwarp();
        if (lane == 0) mbar_arrive(pipe.bar(V_CLEAN));
      }
      kt += all;
      pos = (pos + (uint32_t)all * (KC + 2)) % RING;
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax and output of one tile
    const int i = warp >> 2, r = threadIdx.x & 127;
    const int r_token = PACK ? r / packed : r, r_head = PACK ? r - r_token * packed : 0;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = t_s + i * BN + lanes, o_at = t_o + i * BN + lanes;
    uint32_t ns = 0, nu = 0;                            // key tiles, units with work
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!(ok = pipe.wait_warp(U_FULL + k % NS, (k / NS) & 1))) break;
      const Unit u = read_unit(gbase, k);
      __syncwarp();
      if (lane == 0) mbar_arrive(pipe.bar(U_FREE + k % NS));
      if (u.q0 < 0) break;
      const int n = u.tiles(i), row = u.row + i * tokens + r_token;
      // keys this row sees, and the first and the last row of the warp
      const int64_t off = (int64_t)u.nk - u.nq + 1;
      const int lim = (int)max((int64_t)0, min((int64_t)u.nk, row + off));
      const int first = __shfl_sync(0xffffffffu, lim, 0), last = __shfl_sync(0xffffffffu, lim, 31);
      float m = -INFINITY, l = 0.f;                     // raw scores
      for (int j = 0; j < n; ++j, ++ns) {
        if (!(ok = pipe.wait_warp(S_FULL + i, ns & 1u))) break;
        tc_fence_after();
        // columns that every row of the warp sees, that some row does, and that this row does
        const int c_all = first - j * BN, c_any = last - j * BN, c_row = lim - j * BN;
        const bool whole = c_all >= BN;
        float mx = -INFINITY;
        if (whole) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t s[64];
            tmem_ld64(s_at + h * 64, s);
            tmem_wait_ld();
            mx = fmaxf(mx, max_columns<64>(s));
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < min(BN, c_any); c += 32) {
            uint32_t s[32];
            tmem_ld32(s_at + c, s);
            tmem_wait_ld();
            if (c + 32 > c_all) mask32(s, c_row - c);
            mx = fmaxf(mx, max_columns<32>(s));
          }
        }
        // the maximum in use moves when P would pass 2^8
        const bool rise = j == 0 || (mx - m) * p.scale_log2 > 8.f;
        if (j > 0 && __any_sync(0xffffffffu, rise)) {
          const float mn = rise ? mx : m;
          const float f = rise ? ex2((m - mn) * p.scale_log2) : 1.f;       // m = -inf: 0
          l *= f;
          m = mn;
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t o[32];
            tmem_ld32(o_at + q * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
            tmem_st32(o_at + q * 32, o);
          }
        } else if (j == 0) {
          m = mx;
        }
        const float nm = m == -INFINITY ? 0.f : -m * p.scale_log2;
        float l0 = 0.f, l1 = 0.f;
        // the scores are read once more: held over from the maximum, they would leave no
        // registers to keep more than a few exponentials in flight
        if (whole) {
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t s[64], pk[32];
            tmem_ld64(s_at + h * 64, s);
            tmem_wait_ld();
            exp_columns<64>(s, pk, p.scale_log2, nm, l0, l1);
            tmem_st32(s_at + h * 32, pk);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(pipe.bar(P_FULL + 2 * i + h));
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < BN; c += 32) {
            uint32_t pk[16];
            if (c < c_any) {
              uint32_t s[32];
              tmem_ld32(s_at + c, s);
              tmem_wait_ld();
              if (c + 32 > c_all) mask32(s, c_row - c);
              exp_columns<32>(s, pk, p.scale_log2, nm, l0, l1);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) pk[e] = 0u;
            }
            tmem_st8(s_at + c / 2, pk[0], pk[1], pk[2], pk[3], pk[4], pk[5], pk[6], pk[7]);
            tmem_st8(s_at + c / 2 + 8, pk[8], pk[9], pk[10], pk[11], pk[12], pk[13], pk[14], pk[15]);
            if (c & 32) {
              tmem_wait_st();
              tc_fence_before();
              mbar_arrive(pipe.bar(P_FULL + 2 * i + (c >> 6)));
            }
          }
        }
        l += l0 + l1;
      }
      if (!ok) break;
      const bool mine = row < u.nq && (!PACK || r_token < tokens);      // (128 rows are not all used)
      const int64_t at = (int64_t)(u.q0 + row) * p.H + u.head * packed + r_head;
      if (n > 0) {
        if (!(ok = pipe.wait_warp(O_DONE + i, nu & 1u))) break;
        ++nu;
        tc_fence_after();
        const float inv = 1.f / l;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t o[32];
          tmem_ld32(o_at + q * 32, o);
          tmem_wait_ld();
          if (mine) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                v[e] = lim == 0 ? 0u : pack_bf16x2(__uint_as_float(o[c * 16 + 2 * e]) * inv,
                                                   __uint_as_float(o[c * 16 + 2 * e + 1]) * inv);
              st_global_v8(p.out + at * 128 + q * 32 + c * 16, v);
            }
          }
        }
        tc_fence_before();
      } else if (mine) {
        for (int c = 0; c < 16; ++c) st_global_v4(p.out + at * 128 + c * 8, 0u, 0u, 0u, 0u);
      }
      if (mine) p.lse[at] = lim == 0 ? -INFINITY : m * p.scale + logf(l);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 11) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace pr
}  // namespace kd

using namespace kd;

static bool view_ok(const void* p, int64_t tok, int64_t head, int64_t rows) {
  return p && aligned16(p) && tok >= 0 && head >= 0 && tok % 8 == 0 && head % 8 == 0 && (tok > 0 || rows <= 1);
}

extern "C" int kd_prompt_attn(const kd_bf16_t* q_nope, int64_t qnt, int64_t qnh, const kd_bf16_t* q_rope, int64_t qrt,
                              int64_t qrh, const kd_bf16_t* k_nope, int64_t knt, int64_t knh, const kd_bf16_t* k_rope,
                              int64_t krt, int64_t krh, const kd_bf16_t* v, int64_t vt, int64_t vh,
                              const int32_t* cu_q, const int32_t* cu_k, int B, int T, int Tk, int H, int Hk,
                              float scale, kd_bf16_t* out, float* lse, int32_t* dev_error, cudaStream_t stream) {
  if (B < 1 || B > 65535 || T < 0 || Tk < 0 || H < 1 || H > KD_MAX_HEADS || Hk < 1 || H % Hk ||
      !(scale > 0.f && isfinite(scale)) || (int64_t)T * H > INT32_MAX || (int64_t)Tk * Hk > INT32_MAX)
    return KD_EINVAL;
  if (T == 0) return KD_OK;                       // (tensors without elements may have no address)
  if ((Tk && (q_rope != nullptr) != (k_rope != nullptr)) || !view_ok(q_nope, qnt, qnh, T) || (H > 1 && qnh == 0) || !out || (reinterpret_cast<uintptr_t>(out) & 31u) || !lse || !cu_q ||
      (Tk && (!view_ok(k_nope, knt, knh, Tk) || !view_ok(v, vt, vh, Tk))) ||
      (q_rope && (!view_ok(q_rope, qrt, qrh, T) || (H > 1 && qrh == 0) || (Tk && !view_ok(k_rope, krt, krh, Tk)))))
    return KD_EINVAL;
  // Short prompts' heads that share a key head fill a tile together.  With a head a tile and so:
  // 32 prompts of 1 to 300 tokens, 28 heads on 4, 40 and 32 us; 8 of 1000 to 2000, 32 on 4, 193 and
  // 179; 27 of one or two tokens over 340 keys, 32 on 8, 45 and 20; but 4 of just 1024, 40 on 8,
  // 66 and 68.  Long ones leave few rows empty, and a tile's rows in one piece are faster: 4 of
  // 4096 tokens, 16 heads on 2, 283 and 291, one of 16384 1016 and 1028.  (2048 is between the
  // lengths that gain and those that lose, neither by much: not a sharp bound.)  Nor do groups share a
  // tile that would leave an eighth of it empty (22 or more heads as a rule).
  const int group = H / Hk, full = pr::BM / group * group;
  const int packed = T < (int64_t)2048 * B && full >= pr::BM * 7 / 8 ? group : 1;
  const int tokens = pr::BM / packed, heads = H / packed;
  const int64_t slots = T / (2 * tokens) + (int64_t)B;
  if (slots * heads > INT32_MAX) return KD_EINVAL;
  int st = device_sms(nullptr);
  if (st) return st;
  int dev = 0;
  if ((st = cuda_status(cudaGetDevice(&dev), "cudaGetDevice"))) return st;
  static std::once_flag once[64];
  static std::atomic<int> attr[64];
  std::call_once(once[dev], [&] {
    int s = 0;
    for (const auto kernel : {pr::prompt_kernel<false, false>, pr::prompt_kernel<false, true>,
                              pr::prompt_kernel<true, false>, pr::prompt_kernel<true, true>})
      if (!s)
        s = cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, pr::SMEM),
                        "cudaFuncSetAttribute(prompt_kernel)");
    attr[dev].store(s);
  });
  if ((st = attr[dev].load())) return st;

  pr::Params p{cu_q, cu_k, out, lse, dev_error, B, T, Tk, H, (int)slots, packed, tokens, heads, heads / Hk, knh > 0, krh > 0, vh > 0,
               scale, scale * 1.4426950408889634f};
  const bool rope = q_rope != nullptr;
  CUtensorMap tq, tqr, tk, tkr, tv;
  // without keys the key and value maps are never used: any memory will do
  const kd_bf16_t *kp = Tk ? k_nope : q_nope, *vp = Tk ? v : q_nope, *rp = Tk ? k_rope : q_rope;
  if ((st = make_tmap3(&tq, q_nope, 128, H, T, qnh, qnt, packed, tokens)) ||
      (st = make_tmap3(&tk, kp, 128, knh ? Hk : 1, Tk, knh, knt, 1, pr::BN)) ||
      (st = make_tmap3(&tv, vp, 128, vh ? Hk : 1, Tk, vh, vt, 1, 64)))
    return st;
  if (rope) {
    if ((st = make_tmap3(&tqr, q_rope, 64, H, T, qrh, qrt, packed, tokens)) ||
        (st = make_tmap3(&tkr, rp, 64, krh ? Hk : 1, Tk, krh, krt, 1, pr::BN)))
      return st;
  } else {
    tqr = tq;
    tkr = tk;
  }
  const unsigned grid = (unsigned)(slots * heads);
  const auto kernel = packed > 1 ? (rope ? pr::prompt_kernel<true, true> : pr::prompt_kernel<false, true>)
                            : (rope ? pr::prompt_kernel<true, false> : pr::prompt_kernel<false, false>);
  kernel<<<grid, pr::THREADS, pr::SMEM, stream>>>(tq, tqr, tk, tkr, tv, p);
  return launch_status("prompt_kernel");
}

// Dense causal attention over packed sequences for sm_100a.
//
// What it computes: rows cu[s] .. cu[s+1] - 1 of Q, K and V are sequence s; for its row i and
// query head h (KV head h / G, G = Hq / Hkv)
//   O_i = sum_{j <= i, j in s} softmax_j(q_i.k_j / sqrt(d)) v_j,   lse_i = log sum_j exp(q_i.k_j / sqrt(d)).
// One pass over the keys with a running maximum m and sum l per row; S and O accumulate in
// fp32 (TMEM), l sums the unrounded P.  P is rounded to bf16 for the P.V product, whose operands have one
// type, V's (as in the sparse prefill): O is 1.9e-3 to 2.1e-3 from 64 bits, relative, where its own
// rounding alone makes 1.6e-3.
//
// Design (persistent, one CTA per SM; an item = two 128-row query tiles that walk the same keys):
//   * the two tiles are the same rows of two query heads of one KV head when G is even, else
//     two adjacent row tiles of one head: each K and V tile (128 keys) is loaded once for both;
//   * warps 0-3 run tile A's softmax and epilogue, warps 4-7 tile B's (one thread per row);
//     warp 8 finds the items, one lane of it streams K and V through a ring of NST stages with
//     TMA; warps 9 and 10 issue the tcgen05.mma of tile A and of tile B; warps 11-14 clean the V
//     tiles that reach past what a row may see (V FIX below);
//   * TMEM (all 512 columns): S of each tile in two halves of 64 keys, O_A, O_B of 128 columns;
//     P overwrites the first 32 columns of its half as bf16 pairs.  A half's next S = Q K^T goes
//     out right behind its P V, while the softmax works on the other half;
//   * the running maximum is raised only when it grows by more than 2^8, so O is rescaled almost
//     never.  Weights are 2^(x - m - 8), at most 1 however far m lags: relative roundings are the
//     same, l is at most the number of keys, and O stays inside fp32 wherever it would with an exact
//     maximum (|V| below 2^128 / keys).  With weights up to 2^8, one key of 2^7.9 and a value of
//     2^121 were infinite.  What it costs is at the other end: the largest weight may be 2^-8, so
//     sums lose what is under 2^-118.
// What bounds it: MMA operands and TMA together move about 320 KB of shared memory per 128 keys of an
// item (2500 cycles at 128 bytes), the weights' exponentials take 2048 (16 a cycle); a step of 128
// keys takes 3650 at 32K tokens.  Steps that led here (32 query heads on 8, d 128, one sequence of 32768):
//   one MMA thread, whole tiles of S: 9.0 ms.  The chain P -> P V -> S -> softmax was a step's time
//     (4860 cycles), and the issuing thread was busy for 2700 of them;
//   halves of 64 keys with one thread issuing: 12.8 ms (issue-bound); descriptors as uniform values of a
//     whole warp, one lane elected: 10.0 ms; a warp for each tile: 8.1 ms.
//   Part of the exponentials as polynomials on the multiply-add pipe, spread between the others: d 64 (16 heads,
//     8192 tokens) 0.269 -> 0.234 ms with 5 of 16, d 128 (32768 tokens) 8.33 -> 8.13 ms with 4 of 16.
// Now, in runs of many such calls: 8.35 ms and 0.237 ms.
// V FIX: a hidden key has P = 0, but 0 x infinity is NaN.  The last key tile of a row tile holds
// rows behind the sequence's end (another request's values) and keys that some rows must not
// see; warps 11-14 zero the former, and zero the non-finite elements of the others, noting
// their rows; the epilogue adds those elements to the rows that do see them.
// No cluster, no multicast; every wait is bounded (status word + early exit).
#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "dsa_serve.cuh"

namespace dsa {
namespace {

constexpr int TM = 128;             // query rows of a tile
constexpr int TN = 128;             // keys of a tile
constexpr int TH = 64;              // keys of half a tile: what one softmax step takes
constexpr int SLAB = 128 * 128;     // bytes of 128 rows x 64 bf16 columns
constexpr int CLEAN_WARPS = 4;
constexpr int PACK_THREADS = 352 + 32 * CLEAN_WARPS;
constexpr uint32_t PACK_TMEM = 512;
constexpr uint32_t PACK_O = 256;    // O of tile x at PACK_O + 128 x, S of tile x at 128 x
constexpr int NITEM = 4;            // ItemInfo ring
// Barriers for cleaned V tiles, used in turn.  One MMA warp may be up to two cleaned tiles ahead of the other: it
// cannot pass the next item's Q before the other has issued all of this item's Q K^T, and an item has two of them.
constexpr int NFIX = 4;
constexpr float PACK_RESCALE = 8.0f;  // how far (log2) a row's maximum may lag

struct PackArgs {
  int Hq, G, T, nseq, npairs;
  const int32_t* cu;
  const __nv_bfloat16* V;
  int64_t v_hs, v_ts;
  __nv_bfloat16* O;
  int64_t o_hs, o_ts;
  int o_v8;
  float* lse;
  float scale_log2;
  unsigned* status;
  uint64_t wait_limit_ns;
};

struct PackItem {
  int h[2];     // query head of each tile
  int row0[2];  // first row of each tile, counted in its sequence
  int n[2];     // key tiles of each tile (0: no such tile)
  int start;    // first row of the sequence in the packed tensors; -1: no more items
  int len;      // its rows
  uint32_t bad[2][4];  // rows with non-finite V elements in key tile n[0] - 1 + i
};

template <int D>
struct PackSmem {
  static constexpr int DS = D / 64;
    static constexpr int NST = D == 128 ? 5 : 10;
  static constexpr int STAGE = DS * SLAB;
  static constexpr int Q_OFF = 0;
  static constexpr int KV_OFF = 2 * STAGE;
  static constexpr int ITEM_OFF = KV_OFF + NST * STAGE;
  static constexpr int BAR_OFF = ITEM_OFF + NITEM * (int)sizeof(PackItem);
  static constexpr int NBAR = 2 * NST + 2 * NITEM + 18 + NFIX;
  static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
  static constexpr int BYTES = MISC_OFF + 32 + 1024;
  static_assert(BYTES <= 232448, "shared memory");
  static_assert(sizeof(PackItem) % 8 == 0, "barrier alignment");
  // barriers
  // (SFULL, PFULL and ODONE: 2 * row tile + half.  A parity tells only neighbouring phases apart; with one barrier
  // for each half, no one waits for a phase while the one behind it could be over.)
  static constexpr int QFULL = 0, QEMPTY = 1, SFULL = 2, PFULL = 6, ODONE = 10, FIXREQ = 14, DRAIN = 16, VFIX = 18;
  static constexpr int ITEMFULL = VFIX + NFIX, ITEMFREE = ITEMFULL + NITEM;
  static constexpr int FULL = ITEMFREE + NITEM, EMPTY = FULL + NST;
};

// The whole MMA warp runs the code around these, so that descriptors and addresses are uniform values;
// one elected lane issues.
__device__ __forceinline__ bool pack_elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// S = Q K^T for 64 keys (both K-major, 128-byte swizzle): D / 16 k-steps.  a, b: low words of the descriptors.
template <int D>
__device__ __forceinline__ void pack_mma_qk(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc) {
  if (pack_elect()) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint32_t off = (k >> 2) * (SLAB >> 4) + (k & 3) * 2;
      tc_mma_f16(d, ((uint64_t)hi << 32) | (a + off), ((uint64_t)hi << 32) | (b + off), idesc, k > 0 ? 1u : 0u);
    }
  }
  __syncwarp();
}
// O (+)= P V for 64 keys: P from TMEM, V MN-major, 4 k-steps of 16 keys.
__device__ __forceinline__ void pack_mma_pv(uint32_t d, uint32_t p, uint32_t b, uint32_t hi, uint32_t idesc, uint32_t acc) {
  if (pack_elect()) {
#pragma unroll
    for (int k = 0; k < TH / 16; ++k)
      tc_mma_f16_ts(d, p + 8 * k, ((uint64_t)hi << 32) | (b + k * (2048 >> 4)), idesc, k > 0 ? 1u : acc);
  }
  __syncwarp();
}
__device__ __forceinline__ void pack_arrive(uint64_t* bar) {
  if (pack_elect()) mbar_arrive(bar);
  __syncwarp();
}
__device__ __forceinline__ void pack_commit(uint64_t* bar) {
  if (pack_elect()) tc_commit(bar);
  __syncwarp();
}

template <int D>
__global__ void __launch_bounds__(PACK_THREADS, 1)
packed_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PackArgs a) {
  using L = PackSmem<D>;
  constexpr int DS = L::DS, NST = L::NST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::BAR_OFF);
  PackItem* items = reinterpret_cast<PackItem*>(sm + L::ITEM_OFF);
  int* misc = reinterpret_cast<int*>(sm + L::MISC_OFF);  // [0] TMEM base, [2] abort
  volatile int* abort_flag = misc + 2;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < L::NBAR; ++i) {
      uint32_t cnt = 1;
      if (i >= L::PFULL && i < L::PFULL + 4) cnt = 4;
      if (i >= L::EMPTY || i == L::QEMPTY) cnt = 2;               // both MMA warps
      if (i >= L::ITEMFREE && i < L::ITEMFREE + NITEM) cnt = 10 + CLEAN_WARPS;  // softmax, MMA and cleaning warps
      if (i >= L::VFIX && i < L::VFIX + NFIX) cnt = CLEAN_WARPS;
      mbar_init(&bars[i], cnt);
    }
    fence_barrier_init();
    misc[2] = 0;
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  // Tensor memory is taken behind this wait only: the grid in front may still have to take its own.
  pdl_prologue();
  if (warp == 9) {
    tmem_alloc(reinterpret_cast<uint32_t*>(&misc[0]), PACK_TMEM);
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);
  const uint64_t limit = a.wait_limit_ns;

  if (warp >= 8) {
    if (warp == 8) {
      // ---------------------------------------------------------- items and TMA loads
      const bool by_heads = (a.G & 1) == 0;
      const int rows_per_item = by_heads ? TM : 2 * TM;
      // Row groups are taken in windows of 32 sequences, one per lane, and in each window by their place in the
      // sequence, the last (longest) ones first.
      int win = 0, before = 0;         // first sequence of the window, groups of the windows before it
      int lo = 0, hi = 0, groups = 0;  // this lane's sequence
      int in_win = 0;                  // groups of the window
      int place = 0, longer = 0;       // the place that items are taken from now, groups behind it
      auto load_window = [&]() {
        const int s = win + lane;
        lo = hi = 0;
        if (s < a.nseq) {
          lo = a.cu[s];
          hi = a.cu[s + 1];
          if (lo < 0 || hi < lo || hi > a.T) {
            report(a.status, DSA_ERR_DEVICE, DETAIL_BAD_SEQ);
            hi = lo = 0;
          }
        }
        groups = ceil_div(hi - lo, rows_per_item);
        in_win = warp_sum_int(groups);
        int most = groups;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        place = most - 1;
        longer = 0;
      };
      load_window();
      uint32_t gs = 0;   // ring stages used so far
      int q_last = -1;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        // items are dealt back and forth over the CTAs, so that a CTA's early (long) items pair with late ones
        const int64_t k = (int64_t)it * gridDim.x + ((it & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        const int64_t grp64 = k / a.npairs;
        const int pair = (int)(k - grp64 * a.npairs);
        while (grp64 >= (int64_t)before + in_win && win + 32 < a.nseq) {
          before += in_win;
          win += 32;
          load_window();
        }
        const bool end = grp64 >= (int64_t)before + in_win;
        const int slot = it % NITEM;
        PackItem* item = &items[slot];
        if (it >= NITEM) {
          int w = 1;
          if (lane == 0) w = serve_wait(&bars[L::ITEMFREE + slot], (it / NITEM - 1) & 1, limit, a.status, DETAIL_WAIT_EMPTY, abort_flag);
          if (!__shfl_sync(0xffffffffu, w, 0)) break;
        }
        if (end) {
          if (lane == 0) {
            item->start = -1;
            mbar_arrive(&bars[L::ITEMFULL + slot]);
          }
          break;
        }
        const int grp = (int)(grp64 - before);
        uint32_t has = __ballot_sync(0xffffffffu, groups > place);  // sequences with a group at `place`
        while (grp >= longer + __popc(has)) {
          longer += __popc(has);
          --place;
          has = __ballot_sync(0xffffffffu, groups > place);
        }
        const bool mine = ((has >> lane) & 1u) && __popc(has & ((1u << lane) - 1u)) == grp - longer;
        const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
        const int start = __shfl_sync(0xffffffffu, lo, src);
        const int len = __shfl_sync(0xffffffffu, hi, src) - start;
        const int local = place;
        if (lane == 0) {
          PackItem& w = *item;
          w.start = start;
          w.len = len;
#pragma unroll
          for (int x = 0; x < 8; ++x) w.bad[x >> 2][x & 3] = 0;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int tile = by_heads ? local : 2 * local + x;
            w.h[x] = by_heads ? 2 * pair + x : pair;
            w.row0[x] = tile * TM;
            w.n[x] = tile * TM < len ? tile + 1 : 0;
          }
          const int n = max(w.n[0], w.n[1]);
          const int h0 = w.h[0], h1 = w.h[1], r0 = w.row0[0], r1 = w.row0[1], n1 = w.n[1];
          mbar_arrive(&bars[L::ITEMFULL + slot]);
          const int kvh = h0 / a.G;
          if (it > 0) ok = serve_wait(&bars[L::QEMPTY], (it - 1) & 1, limit, a.status, DETAIL_WAIT_Q, abort_flag);
          for (int t = -1; ok && t < 2 * n; ++t) {
            if (t < 0) {
              mbar_arrive_expect_tx(&bars[L::QFULL], (n1 > 0 ? 2 : 1) * L::STAGE);
              q_last = it;
              for (int c = 0; c < DS; ++c) {
                tma_load_3d(sm + L::Q_OFF + c * SLAB, &tmQ, &bars[L::QFULL], c * 64, start + r0, h0);
                if (n1 > 0) tma_load_3d(sm + L::Q_OFF + L::STAGE + c * SLAB, &tmQ, &bars[L::QFULL], c * 64, start + r1, h1);
              }
              continue;
            }
            const uint32_t st = gs % NST, ph = gs / NST;
            if (ph > 0 && !serve_wait(&bars[L::EMPTY + st], (ph - 1) & 1, limit, a.status, DETAIL_WAIT_EMPTY, abort_flag)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&bars[L::FULL + st], L::STAGE);
            uint8_t* dst = sm + L::KV_OFF + st * L::STAGE;
            const CUtensorMap* map = (t & 1) ? &tmV : &tmK;
            for (int c = 0; c < DS; ++c) tma_load_3d(dst + c * SLAB, map, &bars[L::FULL + st], c * 64, start + (t >> 1) * TN, kvh);
            ++gs;
          }
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      }
      // No load may still be on its way into shared memory when the CTA ends.  Whether another warp gives up before the
      // last ones have landed is not known here, so this warp always waits for them: nothing arms these barriers again,
      // and it has nothing else to do.
      if (lane == 0) {
        if (q_last >= 0) serve_drain(&bars[L::QFULL], q_last & 1);
        for (uint32_t g = gs > NST ? gs - NST : 0; g < gs; ++g) serve_drain(&bars[L::FULL + g % NST], (g / NST) & 1);
      }
      __syncwarp();
    } else if (warp < 11) {
      // ---------------------------------------------------------- MMA issuers
      const int x = __shfl_sync(0xffffffffu, warp, 0) - 9;  // the row tile
      constexpr uint32_t IDESC_QK = idesc_bf16(TM, TH, 0, 0);
      constexpr uint32_t IDESC_PV = idesc_bf16(TM, D, 0, 1);
      const uint64_t q_desc = smem_desc(smem_u32(sm + L::Q_OFF), 16, 1024, SWZ_128B);
      const uint64_t k_desc = smem_desc(smem_u32(sm + L::KV_OFF), 16, 1024, SWZ_128B);
      const uint64_t v_desc = smem_desc(smem_u32(sm + L::KV_OFF), SLAB, 1024, SWZ_128B);
      constexpr uint32_t STG = L::STAGE >> 4;
      const uint32_t q_lo = __shfl_sync(0xffffffffu, (uint32_t)q_desc, 0) + x * STG;
      const uint32_t k_lo = __shfl_sync(0xffffffffu, (uint32_t)k_desc, 0), v_lo = __shfl_sync(0xffffffffu, (uint32_t)v_desc, 0);
      const uint32_t qk_hi = (uint32_t)(q_desc >> 32), pv_hi = (uint32_t)(v_desc >> 32);
      const uint32_t tm_s = __shfl_sync(0xffffffffu, tmem, 0) + 128 * x, tm_o = tm_s + PACK_O;
      uint64_t* const pfull = &bars[L::PFULL + 2 * x];
      uint64_t* const sfull = &bars[L::SFULL + 2 * x];
      uint32_t gs = 0;     // ring stages of the items before this one
      uint32_t np = 0;     // key tiles of this row tile whose P has been taken
      uint32_t nfix = 0;   // V tiles cleaned so far
      int pt = -1;         // the key tile whose P V comes next (-1: none),
      bool p_mine = false, p_fix = false;  // whether this row tile has it, whether its V is cleaned,
      uint32_t pg = 0;     // and the ring place of its V
      bool ok = true;
      // Both warps wait for every load and cleaned tile, used or not: that keeps their phases within a ring turn.
      for (int it = 0; ok; ++it) {
        const int slot = it % NITEM;
        if (!serve_warp_wait(&bars[L::ITEMFULL + slot], (it / NITEM) & 1, limit, a.status, DETAIL_WAIT_Q, abort_flag)) break;
        const PackItem* im = &items[slot];
        const bool last = __shfl_sync(0xffffffffu, im->start, 0) < 0;
        const int n0 = __shfl_sync(0xffffffffu, last ? 0 : im->n[0], 0), n1 = __shfl_sync(0xffffffffu, last ? 0 : im->n[1], 0);
        if (!last) pack_arrive(&bars[L::ITEMFREE + slot]);
        const int n = max(n0, n1), nx = x ? n1 : n0;
        // Step t: for each half, P V of the key tile before, then S of tile t.  At t = 0 the tile before is the previous
        // item's last one; both its halves go first, because this item's Q may still be on its way.
        for (int t = 0; t < n || (last && t == 0); ++t) {
          const uint32_t kst = (gs + 2 * t) % NST, kph = ((gs + 2 * t) / NST) & 1;
          const uint32_t vst = pg % NST, vph = (pg / NST) & 1;
          auto put_pv = [&](int h) {
            if (h == 0) {
              if (p_fix) {
                ok = serve_warp_wait(&bars[L::VFIX + nfix % NFIX], (nfix / NFIX) & 1, limit, a.status, DETAIL_WAIT_V, abort_flag, true);
                ++nfix;
              }
              ok = ok && serve_warp_wait(&bars[L::FULL + vst], vph, limit, a.status, DETAIL_WAIT_V, abort_flag, true);
            }
            if (ok && p_mine) {
              ok = serve_warp_wait(pfull + h, np & 1, limit, a.status, DETAIL_WAIT_P, abort_flag, true);
              if (ok) {
                tc_fence_after();
                pack_mma_pv(tm_o, tm_s + TH * h, v_lo + vst * STG + h * (TH / 16) * (2048 >> 4), pv_hi, IDESC_PV, h > 0 || pt > 0 ? 1u : 0u);
                pack_commit(&bars[L::ODONE + 2 * x + h]);
              }
            }
          };
          auto put_qk = [&](int h) {
            if (h == 0) {
              ok = serve_warp_wait(&bars[L::FULL + kst], kph, limit, a.status, DETAIL_WAIT_K, abort_flag, true);
              tc_fence_after();
            }
            if (ok && t < nx) {
              pack_mma_qk<D>(tm_s + TH * h, q_lo, k_lo + kst * STG + h * ((TH * 128) >> 4), qk_hi, IDESC_QK);
              pack_commit(sfull + h);
            }
          };
          if (t > 0) {
            put_pv(0);
            if (ok) put_qk(0);
            if (ok) put_pv(1);
            if (ok) put_qk(1);
          } else {
            if (pt >= 0) {
              put_pv(0);
              if (ok) put_pv(1);
            }
            if (ok && n > 0) {
              ok = serve_warp_wait(&bars[L::QFULL], it & 1, limit, a.status, DETAIL_WAIT_Q, abort_flag, true);
              if (ok) put_qk(0);
              if (ok) put_qk(1);
            }
          }
          if (!ok) break;
          if (pt >= 0) {
            np += p_mine ? 1 : 0;
            pack_commit(&bars[L::EMPTY + vst]);
          }
          pt = -1;
          if (t < n) {
            pack_commit(&bars[L::EMPTY + kst]);
            if (t == n - 1) pack_commit(&bars[L::QEMPTY]);
            pt = t;
            p_mine = t < nx;
            p_fix = t >= n0 - 1;
            pg = gs + 2 * t + 1;
          }
        }
        if (last) break;
        gs += 2 * n;
      }
      // every MMA issued has finished before TMEM is released (also after an abort)
      pack_commit(&bars[L::DRAIN + x]);
      if (lane == 0) serve_drain(&bars[L::DRAIN + x], 0);
      __syncwarp();
    } else {
      // ---------------------------------------------------------- V cleaner
      uint32_t gs = 0, nfix = 0, nsec = 0;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        const int slot = it % NITEM;
        if (!serve_warp_wait(&bars[L::ITEMFULL + slot], (it / NITEM) & 1, limit, a.status, DETAIL_WAIT_Q, abort_flag)) break;
        PackItem* im = &items[slot];
        if (im->start < 0) break;
        const int n0 = im->n[0], n = max(n0, im->n[1]), len = im->len;
        for (int t = n0 - 1; t < n; ++t) {
          // asked for by the softmax that meets the tile; by then the stage's use before this one is known to be over
          const uint32_t g = gs + 2 * t + 1, st = g % NST;
          const int second = t - (n0 - 1);
          ok = serve_warp_wait(&bars[L::FIXREQ + second], (second ? nsec++ : (uint32_t)it) & 1, limit, a.status, DETAIL_WAIT_V, abort_flag) &&
               serve_warp_wait(&bars[L::FULL + st], (g / NST) & 1, limit, a.status, DETAIL_WAIT_V, abort_flag);
          bool wrote = false;
          if (ok) {
            uint8_t* v = sm + L::KV_OFF + st * L::STAGE;
            const int live = len - t * TN;  // rows from here on are behind the sequence
            const int w0 = warp - 11;       // 16-byte pieces i * 32 + lane, i of this warp: 4 rows each
#pragma unroll 1
            for (int i0 = w0 * 8; i0 < DS * 32; i0 += 8 * CLEAN_WARPS) {
              uint4 w[8];
#pragma unroll
              for (int q = 0; q < 8; ++q) w[q] = *reinterpret_cast<const uint4*>(v + ((i0 + q) * 32 + lane) * 16);
              if (live < TN) {
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                  if ((((i0 + q) * 4 + (lane >> 3)) & 127) >= live) {
                    *reinterpret_cast<uint4*>(v + ((i0 + q) * 32 + lane) * 16) = w[q] = make_uint4(0, 0, 0, 0);
                    wrote = true;
                  }
                }
              }
              // 0 x is 0, or NaN where x is not finite
              const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
              __nv_bfloat162 acc[4] = {zero, zero, zero, zero};
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                acc[0] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w[q].x), zero, acc[0]);
                acc[1] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w[q].y), zero, acc[1]);
                acc[2] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w[q].z), zero, acc[2]);
                acc[3] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w[q].w), zero, acc[3]);
              }
              acc[0] = __hadd2(__hadd2(acc[0], acc[1]), __hadd2(acc[2], acc[3]));
              const float seen = __low2float(acc[0]) + __high2float(acc[0]);
              if (seen != seen) {
                wrote = true;
#pragma unroll 1
                for (int q = 0; q < 8; ++q) {
                  uint16_t* e = reinterpret_cast<uint16_t*>(v + ((i0 + q) * 32 + lane) * 16);
                  const int row = ((i0 + q) * 4 + (lane >> 3)) & 127;
                  bool hit = false;
                  for (int j = 0; j < 8; ++j) {
                    if ((e[j] & 0x7f80u) == 0x7f80u) {
                      e[j] = 0;
                      hit = true;
                    }
                  }
                  if (hit) atomicOr(&im->bad[t - (n0 - 1)][row >> 5], 1u << (row & 31));
                }
              }
            }
            if (wrote) fence_proxy_async_smem();  // (a fence holds back the arrival below by some 1000 cycles)
          }
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(&bars[L::VFIX + nfix % NFIX]);
          ++nfix;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::ITEMFREE + slot]);
        gs += 2 * n;
      }
    }
  } else {
    // ------------------------------------------------------------ softmax and epilogue
    const int x = warp >> 2;
    const int q4 = warp & 3;
    const int r = q4 * 32 + lane;  // row of the tile == TMEM lane
    const uint32_t s_t = tmem + ((uint32_t)(q4 * 32) << 16) + 128 * x;
    const uint32_t o_t = s_t + PACK_O;
    uint32_t ns = 0;  // halves of S tiles seen so far
    bool ok = true;
    for (int it = 0; ok; ++it) {
      const int slot = it % NITEM;
      if (!serve_warp_wait_inline(&bars[L::ITEMFULL + slot], (it / NITEM) & 1, limit, a.status, DETAIL_WAIT_Q, abort_flag)) break;
      const PackItem* im = &items[slot];
      if (im->start < 0) break;
      const int n = im->n[x], start = im->start, row = im->row0[x] + r, h = im->h[x];
      const bool in = n > 0 && row < im->len;
      float m = -INFINITY, l = 0.f;  // m: the running maximum when it was last raised, plus PACK_RESCALE
#pragma unroll 1
      for (int u = 0; u < 2 * n; ++u) {
        const int half = u & 1;
        const uint32_t s_h = s_t + TH * half;
        if (!serve_warp_wait_inline(&bars[L::SFULL + 2 * x + half], (ns >> 1) & 1, limit, a.status, DETAIL_WAIT_S, abort_flag)) { ok = false; break; }
        ++ns;
        tc_fence_after();
        float s[TH];
        tmem_ld32(s_h, s);
        tmem_ld32(s_h + 32, s + 32);
        tmem_wait_ld();
        if (u >= 2 * n - 2) {  // the tile on the diagonal
          if (half == 0 && warp == 4 * x && lane == 0 && (x == 0 || n > im->n[0])) mbar_arrive(&bars[L::FIXREQ + x]);  // its V may be cleaned
          const int seen = r - TH * half;
#pragma unroll
          for (int c = 0; c < TH; ++c) s[c] = c <= seen ? s[c] : -INFINITY;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < TH / 2; ++c) mx[c & 3] = serve_max3(mx[c & 3], s[2 * c], s[2 * c + 1]);
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
        float alpha = 1.f;
        bool need = false;
        if (top > m) {
          const float m_new = top + PACK_RESCALE;
          if (m != -INFINITY) {
            alpha = serve_ex2(m - m_new);
            l *= alpha;
            need = true;
          }
          m = m_new;
        }
        // s * scale - m in one rounding leaves what m's own rounding took, half a step of m: beyond 2^24 that is more
        // than the weights' range bears, so there the product is rounded as m was.  (It stands where O is rescaled; in
        // a branch of its own it costs every half: 3 prompts of up to 4096 tokens, 16 heads of d 64, 121 us, 110 here,
        // 107 without.)
        const bool far = in && fabsf(m) >= 16777216.f;  // (rows behind the sequence may hold anything)
        const float scale = far ? 1.f : a.scale_log2;
        if (__any_sync(0xffffffffu, need || far)) {
          if (u > 0) {
            // P V of the half before: the only one that can be under way
            if (!serve_warp_wait_inline(&bars[L::ODONE + 2 * x + (half ^ 1)], ((ns - 2) >> 1) & 1, limit, a.status, DETAIL_WAIT_O, abort_flag)) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              float o[16];
              serve_tmem_ld16(o_t + c * 16, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= alpha;
              serve_tmem_st16(o_t + c * 16, reinterpret_cast<const uint32_t*>(o));
            }
          }
          if (far) {
#pragma unroll
            for (int c = 0; c < TH; ++c) s[c] *= a.scale_log2;
          }
        }
        const float negm = (m == -INFINITY) ? 0.f : -m;
        float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < TH / 32; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float x0, x1;
            serve_fma2(s[32 * c + 2 * i], s[32 * c + 2 * i + 1], scale, negm, x0, x1);
            float p0, p1;
            if (D == 64 ? i % 3 == 1 : i % 4 == 1) {  // see the measurements above
              serve_ex2_poly2(x0, x1, p0, p1);
            } else {
              p0 = serve_ex2(x0);
              p1 = serve_ex2(x1);
            }
            serve_add2(ls[(i & 1) * 2], ls[(i & 1) * 2 + 1], p0, p1);
            __nv_bfloat162 v2 = __floats2bfloat162_rn(p0, p1);
            pk[i] = *reinterpret_cast<uint32_t*>(&v2);
          }
          serve_tmem_st16(s_h + 16 * c, pk);
        }
        l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::PFULL + 2 * x + half]);
      }
      if (!ok) break;
      if (n > 0) {
        if (!serve_warp_wait_inline(&bars[L::ODONE + 2 * x + 1], ((ns >> 1) - 1) & 1, limit, a.status, DETAIL_WAIT_O, abort_flag)) break;
        tc_fence_after();
        const float inv = (l > 0.f) ? 1.f / l : (l == 0.f ? 0.f : l);  // l is 0 without a key of weight, NaN stays
        const int64_t grow = (int64_t)start + (in ? row : 0);
        // cleaned key tiles that this tile's rows see: the diagonal one, and tile A's diagonal one in front of it
        const int first_bad = im->n[0] - 1;
        uint32_t any_bad = 0;
        for (int i = first_bad; i < n; ++i) {
          const uint32_t* bad = im->bad[i - first_bad];
          any_bad |= bad[0] | bad[1] | bad[2] | bad[3];
        }
        __nv_bfloat16* orow = a.O + (int64_t)h * a.o_hs + grow * a.o_ts;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tmem_ld32(o_t + c * 32, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= inv;
          if (any_bad != 0u && in) {
            // non-finite values of those tiles' keys that this row sees
            const __nv_bfloat16* v = a.V + (int64_t)(h / a.G) * a.v_hs + ((int64_t)start + first_bad * TN) * a.v_ts + c * 32;
            const int seen = (n - 1 - first_bad) * TN + r;
#pragma unroll 1
            for (int j = 0; j <= seen; ++j) {
              if (!((im->bad[j >> 7][(j >> 5) & 3] >> (j & 31)) & 1u)) continue;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float e = __bfloat162float(v[(int64_t)j * a.v_ts + i]);
                if (!(fabsf(e) < INFINITY)) o[i] += e;
              }
            }
          }
          // (rows by way of shared memory, so that a store writes whole lines: no faster)
          if (in) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              __nv_bfloat162 v2 = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
              pk[i] = *reinterpret_cast<uint32_t*>(&v2);
            }
            if (a.o_v8) {
              serve_st_v8(orow + c * 32, pk);
              serve_st_v8(orow + c * 32 + 16, pk + 8);
            } else {
#pragma unroll
              for (int v = 0; v < 4; ++v)
                *reinterpret_cast<uint4*>(orow + c * 32 + v * 8) = make_uint4(pk[4 * v], pk[4 * v + 1], pk[4 * v + 2], pk[4 * v + 3]);
            }
          }
        }
        if (a.lse != nullptr && in)
          a.lse[(int64_t)h * a.T + grow] = (l == 0.f) ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[L::ITEMFREE + slot]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, PACK_TMEM);
  }
}

template <int D>
dsa_status launch_packed(const dsa_problem& p, const void* Q, const void* K, const void* V, const int32_t* cu, int nseq,
                         void* O, float* lse, cudaStream_t stream, unsigned* status) {
  CUtensorMap mq, mk, mv;
  if (!make_tma_map_bf16_3d(&mq, Q, D, p.N, p.Hq, p.q_token_stride, p.q_head_stride, TM) ||
      !make_tma_map_bf16_3d(&mk, K, D, p.N, p.Hkv, p.k_token_stride, p.k_head_stride, TN) ||
      !make_tma_map_bf16_3d(&mv, V, D, p.N, p.Hkv, p.v_token_stride, p.v_head_stride, TN))
    return DSA_ERR_CUDA;
  PackArgs a;
  a.Hq = p.Hq;
  a.G = p.Hq / p.Hkv;
  a.T = p.N;
  a.nseq = nseq;
  a.npairs = (a.G & 1) == 0 ? p.Hq / 2 : p.Hq;
  a.cu = cu;
  a.V = static_cast<const __nv_bfloat16*>(V);
  a.v_hs = p.v_head_stride;
  a.v_ts = p.v_token_stride;
  a.O = static_cast<__nv_bfloat16*>(O);
  a.o_hs = p.o_head_stride;
  a.o_ts = p.o_token_stride;
  a.o_v8 = ((reinterpret_cast<uintptr_t>(O) & 31u) == 0 && p.o_token_stride % 16 == 0 && p.o_head_stride % 16 == 0) ? 1 : 0;
  a.lse = lse;
  a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)D));
  a.status = status;
  a.wait_limit_ns = wait_limit_ns();
  int dev = 0, sms = 0;
  cudaError_t e = serve_sms(&dev, &sms);
  if (e == cudaSuccess) e = serve_allow_smem<packed_attn_kernel<D>>(dev, PackSmem<D>::BYTES);
  if (e != cudaSuccess) return cuda_fail(e);
  // the lengths are on the device: as many items as the rows could need at most
  const int64_t rows = (a.G & 1) == 0 ? TM : 2 * TM;
  const int64_t most = ((int64_t)p.N / rows + nseq) * a.npairs;
  const int grid = most < sms ? (int)most : sms;
  e = launch_pdl(packed_attn_kernel<D>, dim3(grid), dim3(PACK_THREADS), (size_t)PackSmem<D>::BYTES, stream, mq, mk, mv, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e);
  return DSA_OK;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status dsa_packed_prefill(const dsa_problem* p, const void* Q, const void* K, const void* V,
                                         const int32_t* cu_seqlens, int32_t n_seq, void* O, float* lse,
                                         dsa_stream stream) {
  dsa_status s = validate_problem(p);
  if (s != DSA_OK) return s;
  // (the tensor maps of the loads cannot step over heads by 0)
  if ((p->Hq > 1 && (p->q_head_stride == 0 || p->o_head_stride == 0)) ||
      (p->Hkv > 1 && (p->k_head_stride == 0 || p->v_head_stride == 0)))
    return DSA_ERR_INVALID_ARG;
  ServeDim o_dims[2] = {{p->N, p->o_token_stride}, {p->Hq, p->o_head_stride}};
  if (!serve_apart(p->d, o_dims)) return DSA_ERR_INVALID_ARG;  // rows of O overlap
  if (n_seq < 0 || (n_seq > 0 && cu_seqlens == nullptr)) return DSA_ERR_INVALID_ARG;
  if (!Q || !K || !V || !O) return DSA_ERR_INVALID_ARG;
  if (!serve_aligned16(Q) || !serve_aligned16(K) || !serve_aligned16(V) || !serve_aligned16(O)) return DSA_ERR_INVALID_ARG;
  if (n_seq == 0) return DSA_OK;
  unsigned* st = status_ptr((cudaStream_t)stream);
  if (st == nullptr) return cuda_fail(cudaGetLastError());
  return p->d == 128 ? launch_packed<128>(*p, Q, K, V, cu_seqlens, n_seq, O, lse, (cudaStream_t)stream, st)
                     : launch_packed<64>(*p, Q, K, V, cu_seqlens, n_seq, O, lse, (cudaStream_t)stream, st);
}

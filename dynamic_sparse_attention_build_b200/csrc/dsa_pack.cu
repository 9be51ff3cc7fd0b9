// Dense causal attention over packed sequences for sm_100a.
//
// What it computes: rows cu[s] .. cu[s+1] - 1 of Q, K and V are sequence s; for its row i and
// query head h (KV head h / G, G = Hq / Hkv)
//   O_i = sum_{j <= i, j in s} softmax_j(q_i.k_j / sqrt(d)) v_j,   lse_i = log sum_j exp(q_i.k_j / sqrt(d)).
// One pass over the keys with a running maximum m and sum l per row; S and O accumulate in
// fp32 (TMEM), P is rounded to bf16 for the P.V product, l sums the unrounded P.
//
// Design (persistent, one CTA per SM; an item = two 128-row query tiles that walk the same keys):
//   * the two tiles are the same rows of two query heads of one KV head when G is even, else
//     two adjacent row tiles of one head: each K and V tile (128 keys) is loaded once for both;
//   * warp 8 (whole) finds the items, one lane loads Q and streams K and V through a ring of
//     NST stages with TMA; warp 9 (one thread) issues the tcgen05.mma; warps 0-3 run tile A's
//     softmax and epilogue, warps 4-7 tile B's (one thread per row); while one tile is in its
//     softmax the tensor core works on the other;
//   * warp 10 cleans the V tiles that reach past what a row may see (see V FIX below);
//   * TMEM (all 512 columns): S_A, S_B, O_A, O_B of 128 columns each; P overwrites the first
//     64 columns of its S as bf16 pairs; S(t+1) is issued right after P(t) V(t), one thread's
//     MMAs run in issue order;
//   * the running maximum is raised only when it grows by more than 2^8,
//     so O is rescaled almost never: scaling all P of a row by one power of two changes no
//     rounding, and l <= 2^29 and O <= 2^29 |V| stay inside fp32.
// V FIX: a hidden key has P = 0, but 0 x infinity is NaN.  The last key tile of an item holds
// rows behind the sequence's end (another request's values) and keys that some rows must not
// see; warp 10 zeroes the former, and zero the non-finite elements of the others, noting
// their rows; the epilogue adds those elements to the rows that do see them.
// No cluster, no multicast; every wait is bounded (status word + early exit).
#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "dsa_serve.cuh"

namespace dsa {
namespace {

constexpr int TM = 128;             // query rows of a tile
constexpr int TN = 128;             // keys of a tile
constexpr int SLAB = 128 * 128;     // bytes of 128 rows x 64 bf16 columns
constexpr int PACK_THREADS = 352;  // 11 warps: up to 184 registers a thread, which the softmax needs
constexpr uint32_t PACK_TMEM = 512;
constexpr uint32_t PACK_O = 256;    // O of tile x at PACK_O + 128 x, S of tile x at 128 x
constexpr int NITEM = 4;            // ItemInfo ring
constexpr float PACK_RESCALE = 8.0f;

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
  static constexpr int NBAR = 2 * NST + 2 * NITEM + 11;
  static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
  static constexpr int BYTES = MISC_OFF + 32 + 1024;
  static_assert(BYTES <= 232448, "shared memory");
  static_assert(sizeof(PackItem) % 8 == 0, "barrier alignment");
  // barriers
  static constexpr int QFULL = 0, QEMPTY = 1, SFULL = 2, PFULL = 4, ODONE = 6, FIXREQ = 8, VFIX = 9, DRAIN = 10;
  static constexpr int ITEMFULL = 11, ITEMFREE = ITEMFULL + NITEM;
  static constexpr int FULL = ITEMFREE + NITEM, EMPTY = FULL + NST;
};

// S = Q K^T (both K-major, 128-byte swizzle): D / 16 k-steps.
template <int D>
__device__ __forceinline__ void pack_mma_qk(uint32_t d, uint64_t a0, uint64_t b0, uint32_t idesc) {
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    const uint64_t off = (uint64_t)((k >> 2) * (SLAB >> 4) + (k & 3) * 2);
    tc_mma_f16(d, a0 + off, b0 + off, idesc, k > 0 ? 1u : 0u);
  }
}
// O (+)= P V: P from TMEM, V MN-major, 8 k-steps of 16 keys.
__device__ __forceinline__ void pack_mma_pv(uint32_t d, uint32_t p, uint64_t b0, uint32_t idesc, uint32_t acc) {
#pragma unroll
  for (int k = 0; k < TN / 16; ++k) tc_mma_f16_ts(d, p + 8 * k, b0 + (uint64_t)(k * (2048 >> 4)), idesc, k > 0 ? 1u : acc);
}

template <int D>
__global__ void __launch_bounds__(PACK_THREADS, 1)
packed_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PackArgs a) {
  pdl_prologue();
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
      if (i == L::PFULL || i == L::PFULL + 1) cnt = 4;
      if (i >= L::ITEMFREE && i < L::ITEMFREE + NITEM) cnt = 10;  // 8 softmax warps, the cleaner, the MMA thread
      mbar_init(&bars[i], cnt);
    }
    fence_barrier_init();
    misc[2] = 0;
  }
  if (warp == 9) {
    tmem_alloc(reinterpret_cast<uint32_t*>(&misc[0]), PACK_TMEM);
    tc_fence_before();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
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
      int win = 0, before = 0;       // sequence window (32 sequences), items groups before it
      int lo = 0, hi = 0, incl = 0;  // this lane's sequence and the groups up to and with it
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
        incl = ceil_div(hi - lo, rows_per_item);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
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
        int total = __shfl_sync(0xffffffffu, incl, 31);
        while (grp64 >= (int64_t)before + total && win + 32 < a.nseq) {
          before += total;
          win += 32;
          load_window();
          total = __shfl_sync(0xffffffffu, incl, 31);
        }
        const bool end = grp64 >= (int64_t)before + total;
        const int slot = it % NITEM;
        PackItem* item = &items[slot];
        if (it >= NITEM) {
          int w = 1;
          if (lane == 0) w = mbar_wait_ool(&bars[L::ITEMFREE + slot], (it / NITEM - 1) & 1, limit, a.status, DETAIL_WAIT_EMPTY, abort_flag, true);
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
        const int src = __popc(__ballot_sync(0xffffffffu, incl <= grp));  // first sequence whose groups reach past grp
        const int start = __shfl_sync(0xffffffffu, lo, src);
        const int len = __shfl_sync(0xffffffffu, hi, src) - start;
        const int local = __shfl_sync(0xffffffffu, incl, src) - 1 - grp;  // longest rows first
        if (lane == 0) {
          PackItem& w = *item;
          w.start = start;
          w.len = len;
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
          if (it > 0) ok = mbar_wait_ool(&bars[L::QEMPTY], (it - 1) & 1, limit, a.status, DETAIL_WAIT_Q, abort_flag, true);
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
            if (ph > 0 && !mbar_wait_ool(&bars[L::EMPTY + st], (ph - 1) & 1, limit, a.status, DETAIL_WAIT_EMPTY, abort_flag, true)) {
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
      // after an abort no load may still be on its way into shared memory when the CTA ends
      if (lane == 0 && *abort_flag) {
        if (q_last >= 0) serve_drain(&bars[L::QFULL], q_last & 1);
        for (uint32_t g = gs > NST ? gs - NST : 0; g < gs; ++g) serve_drain(&bars[L::FULL + g % NST], (g / NST) & 1);
      }
      __syncwarp();
    } else if (warp == 9) {
      // ---------------------------------------------------------- MMA issuer
      if (lane == 0) {
        constexpr uint32_t IDESC_QK = idesc_bf16(TM, TN, 0, 0);
        constexpr uint32_t IDESC_PV = idesc_bf16(TM, D, 0, 1);
        const uint64_t q_desc = smem_desc(smem_u32(sm + L::Q_OFF), 16, 1024, SWZ_128B);
        const uint64_t k_desc = smem_desc(smem_u32(sm + L::KV_OFF), 16, 1024, SWZ_128B);
        const uint64_t v_desc = smem_desc(smem_u32(sm + L::KV_OFF), SLAB, 1024, SWZ_128B);
        constexpr uint64_t STG = L::STAGE >> 4;
        uint32_t gs = 0;
        uint32_t np[2] = {0, 0};  // P tiles consumed so far
        uint32_t nfix = 0;
        bool ok = true;
        for (int it = 0; ok; ++it) {
          const int slot = it % NITEM;
          if (!mbar_wait_ool(&bars[L::ITEMFULL + slot], (it / NITEM) & 1, limit, a.status, DETAIL_WAIT_Q, abort_flag, true)) break;
          const PackItem* im = &items[slot];
          if (im->start < 0) break;
          const int n0 = im->n[0], n1 = im->n[1];
          mbar_arrive(&bars[L::ITEMFREE + slot]);
          const int n = max(n0, n1);
          if (!mbar_wait_ool(&bars[L::QFULL], it & 1, limit, a.status, DETAIL_WAIT_Q, abort_flag, true)) break;
          // step t: P(t-1) V(t-1) of each tile, followed by its S(t)
          for (int t = 0; ok && t <= n; ++t) {
            const uint32_t kst = (gs + 2 * t) % NST, kph = ((gs + 2 * t) / NST) & 1;
            const uint32_t vg = gs + 2 * t - 1;
            const uint32_t vst = vg % NST, vph = (vg / NST) & 1;
            bool k_seen = false;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int nx = x ? n1 : n0;
              if (ok && t > 0 && t - 1 < nx) {
                ok = mbar_wait_ool(&bars[L::PFULL + x], np[x] & 1, limit, a.status, DETAIL_WAIT_P, abort_flag, true);
                ++np[x];
                if (ok && t - 1 >= n0 - 1 && (x == 0 || t - 1 >= n0)) {  // first use of a cleaned V tile
                  ok = mbar_wait_ool(&bars[L::VFIX], nfix & 1, limit, a.status, DETAIL_WAIT_V, abort_flag, true);
                  ++nfix;
                }
                ok = ok && mbar_wait_ool(&bars[L::FULL + vst], vph, limit, a.status, DETAIL_WAIT_V, abort_flag, true);
                if (!ok) break;
                tc_fence_after();
                pack_mma_pv(tmem + PACK_O + 128 * x, tmem + 128 * x, v_desc + vst * STG, IDESC_PV, t > 1 ? 1u : 0u);
                tc_commit(&bars[L::ODONE + x]);
              }
              if (ok && t < nx) {
                if (!k_seen) ok = mbar_wait_ool(&bars[L::FULL + kst], kph, limit, a.status, DETAIL_WAIT_K, abort_flag, true);
                k_seen = true;
                if (!ok) break;
                tc_fence_after();
                pack_mma_qk<D>(tmem + 128 * x, q_desc + x * STG, k_desc + kst * STG, IDESC_QK);
                tc_commit(&bars[L::SFULL + x]);
              }
            }
            if (!ok) break;
            if (t > 0) tc_commit(&bars[L::EMPTY + vst]);
            if (t < n) tc_commit(&bars[L::EMPTY + kst]);
            if (t == n - 1) tc_commit(&bars[L::QEMPTY]);
            if (t < n && t >= n0 - 1) {
              // the cleaner starts on V(t) while S(t) is in its softmax
              const uint32_t fg = gs + 2 * t + 1;
              ok = mbar_wait_ool(&bars[L::FULL + fg % NST], (fg / NST) & 1, limit, a.status, DETAIL_WAIT_V, abort_flag, true);
              if (ok) mbar_arrive(&bars[L::FIXREQ]);
            }
          }
          gs += 2 * n;
        }
        // every MMA issued has finished before TMEM is released (also after an abort)
        tc_commit(&bars[L::DRAIN]);
        serve_drain(&bars[L::DRAIN], 0);
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------- V cleaner
      uint32_t gs = 0, nfix = 0;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        const int slot = it % NITEM;
        if (!serve_warp_wait(&bars[L::ITEMFULL + slot], (it / NITEM) & 1, limit, a.status, DETAIL_WAIT_Q, abort_flag, true)) break;
        PackItem* im = &items[slot];
        if (im->start < 0) break;
        const int n0 = im->n[0], n = max(n0, im->n[1]), len = im->len;
        if (lane < 8) im->bad[lane >> 2][lane & 3] = 0;
        __syncwarp();
        for (int t = n0 - 1; t < n; ++t) {
          if (!serve_warp_wait(&bars[L::FIXREQ], nfix & 1, limit, a.status, DETAIL_WAIT_V, abort_flag, true)) ok = false;
          ++nfix;
          if (ok) {
            const uint32_t st = (gs + 2 * t + 1) % NST;
            uint8_t* v = sm + L::KV_OFF + st * L::STAGE;
            const int live = len - t * TN;  // rows from here on are behind the sequence
#pragma unroll 1
            for (int i0 = 0; i0 < DS * 32; i0 += 8) {
              uint4 w[8];
#pragma unroll
              for (int q = 0; q < 8; ++q) w[q] = *reinterpret_cast<const uint4*>(v + ((i0 + q) * 32 + lane) * 16);
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                const int row = (((i0 + q) * 32 + lane) >> 3) & 127;
                if (row >= live) {
                  *reinterpret_cast<uint4*>(v + ((i0 + q) * 32 + lane) * 16) = make_uint4(0, 0, 0, 0);
                } else {
                  // a half whose exponent is all ones carries into its top bit
                  const uint32_t hit = (((w[q].x & 0x7f807f80u) + 0x00800080u) | ((w[q].y & 0x7f807f80u) + 0x00800080u) |
                                        ((w[q].z & 0x7f807f80u) + 0x00800080u) | ((w[q].w & 0x7f807f80u) + 0x00800080u)) & 0x80008000u;
                  if (hit) {
                    uint16_t* e = reinterpret_cast<uint16_t*>(v + ((i0 + q) * 32 + lane) * 16);
                    for (int j = 0; j < 8; ++j)
                      if ((e[j] & 0x7f80u) == 0x7f80u) e[j] = 0;
                    atomicOr(&im->bad[t - (n0 - 1)][row >> 5], 1u << (row & 31));
                  }
                }
              }
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(&bars[L::VFIX]);
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
    uint32_t ns = 0;  // S tiles seen so far
    bool ok = true;
    for (int it = 0; ok; ++it) {
      const int slot = it % NITEM;
      if (!serve_warp_wait_inline(&bars[L::ITEMFULL + slot], (it / NITEM) & 1, limit, a.status, DETAIL_WAIT_Q, abort_flag)) break;
      const PackItem* im = &items[slot];
      if (im->start < 0) break;
      const int n = im->n[x], start = im->start, row = im->row0[x] + r, h = im->h[x];
      const bool in = n > 0 && row < im->len;
      float m = -INFINITY, l = 0.f;
      for (int t = 0; t < n; ++t) {
        if (!serve_warp_wait_inline(&bars[L::SFULL + x], ns & 1, limit, a.status, DETAIL_WAIT_S, abort_flag)) { ok = false; break; }
        ++ns;
        tc_fence_after();
        float s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_t + 32 * c, s + 32 * c);
        tmem_wait_ld();
        if (t == n - 1) {  // the tile on the diagonal
#pragma unroll
          for (int c = 0; c < 128; ++c) s[c] = c <= r ? s[c] : -INFINITY;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 64; ++c) mx[c & 3] = serve_max3(mx[c & 3], s[2 * c], s[2 * c + 1]);
        const float m_new = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2);
        float alpha = 1.f;
        bool need = false;
        if (m_new > m + PACK_RESCALE) {
          if (m != -INFINITY) {
            alpha = serve_ex2(m - m_new);
            l *= alpha;
            need = true;
          }
          m = m_new;
        }
        if (t > 0 && __any_sync(0xffffffffu, need)) {
          if (!serve_warp_wait_inline(&bars[L::ODONE + x], (ns - 2) & 1, limit, a.status, DETAIL_WAIT_O, abort_flag)) { ok = false; break; }
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
        const float negm = (m == -INFINITY) ? 0.f : -m;
        float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float x0, x1;
            serve_fma2(s[32 * c + 2 * i], s[32 * c + 2 * i + 1], a.scale_log2, negm, x0, x1);
            const float p0 = serve_ex2(x0), p1 = serve_ex2(x1);
            serve_add2(ls[(i & 1) * 2], ls[(i & 1) * 2 + 1], p0, p1);
            __nv_bfloat162 v2 = __floats2bfloat162_rn(p0, p1);
            pk[i] = *reinterpret_cast<uint32_t*>(&v2);
          }
          serve_tmem_st16(s_t + 16 * c, pk);
        }
        l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::PFULL + x]);
      }
      if (!ok) break;
      if (n > 0) {
        if (!serve_warp_wait_inline(&bars[L::ODONE + x], (ns - 1) & 1, limit, a.status, DETAIL_WAIT_O, abort_flag)) break;
        tc_fence_after();
        const float inv = (l > 0.f) ? 1.f / l : (l == 0.f ? 0.f : l);  // l is 0 without a key of weight, NaN stays
        const int64_t grow = (int64_t)start + (in ? row : 0);
        __nv_bfloat16* orow = a.O + (int64_t)h * a.o_hs + grow * a.o_ts;
        // cleaned key tiles that this tile's rows see: the diagonal one, and tile A's diagonal one in front of it
        const int first_bad = im->n[0] - 1;
        uint32_t any_bad = 0;
        for (int i = first_bad; i < n; ++i) {
          const uint32_t* bad = im->bad[i - first_bad];
          any_bad |= bad[0] | bad[1] | bad[2] | bad[3];
        }
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
  if (n_seq < 0 || (n_seq > 0 && cu_seqlens == nullptr)) return DSA_ERR_INVALID_ARG;
  if (!Q || !K || !V || !O) return DSA_ERR_INVALID_ARG;
  if (!serve_aligned16(Q) || !serve_aligned16(K) || !serve_aligned16(V) || !serve_aligned16(O)) return DSA_ERR_INVALID_ARG;
  if (n_seq == 0) return DSA_OK;
  unsigned* st = status_ptr((cudaStream_t)stream);
  if (st == nullptr) return cuda_fail(cudaGetLastError());
  return p->d == 128 ? launch_packed<128>(*p, Q, K, V, cu_seqlens, n_seq, O, lse, (cudaStream_t)stream, st)
                     : launch_packed<64>(*p, Q, K, V, cu_seqlens, n_seq, O, lse, (cudaStream_t)stream, st);
}

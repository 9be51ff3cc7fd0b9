// The paged 8-bit KV cache of sm_100a serving: page tables and slot maps from the requests'
// lengths, the store of new keys and values, and the attention of each request's newest
// tokens over what is stored.
#include <cuda_fp16.h>

#include "dsa_common.cuh"
#include "dsa_internal.h"
#include "dsa_serve.cuh"

namespace dsa {
namespace {

constexpr int MAX_REQ = 4096;          // requests of one call (their prefix sums sit in shared memory)
constexpr int MIN_EXP = -60, MAX_EXP = 60;  // exponents of the scales the store writes

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The request whose half-open range of a prefix array holds i: pre[b] <= i < pre[b + 1].
__device__ __forceinline__ int owner_of(const int* pre, int n, int i) {
  int lo = 0, hi = n;  // pre[lo] <= i < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------------------
// Page tables.  Released requests (new < 0) push their pages on the free stack; then request b
// takes ceil((l + n) / P) - ceil(l / P) pages from its top, in request order; token i of request
// b goes to slot table[b][(l + i) / P] * P + (l + i) % P.
// Bound by latency: a few hundred kB at most.  Every CTA scans all lengths itself (three prefix sums in shared
// memory); pushes, takes and slots are flattened over all threads (one page or four slots each, found by binary
// search).  Nothing is read that the call writes: a taken page is looked up where it comes from, the old stack or the
// row of the request that gave it back; pushes go behind the old stack, takes behind a row's old pages.  So no step
// waits for another, but for one case: where lengths or count are updated in place, one cluster does all the work,
// and its barrier stands between their reads and writes.
// ---------------------------------------------------------------------------
constexpr int TAB_THREADS = 512;

struct TableArgs {
  int n_req, width, shift, max_tokens, free_cap, in_place;
  const int32_t* lens;
  const int32_t* new_lens;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t* table;
  int32_t* slots;
  int32_t* cu;
  int32_t* lens_out;
  int32_t* count_out;
  unsigned* status;
};

__global__ void __launch_bounds__(TAB_THREADS, 1) k_build_tables(const __grid_constant__ TableArgs a) {
  pdl_prologue();
  extern __shared__ int sh[];
  const int n = a.n_req;
  int* cu = sh;                  // [n + 1] first new token of each request
  int* take = cu + n + 1;        // [n + 1] first page taken
  int* give = take + n + 1;      // [n + 1] first page given back
  int* old = give + n + 1;       // [n] tokens kept
  __shared__ long long part[3][TAB_THREADS / 32];
  __shared__ int bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int page = 1 << a.shift;
  const int rank = blockIdx.x, nthreads = gridDim.x * TAB_THREADS;
  if (tid == 0) bad = 0;
  __syncthreads();

  // thread i scans requests [i * per, (i + 1) * per)
  const int per = ceil_div(n, TAB_THREADS);
  const int b0 = min(n, tid * per), b1 = min(n, b0 + per);
  long long sum[3] = {0, 0, 0};
  int flaw = 0;
  for (int b = b0; b < b1; ++b) {
    const int l = a.lens[b], w = a.new_lens[b];
    const long long held = ((long long)l + page - 1) >> a.shift;
    const long long o = w < 0 ? 0 : l, add = w < 0 ? 0 : w;
    const long long have = (o + page - 1) >> a.shift, all = (o + add + page - 1) >> a.shift;
    if (l < 0) flaw |= 1;
    if (held > a.width || all > a.width || o + add > 0x7fffffffll) flaw |= 2;
    sum[0] += add;
    sum[1] += all - have;
    sum[2] += w < 0 ? held : 0;
    old[b] = (int)o;
  }
  if (flaw) atomicOr(&bad, flaw);
  long long excl[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    long long v = sum[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) part[k][warp] = v;
    excl[k] = v - sum[k];
  }
  __syncthreads();
  long long total[3] = {0, 0, 0};
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    for (int w = 0; w < TAB_THREADS / 32; ++w) {
      if (w < warp) excl[k] += part[k][w];
      total[k] += part[k][w];
    }
  }
  const int count = *a.free_count;
  const bool t_ok = total[0] <= a.max_tokens;
  const bool p_ok = count >= 0 && count + total[2] <= a.free_cap && count + total[2] - total[1] >= 0;
  const bool ok = bad == 0 && t_ok && p_ok;
  if (ok) {  // every sum fits 32 bits now
    for (int b = b0; b < b1; ++b) {
      const int w = a.new_lens[b], o = old[b], add = max(w, 0);
      cu[b] = (int)excl[0];
      take[b] = (int)excl[1];
      give[b] = (int)excl[2];
      excl[0] += add;
      excl[1] += ((o + add + page - 1) >> a.shift) - ((o + page - 1) >> a.shift);
      excl[2] += w < 0 ? (a.lens[b] + page - 1) >> a.shift : 0;
    }
    if (tid == 0) {
      cu[n] = (int)total[0];
      take[n] = (int)total[1];
      give[n] = (int)total[2];
    }
  } else if (rank == 0 && tid == 0) {
    if (bad & 1) report(a.status, DSA_ERR_DEVICE, DETAIL_BAD_LEN);
    else report(a.status, DSA_ERR_CAPACITY, (bad & 2) ? DETAIL_CAP_TABLE : !t_ok ? DETAIL_CAP_TOKENS : DETAIL_CAP_PAGES);
  }
  __syncthreads();
  const int at = rank * TAB_THREADS + tid;
  // the k-th page taken: from the old stack, or from the row of a request that ends
  const int freed = (int)total[2];
  auto taken = [&](int k) {
    const int i = freed - 1 - k;
    if (i < 0) return a.free_pages[count + i];
    const int b = owner_of(give, n, i);
    return a.table[(int64_t)b * a.width + (i - give[b])];
  };
  if (ok) {
    for (int i = at; i < freed; i += nthreads) {
      const int b = owner_of(give, n, i);
      a.free_pages[count + i] = a.table[(int64_t)b * a.width + (i - give[b])];
    }
    for (int i = at; i < (int)total[1]; i += nthreads) {
      const int b = owner_of(take, n, i);
      a.table[(int64_t)b * a.width + ((old[b] + page - 1) >> a.shift) + (i - take[b])] = taken(i);
    }
  }
  // slots, four tokens a thread; a token's page comes from the stack or, for the page that held
  // its request's last token, from the table
  const int live = ok ? (int)total[0] : 0;
  const bool vec = (reinterpret_cast<uintptr_t>(a.slots) & 15u) == 0;
  for (int64_t t0 = 4 * (int64_t)at; t0 < a.max_tokens; t0 += 4 * (int64_t)nthreads) {
    int v[4];
    int b = t0 < live ? owner_of(cu, n, (int)t0) : 0;
    int seen = -1, pg = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int t = (int)t0 + k;
      v[k] = -1;
      if (t < live) {
        if (t >= cu[b + 1]) {
          while (t >= cu[b + 1]) ++b;
          seen = -1;
        }
        const int pos = old[b] + (t - cu[b]);
        const int j = pos >> a.shift, have = (old[b] + page - 1) >> a.shift;
        if (j != seen) {
          pg = j < have ? a.table[(int64_t)b * a.width + j] : taken(take[b] + j - have);
          seen = j;
          if (pg < 0 || pg > (0x7fffffff >> a.shift)) {  // a table or stack that holds no page here
            report(a.status, DSA_ERR_DEVICE, DETAIL_BAD_PAGE);
            pg = -1;
          }
        }
        v[k] = pg < 0 ? -1 : (pg << a.shift) + (pos & (page - 1));
      }
    }
    if (vec && t0 + 4 <= a.max_tokens) {
      *reinterpret_cast<int4*>(a.slots + t0) = make_int4(v[0], v[1], v[2], v[3]);
    } else {
      for (int k = 0; k < 4; ++k)
        if (t0 + k < a.max_tokens) a.slots[t0 + k] = v[k];
    }
  }
  if (a.in_place && gridDim.x > 1) cluster_sync();  // every CTA has read lengths and count
  for (int i = at; i <= n; i += nthreads) {
    a.cu[i] = ok ? cu[i] : 0;
    if (i < n) a.lens_out[i] = ok ? old[i] + (cu[i + 1] - cu[i]) : a.lens[i];
  }
  if (at == 0) *a.count_out = ok ? count + freed - (int)total[1] : count;
}

// ---------------------------------------------------------------------------
// Store.  A run is a stretch of consecutive tokens whose slots ascend by one inside one page; one
// CTA handles a run of one head of K or V: the run's largest magnitude gives the smallest exponent
// e with amax <= 448 * 2^e, the page takes 2^max(e, older) (older: only if tokens before the run
// are in the page, which are rounded again when the scale grows), and the run's values x * 2^-e
// are rounded to e4m3 (nearest, ties to even).  A power of two costs at most one binade of range
// and no precision (e4m3 is relative), makes the scaling exact and lets older values move to a
// larger scale without a second error unless they become subnormal.
// Bound by memory: 2 bytes read and 1 written per element; a page's rows stay in registers between
// the maximum and the rounding.
// ---------------------------------------------------------------------------
constexpr int ST_THREADS = 128;
constexpr int ST_KEEP = 8;  // passes whose rows stay in registers (64 rows at d = 128)

struct StoreArgs {
  const __nv_bfloat16* X[2];
  int64_t hs[2], ts[2];
  uint8_t* data[2];
  float* scale[2];
  int64_t page_stride, head_stride, token_stride;
  const int32_t* slots;
  int T, Hkv, shift, num_pages, chunk;
  unsigned* status;
};

__device__ __forceinline__ uint32_t finite_max2(uint32_t m, uint32_t x) {  // per-half magnitudes, non-finite ones ignored
  x &= 0x7fff7fffu;
  const uint32_t big = ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u;  // halves whose exponent is all ones
  x &= ~((big >> 15) * 0xffffu);
  return __vmaxu2(m, x);
}

__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t x) {  // the low 16 bits
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)x));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_to_e4m3x2(uint32_t x, float f) {
  return to_e4m3x2(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xffff0000u) * f);
}
__device__ __forceinline__ uint32_t rescale_e4m3x4(uint32_t x, float f) {
  const uint32_t a = e4m3x2_to_f16x2(x), b = e4m3x2_to_f16x2(x >> 16);
  const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&b));
  return to_e4m3x2(u.x * f, u.y * f) | (to_e4m3x2(v.x * f, v.y * f) << 16);
}
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ bool good_scale(float s) { return s >= 5.42101086e-20f && s <= 1.84467441e19f; }  // 2^-64 .. 2^64

// The first set bit at or behind `from` in ST_THREADS bits, or -1.
__device__ __forceinline__ int next_bit(const uint32_t* bits, int from) {
  for (int i = from >> 5; i < ST_THREADS / 32; ++i) {
    const uint32_t w = i == from >> 5 ? bits[i] & (~0u << (from & 31)) : bits[i];
    if (w != 0) return i * 32 + __ffs(w) - 1;
  }
  return -1;
}

template <int D>
__global__ void __launch_bounds__(ST_THREADS) k_cache_store(const __grid_constant__ StoreArgs a) {
  pdl_prologue();
  constexpr int LPR = D / 8;                   // lanes of a row (16 bytes of bf16 each)
  constexpr int RPP = ST_THREADS / LPR;        // rows of a pass
  __shared__ int s_end[ST_THREADS / 32];
  __shared__ uint32_t s_max[ST_THREADS / 32];
  __shared__ uint32_t s_starts[ST_THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.y, kv = blockIdx.z;
  const int page = 1 << a.shift;
  const int64_t slots_end = (int64_t)a.num_pages << a.shift;
  const int sub = tid % LPR, r0 = tid / LPR;
  // the runs that begin among this CTA's tokens (at most as many as threads)
  const int c0 = blockIdx.x * a.chunk;
  bool starts = false;
  if (tid < a.chunk && c0 + tid < a.T) {
    const int s = a.slots[c0 + tid];
    starts = s >= 0 && ((s & (page - 1)) == 0 || c0 + tid == 0 || a.slots[c0 + tid - 1] != s - 1);
    if (starts && s >= slots_end) {
      report(a.status, DSA_ERR_DEVICE, DETAIL_BAD_SLOT);
      starts = false;
    }
  }
  const uint32_t ballot = __ballot_sync(0xffffffffu, starts);
  if (lane == 0) s_starts[warp] = ballot;
  __syncthreads();
  for (int c = next_bit(s_starts, 0); c >= 0; c = next_bit(s_starts, c + 1)) {
    const int t = c0 + c;
    const int slot = a.slots[t];
    const int off = slot & (page - 1);
    // tokens of the run
    const int most = min(page - off, a.T - t);
    int n = 0;
    for (int base = 0; base < most; base += ST_THREADS) {
      const int i = base + tid;
      const uint32_t in = __ballot_sync(0xffffffffu, i < most && a.slots[t + i] == slot + i);
      if (lane == 0) s_end[warp] = __ffs(~in) == 0 ? 32 : __ffs(~in) - 1;
      __syncthreads();
      int got = 0;
      for (int w = 0; w < ST_THREADS / 32; ++w) {
        got += s_end[w];
        if (s_end[w] < 32) break;
      }
      __syncthreads();
      n += got;
      if (got < ST_THREADS) break;
    }
    const int pg = slot >> a.shift;
    const __nv_bfloat16* x = a.X[kv] + h * a.hs[kv] + t * a.ts[kv] + sub * 8;
    uint8_t* data = a.data[kv] + pg * a.page_stride + h * a.head_stride;
    float* scale = a.scale[kv] + (int64_t)pg * a.Hkv + h;
    const float was = off > 0 ? *scale : 0.f;
    uint4 keep[ST_KEEP];
    uint32_t mx = 0;
#pragma unroll
    for (int p = 0; p < ST_KEEP; ++p) {
      const int r = p * RPP + r0;
      keep[p] = make_uint4(0, 0, 0, 0);
      if (r < n) keep[p] = *reinterpret_cast<const uint4*>(x + r * a.ts[kv]);
    }
#pragma unroll
    for (int p = 0; p < ST_KEEP; ++p)
      mx = finite_max2(finite_max2(finite_max2(finite_max2(mx, keep[p].x), keep[p].y), keep[p].z), keep[p].w);
    for (int r = ST_KEEP * RPP + r0; r < n; r += RPP) {
      const uint4 v = *reinterpret_cast<const uint4*>(x + r * a.ts[kv]);
      mx = finite_max2(finite_max2(finite_max2(finite_max2(mx, v.x), v.y), v.z), v.w);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane == 0) s_max[warp] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < ST_THREADS / 32; ++w) mx = __vmaxu2(mx, s_max[w]);
    const uint32_t top = max(mx & 0xffffu, mx >> 16);  // the run's largest magnitude as bf16 bits
    // 1.f * 2^E <= 1.75 * 2^(8 + e)
    int e = (int)(top >> 7) - 127 - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0);
    e = max(MIN_EXP, min(MAX_EXP, e));
    float now = pow2f(e);
    if (off > 0) {
      if (good_scale(was)) {
        const uint32_t wb = __float_as_uint(was);
        const int ew = (int)(wb >> 23) - 127 + ((wb & 0x7fffffu) ? 1 : 0);  // the power of two at or above it
        now = pow2f(max(e, ew));
      } else if (tid == 0) {
        report(a.status, DSA_ERR_DEVICE, DETAIL_BAD_SCALE);
      }
      if (now != was) {
        const float f = was / now;
        for (int i = tid; i < off * (D / 16); i += ST_THREADS) {
          uint4* q = reinterpret_cast<uint4*>(data + (i / (D / 16)) * a.token_stride + (i % (D / 16)) * 16);
          uint4 v = *q;
          v.x = rescale_e4m3x4(v.x, f);
          v.y = rescale_e4m3x4(v.y, f);
          v.z = rescale_e4m3x4(v.z, f);
          v.w = rescale_e4m3x4(v.w, f);
          *q = v;
        }
      }
    }
    const float f = 1.f / now;
    uint8_t* dst = data + off * a.token_stride + sub * 8;
    auto put = [&](int r, const uint4& v) {
      const uint32_t lo = bf16x2_to_e4m3x2(v.x, f) | (bf16x2_to_e4m3x2(v.y, f) << 16);
      const uint32_t hi = bf16x2_to_e4m3x2(v.z, f) | (bf16x2_to_e4m3x2(v.w, f) << 16);
      *reinterpret_cast<uint2*>(dst + r * a.token_stride) = make_uint2(lo, hi);
    };
#pragma unroll
    for (int p = 0; p < ST_KEEP; ++p)
      if (p * RPP + r0 < n) put(p * RPP + r0, keep[p]);
    for (int r = ST_KEEP * RPP + r0; r < n; r += RPP) put(r, *reinterpret_cast<const uint4*>(x + r * a.ts[kv]));
    if (tid == 0) *scale = now;
    __syncthreads();  // s_max, s_end are free again
  }
}

// ---------------------------------------------------------------------------
// Attention of the newest n_q tokens of each request over its cached keys (itself among them):
//   O = sum_j softmax_j(q . k_j ks / sqrt(d)) v_j vs,  j <= len - n_q + i for token i,
// k, v: e4m3 values, ks, vs: their page's scales.
// Bound by memory: 2 d bytes per key and KV head, read once.  All query heads of a KV head and all
// n_q tokens are rows of one m16 tile, so each key is converted once; e4m3 is exact in fp16, q is
// scaled by a power of two per row so that its 8 bits are exact in fp16 too, products accumulate
// in fp32 (mma m16n8k16; the tensor work is a fraction of what the legacy path carries).
// Weights: with x = s ks and y = x + log2(vs) (log2 units), P = 2^(y - m + P_OFF) carries the value
// scale, so pages of any scale share one accumulator, and l sums P / vs.  m lags the running
// maximum by at most P_LAG: P <= 2^15 in fp16 (11 bits), underflow 2^-34 below the maximum.
// Split: the work (64-key tiles of all requests, KV heads and row tiles, laid end to end) is
// cut into equal ranges, one per CTA, three CTAs per SM; so a long request spreads over many CTAs
// and short ones share one.  A CTA's four warps take every fourth 16 keys, each through its own
// ring of cp.async stages (no barrier in the loop), and join at the end of a unit; units cut by a
// range's end leave fp32 partials that k_cache_join adds in range order.
// ---------------------------------------------------------------------------
constexpr int AT_THREADS = 128;
constexpr int AT_WARPS = AT_THREADS / 32;
constexpr int AT_KEYS = 16;                  // keys of a warp's step
constexpr int AT_TILE = AT_KEYS * AT_WARPS;  // keys of a CTA's step
constexpr int AT_MAX_CTAS = 444;             // sizes the workspace
constexpr int AT_PER_SM = 3;
constexpr int AT_MIN_TILES = 4;              // a CTA takes at least so many tiles
constexpr float P_OFF = 10.f, P_LAG = 5.f;

struct AttendArgs {
  const __nv_bfloat16* Q;
  int64_t q_hs, q_ts;
  __nv_bfloat16* O;
  int64_t o_hs, o_ts;
  float* lse;
  const uint8_t* K;
  const uint8_t* V;
  const float* k_scale;
  const float* v_scale;
  int64_t page_stride, head_stride, token_stride;
  const int32_t* table;
  const int32_t* lens;
  float* part;  // [CTAs][2][rows][D + 2]: the CTA's first and last unit, if cut
  int n_req, width, Hkv, G, n_q, shift, num_pages, MT, T;
  float scale_log2;
  unsigned* status;
};

template <int D>
struct AttendSmem {
  static constexpr int NST = D == 128 ? 4 : 6;
  static constexpr int STAGE = AT_KEYS * D * 2 + 16;  // K rows, V rows, the two scales
  static constexpr int RING = AT_WARPS * NST * STAGE;
  static constexpr int JOIN = AT_WARPS * 16 * (D + 4) * 4;
  static constexpr int PRE = RING > JOIN ? RING : JOIN;
  static int bytes(int n_req) { return PRE + (n_req + 1) * 4; }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Key tiles of request b; a length that its table row cannot hold is cut.
__device__ __forceinline__ int req_len(const AttendArgs& a, int b, bool tell) {
  const int l = a.lens[b];
  const int64_t most = (int64_t)a.width << a.shift;
  if (l < 0 || l > most) {
    if (tell) report(a.status, DSA_ERR_DEVICE, DETAIL_BAD_LEN);
    return l < 0 ? 0 : (int)most;
  }
  return l;
}

// pre[b] = key tiles of the requests before b; returns their total.
__device__ __forceinline__ int scan_tiles(const AttendArgs& a, int* pre, bool tell) {
  __shared__ int part[AT_WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int base = 0;
  for (int b0 = 0; b0 < a.n_req; b0 += AT_THREADS) {
    const int b = b0 + tid;
    const int c = b < a.n_req ? ceil_div(req_len(a, b, tell), AT_TILE) : 0;
    int v = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) part[warp] = v;
    __syncthreads();
    int sum = 0;
    for (int w = 0; w < AT_WARPS; ++w) {
      if (w < warp) v += part[w];
      sum += part[w];
    }
    if (b < a.n_req) pre[b] = base + v - c;
    base += sum;
    __syncthreads();
  }
  if (tid == 0) pre[a.n_req] = base;
  __syncthreads();
  return base;
}

// First tile of CTA c's range when `total` tiles are cut over `n` CTAs.
__device__ __forceinline__ int64_t cut_at(int64_t total, int n, int c) { return total * c / n; }
__device__ __forceinline__ int used_ctas(int64_t total, int grid) {
  const int64_t want = (total + AT_MIN_TILES - 1) / AT_MIN_TILES;
  return want < grid ? (int)(want < 1 ? 1 : want) : grid;
}

// The row of an m16 tile -> query head and packed token
struct RowAt {
  int head, token;
};
__device__ __forceinline__ RowAt row_at(const AttendArgs& a, int b, int kvh, int row) {
  const int tok = row / a.G;
  return {kvh * a.G + row - tok * a.G, b * a.n_q + tok};
}

template <int D, bool R8>
__global__ void __launch_bounds__(AT_THREADS, AT_PER_SM) k_cache_attend(const __grid_constant__ AttendArgs a) {
  pdl_prologue();
  using L = AttendSmem<D>;
  constexpr int NST = L::NST;
  constexpr int CH = D / 16;      // 16-byte chunks of a row
  constexpr int KS = D / 16;      // k-steps of Q K^T
  constexpr int NT = D / 8;       // n-tiles of P V
  constexpr int ROWS = R8 ? 8 : 16;
  extern __shared__ __align__(16) uint8_t smem[];
  int* pre = reinterpret_cast<int*>(smem + L::PRE);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, tq = lane & 3;
  const int U = a.Hkv * a.MT;
  const int total_req = scan_tiles(a, pre, blockIdx.x == 0);
  const int64_t total = (int64_t)total_req * U;

  // requests without keys: every row is empty
  for (int i = blockIdx.x; i < a.n_req; i += gridDim.x) {
    if (pre[i + 1] > pre[i]) continue;
    for (int j = tid; j < a.n_q * a.Hkv * a.G * (D / 8); j += AT_THREADS) {
      const int row = j / (D / 8), c = j % (D / 8);
      const int head = row / a.n_q;
      const int64_t token = (int64_t)i * a.n_q + row % a.n_q;
      *reinterpret_cast<uint4*>(a.O + head * a.o_hs + token * a.o_ts + c * 8) = make_uint4(0, 0, 0, 0);
      if (c == 0 && a.lse != nullptr) a.lse[(int64_t)head * a.T + token] = -INFINITY;
    }
  }
  const int ctas = used_ctas(total, gridDim.x);
  if (total == 0 || (int)blockIdx.x >= ctas) return;
  const int64_t from = cut_at(total, ctas, blockIdx.x), to = cut_at(total, ctas, blockIdx.x + 1);

  const uint32_t ring = smem_u32(smem) + warp * NST * L::STAGE;
  const uint8_t* ring_p = smem + warp * NST * L::STAGE;

  for (int64_t at = from; at < to;) {
    // the unit (request, KV head, row tile) that holds tile `at`
    const int b = owner_of(pre, a.n_req, (int)(at / U));
    const int tiles = pre[b + 1] - pre[b];
    const int64_t base = (int64_t)pre[b] * U;
    const int unit = (int)((at - base) / tiles);
    const int64_t unit0 = base + (int64_t)unit * tiles;
    const int t0 = (int)(at - unit0);
    const int t1 = (int)min((int64_t)tiles, to - unit0);
    const int kvh = unit / a.MT, mt = unit - kvh * a.MT;
    const int len = req_len(a, b, false);
    const int rows = a.n_q * a.G;
    at = unit0 + t1;

    // Q: this lane's rows g and g + 8, scaled by a power of two per row into fp16
    uint32_t qa[KS][4];
    float rowf[2];
    int limit[2];  // last key that the row sees
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = mt * 16 + g + 8 * x;
      const bool live = row < rows && !(R8 && x == 1);
      limit[x] = live ? len - a.n_q + row / a.G : -1;
      uint32_t w[CH / 4][8];
      const RowAt ra = row_at(a, b, kvh, live ? row : 0);
      const __nv_bfloat16* q = a.Q + ra.head * a.q_hs + (int64_t)ra.token * a.q_ts;
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < CH / 4; ++i) {
        uint4 u = make_uint4(0, 0, 0, 0), v = u;
        if (live) {
          u = *reinterpret_cast<const uint4*>(q + 16 * (tq + 4 * i));
          v = *reinterpret_cast<const uint4*>(q + 16 * (tq + 4 * i) + 8);
        }
        w[i][0] = u.x; w[i][1] = u.y; w[i][2] = u.z; w[i][3] = u.w;
        w[i][4] = v.x; w[i][5] = v.y; w[i][6] = v.z; w[i][7] = v.w;
#pragma unroll
        for (int k = 0; k < 8; ++k) mx = finite_max2(mx, w[i][k]);
      }
      mx = max(mx & 0xffffu, mx >> 16);
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int e = (int)(mx >> 7);                        // biased exponent of the row's largest value
      const int up = e == 0 ? 0 : max(-114, min(110, 127 + 13 - e));  // brings it to [2^13, 2^14)
      const float f = pow2f(up);
      rowf[x] = a.scale_log2 * pow2f(-up);
#pragma unroll
      for (int i = 0; i < CH / 4; ++i) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t p = w[i][2 * s + k];
            qa[4 * i + s][2 * k + x] = f16x2(__uint_as_float(p << 16) * f, __uint_as_float(p & 0xffff0000u) * f);
          }
        }
      }
    }
    const int see_all = len - a.n_q;  // every row sees the keys up to here

    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    const int steps = t1 - t0;
    const int32_t* trow = a.table + (int64_t)b * a.width;
    // page numbers of 32 steps at a time, one per lane
    auto load_pages = [&](int i0) {
      const int key = (t0 + i0 + lane) * AT_TILE + warp * AT_KEYS;
      int pg = -1;
      if (i0 + lane < steps && key < len) {
        pg = trow[key >> a.shift];
        if (pg < 0 || pg >= a.num_pages) {
          report(a.status, DSA_ERR_DEVICE, DETAIL_BAD_PAGE);
          pg = -1;
        }
      }
      return pg;
    };
    int pages = load_pages(0), pages_next = load_pages(32);
    int seen = 0;  // steps whose pages `pages` begins with
    uint32_t have = 0;  // bit: ring stage holds keys

    auto issue = [&](int i) {
      const uint32_t st = (uint32_t)i % NST;
      have &= ~(1u << st);
      if (i < steps) {
        if (i - seen >= 32) {
          seen += 32;
          pages = pages_next;
          pages_next = load_pages(seen + 32);
        }
        const int pg = __shfl_sync(0xffffffffu, pages, i - seen);
        if (pg >= 0) {
          have |= 1u << st;
          const int key = (t0 + i) * AT_TILE + warp * AT_KEYS;
          const int64_t off = pg * a.page_stride + kvh * a.head_stride + (key & ((1 << a.shift) - 1)) * a.token_stride;
          const uint32_t dst = ring + st * L::STAGE;
#pragma unroll
          for (int k = 0; k < AT_KEYS * CH / 32; ++k) {
            const int r = (k * 32 + lane) / CH, c = (k * 32 + lane) % CH;
            // chunk places that keep the reads below free of bank conflicts (rows of 128 bytes)
            const int ck = D == 128 ? c ^ (((r & 1) << 2) | ((r >> 1) & 3)) : c;
            const int cv = D == 128 ? c ^ (((r >> 1) & 3) << 1) : c ^ ((r >> 1) & 3);
            cp_async16(dst + r * D + ck * 16, a.K + off + r * a.token_stride + c * 16);
            cp_async16(dst + AT_KEYS * D + r * D + cv * 16, a.V + off + r * a.token_stride + c * 16);
          }
          if (lane < 2) {
            const float* s = lane ? a.v_scale : a.k_scale;
            cp_async4(dst + AT_KEYS * D * 2 + lane * 4, s + (int64_t)pg * a.Hkv + kvh);
          }
        }
      }
      cp_commit();
    };

#pragma unroll 1
    for (int i = 0; i < NST - 1; ++i) issue(i);
#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
      cp_wait<NST - 2>();
      __syncwarp();
      const uint32_t st = (uint32_t)i % NST;
      const uint8_t* kp = ring_p + st * L::STAGE;
      const uint8_t* vp = kp + AT_KEYS * D;
      const float2 sc = *reinterpret_cast<const float2*>(kp + AT_KEYS * D * 2);
      bool use = (have >> st) & 1u;
      if (use && !(good_scale(sc.x) && good_scale(sc.y))) {
        if (lane == 0) report(a.status, DSA_ERR_DEVICE, DETAIL_BAD_SCALE);
        use = false;
      }
      if (use) {
        const int key0 = (t0 + i) * AT_TILE + warp * AT_KEYS;
        // S = Q K^T: n-tile j holds keys key0 + 8 j + (0 .. 7)
        float s[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
          const int r = 8 * j + g;
#pragma unroll
          for (int i2 = 0; i2 < CH / 4; ++i2) {
            const int c = tq + 4 * i2;
            const int ck = D == 128 ? c ^ (((r & 1) << 2) | ((r >> 1) & 3)) : c;
            const uint4 w = *reinterpret_cast<const uint4*>(kp + r * D + ck * 16);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f16(s[j], qa[4 * i2 + k], e4m3x2_to_f16x2(ww[k]), e4m3x2_to_f16x2(ww[k] >> 16));
          }
        }
        // V: rows 2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9 at this lane's D / 8 values
        uint32_t vw[4][D / 32];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = 2 * tq + (u & 1) + 8 * (u >> 1);
          if constexpr (D == 128) {
            const uint4 w = *reinterpret_cast<const uint4*>(vp + r * D + ((g ^ (((r >> 1) & 3) << 1)) * 16));
            vw[u][0] = w.x; vw[u][1] = w.y; vw[u][2] = w.z; vw[u][3] = w.w;
          } else {
            const uint2 w = *reinterpret_cast<const uint2*>(vp + r * D + (((g >> 1) ^ ((r >> 1) & 3)) * 16 + (g & 1) * 8));
            vw[u][0] = w.x; vw[u][1] = w.y;
          }
        }
        const float lv = log2f(sc.y), iv = 1.f / sc.y;
        float y[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int k = 0; k < 4; ++k) y[j][k] = fmaf(s[j][k], rowf[k >> 1] * sc.x, lv);
        }
        const bool edge = key0 + AT_KEYS - 1 > see_all;  // some row does not see some key
        if (edge) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (key0 + 8 * j + 2 * tq + (k & 1) > limit[k >> 1]) y[j][k] = -INFINITY;
          }
        }
        float top[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) top[x] = fmaxf(fmaxf(y[0][2 * x], y[0][2 * x + 1]), fmaxf(y[1][2 * x], y[1][2 * x + 1]));
        const bool grow = top[0] > m[0] + P_LAG || (!R8 && top[1] > m[1] + P_LAG);
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int x = 0; x < (R8 ? 1 : 2); ++x) {
            float t = fmaxf(m[x], top[x]);
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
            if (t > m[x]) {
              const float f = m[x] == -INFINITY ? 0.f : serve_ex2(m[x] - t);
              m[x] = t;
              l[x] *= f;
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                o[n][2 * x] *= f;
                o[n][2 * x + 1] *= f;
              }
            }
          }
        }
        uint32_t pa[4];
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (R8 && x == 1) {
            pa[1] = pa[3] = 0u;
            continue;
          }
          const float sh = m[x] == -INFINITY ? 0.f : P_OFF - m[x];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float p0 = serve_ex2(y[j][2 * x] + sh), p1 = serve_ex2(y[j][2 * x + 1] + sh);
            sum[x] += p0 + p1;
            pa[2 * j + x] = f16x2(p0, p1);
          }
          l[x] = fmaf(sum[x], iv, l[x]);
        }
        if (edge) {
          // Values that a row must not see: those behind the length become 0; a NaN that only some
          // rows see is taken out of the product (0 x NaN) and brought back to the rows that see it.
          uint32_t nan_any = 0;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const bool behind = key0 + 2 * tq + (u & 1) + 8 * (u >> 1) >= len;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
              if (behind) vw[u][k] = 0u;
              const uint32_t w = vw[u][k];
              nan_any |= ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;  // a byte of 0x7f or 0xff
            }
          }
          if (__any_sync(0xffffffffu, nan_any != 0u)) {
            uint32_t one[4];  // 1 where the row sees the key
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int key = key0 + 8 * j + 2 * tq;
                one[2 * j + x] = (key <= limit[x] ? 0x3c00u : 0u) | (key + 1 <= limit[x] ? 0x3c000000u : 0u);
              }
            }
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
              uint32_t nb[4];
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const uint32_t hit = (((vw[u][k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
                nb[u] = hit * 0x38u;  // e4m3 1.0 where the value is NaN
                vw[u][k] &= ~(hit * 0xffu);
              }
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                const uint32_t sel = z | ((4 + z) << 4);
                float c[4] = {0.f, 0.f, 0.f, 0.f};
                mma_f16(c, one, e4m3x2_to_f16x2(prmt(nb[0], nb[1], sel)), e4m3x2_to_f16x2(prmt(nb[2], nb[3], sel)));
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  if (c[q] > 0.f) o[4 * k + z][q] = __int_as_float(0x7fffffff);
              }
            }
          }
        }
        // O += P V: n-tile e holds value e of every lane's stretch
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          const uint32_t a01 = prmt(vw[0][k], vw[1][k], 0x5140), a23 = prmt(vw[0][k], vw[1][k], 0x7362);
          const uint32_t b01 = prmt(vw[2][k], vw[3][k], 0x5140), b23 = prmt(vw[2][k], vw[3][k], 0x7362);
          mma_f16(o[4 * k], pa, e4m3x2_to_f16x2(a01), e4m3x2_to_f16x2(b01));
          mma_f16(o[4 * k + 1], pa, e4m3x2_to_f16x2(a01 >> 16), e4m3x2_to_f16x2(b01 >> 16));
          mma_f16(o[4 * k + 2], pa, e4m3x2_to_f16x2(a23), e4m3x2_to_f16x2(b23));
          mma_f16(o[4 * k + 3], pa, e4m3x2_to_f16x2(a23 >> 16), e4m3x2_to_f16x2(b23 >> 16));
        }
      }
      __syncwarp();
      issue(i + NST - 1);
    }
    cp_wait<0>();

    // join the warps: O rows, m and l through shared memory
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
    }
    __syncthreads();  // every warp is done with its ring
    float* join = reinterpret_cast<float*>(smem);  // [warp][16][D + 4]: m, l, then O at 4
#pragma unroll
    for (int x = 0; x < (R8 ? 1 : 2); ++x) {
      float* w = join + (warp * 16 + g + 8 * x) * (D + 4);
      if (tq == 0) {
        w[0] = m[x];
        w[1] = l[x];
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        w[4 + (D / 8) * (2 * tq) + n] = o[n][2 * x];
        w[4 + (D / 8) * (2 * tq + 1) + n] = o[n][2 * x + 1];
      }
    }
    __syncthreads();
    const int in_tile = min(ROWS, rows - mt * 16);
    const bool whole = t0 == 0 && t1 == tiles;
    constexpr int TPR = D / 8;  // threads of a row
    for (int i = tid; i < in_tile * TPR; i += AT_THREADS) {
      const int row = i / TPR, c = (i % TPR) * 8;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < AT_WARPS; ++w) M = fmaxf(M, join[(w * 16 + row) * (D + 4)]);
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, lsum = 0.f;
#pragma unroll
      for (int w = 0; w < AT_WARPS; ++w) {
        const float* src = join + (w * 16 + row) * (D + 4);
        const float f = src[0] == -INFINITY ? 0.f : serve_ex2(src[0] - M);
        // a warp without a key of the row has O = 0, or NaN brought back by a masked value
        lsum += src[1] * f;
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] += src[4 + c + k] * f;
      }
      if (whole) {
        const RowAt ra = row_at(a, b, kvh, mt * 16 + row);
        const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
        uint32_t pk[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(acc[2 * k] * inv, acc[2 * k + 1] * inv);
          pk[k] = *reinterpret_cast<const uint32_t*>(&v);
        }
        *reinterpret_cast<uint4*>(a.O + ra.head * a.o_hs + (int64_t)ra.token * a.o_ts + c) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        if (c == 0 && a.lse != nullptr)
          a.lse[(int64_t)ra.head * a.T + ra.token] = lsum == 0.f ? -INFINITY : (M - P_OFF + log2f(lsum)) * 0.69314718055994531f;
      } else {
        float* w = a.part + ((int64_t)(blockIdx.x * 2 + (t0 > 0 ? 0 : 1)) * 16 + row) * (D + 4);
        if (c == 0) {
          w[0] = M;
          w[1] = lsum;
        }
        *reinterpret_cast<float4*>(w + 4 + c) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        *reinterpret_cast<float4*>(w + 8 + c) = make_float4(acc[4], acc[5], acc[6], acc[7]);
      }
    }
    __syncthreads();  // the ring may be filled again
  }
}

// Units that a range's end cut: adds their parts in range order.  A part of the unit's first tiles
// is its CTA's last one (slot 1), every other part is its CTA's first (slot 0).
template <int D>
__global__ void __launch_bounds__(AT_THREADS) k_cache_join(const __grid_constant__ AttendArgs a, int grid) {
  extern __shared__ int pre[];
  // the lengths were written before the kernel in front of this one began, so they can be read before it ends
  const int U = a.Hkv * a.MT;
  const int64_t total = (int64_t)scan_tiles(a, pre, false) * U;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int b = blockIdx.x / U, unit = blockIdx.x - b * U;
  const int tiles = pre[b + 1] - pre[b];
  if (tiles == 0) return;
  const int ctas = used_ctas(total, grid);
  const int64_t u0 = (int64_t)pre[b] * U + (int64_t)unit * tiles, u1 = u0 + tiles;
  // the CTAs whose ranges hold the unit's first and last tile: cut_at(c) <= tile < cut_at(c + 1)
  const int c0 = (int)(((u0 + 1) * ctas - 1) / total), c1 = (int)((u1 * ctas - 1) / total);
  if (c0 == c1) return;
  const int kvh = unit / a.MT, mt = unit - kvh * a.MT;
  const int rows = min(16, a.n_q * a.G - mt * 16);
  constexpr int TPR = D / 4;
  for (int i = threadIdx.x + blockIdx.y * AT_THREADS; i < rows * TPR; i += AT_THREADS * gridDim.y) {
    const int row = i / TPR, c = (i % TPR) * 4;
    float M = -INFINITY;
    for (int k = c0; k <= c1; ++k) {
      const int slot = cut_at(total, ctas, k) <= u0 ? 1 : 0;
      M = fmaxf(M, a.part[((int64_t)(k * 2 + slot) * 16 + row) * (D + 4)]);
    }
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, lsum = 0.f;
    for (int k = c0; k <= c1; ++k) {
      const int slot = cut_at(total, ctas, k) <= u0 ? 1 : 0;
      const float* w = a.part + ((int64_t)(k * 2 + slot) * 16 + row) * (D + 4);
      const float f = w[0] == -INFINITY ? 0.f : serve_ex2(w[0] - M);
      const float4 v = *reinterpret_cast<const float4*>(w + 4 + c);
      lsum += w[1] * f;
      acc[0] += v.x * f;
      acc[1] += v.y * f;
      acc[2] += v.z * f;
      acc[3] += v.w * f;
    }
    const RowAt ra = row_at(a, b, kvh, mt * 16 + row);
    const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
    const __nv_bfloat162 v0 = __floats2bfloat162_rn(acc[0] * inv, acc[1] * inv), v1 = __floats2bfloat162_rn(acc[2] * inv, acc[3] * inv);
    *reinterpret_cast<uint2*>(a.O + ra.head * a.o_hs + (int64_t)ra.token * a.o_ts + c) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&v0), *reinterpret_cast<const uint32_t*>(&v1));
    if (c == 0 && a.lse != nullptr)
      a.lse[(int64_t)ra.head * a.T + ra.token] = lsum == 0.f ? -INFINITY : (M - P_OFF + log2f(lsum)) * 0.69314718055994531f;
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int log2_page(int page) {
  for (int s = 4; s <= 8; ++s)
    if (page == (1 << s)) return s;
  return -1;
}

dsa_status validate_cache(const dsa_cache* c) {
  if (c == nullptr || c->num_pages < 1 || c->Hkv < 1 || log2_page(c->page) < 0) return DSA_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return DSA_ERR_UNSUPPORTED;
  if (c->Hkv > 4096 || (int64_t)c->num_pages * c->page > 0x7fffffffll) return DSA_ERR_UNSUPPORTED;
  if (!c->K || !c->V || !c->k_scale || !c->v_scale || !serve_aligned16(c->K) || !serve_aligned16(c->V)) return DSA_ERR_INVALID_ARG;
  if (c->token_stride < c->d || c->token_stride % 16 || c->head_stride % 16 || c->page_stride % 16) return DSA_ERR_INVALID_ARG;
  if ((c->Hkv > 1 && c->head_stride < c->d) || (c->num_pages > 1 && c->page_stride < c->d)) return DSA_ERR_INVALID_ARG;
  return DSA_OK;
}

template <int D, bool R8>
dsa_status launch_attend(AttendArgs& a, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = serve_sms(&dev, &sms);
  if (e == cudaSuccess) e = serve_allow_smem<k_cache_attend<D, R8>>(dev, AttendSmem<D>::bytes(MAX_REQ));
  const int smem = AttendSmem<D>::bytes(a.n_req);
  const int grid = min(AT_PER_SM * sms, AT_MAX_CTAS);
  if (e == cudaSuccess) e = launch_pdl(k_cache_attend<D, R8>, dim3(grid), dim3(AT_THREADS), (size_t)smem, stream, a);
  const int rows = min(16, a.n_q * a.G);
  const int per_unit = max(1, rows * (D / 4) / AT_THREADS);
  if (e == cudaSuccess)
    e = launch_pdl(k_cache_join<D>, dim3(a.n_req * a.Hkv * a.MT, per_unit), dim3(AT_THREADS), (size_t)(a.n_req + 1) * 4, stream, a, grid);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? DSA_OK : cuda_fail(e);
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

dsa_status dsa_build_tables(int32_t n_req, const int32_t* lens, const int32_t* new_lens, int32_t* free_pages,
                            int32_t free_cap, const int32_t* free_count, int32_t* block_table, int32_t width,
                            int32_t page, int32_t max_tokens, int32_t* slots, int32_t* cu_seqlens, int32_t* lens_out,
                            int32_t* free_count_out, dsa_stream stream) {
  if (n_req < 1 || width < 1 || free_cap < 1 || max_tokens < 0 || log2_page(page) < 0) return DSA_ERR_INVALID_ARG;
  if (n_req > MAX_REQ || max_tokens > (1 << 30)) return DSA_ERR_UNSUPPORTED;
  if (!lens || !new_lens || !free_pages || !free_count || !block_table || !cu_seqlens || !lens_out || !free_count_out ||
      (max_tokens > 0 && !slots))
    return DSA_ERR_INVALID_ARG;
  unsigned* st = status_ptr((cudaStream_t)stream);
  if (st == nullptr) return cuda_fail(cudaGetLastError());
  TableArgs a;
  a.n_req = n_req;
  a.width = width;
  a.shift = log2_page(page);
  a.max_tokens = max_tokens;
  a.free_cap = free_cap;
  a.lens = lens;
  a.new_lens = new_lens;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.table = block_table;
  a.slots = slots;
  a.cu = cu_seqlens;
  a.lens_out = lens_out;
  a.count_out = free_count_out;
  a.status = st;
  // (arrays that overlap in part are not in place, but as safe this way)
  auto meet = [](const int32_t* x, int64_t nx, const int32_t* y, int64_t ny) { return x < y + ny && y < x + nx; };
  a.in_place = meet(lens, n_req, lens_out, n_req) || meet(new_lens, n_req, lens_out, n_req) ||
                       meet(free_count, 1, free_count_out, 1)
                   ? 1
                   : 0;
  const int most = a.in_place ? 8 : 148;
  int ctas = 1;
  while (ctas < most && ctas * TAB_THREADS * 4 < max_tokens) ctas = min(most, ctas * 2);
  const size_t smem = (size_t)(4 * n_req + 3) * 4;
  int dev = 0, sms = 0;
  cudaError_t e = serve_sms(&dev, &sms);
  if (e == cudaSuccess) e = serve_allow_smem<k_build_tables>(dev, (4 * MAX_REQ + 3) * 4);
  if (e == cudaSuccess)
    e = a.in_place && ctas > 1 ? serve_launch_cluster(k_build_tables, dim3(ctas), dim3(TAB_THREADS), ctas, smem, (cudaStream_t)stream, a)
                               : launch_pdl(k_build_tables, dim3(ctas), dim3(TAB_THREADS), smem, (cudaStream_t)stream, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? DSA_OK : cuda_fail(e);
}

dsa_status dsa_cache_write(const dsa_cache* cache, const void* K, const void* V, int64_t k_head_stride,
                           int64_t k_token_stride, int64_t v_head_stride, int64_t v_token_stride,
                           const int32_t* slots, int32_t n_tokens, dsa_stream stream) {
  dsa_status s = validate_cache(cache);
  if (s != DSA_OK) return s;
  if (n_tokens < 0) return DSA_ERR_INVALID_ARG;
  if (n_tokens == 0) return DSA_OK;
  if (!K || !V || !slots || !serve_aligned16(K) || !serve_aligned16(V)) return DSA_ERR_INVALID_ARG;
  if (k_token_stride % 8 || v_token_stride % 8 || k_head_stride % 8 || v_head_stride % 8) return DSA_ERR_INVALID_ARG;
  unsigned* st = status_ptr((cudaStream_t)stream);
  if (st == nullptr) return cuda_fail(cudaGetLastError());
  StoreArgs a;
  a.X[0] = static_cast<const __nv_bfloat16*>(K);
  a.X[1] = static_cast<const __nv_bfloat16*>(V);
  a.hs[0] = k_head_stride;
  a.hs[1] = v_head_stride;
  a.ts[0] = k_token_stride;
  a.ts[1] = v_token_stride;
  a.data[0] = static_cast<uint8_t*>(cache->K);
  a.data[1] = static_cast<uint8_t*>(cache->V);
  a.scale[0] = cache->k_scale;
  a.scale[1] = cache->v_scale;
  a.page_stride = cache->page_stride;
  a.head_stride = cache->head_stride;
  a.token_stride = cache->token_stride;
  a.slots = slots;
  a.T = n_tokens;
  a.Hkv = cache->Hkv;
  a.shift = log2_page(cache->page);
  a.num_pages = cache->num_pages;
  // a token a CTA while CTAs are few (each may be a run of its own), up to 128 once there are enough for every SM
  int chunk = 1;
  while (chunk < ST_THREADS && (int64_t)n_tokens * cache->Hkv * 2 > (int64_t)chunk * 4096) chunk *= 2;
  a.chunk = chunk;
  a.status = st;
  const dim3 grid(ceil_div(n_tokens, a.chunk), cache->Hkv, 2);
  cudaError_t e = cache->d == 128 ? launch_pdl(k_cache_store<128>, grid, dim3(ST_THREADS), 0, (cudaStream_t)stream, a)
                                  : launch_pdl(k_cache_store<64>, grid, dim3(ST_THREADS), 0, (cudaStream_t)stream, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? DSA_OK : cuda_fail(e);
}

int64_t dsa_cache_attention_workspace(int32_t d) { return (int64_t)AT_MAX_CTAS * 2 * 16 * (d + 4) * 4; }

dsa_status dsa_cache_attention(const dsa_cache* cache, const void* Q, int32_t Hq, int64_t q_head_stride,
                               int64_t q_token_stride, const int32_t* block_table, int32_t width,
                               const int32_t* lens, int32_t n_req, int32_t n_q, void* O, int64_t o_head_stride,
                               int64_t o_token_stride, float* lse, void* workspace, size_t workspace_bytes,
                               dsa_stream stream) {
  dsa_status s = validate_cache(cache);
  if (s != DSA_OK) return s;
  if (n_req < 0 || n_q < 1 || Hq < 1 || Hq % cache->Hkv != 0) return DSA_ERR_INVALID_ARG;
  if (n_req == 0) return DSA_OK;
  if (width < 1) return DSA_ERR_INVALID_ARG;
  const int64_t most = (int64_t)width * cache->page;
  if (n_req > MAX_REQ || Hq > 4096 || n_q > 4096 || most > 0x7fffff00ll ||
      (most / AT_TILE + 1) * n_req > 0x7fffffffll)
    return DSA_ERR_UNSUPPORTED;
  if (!Q || !O || !block_table || !lens || !workspace) return DSA_ERR_INVALID_ARG;
  if (!serve_aligned16(Q) || !serve_aligned16(O) || !serve_aligned16(workspace)) return DSA_ERR_INVALID_ARG;
  if (q_head_stride % 8 || q_token_stride % 8 || o_head_stride % 8 || o_token_stride % 8) return DSA_ERR_INVALID_ARG;
  if (o_token_stride < cache->d || (Hq > 1 && o_head_stride < cache->d)) return DSA_ERR_INVALID_ARG;  // rows of O overlap
  if ((int64_t)n_req * cache->Hkv * ceil_div(n_q * (Hq / cache->Hkv), 16) > 0x7fffffffll) return DSA_ERR_UNSUPPORTED;
  if (workspace_bytes < (size_t)dsa_cache_attention_workspace(cache->d)) return DSA_ERR_CAPACITY;
  unsigned* st = status_ptr((cudaStream_t)stream);
  if (st == nullptr) return cuda_fail(cudaGetLastError());
  AttendArgs a;
  a.Q = static_cast<const __nv_bfloat16*>(Q);
  a.q_hs = q_head_stride;
  a.q_ts = q_token_stride;
  a.O = static_cast<__nv_bfloat16*>(O);
  a.o_hs = o_head_stride;
  a.o_ts = o_token_stride;
  a.lse = lse;
  a.K = static_cast<const uint8_t*>(cache->K);
  a.V = static_cast<const uint8_t*>(cache->V);
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.page_stride = cache->page_stride;
  a.head_stride = cache->head_stride;
  a.token_stride = cache->token_stride;
  a.table = block_table;
  a.lens = lens;
  a.part = static_cast<float*>(workspace);
  a.n_req = n_req;
  a.width = width;
  a.Hkv = cache->Hkv;
  a.G = Hq / cache->Hkv;
  a.n_q = n_q;
  a.shift = log2_page(cache->page);
  a.num_pages = cache->num_pages;
  a.MT = ceil_div(n_q * a.G, 16);
  a.T = n_req * n_q;
  a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)cache->d));
  a.status = st;
  const bool r8 = n_q * a.G <= 8;
  if (cache->d == 128) return r8 ? launch_attend<128, true>(a, (cudaStream_t)stream) : launch_attend<128, false>(a, (cudaStream_t)stream);
  return r8 ? launch_attend<64, true>(a, (cudaStream_t)stream) : launch_attend<64, false>(a, (cudaStream_t)stream);
}

}  // extern "C"

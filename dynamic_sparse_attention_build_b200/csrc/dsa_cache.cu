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
// and its barrier stands between their reads and writes.  197K slots of 48 prompts: 4.4 us apart, 17.5 in place (8 CTAs
// write the slots); 256 requests of one token: 9.4 us either way.
// ---------------------------------------------------------------------------
constexpr int TAB_THREADS = 512;

struct TableArgs {
  int n_req, width, shift, max_tokens, free_cap, in_place;
  int prompts;  // 1: a request that gets tokens must hold none; 2: and gets all max_tokens
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
  int* cu = sh;                  // [n + 1] first new token of each request; its length if the call is refused
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
    if (add > 0 && ((a.prompts > 0 && o > 0) || (a.prompts == 2 && add != a.max_tokens))) flaw |= 4;
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
  const bool s_ok = a.prompts != 2 || total[0] == a.max_tokens;
  const bool ok = bad == 0 && t_ok && p_ok && s_ok;
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
  } else {
    for (int b = b0; b < b1; ++b) cu[b] = a.lens[b];  // they stay: kept here, where no write of this call reaches them
    if (rank == 0 && tid == 0) {
      if (bad & 1) report(a.status, DSA_ERR_DEVICE, DETAIL_BAD_LEN);
      else if ((bad & 4) || !s_ok) report(a.status, DSA_ERR_DEVICE, DETAIL_HELD);
      else report(a.status, DSA_ERR_CAPACITY, (bad & 2) ? DETAIL_CAP_TABLE : !t_ok ? DETAIL_CAP_TOKENS : DETAIL_CAP_PAGES);
    }
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
    if (i < n) a.lens_out[i] = ok ? old[i] + (cu[i + 1] - cu[i]) : cu[i];
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
// the maximum and the rounding.  71K tokens of 16 prompts, 8 heads of d 128: 77 us, 86% of a copy's rate; one token
// for each of 64 requests: 5.3 us.
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
// Bound by memory: 2 d bytes per key and KV head, read once where a KV head has up to 16 rows (query heads
// times n_q): they are the columns of one n8 tile (or two), so each key is converted once.  Each further 16
// rows are a unit of their own and read the keys again.  32 requests of up to 8192 keys, 8 KV heads of d 128:
// 51 us with 4 rows, 80 with 16, 137 with 32; 512 tokens of 4 heads behind 16384 keys 936 us.  e4m3 is exact
// in fp16; q is scaled by a power of two per row so that its 8 bits are exact in fp16 too (elements under
// 2^-30 of their row's largest are rounded, by at most 2^-38 of it); products accumulate in fp32.
// Keys (and, in the second product, value dimensions) are the m16 side of mma
// m16n8k16, S^T = K Q^T and O^T = V^T P^T: decoding has few queries, and as the m16 side they would
// leave three quarters of the products and accumulators empty.  The tensor work is a fraction of what
// the legacy path carries; tcgen05 would want 128 rows and both operands of 8 bits in one type.
// Weights: with x = s ks and y = x + log2(vs) (log2 units), P = 2^(y - m + P_OFF) carries the value
// scale, so pages of any scale share one accumulator, and l sums P / vs.  m lags the running
// maximum by at most P_LAG: P <= 2^15 in fp16, underflow 2^-34 below the maximum.  fp16 because it holds
// e4m3 exactly and P to 11 bits, 8 times finer than the output's rounding.
// Split: the work (64-key tiles of all requests, KV heads and row tiles, laid end to end) is
// cut into equal ranges, one per CTA, a few CTAs per SM; so a long request spreads over many CTAs
// and short ones share one.  A CTA's four warps take every fourth 16 keys, each through its own
// ring of TMA stages (two boxes of 16 rows, swizzled so that the reads below have no bank conflicts;
// no barrier between warps in the loop), and join at the end of a unit; units cut by a range's end
// leave fp32 partials that k_cache_join adds in range order.
// ---------------------------------------------------------------------------
constexpr int AT_THREADS = 128;
constexpr int AT_WARPS = AT_THREADS / 32;
constexpr int AT_KEYS = 16;                  // keys of a warp's step
constexpr int AT_TILE = AT_KEYS * AT_WARPS;  // keys of a CTA's step
constexpr int AT_MAX_CTAS = 592;             // sizes the workspace
// A CTA's range is at least so long, in tiles, with the start of a unit counted as AT_START of them; a range that lies in
// a unit's start holds no key, and its CTA nothing to do.  One request of 1000 tokens, 8 KV heads: 9.4 us with 4, 10.9
// with 6, 12.4 with 8; one of 96396 tokens, 1 KV head, whose parts are many: 24, 21 and 20.
constexpr int AT_MIN_TILES = 4;
// A unit costs its tiles and this much for its start (pages, scales, Q): without it, CTAs whose range holds two units
// end last.  32 requests of up to 8192 keys, 8 heads of d 128: 58 us, 79 without; 10 of up to 4000, 16 heads of d 64:
// 19 and 33.
constexpr int AT_START = 4;
constexpr float P_OFF = 10.f, P_LAG = 5.f;
// CTAs of an SM, with at_stages() ring stages each: what counts is the bytes on their way.  d 128, a million keys of 8
// heads: 352 us with 3 CTAs of 4 stages, 409 with 2 of 6, 422 with 4 of 3 (336 now, 98% of a copy's rate; 367 to 389
// after a tenth of a second of such calls, when the power cap has taken the SM clock from 1965 to some 1750 MHz).
// d 64 (boxes half as large), 20 requests of up to 4001 tokens, 16 heads: 37 us with 4 CTAs of 6 stages, 55 with 3 of 8.
__host__ __device__ constexpr int at_per_sm(int d, int nq) { return d == 64 && nq == 1 ? 4 : 3; }
__host__ __device__ constexpr int at_stages(int d) { return d == 128 ? 4 : 6; }

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
  uint64_t wait_limit_ns;
};

template <int D>
struct AttendSmem {
  static constexpr int NST = at_stages(D);
  static constexpr int BOX = AT_KEYS * D;  // 16 rows of K or V
  static constexpr int RING = AT_WARPS * NST * 2 * BOX;
  static constexpr int JOIN = AT_WARPS * 16 * (D + 4) * 4;
  static constexpr int BAR = RING > JOIN ? RING : JOIN;        // uint64 [warp][stage]
  static constexpr int PRE = BAR + AT_WARPS * NST * 8;         // int [requests + 1], int [requests]
  static int bytes(int n_req) { return 1024 + PRE + (2 * n_req + 1) * 4; }
};

// Box of 16 rows at (page, head, token) of K or V.
__device__ __forceinline__ void tma_load_rows(void* dst, const CUtensorMap* map, uint64_t* bar, int token, int head, int page) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(token), "r"(head), "r"(page), "r"(smem_u32(bar))
      : "memory");
}
// Transposes an 8 x 8 matrix of 16-bit values, two a lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// The key that row i (0 .. 7) of an m-tile's half stands for.  Any order of the keys will do as long as both products
// share it; this one keeps 16-byte reads of K (rows i, i + 1 together) and reads of V (rows i, i + 2, ..) free of bank
// conflicts under the swizzles of 128-byte and of 64-byte rows.
template <int D>
__device__ __forceinline__ int key_of(int i) {
  if (D == 128) return (i & 1) ? (i - 1) ^ 5 : i;
  const int e = ((i >> 1) & 1) | ((i >> 2) << 2);
  return (i & 1) ? e ^ 3 : e;
}

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

// The length of request b; one that its table row cannot hold is cut.
__device__ __forceinline__ int req_len(const AttendArgs& a, int b, bool tell) {
  const int l = a.lens[b];
  const int64_t most = (int64_t)a.width << a.shift;
  if (l < 0 || l > most) {
    if (tell) report(a.status, DSA_ERR_DEVICE, DETAIL_BAD_LEN);
    return l < 0 ? 0 : (int)most;
  }
  return l;
}

// pre[b] = the cost of a unit of each request before b, in key tiles; returns their total.  len_of: their lengths.
__device__ __forceinline__ int scan_costs(const AttendArgs& a, int* pre, int* len_of, bool tell) {
  __shared__ int part[AT_WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int base = 0;
  for (int b0 = 0; b0 < a.n_req; b0 += AT_THREADS) {
    const int b = b0 + tid;
    int c = 0;
    if (b < a.n_req) {
      const int len = req_len(a, b, tell);
      if (len_of != nullptr) len_of[b] = len;
      c = len > 0 ? AT_START + ceil_div(len, AT_TILE) : 0;
    }
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

// Divisions of 64-bit numbers that nearly always fit 32 bits (a 64-bit division takes some hundred cycles).
__device__ __forceinline__ int64_t div_by(int64_t x, int64_t y) {
  return ((x | y) >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}
// `total` tiles over n CTAs: the first `rest` get one more than the others.
struct Cut {
  int64_t each;
  int rest;
  __device__ __forceinline__ Cut(int64_t total, int n) : each(div_by(total, n)), rest((int)(total - each * n)) {}
  __device__ __forceinline__ int64_t first(int c) const { return c * each + min(c, rest); }  // of CTA c's range
  __device__ __forceinline__ int holder(int64_t tile) const {                                // the CTA whose range holds it
    const int64_t longer = (each + 1) * rest;
    return (int)(tile < longer ? div_by(tile, each + 1) : rest + div_by(tile - longer, each));
  }
};
__device__ __forceinline__ int used_ctas(int64_t total, int grid) {
  const int64_t want = div_by(total + AT_MIN_TILES - 1, AT_MIN_TILES);
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

// NQ: n8 tiles of query rows (1: up to 8 rows of a KV head and request, 2: 16 at a time)
template <int D, int NQ>
__global__ void __launch_bounds__(AT_THREADS, at_per_sm(D, NQ))
k_cache_attend(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const __grid_constant__ AttendArgs a) {
  using L = AttendSmem<D>;
  constexpr int NST = L::NST;
  constexpr int CH = D / 16;      // 16-byte chunks of a row
  constexpr int KS = D / 16;      // k-steps of K Q^T
  constexpr int MTV = D / 16;     // m-tiles of V^T P^T
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  int* pre = reinterpret_cast<int*>(smem + L::PRE);
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, tq = lane & 3;
  uint8_t* ring = smem + warp * NST * 2 * L::BOX;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::BAR) + warp * NST;
  if (tid == 0) abort_word = 0;
  if (lane == 0) {
    for (int i = 0; i < NST; ++i) mbar_init(&full[i], 1);
    fence_barrier_init();
    if (warp == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int U = a.Hkv * a.MT;
  int* const len_of = pre + a.n_req + 1;
  const int total_req = scan_costs(a, pre, len_of, blockIdx.x == 0);
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
  if (total == 0 || (int)blockIdx.x >= ctas) return;  // (which lets the next grid begin as well)
  const Cut cut(total, ctas);
  const int64_t from = cut.first(blockIdx.x), to = cut.first(blockIdx.x + 1);
  // The join's CTAs may come early where the work is short (one request of 1000 keys: 10.4 us, 11.4 without); where
  // it is long they wait in places that this grid's successors want (128 requests of up to 4000 keys: 152 us, 114
  // without).
  const bool soon = cut.each <= 8;
  if (soon) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint32_t phases = 0;  // bit: parity that the stage's next load completes
  uint32_t flying = 0;  // bit: the stage has a load that nobody has waited for
  bool dead = false;    // a wait ran out: nothing is loaded or computed from here on

  for (int64_t at = from; at < to;) {
    // the unit (request, KV head, row tile) that holds tile `at`
    const int b = owner_of(pre, a.n_req, (int)div_by(at, U));
    const int cost = pre[b + 1] - pre[b], tiles = cost - AT_START;
    const int64_t base = (int64_t)pre[b] * U;
    const int unit = (int)div_by(at - base, cost);
    const int64_t unit0 = base + (int64_t)unit * cost + AT_START;  // its first tile, behind what its start costs
    const int t0 = (int)max((int64_t)0, at - unit0);
    const int t1 = (int)min((int64_t)tiles, to - unit0);
    at = min(to, unit0 + tiles);
    if (t1 <= t0) continue;
    const int kvh = unit / a.MT, mt = unit - kvh * a.MT;
    const int len = len_of[b];
    const int rows = a.n_q * a.G;

    const int steps = t1 - t0;
    const int32_t* trow = a.table + (int64_t)b * a.width;
    // page numbers and scales of 32 steps at a time, one per lane
    auto load_page = [&](int i0) {
      const int key = (t0 + i0 + lane) * AT_TILE + warp * AT_KEYS;
      if (i0 + lane >= steps || key >= len) return -1;
      const int pg = trow[key >> a.shift];
      return pg < 0 || pg >= a.num_pages ? -2 : pg;  // -2: a number that is none
    };
    auto load_scales = [&](int pg) {  // (checked where they are used)
      return pg < 0 ? make_float2(0.f, 0.f)
                    : make_float2(a.k_scale[(int64_t)pg * a.Hkv + kvh], a.v_scale[(int64_t)pg * a.Hkv + kvh]);
    };
    int page = load_page(0), page_next = load_page(32);
    float2 sc_next = make_float2(0.f, 0.f);
    int win = 0;   // steps whose pages `page` begins with
    int put = 0;   // stage of the next step to be loaded
    auto issue = [&](int i) {
      if (i < steps) {
        const int pg = __shfl_sync(0xffffffffu, page, i - win);
        if (pg >= 0 && !dead) {
          flying |= 1u << put;
          if (lane == 0) {
            uint8_t* dst = ring + put * 2 * L::BOX;
            const int token = ((t0 + i) * AT_TILE + warp * AT_KEYS) & ((1 << a.shift) - 1);
            mbar_arrive_expect_tx(&full[put], 2 * L::BOX);
            tma_load_rows(dst, &tmK, &full[put], token, kvh, pg);
            tma_load_rows(dst + L::BOX, &tmV, &full[put], token, kvh, pg);
          }
        }
        if (i - win == 31) {  // the next 32 pages; their scales are wanted a few steps from here
          win += 32;
          if (page_next == -2) report(a.status, DSA_ERR_DEVICE, DETAIL_BAD_PAGE);
          page = page_next;
          sc_next = load_scales(page);
          page_next = load_page(win + 32);
        }
      }
      put = put + 1 == NST ? 0 : put + 1;
    };
    if (page == -2) report(a.status, DSA_ERR_DEVICE, DETAIL_BAD_PAGE);

#pragma unroll 1
    for (int i = 0; i < NST - 1; ++i) issue(i);
    float2 sc = load_scales(page);  // of this lane's step of the window that is computed
    int swin = 0;

    // Q: row 8 n + g of the tile, this lane's 16-byte chunks, scaled by a power of two per row into fp16
    uint32_t qb[NQ][KS][2];
    float rowf[NQ][2];  // what turns a product of row 8 n + 2 tq + x into log2 units (without the key's scale)
    int limit[NQ][2];   // the last key that this row sees
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int row = mt * 16 + 8 * n + g;
      const bool live = row < rows;
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
#pragma unroll
      for (int i = 0; i < CH / 4; ++i) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t p = w[i][2 * s + k];
            qb[n][4 * i + s][k] = f16x2(__uint_as_float(p << 16) * f, __uint_as_float(p & 0xffff0000u) * f);
          }
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        rowf[n][x] = __shfl_sync(0xffffffffu, a.scale_log2 * pow2f(-up), (2 * tq + x) * 4);
        const int r = mt * 16 + 8 * n + 2 * tq + x;
        limit[n][x] = r < rows ? len - a.n_q + r / a.G : -1;
      }
    }
    const int see_all = len - a.n_q;  // every row sees the keys up to here

    float o[NQ][MTV][4];
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int i = 0; i < MTV; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
    float m[NQ][2], l[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
    }

    int got = 0;  // stage of step i
#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
      __syncwarp();
      if (i - swin == 32) {
        swin += 32;
        sc = sc_next;
      }
      const float2 ss = make_float2(__shfl_sync(0xffffffffu, sc.x, i - swin), __shfl_sync(0xffffffffu, sc.y, i - swin));
      const uint8_t* kp = ring + got * 2 * L::BOX;
      const uint8_t* vp = kp + L::BOX;
      bool use = ((flying >> got) & 1u) && !dead;
      if (use) {
        if (!serve_warp_wait(&full[got], (phases >> got) & 1u, a.wait_limit_ns, a.status, DETAIL_WAIT_K, abort_flag, true)) {
          dead = true;
          use = false;
        } else {
          phases ^= 1u << got;
          flying &= ~(1u << got);
          if (!(good_scale(ss.x) && good_scale(ss.y))) {
            if (lane == 0) report(a.status, DSA_ERR_DEVICE, DETAIL_BAD_SCALE);
            use = false;
          }
        }
      }
      if (use) {
        const int key0 = (t0 + i) * AT_TILE + warp * AT_KEYS;
        // S^T = K Q^T: rows g and g + 8 of the m-tile are keys key0 + key_of(g) and 8 more
        float s[NQ][4];
#pragma unroll
        for (int n = 0; n < NQ; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
        const int r0 = key_of<D>(g);
#pragma unroll
        for (int i2 = 0; i2 < CH / 4; ++i2) {
          const int c = tq + 4 * i2;
          const int ck = D == 128 ? c ^ r0 : c ^ ((r0 >> 1) & 3);
          const uint4 w0 = *reinterpret_cast<const uint4*>(kp + r0 * D + ck * 16);
          const uint4 w1 = *reinterpret_cast<const uint4*>(kp + (r0 + 8) * D + ck * 16);
          const uint32_t u0[4] = {w0.x, w0.y, w0.z, w0.w}, u1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t ka[4] = {e4m3x2_to_f16x2(u0[k]), e4m3x2_to_f16x2(u1[k]), e4m3x2_to_f16x2(u0[k] >> 16),
                                    e4m3x2_to_f16x2(u1[k] >> 16)};
#pragma unroll
            for (int n = 0; n < NQ; ++n) mma_f16(s[n], ka, qb[n][4 * i2 + k][0], qb[n][4 * i2 + k][1]);
          }
        }
        // V: the keys of k = 2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9, this lane's D / 8 values (from (D / 8) g on)
        uint32_t vw[4][D / 32];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = key_of<D>(2 * tq + (u & 1)) + 8 * (u >> 1);
          if constexpr (D == 128) {
            const uint4 w = *reinterpret_cast<const uint4*>(vp + r * D + ((g ^ (r & 7)) * 16));
            vw[u][0] = w.x; vw[u][1] = w.y; vw[u][2] = w.z; vw[u][3] = w.w;
          } else {
            const uint2 w = *reinterpret_cast<const uint2*>(vp + r * D + (((g >> 1) ^ ((r >> 1) & 3)) * 16 + (g & 1) * 8));
            vw[u][0] = w.x; vw[u][1] = w.y;
          }
        }
        const float lv = log2f(ss.y), iv = 1.f / ss.y;
        const bool edge = key0 + AT_KEYS - 1 > see_all;  // some row does not see some key
        bool grow = false;
        float y[NQ][4], top[NQ][2];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
#pragma unroll
          for (int k = 0; k < 4; ++k) y[n][k] = fmaf(s[n][k], rowf[n][k & 1] * ss.x, lv);
          if (edge) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (key0 + r0 + 8 * (k >> 1) > limit[n][k & 1]) y[n][k] = -INFINITY;
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            top[n][x] = fmaxf(y[n][x], y[n][2 + x]);
            grow |= top[n][x] - m[n][x] > P_LAG;  // (m + P_LAG would be rounded where m is large)
          }
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float t = fmaxf(m[n][x], top[n][x]);
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
              const float f = t == m[n][x] ? 1.f : m[n][x] == -INFINITY ? 0.f : serve_ex2(m[n][x] - t);
              m[n][x] = t;
              l[n][x] *= f;
#pragma unroll
              for (int i2 = 0; i2 < MTV; ++i2) {
                o[n][i2][x] *= f;
                o[n][i2][2 + x] *= f;
              }
            }
          }
        }
        uint32_t pb[NQ][2];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          float p[4];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            // y - m first: both are as large as the scores, so P_OFF - m would be off by half a step of m, which takes P
            // out of fp16's range from 2^24 on
            const float ref = m[n][x] == -INFINITY ? 0.f : m[n][x];
            p[x] = serve_ex2(y[n][x] - ref + P_OFF);
            p[2 + x] = serve_ex2(y[n][2 + x] - ref + P_OFF);
            l[n][x] = fmaf(p[x] + p[2 + x], iv, l[n][x]);
          }
          pb[n][0] = transpose8x8(f16x2(p[0], p[1]));
          pb[n][1] = transpose8x8(f16x2(p[2], p[3]));
        }
        if (edge) {
          // Values that a row must not see: those behind the length become 0; a NaN that only some
          // rows see is taken out of the product (0 x NaN) and brought back to the rows that see it.
          uint32_t nan_any = 0;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const bool behind = key0 + key_of<D>(2 * tq + (u & 1)) + 8 * (u >> 1) >= len;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
              if (behind) vw[u][k] = 0u;
              nan_any |= ((vw[u][k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;  // a byte of 0x7f or 0xff
            }
          }
          if (__any_sync(0xffffffffu, nan_any != 0u)) {
            uint32_t one[NQ][2];  // 1 where row 8 n + g sees the key
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
              const int r = mt * 16 + 8 * n + g;
              const int lim = r < rows ? len - a.n_q + r / a.G : -1;
#pragma unroll
              for (int j = 0; j < 2; ++j)
                one[n][j] = (key0 + key_of<D>(2 * tq) + 8 * j <= lim ? 0x3c00u : 0u) |
                            (key0 + key_of<D>(2 * tq + 1) + 8 * j <= lim ? 0x3c000000u : 0u);
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
              for (int z = 0; z < 2; ++z) {
                const uint32_t p01 = prmt(nb[0], nb[1], z ? 0x7362 : 0x5140), p89 = prmt(nb[2], nb[3], z ? 0x7362 : 0x5140);
                const uint32_t na[4] = {e4m3x2_to_f16x2(p01), e4m3x2_to_f16x2(p01 >> 16), e4m3x2_to_f16x2(p89), e4m3x2_to_f16x2(p89 >> 16)};
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                  float c[4] = {0.f, 0.f, 0.f, 0.f};
                  mma_f16(c, na, one[n][0], one[n][1]);
#pragma unroll
                  for (int q = 0; q < 4; ++q)
                    if (c[q] > 0.f) o[n][2 * k + z][q] = __int_as_float(0x7fffffff);
                }
              }
            }
          }
        }
        // O^T += V^T P^T: rows g and g + 8 of m-tile t are values 2 t and 2 t + 1 of every lane's stretch
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const uint32_t p01 = prmt(vw[0][k], vw[1][k], z ? 0x7362 : 0x5140), p89 = prmt(vw[2][k], vw[3][k], z ? 0x7362 : 0x5140);
            const uint32_t va[4] = {e4m3x2_to_f16x2(p01), e4m3x2_to_f16x2(p01 >> 16), e4m3x2_to_f16x2(p89), e4m3x2_to_f16x2(p89 >> 16)};
#pragma unroll
            for (int n = 0; n < NQ; ++n) mma_f16(o[n][2 * k + z], va, pb[n][0], pb[n][1]);
          }
        }
      }
      __syncwarp();  // the stage before this one has been read by every lane
      issue(i + NST - 1);
      got = got + 1 == NST ? 0 : got + 1;
    }

    // join the warps: O rows, m and l through shared memory
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[n][x] += __shfl_xor_sync(0xffffffffu, l[n][x], 4);
        l[n][x] += __shfl_xor_sync(0xffffffffu, l[n][x], 8);
        l[n][x] += __shfl_xor_sync(0xffffffffu, l[n][x], 16);
      }
    }
    if (dead) {  // loads under way end before the ring is used for something else
      if (lane == 0)
        for (int i = 0; i < NST; ++i)
          if ((flying >> i) & 1u) serve_drain(&full[i], (phases >> i) & 1u);
      flying = 0;
      __syncwarp();
    }
    __syncthreads();  // every warp is done with its ring
    float* join = reinterpret_cast<float*>(smem);  // [warp][16][D + 4]: m, l, then O at 4
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float* w = join + (warp * 16 + 8 * n + 2 * tq + x) * (D + 4);
        if (g == 0) {
          w[0] = m[n][x];
          w[1] = l[n][x];
        }
#pragma unroll
        for (int i = 0; i < MTV; ++i) {
          w[4 + (D / 8) * g + 2 * i] = o[n][i][x];
          w[4 + (D / 8) * g + 2 * i + 1] = o[n][i][2 + x];
        }
      }
    }
    __syncthreads();
    const int in_tile = min(8 * NQ, rows - mt * 16);
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
    fence_proxy_async_smem();
    __syncthreads();  // the ring may be filled again
  }
  if (!soon) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Units that a range's end cut: adds their parts in range order.  A part of the unit's first tiles
// is its CTA's last one (slot 1), every other part is its CTA's first (slot 0).
// A unit may have as many parts as there are CTAs (one request with one KV head), so a CTA takes one row at a time: its
// groups of D / 4 threads take parts in turn, 4 columns a thread, and meet in shared memory.  (With a warp for each
// row, one request of 96396 keys, 1 KV head, took 121 us.)
template <int D>
__global__ void __launch_bounds__(AT_THREADS) k_cache_join(const __grid_constant__ AttendArgs a, int grid) {
  extern __shared__ int pre[];
  // the lengths were written before the kernel in front of this one began, so they can be read before it ends
  const int U = a.Hkv * a.MT;
  const int64_t total = (int64_t)scan_costs(a, pre, nullptr, false) * U;
  const int b = blockIdx.x / U, unit = blockIdx.x - b * U;
  const int cost = pre[b + 1] - pre[b], tiles = cost - AT_START;
  const int64_t u0 = (int64_t)pre[b] * U + (int64_t)unit * cost + AT_START;
  const Cut cut(max(total, (int64_t)1), used_ctas(total, grid));
  const int c0 = cut.holder(u0), c1 = cut.holder(u0 + max(tiles, 1) - 1);  // the CTAs with the unit's first and last tile
  const int kvh = unit / a.MT, mt = unit - kvh * a.MT;
  const int rows = min(16, a.n_q * a.G - mt * 16);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (cost == 0 || c0 == c1) return;
  constexpr int TPR = D / 4, GROUPS = AT_THREADS / TPR;
  __shared__ float s_max[AT_WARPS];
  __shared__ float s_sum[GROUPS];
  __shared__ __align__(16) float s_acc[GROUPS][D];
  const int tid = threadIdx.x, grp = tid / TPR, c = (tid % TPR) * 4;
  const int n = c1 - c0 + 1;
  for (int row = blockIdx.y; row < rows; row += gridDim.y) {
    auto part = [&](int k) {  // the unit's first part is its CTA's last one, every other its CTA's first
      return a.part + ((int64_t)((c0 + k) * 2 + (k == 0 ? 1 : 0)) * 16 + row) * (D + 4);
    };
    float M = -INFINITY;
    for (int k = tid; k < n; k += AT_THREADS) M = fmaxf(M, part(k)[0]);
    M = warp_max(M);
    if ((tid & 31) == 0) s_max[tid >> 5] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < AT_WARPS; ++w) M = fmaxf(M, s_max[w]);
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, lsum = 0.f;
#pragma unroll 4
    for (int k = grp; k < n; k += GROUPS) {
      const float* w = part(k);
      const float4 v = *reinterpret_cast<const float4*>(w + 4 + c);
      const float f = w[0] == -INFINITY ? 0.f : serve_ex2(w[0] - M);
      lsum += w[1] * f;
      acc[0] += v.x * f;
      acc[1] += v.y * f;
      acc[2] += v.z * f;
      acc[3] += v.w * f;
    }
    *reinterpret_cast<float4*>(&s_acc[grp][c]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    if (c == 0) s_sum[grp] = lsum;
    __syncthreads();
    if (tid < TPR) {
#pragma unroll
      for (int i = 1; i < GROUPS; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(&s_acc[i][c]);
        acc[0] += v.x;
        acc[1] += v.y;
        acc[2] += v.z;
        acc[3] += v.w;
      }
      lsum = 0.f;
#pragma unroll
      for (int i = 0; i < GROUPS; ++i) lsum += s_sum[i];
      const RowAt ra = row_at(a, b, kvh, mt * 16 + row);
      const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
      const __nv_bfloat162 v0 = __floats2bfloat162_rn(acc[0] * inv, acc[1] * inv), v1 = __floats2bfloat162_rn(acc[2] * inv, acc[3] * inv);
      *reinterpret_cast<uint2*>(a.O + ra.head * a.o_hs + (int64_t)ra.token * a.o_ts + c) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&v0), *reinterpret_cast<const uint32_t*>(&v1));
      if (c == 0 && a.lse != nullptr)
        a.lse[(int64_t)ra.head * a.T + ra.token] = lsum == 0.f ? -INFINITY : (M - P_OFF + log2f(lsum)) * 0.69314718055994531f;
    }
    __syncthreads();  // the places are free again
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
  ServeDim dims[3] = {{c->page, c->token_stride}, {c->Hkv, c->head_stride}, {c->num_pages, c->page_stride}};
  if (!serve_apart(c->d, dims)) return DSA_ERR_INVALID_ARG;  // pages would overwrite each other
  return DSA_OK;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Tensor map over K or V of a cache: [page][head][token][byte], boxes of 16 rows.
bool make_cache_map(CUtensorMap* map, void* base, const dsa_cache& c) {
  static const EncodeTiled encode = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess || q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  if (encode == nullptr) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)c.d, (cuuint64_t)c.page, (cuuint64_t)c.Hkv, (cuuint64_t)c.num_pages};
  // strides of dimensions of size 1 are never used, but have to be valid
  const int64_t head = c.Hkv > 1 ? c.head_stride : c.page * c.token_stride;
  const int64_t page = c.num_pages > 1 ? c.page_stride : c.Hkv * head;
  const cuuint64_t strides[3] = {(cuuint64_t)c.token_stride, (cuuint64_t)head, (cuuint64_t)page};
  const cuuint32_t box[4] = {(cuuint32_t)c.d, (cuuint32_t)AT_KEYS, 1, 1}, one[4] = {1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                c.d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NQ>
dsa_status launch_attend(const dsa_cache& c, AttendArgs& a, cudaStream_t stream) {
  CUtensorMap mk, mv;
  if (!make_cache_map(&mk, c.K, c) || !make_cache_map(&mv, c.V, c)) return DSA_ERR_CUDA;
  int dev = 0, sms = 0;
  cudaError_t e = serve_sms(&dev, &sms);
  if (e == cudaSuccess) e = serve_allow_smem<k_cache_attend<D, NQ>>(dev, AttendSmem<D>::bytes(MAX_REQ));
  const int smem = AttendSmem<D>::bytes(a.n_req);
  // As many CTAs as an SM holds while the lengths in shared memory are short.  Above some 860 requests (d 64, one n8
  // tile) or 1250 (d 128) fewer fit and the last ranges wait for the first; nothing depends on their running together.
  // 32 query heads on 8, d 128, up to 300 keys each: 1024 requests 167 us (50 by their bytes), 4096 1226 us (201); the
  // join, whose CTAs each sum all lengths, takes 37 and 334 of them.
  const int grid = min(at_per_sm(D, NQ) * sms, AT_MAX_CTAS);
  if (e == cudaSuccess) e = launch_pdl(k_cache_attend<D, NQ>, dim3(grid), dim3(AT_THREADS), (size_t)smem, stream, mk, mv, a);
  const int rows = min(16, a.n_q * a.G);
  const int units = a.n_req * a.Hkv * a.MT, per_unit = max(1, min(rows, 2048 / units));  // a CTA a row while CTAs are few
  if (e == cudaSuccess)
    e = launch_pdl(k_cache_join<D>, dim3(units, per_unit), dim3(AT_THREADS), (size_t)(a.n_req + 1) * 4, stream, a, grid);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? DSA_OK : cuda_fail(e);
}

dsa_status launch_tables(int32_t n_req, const int32_t* lens, const int32_t* new_lens, int32_t* free_pages,
                         int32_t free_cap, const int32_t* free_count, int32_t* block_table, int32_t width,
                         int32_t page, int32_t max_tokens, int32_t* slots, int32_t* cu_seqlens, int32_t* lens_out,
                         int32_t* free_count_out, int prompts, dsa_stream stream) {
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
  a.prompts = prompts;
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

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

dsa_status dsa_build_tables(int32_t n_req, const int32_t* lens, const int32_t* new_lens, int32_t* free_pages,
                            int32_t free_cap, const int32_t* free_count, int32_t* block_table, int32_t width,
                            int32_t page, int32_t max_tokens, int32_t* slots, int32_t* cu_seqlens, int32_t* lens_out,
                            int32_t* free_count_out, dsa_stream stream) {
  return launch_tables(n_req, lens, new_lens, free_pages, free_cap, free_count, block_table, width, page, max_tokens,
                       slots, cu_seqlens, lens_out, free_count_out, 0, stream);
}

dsa_status dsa_build_prompt_tables(int32_t n_req, const int32_t* lens, const int32_t* new_lens, int32_t* free_pages,
                                   int32_t free_cap, const int32_t* free_count, int32_t* block_table, int32_t width,
                                   int32_t page, int32_t max_tokens, int32_t* slots, int32_t* cu_seqlens,
                                   int32_t* lens_out, int32_t* free_count_out, int32_t single, dsa_stream stream) {
  if (single != 0 && single != 1) return DSA_ERR_INVALID_ARG;
  return launch_tables(n_req, lens, new_lens, free_pages, free_cap, free_count, block_table, width, page, max_tokens,
                       slots, cu_seqlens, lens_out, free_count_out, 1 + single, stream);
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
  // keys and values that overlap (which reading them bears), and their scales
  auto distance = [](const void* x, const void* y) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
    return (int64_t)(a < b ? b - a : a - b);
  };
  ServeDim dims[4] = {{cache->page, cache->token_stride},
                      {cache->Hkv, cache->head_stride},
                      {cache->num_pages, cache->page_stride},
                      {2, distance(cache->K, cache->V)}};
  if (!serve_apart(cache->d, dims) ||
      distance(cache->k_scale, cache->v_scale) < (int64_t)cache->num_pages * cache->Hkv * (int64_t)sizeof(float))
    return DSA_ERR_INVALID_ARG;
  if (n_tokens > (1 << 30)) return DSA_ERR_UNSUPPORTED;
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
  // A token a CTA while CTAs are few (each may be a run of its own), up to 128 once there are enough for every SM.
  // 64 tokens of 64 requests, 8 heads: 5.3 us with 1, 23 with 16, 82 with 128; 71K tokens of 16 prompts: 1177, 107 and 77.
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
      (most / AT_TILE + 1 + AT_START) * n_req > 0x7fffffffll)
    return DSA_ERR_UNSUPPORTED;
  if (!Q || !O || !block_table || !lens || !workspace) return DSA_ERR_INVALID_ARG;
  if (!serve_aligned16(Q) || !serve_aligned16(O) || !serve_aligned16(workspace)) return DSA_ERR_INVALID_ARG;
  if (q_head_stride % 8 || q_token_stride % 8 || o_head_stride % 8 || o_token_stride % 8) return DSA_ERR_INVALID_ARG;
  ServeDim o_dims[2] = {{(int64_t)n_req * n_q, o_token_stride}, {Hq, o_head_stride}};
  if (o_token_stride < cache->d || !serve_apart(cache->d, o_dims)) return DSA_ERR_INVALID_ARG;  // rows of O overlap
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
  a.wait_limit_ns = wait_limit_ns();
  // (one n8 tile where it holds all rows: 64 ragged requests of 4 query heads a KV head 191 us, 272 with two)
  const bool one = n_q * a.G <= 8;
  if (cache->d == 128) return one ? launch_attend<128, 1>(*cache, a, (cudaStream_t)stream) : launch_attend<128, 2>(*cache, a, (cudaStream_t)stream);
  return one ? launch_attend<64, 1>(*cache, a, (cudaStream_t)stream) : launch_attend<64, 2>(*cache, a, (cudaStream_t)stream);
}

}  // extern "C"

// Block tables and slot maps from request lengths, and the write of keys and values into the 8-bit paged cache.
#include "attn.h"
#include "attn.cuh"

#include <algorithm>

namespace moe {
namespace {

// ------------------------------------------------------------------ block tables and slot maps
// One launch: every CTA takes the two exclusive sums over the requests (tokens, blocks) for itself, in shared memory,
// then writes its share of the table and of the tokens' slots. The sums cost a CTA one pass over 8 bytes a request out
// of L2, which is less than a second launch; with 4 CTAs an SM in place of 2, 1024 requests took 11.6 us against
// 7.7. (CTAs of 1024 threads, one an SM: 6.5 us against 7.0 for 1024 requests, 4.0 against 3.5 for 64.)
// What bounds a call is the latency of that chain (lengths, sums, then table or ids) and, before it, the host, which takes
// 8 us to issue a call (five results to allocate). On the GPU 1024 requests with tables of 2048 entries and 131072 new
// tokens take 7.0 us, 6.8 MB; 64 requests 3.6 us.
constexpr int kAssignThreads = 512, kAssignWarps = kAssignThreads / 32;
constexpr int kAssignPiece = 128;  // table entries that a warp writes at a time: 16 bytes a lane

// Sums stop at 2^31 - 1 (so added, values from 0 to there may be added in any order).
__device__ __forceinline__ uint32_t sat_add(uint32_t x, uint32_t y) { return min(x + y, 0x7FFFFFFFu); }
// the lanes' sum
__device__ __forceinline__ uint32_t sat_sum(uint32_t x) {
  const uint32_t lo = __reduce_add_sync(~0u, x & 0xFFFFu), hi = __reduce_add_sync(~0u, x >> 16) + (lo >> 16);
  return hi > 0x7FFFu ? 0x7FFFFFFFu : hi << 16 | (lo & 0xFFFFu);
}

struct Request {
  uint32_t ctx, fresh, n0, n1;  // tokens held and new, blocks held and blocks then needed
};
__device__ __forceinline__ Request request_of(const moe_kv_assign_args& a, int b) {
  Request r;
  r.ctx = static_cast<uint32_t>(max(0, a.ctx_lens[b]));
  r.fresh = static_cast<uint32_t>(max(0, a.new_lens[b]));
  const uint32_t bs = static_cast<uint32_t>(a.block_size), len = r.ctx + r.fresh;  // below 2^32
  r.n0 = r.ctx ? (r.ctx - 1) / bs + 1 : 0;
  r.n1 = len ? (len - 1) / bs + 1 : 0;
  return r;
}

__global__ void __launch_bounds__(kAssignThreads) kv_assign_kernel(const __grid_constant__ moe_kv_assign_args a) {
  extern __shared__ int32_t sm[];
  wait_for_previous();
  const int n = a.n_requests, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* tok0 = sm;             // [n + 1] first token of each request
  int32_t* blk0 = tok0 + n + 1;   // [n + 1] first taken block of each request
  uint32_t* ctx = reinterpret_cast<uint32_t*>(blk0 + n + 1);  // [n] tokens held
  const uint32_t bs = static_cast<uint32_t>(a.block_size);
  auto blocks_held = [&](int b) { return ctx[b] ? (ctx[b] - 1) / bs + 1 : 0u; };
  __shared__ uint32_t warp_tok[kAssignWarps], warp_blk[kAssignWarps];
  const int per = (n + kAssignThreads - 1) / kAssignThreads;
  const int b0 = min(n, tid * per), b1 = min(n, b0 + per);
  uint32_t tok = 0, blk = 0;
  for (int b = b0; b < b1; ++b) {
    const Request r = request_of(a, b);
    tok = sat_add(tok, r.fresh);
    blk = sat_add(blk, r.n1 - r.n0);
  }
  if (warp * 32 * per < n) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t t = __shfl_up_sync(~0u, tok, d), k = __shfl_up_sync(~0u, blk, d);
      if (lane >= d) tok = sat_add(tok, t), blk = sat_add(blk, k);
    }
  }
  if (lane == 31) warp_tok[warp] = tok, warp_blk[warp] = blk;
  const uint32_t tok_up = __shfl_up_sync(~0u, tok, 1), blk_up = __shfl_up_sync(~0u, blk, 1);
  __syncthreads();
  const bool below = lane < warp;  // (there are no more than 32 warps)
  tok = sat_add(sat_sum(below ? warp_tok[lane] : 0u), lane ? tok_up : 0u);
  blk = sat_add(sat_sum(below ? warp_blk[lane] : 0u), lane ? blk_up : 0u);
  for (int b = b0; b < b1; ++b) {
    const Request r = request_of(a, b);
    tok0[b] = static_cast<int32_t>(tok);
    blk0[b] = static_cast<int32_t>(blk);
    ctx[b] = r.ctx;
    if (blockIdx.x == 0) {
      a.cu_new[b] = static_cast<int32_t>(tok);
      a.kv_lens[b] = static_cast<int32_t>(sat_add(r.ctx, r.fresh));
    }
    tok = sat_add(tok, r.fresh);
    blk = sat_add(blk, r.n1 - r.n0);
  }
  if (tid == kAssignThreads - 1) {  // the last thread's sums end at the totals (it may own no request)
    tok0[n] = static_cast<int32_t>(tok);
    blk0[n] = static_cast<int32_t>(blk);
    if (blockIdx.x == 0) a.cu_new[n] = static_cast<int32_t>(tok), a.used[0] = static_cast<int32_t>(blk);
  }
  __syncthreads();

  // the table: a warp takes pieces of a row
  const int pieces = (a.max_blocks + kAssignPiece - 1) / kAssignPiece;
  const bool vec = (reinterpret_cast<uintptr_t>(a.block_table) & 15) == 0 && a.table_stride % 4 == 0;
  const int warps = gridDim.x * kAssignWarps, warp0 = blockIdx.x * kAssignWarps + warp;
  const int step_b = pieces ? warps / pieces : n, step_p = pieces ? warps % pieces : 0;
  for (int b = pieces ? warp0 / pieces : n, p = pieces ? warp0 % pieces : 0; b < n; b += step_b, p += step_p) {
    if (p >= pieces) {
      p -= pieces;
      if (++b >= n) break;
    }
    const int c0 = p * kAssignPiece;
    const uint32_t n0 = blocks_held(b);
    const uint32_t taken = static_cast<uint32_t>(blk0[b + 1] - blk0[b]);  // (past 2^31 blocks all told: none is there)
    if (n0 >= static_cast<uint32_t>(c0) + kAssignPiece) continue;
    int32_t* row = a.block_table + b * a.table_stride + c0;
    if (vec && n0 + taken <= static_cast<uint32_t>(c0) && c0 + kAssignPiece <= a.max_blocks) {
      reinterpret_cast<int4*>(row)[lane] = make_int4(-1, -1, -1, -1);
      continue;
    }
#pragma unroll
    for (int j = 0; j < kAssignPiece; j += 32) {
      const uint32_t c = static_cast<uint32_t>(c0 + j + lane);
      const long long f = static_cast<long long>(blk0[b]) + (c - n0);
      if (c >= n0 && c < static_cast<uint32_t>(a.max_blocks))
        row[j + lane] = (c - n0 < taken && f < a.n_free) ? a.free_blocks[f] : -1;
    }
  }
  // tokens
  const int total = tok0[n];
  for (long long t = static_cast<long long>(blockIdx.x) * kAssignThreads + tid; t < a.max_tokens;
       t += static_cast<long long>(gridDim.x) * kAssignThreads) {
    long long slot = -1;
    int pos = -1;
    if (t < total) {
      int lo = 0, hi = n - 1;  // the last request whose first token is <= t (requests without tokens share theirs)
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tok0[mid] <= t) lo = mid; else hi = mid - 1;
      }
      const uint32_t at = ctx[lo] + static_cast<uint32_t>(t - tok0[lo]);  // below 2^32: its slot is right past 2^31 too
      pos = static_cast<int>(min(at, 0x7FFFFFFFu));
      const uint32_t c = at / bs, n0 = blocks_held(lo);
      int id = -1;
      if (c < static_cast<uint32_t>(a.max_blocks)) {
        if (c < n0) {
          id = a.block_table[lo * a.table_stride + c];
        } else {
          const long long f = static_cast<long long>(blk0[lo]) + (c - n0);
          if (f < a.n_free) id = a.free_blocks[f];
        }
      }
      if (id >= 0) slot = static_cast<long long>(id) * bs + at % bs;
    }
    a.slot_map[t] = slot;
    a.positions[t] = pos;
  }
}

// ------------------------------------------------------------------ the write into the cache
// The unit of work is a run: the call's tokens of one block, for one kv head, K or V. A run's magnitude decides the
// block's scale before any code can be written, so its tokens stay in registers between the two steps (one read). A CTA
// takes the runs that begin in its window of block_size tokens; they end at most a block further on. Its warps take the
// window's tokens in turn whatever runs they belong to, so that their rows are on their way at once: what bounds a call
// is the latency of one chain (slots, rows and scales, barriers, codes), not the bytes. One call after another, 16022
// tokens of 8 heads of 128 take 18.7 us, 98.6 MB, 5.3 TB/s, and 64 single tokens 3.1 us.
constexpr int kAppendThreads = 256, kAppendWarps = kAppendThreads / 32;
// CTAs an SM for all but the largest blocks: more hide more of that latency (16022 tokens: 19.6 us with 5,
// 18.9 with 6; the same chain took 24.5 with 4).
constexpr int kAppendCtas = 6;
// Up to this many tokens a window is a token a warp, as many CTAs as a decode step can use; where they are a prompt all
// the same, the CTA at each block's beginning takes the block. 256 tokens, 8 heads of 128, blocks of 64: as single tokens
// 5.1 us against 9.0 with a block a window, as a prompt 4.9 against 2.5; 512: 7.3 against 9.2, and 5.6 against 2.6.
constexpr int kAppendShort = 256;
constexpr int kMinScaleLog2 = -40, kMaxScaleLog2 = 40;

// log2 of the smallest power of two s (from 2^-40 to 2^40) with amax / s <= 448 = 1.75 * 2^8
__device__ __forceinline__ int scale_log2(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127;
  const int k = e - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(kMaxScaleLog2, max(kMinScaleLog2, k));
}
__device__ __forceinline__ float pow2i(int k) { return __uint_as_float(static_cast<uint32_t>(k + 127) << 23); }

template <int V>
struct Words { uint32_t w[V]; };  // V 32-bit words: 2V values

template <int V>
__device__ __forceinline__ Words<V> load_words(const uint16_t* p) {
  Words<V> r;
  if constexpr (V == 1) r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  if constexpr (V == 2) { const uint2 v = *reinterpret_cast<const uint2*>(p); r.w[0] = v.x; r.w[1] = v.y; }
  if constexpr (V == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
  }
  return r;
}

// The same, issued where it stands (the compiler would move a load to its only use, behind a branch on other loads).
template <int V>
__device__ __forceinline__ Words<V> load_words_here(const uint16_t* p) {
  Words<V> r;
  if constexpr (V == 1) asm volatile("ld.global.b32 %0, [%1];" : "=r"(r.w[0]) : "l"(p));
  if constexpr (V == 2) asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[1]) : "l"(p));
  if constexpr (V == 4)
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]) : "l"(p));
  return r;
}

__device__ __forceinline__ int64_t load_here(const int64_t* p) {
  int64_t v;
  asm volatile("ld.global.b64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float load_here(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}

// the larger magnitudes of two pairs of values; a NaN gives way, an infinity stays
template <class T>
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t x) {
  if constexpr (T::kCode == 0) {
    const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&m),
                                     __habs2(*reinterpret_cast<const __nv_bfloat162*>(&x)));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&m), __habs2(*reinterpret_cast<const __half2*>(&x)));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

// the largest finite magnitude
template <class T, int V>
__device__ __forceinline__ float finite_amax(const Words<V>& x, float m) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float2 f = T::unpack(x.w[i]);
    if (finite_bits(f.x)) m = fmaxf(m, fabsf(f.x));
    if (finite_bits(f.y)) m = fmaxf(m, fabsf(f.y));
  }
  return m;
}

__device__ __forceinline__ float warp_max(float m) {
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
  return m;
}

template <class T, int V>
__device__ __forceinline__ float row_amax(const Words<V>& x) {
  uint32_t m2 = 0;
#pragma unroll
  for (int k = 0; k < V; ++k) m2 = max_abs2<T>(m2, x.w[k]);
  const float2 mm = T::unpack(m2);
  const float m = fmaxf(mm.x, mm.y);
  return finite_bits(m) ? m : finite_amax<T, V>(x, 0.0f);  // seldom: infinities take no part
}

template <class T, int V>
__device__ __forceinline__ void store_codes(uint8_t* dst, const Words<V>& x, float inv) {
  uint32_t c[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float2 f = T::unpack(x.w[i]);
    c[i] = to_e4m3x2(f.x * inv, f.y * inv);
  }
  if constexpr (V == 1) *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(c[0]);
  if constexpr (V == 2) *reinterpret_cast<uint32_t*>(dst) = c[0] | (c[1] << 16);
  if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// codes of one row times ratio (below 1: a power of two, or 0 where the old scale was 0 and so were the values)
template <int V>
__device__ __forceinline__ void rescale_row(uint8_t* row, float ratio) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float2 f = from_e4m3x2(reinterpret_cast<uint16_t*>(row)[i]);
    reinterpret_cast<uint16_t*>(row)[i] = static_cast<uint16_t>(to_e4m3x2(f.x * ratio, f.y * ratio));
  }
}

// HOLD: tokens of a window that a warp holds, block_size / 8
template <class T, int D, int HOLD>
__global__ void __launch_bounds__(kAppendThreads, HOLD * D <= 1024 ? kAppendCtas : 1)
    kv_append_kernel(const __grid_constant__ moe_kv_append_args a, int window) {
  constexpr int V = D / 64;  // words of a row per lane
  constexpr int BS = HOLD * kAppendWarps, BLOCK_LOG2 = HOLD == 2 ? 4 : HOLD == 4 ? 5 : HOLD == 8 ? 6 : 7;
  constexpr int SPAN = 2 * BS, WORDS = SPAN / 32;
  static_assert(BS == 1 << BLOCK_LOG2 && SPAN <= kAppendThreads, "block sizes 16, 32, 64, 128");
  __shared__ float amax_sh[SPAN];
  __shared__ int32_t blk_sh[SPAN];
  __shared__ int16_t off_sh[SPAN], first_sh[SPAN], end_sh[SPAN];
  __shared__ int32_t before_sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const uint16_t* x = static_cast<const uint16_t*>(is_v ? a.v : a.k) + h * (is_v ? a.v_head : a.k_head) + lane * 2 * V;
  const int64_t x_token = is_v ? a.v_token : a.k_token;
  uint8_t* codes = static_cast<uint8_t*>(is_v ? a.v_codes : a.k_codes) + lane * 2 * V;
  float* scales = is_v ? a.v_scale : a.k_scale;
  const int64_t n_slots = static_cast<int64_t>(a.num_blocks) << BLOCK_LOG2;
  auto slot_at = [&](int64_t t) -> int64_t {  // -1: none
    if (t < 0 || t >= a.n_tokens) return -1;
    const int64_t s = a.slot_map[t];
    return s >= 0 && s < n_slots ? s : -1;
  };
  wait_for_previous();
  // token i of the span from the window's first token on; warp w holds i = w, w + 8, ..
  const int64_t window0 = static_cast<int64_t>(gridDim.x - 1 - blockIdx.x) * window;  // a last, ragged window begins first
  Words<V> keep[HOLD];
  auto load_run = [&](int64_t t, int len) {  // its tokens t .. t + len - 1, dealt out to the warps
#pragma unroll
    for (int j = 0; j < HOLD; ++j)
      if (warp + j * kAppendWarps < len) keep[j] = load_words_here<V>(x + (t + warp + j * kAppendWarps) * x_token);
  };
  // the largest finite magnitude of a run whose tokens are held (one barrier)
  auto run_amax = [&](int len) {
    uint32_t m2 = 0;
#pragma unroll
    for (int j = 0; j < HOLD; ++j)
      if (warp + j * kAppendWarps < len)
#pragma unroll
        for (int k = 0; k < V; ++k) m2 = max_abs2<T>(m2, keep[j].w[k]);
    const float2 mm = T::unpack(m2);
    float m = fmaxf(mm.x, mm.y);
    if (!finite_bits(m)) {  // seldom: infinities take no part
      m = 0.0f;
#pragma unroll
      for (int j = 0; j < HOLD; ++j)
        if (warp + j * kAppendWarps < len) m = finite_amax<T, V>(keep[j], m);
    }
    m = warp_max(m);
    if (lane == 0) amax_sh[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAppendWarps; ++w) m = fmaxf(m, amax_sh[w]);
    return m;
  };

  // Most windows of a long prompt are one whole block: nothing to look for, no old scale. Its slots and rows are asked for
  // together.
  const bool early = window == BS && window0 + BS <= a.n_tokens;
  if (early) {
    constexpr int SL = BS < 32 ? 1 : BS / 32;
    const int64_t s0 = load_here(a.slot_map + window0);
    int64_t slot[SL];
#pragma unroll
    for (int i = 0; i < SL; ++i) slot[i] = load_here(a.slot_map + window0 + ((i * 32 + lane) & (BS - 1)));
    load_run(window0, BS);
    bool whole = s0 >= 0 && s0 < n_slots && (s0 & (BS - 1)) == 0;
#pragma unroll
    for (int i = 0; i < SL; ++i) whole &= slot[i] == s0 + ((i * 32 + lane) & (BS - 1));
    if (__all_sync(~0u, whole)) {
      const int64_t at = (s0 >> BLOCK_LOG2) * a.n_kv_heads + h;
      const float scale = pow2i(scale_log2(run_amax(BS))), inv = 1.0f / scale;
      if (threadIdx.x == 0) scales[at] = scale;
      uint8_t* base = codes + ((at << BLOCK_LOG2) + warp) * D;
#pragma unroll
      for (int j = 0; j < HOLD; ++j) store_codes<T, V>(base + j * kAppendWarps * D, keep[j], inv);
      return;
    }
  }

  const int i_own = threadIdx.x;
  if (i_own < SPAN) {
    const int64_t s = slot_at(window0 + i_own);
    blk_sh[i_own] = s >= 0 ? static_cast<int32_t>(s >> BLOCK_LOG2) : -1;
    off_sh[i_own] = static_cast<int16_t>(s & (BS - 1));
  }
  if (threadIdx.x == kAppendThreads - 1) {
    const int64_t s = slot_at(window0 - 1);
    before_sh = s >= 0 ? static_cast<int32_t>(s >> BLOCK_LOG2) : -1;
  }
  __syncthreads();
  // where runs begin, and where one before ends (a run begins, or there is no slot)
  uint32_t begins[WORDS], stops[WORDS];
#pragma unroll
  for (int w = 0; w < WORDS; ++w) {
    const int i = 32 * w + lane, blk = blk_sh[i], prev = i ? blk_sh[i - 1] : before_sh;
    begins[w] = __ballot_sync(~0u, blk >= 0 && blk != prev);
    stops[w] = __ballot_sync(~0u, blk < 0 || blk != prev);
  }
  auto next_stop = [&](int from) {  // the first stop from `from` on, or SPAN
    int at = SPAN;
#pragma unroll
    for (int w = WORDS - 1; w >= 0; --w) {
      const uint32_t m = from <= 32 * w ? stops[w] : from < 32 * w + 32 ? stops[w] & (~0u << (from & 31)) : 0;
      if (m) at = 32 * w + __ffs(m) - 1;
    }
    return at;
  };
  auto last_begin = [&](int to) {  // the last beginning up to `to`, or -1
    int at = -1;
#pragma unroll
    for (int w = 0; w < WORDS; ++w) {
      const uint32_t m = to >= 32 * w + 31 ? begins[w] : to >= 32 * w ? begins[w] & (~0u >> (31 - (to & 31))) : 0;
      if (m) at = 32 * w + 31 - __clz(m);
    }
    return at;
  };
  int first = SPAN;  // the window's first run; its last ends at `end`
#pragma unroll
  for (int w = WORDS - 1; w >= 0; --w)
    if (begins[w]) first = 32 * w + __ffs(begins[w]) - 1;
  if (first >= window) return;
  const int end = next_stop(window);
  if (next_stop(first + 1) == end && end - first <= BS) {  // one run: its magnitude is one maximum over the CTA
    const int len = end - first, off = off_sh[first];
    if (!(early && first == 0)) load_run(window0 + first, len);
    const int64_t at = static_cast<int64_t>(blk_sh[first]) * a.n_kv_heads + h;
    const float old = off > 0 ? load_here(scales + at) : 0.0f;
    const float want = pow2i(scale_log2(run_amax(len)));  // (its barrier: the old scale is read before it is written)
    const float scale = off > 0 && old >= want ? old : want, inv = 1.0f / scale;
    uint8_t* base = codes + (at << BLOCK_LOG2) * D;
    if (off > 0 && scale > old && old >= 0.0f)
      for (int r = warp; r < off; r += kAppendWarps) rescale_row<V>(base + r * D, old / scale);
    if (threadIdx.x == 0) scales[at] = scale;
#pragma unroll
    for (int j = 0; j < HOLD; ++j)
      if (const int i = warp + j * kAppendWarps; i < len) store_codes<T, V>(base + off_sh[first + i] * D, keep[j], inv);
    return;
  }
  if (i_own < SPAN) {
    first_sh[i_own] = static_cast<int16_t>(last_begin(i_own));
    end_sh[i_own] = static_cast<int16_t>(next_stop(i_own + 1));
  }
  // Several runs: each token's magnitude, a barrier, then each token's run's maximum, scale and codes. The loops are kept
  // small and read one token ahead; the second reads the rows again (out of L1). Unrolled over all tokens of a warp, with
  // the rows in registers, a call of 64 single tokens took 11 us, most of it for fetching instructions.
  const int i0 = warp + (max(first - warp, 0) + kAppendWarps - 1) / kAppendWarps * kAppendWarps;
  Words<V> row, next;
  float old = 0.0f, next_old = 0.0f;
  auto ahead = [&](int i, bool scale) {
    if (i < end && blk_sh[i] >= 0) {
      next = load_words_here<V>(x + (window0 + i) * x_token);
      // A run's first token writes the new scale, max(old, what the run wants); for its others it makes no difference
      // whether they read the old or the new.
      if (scale) next_old = load_here(scales + static_cast<int64_t>(blk_sh[i]) * a.n_kv_heads + h);
    }
  };
  ahead(i0, false);
#pragma unroll 1
  for (int i = i0; i < end; i += kAppendWarps) {
    row = next;
    ahead(i + kAppendWarps, false);
    if (blk_sh[i] >= 0) {
      const float m = warp_max(row_amax<T, V>(row));
      if (lane == 0) amax_sh[i] = m;
    }
  }
  ahead(i0, true);
  __syncthreads();
#pragma unroll 1
  for (int i = i0; i < end; i += kAppendWarps) {
    row = next, old = next_old;
    ahead(i + kAppendWarps, true);
    if (blk_sh[i] < 0) continue;
    const int s = first_sh[i], off = off_sh[s];
    const int64_t at = static_cast<int64_t>(blk_sh[i]) * a.n_kv_heads + h;
    float m = 0.0f;
    for (int j = s + lane; j < end_sh[i]; j += 32) m = fmaxf(m, amax_sh[j]);
    const float want = pow2i(scale_log2(warp_max(m)));
    const float scale = off > 0 && old >= want ? old : want;
    uint8_t* base = codes + (at << BLOCK_LOG2) * D;
    if (i == s) {
      if (off > 0 && scale > old && old >= 0.0f)  // the codes that are there, for the larger scale
        for (int r = 0; r < off; ++r) rescale_row<V>(base + r * D, old / scale);
      if (lane == 0) scales[at] = scale;
    }
    store_codes<T, V>(base + off_sh[i] * D, row, 1.0f / scale);
  }
}

template <class T, int D>
cudaError_t append_dim(const moe_kv_append_args& a, cudaStream_t stream) {
  const int window = a.n_tokens <= kAppendShort ? kAppendWarps : a.block_size;
  const dim3 grid((static_cast<uint32_t>(a.n_tokens) + window - 1) / window, a.n_kv_heads, 2);
  switch (a.block_size) {
    case 16: return launch_early(kv_append_kernel<T, D, 2>, grid, dim3(kAppendThreads), 0, stream, a, window);
    case 32: return launch_early(kv_append_kernel<T, D, 4>, grid, dim3(kAppendThreads), 0, stream, a, window);
    case 64: return launch_early(kv_append_kernel<T, D, 8>, grid, dim3(kAppendThreads), 0, stream, a, window);
    default: return launch_early(kv_append_kernel<T, D, 16>, grid, dim3(kAppendThreads), 0, stream, a, window);
  }
}

template <class T>
cudaError_t append_typed(const moe_kv_append_args& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 64: return append_dim<T, 64>(a, stream);
    case 128: return append_dim<T, 128>(a, stream);
    default: return append_dim<T, 256>(a, stream);
  }
}

}  // namespace

cudaError_t launch_kv_assign(const moe_kv_assign_args& a, cudaStream_t stream) {
  const size_t smem = sizeof(int32_t) * (3 * static_cast<size_t>(a.n_requests) + 2);
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kv_assign_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(sizeof(int32_t) * (3 * kAssignMaxRequests + 2)));
    if (e != cudaSuccess) return e;
  }
  const int64_t pieces = static_cast<int64_t>(a.n_requests) * ((a.max_blocks + kAssignPiece - 1) / kAssignPiece);
  const int64_t toks = (static_cast<int64_t>(a.max_tokens) + kAssignThreads - 1) / kAssignThreads;
  const int64_t rows = (pieces + kAssignWarps - 1) / kAssignWarps;
  const int grid = static_cast<int>(std::min<int64_t>(2 * 152, std::max<int64_t>({1, rows, toks})));
  return launch_early(kv_assign_kernel, dim3(grid), dim3(kAssignThreads), smem, stream, a);
}

cudaError_t launch_kv_append(const moe_kv_append_args& a, cudaStream_t stream) {
  return a.dtype == MOE_ATTN_BF16 ? append_typed<Bf16>(a, stream) : append_typed<F16>(a, stream);
}

}  // namespace moe

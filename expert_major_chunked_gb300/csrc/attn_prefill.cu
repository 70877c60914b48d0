// Causal attention over packed prompts with grouped heads.
//
// One pass over the keys of a tile of rows with the running maximum and sum of the softmax:
//   s = scale * q . k,  m' = max(m, max_j s_j),  l' = l 2^(m - m') + sum_j 2^(s_j - m'),
//   o' = o 2^(m - m') + sum_j 2^(s_j - m') v_j
// (in base 2, scale times log2 e), out = o / l. The rows of a tile are the query heads of one kv head for consecutive
// tokens (row = token * heads + head), so a tile reads its keys and values once for the whole group.
//
// What bounds it, head_dim 128 in bf16, one call after another:
//   - long sequences, the two products: 16022 tokens, 16 heads on 2: 607 us, 1.73 PFLOP/s, 90% of a library product's
//     burst rate (the power limit holds the clock in a run of such calls). The last 2048 of as many tokens, 16 heads on
//     4: 168 us; 128 tiles on 152 SMs, and a step of 128 keys takes 2325 cycles of which 2048 are the products.
//   - short sequences, the ends of tiles: 13 of them with 4099 tokens, 32 heads on 8, f16: 35 us, 2.4 TB/s; about 5 us until
//     the first scores are there, and 2500 cycles a tile (5200 with head_dim 256) to divide and write the outputs.
//   - a few tokens, the launch: 40 tokens 6.5 us. The launch is an early one (attn.h): it was 8.2 us without, 35 was 37.
#include "attn.h"
#include "attn.cuh"

#include <algorithm>

namespace moe {
namespace {

// Set when a wait inside the kernel gave up; read and cleared by moe_attn_check.
__device__ int g_attn_error;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void seq_bounds(const int32_t* cu, int b, int total, int& start, int& len) {
  start = min(max(cu[b], 0), total);
  len = max(min(max(cu[b + 1], 0), total) - start, 0);
}

// A CTA's flags in shared memory: abort is raised by a wait that gives up and ends the others; worked is when the CTA last
// got on with its work (another tile, and once in kNote steps of keys, of the search for a tile, or keys of a row
// done by loops, of a microsecond or less each). A tile may have millions of steps, and most roles wait for most of it, so
// how long a wait takes says nothing by itself.
struct Flags {
  uint64_t worked;
  int abort;
};
constexpr int kNote = 1024;
__device__ __forceinline__ void note_work(volatile Flags* f) { f->worked = ptx::globaltimer(); }

// A tile of work: `tokens` tokens of a sequence from tok0 on, for a slice of the query heads of a kv head.
struct TileAt {
  uint32_t index;  // of the CTA whose tile it is
  int valid, q0, q_len, k0, k_len, tok0, kvh, slice;
};

// The tiles of a call in the order in which they are dealt out. Up to 32 sequences: by the keys that a tile sees, most
// first (level = tile number + prefix in tiles), which leaves short tiles for the end; one lane holds one sequence. More
// sequences: from the last to the first, without sorting, which would cost each tile a pass over all of them for every
// step of the search. The (kv head, slice) units of a tile come one after the other. One warp, all lanes.
struct TileOrder {
  const moe_attn_prefill_args& a;
  volatile Flags* flags;
  int tokens, units, slices;
  int q0, q_len, k0, k_len, n_tiles, level0;  // this lane's sequence (up to 32 sequences)
  int total;                                   // tiles of all sequences

  __device__ TileOrder(const moe_attn_prefill_args& args, volatile Flags* flags_, int tokens_, int slices_)
      : a(args), flags(flags_), tokens(tokens_), units(args.n_kv_heads * slices_), slices(slices_) {
    const int lane = threadIdx.x & 31;
    total = 0;
    for (int b0 = 0; b0 < a.n_seqs; b0 += 32) {
      q0 = q_len = k0 = k_len = 0;
      if (b0 + lane < a.n_seqs) {
        seq_bounds(a.cu_q, b0 + lane, a.total_q, q0, q_len);
        if (a.n_seqs <= 32) seq_bounds(a.cu_k, lane, a.total_k, k0, k_len);
      }
      n_tiles = (q_len + tokens - 1) / tokens;
      total += __reduce_add_sync(~0u, n_tiles);
      if (lane == 0 && (b0 / 32) % kNote == kNote - 1) note_work(flags);
    }
    const int shift = k_len - q_len;
    level0 = shift >= 0 ? shift / tokens : -((-shift + tokens - 1) / tokens);
  }
  __device__ int count_from(int level) const {  // tiles of this level or a higher one
    return __reduce_add_sync(~0u, min(max(n_tiles + level0 - level, 0), n_tiles));
  }
  __device__ bool find(uint32_t index, TileAt& t) const {
    const int lane = threadIdx.x & 31, rank = static_cast<int>(index / static_cast<uint32_t>(units)),
              unit = static_cast<int>(index % static_cast<uint32_t>(units));
    if (rank >= total) return false;
    int src, tile;
    if (a.n_seqs <= 32) {
      // the highest level that has more than `rank` tiles from it on
      int lo = __reduce_min_sync(~0u, n_tiles ? level0 : 0x7FFFFFFF);
      int hi = __reduce_max_sync(~0u, n_tiles ? level0 + n_tiles - 1 : static_cast<int>(0x80000000));
      while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (count_from(mid) > rank) lo = mid; else hi = mid - 1;
      }
      const uint32_t has = __ballot_sync(~0u, lo >= level0 && lo < level0 + n_tiles);
      // the lane with this many such lanes below it
      const int nth = rank - count_from(lo + 1);
      const bool is_it = (has >> lane & 1u) && __popc(has & ((1u << lane) - 1u)) == nth;
      src = __ffs(__ballot_sync(~0u, is_it)) - 1;
      tile = lo - __shfl_sync(~0u, level0, src);
      t.q0 = __shfl_sync(~0u, q0, src), t.q_len = __shfl_sync(~0u, q_len, src);
      t.k0 = __shfl_sync(~0u, k0, src), t.k_len = __shfl_sync(~0u, k_len, src);
    } else {
      int left = total - 1 - rank, b0 = 0;
      for (;; b0 += 32) {
        if (b0 >= a.n_seqs) return false;  // (offsets that overlap may add up to anything)
        int s = 0, n = 0;
        if (b0 + lane < a.n_seqs) seq_bounds(a.cu_q, b0 + lane, a.total_q, s, n);
        const int nt = (n + tokens - 1) / tokens;
        int incl = nt;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int v = __shfl_up_sync(~0u, incl, d);
          if (lane >= d) incl += v;
        }
        const uint32_t past = __ballot_sync(~0u, incl > left);
        if (past) {
          src = __ffs(past) - 1;
          tile = left - __shfl_sync(~0u, incl - nt, src);
          t.q0 = __shfl_sync(~0u, s, src), t.q_len = __shfl_sync(~0u, n, src);
          seq_bounds(a.cu_k, b0 + src, a.total_k, t.k0, t.k_len);
          break;
        }
        left -= __shfl_sync(~0u, incl, 31);
        if (lane == 0 && (b0 / 32) % kNote == kNote - 1) note_work(flags);
      }
    }
    t.index = index;
    t.valid = 1;
    t.kvh = unit / slices;
    t.slice = unit % slices;
    t.tok0 = tile * tokens;
    return true;
  }
};

// ------------------------------------------------------------------ rows whose product is not finite
// A hidden value that is NaN or infinite, in the last tiles of keys that a tile of rows reads, meets a probability of
// zero there and makes the row's product NaN. Such rows are noted, and computed again when the CTA is done with its tiles:
// that function called between the tiles costs the kernel registers, and spills in every step (3001 tokens 59.5 us
// against 53.5), whether or not there are such rows.
struct BadRows {
  uint32_t index, rows;  // of the tile; a bit for each of the warp's 32 rows
};
// A warp's list has room for the tiles that are under way when the CTA stops to take further ones (those that have not
// started then start as CTAs of their own).
constexpr int kBadRoom = 8, kBadStop = kBadRoom - 2;

// A warp's 32 rows: row0 .. of the 128 of a sub-tile; row r is token first_tok + r / hpt and head head0 + r % hpt, for
// n_tok tokens and `heads` heads.
struct RowsAt {
  int q0, k0, shift, head0, kvh, first_tok, n_tok, hpt, heads, row0;
};

// The first and the last of the keys `from` .. `to` - 1 whose value has a NaN or an infinity (2^31 - 1, -1: none). One warp;
// with `any`, it stops at the first ones that it meets.
template <class T, int D>
__device__ int2 unfinite_keys(const uint16_t* v, int64_t v_token, int from, int to, bool any, volatile Flags* flags) {
  constexpr int CHUNKS = D / 8, KEYS = 32 / CHUNKS, AHEAD = 8;  // 16 bytes a lane, KEYS keys a pass
  constexpr uint32_t E = T::kCode == 0 ? 0x7F80u : 0x7C00u;     // the exponent's bits
  const int lane = threadIdx.x & 31;
  int2 at = make_int2(0x7FFFFFFF, -1);
  for (int j = from; j < to; j += KEYS * AHEAD) {
    uint4 x[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int key = j + i * KEYS + lane / CHUNKS;
      x[i] = key < to ? *reinterpret_cast<const uint4*>(v + key * v_token + lane % CHUNKS * 8) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      bool hit = false;
#pragma unroll
      for (int k = 0; k < 4; ++k) hit |= (w[k] & E) == E || (w[k] >> 16 & E) == E;
      const int key = j + i * KEYS + lane / CHUNKS;
      if (hit) at = make_int2(min(at.x, key), key);
    }
    if (any && __any_sync(~0u, at.y >= 0)) break;
    if (lane == 0 && (j - from) / (KEYS * AHEAD) % kNote == kNote - 1) note_work(flags);
  }
  return make_int2(__reduce_min_sync(~0u, at.x), __reduce_max_sync(~0u, at.y));
}

// 16 rows (r0 .. of the 128) again, those of `which` written: 16 keys at a time as warp-level matrix products as long as
// every row sees them, then key by key for the rows that see it. A pass makes up to 128 dims of the output (all 256 would
// take more registers than there are).
template <class T, int D>
__device__ __noinline__ void rows_again(const moe_attn_prefill_args& a, const RowsAt& at, int r0, uint32_t which,
                                        float c) {
  constexpr float top = T::kCode == 1 ? 15.0f : 0.0f;  // log2 of the largest weight
  constexpr int CH = D < 128 ? D : 128;
  const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const uint16_t* k = static_cast<const uint16_t*>(a.k) + at.k0 * a.k_token + at.kvh * a.k_head;
  const uint16_t* v = static_cast<const uint16_t*>(a.v) + at.k0 * a.v_token + at.kvh * a.v_head;
  const uint16_t* q[2];  // this lane's rows: r0 + g and r0 + g + 8
  int64_t tok[2];
  int head[2], lim[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = r0 + g + 8 * e, row_tok = r / at.hpt, row_head = r % at.hpt;
    const bool real = row_tok < at.n_tok && row_head < at.heads;
    tok[e] = at.q0 + at.first_tok + row_tok, head[e] = at.head0 + row_head;
    lim[e] = real ? at.first_tok + row_tok + at.shift : -1;
    q[e] = real ? static_cast<const uint16_t*>(a.q) + tok[e] * a.q_token + head[e] * a.q_head : nullptr;
  }
  const int all_see = at.first_tok + r0 / at.hpt + at.shift + 1;  // keys that every row sees: the first row's
  const int blocks = max(all_see, 0) / 16, last = __reduce_max_sync(~0u, max(lim[0], lim[1]));
  auto load = [](const uint16_t* p) { return p ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0); };

#pragma unroll 1
  for (int d0 = 0; d0 < D; d0 += CH) {
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    // Loads are 16 bytes a lane. Of 32 dims of Q and K a lane has 8 t4 .. + 7, four of them for each of two products (their
    // order does not matter as long as it is the same). Of 64 dims of V it has 8 g .. + 7, one for each of eight products: the
    // results are dims 16 t4 + i (o[..][i][0] and [2] for the second row) and 16 t4 + 8 + i ([1] and [3]).
    float o[CH / 64][8][4];
#pragma unroll
    for (int j = 0; j < CH / 64; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) o[j][i][0] = o[j][i][1] = o[j][i][2] = o[j][i][3] = 0.0f;
    auto scale_rows = [&](float f0, float f1) {
      l[0] *= f0, l[1] *= f1;
#pragma unroll
      for (int j = 0; j < CH / 64; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) o[j][i][0] *= f0, o[j][i][1] *= f0, o[j][i][2] *= f1, o[j][i][3] *= f1;
    };

    for (int b = 0; b < blocks; ++b) {
      const uint16_t* kb = k + static_cast<int64_t>(b * 16 + g) * a.k_token + 8 * t4;
      const uint16_t* vb = v + static_cast<int64_t>(b * 16 + 2 * t4) * a.v_token + d0 + 8 * g;
      float s[2][4] = {};
#pragma unroll 4
      for (int kk = 0; kk < D; kk += 32) {
        const uint4 q0 = load(q[0] ? q[0] + kk + 8 * t4 : nullptr), q1 = load(q[1] ? q[1] + kk + 8 * t4 : nullptr);
        const uint32_t a0[4] = {q0.x, q1.x, q0.y, q1.y}, a1[4] = {q0.z, q1.z, q0.w, q1.w};
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const uint4 kw = load(kb + 8 * n * a.k_token + kk);
          mma_16816<T>(s[n], a0, kw.x, kw.y);
          mma_16816<T>(s[n], a1, kw.z, kw.w);
        }
      }
      float f[2], ms[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = fmaxf(fmaxf(s[0][2 * e], s[0][2 * e + 1]), fmaxf(s[1][2 * e], s[1][2 * e + 1]));
        x = fmaxf(x, __shfl_xor_sync(~0u, x, 1));
        x = fmaxf(x, __shfl_xor_sync(~0u, x, 2)) * c;
        const float mn = x > m[e] ? x : m[e];
        ms[e] = mn == -INFINITY ? 0.0f : mn;
        f[e] = exp2_fast(m[e] - ms[e]);
        m[e] = mn;
      }
      if (__any_sync(~0u, f[0] != 1.0f || f[1] != 1.0f)) scale_rows(f[0], f[1]);
      uint32_t p[4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x = exp2_fast(fmaf(s[n][2 * e], c, top - ms[e])), y = exp2_fast(fmaf(s[n][2 * e + 1], c, top - ms[e]));
          l[e] += x + y;
          p[2 * n + e] = T::pack(x, y);
        }
#pragma unroll
      for (int j = 0; j < CH / 64; ++j) {
        const uint4 w0 = load(vb + 64 * j), w1 = load(vb + 64 * j + a.v_token);
        const uint4 w2 = load(vb + 64 * j + 8 * a.v_token), w3 = load(vb + 64 * j + 9 * a.v_token);
        const uint32_t x[4][4] = {{w0.x, w1.x, w2.x, w3.x}, {w0.y, w1.y, w2.y, w3.y}, {w0.z, w1.z, w2.z, w3.z},
                                  {w0.w, w1.w, w2.w, w3.w}};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t half = i & 1 ? 0x7632 : 0x5410, *w = x[i / 2];
          mma_16816<T>(o[j][i], p, __byte_perm(w[0], w[1], half), __byte_perm(w[2], w[3], half));
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(~0u, l[e], 1);
      l[e] += __shfl_xor_sync(~0u, l[e], 2);
    }
    for (int key = blocks * 16; key <= last; ++key) {
      const uint16_t *kr = k + key * a.k_token + 8 * t4, *vr = v + key * a.v_token + d0 + 16 * t4;
      float s[2] = {0.0f, 0.0f};
#pragma unroll 1
      for (int j = 0; j < D; j += 32) {
        const uint4 kw = load(kr + j);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint4 qw = load(q[e] ? q[e] + j + 8 * t4 : nullptr);
          const uint32_t x[4] = {qw.x, qw.y, qw.z, qw.w}, y[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 xf = T::unpack(x[i]), yf = T::unpack(y[i]);
            s[e] = fmaf(xf.x, yf.x, fmaf(xf.y, yf.y, s[e]));
          }
        }
      }
      float f[2], p[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s[e] += __shfl_xor_sync(~0u, s[e], 1);
        s[e] += __shfl_xor_sync(~0u, s[e], 2);
        const bool sees = key <= lim[e];
        const float x = s[e] * c, mn = sees && x > m[e] ? x : m[e], ms = mn == -INFINITY ? 0.0f : mn;
        f[e] = exp2_fast(m[e] - ms);
        p[e] = sees ? exp2_fast(x - ms + top) : 0.0f;
        m[e] = mn;
      }
      scale_rows(f[0], f[1]);
      l[0] += p[0], l[1] += p[1];
#pragma unroll
      for (int j = 0; j < CH / 64; ++j)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint4 vw = load(vr + 64 * j + 8 * half);
          const uint32_t w[4] = {vw.x, vw.y, vw.z, vw.w};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (key > lim[e]) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 x = T::unpack(w[i]);
              o[j][2 * i][2 * e + half] = fmaf(p[e], x.x, o[j][2 * i][2 * e + half]);
              o[j][2 * i + 1][2 * e + half] = fmaf(p[e], x.y, o[j][2 * i + 1][2 * e + half]);
            }
          }
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (!(which >> (g + 8 * e) & 1u)) continue;
      const float il = l[e] == 0.0f ? 0.0f : 1.0f / l[e];
      uint16_t* out = static_cast<uint16_t*>(a.out) + tok[e] * a.out_token + head[e] * a.out_head + d0 + 16 * t4;
#pragma unroll
      for (int j = 0; j < CH / 64; ++j)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = T::pack(o[j][2 * i][2 * e + half] * il, o[j][2 * i + 1][2 * e + half] * il);
          *reinterpret_cast<uint4*>(out + 64 * j + 8 * half) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      if (a.lse && t4 == 0 && d0 == 0)
        a.lse[static_cast<int64_t>(head[e]) * a.total_q + tok[e]] =
            l[e] == 0.0f ? -INFINITY : (m[e] - top + log2_fast(l[e])) * kLn2;
    }
  }
}

// Which of the rows of `which` (a bit a lane, whose row sees keys up to `lim` of v) are to be computed again; their product
// is not finite although their sum is. A row stays as it is where it sees a value that is not finite, unless its tiles of
// `keys` keys have a hidden one as well. (Where there is none at all the sums have overflowed: weights are up to 2^8 there,
// and up to 1 when the row is computed again.)
template <class T, int D>
__device__ __noinline__ uint32_t rows_to_mend(const uint16_t* v, int64_t v_token, int lim, int keys, uint32_t which,
                                              volatile Flags* flags) {
  const int lane = threadIdx.x & 31, all_see = min(max(__shfl_sync(~0u, lim, 0) + 1, 0), keys);
  const int2 late = unfinite_keys<T, D>(v, v_token, all_see, keys, false, flags);
  const bool mine = which >> lane & 1u, hidden = mine && late.y > lim, unclear = mine && !hidden && late.x > lim;
  bool again = hidden;
  if (__any_sync(~0u, unclear) && unfinite_keys<T, D>(v, v_token, 0, all_see, true, flags).y < 0) again |= unclear;
  return __ballot_sync(~0u, again);
}

// ------------------------------------------------------------------ tcgen05 tiles
// A CTA works on two sub-tiles of 128 rows (one for head_dim 256) against tiles of 128 keys. Scores S = Q K^T go to
// TMEM (128 columns a slot), a softmax warpgroup reads them with one row a thread, writes the probabilities over them as
// 16-bit values, and O += P V takes its left operand from there. While the tensor core multiplies for one slot, the
// softmax of the other slot runs. TMEM columns: S of slots 0 and 1 at 0 and 128, O of the sub-tiles from 256 on.
//
// Warps 0-3, 4-7: softmax of slots 0, 1 (head_dim 256: warps 0-3 for both slots in turn); 8: TMA loads of keys and
// values; 9: matrix instructions (and TMEM); 10: which tile comes next; 11: TMA loads of queries.
//
// The grid has a CTA for every tile; one an SM starts and then takes tiles over from those that have not started, longest
// first, so the next tile goes to the first CTA that is free (dealt out in turn: 600 us against 575 on 16022 tokens). Each
// role runs ahead as far as its buffers allow: the next tile's keys, queries and first scores are under way while the
// last rows of this one are written out.
constexpr int kTKeys = 128, kTRows = 128, kTThreads = 384;
// Steps before a tile's end at which the next one is asked for: late enough that it is not promised long before it can
// start (asked for at once: 63 us against 54 on 3001 tokens at head_dim 256), early enough for its first loads.
constexpr int kSoon = 2;
constexpr int64_t kWaitNs = 2000000000;  // a wait gives up when nothing of its CTA has advanced for this long
// A row keeps its reference maximum until a score passes it by more than 2^8: the sums and the 16-bit probabilities
// have the room, and o is multiplied (a pass over TMEM) only then. The choice is each row's own, so a row's bits do not
// depend on the rows beside it.
constexpr float kSlack = 8.0f;
// log2 of the weight at the reference maximum. f16 is normal from 2^-14 to 2^16: with 2^7 there, and 2^8 more while the
// reference lags, the largest weight is from 2^7 to 2^15 and a weight keeps its 11 bits down to 2^-21 of it (with 1 there,
// down to 2^-14 only). bf16 has float32's exponents, so its weights keep their bits wherever they lie.
template <class T>
constexpr float kTop = T::kCode == 1 ? 7.0f : 0.0f;

template <int D>
struct Tc {
  static constexpr int NQ = D <= 128 ? 2 : 1;         // sub-tiles
  static constexpr int DH = D < 128 ? D : 128;
  static constexpr int PARTS = D / DH;                 // ring stages of a tile of keys (by dims), or values (by keys)
  static constexpr int STAGE = kTKeys * DH * 2;
  static constexpr int STAGES = D == 64 ? 8 : 5;
  static constexpr int VKEYS = kTKeys / PARTS;         // keys of a stage of values
  static constexpr int READERS = 4 * NQ + 3;           // warps that read a tile's record
  static constexpr int QBYTES = NQ * kTRows * D * 2;
  static constexpr int SMEM = 1024 + QBYTES + STAGES * STAGE + 1056;
  static_assert(SMEM <= 232448, "shared memory per CTA");
};

struct TcParams {
  CUtensorMap q;     // (64, heads, rows, head_dim / 64), boxes of a sub-tile's heads and tokens
  CUtensorMap k, v;  // (64, rows, head_dim / 64, kv heads)
  moe_attn_prefill_args a;
  int32_t heads_per_tile, slices;
};

__device__ __forceinline__ bool wait_working(uint32_t bar, uint32_t parity, volatile Flags* f) {
  for (uint32_t it = 0;; ++it) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if ((it & 15u) == 15u) {
      const uint64_t since = f->worked;
      if (f->abort || static_cast<int64_t>(ptx::globaltimer() - since) > kWaitNs) return false;
    }
  }
}

__device__ __forceinline__ void raise_wait(volatile Flags* f, int site) {
  f->abort = 1;
  atomicCAS(&g_attn_error, 0, site);
}

// smem descriptor of a V tile [keys][64-wide blocks of dims]: the instruction's N (dims) is the dense dimension.
// Leading offset: from one block of 64 dims to the next; stride offset: from 8 keys to the next 8.
__device__ __forceinline__ uint64_t v_desc(uint32_t addr, uint32_t block_stride) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(block_stride >> 4) << 16 |
         static_cast<uint64_t>(1024u >> 4) << 32 | static_cast<uint64_t>(1u) << 46 | static_cast<uint64_t>(2u) << 61;
}

// kind::f16 with float32 results; both operands bf16 (1) or f16 (0); n_major: B's dense dimension is N
template <class T>
__device__ constexpr uint32_t tc_idesc(uint32_t n, bool n_major) {
  constexpr uint32_t f = T::kCode == 0 ? 1u : 0u;
  return (1u << 4) | (f << 7) | (f << 10) | (n_major ? 1u << 16 : 0u) | ((n >> 3) << 17) | ((kTRows >> 4) << 24);
}

// Asks for a CTA of this grid that has not started (it then never will); the answer (16 bytes) completes on bar.
__device__ __forceinline__ void take_over(uint32_t answer, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
               ::"r"(answer), "r"(bar)
               : "memory");
}
// Whether there was one, and its number.
__device__ __forceinline__ bool took_over(uint32_t answer, uint32_t& cta) {
  uint32_t yes, x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(yes), "=r"(x)
      : "r"(answer)
      : "memory");
  cta = x;
  return yes != 0;
}

// true for one lane of the (converged) warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
      ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One step of a transposition across lanes: a goes to the partner where this lane's bit is set, else b.
__device__ __forceinline__ void swap_piece(uint32_t& a, uint32_t& b, bool bit, int partner) {
  const uint32_t got = __shfl_xor_sync(~0u, bit ? a : b, partner);
  if (bit) a = got; else b = got;
}

// two float32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// NaNs give way, as in fmaxf
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ void write_record(volatile TileAt& r, const TileAt& t) {
  r.index = t.index, r.valid = t.valid, r.q0 = t.q0, r.q_len = t.q_len, r.k0 = t.k0, r.k_len = t.k_len;
  r.tok0 = t.tok0, r.kvh = t.kvh, r.slice = t.slice;
}

// The rows that a softmax warp has noted. 16022 tokens, 16 heads on 2 of 128, with a NaN behind the last: 3.4 ms a call
// against 0.54 without (4.6 with loads of 4 bytes a lane; row after row and key after key 138).
template <class T, int D>
__device__ void mend_rows(const TcParams& p, const volatile BadRows* list, int n, volatile Flags* flags) {
  constexpr int NQ = Tc<D>::NQ;
  const moe_attn_prefill_args& a = p.a;
  const int group = a.n_heads / a.n_kv_heads, hpt = p.heads_per_tile, sub_tokens = kTRows / hpt;
  const int warp = threadIdx.x >> 5, sub = NQ == 2 ? warp >> 2 : 0;
  if (n == 0) return;
  const TileOrder order(a, flags, NQ * sub_tokens, p.slices);
  for (int i = 0; i < n; ++i) {
    TileAt t{};
    if (!order.find(list[i].index, t)) return;
    const int first_tok = t.tok0 + sub * sub_tokens;
    const RowsAt at = {t.q0, t.k0, t.k_len - t.q_len, t.kvh * group + t.slice * hpt, t.kvh, first_tok,
                       max(0, min(sub_tokens, t.q_len - first_tok)), hpt, min(hpt, group - t.slice * hpt), (warp & 3) * 32};
    for (int half = 0; half < 2; ++half)
      if (const uint32_t rows = list[i].rows >> (16 * half) & 0xFFFFu)
        rows_again<T, D>(a, at, at.row0 + 16 * half, rows, a.scale * kLog2e);
  }
}

template <class T, int D>
__global__ void __launch_bounds__(kTThreads, 1) prefill_kernel(const __grid_constant__ TcParams p) {
  using C = Tc<D>;
  constexpr int NQ = C::NQ;
  const moe_attn_prefill_args& a = p.a;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  const uint32_t sq = base, ring = base + C::QBYTES, bars = ring + C::STAGES * C::STAGE;
  // barriers: full[STAGES], empty[STAGES], q_full, q_empty, s_full[2], p_ready[2][2], pv_done[2], rec_full[2],
  // rec_empty[2], drain, taken, soon
  const uint32_t full0 = bars, empty0 = bars + 8u * C::STAGES, q_full = empty0 + 8u * C::STAGES, q_empty = q_full + 8u,
                 s_full = q_empty + 8u, p_ready = s_full + 16u, pv_done = p_ready + 32u, rec_full = pv_done + 16u,
                 rec_empty = rec_full + 16u, drain = rec_empty + 16u, taken = drain + 8u, soon = taken + 8u;
  const uint32_t answer = bars + 448u;  // 16 bytes: the tile taken over from a CTA that has not started
  uint8_t* tail = smem_raw + (soon + 8u - raw);
  volatile Flags* flags = reinterpret_cast<volatile Flags*>(tail);
  volatile TileAt* records = reinterpret_cast<volatile TileAt*>(tail + sizeof(Flags));  // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail + sizeof(Flags) + 2 * sizeof(TileAt));
  static_assert(8 * (2 * C::STAGES + 17) + sizeof(Flags) + 2 * sizeof(TileAt) + 4 <= 448, "barriers and records");
  volatile BadRows* bad_rows = reinterpret_cast<volatile BadRows*>(smem_raw + (bars + 512u - raw));  // [8][kBadRoom]
  volatile int* n_bad = reinterpret_cast<volatile int*>(bad_rows + 8 * kBadRoom);                    // [8]
  static_assert(512 + 8 * kBadRoom * sizeof(BadRows) + 8 * sizeof(int) <= 1056, "lists of rows");
  const int warp = __shfl_sync(~0u, static_cast<int>(threadIdx.x) >> 5, 0), lane = static_cast<int>(threadIdx.x) & 31;
  const int group = a.n_heads / a.n_kv_heads, hpt = p.heads_per_tile, sub_tokens = kTRows / hpt;

  if (warp == 10) {  // the first tile's record, beside the set-up below
    wait_for_previous();
    const TileOrder order(a, flags, NQ * sub_tokens, p.slices);
    TileAt t{};
    order.find(blockIdx.x, t);
    if (lane == 0) write_record(records[0], t);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      ptx::mbar_init(full0 + 8u * s, 1);
      ptx::mbar_init(empty0 + 8u * s, 1);
    }
    ptx::mbar_init(q_full, 1);
    ptx::mbar_init(q_empty, 1);
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(s_full + 8u * s, 1);
      ptx::mbar_init(p_ready + 16u * s, 4);
      ptx::mbar_init(p_ready + 16u * s + 8u, 4);
      ptx::mbar_init(pv_done + 8u * s, 1);
      ptx::mbar_init(rec_full + 8u * s, 1);
      ptx::mbar_init(rec_empty + 8u * s, C::READERS);
    }
    ptx::mbar_init(drain, 1);
    ptx::mbar_init(taken, 1);
    ptx::mbar_init(soon, 1);
    flags->abort = 0;
    for (int w = 0; w < 8; ++w) n_bad[w] = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 8 && lane == 0 && a.total_k > 0) {  // (without keys there are no such maps)
    ptx::tma_prefetch_desc(&p.k);
    ptx::tma_prefetch_desc(&p.v);
  }
  if (warp == 11 && lane == 0) ptx::tma_prefetch_desc(&p.q);
  wait_for_previous();  // nothing above reads what the stream's earlier work writes
  if (warp == 9) {      // (after the wait: a CTA of that work that has yet to ask for its TMEM comes first)
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
    if (lane == 0) note_work(flags);  // (all that the CTA has waited for so far was other work)
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);

  // A tile's record, and what follows from it: tokens of each sub-tile, tiles of keys that any of its rows sees.
  struct Tile {
    TileAt at;
    int n_tok[NQ], n_keys[NQ], most;
  };
  auto read_tile = [&](int it, Tile& t) {  // false: no more tiles (or a wait gave up)
    if (!wait_working(rec_full + 8u * (it & 1), (it >> 1) & 1, flags)) {
      raise_wait(flags, 4);
      return false;
    }
    const volatile TileAt& r = records[it & 1];
    t.at.index = r.index, t.at.valid = r.valid, t.at.q0 = r.q0, t.at.q_len = r.q_len, t.at.k0 = r.k0, t.at.k_len = r.k_len;
    t.at.tok0 = r.tok0, t.at.kvh = r.kvh, t.at.slice = r.slice;
    t.most = 0;
#pragma unroll
    for (int s = 0; s < NQ; ++s) {
      t.n_tok[s] = max(0, min(sub_tokens, t.at.q_len - t.at.tok0 - s * sub_tokens));
      const int seen = t.at.tok0 + s * sub_tokens + t.n_tok[s] + t.at.k_len - t.at.q_len;
      const int keys = t.n_tok[s] ? min(max(seen, 0), t.at.k_len) : 0;
      t.n_keys[s] = (keys + kTKeys - 1) / kTKeys;
      t.most = max(t.most, t.n_keys[s]);
    }
    return t.at.valid != 0;
  };
  auto done_reading = [&](int it) { ptx::mbar_arrive(rec_empty + 8u * (it & 1)); };

  // 384 threads x 168 registers = 256 x 200 + 128 x 104: a softmax thread holds a row of 128 scores. (Nothing moved: the
  // softmax spilled; 208 and 88: the issuing warp spilled, 6% slower on a chunk of 2048 tokens over 16022 keys.)
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 8) {
      // ------------------------------------------------------------ keys and values, in the order in which they are used
      if (lane == 0) {
        uint32_t issued = 0;
        bool failed = false;
        Tile t;
        for (int it = 0; !failed && read_tile(it, t); ++it) {
          done_reading(it);
          auto load = [&](bool is_v, int tile) {
#pragma unroll
            for (int part = 0; part < C::PARTS; ++part) {
              const uint32_t stage = issued % C::STAGES, use = issued / C::STAGES;
              if (failed || !wait_working(empty0 + 8u * stage, (use & 1u) ^ 1u, flags)) {
                if (!failed) raise_wait(flags, 1);
                failed = true;
                return;
              }
              const uint32_t bar = full0 + 8u * stage, dst = ring + stage * C::STAGE;
              ptx::mbar_arrive_expect_tx(bar, C::STAGE);
              if (is_v)
                ptx::tma_load_4d(dst, &p.v, 0, t.at.k0 + tile * kTKeys + part * C::VKEYS, 0, a.v_head ? t.at.kvh : 0, bar);
              else
                ptx::tma_load_4d(dst, &p.k, 0, t.at.k0 + tile * kTKeys, part * (C::DH / 64), a.k_head ? t.at.kvh : 0, bar);
              ++issued;
            }
          };
          if (t.most > 0) load(false, 0);
          if (NQ == 1 && t.most > 1) load(false, 1);
          for (int j = 0; j < t.most && !failed; ++j) {
            load(true, j);
            if (j + 3 - NQ < t.most) load(false, j + 3 - NQ);
          }
        }
        // no copy may land in a CTA that has left, nor a release arrive there
        int no_abort = 0;
        for (uint32_t s = 0; s < C::STAGES; ++s) {
          const uint32_t n = issued / C::STAGES + (s < issued % C::STAGES ? 1u : 0u);
          if (n) ptx::wait_bounded(full0 + 8u * s, (n - 1u) & 1u, kWaitNs, &no_abort);
          if (n && !failed) wait_working(empty0 + 8u * s, (n - 1u) & 1u, flags);
        }
      }
      __syncwarp();
    } else if (warp == 11) {
      // ------------------------------------------------------------ queries
      if (lane == 0) {
        uint32_t n = 0;  // tiles whose queries were loaded
        bool failed = false;
        Tile t;
        for (int it = 0; read_tile(it, t); ++it) {
          done_reading(it);
          if (t.most == 0) continue;
          if (!wait_working(q_empty, (n & 1u) ^ 1u, flags)) {
            raise_wait(flags, 5);
            failed = true;
            break;
          }
          ptx::mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(hpt * sub_tokens * 2 * D * NQ));
          for (int s = 0; s < NQ; ++s)
            for (int i = 0; i < D / 64; ++i)  // row = token * hpt + head; rows of other heads or sequences are not used
              ptx::tma_load_4d(sq + s * (kTRows * D * 2) + i * (kTRows * 128), &p.q, 0,
                               t.at.kvh * group + t.at.slice * hpt, t.at.q0 + t.at.tok0 + s * sub_tokens, i, q_full);
          ++n;
        }
        int no_abort = 0;
        if (n) ptx::wait_bounded(q_full, (n - 1u) & 1u, kWaitNs, &no_abort);
        if (n && !failed) wait_working(q_empty, (n - 1u) & 1u, flags);
      }
      __syncwarp();
    } else if (warp == 10) {
      // ------------------------------------------------------------ which tile comes next
      // The grid has a CTA for every tile, longest first. One CTA an SM starts; when it is ready for another tile it takes
      // one over from a CTA that has not started, so the next tile always goes to the first CTA that is free.
      const TileOrder order(a, flags, NQ * sub_tokens, p.slices);
      if (lane == 0) ptx::mbar_arrive(rec_full);
      uint32_t asked = 0, index = 0;
      bool more = true;     // there may be CTAs that have not started
      auto ask = [&]() {    // false: a wait gave up
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(taken, 16);
          take_over(answer, taken);
        }
        __syncwarp();
        if (!__all_sync(~0u, wait_working(taken, asked++ & 1u, flags))) return false;
        more = took_over(answer, index);
        if (lane == 0) note_work(flags);
        ptx::fence_proxy_async_smem();  // the answer's place may be written again
        __syncwarp();
        return true;
      };
      bool have = records[0].valid != 0, ok = true;
      for (int it = 1; have; ++it) {
        ok = __all_sync(~0u, wait_working(rec_empty + 8u * (it & 1), ((it >> 1) & 1) ^ 1, flags));
        // (the lists are those of tiles up to it - 3: it - 2, it - 1 and this one may add to them)
        if (__any_sync(~0u, n_bad[lane & 7] >= kBadStop))
          more = false;
        else
          ok = ok && __all_sync(~0u, wait_working(soon, (it - 1) & 1, flags)) && ask();
        if (!ok) {
          if (lane == 0) raise_wait(flags, 6);
          break;
        }
        TileAt t{};
        have = more && order.find(index, t);
        if (lane == 0) {
          write_record(records[it & 1], t);
          ptx::mbar_arrive(rec_full + 8u * (it & 1));
        }
      }
      while (ok && more) ok = ask();  // the grid is an upper bound: CTAs without a tile need not start
      __syncwarp();
    } else if (warp == 9) {
      // ------------------------------------------------------------ matrix instructions
      // All lanes run the loops, so that their state and the descriptors stay in uniform registers; one lane issues. With
      // the loops in one lane the issue was the bound: 207 us against 164 on a chunk of 2048 tokens over 16022 keys.
      {
        const bool leader = elect_one();
        constexpr uint32_t idesc_s = tc_idesc<T>(kTKeys, false), idesc_o = tc_idesc<T>(D, true);
        // An instruction takes 64 tensor cycles, so the descriptors are constants added to a stage's base.
        const uint64_t q_desc = ptx::sw128_kmajor_desc(sq), k_desc = ptx::sw128_kmajor_desc(ring),
                       v_base = v_desc(ring, C::VKEYS * 128);
        bool failed = false;
        auto wait = [&](uint32_t bar, uint32_t parity) {
          if (failed) return false;
          if (!__all_sync(~0u, wait_working(bar, parity, flags))) {
            raise_wait(flags, 2);
            failed = true;
          }
          return !failed;
        };
        uint32_t stage = 0, phase = 0;      // the next stage to take
        struct Taken { uint32_t at[C::PARTS]; };
        auto take = [&](Taken& t) {  // the PARTS stages of a tile, once they have arrived
#pragma unroll
          for (int i = 0; i < C::PARTS; ++i) {
            if (!wait(full0 + 8u * stage, phase)) return false;
            t.at[i] = stage;
            if (++stage == C::STAGES) stage = 0, phase ^= 1u;
          }
          ptx::tc_fence_after();
          return true;
        };
        auto release = [&](const Taken& t) {
#pragma unroll
          for (int i = 0; i < C::PARTS; ++i)
            if (leader) ptx::umma_commit(empty0 + 8u * t.at[i]);
        };
        auto scores = [&](int sub, int slot, const Taken& t) {
          const uint64_t qd = q_desc + static_cast<uint32_t>(sub * (kTRows * D * 2 / 16));
          const uint32_t d = tmem + 128u * slot;
#pragma unroll
          for (int i = 0; i < C::PARTS; ++i) {
            const uint64_t kd = k_desc + t.at[i] * static_cast<uint32_t>(C::STAGE / 16);
#pragma unroll
            for (int in = 0; in < C::DH / 16; ++in) {  // a stage: up to 8 steps of 16 dims, 4 to a 128-byte row
              const int kk = i * (C::DH / 16) + in;
              if (leader) ptx::umma_bf16(d, qd + ((kk / 4) * (kTRows * 128) + (kk % 4) * 32) / 16,
                             kd + ((in / 4) * (kTKeys * 128) + (in % 4) * 32) / 16, idesc_s, kk ? 1u : 0u);
            }
          }
          if (leader) ptx::umma_commit(s_full + 8u * slot);
        };
        auto values = [&](int sub, int slot, const Taken& t, bool accumulate, uint32_t parity) {
          const uint32_t d = tmem + 256u + sub * D, pr = tmem + 128u * slot;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (!wait(p_ready + 16u * slot + 8u * half, parity)) return;
            ptx::tc_fence_after();
#pragma unroll
            for (int kk = half * 4; kk < half * 4 + 4; ++kk) {
              const int i = kk / (C::VKEYS / 16), in = kk % (C::VKEYS / 16);
              const uint64_t vd = v_base + t.at[i] * static_cast<uint32_t>(C::STAGE / 16);
              if (leader) umma_ts(d, pr + 8u * kk, vd + in * (2048 / 16), idesc_o, (accumulate || kk) ? 1u : 0u);
            }
          }
          if (leader) ptx::umma_commit(pv_done + 8u * sub);
        };
        bool any = false;
        uint32_t tiles = 0, steps[NQ] = {};  // tiles that had keys; steps of each sub-tile so far
        Tile t;
        for (int it = 0; !failed; ++it) {
          const bool have = read_tile(it, t);
          if (!__all_sync(~0u, have)) break;
          if (leader) done_reading(it);
          t.most = __shfl_sync(~0u, t.most, 0);
#pragma unroll
          for (int s = 0; s < NQ; ++s) t.n_keys[s] = __shfl_sync(~0u, t.n_keys[s], 0);
          if (leader && t.most <= kSoon) ptx::mbar_arrive(soon);
          if (t.most == 0) continue;
          if (!wait(q_full, tiles & 1u)) break;
          Taken kt, vt, kn;
          any = true;
          if constexpr (NQ == 2) {
            if (!take(kt)) break;
            for (int s = 0; s < 2; ++s)
              if (t.n_keys[s] > 0) scores(s, s, kt);
            release(kt);
            if (t.most == 1 && leader) ptx::umma_commit(q_empty);
            for (int j = 0; j < t.most && !failed; ++j) {
              if (leader && j % kNote == kNote - 1) note_work(flags);
              if (leader && j + kSoon + 1 == t.most) ptx::mbar_arrive(soon);
              if (!take(vt)) break;
              bool have_k = false;
#pragma unroll
              for (int s = 0; s < 2; ++s) {
                if (j < t.n_keys[s]) {
                  values(s, s, vt, j > 0, (steps[s] + j) & 1u);
                  if (failed) break;
                }
                if (s == 1) release(vt);
                if (j + 1 < t.n_keys[s]) {
                  if (!have_k && !take(kn)) break;
                  have_k = true;
                  scores(s, s, kn);
                }
              }
              if (failed) break;
              if (have_k) release(kn);
              if (j + 2 == t.most && leader) ptx::umma_commit(q_empty);  // the tile's last scores
            }
            steps[0] += t.n_keys[0];
            steps[NQ - 1] += t.n_keys[NQ - 1];
          } else {
            const uint32_t g = steps[0];
            for (int j = 0; j < min(t.most, 2) && !failed; ++j) {
              if (!take(kt)) break;
              scores(0, (g + j) & 1, kt);
              release(kt);
            }
            if (t.most <= 2 && leader) ptx::umma_commit(q_empty);
            for (int j = 0; j < t.most && !failed; ++j) {
              if (leader && j % kNote == kNote - 1) note_work(flags);
              if (leader && j + kSoon + 1 == t.most) ptx::mbar_arrive(soon);
              const int slot = (g + j) & 1;
              if (!take(vt)) break;
              values(0, slot, vt, j > 0, ((g + j) >> 1) & 1u);
              if (failed) break;
              release(vt);
              if (j + 2 < t.most) {
                if (!take(kn)) break;
                scores(0, slot, kn);
                release(kn);
                if (j + 3 == t.most && leader) ptx::umma_commit(q_empty);
              }
            }
            steps[0] += t.most;
          }
          ++tiles;
        }
        if (failed && any) {
          int no_abort = 0;
          if (leader) ptx::umma_commit(drain);
          ptx::wait_bounded(drain, 0u, kWaitNs, &no_abort);
        }
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    if (NQ == 2 || warp < 4) {
      // ------------------------------------------------------------ softmax: a row a thread
      const int sub = NQ == 2 ? warp >> 2 : 0;
      const int row = (warp & 3) * 32 + lane, row_tok = row / hpt, row_head = row % hpt;
      const float c = a.scale * kLog2e;
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t o_at = tmem + 256u + sub * D + lanes;
      uint32_t steps = 0;  // tiles of keys so far: the phases of s_full, p_ready and pv_done
      bool ok = true;
      Tile t;
      for (int it = 0; ok; ++it) {
        const bool have = read_tile(it, t);
        __syncwarp();
        if (!__all_sync(~0u, have)) break;
        if (lane == 0) done_reading(it);
        const int nt = sub == 0 ? t.n_keys[0] : t.n_keys[NQ - 1], ntk = sub == 0 ? t.n_tok[0] : t.n_tok[NQ - 1];
        const int gs = min(hpt, group - t.at.slice * hpt), shift = t.at.k_len - t.at.q_len;
        const int first_tok = t.at.tok0 + sub * sub_tokens, tok = first_tok + row_tok;  // in the sequence
        const bool real = row_tok < ntk && row_head < gs;
        // the last key that this row sees, and the warp's first row (rows that are not real may see anything)
        const int lim = tok + shift, lim_lo = __shfl_sync(~0u, lim, 0);
        const int h = t.at.kvh * group + t.at.slice * hpt + row_head;
        float m = -INFINITY, l = 0.0f;
        for (int j = 0; j < nt; ++j) {
          const int slot = NQ == 2 ? sub : (steps + j) & 1;
          const uint32_t s_at = tmem + 128u * slot + lanes;
          ok = wait_working(s_full + 8u * slot, (NQ == 2 ? steps + j : (steps + j) >> 1) & 1u, flags);
          ok = __all_sync(~0u, ok);
          if (!ok) break;
          ptx::tc_fence_after();
          uint32_t s[4][32];
#pragma unroll
          for (int i = 0; i < 4; ++i) ptx::tmem_ld32(s_at + 32u * i, s[i]);
          ptx::tmem_ld_wait();
          if (const int rel = lim - j * kTKeys; j * kTKeys + kTKeys - 1 > lim_lo) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int n = min(max(rel - 32 * i + 1, 0), 32);
              const uint32_t keep = n == 32 ? ~0u : (1u << n) - 1u;
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!(keep & (1u << k))) s[i][k] = 0xFF800000u;
            }
          }
          float mx[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mx[i] = __uint_as_float(s[i][0]);
#pragma unroll
            for (int k = 1; k < 31; k += 2)
              mx[i] = max3(mx[i], __uint_as_float(s[i][k]), __uint_as_float(s[i][k + 1]));
            mx[i] = fmaxf(mx[i], __uint_as_float(s[i][31]));
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
          const bool grows = top > m + kSlack;  // also from -inf
          if (__any_sync(~0u, grows)) {
            const float mn = grows ? top : m;
            if (j > 0) {
              const float f = grows ? exp2_fast(m - mn) : 1.0f;
              ok = wait_working(pv_done + 8u * sub, (steps + j - 1u) & 1u, flags);
              ok = __all_sync(~0u, ok);
              if (!ok) break;
              ptx::tc_fence_after();
              l *= f;
#pragma unroll 1
              for (int i = 0; i < D; i += 32) {
                uint32_t o[32];
                ptx::tmem_ld32(o_at + i, o);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tmem_st32(o_at + i, o);
              }
            }
            m = mn;
          }
          const float u = m == -INFINITY ? 0.0f : m;
          const float2 c2 = make_float2(c, c), u2 = make_float2(kTop<T> - u, kTop<T> - u);
          float2 sum[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[i] = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t pk[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int e = q * 64 + 2 * i;
              float2 x = make_float2(__uint_as_float(s[e / 32][e % 32]), __uint_as_float(s[e / 32][e % 32 + 1]));
              x = fma2(x, c2, u2);
              x.x = exp2_fast(x.x);
              x.y = exp2_fast(x.y);
              sum[i & 3] = add2(sum[i & 3], x);
              pk[i] = T::pack(x.x, x.y);
            }
            tmem_st32(s_at + 32u * q, pk);
            tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(p_ready + 16u * slot + 8u * q);
          }
          const float2 t2 = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
          l += t2.x + t2.y;
        }
        steps += nt;
        // With one sub-tile the last scores were asked for before the last but one product with V, so that product may not be
        // done here. A barrier tells apart two phases only, so both have to be waited for, one after the other. (With two
        // sub-tiles each one's scores come after its product before.)
        if (NQ == 1 && ok && nt > 1) {
          ok = wait_working(pv_done, steps & 1u, flags);
          ok = __all_sync(~0u, ok);
        }
        if (ok && nt > 0) {
          ok = wait_working(pv_done + 8u * sub, (steps - 1u) & 1u, flags);
          ok = __all_sync(~0u, ok);
        }
        if (!ok) {
          if (lane == 0) raise_wait(flags, 3);
          break;
        }
        ptx::tc_fence_after();
        const float il = l == 0.0f ? 0.0f : 1.0f / l;  // (NaN from a score that the row sees makes all of it NaN)
        // A row a thread would store 16 bytes of 32 rows at a time: four neighbours exchange their 16-byte pieces first, and
        // then store 64 bytes of 8 rows. Offsets of the four rows, -1 for one that is not there:
        const int64_t own = real ? (t.at.q0 + tok) * a.out_token + h * a.out_head : -1;
        int64_t row_at[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) row_at[k] = __shfl_sync(~0u, own, (lane & ~3) + k);
        const bool odd1 = lane & 1, odd2 = lane & 2;
        float2 zero = make_float2(0.0f, 0.0f);  // stays 0 unless a value is not finite
#pragma unroll 1
        for (int i = 0; i < D; i += 32) {
          uint32_t o[32];
          if (nt > 0) {
            ptx::tmem_ld32(o_at + i, o);
            ptx::tmem_ld_wait();
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0;
          }
          uint32_t w[4][4];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 x = make_float2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1]));
            zero = fma2(x, make_float2(0.0f, 0.0f), zero);
            w[k / 4][k % 4] = T::pack(x.x * il, x.y * il);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // pieces 0|1 and 2|3 with lane ^ 1, then 0|2 and 1|3 with lane ^ 2
            swap_piece(w[0][k], w[1][k], odd1, 1);
            swap_piece(w[2][k], w[3][k], odd1, 1);
            swap_piece(w[0][k], w[2][k], odd2, 2);
            swap_piece(w[1][k], w[3][k], odd2, 2);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (row_at[k] >= 0)
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + row_at[k] + i + (lane & 3) * 8) =
                  make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
        }
        const bool bad = real && finite_bits(l) && !(zero.x == 0.0f && zero.y == 0.0f);
        ptx::tc_fence_before();
        if (real && a.lse)
          a.lse[static_cast<int64_t>(h) * a.total_q + t.at.q0 + tok] =
              l == 0.0f ? -INFINITY : (m - kTop<T> + log2_fast(l)) * kLn2;
        if (const uint32_t which = __ballot_sync(~0u, bad)) {
          const uint16_t* v = static_cast<const uint16_t*>(a.v) + t.at.k0 * a.v_token + t.at.kvh * a.v_head;
          const uint32_t rows = rows_to_mend<T, D>(v, a.v_token, lim, min(nt * kTKeys, a.total_k - t.at.k0), which, flags);
          if (rows && lane == 0) {
            const int n = n_bad[warp];
            bad_rows[warp * kBadRoom + n].index = t.at.index;
            bad_rows[warp * kBadRoom + n].rows = rows;
            n_bad[warp] = n + 1;
          }
        }
      }
      __syncwarp();
      mend_rows<T, D>(p, bad_rows + warp * kBadRoom, n_bad[warp], flags);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// Keys or values as (64, rows, head_dim / 64, kv heads), boxes of box_rows rows of box_blocks blocks of 64 dims: a box
// lands as [box_blocks][box_rows][128 B], swizzled. A dimension that is not walked (one row, one head, or a head
// stride of 0, where the kernel stays at head 0) gets an arbitrary valid stride.
bool encode_rows(CUtensorMap* m, const void* p, int dtype, int dim, int rows, int heads, int64_t token, int64_t head,
                 int box_rows, int box_blocks) {
  const EncodeTiledFn fn = tensor_map_encoder();
  if (!fn) return false;
  if (head == 0) heads = 1;
  const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(dim / 64),
                              static_cast<cuuint64_t>(heads)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(rows > 1 ? token * 2 : dim * 2), 128,
                                 static_cast<cuuint64_t>(heads > 1 ? head * 2 : dim * 2)};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(box_blocks), 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn(m, dtype == MOE_ATTN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
            const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries as (64, heads, rows, head_dim / 64), boxes of `heads` heads of `tokens` tokens: a box lands as
// [tokens][heads][128 B], swizzled.
bool encode_queries(CUtensorMap* m, const moe_attn_prefill_args& a, int heads, int tokens) {
  const EncodeTiledFn fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(a.n_heads), static_cast<cuuint64_t>(a.total_q),
                              static_cast<cuuint64_t>(a.head_dim / 64)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(a.n_heads > 1 ? a.q_head * 2 : a.head_dim * 2),
                                 static_cast<cuuint64_t>(a.total_q > 1 ? a.q_token * 2 : a.head_dim * 2), 128};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(tokens), 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn(m, a.dtype == MOE_ATTN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
            const_cast<void*>(a.q), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T, int D>
cudaError_t launch_tiles(const moe_attn_prefill_args& a, cudaStream_t stream) {
  using C = Tc<D>;
  static OncePerDevice prepared;
  const cudaError_t e = prepared([] {
    return cudaFuncSetAttribute(prefill_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  });
  if (e != cudaSuccess) return e;
  TcParams p;
  p.a = a;
  const int group = a.n_heads / a.n_kv_heads;
  p.heads_per_tile = std::min(group, kTRows);
  p.slices = (group + p.heads_per_tile - 1) / p.heads_per_tile;
  const int sub_tokens = kTRows / p.heads_per_tile;
  bool encoded = encode_queries(&p.q, a, p.heads_per_tile, sub_tokens);
  if (a.total_k > 0) {
    encoded &= encode_rows(&p.k, a.k, a.dtype, D, a.total_k, a.n_kv_heads, a.k_token, a.k_head, kTKeys, C::DH / 64) &&
               encode_rows(&p.v, a.v, a.dtype, D, a.total_k, a.n_kv_heads, a.v_token, a.v_head, C::VKEYS, D / 64);
  } else {
    p.k = CUtensorMap{}, p.v = CUtensorMap{};  // no tile of keys is loaded
  }
  if (!encoded) return cudaErrorInvalidValue;
  // sequences begin new tiles, so there are at most total / tokens + n_seqs
  const int64_t tiles = (static_cast<int64_t>(a.total_q) / (C::NQ * sub_tokens) + a.n_seqs) * a.n_kv_heads * p.slices;
  return launch_early(prefill_kernel<T, D>, dim3(static_cast<unsigned>(tiles)), dim3(kTThreads), C::SMEM, stream, p);
}

}  // namespace

cudaError_t launch_attn_prefill(const moe_attn_prefill_args& a, cudaStream_t stream) {
  const bool b = a.dtype == MOE_ATTN_BF16;
  switch (a.head_dim) {
    case 64: return b ? launch_tiles<Bf16, 64>(a, stream) : launch_tiles<F16, 64>(a, stream);
    case 128: return b ? launch_tiles<Bf16, 128>(a, stream) : launch_tiles<F16, 128>(a, stream);
    default: return b ? launch_tiles<Bf16, 256>(a, stream) : launch_tiles<F16, 256>(a, stream);
  }
}

cudaError_t attn_prefill_take_error(int* site, cudaStream_t stream) {
  const int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(site, g_attn_error, sizeof(int), 0, cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e == cudaSuccess && *site) {
    e = cudaMemcpyToSymbolAsync(g_attn_error, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  }
  return e;
}

}  // namespace moe

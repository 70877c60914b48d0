// Decode attention: one query token a request over the 8-bit paged cache.
//
// With codes c_j, scales sk_j and sv_j (constant over a block) and u_j = scale * log2(e) * sk_j * (q . ck_j):
//   out = sum_j 2^u_j sv_j cv_j / sum_j 2^u_j
// The weights enter the second product as p_j = 2^(u_j + log2 sv_j - m + 15), m the running maximum of u_j + log2 sv_j:
// at most 2^15 whatever the scales are, so p fits f16, and e4m3 codes are exact in f16: both products run on the f16
// tensor path with float32 accumulators. f16 is normal down to 2^-14, so a weight keeps its 11 bits down to 2^-29 of the
// row's largest; with the largest at 1 a token of a block with a small scale beside a block with a large one lost bits
// (2^-14 of the largest weight, while its codes can be 2^17 times the other's). The denominator is sum_j p_j / sv_j, in
// float32 from p before its rounding.
//
// Work: the (request, kv head, slice of 16 query heads, tile of tokens) units of the whole call in one line, cut into as
// many equal ranges as there are CTAs, so that mixed lengths and few requests fill the machine alike. A (request, kv
// head) that lies in one range is finished there; the others leave (m, l, o) pieces that a second kernel joins in range
// order, always the same, so that the same call gives the same bytes.
//
// What bounds it: the bytes of the cache, 2 head_dim a token and kv head, each read once. 64 requests of up to 16384
// tokens, 32 query heads on 8 kv heads of 128: 1.1 GB in 174 us, 6.3 TB/s, 93% of a plain copy's rate. One request of
// 131072 tokens, 16 heads on 2 of 256 (134 MB): 30.4 us, of which about 8 us are the two launches, the first loads'
// latency and the join (20 us would be the bytes alone; two stages a warp and two CTAs an SM measured best, against 3 x 2,
// 2 x 3 and 2 x 4 and against CTAs of 8 warps). One request of 1500 tokens: 6.6 us on the GPU, two launches' latency; the
// host needs about 8 us to issue it. Both kernels are launched early (attn.h; 33.0 us without at 131072 tokens).
#include "attn.h"
#include "attn.cuh"

#include <algorithm>

namespace moe {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kTop = 15.0f;  // log2 of a row's largest weight
constexpr int kDecWarps = 4, kDecThreads = kDecWarps * 32, kDecStages = 2, kDecCtas = 2 * 152;
constexpr int kRows = 16;           // query heads of a tile (the matrix instruction's rows)
constexpr int kCodeBytes = 4096;    // codes of K (and of V) in a warp's stage
constexpr int kStageBytes = 2 * kCodeBytes;
template <int D>
constexpr int kTok = kCodeBytes / D;  // tokens of a stage: 64, 32, 16

struct DecodeGeom {
  int group, slices, rows;  // query heads a kv head, slices of them, heads of a slice
  int units_per_tile;       // n_kv_heads * slices
};
__host__ __device__ inline DecodeGeom decode_geom(int n_heads, int n_kv_heads) {
  DecodeGeom g;
  g.group = n_heads / n_kv_heads;
  g.slices = (g.group + kRows - 1) / kRows;
  g.rows = (g.group + g.slices - 1) / g.slices;
  g.units_per_tile = n_kv_heads * g.slices;
  return g;
}

// workspace: pieces [kDecCtas][2] of (m[16], l[16], o[16][D]), then (first, last) CTA of every (request, kv head, slice)
__host__ __device__ inline size_t piece_floats(int D) { return 2 * kRows + static_cast<size_t>(kRows) * D; }

__device__ __forceinline__ int request_len(const moe_attn_decode_args& a, int b) {
  const long long cap = static_cast<long long>(a.max_blocks) * a.block_size;
  return static_cast<int>(min(static_cast<long long>(max(a.kv_lens[b], 0)), cap));
}
// len / n rounded up; a length may be 2^31 - 1, so the sum is taken without a sign
__device__ __forceinline__ int parts_of(int len, int n) {
  return static_cast<int>((static_cast<uint32_t>(len) + static_cast<uint32_t>(n - 1)) / static_cast<uint32_t>(n));
}

// the first unit of range i of `ranges` (a 64-bit division takes several hundred cycles; few calls need one)
__device__ __forceinline__ long long first_unit(long long total, long long ranges, uint32_t i) {
  if (total < (1ll << 32) / (kDecCtas + 1))
    return static_cast<uint32_t>(total) * i / static_cast<uint32_t>(ranges);
  return total * i / ranges;
}

// byte offset of 16-byte chunk c of row r of a tile of codes: the chunks of a 128-byte line are exchanged so that eight
// consecutive rows of one chunk fall into different banks
template <int D>
__device__ __forceinline__ uint32_t code_at(int r, int c) {
  if constexpr (D == 64) return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  return static_cast<uint32_t>(r * D + ((c ^ (r & 7)) << 4));
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void zero16(uint32_t dst) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0) : "memory");
}

// an 8 x 8 matrix of 16-bit values, two of a row a lane, transposed across the warp
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Both products have the cache as their 16-row operand and 8 query heads (NH times) as columns: S^T = K Q^T and
// O^T = V^T P^T, so a group of up to 8 heads wastes no row. K's 4 consecutive bytes a lane give the operand's columns
// 2t, 2t+1, 2t+8, 2t+9 (the queries are taken in the same order); the transposed load of V gives a lane two tokens of
// two dims, which split into an operand whose rows 0..7 are the even dims and 8..15 the odd ones.
template <class T, int D, int NH>
__global__ void __launch_bounds__(kDecThreads, 2) decode_kernel(const __grid_constant__ moe_attn_decode_args a,
                                                                int block_log2) {
  constexpr int TOK = kTok<D>, TT = TOK / 16, CT = TOK * kDecWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) uint16_t q_sh[8 * NH * (D + 8)];
  __shared__ float q_mul[8 * NH];
  __shared__ float m_sh[kDecWarps][8 * NH], l_sh[kDecWarps][8 * NH];
  __shared__ __align__(16) float scale_sh[kDecWarps][kDecStages][8];
  __shared__ long long warp_sum[kDecWarps];
  __shared__ int start_b;
  __shared__ long long start_base;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const DecodeGeom geo = decode_geom(a.n_heads, a.n_kv_heads);
  wait_for_previous();
  // this CTA's range of units, and the request that it begins in
  const int per = (a.n_requests + kDecThreads - 1) / kDecThreads;
  const int b_lo = min(a.n_requests, tid * per), b_hi = min(a.n_requests, b_lo + per);
  auto tiles_of = [&](int b) { return parts_of(request_len(a, b), CT); };
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += tiles_of(b);
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long v = __shfl_up_sync(~0u, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  total *= geo.units_per_tile;
  // no more ranges than units: every range has a unit, so those that share a (request, kv head) are neighbours
  const long long ranges = min(static_cast<long long>(gridDim.x), total);
  if (blockIdx.x >= ranges) return;
  long long u = first_unit(total, ranges, blockIdx.x);
  const long long u_end = first_unit(total, ranges, blockIdx.x + 1);
  {
    long long base = before * geo.units_per_tile;
    for (int b = b_lo; b < b_hi; ++b) {
      const long long n = static_cast<long long>(tiles_of(b)) * geo.units_per_tile;
      if (u >= base && u < base + n) start_b = b, start_base = base;
      base += n;
    }
  }
  __syncthreads();
  int b = start_b;
  long long base = start_base;

  const uint32_t stage0 = ptx::smem_u32(smem) + warp * (kDecStages * kStageBytes);
  float* pieces = static_cast<float*>(a.workspace);
  int2* owners = reinterpret_cast<int2*>(pieces + piece_floats(D) * 2 * kDecCtas);
  const float sc = a.scale * kLog2e;
  const int g = lane >> 2, t4 = lane & 3;

  while (u < u_end) {
    const int len = request_len(a, b), nt = parts_of(len, CT);
    const long long n_units = static_cast<long long>(nt) * geo.units_per_tile;
    if (u >= base + n_units) {
      base += n_units;
      ++b;
      continue;
    }
    const long long in = u - base;
    const int hs = in >> 32 ? static_cast<int>(in / nt)
                            : static_cast<int>(static_cast<uint32_t>(in) / static_cast<uint32_t>(nt));
    const int first = static_cast<int>(in - static_cast<long long>(hs) * nt);
    const int tiles = static_cast<int>(min(static_cast<long long>(nt - first), u_end - u));
    const int kvh = hs / geo.slices, row0 = (hs % geo.slices) * geo.rows, rows = min(geo.rows, geo.group - row0);
    const int h0 = kvh * geo.group + row0;
    const int tok_end = static_cast<int>(min(static_cast<uint32_t>(len), static_cast<uint32_t>(first + tiles) * CT));
    const int32_t* table = a.block_table + b * a.table_stride;

    // the stage ring: a warp takes every fourth chunk of the segment
    int next_chunk = first * kDecWarps + warp, chunk = next_chunk, fill = 0, take = 0;
    const int chunk_end = parts_of(tok_end, TOK);
    auto block_of = [&](int c) {  // lanes below TT: the block of 16 tokens each
      const uint32_t tok = static_cast<uint32_t>(c) * TOK + lane * 16;  // (c may lie past the end)
      int id = -1;
      if (lane < TT && tok < static_cast<uint32_t>(tok_end)) {
        id = table[tok >> block_log2];
        if (id < 0 || id >= a.num_blocks) id = -1;
      }
      return id;
    };
    int blk = block_of(next_chunk);
    auto issue = [&]() {
      if (next_chunk < chunk_end) {
        constexpr int PER = D / 16, ROWS = 32 / PER, STEPS = 16 / ROWS;  // a step: 32 chunks of 16 bytes, ROWS rows
        const uint32_t dst = stage0 + fill * kStageBytes;
        const int tok0 = next_chunk * TOK, row = lane / PER, col = lane % PER;
#pragma unroll
        for (int i = 0; i < TT; ++i) {  // 16 tokens lie in one block, one after the other
          const int id = __shfl_sync(~0u, blk, i), left = id >= 0 ? tok_end - (tok0 + 16 * i) : 0;
          const int64_t at = ((static_cast<int64_t>(max(id, 0)) * a.n_kv_heads + kvh) << block_log2) +
                             ((tok0 + 16 * i) & (a.block_size - 1)) + row;
          const uint8_t* k = static_cast<const uint8_t*>(a.k_codes) + at * D + col * 16;
          const uint8_t* v = static_cast<const uint8_t*>(a.v_codes) + at * D + col * 16;
#pragma unroll
          for (int j = 0; j < STEPS; ++j) {
            const bool in = row + j * ROWS < left;
            const uint32_t to = dst + code_at<D>(16 * i + j * ROWS + row, col);
            cp_async16(to, in ? k + j * (ROWS * D) : a.k_codes, in ? 16 : 0);
            cp_async16(to + kCodeBytes, in ? v + j * (ROWS * D) : a.v_codes, in ? 16 : 0);
          }
        }
        if (lane < TT) {
          const uint32_t sc_at = ptx::smem_u32(&scale_sh[warp][fill][lane]);
          const int64_t off = blk >= 0 ? static_cast<int64_t>(blk) * a.n_kv_heads + kvh : 0;
          cp_async4(sc_at, a.k_scale + off, blk >= 0 ? 4 : 0);
          cp_async4(sc_at + 16, a.v_scale + off, blk >= 0 ? 4 : 0);
        }
        next_chunk += kDecWarps;
        blk = block_of(next_chunk);
        fill = fill + 1 == kDecStages ? 0 : fill + 1;
      }
      cp_async_commit();
    };
    // The queries' loads go out before the first codes are waited for. They become f16, each row scaled by a power of two
    // to below 2^15: f16 is normal from 2^-14 on, so a value keeps 11 bits down to 2^-28 of the row's largest (with the
    // largest below 2 an f16 query of 0.25 beside one of 60000 lost bits).
    constexpr int QR = 8 * NH / kDecWarps, W = D / 64;
    uint32_t qw[QR][W];
#pragma unroll
    for (int i = 0; i < QR; ++i) {
      const int r = warp + i * kDecWarps;
      const uint16_t* q = static_cast<const uint16_t*>(a.q) + b * a.q_token + (h0 + r) * a.q_head;
#pragma unroll
      for (int w = 0; w < W; ++w) qw[i][w] = r < rows ? *reinterpret_cast<const uint32_t*>(q + 2 * (lane + 32 * w)) : 0;
    }
#pragma unroll
    for (int i = 0; i < kDecStages - 1; ++i) issue();
#pragma unroll
    for (int i = 0; i < QR; ++i) {
      const int r = warp + i * kDecWarps;
      float2 x[W];
      float big = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        x[w] = T::unpack(qw[i][w]);
        if (finite_bits(x[w].x)) big = fmaxf(big, fabsf(x[w].x));
        if (finite_bits(x[w].y)) big = fmaxf(big, fabsf(x[w].y));
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, d));
      const int e = min(max(static_cast<int>(__float_as_uint(big) >> 23), 27), 227) - 127;
      const float down = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
      const float up = __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23);
#pragma unroll
      for (int w = 0; w < W; ++w)
        *reinterpret_cast<uint32_t*>(q_sh + r * (D + 8) + 2 * (lane + 32 * w)) = F16::pack(x[w].x * down, x[w].y * down);
      if (lane == 0) q_mul[r] = up * sc;
    }
    __syncthreads();
    constexpr bool QREG = D * NH <= 256;
    auto q_frag = [&](int kk, int n) {
      return *reinterpret_cast<const uint2*>(q_sh + (8 * n + g) * (D + 8) + kk * 16 + t4 * 4);
    };
    uint2 qf[QREG ? D / 16 : 1][NH];
    if constexpr (QREG) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int n = 0; n < NH; ++n) qf[kk][n] = q_frag(kk, n);
    }
    float mul[NH][2], m[NH][2], l[NH][2];  // of heads 8 n + 2 t4 and + 1
    float o[D / 16][NH][4];
#pragma unroll
    for (int n = 0; n < NH; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) mul[n][e] = q_mul[8 * n + 2 * t4 + e], m[n][e] = -INFINITY, l[n][e] = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.0f;
    }

    for (; chunk < chunk_end; chunk += kDecWarps) {
      issue();
      cp_async_wait<kDecStages - 1>();
      __syncwarp();
      const uint32_t st = stage0 + take * kStageBytes;
      const float* sc_sh = scale_sh[warp][take];
      take = take + 1 == kDecStages ? 0 : take + 1;
      bool full = static_cast<uint32_t>(chunk + 1) * TOK <= static_cast<uint32_t>(tok_end);
#pragma unroll
      for (int i = 0; i < TT; ++i) full &= sc_sh[4 + i] > 0.0f;  // a block outside the cache left zeros
      float s[TT][NH][4];
#pragma unroll
      for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int n = 0; n < NH; ++n) s[i][n][0] = s[i][n][1] = s[i][n][2] = s[i][n][3] = 0.0f;
#pragma unroll
      for (int k2 = 0; k2 < D / 32; ++k2) {
        uint32_t kb[TT][4];  // tokens 0-7, 8-15 of dims 32 k2 .. + 15, then of dims + 16 .. + 31
#pragma unroll
        for (int i = 0; i < TT; ++i) ldsm_x4(kb[i], st + code_at<D>(i * 16 + (lane & 15), 2 * k2 + (lane >> 4)));
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < TT; ++i) {
            const uint32_t af[4] = {ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(kb[i][2 * e])),
                                    ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(kb[i][2 * e + 1])),
                                    ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(kb[i][2 * e] >> 16)),
                                    ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(kb[i][2 * e + 1] >> 16))};
#pragma unroll
            for (int n = 0; n < NH; ++n) {
              const uint2 qb = QREG ? qf[QREG ? 2 * k2 + e : 0][n] : q_frag(2 * k2 + e, n);
              mma_16816<F16>(s[i][n], af, qb.x, qb.y);
            }
          }
      }
      float inv[TT], lg[TT], sk[TT];
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        const float sv = sc_sh[4 + i];
        sk[i] = sc_sh[i];
        lg[i] = sv > 0.0f ? log2_fast(sv) : -INFINITY;  // no block: every weight becomes 0
        inv[i] = sv > 0.0f ? 1.0f / sv : 0.0f;
      }
      float x[NH][2];
#pragma unroll
      for (int n = 0; n < NH; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x[n][e] = m[n][e];
#pragma unroll
          for (int i = 0; i < TT; ++i) {
            const float f = mul[n][e] * sk[i];
            s[i][n][e] = fmaf(s[i][n][e], f, lg[i]);
            s[i][n][e + 2] = fmaf(s[i][n][e + 2], f, lg[i]);
            if (!full) {
              const int tok = chunk * TOK + i * 16 + g;
              if (tok >= tok_end || lg[i] == -INFINITY) s[i][n][e] = -INFINITY;
              if (tok + 8 >= tok_end || lg[i] == -INFINITY) s[i][n][e + 2] = -INFINITY;
            }
            x[n][e] = fmaxf(x[n][e], fmaxf(s[i][n][e], s[i][n][e + 2]));
          }
        }
      }
#pragma unroll
      for (int d = 4; d < 32; d <<= 1)
#pragma unroll
        for (int n = 0; n < NH; ++n) {
          x[n][0] = fmaxf(x[n][0], __shfl_xor_sync(~0u, x[n][0], d));
          x[n][1] = fmaxf(x[n][1], __shfl_xor_sync(~0u, x[n][1], d));
        }
      if (!full) {  // a block that is left out for its scale: its codes may be NaN, which a weight of 0 does not hide
#pragma unroll
        for (int i = 0; i < TT; ++i)
          if (!(sc_sh[4 + i] > 0.0f))
            for (int x = lane; x < D; x += 32)
              zero16(st + kCodeBytes + code_at<D>(i * 16 + x / (D / 16), x % (D / 16)));
        __syncwarp();
      }
      bool grows = false;
#pragma unroll
      for (int n = 0; n < NH; ++n) grows |= x[n][0] > m[n][0] || x[n][1] > m[n][1];
      if (__any_sync(~0u, grows)) {  // seldom after a request's first chunks
#pragma unroll
        for (int n = 0; n < NH; ++n) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            f[e] = exp2_fast(m[n][e] - (x[n][e] == -INFINITY ? 0.0f : x[n][e]));
            m[n][e] = x[n][e];
            l[n][e] *= f[e];
          }
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
            o[i][n][0] *= f[0], o[i][n][1] *= f[1], o[i][n][2] *= f[0], o[i][n][3] *= f[1];
        }
      }
      uint32_t pb[TT][NH][2];
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        const float r0 = (m[n][0] == -INFINITY ? 0.0f : m[n][0]) - kTop,
                    r1 = (m[n][1] == -INFINITY ? 0.0f : m[n][1]) - kTop;
#pragma unroll
        for (int i = 0; i < TT; ++i) {
          const float e0 = exp2_fast(s[i][n][0] - r0), e1 = exp2_fast(s[i][n][1] - r1);
          const float e2 = exp2_fast(s[i][n][2] - r0), e3 = exp2_fast(s[i][n][3] - r1);
          l[n][0] = fmaf(e0 + e2, inv[i], l[n][0]);
          l[n][1] = fmaf(e1 + e3, inv[i], l[n][1]);
          pb[i][n][0] = transpose8x8(F16::pack(e0, e1));
          pb[i][n][1] = transpose8x8(F16::pack(e2, e3));
        }
      }
#pragma unroll
      for (int i = 0; i < TT; ++i) {
#pragma unroll
        for (int d2 = 0; d2 < D / 32; ++d2) {
          uint32_t vb[4];  // tokens 0-7, 8-15 of dims 32 d2 .. + 15, then of dims + 16 .. + 31
          ldsm_x4_t(vb, st + kCodeBytes + code_at<D>(i * 16 + (lane & 15), 2 * d2 + (lane >> 4)));
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t ev = __byte_perm(vb[2 * e], vb[2 * e + 1], 0x6420);
            const uint32_t od = __byte_perm(vb[2 * e], vb[2 * e + 1], 0x7531);
            const uint32_t af[4] = {ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(ev)),
                                    ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(od)),
                                    ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(ev >> 16)),
                                    ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(od >> 16))};
#pragma unroll
            for (int n = 0; n < NH; ++n) mma_16816<F16>(o[2 * d2 + e][n], af, pb[i][n][0], pb[i][n][1]);
          }
        }
      }
      __syncwarp();  // the stage is filled again by the next issue
    }
    cp_async_wait<0>();
    // The join's CTAs may come in. Let in at the kernel's start they take issue slots meanwhile (131072 tokens: 31.7 us
    // against 30.6; before the loop 31.4).
    let_next_start();

    // join the four warps
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[n][e] += __shfl_xor_sync(~0u, l[n][e], d);
        if (g == 0) m_sh[warp][8 * n + 2 * t4 + e] = m[n][e], l_sh[warp][8 * n + 2 * t4 + e] = l[n][e];
      }
    __syncthreads();  // every warp is done with its stages
    constexpr int OD = D + 4;  // (rows apart in their banks)
    float* o_sh = reinterpret_cast<float*>(smem);  // [4][8 NH][OD]
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        float* at = o_sh + (warp * 8 * NH + 8 * n + 2 * t4) * OD + i * 16 + 2 * g;
        *reinterpret_cast<float2*>(at) = make_float2(o[i][n][0], o[i][n][2]);
        *reinterpret_cast<float2*>(at + OD) = make_float2(o[i][n][1], o[i][n][3]);
      }
    __syncthreads();
    const bool whole = tiles == nt;
    float* piece = pieces + piece_floats(D) * (2 * blockIdx.x + (first == 0 ? 1 : 0));
    if (tid == 0) {
      int2* own = owners + static_cast<int64_t>(b) * geo.units_per_tile + hs;
      if (first == 0) own->x = whole ? -1 : static_cast<int>(blockIdx.x);
      if (first + tiles == nt) own->y = static_cast<int>(blockIdx.x);
    }
    for (int i = tid; i < rows * (D / 4); i += kDecThreads) {
      const int r = i / (D / 4), d = (i % (D / 4)) * 4;
      float mm = m_sh[0][r];
#pragma unroll
      for (int w = 1; w < kDecWarps; ++w) mm = fmaxf(mm, m_sh[w][r]);
      const float ms = mm == -INFINITY ? 0.0f : mm;
      float ll = 0.0f;
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float f = exp2_fast(m_sh[w][r] - ms);
        const float4 x = *reinterpret_cast<const float4*>(o_sh + (w * 8 * NH + r) * OD + d);
        ll = fmaf(l_sh[w][r], f, ll);
        acc.x = fmaf(x.x, f, acc.x), acc.y = fmaf(x.y, f, acc.y);
        acc.z = fmaf(x.z, f, acc.z), acc.w = fmaf(x.w, f, acc.w);
      }
      if (whole) {
        const float il = ll == 0.0f ? 0.0f : 1.0f / ll;
        uint16_t* out = static_cast<uint16_t*>(a.out) + b * a.out_token + (h0 + r) * a.out_head + d;
        *reinterpret_cast<uint2*>(out) = make_uint2(T::pack(acc.x * il, acc.y * il), T::pack(acc.z * il, acc.w * il));
        if (a.lse && d == 0)
          a.lse[static_cast<int64_t>(b) * a.n_heads + h0 + r] =
              ll == 0.0f ? -INFINITY : (mm - kTop + log2_fast(ll)) * kLn2;
      } else {
        if (d == 0) piece[r] = mm, piece[kRows + r] = ll;
        *reinterpret_cast<float4*>(piece + 2 * kRows + r * D + d) = acc;
      }
    }
    __syncthreads();
    u += tiles;
  }
}

// Joins the pieces of a (request, kv head, slice) in range order; zeros for a request without tokens. A CTA takes `cols`
// groups of four output values (of one row, or of several whole rows) and deals the pieces out over 256 / cols groups of
// threads, whose sums are added in order. What bounds it is latency: the pieces' (m, l) and the first of their values are
// all asked for at once. cols is small where there are few (request, kv head)s, each with many pieces, so that enough
// CTAs read them.
constexpr int kJoinThreads = 256, kJoinMinCols = 16;

template <class T, int D>
__global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(const __grid_constant__ moe_attn_decode_args a,
                                                                   int cols) {
  constexpr int ROW4 = D / 4, MAX_ROWS = kJoinThreads / ROW4;
  __shared__ float w_sh[MAX_ROWS][kDecCtas], lw_sh[MAX_ROWS][kDecCtas], m_sh[MAX_ROWS], l_sh[MAX_ROWS];
  __shared__ float4 o_sh[kJoinThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.y;
  const DecodeGeom geo = decode_geom(a.n_heads, a.n_kv_heads);
  const int per_unit = (geo.rows * ROW4 + cols - 1) / cols;
  const int hs = blockIdx.x / per_unit, item0 = (blockIdx.x % per_unit) * cols;
  const int head0 = (hs % geo.slices) * geo.rows, rows = min(geo.rows, geo.group - head0);
  const int h0 = (hs / geo.slices) * geo.group + head0;
  const int groups = kJoinThreads / cols, mine = item0 + tid % cols, grp = tid / cols;
  const int r = mine / ROW4, d = (mine % ROW4) * 4;
  const int r_first = item0 / ROW4, r_end = min(rows, (item0 + cols + ROW4 - 1) / ROW4);
  uint16_t* out = static_cast<uint16_t*>(a.out) + b * a.out_token + (h0 + r) * a.out_head + d;
  float* lse = a.lse ? a.lse + static_cast<int64_t>(b) * a.n_heads + h0 + r : nullptr;
  wait_for_previous();  // the pieces' kernel, and what that one has waited for
  if (request_len(a, b) <= 0) {
    if (grp == 0 && r < rows) {
      *reinterpret_cast<uint2*>(out) = make_uint2(0, 0);
      if (lse && d == 0) *lse = -INFINITY;
    }
    return;
  }
  const float* pieces = static_cast<const float*>(a.workspace);
  const int2* owners = reinterpret_cast<const int2*>(pieces + piece_floats(D) * 2 * kDecCtas);
  const int2 own = owners[static_cast<int64_t>(b) * geo.units_per_tile + hs];
  if (own.x < 0) return;
  const int n = own.y - own.x + 1;  // at most kDecCtas
  auto piece = [&](int i) { return pieces + piece_floats(D) * (2 * (own.x + i) + (i == 0 ? 1 : 0)); };
  constexpr int AHEAD = 4;
  float4 x[AHEAD];
#pragma unroll
  for (int k = 0; k < AHEAD; ++k)
    if (const int i = grp + k * groups; i < n && r < rows)
      x[k] = *reinterpret_cast<const float4*>(piece(i) + 2 * kRows + r * D + d);
  for (int i = tid; i < n * (r_end - r_first); i += kJoinThreads) {
    const int q = i / n, j = i % n;
    w_sh[q][j] = piece(j)[r_first + q];
    lw_sh[q][j] = piece(j)[kRows + r_first + q];
  }
  __syncthreads();
  for (int q = warp; q < r_end - r_first; q += kJoinThreads / 32) {
    float m = -INFINITY, l = 0.0f;
    for (int i = lane; i < n; i += 32) m = fmaxf(m, w_sh[q][i]);
#pragma unroll
    for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, k));
    const float ms = m == -INFINITY ? 0.0f : m;
    for (int i = lane; i < n; i += 32) {
      const float w = exp2_fast(w_sh[q][i] - ms);
      w_sh[q][i] = w;
      l = fmaf(lw_sh[q][i], w, l);
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) l += __shfl_xor_sync(~0u, l, k);
    if (lane == 0) m_sh[q] = m, l_sh[q] = l;
  }
  __syncthreads();
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (r < rows) {
    const float* w = w_sh[r - r_first];
    auto add = [&](const float4& v, float f) {
      acc.x = fmaf(v.x, f, acc.x), acc.y = fmaf(v.y, f, acc.y), acc.z = fmaf(v.z, f, acc.z), acc.w = fmaf(v.w, f, acc.w);
    };
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (const int i = grp + k * groups; i < n) add(x[k], w[i]);
#pragma unroll 4
    for (int i = grp + AHEAD * groups; i < n; i += groups)
      add(*reinterpret_cast<const float4*>(piece(i) + 2 * kRows + r * D + d), w[i]);
  }
  o_sh[tid] = acc;
  __syncthreads();
  if (grp == 0 && r < rows) {
    for (int i = 1; i < groups; ++i) {
      const float4 x = o_sh[i * cols + tid];
      acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
    }
    const float l = l_sh[r - r_first], il = l == 0.0f ? 0.0f : 1.0f / l;
    *reinterpret_cast<uint2*>(out) = make_uint2(T::pack(acc.x * il, acc.y * il), T::pack(acc.z * il, acc.w * il));
    if (lse && d == 0) *lse = l == 0.0f ? -INFINITY : (m_sh[r - r_first] - kTop + log2_fast(l)) * kLn2;
  }
}

template <class T, int D, int NH>
cudaError_t launch_decode(const moe_attn_decode_args& a, cudaStream_t stream) {
  constexpr int ring = kDecWarps * kDecStages * kStageBytes, join = kDecWarps * 8 * NH * (D + 4) * 4;
  constexpr int smem = ring > join ? ring : join;
  static OncePerDevice prepared;
  cudaError_t e = prepared([] {
    return cudaFuncSetAttribute(decode_kernel<T, D, NH>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  int block_log2 = 0;
  while ((1 << block_log2) < a.block_size) ++block_log2;
  e = launch_early(decode_kernel<T, D, NH>, dim3(kDecCtas), dim3(kDecThreads), smem, stream, a, block_log2);
  if (e != cudaSuccess) return e;
  const DecodeGeom geo = decode_geom(a.n_heads, a.n_kv_heads);
  const int64_t units = static_cast<int64_t>(geo.units_per_tile) * a.n_requests;
  int cols = kJoinMinCols, per_unit;
  for (;; cols *= 2) {
    per_unit = (geo.rows * (D / 4) + cols - 1) / cols;
    if (cols == kJoinThreads || units * per_unit <= 2 * kDecCtas) break;
  }
  return launch_early(decode_join_kernel<T, D>, dim3(geo.units_per_tile * per_unit, a.n_requests), dim3(kJoinThreads), 0,
                      stream, a, cols);
}

template <class T, int D>
cudaError_t decode_by_rows(const moe_attn_decode_args& a, cudaStream_t stream) {
  return decode_geom(a.n_heads, a.n_kv_heads).rows <= 8 ? launch_decode<T, D, 1>(a, stream)
                                                        : launch_decode<T, D, 2>(a, stream);
}

template <class T>
cudaError_t decode_by_dim(const moe_attn_decode_args& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 64: return decode_by_rows<T, 64>(a, stream);
    case 128: return decode_by_rows<T, 128>(a, stream);
    default: return decode_by_rows<T, 256>(a, stream);
  }
}

}  // namespace

size_t attn_decode_workspace(int n_requests, int n_heads, int n_kv_heads, int head_dim) {
  return piece_floats(head_dim) * 2 * kDecCtas * sizeof(float) +
         sizeof(int2) * static_cast<size_t>(n_requests) * decode_geom(n_heads, n_kv_heads).units_per_tile;
}

cudaError_t launch_attn_decode(const moe_attn_decode_args& a, cudaStream_t stream) {
  return a.dtype == MOE_ATTN_BF16 ? decode_by_dim<Bf16>(a, stream) : decode_by_dim<F16>(a, stream);
}

}  // namespace moe

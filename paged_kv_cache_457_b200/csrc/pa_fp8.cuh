// Decode attention over a paged cache held in 8 bits (e4m3) with one fp32
// scale for each (block, kv head) of K and of V.
//
// With sk(j), sv(j) the scales of token j's block, z_j = scale sk(j) <q, k_j>
// and w_j = 2^(z_j log2 e - m):   out = sum_j w_j sv(j) v_j / sum_j w_j.
// The bytes go to the tensor cores as they are: e4m3's values are fp16 values,
// so K and V are widened exactly to fp16 in registers (one cvt per two) and
// multiplied by mma.sync m16n8k16 with fp32 accumulation; both scales are
// applied to the products in fp32, once per 16 tokens instead of per element:
//   - sk multiplies the scores;
//   - sv joins the exponent: with zv_j = z_j + log2 sv(j) and m the running
//     maximum of zv, p_j = 2^(zv_j - m + 7) is the weight that multiplies the
//     bytes, and l += p_j / sv(j) the normaliser, so that out = acc / l and the
//     weights stay in fp16's range whatever the scales are.  p is rounded to
//     fp16 (half a step: 2^-11 of it; l adds the rounded values, a product of
//     P with a row of ones, so weights still sum to one) -- the bytes carry
//     2^-4.  The 16-bit kernels multiply the rounding's residual as well, which
//     here would double the products of V for an error of fp16 outputs of
//     0.00021 instead of 0.00025, bf16 outputs the same.  Factor 2^7: weights down to 2^-21 of the largest keep their bits,
//     those down to 2^-31 some, and the largest, 2^(7 + RESCALE_SLACK), fits.
// A query row in bf16 is scaled by a power of two to magnitudes in
// [2^14, 2^15) and so becomes fp16 without loss (elements below 2^-28 of the
// row's largest excepted); the power is undone with the score's scale.
//
// Per warp and tile of 32 tokens, 8 columns (below):
//   S^T[32 x 8] = K[32 x d] Q^T,  O^T[d x 8] += V^T[d x 32] P^T[32 x 8].
// The columns are the query heads that share the kv head, G at a time, of one
// token, or of several consecutive new tokens of a sequence (P tokens, P G <=
// 8) when a call brings a few per sequence: a K/V tile is then read and
// widened once for all of them, and a column's mask ends at its own token.
// The contraction over head dims may run in any order as long as K and Q agree:
// lane tig of a row takes d / 4 consecutive bytes, so K fragments are plain
// 16-byte shared-memory loads.  V^T needs pairs of tokens side by side:
// ldmatrix.trans on pairs of bytes, then one byte permute per register.
#pragma once

#include <cuda.h>

#include "pa_append.cuh"
#include "pa_chunk8.h"
#include "pa_kernels.cuh"
#include "pa_mma.cuh"
#include "pa_prefill.cuh"
#include "pa_table_window.h"
#include "pa_tcgen05.cuh"

namespace pa {

struct Decode8Args {
  // d.num_seqs counts row groups; d.q_seq_stride and d.out_seq_stride step from token to token; d.chunk_tiles counts
  // tiles of TILE8 tokens; d.k_cache and d.v_cache are unused
  DecodeArgs d;
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  // FEW kernels: [sequences + 1] first query token of each sequence
  const int32_t *query_start;
  long long num_query_tokens;
  int tokens;  // P: query tokens of a row group
  int groups;  // row groups of a sequence (1 for decode)
};

// Row group v: up to P consecutive query tokens of a sequence, attended together.
struct RowGroup {
  int s;    // sequence (table row)
  int L;    // tokens of the context that the group's last token sees; below 1: its rows are zeros
  int tok;  // first query token
  int cnt;  // query tokens, 0: none
};

// FEW: row groups of several tokens per sequence (query_start); else one token per sequence (decode), and what several
// would take folds away.
template <bool FEW>
__device__ __forceinline__ RowGroup row_group(const Decode8Args &a, int v) {
  RowGroup g;
  if constexpr (!FEW) {
    const int L = __ldg(a.d.context_lens + v);
    g.s = g.tok = v;
    g.cnt = 1;
    g.L = context_ok(a.d, L) ? L : -1;
    return g;
  }
  g.s = v / a.groups;
  const int i0 = (v - g.s * a.groups) * a.tokens;
  const int q0 = __ldg(a.query_start + g.s), n = __ldg(a.query_start + g.s + 1) - q0;
  const int ctx = __ldg(a.d.context_lens + g.s);
  const bool rows_ok = q0 >= 0 && n >= 0 && (long long)q0 + n <= a.num_query_tokens;
  g.tok = q0 + i0;
  g.cnt = rows_ok ? max(0, min(a.tokens, n - i0)) : 0;
  g.L = ctx >= n && (long long)ctx <= (long long)a.d.table_stride * a.d.block_size ? ctx - n + i0 + g.cnt : -1;
  return g;
}
// Status bits of the inputs behind row group v, reported once per sequence.
template <bool FEW>
__device__ __forceinline__ unsigned row_group_errors(const Decode8Args &a, int v) {
  if constexpr (!FEW) {
    const int L = __ldg(a.d.context_lens + v);
    if (context_ok(a.d, L)) return 0;
    return (L < 0 || (long long)L > (long long)a.d.table_stride * a.d.block_size) ? PA_DEV_ERR_CONTEXT
                                                                                  : PA_DEV_ERR_CONTEXT_HINT;
  }
  const int s = v / a.groups;
  if (v != s * a.groups) return 0;
  const int q0 = __ldg(a.query_start + s), n = __ldg(a.query_start + s + 1) - q0;
  if (q0 < 0 || n < 0 || (long long)q0 + n > a.num_query_tokens) return PA_DEV_ERR_CONTEXT;
  const unsigned hint = n > a.groups * a.tokens ? PA_DEV_ERR_CONTEXT_HINT : 0;
  return hint | (n > 0 && row_group<FEW>(a, v).L < 0 ? PA_DEV_ERR_CONTEXT : 0);
}
__device__ __forceinline__ int group_tiles(const RowGroup &g) {
  return g.cnt > 0 && g.L > 0 ? (g.L + TILE8 - 1) / TILE8 : 0;
}

// The cut of the tile stream (see ChunkPlan).
__device__ __forceinline__ ChunkPlan plan_chunks8(const DecodeArgs &a, int tiles_per_head_chunk_set) {
  ChunkPlan p;
  p.total = (long long)tiles_per_head_chunk_set * a.num_kv_heads * a.n_chunks;
  p.c1 = p.c2 = chunk8_tiles(p.total, a.split_warps, a.chunk_tiles, a.max_chunks);
  p.count = ceil_div8(p.total, p.c1);
  p.n1 = min((long long)a.split_warps, p.count);
  return p;
}

// pt[v] = tiles (per head chunk) of the row groups before v; all threads of the block, ends with a barrier.
template <bool FEW>
__device__ __forceinline__ void build_tile_prefix8(const Decode8Args &a, int *pt, int *scratch) {
  const int S = a.d.num_seqs, nth = blockDim.x, tid = threadIdx.x;
  const int per = (S + nth - 1) / nth;
  const int i0 = min(S, tid * per), i1 = min(S, i0 + per);
  int sum = 0;
  for (int i = i0; i < i1; ++i) {
    const int nt = group_tiles(row_group<FEW>(a, i));
    pt[i + 1] = nt;
    sum += nt;
  }
  const int lane = tid & 31, warp = tid >> 5;
  int incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(FULL, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  int run = incl - sum;
  for (int w = 0; w < warp; ++w) run += scratch[w];
  for (int i = i0; i < i1; ++i) {
    run += pt[i + 1];
    pt[i + 1] = run;
  }
  if (tid == 0) pt[0] = 0;
  __syncthreads();
}

// 4-byte asynchronous copy global -> shared, and its arrival on a barrier whose count includes it.
__device__ __forceinline__ void cp_async4(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// Offset of 16-byte chunk c of row r in a tile of D-byte rows with the TMA swizzle of D bytes (64 or 128): reads of
// the same chunks of 8 rows, and of chunks 2 tig and 2 tig + 1 of rows gid, meet every bank once.
template <int D>
__device__ __forceinline__ uint32_t swizzled8(int r, int c) {
  if constexpr (D == 128) return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
  return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

template <int D, int WARPS, int STAGES>
struct Smem8 {
  static constexpr uint32_t TILE_BYTES = TILE8 * D;
  static constexpr uint32_t STAGE_BYTES = 2 * TILE_BYTES;
  static constexpr uint32_t RING = WARPS * STAGES * STAGE_BYTES;
  static constexpr uint32_t SCALES = WARPS * STAGES * 16;  // per slot: K scales of both halves, V scales of both
  static constexpr uint32_t BARS = WARPS * STAGES * 8;
  static __host__ __device__ constexpr uint32_t bytes(int num_seqs) {
    return 1024 + RING + SCALES + BARS + (uint32_t)(num_seqs + 1 + WARPS) * 4u;  // 1024: alignment slack
  }
};
constexpr int BAR8_ARRIVALS = 1 + 4;  // lane 0's (with the tile's bytes) and one per scale

// The columns of a lane: its query row's (column gid) and its accumulators' (a = 2 tig, b = 2 tig + 1).  Column c is
// query head c % G of the unit and token c / G of the row group.
template <bool FEW>
struct Columns {
  int G, gid, tig;
  __device__ __forceinline__ Columns(int G_, int lane) : G(G_), gid(lane >> 2), tig(lane & 3) {}
  __device__ __forceinline__ int tok(int c) const { return FEW ? c / G : (c >= G ? 1 : 0); }
  // Elements from the row group's first row to column c's row of query head hq0 + ..., rows `stride` apart.
  template <int D>
  __device__ __forceinline__ long long offset(int c, int hq0, long long stride) const {
    const int t = FEW ? c / G : 0;
    return t * stride + (long long)(hq0 + c - t * G) * D;
  }
};

// The arithmetic of one piece (a run of tiles of one unit: a row group and a head chunk), one warp.
template <class E, int D, bool FEW>
struct Math8 {
  static constexpr int KSTEPS = D / 16;
  uint32_t qb[KSTEPS][2];
  float o[KSTEPS][4];  // [16 dims][dim 2 gid: column a, b; dim 2 gid + 1: column a, b]
  // per column a, b: the running maximum of zv less 7 (the weights' exponent offset), the normaliser over all lanes,
  // and the score scales (base-2 units)
  float ma, mb, la, lb, qa, qbs;
  float lv_top;     // largest log2 of a V scale so far in the piece
  int La, Lb, least;  // FEW: context tokens that columns a and b see, and the fewest that any column sees

  // The query rows of group g, unit's first head hq0.
  __device__ __forceinline__ void begin(const Decode8Args &args, const RowGroup &g, int hq0, bool ok,
                                        const Columns<FEW> &col) {
    const DecodeArgs &a = args.d;
    const bool live = ok && col.tok(col.gid) < g.cnt;
    uint4 w[D / 32];
    const uint4 *src = reinterpret_cast<const uint4 *>(
        a.q + (live ? (long long)g.tok * a.q_seq_stride + col.offset<D>(col.gid, hq0, a.q_seq_stride) : 0) +
        col.tig * (D / 4));
#pragma unroll
    for (int i = 0; i < D / 32; ++i) w[i] = live ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
    float unit = 1.f;
    if constexpr (std::is_same<E, BF16>::value) {
      float f[D / 4], amax = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        float t[8];
        E::widen8(w[i], t);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f[8 * i + e] = t[e];
          const float x = fabsf(t[e]);
          amax = fmaxf(amax, x < INFINITY ? x : 0.f);
        }
      }
      amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, 2));
      const int shift = min(14 - ((int)(__float_as_uint(amax) >> 23) - 127), 120);  // >= -113
      const float up = __uint_as_float((uint32_t)(127 + shift) << 23);
      unit = __uint_as_float((uint32_t)(127 - shift) << 23);
#pragma unroll
      for (int ks = 0; ks < KSTEPS; ++ks) {
        qb[ks][0] = F16::narrow2(f[4 * ks] * up, f[4 * ks + 1] * up);
        qb[ks][1] = F16::narrow2(f[4 * ks + 2] * up, f[4 * ks + 3] * up);
      }
    } else {
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        qb[2 * i][0] = w[i].x;
        qb[2 * i][1] = w[i].y;
        qb[2 * i + 1][0] = w[i].z;
        qb[2 * i + 1][1] = w[i].w;
      }
    }
    qa = __shfl_sync(FULL, unit, 8 * col.tig) * a.scale_log2;       // a lane of column 2 tig
    qbs = __shfl_sync(FULL, unit, 8 * col.tig + 4) * a.scale_log2;  // column 2 tig + 1
#pragma unroll
    for (int c = 0; c < KSTEPS; ++c) o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.f;
    ma = mb = lv_top = -INFINITY;
    la = lb = 0.f;
    if constexpr (FEW) {
      least = g.L - (g.cnt - 1);
      La = min(g.L, least + col.tok(2 * col.tig));
      Lb = min(g.L, least + col.tok(2 * col.tig + 1));
    }
  }

  // One tile at kt, vt (shared-memory addresses) with its scales (K of tokens 0-15 and 16-31, V likewise); nvalid live
  // rows, tokens j0 and on.  The caller has made sure that the slot's bytes have arrived; it is free again when this
  // returns.
  __device__ __forceinline__ void tile(uint32_t kt, uint32_t vt, float4 sc4, int nvalid, int j0, int lane) {
    // live rows that columns a and b see, and the fewest that any column sees
    const int na = FEW ? La - j0 : nvalid, nb = FEW ? Lb - j0 : nvalid, fewest = FEW ? least - j0 : nvalid;
    const int gid = lane >> 2, tig = lane & 3;
    float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    constexpr int CH = D / 64;  // 16-byte chunks of a row per lane
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      uint4 kw[2][2];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int u = 0; u < 2; ++u) kw[mt][u] = lds128(kt + swizzled8<D>(mt * 16 + u * 8 + gid, tig * CH + i));
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const uint32_t w0 = j == 0 ? kw[mt][0].x : j == 1 ? kw[mt][0].y : j == 2 ? kw[mt][0].z : kw[mt][0].w;
          const uint32_t w1 = j == 0 ? kw[mt][1].x : j == 1 ? kw[mt][1].y : j == 2 ? kw[mt][1].z : kw[mt][1].w;
          const uint32_t af[4] = {e4m3x2_to_f16x2((uint16_t)w0), e4m3x2_to_f16x2((uint16_t)w1),
                                  e4m3x2_to_f16x2((uint16_t)(w0 >> 16)), e4m3x2_to_f16x2((uint16_t)(w1 >> 16))};
          mma_16816_f16(sc[mt], af, qb[4 * i + j][0], qb[4 * i + j][1]);
        }
    }
    if (nvalid < TILE8) {
      if (nvalid <= 16) {  // a half without rows has no scales of its own
        sc4.y = sc4.x;
        sc4.w = sc4.z;
      }
      clear_tail(vt, nvalid, lane);
    }
    // log2 of V's scales; one below 2^-80 counts as zero (l, in units of 1 / scale, then fits fp32 whatever the length).
    // Under such a scale no weight multiplies the bytes, but all count in l: any exponent would do for them, and the
    // largest scale's so far keeps them near the others
    float lr[2] = {lg2(sc4.z), lg2(sc4.w)};
    lv_top = fmax3(lv_top, lr[0], lr[1]);
    const float low = fmaxf(lv_top, -80.f);
    float lv[2];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      if (lr[mt] < -80.f) lr[mt] = -INFINITY;
      lv[mt] = lr[mt] == -INFINITY ? low : lr[mt];
    }
    const float ka[2] = {sc4.x * qa, sc4.y * qa}, kb[2] = {sc4.x * qbs, sc4.y * qbs};
    // exponents of the weights, e = z + lv - (m - 7); dead rows -inf
    float e[2][4];
    auto exponents = [&]() {
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const float ca = lv[mt] - ma, cb = lv[mt] - mb;
        e[mt][0] = fmaf(sc[mt][0], ka[mt], ca);
        e[mt][1] = fmaf(sc[mt][1], kb[mt], cb);
        e[mt][2] = fmaf(sc[mt][2], ka[mt], ca);
        e[mt][3] = fmaf(sc[mt][3], kb[mt], cb);
      }
      if (fewest < TILE8) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          if (mt * 16 + gid >= na) e[mt][0] = -INFINITY;
          if (mt * 16 + gid >= nb) e[mt][1] = -INFINITY;
          if (mt * 16 + 8 + gid >= na) e[mt][2] = -INFINITY;
          if (mt * 16 + 8 + gid >= nb) e[mt][3] = -INFINITY;
        }
      }
    };
    exponents();
    // raise m only when some weight passes 2^(7 + slack): on the piece's first tile (m = -inf) and seldom after it
    const float top = fmaxf(fmax3(fmaxf(e[0][0], e[0][1]), e[0][2], e[0][3]),
                            fmax3(fmaxf(e[1][0], e[1][1]), e[1][2], e[1][3]));
    if (__any_sync(FULL, top > 7.f + RESCALE_SLACK)) {
      const float oa = ma, ob = mb;
      ma = mb = 0.f;
      exponents();  // z + lv themselves
      float ca = fmaxf(fmaxf(e[0][0], e[0][2]), fmaxf(e[1][0], e[1][2]));
      float cb = fmaxf(fmaxf(e[0][1], e[0][3]), fmaxf(e[1][1], e[1][3]));
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        ca = fmaxf(ca, __shfl_xor_sync(FULL, ca, off));
        cb = fmaxf(cb, __shfl_xor_sync(FULL, cb, off));
      }
      ma = fmaxf(oa, ca - 7.f);
      mb = fmaxf(ob, cb - 7.f);
      // 0 on the piece's first tile; a column that has seen no key yet has nothing to scale
      const float fa = ma > -INFINITY ? ex2(oa - ma) : 0.f, fb = mb > -INFINITY ? ex2(ob - mb) : 0.f;
#pragma unroll
      for (int c = 0; c < KSTEPS; ++c) {
        o[c][0] *= fa;
        o[c][1] *= fb;
        o[c][2] *= fa;
        o[c][3] *= fb;
      }
      // l in two steps: it is in units of 1 / scale, and m moves by the quotient of two scales
      const float ha = ma > -INFINITY ? ex2(0.5f * (oa - ma)) : 0.f, hb = mb > -INFINITY ? ex2(0.5f * (ob - mb)) : 0.f;
      la = la * ha * ha;
      lb = lb * hb * hb;
      exponents();
    }
    uint32_t pb[2][2];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const float p0 = ex2(e[mt][0]), p1 = ex2(e[mt][1]), p2 = ex2(e[mt][2]), p3 = ex2(e[mt][3]);
      pb[mt][0] = movmatrix_trans(F16::narrow2(p0, p1));
      pb[mt][1] = movmatrix_trans(F16::narrow2(p2, p3));
      // l: P times ones (every row of the product holds the sums of the rounded weights)
      float ls[4] = {0.f, 0.f, 0.f, 0.f};
      const uint32_t ones[4] = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
      mma_16816_f16(ls, ones, pb[mt][0], pb[mt][1]);
      float sa = ls[0], sb = ls[1], iv = ex2(-lv[mt]);
      if (lr[mt] < low - 10.f) {  // uniform, rare: under a scale this small fp16 has lost weights that count in l
        const float up = fminf(low - lv[mt], 112.f);  // and fp32 too when it is very small
        sa = ex2(e[mt][0] + up) + ex2(e[mt][2] + up);
        sb = ex2(e[mt][1] + up) + ex2(e[mt][3] + up);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          sa += __shfl_xor_sync(FULL, sa, off);
          sb += __shfl_xor_sync(FULL, sb, off);
        }
        iv = ex2(-lv[mt] - up);
        if (lr[mt] == -INFINITY) pb[mt][0] = pb[mt][1] = 0;
      }
      la = fmaf(sa, iv, la);
      lb = fmaf(sb, iv, lb);
    }
#pragma unroll
    for (int c = 0; c < KSTEPS; ++c) {
      uint32_t r[4];
      ldsm_x4_trans(r, vt + swizzled8<D>(lane, c));  // matrix i: tokens 8 i .. 8 i + 7, byte pairs of chunk c
      uint32_t lo[4], hi[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x = __byte_perm(r[i], 0, 0x3120);  // (dim 2 gid of both tokens, dim 2 gid + 1 of both)
        lo[i] = e4m3x2_to_f16x2((uint16_t)x);
        hi[i] = e4m3x2_to_f16x2((uint16_t)(x >> 16));
      }
      const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
      mma_16816_f16(o[c], a0, pb[0][0], pb[0][1]);
      mma_16816_f16(o[c], a1, pb[1][0], pb[1][1]);
    }
  }

  // The normalised rows of group g (zeros when bad).
  __device__ __forceinline__ void store_output(const Decode8Args &args, const RowGroup &g, int hq0, bool bad,
                                               const Columns<FEW> &col) const {
    const DecodeArgs &a = args.d;
    const float ia = 1.f / la, ib = 1.f / lb;
    uint16_t *rows = a.out + (long long)g.tok * a.out_seq_stride;
    uint16_t *ra = rows + col.offset<D>(2 * col.tig, hq0, a.out_seq_stride);
    uint16_t *rb = rows + col.offset<D>(2 * col.tig + 1, hq0, a.out_seq_stride);
    const bool wa = col.tok(2 * col.tig) < g.cnt, wb = col.tok(2 * col.tig + 1) < g.cnt;
#pragma unroll
    for (int c = 0; c < KSTEPS; ++c) {
      const int d = 16 * c + 2 * col.gid;
      if (wa) *reinterpret_cast<uint32_t *>(ra + d) = bad ? 0u : E::narrow2(o[c][0] * ia, o[c][2] * ia);
      if (wb) *reinterpret_cast<uint32_t *>(rb + d) = bad ? 0u : E::narrow2(o[c][1] * ib, o[c][3] * ib);
    }
  }

  // V's rows from nvalid on become zeros in place: they may hold NaN, or bytes never copied, and 0 * NaN is not 0.
  static __device__ __noinline__ void clear_tail(uint32_t vt, int nvalid, int lane) {
    for (int i = nvalid * D + lane * 4; i < TILE8 * D; i += 128)
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(vt + i), "r"(0) : "memory");  // whole rows: the swizzle permutes within one
    fence_proxy_async_smem();
    __syncwarp();
  }
};

// The physical blocks of a unit's tiles, through a 32-entry window of the table row (one entry per lane).  Entries past
// the row group's last block are not read.
struct TileLookup {
  TableWindow win;
  int ent = -1;
  // Tile j of row `s`, of a group that sees L tokens: *p0 the block of its first 16 tokens, *p1 that of the other 16
  // (second: whether there are such).  Returns whether the blocks lie in the pool.
  __device__ __forceinline__ bool find(const DecodeArgs &a, int s, int j, int L, int lane, int *p0, int *p1,
                                       bool *second) {
    const bool two = a.block_size == 16;
    if (win.ask(s, j, L, a.block_size)) {
      const int e = win.base + lane;
      ent = e < win.end && dcheck((long long)e * a.block_size < L && e < a.table_stride)
                ? __ldg(a.block_tables + (long long)s * a.table_stride + e)
                : -1;
    }
    const unsigned nblocks = (unsigned)a.num_blocks;  // below 2^31, as are the rows (checked on the host)
    *second = win.last > win.first;
    *p0 = __shfl_sync(FULL, ent, win.first - win.base);
    *p1 = two ? __shfl_sync(FULL, ent, (win.first + 1 - win.base) & 31) : *p0;
    return (unsigned)*p0 < nblocks && (!*second || (unsigned)*p1 < nblocks);
  }
};

// A piece's normaliser l (in units of 1 / scale) from its own exponent m to M, in two steps: 2^(m - M), with the quotient
// of two scales in it, may leave fp32's range where the product does not.
__device__ __forceinline__ float weighted_sum(float2 ml, float M) {
  const float h = exp2f(0.5f * (ml.x - M));
  return ml.y * h * h;
}

// Decode split kernel: the work decomposition of decode_split_mma_kernel (a balanced stream of tiles cut into chunks,
// pieces merged by a second kernel) on tiles of 32 tokens and units of a row group and a head chunk; K and V tiles
// arrive by TMA, the tile's scales by 4-byte asynchronous copies that complete on the same barrier.
// Bound by HBM on long streams: 8 contexts of 16k-32k tokens (1.68 GB) take 268 us, 0.95 of the measured copy rate; 64
// sequences of 32 heads (476 MB) 89 us, 0.81; 256 of 32 q / 8 kv heads with a long tail of lengths (484 MB) 107 us,
// 0.69: there every warp meets two or three pieces (query rows, partial states) per 31 tiles, and the stream's end is
// uneven.  A tile costs a warp about 2 us at 12 warps on an SM; widening the bytes (128 cvt per tile) and the products
// share the issue slots about evenly.
template <class E, int D, int WARPS, int STAGES, int BLOCKS, bool FEW>
__global__ void __launch_bounds__(WARPS * 32, BLOCKS)
    decode8_split_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                         const Decode8Args args) {
  static_assert(STAGES <= MIN_CHUNK8_TILES, "see there");
  const DecodeArgs &a = args.d;
  using Smem = Smem8<D, WARPS, STAGES>;
  constexpr int KSTEPS = D / 16;

  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);  // swizzle pattern alignment
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  unsigned char *ring = smem + warp * STAGES * Smem::STAGE_BYTES;
  float *scales = reinterpret_cast<float *>(smem + Smem::RING) + warp * STAGES * 4;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Smem::RING + Smem::SCALES) + warp * STAGES;
  int *pt = reinterpret_cast<int *>(smem + Smem::RING + Smem::SCALES + Smem::BARS);
  if (lane == 0) {
#pragma unroll
    for (int st = 0; st < STAGES; ++st) mbar_init(&bars[st], BAR8_ARRIVALS);
    fence_mbar_init();
    prefetch_tensor_map(&tmap_k);
    prefetch_tensor_map(&tmap_v);
  }
  grid_dependency_wait();    // every input may come from the previous kernel in the stream
  grid_launch_dependents();  // the merge kernel may launch now and wait for this grid
  if (blockIdx.x == 0 && threadIdx.x == 0) atomicExch(a.ws_queue, (unsigned long long)a.epoch << 32);
  const int S = a.num_seqs;
  build_tile_prefix8<FEW>(args, pt, pt + S + 1);
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= S; i += blockDim.x) a.ws_tiles[i] = pt[i];
  const ChunkPlan plan = plan_chunks8(a, pt[S]);
  const int HC = a.num_kv_heads * a.n_chunks;
  const Columns<FEW> col(a.heads_per_unit, lane);
  const int C = FEW ? args.tokens * a.heads_per_unit : a.heads_per_unit;  // columns in use

  long long cons_c = (long long)blockIdx.x * WARPS + warp;  // chunk the consumer is in (the first one is static)
  if (cons_c >= plan.count) return;

  ChunkQueue queue{a.ws_queue, a.epoch, (long long)a.split_warps, plan.count, 0ull};
  bool requested = false;  // a ticket for the producer's next chunk is on its way
  long long prod_c = cons_c;
  int prod_left = plan.length(prod_c);
  bool prod_done = false;
  TilePos cp = locate_tile(pt, S, HC, plan.start(cons_c));
  TilePos pos = cp;  // the producer's next tile
  TileLookup look;
  int prod_v = -1, prod_hc = -1, prod_h = 0;
  int prod_row = 0, prod_L = 0;  // table row and context of the producer's row group
  uint32_t bad_slots = 0;
  uint32_t iter = 0, issued = 0;

  // issue the producer's next tile, moving it into its next chunk when the current one is done
  auto issue_next = [&]() {
    if (prod_left == 0) {
      if (prod_done) return;
      if (!requested) queue.request(lane);
      requested = false;
      const long long nc = queue.take(lane, a.wait_limit_ns);
      if (nc >= plan.count) {
        prod_done = true;
        return;
      }
      prod_c = nc;
      prod_left = plan.length(nc);
      pos = locate_tile(pt, S, HC, plan.start(nc));
    }
    const int st = (int)(issued++ % STAGES);
    if (pos.s != prod_v) {
      prod_v = pos.s;
      const RowGroup pg = row_group<FEW>(args, pos.s);
      prod_row = pg.s;
      prod_L = pg.L;
    }
    if (pos.hc != prod_hc) {
      prod_hc = pos.hc;
      prod_h = pos.hc / a.n_chunks;
    }
    const int h = prod_h;
    // a new segment: its query rows on their way to L1, where the consumer will ask for them
    if (pos.j == 0) {
      const RowGroup pg = row_group<FEW>(args, pos.s);
      if (col.tok(col.gid) < pg.cnt)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(a.q + (long long)pg.tok * a.q_seq_stride +
                                                       col.offset<D>(col.gid, chunk_first_head(a, pos.hc), a.q_seq_stride) +
                                                       col.tig * (D / 4)));
    }
    int p0, p1;
    bool second;
    const bool found = look.find(a, prod_row, pos.j, prod_L, lane, &p0, &p1, &second);
    const bool good = found && dcheck(h < a.num_kv_heads && pos.j * TILE8 < prod_L);
    const bool whole = second || a.block_size != 16;  // both halves are copied
    bad_slots = good ? (bad_slots & ~(1u << st)) : (bad_slots | (1u << st));
    if (lane < 4) {
      if (good && (!(lane & 1) || whole))
        cp_async4(scales + st * 4 + lane,
                  ((lane & 2) ? args.v_scale : args.k_scale) + (((lane & 1) ? p1 : p0) * a.num_kv_heads + h));
      cp_async_arrive(&bars[st]);
    }
    if (lane == 0) {
      fence_proxy_async_smem();
      if (good) {
        unsigned char *kd = ring + st * Smem::STAGE_BYTES, *vd = kd + Smem::TILE_BYTES;
        const int r0 = (p0 * a.num_kv_heads + h) * a.block_size;
        mbar_arrive_expect_tx(&bars[st], whole ? Smem::STAGE_BYTES : Smem::STAGE_BYTES / 2);
        tma_load_2d(kd, &tmap_k, 0, r0, &bars[st]);
        tma_load_2d(vd, &tmap_v, 0, r0, &bars[st]);
        if (second) {
          const int r1 = (p1 * a.num_kv_heads + h) * a.block_size;
          tma_load_2d(kd + Smem::TILE_BYTES / 2, &tmap_k, 0, r1, &bars[st]);
          tma_load_2d(vd + Smem::TILE_BYTES / 2, &tmap_v, 0, r1, &bars[st]);
        }
      } else {
        mbar_arrive(&bars[st]);
      }
    }
    advance_tile(pos, pt, S, HC);
    --prod_left;
    if (!requested && prod_left <= TICKET_AHEAD) {
      queue.request(lane);
      requested = true;
    }
  };
  for (int k = 0; k < STAGES; ++k) issue_next();

  Math8<E, D, FEW> cm;
  RowGroup g{};
  int hq0 = 0, slot = 0;
  bool full = false, piece_bad = false;
  int cons_left = plan.length(cons_c);
  int k = 0;  // tile index within the consumer's chunk
  while (true) {
    if (cons_left == 0) {  // the consumer's chunk is done: follow the producer into its next chunk
      if (prod_c == cons_c) break;
      cons_c = prod_c;
      cons_left = plan.length(cons_c);
      cp = locate_tile(pt, S, HC, plan.start(cons_c));
      k = 0;
    }
    if (k == 0 || cp.j == 0) {  // a new piece: segment (cp.s, cp.hc) from tile cp.j on
      const int len = min(cp.nt - cp.j, cons_left);
      full = (cp.j == 0 && len == cp.nt);
      slot = (k == 0) ? 0 : 1;
      hq0 = chunk_first_head(a, cp.hc);
      const bool q_ok = dcheck(cp.s < S && hq0 + col.G <= a.num_q_heads);
      if (q_ok) g = row_group<FEW>(args, cp.s);
      piece_bad = false;
      cm.begin(args, g, hq0, q_ok, col);
    }
    const int st = (int)(iter % STAGES);
    if (!wait_slot<STAGES>(bars, iter, (int)(issued - iter), a.wait_limit_ns, lane)) return;
    piece_bad |= (bad_slots >> st) & 1u;  // warp-uniform
    if (!piece_bad) {
      const uint32_t kt = smem_addr(ring + st * Smem::STAGE_BYTES);
      const float4 sc4 = *reinterpret_cast<const float4 *>(scales + st * 4);
      const int j0 = cp.j * TILE8;
      cm.tile(kt, kt + Smem::TILE_BYTES, sc4, min(TILE8, g.L - j0), j0, lane);
    }
    __syncwarp();
    issue_next();
    ++iter;

    if (cp.j + 1 == cp.nt || cons_left == 1) {  // end of the piece
      if (piece_bad && lane == 0) atomicOr(&g_status, PA_DEV_ERR_BLOCK_ID);
      if (full) {
        if (dcheck(cp.s < S && hq0 + col.G <= a.num_q_heads)) cm.store_output(args, g, hq0, piece_bad, col);
      } else if (dcheck(cons_c < a.max_chunks)) {
        const long long prow = (cons_c * 2 + slot) * C;
        const int ca = 2 * col.tig, cb = ca + 1;
        if (!piece_bad) {
          float *acc = a.ws_acc + prow * D + 2 * col.gid;
#pragma unroll
          for (int c = 0; c < KSTEPS; ++c) {
            if (ca < C) *reinterpret_cast<float2 *>(acc + ca * D + 16 * c) = make_float2(cm.o[c][0], cm.o[c][2]);
            if (cb < C) *reinterpret_cast<float2 *>(acc + cb * D + 16 * c) = make_float2(cm.o[c][1], cm.o[c][3]);
          }
        }
        if (col.gid == 0) {
          if (ca < C) a.ws_ml[prow + ca] = piece_bad ? make_float2(-INFINITY, -1.f) : make_float2(cm.ma, cm.la);
          if (cb < C) a.ws_ml[prow + cb] = piece_bad ? make_float2(-INFINITY, -1.f) : make_float2(cm.mb, cm.lb);
        }
      }
    }
    advance_tile(cp, pt, S, HC);
    --cons_left;
    ++k;
  }
}

// One warp per HW columns of a unit: the zero rows of groups without a context (with the status bits of invalid
// inputs), and the merge of the pieces of units that the split kernel cut:
//   out = sum_p 2^(m_p - M) acc_p / sum_p 2^(m_p - M) l_p,  M = max_p m_p,
// in increasing chunk order (deterministic).  As decode_merge_kernel, for units whose columns are several tokens.
template <class E, int D, int HW, int MB, bool FEW>
__global__ void __launch_bounds__(256, 1) decode8_merge_kernel(const Decode8Args args) {
  static_assert(32 % MB == 0, "a batch of pieces never straddles a 32-piece window");
  const DecodeArgs &a = args.d;
  constexpr int DPL = D / 32;  // dims per lane (4 or 2)
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();  // the split kernel's pieces and tile prefix
  grid_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ws_queue = 0ull;  // leave the chunk counter clear
  const int S = a.num_seqs, HC = a.num_kv_heads * a.n_chunks, G = a.heads_per_unit, C = FEW ? args.tokens * G : G;
  const int subs = C / HW;  // warps per unit
  const long long w = (long long)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
  if (w >= (long long)S * HC * subs) return;
  const long long seg = w / subs;
  const int c0 = (int)(w - seg * subs) * HW;  // first column of this warp
  const int v = (int)(seg / HC), hc = (int)(seg - (long long)v * HC);
  const int pt0 = __ldg(a.ws_tiles + v), pt1 = __ldg(a.ws_tiles + v + 1), pts = __ldg(a.ws_tiles + S);
  const RowGroup g = row_group<FEW>(args, v);
  if (lane == 0 && hc == 0 && c0 == 0) {
    const unsigned err = row_group_errors<FEW>(args, v);
    if (err) atomicOr(&g_status, err);
  }
  if (c0 / G >= g.cnt) return;  // columns of no token
  float o[HW][DPL];
#pragma unroll
  for (int x = 0; x < HW; ++x)
#pragma unroll
    for (int k = 0; k < DPL; ++k) o[x][k] = 0.f;
  if (g.L > 0) {
    const ChunkPlan plan = plan_chunks8(a, pts);
    const int nt = pt1 - pt0;
    const long long seg0 = (long long)pt0 * HC + (long long)hc * nt;
    if (!dcheck(nt > 0 && pt0 >= 0 && pt1 <= pts)) return;  // a group with a context owns tiles
    const long long c_first = plan.chunk_of(seg0), c_last = plan.chunk_of(seg0 + nt - 1);
    if (c_first == c_last) return;  // one chunk held the whole unit: the split kernel wrote the rows
    if (!dcheck(c_first >= 0 && c_last < plan.count && c_last < a.max_chunks)) return;
    const int n = (int)(c_last - c_first + 1);
    const int first_slot = seg0 > plan.start(c_first) ? 1 : 0;
    auto piece_row = [&](int p) -> long long {  // partial row of this warp's first column in piece p
      return ((c_first + p) * 2 + (p == 0 ? first_slot : 0)) * C + c0;
    };
    // (m, l) of the first 32 pieces (lane p holds piece p) and the partial rows of the first batch, together
    float2 ml0[HW];
#pragma unroll
    for (int x = 0; x < HW; ++x) ml0[x] = make_float2(-INFINITY, 0.f);
    if (lane < n) {
      const long long r = piece_row(lane);
#pragma unroll
      for (int x = 0; x < HW; ++x) ml0[x] = __ldg(a.ws_ml + r + x);
    }
    float t[MB][HW][DPL];
    auto load_batch = [&](int base) {
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const bool ok = base + i < n;
        const long long r = ok ? piece_row(base + i) : 0;
#pragma unroll
        for (int x = 0; x < HW; ++x) {
          const float *src = a.ws_acc + (r + x) * D + lane * DPL;
          if constexpr (DPL == 4) {
            const float4 q = ok ? __ldg(reinterpret_cast<const float4 *>(src)) : make_float4(0.f, 0.f, 0.f, 0.f);
            t[i][x][0] = q.x;
            t[i][x][1] = q.y;
            t[i][x][2] = q.z;
            t[i][x][3] = q.w;
          } else {
            const float2 q = ok ? __ldg(reinterpret_cast<const float2 *>(src)) : make_float2(0.f, 0.f);
            t[i][x][0] = q.x;
            t[i][x][1] = q.y;
          }
        }
      }
    };
    load_batch(0);
    // maximum and validity over all pieces, per column
    float M[HW];
    bool err = false;
#pragma unroll
    for (int x = 0; x < HW; ++x) {
      M[x] = ml0[x].x;
      err |= lane < n && ml0[x].y < 0.f;
    }
    for (int p = lane + 32; p < n; p += 32) {
      const long long r = piece_row(p);
#pragma unroll
      for (int x = 0; x < HW; ++x) {
        const float2 ml = __ldg(a.ws_ml + r + x);
        M[x] = fmaxf(M[x], ml.x);
        err |= ml.y < 0.f;
      }
    }
#pragma unroll
    for (int x = 0; x < HW; ++x)
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) M[x] = fmaxf(M[x], __shfl_xor_sync(FULL, M[x], off));
    if (!__any_sync(FULL, err)) {
      // lane p of the current 32-piece window holds piece p's weight per column; weighted l sums run per lane
      float wt[HW], l[HW];
#pragma unroll
      for (int x = 0; x < HW; ++x) {
        wt[x] = lane < n ? exp2f(ml0[x].x - M[x]) : 0.f;
        l[x] = lane < n ? weighted_sum(ml0[x], M[x]) : 0.f;
      }
      for (int base = 0; base < n; base += MB) {
        if (base > 0) {
          if ((base & 31) == 0) {  // next window of 32 pieces: their (m, l)
            const int p = base + lane;
            const long long r = p < n ? piece_row(p) : 0;
#pragma unroll
            for (int x = 0; x < HW; ++x) {
              const float2 ml = p < n ? __ldg(a.ws_ml + r + x) : make_float2(-INFINITY, 0.f);
              wt[x] = p < n ? exp2f(ml.x - M[x]) : 0.f;
              if (p < n) l[x] += weighted_sum(ml, M[x]);
            }
          }
          load_batch(base);
        }
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          const int src_lane = (base + i) & 31;
#pragma unroll
          for (int x = 0; x < HW; ++x) {
            const float wq = __shfl_sync(FULL, wt[x], src_lane);  // 0 past the last piece
#pragma unroll
            for (int k = 0; k < DPL; ++k) o[x][k] = fmaf(wq, t[i][x][k], o[x][k]);
          }
        }
      }
#pragma unroll
      for (int x = 0; x < HW; ++x) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) l[x] += __shfl_xor_sync(FULL, l[x], off);
#pragma unroll
        for (int k = 0; k < DPL; ++k) o[x][k] = o[x][k] / l[x];
      }
    }
  }
#pragma unroll
  for (int x = 0; x < HW; ++x) {
    const int tok = (c0 + x) / G, head = chunk_first_head(a, hc) + (c0 + x) - tok * G;
    if (tok >= g.cnt) break;
    uint16_t *dst = a.out + (long long)(g.tok + tok) * a.out_seq_stride + (long long)head * D + lane * DPL;
    if constexpr (DPL == 4) {
      *reinterpret_cast<uint2 *>(dst) = make_uint2(E::narrow2(o[x][0], o[x][1]), E::narrow2(o[x][2], o[x][3]));
    } else {
      *reinterpret_cast<uint32_t *>(dst) = E::narrow2(o[x][0], o[x][1]);
    }
  }
}

// Small calls: one block per unit, its WARPS warps take the unit's tiles in turn (tile j to warp j mod WARPS), and
// their softmax states are merged in shared memory, in warp order (deterministic).  No workspace, no tensor map, no
// second launch: chosen when all units fit one wave of blocks and none is long, where the split kernel's tile prefix,
// queue and merge would cost more than the work.  Tiles come in by 16-byte asynchronous copies, placed as TMA's
// swizzle would.
template <int D, int WARPS>
struct SegSmem8 {
  static constexpr int STAGES = 2;
  static constexpr uint32_t TILE_BYTES = TILE8 * D;
  static constexpr uint32_t STAGE_BYTES = 2 * TILE_BYTES + 16;  // and the tile's four scales
  static constexpr uint32_t RING = WARPS * STAGES * STAGE_BYTES;
  static constexpr uint32_t MERGE = WARPS * 8 * (D + 2) * 4 + WARPS * 4;
  static constexpr uint32_t BYTES = RING > MERGE ? RING : MERGE;
};

template <class E, int D, int WARPS, bool FEW>
__global__ void __launch_bounds__(WARPS * 32, 3) decode8_segment_kernel(const Decode8Args args) {
  const DecodeArgs &a = args.d;
  using Smem = SegSmem8<D, WARPS>;
  constexpr int KSTEPS = D / 16, CPR = D / 16;  // 16-byte pieces of a row
  extern __shared__ __align__(128) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependency_wait();  // every input may come from the previous kernel in the stream
  grid_launch_dependents();
  const int HC = a.num_kv_heads * a.n_chunks;
  const int v = (int)(blockIdx.x / HC), hc = (int)(blockIdx.x - (unsigned)v * HC);
  const int hq0 = chunk_first_head(a, hc), h = hc / a.n_chunks;
  const Columns<FEW> col(a.heads_per_unit, lane);
  const RowGroup g = row_group<FEW>(args, v);
  if (hc == 0 && threadIdx.x == 0) {
    const unsigned err = row_group_errors<FEW>(args, v);
    if (err) atomicOr(&g_status, err);
  }
  const int C = g.cnt * col.G;  // live columns
  const int nt = group_tiles(g);
  auto out_row = [&](int c) {
    const int tok = c / col.G;
    return a.out + (long long)(g.tok + tok) * a.out_seq_stride + (long long)(hq0 + c - tok * col.G) * D;
  };
  if (nt == 0) {  // zero rows, or none
    for (int i = threadIdx.x; i < C * (D / 8); i += WARPS * 32)
      reinterpret_cast<uint4 *>(out_row(i / (D / 8)))[i % (D / 8)] = make_uint4(0, 0, 0, 0);
    return;
  }
  const int mine = warp < nt ? (nt - warp + WARPS - 1) / WARPS : 0;
  unsigned char *ring = smem + warp * Smem::STAGES * Smem::STAGE_BYTES;
  TileLookup look;
  bool bad = false;
  // this warp's t-th tile into slot t % 2; rows of a missing half are left alone (the arithmetic clears them)
  auto fetch = [&](int t) {
    const int j = warp + t * WARPS;
    int p0, p1;
    bool second;
    const bool good = look.find(a, g.s, j, g.L, lane, &p0, &p1, &second) && dcheck(h < a.num_kv_heads);
    bad |= !good;
    unsigned char *kd = ring + (t % Smem::STAGES) * Smem::STAGE_BYTES;
    if (good) {
      const int rows = second || a.block_size != 16 ? TILE8 : 16;
      const long long s0 = (long long)p0 * a.num_kv_heads + h, s1 = (long long)p1 * a.num_kv_heads + h;
      // row 16 + r of the tile: row r of the second block, or of the block's second half
      const long long b0 = s0 * a.block_size * D, b1 = a.block_size == 16 ? s1 * 16 * D : b0 + 16 * D;
#pragma unroll
      for (int i = 0; i < TILE8 * CPR / 32; ++i) {
        const int r = (i * 32 + lane) / CPR, c = (i * 32 + lane) % CPR;
        if (r >= rows) break;
        const long long src = (r < 16 ? b0 + r * D : b1 + (r - 16) * D) + c * 16;
        const uint32_t at = swizzled8<D>(r, c);
        cp_async16(kd + at, args.k_cache + src, true);
        cp_async16(kd + Smem::TILE_BYTES + at, args.v_cache + src, true);
      }
      if (lane < 4) {
        if (!(lane & 1) || rows == TILE8)
          cp_async4(kd + 2 * Smem::TILE_BYTES + lane * 4,
                    ((lane & 2) ? args.v_scale : args.k_scale) + ((lane & 1) ? s1 : s0));
      }
    }
    cp_async_commit();
  };
  if (mine > 0) fetch(0);
  Math8<E, D, FEW> cm;
  cm.begin(args, g, hq0, dcheck(hq0 + col.G <= a.num_q_heads), col);
  for (int t = 0; t < mine && !bad; ++t) {
    if (t + 1 < mine) {
      fetch(t + 1);
      cp_async_wait<1>();
    } else {
      cp_async_wait<0>();
    }
    __syncwarp();
    const unsigned char *kd = ring + (t % Smem::STAGES) * Smem::STAGE_BYTES;
    const float4 sc4 = *reinterpret_cast<const float4 *>(kd + 2 * Smem::TILE_BYTES);
    const int j0 = (warp + t * WARPS) * TILE8;
    cm.tile(smem_addr(kd), smem_addr(kd) + Smem::TILE_BYTES, sc4, min(TILE8, g.L - j0), j0, lane);
    __syncwarp();
  }
  cp_async_wait<0>();
  // the warps' states through shared memory (every copy has landed)
  __syncthreads();
  float *x_acc = reinterpret_cast<float *>(smem);  // [WARPS][8][D]
  float2 *x_ml = reinterpret_cast<float2 *>(x_acc + WARPS * 8 * D);
  int *x_bad = reinterpret_cast<int *>(x_ml + WARPS * 8);
  float *acc = x_acc + (warp * 8 + 2 * col.tig) * D + 2 * col.gid;
#pragma unroll
  for (int c = 0; c < KSTEPS; ++c) {
    *reinterpret_cast<float2 *>(acc + 16 * c) = make_float2(cm.o[c][0], cm.o[c][2]);
    *reinterpret_cast<float2 *>(acc + D + 16 * c) = make_float2(cm.o[c][1], cm.o[c][3]);
  }
  if (col.gid == 0) {
    x_ml[warp * 8 + 2 * col.tig] = make_float2(cm.ma, cm.la);
    x_ml[warp * 8 + 2 * col.tig + 1] = make_float2(cm.mb, cm.lb);
  }
  if (lane == 0) x_bad[warp] = bad ? 1 : 0;
  __syncthreads();
  bool any_bad = false;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) any_bad |= x_bad[w] != 0;
  if (any_bad && threadIdx.x == 0) atomicOr(&g_status, PA_DEV_ERR_BLOCK_ID);
  for (int i = threadIdx.x; i < C * (D / 8); i += WARPS * 32) {
    const int c = i / (D / 8), d0 = (i % (D / 8)) * 8;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, x_ml[w * 8 + c].x);
    float l = 0.f, f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float2 ml = x_ml[w * 8 + c];
      const float wt = ml.y != 0.f ? exp2f(ml.x - M) : 0.f;  // a warp without keys for this column: m = -inf, l = 0
      if (ml.y != 0.f) l += weighted_sum(ml, M);
      const float *src = x_acc + (w * 8 + c) * D + d0;
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = fmaf(wt, src[e], f[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = any_bad ? 0.f : f[e] / l;
    *reinterpret_cast<uint4 *>(out_row(c) + d0) = narrow8<E>(f);
  }
}

}  // namespace pa

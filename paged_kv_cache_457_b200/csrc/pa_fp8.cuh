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
//     2^-4.  Factor 2^7: weights down to
//     2^-31 of the largest are kept, and the largest, 2^(7 + RESCALE_SLACK),
//     fits.
// A query row in bf16 is scaled by a power of two to magnitudes in
// [2^14, 2^15) and so becomes fp16 without loss (elements below 2^-28 of the
// row's largest excepted); the power is undone with the score's scale.
//
// Per warp and tile of 32 tokens (G <= 8 query heads as the 8 columns):
//   S^T[32 x 8] = K[32 x d] Q^T,  O^T[d x 8] += V^T[d x 32] P^T[32 x 8].
// The contraction over head dims may run in any order as long as K and Q agree:
// lane tig of a row takes d / 4 consecutive bytes, so K fragments are plain
// 16-byte shared-memory loads.  V^T needs pairs of tokens side by side:
// ldmatrix.trans on pairs of bytes, then one byte permute per register.
#pragma once

#include <cuda.h>

#include "pa_append.cuh"
#include "pa_kernels.cuh"
#include "pa_mma.cuh"
#include "pa_prefill.cuh"
#include "pa_tcgen05.cuh"

namespace pa {

constexpr int TILE8 = 32;  // tokens per tile of the 8-bit kernels

struct Decode8Args {
  DecodeArgs d;  // k_cache / v_cache unused (tensor maps); chunk_tiles counts tiles of TILE8 tokens
  const float *k_scale, *v_scale;
};

__device__ __forceinline__ int seq_tiles8(const DecodeArgs &a, int L) {
  return (context_ok(a, L) && L > 0) ? (L + TILE8 - 1) / TILE8 : 0;
}

// pt[s] = tiles (per head chunk) of the sequences before s; all threads of the block, ends with a barrier.
__device__ __forceinline__ void build_tile_prefix8(const DecodeArgs &a, int *pt, int *scratch) {
  const int S = a.num_seqs, nth = blockDim.x, tid = threadIdx.x;
  const int per = (S + nth - 1) / nth;
  const int i0 = min(S, tid * per), i1 = min(S, i0 + per);
  int sum = 0;
  for (int i = i0; i < i1; ++i) {
    const int nt = seq_tiles8(a, __ldg(a.context_lens + i));
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

// The arithmetic of one piece (a run of tiles of one head chunk of G <= 8 query heads), one warp.
template <class E, int D>
struct Math8 {
  static constexpr int KSTEPS = D / 16;
  uint32_t qb[KSTEPS][2];
  float o[KSTEPS][4];  // [16 dims][dim 2 gid: head a, head b; dim 2 gid + 1: head a, head b]
  // per head column a = 2 tig, b = 2 tig + 1: the running maximum of zv less 7 (the weights' exponent offset), the
  // normaliser over all lanes, and the score scales (base-2 units)
  float ma, mb, la, lb, qa, qbs;
  float lv_top;  // largest log2 of a V scale so far in the piece

  // Query rows qrow + g * D of heads g < G.
  __device__ __forceinline__ void begin(const uint16_t *qrow, int G, bool ok, float scale_log2, int lane) {
    const int gid = lane >> 2, tig = lane & 3;
    const bool live = ok && gid < G;
    uint4 w[D / 32];
    const uint4 *src = reinterpret_cast<const uint4 *>(qrow + (long long)(live ? gid : 0) * D + tig * (D / 4));
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
    qa = __shfl_sync(FULL, unit, 8 * tig) * scale_log2;       // lane of head 2 tig, any of its four
    qbs = __shfl_sync(FULL, unit, 8 * tig + 4) * scale_log2;  // head 2 tig + 1
#pragma unroll
    for (int c = 0; c < KSTEPS; ++c) o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.f;
    ma = mb = lv_top = -INFINITY;
    la = lb = 0.f;
  }

  // One tile at kt, vt (shared-memory addresses) with its scales (K of tokens 0-15 and 16-31, V likewise); nvalid live
  // rows.  The caller has made sure that the slot's bytes have arrived; it is free again when this returns.
  __device__ __forceinline__ void tile(uint32_t kt, uint32_t vt, float4 sc4, int nvalid, int lane) {
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
    // a scale of zero (a block of zeros) would send the exponent to -inf: its bytes are zeros, any small scale will do
    const float lv[2] = {lg2(fmaxf(sc4.z, 5.421011e-20f)), lg2(fmaxf(sc4.w, 5.421011e-20f))};
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
      if (nvalid < TILE8) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          if (mt * 16 + gid >= nvalid) e[mt][0] = e[mt][1] = -INFINITY;
          if (mt * 16 + 8 + gid >= nvalid) e[mt][2] = e[mt][3] = -INFINITY;
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
      const float fa = ex2(oa - ma), fb = ex2(ob - mb);  // 0 on the piece's first tile
#pragma unroll
      for (int c = 0; c < KSTEPS; ++c) {
        o[c][0] *= fa;
        o[c][1] *= fb;
        o[c][2] *= fa;
        o[c][3] *= fb;
      }
      la *= fa;
      lb *= fb;
      exponents();
    }
    lv_top = fmax3(lv_top, lv[0], lv[1]);
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
      float sa = ls[0], sb = ls[1];
      if (lv[mt] < lv_top - 10.f) {  // uniform, rare: under a scale this small fp16 has lost weights that count in l
        sa = p0 + p2;
        sb = p1 + p3;
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          sa += __shfl_xor_sync(FULL, sa, off);
          sb += __shfl_xor_sync(FULL, sb, off);
        }
      }
      const float iv = ex2(-lv[mt]);
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

  // V's rows from nvalid on become zeros in place: they may hold NaN, or bytes never copied, and 0 * NaN is not 0.
  static __device__ __noinline__ void clear_tail(uint32_t vt, int nvalid, int lane) {
    for (int i = nvalid * D + lane * 4; i < TILE8 * D; i += 128)
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(vt + i), "r"(0) : "memory");  // whole rows: the swizzle permutes within one
    fence_proxy_async_smem();
    __syncwarp();
  }
};

// Decode split kernel: the work decomposition of decode_split_mma_kernel (a balanced stream of tiles cut into chunks,
// pieces merged by decode_merge_kernel) on tiles of 32 tokens; K and V tiles arrive by TMA, the tile's scales by
// 4-byte asynchronous copies that complete on the same barrier.
template <class E, int D, int WARPS, int STAGES, int BLOCKS>
__global__ void __launch_bounds__(WARPS * 32, BLOCKS)
    decode8_split_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                         const Decode8Args args) {
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
  build_tile_prefix8(a, pt, pt + S + 1);
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= S; i += blockDim.x) a.ws_tiles[i] = pt[i];
  const ChunkPlan plan = plan_chunks(a, pt[S]);
  const int HC = a.num_kv_heads * a.n_chunks;
  const int G = a.heads_per_unit;
  const bool two = a.block_size == 16;  // a tile spans two blocks

  long long cons_c = (long long)blockIdx.x * WARPS + warp;  // chunk the consumer is in (the first one is static)
  if (cons_c >= plan.count) return;

  ChunkQueue queue{a.ws_queue, a.epoch, (long long)a.split_warps, plan.count, 0ull};
  bool requested = false;  // a ticket for the producer's next chunk is on its way
  long long prod_c = cons_c;
  int prod_left = plan.length(prod_c);
  bool prod_done = false;
  TilePos cp = locate_tile(pt, S, HC, plan.start(cons_c));
  TilePos pos = cp;  // the producer's next tile
  int win_s = -1, win_base = 0, ent = -1, prod_L = 0, prod_hc = -1, prod_h = 0;
  const unsigned nblocks = (unsigned)a.num_blocks;  // below 2^31, as are the rows (checked on the host)
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
    const int b0 = two ? 2 * pos.j : pos.j;
    if (pos.s != win_s || b0 < win_base || b0 >= win_base + 32) {
      // a window of 32 entries of the row; those past the sequence's last tile are not read, and the one past its last
      // block (an odd count of 16-token blocks) is never used
      if (pos.s != win_s) prod_L = __ldg(a.context_lens + pos.s);
      win_s = pos.s;
      win_base = b0 & ~31;
      const int n = min(a.table_stride, two ? 2 * pos.nt : pos.nt);
      ent = (win_base + lane < n && dcheck(pos.s < S))
                ? __ldg(a.block_tables + (long long)pos.s * a.table_stride + win_base + lane)
                : -1;
    }
    const int p0 = __shfl_sync(FULL, ent, b0 - win_base);
    const int p1 = two ? __shfl_sync(FULL, ent, (b0 + 1 - win_base) & 31) : p0;  // b0 is even: the same window
    const bool second = two && pos.j * TILE8 + 16 < prod_L;
    if (pos.hc != prod_hc) {
      prod_hc = pos.hc;
      prod_h = pos.hc / a.n_chunks;
    }
    if (pos.j == 0) {  // a new segment: its query rows on their way to L1, where the consumer will ask for them
      const int g = lane >> 2;
      if (g < G)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(a.q + (long long)pos.s * a.q_seq_stride +
                                                       (long long)(chunk_first_head(a, pos.hc) + g) * D + (lane & 3) * (D / 4)));
    }
    const int h = prod_h;
    const bool good = (unsigned)p0 < nblocks && (!second || (unsigned)p1 < nblocks) && dcheck(h < a.num_kv_heads);
    bad_slots = good ? (bad_slots & ~(1u << st)) : (bad_slots | (1u << st));
    if (lane < 4) {
      if (good && (!(lane & 1) || second || !two))
        cp_async4(scales + st * 4 + lane,
                  ((lane & 2) ? args.v_scale : args.k_scale) + (((lane & 1) ? p1 : p0) * a.num_kv_heads + h));
      cp_async_arrive(&bars[st]);
    }
    if (lane == 0) {
      fence_proxy_async_smem();
      if (good) {
        unsigned char *kd = ring + st * Smem::STAGE_BYTES, *vd = kd + Smem::TILE_BYTES;
        const int r0 = (p0 * a.num_kv_heads + h) * a.block_size;
        mbar_arrive_expect_tx(&bars[st], (second || !two) ? Smem::STAGE_BYTES : Smem::STAGE_BYTES / 2);
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

  Math8<E, D> cm;
  int L = 0, hq0 = 0, slot = 0;
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
      const bool q_ok = dcheck(cp.s < S && hq0 + G <= a.num_q_heads);
      L = q_ok ? __ldg(a.context_lens + cp.s) : 0;
      piece_bad = false;
      cm.begin(a.q + (long long)cp.s * a.q_seq_stride + (long long)hq0 * D, G, q_ok, a.scale_log2, lane);
    }
    const int st = (int)(iter % STAGES);
    if (!wait_slot<STAGES>(bars, iter, (int)(issued - iter), a.wait_limit_ns, lane)) return;
    piece_bad |= (bad_slots >> st) & 1u;  // warp-uniform
    if (!piece_bad) {
      const uint32_t kt = smem_addr(ring + st * Smem::STAGE_BYTES);
      const float4 sc4 = *reinterpret_cast<const float4 *>(scales + st * 4);
      cm.tile(kt, kt + Smem::TILE_BYTES, sc4, min(TILE8, L - cp.j * TILE8), lane);
    }
    __syncwarp();
    issue_next();
    ++iter;

    if (cp.j + 1 == cp.nt || cons_left == 1) {  // end of the piece
      if (piece_bad && lane == 0) atomicOr(&g_status, PA_DEV_ERR_BLOCK_ID);
      const int gid = lane >> 2, ha = 2 * (lane & 3), hb = ha + 1;
      if (full) {
        const float ia = 1.f / cm.la, ib = 1.f / cm.lb;
        uint16_t *orow = a.out + (long long)cp.s * a.out_seq_stride + (long long)hq0 * D + 2 * gid;
        if (dcheck(cp.s < S && hq0 + G <= a.num_q_heads)) {
#pragma unroll
          for (int c = 0; c < KSTEPS; ++c) {
            if (ha < G)
              *reinterpret_cast<uint32_t *>(orow + ha * D + 16 * c) =
                  piece_bad ? 0u : E::narrow2(cm.o[c][0] * ia, cm.o[c][2] * ia);
            if (hb < G)
              *reinterpret_cast<uint32_t *>(orow + hb * D + 16 * c) =
                  piece_bad ? 0u : E::narrow2(cm.o[c][1] * ib, cm.o[c][3] * ib);
          }
        }
      } else if (dcheck(cons_c < a.max_chunks)) {
        const long long prow = (cons_c * 2 + slot) * G;
        if (!piece_bad) {
          float *acc = a.ws_acc + prow * D + 2 * gid;
#pragma unroll
          for (int c = 0; c < KSTEPS; ++c) {
            if (ha < G) *reinterpret_cast<float2 *>(acc + ha * D + 16 * c) = make_float2(cm.o[c][0], cm.o[c][2]);
            if (hb < G) *reinterpret_cast<float2 *>(acc + hb * D + 16 * c) = make_float2(cm.o[c][1], cm.o[c][3]);
          }
        }
        if (gid == 0) {
          if (ha < G) a.ws_ml[prow + ha] = piece_bad ? make_float2(-INFINITY, -1.f) : make_float2(cm.ma, cm.la);
          if (hb < G) a.ws_ml[prow + hb] = piece_bad ? make_float2(-INFINITY, -1.f) : make_float2(cm.mb, cm.lb);
        }
      }
    }
    advance_tile(cp, pt, S, HC);
    --cons_left;
    ++k;
  }
}

}  // namespace pa

// Causal prefill / chunked prefill over a paged cache held in 8 bits.
//
// The pipeline of prefill_tc_kernel (two 128-row sub-tiles of one query head
// against 128-key tiles, tcgen05 with accumulators in tensor memory, one
// softmax warpgroup per sub-tile), with the page tiles brought in by seven
// loader warps instead of TMA: they read e4m3 rows (16 bytes a lane, whole
// 128-byte lines a warp), widen them, multiply by the block's scale in fp32,
// round to the storage type and store them in the 128-byte swizzle the tensor
// cores read.  The rounding changes nothing where the scale is a power of two
// and the value a normal number of the type (every cache the appends fill, in
// bf16; from scales of 2^-15 on in fp16); other scales cost half a step of the
// storage type, far below the bytes' own 2^-4.  Rows past the context are
// stored as zeros whatever the pool holds there.
//
// Why not the tensor cores' own 8-bit kinds: they would need Q and P in 8 bits
// too.
//
// Softmax weights are rounded to the storage type as well: the 16-bit kind
// takes both operands of a product in one type.  The normaliser sums the
// rounded weights, so an output is still a mean of V.  Relative error against
// 64-bit arithmetic, output rounding included, with this and with 32-bit
// weights: 0.0021 and 0.0017 in bf16, 0.00024 and 0.00021 in fp16.
//
// 32 chunks of 512 tokens behind 0-3584, 32 q / 8 kv heads, take 742 us (735
// TFLOP/s); with the bytes stored unwidened in a scratch copy, 693.
//
// Work items are taken from a counter in the call's workspace.  The warp that
// takes an item checks all of its table entries first, so that the other roles
// never meet a missing page: such an item's rows are zeroed there and then.
#pragma once

#include "pa_append.cuh"
#include "pa_prefill.cuh"

namespace pa {

struct Prefill8Args {
  PrefillArgs p;
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  float k_sign;  // sign of the softmax scale (0 for a scale of 0), multiplied into K: p.scale_log2 is then positive
};

constexpr int PF8_THREADS = 16 * 32;  // 8 softmax warps, 8 / 9 / 11-15 loaders, 10 MMA issue
constexpr int PF8_LOADERS = 7;
constexpr int PF8_ITEM_READERS = 15;  // six loaders, MMA lane, 8 softmax warps
// Registers per thread: 128 at launch (512 threads fill the file); the two softmax warpgroups take 48 more each from
// the two others: 256 * 176 + 256 * 80 = 512 * 128.
constexpr int PF8_SOFTMAX_REGS = 176, PF8_OTHER_REGS = 80;
constexpr int PF8_QUARTERS = 4;       // a K or V tile is brought in as four units of 32 rows

// Rings of K and V tiles.  What shared memory does not take is L1, which the loaders' 16-byte reads want: a third slot
// for K or for V costs more than it gives (783 and 780 against 742 us for 32 chunks of 512 tokens behind 0-3584).
constexpr int PF8_KST = 2, PF8_VST = 2;

template <int D>
struct Prefill8Smem {
  static constexpr uint32_t REGION = 128 * 128;  // 128 rows of 128 bytes (64 elements)
  static constexpr uint32_t HALVES = D / 64;
  static constexpr uint32_t Q = 0;  // sub-tiles A and B
  static constexpr uint32_t K = Q + 2 * HALVES * REGION;
  static constexpr uint32_t V = K + PF8_KST * HALVES * REGION;
  static constexpr uint32_t BARS = V + PF8_VST * HALVES * REGION;
  static constexpr uint32_t BYTES = BARS + 512;  // 25 mbarriers, the item ring, the tensor-memory address, flags
  // + alignment slack; at least 120 KB so that one CTA holds an SM (and its tensor memory) alone
  static constexpr uint32_t ALLOC = (BYTES + 1024 > 120 * 1024) ? BYTES + 1024 : 120 * 1024;
  // tensor memory columns
  static constexpr uint32_t T_S = 0;      // S_x at T_S + x * 128; P_x in its first 64 columns
  static constexpr uint32_t T_O = 256;    // O_x at T_O + x * D
};
static_assert(Prefill8Smem<128>::ALLOC <= 232448, "prefill smem over the per-block opt-in limit");

template <int N>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Two fp32 values to the storage type, saturating (a re-scaled byte can pass fp16's largest value by a rounding).
template <class E>
__device__ __forceinline__ uint32_t narrow2_sat(float lo, float hi) {
  if constexpr (std::is_same<E, F16>::value) {
    uint32_t d;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
  }
  return E::narrow2(lo, hi);
}

// Two e4m3 values times a scale, in the storage type.  `s16`: the scale in fp16 when FAST (it is then exact there and
// no product overflows): fp16 by one packed product, bf16 by mixed-precision ones.
template <class E, bool FAST>
__device__ __forceinline__ uint32_t scaled2(uint16_t x, float s, uint32_t s16) {
  const uint32_t h = e4m3x2_to_f16x2(x);
  if constexpr (FAST && std::is_same<E, F16>::value) {
    const __half2 p = __hmul2(*reinterpret_cast<const __half2 *>(&h), *reinterpret_cast<const __half2 *>(&s16));
    return *reinterpret_cast<const uint32_t *>(&p);
  } else if constexpr (FAST) {
    float lo, hi;
    asm("{\n\t.reg .b16 a, b, s, t;\n\tmov.b32 {a, b}, %2;\n\tmov.b32 {s, t}, %3;\n\t"
        "fma.rn.f32.f16 %0, a, s, 0f00000000;\n\tfma.rn.f32.f16 %1, b, s, 0f00000000;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h), "r"(s16));
    return E::narrow2(lo, hi);
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    return narrow2_sat<E>(f.x * s, f.y * s);
  }
}
// Whether a scale is an exact fp16 power of two (or zero) whose products with e4m3 values stay below fp16's largest
// value and normal scale: |s| in [2^-14, 2^7].
__device__ __forceinline__ bool scale_is_plain(float s) {
  const float a = fabsf(s);
  return s == 0.f || ((__float_as_uint(s) & 0x7fffffu) == 0 && a >= 6.103515625e-5f && a <= 128.f);
}

// One unit: 32 rows of a K or V tile, held by the warp as pieces of 16 bytes.
template <class E, int D>
struct LoadUnit {
  static constexpr int LPR = D / 16;       // lanes of a row
  static constexpr int N = LPR;            // pieces per lane: 32 rows * LPR / 32 lanes
  static constexpr int STEP = 32 / LPR;    // rows between a lane's pieces
  uint4 w[N];
  float s[2];  // scales of rows 0-15 and 16-31

  // Rows tok0 .. tok0 + 31 of the item's context; p0, p1: physical blocks of the two halves (-1: past the context).
  __device__ __forceinline__ void load(const uint8_t *cache, const float *scale, const PrefillArgs &a, int h, int p0,
                                       int p1, int tok0, int kmax, int lane) {
    // the unit's two halves of 16 rows: blocks p0 and p1, or the two halves of block p0
    const long long slab0 = (long long)p0 * a.num_kv_heads + h, slab1 = (long long)p1 * a.num_kv_heads + h;
    s[0] = p0 >= 0 ? __ldg(scale + slab0) : 0.f;
    s[1] = p1 >= 0 ? __ldg(scale + slab1) : 0.f;
    const int off = (lane / LPR) * D + (lane % LPR) * 16;
    const uint8_t *half0 = cache + slab0 * a.block_size * D + off;
    const uint8_t *half1 = cache + slab1 * a.block_size * D + (a.block_size == 16 ? 0 : 16 * D) + off;
    const int live = kmax - tok0 - lane / LPR;  // rows of this lane's column that lie in the context
#pragma unroll
    for (int i = 0; i < N; ++i)
      w[i] = i * STEP < live ? __ldg(reinterpret_cast<const uint4 *>((i < N / 2 ? half0 : half1) + (i % (N / 2)) * STEP * D))
                             : make_uint4(0, 0, 0, 0);
  }
  // A piece becomes chunks c0 and c0 + 1 of its 64-element region.  The two regions' chunks of a row fall on the same
  // banks (two-way conflicts); swapping the order for one region cost more in selects, or in 8-byte loads (5 and
  // 20 us more for 32 chunks of 512 tokens).
  template <bool FAST>
  __device__ __forceinline__ void store_as(uint8_t *tile, int row0, float s0, float s1, int lane) const {
    uint8_t *region = tile + ((lane % LPR) / 4) * 128 * 128;
    const int c0 = ((lane % LPR) % 4) * 2;
    const uint32_t h0 = F16::narrow2(s0, s0), h1 = F16::narrow2(s1, s1);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float sc = i < N / 2 ? s0 : s1;
      const uint32_t hc = i < N / 2 ? h0 : h1;
      const int row = row0 + i * STEP + lane / LPR, sw = row & 7;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint2 x = k == 0 ? make_uint2(w[i].x, w[i].y) : make_uint2(w[i].z, w[i].w);
        *reinterpret_cast<uint4 *>(region + row * 128 + (((c0 + k) ^ sw) << 4)) =
            make_uint4(scaled2<E, FAST>((uint16_t)x.x, sc, hc), scaled2<E, FAST>((uint16_t)(x.x >> 16), sc, hc),
                       scaled2<E, FAST>((uint16_t)x.y, sc, hc), scaled2<E, FAST>((uint16_t)(x.y >> 16), sc, hc));
      }
    }
  }
  // Into rows row0 .. row0 + 31 of a tile stored as D / 64 regions of [128 rows][128 bytes], swizzled.
  __device__ __forceinline__ void store(uint8_t *tile, int row0, float factor, int lane) const {
    const float s0 = s[0] * factor, s1 = s[1] * factor;
    if (scale_is_plain(s0) && scale_is_plain(s1))  // uniform
      store_as<true>(tile, row0, s0, s1, lane);
    else
      store_as<false>(tile, row0, s0, s1, lane);
  }
};

template <class E, int D>
__global__ void __launch_bounds__(PF8_THREADS, 1)
    prefill8_tc_kernel(const __grid_constant__ CUtensorMap tmap_q, const Prefill8Args args) {
  const PrefillArgs &a = args.p;
  using L = Prefill8Smem<D>;
  constexpr int HALVES = D / 64;
  constexpr uint32_t REGION = L::REGION;
  constexpr bool kBf16 = std::is_same<E, BF16>::value;

  grid_dependency_wait();  // inputs may come from the previous kernel in the stream

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  uint8_t *sm = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const uint32_t sbase = smem_addr(sm);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BARS);
  uint64_t *q_full = bars;
  uint64_t *q_empty = q_full + 1;
  uint64_t *k_full = q_empty + 1;       // [PF8_KST]
  uint64_t *k_empty = k_full + PF8_KST;  // [PF8_KST]
  uint64_t *v_full = k_empty + PF8_KST;  // [PF8_VST]
  uint64_t *v_empty = v_full + PF8_VST;  // [PF8_VST]
  uint64_t *s_full = v_empty + PF8_VST;  // [2]: S_A, S_B written (and every earlier MMA done)
  uint64_t *p_full = s_full + 2;        // [2]: P_A, P_B written
  uint64_t *o_done = p_full + 2;        // [2]: an item's last PV of A, of B done
  uint64_t *drained = o_done + 2;
  uint64_t *item_full = drained + 1;   // [4]: the ring of items handed out by the first loader
  uint64_t *item_empty = item_full + 4;
  volatile long long *items = reinterpret_cast<volatile long long *>(item_empty + 4);  // [4]
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(const_cast<long long *>(items + 4));
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < PF8_KST; ++i) {
      mbar_init(&k_full[i], PF8_QUARTERS);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < PF8_VST; ++i) {
      mbar_init(&v_full[i], PF8_QUARTERS);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_done[i], 1);
    }
    mbar_init(drained, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], PF8_ITEM_READERS);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 10) {
    tc::alloc(tmem_slot, PF_TMEM_COLS);
    tc::relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const unsigned long long limit = a.wait_limit_ns;
  // The k-th item the first loader handed out (-1: none left), for one warp or one lane.
  auto take_item = [&](int k, bool whole_warp, long long *idx) -> bool {
    const int slot = k & 3;
    const bool ok = whole_warp ? warp_wait(&item_full[slot], (uint32_t)((k >> 2) & 1), limit)
                               : mbar_wait_bounded(&item_full[slot], (uint32_t)((k >> 2) & 1), limit);
    *idx = items[slot];
    if (whole_warp) __syncwarp();
    if (!whole_warp || lane == 0) mbar_arrive(&item_empty[slot]);
    return ok;
  };

  // One instruction per warpgroup (8-11 and 12-15 give, 0-3 and 4-7 take), all of its warps together.
  if (warp >= 8) {
    give_registers<PF8_OTHER_REGS>();
    if (warp != 10) {
      // ------------------------------------------------------------ loaders (warp 8 also takes the items and loads Q)
      const int w = warp > 10 ? warp - 9 : warp - 8;
      if (w == 0 && lane == 0) prefetch_tensor_map(&tmap_q);
      long long g = 0;  // K/V tiles of the items before
      int n_items = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        long long item;
        PrefillItem it;
        if (w == 0) {
          // the next item with work; items whose rows, context or pages are invalid are settled here
          const int slot = k & 3;
          if (k >= 4 && !(ok = warp_wait(&item_empty[slot], (uint32_t)(((k >> 2) - 1) & 1), limit))) break;
          for (;;) {
            unsigned int t = 0;
            if (lane == 0) t = atomicAdd(a.queue, 1u);
            item = (long long)__shfl_sync(FULL, t, 0);
            if (item >= a.num_items) {
              item = -1;
              break;
            }
            it = prefill_item(a, item);
            if (!dcheck(it.s < a.num_seqs && it.hq < a.num_q_heads)) continue;
            if (it.past_grid && it.t0 == 0 && it.hq == 0 && lane == 0) atomicOr(&g_status, PA_DEV_ERR_CONTEXT_HINT);
            bool zero = it.bad_ctx;
            if (it.work) {
              const int pages = (it.kmax + a.block_size - 1) / a.block_size;
              const int32_t *row = a.block_tables + (long long)it.s * a.table_stride;
              bool bad = false;
#pragma unroll 4
              for (int p = lane; p < pages; p += 32) {
                const int blk = __ldg(row + p);
                bad |= blk < 0 || (long long)blk >= a.num_blocks;
              }
              zero = __any_sync(FULL, bad);
              if (!zero) break;
            } else if (!zero && lane == 0) {
              // no rows of this sequence at this query tile (or no valid rows at all): the same holds for the
              // sequence's remaining heads, which are the next items; move the counter past them
              atomicMax(a.queue, (unsigned int)(item + a.num_q_heads - it.hq));
              if (it.bad_rows) atomicOr(&g_status, PA_DEV_ERR_CONTEXT);
            }
            if (zero) {  // zero the item's rows
              if (lane == 0) atomicOr(&g_status, it.bad_ctx ? PA_DEV_ERR_CONTEXT : PA_DEV_ERR_BLOCK_ID);
              for (int r = lane; r < it.rows; r += 32) {
                if (!dcheck((long long)it.q0 + it.t0 + r < a.num_query_tokens)) break;
                uint4 *dst = reinterpret_cast<uint4 *>(a.out + (long long)(it.q0 + it.t0 + r) * a.out_token_stride +
                                                       (long long)it.hq * D);
#pragma unroll
                for (int c = 0; c < D / 8; ++c) dst[c] = make_uint4(0, 0, 0, 0);
              }
            }
          }
          if (lane == 0) {
            items[slot] = item;
            mbar_arrive(&item_full[slot]);  // release: the item index is visible to the readers
          }
          if (item < 0) break;
          if (n_items >= 1 && !(ok = warp_wait(q_empty, (uint32_t)((n_items - 1) & 1), limit))) break;
          if (lane == 0) mbar_arrive_expect_tx(q_full, 2 * PF_BM * D * 2);
          __syncwarp();
          if (lane < 2 * HALVES) {  // lane = sub-tile * HALVES + half
            const int x = lane / HALVES, hh = lane % HALVES;
            tc::tma_load_3d(sm + L::Q + lane * REGION, &tmap_q, hh * 64, it.hq, it.q0 + it.t0 + x * PF_BM, q_full);
          }
        } else {
          if (!(ok = take_item(k, true, &item))) break;
          if (item < 0) break;
          it = prefill_item(a, item);
        }
        // The item's units: per key tile four of K, then four of V; unit number modulo PF8_LOADERS names the warp.
        const int32_t *row = a.block_tables + (long long)it.s * a.table_stride;
        const int pages = (it.kmax + a.block_size - 1) / a.block_size;
        int win = -1, ent = -1, ent_next = -1;  // 32 table entries from page 32 win on, and the 32 after them
        auto entries = [&](int wi) {
          return wi * 32 + lane < pages && dcheck(pages <= a.table_stride) ? __ldg(row + wi * 32 + lane) : -1;
        };
        auto load = [&](int u, LoadUnit<E, D> &x) {
          const int tok0 = (u >> 3) * PF_BN + (u & 3) * 32;
          const int page = tok0 / a.block_size, wi = page >> 5;
          if (wi != win) {
            ent = wi == win + 1 && win >= 0 ? ent_next : entries(wi);
            win = wi;
            ent_next = entries(wi + 1);
          }
          const int p0 = __shfl_sync(FULL, ent, page & 31);
          const int p1 = a.block_size == 16 ? __shfl_sync(FULL, ent, (page + 1) & 31) : p0;
          const bool is_v = (u >> 2) & 1;
          x.load(is_v ? args.v_cache : args.k_cache, is_v ? args.v_scale : args.k_scale, a, it.h, p0, p1, tok0, it.kmax,
                 lane);
        };
        const int units = it.nt * 8;
        const int u0 = (int)((w + PF8_LOADERS - (g * 8) % PF8_LOADERS) % PF8_LOADERS);
        LoadUnit<E, D> x;
        for (int u = u0; u < units; u += PF8_LOADERS) {
          load(u, x);  // in flight while the slot is waited for
          const long long t = g + (u >> 3);
          const bool is_v = (u >> 2) & 1;
          const int nst = is_v ? PF8_VST : PF8_KST;
          const int st = (int)(t % nst);
          if (t >= nst && !(ok = warp_wait(&(is_v ? v_empty : k_empty)[st], (uint32_t)(((t / nst) - 1) & 1), limit))) break;
          if (__any_sync(FULL, *abort_flag != 0)) {
            ok = false;
            break;
          }
          x.store(sm + (is_v ? L::V : L::K) + st * HALVES * REGION, (u & 3) * 32, is_v ? 1.f : args.k_sign, lane);
          fence_proxy_async_smem();  // the tensor cores read the rows through the async proxy
          __syncwarp();
          if (lane == 0) mbar_arrive(&(is_v ? v_full : k_full)[st]);
        }
        g += it.nt;
        ++n_items;
      }
      if (!ok && lane == 0) {
        *abort_flag = 1;
        atomicOr(&g_status, PA_DEV_ERR_TIMEOUT);
      }
      // Q's copies have landed before the CTA's smem is given back
      if (w == 0 && n_items > 0 && !warp_wait(q_full, (uint32_t)((n_items - 1) & 1), limit) && lane == 0)
        atomicOr(&g_status, PA_DEV_ERR_TIMEOUT);
    } else {
      // ------------------------------------------------------------ MMA issue (one lane)
      if (lane == 0) {
        constexpr uint32_t idesc_qk = tc::idesc_f16(kBf16, false, PF_BM, PF_BN);
        constexpr uint32_t idesc_pv = tc::idesc_f16(kBf16, true, PF_BM, D);
        const uint32_t qs = sbase + L::Q;
        long long g = 0;           // K/V tiles
        long long gx[2] = {0, 0};  // tiles of sub-tile A, B
        int n_items = 0;
        bool ok = true;
        // S_x = Q_x K(t)^T
        auto issue_qk = [&](int x, long long t) {
          const uint32_t ks = sbase + L::K + (uint32_t)(t % PF8_KST) * HALVES * REGION;
          const uint32_t qx = qs + x * HALVES * REGION;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k / 4) * REGION + (k % 4) * 32;
            tc::mma_ss(tmem + L::T_S + x * 128, tc::desc_sw128(qx + off, 16, 1024), tc::desc_sw128(ks + off, 16, 1024),
                       idesc_qk, k > 0);
          }
          tc::commit(&s_full[x]);
        };
        // O_x += P_x V(t), once softmax_x has written P_x for its tile gx
        auto issue_pv = [&](int x, long long t, long long tx, bool first_of_item) -> bool {
          if (!mbar_wait_bounded(&p_full[x], (uint32_t)(tx & 1), limit)) return false;
          const int st = (int)(t % PF8_VST);
          if (!mbar_wait_bounded(&v_full[st], (uint32_t)((t / PF8_VST) & 1), limit)) return false;
          tc::fence_after_sync();
          const uint32_t vs = sbase + L::V + st * HALVES * REGION;
#pragma unroll
          for (int k = 0; k < PF_BN / 16; ++k)
            tc::mma_ts(tmem + L::T_O + x * D, tmem + L::T_S + x * 128 + k * 8,
                       tc::desc_sw128(vs + k * 16 * 128, REGION, 1024), idesc_pv, !first_of_item || k > 0);
          return true;
        };
        for (int k = 0; ok; ++k) {
          long long item;
          if (!(ok = take_item(k, false, &item))) break;
          if (item < 0) break;
          const PrefillItem it = prefill_item(a, item);
          if (!(ok = mbar_wait_bounded(q_full, (uint32_t)(n_items & 1), limit))) break;
          long long pend_t = -1, pend_tb = 0;  // PV_B due next: K/V tile and B's tile
          bool pend_first = false;
          for (int j = 0; j < it.nt; ++j, ++g) {
            if (*abort_flag) {
              ok = false;
              break;
            }
            const bool a_on = j < it.nt_a, b_on = it.has_b;
            if (!(ok = mbar_wait_bounded(&k_full[g % PF8_KST], (uint32_t)((g / PF8_KST) & 1), limit))) break;
            tc::fence_after_sync();
            if (a_on) issue_qk(0, g);
            if (pend_t >= 0) {
              if (!(ok = issue_pv(1, pend_t, pend_tb, pend_first))) break;
              tc::commit(&v_empty[pend_t % PF8_VST]);
              pend_t = -1;
            }
            if (b_on) issue_qk(1, g);
            tc::commit(&k_empty[g % PF8_KST]);
            if (j == it.nt - 1) tc::commit(q_empty);
            if (a_on) {
              if (!(ok = issue_pv(0, g, gx[0], j == 0))) break;
              if (j == it.nt_a - 1) tc::commit(&o_done[0]);
              if (!b_on) tc::commit(&v_empty[g % PF8_VST]);
              ++gx[0];
            }
            if (b_on) {
              pend_t = g;
              pend_tb = gx[1]++;
              pend_first = j == 0;
            }
          }
          if (ok && pend_t >= 0) {  // the item's last PV_B
            if ((ok = issue_pv(1, pend_t, pend_tb, pend_first))) {
              tc::commit(&v_empty[pend_t % PF8_VST]);
              tc::commit(&o_done[1]);
            }
          }
          ++n_items;
        }
        if (!ok) {
          *abort_flag = 1;
          atomicOr(&g_status, PA_DEV_ERR_TIMEOUT);
        }
        // Every MMA issued has finished before tensor memory and smem are released.
        tc::commit(drained);
        if (!mbar_wait_bounded(drained, 0, limit)) atomicOr(&g_status, PA_DEV_ERR_TIMEOUT);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax and epilogue of sub-tile x (warps 0-3: A, 4-7: B)
    take_registers<PF8_SOFTMAX_REGS>();
    const int x = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + L::T_S + x * 128, t_o = tmem + lanes + L::T_O + x * D;
    long long gx = 0;  // this sub-tile's tiles
    int nx_items = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      long long item;
      if (!(ok = take_item(k, true, &item))) break;
      if (item < 0) break;
      const PrefillItem it = prefill_item(a, item);
      const int ntx = x == 0 ? it.nt_a : (it.has_b ? it.nt : 0);
      // last key this row sees; rows past the item's tokens stop at kmax - 1 too, so that no row
      // reads a page the producers did not load
      const int pos0 = it.pos0 + x * PF_BM;
      const int vis = min(pos0 + r, it.kmax - 1);
      const int vis_min = min(pos0, it.kmax - 1);
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < ntx; ++j, ++gx) {
        if (__any_sync(FULL, *abort_flag != 0)) {
          ok = false;
          break;
        }
        // S_x(j) is in tensor memory, and every earlier MMA (PV_x of the previous tile) is done
        if (!(ok = warp_wait(&s_full[x], (uint32_t)(gx & 1), limit))) break;
        tc::fence_after_sync();
        const int key0 = j * PF_BN;
        const bool masked = key0 + PF_BN - 1 > vis_min;  // a tile on the diagonal or at the end (uniform)
        // the row of S_x: four loads, one wait
        float sv[PF_BN];
#pragma unroll
        for (int c = 0; c < PF_BN / 32; ++c) tc::ld32(t_s + c * 32, *reinterpret_cast<float(*)[32]>(&sv[c * 32]));
        tc::wait_ld();
        if (masked) {
#pragma unroll
          for (int c = 0; c < PF_BN; ++c)
            if (key0 + c > vis) sv[c] = -INFINITY;
        }
        // row max of the raw scores in four chains, two scores per three-input max (scale_log2 > 0 keeps the order)
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < PF_BN; c += 8)
#pragma unroll
          for (int u = 0; u < 4; ++u) mx4[u] = fmax3(mx4[u], sv[c + u], sv[c + 4 + u]);
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * a.scale_log2;
        const float m_new = fmaxf(m, mx);
        const bool need = m_new > m + RESCALE_SLACK;
        float factor = 1.f;
        if (need) {
          factor = ex2(m - m_new);
          m = m_new;
        }
        // p = 2^(s * scale_log2 - m) (0 where masked), rounded to the storage type (see the top), into P_x: the
        // first 64 columns of S_x, whose scores are all in registers by now.
        float sum4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < PF_BN / 32; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            // masked scores are -inf: 2^-inf = 0
            // scale and shift two scores in one packed fma
            const float2 x = __ffma2_rn(make_float2(sv[c * 32 + 2 * i], sv[c * 32 + 2 * i + 1]),
                                        make_float2(a.scale_log2, a.scale_log2), make_float2(-m, -m));
            const float p0 = ex2(x.x);
            const float p1 = ex2(x.y);
            pk[i] = E::narrow2(p0, p1);
            sum4[i & 3] = add_packed<E>(pk[i], sum4[i & 3]);
          }
          tc::st16(t_s + c * 16, pk);
        }
        const float rowsum = (sum4[0] + sum4[1]) + (sum4[2] + sum4[3]);
        if (j > 0 && __any_sync(FULL, need)) {  // O_x is settled: the previous PV_x is done
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tc::ld32(t_o + c * 32, o);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= factor;
            tc::st32(t_o + c * 32, o);
          }
        }
        tc::wait_st();
        l = l * factor + rowsum;
        tc::fence_before_sync();
        mbar_arrive(&p_full[x]);
      }
      if (!ok) break;
      if (ntx == 0) continue;
      // epilogue: O_x after the item's last PV_x, normalised
      if (!(ok = warp_wait(&o_done[x], (uint32_t)(nx_items & 1), limit))) break;
      tc::fence_after_sync();
      const int row = x * PF_BM + r;
      uint16_t *dst = a.out + (long long)(it.q0 + it.t0 + row) * a.out_token_stride + (long long)it.hq * D;
      const float inv = 1.f / l;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        float o[32];
        tc::ld32(t_o + c * 32, o);  // every lane: the load is warp-collective
        tc::wait_ld();
        if (row < it.rows && dcheck((long long)it.q0 + it.t0 + row < a.num_query_tokens)) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = o[i * 8 + e] * inv;
            *reinterpret_cast<uint4 *>(dst + c * 32 + i * 8) = narrow8<E>(f);
          }
        }
      }
      tc::fence_before_sync();
      ++nx_items;
    }
    if (!ok) {
      *abort_flag = 1;
      if (lane == 0) atomicOr(&g_status, PA_DEV_ERR_TIMEOUT);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 10) {
    __syncwarp();
    tc::fence_after_sync();
    tc::dealloc(tmem, PF_TMEM_COLS);
  }
}

}  // namespace pa

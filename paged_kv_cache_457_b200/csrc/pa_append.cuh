// Appending a step's keys and values to the paged cache with the position
// rotation applied on the way, into 16-bit caches and into caches held in 8
// bits (e4m3) with one scale for each (block, kv head).
//
// Rotation of a row x of token t, position p = positions[t], over its first
// r = rot_dim dims; pairs (x_i, x_{i + r/2}) (halves) or (x_{2i}, x_{2i+1})
// (interleaved), i < r / 2, with c = cos_sin[p][i], s = cos_sin[p][r/2 + i]:
//   x_a' = x_a c - x_b s,   x_b' = x_b c + x_a s,
// in fp32, products and sums rounded separately (no contraction, so the
// result is the one that elementary fp32 operations give, bit for bit).
//
// rope_write_kv_kernel      16-bit caches: q' out, k' and v to their slots.
// append_fp8_kernel         8-bit caches: k' and v quantised to their slots,
//                           q' out in the same launch (later blocks) for short
//                           inputs, by rope_write_kv_kernel for long ones.
//
// A unit of work of a row is 16 elements: two 16-byte chunks that hold both
// members of 8 pairs, with their 8 cosines and 8 sines.
#pragma once

#include <cstdint>
#include <type_traits>

#include "pa_kernels.cuh"

namespace pa {

struct AppendArgs {
  const uint16_t *q, *k, *v;
  uint16_t *q_out;
  void *k_cache, *v_cache;    // 2-byte elements, or e4m3 bytes
  float *k_scale, *v_scale;   // [num_blocks][num_kv_heads], 8-bit caches only
  const int64_t *slot_mapping, *positions;
  const float *cos_sin;       // [max_positions][rot_dim]: cosines, then sines
  long long num_tokens, num_blocks, max_positions;
  long long q_stride, k_stride, v_stride, q_out_stride;
  long long kv_blocks;        // append_fp8_kernel: grid blocks of the K/V part
  int num_q_heads, num_kv_heads, block_size, rot_dim;
  int rows;                   // rope_write_kv_kernel: rows of a token it handles (q heads alone, or all)
  int tokens_per_cta;         // row part: consecutive tokens of one block of threads
  int tokens_per_warp;        // append_fp8_kernel: consecutive tokens of one warp (1 or block_size)
  int heads_per_warp;         // append_fp8_kernel: (kv head, K or V) pairs of one warp
};

// ---------------------------------------------------------------- e4m3
// Two fp32 values to packed e4m3 (lo in the low byte), nearest even, saturating at +-448; NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
// Two packed e4m3 values to packed fp16 (exact: e4m3's values are fp16 values).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t x) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(x));
  return d;
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t x) {
  const uint32_t h = e4m3x2_to_f16x2(x);
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// The smallest power of two s in [2^-64, 2^120] with amax <= 448 s (amax finite, >= 0).  448 = 1.75 * 2^8:
// with amax = m 2^x, s = 2^(x - 8) while m <= 1.75, else 2^(x - 7).  Powers of two because scaling by one is
// exact: x / s has x's bits, so a value is rounded once, to e4m3, and bytes re-scaled when a later row of the
// block needs a larger s keep their bits unless they leave e4m3's normal range.  The price is at most one bit of
// e4m3's 17-binade range, none of its precision.
__device__ __forceinline__ float pow2_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, -64);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// ---------------------------------------------------------------- rotation
// The 16-byte chunks (8 elements each) of unit c of a row, and whether the unit is rotated.
struct Unit {
  int c0, c1;
  bool rotated;
};
template <bool INTERLEAVED>
__device__ __forceinline__ Unit unit_of(int c, int rot_dim) {
  const int ru = rot_dim / 16;
  if (INTERLEAVED) return Unit{2 * c, 2 * c + 1, c < ru};
  return c < ru ? Unit{c, c + ru, true} : Unit{2 * c, 2 * c + 1, false};
}

struct Angles {
  float c[8], s[8];
};
// Cosines and sines of a rotated unit c at position p (rows of rot_dim floats, rot_dim a multiple of 16).
__device__ __forceinline__ Angles load_angles(const AppendArgs &a, long long p, int c) {
  Angles g;
  const float4 *cs = reinterpret_cast<const float4 *>(a.cos_sin + p * a.rot_dim + 8 * c);
  const float4 *sn = reinterpret_cast<const float4 *>(a.cos_sin + p * a.rot_dim + a.rot_dim / 2 + 8 * c);
  const float4 c0 = __ldg(cs), c1 = __ldg(cs + 1), s0 = __ldg(sn), s1 = __ldg(sn + 1);
  g.c[0] = c0.x, g.c[1] = c0.y, g.c[2] = c0.z, g.c[3] = c0.w;
  g.c[4] = c1.x, g.c[5] = c1.y, g.c[6] = c1.z, g.c[7] = c1.w;
  g.s[0] = s0.x, g.s[1] = s0.y, g.s[2] = s0.z, g.s[3] = s0.w;
  g.s[4] = s1.x, g.s[5] = s1.y, g.s[6] = s1.z, g.s[7] = s1.w;
  return g;
}

// Packed fp32 products.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\t"
      "mov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Turns the unit's 16 elements (chunks lo and hi) in place.
template <bool INTERLEAVED>
__device__ __forceinline__ void turn(float (&lo)[8], float (&hi)[8], const Angles &g) {
  // Pairs i and i + 1 at once: packed products, scalar sums -- a packed product followed by a packed sum is contracted
  // into a fused one, whatever their rounding suffix.
  auto two = [&](float &x0, float &y0, float &x1, float &y1, int i) {
    const float2 x = make_float2(x0, x1), y = make_float2(y0, y1);
    const float2 c = make_float2(g.c[i], g.c[i + 1]), s = make_float2(g.s[i], g.s[i + 1]);
    const float2 xc = mul2(x, c), ys = mul2(y, s), yc = mul2(y, c), xs = mul2(x, s);
    x0 = __fsub_rn(xc.x, ys.x), x1 = __fsub_rn(xc.y, ys.y);
    y0 = __fadd_rn(yc.x, xs.x), y1 = __fadd_rn(yc.y, xs.y);
  };
  if (INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      two(lo[2 * i], lo[2 * i + 1], lo[2 * i + 2], lo[2 * i + 3], i);
      two(hi[2 * i], hi[2 * i + 1], hi[2 * i + 2], hi[2 * i + 3], 4 + i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i += 2) two(lo[i], hi[i], lo[i + 1], hi[i + 1], i);
  }
}

// ---------------------------------------------------------------- 16-bit rows
// One item: unit c of NR rows of token t, r0, r0 + apart, ... (rows: q heads, then k heads, then v heads).  The rows
// share the angles and keep 2 NR 16-byte loads in flight.  q_out may be q itself: a thread reads the two chunks of a
// row that it alone writes, before it writes them.
template <class E, int D, bool INTERLEAVED, int NR>
__device__ __forceinline__ void append_rows(const AppendArgs &a, long long t, int r0, int apart, int rows, int c) {
  const long long pos = a.positions[t];
  if (pos < 0) return;  // padding: nothing of the token is touched
  const bool pos_ok = pos < a.max_positions;
  const bool kv = rows > a.num_q_heads;  // this launch stores K and V too
  const long long slot = kv ? a.slot_mapping[t] : -1;
  const bool slot_ok = slot >= 0 && slot < a.num_blocks * a.block_size;
  if (r0 == 0 && c == 0) {
    if (!pos_ok) atomicOr(&g_status, PA_DEV_ERR_POSITION);
    if (slot >= 0 && !slot_ok) atomicOr(&g_status, PA_DEV_ERR_SLOT);
  }
  const Unit u = unit_of<INTERLEAVED>(c, a.rot_dim);
  const long long blk = slot_ok ? slot / a.block_size : 0;
  const int row = slot_ok ? (int)(slot - blk * a.block_size) : 0;
  uint16_t *dst[NR];
  uint4 w[NR][2];
  // chunks of row r: a V row keeps its own in order
  auto chunks = [&](int r) {
    const bool v = r >= a.num_q_heads + a.num_kv_heads;
    return make_int2(v ? 2 * c : u.c0, v ? 2 * c + 1 : u.c1);
  };
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int r = r0 + i * apart;
    const int hk = r - a.num_q_heads, hv = hk - a.num_kv_heads;
    const uint16_t *src = nullptr;
    dst[i] = nullptr;
    if (r < rows) {
      if (hk < 0) {
        src = a.q + t * a.q_stride + (long long)r * D;
        dst[i] = a.q_out + t * a.q_out_stride + (long long)r * D;
      } else if (slot_ok && pos_ok && dcheck(blk < a.num_blocks && row < a.block_size && hv < a.num_kv_heads)) {
        const int h = hv < 0 ? hk : hv;
        src = (hv < 0 ? a.k + t * a.k_stride : a.v + t * a.v_stride) + (long long)h * D;
        dst[i] = static_cast<uint16_t *>(hv < 0 ? a.k_cache : a.v_cache) +
                 ((blk * a.num_kv_heads + h) * a.block_size + row) * D;
      }
    }
    if (src) {
      const int2 cc = chunks(r);
      w[i][0] = *reinterpret_cast<const uint4 *>(src + cc.x * 8);
      w[i][1] = *reinterpret_cast<const uint4 *>(src + cc.y * 8);
    }
  }
  Angles g;
  if (u.rotated && pos_ok) g = load_angles(a, pos, c);
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    if (!dst[i]) continue;
    const int r = r0 + i * apart;
    if (u.rotated && pos_ok && r < a.num_q_heads + a.num_kv_heads) {
      float lo[8], hi[8];
      E::widen8(w[i][0], lo);
      E::widen8(w[i][1], hi);
      turn<INTERLEAVED>(lo, hi, g);
      w[i][0] = narrow8<E>(lo);
      w[i][1] = narrow8<E>(hi);
    }
    if (!pos_ok) w[i][0] = w[i][1] = make_uint4(0, 0, 0, 0);  // only q rows get here: zeros for a bad position
    const int2 cc = chunks(r);
    *reinterpret_cast<uint4 *>(dst[i] + cc.x * 8) = w[i][0];
    *reinterpret_cast<uint4 *>(dst[i] + cc.y * 8) = w[i][1];
  }
}

// The row part of a launch: grid block b takes tokens b * tokens_per_cta .. of the first `rows` rows.
template <class E, int D, bool INTERLEAVED>
__device__ __forceinline__ void append_row_block(const AppendArgs &a, long long b, int rows) {
  constexpr int UNITS = D / 16;
  const long long t0 = b * a.tokens_per_cta;
  const int nt = (int)min((long long)a.tokens_per_cta, a.num_tokens - t0);
  constexpr int NR = 2;
  const int apart = (rows + NR - 1) / NR;
  const int per = apart * UNITS;
  for (int i = threadIdx.x; i < nt * per; i += blockDim.x) {
    const int t = i / per, rem = i - t * per;
    append_rows<E, D, INTERLEAVED, NR>(a, t0 + t, rem / UNITS, apart, rows, rem % UNITS);
  }
}

constexpr int ROW_THREADS = 256;

// Bound by HBM: 16384 tokens of 32 q and 8 kv heads (411 MB) take 70.4 us, 0.89 of the measured copy rate, with four
// blocks on an SM (64 registers); 79 with three, 119 with five (spills), 89 with four rows per thread.
template <class E, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(ROW_THREADS, 4) rope_write_kv_kernel(const AppendArgs a) {
  grid_dependency_wait();  // the rows may come from the previous kernel in the stream
  grid_launch_dependents();
  append_row_block<E, D, INTERLEAVED>(a, blockIdx.x, a.rows);
}

// ---------------------------------------------------------------- 8-bit rows
// A run is a stretch of tokens whose slots lie in one block, whatever skipped tokens stand between them; one warp
// handles a run for one kv head of K or of V, so a block's scale has one writer and no atomics are needed.  With x'
// the run's rows (rotated K in fp32, V as is):
//   amax  = largest finite |x'|,
//   s_new = pow2_scale(amax) if the run holds the block's row 0 (the block starts anew), else
//           max(s_old, pow2_scale(amax)); where s_new > s_old the block's bytes become rn(byte * s_old / s_new),
//   bytes = rn_sat(x' / s_new) to the run's rows.
// Rows are read in windows of BS tokens by 16-byte asynchronous copies into shared memory, from where each lane reads
// back what it copied, once for the magnitude and once for the bytes, and a warp's next head is on its way while it
// works on this one.  A run is one window unless skipped tokens or a slot named twice stretch it, and only then are
// rows fetched twice.
// Bound by latency at 16 warps on an SM, not by HBM (16 prompts of a 32-head model: K/V part about 120 us for 381 MB,
// 0.48 of the copy rate).  Measured on that case, the whole call: 164 us; 277 with rows in registers, one head per warp
// and the neighbours looked up in turn; 173 with rows in registers; 210, 186, 165 and 179 with 1, 2, 8 and 16 heads per
// warp; 201 with the rotated values kept in fp32 for the second step (they spill, or leave 12 warps); 170 to 185 with
// 20 or 24 warps.

// Token t of the call: its block (-1: not written), row in the block and position.  `flags`: set the status bits.
template <int BS, bool ROPE>
__device__ __forceinline__ int append_token(const AppendArgs &a, long long t, bool flags, int &row, long long &pos) {
  row = -1;
  pos = 0;
  if (t < 0 || t >= a.num_tokens) return -1;
  const long long slot = __ldg(reinterpret_cast<const long long *>(a.slot_mapping) + t);
  if (ROPE) pos = __ldg(reinterpret_cast<const long long *>(a.positions) + t);
  if (pos < 0) return -1;  // padding
  const bool slot_high = slot >= a.num_blocks * BS, pos_high = ROPE && pos >= a.max_positions;
  if (flags && slot_high) atomicOr(&g_status, PA_DEV_ERR_SLOT);
  if (flags && pos_high) atomicOr(&g_status, PA_DEV_ERR_POSITION);
  if (slot < 0 || slot_high || pos_high) return -1;
  row = (int)(slot % BS);
  return (int)(slot / BS);  // num_blocks is at most 2^31 - 1
}

// The largest of |f[i]| and m; NaN counts as nothing.
__device__ __forceinline__ float amax8(const float (&f)[8], float m) {
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    asm("{\n\t.reg .f32 x, y;\n\tabs.f32 x, %1;\n\tabs.f32 y, %2;\n\tmax.f32 %0, x, y, %3;\n\t}"
        : "=f"(m)
        : "f"(f[i]), "f"(f[i + 1]), "f"(m));
  return m;
}

// 16-byte asynchronous copy global -> shared (zeros when !ok), past L1; a thread's copies and its wait for all but the
// last N groups of them.
__device__ __forceinline__ void cp_async16(void *dst, const void *src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(ok ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <class E, int D, int BS, bool INTERLEAVED, bool ROPE>
struct RunWindow {
  static constexpr int LPR = D / 16;    // lanes (units) of a row
  static constexpr int RPI = 32 / LPR;  // rows of one pass of the warp
  static constexpr int PASSES = BS / RPI;
  static constexpr int ROWS = BS;
  static constexpr uint32_t BYTES = BS * D * 2;  // one buffer: [pass][chunk][lane] pieces of 16 bytes
  int my_row;        // lane i: row of the window's token i in the block, -1: none of the run's
  int my_pos;        // its position (below max_positions, at most 2^31 - 1)
  unsigned live;     // lanes with such a row

  // Tokens ts .. ts + ROWS - 1 of the run [ts, te) of block blk.
  __device__ __forceinline__ void tokens(const AppendArgs &a, long long ts, long long te, int blk, int lane) {
    long long pos;
    const int b = append_token<BS, ROPE>(a, lane < ROWS && ts + lane < te ? ts + lane : -1, false, my_row, pos);
    my_pos = (int)pos;
    if (b != blk) my_row = -1;
    live = __ballot_sync(FULL, my_row >= 0);
  }
  // Starts the copies of the window's rows from `base` (token ts, this head) into `buf`, dead rows as zeros.
  __device__ __forceinline__ void fetch(uint8_t *buf, const uint16_t *base, long long stride, const Unit &u,
                                        int lane) const {
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int r = p * RPI + lane / LPR;
      const bool ok = (live >> r) & 1u;
      const uint16_t *src = ok ? base + r * stride : base;
      cp_async16(buf + (2 * p) * 512 + lane * 16, src + u.c0 * 8, ok);
      cp_async16(buf + (2 * p + 1) * 512 + lane * 16, src + u.c1 * 8, ok);
    }
    cp_async_commit();
  }
  // This lane's 16 values of pass p in fp32, rotated when `turned` (the angles come from L1 the second time).
  __device__ __forceinline__ void values(const AppendArgs &a, const uint8_t *buf, int p, const Unit &u, bool turned,
                                         int lane, float (&lo)[8], float (&hi)[8]) const {
    E::widen8(*reinterpret_cast<const uint4 *>(buf + (2 * p) * 512 + lane * 16), lo);
    E::widen8(*reinterpret_cast<const uint4 *>(buf + (2 * p + 1) * 512 + lane * 16), hi);
    if (turned) {
      const int r = p * RPI + lane / LPR;
      const int pos = __shfl_sync(FULL, my_pos, r);
      if (u.rotated && ((live >> r) & 1u)) turn<INTERLEAVED>(lo, hi, load_angles(a, pos, lane % LPR));
    }
  }
  // Largest finite magnitude of this lane's values.
  __device__ __forceinline__ float amax(const AppendArgs &a, const uint8_t *buf, const Unit &u, bool turned,
                                        int lane) const {
    float m = 0.f;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      if ((live >> (p * RPI)) == 0) break;
      float lo[8], hi[8];
      values(a, buf, p, u, turned, lane, lo, hi);
      const float all = amax8(hi, amax8(lo, 0.f));
      if (all < INFINITY) {
        m = fmaxf(m, all);
      } else {  // infinite values do not count
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = fabsf(lo[i]), y = fabsf(hi[i]);
          m = fmaxf(m, fmaxf(x < INFINITY ? x : 0.f, y < INFINITY ? y : 0.f));
        }
      }
    }
    return m;
  }
  __device__ __forceinline__ void store(const AppendArgs &a, const uint8_t *buf, uint8_t *slab, const Unit &u,
                                        bool turned, float s, int lane) const {
    // x / s: by the exact reciprocal where s is a power of two (always, unless the caller's own scale stands)
    const bool pow2 = (__float_as_uint(s) & 0x7fffffu) == 0;
    const float inv = __fdiv_rn(1.f, s);
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      if ((live >> (p * RPI)) == 0) break;
      float lo[8], hi[8];
      values(a, buf, p, u, turned, lane, lo, hi);
      const int row = __shfl_sync(FULL, my_row, p * RPI + lane / LPR);
      if (pow2) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float2 x = mul2(make_float2(lo[i], lo[i + 1]), make_float2(inv, inv));
          const float2 y = mul2(make_float2(hi[i], hi[i + 1]), make_float2(inv, inv));
          lo[i] = x.x, lo[i + 1] = x.y, hi[i] = y.x, hi[i + 1] = y.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          lo[i] = __fdiv_rn(lo[i], s);
          hi[i] = __fdiv_rn(hi[i], s);
        }
      }
      uint2 b0, b1;
      b0.x = to_e4m3x2(lo[0], lo[1]) | (to_e4m3x2(lo[2], lo[3]) << 16);
      b0.y = to_e4m3x2(lo[4], lo[5]) | (to_e4m3x2(lo[6], lo[7]) << 16);
      b1.x = to_e4m3x2(hi[0], hi[1]) | (to_e4m3x2(hi[2], hi[3]) << 16);
      b1.y = to_e4m3x2(hi[4], hi[5]) | (to_e4m3x2(hi[6], hi[7]) << 16);
      if (row >= 0 && dcheck(row < BS)) {
        *reinterpret_cast<uint2 *>(slab + row * D + u.c0 * 8) = b0;
        *reinterpret_cast<uint2 *>(slab + row * D + u.c1 * 8) = b1;
      }
    }
  }
};

// Rows of earlier calls in units of a larger scale: bytes b become rn(b * ratio).
template <int BYTES>
__device__ __forceinline__ void rescale_slab(uint8_t *slab, float ratio, int lane) {
  const float2 r2 = make_float2(ratio, ratio);
  uint4 *b = reinterpret_cast<uint4 *>(slab) + lane;
  uint4 x[BYTES / 512];
#pragma unroll
  for (int i = 0; i < BYTES / 512; ++i) x[i] = b[i * 32];
#pragma unroll
  for (int i = 0; i < BYTES / 512; ++i) {
    const uint32_t in[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f0 = __fmul2_rn(e4m3x2_to_float2((uint16_t)in[j]), r2);
      const float2 f1 = __fmul2_rn(e4m3x2_to_float2((uint16_t)(in[j] >> 16)), r2);
      out[j] = to_e4m3x2(f0.x, f0.y) | (to_e4m3x2(f1.x, f1.y) << 16);
    }
    b[i * 32] = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

// One kv head of K or of V of a run that starts at token ts in block blk.
template <class E, int D, int BS>
struct RunHead {
  const uint16_t *base;
  long long stride;
  float *scale;
  uint8_t *slab;
  Unit u;
  bool turned;
  float s_old;
  template <bool INTERLEAVED, bool ROPE>
  __device__ __forceinline__ void set(const AppendArgs &a, int hw, long long ts, int blk, int lane) {
    const bool is_v = hw >= a.num_kv_heads;
    const int h = is_v ? hw - a.num_kv_heads : hw;
    const int c = lane % (D / 16);
    turned = ROPE && !is_v;
    u = turned ? unit_of<INTERLEAVED>(c, a.rot_dim) : Unit{2 * c, 2 * c + 1, false};
    stride = is_v ? a.v_stride : a.k_stride;
    base = (is_v ? a.v : a.k) + ts * stride + (long long)h * D;
    const long long head = (long long)blk * a.num_kv_heads + h;
    scale = (is_v ? a.v_scale : a.k_scale) + head;
    slab = static_cast<uint8_t *>(is_v ? a.v_cache : a.k_cache) + head * BS * D;
    s_old = *scale;
  }
};

constexpr int APPEND_WARPS = 4;

// Dynamic shared memory of append_fp8_kernel: two windows per warp.
__host__ __device__ constexpr uint32_t append_smem(int head_dim, int block_size) {
  return APPEND_WARPS * 2u * (uint32_t)(block_size * head_dim * 2);
}

// K/V part: warp w of the part takes tokens [i * tokens_per_warp, +tokens_per_warp) of heads_per_warp (kv head, K or
// V) pairs, and the runs that START among them (a run's later tokens may lie in the next warps' stretches, which then
// leave them alone).  With Q, grid blocks from kv_blocks on take the q heads' rows: one launch for a decode step.
template <class E, int D, int BS, bool INTERLEAVED, bool ROPE, bool Q>
__global__ void __launch_bounds__(APPEND_WARPS * 32, 4) append_fp8_kernel(const AppendArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  if (Q && (long long)blockIdx.x >= a.kv_blocks) {
    append_row_block<E, D, INTERLEAVED>(a, (long long)blockIdx.x - a.kv_blocks, a.num_q_heads);
    return;
  }
  using Window = RunWindow<E, D, BS, INTERLEAVED, ROPE>;
  extern __shared__ __align__(16) uint8_t append_buf[];
  uint8_t *buf = append_buf + (threadIdx.x >> 5) * 2 * Window::BYTES;
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int pairs = 2 * a.num_kv_heads;
  const int per = (pairs + a.heads_per_warp - 1) / a.heads_per_warp;  // warps of a stretch
  const long long t0 = (w / per) * a.tokens_per_warp;
  if (t0 >= a.num_tokens) return;
  const int hw0 = (int)(w % per);
  // The stretch and its neighbours in one load: lane i holds token tb + i, the stretch is lanes [lead, lead + its
  // length).  Most runs are settled by what the lanes hold; the loops below are for longer ones.
  const int lead = (32 - a.tokens_per_warp) / 2;
  const long long tb = t0 - lead;
  int row;
  long long pos;
  const bool inside = lane >= lead && lane < lead + a.tokens_per_warp;
  const int blk_l = append_token<BS, ROPE>(a, tb + lane, hw0 == 0 && inside, row, pos);
  const unsigned written = __ballot_sync(FULL, blk_l >= 0);
  const unsigned stretch = __ballot_sync(FULL, inside && blk_l >= 0);
  if (!stretch) return;
  // block of the last written token before the lanes' first, where the stretch's first written token needs it
  int before = -1;
  if ((written & ((1u << (__ffs(stretch) - 1)) - 1u)) == 0) {
    for (long long t = tb - 1; t >= 0; t -= 32) {
      int r;
      long long p;
      const int b = append_token<BS, ROPE>(a, t - lane, false, r, p);
      const unsigned m = __ballot_sync(FULL, b >= 0);
      if (m) {
        before = __shfl_sync(FULL, b, __ffs(m) - 1);
        break;
      }
    }
  }
  // a written token starts a run where the written token before it lies in another block
  const unsigned below = written & ((1u << lane) - 1u);
  const int prev = __shfl_sync(FULL, blk_l, below ? 31 - __clz(below) : 0);
  unsigned heads = __ballot_sync(FULL, inside && blk_l >= 0 && blk_l != (below ? prev : before));
  while (heads) {
    const int i = __ffs(heads) - 1;
    heads &= heads - 1;
    const int blk = __shfl_sync(FULL, blk_l, i);
    const long long ts = tb + i;
    // the run ends before the next written token of another block; `te` is one past its last token
    unsigned other = __ballot_sync(FULL, lane > i && blk_l >= 0 && blk_l != blk);
    unsigned same = __ballot_sync(FULL, lane >= i && blk_l == blk);
    if (other) same &= (other & (0u - other)) - 1u;  // those before the first of another block
    long long te = tb + 32 - __clz(same);
    const bool settled = other != 0;
    bool fresh = __any_sync(FULL, ((same >> lane) & 1u) && row == 0);
    if (!settled) {
      for (long long t = tb + 32; t < a.num_tokens; t += 32) {
        int r;
        long long p;
        const int b = append_token<BS, ROPE>(a, t + lane, false, r, p);
        other = __ballot_sync(FULL, b >= 0 && b != blk);
        same = __ballot_sync(FULL, b == blk);
        if (other) same &= (other & (0u - other)) - 1u;
        if (same) te = t + 32 - __clz(same);
        fresh |= __any_sync(FULL, ((same >> lane) & 1u) && r == 0);
        if (other) break;
      }
    }
    Window win;
    if (te - tb <= 32) {  // the first window's tokens are in the lanes
      const int src = i + lane;
      const int b = __shfl_sync(FULL, blk_l, src & 31), r = __shfl_sync(FULL, row, src & 31);
      win.my_pos = __shfl_sync(FULL, (int)pos, src & 31);
      win.my_row = lane < Window::ROWS && ts + lane < te && b == blk ? r : -1;
      win.live = __ballot_sync(FULL, win.my_row >= 0);
    } else {
      win.tokens(a, ts, te, blk, lane);
    }
    if (!dcheck(blk < a.num_blocks)) continue;
    const bool one = te - ts <= Window::ROWS;
    RunHead<E, D, BS> cur, next;
    cur.template set<INTERLEAVED, ROPE>(a, hw0, ts, blk, lane);
    win.fetch(buf, cur.base, cur.stride, cur.u, lane);
    int at = 0;  // buffer of the current head
    for (int hw = hw0; hw < pairs; hw += per) {
      uint8_t *b = buf + at * Window::BYTES;
      const bool more = one && hw + per < pairs;
      if (more) {  // the next head's rows, while this one is worked on
        next.template set<INTERLEAVED, ROPE>(a, hw + per, ts, blk, lane);
        win.fetch(buf + (at ^ 1) * Window::BYTES, next.base, next.stride, next.u, lane);
        cp_async_wait<1>();
      } else {
        cp_async_wait<0>();
      }
      float amax = win.amax(a, b, cur.u, cur.turned, lane);
      if (!one) {
        for (long long t = ts + Window::ROWS; t < te; t += Window::ROWS) {
          win.tokens(a, t, te, blk, lane);
          win.fetch(b, cur.base + (t - ts) * cur.stride, cur.stride, cur.u, lane);
          cp_async_wait<0>();
          amax = fmaxf(amax, win.amax(a, b, cur.u, cur.turned, lane));
        }
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, off));
      const float want = pow2_scale(amax);
      const float s_new = fresh ? want : fmaxf(cur.s_old, want);
      if (!fresh && s_new > cur.s_old) {
        rescale_slab<BS * D>(cur.slab, __fdiv_rn(cur.s_old, s_new), lane);
        __syncwarp();  // before the run's own rows are written over theirs
      }
      if (one) {
        win.store(a, b, cur.slab, cur.u, cur.turned, s_new, lane);
      } else {
        for (long long t = ts; t < te; t += Window::ROWS) {
          win.tokens(a, t, te, blk, lane);
          win.fetch(b, cur.base + (t - ts) * cur.stride, cur.stride, cur.u, lane);
          cp_async_wait<0>();
          win.store(a, b, cur.slab, cur.u, cur.turned, s_new, lane);
          __syncwarp();
        }
        win.tokens(a, ts, te, blk, lane);
        if (hw + per < pairs) {
          next.template set<INTERLEAVED, ROPE>(a, hw + per, ts, blk, lane);
          win.fetch(b, next.base, next.stride, next.u, lane);
        }
      }
      if (lane == 0) *cur.scale = s_new;
      cur = next;
      if (one) at ^= 1;
    }
  }
}

}  // namespace pa

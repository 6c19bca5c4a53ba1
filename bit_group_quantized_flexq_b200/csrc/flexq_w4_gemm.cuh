// flexq_w4_gemm.cuh -- 4-bit linear layers for batches beyond the streaming
// kernel's, on the tensor core's tcgen05 MMA.
//
// One CTA: RB blocks of 128 weight rows x T tokens over its share of the
// columns.  The weights are the MMA's A operand, in tensor memory: unpack warps
// turn a tile of 128 rows x 128 columns (8 KB of codes, one TMA box) into FP16
// or BF16 values and store them there; the activations are the B operand, in
// shared memory as TMA brings them; one FP32 accumulator of T columns per row
// block takes the whole share.  Two row blocks read each tile of activations
// once: with one, 128 tokens bring 32 KB from L2 for 512 cycles of MMA, more
// than an SM receives in them.  An unpacked weight is the rounded product of
// code and scale, half a step of the activations' type: keeping the codes whole
// and scaling each group's sum instead would read the accumulator back once per
// group, which costs a tile of 128 tokens more time than its MMAs, and a second
// MMA for the rounding's rest would take as long as the first.  The error of a
// result grows from that of its own rounding, 0.0017 in BF16 and 0.00021 in FP16
// of the result's root mean square, to 0.0023 and 0.00027.
//
// With fewer tiles than the machine has room for, a cluster of CTAs shares a
// tile's columns; each leaves its sums in its shared memory, and the CTAs add
// them up in the order of the columns, a share of the tokens each.
//
// Bound by unpacking: 13 instructions per word of eight codes in FP16, 19 in
// BF16, and about as many around them (waits, addresses, scales), at 0.65
// instructions per cycle and scheduler.  Measured (device time): 11008 x 4096 at
// 32 tokens 15.8 us, at 256 30.4 us (BF16 33.9), at 2048 152 us, 1215 TFLOP/s, in
// short runs and 176 us, 1050, in a long one that meets the power cap; 28672 x
// 8192 at 64 tokens 53 us.  A warp's time per tile does not fall with
// fewer warps beside it (tiles of 160 rows, which fill 138 SMs at 256 tokens
// where those of 256 fill 86: 31.5 and 33.8 us), nor with three slots of
// unpacked weights for two; leaving the wait for a tile's stores until the next
// one is unpacked took 36 us for 30.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "flexq_gemm.cuh"
#include "flexq_w4.cuh"

namespace flexq {

__device__ __forceinline__ void mma_f16_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                               uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %6, %7, %8}, "
      "p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(0u), "r"(0u),
      "r"(0u), "r"(0u)
      : "memory");
}

__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(x),
               "r"(y), "r"(z)
               : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// 16 lanes x 256 bits twice along the columns (16 columns): thread t gets lane
// t/4, columns 8i + 2(t%4) and the one behind, and the same of lane t/4 + 8,
// in r[4i .. 4i+3] for i = 0, 1.
__device__ __forceinline__ void tmem_ld_16x256b_x2(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}

// Four 8 x 8 blocks of 16-bit values, each stored transposed: lane 8 b + i
// gives the address of the eight values that were column i of block b.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, const uint32_t (&p)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(p[0]), "r"(p[1]), "r"(p[2]), "r"(p[3])
               : "memory");
}

// Instruction descriptor: FP16 or BF16 operands, FP32 accumulator, both
// K-major, M x N.
template <typename T>
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
  constexpr uint32_t ab = std::is_same<T, __half>::value ? 0u : 1u;
  return (1u << 4) | (ab << 7) | (ab << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// A row's scale for one group, ready for its codes.
template <typename T>
struct RowScale;

template <>
struct RowScale<__half> {
  __half2 s;
  __device__ __forceinline__ explicit RowScale(uint32_t bits)
      : s(__half2half2(__ushort_as_half(static_cast<unsigned short>(bits)))) {}
  // The quantizer's largest scale, of a group whose maximum is near 65504: 7 *
  // 9360 = 65520 would round to infinity.  The largest finite value is as near
  // as a rounding may be (16 off, half a step is 32 there).
  static __device__ __forceinline__ bool overflows(uint32_t bits) { return bits == 0x7092; }
  static __device__ __forceinline__ uint32_t finite(uint32_t w) {
    const __half2 most = __half2half2(__ushort_as_half(0x7BFF));
    const __half2 v = __hmax2(__hmin2(*reinterpret_cast<const __half2*>(&w), most), __hneg2(most));
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  // eight codes of a word -> four pairs code * scale, each rounded once
  __device__ __forceinline__ void apply(uint32_t w, uint32_t* out) const {
    uint32_t p[4];
    Elem<__half>::codes(w, p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&p[i]), s);
      out[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
};

template <>
struct RowScale<__nv_bfloat16> {
  // an FP16 scale as a sum of two BF16 values (11 bits of mantissa in 8 + 8)
  __nv_bfloat162 hi, lo;
  __device__ __forceinline__ explicit RowScale(uint32_t bits) {
    const float f = __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
    const __nv_bfloat16 h = __float2bfloat16_rn(f);
    hi = __bfloat162bfloat162(h);
    lo = __bfloat162bfloat162(__float2bfloat16_rn(f - __bfloat162float(h)));
  }
  static __device__ __forceinline__ bool overflows(uint32_t) { return false; }   // BF16 holds them all
  static __device__ __forceinline__ uint32_t finite(uint32_t w) { return w; }
  // code * lo is exact (4 + 3 bits), so the sum rounds code * scale once
  __device__ __forceinline__ void apply(uint32_t w, uint32_t* out) const {
    uint32_t p[4];
    Elem<__nv_bfloat16>::codes(w, p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 q = *reinterpret_cast<const __nv_bfloat162*>(&p[i]);
      const __nv_bfloat162 v = __hfma2(q, hi, __hmul2(q, lo));
      out[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
};

template <int T, int RB>
struct W4MmaCfg {
  // Warps: 0 producer, 1 .. RB MMA, idle up to 3; the others unpack and write
  // the sums out, eight to a row block: two to a quarter of its rows with half
  // a tile's columns each (with one, unpacking took longer than the MMAs).
  static constexpr int kUnpackWarps = 8 * RB;
  static constexpr int kThreads = 128 + 32 * kUnpackWarps;
  static constexpr int kCtasPerSm = 2 / RB;
  static constexpr int kRows = 128 * RB;
  static constexpr int kXBox = T * 128;                 // 64 columns of T tokens
  static constexpr int kXSlot = 2 * kXBox;
  static constexpr int kXSlots = RB == 2 ? (T == 128 ? 4 : 6) : T == 128 ? 2 : T == 64 ? 4 : T == 32 ? 6 : 8;
  static constexpr int kWSlot = 8 * RB * kW4TileBytes;  // 128 columns of the rows
  static constexpr int kWSlots = T == 128 ? 4 : RB == 2 ? 6 : T == 16 ? 6 : 5;
  static constexpr int kXBytes = kXSlots * kXSlot;
  static constexpr int kWBytes = kWSlots * kWSlot;
  // results lie over the operand slots before they leave, or FP32 sums for
  // the cluster; a token's results start half a bank line after the last one's
  static constexpr int kOutPitch = kRows * 2 + 16;
  static constexpr int kMain = kXBytes + kWBytes > T * kRows * 4 ? kXBytes + kWBytes : T * kRows * 4;
  static constexpr int kSmem = kMain + 1024;            // aligned to the swizzle's 1024 bytes
  static constexpr int kAccCols = T < 32 ? 32 : T;
  static constexpr int kACols = 64;                     // 128 columns of weights
  static constexpr int kASlots = 2;
  static constexpr int kTmemCols = 256 * RB;            // of an SM's 512
  static_assert(RB * (kAccCols + kASlots * kACols) <= kTmemCols, "tensor memory");
  // one CTA more on the SM would wait for tensor memory
  static_assert((kCtasPerSm + 1) * kSmem > 227 * 1024 && kCtasPerSm * (kSmem + 2048) <= 228 * 1024,
                "CTAs per SM");
};

struct W4MmaArgs {
  CUtensorMap x;                        // [M][K], boxes of 64 columns x T tokens, 128-byte swizzle
  CUtensorMap w[kW4MaxLayers];          // [strip][16 kbs rows][64 bytes], boxes of 8 RB strips, 64-byte swizzle
  const __half* ws[kW4MaxLayers];
  void* y[kW4MaxLayers];
  long long ldy[kW4MaxLayers];
  int N[kW4MaxLayers];
  int tile0[kW4MaxLayers + 1];          // first tile of 128 RB rows of each layer
  int n;
  int M, K, G, kbs, gs_shift;
  int split;                            // CTAs of a cluster, which share a tile's columns
  int token_tiles;
  int first_wave;                       // CTAs that start together
  int stall;                            // test hook: the first tile is withheld
  unsigned int* status;
  unsigned long long wait_limit_ns;
};

template <typename E, int T, int RB>
__global__ void __launch_bounds__(W4MmaCfg<T, RB>::kThreads, W4MmaCfg<T, RB>::kCtasPerSm)
    w4_mma_kernel(const __grid_constant__ W4MmaArgs a) {
  using Cfg = W4MmaCfg<T, RB>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t x_full[Cfg::kXSlots], x_empty[Cfg::kXSlots];
  __shared__ uint64_t w_full[Cfg::kWSlots], w_empty[Cfg::kWSlots];
  __shared__ uint64_t a_full[RB][Cfg::kASlots], a_empty[RB][Cfg::kASlots];
  __shared__ uint64_t acc_full[RB];
  __shared__ uint32_t tmem_at;
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* x_mem = base;
  uint8_t* w_mem = base + Cfg::kXBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t lim = a.wait_limit_ns;

  // the tile: token tiles vary fastest, so that the CTAs in flight share weights
  const int rank = blockIdx.x % a.split, tile = blockIdx.x / a.split;
  const int mt = tile % a.token_tiles, rt = tile / a.token_tiles;
  int l = 0;
  while (l + 1 < a.n && rt >= a.tile0[l + 1]) ++l;
  const int strip0 = (rt - a.tile0[l]) * 8 * RB;
  const int kb0 = static_cast<int>(static_cast<long long>(rank) * a.kbs / a.split);
  const int nk = static_cast<int>(static_cast<long long>(rank + 1) * a.kbs / a.split) - kb0;

  auto load_w = [&](int i) {
    if (a.stall && i == 0) return;
    uint64_t* bar = &w_full[i % Cfg::kWSlots];
    mbar_arrive_expect_tx(bar, Cfg::kWSlot);
    tma_load_3d(w_mem + i % Cfg::kWSlots * Cfg::kWSlot, &a.w[l], bar, 0, (kb0 + i) * 16, strip0);
  };
  auto load_x = [&](int i) {
    uint64_t* bar = &x_full[i % Cfg::kXSlots];
    uint8_t* dst = x_mem + i % Cfg::kXSlots * Cfg::kXSlot;
    mbar_arrive_expect_tx(bar, Cfg::kXSlot);
    tma_load_2d(dst, &a.x, bar, (kb0 + i) * 128, mt * T);
    tma_load_2d(dst + Cfg::kXBox, &a.x, bar, (kb0 + i) * 128 + 64, mt * T);
  };
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < Cfg::kXSlots; ++i) {
      mbar_init(&x_full[i], 1);
      mbar_init(&x_empty[i], RB);
    }
    for (int i = 0; i < Cfg::kWSlots; ++i) {
      mbar_init(&w_full[i], 1);
      mbar_init(&w_empty[i], Cfg::kUnpackWarps);
    }
    for (int rb = 0; rb < RB; ++rb) {
      for (int i = 0; i < Cfg::kASlots; ++i) {
        mbar_init(&a_full[rb][i], 8);
        mbar_init(&a_empty[rb][i], 1);
      }
      mbar_init(&acc_full[rb], 1);
    }
    fence_barrier_init();
    // towards L2 while the kernel before ends; its results are read behind the
    // wait alone
    if (static_cast<int>(blockIdx.x) < a.first_wave)
      for (int i = 0; i < Cfg::kWSlots && i < nk; ++i) tma_prefetch_3d(&a.w[l], 0, (kb0 + i) * 16, strip0);
    grid_wait_dependencies();
    for (int i = 0; i < Cfg::kWSlots && i < nk; ++i) load_w(i);
    for (int i = 0; i < Cfg::kXSlots && i < nk; ++i) load_x(i);
  }
  // an unpack warp's quarter q of row block rb, and its half h of a tile's columns
  const int q = warp & 3, h = (warp - 4) >> 2 & 1, rb = max(warp - 4, 0) >> 3;
  const int row = rb * 128 + q * 32 + lane;
  // Where the scales of words 2 h and 2 h + 1 of this row lie, for the even
  // and the odd tiles: two tiles on is `step` scales on.  A row behind the
  // last takes that one's (its sums are dropped).
  const int n_row = min(strip0 * 16 + row, a.N[l] - 1), step = 256 >> a.gs_shift;
  const unsigned short* sp[2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
    sp[j] = reinterpret_cast<const unsigned short*>(a.ws[l]) + static_cast<size_t>(n_row) * a.G +
            (((kb0 + j) * 128 + h * 64) >> a.gs_shift);
  const bool two = a.gs_shift < 6;              // words with a group each
  // words of the last tile behind K have no scale (their codes are zeros)
  const int last = a.kbs - kb0 - 1, last_words = (a.K - (a.kbs - 1) * 128 + 31) / 32 - 2 * h;
  auto scales = [&](int i, int j, uint32_t (&s)[2]) {
    const int words = i == last ? last_words : 2;
    if (i < nk && words > 0) {
      s[0] = s[1] = __ldg(sp[j]);
      if (two && words > 1) s[1] = __ldg(sp[j] + 1);
    }
    sp[j] += step;
  };
  uint32_t s0[2] = {}, s1[2] = {};
  if (warp >= 4) {
    if (last > 0 || last_words > 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(sp[0]));
    grid_wait_dependencies();
    scales(0, 0, s0);
    scales(1, 1, s1);
  }
  // Tensor memory is taken after the kernel before has ended and before the
  // next may begin: one that takes its own while others still wait for theirs
  // would keep it until they end.
  if (warp == 1) {
    grid_wait_dependencies();
    tmem_alloc(&tmem_at, Cfg::kTmemCols);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  const uint32_t acc_col = tmem, a_col0 = tmem + RB * Cfg::kAccCols;
  grid_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------- producer -----
    if (lane == 0) {
      int w_issued = min(nk, Cfg::kWSlots), x_issued = min(nk, Cfg::kXSlots);
      bool ok = true;
      for (int i = 0; ok && i < nk; ++i) {
        if (i + Cfg::kWSlots < nk) {
          ok = mbar_wait(&w_empty[i % Cfg::kWSlots], (i / Cfg::kWSlots) & 1, lim);
          if (ok) {
            load_w(i + Cfg::kWSlots);
            ++w_issued;
          }
        }
        if (ok && i + Cfg::kXSlots < nk) {
          ok = mbar_wait(&x_empty[i % Cfg::kXSlots], (i / Cfg::kXSlots) & 1, lim);
          if (ok) {
            load_x(i + Cfg::kXSlots);
            ++x_issued;
          }
        }
      }
      if (!ok) record_status(a.status, kStatusTimeout, 0);
      // every issued copy must land before the CTA may finish
      for (int i = max(0, w_issued - Cfg::kWSlots); i < w_issued; ++i)
        mbar_wait(&w_full[i % Cfg::kWSlots], (i / Cfg::kWSlots) & 1, lim);
      for (int i = max(0, x_issued - Cfg::kXSlots); i < x_issued; ++i)
        mbar_wait(&x_full[i % Cfg::kXSlots], (i / Cfg::kXSlots) & 1, lim);
    }
    __syncwarp();
  } else if (warp <= RB) {
    // ------------------------------------------------------------ MMA -----
    // A warp per row block: while one waits at its barriers the other's MMAs
    // run.  The whole warp waits and one elected lane issues, so that the
    // compiler knows the operands to be uniform.
    const int rb = warp - 1;
    constexpr uint32_t idesc = idesc_f16<E>(128, T);
    const uint64_t desc0 = smem_desc_k_sw128(smem_u32(x_mem));
    const uint32_t acc = acc_col + rb * Cfg::kAccCols;
    RingPos<Cfg::kXSlots> xp;
    RingPos<Cfg::kASlots> as;
    bool ok = true;
    for (int i = 0; i < nk; ++i) {
      ok = warp_wait(&x_full[xp.idx], xp.phase, lim) && warp_wait(&a_full[rb][as.idx], as.phase, lim);
      if (!ok) break;
      tc_fence_after();
      const uint64_t desc = desc0 + ((xp.idx * Cfg::kXSlot) >> 4);
      const uint32_t a_col = a_col0 + (as.idx * RB + rb) * Cfg::kACols;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 8; ++k)             // 16 columns each: 8 TMEM columns, 32 bytes of x
          mma_f16_tmem_a(acc, a_col + k * 8, desc + (((k >> 2) * Cfg::kXBox + (k & 3) * 32) >> 4),
                         idesc, i == 0 && k == 0 ? 0u : 1u);
        mma_commit(&x_empty[xp.idx]);
        mma_commit(&a_empty[rb][as.idx]);
      }
      __syncwarp();
      xp.next();
      as.next();
    }
    if (!ok && lane == 0) record_status(a.status, kStatusTimeout, 1);
    // all issued MMAs finish before the sums are read or TMEM is released
    if (elect_one()) mma_commit(&acc_full[rb]);
    warp_wait(&acc_full[rb], 0, lim);
  } else if (warp >= 4) {
    // --------------------------------------------------------- unpack -----
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    RingPos<Cfg::kWSlots> wp;
    uint32_t phase = 1;                         // of the A slots' release
    auto unpack = [&](int i, int slot, uint32_t (&s)[2]) -> bool {
      if (!warp_wait(&w_full[wp.idx], wp.phase, lim)) return false;
      // chunk t of the row lies at t ^ (row / 2 % 4): the box's 64-byte swizzle
      const uint2* src = reinterpret_cast<const uint2*>(w_mem + wp.idx * Cfg::kWSlot + row * 64) + h;
      uint2 c[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) c[t] = src[(t ^ ((row >> 1) & 3)) * 2];
      __syncwarp();
      if (lane == 0) mbar_arrive(&w_empty[wp.idx]);
      wp.next();
      // columns 64 h .. +63; chunk t's eight of word j at 32 j + 8 t
      uint32_t out[32];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const RowScale<E> scale(s[j]);
#pragma unroll
        for (int t = 0; t < 4; ++t) scale.apply(j == 0 ? c[t].x : c[t].y, out + 16 * j + 4 * t);
      }
      // One test per lane and tile, so that other weights pay no clamping (64
      // tokens x 28672 x 8192 53 us with it, 51 without; 512 x 8192 x 8192 58.5
      // and 57.9, and 59.8 with every word clamped).
      if (__builtin_expect(RowScale<E>::overflows(s[0]) | RowScale<E>::overflows(s[1]), 0)) {
#pragma unroll
        for (int w = 0; w < 32; ++w) out[w] = RowScale<E>::finite(out[w]);
      }
      scales(i + Cfg::kASlots, slot, s);        // for this slot's next tile
      if (!warp_wait(&a_empty[rb][slot], phase, lim)) return false;
      tc_fence_after();
      tmem_st32(lane_base + a_col0 + (slot * RB + rb) * Cfg::kACols + 32 * h, out);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&a_full[rb][slot]);
      return true;
    };
    bool ok = true;
    static_assert(Cfg::kASlots == 2, "the loop below takes two tiles at a time");
    for (int i = 0; ok && i < nk; i += 2, phase ^= 1) {
      ok = unpack(i, 0, s0);
      if (ok && i + 1 < nk) ok = unpack(i + 1, 1, s1);
    }
    // ------------------------------------------------------- epilogue -----
    // The sums go to shared memory, over the operands: as results of the
    // activations' type, token by token, or in FP32 for the cluster to add up.
    // The other row block's MMAs may still read the operands there.
    for (int r = 0; ok && r < RB; ++r) ok = warp_wait(&acc_full[r], 0, lim);
    if (!ok && lane == 0) record_status(a.status, kStatusTimeout, 2);
    if (ok) {
      tc_fence_after();
      const uint32_t acc = lane_base + acc_col + rb * Cfg::kAccCols;
#pragma unroll 1
      for (int c0 = 16 * h; c0 < T; c0 += 32) {         // the two warps of a quarter take turns
        if (a.split > 1) {
          uint32_t v[16];
          tmem_ld16(acc + c0, v);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            reinterpret_cast<float*>(base)[(c0 + j) * Cfg::kRows + row] = __uint_as_float(v[j]);
        } else {
          // thread t holds tokens 2 (t % 4) + {0, 1} (+ 8 for the second four) of
          // rows t / 4 and t / 4 + 8: 8 x 8 blocks as stmatrix takes them
          uint32_t v[2][8];
          tmem_ld_16x256b_x2(acc + c0, v[0]);
          tmem_ld_16x256b_x2(acc + c0 + (16u << 16), v[1]);
          tmem_wait_ld();
          // lane 8 b + i gives the place of token i of block b: rows 8 (b % 2), tokens 8 (b / 2)
          const uint32_t at = smem_u32(base) + (c0 + (lane >> 4) * 8 + (lane & 7)) * Cfg::kOutPitch +
                              (rb * 128 + q * 32 + (lane >> 3 & 1) * 8) * 2;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            uint32_t p[4];
#pragma unroll
            for (int b = 0; b < 4; ++b)
              p[b] = Elem<E>::pack(__uint_as_float(v[r][2 * b]), __uint_as_float(v[r][2 * b + 1]));
            stmatrix_x4_trans(at + r * 32, p);
          }
        }
      }
    }
  }

  // ------------------------------------------------------------ teardown --
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::kTmemCols);
  }
  // results leave in pieces of eight rows (of the weights) of a token
  E* const y = static_cast<E*>(a.y[l]);
  const long long ldy = a.ldy[l];
  const int n0 = strip0 * 16, N = a.N[l];
  const bool wide = ((ldy * 2) | static_cast<long long>(reinterpret_cast<uintptr_t>(y))) % 16 == 0;
  auto write = [&](int token, int piece, const uint4& v) {
    const int m = mt * T + token, n = n0 + piece * 8;
    if (m >= a.M || n >= N) return;
    E* at = y + m * ldy + n;
    if (wide && n + 8 <= N) {
      *reinterpret_cast<uint4*>(at) = v;
    } else {
      const E* e = reinterpret_cast<const E*>(&v);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (n + j < N) at[j] = e[j];
    }
  };
  constexpr int kPieces = Cfg::kRows / 8;
  if (a.split == 1) {
    for (int i = threadIdx.x; i < T * kPieces; i += Cfg::kThreads)
      write(i / kPieces, i % kPieces,
            *reinterpret_cast<const uint4*>(base + i / kPieces * Cfg::kOutPitch + i % kPieces * 16));
    return;
  }
  cluster_sync_all();
  // every rank adds up the ranks' sums for its share of the tokens
  const int t0 = rank * T / a.split, t1 = (rank + 1) * T / a.split;
  for (int i = t0 * kPieces + threadIdx.x; i < t1 * kPieces; i += Cfg::kThreads) {
    const uint32_t at = smem_u32(base) + static_cast<uint32_t>(i) * 32;
    float sum[8] = {};
    for (int r0 = 0; r0 < a.split; r0 += 4) {           // four ranks' sums in flight
      float v[4][8];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (r0 + r >= a.split) break;
        const uint32_t p = map_to_rank(at, r0 + r);
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v[r][0]), "=f"(v[r][1]), "=f"(v[r][2]), "=f"(v[r][3]) : "r"(p) : "memory");
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v[r][4]), "=f"(v[r][5]), "=f"(v[r][6]), "=f"(v[r][7]) : "r"(p + 16) : "memory");
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (r0 + r >= a.split) break;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += v[r][j];
      }
    }
    uint4 o;
    o.x = Elem<E>::pack(sum[0], sum[1]);
    o.y = Elem<E>::pack(sum[2], sum[3]);
    o.z = Elem<E>::pack(sum[4], sum[5]);
    o.w = Elem<E>::pack(sum[6], sum[7]);
    write(i / kPieces, i % kPieces, o);
  }
  cluster_sync_all();                   // no CTA leaves while another reads its sums
}

}  // namespace flexq

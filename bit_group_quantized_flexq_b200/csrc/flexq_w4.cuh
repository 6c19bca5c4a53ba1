// flexq_w4.cuh -- weight-only 4-bit linear layers: the packed form, its
// quantizer and the matrix-vector product for small batches.
//
// A weight row is cut into groups of gs consecutive values that share one
// FP16 scale s = fp16_rne(absmax / 7); a code is q = clamp(rne(w / s), -7, 7)
// (-8 is never produced but multiplied exactly).  The layer's output is
//   y[m,n] = sum_g s[n,g] * sum_{k in g} x[m,k] * q[n,k]
// with FP16 or BF16 activations that are not quantized.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "flexq_gemm.cuh"
#include "flexq_ptx.cuh"
#include "flexq_quant.cuh"

namespace flexq {

// ------------------------------------------------------------ packed form --
// Rows are padded to a multiple of 16 and columns to a multiple of 128 (code
// 0).  Tile (nt, kb) = rows 16 nt .. +15, columns 128 kb .. +127 is 1024
// contiguous bytes at (nt * kbs + kb) * 1024; row r of it is 64 bytes at
// 64 r; its 16-byte chunk t holds four little-endian words, and word w the
// eight codes of columns 32 w + 8 t .. +7 as u = q + 8: columns 0, 2, 4 and 6
// in nibbles 0, 2, 1 and 3, the odd column behind each four nibbles higher.
//
// Why: a warp's 16-byte loads of a tile cover 512 contiguous bytes, lane
// (4 r + t) holding row r's chunk t, which is the register layout of an
// m16n8k16 MMA's A operand up to the order of k; that order is chosen so that
// the lane's activations for one word are 16 contiguous bytes too.  The
// nibble order puts consecutive columns into the two halves of a register
// with one mask, and columns 0 .. 3 and 4 .. 7 into the same bits of them.  A
// row's 128 codes stay within 64 aligned bytes (two DRAM sectors), so that
// rows can also be looked up alone.
constexpr int kW4TileCols = 128;
constexpr int kW4TileBytes = 1024;

__host__ __device__ inline int w4_row_tiles(int N) { return (N + 15) / 16; }
__host__ __device__ inline int w4_col_tiles(int K) { return (K + 127) / 128; }

// The bit at which code i (0..7) of a word begins.
__host__ __device__ constexpr int w4_shift(int i) {
  return 4 * ((i >> 1 & 1) * 2 + (i >> 2) + 4 * (i & 1));
}

// --------------------------------------------------------------- quantizer --
// Offline, once per layer: two passes over W, the scales and then the codes.  A
// warp reads 64 bytes at a time in the first, a thread 16 in the second: 28672 x
// 8192 takes 485 us, a fifth of a copy's rate.
__global__ void w4_scale_kernel(const __half* __restrict__ w, __half* __restrict__ scales,
                                long long groups, int gs) {
  const long long grp = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) / 32;
  if (grp >= groups) return;
  const int lane = threadIdx.x & 31;
  float amax = 0.0f;
  for (int i = lane; i < gs; i += 32) amax = fmaxf(amax, fabsf(__half2float(w[grp * gs + i])));
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  if (lane == 0) scales[grp] = group_scale(amax, 7.0f);
}

// One thread per word of the packed form, padding included.
__global__ void w4_pack_kernel(const __half* __restrict__ w, const __half* __restrict__ scales,
                               uint32_t* __restrict__ packed, int N, int K, int kbs, int gs,
                               long long words) {
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= words) return;
  const long long tile = i >> 8;
  const int r = static_cast<int>(i >> 4) & 15, t = static_cast<int>(i >> 2) & 3, wd = static_cast<int>(i) & 3;
  const int n = static_cast<int>(tile / kbs) * 16 + r;
  const int k = static_cast<int>(tile % kbs) * 128 + wd * 32 + t * 8;
  uint32_t word = 0x88888888u;
  if (n < N && k < K) {
    const float s = __half2float(scales[static_cast<size_t>(n) * (K / gs) + k / gs]);
    const uint4 v = *reinterpret_cast<const uint4*>(w + static_cast<size_t>(n) * K + k);
    const __half* h = reinterpret_cast<const __half*>(&v);
    word = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int q = quant_code_div(__half2float(h[j]), s, 7);
      word |= static_cast<uint32_t>(q + 8) << w4_shift(j);
    }
  }
  packed[i] = word;
}

// ---------------------------------------------------------- element types --
// (w & mask) | bits in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(bits));
  return r;
}

template <typename T>
struct Elem;

template <>
struct Elem<__half> {
  static __device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
  // d = a . b + c
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1, const float (&c)[4]) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]),
          "f"(c[2]), "f"(c[3]));
  }
  // The eight codes of a word as exact FP16 pairs of consecutive columns, by
  // the common way of putting an integer's bits into the mantissa of a power
  // of two: a nibble in the low mantissa bits of 1024 is 1024 + u; four bits
  // further up it is 1024 + 16 u, brought down by an exact multiply-add.
  static __device__ __forceinline__ void codes(uint32_t w, uint32_t (&p)[4]) {
    const __half2 off = __half2half2(__ushort_as_half(0x6408));      // 1032
    const __half2 sixteenth = __half2half2(__ushort_as_half(0x2C00));   // 1/16
    const __half2 off16 = __half2half2(__ushort_as_half(0xD480));    // -72
    const uint32_t v = w >> 8;
    uint32_t b[4];
    b[0] = and_or(w, 0x000F000Fu, 0x64006400u);
    b[1] = and_or(w, 0x00F000F0u, 0x64006400u);
    b[2] = and_or(v, 0x000F000Fu, 0x64006400u);
    b[3] = and_or(v, 0x00F000F0u, 0x64006400u);
    __half2* h = reinterpret_cast<__half2*>(b);
    __half2* o = reinterpret_cast<__half2*>(p);
    o[0] = __hsub2(h[0], off);
    o[1] = __hsub2(h[2], off);
    o[2] = __hfma2(h[1], sixteenth, off16);
    o[3] = __hfma2(h[3], sixteenth, off16);
  }
  // The streaming kernel's operand: the codes as they are.
  static constexpr float kUnit = 1.0f;
  static __device__ __forceinline__ void operand(uint32_t w, uint32_t (&p)[4]) { codes(w, p); }
};

template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  }
  // d = a . b + c
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1, const float (&c)[4]) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]),
          "f"(c[2]), "f"(c[3]));
  }
  // BF16 has 7 mantissa bits: a nibble in the low ones of 128 is 128 + u; the
  // other nibbles are shifted there first.  DOWN: in units of 2^-DOWN.
  template <int DOWN = 0>
  static __device__ __forceinline__ void codes(uint32_t w, uint32_t (&p)[4]) {
    constexpr uint32_t base = 0x4300u - (DOWN << 7);                           // 128
    const __nv_bfloat162 off = __bfloat162bfloat162(__ushort_as_bfloat16(base + 8));   // 136
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = and_or(w >> w4_shift(2 * i), 0x000F000Fu, base << 16 | base);
      const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&b), off);
      p[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
  // The streaming kernel's operand: codes in units of 2^-11, so that a group's
  // sum, of at most 256 terms of at most 8 |x|, is at most the largest |x| and
  // no finite activation overflows it.
  static constexpr float kUnit = 2048.0f;
  static __device__ __forceinline__ void operand(uint32_t w, uint32_t (&p)[4]) { codes<11>(w, p); }
};

// ---------------------------------------------------- matrix-vector product --
constexpr int kW4MaxLayers = 4;

// The layers of one launch: they read the same activations.  Strips of 16
// rows are numbered layer after layer.
struct W4Layers {
  const uint4* wp[kW4MaxLayers];
  const __half* ws[kW4MaxLayers];
  void* y[kW4MaxLayers];
  long long ldy[kW4MaxLayers];
  int N[kW4MaxLayers];
  int strip0[kW4MaxLayers + 1];
  int n;
};

struct W4Args {
  const void* x;
  long long ldx;
  int M, K, G, kbs, gs_shift;     // kbs: tiles of 128 columns; gs = 1 << gs_shift
  int split, rounds;              // streaming kernel: CTAs of a cluster, parts of its strips
  int stall;                      // test hook: every warp's first copy is withheld
  unsigned int* status;           // device status word
  unsigned long long wait_limit_ns;
};

// Brings bytes (a multiple of 16, 16-byte aligned) towards the L2 cache, where
// what a kernel before writes into them meanwhile is seen too.
__device__ __forceinline__ void prefetch_l2(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// The product for batches of up to 16 tokens streams the weights once, so it
// is bound by HBM; every SM must keep tens of KB of loads in flight from its
// first to its last cycle.  A strip's tiles are cut into chunks of four tiles
// (16 rows x 512 columns, 4 KB, one bulk copy).  A cluster of one to eight
// CTAs, one per SM, takes a run of strips; each of its CTAs takes a share of
// their columns, whose activations it keeps in shared memory, and divides its
// chunks evenly among 16 warps, wherever strips begin or end: no warp waits
// for another before the end.  A warp brings a chunk into a buffer of its own
// while it multiplies the one before in registers.  Codes are exact in FP16
// and BF16; the tensor core adds a group's products in FP32, and the group's
// sum times the scale is added in FP32.  What a warp has of a strip that it
// shares with others is added, in the order of the columns, by the warp that
// holds the strip's first chunk, and so are the CTAs' sums of a strip.  Where
// shared memory does not hold those of all its strips, a cluster takes them in
// rounds.
//
// Taking a code apart has to cost little: at HBM's rate an SM has about 44
// cycles per tile.  Yet the tensor core multiplies the signed codes, 9 (FP16)
// and 11 (BF16) instructions per word: multiplying u = q + 8 and starting a
// group from -8 times the sum of its activations takes 5, but those sums
// cancel, so that a large activation on a zero code costs all other terms of
// its group bits.  (That way one token x 28672 x 8192 took 25.8 us, 8 x 8192 x
// 8192 13.1 and 16 x 4096 x 4096 11.1, for 27.9, 12.2 and 7.3: the sums of the
// activations have their price too.)
//
// Measured (device time, weights cold): 28672 x 8192 at one token 27.9 us, 4.3
// TB/s or 0.66 of a copy's rate; the same kernel without its arithmetic takes
// 21.4 us.  Between the two is the time from a chunk's arrival to the next
// request, with the four warps that a scheduler has: it issues in 55 % of its
// cycles, ALU 38 % and tensor core 22 % busy.  20 and 24 warps take 29.7
// and 33.3 us, chunks of two tiles 30.6.  4096 x 4096 takes 5.2 us, of which
// its stream is 1.3: launch, the first bytes and the final sums are the rest.
// 16 tokens x 28672 columns take 51 us: a lane reads its activations from
// shared memory four times as often as its codes, and 15 clusters of eight,
// which is what their activations need, fill 120 of 148 SMs.  (Chunks of two
// tiles take 44.6 there, but 5 to 10 % more at one token.)
constexpr int kGemvWarps = 16;
constexpr int kGemvThreads = kGemvWarps * 32;
constexpr int kGemvChunk = 4;                 // tiles
constexpr int kGemvChunkCols = kGemvChunk * kW4TileCols;
constexpr int kGemvChunkBytes = kGemvChunk * kW4TileBytes;
constexpr int kGemvBufferBytes = kGemvWarps * kGemvChunkBytes;

// The scales of a row for a chunk: NS of them, as FP16 bits in pairs.
template <int NS>
struct ChunkScales {
  uint32_t v[(NS + 1) / 2];
  __device__ __forceinline__ float get(int i) const {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(v[i / 2] >> (16 * (i & 1)))));
  }
  // `left` scales from p on belong to the row (none: a row behind the last).
  // `even`: every chunk is whole and its scales are aligned for wide loads.
  __device__ __forceinline__ void load(const __half* p, int left, bool even) {
    if (even && left > 0) {
      if constexpr (NS == 1) {
        v[0] = __ldg(reinterpret_cast<const unsigned short*>(p));
      } else if constexpr (NS == 2) {
        v[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
      } else if constexpr (NS == 4) {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
        v[0] = u.x;
        v[1] = u.y;
      } else {
#pragma unroll
        for (int i = 0; i < NS / 8; ++i) {
          const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + i);
          v[4 * i] = u.x;
          v[4 * i + 1] = u.y;
          v[4 * i + 2] = u.z;
          v[4 * i + 3] = u.w;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NS; i += 2) {
        uint32_t lo = 0, hi = 0;
        if (i < left) lo = __ldg(reinterpret_cast<const unsigned short*>(p) + i);
        if (NS > 1 && i + 1 < left) hi = __ldg(reinterpret_cast<const unsigned short*>(p) + i + 1);
        v[i / 2] = lo | hi << 16;
      }
    }
  }
};

// acc += one 16 x 128 tile times the activations of 8 NT tokens.  x: the
// lane's activations of the chunk, those of the n-th eight tokens xo[n] bytes
// on; c0, c1: scales of rows g and g + 8; WPG: words (of 32 columns) per
// group, 8 where a group is two tiles.
//
// Two chains of MMAs are in flight: of the words' halves where there is one
// eight of tokens and a group has several words, else one for each eight (two
// words' halves then cost their addition per group and registers: 16 tokens x
// 28672 columns 53.1 us with them and 51.0 without, 5 tokens x 32003 x 4096 in
// groups of 64 17.6 and 16.9; one token x 28672 x 8192 in groups of 128 27.6
// and 28.0).
template <typename T, int WPG, int NS, int NT>
__device__ __forceinline__ void gemv_tile(float (&acc)[NT][4], const uint4& w0, const uint4& w1,
                                          const uint8_t* x, const int (&xo)[NT],
                                          const ChunkScales<NS>& c0,
                                          const ChunkScales<NS>& c1, int tile) {
  constexpr bool kHalves = NT == 1 && WPG >= 4;
  float sum[NT][4], upper[4];           // upper: columns 4 .. 7 of the words, where they are apart
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t lo[4], hi[4];
    Elem<T>::operand(reinterpret_cast<const uint32_t*>(&w0)[j], lo);
    Elem<T>::operand(reinterpret_cast<const uint32_t*>(&w1)[j], hi);
    const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]};
    const uint32_t a1[4] = {lo[2], hi[2], lo[3], hi[3]};
    const int i = (tile * 4 + j) / WPG;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint4 xv = *reinterpret_cast<const uint4*>(x + xo[n] + tile * 256 + j * 64);
      if (j % WPG == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[n][e] = upper[e] = 0.0f;
      }
      Elem<T>::mma(sum[n], a0, xv.x, xv.y, sum[n]);
      if (kHalves) Elem<T>::mma(upper, a1, xv.z, xv.w, upper);
      else Elem<T>::mma(sum[n], a1, xv.z, xv.w, sum[n]);
      if ((j + 1) % WPG == 0 || j == 3) {
        const float f0 = c0.get(i), f1 = c1.get(i);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[n][e] = fmaf(kHalves ? sum[n][e] + upper[e] : sum[n][e], e < 2 ? f0 : f1, acc[n][e]);
      }
    }
  }
}

// Chunks of a strip, and those a CTA of a cluster takes at most.
__host__ __device__ constexpr int gemv_chunks(int kbs) { return (kbs + kGemvChunk - 1) / kGemvChunk; }
__host__ __device__ constexpr int gemv_share(int kbs, int split) {
  return (gemv_chunks(kbs) + split - 1) / split;
}

// Bytes of a token's activations in shared memory: whole chunks (zeros behind
// K), and half a bank line so that tokens' rows start in different banks.
__host__ __device__ constexpr int gemv_x_stride(int chunks) { return chunks * kGemvChunkCols * 2 + 64; }

// Eights of tokens that the kernel multiplies at once.
__host__ __device__ constexpr int gemv_eights(int M) { return M <= 8 ? 1 : 2; }

// Shared memory: the warps' buffers, the activations, and with a cluster the
// sums of the strips of a round.
__host__ __device__ constexpr long long gemv_smem(int M, int kbs, int split, int strips) {
  return kGemvBufferBytes + static_cast<long long>(M) * gemv_x_stride(gemv_share(kbs, split)) +
         (split > 1 ? static_cast<long long>(strips) * gemv_eights(M) * 512 : 0);
}

// MANY: several rounds (a kernel of its own: the loop costs one round's launch
// of 4096 x 4096 at one token 0.4 of 5.3 us).
template <typename T, int WPG, int NT, bool MANY>
__global__ void __launch_bounds__(kGemvThreads, 1) w4_gemv_kernel(const __grid_constant__ W4Layers L,
                                                                 const W4Args a) {
  constexpr int NS = 4 * kGemvChunk / WPG;        // scales of a row per chunk
  extern __shared__ __align__(128) uint8_t buffers[];
  __shared__ uint64_t full[kGemvWarps];
  __shared__ uint64_t x_full;
  __shared__ float4 head_of[kGemvWarps][NT][32];  // of a strip begun by an earlier warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int kbs = a.kbs, rank = blockIdx.x % a.split;
  const long long cluster = blockIdx.x / a.split, clusters = gridDim.x / a.split;
  const int strips = L.strip0[L.n];
  // the cluster's strips, and this CTA's chunks of each
  const int strip_lo = static_cast<int>(cluster * strips / clusters);
  const int strip_n = static_cast<int>((cluster + 1) * strips / clusters) - strip_lo;
  const int per_strip = gemv_chunks(kbs);
  const int c_lo = rank * per_strip / a.split, chunks = (rank + 1) * per_strip / a.split - c_lo;
  // tiles of the last of them
  const int end_tiles = min(kGemvChunk, kbs - (c_lo + chunks - 1) * kGemvChunk);
  auto layer_of = [&](int strip) {
    int l = 0;
    while (l + 1 < L.n && strip >= L.strip0[l + 1]) ++l;
    return l;
  };
  // shared memory is laid out for the largest share, alike in all CTAs
  const int room = gemv_share(kbs, a.split), x_stride = gemv_x_stride(room);
  uint8_t* buffer = buffers + warp * kGemvChunkBytes;
  uint8_t* xs_mem = buffers + kGemvBufferBytes;                           // [M][x_stride]
  float4* slab = reinterpret_cast<float4*>(xs_mem + a.M * x_stride);      // [count][NT][32]

  int first = 0, count = 0, units = 0;   // the round's strips and this CTA's chunks of them
  int u0 = 0, u1 = 0;               // this warp's chunks
  int c = 0, strip = 0;             // of the chunk in hand
  // the next chunk to request, its place in the share and in memory
  int ru = 0, rc = 0, rs = 0, asked = 0;
  bool ok = true;                   // no wait ran out
  const uint4* rp = nullptr;
  auto stream_at = [&](int strip, int c) {
    const int l = layer_of(strip);
    return L.wp[l] + (static_cast<size_t>(strip - L.strip0[l]) * kbs + (c_lo + c) * kGemvChunk) * (kW4TileBytes / 16);
  };
  auto request = [&]() {
    if (ru >= u1) return;
    const bool end = rc + 1 == chunks;
    if (lane == 0 && !(a.stall && asked == 0)) {
      const uint32_t bytes = (end ? end_tiles : kGemvChunk) * kW4TileBytes;
      mbar_arrive_expect_tx(&full[warp], bytes);
      bulk_load(buffer, rp, bytes, &full[warp]);
    }
    ++asked;
    ++ru;
    ++rc;
    rp += kGemvChunkBytes / 16;
    if (end) {
      rc = 0;
      ++rs;
      if (ru < u1) rp = stream_at(rs, 0);
    }
  };
  auto begin = [&](int round) {
    first = strip_lo;
    count = strip_n;
    if (MANY) {
      first += static_cast<int>(static_cast<long long>(round) * strip_n / a.rounds);
      count = strip_lo + static_cast<int>(static_cast<long long>(round + 1) * strip_n / a.rounds) - first;
    }
    units = count * chunks;
    u0 = static_cast<int>(static_cast<long long>(warp) * units / kGemvWarps);
    u1 = static_cast<int>(static_cast<long long>(warp + 1) * units / kGemvWarps);
    ru = u0;
    rc = c = u0 % chunks;
    rs = strip = first + u0 / chunks;
    if (u0 < u1) rp = stream_at(strip, c);
  };
  if (lane == 0) {
    mbar_init(&full[warp], 1);
    if (warp == 0) mbar_init(&x_full, 1);
    fence_barrier_init();
  }
  __syncwarp();
  begin(0);
  if (lane == 0 && u0 < u1) prefetch_l2(rp, (c + 1 == chunks ? end_tiles : kGemvChunk) * kW4TileBytes);

  // where the scales of rows g and g + 8 lie, from the next chunk on
  const bool even = a.K % kGemvChunkCols == 0;
  const __half *p0 = nullptr, *p1 = nullptr;
  int left0 = 0, left1 = 0;                       // of the row; none behind the last row
  auto rows_of = [&](int strip, int c) {
    const int l = layer_of(strip);
    const int row = (strip - L.strip0[l]) * 16 + g, at = (c_lo + c) * NS;
    p0 = L.ws[l] + static_cast<size_t>(row) * a.G + at;
    p1 = p0 + static_cast<size_t>(8) * a.G;
    left0 = row < L.N[l] ? a.G - at : 0;
    left1 = row + 8 < L.N[l] ? a.G - at : 0;
  };
  ChunkScales<NS> c0, c1, n0, n1;
  auto first_scales = [&]() {
    if (u0 >= u1) return;
    rows_of(strip, c);
    c0.load(p0, left0, even);
    c1.load(p1, left1, even);
  };
  // activations to shared memory; columns behind K are zeros
  const int padded = chunks * kGemvChunkCols;
  const int row_bytes = min(padded, a.K - c_lo * kGemvChunkCols) * 2, pad16 = (padded * 2 - row_bytes) / 16;
  for (int i = threadIdx.x; i < a.M * pad16; i += kGemvThreads)
    *reinterpret_cast<uint4*>(xs_mem + i / pad16 * x_stride + row_bytes + i % pad16 * 16) = make_uint4(0, 0, 0, 0);
  grid_launch_dependents();
  grid_wait_dependencies();         // whatever the call reads may have been written just before
  request();
  if (threadIdx.x == 0) {
    mbar_arrive_expect_tx(&x_full, a.M * row_bytes);
    for (int m = 0; m < a.M; ++m)
      bulk_load(xs_mem + m * x_stride, static_cast<const T*>(a.x) + m * a.ldx + c_lo * kGemvChunkCols,
                row_bytes, &x_full);
  }
  first_scales();
  __syncthreads();                  // x_full is initialised; the padding is written
  ok = __syncthreads_and(mbar_wait(&x_full, 0, a.wait_limit_ns));
  if (!ok && threadIdx.x == 0) record_status(a.status, kStatusTimeout, 2);

  // a column of the product without a token is computed and dropped
  const uint8_t* x = xs_mem + min(g, a.M - 1) * x_stride + t * 16;
  int xo[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) xo[n] = g + 8 * n < a.M ? 8 * n * x_stride : 0;
  auto store = [&](int strip, int n, const float4& f) {
    const int l = layer_of(strip);
    const int row = (strip - L.strip0[l]) * 16 + g;
    T* y = static_cast<T*>(L.y[l]) + row;
    const float v[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = n * 8 + 2 * t + (i & 1);
      if (m < a.M && row + 8 * (i >> 1) < L.N[l])
        y[m * L.ldy[l] + 8 * (i >> 1)] = Elem<T>::from_float(v[i] * Elem<T>::kUnit);
    }
  };
  // a CTA's sums of a strip: results without a cluster
  auto finish = [&](int strip, const float (&v)[NT][4]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float4 f = make_float4(v[n][0], v[n][1], v[n][2], v[n][3]);
      if (a.split == 1) store(strip, n, f);
      else slab[((strip - first) * NT + n) * 32 + lane] = f;
    }
  };
  uint32_t parity = 0;
#pragma unroll 1
  for (int round = 0;;) {
  float acc[NT][4] = {};
  bool whole = c == 0;              // the strip's first chunk is this warp's
#pragma unroll 1
  for (int u = u0; ok && u < u1; ++u, parity ^= 1) {
    const bool end = c + 1 == chunks;
    if (u + 1 < u1) {               // the next chunk's scales
      if (end) {
        rows_of(strip + 1, 0);
      } else {
        p0 += NS;
        p1 += NS;
        left0 -= NS;
        left1 -= NS;
      }
      n0.load(p0, left0, even);
      n1.load(p1, left1, even);
    }
    if (!__all_sync(0xFFFFFFFFu, mbar_test_wait(smem_u32(&full[warp]), parity))) {
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&full[warp], parity, a.wait_limit_ns));
      if (!ok) {
        if (lane == 0) record_status(a.status, kStatusTimeout, 2);
        break;
      }
    }
    const uint4* tile = reinterpret_cast<const uint4*>(buffer) + lane;
    uint4 w[kGemvChunk][2];
#pragma unroll
    for (int i = 0; i < kGemvChunk; ++i) {
      w[i][0] = tile[i * 64];
      w[i][1] = tile[i * 64 + 32];
    }
    __syncwarp();                   // every lane holds the chunk
    request();                      // the next one comes while this one is multiplied
    const uint8_t* xp = x + c * (kGemvChunkCols * 2);
    if (!end || end_tiles == kGemvChunk) {
#pragma unroll
      for (int i = 0; i < kGemvChunk; ++i)
        gemv_tile<T, WPG, NS, NT>(acc, w[i][0], w[i][1], xp, xo, c0, c1, i);
    } else {
#pragma unroll
      for (int i = 0; i < kGemvChunk; ++i)
        if (i < end_tiles) gemv_tile<T, WPG, NS, NT>(acc, w[i][0], w[i][1], xp, xo, c0, c1, i);
    }
    c0 = n0;
    c1 = n1;
    ++c;
    if (end) {
      if (whole) {
        finish(strip, acc);
      } else {
#pragma unroll
        for (int n = 0; n < NT; ++n)
          head_of[warp][n][lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
      }
      whole = true;
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
      c = 0;
      ++strip;
    }
  }
  if (!ok) {                        // let the copies in flight land
    mbar_wait(&x_full, 0, a.wait_limit_ns);
    if (asked > 0) mbar_wait(&full[warp], (asked - 1) & 1, a.wait_limit_ns);
  }
  const bool open = u0 < u1 && c > 0;           // the last strip goes on behind this warp
  if (open && !whole) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
      head_of[warp][n][lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
  }
  __syncthreads();
  if (open && whole) {
    const int end = (strip - first + 1) * chunks;
    for (int w2 = warp + 1; w2 < kGemvWarps; ++w2) {
      const int b0 = static_cast<int>(static_cast<long long>(w2) * units / kGemvWarps);
      const int b1 = static_cast<int>(static_cast<long long>(w2 + 1) * units / kGemvWarps);
      if (b0 >= end) break;
      if (b0 == b1) continue;                   // a warp without chunks
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float4 v = head_of[w2][n][lane];
        acc[n][0] += v.x;
        acc[n][1] += v.y;
        acc[n][2] += v.z;
        acc[n][3] += v.w;
      }
    }
    finish(strip, acc);
  }
  if (a.split == 1) return;         // in one round
  const int round_first = first, round_count = count;
  if (MANY && ++round < a.rounds) { // its first chunk comes while the sums are added
    begin(round);
    if (ok) request();
    first_scales();
  }
  cluster_sync_all();
  // the ranks' sums of every strip, a share of them each
  for (int i = rank * kGemvWarps + warp; i < round_count * NT; i += a.split * kGemvWarps) {
    const uint32_t at = smem_u32(slab + i * 32 + lane);
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float4 v[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      v[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (r < a.split)
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v[r].x), "=f"(v[r].y), "=f"(v[r].z), "=f"(v[r].w)
                     : "r"(map_to_rank(at, r)) : "memory");
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      sum.x += v[r].x;
      sum.y += v[r].y;
      sum.z += v[r].z;
      sum.w += v[r].w;
    }
    store(round_first + i / NT, i % NT, sum);
  }
  // no CTA leaves, or writes its sums again, while another reads them
  cluster_sync_all();
  if (!MANY || round == a.rounds) return;
  }
}

}  // namespace flexq

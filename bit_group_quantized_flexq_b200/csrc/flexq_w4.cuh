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

#include "flexq_ptx.cuh"
#include "flexq_quant.cuh"

namespace flexq {

// ------------------------------------------------------------ packed form --
// Rows are padded to a multiple of 16 and columns to a multiple of 128 (code
// 0).  Tile (nt, kb) = rows 16 nt .. +15, columns 128 kb .. +127 is 1024
// contiguous bytes at (nt * kbs + kb) * 1024; row r of it is 64 bytes at
// 64 r; its 16-byte chunk t holds four little-endian words, and word w the
// eight codes of columns 32 w + 8 t .. +7 as u = q + 8, column i in nibble
// i / 2 + 4 * (i % 2).
//
// Why: a warp's 16-byte loads of a tile cover 512 contiguous bytes, lane
// (4 r + t) holding row r's chunk t, which is the register layout of an
// m16n8k16 MMA's A operand up to the order of k; that order is chosen so that
// the lane's activations for one word are 16 contiguous bytes too.  The
// nibble order puts consecutive columns into the two halves of a register
// with one mask.  A row's 128 codes stay within 64 aligned bytes (two DRAM
// sectors), so that rows can also be looked up alone.
constexpr int kW4TileRows = 16;
constexpr int kW4TileCols = 128;
constexpr int kW4TileBytes = 1024;

__host__ __device__ inline int w4_row_tiles(int N) { return (N + 15) / 16; }
__host__ __device__ inline int w4_col_tiles(int K) { return (K + 127) / 128; }

// Byte offset of the word of columns k .. k+7 (k % 8 == 0) of row n.
__device__ __forceinline__ size_t w4_word_offset(int n, int k, int kbs) {
  return (static_cast<size_t>(n >> 4) * kbs + (k >> 7)) * kW4TileBytes + (n & 15) * 64 +
         ((k >> 3) & 3) * 16 + ((k >> 5) & 3) * 4;
}

// Code i (0..7) of a word.
__device__ __forceinline__ int w4_code(uint32_t word, int i) {
  return static_cast<int>((word >> (4 * (i / 2 + 4 * (i & 1)))) & 15u) - 8;
}

// --------------------------------------------------------------- quantizer --
// Offline, two passes over W (the scales, then the codes): not timed.
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
      word |= static_cast<uint32_t>(q + 8) << (4 * (j / 2 + 4 * (j & 1)));
    }
  }
  packed[i] = word;
}

// ---------------------------------------------------------- element types --
template <typename T>
struct Elem;

template <>
struct Elem<__half> {
  using Pair = __half2;
  static __device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  // The eight codes of a word as exact FP16 pairs of consecutive columns.  A
  // nibble in the low mantissa bits of 1024 is 1024 + u; four bits further up
  // it is 1024 + 16 u, brought down by an exact multiply-add.
  static __device__ __forceinline__ void codes(uint32_t w, uint32_t (&p)[4]) {
    const __half2 off = __half2half2(__ushort_as_half(0x6408));      // 1032
    const __half2 sixteenth = __half2half2(__ushort_as_half(0x2C00));   // 1/16
    const __half2 off16 = __half2half2(__ushort_as_half(0xD480));    // -72
    const uint32_t v = w >> 8;
    uint32_t b[4];
    b[0] = (w & 0x000F000Fu) | 0x64006400u;
    b[1] = (w & 0x00F000F0u) | 0x64006400u;
    b[2] = (v & 0x000F000Fu) | 0x64006400u;
    b[3] = (v & 0x00F000F0u) | 0x64006400u;
    __half2* h = reinterpret_cast<__half2*>(b);
    __half2* o = reinterpret_cast<__half2*>(p);
    o[0] = __hsub2(h[0], off);
    o[1] = __hfma2(h[1], sixteenth, off16);
    o[2] = __hsub2(h[2], off);
    o[3] = __hfma2(h[3], sixteenth, off16);
  }
};

template <>
struct Elem<__nv_bfloat16> {
  using Pair = __nv_bfloat162;
  static __device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  // BF16 has 7 mantissa bits: a nibble in the low ones of 128 is 128 + u; the
  // other nibbles are shifted there first.
  static __device__ __forceinline__ void codes(uint32_t w, uint32_t (&p)[4]) {
    const __nv_bfloat162 off = __bfloat162bfloat162(__ushort_as_bfloat16(0x4308));   // 136
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
      const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&b), off);
      p[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
};

// ---------------------------------------------------- matrix-vector product --
constexpr int kW4MaxLayers = 4;
constexpr int kGemvWarps = 8;
constexpr int kGemvThreads = kGemvWarps * 32;

// The layers of one launch: they read the same activations.
struct W4Layers {
  const uint4* wp[kW4MaxLayers];
  const __half* ws[kW4MaxLayers];
  void* y[kW4MaxLayers];
  long long ldy[kW4MaxLayers];
  int N[kW4MaxLayers];
  int block0[kW4MaxLayers + 1];   // first block (in x) of each layer
  int n;
};

struct GemvArgs {
  const void* x;
  long long ldx;
  int M, K, G, kbs, gs_shift;     // kbs: tiles of 128 columns; gs = 1 << gs_shift
};

// Registers of one step: a 16 x 128 tile per strip and the batch's
// activations for its columns.
template <int NT, int S>
struct GemvStep {
  uint4 w[S][2];                  // rows g and g + 8 of each strip
  uint4 x[NT][4];                 // per word: eight columns of token g
};

// One CTA: S * 16 rows of one layer, all of K (or its cluster rank's share),
// NT * 8 tokens.  The warps take the tiles of 128 columns in turn; each
// multiplies its codes (exact in FP16 and BF16) with the activations on the
// tensor core in FP32 and adds a group's sum times the scale, in FP32, to its
// totals.  The warps' totals are added in shared memory, the cluster's in
// distributed shared memory, always in the same order.
template <typename T, int NT, int S, int WPG>
__global__ void __launch_bounds__(kGemvThreads) w4_gemv_kernel(const __grid_constant__ W4Layers L,
                                                              const GemvArgs a) {
  constexpr int kRows = 16 * S, kTok = 8 * NT;
  __shared__ float red[kGemvWarps][S * NT * 4][32];
  __shared__ float tot[kRows * kTok];
  int l = 0;
  while (l + 1 < L.n && static_cast<int>(blockIdx.x) >= L.block0[l + 1]) ++l;
  const int strip0 = (static_cast<int>(blockIdx.x) - L.block0[l]) * S;
  const int N = L.N[l], strips = w4_row_tiles(N);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int m0 = blockIdx.y * kTok;
  const int ks = gridDim.z, rank = blockIdx.z;
  const T* x = static_cast<const T*>(a.x);
  const uint4* wp = L.wp[l] + static_cast<size_t>(strip0) * a.kbs * (kW4TileBytes / 16);
  const __half* ws = L.ws[l];

  float acc[S][NT][4] = {};
  auto load = [&](GemvStep<NT, S>& st, int kb) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const bool in = strip0 + s < strips;
      const uint4* p = wp + (static_cast<size_t>(s) * a.kbs + kb) * (kW4TileBytes / 16) + lane;
      const uint4 zero = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
      st.w[s][0] = in ? __ldcs(p) : zero;
      st.w[s][1] = in ? __ldcs(p + 32) : zero;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int m = m0 + nt * 8 + g;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int k = kb * 128 + w * 32 + t * 8;
        st.x[nt][w] = (m < a.M && k < a.K)
                          ? __ldg(reinterpret_cast<const uint4*>(x + m * a.ldx + k))
                          : make_uint4(0, 0, 0, 0);
      }
    }
  };
  const int stride = kGemvWarps * ks;
  int kb = rank * kGemvWarps + warp;
  GemvStep<NT, S> cur, nxt;
  if (kb < a.kbs) load(cur, kb);
  for (; kb < a.kbs; kb += stride) {
    if (kb + stride < a.kbs) load(nxt, kb + stride);
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int row = (strip0 + s) * 16 + g;
      float part[NT][4] = {};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t lo[4], hi[4];
        const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&cur.w[s][0]);
        const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&cur.w[s][1]);
        Elem<T>::codes(w0[w], lo);
        Elem<T>::codes(w1[w], hi);
        const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]};
        const uint32_t a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          Elem<T>::mma(part[nt], a0, cur.x[nt][w].x, cur.x[nt][w].y);
          Elem<T>::mma(part[nt], a1, cur.x[nt][w].z, cur.x[nt][w].w);
        }
        if ((w + 1) % WPG == 0) {
          const int k = kb * 128 + w * 32;
          const int grp = k >> a.gs_shift;
          const float s0 = (row < N && k < a.K)
                               ? __half2float(__ldg(ws + static_cast<size_t>(row) * a.G + grp)) : 0.0f;
          const float s1 = (row + 8 < N && k < a.K)
                               ? __half2float(__ldg(ws + static_cast<size_t>(row + 8) * a.G + grp)) : 0.0f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            acc[s][nt][0] = fmaf(part[nt][0], s0, acc[s][nt][0]);
            acc[s][nt][1] = fmaf(part[nt][1], s0, acc[s][nt][1]);
            acc[s][nt][2] = fmaf(part[nt][2], s1, acc[s][nt][2]);
            acc[s][nt][3] = fmaf(part[nt][3], s1, acc[s][nt][3]);
            part[nt][0] = part[nt][1] = part[nt][2] = part[nt][3] = 0.0f;
          }
        }
      }
    }
    cur = nxt;
  }
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[warp][(s * NT + nt) * 4 + i][lane] = acc[s][nt][i];
  __syncthreads();
  // tot[token][row]: value i of lane (g, t) is row g + 8 (i / 2), token 2 t + i % 2
  for (int o = threadIdx.x; o < kRows * kTok; o += kGemvThreads) {
    const int row = o % kRows, tok = o / kRows;
    const int s = row >> 4, nt = tok >> 3;
    const int i = ((row >> 3) & 1) * 2 + (tok & 1), ln = (row & 7) * 4 + ((tok & 7) >> 1);
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kGemvWarps; ++w) v += red[w][(s * NT + nt) * 4 + i][ln];
    tot[o] = v;
  }
  if (ks > 1) cluster_sync_all(); else __syncthreads();
  // the cluster's CTAs share the outputs; each adds the ranks' totals in order
  T* y = static_cast<T*>(L.y[l]);
  for (int o = rank * kGemvThreads + threadIdx.x; o < kRows * kTok; o += kGemvThreads * ks) {
    const int row = strip0 * 16 + o % kRows, m = m0 + o / kRows;
    float v = 0.0f;
    if (ks == 1) {
      v = tot[o];
    } else {
      for (int r = 0; r < ks; ++r) {
        const uint32_t p = map_to_rank(smem_u32(&tot[o]), r);
        float u;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(u) : "r"(p) : "memory");
        v += u;
      }
    }
    if (row < N && m < a.M) y[m * L.ldy[l] + row] = Elem<T>::from_float(v);
  }
  if (ks > 1) cluster_sync_all();   // no CTA leaves while another reads its totals
}

}  // namespace flexq

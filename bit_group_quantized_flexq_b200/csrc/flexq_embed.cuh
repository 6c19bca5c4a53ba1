// flexq_embed.cuh -- rows of a packed weight table: lookup with scaling, and
// its gradient by sorted tokens.
//
//   y[t,k]  = a * q[id_t,k] * s[id_t, k / gs]
//   D[v,k]  = a * sum over t with id_t = v of dy[t,k]   (in the order of t)
//   ds[v,g] = sum over k in g of D[v,k] * q[v,k]
//
// The codes are constants; D is the gradient of the rows of a latent table
// whose rounding is passed through, ds the exact gradient of the scales.  A
// token outside [0, V) is padding: a zero row, and no gradient.  Tables are
// in the 4-bit form of flexq_w4.cuh (scales [V, G]) or in the byte-aligned
// 6-bit form of flexq_quant.cuh (scales [G, V]).
#pragma once

#include "flexq_w4.cuh"

namespace flexq {

struct Table {
  const uint8_t* packed;
  const __half* scales;
  int V, K, G, kbs, gs_shift;       // kbs: tiles of 128 columns, gs = 1 << gs_shift
};

// Where a row's codes begin in a table.
template <int BITS>
__device__ __forceinline__ size_t row_offset(const Table& tb, int v) {
  return BITS == 4 ? static_cast<size_t>(v >> 4) * tb.kbs * kW4TileBytes + (v & 15) * 64
                   : static_cast<size_t>(v >> 7) * tb.kbs * 12288 + (v & 127) * 16;
}

// The packed codes of eight columns k .. k+7 (k % 8 == 0) of a row: one word of
// the 4-bit form, or the three words of the 16-code block that holds them.
template <int BITS>
struct Codes8 {
  static constexpr int kWords = BITS == 4 ? 1 : 3;
  uint32_t w[kWords];

  // The words' places from the row's beginning.
  static __device__ __forceinline__ void places(int k, uint32_t (&at)[kWords]) {
    if (BITS == 4) {
      at[0] = static_cast<uint32_t>(k >> 7) * kW4TileBytes + ((k >> 3) & 3) * 16 + ((k >> 5) & 3) * 4;
    } else {
      // a row's 96 bytes of 128 codes lie in 16-byte chunks 128 rows apart
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int o = 12 * ((k >> 4) & 7) + 4 * i;
        at[i] = static_cast<uint32_t>(k >> 7) * 12288 + (o >> 4) * 2048 + (o & 15);
      }
    }
  }
  __device__ __forceinline__ void load(const uint8_t* row, const uint32_t (&at)[kWords]) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(row + at[i]));
  }
  __device__ __forceinline__ void load(const Table& tb, int v, int k) {
    uint32_t at[kWords];
    places(k, at);
    load(tb.packed + row_offset<BITS>(tb, v), at);
  }

  // The codes as FP32.
  __device__ __forceinline__ void get(int k, float (&q)[8]) const {
    if (BITS == 4) {
      uint32_t p[4];
      Elem<__half>::codes(w[0], p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = Elem<__half>::unpack(p[i]);
        q[2 * i] = f.x;
        q[2 * i + 1] = f.y;
      }
    } else {
      // byte t of word i holds code 4 i + t in bits [7:2] and bits [2i+1:2i] of
      // code 12 + t in bits [1:0]
      const uint32_t w0 = w[0], w1 = w[kWords / 2], w2 = w[kWords - 1];
      const bool upper = k & 8;
      const uint32_t first = upper ? w2 : w0;
      const uint32_t last = (w0 & 0x03030303u) << 2 | (w1 & 0x03030303u) << 4 | (w2 & 0x03030303u) << 6;
      const uint32_t second = upper ? last : w1;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        q[t] = static_cast<float>(static_cast<int8_t>(first >> (8 * t)) >> 2);
        q[4 + t] = static_cast<float>(static_cast<int8_t>(second >> (8 * t)) >> 2);
      }
    }
  }
};

template <int BITS>
__device__ __forceinline__ size_t scale_index(const Table& tb, int v, int grp) {
  return BITS == 4 ? static_cast<size_t>(v) * tb.G + grp : static_cast<size_t>(grp) * tb.V + v;
}

// The token's row, or -1 for padding.
__device__ __forceinline__ int token_row(const void* ids, int id_bytes, long long t, int V) {
  const long long id = id_bytes == 8 ? __ldg(static_cast<const long long*>(ids) + t)
                                     : __ldg(static_cast<const int*>(ids) + t);
  return id >= 0 && id < V ? static_cast<int>(id) : -1;
}

// ------------------------------------------------------------------ lookup --
// Bound by writing the rows: 16 bytes a thread, consecutive threads and then
// consecutive CTAs write consecutive pieces.  A thread keeps its columns and takes
// a few tokens at a time, so that their ids, then their codes and scales, are in
// flight together: four with 4 bits (16384 tokens x 8192 take 62 us, with two 69),
// two with 6, whose codes are three words (4096 tokens x 4096 15.4 us, with four
// 16.3).  62 us are 4.7 TB/s; asking for the next tokens' ids meanwhile costs more
// in registers than it hides (66 to 76 us).  One token takes 1.7 us.
constexpr int kLookThreads = 256;
constexpr int kLookCols = kLookThreads * 8;
__host__ __device__ constexpr int look_ahead(int bits) { return bits == 4 ? 4 : 2; }

template <typename T, int BITS>
__global__ void __launch_bounds__(kLookThreads) embed_kernel(const Table tb, const void* __restrict__ ids,
                                                             int id_bytes, int tokens, float scale,
                                                             T* __restrict__ out) {
  constexpr int kLookAhead = look_ahead(BITS);
  const int k = blockIdx.x * kLookCols + threadIdx.x * 8;   // consecutive CTAs write a row's pieces
  if (k >= tb.K) return;
  const int grp = k >> tb.gs_shift;
  for (long long t0 = static_cast<long long>(blockIdx.y) * kLookAhead; t0 < tokens;
       t0 += static_cast<long long>(gridDim.y) * kLookAhead) {
    int v[kLookAhead];
#pragma unroll
    for (int j = 0; j < kLookAhead; ++j)
      v[j] = t0 + j < tokens ? token_row(ids, id_bytes, t0 + j, tb.V) : -1;
    Codes8<BITS> c[kLookAhead];
    __half s[kLookAhead];
#pragma unroll
    for (int j = 0; j < kLookAhead; ++j)
      if (v[j] >= 0) {
        c[j].load(tb, v[j], k);
        s[j] = __ldg(tb.scales + scale_index<BITS>(tb, v[j], grp));
      }
#pragma unroll
    for (int j = 0; j < kLookAhead; ++j) {
      if (t0 + j >= tokens) break;
      uint4 o = make_uint4(0, 0, 0, 0);
      if (v[j] >= 0) {
        float q[8];
        c[j].get(k, q);
        const float f = __half2float(s[j]);
        uint32_t* p = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
        for (int i = 0; i < 4; ++i) {    // code * scale is exact in FP32
          const float2 x = __fmul2_rn(__fmul2_rn(make_float2(q[2 * i], q[2 * i + 1]), make_float2(f, f)),
                                      make_float2(scale, scale));
          p[i] = Elem<T>::pack(x.x, x.y);
        }
      }
      __stcs(reinterpret_cast<uint4*>(out + static_cast<size_t>(t0 + j) * tb.K + k), o);
    }
  }
}

// -------------------------------------------------------------------- sort --
// Tokens sorted by row, equal rows in the order of the tokens (stable), by a
// least-significant-digit radix sort of 8-bit digits.  One cluster sorts;
// its CTAs exchange digit counts in distributed shared memory and meet at
// the cluster's barrier, so that one launch does every pass.  The grid's
// other clusters meanwhile zero the scales' gradient and what of the rows'
// they can in that time; the rest of it, but for the rows with a token, is
// zeroed beside the sums.  Bound by latency: 8192 tokens of 32000 rows take two
// passes and 17 us, the chain of digit counts, barriers and places of each.  More
// CTAs than a cluster holds would meet in global memory.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortDigits = 256;

struct SortArgs {
  const void* ids;
  int id_bytes;
  int T, V, passes;
  uint2* buf[2];                  // (row, token); padding has row V
  uint4* fill[2];                 // outputs to zero, in 16-byte pieces, and their ends
  long long fill_n[2];
  float* tail;                    // the last 0..3 floats of the second output
  int tail_n;
  unsigned* present;              // a bit per row that has a token, or null
  int clusters_size;              // CTAs of the sorting cluster
};

__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const SortArgs a) {
  __shared__ unsigned hist[kSortWarps][kSortDigits + 1];   // the odd stride spreads a digit's column
  __shared__ unsigned total[kSortDigits];
  __shared__ unsigned base[kSortDigits];
  __shared__ unsigned warp_sum[kSortDigits / 32];
  const int C = a.clusters_size;
  grid_launch_dependents();         // the sums wait for this kernel's end
  if (static_cast<int>(blockIdx.x) >= C) {
    const long long stride = static_cast<long long>(gridDim.x - C) * kSortThreads;
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll 4
      for (long long i = static_cast<long long>(blockIdx.x - C) * kSortThreads + threadIdx.x;
           i < a.fill_n[f]; i += stride)
        a.fill[f][i] = make_uint4(0, 0, 0, 0);
    if (static_cast<int>(blockIdx.x) == C && static_cast<int>(threadIdx.x) < a.tail_n)
      a.tail[threadIdx.x] = 0.0f;
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned below = (1u << lane) - 1u;
  const int rank = blockIdx.x;
  // each warp owns a run of consecutive tokens; the first kKeep of a lane stay
  // in registers between counting and placing them
  constexpr int kKeep = 4;
  const long long per_warp = ((static_cast<long long>(a.T) + kSortWarps * C - 1) / (kSortWarps * C) + 31) / 32 * 32;
  const long long lo = min(static_cast<long long>(a.T), (static_cast<long long>(rank) * kSortWarps + warp) * per_warp);
  const long long hi = min(static_cast<long long>(a.T), lo + per_warp);

  if (a.present)                    // in place before the first tokens are placed
    for (int i = rank * kSortThreads + threadIdx.x; i < (a.V + 31) / 32; i += C * kSortThreads) a.present[i] = 0;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = 8 * pass;
    const uint2* src = a.buf[(pass + 1) & 1];
    uint2* dst = a.buf[pass & 1];
    auto item = [&](long long i) {
      if (i >= hi) return make_uint2(0, 0);
      if (pass == 0) {
        const int v = token_row(a.ids, a.id_bytes, i, a.V);
        return make_uint2(v < 0 ? a.V : v, static_cast<unsigned>(i));
      }
      return __ldcg(src + i);
    };
    // the lanes whose token has this lane's digit
    auto alike = [&](unsigned d, bool in) {
      unsigned same = __ballot_sync(0xFFFFFFFFu, in);
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        const unsigned set = __ballot_sync(0xFFFFFFFFu, d >> b & 1u);
        same &= d >> b & 1u ? set : ~set;
      }
      return same;
    };
    auto count = [&](const uint2& it, bool in) {
      const unsigned d = (it.x >> shift) & 255u, same = alike(d, in);
      if (in && (same & below) == 0) hist[warp][d] += __popc(same);
      __syncwarp();
    };
    auto place = [&](const uint2& it, bool in) {
      const unsigned d = (it.x >> shift) & 255u, same = alike(d, in);
      const unsigned at = hist[warp][d];
      __syncwarp();
      if (in) {
        dst[base[d] + at + __popc(same & below)] = it;
        if (pass == 0 && a.present && it.x < static_cast<unsigned>(a.V)) atomicOr(&a.present[it.x >> 5], 1u << (it.x & 31));
        if ((same & below) == 0) hist[warp][d] = at + __popc(same);
      }
      __syncwarp();
    };
    uint2 kept[kKeep];
#pragma unroll
    for (int r = 0; r < kKeep; ++r) kept[r] = item(lo + 32 * r + lane);
    for (int i = lane; i < kSortDigits; i += 32) hist[warp][i] = 0;
    __syncwarp();
#pragma unroll
    for (int r = 0; r < kKeep; ++r)
      if (lo + 32 * r < hi) count(kept[r], lo + 32 * r + lane < hi);
    for (long long i0 = lo + 32 * kKeep; i0 < hi; i0 += 32) count(item(i0 + lane), i0 + lane < hi);
    __syncthreads();
    {                               // each warp's first place within the CTA, four threads to a digit
      const int d = threadIdx.x >> 2, q = threadIdx.x & 3;
      unsigned c[8], sum = 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        c[w] = hist[8 * q + w][d];
        sum += c[w];
      }
      unsigned incl = sum;
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        const unsigned up = __shfl_up_sync(0xFFFFFFFFu, incl, o, 4);
        if (q >= o) incl += up;
      }
      unsigned at = incl - sum;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        hist[8 * q + w][d] = at;
        at += c[w];
      }
      if (q == 3) total[d] = incl;
    }
    if (C > 1) cluster_sync_all(); else __syncthreads();
    unsigned all = 0, before = 0, incl = 0;
    if (threadIdx.x < kSortDigits) {
      if (C > 1) {
        unsigned c[8];              // all at once; C is 8
#pragma unroll
        for (int r = 0; r < 8; ++r)
          asm volatile("ld.shared::cluster.u32 %0, [%1];"
                       : "=r"(c[r]) : "r"(map_to_rank(smem_u32(&total[threadIdx.x]), r)) : "memory");
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          all += c[r];
          if (r < rank) before += c[r];
        }
      } else {
        all = total[threadIdx.x];
      }
      incl = all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += up;
      }
      if (lane == 31) warp_sum[warp] = incl;
    }
    __syncthreads();
    if (threadIdx.x < kSortDigits) {
      unsigned low = 0;
#pragma unroll
      for (int w = 0; w < kSortDigits / 32; ++w)
        if (w < warp) low += warp_sum[w];
      base[threadIdx.x] = low + incl - all + before;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kKeep; ++r)
      if (lo + 32 * r < hi) place(kept[r], lo + 32 * r + lane < hi);
    for (long long i0 = lo + 32 * kKeep; i0 < hi; i0 += 32) place(item(i0 + lane), i0 + lane < hi);
    // the next pass reads what every CTA of the cluster wrote, and none
    // clears its counts while another reads them
    if (C > 1) cluster_sync_all(); else __syncthreads();
  }
}

// -------------------------------------------------------------------- sums --
constexpr int kSumThreads = 256;
constexpr int kSumCols = kSumThreads * 8;
constexpr int kSumMaxTile = 64;

struct SumArgs {
  const uint2* sorted;
  const void* dy;
  int T, tile;                    // sorted tokens per CTA
  float scale;
  float* partial;                 // [tiles][2][K]: a tile's part of a run it shares with others
  void* table;                    // row gradient, or null
  float* scales;                  // scale gradient, or null
  const unsigned* present;        // rows of the table with a token
  int fill_row, sum_ctas, fill_ctas;    // rows from fill_row on are zeroed beside the sums
};

// Writes the finished sums of columns k .. k+7 of row v; codes: the row's, where
// the scales' gradient is wanted.  All threads of a warp take part (the group
// sums are shuffled); `in` says whose columns exist.
template <typename T, typename TO, int BITS>
__device__ __forceinline__ void embed_finish(const Table& tb, const SumArgs& a, int v, int k, bool in,
                                             const float (&acc)[8], const Codes8<BITS>& codes) {
  if (a.table && in) {
    float d[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = acc[i] * a.scale;
    TO* row = static_cast<TO*>(a.table) + static_cast<size_t>(v) * tb.K + k;
    if constexpr (sizeof(TO) == 4) {
      reinterpret_cast<float4*>(row)[0] = make_float4(d[0], d[1], d[2], d[3]);
      reinterpret_cast<float4*>(row)[1] = make_float4(d[4], d[5], d[6], d[7]);
    } else {
      uint4 o;
      o.x = Elem<T>::pack(d[0], d[1]);
      o.y = Elem<T>::pack(d[2], d[3]);
      o.z = Elem<T>::pack(d[4], d[5]);
      o.w = Elem<T>::pack(d[6], d[7]);
      *reinterpret_cast<uint4*>(row) = o;
    }
  }
  if (a.scales) {
    float sum = 0.0f;
    if (in) {
      float q[8];
      codes.get(k, q);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(acc[i], q[i], sum);
    }
    // gs / 8 threads per group: 4 .. 32
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
    if (tb.gs_shift > 5) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 4);
    if (tb.gs_shift > 6) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 8);
    if (tb.gs_shift > 7) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
    if (in && (k & ((1 << tb.gs_shift) - 1)) == 0)
      a.scales[scale_index<BITS>(tb, v, k >> tb.gs_shift)] = sum * a.scale;
  }
}

template <typename T>
__device__ __forceinline__ void add8(float (&acc)[8], const uint4& x) {
  const uint32_t* p = reinterpret_cast<const uint32_t*>(&x);
  float2* a = reinterpret_cast<float2*>(acc);
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = __fadd2_rn(a[i], Elem<T>::unpack(p[i]));
}

// Copies into shared memory that the copying thread alone reads: it waits for
// its own groups of them.
__device__ __forceinline__ void async_copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void async_copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One CTA: a tile of consecutive sorted tokens, 4096 columns.  Runs of equal
// rows inside the tile are finished here; what a run has in a tile that it
// shares with others goes to `partial` and is joined by embed_join_kernel, so
// that a row with many tokens is spread over many CTAs and every sum has one
// fixed order.  Bound by reading dY: a thread takes two pieces of eight
// columns, 2048 apart, and keeps six tokens' values (and the codes of the rows
// that end with them) on the way into shared memory; what there is to know of
// a token is worked out once per tile.  (With the values on the way to
// registers instead, a wait for one token's waited for the next ones' too:
// 16384 tokens x 8192 took 100 us for 66.)  The zeros of the rows without a
// token are written by CTAs in between: 8192 tokens and 32000 x 4096 BF16 rows
// take 73 us in all three launches, FP32 rows 108; the bytes alone (262 or 524
// MB of rows, 67 of dY) are 51 and 91 us at a copy's rate.
template <int BITS>
struct SumRing {
  static constexpr int kStages = 6;
  uint4 x[kStages][2][kSumThreads];
  uint32_t codes[kStages][2][Codes8<BITS>::kWords][kSumThreads];
};

template <typename T, typename TO, int BITS>
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const Table tb, const SumArgs a) {
  enum { kGoOn, kFinish, kBegun, kOpen };             // what follows a token's values
  struct __align__(16) Item {
    const T* dy;                                      // its values
    const uint8_t* codes;                             // its row's
    int row, next;
  };
  extern __shared__ __align__(16) uint8_t ring_mem[];
  SumRing<BITS>& ring = *reinterpret_cast<SumRing<BITS>*>(ring_mem);
  constexpr int D = SumRing<BITS>::kStages;
  __shared__ Item items[kSumMaxTile];
  __shared__ int valid;
  const int tid = threadIdx.x;
  grid_launch_dependents();
  grid_wait_dependencies();
  // sums and zeros take turns, so that dY is read while zeros are written
  const int pairs = min(a.sum_ctas, a.fill_ctas), block = blockIdx.x;
  const bool fills = block < 2 * pairs ? block & 1 : a.fill_ctas > a.sum_ctas;
  const int id = block < 2 * pairs ? block >> 1 : block - pairs;
  if (fills) {
    const int rows = tb.V - a.fill_row;
    const int lo = a.fill_row + static_cast<int>(static_cast<long long>(id) * rows / a.fill_ctas);
    const int hi = a.fill_row + static_cast<int>(static_cast<long long>(id + 1) * rows / a.fill_ctas);
    const int pieces = tb.K * static_cast<int>(sizeof(TO)) / 16;
    for (int v = lo; v < hi; ++v) {
      if (a.present[v >> 5] >> (v & 31) & 1u) continue;
      uint4* row = reinterpret_cast<uint4*>(static_cast<TO*>(a.table) + static_cast<size_t>(v) * tb.K);
      for (int i = tid; i < pieces; i += kSumThreads) row[i] = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const int tiles = static_cast<int>((static_cast<long long>(a.T) + a.tile - 1) / a.tile);
  const int tile = id % tiles, column = id / tiles;
  const long long p0 = static_cast<long long>(tile) * a.tile;
  if (tid == 0) valid = 0;
  __syncthreads();
  if (tid < a.tile && p0 + tid < a.T) {
    const long long p = p0 + tid, end = min(p0 + a.tile, static_cast<long long>(a.T));
    const uint2 it = a.sorted[p];
    if (it.x < static_cast<unsigned>(tb.V)) {         // padding sorts last
      const unsigned behind = p + 1 < a.T ? a.sorted[p + 1].x : 0xFFFFFFFFu;
      const bool begun = p0 > 0 && a.sorted[p0 - 1].x == it.x;
      Item item;
      item.dy = static_cast<const T*>(a.dy) + static_cast<size_t>(it.y) * tb.K;
      item.codes = tb.packed + row_offset<BITS>(tb, static_cast<int>(it.x));
      item.row = static_cast<int>(it.x);
      item.next = behind == it.x && p + 1 < end ? kGoOn : begun ? kBegun : behind == it.x ? kOpen : kFinish;
      items[tid] = item;
      atomicMax(&valid, tid + 1);
    }
  }
  __syncthreads();
  const int n = valid;
  const int k0 = column * (2 * kSumCols) + tid * 8;
  uint32_t at[2][Codes8<BITS>::kWords];
  Codes8<BITS>::places(k0, at[0]);
  Codes8<BITS>::places(k0 + kSumCols, at[1]);
  auto request = [&](int i, int slot) {
    if (i < n) {
      const Item& it = items[i];
      const bool codes = a.scales && it.next == kFinish;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int k = k0 + u * kSumCols;
        if (k < tb.K) {
          async_copy16(smem_u32(&ring.x[slot][u][tid]), it.dy + k);
          if (codes)
#pragma unroll
            for (int w = 0; w < Codes8<BITS>::kWords; ++w)
              async_copy4(smem_u32(&ring.codes[slot][u][w][tid]), it.codes + at[u][w]);
        }
      }
    }
    async_commit();
  };
#pragma unroll
  for (int i = 0; i < D; ++i) request(i, i);
  float acc[2][8] = {};
  int slot = 0;
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    async_wait<D - 1>();
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (k0 + u * kSumCols < tb.K) add8<T>(acc[u], ring.x[slot][u][tid]);
    const int next = items[i].next;
    if (next != kGoOn) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int k = k0 + u * kSumCols;
        if (next == kFinish) {
          Codes8<BITS> codes;
#pragma unroll
          for (int w = 0; w < Codes8<BITS>::kWords; ++w) codes.w[w] = ring.codes[slot][u][w][tid];
          embed_finish<T, TO, BITS>(tb, a, items[i].row, k, k < tb.K, acc[u], codes);
        } else if (k < tb.K) {
          float4* p = reinterpret_cast<float4*>(
              a.partial + (static_cast<size_t>(tile) * 2 + (next == kOpen ? 1 : 0)) * tb.K + k);
          p[0] = make_float4(acc[u][0], acc[u][1], acc[u][2], acc[u][3]);
          p[1] = make_float4(acc[u][4], acc[u][5], acc[u][6], acc[u][7]);
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[u][c] = 0.0f;
      }
    }
    request(i + D, slot);
    if (++slot == D) slot = 0;
  }
  async_wait<0>();
}

// Joins the run that starts in tile blockIdx.x and goes on into the next.  A
// chain of loads as long as the longest run, about 10 us for 8192 tokens with a
// few frequent rows.  (Sixteen parts at a time instead of eight, and zeros
// written beside them, took 5 to 12 us more.)
template <typename T, typename TO, int BITS>
__global__ void __launch_bounds__(kSumThreads) embed_join_kernel(const Table tb, const SumArgs a) {
  const long long end = (static_cast<long long>(blockIdx.x) + 1) * a.tile;   // of the tile
  grid_wait_dependencies();
  if (end >= a.T) return;
  const unsigned v = a.sorted[end - 1].x;
  if (v >= static_cast<unsigned>(tb.V) || a.sorted[end].x != v) return;
  const long long begin = end - a.tile;
  if (begin > 0 && a.sorted[begin].x == v && a.sorted[begin - 1].x == v) return;   // starts earlier
  const int k = blockIdx.y * kSumCols + threadIdx.x * 8;
  const bool in = k < tb.K;
  Codes8<BITS> codes;
  if (in && a.scales) codes.load(tb, static_cast<int>(v), k);
  float acc[8] = {};
  auto get = [&](size_t slot, float4 (&x)[2]) {
    const float4* p = reinterpret_cast<const float4*>(a.partial + slot * tb.K + k);
    x[0] = p[0];
    x[1] = p[1];
  };
  auto add = [&](const float4 (&x)[2]) {
    acc[0] += x[0].x; acc[1] += x[0].y; acc[2] += x[0].z; acc[3] += x[0].w;
    acc[4] += x[1].x; acc[5] += x[1].y; acc[6] += x[1].z; acc[7] += x[1].w;
  };
  if (in) {
    float4 x[2];
    get(static_cast<size_t>(blockIdx.x) * 2 + 1, x);
    add(x);
  }
  // the tiles behind that begin with v: 32 of them are asked at once, and
  // their parts come eight at a time
  const long long tiles = (static_cast<long long>(a.T) + a.tile - 1) / a.tile;
  for (long long t0 = static_cast<long long>(blockIdx.x) + 1;; t0 += 32) {
    const long long t = t0 + (threadIdx.x & 31);
    const unsigned same = __ballot_sync(0xFFFFFFFFu, t < tiles && a.sorted[t * a.tile].x == v);
    const int run = same == 0xFFFFFFFFu ? 32 : __ffs(~same) - 1;
    if (in)
      for (int i = 0; i < run; i += 8) {
        float4 x[8][2];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (i + j < run) get(static_cast<size_t>(t0 + i + j) * 2, x[j]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (i + j < run) add(x[j]);
      }
    if (run < 32) break;
  }
  embed_finish<T, TO, BITS>(tb, a, static_cast<int>(v), k, in, acc, codes);
}

// ------------------------------------------------------------- few tokens ----
// Up to 256 tokens take one launch: every CTA sorts them all by comparing each
// with each (about a microsecond for 256, less than the launches above), then
// takes its share of the runs' 2048-column pieces, and of the rows without a
// token, whose gradients it zeroes.  37 tokens and the scales of 32000 x 4096 in
// groups of 64: 7.5 us (9.3 with the three launches), 200 tokens 11.6 (19.8).
constexpr int kFewTokens = 256;

struct FewArgs {
  SumArgs sum;
  const void* ids;
  int id_bytes;
};

template <typename T, typename TO, int BITS>
__global__ void __launch_bounds__(kSumThreads) embed_few_kernel(const Table tb, const FewArgs f) {
  const SumArgs& a = f.sum;
  __shared__ int row_of[kFewTokens];                  // of each token; V for padding
  __shared__ uint2 items[kFewTokens + 1];             // sorted
  __shared__ int start[kFewTokens];                   // of each run, in the order of the rows
  __shared__ int runs_of[kFewTokens / 32];
  const int n = a.T, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < n) {
    const int v = token_row(f.ids, f.id_bytes, tid, tb.V);
    row_of[tid] = v < 0 ? tb.V : v;
  }
  __syncthreads();
  if (tid < n) {
    const int v = row_of[tid];
    int at = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) at += row_of[j] < v || (row_of[j] == v && j < tid);
    items[at] = make_uint2(static_cast<unsigned>(v), static_cast<unsigned>(tid));
  }
  if (tid == 0) items[n] = make_uint2(0xFFFFFFFFu, 0);
  __syncthreads();
  bool first = false;
  unsigned here = 0;
  if (warp < kFewTokens / 32) {
    first = tid < n && items[tid].x < static_cast<unsigned>(tb.V) && (tid == 0 || items[tid - 1].x != items[tid].x);
    here = __ballot_sync(0xFFFFFFFFu, first);
    if (lane == 0) runs_of[warp] = __popc(here);
  }
  __syncthreads();
  int runs = 0;
  for (int w = 0; w < kFewTokens / 32; ++w) {
    if (w == warp && first) start[runs + __popc(here & ((1u << lane) - 1u))] = tid;
    runs += runs_of[w];
  }
  __syncthreads();

  const int pieces = (tb.K + kSumCols - 1) / kSumCols;
  const T* dy = static_cast<const T*>(a.dy);
  for (int w = blockIdx.x; w < runs * pieces; w += gridDim.x) {
    const int p = start[w / pieces], k = w % pieces * kSumCols + tid * 8;
    const unsigned v = items[p].x;
    const bool in = k < tb.K;
    Codes8<BITS> codes;
    if (in && a.scales) codes.load(tb, static_cast<int>(v), k);
    float acc[8] = {};
    constexpr int kAhead = 8;
    for (int i0 = p; items[i0].x == v; i0 += kAhead) {
      uint4 x[kAhead];
      int m = 0;                                      // of them that belong to the run
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (m == j && i0 + j < n && items[i0 + j].x == v) {
          if (in) x[j] = *reinterpret_cast<const uint4*>(dy + static_cast<size_t>(items[i0 + j].y) * tb.K + k);
          m = j + 1;
        }
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (j < m && in) add8<T>(acc, x[j]);
      if (m < kAhead || i0 + kAhead >= n) break;
    }
    embed_finish<T, TO, BITS>(tb, a, static_cast<int>(v), k, in, acc, codes);
  }

  // this CTA's share of the rows, less those of the runs
  auto zero_rows = [&](int lo, int hi) {
    if (a.table) {
      uint4* p = reinterpret_cast<uint4*>(static_cast<TO*>(a.table) + static_cast<size_t>(lo) * tb.K);
      const long long m = static_cast<long long>(hi - lo) * tb.K * static_cast<int>(sizeof(TO)) / 16;
      for (long long i = tid; i < m; i += kSumThreads) p[i] = make_uint4(0, 0, 0, 0);
    }
    if (a.scales) {
      if (BITS == 4) {
        float* p = a.scales + static_cast<size_t>(lo) * tb.G;
        const long long m = static_cast<long long>(hi - lo) * tb.G;
        for (long long i = tid; i < m; i += kSumThreads) p[i] = 0.0f;
      } else {
        for (int g = warp; g < tb.G; g += kSumThreads / 32)
          for (int v = lo + lane; v < hi; v += 32) a.scales[static_cast<size_t>(g) * tb.V + v] = 0.0f;
      }
    }
  };
  const int share_lo = static_cast<int>(static_cast<long long>(blockIdx.x) * tb.V / gridDim.x);
  const int share_hi = static_cast<int>(static_cast<long long>(blockIdx.x + 1) * tb.V / gridDim.x);
  int lo = share_lo, r0 = 0, r1 = runs;               // the first run from here on
  while (r0 < r1) {
    const int mid = (r0 + r1) / 2;
    if (static_cast<int>(items[start[mid]].x) < share_lo) r0 = mid + 1; else r1 = mid;
  }
  for (int r = r0; r <= runs && lo < share_hi; ++r) {
    const int row = r < runs ? static_cast<int>(items[start[r]].x) : tb.V;
    const int hi = min(row, share_hi);
    if (lo < hi) zero_rows(lo, hi);
    lo = row + 1;
  }
}

}  // namespace flexq

// gfx950 kernels that quantise matrices to microscaled 4-bit floating point and
// average or read back quantised ones.  The arithmetic contract is stated in
// include/ob_mx4.h.
//
// A block of 32 elements shares a scale.  Along a row its elements lie on four
// neighbouring lanes, 8 consecutive ones each, so its maximum is two
// permutations within a quad of lanes; down a column (the transposed matrix)
// one lane holds all 32.  The codes come from the conversion instructions,
// which round to nearest even, or stochastically by the 16 random bits placed
// on top of their 32.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ob_mx4_device.h"
#include "ob_mx4_kernels.h"

namespace ob {
namespace mx4 {
namespace {

constexpr int kThreads = 256;
constexpr int kLaneElems = 8;  // consecutive elements of a row that a lane takes

__device__ __forceinline__ Keys call_keys(const QuantizeArgs& a) {
  return keys_of(a.seed_device != nullptr ? *a.seed_device : a.seed, 0);
}

// A lane's place in a matrix whose rows are `groups` groups of 8: the u-th of
// a block's kThreads * U consecutive groups.  One division a block, which is
// uniform, and a short one where a block spans rows.
struct Place {
  int64_t row, group;
};
struct Start {
  int64_t row, group;
};
__device__ __forceinline__ Start start_of(int64_t first, int64_t rows, int64_t groups) {
  if (rows == 1) return {0, first};
  const int64_t r = first / groups;
  return {r, first - r * groups};
}
__device__ __forceinline__ Place place_of(Start s, int64_t rows, int64_t groups, uint32_t local) {
  Place p = {s.row, s.group + local};
  if (p.group >= groups) {
    if (rows == 1) return {1, 0};
    // local < 2^12: past 2^31 groups a row this is one subtraction
    if (groups < (int64_t(1) << 31)) {
      const uint32_t q = (uint32_t)p.group / (uint32_t)groups;
      p.row += q;
      p.group -= (int64_t)q * groups;
    } else {
      p.row += 1;
      p.group -= groups;
    }
  }
  return p;
}

// Rows of x, 8 elements a lane.  Bound by memory: 110M fp32 elements in 89 us (5.6
// TB/s), with a residual 253 us (5.5 TB/s; its tensors are touched once, so they go
// past the caches: 262 through them), stochastically the same.
template <typename T, bool RESIDUAL, bool STOCHASTIC, bool WIDE, int U>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(QuantizeArgs a) {
  const int64_t groups = padded(a.cols) / kLaneElems;
  const int64_t rc = row_codes(a.cols), rs = row_scales(a.cols);
  const Start s = start_of((int64_t)blockIdx.x * (kThreads * U), a.rows, groups);
  Keys keys{};
  if (STOCHASTIC) keys = call_keys(a);
  Place at[U];
  float c[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    at[u] = place_of(s, a.rows, groups, u * kThreads + threadIdx.x);
    if (at[u].row >= a.rows) continue;
    const int64_t col = at[u].group * kLaneElems;
    const T* x = (const T*)a.x + at[u].row * a.stride + col;
    if (col + kLaneElems <= a.cols)
      RESIDUAL ? load8_stream(x, c[u]) : load8(x, c[u]);
    else
      load8_some(x, (int)(a.cols > col ? a.cols - col : 0), c[u]);
    if (RESIDUAL) {
      float e[8];
      const float* r = a.residual + at[u].row * a.cols + col;
      if (col + kLaneElems <= a.cols)
        load8_stream(r, e);
      else
        load8_some(r, (int)(a.cols > col ? a.cols - col : 0), e);
#pragma unroll
      for (int i = 0; i < 8; ++i) c[u][i] += e[i];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    // groups come in blocks of 4 on a quad of lanes, so a quad goes together
    if (at[u].row >= a.rows) continue;
    const uint32_t byte = scale_byte<STOCHASTIC>(quad_max(largest<8>(c[u])));
    const int64_t g = at[u].group;
    const uint32_t codes =
        STOCHASTIC ? encode8_stochastic<WIDE>(c[u], byte, (uint64_t)(at[u].row * groups + g) * 2,
                                              keys)
                   : encode8(c[u], byte);
    *(uint32_t*)(a.codes + at[u].row * rc + g * 4) = codes;
    if ((threadIdx.x & 3) == 0) {
      uint8_t* scales = a.scales + at[u].row * rs;
      scales[g / 4] = (uint8_t)byte;
      if (g + 4 == groups)
        for (int64_t i = groups / 4; i < rs; ++i) scales[i] = 0;
    }
    if (RESIDUAL) {
      float v[8];
      grid8(codes, v);
      const int64_t col = g * kLaneElems;
      float* r = a.residual + at[u].row * a.cols + col;
      // the value itself may be 2^128, past fp32: it is subtracted as it is multiplied
      const float scale = scale_of(byte);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __builtin_fmaf(-v[i], scale, c[u][i]);
      if (col + kLaneElems <= a.cols) {
        store8_stream(r, v);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col + i < a.cols) r[i] = v[i];
      }
    }
  }
}

// The transposed matrix, and the rows too where codes is not null, from one
// read: a wave holds 32 rows of 128 columns in registers, 16 rows of 4 columns a
// lane (the upper lanes the lower rows), so that a block down a column lies on
// two lanes and one along a row on 8.  The transposed codes of 4 waves go through
// LDS to be written as 64 bytes of a column, the scales of both as words.
// 16384 x 6400 bfloat16 elements in 75 us (4.3 TB/s; with the tile itself in
// LDS 131), 4096 x 1024 in 6.4.  Stochastically 100 us: 23 instructions an element for
// two results, half of them the hash.  32 rows of 256 columns a wave: 79 and
// 104 us, 4096 x 1024 8.0, where they are too few.  Neighbours on one die merge
// their halves of lines: 75 against 78 without (fp32, whose lines are whole, 131
// against 120 at this size, 23 against 25 at a quarter of it).
constexpr int kTileCols = 128, kTileWaves = 4, kTileRows = kTileWaves * kBlockElems;
constexpr int kLaneRows = 16;
template <typename T>
struct Four;  // 4 neighbouring elements
template <>
struct Four<float> {
  f32x4 w;
  __device__ __forceinline__ void clear() { w = f32x4{0.0f, 0.0f, 0.0f, 0.0f}; }
  __device__ __forceinline__ void load(const float* p) { w = *(const f32x4_at4*)p; }
  // The first n, 1 to 3.
  __device__ __forceinline__ void load_some(const float* p, int n) {
    w[0] = p[0];
    if (n > 1) w[1] = p[1];
    if (n > 2) w[2] = p[2];
  }
  __device__ __forceinline__ uint32_t top() const {
    const float c[4] = {w[0], w[1], w[2], w[3]};
    return largest<4>(c);
  }
  __device__ __forceinline__ uint32_t encode(uint32_t byte) const {
    const float c[4] = {w[0], w[1], w[2], w[3]};
    return encode4(c, byte);
  }
  template <bool WIDE>
  __device__ __forceinline__ uint32_t stochastic(uint32_t byte, uint64_t quad, Keys k) const {
    const float c[4] = {w[0], w[1], w[2], w[3]};
    return encode4_stochastic<WIDE>(c, byte, quad, k);
  }
};
template <>
struct Four<bf16> {
  u32x2 w;
  __device__ __forceinline__ void clear() { w = u32x2{0u, 0u}; }
  __device__ __forceinline__ void load(const bf16* p) { w = *(const u32x2_at2*)p; }
  __device__ __forceinline__ void load_some(const bf16* p, int n) {
    w[0] = p[0].bits;
    if (n > 1) w[0] |= (uint32_t)p[1].bits << 16;
    if (n > 2) w[1] = p[2].bits;
  }
  __device__ __forceinline__ uint32_t top() const {
    return larger(__builtin_elementwise_max(magnitudes(w[0]), magnitudes(w[1])));
  }
  __device__ __forceinline__ uint32_t encode(uint32_t byte) const { return encode4(w, byte); }
  template <bool WIDE>
  __device__ __forceinline__ uint32_t stochastic(uint32_t byte, uint64_t quad, Keys k) const {
    return encode4_stochastic<WIDE>(w, byte, quad, k);
  }
};

// Column j of a lane's 16 rows: its largest magnitude, and 8 of its codes at a time.
__device__ __forceinline__ uint32_t column_top(const Four<float>* x, int j) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kLaneRows; ++i) {
    const uint32_t w = magnitude(x[i].w[j]);
    top = w > top ? w : top;
  }
  return top;
}
__device__ __forceinline__ uint32_t column_top(const Four<bf16>* x, int j) {
  u16x2 top = magnitudes(x[0].w[j >> 1]);  // of two columns, once for both
#pragma unroll
  for (int i = 1; i < kLaneRows; ++i)
    top = __builtin_elementwise_max(top, magnitudes(x[i].w[j >> 1]));
  return (uint32_t)top[j & 1] << 16;
}
template <bool STOCHASTIC, bool WIDE>
__device__ __forceinline__ uint32_t column_codes(const Four<float>* x, int j, uint32_t byte,
                                                 uint64_t quad, Keys k) {
  float c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = x[i].w[j];
  return STOCHASTIC ? encode8_stochastic<WIDE>(c, byte, quad, k) : encode8(c, byte);
}
template <bool STOCHASTIC, bool WIDE>
__device__ __forceinline__ uint32_t column_codes(const Four<bf16>* x, int j, uint32_t byte,
                                                 uint64_t quad, Keys k) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i)  // the low or the high halves of two rows
    w[i] = __builtin_amdgcn_perm(x[2 * i + 1].w[j >> 1], x[2 * i].w[j >> 1],
                                 j & 1 ? 0x07060302u : 0x05040100u);
  return STOCHASTIC ? encode8_stochastic<WIDE>(w, byte, quad, k) : encode8(w, byte);
}

template <typename T, bool STOCHASTIC, bool WIDE>
__global__ void __launch_bounds__(kTileWaves * 64) quantize_tiles_kernel(QuantizeArgs a) {
  constexpr int kPieces = kTileRows / kLaneRows;  // 8 bytes each of a column's codes
  __shared__ __attribute__((aligned(16))) u32x2 out[kTileCols * kPieces];
  __shared__ __attribute__((aligned(4))) uint8_t out_scale[kTileCols * kTileWaves];
  __shared__ __attribute__((aligned(4))) uint8_t row_scale[kTileRows * (kTileCols / kBlockElems)];
  const int64_t tiles_c = (a.cols + kTileCols - 1) / kTileCols;
  const uint32_t tile = on_one_die(blockIdx.x, gridDim.x);
  const int64_t tr = (int64_t)tile / tiles_c, tc = (int64_t)tile - tr * tiles_c;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int lane = (int)threadIdx.x & 31, half = (int)threadIdx.x >> 5 & 1;
  const int64_t first_row = tr * kTileRows, c0 = tc * kTileCols, col = c0 + lane * 4;
  const int lr0 = wave * kBlockElems + half * kLaneRows;  // in the tile
  const int64_t r0 = first_row + lr0;
  const int64_t rc = row_codes(a.cols), rs = row_scales(a.cols);
  Keys keys{};
  if (STOCHASTIC) keys = call_keys(a);
  Four<T> x[kLaneRows];
  const T* from = (const T*)a.x + r0 * a.stride + col;
  if (first_row + kTileRows <= a.rows && c0 + kTileCols <= a.cols) {
#pragma unroll
    for (int i = 0; i < kLaneRows; ++i) x[i].load(from + i * a.stride);
  } else {
    // at an edge: zeros where there are no elements
#pragma unroll
    for (int i = 0; i < kLaneRows; ++i) x[i].clear();
    if (col + 4 <= a.cols) {
#pragma unroll
      for (int i = 0; i < kLaneRows; ++i)
        if (r0 + i < a.rows) x[i].load(from + i * a.stride);
    } else if (col < a.cols) {
#pragma unroll
      for (int i = 0; i < kLaneRows; ++i)
        if (r0 + i < a.rows) x[i].load_some(from + i * a.stride, (int)(a.cols - col));
    }
  }
  if (a.codes != nullptr) {
    uint8_t* to = a.codes + r0 * rc + col / 2;
    const uint64_t quad = (uint64_t)(r0 * (padded(a.cols) / 4) + col / 4);
#pragma unroll
    for (int i = 0; i < kLaneRows; ++i) {
      const uint32_t byte = scale_byte<STOCHASTIC>(oct_max(x[i].top()));
      const uint32_t codes =
          STOCHASTIC ? x[i].template stochastic<WIDE>(
                           byte, quad + (uint64_t)i * (uint64_t)(padded(a.cols) / 4), keys)
                     : x[i].encode(byte);
      // the columns of a tile are those of the padding
      if (r0 + i < a.rows) *(uint16_t*)(to + i * rc) = (uint16_t)codes;
      if ((lane & 7) == 0) row_scale[(lr0 + i) * 4 + lane / 8] = (uint8_t)byte;
      // few rows at a time, so that the registers do
      if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);
    }
  }
  // The values are taken apart again from here on: kept from the rows they would
  // take twice the registers.
#pragma unroll
  for (int i = 0; i < kLaneRows; ++i) asm volatile("" : "+v"(x[i].w));
  const int64_t trc = row_codes(a.rows), trs = row_scales(a.rows);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t top = column_top(x, j);
    const u32x2 both =
        __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(top, top, false, false));
    const uint32_t byte = scale_byte<STOCHASTIC>(both.x > both.y ? both.x : both.y);
    const uint64_t quad = (uint64_t)((col + j) * (padded(a.rows) / 4) + r0 / 4);
    u32x2 codes;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      codes[k] = column_codes<STOCHASTIC, WIDE>(x + 8 * k, j, byte, quad + 2 * k, keys);
    // lanes that write together are 4 columns apart: their pieces are permuted
    out[(lane * 4 + j) * kPieces + ((wave ^ (lane & 3)) * 2 + half)] = codes;
    if (half == 0) out_scale[(lane * 4 + j) * kTileWaves + wave] = (uint8_t)byte;
    __builtin_amdgcn_sched_barrier(0);
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < kTileCols / 64; ++t) {
    const int i = t * kTileWaves * 64 + (int)threadIdx.x, lc = i / 4, piece = i % 4;
    if (c0 + lc < a.cols)
      *(u32x4*)(a.codes_t + (c0 + lc) * trc + first_row / 2 + piece * 16) =
          *(const u32x4*)&out[lc * kPieces + (piece ^ (lc / 4 & 3)) * 2];
  }
  // a word of scales for a column, one for a row; the last tile's go on to the
  // end of the padding
  const int i = (int)threadIdx.x & 127;
  if (threadIdx.x < 128) {
    if (c0 + i < a.cols) {
      uint32_t* to = (uint32_t*)(a.scales_t + (c0 + i) * trs);
      to[tr] = *(const uint32_t*)&out_scale[i * 4];
      if (first_row + kTileRows >= a.rows)
        for (int64_t k = tr + 1; k < trs / 4; ++k) to[k] = 0;
    }
  } else if (a.codes != nullptr && first_row + i < a.rows) {
    uint32_t* to = (uint32_t*)(a.scales + (first_row + i) * rs);
    to[tc] = *(const uint32_t*)&row_scale[i * 4];
    if (tc == tiles_c - 1)
      for (int64_t k = tc + 1; k < rs / 4; ++k) to[k] = 0;
  }
}
static_assert(kTileRows == 128 && kTileCols == 128, "a thread for each row and column's scales");

// Mean of n messages, 8 elements a lane; the loads of kAhead messages at a time: 8
// messages of 110M elements in 165-176 us (5.2-5.5 TB/s; one message after the
// other 222), one read back as bfloat16 in 47 us (5.9 TB/s).
constexpr int kAhead = 8;
template <typename T, int U>
__global__ void __launch_bounds__(kThreads) average_kernel(AverageArgs a) {
  const int64_t groups = padded(a.cols) / kLaneElems;
  const int64_t rc = row_codes(a.cols), rs = row_scales(a.cols);
  const Start s = start_of((int64_t)blockIdx.x * (kThreads * U), a.rows, groups);
  Place at[U];
  int64_t code_at[U], scale_at[U];
  float sum[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    at[u] = place_of(s, a.rows, groups, u * kThreads + threadIdx.x);
    // lanes behind the last row or column read what the first lane of all does
    const bool inside = at[u].row < a.rows && at[u].group * kLaneElems < a.cols;
    code_at[u] = inside ? at[u].row * rc + at[u].group * 4 : 0;
    scale_at[u] = inside ? at[u].row * rs + at[u].group / 4 : 0;
    if (!inside) at[u].row = a.rows;
  }
  for (int i0 = 0; i0 < a.n; i0 += kAhead) {
    uint32_t codes[kAhead][U], bytes[kAhead][U];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i >= a.n) continue;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        codes[i][u] = *(const uint32_t*)(a.codes[i0 + i] + code_at[u]);
        bytes[i][u] = a.scales[i0 + i][scale_at[u]];
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i >= a.n) continue;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[8];
        decode8(codes[i][u], scale_of(bytes[i][u]), v);
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[u][k] = i0 + i == 0 ? v[k] : sum[u][k] + v[k];
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (at[u].row >= a.rows) continue;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[u][k] *= a.factor;
    const int64_t col = at[u].group * kLaneElems;
    T* out = (T*)a.out + at[u].row * a.stride + col;
    if (col + kLaneElems <= a.cols) {
      store8(out, sum[u]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (col + k < a.cols) store1(out + k, sum[u][k]);
    }
  }
}

// Blocks of a kernel that takes `per` groups of 8 elements a block.
int64_t blocks_for(int64_t rows, int64_t cols, int64_t per) {
  return (rows * (padded(cols) / kLaneElems) + per - 1) / per;
}
constexpr int kUnroll = 2;

// Whether the index of four elements of rows x cols, padded, may pass 2^32.
bool wide(int64_t rows, int64_t cols) { return rows * (padded(cols) / 4) > int64_t(1) << 32; }

template <typename T, bool STOCHASTIC, bool WIDE>
hipError_t quantize_rows(const QuantizeArgs& a, hipStream_t stream) {
  const dim3 grid((uint32_t)blocks_for(a.rows, a.cols, kThreads * kUnroll));
  if (a.residual != nullptr)
    quantize_rows_kernel<T, true, STOCHASTIC, WIDE, kUnroll><<<grid, kThreads, 0, stream>>>(a);
  else
    quantize_rows_kernel<T, false, STOCHASTIC, WIDE, kUnroll><<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}
template <typename T>
hipError_t quantize_rows(const QuantizeArgs& a, bool stochastic, hipStream_t stream) {
  if (!stochastic) return quantize_rows<T, false, false>(a, stream);
  return wide(a.rows, a.cols) ? quantize_rows<T, true, true>(a, stream)
                              : quantize_rows<T, true, false>(a, stream);
}

template <typename T, bool STOCHASTIC, bool WIDE>
hipError_t quantize_tiles(const QuantizeArgs& a, hipStream_t stream) {
  const int64_t tr = (a.rows + kTileRows - 1) / kTileRows;
  const dim3 grid((uint32_t)(tr * ((a.cols + kTileCols - 1) / kTileCols)));
  quantize_tiles_kernel<T, STOCHASTIC, WIDE><<<grid, kTileWaves * 64, 0, stream>>>(a);
  return hipGetLastError();
}
template <typename T>
hipError_t quantize_tiles(const QuantizeArgs& a, bool stochastic, hipStream_t stream) {
  if (!stochastic) return quantize_tiles<T, false, false>(a, stream);
  return wide(a.rows, a.cols) || wide(a.cols, a.rows) ? quantize_tiles<T, true, true>(a, stream)
                                                      : quantize_tiles<T, true, false>(a, stream);
}

}  // namespace

hipError_t launch_quantize_rows(const QuantizeArgs& a, bool is_bf16, bool stochastic,
                                hipStream_t stream) {
  return is_bf16 ? quantize_rows<bf16>(a, stochastic, stream)
                 : quantize_rows<float>(a, stochastic, stream);
}

hipError_t launch_quantize_tiles(const QuantizeArgs& a, bool is_bf16, bool stochastic,
                                 hipStream_t stream) {
  return is_bf16 ? quantize_tiles<bf16>(a, stochastic, stream)
                 : quantize_tiles<float>(a, stochastic, stream);
}

hipError_t launch_average(const AverageArgs& a, bool is_bf16, hipStream_t stream) {
  const dim3 grid((uint32_t)blocks_for(a.rows, a.cols, kThreads * kUnroll));
  if (is_bf16)
    average_kernel<bf16, kUnroll><<<grid, kThreads, 0, stream>>>(a);
  else
    average_kernel<float, kUnroll><<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace mx4
}  // namespace ob

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

// Rows of x, 8 elements a lane.
template <typename T, bool RESIDUAL, bool STOCHASTIC, int U>
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
      load8(x, c[u]);
    else
      load8_some(x, (int)(a.cols > col ? a.cols - col : 0), c[u]);
    if (RESIDUAL) {
      float e[8];
      const float* r = a.residual + at[u].row * a.cols + col;
      if (col + kLaneElems <= a.cols)
        load8(r, e);
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
    const uint32_t byte = scale_byte<STOCHASTIC>(quad_max(largest8(c[u])));
    const float inv = inverse_scale(byte);
    const int64_t g = at[u].group;
    const uint32_t codes =
        STOCHASTIC
            ? encode8_stochastic(c[u], inv, (uint64_t)(at[u].row * groups + g) * 2, keys)
            : encode8(c[u], inv);
    *(uint32_t*)(a.codes + at[u].row * rc + g * 4) = codes;
    if ((threadIdx.x & 3) == 0) {
      uint8_t* scales = a.scales + at[u].row * rs;
      scales[g / 4] = (uint8_t)byte;
      if (g + 4 == groups)
        for (int64_t i = groups / 4; i < rs; ++i) scales[i] = 0;
    }
    if (RESIDUAL) {
      float v[8];
      decode8(codes, scale_of(byte), v);
      const int64_t col = g * kLaneElems;
      float* r = a.residual + at[u].row * a.cols + col;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = c[u][i] - v[i];
      if (col + kLaneElems <= a.cols) {
        store8(r, v);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col + i < a.cols) r[i] = v[i];
      }
    }
  }
}

// The transposed matrix, and the rows too where codes is not null, from one
// read: a block takes a tile of 128 x 128, quantises the rows on their way
// into LDS, then every lane reads 32 elements down a column.  The transposed
// codes go through LDS so that a column's 64 bytes are written together.
constexpr int kTile = 128;
template <typename T, bool STOCHASTIC>
__global__ void __launch_bounds__(kThreads) quantize_tiles_kernel(QuantizeArgs a) {
  constexpr int kWords = kTile * (int)sizeof(T) / 4;      // 32-bit words of a tile's row
  constexpr int kPerWord = 4 / (int)sizeof(T);            // columns in one of them
  __shared__ __attribute__((aligned(16))) uint32_t tile[kTile * kWords];
  __shared__ __attribute__((aligned(16))) u32x4 out[kTile * 4];
  __shared__ uint8_t out_scale[kTile * 4];
  const int64_t tiles_c = padded(a.cols) / kTile;
  const int64_t tr = (int64_t)blockIdx.x / tiles_c, tc = (int64_t)blockIdx.x - tr * tiles_c;
  const int64_t r0 = tr * kTile, c0 = tc * kTile;
  const int64_t rc = row_codes(a.cols), rs = row_scales(a.cols);
  Keys keys{};
  if (STOCHASTIC) keys = call_keys(a);
  const int tid = (int)threadIdx.x;
  // 16 lanes take a row, 16 rows a round
  const int lane_col = (tid & 15) * kLaneElems, lane_row = tid >> 4;
#pragma unroll 4
  for (int i = 0; i < kTile / 16; ++i) {
    const int lr = i * 16 + lane_row;
    const int64_t row = r0 + lr, col = c0 + lane_col;
    float c[8];
    if (row < a.rows && col + kLaneElems <= a.cols) {
      load8((const T*)a.x + row * a.stride + col, c);
    } else {
      const int n = row < a.rows && col < a.cols ? (int)(a.cols - col) : 0;
      load8_some((const T*)a.x + (n > 0 ? row * a.stride + col : 0), n, c);
    }
    if constexpr (sizeof(T) == 4) {
      *(f32x4*)&tile[lr * kWords + lane_col] = f32x4{c[0], c[1], c[2], c[3]};
      *(f32x4*)&tile[lr * kWords + lane_col + 4] = f32x4{c[4], c[5], c[6], c[7]};
    } else {
      u32x4 w;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = (__float_as_uint(c[2 * k]) >> 16) | __float_as_uint(c[2 * k + 1]);
      *(u32x4*)&tile[lr * kWords + lane_col / 2] = w;
    }
    if (a.codes != nullptr) {
      const uint32_t byte = scale_byte<STOCHASTIC>(quad_max(largest8(c)));
      const float inv = inverse_scale(byte);
      if (row < a.rows) {
        const uint32_t codes =
            STOCHASTIC ? encode8_stochastic(c, inv, (uint64_t)(row * padded(a.cols) + col) / 4, keys)
                       : encode8(c, inv);
        *(uint32_t*)(a.codes + row * rc + col / 2) = codes;
        if ((tid & 3) == 0) a.scales[row * rs + col / kBlockElems] = (uint8_t)byte;
        if ((tid & 15) == 0 && tc == tiles_c - 1)
          for (int64_t k = tiles_c * 4; k < rs; ++k) a.scales[row * rs + k] = 0;
      }
    }
  }
  __syncthreads();
  const int64_t trc = row_codes(a.rows), trs = row_scales(a.rows);
  const int64_t tiles_r = padded(a.rows) / kTile;
  constexpr int kTasks = kWords * 4;  // words across the tile, times blocks down it
#pragma unroll
  for (int t = 0; t < kTasks / kThreads; ++t) {
    const int word = (tid + t * kThreads) % kWords, block = (tid + t * kThreads) / kWords;
    uint32_t w[kBlockElems];
#pragma unroll
    for (int i = 0; i < kBlockElems; ++i) w[i] = tile[(block * kBlockElems + i) * kWords + word];
#pragma unroll
    for (int p = 0; p < kPerWord; ++p) {
      float c[kBlockElems];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < kBlockElems; ++i) {
        const uint32_t bits = kPerWord == 1 ? w[i] : p == 0 ? w[i] << 16 : w[i] & 0xffff0000u;
        c[i] = __uint_as_float(bits);
        top = (bits & 0x7fffffffu) > top ? bits & 0x7fffffffu : top;
      }
      const uint32_t byte = scale_byte<STOCHASTIC>(top);
      const float inv = inverse_scale(byte);
      const int lc = word * kPerWord + p;
      u32x4 codes;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint64_t at = (uint64_t)((c0 + lc) * padded(a.rows) + r0 + block * kBlockElems) / 4;
        codes[k] = STOCHASTIC ? encode8_stochastic(c + 8 * k, inv, at + 2 * k, keys)
                              : encode8(c + 8 * k, inv);
      }
      out[lc * 4 + block] = codes;
      out_scale[lc * 4 + block] = (uint8_t)byte;
    }
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < kTile * 4 / kThreads; ++t) {
    const int i = t * kThreads + tid, lc = i >> 2, piece = i & 3;
    const int64_t row = c0 + lc;
    if (row >= a.cols) continue;
    *(u32x4*)(a.codes_t + row * trc + r0 / 2 + piece * 16) = out[i];
    a.scales_t[row * trs + r0 / kBlockElems + piece] = out_scale[i];
    if (piece == 0 && tr == tiles_r - 1)
      for (int64_t k = tiles_r * 4; k < trs; ++k) a.scales_t[row * trs + k] = 0;
  }
}

// Mean of n messages, 8 elements a lane.
template <typename T, int U>
__global__ void __launch_bounds__(kThreads) average_kernel(AverageArgs a) {
  const int64_t groups = padded(a.cols) / kLaneElems;
  const int64_t rc = row_codes(a.cols), rs = row_scales(a.cols);
  const Start s = start_of((int64_t)blockIdx.x * (kThreads * U), a.rows, groups);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Place at = place_of(s, a.rows, groups, u * kThreads + threadIdx.x);
    const int64_t col = at.group * kLaneElems;
    if (at.row >= a.rows || col >= a.cols) continue;
    float sum[8];
    for (int i = 0; i < a.n; ++i) {
      const uint32_t codes = *(const uint32_t*)(a.codes[i] + at.row * rc + at.group * 4);
      const float scale = scale_of(a.scales[i][at.row * rs + at.group / 4]);
      float v[8];
      decode8(codes, scale, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[k] = i == 0 ? v[k] : sum[k] + v[k];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[k] *= a.factor;
    T* out = (T*)a.out + at.row * a.stride + col;
    if (col + kLaneElems <= a.cols) {
      store8(out, sum);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (col + k < a.cols) store1(out + k, sum[k]);
    }
  }
}

// Blocks of a kernel that takes `per` groups of 8 elements a block.
int64_t blocks_for(int64_t rows, int64_t cols, int64_t per) {
  return (rows * (padded(cols) / kLaneElems) + per - 1) / per;
}
// A grid's first dimension holds 2^31 - 1 blocks: 2^40 elements in blocks of 2048
// and more stay below it.
constexpr int kUnroll = 2;

template <typename T, bool STOCHASTIC>
hipError_t quantize_rows(const QuantizeArgs& a, hipStream_t stream) {
  const dim3 grid((uint32_t)blocks_for(a.rows, a.cols, kThreads * kUnroll));
  if (a.residual != nullptr)
    quantize_rows_kernel<T, true, STOCHASTIC, kUnroll><<<grid, kThreads, 0, stream>>>(a);
  else
    quantize_rows_kernel<T, false, STOCHASTIC, kUnroll><<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

template <typename T, bool STOCHASTIC>
hipError_t quantize_tiles(const QuantizeArgs& a, hipStream_t stream) {
  const dim3 grid((uint32_t)(padded(a.rows) / kTile * (padded(a.cols) / kTile)));
  quantize_tiles_kernel<T, STOCHASTIC><<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_rows(const QuantizeArgs& a, bool is_bf16, bool stochastic,
                                hipStream_t stream) {
  if (is_bf16)
    return stochastic ? quantize_rows<bf16, true>(a, stream) : quantize_rows<bf16, false>(a, stream);
  return stochastic ? quantize_rows<float, true>(a, stream) : quantize_rows<float, false>(a, stream);
}

hipError_t launch_quantize_tiles(const QuantizeArgs& a, bool is_bf16, bool stochastic,
                                 hipStream_t stream) {
  if (is_bf16)
    return stochastic ? quantize_tiles<bf16, true>(a, stream)
                      : quantize_tiles<bf16, false>(a, stream);
  return stochastic ? quantize_tiles<float, true>(a, stream)
                    : quantize_tiles<float, false>(a, stream);
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

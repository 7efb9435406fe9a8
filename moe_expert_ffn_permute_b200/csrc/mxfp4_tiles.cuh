// mxfp4_tiles.cuh -- what the two MXFP4 product kernels share: the tiles of a
// grouped product, derived on the device from the row offsets, and the epilogue
// that takes a 128-feature x n-token accumulator from registers to the output.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "sm100.cuh"

namespace moe {
namespace mx {

constexpr int kKBytes = 128;   // bytes of a row per stage: 256 codes

// The value on lane 0: the same on every lane, and the compiler knows it.
template <class T>
__device__ __forceinline__ T uniform(T v) {
  return __shfl_sync(0xffffffffu, v, 0);
}

// Row offsets and token tiles of the groups, in shared memory.
struct Groups {
  int row_off[kMxMaxExperts + 1];    // first row of each expert, made monotone
  int tile_off[kMxMaxExperts + 1];   // token tiles before each expert
};

struct Tile {
  int e, nb, row, rows;   // expert, weight block(s), first row, rows (1..cap)
};

// Token tiles of a group of `rows` rows, at most `cap` tokens each, and the tokens
// that each of a group's `tiles` tiles has (a multiple of 16; the last may have
// fewer).  Unsigned: a group may have all of the 2^31 - 1 rows, and the sums that
// round up pass 2^31 - 1 then.
__host__ __device__ __forceinline__ int token_tiles(int rows, int cap) {
  return static_cast<int>((static_cast<uint32_t>(rows) + cap - 1u) / cap);
}
__host__ __device__ __forceinline__ int tile_size(int rows, int tiles) {
  return static_cast<int>(((static_cast<uint32_t>(rows) + tiles - 1u) / tiles + 15u) & ~15u);
}

// By one whole warp: row offsets clamped to [0, R] and made monotone (a running
// maximum), so that no content of the array can lead outside the buffers; then
// the prefix sums of the token tiles, at most `cap` tokens each.
__device__ __forceinline__ void find_groups(Groups& g, const int32_t* offsets, int R, int E,
                                            int cap) {
  const int lane = threadIdx.x & 31;
  if (offsets == nullptr) {
    if (lane == 0) {
      g.row_off[0] = 0;
      g.row_off[1] = R;
    }
  } else {
    int carry = 0;
    for (int b = 0; b <= E; b += 32) {
      const int i = b + lane;
      int v = i <= E ? min(max(__ldg(&offsets[i]), 0), R) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v = max(v, u);
      }
      v = max(v, carry);
      carry = __shfl_sync(0xffffffffu, v, 31);
      if (i <= E) g.row_off[i] = v;
    }
  }
  __syncwarp();
  int carry = 0;
  for (int b = 0; b < E; b += 32) {
    const int i = b + lane;
    const int rows = i < E ? g.row_off[i + 1] - g.row_off[i] : 0;
    const int own = token_tiles(rows, cap);
    int v = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (i < E) g.tile_off[i] = carry + v - own;
    carry += __shfl_sync(0xffffffffu, v, 31);
  }
  if (lane == 0) g.tile_off[E] = carry;
}

// Tile `id`: the groups' token tiles in order, each with its `nb_n` weight
// blocks.  A group is cut into tiles of equal size (a multiple of 16).
__device__ __forceinline__ Tile tile_at(const Groups& g, int E, int nb_n, long long id) {
  Tile t;
  const int tt = static_cast<int>(id / nb_n);
  t.nb = static_cast<int>(id - static_cast<long long>(tt) * nb_n);
  int lo = 0, hi = E - 1;   // the last expert whose tiles start at or before tt
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.tile_off[mid] <= tt) lo = mid;
    else hi = mid - 1;
  }
  // (Experts without rows start where their successor does: the search lands on
  // the last of equals, which is the one that has the tile.)
  t.e = lo;
  const int n = g.row_off[lo + 1] - g.row_off[lo];
  const int tiles = g.tile_off[lo + 1] - g.tile_off[lo];
  const int size = tile_size(n, tiles);
  const int local = (tt - g.tile_off[lo]) * size;
  t.row = g.row_off[lo] + local;
  t.rows = min(size, n - local);
  return t;
}

// First row of a half (0 or 1) of a tile whose MMA has n columns; past the last
// row it is R, whose rows arrive as zeros (t.row + n / 2 may pass 2^31 - 1).
__host__ __device__ __forceinline__ int half_row(int row, int n, int half, int R) {
  const uint32_t first = static_cast<uint32_t>(row) + static_cast<uint32_t>(half * (n / 2));
  return static_cast<int>(first < static_cast<uint32_t>(R) ? first : static_cast<uint32_t>(R));
}

// Two fp32 -> two 16-bit floats, round to nearest even; `lo` in the low half.
template <bool kFp16>
__device__ __forceinline__ uint32_t pack_out(float lo, float hi) {
  if constexpr (kFp16) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  } else {
    return pack_bf16x2(lo, hi);
  }
}

// Token columns of an accumulator of n columns: half 0 has [0, half_begin(n, 1)),
// half 1 the rest (the two warps of a TMEM sub-partition share a tile's tokens
// evenly).
__device__ __forceinline__ int half_begin(int n, int h) { return h ? (n / 2 + 7) & ~7 : 0; }

// One warp's part of a tile: lane = feature, v[j] = token c0 + j, `cols` of them.
// Neighbouring lanes trade halves of a pair of tokens so that an even lane holds
// two features of the first and an odd lane of the second: 4-byte stores, 64
// contiguous bytes per token.  Unrolled straight-line code, so it is kept short
// (one conversion, shuffle, permute and store per pair): with a runtime choice of
// the output type in it a tile's epilogue took 5 us, mostly instruction fetches.
template <int kCols, bool kFp16>
__device__ __forceinline__ void store_tile(const uint32_t (&v)[kCols], uint16_t* out, int N,
                                           int feature0, const Tile& t, int c0, int cols) {
  const int lane = threadIdx.x & 31;
  const int odd = lane & 1;
  const uint32_t pick = odd ? 0x3276u : 0x5410u;
  const int f = feature0 + (lane & ~1);
  uint16_t* dst = out + (static_cast<size_t>(t.row) + c0 + odd) * N + f;
  const size_t step = 2 * static_cast<size_t>(N);
  // Tokens of this half, counted from the lane's first.
  const int left = f < N ? min(cols, t.rows - c0) - odd : 0;
#pragma unroll
  for (int c = 0; c < kCols / 32; ++c) {
    if (32 * c >= cols) break;
#pragma unroll
    for (int j = 32 * c; j < 32 * c + 32; j += 2) {
      const uint32_t own = pack_out<kFp16>(__uint_as_float(v[j]), __uint_as_float(v[j + 1]));
      const uint32_t got = __shfl_xor_sync(0xffffffffu, own, 1);
      if (j < left) *reinterpret_cast<uint32_t*>(dst) = __byte_perm(own, got, pick);
      dst += step;
    }
  }
}

// --------------------------------------------------------------- host side
// A map of u8 rows [rows, width] with boxes of box_rows rows of `box` bytes.
bool map_rows(CUtensorMap* m, const void* base, uint64_t width, uint64_t rows, uint32_t box,
              uint32_t box_rows, bool swizzle128);

}  // namespace mx

// What a product launch needs (both kernels).
struct MxGemm {
  int R, E, N, K;
  int cap;                    // most tokens of a tile (a multiple of 16)
  int nb_n, kb_n;             // 128-row weight blocks, 256-wide K blocks
  int fault;                  // test hook: the MMA issuers wait for what never comes
  const int32_t* offsets;     // null: one group of all rows
  const uint8_t* codes;
  const uint8_t* scales;      // token scales, group-major [ceil(K/128)][R][4]
  const uint8_t* w;           // prepacked tiles
  const uint8_t* w_sf;        // prepacked scale chunks
  uint16_t* out;
  uint32_t* err;
  uint8_t* records;           // pairs: token scales in the tensor core's layout
};

// Bytes of the pair kernel's token scale records.
size_t mx_pair_record_bytes(int R, int E, int K);
// The product on CTA pairs (two launches: scale records, product).
cudaError_t launch_mx_pairs(const MxGemm& p, bool fp16, cudaStream_t st);

}  // namespace moe

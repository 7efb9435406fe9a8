// mxfp4_gemm.cu -- grouped product with both operands in MXFP4:
//   out[r, n] = sum_k a[r, k] * w[e, n, k]   for the rows r of expert e,
//   offsets[e] <= r < offsets[e + 1],
// fp32 sums, rounded once to bf16 or fp16.  tcgen05.mma.kind::mxf4 takes the
// packed codes and applies both UE8M0 scales itself: K = 64 per instruction,
// twice the rate of the FP8 x MXFP4 product in gemm.cu.
//
// The weights are the MMA's A operand (128 rows, prepacked tiles) and a tile's
// token rows its B operand, N = their count rounded up to 16: one form serves a
// single token and a full tile, and the tensor work follows the tokens.  An
// accumulator lane is then an output feature and a column a token.
//   Tokens are read where they lie: a tile starts at any row (2-D TMA, 128-byte
//   swizzle, rows past R and codes past K arrive as zeros); rows of the next
//   group that a box brings along are computed and not stored.
//
// One persistent CTA per SM; tile i of CTA b is b + i * grid, the 128-row weight
// blocks of a token tile next to one another.  Every role derives the tiles from
// the same prefix sums in shared memory.  Warps:
//   0      operands: weight tile and its scale chunks (bulk copies), token boxes
//   1      MMA issuer (one lane); owns the tensor-memory allocation
//   2, 3   token scales: warp 2 + h brings 128-wide half h of the stage's 256
//          codes, one word (four scale bytes) per row, by cp.async
//   4-11   epilogue: two warps per 32-lane TMEM sub-partition
// Every wait is bounded; on expiry the error word gets MOE_ERR_DEVICE_TIMEOUT
// and the CTA winds down.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "elem.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace moe {
namespace {

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr uint32_t kTmemCols = 512;
constexpr int kKBytes = 128;             // bytes of a row per stage: 256 codes
// TMEM: the accumulator takes columns 0..255; two scale sets, used in turn so
// that a copy never lands in the set that MMAs just issued may still read.  A
// set holds 2 x 4 columns of weight scales and 2 x 8 of token scales (rows
// 0..127 and 128..255 of the tile, for each half of the stage's K).
constexpr uint32_t kSfCol = 256, kSfSet = 32, kSfTokens = 8;

// kTok: most tokens of a tile.  256: the fewest weight reads per token; 64: twice
// the stages in flight where an expert has few tokens and the weights stream.
template <int kTok>
struct Cfg {
  static constexpr int kStages = kTok == 256 ? 4 : 8;
  static constexpr int kBox = kTok == 256 ? 64 : 32;   // rows of a token box
  static constexpr int kChunks = (kTok + 127) / 128;   // 128-row scale chunks
};

template <int kTok>
struct __align__(1024) Smem {
  using C = Cfg<kTok>;
  uint8_t w[C::kStages][kTileBytes];
  uint8_t t[C::kStages][kTok * kKBytes];
  uint8_t sfw[C::kStages][1024];
  uint8_t sft[C::kStages][2 * C::kChunks * 512];   // [half][chunk]
  uint64_t full[C::kStages];      // the operand warp's copies
  uint64_t full_sf[C::kStages];   // the scale warps' copies
  uint64_t empty[C::kStages];
  uint64_t tmem_full, tmem_empty, drain;
  int row_off[kMxMaxExperts + 1];    // first row of each expert, made monotone
  int tile_off[kMxMaxExperts + 1];   // token tiles before each expert
  uint32_t tmem_base;
  int abort_flag;
};

struct Params {
  int R, E, N, K;
  int cap;                    // most tokens of a tile (a multiple of 16, at most kTok)
  int nb_n, kb_n;             // 128-row weight blocks, 256-wide K blocks
  const int32_t* offsets;     // null: one group of all rows
  const uint8_t* w;           // prepacked tiles
  const uint8_t* w_sf;        // prepacked scale chunks
  const uint8_t* scales;      // token scales, group-major [ceil(K/128)][R][4]
  uint16_t* out;
  uint32_t* err;
};

struct Tile {
  int e, nb, row, rows;       // expert, weight block, first row, rows (1..cap)
};

// Tile `id` of the launch: the groups' token tiles in order, each with all its
// weight blocks.  A group is cut into tiles of equal size (a multiple of 16).
template <int kTok>
__device__ __forceinline__ Tile tile_at(const Smem<kTok>& sm, const Params& p, long long id) {
  Tile t;
  const int tt = static_cast<int>(id / p.nb_n);
  t.nb = static_cast<int>(id - static_cast<long long>(tt) * p.nb_n);
  int lo = 0, hi = p.E - 1;   // the last expert whose tiles start at or before tt
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sm.tile_off[mid] <= tt) lo = mid;
    else hi = mid - 1;
  }
  // Experts without rows share their successor's start: the search lands on the
  // last of equals, which is the one that has the tile.
  t.e = lo;
  const int n = sm.row_off[lo + 1] - sm.row_off[lo];
  const int tiles = sm.tile_off[lo + 1] - sm.tile_off[lo];
  const int size = ((n + tiles - 1) / tiles + 15) & ~15;
  const int local = (tt - sm.tile_off[lo]) * size;
  t.row = sm.row_off[lo] + local;
  t.rows = min(size, n - local);
  return t;
}

// The value on lane 0: the same on every lane, and the compiler knows it.
template <class T>
__device__ __forceinline__ T uniform(T v) {
  return __shfl_sync(0xffffffffu, v, 0);
}

__device__ __forceinline__ uint32_t mma_n(int rows) {
  return static_cast<uint32_t>((rows + 15) & ~15);
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

// Token columns [c0, c0 + cols) of an accumulator of n columns are half h's: the
// two warps of a sub-partition share a tile's tokens evenly.
__device__ __forceinline__ int half_begin(int n, int h) { return h ? (n / 2 + 7) & ~7 : 0; }

template <int kTok, bool kFp16>
__global__ void __launch_bounds__(kThreads, 1)
    mxfp4_gemm_kernel(const __grid_constant__ CUtensorMap tmap, const Params p) {
  using C = Cfg<kTok>;
  constexpr int STAGES = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  griddep_launch_dependents();
  Smem<kTok>& sm = *reinterpret_cast<Smem<kTok>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  // (The shuffle makes the warp's number uniform to the compiler.)
  const int warp = uniform(static_cast<int>(threadIdx.x >> 5));
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.full_sf[s], 64);
      mbar_init(&sm.empty[s], 1);
    }
    mbar_init(&sm.tmem_full, 1);
    mbar_init(&sm.tmem_empty, kEpiWarps);
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmap);
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  // Everything above is local set-up that overlaps the previous kernel's tail.
  griddep_wait();
  if (warp == 2) {
    // Row offsets, clamped to [0, R] and made monotone (a running maximum), so
    // that no content of the array can lead outside the buffers; then the
    // prefix sums of the token tiles.
    if (p.offsets == nullptr) {
      if (lane == 0) {
        sm.row_off[0] = 0;
        sm.row_off[1] = p.R;
      }
    } else {
      int carry = 0;
      for (int b = 0; b <= p.E; b += 32) {
        const int i = b + lane;
        int v = i <= p.E ? min(max(__ldg(&p.offsets[i]), 0), p.R) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v = max(v, u);
        }
        v = max(v, carry);
        carry = __shfl_sync(0xffffffffu, v, 31);
        if (i <= p.E) sm.row_off[i] = v;
      }
    }
    __syncwarp();
    int carry = 0;
    for (int b = 0; b < p.E; b += 32) {
      const int i = b + lane;
      const int rows = i < p.E ? sm.row_off[i + 1] - sm.row_off[i] : 0;
      const int own = (rows + p.cap - 1) / p.cap;
      int v = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      if (i < p.E) sm.tile_off[i] = carry + v - own;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) sm.tile_off[p.E] = carry;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const int kb_n = p.kb_n;
  const long long tiles = static_cast<long long>(sm.tile_off[p.E]) * p.nb_n;
  const int my_tiles = uniform(
      static_cast<int>((tiles - blockIdx.x + gridDim.x - 1) / gridDim.x));   // may be <= 0

  // The issuing warps run warp-uniform loops and elect a lane for the copies and
  // MMAs alone (elect_one() says what that saves).
  if (warp == 0) {
    // ------------------------------------------------------------- operands
    const uint64_t pol_tok = l2_policy_evict_last();
    const uint64_t pol_once = l2_policy_evict_first();
    const uint64_t pol_reused = l2_policy_evict_normal();
    int stage = 0;
    uint32_t phase = 0;
    long long issued = 0;   // stages filled
    bool ok = true;
    for (int i = 0; ok && i < my_tiles; ++i) {
      const Tile t = tile_at<kTok>(sm, p, blockIdx.x + static_cast<long long>(i) * gridDim.x);
      // Weights of an expert with one token tile are read once.
      const uint64_t pol_w = sm.tile_off[t.e + 1] - sm.tile_off[t.e] > 1 ? pol_reused : pol_once;
      const int boxes = uniform((t.rows + C::kBox - 1) / C::kBox);
      const uint32_t bytes = kTileBytes + 1024 + boxes * C::kBox * kKBytes;
      const long long block = uniform((static_cast<long long>(t.e) * p.nb_n + t.nb) * kb_n);
      const int row = uniform(t.row);
      for (int kb = 0; kb < kb_n; ++kb) {
        if (!mbar_wait_warp(&sm.empty[stage], phase ^ 1u, p.err, &sm.abort_flag)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          mbar_arrive_expect_tx(&sm.full[stage], bytes);
          bulk_load_hint(sm.w[stage], p.w + (block + kb) * kTileBytes, kTileBytes, &sm.full[stage],
                         pol_w);
          bulk_load_hint(sm.sfw[stage], p.w_sf + (block + kb) * 1024, 1024, &sm.full[stage], pol_w);
          for (int b = 0; b < boxes; ++b)
            tma_load_2d(sm.t[stage] + b * C::kBox * kKBytes, &tmap, kb * kKBytes,
                        row + b * C::kBox, &sm.full[stage], pol_tok);
        }
        __syncwarp();
        ++issued;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // On the way out of an aborted CTA: its copies in flight land before its
    // shared memory is given back.
    for (int s = 0; !ok && s < STAGES && s < issued; ++s) {
      if (--stage < 0) {
        stage = STAGES - 1;
        phase ^= 1u;
      }
      mbar_wait_limited(&sm.full[stage], phase, kWaitLimitNs);
    }
    __syncwarp();
  } else if (warp == 2 || warp == 3) {
    // --------------------------------------------------------- token scales
    const int h = warp - 2;
    const int groups = (p.K + 127) / 128;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int i = 0; ok && i < my_tiles; ++i) {
      const Tile t = tile_at<kTok>(sm, p, blockIdx.x + static_cast<long long>(i) * gridDim.x);
      const int quads = (t.rows + 31) / 32;
      for (int kb = 0; kb < kb_n; ++kb) {
        if (!mbar_wait(&sm.empty[stage], phase ^ 1u, p.err, &sm.abort_flag)) {
          ok = false;
          break;
        }
        const int g = 2 * kb + h;
        const bool in_k = g < groups;
        // Row 32q + lane of the tile: word `q % 4` of the lane's 16 bytes in
        // chunk q / 4.
        const uint8_t* src = p.scales + (static_cast<size_t>(in_k ? g : 0) * p.R + t.row) * 4;
        uint8_t* dst = sm.sft[stage] + h * C::kChunks * 512 + lane * 16;
        for (int q = 0; q < quads; ++q) {
          const int r = 32 * q + lane;
          const bool in = in_k && r < t.rows;
          cp_async_4_zfill(dst + (q >> 2) * 512 + (q & 3) * 4, src + (in ? r * 4 : 0), in);
        }
        cp_async_mbar_arrive_noinc(&sm.full_sf[stage]);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // No copy of this thread is in flight when the CTA ends.
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issue
    int stage = 0;
    uint32_t phase = 0, acc_phase = 0, set = 0;
    const uint32_t acc = uniform(tmem);
    const uint64_t w_desc0 = umma_desc_sw128(smem_u32(sm.w[0]));
    const uint64_t t_desc0 = umma_desc_sw128(smem_u32(sm.t[0]));
    const uint64_t sfw_desc0 = sf_desc(smem_u32(sm.sfw[0]));
    const uint64_t sft_desc0 = sf_desc(smem_u32(sm.sft[0]));
    constexpr uint64_t kKStep = 32 >> 4, kSfChunk = 512 >> 4;
    bool ok = true;
    for (int i = 0; ok && i < my_tiles; ++i) {
      const Tile t = tile_at<kTok>(sm, p, blockIdx.x + static_cast<long long>(i) * gridDim.x);
      const uint32_t n = uniform(mma_n(t.rows));
      const uint32_t idesc0 = mxf4_idesc(n, 0);
      if (!mbar_wait_warp(&sm.tmem_empty, acc_phase ^ 1u, p.err, &sm.abort_flag)) break;
      tc_fence_after();
      for (int kb = 0; kb < kb_n; ++kb) {
        if (!mbar_wait_warp(&sm.full[stage], phase, p.err, &sm.abort_flag) ||
            !mbar_wait_warp(&sm.full_sf[stage], phase, p.err, &sm.abort_flag)) {
          ok = false;
          break;
        }
        // The token scales land by cp.async (generic proxy): order them before
        // the tensor core's (async proxy) reads.
        fence_proxy_async_smem();
        tc_fence_after();
        if (elect_one()) {
          const uint32_t sfw = acc + kSfCol + set * kSfSet;
          const uint32_t sft = sfw + kSfTokens;
          const uint64_t sfwd = sfw_desc0 + static_cast<uint64_t>(stage) * (1024 >> 4);
          const uint64_t sftd =
              sft_desc0 + static_cast<uint64_t>(stage) * (2 * C::kChunks * 512 >> 4);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            tmem_cp_32x128b_warpx4(sfw + 4 * h, sfwd + h * kSfChunk);
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
              if (c == 0 || n > 128)
                tmem_cp_32x128b_warpx4(sft + 8 * h + 4 * c,
                                       sftd + (h * C::kChunks + c) * kSfChunk);
          }
          const uint64_t wd = w_desc0 + static_cast<uint64_t>(stage) * (kTileBytes >> 4);
          const uint64_t td = t_desc0 + static_cast<uint64_t>(stage) * (kTok * kKBytes >> 4);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint32_t h = ks >> 1, sf_id = (ks & 1) * 2;
            mma_mxf4(acc, wd + ks * kKStep, td + ks * kKStep,
                     idesc0 | (sf_id << 4) | (sf_id << 29), (sfw + 4 * h) | (sf_id << 30),
                     (sft + 8 * h) | (sf_id << 30), (kb > 0 || ks > 0) ? 1u : 0u);
          }
          tc_commit(&sm.empty[stage]);
        }
        __syncwarp();
        set ^= 1u;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (elect_one()) tc_commit(&sm.tmem_full);
      __syncwarp();
      acc_phase ^= 1u;
    }
    // Everything issued above completes before the TMEM is freed.
    if (elect_one()) {
      tc_commit(&sm.drain);
      if (!mbar_wait_limited(&sm.drain, 0, kWaitLimitNs)) atomicOr(p.err, kErrTimeoutBit);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- epilogue
    const int q = warp & 3;              // TMEM sub-partition: lanes 32q..32q+31
    const int half = (warp - 4) >> 2;    // which half of the tile's token columns
    constexpr int kCols = kTok / 2;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const bool odd = lane & 1;
    const uint32_t pick = odd ? 0x3276u : 0x5410u;
    uint32_t acc_phase = 0;
    for (int i = 0; i < my_tiles; ++i) {
      const Tile t = tile_at<kTok>(sm, p, blockIdx.x + static_cast<long long>(i) * gridDim.x);
      const int n = static_cast<int>(mma_n(t.rows));
      const int c0 = half_begin(n, half), cols = half ? n - c0 : half_begin(n, 1);
      if (!mbar_wait(&sm.tmem_full, acc_phase, p.err, &sm.abort_flag)) break;
      acc_phase ^= 1u;
      tc_fence_after();
      // (kCols columns are loaded whatever the tile holds: they are always
      // addressable, and a conditional load would put the array in local
      // memory.)
      uint32_t v[kCols];
#pragma unroll
      for (int c = 0; c < kCols / 32; ++c)
        tmem_ld_32x32b_x32(lanes + c0 + c * 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32 * c));
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.tmem_empty);
      // Lane = feature, register = token.  Neighbouring lanes trade halves of a
      // pair of tokens so that an even lane holds two features of the first and
      // an odd lane of the second: 4-byte stores, 64 contiguous bytes per token.
      const int f = t.nb * 128 + q * 32 + (lane & ~1);
      uint16_t* dst = p.out + (static_cast<size_t>(t.row) + c0 + (odd ? 1 : 0)) * p.N + f;
      const size_t step = 2 * static_cast<size_t>(p.N);
      // Tokens of this half, counted from the lane's first.
      const int left = f < p.N ? min(cols, t.rows - c0) - (odd ? 1 : 0) : 0;
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
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// --------------------------------------------------------------- host side
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault,
                                            &q) == cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<EncodeTiledFn>(ptr) : nullptr;
  }();
  return fn;
}

template <int kTok, bool kFp16>
cudaError_t launch(const Params& p, const uint8_t* codes, cudaStream_t st) {
  const EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return cudaErrorNotSupported;
  CUtensorMap map;
  std::memset(&map, 0, sizeof(map));
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.K / 2), static_cast<cuuint64_t>(p.R)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.K / 2)};
  const cuuint32_t box[2] = {kKBytes, Cfg<kTok>::kBox};
  const cuuint32_t estr[2] = {1, 1};
  if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, box,
          estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const size_t smem = sizeof(Smem<kTok>) + 1024;
  static_assert(sizeof(Smem<kTok>) + 1024 <= 232448, "shared memory of a CTA");
  auto kern = mxfp4_gemm_kernel<kTok, kFp16>;
  const cudaError_t e =
      ensure_max_dynamic_smem(reinterpret_cast<const void*>(kern), static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  // No more CTAs than tiles there can be.
  const long long most = (p.R / p.cap + std::min(p.E, p.R)) * static_cast<long long>(p.nb_n);
  const int grid = static_cast<int>(std::min<long long>(sm_count(), most));
  return launch_pdl(kern, dim3(grid), dim3(kThreads), smem, st, map, p);
}

// Small token tiles (twice the stages) while the average group fits one.
bool small_tiles(int R, int E) { return R <= 64ll * E; }

// Most tokens of a tile of the large variant.  A K block of a tile of n tokens
// costs about kBlockClocks + kTokenClocks * n clocks, and a launch as many tiles
// one after another as there are waves; group sizes are known on the device
// only, so the groups are taken as equal.
constexpr double kBlockClocks = 300, kTokenClocks = 1.75;
int tile_cap(int R, int E, int nb_n) {
  const long long groups = std::min(E, R), rows = (R + groups - 1) / groups;
  const int ctas = sm_count();
  int best = 256;
  double least = 0;
  for (int cap = 256; cap >= 64; cap -= 16) {
    const long long per = (rows + cap - 1) / cap, tiles = per * groups * nb_n;
    const long long size = ((rows + per - 1) / per + 15) / 16 * 16;
    const double cost =
        static_cast<double>((tiles + ctas - 1) / ctas) * (kBlockClocks + kTokenClocks * size);
    if (cap == 256 || cost < least) {
      least = cost;
      best = cap;
    }
  }
  return best;
}

bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_mxfp4_clear_error(void* workspace, moe_stream_t stream) {
  if (workspace == nullptr) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned_to(workspace, 256)) return MOE_ERR_ALIGNMENT;
  return cudaMemsetAsync(workspace, 0, 256, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

moe_status moe_mxfp4_check_error(const void* workspace, moe_stream_t stream) {
  if (workspace == nullptr) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned_to(workspace, 256)) return MOE_ERR_ALIGNMENT;
  uint32_t word = 0;
  auto st = reinterpret_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(&word, workspace, 4, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return MOE_ERR_CUDA;
  return word & moe::kErrTimeoutBit ? MOE_ERR_DEVICE_TIMEOUT : MOE_OK;
}

size_t moe_mxfp4_workspace_bytes(int R, int E, int N, int K) {
  return R >= 1 && moe::mx_gemm_sizes_ok(E, N, K) ? 256 : 0;
}

moe_status moe_mxfp4_gemm(const uint8_t* codes, const uint8_t* scales, const int32_t* offsets,
                          int R, int E, int N, int K, const uint8_t* w_tiled,
                          const uint8_t* w_scales_chunked, int dtype, void* out, void* workspace,
                          moe_stream_t stream) {
  if (codes == nullptr || scales == nullptr || w_tiled == nullptr || w_scales_chunked == nullptr ||
      out == nullptr || workspace == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (R < 1 || E < 1 || N < 1 || K < 1 || !moe::elem_ok(dtype)) return MOE_ERR_INVALID_ARG;
  if (offsets == nullptr && E != 1) return MOE_ERR_INVALID_ARG;
  if (!moe::mx_gemm_sizes_ok(E, N, K) || dtype == MOE_T_FP32) return MOE_ERR_UNSUPPORTED;
  if (!moe::aligned_to(codes, 16) || !moe::aligned_to(scales, 4) ||
      !moe::aligned_to(offsets, 4) || !moe::aligned_to(w_tiled, 16) ||
      !moe::aligned_to(w_scales_chunked, 16) || !moe::aligned_to(out, 16) ||
      !moe::aligned_to(workspace, 256))
    return MOE_ERR_ALIGNMENT;
  const long long rb = R;
  if (moe::buffers_overlap(out, rb * N * 2, codes, rb * (K / 2)) ||
      moe::buffers_overlap(out, rb * N * 2, scales, (K + 127) / 128 * rb * 4))
    return MOE_ERR_INVALID_ARG;
  moe::Params p{};
  p.R = R;
  p.E = E;
  p.N = N;
  p.K = K;
  p.nb_n = (N + 127) / 128;
  p.kb_n = (K + 255) / 256;
  p.offsets = offsets;
  p.w = w_tiled;
  p.w_sf = w_scales_chunked;
  p.scales = scales;
  p.out = static_cast<uint16_t*>(out);
  p.err = static_cast<uint32_t*>(workspace);
  const bool small = moe::small_tiles(R, E);
  p.cap = small ? 64 : moe::tile_cap(R, E, p.nb_n);
  auto st = reinterpret_cast<cudaStream_t>(stream);
  const bool fp16 = dtype == MOE_T_FP16;
  const cudaError_t e = small ? (fp16 ? moe::launch<64, true>(p, codes, st)
                                      : moe::launch<64, false>(p, codes, st))
                              : (fp16 ? moe::launch<256, true>(p, codes, st)
                                      : moe::launch<256, false>(p, codes, st));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"

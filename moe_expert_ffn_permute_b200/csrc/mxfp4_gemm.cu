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
//
// Few tokens: bound by the weight stream.  One token through 8 experts, 7168 ->
// 4096, 23.8 us (125 MB, 5.2 TB/s; 1.8 us until the first weights, 1.5 us from the
// last MMA to the next kernel), 2048 -> 7168 15.9 us (63 MB in four rounds of tiles);
// a skewed batch of 128 tokens, 28 of 32 experts, 75 to 78 us (449 MB, 5.9 TB/s), 70
// without its MMAs, and 42 us 2048 -> 7168 (39 without its stores).  Many tokens:
// operand delivery into shared memory (52 KB per SM and K block) and then the power
// cap; mxfp4_pair.cu takes those.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "args.h"
#include "internal.h"
#include "mxfp4_tiles.cuh"
#include "sm100.cuh"

namespace moe {
namespace {

using mx::kKBytes;
using mx::Tile;
using mx::tile_at;
using mx::uniform;

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr uint32_t kTmemCols = 512;
// TMEM: the accumulator takes columns 0..255; two scale sets, used in turn so
// that a copy never lands in the set that MMAs just issued may still read.  A
// set holds 2 x 4 columns of weight scales and 2 x 8 of token scales (rows
// 0..127 and 128..255 of the tile, for each half of the stage's K).  (With tiles of
// 128 tokens two accumulators used in turn measured the same as one, on decode
// batches and groups of 32 to 144 rows: the epilogue frees TMEM as soon as it has
// loaded.  Not measured on large tiles of short K.)
constexpr uint32_t kSfCol = 256, kSfSet = 32, kSfTokens = 8;

// kTok: most tokens of a tile.  256: the fewest weight reads per token; 128: half
// as many stages again where groups have few tokens and the weights stream (with
// 64, eight stages, one token took 1% less, but a skewed batch of 128 tokens 81 us
// against 77, reading the weights of its busy experts twice).
template <int kTok>
struct Cfg {
  static constexpr int kStages = kTok == 256 ? 4 : 6;
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
  mx::Groups groups;
  uint32_t tmem_base;
  int abort_flag;
};

__device__ __forceinline__ uint32_t mma_n(int rows) {
  return static_cast<uint32_t>((rows + 15) & ~15);
}

template <int kTok, bool kFp16>
__global__ void __launch_bounds__(kThreads, 1)
    mxfp4_gemm_kernel(const __grid_constant__ CUtensorMap tmap, const MxGemm p) {
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
  if (warp == 2) mx::find_groups(sm.groups, p.offsets, p.R, p.E, p.cap);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const int kb_n = p.kb_n;
  const long long tiles = static_cast<long long>(sm.groups.tile_off[p.E]) * p.nb_n;
  const int my_tiles = uniform(
      static_cast<int>((tiles - blockIdx.x + gridDim.x - 1) / gridDim.x));   // may be <= 0

  // The issuing loops run on one elected lane (elect_one() says why not on lane 0).
  if (warp == 0) {
    // ------------------------------------------------------------- operands
    if (elect_one()) {
      // Codes and weights that a kernel before this one wrote (generic proxy) are
      // read by the copy engine (async proxy).
      fence_proxy_async_global();
      const uint64_t pol_tok = l2_policy_evict_last();
      const uint64_t pol_once = l2_policy_evict_first();
      const uint64_t pol_reused = l2_policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0;
      long long issued = 0;   // stages filled
      bool ok = true;
      for (int i = 0; ok && i < my_tiles; ++i) {
        const Tile t =
            tile_at(sm.groups, p.E, p.nb_n, blockIdx.x + static_cast<long long>(i) * gridDim.x);
        // Weights of an expert with one token tile are read once.
        const uint64_t pol_w =
            sm.groups.tile_off[t.e + 1] - sm.groups.tile_off[t.e] > 1 ? pol_reused : pol_once;
        const int boxes = (t.rows + C::kBox - 1) / C::kBox;
        const uint32_t bytes = kTileBytes + 1024 + boxes * C::kBox * kKBytes;
        const long long block = (static_cast<long long>(t.e) * p.nb_n + t.nb) * kb_n;
        for (int kb = 0; kb < kb_n; ++kb) {
          if (!mbar_wait(&sm.empty[stage], phase ^ 1u, p.err, &sm.abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&sm.full[stage], bytes);
          bulk_load_hint(sm.w[stage], p.w + (block + kb) * kTileBytes, kTileBytes, &sm.full[stage],
                         pol_w);
          bulk_load_hint(sm.sfw[stage], p.w_sf + (block + kb) * 1024, 1024, &sm.full[stage], pol_w);
          for (int b = 0; b < boxes; ++b)
            tma_load_2d(sm.t[stage] + b * C::kBox * kKBytes, &tmap, kb * kKBytes,
                        t.row + b * C::kBox, &sm.full[stage], pol_tok);
          ++issued;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // The copies land before the CTA gives its shared memory back, also where
      // it was another warp that gave up (else they have landed long since).
      for (int s = 0; s < STAGES && s < issued; ++s) {
        if (--stage < 0) {
          stage = STAGES - 1;
          phase ^= 1u;
        }
        mbar_wait_limited(&sm.full[stage], phase, kWaitLimitNs);
      }
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
      const Tile t =
          tile_at(sm.groups, p.E, p.nb_n, blockIdx.x + static_cast<long long>(i) * gridDim.x);
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
    __syncwarp();   // (lanes may leave an aborted loop apart)
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issue
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0, acc_phase = 0, set = 0;
      const uint32_t acc = tmem;
      const uint64_t w_desc0 = umma_desc_sw128(smem_u32(sm.w[0]));
      const uint64_t t_desc0 = umma_desc_sw128(smem_u32(sm.t[0]));
      const uint64_t sfw_desc0 = sf_desc(smem_u32(sm.sfw[0]));
      const uint64_t sft_desc0 = sf_desc(smem_u32(sm.sft[0]));
      constexpr uint64_t kKStep = 32 >> 4, kSfChunk = 512 >> 4;
      // (Nothing arrives on `drain` before the end of this branch.)
      bool ok = p.fault == 0 || mbar_wait(&sm.drain, 0, p.err, &sm.abort_flag);
      for (int i = 0; ok && i < my_tiles; ++i) {
        const Tile t =
            tile_at(sm.groups, p.E, p.nb_n, blockIdx.x + static_cast<long long>(i) * gridDim.x);
        const uint32_t n = mma_n(t.rows);
        const uint32_t idesc0 = mxf4_idesc(n, 0);
        if (!mbar_wait(&sm.tmem_empty, acc_phase ^ 1u, p.err, &sm.abort_flag)) break;
        tc_fence_after();
        for (int kb = 0; kb < kb_n; ++kb) {
          if (!mbar_wait(&sm.full[stage], phase, p.err, &sm.abort_flag) ||
              !mbar_wait(&sm.full_sf[stage], phase, p.err, &sm.abort_flag)) {
            ok = false;
            break;
          }
          // The token scales land by cp.async (generic proxy): order them before
          // the tensor core's (async proxy) reads.
          fence_proxy_async_smem();
          tc_fence_after();
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
          set ^= 1u;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        tc_commit(&sm.tmem_full);
        acc_phase ^= 1u;
      }
      // Everything issued above completes before the TMEM is freed.
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
    uint32_t acc_phase = 0;
    for (int i = 0; i < my_tiles; ++i) {
      const Tile t =
          tile_at(sm.groups, p.E, p.nb_n, blockIdx.x + static_cast<long long>(i) * gridDim.x);
      const int n = static_cast<int>(mma_n(t.rows));
      const int c0 = mx::half_begin(n, half), cols = half ? n - c0 : mx::half_begin(n, 1);
      if (!mbar_wait_warp(&sm.tmem_full, acc_phase, p.err, &sm.abort_flag)) break;
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
      mx::store_tile<kCols, kFp16>(v, p.out, p.N, t.nb * 128 + q * 32, t, c0, cols);
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
thread_local int g_debug_fault = 0;   // moe_mxfp4_set_debug

template <int kTok, bool kFp16>
cudaError_t launch(const MxGemm& p, cudaStream_t st) {
  CUtensorMap map;
  if (!mx::map_rows(&map, p.codes, p.K / 2, p.R, kKBytes, Cfg<kTok>::kBox, true))
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

// Most tokens of a tile.  A K block of a tile of n tokens costs about
// kBlockClocks + kTokenClocks * n clocks, and a launch as many tiles one after
// another as there are waves; group sizes are known on the device only, so the
// groups are taken as equal (one group of 1001 rows, 2080 -> 1544: 104 tiles of 128
// tokens or 143 of 96 take 7.0 us, 52 of 256 take 9.2).  Several groups with up to
// kFewRows rows on average get tiles of 128: their sizes scatter, and a group cut in
// two reads its weights twice (96 rows per group: 92 us against 97 with 256 and four
// stages; 128 per group: 33 against 31).
constexpr double kBlockClocks = 300, kTokenClocks = 1.75;
constexpr long long kFewRows = 96;
int tile_cap(int R, int E, int nb_n) {
  if (E > 1 && R <= kFewRows * E) return 128;
  const long long groups = std::min(E, R), rows = (R + groups - 1) / groups;
  const int ctas = sm_count();
  long long best = 256, best_size = 256;
  double least = 0;
  for (long long cap = 256; cap >= 64; cap -= 16) {
    const long long per = (rows + cap - 1) / cap, tiles = per * groups * nb_n;
    const long long size = ((rows + per - 1) / per + 15) / 16 * 16;
    const double cost =
        static_cast<double>((tiles + ctas - 1) / ctas) * (kBlockClocks + kTokenClocks * size);
    if (cap == 256 || cost < least) {
      least = cost;
      best = cap;
      best_size = size;
    }
  }
  // One group's tiles have just the size they were given; several groups get the
  // largest cap of the same cost, so that one a little over the average is not
  // cut in two (144 rows per group: 79 us, 94 with tiles of 144).
  return static_cast<int>(E == 1 ? best_size : best);
}

// CTA pairs (mxfp4_pair.cu) where the average group fills most of a 256-row tile
// and either K is long (kLongBlocks K blocks) and the 256 x 256 tiles make two
// waves of pairs, or they make forty.  Pairs against this kernel, power-capped, us:
//   7168 -> 4096: 2048 rows x 32 groups 827 / 892, 256 x 32 152 / 161, 768 x 4 (2.6
//   waves) 50 / 53; one group of 1024 rows (under a wave) 17.6 / 15.4
//   4096 -> 4096: 2048 x 8 134 / 139, 8192 x 1 64 / 64; 2816 -> 4096: 2048 x 8 100 / 105
//   2048 -> 7168: 2048 x 32 (97 waves) 546 / 566, 1024 x 8 (12 waves) 76.7 / 76.1;
//   2048 -> 4096: 8192 x 8 (55 waves) 300 / 307, 512 x 64 (27) 195 / 191, 192 x 64
//   92 / 88; 2048 -> 8192: 4096 x 1 (7 waves) 40 / 38.6
constexpr int kLongBlocks = 11;
bool use_pairs(int R, int E, int N, int K) {
  const long long tiles = (R / 256) * ((N + 255ll) / 256);
  const int waves = (K + 255) / 256 >= kLongBlocks ? 2 : 40;   // of sm_count() / 2 pairs
  return R >= 224ll * E && 2 * tiles >= static_cast<long long>(waves) * sm_count();
}

}  // namespace

bool mx::map_rows(CUtensorMap* m, const void* base, uint64_t width, uint64_t rows, uint32_t box,
                  uint32_t box_rows, bool swizzle128) {
  const EncodeTiledFn enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  std::memset(m, 0, sizeof(*m));
  const cuuint64_t dims[2] = {width, rows};
  const cuuint64_t strides[1] = {width};
  const cuuint32_t boxes[2] = {box, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, boxes,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace moe

extern "C" {

moe_status moe_mxfp4_set_debug(int flags) {
  if (flags & ~1) return MOE_ERR_INVALID_ARG;
  moe::g_debug_fault = flags & 1;
  return MOE_OK;
}

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
  if (R < 1 || !moe::mx_gemm_sizes_ok(E, N, K)) return 0;
  return 256 + (moe::use_pairs(R, E, N, K) ? moe::mx_pair_record_bytes(R, E, K) : 0);
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
  const long long tiles = static_cast<long long>(E) * ((N + 127) / 128) * ((K + 255) / 256);
  const moe::Buffer buffers[] = {
      {codes, rb * (K / 2), false},
      {scales, (K + 127) / 128 * rb * 4, false},
      {offsets, (E + 1) * 4ll, false},
      {w_tiled, tiles * static_cast<long long>(moe::kTileBytes), false},
      {w_scales_chunked, tiles * 1024, false},
      {out, rb * N * 2, true},
      {workspace, static_cast<long long>(moe_mxfp4_workspace_bytes(R, E, N, K)), true}};
  if (moe::outputs_overlap(buffers)) return MOE_ERR_INVALID_ARG;
  moe::MxGemm p{};
  p.R = R;
  p.E = E;
  p.N = N;
  p.K = K;
  p.nb_n = (N + 127) / 128;
  p.kb_n = (K + 255) / 256;
  p.offsets = offsets;
  p.w = w_tiled;
  p.w_sf = w_scales_chunked;
  p.codes = codes;
  p.scales = scales;
  p.out = static_cast<uint16_t*>(out);
  p.err = static_cast<uint32_t*>(workspace);
  p.records = static_cast<uint8_t*>(workspace) + 256;
  p.fault = moe::g_debug_fault;
  p.cap = moe::tile_cap(R, E, p.nb_n);
  auto st = reinterpret_cast<cudaStream_t>(stream);
  const bool fp16 = dtype == MOE_T_FP16;
  if (moe::use_pairs(R, E, N, K)) {
    p.cap = 256;
    return moe::launch_mx_pairs(p, fp16, st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  cudaError_t e;
  if (p.cap <= 128)
    e = fp16 ? moe::launch<128, true>(p, st) : moe::launch<128, false>(p, st);
  else
    e = fp16 ? moe::launch<256, true>(p, st) : moe::launch<256, false>(p, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"

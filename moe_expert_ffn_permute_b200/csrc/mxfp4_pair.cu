// mxfp4_pair.cu -- the MXFP4 product (mxfp4_gemm.cu) on CTA pairs, for groups
// with many rows: two SMs compute 256 weight rows x up to 256 tokens with
// tcgen05.mma.cta_group::2.  Each SM loads its own 128 weight rows and half of
// the tile's tokens, so a K block moves 35 KB per SM instead of 52 KB and a
// token row is read from shared memory once for 256 features.
//
// All of a stage's operands arrive by TMA on the leader's barrier.  The token
// scales' group-major words cannot be brought into the tensor core's layout by a
// TMA box (4-byte pieces), so a first launch writes them as records, 2 KB per
// token tile and K block (1/16 of the codes' bytes); both SMs of a pair read the
// whole record, since each applies the scales of all the tile's tokens.
//
// 65536 rows, 7168 -> 4096, 32 experts: 705 us (5.5 PFLOP/s) for a first call, 814
// under the 1 kW cap at 1.35 GHz, where every byte moved costs clocks: without the
// MMAs 505 us, without the output's stores 765, without the token loads 700.  Short K
// is bound by the output, 4 bytes a lane and store: 2048 -> 7168, 65536 rows, 32
// experts, 550 us, 453 without the stores (289 at the tensor rate, 337 under the cap).
//
// Tiles, warps and the epilogue are those of mxfp4_gemm.cu; the MMA warp of the
// leader (rank 0) issues for both SMs.  No TMA load uses cluster multicast.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "internal.h"
#include "mxfp4_tiles.cuh"
#include "sm100_pair.cuh"

namespace moe {
namespace {

using mx::kKBytes;
using mx::Tile;
using mx::tile_at;
using mx::uniform;

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kStages = 6;
constexpr int kHalfTok = 128;            // most tokens of a tile's half
constexpr int kRecordBytes = 2048;       // [128-wide half][128-row chunk][512]
constexpr uint32_t kTmemCols = 512;
// TMEM columns as in mxfp4_gemm.cu: the accumulator, then two scale sets.
constexpr uint32_t kSfCol = 256, kSfSet = 32, kSfTokens = 8;
// Bytes of a stage that land in both CTAs together.
constexpr uint32_t kStageTx = 2 * (kTileBytes + kHalfTok * kKBytes + 1024 + kRecordBytes);

struct __align__(1024) Smem {
  uint8_t w[kStages][kTileBytes];
  uint8_t t[kStages][kHalfTok * kKBytes];
  uint8_t sfw[kStages][1024];
  uint8_t sft[kStages][kRecordBytes];
  uint64_t full[kStages];    // leader only: the copies of both CTAs
  uint64_t empty[kStages];   // each CTA
  uint64_t tmem_full;        // each CTA
  uint64_t tmem_empty;       // leader only: the epilogue warps of both
  uint64_t drain;            // leader only
  mx::Groups groups;
  uint32_t tmem_base;
  int abort_flag;
};

struct Maps {
  CUtensorMap w, t, sfw, sft;
};

// A tile's MMA columns: its tokens rounded up to 16 (each CTA has half of them).
__device__ __forceinline__ int mma_n(int rows) { return (rows + 15) & ~15; }

// Token scales -> records.  One thread per 16 bytes: lane l of a chunk holds the
// words of rows l, l + 32, l + 64, l + 96.
__global__ void __launch_bounds__(256) scale_records_kernel(const MxGemm p) {
  __shared__ mx::Groups groups;
  griddep_launch_dependents();
  griddep_wait();
  if (threadIdx.x < 32) mx::find_groups(groups, p.offsets, p.R, p.E, p.cap);
  __syncthreads();
  const int k_groups = (p.K + 127) / 128;
  const long long n = static_cast<long long>(groups.tile_off[p.E]) * p.kb_n * (kRecordBytes / 16);
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
    const int l = static_cast<int>(i & 31), c = static_cast<int>(i >> 5) & 1;
    const int h = static_cast<int>(i >> 6) & 1;
    const long long rec = i >> 7;
    const long long tt = rec / p.kb_n;
    const int g = 2 * static_cast<int>(rec - tt * p.kb_n) + h;
    const Tile t = tile_at(groups, p.E, 1, tt);
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = 128 * c + 32 * q + l;
      // (Rows past the tile and blocks past K: byte 0, a finite scale.)
      w[q] = r < t.rows && g < k_groups
                 ? __ldg(reinterpret_cast<const uint32_t*>(p.scales) +
                         static_cast<size_t>(g) * p.R + t.row + r)
                 : 0u;
    }
    reinterpret_cast<uint4*>(p.records)[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <bool kFp16>
__global__ void __launch_bounds__(kThreads, 1)
    mxfp4_pair_kernel(const __grid_constant__ Maps tm, const MxGemm p) {
  extern __shared__ uint8_t smem_raw[];
  griddep_launch_dependents();
  Smem& sm = *reinterpret_cast<Smem*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = uniform(static_cast<int>(threadIdx.x >> 5));
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.full[s], 1);   // the leader's expect-tx arrive; bytes from both CTAs
      mbar_init(&sm.empty[s], 1);
    }
    mbar_init(&sm.tmem_full, 1);
    mbar_init(&sm.tmem_empty, 2 * kEpiWarps);
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tm.w);
    tma_prefetch_desc(&tm.t);
    tma_prefetch_desc(&tm.sfw);
    tma_prefetch_desc(&tm.sft);
  }
  if (warp == 1) {
    tmem_alloc_pair(&sm.tmem_base, kTmemCols);
    tmem_relinquish_pair();
  }
  griddep_wait();
  if (warp == 2) mx::find_groups(sm.groups, p.offsets, p.R, p.E, p.cap);
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers exist before any remote operation
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const int kb_n = p.kb_n;
  const int pairs_n = (p.nb_n + 1) / 2;   // 256-row weight blocks per token tile
  const long long tiles = static_cast<long long>(sm.groups.tile_off[p.E]) * pairs_n;
  const int clusters = gridDim.x / 2, cluster = blockIdx.x / 2;
  const int my_tiles = uniform(static_cast<int>((tiles - cluster + clusters - 1) / clusters));
  auto tile = [&](int i) {
    return tile_at(sm.groups, p.E, pairs_n, cluster + static_cast<long long>(i) * clusters);
  };

  if (warp == 0) {
    // ------------------------------------------------------------- operands
    if (elect_one()) {
      // Codes, records and weights that a kernel before this one wrote (generic
      // proxy) are read by the copy engine (async proxy).
      fence_proxy_async_global();
      const uint64_t pol_tok = l2_policy_evict_last();
      const uint64_t pol_w = l2_policy_evict_normal();
      const uint32_t lead_full0 = mapa_shared(smem_u32(&sm.full[0]), 0);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int i = 0; ok && i < my_tiles; ++i) {
        const Tile t = tile(i);
        // A pair whose second block is past N reads some other block (or zeros
        // past the last one) and stores nothing of it.
        const long long nb = 2ll * t.nb + rank;
        const int block = static_cast<int>((static_cast<long long>(t.e) * p.nb_n + nb) * kb_n);
        const int row = mx::half_row(t.row, mma_n(t.rows), rank, p.R);
        const int rec = static_cast<int>(
            (cluster + static_cast<long long>(i) * clusters) / pairs_n * kb_n);
        for (int kb = 0; kb < kb_n; ++kb) {
          if (!mbar_wait(&sm.empty[stage], phase ^ 1u, p.err, &sm.abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t bar = lead_full0 + stage * 8;
          if (leader) mbar_arrive_expect_tx(&sm.full[stage], kStageTx);
          tma_load_2d_pair(sm.w[stage], &tm.w, 0, (block + kb) * 128, bar, pol_w);
          tma_load_2d_pair(sm.t[stage], &tm.t, kb * kKBytes, row, bar, pol_tok);
          tma_load_2d_pair(sm.sfw[stage], &tm.sfw, 0, (block + kb) * 4, bar, pol_w);
          tma_load_2d_pair(sm.sft[stage], &tm.sft, 0, (rec + kb) * 8, bar, pol_tok);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issue
    if (leader && elect_one()) {
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
        const uint32_t n = static_cast<uint32_t>(mma_n(tile(i).rows));
        const uint32_t idesc0 = mxf4_idesc_m256(n, 0);
        if (!mbar_wait_cluster(&sm.tmem_empty, acc_phase ^ 1u, p.err, &sm.abort_flag)) break;
        tc_fence_after();
        for (int kb = 0; kb < kb_n; ++kb) {
          if (!mbar_wait(&sm.full[stage], phase, p.err, &sm.abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sfw = acc + kSfCol + set * kSfSet;
          const uint32_t sft = sfw + kSfTokens;
          const uint64_t sfwd = sfw_desc0 + static_cast<uint64_t>(stage) * (1024 >> 4);
          const uint64_t sftd = sft_desc0 + static_cast<uint64_t>(stage) * (kRecordBytes >> 4);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            tmem_cp_pair_32x128b_warpx4(sfw + 4 * h, sfwd + h * kSfChunk);
            tmem_cp_pair_32x128b_warpx4(sft + 8 * h, sftd + 2 * h * kSfChunk);
            if (n > 128)
              tmem_cp_pair_32x128b_warpx4(sft + 8 * h + 4, sftd + (2 * h + 1) * kSfChunk);
          }
          const uint64_t wd = w_desc0 + static_cast<uint64_t>(stage) * (kTileBytes >> 4);
          const uint64_t td = t_desc0 + static_cast<uint64_t>(stage) * (kHalfTok * kKBytes >> 4);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint32_t h = ks >> 1, sf_id = (ks & 1) * 2;
            mma_mxf4_pair(acc, wd + ks * kKStep, td + ks * kKStep,
                          idesc0 | (sf_id << 4) | (sf_id << 29), (sfw + 4 * h) | (sf_id << 30),
                          (sft + 8 * h) | (sf_id << 30), (kb > 0 || ks > 0) ? 1u : 0u);
          }
          tc_commit_pair_multicast(&sm.empty[stage], 0x3);
          set ^= 1u;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        tc_commit_pair_multicast(&sm.tmem_full, 0x3);
        acc_phase ^= 1u;
      }
      // Everything issued above (into both CTAs' TMEM) completes before the pair
      // frees its TMEM.
      tc_commit_pair_multicast(&sm.drain, 0x1);
      if (!mbar_wait_limited(&sm.drain, 0, kWaitLimitNs)) atomicOr(p.err, kErrTimeoutBit);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------- epilogue
    const int q = warp & 3;              // TMEM sub-partition: lanes 32q..32q+31
    const int half = (warp - 4) >> 2;    // which half of the tile's token columns
    constexpr int kCols = 128;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const uint32_t lead_tmem_empty = mapa_shared(smem_u32(&sm.tmem_empty), 0);
    uint32_t acc_phase = 0;
    for (int i = 0; i < my_tiles; ++i) {
      const Tile t = tile(i);
      const int n = mma_n(t.rows);
      const int c0 = mx::half_begin(n, half), cols = half ? n - c0 : mx::half_begin(n, 1);
      if (!mbar_wait_warp(&sm.tmem_full, acc_phase, p.err, &sm.abort_flag)) break;
      acc_phase ^= 1u;
      tc_fence_after();
      uint32_t v[kCols];
#pragma unroll
      for (int c = 0; c < kCols / 32; ++c)
        tmem_ld_32x32b_x32(lanes + c0 + c * 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32 * c));
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(lead_tmem_empty);
      mx::store_tile<kCols, kFp16>(v, p.out, p.N, (2 * t.nb + rank) * 128 + q * 32, t, c0, cols);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (sm.abort_flag) {
    // Copies in flight (microseconds) land before the shared memory is given back,
    // whichever warp gave up.  Their barrier is the leader's and may never
    // complete, so this waits by time.
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 1000000ull) __nanosleep(1000);
    __syncthreads();
  }
  cluster_sync();   // no remote operation targets a CTA that has left
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// Token tiles there can be.
long long most_token_tiles(int R, int E, int cap) { return R / cap + std::min(E, R); }

}  // namespace

size_t mx_pair_record_bytes(int R, int E, int K) {
  return static_cast<size_t>(most_token_tiles(R, E, 2 * kHalfTok)) * ((K + 255) / 256) *
         kRecordBytes;
}

cudaError_t launch_mx_pairs(const MxGemm& p, bool fp16, cudaStream_t st) {
  const long long token_tiles = most_token_tiles(p.R, p.E, p.cap);
  const uint64_t blocks = static_cast<uint64_t>(p.E) * p.nb_n * p.kb_n;
  Maps m;
  if (!mx::map_rows(&m.w, p.w, 128, blocks * 128, 128, 128, false) ||
      !mx::map_rows(&m.t, p.codes, p.K / 2, p.R, kKBytes, kHalfTok, true) ||
      !mx::map_rows(&m.sfw, p.w_sf, 256, blocks * 4, 256, 4, false) ||
      !mx::map_rows(&m.sft, p.records, 256, token_tiles * p.kb_n * 8, 256, 8, false))
    return cudaErrorInvalidValue;
  const long long units = token_tiles * p.kb_n * (kRecordBytes / 16);
  const int record_blocks =
      static_cast<int>(std::min<long long>((units + 255) / 256, 4ll * sm_count()));
  cudaError_t e = launch_pdl(scale_records_kernel, dim3(record_blocks), dim3(256), 0, st, p);
  if (e != cudaSuccess) return e;
  auto kern = fp16 ? mxfp4_pair_kernel<true> : mxfp4_pair_kernel<false>;
  const size_t smem = sizeof(Smem) + 1024;
  static_assert(sizeof(Smem) + 1024 <= 232448, "shared memory of a CTA");
  e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(kern), static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const long long most = token_tiles * ((p.nb_n + 1) / 2);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * static_cast<unsigned>(std::min<long long>(sm_count() / 2, most)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, m, p);
}

}  // namespace moe

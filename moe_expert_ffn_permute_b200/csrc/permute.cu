// permute.cu -- token rows copied into expert order and back, and the
// gradients of both, on plain row-major tensors outside the fused layer:
//   moe_permute            rows[inv[t,j]] = x[t]
//   moe_permute_backward   dx[t]  = sum_j drows[inv[t,j]]
//   moe_unpermute          out[t] = sum_j w[t,j] * rows[inv[t,j]]
//   moe_unpermute_backward drows[inv[t,j]] = w[t,j] * dout[t],
//                          dw[t,j] = <dout[t], rows[inv[t,j]]>
// inv is what moe_route() computes (position of slot t*k + j in expert order,
// -1 for a slot that is not routed); positions outside [0, T*k) are skipped
// like -1, so no index can leave a buffer.  Sums run in fp32 with j ascending
// and no atomics: the results do not depend on the order blocks run in.
// All of it is HBM-bound: every kernel is one pass that reads each input row
// once and writes each output row once.
#include <cuda_runtime.h>

#include <algorithm>

#include "args.h"
#include "elem.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kSlotGroup = 8;   // slots whose stores the copy issues together
// Slots whose rows the sum loads together (8192 tokens, top-8, 7168 wide: 152 us;
// eight take 157, their 114 registers leave two blocks per SM; two 155).
constexpr int kSumGroup = 4;
// 16-byte chunks of a row per thread of the copy and the sum (one in each half
// of the row), as in the layer's combine.
constexpr int kCpt = 2;

__device__ __forceinline__ bool routed(int p, long long S) { return p >= 0 && p < S; }

// One thread per (token, pair of chunks): the token's chunk is read once and
// written to each of its slots' rows.  Bound by the writes: 8192 tokens to 8 slots
// each, 7168 wide in bf16, take 170 us, 6.2 TB/s of their 1.06 GB.  Streaming
// stores (the rows exceed L2 where the time matters) took 1.5% off.
template <class V>
__global__ void __launch_bounds__(kThreads) permute_kernel(const V* __restrict__ x,
                                                           const int32_t* __restrict__ inv, int T,
                                                           long long vecs, int k,
                                                           V* __restrict__ rows) {
  griddep_launch_dependents();
  griddep_wait();
  const long long half = (vecs + kCpt - 1) / kCpt;
  const long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x;
  if (i >= T * half) return;
  const long long t = i / half;
  const long long c = i - t * half;
  const bool second = c + half < vecs;
  const long long S = static_cast<long long>(T) * k;
  const V v0 = __ldg(x + t * vecs + c);
  V v1 = v0;
  if (second) v1 = __ldg(x + t * vecs + c + half);
  for (int j0 = 0; j0 < k; j0 += kSlotGroup) {
    int p[kSlotGroup];
#pragma unroll
    for (int j = 0; j < kSlotGroup; ++j) p[j] = j0 + j < k ? __ldg(&inv[t * k + j0 + j]) : -1;
#pragma unroll
    for (int j = 0; j < kSlotGroup; ++j) {
      if (!routed(p[j], S)) continue;
      V* row = rows + p[j] * vecs;
      __stcs(row + c, v0);
      if (second) __stcs(row + c + half, v1);
    }
  }
}

// The same thread layout the other way round: kSumGroup rows' chunks are loaded
// together and summed in fp32, j ascending.  topk_w == nullptr: weights 1.  Bound
// by the reads: the copy's size above, 5% of the slots masked, takes 152 us, 6.65
// TB/s of its 1.01 GB (156 where one of a thread's two stores does not stream).
template <int kDtype>
__global__ void __launch_bounds__(kThreads) unpermute_kernel(
    const uint4* __restrict__ rows, const int32_t* __restrict__ inv,
    const float* __restrict__ topk_w, int T, long long vecs, int k, uint4* __restrict__ out) {
  using E = Elem<kDtype>;
  griddep_launch_dependents();
  griddep_wait();
  const long long half = (vecs + kCpt - 1) / kCpt;
  const long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x;
  if (i >= T * half) return;
  const long long t = i / half;
  const long long c = i - t * half;
  const bool second = c + half < vecs;
  const long long S = static_cast<long long>(T) * k;
  float acc[kCpt][E::kPerVec];
#pragma unroll
  for (int h = 0; h < kCpt; ++h)
#pragma unroll
    for (int q = 0; q < E::kPerVec; ++q) acc[h][q] = 0.0f;
  for (int j0 = 0; j0 < k; j0 += kSumGroup) {
    int p[kSumGroup];
    float w[kSumGroup];
    uint4 v[kSumGroup][kCpt];
#pragma unroll
    for (int j = 0; j < kSumGroup; ++j) {
      const bool in = j0 + j < k;
      p[j] = in ? __ldg(&inv[t * k + j0 + j]) : -1;
      w[j] = in && topk_w != nullptr ? __ldg(&topk_w[t * k + j0 + j]) : 1.0f;
    }
#pragma unroll
    for (int j = 0; j < kSumGroup; ++j) {
      const bool in = routed(p[j], S);
      const uint4* row = rows + static_cast<long long>(in ? p[j] : 0) * vecs;
      v[j][0] = in ? __ldcs(row + c) : make_uint4(0, 0, 0, 0);
      v[j][1] = in && second ? __ldcs(row + c + half) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < kSumGroup; ++j) {
      // A skipped slot adds nothing (no product with 0: its weight may be NaN).
      if (!routed(p[j], S)) continue;
#pragma unroll
      for (int h = 0; h < kCpt; ++h) {
        float f[E::kPerVec];
        E::unpack(v[j][h], f);
#pragma unroll
        for (int q = 0; q < E::kPerVec; ++q) acc[h][q] = fmaf(w[j], f[q], acc[h][q]);
      }
    }
  }
  __stcs(out + t * vecs + c, E::pack(acc[0]));
  if (second) __stcs(out + t * vecs + c + half, E::pack(acc[1]));
}

// One block per (token, group of kJ slots): dout's row is read once for the
// group, each slot's row once; the dot products are summed over the block in a
// fixed order.  4096 tokens, top-8, 7168 wide in bf16: 150 us, 6.35 TB/s of its
// 0.95 GB.  drows or dw may be null (rows is read only for dw).
template <int kDtype, int kJ>
__global__ void __launch_bounds__(kThreads) unpermute_backward_kernel(
    const uint4* __restrict__ dout, const uint4* __restrict__ rows,
    const int32_t* __restrict__ inv, const float* __restrict__ topk_w, int T, long long vecs, int k,
    uint4* __restrict__ drows, float* __restrict__ dw) {
  using E = Elem<kDtype>;
  __shared__ float part[kThreads / 32][kJ];
  griddep_launch_dependents();
  griddep_wait();
  const int groups = (k + kJ - 1) / kJ;
  const long long t = blockIdx.x / groups;
  const int j0 = static_cast<int>(blockIdx.x - t * groups) * kJ;
  const long long S = static_cast<long long>(T) * k;
  long long p[kJ];
  float w[kJ], dot[kJ];
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
    const bool in = j0 + j < k;
    const int pj = in ? __ldg(&inv[t * k + j0 + j]) : -1;
    p[j] = routed(pj, S) ? pj * vecs : -1;
    w[j] = in ? __ldg(&topk_w[t * k + j0 + j]) : 0.0f;
    dot[j] = 0.0f;
  }
  for (long long c = threadIdx.x; c < vecs; c += blockDim.x) {
    const uint4 dv = __ldg(dout + t * vecs + c);
    uint4 v[kJ];
    if (dw != nullptr) {
#pragma unroll
      for (int j = 0; j < kJ; ++j)
        v[j] = p[j] >= 0 ? __ldcs(rows + p[j] + c) : make_uint4(0, 0, 0, 0);
    }
    float d[E::kPerVec];
    E::unpack(dv, d);
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      if (p[j] < 0) continue;
      if (dw != nullptr) {
        float f[E::kPerVec];
        E::unpack(v[j], f);
#pragma unroll
        for (int q = 0; q < E::kPerVec; ++q) dot[j] = fmaf(d[q], f[q], dot[j]);
      }
      if (drows != nullptr) {
        float g[E::kPerVec];
#pragma unroll
        for (int q = 0; q < E::kPerVec; ++q) g[q] = w[j] * d[q];
        __stcs(drows + p[j] + c, E::pack(g));
      }
    }
  }
  if (dw == nullptr) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < kJ; ++j) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
    if (lane == 0) part[warp][j] = dot[j];
  }
  __syncthreads();
  const int j = threadIdx.x;
  if (j < kJ && j0 + j < k) {
    float sum = 0.0f;
    for (int q = 0; q < static_cast<int>(blockDim.x) / 32; ++q) sum += part[q][j];
    dw[t * k + j0 + j] = sum;   // a slot that is not routed: 0
  }
}

// Blocks of kThreads for one thread per (token, pair of chunks); 0 if the grid
// would exceed its limit, or the rows' bytes 64 bits.
unsigned copy_blocks(int T, long long vecs, int k) {
  const long long half = (vecs + kCpt - 1) / kCpt;
  if (vecs > (1ll << 58) / T / k) return 0;
  const long long blocks = (T * half + kThreads - 1) / kThreads;
  return blocks < (1ll << 31) ? static_cast<unsigned>(blocks) : 0u;
}

// Sizes shared by the calls on rows of H elements.
moe_status check_rows(int dtype, int T, int H, int k) {
  if (!elem_ok(dtype) || T < 1 || H < 1 || k < 1) return MOE_ERR_INVALID_ARG;
  if (static_cast<long long>(T) * k >= (1ll << 31)) return MOE_ERR_INVALID_ARG;
  const long long row_bytes = static_cast<long long>(H) * elem_bytes(dtype);
  if (k > kMaxSlotsPerToken) return MOE_ERR_UNSUPPORTED;
  if (row_bytes % 16 != 0 || copy_blocks(T, row_bytes / 16, k) == 0) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status sum_rows(const void* rows, int dtype, int T, int H, int k, const int32_t* inv,
                    const float* topk_w, void* out, moe_stream_t stream) {
  if (rows == nullptr || inv == nullptr || out == nullptr) return MOE_ERR_INVALID_ARG;
  const moe_status s = check_rows(dtype, T, H, k);
  if (s != MOE_OK) return s;
  if (!aligned_to(rows, 16) || !aligned_to(out, 16) || !aligned_to(inv, 4) ||
      !aligned_to(topk_w, 4))
    return MOE_ERR_ALIGNMENT;
  const long long vecs = static_cast<long long>(H) * elem_bytes(dtype) / 16;
  const unsigned blocks = copy_blocks(T, vecs, k);
  const long long S = static_cast<long long>(T) * k;
  const Buffer buffers[] = {{rows, S * vecs * 16, false},
                            {inv, S * 4, false},
                            {topk_w, S * 4, false},
                            {out, T * vecs * 16, true}};
  if (outputs_overlap(buffers)) return MOE_ERR_INVALID_ARG;
  auto kern = dtype == MOE_T_BF16   ? unpermute_kernel<MOE_T_BF16>
              : dtype == MOE_T_FP16 ? unpermute_kernel<MOE_T_FP16>
                                    : unpermute_kernel<MOE_T_FP32>;
  const cudaError_t e = launch_pdl(kern, dim3(blocks), dim3(kThreads), 0,
                                   reinterpret_cast<cudaStream_t>(stream),
                                   static_cast<const uint4*>(rows), inv, topk_w, T, vecs, k,
                                   static_cast<uint4*>(out));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <int kDtype, int kJ>
cudaError_t launch_backward(const void* dout, const void* rows, const int32_t* inv,
                            const float* topk_w, int T, long long vecs, int k, void* drows,
                            float* dw, cudaStream_t st) {
  // Threads that each take the same number of chunks of the row: as many as
  // there may be where a block has one slot; with four, blocks of about seven
  // chunks a thread (128 threads on rows of 14 KB: 150 us against 155 with 224;
  // 256 on rows of 28 KB: 84 us against 88 with 128).
  const long long fewest = (vecs + kThreads - 1) / kThreads;
  const long long rounds =
      kJ == 1 ? fewest : std::max(fewest, std::min(7ll, (vecs + 127) / 128));
  const unsigned threads = static_cast<unsigned>(((vecs + rounds - 1) / rounds + 31) / 32 * 32);
  const unsigned blocks = static_cast<unsigned>(T) * ((k + kJ - 1) / kJ);
  return launch_pdl(unpermute_backward_kernel<kDtype, kJ>, dim3(blocks), dim3(threads), 0, st,
                    static_cast<const uint4*>(dout), static_cast<const uint4*>(rows), inv, topk_w,
                    T, vecs, k, static_cast<uint4*>(drows), dw);
}

// Slots of a token that a block of the gradient takes: four (4096 tokens, top-8,
// 7168 wide in bf16: 150 us; eight take 163, their 109 registers leave few blocks
// per SM; two 171, one 173, re-reading dout), or one below two tokens per SM, where
// a token's slots should spread over the SMs (148 SMs, one slot / four, same width: 37
// tokens 3.4 / 5.4 us, 200 8.5 / 10.4, 296 11.5 / 12.1, 400 15.0 / 13.7; rows of
// 6 KB cross over earlier, at most 0.6 us apart).
constexpr int kBackSlots = 4;

template <int kDtype>
cudaError_t launch_backward_any(const void* dout, const void* rows, const int32_t* inv,
                                const float* topk_w, int T, long long vecs, int k, void* drows,
                                float* dw, cudaStream_t st) {
  if (T < 2 * sm_count() || k == 1)
    return launch_backward<kDtype, 1>(dout, rows, inv, topk_w, T, vecs, k, drows, dw, st);
  return launch_backward<kDtype, kBackSlots>(dout, rows, inv, topk_w, T, vecs, k, drows, dw, st);
}

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_permute(const void* x, int T, int64_t row_bytes, int k, const int32_t* inv,
                       void* rows, moe_stream_t stream) {
  if (x == nullptr || inv == nullptr || rows == nullptr) return MOE_ERR_INVALID_ARG;
  if (T < 1 || row_bytes < 1 || k < 1 || static_cast<long long>(T) * k >= (1ll << 31))
    return MOE_ERR_INVALID_ARG;
  if (row_bytes % 4 != 0 || k > moe::kMaxSlotsPerToken) return MOE_ERR_UNSUPPORTED;
  if (!moe::aligned_to(x, 16) || !moe::aligned_to(rows, 16) || !moe::aligned_to(inv, 4))
    return MOE_ERR_ALIGNMENT;
  auto st = reinterpret_cast<cudaStream_t>(stream);
  // Rows of whole 16-byte vectors keep every row 16-byte aligned; others
  // (scale bytes of odd sizes) go word by word, at about half the rate (65536
  // tokens, top-8: rows of 1792 bytes 189 us, of 1796 bytes 358; 224 and 228
  // bytes 28 and 58).
  const bool wide = row_bytes % 16 == 0;
  const long long vecs = row_bytes / (wide ? 16 : 4);
  const unsigned blocks = moe::copy_blocks(T, vecs, k);
  if (blocks == 0) return MOE_ERR_UNSUPPORTED;
  const long long S = static_cast<long long>(T) * k;
  const moe::Buffer buffers[] = {
      {x, T * row_bytes, false}, {inv, S * 4, false}, {rows, S * row_bytes, true}};
  if (moe::outputs_overlap(buffers)) return MOE_ERR_INVALID_ARG;
  const cudaError_t e =
      wide ? moe::launch_pdl(moe::permute_kernel<uint4>, dim3(blocks), dim3(moe::kThreads), 0, st,
                             static_cast<const uint4*>(x), inv, T, vecs, k,
                             static_cast<uint4*>(rows))
           : moe::launch_pdl(moe::permute_kernel<uint32_t>, dim3(blocks), dim3(moe::kThreads), 0,
                             st, static_cast<const uint32_t*>(x), inv, T, vecs, k,
                             static_cast<uint32_t*>(rows));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_permute_backward(const void* drows, int dtype, int T, int H, int k,
                                const int32_t* inv, void* dx, moe_stream_t stream) {
  return moe::sum_rows(drows, dtype, T, H, k, inv, nullptr, dx, stream);
}

moe_status moe_unpermute(const void* rows, int dtype, int T, int H, int k, const int32_t* inv,
                         const float* topk_w, void* out, moe_stream_t stream) {
  if (topk_w == nullptr) return MOE_ERR_INVALID_ARG;
  return moe::sum_rows(rows, dtype, T, H, k, inv, topk_w, out, stream);
}

moe_status moe_unpermute_backward(const void* dout, const void* rows, int dtype, int T, int H,
                                  int k, const int32_t* inv, const float* topk_w, void* drows,
                                  float* dw, moe_stream_t stream) {
  if (dout == nullptr || inv == nullptr || topk_w == nullptr) return MOE_ERR_INVALID_ARG;
  if (drows == nullptr && dw == nullptr) return MOE_ERR_INVALID_ARG;
  if (dw != nullptr && rows == nullptr) return MOE_ERR_INVALID_ARG;
  const moe_status s = moe::check_rows(dtype, T, H, k);
  if (s != MOE_OK) return s;
  if (!moe::aligned_to(dout, 16) || !moe::aligned_to(rows, 16) || !moe::aligned_to(drows, 16) ||
      !moe::aligned_to(inv, 4) || !moe::aligned_to(topk_w, 4) || !moe::aligned_to(dw, 4))
    return MOE_ERR_ALIGNMENT;
  const long long vecs = static_cast<long long>(H) * moe::elem_bytes(dtype) / 16;
  const long long S = static_cast<long long>(T) * k;
  const moe::Buffer buffers[] = {{dout, T * vecs * 16, false},
                                 {dw != nullptr ? rows : nullptr, S * vecs * 16, false},
                                 {inv, S * 4, false},
                                 {topk_w, S * 4, false},
                                 {drows, S * vecs * 16, true},
                                 {dw, S * 4, true}};
  if (moe::outputs_overlap(buffers)) return MOE_ERR_INVALID_ARG;
  auto st = reinterpret_cast<cudaStream_t>(stream);
  auto launch = dtype == MOE_T_BF16   ? moe::launch_backward_any<MOE_T_BF16>
                : dtype == MOE_T_FP16 ? moe::launch_backward_any<MOE_T_FP16>
                                      : moe::launch_backward_any<MOE_T_FP32>;
  const cudaError_t e = launch(dout, rows, inv, topk_w, T, vecs, k, drows, dw, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"

// mxfp4.cu -- MXFP4 on the GPU: E2M1 codes, two to a byte, with one UE8M0 scale
// per 32 elements of a row.
//   quantise:   n = the smallest integer >= -127 with amax <= 6 * 2^n over the
//               32 elements, scale byte n + 127, codes = E2M1 of x / 2^n, to
//               nearest with ties to even (x / 2^n <= 6: nothing saturates).
//               A block that holds a NaN or an infinity gets scale byte 255
//               (NaN) and codes 0: all its values are NaN.
//   dequantise: value = E2M1 * 2^(byte - 127), exact in bf16 and fp32 (infinity
//               from 2^128 on).
//   prepack:    weights into the tiles and scale chunks the MXFP4 product reads,
//               once per weight set (32 x 4096 x 7168: 217 us for both launches,
//               4.6 TB/s; the scales, read by bytes, take 59 of them).
// The division by 2^n is exact, so the codes depend on the inputs alone.
// HBM-bound: quantise reads an element once and writes 17/32 byte for it, once
// per slot when it also copies the rows into expert order (8192 x 7168 bf16: in
// order 27 us, 5.5 TB/s; to 8 slots each 68 us, 5.4 TB/s, group-major scales, of
// which each row's words lie apart, costing 5 of them); dequantise 65536 x 7168
// to bf16 177 us, 6.7 TB/s.  32-byte loads and stores: with 16 bytes a thread's two
// accesses each touch half of their sectors.
#include <cuda_runtime.h>

#include "args.h"
#include "elem.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kSlotGroup = 8;    // slots whose stores are issued together
constexpr int kUnit = 16;        // elements a thread owns: half a block
constexpr int kGroupUnits = 8;   // threads of a 128-wide group (four blocks)
constexpr int kMaxRow = 1 << 28; // elements of a row (bytes of 2^31 rows fit 64 bits)

// UE8M0 byte of a block from the largest magnitude's fp32 bits: 6 = 1.5 * 2^2,
// so with amax = m * 2^e, m in [1, 2), n = e - 2 if m <= 1.5, else e - 1.
__device__ __forceinline__ int mx_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return 255;
  const int e = static_cast<int>(amax_bits >> 23);   // biased; 0 below 2^-126
  const int byte = (amax_bits & 0x7FFFFFu) <= 0x400000u ? e - 2 : e - 1;
  return byte < 0 ? 0 : byte;
}

// Eight fp32 -> eight E2M1 codes, round to nearest even, the first in the lowest
// nibble.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&f)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

// 32 bytes in one instruction: a thread's 16-bit unit, or half of its fp32 one.
struct alignas(32) Vec32 {
  uint32_t w[8];
};
__device__ __forceinline__ Vec32 load32_stream(const Vec32* p) {
  Vec32 v;
  asm volatile("ld.global.cs.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]),
                 "=r"(v.w[5]), "=r"(v.w[6]), "=r"(v.w[7])
               : "l"(p));
  return v;
}
__device__ __forceinline__ void store32(Vec32* p, const Vec32& v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v.w[0]),
               "r"(v.w[1]), "r"(v.w[2]), "r"(v.w[3]), "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]),
               "r"(v.w[7])
               : "memory");
}

// i / d and i % d; in 32 bits where i fits them (a 64-bit division costs more
// than the rest of an index).
__device__ __forceinline__ long long divide(long long i, int d, int& rest) {
  if (i >> 32 == 0) {
    const uint32_t q = static_cast<uint32_t>(i) / static_cast<uint32_t>(d);
    rest = static_cast<int>(static_cast<uint32_t>(i) - q * d);
    return q;
  }
  const long long q = i / d;
  rest = static_cast<int>(i - q * d);
  return q;
}

// Address of the scale byte of row r, 32-wide block b, in one of the layouts.
template <bool kGroupMajor>
__device__ __forceinline__ long long scale_at(long long r, int b, long long R, int blocks) {
  return kGroupMajor ? ((b >> 2) * R + r) * 4 + (b & 3) : r * blocks + b;
}

// What a thread reads of a unit, its largest magnitude (as fp32 bits: compared
// as integers, infinities and NaN rank above all others; 16-bit types two at a
// time) and its elements in fp32.
template <int kDtype>
struct Unit {
  static constexpr int kVecs = kDtype == MOE_T_FP32 ? 2 : 1;
  Vec32 v[kVecs];

  __device__ __forceinline__ uint32_t amax_bits() const {
    uint32_t top = 0;
    if constexpr (kDtype == MOE_T_FP32) {
#pragma unroll
      for (int c = 0; c < 16; ++c) top = max(top, v[c >> 3].w[c & 7] & 0x7FFFFFFFu);
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c) top = __vmaxu2(top, v[0].w[c] & 0x7FFF7FFFu);
      top = max(top >> 16, top & 0xFFFFu);
      if constexpr (kDtype == MOE_T_BF16)
        top <<= 16;
      else
        top = __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(top))));
    }
    return top;
  }
  // Elements 8h .. 8h + 7.
  __device__ __forceinline__ void get(int h, float (&f)[8]) const {
    if constexpr (kDtype == MOE_T_FP32) {
#pragma unroll
      for (int c = 0; c < 8; ++c) f[c] = __uint_as_float(v[h].w[c]);
    } else {
      Elem<kDtype>::unpack(
          make_uint4(v[0].w[4 * h], v[0].w[4 * h + 1], v[0].w[4 * h + 2], v[0].w[4 * h + 3]), f);
    }
  }
};

// One thread per 16 elements; eight consecutive threads share a 128-wide group
// of a row and write its four scale bytes as one word.  The threads of a row are
// rounded up to whole groups, so a group never straddles two rows.
template <int kDtype, bool kGroupMajor>
__global__ void __launch_bounds__(kThreads) quantize_mxfp4_kernel(
    const Vec32* __restrict__ x, const int32_t* __restrict__ inv, int T, int K, int k,
    uint2* __restrict__ codes, uint8_t* __restrict__ scales) {
  griddep_launch_dependents();
  griddep_wait();
  const int units = K / kUnit, blocks = K / 32;
  const long long R = static_cast<long long>(T) * k;
  const long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x;
  const int lane8 = threadIdx.x % kGroupUnits;
  int g;
  const long long t = divide(i / kGroupUnits, (K + 127) / 128, g);
  const int u = g * kGroupUnits + lane8;
  const bool live = t < T && u < units;
  Unit<kDtype> unit;
#pragma unroll
  for (int q = 0; q < Unit<kDtype>::kVecs; ++q)
    unit.v[q] = live ? load32_stream(x + (t * units + u) * Unit<kDtype>::kVecs + q) : Vec32{};
  uint32_t amax = unit.amax_bits();
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  const int byte = mx_scale_byte(amax);
  const float inv_scale = __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);   // 2^-n
  uint32_t out[2] = {0, 0};
  if (byte != 255) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float f[8];
      unit.get(h, f);
#pragma unroll
      for (int c = 0; c < 8; ++c) f[c] *= inv_scale;
      out[h] = cvt_e2m1x8(f);
    }
  }
  // The group's four bytes (0 for blocks past K).
  uint32_t word = live ? static_cast<uint32_t>(byte) << (8 * (lane8 >> 1)) : 0u;
  word |= __shfl_xor_sync(0xffffffffu, word, 2);
  word |= __shfl_xor_sync(0xffffffffu, word, 4);
  if (t >= T) return;
  auto write = [&](long long r) {
    if (r < 0 || r >= R) return;
    if (live) codes[r * units + u] = make_uint2(out[0], out[1]);
    if (kGroupMajor || blocks % 4 == 0) {
      if (lane8 == 0)
        *reinterpret_cast<uint32_t*>(scales + scale_at<kGroupMajor>(r, 4 * g, R, blocks)) = word;
    } else if (live && (lane8 & 1) == 0) {
      scales[scale_at<false>(r, u >> 1, R, blocks)] = static_cast<uint8_t>(byte);
    }
  };
  if (inv == nullptr) {
    write(t);
    return;
  }
  for (int j0 = 0; j0 < k; j0 += kSlotGroup) {
    int p[kSlotGroup];
#pragma unroll
    for (int j = 0; j < kSlotGroup; ++j) p[j] = j0 + j < k ? __ldg(&inv[t * k + j0 + j]) : -1;
#pragma unroll
    for (int j = 0; j < kSlotGroup; ++j) write(p[j]);
  }
}

// 16 codes a unit; a thread takes kPer units, `stride` apart, and loads them all
// before it uses any.
template <int kDtype, bool kGroupMajor, int kPer>
__global__ void __launch_bounds__(kThreads) dequantize_mxfp4_kernel(
    const uint2* __restrict__ codes, const uint8_t* __restrict__ scales, long long R, int K,
    long long stride, Vec32* __restrict__ out) {
  using E = Elem<kDtype>;
  constexpr int kVals = 32 / E::kBytes;   // values of a 32-byte store
  griddep_launch_dependents();
  griddep_wait();
  const int units = K / kUnit;
  const long long total = R * units;
  const long long first = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x;
  if (first >= stride) return;
  uint2 code[kPer];
  int byte[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const long long i = first + e * stride;
    code[e] = make_uint2(0, 0);
    byte[e] = 0;
    if (i < total) {
      int u;
      const long long r = divide(i, units, u);
      code[e] = __ldcs(codes + i);
      byte[e] = __ldg(scales + scale_at<kGroupMajor>(r, u >> 1, R, K / 32));
    }
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const long long i = first + e * stride;
    if (i >= total) return;
    // 2^(byte - 127): byte 0 is a subnormal, byte 255 NaN.
    const float scale =
        byte[e] == 255 ? __uint_as_float(0x7FC00000u)
                       : __uint_as_float(byte[e] == 0 ? 0x00400000u
                                                      : static_cast<uint32_t>(byte[e]) << 23);
    const uint32_t w[2] = {code[e].x, code[e].y};
#pragma unroll
    for (int q = 0; q < kUnit / kVals; ++q) {
      Vec32 o;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float f[E::kPerVec];
#pragma unroll
        for (int c = 0; c < E::kPerVec; ++c) {
          const int at = q * kVals + h * E::kPerVec + c;
          const uint32_t code4 = (w[at >> 3] >> (4 * (at & 7))) & 15u;
          // Exponent and mantissa bits read as an fp32 of exponent bias 127:
          // times 2^126 they have E2M1's bias 1, its subnormal 0.5 included.
          const float mag = __uint_as_float((code4 & 7u) << 22) * 8.507059173023462e37f;
          f[c] = __uint_as_float(__float_as_uint(mag) | (code4 & 8u) << 28) * scale;
        }
        const uint4 half = E::pack(f);
        o.w[4 * h] = half.x;
        o.w[4 * h + 1] = half.y;
        o.w[4 * h + 2] = half.z;
        o.w[4 * h + 3] = half.w;
      }
      store32(out + i * (kUnit / kVals) + q, o);
    }
  }
}

// Row-major codes w [E, N, K/2] -> 16 KB tiles of 128 rows x 128 bytes (256
// codes), tile (e, nb, kb) at ((e * NB + nb) * KB + kb) * 16 KB in the
// 128-byte-swizzled image the tensor core reads; rows past N and bytes past
// K/2 are zero.  One thread per 16-byte chunk of the tiles.
__global__ void __launch_bounds__(kThreads) prepack_mxfp4_kernel(const uint4* __restrict__ w,
                                                                 long long tiles, int N, int K,
                                                                 uint4* __restrict__ dst) {
  griddep_launch_dependents();
  griddep_wait();
  const int row_vecs = K / 32;
  const int KB = (K + 255) / 256, NB = (N + 127) / 128;
  const long long n = tiles * (kTileBytes / 16);
  for (long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; i < n;
       i += static_cast<long long>(gridDim.x) * kThreads) {
    const long long tile = i / (kTileBytes / 16);
    const int at = static_cast<int>(i % (kTileBytes / 16));
    const int r = at >> 3, c = at & 7;
    const long long block = tile / KB;
    const int kb = static_cast<int>(tile - block * KB);
    const long long e = block / NB;
    const int row = static_cast<int>(block - e * NB) * 128 + r;
    const int col = kb * 8 + c;
    const bool in = row < N && col < row_vecs;
    dst[tile * (kTileBytes / 16) + swz128(r, c) / 16] =
        in ? __ldg(w + (e * N + row) * row_vecs + col) : make_uint4(0, 0, 0, 0);
  }
}

// Row-major scales [E, N, K/32] -> two 512-byte chunks per tile, one per
// 128-wide half h of its 256 codes: row r's four bytes at
// tile * 1024 + h * 512 + (r % 32) * 16 + (r / 32) * 4, the layout the tensor
// core's scale copy reads; missing rows and blocks are byte 0 (a finite scale,
// on codes that are zero).  One thread per word.
__global__ void __launch_bounds__(kThreads) prepack_mxfp4_scales_kernel(
    const uint8_t* __restrict__ ws, long long tiles, int N, int K, uint32_t* __restrict__ dst) {
  griddep_launch_dependents();
  griddep_wait();
  const int blocks = K / 32;
  const int KB = (K + 255) / 256, NB = (N + 127) / 128;
  const long long n = tiles * 256;
  for (long long i = blockIdx.x * static_cast<long long>(kThreads) + threadIdx.x; i < n;
       i += static_cast<long long>(gridDim.x) * kThreads) {
    const long long tile = i / 256;
    const int at = static_cast<int>(i % 256);
    const int h = at >> 7, r = at & 127;
    const long long block = tile / KB;
    const int kb = static_cast<int>(tile - block * KB);
    const long long e = block / NB;
    const int row = static_cast<int>(block - e * NB) * 128 + r;
    uint32_t word = 0;
    if (row < N) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int b = (2 * kb + h) * 4 + j;
        if (b < blocks) word |= static_cast<uint32_t>(ws[(e * N + row) * blocks + b]) << (8 * j);
      }
    }
    dst[tile * 256 + h * 128 + (r & 31) * 4 + (r >> 5)] = word;
  }
}

bool layout_ok(int layout) {
  return layout == MOE_SCALES_ROW_MAJOR || layout == MOE_SCALES_GROUP_MAJOR;
}

long long scale_bytes(long long R, int K, int layout) {
  return layout == MOE_SCALES_GROUP_MAJOR ? (K + 127) / 128 * R * 4 : R * (K / 32);
}

// Blocks of kThreads for n threads; 0 if the grid would exceed its limit.
unsigned blocks_of(long long n) {
  const long long b = (n + kThreads - 1) / kThreads;
  return b < (1ll << 31) ? static_cast<unsigned>(b) : 0u;
}

template <int kDtype>
cudaError_t launch_quantize(bool group_major, unsigned blocks, cudaStream_t st, const void* x,
                            const int32_t* inv, int T, int K, int k, uint8_t* codes,
                            uint8_t* scales) {
  auto kern = group_major ? quantize_mxfp4_kernel<kDtype, true>
                          : quantize_mxfp4_kernel<kDtype, false>;
  return launch_pdl(kern, dim3(blocks), dim3(kThreads), 0, st, static_cast<const Vec32*>(x), inv,
                    T, K, k, reinterpret_cast<uint2*>(codes), scales);
}

template <int kDtype, int kPer>
cudaError_t launch_dequantize_per(bool group_major, cudaStream_t st, const uint8_t* codes,
                                  const uint8_t* scales, int R, int K, void* out) {
  const long long total = static_cast<long long>(R) * (K / kUnit);
  const long long stride = (total + kPer - 1) / kPer;
  const unsigned blocks = blocks_of(stride);
  if (blocks == 0) return cudaErrorInvalidConfiguration;
  auto kern = group_major ? dequantize_mxfp4_kernel<kDtype, true, kPer>
                          : dequantize_mxfp4_kernel<kDtype, false, kPer>;
  return launch_pdl(kern, dim3(blocks), dim3(kThreads), 0, st,
                    reinterpret_cast<const uint2*>(codes), scales, static_cast<long long>(R), K,
                    stride, static_cast<Vec32*>(out));
}

template <int kDtype>
cudaError_t launch_dequantize(bool group_major, cudaStream_t st, const uint8_t* codes,
                              const uint8_t* scales, int R, int K, void* out) {
  // Two units a thread once that leaves every SM full of threads (65536 x 7168 to
  // bf16: 180 us against 204 with one; 333 x 1568: 2.1 against 1.8).
  const long long total = static_cast<long long>(R) * (K / kUnit);
  return total >= 2ll * 2048 * sm_count()
             ? launch_dequantize_per<kDtype, 2>(group_major, st, codes, scales, R, K, out)
             : launch_dequantize_per<kDtype, 1>(group_major, st, codes, scales, R, K, out);
}

// Tiles of prepacked weights, or 0 for sizes the product does not take.
long long weight_tiles(int E, int N, int K) {
  if (!mx_gemm_sizes_ok(E, N, K)) return 0;
  return static_cast<long long>(E) * ((N + 127ll) / 128) * ((K + 255ll) / 256);
}

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_quantize_mxfp4(const void* x, int dtype, int T, int K, int k, const int32_t* inv,
                              uint8_t* codes, uint8_t* scales, int scale_layout,
                              moe_stream_t stream) {
  if (x == nullptr || codes == nullptr || scales == nullptr) return MOE_ERR_INVALID_ARG;
  if (!moe::elem_ok(dtype) || !moe::layout_ok(scale_layout)) return MOE_ERR_INVALID_ARG;
  if (T < 1 || K < 1 || k < 1 || static_cast<long long>(T) * k >= (1ll << 31))
    return MOE_ERR_INVALID_ARG;
  if (inv == nullptr && k != 1) return MOE_ERR_INVALID_ARG;
  if (K % 32 != 0 || K > moe::kMaxRow || k > moe::kMaxSlotsPerToken) return MOE_ERR_UNSUPPORTED;
  if (!moe::aligned_to(x, 32) || !moe::aligned_to(codes, 16) || !moe::aligned_to(scales, 4) ||
      !moe::aligned_to(inv, 4))
    return MOE_ERR_ALIGNMENT;
  const long long R = static_cast<long long>(T) * k;
  const long long xb = static_cast<long long>(T) * K * moe::elem_bytes(dtype), cb = R * (K / 2);
  const long long sb = moe::scale_bytes(R, K, scale_layout);
  const moe::Buffer buffers[] = {
      {x, xb, false}, {inv, R * 4, false}, {codes, cb, true}, {scales, sb, true}};
  if (moe::outputs_overlap(buffers)) return MOE_ERR_INVALID_ARG;
  const unsigned blocks = moe::blocks_of(T * ((K + 127ll) / 128) * moe::kGroupUnits);
  if (blocks == 0) return MOE_ERR_UNSUPPORTED;
  auto launch = dtype == MOE_T_BF16   ? moe::launch_quantize<MOE_T_BF16>
                : dtype == MOE_T_FP16 ? moe::launch_quantize<MOE_T_FP16>
                                      : moe::launch_quantize<MOE_T_FP32>;
  const cudaError_t e = launch(scale_layout == MOE_SCALES_GROUP_MAJOR, blocks,
                               reinterpret_cast<cudaStream_t>(stream), x, inv, T, K, k, codes,
                               scales);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_dequantize_mxfp4(const uint8_t* codes, const uint8_t* scales, int scale_layout,
                                int R, int K, int dtype, void* out, moe_stream_t stream) {
  if (codes == nullptr || scales == nullptr || out == nullptr) return MOE_ERR_INVALID_ARG;
  if (!moe::elem_ok(dtype) || !moe::layout_ok(scale_layout) || R < 1 || K < 1)
    return MOE_ERR_INVALID_ARG;
  if (K % 32 != 0 || K > moe::kMaxRow) return MOE_ERR_UNSUPPORTED;
  if (!moe::aligned_to(codes, 16) || !moe::aligned_to(out, 32)) return MOE_ERR_ALIGNMENT;
  const long long n = R * static_cast<long long>(K);
  const moe::Buffer buffers[] = {{codes, n / 2, false},
                                 {scales, moe::scale_bytes(R, K, scale_layout), false},
                                 {out, n * moe::elem_bytes(dtype), true}};
  if (moe::outputs_overlap(buffers)) return MOE_ERR_INVALID_ARG;
  if (n / moe::kUnit > (1ll << 38)) return MOE_ERR_UNSUPPORTED;   // the grid's limit
  auto launch = dtype == MOE_T_BF16   ? moe::launch_dequantize<MOE_T_BF16>
                : dtype == MOE_T_FP16 ? moe::launch_dequantize<MOE_T_FP16>
                                      : moe::launch_dequantize<MOE_T_FP32>;
  const cudaError_t e = launch(scale_layout == MOE_SCALES_GROUP_MAJOR,
                               reinterpret_cast<cudaStream_t>(stream), codes, scales, R, K, out);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_mxfp4_weight_bytes(int E, int N, int K) {
  return static_cast<size_t>(moe::weight_tiles(E, N, K)) * moe::kTileBytes;
}

size_t moe_mxfp4_weight_scale_bytes(int E, int N, int K) {
  return static_cast<size_t>(moe::weight_tiles(E, N, K)) * 1024;
}

moe_status moe_mxfp4_prepack(const uint8_t* w, const uint8_t* w_scales, int E, int N, int K,
                             uint8_t* w_tiled, uint8_t* w_scales_chunked, moe_stream_t stream) {
  if (w == nullptr || w_scales == nullptr || w_tiled == nullptr || w_scales_chunked == nullptr)
    return MOE_ERR_INVALID_ARG;
  if (E < 1 || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
  const long long tiles = moe::weight_tiles(E, N, K);
  if (tiles == 0) return MOE_ERR_UNSUPPORTED;
  if (!moe::aligned_to(w, 16) || !moe::aligned_to(w_tiled, 16) ||
      !moe::aligned_to(w_scales_chunked, 16))
    return MOE_ERR_ALIGNMENT;
  const long long rows = static_cast<long long>(E) * N;
  const moe::Buffer buffers[] = {{w, rows * (K / 2), false},
                                 {w_scales, rows * (K / 32), false},
                                 {w_tiled, tiles * static_cast<long long>(moe::kTileBytes), true},
                                 {w_scales_chunked, tiles * 1024, true}};
  if (moe::outputs_overlap(buffers)) return MOE_ERR_INVALID_ARG;
  auto st = reinterpret_cast<cudaStream_t>(stream);
  const unsigned most = static_cast<unsigned>(moe::sm_count()) * 16;
  const long long cb = tiles * static_cast<long long>(moe::kTileBytes / 16) / moe::kThreads;
  const unsigned code_blocks = cb < most ? static_cast<unsigned>(cb) : most;
  const unsigned scale_blocks = tiles < most ? static_cast<unsigned>(tiles) : most;
  cudaError_t e = moe::launch_pdl(moe::prepack_mxfp4_kernel, dim3(code_blocks),
                                  dim3(moe::kThreads), 0, st, reinterpret_cast<const uint4*>(w),
                                  tiles, N, K, reinterpret_cast<uint4*>(w_tiled));
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  e = moe::launch_pdl(moe::prepack_mxfp4_scales_kernel, dim3(scale_blocks), dim3(moe::kThreads), 0,
                      st, w_scales, tiles, N, K, reinterpret_cast<uint32_t*>(w_scales_chunked));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"

// int8 encoding and decoding on gfx950 (page "deepseek-v4-mxfp4-int8
// config.json", quantization_config, linears_w8a16: int8, symmetric, one scale
// per output channel; here one scale per row, a weight's channel or an
// activation's token): per row with largest magnitude m,
//   s = m / 127 (fp32, rounded once; 1 if m = 0; at least 2^-126),
//   code = v / s rounded to the nearest whole number, ties to even.
// A row with an Inf or NaN gets the scale NaN and codes 0, and reads as NaN.
//
// The code is that of the exact quotient: a product with 1 / s lies within a few
// units in its last place, so it can only miss a code next to a border, and the
// remainder v - c s, exact in one fma (|v - c s| <= s and both are multiples of
// the smaller one's last place), says on which side v lies.
//
// Memory-bound both ways: a row is read once and held in registers between its
// maximum and its codes. Measured (a large copy: 5.0 to 5.1 TB/s): 16384 x 4096 fp32
// 61 us to encode and 61 to decode again and again (part of it from the
// last-level cache; on inputs in turn 82, 4.1 TB/s, and 54), bf16 37 and 38; 8192
// x 4096 bf16 18 to 20; 33 x 8192 bf16 3.5, 64 x 4096 2.9 (launch and one round of
// load latency).
#include <type_traits>

#include "device.h"
#include "internal.h"

namespace moe {

namespace {

template <int DT>
constexpr int kPer = DT == kDtF32 ? 4 : 8;  // values of a 16-byte piece

template <int DT>
__device__ __forceinline__ float value_of(const u32x4_t& p, int i) {
  if constexpr (DT == kDtF32) return __uint_as_float(p[i]);
  const uint32_t h = i & 1 ? p[i >> 1] >> 16 : p[i >> 1] & 0xffffu;
  return DT == kDtBf16 ? __uint_as_float(h << 16) : f16_bits_to_f32(h);
}

// Largest magnitude as bits: magnitudes compare as integers, Inf and NaN above every finite value.
template <int DT>
__device__ __forceinline__ uint32_t piece_top(const u32x4_t& p, uint32_t m) {
#pragma unroll
  for (int i = 0; i < kPer<DT>; ++i) m = max(m, __float_as_uint(value_of<DT>(p, i)) & 0x7fffffffu);
  return m;
}

// The codes of a piece: 8 bytes (16-bit values) or 4.
template <int DT>
__device__ __forceinline__ uint2 piece_codes(const u32x4_t& p, const RowScale& s) {
  uint2 o = make_uint2(0u, 0u);
  f32x4_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = value_of<DT>(p, i);
  o.x = int8_codes4(v, s);
  if constexpr (kPer<DT> == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = value_of<DT>(p, 4 + i);
    o.y = int8_codes4(v, s);
  }
  return o;
}

template <int DT>
__device__ __forceinline__ void put_codes(int8_t* row, int piece, const uint2& c) {
  if constexpr (DT == kDtF32) *reinterpret_cast<uint32_t*>(row + 4 * piece) = c.x;
  else *reinterpret_cast<uint2*>(row + 8 * piece) = c;
}

// TPR threads per row (8 to 64: a part of a wave; 256, 1024: whole waves), PER pieces per thread.
template <int DT, int TPR, int PER>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void k_int8_quantize(long long rows, int K, const char* __restrict__ x,
                                                       long long ld_bytes, int8_t* __restrict__ codes,
                                                       float* __restrict__ scales) {
  constexpr int BLOCK = TPR > 256 ? TPR : 256, WPR = TPR / 64;
  const int lane = (int)threadIdx.x % TPR, sub = (int)threadIdx.x / TPR;
  const long long row = (long long)blockIdx.x * (BLOCK / TPR) + sub;
  const bool live = row < rows;
  const int P = live ? K / kPer<DT> : 0;
  const u32x4_t* src = reinterpret_cast<const u32x4_t*>(x + (live ? row : 0) * ld_bytes);
  u32x4_t v[PER];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) v[i] = lane + i * TPR < P ? src[lane + i * TPR] : (u32x4_t){0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < PER; ++i) top = piece_top<DT>(v[i], top);
#pragma unroll
  for (int o = (TPR < 64 ? TPR : 64) / 2; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
  if constexpr (WPR > 1) {
    __shared__ uint32_t tops[WPR];
    if (threadIdx.x % 64 == 0) tops[threadIdx.x / 64] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WPR; ++i) top = max(top, tops[i]);
  }
  if (!live) return;
  const RowScale s = row_scale(top);
  int8_t* out = codes + row * K;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (lane + i * TPR < P) put_codes<DT>(out, lane + i * TPR, piece_codes<DT>(v[i], s));
  if (lane == 0) scales[row] = s.scale;
}

constexpr long long kMaxThreads = 1ll << 31;  // of a launch (the runtime takes fewer than 2^32); more rows, more launches

template <int DT>
hipError_t quantize(long long rows, int K, const char* x, long long ld, int8_t* codes, float* scales, hipStream_t st) {
  const int P = K / kPer<DT>;
  auto go = [&](auto tpr, auto per) {
    constexpr int threads = tpr > 256 ? tpr : 256, rpb = threads / tpr;
    constexpr long long most = kMaxThreads / tpr;
    for (long long r = 0; r < rows; r += most) {
      const long long n = rows - r < most ? rows - r : most;
      k_int8_quantize<DT, tpr, per><<<(unsigned)((n + rpb - 1) / rpb), threads, 0, st>>>(n, K, x + r * ld, ld, codes + r * K,
                                                                                        scales + r);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  };
#define ROW(tpr, per) go(std::integral_constant<int, tpr>{}, std::integral_constant<int, per>{})
  // Few rows: latency counts, and a row's pieces are spread over 1024 threads (33 x 8192 bf16 5.3 -> 3.4 us); rows past
  // 2048 pieces take as many anyway.
  if ((rows <= 512 && P > 256) || P > 2048) {
    if (P <= 1024) return ROW(1024, 1);
    if (P <= 2048) return ROW(1024, 2);
    if (P <= 4096) return ROW(1024, 4);
    if (P <= 8192) return ROW(1024, 8);
    return ROW(1024, 16);  // fp32, K up to 65536
  }
  // as many lanes as a short row has pieces, a wave while they hold two each, then a block per row
  if (P <= 8) return ROW(8, 1);
  if (P <= 16) return ROW(16, 1);
  if (P <= 32) return ROW(32, 1);
  if (P <= 64) return ROW(64, 1);
  if (P <= 128) return ROW(64, 2);
  if (P <= 256) return ROW(256, 1);
  if (P <= 512) return ROW(256, 2);
  if (P <= 1024) return ROW(256, 4);
  return ROW(256, 8);
#undef ROW
}

// A thread takes pieces of 16 output bytes. Rows of fewer than 256 pieces share a block (RPB rows), longer ones are cut
// into segments of 256 * AHEAD pieces.
constexpr int kDeqAhead = 4;

template <bool F32>
__global__ __launch_bounds__(256) void k_int8_dequantize(long long rows, int K, int rpb, int segs,
                                                         const int8_t* __restrict__ codes,
                                                         const float* __restrict__ scales, void* __restrict__ out) {
  constexpr int V = F32 ? 4 : 8;
  const int P = K / V;
  long long row;
  int first, step;
  if (rpb > 1) {
    const int sub = (int)threadIdx.x / P;
    row = (long long)blockIdx.x * rpb + sub;
    if (sub >= rpb || row >= rows) return;
    first = (int)threadIdx.x - sub * P;
    step = P;  // one piece each
  } else {
    row = blockIdx.x / (unsigned)segs;
    first = (int)(blockIdx.x - (unsigned)row * (unsigned)segs) * 256 * kDeqAhead + (int)threadIdx.x;
    step = 256;
  }
  const float s = scales[row];
  const int8_t* c = codes + row * K;
  uint2 q[kDeqAhead];
#pragma unroll
  for (int i = 0; i < kDeqAhead; ++i) {
    const int p = first + i * step;
    q[i] = make_uint2(0u, 0u);
    if (p >= P) continue;
    if constexpr (F32) q[i].x = *reinterpret_cast<const uint32_t*>(c + 4 * p);
    else q[i] = *reinterpret_cast<const uint2*>(c + 8 * p);
  }
#pragma unroll
  for (int i = 0; i < kDeqAhead; ++i) {
    const int p = first + i * step;
    if (p >= P) continue;
    float f[V];
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = (float)(int8_t)((j < 4 ? q[i].x : q[i].y) >> (8 * (j & 3))) * s;
    u32x4_t o;
    if constexpr (F32) {
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = __float_as_uint(f[j]);
      reinterpret_cast<u32x4_t*>(static_cast<float*>(out) + row * K)[p] = o;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = bf16x2_rne(f[2 * j], f[2 * j + 1]);
      reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(out) + row * K)[p] = o;
    }
  }
}

}  // namespace

hipError_t launch_int8_quantize(long long rows, int K, int dtype, const void* x, long long ldx, int8_t* codes,
                                float* scales, hipStream_t st) {
  if (rows <= 0 || K <= 0 || K % 16 || rows > (1ll << 32)) return hipErrorInvalidValue;
  const char* p = static_cast<const char*>(x);
  if (dtype == kDtF32) return quantize<kDtF32>(rows, K, p, ldx * 4, codes, scales, st);
  if (dtype == kDtBf16) return quantize<kDtBf16>(rows, K, p, ldx * 2, codes, scales, st);
  return quantize<kDtF16>(rows, K, p, ldx * 2, codes, scales, st);
}

hipError_t launch_int8_dequantize(long long rows, int K, const int8_t* codes, const float* scales, int dtype, void* out,
                                  hipStream_t st) {
  if (rows <= 0 || K <= 0 || K % 16 || rows > (1ll << 32)) return hipErrorInvalidValue;
  const int P = K / (dtype == kDtF32 ? 4 : 8);
  const int rpb = P <= 128 ? 256 / P : 1;
  const int segs = rpb > 1 ? 1 : (P + 256 * kDeqAhead - 1) / (256 * kDeqAhead);
  const long long most = kMaxThreads / 256 / segs * rpb;
  for (long long r = 0; r < rows; r += most) {
    const long long n = rows - r < most ? rows - r : most;
    const unsigned nb = (unsigned)((n + rpb - 1) / rpb * segs);
    if (dtype == kDtF32)
      k_int8_dequantize<true><<<nb, 256, 0, st>>>(n, K, rpb, segs, codes + r * K, scales + r, static_cast<float*>(out) + r * K);
    else
      k_int8_dequantize<false><<<nb, 256, 0, st>>>(n, K, rpb, segs, codes + r * K, scales + r,
                                                   static_cast<uint16_t*>(out) + r * K);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe

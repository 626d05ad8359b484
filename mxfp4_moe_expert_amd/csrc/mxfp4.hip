// MXFP4 encoding and decoding on gfx950 (page "deepseek-v4-mxfp4-int8
// config.json", quantization_config, experts_w4a16; OCP Microscaling Formats
// v1.0): per 32 consecutive values along K with largest magnitude m,
//   X = max(floor(log2 m) - 2, -127), exponent byte X + 127,
//   code = E2M1 value nearest to v / 2^X, ties to the even code, at most 6.
// floor(log2 m) is the exponent field of m as fp32 (a subnormal m has field 0
// and ends at X = -127 like every m below 2^-125), and v / 2^X is exact inside
// the hardware's scaled conversion, so no rounding happens but the one to
// E2M1. A group with an Inf or NaN gets the byte 255 (NaN), and reads back as
// NaN; its codes are 0.
//
// Memory-bound in both directions. A lane takes 16 bytes per load (8 values of
// 16 bits or 4 of 32), consecutive lanes consecutive bytes, so 4 or 8 lanes
// share a group and its maximum is two or three lane exchanges. Measured,
// 16384 x 4096 fp32: encoding 75 us (4.0 TB/s), decoding 56 to 58 us (5.2);
// 4096 x 4096 weights to bf16 8.4 us (5.0); the operands of the 4-bit product
// with 8192 x 4096 activations 16.5 to 17.4 us (4.9). A large copy: 5.1 TB/s.
#include "device.h"
#include "internal.h"

namespace moe {

typedef __attribute__((ext_vector_type(8))) float f32x8_t;

// Eight 16-bit values as fp32.
template <int DT>
__device__ __forceinline__ f32x8_t widen8(const u32x4_t& a) {
  f32x8_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == kDtBf16) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    } else {
      v[2 * i] = f16_bits_to_f32(a[i] & 0xffffu);
      v[2 * i + 1] = f16_bits_to_f32(a[i] >> 16);
    }
  }
  return v;
}

// Largest magnitude of a lane's values as bits: magnitudes compare as integers, Inf and NaN above every finite value.
template <class V, int N>
__device__ __forceinline__ uint32_t top_bits(const V& v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}
template <int CTRL>
__device__ __forceinline__ uint32_t lane_max(uint32_t m) {
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  return lane_max<0x4E>(lane_max<0xB1>(m));  // quad_perm [1,0,3,2], then [2,3,0,1]
}
// The exponent byte of a group with largest magnitude m (bits): 255 if it is not finite. scale: for the conversion.
__device__ __forceinline__ uint32_t group_byte(uint32_t m, float& scale) {
  const uint32_t field = m >> 23, e = field > 2u ? field - 2u : 0u;
  scale = e8m0_scale_operand(e);
  return field == 255u ? 255u : e;
}

// The quad's four lanes hold one group, eight values each -> the lane's codes
// (one dword) and the group's exponent byte.
__device__ __forceinline__ uint32_t quad_encode(const f32x8_t& v, uint32_t& byte) {
  float sc;
  byte = group_byte(quad_max(top_bits<f32x8_t, 8>(v)), sc);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], sc, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], sc, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], sc, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], sc, 3);
  return byte == 255u ? 0u : c;
}
// Eight lanes hold one group, four values each -> the lane's codes (16 bits) and the exponent byte.
__device__ __forceinline__ uint32_t oct_encode(const f32x4_t& v, uint32_t& byte) {
  float sc;
  byte = group_byte(lane_max<0x141>(quad_max(top_bits<f32x4_t, 4>(v))), sc);  // row_half_mirror: the other quad of 8
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], sc, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], sc, 1);
  return byte == 255u ? 0u : c;
}

// Units of 16 bytes of x; a thread takes kQuantUnits of them, 256 apart, and
// has all their loads in flight together.
constexpr int kQuantUnits = 8;
constexpr long long kMaxBlocks = 0xffffff;  // of 256 threads: a grid holds fewer than 2^32 threads

template <int DT>
__global__ __launch_bounds__(256) void k_mxfp4_quantize(const void* x, long long units, int upr, long long ldx,
                                                        uint8_t* codes, uint8_t* scales) {
  constexpr int V = DT == kDtF32 ? 4 : 8, LPG = kMxGroup / V;  // values per unit, lanes per group
  const long long u0 = (long long)blockIdx.x * (256 * kQuantUnits) + threadIdx.x;
  u32x4_t v[kQuantUnits];
#pragma unroll
  for (int i = 0; i < kQuantUnits; ++i) {
    const long long u = min(u0 + i * 256, units - 1);
    size_t at = (size_t)u * V;
    if (ldx != (long long)upr * V) {
      const long long row = u / upr;
      at = (size_t)row * ldx + (size_t)(u - row * upr) * V;
    }
    v[i] = *reinterpret_cast<const u32x4_t*>(static_cast<const uint8_t*>(x) + at * (16 / V));
  }
#pragma unroll
  for (int i = 0; i < kQuantUnits; ++i) {
    const long long u = u0 + i * 256;
    if (u >= units) continue;  // units are whole groups: a group's lanes are live or not as one
    uint32_t byte;
    if constexpr (DT == kDtF32) {
      const uint32_t c = oct_encode(__builtin_bit_cast(f32x4_t, v[i]), byte);
      reinterpret_cast<uint16_t*>(codes)[u] = (uint16_t)c;
    } else {
      reinterpret_cast<uint32_t*>(codes)[u] = quad_encode(widen8<DT>(v[i]), byte);
    }
    if ((u & (LPG - 1)) == 0) scales[u / LPG] = (uint8_t)byte;
  }
}

hipError_t launch_mxfp4_quantize(long long rows, int K, int dtype, const void* x, long long ldx, uint8_t* codes,
                                 uint8_t* scales, hipStream_t st) {
  const int upr = K / (dtype == kDtF32 ? 4 : 8);
  const long long units = rows * upr;
  if (K % kMxGroup || ldx < K) return hipErrorInvalidValue;
  if (units <= 0) return hipSuccess;
  const long long nb = (units + 256 * kQuantUnits - 1) / (256 * kQuantUnits);
  if (nb > kMaxBlocks) return hipErrorInvalidValue;
  if (dtype == kDtBf16) k_mxfp4_quantize<kDtBf16><<<(unsigned)nb, 256, 0, st>>>(x, units, upr, ldx, codes, scales);
  else if (dtype == kDtF32) k_mxfp4_quantize<kDtF32><<<(unsigned)nb, 256, 0, st>>>(x, units, upr, ldx, codes, scales);
  else if (dtype == kDtF16) k_mxfp4_quantize<kDtF16><<<(unsigned)nb, 256, 0, st>>>(x, units, upr, ldx, codes, scales);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

constexpr int kDecodeUnits = 4;

// Decoding: a unit is 8 codes (one dword) and its group's byte. Byte 255
// makes the hardware conversion return NaN.
template <int DT>
__device__ __forceinline__ void decode_unit(uint32_t c, uint32_t byte, void* out, size_t at) {
  const float sc = e8m0_scale_operand(byte);
  const bf16x8_t v = fp4x8_to_bf16x8(c, sc);
  if constexpr (DT == kDtBf16) {
    *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(out) + at) = __builtin_bit_cast(u32x4_t, v);
  } else {
    const u32x4_t b = __builtin_bit_cast(u32x4_t, v);
    f32x4_t lo, hi;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      lo[2 * i] = __uint_as_float(b[i] << 16);
      lo[2 * i + 1] = __uint_as_float(b[i] & 0xffff0000u);
      hi[2 * i] = __uint_as_float(b[2 + i] << 16);
      hi[2 * i + 1] = __uint_as_float(b[2 + i] & 0xffff0000u);
    }
    f32x4_t* o = reinterpret_cast<f32x4_t*>(static_cast<float*>(out) + at);
    o[0] = lo;
    o[1] = hi;
  }
}

template <int DT>
__global__ __launch_bounds__(256) void k_mxfp4_dequantize(const uint32_t* codes, const uint8_t* scales,
                                                          long long units, void* out) {
  const long long u0 = (long long)blockIdx.x * (256 * kDecodeUnits) + threadIdx.x;
  uint32_t c[kDecodeUnits], b[kDecodeUnits];
#pragma unroll
  for (int i = 0; i < kDecodeUnits; ++i) {
    const long long u = min(u0 + i * 256, units - 1);
    c[i] = codes[u];
    b[i] = scales[u >> 2];
  }
#pragma unroll
  for (int i = 0; i < kDecodeUnits; ++i) {
    const long long u = u0 + i * 256;
    if (u < units) decode_unit<DT>(c[i], b[i], out, (size_t)u * 8);
  }
}

hipError_t launch_mxfp4_dequantize(long long rows, int K, const uint8_t* codes, const uint8_t* scales, int dtype,
                                   void* out, hipStream_t st) {
  const long long units = rows * (K / 8);
  if (K % kMxGroup) return hipErrorInvalidValue;
  if (units <= 0) return hipSuccess;
  const long long nb = (units + 256 * kDecodeUnits - 1) / (256 * kDecodeUnits);
  if (nb > kMaxBlocks) return hipErrorInvalidValue;
  const uint32_t* c = reinterpret_cast<const uint32_t*>(codes);
  if (dtype == kDtBf16) k_mxfp4_dequantize<kDtBf16><<<(unsigned)nb, 256, 0, st>>>(c, scales, units, out);
  else if (dtype == kDtF32) k_mxfp4_dequantize<kDtF32><<<(unsigned)nb, 256, 0, st>>>(c, scales, units, out);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

// ---- operands of the 4-bit x 4-bit product
//
// Packed scales: the product's k-step j (128 values) of two stages p (512
// values) takes, in lane (r, g), the exponent byte of row 16 b + r, group
// 16 p + 4 j + g. Packed as u32 [p][b][16 g + r], byte j: the scales of
// consecutive row blocks are contiguous and lane-ordered. Groups past K get
// the byte 0 (their codes are zeros, and 2^-127 keeps the products zero).
//
// Blocks [0, xblocks): x [T][K] bf16 to codes and packed scales, a block per
// 16 rows and 512 values, each wave a row at a time (1 KB per load): the
// block's 256 scale bytes meet in LDS and are stored as one piece (stored byte
// by byte, the rows' blocks on several XCDs shared their lines). Blocks from
// xblocks on: the weights' exponent bytes to the packed order, a dword per
// thread in its place's order.
__global__ __launch_bounds__(256) void k_mxfp4_prep(int T, int K, const uint16_t* x, uint32_t* xcodes, uint32_t* xpack,
                                                    unsigned xblocks, int N, const uint8_t* wscales, uint32_t* wpack) {
  const int pairs = mxfp4_pairs(K);
  if (blockIdx.x < xblocks) {
    __shared__ __align__(16) uint8_t pack[256];
    const int tb = (T + 15) / 16, p = (int)(blockIdx.x / tb), b = (int)(blockIdx.x - (unsigned)p * tb);
    const int unit = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = p * 64 + unit;  // K % 32 == 0: a quad is in or out as one
    u32x4_t v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = 16 * b + 4 * j + wave;
      v[j] = (u32x4_t){0u, 0u, 0u, 0u};
      if (row < T && col * 8 < K) v[j] = *reinterpret_cast<const u32x4_t*>(x + (size_t)row * K + (size_t)col * 8);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 4 * j + wave, row = 16 * b + r, group = unit >> 2;
      uint32_t byte;
      const uint32_t c = quad_encode(widen8<kDtBf16>(v[j]), byte);
      if (row < T && col * 8 < K) xcodes[(size_t)row * (K / 8) + col] = c;
      if ((unit & 3) == 0) pack[((group & 3) * 16 + r) * 4 + (group >> 2)] = col * 8 < K ? (uint8_t)byte : (uint8_t)0;
    }
    __syncthreads();
    if (threadIdx.x < 64) xpack[((size_t)p * tb + b) * 64 + threadIdx.x] = reinterpret_cast<const uint32_t*>(pack)[threadIdx.x];
  } else {
    const int nb = (N + 15) / 16;
    const long long u = (long long)(blockIdx.x - xblocks) * 256 + threadIdx.x;
    const long long blk = u >> 6;  // p * nb + b
    const int p = (int)(blk / nb), row = (int)(blk - (long long)p * nb) * 16 + ((int)u & 15), g = ((int)u >> 4) & 3;
    if (p >= pairs || row >= N) return;
    const int G = K / kMxGroup, g0 = p * 16 + g;
    uint32_t d = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (g0 + 4 * j < G) d |= (uint32_t)wscales[(size_t)row * G + g0 + 4 * j] << (8 * j);
    wpack[u] = d;
  }
}

hipError_t launch_mxfp4_prep(int T, int K, const uint16_t* x, uint8_t* xcodes, uint32_t* xpack, int N,
                             const uint8_t* wscales, uint32_t* wpack, hipStream_t st) {
  if (K % kMxGroup || T <= 0 || N <= 0) return hipErrorInvalidValue;
  const long long pairs = mxfp4_pairs(K);
  const long long xb = pairs * mxfp4_blocks(T), wb = (pairs * mxfp4_blocks(N) * 64 + 255) / 256;
  if (xb + wb > kMaxBlocks) return hipErrorInvalidValue;
  k_mxfp4_prep<<<(unsigned)(xb + wb), 256, 0, st>>>(T, K, x, reinterpret_cast<uint32_t*>(xcodes), xpack, (unsigned)xb, N,
                                                    wscales, wpack);
  return hipGetLastError();
}

// Weights to bf16 [N][K] for the bf16 product of many rows, and (blocks from
// wblocks on) dy [T][N] to rows of ld values, zero-padded, where N is not a
// multiple of 8 (the product reads 16-byte pieces of each row).
__global__ __launch_bounds__(256) void k_mxfp4_expand(const uint32_t* codes, const uint8_t* scales, long long units,
                                                      uint16_t* w, unsigned wblocks, int T, int N, const uint16_t* dy,
                                                      uint16_t* dyp, int ld) {
  if (blockIdx.x < wblocks) {
    const long long u0 = (long long)blockIdx.x * (256 * kDecodeUnits) + threadIdx.x;
    uint32_t c[kDecodeUnits], b[kDecodeUnits];
#pragma unroll
    for (int i = 0; i < kDecodeUnits; ++i) {
      const long long u = min(u0 + i * 256, units - 1);
      c[i] = codes[u];
      b[i] = scales[u >> 2];
    }
#pragma unroll
    for (int i = 0; i < kDecodeUnits; ++i) {
      const long long u = u0 + i * 256;
      if (u < units) decode_unit<kDtBf16>(c[i], b[i], w, (size_t)u * 8);
    }
  } else {
    const long long i = (long long)(blockIdx.x - wblocks) * 256 + threadIdx.x;  // 8 values of a padded row
    const long long row = i / (ld / 8);
    const int col = (int)(i - row * (ld / 8)) * 8;
    if (row >= T) return;
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = col + j < N ? dy[row * N + col + j] : 0u;
    *reinterpret_cast<u32x4_t*>(dyp + i * 8) =
        (u32x4_t){v[0] | (v[1] << 16), v[2] | (v[3] << 16), v[4] | (v[5] << 16), v[6] | (v[7] << 16)};
  }
}

hipError_t launch_mxfp4_expand(int N, int K, const uint8_t* codes, const uint8_t* scales, uint16_t* w, int T,
                               const uint16_t* dy, uint16_t* dyp, int ld, hipStream_t st) {
  if (K % kMxGroup || N <= 0) return hipErrorInvalidValue;
  const long long units = (long long)N * (K / 8);
  const long long wb = (units + 256 * kDecodeUnits - 1) / (256 * kDecodeUnits);
  const long long db = dy ? ((long long)T * (ld / 8) + 255) / 256 : 0;
  if (ld % 8 || wb + db > kMaxBlocks) return hipErrorInvalidValue;
  k_mxfp4_expand<<<(unsigned)(wb + db), 256, 0, st>>>(reinterpret_cast<const uint32_t*>(codes), scales, units, w,
                                                      (unsigned)wb, T, N, dy, dyp, ld);
  return hipGetLastError();
}

}  // namespace moe

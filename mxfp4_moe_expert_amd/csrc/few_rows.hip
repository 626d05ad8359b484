// Products of at most 32 rows with a weight matrix that is streamed once:
// MXFP4 weights (moe_linear_mxfp4) and bf16 weights (the gated block).
//
// A block owns 16 weight rows (gate: 8 gate rows and the matching 8 up rows)
// and its NW waves split K, wave w taking k-steps w, w + NW, ...: a block
// reads NW consecutive pieces of each row at a time, all its loads in flight
// at once for the usual K, and needs neither LDS staging (no wave shares
// activations with another) nor a second launch: the waves' fp32 sums meet
// in LDS and are added in wave order, so results do not depend on timing.
//   MXFP4: a k-step is 128 values; lane (r, g) reads 16 bytes, exactly group
//     g of row r. Activations in bf16: the codes are converted to bf16 (exact)
//     for four MFMA 16x16x32. Activations rounded to MXFP4: lane (t, g) holds
//     exactly one group of token t, encodes it, and the codes of both sides
//     go to one scaled MFMA 16x16x128.
//   bf16: a k-step is 64 values; lane (r, g) reads 32 bytes of row r. The gated
//     block's h enters its second product as two bf16 values, the nearest and
//     the nearest to what that leaves (16 bits together): the weights bound the
//     pass, and h rounded to bf16 alone would cost the output as much again as
//     its own rounding (relative L2 2.4e-3 against 1.7e-3). The parts' sums stay
//     apart until the first is known to be finite (two_parts).
// Bound by the weight bytes; at one token by launch and load latency; with
// more tokens by every block's reading all activations. Measured (kernels in a
// trace, median and least of 20): 1 x 4096 -> 1536 (MXFP4) 6.0 and 5.8 us; the
// gated block, 1 x 4096 x 2048, 9.0 and 8.7 us for gate and up (3.7 TB/s of
// weights), 5.6 and 4.5 for down (3.0).
#include "dense.h"

namespace moe {

// x [32 values of one group, as 4 x 8 bf16] -> E2M1 codes and exponent byte,
// all in one lane (the encoding of mxfp4.hip).
__device__ __forceinline__ u32x4_t lane_encode(const u32x4_t (&x)[4], uint32_t& byte) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max(m, max((x[i][j] << 16) & 0x7fff0000u, x[i][j] & 0x7fff0000u));
  const uint32_t field = m >> 23;
  const bool bad = field == 255u;
  const uint32_t e = field > 2u ? field - 2u : 0u;
  byte = bad ? 255u : e;
  const float sc = e8m0_scale_operand(e);
  u32x4_t c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t d = 0;
    d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, __uint_as_float(x[i][0] << 16),
                                                 __uint_as_float(x[i][0] & 0xffff0000u), sc, 0);
    d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, __uint_as_float(x[i][1] << 16),
                                                 __uint_as_float(x[i][1] & 0xffff0000u), sc, 1);
    d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, __uint_as_float(x[i][2] << 16),
                                                 __uint_as_float(x[i][2] & 0xffff0000u), sc, 2);
    d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, __uint_as_float(x[i][3] << 16),
                                                 __uint_as_float(x[i][3] & 0xffff0000u), sc, 3);
    c[i] = bad ? 0u : d;
  }
  return c;
}

// The sum of h's first parts and that of the second. An infinite weight, or a product past the largest value, makes the
// first infinite and the second NaN (a second part of 0) or infinite with either sign: the first alone is the answer.
// Where the first is finite so is the second, 2^-8 of it term by term.
__device__ __forceinline__ float two_parts(float hi, float lo) {
  return __builtin_fabsf(hi) < __builtin_inff() ? hi + lo : hi;
}

// The value of the lane 8 further on in its 16.
__device__ __forceinline__ float from_lane_8_on(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x128, 0xf, 0xf, true));  // row_ror:8
}

enum RowsFmt {
  kRowsGate = 0,   // bf16 weights and activations, gated
  kRowsMx = 1,     // MXFP4 weights, bf16 activations
  kRowsMxA4 = 2,   // MXFP4 weights, activations encoded to MXFP4
  kRowsTwo = 3,    // bf16 weights, activations the sum of two bf16
  kRowsPair = 4,   // the same for up to 8 tokens: the second parts are tokens 8 .. 15 of the MFMA, at no cost
};

template <int FMT, int CT, int NW>
__global__ __launch_bounds__(NW * 64) void k_few_rows(FewRowsArgs a) {
  constexpr bool GATE = FMT == kRowsGate, BF = GATE || FMT == kRowsTwo || FMT == kRowsPair;
  constexpr int STEP = BF ? 64 : 128;                  // k values per step
  constexpr int PV = STEP / 32;                        // 16-byte activation pieces per lane, token block and step
  constexpr int XV = FMT == kRowsTwo ? 2 * PV : PV;    // and those of the second part
  constexpr int WV = BF ? 2 : 1;                       // 16-byte weight pieces per lane and step
  constexpr int U = CT == 1 ? 4 : 2;                   // steps whose loads are in flight together
  __shared__ __align__(16) float red[NW][CT * 256];
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = blockIdx.x * (GATE ? 8 : 16);
  int row;  // the lane's weight row (past the end: the last row again, never stored)
  if constexpr (GATE) row = (r < 8 ? 0 : a.N) + n0 + (r & 7);  // N % 8 == 0
  else row = min(n0 + r, a.N - 1);
  const int S = (a.K + STEP - 1) / STEP;
  const int kl = g * (STEP / 4);  // the lane's first k of a step
  const uint8_t* wrow;
  const uint8_t* srow = nullptr;
  if constexpr (BF) {
    wrow = reinterpret_cast<const uint8_t*>(a.w + (size_t)row * a.K + kl);
  } else {
    wrow = a.codes + (size_t)row * (a.K / 2) + kl / 2;
    srow = a.scales + (size_t)row * (a.K / 32) + g;
  }
  const uint16_t *xrow[CT], *lorow[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int t = min(FMT == kRowsPair ? r & 7 : 16 * c + r, a.T - 1);
    xrow[c] = (FMT == kRowsPair && r >= 8 ? a.x_lo : a.x) + (size_t)t * a.K + kl;
    if constexpr (FMT == kRowsTwo) lorow[c] = a.x_lo + (size_t)t * a.K + kl;
  }

  constexpr int LOW = FMT == kRowsTwo ? CT : 0;  // the second parts' sums
  f32x4_t acc[CT + LOW];
#pragma unroll
  for (int c = 0; c < CT + LOW; ++c) acc[c] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  const u32x4_t zero = {0u, 0u, 0u, 0u};

  for (int s0 = wave; s0 < S; s0 += NW * U) {
    u32x4_t w[U][WV], x[U][CT][XV];
    uint32_t sc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = s0 + u * NW, k = s * STEP + kl;
#pragma unroll
      for (int v = 0; v < WV; ++v) {
        // a piece past K is zeros on both sides (K % 8 == 0; MXFP4: K % 32 == 0)
        const bool in = k + v * 8 < a.K;
        w[u][v] = in ? *reinterpret_cast<const u32x4_t*>(wrow + (size_t)s * (BF ? 128 : 64) + v * 16) : zero;
      }
      if constexpr (!BF) sc[u] = k < a.K ? srow[s * 4] : 0u;
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int v = 0; v < XV; ++v) {
          const int at = v % PV * 8;
          const uint16_t* from = (v < PV ? xrow[c] : lorow[c]) + (size_t)s * STEP + at;
          x[u][c][v] = k + at < a.K ? *reinterpret_cast<const u32x4_t*>(from) : zero;
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (BF) {
#pragma unroll
        for (int v = 0; v < XV; ++v)
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            f32x4_t& to = acc[v < PV ? c : c + LOW];
            to = mfma_bf16(w[u][v % PV], x[u][c][v], to);
          }
      } else if constexpr (FMT == kRowsMx) {
        const float sv = e8m0_scale_operand(sc[u]);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const u32x4_t wf = __builtin_bit_cast(u32x4_t, fp4x8_to_bf16x8(w[u][0][v], sv));
#pragma unroll
          for (int c = 0; c < CT; ++c) acc[c] = mfma_bf16(wf, x[u][c][v], acc[c]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          uint32_t sx;
          const u32x4_t xc = lane_encode(x[u][c], sx);
          acc[c] = mfma_mx4<0>(w[u][0], xc, acc[c], sc[u], sx);
        }
      }
    }
  }
#pragma unroll
  for (int c = 0; c < LOW; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[c][i] = two_parts(acc[c][i], acc[c + LOW][i]);
  if constexpr (FMT == kRowsPair) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[0][i] = two_parts(acc[0][i], from_lane_8_on(acc[0][i]));
  }
#pragma unroll
  for (int c = 0; c < CT; ++c) *reinterpret_cast<f32x4_t*>(&red[wave][(c * 64 + lane) * 4]) = acc[c];
  __syncthreads();
  // value j: row 4 (lane / 16) + j % 4, token 16 c + lane % 16, where (c, lane) = j / 4
  for (int j = tid; j < CT * 256; j += NW * 64) {
    const int l = (j >> 2) & 63, t = (j >> 8) * 16 + (l & 15), n = 4 * (l >> 4) + (j & 3);
    if (t >= a.T) continue;
    if constexpr (GATE) {
      if (n >= 8) continue;
      float gv = 0.0f, uv = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        gv += red[w][j];
        uv += red[w][j + 128];  // row n + 8
      }
      const size_t at = (size_t)t * a.N + n0 + n;
      const float h = ffn_act(gv, uv, a.limit);
      const uint16_t hi = f32_to_bf16(h);
      const float top = __uint_as_float((uint32_t)hi << 16);
      static_cast<uint16_t*>(a.out)[at] = hi;
      a.out_lo[at] = f32_to_bf16(__builtin_fabsf(top) < __builtin_inff() ? h - top : 0.0f);  // none beside Inf or NaN
      if (a.gu_out) {
        float* o = a.gu_out + (size_t)t * 2 * a.N + n0 + n;
        o[0] = gv;
        o[a.N] = uv;
      }
    } else {
      if (n0 + n >= a.N) continue;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) v += red[w][j];
      const size_t at = (size_t)t * a.N + n0 + n;
      if (a.out_is_fp32) static_cast<float*>(a.out)[at] = v;
      else static_cast<uint16_t*>(a.out)[at] = f32_to_bf16(v);
    }
  }
}

// Waves per block: enough that the blocks of 16 rows give each of the 256 CUs
// about 16 waves. (Where K has fewer steps than the block has waves, the others
// add zeros.) With 17 and more rows the gated block runs as tile products before
// it has more than 640 blocks: its estimate is 16 % above theirs at the least.
template <int FMT, int CT>
static hipError_t go_waves(const FewRowsArgs& a, hipStream_t st) {
  constexpr bool FOUR = CT == 1 || FMT == kRowsMx || FMT == kRowsMxA4;
  const int blocks = FMT == kRowsGate ? a.N / 8 : (a.N + 15) / 16;
  if (blocks <= 320) k_few_rows<FMT, CT, 16><<<blocks, 16 * 64, 0, st>>>(a);
  else if (blocks <= 640 || !FOUR) k_few_rows<FMT, CT, 8><<<blocks, 8 * 64, 0, st>>>(a);
  else if constexpr (FOUR) k_few_rows<FMT, CT, 4><<<blocks, 4 * 64, 0, st>>>(a);
  return hipGetLastError();
}

template <int FMT>
static hipError_t go_tokens(const FewRowsArgs& a, hipStream_t st) {
  if (a.T <= 16) return go_waves<FMT, 1>(a, st);
  return go_waves<FMT, 2>(a, st);
}

static bool few_rows_ok(const FewRowsArgs& a, int step) {
  return a.T > 0 && a.T <= kFewRows && a.N > 0 && a.K > 0 && a.K % step == 0;
}

hipError_t launch_few_rows_mxfp4(const FewRowsArgs& a, hipStream_t st) {
  if (!few_rows_ok(a, 32)) return hipErrorInvalidValue;
  return a.act_mxfp4 ? go_tokens<kRowsMxA4>(a, st) : go_tokens<kRowsMx>(a, st);
}

hipError_t launch_few_rows_gate(const FewRowsArgs& a, hipStream_t st) {
  if (!few_rows_ok(a, 8) || a.N % 8 || !a.out_lo) return hipErrorInvalidValue;
  return go_tokens<kRowsGate>(a, st);
}

hipError_t launch_few_rows_two(const FewRowsArgs& a, hipStream_t st) {
  if (!few_rows_ok(a, 8) || !a.x_lo) return hipErrorInvalidValue;
  if (a.T <= 8) return go_waves<kRowsPair, 1>(a, st);
  return go_tokens<kRowsTwo>(a, st);
}

}  // namespace moe

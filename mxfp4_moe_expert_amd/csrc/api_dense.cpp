// Host entry points of the plain MXFP4 operators and the gated block
// (include/moe.h): argument checks, workspace carving and dispatch on the
// caller's stream. Nothing here allocates device memory or synchronises.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include "internal.h"
#include "moe.h"

namespace {

using namespace moe;

constexpr int kMaxRows = 65536;   // T
constexpr int kMaxLinear = 65536; // K and N of a linear
constexpr int kMaxFfn = 16384;    // H and I of the gated block: 2 I H values stay below 2^30

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline int status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_EHIP; }
inline size_t max_of(size_t a, size_t b) { return a > b ? a : b; }

template <class P>
inline P* at(void* ws, size_t off) {
  return reinterpret_cast<P*>(static_cast<char*>(ws) + off);
}

// MOE_OK if the workspace holds `need` bytes at 256-byte alignment.
int check_ws(const void* ws, size_t have, size_t need) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255)) return MOE_EINVAL;
  return have < need ? MOE_EWORKSPACE : MOE_OK;
}

bool linear_ok(int T, int K, int N) {
  return T >= 0 && T <= kMaxRows && K >= kMxGroup && K % kMxGroup == 0 && K <= kMaxLinear && N >= 1 &&
         N <= kMaxLinear;
}

// Rows up to which a product runs in the streaming pass (few_rows.hip) rather than as a tile product. Every block of
// the pass reads all activations, T K values, through its CU's share of the L2, while the tile product splits K over
// blocks at the price of a second launch: at 4096 x 4096 (MXFP4, bf16 activations) 9.8 us at 24 rows and 11.1 at 32
// against 10.9 at 33, at K = 8192 11.9 at 12 rows and 13.2 at 16 against 12.1 at 17, at 2048 x 2048 6.7 against 7.6 at 32
// rows. The rule does not know N: at 4096 -> 1536 tiles lead from about 18 rows on (9.6 us streamed at 24 rows, 8.6 in
// tiles at 28), at 1024 -> 8192 the pass still does at 32 (6.9 us; tiles 8.8 at 33).
// Activations that the pass encodes to MXFP4 itself cost it more. 81920 lies between 4096 x 4096, where it would lead at
// 24 rows (10.6 us; tiles 11.1 at 28), and K = 8192, where it would trail at 12 (12.4 us; tiles 11.5 at 16); at 1024 ->
// 8192 it trails from 17 rows on (8.0 us at 32; tiles 6.8 at 33).
bool linear_few(int T, int K, int act) {
  return T <= kFewRows && (long long)T * K <= (act == MOE_ACT_MXFP4 ? 81920 : 98304);
}
// The gated block: two passes, by their weights and by what each CU's blocks (of 8 gate and 8 up rows; of 16) read of the
// activations (h in two parts), against the tile products' estimate. 4096 x 2048 (hidden x intermediate):
// 20.1 us at 17 rows and 22.5 at 24 against 20.8 at 24; 2048 x 1024: 12.7 at 24 and 14.1 at 32 against 13.6 at 33; 1024 x
// 4096: 14.4 at 8 and 16.8 at 12 against 14.4 at 17.
bool ffn_few(int T, int H, int I) {
  if (T <= 8 || T > kFewRows) return T <= 8;  // without the estimates' microsecond on the host where calls are shortest
  const double values = (double)T * ((double)H * ((I + 2047) / 2048) + 2.0 * I * ((H + 4095) / 4096));
  const double few_us = 7.0 + 6.0 * H * I / 1e7 + 5.7e-5 * values;
  double up_us, down_us;
  dense_plan(kDenseBf16, kDenseNT, T, 2 * I, H, &up_us);
  dense_plan(kDenseBf16, kDenseNT, T, H, I, &down_us);
  return few_us < up_us + down_us;
}

// ---- workspace layouts

constexpr size_t kNoWorkspace = 256;  // the stated size where none is used (0 stands for unsupported)

struct LinearLayout {
  DensePlan plan;
  bool codes_direct;            // act bf16: the product reads W's codes (dense_w4.hip)
  size_t w;                     // act bf16 otherwise: W as bf16 [N][K]
  size_t codes, xpack, wpack;   // act mxfp4: activation codes, packed scales of both sides
  size_t part, total;
};

LinearLayout linear_layout(int T, int K, int N, int act) {
  LinearLayout L;
  memset(&L, 0, sizeof(L));
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t p = o;
    o = align256(o + bytes);
    return p;
  };
  if (T > 0 && !linear_few(T, K, act)) {
    double us;
    L.plan = dense_plan(act == MOE_ACT_MXFP4 ? kDenseFp4 : kDenseBf16, kDenseNT, T, N, K, &us);
    if (act == MOE_ACT_BF16) {
      // expanding W: a launch, and 17/32 of a byte read and 2 written per weight
      const double expand_us = 3.0 + (double)N * K * (17.0 / 32 + 2) / 4.5e6;
      double direct_us;
      const DensePlan direct = dense_w4_plan(T, N, K, &direct_us);
      L.codes_direct = direct.tile >= 0 && direct_us < us + expand_us;
      if (L.codes_direct) L.plan = direct;
    }
    if (act == MOE_ACT_MXFP4) {
      L.codes = take((size_t)T * K / 2);
      L.xpack = take(mxfp4_pack_bytes(T, K));
      L.wpack = take(mxfp4_pack_bytes(N, K));
    } else if (!L.codes_direct) {
      L.w = take((size_t)N * K * 2);
    }
    L.part = take(dense_part_bytes(L.plan, T, N));
  }
  L.total = o == 0 ? kNoWorkspace : o < 512 ? 512 : o;
  return L;
}

struct DxLayout {
  DensePlan plan;
  int ldy;  // values per row of dy in the product
  size_t w, dyp, part, total;
};

DxLayout dx_layout(int T, int K, int N) {
  DxLayout L;
  memset(&L, 0, sizeof(L));
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t p = o;
    o = align256(o + bytes);
    return p;
  };
  L.ldy = (N + 7) & ~7;
  L.plan = dense_plan(kDenseBf16, kDenseNN, T > 0 ? T : 1, K, N);
  L.w = take((size_t)N * K * 2);
  L.dyp = take(L.ldy != N ? (size_t)T * L.ldy * 2 : 0);
  L.part = take(dense_part_bytes(L.plan, T, K));
  L.total = o;
  return L;
}

bool ffn_ok(int T, int H, int I) {
  return T >= 0 && T <= kMaxRows && H >= 8 && H % 8 == 0 && H <= kMaxFfn && I >= 8 && I % 8 == 0 && I <= kMaxFfn;
}

constexpr int kStore = 0, kGate = 1, kGrad = 2;  // epilogues of dense.h

struct FfnLayout {
  DensePlan up, down;
  bool few;               // streamed
  size_t h, part, total;  // h: [T][I] bf16; of few rows followed by what its rounding left, another [T][I]
};

FfnLayout ffn_layout(int T, int H, int I) {
  FfnLayout L;
  memset(&L, 0, sizeof(L));
  L.h = 0;
  L.few = ffn_few(T, H, I);
  size_t o = align256((size_t)T * I * (L.few ? 4 : 2));
  L.part = o;
  if (!L.few) {
    L.up = dense_plan(kDenseBf16, kDenseNT, T, 2 * I, H);
    L.down = dense_plan(kDenseBf16, kDenseNT, T, H, I);
    o = align256(o + max_of(dense_part_bytes(L.up, T, 2 * I), dense_part_bytes(L.down, T, H)));
  }
  L.total = o < 256 ? 256 : o;
  return L;
}

// The plan of one product of a pair whose other gradient is not wanted: cut as in the pair (a split K would add in
// another order), so a gradient's bits do not depend on which others are computed.
DensePlan alone_a(const DensePairPlan& p) { return p.tile >= 0 ? DensePlan{p.tile, 1} : p.a; }
DensePlan alone_b(const DensePairPlan& p) { return p.tile >= 0 ? DensePlan{p.tile, 1} : p.b; }

struct FfnGradLayout {
  DensePairPlan first, second;  // dw2 with dgu (from dh); dw13 with dx
  size_t dgu, part, total;
};

FfnGradLayout ffn_grad_layout(int T, int H, int I) {
  FfnGradLayout L;
  memset(&L, 0, sizeof(L));
  const int t = T > 0 ? T : 1;
  L.first = dense_pair_plan(H, I, t, t, I, H, 2 * 4 + 2);  // g and u read, a second bf16 value written
  L.second = dense_pair_plan(2 * I, H, t, t, H, 2 * I, 0);
  L.dgu = 0;
  L.part = align256((size_t)T * 2 * I * 2);
  size_t p = max_of(dense_part_bytes(alone_a(L.first), H, I), dense_part_bytes(alone_b(L.first), t, I));
  p = max_of(p, max_of(dense_part_bytes(alone_a(L.second), 2 * I, H), dense_part_bytes(alone_b(L.second), t, H)));
  L.total = L.part + align256(p);
  if (L.total < 256) L.total = 256;
  return L;
}

// A bf16 product on contiguous operands.
DenseArgs dense_args(const void* x, size_t x_cols, const void* w, size_t w_cols, int M, int N, int K, void* out,
                     int fp32, float* part) {
  DenseArgs a;
  memset(&a, 0, sizeof(a));
  a.x = x;
  a.w = w;
  a.x_ld = (uint32_t)(x_cols * 2);
  a.w_ld = (uint32_t)(w_cols * 2);
  a.M = M;
  a.N = N;
  a.K = K;
  a.out = out;
  a.out_is_fp32 = fp32 ? 1 : 0;
  a.part = part;
  return a;
}

}  // namespace

extern "C" {

int moe_mxfp4_quantize(int64_t rows, int32_t K, int32_t dtype, const void* x, int64_t ldx, uint8_t* codes,
                       uint8_t* scales, void* stream) {
  if (rows < 0 || K <= 0 || ldx < K) return MOE_EINVAL;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_F16) return MOE_EUNSUPPORTED;
  if (K % kMxGroup || K > kMaxLinear || rows > ((int64_t)1 << 36) / K) return MOE_EUNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scales || !aligned16(x) || !aligned16(codes) || !aligned16(scales)) return MOE_EINVAL;
  if (ldx % (dtype == MOE_DTYPE_F32 ? 4 : 8)) return MOE_EINVAL;
  return status(launch_mxfp4_quantize(rows, K, dtype, x, ldx, codes, scales, static_cast<hipStream_t>(stream)));
}

int moe_mxfp4_dequantize(int64_t rows, int32_t K, const uint8_t* codes, const uint8_t* scales, int32_t dtype,
                         void* out, void* stream) {
  if (rows < 0 || K <= 0) return MOE_EINVAL;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F32) return MOE_EUNSUPPORTED;
  if (K % kMxGroup || K > kMaxLinear || rows > ((int64_t)1 << 36) / K) return MOE_EUNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!out || !codes || !scales || !aligned16(out) || !aligned16(codes) || !aligned16(scales)) return MOE_EINVAL;
  return status(launch_mxfp4_dequantize(rows, K, codes, scales, dtype, out, static_cast<hipStream_t>(stream)));
}

size_t moe_linear_mxfp4_workspace_size(int32_t T, int32_t K, int32_t N, int32_t act) {
  if (!linear_ok(T, K, N) || (act != MOE_ACT_BF16 && act != MOE_ACT_MXFP4)) return 0;
  return linear_layout(T, K, N, act).total;
}

int moe_linear_mxfp4(int32_t T, int32_t K, int32_t N, const uint16_t* x, const uint8_t* codes, const uint8_t* scales,
                     int32_t act, void* out, int32_t out_is_fp32, void* workspace, size_t workspace_bytes,
                     void* stream) {
  if (T < 0 || K <= 0 || N <= 0) return MOE_EINVAL;
  if (!linear_ok(T, K, N) || (act != MOE_ACT_BF16 && act != MOE_ACT_MXFP4)) return MOE_EUNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !codes || !scales || !out) return MOE_EINVAL;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales) || !aligned16(out)) return MOE_EINVAL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (linear_few(T, K, act)) {
    FewRowsArgs a;
    memset(&a, 0, sizeof(a));
    a.T = T;
    a.N = N;
    a.K = K;
    a.x = x;
    a.codes = codes;
    a.scales = scales;
    a.act_mxfp4 = act == MOE_ACT_MXFP4;
    a.out = out;
    a.out_is_fp32 = out_is_fp32 ? 1 : 0;
    return status(launch_few_rows_mxfp4(a, st));
  }
  const LinearLayout L = linear_layout(T, K, N, act);
  if (L.total != kNoWorkspace) {
    const int rc = check_ws(workspace, workspace_bytes, L.total);
    if (rc) return rc;
  }
  float* part = at<float>(workspace, L.part);
  if (act == MOE_ACT_MXFP4) {
    uint8_t* xc = at<uint8_t>(workspace, L.codes);
    uint32_t* xp = at<uint32_t>(workspace, L.xpack);
    uint32_t* wp = at<uint32_t>(workspace, L.wpack);
    const hipError_t e = launch_mxfp4_prep(T, K, x, xc, xp, N, scales, wp, st);
    if (e != hipSuccess) return status(e);
    DenseArgs a = dense_args(xc, (size_t)K / 4, codes, (size_t)K / 4, T, N, K, out, out_is_fp32, part);
    a.x_scales = xp;
    a.w_scales = wp;
    a.x_blocks = mxfp4_blocks(T);
    a.w_blocks = mxfp4_blocks(N);
    return status(launch_dense(kDenseFp4, kDenseNT, kStore, L.plan, a, st));
  }
  if (L.codes_direct)
    return status(launch_dense_w4(L.plan, dense_args(x, K, codes, (size_t)K / 4, T, N, K, out, out_is_fp32, part),
                                  scales, st));
  uint16_t* w = at<uint16_t>(workspace, L.w);
  const hipError_t e = launch_mxfp4_expand(N, K, codes, scales, w, 0, nullptr, nullptr, 8, st);
  if (e != hipSuccess) return status(e);
  return status(launch_dense(kDenseBf16, kDenseNT, kStore, L.plan,
                             dense_args(x, K, w, K, T, N, K, out, out_is_fp32, part), st));
}

size_t moe_linear_mxfp4_dx_workspace_size(int32_t T, int32_t K, int32_t N) {
  return linear_ok(T, K, N) ? dx_layout(T, K, N).total : 0;
}

int moe_linear_mxfp4_dx(int32_t T, int32_t K, int32_t N, const uint16_t* dy, const uint8_t* codes,
                        const uint8_t* scales, void* dx, int32_t out_is_fp32, void* workspace, size_t workspace_bytes,
                        void* stream) {
  if (T < 0 || K <= 0 || N <= 0) return MOE_EINVAL;
  if (!linear_ok(T, K, N)) return MOE_EUNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!dy || !codes || !scales || !dx) return MOE_EINVAL;
  if (!aligned16(dy) || !aligned16(codes) || !aligned16(scales) || !aligned16(dx)) return MOE_EINVAL;
  const DxLayout L = dx_layout(T, K, N);
  const int rc = check_ws(workspace, workspace_bytes, L.total);
  if (rc) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  uint16_t* w = at<uint16_t>(workspace, L.w);
  const bool pad = L.ldy != N;
  uint16_t* dyp = at<uint16_t>(workspace, L.dyp);
  const hipError_t e = launch_mxfp4_expand(N, K, codes, scales, w, T, pad ? dy : nullptr, dyp, L.ldy, st);
  if (e != hipSuccess) return status(e);
  return status(launch_dense(kDenseBf16, kDenseNN, kStore, L.plan,
                             dense_args(pad ? dyp : dy, L.ldy, w, K, T, K, N, dx, out_is_fp32,
                                        at<float>(workspace, L.part)), st));
}

size_t moe_gated_ffn_workspace_size(int32_t T, int32_t H, int32_t I) {
  return ffn_ok(T, H, I) ? ffn_layout(T, H, I).total : 0;
}

int moe_gated_ffn(int32_t T, int32_t H, int32_t I, float limit, const uint16_t* x, const uint16_t* w13,
                  const uint16_t* w2, float* gu_saved, uint16_t* h_saved, void* out, int32_t out_is_fp32,
                  void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 0 || H <= 0 || I <= 0 || !(limit > 0.0f)) return MOE_EINVAL;
  if (!ffn_ok(T, H, I)) return MOE_EUNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !w13 || !w2 || !out || (gu_saved == nullptr) != (h_saved == nullptr)) return MOE_EINVAL;
  if (!aligned16(x) || !aligned16(w13) || !aligned16(w2) || !aligned16(out) || !aligned16(gu_saved) ||
      !aligned16(h_saved))
    return MOE_EINVAL;
  const FfnLayout L = ffn_layout(T, H, I);
  const int rc = check_ws(workspace, workspace_bytes, L.total);
  if (rc) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  uint16_t* h = h_saved ? h_saved : at<uint16_t>(workspace, L.h);
  if (L.few) {
    uint16_t* h_lo = at<uint16_t>(workspace, L.h) + (size_t)T * I;
    FewRowsArgs a;
    memset(&a, 0, sizeof(a));
    a.T = T;
    a.N = I;
    a.K = H;
    a.x = x;
    a.w = w13;
    a.out = h;
    a.out_lo = h_lo;
    a.limit = limit;
    a.gu_out = gu_saved;
    const hipError_t e = launch_few_rows_gate(a, st);
    if (e != hipSuccess) return status(e);
    memset(&a, 0, sizeof(a));
    a.T = T;
    a.N = H;
    a.K = I;
    a.x = h;
    a.x_lo = h_lo;
    a.w = w2;
    a.out = out;
    a.out_is_fp32 = out_is_fp32 ? 1 : 0;
    return status(launch_few_rows_two(a, st));
  }
  float* part = at<float>(workspace, L.part);
  DenseArgs a = dense_args(x, H, w13, H, T, 2 * I, H, h, 0, part);
  a.I = I;
  a.limit = limit;
  a.gu_out = gu_saved;
  const hipError_t e = launch_dense(kDenseBf16, kDenseNT, kGate, L.up, a, st);
  if (e != hipSuccess) return status(e);
  return status(launch_dense(kDenseBf16, kDenseNT, kStore, L.down,
                             dense_args(h, I, w2, I, T, H, I, out, out_is_fp32, part), st));
}

size_t moe_gated_ffn_backward_workspace_size(int32_t T, int32_t H, int32_t I) {
  return ffn_ok(T, H, I) ? ffn_grad_layout(T, H, I).total : 0;
}

int moe_gated_ffn_backward(int32_t T, int32_t H, int32_t I, float limit, const uint16_t* dy, const uint16_t* x,
                           const uint16_t* w13, const uint16_t* w2, const float* gu_saved,
                           const uint16_t* h_saved, uint16_t* dx, void* dw13, void* dw2, int32_t dw_is_fp32,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 0 || H <= 0 || I <= 0 || !(limit > 0.0f)) return MOE_EINVAL;
  if (!ffn_ok(T, H, I)) return MOE_EUNSUPPORTED;
  if (!aligned16(dx) || !aligned16(dw13) || !aligned16(dw2)) return MOE_EINVAL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (T == 0) {
    const size_t el = dw_is_fp32 ? 4 : 2;
    if (dw13) {
      const hipError_t e = launch_fill_zero(dw13, (size_t)2 * I * H * el, st);
      if (e != hipSuccess) return status(e);
    }
    return dw2 ? status(launch_fill_zero(dw2, (size_t)I * H * el, st)) : MOE_OK;
  }
  if (!dy || !x || !w13 || !w2 || !gu_saved || !h_saved) return MOE_EINVAL;
  if (!aligned16(dy) || !aligned16(x) || !aligned16(w13) || !aligned16(w2) || !aligned16(gu_saved) ||
      !aligned16(h_saved))
    return MOE_EINVAL;
  const FfnGradLayout L = ffn_grad_layout(T, H, I);
  const int rc = check_ws(workspace, workspace_bytes, L.total);
  if (rc) return rc;
  uint16_t* dgu = at<uint16_t>(workspace, L.dgu);
  float* part = at<float>(workspace, L.part);
  hipError_t e = hipSuccess;
  const DenseArgs gw2 = dense_args(dy, H, h_saved, I, H, I, T, dw2, dw_is_fp32, part);
  DenseArgs gdgu = dense_args(dy, H, w2, I, T, I, H, dgu, 0, part);
  gdgu.I = I;
  gdgu.limit = limit;
  gdgu.gu_in = gu_saved;
  const bool inner = dx || dw13;
  if (dw2 && inner) e = launch_dense_pair(kGrad, L.first, gw2, gdgu, st);
  else if (dw2) e = launch_dense(kDenseBf16, kDenseTN, kStore, alone_a(L.first), gw2, st);
  else if (inner) e = launch_dense(kDenseBf16, kDenseNN, kGrad, alone_b(L.first), gdgu, st);
  if (e != hipSuccess || !inner) return status(e);
  const DenseArgs gw13 = dense_args(dgu, 2 * I, x, H, 2 * I, H, T, dw13, dw_is_fp32, part);
  const DenseArgs gx = dense_args(dgu, 2 * I, w13, H, T, H, 2 * I, dx, 0, part);
  if (dx && dw13) e = launch_dense_pair(kStore, L.second, gw13, gx, st);
  else if (dw13) e = launch_dense(kDenseBf16, kDenseTN, kStore, alone_a(L.second), gw13, st);
  else e = launch_dense(kDenseBf16, kDenseNN, kStore, alone_b(L.second), gx, st);
  return status(e);
}

}  // extern "C"

// y = x W^T for rows that are many for the streaming pass (few_rows.hip) and
// few for expanding W to bf16 first: the tile product of dense.h with W read
// as it is stored. W's tile holds the 16 bytes of codes that a row has per
// group of 32 values, eight groups (128-byte lines) per ring stage; lane
// (r, g) of a k-step reads the 4 bytes of its 8 values and converts them to
// bf16 (exact) under the previous k-step's last MFMAs. Conversions and MFMAs
// share the SIMD's issue, so at 64 rows every wave takes all of them and
// converts its own 16 columns only (0.375 against 0.40 us a stage with two
// waves per column block; the bf16 product: 0.30). The tile's exponent bytes
// are copied to LDS once, before the K loop (a byte per row and k-step is then
// one LDS read).
//
// Measured (the kernel in a trace, medians): 33 x 8192 -> 4096, eight slices of
// K, 12.7 us, of which the 16 stages are 6 (0.37 us each: LDS latency, which a
// wave's four MFMAs a k-step do not cover) and the rest is before and after
// them: the exponent bytes pass through registers, everything loaded first is
// waited for together, and 4 MB of partial sums are stored. 1000 x 4096 ->
// 4096 41.9 us (0.80 PFLOP/s; untraced, a call among others 37 to 39 us; the
// bf16 product with W expanded before it: 34.7 + 8.6).
#include "dense.h"

namespace moe {

constexpr int kWStage = 4;  // X stages (64 k) per W ring stage (256 k)

// One 16-row block of W for k-step t (0..7) of a ring stage.
__device__ __forceinline__ uint32_t read_codes(const lds_u8* tile, uint32_t row_off, uint32_t key, int t) {
  return *(const lds_u32*)(tile + row_off + ((((uint32_t)t << 4) ^ key)));
}

template <int BM, int BN, int WGM, int WGN, int NX, int EPI>
__global__ __launch_bounds__(WGM* WGN * 64) void k_dense_w4(DenseArgs a, const uint8_t* scales, int scld) {
  constexpr int W = WGM * WGN;
  constexpr int MB = BM / WGM / 16, NB = BN / WGN / 16;
  constexpr int XB = BM * kStageB, WB = BN * kStageB;
  constexpr uint32_t WBASE = NX * XB, SCALES = WBASE + 2 * WB;  // LDS: X ring, W ring, exponent bytes [BN][scld]
  using SX = Stager<false, BM, W>;
  using SW = Stager<false, BN, W>;
  static_assert(NX >= 3 && NX <= 5, "W of the next ring stage is loaded before the X loads that may be outstanding");
  extern __shared__ __align__(16) unsigned char smem[];
  lds_u8* const lds = (lds_u8*)smem;
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;

  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int im, in;
  dense_tile(blockIdx.x, a.tm, a.tn, im, in);
  const int m0 = im * BM, n0 = in * BN;
  const int st0 = blockIdx.y * a.slice_stages;  // a multiple of kWStage
  const int nst = min(a.slice_stages, a.stages - st0);

  SX sx;
  SW sw;
  sx.init_kc(wave, lane, a.x_ld, [&](int i) { return m0 + i < a.M ? i : -1; });
  sw.init_kc(wave, lane, a.w_ld, [&](int i) { return n0 + i < a.N ? i : -1; });
  const char* wbase = static_cast<const char*>(a.w) + (size_t)n0 * a.w_ld;
  const int xat = SX::first_k(wave, lane), wat = SW::first_k(wave, lane);

  // the next X stage to load: from, bytes of k left in the slice (0 or less: nothing is read), ring place
  const char* xsrc = static_cast<const char*>(a.x) + (size_t)m0 * a.x_ld + (size_t)st0 * kStageB;
  int xleft = min(2 * a.K, (st0 + nst) * kStageB) - st0 * kStageB;
  uint32_t xat_lds = lds0;
  auto load_x = [&](int op) { sx.load(op, buffer_of(xsrc), xat_lds, wave, xat, xleft); };
  auto next_x = [&]() {
    xsrc += kStageB;
    xleft -= kStageB;
    xat_lds = xat_lds == lds0 + (NX - 1) * XB ? lds0 : xat_lds + XB;
  };
  auto load_w = [&](int j) {  // ring stage j: X stages 4 j .. 4 j + 3 of the slice
    const bool live = j * kWStage < nst;
    const int st = live ? st0 / kWStage + j : 0;
    const u32x4_t rs = buffer_of(wbase + (size_t)st * kStageB);
#pragma unroll
    for (int op = 0; op < SW::NI; ++op)
      sw.load(op, rs, lds0 + WBASE + (uint32_t)(j & 1) * WB, wave, wat, live ? a.K / 2 - st * kStageB : 0);
  };

  const int wm = wave / WGN, wn = wave % WGN;
  Reader<false, BM, MB> rx;
  rx.init(wm * MB * 16, lane);
  const uint32_t wrow = (uint32_t)((wn * NB * 16 + r) * kStageB + g * 4), wkey = (uint32_t)(r >> 1) << 4;
  const lds_u8* srow = lds + SCALES + (wn * NB * 16 + r) * scld;

  f32x4_t acc[NB][MB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int c = 0; c < MB; ++c) acc[b][c] = (f32x4_t){0.f, 0.f, 0.f, 0.f};

  // Loads in flight before the scales are fetched: W(0), X(0) .. X(NX - 2)
  load_w(0);
#pragma unroll
  for (int i = 0; i < NX - 1; ++i) {
#pragma unroll
    for (int op = 0; op < SX::NI; ++op) load_x(op);
    next_x();
  }
  {
    // exponent bytes of the slice; groups past K as 0 (their codes are zeros). scld is a multiple of 4.
    const int G = a.K / kMxGroup, g0 = st0 * 2, ng = min(nst * 2, G - g0);
    const int wide = (G & 3) == 0 ? scld >> 2 : 0;  // dwords where rows are aligned so (g0 is a multiple of 8)
    if (wide) {
      for (int i = tid; i < BN * wide; i += W * 64) {
        const int row = i / wide, q = i - row * wide;
        const uint8_t* s = scales + (size_t)min(n0 + row, a.N - 1) * G + g0 + 4 * q;
        *(lds_u32*)(lds + SCALES + row * scld + 4 * q) = 4 * q < ng ? *reinterpret_cast<const uint32_t*>(s) : 0u;
      }
    } else {
      for (int i = tid; i < BN * scld; i += W * 64) {
        const int row = i / scld, q = i - row * scld;
        lds[SCALES + row * scld + q] = q < ng ? scales[(size_t)min(n0 + row, a.N - 1) * G + g0 + q] : (uint8_t)0;
      }
    }
  }
  dense_wait<0>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");

  u32x4_t xf[2][MB], wf[2][NB];
  uint32_t wq[NB], ws[NB];  // the next k-step's codes and exponent bytes
  auto read_w = [&](int b, int t) {
    wq[b] = read_codes(lds + WBASE + ((t >> 3) & 1) * WB, wrow + b * (16 * kStageB), wkey, t & 7);
    ws[b] = srow[b * 16 * scld + t];
  };
  auto convert = [&](int b) {
    return __builtin_bit_cast(u32x4_t, fp4x8_to_bf16x8(wq[b], e8m0_scale_operand(ws[b])));
  };
#pragma unroll
  for (int b = 0; b < NB; ++b) read_w(b, 0);
#pragma unroll
  for (int c = 0; c < MB; ++c) xf[0][c] = rx.read(lds, c, 0);
#pragma unroll
  for (int b = 0; b < NB; ++b) wf[0][b] = convert(b);

  // The MFMAs of k-step kk; between them the loads, the reads of k-step t (of the slice) into the other register set
  // (X from tile xt), and late enough for those to have arrived the conversions of its W operands.
  auto step = [&](auto kk, const lds_u8* xt, int t, auto nload) {
    constexpr int NM = MB * NB, NR = NB + MB, CV = NM - NB;
    static_assert(nload <= CV, "the loads end before the conversions begin");
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      const int c = m / NB, b = m % NB;
      acc[b][c] = mfma_bf16(wf[kk][b], xf[kk][c], acc[b][c]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = spread(m - 1, CV, nload); i < spread(m, CV, nload); ++i) load_x(i);
#pragma unroll
      for (int i = spread(2 * m - 2, NM, NR); i < spread(2 * m, NM, NR); ++i) {
        if (i < NB) read_w(i, t);
        else xf[1 - kk][i - NB] = rx.read(xt, i - NB, 1 - kk);
      }
      if (nload > 0 && m == CV) next_x();
      if (m >= CV) wf[1 - kk][m - CV] = convert(m - CV);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  using K0 = std::integral_constant<int, 0>;
  using K1 = std::integral_constant<int, 1>;
  int bx = 0;
  for (int i = 0; i < nst; ++i) {
    const int nx = bx + 1 == NX ? 0 : bx + 1;
    // X of stage i - 1 + NX is loaded where stage i - 1 was
    step(K0{}, lds + bx * XB, 2 * i + 1, std::integral_constant<int, SX::NI>{});
    // X of stage i + 1 has landed (W of its ring stage was loaded before it) and this wave has read stage i, then
    // every wave
    dense_wait<(NX - 2) * SX::NI>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (i % kWStage == 0) load_w(i / kWStage + 1);  // over ring stage i / 4 - 1, which every wave has read
    step(K1{}, lds + nx * XB, 2 * i + 2, K0{});
    bx = nx;
  }
  dense_wait<0>();  // nothing may still write this block's LDS when it ends
  void* out = EPI == kEpiPartial ? static_cast<void*>(a.part + (size_t)blockIdx.y * a.M * a.N) : a.out;
  store_tile<MB, NB>(acc, out, EPI == kEpiPartial || a.out_is_fp32, a.M, a.N, m0 + wm * MB * 16, n0 + wn * NB * 16,
                     lane);
}

namespace {

struct W4Cfg {
  int bm, bn, nx;
};
constexpr W4Cfg kW4[] = {{64, 128, 4}, {128, 128, 4}, {256, 128, 3}};
constexpr int kNumW4 = 3;
constexpr int kW4Threads = 512;

inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// bytes per row of the exponent bytes of a slice: an odd number of dwords, so that the 16 rows a wave reads at once
// lie in different banks, with room for the k-step after the last
inline int w4_scld(int slice_stages) { return ((2 * slice_stages + 4) / 4 | 1) * 4; }
inline size_t w4_lds(const W4Cfg& t, int slice_stages) {
  return ((size_t)t.nx * t.bm + 2 * t.bn) * kStageB + (size_t)t.bn * w4_scld(slice_stages);
}
inline int w4_slice_stages(int nst, int slices) { return (ceil_div(nst, slices) + kWStage - 1) / kWStage * kWStage; }

template <int EPI>
hipError_t go(int tile, int slices, const DenseArgs& a, const uint8_t* scales, size_t lds, hipStream_t st) {
  auto run = [&](auto kern) -> hipError_t {
    const hipError_t e = allow_lds<decltype(kern)::value>(kLdsBlockMax);  // lds differs from call to call
    if (e != hipSuccess) return e;
    decltype(kern)::value<<<dim3((unsigned)(a.tm * a.tn), (unsigned)slices), kW4Threads, lds, st>>>(
        a, scales, w4_scld(a.slice_stages));
    return hipGetLastError();
  };
  if (tile == 0) return run(Kernel<&k_dense_w4<64, 128, 1, 8, kW4[0].nx, EPI>>{});
  if (tile == 1) return run(Kernel<&k_dense_w4<128, 128, 2, 4, kW4[1].nx, EPI>>{});
  return run(Kernel<&k_dense_w4<256, 128, 2, 4, kW4[2].nx, EPI>>{});
}

}  // namespace

DensePlan dense_w4_plan(int M, int N, int K, double* us_out) {
  const int nst = (K + 63) / 64;
  // full-chip stage times at 4096 x 4096 weights, 1000 rows of 128 x 128 tiles and 2048 of 256 x 128
  constexpr double stage_us[kNumW4] = {0.38, 0.53, 0.83}, start_us = 4.0;
  DensePlan best = {-1, 0};
  double best_us = 1e30;
  for (int t = 0; t < kNumW4; ++t) {
    const long long tiles = (long long)ceil_div(M, kW4[t].bm) * ceil_div(N, kW4[t].bn);
    for (int s = 1; s <= 16; s *= 2) {
      const int per = w4_slice_stages(nst, s), slices = ceil_div(nst, per);
      if (w4_lds(kW4[t], per) > kLdsBlockMax) continue;
      const long long blocks = tiles * slices;
      double us = (double)((blocks + 255) / 256) * (per * stage_us[t] + start_us);
      if (slices > 1) us += 2.5 + 2.0 * slices * M * (double)N * 4 / 4e6;
      if (us < best_us) {
        best_us = us;
        best = {t, slices};
      }
    }
  }
  if (us_out) *us_out = best_us;
  return best;
}

hipError_t launch_dense_w4(const DensePlan& p, DenseArgs a, const uint8_t* scales, hipStream_t st) {
  if (a.M <= 0 || a.N <= 0 || a.K <= 0 || a.K % kMxGroup || p.tile < 0 || p.tile >= kNumW4 || p.slices < 1 ||
      (p.slices > 1 && !a.part))
    return hipErrorInvalidValue;
  const W4Cfg& t = kW4[p.tile];
  a.stages = (a.K + 63) / 64;
  a.slice_stages = w4_slice_stages(a.stages, p.slices);
  const size_t lds = w4_lds(t, a.slice_stages);
  a.tm = ceil_div(a.M, t.bm);
  a.tn = ceil_div(a.N, t.bn);
  if (ceil_div(a.stages, a.slice_stages) != p.slices || lds > kLdsBlockMax || (long long)a.tm * a.tn > 0x3fffff)
    return hipErrorInvalidValue;
  if (p.slices == 1) return go<kEpiStore>(p.tile, 1, a, scales, lds, st);
  const hipError_t e = go<kEpiPartial>(p.tile, p.slices, a, scales, lds, st);
  return e != hipSuccess ? e : launch_dense_reduce(kEpiStore, a, p.slices, st);
}

}  // namespace moe

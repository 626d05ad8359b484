// Launching the dense products of dense.h: tile configurations, the split of
// K for products with few tiles, and its reduction.
#include "dense.h"

namespace moe {

namespace {

struct TileCfg {
  int bm, bn, nx, nw;  // nx, nw: stages of X and W in LDS
  int scale_sets;      // MXFP4: sets of scales of two stages
};
// The rings fill the 160 KB of a CU (64 x 128: half of it, two blocks per CU). MXFP4: the scales take the place of a
// stage of X in the largest tile.
constexpr TileCfg kTiles[] = {{256, 256, 3, 2, 2}, {256, 128, 3, 3, 2}, {128, 128, 4, 4, 3}, {64, 128, 3, 3, 2}};
constexpr TileCfg kTilesFp4[] = {{256, 256, 2, 2, 2}, {256, 128, 3, 3, 2}, {128, 128, 4, 4, 3}, {64, 128, 3, 3, 2}};
constexpr int kNumTiles = 4;
constexpr int kTileThreads = 512;

constexpr size_t tile_lds(const TileCfg& t, bool fp4) {
  return ((size_t)t.nx * t.bm + (size_t)t.nw * t.bn) * kStageB + (fp4 ? (size_t)t.scale_sets * (t.bm + t.bn) * 16 : 0);
}

// Sums the slices of a split K in order, then the epilogue of the product.
// Thread: four consecutive columns of one row.
template <int EPI>
__global__ __launch_bounds__(64) void k_dense_reduce(DenseArgs a, int slices) {
  const int cols = EPI == kEpiGate ? a.I : a.N;
  const int per = (cols + 3) / 4;
  const long long id = (long long)blockIdx.x * 64 + threadIdx.x;
  const int m = (int)(id / per), n = (int)(id - (long long)m * per) * 4;
  if (m >= a.M) return;
  const size_t plane = (size_t)a.M * a.N;
  const bool wide = (a.N & 3) == 0;
  auto sum = [&](int col) {
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    const float* p = a.part + (size_t)m * a.N + col;
    if (wide) {
      // eight slices' loads in flight together (past the last slice: the last again, not added)
      constexpr int AHEAD = 8;
      for (int s0 = 0; s0 < slices; s0 += AHEAD) {
        f32x4_t t[AHEAD];
#pragma unroll
        for (int s = 0; s < AHEAD; ++s)
          t[s] = *reinterpret_cast<const f32x4_t*>(p + (size_t)min(s0 + s, slices - 1) * plane);
#pragma unroll
        for (int s = 0; s < AHEAD; ++s)
          if (s0 + s < slices) v += t[s];
      }
    } else {
      for (int s = 0; s < slices; ++s, p += plane) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (col + i < a.N) v[i] += p[i];
      }
    }
    return v;
  };
  if constexpr (EPI == kEpiGate) {
    const f32x4_t g = sum(n), u = sum(a.I + n);
    f32x4_t h;
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = ffn_act(g[i], u[i], a.limit);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + (size_t)m * a.I + n) = pack4_bf16(h);
    if (a.gu_out) {
      float* o = a.gu_out + (size_t)m * 2 * a.I + n;
      *reinterpret_cast<f32x4_t*>(o) = g;
      *reinterpret_cast<f32x4_t*>(o + a.I) = u;
    }
  } else if constexpr (EPI == kEpiGrad) {
    const float* s = a.gu_in + (size_t)m * 2 * a.I + n;
    const f32x4_t g = *reinterpret_cast<const f32x4_t*>(s), u = *reinterpret_cast<const f32x4_t*>(s + a.I);
    f32x4_t dg, du;
    ffn_act_grad4(g, u, sum(n), a.limit, dg, du);
    uint16_t* o = static_cast<uint16_t*>(a.out) + (size_t)m * 2 * a.I + n;
    *reinterpret_cast<uint2*>(o) = pack4_bf16(dg);
    *reinterpret_cast<uint2*>(o + a.I) = pack4_bf16(du);
  } else {
    store4(a.out, a.out_is_fp32, (size_t)m * a.N + n, sum(n), a.N - n, wide);
  }
}

template <auto KERNEL>
hipError_t run(const TileCfg& t, bool fp4, int slices, const DenseArgs& a, hipStream_t st) {
  const size_t lds = tile_lds(t, fp4);
  const hipError_t e = allow_lds<KERNEL>((int)lds);
  if (e != hipSuccess) return e;
  KERNEL<<<dim3((unsigned)(a.tm * a.tn), (unsigned)slices), kTileThreads, lds, st>>>(a);
  return hipGetLastError();
}

template <bool XT, bool WT, bool FP4, int EPI>
hipError_t run_tile(int tile, int slices, const DenseArgs& a, hipStream_t st) {
  constexpr const TileCfg* t = FP4 ? kTilesFp4 : kTiles;
  if (tile == 0) return run<&k_dense<XT, WT, 256, 256, 2, 4, t[0].nx, t[0].nw, FP4, EPI>>(t[0], FP4, slices, a, st);
  if (tile == 1) return run<&k_dense<XT, WT, 256, 128, 2, 4, t[1].nx, t[1].nw, FP4, EPI>>(t[1], FP4, slices, a, st);
  if (tile == 2) return run<&k_dense<XT, WT, 128, 128, 2, 4, t[2].nx, t[2].nw, FP4, EPI>>(t[2], FP4, slices, a, st);
  return run<&k_dense<XT, WT, 64, 128, 2, 4, t[3].nx, t[3].nw, FP4, EPI>>(t[3], FP4, slices, a, st);
}

template <int EPI>
hipError_t run_bf16(DenseLayout layout, int tile, int slices, const DenseArgs& a, hipStream_t st) {
  if constexpr (EPI == kEpiGate) {
    return layout == kDenseNT ? run_tile<false, false, false, EPI>(tile, slices, a, st) : hipErrorInvalidValue;
  } else if constexpr (EPI == kEpiGrad) {
    return layout == kDenseNN ? run_tile<false, true, false, EPI>(tile, slices, a, st) : hipErrorInvalidValue;
  } else {
    if (layout == kDenseNT) return run_tile<false, false, false, EPI>(tile, slices, a, st);
    if (layout == kDenseNN) return run_tile<false, true, false, EPI>(tile, slices, a, st);
    return run_tile<true, true, false, EPI>(tile, slices, a, st);
  }
}

inline int stages_of(DenseKind kind, int K) { return kind == kDenseFp4 ? (K + 255) / 256 : (K + 63) / 64; }
inline int ceil_div(int a, int b) { return (a + b - 1) / b; }
// stages per slice; MXFP4 slices are whole pairs of stages (their scales are packed so)
inline int slice_stages(DenseKind kind, int nst, int slices) {
  const int per = ceil_div(nst, slices);
  return kind == kDenseFp4 && slices > 1 ? (per + 1) & ~1 : per;
}

}  // namespace

// Microseconds per stage of a block, by tile, where few CUs are busy and on a full chip, and the rest of a block's time
// (launch, first loads, epilogue). A block is bound by its share of the L2 -> LDS path, then by the matrix cores.
// Measured on 4096 x 4096 weights at 33 to 4096 rows: of the cuts tried for each size, the rule takes the fastest or one
// within a few percent of it. MXFP4 products are cut by the same times, though a stage of theirs is other work; their
// cuts were not timed one against another.
constexpr double kFewUs[kNumTiles] = {0.95, 0.47, 0.32, 0.26}, kFullUs[kNumTiles] = {1.45, 0.80, 0.47, 0.34};
constexpr double kStartUs = 4.5;
constexpr double kPairUs = 0.56;  // 64 x 128: a stage of both blocks of a CU
constexpr double kTnCost = 1.12;  // a stage with both operands transposed (7 to 16 % by tile at 4096 x 4096 x 8192)
inline double stage_us(int tile, double blocks) {
  const double full = blocks < 256 ? blocks / 256 : 1.0;
  if (tile == 3 && blocks > 256) return kFullUs[3] + (blocks > 512 ? 1.0 : (blocks - 256) / 256) * (kPairUs - kFullUs[3]);
  return kFewUs[tile] + full * (kFullUs[tile] - kFewUs[tile]);
}
inline int places(int tile) { return tile == 3 ? 512 : 256; }  // blocks the chip holds

// The plan with the least estimated time: rounds of blocks over the 256 CUs times the stages each runs, plus the
// partial sums' traffic (written and read at about 4 TB/s) and launch for a split.
DensePlan dense_plan(DenseKind kind, DenseLayout layout, int M, int N, int K, double* us_out) {
  const int nst = stages_of(kind, K);
  DensePlan best = {0, 1};
  double best_us = 1e30;
  for (int t = 0; t < kNumTiles; ++t) {
    const long long tiles = (long long)ceil_div(M, kTiles[t].bm) * ceil_div(N, kTiles[t].bn);
    for (int s = 1; s <= 16 && s * 4 <= nst + 3; s *= 2) {
      const int per = slice_stages(kind, nst, s), slices = ceil_div(nst, per);
      const long long blocks = tiles * slices;
      const double stage = stage_us(t, (double)blocks) * (layout == kDenseTN ? kTnCost : 1.0);
      double us = (double)((blocks + places(t) - 1) / places(t)) * (per * stage + kStartUs);
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

size_t dense_part_bytes(const DensePlan& p, int M, int N) {
  return p.slices > 1 ? (size_t)p.slices * M * N * sizeof(float) : 0;
}

hipError_t launch_dense(DenseKind kind, DenseLayout layout, int epi, const DensePlan& p, DenseArgs a, hipStream_t st) {
  if (a.M <= 0 || a.N <= 0 || a.K <= 0 || p.tile < 0 || p.tile >= kNumTiles || p.slices < 1 ||
      (p.slices > 1 && !a.part))
    return hipErrorInvalidValue;
  const TileCfg& t = kTiles[p.tile];
  a.stages = stages_of(kind, a.K);
  a.slice_stages = slice_stages(kind, a.stages, p.slices);
  if (ceil_div(a.stages, a.slice_stages) != p.slices) return hipErrorInvalidValue;
  const bool split = p.slices > 1;
  a.tm = ceil_div(a.M, t.bm);
  // the gate epilogue pairs gate and up rows in a tile; its split product is a plain [M][2I]
  const bool gate = epi == kEpiGate && !split;
  a.tn = gate ? ceil_div(a.I, t.bn / 2) : ceil_div(a.N, t.bn);
  if ((long long)a.tm * a.tn > 0x3fffff) return hipErrorInvalidValue;
  hipError_t e;
  const int first = split ? (int)kEpiPartial : epi;
  if (kind == kDenseFp4) {
    if (layout != kDenseNT || epi != kEpiStore) return hipErrorInvalidValue;
    e = split ? run_tile<false, false, true, kEpiPartial>(p.tile, p.slices, a, st)
              : run_tile<false, false, true, kEpiStore>(p.tile, p.slices, a, st);
  } else if (first == kEpiGate) {
    e = run_bf16<kEpiGate>(layout, p.tile, p.slices, a, st);
  } else if (first == kEpiGrad) {
    e = run_bf16<kEpiGrad>(layout, p.tile, p.slices, a, st);
  } else if (first == kEpiPartial) {
    e = run_bf16<kEpiPartial>(layout, p.tile, p.slices, a, st);
  } else {
    e = run_bf16<kEpiStore>(layout, p.tile, p.slices, a, st);
  }
  return e != hipSuccess || !split ? e : launch_dense_reduce(epi, a, p.slices, st);
}

namespace {

template <int EPI>
hipError_t run_pair(int tile, const DenseArgs& a, const DenseArgs& b, hipStream_t st) {
  const int na = a.tm * a.tn, nb = b.tm * b.tn;
  const int b_first = b.stages > a.stages;
  const int second = ((b_first ? nb : na) + 7) & ~7;
  const unsigned grid = (unsigned)(second + (b_first ? na : nb));
  auto go = [&](auto kern) -> hipError_t {
    const size_t lds = tile_lds(kTiles[tile], false);
    const hipError_t e = allow_lds<decltype(kern)::value>((int)lds);
    if (e != hipSuccess) return e;
    decltype(kern)::value<<<grid, kTileThreads, lds, st>>>(a, b, second, b_first);
    return hipGetLastError();
  };
  constexpr const TileCfg* t = kTiles;
  if (tile == 0) return go(Kernel<&k_dense_pair<256, 256, 2, 4, t[0].nx, t[0].nw, EPI>>{});
  if (tile == 1) return go(Kernel<&k_dense_pair<256, 128, 2, 4, t[1].nx, t[1].nw, EPI>>{});
  if (tile == 2) return go(Kernel<&k_dense_pair<128, 128, 2, 4, t[2].nx, t[2].nw, EPI>>{});
  return go(Kernel<&k_dense_pair<64, 128, 2, 4, t[3].nx, t[3].nw, EPI>>{});
}

}  // namespace

// When n1 blocks of time c1, then n2 of time c2 <= c1, started in order as places come free, have all ended.
static double makespan(long long n1, double c1, long long n2, double c2, long long places) {
  const long long q = n1 / places, r = n1 % places;  // places - r come free at q c1, r at (q + 1) c1
  const double early = q * c1, late = r ? early + c1 : early;
  // the end is a whole number of c2 after early or after late
  auto first_end = [&](double from) {
    for (double end = from;; end += c2) {
      if (end < late) continue;
      const long long a = (long long)((end - early) / c2 + 1e-6), b = (long long)((end - late) / c2 + 1e-6);
      if (a * (places - r) + b * r >= n2) return end;
    }
  };
  const double x = first_end(early), y = first_end(late);
  return x < y ? x : y;
}

// Blocks reach an epilogue that moves many bytes together, at the memory's rate, unless others run beside them: its
// cost grows with b's share of the blocks at work. dw2 with the gradients of g and u, hidden 4096, intermediate 2048,
// in one launch against two of the products' best tiles: 255 against 289 us at 8192 tokens, 117 / 138 at 4096, 72 / 83
// at 2048, 30 / 37 at 512; dw13 with dx: 393 / 420, 199 / 204, 110 / 116 (at 6000 tokens 205 / 206: two launches).
DensePairPlan dense_pair_plan(int Ma, int Na, int Ka, int Mb, int Nb, int Kb, int epi_bytes) {
  DensePairPlan best;
  double ua, ub;
  best.a = dense_plan(kDenseBf16, kDenseTN, Ma, Na, Ka, &ua);
  best.b = dense_plan(kDenseBf16, kDenseNN, Mb, Nb, Kb, &ub);
  best.tile = -1;
  constexpr double kBytesPerUs = 5.1e6, kEpiUs = 2.1e-4;
  constexpr double kTwoLaunches = 1.07;  // measured over the sum of the estimates: 2 to 13 % more
  // the epilogue of a block of tile t, with `blocks` of them at a time: its bytes, or its arithmetic
  auto epi_us = [&](int t, double blocks) {
    const double values = (double)kTiles[t].bm * kTiles[t].bn, bytes = blocks * epi_bytes * values / kBytesPerUs;
    return !epi_bytes || bytes > kEpiUs * values ? bytes : kEpiUs * values;
  };
  double best_us = kTwoLaunches * (ua + ub) + epi_us(best.b.tile, (double)Mb * Nb / kTiles[best.b.tile].bm / kTiles[best.b.tile].bn);
  const int sa = stages_of(kDenseBf16, Ka), sb = stages_of(kDenseBf16, Kb);
  for (int t = kNumTiles - 1; t >= 0; --t) {
    const long long na = (long long)ceil_div(Ma, kTiles[t].bm) * ceil_div(Na, kTiles[t].bn);
    const long long nb = (long long)ceil_div(Mb, kTiles[t].bm) * ceil_div(Nb, kTiles[t].bn);
    // blocks at work at a time, over the longer product's stages
    const double n = ((double)na * sa + (double)nb * sb) / (sa > sb ? sa : sb), c = stage_us(t, n);
    const double ca = sa * c * kTnCost + kStartUs;
    const double cb = sb * c + kStartUs + epi_us(t, (n < places(t) ? n : places(t)) * nb / (double)(na + nb));
    const double us = sa > sb ? makespan(na, ca, nb, cb, places(t)) : makespan(nb, cb, na, ca, places(t));
    if (us < 0.97 * best_us) {  // near ties: separate, then the smaller tile, whose blocks mix better
      best_us = us;
      best.tile = t;
    }
  }
  return best;
}

hipError_t launch_dense_pair(int epi, const DensePairPlan& p, DenseArgs a, DenseArgs b, hipStream_t st) {
  if (p.tile < 0) {
    const hipError_t e = launch_dense(kDenseBf16, kDenseTN, kEpiStore, p.a, a, st);
    return e != hipSuccess ? e : launch_dense(kDenseBf16, kDenseNN, epi, p.b, b, st);
  }
  if (p.tile >= kNumTiles || (epi != kEpiStore && epi != kEpiGrad)) return hipErrorInvalidValue;
  const TileCfg& t = kTiles[p.tile];
  for (DenseArgs* x : {&a, &b}) {
    if (x->M <= 0 || x->N <= 0 || x->K <= 0) return hipErrorInvalidValue;
    x->stages = x->slice_stages = stages_of(kDenseBf16, x->K);
    x->tm = ceil_div(x->M, t.bm);
    x->tn = ceil_div(x->N, t.bn);
    if ((long long)x->tm * x->tn > 0x1fffff) return hipErrorInvalidValue;
  }
  return epi == kEpiGrad ? run_pair<kEpiGrad>(p.tile, a, b, st) : run_pair<kEpiStore>(p.tile, a, b, st);
}

hipError_t launch_dense_reduce(int epi, const DenseArgs& a, int slices, hipStream_t st) {
  const int cols = epi == kEpiGate ? a.I : a.N;
  const long long threads = (long long)a.M * ((cols + 3) / 4);
  const unsigned nb = (unsigned)((threads + 63) / 64);
  if (epi == kEpiGate) k_dense_reduce<kEpiGate><<<nb, 64, 0, st>>>(a, slices);
  else if (epi == kEpiGrad) k_dense_reduce<kEpiGrad><<<nb, 64, 0, st>>>(a, slices);
  else k_dense_reduce<kEpiStore><<<nb, 64, 0, st>>>(a, slices);
  return hipGetLastError();
}

}  // namespace moe

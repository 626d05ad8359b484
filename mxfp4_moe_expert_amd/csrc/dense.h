// Dense matrix products of the trainable gated block and of the plain MXFP4
// projections on gfx950's matrix cores: one kernel template,
//   C[m][n] = sum_k X(m, k) W(n, k),
// with each operand stored either along k ([row][k], "K-contiguous") or
// across it ([k][row], "transposed"), in bf16 or (both K-contiguous) MXFP4.
//
// Tile BM x BN, one block of WGM x WGN waves. K runs in stages of two MFMA
// k-steps (128 bytes per row: 64 bf16 or 256 E2M1 values); LDS holds NX stages
// of the X tile and NW of the W tile:
//   - Operands go from global memory straight to LDS (16 bytes per lane, the
//     64 lanes of a wave filling 1 KB), whole 128-byte lines at a time (half
//     lines cost as much L2 bandwidth as whole ones). The loads are raw
//     buffer loads whose out-of-range lanes (rows, columns or k past the end)
//     write zeros, so no tail needs code in the K loop.
//   - The MFMAs of a k-step run on operands already in registers, with the
//     LDS reads of the next k-step's operands and a share of a later stage's
//     loads spread between them: a burst of either stalls the waves (the
//     loads of a CU share one 64 B/clock path), and MFMAs behind a stalled
//     instruction do not issue. X is loaded in the first k-step and W in the
//     second; one barrier per stage, between them.
//   - The eight 16-byte pieces of a K-contiguous row i are stored at piece ^
//     (i / 2) % 8, so the 16 rows of an MFMA operand lie in different banks
//     (no conflicts counted in any product). A transposed operand keeps its
//     k rows; its 32-byte units are stored at unit ^ f(k), and the LDS
//     transposing read (16 lanes x 4 elements) hands each lane 4 consecutive
//     k of its row.
//   - MFMA 16x16x32 (bf16) or 16x16x128 with E8M0 scales (MXFP4), W as the A
//     operand: lane (r, g) ends with 4 consecutive n of one m; two blocks'
//     lanes are joined to 16-byte stores.
//
// Measured (MI355X; a large copy runs at 5.1 TB/s, a large library bf16
// product at 1.26 PFLOP/s): 8192 x 4096 x 4096, transposed W, 256 x 256 tiles
// 205 us, 1.34 PFLOP/s, matrix cores busy 64 % of the cycles; both transposed
// 205 us; 1000 x 4096 x 4096, 128 x 128: 34.7 us, 0.97; 300 x 4096 x 4096,
// 64 x 128: 22.7 us; MXFP4 8192 x 4096 x 4096: 72 to 76 us, 3.6 to 3.8
// PFLOP/s. Large tiles are bound by the MFMAs and, where a launch is one or
// two rounds of blocks, by epilogues that nothing covers (6.5 us a round of
// bf16 stores); the smaller ones by the L2 -> LDS path (a stage of 64 x 128
// takes 0.26 to 0.34 us, 128 x 128 0.32 to 0.47, 256 x 128 0.47 to 0.80, 256 x
// 256 0.95 to 1.45, with few and with all CUs at work). MXFP4 at 256 x 256 fills
// neither: a stage of 64 KB takes about 1.6 us (40 KB/us per CU, where the small
// tiles reach 70), its MFMAs about half of that. Its ring holds two stages, so
// each load is waited for one stage after its issue.
#pragma once

#include <atomic>
#include <type_traits>

#include "device.h"
#include "internal.h"

namespace moe {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((ext_vector_type(4))) short s16x4_t;
typedef __attribute__((address_space(3))) unsigned char lds_u8;
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
typedef __attribute__((address_space(3))) u32x4_t lds_u32x4;
typedef __attribute__((address_space(3))) uint32_t lds_u32;

constexpr uint32_t kLaneOff = 0x80000000u;  // a lane offset past every buffer: reads zero
constexpr int kStageB = 128;                // K bytes per row and stage
constexpr int kStageK = 64;                 // k rows of a transposed operand per stage

// 16 bytes per lane from buffer offset voff to LDS byte m0 + lane * 16.
// No output registers: the data is waited for with dense_wait before a barrier.
// (m0 is a reserved register: the compiler sets it right before each use of its own.)
__device__ __forceinline__ void load_lds16(u32x4_t rsrc, uint32_t voff, uint32_t lds_at) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane((int)lds_at)), "v"(voff), "s"(rsrc)
               : "memory");
}
// At most N of the wave's vector loads outstanding, and its LDS reads done.
template <int N>
__device__ __forceinline__ void dense_wait() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(N) : "memory");
}

__device__ __forceinline__ u32x4_t buffer_of(const void* p) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  return (u32x4_t){(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
                   (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xffffu)), 0x7fffffffu,
                   0x00027000u};
}

// Staging of one operand tile of ROWS rows (W waves). Rows past `rows` and k
// past `kb` (bytes along k, K-contiguous) or `kn` (k rows, transposed) read
// as zeros.
template <bool TR, int ROWS, int W>
struct Stager {
  static constexpr int NI = ROWS * kStageB / 1024 / W;  // 1 KB loads per wave and stage
  static constexpr int PPR = TR ? ROWS / 8 : 8;         // 16-byte pieces per stored row
  static_assert(W % 4 == 0 && (W * 64) % PPR == 0, "loads of a wave share their k offsets");
  uint32_t voff[NI];

  static __device__ __forceinline__ int slot(int i, int wave, int lane) { return (i * W + wave) * 64 + lane; }
  // the 16-byte piece that slot s holds of its stored row (row of the tile, or k row)
  static __device__ __forceinline__ int piece(int s) {
    const int row = s / PPR, pos = s % PPR;
    if constexpr (TR) {
      const int f = ((row & 3) | (((row >> 3) & 1) << 2)) & (ROWS / 16 - 1);
      return ((((pos >> 1) ^ f) << 1) | (pos & 1));
    } else {
      return pos ^ ((row >> 1) & 7);
    }
  }

  // row_of(i): the stored row of tile row i (K-contiguous), or -1 for none
  template <class F>
  __device__ __forceinline__ void init_kc(int wave, int lane, uint32_t ld, F row_of) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int s = slot(i, wave, lane);
      const int row = row_of(s / PPR);
      voff[i] = row < 0 ? kLaneOff : (uint32_t)row * ld + (uint32_t)piece(s) * 16;
    }
  }
  __device__ __forceinline__ void init_tr(int wave, int lane, uint32_t ld, int cols) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int s = slot(i, wave, lane);
      voff[i] = piece(s) * 8 < cols ? (uint32_t)(s / PPR) * ld + (uint32_t)piece(s) * 16 : kLaneOff;
    }
  }
  // Load i of a stage. kleft: bytes (K-contiguous) or k rows (transposed) from the stage's start to the end of k;
  // lanes past it read zeros. `at` is the lane's first k of load 0: the others differ by a constant.
  __device__ __forceinline__ void load(int i, u32x4_t rsrc, uint32_t lds_at, int wave, int at, int kleft) const {
    const int step = TR ? W * 64 / PPR : 0;  // K-contiguous: the piece is the same in every load (W % 4 == 0)
    load_lds16(rsrc, at < kleft - i * step ? voff[i] : kLaneOff, lds_at + (uint32_t)((i * W + wave) * 1024));
  }
  static __device__ __forceinline__ int first_k(int wave, int lane) {
    const int s = slot(0, wave, lane);
    return TR ? s / PPR : piece(s) * 16;
  }
};

// Reading MFMA operands of 16 tile rows from a staged tile.
template <bool TR, int ROWS, int NB>
struct Reader {
  // K-contiguous: offsets of the lane's piece for the two k-steps; transposed: one per row block
  uint32_t off[TR ? NB : 2];
  __device__ __forceinline__ void init(int row0, int lane) {
    const int r = lane & 15, g = lane >> 4;
    if constexpr (TR) {
      const int j = r >> 2, q = r & 3, f = (j | ((g & 1) << 2)) & (ROWS / 16 - 1);
#pragma unroll
      for (int b = 0; b < NB; ++b)
        off[b] = (uint32_t)((8 * g + j) * (ROWS * 2) + (((row0 >> 4) + b) ^ f) * 32 + q * 8);
    } else {
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
        off[kk] = (uint32_t)((row0 + r) * kStageB + (((kk * 4 + g) ^ (r >> 1)) * 16));
    }
  }
  __device__ __forceinline__ u32x4_t read(const lds_u8* tile, int b, int kk) const {
    if constexpr (TR) {
      const lds_u8* p = tile + off[b] + kk * 32 * (ROWS * 2);
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * (ROWS * 2)));
      const uint2 a = __builtin_bit_cast(uint2, lo), c = __builtin_bit_cast(uint2, hi);
      return (u32x4_t){a.x, a.y, c.x, c.y};
    } else {
      return *(const lds_u32x4*)(tile + off[kk] + b * (16 * kStageB));
    }
  }
};

__device__ __forceinline__ f32x4_t mfma_bf16(const u32x4_t& a, const u32x4_t& b, const f32x4_t& c) {
  return mfma_16x16x32(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c);
}
template <int KK>
__device__ __forceinline__ f32x4_t mfma_mx4(const u32x4_t& a, const u32x4_t& b, const f32x4_t& c, uint32_t sa,
                                            uint32_t sb) {
  const i32x8_t a8 = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8_t b8 = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, KK, (int)sa, KK, (int)sb);
}

__device__ __forceinline__ uint2 pack4_bf16(const f32x4_t& v) {
  return make_uint2(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]));
}

// Lane row g of a wave holds columns 4 g .. 4 g + 3 (8 bytes) of two 16-column blocks -> columns 8 g .. 8 g + 7 of the 32
// (16 bytes), so that a store covers 64 consecutive bytes of each of 16 rows.
__device__ __forceinline__ u32x4_t join_blocks(const uint2& p, const uint2& q) {
  const auto a = __builtin_amdgcn_permlane32_swap(p.x, q.x, false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(p.y, q.y, false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], a[1], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(b[0], b[1], false, false);
  return (u32x4_t){c[0], d[0], c[1], d[1]};
}
// Four consecutive outputs out[at .. at+3], of which `live` (1..4) exist;
// wide: at is a multiple of 4 elements and all four exist.
__device__ __forceinline__ void store4(void* out, bool fp32, size_t at, const f32x4_t& v, int live, bool wide) {
  if (fp32) {
    float* o = static_cast<float*>(out) + at;
    if (wide) {
      *reinterpret_cast<f32x4_t*>(o) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < live) o[i] = v[i];
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(out) + at;
    if (wide) {
      *reinterpret_cast<uint2*>(o) = pack4_bf16(v);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < live) o[i] = f32_to_bf16(v[i]);
    }
  }
}

// min(v, L) and clamp(v, -L, L), one and two instructions; NaN stays NaN.
__device__ __forceinline__ float at_most(float v, float L) { return __builtin_elementwise_minimum(v, L); }
__device__ __forceinline__ float clamped(float v, float L) { return __builtin_elementwise_maximum(at_most(v, L), -L); }

// h = silu(min(g, L)) * clamp(u, -L, L); NaN operands give NaN.
__device__ __forceinline__ float ffn_act(float g, float u, float L) { return silu(at_most(g, L)) * clamped(u, L); }

// Gradients of the gated product at the saved (g, u) for dh, four columns: with s = sigmoid(g) and t = silu(g) = g s,
// du = dh t and dg = dh u (s + t (1 - s)). 1 - s is taken first: it is exact from s = 1/2 on and 0 where s is 1, so no
// part of a large t is left over (as s + t - t s, 1 is lost beside a t of 2^24 and more).
// Few instructions count here: where all blocks of a launch end together, a
// 256 x 256 tile's 128 exponentials and reciprocals per lane are bare (14 us of a launch; 17 with clamps by comparison).
// g and u are saved in fp32: rounded to bf16 they would cost the gradients as much precision again as the rounding of
// dg and du (relative L2 error of dx 3.0e-3 against 2.4e-3), and a value next to the clamp could cross it.
__device__ __forceinline__ void ffn_act_grad4(const f32x4_t& g4, const f32x4_t& u4, const f32x4_t& dh, float L,
                                              f32x4_t& dg, f32x4_t& du) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float gc = at_most(g4[i], L);
    const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-gc * 1.4426950408889634f));
    const float t = gc * s;
    dg[i] = g4[i] > L ? 0.0f : dh[i] * clamped(u4[i], L) * __builtin_fmaf(t, 1.0f - s, s);
    du[i] = __builtin_fabsf(u4[i]) > L ? 0.0f : dh[i] * t;
  }
}

// The wave's accumulators to out [M][N]: lane (r, g) holds acc[b][c][i] = C[m0 + 16 c + r][n0 + 16 b + 4 g + i].
template <int MB, int NB>
__device__ __forceinline__ void store_tile(const f32x4_t (&acc)[NB][MB], void* out, bool fp32, int M, int N, int m0,
                                           int n0, int lane) {
  const int r = lane & 15, g = lane >> 4;
  // 16-byte pieces of bf16 rows exist whole or not at all
  const bool joined = NB % 2 == 0 && !fp32 && (N & 7) == 0;
#pragma unroll
  for (int c = 0; c < MB; ++c) {
    const int m = m0 + c * 16 + r;
    if (joined) {
      uint16_t* row = static_cast<uint16_t*>(out) + (size_t)m * N;
#pragma unroll
      for (int b = 0; b + 1 < NB; b += 2) {
        const int n = n0 + b * 16 + 8 * g;
        const u32x4_t v = join_blocks(pack4_bf16(acc[b][c]), pack4_bf16(acc[b + 1][c]));
        if (m < M && n < N) *reinterpret_cast<u32x4_t*>(row + n) = v;
      }
    } else if (m < M) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int n = n0 + b * 16 + 4 * g;
        if (n >= N) continue;
        store4(out, fp32, (size_t)m * N + n, acc[b][c], N - n, (N & 3) == 0);
      }
    }
  }
}

enum DenseEpi {
  kEpiStore = 0,    // out [M][N] bf16 or fp32
  kEpiGate = 1,     // gate / up rows interleaved: h [M][I] bf16 (and gu [M][2I] fp32)
  kEpiGrad = 2,     // dh -> dgu [M][2I] from gu
  kEpiPartial = 3,  // fp32 partial sums [slice][M][N] (of a split K)
};

// Of n operations spread evenly over nm places: how many are done by place m (at m < 0: none).
__device__ constexpr int spread(int m, int nm, int n) {
  return m < 0 ? 0 : (m * n / nm + 1 < n ? m * n / nm + 1 : n);
}

// Logical tile of a block: XCD x (block % 8) walks a contiguous run of the
// tiles, ordered in bands of 8 row tiles, so that the tiles an XCD's blocks
// run at once share operand rows in its L2.
__device__ __forceinline__ void dense_tile(int bid, int tm, int tn, int& im, int& in) {
  const int n = tm * tn, per = n >> 3, extra = n & 7, x = bid & 7;
  const int t = x * per + min(x, extra) + (bid >> 3);
  constexpr int BAND = 8;
  const int band = t / (BAND * tn), left = tm - band * BAND;
  const int h = left < BAND ? left : BAND;
  const int o = t - band * BAND * tn;
  im = band * BAND + o % h;
  in = o / h;
}

// The LDS rings of a tile and the loads that fill them: NX stages of X, NW of W, then (MXFP4) NS sets of the packed
// scales of two stages (see mxfp4.hip). Past the slice's stages a load writes zeros, so that every stage has its loads
// and the waits can count them.
template <bool XT, bool WT, int BM, int BN, int W, int NX, int NW, bool FP4, int NS, bool GATE>
struct TileLoads {
  static constexpr int XB = BM * kStageB, WB = BN * kStageB;              // bytes per stage
  static constexpr int SXB = FP4 ? BM * 16 : 0, SWB = FP4 ? BN * 16 : 0;  // scales of two stages
  static constexpr uint32_t WBASE = NX * XB, SCALES = WBASE + NW * WB, SCB = SXB + SWB;
  using SX = Stager<XT, BM, W>;
  using SW = Stager<WT, BN, W>;
  static constexpr int LX = SX::NI, LW = SW::NI;  // loads per wave and stage
  static_assert(LX * 1024 * W == XB && LW * 1024 * W == WB, "tiles split evenly over the waves");
  static_assert(!FP4 || (!XT && !WT), "MXFP4 operands are K-contiguous");
  // Where the next stage of one operand comes from and goes to. Past the slice kleft is 0 or less: every lane is out of
  // range and nothing is read.
  struct Feed {
    const char* src;
    int kleft;    // bytes (K-contiguous) or k rows (transposed) from the stage's start to the slice's end
    uint32_t at;  // ring place, LDS bytes
  };

  SX sx;
  SW sw;
  Feed fx, fw;
  size_t xstep, wstep;
  int xat, wat;
  uint32_t lds0;
  int wave, lane, st0, nst, im, in;

  __device__ __forceinline__ void init(const DenseArgs& a, uint32_t lds, int wave_, int lane_, int im_, int in_) {
    lds0 = lds;
    wave = wave_;
    lane = lane_;
    im = im_;
    in = in_;
    st0 = blockIdx.y * a.slice_stages;
    nst = min(a.slice_stages, a.stages - st0);
    const int m0 = im * BM, n0 = in * (GATE ? BN / 2 : BN);
    const int kb = a.K * 2 / (FP4 ? 4 : 1);  // bytes along k (K-contiguous operands)
    const char *xbase = static_cast<const char*>(a.x), *wbase = static_cast<const char*>(a.w);
    if constexpr (XT) {
      sx.init_tr(wave, lane, a.x_ld, a.M - m0);
      xbase += (size_t)m0 * 2;
    } else {
      sx.init_kc(wave, lane, a.x_ld, [&](int i) { return m0 + i < a.M ? i : -1; });
      xbase += (size_t)m0 * a.x_ld;
    }
    if constexpr (WT) {
      sw.init_tr(wave, lane, a.w_ld, a.N - n0);
      wbase += (size_t)n0 * 2;
    } else if constexpr (GATE) {
      // tile rows: 16 gate rows, then the matching 16 up rows, and so on
      sw.init_kc(wave, lane, a.w_ld, [&](int i) {
        const int c = n0 + (i >> 5) * 16 + (i & 15);
        return c < a.I ? ((i >> 4) & 1) * a.I + c : -1;
      });
    } else {
      sw.init_kc(wave, lane, a.w_ld, [&](int i) { return n0 + i < a.N ? i : -1; });
      wbase += (size_t)n0 * a.w_ld;
    }
    xstep = XT ? (size_t)kStageK * a.x_ld : kStageB;
    wstep = WT ? (size_t)kStageK * a.w_ld : kStageB;
    xat = SX::first_k(wave, lane);
    wat = SW::first_k(wave, lane);
    constexpr int xk = XT ? kStageK : kStageB, wk = WT ? kStageK : kStageB;
    const int end = st0 + nst;  // K up to the slice's end
    fx = {xbase + (size_t)st0 * xstep, min(XT ? a.K : kb, end * xk) - st0 * xk, lds0};
    fw = {wbase + (size_t)st0 * wstep, min(WT ? a.K : kb, end * wk) - st0 * wk, lds0 + WBASE};
  }
  // The loads 0 .. LX - 1 (LW - 1) of the next stage, then the step to the one after it
  __device__ __forceinline__ void load_x(int op) const { sx.load(op, buffer_of(fx.src), fx.at, wave, xat, fx.kleft); }
  __device__ __forceinline__ void load_w(int op) const { sw.load(op, buffer_of(fw.src), fw.at, wave, wat, fw.kleft); }
  __device__ __forceinline__ void next_x() {
    fx.src += xstep;
    fx.kleft -= XT ? kStageK : kStageB;
    fx.at = fx.at == lds0 + (NX - 1) * XB ? lds0 : fx.at + XB;
  }
  __device__ __forceinline__ void next_w() {
    fw.src += wstep;
    fw.kleft -= WT ? kStageK : kStageB;
    fw.at = fw.at == lds0 + WBASE + (NW - 1) * WB ? lds0 + WBASE : fw.at + WB;
  }
  // The scales of stages i and i + 1, i even: [two stages][16-row block][lane] u32, the tile's blocks contiguous
  __device__ __forceinline__ void load_scales(const DenseArgs& a, int i) const {
    const bool live = i < nst;
    const size_t pr = live ? (size_t)((st0 + i) >> 1) : 0;
    const u32x4_t rx = buffer_of(a.x_scales + (pr * a.x_blocks + (size_t)im * (BM / 16)) * 64);
    const u32x4_t rw = buffer_of(a.w_scales + (pr * a.w_blocks + (size_t)in * (BN / 16)) * 64);
    const uint32_t endx = (uint32_t)(a.x_blocks - im * (BM / 16)) * 256;
    const uint32_t endw = (uint32_t)(a.w_blocks - in * (BN / 16)) * 256;
    for (uint32_t o = (uint32_t)wave * 1024; o < SCB; o += W * 1024) {  // byte of the set
      const bool isw = o >= SXB;
      const uint32_t off = (isw ? o - SXB : o) + (uint32_t)lane * 16;
      load_lds16(isw ? rw : rx, live && off < (isw ? endw : endx) ? off : kLaneOff,
                 lds0 + SCALES + (uint32_t)((i >> 1) % NS) * SCB + o);
    }
  }
};

// What a wave does with its sums: lane (r, g) holds acc[b][c][i] = C[m0 + 16 c + r][n0 + 16 b + 4 g + i] (gate: blocks b
// alternate between gate and up, n0 is the first h column).
template <int EPI, int MB, int NB>
__device__ __forceinline__ void dense_epilogue(const DenseArgs& a, const f32x4_t (&acc)[NB][MB], int m0, int n0,
                                               int lane) {
  if constexpr (EPI == kEpiStore || EPI == kEpiPartial) {
    void* out = EPI == kEpiPartial ? static_cast<void*>(a.part + (size_t)blockIdx.y * a.M * a.N) : a.out;
    store_tile<MB, NB>(acc, out, EPI == kEpiPartial || a.out_is_fp32, a.M, a.N, m0, n0, lane);
    return;
  }
  // N and I are multiples of 8: 16-byte pieces exist whole or not at all
  const int r = lane & 15, g = lane >> 4;
  auto put = [&](uint16_t* p, const u32x4_t& v, bool live) {
    if (live) *reinterpret_cast<u32x4_t*>(p) = v;
  };
  if constexpr (EPI == kEpiGate) {
#pragma unroll
    for (int c = 0; c < MB; ++c) {
      const int m = m0 + c * 16 + r;
      uint16_t* hrow = static_cast<uint16_t*>(a.out) + (size_t)m * a.I;
      auto act = [&](int b) {
        f32x4_t h;
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = ffn_act(acc[b][c][i], acc[b + 1][c][i], a.limit);
        return pack4_bf16(h);
      };
      if constexpr (NB % 4 == 0) {
#pragma unroll
        for (int b = 0; b < NB; b += 4) {
          const int n = n0 + b * 8 + 8 * g;  // h column
          put(hrow + n, join_blocks(act(b), act(b + 2)), m < a.M && n < a.I);
        }
      } else {
#pragma unroll
        for (int b = 0; b < NB; b += 2) {
          const int n = n0 + b * 8 + 4 * g;
          if (m < a.M && n < a.I) *reinterpret_cast<uint2*>(hrow + n) = act(b);
        }
      }
      if (a.gu_out) {
        float* grow = a.gu_out + (size_t)m * 2 * a.I;
#pragma unroll
        for (int b = 0; b < NB; b += 2) {
          const int n = n0 + b * 8 + 4 * g;
          if (m >= a.M || n >= a.I) continue;
          *reinterpret_cast<f32x4_t*>(grow + n) = acc[b][c];
          *reinterpret_cast<f32x4_t*>(grow + a.I + n) = acc[b + 1][c];
        }
      }
    }
  } else {
    // g and u of the next 16 rows are fetched before this one's stores, which the compiler may not move loads across
    f32x4_t gv[2][NB], uv[2][NB];
    auto fetch = [&](int c) {  // past the edges: the last row, the first column (never stored)
      const float* s = a.gu_in + (size_t)min(m0 + c * 16 + r, a.M - 1) * 2 * a.I;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int n = n0 + b * 16 + 4 * g, col = n < a.N ? n : 0;
        gv[c & 1][b] = *reinterpret_cast<const f32x4_t*>(s + col);
        uv[c & 1][b] = *reinterpret_cast<const f32x4_t*>(s + a.I + col);
      }
    };
    fetch(0);
#pragma unroll
    for (int c = 0; c < MB; ++c) {
      if (c + 1 < MB) fetch(c + 1);
      const int m = m0 + c * 16 + r;
      uint16_t* o = static_cast<uint16_t*>(a.out) + (size_t)m * 2 * a.I;
#pragma unroll
      for (int b = 0; b < NB; b += 2) {
        uint2 dgv[2], duv[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          f32x4_t dg, du;
          ffn_act_grad4(gv[c & 1][b + j], uv[c & 1][b + j], acc[b + j][c], a.limit, dg, du);
          dgv[j] = pack4_bf16(dg);
          duv[j] = pack4_bf16(du);
        }
        const int n = n0 + b * 16 + 8 * g;
        const bool live = m < a.M && n < a.N;
        put(o + n, join_blocks(dgv[0], dgv[1]), live);
        put(o + a.I + n, join_blocks(duv[0], duv[1]), live);
      }
    }
  }
}

// One tile (block `bid` of the product's a.tm a.tn) of the product. FP4: both operands MXFP4 K-contiguous, with packed
// scales.
template <bool XT, bool WT, int BM, int BN, int WGM, int WGN, int NX, int NW, bool FP4, int EPI>
__device__ __forceinline__ void dense_block(const DenseArgs& a, int bid) {
  constexpr int W = WGM * WGN;
  constexpr int MB = BM / WGM / 16, NB = BN / WGN / 16;  // 16-row blocks per wave
  // scales are loaded SD pairs of stages ahead, so that the waits below cover them
  constexpr int SD = NW <= 2 ? 1 : (NW + 1) / 2 - (NW & 1);
  using L = TileLoads<XT, WT, BM, BN, W, NX, NW, FP4, SD + 1, EPI == kEpiGate>;
  constexpr int XB = L::XB, WB = L::WB, LX = L::LX, LW = L::LW;
  constexpr uint32_t WBASE = L::WBASE;
  static_assert(2 * SD - 1 >= NW - 2, "a stage's scales land with it");
  static_assert(NW >= 2 && (NX == NW || NX == NW + 1), "the waits below assume it");
  // X is loaded in the first k-step; with two stages of both, a load there would be waited for in the same stage, and
  // both operands are loaded in the second
  constexpr bool XK0 = NX > NW || NW > 2;
  extern __shared__ __align__(16) unsigned char smem[];
  lds_u8* const lds = (lds_u8*)smem;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int im, in;
  dense_tile(bid, a.tm, a.tn, im, in);
  L t;
  t.init(a, (uint32_t)(uintptr_t)lds, wave, lane, im, in);
  const int nst = t.nst;

  const int wm = wave / WGN, wn = wave % WGN;
  Reader<XT, BM, MB> rx;
  Reader<WT, BN, NB> rw;
  rx.init(wm * MB * 16, lane);
  rw.init(wn * NB * 16, lane);

  f32x4_t acc[NB][MB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int c = 0; c < MB; ++c) acc[b][c] = (f32x4_t){0.f, 0.f, 0.f, 0.f};

  // Registers: the W operands of this k-step and the next; of the X operands the first half once (xr[c] is read again,
  // for the next k-step, after its last MFMA of this one) and the second half twice, so that every read of a k-step is
  // issued by the middle of the one before.
  constexpr int XR = MB / 2;
  u32x4_t xr[XR], xd[2][MB - XR], wf[2][NB];
  uint32_t sxv[MB], swv[NB];  // MXFP4: the lane's scale bytes of two stages, one per k-step
  auto read_scales = [&](int i) {
    const lds_u8* sc = lds + L::SCALES + (uint32_t)((i >> 1) % (SD + 1)) * L::SCB;
#pragma unroll
    for (int c = 0; c < MB; ++c) sxv[c] = *(const lds_u32*)(sc + ((wm * MB + c) * 64 + lane) * 4);
#pragma unroll
    for (int b = 0; b < NB; ++b) swv[b] = *(const lds_u32*)(sc + L::SXB + ((wn * NB + b) * 64 + lane) * 4);
  };
  // The MFMAs of k-step kk (parity q of its stage), reading the next k-step's operands from the tiles xt and wt and
  // issuing the loads load(0) .. load(nload - 1). The order is pinned, or the compiler gathers the memory operations.
  auto step = [&](auto kk, auto q, const lds_u8* xt, const lds_u8* wt, auto nload, auto&& load, auto&& next) {
    constexpr int NM = MB * NB, NR = NB + MB - XR;
    // the loads' places; then the sources move on, in the shadow of the last MFMAs
    constexpr int NP = XK0 ? NM * 3 / 4 : NM - 2;
    static_assert(nload <= NP, "one load per MFMA at most");
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      const int c = m / NB, b = m % NB;
      const u32x4_t& x = c < XR ? xr[c < XR ? c : 0] : xd[kk][c < XR ? 0 : c - XR];
      if constexpr (FP4) acc[b][c] = mfma_mx4<kk + 2 * q>(wf[kk][b], x, acc[b][c], swv[b], sxv[c]);
      else acc[b][c] = mfma_bf16(wf[kk][b], x, acc[b][c]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = spread(m - 1, NP, nload); i < spread(m, NP, nload); ++i) load(i);
      if (m == NP) next();
#pragma unroll
      for (int i = spread(2 * m - 2, NM, NR); i < spread(2 * m, NM, NR); ++i) {
        if (i < NB) wf[1 - kk][i] = rw.read(wt, i, 1 - kk);
        else xd[1 - kk][i - NB] = rx.read(xt, i - NB + XR, 1 - kk);
      }
      if (b == NB - 1 && c < XR) xr[c < XR ? c : 0] = rx.read(xt, c, 1 - kk);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  using K0 = std::integral_constant<int, 0>;
  using K1 = std::integral_constant<int, 1>;

  // Loads in order X(0) W(0) X(1) W(1) ..., as the loop continues it
  if constexpr (FP4) {
#pragma unroll
    for (int d = 0; d < SD; ++d) t.load_scales(a, 2 * d);
  }
#pragma unroll
  for (int i = 0; i < (NX > NW ? NX : NW); ++i) {
    if (i < (XK0 ? NX - 1 : NX)) {
#pragma unroll
      for (int op = 0; op < LX; ++op) t.load_x(op);
      t.next_x();
    }
    if (i < NW) {
#pragma unroll
      for (int op = 0; op < LW; ++op) t.load_w(op);
      t.next_w();
    }
  }
  dense_wait<(XK0 ? NX - 2 : NX - 1) * LX + (NW - 1) * LW>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int b = 0; b < NB; ++b) wf[0][b] = rw.read(lds + WBASE, b, 0);
#pragma unroll
  for (int c = 0; c < MB; ++c) (c < XR ? xr[c] : xd[0][c - XR]) = rx.read(lds, c, 0);
  int bx = 0, bw = 0;  // buffers of stage i
  auto stage = [&](int i, auto q) {
    if constexpr (FP4 && q == 0) read_scales(i);
    const int nx = bx + 1 == NX ? 0 : bx + 1, nw = bw + 1 == NW ? 0 : bw + 1;
    if constexpr (XK0) {  // X of stage i - 1 + NX, where stage i - 1 was
      step(K0{}, q, lds + bx * XB, lds + WBASE + bw * WB, std::integral_constant<int, LX>{},
           [&](int op) { t.load_x(op); }, [&]() { t.next_x(); });
    } else {
      step(K0{}, q, lds + bx * XB, lds + WBASE + bw * WB, K0{}, [](int) {}, []() {});
    }
    // stage i + 1 has landed (this wave's part) and this wave has read stage i, then every wave
    dense_wait<(NW - 2) * (LX + LW) + (NX > NW ? LX : 0)>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if constexpr (FP4 && q == 0) t.load_scales(a, i + 2 * SD);
    if constexpr (XK0) {
      step(K1{}, q, lds + nx * XB, lds + WBASE + nw * WB, std::integral_constant<int, LW>{},
           [&](int op) { t.load_w(op); }, [&]() { t.next_w(); });
    } else {
      step(K1{}, q, lds + nx * XB, lds + WBASE + nw * WB, std::integral_constant<int, LX + LW>{},
           [&](int op) {
             if (op < LX) t.load_x(op);
             else t.load_w(op - LX);
           },
           [&]() {
             t.next_x();
             t.next_w();
           });
    }
    bx = nx;
    bw = nw;
  };
  if constexpr (FP4) {
    for (int i = 0; i < nst; i += 2) {
      stage(i, K0{});
      if (i + 1 < nst) stage(i + 1, K1{});
    }
  } else {
    for (int i = 0; i < nst; ++i) stage(i, K0{});
  }
  dense_wait<0>();  // nothing may still write this block's LDS when it ends
  dense_epilogue<EPI, MB, NB>(a, acc, im * BM + wm * MB * 16,
                              EPI == kEpiGate ? in * (BN / 2) + wn * NB * 8 : in * BN + wn * NB * 16, lane);
}

template <bool XT, bool WT, int BM, int BN, int WGM, int WGN, int NX, int NW, bool FP4, int EPI>
__global__ __launch_bounds__(WGM* WGN * 64) void k_dense(DenseArgs a) {
  dense_block<XT, WT, BM, BN, WGM, WGN, NX, NW, FP4, EPI>(a, blockIdx.x);
}

// Two independent products in one launch: the weight gradient `a` (both operands transposed) and a product `b` with W
// transposed. One's blocks come first, the other's from block `second` on (a multiple of 8, so that blocks keep their
// XCDs). Blocks start in order: the product with the longer K goes first, and the other's blocks fill up behind it.
template <int BM, int BN, int WGM, int WGN, int NX, int NW, int EPI>
__global__ __launch_bounds__(WGM* WGN * 64) void k_dense_pair(DenseArgs a, DenseArgs b, int second, int b_first) {
  const int in_first = (int)blockIdx.x < second;
  const int bid = in_first ? (int)blockIdx.x : (int)blockIdx.x - second;
  if (in_first != b_first) {
    if (bid < a.tm * a.tn) dense_block<true, true, BM, BN, WGM, WGN, NX, NW, false, kEpiStore>(a, bid);
  } else {
    if (bid < b.tm * b.tn) dense_block<false, true, BM, BN, WGM, WGN, NX, NW, false, EPI>(b, bid);
  }
}

// Allows KERNEL `bytes` of dynamic LDS on the current device, asking the runtime once per device and kernel (the call
// is not needed again, and costs a small product part of its time).
template <auto KERNEL>
inline hipError_t allow_lds(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(KERNEL), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// A kernel as a value that a function can take.
template <auto KERNEL>
struct Kernel {
  static constexpr auto value = KERNEL;
};

}  // namespace moe

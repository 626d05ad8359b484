// The router's training operators on gfx950: the balance loss of a routed
// batch with its per-expert counts, and the gradient of the logits.
//
// With scores s = sqrt(softplus(z)) of token t's logits z (route.hip), shares
// p_te = s_te / sum_j s_tj, and per sequence q of n_q tokens c_qe slots on
// expert e:
//   f_qe = c_qe E / (k n_q),  P_qe = (1 / n_q) sum_t p_te,
//   loss = alpha / Q sum_q sum_e f_qe P_qe   (Q sequences that are not empty).
// The counts pass no gradient. With g_qe = alpha f_qe / (Q n_q),
//   d loss / d s_te = (g_qe - sum_j g_qj p_tj) / sum_j s_tj,
// and from the routing weights w_tj = scale s_j / N, N = sum_i s_i over the
// token's k slots, dw_tj given:
//   d s_j += scale (dw_j - sum_i dw_i s_i / N) / N   for each slot's expert,
//   dz = ds sigmoid(z) / (2 s).
//
// Forward: a block takes a run of tokens and, for each sequence in it, adds the
// shares of its tokens in registers (a group of G lanes per token, four experts
// per lane), then over the block in LDS, and writes one partial row per (run,
// sequence). A second launch adds each sequence's partial rows in order and the
// losses of the sequences in order: results do not depend on timing. Backward:
// one pass over the logits.
#include <type_traits>

#include "device.h"
#include "internal.h"

namespace moe {

namespace {

constexpr int kBalWaves = 16, kBalThreads = kBalWaves * 64;
constexpr int kBalRuns = 256;    // runs of tokens at most: one block per CU
constexpr int kBalRunMin = 32;

// h = exp(-|z| / 2), one hardware exponential. Above, e = h h = exp(-|z|): softplus(z) = max(z, 0) + log1p(e), with
// log1p(e) = log(1 + e) + what 1 + e lost of e (exact; it matters where e is small, and there its slope is 1). Below
// z = -17, softplus is e and its root h to fp32's last place, for every z down to where h itself ends.
struct Score {
  float h, e, sp, s;
};
__device__ __forceinline__ Score score_of(float z) {
  Score v;
  v.h = __builtin_amdgcn_exp2f(__builtin_fabsf(z) * -0.72134752044448170f);
  v.e = v.h * v.h;
  const float u = 1.0f + v.e;
  v.sp = fmaxf(z, 0.0f) + __builtin_fmaf(__builtin_amdgcn_logf(u), 0.69314718055994531f, v.e - (u - 1.0f));
  v.s = z < -17.0f ? v.h : __builtin_amdgcn_sqrtf(v.sp);
  return v;
}
// ds/dz = sigmoid(z) / (2 s)
__device__ __forceinline__ float score_slope(float z, const Score& v) {
  const float sig = (z < 0.0f ? v.e : 1.0f) * __builtin_amdgcn_rcpf(1.0f + v.e);
  return z < -17.0f ? 0.5f * v.h : 0.5f * sig * __builtin_amdgcn_rsqf(v.sp);
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// A token's four logits of lane l of its group; experts past E as -inf (score 0).
template <bool VEC>
__device__ __forceinline__ f32x4_t four_logits(const float* row, int l, int E) {
  f32x4_t z;
  if constexpr (VEC) {
    const bool in = 4 * l < E;
    z = *reinterpret_cast<const f32x4_t*>(row + (in ? 4 * l : 0));
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = in ? z[i] : -__builtin_inff();
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = 4 * l + i < E ? row[4 * l + i] : -__builtin_inff();
  }
  return z;
}

// Offsets come from the caller: used within [0, T]. Without any, one sequence of all tokens.
__device__ __forceinline__ int offset_of(const BalanceArgs& a, int q) {
  return a.offsets ? min(max(a.offsets[q], 0), a.T) : q > 0 ? a.T : 0;
}
// The last sequence that starts at or before t (-1: none).
__device__ __forceinline__ int sequence_of(const BalanceArgs& a, int t) {
  int lo = 0, hi = a.S;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (offset_of(a, mid) <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo - 1;
}

template <int G, bool VEC>
__global__ __launch_bounds__(kBalThreads) void k_balance_runs(BalanceArgs a) {
  constexpr int TPW = 64 / G, NG = kBalWaves * TPW;  // tokens per wave and block at a time
  __shared__ __align__(16) float red[kBalWaves][256];
  __shared__ int hist[256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l = lane & (G - 1);
  const int group = wave * TPW + lane / G;
  if (blockIdx.x == 0) {  // for the next launch
    if (tid < a.E) a.counts[tid] = 0;
    if (tid == 0) *a.ticket = 0;
  }
  const int t0 = blockIdx.x * a.run, t1 = min(t0 + a.run, a.T);
  int q = max(sequence_of(a, t0), 0);
  for (int t = t0; t < t1 && q < a.S; ++q) {
    const int first = max(t, offset_of(a, q)), end = min(t1, offset_of(a, q + 1));
    if (first >= end) continue;
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
    constexpr int U = 4;  // tokens whose logits are in flight together
    for (int b = first + group; b < end; b += U * NG) {
      f32x4_t z[U];
#pragma unroll
      for (int u = 0; u < U; ++u) z[u] = four_logits<VEC>(a.logits + (size_t)min(b + u * NG, end - 1) * a.E, l, a.E);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        f32x4_t s;
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = score_of(z[u][i]).s;
        const float total = group_sum<G>((s[0] + s[1]) + (s[2] + s[3]));
        // a row whose scores are all 0 has no shares
        const float inv = b + u * NG < end && total != 0.0f ? 1.0f / total : 0.0f;
        if (b + u * NG < end) sum += s * inv;
      }
    }
    *reinterpret_cast<f32x4_t*>(&red[wave][lane * 4]) = sum;
    for (int i = first * a.k + tid; i < end * a.k; i += kBalThreads) {
      const int e = a.ids[i];
      if ((unsigned)e < (unsigned)a.E) atomicAdd(&hist[e], 1);
      else if (a.flags) atomicOr(a.flags, kFlagExpertId);
    }
    __syncthreads();
    if (tid < a.E) {
      float v = 0.0f;
#pragma unroll 8
      for (int w = 0; w < NG; ++w) v += red[w / TPW][(w % TPW) * (4 * G) + tid];
      const size_t at = (size_t)(blockIdx.x + q) * a.E + tid;
      a.part_sum[at] = v;
      a.part_count[at] = hist[tid];
    }
    __syncthreads();
    t = end;
  }
}

// Sum over the block in a fixed order; every thread has the result.
__device__ __forceinline__ float block_sum(float v, float* lds) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < kBalWaves; ++w) s += lds[w];
  return s;
}

// Block q: sequence q's partial rows -> its loss, its coefficients (alpha f / n; 1 / Q follows them) and its counts; the
// last block to end adds the sequences' losses.
__global__ __launch_bounds__(kBalThreads) void k_balance_fold(BalanceArgs a) {
  constexpr int SUB = kBalThreads / 256;
  __shared__ float psum[SUB][256], lds[kBalWaves];
  __shared__ int pcount[SUB][256], last;
  const int tid = threadIdx.x, e = tid & 255, sub = tid >> 8, q = blockIdx.x;
  const int b = offset_of(a, q), end = offset_of(a, q + 1), n = end - b;
  bool bad = false;
  if (a.offsets) {
    const int lo = a.offsets[q], hi = a.offsets[q + 1];
    bad = lo < 0 || hi < lo || hi > a.T;
    if (bad && tid == 0 && a.flags) atomicOr(a.flags, kFlagSequence);
  }
  float sum = 0.0f;
  int count = 0;
  if (n > 0 && e < a.E) {
    const int r0 = b / a.run, r1 = (end - 1) / a.run;
    const float* ps = a.part_sum + (size_t)q * a.E + e;
    const int* pc = a.part_count + (size_t)q * a.E + e;
    constexpr int AHEAD = 8;
    for (int r = r0 + sub; r <= r1; r += SUB * AHEAD) {
      float v[AHEAD];
      int c[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const size_t at = (size_t)min(r + i * SUB, r1) * a.E;
        v[i] = ps[at];
        c[i] = pc[at];
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (r + i * SUB > r1) continue;
        sum += v[i];
        count += c[i];
      }
    }
  }
  psum[sub][e] = sum;
  pcount[sub][e] = count;
  __syncthreads();
  float loss = 0.0f;
  if (sub == 0 && e < a.E) {
#pragma unroll
    for (int i = 1; i < SUB; ++i) {
      sum += psum[i][e];
      count += pcount[i][e];
    }
    const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
    const float f = (float)count * ((float)a.E / (float)a.k) * inv;
    loss = f * (sum * inv);
    a.coef[(size_t)q * a.E + e] = a.alpha * f * inv;
    if (count) atomicAdd(&a.counts[e], count);
  }
  loss = block_sum(loss, lds);
  if (bad) loss = __uint_as_float(0x7fc00000u);
  if (tid == 0) {
    __hip_atomic_store(&a.seq_loss[q], loss, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __threadfence();
    last = atomicAdd(a.ticket, 1) == a.S - 1;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  float total = 0.0f, live = 0.0f;
  for (int i = tid; i < a.S; i += kBalThreads) {
    total += __hip_atomic_load(&a.seq_loss[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    live += offset_of(a, i + 1) > offset_of(a, i) ? 1.0f : 0.0f;
  }
  total = block_sum(total, lds);
  live = fmaxf(block_sum(live, lds), 1.0f);
  if (tid == 0) {
    *a.loss = a.alpha * total / live;
    a.coef[(size_t)a.S * a.E] = 1.0f / live;
  }
}

// The gradient of the logits. A group of G lanes takes the tokens of a run one after another.
constexpr int kGradWaves = 4;

template <int G, bool VEC, bool DW>
__global__ __launch_bounds__(kGradWaves * 64) void k_route_backward(BalanceArgs a, int per_group) {
  constexpr int TPW = 64 / G;
  const int lane = threadIdx.x & 63, l = lane & (G - 1);
  const long long group = ((long long)blockIdx.x * kGradWaves + (threadIdx.x >> 6)) * TPW + lane / G;
  const int t0 = (int)min(group * per_group, (long long)a.T), t1 = min(t0 + per_group, a.T);
  const float lead = a.coef ? a.coef[(size_t)a.S * a.E] * (a.dloss ? *a.dloss : 1.0f) : 0.0f;
  int q = t0 < t1 ? sequence_of(a, t0) : a.S, begin = 0, end = 0;  // tokens [begin, end) are sequence q's
  if (q < 0) q = 0;
  f32x4_t g = {0.f, 0.f, 0.f, 0.f};
  auto enter = [&]() {
    begin = offset_of(a, q);
    end = offset_of(a, q + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      g[i] = a.coef && 4 * l + i < a.E ? a.coef[(size_t)q * a.E + 4 * l + i] * lead : 0.0f;
  };
  if (q < a.S) enter();
  constexpr int U = 2;  // tokens whose logits are in flight together
  // every group makes the same number of steps: the lanes of a wave exchange values
  for (int b = 0; b < per_group; b += U) {
    f32x4_t z[U];
    int id[U];
    float dw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = min(t0 + b + u, a.T - 1);
      z[u] = four_logits<VEC>(a.logits + (size_t)t * a.E, l, a.E);
      if constexpr (DW) {
        id[u] = l < a.k ? a.ids[(size_t)t * a.k + l] : -1;
        dw[u] = l < a.k ? a.dw[(size_t)t * a.k + l] : 0.0f;
        if ((unsigned)id[u] >= (unsigned)a.E) {
          if (l < a.k && a.flags) atomicOr(a.flags, kFlagExpertId);
          id[u] = -1;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + b + u;
      while (t < t1 && t >= end && q + 1 < a.S) {
        ++q;
        enter();
      }
      const bool live = t < t1 && t >= begin && t < end;
      Score v[4];
      f32x4_t ds;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = score_of(z[u][i]);
      const float total = group_sum<G>((v[0].s + v[1].s) + (v[2].s + v[3].s));
      const float dot = group_sum<G>((g[0] * v[0].s + g[1] * v[1].s) + (g[2] * v[2].s + g[3] * v[3].s));
      const float inv = total != 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) ds[i] = (g[i] - dot * inv) * inv;
      if constexpr (DW) {
        // lane j of the group: slot j's score, from the lane that holds its expert
        const int from = (lane & ~(G - 1)) + (id[u] < 0 ? 0 : id[u] >> 2), c = id[u] & 3;
        const float a0 = __shfl(v[0].s, from), a1 = __shfl(v[1].s, from), a2 = __shfl(v[2].s, from),
                    a3 = __shfl(v[3].s, from);
        const float sj = id[u] < 0 ? 0.0f : c == 0 ? a0 : c == 1 ? a1 : c == 2 ? a2 : a3;
        const float norm = group_sum<8>(sj), wdot = group_sum<8>(id[u] < 0 ? 0.0f : dw[u] * sj);
        const float ninv = norm != 0.0f ? 1.0f / norm : 0.0f;
        const float dsj = a.scale * ninv * (dw[u] - wdot * ninv);
        for (int j = 0; j < a.k; ++j) {  // in slot order
          const int at = (lane & ~(G - 1)) + j, ej = __shfl(id[u], at);
          const float dj = __shfl(dsj, at);
#pragma unroll
          for (int i = 0; i < 4; ++i) ds[i] += ej == 4 * l + i ? dj : 0.0f;
        }
      }
      if (t >= t1) continue;
      f32x4_t o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = live ? ds[i] * score_slope(z[u][i], v[i]) : 0.0f;
      float* row = a.dlogits + (size_t)t * a.E;
      if constexpr (VEC) {
        if (4 * l < a.E) *reinterpret_cast<f32x4_t*>(row + 4 * l) = o;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * l + i < a.E) row[4 * l + i] = o[i];
      }
    }
  }
}

// Lanes per token: four experts each, eight lanes at least (a token's slots lie in the first eight).
template <class F>
hipError_t by_group(int E, F&& f) {
  if (E > 128) f(std::integral_constant<int, 64>{});
  else if (E > 64) f(std::integral_constant<int, 32>{});
  else if (E > 32) f(std::integral_constant<int, 16>{});
  else f(std::integral_constant<int, 8>{});
  return hipGetLastError();
}

bool balance_args_ok(const BalanceArgs& a) {
  return a.T >= 0 && a.E > 0 && a.E <= 256 && a.k > 0 && a.k <= kTopKMax && a.S > 0 && (a.offsets || a.S == 1);
}

}  // namespace

int balance_run(int T) {
  const int run = (T + kBalRuns - 1) / kBalRuns;
  return run < kBalRunMin ? kBalRunMin : run;
}
int balance_rows(int T, int S) {
  const int run = balance_run(T);
  return (T > 0 ? (T + run - 1) / run : 1) + S;
}

hipError_t launch_balance(BalanceArgs a, hipStream_t st) {
  if (!balance_args_ok(a)) return hipErrorInvalidValue;
  a.run = balance_run(a.T);
  const unsigned runs = (unsigned)(balance_rows(a.T, a.S) - a.S);
  const hipError_t e = by_group(a.E, [&](auto g) {
    if (a.E % 4 == 0) k_balance_runs<g, true><<<runs, kBalThreads, 0, st>>>(a);
    else k_balance_runs<g, false><<<runs, kBalThreads, 0, st>>>(a);
  });
  if (e != hipSuccess) return e;
  k_balance_fold<<<(unsigned)a.S, kBalThreads, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_route_backward(const BalanceArgs& a, hipStream_t st) {
  if (!balance_args_ok(a) || a.T == 0) return hipErrorInvalidValue;
  return by_group(a.E, [&](auto g) {
    constexpr int TPW = 64 / decltype(g)::value;
    // a run per group: enough of them for 16 waves per CU, an even number of tokens each
    const long long groups = 256ll * 16 * TPW;
    int per = (int)((a.T + groups - 1) / groups);
    per = (per + 1) & ~1;
    const long long need = (a.T + per - 1) / per, per_block = kGradWaves * TPW;
    const unsigned nb = (unsigned)((need + per_block - 1) / per_block);
    constexpr int NT = kGradWaves * 64;
    if (a.E % 4 == 0) {
      if (a.dw) k_route_backward<g, true, true><<<nb, NT, 0, st>>>(a, per);
      else k_route_backward<g, true, false><<<nb, NT, 0, st>>>(a, per);
    } else {
      if (a.dw) k_route_backward<g, false, true><<<nb, NT, 0, st>>>(a, per);
      else k_route_backward<g, false, false><<<nb, NT, 0, st>>>(a, per);
    }
  });
}

}  // namespace moe

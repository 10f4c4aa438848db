// The load-balance loss of a router with its per-expert counts, and the loss's
// gradient with respect to the logits, over a batch of ragged sequences.
//
// For each sequence s (the whole batch without cu_seqlens), over its n tokens
// that the token mask keeps:
//   p_t  = softmax(r_t)                       (RENORM, RAW)
//        = sigmoid(r_t) / sum_j sigmoid(r_tj) (SIGMOID)
//   c_i  = #{(t, slot): topk_idx = i},  f_i = c_i / (n k),  P_i = mean_t p_ti
//   L    = E sum_i f_i P_i
//   dL/dr_tj = (E / n) p_tj (f_j - sum_i f_i p_ti)   [SIGMOID: times 1 - sigmoid(r_tj)]
// Sources: kevinluzbetak "Mixture-Of-Experts", balancing list (E sum f P, the
// gradient flows through P alone: f is a count); AI Engineering Illustrated,
// "Fix 1" and the sequence-level loss of DeepSeek-V3.
//
// Bound: memory in principle (15 us for 32768 rows of 256 experts, both ways),
// in fact the instructions of a row and the three launches: 37 us. The forward
// pass reads the logits once, the gradient reads them once more and writes as
// much (it needs f, a count over the whole sequence). A row's softmax stays in the registers of one group of lanes.
// Determinism: every sum has a fixed order (lane, then warp, then chunk);
// counts are integers. The probability sums of a warp are fp32 over at most
// WARP_ROWS rows; everything above is added in fp64, and rounded once to fp32
// where a block leaves its sum of a sequence to balance_finish_kernel. All terms
// are positive, so P is off by at most WARP_ROWS + 3 half ulps beside the
// probabilities' own error, however long the batch. (Sums left in fp64 would save
// one of the 67 and cost that kernel twice the bytes: 13831 tokens, 475 experts,
// 2 sequences 44 -> 51 us both ways.)
#pragma once
#include "common.cuh"
#include "router.cuh"

namespace moe {
namespace bal {

struct BalParams {
  const void* logits;
  int64_t ld;              // elements from a row of logits to the next
  const int32_t* idx;      // [T, k]; entries outside [0, E) count for no expert
  const uint8_t* mask;     // [T], nonzero = the token counts; NULL = all do
  const int32_t* cu;       // [S + 1] first token of each sequence; NULL = one sequence
  int T, E, k, S;
  int chunk, nchunks;      // tokens per block of the forward kernel, and blocks
  float* part_psum;        // [nchunks + S][E]: slot (chunk + sequence)
  int32_t* part_counts;    // [nchunks + S][E]
  int32_t* part_tokens;    // [nchunks + S]
  float* loss;             // [S]
  int32_t* counts;         // [S, E]
  int32_t* tokens;         // [S]
};

// Sequence bounds, clamped so that any contents of cu stay inside the batch.
__device__ __forceinline__ int seq_begin(const int32_t* cu, int s, int T) {
  if (cu == nullptr) return 0;
  const int v = cu[s];
  return v < 0 ? 0 : (v > T ? T : v);
}
__device__ __forceinline__ int seq_end(const int32_t* cu, int s, int T) {
  if (cu == nullptr) return T;
  const int v = cu[s + 1], b = seq_begin(cu, s, T);
  return v < b ? b : (v > T ? T : v);
}
// First sequence that ends behind token t (S when none does).
__device__ __forceinline__ int first_seq_past(const int32_t* cu, int S, int t) {
  if (cu == nullptr) return 0;
  int lo = 0, hi = S;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid + 1] > t) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// 2^x and 1/x by the hardware: off by 2 ulp and 1 ulp, results below 2^-126 are
// zero: a few 2^-23 of a probability, of the order of its other roundings. (The
// layer's own statistic takes expf and divisions; the two agree to that.) With the library's expf and a true division, and a test of every
// expert's index, a row of 256 took 540 instructions forward and 740 backward
// and these kernels were bound by issuing them: 34 and 40 us for 32768 rows.
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The terms of one row's probabilities in place of its logits; returns the
// factor that makes them probabilities. SIGMOID: also the slope 1 - sigmoid(r).
// Lane l of a group of G holds experts l, l + G, ... (NV of them; those past E
// hold -inf). A softmax is scaled by the row's largest logit: 2^((r - max)
// log2e). The difference is taken first, in logits: it is exact near the maximum
// and finite or -inf for any finite row. As one fused r log2e - max log2e, the
// rounding of max log2e passes the exponent's range from logits of 1e9 on (rows
// of 1e10 had no probabilities, or NaN). sigmoid(r) = e^min(r,0) / (1 + e^-|r|)
// needs one exponential where the row has a logit >= 0; a row below zero is
// scaled by its largest logit too, so that it keeps its ratios where the
// sigmoids underflow. A row of only -inf has no probabilities: all zero. NaN
// gives NaN, as does +inf under the softmax.
// U rows at once, so that their shuffles overlap.
template <int G, int NV, int U, bool SIG>
__device__ __forceinline__ void row_terms(float (*v)[NV], float (*slope)[NV], float* inv) {
  constexpr float L2E = 1.4426950408889634f;
  float m[U], s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    m[u] = v[u][0];
#pragma unroll
    for (int i = 1; i < NV; ++i) m[u] = fmaxf(m[u], v[u][i]);
  }
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1)
#pragma unroll
    for (int u = 0; u < U; ++u) m[u] = fmaxf(m[u], __shfl_xor_sync(0xffffffffu, m[u], o));
#pragma unroll
  for (int u = 0; u < U; ++u) {
    s[u] = 0.f;
    if (SIG) {
      const bool below = __any_sync(0xffffffffu, m[u] < 0.f);  // warp-uniform
      const float top_r = m[u] < 0.f && m[u] != -INFINITY ? m[u] : 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float e = ex2(fabsf(v[u][i]) * -L2E), r1 = rcp(1.f + e);
        const bool pos = v[u][i] >= 0.f;
        float top = pos ? 1.f : e;
        if (below && !pos) top = ex2((v[u][i] - top_r) * L2E);
        slope[u][i] = (pos ? e : 1.f) * r1;
        v[u][i] = top * r1;
        s[u] += v[u][i];
      }
    } else {
      const float top_r = m[u] != -INFINITY ? m[u] : 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        v[u][i] = ex2((v[u][i] - top_r) * L2E);
        s[u] += v[u][i];
      }
    }
  }
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1)
#pragma unroll
    for (int u = 0; u < U; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], o);
#pragma unroll
  for (int u = 0; u < U; ++u) inv[u] = s[u] == 0.f ? 0.f : rcp(s[u]);
}
// Rows a group of lanes works on at once.
template <int NV> constexpr int ROWS_AT_ONCE = NV <= 2 ? 4 : (NV == 4 ? 2 : 1);

// One row's logits into registers (experts past E: -inf); rows that do not
// exist or do not count: zeros, whatever they hold.
template <typename TL, int G, int NV>
__device__ __forceinline__ void load_row(const TL* row, bool ok, int sub, int E, float* v) {
  const TL* p = row + sub;
  if (E == G * NV) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = 0.f;
    if (ok) {
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = to_f32(p[G * i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      v[i] = sub + G * i < E ? (ok ? to_f32(p[G * i]) : 0.f) : -INFINITY;
  }
}

// Deterministic block sum of a double (all threads get it); red holds 32.
__device__ __forceinline__ double block_sum(double v, double* red) {
  const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[warp] = v;
  __syncthreads();
  v = (int)(threadIdx.x & 31) < nw ? red[threadIdx.x & 31] : 0.0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// L = E sum_i c_i psum_i / (n^2 k) from a block-wide sum of c_i psum_i.
__device__ __forceinline__ float loss_of(double dot, int n, int E, int k) {
  if (n == 0) return 0.f;
  return (float)((double)E * dot / ((double)n * (double)n * (double)k));
}

// One block per chunk of tokens; warps take the chunk's tokens in turn, 32 / G
// times ROWS_AT_ONCE at a time. The block walks the sequences that its chunk
// meets; each leaves its sums in slot (chunk + sequence), which no other pair has, or, when the
// sequence lies inside the chunk, its results at once.
// The fp32 sums of a warp's rows end after WARP_ROWS of them, so that their error
// (at most WARP_ROWS half ulps) does not grow with the batch; a chunk holds more
// than one such span of rows from some 300 thousand tokens on (32 warps a block).
// Dynamic shared memory: double total[E] (the spans before the last), float
// psum[warps][E], int32 counts[E].
constexpr int WARP_ROWS = 64;
template <typename TL, int G, int NV, bool SIG>
__global__ void __launch_bounds__(NV > 8 ? 8192 / NV : 1024) balance_kernel(const BalParams p) {
  pdl_wait();
  pdl_launch_dependents();
  extern __shared__ __align__(16) uint8_t bal_smem[];
  constexpr int U = ROWS_AT_ONCE<NV>, PER = 32 / G * U;
  const int THREADS = blockDim.x, WARPS = THREADS / 32;
  double* s_total = reinterpret_cast<double*>(bal_smem);
  float* s_psum = reinterpret_cast<float*>(s_total + p.E);
  int32_t* s_cnt = reinterpret_cast<int32_t*>(s_psum + (size_t)WARPS * p.E);
  __shared__ double s_red[32];
  __shared__ int s_n;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane & (G - 1), grp = lane / G;
  const TL* logits = static_cast<const TL*>(p.logits);
  const int c0 = blockIdx.x * p.chunk;
  const int c1 = min(p.T, c0 + p.chunk);
  if (p.nchunks == 1 && (p.cu != nullptr || p.T == 0)) {  // empty sequences: no other kernel sees them
    for (int s = warp; s < p.S; s += WARPS) {
      if (seq_begin(p.cu, s, p.T) < seq_end(p.cu, s, p.T)) continue;
      for (int i = lane; i < p.E; i += 32) p.counts[(size_t)s * p.E + i] = 0;
      if (lane == 0) {
        p.tokens[s] = 0;
        p.loss[s] = 0.f;
      }
    }
  }
  for (int s = first_seq_past(p.cu, p.S, c0); s < p.S; ++s) {
    const int qb = seq_begin(p.cu, s, p.T), qe = seq_end(p.cu, s, p.T);
    if (qb >= c1) break;
    int b = max(qb, c0), e = min(qe, c1);
    if (b >= e) continue;
    const int last = e, span = WARPS * WARP_ROWS;
    const bool spans = e - b > span;
    __syncthreads();
    for (int i = threadIdx.x; i < p.E; i += THREADS) {
      s_cnt[i] = 0;
      if (spans) s_total[i] = 0.0;
    }
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
    float ps[NV], next[U][NV];
    bool next_live[U];
    int mine = 0;
    // the next rows' logits are loaded before these are worked on
    auto load = [&](int t0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = t0 + u * (32 / G) + grp;
        next_live[u] = t < e && (p.mask == nullptr || p.mask[t] != 0);
        load_row<TL, G, NV>(logits + (int64_t)t * p.ld, next_live[u], sub, p.E, next[u]);
      }
    };
    for (;; b = e) {  // spans of rows, mostly one
      e = min(last, b + span);
#pragma unroll
      for (int i = 0; i < NV; ++i) ps[i] = 0.f;
      load(b + warp * PER);
      for (int t0 = b + warp * PER; t0 < e; t0 += WARPS * PER) {
        float v[U][NV], slope[U][NV], inv[U];
        bool live[U];
        int chosen[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          live[u] = next_live[u];
#pragma unroll
          for (int i = 0; i < NV; ++i) v[u][i] = next[u][i];
          const int t = t0 + u * (32 / G) + grp;
          chosen[u] = live[u] && sub < p.k ? p.idx[(int64_t)t * p.k + sub] : -1;
        }
        load(t0 + WARPS * PER);
        row_terms<G, NV, U, SIG>(v, slope, inv);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (!live[u]) continue;
          const int t = t0 + u * (32 / G) + grp;
          if ((unsigned)chosen[u] < (unsigned)p.E) atomicAdd(&s_cnt[chosen[u]], 1);
          for (int j = sub + G; j < p.k; j += G) {
            const int x = p.idx[(int64_t)t * p.k + j];
            if ((unsigned)x < (unsigned)p.E) atomicAdd(&s_cnt[x], 1);
          }
          mine += sub == 0;
#pragma unroll
          for (int i = 0; i < NV; ++i) ps[i] = fmaf(v[u][i], inv[u], ps[i]);
        }
      }
      // the groups of a warp hold the same experts: add them up
#pragma unroll
      for (int o = G; o < 32; o <<= 1) ps[0] += __shfl_xor_sync(0xffffffffu, ps[0], o);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (lane < G && sub + G * i < p.E) s_psum[(size_t)warp * p.E + sub + G * i] = ps[i];
      if (e == last) break;
      __syncthreads();
      for (int i = threadIdx.x; i < p.E; i += THREADS) {
        double acc = 0.0;
        for (int w = 0; w < WARPS; ++w) acc += (double)s_psum[(size_t)w * p.E + i];
        s_total[i] += acc;
      }
      __syncthreads();
    }
    if (mine) atomicAdd(&s_n, mine);
    __syncthreads();
    const bool whole = qb >= c0 && qe <= c1;
    const size_t slot = (size_t)blockIdx.x + s;
    const int n = s_n;
    double dot = 0.0;
    for (int i = threadIdx.x; i < p.E; i += THREADS) {
      double acc = 0.0;
#pragma unroll 8
      for (int w = 0; w < WARPS; ++w) acc += (double)s_psum[(size_t)w * p.E + i];
      if (spans) acc += s_total[i];
      const int c = s_cnt[i];
      if (whole) {
        p.counts[(size_t)s * p.E + i] = c;
        dot += (double)c * acc;
      } else {
        p.part_psum[slot * p.E + i] = (float)acc;
        p.part_counts[slot * p.E + i] = c;
      }
    }
    if (whole) {
      dot = block_sum(dot, s_red);
      if (threadIdx.x == 0) {
        p.tokens[s] = n;
        p.loss[s] = loss_of(dot, n, p.E, p.k);
      }
    } else if (threadIdx.x == 0) {
      p.part_tokens[slot] = n;
    }
  }
}

// One block per sequence: those that met several chunks add
// their slots up, empty ones get zeros. A thread per expert (rounded up to a
// warp) and part of the slots; the parts are added in order.
__global__ void __launch_bounds__(1024) balance_finish_kernel(const BalParams p) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ double s_ps[1024];
  __shared__ int s_c[1024];
  __shared__ double s_red[32];
  const int s = blockIdx.x;
  const int qb = seq_begin(p.cu, s, p.T), qe = seq_end(p.cu, s, p.T);
  const bool empty = qb >= qe;
  const int f = empty ? 0 : qb / p.chunk, l = empty ? -1 : (qe - 1) / p.chunk;
  if (!empty && f == l) return;  // finished where it was read
  const int width = (p.E + 31) & ~31, parts = blockDim.x / width;
  const int e = threadIdx.x % width, part = threadIdx.x / width;
  double ps = 0.0;
  int c = 0;
  if (e < p.E && part < parts) {
#pragma unroll 4
    for (int j = f + part; j <= l; j += parts) {
      ps += (double)p.part_psum[((size_t)j + s) * p.E + e];
      c += p.part_counts[((size_t)j + s) * p.E + e];
    }
  }
  s_ps[threadIdx.x] = ps;
  s_c[threadIdx.x] = c;
  __syncthreads();
  double dot = 0.0;
  if (part == 0 && e < p.E) {
    for (int w = 1; w < parts; ++w) {
      ps += s_ps[w * width + e];
      c += s_c[w * width + e];
    }
    p.counts[(size_t)s * p.E + e] = c;
    dot = (double)c * ps;
  }
  int n = 0;
  for (int j = f + (int)threadIdx.x; j <= l; j += blockDim.x) n += p.part_tokens[(size_t)j + s];
  dot = block_sum(dot, s_red);
  const int total = (int)block_sum((double)n, s_red);
  if (threadIdx.x == 0) {
    p.tokens[s] = total;
    p.loss[s] = loss_of(dot, total, p.E, p.k);
  }
}

// The gradient: each warp takes `run` consecutive tokens, as many at a time.
// f - 1/E stands for f: the p of a row add up to 1, so the difference is the
// same, and (c E - n k) is an exact integer, so an f near 1/E does not cancel.
// Rows that are masked or lie in no sequence get zeros, whatever they hold.
template <typename TL, int G, int NV, bool SIG>
__global__ void __launch_bounds__(256) balance_backward_kernel(const BalParams p, const float* dloss,
                                                               TL* dlogits, int run) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int U = ROWS_AT_ONCE<NV>, PER = 32 / G * U;
  const int lane = threadIdx.x & 31, sub = lane & (G - 1), grp = lane / G;
  const int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int64_t b64 = w * run;
  if (b64 >= p.T) return;  // warp-uniform
  const int b = (int)b64, e = min(p.T, b + run);
  const TL* logits = static_cast<const TL*>(p.logits);
  // the next rows' logits are loaded before these are worked on, and the first
  // before their sequence is looked up: rows that do not count are read as well
  float next[U][NV];
  auto load = [&](int t0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * (32 / G) + grp;
      load_row<TL, G, NV>(logits + (int64_t)t * p.ld, t < e, sub, p.E, next[u]);
    }
  };
  load(b);
  int s = first_seq_past(p.cu, p.S, min(b + grp, p.T - 1)), have = -1;
  int qb = 0, qe = 0;
  float f[NV], coef = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) f[i] = 0.f;
  if (s < p.S) { qb = seq_begin(p.cu, s, p.T); qe = seq_end(p.cu, s, p.T); }
  for (int t0 = b; t0 < e; t0 += PER) {
    float v[U][NV], slope[U][NV], inv[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NV; ++i) v[u][i] = next[u][i];
    load(t0 + PER);
    row_terms<G, NV, U, SIG>(v, slope, inv);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * (32 / G) + grp;
      while (s < p.S && t >= qe) {
        if (++s < p.S) { qb = seq_begin(p.cu, s, p.T); qe = seq_end(p.cu, s, p.T); }
      }
      const bool live =
          t < e && s < p.S && t >= qb && (p.mask == nullptr || p.mask[t] != 0);
      if (live && have != s) {
        have = s;
        const int n = p.tokens[s];
        const int64_t nk = (int64_t)n * p.k;
        coef = n > 0 ? (float)((double)dloss[s] * (double)p.E / (double)n) : 0.f;
        const float over = n > 0 ? (float)(1.0 / ((double)nk * (double)p.E)) : 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int x = sub + G * i;
          f[i] = x < p.E ? (float)((int64_t)p.counts[(size_t)s * p.E + x] * p.E - nk) * over : 0.f;
        }
      }
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) dot = fmaf(f[i], v[u][i], dot);
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      dot *= inv[u];
      const float k = coef * inv[u];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float d = v[u][i] * k * (f[i] - dot);
        if (SIG) d *= slope[u][i];
        v[u][i] = live ? d : 0.f;
      }
      if (t < e) {
        TL* o = dlogits + (int64_t)t * p.E + sub;
        if (p.E == G * NV) {
#pragma unroll
          for (int i = 0; i < NV; ++i) o[G * i] = from_f32<TL>(v[u][i]);
        } else {
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if (sub + G * i < p.E) o[G * i] = from_f32<TL>(v[u][i]);
        }
      }
    }
  }
}

}  // namespace bal
}  // namespace moe

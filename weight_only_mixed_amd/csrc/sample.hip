// Next-token choice: temperature, top-k, top-p, min-p, from given uniform
// numbers (semantics in slq_serve.h).
//
// Weights w = exp((l - max) / T) are fp64, then whole numbers floor(w * 2^S)
// with S = 62 - ceil(log2 vocab): sums of them are exact, so histograms may be
// filled with atomics and partial sums taken in any order without changing a
// result, and a cut falls where the 64-bit definition puts it.
//
// One workgroup per row.  The three cuts are prefixes of one order (logit
// descending, index ascending), so the kept set is "key above tau, or equal to
// tau and among the first ties by index", with w >= min_p on top.  tau comes
// from a radix descent over the 32-bit ordered keys with a (count, mass)
// histogram per digit; the draw descends over index segments, one per wave.
#include <float.h>

#include "serve.h"
#include "slq_device.h"

namespace slq {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr int kBins = 2048;

template <int T>
__device__ __forceinline__ float load_logit(const void *row, int64_t i) {
  float v;
  if constexpr (T == kElemF32) v = static_cast<const float *>(row)[i];
  else if constexpr (T == kElemBf16)
    v = __builtin_bit_cast(float, (uint32_t) static_cast<const uint16_t *>(row)[i] << 16);
  else v = (float)static_cast<const _Float16 *>(row)[i];
  return fminf(v == v ? v : -INFINITY, FLT_MAX);   // NaN -> -inf, +inf -> finite
}

// Order-preserving 32-bit key (-0 and +0 are equal logits).
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.f);
  return b ^ (b & 0x80000000u ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __builtin_bit_cast(float, k ^ (k & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu));
}

// exp(x) for x <= 0 in fp64: x = n ln 2 + f, |f| <= ln 2 / 2, Taylor series of
// degree 12 (remainder below 2e-16).  Below 2^-64 it is 0.
__device__ __forceinline__ double exp_neg(double x) {
  const double n = rint(x * 1.4426950408889634);
  if (!(n > -64.0)) return 0.0;
  const double f = fma(n, -2.3190468138462996e-17, fma(n, -0.6931471805599453, x));
  double r = 1.0 / 479001600;
  r = fma(r, f, 1.0 / 39916800);
  r = fma(r, f, 1.0 / 3628800);
  r = fma(r, f, 1.0 / 362880);
  r = fma(r, f, 1.0 / 40320);
  r = fma(r, f, 1.0 / 5040);
  r = fma(r, f, 1.0 / 720);
  r = fma(r, f, 1.0 / 120);
  r = fma(r, f, 1.0 / 24);
  r = fma(r, f, 1.0 / 6);
  r = fma(r, f, 0.5);
  r = fma(r, f, 1.0);
  r = fma(r, f, 1.0);
  return ldexp(r, (int)n);
}

struct Weigh {
  double max, inv_t, unit;
  __device__ __forceinline__ double weight(float v) const {
    return v == -INFINITY ? 0.0 : exp_neg(((double)v - max) * inv_t);
  }
  __device__ __forceinline__ uint64_t mass(double w) const { return (uint64_t)(w * unit); }
};

__device__ __forceinline__ uint64_t wave_sum_u64(uint64_t v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor((unsigned long long)v, o, kWave);
  return v;
}
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const uint64_t t = __shfl_xor((unsigned long long)v, o, kWave);
    v = t > v ? t : v;
  }
  return v;
}

struct Shared {
  uint32_t count[kBins];
  unsigned long long mass[kBins];
  uint64_t a[kWaves], b[kWaves];
  uint32_t digit;
  uint64_t above_n, above_m;
};

// The elements strictly above key tau number `above_n` and weigh `above_m`;
// `ties` elements equal it.
struct Cut {
  uint32_t tau;
  uint64_t above_n, above_m, ties;
};

// Descends to the key at which the running count reaches `want_n` (by_mass
// false) or the running mass reaches `want_m` (by_mass true).  Every thread
// returns the same cut.  The wanted amount is at most the total.
template <int T>
__device__ Cut descend(const void *row, int64_t vocab, const Weigh &wg, bool by_mass,
                       uint64_t want_n, double want_m, Shared &sh) {
  uint32_t prefix = 0;
  uint64_t above_n = 0, above_m = 0, ties = 0;
  int shift = 32;
  const int bits[3] = {11, 11, 10};
#pragma unroll
  for (int level = 0; level < 3; ++level) {
    const int next = shift - bits[level];
    const uint32_t bins = 1u << bits[level];
    for (uint32_t i = threadIdx.x; i < bins; i += kThreads) {
      sh.count[i] = 0;
      sh.mass[i] = 0;
    }
    __syncthreads();
    for (int64_t i = threadIdx.x; i < vocab; i += kThreads) {
      const float v = load_logit<T>(row, i);
      const uint32_t k = key_of(v);
      if (level == 0 || k >> shift == prefix) {
        const uint32_t d = (k >> next) & (bins - 1);
        atomicAdd(&sh.count[d], 1u);
        atomicAdd(&sh.mass[d], (unsigned long long)wg.mass(wg.weight(v)));
      }
    }
    __syncthreads();
    if (threadIdx.x < kWave) {   // wave 0 scans the bins from the top, 64 at a time
      const int lane = threadIdx.x;
      bool done = false;
      for (int base = (int)bins - kWave; base >= 0 && !done; base -= kWave) {
        const int d = base + kWave - 1 - lane;
        uint64_t n = sh.count[d], m = sh.mass[d];
        const uint64_t n0 = n, m0 = m;
#pragma unroll
        for (int o = 1; o < kWave; o <<= 1) {
          const uint64_t tn = __shfl_up((unsigned long long)n, o, kWave);
          const uint64_t tm = __shfl_up((unsigned long long)m, o, kWave);
          if (lane >= o) {
            n += tn;
            m += tm;
          }
        }
        const bool hit = n0 > 0 && (by_mass ? (double)(above_m + m) >= want_m : above_n + n >= want_n);
        const uint64_t mask = __ballot(hit);
        if (mask) {
          const int first = __builtin_ctzll(mask);
          if (lane == first) {
            sh.digit = (uint32_t)d;
            sh.above_n = above_n + n - n0;
            sh.above_m = above_m + m - m0;
          }
          done = true;
        } else {
          above_n += __shfl((unsigned long long)n, kWave - 1, kWave);
          above_m += __shfl((unsigned long long)m, kWave - 1, kWave);
        }
      }
      if (!done && lane == 0) {   // rounding put the wanted mass behind the last element
        uint32_t d = 0;
        while (d + 1 < bins && sh.count[d] == 0) ++d;
        sh.digit = d;
        sh.above_n = above_n - sh.count[d];
        sh.above_m = above_m - sh.mass[d];
      }
    }
    __syncthreads();
    const uint32_t d = sh.digit;
    above_n = sh.above_n;
    above_m = sh.above_m;
    ties = sh.count[d];
    prefix = level == 0 ? d : prefix << bits[level] | d;
    shift = next;
    __syncthreads();
  }
  return Cut{prefix, above_n, above_m, ties};
}

template <int T>
__global__ __launch_bounds__(kThreads) void sample_row_kernel(SampleArgs a) {
  __shared__ Shared sh;
  const int64_t r = blockIdx.x;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const void *row = static_cast<const char *>(a.logits) + r * a.row_stride * (T == kElemF32 ? 4 : 2);

  uint64_t best = 0;   // (key, ~index): the largest logit, its lowest index
  for (int64_t i = threadIdx.x; i < a.vocab; i += kThreads) {
    const uint64_t k = (uint64_t)key_of(load_logit<T>(row, i)) << 32 | (uint32_t)~(uint32_t)i;
    best = k > best ? k : best;
  }
  best = wave_max_u64(best);
  if (lane == 0) sh.a[wave] = best;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) best = sh.a[w] > best ? sh.a[w] : best;
  __syncthreads();
  const float top = value_of((uint32_t)(best >> 32));
  const float temp = a.temperature ? a.temperature[r] : 1.f;
  if (top == -INFINITY || !(temp > 0.f)) {
    if (threadIdx.x == 0) {
      a.tokens[r] = top == -INFINITY ? -1 : (int32_t)~(uint32_t)best;
      if (a.logprobs) a.logprobs[r] = top == -INFINITY ? -INFINITY : 0.f;
    }
    return;
  }
  const int s = 62 - (a.vocab > 1 ? 64 - __builtin_clzll((uint64_t)a.vocab - 1) : 0);
  const Weigh wg{(double)top, 1.0 / (double)temp, ldexp(1.0, s)};
  const int64_t k = a.top_k ? a.top_k[r] : 0;
  const float p = a.top_p ? a.top_p[r] : 1.f;
  const float mp = a.min_p ? a.min_p[r] : 0.f;
  const double min_w = mp > 0.f ? fmin((double)mp, 1.0) : 0.0;

  uint32_t tau = 0;                 // kept: key > tau, or == tau and among the first `quota` ties
  uint64_t quota = (uint64_t)a.vocab;
  double of_mass = -1.0;            // mass that top_p refers to
  if (k > 0 && k < a.vocab) {
    const Cut c = descend<T>(row, a.vocab, wg, false, (uint64_t)k, 0.0, sh);
    tau = c.tau;
    quota = (uint64_t)k - c.above_n;
    of_mass = (double)(c.above_m + quota * wg.mass(wg.weight(value_of(tau))));
  }
  if (p < 1.f) {
    if (of_mass < 0.0) {
      uint64_t m = 0;
      for (int64_t i = threadIdx.x; i < a.vocab; i += kThreads)
        m += wg.mass(wg.weight(load_logit<T>(row, i)));
      m = wave_sum_u64(m);
      if (lane == 0) sh.a[wave] = m;
      __syncthreads();
      m = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) m += sh.a[w];
      __syncthreads();
      of_mass = (double)m;
    }
    // shortest prefix with mass >= p * of_mass; at least one token
    const double want = fmax((double)p * of_mass, 1.0);
    const Cut c = descend<T>(row, a.vocab, wg, true, 0, want, sh);
    const uint64_t w = wg.mass(wg.weight(value_of(c.tau)));
    const double need = want - (double)c.above_m;
    uint64_t q = w > 0 ? (uint64_t)ceil(need / (double)w) : c.ties;
    if (q < 1) q = 1;
    if (q > c.ties) q = c.ties;
    if (c.tau > tau) {
      tau = c.tau;
      quota = q;
    } else if (c.tau == tau && q < quota) {
      quota = q;
    }
  }

  // draw: descend over index segments, one per wave
  int64_t beg = 0, end = a.vocab;
  const uint64_t w_tau = [&] {
    const double w = wg.weight(value_of(tau));
    return w >= min_w ? wg.mass(w) : 0;
  }();
  uint64_t ties_before = 0, mass_before = 0, total = 0;
  double target = 0.0;
  for (bool first = true;; first = false) {
    const int64_t seg = (((end - beg + kWaves - 1) / kWaves) + kWave - 1) / kWave * kWave;
    const int64_t s0 = min(beg + seg * wave, end), s1 = min(s0 + seg, end);
    uint64_t m = 0, t = 0;
    for (int64_t i = s0 + lane; i < s1; i += kWave) {
      const float v = load_logit<T>(row, i);
      const uint32_t kk = key_of(v);
      if (kk > tau) {
        const double w = wg.weight(v);
        m += w >= min_w ? wg.mass(w) : 0;
      } else if (kk == tau) {
        ++t;
      }
    }
    m = wave_sum_u64(m);
    t = wave_sum_u64(t);
    __syncthreads();
    if (lane == 0) {
      sh.a[wave] = m;
      sh.b[wave] = t;
    }
    __syncthreads();
    // a segment keeps the ties that the quota still covers
    auto seg_mass = [&](int w, uint64_t before) {
      const uint64_t left = quota > before ? quota - before : 0;
      return sh.a[w] + (sh.b[w] < left ? sh.b[w] : left) * w_tau;
    };
    if (first) {
      uint64_t tb = 0;
      for (int w = 0; w < kWaves; ++w) {
        total += seg_mass(w, tb);
        tb += sh.b[w];
      }
      const float u = a.u[r];
      target = fmin((double)(u > 0.f ? u : 0.f) * (double)total, (double)(total - 1));
    }
    int pick = -1;
    uint64_t tb = ties_before, mb = mass_before;
    int last = 0;
    uint64_t last_tb = tb, last_mb = mb;
    for (int w = 0; w < kWaves; ++w) {
      const uint64_t sm = seg_mass(w, tb);
      if (sm > 0) {
        last = w;
        last_tb = tb;
        last_mb = mb;
        if ((double)(mb + sm) > target) {
          pick = w;
          break;
        }
      }
      mb += sm;
      tb += sh.b[w];
    }
    if (pick < 0) {
      pick = last;
      tb = last_tb;
      mb = last_mb;
    }
    ties_before = tb;
    mass_before = mb;
    const int64_t n0 = min(beg + seg * pick, end);
    end = min(n0 + seg, end);
    beg = n0;
    if (end - beg <= kWave) break;
  }
  if (wave == 0) {
    const int64_t i = beg + lane;
    uint64_t m = 0;
    bool tie = false;
    float v = -INFINITY;
    if (i < end) {
      v = load_logit<T>(row, i);
      const uint32_t kk = key_of(v);
      tie = kk == tau;
      if (kk > tau) {
        const double w = wg.weight(v);
        m = w >= min_w ? wg.mass(w) : 0;
      }
    }
    const uint64_t tm = __ballot(tie);
    if (tie && ties_before + __popcll(tm & ((1ull << lane) - 1)) < quota) m = w_tau;
    uint64_t c = m;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const uint64_t t = __shfl_up((unsigned long long)c, o, kWave);
      if (lane >= o) c += t;
    }
    uint64_t hit = __ballot(m > 0 && (double)(mass_before + c) > target);
    const uint64_t some = __ballot(m > 0);
    const int who = hit ? __builtin_ctzll(hit) : 63 - __builtin_clzll(some | 1ull);
    if (lane == who) {
      a.tokens[r] = (int32_t)i;
      if (a.logprobs)
        a.logprobs[r] = (float)(((double)v - wg.max) * wg.inv_t - log((double)total / wg.unit));
    }
  }
}

}  // namespace

size_t sample_workspace(int64_t, int64_t) { return 0; }

hipError_t launch_sample(const SampleArgs &a, int type, void *, hipStream_t st) {
  const dim3 grid((unsigned)a.rows), block(kThreads);
  if (type == kElemF32) hipLaunchKernelGGL((sample_row_kernel<kElemF32>), grid, block, 0, st, a);
  else if (type == kElemBf16) hipLaunchKernelGGL((sample_row_kernel<kElemBf16>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((sample_row_kernel<kElemF16>), grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace slq

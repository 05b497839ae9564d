// Next-token choice: temperature, top-k, top-p, min-p, from given uniform
// numbers (semantics in slq_serve.h).
//
// Weights w = exp((l - max) / T) are fp64, then whole numbers, w * 2^S rounded,
// with S = min(50, 62 - ceil(log2 vocab)): sums of them are exact, so histograms may be
// filled with atomics and partial sums taken in any order without changing a
// result, and a cut falls where the 64-bit definition puts it.
//
// The three cuts are prefixes of one order (logit descending, index
// ascending).  Two launches:
//  1. sample_units_kernel streams the logits once.  Each wave takes one unit of
//     1024 * U consecutive elements and leaves a list of all its elements above
//     a bound that rises as the unit goes by (about the unit's 16 or 32 largest),
//     its best element, and where the row's settings need it the unit's mass.
//  2. sample_pick_kernel, one workgroup per row, takes the listed elements above
//     the largest of the row's bounds: all of the row's elements above it, so a
//     prefix of the order, usually hundreds of elements long.  A kept set that
//     ends inside it is narrowed down by a histogram of keys, cut and drawn from
//     there, by comparing all pairs (up to kPairs elements: 16 us for a row
//     where sorting the whole prefix took 31) or by sorting.  Without any cut the
//     units' masses name the unit, and only that is read again.  A kept set that
//     ends outside (a wide nucleus) is found from a histogram of the row's values
//     and the one bin where the cut falls, or (a bin of thousands of ties) by a
//     radix descent over the 32-bit ordered keys, and drawn by a descent over
//     index segments.
// A row of at most kList elements needs no first launch: it is sorted whole.
//
// Bound: HBM for many rows, latency for few.  Measured (kernel times): 512 rows of
// 151936 in fp32 (311 MB) 67 us for the lists, 4.6 TB/s, and 33 for the picks; one
// such row 6 + 16 us.  A wide nucleus costs the row's workgroup two passes of 64-bit
// exponentials over the row: 64 rows of 50257 in bf16 of which a fifth have one take
// 11 + 89 us.
#include <float.h>

#include <algorithm>

#include "serve.h"
#include "slq_device.h"

namespace slq {
namespace {

constexpr int kThreads = 1024;           // sample_pick_kernel
constexpr int kWaves = kThreads / kWave;
constexpr int kBins = 2048;
constexpr int kUnitThreads = 256;        // sample_units_kernel: four units
constexpr int kBatch = 1024;             // elements of a wave's step, 16 per lane
constexpr int kCand = 128;               // list entries of a unit
constexpr int kList = 2048;              // sorted entries of a row
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;   // key_of(-inf): the smallest key

struct Unit {
  double mass;       // sum of exp((l - top) / T), where the row needs it
  float top;         // the largest element
  uint32_t bound;    // every element with a key above it is listed
  uint32_t count;
  uint32_t pad;
};

template <int T>
struct Logit;
template <>
struct Logit<kElemF32> {
  typedef f32x4_t Vec;
  static constexpr int kBytes = 4, kPer = 4;
  static constexpr float kNegInf = -INFINITY;
  static __device__ __forceinline__ float get(Vec v, int i) { return v[i]; }
  static __device__ __forceinline__ float bits(const char *p) { return *reinterpret_cast<const float *>(p); }
  static __device__ __forceinline__ void set(Vec &v, int i, float x) { v[i] = x; }
  static __device__ __forceinline__ float one(const char *p) { return *reinterpret_cast<const float *>(p); }
};
template <>
struct Logit<kElemBf16> {
  typedef u32x4_t Vec;
  static constexpr int kBytes = 2, kPer = 8;
  static constexpr uint32_t kNegInf = 0xFF80u;
  static __device__ __forceinline__ uint32_t bits(const char *p) {
    return *reinterpret_cast<const uint16_t *>(p);
  }
  static __device__ __forceinline__ void set(Vec &v, int i, uint32_t x) {
    v[i >> 1] = i & 1 ? v[i >> 1] | x << 16 : x;
  }
  static __device__ __forceinline__ float get(Vec v, int i) {
    return __builtin_bit_cast(float, i & 1 ? v[i >> 1] & 0xFFFF0000u : v[i >> 1] << 16);
  }
  static __device__ __forceinline__ float one(const char *p) {
    return __builtin_bit_cast(float, (uint32_t) * reinterpret_cast<const uint16_t *>(p) << 16);
  }
};
template <>
struct Logit<kElemF16> {
  typedef u32x4_t Vec;
  static constexpr int kBytes = 2, kPer = 8;
  static constexpr uint32_t kNegInf = 0xFC00u;
  static __device__ __forceinline__ uint32_t bits(const char *p) {
    return *reinterpret_cast<const uint16_t *>(p);
  }
  static __device__ __forceinline__ void set(Vec &v, int i, uint32_t x) {
    v[i >> 1] = i & 1 ? v[i >> 1] | x << 16 : x;
  }
  static __device__ __forceinline__ float get(Vec v, int i) {
    return f16_bits_to_f32(i & 1 ? v[i >> 1] >> 16 : v[i >> 1] & 0xFFFFu);
  }
  static __device__ __forceinline__ float one(const char *p) {
    return (float)*reinterpret_cast<const _Float16 *>(p);
  }
};

// NaN -> -inf, +inf -> the largest finite value.
__device__ __forceinline__ float tame(float v) { return fminf(v == v ? v : -INFINITY, FLT_MAX); }

// A row of logits as 16-byte vectors: slot i of the window is element i -
// `skip`, the window starting at the 16-byte boundary at or before the row.
// Vectors that stick out of the row are read element by element, so nothing
// outside it is touched; slots outside it read as -inf.
template <int T>
struct Row {
  typedef typename Logit<T>::Vec Vec;
  const char *base;   // the boundary
  int skip;           // slots before element 0
  int end;            // slot behind the last element (vocab <= 2^24)
  __device__ __forceinline__ Row(const SampleArgs &a, int64_t r) {
    const char *p = static_cast<const char *>(a.logits) + r * a.row_stride * Logit<T>::kBytes;
    skip = (int)((uintptr_t)p & 15) / Logit<T>::kBytes;
    base = p - skip * Logit<T>::kBytes;
    end = (int)a.vocab + skip;
  }
  __device__ __forceinline__ float at(int slot) const {
    return slot >= skip && slot < end ? tame(Logit<T>::one(base + (uint32_t)(slot * Logit<T>::kBytes))) : -INFINITY;
  }
  // whether slots [lo, hi) are all elements of the row
  __device__ __forceinline__ bool inside(int lo, int hi) const { return lo >= skip && hi <= end; }
  // kPer slots from `slot`, a multiple of kPer, wholly inside the row: one load,
  // nothing done with it yet
  __device__ __forceinline__ Vec raw(int slot) const {
    return *reinterpret_cast<const Vec *>(base + (uint32_t)(slot * Logit<T>::kBytes));
  }
  // the same anywhere
  __device__ __forceinline__ Vec any(int slot) const {
    if (inside(slot, slot + Logit<T>::kPer)) return raw(slot);
    Vec w;
#pragma unroll
    for (int i = 0; i < Logit<T>::kPer; ++i)
      Logit<T>::set(w, i, slot + i >= skip && slot + i < end
                              ? Logit<T>::bits(base + (uint32_t)((slot + i) * Logit<T>::kBytes))
                              : Logit<T>::kNegInf);
    return w;
  }
  __device__ __forceinline__ void load(int slot, float *v) const {
    const Vec w = any(slot);
#pragma unroll
    for (int i = 0; i < Logit<T>::kPer; ++i) v[i] = tame(Logit<T>::get(w, i));
  }
  // f(v, slot) for the elements of the vectors at slots first, first + step, ..
  // below `stop`, which ends at a vector's end or the row's (slots behind the
  // row read as -inf); kU loads in flight
  template <int kU, typename F>
  __device__ __forceinline__ void each(int first, int step, int stop, F &&f) const {
    constexpr int P = Logit<T>::kPer;
    for (int s = first; s < stop; s += kU * step) {
      Vec w[kU];
      // one branch for all: a load inside a divergent branch waits there
      if (__all(inside(s, s + (kU - 1) * step + P))) {
#pragma unroll
        for (int u = 0; u < kU; ++u) w[u] = raw(s + u * step);
      } else {
#pragma unroll
        for (int u = 0; u < kU; ++u) w[u] = any(s + u * step);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (s + u * step < stop)
#pragma unroll
          for (int i = 0; i < P; ++i) f(tame(Logit<T>::get(w[u], i)), s + u * step + i);
    }
  }
};

// Order-preserving 32-bit key (-0 and +0 are equal logits).
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.f);
  return b ^ (b & 0x80000000u ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __builtin_bit_cast(float, k ^ (k & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu));
}

// The float that v > limit compares with where key_of(v) > k is meant: +0 is the
// key after that of -0, which no logit has.
__device__ __forceinline__ float limit_of(uint32_t k) { return value_of(k == 0x7FFFFFFFu ? k - 1 : k); }

// 2^y for y <= 0 in fp64: y = n + f, |f| <= 1/2, and the series of 2^f =
// exp(f ln 2) to degree 11 (coefficients ln(2)^k / k!, remainder below 1e-14).
// Below 2^-64 it is 0.
__device__ __forceinline__ double exp2_neg(double y) {
  const double n = rint(y);
  if (!(n > -64.0)) return 0.0;
  const double f = y - n;
  double r = 4.44553827187081e-10;
  r = fma(r, f, 7.054911620801121e-09);
  r = fma(r, f, 1.0178086009239696e-07);
  r = fma(r, f, 1.3215486790144305e-06);
  r = fma(r, f, 1.5252733804059838e-05);
  r = fma(r, f, 0.00015403530393381606);
  r = fma(r, f, 0.0013333558146428441);
  r = fma(r, f, 0.009618129107628477);
  r = fma(r, f, 0.055504108664821576);
  r = fma(r, f, 0.2402265069591007);
  r = fma(r, f, 0.6931471805599453);
  r = fma(r, f, 1.0);
  return ldexp(r, (int)n);
}

constexpr double kLog2e = 1.4426950408889634;

// w = exp((l - max) / T) and its mass, w * 2^S to the nearest whole number.
// S <= 50, so the mass is what adding 2^52 leaves in the low bits of a double.
struct Weigh {
  double max, inv_t, scale, unit;   // scale = log2(e) / T, unit = 2^S
  __device__ __forceinline__ double weight(float v) const {
    return v == -INFINITY ? 0.0 : exp2_neg(((double)v - max) * scale);
  }
  __device__ __forceinline__ uint64_t mass(double w) const {
    return __builtin_bit_cast(uint64_t, fma(w, unit, 0x1p52)) & 0xFFFFFFFFFFFFFull;
  }
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


// A row's settings.
struct Cuts {
  float temp;
  int64_t k;       // vocab: no limit
  double p;        // 1: all
  double min_w;    // 0: all
  __device__ __forceinline__ Cuts(const SampleArgs &a, int64_t r) {
    temp = a.temperature ? a.temperature[r] : 1.f;
    const int64_t kk = a.top_k ? a.top_k[r] : 0;
    k = kk > 0 && kk < a.vocab ? kk : a.vocab;
    const float pp = a.top_p ? a.top_p[r] : 1.f, m = a.min_p ? a.min_p[r] : 0.f;
    p = pp < 1.f ? (double)pp : 1.0;
    min_w = m > 0.f ? fmin((double)m, 1.0) : 0.0;
  }
  __device__ __forceinline__ bool greedy() const { return !(temp > 0.f); }
  // whether the mass of the whole row is asked for
  __device__ __forceinline__ bool row_mass(int64_t vocab) const {
    return !greedy() && k == vocab && (p < 1.0 || min_w == 0.0);
  }
};

// The n-th largest of the wave's keys, n <= their number, cut to its bits above
// `low`: at least n keys are not below it.
template <int PER>
__device__ uint32_t wave_nth(const uint32_t (&key)[PER], int n, int low) {
  uint32_t t = 0;
  for (int b = 31; b >= low; --b) {
    const uint32_t c = t | 1u << b;
    int have = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) have += __popcll(__ballot(key[i] >= c));
    if (have >= n) t = c;
  }
  return t;
}

// Values are compared as they are loaded: a NaN exceeds no bound and is never
// listed, an infinity is tamed where it is used.
template <int T>
__global__ __launch_bounds__(kUnitThreads, 4) void sample_units_kernel(SampleArgs a, Unit *units,
                                                                       uint64_t *lists, int per_row,
                                                                       int steps, int keep) {
  __shared__ uint64_t lds[kUnitThreads / kWave][kCand];
  constexpr int P = Logit<T>::kPer, V = 16 / P;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  uint64_t *list = lds[wave];
  const uint64_t below = (1ull << lane) - 1;
  const int groups = (per_row + kUnitThreads / kWave - 1) / (kUnitThreads / kWave);
  for (int64_t task = blockIdx.x; task < a.rows * groups; task += gridDim.x) {
    const int64_t r = task / groups;
    const int unit = (int)(task % groups) * (kUnitThreads / kWave) + wave;
    if (unit >= per_row) continue;
    const Row<T> row(a, r);
    const Cuts cuts(a, r);
    const bool with_mass = cuts.row_mass(a.vocab);
    const double scale = with_mass ? 1.0 / (double)cuts.temp * kLog2e : 0.0;
    const int beg = unit * steps * kBatch;   // slots fit an int: vocab <= 2^24
    uint32_t bound = kKeyNegInf;
    float limit = -INFINITY;                 // v > limit: key above the bound
    int n = 0;
    double mass = 0.0;
    float top = -INFINITY, lane_top = -INFINITY;
    typename Logit<T>::Vec next[V];
    auto fetch = [&](int at) {
      if (row.inside(at, at + kBatch)) {
#pragma unroll
        for (int j = 0; j < V; ++j) next[j] = row.raw(at + (j * kWave + lane) * P);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) next[j] = row.any(at + (j * kWave + lane) * P);
      }
    };
    fetch(beg);
    for (int s = 0; s < steps; ++s) {
      const int at = beg + s * kBatch;
      if (at >= row.end) break;
      float v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = Logit<T>::get(next[e / P], e % P);
      if (s + 1 < steps) fetch(at + kBatch);
      float mx = v[0];
#pragma unroll
      for (int e = 1; e < 16; ++e) mx = fmaxf(mx, v[e]);
      mx = tame(mx);
      lane_top = fmaxf(lane_top, mx);
      if (s == 0) {
        // `keep` distinct elements are at least the keep-th largest lane maximum
        const uint32_t one[1] = {key_of(mx)};
        if (__popcll(__ballot(mx > -INFINITY)) >= keep) {
          bound = max(wave_nth(one, keep, 14), kKeyNegInf + 1) - 1;
          limit = limit_of(bound);
        }
      }
      if (with_mass) {
        const float t = wave_max(mx);
        if (t > top) {
          if (top != -INFINITY) mass *= exp2_neg(((double)top - (double)t) * scale);
          top = t;
        }
        if (top != -INFINITY) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float x = tame(v[e]);
            mass += x == -INFINITY ? 0.0 : exp2_neg(((double)x - (double)top) * scale);
          }
        }
      }
      if (!__any(mx > limit)) continue;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        uint64_t m = __ballot(v[e] > limit);
        if (!m) continue;
        if (n + __popcll(m) > kCand) {
          // full: the bound moves to the list's keep-th largest, what is above it
          // (less than keep) stays
          uint64_t old[2];
          uint32_t key[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            old[h] = h * kWave + lane < n ? list[h * kWave + lane] : 0;
            key[h] = (uint32_t)(old[h] >> 32);
          }
          bound = wave_nth(key, keep, 0);
          limit = limit_of(bound);
          n = 0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const bool in = key[h] > bound;
            const uint64_t k = __ballot(in);
            if (in) list[n + __popcll(k & below)] = old[h];
            n += __popcll(k);
          }
        }
        const float x = tame(v[e]);
        m = __ballot(x > limit);
        if (x > limit) {
          const int i = at + ((e / P) * kWave + lane) * P + e % P - row.skip;
          list[n + __popcll(m & below)] = (uint64_t)key_of(x) << 32 | (uint32_t)~(uint32_t)i;
        }
        n += __popcll(m);
      }
    }
    top = wave_max(lane_top);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) mass += __shfl_xor(mass, o, kWave);
    const int64_t slot = r * per_row + unit;
    if (lane == 0) units[slot] = Unit{mass, top, bound, (uint32_t)n, 0u};
    for (int e = lane; e < n; e += kWave) lists[slot * kCand + e] = list[e];
  }
}

struct Shared {
  union {
    struct {
      uint32_t count[kBins];
      unsigned long long mass[kBins];
    } hist;
    struct {
      uint64_t entry[kList];          // (key, ~index)
      unsigned long long mass[kList];
      union {
        uint64_t order[kList];
        uint32_t count[kBins];
      };
    } list;
  };
  uint64_t a[kWaves], b[kWaves];
  double d[kWaves];
  uint32_t digit, listed, some;
  uint64_t above_n, above_m;
  int64_t pos;
};

// Inclusive sum over the threads before and at this one; `total` over all.
__device__ __forceinline__ uint64_t block_scan_u64(uint64_t v, uint64_t &total, Shared &sh) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const uint64_t up = __shfl_up((unsigned long long)v, o, kWave);
    if (lane >= o) v += up;
  }
  __syncthreads();
  if (lane == kWave - 1) sh.a[wave] = v;
  __syncthreads();
  total = 0;
  uint64_t before = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w == wave) before = total;
    total += sh.a[w];
  }
  return v + before;
}

__device__ __forceinline__ uint64_t block_max_u64(uint64_t v, Shared &sh) {
  v = wave_max_u64(v);
  __syncthreads();
  if ((threadIdx.x & (kWave - 1)) == 0) sh.a[threadIdx.x / kWave] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) v = sh.a[w] > v ? sh.a[w] : v;
  return v;
}

// Descending bitonic sort of n (a power of two, 64 .. kList) words.  Exchanges
// of distance <= 64 stay within the 128 words that one wave's 64 pairs cover.
__device__ void block_sort(uint64_t *x, int n) {
  int before = kList;   // distance of the previous step
  for (int k = 2; k <= n; k <<= 1)
    for (int j = k >> 1; j >= 1; j >>= 1) {
      if (j > kWave || before > kWave) __syncthreads();
      else __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      before = j;
      const int p = threadIdx.x;
      if (p < n / 2) {
        const int lo = 2 * p - (p & (j - 1)), hi = lo + j;
        const uint64_t u = x[lo], w = x[hi];
        if ((u < w) == ((lo & k) == 0)) {
          x[lo] = w;
          x[hi] = u;
        }
      }
    }
  __syncthreads();
}

// The elements strictly above key tau number `above_n` and weigh `above_m`
// (0 without masses); `ties` elements equal it.
struct Cut {
  uint32_t tau;
  uint64_t above_n, above_m, ties;
};

// Descends to the key at which the running count reaches `want_n` (by_mass
// false) or the running mass reaches `want_m` (by_mass true).  Every thread
// returns the same cut.  The wanted amount is at most the total.
template <int T>
__device__ Cut descend(const Row<T> &row, const Weigh &wg, bool by_mass, bool with_mass,
                       uint64_t want_n, double want_m, Shared &sh) {
  constexpr int P = Logit<T>::kPer;
  uint32_t prefix = 0;
  uint64_t above_n = 0, above_m = 0, ties = 0;
  int shift = 32;
  for (int level = 0; level < 3; ++level) {
    const int bits = level < 2 ? 11 : 10;
    const int next = shift - bits;
    const uint32_t bins = 1u << bits;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < bins; i += kThreads) {
      sh.hist.count[i] = 0;
      sh.hist.mass[i] = 0;
    }
    __syncthreads();
    row.template each<16 / P>((int)threadIdx.x * P, kThreads * P, row.end, [&](float v, int) {
      const uint32_t k = key_of(v);
      if (k > kKeyNegInf && (level == 0 || k >> shift == prefix)) {
        const uint32_t d = (k >> next) & (bins - 1);
        atomicAdd(&sh.hist.count[d], 1u);
        if (with_mass) atomicAdd(&sh.hist.mass[d], (unsigned long long)wg.mass(wg.weight(v)));
      }
    });
    __syncthreads();
    if (threadIdx.x < kWave) {   // wave 0 scans the bins from the top, 64 at a time
      const int lane = threadIdx.x;
      bool done = false;
      for (int base = (int)bins - kWave; base >= 0 && !done; base -= kWave) {
        const int d = base + kWave - 1 - lane;
        uint64_t n = sh.hist.count[d], m = sh.hist.mass[d];
        if (!__any(n > 0)) continue;
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
        while (d + 1 < bins && sh.hist.count[d] == 0) ++d;
        sh.digit = d;
        sh.above_n = above_n - sh.hist.count[d];
        sh.above_m = above_m - sh.hist.mass[d];
      }
    }
    __syncthreads();
    const uint32_t d = sh.digit;
    above_n = sh.above_n;
    above_m = sh.above_m;
    ties = sh.hist.count[d];
    prefix = level == 0 ? d : prefix << bits | d;
    shift = next;
  }
  return Cut{prefix, above_n, above_m, ties};
}

// The kept prefix that a count or a mass asks for: keys above tau and the first
// `quota` elements equal to it, weighing `mass`.
struct Prefix {
  uint32_t tau;
  uint64_t quota, mass;
};

// The shortest prefix of the row's order with want_n elements (by_mass false)
// or of mass want_m.  One histogram over 2048 bins of (max - l) / T, 1/64 wide
// (the map is monotone in l, so bins are runs of the order), then only the
// bin where the cut falls is gathered and sorted.  A bin of more than kList
// elements (ties, or the far tail in the last bin) takes the radix descent.
template <int T>
__device__ Prefix row_prefix(const Row<T> &row, const Weigh &wg, bool by_mass, bool with_mass,
                             uint64_t want_n, double want_m, Shared &sh) {
  constexpr int P = Logit<T>::kPer;
  const float top = (float)wg.max, step = (float)fmin(64.0 * wg.inv_t, 1e30);
  auto bin_of = [&](float v) { return (int)fminf((top - v) * step, (float)(kBins - 1)); };
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kThreads) {
    sh.hist.count[i] = 0;
    sh.hist.mass[i] = 0;
  }
  if (threadIdx.x == 0) {
    sh.listed = 0;
    sh.digit = kBins;
  }
  __syncthreads();
  row.template each<16 / P>((int)threadIdx.x * P, kThreads * P, row.end, [&](float v, int) {
    if (v == -INFINITY) return;
    const int d = bin_of(v);
    if (!by_mass) atomicAdd(&sh.hist.count[d], 1u);
    if (with_mass) atomicAdd(&sh.hist.mass[d], (unsigned long long)wg.mass(wg.weight(v)));
  });
  __syncthreads();
  const int b0 = 2 * threadIdx.x;
  uint64_t n[2] = {sh.hist.count[b0], sh.hist.count[b0 + 1]};
  uint64_t m[2] = {sh.hist.mass[b0], sh.hist.mass[b0 + 1]};
  uint64_t total;
  const uint64_t run_n = block_scan_u64(n[0] + n[1], total, sh);
  const uint64_t run_m = with_mass ? block_scan_u64(m[0] + m[1], total, sh) : 0;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const uint64_t through_n = e ? run_n : run_n - n[1], through_m = e ? run_m : run_m - m[1];
    const bool hit = by_mass ? (double)through_m >= want_m && !((double)(through_m - m[e]) >= want_m)
                             : through_n >= want_n && through_n - n[e] < want_n;
    if (hit) {   // one bin, or none where rounding put the mass behind the last
      sh.digit = (uint32_t)(b0 + e);
      sh.above_n = through_n - n[e];
      sh.above_m = through_m - m[e];
    }
  }
  __syncthreads();
  const int bin = (int)sh.digit;
  const uint64_t above_n = sh.above_n, above_m = sh.above_m;
  if (bin < kBins - 1) {
    row.template each<16 / P>((int)threadIdx.x * P, kThreads * P, row.end, [&](float v, int slot) {
      if (v == -INFINITY || bin_of(v) != bin) return;
      const uint32_t at = atomicAdd(&sh.listed, 1u);
      if (at < kList)
        sh.list.entry[at] = (uint64_t)key_of(v) << 32 | (uint32_t)~(uint32_t)(slot - row.skip);
    });
    __syncthreads();
    const int listed = (int)sh.listed;
    if (listed <= kList) {
      int size = kWave;
      while (size < listed) size <<= 1;
      for (int i = listed + threadIdx.x; i < size; i += kThreads) sh.list.entry[i] = 0;
      block_sort(sh.list.entry, size);
      uint64_t w[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (with_mass && b0 + e < listed)
          w[e] = wg.mass(wg.weight(value_of((uint32_t)(sh.list.entry[b0 + e] >> 32))));
      const uint64_t run = with_mass ? block_scan_u64(w[0] + w[1], total, sh) + above_m : above_m;
      if (threadIdx.x == 0) sh.pos = -1;
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint64_t through = e ? run : run - w[1];
        const bool hit = b0 + e < listed &&
                         (by_mass ? (double)through >= want_m && !((double)(through - w[e]) >= want_m)
                                  : (uint64_t)(b0 + e) == want_n - above_n - 1);
        if (hit) {
          sh.pos = b0 + e;
          sh.above_m = through;
        }
      }
      __syncthreads();
      const int at = (int)sh.pos;
      if (at >= 0) {
        const uint32_t tau = (uint32_t)(sh.list.entry[at] >> 32);
        // entries equal to tau up to the cut
        uint64_t q = 0;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          q += b0 + e <= at && (uint32_t)(sh.list.entry[b0 + e] >> 32) == tau;
        block_scan_u64(q, total, sh);
        const Prefix out{tau, total, sh.above_m};
        __syncthreads();
        return out;
      }
    }
  }
  const Cut c = descend<T>(row, wg, by_mass, with_mass, want_n, want_m, sh);
  const uint64_t w = with_mass ? wg.mass(wg.weight(value_of(c.tau))) : 0;
  uint64_t q;
  if (by_mass) {
    const double need = want_m - (double)c.above_m;
    q = w > 0 ? need > 0.0 ? (uint64_t)ceil(need / (double)w) : 1 : c.ties;
    if (q < 1) q = 1;
  } else {
    q = want_n > c.above_n ? want_n - c.above_n : 0;
  }
  if (q > c.ties) q = c.ties;
  return Prefix{c.tau, q, c.above_m + q * w};
}

// Draws from the elements with key > tau and the first `quota` ones equal to
// it, of weight >= min_w, among slots [beg, end): a descent over index
// segments, one per wave, to the 64 slots that hold the answer.  `target` < 0:
// u times the mass found (the range is the whole row); else the mass that the
// range's elements must exceed.  `total`: the mass that the token's share is
// taken of (0: the mass found).
template <int T>
__device__ void draw(const SampleArgs &a, int64_t r, const Row<T> &row, const Weigh &wg,
                     uint32_t tau, uint64_t quota, double min_w, int beg, int end,
                     double target, double total, Shared &sh) {
  constexpr int P = Logit<T>::kPer;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const double wt = wg.weight(value_of(tau));
  const uint64_t w_tau = wt >= min_w ? wg.mass(wt) : 0;
  uint64_t ties_before = 0, mass_before = 0;
  auto take = [&](float v, uint64_t &m, uint64_t &t) {
    const uint32_t k = key_of(v);
    if (k > tau) {
      const double w = wg.weight(v);
      m += w >= min_w ? wg.mass(w) : 0;
    } else if (k == tau) {
      ++t;
    }
  };
  do {
    const int len = end - beg;
    const bool wide = len > kWave * kWaves;   // whole vectors per lane
    const int grain = wide ? kWave * P : kWave;
    const int seg = ((len + kWaves - 1) / kWaves + grain - 1) / grain * grain;
    const int s0 = min(beg + seg * wave, end), s1 = min(s0 + seg, end);
    uint64_t m = 0, t = 0;
    if (wide) {
      row.template each<16 / P>(s0 + lane * P, kWave * P, s1, [&](float v, int) { take(v, m, t); });
    } else {
      for (int s = s0 + lane; s < s1; s += kWave) take(row.at(s), m, t);
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
    if (target < 0.0) {
      uint64_t tb = 0, sum = 0;
      for (int w = 0; w < kWaves; ++w) {
        sum += seg_mass(w, tb);
        tb += sh.b[w];
      }
      const float u = a.u[r];
      target = fmin((double)(u > 0.f ? u : 0.f) * (double)sum, (double)(sum - 1));
      if (total == 0.0) total = (double)sum;
    }
    int pick = -1, last = 0;
    uint64_t tb = ties_before, mb = mass_before, last_tb = tb, last_mb = mb;
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
    ties_before = pick < 0 ? last_tb : tb;
    mass_before = pick < 0 ? last_mb : mb;
    const int n0 = min(beg + seg * (pick < 0 ? last : pick), end);
    end = min(n0 + seg, end);
    beg = n0;
  } while (end - beg > kWave);
  if (wave == 0) {
    const int slot = beg + lane;
    const float v = slot < end ? row.at(slot) : -INFINITY;
    uint64_t m = 0, t = 0;
    if (slot < end) take(v, m, t);
    const uint64_t tm = __ballot(t > 0);
    if (t > 0 && ties_before + __popcll(tm & ((1ull << lane) - 1)) < quota) m = w_tau;
    uint64_t c = m;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const uint64_t up = __shfl_up((unsigned long long)c, o, kWave);
      if (lane >= o) c += up;
    }
    const uint64_t hit = __ballot(m > 0 && (double)(mass_before + c) > target);
    const uint64_t some = __ballot(m > 0);
    const int who = hit ? __builtin_ctzll(hit) : 63 - __builtin_clzll(some | 1ull);
    if (lane == who) {
      a.tokens[r] = (int32_t)(slot - row.skip);
      if (a.logprobs)
        a.logprobs[r] = (float)(((double)v - wg.max) * wg.inv_t - log(total / wg.unit));
    }
  }
}

// The first n entries of the sorted list are kept: draw from them by index.
__device__ void draw_listed(const SampleArgs &a, int64_t r, const Weigh &wg, int n, Shared &sh) {
  int size = kWave;
  while (size < n) size <<= 1;
  for (int i = threadIdx.x; i < size; i += kThreads)   // ~index descending: index ascending
    sh.list.order[i] = i < n ? (sh.list.entry[i] & 0xFFFFFFFFull) << 32 | (uint32_t)i : 0;
  block_sort(sh.list.order, size);   // starts with a barrier
  // each thread two neighbours, a scan over threads
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int i0 = 2 * threadIdx.x;
  uint64_t m[2];
#pragma unroll
  for (int e = 0; e < 2; ++e)
    m[e] = i0 + e < n ? sh.list.mass[(uint32_t)sh.list.order[i0 + e]] : 0;
  uint64_t c = m[0] + m[1];
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const uint64_t up = __shfl_up((unsigned long long)c, o, kWave);
    if (lane >= o) c += up;
  }
  __syncthreads();
  if (lane == kWave - 1) sh.a[wave] = c;
  __syncthreads();
  uint64_t total = 0, mine = 0;
  for (int w = 0; w < kWaves; ++w) {
    if (w == wave) mine = total;
    total += sh.a[w];
  }
  c += mine;
  const float u = a.u[r];
  const double target = fmin((double)(u > 0.f ? u : 0.f) * (double)total, (double)(total - 1));
  const uint64_t c1 = c, c0 = c - m[1];   // running mass through each neighbour
  // the last entry with any mass, where rounding puts the target at the total
  if (m[0] > 0 && c0 == total) sh.pos = i0;
  if (m[1] > 0 && c1 == total) sh.pos = i0 + 1;
  __syncthreads();
  if (m[0] > 0 && (double)c0 > target && !((double)(c0 - m[0]) > target)) sh.pos = i0;
  else if (m[1] > 0 && (double)c1 > target && !((double)(c1 - m[1]) > target)) sh.pos = i0 + 1;
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint64_t e = sh.list.entry[(uint32_t)sh.list.order[sh.pos]];
    a.tokens[r] = (int32_t)~(uint32_t)e;
    if (a.logprobs)
      a.logprobs[r] = (float)(((double)value_of((uint32_t)(e >> 32)) - wg.max) * wg.inv_t -
                              log((double)total / wg.unit));
  }
}

// At most this many listed elements are ranked by comparing all pairs.
constexpr int kPairs = 256;

// Cuts and draws among n <= kPairs listed elements, in any order: kThreads / n
// threads share an element and compare it with all others.  n_k: elements that
// top_k leaves; want < 0: no top_p; `of_list`: want is p of the mass of the
// first n_k, not a mass.
__device__ void cut_pairs(const SampleArgs &a, int64_t r, const Weigh &wg, int n, int64_t n_k,
                          double want, bool of_list, double min_w, Shared &sh) {
  int size = 16;
  while (size < n) size <<= 1;
  const int per = kThreads / size;               // 4 .. 64 neighbouring lanes
  const int i = threadIdx.x / per, part = threadIdx.x % per;
  const bool real = i < n;
  const uint64_t x = real ? sh.list.entry[i] : 0;
  double w = 0.0;
  uint64_t m = 0;
  if (real) {
    w = wg.weight(value_of((uint32_t)(x >> 32)));
    m = wg.mass(w);
    if (part == 0) sh.list.mass[i] = m;
  }
  __syncthreads();
  uint32_t rank = 0;
  uint64_t run = 0;                              // mass of the elements before it and its own
  for (int j = part; j < n; j += per) {
    const uint64_t y = sh.list.entry[j];
    if (y >= x) {
      rank += y > x;
      run += sh.list.mass[j];
    }
  }
  for (int o = 1; o < per; o <<= 1) {
    rank += __shfl_xor(rank, o, kWave);
    run += __shfl_xor((unsigned long long)run, o, kWave);
  }
  if (real && part == 0 && rank == n_k - 1) sh.above_m = run;
  __syncthreads();
  if (of_list) want = fmax(want * (double)sh.above_m, 1.0);
  const bool keep = real && rank < n_k && w >= min_w &&
                    (want < 0.0 || rank == 0 || (double)(run - m) < want);
  if (real && part == 0 && !keep) sh.list.mass[i] = 0;
  __syncthreads();
  uint64_t cum = 0, total = 0;                   // by index: ~index not below its own
  for (int j = part; j < n; j += per) {
    const uint64_t mj = sh.list.mass[j];
    total += mj;
    if ((uint32_t)sh.list.entry[j] >= (uint32_t)x) cum += mj;
  }
  for (int o = 1; o < per; o <<= 1) {
    cum += __shfl_xor((unsigned long long)cum, o, kWave);
    total += __shfl_xor((unsigned long long)total, o, kWave);
  }
  const float u = a.u[r];
  const double target = fmin((double)(u > 0.f ? u : 0.f) * (double)total, (double)(total - 1));
  // the element whose share holds the target, or (rounding) the last of any mass
  const bool holds = keep && m > 0 && part == 0;
  if (holds && cum == total) sh.pos = i;
  __syncthreads();
  if (holds && (double)cum > target && !((double)(cum - m) > target)) sh.pos = i;
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint64_t e = sh.list.entry[sh.pos];
    a.tokens[r] = (int32_t)~(uint32_t)e;
    if (a.logprobs)
      a.logprobs[r] = (float)(((double)value_of((uint32_t)(e >> 32)) - wg.max) * wg.inv_t -
                              log((double)total / wg.unit));
  }
}

// per_row = 0: the row is listed whole, no units.
template <int T>
__global__ __launch_bounds__(kThreads) void sample_pick_kernel(SampleArgs a, const Unit *units,
                                                               const uint64_t *lists, int per_row,
                                                               int steps) {
  __shared__ Shared sh;
  constexpr int P = Logit<T>::kPer;
  const int64_t r = blockIdx.x;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const Row<T> row(a, r);
  const Cuts cuts(a, r);
  const int unit_slots = steps * kBatch;
  units += r * per_row;
  lists += r * per_row * kCand;

  // the largest logit and the bound above which every element is listed
  uint32_t bound = kKeyNegInf;
  uint64_t best = 0;                   // (key, bound) or (key, ~index)
  if (threadIdx.x == 0) {
    sh.listed = 0;
    sh.some = 0;
  }
  __syncthreads();
  if (per_row == 0) {
    for (int s = threadIdx.x * P; s < row.end; s += kThreads * P) {
      float v[P];
      row.load(s, v);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        if (s + e < row.skip || s + e >= row.end) continue;
        const uint32_t k = key_of(v[e]);
        const uint64_t x = (uint64_t)k << 32 | (uint32_t)~(uint32_t)(s + e - row.skip);
        best = x > best ? x : best;
        if (k > kKeyNegInf) sh.list.entry[atomicAdd(&sh.listed, 1u)] = x;
      }
    }
    best = block_max_u64(best, sh);
  } else {
    uint32_t key = 0;
    for (int i = threadIdx.x; i < per_row; i += kThreads) {
      key = max(key, key_of(units[i].top));
      bound = max(bound, units[i].bound);
    }
    best = block_max_u64((uint64_t)key << 32, sh);
    bound = (uint32_t)block_max_u64(bound, sh);
  }
  const float top = value_of((uint32_t)(best >> 32));
  if (top == -INFINITY || cuts.greedy()) {
    if (per_row > 0 && top != -INFINITY) {
      // its lowest index: in the first unit that reaches it
      uint64_t first = 0;
      for (int i = threadIdx.x; i < per_row; i += kThreads)
        if (units[i].top == top) first = max(first, (uint64_t)(uint32_t)~(uint32_t)i);
      const int unit = (int)~(uint32_t)block_max_u64(first, sh);
      const int s0 = unit * unit_slots, s1 = min(s0 + unit_slots, row.end);
      best = 0;
      for (int s = s0 + threadIdx.x; s < s1; s += kThreads)
        if (row.at(s) == top) best = max(best, (uint64_t)(uint32_t)~(uint32_t)(s - row.skip));
      best = block_max_u64(best, sh);
    }
    if (threadIdx.x == 0) {
      a.tokens[r] = top == -INFINITY ? -1 : (int32_t)~(uint32_t)best;
      if (a.logprobs) a.logprobs[r] = top == -INFINITY ? -INFINITY : 0.f;
    }
    return;
  }
  const int s = min(50, 62 - (a.vocab > 1 ? 64 - __builtin_clzll((uint64_t)a.vocab - 1) : 0));
  const double inv_t = 1.0 / (double)cuts.temp;
  const Weigh wg{(double)top, inv_t, inv_t * kLog2e, ldexp(1.0, s)};

  // the row's mass, in the order of the units
  double row_mass = 0.0;
  const bool free_draw = cuts.k == a.vocab && !(cuts.p < 1.0) && cuts.min_w == 0.0;
  if (per_row > 0 && cuts.row_mass(a.vocab)) {
    // thread w * 64 + l takes units l + 64 w + 1024 n ...: a fixed order
    double m = 0.0;
    for (int i = threadIdx.x; i < per_row; i += kThreads)
      if (units[i].top != -INFINITY) m += units[i].mass * wg.weight(units[i].top);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) m += __shfl_xor(m, o, kWave);
    __syncthreads();
    if (lane == 0) sh.d[wave] = m;
    __syncthreads();
    for (int w = 0; w < kWaves; ++w) row_mass += sh.d[w];
    row_mass *= wg.unit;
  }

  // what the draw at the end takes: by default the whole row
  int beg = 0, end = row.end;
  double target = -1.0, total = 0.0;
  if (per_row > 0 && free_draw) {
    // the unit that holds the draw: wave 0 scans the units' masses by index
    const float u = a.u[r];
    target = fmin((double)(u > 0.f ? u : 0.f), 1.0 - 0x1p-53) * row_mass;
    __syncthreads();
    if (wave == 0) {
      double before = 0.0;
      int64_t pick = -1, last = 0;
      double pick_before = 0.0, last_before = 0.0;
      for (int base = 0; base < per_row && pick < 0; base += kWave) {
        const int i = base + lane;
        const double m = i < per_row && units[i].top != -INFINITY
                             ? units[i].mass * wg.weight(units[i].top) * wg.unit : 0.0;
        double c = m;
#pragma unroll
        for (int o = 1; o < kWave; o <<= 1) {
          const double up = __shfl_up(c, o, kWave);
          if (lane >= o) c += up;
        }
        // (a unit of less mass than elements may hold no element of any)
        const bool holds = m >= (double)unit_slots;
        const uint64_t some = __ballot(holds);
        const uint64_t hit = __ballot(holds && before + c > target);
        if (hit) {
          const int who = __builtin_ctzll(hit);
          pick = base + who;
          pick_before = before + __shfl(c - m, who, kWave);
        } else if (some) {
          const int who = 63 - __builtin_clzll(some);
          last = base + who;
          last_before = before + __shfl(c - m, who, kWave);
        }
        before += __shfl(c, kWave - 1, kWave);
      }
      if (lane == 0) {
        sh.pos = pick < 0 ? last : pick;
        sh.d[0] = pick < 0 ? last_before : pick_before;
      }
    }
    __syncthreads();
    beg = (int)sh.pos * unit_slots;
    end = min(beg + unit_slots, row.end);
    target = fmax(target - sh.d[0], 0.0);
    total = row_mass;
    __syncthreads();
  }

  // the listed elements above the bound
  if (per_row > 0 && !free_draw) {
    // a wave takes units wave, wave + 16, ..; lists are read whole (entries
    // behind a unit's count are whatever the workspace held) so that count and
    // entries are one round trip
    constexpr int kU = 5;
    for (int base = wave; base < per_row; base += kU * kWaves) {
      uint64_t x[kU][2];
      uint32_t n[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int unit = min(base + u * kWaves, per_row - 1);
        n[u] = base + u * kWaves < per_row ? units[unit].count : 0;
#pragma unroll
        for (int e = 0; e < 2; ++e) x[u][e] = lists[(int64_t)unit * kCand + e * kWave + lane];
      }
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool in = e * kWave + lane < (int)n[u] && (uint32_t)(x[u][e] >> 32) > bound;
          const uint64_t m = __ballot(in);
          if (!m) continue;
          uint32_t at = 0;
          if (lane == 0) at = atomicAdd(&sh.listed, (uint32_t)__popcll(m));
          at = __shfl(at, 0, kWave) + __popcll(m & ((1ull << lane) - 1));
          if (in && at < kList) sh.list.entry[at] = x[u][e];
        }
    }
  }
  __syncthreads();
  int listed = (int)sh.listed;
  const bool whole = bound == kKeyNegInf && listed <= kList;   // every element above -inf
  const bool k_inside = listed <= kList && (cuts.k <= listed || whole);
  const int64_t n_k = min<int64_t>(cuts.k, listed);
  const int i0 = 2 * threadIdx.x;
  // whether the kept set is known to end inside the list
  bool inside = listed > 0 && listed <= kList && (per_row == 0 || !free_draw);
  if (inside && (listed > kPairs || !k_inside)) {
    // Narrow the list to a shorter prefix that still holds the kept set, by a
    // histogram of its keys: through the n_k-th element, or the nucleus; and
    // where no mass of the first k is asked for, to the elements that min_p
    // leaves.
    const uint32_t top_key = (uint32_t)(best >> 32), span = top_key - bound - 1;
    const int shift = max(0, 32 - 11 - (span ? __builtin_clz(span) : 32));
    uint64_t x[2], m[2];
    bool heavy[2];
    for (int i = threadIdx.x; i < kBins; i += kThreads) sh.list.count[i] = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      x[e] = i0 + e < listed ? sh.list.entry[i0 + e] : 0;
      const double w = i0 + e < listed && !k_inside ? wg.weight(value_of((uint32_t)(x[e] >> 32))) : 0.0;
      heavy[e] = w >= cuts.min_w;
      m[e] = wg.mass(w);
      sh.list.mass[i0 + e] = 0;   // the histogram's masses (kBins == kList)
      if (i0 + e < listed && !k_inside && !heavy[e]) sh.some = 1;   // min_p ends inside
    }
    auto bin_of = [&](uint64_t v) { return (int)((top_key - (uint32_t)(v >> 32)) >> shift); };
    __syncthreads();
    const bool by_mass = !k_inside && cuts.p < 1.0;
    if (k_inside || by_mass) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (i0 + e < listed) {
          if (by_mass) atomicAdd(&sh.list.mass[bin_of(x[e])], (unsigned long long)m[e]);
          else atomicAdd(&sh.list.count[bin_of(x[e])], 1u);
        }
    }
    if (threadIdx.x == 0) {
      sh.digit = kBins;
      sh.listed = 0;
    }
    __syncthreads();
    if (k_inside || by_mass) {
      const uint64_t h0 = by_mass ? sh.list.mass[i0] : sh.list.count[i0];
      const uint64_t h1 = by_mass ? sh.list.mass[i0 + 1] : sh.list.count[i0 + 1];
      uint64_t all;
      const uint64_t run1 = block_scan_u64(h0 + h1, all, sh), run0 = run1 - h1;
      const double want = by_mass ? fmax(cuts.p * row_mass, 1.0) : (double)n_k;
      if ((double)run0 >= want && !((double)(run0 - h0) >= want)) sh.digit = (uint32_t)i0;
      else if ((double)run1 >= want && !((double)(run1 - h1) >= want)) sh.digit = (uint32_t)i0 + 1;
      __syncthreads();
    }
    const int through = (int)sh.digit;    // the last bin that the prefix needs
    const bool min_ends = sh.some != 0;
    if (!k_inside)
      inside = cuts.k == a.vocab ? (by_mass && through < kBins) || min_ends
                                 : !(cuts.p < 1.0) && min_ends;
    __syncthreads();
    if (inside) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (i0 + e < listed && (k_inside || heavy[e]) && bin_of(x[e]) <= through)
          sh.list.entry[atomicAdd(&sh.listed, 1u)] = x[e];
      __syncthreads();
      listed = (int)sh.listed;
    }
  }
  if (inside) {
    const bool nucleus = cuts.p < 1.0;
    const double want = !nucleus ? -1.0 : k_inside ? cuts.p : fmax(cuts.p * row_mass, 1.0);
    const int64_t first = min<int64_t>(n_k, listed);
    if (listed <= kPairs) {
      cut_pairs(a, r, wg, listed, first, want, nucleus && k_inside, cuts.min_w, sh);
      return;
    }
    int size = kWave;
    while (size < listed) size <<= 1;
    for (int i = listed + threadIdx.x; i < size; i += kThreads) sh.list.entry[i] = 0;
    block_sort(sh.list.entry, size);
    // masses, their running sum, and where each cut falls
    uint64_t m[2];
    int heavy = 0;   // entries of weight >= min_w
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[e] = 0;
      if (i0 + e < listed) {
        const double w = wg.weight(value_of((uint32_t)(sh.list.entry[i0 + e] >> 32)));
        m[e] = wg.mass(w);
        sh.list.mass[i0 + e] = m[e];
        heavy += w >= cuts.min_w;
      }
    }
    uint64_t all, n_min;
    block_scan_u64((uint64_t)heavy, n_min, sh);
    const uint64_t run1 = block_scan_u64(m[0] + m[1], all, sh), run0 = run1 - m[1];
    if (i0 == first - 1) sh.above_m = run0;      // mass of the first k
    if (i0 + 1 == first - 1) sh.above_m = run1;
    if (threadIdx.x == 0) sh.pos = listed;
    __syncthreads();
    int64_t n = min<int64_t>(first, (int64_t)n_min);
    if (nucleus) {
      const double mass = k_inside ? fmax(want * (double)sh.above_m, 1.0) : want;
      // the first entry whose running mass reaches the wanted one
      if (i0 < listed && (double)run0 >= mass && !((double)(run0 - m[0]) >= mass)) sh.pos = i0;
      else if (i0 + 1 < listed && (double)run1 >= mass && !((double)(run1 - m[1]) >= mass))
        sh.pos = i0 + 1;
      __syncthreads();
      n = min<int64_t>(n, sh.pos + 1);
      __syncthreads();
    }
    draw_listed(a, r, wg, (int)n, sh);
    return;
  }

  // the kept set ends outside the list (or is the whole row)
  uint32_t tau = 0;                 // kept: key > tau, or == tau and among the first `quota` ties
  uint64_t quota = 0;
  double of_mass = row_mass;
#pragma unroll 1
  for (int cut = 0; cut < 2; ++cut) {   // top_k, then top_p (one copy of the code)
    const bool by_mass = cut == 1;
    if (by_mass ? !(cuts.p < 1.0) : cuts.k == a.vocab) continue;
    // the shortest prefix with mass >= p * of_mass has at least one token
    const Prefix c = row_prefix<T>(row, wg, by_mass, by_mass || cuts.p < 1.0, (uint64_t)cuts.k,
                                   fmax(cuts.p * of_mass, 1.0), sh);
    if (c.tau > tau) {
      tau = c.tau;
      quota = c.quota;
    } else if (c.tau == tau && c.quota < quota) {
      quota = c.quota;
    }
    of_mass = (double)c.mass;
  }
  __syncthreads();
  draw<T>(a, r, row, wg, tau, quota, cuts.min_w, beg, end, target, total, sh);
}

struct SamplePlan {
  int per_row;   // units per row (0: rows short enough to be listed whole)
  int steps;     // 1024-element steps per unit
  int keep;
};
// Units of one step where rows are few (149 waves for one row of 151936), of
// up to eight where they are many (110 us against 122 for four and 125 for
// sixteen on 512 rows): fewer, longer units list fewer elements per row.
SamplePlan sample_plan(int64_t rows, int64_t vocab) {
  SamplePlan p{0, 1, 16};
  if (vocab <= kList) return p;
  const int64_t slots = vocab + 7;   // a row may start up to 7 elements behind a boundary
  int64_t steps = 1;
  while (steps < 8 && rows * ((slots + steps * kBatch - 1) / (steps * kBatch)) > 8192) steps *= 2;
  while ((slots + steps * kBatch - 1) / (steps * kBatch) > 4096) steps *= 2;
  p.steps = (int)steps;
  p.per_row = (int)((slots + steps * kBatch - 1) / (steps * kBatch));
  p.keep = steps == 1 ? 16 : 32;
  return p;
}

template <int T>
hipError_t launch_type(const SampleArgs &a, void *ws, hipStream_t st) {
  const SamplePlan p = sample_plan(a.rows, a.vocab);
  const size_t n = (size_t)a.rows * p.per_row;
  uint64_t *lists = static_cast<uint64_t *>(ws);
  Unit *units = reinterpret_cast<Unit *>(lists + n * kCand);
  if (p.per_row > 0) {
    const int64_t tasks = a.rows * ((p.per_row + 3) / 4);
    hipLaunchKernelGGL((sample_units_kernel<T>), dim3((unsigned)std::min<int64_t>(tasks, 1 << 20)),
                       dim3(kUnitThreads), 0, st, a, units, lists, p.per_row, p.steps, p.keep);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((sample_pick_kernel<T>), dim3((unsigned)a.rows), dim3(kThreads), 0, st, a, units,
                     lists, p.per_row, p.steps);
  return hipGetLastError();
}

}  // namespace

size_t sample_workspace(int64_t rows, int64_t vocab) {
  const SamplePlan p = sample_plan(rows, vocab);
  return (size_t)rows * p.per_row * (kCand * sizeof(uint64_t) + sizeof(Unit));
}

hipError_t launch_sample(const SampleArgs &a, int type, void *ws, hipStream_t st) {
  if (type == kElemF32) return launch_type<kElemF32>(a, ws, st);
  if (type == kElemBf16) return launch_type<kElemBf16>(a, ws, st);
  return launch_type<kElemF16>(a, ws, st);
}

}  // namespace slq

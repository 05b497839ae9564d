// Writing and reading the paged 8-bit key/value cache.
//
// Write: one workgroup per (sequence, touched page, head, K or V).  It takes
// the largest magnitude of the page's new rows, derives the page's scale (the
// old one or a larger one), encodes the new rows, and moves older codes of the
// page to a grown scale.  A page belongs to one workgroup, so nothing is
// shared and the result does not depend on any order.
// The scale is max|x| times the fp32 reciprocal of the largest code (a constant:
// one multiplication, at most one unit in the last place from the quotient); it
// is applied as the weight quantizer's is: a code is the nearest grid point of
// the IEEE fp32 quotient x / s.
//
// Bound: HBM for prompts, one chain of dependent reads (offsets, page number,
// rows) for single tokens.  Measured: 18971 rows of 8 heads x 128 in fp32 to E4M3
// (194 MB read and written) 43 us, 4.5 TB/s against 5.2 of a plain copy; one token
// each for 64 sequences 5.6 us.  Reading 112978 rows back as bf16 (694 MB) 139 us,
// 5.0 TB/s.
#include <float.h>

#include <algorithm>

#include "serve.h"
#include "slq_device.h"

namespace slq {
namespace {

constexpr int kThreads = 256;

template <int T>
struct Elem;   // 8 consecutive elements as fp32
template <>
struct Elem<kElemF32> {
  static constexpr int kBytes = 4;
  static __device__ __forceinline__ void load8(const void *p, float (&x)[8]) {
    const float4 a = static_cast<const float4 *>(p)[0], b = static_cast<const float4 *>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  static __device__ __forceinline__ void store8(void *p, const float (&x)[8]) {
    static_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    static_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
};
template <>
struct Elem<kElemBf16> {
  static constexpr int kBytes = 2;
  static __device__ __forceinline__ void load8(const void *p, float (&x)[8]) {
    const u32x4_t w = *static_cast<const u32x4_t *>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __builtin_bit_cast(float, w[i] << 16);
      x[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void store8(void *p, const float (&x)[8]) {
    bf16x8_t o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (__bf16)x[i];
    *static_cast<bf16x8_t *>(p) = o;
  }
};
template <>
struct Elem<kElemF16> {
  static constexpr int kBytes = 2;
  typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ void load8(const void *p, float (&x)[8]) {
    const f16x8 w = *static_cast<const f16x8 *>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)w[i];
  }
  static __device__ __forceinline__ void store8(void *p, const float (&x)[8]) {
    f16x8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (_Float16)x[i];
    *static_cast<f16x8 *>(p) = o;
  }
};

// NaN -> 0, infinities -> the largest finite value.
__device__ __forceinline__ float finite(float x) {
  return fminf(fmaxf(x == x ? x : 0.f, -FLT_MAX), FLT_MAX);
}

// Four codes of one word.
template <bool E4M3>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  if constexpr (E4M3) {
    auto sat = [](float x) { return fminf(fmaxf(x, -448.f), 448.f); };
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(sat(a), sat(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(sat(c), sat(d), w, true);
  } else {
    auto code = [](float x) {
      return (uint32_t)(int)fminf(fmaxf(rintf(x), -127.f), 127.f) & 0xFFu;
    };
    return code(a) | code(b) << 8 | code(c) << 16 | code(d) << 24;
  }
}

template <bool E4M3>
__device__ __forceinline__ void decode4(uint32_t w, float (&x)[4]) {
  if constexpr (E4M3) {
    x[0] = __builtin_amdgcn_cvt_f32_fp8((int)w, 0);
    x[1] = __builtin_amdgcn_cvt_f32_fp8((int)w, 1);
    x[2] = __builtin_amdgcn_cvt_f32_fp8((int)w, 2);
    x[3] = __builtin_amdgcn_cvt_f32_fp8((int)w, 3);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (float)(int8_t)(w >> (8 * i));
  }
}

// x / s, correctly rounded, for many x at one s: with y = fl(1 / s), q = fl(x y)
// is within an ulp of the quotient, its remainder x - q s is exact in one fused
// operation, and fl(q + remainder y) is the rounded quotient (Markstein, "Computation
// of elementary functions on the IBM RISC System/6000 processor", 1990).  That
// needs the remainder above the subnormal range, so it serves 2^-60 <= s <= 2^60
// (where a quotient too small for that has code 0 either way); other scales
// divide.  8 divisions a vector took as long as the memory traffic.
struct Divider {
  float s, y;
  bool fast;
  __device__ __forceinline__ explicit Divider(float scale) : s(scale) {
    fast = s >= 0x1p-60f && s <= 0x1p60f;
    y = fast ? 1.f / s : 0.f;
  }
  __device__ __forceinline__ float operator()(float x) const {
    if (fast) {
      const float q = x * y;
      // (the sum of a zero remainder and -0 is +0: the sign is x's)
      return copysignf(__builtin_fmaf(__builtin_fmaf(-q, s, x), y, q), x);
    }
    return s > 0.f ? x / s : 0.f;
  }
};

struct WriteArgs {
  KvView c;
  SeqView s;
  const char *x[2];
  int64_t row[2], head[2];   // bytes
  int32_t per;               // workgroups per sequence
};

template <int T, bool E4M3>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(WriteArgs a) {
  __shared__ float red[kThreads / kWave];
  const int b = blockIdx.x / a.per, j = blockIdx.x % a.per;
  const int h = blockIdx.y >> 1, kv = blockIdx.y & 1;
  const KvSpan sp = kv_span(a.s, a.c.shift, b);
  const int last = kv_last_page(sp, a.c.shift);
  const int vpr = a.c.dim / 8;   // 8-element vectors per row: 8, 16 or 32
  const int vs = __builtin_ctz(vpr);
  constexpr float kStep = 1.f / (E4M3 ? 448.f : 127.f);
  for (int p = kv_first_page(sp, a.c.shift) + j; p <= last; p += a.per) {
    const int id = kv_page(a.s, a.c.pages, b, p);
    if (id < 0) continue;
    const KvPart part = kv_part(sp, a.c.shift, p);
    const char *src = a.x[kv] + (int64_t)part.row * a.row[kv] + (int64_t)h * a.head[kv];
    uint8_t *dst = a.c.codes[kv] + (int64_t)id * a.c.page_stride + (int64_t)h * a.c.head_stride;
    float *scale = a.c.scales[kv] + (int64_t)id * a.c.heads + h;
    const float old = part.lo > 0 ? *scale : 0.f;
    const int nvec = (part.hi - part.lo) << vs;
    // a thread's first kHold vectors stay in registers between the two passes
    // (a whole page of 64 tokens and 128 dims); more are read again
    constexpr int kHold = 4;
    auto at = [&](int i) {
      return src + (int64_t)(i >> vs) * a.row[kv] + (i & (vpr - 1)) * (8 * Elem<T>::kBytes);
    };
    float hold[kHold][8], mx = 0.f;
#pragma unroll
    for (int u = 0; u < kHold; ++u) {
      const int i = threadIdx.x + u * kThreads;
      if (i < nvec) Elem<T>::load8(at(i), hold[u]);
      else
#pragma unroll
        for (int e = 0; e < 8; ++e) hold[u][e] = 0.f;
    }
#pragma unroll
    for (int u = 0; u < kHold; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        hold[u][e] = finite(hold[u][e]);
        mx = fmaxf(mx, fabsf(hold[u][e]));
      }
    for (int i = threadIdx.x + kHold * kThreads; i < nvec; i += kThreads) {
      float x[8];
      Elem<T>::load8(at(i), x);
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(finite(x[e])));
    }
    mx = wave_max(mx);
    __syncthreads();   // the previous page's readers of red, and of *scale
    if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x / kWave] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / kWave; ++w) mx = fmaxf(mx, red[w]);
    const float s = fmaxf(mx * kStep, old);
    const Divider by(s);
    auto put = [&](int i, const float (&x)[8]) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = by(x[e]);
      u32x2_t w;
      w[0] = encode4<E4M3>(y[0], y[1], y[2], y[3]);
      w[1] = encode4<E4M3>(y[4], y[5], y[6], y[7]);
      *reinterpret_cast<u32x2_t *>(dst + (int64_t)(part.lo + (i >> vs)) * a.c.token_stride +
                                   8 * (i & (vpr - 1))) = w;
    };
#pragma unroll
    for (int u = 0; u < kHold; ++u) {
      const int i = threadIdx.x + u * kThreads;
      if (i < nvec) put(i, hold[u]);
    }
    for (int i = threadIdx.x + kHold * kThreads; i < nvec; i += kThreads) {
      float x[8];
      Elem<T>::load8(at(i), x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = finite(x[e]);
      put(i, x);
    }
    if (part.lo > 0 && s > old) {   // older codes of the page move to the new scale
      for (int i = threadIdx.x; i < part.lo << vs; i += kThreads) {
        u32x2_t *at = reinterpret_cast<u32x2_t *>(dst + (int64_t)(i >> vs) * a.c.token_stride +
                                                  8 * (i & (vpr - 1)));
        u32x2_t w = *at;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float x[4];
          decode4<E4M3>(w[k], x);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = (x[e] * old) / s;
          w[k] = encode4<E4M3>(x[0], x[1], x[2], x[3]);
        }
        *at = w;
      }
    }
    if (threadIdx.x == 0) *scale = s;
  }
}

struct ReadArgs {
  KvView c;
  SeqView s;
  char *out[2];
  int32_t per;
};

// Read: the same division of the work; rows that do not exist become 0.
template <int T, bool E4M3>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(ReadArgs a) {
  const int b = blockIdx.x / a.per, j = blockIdx.x % a.per;
  const int h = blockIdx.y >> 1, kv = blockIdx.y & 1;
  const KvSpan sp = kv_span(a.s, a.c.shift, b);
  const int last = kv_last_page(sp, a.c.shift);
  const int vpr = a.c.dim / 8;
  const int vs = __builtin_ctz(vpr);
  const int64_t orow = (int64_t)a.c.heads * a.c.dim * Elem<T>::kBytes;
  char *out = a.out[kv] + (int64_t)h * a.c.dim * Elem<T>::kBytes;
  if (j == 0) {   // rows at negative positions
    const int none = sp.pos0 < 0 ? (-sp.pos0 < sp.n ? -sp.pos0 : sp.n) : 0;
    const float zero[8] = {};
    for (int64_t i = threadIdx.x; i < (int64_t)none << vs; i += kThreads)
      Elem<T>::store8(out + (sp.row0 + (i >> vs)) * orow + (i & (vpr - 1)) * (8 * Elem<T>::kBytes), zero);
  }
  for (int p = kv_first_page(sp, a.c.shift) + j; p <= last; p += a.per) {
    const int id = kv_page(a.s, a.c.pages, b, p);
    const KvPart part = kv_part(sp, a.c.shift, p);
    const int64_t at = id < 0 ? 0 : (int64_t)id;
    const uint8_t *src = a.c.codes[kv] + at * a.c.page_stride + (int64_t)h * a.c.head_stride;
    const float s = id < 0 ? 0.f : a.c.scales[kv][at * a.c.heads + h];
    const int nvec = (part.hi - part.lo) << vs;
    for (int i = threadIdx.x; i < nvec; i += kThreads) {
      const int r = i >> vs, v = i & (vpr - 1);
      float x[8] = {};
      if (id >= 0) {
        const u32x2_t w = *reinterpret_cast<const u32x2_t *>(
            src + (int64_t)(part.lo + r) * a.c.token_stride + 8 * v);
        float lo[4], hi[4];
        decode4<E4M3>(w[0], lo);
        decode4<E4M3>(w[1], hi);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = lo[e] * s;
          x[4 + e] = hi[e] * s;
        }
      }
      Elem<T>::store8(out + (int64_t)(part.row + r) * orow + v * (8 * Elem<T>::kBytes), x);
    }
  }
}

// Workgroups per sequence for n rows: the pages that n consecutive rows can
// touch, held to 2^32 threads along x (a workgroup goes on to further pages).
int32_t pages_touched(int64_t n, int shift, int batch) {
  const int64_t page = (int64_t)1 << shift;
  const int64_t per = (n + page - 2) / page + 1;
  return (int32_t)std::max<int64_t>(1, std::min<int64_t>(per, 0xFFFFFF / batch));
}

template <typename F>
hipError_t by_type(int type, bool e4m3, F &&f) {
  switch (type) {
    case kElemF32:
      return e4m3 ? f(std::integral_constant<int, kElemF32>(), std::true_type())
                  : f(std::integral_constant<int, kElemF32>(), std::false_type());
    case kElemBf16:
      return e4m3 ? f(std::integral_constant<int, kElemBf16>(), std::true_type())
                  : f(std::integral_constant<int, kElemBf16>(), std::false_type());
    default:
      return e4m3 ? f(std::integral_constant<int, kElemF16>(), std::true_type())
                  : f(std::integral_constant<int, kElemF16>(), std::false_type());
  }
}

}  // namespace

hipError_t launch_kv_write(const KvView &c, const SeqView &s, bool e4m3, const void *k,
                           const void *v, int type, int64_t k_row, int64_t k_head, int64_t v_row,
                           int64_t v_head, int64_t max_new, hipStream_t st) {
  const int64_t eb = type == kElemF32 ? 4 : 2;
  WriteArgs a{c, s, {static_cast<const char *>(k), static_cast<const char *>(v)},
              {k_row * eb, v_row * eb}, {k_head * eb, v_head * eb},
              pages_touched(std::min<int64_t>(max_new, s.rows), c.shift, s.batch)};
  const dim3 grid((unsigned)a.per * (unsigned)s.batch, (unsigned)(2 * c.heads));
  return by_type(type, e4m3, [&](auto t, auto f) {
    hipLaunchKernelGGL((kv_write_kernel<decltype(t)::value, decltype(f)::value>), grid,
                       dim3(kThreads), 0, st, a);
    return hipGetLastError();
  });
}

hipError_t launch_kv_read(const KvView &c, const SeqView &s, bool e4m3, void *k, void *v, int type,
                          int64_t max_rows, hipStream_t st) {
  ReadArgs a{c, s, {static_cast<char *>(k), static_cast<char *>(v)},
             pages_touched(std::min<int64_t>(max_rows, s.rows), c.shift, s.batch)};
  const dim3 grid((unsigned)a.per * (unsigned)s.batch, (unsigned)(2 * c.heads));
  return by_type(type, e4m3, [&](auto t, auto f) {
    hipLaunchKernelGGL((kv_read_kernel<decltype(t)::value, decltype(f)::value>), grid,
                       dim3(kThreads), 0, st, a);
    return hipGetLastError();
  });
}

}  // namespace slq

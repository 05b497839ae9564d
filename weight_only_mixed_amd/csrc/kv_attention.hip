// Causal attention of ragged queries over the paged 8-bit cache.
//
//   s_j = scale * sk(page j) * (q . kcode_j),  p = softmax(s),
//   o   = sum_j p_j * sv(page j) * vcode_j
//
// The query heads that share a kv head are rows of one product (row = query *
// group + head in group), so each cached byte is read once per kv head.
// Codes go to binary16 (exact: at most 8 significant bits, |code| <= 448) and
// feed 16x16x32 MFMAs; q goes there too, after its row is shifted by a power
// of two to a largest element in [1, 2), which keeps every product exact down
// to 2^-25 of the row's largest element whatever the range of q.
//
// Scores are computed transposed, S^T = K q^T (rows: tokens, columns:
// queries): lane l then holds, for query l % 16, tokens 4 (l/16) + v of each
// 16-token tile, which is the operand layout of the second product
// O^T = V^T P^T if its 32 k slots are numbered as the tokens of two such tiles
// (slot 8 g + t: token 4 g + t of tile 0 for t < 4, token 4 g + t - 4 of tile
// 1 above).  So probabilities never leave their lane, and the softmax
// statistics of a query live in the lanes that hold its accumulators.  V rows
// are loaded token by token, each lane taking the same dim / 16 bytes of the 8
// tokens of its slots; the byte transposition is part of the conversion.
// Nothing passes through shared memory before the epilogue.
//
// Bound of single tokens: HBM.  Measured, 64 sequences of 300 .. 8192 tokens, 8 kv
// heads of 4 query heads x 128, INT8 (597 MB): 140 us and 9 us of joining, 4.3 TB/s
// against 6.3 of a plain read; two sequences of about 131072, 8 query heads per kv
// head, E4M3 (513 MB): 105 + 9 us, 4.9 TB/s.  Conversions and softmax take about
// half of the vector issue slots while the loads are out; waves in flight (four per
// SIMD), not their arithmetic, set the rate.  One sequence of 1003 tokens: 13 us.
//
// Probabilities are taken relative to a reference m that a score has reached,
// and that follows the running maximum only when that has risen by more than
// 2^4 (otherwise some query of a tile has a new maximum nearly every time, and
// all accumulators would be rescaled for a change of no consequence).  They
// enter the second product as binary16 of p * 2^11 * sv / R with R the largest
// sv met so far (folded into the accumulator when it grows): at most 2^15, and
// each loses at most 2^-36 of m's weight where binary16 runs out of exponent.
#include <float.h>

#include <algorithm>
#include <utility>

#include "serve.h"
#include "slq_device.h"

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

namespace slq {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kBlock = 32;            // tokens per wave and step
constexpr int kWideSpan = 1280;       // tokens that 8 waves take in one piece
constexpr float kPUnit = 2048.f;      // probabilities are held times this
constexpr float kSlack = 4.f;         // and may reach 2^kSlack
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_hw(float v) { return __builtin_amdgcn_exp2f(v); }

__device__ __forceinline__ f32x4_t mfma16h(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t h2_bits(f16x2_t v) { return __builtin_bit_cast(uint32_t, v); }

// 1024 + (b + 128) in both halves, minus 1152: two signed bytes as binary16.
// `v`: the bytes in bits 0..7 and 16..23, zero elsewhere.
__device__ __forceinline__ uint32_t int8_pair(uint32_t v) {
  const f16x2_t bias = {(_Float16)1152.f, (_Float16)1152.f};
  return h2_bits(__builtin_bit_cast(f16x2_t, v ^ 0x64806480u) - bias);
}

// Four codes of a word as binary16.
template <bool E4M3>
__device__ __forceinline__ u32x2_t codes4(uint32_t w) {
  u32x2_t r;
  if constexpr (E4M3) {
    r[0] = h2_bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, false));
    r[1] = h2_bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, true));
  } else {
    const f16x2_t bias = {(_Float16)1152.f, (_Float16)1152.f};
    const uint32_t u = w ^ 0x80808080u;   // b + 128; 0x64 above it makes 1024 + (b + 128)
    r[0] = h2_bits(__builtin_bit_cast(f16x2_t, perm(0x64646464u, u, 0x04010400u)) - bias);
    r[1] = h2_bits(__builtin_bit_cast(f16x2_t, perm(0x64646464u, u, 0x04030402u)) - bias);
  }
  return r;
}

// Column c (0..3) of two words of different tokens: (a's byte c, b's byte c).
// E4M3 converts the pairs of columns 0/1 and 2/3 of one permuted word.
template <bool E4M3, int C>
__device__ __forceinline__ uint32_t column_pair(uint32_t a, uint32_t b) {
  if constexpr (E4M3) {
    const uint32_t w = C < 2 ? perm(b, a, 0x05010400u) : perm(b, a, 0x07030602u);
    return h2_bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, (C & 1) != 0));
  } else {
    return int8_pair(perm(b, a, 0x0c000c00u | (uint32_t)C | (uint32_t)(4 + C) << 16));
  }
}

// A load through the scalar cache, of memory that no one writes while the kernel
// runs and from an address that is the same in every lane: it takes no vector
// register and does not queue behind the loads of codes.
template <typename T>
__device__ __forceinline__ T uniform_load(const T *p) {
  typedef const __attribute__((address_space(4))) T *Const;
  return *(Const)(uintptr_t)p;
}

template <typename F, int... I>
__device__ __forceinline__ void for_each_int(F &f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>()), ...);
}

__device__ __forceinline__ float shfl_x(float v, int o) { return __shfl_xor(v, o, kWave); }
// Over the four lanes that hold one query (l, l^16, l^32, l^48).
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, shfl_x(v, 16));
  return fmaxf(v, shfl_x(v, 32));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += shfl_x(v, 16);
  return v + shfl_x(v, 32);
}

__device__ __forceinline__ uint16_t to_out(float v, bool bf16) {
  return bf16 ? __builtin_bit_cast(uint16_t, (__bf16)v) : __builtin_bit_cast(uint16_t, (_Float16)v);
}

__device__ __forceinline__ KvSpan uniform_span(const KvAttnArgs &a, int b) {
  // kv_span on copies of the three entries it reads
  const int32_t cu[2] = {uniform_load(a.s.cu + b), uniform_load(a.s.cu + b + 1)};
  const int32_t len = uniform_load(a.s.lens + b);
  SeqView one = a.s;
  one.cu = cu;
  one.lens = &len;
  return kv_span(one, a.c.shift, 0);
}

// Tokens per split.  The host knows bounds, not lengths, and a split size that
// fits the longest sequence leaves the chip half idle on ragged batches (64
// lengths of 300 .. 8192: 163 us, the compute units busy for 105 of them), so
// every workgroup sums the lengths itself: an even share of all visible tokens
// for each of a.share workgroups.  Whole numbers and one division of doubles:
// the joining kernel comes to the same size.  Every lane returns it.
__device__ __forceinline__ int split_size(const KvAttnArgs &a) {
  if (a.share == 0) return a.chunk;
  double total = 0.0;
  for (int b = threadIdx.x & (kWave - 1); b < a.s.batch; b += kWave) {
    const KvSpan sp = kv_span(a.s, a.c.shift, b);
    if (sp.n > 0) {
      const KvRange r = kv_visible(sp, a.window, 0, sp.n - 1);
      total += (double)(r.hi - r.lo);
    }
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) total += __shfl_xor(total, o, kWave);
  const double size = ceil(total * (double)(a.c.heads * a.tiles) / (double)a.share);
  // the same in every lane; said so, or all addresses become per-lane values
  return __builtin_amdgcn_readfirstlane((int)fmin(fmax(size, (double)a.chunk), 1073741824.0));
}

// What the workgroups of one (sequence, tile of query rows) share: the token
// range, how many splits of it hold any token, and their size.
struct TileRange {
  int lo, hi, start, active, chunk;
};
__device__ __forceinline__ TileRange tile_range(const KvAttnArgs &a, const KvSpan &sp, int rho0,
                                                int rho1, int size) {
  const KvRange r = kv_visible(sp, a.window, rho0 / a.group, (rho1 - 1) / a.group);
  TileRange t;
  t.lo = r.lo;
  t.hi = r.hi;
  t.start = r.hi > r.lo ? r.lo & ~(kBlock - 1) : r.hi;   // nothing to walk where empty
  const int n = r.hi - t.start;
  // as many splits as `size` asks for, within the grid, of equal size
  const int want = min(max((n - 1) / size + 1, 1), a.splits);
  t.chunk = ((n - 1) / want + a.grain) / a.grain * a.grain;
  t.chunk = max(t.chunk, a.grain);
  t.active = n > 0 ? min((n - 1) / t.chunk + 1, a.splits) : 0;
  return t;
}

// Four waves per SIMD for single tokens: what hides the loads is waves, not
// blocks in flight per wave.
// W waves share a workgroup's tokens: 4, or 8 for a short sequence in one piece.
template <int D, bool E4M3, int NT, int W>
__global__ __launch_bounds__(W *kWave, (D <= 128 && NT == 1 && W == 4 ? 4 : 1)) void kv_attn_kernel(KvAttnArgs a) {
  constexpr int KS = D / 32;      // MFMA k steps of q . k
  constexpr int VJ = D / 16;      // bytes of a V row per lane, and MFMAs of p . v
  constexpr int KL = D / 64;      // 16-byte K loads per token and lane
  constexpr int VW = VJ / 4;      // 32-bit words of a V row per lane
  constexpr int ROWS = 16 * NT;
  constexpr int OP = D + 4;       // pitch of a query's outputs in LDS
  __shared__ float o_lds[W][16 * OP];
  __shared__ float m_lds[W][16], l_lds[W][16];

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int col = lane & 15, g = lane >> 4;
  const int slot = a.heads_first ? blockIdx.y : blockIdx.x;
  const int b = slot / a.splits, split = slot % a.splits;
  const int h = a.heads_first ? blockIdx.x : blockIdx.y;
  const int size = split_size(a);
  const KvSpan sp = uniform_span(a, b);
  const int total = sp.n * a.group;
  const uint8_t *kbase = a.c.codes[0] + (int64_t)h * a.c.head_stride;
  const uint8_t *vbase = a.c.codes[1] + (int64_t)h * a.c.head_stride;
  // lane offsets into a 16-token tile: 16 bytes of K row col, V rows 4 g ..
  const uint32_t koff = (uint32_t)(col * (int)a.c.token_stride + 16 * g);
  const uint32_t voff = (uint32_t)(4 * g * (int)a.c.token_stride + VJ * col);

  for (int rho0 = blockIdx.z * ROWS; rho0 < total; rho0 += a.tiles * ROWS) {
    const int rho1 = min(rho0 + ROWS, total);
    const TileRange tr = tile_range(a, sp, rho0, rho1, size);
    if (split >= max(tr.active, a.splits == 1 ? 1 : 0)) continue;   // nothing here (uniform)
    const int t0 = tr.start + split * tr.chunk;
    const int t1 = split == a.splits - 1 ? tr.hi : min(tr.hi, t0 + tr.chunk);

    // queries: lane (col, g) holds dims 64 h2 + 16 g + 8 e + t of query col
    u32x4_t qf[NT][KS];
    float qs[NT];
    int pos[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int rho = rho0 + 16 * n + col;
      const bool ok = rho < rho1;
      const int i = (ok ? rho : rho0) / a.group, hd = (ok ? rho : rho0) % a.group;
      pos[n] = ok ? sp.pos0 + i : -1;
      const uint16_t *qp = a.q + (int64_t)(sp.row0 + i) * a.q_row +
                           (int64_t)(h * a.group + hd) * a.q_head + 16 * g;
      u32x4_t raw[KS];
#pragma unroll
      for (int k = 0; k < KS; ++k)
        raw[k] = ok ? *reinterpret_cast<const u32x4_t *>(qp + 64 * (k >> 1) + 8 * (k & 1))
                    : u32x4_t{0, 0, 0, 0};
      qs[n] = a.scale_log2;
      if (a.bf16) {
        float mx = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int w = 0; w < 4; ++w)
            mx = fmaxf(mx, fmaxf(__builtin_bit_cast(float, (raw[k][w] << 16) & 0x7FFFFFFFu),
                                 __builtin_bit_cast(float, raw[k][w] & 0x7FFF0000u)));
        mx = quad_max(mx);
        const int e = (int)(__builtin_bit_cast(uint32_t, mx) >> 23) - 127;
        const float down = ldexpf(1.f, -(e / 2)), down2 = ldexpf(1.f, -(e - e / 2));
        qs[n] = a.scale_log2 * ldexpf(1.f, e / 2) * ldexpf(1.f, e - e / 2);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float lo = __builtin_bit_cast(float, raw[k][w] << 16) * down * down2;
            const float hi = __builtin_bit_cast(float, raw[k][w] & 0xFFFF0000u) * down * down2;
            qf[n][k][w] = h2_bits(f16x2_t{(_Float16)lo, (_Float16)hi});
          }
      } else {
#pragma unroll
        for (int k = 0; k < KS; ++k) qf[n][k] = raw[k];
      }
    }

    f32x4_t acc[NT][VJ];
    float m[NT], l[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n] = -FLT_MAX;
      l[n] = 0.f;
#pragma unroll
      for (int j = 0; j < VJ; ++j) acc[n][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    float unit = 0.f, inv_unit = 0.f;   // R and kPUnit / R
    // tokens every query of this tile sees
    const int all_hi = min(tr.hi, sp.pos0 + rho0 / a.group + 1);
    const int last_pos = sp.pos0 + (rho1 - 1) / a.group;
    const int all_lo = a.window > 0 ? max(tr.lo, last_pos - a.window + 1) : tr.lo;

    // the two 16-token tiles of a wave's step: their pages (a tile never crosses
    // a page), scales and codes
    struct Block {
      int id[2];
      float sk[2], sv[2];
      u32x4_t kw[2][KL];
      uint32_t vw[2][4][VW];
    };
    auto entries = [&](int blk, int (&e)[2]) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
        e[u] = uniform_load(a.s.table + kv_entry(a.s, b, (blk + 16 * u) >> a.c.shift));
    };
    auto load = [&](int blk, const int (&e)[2], Block &x) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int tok = blk + 16 * u;
        // a tile wholly outside the visible range is not looked at: its page may
        // belong to someone else by now
        x.id[u] = tok < tr.hi && tok + 16 > tr.lo
                      ? kv_page_of(a.s, a.c.pages, tok >> a.c.shift, e[u]) : -1;
        x.sk[u] = x.sv[u] = 0.f;
        if (x.id[u] >= 0) {
          const int64_t at = (int64_t)x.id[u] * a.c.page_stride +
                             (int64_t)(tok & ((1 << a.c.shift) - 1)) * a.c.token_stride;
          x.sk[u] = uniform_load(a.c.scales[0] + (int64_t)x.id[u] * a.c.heads + h);
          x.sv[u] = uniform_load(a.c.scales[1] + (int64_t)x.id[u] * a.c.heads + h);
          const uint8_t *kp = kbase + at, *vp = vbase + at;
#pragma unroll
          for (int k = 0; k < KL; ++k) x.kw[u][k] = *reinterpret_cast<const u32x4_t *>(kp + koff + 64 * k);
#pragma unroll
          for (int t = 0; t < 4; ++t, vp += a.c.token_stride) {
            if constexpr (VW == 1) x.vw[u][t][0] = *reinterpret_cast<const uint32_t *>(vp + voff);
            else if constexpr (VW == 2) {
              const u32x2_t w = *reinterpret_cast<const u32x2_t *>(vp + voff);
              x.vw[u][t][0] = w[0];
              x.vw[u][t][1] = w[1];
            } else {
              const u32x4_t w = *reinterpret_cast<const u32x4_t *>(vp + voff);
#pragma unroll
              for (int i = 0; i < 4; ++i) x.vw[u][t][i] = w[i];
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < KL; ++k) x.kw[u][k] = u32x4_t{0, 0, 0, 0};
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < VW; ++i) x.vw[u][t][i] = 0u;
        }
      }
    };
    auto step = [&](int blk, Block &x) {
      const int (&id)[2] = x.id;
      const float (&sk)[2] = x.sk, (&sv)[2] = x.sv;
      const u32x4_t (&kw)[2][KL] = x.kw;
      uint32_t (&vw)[2][4][VW] = x.vw;
      const bool plain = blk >= all_lo && blk + kBlock <= all_hi && id[0] >= 0 && id[1] >= 0;
      if (!plain) {   // rows outside every query's range may hold anything: 0 * NaN
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const int tok = blk + 16 * u + 4 * g + t;
            const bool in = tok >= tr.lo && tok < tr.hi;
#pragma unroll
            for (int i = 0; i < VW; ++i) vw[u][t][i] = in ? vw[u][t][i] : 0u;
          }
      }
      const float grown = fmaxf(unit, fmaxf(sv[0], sv[1]));
      if (grown > unit) {
        const float f = unit / grown;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < VJ; ++j) acc[n][j] *= f;
        unit = grown;
        inv_unit = kPUnit / grown;
      }

      f32x4_t s[NT][2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int n = 0; n < NT; ++n) s[n][u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const u32x2_t c0 = codes4<E4M3>(kw[u][k >> 1][2 * (k & 1)]);
          const u32x2_t c1 = codes4<E4M3>(kw[u][k >> 1][2 * (k & 1) + 1]);
          const u32x4_t kf = {c0[0], c0[1], c1[0], c1[1]};
#pragma unroll
          for (int n = 0; n < NT; ++n) s[n][u] = mfma16h(kf, qf[n][k], s[n][u]);
        }
      }
      u32x4_t pf[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float f = sk[u] * qs[n];
#pragma unroll
          for (int v = 0; v < 4; ++v) s[n][u][v] *= f;
        }
        if (!plain) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const int tok = blk + 16 * u + 4 * g + v;
              const bool in = id[u] >= 0 && tok <= pos[n] && tok < tr.hi && tok >= tr.lo &&
                              (a.window <= 0 || tok > pos[n] - a.window);
              s[n][u][v] = in ? s[n][u][v] : -INFINITY;
            }
        }
        float mx = s[n][0][0];
#pragma unroll
        for (int v = 1; v < 8; ++v) mx = fmaxf(mx, s[n][v >> 2][v & 3]);
        if (__any(mx > m[n] + kSlack)) {
          const float mn = fmaxf(m[n], quad_max(mx));
          const float f = exp2_hw(m[n] - mn);
          l[n] *= f;
#pragma unroll
          for (int j = 0; j < VJ; ++j) acc[n][j] *= f;
          m[n] = mn;
        }
        float p[8];
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          p[v] = exp2_hw(s[n][v >> 2][v & 3] - m[n]);
          l[n] += p[v];
          p[v] *= sv[v >> 2] * inv_unit;
        }
#pragma unroll
        for (int w = 0; w < 4; ++w)
          pf[n][w] = h2_bits(f16x2_t{(_Float16)p[2 * w], (_Float16)p[2 * w + 1]});
      }
      auto column = [&](auto jc) {
        constexpr int J = decltype(jc)::value, I = J / 4, C = J % 4;
        const u32x4_t vf = {column_pair<E4M3, C>(vw[0][0][I], vw[0][1][I]),
                            column_pair<E4M3, C>(vw[0][2][I], vw[0][3][I]),
                            column_pair<E4M3, C>(vw[1][0][I], vw[1][1][I]),
                            column_pair<E4M3, C>(vw[1][2][I], vw[1][3][I])};
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n][J] = mfma16h(vf, pf[n], acc[n][J]);
      };
      for_each_int(column, std::make_integer_sequence<int, VJ>());
    };
    // (a second block in flight per wave costs more occupancy than it hides:
    // 237 us against 188 for 64 sequences of up to 8192 tokens)
    int e[2];   // table entries, read a step ahead
    entries(t0 + kBlock * wave, e);
    for (int blk = t0 + kBlock * wave; blk < t1; blk += kBlock * W) {
      Block x;
      load(blk, e, x);
      entries(blk + kBlock * W, e);
      step(blk, x);
    }

    // the four waves' parts of each query, joined in wave order
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float lt = quad_sum(l[n]), f = unit * (1.f / kPUnit);
      __syncthreads();
#pragma unroll
      for (int v = 0; v < 4; ++v)
#pragma unroll
        for (int j = 0; j < VJ; j += 4)
          *reinterpret_cast<f32x4_t *>(&o_lds[wave][col * OP + (4 * g + v) * VJ + j]) =
              f32x4_t{acc[n][j][v] * f, acc[n][j + 1][v] * f, acc[n][j + 2][v] * f,
                      acc[n][j + 3][v] * f};
      if (g == 0) {
        m_lds[wave][col] = m[n];
        l_lds[wave][col] = lt;
      }
      __syncthreads();
      const int qc = threadIdx.x / 16, d0 = (threadIdx.x % 16) * VJ;
      const int rho = rho0 + 16 * n + qc;
      if (threadIdx.x < 256 && rho < rho1) {
        float mt = m_lds[0][qc];
#pragma unroll
        for (int w = 1; w < W; ++w) mt = fmaxf(mt, m_lds[w][qc]);
        float lsum = 0.f, o[VJ] = {};
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float f2 = l_lds[w][qc] > 0.f ? exp2_hw(m_lds[w][qc] - mt) : l_lds[w][qc];
          lsum += f2 * l_lds[w][qc];
#pragma unroll
          for (int j = 0; j < VJ; ++j) o[j] += f2 * o_lds[w][qc * OP + d0 + j];
        }
        const bool none = lsum == 0.f;
        const float inv = none ? 0.f : 1.f / lsum;
        const float lse2 = none ? -INFINITY : mt + log2f(lsum);
        const int i = rho / a.group, hd = rho % a.group;
        const int64_t row = (int64_t)(sp.row0 + i) * a.heads_q + h * a.group + hd;
        if (a.splits == 1) {
          uint16_t *op = a.out + row * D + d0;
          union {
            uint16_t e[VJ];
            u32x2_t w[VJ / 4];
          } t;
#pragma unroll
          for (int j = 0; j < VJ; ++j) t.e[j] = to_out(o[j] * inv, a.bf16);
#pragma unroll
          for (int j = 0; j < VJ / 4; ++j) reinterpret_cast<u32x2_t *>(op)[j] = t.w[j];
          if (a.lse && d0 == 0) a.lse[row] = lse2 * kLn2;
        } else {
          const int64_t at = (int64_t)split * a.s.rows * a.heads_q + row;
#pragma unroll
          for (int j = 0; j < VJ; j += 4)
            *reinterpret_cast<f32x4_t *>(a.part_o + at * D + d0 + j) =
                f32x4_t{o[j] * inv, o[j + 1] * inv, o[j + 2] * inv, o[j + 3] * inv};
          if (d0 == 0) a.part_lse[at] = lse2;
        }
      }
    }
  }
}

// ---- prompt chunks: many query rows per kv head ----
//
// One workgroup of 8 waves takes 256 query rows of a kv head, 32 per wave, and
// walks the tokens in tiles of 8192 / dim.  A tile's codes are converted once
// for all waves: every thread loads 16 bytes of K and a 4 x 4 block of V a tile
// ahead, and writes binary16 to one of two buffers in shared memory, K as
// [token][dim], V transposed as [dim][token] with the tokens of each 16 in the
// order of the second product's k slots.  The products are 32x32x16 MFMAs in
// the transposed form of the decode kernel (S^T = K q^T, O^T = V^T P^T), so
// probabilities stay in their lane here too and a wave's outputs need no
// other wave.  Rows in shared memory are swizzled in 16-byte chunks so that
// both the operand reads (neighbouring rows) and the transposed writes (every
// fourth row) spread over the banks.
//
// Measured, 4 x 2048 rows of 4 query heads per kv head against 4212 .. 8192 tokens,
// 8 kv heads x 128, INT8 (768 GFLOP): 1.00 to 1.14 ms, 670 to 770 TFLOP/s (a large
// library product reaches 1296 here).  The matrix units are busy for 40% of the
// cycles and the vector units for 56%; shared memory serves operands in 41%.  With
// the conversions taken out it takes 0.91 ms instead of 1.18, without softmax 1.04,
// without both 0.77: operand reads from shared memory, conversion and softmax share
// the rest.  Two waves of a SIMD half a tile apart behind two barriers a tile (one
// in its products while the other does softmax) was slower, 1.38 ms against 1.23.
constexpr int kPromptThreads = 512;
constexpr int kPromptRows = 256;

typedef float f32x16v __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16v mfma32h(u32x4_t a, u32x4_t b, f32x16v c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a),
                                                __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

template <int D>
struct PromptTile {
  static constexpr int kTok = 8192 / D;          // tokens per tile: 128, 64, 32
  static constexpr int kGroups = kTok / 16;      // 16-token groups (one page each)
  static constexpr int kBytes = kTok * D * 2;    // of K, and of V
  // 16-byte chunk c of K row `tok`
  static __device__ __forceinline__ int k_at(int tok, int c) {
    return tok * (D * 2) + ((c ^ (tok & 7)) << 4);
  }
  // 16-byte chunk c of V^T row d
  static __device__ __forceinline__ int v_at(int d, int c) {
    const int f = D == 256 ? ((d >> 1) ^ (d >> 3)) & 3 : ((d >> 2) ^ (d << 1)) & 7;
    return d * (kTok * 2) + ((c ^ f) << 4);
  }
};

template <int D, bool E4M3>
__global__ __launch_bounds__(kPromptThreads, 2) void kv_prompt_kernel(KvAttnArgs a) {
  typedef PromptTile<D> Tile;
  constexpr int TOK = Tile::kTok, GR = Tile::kGroups;
  constexpr int TT = TOK / 32;      // 32-token tiles of S
  constexpr int ST = TT < 2 ? TT : 2, SG = 2 * ST;   // of these at a time, and their groups
  constexpr int KS = D / 16;        // k steps of q . k
  constexpr int DT = D / 32;        // 32-dim tiles of the output
  __shared__ __attribute__((aligned(16))) unsigned char k_lds[2][Tile::kBytes];
  __shared__ __attribute__((aligned(16))) unsigned char v_lds[2][Tile::kBytes];
  __shared__ float sk_lds[2][GR], sv_lds[2][GR];   // scales per group; sk < 0: no such tokens

  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int col = lane & 31, half = lane >> 5;
  // heads vary fastest over the workgroups: neighbours go to different chiplets,
  // and the tiles of one head's tokens share a chiplet's L2
  const int h = blockIdx.x, b = blockIdx.y / a.splits, split = blockIdx.y % a.splits;
  const int size = split_size(a);
  const KvSpan sp = uniform_span(a, b);
  const int total = sp.n * a.group;
  const uint8_t *kbase = a.c.codes[0] + (int64_t)h * a.c.head_stride;
  const uint8_t *vbase = a.c.codes[1] + (int64_t)h * a.c.head_stride;

  // what this thread loads: 16 bytes of K row kt, words of 4 V rows from vt on
  const int kt = tid / (D / 16), kc = tid % (D / 16);
  const int vt = 4 * (tid / (D / 4)), vd = 4 * (tid % (D / 4));
  const int wtok = wave * (TOK / 8);   // the wave's tokens lie in one group of 16
  // offsets from the wave's first row: the same for every tile
  const uint32_t koff = (uint32_t)((kt - wtok) * (int)a.c.token_stride + 16 * kc);
  const uint32_t voff = (uint32_t)((vt - wtok) * (int)a.c.token_stride + vd);
  // where the converted codes go (in_vgpr: kept, not recomputed every tile)
  const int quad = (vt >> 2) & 3, chunk = 2 * (vt >> 4) + (quad & 1), part = 8 * (quad >> 1);
  const uint32_t kdst0 = in_vgpr(Tile::k_at(kt, 2 * kc)), kdst1 = in_vgpr(Tile::k_at(kt, 2 * kc + 1));
  uint32_t vdst[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) vdst[c] = in_vgpr(Tile::v_at(vd + c, chunk) + part);

  // where a lane reads operands: chunk 2 k + half of K row 32 t + col is at ksrc ^
  // 32 k, plus t rows of 32, and chunk 2 g + half of V^T row 32 j + col likewise
  // (a swizzle depends on the row's low bits only)
  const uint32_t ksrc = Tile::k_at(col, half), vsrc = Tile::v_at(col, half);

  // late tiles see the most tokens: they start first
  const int ntiles = (total + kPromptRows - 1) / kPromptRows;
  for (int tile = ntiles - 1 - (int)blockIdx.z; tile >= 0; tile -= a.tiles) {
    const int rho0 = tile * kPromptRows, rho1 = min(rho0 + kPromptRows, total);
    const TileRange tr = tile_range(a, sp, rho0, rho1, size);
    if (split >= max(tr.active, a.splits == 1 ? 1 : 0)) continue;   // nothing here (uniform)
    const int t0 = tr.start + split * tr.chunk;
    const int t1 = split == a.splits - 1 ? tr.hi : min(tr.hi, t0 + tr.chunk);

    // queries: lane (col, half) holds dims 16 k + 8 half + t of query col
    const int rho = rho0 + 32 * wave + col;
    const bool mine = rho < rho1;
    const int qi = (mine ? rho : rho0) / a.group, qh = (mine ? rho : rho0) % a.group;
    const int pos = mine ? sp.pos0 + qi : -1;
    u32x4_t qf[KS];
    float qs;
    {
      const uint16_t *qp = a.q + (int64_t)(sp.row0 + qi) * a.q_row +
                           (int64_t)(h * a.group + qh) * a.q_head + 8 * half;
#pragma unroll
      for (int k = 0; k < KS; ++k)
        qf[k] = mine ? *reinterpret_cast<const u32x4_t *>(qp + 16 * k) : u32x4_t{0, 0, 0, 0};
      qs = fabsf(a.scale_log2);
      if (a.bf16) {
        float mx = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int w = 0; w < 4; ++w)
            mx = fmaxf(mx, fmaxf(__builtin_bit_cast(float, (qf[k][w] << 16) & 0x7FFFFFFFu),
                                 __builtin_bit_cast(float, qf[k][w] & 0x7FFF0000u)));
        mx = fmaxf(mx, shfl_x(mx, 32));
        const int e = (int)(__builtin_bit_cast(uint32_t, mx) >> 23) - 127;
        const float down = ldexpf(1.f, -(e / 2)), down2 = ldexpf(1.f, -(e - e / 2));
        qs = qs * ldexpf(1.f, e / 2) * ldexpf(1.f, e - e / 2);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float lo = __builtin_bit_cast(float, qf[k][w] << 16) * down * down2;
            const float hi = __builtin_bit_cast(float, qf[k][w] & 0xFFFF0000u) * down * down2;
            qf[k][w] = h2_bits(f16x2_t{(_Float16)lo, (_Float16)hi});
          }
      }
      // the sign of the scale goes to q, so that score factors are not negative
      const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int w = 0; w < 4; ++w) qf[k][w] ^= flip;
    }
    // tokens that all of the wave's queries see, and that any of them sees
    const int wr0 = min(rho0 + 32 * wave, rho1 - 1), wr1 = min(rho0 + 32 * wave + 32, rho1) - 1;
    const bool wave_on = rho0 + 32 * wave < rho1;
    const int first_pos = sp.pos0 + wr0 / a.group, last_pos = sp.pos0 + wr1 / a.group;
    const int all_hi = min(tr.hi, first_pos + 1);
    const int all_lo = a.window > 0 ? max(tr.lo, last_pos - a.window + 1) : tr.lo;
    const int any_hi = min(tr.hi, last_pos + 1);
    const int any_lo = a.window > 0 ? max(tr.lo, first_pos - a.window + 1) : tr.lo;

    f32x16v acc[DT];
#pragma unroll
    for (int j = 0; j < DT; ++j) acc[j] = f32x16v{};
    float m = -FLT_MAX, l = 0.f, unit = 0.f, inv_unit = 0.f;

    u32x4_t kreg;
    uint32_t vreg[4];
    float skreg, svreg;
    auto entry = [&](int base) {
      return uniform_load(a.s.table + kv_entry(a.s, b, (base + wtok) >> a.c.shift));
    };
    auto load = [&](int base, int e) {
      const int tok = (base + wtok) & ~15;   // the group's first: its waves agree
      const int id = tok < t1 && tok + 16 > tr.lo
                         ? kv_page_of(a.s, a.c.pages, tok >> a.c.shift, e) : -1;
      kreg = u32x4_t{0, 0, 0, 0};
      vreg[0] = vreg[1] = vreg[2] = vreg[3] = 0u;
      skreg = -1.f;
      svreg = 0.f;
      if (id >= 0) {
        const int slot = (base + wtok) & ((1 << a.c.shift) - 1);
        const int64_t at = (int64_t)id * a.c.page_stride + (int64_t)slot * a.c.token_stride;
        kreg = *reinterpret_cast<const u32x4_t *>(kbase + at + koff);
        const uint8_t *vp = vbase + at;
#pragma unroll
        for (int t = 0; t < 4; ++t, vp += a.c.token_stride)
          vreg[t] = *reinterpret_cast<const uint32_t *>(vp + voff);
        skreg = uniform_load(a.c.scales[0] + (int64_t)id * a.c.heads + h);
        svreg = uniform_load(a.c.scales[1] + (int64_t)id * a.c.heads + h);
      }
    };
    auto store = [&](int base, int buf) {
      const u32x2_t c0 = codes4<E4M3>(kreg[0]), c1 = codes4<E4M3>(kreg[1]);
      const u32x2_t c2 = codes4<E4M3>(kreg[2]), c3 = codes4<E4M3>(kreg[3]);
      *reinterpret_cast<u32x4_t *>(&k_lds[buf][kdst0]) =
          u32x4_t{c0[0], c0[1], c1[0], c1[1]};
      *reinterpret_cast<u32x4_t *>(&k_lds[buf][kdst1]) =
          u32x4_t{c2[0], c2[1], c3[0], c3[1]};
      // rows outside the visible range may hold anything: 0 * NaN
      if (base + wtok < tr.lo || base + wtok + TOK / 8 > tr.hi) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (base + vt + t < tr.lo || base + vt + t >= tr.hi) vreg[t] = 0u;
      }
      *reinterpret_cast<u32x2_t *>(&v_lds[buf][vdst[0]]) =
          u32x2_t{column_pair<E4M3, 0>(vreg[0], vreg[1]), column_pair<E4M3, 0>(vreg[2], vreg[3])};
      *reinterpret_cast<u32x2_t *>(&v_lds[buf][vdst[1]]) =
          u32x2_t{column_pair<E4M3, 1>(vreg[0], vreg[1]), column_pair<E4M3, 1>(vreg[2], vreg[3])};
      *reinterpret_cast<u32x2_t *>(&v_lds[buf][vdst[2]]) =
          u32x2_t{column_pair<E4M3, 2>(vreg[0], vreg[1]), column_pair<E4M3, 2>(vreg[2], vreg[3])};
      *reinterpret_cast<u32x2_t *>(&v_lds[buf][vdst[3]]) =
          u32x2_t{column_pair<E4M3, 3>(vreg[0], vreg[1]), column_pair<E4M3, 3>(vreg[2], vreg[3])};
      if (lane == 0) {   // waves of one group write the same values
        sk_lds[buf][wtok >> 4] = skreg;
        sv_lds[buf][wtok >> 4] = svreg;
      }
    };

    int e_next = entry(t0 + TOK);   // table entries, read a tile ahead
    __syncthreads();   // the previous tile's last readers
    load(t0, entry(t0));
    store(t0, 0);
    __syncthreads();
    for (int base = t0, buf = 0; base < t1; base += TOK, buf ^= 1) {
      const bool more = base + TOK < t1;
      if (more) {
        load(base + TOK, e_next);
        e_next = entry(base + 2 * TOK);
      }
      // at most 64 tokens at a time: scores and probabilities of more do not fit
      // beside the accumulators
#pragma unroll 1
      for (int sub = 0; sub < TT / ST; ++sub) {
        const int sbase = base + 32 * ST * sub;
        if (!wave_on || sbase >= any_hi || sbase + 32 * ST <= any_lo) continue;
        float f[SG], sv[SG];
        bool plain = sbase >= all_lo && sbase + 32 * ST <= all_hi;
        float grown = unit;
#pragma unroll
        for (int g = 0; g < SG; ++g) {
          f[g] = sk_lds[buf][SG * sub + g];
          sv[g] = sv_lds[buf][SG * sub + g];
          plain = plain && f[g] >= 0.f;
          grown = fmaxf(grown, sv[g]);
        }
        if (__any(grown > unit)) {   // the same in every lane
          const float c = unit / grown;
#pragma unroll
          for (int j = 0; j < DT; ++j) acc[j] *= c;
          unit = grown;
          inv_unit = kPUnit / grown;
        }
        // operand reads run kAhead products ahead: the compiler left alone reads
        // each operand right before its product and waits the whole read out
        constexpr int kAhead = 4, NS = KS * ST, NP = SG * DT;
        u32x4_t op[kAhead];
        auto k_op = [&](int i) {
          return *reinterpret_cast<const u32x4_t *>(
              &k_lds[buf][(ksrc ^ (uint32_t)(i / ST) << 5) + 32 * (ST * sub + i % ST) * (D * 2)]);
        };
        auto v_op = [&](int i) {
          return *reinterpret_cast<const u32x4_t *>(
              &v_lds[buf][(vsrc ^ (uint32_t)(SG * sub + i / DT) << 5) + 32 * (i % DT) * (TOK * 2)]);
        };
        f32x16v s[ST];
#pragma unroll
        for (int t = 0; t < ST; ++t) s[t] = f32x16v{};
#pragma unroll
        for (int i = 0; i < kAhead; ++i) op[i] = k_op(i);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          s[i % ST] = mfma32h(op[i % kAhead], qf[i / ST], s[i % ST]);
          op[i % kAhead] = i + kAhead < NS ? k_op(i + kAhead) : v_op(i + kAhead - NS);
          __builtin_amdgcn_sched_barrier(0);
        }
        // register v of tile t: token 32 t + 8 (v / 4) + 4 half + v % 4, group 2 t + v / 8
        if (__all(plain)) {
#pragma unroll
          for (int g = 0; g < SG; ++g) f[g] *= qs;
        } else {
#pragma unroll
          for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
              const int tok = sbase + 32 * t + 8 * (v >> 2) + 4 * half + (v & 3);
              const bool in = f[2 * t + (v >> 3)] >= 0.f && tok <= pos && tok < tr.hi &&
                              tok >= tr.lo && (a.window <= 0 || tok > pos - a.window);
              s[t][v] = in ? s[t][v] * (f[2 * t + (v >> 3)] * qs) : -INFINITY;
            }
#pragma unroll
          for (int g = 0; g < SG; ++g) f[g] = 1.f;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int g = 0; g < SG; ++g) {
          float x = s[g >> 1][8 * (g & 1)];
#pragma unroll
          for (int v = 1; v < 8; ++v) x = fmaxf(x, s[g >> 1][8 * (g & 1) + v]);
          mx = fmaxf(mx, x * f[g]);
        }
        if (__any(mx > m + kSlack)) {
          const float mn = fmaxf(m, fmaxf(mx, shfl_x(mx, 32)));
          const float c = exp2_hw(m - mn);
          l *= c;
#pragma unroll
          for (int j = 0; j < DT; ++j) acc[j] *= c;
          m = mn;
        }
        u32x4_t pf[SG];   // one k step of p . v per group of 16 tokens
#pragma unroll
        for (int g = 0; g < SG; ++g) {
          const float c = sv[g] * inv_unit;
          float p[8];
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            p[v] = exp2_hw(__builtin_fmaf(s[g >> 1][8 * (g & 1) + v], f[g], -m));
            l += p[v];
            p[v] *= c;
          }
#pragma unroll
          for (int w = 0; w < 4; ++w)
            pf[g][w] = h2_bits(f16x2_t{(_Float16)p[2 * w], (_Float16)p[2 * w + 1]});
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          acc[i % DT] = mfma32h(op[i % kAhead], pf[i / DT], acc[i % DT]);
          if (i + kAhead < NP) op[i % kAhead] = v_op(i + kAhead);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if (more) store(base + TOK, buf ^ 1);
      __syncthreads();
    }

    const float lsum = l + shfl_x(l, 32);
    if (mine) {
      const bool none = lsum == 0.f;
      const float inv = none ? 0.f : unit * (1.f / kPUnit) / lsum;
      const float lse2 = none ? -INFINITY : m + log2f(lsum);
      const int64_t row = (int64_t)(sp.row0 + qi) * a.heads_q + h * a.group + qh;
      if (a.splits == 1) {
#pragma unroll
        for (int j = 0; j < DT; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            union {
              uint16_t e[4];
              u32x2_t w;
            } t;
#pragma unroll
            for (int v = 0; v < 4; ++v) t.e[v] = to_out(acc[j][4 * i + v] * inv, a.bf16);
            *reinterpret_cast<u32x2_t *>(a.out + row * D + 32 * j + 8 * i + 4 * half) = t.w;
          }
        if (a.lse && half == 0) a.lse[row] = lse2 * kLn2;
      } else {
        const int64_t at = (int64_t)split * a.s.rows * a.heads_q + row;
#pragma unroll
        for (int j = 0; j < DT; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<f32x4_t *>(a.part_o + at * D + 32 * j + 8 * i + 4 * half) =
                f32x4_t{acc[j][4 * i] * inv, acc[j][4 * i + 1] * inv, acc[j][4 * i + 2] * inv,
                        acc[j][4 * i + 3] * inv};
        if (half == 0) a.part_lse[at] = lse2;
      }
    }
  }
}

// Joins the splits of each query row: one workgroup per row (9 us for 2048 rows; with
// one workgroup per 16 rows and splits read one after another it took 68 us at 128
// splits), the splits dealt to
// its four waves (fixed sums: split order within a wave, then wave order).  A
// row whose tile had no token (no split was active) gets 0 and -inf.
template <int D>
__global__ __launch_bounds__(kThreads) void kv_attn_join_kernel(KvAttnArgs a, int tile_rows) {
  constexpr int PER = D / kWave;   // outputs per lane
  constexpr int kU = 8;            // splits in flight per wave
  __shared__ float o_lds[kWaves][D];
  __shared__ float m_lds[kWaves], l_lds[kWaves];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int b = blockIdx.x, h = blockIdx.y;
  const int size = split_size(a);
  const KvSpan sp = uniform_span(a, b);
  const int total = sp.n * a.group;
  const int64_t step = (int64_t)a.s.rows * a.heads_q;
  for (int rho = blockIdx.z; rho < total; rho += gridDim.z) {
    const int rho0 = rho / tile_rows * tile_rows;
    const TileRange tr = tile_range(a, sp, rho0, min(rho0 + tile_rows, total), size);
    const int i = rho / a.group, hd = rho % a.group;
    const int64_t row = (int64_t)(sp.row0 + i) * a.heads_q + h * a.group + hd;
    float m = -INFINITY, l = 0.f, o[PER] = {};
    for (int base = wave; base < tr.active; base += kU * kWaves) {
      float e[kU], x[kU][PER];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int s = base + u * kWaves;
        const int64_t at = min(s, tr.active - 1) * step + row;
        e[u] = s < tr.active ? a.part_lse[at] : -INFINITY;
#pragma unroll
        for (int j = 0; j < PER; ++j) x[u][j] = a.part_o[at * D + lane * PER + j];
      }
      float top = m;
#pragma unroll
      for (int u = 0; u < kU; ++u) top = fmaxf(top, e[u]);
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (e[u] != e[u]) l = e[u];   // a maximum does not show it
      if (top == -INFINITY) continue;
      const float f = exp2_hw(m - top);
      l *= f;
#pragma unroll
      for (int j = 0; j < PER; ++j) o[j] *= f;
      m = top;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const float w = exp2_hw(e[u] - m);   // NaN where the split's sum was
        l += w;
        if (e[u] != -INFINITY)
#pragma unroll
          for (int j = 0; j < PER; ++j) o[j] += w * x[u][j];
      }
    }
    __syncthreads();   // the previous row's readers
    if (lane == 0) {
      m_lds[wave] = m;
      l_lds[wave] = l;
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) o_lds[wave][lane * PER + j] = o[j];
    __syncthreads();
    float top = m_lds[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) top = fmaxf(top, m_lds[w]);
    for (int d = threadIdx.x; d < D; d += kThreads) {
      float lsum = 0.f, v = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = m_lds[w] == -INFINITY && l_lds[w] == 0.f ? 0.f : exp2_hw(m_lds[w] - top);
        lsum += f * l_lds[w];
        v += f * o_lds[w][d];
      }
      a.out[row * D + d] = to_out(lsum == 0.f ? 0.f : v / lsum, a.bf16);
      if (a.lse && d == 0) a.lse[row] = lsum == 0.f ? -INFINITY : (top + log2f(lsum)) * kLn2;
    }
  }
}

template <int D, int NT, int W = kWaves>
void launch_decode(const KvAttnArgs &a, bool e4m3, hipStream_t st) {
  const unsigned slots = (unsigned)a.s.batch * (unsigned)a.splits, heads = (unsigned)a.c.heads;
  const dim3 grid(a.heads_first ? heads : slots, a.heads_first ? slots : heads, (unsigned)a.tiles);
  if (e4m3)
    hipLaunchKernelGGL((kv_attn_kernel<D, true, NT, W>), grid, dim3(W * kWave), 0, st, a);
  else
    hipLaunchKernelGGL((kv_attn_kernel<D, false, NT, W>), grid, dim3(W * kWave), 0, st, a);
}

template <int D>
void launch_prompt(const KvAttnArgs &a, bool e4m3, hipStream_t st) {
  const dim3 grid((unsigned)a.c.heads, (unsigned)a.s.batch * (unsigned)a.splits, (unsigned)a.tiles);
  if (e4m3)
    hipLaunchKernelGGL((kv_prompt_kernel<D, true>), grid, dim3(kPromptThreads), 0, st, a);
  else
    hipLaunchKernelGGL((kv_prompt_kernel<D, false>), grid, dim3(kPromptThreads), 0, st, a);
}

template <int D>
hipError_t launch_dim(const KvAttnArgs &a, bool e4m3, int nt, bool wide, hipStream_t st) {
  if (nt == 0) launch_prompt<D>(a, e4m3, st);
  else if (nt == 1 && wide) launch_decode<D, 1, 8>(a, e4m3, st);
  else if (nt == 1) launch_decode<D, 1>(a, e4m3, st);
  else if (nt == 2) {
    if constexpr (D <= 128) launch_decode<D, 2>(a, e4m3, st);
  } else if constexpr (D == 64) {
    launch_decode<D, 4>(a, e4m3, st);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const int tile_rows = nt == 0 ? kPromptRows : 16 * nt;
  hipLaunchKernelGGL((kv_attn_join_kernel<D>),
                     dim3((unsigned)a.s.batch, (unsigned)a.c.heads,
                          (unsigned)std::min<int64_t>(a.join_rows, 65535)),
                     dim3(kThreads), 0, st, a, tile_rows);
  return hipGetLastError();
}

}  // namespace

KvAttnPlan kv_attn_plan(int batch, int heads, int dim, int64_t capacity, int64_t rows, int heads_q,
                        int window, int64_t max_q, int64_t max_len) {
  KvAttnPlan p{};
  const int64_t group = heads_q / heads;
  // some sequence has at least its share of the rows, whatever max_q says (and
  // the workspace of splits is for all rows)
  const int64_t q = std::max(std::min(max_q, rows), (rows + batch - 1) / batch);
  const int64_t qrows = q * group;
  p.rows = (int)std::min<int64_t>(qrows, 65535);
  // As many query tiles per workgroup as the accumulators of 256 vector registers
  // allow.  (Wider instances, four tiles of 128 dims or two of 256, overflowed into
  // the accumulation registers; built with results in vector registers, those gave
  // wrong rows in the second pass of their tile loop.)
  const int widest = dim == 64 ? 4 : dim == 128 ? 2 : 1;
  p.nt = qrows > 64 ? 0 : std::min(widest, qrows <= 16 ? 1 : qrows <= 32 ? 2 : 4);
  const int tile_rows = p.nt == 0 ? kPromptRows : 16 * p.nt;
  p.tiles = (int)std::min<int64_t>((qrows + tile_rows - 1) / tile_rows, 65535);
  int64_t span = std::min(max_len, capacity);
  if (window > 0) span = std::min<int64_t>(span, (int64_t)window + tile_rows / group + 1);
  span += kBlock - 1;   // a range may start up to 31 tokens before its first visible one
  const int64_t base = (int64_t)batch * heads * p.tiles;
  // one step of every wave
  p.grain = p.nt == 0 ? 8192 / dim : kBlock * kWaves;
  // Workgroups to aim for: one per compute unit for the prompt kernel, two
  // rounds of those that run at once for the decode kernel (64 sequences of 300
  // .. 8192 tokens: 185 us with one round, 164 with two, 169 with four).
  const int64_t slots = p.nt == 0 ? 256 : p.nt == 1 && dim <= 128 ? 2048 : 1024;
  // Splits per sequence: room for one that is four times the mean; more
  // workgroups than slots need no splitting.  Each sequence's last split is
  // half full on average, hence the share.
  int64_t splits = std::min<int64_t>((4 * slots + base - 1) / base, (span + p.grain - 1) / p.grain);
  if (base >= (p.nt == 0 ? slots : 2 * slots)) splits = 1;
  // Short sequences, few of them: 8 waves on one piece instead of splits and a
  // second launch to join them.
  p.wide = p.nt == 1 && splits > 1 && span <= kWideSpan;
  if (p.wide) splits = 1;
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(splits, 256));
  p.share = p.splits > 1 ? (int)std::max<int64_t>(slots - base / 2, slots / 2) : 0;
  p.chunk = p.splits > 1 ? p.grain : 1 << 30;
  if (p.splits > 1)
    p.ws_bytes = (size_t)p.splits * (size_t)rows * (size_t)heads_q * (size_t)(dim + 1) * sizeof(float);
  return p;
}

hipError_t launch_kv_attention(KvAttnArgs a, bool e4m3, const KvAttnPlan &plan, void *ws,
                               hipStream_t st) {
  a.splits = plan.splits;
  a.chunk = plan.chunk;
  a.grain = plan.grain;
  a.share = plan.share;
  // Pages that keep a head's tokens together: neighbouring workgroups take the
  // heads of one page (168 us against 175); pages that keep a token's heads
  // together: neighbours take tokens (129 us against 145).
  a.heads_first = a.c.head_stride >= a.c.token_stride && (int64_t)a.s.batch * a.splits <= 65535;
  a.tiles = plan.tiles;
  a.join_rows = plan.rows;
  a.part_o = static_cast<float *>(ws);
  a.part_lse = plan.splits > 1
                   ? a.part_o + (size_t)plan.splits * a.s.rows * a.heads_q * a.c.dim
                   : nullptr;
  switch (a.c.dim) {
    case 64: return launch_dim<64>(a, e4m3, plan.nt, plan.wide, st);
    case 128: return launch_dim<128>(a, e4m3, plan.nt, plan.wide, st);
    default: return launch_dim<256>(a, e4m3, plan.nt, plan.wide, st);
  }
}

}  // namespace slq

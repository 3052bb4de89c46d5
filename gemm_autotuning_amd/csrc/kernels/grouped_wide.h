// grouped_wide.h -- the products of grouped.h where many rows name the same
// 16-bit matrix: tiles of 64 rows, so that the weights are read a quarter as
// often.
//
// A workgroup's eight waves take a pair of column tiles each and walk K
// together, 128 of it a step: the rows' piece lies in LDS for all of them,
// two buffers in turn, and each wave's weights come as in grouped.h.  A wave
// has its columns' whole sums (64 rows x 32 columns in registers), so nothing
// is joined.  8 experts 4096 x 2048 bf16, two to a token: 64 tokens 97 us (120
// with tiles of 16 rows), 256 tokens 160 (299), 512 tokens 274 to 291 (582): at 64
// tokens 402 MB of weights are 4.1 TB/s, at 512 the products' 77 GFLOP (the
// second one's rows are parts) and the waits of eight waves for each other
// bound it.  Halving K between the waves (256 workgroups instead of 128 for
// the first product) and loading the rows' pieces two steps ahead changed
// nothing or lost.
#pragma once

#include "grouped.h"

namespace gtk {

// PARTS: of an fp32 row's value (ValueParts).  bf16's three are all of it, for an
// fp32 y; two, 16 bits, are enough below a y that is rounded to 16 bits itself,
// and save a third of the second product's matrix-core work (256 tokens 159 us and
// 171 with three, 512 tokens 290 and 310).
template <int PHASE, int XT, int PARTS>
__global__ __launch_bounds__(512, 2) void grouped_wide_kernel(GroupedParams p) {
  typedef UnitOf<GROUPED_16, 256> Unit;
  typedef PairWeights<PHASE, GROUPED_16, 256, 128, 0> Weights;
  typedef W4Operand<XT, W4_E2M1> Op;  // elements in order
  constexpr int D = 4, R = D / 2;  // halves of units in flight; steps unrolled
  constexpr bool kSplit = PHASE == GROUPED_DOWN, kScaled = kSplit && XT == DT_F16;
  constexpr int kParts = kSplit ? PARTS : 1;
  constexpr int kPitch = 272;  // bytes of a row's 128 elements
  __shared__ TileSearch tile;
  __shared__ GroupedStage stages[8];
  __shared__ alignas(16) char xt[2][kParts][64 * kPitch];
  __shared__ float unscale[64];

  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool search = PHASE != GROUPED_DOWN && p.ix.n <= kFewRows;
  Part part = first_part(p, search, wave, tile);
  char* const st = stages[wave].q;
  for (bool found = search; part.left > 0; found = false) {
    const Stretch stretch = next_stretch(p, search, found, wave, part, tile);
    const int matrix = __builtin_amdgcn_readfirstlane(tile.matrix);
    if (matrix >= p.ix.matrices) continue;
    const int rows = __builtin_amdgcn_readfirstlane(tile.count);
    int lane = tid & 63;
    asm volatile("" : "+v"(lane));  // what follows from it is not kept over the search above
    const int r = lane & 15, kq = lane >> 4;
    Weights w(p, matrix, wave, stretch.g1, lane, st, nullptr);
    w.slice(stretch.slice);

    // ---- the rows' next 128 elements: eight threads to a row, 16 elements each
    const int xr = tid >> 3, xc = tid & 7, row = tile.rows[min(xr, rows - 1)];
    const char* const x = static_cast<const char*>(p.x) + (kSplit ? row * p.ldx * 4 : row_of(p.ix, row) * p.ldx * 2);
    constexpr int kRaw = kSplit ? 4 : 2;
    typedef u32x4 Raw[kRaw];
    auto load_x = [&](int un, Raw& raw) __attribute__((always_inline)) {
      const int k = (w.c0 + un) * 128 + 16 * xc;
#pragma unroll
      for (int i = 0; i < kRaw; ++i)
        raw[i] = *reinterpret_cast<const u32x4_any*>(x + (kSplit ? 4 * min(k + 4 * i, (p.K - 1) & ~3) : 2 * min(k + 8 * i, p.K - 8)));
    };
    float scale = 1.f;
    auto values = [&](int un, const Raw& raw, float (&v)[16]) __attribute__((always_inline)) {
      const int k = (w.c0 + un) * 128 + 16 * xc;
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = k + e < p.K ? __uint_as_float(raw[e / 4][e % 4]) : 0.f;
    };
    auto place_x = [&](int un, Raw& raw, int buf) __attribute__((always_inline)) {
      char* const at = xt[buf][0] + xr * kPitch + 32 * xc;
      if constexpr (!kSplit) {
        const int k = (w.c0 + un) * 128 + 16 * xc;
#pragma unroll
        for (int i = 0; i < kRaw; ++i) {
          if ((w.c0 + un + 1) * 128 > p.K) raw[i] = bytes_from(raw[i], min(max(0, 2 * (k + 8 * i - (p.K - 8))), 16));
          const Chunk c = Op::order(raw[i]);
          __builtin_memcpy(at + 16 * i, &c, 16);
        }
      } else {
        float v[16];
        values(un, raw, v);
#pragma unroll
        for (int part = 0; part < kParts; ++part)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint16_t h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float& f = v[8 * i + e];
              if (kScaled && part == 0) f *= scale;
              // of two, bf16's second is rounded
              h[e] = XT == DT_BF16 && kParts == 2 && part == 1 ? f32_to_bf16_bits(f) : take_part<XT>(f);
            }
            u32x4 b;
            __builtin_memcpy(&b, h, 16);
            const Chunk c = Op::order(b);
            __builtin_memcpy(at + part * (64 * kPitch) + 16 * i, &c, 16);
          }
      }
    };
    Raw raw;
    if constexpr (kScaled) {
      // a row's power of two, for its whole slice: its sums run over all of it
      uint32_t most = 0;
      for (int un = 0; un < w.nc; ++un) {
        float v[16];
        load_x(un, raw);
        values(un, raw, v);
#pragma unroll
        for (int e = 0; e < 16; ++e) most = max(most, __float_as_uint(v[e]) & 0x7fffffffu);
      }
      most = max(most, dpp<0xB1>(most));
      most = max(most, dpp<0x4E>(most));
      most = max(most, dpp<0x141>(most));
      const uint32_t to = row_power(most);
      scale = __uint_as_float(to << 23);
      if (xc == 0) unscale[xr] = __uint_as_float((254u - to) << 23);
    }

    // ---- weights: the next half to load is of unit load_u
    u32x4 ring[D][Unit::kLoads];
    typename Weights::Scale ring_s[D][Weights::kScales];
    int load_u = 0;
    auto load_half = [&](int place) __attribute__((always_inline)) {
      w.load(true, place & 1, load_u, ring[place], ring_s[place]);
      if (place & 1)
        if (++load_u == w.nc) {
          load_u = 0;
          w.load_next_pair();
        }
    };
    w.load_from(stretch.g0);
    load_x(0, raw);
#pragma unroll
    for (int d = 0; d < D; ++d) load_half(d);
    place_x(0, raw, 0);
    __syncthreads();

    f32x4 acc[2][4];
    auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[half][b] = f32x4{0.f, 0.f, 0.f, 0.f};
    };
    clear();
    int g = stretch.g0, u = 0, buf = 0;
    const int steps = (stretch.g1 - stretch.g0) * w.nc;
#pragma unroll 1
    for (int n = 0; n < steps; n += R)
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (n + i >= steps) break;
        const int next = u + 1 < w.nc ? u + 1 : 0;
        load_x(next, raw);
        // both halves' operands; of a pair that is not there nothing is stored
        Chunk f[2][4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          w.stage(max(w.last_of(g, half), 0), u, ring[2 * i + half], ring_s[2 * i + half]);
#pragma unroll
          for (int j = 0; j < 4; ++j) __builtin_memcpy(&f[half][j], st + r * Unit::kPitch + 16 * (4 * j + kq), 16);
          wave_lds_order();
          load_half(2 * i + half);
        }
        const char* const xb = xt[buf][0] + r * kPitch;
        auto x_at = [&](int b, int j, int part) {
          Chunk c;
          __builtin_memcpy(&c, xb + part * (64 * kPitch) + 16 * b * kPitch + 16 * (4 * j + kq), 16);
          return c;
        };
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (16 * b < rows)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int part = 0; part < kParts; ++part) {
                const Chunk c = x_at(b, j, part);
                Op::mma(acc[0][b], c, f[0][j]);
                Op::mma(acc[1][b], c, f[1][j]);
              }
        buf ^= 1;
        place_x(next, raw, buf);
        __syncthreads();
        if (++u == w.nc) {
#pragma unroll
          for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int m = 16 * b + 4 * kq + e;
              if (m < rows) {
                float* const out = p.out + tile.rows[m] * p.ld_out + stretch.slice * p.out_slice;
                if constexpr (PHASE == GROUPED_GATE_UP) {
                  if (r <= w.last_of(g, 0)) out[w.column_of(g, 0) + r] = activated(acc[0][b][e], acc[1][b][e], p.activation);
                } else {
                  const float s = kScaled ? unscale[m] : 1.f;
#pragma unroll
                  for (int half = 0; half < 2; ++half)
                    if (r <= w.last_of(g, half)) out[w.column_of(g, half) + r] = acc[half][b][e] * s;
                }
              }
            }
          clear();
          u = 0;
          ++g;
        }
      }
  }
}

template <int XT>
int grouped_wide_launch(const GroupedParams& p, int phase, bool whole, hipStream_t stream) {
  if (phase == GROUPED_GATE_UP)
    hipLaunchKernelGGL((grouped_wide_kernel<GROUPED_GATE_UP, XT, 1>), dim3(p.workgroups.n), dim3(512), 0, stream, p);
  else if (whole)
    hipLaunchKernelGGL((grouped_wide_kernel<GROUPED_DOWN, XT, ValueParts<XT>::n>), dim3(p.workgroups.n), dim3(512), 0, stream, p);
  else
    hipLaunchKernelGGL((grouped_wide_kernel<GROUPED_DOWN, XT, 2>), dim3(p.workgroups.n), dim3(512), 0, stream, p);
  return hipGetLastError() == hipSuccess ? gt::LS_OK : gt::LS_HIP_ERROR;
}

}  // namespace gtk

namespace gt {
// whole: all of an fp32 row's values, not 16 bits of them
int grouped_wide_bf16(const gtk::GroupedParams& p, int phase, bool whole, hipStream_t stream);
int grouped_wide_f16(const gtk::GroupedParams& p, int phase, bool whole, hipStream_t stream);
}  // namespace gt

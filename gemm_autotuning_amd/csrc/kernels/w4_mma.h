// w4_mma.h -- rows times 4-bit weights on the matrix cores.
//
//   y[m,n] = f[m] * sum_g s[n,g] * (sum_{k in g} x[m,k] * v(q[n,k]))
//
// The weights are read once from HBM and bound the time (half a byte each);
// everything else is arranged around that stream.  A wave owns a slice of K
// (at most C chunks of 128) and keeps the rows' slice in registers, as the A
// operands of 16x16x32 matrix-core blocks (T blocks of 16 rows); it then
// walks tiles of 16 columns, loading 16 bytes per lane and chunk (a column's
// 32 consecutive k), one tile ahead of the arithmetic.  The workgroup's waves
// hold consecutive slices, so a tile ends with a sum over the waves in LDS;
// when K is longer than a workgroup's slices, S workgroups share a tile and
// the last to finish adds their partial sums in order (slices.h).
//
// The values are expanded exactly: integers through e4m3 (below), e2m1
// through the conversion instructions.  A group's products are summed in the
// matrix core's fp32 accumulators and the group's scale multiplies that sum.
#pragma once

#include "elements.h"
#include "slices.h"

namespace gtk {

constexpr int kW4Waves = 8;     // most waves of a workgroup
constexpr int kW4Chunk = 128;   // k of one 16-byte load of the four lanes of a column
enum { W4_INT4 = 0, W4_E2M1 = 1 };

struct W4Params {
  gt::W4Args a;
  float* ws;           // S x M x N partial sums (S > 1)
  unsigned* counters;  // one per workgroup of columns and rows, zero between launches (S > 1)
  int S, waves;
  int tiles, tiles_per_wg, chunks;
};

// The low nibble of each byte, two's complement, as four e4m3 bytes of value
// nibble / 512: e4m3 is linear below 2^-5 (magnitudes 0..15 in steps of 2^-9
// are the bytes 0..15), so the magnitude itself is the code.  A negative c in
// -8..-1 has the bits 8 + j and the magnitude 8 - j = (j ^ 7) + 1.
__device__ __forceinline__ uint32_t int4_to_e4m3(uint32_t u) {
  const uint32_t t = u & 0x08080808u, one = t >> 3;
  return (((u & 0x07070707u) ^ (t - one)) + one) | (t << 4);
}
// The operands of one 16x16x32 matrix-core block: eight k of a lane.  Rows of
// f16 stay f16; bf16 rows and e4m3 rows (exact in bf16) run as bf16.  The
// 8-bit matrix-core instructions would take e4m3 rows as they are, but their
// sums are held in fewer bits than fp32: on rows with a few large elements
// they were off by 2^-16 of the terms' magnitudes.
template <int XT>
struct W4Rows {
  static constexpr bool kF16 = XT == DT_F16;
  static __device__ __forceinline__ void mma(f32x4& acc, const Chunk& x, const Chunk& w) {
    if constexpr (kF16)
      Mfma16<TraitsF16>::mma(acc, x, w);
    else
      Mfma16<TraitsBF16>::mma(acc, x, w);
  }
  template <class V>
  static __device__ __forceinline__ uint32_t bits(V v) {
    uint32_t r;
    __builtin_memcpy(&r, &v, 4);
    return r;
  }
  // two e4m3 bytes times 2^e (scale = 2^e), the low or the high half of b
  template <bool HIGH>
  static __device__ __forceinline__ uint32_t from_e4m3(uint32_t b, float scale) {
    if constexpr (kF16)
      return bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, scale, HIGH));
    else
      return bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, HIGH));
  }
  // eight elements of a row, `valid` of them inside it
  static __device__ __forceinline__ Chunk load(const void* p, int64_t i, int valid) {
    Chunk f = {{0, 0, 0, 0}};
    if constexpr (XT == DT_E4M3) {
      const uint8_t* s = reinterpret_cast<const uint8_t*>(p) + i;
      uint32_t b[2] = {0, 0};
      if (valid >= 8) {
        __builtin_memcpy(b, s, 8);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < valid) b[e >> 2] |= (uint32_t)s[e] << (8 * (e & 3));
      }
      f.w[0] = from_e4m3<false>(b[0], 1.f);
      f.w[1] = from_e4m3<true>(b[0], 1.f);
      f.w[2] = from_e4m3<false>(b[1], 1.f);
      f.w[3] = from_e4m3<true>(b[1], 1.f);
    } else {
      const uint16_t* s = reinterpret_cast<const uint16_t*>(p) + i;
      if (valid >= 8) {
        __builtin_memcpy(&f, s, 16);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < valid) f.w[e >> 1] |= (uint32_t)s[e] << (16 * (e & 1));
      }
    }
    return f;
  }
};

// Eight weights from a dword of nibbles, and the rows' elements in the order
// of k they come in.
template <int XT, int FMT>
struct W4Operand : W4Rows<XT> {
  typedef W4Rows<XT> R;
  static __device__ __forceinline__ Chunk weights(uint32_t u) {
    Chunk f;
    if constexpr (FMT == W4_INT4) {
      const uint32_t lo = int4_to_e4m3(u), hi = int4_to_e4m3(u >> 4);
      f.w[0] = R::template from_e4m3<false>(lo, 512.f);
      f.w[1] = R::template from_e4m3<true>(lo, 512.f);
      f.w[2] = R::template from_e4m3<false>(hi, 512.f);
      f.w[3] = R::template from_e4m3<true>(hi, 512.f);
    } else if constexpr (R::kF16) {
      f.w[0] = R::bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(u, 1.f, 0));
      f.w[1] = R::bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(u, 1.f, 1));
      f.w[2] = R::bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(u, 1.f, 2));
      f.w[3] = R::bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(u, 1.f, 3));
    } else {
      f.w[0] = R::bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(u, 1.f, 0));
      f.w[1] = R::bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(u, 1.f, 1));
      f.w[2] = R::bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(u, 1.f, 2));
      f.w[3] = R::bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(u, 1.f, 3));
    }
    return f;
  }
  // integers: the low nibbles (even k), then the high ones; e2m1: as stored
  static __device__ __forceinline__ Chunk order(const Chunk& x) {
    if constexpr (FMT == W4_E2M1) return x;
    Chunk f;
    f.w[0] = __builtin_amdgcn_perm(x.w[1], x.w[0], 0x05040100u);
    f.w[1] = __builtin_amdgcn_perm(x.w[3], x.w[2], 0x05040100u);
    f.w[2] = __builtin_amdgcn_perm(x.w[1], x.w[0], 0x07060302u);
    f.w[3] = __builtin_amdgcn_perm(x.w[3], x.w[2], 0x07060302u);
    return f;
  }
};

// Dwords of a 4 x 4 grid (16-lane row of the wave, index) transposed: lane
// row r's d[j] becomes lane row j's d[r].
__device__ __forceinline__ void transpose_lane_rows(uint32_t (&d)[4]) {
  auto swap32 = [](uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
  };
  auto swap16 = [](uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
  };
  swap32(d[0], d[2]);
  swap32(d[1], d[3]);
  swap16(d[0], d[1]);
  swap16(d[2], d[3]);
}

// What a wave loads of one tile: C chunks of its columns and their scales.
template <int G, int C>
struct W4Tile {
  Chunk q[C];
  uint32_t s[C][kW4Chunk / G];
};

// Bytes [0, valid) of 16 at p (the rest zero: the rows are zero there).
__device__ __forceinline__ Chunk load_nibbles(const uint8_t* p, int valid) {
  Chunk c = {{0, 0, 0, 0}};
  if (valid >= 16) {
    __builtin_memcpy(&c, p, 16);
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (e < valid) c.w[e >> 2] |= (uint32_t)p[e] << (8 * (e & 3));
  }
  return c;
}

template <int XT, int FMT, int G, int WIDE, int T, int C>
__global__ __launch_bounds__(64 * kW4Waves) void w4_mma_kernel(W4Params p) {
  typedef W4Operand<XT, FMT> Op;
  constexpr int kPer = kW4Chunk / G;  // groups of a chunk
  __shared__ float red[2][kW4Waves][T][256];
  __shared__ int is_last;
  const gt::W4Args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, kq = lane >> 4;
  const int slice = blockIdx.y * p.waves + wave;
  // the slices' chunks differ by at most one
  const int c0 = (int)((int64_t)slice * p.chunks / (p.S * p.waves));
  const int nc = (int)((int64_t)(slice + 1) * p.chunks / (p.S * p.waves)) - c0;
  const int64_t m0 = (int64_t)blockIdx.z * (16 * T);
  const int64_t K = a.w.K, N = a.w.N;
  // the k of step j of a chunk: with one group to a chunk a lane's 32
  // consecutive k give four steps of eight; with more, a step's 32 k must
  // be of one group, so the dwords are exchanged between the lane rows
  auto k_of = [&](int c, int j) { return (int64_t)(c0 + c) * kW4Chunk + (G == kW4Chunk ? 32 * kq + 8 * j : 32 * j + 8 * kq); };

  Chunk x[C][4][T];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const int64_t m = m0 + 16 * t + r, k = k_of(c, j);
        const int64_t left = m < a.M && c < nc ? K - k : 0;
        x[c][j][t] = Op::order(Op::load(a.x, m * a.ldx + k, (int)(left < 8 ? (left < 0 ? 0 : left) : 8)));
      }

  const int64_t row_bytes = (K + 1) / 2;
  const int groups = (int)((K + G - 1) / G);
  auto load_tile = [&](int tile, W4Tile<G, C>& w) {
    int64_t n = (int64_t)tile * 16 + r;
    if (n >= N) n = N - 1;  // a column past the last is computed and not stored
    const uint8_t* q = a.w.q + n * a.w.ldq;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c < nc) {
        const int64_t b = (int64_t)(c0 + c) * (kW4Chunk / 2) + 16 * kq;
        if ((int64_t)(c0 + c + 1) * kW4Chunk <= K) {
          __builtin_memcpy(&w.q[c], q + b, 16);
        } else {
          const int64_t left = row_bytes - b;
          w.q[c] = load_nibbles(q + b, (int)(left < 16 ? (left < 0 ? 0 : left) : 16));
        }
#pragma unroll
        for (int g = 0; g < kPer; ++g) {
          const int gi = (c0 + c) * kPer + g;
          const int64_t i = n * a.w.lds_n + (gi < groups ? gi : groups - 1) * a.w.lds_g;
          if constexpr (WIDE)
            w.s[c][g] = reinterpret_cast<const uint32_t*>(a.w.scales)[i];
          else
            w.s[c][g] = reinterpret_cast<const uint16_t*>(a.w.scales)[i];
          if (gi >= groups) w.s[c][g] = 0;  // past K: nothing times zero, whatever the last group's scale is
        }
      }
  };

  const int tile0 = blockIdx.x * p.tiles_per_wg;
  const int tile1 = min(tile0 + p.tiles_per_wg, p.tiles);
  const bool bf16_scales = a.w.scale_dtype == DT_BF16;
  W4Tile<G, C> cur, next;
  load_tile(tile0, cur);
  for (int tile = tile0; tile < tile1; ++tile) {
    if (tile + 1 < tile1) load_tile(tile + 1, next);
    f32x4 acc[T];
#pragma unroll
    for (int t = 0; t < T; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c < nc) {
        uint32_t d[4] = {cur.q[c].w[0], cur.q[c].w[1], cur.q[c].w[2], cur.q[c].w[3]};
        if constexpr (G < kW4Chunk) transpose_lane_rows(d);
#pragma unroll
        for (int g = 0; g < kPer; ++g) {
          f32x4 sum[T];
#pragma unroll
          for (int t = 0; t < T; ++t) sum[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 4 / kPer; ++j) {
            const Chunk w = Op::weights(d[g * (4 / kPer) + j]);
#pragma unroll
            for (int t = 0; t < T; ++t) Op::mma(sum[t], x[c][g * (4 / kPer) + j][t], w);
          }
          const uint32_t sb = cur.s[c][g];
          const float s = WIDE ? __uint_as_float(sb) : (bf16_scales ? bf16_bits_to_f32((uint16_t)sb) : f16_bits_to_f32((uint16_t)sb));
#pragma unroll
          for (int t = 0; t < T; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][i] += s * sum[t][i];
        }
      }
    // the waves' sums of this tile; the two buffers take turns, so one
    // barrier a tile keeps a buffer's readers ahead of its next writers
    const int buf = (tile - tile0) & 1;
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[buf][wave][t][64 * i + lane] = acc[t][i];
    __syncthreads();
    for (int o = tid; o < 256 * T; o += 64 * p.waves) {
      const int t = o >> 8, e = o & 255;
      float v = 0.f;
      for (int w = 0; w < p.waves; ++w) v += red[buf][w][t][e];
      const int64_t m = m0 + 16 * t + 4 * ((e >> 4) & 3) + (e >> 6), n = (int64_t)tile * 16 + (e & 15);
      if (m < a.M && n < N) {
        if (p.S == 1)
          store_out(a.y, m * a.ldy + n, v * a.x_scale * (a.row_scale ? a.row_scale[m] : 1.f), a.out_dtype);
        else
          __hip_atomic_store(&p.ws[((int64_t)blockIdx.y * a.M + m) * N + n], v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    cur = next;
  }
  if (p.S == 1) return;
  unsigned* counter = p.counters + blockIdx.z * gridDim.x + blockIdx.x;
  last_slice_handshake(counter, p.S, tid, is_last);
  if (!is_last) return;
  const int cols = (int)(min((int64_t)tile1 * 16, N) - (int64_t)tile0 * 16);
  const int rows = (int)min((int64_t)(16 * T), a.M - m0);
  for (int o = tid; o < rows * cols; o += 64 * p.waves) {
    const int64_t m = m0 + o / cols, n = (int64_t)tile0 * 16 + o % cols;
    const float v = sum_slices<8>(p.ws + m * N + n, a.M * N, p.S);
    store_out(a.y, m * a.ldy + n, v * a.x_scale * (a.row_scale ? a.row_scale[m] : 1.f), a.out_dtype);
  }
  if (tid == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Launch for rows of type XT; T and C as chosen by the caller.
template <int XT, int FMT, int G, int WIDE>
int w4_mma_sizes(const W4Params& p, dim3 grid, int T, int C) {
  const dim3 block(64 * p.waves);
  if (T == 1 && C == 1)
    hipLaunchKernelGGL((w4_mma_kernel<XT, FMT, G, WIDE, 1, 1>), grid, block, 0, p.a.stream, p);
  else if (T == 1 && C == 4)
    hipLaunchKernelGGL((w4_mma_kernel<XT, FMT, G, WIDE, 1, 4>), grid, block, 0, p.a.stream, p);
  else if (T == 2 && C == 2)
    hipLaunchKernelGGL((w4_mma_kernel<XT, FMT, G, WIDE, 2, 2>), grid, block, 0, p.a.stream, p);
  else if (T == 4 && C == 2)
    hipLaunchKernelGGL((w4_mma_kernel<XT, FMT, G, WIDE, 4, 2>), grid, block, 0, p.a.stream, p);
  else
    return gt::LS_UNSUPPORTED;
  return hipGetLastError() == hipSuccess ? gt::LS_OK : gt::LS_HIP_ERROR;
}
template <int XT, int FMT, int G>
int w4_mma_scales(const W4Params& p, dim3 grid, int T, int C) {
  return p.a.w.scale_dtype == DT_F32 ? w4_mma_sizes<XT, FMT, G, 1>(p, grid, T, C) : w4_mma_sizes<XT, FMT, G, 0>(p, grid, T, C);
}
template <int XT, int FMT>
int w4_mma_group(const W4Params& p, dim3 grid, int T, int C) {
  switch (p.a.w.group) {
    case 32: return w4_mma_scales<XT, FMT, 32>(p, grid, T, C);
    case 64: return w4_mma_scales<XT, FMT, 64>(p, grid, T, C);
    default: return w4_mma_scales<XT, FMT, 128>(p, grid, T, C);
  }
}
// One source file per row type and format defines its launcher.
#define GT_W4_LAUNCHER(name, XT, FMT) \
  int name(const gtk::W4Params& p, dim3 grid, int T, int C) { return gtk::w4_mma_group<XT, FMT>(p, grid, T, C); }

}  // namespace gtk

namespace gt {
int w4_mma_bf16_int4(const gtk::W4Params& p, dim3 grid, int T, int C);
int w4_mma_bf16_e2m1(const gtk::W4Params& p, dim3 grid, int T, int C);
int w4_mma_f16_int4(const gtk::W4Params& p, dim3 grid, int T, int C);
int w4_mma_f16_e2m1(const gtk::W4Params& p, dim3 grid, int T, int C);
int w4_mma_e4m3_int4(const gtk::W4Params& p, dim3 grid, int T, int C);
int w4_mma_e4m3_e2m1(const gtk::W4Params& p, dim3 grid, int T, int C);
}  // namespace gt

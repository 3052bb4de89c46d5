// w4_mma.h -- rows times 4-bit weights on the matrix cores.
//
//   y[m,n] = f[m] * sum_g s[n,g] * (sum_{k in g} x[m,k] * v(q[n,k]))
//
// The weights are read once from HBM and bound the time (half a byte each);
// everything else is arranged around that stream.  A wave owns a slice of K
// (at most C chunks of 128) and keeps the rows' slice in registers, as the A
// operands of 16x16x32 matrix-core blocks (T blocks of 16 rows); it then
// walks tiles of 16 columns, loading 16 bytes per lane and chunk (32
// consecutive k of a column) D tiles ahead of the arithmetic.  The
// workgroup's waves hold consecutive slices, so tiles end with a sum over the
// waves in LDS, several tiles to a barrier; when K is longer than a
// workgroup's slices, S workgroups share a tile and a second launch adds
// their partial sums in order.
//
// 4 x 65536 x 8192 bf16 (group 128) takes 56 us, 5.0 TB/s, a copy's rate:
// HBM.  One row of 16384 x 4096 takes 10.8 us, of which 2.4 are a launch and
// 2.8 the time until the rows are laid out.  61 x 11001 x 4100 takes 24.3 us:
// with four row blocks a tile's expansion, products, the waves' sums and the
// barrier follow each other (1.3 us a tile, about four times what its bytes
// take), and two waves a SIMD hide little of it: vector instructions are under
// way in 0.22 of the waves' cycles, LDS in 0.06, the matrix cores are busy for
// 0.09 of the dispatch.
//
// The values are expanded exactly, and a group's products are summed in the
// matrix core's fp32 accumulators before the group's scale multiplies them.
#pragma once

#include <type_traits>

#include "elements.h"

namespace gtk {

constexpr int kW4Waves = 8;     // most waves of a workgroup
constexpr int kW4Chunk = 128;   // k of one 16-byte load of the four lanes of a column
constexpr int kW4LeastK = 32;   // 16 bytes of a row: what a lane loads
enum { W4_INT4 = 0, W4_E2M1 = 1 };
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef u32x4 u32x4_any __attribute__((aligned(1)));  // at any byte

struct W4Params {
  gt::W4Args a;
  float* ws;           // S x M x ws_ld partial sums (S > 1)
  int64_t ws_ld;       // N rounded up to whole tiles
  int S, waves, groups, tiles;  // waves side by side along K, groups of them side by side along N
  int waves_inverse;            // 2^16 / waves, rounded up: exact for what is divided (at most 64)
  int chunks_each, chunks_rest;  // of a workgroup's slice: the first `rest` of S have one more
  int tiles_each, tiles_rest;    // of a group's columns
};

// Eight two's complement nibbles as e4m3 bytes of value nibble / 512, those of
// the bytes' low nibbles and those of the high ones: e4m3 is linear below 2^-5
// (magnitudes 0..15 in steps of 2^-9 are the bytes 0..15), so the magnitude
// itself is the code.  A negative c in -8..-1 has the bits 8 + j and the
// magnitude 8 - j = (j ^ 7) + 1.
__device__ __forceinline__ void int4_to_e4m3(uint32_t u, uint32_t* lo, uint32_t* hi) {
  uint32_t sign = u & 0x88888888u;
  const uint32_t one = sign >> 3;
  asm("" : "+v"(sign));  // else its known bits make two instructions of each selection below
  const uint32_t mag = ((u & 0x77777777u) ^ (sign - one)) + one;
  *lo = (mag & 0x0f0f0f0fu) | (sign << 4 & 0xf0f0f0f0u);
  *hi = (mag >> 4 & 0x0f0f0f0fu) | (sign & 0xf0f0f0f0u);
}
template <class V>
__device__ __forceinline__ uint32_t bits_of(V v) {
  uint32_t r;
  __builtin_memcpy(&r, &v, 4);
  return r;
}

// A row's operand of one 16x16x32 block: eight k of a lane.  f16 rows stay
// f16 and bf16 rows bf16; e4m3 rows run as f16, which holds them exactly.
// The 8-bit matrix-core instructions would take e4m3 rows as they are, but
// their sums are held in fewer bits than fp32: on rows with a few large
// elements they were off by 2^-16 of the terms' magnitudes.
template <int XT>
struct W4Rows {
  static constexpr bool kF16 = XT != DT_BF16;
  static constexpr int kBytes = XT == DT_E4M3 ? 1 : 2;
  typedef __attribute__((ext_vector_type(2 * kBytes))) uint32_t Raw;  // eight elements
  typedef Raw RawAny __attribute__((aligned(1)));
  static __device__ __forceinline__ void mma(f32x4& acc, const Chunk& x, const Chunk& w) {
    if constexpr (kF16)
      Mfma16<TraitsF16>::mma(acc, x, w);
    else
      Mfma16<TraitsBF16>::mma(acc, x, w);
  }
  static __device__ __forceinline__ Raw load(const void* p, int64_t i) {
    return *reinterpret_cast<const RawAny*>(static_cast<const char*>(p) + i * kBytes);
  }
  // the elements d.. of r in front (0 <= d), zeros after them, then the
  // first lo zeroed: both count to 8 and past it
  static __device__ __forceinline__ Raw window(Raw r, int d, int lo) {
    unsigned __int128 v = 0;
    __builtin_memcpy(&v, &r, sizeof(r));
    constexpr int kBits = 8 * kBytes;
    v = d < 8 ? v >> (kBits * d) : 0;
    if (lo > 0) v = lo < 8 ? v >> (kBits * lo) << (kBits * lo) : 0;
    Raw o;
    __builtin_memcpy(&o, &v, sizeof(o));
    return o;
  }
  static __device__ __forceinline__ u32x4 widen(Raw r) {
    if constexpr (XT == DT_E4M3)
      return u32x4{bits_of(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(r[0], 1.f, false)),
                   bits_of(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(r[0], 1.f, true)),
                   bits_of(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(r[1], 1.f, false)),
                   bits_of(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(r[1], 1.f, true))};
    else
      return r;
  }
};

// Eight weights from a dword of nibbles, and the rows' elements in the order
// of k they come in.  Instructions per dword, which the arithmetic of one row
// block hardly hides: e2m1 four (conversions); integers nine with f16 rows,
// thirteen with bf16 ones (value + 8 would take seven there, but its sums hold
// eight times the row's elements, and a large one at a weight of zero costs
// the others their last bits).
template <int XT, int FMT>
struct W4Operand : W4Rows<XT> {
  typedef W4Rows<XT> R;
  static __device__ __forceinline__ Chunk weights(uint32_t u) {
    Chunk f;
    if constexpr (FMT == W4_E2M1) {
      if constexpr (R::kF16) {
        f.w[0] = bits_of(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(u, 1.f, 0));
        f.w[1] = bits_of(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(u, 1.f, 1));
        f.w[2] = bits_of(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(u, 1.f, 2));
        f.w[3] = bits_of(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(u, 1.f, 3));
      } else {
        f.w[0] = bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(u, 1.f, 0));
        f.w[1] = bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(u, 1.f, 1));
        f.w[2] = bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(u, 1.f, 2));
        f.w[3] = bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(u, 1.f, 3));
      }
    } else if constexpr (R::kF16) {
      // a nibble with its sign bit flipped is value + 8; under the exponent of
      // 1024 it adds that (or 16 times that) to 1024, and one fused step
      // takes the rest off, exactly
      const uint32_t h = u >> 8;
      f.w[0] = low(u & 0x000f000fu);
      f.w[1] = high(u & 0x00f000f0u);
      f.w[2] = low(h & 0x000f000fu);
      f.w[3] = high(h & 0x00f000f0u);
    } else {
      uint32_t lo, hi;
      int4_to_e4m3(u, &lo, &hi);
      f.w[0] = bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.f, false));
      f.w[1] = bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.f, true));
      f.w[2] = bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.f, false));
      f.w[3] = bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.f, true));
    }
    return f;
  }
  static __device__ __forceinline__ uint32_t low(uint32_t b) {
    b ^= 0x64086408u;
    f16x2v f;
    __builtin_memcpy(&f, &b, 4);
    return bits_of(f + f16x2v{(_Float16)-1032.f, (_Float16)-1032.f});
  }
  static __device__ __forceinline__ uint32_t high(uint32_t b) {
    b ^= 0x64806480u;
    f16x2v f;
    __builtin_memcpy(&f, &b, 4);
    return bits_of(__builtin_elementwise_fma(f, f16x2v{(_Float16)0.0625f, (_Float16)0.0625f},
                                             f16x2v{(_Float16)-72.f, (_Float16)-72.f}));
  }
  // e2m1: as stored.  Integers: f16 pairs k with k + 4; bf16 takes the even
  // k (the bytes' low nibbles), then the odd ones.
  static __device__ __forceinline__ Chunk order(u32x4 x) {
    Chunk f = {{x[0], x[1], x[2], x[3]}};
    if constexpr (FMT == W4_E2M1) return f;
    if constexpr (R::kF16) {
      f.w[0] = __builtin_amdgcn_perm(x[2], x[0], 0x05040100u);
      f.w[1] = __builtin_amdgcn_perm(x[2], x[0], 0x07060302u);
      f.w[2] = __builtin_amdgcn_perm(x[3], x[1], 0x05040100u);
      f.w[3] = __builtin_amdgcn_perm(x[3], x[1], 0x07060302u);
    } else {
      f.w[0] = __builtin_amdgcn_perm(x[1], x[0], 0x05040100u);
      f.w[1] = __builtin_amdgcn_perm(x[3], x[2], 0x05040100u);
      f.w[2] = __builtin_amdgcn_perm(x[1], x[0], 0x07060302u);
      f.w[3] = __builtin_amdgcn_perm(x[3], x[2], 0x07060302u);
    }
    return f;
  }
};

// How a wave takes a tile from memory.  The operand layout has a column to a
// lane and neighbouring lanes in different columns, where the L1 would serve
// each lane's 16 bytes by themselves; so a load has kLanes neighbouring lanes
// on one column's consecutive bytes, and the pieces go through an LDS region
// of the wave's own, whose columns lie a piece further apart than their
// length (the reads of 16 columns fall on different banks).  A chunk's scales
// take the same way, already as floats.
template <int G, int C, int WIDE>
struct W4Stage {
  typedef typename std::conditional<WIDE, uint32_t, uint16_t>::type Scale;
  static constexpr int kPer = kW4Chunk / G;  // groups of a chunk
  static constexpr int kLanes = C < 4 ? 4 * C : 16, kCols = 64 / kLanes, kRuns = 4 * C / kLanes;
  static constexpr int kScales = C * kPer < 4 ? 1 : C * kPer / 4;  // of a lane: every fourth
  alignas(16) uint32_t q[16][(4 * C + 1) * 4];
  alignas(16) float s[16][4 * kScales + 4];
};

// Between LDS accesses of a wave's lanes to each other's places: the hardware
// serves a wave's accesses in order, and the compiler must keep it.
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ONCE: the weights pass by the caches.  It pays where each row of them starts
// a cache line and a wave reads whole ones, so that no line is read by two
// loads far apart (4 x 65536 x 8192 f16: 55.4 us, 62.0 through the caches; 16 x
// 32768 x 2048 12.4 and 13.5; rows of 2050 bytes lose, 27.1 and 24.3), and
// with one row block (64 x 32768 x 4096 39.1 and 37.2).
template <int XT, int FMT, int G, int WIDE, int T, int C, int D, int ONCE>
__global__ __launch_bounds__(64 * kW4Waves) void w4_mma_kernel(W4Params p) {
  typedef W4Operand<XT, FMT> Op;
  typedef W4Stage<G, C, WIDE> Stage;
  constexpr int kPer = Stage::kPer;
  constexpr int kBatch = T == 4 ? 2 : 4;  // tiles to a barrier
  constexpr int kRound = kBatch > D ? kBatch : D;  // tiles that are unrolled
  static_assert(kRound % kBatch == 0 && kRound % D == 0, "a round is a whole number of both");
  __shared__ float red[kW4Waves][2][kBatch][T][256];
  __shared__ Stage stages[kW4Waves];
  const gt::W4Args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, kq = lane >> 4;
  // With fewer chunks than waves, groups of waves have columns of their own.
  // The slices' chunks differ by at most one, and so do their waves' and the
  // groups' tiles; a wave has at least C / 2 chunks and at most C.
  const int group = (wave * p.waves_inverse) >> 16, turn = wave - group * p.waves, part = blockIdx.y;
  const int cols = blockIdx.x * p.groups + group;
  const int chunks = p.chunks_each + (part < p.chunks_rest);
  const int each = (chunks * p.waves_inverse) >> 16, rest = chunks - each * p.waves;
  const int nc = each + (turn < rest);
  const int c0 = part * p.chunks_each + min(part, p.chunks_rest) + turn * each + min(turn, rest);
  const int tile0 = cols * p.tiles_each + min(cols, p.tiles_rest), tile1 = tile0 + p.tiles_each + (cols < p.tiles_rest);
  const int most_tiles = p.groups == 1 ? tile1 - tile0 : p.tiles_each + (p.tiles_rest > 0);  // of the workgroup's groups
  const int64_t K = a.w.K, N = a.w.N;
  const int64_t row0 = (int64_t)blockIdx.z * (16 * T);
  const int rows = (int)min(a.M - row0, (int64_t)(16 * T));

  // The rows.  A chunk's k come in pieces of eight, and weight bytes in 16: a
  // column's last 16 bytes end with the row, so in the last chunk they reach
  // back over bytes that belong to others, and the rows' elements at those
  // places are zero.  Sixteen neighbouring lanes load a row's chunk; a row
  // past the last is computed and not stored.
  //
  // No load is under a condition (what there is nothing for reads a place
  // that is read anyway): the wait for one then leaves the later ones in
  // flight, where a load that may not have happened would mean a wait for all.
  //
  // The wave's first chunk here is its slice's last (then the others in
  // order), so that the special case is in one place of the code.
  const int64_t row_bytes = (K + 1) / 2;
  auto chunk = [&](int c) { return c0 + (c ? c - 1 : nc - 1); };
  auto k_of = [&](int c, int piece) {
    const int64_t b = (int64_t)chunk(c) * (kW4Chunk / 2) + 16 * (piece >> 2);
    return 2 * (b < row_bytes - 16 ? b : row_bytes - 16) + 8 * (piece & 3);
  };
  typename Op::Raw raw[C][T][4];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t k = k_of(c, r);
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        raw[c][t][i] = Op::load(a.x, (row0 + min(16 * t + 4 * i + kq, rows - 1)) * a.ldx + (k < K - 8 ? k : K - 8));
  }

  Stage& stage = stages[wave];
  constexpr int kScale = sizeof(typename Stage::Scale);
  const int groups = (int)((K + G - 1) / G), g0 = c0 * kPer;
  const int64_t b0 = min((int64_t)c0 * (kW4Chunk / 2), row_bytes - 16);
  const uint32_t ldq = (uint32_t)a.w.ldq, lds_n = (uint32_t)a.w.lds_n * kScale, lds_g = (uint32_t)a.w.lds_g * kScale;
  uint32_t q_off[Stage::kRuns];  // the lane's bytes of its first column
#pragma unroll
  for (int i = 0; i < Stage::kRuns; ++i) {
    const int piece = i * Stage::kLanes + lane % Stage::kLanes;
    q_off[i] = (uint32_t)(min((int64_t)chunk(piece >> 2) * (kW4Chunk / 2) + 16 * (piece & 3), row_bytes - 16) - b0) +
               lane / Stage::kLanes * ldq;
  }
  auto scale_of = [&](int i) {  // of the slice's groups of k: that of the lane's i-th scale
    const int g = 4 * i + (lane & 3);
    return g < kPer ? (nc - 1) * kPer + g : g - kPer;
  };
  const uint32_t s_most = (uint32_t)min(groups - 1 - g0, 4 * Stage::kScales) * lds_g;
  const int64_t n0 = (int64_t)min(tile0, p.tiles - 1) * 16;  // a group may have no tile
  const uint8_t* const q0 = a.w.q + n0 * a.w.ldq + b0;
  const char* const s0 = static_cast<const char*>(a.w.scales) + (n0 * a.w.lds_n + g0 * a.w.lds_g) * kScale;
  const uint8_t* q_next = q0;
  const char* s_next = s0;
  // the group's next tile; past its last, the first bytes of its first
  auto load_tile = [&](int tile, u32x4 (&wq)[C], typename Stage::Scale (&ws)[Stage::kScales]) __attribute__((always_inline)) {
    const uint32_t some = tile < tile1 ? ~0u : 0u;
    const uint32_t last = tile == p.tiles - 1 ? (uint32_t)(N - 1) & 15u : 15u;  // a column past it is computed and not stored
    const uint8_t* q = some ? q_next : q0;
    const char* s = some ? s_next : s0;
    q_next += 16 * a.w.ldq;
    s_next += 16 * a.w.lds_n * kScale;
    uint32_t most[Stage::kRuns];
#pragma unroll
    for (int i = 0; i < Stage::kRuns; ++i)
      most[i] = ((last - lane / Stage::kLanes) * ldq + q_off[i]) &
                (i * Stage::kLanes + lane % Stage::kLanes < 4 * nc ? some : 0u);
    const uint32_t step = ldq * Stage::kCols;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int run = i % Stage::kRuns;
      const u32x4_any* at = reinterpret_cast<const u32x4_any*>(q + min(i / Stage::kRuns * step + q_off[run], most[run]));
      if constexpr (ONCE)
        wq[i] = __builtin_nontemporal_load(at);
      else
        wq[i] = *at;
    }
    const uint32_t col = min((uint32_t)lane >> 2, last) * lds_n;
#pragma unroll
    for (int i = 0; i < Stage::kScales; ++i) {
      const uint32_t off = (col + min(scale_of(i) * lds_g, s_most)) & some;
      ws[i] = *reinterpret_cast<const typename Stage::Scale*>(s + off);
    }
  };
  const uint32_t bf16_scales = a.w.scale_dtype == DT_BF16 ? ~0u : 0u;
  auto stage_tile = [&](const u32x4 (&wq)[C], const typename Stage::Scale (&ws)[Stage::kScales]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < C; ++i)
      *reinterpret_cast<u32x4*>(&stage.q[i / Stage::kRuns * Stage::kCols + lane / Stage::kLanes]
                                        [4 * (i % Stage::kRuns * Stage::kLanes + lane % Stage::kLanes)]) = wq[i];
#pragma unroll
    for (int i = 0; i < Stage::kScales; ++i) {
      typename Stage::Scale b = ws[i];
      asm volatile("" : "+v"(b));  // converted here and not where it was loaded, which would wait for it there
      float f;
      if constexpr (WIDE)
        f = __uint_as_float(b);
      else  // both conversions and a selection by bits: a branch here would split the tile's code
        f = __uint_as_float(((uint32_t)b << 16 & bf16_scales) | (__float_as_uint(f16_bits_to_f32(b)) & ~bf16_scales));
      // past K: nothing times zero, whatever the last group's scale is
      stage.s[lane >> 2][4 * i + (lane & 3)] = g0 + scale_of(i) < groups ? f : 0.f;
    }
    wave_lds_order();
  };
  u32x4 ring_q[D][C];
  typename Stage::Scale ring_s[D][Stage::kScales];
#pragma unroll
  for (int d = 0; d < D; ++d) load_tile(tile0 + d, ring_q[d], ring_s[d]);

  // Into operand layout through LDS (the wave's part of the sums, still
  // unused): a
  // lane has row r, and of a chunk with one group its own 32 k, eight to a
  // step; with more groups a step's 32 k must be of one group.
  Chunk x[C][4][T];
  {
    static_assert(sizeof(red[0]) >= 16 * 16 * sizeof(u32x4), "a chunk of 16 rows fits");
    auto place = [](int row, int piece) { return 16 * row + (piece ^ row); };  // a piece of all rows on different banks
    u32x4* own = reinterpret_cast<u32x4*>(&red[wave][0][0][0][0]);
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int t = 0; t < T; ++t) {
        if (c == 0 && (int64_t)(chunk(0) + 1) * kW4Chunk > K) {
          const int64_t k = k_of(0, r);
          const int d = (int)(k < K - 8 ? 0 : k - (K - 8)), lo = (int)((int64_t)chunk(0) * kW4Chunk + 32 * (r >> 2) - k);
#pragma unroll
          for (int i = 0; i < 4; ++i) raw[c][t][i] = Op::window(raw[c][t][i], d, lo);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) own[place(4 * i + kq, r)] = Op::widen(raw[c][t][i]);
        wave_lds_order();
#pragma unroll
        for (int j = 0; j < 4; ++j) x[c][j][t] = Op::order(own[place(r, kPer == 1 ? 4 * kq + j : 4 * j + kq)]);
        wave_lds_order();
      }
    }
  }
  // a tile is staged before its turn, so that the load that takes its place
  // in the ring is under way
  stage_tile(ring_q[0], ring_s[0]);
  load_tile(tile0 + D, ring_q[0], ring_s[0]);

  // the staged tile's sums over this wave's k, into LDS
  auto multiply_tile = [&](float (&out)[T][256]) __attribute__((always_inline)) {
    f32x4 acc[T];
#pragma unroll
    for (int t = 0; t < T; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c < C / 2 || c < nc) {
        uint32_t u[4];
        if constexpr (kPer == 1) {
          __builtin_memcpy(u, &stage.q[r][4 * (4 * c + kq)], 16);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) u[j] = stage.q[r][4 * (4 * c + j) + kq];
        }
#pragma unroll
        for (int g = 0; g < kPer; ++g) {
          constexpr int kSteps = 4 / kPer;
          f32x4 sum[T];
#pragma unroll
          for (int t = 0; t < T; ++t) sum[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < kSteps; ++j) {
            const uint32_t v = u[g * kSteps + j];
            const Chunk w = Op::weights(v);
#pragma unroll
            for (int t = 0; t < T; ++t) Op::mma(sum[t], x[c][g * kSteps + j][t], w);
          }
#pragma unroll
          for (int t = 0; t < T; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][i] += stage.s[r][c * kPer + g] * sum[t][i];
        }
      }
#pragma unroll
    for (int t = 0; t < T; ++t)
      if (16 * t + 4 * kq < rows) *reinterpret_cast<f32x4*>(&out[t][4 * lane]) = acc[t];
  };
  // The waves' sums of a batch of tiles.  The two buffers take turns, so one
  // barrier a batch keeps a buffer's readers ahead of its next writers.
  int buf = 0;
  const int64_t y0 = row0 * a.ldy;
  float* const ws0 = p.ws + (part * a.M + row0) * p.ws_ld;
  auto join = [&](int tile) __attribute__((always_inline)) {
    __syncthreads();
    const int first = group * p.waves * 64;
    auto wave_of = [&](int w) { return (group * p.waves + w) & (kW4Waves - 1); };  // past the group's, any that is there
    auto put = [&](int m, int64_t n, float v) __attribute__((always_inline)) {
      if (p.S == 1)
        store_out(a.y, y0 + m * a.ldy + n, v * a.x_scale * (a.row_scale ? a.row_scale[row0 + m] : 1.f), a.out_dtype);
      else
        ws0[m * p.ws_ld + n] = v;
    };
    // Up to four rows an output to a thread, else four rows of a column: 4 x
    // 65536 x 8192 takes 53.7 and 57.1 us, 61 x 11001 x 4100 28.0 and 25.5.
    if (T == 1 && rows <= 4) {
      constexpr int kCols = 16 * kBatch;
      for (int o = tid - first; o < kCols * rows; o += 64 * p.waves) {
        const int m = o / kCols, i = o / 16 % kBatch, l = o & 15;
        const int64_t n = (int64_t)(tile + i) * 16 + l;
        float v = 0.f, waves[kW4Waves];
#pragma unroll
        for (int w = 0; w < kW4Waves; ++w) waves[w] = red[wave_of(w)][buf][i][0][4 * l + m];
#pragma unroll
        for (int w = 0; w < kW4Waves; ++w) v += w < p.waves ? waves[w] : 0.f;
        if (tile + i < tile1 && n < N) put(m, n, v);
      }
    } else {
      constexpr int kItems = kBatch * T * 64;
      for (int o = tid - first; o < kItems; o += 64 * p.waves) {
        const int l = o & 63, t = o / 64 % T, i = o / (64 * T);
        const int m = 16 * t + 4 * (l >> 4);
        const int64_t n = (int64_t)(tile + i) * 16 + (l & 15);
        if (tile + i < tile1 && m < rows && n < N) {
          f32x4 v = {0.f, 0.f, 0.f, 0.f}, waves[kW4Waves];
#pragma unroll
          for (int w = 0; w < kW4Waves; ++w) waves[w] = *reinterpret_cast<const f32x4*>(&red[wave_of(w)][buf][i][t][4 * l]);
#pragma unroll
          for (int w = 0; w < kW4Waves; ++w)
            if (w < p.waves) v += waves[w];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (m + e < rows) put(m + e, n, v[e]);
        }
      }
    }
    buf ^= 1;
  };

  for (int done = 0; done < most_tiles; done += kRound) {
    const int tile = tile0 + done;
#pragma unroll
    for (int b = 0; b < kRound; b += kBatch) {
#pragma unroll
      for (int d = b; d < b + kBatch; ++d) {
        if (tile + d < tile1) multiply_tile(red[wave][buf][d - b]);
        stage_tile(ring_q[(d + 1) % D], ring_s[(d + 1) % D]);
        load_tile(tile + d + 1 + D, ring_q[(d + 1) % D], ring_s[(d + 1) % D]);
      }
      if (done + b < most_tiles) join(tile + b);
    }
  }
}

// Launch for rows of type XT; T and C as chosen by the caller.
template <int XT, int FMT, int G, int WIDE>
int w4_mma_sizes(const W4Params& p, dim3 grid, int T, int C) {
  const dim3 block(64 * p.waves * p.groups);
  const bool lines = p.a.w.ldq % 128 == 0 && (uintptr_t)p.a.w.q % 128 == 0;
  switch (16 * T + C) {
#define GT_W4_RUN(T, C, D, ONCE) \
  hipLaunchKernelGGL((w4_mma_kernel<XT, FMT, G, WIDE, T, C, D, ONCE>), grid, block, 0, p.a.stream, p)
#define GT_W4_SIZE(T, C, D) \
  case 16 * T + C: GT_W4_RUN(T, C, D, 0); break;
#define GT_W4_LINES(T, C, D)   \
  case 16 * T + C:             \
    if (lines)                 \
      GT_W4_RUN(T, C, D, 1);   \
    else                       \
      GT_W4_RUN(T, C, D, 0);   \
    break;
    GT_W4_SIZE(1, 1, 4)
    GT_W4_LINES(1, 2, 4)
    GT_W4_LINES(1, 4, 2)
    GT_W4_SIZE(2, 1, 4)
    GT_W4_SIZE(2, 2, 4)
    GT_W4_SIZE(4, 1, 2)
    GT_W4_SIZE(4, 2, 2)
#undef GT_W4_LINES
#undef GT_W4_SIZE
#undef GT_W4_RUN
    default: return gt::LS_UNSUPPORTED;
  }
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

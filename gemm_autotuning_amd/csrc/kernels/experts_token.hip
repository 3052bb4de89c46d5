// experts_token.hip -- a layer of gated experts for a token or so few that they
// hardly share an expert: two launches of dot products instead of grouped.h's
// three of tiles.
//
//   up:   act[j, h] = act(gate_e x) * (up_e x), a workgroup to four h of slot j
//   down: y[n] = base[n] + sum_j sum_h (weight[j] act[j, h]) down_e[n, h], a
//         workgroup to eight n, all slots in it
//
// The weights bound it.  A wave takes units of its workgroup's eight rows,
// 1 KB of each, 16 bytes to a lane, and multiplies them in fp32 by the
// activations that it loads with them (the second product's times their slot's
// weight).  It has one unit at a time: four waves and more to a SIMD cover
// each other's loads better than half as many with two units each (one token
// of 128 experts 2048 x 768 bf16, eight of them named: 18.4 us so, 19.5 with
// two; 4 of int4 experts 4096 x 2048 20.8 and 23.1).  Those 18.4 us are 75 MB
// at 4.1 TB/s, of which the two launches' starts and ends, 2.5 us each, and
// the chain from the choice over the loads to the joined sums are most of what
// lies above 12; the int4 ones' 53 MB take 18 instructions to eight weights
// besides, some 6 us of the 20.8, and each wave has one unit, so that nothing is
// loaded behind the choice's latency or between the launches.  The lanes' sums
// are joined at the end, the waves' through LDS, in order.
#include "elements.h"
#include "grouped.h"
#include "launchers.h"

namespace gtk {
namespace {

constexpr int kRows = 8;  // of weights, to a workgroup

// The eight weights of a dword of codes, in order: e2m1 as they are, integers by
// way of e4m3 (w4_mma.h), 18 instructions with the products where conversions
// of single nibbles make 24 (2 tokens, 4 of 64 experts 4096 x 2048, 32.9 us and 33.9).
template <int FMT>
__device__ __forceinline__ void codes(uint32_t u, float (&w)[8]) {
  if constexpr (FMT == W4_E2M1) {
    const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.f, 1);
    const auto c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.f, 3);
    w[0] = a[0], w[1] = a[1], w[2] = b[0], w[3] = b[1], w[4] = c[0], w[5] = c[1], w[6] = d[0], w[7] = d[1];
  } else {
    uint32_t lo, hi;
    int4_to_e4m3(u, &lo, &hi);
    const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo, 512.f, false), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo, 512.f, true);
    const auto c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, 512.f, false), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, 512.f, true);
    w[0] = a[0], w[2] = a[1], w[4] = b[0], w[6] = b[1], w[1] = c[0], w[3] = c[1], w[5] = d[0], w[7] = d[1];
  }
}

// WIDE: the scales are fp32.
template <int PHASE, int XT, int FMT, int WIDE>
__global__ __launch_bounds__(512, 4) void token_kernel(gt::MoeArgs a, float* act, int64_t act_ld) {
  constexpr bool k4 = FMT != GROUPED_16, kDown = PHASE == GROUPED_DOWN;
  constexpr int kEach = k4 ? 32 : 8;              // elements of a row to a lane
  constexpr int kPieces = kDown ? kEach / 4 : kEach / 8;  // of 16 bytes, that the activations come in
  typedef typename std::conditional<WIDE, uint32_t, uint16_t>::type Scale;
  __shared__ float sums[8][kRows];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
  const int64_t t = blockIdx.z;
  const gt::ExpertWeights& w = kDown ? a.down : a.gate_up;
  const int K = (int)(kDown ? a.H : a.K), row_bytes = k4 ? (K + 1) / 2 : 2 * K;
  const int of_slot = (K + 64 * kEach - 1) / (64 * kEach), units = kDown ? of_slot * a.topk : of_slot;
  const int slots = lane < a.topk ? a.index[t * a.ldi + lane] : -1;
  const float weights = kDown && lane < a.topk ? a.weight[t * a.ldw + lane] : 1.f;
  const int first = kDown ? 0 : blockIdx.y;
  if (!kDown) {
    const int e = __builtin_amdgcn_readlane(slots, first);
    if (e < 0 || e >= a.E) return;
  }
  const int64_t n0 = (int64_t)blockIdx.x * (kDown ? kRows : kRows / 2);
  auto row = [&](int i) {
    return kDown ? min(n0 + i, a.K - 1) : (i < kRows / 2 ? min(n0 + i, a.H - 1) : a.H + min(n0 + i - kRows / 2, a.H - 1));
  };
  struct Unit {
    u32x4 q[kRows], x[kPieces];
    Scale s[kRows];
    int slot, k0;  // of the lane
  };
  auto load = [&](int unit, Unit& u) __attribute__((always_inline)) {
    u.slot = first + (kDown ? unit / of_slot : 0);
    const int c = kDown ? unit % of_slot : unit, at = min(1024 * c + 16 * lane, row_bytes - 16);
    const int named = __builtin_amdgcn_readlane(slots, u.slot), e = named >= 0 && named < a.E ? named : 0;
    u.k0 = (64 * c + lane) * kEach;
    const char* const p = w.p + e * w.stride;
#pragma unroll
    for (int i = 0; i < kRows; ++i) u.q[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p + row(i) * w.ld + at));
    if constexpr (k4) {
      const int64_t g = min(u.k0, K - 1) >> a.group_lg;
      const Scale* const s = static_cast<const Scale*>(w.scales) + e * w.s_lde + g * w.s_ldg;
#pragma unroll
      for (int i = 0; i < kRows; ++i) u.s[i] = s[row(i) * w.s_ldn];
    }
    const char* const x = kDown ? reinterpret_cast<const char*>(act + (t * a.topk + u.slot) * act_ld)
                                : static_cast<const char*>(a.x) + t * a.ldx * 2;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      u.x[i] = *reinterpret_cast<const u32x4_any*>(x + (kDown ? 4 * min(u.k0 + 4 * i, (K - 1) & ~3) : 2 * min(u.k0 + 8 * i, K - 8)));
  };
  float acc[kRows] = {};
  auto multiply = [&](Unit& u) __attribute__((always_inline)) {
    float x[kEach];
    const int named = __builtin_amdgcn_readlane(slots, u.slot);
    if (kDown && (named < 0 || named >= a.E)) return;
    const bool tail = __builtin_amdgcn_readlane(u.k0, 63) + kEach > K;
    if (tail) {
      // what lies past the row's end becomes zero, of the weights and of x
      const int at = 16 * (u.k0 / kEach), past = at - min(at, row_bytes - 16);
#pragma unroll
      for (int i = 0; i < kRows; ++i) u.q[i] = bytes_from(u.q[i], past);
      if constexpr (!kDown)
#pragma unroll
        for (int i = 0; i < kPieces; ++i) u.x[i] = bytes_from(u.x[i], 2 * max(0, u.k0 + 8 * i - (K - 8)));
    }
    const float f = kDown ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(weights), u.slot)) : 1.f;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      if constexpr (kDown) {
        x[e] = __uint_as_float(u.x[e / 4][e % 4]) * f;
        if (tail && u.k0 + e >= K) x[e] = 0.f;
      } else {
        x[e] = half_to_f32<XT>(u.x[e / 8][e / 2 % 4], e & 1);
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if constexpr (k4) {
        float sum = 0.f, v[8];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          codes<FMT>(u.q[i][d], v);
#pragma unroll
          for (int e = 0; e < 8; ++e) sum = fmaf(v[e], x[8 * d + e], sum);
        }
        float s;
        if constexpr (WIDE)
          s = __uint_as_float(u.s[i]);
        else
          s = a.scale_dtype == DT_BF16 ? __uint_as_float((uint32_t)u.s[i] << 16) : f16_bits_to_f32(u.s[i]);
        acc[i] += u.k0 < K ? s * sum : 0.f;  // past the end nothing, whatever the last scale is
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i] = fmaf(half_to_f32<XT>(u.q[i][e / 2], e & 1), x[e], acc[i]);
      }
    }
  };
  Unit u;
  for (int unit = wave; unit < units; unit += waves) {
    load(unit, u);
    multiply(u);
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const float v = wave_sum(acc[i]);
    if (lane == 0) sums[wave][i] = v;
  }
  __syncthreads();
  if constexpr (kDown) {
    const int64_t n = n0 + tid;
    if (tid >= kRows || n >= a.K) return;
    float y = a.base ? load_any(a.base, t * a.ldb + n, a.out_dtype) : 0.f;
    for (int v = 0; v < waves; ++v) y += sums[v][tid];
    store_out(a.y, t * a.ldy + n, y, a.out_dtype);
  } else {
    const int64_t h = n0 + tid;
    if (tid >= kRows / 2 || h >= a.H) return;
    float g = 0.f, u = 0.f;
    for (int v = 0; v < waves; ++v) {
      g += sums[v][tid];
      u += sums[v][kRows / 2 + tid];
    }
    act[(t * a.topk + first) * act_ld + h] = activated(g, u, a.activation);
  }
}

}  // namespace
}  // namespace gtk

namespace gt {
namespace {

template <int XT, int FMT, int WIDE>
int token(const MoeArgs& a, float* act, int64_t act_ld) {
  const int64_t each = 64 * (FMT == gtk::GROUPED_16 ? 8 : 32);
  const int up = (int)std::min<int64_t>(4, (a.K + each - 1) / each),
            down = (int)std::min<int64_t>(8, (a.H + each - 1) / each * a.topk);
  hipLaunchKernelGGL((gtk::token_kernel<gtk::GROUPED_GATE_UP, XT, FMT, WIDE>), dim3((unsigned)((a.H + 3) / 4), (unsigned)a.topk, (unsigned)a.M),
                     dim3(64 * up), 0, a.stream, a, act, act_ld);
  hipLaunchKernelGGL((gtk::token_kernel<gtk::GROUPED_DOWN, XT, FMT, WIDE>), dim3((unsigned)((a.K + 7) / 8), 1, (unsigned)a.M), dim3(64 * down),
                     0, a.stream, a, act, act_ld);
  return hipGetLastError() == hipSuccess ? LS_OK : LS_HIP_ERROR;
}
template <int XT>
int token(const MoeArgs& a, float* act, int64_t act_ld) {
  const bool wide = a.scale_dtype == DT_F32;
  if (a.format == gtk::W4_INT4) return wide ? token<XT, gtk::W4_INT4, 1>(a, act, act_ld) : token<XT, gtk::W4_INT4, 0>(a, act, act_ld);
  if (a.format == gtk::W4_E2M1) return wide ? token<XT, gtk::W4_E2M1, 1>(a, act, act_ld) : token<XT, gtk::W4_E2M1, 0>(a, act, act_ld);
  return token<XT, gtk::GROUPED_16, 0>(a, act, act_ld);
}

}  // namespace

int launch_moe_tokens(const MoeArgs& a, float* act, int64_t act_ld) {
  return a.x_dtype == DT_BF16 ? token<DT_BF16>(a, act, act_ld) : token<DT_F16>(a, act, act_ld);
}

}  // namespace gt

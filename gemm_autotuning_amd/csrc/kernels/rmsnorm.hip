// rmsnorm.hip -- the RMS norm with the residual's addition, and its backward
// pass.
//
//   h = x + r,  rstd = 1/sqrt(mean h^2 + eps),  y = h * rstd * (w + offset)
//
// Few operations per byte: HBM bounds both directions, and the rule is one
// trip over the data.  A row belongs to NT threads (a wave or a workgroup),
// which hold it in registers, C pieces of 16 input bytes each, while its sum
// of squares is joined; nothing is read twice.  8192 x 4096 bf16 with the
// residual and its sum: 48.5 us, 5.5 TB/s, where a copy of 2 GiB reaches 5.0.
#include "elements.h"
#include "launchers.h"

namespace gtk {

// A value of each of the NT threads of a row joined over them.  Two parts of
// LDS take turns, so that one barrier a sum keeps a part's readers ahead of
// its next writers.  NT = 64 needs neither.
template <int NT>
struct RowJoin {
  static constexpr int kWaves = NT / 64;
  uint32_t* part;  // 2 * kWaves
  int turn = 0;
  template <class F>
  __device__ __forceinline__ uint32_t join(uint32_t v, F f) {
    v = wave_join(v, f);
    if constexpr (kWaves == 1) {
      return v;
    } else {
      uint32_t* p = part + turn * kWaves;
      turn ^= 1;
      if ((threadIdx.x & 63) == 0) p[threadIdx.x >> 6] = v;
      __syncthreads();
      v = p[0];
#pragma unroll
      for (int i = 1; i < kWaves; ++i) v = f(v, p[i]);
      return v;
    }
  }
  __device__ __forceinline__ float sum(float v) {
    return __uint_as_float(join(__float_as_uint(v), [](uint32_t a, uint32_t b) {
      return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
  }
  // largest |v| by the bits below the sign: NaN above infinity above the finite
  __device__ __forceinline__ uint32_t max_bits(uint32_t v) {
    return join(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
  }
};

// The row's last N % E elements go one to a thread beside its pieces, so no
// piece is ever partial.
template <int IN, int OUT, int NT, int C>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void rmsnorm_kernel(gt::NormArgs a) {
  constexpr int kRows = NT < 256 ? 256 / NT : 1;  // rows a workgroup takes at a time
  constexpr unsigned E = 16 / sizeof(typename Elem<IN>::T);
  constexpr bool kEarlyWeights = C * E <= 16;  // in flight with the row where registers allow
  typedef typename Elem<IN>::T TI;
  typedef typename Elem<OUT>::T TO;
  __shared__ uint32_t part[2 * (NT / 64)];
  RowJoin<NT> row{part};
  const unsigned t = threadIdx.x % NT, N = (unsigned)a.N;
  const unsigned whole = N / E * E, last = whole + t;  // this thread's single element, if it is in the row
  for (int64_t m = (int64_t)blockIdx.x * kRows + threadIdx.x / NT; m < a.M; m += (int64_t)gridDim.x * kRows) {
    const TI* x = reinterpret_cast<const TI*>(a.x) + m * a.ldx;
    const TI* r = a.r ? reinterpret_cast<const TI*>(a.r) + m * a.ldr : nullptr;
    Piece<IN, E> px[C], pr[C];
    TI xl = 0, rl = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const unsigned n = (t + c * NT) * E;
      px[c].clear();
      pr[c].clear();
      if (n < whole) px[c].load(x + n);
    }
    if (last < N) xl = x[last];
    if (r) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const unsigned n = (t + c * NT) * E;
        if (n < whole) pr[c].load(r + n);
      }
      if (last < N) rl = r[last];
    }
    float w[kEarlyWeights ? C * E : E];
    auto gain = [&](int c) {
      const unsigned n = (t + c * NT) * E;
      float* g = w + (kEarlyWeights ? c * E : 0);
      if (a.w && n < whole) load_weights<E>(a.w, n, a.w_dtype, g);
    };
    if constexpr (kEarlyWeights) {
#pragma unroll
      for (int c = 0; c < C; ++c) gain(c);
    }
    float wl = 1.f;
    if (a.w && last < N) wl = load_any(a.w, last, a.w_dtype) + a.offset;
    float h[C * E], hl = Elem<IN>::get(xl) + (r ? Elem<IN>::get(rl) : 0.f);
    float q = hl * hl;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float v = px[c].get(e) + (r ? pr[c].get(e) : 0.f);
        h[c * E + e] = v;
        q += v * v;
      }
    if (a.sum) {
      TI* s = reinterpret_cast<TI*>(a.sum) + m * a.lds;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const unsigned n = (t + c * NT) * E;
        if (n < whole) store_piece<IN, E>(s + n, h + c * E, a.past_caches);
      }
      if (last < N) s[last] = Elem<IN>::put(hl);
    }
    const float rstd = 1.0f / sqrtf(row.sum(q) / (float)N + a.eps);
    if (t == 0 && a.rstd) a.rstd[m] = rstd;
    const float near = OUT == DT_E4M3 ? a.near : 1.f;
    hl = hl * rstd * near * wl;
    uint32_t big = last < N ? __float_as_uint(hl) & 0x7fffffffu : 0u;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if constexpr (!kEarlyWeights) gain(c);
      const float* g = w + (kEarlyWeights ? c * E : 0);
      uint32_t most = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float& v = h[c * E + e];
        v *= rstd;
        if constexpr (OUT == DT_E4M3) v *= near;
        if (a.w) v *= g[e] + a.offset;
        if constexpr (OUT == DT_E4M3) most = max(most, __float_as_uint(v) & 0x7fffffffu);
      }
      if ((t + c * NT) * E < whole) big = max(big, most);
    }
    if constexpr (OUT == DT_E4M3) {
      float inv;
      if (a.row_scale) {
        const float amax = __uint_as_float(row.max_bits(big));
        const float scale = (amax < 0x1p-100f ? 0x1p-100f : amax) / 448.f;
        if (t == 0) a.row_scale[m] = scale;
        inv = 1.0f / scale;
      } else {
        inv = 1.0f / (a.scale * near);
      }
      hl *= inv;
#pragma unroll
      for (int e = 0; e < C * E; ++e) h[e] *= inv;
    }
    TO* y = reinterpret_cast<TO*>(a.y) + m * a.ldy;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const unsigned n = (t + c * NT) * E;
      if (n < whole) store_piece<OUT, E>(y + n, h + c * E, a.past_caches);
    }
    if (last < N) y[last] = Elem<OUT>::put(hl);
  }
}

// Rows too long for a workgroup's registers: the row is read again (from the
// caches) for its scale and for its output.  A thread writes an element only
// after its last read of it, so results may lie over inputs here too.
constexpr int kLongNT = 1024;
template <int IN, int OUT>
__global__ __launch_bounds__(kLongNT) void rmsnorm_long_kernel(gt::NormArgs a) {
  typedef typename Elem<IN>::T TI;
  typedef typename Elem<OUT>::T TO;
  __shared__ uint32_t part[2 * (kLongNT / 64)];
  RowJoin<kLongNT> row{part};
  const unsigned N = (unsigned)a.N;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const TI* x = reinterpret_cast<const TI*>(a.x) + m * a.ldx;
    const TI* r = a.r ? reinterpret_cast<const TI*>(a.r) + m * a.ldr : nullptr;
    TI* s = a.sum ? reinterpret_cast<TI*>(a.sum) + m * a.lds : nullptr;
    TO* y = reinterpret_cast<TO*>(a.y) + m * a.ldy;
    auto h_of = [&](unsigned n) { return Elem<IN>::get(x[n]) + (r ? Elem<IN>::get(r[n]) : 0.f); };
    auto w_of = [&](unsigned n) { return a.w ? load_any(a.w, n, a.w_dtype) + a.offset : 1.f; };
    float q = 0;
#pragma unroll 8
    for (unsigned n = threadIdx.x; n < N; n += kLongNT) {
      const float h = h_of(n);
      q += h * h;
    }
    const float rstd = 1.0f / sqrtf(row.sum(q) / (float)N + a.eps);
    if (threadIdx.x == 0 && a.rstd) a.rstd[m] = rstd;
    float inv = 1.0f;
    if constexpr (OUT == DT_E4M3) {
      inv = 1.0f / (a.scale * a.near);
      if (a.row_scale) {
        uint32_t big = 0;
#pragma unroll 8
        for (unsigned n = threadIdx.x; n < N; n += kLongNT)
          big = max(big, __float_as_uint(h_of(n) * rstd * w_of(n)) & 0x7fffffffu);
        const float amax = __uint_as_float(row.max_bits(big));
        const float scale = (amax < 0x1p-100f ? 0x1p-100f : amax) / 448.f;
        if (threadIdx.x == 0) a.row_scale[m] = scale;
        inv = 1.0f / scale;
      }
    }
    for (unsigned n = threadIdx.x; n < N; n += kLongNT) {
      const float h = h_of(n);
      const float v = h * rstd * (OUT == DT_E4M3 ? a.near : 1.f) * w_of(n);
      if (s) s[n] = Elem<IN>::put(h);
      y[n] = Elem<OUT>::put(OUT == DT_E4M3 ? v * inv : v);
    }
  }
}

// ---- backward
//
//   g = dy * (w + offset), n = h * rstd
//   dx = rstd * (g - n * mean(g * n)) + dsum,   dw = sum over rows of dy * n
//
// One pass for both: a workgroup walks rows gridDim apart, its threads own
// columns, so dw's partial sums stay in registers and go to the workspace
// once (blocks x N floats), where rmsnorm_join_kernel adds them in block
// order.  Where registers allow, a row's successor is loaded while the row's
// mean is joined.  8192 x 4096 bf16 with dsum: 51.8 us, 5.2 TB/s.
//
// That second launch is most of the time of a small gradient (500 x 1000 f16:
// 7.0 us of both, 4.0 of one launch).  Where a workgroup reads 32 columns of
// all rows in about the time a launch takes, the first dw_blocks workgroups
// do that instead, and the others only make dx.
constexpr unsigned kDwCols = 32;
template <int IN, int DY, int THREADS>
__device__ void dw_columns(const gt::NormBwdArgs& a, unsigned block) {
  constexpr unsigned E = 16 / sizeof(typename Elem<IN>::T), kLanes = kDwCols / E, kAt = THREADS / kLanes, kSegs = THREADS / kDwCols;
  typedef typename Elem<IN>::T TI;
  typedef typename Elem<DY>::T TD;
  __shared__ float part[kAt][kDwCols + 1];
  __shared__ float segs[kSegs][kDwCols];
  const unsigned t = threadIdx.x, N = (unsigned)a.N, M = (unsigned)a.M;
  const unsigned n = block * kDwCols + t % kLanes * E;
  float s[E];
#pragma unroll
  for (int e = 0; e < E; ++e) s[e] = 0.f;
  for (unsigned m0 = t / kLanes; m0 < M; m0 += 4 * kAt) {
    Piece<IN, E> h[4];
    Piece<DY, E> dy[4];
    float rstd[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned m = min(m0 + i * kAt, M - 1);
      h[i].clear();
      dy[i].clear();
      if (n + E <= N) {
        h[i].load(reinterpret_cast<const TI*>(a.h) + m * a.ldh + n);
        dy[i].load(reinterpret_cast<const TD*>(a.dy) + m * a.lddy + n);
      }
      rstd[i] = a.rstd[m];
    }
    if (N % E && block == N / kDwCols) {  // after every whole piece's load is under way
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n < N && n + E > N) {
          const unsigned m = min(m0 + i * kAt, M - 1);
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (n + e < N) {
              h[i].set(e, reinterpret_cast<const TI*>(a.h)[m * a.ldh + n + e]);
              dy[i].set(e, reinterpret_cast<const TD*>(a.dy)[m * a.lddy + n + e]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (m0 + i * kAt < M)
#pragma unroll
        for (int e = 0; e < E; ++e) s[e] += dy[i].get(e) * (h[i].get(e) * rstd[i]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) part[t / kLanes][t % kLanes * E + e] = s[e];
  __syncthreads();
  const unsigned col = t % kDwCols, seg = t / kDwCols;
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < kAt / kSegs; ++i) v += part[seg * (kAt / kSegs) + i][col];
  segs[seg][col] = v;
  __syncthreads();
  if (seg == 0 && block * kDwCols + col < N) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kSegs; ++i) v += segs[i][col];
    store_out(a.dw, block * kDwCols + col, v, a.dw_dtype);
  }
}

template <int IN, int DY, int NT, int C>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void rmsnorm_bwd_kernel(gt::NormBwdArgs a) {
  constexpr int kRows = NT < 256 ? 256 / NT : 1;
  constexpr unsigned E = 16 / sizeof(typename Elem<IN>::T);
  constexpr bool kAhead = C * (2 * 4 + Piece<DY, E>::kWords) <= 64;
  typedef typename Elem<IN>::T TI;
  typedef typename Elem<DY>::T TD;
  __shared__ uint32_t part[2 * (NT / 64)];
  __shared__ float joined[kRows > 1 ? kRows * (C * E * NT + E) : 1];
  RowJoin<NT> row{part};
  const unsigned t = threadIdx.x % NT, N = (unsigned)a.N;
  const unsigned whole = N / E * E, last = whole + t;
  struct Raw {
    Piece<IN, E> h[C], ds[C];
    Piece<DY, E> dy[C];
    TI hl, dsl;
    TD dyl;
    float rstd;
  };
  if (blockIdx.x < (unsigned)a.dw_blocks) return dw_columns<IN, DY, (NT < 256 ? 256 : NT)>(a, blockIdx.x);
  const unsigned block = blockIdx.x - a.dw_blocks, blocks = gridDim.x - a.dw_blocks;
  auto load = [&](int64_t m, Raw& v) {
    const TI* h = reinterpret_cast<const TI*>(a.h) + m * a.ldh;
    const TD* dy = reinterpret_cast<const TD*>(a.dy) + m * a.lddy;
    const TI* ds = a.dsum ? reinterpret_cast<const TI*>(a.dsum) + m * a.ldds : nullptr;
    v.hl = v.dsl = 0;
    v.dyl = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const unsigned n = (t + c * NT) * E;
      v.h[c].clear();
      v.dy[c].clear();
      v.ds[c].clear();
      if (n < whole) {
        v.h[c].load(h + n);
        v.dy[c].load(dy + n);
      }
    }
    if (ds) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const unsigned n = (t + c * NT) * E;
        if (n < whole) v.ds[c].load(ds + n);
      }
    }
    if (last < N) {
      v.hl = h[last];
      v.dyl = dy[last];
      if (ds) v.dsl = ds[last];
    }
    v.rstd = a.rstd[m];
  };
  const int64_t step = (int64_t)blocks * kRows;
  int64_t m = (int64_t)block * kRows + threadIdx.x / NT;
  Raw v;
  if (m < a.M) load(m, v);
  float w[C][E], dw[C * E], wl = 1.f, dwl = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const unsigned n = (t + c * NT) * E;
    if (a.w && n < whole) load_weights<E>(a.w, n, a.w_dtype, w[c]);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      w[c][e] = a.w ? w[c][e] + a.offset : 1.f;
      dw[c * E + e] = 0.f;
    }
  }
  if (a.w && last < N) wl = load_any(a.w, last, a.w_dtype) + a.offset;
  for (; m < a.M; m += step) {
    Raw next;
    if (kAhead && m + step < a.M) load(m + step, next);
    const float dyl = Elem<DY>::get(v.dyl), nl = Elem<IN>::get(v.hl) * v.rstd;
    float q = 0;
    if (last < N) {
      dwl += dyl * nl;
      q = dyl * wl * nl;
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
      if ((t + c * NT) * E < whole) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float dy = v.dy[c].get(e), n = v.h[c].get(e) * v.rstd;
          dw[c * E + e] += dy * n;
          q += dy * w[c][e] * n;
        }
      }
    if (a.dx) {
      TI* dx = reinterpret_cast<TI*>(a.dx) + m * a.lddx;
      const float mean = row.sum(q) / (float)N;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const unsigned i = (t + c * NT) * E;
        float o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float g = v.dy[c].get(e) * w[c][e], n = v.h[c].get(e) * v.rstd;
          o[e] = v.rstd * (g - n * mean) + v.ds[c].get(e);
        }
        if (i < whole) store_piece<IN, E>(dx + i, o, a.past_caches);
      }
      if (last < N) dx[last] = Elem<IN>::put(v.rstd * (dyl * wl - nl * mean) + Elem<IN>::get(v.dsl));
    }
    if constexpr (kAhead)
      v = next;
    else if (m + step < a.M)
      load(m + step, v);
  }
  if (!a.dw || a.dw_blocks) return;
  if constexpr (kRows > 1) {  // the workgroup's rows first, in order
    constexpr unsigned kSpan = C * E * NT + E;
    float* mine = joined + (threadIdx.x / NT) * kSpan;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const unsigned n = (t + c * NT) * E;
      if (n < whole)
#pragma unroll
        for (int e = 0; e < E; ++e) mine[n + e] = dw[c * E + e];
    }
    if (last < N) mine[last] = dwl;
    __syncthreads();
    for (unsigned n = threadIdx.x; n < N; n += NT * kRows) {
      float s = joined[n];
#pragma unroll
      for (int k = 1; k < kRows; ++k) s += joined[k * kSpan + n];
      a.ws[(int64_t)blockIdx.x * N + n] = s;
    }
  } else {
    float* p = a.ws + (int64_t)blockIdx.x * N;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const unsigned n = (t + c * NT) * E;
      if (n < whole) store_piece<DT_F32, E>(p + n, dw + c * E);
    }
    if (last < N) p[last] = dwl;
  }
}

// dw from the blocks' partial sums: 16 columns to a workgroup (64 bytes of a
// block's row), 32 slices of the blocks side by side, then the slices in order.
constexpr int kJoinCols = 16, kJoinSlices = 32;
__global__ __launch_bounds__(kJoinCols* kJoinSlices) void rmsnorm_join_kernel(const float* ws, void* dw, int blocks, int N,
                                                                              int dtype) {
  __shared__ float part[kJoinSlices][kJoinCols];
  const int c = threadIdx.x % kJoinCols, s = threadIdx.x / kJoinCols;
  const int n = blockIdx.x * kJoinCols + c;
  float v = 0;
  if (n < N) {
    int b = s;
    for (; b + 7 * kJoinSlices < blocks; b += 8 * kJoinSlices) {
      float p[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = ws[(int64_t)(b + j * kJoinSlices) * N + n];
#pragma unroll
      for (int j = 0; j < 8; ++j) v += p[j];
    }
    for (; b < blocks; b += kJoinSlices) v += ws[(int64_t)b * N + n];
  }
  part[s][c] = v;
  __syncthreads();
  if (s == 0 && n < N) {
#pragma unroll
    for (int i = 1; i < kJoinSlices; ++i) v += part[i][c];
    store_out(dw, n, v, dtype);
  }
}

// Rows too long for one workgroup's registers: dx reads its row twice (the
// second time from the caches), dw is a pass of its own with a thread to a
// column and rows gridDim.y apart.
template <int IN, int DY>
__global__ __launch_bounds__(kLongNT) void rmsnorm_long_dx_kernel(gt::NormBwdArgs a) {
  __shared__ uint32_t part[2 * (kLongNT / 64)];
  RowJoin<kLongNT> row{part};
  typedef typename Elem<IN>::T TI;
  typedef typename Elem<DY>::T TD;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const TD* dy = reinterpret_cast<const TD*>(a.dy) + m * a.lddy;
    const TI* h = reinterpret_cast<const TI*>(a.h) + m * a.ldh;
    const TI* ds = a.dsum ? reinterpret_cast<const TI*>(a.dsum) + m * a.ldds : nullptr;
    TI* dx = reinterpret_cast<TI*>(a.dx) + m * a.lddx;
    const float rstd = a.rstd[m];
    auto g_of = [&](int64_t n) {
      return Elem<DY>::get(dy[n]) * (a.w ? load_any(a.w, n, a.w_dtype) + a.offset : 1.f);
    };
    float q = 0;
    for (int64_t n = threadIdx.x; n < a.N; n += kLongNT) q += g_of(n) * (Elem<IN>::get(h[n]) * rstd);
    const float mean = row.sum(q) / (float)a.N;
    for (int64_t n = threadIdx.x; n < a.N; n += kLongNT) {
      const float v = rstd * (g_of(n) - Elem<IN>::get(h[n]) * rstd * mean);
      dx[n] = Elem<IN>::put(v + (ds ? Elem<IN>::get(ds[n]) : 0.f));
    }
  }
}
template <int IN, int DY>
__global__ __launch_bounds__(256) void rmsnorm_long_dw_kernel(gt::NormBwdArgs a) {
  typedef typename Elem<IN>::T TI;
  typedef typename Elem<DY>::T TD;
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (n >= a.N) return;
  float s = 0;
  for (int64_t m = blockIdx.y; m < a.M; m += gridDim.y)
    s += Elem<DY>::get(reinterpret_cast<const TD*>(a.dy)[m * a.lddy + n]) *
         (Elem<IN>::get(reinterpret_cast<const TI*>(a.h)[m * a.ldh + n]) * a.rstd[m]);
  a.ws[(int64_t)blockIdx.y * a.N + n] = s;
}

}  // namespace gtk

namespace gt {

namespace {
int status() { return hipGetLastError() == hipSuccess ? LS_OK : LS_HIP_ERROR; }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Threads of a row, by its pieces of 16 input bytes: a wave where two pieces a
// lane hold it (no barrier), else a workgroup.  With fewer rows than CUs a
// longer row's own latency counts, and more threads share it: one row of 8192
// bf16 to e4m3 takes 3.8 us with 1024 threads and 4.5 with 256 (shorter rows
// gain nothing: 4096 elements 3.5 and 3.3).
constexpr int64_t kMostPieces = 4096;
bool long_rows(int64_t N, int elem) { return ceil_div(N * elem, 16) > kMostPieces; }
struct RowShape {
  int NT, C;
};
RowShape row_shape(int64_t N, int64_t M, int elem, int cus) {
  const int64_t pieces = ceil_div(N * elem, 16);
  if (pieces <= 64) return {64, 1};
  if (pieces <= 128) return {64, 2};
  if (pieces <= 256) return {256, 1};
  if (pieces <= 512) return {256, 2};
  if (pieces <= 1024) return M < cus ? RowShape{1024, 1} : RowShape{256, 4};
  if (pieces <= 2048) return {512, 4};
  return {1024, 4};
}

// Workgroups of a launch, whose threads must be fewer than 2^32: those of up to
// 1024 threads walk the rows past them.
constexpr int64_t kMostGroups = 1 << 21;

template <int IN, int OUT, int NT, int C>
int norm_launch(const NormArgs& a) {
  constexpr int kRows = NT < 256 ? 256 / NT : 1;
  const int64_t wgs = ceil_div(a.M, kRows);
  const dim3 g((unsigned)(wgs < kMostGroups ? wgs : kMostGroups)), b(NT < 256 ? 256 : NT);
  hipLaunchKernelGGL((gtk::rmsnorm_kernel<IN, OUT, NT, C>), g, b, 0, a.stream, a);
  return status();
}
template <int IN, int OUT>
int norm_shape(const NormArgs& a) {
  if (long_rows(a.N, elem_bytes(IN))) {
    const dim3 g((unsigned)(a.M < kMostGroups ? a.M : kMostGroups));
    hipLaunchKernelGGL((gtk::rmsnorm_long_kernel<IN, OUT>), g, dim3(gtk::kLongNT), 0, a.stream, a);
    return status();
  }
  const RowShape s = row_shape(a.N, a.M, elem_bytes(IN), a.cus);
  switch (s.NT * 32 + s.C) {
    case 64 * 32 + 1: return norm_launch<IN, OUT, 64, 1>(a);
    case 64 * 32 + 2: return norm_launch<IN, OUT, 64, 2>(a);
    case 256 * 32 + 1: return norm_launch<IN, OUT, 256, 1>(a);
    case 256 * 32 + 2: return norm_launch<IN, OUT, 256, 2>(a);
    case 256 * 32 + 4: return norm_launch<IN, OUT, 256, 4>(a);
    case 1024 * 32 + 1: return norm_launch<IN, OUT, 1024, 1>(a);
    case 512 * 32 + 4: return norm_launch<IN, OUT, 512, 4>(a);
    default: return norm_launch<IN, OUT, 1024, 4>(a);
  }
}
template <int IN>
int norm_in(const NormArgs& a) {
  switch (a.out_dtype) {
    case DT_F32: return norm_shape<IN, DT_F32>(a);
    case DT_F16: return norm_shape<IN, DT_F16>(a);
    case DT_BF16: return norm_shape<IN, DT_BF16>(a);
    default: return norm_shape<IN, DT_E4M3>(a);
  }
}

// Longest rows that the one-pass kernel holds: h, dy, dsum, w and dw of a row
// in the registers of 512 threads (f32 rows have half the elements a piece).
bool bwd_long(const NormBwdArgs& a) { return a.N > 16384; }
RowShape bwd_shape(const NormBwdArgs& a) {
  const RowShape s = row_shape(a.N, a.M, elem_bytes(a.in_dtype), 0);
  return s.NT == 1024 ? RowShape{512, 8} : s;
}
// Workgroups of the backward pass: each leaves N partial sums of dw, so they
// are as few as keep the memory busy.
int bwd_blocks(const NormBwdArgs& a) {
  if (bwd_long(a)) return (int)(a.M < 64 ? a.M : 64);
  const RowShape s = bwd_shape(a);
  // 8192 x 4096 bf16 (C = 2) with one, two, four a CU: 42.6, 44.5, 48.5 us;
  // 16384 x 2048 (C = 1): 52.1, 41.7, 44.6; 2048 x 16384 (C = 4): 50.6, 59.5
  const int64_t b = ceil_div(a.M, s.NT < 256 ? 256 / s.NT : 1), most = (int64_t)a.cus * (s.C == 1 ? 2 : 1);
  return (int)(b < most ? b : most);
}
// dw by columns beside dx: few rows (four round trips of a workgroup's loads;
// 1000 x 2000 f16 7.3 us, 9.8 in two launches; 1000 x 1000 f32, twice the
// bytes a row, 9.4 and 8.1), a second reading that the caches serve, and dx
// not written over what it reads.
int bwd_dw_blocks(const NormBwdArgs& a) {
  const bool small = a.M * elem_bytes(a.in_dtype) <= 2048 && a.M * a.N <= (1 << 21) && !bwd_long(a);
  return a.dw && small && a.dx != a.dy && a.dx != a.h ? (int)ceil_div(a.N, gtk::kDwCols) : 0;
}

template <int IN, int DY>
int bwd_types(const NormBwdArgs& a) {
  const int blocks = bwd_blocks(a);
  if (bwd_long(a)) {
    // dw first: dx may be written over dy or h
    if (a.dw) {
      const dim3 g((unsigned)ceil_div(a.N, 256), (unsigned)blocks);
      hipLaunchKernelGGL((gtk::rmsnorm_long_dw_kernel<IN, DY>), g, dim3(256), 0, a.stream, a);
    }
    if (a.dx) {
      const dim3 g((unsigned)(a.M < 65536 ? a.M : 65536));
      hipLaunchKernelGGL((gtk::rmsnorm_long_dx_kernel<IN, DY>), g, dim3(gtk::kLongNT), 0, a.stream, a);
    }
  } else {
    const RowShape s = bwd_shape(a);
    const dim3 g((unsigned)((a.dx || !a.dw_blocks ? blocks : 0) + a.dw_blocks)), b(s.NT < 256 ? 256 : s.NT);
    switch (s.NT * 32 + s.C) {
#define GT_BWD(NT, C) \
  case NT * 32 + C: hipLaunchKernelGGL((gtk::rmsnorm_bwd_kernel<IN, DY, NT, C>), g, b, 0, a.stream, a); break;
      GT_BWD(64, 1)
      GT_BWD(64, 2)
      GT_BWD(256, 1)
      GT_BWD(256, 2)
      GT_BWD(256, 4)
      GT_BWD(512, 4)
      default:
        if constexpr (IN == DT_F32)
          hipLaunchKernelGGL((gtk::rmsnorm_bwd_kernel<IN, DY, 512, 8>), g, b, 0, a.stream, a);
        else
          return LS_UNSUPPORTED;
#undef GT_BWD
    }
  }
  if (a.dw && !a.dw_blocks) {
    const dim3 g((unsigned)ceil_div(a.N, gtk::kJoinCols));
    hipLaunchKernelGGL(gtk::rmsnorm_join_kernel, g, dim3(gtk::kJoinCols * gtk::kJoinSlices), 0, a.stream, a.ws, a.dw, blocks,
                       (int)a.N, a.dw_dtype);
  }
  return status();
}
}  // namespace

int launch_rmsnorm(const NormArgs& args) {
  NormArgs a = args;
  const int e = elem_bytes(a.in_dtype);
  a.past_caches = (double)a.M * a.N * (e * (1 + !!a.r + !!a.sum) + elem_bytes(a.out_dtype)) > gtk::kPastCaches;
  // The quotient by a given scale is a product with its reciprocal, which
  // leaves fp32's normal numbers for scales near the ends of its range, as the
  // weighted value may; a power of two keeps both inside.
  const bool given = !a.row_scale && a.out_dtype == DT_E4M3;
  a.near = given && a.scale < 0x1p-64f ? 0x1p64f : (given && a.scale > 0x1p64f ? 0x1p-64f : 1.f);
  switch (a.in_dtype) {
    case DT_F32: return norm_in<DT_F32>(a);
    case DT_F16: return norm_in<DT_F16>(a);
    default: return norm_in<DT_BF16>(a);
  }
}

size_t rmsnorm_bwd_workspace_bytes(const NormBwdArgs& a) {
  return a.dw && !bwd_dw_blocks(a) ? (size_t)bwd_blocks(a) * a.N * 4 : 0;
}

int launch_rmsnorm_bwd(const NormBwdArgs& args) {
  NormBwdArgs a = args;
  a.dw_blocks = bwd_dw_blocks(a);
  const int e = elem_bytes(a.in_dtype);
  a.past_caches = (double)a.M * a.N * (e * (1 + !!a.dsum + !!a.dx) + elem_bytes(a.dy_dtype)) > gtk::kPastCaches;
  const bool wide = a.dy_dtype == DT_F32;
  switch (a.in_dtype) {
    case DT_F32: return bwd_types<DT_F32, DT_F32>(a);
    case DT_F16: return wide ? bwd_types<DT_F16, DT_F32>(a) : bwd_types<DT_F16, DT_F16>(a);
    default: return wide ? bwd_types<DT_BF16, DT_F32>(a) : bwd_types<DT_BF16, DT_BF16>(a);
  }
}

}  // namespace gt

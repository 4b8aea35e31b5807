// Norms at a block's boundary: the norm after the block with its gate, the
// residual scale and sum, and the next block's norm, in one pass over a row.
//
//   rms(v) = v r,  r = 1 / sqrt(mean(v^2) + eps)
//   h = x [act(g)];  p = rms(h) w_post [act(g)];  out = res + s p;
//   normed = rms(out) w_pre
// Backward of y = rms(v) w:  dv = r (dy w - vhat mean(dy w vhat)),
// dw = sum over rows of dy vhat, with vhat = v r.
//
// A row is read once and its elements stay in registers across both norms (up
// to 8192 columns; wider rows hold 32 elements a thread, and all but the
// aligned forward without a gate spill some of them: 4096 x 16384 forward 189
// us, 55 % of a copy's rate, backward 1104 us), so HBM is the bound; to reach
// it, a row's fixed cost (its sums over threads, its addresses) must be spread
// over many elements a thread.  Work split: TPR threads own a row (part of a
// warp for a head's row, a block for a wide one) with 16 elements a thread (32
// in the widest rows), and several blocks an SM, so that one row's loads run
// under another's sums.  (With 8 elements a thread and one or two blocks an SM,
// rows prefetched through registers or an asynchronous ring included, 16384 x
// 4096 took 0.21 to 0.33 ms.)  Each thread meets the same elements of every
// row, so the weights' gradients are sums of its own, kept in shared memory
// backward; the weights come out of L1, where the rows do not stay.  The grid
// is the resident blocks only.  Measured, in shares of a copy's rate: 16384 x
// 4096 with an fp32 residual 178 us (82 %), 524288 rows of 128 with a gate 85
// us (73 %), backward of 8192 x 4096 143 us (58 %; issue slots half used: three
// sums over the block a pair of rows, with one block of 16 warps an SM and
// nothing to run under them).
#include "kda_layer.cuh"

namespace kda {

namespace {

struct Gate {
  bool none, silu;
  // act(g) of a pair
  __device__ __forceinline__ f32x2 f(f32x2 g) const {
    if (none) return g;
    const f32x2 s = sigmoid2(g);
    return silu ? mul2(s, g) : s;
  }
  // s: sigmoid(g) -> act(g) and act'(g) = s (k + m (1 - s)) with act = s m:
  // m = 1, k = 0 for the sigmoid, m = g, k = 1 for SiLU
  __device__ __forceinline__ void fd(f32x2 g, f32x2 s, f32x2& f_, f32x2& d_) const {
    if (none) {
      f_ = g;
      d_ = both(1.f);
      return;
    }
    const f32x2 t = fma2(s, both(-1.f), both(1.f));
    f_ = silu ? mul2(s, g) : s;
    d_ = mul2(s, silu ? fma2(g, t, both(1.f)) : t);
  }
};

// Sums of N <= 4 values over the TPR threads of a row, in every one of them.
// TPR <= 32: exchanges.  Above, the row is the whole block: per-warp sums
// through shared memory; `turn` alternates between two buffers, so that one
// barrier per sum is enough (a buffer is written again only behind the next
// sum's barrier).  Every warp adds the warps' values in the same order.
struct RowSum {
  int tpr;
  int turn;
  float4* buf;  // [2][16]
  template <int N>
  __device__ __forceinline__ void operator()(float (&v)[N]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (tpr > o)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (tpr <= 32) return;
    float4* s = buf + turn * 16;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0)
      s[threadIdx.x >> 5] = make_float4(v[0], v[1 % N], v[2 % N], v[3 % N]);
    __syncthreads();
    const int warps = tpr >> 5;
    if (warps <= 4) {
      float4 t = s[0];
      for (int i = 1; i < warps; ++i) {
        const float4 u = s[i];
        t.x += u.x;
        if (N > 1) t.y += u.y;
        if (N > 2) t.z += u.z;
        if (N > 3) t.w += u.w;
      }
      v[0] = t.x;
      if (N > 1) v[1 % N] = t.y;
      if (N > 2) v[2 % N] = t.z;
      if (N > 3) v[3 % N] = t.w;
    } else {  // up to 16 warps: one value a lane, and exchanges
      const int lane = threadIdx.x & 15;
      float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
      if (lane < warps) t = s[lane];
      v[0] = t.x;
      if (N > 1) v[1 % N] = t.y;
      if (N > 2) v[2 % N] = t.z;
      if (N > 3) v[3 % N] = t.w;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
  }
};

// A row's elements pass once: they do not stay in L1.
template <typename T, int N>
__device__ __forceinline__ Raw<T, N> load_once(const T* p) {
  constexpr int BYTES = N * (int)sizeof(T);
  Raw<T, N> r;
  if constexpr (BYTES % 16 == 0) {
    uint4* q = reinterpret_cast<uint4*>(&r);
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i)
      asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(q[i].x), "=r"(q[i].y), "=r"(q[i].z), "=r"(q[i].w)
                   : "l"(reinterpret_cast<const uint4*>(p) + i));
  } else {
    r = load_raw<T, N>(p);
  }
  return r;
}

// What a thread holds of its row: ITER vectors of VEC elements, each in
// accesses of UNIT neighbouring elements (VEC where rows are aligned, 2 where
// only the width is even, else 1); access k of vector i starts at column
// (lane + (i VEC / UNIT + k) TPR) UNIT, so that a warp's accesses are next to
// each other.  Elements behind the row's end load as 0 and are not stored.
template <int VEC, int ITER, int UNIT>
struct Place {
  static constexpr int P = VEC / 2, N = VEC / UNIT;
  int rows_per_block, sub, col0, stride, width;
  __device__ __forceinline__ Place(int tpr, int width_) {
    sub = threadIdx.x / tpr;
    rows_per_block = blockDim.x / tpr;
    col0 = threadIdx.x % tpr * UNIT;
    stride = tpr * UNIT;
    width = width_;
  }
  __device__ __forceinline__ int col(int i, int k) const { return col0 + (i * N + k) * stride; }
  __device__ __forceinline__ bool on(int i, int k) const { return col(i, k) < width; }

  template <typename T>
  struct Row {  // as loaded
    Raw<T, UNIT> v[ITER][N];
  };
  template <typename T>
  __device__ __forceinline__ void load(const T* row, Row<T>& r) const {
#pragma unroll
    for (int i = 0; i < ITER; ++i)
#pragma unroll
      for (int k = 0; k < N; ++k) {
        r.v[i][k] = Raw<T, UNIT>{};
        if (row && on(i, k)) r.v[i][k] = load_once<T, UNIT>(row + col(i, k));
      }
  }
  template <typename T>
  __device__ __forceinline__ static void unpack_row(const Row<T>& r, int i, f32x2 (&v)[P]) {
    float f[VEC];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float u[UNIT];
      unpack(r.v[i][k], u);
#pragma unroll
      for (int j = 0; j < UNIT; ++j) f[k * UNIT + j] = u[j];
    }
#pragma unroll
    for (int c = 0; c < P; ++c) v[c] = pack2(f[2 * c], f[2 * c + 1]);
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, int i, const f32x2 (&v)[P]) const {
    float f[VEC];
#pragma unroll
    for (int c = 0; c < P; ++c) unpack2(v[c], f[2 * c], f[2 * c + 1]);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float u[UNIT];
#pragma unroll
      for (int j = 0; j < UNIT; ++j) u[j] = f[k * UNIT + j];
      if (on(i, k)) store_vec<T, UNIT>(row + col(i, k), u);
    }
  }
  // a weight's values, or 1 without it; `vec`: 16-byte aligned
  __device__ __forceinline__ void weight(const float* w, bool vec, int i, f32x2 (&v)[P]) const {
    if (!w) {
#pragma unroll
      for (int c = 0; c < P; ++c) v[c] = both(1.f);
      return;
    }
    float f[VEC];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float* q = w + col(i, k);
      const bool real = on(i, k);
      if (UNIT >= 4 && vec) {
#pragma unroll
        for (int j = 0; j < UNIT; j += 4) {
          float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
          if (real) t = __ldg(reinterpret_cast<const float4*>(q + j));
          f[k * UNIT + j] = t.x;
          f[(k * UNIT + j + 1) % VEC] = t.y;
          f[(k * UNIT + j + 2) % VEC] = t.z;
          f[(k * UNIT + j + 3) % VEC] = t.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < UNIT; ++j) f[k * UNIT + j] = real ? __ldg(q + j) : 0.f;
      }
    }
#pragma unroll
    for (int c = 0; c < P; ++c) v[c] = pack2(f[2 * c], f[2 * c + 1]);
  }
  // s[columns] += t u, in shared memory that no other thread touches
  __device__ __forceinline__ void add(float* s, int i, const f32x2 (&t)[P],
                                      const f32x2 (&u)[P]) const {
    if constexpr (UNIT >= 4) {
#pragma unroll
      for (int j = 0; j < VEC / 4; ++j) {
        if (!on(i, 0)) break;
        ulonglong2* q = reinterpret_cast<ulonglong2*>(s + col(i, 0)) + j;
        ulonglong2 v = *q;
        v.x = fma2(t[2 * j], u[2 * j], v.x);
        v.y = fma2(t[2 * j + 1], u[2 * j + 1], v.y);
        *q = v;
      }
    } else {
#pragma unroll
      for (int c = 0; c < P; ++c) {
        float lo, hi;
        unpack2(mul2(t[c], u[c]), lo, hi);
        if (UNIT == 2) {
          if (!on(i, c)) break;
          float2* q = reinterpret_cast<float2*>(s + col(i, c));
          const float2 v = *q;
          *q = make_float2(v.x + lo, v.y + hi);
        } else {
          if (on(i, 2 * c)) s[col(i, 2 * c)] += lo;
          if (on(i, 2 * c + 1)) s[col(i, 2 * c + 1)] += hi;
        }
      }
    }
  }
};

__device__ __forceinline__ int64_t strided(const NormArgs& a, int64_t row, int64_t stride) {
  if (a.heads == 1) return row * stride;
  const int64_t t = row / a.heads;
  return t * stride + (row - t * a.heads) * a.width;
}

__device__ __forceinline__ bool aligned16(const void* a, const void* b, const void* c) {
  return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) |
           reinterpret_cast<uintptr_t>(c)) & 15) == 0;
}

// GATE: 0 none, 1 behind the norm, 2 before it.
template <typename IO, typename RT, int VEC, int ITER, int UNIT, int GATE>
__global__ void __launch_bounds__(512) norm_fwd_kernel(NormArgs a, int tpr) {
  using At = Place<VEC, ITER, UNIT>;
  constexpr int P = At::P;
  __shared__ float4 s_sum[32];
  const At p(tpr, a.width);
  RowSum sum{tpr, 0, s_sum};
  const Gate act{a.act == kActNone, a.act == kActSilu};
  const int64_t rows = a.tokens * a.heads;
  const float inv_w = 1.f / (float)a.width;
  const bool wvec = aligned16(a.post_weight, a.scale, a.pre_weight);
  const IO* x = static_cast<const IO*>(a.x);
  const IO* gate = static_cast<const IO*>(a.gate);
  const RT* res = static_cast<const RT*>(a.residual);
  for (int64_t base = (int64_t)blockIdx.x * p.rows_per_block; base < rows;
       base += (int64_t)gridDim.x * p.rows_per_block) {
    const int64_t row = base + p.sub, at = row * a.width;
    const bool row_on = row < rows;
    typename At::template Row<IO> rx, rg;
    typename At::template Row<RT> rr;
    p.load(row_on ? x + strided(a, row, a.x_stride) : nullptr, rx);
    if constexpr (GATE != 0)
      p.load(row_on ? gate + strided(a, row, a.gate_stride) : nullptr, rg);
    p.load(row_on && res ? res + at : nullptr, rr);
    f32x2 h[ITER][P];
    float s[1];
    f32x2 acc = both(0.f);
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      p.unpack_row(rx, i, h[i]);
      if constexpr (GATE == 2) {
        f32x2 g[P];
        p.unpack_row(rg, i, g);
#pragma unroll
        for (int c = 0; c < P; ++c) h[i][c] = mul2(h[i][c], act.f(g[c]));
      }
#pragma unroll
      for (int c = 0; c < P; ++c) acc = fma2(h[i][c], h[i][c], acc);
    }
    float r1 = 1.f;
    if (a.post_weight) {
      s[0] = sum2(acc);
      sum(s);
      r1 = rsqrtf(s[0] * inv_w + a.eps);
    }
    acc = both(0.f);
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      f32x2 w[P], sc[P], r[P];
      p.weight(a.post_weight, wvec, i, w);
      p.weight(a.scale, wvec, i, sc);
      p.unpack_row(rr, i, r);
#pragma unroll
      for (int c = 0; c < P; ++c) h[i][c] = mul2(mul2(h[i][c], both(r1)), w[c]);
      if constexpr (GATE == 1) {
        f32x2 g[P];
        p.unpack_row(rg, i, g);
#pragma unroll
        for (int c = 0; c < P; ++c) h[i][c] = mul2(h[i][c], act.f(g[c]));
      }
#pragma unroll
      for (int c = 0; c < P; ++c) {
        h[i][c] = fma2(sc[c], h[i][c], r[c]);
        acc = fma2(h[i][c], h[i][c], acc);
      }
      if (row_on) p.store(static_cast<RT*>(a.out) + at, i, h[i]);
    }
    if (a.pre_weight) {
      s[0] = sum2(acc);
      sum(s);
      const float r2 = rsqrtf(s[0] * inv_w + a.eps);
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
          f32x2 w[P];
        p.weight(a.pre_weight, wvec, i, w);
#pragma unroll
        for (int c = 0; c < P; ++c) h[i][c] = mul2(mul2(h[i][c], both(r2)), w[c]);
        if (row_on) p.store(static_cast<IO*>(a.normed) + at, i, h[i]);
      }
    }
  }
}

// part[block * rows_per_block + sub][3][width]: the weights' gradients of one
// row place's rows; norm_weight_sum_kernel sums them in a fixed order.
template <typename IO, typename RT, int VEC, int ITER, int UNIT, int GATE>
__global__ void __launch_bounds__(512)
    norm_bwd_kernel(NormArgs a, int tpr, float* __restrict__ part) {
  using At = Place<VEC, ITER, UNIT>;
  constexpr int P = At::P;
  __shared__ float4 s_sum[32];
  extern __shared__ __align__(16) float s_cols[];  // [rows of the block][3][padded width]
  const At p(tpr, a.width);
  RowSum sum{tpr, 0, s_sum};
  const Gate act{a.act == kActNone, a.act == kActSilu};
  const int64_t rows = a.tokens * a.heads;
  const float inv_w = 1.f / (float)a.width;
  const bool wvec = aligned16(a.post_weight, a.scale, a.pre_weight);
  const int pitch = (a.width + 3) & ~3;
  float* c_post = s_cols + p.sub * 3 * pitch;
  float* c_scale = c_post + pitch;
  float* c_pre = c_scale + pitch;
#pragma unroll
  for (int i = 0; i < ITER; ++i)
#pragma unroll
    for (int e = 0; e < At::N; ++e)
      if (p.on(i, e))
#pragma unroll
        for (int j = 0; j < UNIT; ++j) {
          const int c = p.col(i, e) + j;
          c_post[c] = c_scale[c] = c_pre[c] = 0.f;
        }
  const IO* x = static_cast<const IO*>(a.x);
  const IO* gate = static_cast<const IO*>(a.gate);
  const RT* res = static_cast<const RT*>(a.residual);
  const RT* dout = static_cast<const RT*>(a.d_out);
  const IO* dnorm = static_cast<const IO*>(a.d_normed);
  const bool pre = a.pre_weight && dnorm;
  for (int64_t base = (int64_t)blockIdx.x * p.rows_per_block; base < rows;
       base += (int64_t)gridDim.x * p.rows_per_block) {
    const int64_t row = base + p.sub, at = row * a.width;
    const bool row_on = row < rows;
    typename At::template Row<IO> rx, rg, rn;
    typename At::template Row<RT> rr, ro;
    p.load(row_on ? x + strided(a, row, a.x_stride) : nullptr, rx);
    if constexpr (GATE != 0)
      p.load(row_on ? gate + strided(a, row, a.gate_stride) : nullptr, rg);
    p.load(row_on && pre ? dnorm + at : nullptr, rn);
    p.load(row_on && pre && res ? res + at : nullptr, rr);
    p.load(row_on && dout ? dout + at : nullptr, ro);
    // sg: sigmoid(gate); hat: x [act(gate)] r1; d: the gradient from out to x
    f32x2 sg[GATE ? ITER : 1][P], out[ITER][P], d[ITER][P];
    float r1 = 1.f;
    auto h_of = [&](int i, f32x2(&h)[P]) {
      p.unpack_row(rx, i, h);
      if constexpr (GATE == 2) {
        f32x2 g[P], f, fd;
        p.unpack_row(rg, i, g);
#pragma unroll
        for (int c = 0; c < P; ++c) {
          act.fd(g[c], sg[i][c], f, fd);
          h[c] = mul2(h[c], f);
        }
      }
    };
    if constexpr (GATE != 0)
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        f32x2 g[P];
        p.unpack_row(rg, i, g);
#pragma unroll
        for (int c = 0; c < P; ++c) sg[i][c] = act.none ? both(0.f) : sigmoid2(g[c]);
      }
    if (a.post_weight) {
      f32x2 acc = both(0.f);
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        f32x2 h[P];
        h_of(i, h);
#pragma unroll
        for (int c = 0; c < P; ++c) acc = fma2(h[c], h[c], acc);
      }
      float s[1] = {sum2(acc)};
      sum(s);
      // with eps 0 an absent row must not add 0 * inf
      r1 = row_on ? rsqrtf(s[0] * inv_w + a.eps) : 0.f;
    }
    float r2 = 0.f, m2 = 0.f;
    if (pre) {
      f32x2 acc1 = both(0.f), acc2 = both(0.f);
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        f32x2 w[P], sc[P], wn[P], h[P], n[P], r[P];
        p.weight(a.post_weight, wvec, i, w);
        p.weight(a.scale, wvec, i, sc);
        p.weight(a.pre_weight, wvec, i, wn);
        h_of(i, h);
        p.unpack_row(rn, i, n);
        p.unpack_row(rr, i, r);
        f32x2 g[P];
        if constexpr (GATE == 1) p.unpack_row(rg, i, g);
#pragma unroll
        for (int c = 0; c < P; ++c) {
          f32x2 q = mul2(mul2(h[c], both(r1)), w[c]);
          if constexpr (GATE == 1) {
            f32x2 f, fd;
            act.fd(g[c], sg[i][c], f, fd);
            q = mul2(q, f);
          }
          out[i][c] = fma2(sc[c], q, r[c]);
          acc1 = fma2(out[i][c], out[i][c], acc1);
          acc2 = fma2(mul2(n[c], wn[c]), out[i][c], acc2);
        }
      }
      float s[2] = {sum2(acc1), sum2(acc2)};
      sum(s);
      // d out += r2 (dn w - out r2 mean(dn w out r2))
      r2 = row_on ? rsqrtf(s[0] * inv_w + a.eps) : 0.f;
      m2 = -(s[1] * inv_w * r2 * r2);
    }
    f32x2 acc = both(0.f);
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      p.unpack_row(ro, i, d[i]);
      if (pre) {
        f32x2 wn[P], n[P], o2[P];
        p.weight(a.pre_weight, wvec, i, wn);
        p.unpack_row(rn, i, n);
#pragma unroll
        for (int c = 0; c < P; ++c) {
          d[i][c] = fma2(both(r2), fma2(out[i][c], both(m2), mul2(n[c], wn[c])), d[i][c]);
          o2[c] = mul2(out[i][c], both(r2));
        }
        p.add(c_pre, i, n, o2);
      }
      if (a.dres && row_on) p.store(static_cast<RT*>(a.dres) + at, i, d[i]);
      f32x2 w[P], sc[P], h[P], q[P], f[P], fd[P];
      p.weight(a.post_weight, wvec, i, w);
      p.weight(a.scale, wvec, i, sc);
      h_of(i, h);
      if constexpr (GATE == 1) {
        f32x2 g[P];
        p.unpack_row(rg, i, g);
#pragma unroll
        for (int c = 0; c < P; ++c) act.fd(g[c], sg[i][c], f[c], fd[c]);
      }
#pragma unroll
      for (int c = 0; c < P; ++c) {
        h[c] = mul2(h[c], both(r1));
        q[c] = mul2(h[c], w[c]);
        if constexpr (GATE == 1) {
          fd[c] = mul2(fd[c], q[c]);
          q[c] = mul2(q[c], f[c]);
        }
      }
      if (a.dscale) p.add(c_scale, i, d[i], q);
#pragma unroll
      for (int c = 0; c < P; ++c) {
        d[i][c] = mul2(d[i][c], sc[c]);
        if constexpr (GATE == 1) {
          fd[c] = mul2(fd[c], d[i][c]);
          d[i][c] = mul2(d[i][c], f[c]);
        }
      }
      if constexpr (GATE == 1)
        if (row_on) p.store(static_cast<IO*>(a.dgate) + at, i, fd);
      if (a.dpost) p.add(c_post, i, d[i], h);
#pragma unroll
      for (int c = 0; c < P; ++c) {
        d[i][c] = mul2(d[i][c], w[c]);
        acc = fma2(d[i][c], h[c], acc);
      }
    }
    float m1 = 0.f;
    if (a.post_weight) {
      float s[1] = {sum2(acc)};
      sum(s);
      m1 = -(s[0] * inv_w * r1);  // hat = h r1
    }
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      if (!row_on) continue;
      if (a.post_weight) {
        f32x2 h[P];
        h_of(i, h);
#pragma unroll
        for (int c = 0; c < P; ++c)
          d[i][c] = mul2(both(r1), fma2(h[c], both(m1), d[i][c]));
      }
      if constexpr (GATE == 2) {  // d is the gradient of h = x act(g)
        f32x2 g[P], xv[P], dg[P];
        p.unpack_row(rg, i, g);
        p.unpack_row(rx, i, xv);
#pragma unroll
        for (int c = 0; c < P; ++c) {
          f32x2 f, fd;
          act.fd(g[c], sg[i][c], f, fd);
          dg[c] = mul2(mul2(fd, xv[c]), d[i][c]);
          d[i][c] = mul2(d[i][c], f);
        }
        p.store(static_cast<IO*>(a.dgate) + at, i, dg);
      }
      p.store(static_cast<IO*>(a.dx) + at, i, d[i]);
    }
  }
  float* o = part + ((int64_t)blockIdx.x * p.rows_per_block + p.sub) * 3 * a.width;
#pragma unroll
  for (int i = 0; i < ITER; ++i)
#pragma unroll
    for (int e = 0; e < At::N; ++e)
      if (p.on(i, e))
#pragma unroll
        for (int j = 0; j < UNIT; ++j) {
          const int c = p.col(i, e) + j;
          if (a.dpost) o[c] = c_post[c];
          if (a.dscale) o[a.width + c] = c_scale[c];
          if (a.dpre) o[2 * a.width + c] = c_pre[c];
        }
}

// The backward for wide rows (every thread VEC columns, no gaps): two rows at a
// time, so that the weights' loads, the sums' barriers and the addresses serve
// both.  The rows arrive through two slots of shared memory, filled by
// asynchronous copies of 16 bytes: a thread copies just the elements that it
// will read (no barrier), the next pair while it works on this one, and reads
// them again wherever they are needed instead of holding them.  The weights
// are in shared memory, their gradients in registers.
constexpr int kPairRows = 2;

template <typename T, int VEC>
constexpr int kUnits = VEC * (int)sizeof(T) / 16;  // 16-byte units of a vector

template <typename T, int VEC>
__device__ __forceinline__ void send_vec(unsigned dst, int unit, const T* p) {
#pragma unroll
  for (int k = 0; k < kUnits<T, VEC>; ++k)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + k * unit),
                 "l"(reinterpret_cast<const uint4*>(p) + k)
                 : "memory");
}
template <typename T, int VEC>
__device__ __forceinline__ void take_vec(const unsigned char* s, int unit, bool on,
                                         f32x2 (&v)[kPairs<VEC>]) {
  Raw<T, VEC> raw{};
  if (on) {
    uint4* q = reinterpret_cast<uint4*>(&raw);
#pragma unroll
    for (int k = 0; k < kUnits<T, VEC>; ++k) q[k] = *reinterpret_cast<const uint4*>(s + k * unit);
  }
  unpack_pairs<T, VEC>(raw, v);
}
template <int VEC>
__device__ __forceinline__ void shared_weight(const float* s, f32x2 (&v)[kPairs<VEC>]) {
#pragma unroll
  for (int i = 0; i < VEC / 4; ++i) {
    const ulonglong2 t = reinterpret_cast<const ulonglong2*>(s)[i];
    v[2 * i] = t.x;
    v[2 * i + 1] = t.y;
  }
}

template <typename IO, typename RT, int VEC, int GATE, bool SILU>
__global__ void __launch_bounds__(512)
    norm_bwd_pair_kernel(NormArgs a, int slot_bytes, float* __restrict__ part) {
  constexpr int P = kPairs<VEC>, R = kPairRows;
  extern __shared__ __align__(16) unsigned char s_mem[];
  __shared__ float4 s_sum[32];
  RowSum sum{(int)blockDim.x, 0, s_sum};
  const int col = threadIdx.x * VEC, unit = blockDim.x * 16;
  const float inv_w = 1.f / (float)a.width;
  float* s_post = reinterpret_cast<float*>(s_mem + 2 * slot_bytes);
  float* s_scale = s_post + a.width;
  float* s_pre = s_scale + a.width;
  for (int i = threadIdx.x; i < a.width; i += blockDim.x) {
    s_post[i] = a.post_weight ? a.post_weight[i] : 1.f;
    s_scale[i] = a.scale ? a.scale[i] : 1.f;
    s_pre[i] = a.pre_weight ? a.pre_weight[i] : 1.f;
  }
  const bool pre = a.pre_weight && a.d_normed, res = pre && a.residual, dout = a.d_out;
  // units before each array in a slot's row
  constexpr int UX = kUnits<IO, VEC>, UR = kUnits<RT, VEC>;
  const int at_n = GATE ? 2 * UX : UX, at_r = at_n + (pre ? UX : 0), at_o = at_r + (res ? UR : 0),
            row_units = at_o + (dout ? UR : 0);
  const int64_t rows = a.tokens * a.heads, pairs = (rows + R - 1) / R;
  unsigned char* mine = s_mem + threadIdx.x * 16;
  const unsigned dst0 = (unsigned)__cvta_generic_to_shared(mine);
  // where the next pair to fetch lies; one step is the grid's pairs
  const int64_t step = (int64_t)gridDim.x * R;
  int64_t next = (int64_t)blockIdx.x * R, next_at = next * a.width + col;
  const int64_t step_at = step * a.width;
  const IO* next_x = static_cast<const IO*>(a.x) + next * a.x_stride + col;
  const IO* next_g = static_cast<const IO*>(a.gate) + next * a.gate_stride + col;
  const int64_t step_x = step * a.x_stride, step_g = step * a.gate_stride;
  auto fetch = [&](int slot) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (next + j < rows) {
        const unsigned dst = dst0 + slot * slot_bytes + j * row_units * unit;
        const int64_t at = next_at + j * a.width;
        const IO *px = next_x + j * a.x_stride, *pg = next_g + j * a.gate_stride;
        if (a.heads != 1) {
          px = static_cast<const IO*>(a.x) + strided(a, next + j, a.x_stride) + col;
          pg = static_cast<const IO*>(a.gate) + strided(a, next + j, a.gate_stride) + col;
        }
        send_vec<IO, VEC>(dst, unit, px);
        if (GATE) send_vec<IO, VEC>(dst + UX * unit, unit, pg);
        if (pre) send_vec<IO, VEC>(dst + at_n * unit, unit, static_cast<const IO*>(a.d_normed) + at);
        if (res) send_vec<RT, VEC>(dst + at_r * unit, unit, static_cast<const RT*>(a.residual) + at);
        if (dout) send_vec<RT, VEC>(dst + at_o * unit, unit, static_cast<const RT*>(a.d_out) + at);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    next += step;
    next_at += step_at;
    next_x += step_x;
    next_g += step_g;
  };
  f32x2 dpost[P], dscale[P], dpre[P];
#pragma unroll
  for (int c = 0; c < P; ++c) dpost[c] = dscale[c] = dpre[c] = both(0.f);
  int slot = 0;
  if (blockIdx.x < pairs) fetch(0);
  __syncthreads();
  for (int64_t pair = blockIdx.x; pair < pairs; pair += gridDim.x, slot ^= 1) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    // the other slot's last reads lie behind the last pair's barriers
    if (pair + gridDim.x < pairs) fetch(slot ^ 1);
    const int64_t at = pair * R * a.width + col;
    const unsigned char* from = mine + slot * slot_bytes;
    bool on[R];
    const unsigned char* src[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      on[j] = pair * R + j < rows;
      src[j] = from + j * row_units * unit;
    }
    // hat: x [act(gate)] r1; sg: sigmoid(gate); d: the gradient from out to x
    f32x2 hat[R][P], sg[GATE ? R : 1][P], out[R][P];
    float r1[R], r2[R], m[R], s2[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      f32x2 acc = both(0.f);
      take_vec<IO, VEC>(src[j], unit, on[j], hat[j]);
      if constexpr (GATE != 0) {
        f32x2 g[P];
        take_vec<IO, VEC>(src[j] + UX * unit, unit, on[j], g);
#pragma unroll
        for (int c = 0; c < P; ++c) {
          sg[j][c] = sigmoid2(g[c]);
          if (GATE == 2) hat[j][c] = mul2(hat[j][c], SILU ? mul2(sg[j][c], g[c]) : sg[j][c]);
        }
      }
#pragma unroll
      for (int c = 0; c < P; ++c) acc = fma2(hat[j][c], hat[j][c], acc);
      s2[j] = sum2(acc);
      r1[j] = 1.f;
    }
    if (a.post_weight) {
      sum(s2);
#pragma unroll
      for (int j = 0; j < R; ++j) {
        // with eps 0 an absent row must not add 0 * inf
        r1[j] = on[j] ? rsqrtf(s2[j] * inv_w + a.eps) : 0.f;
#pragma unroll
        for (int c = 0; c < P; ++c) hat[j][c] = mul2(hat[j][c], both(r1[j]));
      }
    }
    f32x2 w[P], sc[P];
    shared_weight<VEC>(s_post + col, w);
    shared_weight<VEC>(s_scale + col, sc);
    if (pre) {
      f32x2 wn[P];
      shared_weight<VEC>(s_pre + col, wn);
      float s4[2 * R];
#pragma unroll
      for (int j = 0; j < R; ++j) {
        f32x2 n[P], acc1 = both(0.f), acc2 = both(0.f);
        take_vec<IO, VEC>(src[j] + at_n * unit, unit, on[j], n);
        take_vec<RT, VEC>(src[j] + at_r * unit, unit, on[j] && res, out[j]);
        f32x2 g[P];
        if constexpr (GATE == 1 && SILU) take_vec<IO, VEC>(src[j] + UX * unit, unit, on[j], g);
#pragma unroll
        for (int c = 0; c < P; ++c) {
          f32x2 q = mul2(hat[j][c], w[c]);
          if constexpr (GATE == 1) q = mul2(q, SILU ? mul2(sg[j][c], g[c]) : sg[j][c]);
          out[j][c] = fma2(sc[c], q, out[j][c]);
          acc1 = fma2(out[j][c], out[j][c], acc1);
          acc2 = fma2(mul2(n[c], wn[c]), out[j][c], acc2);
        }
        s4[2 * j] = sum2(acc1);
        s4[2 * j + 1] = sum2(acc2);
      }
      sum(s4);
      // d out += r2 (dn w - out r2 mean(dn w out r2))
#pragma unroll
      for (int j = 0; j < R; ++j) {
        r2[j] = on[j] ? rsqrtf(s4[2 * j] * inv_w + a.eps) : 0.f;
        m[j] = -(s4[2 * j + 1] * inv_w * r2[j] * r2[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      f32x2 d[P], acc = both(0.f);
      take_vec<RT, VEC>(src[j] + at_o * unit, unit, on[j] && dout, d);
      if (pre) {
        f32x2 n[P], wn[P];
        take_vec<IO, VEC>(src[j] + at_n * unit, unit, on[j], n);
        shared_weight<VEC>(s_pre + col, wn);
#pragma unroll
        for (int c = 0; c < P; ++c) {
          d[c] = fma2(both(r2[j]), fma2(out[j][c], both(m[j]), mul2(n[c], wn[c])), d[c]);
          dpre[c] = fma2(n[c], mul2(out[j][c], both(r2[j])), dpre[c]);
        }
      }
      if (a.dres && on[j]) store_pairs<RT, VEC>(static_cast<RT*>(a.dres) + at + j * a.width, d);
      f32x2 g[P], dg[P];
      if constexpr (GATE == 1 && SILU) take_vec<IO, VEC>(src[j] + UX * unit, unit, on[j], g);
#pragma unroll
      for (int c = 0; c < P; ++c) {
        f32x2 q = mul2(hat[j][c], w[c]);
        if constexpr (GATE == 1) {
          const f32x2 s = sg[j][c], t = fma2(s, both(-1.f), both(1.f));
          const f32x2 f = SILU ? mul2(s, g[c]) : s;
          dg[c] = mul2(mul2(s, SILU ? fma2(g[c], t, both(1.f)) : t), q);  // act'(g) q
          q = mul2(q, f);
          dscale[c] = fma2(d[c], q, dscale[c]);
          d[c] = mul2(d[c], sc[c]);
          dg[c] = mul2(dg[c], d[c]);
          d[c] = mul2(d[c], f);
        } else {
          dscale[c] = fma2(d[c], q, dscale[c]);
          d[c] = mul2(d[c], sc[c]);
        }
        dpost[c] = fma2(d[c], hat[j][c], dpost[c]);
        d[c] = mul2(d[c], w[c]);
        acc = fma2(d[c], hat[j][c], acc);
        out[j][c] = d[c];
      }
      if constexpr (GATE == 1)
        if (on[j]) store_pairs<IO, VEC>(static_cast<IO*>(a.dgate) + at + j * a.width, dg);
      s2[j] = sum2(acc);
    }
    if (a.post_weight) sum(s2);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (!on[j]) continue;
      f32x2 (&d)[P] = out[j];
      if (a.post_weight) {
        const float mean = -(s2[j] * inv_w);
#pragma unroll
        for (int c = 0; c < P; ++c)
          d[c] = mul2(both(r1[j]), fma2(hat[j][c], both(mean), d[c]));
      }
      if constexpr (GATE == 2) {  // d is the gradient of h = x act(g)
        f32x2 g[P], xv[P], dg[P];
        take_vec<IO, VEC>(src[j], unit, true, xv);
        take_vec<IO, VEC>(src[j] + UX * unit, unit, true, g);
#pragma unroll
        for (int c = 0; c < P; ++c) {
          const f32x2 s = sg[j][c], t = fma2(s, both(-1.f), both(1.f));
          dg[c] = mul2(mul2(mul2(s, SILU ? fma2(g[c], t, both(1.f)) : t), xv[c]), d[c]);
          d[c] = mul2(d[c], SILU ? mul2(s, g[c]) : s);
        }
        store_pairs<IO, VEC>(static_cast<IO*>(a.dgate) + at + j * a.width, dg);
      }
      store_pairs<IO, VEC>(static_cast<IO*>(a.dx) + at + j * a.width, d);
    }
    // without a sum nothing else separates this slot's reads from its refill,
    // but they are this thread's own
  }
  float* o = part + (int64_t)blockIdx.x * 3 * a.width + col;
  if (a.dpost) store_pairs<float, VEC>(o, dpost);
  if (a.dscale) store_pairs<float, VEC>(o + a.width, dscale);
  if (a.dpre) store_pairs<float, VEC>(o + 2 * a.width, dpre);
}

__global__ void norm_weight_sum_kernel(const float* __restrict__ part, int slots, int width,
                                       float* dpost, float* dscale, float* dpre) {
  __shared__ float s[16][33];
  float* out = blockIdx.y == 0 ? dpost : blockIdx.y == 1 ? dscale : dpre;
  if (!out) return;
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (c < width)
    for (int b = threadIdx.y; b < slots; b += 16)
      v += part[((int64_t)b * 3 + blockIdx.y) * width + c];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && c < width) {
    for (int i = 1; i < 16; ++i) v += s[i][threadIdx.x];
    out[c] = v;
  }
}

// Threads per row and vectors per thread.  Up to 32 threads a row is part of a
// warp (the block holds several rows); above, the block is one row.
struct Shape {
  int tpr, block, iter;
};
// `iters`: the vectors a thread may hold, the wanted number first, smaller
// ones (for few rows: more threads a row) behind it, larger ones (for rows of
// more than 512 threads) last.
Shape row_shape(const NormArgs& a, int vec, const int* iters, int n) {
  const int nvec = (a.width + vec - 1) / vec;
  const int64_t rows = a.tokens * a.heads;
  auto at = [&](int iter) {
    Shape s{4, 0, iter};
    while (s.tpr < 512 && s.tpr * iter < nvec) s.tpr *= 2;
    s.block = s.tpr <= 32 ? 128 : s.tpr;
    return s;
  };
  Shape best = at(iters[0]);
  for (int k = 1; k < n; ++k) {
    const bool fits = best.tpr * best.iter >= nvec;
    if (fits && (rows * best.tpr >= 148 * 256 || iters[k] > best.iter)) continue;
    const Shape s = at(iters[k]);
    if (!fits || s.tpr * s.iter >= nvec) best = s;
  }
  return best;
}

// Resident blocks of a launch on the whole device.  Every device that this
// library serves is the same chip, so what the runtime said for a kernel is
// remembered for the thread's next calls.
template <typename K>
int resident_blocks(K kernel, int block, int sms, size_t shared) {
  struct Known {
    const void* kernel;
    int block, per;
    size_t shared;
  };
  static thread_local Known known[8];
  static thread_local int next = 0;
  const void* key = reinterpret_cast<const void*>(kernel);
  for (const Known& k : known)
    if (k.kernel == key && k.block == block && k.shared == shared) return k.per * sms;
  int per = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, block, shared) != cudaSuccess ||
      per < 1)
    return sms;
  known[next] = Known{key, block, per, shared};
  next = (next + 1) % 8;
  return per * sms;
}

template <typename IO, typename RT, int VEC, int ITER, int UNIT>
cudaError_t fwd_launch(const NormArgs& a, const Shape& s, cudaStream_t stream) {
  auto* k = !a.gate          ? norm_fwd_kernel<IO, RT, VEC, ITER, UNIT, 0>
            : !a.gate_first  ? norm_fwd_kernel<IO, RT, VEC, ITER, UNIT, 1>
                             : norm_fwd_kernel<IO, RT, VEC, ITER, UNIT, 2>;
  const int64_t need = (a.tokens * a.heads + s.block / s.tpr - 1) / (s.block / s.tpr);
  const int64_t most = resident_blocks(k, s.block, sm_count(), 0);
  k<<<(unsigned)(need < most ? need : most), s.block, 0, stream>>>(a, s.tpr);
  return cudaGetLastError();
}

// What these kernels may take: their sums have half a KB of static memory.
constexpr int kMostShared = kBlockShared - 1024;

// Shared memory of the backward for wide rows; 0 where it does not take them:
// rows of 64 to 512 whole vectors in whole warps, a gate with a sigmoid, and
// two slots that fit beside the weights.
struct PairShape {
  int threads, slot_bytes, bytes;
};
PairShape pair_shape(const NormArgs& a, int vec) {
  const int threads = a.width / vec, e = a.bf16 ? 2 : 4, r = a.res_bf16 ? 2 : 4;
  const bool pre = a.pre_weight && a.d_normed;
  if (vec == 1 || a.width % (32 * vec) || threads < 64 || threads > 512 ||
      (a.gate && a.act == kActNone))
    return PairShape{0, 0, 0};
  const int row = a.width * (e * (1 + (a.gate ? 1 : 0) + (pre ? 1 : 0)) +
                             r * ((pre && a.residual ? 1 : 0) + (a.d_out ? 1 : 0)));
  const PairShape s{threads, kPairRows * row, 2 * kPairRows * row + 12 * a.width};
  return s.bytes <= kMostShared ? s : PairShape{0, 0, 0};
}

// The most blocks of a backward launch: what its workspace holds parts for.
int64_t bwd_blocks(const NormArgs& a, const Shape& s, int sms) {
  const int per = s.block / s.tpr;
  const int64_t need = (a.tokens * a.heads + per - 1) / per, cap = (int64_t)sms * (1024 / s.block);
  return need < cap ? need : cap;
}

template <typename IO, typename RT, int VEC, int ITER, int UNIT>
cudaError_t bwd_launch(const NormArgs& a, const Shape& s, int sms, float* part,
                       cudaStream_t stream) {
  auto* k = !a.gate          ? norm_bwd_kernel<IO, RT, VEC, ITER, UNIT, 0>
            : !a.gate_first  ? norm_bwd_kernel<IO, RT, VEC, ITER, UNIT, 1>
                             : norm_bwd_kernel<IO, RT, VEC, ITER, UNIT, 2>;
  const int per = s.block / s.tpr;
  const int bytes = per * 3 * ((a.width + 3) & ~3) * (int)sizeof(float);
  cudaError_t e = cudaSuccess;
  if (bytes > 47 * 1024) e = allow_shared(k, kMostShared);  // the static part comes on top
  if (e != cudaSuccess) return e;
  int64_t blocks = resident_blocks(k, s.block, sms, bytes);
  const int64_t most = bwd_blocks(a, s, sms);
  blocks = blocks < most ? blocks : most;
  if (blocks > 0) k<<<(unsigned)blocks, s.block, bytes, stream>>>(a, s.tpr, part);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (a.dpost || a.dscale || a.dpre)
    norm_weight_sum_kernel<<<dim3((a.width + 31) / 32, 3), dim3(32, 16), 0, stream>>>(
        part, (int)(blocks * per), a.width, a.dpost, a.dscale, a.dpre);
  return cudaGetLastError();
}

template <typename IO, typename RT, int VEC>
cudaError_t pair_launch(const NormArgs& a, const PairShape& s, int sms, float* part,
                        cudaStream_t stream) {
  const bool silu = a.act == kActSilu;
  auto* k = !a.gate ? norm_bwd_pair_kernel<IO, RT, VEC, 0, false>
            : a.gate_first ? (silu ? norm_bwd_pair_kernel<IO, RT, VEC, 2, true>
                                   : norm_bwd_pair_kernel<IO, RT, VEC, 2, false>)
                           : (silu ? norm_bwd_pair_kernel<IO, RT, VEC, 1, true>
                                   : norm_bwd_pair_kernel<IO, RT, VEC, 1, false>);
  cudaError_t e = allow_shared(k, kMostShared);
  if (e != cudaSuccess) return e;
  const int64_t need = (a.tokens * a.heads + kPairRows - 1) / kPairRows;
  int64_t blocks = resident_blocks(k, s.threads, sms, s.bytes);
  const int64_t cap = (int64_t)sms * (1024 / s.threads);
  blocks = blocks < need ? blocks : need;
  blocks = blocks < cap ? blocks : cap;
  if (blocks > 0) k<<<(unsigned)blocks, s.threads, s.bytes, stream>>>(a, s.slot_bytes, part);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (a.dpost || a.dscale || a.dpre)
    norm_weight_sum_kernel<<<dim3((a.width + 31) / 32, 3), dim3(32, 16), 0, stream>>>(
        part, (int)blocks, a.width, a.dpost, a.dscale, a.dpre);
  return cudaGetLastError();
}

constexpr int kFwd8[] = {2, 1, 4}, kFwd4[] = {4, 1, 8}, kBwd8[] = {2, 1, 4}, kBwd4[] = {2, 1, 4, 8};
// rows that are not aligned: 16 elements a thread as far as 512 threads go,
// forward also one vector a thread for few rows
constexpr int kOddFwd8[] = {2, 1, 4}, kOddFwd4[] = {4, 1, 8}, kOdd8[] = {2, 4}, kOdd4[] = {4, 8};

// Neighbouring elements an access can take: 16 bytes of io where every
// pointer, stride and the width allow it, 2 elements where they allow that.
int unit_of(const NormArgs& a) {
  const int vec = a.bf16 ? 8 : 4;
  const void* io[] = {a.x, a.gate, a.normed, a.d_normed, a.dx, a.dgate};
  const void* res[] = {a.residual, a.out, a.d_out, a.dres};
  for (const int u : {vec, 2}) {
    const size_t e = a.bf16 ? 2 : 4, r = a.res_bf16 ? 2 : 4;
    bool ok = a.width % u == 0 && a.x_stride % u == 0 && a.gate_stride % u == 0;
    for (const void* p : io) ok = ok && aligned_to(p, u * e);
    for (const void* p : res) ok = ok && aligned_to(p, u * r > 16 ? 16 : u * r);
    if (ok) return u;
  }
  return 1;
}

Shape shape_of(const NormArgs& a, bool bwd, int unit) {
  if (a.bf16)
    return unit < 8 ? bwd ? row_shape(a, 8, kOdd8, 2) : row_shape(a, 8, kOddFwd8, 3)
                    : bwd ? row_shape(a, 8, kBwd8, 3) : row_shape(a, 8, kFwd8, 3);
  return unit < 4 ? bwd ? row_shape(a, 4, kOdd4, 2) : row_shape(a, 4, kOddFwd4, 3)
                  : bwd ? row_shape(a, 4, kBwd4, 4) : row_shape(a, 4, kFwd4, 3);
}

template <typename IO, typename RT, int VEC, int UNIT>
cudaError_t fwd_pick(const NormArgs& a, cudaStream_t st) {
  const Shape s = shape_of(a, false, UNIT);
  if (s.iter == 1) return fwd_launch<IO, RT, VEC, 1, UNIT>(a, s, st);
  if constexpr (VEC == 8)
    if (s.iter == 2) return fwd_launch<IO, RT, VEC, 2, UNIT>(a, s, st);
  if (s.iter == 4) return fwd_launch<IO, RT, VEC, 4, UNIT>(a, s, st);
  if constexpr (VEC == 4)
    if (s.iter == 8) return fwd_launch<IO, RT, VEC, 8, UNIT>(a, s, st);
  return cudaErrorInvalidValue;
}
template <typename IO, typename RT, int VEC>
cudaError_t fwd_unit(const NormArgs& a, cudaStream_t st) {
  const int u = unit_of(a);
  return u == VEC ? fwd_pick<IO, RT, VEC, VEC>(a, st)
         : u == 2 ? fwd_pick<IO, RT, VEC, 2>(a, st)
                  : fwd_pick<IO, RT, VEC, 1>(a, st);
}

template <typename IO, typename RT, int VEC, int UNIT>
cudaError_t bwd_pick(const NormArgs& a, int sms, float* part, cudaStream_t st) {
  const Shape s = shape_of(a, true, UNIT);
  if constexpr (UNIT == VEC)
    if (s.iter == 1) return bwd_launch<IO, RT, VEC, 1, UNIT>(a, s, sms, part, st);
  if constexpr (UNIT == VEC || VEC == 8)
    if (s.iter == 2) return bwd_launch<IO, RT, VEC, 2, UNIT>(a, s, sms, part, st);
  if (s.iter == 4) return bwd_launch<IO, RT, VEC, 4, UNIT>(a, s, sms, part, st);
  if constexpr (VEC == 4)
    if (s.iter == 8) return bwd_launch<IO, RT, VEC, 8, UNIT>(a, s, sms, part, st);
  return cudaErrorInvalidValue;
}
template <typename IO, typename RT, int VEC>
cudaError_t bwd_unit(const NormArgs& a, int sms, float* part, cudaStream_t st) {
  const int u = unit_of(a);
  if (const PairShape q = pair_shape(a, u == VEC ? VEC : 1); q.threads)
    return pair_launch<IO, RT, VEC>(a, q, sms, part, st);
  return u == VEC ? bwd_pick<IO, RT, VEC, VEC>(a, sms, part, st)
         : u == 2 ? bwd_pick<IO, RT, VEC, 2>(a, sms, part, st)
                  : bwd_pick<IO, RT, VEC, 1>(a, sms, part, st);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t st) {
  if (a.tokens == 0) return cudaSuccess;
  using bf = __nv_bfloat16;
  return a.bf16 && a.res_bf16 ? fwd_unit<bf, bf, 8>(a, st)
         : a.bf16             ? fwd_unit<bf, float, 8>(a, st)
                              : fwd_unit<float, float, 4>(a, st);
}

size_t norm_bwd_workspace_bytes(const NormArgs& a, int sms) {
  if (!a.dpost && !a.dscale && !a.dpre) return 0;
  const int vec = a.bf16 ? 8 : 4, unit = unit_of(a);
  if (const PairShape q = pair_shape(a, unit == vec ? vec : 1); q.threads) {
    const int64_t need = (a.tokens * a.heads + kPairRows - 1) / kPairRows,
                  cap = (int64_t)sms * (1024 / q.threads);
    return (size_t)(need < cap ? need : cap) * 3 * a.width * sizeof(float);
  }
  const Shape s = shape_of(a, true, unit);
  return (size_t)bwd_blocks(a, s, sms) * (s.block / s.tpr) * 3 * a.width * sizeof(float);
}

cudaError_t launch_norm_bwd(const NormArgs& a, void* ws, int sms, cudaStream_t st) {
  using bf = __nv_bfloat16;
  float* part = static_cast<float*>(ws);
  return a.bf16 && a.res_bf16 ? bwd_unit<bf, bf, 8>(a, sms, part, st)
         : a.bf16             ? bwd_unit<bf, float, 8>(a, sms, part, st)
                              : bwd_unit<float, float, 4>(a, sms, part, st);
}

}  // namespace kda

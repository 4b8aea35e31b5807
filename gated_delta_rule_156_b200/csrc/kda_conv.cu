// Short causal convolution: forward, backward and the step for new tokens.
//
//   pre_t = bias + sum_j w_j x_{t-(W-1)+j},   out_t = act(pre_t)
// per channel, with x at the W - 1 places before a sequence taken from its
// initial state.  W is 2, 3 or 4, so an element costs 2 W flops and an
// activation against 2 * sizeof(io) bytes: the kernels are bound by HBM.
//
// Work split: a thread owns VEC neighbouring channels and a run of consecutive
// tokens, over which the last W - 1 inputs stay in registers.  The run's first
// W - 1 inputs are read by the run before it as well; those reads come out of
// L2.  Measured for bf16, in shares of a copy's rate: 2 x 8192 x 4096 forward
// 55 us (76 %), 8200 x 4096 packed backward 70 us (45 %, bound by the latency
// of the sigmoid's chain), 256 x 12288 step 11.6 us (67 %).
#include "kda_layer.cuh"

namespace kda {

namespace {

// Tokens on their way: a ring of kStages groups of kGroup tokens in shared
// memory, filled by asynchronous copies.  A thread copies just what it will
// read itself (no barrier; the copies are statements that the compiler moves no
// read across), and three groups in flight cost it no registers
// (2 x 8192 x 4096 forward: 55 us, 63 with the next group in registers).
// Vectors of 4 elements; single elements are loaded 8 tokens at a time.
constexpr int kGroup = 4, kStages = 4;
template <typename IO, int VEC>
struct Ring {
  static constexpr int BYTES = VEC * (int)sizeof(IO);
  static constexpr bool ON = BYTES >= 8;
  unsigned char* at;  // this thread's first vector
  int step;           // to its next one
  __device__ __forceinline__ Ring(unsigned char* base, int tid, int threads)
      : at(base + tid * BYTES), step(threads * BYTES) {}
  // vector i of a group of `arrays` * kGroup vectors
  __device__ __forceinline__ unsigned char* place(int stage, int n, int i) const {
    return at + (stage * n + i) * step;
  }
  __device__ __forceinline__ static void send(unsigned char* to, const IO* from) {
    const unsigned dst = (unsigned)__cvta_generic_to_shared(to);
    if constexpr (BYTES == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(from) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(from) : "memory");
  }
  __device__ __forceinline__ static void commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ static void wait() {  // for the oldest group in flight
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
  }
  __device__ __forceinline__ static Raw<IO, VEC> take(const unsigned char* from) {
    return *reinterpret_cast<const Raw<IO, VEC>*>(from);
  }
};

// A thread's channels go in pairs through the packed fp32 arithmetic.
template <typename IO, int W, int VEC>
struct Taps {
  static constexpr int P = kPairs<VEC>;
  f32x2 w[W][P], b[P];
  __device__ __forceinline__ void load(const ConvArgs& a, int c0) {
    float t[2 * P][W];
    const float* p = a.weight + (size_t)c0 * W;
    if (W == 4 && (reinterpret_cast<uintptr_t>(a.weight) & 15) == 0) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {  // a channel's taps are 16 bytes
        const float4 v = reinterpret_cast<const float4*>(p)[i];
        t[i][0] = v.x;
        t[i][1] = v.y;
        t[i][2 % W] = v.z;
        t[i][W - 1] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) t[i][j] = p[i * W + j];
    }
    if (VEC == 1)
#pragma unroll
      for (int j = 0; j < W; ++j) t[2 * P - 1][j] = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][i] = pack2(t[2 * i][j], t[2 * i + 1][j]);
      b[i] = a.bias ? pack2(a.bias[c0 + 2 * i], VEC > 1 ? a.bias[c0 + 2 * i + 1] : 0.f) : both(0.f);
    }
  }
};

// Input at position t of a sequence (t >= start - (W-1)): x, or the past.
template <typename IO, int W, int VEC>
__device__ __forceinline__ void input_at(const ConvArgs& a, const SeqCursor& q, int t, int c0,
                                         f32x2 (&v)[kPairs<VEC>]) {
  if (t >= q.start) {
    load_pairs<IO, VEC>(static_cast<const IO*>(a.x) + (int64_t)t * a.x_stride + c0, v);
  } else if (a.past) {
    const int64_t row = (int64_t)q.s * (W - 1) + (t - q.start + W - 1);
    load_pairs<IO, VEC>(static_cast<const IO*>(a.past) + row * a.D + c0, v);
  } else {
#pragma unroll
    for (int i = 0; i < kPairs<VEC>; ++i) v[i] = both(0.f);
  }
}

__device__ __forceinline__ f32x2 act2(f32x2 x, int act) {
  return act == kActSilu ? mul2(x, sigmoid2(x)) : x;
}
// d act(x) / dx: s (1 + x (1 - s)) for SiLU
__device__ __forceinline__ f32x2 act_grad2(f32x2 x, int act) {
  if (act != kActSilu) return both(1.f);
  const f32x2 s = sigmoid2(x);
  return mul2(s, fma2(x, fma2(s, both(-1.f), both(1.f)), both(1.f)));
}

template <typename IO, int W, int VEC, int P>
__device__ __forceinline__ void taps_dot(const Taps<IO, W, VEC>& k, const f32x2 (&win)[W - 1][P],
                                         const f32x2 (&x)[P], f32x2 (&pre)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    f32x2 p = k.b[i];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) p = fma2(k.w[j][i], win[j][i], p);
    pre[i] = fma2(k.w[W - 1][i], x[i], p);
  }
}

template <int W, int P>
__device__ __forceinline__ void slide(f32x2 (&win)[W - 1][P], const f32x2 (&x)[P]) {
#pragma unroll
  for (int j = 0; j + 1 < W - 1; ++j)
#pragma unroll
    for (int i = 0; i < P; ++i) win[j][i] = win[j + 1][i];
#pragma unroll
  for (int i = 0; i < P; ++i) win[W - 2][i] = x[i];
}

// Block (channel vectors, runs); the grid's runs go over all tokens, then
// over the n_seqs * (W - 1) rows of the final states.
template <typename IO, int W, int VEC>
__global__ void __launch_bounds__(256, 4)
    conv_fwd_kernel(ConvArgs a, int nvec, int run, int64_t n_runs) {
  constexpr int P = kPairs<VEC>;
  using R = Ring<IO, VEC>;
  extern __shared__ __align__(16) unsigned char s_ring[];
  const R ring(s_ring, threadIdx.y * blockDim.x + threadIdx.x, 256);
  const int cv = blockIdx.y * blockDim.x + threadIdx.x;
  int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (cv >= nvec) return;
  const int c0 = cv * VEC;
  if (r >= n_runs) {  // final state row
    r -= n_runs;
    if (!a.final_state || r >= (int64_t)a.n_seqs * (W - 1)) return;
    SeqCursor q;
    q.s = (int)(r / (W - 1));
    seq_range(a.cu, q.s, a.T, &q.start, &q.end);
    f32x2 v[P];
    input_at<IO, W, VEC>(a, q, q.end - (W - 1) + (int)(r % (W - 1)), c0, v);
    store_pairs<IO, VEC>(static_cast<IO*>(a.final_state) + r * a.D + c0, v);
    return;
  }
  Taps<IO, W, VEC> k;
  k.load(a, c0);
  const IO* x = static_cast<const IO*>(a.x) + c0;
  IO* out = static_cast<IO*>(a.out) + c0;
  int64_t t = r * run;
  const int64_t t1 = min(t + run, a.tokens);
  while (t < t1) {
    SeqCursor q;
    if (!find_seq(a.cu, a.n_seqs, a.T, (int)t, &q)) return;
    if (t < q.start) t = q.start;
    const int64_t e = min((int64_t)q.end, t1);
    if (t >= e) break;
    f32x2 win[W - 1][P];
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      input_at<IO, W, VEC>(a, q, (int)t - (W - 1) + j, c0, win[j]);
    const IO* px = x + t * a.x_stride;
    IO* po = out + t * a.D;
    auto token = [&](const Raw<IO, VEC>& raw) {
      f32x2 v[P], pre[P];
      unpack_pairs<IO, VEC>(raw, v);
      taps_dot<IO, W, VEC>(k, win, v, pre);
#pragma unroll
      for (int i = 0; i < P; ++i) pre[i] = act2(pre[i], a.act);
      store_pairs<IO, VEC>(po, pre);
      slide<W>(win, v);
      po += a.D;
    };
    int left = (int)(e - t);
    if constexpr (R::ON) {
      const int groups = left / kGroup;
      auto fetch = [&](int n) {
        if (n < groups)
#pragma unroll
          for (int i = 0; i < kGroup; ++i)
            R::send(ring.place(n % kStages, kGroup, i), px + (n * kGroup + i) * a.x_stride);
        R::commit();
      };
#pragma unroll
      for (int n = 0; n < kStages - 1; ++n) fetch(n);
      for (int n = 0; n < groups; ++n) {
        R::wait();
        fetch(n + kStages - 1);
#pragma unroll
        for (int i = 0; i < kGroup; ++i) token(R::take(ring.place(n % kStages, kGroup, i)));
      }
      px += groups * kGroup * a.x_stride;
      left -= groups * kGroup;
    } else {
      for (; left >= 2 * kGroup; left -= 2 * kGroup) {
        Raw<IO, VEC> raw[2 * kGroup];
#pragma unroll
        for (int i = 0; i < 2 * kGroup; ++i) raw[i] = load_raw<IO, VEC>(px + i * a.x_stride);
        px += 2 * kGroup * a.x_stride;
#pragma unroll
        for (int i = 0; i < 2 * kGroup; ++i) token(raw[i]);
      }
    }
    for (; left > 0; --left) {
      token(load_raw<IO, VEC>(px));
      px += a.x_stride;
    }
    t = e;
  }
}

// Gradients.  dpre_t = d_out_t act'(pre_t) reaches dx at the W places
// t-(W-1) .. t; the thread walks its run and W - 1 tokens further, carrying
// the W - 1 unfinished dx in registers, and sums dw_j += dpre_t x_{t-(W-1)+j}
// and db over the run itself.  The block's runs are summed in shared memory
// in a fixed order; conv_weight_sum_kernel sums the blocks.  The rows of
// d_initial_state are independent of the runs and have threads of their own.
constexpr int kBwdLanes = 32, kBwdRuns = 8;

template <typename IO, int W, int VEC>
__device__ void past_grad(const ConvArgs& a, const Taps<IO, W, VEC>& k, int64_t row,
                          int c0) {
  SeqCursor q;
  q.s = (int)(row / (W - 1));
  const int r = (int)(row % (W - 1));
  seq_range(a.cu, q.s, a.T, &q.start, &q.end);
  const int len = q.end - q.start;
  constexpr int P = kPairs<VEC>;
  f32x2 g[P];
#pragma unroll
  for (int i = 0; i < P; ++i) g[i] = both(0.f);
  // row r of the past is input r-(W-1); token tau <= r reads it with tap r-tau
  for (int tau = 0; tau <= r && tau < len; ++tau) {
    f32x2 win[W - 1][P], x[P], pre[P], dy[P];
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      input_at<IO, W, VEC>(a, q, q.start + tau - (W - 1) + j, c0, win[j]);
    input_at<IO, W, VEC>(a, q, q.start + tau, c0, x);
    taps_dot<IO, W, VEC>(k, win, x, pre);
    load_pairs<IO, VEC>(static_cast<const IO*>(a.d_out) + (int64_t)(q.start + tau) * a.D + c0,
                        dy);
#pragma unroll
    for (int j = 0; j < W; ++j)
      if (j == r - tau)
#pragma unroll
        for (int i = 0; i < P; ++i)
          g[i] = fma2(k.w[j][i], mul2(dy[i], act_grad2(pre[i], a.act)), g[i]);
  }
  if (a.d_final && r >= len) {  // a short sequence keeps this row
    f32x2 v[P];
    load_pairs<IO, VEC>(static_cast<const IO*>(a.d_final) + (row - len) * a.D + c0, v);
#pragma unroll
    for (int i = 0; i < P; ++i) g[i] = add2(g[i], v[i]);
  }
  store_pairs<IO, VEC>(static_cast<IO*>(a.d_past) + row * a.D + c0, g);
}

template <typename IO, int W, int VEC>
__global__ void __launch_bounds__(kBwdLanes* kBwdRuns, 2)
    conv_bwd_kernel(ConvArgs a, int nvec, int run, int64_t n_blocks,
                    float* __restrict__ part) {
  __shared__ float s_part[kBwdRuns][W + 1][kBwdLanes][VEC];
  using R = Ring<IO, VEC>;
  extern __shared__ __align__(16) unsigned char s_ring[];
  const R ring(s_ring, threadIdx.y * kBwdLanes + threadIdx.x, kBwdLanes * kBwdRuns);
  const int cv = blockIdx.y * kBwdLanes + threadIdx.x;
  const bool on = cv < nvec;
  const int c0 = on ? cv * VEC : 0;
  Taps<IO, W, VEC> k;
  k.load(a, c0);
  if ((int64_t)blockIdx.x >= n_blocks) {  // rows of d_initial_state
    const int64_t row = ((int64_t)blockIdx.x - n_blocks) * kBwdRuns + threadIdx.y;
    if (on && row < (int64_t)a.n_seqs * (W - 1)) past_grad<IO, W, VEC>(a, k, row, c0);
    return;
  }
  constexpr int P = kPairs<VEC>;
  f32x2 dw[W][P], db[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    db[i] = both(0.f);
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][i] = both(0.f);
  }
  const IO* x = static_cast<const IO*>(a.x) + c0;
  const IO* dy = static_cast<const IO*>(a.d_out) + c0;
  IO* dx = static_cast<IO*>(a.dx) + c0;
  int64_t t = ((int64_t)blockIdx.x * kBwdRuns + threadIdx.y) * run;
  const int64_t t1 = on ? min(t + run, a.tokens) : t;
  while (t < t1) {
    SeqCursor q;
    if (!find_seq(a.cu, a.n_seqs, a.T, (int)t, &q)) break;
    if (t < q.start) t = q.start;
    const int64_t e = min((int64_t)q.end, t1);
    if (t >= e) break;
    const int64_t stop = min((int64_t)q.end, e + W - 1);
    f32x2 win[W - 1][P], g[W - 1][P];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      input_at<IO, W, VEC>(a, q, (int)t - (W - 1) + j, c0, win[j]);
#pragma unroll
      for (int i = 0; i < P; ++i) g[j][i] = both(0.f);
    }
    const IO* px = x + t * a.x_stride;
    const IO* py = dy + t * a.D;
    IO* po = dx + (t - (W - 1)) * a.D;
    int skip = W - 1;  // places before the run, finished by others
    auto token = [&](const Raw<IO, VEC>& rx, const Raw<IO, VEC>& ry, bool mine) {
      f32x2 xv[P], dp[P], pre[P], done[P];
      unpack_pairs<IO, VEC>(rx, xv);
      unpack_pairs<IO, VEC>(ry, dp);
      taps_dot<IO, W, VEC>(k, win, xv, pre);
#pragma unroll
      for (int c = 0; c < P; ++c) {
        dp[c] = mul2(dp[c], act_grad2(pre[c], a.act));
        if (mine) {
          db[c] = add2(db[c], dp[c]);
#pragma unroll
          for (int j = 0; j < W - 1; ++j) dw[j][c] = fma2(dp[c], win[j][c], dw[j][c]);
          dw[W - 1][c] = fma2(dp[c], xv[c], dw[W - 1][c]);
        }
        done[c] = fma2(k.w[0][c], dp[c], g[0][c]);
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) g[j][c] = fma2(k.w[j + 1][c], dp[c], g[j + 1][c]);
        g[W - 2][c] = mul2(k.w[W - 1][c], dp[c]);
      }
      if (skip > 0)
        --skip;
      else
        store_pairs<IO, VEC>(po, done);
      po += a.D;
      slide<W>(win, xv);
    };
    int left = (int)(e - t);
    if constexpr (R::ON) {
      const int groups = left / kGroup;
      auto fetch = [&](int n) {
        if (n < groups)
#pragma unroll
          for (int i = 0; i < kGroup; ++i) {
            R::send(ring.place(n % kStages, 2 * kGroup, i), px + (n * kGroup + i) * a.x_stride);
            R::send(ring.place(n % kStages, 2 * kGroup, kGroup + i),
                    py + (n * kGroup + i) * (int64_t)a.D);
          }
        R::commit();
      };
#pragma unroll
      for (int n = 0; n < kStages - 1; ++n) fetch(n);
      for (int n = 0; n < groups; ++n) {
        R::wait();
        fetch(n + kStages - 1);
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
          token(R::take(ring.place(n % kStages, 2 * kGroup, i)),
                R::take(ring.place(n % kStages, 2 * kGroup, kGroup + i)), true);
      }
      px += groups * kGroup * a.x_stride;
      py += groups * kGroup * (int64_t)a.D;
      left -= groups * kGroup;
    } else {
      for (; left >= 2 * kGroup; left -= 2 * kGroup) {
        Raw<IO, VEC> rx[2 * kGroup], ry[2 * kGroup];
#pragma unroll
        for (int i = 0; i < 2 * kGroup; ++i) {
          rx[i] = load_raw<IO, VEC>(px + i * a.x_stride);
          ry[i] = load_raw<IO, VEC>(py + i * (int64_t)a.D);
        }
        px += 2 * kGroup * a.x_stride;
        py += 2 * kGroup * (int64_t)a.D;
#pragma unroll
        for (int i = 0; i < 2 * kGroup; ++i) token(rx[i], ry[i], true);
      }
    }
    for (int i = left + (int)(stop - e); i > 0; --i) {
      token(load_raw<IO, VEC>(px), load_raw<IO, VEC>(py), left-- > 0);
      px += a.x_stride;
      py += a.D;
    }
    if (stop == q.end) {  // the sequence's last W - 1 places
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        const int64_t at = stop - (W - 1) + j;
        if (at >= t && at < e) {
          if (a.d_final) {
            f32x2 v[P];
            load_pairs<IO, VEC>(static_cast<const IO*>(a.d_final) +
                                    ((int64_t)q.s * (W - 1) + j) * a.D + c0, v);
#pragma unroll
            for (int i = 0; i < P; ++i) g[j][i] = add2(g[j][i], v[i]);
          }
          store_pairs<IO, VEC>(dx + at * a.D, g[j]);
        }
      }
    }
    t = e;
  }
#pragma unroll
  for (int j = 0; j <= W; ++j)
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float lo, hi;
      unpack2(j < W ? dw[j % W][i] : db[i], lo, hi);
      s_part[threadIdx.y][j][threadIdx.x][2 * i] = lo;
      if (VEC > 1) s_part[threadIdx.y][j][threadIdx.x][(2 * i + 1) % VEC] = hi;
    }
  __syncthreads();
  // part[block][tap or bias][channel]
  const int tid = threadIdx.y * kBwdLanes + threadIdx.x;
  for (int o = tid; o < (W + 1) * kBwdLanes * VEC; o += kBwdLanes * kBwdRuns) {
    const int j = o / (kBwdLanes * VEC), c = o % (kBwdLanes * VEC);
    const int ch = blockIdx.y * kBwdLanes * VEC + c;
    if (ch >= a.D) continue;
    float s = 0.f;
#pragma unroll
    for (int rr = 0; rr < kBwdRuns; ++rr) s += s_part[rr][j][c / VEC][c % VEC];
    part[((int64_t)blockIdx.x * (W + 1) + j) * a.D + ch] = s;
  }
}

// dw[c][j] and db[c]: the blocks' parts summed in a fixed order.
__global__ void conv_weight_sum_kernel(const float* __restrict__ part, int64_t n_blocks, int W,
                                       int D, float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float s[8][32];
  const int c = blockIdx.x * 32 + threadIdx.x, j = blockIdx.y;
  float v = 0.f;
  if (c < D)
    for (int64_t b = threadIdx.y; b < n_blocks; b += 8) v += part[(b * (W + 1) + j) * D + c];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && c < D) {
    for (int i = 1; i < 8; ++i) v += s[i][threadIdx.x];
    if (j < W)
      dw[(int64_t)c * W + j] = v;
    else if (db)
      db[c] = v;
  }
}

// T new tokens, state in place.  A thread owns VEC channels of NS sequences,
// whose loads it issues together; the taps are read once for all of them.
template <typename IO, int W, int VEC, int NS>
__global__ void __launch_bounds__(256) conv_step_kernel(ConvArgs a, int nvec) {
  const int cv = blockIdx.y * blockDim.x + threadIdx.x;
  const int64_t n0 = ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * NS;
  if (cv >= nvec || n0 >= a.n_seqs) return;
  constexpr int P = kPairs<VEC>;
  const int c0 = cv * VEC;
  const int64_t row = (int64_t)(W - 1) * a.D, xs = (int64_t)a.T * a.x_stride;
  IO* st = static_cast<IO*>(a.final_state) + n0 * row + c0;
  const IO* x = static_cast<const IO*>(a.x) + n0 * xs + c0;
  IO* out = static_cast<IO*>(a.out) + n0 * a.T * a.D + c0;
  Raw<IO, VEC> keep[NS][W - 1], rx[NS];
#pragma unroll
  for (int k = 0; k < NS; ++k)
    if (n0 + k < a.n_seqs) {
      rx[k] = load_raw<IO, VEC>(x + k * xs);
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        keep[k][j] = load_raw<IO, VEC>(st + k * row + (int64_t)j * a.D);
    }
  Taps<IO, W, VEC> taps;
  taps.load(a, c0);
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    if (n0 + k >= a.n_seqs) return;
    f32x2 win[W - 1][P];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) unpack_pairs<IO, VEC>(keep[k][j], win[j]);
    for (int t = 0; t < a.T; ++t) {
      f32x2 v[P], pre[P];
      unpack_pairs<IO, VEC>(rx[k], v);
      if (t + 1 < a.T) rx[k] = load_raw<IO, VEC>(x + k * xs + (int64_t)(t + 1) * a.x_stride);
      taps_dot<IO, W, VEC>(taps, win, v, pre);
#pragma unroll
      for (int c = 0; c < P; ++c) pre[c] = act2(pre[c], a.act);
      store_pairs<IO, VEC>(out + ((int64_t)k * a.T + t) * a.D, pre);
      slide<W>(win, v);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      store_pairs<IO, VEC>(st + k * row + (int64_t)j * a.D, win[j]);
  }
}

// Channel lanes of a 256-thread block: the smallest power of two that covers
// the channel vectors, so that narrow tensors put several runs in a block.
dim3 block_shape(int nvec) {
  int lx = 32;
  while (lx < 256 && lx < nvec) lx *= 2;
  return dim3(lx, 256 / lx);
}

template <typename K>
cudaError_t allow_shared(K kernel, int bytes, int fixed) {  // fixed: static
  if (bytes + fixed <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

bool vec_ok(const ConvArgs& a, int vec, size_t bytes) {
  const void* ps[] = {a.x, a.past, a.out, a.final_state, a.d_out, a.d_final, a.dx, a.d_past};
  for (const void* p : ps)
    if (p && !aligned_to(p, bytes)) return false;
  return a.D % vec == 0 && a.x_stride % vec == 0;
}

template <typename IO, int W, int VEC>
cudaError_t fwd_launch(const ConvArgs& a, cudaStream_t stream) {
  const int nvec = a.D / VEC;
  const dim3 block = block_shape(nvec);
  // 32 tokens a run re-read 3 of 35 inputs from L2; shorter runs when the
  // tokens would not give every SM its 2048 threads
  int run = 32;
  while (run > 4 && (a.tokens + run - 1) / run * nvec < (int64_t)148 * 2048) run /= 2;
  const int64_t n_runs = (a.tokens + run - 1) / run;
  const int64_t rows = n_runs + (a.final_state ? (int64_t)a.n_seqs * (W - 1) : 0);
  const dim3 grid((unsigned)((rows + block.y - 1) / block.y), (nvec + block.x - 1) / block.x);
  constexpr int bytes = Ring<IO, VEC>::ON ? kStages * kGroup * 256 * Ring<IO, VEC>::BYTES : 0;
  auto* k = conv_fwd_kernel<IO, W, VEC>;
  const cudaError_t e = allow_shared(k, bytes, 0);
  if (e != cudaSuccess) return e;
  if (rows) k<<<grid, block, bytes, stream>>>(a, nvec, run, n_runs);
  return cudaGetLastError();
}

template <typename IO, int W, int VEC>
cudaError_t step_launch(const ConvArgs& a, cudaStream_t stream) {
  const int nvec = a.D / VEC;
  const dim3 block = block_shape(nvec);
  // four sequences a thread where that still fills the SMs
  const int ns = (int64_t)a.n_seqs * nvec >= (int64_t)4 * 148 * 1024 ? 4 : 1;
  const int64_t rows = (a.n_seqs + ns - 1) / ns;
  const dim3 grid((unsigned)((rows + block.y - 1) / block.y), (nvec + block.x - 1) / block.x);
  if (ns == 4)
    conv_step_kernel<IO, W, VEC, 4><<<grid, block, 0, stream>>>(a, nvec);
  else
    conv_step_kernel<IO, W, VEC, 1><<<grid, block, 0, stream>>>(a, nvec);
  return cudaGetLastError();
}

// Tokens a thread takes backward: 64 (which reads 3 of 67 again and sums 512
// tokens before a part is written), fewer where that would not give every SM
// its two blocks (in fp32 one: the ring's 128 KB and the parts' 20 leave no room
// for a second).
int bwd_run(const ConvArgs& a) {
  int run = 64;
  while (run > 8 && a.tokens / run * (a.D / 4) < (int64_t)148 * 512) run /= 2;
  return run;
}
int64_t bwd_blocks(const ConvArgs& a) {
  const int64_t per = (int64_t)bwd_run(a) * kBwdRuns;
  return (a.tokens + per - 1) / per;
}

template <typename IO, int W, int VEC>
cudaError_t bwd_launch(const ConvArgs& a, float* part, cudaStream_t stream) {
  const int nvec = a.D / VEC;
  const int64_t blocks = bwd_blocks(a);
  const int64_t rows = a.d_past ? (int64_t)a.n_seqs * (W - 1) : 0;
  const dim3 block(kBwdLanes, kBwdRuns);
  const dim3 grid((unsigned)(blocks + (rows + kBwdRuns - 1) / kBwdRuns),
                  (nvec + kBwdLanes - 1) / kBwdLanes);
  constexpr int bytes = Ring<IO, VEC>::ON ? kStages * 2 * kGroup * 256 * Ring<IO, VEC>::BYTES : 0;
  auto* k = conv_bwd_kernel<IO, W, VEC>;
  cudaError_t e = allow_shared(k, bytes, kBwdRuns * (W + 1) * kBwdLanes * VEC * 4);
  if (e != cudaSuccess) return e;
  if (grid.x) k<<<grid, block, bytes, stream>>>(a, nvec, bwd_run(a), blocks, part);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  conv_weight_sum_kernel<<<dim3((a.D + 31) / 32, W + 1), dim3(32, 8), 0, stream>>>(
      part, blocks, W, a.D, a.dw, a.db);
  return cudaGetLastError();
}

#define KDA_CONV_W(FN, IO, VEC, ...)                          \
  (a.W == 2   ? FN<IO, 2, VEC>(__VA_ARGS__)                   \
   : a.W == 3 ? FN<IO, 3, VEC>(__VA_ARGS__)                   \
   : a.W == 4 ? FN<IO, 4, VEC>(__VA_ARGS__)                   \
              : cudaErrorInvalidValue)

}  // namespace

cudaError_t launch_conv_fwd(const ConvArgs& a, cudaStream_t stream) {
  if (a.bf16)
    return vec_ok(a, 4, 8) ? KDA_CONV_W(fwd_launch, __nv_bfloat16, 4, a, stream)
                            : KDA_CONV_W(fwd_launch, __nv_bfloat16, 1, a, stream);
  return vec_ok(a, 4, 16) ? KDA_CONV_W(fwd_launch, float, 4, a, stream)
                          : KDA_CONV_W(fwd_launch, float, 1, a, stream);
}

cudaError_t launch_conv_step(const ConvArgs& a, cudaStream_t stream) {
  if (a.n_seqs == 0 || a.T == 0) return cudaSuccess;
  if (a.bf16)
    return vec_ok(a, 4, 8) ? KDA_CONV_W(step_launch, __nv_bfloat16, 4, a, stream)
                            : KDA_CONV_W(step_launch, __nv_bfloat16, 1, a, stream);
  return vec_ok(a, 4, 16) ? KDA_CONV_W(step_launch, float, 4, a, stream)
                          : KDA_CONV_W(step_launch, float, 1, a, stream);
}

size_t conv_bwd_workspace_bytes(const ConvArgs& a) {
  return (size_t)bwd_blocks(a) * (a.W + 1) * a.D * sizeof(float);
}

cudaError_t launch_conv_bwd(const ConvArgs& a, void* ws, cudaStream_t stream) {
  float* part = static_cast<float*>(ws);
  if (a.bf16)
    return vec_ok(a, 4, 8) ? KDA_CONV_W(bwd_launch, __nv_bfloat16, 4, a, part, stream)
                           : KDA_CONV_W(bwd_launch, __nv_bfloat16, 1, a, part, stream);
  return vec_ok(a, 4, 16) ? KDA_CONV_W(bwd_launch, float, 4, a, part, stream)
                          : KDA_CONV_W(bwd_launch, float, 1, a, part, stream);
}

}  // namespace kda

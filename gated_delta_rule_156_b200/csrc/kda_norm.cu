// Norms at a block's boundary: the norm after the block with its gate, the
// residual scale and sum, and the next block's norm, in one pass over a row.
//
//   rms(v) = v r,  r = 1 / sqrt(mean(v^2) + eps)
//   h = x [act(g)];  p = rms(h) w_post [act(g)];  out = res + s p;
//   normed = rms(out) w_pre
// Backward of y = rms(v) w:  dv = r (dy w - vhat mean(dy w vhat)),
// dw = sum over rows of dy vhat, with vhat = v r.
//
// A row is read once and its elements stay in registers across both norms, so
// the kernels are bound by HBM.  Work split: TPR threads own a row (part of a
// warp for a head's row, a whole block for a wide one) and each of them the
// same elements of every row it meets, so weights are loaded once and the
// weights' gradients are register sums; the grid is the resident blocks only.
#include "kda_layer.cuh"

namespace kda {

namespace {

struct Act2 {
  float f, d;  // act(g) and its derivative
};
__device__ __forceinline__ float gate_f(float g, int act) {
  if (act == kActNone) return g;
  const float s = sigmoid_f(g);
  return act == kActSilu ? g * s : s;
}
__device__ __forceinline__ Act2 gate_fd(float g, int act) {
  if (act == kActNone) return Act2{g, 1.f};
  const float s = sigmoid_f(g);
  return act == kActSilu ? Act2{g * s, silu_grad(g, s)} : Act2{s, s * (1.f - s)};
}

// Sum of one value (or two) over the TPR threads of a row, in every one of them.  TPR <= 32:
// shuffles.  Above, the row is the whole block: per-warp sums through shared
// memory; `turn` alternates between two buffers, so that one barrier per sum
// is enough (a buffer is written again only behind the next sum's barrier).
struct RowSum {
  int tpr;
  int turn;
  float2* buf;  // [2][32]
  __device__ __forceinline__ float2 two(float a, float b) {
    const int w = tpr < 32 ? tpr : 32;
    for (int o = w >> 1; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (tpr <= 32) return make_float2(a, b);
    float2* s = buf + turn * 32;
    turn ^= 1;
    const int warps = tpr >> 5;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    // every warp sums the warps' values with the same tree
    const int lane = threadIdx.x & 31;
    float2 v = lane < warps ? s[lane] : make_float2(0.f, 0.f);
    for (int o = 16; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    return v;
  }
  __device__ __forceinline__ float one(float a) { return two(a, 0.f).x; }
};

// Element offsets of a thread's vectors and the rows of its block.
template <int VEC, int ITER>
struct Place {
  int lane, rows_per_block, sub;
  int col[ITER];
  bool on[ITER];
  __device__ __forceinline__ Place(int tpr, int width) {
    lane = threadIdx.x % tpr;
    sub = threadIdx.x / tpr;
    rows_per_block = blockDim.x / tpr;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int c = (lane + i * tpr) * VEC;
      on[i] = c < width;
      col[i] = on[i] ? c : 0;
    }
  }
};

template <int VEC, int ITER>
__device__ __forceinline__ void load_weight(const float* w, const Place<VEC, ITER>& p,
                                            float none, float (&v)[ITER][VEC]) {
#pragma unroll
  for (int i = 0; i < ITER; ++i)
#pragma unroll
    for (int c = 0; c < VEC; ++c) v[i][c] = w ? w[p.col[i] + c] : none;
}

template <typename IO, int VEC, int ITER>
__device__ __forceinline__ void load_row(const IO* row, const Place<VEC, ITER>& p, bool row_on,
                                         Raw<IO, VEC> (&v)[ITER]) {
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    if (row && row_on && p.on[i])
      v[i] = load_raw<IO, VEC>(row + p.col[i]);
    else
      v[i] = Raw<IO, VEC>{};
  }
}

template <typename IO, int VEC, int ITER>
__device__ __forceinline__ void store_row(IO* row, const Place<VEC, ITER>& p, bool row_on,
                                          const float (&v)[ITER][VEC]) {
#pragma unroll
  for (int i = 0; i < ITER; ++i)
    if (row_on && p.on[i]) store_vec<IO, VEC>(row + p.col[i], v[i]);
}

__device__ __forceinline__ int64_t strided(const NormArgs& a, int64_t row, int64_t stride) {
  if (a.heads == 1) return row * stride;
  const int64_t t = row / a.heads;
  return t * stride + (row - t * a.heads) * a.width;
}

template <typename IO, typename RT, int VEC, int ITER>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(NormArgs a, int tpr) {
  __shared__ float2 s_sum[64];
  const Place<VEC, ITER> p(tpr, a.width);
  RowSum sum{tpr, 0, s_sum};
  const int64_t rows = a.tokens * a.heads;
  const float inv_w = 1.f / (float)a.width;
  float wpost[ITER][VEC], scale[ITER][VEC], wpre[ITER][VEC];
  load_weight(a.post_weight, p, 1.f, wpost);
  load_weight(a.scale, p, 1.f, scale);
  load_weight(a.pre_weight, p, 1.f, wpre);
  const IO* x = static_cast<const IO*>(a.x);
  const IO* gate = static_cast<const IO*>(a.gate);
  const RT* res = static_cast<const RT*>(a.residual);
  for (int64_t base = (int64_t)blockIdx.x * p.rows_per_block; base < rows;
       base += (int64_t)gridDim.x * p.rows_per_block) {
    const int64_t row = base + p.sub;
    const bool on = row < rows;
    Raw<IO, VEC> rx[ITER], rg[ITER];
    Raw<RT, VEC> rr[ITER];
    load_row<IO>(x + (on ? strided(a, row, a.x_stride) : 0), p, on, rx);
    load_row<IO>(gate ? gate + (on ? strided(a, row, a.gate_stride) : 0) : gate, p, on, rg);
    load_row<RT>(res ? res + (on ? row : 0) * a.width : res, p, on, rr);
    float h[ITER][VEC], act[ITER][VEC];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      unpack(rx[i], h[i]);
      unpack(rg[i], act[i]);
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        act[i][c] = gate ? gate_f(act[i][c], a.act) : 1.f;
        if (a.gate_first) {
          h[i][c] *= act[i][c];
          act[i][c] = 1.f;
        }
        ss = fmaf(h[i][c], h[i][c], ss);
      }
    }
    float r1 = 1.f;
    if (a.post_weight) r1 = rsqrtf(sum.one(ss) * inv_w + a.eps);
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      float v[VEC];
      unpack(rr[i], v);
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        const float q = h[i][c] * r1 * wpost[i][c] * act[i][c];
        h[i][c] = fmaf(scale[i][c], q, v[c]);
        if (p.on[i]) ss = fmaf(h[i][c], h[i][c], ss);
      }
    }
    store_row<RT>(static_cast<RT*>(a.out) + (on ? row : 0) * a.width, p, on, h);
    if (a.pre_weight) {
      const float r2 = rsqrtf(sum.one(ss) * inv_w + a.eps);
#pragma unroll
      for (int i = 0; i < ITER; ++i)
#pragma unroll
        for (int c = 0; c < VEC; ++c) h[i][c] *= r2 * wpre[i][c];
      store_row<IO>(static_cast<IO*>(a.normed) + (on ? row : 0) * a.width, p, on, h);
    }
  }
}

// part[block * rows_per_block + sub][3][width]: the weights' gradients of one
// thread's rows; norm_weight_sum_kernel sums them in a fixed order.
template <typename IO, typename RT, int VEC, int ITER>
__global__ void __launch_bounds__(512)
    norm_bwd_kernel(NormArgs a, int tpr, float* __restrict__ part) {
  __shared__ float2 s_sum[64];
  const Place<VEC, ITER> p(tpr, a.width);
  RowSum sum{tpr, 0, s_sum};
  const int64_t rows = a.tokens * a.heads;
  const float inv_w = 1.f / (float)a.width;
  float wpost[ITER][VEC], scale[ITER][VEC], wpre[ITER][VEC];
  load_weight(a.post_weight, p, 1.f, wpost);
  load_weight(a.scale, p, 1.f, scale);
  load_weight(a.pre_weight, p, 1.f, wpre);
  float dpost[ITER][VEC] = {}, dscale[ITER][VEC] = {}, dpre[ITER][VEC] = {};
  const IO* x = static_cast<const IO*>(a.x);
  const IO* gate = static_cast<const IO*>(a.gate);
  const RT* res = static_cast<const RT*>(a.residual);
  const RT* dout = static_cast<const RT*>(a.d_out);
  const IO* dnorm = static_cast<const IO*>(a.d_normed);
  const bool pre = a.pre_weight && dnorm;
  for (int64_t base = (int64_t)blockIdx.x * p.rows_per_block; base < rows;
       base += (int64_t)gridDim.x * p.rows_per_block) {
    const int64_t row = base + p.sub;
    const bool on = row < rows;
    const int64_t at = (on ? row : 0) * a.width;
    Raw<IO, VEC> rx[ITER], rg[ITER], rn[ITER];
    Raw<RT, VEC> rr[ITER], ro[ITER];
    load_row<IO>(x + (on ? strided(a, row, a.x_stride) : 0), p, on, rx);
    load_row<IO>(gate ? gate + (on ? strided(a, row, a.gate_stride) : 0) : gate, p, on, rg);
    load_row<RT>(res ? res + at : res, p, on, rr);
    load_row<RT>(dout ? dout + at : dout, p, on, ro);
    load_row<IO>(dnorm ? dnorm + at : dnorm, p, on, rn);
    float r1 = 1.f, r2 = 0.f, ss = 0.f;
    if (a.post_weight) {
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        float v[VEC], g[VEC];
        unpack(rx[i], v);
        unpack(rg[i], g);
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          if (gate && a.gate_first) v[c] *= gate_f(g[c], a.act);
          ss = fmaf(v[c], v[c], ss);
        }
      }
      r1 = rsqrtf(sum.one(ss) * inv_w + a.eps);
      if (!on) r1 = 0.f;  // with eps 0 an absent row must not add 0 * inf
    }
    // hat: h r1; q: hat w_post (before a gate behind the norm); d: d out
    float hat[ITER][VEC], d[ITER][VEC], q[ITER][VEC];
    Act2 act[ITER][VEC];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      float v[VEC], g[VEC], o[VEC], n[VEC], r[VEC];
      unpack(rx[i], v);
      unpack(rg[i], g);
      unpack(rr[i], r);
      unpack(ro[i], o);
      unpack(rn[i], n);
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        act[i][c] = gate ? gate_fd(g[c], a.act) : Act2{1.f, 0.f};
        const float first = a.gate_first ? act[i][c].f : 1.f;
        const float behind = a.gate_first ? 1.f : act[i][c].f;
        hat[i][c] = v[c] * first * r1;
        q[i][c] = hat[i][c] * wpost[i][c];
        d[i][c] = o[c];
        if (pre) {
          const float out = fmaf(scale[i][c], q[i][c] * behind, r[c]);
          if (p.on[i]) {
            s1 = fmaf(out, out, s1);
            s2 = fmaf(n[c] * wpre[i][c], out, s2);
          }
        }
      }
    }
    if (pre) {
      const float2 t = sum.two(s1, s2);
      r2 = on ? rsqrtf(t.x * inv_w + a.eps) : 0.f;
      // d out += r2 (dn w - out r2 mean(dn w out r2))
      const float m = t.y * inv_w * r2 * r2;
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        float n[VEC], r[VEC];
        unpack(rn[i], n);
        unpack(rr[i], r);
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          const float behind = a.gate_first ? 1.f : act[i][c].f;
          const float out = fmaf(scale[i][c], q[i][c] * behind, r[c]);
          dpre[i][c] = fmaf(n[c], out * r2, dpre[i][c]);
          d[i][c] = fmaf(r2, n[c] * wpre[i][c] - out * m, d[i][c]);
        }
      }
    }
    if (a.dres) store_row<RT>(static_cast<RT*>(a.dres) + at, p, on, d);
    float s3 = 0.f;
    float dg[ITER][VEC];
#pragma unroll
    for (int i = 0; i < ITER; ++i)
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        const float behind = a.gate_first ? 1.f : act[i][c].f;
        dscale[i][c] = fmaf(d[i][c], q[i][c] * behind, dscale[i][c]);
        const float dp = d[i][c] * scale[i][c];
        dg[i][c] = dp * q[i][c] * act[i][c].d;  // the gate behind the norm
        d[i][c] = dp * behind;                  // into q
        dpost[i][c] = fmaf(d[i][c], hat[i][c], dpost[i][c]);
        if (p.on[i]) s3 = fmaf(d[i][c] * wpost[i][c], hat[i][c], s3);
      }
    if (a.post_weight) {
      const float m = sum.one(s3) * inv_w;
#pragma unroll
      for (int i = 0; i < ITER; ++i)
#pragma unroll
        for (int c = 0; c < VEC; ++c)
          d[i][c] = r1 * (d[i][c] * wpost[i][c] - hat[i][c] * m);
    }
    if (a.gate_first) {  // d is the gradient of h = x act(g)
#pragma unroll
      for (int i = 0; i < ITER; ++i) {
        float v[VEC];
        unpack(rx[i], v);
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          dg[i][c] = d[i][c] * v[c] * act[i][c].d;
          d[i][c] *= act[i][c].f;
        }
      }
    }
    if (gate) store_row<IO>(static_cast<IO*>(a.dgate) + at, p, on, dg);
    store_row<IO>(static_cast<IO*>(a.dx) + at, p, on, d);
  }
  const int64_t slot = (int64_t)blockIdx.x * p.rows_per_block + p.sub;
  float* o = part + slot * 3 * a.width;
#pragma unroll
  for (int i = 0; i < ITER; ++i)
    if (p.on[i])
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        if (a.dpost) o[p.col[i] + c] = dpost[i][c];
        if (a.dscale) o[a.width + p.col[i] + c] = dscale[i][c];
        if (a.dpre) o[2 * a.width + p.col[i] + c] = dpre[i][c];
      }
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

// Threads per row and vectors per thread.  Up to 32 vectors a row is part of
// a warp (the block holds several rows); above, the block is one row.
struct Shape {
  int tpr, block, iter;
};
Shape row_shape(int width, int vec, const int* iters, int n_iter, int max_tpr) {
  const int nvec = (width + vec - 1) / vec;
  Shape s{8, 0, 0};
  for (int k = 0; k < n_iter; ++k) {
    s.iter = iters[k];
    s.tpr = 8;
    while (s.tpr < max_tpr && s.tpr * s.iter < nvec) s.tpr *= 2;
    if (s.tpr * s.iter >= nvec) break;
  }
  s.block = s.tpr <= 32 ? 256 : s.tpr;
  return s;
}

template <typename K>
int resident_blocks(K kernel, int block, int sms) {
  int per = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, block, 0) != cudaSuccess ||
      per < 1)
    per = 1;
  return per * sms;
}

template <typename IO, typename RT, int VEC, int ITER>
cudaError_t fwd_launch(const NormArgs& a, const Shape& s, cudaStream_t stream) {
  auto* k = norm_fwd_kernel<IO, RT, VEC, ITER>;
  const int64_t need = (a.tokens * a.heads + s.block / s.tpr - 1) / (s.block / s.tpr);
  const int64_t most = resident_blocks(k, s.block, sm_count());
  k<<<(unsigned)(need < most ? need : most), s.block, 0, stream>>>(a, s.tpr);
  return cudaGetLastError();
}

template <typename IO, typename RT, int VEC, int ITER>
cudaError_t bwd_launch(const NormArgs& a, const Shape& s, int sms, float* part,
                       cudaStream_t stream) {
  auto* k = norm_bwd_kernel<IO, RT, VEC, ITER>;
  const int per = s.block / s.tpr;
  const int64_t need = (a.tokens * a.heads + per - 1) / per;
  int64_t blocks = resident_blocks(k, s.block, sms);
  const int64_t cap = (int64_t)sms * (2048 / s.block);
  blocks = blocks < need ? blocks : need;
  blocks = blocks < cap ? blocks : cap;
  if (blocks > 0) k<<<(unsigned)blocks, s.block, 0, stream>>>(a, s.tpr, part);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (a.dpost || a.dscale || a.dpre)
    norm_weight_sum_kernel<<<dim3((a.width + 31) / 32, 3), dim3(32, 16), 0, stream>>>(
        part, (int)(blocks * per), a.width, a.dpost, a.dscale, a.dpre);
  return cudaGetLastError();
}

constexpr int kVecIters[] = {1, 2, 4}, kOneIters[] = {4, 16};
constexpr int kBwdVecIters[] = {1, 2, 4, 8}, kBwdOneIters[] = {4, 32};

// 16 bytes of io a load where every pointer, stride and the width allow it,
// single elements otherwise.
bool vec_ok(const NormArgs& a, int vec) {
  const void* io[] = {a.x, a.gate, a.normed, a.d_normed, a.dx, a.dgate,
                      a.residual, a.out, a.d_out, a.dres};
  for (const void* p : io)
    if (p && !aligned_to(p, 16)) return false;
  return a.width % vec == 0 && a.x_stride % vec == 0 && a.gate_stride % vec == 0;
}

Shape bwd_shape(const NormArgs& a, bool vec) {
  const int v = vec ? (a.bf16 ? 8 : 4) : 1;
  return vec ? row_shape(a.width, v, kBwdVecIters, 4, 512)
             : row_shape(a.width, v, kBwdOneIters, 2, 512);
}

template <typename IO, typename RT, int VEC>
cudaError_t fwd_pick(const NormArgs& a, cudaStream_t st) {
  if (VEC > 1) {
    const Shape s = row_shape(a.width, VEC, kVecIters, 3, 1024);
    if (s.iter == 1) return fwd_launch<IO, RT, VEC, 1>(a, s, st);
    if (s.iter == 2) return fwd_launch<IO, RT, VEC, 2>(a, s, st);
    return fwd_launch<IO, RT, VEC, 4>(a, s, st);
  }
  const Shape s = row_shape(a.width, 1, kOneIters, 2, 1024);
  if (s.iter == 4) return fwd_launch<IO, RT, 1, 4>(a, s, st);
  return fwd_launch<IO, RT, 1, 16>(a, s, st);
}

template <typename IO, typename RT, int VEC>
cudaError_t bwd_pick(const NormArgs& a, int sms, float* part, cudaStream_t st) {
  const Shape s = bwd_shape(a, VEC > 1);
  if (VEC > 1) {
    if (s.iter == 1) return bwd_launch<IO, RT, VEC, 1>(a, s, sms, part, st);
    if (s.iter == 2) return bwd_launch<IO, RT, VEC, 2>(a, s, sms, part, st);
    if (s.iter == 4) return bwd_launch<IO, RT, VEC, 4>(a, s, sms, part, st);
    return bwd_launch<IO, RT, VEC, 8>(a, s, sms, part, st);
  }
  if (s.iter == 4) return bwd_launch<IO, RT, 1, 4>(a, s, sms, part, st);
  return bwd_launch<IO, RT, 1, 32>(a, s, sms, part, st);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t st) {
  if (a.tokens == 0) return cudaSuccess;
  using bf = __nv_bfloat16;
  if (a.bf16 && a.res_bf16)
    return vec_ok(a, 8) ? fwd_pick<bf, bf, 8>(a, st) : fwd_pick<bf, bf, 1>(a, st);
  if (a.bf16) return vec_ok(a, 8) ? fwd_pick<bf, float, 8>(a, st) : fwd_pick<bf, float, 1>(a, st);
  return vec_ok(a, 4) ? fwd_pick<float, float, 4>(a, st) : fwd_pick<float, float, 1>(a, st);
}

size_t norm_bwd_workspace_bytes(const NormArgs& a, int sms) {
  if (!a.dpost && !a.dscale && !a.dpre) return 0;
  const Shape s = bwd_shape(a, vec_ok(a, a.bf16 ? 8 : 4));
  const int per = s.block / s.tpr;
  const int64_t need = (a.tokens * a.heads + per - 1) / per;
  const int64_t cap = (int64_t)sms * (2048 / s.block);
  return (size_t)(need < cap ? need : cap) * per * 3 * a.width * sizeof(float);
}

cudaError_t launch_norm_bwd(const NormArgs& a, void* ws, int sms, cudaStream_t st) {
  using bf = __nv_bfloat16;
  float* part = static_cast<float*>(ws);
  if (a.bf16 && a.res_bf16)
    return vec_ok(a, 8) ? bwd_pick<bf, bf, 8>(a, sms, part, st)
                        : bwd_pick<bf, bf, 1>(a, sms, part, st);
  if (a.bf16)
    return vec_ok(a, 8) ? bwd_pick<bf, float, 8>(a, sms, part, st)
                        : bwd_pick<bf, float, 1>(a, sms, part, st);
  return vec_ok(a, 4) ? bwd_pick<float, float, 4>(a, sms, part, st)
                      : bwd_pick<float, float, 1>(a, sms, part, st);
}

}  // namespace kda

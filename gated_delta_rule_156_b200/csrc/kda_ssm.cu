// Selective state space scan: the forward over prompts, the first pass of the
// backward (which saves states), and the step for new tokens.  The recurrence
// and its split over lanes are in kda_ssm.cuh.
//
// Bound: an update costs one exponential and about 6 flops.  The special
// function unit gives 16 a cycle and SM, so 16 states a channel cost more
// there (0.24 ms for 2 x 8192 tokens of 4096 channels at 1.9 GHz) than the
// 8 bytes a token and channel cost in HBM (0.08 ms).
#include "kda_ssm.cuh"

namespace kda {

namespace {

constexpr int kTile = 32;  // tokens per tile

template <typename IO, int L, int MODE>
__global__ void __launch_bounds__(kSsmThreads) ssm_fwd_kernel(SsmArgs a, SsmSave save) {
  constexpr int CH = kSsmThreads / L, SW = L * kSsmStates;
  __shared__ float2 s_dt[kTile][CH];
  __shared__ float s_y[kTile][CH];
  __shared__ __align__(16) float s_b[kTile][SW], s_c[kTile][SW];
  const int tid = threadIdx.x, l = tid % L, ch = tid / L;
  const int n_blk = ssm_blocks(a, CH);
  const int seq = blockIdx.x / n_blk;
  const SsmBlock blk(a, CH, blockIdx.x % n_blk);
  int start, end;
  seq_range(a.cu, seq, a.T, &start, &end);

  const IO* u = static_cast<const IO*>(a.u);
  const IO* delta = static_cast<const IO*>(a.delta);
  const IO* z = static_cast<const IO*>(a.z);
  const IO* B = static_cast<const IO*>(a.B) + (int64_t)blk.g * a.b_group;
  const IO* C = static_cast<const IO*>(a.C) + (int64_t)blk.g * a.c_group;
  const bool on = ch < blk.n;
  const int d = blk.c0 + (on ? ch : 0);
  float A2[kSsmStates], h[kSsmStates];
#pragma unroll
  for (int i = 0; i < kSsmStates; ++i) {
    const int n = l * kSsmStates + i;
    const bool real = on && n < a.S;
    A2[i] = real ? a.A[(int64_t)d * a.S + n] * kLog2e : 0.f;
    h[i] = real && a.h0 ? a.h0[((int64_t)seq * a.D + d) * a.S + n] : 0.f;
  }

  for (int t0 = start; t0 < end; t0 += kTile) {
    const int m = min(kTile, end - t0);
    for (int i = tid; i < kTile * CH; i += kSsmThreads) {
      const int t = i / CH, c = i % CH;
      float2 v = make_float2(0.f, 0.f);
      if (t < m && c < blk.n) {
        const int64_t tok = t0 + t;
        const float raw = to_f32(delta[tok * a.delta_stride + blk.c0 + c]) +
                          (a.bias ? a.bias[blk.c0 + c] : 0.f);
        v.x = a.softplus ? softplus_f(raw) : raw;
        v.y = v.x * to_f32(u[tok * a.u_stride + blk.c0 + c]);
      }
      s_dt[t][c] = v;
    }
    for (int i = tid; i < kTile * SW; i += kSsmThreads) {
      const int t = i / SW, n = i % SW;
      const bool real = t < m && n < a.S;
      s_b[t][n] = real ? to_f32(B[(int64_t)(t0 + t) * a.b_stride + n]) : 0.f;
      s_c[t][n] = real ? to_f32(C[(int64_t)(t0 + t) * a.c_stride + n]) : 0.f;
    }
    __syncthreads();
    for (int t = 0; t < m; t += 4) {
      if (MODE == kSsmSave && t % kSsmChunk == 0) {
        const int64_t id = ssm_chunk_id(seq, start, (t0 - start + t) / kSsmChunk);
#pragma unroll
        for (int i = 0; i < kSsmStates; ++i)
          if (on && l * kSsmStates + i < a.S)
            save.states[(id * a.D + d) * a.S + l * kSsmStates + i] = h[i];
      }
      float y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // behind the last token: step 0 keeps the state
        const float2 v = s_dt[t + j][ch];
        const float4 b = *reinterpret_cast<const float4*>(&s_b[t + j][l * kSsmStates]);
        const float4 c = *reinterpret_cast<const float4*>(&s_c[t + j][l * kSsmStates]);
        h[0] = fmaf(ex2_f(v.x * A2[0]), h[0], v.y * b.x);
        h[1] = fmaf(ex2_f(v.x * A2[1]), h[1], v.y * b.y);
        h[2] = fmaf(ex2_f(v.x * A2[2]), h[2], v.y * b.z);
        h[3] = fmaf(ex2_f(v.x * A2[3]), h[3], v.y * b.w);
        y[j] = fmaf(h[0], c.x, h[1] * c.y) + fmaf(h[2], c.z, h[3] * c.w);
      }
      int first = 0;
      SpreadSum<4, 1, L>::run(y, l, first);
      constexpr int LEFT = L >= 4 ? 1 : 4 / L;
      if (l < 4)
#pragma unroll
        for (int j = 0; j < LEFT; ++j) s_y[t + first + j][ch] = y[j];
    }
    __syncthreads();
    if (MODE == kSsmOut || save.dz) {
      for (int i = tid; i < m * CH; i += kSsmThreads) {
        const int t = i / CH, c = i % CH;
        if (c >= blk.n) continue;
        const int64_t tok = t0 + t;
        const int dd = blk.c0 + c;
        float y = s_y[t][c];
        if (a.skip) y = fmaf(a.skip[dd], to_f32(u[tok * a.u_stride + dd]), y);
        if (MODE == kSsmOut) {
          if (z) {
            const float g = to_f32(z[tok * a.z_stride + dd]);
            y *= g * sigmoid_f(g);
          }
          static_cast<IO*>(a.out)[tok * a.D + dd] = from_f32<IO>(y);
        } else {
          const float g = to_f32(z[tok * a.z_stride + dd]);
          const float dout = to_f32(static_cast<const IO*>(save.d_out)[tok * a.D + dd]);
          static_cast<IO*>(save.dz)[tok * a.D + dd] =
              from_f32<IO>(dout * y * silu_grad(g, sigmoid_f(g)));
        }
      }
    }
  }
  if (MODE == kSsmOut && a.h_out && on) {
#pragma unroll
    for (int i = 0; i < kSsmStates; ++i)
      if (l * kSsmStates + i < a.S)
        a.h_out[((int64_t)seq * a.D + d) * a.S + l * kSsmStates + i] = h[i];
  }
}

// New tokens: L lanes own a channel of a sequence and stream its state, read
// and written once per call.
template <typename IO, int L>
__global__ void __launch_bounds__(256) ssm_step_kernel(SsmArgs a) {
  const int l = threadIdx.x % L;
  const int64_t id = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / L;
  const bool on = id < (int64_t)a.n_seqs * a.D;
  const int64_t at = on ? id : 0;
  const int seq = (int)(at / a.D), d = (int)(at - (int64_t)seq * a.D);
  const int g = d / (a.D / a.G);
  float A2[kSsmStates], h[kSsmStates];
  const bool vec = (a.S & 3) == 0;
  float* st = a.h_out + at * a.S + l * kSsmStates;
  const bool real4 = on && l * kSsmStates < a.S;
  if (vec) {
    const float4 z4 = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 hv = real4 ? *reinterpret_cast<const float4*>(st) : z4;
    const float4 av = real4 ? *reinterpret_cast<const float4*>(
                                  a.A + (int64_t)d * a.S + l * kSsmStates) : z4;
    h[0] = hv.x; h[1] = hv.y; h[2] = hv.z; h[3] = hv.w;
    A2[0] = av.x; A2[1] = av.y; A2[2] = av.z; A2[3] = av.w;
  } else {
#pragma unroll
    for (int i = 0; i < kSsmStates; ++i) {
      const bool real = on && l * kSsmStates + i < a.S;
      h[i] = real ? st[i] : 0.f;
      A2[i] = real ? a.A[(int64_t)d * a.S + l * kSsmStates + i] : 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < kSsmStates; ++i) A2[i] *= kLog2e;
  const float bias = a.bias ? a.bias[d] : 0.f, skip = a.skip ? a.skip[d] : 0.f;
  for (int t = 0; t < a.T; ++t) {
    const int64_t tok = (int64_t)seq * a.T + t;
    const float raw = to_f32(static_cast<const IO*>(a.delta)[tok * a.delta_stride + d]) + bias;
    const float uu = to_f32(static_cast<const IO*>(a.u)[tok * a.u_stride + d]);
    const IO* B = static_cast<const IO*>(a.B) + tok * a.b_stride + (int64_t)g * a.b_group;
    const IO* C = static_cast<const IO*>(a.C) + tok * a.c_stride + (int64_t)g * a.c_group;
    const float dt = a.softplus ? softplus_f(raw) : raw, dtu = dt * uu;
    float y = 0.f;
#pragma unroll
    for (int i = 0; i < kSsmStates; ++i) {
      const int n = l * kSsmStates + i;
      if (n < a.S) {
        h[i] = fmaf(ex2_f(dt * A2[i]), h[i], dtu * to_f32(B[n]));
        y = fmaf(h[i], to_f32(C[n]), y);
      }
    }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (on && l == 0) {
      y = fmaf(skip, uu, y);
      if (a.z) {
        const float gz = to_f32(static_cast<const IO*>(a.z)[tok * a.z_stride + d]);
        y *= gz * sigmoid_f(gz);
      }
      static_cast<IO*>(a.out)[tok * a.D + d] = from_f32<IO>(y);
    }
  }
  if (vec) {
    if (real4) *reinterpret_cast<float4*>(st) = make_float4(h[0], h[1], h[2], h[3]);
  } else {
#pragma unroll
    for (int i = 0; i < kSsmStates; ++i)
      if (on && l * kSsmStates + i < a.S) st[i] = h[i];
  }
}

template <typename IO, int L, int MODE>
cudaError_t fwd_launch(const SsmArgs& a, const SsmSave& save, cudaStream_t st) {
  const unsigned grid = (unsigned)ssm_blocks(a, kSsmThreads / L) * (unsigned)a.n_seqs;
  ssm_fwd_kernel<IO, L, MODE><<<grid, kSsmThreads, 0, st>>>(a, save);
  return cudaGetLastError();
}

template <typename IO, int MODE>
cudaError_t fwd_pick(const SsmArgs& a, const SsmSave& save, cudaStream_t st) {
  switch (ssm_lanes(a.S)) {
    case 2: return fwd_launch<IO, 2, MODE>(a, save, st);
    case 4: return fwd_launch<IO, 4, MODE>(a, save, st);
    case 8: return fwd_launch<IO, 8, MODE>(a, save, st);
    case 16: return fwd_launch<IO, 16, MODE>(a, save, st);
    case 32: return fwd_launch<IO, 32, MODE>(a, save, st);
  }
  return cudaErrorInvalidValue;
}

template <typename IO, int L>
cudaError_t step_launch(const SsmArgs& a, cudaStream_t st) {
  const int64_t threads = (int64_t)a.n_seqs * a.D * L;
  ssm_step_kernel<IO, L><<<(unsigned)((threads + 255) / 256), 256, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename IO>
cudaError_t step_pick(const SsmArgs& a, cudaStream_t st) {
  switch (ssm_lanes(a.S)) {
    case 2: return step_launch<IO, 2>(a, st);
    case 4: return step_launch<IO, 4>(a, st);
    case 8: return step_launch<IO, 8>(a, st);
    case 16: return step_launch<IO, 16>(a, st);
    case 32: return step_launch<IO, 32>(a, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_ssm_fwd(const SsmArgs& a, cudaStream_t st) {
  if (a.n_seqs == 0) return cudaSuccess;
  const SsmSave none{};
  return a.bf16 ? fwd_pick<__nv_bfloat16, kSsmOut>(a, none, st)
                : fwd_pick<float, kSsmOut>(a, none, st);
}

cudaError_t launch_ssm_save(const SsmArgs& a, const SsmSave& save, cudaStream_t st) {
  if (a.n_seqs == 0) return cudaSuccess;
  return a.bf16 ? fwd_pick<__nv_bfloat16, kSsmSave>(a, save, st)
                : fwd_pick<float, kSsmSave>(a, save, st);
}

cudaError_t launch_ssm_step(const SsmArgs& a, cudaStream_t st) {
  if (a.n_seqs == 0 || a.T == 0) return cudaSuccess;
  return a.bf16 ? step_pick<__nv_bfloat16>(a, st) : step_pick<float>(a, st);
}

}  // namespace kda

// Selective state space scan, backward.  With dy_t = d_out_t silu(z_t) and
// going from the last token to the first:
//   dh_t = dy_t C_t + a_{t+1} dh_{t+1}        (d_final behind the last token)
//   dC_t = sum_d dy_t h_t,   dB_t = sum_d dh_t step_t u_t
//   fed_t = sum_n dh_t B_t,  q_t[n] = dh_t a_t h_{t-1}
//   du_t = fed_t step_t + dy_t skip,  dstep_t = sum_n q_t A + fed_t u_t
//   dA = sum_t q_t step_t,  ddelta_t = dstep_t sigmoid(delta_t + bias)
// Two passes: the forward recurrence once more, which keeps the state at
// every 8th token (and writes dz, which needs y); then, chunk by chunk of 8
// tokens from the end, the chunk's states and decays again in registers and
// the sums above.  Sums over a channel's states are exchanges between its
// lanes, sums over channels (dB, dC) exchanges between the warp's channels,
// then shared memory, then one part per channel block in the workspace, which
// a last kernel adds up: every order is fixed.
#include "kda_ssm.cuh"

namespace kda {

namespace {

constexpr float kLn2 = 0.6931471805599453f;

struct BwdParts {
  float* states;  // [chunk ids][D][S]
  float* bc;      // [channel block][token][2][S]
  float* dA;      // [n_seqs][D][S]
  float* dskip;   // [n_seqs][D]
  float* dbias;   // [n_seqs][D]
};

template <typename IO, int L>
__global__ void __launch_bounds__(kSsmThreads) ssm_bwd_kernel(SsmBwdArgs b, BwdParts part) {
  constexpr int CH = kSsmThreads / L, SW = L * kSsmStates, K = kSsmChunk;
  constexpr int WARPS = kSsmThreads / 32;
  const SsmArgs& a = b.f;
  __shared__ float2 s_dt[K][CH];
  __shared__ float s_dy[K][CH], s_fed[K][CH], s_qa[K][CH];
  __shared__ __align__(16) float s_b[K][SW], s_c[K][SW];
  __shared__ float s_part[WARPS][K][2][SW];
  const int tid = threadIdx.x, l = tid % L, ch = tid / L, warp = tid / 32;
  const int n_blk = ssm_blocks(a, CH);
  const int seq = blockIdx.x / n_blk, block = blockIdx.x % n_blk;
  const SsmBlock blk(a, CH, block);
  int start, end;
  seq_range(a.cu, seq, a.T, &start, &end);

  const IO* u = static_cast<const IO*>(a.u);
  const IO* delta = static_cast<const IO*>(a.delta);
  const IO* z = static_cast<const IO*>(a.z);
  const IO* dout = static_cast<const IO*>(b.d_out);
  const IO* B = static_cast<const IO*>(a.B) + (int64_t)blk.g * a.b_group;
  const IO* C = static_cast<const IO*>(a.C) + (int64_t)blk.g * a.c_group;
  const bool on = ch < blk.n;
  const int d = blk.c0 + (on ? ch : 0);
  float A2[kSsmStates], dh[kSsmStates], dA[kSsmStates];
#pragma unroll
  for (int i = 0; i < kSsmStates; ++i) {
    const int n = l * kSsmStates + i;
    const bool real = on && n < a.S;
    A2[i] = real ? a.A[(int64_t)d * a.S + n] * kLog2e : 0.f;
    dh[i] = real && b.d_final ? b.d_final[((int64_t)seq * a.D + d) * a.S + n] : 0.f;
    dA[i] = 0.f;
  }
  // the channel this thread finishes tokens of
  const int oc = tid % CH;
  const bool out_on = oc < blk.n;
  const int od = blk.c0 + (out_on ? oc : 0);
  const float bias = a.bias ? a.bias[od] : 0.f, skip = a.skip ? a.skip[od] : 0.f;
  float dskip = 0.f, dbias = 0.f;

  const int chunks = (end - start + K - 1) / K;
  for (int k = chunks - 1; k >= 0; --k) {
    const int t0 = start + k * K, m = min(K, end - t0);
    for (int i = tid; i < K * CH; i += kSsmThreads) {
      const int t = i / CH;
      float2 v = make_float2(0.f, 0.f);
      float dy = 0.f;
      if (t < m && out_on) {
        const int64_t tok = t0 + t;
        const float raw = to_f32(delta[tok * a.delta_stride + od]) + bias;
        v.x = a.softplus ? softplus_f(raw) : raw;
        v.y = v.x * to_f32(u[tok * a.u_stride + od]);
        dy = to_f32(dout[tok * a.D + od]);
        if (z) {
          const float g = to_f32(z[tok * a.z_stride + od]);
          dy *= g * sigmoid_f(g);
        }
      }
      s_dt[t][oc] = v;
      s_dy[t][oc] = dy;
    }
    for (int i = tid; i < K * SW; i += kSsmThreads) {
      const int t = i / SW, n = i % SW;
      const bool real = t < m && n < a.S;
      s_b[t][n] = real ? to_f32(B[(int64_t)(t0 + t) * a.b_stride + n]) : 0.f;
      s_c[t][n] = real ? to_f32(C[(int64_t)(t0 + t) * a.c_stride + n]) : 0.f;
    }
    float hp[K + 1][kSsmStates], av[K][kSsmStates];
    const float* hs = part.states + (ssm_piece_id(seq, start, K, k) * a.D + d) * a.S;
#pragma unroll
    for (int i = 0; i < kSsmStates; ++i)
      hp[0][i] = on && l * kSsmStates + i < a.S ? hs[l * kSsmStates + i] : 0.f;
    __syncthreads();
#pragma unroll
    for (int t = 0; t < K; ++t) {
      const float2 v = s_dt[t][ch];
      const float4 bv = *reinterpret_cast<const float4*>(&s_b[t][l * kSsmStates]);
      const float bb[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
      for (int i = 0; i < kSsmStates; ++i) {
        av[t][i] = ex2_f(v.x * A2[i]);
        hp[t + 1][i] = fmaf(av[t][i], hp[t][i], v.y * bb[i]);
      }
    }
    float fed[K], qa[K], dAc[kSsmStates] = {};
#pragma unroll
    for (int t = K - 1; t >= 0; --t) {
      const float2 v = s_dt[t][ch];
      const float dy = s_dy[t][ch];
      const float4 bv = *reinterpret_cast<const float4*>(&s_b[t][l * kSsmStates]);
      const float4 cv = *reinterpret_cast<const float4*>(&s_c[t][l * kSsmStates]);
      const float bb[4] = {bv.x, bv.y, bv.z, bv.w}, cc[4] = {cv.x, cv.y, cv.z, cv.w};
      float bc[2 * kSsmStates];
      fed[t] = 0.f;
      qa[t] = 0.f;
#pragma unroll
      for (int i = 0; i < kSsmStates; ++i) {
        dh[i] = fmaf(dy, cc[i], dh[i]);
        bc[i] = dh[i] * v.y;
        bc[kSsmStates + i] = dy * hp[t + 1][i];
        fed[t] = fmaf(dh[i], bb[i], fed[t]);
        dh[i] *= av[t][i];
        const float q = dh[i] * hp[t][i];
        qa[t] = fmaf(q, A2[i], qa[t]);
        dAc[i] = fmaf(q, v.x, dAc[i]);
      }
      int first = 0;
      SpreadSum<2 * kSsmStates, L, 32>::run(bc, tid, first);
      constexpr int LEFT = 2 * kSsmStates / (32 / L) > 1 ? 2 * kSsmStates / (32 / L) : 1;
#pragma unroll
      for (int i = 0; i < LEFT; ++i) {
        const int e = first + i;
        s_part[warp][t][e / kSsmStates][l * kSsmStates + e % kSsmStates] = bc[i];
      }
    }
#pragma unroll
    for (int i = 0; i < kSsmStates; ++i) dA[i] += dAc[i];
    int first = 0, first2 = 0;
    SpreadSum<K, 1, L>::run(fed, l, first);
    SpreadSum<K, 1, L>::run(qa, l, first2);
    constexpr int LEFT = K / L > 1 ? K / L : 1;
#pragma unroll
    for (int i = 0; i < LEFT; ++i) {
      s_fed[first + i][ch] = fed[i];
      s_qa[first + i][ch] = qa[i];
    }
    __syncthreads();
    for (int i = tid; i < m * CH; i += kSsmThreads) {
      const int t = i / CH;
      if (!out_on) continue;
      const int64_t tok = t0 + t;
      const float raw = to_f32(delta[tok * a.delta_stride + od]) + bias;
      const float uu = to_f32(u[tok * a.u_stride + od]);
      const float dy = s_dy[t][oc], f = s_fed[t][oc];
      float dd = fmaf(f, uu, kLn2 * s_qa[t][oc]);
      if (a.softplus) dd *= sigmoid_f(raw);
      dskip = fmaf(dy, uu, dskip);
      dbias += dd;
      static_cast<IO*>(b.du)[tok * a.D + od] = from_f32<IO>(fmaf(f, s_dt[t][oc].x, dy * skip));
      static_cast<IO*>(b.ddelta)[tok * a.D + od] = from_f32<IO>(dd);
    }
    for (int i = tid; i < m * 2 * SW; i += kSsmThreads) {
      const int t = i / (2 * SW), which = i / SW % 2, n = i % SW;
      if (n >= a.S) continue;
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) s += s_part[w][t][which][n];
      part.bc[(((int64_t)block * a.tokens + t0 + t) * 2 + which) * a.S + n] = s;
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < kSsmStates; ++i) {
    const int n = l * kSsmStates + i;
    if (!on || n >= a.S) continue;
    const int64_t at = ((int64_t)seq * a.D + d) * a.S + n;
    part.dA[at] = dA[i];
    if (b.dh0) b.dh0[at] = dh[i];
  }
  // sums over the threads that finished tokens of one channel
  float* sum = &s_part[0][0][0][0];
  sum[tid] = dskip;
  sum[kSsmThreads + tid] = dbias;
  __syncthreads();
  if (tid < CH && tid < blk.n) {
    float x = 0.f, y = 0.f;
    for (int i = tid; i < kSsmThreads; i += CH) {
      x += sum[i];
      y += sum[kSsmThreads + i];
    }
    part.dskip[(int64_t)seq * a.D + blk.c0 + tid] = x;
    part.dbias[(int64_t)seq * a.D + blk.c0 + tid] = y;
  }
}

// dB and dC of a token's group: the channel blocks' parts.
template <typename IO>
__global__ void ssm_bc_sum_kernel(SsmBwdArgs b, const float* __restrict__ bc, int blocks_per_group) {
  const SsmArgs& a = b.f;
  const int64_t per = (int64_t)2 * a.S;
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (id >= a.tokens * a.G * per) return;
  const int e = (int)(id % per);
  const int64_t tg = id / per;
  const int g = (int)(tg % a.G);
  const int64_t tok = tg / a.G;
  SeqCursor q;
  if (!find_seq(a.cu, a.n_seqs, a.T, (int)tok, &q) || tok < q.start) return;
  float s = 0.f;
  for (int i = 0; i < blocks_per_group; ++i)
    s += bc[((int64_t)(g * blocks_per_group + i) * a.tokens + tok) * per + e];
  IO* out = static_cast<IO*>(e < a.S ? b.dB : b.dC);
  out[(tok * a.G + g) * a.S + e % a.S] = from_f32<IO>(s);
}

// out[i] = sum over sequences of part[seq][i]
__global__ void ssm_seq_sum_kernel(const float* __restrict__ part, int n_seqs, int64_t n,
                                   float* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  float s = 0.f;
  for (int k = 0; k < n_seqs; ++k) s += part[k * n + i];
  out[i] = s;
}

size_t up(size_t x) { return (x + 255) & ~(size_t)255; }

struct Layout {
  size_t states, bc, dA, dskip, dbias, total;
};
Layout layout(const SsmBwdArgs& b) {
  const SsmArgs& a = b.f;
  const size_t ids = (size_t)a.tokens / kSsmChunk + a.n_seqs + 1;
  // dense sequences count their chunks by the same ids
  const size_t blocks = ssm_blocks(a, kSsmThreads / ssm_lanes(a.S));
  Layout o;
  o.states = 0;
  o.bc = o.states + up(ids * a.D * a.S * 4);
  o.dA = o.bc + up(blocks * a.tokens * 2 * a.S * 4);
  o.dskip = o.dA + up((size_t)a.n_seqs * a.D * a.S * 4);
  o.dbias = o.dskip + up((size_t)a.n_seqs * a.D * 4);
  o.total = o.dbias + up((size_t)a.n_seqs * a.D * 4);
  return o;
}

template <typename IO, int L>
cudaError_t bwd_launch(const SsmBwdArgs& b, const BwdParts& part, cudaStream_t st) {
  const unsigned grid = (unsigned)ssm_blocks(b.f, kSsmThreads / L) * (unsigned)b.f.n_seqs;
  if (grid) ssm_bwd_kernel<IO, L><<<grid, kSsmThreads, 0, st>>>(b, part);
  return cudaGetLastError();
}

template <typename IO>
cudaError_t bwd_pick(const SsmBwdArgs& b, const BwdParts& part, cudaStream_t st) {
  cudaError_t e = cudaErrorInvalidValue;
  switch (ssm_lanes(b.f.S)) {
    case 2: e = bwd_launch<IO, 2>(b, part, st); break;
    case 4: e = bwd_launch<IO, 4>(b, part, st); break;
    case 8: e = bwd_launch<IO, 8>(b, part, st); break;
    case 16: e = bwd_launch<IO, 16>(b, part, st); break;
    case 32: e = bwd_launch<IO, 32>(b, part, st); break;
  }
  if (e != cudaSuccess) return e;
  const int64_t n = b.f.tokens * b.f.G * 2 * b.f.S;
  const int per_group = ssm_blocks(b.f, kSsmThreads / ssm_lanes(b.f.S)) / b.f.G;
  if (n) ssm_bc_sum_kernel<IO><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(b, part.bc, per_group);
  return cudaGetLastError();
}

cudaError_t seq_sum(const float* part, const SsmArgs& a, int64_t n, float* out, cudaStream_t st) {
  if (!out) return cudaSuccess;
  ssm_seq_sum_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(part, a.n_seqs, n, out);
  return cudaGetLastError();
}

}  // namespace

size_t ssm_bwd_workspace_bytes(const SsmBwdArgs& b) { return layout(b).total; }

int ssm_bwd_kernel_count(const SsmBwdArgs& b) {
  return (b.f.n_seqs ? 2 : 0) + (b.f.tokens ? 1 : 0) + 1 + (b.dskip ? 1 : 0) + (b.dbias ? 1 : 0);
}

cudaError_t launch_ssm_bwd(const SsmBwdArgs& b, void* ws, cudaStream_t st) {
  const Layout o = layout(b);
  char* w = static_cast<char*>(ws);
  BwdParts part{reinterpret_cast<float*>(w + o.states), reinterpret_cast<float*>(w + o.bc),
                reinterpret_cast<float*>(w + o.dA), reinterpret_cast<float*>(w + o.dskip),
                reinterpret_cast<float*>(w + o.dbias)};
  SsmSave save{part.states, b.d_out, b.f.z ? b.dz : nullptr};
  const SsmSplit whole{INT32_MAX, nullptr, nullptr};
  cudaError_t e = launch_ssm_save(b.f, save, whole, st);
  if (e == cudaSuccess)
    e = b.f.bf16 ? bwd_pick<__nv_bfloat16>(b, part, st) : bwd_pick<float>(b, part, st);
  if (e == cudaSuccess) e = seq_sum(part.dA, b.f, (int64_t)b.f.D * b.f.S, b.dA, st);
  if (e == cudaSuccess) e = seq_sum(part.dskip, b.f, b.f.D, b.dskip, st);
  if (e == cudaSuccess) e = seq_sum(part.dbias, b.f, b.f.D, b.dbias, st);
  return e;
}

}  // namespace kda

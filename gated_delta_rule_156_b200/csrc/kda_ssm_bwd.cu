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
// a last kernel adds up: every order is fixed.  Measured: 1.29 ms for 2 x 4096
// tokens of 4096 channels with 16 states (0.35 the saving pass, 0.9 the pass
// back), against 0.07 ms for the bytes alone; 1.34 ms in fp32.
#include "kda_ssm.cuh"

namespace kda {

namespace {

struct BwdParts {
  float* states;   // [piece ids of 8 tokens][D][S]
  float* bc;       // [channel block][token][2][S]
  float* small;    // [segment id][D (S + 2)]: dA, dskip, dbias of a segment
  SsmSplit split;  // the segments; ends and steps of the backward's first pass
};

template <int L>
struct BwdShared {
  static constexpr int TILE = tile_of(L), CH = kSsmThreads / L, SW = L * kSsmStates;
  static constexpr int YP = CH + 8;
  static constexpr int WARPS = kSsmThreads / 32;
  // one buffer of the warps' sums where two would not fit (S > 64); the tile
  // then waits for the helpers to have read the last one's
  static constexpr int PARTS = L == 32 ? 1 : 2;
  float2 dt[2][TILE][CH];              // step, step * u
  float dy[2][TILE][CH];
  float b[2][TILE][SW], c[2][TILE][SW];
  float fed[2][TILE][YP], qa[2][TILE][YP];
  float part[PARTS][WARPS][TILE][2][SW];  // a warp's dB and dC
  float4 state[2][TILE / kSsmChunk][kSsmThreads];
};

// Like the forward's CTA (see kda_ssm.cu): 4 warps run the recurrence, here
// tile by tile from the end, 4 helper warps turn the next tile into step, step
// * u, dy, B and C and finish the previous one.  A recurrence thread's start
// states of a tile's chunks come by asynchronous copies of its own, a tile
// ahead.
//
// Per chunk of 8 tokens a thread runs its 4 states forward, keeping them and
// their decays in registers, and then back.  dB and dC are summed over the
// warp's channels by exchanges: 8 values a token in 7 of them.  (Products with
// a row of ones on the tensor cores, mma.sync in tf32, take fewer instructions
// but were slower, 1.39 against 1.23 ms for 2 x 4096 tokens of 4096 channels
// at the time, and less exact.)  No unit is full (issue slots 48 % used, shared
// memory 45, FMA pipe 32, special function unit 20): what bounds the kernel is
// latency at the 16 warps an SM that 128 registers leave, and the barrier a tile
// that ties the recurrence to its helpers, the largest stall.  At those 128
// registers every variant spills, 4 to 100 bytes a thread in bf16 and up to 232
// in fp32.
//
// ENDS: a split scan's first pass backward (see SsmSplit): each segment's
// gradient into its start state from none at its end, and its sum of steps.
template <typename IO, int L, bool VEC, bool ENDS>
__global__ void __launch_bounds__(kSsmThreads + kHelpers, 2)
    ssm_bwd_kernel(SsmBwdArgs b, BwdParts part) {
  using Shared = BwdShared<L>;
  constexpr int CH = Shared::CH, SW = Shared::SW, kTile = Shared::TILE, K = kSsmChunk;
  constexpr int WARPS = Shared::WARPS, PARTS = Shared::PARTS, CHUNKS = kTile / K;
  constexpr int E = kTile * CH / kHelpers;   // (token, channel) pairs a helper
  constexpr int BN = kTile * SW / kHelpers;  // values of B (and of C) a helper
  constexpr int TPT = kHelpers / kTile;      // helpers a token (VEC)
  constexpr int TSTEP = kHelpers / CH;       // tokens between two of a helper's (not VEC)
  extern __shared__ __align__(16) unsigned char s_raw[];
  Shared& sh = *reinterpret_cast<Shared*>(s_raw);
  const SsmArgs& a = b.f;
  const int tid = threadIdx.x;
  const int n_blk = ssm_blocks(a, CH), block = blockIdx.x % n_blk;
  const int64_t id = blockIdx.x / n_blk;
  const SsmBlock blk(a, CH, block);
  float* small = part.small + id * a.D * (a.S + 2);  // of this segment
  const SsmSplit& split = part.split;
  const bool cut = split.seg != INT32_MAX;
  int seq, piece, seq_start, seq_end;
  if (!ssm_piece(a, split.seg, id, &seq, &piece, &seq_start, &seq_end)) {
    if (!ENDS) {  // an id without a segment adds nothing to the sums
      for (int i = tid; i < blk.n * a.S; i += kSsmThreads + kHelpers)
        small[(int64_t)blk.c0 * a.S + i] = 0.f;
      for (int i = tid; i < 2 * blk.n; i += kSsmThreads + kHelpers)
        small[(int64_t)a.D * (a.S + i / blk.n) + blk.c0 + i % blk.n] = 0.f;
    }
    return;
  }
  if (ENDS && piece == 0) return;  // nothing lies before it
  const int start = seq_start + piece * (cut ? split.seg : 0);
  const int end = min(seq_end, (int)min((int64_t)start + split.seg, (int64_t)INT32_MAX));
  const int tiles = (end - start + kTile - 1) / kTile;
  auto slot = [](int t, int c) {  // see the forward kernel
    if (L != 4) return c;
    const int p = c >> 1, o = p >> 2;
    return ((o << 2 | ((p ^ o ^ t) & 1) | ((p ^ o) & 2)) << 1) | (c & 1);
  };

  if (tid >= kSsmThreads) {
    const int hid = tid - kSsmThreads;
    const IO* u = static_cast<const IO*>(a.u) + blk.c0;
    const IO* delta = static_cast<const IO*>(a.delta) + blk.c0;
    const IO* z = a.z ? static_cast<const IO*>(a.z) + blk.c0 : nullptr;
    const IO* dout = static_cast<const IO*>(b.d_out) + blk.c0;
    const IO* B = static_cast<const IO*>(a.B) + (int64_t)blk.g * a.b_group;
    const IO* C = static_cast<const IO*>(a.C) + (int64_t)blk.g * a.c_group;
    IO* du = static_cast<IO*>(b.du) + blk.c0;
    IO* ddelta = static_cast<IO*>(b.ddelta) + blk.c0;
    const bool bc_vec = a.S % BN == 0 && a.b_stride % BN == 0 && a.c_stride % BN == 0 &&
                        a.b_group % BN == 0 && a.c_group % BN == 0 &&
                        (reinterpret_cast<uintptr_t>(a.B) | reinterpret_cast<uintptr_t>(a.C)) %
                                Held<IO, BN, true>::ALIGN == 0;
    auto tok_of = [&](int j) { return VEC ? hid / TPT : (j * kHelpers + hid) / CH; };
    auto ch_of = [&](int j) { return VEC ? hid % TPT * E + j : (j * kHelpers + hid) % CH; };
    const int bt = hid / TPT, bn = hid % TPT * BN;
    constexpr int EC = VEC ? E : 1;  // channels a helper finishes
    float bias[EC], skip[EC], dskip[EC], dbias[EC];
#pragma unroll
    for (int j = 0; j < EC; ++j) {
      const int c = ch_of(j);
      bias[j] = a.bias && c < blk.n ? a.bias[blk.c0 + c] : 0.f;
      skip[j] = a.skip && c < blk.n ? a.skip[blk.c0 + c] : 0.f;
      dskip[j] = dbias[j] = 0.f;
    }
    constexpr bool ONE = sizeof(IO) == 4;
    struct Keep {  // what finish() needs of a tile
      Held<IO, E, VEC> u, d;
    } keep[2];
    Held<IO, E, VEC> ru, rd, rz, ro;
    Held<IO, BN, true> rb, rc;   // bc_vec, and fp32 either way
    Held<IO, BN, false> sb, sc;  // bf16 otherwise
    auto load_e = [&](const IO* p, int64_t stride, int t0, int m, Held<IO, E, VEC>& r) {
      r.clear();
      if (VEC) {
        if (tok_of(0) < m && ch_of(0) < blk.n)
          r.all(p + (t0 + tok_of(0)) * stride + ch_of(0));
      } else {
        const IO* q = p + (t0 + tok_of(0)) * stride + ch_of(0);
        const int left = ch_of(0) < blk.n ? m - tok_of(0) : 0;
#pragma unroll
        for (int j = 0; j < E; ++j)
          if (j * TSTEP < left) r.one(j, q + j * (TSTEP * stride));
      }
    };
    auto load_bc = [&](const IO* p, int64_t stride, int t0, int m, Held<IO, BN, true>& r,
                       Held<IO, BN, false>& s) {
      const IO* q = p + (int64_t)(t0 + bt) * stride + bn;
      if (bc_vec) {
        r.clear();
        if (bt < m && bn < a.S) r.all(q);
      } else {
        if (ONE)
          r.clear();
        else
          s.clear();
#pragma unroll
        for (int j = 0; j < BN; ++j)
          if (bt < m && bn + j < a.S) {
            if (ONE)
              r.one(j, q + j);
            else
              s.one(j, q + j);
          }
      }
    };
    auto load = [&](int i) {
      const int t0 = start + i * kTile, m = min(kTile, end - t0);
      load_e(delta, a.delta_stride, t0, m, rd);
      if (!ENDS) load_e(u, a.u_stride, t0, m, ru);
      load_e(dout, a.D, t0, m, ro);
      if (z) load_e(z, a.z_stride, t0, m, rz);
      if (!ENDS) load_bc(B, a.b_stride, t0, m, rb, sb);
      load_bc(C, a.c_stride, t0, m, rc, sc);
    };
    auto convert = [&](int i, int w, Keep& k) {
      const int t0 = start + i * kTile, m = min(kTile, end - t0);
      float dt[E], dtu[E], dy[E];
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float raw = rd.get(j) + bias[VEC ? j : 0];
        const bool real = tok_of(j) < m && ch_of(j) < blk.n;
        dt[j] = real ? (a.softplus ? softplus_f<IO>(raw) : raw) : 0.f;
        dtu[j] = ENDS ? 0.f : dt[j] * ru.get(j);
        dy[j] = ro.get(j);
        if (z) {
          const float g = rz.get(j);
          dy[j] *= g * sigmoid_f(g);
        }
      }
      if (!ENDS) {
        k.u = ru;
        k.d = rd;
      }
      if (VEC && E >= 2) {
#pragma unroll
        for (int j = 0; j < E; j += 2)
          *reinterpret_cast<float4*>(&sh.dt[w][tok_of(0)][slot(tok_of(0), ch_of(j))]) =
              make_float4(dt[j], dtu[j], dt[j + 1], dtu[j + 1]);
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j)
          sh.dt[w][tok_of(j)][slot(tok_of(j), ch_of(j))] = make_float2(dt[j], dtu[j]);
      }
      if (VEC) {
        store_floats<E>(&sh.dy[w][tok_of(0)][ch_of(0)], dy);
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j) sh.dy[w][tok_of(j)][ch_of(j)] = dy[j];
      }
      float vb[BN], vc[BN];
#pragma unroll
      for (int j = 0; j < BN; ++j) {
        if (!ENDS) vb[j] = ONE || bc_vec ? rb.get(j) : sb.get(j);
        vc[j] = ONE || bc_vec ? rc.get(j) : sc.get(j);
      }
      if (!ENDS) store_floats<BN>(&sh.b[w][bt][bn], vb);
      store_floats<BN>(&sh.c[w][bt][bn], vc);
    };
    // reads only this thread's own elements of dt and dy, before convert()
    // writes them again
    auto finish = [&](int i, int w, const Keep& k) {
      const int t0 = start + i * kTile, m = min(kTile, end - t0);
      float ru_[E], rd_[E];
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const int t = tok_of(j), c = ch_of(j);
        const float uu = k.u.get(j), raw = k.d.get(j) + bias[VEC ? j : 0];
        const float f = sh.fed[w][t][c], dy = sh.dy[w][t][c];
        float dd = fmaf(f, uu, kLn2 * sh.qa[w][t][c]);
        if (a.softplus) dd *= sigmoid_f(raw);
        if (t < m && c < blk.n) {
          dskip[VEC ? j : 0] = fmaf(dy, uu, dskip[VEC ? j : 0]);
          dbias[VEC ? j : 0] += dd;
        }
        ru_[j] = fmaf(f, sh.dt[w][t][slot(t, c)].x, dy * skip[VEC ? j : 0]);
        rd_[j] = dd;
      }
      if (VEC) {
        if (tok_of(0) < m && ch_of(0) < blk.n) {
          const int64_t at = (int64_t)(t0 + tok_of(0)) * a.D + ch_of(0);
          store_vec<IO, E>(du + at, ru_);
          store_vec<IO, E>(ddelta + at, rd_);
        }
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j)
          if (tok_of(j) < m && ch_of(j) < blk.n) {
            const int64_t at = (int64_t)(t0 + tok_of(j)) * a.D + ch_of(j);
            du[at] = from_f32<IO>(ru_[j]);
            ddelta[at] = from_f32<IO>(rd_[j]);
          }
      }
      // the warps' dB and dC
      float* to = part.bc + ((int64_t)block * a.tokens + t0) * 2 * a.S;
      if (a.S == SW) {
        for (int e = hid * 4; e < m * 2 * SW; e += kHelpers * 4) {
          float4 s = *reinterpret_cast<const float4*>(&sh.part[w % PARTS][0][0][0][0] + e);
#pragma unroll
          for (int q = 1; q < WARPS; ++q) {
            const float4 v = *reinterpret_cast<const float4*>(&sh.part[w % PARTS][q][0][0][0] + e);
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
          }
          *reinterpret_cast<float4*>(to + e) = s;
        }
      } else {
        for (int e = hid; e < m * 2 * SW; e += kHelpers) {
          const int n = e % SW;
          if (n >= a.S) continue;
          float s = 0.f;
#pragma unroll
          for (int q = 0; q < WARPS; ++q) s += (&sh.part[w % PARTS][q][0][0][0])[e];
          to[e / SW * a.S + n] = s;
        }
      }
    };
    if (tiles > 0) {
      load(tiles - 1);
      convert(tiles - 1, 0, keep[0]);
      if (tiles > 1) load(tiles - 2);
    }
    __syncthreads();
    for (int n = 0; n < tiles; n += 2) {  // tile tiles - 1 - n - k in buffer k
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = tiles - 1 - n - k;
        if (i < 0) break;
        if (!ENDS && n + k > 0) finish(i + 1, 1 - k, keep[1 - k]);
        if (PARTS == 1) __syncthreads();
        if (i > 0) {
          convert(i - 1, 1 - k, keep[1 - k]);
          if (i > 1) load(i - 2);
        }
        __syncthreads();
      }
    }
    if (ENDS) return;
    if (tiles > 0) {
      if (tiles & 1)
        finish(0, 0, keep[0]);
      else
        finish(0, 1, keep[1]);
    }
    // sums over the helpers of one channel, in the order of the helpers
    float* s_sum = &sh.dt[0][0][0].x;  // [2][kHelpers][EC]
    asm volatile("bar.sync 1, %0;" ::"n"(kHelpers) : "memory");
#pragma unroll
    for (int j = 0; j < EC; ++j) {
      s_sum[hid * EC + j] = dskip[j];
      s_sum[(kHelpers + hid) * EC + j] = dbias[j];
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kHelpers) : "memory");
    for (int c = hid; c < blk.n; c += kHelpers) {
      float x = 0.f, y = 0.f;
      const int first = VEC ? c / E : c, step = VEC ? TPT : CH, j = VEC ? c % E : 0;
      for (int h = first; h < kHelpers; h += step) {
        x += s_sum[h * EC + j];
        y += s_sum[(kHelpers + h) * EC + j];
      }
      small[(int64_t)a.D * a.S + blk.c0 + c] = x;
      small[(int64_t)a.D * (a.S + 1) + blk.c0 + c] = y;
    }
    return;
  }

  constexpr int CW = 32 / L;  // channels a warp, in the low lane bits
  const int warp = tid / 32, lane = tid % 32, l = lane / CW, ch = warp * CW + lane % CW;
  const bool on = ch < blk.n;
  const int d = blk.c0 + (on ? ch : 0), n0 = l * kSsmStates;
  const int slot0 = slot(0, ch), slot1 = slot(1, ch);
  const bool st_vec = a.S % 4 == 0;
  float A2[kSsmStates], g0[kSsmStates];
#pragma unroll
  for (int i = 0; i < kSsmStates; ++i) {
    const bool real = on && n0 + i < a.S;
    A2[i] = real ? a.A[(int64_t)d * a.S + n0 + i] * kLog2e : 0.f;
    g0[i] = real && b.d_final && !ENDS ? b.d_final[((int64_t)seq * a.D + d) * a.S + n0 + i] : 0.f;
  }
  if (cut && !ENDS) {  // through the segments behind this one
    const int n = (int)(((int64_t)seq_end - seq_start + split.seg - 1) / split.seg);
    for (int k = n - 1; k > piece; --k) {
      const int64_t row = (id - piece + k) * a.D + d;
      const float sum = split.steps[row];
#pragma unroll
      for (int i = 0; i < kSsmStates; ++i)
        if (on && n0 + i < a.S)
          g0[i] = segment_join(ex2_f(sum * A2[i]), g0[i], split.ends[row * a.S + n0 + i]);
    }
  }
  const f32x2 A01 = pack2(A2[0], A2[1]), A23 = pack2(A2[2], A2[3]);
  f32x2 dh01 = pack2(g0[0], g0[1]), dh23 = pack2(g0[2], g0[3]);
  f32x2 dA01 = both(0.f), dA23 = both(0.f);
  float steps = 0.f;
  auto fetch = [&](int i, int w) {  // the start states of tile i's chunks
    if (ENDS || !st_vec || !on || n0 >= a.S) return;
    const int t0 = i * kTile, m = min(kTile, end - start - t0);
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
      if (c * K < m) {
        const float* p = part.states +
                         (ssm_piece_id(seq, seq_start, K, (start - seq_start + t0) / K + c) * a.D + d) *
                             a.S + n0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::
                     "r"((unsigned)__cvta_generic_to_shared(&sh.state[w][c][tid])), "l"(p)
                     : "memory");
      }
  };
  if (tiles > 0) fetch(tiles - 1, 0);
  asm volatile("cp.async.commit_group;" ::: "memory");
  __syncthreads();
  for (int n = 0; n < tiles; ++n) {
    const int i = tiles - 1 - n, w = n & 1, m = min(kTile, end - start - i * kTile);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (i > 0) fetch(i - 1, w ^ 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (PARTS == 1) __syncthreads();
    for (int c = (m - 1) / K; c >= 0; --c) {
      const int tc = c * K;
      // the chunk's decay is put right at its end, as in the forward kernel
      const f32x2 g01 = dh01, g23 = dh23;
      f32x2 p01 = both(1.f), p23 = both(1.f);
      float sum = 0.f;
      if constexpr (ENDS) {
#pragma unroll
        for (int t = K - 1; t >= 0; --t) {
          const float dt = sh.dt[w][tc + t][t & 1 ? slot1 : slot0].x;
          const ulonglong2 cv = *reinterpret_cast<const ulonglong2*>(&sh.c[w][tc + t][n0]);
          const f32x2 dy = both(sh.dy[w][tc + t][ch]);
          float p[4];
          unpack2(mul2(both(dt), A01), p[0], p[1]);
          unpack2(mul2(both(dt), A23), p[2], p[3]);
          const f32x2 e01 = pack2(ex2_f(p[0]), ex2_f(p[1])), e23 = pack2(ex2_f(p[2]), ex2_f(p[3]));
          dh01 = mul2(fma2(dy, cv.x, dh01), e01);
          dh23 = mul2(fma2(dy, cv.y, dh23), e23);
          p01 = mul2(p01, e01);
          p23 = mul2(p23, e23);
          sum += dt;
        }
        steps += sum;
        chunk_decay(sum, A01, A23, p01, p23);
        chunk_add(p01, g01, dh01);
        chunk_add(p23, g23, dh23);
        continue;
      }
      f32x2 h01[K + 1], h23[K + 1], e01[K], e23[K];
      if (st_vec) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (on && n0 < a.S) v = sh.state[w][c][tid];
        h01[0] = pack2(v.x, v.y);
        h23[0] = pack2(v.z, v.w);
      } else {
        const float* p =
            part.states +
            (ssm_piece_id(seq, seq_start, K, (start - seq_start) / K + i * CHUNKS + c) * a.D + d) *
                a.S + n0;
        float v[kSsmStates];
#pragma unroll
        for (int k = 0; k < kSsmStates; ++k) v[k] = on && n0 + k < a.S ? p[k] : 0.f;
        h01[0] = pack2(v[0], v[1]);
        h23[0] = pack2(v[2], v[3]);
      }
#pragma unroll
      for (int t = 0; t < K; ++t) {
        const float2 v = sh.dt[w][tc + t][t & 1 ? slot1 : slot0];
        const ulonglong2 bv = *reinterpret_cast<const ulonglong2*>(&sh.b[w][tc + t][n0]);
        const f32x2 dt = both(v.x), dtu = both(v.y);
        float p[4];
        unpack2(mul2(dt, A01), p[0], p[1]);
        unpack2(mul2(dt, A23), p[2], p[3]);
        e01[t] = pack2(ex2_f(p[0]), ex2_f(p[1]));
        e23[t] = pack2(ex2_f(p[2]), ex2_f(p[3]));
        h01[t + 1] = fma2(e01[t], h01[t], mul2(dtu, bv.x));
        h23[t + 1] = fma2(e23[t], h23[t], mul2(dtu, bv.y));
        p01 = mul2(p01, e01[t]);
        p23 = mul2(p23, e23[t]);
        sum += v.x;
      }
      f32x2 s01 = both(0.f), s23 = both(0.f);  // dA of the chunk
      float fed[4], qa[4];
#pragma unroll
      for (int t = K - 1; t >= 0; --t) {
        const float2 v = sh.dt[w][tc + t][t & 1 ? slot1 : slot0];
        const ulonglong2 bv = *reinterpret_cast<const ulonglong2*>(&sh.b[w][tc + t][n0]);
        const ulonglong2 cv = *reinterpret_cast<const ulonglong2*>(&sh.c[w][tc + t][n0]);
        const f32x2 dy = both(sh.dy[w][tc + t][ch]), dt = both(v.x), dtu = both(v.y);
        dh01 = fma2(dy, cv.x, dh01);
        dh23 = fma2(dy, cv.y, dh23);
        float bc[8];
        unpack2(mul2(dh01, dtu), bc[0], bc[1]);
        unpack2(mul2(dh23, dtu), bc[2], bc[3]);
        unpack2(mul2(dy, h01[t + 1]), bc[4], bc[5]);
        unpack2(mul2(dy, h23[t + 1]), bc[6], bc[7]);
        fed[t & 3] = sum2(fma2(dh01, bv.x, mul2(dh23, bv.y)));
        dh01 = mul2(dh01, e01[t]);
        dh23 = mul2(dh23, e23[t]);
        const f32x2 q01 = mul2(dh01, h01[t]), q23 = mul2(dh23, h23[t]);
        qa[t & 3] = sum2(fma2(q01, A01, mul2(q23, A23)));
        s01 = fma2(q01, dt, s01);
        s23 = fma2(q23, dt, s23);
        {
          int f = 0;
          SpreadSum<8, 1, CW>::run(bc, lane, f);
          constexpr int LEFT = 8 / CW > 1 ? 8 / CW : 1;
#pragma unroll
          for (int k = 0; k < LEFT; ++k)
            sh.part[w % PARTS][warp][tc + t][(f + k) / 4][n0 + (f + k) % 4] = bc[k];
        }
        if ((t & 3) == 0) {  // four tokens' sums over the state groups
          int f = 0, f2 = 0;
          SpreadSum<4, CW, 32>::run(fed, lane, f);
          SpreadSum<4, CW, 32>::run(qa, lane, f2);
          constexpr int LEFT = L >= 4 ? 1 : 4 / L;
          if (l < 4)
#pragma unroll
            for (int k = 0; k < LEFT; ++k) {
              sh.fed[w][tc + t + f + k][ch] = fed[k];
              sh.qa[w][tc + t + f + k][ch] = qa[k];
            }
        }
      }
      dA01 = add2(dA01, s01);
      dA23 = add2(dA23, s23);
      chunk_decay(sum, A01, A23, p01, p23);
      chunk_add(p01, g01, dh01);
      chunk_add(p23, g23, dh23);
    }
    __syncthreads();
  }
  float dA[kSsmStates], dh[kSsmStates];
  unpack2(dA01, dA[0], dA[1]);
  unpack2(dA23, dA[2], dA[3]);
  unpack2(dh01, dh[0], dh[1]);
  unpack2(dh23, dh[2], dh[3]);
#pragma unroll
  for (int k = 0; k < kSsmStates; ++k) {
    if (!on || n0 + k >= a.S) continue;
    if (ENDS) {
      split.ends[(id * a.D + d) * a.S + n0 + k] = dh[k];
      continue;
    }
    small[(int64_t)d * a.S + n0 + k] = dA[k];
    if (b.dh0 && piece == 0) b.dh0[((int64_t)seq * a.D + d) * a.S + n0 + k] = dh[k];
  }
  if (ENDS && on && l == 0) split.steps[id * a.D + d] = steps;
}

// dB and dC of a token's group: the channel blocks' parts, N values a thread.
template <typename IO, int N>
__global__ void __launch_bounds__(256)
    ssm_bc_sum_kernel(SsmBwdArgs b, const float* __restrict__ bc, int blocks_per_group) {
  const SsmArgs& a = b.f;
  const int per = 2 * a.S / N;  // threads a token and group
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, tg = id / per;
  const int e = (int)(id - tg * per) * N;
  const int64_t tok = tg / a.G;
  const int g = (int)(tg - tok * a.G);
  if (tok >= a.tokens) return;
  SeqCursor q;
  if (!find_seq(a.cu, a.n_seqs, a.T, (int)tok, &q) || tok < q.start) return;
  const int64_t step = a.tokens * 2 * a.S;
  const float* p = bc + g * blocks_per_group * step + tok * 2 * a.S + e;
  float s[N] = {};
#pragma unroll 8
  for (int i = 0; i < blocks_per_group; ++i) {
    float v[N];
    load_vec<float, N>(p + i * step, v);
#pragma unroll
    for (int j = 0; j < N; ++j) s[j] += v[j];
  }
  IO* out = static_cast<IO*>(e < a.S ? b.dB : b.dC) + (tok * a.G + g) * a.S + e % a.S;
#pragma unroll
  for (int j = 0; j < N; ++j) out[j] = from_f32<IO>(s[j]);
}

// dA, dskip and dbias: the segments' parts, 8 rows of threads and then their
// sums in order.
__global__ void ssm_small_sum_kernel(const float* __restrict__ part, int64_t ids, int D, int S,
                                     float* __restrict__ dA, float* __restrict__ dskip,
                                     float* __restrict__ dbias) {
  __shared__ float s[8][32];
  const int64_t n = (int64_t)D * (S + 2), i = (int64_t)blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (i < n)
    for (int64_t k = threadIdx.y; k < ids; k += 8) v += part[k * n + i];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y || i >= n) return;
  for (int k = 1; k < 8; ++k) v += s[k][threadIdx.x];
  const int64_t m = (int64_t)D * S;
  if (i < m)
    dA[i] = v;
  else if (i < m + D) {
    if (dskip) dskip[i - m] = v;
  } else if (dbias) {
    dbias[i - m - D] = v;
  }
}

size_t up(size_t x) { return (x + 255) & ~(size_t)255; }

// A backward's segments: its passes over the recurrence cost about three times
// a split's, so two segments a sequence are worth it.
int bwd_segment(const SsmBwdArgs& b, int sms) { return ssm_segment(b.f, sms, 2.0); }
int64_t bwd_ids(const SsmArgs& a, int seg) {
  return seg == INT32_MAX ? a.n_seqs : ssm_segments(a, seg);
}

struct Layout {
  size_t states, bc, small, fwd_ends, bwd_ends, total;
};
Layout layout(const SsmBwdArgs& b, int seg) {
  const SsmArgs& a = b.f;
  const size_t chunks = (size_t)a.tokens / kSsmChunk + a.n_seqs + 1;
  const size_t blocks = ssm_blocks(a, kSsmThreads / ssm_lanes(a.S));
  Layout o;
  o.states = 0;
  o.bc = o.states + up(chunks * a.D * a.S * 4);
  o.small = o.bc + up(blocks * a.tokens * 2 * a.S * 4);
  o.fwd_ends = o.small + up((size_t)bwd_ids(a, seg) * a.D * (a.S + 2) * 4);
  o.bwd_ends = o.fwd_ends + up(ssm_split_bytes(a, seg));
  o.total = o.bwd_ends + up(ssm_split_bytes(a, seg));
  return o;
}

template <typename IO, int E>
bool vec_ok(const SsmBwdArgs& b) {
  const SsmArgs& a = b.f;
  const void* ps[] = {a.u, a.delta, a.z, b.d_out, b.du, b.ddelta};
  for (const void* p : ps)
    if (p && !aligned_to(p, Held<IO, E, true>::ALIGN)) return false;
  return a.D / a.G % E == 0 && a.D % E == 0 && a.u_stride % E == 0 && a.delta_stride % E == 0 &&
         a.z_stride % E == 0;
}

template <typename IO, int L, bool ENDS>
cudaError_t pass_launch(const SsmBwdArgs& b, const BwdParts& part, cudaStream_t st) {
  const unsigned grid =
      (unsigned)(bwd_ids(b.f, part.split.seg) * ssm_blocks(b.f, kSsmThreads / L));
  constexpr int E = tile_of(L) * (kSsmThreads / L) / kHelpers;
  auto* k = vec_ok<IO, E>(b) ? ssm_bwd_kernel<IO, L, true, ENDS>
                             : ssm_bwd_kernel<IO, L, false, ENDS>;
  constexpr int bytes = sizeof(BwdShared<L>);
  static_assert(bytes <= 227 * 1024, "shared memory of an SM");
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  k<<<grid, kSsmThreads + kHelpers, bytes, st>>>(b, part);
  return cudaGetLastError();
}
template <typename IO, int L>
cudaError_t bwd_launch(const SsmBwdArgs& b, const BwdParts& part, cudaStream_t st) {
  if (b.f.n_seqs == 0) return cudaSuccess;
  if (part.split.seg != INT32_MAX) {
    const cudaError_t e = pass_launch<IO, L, true>(b, part, st);
    if (e != cudaSuccess) return e;
  }
  return pass_launch<IO, L, false>(b, part, st);
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
  if (n && b.f.S % 4 == 0)
    ssm_bc_sum_kernel<IO, 4><<<(unsigned)((n / 4 + 255) / 256), 256, 0, st>>>(b, part.bc, per_group);
  else if (n)
    ssm_bc_sum_kernel<IO, 1><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(b, part.bc, per_group);
  return cudaGetLastError();
}

}  // namespace

size_t ssm_bwd_workspace_bytes(const SsmBwdArgs& b, int sms) {
  return layout(b, bwd_segment(b, sms)).total;
}

int ssm_bwd_kernel_count(const SsmBwdArgs& b, int sms) {
  const bool cut = bwd_segment(b, sms) != INT32_MAX;
  return (b.f.n_seqs ? cut ? 4 : 2 : 0) + (b.f.tokens ? 1 : 0) + 1;
}

cudaError_t launch_ssm_bwd(const SsmBwdArgs& b, void* ws, int sms, cudaStream_t st) {
  const int seg = bwd_segment(b, sms);
  const Layout o = layout(b, seg);
  char* w = static_cast<char*>(ws);
  const BwdParts part{reinterpret_cast<float*>(w + o.states), reinterpret_cast<float*>(w + o.bc),
                      reinterpret_cast<float*>(w + o.small),
                      ssm_split_at(b.f, seg, w + o.bwd_ends)};
  const SsmSave save{part.states, b.d_out, b.f.z ? b.dz : nullptr};
  cudaError_t e = launch_ssm_save(b.f, save, ssm_split_at(b.f, seg, w + o.fwd_ends), st);
  if (e == cudaSuccess)
    e = b.f.bf16 ? bwd_pick<__nv_bfloat16>(b, part, st) : bwd_pick<float>(b, part, st);
  if (e != cudaSuccess) return e;
  const int64_t n = (int64_t)b.f.D * (b.f.S + 2);
  ssm_small_sum_kernel<<<(unsigned)((n + 31) / 32), dim3(32, 8), 0, st>>>(
      part.small, bwd_ids(b.f, seg), b.f.D, b.f.S, b.dA, b.dskip, b.dbias);
  return cudaGetLastError();
}

}  // namespace kda

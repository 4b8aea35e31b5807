// Selective state space scan: the forward over prompts, the first pass of the
// backward (which saves states), and the step for new tokens.  The recurrence
// and its split over lanes are in kda_ssm.cuh.
//
// Bound: an update costs one exponential and about 6 flops.  The special
// function unit gives 16 a cycle and SM, so 16 states a channel cost more
// there (0.24 ms for 2 x 8192 tokens of 4096 channels at 1.9 GHz) than the
// 8 bytes a token and channel cost in HBM (0.08 ms).  Measured: 0.50 ms (fp32,
// see EXACT below: 0.58).  Neither is full then: an SM with two CTAs uses 71 %
// of its special function unit and 61 % of its issue slots, 256 CTAs give 40 of
// 148 SMs only one, and the rest is latency at 16 warps an SM.  More than 64
// states in bf16 spill about 550 bytes a thread.
#include "kda_ssm.cuh"

namespace kda {

namespace {

constexpr int kMinSegment = 128;  // tokens: below, a split's passes are all latency

// A CTA's shared memory, two of each: the tile in work and the next.
template <int L, bool WANT_Y>
struct FwdShared {
  static constexpr int TILE = tile_of(L), CH = kSsmThreads / L, SW = L * kSsmStates;
  static constexpr int YP = CH + 8;  // row pitch of y: 4 tokens of 8 channels on 32 banks
  float2 dt[2][TILE][CH];            // step, step * u
  float b[2][TILE][SW];
  float c[2][WANT_Y ? TILE : 1][SW];
  float y[2][WANT_Y ? TILE : 1][YP];
};

// CTA: 4 warps run the recurrence, 4 helper warps feed them and finish their
// results, tile by tile of 32 tokens with one barrier a tile: while the
// recurrence runs tile i, the helpers finish and store tile i - 1, turn tile
// i + 1 (its loads were issued a tile earlier and wait in registers) into
// step, step * u, B and C, and issue the loads of tile i + 2.  A helper thread
// keeps what a token's result needs besides y (skip * u, silu(z)) in
// registers, since it stores the same elements it loaded.
template <typename IO, int L, int MODE, bool VEC>
__global__ void __launch_bounds__(kSsmThreads + kHelpers, 2)
    ssm_fwd_kernel(SsmArgs a, SsmSave save, SsmSplit split) {
  constexpr bool WANT_Y = MODE == kSsmOut || MODE == kSsmSaveDz;
  using Shared = FwdShared<L, WANT_Y>;
  constexpr int CH = Shared::CH, SW = Shared::SW, kTile = Shared::TILE;
  constexpr int E = kTile * CH / kHelpers;   // (token, channel) pairs a helper
  constexpr int BN = kTile * SW / kHelpers;  // values of B (and of C) a helper
  constexpr int TPT = kHelpers / kTile;      // helpers a token (VEC)
  constexpr int TSTEP = kHelpers / CH;       // tokens between two of a helper's (not VEC)
  extern __shared__ __align__(16) unsigned char s_raw[];
  Shared& sh = *reinterpret_cast<Shared*>(s_raw);
  auto& s_dt = sh.dt;
  auto& s_b = sh.b;
  auto& s_c = sh.c;
  auto& s_y = sh.y;
  const int tid = threadIdx.x;
  const int n_blk = ssm_blocks(a, CH);
  const int64_t id = blockIdx.x / n_blk;
  const SsmBlock blk(a, CH, blockIdx.x % n_blk);
  int seq, piece, start, end;
  if (!ssm_piece(a, split.seg, id, &seq, &piece, &start, &end)) return;
  const int first = start + piece * (split.seg < end - start ? split.seg : 0);
  const int last = min(end, (int)min((int64_t)first + split.seg, (int64_t)INT32_MAX));
  const bool cut = split.seg != INT32_MAX;
  // a sequence's last segment has no end to hand on: in its place stands the
  // sequence's start state, read from here by the second pass, which may be
  // writing final states over the initial ones
  const int tiles = MODE == kSsmEnds && last == end ? 0 : (last - first + kTile - 1) / kTile;
  // a pair of channels is 16 bytes; the order of a row's pairs is turned so
  // that 8 helper lanes writing one each never meet on a bank
  auto slot = [](int t, int c) {
    if (L != 4) return c;
    const int p = c >> 1, o = p >> 2;
    return ((o << 2 | ((p ^ o ^ t) & 1) | ((p ^ o) & 2)) << 1) | (c & 1);
  };

  if (tid >= kSsmThreads) {
    const int hid = tid - kSsmThreads;
    const IO* u = static_cast<const IO*>(a.u) + blk.c0;
    const IO* delta = static_cast<const IO*>(a.delta) + blk.c0;
    const IO* z = a.z ? static_cast<const IO*>(a.z) + blk.c0 : nullptr;
    const IO* dout = static_cast<const IO*>(save.d_out) + blk.c0;
    const IO* B = static_cast<const IO*>(a.B) + (int64_t)blk.g * a.b_group;
    const IO* C = static_cast<const IO*>(a.C) + (int64_t)blk.g * a.c_group;
    IO* out = static_cast<IO*>(MODE == kSsmOut ? a.out : save.dz) + blk.c0;
    const bool bc_vec = a.S % BN == 0 && a.b_stride % BN == 0 && a.c_stride % BN == 0 &&
                        a.b_group % BN == 0 && a.c_group % BN == 0 &&
                        (reinterpret_cast<uintptr_t>(a.B) | reinterpret_cast<uintptr_t>(a.C)) %
                                Held<IO, BN, true>::ALIGN == 0;
    // element j of this thread in a tile: VEC E neighbouring channels of one
    // token, else one channel (or few) of E tokens
    auto tok_of = [&](int j) { return VEC ? hid / TPT : (j * kHelpers + hid) / CH; };
    auto ch_of = [&](int j) { return VEC ? hid % TPT * E + j : (j * kHelpers + hid) % CH; };
    const int bt = hid / TPT, bn = hid % TPT * BN;
    float bias[VEC ? E : 1], skip[VEC ? E : 1];
#pragma unroll
    for (int j = 0; j < (VEC ? E : 1); ++j) {
      const int c = ch_of(j);
      bias[j] = a.bias && c < blk.n ? a.bias[blk.c0 + c] : 0.f;
      skip[j] = a.skip && c < blk.n ? a.skip[blk.c0 + c] : 0.f;
    }
    struct Set {  // a tile's values on their way
      Held<IO, E, VEC> u, d, z, o;
      Held<IO, BN, true> b, c;     // bc_vec, and fp32 either way
      Held<IO, BN, false> b1, c1;  // bf16 otherwise
    } set;
    constexpr bool ONE = sizeof(IO) == 4;
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
    auto load = [&](int i, Set& r) {
      const int t0 = first + i * kTile, m = min(kTile, last - t0);
      load_e(delta, a.delta_stride, t0, m, r.d);
      load_e(u, a.u_stride, t0, m, r.u);
      load_bc(B, a.b_stride, t0, m, r.b, r.b1);
      if (WANT_Y) {
        load_bc(C, a.c_stride, t0, m, r.c, r.c1);
        if (z) load_e(z, a.z_stride, t0, m, r.z);
      }
      if (MODE == kSsmSaveDz) load_e(dout, a.D, t0, m, r.o);
    };
    // what turns y into the result: (y + add) * mul, of the tile being
    // converted and of the one before
    float add[2][E], mul[2][E];
    auto convert = [&](int i, const Set& r, float (&add_)[E], float (&mul_)[E]) {
      const int t0 = first + i * kTile, m = min(kTile, last - t0), w = i & 1;
      float dt[E], dtu[E];
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float raw = r.d.get(j) + bias[VEC ? j : 0], uu = r.u.get(j);
        const bool real = tok_of(j) < m && ch_of(j) < blk.n;
        dt[j] = real ? (a.softplus ? softplus_f<IO>(raw) : raw) : 0.f;
        dtu[j] = dt[j] * uu;
        if (WANT_Y) {
          add_[j] = skip[VEC ? j : 0] * uu;
          float k = 1.f;
          if (z) {
            const float g = r.z.get(j), s = sigmoid_f(g);
            k = MODE == kSsmOut ? g * s : r.o.get(j) * silu_grad(g, s);
          }
          mul_[j] = k;
        }
      }
      if (VEC && E >= 2) {
#pragma unroll
        for (int j = 0; j < E; j += 2)
          *reinterpret_cast<float4*>(&s_dt[w][tok_of(0)][slot(tok_of(0), ch_of(j))]) =
              make_float4(dt[j], dtu[j], dt[j + 1], dtu[j + 1]);
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j)
          s_dt[w][tok_of(j)][slot(tok_of(j), ch_of(j))] = make_float2(dt[j], dtu[j]);
      }
      float v[BN];
#pragma unroll
      for (int j = 0; j < BN; ++j) v[j] = ONE || bc_vec ? r.b.get(j) : r.b1.get(j);
      store_floats<BN>(&s_b[w][bt][bn], v);
      if (WANT_Y) {
#pragma unroll
        for (int j = 0; j < BN; ++j) v[j] = ONE || bc_vec ? r.c.get(j) : r.c1.get(j);
        store_floats<BN>(&s_c[w][bt][bn], v);
      }
    };
    auto finish = [&](int i, const float (&add_)[E], const float (&mul_)[E]) {
      const int t0 = first + i * kTile, m = min(kTile, last - t0), w = i & 1;
      if (VEC) {
        const int t = tok_of(0), c = ch_of(0);
        if (t < m && c < blk.n) {
          float r[E];
#pragma unroll
          for (int j = 0; j < E; ++j) r[j] = (s_y[w][t][c + j] + add_[j]) * mul_[j];
          store_vec<IO, E>(out + (int64_t)(t0 + t) * a.D + c, r);
        }
      } else {
        const int c = ch_of(0), left = c < blk.n ? m - tok_of(0) : 0;
        IO* q = out + (int64_t)(t0 + tok_of(0)) * a.D + c;
#pragma unroll
        for (int j = 0; j < E; ++j)
          if (j * TSTEP < left)
            q[j * (TSTEP * (int64_t)a.D)] =
                from_f32<IO>((s_y[w][tok_of(j)][c] + add_[j]) * mul_[j]);
      }
    };
    if (tiles > 0) {
      load(0, set);
      convert(0, set, add[0], mul[0]);
      if (tiles > 1) load(1, set);
    }
    __syncthreads();
    for (int i = 0; i < tiles; i += 2) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // tile i + k: parity k
        if (i + k >= tiles) break;
        if (WANT_Y && i + k > 0) finish(i + k - 1, add[1 - k], mul[1 - k]);
        if (i + k + 1 < tiles) {
          convert(i + k + 1, set, add[1 - k], mul[1 - k]);
          if (i + k + 2 < tiles) load(i + k + 2, set);
        }
        __syncthreads();
      }
    }
    if (WANT_Y && tiles > 0) {
      if (tiles & 1)
        finish(tiles - 1, add[0], mul[0]);
      else
        finish(tiles - 1, add[1], mul[1]);
    }
    return;
  }

  // a warp's channels in the low lane bits, the groups of 4 states in the high
  // ones: neighbouring lanes then share the words of B and C, which a 16-byte
  // shared load serves in two wavefronts (four the other way round)
  constexpr int CW = 32 / L;  // channels a warp
  const int lane = tid % 32, l = lane / CW, ch = tid / 32 * CW + lane % CW;
  const bool on = ch < blk.n;
  const int d = blk.c0 + (on ? ch : 0), n0 = l * kSsmStates;
  float A2[kSsmStates], h[kSsmStates];
#pragma unroll
  for (int i = 0; i < kSsmStates; ++i) {
    const bool real = on && n0 + i < a.S;
    A2[i] = real ? a.A[(int64_t)d * a.S + n0 + i] * kLog2e : 0.f;
    h[i] = real && a.h0 && (!cut || (MODE == kSsmEnds && last == end))
               ? a.h0[((int64_t)seq * a.D + d) * a.S + n0 + i] : 0.f;
  }
  if (cut && MODE != kSsmEnds) {  // the start state and the segments before this one
    const int64_t n = max((int64_t)1, ((int64_t)(end - start) + split.seg - 1) / split.seg);
#pragma unroll
    for (int i = 0; i < kSsmStates; ++i)
      if (n0 + i < a.S) h[i] = split.ends[((id - piece + n - 1) * a.D + d) * a.S + n0 + i];
    for (int k = 0; k < piece; ++k) {
      const int64_t row = (id - piece + k) * a.D + d;
      const float sum = split.steps[row];
#pragma unroll
      for (int i = 0; i < kSsmStates; ++i)
        if (n0 + i < a.S)
          h[i] = segment_join(ex2_f(sum * A2[i]), h[i], split.ends[row * a.S + n0 + i]);
    }
    if (!on)
#pragma unroll
      for (int i = 0; i < kSsmStates; ++i) h[i] = 0.f;
  }
  f32x2 h01 = pack2(h[0], h[1]), h23 = pack2(h[2], h[3]);
  const f32x2 A01 = pack2(A2[0], A2[1]), A23 = pack2(A2[2], A2[3]);
  float steps = 0.f;
  const int slot0 = slot(0, ch), slot1 = slot(1, ch);
  __syncthreads();
  for (int i = 0; i < tiles; ++i) {
    const int t0 = first + i * kTile, m = min(kTile, last - t0), w = i & 1;
    // Four tokens at a time: their decays and inputs, one step ahead of the
    // recurrence through the four before, in one straight run of the tile, so
    // that exponentials and the rest alternate (a loop over 8 tokens: 0.54 ms
    // against 0.50 for 2 x 8192 tokens of 4096 channels).  A polynomial in
    // place of every eighth or fourth exponential frees the special function
    // unit but is slower (0.51, 0.53 ms): the instructions it takes cost more than
    // the unit's share that it frees.
    f32x2 e01[2][4], e23[2][4], x01[2][4], x23[2][4];
    // A chunk's decay is put right at its end: the rounding of 8 exponentials,
    // which would add up over a state's memory, gives way to that of one of the
    // 8 steps' sum.  Without it in bf16 prompts alone: a bf16 step is itself off
    // by 2^-9 of its value, so its decay by 2^-9 of its exponent, where 8
    // exponentials' rounding is 2^-19 at most; the correction costs 8 % there
    // (541 against 499 us, 2 x 8192 x 4096).  In fp32 it takes the state's error
    // from 1.3e-6 to 5e-7 (8 x 1024 tokens, steps of 0.001 to 0.1), below what
    // correctly rounded exponentials leave (2.3e-6), and costs 10 % together with
    // the longer softplus (525 -> 578 us, 2 x 8192 x 4096).
    constexpr bool EXACT = MODE != kSsmOut || sizeof(IO) == 4;
    f32x2 c01, c23, p01, p23;  // the chunk's start state, its product of decays
    float sum4[2], chunk_sum = 0.f;
#pragma unroll
    for (int q = 0; q <= kTile; q += 4) {
      const int next = q / 4 & 1, cur = next ^ 1;
      if (q < kTile) {
        sum4[next] = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // behind the last token: step 0 keeps the state
          const float2 v = s_dt[w][q + j][j & 1 ? slot1 : slot0];
          const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(&s_b[w][q + j][n0]);
          const f32x2 dt = pack2(v.x, v.x), dtu = pack2(v.y, v.y);
          float p[4];
          unpack2(mul2(dt, A01), p[0], p[1]);
          unpack2(mul2(dt, A23), p[2], p[3]);
          e01[next][j] = pack2(ex2_f(p[0]), ex2_f(p[1]));
          e23[next][j] = pack2(ex2_f(p[2]), ex2_f(p[3]));
          x01[next][j] = mul2(dtu, b.x);
          x23[next][j] = mul2(dtu, b.y);
          if (EXACT) sum4[next] += v.x;
        }
      }
      if (q > 0) {
        const int t4 = q - 4;
        if ((MODE == kSsmSave || MODE == kSsmSaveDz) && t4 % kSsmChunk == 0 && t4 < m) {
          float* st = save.states + (ssm_piece_id(seq, start, kSsmChunk,
                                                  (t0 - start + t4) / kSsmChunk) * a.D + d) *
                                        a.S + n0;
          float v[4];
          unpack2(h01, v[0], v[1]);
          unpack2(h23, v[2], v[3]);
          if (a.S % 4 == 0) {
            if (on && n0 < a.S)
              *reinterpret_cast<float4*>(st) = make_float4(v[0], v[1], v[2], v[3]);
          } else {
#pragma unroll
            for (int k = 0; k < kSsmStates; ++k)
              if (on && n0 + k < a.S) st[k] = v[k];
          }
        }
        if (EXACT && t4 % kSsmChunk == 0) {
          c01 = h01;
          c23 = h23;
          p01 = p23 = both(1.f);
          chunk_sum = 0.f;
        }
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h01 = fma2(e01[cur][j], h01, x01[cur][j]);
          h23 = fma2(e23[cur][j], h23, x23[cur][j]);
          if (EXACT) {
            p01 = mul2(p01, e01[cur][j]);
            p23 = mul2(p23, e23[cur][j]);
          }
          if (WANT_Y) {
            const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(&s_c[w][t4 + j][n0]);
            float lo, hi;
            unpack2(fma2(h01, c.x, mul2(h23, c.y)), lo, hi);
            y[j] = lo + hi;
          }
        }
        if (EXACT) {
          chunk_sum += sum4[cur];
          if (t4 % kSsmChunk == kSsmChunk - 4) {
            chunk_decay(chunk_sum, A01, A23, p01, p23);
            chunk_add(p01, c01, h01);
            chunk_add(p23, c23, h23);
            if (MODE == kSsmEnds) steps += chunk_sum;
          }
        }
        if (WANT_Y) {
          int f = 0;
          SpreadSum<4, CW, 32>::run(y, lane, f);
          constexpr int LEFT = L >= 4 ? 1 : 4 / L;
          if (l < 4)
#pragma unroll
            for (int j = 0; j < LEFT; ++j) s_y[w][t4 + f + j][ch] = y[j];
        }
      }
    }
    __syncthreads();
  }
  unpack2(h01, h[0], h[1]);
  unpack2(h23, h[2], h[3]);
  float* fin = nullptr;
  if (MODE == kSsmOut && a.h_out && last == end)
    fin = a.h_out + ((int64_t)seq * a.D + d) * a.S + n0;
  if (MODE == kSsmEnds) {
    fin = split.ends + (id * a.D + d) * a.S + n0;
    if (on && l == 0) split.steps[id * a.D + d] = steps;
  }
  if (fin && on) {
#pragma unroll
    for (int i = 0; i < kSsmStates; ++i)
      if (n0 + i < a.S) fin[i] = h[i];
  }
}

// New tokens: L lanes own a channel and stream the states of NS sequences, read
// and written once per call; A is read once for all of them, and each lane
// forms the step and the result of one of the sequences.  VEC: 4 states of B,
// C and the state are one access each.  Bound by HBM: 32 us for 256 sequences
// of 4096 channels with 16 states, 69 % of a copy's rate.
template <typename IO, int L, int NS, bool VEC>
__global__ void __launch_bounds__(256) ssm_step_kernel(SsmArgs a) {
  constexpr int SL = kSsmStates;
  const int l = threadIdx.x % L, n0 = l * SL;
  const int dd = (blockIdx.x * 256 + threadIdx.x) / L;
  const bool mine = dd < a.D;
  const int d = mine ? dd : 0, g = d / (a.D / a.G);
  float A2[SL];
#pragma unroll
  for (int i = 0; i < SL; ++i)
    A2[i] = mine && n0 + i < a.S ? a.A[(int64_t)d * a.S + n0 + i] * kLog2e : 0.f;
  const float bias = a.bias ? a.bias[d] : 0.f, skip = a.skip ? a.skip[d] : 0.f;
  const IO* B = static_cast<const IO*>(a.B) + g * a.b_group + n0;
  const IO* C = static_cast<const IO*>(a.C) + g * a.c_group + n0;
  const bool lane_on = mine && n0 < a.S;
  // where SpreadSum leaves sequence k's sum
  const int own = NS == 4 ? (l & 1) * 2 + (l >> 1 & 1) : l % NS;
  for (int s0 = blockIdx.y * NS; s0 < a.n_seqs; s0 += gridDim.y * NS) {
    float h[NS][SL];
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      const float* st = a.h_out + ((int64_t)(s0 + k) * a.D + d) * a.S + n0;
      const bool on = lane_on && s0 + k < a.n_seqs;
      if (VEC) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (on) v = __ldcs(reinterpret_cast<const float4*>(st));
        h[k][0] = v.x; h[k][1] = v.y; h[k][2] = v.z; h[k][3] = v.w;
      } else {
#pragma unroll
        for (int i = 0; i < SL; ++i) h[k][i] = on && n0 + i < a.S ? st[i] : 0.f;
      }
    }
    for (int t = 0; t < a.T; ++t) {
      Held<IO, SL, VEC> rb[NS], rc[NS];
#pragma unroll
      for (int k = 0; k < NS; ++k) {
        const int64_t tok = (int64_t)min(s0 + k, a.n_seqs - 1) * a.T + t;
        rb[k].clear();
        rc[k].clear();
        if (VEC) {
          if (n0 < a.S) {
            rb[k].all(B + tok * a.b_stride);
            rc[k].all(C + tok * a.c_stride);
          }
        } else {
#pragma unroll
          for (int i = 0; i < SL; ++i)
            if (n0 + i < a.S) {
              rb[k].one(i, B + tok * a.b_stride + i);
              rc[k].one(i, C + tok * a.c_stride + i);
            }
        }
      }
      // the step and the result of sequence `own` are this lane's
      const int64_t tok = (int64_t)min(s0 + own, a.n_seqs - 1) * a.T + t;
      const float raw = to_f32(static_cast<const IO*>(a.delta)[tok * a.delta_stride + d]) + bias;
      const float uu = to_f32(static_cast<const IO*>(a.u)[tok * a.u_stride + d]);
      const float gz = a.z ? to_f32(static_cast<const IO*>(a.z)[tok * a.z_stride + d]) : 0.f;
      const float dt0 = a.softplus ? softplus_f<IO>(raw) : raw, dtu0 = dt0 * uu;
      float y[NS];
#pragma unroll
      for (int k = 0; k < NS; ++k) {
        const int from = NS == 4 ? (k >> 1) | (k & 1) << 1 : k;  // the lane with own == k
        const float dt = NS == 1 ? dt0 : __shfl_sync(0xffffffffu, dt0, from, L);
        const float dtu = NS == 1 ? dtu0 : __shfl_sync(0xffffffffu, dtu0, from, L);
        y[k] = 0.f;
#pragma unroll
        for (int i = 0; i < SL; ++i) {
          h[k][i] = fmaf(ex2_f(dt * A2[i]), h[k][i], dtu * rb[k].get(i));
          y[k] = fmaf(h[k][i], rc[k].get(i), y[k]);
        }
      }
      int f = 0;
      SpreadSum<NS, 1, L>::run(y, l, f);
      if (mine && l < NS && s0 + own < a.n_seqs) {
        float r = fmaf(skip, uu, y[0]);
        if (a.z) r *= gz * sigmoid_f(gz);
        static_cast<IO*>(a.out)[tok * a.D + d] = from_f32<IO>(r);
      }
    }
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      float* st = a.h_out + ((int64_t)(s0 + k) * a.D + d) * a.S + n0;
      if (!lane_on || s0 + k >= a.n_seqs) continue;
      if (VEC) {
        __stcs(reinterpret_cast<float4*>(st), make_float4(h[k][0], h[k][1], h[k][2], h[k][3]));
      } else {
#pragma unroll
        for (int i = 0; i < SL; ++i)
          if (n0 + i < a.S) st[i] = h[k][i];
      }
    }
  }
}

// Whole vectors of E channels: aligned pointers and strides, and channel
// blocks that start and end on them.
template <typename IO, int E>
bool vec_ok(const SsmArgs& a, const SsmSave& save) {
  const void* ps[] = {a.u, a.delta, a.z, a.out, save.d_out, save.dz};
  for (const void* p : ps)
    if (p && !aligned_to(p, Held<IO, E, true>::ALIGN)) return false;
  return a.D / a.G % E == 0 && a.D % E == 0 && a.u_stride % E == 0 && a.delta_stride % E == 0 &&
         a.z_stride % E == 0;
}

template <typename IO, int L, int MODE>
cudaError_t fwd_launch(const SsmArgs& a, const SsmSave& save, const SsmSplit& split,
                       cudaStream_t st) {
  const int64_t ids = split.seg == INT32_MAX ? a.n_seqs : ssm_segments(a, split.seg);
  const unsigned grid = (unsigned)(ids * ssm_blocks(a, kSsmThreads / L));
  constexpr int E = tile_of(L) * (kSsmThreads / L) / kHelpers;
  auto* k = vec_ok<IO, E>(a, save) ? ssm_fwd_kernel<IO, L, MODE, true>
                                   : ssm_fwd_kernel<IO, L, MODE, false>;
  constexpr int bytes = sizeof(FwdShared<L, MODE == kSsmOut || MODE == kSsmSaveDz>);
  if (bytes > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
  }
  k<<<grid, kSsmThreads + kHelpers, bytes, st>>>(a, save, split);
  return cudaGetLastError();
}

template <typename IO, int MODE>
cudaError_t fwd_pick(const SsmArgs& a, const SsmSave& save, const SsmSplit& split,
                     cudaStream_t st) {
  switch (ssm_lanes(a.S)) {
    case 2: return fwd_launch<IO, 2, MODE>(a, save, split, st);
    case 4: return fwd_launch<IO, 4, MODE>(a, save, split, st);
    case 8: return fwd_launch<IO, 8, MODE>(a, save, split, st);
    case 16: return fwd_launch<IO, 16, MODE>(a, save, split, st);
    case 32: return fwd_launch<IO, 32, MODE>(a, save, split, st);
  }
  return cudaErrorInvalidValue;
}

template <typename IO, int L>
cudaError_t step_launch(const SsmArgs& a, cudaStream_t st) {
  // four sequences a thread (two for two lanes) where that still fills the SMs
  constexpr int NS = L >= 4 ? 4 : 2;
  const bool many = (int64_t)a.n_seqs * a.D * L >= (int64_t)4 * 148 * 2048;
  const int ns = many ? NS : 1;
  const bool vec = a.S % 4 == 0 && a.b_stride % 4 == 0 && a.c_stride % 4 == 0 &&
                   a.b_group % 4 == 0 && a.c_group % 4 == 0 && aligned_to(a.h_out, 16) &&
                   aligned_to(a.B, 4 * sizeof(IO)) && aligned_to(a.C, 4 * sizeof(IO));
  const int64_t groups = (a.n_seqs + ns - 1) / ns;
  const dim3 grid((unsigned)(((int64_t)a.D * L + 255) / 256),
                  (unsigned)(groups < 65535 ? groups : 65535));
  auto* k = many ? (vec ? ssm_step_kernel<IO, L, NS, true> : ssm_step_kernel<IO, L, NS, false>)
                 : (vec ? ssm_step_kernel<IO, L, 1, true> : ssm_step_kernel<IO, L, 1, false>);
  k<<<grid, 256, 0, st>>>(a);
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

// Splitting costs a second pass over the recurrence (without its outputs), so
// it pays where the sequences' own CTAs leave most of the SMs idle: a segment
// is what each of the SMs' CTA slots (two an SM) would get of the whole, and
// sequences are cut where they hold `least` of them, three for the forward.  One sequence of 4096 tokens
// whole and split: 159 and 27 us with 256 channels, 161 and 122 us with 2048;
// with 4096 channels, 2.3 segments, 198 and 230 us.  Packed lengths are not
// known on the host; their longest is taken to be 2.5 times the mean.
int ssm_segment(const SsmArgs& a, int sms, double least) {
  if (a.n_seqs < 1) return INT32_MAX;
  const int64_t blocks = ssm_blocks(a, kSsmThreads / ssm_lanes(a.S)), slots = 2 * (int64_t)sms;
  int64_t seg = (a.tokens * blocks + slots - 1) / slots;
  seg = seg < kMinSegment ? kMinSegment : (seg + 31) / 32 * 32;
  const double longest = (double)a.tokens / a.n_seqs * (a.cu && a.n_seqs > 1 ? 2.5 : 1.0);
  return longest >= least * seg ? (int)seg : INT32_MAX;
}

size_t ssm_split_bytes(const SsmArgs& a, int seg) {
  return seg == INT32_MAX ? 0 : (size_t)ssm_segments(a, seg) * a.D * (a.S + 1) * sizeof(float);
}

SsmSplit ssm_split_at(const SsmArgs& a, int seg, void* workspace) {
  SsmSplit s{seg, static_cast<float*>(workspace), nullptr};
  if (seg != INT32_MAX) s.steps = s.ends + ssm_segments(a, seg) * a.D * a.S;
  return s;
}

namespace {
template <typename IO>
cudaError_t ends_pass(const SsmArgs& a, const SsmSplit& split, cudaStream_t st) {
  return split.seg == INT32_MAX ? cudaSuccess
                                : fwd_pick<IO, kSsmEnds>(a, SsmSave{}, split, st);
}
template <typename IO>
cudaError_t scan(const SsmArgs& a, const SsmSave* save, const SsmSplit& split, cudaStream_t st) {
  cudaError_t e = ends_pass<IO>(a, split, st);
  if (e != cudaSuccess) return e;
  if (!save) return fwd_pick<IO, kSsmOut>(a, SsmSave{}, split, st);
  return save->dz ? fwd_pick<IO, kSsmSaveDz>(a, *save, split, st)
                  : fwd_pick<IO, kSsmSave>(a, *save, split, st);
}
}  // namespace

size_t ssm_fwd_workspace_bytes(const SsmArgs& a, int sms) {
  return ssm_split_bytes(a, ssm_segment(a, sms, 3.0));
}

cudaError_t launch_ssm_fwd(const SsmArgs& a, void* workspace, int sms, cudaStream_t st) {
  if (a.n_seqs == 0) return cudaSuccess;
  const SsmSplit split = ssm_split_at(a, ssm_segment(a, sms, 3.0), workspace);
  return a.bf16 ? scan<__nv_bfloat16>(a, nullptr, split, st) : scan<float>(a, nullptr, split, st);
}

cudaError_t launch_ssm_save(const SsmArgs& a, const SsmSave& save, const SsmSplit& split,
                            cudaStream_t st) {
  if (a.n_seqs == 0) return cudaSuccess;
  return a.bf16 ? scan<__nv_bfloat16>(a, &save, split, st) : scan<float>(a, &save, split, st);
}

cudaError_t launch_ssm_step(const SsmArgs& a, cudaStream_t st) {
  if (a.n_seqs == 0 || a.T == 0) return cudaSuccess;
  return a.bf16 ? step_pick<__nv_bfloat16>(a, st) : step_pick<float>(a, st);
}

}  // namespace kda

// Shared by the selective scan's forward and backward: the split of channels
// and states over lanes, the staged tile of one token range, and sums over
// lanes.
//
//   step_t = softplus(delta_t + bias);  a_t[n] = exp(step_t A[n])
//   h_t[n] = a_t[n] h_{t-1}[n] + step_t u_t B_t[n];  y_t = sum_n C_t[n] h_t[n]
//
// A lane owns 4 states of one channel; L lanes hold a channel's states
// (4 L >= S, absent states have A = B = C = 0 and stay 0), 128 threads hold
// 128 / L channels of one group and one sequence and walk the sequence in
// tiles of tokens.  Per (token, channel) a tile keeps step and step * u, per
// token the 4 L values of B and of C, all fp32 in shared memory.
#pragma once

#include "kda_layer.cuh"

namespace kda {

constexpr float kMaxFinite = 3.402823466e38f;
constexpr int kSsmThreads = 128;
constexpr int kSsmStates = 4;  // states per lane
constexpr int kHelpers = 128;  // threads that feed the recurrence's 128

// Tokens per tile: 32; 16 where two lanes a channel give the CTA 64 channels
// (a helper then holds 8 pairs as with four lanes, 16 with a tile of 32).
constexpr int tile_of(int lanes) { return lanes == 2 ? 16 : 32; }

// N elements on their way from memory, as the 32-bit registers that the loads
// write: nothing touches them before get(), so that every load of a tile is
// in flight at once.  VEC: neighbouring elements, aligned to their whole size
// (16 bytes at most), else one register each.
template <typename IO, int N, bool VEC>
struct Held {
  static constexpr int BYTES = N * (int)sizeof(IO);
  static constexpr bool PACKED = VEC && BYTES % 4 == 0;
  static constexpr int WORDS = PACKED ? BYTES / 4 : N;
  static constexpr int ALIGN = VEC ? (BYTES > 16 ? 16 : BYTES) : (int)sizeof(IO);
  uint32_t w[WORDS];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void one(int j, const IO* p) {
    if constexpr (sizeof(IO) == 2)
      w[j] = *reinterpret_cast<const uint16_t*>(p);
    else
      w[j] = *reinterpret_cast<const uint32_t*>(p);
  }
  __device__ __forceinline__ void all(const IO* p) {
    if constexpr (!PACKED) {
      one(0, p);
    } else if constexpr (WORDS == 1) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (WORDS == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x;
      w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < WORDS; i += 4) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i / 4];
        w[i] = v.x;
        w[i + 1] = v.y;
        w[i + 2] = v.z;
        w[i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (sizeof(IO) == 4) return __uint_as_float(w[j]);
    if constexpr (!PACKED) return __uint_as_float(w[j] << 16);
    return j & 1 ? bf_hi(w[j / 2]) : bf_lo(w[j / 2]);
  }
};

// N consecutive floats to shared memory (aligned to 4 N bytes, 16 at most).
template <int N>
__device__ __forceinline__ void store_floats(float* p, const float (&v)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else if constexpr (N == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = v[i];
  }
}

// The channels of a CTA: channel blocks are counted group by group.
struct SsmBlock {
  int g, c0, n;  // group, first channel, channels (<= CH)
  __device__ __forceinline__ SsmBlock(const SsmArgs& a, int ch, int block) {
    const int per = a.D / a.G, nb = (per + ch - 1) / ch;
    g = block / nb;
    const int k = block % nb;
    c0 = g * per + k * ch;
    n = min(ch, per - k * ch);
  }
};

// p: a chunk's product of decays, as multiplied up; becomes what its decay
// exp(sum of steps * A) has more than that.
__device__ __forceinline__ void chunk_decay(float sum, f32x2 A01, f32x2 A23, f32x2& p01,
                                            f32x2& p23) {
  float x[4];
  unpack2(mul2(both(sum), A01), x[0], x[1]);
  unpack2(mul2(both(sum), A23), x[2], x[3]);
  p01 = fma2(p01, both(-1.f), pack2(ex2_f(x[0]), ex2_f(x[1])));
  p23 = fma2(p23, both(-1.f), pack2(ex2_f(x[2]), ex2_f(x[3])));
}
// Adds what the chunk's decay has more, p, times the chunk's start state c.
// Where that is not finite nothing is added: with an infinite c the state is
// what the single decays made of it, and a p that is not finite (a growth
// beyond fp32) says nothing about a c of 0.
__device__ __forceinline__ void chunk_add(f32x2 p, f32x2 c, f32x2& h) {
  float lo, hi;
  unpack2(mul2(p, c), lo, hi);
  h = add2(h, pack2(fabsf(lo) <= kMaxFinite ? lo : 0.f, fabsf(hi) <= kMaxFinite ? hi : 0.f));
}
// A segment's end state from its start state h: decay * h + end, where an
// infinite h stays infinite and a h of 0 stays 0, though the decay of all the
// segment's tokens may be below or beyond what fp32 holds.
__device__ __forceinline__ float segment_join(float decay, float h, float end) {
  return isnan(decay * h) ? h + end : fmaf(decay, h, end);
}

// Sum of NV values over the lanes that differ in the bits of `mask`, spread:
// while there are values to halve, each exchange keeps one half of them; the
// rest are plain exchanges.  Returns with v[0 .. NV/lanes) (at least one)
// holding the totals of values first .. first + that many.
template <int NV, int LOW, int HIGH>
struct SpreadSum {  // lanes LOW, 2 LOW, ... < HIGH
  static __device__ __forceinline__ void run(float (&v)[NV], int lane, int& first) {
    if constexpr (LOW < HIGH) {
      if constexpr (NV > 1) {
        constexpr int HALF = NV / 2;
        const bool up = lane & LOW;
        float w[HALF];
#pragma unroll
        for (int i = 0; i < HALF; ++i) {
          const float keep = up ? v[i + HALF] : v[i];
          const float give = up ? v[i] : v[i + HALF];
          w[i] = keep + __shfl_xor_sync(0xffffffffu, give, LOW);
        }
        if (up) first += HALF;
        SpreadSum<HALF, LOW * 2, HIGH>::run(w, lane, first);
#pragma unroll
        for (int i = 0; i < HALF; ++i) v[i] = w[i];
      } else {
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], LOW);
        SpreadSum<1, LOW * 2, HIGH>::run(v, lane, first);
      }
    }
  }
};

// Pieces of n tokens of every sequence (the backward's saved states every 8
// tokens; the segments of a split scan): piece c of sequence s has the id
// start_s / n + s + c.  A sequence has max(1, ceil(len / n)) pieces; the ids of
// two sequences never meet, since floor((start + len) / n) + 1 >=
// floor(start / n) + max(1, ceil(len / n)), and are below tokens / n + n_seqs
// + 1.
__host__ __device__ __forceinline__ int64_t ssm_piece_id(int s, int start, int n, int c) {
  return (int64_t)(start / n) + s + c;
}
constexpr int kSsmChunk = 8;

// The sequence and piece of an id; false where the id has none.
__device__ __forceinline__ bool ssm_piece(const SsmArgs& a, int n, int64_t id, int* seq, int* c,
                                          int* start, int* end) {
  int lo = 0, hi = a.n_seqs;  // the last sequence whose first id is <= id
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    int s, e;
    seq_range(a.cu, mid, a.T, &s, &e);
    if (ssm_piece_id(mid, s, n, 0) <= id)
      lo = mid;
    else
      hi = mid;
  }
  seq_range(a.cu, lo, a.T, start, end);
  const int64_t k = id - ssm_piece_id(lo, *start, n, 0);
  const int len = *end - *start;
  *seq = lo;
  *c = (int)k;
  return k >= 0 && k < max((int64_t)1, ((int64_t)len + n - 1) / n);
}

// What one pass of the forward kernel is for.
enum SsmMode {
  kSsmOut,     // out = y silu(z), final states
  kSsmSave,    // the backward's first pass: the state at every 8th token
  kSsmSaveDz,  // the same, and dz = d_out y silu'(z)
  kSsmEnds,    // a split scan's first pass: each segment's end from state 0
};
// A split scan: segments of `seg` tokens; ends [segment id][D][S] their states
// from zero, steps [segment id][D] their sums of steps (a segment's decay is
// exp(A * sum of steps)).  The row of a sequence's last segment holds the
// sequence's start state.
struct SsmSplit {
  int seg;  // INT32_MAX: not split
  float* ends;
  float* steps;
};
struct SsmSave {
  float* states;      // [piece ids of 8 tokens][D][S]
  const void* d_out;  // for dz
  void* dz;
};
// Tokens per segment of a scan over `a` on a device of `sms` SMs where a
// sequence makes `least` of them, else INT32_MAX (not split); an upper bound of
// the segment ids, and the workspace that a split takes.
int ssm_segment(const SsmArgs& a, int sms, double least);
inline int64_t ssm_segments(const SsmArgs& a, int seg) { return a.tokens / seg + a.n_seqs + 1; }
size_t ssm_split_bytes(const SsmArgs& a, int seg);
SsmSplit ssm_split_at(const SsmArgs& a, int seg, void* workspace);
cudaError_t launch_ssm_save(const SsmArgs& a, const SsmSave& save, const SsmSplit& split,
                            cudaStream_t stream);

// Lanes per channel for S states: the smallest power of two >= S / 4, at
// least 2 (so that a CTA never holds more than 64 channels).
inline int ssm_lanes(int S) {
  int l = 2;
  while (l * kSsmStates < S) l *= 2;
  return l;
}
__host__ __device__ inline int ssm_blocks(const SsmArgs& a, int ch) {
  const int per = a.D / a.G;
  return a.G * ((per + ch - 1) / ch);
}

}  // namespace kda

// Beam search's selection over beams and vocabulary, and which slot each new beam lives in, gfx950.
//
// A candidate (beam b, token t) of a request has the score
//   score_b + x_bt - log sum_t' e^(x_bt'),
// and the request keeps its `beams` best, ties going to the lowest b * vocab + t; a finished beam
// has the one candidate (b, eos) at its own score.  The best `beams` of a row are the best of its
// logits, so the vocabulary is read once, without the row's sum being known:
//   1. beam_scan_kernel   per (row, tile of the vocabulary): largest logit, sum of exponentials and
//                         the tile's best logits with their tokens;
//   2. beam_pick_kernel   per request: log-sum-exp of every beam, the candidates' scores in fp64
//                         (neighbouring scores decide ranks, and a score is a small difference of
//                         large numbers), the best of them, and the slots.
// Only the exponentials and their sums inside a thread are fp32.
// A recurrent state cannot be shared by two beams, but a beam that goes on keeps its slot: a
// parent's first child stays where the state is, and each further child takes the slot of a beam
// that lost all its children.  Only those states are copied (by the slot copy that follows), and no
// copy reads a slot that another one writes.
//
// A tile's best come by a threshold rather than by sorting: the beams-th largest of a wave's 64
// lane maxima is at most the beams-th largest logit, and few logits reach it.
//
// Measured: 256 rows of 131072 bf16 logits, of which 15% belong to finished beams, scan 34 us (58 MB,
// 1.7 TB/s; 710 VALU instructions a wave are 20 us of issue, which keeps it from the 9 us of the copy's
// rate), pick 14 us, the copies of the states of two wide layers 93 us (566 MB, 6.1 TB/s); 4 rows of 32003
// fp32 logits 7 + 6 + 2 us, all latency.
#include "beam.h"
#include "device_common.h"

namespace m2 {
namespace {

constexpr int kWaves = kBeamThreads / 64;
constexpr int kListCap = 1024;   // logits or candidates that reach the threshold, in LDS
constexpr int kHeldCap = 4096;   // candidates whose scores stay in LDS between the two looks at them

// A float as an unsigned integer of the same order; -0 counts as 0.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint64_t ordered(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return b ^ ((b >> 63) ? ~0ull : 0x8000000000000000ull);
}

// Reductions over a wave, in every lane: inside 16 lanes by data-parallel primitives (quads, then the
// mirrored half row and row), across them by two exchanges.
template <typename T, typename F> __device__ __forceinline__ T wave_reduce(T v, F&& f) {
  v = f(v, dpp<0xB1>(v));
  v = f(v, dpp<0x4E>(v));
  v = f(v, dpp<0x141>(v));
  v = f(v, dpp<0x140>(v));
  v = f(v, __shfl_xor(v, 16));
  return f(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ double wave_sum(double v) {
  return wave_reduce(v, [](double a, double b) { return a + b; });
}

// The upper bits [31:32-BITS] of the k-th largest of a wave's values, the rest zero: at most that
// value.  0 if fewer than k lanes hold one above 0.
template <int BITS> __device__ __forceinline__ uint32_t kth_largest(uint32_t v, int k) {
  uint32_t thr = 0;
#pragma unroll
  for (int b = 31; b > 31 - BITS; --b) {
    const uint32_t t = thr | (1u << b);
    if (__popcll(__ballot(v >= t)) >= k) thr = t;
  }
  return thr;
}

// One 16-byte piece of a row as fp32 values, at the alignment of its elements.
template <bool BF16> struct Piece;
template <> struct Piece<true> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void load(const void* p, int64_t i, float* o) {
    typedef bf16 piece __attribute__((ext_vector_type(8), aligned(2)));
    const piece v = __builtin_nontemporal_load(reinterpret_cast<const piece*>(static_cast<const bf16*>(p) + i));
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = static_cast<float>(v[e]);
  }
};
template <> struct Piece<false> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void load(const void* p, int64_t i, float* o) {
    typedef float piece __attribute__((ext_vector_type(4), aligned(4)));
    const piece v = __builtin_nontemporal_load(reinterpret_cast<const piece*>(static_cast<const float*>(p) + i));
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = v[e];
  }
};

// A beam none of whose continuations can be taken.
__device__ __forceinline__ bool dead(float score) { return !(score > -INFINITY && score < INFINITY); }

template <bool BF16> __global__ __launch_bounds__(kBeamThreads) void beam_scan_kernel(BeamParams p) {
  constexpr int N = Piece<BF16>::N, PIECES = kBeamPerThread / N;
  __shared__ float s_val[kListCap];
  __shared__ int s_tok[kListCap];
  __shared__ float s_max[kWaves];
  __shared__ double s_sum[kWaves];
  __shared__ uint32_t s_thr[kWaves];
  __shared__ uint64_t s_best[kWaves];
  __shared__ int s_n;
  const int tile = blockIdx.x % p.tiles, row = blockIdx.x / p.tiles;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t out = (int64_t)row * p.tiles + tile;
  float* cv = p.cand_val + out * p.beams;
  int32_t* ct = p.cand_tok + out * p.beams;
  if (dead(p.scores[row]) || (p.finished && p.finished[row])) {   // its logits are not looked at
    if (tid == 0) p.part_max[out] = -INFINITY, p.part_sum[out] = 0.0;
    for (int i = tid; i < p.beams; i += kBeamThreads) ct[i] = -1;
    return;
  }
  // Piece i of the row holds its tokens i N .. i N + N-1, wherever in memory the row starts: which
  // logits are summed together depends on their tokens alone, so that equal rows have the same sum to
  // the last bit and their beams tie.  (The whole step over 256 bf16 rows of 131071, half of them off 4 bytes:
  // 109 us with pieces at their elements' alignment, 104 with pieces from the row's first 16-byte boundary.)
  const char* base = static_cast<const char*>(p.logits) + (int64_t)row * p.logits_stride * (BF16 ? 2 : 4);
  const int whole = p.vocab / N;
  float x[PIECES][N], mx[PIECES];
  auto piece_of = [&](int j) { return tile * (kBeamTile / N) + j * kBeamThreads + tid; };
  auto token_of = [&](int j) { return (int)((unsigned)piece_of(j) * N); };   // the piece's first
#pragma unroll
  for (int j = 0; j < PIECES; ++j) {
    const int pc = piece_of(j);
    if (pc < whole) {
      Piece<BF16>::load(base, (int64_t)pc * N, x[j]);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) x[j][e] = -INFINITY;
    }
  }
  if (tile == p.tiles - 1 && p.vocab % N) {   // the row's last piece, a part of one
#pragma unroll
    for (int j = 0; j < PIECES; ++j)
      if (piece_of(j) == whole) {
#pragma unroll
        for (int e = 0; e < N - 1; ++e)
          if (e < p.vocab % N) x[j][e] = load_any(base, (int64_t)whole * N + e, BF16);
      }
  }
  // largest logit (NaN are passed over here and make the sum NaN)
  float lm = -INFINITY;
#pragma unroll
  for (int j = 0; j < PIECES; ++j) {
    mx[j] = x[j][0];
#pragma unroll
    for (int e = 1; e < N; ++e) mx[j] = fmaxf(mx[j], x[j][e]);
    lm = fmaxf(lm, mx[j]);
  }
  const float wm = wave_max(lm);
  const uint32_t wt = kth_largest<16>(lm > -INFINITY ? ordered(lm) : 0u, p.beams);
  if (lane == 0) s_max[wave] = wm, s_thr[wave] = wt;
  if (tid == 0) s_n = 0;
  __syncthreads();
  float m = s_max[0];
  uint32_t thr = s_thr[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) {
    m = fmaxf(m, s_max[w]);
    thr = thr > s_thr[w] ? thr : s_thr[w];
  }
  // sum of e^(x - m).  The largest terms, exactly 1, are counted apart: next to them the others
  // would lose their last bits, and the log of the sum is compared between beams.  log2 e has two
  // parts: rounded to one, it would push every term the same way (by 1.3e-8 |x - m| of it).  Of the
  // sum, a term's difference and argument are off by 2^-24 |x - m| each, its exponential by 2^-23 and the
  // 12 additions by 2^-24 each; of 8192 terms the mean |x - m| is 6.2 at most: 1.6e-6 at worst, and about
  // 1e-8 where the roundings differ from term to term.
  float sum = 0.f;
  int ones = 0;
  auto term = [&](float v) {
    const float d = v - m;
    const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(d, 1.44269502f, d * 1.92596303e-8f));
    const bool one = v == m;
    ones += one;
    return one ? 0.f : e;
  };
#pragma unroll
  for (int j = 0; j < PIECES; ++j) {
    float part = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) part += term(x[j][e]);
    sum += part;
  }
  const double ws = wave_sum(m > -INFINITY ? (double)sum + (double)ones : sum == sum ? 0.0 : (double)sum);
  if (lane == 0) s_sum[wave] = ws;
  // logits that reach the threshold
  thr = thr ? thr : 1u;
  auto offer = [&](float v, int tok) {
    if (v > -INFINITY && ordered(v) >= thr) {
      const int i = atomicAdd(&s_n, 1);
      if (i < kListCap) s_val[i] = v, s_tok[i] = tok;
    }
  };
#pragma unroll
  for (int j = 0; j < PIECES; ++j) {
    if (mx[j] > -INFINITY && ordered(mx[j]) >= thr) {
      const int t0 = token_of(j);
#pragma unroll
      for (int e = 0; e < N; ++e) offer(x[j][e], t0 + e);
    }
  }
  __syncthreads();
  if (tid == 0) {
    double t = 0.0;
    for (int w = 0; w < kWaves; ++w) t += s_sum[w];
    p.part_max[out] = m;
    p.part_sum[out] = t;
  }
  const int n = s_n;
  if (n <= kListCap) {
    // rank each listed logit among the others; the order they were listed in does not matter
    for (int i = tid; i < n; i += kBeamThreads) {
      const uint32_t k = ordered(s_val[i]);
      const int tok = s_tok[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) {
        const uint32_t o = ordered(s_val[j]);
        rank += o > k || (o == k && s_tok[j] < tok);
      }
      if (rank < p.beams) cv[rank] = s_val[i], ct[rank] = tok;
    }
    for (int i = n + tid; i < p.beams; i += kBeamThreads) ct[i] = -1;
    return;
  }
  // So many equal logits that the list overflows (a constant row): one at a time, in order.
  uint64_t last = ~0ull;
  for (int r = 0; r < p.beams; ++r) {
    uint64_t best = 0;
    auto look = [&](float v, int tok) {
      const uint64_t k = ((uint64_t)ordered(v) << 32) | (uint32_t)~tok;
      if (v > -INFINITY && k < last && k > best) best = k;
    };
#pragma unroll
    for (int j = 0; j < PIECES; ++j) {
      const int t0 = token_of(j);
#pragma unroll
      for (int e = 0; e < N; ++e) look(x[j][e], t0 + e);
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) {
      const uint64_t up = __shfl_xor(best, o);
      best = up > best ? up : best;
    }
    if (lane == 0) s_best[wave] = best;
    __syncthreads();
    best = s_best[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) best = s_best[w] > best ? s_best[w] : best;
    if (tid == 0) {
      const uint32_t k = (uint32_t)(best >> 32);
      cv[r] = __uint_as_float((k >> 31) ? k ^ 0x80000000u : ~k);
      ct[r] = (int32_t)~(uint32_t)best;
    }
    last = best;
    __syncthreads();
  }
}

__global__ __launch_bounds__(kBeamThreads) void beam_pick_kernel(BeamParams p) {
  __shared__ double s_lse[kMaxBeams];
  __shared__ double s_held[kHeldCap];
  __shared__ double s_val[kListCap];
  __shared__ int64_t s_at[kListCap];
  __shared__ uint32_t s_thr[kWaves];
  __shared__ uint64_t s_key[kWaves];
  __shared__ int64_t s_pos[kWaves];
  __shared__ int s_n;
  __shared__ double r_val[kMaxBeams];
  __shared__ int64_t r_at[kMaxBeams];
  const int req = blockIdx.x, K = p.beams;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row0 = (int64_t)req * K;

  // log-sum-exp of each beam: a wave per beam, lanes over its tiles
  for (int b = wave; b < K; b += kWaves) {
    const float* pm = p.part_max + (row0 + b) * p.tiles;
    const double* ps = p.part_sum + (row0 + b) * p.tiles;
    float m = -INFINITY;
    for (int t = lane; t < p.tiles; t += 64) m = fmaxf(m, pm[t]);
    m = wave_max(m);
    double s = 0.0;
    for (int t = lane; t < p.tiles; t += 64)
      if (pm[t] > -INFINITY || !(ps[t] == 0.0)) s += ps[t] * exp((double)pm[t] - (double)m);
    s = wave_sum(s);
    if (lane == 0) s_lse[b] = (double)m + log(s);
  }
  if (tid == 0) s_n = 0;
  if (tid < K) r_val[tid] = -INFINITY, r_at[tid] = -1;
  __syncthreads();

  // candidate c: the (c % beams)-th best of tile (c / beams) of the request's rows.  A finished beam's
  // one candidate stands at the place of the first of its first tile.
  const int per = p.tiles * K, total = K * per;
  auto candidate = [&](int c, double& v, int64_t& at) {   // -inf where there is none
    const int b = c / per, i = c - b * per;
    const float sc = p.scores[row0 + b], x = p.cand_val[(row0 + b) * per + i];
    const int tok = p.cand_tok[(row0 + b) * per + i];
    const bool fin = p.finished && p.finished[row0 + b];
    at = (int64_t)b * p.vocab + (fin ? p.eos : tok);
    v = fin ? (double)sc : (double)sc + ((double)x - s_lse[b]);
    // a NaN among the row's logits, or an infinite one: none of its candidates
    if (dead(sc) || (fin ? i != 0 : tok < 0) || !(v > -INFINITY)) v = -INFINITY;
  };
  const bool hold = total <= kHeldCap;
  uint32_t lm = 0;
#pragma unroll 4
  for (int c = tid; c < total; c += kBeamThreads) {
    double v;
    int64_t at;
    candidate(c, v, at);
    if (hold) s_held[c] = v;
    const uint32_t k = v > -INFINITY ? (uint32_t)(ordered(v) >> 32) : 0u;
    lm = k > lm ? k : lm;
  }
  const uint32_t wt = kth_largest<32>(lm, K);
  if (lane == 0) s_thr[wave] = wt;
  __syncthreads();
  uint32_t thr = 1;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) thr = s_thr[w] > thr ? s_thr[w] : thr;
  for (int c = tid; c < total; c += kBeamThreads) {
    double v;
    int64_t at;
    if (hold) {
      v = s_held[c];
      if (!(v > -INFINITY && (uint32_t)(ordered(v) >> 32) >= thr)) continue;
    }
    candidate(c, v, at);
    if (v > -INFINITY && (uint32_t)(ordered(v) >> 32) >= thr) {
      const int i = atomicAdd(&s_n, 1);
      if (i < kListCap) s_val[i] = v, s_at[i] = at;
    }
  }
  __syncthreads();
  const int n = s_n;
  if (n <= kListCap) {
    for (int i = tid; i < n; i += kBeamThreads) {
      const double v = s_val[i];
      const int64_t at = s_at[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += s_val[j] > v || (s_val[j] == v && s_at[j] < at);
      if (rank < K) r_val[rank] = v, r_at[rank] = at;
    }
  } else {
    // more ties than the list holds: one at a time, in order
    uint64_t lastk = ~0ull;
    int64_t lastp = -1;
    for (int r = 0; r < K; ++r) {
      uint64_t bk = 0;
      int64_t bp = INT64_MAX;
      for (int c = tid; c < total; c += kBeamThreads) {
        double v;
        int64_t at;
        candidate(c, v, at);
        if (!(v > -INFINITY)) continue;
        const uint64_t k = ordered(v);
        if ((k < lastk || (k == lastk && at > lastp)) && (k > bk || (k == bk && at < bp))) bk = k, bp = at;
      }
#pragma unroll
      for (int o = 32; o; o >>= 1) {
        const uint64_t k = __shfl_xor(bk, o);
        const int64_t a = __shfl_xor(bp, o);
        if (k > bk || (k == bk && a < bp)) bk = k, bp = a;
      }
      if (lane == 0) s_key[wave] = bk, s_pos[wave] = bp;
      __syncthreads();
      bk = s_key[0], bp = s_pos[0];
#pragma unroll
      for (int w = 1; w < kWaves; ++w)
        if (s_key[w] > bk || (s_key[w] == bk && s_pos[w] < bp)) bk = s_key[w], bp = s_pos[w];
      if (tid == 0 && bk) {
        r_val[r] = __longlong_as_double((long long)((bk >> 63) ? bk ^ 0x8000000000000000ull : ~bk));
        r_at[r] = bp;
      }
      lastk = bk, lastp = bp;
      __syncthreads();
    }
  }
  __syncthreads();

  // the new beams, lane j the j-th: everything of the request's rows is read before any is written,
  // so outputs may be the inputs' own arrays
  if (wave == 0) {
    const bool mine = lane < K;
    const int64_t at = mine ? r_at[lane] : -1;
    const int parent = at >= 0 ? (int)(at / p.vocab) : -1, token = at >= 0 ? (int)(at % p.vocab) : -1;
    const int slot = mine ? p.slots[row0 + lane] : -1;
    const int done = mine && parent >= 0 && p.finished ? p.finished[row0 + parent] : 0;
    bool first = parent >= 0;
    uint32_t has_child = 0;
    for (int j = 0; j < K; ++j) {
      const int pj = __shfl(parent, j);
      if (pj >= 0) has_child |= 1u << pj;
      if (j < lane && pj == parent) first = false;
    }
    // children without their parent's slot take the childless beams' slots, both in order
    const uint64_t need = __ballot(mine && !first);
    const int turn = __popcll(need & ((1ull << lane) - 1));
    int home = parent, left = turn;
    if (!first)
      for (int j = 0; j < K; ++j)
        if (!((has_child >> j) & 1) && left-- == 0) home = j;
    const int to = __shfl(slot, home < 0 ? 0 : home), from = __shfl(slot, parent < 0 ? 0 : parent);
    if (mine) {
      const int64_t r = row0 + lane;
      p.tokens[r] = token;
      p.parents[r] = parent;
      p.scores_out[r] = (float)r_val[lane];
      if (p.finished_out) p.finished_out[r] = done || (parent >= 0 && token == p.eos) ? 1 : 0;
      p.slots_out[r] = to;
      p.copy_src[r] = !first && parent >= 0 ? from : -1;
      p.copy_dst[r] = !first && parent >= 0 ? to : -1;
    }
  }
}

}  // namespace

hipError_t launch_beam_select(const BeamParams& p, hipStream_t s) {
  const int rows = p.batch * p.beams;
  if (p.logits_bf16)
    hipLaunchKernelGGL(beam_scan_kernel<true>, dim3(rows * p.tiles), dim3(kBeamThreads), 0, s, p);
  else
    hipLaunchKernelGGL(beam_scan_kernel<false>, dim3(rows * p.tiles), dim3(kBeamThreads), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(beam_pick_kernel, dim3(p.batch), dim3(kBeamThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace m2

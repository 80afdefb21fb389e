// Gated delta rule, chunked prefill of packed variable-length sequences, gfx950.
//
// Per value head h of key head g = h / (Hv/Hk), with S the state as a (dk, dv) matrix:
//   S_t = alpha_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,   o_t = S_t^T q_t.
// A chunk of C <= 64 rows that starts from S0 has, with gamma_i the inclusive sum of log alpha,
//   L_ij = beta_i e^(gamma_i - gamma_j) k_i.k_j  (j < i),      T = (I + L)^-1,
//   U = T (beta o (V - e^gamma o K S0)),
//   O = e^gamma o Q S0 + (Q K^T o e^(gamma_i - gamma_j), j <= i) U,
//   S1 = e^gamma_C S0 + K^T (e^(gamma_C - gamma) o U),
// so that all work of a chunk is matrix products, and only K S0 -> U -> S1 is sequential.
//
// Two launches on one stream:
//   1. prep_kernel  per (chunk, key head): conv, SiLU and norms of q and k; K K^T and Q K^T; per
//                   value head the gates, T and the masked Q K^T; written to the workspace as
//                   MFMA operands in the order the second launch loads them;
//   2. the walk     per (sequence, value head, part of its dv columns): the chunks in order, the
//                   state in MFMA accumulators.  An accumulator tile pair is, with the K order
//                   kmap of the fragments, an operand of the next product as it stands, so the
//                   chain S0 -> K S0 -> U -> S1 never leaves a wave's registers.  role_walk_kernel
//                   for bf16 rows and dk <= 128, walk_kernel otherwise (one wave does all the work
//                   of its columns).
// Measured at 32 value heads of 128 x 128 over 16 key heads: 8192 rows of one sequence 257 us (launch 1
// 77 us: 31 of them VALU issue, 2220 instructions a wave, the rest latency that three workgroups a CU do
// not cover; it writes 168 MB, 44 of them spilled registers; launch 2 189 us, 1.5 us a chunk), 16 x 1024
// rows 393 us.
// Operands are fp16, one plane each, with fp32 accumulation; or, when q, k, v or o are fp32, three bf16
// planes whose sum is the fp32 value, and six MFMAs a product (the terms above 2^-24 of it).
// fp16 because K, Q, T, the masked Q K^T and the gates are at most 1 and everything else can be put in
// units (below): its 11 bits leave o and the states 3e-4 of the 2-norm off before their own rounding to
// bf16, 1.7e-3, 6e-4 where nothing decays.  With bf16 operands, U, e^(G-g) U, T and the masked Q K^T in
// two planes, it was 1.5e-3 to 2e-3, most of it from K and Q, and 8192 rows took 304 us.
// What the diagonals of T and Q K^T carry stays fp32 throughout: U starts from the unrounded R, and
// O takes q_i.k_i u_i elementwise, q_i.k_i from the unrounded rows.  The diagonal terms are the
// largest of their sums, and it costs no product.  Where keys repeat, U holds differences of
// neighbouring v whose sum over the chunk must telescope, and T's roundings, each repeated down a
// column, add up instead: one key written 150 times without decay is 2.4e-3 off, rounding included.
// State, gates, T and all sums are fp32, the sum of log alpha fp64: differences of it far behind a
// strong decay would lose the digits of the weak ones after it.
#include <cstddef>
#include <cstring>
#include <type_traits>

#include "device_common.h"
#include "gdn.h"

namespace m2 {
namespace {

constexpr int C = kGdnChunk;
constexpr int kPrepThreads = 256;
constexpr int LDL = C + 4;            // row pitch of the fp32 C x C matrices in LDS
constexpr int kTri = kGdnTriFrags * 512;   // elements of a plane of T or of the masked Q K^T
// In fp16, T and the masked Q K^T, which are at most 1, are stored times 2^15: entries behind a strong decay
// keep their digits down to 2^-29 and are 0 below 2^-40.  The factor goes on in U, and ends in the gates of
// the state and in the output's unit.
template <int NP> constexpr float kLift = NP == 1 ? 0x1p15f : 1.f;

struct alignas(16) PrepArgs {   // the first launch's one argument
  GdnPrefillParams p;
  int32_t tab[kGdnInlineBytes / 4];
};

typedef uint16_t u16;
typedef u16 u16x4 __attribute__((ext_vector_type(4)));
typedef u16 u16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16;
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef float floatx2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u16 bits(bf16 v) { return __builtin_bit_cast(u16, v); }

// An operand: one plane in fp16, or NP in bf16, the largest first: each is the rounding of what the ones
// before it leave.
template <int NP> struct Op {
  typedef bf16x8 vec;
  vec p[NP];
};
template <> struct Op<1> {
  typedef f16x8 vec;
  vec p[1];
};
template <int NP> __device__ __forceinline__ Op<NP> make_op(const float (&v)[8]) {
  Op<NP> o;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (NP == 1) {
      o.p[0][e] = static_cast<f16>(v[e]);
    } else {
      float rest = v[e];
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        o.p[i][e] = from_f32<bf16>(rest);
        if (i + 1 < NP) rest -= static_cast<float>(o.p[i][e]);
      }
    }
  }
  return o;
}
__device__ __forceinline__ floatx4 mfma(const bf16x8& a, const bf16x8& b, floatx4 acc) { return mfma_bf16(a, b, acc); }
__device__ __forceinline__ floatx4 mfma(const f16x8& a, const f16x8& b, floatx4 acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, acc, 0, 0, 0);
}
// acc += a b, without the plane products below 2^-8 per plane of it; the small ones first.
template <int NP> __device__ __forceinline__ floatx4 mul(const Op<NP>& a, const Op<NP>& b, floatx4 acc) {
#pragma unroll
  for (int s = NP - 1; s >= 0; --s)
#pragma unroll
    for (int i = s; i >= 0; --i) acc = mfma(a.p[i], b.p[s - i], acc);
  return acc;
}
// Waits until MFMA results in flight are in their registers.  The compiler places such waits by
// itself, but only along one of the paths that meet behind a branch, so this follows products whose
// results the code on the far side of a branch reads: `pin` each of them, then `settle`.
template <int N> __device__ __forceinline__ void pin(floatx4 (&a)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(a[i]));
}
__device__ __forceinline__ void settle() { asm volatile("s_nop 15"); }

// Launch tables are read through the constant address space (scalar loads).
typedef const __attribute__((address_space(4))) char cchar;
template <typename T> __device__ __forceinline__ T load_uniform(cchar* p) {
  typedef const __attribute__((address_space(4))) int cint;
  cint* q = (cint*)p;
  struct Words { int w[sizeof(T) / 4]; } w;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 4); ++i) w.w[i] = q[i];
  return __builtin_bit_cast(T, w);
}

// LDS of prep_kernel.  Rows of q and k are kept in the operands' own bf16, or in fp32 where an
// operand takes three planes (split as it is read).  Two value heads are worked on at a time.
template <int DK, int NP> struct PrepLds {
  typedef typename std::conditional<NP == 1, u16, float>::type row_t;
  static constexpr int LDK = DK + (NP == 1 ? 8 : 4);   // row pitch of q and k
  union {   // q and k are done with once the products are in registers
    struct {
      row_t k[C * LDK], q[C * LDK];
    };
    struct {
      float lt[2][C * LDL];                            // L transposed: row j, column i
      float xt[2][4 * 16 * 20];                        // inverses of the diagonal blocks of I + L, transposed
    };
  };
  double g[2][C];                                      // inclusive sums of log alpha
  float beta[2][C];
  // e^(g_i - g_j) of rows in different 16-row tiles is a product of two factors <= 1 about the last
  // row of the lower tile t: up[t][i] = e^(g_i - g_(16t+15)), down[j] = e^(g_(16 t(j) + 15) - g_j)
  float up[2][3][C], down[2][C];
  float diag[C];                                       // q_i.k_i
};
// Elements of a row in LDS -> an operand: two runs of four, `gap` apart.
template <int NP> __device__ __forceinline__ Op<NP> lds_op(const u16* p, int gap) {
  Op<1> o;
#pragma unroll
  for (int e = 0; e < 8; ++e) o.p[0][e] = __builtin_bit_cast(f16, p[(e >> 2) * gap + (e & 3)]);
  return o;
}
template <int NP> __device__ __forceinline__ Op<NP> lds_op(const float* p, int gap) {
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = p[(e >> 2) * gap + (e & 3)];
  return make_op<NP>(v);
}
// Lane `lane`'s part of fragment f of an array of planes `plane` elements apart.
template <int NP> __device__ __forceinline__ void put_op(u16* base, int plane, int f, int lane, const Op<NP>& o) {
#pragma unroll
  for (int i = 0; i < NP; ++i) *reinterpret_cast<typename Op<NP>::vec*>(base + i * plane + (f * 64 + lane) * 8) = o.p[i];
}
template <int NP> __device__ __forceinline__ Op<NP> get_op(const u16* base, int plane, int f, int lane) {
  Op<NP> o;
#pragma unroll
  for (int i = 0; i < NP; ++i) o.p[i] = *reinterpret_cast<const typename Op<NP>::vec*>(base + i * plane + (f * 64 + lane) * 8);
  return o;
}

// The value `O` lanes away (lane ^ O).
template <int O> __device__ __forceinline__ float lane_xor(float v) {
  if constexpr (O == 4) return dpp<0x1B>(dpp<0x141>(v));        // mirrored half row, then mirrored quads
  else if constexpr (O == 8) return dpp<0x128>(v);              // row rotated by 8
  else return __shfl_xor(v, O);
}

// One (chunk, key head).
template <int DK, int W, int NP, typename IO>
__global__ __launch_bounds__(kPrepThreads) __attribute__((amdgpu_waves_per_eu(3)))
void prep_kernel(PrepArgs args) {
  typedef PrepLds<DK, NP> Lds;
  typedef typename Lds::row_t row_t;
  constexpr int LDK = Lds::LDK;
  constexpr int LPR = DK / 8, KS = DK / 32, RR = DK / 16;   // lanes a row, K steps, rows a thread
  constexpr int RB = RR < 8 ? RR : 8;                       // rows a thread takes at a time
  const GdnPrefillParams& p = args.p;
  extern __shared__ char smem[];
  Lds& s = *reinterpret_cast<Lds*>(smem);
  const int tid = threadIdx.x, lane = tid & 63, q4 = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  const int units = p.num_chunks * p.sh.Hk;
  cchar* const inl = (cchar*)__builtin_amdgcn_kernarg_segment_ptr() + offsetof(PrepArgs, tab);
  if ((int)blockIdx.x == units) {   // the extra workgroup of inline tables: write them out for launch 2
    typedef const __attribute__((address_space(4))) int cint;
    for (int i = tid; i < p.tab_inline / 4; i += kPrepThreads)
      reinterpret_cast<int*>(const_cast<GdnSeq*>(p.seqs))[i] = ((cint*)inl)[i];
    return;
  }
  const int c = blockIdx.x / p.sh.Hk, g = blockIdx.x % p.sh.Hk;
  cchar* const tabs = p.tab_inline ? inl : (cchar*)p.seqs;
  const GdnChunk ce = load_uniform<GdnChunk>(tabs + p.tab_chunks + (size_t)c * sizeof(GdnChunk));
  const GdnSeq se = load_uniform<GdnSeq>(tabs + (size_t)ce.seq * sizeof(GdnSeq));
  const int len = ce.len;
  const int rep = p.sh.Hv / p.sh.Hk;

  // ---------------------------------------------------------------- conv, SiLU, norms of q and k
  {
    const int sub = tid % LPR, isk = (tid / LPR) & 1, r0 = tid / (2 * LPR) * RR;
    const int64_t col = (int64_t)g * DK + sub * 8;
    const int gc = (isk ? p.sh.Hk * DK : 0) + (int)col;
    const int64_t stride = isk ? p.k_stride : p.q_stride;
    typedef IO row8 __attribute__((ext_vector_type(8)));
    const IO* const src = static_cast<const IO*>(isk ? p.k : p.q) + (int64_t)se.t0 * stride + col;   // the sequence's rows
    float wt[8 * W], bias[8];
    const floatx4* wq = reinterpret_cast<const floatx4*>(p.conv_w + (int64_t)gc * W);
#pragma unroll
    for (int v = 0; v < 2 * W; ++v) {
      const floatx4 x = wq[v];
#pragma unroll
      for (int e = 0; e < 4; ++e) wt[4 * v + e] = x[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) bias[e] = p.conv_b ? p.conv_b[gc + e] : 0.f;
    const float scale = isk ? 1.f : __builtin_amdgcn_rsqf((float)DK);
    const bool whole = ce.tau0 >= W - 1 && len == C;      // every row and halo row is one of the sequence
#pragma unroll
    for (int rb = 0; rb < RR; rb += RB) {
      row8 raw[RB + W - 1];
      if (whole) {
        const IO* const from = src + (int64_t)(ce.tau0 + r0 + rb - (W - 1)) * stride;
#pragma unroll
        for (int i = 0; i < RB + W - 1; ++i) raw[i] = *reinterpret_cast<const row8*>(from + i * stride);
      } else {
#pragma unroll
        for (int i = 0; i < RB + W - 1; ++i) {
          const int tau = ce.tau0 + r0 + rb + i - (W - 1);
          raw[i] = *reinterpret_cast<const row8*>(src + (int64_t)(tau < 0 ? 0 : tau >= se.len ? se.len - 1 : tau) * stride);
          if (tau < 0) {                                  // ahead of the sequence: the slot's window, or zeros
            const bf16* wp = static_cast<const bf16*>(p.conv) + ((int64_t)se.slot * p.sh.Cd + gc) * (W - 1) + W - 1 + tau;
#pragma unroll
            for (int e = 0; e < 8; ++e) raw[i][e] = static_cast<IO>(se.has_init ? static_cast<float>(wp[e * (W - 1)]) : 0.f);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const int row = r0 + rb + i;
        float act[8], ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float x = bias[e];
#pragma unroll
          for (int j = 0; j < W; ++j) x += wt[e * W + j] * to_f32(raw[i + j][e]);
          act[e] = silu(x);
          ss += act[e] * act[e];
        }
        const float rn = __builtin_amdgcn_rsqf(group_sum<LPR>(ss) + 1e-6f) * scale;
        // rows behind the chunk are zero: they write nothing into the state
        float kq = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          act[e] = row < len ? act[e] * rn : 0.f;
          kq += act[e] * lane_xor<LPR>(act[e]);
        }
        kq = group_sum<LPR>(kq);
        if (sub == 0 && !isk) s.diag[row] = kq;
        row_t* dst = (isk ? s.k : s.q) + row * LDK + sub * 8;
        if constexpr (NP == 1) {
          *reinterpret_cast<f16x8*>(dst) = make_op<1>(act).p[0];
        } else {
          *reinterpret_cast<floatx4*>(dst) = floatx4{act[0], act[1], act[2], act[3]};
          *reinterpret_cast<floatx4*>(dst + 4) = floatx4{act[4], act[5], act[6], act[7]};
        }
      }
    }
  }

  // where value head `hl` of this chunk's operands go
  auto t_of = [&](int hl) {
    return reinterpret_cast<u16*>(p.head + ((int64_t)c * p.sh.Hv + g * rep + hl) * gdn_head_bytes(NP));
  };
  // Gates of value head `hl` into place z: one wave, lane i row i.
  auto gates = [&](int hl, int z) {
    const int h = g * rep + hl;
    double ga = 0.0;
    float be = 0.f;
    if (lane < len) {
      const int64_t r = (int64_t)se.t0 + ce.tau0 + lane;
      const float la = p.A[h] * softplus(load_any(p.a, r * p.a_stride + h, p.io_bf16) + p.dt_bias[h]);
      ga = (double)(la < -1e4f ? -1e4f : la);   // a decay below e^-1e4 is 0 in fp32 either way
      be = __builtin_amdgcn_rcpf(1.f + __expf(-load_any(p.b, r * p.b_stride + h, p.io_bf16)));
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const double up = __shfl_up(ga, o);
      if (lane >= o) ga += up;
    }
    s.g[z][lane] = ga;
    s.beta[z][lane] = be;
    const double G = __shfl(ga, 63);
    s.down[z][lane] = expf((float)(__shfl(ga, lane | 15) - ga));
#pragma unroll
    for (int t = 0; t < 3; ++t) {
      const double at = __shfl(ga, 16 * t + 15);
      s.up[z][t][lane] = expf((float)(lane > 16 * t + 15 ? ga - at : 0.0));
    }
    const float eg = expf((float)ga);
    u16* const tout = t_of(hl);
    float* const g1 = reinterpret_cast<float*>(tout + NP * kTri);
    g1[lane] = be;
    g1[C + lane] = be * eg;
    g1[2 * C + lane] = expf((float)(G - ga)) / kLift<NP>;
    g1[3 * C + lane] = __shfl(eg, 63);
    float* const g2 = reinterpret_cast<float*>(tout + gdn_t_bytes(NP) / 2 + NP * kTri);
    g2[lane] = eg;
  };
  if (wave < 2 && wave < rep) gates(wave, wave);
  __syncthreads();

  // ---------------------------------------------------------------- K tiles, Q fragments
  u16* const kout = reinterpret_cast<u16*>(p.kq + ((int64_t)c * p.sh.Hk + g) * gdn_kq_bytes(DK, NP));
  u16* const qout = kout + NP * C * DK;
  for (int f = wave; f < 4 * KS; f += 4) {
    const int o = (16 * (f / KS) + l16) * LDK + 32 * (f % KS) + 4 * q4;
    const Op<NP> k = lds_op<NP>(s.k + o, 16), q = lds_op<NP>(s.q + o, 16);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const u16x8 w = __builtin_bit_cast(u16x8, k.p[i]);
      u16* kt = kout + i * C * DK + f * 512 + lane * 4;   // tiles 2f and 2f + 1
      *reinterpret_cast<u16x4*>(kt) = u16x4{w[0], w[1], w[2], w[3]};
      *reinterpret_cast<u16x4*>(kt + 256) = u16x4{w[4], w[5], w[6], w[7]};
    }
    put_op<NP>(qout, C * DK, f, lane, q);
  }

  // ---------------------------------------------------------------- K K^T and Q K^T, lower tiles
  // Five products a wave, kept in registers for all value heads:
  //   slots 1, 2  Q K^T, row tile qi, column tiles 2 qp and 2 qp + 1: one fragment of the masked Q K^T
  //   slot 0      waves 0, 3: Q K^T tile (z0, z0), the lower half of a fragment whose upper half is
  //               above the diagonal; waves 1, 2: K K^T tile
  //   slots 3, 4  K K^T tiles
  // A Q K^T tile is computed transposed (rows j), so that a lane holds four columns of one row, as
  // the fragments do; a K K^T tile with rows i, so that a lane holds four of L^T.
  const int qi = wave == 0 ? 1 : wave == 1 ? 2 : 3, qp = wave == 3 ? 1 : 0;
  const bool zq = wave == 0 || wave == 3;
  int ki[5], kj[5];
  ki[0] = wave == 0 ? 0 : wave == 1 ? 1 : wave == 2 ? 3 : 2, kj[0] = wave == 0 || wave == 1 ? 0 : 2;
  ki[1] = ki[2] = qi, kj[1] = 2 * qp, kj[2] = 2 * qp + 1;
  ki[3] = wave == 0 ? 0 : wave == 1 ? 2 : wave == 2 ? 3 : 2, kj[3] = wave == 3 ? 2 : 0;
  ki[4] = wave == 0 ? 1 : wave == 1 ? 2 : 3, kj[4] = wave == 3 ? 3 : 1;
  floatx4 acc[5];
#pragma unroll
  for (int m = 0; m < 5; ++m) {
    const bool q = m == 1 || m == 2 || (m == 0 && zq);
    const row_t* A = s.k + (16 * (q ? kj[m] : ki[m]) + l16) * LDK + 8 * q4;
    const row_t* B = (q ? s.q : s.k) + (16 * (q ? ki[m] : kj[m]) + l16) * LDK + 8 * q4;
    acc[m] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) acc[m] = mul(lds_op<NP>(A + 32 * ks, 4), lds_op<NP>(B + 32 * ks, 4), acc[m]);
  }
  pin(acc);
  settle();
  acc[1] = acc[1] * kLift<NP>;
  acc[2] = acc[2] * kLift<NP>;
  if (zq) acc[0] = acc[0] * kLift<NP>;

  // ---------------------------------------------------------------- value heads, two at a time
  for (int h0 = 0; h0 < rep; h0 += 2) {
    const int nh = rep - h0 < 2 ? 1 : 2;
    if (h0 > 0) {
      __syncthreads();   // the heads before are done with everything
      if (wave < nh) gates(h0 + wave, wave);
    }
    __syncthreads();
    for (int z = 0; z < nh; ++z) {
      u16* const aout = t_of(h0 + z) + gdn_t_bytes(NP) / 2;
      if (wave == 0) reinterpret_cast<float*>(aout + NP * kTri)[C + lane] = s.diag[lane];
      // four values of the tile (it, jt): e^(g_i - g_j) below the diagonal, else 0.  COLS: columns j =
      // 4 q + r of row i = l; else rows i = 4 q + r of column j = l.
      auto decays = [&](int it, int jt, bool cols) {
        floatx4 d;
        if (it != jt) {
          if (cols) d = s.up[z][jt][16 * it + l16] * *reinterpret_cast<const floatx4*>(&s.down[z][16 * jt + 4 * q4]);
          else d = *reinterpret_cast<const floatx4*>(&s.up[z][jt][16 * it + 4 * q4]) * s.down[z][16 * jt + l16];
        } else {
          const double at = s.g[z][16 * it + l16];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const double o = s.g[z][16 * it + 4 * q4 + r];
            const bool below = cols ? 4 * q4 + r < l16 : l16 < 4 * q4 + r;
            d[r] = below ? expf((float)(cols ? at - o : o - at)) : 0.f;
          }
        }
        return d;
      };
      auto put_l = [&](int m) {
        const floatx4 be = *reinterpret_cast<const floatx4*>(&s.beta[z][16 * ki[m] + 4 * q4]);
        *reinterpret_cast<floatx4*>(&s.lt[z][(16 * kj[m] + l16) * LDL + 16 * ki[m] + 4 * q4]) =
            be * decays(ki[m], kj[m], false) * acc[m];
      };
      const floatx4 none = {0.f, 0.f, 0.f, 0.f};
      const floatx4 a1 = decays(qi, kj[1], true) * acc[1], a2 = decays(qi, kj[2], true) * acc[2];
      const float pair[8] = {a1[0], a1[1], a1[2], a1[3], a2[0], a2[1], a2[2], a2[3]};
      put_op<NP>(aout, kTri, gdn_tri(qi, qp), lane, make_op<NP>(pair));
      if (zq) {
        const floatx4 a0 = decays(ki[0], ki[0], true) * acc[0];
        const float half[8] = {a0[0], a0[1], a0[2], a0[3], none[0], none[1], none[2], none[3]};
        put_op<NP>(aout, kTri, gdn_tri(ki[0], ki[0] / 2), lane, make_op<NP>(half));
      } else {
        put_l(0);
      }
      put_l(3);
      put_l(4);
    }
    __syncthreads();
    // T = (I + L)^-1, held transposed.  The diagonal block `wave` of both heads by substitution: lane
    // group z, lane l the column l of the inverse.  Substitution in fp32 keeps the entries as exact
    // as L, where a power series would lose digits on strongly correlated keys.
    {
      const int z = q4 & 1;
      const float* lb = s.lt[z] + (16 * wave) * LDL + 16 * wave;
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = i == l16 ? 1.f : 0.f;
#pragma unroll
      for (int j = 0; j < 15; ++j) {
#pragma unroll
        for (int i4 = (j + 1) / 4 * 4; i4 < 16; i4 += 4) {
          const floatx4 l = *reinterpret_cast<const floatx4*>(lb + j * LDL + i4);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (i4 + e > j) x[i4 + e] -= l[e] * x[j];
        }
      }
      if (q4 < nh) {
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<floatx4*>(&s.xt[z][(16 * wave + l16) * 20 + i]) = floatx4{x[i], x[i + 1], x[i + 2], x[i + 3]};
      }
    }
    __syncthreads();
    // Row tile I of T, transposed: Y_I = X_I as it is, Y_j = -X_j sum_{j<k<=I} (L^T)_jk Y_k, in fp32
    // MFMA.  An accumulator (rows 4q + r) is the next product's operand if step r takes the K
    // positions 4q + r, so left operands are read as row l % 16, columns 4q .. 4q + 3; and four of its
    // rows in a lane are four columns of T's row, as in T's fragments.
    auto row_tile = [&](auto tile, int z) {
      constexpr int I = decltype(tile)::value;
      const float *lt = s.lt[z], *xt = s.xt[z];
      floatx4 Y[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) Y[I][r] = xt[(16 * I + 4 * q4 + r) * 20 + l16] * kLift<NP>;
#pragma unroll
      for (int j = I - 1; j >= 0; --j) {
        floatx4 m = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = j + 1; k <= I; ++k) {
          const floatx4 l = *reinterpret_cast<const floatx4*>(lt + (16 * j + l16) * LDL + 16 * k + 4 * q4);
#pragma unroll
          for (int r = 0; r < 4; ++r) m = __builtin_amdgcn_mfma_f32_16x16x4f32(l[r], Y[k][r], m, 0, 0, 0);
        }
        const floatx4 x = *reinterpret_cast<const floatx4*>(xt + (16 * j + l16) * 20 + 4 * q4);
        Y[j] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int r = 0; r < 4; ++r) Y[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(-x[r], m[r], Y[j], 0, 0, 0);
      }
      u16* const tout = t_of(h0 + z);
#pragma unroll
      for (int ks = 0; ks <= I / 2; ++ks) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int j = 2 * ks + (e >> 2);
          // the unit diagonal is left out: U takes R itself there
          v[e] = j > I ? 0.f : j == I ? (4 * q4 + (e & 3) < l16 ? Y[I][e & 3] : 0.f) : Y[j][e & 3];
        }
        put_op<NP>(tout, kTri, gdn_tri(I, ks), lane, make_op<NP>(v));
      }
    };
    // tiles I cost 0, 2, 5 and 9 products: the second head takes them the other way round
    auto wave_tiles = [&](auto lo) {
      row_tile(lo, 0);
      if (nh > 1) row_tile(std::integral_constant<int, 3 - decltype(lo)::value>(), 1);
    };
    switch (wave) {
      case 0: wave_tiles(std::integral_constant<int, 0>()); break;
      case 1: wave_tiles(std::integral_constant<int, 1>()); break;
      case 2: wave_tiles(std::integral_constant<int, 2>()); break;
      default: wave_tiles(std::integral_constant<int, 3>());
    }
  }
}

// Two accumulator tiles (rows 0-15 and 16-31 of a 32-row K step) as an operand.
template <int NP> __device__ __forceinline__ Op<NP> acc_op(const floatx4& a, const floatx4& b) {
  const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  return make_op<NP>(v);
}

// 16 bytes per lane from global memory to LDS at `l` + 16 lane, without passing registers.
__device__ __forceinline__ void dma16(const void* g, void* l) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)g,
                                   (__attribute__((address_space(3))) void*)l, 16, 0, 0);
}
__device__ __forceinline__ void wait_dma() { __builtin_amdgcn_s_waitcnt(0x0f70); }   // vmcnt(0)

// K^T out of the K tiles by transposing reads: lane l of 16 lanes gets column l of four rows.  `t` is
// the lane's piece of the tile of the lower 16 rows, `step` elements ahead of that of the upper 16.
template <typename V> __device__ __forceinline__ V tr_frag(const u16* t, int step) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  typedef __attribute__((address_space(3))) s16x4 lds4;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)t);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(t + step));
  return __builtin_bit_cast(V, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
}

// ---- Units of the fp16 form.  Everything that the walk does to a column of dv is linear in that column of
// V and S, so its fp16 operands are in units of the column's own, powers of two: S0 in one that puts its
// largest element between 2^14 and 2^15; R, U and e^(G-g) U in one that puts the largest of R between 2^8 and
// 2^9.  |k| <= 1 and gates <= 1 bound T by 1, so that |U| <= 64 max |R| < 2^15 in that unit: nothing
// overflows, and 2^-22 of the largest still has all its digits.
struct Unit {
  float size, inverse;
};
template <int E> __device__ __forceinline__ Unit unit_of(float largest) {   // largest / size in [2^E, 2^(E+1))
  const uint32_t e = __float_as_uint(fminf(fmaxf(largest, 0x1p-100f), 0x1p126f)) & 0x7f800000u;   // 2^floor(log2)
  const uint32_t u = e - ((uint32_t)E << 23);
  return {__uint_as_float(u), __uint_as_float((254u << 23) - u)};
}
// The unit of R.  The next state is in it too: what is left of S0 in it, at most `rest`, must not overflow
// fp32.  It exceeds R by 2^110 only where R does not count beside it, in the state as in the outputs.
__device__ __forceinline__ Unit unit_of_r(float largest, float rest) { return unit_of<8>(fmaxf(largest, rest * 0x1p-110f)); }
// A ratio of units, finite, so that what it multiplies stays zero if it is.
__device__ __forceinline__ float finite(float ratio) { return fminf(ratio, 0x1p127f); }
// The largest of the four lanes that have a column (lane, lane ^ 16, ^ 32, ^ 48).
__device__ __forceinline__ float column_max(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
template <int N> __device__ __forceinline__ float largest(const floatx4 (&x)[N]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) m = fmaxf(m, fabsf(x[i][r]));
  return m;
}

constexpr int kWalkWaves = 2;   // of a walk_kernel workgroup, 16 columns of dv each

// What a walk workgroup stages in LDS per chunk: K, Q, T, the masked Q K^T and the gates as they lie
// in the workspace, and per wave the raw v rows of its columns with the W-1 rows ahead of them.  Row
// i of those is at slot (i % 4) * 17 + i / 4: the four lane groups of an accumulator tile read rows
// 4 apart, which so lie side by side in the banks.
template <int DK, int NP, typename IO> struct Stage {
  static constexpr int KQ = gdn_kq_bytes(DK, NP), HEAD = gdn_head_bytes(NP);
  static constexpr int SLOTS = 68, SLOT_BYTES = 16 * (int)sizeof(IO);
  static constexpr int V_OPS = (SLOTS * SLOT_BYTES + 1023) / 1024;   // wave-wide copies of one wave's v
  // Q stays in global memory where all of it does not fit (dk 256 in three planes)
  static constexpr bool Q_IN = KQ + HEAD + kWalkWaves * V_OPS * 1024 <= (int)kMaxLdsBytes;
  static constexpr int KIN = Q_IN ? KQ : KQ / 2;
  static constexpr int BYTES = KIN + HEAD + kWalkWaves * V_OPS * 1024;
  static constexpr int PIECES = (KIN + HEAD) / 1024;
  static_assert(BYTES <= (int)kMaxLdsBytes, "LDS of a walk workgroup");
  static_assert(KQ % 1024 == 0 && HEAD % 1024 == 0, "whole pieces");
};

// One workgroup of kWalkWaves waves per (sequence, value head, 32 columns of dv); lane l of a wave has
// the column l % 16 of the wave's 16.  NB stages in LDS: with two, the next chunk's operands travel while
// this one is computed.
template <int DK, int W, int NP, int NB, typename IO>
__global__ __launch_bounds__(64 * kWalkWaves) void walk_kernel(GdnPrefillParams p, int parts, int groups) {
  typedef Stage<DK, NP, IO> St;
  constexpr int KS = DK / 32, NT = DK / 16;
  extern __shared__ char smem[];
  const int lane = threadIdx.x & 63, q4 = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rep = p.sh.Hv / p.sh.Hk, dv = p.sh.dv;
  // The workgroups of a (sequence, key head), which read the same K and Q, go to one XCD (workgroups
  // are dealt over the 8 XCDs in turn), so that they meet in its L2.
  const int per = rep * parts, turn = blockIdx.x >> 3;
  const int grp = turn / per * 8 + (blockIdx.x & 7), in = turn % per;
  if (grp >= groups) return;
  const int g = grp % p.sh.Hk, h = g * rep + in / parts;
  const GdnSeq se = load_uniform<GdnSeq>((cchar*)(p.seqs + grp / p.sh.Hk));
  if (se.nchunk == 0) return;
  const int c0 = (in % parts * kWalkWaves + wave) * 16;   // the wave's first column of dv
  const bool active = c0 < dv;
  bf16* const ssm = static_cast<bf16*>(p.ssm);
  bf16* const conv = static_cast<bf16*>(p.conv);
  const bool has = c0 + l16 < dv;
  const int col = has ? c0 + l16 : dv - 1;                // a lane without a column repeats the last one
  const int gc = 2 * p.sh.Hk * DK + h * dv + col;         // its conv channel
  float wt[W], win[W - 1];
  floatx4 S[NT];      // in units of `unit` (three planes: of 1)
  float unit = 1.f;
#pragma unroll
  for (int j = 0; j < W; ++j) wt[j] = p.conv_w[(int64_t)gc * W + j];
  const float bias = p.conv_b ? p.conv_b[gc] : 0.f;
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
    win[j] = se.has_init ? static_cast<float>(conv[((int64_t)se.slot * p.sh.Cd + gc) * (W - 1) + j]) : 0.f;
  const bf16* sp = ssm + (((int64_t)se.slot * p.sh.Hv + h) * dv + col) * DK + 4 * q4;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const u16x4 x = se.has_init ? *reinterpret_cast<const u16x4*>(sp + 16 * i) : u16x4{0, 0, 0, 0};
#pragma unroll
    for (int r = 0; r < 4; ++r) S[i][r] = static_cast<float>(__builtin_bit_cast(bf16, (u16)x[r]));
  }
  const IO* const vbase = static_cast<const IO*>(p.v) + (int64_t)se.t0 * p.v_stride + h * dv;

  auto put_slot = [&](int slot, int end) {   // state and window after `end` rows of the sequence
    if (has) {
      bf16* sp = ssm + (((int64_t)slot * p.sh.Hv + h) * dv + col) * DK + 4 * q4;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        u16x4 o;
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] = bits(from_f32<bf16>(S[i][r] * unit));
        *reinterpret_cast<u16x4*>(sp + 16 * i) = o;
      }
      if (q4 == 0) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
          const int tau = end - (W - 1) + j;
          float x = 0.f;
          if (tau >= 0) {
            x = to_f32(vbase[(int64_t)tau * p.v_stride + col]);
          } else {
#pragma unroll
            for (int i = 0; i < W - 1; ++i) x = tau == i - (W - 1) ? win[i] : x;
          }
          conv[((int64_t)slot * p.sh.Cd + gc) * (W - 1) + j] = from_f32<bf16>(x);
        }
      }
    }
    if (c0 == 0 && h % rep == 0) {   // the key head's q and k channels
      for (int i = lane; i < 2 * DK; i += 64) {
        const int isk = i >= DK, kc = g * DK + (isk ? i - DK : i);
        const int64_t ch = (isk ? p.sh.Hk * DK : 0) + kc;
        float keep[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
          const int tau = end - (W - 1) + j;
          if (tau >= 0)
            keep[j] = to_f32(static_cast<const IO*>(isk ? p.k : p.q)[((int64_t)se.t0 + tau) * (isk ? p.k_stride : p.q_stride) + kc]);
          else
            keep[j] = se.has_init ? static_cast<float>(conv[((int64_t)se.slot * p.sh.Cd + ch) * (W - 1) + W - 1 + tau]) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) conv[((int64_t)slot * p.sh.Cd + ch) * (W - 1) + j] = from_f32<bf16>(keep[j]);
      }
    }
  };

  // ---------------------------------------------------------------- staging
  auto stage = [&](int c, int tau0, char* to) {
    const char* kq = p.kq + ((int64_t)c * p.sh.Hk + g) * St::KQ;
    const char* hd = p.head + ((int64_t)c * p.sh.Hv + h) * St::HEAD;
#pragma unroll
    for (int i = 0; i < (St::PIECES + kWalkWaves - 1) / kWalkWaves; ++i) {
      const int pc = i * kWalkWaves + wave;
      if (pc < St::PIECES)
        dma16((pc * 1024 < St::KIN ? kq + pc * 1024 : hd + (pc * 1024 - St::KIN)) + lane * 16, to + pc * 1024);
    }
    constexpr int PP = St::SLOT_BYTES / 16, EP = 16 / (int)sizeof(IO);   // 16-byte parts of a slot, elements of a part
    const int last = dv / EP - 1;
#pragma unroll
    for (int i = 0; i < St::V_OPS; ++i) {
      const int n = i * 64 + lane, sl = n / PP, part = c0 / EP + n % PP;
      int tau = tau0 - (W - 1) + (sl % 17 * 4 + sl / 17);   // beyond either end: a row of the sequence, masked later
      tau = tau < 0 ? 0 : tau >= se.len ? se.len - 1 : tau;
      dma16(vbase + (int64_t)tau * p.v_stride + (part < last ? part : last) * EP,
            to + St::KIN + St::HEAD + (wave * St::V_OPS + i) * 1024);
    }
  };

  GdnChunk ce = load_uniform<GdnChunk>((cchar*)(p.chunks + se.chunk0));
  stage(se.chunk0, ce.tau0, smem);
  for (int n = 0; n < se.nchunk; ++n) {
    const int c = se.chunk0 + n;
    const char* const st = smem + (NB == 2 ? (n & 1) * St::BYTES : 0);
    GdnChunk next = ce;
    if (n + 1 < se.nchunk) next = load_uniform<GdnChunk>((cchar*)(p.chunks + c + 1));
    wait_dma();
    __syncthreads();
    if (NB == 2 && n + 1 < se.nchunk) stage(c + 1, next.tau0, smem + ((n + 1) & 1) * St::BYTES);
    if (active) {
      const u16* const Kt = reinterpret_cast<const u16*>(st);
      const u16* const Qf = St::Q_IN ? Kt + NP * C * DK
                                     : reinterpret_cast<const u16*>(p.kq + ((int64_t)c * p.sh.Hk + g) * St::KQ) + NP * C * DK;
      const u16* const Tf = reinterpret_cast<const u16*>(st + St::KIN);
      const u16* const Af = Tf + gdn_t_bytes(NP) / 2;
      const float* const g1 = reinterpret_cast<const float*>(Tf + NP * kTri) + 4 * q4;
      const float* const g2 = reinterpret_cast<const float*>(Af + NP * kTri) + 4 * q4;
      const IO* const vs = reinterpret_cast<const IO*>(st + St::KIN + St::HEAD + wave * St::V_OPS * 1024) + l16;
      // SiLU(conv) of rows 16 rt + 4 q4 .. +3 of the lane's column
      auto conv_tile = [&](int rt) {
        float v[W + 3];
#pragma unroll
        for (int j = 0; j < W + 3; ++j) {
          const IO* vr = vs + ((j & 3) * 17 + 4 * rt + q4 + (j >> 2)) * 16;   // row 16 rt + 4 q4 + j - (W-1)
          const int tau = ce.tau0 + 16 * rt + 4 * q4 + j - (W - 1);
          float x = to_f32(*vr);
          if (rt == 0 && j < W - 1) {                    // rows ahead of the sequence: the window
#pragma unroll
            for (int i = 0; i < W - 1; ++i) x = tau == i - (W - 1) ? win[i] : x;
          }
          v[j] = x;
        }
        floatx4 o;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float x = bias;
#pragma unroll
          for (int j = 0; j < W; ++j) x += wt[j] * v[r + j];
          // a row behind the chunk, perhaps one of the next chunk, may hold a NaN, which must not reach this
          // chunk's end state
          o[r] = 16 * rt + 4 * q4 + r < ce.len ? silu(x) : 0.f;
        }
        return o;
      };
      float most = 0.f;
      Unit su = {1.f, 1.f};
      if constexpr (NP == 1) {
        most = column_max(largest(S));
        su = unit_of<14>(most);
      }
      // K S0 and Q S0
      floatx4 X[4], Y[4];
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) X[rt] = Y[rt] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const Op<NP> sf = acc_op<NP>(S[2 * ks] * su.inverse, S[2 * ks + 1] * su.inverse);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
          Op<NP> k;
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const u16* t = Kt + i * C * DK + (rt * NT + 2 * ks) * 256 + lane * 4;
            const u16x4 lo = *reinterpret_cast<const u16x4*>(t), hi = *reinterpret_cast<const u16x4*>(t + 256);
            k.p[i] = __builtin_bit_cast(typename Op<NP>::vec, u16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
          }
          const Op<NP> q = get_op<NP>(Qf, C * DK, rt * KS + ks, lane);
          X[rt] = mul(k, sf, X[rt]);
          Y[rt] = mul(q, sf, Y[rt]);
        }
      }
      // R = beta (V - e^g K S0)
      const float xs = NP == 1 ? su.size * unit : 1.f;
      floatx4 U[4];
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) {
        const floatx4 be = *reinterpret_cast<const floatx4*>(g1 + 16 * rt);
        const floatx4 bg = *reinterpret_cast<const floatx4*>(g1 + C + 16 * rt);
        U[rt] = be * conv_tile(rt) - bg * (X[rt] * xs);    // beta is 0 behind the chunk
      }
      // from here on R, U and the state are in the column's unit
      const float decay = g1[3 * C];
      Unit ru = {1.f, 1.f};
      if constexpr (NP == 1) ru = unit_of_r(column_max(largest(U)), decay * most * unit);
      const float keep = NP == 1 ? decay * finite(unit * ru.inverse) : decay;
      unit = NP == 1 ? ru.size : 1.f;
      // U = R + (T - I) R
      {
        if constexpr (NP == 1) {
#pragma unroll
          for (int rt = 0; rt < 4; ++rt) U[rt] = U[rt] * ru.inverse;
        }
        const Op<NP> rf[2] = {acc_op<NP>(U[0], U[1]), acc_op<NP>(U[2], U[3])};
        if constexpr (NP == 1) {
#pragma unroll
          for (int rt = 0; rt < 4; ++rt) U[rt] = U[rt] * kLift<NP>;
        }
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
#pragma unroll
          for (int ks = 0; ks <= rt / 2; ++ks) {
            const Op<NP> t = get_op<NP>(Tf, kTri, gdn_tri(rt, ks), lane);
            U[rt] = mul(t, rf[ks], U[rt]);
          }
      }
      // S1 = e^G S0 + K^T (e^(G-g) U)
      {
        floatx4 w[4];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
          const floatx4 eG = *reinterpret_cast<const floatx4*>(g1 + 2 * C + 16 * rt);
          w[rt] = U[rt] * eG;
        }
        const Op<NP> uf[2] = {acc_op<NP>(w[0], w[1]), acc_op<NP>(w[2], w[3])};
        const u16* const tr = Kt + ((l16 & 3) * 16 + 4 * q4 + (l16 >> 2)) * 4;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          S[i] = S[i] * keep;
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            Op<NP> k;
#pragma unroll
            for (int pl = 0; pl < NP; ++pl) k.p[pl] = tr_frag<typename Op<NP>::vec>(tr + pl * C * DK + (2 * ks * NT + i) * 256, NT * 256);
            S[i] = mul(k, uf[ks], S[i]);
          }
        }
      }
      // O = e^g Q S0 + q.k U + (Q K^T below the diagonal) U
      {
        constexpr float lower = 1.f / kLift<NP>;
        const Op<NP> uf[2] = {acc_op<NP>(U[0] * lower, U[1] * lower), acc_op<NP>(U[2] * lower, U[3] * lower)};
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
          const floatx4 eg = *reinterpret_cast<const floatx4*>(g2 + 16 * rt);
          const floatx4 qk = *reinterpret_cast<const floatx4*>(g2 + C + 16 * rt);
          floatx4 Z = qk * U[rt];
#pragma unroll
          for (int ks = 0; ks <= rt / 2; ++ks) {
            const Op<NP> a = get_op<NP>(Af, kTri, gdn_tri(rt, ks), lane);
            Z = mul(a, uf[ks], Z);
          }
          Y[rt] = eg * xs * Y[rt] + Z * (unit / kLift<NP>);
        }
      }
      pin(S);
      pin(Y);
      settle();
#pragma unroll
      for (int rt = 0; rt < 4; ++rt)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = 16 * rt + 4 * q4 + r;
          if (i < ce.len) {
            const int64_t at = ((int64_t)se.t0 + ce.tau0 + i) * p.o_stride + h * dv;
            if (has) store_any(p.o, at + col, Y[rt][r], NP == 1 ? 1 : p.o_bf16);
          }
        }
      if (ce.ckpt_slot >= 0) put_slot(ce.ckpt_slot, ce.tau0 + ce.len);
    }
    if (NB == 1 && n + 1 < se.nchunk) {
      __syncthreads();   // everyone is done with the stage
      stage(c + 1, next.tau0, smem);
    }
    ce = next;
  }
  if (active) put_slot(se.slot, se.len);
}

template <int DK, int W, int NP, typename IO> hipError_t launch_walk(const GdnPrefillParams& p, hipStream_t s) {
  typedef Stage<DK, NP, IO> St;
  constexpr int NB = 2 * St::BYTES <= (int)kMaxLdsBytes ? 2 : 1;
  const auto f = &walk_kernel<DK, W, NP, NB, IO>;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(f), hipFuncAttributeMaxDynamicSharedMemorySize,
                                           NB * St::BYTES);
  if (e != hipSuccess) return e;
  const int parts = (p.sh.dv + kWalkWaves * 16 - 1) / (kWalkWaves * 16), groups = p.num_seqs * p.sh.Hk;
  const int grid = (groups + 7) / 8 * 8 * (p.sh.Hv / p.sh.Hk) * parts;
  hipLaunchKernelGGL(f, dim3(grid), dim3(64 * kWalkWaves), NB * St::BYTES, s, p, parts, groups);
  return hipGetLastError();
}

// ------------------------------------------------------------------ walk with roles
// The walk for bf16 rows and dk <= 128, where one prompt's heads leave most of the chip idle and what
// counts is how fast one chunk follows another.  One workgroup of 8 waves per (sequence, value head,
// 32 columns of dv), whose waves take different parts of the work, one chunk apart:
//   waves 0-1  the state's chain of chunk n, 16 columns each: X = K S0, R, U, S1, in registers;
//   waves 2-3  the output of chunk n-1, two row tiles each, from S0 and U that the chain left in LDS;
//   waves 4-7  conv and SiLU of the v rows of chunk n+1, 16 rows each, and the windows of slots.
// Waves 2-7 also copy the operands of the next step from the workspace to LDS.  One barrier a step.
// The columns of tile ct are 2 l + ct, so that an output lane has two adjacent ones.
// Measured on 8192 rows of one sequence (128 workgroups): 1.5 us a step, bound by the instructions
// of the chain (38 MFMAs, two searches for a column's largest, some 95 LDS accesses) and what waits for
// the copies and the barrier.  With bf16 operands, T, U and Q K^T in two planes 1.7 us, in one plane 1.4 us;
// in that form one wave doing all the work of 16 columns took 4.2 us, these roles with the loads left to
// the compiler's order 2.7 us, and ten or twelve waves, which leave a wave 168 registers instead of
// 256, 2.0 us and more.  One workgroup's LDS is 133 KB at dk 128, so that the next one of a CU starts
// when this one ends.
template <int DK> struct Roles {
  static constexpr int A = 2 * C * DK + gdn_t_bytes(1);       // K, T, gates: the chain's, per chunk
  static constexpr int B = 2 * C * DK + gdn_a_bytes(1);       // Q, Q K^T, gates: the output's
  static constexpr int V = 2 * C * 16 * 4;                    // v rows [ct][64/16][64 lanes][4], then U, lifted
  static constexpr int S = 2 * DK * 16 * 2;                   // S0 operands [ct][dk/32][64 lanes][8]
  static constexpr int UN = 2 * 16 * 8;                       // [ct][16]: the units of S0 and of the lifted U
  // three places for v rows: the chain puts U where it found them, and the output reads that a step
  // later, while the rows after the next come in
  static constexpr int OFF_B = 2 * A, OFF_V = OFF_B + 2 * B, OFF_S = OFF_V + 3 * V, OFF_UN = OFF_S + 2 * S;
  static constexpr int BYTES = OFF_UN + 2 * UN;
  static_assert(BYTES <= (int)kMaxLdsBytes && A % 1024 == 0 && B % 1024 == 0, "LDS of a role walk workgroup");
};

// What the waves of a workgroup know of their unit.
struct RoleUnit {
  GdnSeq se;
  int g, h, rep, c0;     // key head, value head, value heads per key head, first column of dv
  int wave, lane, q4, l16;
  char* smem;
};

// `PIECES` <= 4 KiB from global memory to LDS, 16 bytes per lane: one address, offsets on both sides.
template <int PIECES> __device__ __forceinline__ void copy_run(const char* g, char* l) {
  const auto* from = (const __attribute__((address_space(1))) void*)g;
  auto* to = (__attribute__((address_space(3))) void*)l;
  constexpr int kPiece = 1024;   // bytes one instruction moves: 64 lanes of 16
  __builtin_amdgcn_global_load_lds(from, to, 16, 0, 0);
  if constexpr (PIECES > 1) __builtin_amdgcn_global_load_lds(from, to, 16, 1 * kPiece, 0);
  if constexpr (PIECES > 2) __builtin_amdgcn_global_load_lds(from, to, 16, 2 * kPiece, 0);
  if constexpr (PIECES > 3) __builtin_amdgcn_global_load_lds(from, to, 16, 3 * kPiece, 0);
}
// The copies of waves 2-7 at step n: the chain's operands of chunk n+1 and the output's of chunk n.
// WHO 0..5 has every sixth of the 4 KiB runs, numbered through K, T with gates, Q, the masked Q K^T
// with gates.
template <int DK, int WHO> __device__ __forceinline__ void role_copies(const GdnPrefillParams& p, const RoleUnit& u, int n) {
  typedef Roles<DK> Ro;
  constexpr int KB = 2 * C * DK / 1024, TB = gdn_t_bytes(1) / 1024, AB = gdn_a_bytes(1) / 1024;   // pieces
  constexpr int KR = (KB + 3) / 4, TR = (TB + 3) / 4, AR = (AB + 3) / 4;                          // runs
  const int64_t c = u.se.chunk0 + n;
  const int lo = u.lane * 16;
  if (n + 1 < u.se.nchunk) {
    const char* kq = p.kq + ((c + 1) * p.sh.Hk + u.g) * gdn_kq_bytes(DK, 1) + lo;
    const char* hd = p.head + ((c + 1) * p.sh.Hv + u.h) * gdn_head_bytes(1) + lo;
    char* to = u.smem + ((n + 1) & 1) * Ro::A;
#pragma unroll
    for (int r = 0; r < KR; ++r)
      if (r % 6 == WHO) copy_run<(KB < 4 ? KB : 4)>(kq + r * 4096, to + r * 4096);
#pragma unroll
    for (int r = 0; r < TR; ++r)
      if ((KR + r) % 6 == WHO) {
        if (4 * r + 4 <= TB) copy_run<4>(hd + r * 4096, to + KB * 1024 + r * 4096);
        else copy_run<(TB % 4 ? TB % 4 : 4)>(hd + r * 4096, to + KB * 1024 + r * 4096);
      }
  }
  if (n >= 0 && n < u.se.nchunk) {
    const char* kq = p.kq + (c * p.sh.Hk + u.g) * gdn_kq_bytes(DK, 1) + 2 * C * DK + lo;
    const char* hd = p.head + (c * p.sh.Hv + u.h) * gdn_head_bytes(1) + gdn_t_bytes(1) + lo;
    char* to = u.smem + Ro::OFF_B + (n & 1) * Ro::B;
#pragma unroll
    for (int r = 0; r < KR; ++r)
      if ((KR + TR + r) % 6 == WHO) copy_run<(KB < 4 ? KB : 4)>(kq + r * 4096, to + r * 4096);
#pragma unroll
    for (int r = 0; r < AR; ++r)
      if ((2 * KR + TR + r) % 6 == WHO) {
        if (4 * r + 4 <= AB) copy_run<4>(hd + r * 4096, to + KB * 1024 + r * 4096);
        else copy_run<(AB % 4 ? AB % 4 : 4)>(hd + r * 4096, to + KB * 1024 + r * 4096);
      }
  }
}
// Keeps the compiler from moving loads from one side to the other: operands are asked for ahead of
// the products that cover their latency.
__device__ __forceinline__ void fence_order() { __builtin_amdgcn_sched_barrier(0); }

template <int DK> __device__ __forceinline__ void chain_role(const GdnPrefillParams& p, const RoleUnit& u) {
  typedef Roles<DK> Ro;
  constexpr int KS = DK / 32, NT = DK / 16;
  const GdnSeq& se = u.se;
  const int lane = u.lane, q4 = u.q4, l16 = u.l16, dv = p.sh.dv;
  const int col = u.c0 + 2 * l16 + u.wave;
  const bool has = col < dv;
  bf16* const ssm = static_cast<bf16*>(p.ssm);
  floatx4 S[NT];      // in units of `unit`
  float unit = 1.f;
  {
    const bf16* sp = ssm + (((int64_t)se.slot * p.sh.Hv + u.h) * dv + (has ? col : dv - 1)) * DK + 4 * q4;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const u16x4 x = se.has_init ? *reinterpret_cast<const u16x4*>(sp + 16 * i) : u16x4{0, 0, 0, 0};
#pragma unroll
      for (int r = 0; r < 4; ++r) S[i][r] = static_cast<float>(__builtin_bit_cast(bf16, (u16)x[r]));
    }
  }
  auto put_state = [&](int slot) {
    if (!has) return;
    bf16* sp = ssm + (((int64_t)slot * p.sh.Hv + u.h) * dv + col) * DK + 4 * q4;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      u16x4 o;
#pragma unroll
      for (int r = 0; r < 4; ++r) o[r] = bits(from_f32<bf16>(S[i][r] * unit));
      *reinterpret_cast<u16x4*>(sp + 16 * i) = o;
    }
  };
  // Entries of the chunk table are read at the end of a step for the next one: a scalar load in flight
  // shares the counter of the LDS reads and, returning out of order, would make every wait for an
  // operand a wait for all of them.
  auto ckpt_of = [&](int n) {
    return load_uniform<GdnChunk>((cchar*)(p.chunks + se.chunk0 + (n < se.nchunk ? n : se.nchunk - 1))).ckpt_slot;
  };
  int ckpt = ckpt_of(0);
  __syncthreads();
  for (int n = 0; n < se.nchunk; ++n) {
    const int now = n & 1;
    const char* const sa = u.smem + now * Ro::A;
    const u16* const Kt = reinterpret_cast<const u16*>(sa) + lane * 4;
    const u16* const tr = reinterpret_cast<const u16*>(sa) + ((l16 & 3) * 16 + 4 * q4 + (l16 >> 2)) * 4;
    const u16* const Tf = reinterpret_cast<const u16*>(sa) + C * DK;
    const float* const g1 = reinterpret_cast<const float*>(Tf + kTri) + 4 * q4;
    char* const vs = u.smem + Ro::OFF_V + n % 3 * Ro::V + (u.wave * 4 * 64 + lane) * 16;
    u16* const sf = reinterpret_cast<u16*>(u.smem + Ro::OFF_S + now * Ro::S) + (u.wave * KS * 64 + lane) * 8;
    u16x8 k[KS][4];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) {
        const u16* t = Kt + (rt * NT + 2 * ks) * 256;
        const u16x4 lo = *reinterpret_cast<const u16x4*>(t), hi = *reinterpret_cast<const u16x4*>(t + 256);
        k[ks][rt] = u16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      }
    const float most = column_max(largest(S));
    const Unit su = unit_of<14>(most);
    const float xs = su.size * unit;
    f16x8 s0[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      s0[ks] = acc_op<1>(S[2 * ks] * su.inverse, S[2 * ks + 1] * su.inverse).p[0];
      *reinterpret_cast<f16x8*>(sf + ks * 512) = s0[ks];
    }
    fence_order();
    floatx4 be[4], bg[4], eG[4], v[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      v[rt] = *reinterpret_cast<const floatx4*>(vs + rt * 1024);
      be[rt] = *reinterpret_cast<const floatx4*>(g1 + 16 * rt);
      bg[rt] = *reinterpret_cast<const floatx4*>(g1 + C + 16 * rt);
    }
    fence_order();
    floatx4 X[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) X[rt] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) X[rt] = mfma(__builtin_bit_cast(f16x8, k[ks][rt]), s0[ks], X[rt]);
    fence_order();
    Op<1> t[kGdnTriFrags];
#pragma unroll
    for (int f = 0; f < kGdnTriFrags; ++f) t[f] = get_op<1>(Tf, kTri, f, lane);
    fence_order();
    floatx4 U[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) U[rt] = be[rt] * v[rt] - bg[rt] * (X[rt] * xs);   // R; beta is 0 behind the chunk
    // from here on R, U and the state are in the column's unit
    const float decay = g1[3 * C];
    const Unit ru = unit_of_r(column_max(largest(U)), decay * most * unit);
    const float keep = decay * finite(unit * ru.inverse);
    unit = ru.size;
    if (q4 == 0)
      *reinterpret_cast<floatx2*>(u.smem + Ro::OFF_UN + now * Ro::UN + (u.wave * 16 + l16) * 8) =
          floatx2{xs, unit / kLift<1>};
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) U[rt] = U[rt] * ru.inverse;
    const Op<1> r0 = acc_op<1>(U[0], U[1]), r1 = acc_op<1>(U[2], U[3]);
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) U[rt] = U[rt] * kLift<1>;
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) eG[rt] = *reinterpret_cast<const floatx4*>(g1 + 2 * C + 16 * rt);
    fence_order();
    // T R in an order that keeps products of one sum apart
    U[0] = mul(t[0], r0, U[0]);
    U[1] = mul(t[1], r0, U[1]);
    U[2] = mul(t[2], r0, U[2]);
    U[3] = mul(t[4], r0, U[3]);
    U[2] = mul(t[3], r1, U[2]);
    U[3] = mul(t[5], r1, U[3]);
    f16x8 kt[2][NT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) kt[ks][i] = tr_frag<f16x8>(tr + (2 * ks * NT + i) * 256, NT * 256);
#pragma unroll
    for (int i = 0; i < NT; ++i) S[i] = S[i] * keep;
    fence_order();
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      *reinterpret_cast<floatx4*>(vs + rt * 1024) = U[rt];
      U[rt] = U[rt] * eG[rt];
    }
    const Op<1> w[2] = {acc_op<1>(U[0], U[1]), acc_op<1>(U[2], U[3])};
    fence_order();
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int i = 0; i < NT; ++i) S[i] = mfma(kt[ks][i], w[ks].p[0], S[i]);
    pin(S);
    settle();
    if (ckpt >= 0) put_state(ckpt);
    ckpt = ckpt_of(n + 1);
    __syncthreads();
  }
  put_state(se.slot);
  __syncthreads();
}

template <int DK, int WHO> __device__ __forceinline__ void output_role(const GdnPrefillParams& p, const RoleUnit& u) {
  typedef Roles<DK> Ro;
  constexpr int KS = DK / 32;
  const GdnSeq& se = u.se;
  const int lane = u.lane, q4 = u.q4;
  // row tiles 0 and 3, or 1 and 2: three fragments of the masked Q K^T either way
  constexpr int RT[2] = {WHO, 3 - WHO};
  const bool has = u.c0 + 2 * u.l16 < p.sh.dv;
  uint32_t out[2][4];
  int64_t row = 0;
  int len = 0;
  bf16* const base = static_cast<bf16*>(p.o) + u.h * p.sh.dv + u.c0 + 2 * u.l16 + 4 * q4 * p.o_stride;
  auto store_out = [&]() {
    bf16* const to = base + row * p.o_stride;
    const int left = has ? len - 4 * q4 : 0;                    // this lane's row 16 rt + r is there if below it
    if (p.o_pairs) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (16 * RT[t] + r < left) *reinterpret_cast<uint32_t*>(to + (16 * RT[t] + r) * p.o_stride) = out[t][r];
    } else {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (16 * RT[t] + r < left) {
            u16* const w = reinterpret_cast<u16*>(to + (16 * RT[t] + r) * p.o_stride);
            w[0] = (u16)out[t][r];
            w[1] = (u16)(out[t][r] >> 16);
          }
    }
  };
  role_copies<DK, WHO>(p, u, -1);
  GdnChunk ce = {0, 0, 0, -1};                                   // chunk n - 1
  wait_dma();
  __syncthreads();
  for (int n = 0; n <= se.nchunk; ++n) {
    const int was = (n - 1) & 1;
    role_copies<DK, WHO>(p, u, n);
    if (n > 0) {
      // the rows of chunk n - 2 go out while the operands of chunk n - 1 come in
      const char* const sb = u.smem + Ro::OFF_B + was * Ro::B;
      const u16* const Qf = reinterpret_cast<const u16*>(sb);
      const u16* const Af = Qf + C * DK;
      const float* const g2 = reinterpret_cast<const float*>(Af + kTri) + 4 * q4;
      const u16* const sf = reinterpret_cast<const u16*>(u.smem + Ro::OFF_S + was * Ro::S);
      const char* const uf = u.smem + Ro::OFF_V + (n - 1) % 3 * Ro::V;
      f16x8 s0[KS][2], q[KS][2];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          s0[ks][t] = get_op<1>(sf, 0, t * KS + ks, lane).p[0];
          q[ks][t] = get_op<1>(Qf, 0, RT[t] * KS + ks, lane).p[0];
        }
      fence_order();
      store_out();
      floatx4 Y[2][2], Z[2][2];
#pragma unroll
      for (int t = 0; t < 2; ++t) Y[t][0] = Y[t][1] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int ct = 0; ct < 2; ++ct) Y[t][ct] = mfma(q[ks][t], s0[ks][ct], Y[t][ct]);
      floatx4 U[2][4], eg[2], qk[2];
      floatx2 unit[2];   // of S0 and of the lifted U
      Op<1> a[2], a1;
#pragma unroll
      for (int ct = 0; ct < 2; ++ct)
        unit[ct] = *reinterpret_cast<const floatx2*>(u.smem + Ro::OFF_UN + was * Ro::UN + (ct * 16 + u.l16) * 8);
#pragma unroll
      for (int ct = 0; ct < 2; ++ct)
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
          U[ct][rt] = *reinterpret_cast<const floatx4*>(uf + ((ct * 4 + rt) * 64 + lane) * 16);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int rt = RT[t];
        eg[t] = *reinterpret_cast<const floatx4*>(g2 + 16 * rt);
        qk[t] = *reinterpret_cast<const floatx4*>(g2 + C + 16 * rt);
        a[t] = get_op<1>(Af, kTri, gdn_tri(rt, 0), lane);
      }
      a1 = get_op<1>(Af, kTri, gdn_tri(RT[1], 1), lane);
      fence_order();
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) {
        constexpr float lower = 1.f / kLift<1>;
        const Op<1> u0 = acc_op<1>(U[ct][0] * lower, U[ct][1] * lower);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          Z[t][ct] = qk[t] * U[ct][RT[t]];
          Z[t][ct] = mul(a[t], u0, Z[t][ct]);
        }
        Z[1][ct] = mul(a1, acc_op<1>(U[ct][2] * lower, U[ct][3] * lower), Z[1][ct]);
      }
      pin(Z[0]);
      pin(Z[1]);
      settle();
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) Y[t][ct] = eg[t] * unit[ct][0] * Y[t][ct] + Z[t][ct] * unit[ct][1];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          out[t][r] = bits(from_f32<bf16>(Y[t][0][r])) | (uint32_t)bits(from_f32<bf16>(Y[t][1][r])) << 16;
      row = (int64_t)se.t0 + ce.tau0;
      len = ce.len;
    }
    if (n < se.nchunk) ce = load_uniform<GdnChunk>((cchar*)(p.chunks + se.chunk0 + n));
    wait_dma();
    __syncthreads();
  }
  store_out();
}

template <int DK, int W, int WHO> __device__ __forceinline__ void conv_role(const GdnPrefillParams& p, const RoleUnit& u) {
  typedef Roles<DK> Ro;
  const GdnSeq& se = u.se;
  const int lane = u.lane, q4 = u.q4, dv = p.sh.dv, c0 = u.c0;
  constexpr int rt = WHO - 2;
  bf16* const conv = static_cast<bf16*>(p.conv);
  // rows 16 rt + 4 q4 .. +3, columns c0 + 2 l and the next (dv is even)
  const int col = c0 + 2 * u.l16 < dv ? c0 + 2 * u.l16 : dv - 2;
  const int64_t vch = 2 * p.sh.Hk * DK + (int64_t)u.h * dv + col;   // conv channel
  const bf16* const vbase = static_cast<const bf16*>(p.v) + (int64_t)se.t0 * p.v_stride + u.h * dv;
  float wt[2][W], bias[2], win[2][W - 1];
  uint32_t rows[W + 3], ahead[W + 3];                               // raw rows, two columns each
  // the lane's rows of the chunk at tau0 and the W-1 ahead of them; beyond either end of the
  // sequence a row of it, which is masked or replaced later
  const bf16* const vlane = vbase + (16 * rt + 4 * q4 - (W - 1)) * p.v_stride + col;
  auto load_rows = [&](int tau0, uint32_t (&x)[W + 3]) {
    if (tau0 >= W - 1 && tau0 + C <= se.len) {
      const bf16* const from = vlane + (int64_t)tau0 * p.v_stride;
#pragma unroll
      for (int j = 0; j < W + 3; ++j) x[j] = *reinterpret_cast<const uint32_t*>(from + j * p.v_stride);
    } else {
#pragma unroll
      for (int j = 0; j < W + 3; ++j) {
        int tau = tau0 + 16 * rt + 4 * q4 + j - (W - 1);
        tau = tau < 0 ? 0 : tau >= se.len ? se.len - 1 : tau;
        x[j] = *reinterpret_cast<const uint32_t*>(vbase + (int64_t)tau * p.v_stride + col);
      }
    }
  };
  // SiLU(conv) of the rows held, of the chunk of `len` rows at tau0.  Rows behind the chunk, perhaps of
  // the next one, come out as 0: they may hold a NaN, which must not reach this chunk's end state.
  auto conv_rows = [&](int tau0, int len, char* to) {
    float x[2][W + 3];
#pragma unroll
    for (int j = 0; j < W + 3; ++j) {
      x[0][j] = __uint_as_float(rows[j] << 16);
      x[1][j] = __uint_as_float(rows[j] & 0xffff0000u);
    }
    if (tau0 < W - 1) {                                             // rows ahead of the sequence: the window
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        const int tau = tau0 + 16 * rt + 4 * q4 + j - (W - 1);
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
          x[0][j] = tau == i - (W - 1) ? win[0][i] : x[0][j];
          x[1][j] = tau == i - (W - 1) ? win[1][i] : x[1][j];
        }
      }
    }
#pragma unroll
    for (int ct = 0; ct < 2; ++ct) {
      floatx4 o;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float y = bias[ct];
#pragma unroll
        for (int j = 0; j < W; ++j) y += wt[ct][j] * x[ct][r + j];
        o[r] = 16 * rt + 4 * q4 + r < len ? silu(y) : 0.f;
      }
      *reinterpret_cast<floatx4*>(to + ((ct * 4 + rt) * 64 + lane) * 16) = o;
    }
  };
  // window of a slot after `end` rows: v channels by wave 4, the key head's q and k by waves 5-7 of
  // the workgroup of its first columns
  auto put_window = [&](int slot, int end) {
    const bool qk = rt > 0;
    if (qk && (c0 != 0 || u.h % u.rep != 0)) return;
    const int n = qk ? 2 * DK : (dv - c0 < 32 ? dv - c0 : 32);
    for (int i = qk ? (rt - 1) * 64 + lane : lane; i < n; i += qk ? 192 : 64) {
      const bf16* src;
      int64_t stride, ch;
      if (qk) {
        const int kc = u.g * DK + (i >= DK ? i - DK : i);
        stride = i >= DK ? p.k_stride : p.q_stride;
        ch = (i >= DK ? p.sh.Hk * DK : 0) + kc;
        src = static_cast<const bf16*>(i >= DK ? p.k : p.q) + (int64_t)se.t0 * stride + kc;
      } else {
        src = vbase + c0 + i;
        stride = p.v_stride;
        ch = 2 * p.sh.Hk * DK + (int64_t)u.h * dv + c0 + i;
      }
      bf16 keep[W - 1];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        const int tau = end - (W - 1) + j;
        keep[j] = tau >= 0 ? src[tau * stride]
                  : se.has_init ? conv[((int64_t)se.slot * p.sh.Cd + ch) * (W - 1) + W - 1 + tau] : static_cast<bf16>(0.f);
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j) conv[((int64_t)slot * p.sh.Cd + ch) * (W - 1) + j] = keep[j];
    }
  };
  auto chunk = [&](int n) { return load_uniform<GdnChunk>((cchar*)(p.chunks + se.chunk0 + n)); };

  load_rows(0, rows);
  role_copies<DK, WHO>(p, u, -1);
#pragma unroll
  for (int ct = 0; ct < 2; ++ct) {
#pragma unroll
    for (int j = 0; j < W; ++j) wt[ct][j] = p.conv_w[(vch + ct) * W + j];
    bias[ct] = p.conv_b ? p.conv_b[vch + ct] : 0.f;
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      win[ct][j] = se.has_init ? static_cast<float>(conv[((int64_t)se.slot * p.sh.Cd + vch + ct) * (W - 1) + j]) : 0.f;
  }
  GdnChunk ce = chunk(0), next = ce, after = ce;
  conv_rows(0, ce.len, u.smem + Ro::OFF_V);
  if (se.nchunk > 1) {
    next = chunk(1);
    load_rows(next.tau0, rows);
  }
  if (se.nchunk > 2) after = chunk(2);
  wait_dma();
  __syncthreads();
  for (int n = 0; n <= se.nchunk; ++n) {
    role_copies<DK, WHO>(p, u, n);
    if (n + 2 < se.nchunk) load_rows(after.tau0, ahead);
    if (n + 1 < se.nchunk) conv_rows(next.tau0, next.len, u.smem + Ro::OFF_V + (n + 1) % 3 * Ro::V);
    if (n < se.nchunk && ce.ckpt_slot >= 0) put_window(ce.ckpt_slot, ce.tau0 + ce.len);
#pragma unroll
    for (int j = 0; j < W + 3; ++j) rows[j] = ahead[j];
    ce = next;
    next = after;
    if (n + 3 < se.nchunk) after = chunk(n + 3);
    wait_dma();
    __syncthreads();
  }
  put_window(se.slot, se.len);
}

template <int DK, int W>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2)))
void role_walk_kernel(GdnPrefillParams p, int parts, int groups) {
  extern __shared__ char smem[];
  RoleUnit u;
  u.smem = smem;
  u.lane = threadIdx.x & 63;
  u.q4 = u.lane >> 4;
  u.l16 = u.lane & 15;
  u.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  u.rep = p.sh.Hv / p.sh.Hk;
  // workgroups of one (sequence, key head) on one XCD, as above
  const int per = u.rep * parts, turn = blockIdx.x >> 3;
  const int grp = turn / per * 8 + (blockIdx.x & 7), in = turn % per;
  if (grp >= groups) return;
  u.g = grp % p.sh.Hk;
  u.h = u.g * u.rep + in / parts;
  u.se = load_uniform<GdnSeq>((cchar*)(p.seqs + grp / p.sh.Hk));
  if (u.se.nchunk == 0) return;
  u.c0 = in % parts * 32;
  // every role passes nchunk + 2 barriers
  switch (u.wave) {
    case 0:
    case 1: chain_role<DK>(p, u); break;
    case 2: output_role<DK, 0>(p, u); break;
    case 3: output_role<DK, 1>(p, u); break;
    case 4: conv_role<DK, W, 2>(p, u); break;
    case 5: conv_role<DK, W, 3>(p, u); break;
    case 6: conv_role<DK, W, 4>(p, u); break;
    default: conv_role<DK, W, 5>(p, u);
  }
}

template <int DK, int W, int NP, typename IO> hipError_t launch_prep(const PrepArgs& a, hipStream_t s) {
  constexpr size_t lds = sizeof(PrepLds<DK, NP>);
  static_assert(lds <= kMaxLdsBytes, "prep_kernel LDS");
  const auto f = &prep_kernel<DK, W, NP, IO>;
  if (lds > 65536) {
    const hipError_t e =
        hipFuncSetAttribute(reinterpret_cast<const void*>(f), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  const int units = a.p.num_chunks * a.p.sh.Hk + (a.p.tab_inline ? 1 : 0);
  hipLaunchKernelGGL(f, dim3(units), dim3(kPrepThreads), lds, s, a);
  return hipGetLastError();
}

template <int DK, int W> hipError_t launch_role_walk(const GdnPrefillParams& p, hipStream_t s) {
  const auto f = &role_walk_kernel<DK, W>;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(f), hipFuncAttributeMaxDynamicSharedMemorySize,
                                           Roles<DK>::BYTES);
  if (e != hipSuccess) return e;
  const int parts = (p.sh.dv + 31) / 32, groups = p.num_seqs * p.sh.Hk;
  const int grid = (groups + 7) / 8 * 8 * (p.sh.Hv / p.sh.Hk) * parts;
  hipLaunchKernelGGL(f, dim3(grid), dim3(512), Roles<DK>::BYTES, s, p, parts, groups);
  return hipGetLastError();
}

template <int DK, int W, int NP, typename IO> hipError_t launch_io(const PrepArgs& a, hipStream_t s) {
  const hipError_t e = launch_prep<DK, W, NP, IO>(a, s);
  if (e != hipSuccess) return e;
  // dk 256 leaves no room for the roles' stages in LDS, three planes neither
  if constexpr (NP == 1 && DK <= 128) return launch_role_walk<DK, W>(a.p, s);
  else return launch_walk<DK, W, NP, IO>(a.p, s);
}
template <int DK, int W, int NP> hipError_t launch(const PrepArgs& a, hipStream_t s) {
  if constexpr (NP == 1) return launch_io<DK, W, 1, bf16>(a, s);
  else return a.p.io_bf16 ? launch_io<DK, W, NP, bf16>(a, s) : launch_io<DK, W, NP, float>(a, s);
}
template <int DK, int NP> hipError_t launch_w(const PrepArgs& a, hipStream_t s) {
  switch (a.p.sh.W) {
    case 2: return launch<DK, 2, NP>(a, s);
    case 3: return launch<DK, 3, NP>(a, s);
    case 4: return launch<DK, 4, NP>(a, s);
    default: return hipErrorInvalidValue;
  }
}
template <int NP> hipError_t launch_dk(const PrepArgs& a, hipStream_t s) {
  switch (a.p.sh.dk) {
    case 32: return launch_w<32, NP>(a, s);
    case 64: return launch_w<64, NP>(a, s);
    case 128: return launch_w<128, NP>(a, s);
    case 256: return launch_w<256, NP>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_gdn_prefill(const GdnPrefillParams& p, const void* tables, bool split, hipStream_t s) {
  PrepArgs a;
  a.p = p;
  if (p.tab_inline > 0) memcpy(a.tab, tables, p.tab_inline);
  return split ? launch_dk<kGdnSplitPlanes>(a, s) : launch_dk<1>(a, s);
}

}  // namespace m2

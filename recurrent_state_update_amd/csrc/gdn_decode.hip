// Gated delta rule, recurrent form over a slot pool: one token, or up to 8 draft tokens, per
// sequence, gfx950.
//
// Per value head h of key head g = h / (Hv/Hk), with S the (dv, dk) state of the row's slot:
//   [q | k | v] = SiLU(conv window)      q^ = q / |q| / sqrt(dk)     k^ = k / |k|
//   alpha = exp(A softplus(a + dt_bias))  beta = sigmoid(b)
//   S' = alpha S + d k^T,  d = beta (v - alpha S k^)                 o = S' q^
// The readout needs no second pass over the new state: with s = S k^ and t = S q^ taken together,
//   d = beta (v - alpha s),  o = alpha t + d (k^ . q^),  S' = alpha S + d k^T,
// so each state row is read once, reduced twice over its dk values and written once.
//
// One workgroup per (sequence, key head): the value heads of a key head share its q and k, and one
// workgroup owns the conv windows of all channels it reads, which it shifts in place.  Phase 1
// (conv, SiLU, norms, gates) stages K tokens in LDS while the first state tile is already on its
// way; phase 2 streams the state with 16-byte accesses, dk/8 lanes to a row.  What bounds it is
// the state's trip through HBM: one read and, per token, one write.  At 32 value heads of 128 x 128:
// 256 sequences 102 us (569 MB, 5.6 TB/s), 64 sequences x 8 tokens 135 us (645 MB, nine tenths of it
// writes, 4.8 TB/s); one sequence is a launch and one pass of latency.
#include "device_common.h"
#include "gdn.h"

namespace m2 {

// Threads of a workgroup.  A single token streams best from small workgroups that hold the next tile
// already (256 sequences of the wide layer: 102 us; with 128 or 512 threads 108, with 256 and no tile
// held 103); with several tokens a tile is worked on for longer and its latency counts (64 x 8 tokens:
// 135 us with 512 threads, 144 with 256, 152 with 1024).
constexpr int kGdnDecodeThreads = 256, kGdnMultiThreads = 512;

bool gdn_supported(int dk, int dv, int W) {
  return (dk == 32 || dk == 64 || dk == 128 || dk == 256) && dv >= 16 && dv % 16 == 0 && W >= 2 && W <= 4;
}

namespace {

// A wave-uniform int32 through the constant address space (a scalar load).
__device__ __forceinline__ int uniform_i32(const int32_t* p) {
  typedef const __attribute__((address_space(4))) int32_t cint;
  return *(const cint*)p;
}

__device__ __forceinline__ float sigmoid(float v) { return __builtin_amdgcn_rcpf(1.0f + __expf(-v)); }

// DK: head_k_dim.  MULTI: K tokens with a snapshot slot each; else one token in place.
template <int DK, int W, bool MULTI>
__global__ __launch_bounds__(MULTI ? kGdnMultiThreads : kGdnDecodeThreads) void gdn_decode_kernel(GdnDecodeParams p) {
  constexpr int THREADS = MULTI ? kGdnMultiThreads : kGdnDecodeThreads;
  constexpr int LPR = DK / 8;                     // lanes per state row
  constexpr int RPI = 64 / LPR;                   // rows per wave-wide access
  constexpr int U = DK / 16 > 8 ? 8 : DK / 16;    // accesses in flight per lane
  constexpr int RB = RPI * U;                     // rows per tile (32; 16 for dk 256)
  static_assert(U <= LPR, "one readout per lane and tile");
  const int b = blockIdx.x, g = blockIdx.y;       // rows fastest
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int nwaves = THREADS / 64;
  const int K = MULTI ? p.K : 1;
  const int rep = p.Hv / p.Hk, dv = p.dv, nv = rep * dv;
  const int slot = uniform_i32(p.slots_in + b);

  if (slot < 0 || slot >= p.num_slots) {          // padding row: no pool access, zero outputs
    for (int t = 0; t < K; ++t)
      for (int i = tid; i < nv; i += THREADS)
        store_any(p.o, ((int64_t)b * K + t) * p.o_stride + (int64_t)g * nv + i, 0.f, p.o_bf16);
    return;
  }

  extern __shared__ float smem[];
  const int trow = 2 * DK + nv;                   // per token: q^, k^, v
  float* s_act = smem;                            // [K][trow]
  float* s_alpha = s_act + (size_t)K * trow;      // [K][rep]
  float* s_beta = s_alpha + K * rep;              // [K][rep]
  float* s_kq = s_beta + K * rep;                 // [K]

  // ---------------------------------------------------------------- first state tile on its way
  const int sub = lane % LPR, rsub = lane / LPR, n0 = sub * 8;
  bf16* const ssm = static_cast<bf16*>(p.ssm);
  const int64_t head0 = (int64_t)g * rep;
  const bf16* const base = ssm + ((int64_t)slot * p.Hv + head0) * dv * DK;
  const int nbat = (dv + RB - 1) / RB;
  const int ntile = rep * nbat;
  bf16x8 data[U], next[U];   // the tile in use and the one after it
  auto load_tile = [&](int t, bf16x8 (&data)[U]) {
    const int hl = t / nbat, r0 = (t % nbat) * RB;
    const bf16* st = base + (int64_t)hl * dv * DK;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int row = r0 + j * RPI + rsub;
      if (row < dv) data[j] = __builtin_nontemporal_load(reinterpret_cast<const bf16x8*>(st + (int64_t)row * DK + n0));
    }
  };
  if (wave < ntile) load_tile(wave, next);

  // ---------------------------------------------------------------- conv, norms, gates
  // Wave 0 takes q (its first dk/8 lanes) and k (the next dk/8), the other waves v, 8 channels a
  // thread.
  const int cd = 2 * p.Hk * DK + p.Hv * dv;
  const bool qk = wave == 0;
  for (int c = qk ? lane * 8 : (tid - 64) * 8; c < (qk ? 2 * DK : nv); c += qk ? 512 : (THREADS - 64) * 8) {
    const void* src;
    int64_t col, stride;
    int gc;
    if (qk && c < DK) {
      col = (int64_t)g * DK + c, src = p.q, stride = p.q_stride, gc = (int)col;
    } else if (qk) {
      col = (int64_t)g * DK + c - DK, src = p.k, stride = p.k_stride, gc = p.Hk * DK + (int)col;
    } else {
      col = (int64_t)g * nv + c, src = p.v, stride = p.v_stride, gc = 2 * p.Hk * DK + (int)col;
    }
    // 8 channels x (W-1) window values, contiguous and 16-byte aligned
    float win[8 * (W - 1)];
    const bf16x8* wp = reinterpret_cast<const bf16x8*>(static_cast<const bf16*>(p.conv) + ((int64_t)slot * cd + gc) * (W - 1));
#pragma unroll
    for (int v = 0; v < W - 1; ++v) {
      const bf16x8 x = wp[v];
#pragma unroll
      for (int e = 0; e < 8; ++e) win[8 * v + e] = static_cast<float>(x[e]);
    }
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
    for (int t = 0; t < K; ++t) {
      float u[8], act[8];
      load8_any(src, ((int64_t)b * K + t) * stride + col, p.io_bf16, u);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float x = bias[e];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) x += wt[e * W + j] * win[e * (W - 1) + j];
        x += wt[e * W + W - 1] * u[e];
        act[e] = silu(x);
        // the window after this token, in the slot's type: the next token reads it so
#pragma unroll
        for (int j = 0; j < W - 2; ++j) win[e * (W - 1) + j] = win[e * (W - 1) + j + 1];
        win[e * (W - 1) + W - 2] = static_cast<float>(from_f32<bf16>(u[e]));
      }
      const int so = MULTI ? uniform_i32(p.slots_out + (int64_t)b * K + t) : slot;
      if (so >= 0 && so < p.num_slots) {
        bf16x8* op = reinterpret_cast<bf16x8*>(static_cast<bf16*>(p.conv) + ((int64_t)so * cd + gc) * (W - 1));
#pragma unroll
        for (int v = 0; v < W - 1; ++v) {
          bf16x8 x;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = from_f32<bf16>(win[8 * v + e]);
          op[v] = x;
        }
      }
      float* dst = s_act + (size_t)t * trow + (qk ? c : 2 * DK + c);
      if (qk) {
        // norms over the dk/8 lanes of q and of k; the q lanes also carry 1/sqrt(dk)
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += act[e] * act[e];
        const float rn = __builtin_amdgcn_rsqf(group_sum<LPR>(ss) + 1e-6f) * (c < DK ? __builtin_amdgcn_rsqf((float)DK) : 1.f);
        float kq = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          act[e] *= rn;
          kq += act[e] * __shfl_xor(act[e], LPR);
        }
        kq = group_sum<LPR>(kq);
        if (lane == 0) s_kq[t] = kq;
      }
#pragma unroll
      for (int e = 0; e < 8; e += 4) *reinterpret_cast<floatx4*>(dst + e) = floatx4{act[e], act[e + 1], act[e + 2], act[e + 3]};
    }
  }
  for (int i = tid; i < K * rep; i += THREADS) {
    const int t = i / rep, h = g * rep + i % rep;
    const int64_t r = (int64_t)b * K + t;
    s_alpha[i] = expf(p.A[h] * softplus(load_any(p.a, r * p.a_stride + h, p.io_bf16) + p.dt_bias[h]));
    s_beta[i] = sigmoid(load_any(p.b, r * p.b_stride + h, p.io_bf16));
  }
  __syncthreads();

  // ---------------------------------------------------------------- state
  for (int ti = wave; ti < ntile; ti += nwaves) {
#pragma unroll
    for (int j = 0; j < U; ++j) data[j] = next[j];
    if (ti + nwaves < ntile) load_tile(ti + nwaves, next);
    const int hl = ti / nbat, r0 = (ti % nbat) * RB;
    for (int t = 0; t < K; ++t) {
      const float* act = s_act + (size_t)t * trow;
      float qv[8], kv[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        qv[e] = act[n0 + e];
        kv[e] = act[DK + n0 + e];
      }
      const float alpha = s_alpha[t * rep + hl], beta = s_beta[t * rep + hl], kq = s_kq[t];
      const float* vs = act + 2 * DK + hl * dv;
      const int so = MULTI ? uniform_i32(p.slots_out + (int64_t)b * K + t) : slot;
      const bool keep = so >= 0 && so < p.num_slots;
      bf16* const ost = ssm + ((int64_t)(keep ? so : 0) * p.Hv + head0 + hl) * dv * DK;
      float out = 0.f;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int row = r0 + j * RPI + rsub;
        float s = 0.f, tq = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = to_f32(data[j][e]);
          s += x * kv[e];
          tq += x * qv[e];
        }
        s = group_sum<LPR>(s);
        tq = group_sum<LPR>(tq);
        const float d = row < dv ? beta * (vs[row] - alpha * s) : 0.f;
        if (sub == j) out = alpha * tq + d * kq;
        bf16x8 nvv;
#pragma unroll
        for (int e = 0; e < 8; ++e) nvv[e] = from_f32<bf16>(alpha * to_f32(data[j][e]) + d * kv[e]);
        if (MULTI) data[j] = nvv;
        if (keep && row < dv) __builtin_nontemporal_store(nvv, reinterpret_cast<bf16x8*>(ost + (int64_t)row * DK + n0));
      }
      const int row = r0 + sub * RPI + rsub;
      if (sub < U && row < dv)
        store_any(p.o, ((int64_t)b * K + t) * p.o_stride + (head0 + hl) * dv + row, out, p.o_bf16);
    }
  }
}

template <int DK, int W, bool MULTI> hipError_t launch(const GdnDecodeParams& p, int batch, hipStream_t s) {
  const int rep = p.Hv / p.Hk;
  const size_t lds = gdn_decode_lds_bytes(rep, p.dv, DK, p.K);
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&gdn_decode_kernel<DK, W, MULTI>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((gdn_decode_kernel<DK, W, MULTI>), dim3(batch, p.Hk), dim3(MULTI ? kGdnMultiThreads : kGdnDecodeThreads), lds, s, p);
  return hipGetLastError();
}
template <int DK, bool MULTI> hipError_t launch_w(const GdnDecodeParams& p, int W, int batch, hipStream_t s) {
  switch (W) {
    case 2: return launch<DK, 2, MULTI>(p, batch, s);
    case 3: return launch<DK, 3, MULTI>(p, batch, s);
    case 4: return launch<DK, 4, MULTI>(p, batch, s);
    default: return hipErrorInvalidValue;
  }
}
template <bool MULTI> hipError_t launch_dk(const GdnDecodeParams& p, int dk, int W, int batch, hipStream_t s) {
  switch (dk) {
    case 32: return launch_w<32, MULTI>(p, W, batch, s);
    case 64: return launch_w<64, MULTI>(p, W, batch, s);
    case 128: return launch_w<128, MULTI>(p, W, batch, s);
    case 256: return launch_w<256, MULTI>(p, W, batch, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_gdn_decode(const GdnDecodeParams& p, int dk, int W, int batch, bool multi, hipStream_t s) {
  if (batch == 0) return hipSuccess;
  return multi ? launch_dk<true>(p, dk, W, batch, s) : launch_dk<false>(p, dk, W, batch, s);
}

}  // namespace m2

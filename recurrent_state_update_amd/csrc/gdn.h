// Internal launch interface between the C ABI (api.cpp) and the gfx950 gated-delta-rule kernels.
#pragma once
#include "prefill.h"

namespace m2 {

// Shape of a gated-delta layer: Hv value heads of dv, Hk key heads of dk, conv width W over the
// Cd = 2 Hk dk + Hv dv channels [q | k | v].
struct GdnShape {
  int Hv, Hk, dv, dk, W, Cd;
};

// One decode step (K = 1, slots_out = slots_in) or a multi-token one.  ssm/conv point at the
// layer's first slot (both bf16).  Rows b*K + t of q, k, v, a, b and o.
struct GdnDecodeParams {
  void* ssm;
  void* conv;
  int num_slots;
  int io_bf16, o_bf16;
  int Hv, Hk, dv;
  int K;
  const int32_t* slots_in;
  const int32_t* slots_out;
  const void* q;
  const void* k;
  const void* v;
  const void* a;
  const void* b;
  int64_t q_stride, k_stride, v_stride, a_stride, b_stride;
  void* o;
  int64_t o_stride;
  const float* A;
  const float* dt_bias;
  const float* conv_w;
  const float* conv_b;   // may be NULL
};
bool gdn_supported(int dk, int dv, int W);
// LDS of one decode workgroup for K tokens: per token the normalised q and k, the group's v, per
// head alpha and beta, and k.q.
inline size_t gdn_decode_lds_bytes(int rep, int dv, int dk, int K) {
  return sizeof(float) * (size_t)K * (2 * (size_t)dk + (size_t)rep * dv + 2 * (size_t)rep + 1);
}
hipError_t launch_gdn_decode(const GdnDecodeParams& p, int dk, int W, int batch, bool multi, hipStream_t s);

// Chunked prefill: sequences in chunks of at most kGdnChunk rows.
constexpr int kGdnChunk = 64;
using GdnSeq = SeqEntry;   // first packed row, rows, final slot, seed from slot, first chunk, chunks
struct GdnChunk {   // one per chunk
  int32_t seq, tau0, len, ckpt_slot;  // entry of its sequence, offset inside it, rows, -1 or a slot
};
// Operands of one chunk in the workspace, in 1 KiB pieces as the walk's waves take them: one plane in
// fp16, or three in bf16 whose sum is the fp32 value:
//   per key head   K [planes][64/16][dk/16][64 lanes][4]: the 16 x 16 tile (rt, dt) of the rows, lane l
//                  holds row l % 16, columns 4 (l / 16) ..+3
//                  Q [planes][64/16][dk/32][64 lanes][8]: MFMA fragments
//   per value head T and the masked Q K^T, both below the diagonal, [planes][6][64 lanes][8]: fragments
//                  of the 16-row tile rt, 32-column steps 0 .. rt/2; behind T the gates of the
//                  state's chain (beta, beta e^g, e^(G-g), e^G), behind Q K^T those of the output
//                  (e^g, q.k), kGdnChunk floats each.
constexpr int kGdnTriFrags = 6;
__host__ __device__ constexpr int gdn_tri(int rt, int ks) { return rt < 2 ? rt : 2 * rt - 2 + ks; }
constexpr int kGdnSplitPlanes = 3;
// bytes per (chunk, key head) and per (chunk, value head)
__host__ __device__ constexpr int gdn_kq_bytes(int dk, int planes) { return 2 * planes * kGdnChunk * dk * 2; }
__host__ __device__ constexpr int gdn_t_bytes(int planes) { return (planes * kGdnTriFrags + 1) * 1024; }
__host__ __device__ constexpr int gdn_a_bytes(int planes) { return gdn_t_bytes(planes); }
__host__ __device__ constexpr int gdn_head_bytes(int planes) { return gdn_t_bytes(planes) + gdn_a_bytes(planes); }

struct GdnPrefillParams {
  void* ssm;
  void* conv;
  int io_bf16, o_bf16;
  GdnShape sh;
  int num_seqs, num_chunks;
  int o_pairs;                 // bf16 o: two adjacent elements may be stored as one dword
  const GdnSeq* seqs;
  const GdnChunk* chunks;
  int tab_chunks;              // byte offset of the chunk table from the sequence table
  int tab_inline;              // > 0: the tables ride in the first launch's arguments
  const void* q;
  const void* k;
  const void* v;
  const void* a;
  const void* b;
  int64_t q_stride, k_stride, v_stride, a_stride, b_stride;
  void* o;
  int64_t o_stride;
  const float* A;
  const float* dt_bias;
  const float* conv_w;
  const float* conv_b;         // may be NULL
  char* kq;                    // workspace: [chunks][Hk][gdn_kq_bytes]
  char* head;                  // [chunks][Hv][gdn_head_bytes]
};
// Tables of up to kGdnInlineBytes travel inside the first launch's kernel arguments (`tables`, when
// p.tab_inline > 0).  split: operands of three planes.
constexpr int kGdnInlineBytes = kInlineTableBytes;
hipError_t launch_gdn_prefill(const GdnPrefillParams& p, const void* tables, bool split, hipStream_t s);

}  // namespace m2

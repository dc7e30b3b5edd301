// nq_internal.h -- launch descriptors shared by the C ABI layer (nq_abi.cu)
// and the kernel files.  Arguments are validated by the ABI layer before any
// launcher below is called.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/nq.h"
#include "nq_device.cuh"

namespace nq {

// Heads per CTA of the tiled kernels (one warp per head): the largest divisor
// of the head count up to 8.
inline int pick_head_group(int heads) {
  for (int g = 8; g >= 1; --g)
    if (heads % g == 0) return g;
  return 1;
}

// Division by a fixed divisor for numerators below 2^31 (round-up method of
// Granlund and Montgomery): q = (n * m) >> (31 + l), l = ceil(log2 d),
// m = floor(2^(31+l) / d) + 1.
struct FastDiv {
  uint64_t m;
  uint32_t d, shift;
};

inline FastDiv make_fastdiv(uint32_t d) {
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  FastDiv f;
  f.d = d;
  f.shift = 31 + l;
  f.m = ((1ull << f.shift) / d) + 1;
  return f;
}

__device__ __forceinline__ uint32_t fdiv(uint32_t n, const FastDiv& f) {
  return static_cast<uint32_t>((static_cast<uint64_t>(n) * f.m) >> f.shift);
}

struct EncodeLaunch {
  const void* K;
  nq_kv_strides ks;
  const void* V;
  nq_kv_strides vs;
  int units, heads;
  int64_t T_in, n;
  const int32_t* kept;
  int64_t kept_stride;
  int64_t pos_base;
  const float* rope_tab;
  int64_t rope_max_pos;
  nq_packed k_out, v_out;  // exact layout: meta points to the uint16 scales
  int64_t slot0;
  bool exact;
};

struct DecodeLaunch {
  nq_packed k_in, v_in;  // exact layout: meta points to the uint16 scales
  bool exact;
  int units, heads;
  int64_t n, slot0;
  const int32_t* positions;
  int64_t pos_stride;
  int64_t pos_base;
  const float* rope_tab;
  int64_t rope_max_pos;
  void* K_out;
  nq_kv_strides kos;
  void* V_out;
  nq_kv_strides vos;
};

struct AttendLaunch {
  const float* q;
  int units, heads, G;
  nq_packed k_in, v_in;
  int64_t n, slot0;
  const int32_t* positions;
  int64_t pos_stride, pos_base;
  const float* rope_tab;
  int64_t rope_max_pos;
  float scale;
  float* out;
  float* lse;
  void* ws;
};

struct EncodeSlotsLaunch {
  const void* K;
  nq_kv_strides ks;
  const void* V;
  nq_kv_strides vs;
  int heads;
  int64_t rows;
  const int32_t* slots;
  const int32_t* positions;
  int page_size;
  int64_t pages;
  const float* rope_tab;
  int64_t rope_max_pos;
  nq_packed k_out, v_out;
};

struct PageTablesLaunch {
  const int32_t *lens, *counts;
  int requests, page_size;
  const int32_t* free_pages;
  int64_t n_free;
  const int32_t* taken;
  int32_t* table;
  int64_t table_stride;
  int32_t *lens_out, *starts, *slots, *positions;
  int64_t max_rows;
  int32_t* used;
};

struct NormRopeLaunch {
  const void *q, *k;
  nq_kv_strides qs, ks;
  int q_heads, k_heads;
  bool in_f32, q_f32, k_f32;
  int units;
  int64_t rows;
  const float *q_weight, *k_weight;
  float eps;
  const int32_t* positions;
  int64_t pos_stride, pos_base;
  const float* rope_tab;
  int64_t rope_max_pos;
  void *q_out, *k_out;
  nq_kv_strides qos, kos;
};

struct TreeLaunch {
  const void *q, *K_new, *V_new;
  nq_kv_strides qs, kns, vns;
  int units, heads, G, nodes;
  nq_packed k_in, v_in;
  int64_t n;
  const int32_t* lens;
  const int32_t* table;
  int64_t table_stride;
  int page_size;
  int64_t pages;
  const int32_t* positions;
  int64_t pos_stride, pos_base;
  const float* rope_tab;
  int64_t rope_max_pos;
  const uint64_t* mask;
  int64_t mask_stride;
  float scale;
  void* out;
  nq_kv_strides os;
  float* lse;
  void* ws;
};

cudaError_t launch_encode(const EncodeLaunch& L, cudaStream_t stream);
cudaError_t launch_decode(const DecodeLaunch& L, cudaStream_t stream);
cudaError_t launch_encode_slots(const EncodeSlotsLaunch& L, cudaStream_t stream);
cudaError_t launch_page_tables(const PageTablesLaunch& L, cudaStream_t stream);
cudaError_t launch_norm_rope(const NormRopeLaunch& L, cudaStream_t stream);
size_t tree_workspace_bytes(int units, int heads, int G, int nodes, int64_t n, bool shared,
                            bool ragged);
int64_t tree_ctas(int units, int heads, int G, int nodes, int64_t n, bool ragged);  // of its largest launch
cudaError_t tree_read_clear_error(uint32_t* flags);  // after a synchronisation
cudaError_t launch_tree_attend(const TreeLaunch& L, cudaStream_t stream);

cudaError_t codec_read_clear_error(uint32_t* flags);
// Decode engine (nq_decode_engine values), read at each decode launch.
void set_decode_engine(int engine);
int decode_engine();
size_t attend_workspace_floats(int units, int heads, int G, int64_t n);
int64_t attend_ctas(int units, int heads, int64_t n);  // CTAs of the partial kernel
cudaError_t launch_attend(const AttendLaunch& L, cudaStream_t stream);
cudaError_t launch_e8_quantise(const float* y, int64_t groups, int bits, uint32_t* codes,
                               uint8_t* coset, cudaStream_t stream);
cudaError_t launch_e8_box_quantise(const float* y, int64_t groups, int bits, uint32_t* codes,
                                   uint8_t* coset, cudaStream_t stream);

int64_t entropy_streams(int units, int heads, int64_t n);
int64_t entropy_max_words(int units, int heads, int64_t n);
size_t entropy_workspace_bytes(int units, int heads, int64_t n);
cudaError_t launch_entropy_encode(const nq_packed& in, int units, int heads, int64_t n,
                                  int64_t slot0, int delta, uint16_t* freq, uint32_t* offsets,
                                  uint16_t* words, void* ws, cudaStream_t stream);
cudaError_t launch_entropy_decode(const uint16_t* words, const uint32_t* offsets,
                                  const uint16_t* freq, int units, int heads, int64_t n,
                                  int delta, const nq_packed& out, int64_t slot0,
                                  cudaStream_t stream);

cudaError_t launch_score(const void* K, nq_kv_strides ks, int units, int heads, int64_t T, int W,
                         double* scores, float* mean_ws, cudaStream_t stream);
cudaError_t launch_score_static(const void* K, nq_kv_strides ks, int units, int heads, int64_t T,
                                int W, double* scores, cudaStream_t stream);
cudaError_t launch_select(const double* scores, int units, int64_t T, int W, int evict_pct,
                          int64_t n_kept, int32_t* kept, int64_t kept_stride,
                          cudaStream_t stream);

}  // namespace nq

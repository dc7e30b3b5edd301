// nq_serve.cu -- the steps of a serving loop around the packed cache
// (sm_100a): page tables and slot maps from request lengths, and the norms of
// queries and keys with the rotary embedding.  Formulas: include/nq.h.
#include "nq_internal.h"

namespace nq {

// ------------------------------------------------- page tables and slot maps
// Two exclusive prefix sums over the requests (new tokens, fresh pages), then
// one independent slot per row.  There is nothing to compute and, at serving
// sizes, little to move (8 bytes per row), so the launch is what costs: every
// CTA repeats the scan in its shared memory (12 bytes per request) instead of
// a second kernel waiting for it, CTA 0 writes the scan's own results, and a
// page is found without the table entries that other CTAs write: below have_s
// from the table, above it straight from the free list.  7 us for 64
// requests of one token, 15 us for 1021 requests with 767 000 rows.
constexpr int kPageThreads = 512;

struct PageScan {
  int64_t tokens, pages;
};

__device__ __forceinline__ int32_t sat31(int64_t v) {
  return v > 0x7FFFFFFF ? 0x7FFFFFFF : static_cast<int32_t>(v);
}

struct PageRequest {
  int64_t len, count, have, need;  // need: pages of the table's row in use after the call
  bool beyond;                     // some new token lies past the table's row
};
__device__ __forceinline__ PageRequest page_request(int32_t len, int32_t count, int page_size,
                                                    int64_t stride) {
  PageRequest r;
  r.len = len < 0 ? 0 : len;
  r.count = count < 0 ? 0 : count;
  r.have = (r.len + page_size - 1) / page_size;
  const int64_t want = (r.len + r.count + page_size - 1) / page_size;
  r.beyond = r.count > 0 && want > stride;
  r.need = want < stride ? want : stride;
  return r;
}

__global__ void __launch_bounds__(kPageThreads) page_tables_kernel(const PageTablesLaunch a) {
  extern __shared__ int32_t page_smem[];
  __shared__ PageScan warp_sum[kPageThreads / 32];
  int32_t* s_len = page_smem;              // [S]
  int32_t* s_base = s_len + a.requests;    // [S] free-list index of the first fresh page
  int32_t* s_start = s_base + a.requests;  // [S + 1]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = a.requests, P = a.page_size;
  const bool lead = blockIdx.x == 0;

  // each thread sums a run of consecutive requests, the CTA scans the runs
  const int per = (S + kPageThreads - 1) / kPageThreads;
  const int r0 = min(tid * per, S), r1 = min(r0 + per, S);
  PageScan mine = {0, 0};
  bool bad = false;
  for (int r = r0; r < r1; ++r) {
    const PageRequest q = page_request(a.lens[r], a.counts[r], P, a.table_stride);
    mine.tokens += q.count;
    mine.pages += q.need > q.have ? q.need - q.have : 0;
    if (lead) {
      bad |= q.beyond;
      const int64_t j = q.len / P;  // the page that the first new token shares with older ones
      if (q.count > 0 && j < q.have && j < a.table_stride)
        bad |= a.table[r * a.table_stride + j] < 0;
    }
  }
  PageScan run = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, run.tokens, o);
    const int64_t p = __shfl_up_sync(0xffffffffu, run.pages, o);
    if (lane >= o) {
      run.tokens += t;
      run.pages += p;
    }
  }
  if (lane == 31) warp_sum[warp] = run;
  __syncthreads();
  const int64_t taken = a.taken ? max(__ldg(a.taken), 0) : 0;
  PageScan at = {run.tokens - mine.tokens, taken + run.pages - mine.pages}, total = {0, taken};
  for (int w = 0; w < kPageThreads / 32; ++w) {
    if (w < warp) {
      at.tokens += warp_sum[w].tokens;
      at.pages += warp_sum[w].pages;
    }
    total.tokens += warp_sum[w].tokens;
    total.pages += warp_sum[w].pages;
  }
  for (int r = r0; r < r1; ++r) {
    const PageRequest q = page_request(a.lens[r], a.counts[r], P, a.table_stride);
    s_len[r] = static_cast<int32_t>(q.len);
    s_base[r] = sat31(at.pages);
    s_start[r] = sat31(at.tokens);
    if (lead) {
      a.lens_out[r] = sat31(q.len + q.count);
      a.starts[r] = sat31(at.tokens);
    }
    at.tokens += q.count;
    at.pages += q.need > q.have ? q.need - q.have : 0;
  }
  if (tid == 0) s_start[S] = sat31(total.tokens);
  const bool any_bad = __syncthreads_or(bad);
  if (lead && tid == 0) {
    a.starts[S] = sat31(total.tokens);
    a.used[0] = sat31(total.pages);
    a.used[1] = (total.pages > a.n_free ? 1 : 0) | (any_bad ? 2 : 0) |
                (total.tokens > a.max_rows ? 4 : 0);
  }

  // fresh table entries: one warp per request
  const int nwarps = kPageThreads / 32;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * nwarps + warp; r < S;
       r += static_cast<int64_t>(gridDim.x) * nwarps) {
    const PageRequest q = page_request(s_len[r], a.counts[r], P, a.table_stride);
    for (int64_t j = q.have + lane; j < q.need; j += 32) {
      const int64_t f = s_base[r] + (j - q.have);
      a.table[r * a.table_stride + j] = f < a.n_free ? a.free_pages[f] : -1;
    }
  }

  // rows, four consecutive ones per thread (one search for the first)
  const int64_t rows4 = (a.max_rows + 3) / 4;
  const int64_t tokens = s_start[S];
  for (int64_t x = static_cast<int64_t>(blockIdx.x) * kPageThreads + tid; x < rows4;
       x += static_cast<int64_t>(gridDim.x) * kPageThreads) {
    const int64_t first = 4 * x;
    int slot[4], pos[4];
    int r = 0;
    if (first < tokens) {  // the last request that starts at or before the row
      int lo = 0, hi = S;  // s_start[lo] <= first < s_start[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_start[mid] <= first) lo = mid;
        else hi = mid;
      }
      r = lo;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = first + i;
      slot[i] = -1;
      pos[i] = 0;
      if (row >= tokens) continue;
      while (s_start[r + 1] <= row) ++r;  // ends: row < s_start[S]
      const int64_t len = s_len[r], t = len + (row - s_start[r]);
      const uint32_t j = static_cast<uint32_t>(t) / static_cast<uint32_t>(P);
      const int64_t have = (len + P - 1) / P;
      int32_t page = -1;
      if (j < a.table_stride) {
        if (j < have) {
          page = a.table[r * a.table_stride + j];
        } else {
          const int64_t f = s_base[r] + (j - have);
          if (f < a.n_free) page = a.free_pages[f];
        }
      }
      const int64_t s = static_cast<int64_t>(page) * P + (static_cast<uint32_t>(t) - j * P);
      if (page >= 0 && s <= 0x7FFFFFFF) slot[i] = static_cast<int>(s);
      pos[i] = static_cast<int>(t > 0x7FFFFFFF ? 0x7FFFFFFF : t);
    }
    if (first + 4 <= a.max_rows &&
        ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions)) & 15) == 0) {
      *reinterpret_cast<int4*>(a.slots + first) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.positions + first) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (first + i < a.max_rows) {
          a.slots[first + i] = slot[i];
          a.positions[first + i] = pos[i];
        }
    }
  }
}

cudaError_t launch_page_tables(const PageTablesLaunch& L, cudaStream_t stream) {
  const int smem = (3 * L.requests + 1) * static_cast<int>(sizeof(int32_t));
  if (smem > 48 * 1024) {
    const cudaError_t err = cudaFuncSetAttribute(
        page_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
  }
  int64_t grid = (L.max_rows + 4 * kPageThreads - 1) / (4 * kPageThreads);
  const int64_t by_requests = (L.requests + kPageThreads / 32 - 1) / (kPageThreads / 32);
  if (grid < by_requests) grid = by_requests;
  // at most two CTAs per SM of 148: more would only repeat the scan
  grid = grid < 1 ? 1 : min64(grid, 2 * 148);
  page_tables_kernel<<<static_cast<unsigned>(grid), kPageThreads, smem, stream>>>(L);
  return cudaGetLastError();
}

// ------------------------------------------------- per-head norm + rotation
// Streaming work: every element is read once and written once, and the table
// rows of a token come from L2.  Eight lanes own one 128-vector: lane l holds
// coordinates 8l..8l+7 and their RoPE partners 64+8l..64+8l+7, so the rotation
// stays in the lane, the sum of squares takes three shuffles, and each half
// row is one 128-byte run of 16-byte accesses.  A group keeps its token's
// (cos, sin) in registers for several heads and has the next four heads' rows
// (fp32: the next) under way in a ring of shared memory: what bounds a long
// call is the bytes under way.  32 768 tokens x 40 heads, bf16 (671 MB moved):
// 133 us per call, 5.0 TB/s, 77 % of the measured copy rate; with two heads
// ahead in registers it took 145 us, with loads after the work 220.  fp32 rows
// have half as many bytes under way (two stages are what 48 KB hold beside the
// weights): 303 us to fp32 and 238 us to bf16, 4.4 and 4.2 TB/s.
constexpr int kNormThreads = 256;

struct NormArgs {
  NormRopeLaunch L;
  int64_t n_a, items;  // items: groups of heads of one token, over all tokens and units
  int per;             // heads per item
  int chunks;          // items per token
};

// A lane's share of a row as it is in memory: coordinates 8l .. 8l+7, then
// their partners.
template <bool F32>
struct NormRaw {
  uint4 v[F32 ? 4 : 2];
};

// Asynchronous copy of the lane's share into its own slots of a ring stage
// (chunk c of thread i at c * kNormThreads * 16 + i * 16: nothing is shared
// between threads, so each waits for its own copies only).
template <bool F32>
__device__ __forceinline__ void norm_fetch(const void* p, int64_t off, int l, uint32_t dst) {
  constexpr int kChunks = F32 ? 4 : 2;
  const char* s = static_cast<const char*>(p) + off * (F32 ? 4 : 2);
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int chunk = F32 ? (c < 2 ? 2 * l + c : 16 + 2 * l + c - 2) : l + 8 * c;
    cp_async16(dst + c * (kNormThreads * 16), s + chunk * 16);
  }
}

template <bool F32>
__device__ __forceinline__ void norm_floats(const NormRaw<F32>& r, float (&x)[16]) {
#pragma unroll
  for (int c = 0; c < (F32 ? 4 : 2); ++c) {
    const uint32_t w[4] = {r.v[c].x, r.v[c].y, r.v[c].z, r.v[c].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (F32) {
        x[4 * c + i] = __uint_as_float(w[i]);
      } else {
        x[8 * c + 2 * i] = bf16lo(w[i]);
        x[8 * c + 2 * i + 1] = bf16hi(w[i]);
      }
    }
  }
}

__device__ __forceinline__ void norm_store(void* p, int64_t off, int l, bool f32,
                                           const float (&o)[16]) {
  if (f32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + off);
#pragma unroll
    for (int c = 0; c < 4; ++c)
      d[c < 2 ? 2 * l + c : 16 + 2 * l + c - 2] =
          make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
  } else {
    uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + off);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(o[8 * c + 2 * i], o[8 * c + 2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      d[l + 8 * c] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

template <bool F32>
__global__ void __launch_bounds__(kNormThreads, 3) norm_rope_kernel(const NormArgs a) {
  // Stages of a head each, all but one under way: 3 CTAs x 256 threads x 4 x 32
  // bytes = 98 KB per SM (fp32: 49 KB).
  constexpr int kStages = F32 ? 2 : 5, kStage = (F32 ? 4 : 2) * kNormThreads * 16;
  extern __shared__ __align__(16) unsigned char norm_smem[];
  __shared__ __align__(16) float weights[2][kD];  // of the queries, of the keys
  const NormRopeLaunch& L = a.L;
  {
    const int i = threadIdx.x & 127;
    const float* w = threadIdx.x < 128 ? L.q_weight : L.k_weight;
    weights[threadIdx.x >> 7][i] = w ? __ldg(w + i) : 1.0f;
  }
  __syncthreads();
  const int l = threadIdx.x & 7;
  const int64_t item = (static_cast<int64_t>(blockIdx.x) * kNormThreads + threadIdx.x) >> 3;
  if (item >= a.items) return;  // a whole group
  const int chunk = static_cast<int>(item % a.chunks);
  const int64_t ut = item / a.chunks, u = ut / L.rows, t = ut - u * L.rows;
  int64_t pos = L.pos_base + t;
  if (L.positions) pos = L.pos_base + __ldg(L.positions + u * L.pos_stride + t);
  int64_t hi = pos >> 8;
  hi = hi < 0 ? 0 : (hi >= a.n_a ? a.n_a - 1 : hi);  // out-of-contract positions stay in bounds
  const float4* ta = reinterpret_cast<const float4*>(L.rope_tab) + hi * (kHalf / 2) + 4 * l;
  const float4* tb =
      reinterpret_cast<const float4*>(L.rope_tab) + (a.n_a + (pos & 255)) * (kHalf / 2) + 4 * l;
  float c[8], s[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 A = __ldg(ta + j), B = __ldg(tb + j);
    c[2 * j] = __fmaf_rn(A.x, B.x, -__fmul_rn(A.y, B.y));
    s[2 * j] = __fmaf_rn(A.y, B.x, __fmul_rn(A.x, B.y));
    c[2 * j + 1] = __fmaf_rn(A.z, B.z, -__fmul_rn(A.w, B.w));
    s[2 * j + 1] = __fmaf_rn(A.w, B.z, __fmul_rn(A.z, B.w));
  }
  const int heads = L.q_heads + L.k_heads;
  const int h0 = chunk * a.per, h1 = min(h0 + a.per, heads);
  // the groups of a warp may run different numbers of heads: each shuffles alone
  const uint32_t lanes = 0xFFu << (threadIdx.x & 24);
  const uint32_t ring = smem_u32(norm_smem) + threadIdx.x * 16;
  auto fetch = [&](int h) {
    if (h < h1) {
      const uint32_t dst = ring + ((h - h0) % kStages) * kStage;
      if (h < L.q_heads)
        norm_fetch<F32>(L.q, u * L.qs.unit + h * L.qs.head + t * L.qs.token, l, dst);
      else
        norm_fetch<F32>(L.k, u * L.ks.unit + (h - L.q_heads) * L.ks.head + t * L.ks.token, l, dst);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(h0 + i);
  for (int hh = h0; hh < h1; ++hh) {
    fetch(hh + kStages - 1);  // into the stage that the last head left
    cp_async_wait<kStages - 1>();
    {
      const bool is_q = hh < L.q_heads;
      NormRaw<F32> raw;
      const uint32_t src = ring + ((hh - h0) % kStages) * kStage;
#pragma unroll
      for (int c2 = 0; c2 < (F32 ? 4 : 2); ++c2) raw.v[c2] = lds128(src + c2 * (kNormThreads * 16));
      float x[16], o[16];
      norm_floats<F32>(raw, x);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) ss = __fmaf_rn(x[e], x[e], ss);
#pragma unroll
      for (int o2 = 4; o2 >= 1; o2 >>= 1) ss += __shfl_xor_sync(lanes, ss, o2);
      const float r = __frsqrt_rn(__fmaf_rn(ss, 1.0f / 128.0f, L.eps));
      const float4* g = reinterpret_cast<const float4*>(weights[is_q ? 0 : 1]) + 2 * l;
#pragma unroll
      for (int e4 = 0; e4 < 2; ++e4) {
        const float4 ga = g[e4], gb = g[16 + e4];
        const float wa[4] = {ga.x, ga.y, ga.z, ga.w}, wb[4] = {gb.x, gb.y, gb.z, gb.w};
#pragma unroll
        for (int e2 = 0; e2 < 4; ++e2) {
          const int e = 4 * e4 + e2;
          const float y0 = x[e] * r * wa[e2], y1 = x[e + 8] * r * wb[e2];
          o[e] = __fmaf_rn(y0, c[e], -__fmul_rn(y1, s[e]));
          o[e + 8] = __fmaf_rn(y1, c[e], __fmul_rn(y0, s[e]));
        }
      }
      if (is_q)
        norm_store(L.q_out, u * L.qos.unit + hh * L.qos.head + t * L.qos.token, l, L.q_f32, o);
      else
        norm_store(L.k_out, u * L.kos.unit + (hh - L.q_heads) * L.kos.head + t * L.kos.token, l,
                   L.k_f32, o);
    }
  }
}

cudaError_t launch_norm_rope(const NormRopeLaunch& L, cudaStream_t stream) {
  NormArgs a{};
  a.L = L;
  a.n_a = (L.rope_max_pos + 255) / 256;
  const int heads = L.q_heads + L.k_heads;
  const int64_t tokens = static_cast<int64_t>(L.units) * L.rows;
  // Heads per group: enough groups to fill the GPU first (148 SMs x 16 warps
  // x 4 groups, twice over), then up to sixteen heads share one token's angles.
  int64_t per = tokens * heads / (148 * 16 * 4 * 2);
  per = per < 1 ? 1 : (per > 16 ? 16 : per);
  a.per = static_cast<int>(per > heads ? heads : per);
  a.chunks = (heads + a.per - 1) / a.per;
  a.items = tokens * a.chunks;
  const int64_t grid = (a.items * 8 + kNormThreads - 1) / kNormThreads;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  // shared bytes of the rings, within the 48 KB that need no attribute
  constexpr int kRow = kNormThreads * 16;
  if (L.in_f32)
    norm_rope_kernel<true><<<static_cast<unsigned>(grid), kNormThreads, 2 * 4 * kRow, stream>>>(a);
  else
    norm_rope_kernel<false><<<static_cast<unsigned>(grid), kNormThreads, 5 * 2 * kRow, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace nq

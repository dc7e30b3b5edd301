// nq_tree.cu -- attention of a tree of drafted tokens over the packed cache
// (sm_100a).  Formulas: include/nq.h, nq_tree_attend.
#include "nq_codec_math.cuh"
#include "nq_internal.h"

namespace nq {

constexpr int kTreeTile = 128;            // tokens per tile
constexpr int kTreePart = 2 + kD;         // a split's m (log2 units), l, sums[128]
constexpr int kTreePitch = kD + 4;        // floats per staged row
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct TreeArgs {
  TreeLaunch L;
  int rows;  // nodes * G rows per KV head, row = node * G + g
  int64_t n_a, chunk, nsplit;
  float* part;  // [units * heads][rows][nsplit][kTreePart]
};

__device__ __forceinline__ int64_t tree_len(const TreeLaunch& L, int64_t u) {
  if (!L.lens) return L.n;
  const int64_t v = __ldg(L.lens + u);
  return v < 0 ? 0 : (v > L.n ? L.n : v);
}

// Vector index of token t of unit u, head h; -1 when its page is out of range.
__device__ __forceinline__ int64_t tree_vec(const TreeLaunch& L, const nq_packed& p, int64_t u,
                                            int h, int64_t t) {
  if (!L.table) return u * p.unit_stride + h * p.head_stride + t;
  const uint32_t j = static_cast<uint32_t>(t) / static_cast<uint32_t>(L.page_size);
  const int64_t page = __ldg(L.table + u * L.table_stride + j);
  if (page < 0 || page >= L.pages) return -1;
  return page * p.unit_stride + h * p.head_stride + (t - static_cast<int64_t>(j) * L.page_size);
}

template <int BITS>
__device__ __forceinline__ void tree_codes(const nq_packed& p, int64_t vec,
                                           uint32_t (&w)[4 * BITS], uint32_t& meta) {
#pragma unroll
  for (int c = 0; c < 4 * BITS; ++c) w[c] = vec < 0 ? 0u : __ldg(p.codes + vec * (4 * BITS) + c);
  meta = vec < 0 ? 0u : __ldg(p.meta + vec);
}

template <int BK, int BV>
__global__ void __launch_bounds__(256, 1) tree_partial_kernel(const TreeArgs a) {
  extern __shared__ __align__(16) float tree_smem[];
  float* ks = tree_smem;
  float* vs = ks + kTreeTile * kTreePitch;
  float* qs = vs + kTreeTile * kTreePitch;  // [8 warps][128]
  float* ps = qs + 8 * kD;                  // [8 warps][128]
  const TreeLaunch& L = a.L;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slot_l = lane & 15, half = lane >> 4;
  const int64_t split = blockIdx.x % a.nsplit, uh = blockIdx.x / a.nsplit;
  const int64_t u = uh / L.heads;
  const int h = static_cast<int>(uh % L.heads);
  const int64_t len = tree_len(L, u);
  const int64_t t0 = split * a.chunk, t1 = min64(t0 + a.chunk, len);
  const float2* tab = reinterpret_cast<const float2*>(L.rope_tab);

  for (int64_t tile = t0; tile < t1 || tile == t0; tile += kTreeTile) {
    __syncthreads();
    const int tok = warp * kSlots + slot_l;
    const int64_t t = tile + tok;
    {
      const bool in = t < t1;
      uint32_t wk[4 * BK], wv[4 * BV], mk, mv;
      const int64_t vk = in ? tree_vec(L, L.k_in, u, h, t) : -1;
      const int64_t vv = in ? tree_vec(L, L.v_in, u, h, t) : -1;
      tree_codes<BK>(L.k_in, vk, wk, mk);
      tree_codes<BV>(L.v_in, vv, wv, mv);
      float2 v[32];
      reconstruct_half<BK>(wk, mk, half, v);
      int64_t pos = 0;
      if (in) {
        int32_t p = L.positions ? __ldg(L.positions + u * L.pos_stride + t) : static_cast<int32_t>(t);
        pos = L.pos_base + (p < 0 ? 0 : p);
      }
      int64_t hi = pos >> 8;
      hi = hi >= a.n_a ? a.n_a - 1 : hi;
      const float2* ra = tab + hi * kHalf + 32 * half;
      const float2* rb = tab + (a.n_a + (pos & 255)) * kHalf + 32 * half;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float2 A = __ldg(ra + j), B = __ldg(rb + j);
        const float c = __fmaf_rn(A.x, B.x, -__fmul_rn(A.y, B.y));
        const float s = __fmaf_rn(A.y, B.x, __fmul_rn(A.x, B.y));
        const float x = v[j].x, y = v[j].y;
        ks[tok * kTreePitch + 32 * half + j] = __fmaf_rn(x, c, -__fmul_rn(y, s));
        ks[tok * kTreePitch + 64 + 32 * half + j] = __fmaf_rn(y, c, __fmul_rn(x, s));
      }
      reconstruct_half<BV>(wv, mv, half, v);
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        vs[tok * kTreePitch + 32 * half + j] = v[j].x;
        vs[tok * kTreePitch + 64 + 32 * half + j] = v[j].y;
      }
    }
    __syncthreads();
    float* q = qs + warp * kD;
    float* p = ps + warp * kD;
    for (int r = warp; r < a.rows; r += 8) {
      const int node = r / L.G, j = h * L.G + r % L.G;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(L.q) + u * L.qs.unit +
                                 j * L.qs.head + node * L.qs.token;
      for (int c = lane; c < kD; c += 32) q[c] = __bfloat162float(src[c]);
      __syncwarp();
      float* st = a.part + ((uh * a.rows + r) * a.nsplit + split) * kTreePart;
      float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
      if (tile != t0) {
        m = st[0];
        l = st[1];
        for (int c = 0; c < 4; ++c) o[c] = st[2 + lane + 32 * c];
      }
      float s[4], mt = -INFINITY;
      for (int k = 0; k < 4; ++k) {
        const int tk = lane + 32 * k;
        float d = 0.f;
        for (int c = 0; c < kD; ++c) d = __fmaf_rn(q[c], ks[tk * kTreePitch + c], d);
        const bool ok = tile + tk < t1 && tree_vec(L, L.k_in, u, h, tile + tk) >= 0;
        s[k] = ok ? d * (L.scale * kLog2e) : -INFINITY;
        mt = fmaxf(mt, s[k]);
      }
      for (int x = 16; x >= 1; x >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
      const float mn = fmaxf(m, mt), ref = mn == -INFINITY ? 0.f : mn;
      const float al = exp2f(m - ref);
      float ls = 0.f;
      for (int k = 0; k < 4; ++k) {
        const float e = exp2f(s[k] - ref);
        p[lane + 32 * k] = e;
        ls += e;
      }
      for (int x = 16; x >= 1; x >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, x);
      __syncwarp();
      for (int c = 0; c < 4; ++c) o[c] *= al;
      for (int tk = 0; tk < kTreeTile; ++tk)
        for (int c = 0; c < 4; ++c)
          o[c] = __fmaf_rn(p[tk], vs[tk * kTreePitch + lane + 32 * c], o[c]);
      __syncwarp();
      if (lane == 0) {
        st[0] = mn;
        st[1] = __fmaf_rn(l, al, ls);
      }
      for (int c = 0; c < 4; ++c) st[2 + lane + 32 * c] = o[c];
    }
  }
}

// One warp per row: merge the splits, then attend the draft nodes that the
// row sees one by one (fp32), lane l holding coordinates l, l+32, l+64, l+96.
__global__ void __launch_bounds__(256) tree_combine_kernel(const TreeArgs a) {
  const TreeLaunch& L = a.L;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (w >= static_cast<int64_t>(L.units) * L.heads * a.rows) return;
  const int r = static_cast<int>(w % a.rows);
  const int64_t uh = w / a.rows, u = uh / L.heads;
  const int h = static_cast<int>(uh % L.heads), node = r / L.G, j = h * L.G + r % L.G;
  const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(L.q) + u * L.qs.unit +
                            j * L.qs.head + node * L.qs.token;
  float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
  for (int c = 0; c < 4; ++c) q[c] = __bfloat162float(qp[lane + 32 * c]) * (L.scale * kLog2e);
  for (int64_t s = 0; s < a.nsplit; ++s) {
    const float* p = a.part + (w * a.nsplit + s) * kTreePart;
    const float mn = fmaxf(m, p[0]), ref = mn == -INFINITY ? 0.f : mn;
    const float f = exp2f(m - ref), g = exp2f(p[0] - ref);
    l = l * f + g * p[1];
    for (int c = 0; c < 4; ++c) o[c] = o[c] * f + g * p[2 + lane + 32 * c];
    m = mn;
  }
  const int words = (L.nodes + 63) / 64;
  for (int x = 0; x < words; ++x) {
    const int left = L.mask ? L.nodes - 64 * x : node + 1 - 64 * x;
    unsigned long long bits = left >= 64 ? ~0ull : (left <= 0 ? 0ull : (1ull << left) - 1);
    if (L.mask) bits &= L.mask[u * L.mask_stride + static_cast<int64_t>(node) * words + x];
    while (bits) {
      const int k = 64 * x + __ffsll(static_cast<long long>(bits)) - 1;
      bits &= bits - 1;
      const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(L.K_new) + u * L.kns.unit +
                                h * L.kns.head + k * L.kns.token;
      const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(L.V_new) + u * L.vns.unit +
                                h * L.vns.head + k * L.vns.token;
      float s = 0.f;
      for (int c = 0; c < 4; ++c) s = __fmaf_rn(q[c], __bfloat162float(kp[lane + 32 * c]), s);
      for (int x2 = 16; x2 >= 1; x2 >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x2);
      const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m - ref), g = exp2f(s - ref);
      l = l * f + g;
      for (int c = 0; c < 4; ++c) o[c] = o[c] * f + g * __bfloat162float(vp[lane + 32 * c]);
      m = mn;
    }
  }
  const float inv = l > 0.f ? 1.0f / l : 0.f;
  __nv_bfloat16* op = static_cast<__nv_bfloat16*>(L.out) + u * L.os.unit + j * L.os.head +
                      node * L.os.token;
  for (int c = 0; c < 4; ++c) op[lane + 32 * c] = __float2bfloat16_rn(o[c] * inv);
  if (L.lse && lane == 0)
    L.lse[(u * L.heads * L.G + j) * L.nodes + node] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

static int64_t tree_chunk(int units, int heads, int64_t n) {
  const int64_t uh = static_cast<int64_t>(units) * heads;
  const int64_t want = uh > 0 ? (2 * 148 + uh - 1) / uh : 1;
  int64_t chunk = (n + want - 1) / want;
  chunk = (chunk + kTreeTile - 1) / kTreeTile * kTreeTile;
  return chunk < kTreeTile ? kTreeTile : chunk;
}

static int64_t tree_splits(int units, int heads, int64_t n) {
  const int64_t c = tree_chunk(units, heads, n);
  return (n + c - 1) / c;
}

size_t tree_workspace_bytes(int units, int heads, int G, int nodes, int64_t n, bool) {
  return static_cast<size_t>(units) * heads * G * nodes * tree_splits(units, heads, n) *
         kTreePart * sizeof(float);
}

int64_t tree_ctas(int units, int heads, int G, int nodes, int64_t n) {
  const int64_t uh = static_cast<int64_t>(units) * heads;
  const int64_t a = uh * tree_splits(units, heads, n), b = (uh * G * nodes + 7) / 8;
  return a > b ? a : b;
}

template <int BK, int BV>
static cudaError_t launch_tree_partial(const TreeArgs& a, cudaStream_t stream) {
  constexpr int smem = (2 * kTreeTile * kTreePitch + 16 * kD) * static_cast<int>(sizeof(float));
  cudaError_t err = cudaFuncSetAttribute(tree_partial_kernel<BK, BV>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  const int64_t grid = static_cast<int64_t>(a.L.units) * a.L.heads * a.nsplit;
  tree_partial_kernel<BK, BV><<<static_cast<unsigned>(grid), 256, smem, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_tree_attend(const TreeLaunch& L, cudaStream_t stream) {
  TreeArgs a{};
  a.L = L;
  a.rows = L.nodes * L.G;
  a.n_a = (L.rope_max_pos + 255) / 256;
  a.chunk = tree_chunk(L.units, L.heads, L.n);
  a.nsplit = tree_splits(L.units, L.heads, L.n);
  a.part = static_cast<float*>(L.ws);
  if (L.n > 0) {
    const int bk = L.k_in.bits, bv = L.v_in.bits;
    const cudaError_t err = bk == 3 ? (bv == 3 ? launch_tree_partial<3, 3>(a, stream)
                                               : launch_tree_partial<3, 2>(a, stream))
                                    : (bv == 3 ? launch_tree_partial<2, 3>(a, stream)
                                               : launch_tree_partial<2, 2>(a, stream));
    if (err != cudaSuccess) return err;
  }
  const int64_t rows = static_cast<int64_t>(L.units) * L.heads * a.rows;
  tree_combine_kernel<<<static_cast<unsigned>((rows + 7) / 8), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace nq

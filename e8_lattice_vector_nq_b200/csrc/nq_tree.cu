// nq_tree.cu -- attention of a tree of drafted tokens over the packed cache
// (sm_100a).  Formulas: include/nq.h, nq_tree_attend.
//
// The R = nodes * G query rows of one KV head share the head's tokens, so a
// token is unpacked once for all of them and the two products run on the
// tensor cores with the TOKENS as the 128 rows of the MMA and the query rows
// as its N columns (N = 16 .. 128 as the call needs, so a single new token
// does not pay for 128 rows).  Per tile of 128 tokens and one KV head:
//   1. keys: codes -> t = 2q, q the lattice point (f16 integers, exact); X = t H on the tensor
//      cores: with H128 = [[H64, H64], [H64, -H64]] the two halves u = H64 t_lo
//      and v = H64 t_hi take half the products, and the last butterfly costs
//      nothing inside the rotation:
//        o_i = u c' + v s',  o_{i+64} = u s' - v c',  c' = c - s, s' = c + s.
//      o is rounded to f16 (|o| < 1268: no scale is applied before the product,
//      so no scale can overflow it) and the key's scale kappa_t multiplies the
//      score, where a thread has one token and kappa_t is its scalar.  c', s'
//      and the rotation are f16 too (two coordinates per instruction): o_i is
//      off by up to 2^-11 (2 r + |o_i|), r its pair's length; with unit-normal
//      rows and scale 128^-1/2 that moves a score by 2^-11 sqrt 2 (RMS, at
//      most), against 2^-8 of an output's rounding to bf16;
//   2. S^T = o Q^T (fp32 in TMEM), Q scaled per row by a power of two;
//   3. y = S f_r kappa_t - m_r in log2 units, p = 2^y; the sum over tokens is
//      kept per thread and reduced once at the end;
//   4. O^T += V' P, V' = 2^(e-2) t and P = f16(p m) for the value's scale sigma
//      = 2^e m, so V' is exact and a token's weight is rounded once (no
//      transform: the codes' coordinates are summed, and H is applied once per
//      row at the end).
// m_r is not the running maximum but a reference kept near it: a column's
// largest p starts at 2^4 and stays below 2^14, so the maximum may grow by
// 2^10 before the sums are rescaled, and f16 holds p down to 2^-28 of the
// maximum.  A tile whose scores leave that range (the first one always) takes
// the exact maxima of those columns; the others only compare (one vote per
// tile and warpgroup).
//
// One CTA per SM, its warpgroups specialised so that the phases of different
// tiles overlap: two or four warpgroups make keys (a token per thread and a
// part of its coordinates: codes -> t, then X -> rotated keys), one makes
// values, two or four do the softmax (a part of the query rows each), and the
// last one's warps issue the three products.  X is double buffered in TMEM (up
// to 64 columns), so the codes of tile j+1 go to the tensor cores before tile j
// is rotated.  Registers are moved to the softmax warpgroups, which hold a sum
// per query row.  The work of a launch is split over the tokens (flash
// decoding) to fill the 148 SMs; tree_combine_kernel merges the splits, applies
// H and attends the draft nodes in fp32 on the CUDA cores, a warp per row: 1.43
// of the 2.05 ms that 1024 nodes x 4 heads take over 16 384 tokens of 8 KV heads.
//
// What bounds it: the instructions of the warps that unpack and rotate (16, 64
// and 128 columns take 2890, 3340 and 4380 cycles per tile and issue in 77, 73
// and 64 % of the cycles, part of it polls of the waits; tensor pipe 14 to 29 %,
// DRAM 9 to 15 %).  Per call with 8 KV heads, 3-bit keys and 2-bit
// values: 32 units x 13 147 tokens, one node of 4 heads (16 columns), 350 us
// against 45 us for the bytes alone (296 MB at 6567 GB/s); a tree of 64 nodes x
// 4 heads over 131 072 tokens, 340 to 360 us, 380 to 400 TFLOP/s of the attention's own
// 4 R n 128 operations per KV head.
//
// The angles of a tile are needed by every KV head and every row block:
// tree_angles_kernel writes (c', s') once per call as f16 pairs in the order
// in which the compute threads read them.
#include "nq_codec_math.cuh"
#include "nq_internal.h"
#include "nq_tcgen05.cuh"

namespace nq {

constexpr int kTreeTile = 128;     // tokens per tile
constexpr int kTreePart = 2 + kD;  // a split's m (log2 units), l, sums[128] in the code domain
constexpr float kTreeStart = 4.0f, kTreeTop = 14.0f;  // log2 of a column's largest weight
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTreeMaxSplits = 4 * 148;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kTreeWaitLimit = 1u << 12, kTreePolls = 256;  // 2^20 polls
constexpr uint32_t kErrTreeTimeout = 4u;

struct TreeArgs {
  TreeLaunch L;
  int rows;         // nodes * G rows per KV head, row = node * G + g
  int ncols;        // query rows per CTA
  int rblocks;      // CTAs per (unit, KV head, split)
  int64_t n_a;
  int64_t tiles;    // ceil(n / 128)
  int64_t per;      // tiles per split
  int64_t nsplit;
  float* part;      // [units * heads][rows][nsplit][kTreePart]
  uint4* angles;    // [units or 1][tiles][4][4][128]
  FastDiv page;     // division by the page size
  int64_t angle_stride;  // entries per unit, 0 when shared
};

__device__ __forceinline__ int64_t tree_len(const TreeLaunch& L, int64_t u) {
  if (!L.lens) return L.n;
  const int64_t v = __ldg(L.lens + u);
  return v < 0 ? 0 : (v > L.n ? L.n : v);
}

// ------------------------------------------------------------------ angles
// Per token c' = c - s and s' = c + s of the 64 frequencies as f16 pairs:
// entry e (16 bytes) holds frequencies 4e .. 4e+3 as (c' pair, s' pair, c'
// pair, s' pair), the 128 tokens of a tile side by side.  A warp reads each
// token's two table rows whole (lane l: frequencies 2l, 2l+1) and the tile
// goes through shared memory, so that both sides are contiguous.  32 lists
// of 13 147 positions, 108 MB written: 36 us, 3.0 TB/s.
constexpr int kAngleThreads = 256;
constexpr int kAnglePitch = 256 + 16;  // bytes per token: neither side has bank conflicts
__global__ void __launch_bounds__(kAngleThreads) tree_angles_kernel(const TreeArgs a) {
  __shared__ __align__(16) unsigned char rows[kTreeTile * kAnglePitch];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t tile = blockIdx.x % a.tiles, u = blockIdx.x / a.tiles;
  constexpr int kPer = kTreeTile / (kAngleThreads / 32);  // tokens per warp
  const int first = warp * kPer;
  int64_t mine = 0;  // lane l: the position of the warp's token l
  {
    const int64_t tok = tile * kTreeTile + first + lane;
    if (lane < kPer && tok < a.L.n) {
      const int32_t p = a.L.positions ? __ldg(a.L.positions + u * a.L.pos_stride + tok)
                                      : static_cast<int32_t>(tok);
      mine = a.L.pos_base + (p < 0 ? 0 : p);
    }
  }
  // out-of-contract positions stay in bounds
  mine = min64(mine, min64(a.n_a * 256 - 1, 0x7FFFFFFF));
  const float4* tab = reinterpret_cast<const float4*>(a.L.rope_tab);
  const int pos32 = static_cast<int>(mine);
  // eight fine rows in flight; nearby positions share the coarse row, which is
  // read again only when it changes
  int64_t row = __shfl_sync(0xffffffffu, pos32, 0) >> 8;
  float4 A = __ldg(tab + row * 32 + lane);
#pragma unroll
  for (int i0 = 0; i0 < kPer; i0 += 8) {
    float4 B[8];
    int pos[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      pos[i] = __shfl_sync(0xffffffffu, pos32, i0 + i);
      B[i] = __ldg(tab + (a.n_a + (pos[i] & 255)) * 32 + lane);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t hi = pos[i] >> 8;
      if (hi != row) A = __ldg(tab + hi * 32 + lane);
      row = hi;
      const float c0 = __fmaf_rn(A.x, B[i].x, -__fmul_rn(A.y, B[i].y));
      const float s0 = __fmaf_rn(A.y, B[i].x, __fmul_rn(A.x, B[i].y));
      const float c1 = __fmaf_rn(A.z, B[i].z, -__fmul_rn(A.w, B[i].w));
      const float s1 = __fmaf_rn(A.w, B[i].z, __fmul_rn(A.z, B[i].w));
      const __half2 cc = __floats2half2_rn(c0 - s0, c1 - s1);
      const __half2 ss = __floats2half2_rn(c0 + s0, c1 + s1);
      *reinterpret_cast<uint2*>(rows + (first + i0 + i) * kAnglePitch + lane * 8) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&cc), *reinterpret_cast<const uint32_t*>(&ss));
    }
  }
  __syncthreads();
  uint4* out = a.angles + u * a.angle_stride + tile * (16 * kTreeTile);
#pragma unroll
  for (int i = 0; i < 16 * kTreeTile / kAngleThreads; ++i) {
    const int e = (i * kAngleThreads + threadIdx.x) >> 7, t = threadIdx.x & 127;
    out[e * kTreeTile + t] = *reinterpret_cast<const uint4*>(rows + t * kAnglePitch + e * 16);
  }
}

// ------------------------------------------------------------------- codes
// 32 consecutive codes as 16 f16 pairs.  A code sits in the mantissa of an f16
// whose exponent is that of 1024, at bit d >= 1 (1024 + j 2^d), two codes 16
// bits apart per register, so one AND-OR turns a shifted view of the words
// into a pair and one exact fma into t = 2j - (2^b - 2) - h:
//   b = 3: pairs (a, a+5) of each run of ten codes (15 bits apart: d differs
//          by one between the lanes), the last pair (30, 31) from its own bits;
//   b = 2: pairs (i, i+8) of each word.
// tree_slot gives the code that slot p of the 32 holds.
template <int BITS>
__host__ __device__ constexpr int tree_slot(int p) {
  const int q = p >> 1, lane = p & 1;
  if (BITS == 2) return 16 * (q >> 3) + (q & 7) + 8 * lane;
  return q < 15 ? 10 * (q / 5) + q % 5 + 5 * lane : 30 + lane;
}

// f16 bits of +-2^e * m for values that f16 holds exactly (compile time).
__host__ __device__ constexpr uint32_t f16_bits(float v) {
  uint32_t s = 0;
  if (v < 0) {
    s = 0x8000u;
    v = -v;
  }
  int e = 15;
  while (v >= 2.0f) {
    v *= 0.5f;
    ++e;
  }
  while (v < 1.0f) {
    v *= 2.0f;
    --e;
  }
  return s | (static_cast<uint32_t>(e) << 10) | static_cast<uint32_t>((v - 1.0f) * 1024.0f);
}
__host__ __device__ constexpr uint32_t f16_pair(float lo, float hi) { return f16_bits(lo) | (f16_bits(hi) << 16); }

__device__ __forceinline__ uint32_t hmul2u(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hfma2u(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// The f16 pairs of coset bits that a 32-code run needs: byte g of z has the
// coset bit of group g in its top bit; a byte permute that repeats top bits
// makes the lanes' masks.
__device__ __forceinline__ uint32_t coset_bytes(uint32_t bits4) { return (bits4 & 15u) * 0x10204080u; }
__device__ __forceinline__ uint32_t coset_mask(uint32_t z, int ga, int gb) {
  uint32_t m;  // (prmt's sign mode: __byte_perm has no form of it)
  asm("prmt.b32 %0, %1, %1, %2;"
      : "=r"(m)
      : "r"(z), "r"(0x8888u | (ga * 0x11u) | (gb * 0x1100u)));
  return m;
}

// The pair with fields at bits dl (low lane) and 16 + dh of v -> 2j - (2^b - 2)
// - h, h the lanes' coset bits as a mask.  The addend -(1024 * 2^(1-d) + 2^b - 2)
// has a zero bit where 1.0 is added to its magnitude (2^b - 2 is even and small
// against the power of two), so an OR takes h off.
template <int BITS, int DL, int DH>
__device__ __forceinline__ uint32_t tree_pair(uint32_t v, uint32_t hmask) {
  constexpr uint32_t kMask = (((1u << BITS) - 1u) << DL) | (((1u << BITS) - 1u) << (16 + DH));
  constexpr float kOff = static_cast<float>((1 << BITS) - 2);
  constexpr float kScaleL = 2.0f / (1 << DL), kScaleH = 2.0f / (1 << DH);
  constexpr uint32_t kMul = f16_pair(kScaleL, kScaleH);
  constexpr uint32_t kAdd = f16_pair(-(1024.0f * kScaleL + kOff), -(1024.0f * kScaleH + kOff));
  constexpr uint32_t kAdd1 = f16_pair(-(1024.0f * kScaleL + kOff + 1.0f), -(1024.0f * kScaleH + kOff + 1.0f));
  static_assert((kAdd1 & kAdd) == kAdd, "the coset bit is an OR");
  return hfma2u((v & kMask) | 0x64006400u, kMul, kAdd | (hmask & (kAdd1 ^ kAdd)));
}

template <int BITS>
__device__ __forceinline__ void tree_unpack(const uint32_t (&w)[BITS], uint32_t cosets,
                                            uint32_t (&h)[16]) {
  const uint32_t z = coset_bytes(cosets);
  auto hm = [&](int q) {
    return coset_mask(z, tree_slot<BITS>(2 * q) >> 3, tree_slot<BITS>(2 * q + 1) >> 3);
  };
  if constexpr (BITS == 2) {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint32_t v0 = w[m] << 1, v1 = w[m] >> 7;
      h[8 * m] = tree_pair<2, 1, 1>(v0, hm(8 * m));
      h[8 * m + 1] = tree_pair<2, 3, 3>(v0, hm(8 * m + 1));
      h[8 * m + 2] = tree_pair<2, 5, 5>(v0, hm(8 * m + 2));
      h[8 * m + 3] = tree_pair<2, 7, 7>(v0, hm(8 * m + 3));
      h[8 * m + 4] = tree_pair<2, 1, 1>(v1, hm(8 * m + 4));
      h[8 * m + 5] = tree_pair<2, 3, 3>(v1, hm(8 * m + 5));
      h[8 * m + 6] = tree_pair<2, 5, 5>(v1, hm(8 * m + 6));
      h[8 * m + 7] = tree_pair<2, 7, 7>(v1, hm(8 * m + 7));
    }
  } else {
    auto window = [&](int s) -> uint32_t {  // bits [s, s + 32) of the 96
      if (s < 0) return w[0] << (-s);
      const int i = s >> 5, o = s & 31;
      const uint32_t lo = w[i], hi = i + 1 < 3 ? w[i + 1 < 3 ? i + 1 : 2] : 0u;
      return o == 0 ? lo : __funnelshift_r(lo, hi, o);
    };
#pragma unroll
    for (int b = 0; b < 3; ++b) {
      const uint32_t v0 = window(30 * b - 2), v1 = window(30 * b + 4), v2 = window(30 * b + 10);
      h[5 * b] = tree_pair<3, 2, 1>(v0, hm(5 * b));
      h[5 * b + 1] = tree_pair<3, 5, 4>(v0, hm(5 * b + 1));
      h[5 * b + 2] = tree_pair<3, 2, 1>(v1, hm(5 * b + 2));
      h[5 * b + 3] = tree_pair<3, 5, 4>(v1, hm(5 * b + 3));
      h[5 * b + 4] = tree_pair<3, 2, 1>(v2, hm(5 * b + 4));
    }
    h[15] = tree_pair<3, 2, 1>(((w[2] >> 24) & 0x1Cu) | ((w[2] >> 12) & 0xE0000u), hm(15));
  }
}

// Row t, 16-byte chunk c of an operand of 128-byte swizzled rows (K-major: an
// output row per row; MN-major: a token, the k index, per row).
__device__ __forceinline__ uint32_t row_chunk(int t, int c) {
  return static_cast<uint32_t>((t >> 3) * 1024 + (t & 7) * 128 + ((c ^ (t & 7)) << 4));
}

// The reduction over the warp's lanes of each of C columns (C a power of two
// up to 32) that every lane holds a value of: lane c (mod C) returns column
// c's.  Each step halves the columns that a lane carries, so C columns take
// about C shuffles instead of 5 C.
template <int C, class F>
__device__ __forceinline__ float column_reduce(float (&x)[C], int lane, F f) {
#pragma unroll
  for (int o = C / 2; o >= 1; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int c = 0; c < o; ++c) {
      const float keep = up ? x[c + o] : x[c], give = up ? x[c] : x[c + o];
      x[c] = f(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
  float v = x[0];
#pragma unroll
  for (int o = 16; o >= C; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// ------------------------------------------------------------ shared memory
template <int BK, int BV, int N>
struct TreeSmem {
  static constexpr int V = 0;                           // scaled value codes, two tiles of
                                                        // 2 x (128 rows x 128 B)
  static constexpr int PBytes = (N > 64 ? 2 : 1) * 16384;  // weights: N/64 blocks of 128 rows
  static constexpr int P = V + 2 * 32768;               // of two tiles
  static constexpr int Q = P + 2 * PBytes;              // queries: 2 x (N rows x 128 B)
  static constexpr int H = Q + N * 256;                 // H64, 64 rows x 128 B
  static constexpr int Kap = H + 8192;                  // key scales of 8 tiles (-1: no token)
  static constexpr int Vm = Kap + 8 * 512;              // value scale mantissas of 8 tiles
  static constexpr int FM = Vm + 8 * 512;               // (f0, f1, -m0, -m1) per row pair
  static constexpr int WMax = FM + N * 8;               // [N][4 warps]
  static constexpr int WOr = WMax + N * 16;             // [4][4 warps]
  static constexpr int Bars = WOr + 64;
  static constexpr int Bytes = Bars + 128 + 1024;       // 1 KB of slack to align the base
  static_assert(Bytes <= 232448, "one CTA per SM within 227 KB");
  // TMEM columns (all 512 are allocated): X (one or two tiles), S, O, and the
  // A operands T and K (two f16 per column)
  static constexpr int XBufs = N > 64 ? 1 : 2, KBufs = N > 32 ? 1 : 2;
  static constexpr uint32_t tX = 0, tS = XBufs * 128, tO = tS + N, tT = tO + N, tK = tT + 64;
  static_assert(tK + KBufs * 64 <= 512, "tensor memory");
};

// Bounded wait; past the limit the error word is set and `dead` makes every
// later wait of the CTA return at once (its results are then unspecified).
// A wait names its phase by parity, so a barrier must neither be a phase
// further than the one waited for nor a phase behind: each barrier's next
// phase needs something that its waiters do after their wait for this one,
// and every waiter takes the phases in order.
__device__ __forceinline__ void tree_wait(uint32_t bar, uint32_t parity, volatile uint32_t* dead) {
  bool done = mbar_poll(bar, parity, kTreePolls);
  for (uint32_t i = 1; !done && i < kTreeWaitLimit; ++i)
    done = mbar_poll(bar, parity, kTreePolls) || *dead;
  if (!done) {
    *dead = 1u;
    atomicOr(&g_nq_error, kErrTreeTimeout);
  }
  __syncwarp();
}

// A 128-byte swizzled operand whose first row is at 16 * addr4, groups of 8
// rows 1024 bytes apart: K-major (see desc_sw128), or MN-major, a row of 128
// bytes (64 elements along M or N) per k, the next 64 elements 16 * lbo4 bytes on.
__device__ __forceinline__ uint64_t tree_desc(uint32_t addr4, uint32_t lbo4) {
  constexpr uint32_t kHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
  return (static_cast<uint64_t>(kHigh) << 32) | (addr4 | (lbo4 << 16));
}

// One arrival for the warp, after its threads' shared-memory writes (fenced
// for the MMA by the callers that wrote operands).
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

template <int REGS>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}
// Warpgroups of the roles (KW: threads that share a token's key, SW: that
// share its scores) and their registers per thread, out of Launch x threads
// that the block starts with.  Up to 64 columns the key warpgroups bound the
// pipeline, so they are four; with 128 the softmax would, and gets four.  The
// split with 128 columns: 64 registers for the keys and 80 for the softmax take
// 353 us on 64 nodes x 4 heads over 131 072 tokens, 48 and 88 take 392, 64 and
// 72 take 368.  With 64 columns 56 and 96 take 344 us on 32 ragged units of up
// to 16 384 tokens, 64 and 88 take 361.
template <int N>
struct TreeRoles {
  static constexpr int KW = N > 64 ? 2 : 4, SW = N > 64 ? 4 : 2;
  static constexpr int Values0 = 4 * KW, Softmax0 = Values0 + 4, Issue0 = Softmax0 + 4 * SW;  // warps
  static constexpr int Threads = 32 * (Issue0 + 4), Launch = 64;
  static_assert(Threads == 1024, "eight warpgroups");
  static constexpr int Softmax = N > 64 ? 80 : (N > 32 ? 96 : 64), Keys = N > 64 ? 64 : (N > 32 ? 56 : 64),
                       Values = N > 64 ? 40 : (N > 32 ? 56 : 64), Issue = N > 64 ? 24 : (N > 32 ? 32 : 64);
  static_assert(SW * Softmax + KW * Keys + Values + Issue <= 8 * Launch, "the launch's registers");
  // only the softmax takes more than it was launched with, and only after the
  // setup's barrier, behind which the others wait for nothing before they give
  static_assert(Keys <= Launch && Values <= Launch && Issue <= Launch, "no wait for registers before the barrier");
};
template <int LAUNCH, int WANT>
__device__ __forceinline__ void set_regs() {
  if constexpr (WANT > LAUNCH) regs_inc<WANT>();
  if constexpr (WANT < LAUNCH) regs_dec<WANT>();
}

// The tokens of one thread, tile by tile: the unit or page that holds the
// token (-1: no token) and its slot there.  The page entry of the next tile is
// in flight.
struct TokenWalk {
  const int32_t* row;  // the unit's row of the page table, or NULL
  const FastDiv& div;
  int64_t pages;
  uint32_t t, t1;  // this thread's token of the tile that `page` belongs to; end of the split
  int32_t page;

  __device__ __forceinline__ TokenWalk(const TreeArgs& a, int64_t u, int64_t tok, int64_t end)
      : div(a.page), pages(a.L.pages), t(static_cast<uint32_t>(tok)), t1(static_cast<uint32_t>(end)) {
    row = a.L.table ? a.L.table + u * a.L.table_stride : nullptr;
    page = static_cast<int32_t>(u);
    fetch();
  }
  __device__ __forceinline__ void fetch() {
    if (row && t < t1) page = __ldg(row + fdiv(t, div));
  }
  __device__ __forceinline__ void next(int32_t& lead, uint32_t& slot) {
    lead = t < t1 ? page : -1;
    slot = t;
    if (row) {  // (uniform: a contiguous unit costs none of this)
      if (page < 0 || page >= pages) lead = -1;
      slot = t - fdiv(t, div) * div.d;
    }
    t += kTreeTile;
    fetch();
  }
};

// A value's scale sigma = 2^e m with e >= -22 (so that 2^(e-2) t is exact in
// f16), 1 <= m < 2 (or below for the smallest scales); 7 * 2^13 stays in range.
__device__ __forceinline__ void value_scale(uint32_t meta, float& m, int& e) {
  const float sig = __half2float(__ushort_as_half(static_cast<unsigned short>(meta >> 16)));
  e = max(static_cast<int>(__float_as_uint(sig) >> 23) - 127, -22);
  m = sig * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

template <int V>
struct Parity {
  static constexpr int value = V;
};

template <int BK, int BV, int N>
__global__ void __launch_bounds__(TreeRoles<N>::Threads, 1) tree_partial_kernel(const TreeArgs a) {
  using S = TreeSmem<BK, BV, N>;
  using R = TreeRoles<N>;
  constexpr int KW = R::KW;
  extern __shared__ __align__(1024) unsigned char tree_smem[];
  const uint32_t raw = smem_u32(tree_smem);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* gen = tree_smem + (base - raw);  // generic pointer of the aligned base
  const TreeLaunch& L = a.L;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // barriers: codes written, X done, keys written, S done, S read, values
  // written, weights written, O done (the scales of a tile are written with
  // its codes).  Where a buffer is double, so is its barrier: tile j uses
  // barrier j & 1 in its phase j >> 1.
  const uint32_t bar_t = base + S::Bars, bar_x = bar_t + 8, bar_sf = bar_t + 16;
  const uint32_t bar_xf = bar_t + 24;  // X read (where it is single)
  auto bar_k = [&](int j) { return bar_t + 32 + 8 * (j & 1); };
  auto bar_s = [&](int j) { return bar_t + 48 + 8 * (j & 1); };
  auto bar_v = [&](int j) { return bar_t + 64 + 8 * (j & 1); };
  auto bar_o = [&](int j) { return bar_t + 80 + 8 * (j & 1); };
  auto bar_p = [&](int j) { return bar_t + 96 + 8 * (j & 1); };
  const uint32_t tslot = bar_t + 112;
  volatile uint32_t* dead = reinterpret_cast<volatile uint32_t*>(gen + S::Bars + 116);

  // block index -> (split, unit * heads + head, row block): the row blocks and
  // heads of the same tokens are neighbours (their codes and angles meet in L2)
  const int rb = static_cast<int>(blockIdx.x % a.rblocks);
  const int64_t rest = blockIdx.x / a.rblocks;
  const int64_t UH = static_cast<int64_t>(L.units) * L.heads;
  const int64_t uh = rest % UH, split = rest / UH;
  const int64_t u = uh / L.heads;
  const int h = static_cast<int>(uh % L.heads);
  const int64_t len = tree_len(L, u);
  const int64_t t0 = split * a.per * kTreeTile, t1 = min64(t0 + a.per * kTreeTile, len);
  const int nt = t1 > t0 ? static_cast<int>((t1 - t0 + kTreeTile - 1) / kTreeTile) : 0;
  const int row0 = rb * N;
  float* part = a.part + ((uh * a.rows + row0) * a.nsplit + split) * kTreePart;
  const int64_t part_row = a.nsplit * kTreePart;

  if (nt == 0) {  // nothing held in this split
    if (tid < N && row0 + tid < a.rows) {
      part[tid * part_row] = -INFINITY;
      part[tid * part_row + 1] = 0.f;
    }
    return;
  }

  // ---- setup: barriers, TMEM, constant operands, queries
  constexpr uint32_t kCols = 512;
  if (warp == R::Issue0) {
    tmem_alloc(tslot, kCols);
    tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(bar_t, 4 * KW);
    mbar_init(bar_x, 1);
    mbar_init(bar_xf, 4 * KW);
    mbar_init(bar_sf, 4 * R::SW);
    for (int j = 0; j < 2; ++j) {
      mbar_init(bar_k(j), 4 * KW);
      mbar_init(bar_s(j), 2);  // the products, and their issuer (see there)
      mbar_init(bar_v(j), 4);
      mbar_init(bar_p(j), 4 * R::SW);
      mbar_init(bar_o(j), 1);
    }
    *dead = 0u;
    fence_mbar_init();
  }
  constexpr int kRows = (N + R::Threads / 32 - 1) / (R::Threads / 32);  // query rows per warp
  uint2 qv[kRows];  // all of the warp's rows in flight together
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = warp + i * (R::Threads / 32), row = row0 + r;
    qv[i] = make_uint2(0u, 0u);
    if (r < N && row < a.rows) {
      const int node = row / L.G, j = h * L.G + row % L.G;
      qv[i] = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(L.q) +
                                                   u * L.qs.unit + j * L.qs.head +
                                                   node * L.qs.token) + lane);
    }
  }
  if (tid < 512) {  // H64: row n, chunk c (8 slots)
    const int n = tid >> 3, c = tid & 7;
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t pr = 0u;
#pragma unroll
      for (int l = 0; l < 2; ++l) {
        const int s = 8 * c + 2 * i + l;
        const int code = 32 * (s >> 5) + tree_slot<BK>(s & 31);
        pr |= (0x3C00u | (static_cast<uint32_t>(__popc(n & code) & 1) << 15)) << (16 * l);
      }
      v[i] = pr;
    }
    sts128(base + S::H + row_chunk(n, c), make_uint4(v[0], v[1], v[2], v[3]));
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = warp + i * (R::Threads / 32);
    if (r >= N) break;
    const float q[4] = {bf16lo(qv[i].x), bf16hi(qv[i].x), bf16lo(qv[i].y), bf16hi(qv[i].y)};
    float m = fmaxf(fmaxf(fabsf(q[0]), fabsf(q[1])), fmaxf(fabsf(q[2]), fabsf(q[3])));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // |q| 2^-e in [2^13, 2^14): a bf16 value is exact in f16 down to 2^-29 of
    // the row's largest
    const int e = m > 0.f && m < INFINITY ? static_cast<int>(__float_as_uint(m) >> 23) - 127 - 13 : 0;
    const float down = e >= -126 && e <= 126 ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : 0.f;
    const __half2 p0 = __floats2half2_rn(q[0] * down, q[1] * down);
    const __half2 p1 = __floats2half2_rn(q[2] * down, q[3] * down);
    const int c = lane >> 1;  // chunk of 8 coordinates, this lane's half of it
    const uint32_t dst = base + S::Q + (c >> 3) * (N * 128) + row_chunk(r, c & 7) + (lane & 1) * 8;
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(dst),
                 "r"(*reinterpret_cast<const uint32_t*>(&p0)),
                 "r"(*reinterpret_cast<const uint32_t*>(&p1))
                 : "memory");
    if (lane == 0) {
      float* fm = reinterpret_cast<float*>(gen + S::FM) + (r >> 1) * 4 + (r & 1);
      const float up = down > 0.f ? __uint_as_float(static_cast<uint32_t>(127 + e) << 23) : 0.f;
      fm[0] = L.scale * kLog2e * up;
      fm[2] = 0.f;
    }
  }
  // every role calls this once, the loading ones after their first loads
  auto setup_done = [&]() {
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  };
  // the whole of TMEM is allocated (512 columns), so it starts at column 0
  constexpr uint32_t tS = S::tS, tO = S::tO;
  const int t = tid & 127;
  const uint32_t t_lane = static_cast<uint32_t>(32 * (warp & 3)) << 16;

  if (warp < R::Values0) {
    // ------------------------------------------------------------- keys
    // Thread (t, kw): token t, 128 / KW codes and 64 / KW frequencies.
    set_regs<R::Launch, R::Keys>();
    constexpr int NU = 4 / KW;           // runs of 32 codes
    constexpr int NQ = 8 / KW;           // runs of 8 frequencies
    const int kw = warp >> 2;
    const uint4* ang = a.angles + u * a.angle_stride + ((split * a.per * 4) * 4 + 2 * NQ * kw) * 128 + t;
    TokenWalk walk(a, u, t0 + t, t1);
    // a quarter of a 3-bit vector is three words out of one or two 16-byte
    // chunks: these are loaded whole (one strided access instead of three) and
    // picked from when they are used, so that nothing waits for the loads
    constexpr bool kChunks = NU * BK == 3;
    uint32_t wd[kChunks ? 8 : NU * BK], meta, vmeta;
    int32_t lead;  // where the token of the tile after the loaded one is
    uint32_t slot;
    const int64_t khead = h * L.k_in.head_stride, vhead = h * L.v_in.head_stride;
    // Loads whatever the token: without one, vector 0, whose bits are not used
    // (a branch here makes the compiler move the loaded values at its end,
    // which waits for them).
    bool held;  // the loaded tile's token exists
    auto load = [&]() {
      held = lead >= 0;
      const int64_t v = held ? lead * L.k_in.unit_stride + khead + slot : 0;
      const uint32_t* src = L.k_in.codes + v * (4 * BK) + (kChunks ? (3 * kw) / 4 * 4 : kw * (NU * BK));
      if constexpr (NU * BK == 4 || kChunks) {
#pragma unroll
        for (int i = 0; i < (kChunks ? 2 : 1); ++i) {
          // (the second chunk of an outer quarter is not used: the first again)
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(src) + (kw == 1 || kw == 2 ? i : 0));
          wd[4 * i] = x.x, wd[4 * i + 1] = x.y, wd[4 * i + 2] = x.z, wd[4 * i + 3] = x.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < NU * BK / 2; ++i) {
          const uint2 x = __ldg(reinterpret_cast<const uint2*>(src) + i);
          wd[2 * i] = x.x, wd[2 * i + 1] = x.y;
        }
      }
      meta = __ldg(L.k_in.meta + v);
      if (kw == KW - 1)
        vmeta = __ldg(L.v_in.meta + (held ? lead * L.v_in.unit_stride + vhead + slot : 0));
    };
    // codes of tile j -> T; then the loads of tile j+1
    auto write_t = [&](int j) {
#pragma unroll
      for (int s = 0; s < NU; ++s) {
        const int run = NU * kw + s;  // codes 32 run .. 32 run + 31
        uint32_t w[BK], hh[16];
#pragma unroll
        for (int i = 0; i < BK; ++i)
          w[i] = !kChunks ? wd[s * BK + i]
                          : (kw == 0 ? wd[i] : (kw == 1 ? wd[i + 3] : (kw == 2 ? wd[i + 2] : wd[i + 1])));
        tree_unpack<BK>(w, meta >> (4 * run), hh);
        tmem_st(S::tT + t_lane + 16 * run, hh);
      }
      if (kw == KW - 2) {
        const float sig = __half2float(__ushort_as_half(static_cast<unsigned short>(meta >> 16)));
        const float kap = __fmul_rn(__fmul_rn(sig, 0.5f), __uint_as_float(kCBits));
        reinterpret_cast<float*>(gen + S::Kap)[(j & 7) * 128 + t] = held ? kap : -1.0f;
      }
      if (kw == KW - 1) {
        float m;
        int e;
        value_scale(held ? vmeta : 0u, m, e);
        reinterpret_cast<float*>(gen + S::Vm)[(j & 7) * 128 + t] = m;
      }
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(bar_t, lane);
      load();
      walk.next(lead, slot);
    };
    walk.next(lead, slot);
    load();
    walk.next(lead, slot);
    setup_done();
    write_t(0);
    for (int j = 0; j < nt; ++j) {
      // the angles of two runs of frequencies, those of the next two follow
      uint4 cs[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) cs[x] = __ldg(ang + x * 128);
      tree_wait(bar_x, j & 1, dead);
      tc_fence_after();
      if (j + 1 < nt) write_t(j + 1);
      // the keys that this buffer held have been read
      if (j >= S::KBufs) tree_wait(bar_s(j - S::KBufs), ((j - S::KBufs) >> 1) & 1, dead);
      tc_fence_after();
      const uint32_t kb = S::tK + t_lane + (j % S::KBufs) * 64 + 4 * NQ * kw;
      const uint32_t x0 = S::tX + t_lane + (j % S::XBufs) * 128 + 8 * NQ * kw;
      // (a key thread of 128 columns has no registers for a second buffer: with
      // one it takes 402 us where one buffer takes 353)
      constexpr int XB = N > 64 ? 1 : 2;
      uint32_t uu[XB][8], vv[XB][8];
      tmem_ld(x0, uu[0]);
      tmem_ld(x0 + 64, vv[0]);
#pragma unroll
      for (int q = 0; q < NQ; ++q) {  // eight frequencies at a time
        if (XB == 1 && q > 0) {
          tmem_ld(x0 + 8 * q, uu[0]);
          tmem_ld(x0 + 64 + 8 * q, vv[0]);
        }
        tmem_wait_ld(uu[q % XB]);
        tmem_wait_ld(vv[q % XB]);
        if (XB == 2 && q + 1 < NQ) {
          tmem_ld(x0 + 8 * (q + 1), uu[(q + 1) % XB]);
          tmem_ld(x0 + 64 + 8 * (q + 1), vv[(q + 1) % XB]);
        }
        if (S::XBufs == 1 && q + 1 == NQ) {  // X has been read
          tc_fence_before();
          warp_arrive(bar_xf, lane);
        }
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const uint4& e = cs[2 * (q & 1) + (f >> 1)];
          const uint32_t cw = (f & 1) ? e.z : e.x, sw = (f & 1) ? e.w : e.y;
          const __half2 c = *reinterpret_cast<const __half2*>(&cw);
          const __half2 s = *reinterpret_cast<const __half2*>(&sw);
          // u and v are integers up to 448: exact in f16
          const __half2 U = __floats2half2_rn(__uint_as_float(uu[q % XB][2 * f]),
                                              __uint_as_float(uu[q % XB][2 * f + 1]));
          const __half2 V = __floats2half2_rn(__uint_as_float(vv[q % XB][2 * f]),
                                              __uint_as_float(vv[q % XB][2 * f + 1]));
          const __half2 a0 = __hfma2(U, c, __hmul2(V, s));
          const __half2 a1 = __hfma2(__hneg2(V), c, __hmul2(U, s));
          lo[f] = *reinterpret_cast<const uint32_t*>(&a0);
          hi[f] = *reinterpret_cast<const uint32_t*>(&a1);
        }
        if (q + 2 < NQ) {
          cs[2 * q] = __ldg(ang + (4 + 2 * q) * 128);
          cs[2 * q + 1] = __ldg(ang + (5 + 2 * q) * 128);
        }
        tmem_st(kb + 4 * q, lo);
        tmem_st(kb + 32 + 4 * q, hi);
      }
      ang += 16 * 128;
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(bar_k(j), lane);
    }
  } else if (warp < R::Softmax0) {
    // ------------------------------------------------------------ values
    set_regs<R::Launch, R::Values>();
    TokenWalk walk(a, u, t0 + t, t1);
    uint32_t wd[4 * BV], meta;
    int32_t lead;
    uint32_t slot;
    const int64_t vhead = h * L.v_in.head_stride;
    bool held;
    auto load = [&]() {  // (without a token vector 0, as for the keys)
      held = lead >= 0;
      const int64_t v = held ? lead * L.v_in.unit_stride + vhead + slot : 0;
#pragma unroll
      for (int i = 0; i < BV; ++i) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(L.v_in.codes + v * (4 * BV)) + i);
        wd[4 * i] = x.x, wd[4 * i + 1] = x.y, wd[4 * i + 2] = x.z, wd[4 * i + 3] = x.w;
      }
      meta = __ldg(L.v_in.meta + v);
    };
    walk.next(lead, slot);
    load();
    walk.next(lead, slot);
    setup_done();
    for (int j = 0; j < nt; ++j) {
      if (j > 1) tree_wait(bar_o(j), ((j >> 1) - 1) & 1, dead);  // the values of tile j-2 have been read
      float m;
      int e;
      if (!held) meta = 0u;  // a weight of 0 must meet a finite value
      value_scale(meta, m, e);
      const uint32_t s16 = __half_as_ushort(
          __float2half_rn(__uint_as_float(static_cast<uint32_t>(125 + e) << 23)));
      const uint32_t ss = s16 | (s16 << 16);
#pragma unroll
      for (int w = 0; w < 4; ++w) {  // 32 codes at a time
        uint32_t x[BV], hh[16];
#pragma unroll
        for (int i = 0; i < BV; ++i) x[i] = wd[w * BV + i];
        tree_unpack<BV>(x, meta >> (4 * w), hh);
#pragma unroll
        for (int q = 0; q < 16; ++q) hh[q] = hmul2u(hh[q], ss);
        const uint32_t dst = base + S::V + (j & 1) * 32768 + (w >> 1) * 16384;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          sts128(dst + row_chunk(t, (w & 1) * 4 + c),
                 make_uint4(hh[4 * c], hh[4 * c + 1], hh[4 * c + 2], hh[4 * c + 3]));
      }
      fence_proxy_async_smem();
      warp_arrive(bar_v(j), lane);
      load();
      walk.next(lead, slot);
    }
  } else if (warp < R::Issue0) {
    // ----------------------------------------------------------- softmax
    // Thread (t, w): token t, query rows HN w .. HN w + HN - 1 of the block.
    setup_done();
    set_regs<R::Launch, R::Softmax>();
    constexpr int HN = N / R::SW;
    static_assert(HN <= 32, "a warp's lanes hold a column each");
    const int w = (warp - R::Softmax0) >> 2, wl = warp & 3;
    const uint32_t bid = 1 + w;  // this warpgroup's named barrier
    float4* fm = reinterpret_cast<float4*>(gen + S::FM) + w * (HN / 2);
    int* wmax = reinterpret_cast<int*>(gen + S::WMax) + w * (HN * 4);
    float l[HN];
#pragma unroll
    for (int c = 0; c < HN; ++c) l[c] = 0.f;
    bool started = false;  // some token of the split was valid

    for (int j = 0; j < nt; ++j) {
      tree_wait(bar_s(j), (j >> 1) & 1, dead);
      tc_fence_after();
      const float kv = reinterpret_cast<const float*>(gen + S::Kap)[(j & 7) * 128 + t];
      const bool valid = kv >= 0.f;
      const float vm = reinterpret_cast<const float*>(gen + S::Vm)[(j & 7) * 128 + t];
      bool raised = false;
      float y[HN];
      {
        constexpr int LD = HN < 16 ? HN : 16;
#pragma unroll
        for (int c0 = 0; c0 < HN; c0 += LD) {
          uint32_t s[LD];
          tmem_ld(tS + t_lane + w * HN + c0, s);
          tmem_wait_ld(s);
#pragma unroll
          for (int c = 0; c < LD; c += 2) {
            const float4 f = fm[(c0 + c) / 2];
            const float2 g = mul2(make_float2(f.x, f.y), make_float2(kv, kv));
            const float2 v = fma2(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])),
                                  g, make_float2(f.z, f.w));
            y[c0 + c] = v.x;
            y[c0 + c + 1] = v.y;
          }
        }
      }
      tc_fence_before();  // S has been read
      warp_arrive(bar_sf, lane);
      if (!valid) {
#pragma unroll
        for (int c = 0; c < HN; ++c) y[c] = -INFINITY;
      }
      float top = y[0];
#pragma unroll
      for (int c = 1; c < HN; ++c) top = fmaxf(top, y[c]);
      const bool raise = named_bar_or(bid, 128, top > kTreeTop || (!started && valid));
      if (j > 1)  // the weights of tile j-2 have been read
        tree_wait(bar_o(j), ((j >> 1) - 1) & 1, dead);
      if (raise && !started) {
        // the first tokens of the split: every column's exact maximum (lane c
        // of a warp: column c), before which the references are 0
        raised = true;
        float x[HN];
#pragma unroll
        for (int c = 0; c < HN; ++c) x[c] = y[c];
        const float k = column_reduce<HN>(x, lane, [](float p, float q) { return fmaxf(p, q); });
        float* fmax4 = reinterpret_cast<float*>(wmax);
        if (lane < HN) fmax4[lane * 4 + wl] = k;
        named_bar_sync(bid, 128);
        if (wl == 0 && lane < HN) {
          const float4 k4 = *reinterpret_cast<const float4*>(fmax4 + lane * 4);
          float* m = reinterpret_cast<float*>(fm + (lane >> 1)) + 2 + (lane & 1);
          *m = kTreeStart - fmaxf(fmaxf(k4.x, k4.y), fmaxf(k4.z, k4.w));
        }
        named_bar_sync(bid, 128);  // the references are written, wmax is free
#pragma unroll
        for (int c = 0; c < HN; c += 2) {
          const float4 f = fm[c / 2];
          y[c] += f.z;
          y[c + 1] += f.w;
        }
      } else if (raise) {
        // the sums are to be rescaled: O at rest (the wait above keeps this
        // barrier from being a phase further)
        if (j > 0) tree_wait(bar_o(j - 1), ((j - 1) >> 1) & 1, dead);
        tc_fence_after();
        raised = true;
        // the columns to move: those past the range
        uint32_t cols = 0u;
#pragma unroll
        for (int c = 0; c < HN; ++c)
          if (y[c] > kTreeTop) cols |= 1u << c;
        cols = __reduce_or_sync(0xffffffffu, cols);
        uint32_t* wor = reinterpret_cast<uint32_t*>(gen + S::WOr) + w * 4;
        if (lane == 0) wor[wl] = cols;
        named_bar_sync(bid, 128);
        const uint4 o4 = *reinterpret_cast<const uint4*>(wor);
        cols = (o4.x | o4.y) | (o4.z | o4.w);
        // their exact maxima over the tile, as ordered integers
#pragma unroll
        for (int c = 0; c < HN; ++c)
          if (cols >> c & 1u) {
            const int i = __float_as_int(y[c]);
            const int k = __reduce_max_sync(0xffffffffu, i ^ ((i >> 31) & 0x7FFFFFFF));
            if (lane == 0) wmax[c * 4 + wl] = k;
          }
        named_bar_sync(bid, 128);
        auto delta_of = [&](int c) {
          const int4 k4 = *reinterpret_cast<const int4*>(wmax + c * 4);
          const int k = max(max(k4.x, k4.y), max(k4.z, k4.w));
          return __int_as_float(k ^ ((k >> 31) & 0x7FFFFFFF)) - kTreeStart;
        };
        if (t < HN && (cols >> t & 1u)) {
          float* m = reinterpret_cast<float*>(fm + (t >> 1)) + 2 + (t & 1);
          *m -= delta_of(t);
        }
#pragma unroll
        for (int c0 = 0; c0 < HN; c0 += 4) {
          if ((cols >> c0 & 15u) == 0u) continue;
          float al[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            al[c] = 1.0f;
            if (cols >> (c0 + c) & 1u) {
              const float d = delta_of(c0 + c);
              y[c0 + c] -= d;
              al[c] = ex2(-d);
              l[c0 + c] *= al[c];
            }
          }
          uint32_t o[4];
          tmem_ld(tO + t_lane + w * HN + c0, o);
          tmem_wait_ld(o);
#pragma unroll
          for (int c = 0; c < 4; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * al[c]);
          tmem_st(tO + t_lane + w * HN + c0, o);
        }
        tmem_wait_st();
        named_bar_sync(bid, 128);  // the references are written, wmax is free
      }
      uint32_t pk[HN / 2];
#pragma unroll
      for (int c = 0; c < HN; c += 2) {
        const float2 p = make_float2(ex2(y[c]), ex2(y[c + 1]));
        const float2 s2 = add2(make_float2(l[c], l[c + 1]), p);
        l[c] = s2.x;
        l[c + 1] = s2.y;
        const float2 pm = mul2(p, make_float2(vm, vm));
        const __half2 ph = __floats2half2_rn(pm.x, pm.y);
        pk[c / 2] = *reinterpret_cast<const uint32_t*>(&ph);
      }
#pragma unroll
      for (int c = 0; c < HN; c += 8) {
        const int col = w * HN + c;
        sts128(base + S::P + (j & 1) * S::PBytes + (col / 64) * 16384 + row_chunk(t, (col % 64) >> 3),
               make_uint4(pk[c / 2], pk[c / 2 + 1], pk[c / 2 + 2], pk[c / 2 + 3]));
      }
      started = started || raised;
      fence_proxy_async_smem();
      tc_fence_before();
      warp_arrive(bar_p(j), lane);
    }
    tree_wait(bar_o(nt - 1), ((nt - 1) >> 1) & 1, dead);
    tc_fence_after();

    // ---- the split's sums: lane = code coordinate of this thread's TMEM lane
    const int coord = 32 * (t >> 5) + tree_slot<BV>(t & 31);
    float* out = part + w * HN * part_row + 2 + coord;
    const int left = a.rows - row0 - w * HN;  // rows of this warpgroup's that exist
#pragma unroll
    for (int c0 = 0; c0 < HN; c0 += 8) {
      uint32_t o[8];
      tmem_ld(tO + t_lane + w * HN + c0, o);
      tmem_wait_ld(o);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if (c0 + c < left) *out = __uint_as_float(o[c]);
        out += part_row;
      }
    }
    float* wsum = reinterpret_cast<float*>(wmax);
    const float k = column_reduce<HN>(l, lane, [](float p, float q) { return p + q; });
    if (lane < HN) wsum[lane * 4 + wl] = k;
    named_bar_sync(bid, 128);
    if (t < HN && row0 + w * HN + t < a.rows) {
      const float4 s = *reinterpret_cast<const float4*>(wsum + t * 4);
      const float* m = reinterpret_cast<const float*>(fm + (t >> 1)) + 2 + (t & 1);
      float* p = part + (w * HN + t) * part_row;
      p[0] = started ? -*m : -INFINITY;
      p[1] = (s.x + s.y) + (s.z + s.w);
    }
    tc_fence_before();
  } else {
    // ---------------------------------------------------------- the MMAs
    setup_done();
    set_regs<R::Launch, R::Issue>();
    // low words of the matrix descriptors (address >> 4, leading offset above
    // bit 16), so that an instruction costs one addition per operand
    const uint32_t b4 = base >> 4;
    constexpr uint32_t iX = idesc_f16_f32(128, 64);
    constexpr uint32_t iS = idesc_f16_f32(128, N), iO = idesc_f16_f32(128, N) | kIdescAMn | kIdescBMn;
    const uint32_t one = elect_lane();
    // two tiles per round, so that everything that an instruction names by
    // the tile's parity is a constant
    if (warp == R::Issue0) {  // X = t H
      auto step = [&](int j, auto parity) {
        constexpr uint32_t d = S::tX + (decltype(parity)::value % S::XBufs) * 128;
        tree_wait(bar_t, j & 1, dead);
        if (S::XBufs == 1 && j > 0) tree_wait(bar_xf, (j - 1) & 1, dead);
        tc_fence_after();
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_f16_ta_if(one, d + 64 * hf, S::tT + 32 * hf + 8 * k,
                           tree_desc(b4 + ((S::H + k * 32) >> 4), 1u), iX, k > 0);
        umma_commit_if(one, bar_x);
      };
      for (int j = 0; j < nt; j += 2) {
        step(j, Parity<0>());
        if (j + 1 < nt) step(j + 1, Parity<1>());
      }
    } else if (warp == R::Issue0 + 1) {  // S = keys Q^T
      auto step = [&](int j, auto parity) {
        constexpr int q = decltype(parity)::value;
        tree_wait(bar_k(q), (j >> 1) & 1, dead);
        if (j > 0) tree_wait(bar_sf, (j - 1) & 1, dead);
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 8; ++k)
          umma_f16_ta_if(one, tS, S::tK + (q % S::KBufs) * 64 + 8 * k,
                         tree_desc(b4 + ((S::Q + (k >> 2) * (N * 128) + (k & 3) * 32) >> 4), 1u), iS,
                         k > 0);
        umma_commit_if(one, bar_s(q));
        // orders the key scales, which this warp's wait for the keys has
        // acquired, before the softmax threads' reads
        if (lane == 0) mbar_arrive(bar_s(q));
        __syncwarp();
      };
      for (int j = 0; j < nt; j += 2) {
        step(j, Parity<0>());
        if (j + 1 < nt) step(j + 1, Parity<1>());
      }
    } else if (warp == R::Issue0 + 2) {  // O += V P
      auto step = [&](int j, auto parity) {
        constexpr int q = decltype(parity)::value;
        tree_wait(bar_v(q), (j >> 1) & 1, dead);
        tree_wait(bar_p(q), (j >> 1) & 1, dead);
        tc_fence_after();
        const uint32_t more = j > 0;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          umma_f16_if(one, tO, tree_desc(b4 + ((S::V + q * 32768 + k * 2048) >> 4), 16384u >> 4),
                      tree_desc(b4 + ((S::P + q * S::PBytes + k * 2048) >> 4), 16384u >> 4), iO,
                      k > 0 ? 1u : more);
        umma_commit_if(one, bar_o(q));
      };
      for (int j = 0; j < nt; j += 2) {
        step(j, Parity<0>());
        if (j + 1 < nt) step(j + 1, Parity<1>());
      }
    }
  }
  __syncthreads();
  if (warp == R::Issue0) {
    tc_fence_after();
    tmem_dealloc(0u, kCols);
  }
}

// One warp per row: merge the splits, apply H, attend the draft nodes that
// the row sees (fp32).  Lane l owns coordinates l, l+32, l+64, l+96; a draft
// score takes eight lanes (16 coordinates each).  Latency counts here: the
// loads of a phase are independent of each other.  8 to 22 us in the calls
// above, a launch of latency in the shortest ones.
constexpr int kCombineWarps = 4;

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Shared words of a warp: split factors, the draft nodes seen, their scores
// (then weights), the query.
__host__ __device__ constexpr int combine_floats(int nsplit, int nodes) {
  return (nsplit + 2 * nodes + 3) / 4 * 4 + kD;  // the query 16-byte aligned
}

__global__ void __launch_bounds__(32 * kCombineWarps) tree_combine_kernel(const TreeArgs a) {
  extern __shared__ float combine_smem[];
  const TreeLaunch& L = a.L;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kCombineWarps + (threadIdx.x >> 5);
  if (w >= static_cast<int64_t>(L.units) * L.heads * a.rows) return;
  const int ns = static_cast<int>(a.nsplit);
  float* fac = combine_smem + (threadIdx.x >> 5) * combine_floats(ns, L.nodes);
  float* sc = fac + ns;
  int* list = reinterpret_cast<int*>(sc + L.nodes);
  float* qs = fac + combine_floats(ns, L.nodes) - kD;
  const int r = static_cast<int>(w % a.rows);
  const int64_t uh = w / a.rows, u = uh / L.heads;
  const int h = static_cast<int>(uh % L.heads), node = r / L.G, j = h * L.G + r % L.G;
  const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(L.q) + u * L.qs.unit +
                            j * L.qs.head + node * L.qs.token;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    qs[lane + 32 * i] = __bfloat162float(qp[lane + 32 * i]) * (L.scale * kLog2e);
  const float* part = a.part + w * a.nsplit * kTreePart;
  float top = -INFINITY;
  for (int s = lane; s < ns; s += 32) {
    const float m = part[static_cast<int64_t>(s) * kTreePart];
    fac[s] = m;
    top = fmaxf(top, m);
  }
  __syncwarp();

  // the nodes that the row sees, in order
  const int words = (L.nodes + 63) / 64;
  int seen = 0;
  if (!L.mask) {  // a chain sees nodes 0 .. node
    seen = node + 1;
    for (int k = lane; k < seen; k += 32) list[k] = k;
  } else {
    const uint32_t* mask = reinterpret_cast<const uint32_t*>(
        L.mask + u * L.mask_stride + static_cast<int64_t>(node) * words);
    for (int k0 = 0; k0 < L.nodes; k0 += 32) {
      uint32_t bits = __ldg(mask + (k0 >> 5));
      if (L.nodes - k0 < 32) bits &= (1u << (L.nodes - k0)) - 1u;
      if (bits >> lane & 1u) list[seen + __popc(bits & ((1u << lane) - 1u))] = k0 + lane;
      seen += __popc(bits);
    }
  }
  __syncwarp();

  // their scores, four nodes at a time
  const __nv_bfloat16* Kn = static_cast<const __nv_bfloat16*>(L.K_new) + u * L.kns.unit + h * L.kns.head;
  const __nv_bfloat16* Vn = static_cast<const __nv_bfloat16*>(L.V_new) + u * L.vns.unit + h * L.vns.head;
#pragma unroll 2
  for (int k0 = 0; k0 < seen; k0 += 4) {
    const int k = k0 + (lane >> 3), e = lane & 7;  // lane e: coordinates 8e .. +7, 64 + 8e .. +7
    float s = 0.f;
    if (k < seen) {
      const uint4* src = reinterpret_cast<const uint4*>(Kn + list[k] * L.kns.token);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const uint4 v = __ldg(src + 8 * hf + e);
        const float4 q0 = *reinterpret_cast<const float4*>(qs + 64 * hf + 8 * e);
        const float4 q1 = *reinterpret_cast<const float4*>(qs + 64 * hf + 8 * e + 4);
        s = __fmaf_rn(bf16lo(v.x), q0.x, s);
        s = __fmaf_rn(bf16hi(v.x), q0.y, s);
        s = __fmaf_rn(bf16lo(v.y), q0.z, s);
        s = __fmaf_rn(bf16hi(v.y), q0.w, s);
        s = __fmaf_rn(bf16lo(v.z), q1.x, s);
        s = __fmaf_rn(bf16hi(v.z), q1.y, s);
        s = __fmaf_rn(bf16lo(v.w), q1.z, s);
        s = __fmaf_rn(bf16hi(v.w), q1.w, s);
      }
    }
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (k < seen) {
      if (e == 0) sc[k] = s;
      top = fmaxf(top, s);
    }
  }

  // the common reference of the splits and the draft, then the factors
  const float M = warp_max(top), ref = M == -INFINITY ? 0.f : M;
  __syncwarp();
  float l = 0.f;
  for (int s = lane; s < ns; s += 32) {
    const float f = exp2f(fac[s] - ref);  // 0 for a split without tokens
    fac[s] = f;
    if (f > 0.f) l = __fmaf_rn(f, part[static_cast<int64_t>(s) * kTreePart + 1], l);
  }
  for (int k = lane; k < seen; k += 32) {
    const float p = exp2f(sc[k] - ref);
    sc[k] = p;
    l += p;
  }
  const float sum = warp_sum(l);
  __syncwarp();

  float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < ns; ++s) {
    const float f = fac[s];
    if (f > 0.f) {
      const float* p = part + static_cast<int64_t>(s) * kTreePart + 2 + lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = __fmaf_rn(f, p[32 * i], o[i]);
    }
  }
  // H: stages 1 .. 16 across lanes, 32 and 64 in the lane
#pragma unroll
  for (int st = 1; st < 32; st <<= 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = __shfl_xor_sync(0xffffffffu, o[i], st);
      o[i] = (lane & st) ? x - o[i] : o[i] + x;
    }
  }
  // the sums are of sigma t / 4: v = (sigma / 2) C H t
  const float kv = 2.0f * __uint_as_float(kCBits);
  const float x0 = (o[0] + o[1]) * kv, x1 = (o[0] - o[1]) * kv;
  const float x2 = (o[2] + o[3]) * kv, x3 = (o[2] - o[3]) * kv;
  o[0] = x0 + x2;
  o[2] = x0 - x2;
  o[1] = x1 + x3;
  o[3] = x1 - x3;

#pragma unroll 4
  for (int k = 0; k < seen; ++k) {
    const float p = sc[k];
    const __nv_bfloat16* v = Vn + list[k] * L.vns.token + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __fmaf_rn(p, __bfloat162float(v[32 * i]), o[i]);
  }
  const float inv = sum > 0.f ? 1.0f / sum : 0.f;
  __nv_bfloat16* op = static_cast<__nv_bfloat16*>(L.out) + u * L.os.unit + j * L.os.head +
                      node * L.os.token;
#pragma unroll
  for (int i = 0; i < 4; ++i) op[lane + 32 * i] = __float2bfloat16_rn(o[i] * inv);
  if (L.lse && lane == 0)
    L.lse[(u * L.heads * L.G + j) * L.nodes + node] =
        sum > 0.f ? (ref + log2f(sum)) * kLn2 : -INFINITY;
}

// ------------------------------------------------------------------ launch
constexpr int kTreeTileCost[4] = {31, 33, 41, 59};

struct TreePlan {
  int cols, rblocks;
  int64_t tiles, per, nsplit;
};

// Rows per CTA (columns of the products): the width whose blocks take the
// least time together.  A tile takes 31, 33, 41 and 59 units with 16, 32, 64
// and 128 columns (measured on 32 x 8 x 13 147 tokens: 306, 330, 405, 592 us of
// this kernel; below 64 columns the keys are the work), so two blocks of 64
// lose to one of 128, and three to two (160 rows on that shape: 1200 against
// 1100 us per call; 132 rows, 1180 against 1075).
// Splits: the launch costs (waves of 148 CTAs) * (tiles per CTA + setup, about
// three tiles); the smallest cost, the fewest splits among equals.  Units that
// may hold fewer than n tokens (their lengths are on the device) even out only
// over CTAs much shorter than the launch: there a CTA takes at most a fourth
// of an SM's even share, but 12 tiles at least.
static TreePlan tree_plan(int units, int heads, int G, int nodes, int64_t n, bool ragged) {
  TreePlan p{};
  const int64_t rows = static_cast<int64_t>(nodes) * G;
  int64_t least = -1;
  for (int i = 0; i < 4; ++i) {
    const int cols = 16 << i;
    const int64_t blocks = (rows + cols - 1) / cols, cost = blocks * kTreeTileCost[i];
    if (least < 0 || cost < least) {
      least = cost;
      p.cols = cols;
      p.rblocks = static_cast<int>(blocks);
    }
  }
  p.tiles = (n + kTreeTile - 1) / kTreeTile;
  if (p.tiles < 1) p.tiles = 1;
  const int64_t ctas = static_cast<int64_t>(units) * heads * p.rblocks;
  int64_t most = p.tiles;
  if (ragged && units > 1) {
    most = ctas * p.tiles / (148 * 4);
    most = most < 12 ? 12 : most;
  }
  int64_t best = -1;
  for (int64_t s = 1; s <= p.tiles && s <= kTreeMaxSplits; ++s) {
    const int64_t per = (p.tiles + s - 1) / s, ns = (p.tiles + per - 1) / per;
    if (per > most && s < p.tiles && s < kTreeMaxSplits) continue;
    const int64_t cost = (ctas * ns + 147) / 148 * (per + 3);
    if (best < 0 || cost < best) {
      best = cost;
      p.per = per;
      p.nsplit = ns;
    }
    if (best >= 0 && ctas * s >= 8 * 148 && s > 1) break;  // finer splits only add setup
  }
  return p;
}

static size_t tree_part_bytes(int units, int heads, int G, int nodes, const TreePlan& p) {
  const size_t b = static_cast<size_t>(units) * heads * G * nodes * p.nsplit * kTreePart * sizeof(float);
  return (b + 255) / 256 * 256;
}

size_t tree_workspace_bytes(int units, int heads, int G, int nodes, int64_t n, bool shared,
                            bool ragged) {
  const TreePlan p = tree_plan(units, heads, G, nodes, n, ragged);
  return tree_part_bytes(units, heads, G, nodes, p) +
         static_cast<size_t>(shared ? 1 : units) * p.tiles * 16 * 128 * sizeof(uint4);
}

int64_t tree_ctas(int units, int heads, int G, int nodes, int64_t n, bool ragged) {
  const TreePlan p = tree_plan(units, heads, G, nodes, n, ragged);
  const int64_t a = static_cast<int64_t>(units) * heads * p.rblocks * p.nsplit;
  const int64_t b = static_cast<int64_t>(units) * p.tiles;
  return a > b ? a : b;
}

template <int BK, int BV, int N>
static cudaError_t launch_tree_n(const TreeArgs& a, int64_t grid, cudaStream_t stream) {
  constexpr int smem = TreeSmem<BK, BV, N>::Bytes;
  cudaError_t err = cudaFuncSetAttribute(tree_partial_kernel<BK, BV, N>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  tree_partial_kernel<BK, BV, N><<<static_cast<unsigned>(grid), TreeRoles<N>::Threads, smem, stream>>>(a);
  return cudaGetLastError();
}

template <int BK, int BV>
static cudaError_t launch_tree_partial(const TreeArgs& a, int64_t grid, cudaStream_t stream) {
  switch (a.ncols) {
    case 16: return launch_tree_n<BK, BV, 16>(a, grid, stream);
    case 32: return launch_tree_n<BK, BV, 32>(a, grid, stream);
    case 64: return launch_tree_n<BK, BV, 64>(a, grid, stream);
    default: return launch_tree_n<BK, BV, 128>(a, grid, stream);
  }
}

cudaError_t launch_tree_attend(const TreeLaunch& L, cudaStream_t stream) {
  TreeArgs a{};
  a.L = L;
  a.rows = L.nodes * L.G;
  a.n_a = (L.rope_max_pos + 255) / 256;
  if (L.n > 0) {
    const TreePlan p = tree_plan(L.units, L.heads, L.G, L.nodes, L.n, L.lens != nullptr);
    a.ncols = p.cols;
    a.page = make_fastdiv(static_cast<uint32_t>(L.table ? L.page_size : 1));
    a.rblocks = p.rblocks;
    a.tiles = p.tiles;
    a.per = p.per;
    a.nsplit = p.nsplit;
    a.part = static_cast<float*>(L.ws);
    a.angles = reinterpret_cast<uint4*>(static_cast<char*>(L.ws) +
                                        tree_part_bytes(L.units, L.heads, L.G, L.nodes, p));
    a.angle_stride = L.positions ? p.tiles * 16 * 128 : 0;
    const int64_t agrid = p.tiles * (L.positions ? L.units : 1);
    tree_angles_kernel<<<static_cast<unsigned>(agrid), kAngleThreads, 0, stream>>>(a);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    const int64_t grid = static_cast<int64_t>(L.units) * L.heads * p.rblocks * p.nsplit;
    const int bk = L.k_in.bits, bv = L.v_in.bits;
    err = bk == 3 ? (bv == 3 ? launch_tree_partial<3, 3>(a, grid, stream)
                             : launch_tree_partial<3, 2>(a, grid, stream))
                  : (bv == 3 ? launch_tree_partial<2, 3>(a, grid, stream)
                             : launch_tree_partial<2, 2>(a, grid, stream));
    if (err != cudaSuccess) return err;
  }
  const int64_t rows = static_cast<int64_t>(L.units) * L.heads * a.rows;
  const int smem = kCombineWarps * combine_floats(static_cast<int>(a.nsplit), L.nodes) *
                   static_cast<int>(sizeof(float));  // at most 44 KB
  tree_combine_kernel<<<static_cast<unsigned>((rows + kCombineWarps - 1) / kCombineWarps),
                        32 * kCombineWarps, smem, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t tree_read_clear_error(uint32_t* flags) {
  unsigned int v = 0, zero = 0;
  cudaError_t err = cudaMemcpyFromSymbol(&v, g_nq_error, sizeof(v));
  if (err != cudaSuccess) return err;
  if ((err = cudaMemcpyToSymbol(g_nq_error, &zero, sizeof(zero))) != cudaSuccess) return err;
  *flags = v;
  return cudaSuccess;
}

}  // namespace nq

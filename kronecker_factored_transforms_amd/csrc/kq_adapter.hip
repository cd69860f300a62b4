// kq_adapter.hip -- low-rank adapters of many requests at once, beside a shared projection:
//
//   out[t] = cvt( base[t] + scaling[l] * B[l] (A[l] x[t]) ),   l = adapter[t].
//
// Two kernels. The first forms the low-rank vectors h[t] = A[l] x[t] (K long, r short) and splits
// K over workgroups where tokens are few; each part goes to the workspace as fp32. The second
// adds the parts up in their order (no atomics: the result does not depend on which workgroup
// ends first), scales, and forms B[l] h + base. (From 1024 to 4095 tokens a third in between adds
// up the parts.) Rounded to 16 bits, h would lose what fp32 sums gained: it enters the second
// product as two 16-bit terms, hi + lo, on twice the instructions, which the memory's time hides.
//
// Up to 16 tokens on few small adapters take one kernel that does both (see there).
//
// Bound by memory for prompts (x, base and out once): 8192 tokens, K = N = 4096, r 16 48 us, 0.81
// of the time that their bytes take at a copy's rate (5.2 TB/s); K 4096, N 14336, r 64 150 us,
// 0.71: there h's operands, B and the products add to each wave's chain. By the two kernels'
// latency for decode: 128 tokens on 32 adapters, r 16, K = N = 8192 15.6 us;
// one token, r 16, K = N = 4096 5.2 us.
//
// Both take blocks of 16 tokens as they stand: for each adapter that occurs among them, one
// product of its matrix with all 16 columns, of which the tokens of that adapter keep theirs (a
// selection, not a product with zero: another adapter's infinities and NaN stay out). The tokens
// of a prompt stand together, so most of its blocks have one adapter; the many of a decode
// batch's blocks are loaded several at a time.
#include "kq_internal.h"
#include "kq_device.h"
#include "kq_linear.h"

namespace {

constexpr int kMaxRank = 256;
constexpr int64_t kMaxDim = 1 << 20;
constexpr int64_t kMaxTokens = 1 << 27;  // the grid's threads stay below 2^32

template <int DT>
struct Half;
template <>
struct Half<0> {  // bf16
  typedef bf16x8 vec;
  typedef __bf16 one;
  static __device__ __forceinline__ f32x4 mma(const vec &a, const vec &b, const f32x4 &c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ one round(float v) { return (one)v; }
};
template <>
struct Half<1> {  // fp16
  typedef f16x8 vec;
  typedef _Float16 one;
  static __device__ __forceinline__ f32x4 mma(const vec &a, const vec &b, const f32x4 &c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ one round(float v) { return half_rne(v); }
};

struct AdapterArgs {
  const void *x, *A, *B, *base;
  const int32_t *adapter;
  const float *scaling;
  void *out;
  float *part;  // h's parts, and h as operands: what lies between the kernels, see below
  void *ops;
  int64_t ldx, ldb, ldo, T;
  int K, N, r, L, splits, split_steps;  // a step: kStep values of K
  int tiles_per_group;                  // up: token tiles of one workgroup
};

// What lies between the kernels. The parts of h over K, fp32, [splits][T][ranks up to a multiple
// of 16]; and h as the last product's operands, [tile of 16 tokens][steps of 32 ranks][first,
// second term][lane][8 values], with the exponent of the power of two that each token's h was
// multiplied by, [tile][16]. Few tokens: parts, which the last kernel adds up itself; from kJoin
// tokens on: parts, and a kernel in between that makes the operands of them (each would be added
// up for every 256 columns otherwise); from kWide on: K is whole, and the first kernel makes them.
constexpr int64_t kJoin = 1024, kWide = 4096;

constexpr int kParts = 8;  // of K, at most

__device__ __forceinline__ int round16(int r) { return (r + 15) / 16 * 16; }

// Token t's adapter, -1 for none
__device__ __forceinline__ int token_adapter(const AdapterArgs &p, int64_t t) {
  const int l = t < p.T ? p.adapter[t] : -1;
  return l >= 0 && l < p.L ? l : -1;
}

// The next adapter of `left` (one bit per token of a tile, `l` its adapters), -1 at the end;
// wave-uniform
__device__ __forceinline__ int next_adapter(unsigned long long &left, int l) {
  if (!left) return -1;
  const int a = __builtin_amdgcn_readlane(l, __builtin_ctzll(left));
  left &= ~__ballot(l == a);
  return a;
}

// h of one token (lane: ranks 32 s + 8 g + 0..7) as two 16-bit terms. fp16: a power of two per
// token brings its h into the type's range (exact; undone on the sums), so that neither term
// overflows or loses bits; returns its exponent. bf16 has fp32's range.
template <int DT, int RS>
__device__ __forceinline__ int two_terms(const float (&h)[RS][8], typename Half<DT>::vec (&hi)[RS],
                                         typename Half<DT>::vec (&lo)[RS]) {
  typedef typename Half<DT>::one one;
  int ex = 0;
  if constexpr (DT == 1) {
    float top = 0.f;
#pragma unroll
    for (int s = 0; s < RS; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(h[s][e]));
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const int be = (int)(__float_as_uint(top) >> 23);
    ex = be == 0 || be == 255 ? 0 : 127 + 14 - be;
  }
#pragma unroll
  for (int s = 0; s < RS; ++s)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float v = DT == 1 ? __builtin_ldexpf(h[s][e], ex) : h[s][e];
      const one a = Half<DT>::round(v);
      hi[s][e] = a;
      lo[s][e] = Half<DT>::round(__builtin_isfinite((float)a) ? __fsub_rn(v, (float)a) : 0.f);
    }
  return ex;
}

// A tile's operands: the terms of two_terms() as the lanes hold them, and the exponents
template <int DT, int RS>
__device__ __forceinline__ void store_operands(const AdapterArgs &p, int64_t tile, int64_t tiles,
                                               const typename Half<DT>::vec (&hi)[RS],
                                               const typename Half<DT>::vec (&lo)[RS], int ex) {
  const int lane = threadIdx.x & 63;
  auto *o = reinterpret_cast<typename Half<DT>::vec *>(p.ops);
#pragma unroll
  for (int s = 0; s < RS; ++s) {
    o[tile * (RS * 2 * 64) + (2 * s) * 64 + lane] = hi[s];
    o[tile * (RS * 2 * 64) + (2 * s + 1) * 64 + lane] = lo[s];
  }
  if (lane < 16) reinterpret_cast<int *>(o + tiles * (RS * 2 * 64))[tile * 16 + lane] = ex;
}

constexpr int kStep = 64;  // values of K per step: rows of 128 bytes in LDS

// The products of DD adapters' A (numbers a[]) with TF blocks of 16 tokens, over one wave's steps
// s0, s0 + WAVES, .. of K below s1; RB blocks of 16 ranks. Rows come by DMA into the wave's own
// ring of LDS (no barrier), 8 rows of 128 bytes at a time: read straight into the operands, 16
// rows lie behind each other's 16 bytes and every lane is a memory access of its own. Piece p of
// row R lies at position p ^ ((R / 2) % 8): the 16 rows of a fragment read spread over all banks.
template <int DT, int RB, int TF, int WAVES, int DD, int RING>
__device__ __forceinline__ void down_product(const AdapterArgs &p, int64_t t0, const int *a, int s0, int s1,
                                             unsigned char *ring, f32x4 (&acc)[DD][RB][TF]) {
  typedef typename Half<DT>::vec vec;
  constexpr int kX = 2 * TF, kA = 2 * RB;           // DMA instructions for x, for one A
  constexpr int kLoads = kX + DD * kA;              // per step
  constexpr int kMost = RING / (kLoads * 1024);
  constexpr int kStages = kMost > 4 ? 4 : kMost;
  static_assert(kStages >= 2 && kLoads * (kStages - 1) < 64, "two steps in LDS, loads within the counter");
  const int lane = threadIdx.x & 63, g = lane >> 4, lr = lane & 15;
  // offsets from x's row t0 and from A's first row; rows past the end read a valid row, and
  // what comes of them is dropped
  uint32_t vx[kX], va[kA];
  int piece[2];  // of an even and an odd instruction's rows
#pragma unroll
  for (int j = 0; j < 2; ++j) piece[j] = (lane % 8) ^ (((8 * j + lane / 8) >> 1) & 7);
#pragma unroll
  for (int j = 0; j < kX; ++j) {
    const int R = 8 * j + lane / 8;
    const int64_t row = t0 + R < p.T ? R : p.T - 1 - t0;
    vx[j] = (uint32_t)(row * p.ldx * 2 + piece[j % 2] * 16);
  }
#pragma unroll
  for (int j = 0; j < kA; ++j) va[j] = (uint32_t)min(8 * j + lane / 8, p.r - 1) * (uint32_t)(p.K * 2) + piece[j % 2] * 16;
  const unsigned char *x = uniform(reinterpret_cast<const uint16_t *>(p.x) + t0 * p.ldx);
  const unsigned char *am[DD];
#pragma unroll
  for (int d = 0; d < DD; ++d)
    am[d] = uniform(reinterpret_cast<const uint16_t *>(p.A) + (int64_t)a[d] * p.r * p.K);
#pragma unroll
  for (int d = 0; d < DD; ++d)
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int f = 0; f < TF; ++f) acc[d][b][f] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int pieces = p.K / 8;
  auto load_step = [&](int s, int b) {
    unsigned char *to = ring + b * (kLoads * 1024);
    const int64_t o = (int64_t)s * (kStep * 2);
    if (s * 8 + 8 <= pieces) {
#pragma unroll
      for (int j = 0; j < kX; ++j) dma16<false>(x + o, vx[j], lds_addr(to + j * 1024));
#pragma unroll
      for (int d = 0; d < DD; ++d)
#pragma unroll
        for (int j = 0; j < kA; ++j) dma16<false>(am[d] + o, va[j], lds_addr(to + (kX + d * kA + j) * 1024));
    } else {  // the rows end inside this step: the rest comes from a block of zeros
#pragma unroll
      for (int j = 0; j < kX; ++j)
        dma16_addr<false>(s * 8 + piece[j % 2] < pieces ? x + o + vx[j] : kZeros, lds_addr(to + j * 1024));
#pragma unroll
      for (int d = 0; d < DD; ++d)
#pragma unroll
        for (int j = 0; j < kA; ++j)
          dma16_addr<false>(s * 8 + piece[j % 2] < pieces ? am[d] + o + va[j] : kZeros,
                            lds_addr(to + (kX + d * kA + j) * 1024));
    }
  };
  const int steps = s0 < s1 ? (s1 - s0 + WAVES - 1) / WAVES : 0;
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k)
    if (k < steps) load_step(s0 + k * WAVES, k);
  const int sw = (lr >> 1) & 7;
  int b = 0;
  for (int k = 0; k < steps; ++k) {
    if (k + kStages - 1 < steps) {
      load_step(s0 + (k + kStages - 1) * WAVES, b == 0 ? kStages - 1 : b - 1);
      wait_and_fence<wait_vm_imm(kLoads * (kStages - 1))>();
    } else {
      wait_and_fence<kWaitVm0>();
    }
    const unsigned char *from = ring + b * (kLoads * 1024);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int off = lr * 128 + ((4 * q + g) ^ sw) * 16;
      vec xv[TF];
#pragma unroll
      for (int f = 0; f < TF; ++f) xv[f] = *reinterpret_cast<const vec *>(from + f * 2048 + off);
#pragma unroll
      for (int d = 0; d < DD; ++d)
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
          const vec av = *reinterpret_cast<const vec *>(from + (kX + d * kA + 2 * rb) * 1024 + off);
#pragma unroll
          for (int f = 0; f < TF; ++f) acc[d][rb][f] = Half<DT>::mma(av, xv[f], acc[d][rb][f]);
        }
    }
    wait_and_fence<kWaitLgkm0>();  // this step's reads have returned: its place may be overwritten
    b = b + 1 == kStages ? 0 : b + 1;
  }
}

// h of TF blocks of 16 tokens over a share of K, which the waves split again and add up in LDS;
// D adapters at a time. OPERANDS: h is whole, and is left scaled and as operands.
template <int DT, int RB, int TF, int WAVES, int D, int RING, bool OPERANDS>
__global__ __launch_bounds__(WAVES * 64) void kq_adapter_down_kernel(const AdapterArgs p) {
  constexpr int RS = (RB + 1) / 2;
  constexpr int kRow = 32 * RS + 4;  // of h in LDS, floats: rows 4 banks apart
  constexpr int kSum = WAVES * D * RB * TF * 1024, kH = OPERANDS ? 16 * TF * kRow * 4 : 0;
  constexpr int kAcc = kSum + kH;
  constexpr int kLds = WAVES * RING > kAcc ? WAVES * RING : kAcc;
  __shared__ __align__(16) unsigned char s_mem[kLds];
  f32x4 *s_acc = reinterpret_cast<f32x4 *>(s_mem);           // [WAVES][D RB TF][64], behind the rings' use
  float *s_h = reinterpret_cast<float *>(s_mem + kLds - kH);  // [16 TF][kRow]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, lr = lane & 15;
  const int64_t t0 = (int64_t)blockIdx.x * (16 * TF);
  // lanes 0..15 of the wave stand for block 0's tokens, 16..31 for block 1's
  const int mine = token_adapter(p, t0 + (lane & (16 * TF - 1)));
  int l[TF];
#pragma unroll
  for (int f = 0; f < TF; ++f) l[f] = __shfl(mine, 16 * f + lr, 64);
  const int s0 = blockIdx.y * p.split_steps + wave;
  const int s1 = min((p.K + kStep - 1) / kStep, ((int)blockIdx.y + 1) * p.split_steps);
  f32x4 kept[OPERANDS ? (RB * TF + WAVES - 1) / WAVES : 1];  // this wave's blocks of h, of all adapters
#pragma unroll
  for (f32x4 &v : kept) v = f32x4{0.f, 0.f, 0.f, 0.f};
  unsigned long long left = __ballot(mine >= 0) & ((1ull << (16 * TF)) - 1);
  auto put = [&](int d, const f32x4 (&acc)[RB][TF]) {  // one adapter's accumulators of this wave
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int f = 0; f < TF; ++f) s_acc[((wave * D + d) * RB * TF + b * TF + f) * 64 + lane] = acc[b][f];
  };
  auto sum = [&](int a, int d) {  // lane: ranks 16 b + 4 g + 0..3 of token 16 f + lr
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int f = 0; f < TF; ++f) {
        const int i = b * TF + f;
        if (i % WAVES != wave) continue;
        f32x4 v = s_acc[(d * RB * TF + i) * 64 + lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) v += s_acc[((w * D + d) * RB * TF + i) * 64 + lane];
        if (l[f] != a) continue;
        if constexpr (OPERANDS)
          kept[i / WAVES] = v;
        else if (16 * b < round16(p.r))
          *reinterpret_cast<f32x4 *>(p.part +
                                     ((int64_t)blockIdx.y * p.T + t0 + 16 * f + lr) * round16(p.r) + 16 * b +
                                     4 * g) = v;
      }
  };
  for (int group = 0; left; ++group) {
    int a[D], n = 0;
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int next = next_adapter(left, mine);
      a[d] = next < 0 ? a[0] : next;  // a short group's rest: its first adapter again, dropped
      n += next >= 0;
    }
    if (group % (int)gridDim.z != (int)blockIdx.z) continue;  // another workgroup's
    unsigned char *ring = s_mem + wave * RING;
    if (n == 1) {
      f32x4 acc[1][RB][TF];
      down_product<DT, RB, TF, WAVES, 1, RING>(p, t0, a, s0, s1, ring, acc);
      lds_barrier();
      put(0, acc[0]);
    } else if constexpr (D > 1) {
      f32x4 acc[D][RB][TF];
      down_product<DT, RB, TF, WAVES, D, RING>(p, t0, a, s0, s1, ring, acc);
      lds_barrier();
#pragma unroll
      for (int d = 0; d < D; ++d) put(d, acc[d]);
    }
    lds_barrier();
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (d < n) sum(a[d], d);
    lds_barrier();  // before the rings are written again
  }
  if constexpr (OPERANDS) {
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int f = 0; f < TF; ++f) {
        const int i = b * TF + f;
        if (i % WAVES == wave)
          *reinterpret_cast<f32x4 *>(s_h + (16 * f + lr) * kRow + 16 * b + 4 * g) = kept[i / WAVES];
      }
    lds_barrier();
    for (int f = wave; f < TF; f += WAVES) {
      const int lf = __shfl(mine, 16 * f + lr, 64);
      const float sc = lf >= 0 && p.scaling ? p.scaling[lf] : 1.0f;
      float h[RS][8];
#pragma unroll
      for (int s = 0; s < RS; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int k = 32 * s + 8 * g + e;
          h[s][e] = k < p.r ? __fmul_rn(s_h[(16 * f + lr) * kRow + k], sc) : 0.f;
        }
      typename Half<DT>::vec hi[RS], lo[RS];
      const int ex = two_terms<DT, RS>(h, hi, lo);
      const int64_t tile = t0 / 16 + f, tiles = (p.T + 15) / 16;
      if (tile < tiles) store_operands<DT, RS>(p, tile, tiles, hi, lo, ex);
    }
  }
}

// The operands of one tile of 16 tokens, from the parts of its h: one wave
template <int DT, int RS>
__global__ __launch_bounds__(64) void kq_adapter_join_kernel(const AdapterArgs p) {
  const int lane = threadIdx.x & 63, g = lane >> 4, lr = lane & 15;
  const int64_t tile = blockIdx.x, t = tile * 16 + lr, tc = t < p.T ? t : p.T - 1;
  const int l = token_adapter(p, t), r16 = round16(p.r);
  const float sc = l >= 0 && p.scaling ? p.scaling[l] : 1.0f;
  const float *q = p.part + tc * r16;
  float h[RS][8];
#pragma unroll
  for (int s = 0; s < RS; ++s) {
    const int k = 32 * s + 8 * g;
    const bool in = k < p.r;
    f32x4 w[kParts][2];
#pragma unroll
    for (int i = 0; i < kParts; ++i)
      if (i < p.splits)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          w[i][e] = *reinterpret_cast<const f32x4 *>(q + i * (p.T * r16) + (in ? k : 0) + 4 * e);
#pragma unroll
    for (int i = 1; i < kParts; ++i)
      if (i < p.splits)
#pragma unroll
        for (int e = 0; e < 2; ++e) w[0][e] += w[i][e];
    // what a token without an adapter has there is not written, and dropped
#pragma unroll
    for (int e = 0; e < 8; ++e) h[s][e] = l >= 0 && in ? __fmul_rn(w[0][e / 4][e % 4], sc) : 0.f;
  }
  typename Half<DT>::vec hi[RS], lo[RS];
  const int ex = two_terms<DT, RS>(h, hi, lo);
  store_operands<DT, RS>(p, tile, (p.T + 15) / 16, hi, lo, ex);
}

constexpr int kUpWaves = 4;

// out. A workgroup takes 256 columns (64 per wave; 32 beyond 64 ranks) of tiles_per_group tiles
// of 16 tokens; RS steps of 32 ranks; D adapters' B at a time. A tile's sums go through the
// wave's own part of LDS, so that 8 (4) lanes read and write the 128 (64) bytes of one row of
// base and out: in the product's own layout every lane is a row of its own, and each 16 bytes a
// memory access of its own. A tile's base and h are on their way while the one before it is
// computed. OPERANDS: what lies between the kernels, see above.
template <int DT, int RS, int NB, int D, bool OPERANDS>
__global__ __launch_bounds__(kUpWaves * 64) void kq_adapter_up_kernel(const AdapterArgs p) {
  typedef typename Half<DT>::vec vec;
  typedef typename Half<DT>::one one;
  constexpr int kRow = 16 * NB + 4;                      // floats of a row in LDS: all banks in turn
  constexpr int kLanes = 2 * NB, kPasses = NB / 2;       // lanes of a row of base and out
  constexpr int kHRow = 32 * RS + 4;
  __shared__ __align__(16) float s_out[kUpWaves][16 * kRow];
  __shared__ __align__(16) float s_h[OPERANDS ? 1 : 2][OPERANDS ? 4 : 16 * kHRow];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, lr = lane & 15;
  const int n0 = (int)(blockIdx.x * kUpWaves + wave) * 16 * NB;
  if (OPERANDS && n0 >= p.N) return;  // whole waves; there is no barrier then
  int64_t tile = (int64_t)blockIdx.y * p.tiles_per_group;
  const int64_t tiles = (p.T + 15) / 16, last = min(tile + p.tiles_per_group, tiles);
  uint32_t brow[NB];  // this lane's rows of B, in values; columns past N: dropped below
#pragma unroll
  for (int j = 0; j < NB; ++j) brow[j] = (uint32_t)min(n0 + 16 * j + lr, p.N - 1) * (uint32_t)p.r;
  uint32_t rank[RS];  // this lane's 8 ranks of step s; past r: the first ones, made 0
#pragma unroll
  for (int s = 0; s < RS; ++s) rank[s] = 32 * s + 8 * g < p.r ? 32 * s + 8 * g : 0;
  const int tr = lane / kLanes, nc = n0 + 8 * (lane % kLanes);  // base and out: this lane's token and columns
  const bool in = nc < p.N;  // N is a multiple of 8: a word is all in or all out
  float *mine = s_out[wave];

  u32x4_t base[2][kPasses];  // of this tile and the next
  auto load_base = [&](int64_t tile, u32x4_t (&to)[kPasses]) {
#pragma unroll
    for (int w = 0; w < kPasses; ++w) {
      const int64_t t = tile * 16 + tr + 64 / kLanes * w;
      to[w] = u32x4_t{0, 0, 0, 0};
      if (p.base && in && t < p.T) {
        const auto *b = reinterpret_cast<const u32x4_t *>(reinterpret_cast<const one *>(p.base) + t * p.ldb + nc);
        // many tokens: base and out pass once and would push h and B out of the caches
        to[w] = OPERANDS ? __builtin_nontemporal_load(b) : *b;
      }
    }
  };
  int l, ex = 0;
  vec hi[RS], lo[RS];
  auto load_h = [&](int64_t tile) {
    l = token_adapter(p, tile * 16 + lr);
    if constexpr (OPERANDS) {
      const vec *o = reinterpret_cast<const vec *>(p.ops) + tile * (RS * 2 * 64) + lane;
#pragma unroll
      for (int s = 0; s < RS; ++s) {
        hi[s] = o[(2 * s) * 64];
        lo[s] = o[(2 * s + 1) * 64];
      }
      if constexpr (DT == 1)
        ex = (reinterpret_cast<const int *>(reinterpret_cast<const vec *>(p.ops) + tiles * (RS * 2 * 64)))[tile * 16 + lr];
    }
  };
  // The parts' sums, by the whole workgroup: 16 tokens of r16 ranks stand one behind another in
  // each part. What a token without an adapter has there is dropped.
  auto sum_parts = [&](int64_t tile, float *to) {
    const int r4 = round16(p.r) / 4, quads = (int)min((int64_t)16, p.T - tile * 16) * r4;
    const f32x4 *q = reinterpret_cast<const f32x4 *>(p.part) + tile * 16 * r4;
    const int64_t part = p.T * r4;
    for (int i = threadIdx.x; i < quads; i += kUpWaves * 64) {
      f32x4 w[kParts];
#pragma unroll
      for (int k = 0; k < kParts; ++k)
        if (k < p.splits) w[k] = q[k * part + i];
      f32x4 h = w[0];
#pragma unroll
      for (int k = 1; k < kParts; ++k)
        if (k < p.splits) h += w[k];
      *reinterpret_cast<f32x4 *>(to + i / r4 * kHRow + i % r4 * 4) = h;
    }
  };

  u32x4_t bv[D][NB][RS];
  int held = -1;  // the adapter in bv[0]
  auto load_b = [&](const int (&a)[D]) {
#pragma unroll
    for (int k = 0; k < D; ++k) {
      if (a[k] < 0 || (k == 0 && a[0] == held)) continue;
      const uint16_t *bm = reinterpret_cast<const uint16_t *>(p.B) + (int64_t)a[k] * p.N * p.r;
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int s = 0; s < RS; ++s) bv[k][j][s] = *reinterpret_cast<const u32x4_t *>(bm + brow[j] + rank[s]);
    }
    held = a[0];
  };
  const bool ragged = p.r < 32 * RS;  // ranks past r: 0 on both sides
  load_h(tile);
  load_base(tile, base[0]);
  for (int turn = 0; tile < last; ++tile, turn ^= 1) {
    // the first adapters' B before anything that waits
    unsigned long long left = __ballot(l >= 0) & 0xFFFFull;
    const bool any = left != 0;
    int a[D];
#pragma unroll
    for (int k = 0; k < D; ++k) a[k] = next_adapter(left, l);
    if (any) load_b(a);
    if (tile + 1 < last) load_base(tile + 1, base[1]);
    if constexpr (!OPERANDS) {
      sum_parts(tile, s_h[turn]);
      const float sc = l >= 0 && p.scaling ? p.scaling[l] : 1.0f;
      lds_barrier();  // two buffers in turn: one barrier per tile
      float h[RS][8];
#pragma unroll
      for (int s = 0; s < RS; ++s) {
        const f32x4 *q = reinterpret_cast<const f32x4 *>(s_h[turn] + lr * kHRow + rank[s]);
        const f32x4 v[2] = {q[0], q[1]};
#pragma unroll
        for (int e = 0; e < 8; ++e) h[s][e] = l >= 0 && 32 * s + 8 * g < p.r ? __fmul_rn(v[e / 4][e % 4], sc) : 0.f;
      }
      ex = two_terms<DT, RS>(h, hi, lo);
    }
    f32x4 d[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) d[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    while (any) {
#pragma unroll
      for (int k = 0; k < D; ++k) {
        if (a[k] < 0) continue;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < RS; ++s) {
            u32x4_t b = bv[k][j][s];
            if (ragged) b = 32 * s + 8 * g < p.r ? b : u32x4_t{0, 0, 0, 0};
            acc = Half<DT>::mma(__builtin_bit_cast(vec, b), lo[s], acc);
            acc = Half<DT>::mma(__builtin_bit_cast(vec, b), hi[s], acc);
          }
          if (l == a[k]) d[j] = acc;
        }
      }
      if (!left) break;
#pragma unroll
      for (int k = 0; k < D; ++k) a[k] = next_adapter(left, l);
      load_b(a);
    }
    // a row's adapter for the lanes that write it; then the next tile's h into the registers
    int lt[kPasses];
#pragma unroll
    for (int w = 0; w < kPasses; ++w) lt[w] = __shfl(l, tr + 64 / kLanes * w, 64);
    // lane: columns 16 j + 4 g + 0..3 of token lr; the wave's own rows, in its program order
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      if constexpr (DT == 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[j][e] = __builtin_ldexpf(d[j][e], -ex);
      *reinterpret_cast<f32x4 *>(mine + lr * kRow + 16 * j + 4 * g) = d[j];
    }
    if (tile + 1 < last) load_h(tile + 1);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int w = 0; w < kPasses; ++w) {
      const int row = tr + 64 / kLanes * w;
      const int64_t t = tile * 16 + row;
      u32x4_t o = base[0][w];
      if (lt[w] >= 0) {
        const f32x4 *q = reinterpret_cast<const f32x4 *>(mine + row * kRow + 8 * (lane % kLanes));
        const f32x4 add[2] = {q[0], q[1]};
        const one *b = reinterpret_cast<const one *>(&base[0][w]);
        one v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = Half<DT>::round(__fadd_rn((float)b[e], add[e / 4][e % 4]));
        o = *reinterpret_cast<const u32x4_t *>(v);
      }
      if (in && t < p.T) {
        auto *to = reinterpret_cast<u32x4_t *>(reinterpret_cast<one *>(p.out) + t * p.ldo + nc);
        if constexpr (OPERANDS) __builtin_nontemporal_store(o, to);
        else *to = o;
      }
      base[0][w] = base[1][w];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

constexpr int kFewWaves = 8, kFewRing = 16 * 1024, kFewCols = 16 * kFewWaves;

// Up to 16 tokens in one kernel: every workgroup forms the whole of h for itself (its waves split
// K) and takes 16 columns a wave of the second product. A is read by all of them, from the caches;
// what it saves is the second kernel's launch and the parts' way through memory.
template <int DT, int RB>
__global__ __launch_bounds__(kFewWaves * 64) void kq_adapter_few_kernel(const AdapterArgs p) {
  typedef typename Half<DT>::vec vec;
  typedef typename Half<DT>::one one;
  constexpr int RS = (RB + 1) / 2, kRow = 32 * RS + 4;
  typedef one one4 __attribute__((ext_vector_type(4)));
  __shared__ __align__(16) unsigned char s_mem[kFewWaves * kFewRing];
  __shared__ __align__(16) float s_h[16 * kRow];
  f32x4 *s_acc = reinterpret_cast<f32x4 *>(s_mem);  // [kFewWaves][RB][64], behind the rings' use
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, lr = lane & 15;
  const int n0 = (int)(blockIdx.x * kFewWaves + wave) * 16;
  const int l = token_adapter(p, lr);
  // lane: columns c .. c+3 of token lr; its row of B; the ranks of its operands
  const int c = n0 + 4 * g;
  const bool live = c < p.N && lr < p.T;  // N is a multiple of 8
  const uint32_t brow = (uint32_t)min(n0 + lr, p.N - 1) * (uint32_t)p.r;
  uint32_t rank[RS];
#pragma unroll
  for (int s = 0; s < RS; ++s) rank[s] = 32 * s + 8 * g < p.r ? 32 * s + 8 * g : 0;
  auto load_b = [&](int a, u32x4_t (&b)[RS]) {
    const uint16_t *bm = reinterpret_cast<const uint16_t *>(p.B) + (int64_t)a * p.N * p.r;
#pragma unroll
    for (int s = 0; s < RS; ++s) b[s] = *reinterpret_cast<const u32x4_t *>(bm + brow + rank[s]);
  };
  const unsigned long long all = __ballot(l >= 0) & 0xFFFFull;
  one4 base = {};
  if (live && p.base) base = *reinterpret_cast<const one4 *>(reinterpret_cast<const one *>(p.base) + lr * p.ldb + c);
  const float sc = l >= 0 && p.scaling ? p.scaling[l] : 1.0f;
  u32x4_t b[RS] = {};
  unsigned long long left = all;
  int a = next_adapter(left, l);
  if (a >= 0) load_b(a, b);  // on its way while h is formed
  for (int now = a; now >= 0; now = next_adapter(left, l)) {
    f32x4 acc[1][RB][1];
    down_product<DT, RB, 1, kFewWaves, 1, kFewRing>(p, 0, &now, wave, (p.K + kStep - 1) / kStep,
                                                    s_mem + wave * kFewRing, acc);
    lds_barrier();  // the rings are read
#pragma unroll
    for (int i = 0; i < RB; ++i) s_acc[(wave * RB + i) * 64 + lane] = acc[0][i][0];
    lds_barrier();
    if (wave < RB) {
      f32x4 v = s_acc[wave * 64 + lane];
#pragma unroll
      for (int w = 1; w < kFewWaves; ++w) v += s_acc[(w * RB + wave) * 64 + lane];
      if (l == now) *reinterpret_cast<f32x4 *>(s_h + lr * kRow + 16 * wave + 4 * g) = v;
    }
    lds_barrier();  // before the rings are written again, and h is read
  }
  float h[RS][8];
#pragma unroll
  for (int s = 0; s < RS; ++s) {
    const f32x4 *q = reinterpret_cast<const f32x4 *>(s_h + lr * kRow + rank[s]);
    const f32x4 v[2] = {q[0], q[1]};
#pragma unroll
    for (int e = 0; e < 8; ++e) h[s][e] = l >= 0 && 32 * s + 8 * g < p.r ? __fmul_rn(v[e / 4][e % 4], sc) : 0.f;
  }
  vec hi[RS], lo[RS];
  const int ex = two_terms<DT, RS>(h, hi, lo);
  f32x4 d = {0.f, 0.f, 0.f, 0.f};
  left = all;
  for (int now = next_adapter(left, l); now >= 0; now = next_adapter(left, l)) {
    if (now != a) load_b(now, b);
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < RS; ++s) {
      const u32x4_t w = 32 * s + 8 * g < p.r ? b[s] : u32x4_t{0, 0, 0, 0};
      acc = Half<DT>::mma(__builtin_bit_cast(vec, w), lo[s], acc);
      acc = Half<DT>::mma(__builtin_bit_cast(vec, w), hi[s], acc);
    }
    if (l == now) d = acc;
  }
  if (!live) return;
  one4 o = base;
  if (l >= 0) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = Half<DT>::round(__fadd_rn((float)base[e], DT == 1 ? __builtin_ldexpf(d[e], -ex) : d[e]));
  }
  *reinterpret_cast<one4 *>(reinterpret_cast<one *>(p.out) + lr * p.ldo + c) = o;
}

// Parts of K: enough workgroups to fill the card where tokens are few, a step a wave at least,
// and no more parts than the second kernel adds up at ease.
int split_count(int64_t T, int64_t K) {
  if (T >= kWide) return 1;
  const int64_t tiles = (T + 15) / 16, steps = (K + kStep - 1) / kStep;
  int64_t s = 512 / tiles;
  if (s > steps / 4) s = steps / 4;
  return (int)(s < 1 ? 1 : s > kParts ? kParts : s);
}

// Whether the one kernel of few tokens is used: a single adapter of up to 2^17 values of A or up to
// 4 of 2^16 together, and a compute unit for every workgroup. Measured in graphs, this kernel against the two (us; where
// the host's launches are the bound, one launch saves 3.4 more):
//   1 token: K 1024, N 1024, r 8 3.5, 6.1; K 4096, N 4096, r 16 5.2, 6.5, r 32 5.8, 6.6; N 32768,
//   r 16 5.4, 6.5; K 8192, N 8192, r 16 7.3, 6.9; but K 14336, r 32 14.1, 7.9;
//   4 tokens on 4 adapters: K 1024, r 8 5.6, 7.3; but K 4096, r 16 10.2, 7.7;
//   16 tokens: 2 adapters, K 1024, r 8 4.9, 7.2; but K 4096, r 16 8.3, 7.7; 14 adapters, K 1024,
//   r 8 20.0, 11.7.
bool few(const AdapterArgs &a) {
  const int64_t most = a.T < a.L ? a.T : a.L;
  return a.T <= 16 && most <= 4 && most * a.r * a.K <= (most == 1 ? 1 << 17 : 1 << 16) && a.N <= 256 * kFewCols;
}

// The first kernel's waves and each one's ring of LDS: three steps of a single adapter's rows
// where 32 tokens go at once, two of several adapters' where 16 do (two workgroups then share a
// compute unit's 160 KiB up to 64 ranks)
template <int RB>
struct Down {
  static constexpr int kWideWaves = RB == 1 ? 8 : RB <= 8 ? 4 : 2;
  static constexpr int kWideD = RB <= 4 ? 2 : 1;  // a tile where two prompts meet has two
  static constexpr int kWideRing = 2 * (4 + kWideD * 2 * RB) * 1024;
  static constexpr int kD = RB == 1 ? 4 : RB == 2 ? 2 : 1;
  static constexpr int kWaves = RB <= 8 ? 4 : 2;
  static constexpr int kRing = 2 * (2 + kD * 2 * RB) * 1024;
};

template <int DT, int RS, int NB, int D, bool OPERANDS>
hipError_t launch_up(AdapterArgs a, hipStream_t s) {
  constexpr int kCols = 16 * NB * kUpWaves;
  const int64_t t16 = (a.T + 15) / 16, cols = (a.N + kCols - 1) / kCols;
  // some 4096 workgroups, each over a run of tiles whose adapter's B it keeps (8192 tokens, N
  // 14336, r 64: 151 us for both kernels; one round of 1024 workgroups 170, 8192 workgroups 164)
  int64_t run = t16 * cols / 4096;
  if (run < 1) run = 1;
  if (run > 64) run = 64;
  while ((t16 + run - 1) / run > 65535) run *= 2;  // the grid's second dimension
  a.tiles_per_group = (int)run;
  hipLaunchKernelGGL((kq_adapter_up_kernel<DT, RS, NB, D, OPERANDS>),
                     dim3((unsigned)cols, (unsigned)((t16 + run - 1) / run)), dim3(kUpWaves * 64), 0, s, a);
  return hipGetLastError();
}

template <int DT, int RB>
hipError_t launch(AdapterArgs a, hipStream_t s) {
  typedef Down<RB> C;
  constexpr int RS = (RB + 1) / 2;
  if (a.T >= kWide) {
    hipLaunchKernelGGL((kq_adapter_down_kernel<DT, RB, 2, C::kWideWaves, C::kWideD, C::kWideRing, true>),
                       dim3((unsigned)((a.T + 31) / 32)), dim3(C::kWideWaves * 64), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return launch_up<DT, RS, RS <= 2 ? 4 : 2, 1, true>(a, s);
  }
  if constexpr (RB <= 2) {
    if (few(a)) {
      hipLaunchKernelGGL((kq_adapter_few_kernel<DT, RB>), dim3((unsigned)((a.N + kFewCols - 1) / kFewCols)),
                         dim3(kFewWaves * 64), 0, s, a);
      return hipGetLastError();
    }
  }
  // a decode batch's tile may have 16 adapters: workgroups share them out, up to some 1024
  const int64_t t16 = (a.T + 15) / 16;
  const int64_t most = (a.T < 16 ? a.T + C::kD - 1 : 16) / C::kD, room = 1024 / (t16 * a.splits);
  const unsigned groups = (unsigned)(room < 1 ? 1 : room < most ? room : most);
  hipLaunchKernelGGL((kq_adapter_down_kernel<DT, RB, 1, C::kWaves, C::kD, C::kRing, false>),
                     dim3((unsigned)t16, (unsigned)a.splits, groups), dim3(C::kWaves * 64), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  constexpr int D = RB <= 2 ? 4 : RB <= 8 ? 2 : 1;
  if (a.T < kJoin) {
    // 32 columns a wave where 64 leave the card half empty (us in a graph, 32 and 64 columns: 128
    // tokens on 64 adapters, K = N = 4096, r 16 14.8, 16.6; 512 on 4 12.7, 13.1; but 256 on 64, N
    // 14336 33.0, 32.4)
    if (RS <= 2 && t16 * ((a.N + 255) / 256) <= 512) return launch_up<DT, RS, 2, D, false>(a, s);
    return launch_up<DT, RS, RS <= 2 ? 4 : 2, D, false>(a, s);
  }
  hipLaunchKernelGGL((kq_adapter_join_kernel<DT, RS>), dim3((unsigned)t16), dim3(64), 0, s, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_up<DT, RS, RS <= 2 ? 4 : 2, D, true>(a, s);
}

template <int DT>
hipError_t dispatch(const AdapterArgs &a, hipStream_t s) {
  if (a.r <= 16) return launch<DT, 1>(a, s);
  if (a.r <= 32) return launch<DT, 2>(a, s);
  if (a.r <= 64) return launch<DT, 4>(a, s);
  if (a.r <= 128) return launch<DT, 8>(a, s);
  return launch<DT, 16>(a, s);
}

constexpr int64_t kMax31 = 0x7FFFFFFF;

bool off(const void *p, size_t a) { return ((uintptr_t)p % a) != 0; }

int64_t part_bytes(int64_t T, int64_t K, int64_t r) {
  return T >= kWide ? 0 : (split_count(T, K) * T * ((r + 15) / 16 * 16) * 4 + 255) / 256 * 256;
}

int64_t workspace_bytes(int64_t T, int64_t K, int64_t r) {
  // operands: 32 ranks of two 2-byte terms, and a 4-byte exponent, per token of whole tiles
  const int64_t steps = r <= 32 ? 1 : r <= 64 ? 2 : r <= 128 ? 4 : 8, t16 = (T + 15) / 16 * 16;
  return part_bytes(T, K, r) + (T >= kJoin ? (t16 * (steps * 128 + 4) + 255) / 256 * 256 : 0);
}

kq_status check_sizes(int64_t T, int64_t K, int64_t r) {
  if (T < 0 || K < 1 || r < 1) return KQ_ERR_INVALID_ARG;
  if (K % 8 != 0 || r % 8 != 0 || K > kMaxDim || r > kMaxRank || T > kMaxTokens) return KQ_ERR_UNSUPPORTED;
  return KQ_OK;
}

}  // namespace

extern "C" kq_status kq_adapter_workspace_size(int64_t T, int64_t K, int64_t r, size_t *bytes) {
  if (!bytes) return KQ_ERR_INVALID_ARG;
  const kq_status st = check_sizes(T, K, r);
  if (st != KQ_OK) return st;
  *bytes = T == 0 ? 0 : (size_t)workspace_bytes(T, K, r);
  return KQ_OK;
}

static kq_status adapter_add_impl(const void *x, int64_t ldx, const void *A, const void *B,
                                  const int32_t *adapter, const float *scaling, const void *base,
                                  int64_t ldb, int64_t T, int64_t K, int64_t N, int64_t r, int64_t L,
                                  kq_dtype dtype, void *out, int64_t ldo, void *workspace,
                                  size_t ws_bytes, void *stream) {
  if (N < 0 || L < 1) return KQ_ERR_INVALID_ARG;
  if (dtype != KQ_BF16 && dtype != KQ_FP16) return KQ_ERR_INVALID_ARG;
  const kq_status st = check_sizes(T, K, r);
  if (st != KQ_OK) return st;
  if (N % 8 != 0 || N > kMaxDim || L > kMax31) return KQ_ERR_UNSUPPORTED;
  if (T == 0 || N == 0) return KQ_OK;
  if (!x || !A || !B || !adapter || !out) return KQ_ERR_INVALID_ARG;
  if (ldx < K || (base && ldb < N) || ldo < N) return KQ_ERR_INVALID_ARG;
  // 32 rows of x within 32 bits of byte offset
  if (ldx > (1 << 25) || (base && ldb > kMax31) || ldo > kMax31) return KQ_ERR_UNSUPPORTED;
  if (off(x, 16) || off(A, 16) || off(B, 16) || off(base, 16) || off(out, 16) || ldx % 8 != 0 ||
      (base && ldb % 8 != 0) || ldo % 8 != 0 || off(adapter, 4) || off(scaling, 4))
    return KQ_ERR_ALIGNMENT;
  const kq_span o = kq_rows_span(out, T, ldo, N, 2), b = kq_rows_span(base, T, ldb, N, 2);
  const kq_span in[5] = {kq_rows_span(x, T, ldx, K, 2), kq_rows_span(A, 1, L * r * K, L * r * K, 2),
                         kq_rows_span(B, 1, L * N * r, L * N * r, 2), kq_rows_span(adapter, 1, T, T, 4),
                         kq_rows_span(scaling, 1, L, L, 4)};
  for (const kq_span &i : in)
    if (kq_overlap(o, i)) return KQ_ERR_INVALID_ARG;
  if (kq_overlap(o, b) && !(out == base && ldo == ldb)) return KQ_ERR_INVALID_ARG;
  const int64_t need = workspace_bytes(T, K, r);
  if (!workspace || ws_bytes < (size_t)need) return KQ_ERR_WORKSPACE;
  if (off(workspace, 256)) return KQ_ERR_ALIGNMENT;
  const kq_span ws = kq_rows_span(workspace, 1, need, need, 1);
  for (const kq_span &i : in)
    if (kq_overlap(ws, i)) return KQ_ERR_INVALID_ARG;
  if (kq_overlap(ws, o) || kq_overlap(ws, b)) return KQ_ERR_INVALID_ARG;
  const int splits = split_count(T, K), steps = (int)((K + kStep - 1) / kStep);
  const AdapterArgs a = {x, A, B, base, adapter, scaling, out, static_cast<float *>(workspace),
                         static_cast<char *>(workspace) + part_bytes(T, K, r), ldx, ldb, ldo, T, (int)K,
                         (int)N, (int)r, (int)L, splits, (steps + splits - 1) / splits, 1};
  hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = dtype == KQ_BF16 ? dispatch<0>(a, s) : dispatch<1>(a, s);
  return e == hipSuccess ? KQ_OK : KQ_ERR_HIP;
}

extern "C" kq_status kq_adapter_add(const void *x, int64_t ldx, const void *A, const void *B,
                                    const int32_t *adapter, const float *scaling, const void *base,
                                    int64_t ldb, int64_t T, int64_t K, int64_t N, int64_t r, int64_t L,
                                    kq_dtype dtype, void *out, int64_t ldo, void *workspace,
                                    size_t workspace_bytes, void *stream) {
  const kq_status st = adapter_add_impl(x, ldx, A, B, adapter, scaling, base, ldb, T, K, N, r, L, dtype,
                                        out, ldo, workspace, workspace_bytes, stream);
  if (kq_log_on())
    kq_logf("adapter_add T=%lld K=%lld N=%lld r=%lld L=%lld: %s", (long long)T, (long long)K,
            (long long)N, (long long)r, (long long)L, kq_status_string(st));
  return st;
}

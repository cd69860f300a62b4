// kq_grouped.hip -- products of INT4 or INT8 codes grouped by expert, with ragged sizes, on
// the gfx950 int8 matrix cores.
//
//   out[i][j] = cvt( fp32( fp32( fp32(acc) * sx[t] ) * sw[e][j] ) ),  t = rows[i],
//   acc = sum_k qx[t][k] * qw[e][j][k]   (exact, int32), e the group of row i.
//
// The groups' ends are read on the device (nothing waits for the host): a workgroup finds the
// group and the row tile of its number by a scan of the groups' tile counts. The grid holds
// one tile per TILE rows and one more per group, which is as many as ragged ends can make;
// the workgroups behind the last tile end at once.
//
// Few rows per group: bound by the weights' stream (64 experts of 4096 x 7168 INT4, 4 to 16 rows
// each: 162-166 us, 5.7-5.8 TB/s). Many: by the matrix cores and what feeds them (16384 rows, 8
// experts, N 14336, K 4096: INT4 815-830 us, 2.3-2.36 POP/s; INT8 996-1010 us, 1.9 POP/s; the
// library's dense INT8 product of that size 848 us). INT4 spends 2.3 instructions a product on
// unpacking; INT8 reads twice the bytes from LDS, whose writes and reads take as long as its
// products.
#include "kq_internal.h"
#include "kq_device.h"
#include "kq_linear.h"

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

struct GroupedArgs {
  const uint8_t *xq, *wq;
  const void *sx, *sw;
  const int32_t *rows, *offsets;
  void *out;
  int64_t ldxq, ldwq, ldwe, T, R, N, ldo;
  int pieces;  // 16-byte pieces of a row of codes
  int E, scale_fp16, out_dtype;
};

struct RowTile {
  int e;          // expert; -1: no tile of this number
  int64_t begin;  // first row of the tile
  int count;      // rows, 1 .. TILE
};

// Tile `want` of the groups cut into tiles of TILE rows: the wave's lanes take 64 groups at a
// time, scan their tile counts, and the lane whose range holds `want` answers. Wave-uniform.
template <int TILE>
__device__ __forceinline__ RowTile find_tile(const int32_t *offsets, int E, int64_t R, int want) {
  const int lane = threadIdx.x & 63;
  const int last = (int)(R < 0x7FFFFFFF ? R : 0x7FFFFFFF);
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    int b = 0, n = 0;
    if (e < E) {
      b = min(max(offsets[e], 0), last);
      n = max(min(max(offsets[e + 1], 0), last) - b, 0);
    }
    const int tiles = n / TILE + (n % TILE ? 1 : 0);
    int sum = tiles;  // tiles up to and with this lane's group
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(sum, o, 64);
      if (lane >= o) sum += v;
    }
    const unsigned long long after = __ballot(sum > want);
    if (after) {
      const int l = __builtin_ctzll(after);
      const int k = want - __shfl(sum - tiles, l, 64);
      const int first = __shfl(b, l, 64), rows = __shfl(n, l, 64);
      return {__builtin_amdgcn_readfirstlane(e0 + l),
              (int64_t)__builtin_amdgcn_readfirstlane(first) + (int64_t)__builtin_amdgcn_readfirstlane(k) * TILE,
              __builtin_amdgcn_readfirstlane(min(rows - k * TILE, TILE))};
    }
    want -= __shfl(sum, 63, 64);
  }
  return {-1, 0, 0};
}

__device__ __forceinline__ float load_step(const void *p, int64_t i, int fp16) {
  return fp16 ? (float)reinterpret_cast<const _Float16 *>(p)[i] : reinterpret_cast<const float *>(p)[i];
}

__device__ __forceinline__ void store_out(void *out, int64_t i, float v, int dtype) {
  if (dtype == KQ_FP32) reinterpret_cast<float *>(out)[i] = v;
  else if (dtype == KQ_BF16) reinterpret_cast<__bf16 *>(out)[i] = (__bf16)v;
  else reinterpret_cast<_Float16 *>(out)[i] = half_rne(v);
}

// 4 consecutive outputs of a row, of which the first `left` exist; any alignment of the
// output type (global memory takes a vector access at any address)
template <int OUT>
__device__ __forceinline__ void store_out4(void *out, int64_t i, const float (&v)[4], int64_t left) {
  typedef u32x4_t any16 __attribute__((aligned(4)));
  typedef u32x2_t any8 __attribute__((aligned(2)));
  if (left >= 4) {
    if constexpr (OUT == KQ_FP32) {
      *reinterpret_cast<any16 *>(reinterpret_cast<float *>(out) + i) =
          u32x4_t{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    } else if constexpr (OUT == KQ_BF16) {
      const __bf16 h[4] = {(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
      *reinterpret_cast<any8 *>(reinterpret_cast<__bf16 *>(out) + i) = __builtin_bit_cast(u32x2_t, h);
    } else {
      const _Float16 h[4] = {half_rne(v[0]), half_rne(v[1]), half_rne(v[2]), half_rne(v[3])};
      *reinterpret_cast<any8 *>(reinterpret_cast<_Float16 *>(out) + i) = __builtin_bit_cast(u32x2_t, h);
    }
  } else {
#pragma unroll
    for (int r = 0; r < 3; ++r)
      if (r < left) store_out(out, i + r, v[r], OUT);
  }
}

// 16 bytes of finished outputs, of which the first `left` values exist, to out[i]
template <int OUT>
__device__ __forceinline__ void store_piece(void *out, int64_t i, const u32x4_t &v, int64_t left) {
  if constexpr (OUT == KQ_FP32) {
    typedef u32x4_t any __attribute__((aligned(4)));
    float *o = reinterpret_cast<float *>(out) + i;
    if (left >= 4) {
      *reinterpret_cast<any *>(o) = v;
    } else {
#pragma unroll
      for (int r = 0; r < 3; ++r)
        if (r < left) o[r] = __uint_as_float(v[r]);
    }
  } else {
    typedef u32x4_t any __attribute__((aligned(2)));
    uint16_t *o = reinterpret_cast<uint16_t *>(out) + i;
    if (left >= 8) {
      *reinterpret_cast<any *>(o) = v;
    } else {
#pragma unroll
      for (int r = 0; r < 7; ++r)
        if (r < left) o[r] = (uint16_t)(v[r / 2] >> (16 * (r % 2)));
    }
  }
}

// Steps of Q groups of 4 channels, group q from channel n + at(q) on, of a row of N steps that
// starts at `row`; channels past N get 0 (their outputs are not written).
template <int Q, typename At>
__device__ __forceinline__ void load_steps(const void *p, int64_t row, int64_t n, int64_t N, int fp16, At at,
                                           float (&v)[Q][4]) {
  typedef u32x4_t any16 __attribute__((aligned(4)));
  typedef u32x2_t any8 __attribute__((aligned(2)));
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int64_t c = n + at(q);
    if (c + 4 <= N) {
      if (fp16) {
        const u32x2_t w = *reinterpret_cast<const any8 *>(reinterpret_cast<const _Float16 *>(p) + row + c);
        const _Float16 *h = reinterpret_cast<const _Float16 *>(&w);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[q][r] = (float)h[r];
      } else {
        const u32x4_t w = *reinterpret_cast<const any16 *>(reinterpret_cast<const float *>(p) + row + c);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[q][r] = __uint_as_float(w[r]);
      }
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) v[q][r] = c + r < N ? load_step(p, row + c + r, fp16) : 0.f;
    }
  }
}

// INT4: a code moved into the high nibble of a byte is the int8 value 16 q, so one dword of 8
// codes becomes two operand dwords (even codes, odd codes) by a shift and two masks, the
// products carry 256 q q' and the sum is shifted back by 8 (exact: |sum| < 2^31 for K <= 65536).
template <int BITS>
__device__ __forceinline__ void mfma_piece(const u32x4_t &a, const u32x4_t &b, i32x4 &acc) {
  if constexpr (BITS == 8) {
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a),
                                                __builtin_bit_cast(i32x4, b), acc, 0, 0, 0);
  } else {
    constexpr unsigned kHi = 0xF0F0F0F0u;
    const u32x4_t a0 = (a << 4) & kHi, a1 = a & kHi, b0 = (b << 4) & kHi, b1 = b & kHi;
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a0),
                                                __builtin_bit_cast(i32x4, b0), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a1),
                                                __builtin_bit_cast(i32x4, b1), acc, 0, 0, 0);
  }
}

// A workgroup: 16 MI output channels x 16 NI rows of one group; its waves split the reduction (U
// steps of 64 bytes of a row in turn) and add their parts up in LDS (integers: any order). Bound by
// the weights' stream: the operands come straight from memory, the weights of the next steps before
// the products of these, and as many waves as fit keep their loads going (8 of them a workgroup: 2
// rows of 4096 x 4096 INT8 8.7 us, 4 waves 10.3).
template <int BITS, int MI, int NI, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void kq_grouped_stream_kernel(const GroupedArgs p, int tiles_m) {
  constexpr int U = MI == 1 ? 2 : 1;
  __shared__ i32x4 s_acc[WAVES][MI * NI][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, lr = lane & 15;
  const RowTile tile = find_tile<16 * NI>(p.offsets, p.E, p.R, (int)(blockIdx.x / tiles_m));
  if (tile.e < 0) return;
  const int64_t n0 = (int64_t)(blockIdx.x % tiles_m) * (16 * MI);

  // rows past the end of the matrix, of the group or of the codes read a valid row instead;
  // their products are dropped
  const uint8_t *wrow[MI], *xrow[NI];
#pragma unroll
  for (int m = 0; m < MI; ++m) {
    const int64_t n = n0 + 16 * m + lr;
    wrow[m] = p.wq + tile.e * p.ldwe + (n < p.N ? n : p.N - 1) * p.ldwq + g * 16;
  }
  // a row's last step may have fewer than 4 pieces, and a wave's last steps may lie behind it
  auto in_row = [&](int s) { return s * 4 + g < p.pieces; };
  auto load_a = [&](int s0, u32x4_t (&a)[U][MI]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t o = in_row(s0 + u) ? (int64_t)(s0 + u) * 64 : -(int64_t)g * 16;
#pragma unroll
      for (int m = 0; m < MI; ++m) a[u][m] = *reinterpret_cast<const u32x4_t *>(wrow[m] + o);
    }
  };
  u32x4_t a[U][MI];
  load_a(wave * U, a);  // on their way before the rows' numbers are known
  int64_t src[NI];
#pragma unroll
  for (int j = 0; j < NI; ++j) {
    const int i = 16 * j + lr;
    int64_t t = -1;
    if (i < tile.count) t = p.rows ? (int64_t)p.rows[tile.begin + i] : tile.begin + i;
    src[j] = t >= 0 && t < p.T ? t : -1;
    xrow[j] = p.xq + (src[j] < 0 ? 0 : src[j]) * p.ldxq + g * 16;
  }
  i32x4 acc[MI][NI];
#pragma unroll
  for (int m = 0; m < MI; ++m)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[m][j] = i32x4{0, 0, 0, 0};
  const u32x4_t zero = {0, 0, 0, 0};
  for (int s0 = wave * U; s0 * 4 < p.pieces; s0 += WAVES * U) {
    u32x4_t b[U][NI], next[U][MI] = {};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t o = in_row(s0 + u) ? (int64_t)(s0 + u) * 64 : -(int64_t)g * 16;
#pragma unroll
      for (int j = 0; j < NI; ++j) b[u][j] = *reinterpret_cast<const u32x4_t *>(xrow[j] + o);
    }
    if ((s0 + WAVES * U) * 4 < p.pieces) load_a(s0 + WAVES * U, next);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int m = 0; m < MI; ++m) mfma_piece<BITS>(a[u][m], in_row(s0 + u) ? b[u][j] : zero, acc[m][j]);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < MI; ++m) a[u][m] = next[u][m];
  }
#pragma unroll
  for (int m = 0; m < MI; ++m)
#pragma unroll
    for (int j = 0; j < NI; ++j) s_acc[wave][m * NI + j][lane] = acc[m][j];
  __syncthreads();
  // lane: channels n0 + 16 m + 4 g + 0..3 of row 16 j + lr
#pragma unroll
  for (int m = 0; m < MI; ++m)
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      if ((m * NI + j) % WAVES != wave || src[j] < 0) continue;
      i32x4 v = s_acc[0][m * NI + j][lane];
#pragma unroll
      for (int k = 1; k < WAVES; ++k) v += s_acc[k][m * NI + j][lane];
      const float sx = load_step(p.sx, src[j], p.scale_fp16);
      const int64_t row = (tile.begin + 16 * j + lr) * p.ldo;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t n = n0 + 16 * m + 4 * g + r;
        if (n >= p.N) continue;
        const int sum = BITS == 8 ? v[r] : v[r] >> 8;
        const float sw = load_step(p.sw, tile.e * p.N + n, p.scale_fp16);
        store_out(p.out, row + n, __fmul_rn(__fmul_rn((float)sum, sx), sw), p.out_dtype);
      }
    }
}

// ---- the tile kernels: 256 output channels x up to 256 rows of one group, or 128 x 128 ----
constexpr int kStep = 128;  // bytes of every row per step of the reduction

typedef int i32x16 __attribute__((ext_vector_type(16)));

// 16 int8 operand bytes from one dword pair of INT4 codes (16 codes)
__device__ __forceinline__ i32x4 unpack16(unsigned x, unsigned y) {
  constexpr unsigned kHi = 0xF0F0F0F0u;
  return i32x4{(int)((x << 4) & kHi), (int)(x & kHi), (int)((y << 4) & kHi), (int)(y & kHi)};
}

// The tiles and the waves' shares of them: kMI blocks of kSide channels by kBlocks blocks of kSide
// rows per wave, INT4 on 16x16x64 instructions, INT8 on 32x32x32. A wave's blocks stand kApart
// rows apart, so with NU blocks each the waves cover the first NU kApart rows of the tile and a
// group's short last tile costs what it holds.
template <int BITS, int SIDE>
struct Share;
template <>
struct Share<4, 256> {
  static constexpr int kWM = 2, kWN = 4, kSide = 16;
  typedef i32x4 acc_t;
};
template <>
struct Share<8, 256> {
  static constexpr int kWM = 4, kWN = 2, kSide = 32;
  typedef i32x16 acc_t;
};
template <>
struct Share<4, 128> {
  static constexpr int kWM = 2, kWN = 2, kSide = 16;
  typedef i32x4 acc_t;
};
template <>
struct Share<8, 128> {
  static constexpr int kWM = 2, kWN = 2, kSide = 32;
  typedef i32x16 acc_t;
};
template <int BITS, int SIDE>
struct Tiling : Share<BITS, SIDE> {
  typedef Share<BITS, SIDE> S;
  static constexpr int kWaves = S::kWM * S::kWN;
  static constexpr int kMI = SIDE / S::kWM / S::kSide, kApart = S::kWN * S::kSide, kBlocks = SIDE / kApart;
  static constexpr int kOpBytes = SIDE * kStep;  // per operand and step in LDS
  static constexpr int kOutBytes = 2 * kApart * (SIDE * 4 + 16);  // two blocks of fp32 output rows
  // Weights come from memory, rows of x from the caches: an INT8 tile of 256 that is not full, and so
  // waits for its weights rather than for its products, has them a step further ahead than x (3062
  // rows over 16 experts, N 11008, K 4096 220 us, 229 without; full tiles are slower with it, 16384
  // rows over 8 experts, N 14336, K 4096 1030, 996, and so is INT4)
  static constexpr bool kFar = BITS == 8 && SIDE == 256;
  template <int STAGES>
  static constexpr int kInts = (2 * STAGES + (kFar ? 1 : 0)) * kOpBytes;
  template <int STAGES>
  static constexpr int kLds = kInts<STAGES> > kOutBytes + SIDE ? kInts<STAGES> : kOutBytes + SIDE;
  static constexpr int kLoads = kOpBytes / 1024 / kWaves;
  static_assert(kLoads * 1024 * kWaves == kOpBytes, "the tile splits evenly over the waves");
};

// Wait until a step's operands have landed, `left` steps before the last one, where the loads of up
// to MOST pairs (x of a step, W of the step MORE behind it) may still be on their way behind them:
// those pairs' and, with MORE, the weights that came with the step's own x.
template <int W, int X, int MORE, int MOST>
__device__ __forceinline__ void wait_pairs(int left) {
  static_assert(MORE * W + (W + X) * MOST < 64, "fits the wait counter");
  static_assert(MORE <= 1, "the weights one step ahead of x, or none");
  if (left >= MOST + MORE) {
    wait_and_fence<wait_vm_imm(MORE * W + (W + X) * MOST)>();
  } else if constexpr (MOST == 0) {
    wait_and_fence<kWaitVm0>();
  } else if (MORE && left == MOST) {  // the last pair has no weights
    wait_and_fence<wait_vm_imm((W + X) * MOST)>();
  } else {
    wait_pairs<W, X, MORE, MOST - 1>(left);
  }
}

template <int BITS, int SIDE, int STAGES, int OUT, int NU>
__device__ __forceinline__ void tile_product(const GroupedArgs &p, const RowTile &tile, int64_t n0,
                                             unsigned char *s_buf) {
  typedef Tiling<BITS, SIDE> S;
  typedef typename S::acc_t acc_t;
  constexpr int kOpBytes = S::kOpBytes, kLoads = S::kLoads, kXLoads = kLoads * NU / S::kBlocks;
  constexpr int kRegs = sizeof(acc_t) / 4;
  constexpr int kChunks = kStep / 16, kRowsPer = 1024 / kStep;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane / S::kSide, lr = lane % S::kSide;
  const int wm = wave % S::kWM, wn = wave / S::kWM;
  constexpr int kMore = S::kFar && NU < S::kBlocks ? 1 : 0, kWStages = STAGES + kMore;
  auto w_place = [&](int b) { return s_buf + b * kOpBytes; };
  auto x_place = [&](int b) { return s_buf + (kWStages + b) * kOpBytes; };
  auto plus = [](int b, int n, int places) { return b + n < places ? b + n : b + n - places; };

  // DMA: instruction J = wave kLoads + j of an operand fills kRowsPer tile rows; a lane lands
  // at position lane % kChunks of row R and reads piece (lane % kChunks) ^ swz(R) of that row,
  // so that the rows of one fragment read spread over all banks. Rows past the end of the
  // weight or of the group read a valid row; their products are dropped.
  auto swz = [](int R) { return (R >> 1) & 7; };
  auto row_of = [&](int loads, int j) { return (wave * loads + j) * kRowsPer + lane / kChunks; };
  auto piece_of = [&](int loads, int j) { return (lane % kChunks) ^ swz(row_of(loads, j)); };
  const uint8_t *wbase = uniform(p.wq + tile.e * p.ldwe + n0 * p.ldwq);
  uint32_t vw[kLoads];  // 256 rows of at most 16 MiB (checked on the host): 32 bits
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int R = row_of(kLoads, j);
    const int64_t n = n0 + R < p.N ? R : p.N - 1 - n0;
    vw[j] = (uint32_t)(n * p.ldwq + piece_of(kLoads, j) * 16);
  }
  const uint8_t *ax[kXLoads];  // of the NU blocks' rows
#pragma unroll
  for (int j = 0; j < kXLoads; ++j) {
    const int R = row_of(kXLoads, j);
    int64_t t = tile.begin + (R < tile.count ? R : 0);
    if (p.rows) t = p.rows[t];
    if (t < 0 || t >= p.T) t = 0;
    ax[j] = p.xq + t * p.ldxq + piece_of(kXLoads, j) * 16;
  }
  const int steps = (p.pieces + kChunks - 1) / kChunks;
  // One load of step s, whole (inside the row for all lanes), or ending in it: the rest comes from a
  // block of zeros. Steps come in order, and x's addresses move along.
  auto load_w = [&](int s, int b, int j, bool whole) {
    unsigned char *to = w_place(b) + (wave * kLoads + j) * 1024;
    const uint8_t *w = wbase + (int64_t)s * kStep;
    if (whole) dma16<false>(w, vw[j], lds_addr(to));
    else dma16_addr<false>(s * kChunks + piece_of(kLoads, j) < p.pieces ? w + vw[j] : kZeros, lds_addr(to));
  };
  auto load_x = [&](int s, int b, int j, bool whole) {
    unsigned char *to = x_place(b) + (wave * kXLoads + j) * 1024;
    dma16_addr<false>(whole || s * kChunks + piece_of(kXLoads, j) < p.pieces ? ax[j] : kZeros, lds_addr(to));
    ax[j] += kStep;
  };
  // x of step s and the weights of step s + kMore; the weights that are further ahead go last, so
  // that a wait for x leaves them on their way
  auto load_pair = [&](int s, int bx, int bw) {
    if ((s + kMore + 1) * kChunks <= p.pieces) {
      if constexpr (kMore == 0) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
          load_w(s, bw, j, true);
          if (j < kXLoads) load_x(s, bx, j, true);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kXLoads; ++j) load_x(s, bx, j, true);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) load_w(s + kMore, bw, j, true);
      }
    } else {
      if (s < steps)
#pragma unroll
        for (int j = 0; j < kXLoads; ++j) load_x(s, bx, j, false);
      if (s + kMore < steps)
#pragma unroll
        for (int j = 0; j < kLoads; ++j) load_w(s + kMore, bw, j, false);
    }
  };
  auto load_first = [&]() {  // the weights of the steps that no pair has
    if constexpr (kMore == 1)
#pragma unroll
      for (int j = 0; j < kLoads; ++j) load_w(0, 0, j, kChunks <= p.pieces);
  };

  acc_t acc[S::kMI][NU];
#pragma unroll
  for (int m = 0; m < S::kMI; ++m)
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int r = 0; r < kRegs; ++r) acc[m][i][r] = 0;

  // rows of this lane's fragments: swz is swz(lr) for all of them
  const int sl = swz(lr);
  const int row_w = wm * (SIDE / S::kWM) + lr, row_x = wn * S::kSide + lr;
  // The steps of this lane's rows, and which of them are written: loaded here, so that the
  // epilogue does not wait for them (a row's number, then its step) row by row.
  float sx[NU];
  bool written[NU];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int R = row_x + i * S::kApart;
    int64_t t = tile.begin + (R < tile.count ? R : 0);
    if (p.rows) t = p.rows[t];
    const bool in = t >= 0 && t < p.T;
    sx[i] = load_step(p.sx, in ? t : 0, p.scale_fp16);
    written[i] = R < tile.count && in;
  }

  // A step's fragments come in kParts parts, each read while the part before it multiplies;
  // the first part of the next step is read before the last one of this step multiplies.
  constexpr int kParts = kStep / (1024 / S::kSide);
  struct Part {
    u32x4_t w[S::kMI], x[NU];
  };
  auto read_part = [&](int bw, int bx, int q) {
    const unsigned char *w = w_place(bw), *x = x_place(bx);
    Part f;
    const int off = ((64 / S::kSide * q + g) ^ sl) * 16;
#pragma unroll
    for (int m = 0; m < S::kMI; ++m)
      f.w[m] = *reinterpret_cast<const u32x4_t *>(w + (row_w + m * S::kSide) * kStep + off);
#pragma unroll
    for (int i = 0; i < NU; ++i)
      f.x[i] = *reinterpret_cast<const u32x4_t *>(x + (row_x + i * S::kApart) * kStep + off);
    return f;
  };
  auto multiply = [&](const Part &f) {
    if constexpr (BITS == 4) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        i32x4 a[S::kMI], bx[NU];
#pragma unroll
        for (int m = 0; m < S::kMI; ++m)
          a[m] = h ? unpack16(f.w[m].z, f.w[m].w) : unpack16(f.w[m].x, f.w[m].y);
#pragma unroll
        for (int i = 0; i < NU; ++i)
          bx[i] = h ? unpack16(f.x[i].z, f.x[i].w) : unpack16(f.x[i].x, f.x[i].y);
#pragma unroll
        for (int m = 0; m < S::kMI; ++m)
#pragma unroll
          for (int i = 0; i < NU; ++i)
            acc[m][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[m], bx[i], acc[m][i], 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int m = 0; m < S::kMI; ++m)
#pragma unroll
        for (int i = 0; i < NU; ++i)
          acc[m][i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(
              __builtin_bit_cast(i32x4, f.w[m]), __builtin_bit_cast(i32x4, f.x[i]), acc[m][i], 0, 0, 0);
    }
  };
  auto sync = [] {
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
  };
  if constexpr (BITS == 4) {
    // the unpacking between reads and products covers the reads; a second part in registers costs
    // more than it gives (256: it spills, 2042 against 841 us; 128: 67 against 63 us on R 8192,
    // N 512, K 8192)
    load_first();
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) load_pair(k, k, k + kMore);
    int bw = 0, bx = 0;  // this step's places
    for (int ks = 0; ks < steps; ++ks) {
      wait_pairs<kLoads, kXLoads, kMore, STAGES - 2>(steps - 1 - ks);
      sync();  // this step has landed for every wave, and every wave is done with the one before
      load_pair(ks + STAGES - 1, plus(bx, STAGES - 1, STAGES), plus(bw, kWStages - 1, kWStages));
#pragma unroll
      for (int q = 0; q < kParts; ++q) multiply(read_part(bw, bx, q));
      wait_and_fence<kWaitLgkm0>();
      bw = plus(bw, 1, kWStages);
      bx = plus(bx, 1, STAGES);
    }
  } else {
    // each part is read while the one before it multiplies, across the steps
    load_first();
#pragma unroll
    for (int k = 0; k < STAGES; ++k) load_pair(k, k, k + kMore);
    wait_pairs<kLoads, kXLoads, kMore, STAGES - 1>(steps - 1);
    sync();
    Part f = read_part(0, 0, 0);
    int bw = 0, bx = 0;  // this step's places
    for (int ks = 0; ks < steps; ++ks) {
      const int w_after = plus(bw, 1, kWStages), x_after = plus(bx, 1, STAGES);
#pragma unroll
      for (int q = 0; q < kParts; ++q) {
        Part next = f;
        if (q + 1 < kParts) {
          next = read_part(bw, bx, q + 1);
        } else if (ks + 1 < steps) {
          // this wave's reads of this step have returned, and its loads of the next step have
          // landed; behind the barrier that holds for every wave, so this step's places may be
          // overwritten and the next ones read
          wait_and_fence<kWaitLgkm0>();
          wait_pairs<kLoads, kXLoads, kMore, STAGES - 2>(steps - 2 - ks);
          sync();
          next = read_part(w_after, x_after, 0);
          load_pair(ks + STAGES, bx, bw);
        }
        __builtin_amdgcn_sched_barrier(0);
        multiply(f);
        __builtin_amdgcn_sched_barrier(0);
        f = next;
      }
      bw = w_after;
      bx = x_after;
    }
  }

  // Epilogue, kApart rows at a time (block i of every wave): a lane holds one row's 4 consecutive
  // channels per group of 4 registers, 8 bytes of 16 or 32 different lines an instruction. Through
  // LDS a wave stores whole rows of the tile, 16 bytes a lane. Two places in turn, one barrier per
  // block.
  constexpr int kQ = S::kMI * kRegs / 4;  // groups of 4 channels
  constexpr int kSize = OUT == KQ_FP32 ? 4 : 2, kRowBytes = SIDE * kSize + 16;
  constexpr int kRowLanes = SIDE * kSize / 16, kAtOnce = 64 / kRowLanes, kPer = 16 / kSize;
  static_assert(2 * S::kApart * kRowBytes <= S::kOutBytes, "two places of rows");
  const int ml = wm * (SIDE / S::kWM) + 4 * g;  // this lane's channels: ml + group_at(q)
  auto group_at = [](int q) { return q / (kRegs / 4) * S::kSide + q % (kRegs / 4) * 4 * (64 / S::kSide); };
  float sw[kQ][4];
  load_steps<kQ>(p.sw, tile.e * p.N, n0 + ml, p.N, p.scale_fp16, group_at, sw);
  const int64_t nc = n0 + lane % kRowLanes * kPer;  // the channels this lane stores
  wait_and_fence<kWaitLgkm0>();
  sync();  // every wave has read the last step
  unsigned char *s_ok = s_buf + S::kOutBytes;  // which rows of the tile are written
#pragma unroll
  for (int i = 0; i < NU; ++i)
    if (wm == 0 && g == 0) s_ok[row_x + i * S::kApart] = written[i];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    unsigned char *rows = s_buf + (i & 1) * (S::kApart * kRowBytes);
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      float v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int a = acc[q / (kRegs / 4)][i][q % (kRegs / 4) * 4 + r];
        v[r] = __fmul_rn(__fmul_rn((float)(BITS == 8 ? a : a >> 8), sx[i]), sw[q][r]);
      }
      store_out4<OUT>(rows + row_x * kRowBytes, ml + group_at(q), v, 4);
    }
    wait_and_fence<kWaitLgkm0>();
    sync();
    const unsigned long long ok = __ballot(lane < S::kApart && s_ok[i * S::kApart + lane % S::kApart]);
#pragma unroll
    for (int k = 0; k < S::kApart / (kAtOnce * S::kWaves); ++k) {
      const int r = (k * S::kWaves + wave) * kAtOnce + lane / kRowLanes;
      if (ok >> r & 1)
        store_piece<OUT>(p.out, (tile.begin + i * S::kApart + r) * p.ldo + nc,
                         *reinterpret_cast<const u32x4_t *>(rows + r * kRowBytes + lane % kRowLanes * 16),
                         p.N - nc);
    }
  }
}

template <int BITS, int SIDE, int STAGES, int OUT>
__global__ __launch_bounds__((Tiling<BITS, SIDE>::kWaves * 64)) void kq_grouped_tile_kernel(const GroupedArgs p, int tiles_m) {
  typedef Tiling<BITS, SIDE> S;
  __shared__ __align__(16) unsigned char s_buf[S::template kLds<STAGES>];
  const RowTile tile = find_tile<SIDE>(p.offsets, p.E, p.R, (int)(blockIdx.x / tiles_m));
  if (tile.e < 0) return;
  const int64_t n0 = (int64_t)(blockIdx.x % tiles_m) * SIDE;
  if constexpr (S::kBlocks == 4) {
    if (tile.count > 3 * S::kApart) tile_product<BITS, SIDE, STAGES, OUT, 4>(p, tile, n0, s_buf);
    else if (tile.count > 2 * S::kApart) tile_product<BITS, SIDE, STAGES, OUT, 3>(p, tile, n0, s_buf);
    else if (tile.count > S::kApart) tile_product<BITS, SIDE, STAGES, OUT, 2>(p, tile, n0, s_buf);
    else tile_product<BITS, SIDE, STAGES, OUT, 1>(p, tile, n0, s_buf);
  } else {
    static_assert(S::kBlocks == 2, "blocks of a wave");
    if (tile.count > S::kApart) tile_product<BITS, SIDE, STAGES, OUT, 2>(p, tile, n0, s_buf);
    else tile_product<BITS, SIDE, STAGES, OUT, 1>(p, tile, n0, s_buf);
  }
}

template <int BITS, int MI, int NI>
kq_status launch_stream(const GroupedArgs &a, hipStream_t s) {
  constexpr int WAVES = 8;
  const int64_t tiles_m = (a.N + 16 * MI - 1) / (16 * MI);
  const int64_t tiles = a.R / (16 * NI) + (a.R < a.E ? a.R : a.E);
  if (tiles_m * tiles > 0x7FFFFFFF / (WAVES * 64)) return KQ_ERR_UNSUPPORTED;
  hipLaunchKernelGGL((kq_grouped_stream_kernel<BITS, MI, NI, WAVES>), dim3((unsigned)(tiles_m * tiles)),
                     dim3(WAVES * 64), 0, s, a, (int)tiles_m);
  return hipGetLastError() == hipSuccess ? KQ_OK : KQ_ERR_HIP;
}

// 16 channels a workgroup instead of 32 where many INT8 weights of one or two rows a group stream
// by, or where half a card has no workgroup (us, 16 against 32; weights from memory, and in brackets
// from the last cache, where reading x twice as often costs more):
//   8 rows over 8 experts of 4096 x 4096 INT8 29.7, 32.7 (18.8, 16.4); 2 rows of 14336 x 4096 INT8
//   26.3, 29.6; 6 of 2048 x 7168 INT8 21.5, 22.7 (17.6, 18.8); but 2 of 4096 x 4096 INT8 (256
//   workgroups of 32) 12.0, 10.8; 64 rows over 8 experts 33.6, 35.3 (34.0, 26.8); 8 over 8 INT4 19.2,
//   17.0;
//   32 rows over 4 experts, N 1024, INT8 7.8, 9.1 (8.8, 9.2), INT4 6.2, 7.0; but 2040 rows over 2, N
//   88, K 8576 INT4 (192 workgroups of 32) 13.6, 10.8.
template <int BITS, int NI>
kq_status launch_stream(const GroupedArgs &a, int64_t groups, int64_t per_group, hipStream_t s) {
  const int64_t tiles = (a.N + 31) / 32 * groups * ((per_group + 16 * NI - 1) / (16 * NI));
  if ((BITS == 8 && per_group <= 2 && tiles > 256) || tiles <= 128) return launch_stream<BITS, 1, NI>(a, s);
  return launch_stream<BITS, 2, NI>(a, s);
}

template <int BITS, int SIDE, int STAGES>
kq_status launch_tile(const GroupedArgs &a, hipStream_t s) {
  constexpr int kThreads = Tiling<BITS, SIDE>::kWaves * 64;
  const int64_t tiles_m = (a.N + SIDE - 1) / SIDE;
  const int64_t tiles = a.R / SIDE + (a.R < a.E ? a.R : a.E);
  if (tiles_m * tiles > 0x7FFFFFFF / kThreads) return KQ_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)(tiles_m * tiles)), block(kThreads);
  if (a.out_dtype == KQ_FP32)
    hipLaunchKernelGGL((kq_grouped_tile_kernel<BITS, SIDE, STAGES, KQ_FP32>), grid, block, 0, s, a, (int)tiles_m);
  else if (a.out_dtype == KQ_BF16)
    hipLaunchKernelGGL((kq_grouped_tile_kernel<BITS, SIDE, STAGES, KQ_BF16>), grid, block, 0, s, a, (int)tiles_m);
  else
    hipLaunchKernelGGL((kq_grouped_tile_kernel<BITS, SIDE, STAGES, KQ_FP16>), grid, block, 0, s, a, (int)tiles_m);
  return hipGetLastError() == hipSuccess ? KQ_OK : KQ_ERR_HIP;
}

// Which kernel, by the rows per group and the workgroups that each tile size would make (us; R
// rows, E groups):
//   the stream kernel, where 128 x 128 tiles are too few to keep the card's loads going and the
//   rows too few to ask for more than loads, or where such tiles are very few:
//     R 8, E 8, N 4096, K 4096 INT8 (256 tiles of 128): 16.5 against 24.6; R 64: 26.9, 32.5;
//     R 2040, E 2, N 88, K 8576 INT4 (17 tiles): 10.4 against 45;
//     but R 256, E 32, N 2048, K 7168 INT8 (544 tiles): 104 against 82; R 300, E 2, N 4096,
//     K 4096 INT8 (128 tiles, 150 rows a group): 43 against 34;
//   256 x 256 tiles, where the groups fill them and there are enough for the 256 compute units:
//     R 16384, E 8, N 14336, K 4096: INT4 858 against 911, INT8 1054 against 1254;
//     but R 8192, E 4, N 512, K 8192 INT8 (72 tiles of 256): 110 against 73; R 2048, E 64,
//     N 4096, K 7168 INT4 (32 rows a group): 222 against 182;
//   128 x 128 tiles otherwise; two workgroups of them share a compute unit. Up to 256 of them each
//   has one to itself, and four steps in LDS: R 128, E 4, N 4096, K 4096 INT8 22.3 against 35.3,
//   R 2000, E 8, N 1024, K 2048 16.3 against 17.4 (INT4 within 3 %); but R 8192, E 4, N 512,
//   K 8192 INT8 (272 tiles) 83 against 72.
template <int BITS>
kq_status launch(const GroupedArgs &a, hipStream_t s) {
  const int64_t groups = a.R < a.E ? a.R : a.E, per_group = a.R / groups;
  const int64_t tiles128 = (a.N + 127) / 128 * (a.R / 128 + groups);
  const int64_t tiles256 = (a.N + 255) / 256 * (a.R / 256 + groups);
  if (tiles128 < 64 || (tiles128 < 512 && per_group <= 16))
    return per_group <= 8 ? launch_stream<BITS, 1>(a, groups, per_group, s)
                          : launch_stream<BITS, 2>(a, groups, per_group, s);
  if (per_group >= 96 && tiles256 >= 192) return launch_tile<BITS, 256, 2>(a, s);
  return tiles128 <= 256 ? launch_tile<BITS, 128, 4>(a, s) : launch_tile<BITS, 128, 2>(a, s);
}

constexpr int64_t kMax31 = 0x7FFFFFFF;
constexpr int64_t kMaxLdw = (1 << 24) - 256;  // 256 rows within 32 bits of offset

bool off(const void *p, size_t a) { return ((uintptr_t)p % a) != 0; }

}  // namespace

static kq_status grouped_gemm_impl(const uint8_t *xq, int64_t ldxq, const void *sx, int64_t T,
                                   const int32_t *rows, int64_t R, const uint8_t *wq, int64_t ldwq,
                                   int64_t ldwe, const void *sw, int64_t N, int64_t K, int64_t E,
                                   const int32_t *offsets, int bits, kq_dtype scale_dtype,
                                   kq_dtype out_dtype, void *out, int64_t ldo, void *stream) {
  if (T < 0 || R < 0 || N < 0 || K <= 0 || E < 1) return KQ_ERR_INVALID_ARG;
  if (bits != 4 && bits != 8) return KQ_ERR_INVALID_ARG;
  if (scale_dtype != KQ_FP16 && scale_dtype != KQ_FP32) return KQ_ERR_INVALID_ARG;
  if (out_dtype != KQ_FP32 && out_dtype != KQ_BF16 && out_dtype != KQ_FP16)
    return KQ_ERR_INVALID_ARG;
  if (!rows && R > T) return KQ_ERR_INVALID_ARG;
  if (K > 65536 || (K * bits) % 128 != 0 || E > 4096)
    return KQ_ERR_UNSUPPORTED;
  if (R > kMax31 || T > kMax31 || N > kMax31) return KQ_ERR_UNSUPPORTED;
  if (R == 0 || N == 0) return KQ_OK;
  if (!xq || !wq || !sx || !sw || !offsets || !out || T == 0) return KQ_ERR_INVALID_ARG;
  const int64_t rb = K * bits / 8;
  if (ldxq < rb || ldwq < rb || ldo < N) return KQ_ERR_INVALID_ARG;
  // no product of a row and a stride passes 2^62
  if (ldxq > kMax31 || ldwq > kMaxLdw || ldo > kMax31 || ldwe > ((int64_t)1 << 48))
    return KQ_ERR_UNSUPPORTED;
  if (E > 1 && ldwe < (N - 1) * ldwq + rb) return KQ_ERR_INVALID_ARG;
  const size_t ss = scale_dtype == KQ_FP16 ? 2 : 4, os = out_dtype == KQ_FP32 ? 4 : 2;
  if (off(xq, 16) || off(wq, 16) || ldxq % 16 != 0 || ldwq % 16 != 0 || (E > 1 && ldwe % 16 != 0))
    return KQ_ERR_ALIGNMENT;
  if (off(sx, ss) || off(sw, ss) || off(out, os) || off(rows, 4) || off(offsets, 4))
    return KQ_ERR_ALIGNMENT;
  const int64_t wb = (E - 1) * ldwe * (E > 1) + (N - 1) * ldwq + rb;
  const kq_span o = kq_rows_span(out, R, ldo, N, os);
  const kq_span in[6] = {kq_rows_span(xq, T, ldxq, rb, 1), kq_rows_span(sx, 1, T, T, ss),
                         kq_rows_span(rows, 1, R, R, 4), kq_rows_span(wq, 1, wb, wb, 1),
                         kq_rows_span(sw, 1, E * N, E * N, ss), kq_rows_span(offsets, 1, E + 1, E + 1, 4)};
  for (const kq_span &i : in)
    if (kq_overlap(o, i)) return KQ_ERR_INVALID_ARG;
  const GroupedArgs a = {xq, wq, sx, sw, rows, offsets, out, ldxq, ldwq, E > 1 ? ldwe : 0, T, R, N, ldo,
                         (int)(rb / 16), (int)E, scale_dtype == KQ_FP16 ? 1 : 0, (int)out_dtype};
  hipStream_t s = static_cast<hipStream_t>(stream);
  return bits == 8 ? launch<8>(a, s) : launch<4>(a, s);
}

extern "C" kq_status kq_grouped_gemm(const uint8_t *xq, int64_t ldxq, const void *sx, int64_t T,
                                     const int32_t *rows, int64_t R, const uint8_t *wq,
                                     int64_t ldwq, int64_t ldwe, const void *sw, int64_t N,
                                     int64_t K, int64_t E, const int32_t *offsets, int bits,
                                     kq_dtype scale_dtype, kq_dtype out_dtype, void *out,
                                     int64_t ldo, void *stream) {
  const kq_status st = grouped_gemm_impl(xq, ldxq, sx, T, rows, R, wq, ldwq, ldwe, sw, N, K, E,
                                         offsets, bits, scale_dtype, out_dtype, out, ldo, stream);
  if (kq_log_on())
    kq_logf("grouped_gemm R=%lld E=%lld N=%lld K=%lld bits=%d: %s", (long long)R, (long long)E,
            (long long)N, (long long)K, bits, kq_status_string(st));
  return st;
}

// kq_grouped.hip -- products of INT4 or INT8 codes grouped by expert, with ragged sizes, on
// the gfx950 int8 matrix cores.
//
//   out[i][j] = cvt( fp32( fp32( fp32(acc) * sx[t] ) * sw[e][j] ) ),  t = rows[i],
//   acc = sum_k qx[t][k] * qw[e][j][k]   (exact, int32), e the group of row i.
//
// The groups' ends are read on the device (nothing waits for the host): a workgroup finds the
// group and the row tile of its number by a scan of the groups' tile counts. The grid holds
// one tile per kTile rows and one more per group, which is as many as ragged ends can make;
// the workgroups behind the last tile end at once.
#include "kq_internal.h"
#include "kq_device.h"

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

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
  else reinterpret_cast<_Float16 *>(out)[i] = (_Float16)v;
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

// A workgroup: 16 MI output channels x 16 NI rows of one group; its waves split the reduction
// (64 bytes of a row in turn) and add their parts up in LDS (integers: any order).
template <int BITS, int MI, int NI, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void kq_grouped_stream_kernel(const GroupedArgs p, int tiles_m) {
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
  const int used = (tile.count + 15) / 16;  // 16-row blocks with a row in them
  for (int s = wave; s * 4 < p.pieces; s += WAVES) {
    const bool in = s * 4 + g < p.pieces;  // the last step may have fewer than 4 pieces
    const u32x4_t zero = {0, 0, 0, 0};
    u32x4_t a[MI];
#pragma unroll
    for (int m = 0; m < MI; ++m)
      a[m] = in ? *reinterpret_cast<const u32x4_t *>(wrow[m] + (int64_t)s * 64) : zero;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      if (j >= used) break;
      const u32x4_t b = in ? *reinterpret_cast<const u32x4_t *>(xrow[j] + (int64_t)s * 64) : zero;
#pragma unroll
      for (int m = 0; m < MI; ++m) mfma_piece<BITS>(a[m], b, acc[m][j]);
    }
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

template <int BITS>
kq_status launch(const GroupedArgs &a, hipStream_t s) {
  constexpr int MI = 2, NI = 2, WAVES = 4;
  const int64_t tiles_m = (a.N + 16 * MI - 1) / (16 * MI);
  const int64_t tiles = a.R / (16 * NI) + (a.R < a.E ? a.R : a.E);
  if (tiles_m * tiles > 0x7FFFFFFF / (WAVES * 64)) return KQ_ERR_UNSUPPORTED;
  hipLaunchKernelGGL((kq_grouped_stream_kernel<BITS, MI, NI, WAVES>), dim3((unsigned)(tiles_m * tiles)),
                     dim3(WAVES * 64), 0, s, a, (int)tiles_m);
  return hipGetLastError() == hipSuccess ? KQ_OK : KQ_ERR_HIP;
}

constexpr int64_t kMax31 = 0x7FFFFFFF;

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
  if (ldxq > kMax31 || ldwq > kMax31 || ldo > kMax31 || ldwe > ((int64_t)1 << 48))
    return KQ_ERR_UNSUPPORTED;
  if (E > 1 && ldwe < (N - 1) * ldwq + rb) return KQ_ERR_INVALID_ARG;
  const size_t ss = scale_dtype == KQ_FP16 ? 2 : 4, os = out_dtype == KQ_FP32 ? 4 : 2;
  if (off(xq, 16) || off(wq, 16) || ldxq % 16 != 0 || ldwq % 16 != 0 || (E > 1 && ldwe % 16 != 0))
    return KQ_ERR_ALIGNMENT;
  if (off(sx, ss) || off(sw, ss) || off(out, os) || off(rows, 4) || off(offsets, 4))
    return KQ_ERR_ALIGNMENT;
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

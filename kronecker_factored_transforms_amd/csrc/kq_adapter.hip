// kq_adapter.hip -- low-rank adapters of many requests at once, beside a shared projection:
//
//   out[t] = cvt( base[t] + scaling[l] * B[l] (A[l] x[t]) ),   l = adapter[t].
//
// Two kernels. The first forms the low-rank vectors h[t] = A[l] x[t] (K long, r short) and
// splits K over workgroups where tokens are few; each part goes to the workspace as fp32. The
// second adds the parts up in their order (no atomics: the result does not depend on which
// workgroup ends first), scales, and forms B[l] h + base.
//
// Both take 16 tokens at a time, in whatever order their adapters stand: for each adapter that
// occurs among the 16, one product of its matrix with all 16 columns, of which the tokens of
// that adapter keep theirs (a selection, not a product with zero: another adapter's infinities
// and NaN stay out). Tokens of one prompt stand together, so most tiles have one adapter.
#include "kq_internal.h"
#include "kq_common.h"

namespace {

constexpr int kTile = 16;         // tokens per tile
constexpr int kAdapterWaves = 4;
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
};
template <>
struct Half<1> {  // fp16
  typedef f16x8 vec;
  typedef _Float16 one;
  static __device__ __forceinline__ f32x4 mma(const vec &a, const vec &b, const f32x4 &c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};

struct AdapterArgs {
  const void *x, *A, *B, *base;
  const int32_t *adapter;
  const float *scaling;
  void *out;
  float *part;  // [splits][T][r16] parts of h
  int64_t ldx, ldb, ldo, T;
  int K, N, r, r16, L, splits, steps_per_split;  // a step: 32 values of K
};

// This lane's token's adapter (token t0 + lane % 16), -1 for none
__device__ __forceinline__ int token_adapter(const AdapterArgs &p, int64_t t0) {
  const int64_t t = t0 + (threadIdx.x & 15);
  const int l = t < p.T ? p.adapter[t] : -1;
  return l >= 0 && l < p.L ? l : -1;
}

// h's parts: grid (tiles, splits); RB blocks of 16 ranks
template <int DT, int RB>
__global__ __launch_bounds__(kAdapterWaves * 64) void kq_adapter_down_kernel(const AdapterArgs p) {
  typedef typename Half<DT>::vec vec;
  __shared__ f32x4 s_acc[kAdapterWaves][RB][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, lr = lane & 15;
  const int64_t t0 = (int64_t)blockIdx.x * kTile;
  const int l = token_adapter(p, t0);
  const int64_t t = t0 + lr < p.T ? t0 + lr : p.T - 1;
  const uint16_t *xrow = reinterpret_cast<const uint16_t *>(p.x) + t * p.ldx;
  const int s0 = blockIdx.y * p.steps_per_split;
  const int steps = min((p.K + 31) / 32 - s0, p.steps_per_split);
  unsigned long long left = __ballot(l >= 0) & 0xFFFFull;
  while (left) {
    const int a = __builtin_amdgcn_readlane(l, __builtin_ctzll(left));
    left &= ~__ballot(l == a);
    const uint16_t *am = reinterpret_cast<const uint16_t *>(p.A) + (int64_t)a * p.r * p.K;
    f32x4 acc[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s = wave; s < steps; s += kAdapterWaves) {
      const int k = (s0 + s) * 32 + g * 8;
      const bool in = k < p.K;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      const uint4 xv = in ? *reinterpret_cast<const uint4 *>(xrow + k) : zero;
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        const int row = min(16 * b + lr, p.r - 1);  // ranks past r: dropped below
        const uint4 av = in ? *reinterpret_cast<const uint4 *>(am + (int64_t)row * p.K + k) : zero;
        acc[b] = Half<DT>::mma(__builtin_bit_cast(vec, av), __builtin_bit_cast(vec, xv), acc[b]);
      }
    }
#pragma unroll
    for (int b = 0; b < RB; ++b) s_acc[wave][b][lane] = acc[b];
    __syncthreads();
    // lane: ranks 16 b + 4 g + 0..3 of token lr
    for (int b = wave; b < RB; b += kAdapterWaves) {
      f32x4 v = s_acc[0][b][lane];
#pragma unroll
      for (int w = 1; w < kAdapterWaves; ++w) v += s_acc[w][b][lane];
      if (l == a && 16 * b < p.r16)
        *reinterpret_cast<f32x4 *>(p.part + ((int64_t)blockIdx.y * p.T + t0 + lr) * p.r16 + 16 * b + 4 * g) = v;
    }
    __syncthreads();
  }
}

// out's tile: grid (tiles, column blocks); a wave makes 16 NB columns; RS steps of 32 ranks
template <int DT, int RS, int NB>
__global__ __launch_bounds__(kAdapterWaves * 64) void kq_adapter_up_kernel(const AdapterArgs p) {
  typedef typename Half<DT>::vec vec;
  typedef typename Half<DT>::one one;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, lr = lane & 15;
  const int64_t t0 = (int64_t)blockIdx.x * kTile;
  const int64_t t = t0 + lr;
  const int l = token_adapter(p, t0);
  const int n0 = (int)(blockIdx.y * kAdapterWaves + wave) * 16 * NB;

  // h of token lr, ranks 32 s + 8 g + 0..7, as two 16-bit terms
  vec hi[RS], lo[RS];
  float h[RS][8];
  float top = 0.f;
  const float sc = l >= 0 && p.scaling ? p.scaling[l] : 1.0f;
#pragma unroll
  for (int s = 0; s < RS; ++s) {
#pragma unroll
    for (int e = 0; e < 8; ++e) h[s][e] = 0.f;
    const int k = 32 * s + 8 * g;
    if (l >= 0 && k < p.r) {
      for (int i = 0; i < p.splits; ++i) {
        const f32x4 *q = reinterpret_cast<const f32x4 *>(p.part + ((int64_t)i * p.T + t) * p.r16 + k);
        const f32x4 a = q[0], b = q[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          h[s][e] += a[e];
          h[s][4 + e] += b[e];
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[s][e] = __fmul_rn(h[s][e], sc);
      top = fmaxf(top, fabsf(h[s][e]));
    }
  }
  // fp16: a power of two per token brings its h into the type's range (exact; undone on the
  // sums), so that neither term overflows or loses bits. bf16 has fp32's range.
  int ex = 0;
  if constexpr (DT == 1) {
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
      const one a = (one)v;
      hi[s][e] = a;
      lo[s][e] = (one)(__builtin_isfinite((float)a) ? __fsub_rn(v, (float)a) : 0.f);
    }

  f32x4 d[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) d[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  unsigned long long left = __ballot(l >= 0) & 0xFFFFull;
  while (left) {
    const int a = __builtin_amdgcn_readlane(l, __builtin_ctzll(left));
    left &= ~__ballot(l == a);
    const uint16_t *bm = reinterpret_cast<const uint16_t *>(p.B) + (int64_t)a * p.N * p.r;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int n = min(n0 + 16 * j + lr, p.N - 1);  // columns past N: dropped below
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < RS; ++s) {
        const int k = 32 * s + 8 * g;
        const uint4 bv = k < p.r ? *reinterpret_cast<const uint4 *>(bm + (int64_t)n * p.r + k)
                                 : make_uint4(0, 0, 0, 0);
        acc = Half<DT>::mma(__builtin_bit_cast(vec, bv), lo[s], acc);
        acc = Half<DT>::mma(__builtin_bit_cast(vec, bv), hi[s], acc);
      }
      if (l == a) d[j] = acc;
    }
  }
  if (t >= p.T) return;
  // lane: columns n0 + 16 j + 4 g + 0..3 of token lr (N is a multiple of 8: all in or all out)
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int n = n0 + 16 * j + 4 * g;
    if (n >= p.N) continue;
    union { uint2 u; one v[4]; } b, o;
    b.u = p.base ? *reinterpret_cast<const uint2 *>(reinterpret_cast<const one *>(p.base) + t * p.ldb + n)
                 : make_uint2(0, 0);
    if (l >= 0) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o.v[e] = (one)__fadd_rn((float)b.v[e], DT == 1 ? __builtin_ldexpf(d[j][e], -ex) : d[j][e]);
    } else {
      o.u = b.u;
    }
    *reinterpret_cast<uint2 *>(reinterpret_cast<one *>(p.out) + t * p.ldo + n) = o.u;
  }
}

// Parts of K: enough workgroups to fill the card where tokens are few, of 8 steps of 32 at least.
int split_count(int64_t T, int64_t K) {
  const int64_t tiles = (T + kTile - 1) / kTile, steps = (K + 31) / 32;
  int64_t s = tiles >= 512 ? 1 : 512 / tiles;
  if (s > steps / 8) s = steps / 8;
  return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

template <int DT, int RB>
hipError_t launch(const AdapterArgs &a, hipStream_t s) {
  constexpr int NB = 4;
  const unsigned tiles = (unsigned)((a.T + kTile - 1) / kTile);
  const unsigned cols = (unsigned)((a.N + 16 * NB * kAdapterWaves - 1) / (16 * NB * kAdapterWaves));
  hipLaunchKernelGGL((kq_adapter_down_kernel<DT, RB>), dim3(tiles, (unsigned)a.splits),
                     dim3(kAdapterWaves * 64), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((kq_adapter_up_kernel<DT, (RB + 1) / 2, NB>), dim3(tiles, cols),
                     dim3(kAdapterWaves * 64), 0, s, a);
  return hipGetLastError();
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

int64_t workspace_bytes(int64_t T, int64_t K, int64_t r) {
  const int64_t b = split_count(T, K) * T * ((r + 15) / 16 * 16) * 4;
  return (b + 255) / 256 * 256;
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
  if (ldx > kMax31 || (base && ldb > kMax31) || ldo > kMax31) return KQ_ERR_UNSUPPORTED;
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
  const int splits = split_count(T, K), steps = (int)((K + 31) / 32);
  const AdapterArgs a = {x, A, B, base, adapter, scaling, out, static_cast<float *>(workspace), ldx, ldb,
                         ldo, T, (int)K, (int)N, (int)r, (int)((r + 15) / 16 * 16), (int)L, splits,
                         (steps + splits - 1) / splits};
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

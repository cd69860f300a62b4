// kq_adapter.hip -- low-rank adapters of many requests at once, beside a shared projection:
//
//   out[t] = cvt( base[t] + scaling[l] * B[l] (A[l] x[t]) ),   l = adapter[t].
//
// Two kernels. The first forms the low-rank vectors h[t] = A[l] x[t] (K long, r short) and
// splits K over workgroups where tokens are few; each part goes to the workspace as fp32. The
// second adds the parts up in their order (no atomics: the result does not depend on which
// workgroup ends first), scales, and forms B[l] h + base.
//
// Both take blocks of 16 tokens as they stand: for each adapter that occurs among them, one
// product of its matrix with all 16 columns, of which the tokens of that adapter keep theirs (a
// selection, not a product with zero: another adapter's infinities and NaN stay out). The tokens
// of a prompt stand together, so most of its blocks have one adapter; the many of a decode
// batch's blocks are loaded several at a time.
#include "kq_internal.h"
#include "kq_common.h"

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
  float *part;  // [splits][T][r16] parts of h
  int64_t ldx, ldb, ldo, T;
  int K, N, r, r16, L, splits, split_steps;  // a step: 32 values of K
  int tiles_per_group;                       // up: token tiles of one workgroup
};

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

// h's parts. A workgroup takes TF blocks of 16 tokens and a share of K, which its waves split
// again and add up in LDS. D adapters at a time (their matrices' loads overlap), RB blocks of 16
// ranks, U steps of K in flight.
template <int DT, int RB, int TF, int WAVES, int D, int U>
__global__ __launch_bounds__(WAVES * 64) void kq_adapter_down_kernel(const AdapterArgs p) {
  typedef typename Half<DT>::vec vec;
  __shared__ f32x4 s_acc[WAVES][D * RB * TF][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, lr = lane & 15;
  const int64_t t0 = (int64_t)blockIdx.x * (16 * TF);
  int l[TF];
  const uint16_t *xrow[TF];
  // lanes 0..15 of the wave stand for block 0's tokens, 16..31 for block 1's
  const int mine = token_adapter(p, t0 + (lane & (16 * TF - 1)));
#pragma unroll
  for (int f = 0; f < TF; ++f) {
    l[f] = __shfl(mine, 16 * f + lr, 64);
    const int64_t t = t0 + 16 * f + lr;
    xrow[f] = reinterpret_cast<const uint16_t *>(p.x) + (t < p.T ? t : p.T - 1) * p.ldx;
  }
  const int s0 = blockIdx.y * p.split_steps;
  const int s1 = min((p.K + 31) / 32, s0 + p.split_steps);
  unsigned long long left = __ballot(mine >= 0) & ((1ull << (16 * TF)) - 1);
  while (left) {
    int a[D];
    const uint16_t *am[D];
#pragma unroll
    for (int d = 0; d < D; ++d) {
      a[d] = next_adapter(left, mine);
      am[d] = reinterpret_cast<const uint16_t *>(p.A) + (int64_t)max(a[d], 0) * p.r * p.K;
    }
    f32x4 acc[D][RB][TF];
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int f = 0; f < TF; ++f) acc[d][b][f] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s = s0 + wave; s < s1; s += WAVES * U) {
      u32x4_t xv[U][TF], av[U][D][RB];
      const u32x4_t zero = {0, 0, 0, 0};
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = (s + u * WAVES) * 32 + g * 8;
        const bool in = s + u * WAVES < s1 && k < p.K;  // behind the end: zeros on both sides
#pragma unroll
        for (int f = 0; f < TF; ++f)
          xv[u][f] = in ? *reinterpret_cast<const u32x4_t *>(xrow[f] + k) : zero;
#pragma unroll
        for (int d = 0; d < D; ++d)
#pragma unroll
          for (int b = 0; b < RB; ++b) {
            const int row = min(16 * b + lr, p.r - 1);  // ranks past r: dropped below
            av[u][d][b] = in && a[d] >= 0
                              ? *reinterpret_cast<const u32x4_t *>(am[d] + (int64_t)row * p.K + k)
                              : zero;
          }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int d = 0; d < D; ++d)
#pragma unroll
          for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int f = 0; f < TF; ++f)
              acc[d][b][f] = Half<DT>::mma(__builtin_bit_cast(vec, av[u][d][b]),
                                           __builtin_bit_cast(vec, xv[u][f]), acc[d][b][f]);
    }
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int f = 0; f < TF; ++f) s_acc[wave][(d * RB + b) * TF + f][lane] = acc[d][b][f];
    lds_barrier();
    // lane: ranks 16 b + 4 g + 0..3 of token 16 f + lr
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int f = 0; f < TF; ++f) {
          const int i = (d * RB + b) * TF + f;
          if (i % WAVES != wave) continue;
          f32x4 v = s_acc[0][i][lane];
#pragma unroll
          for (int w = 1; w < WAVES; ++w) v += s_acc[w][i][lane];
          if (a[d] >= 0 && l[f] == a[d] && 16 * b < p.r16)
            *reinterpret_cast<f32x4 *>(p.part + ((int64_t)blockIdx.y * p.T + t0 + 16 * f + lr) * p.r16 +
                                       16 * b + 4 * g) = v;
        }
    if (left) lds_barrier();  // before s_acc is written again
  }
}

constexpr int kUpWaves = 4;

// out. A workgroup takes 64 NB columns (16 NB per wave) of tiles_per_group tiles of 16 tokens; RS
// steps of 32 ranks; D adapters' B at a time. The rows of a B block are dealt so that a lane
// ends with 4 NB consecutive columns of one token.
template <int DT, int RS, int NB, int D>
__global__ __launch_bounds__(kUpWaves * 64) void kq_adapter_up_kernel(const AdapterArgs p) {
  typedef typename Half<DT>::vec vec;
  typedef typename Half<DT>::one one;
  constexpr int kW = 4 * NB / 8;  // 16-byte words of a lane's columns
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, lr = lane & 15;
  const int n0 = (int)(blockIdx.x * kUpWaves + wave) * 16 * NB;
  if (n0 >= p.N) return;  // whole waves; there is no barrier here
  int64_t tile = (int64_t)blockIdx.y * p.tiles_per_group;
  const int64_t last = min(tile + p.tiles_per_group, (p.T + 15) / 16);
  const uint32_t col = (uint32_t)(4 * NB * (lr >> 2) + (lr & 3));  // of block j: + 4 j
  const int nl = n0 + 4 * NB * g;                                  // this lane's first column
  u32x4_t bv[D][NB][RS];
  int held = -1;  // the adapter in bv[0]
  for (; tile < last; ++tile) {
    const int64_t t = tile * 16 + lr;
    const bool live = t < p.T;
    // everything that does not wait for something else first: the adapter, base, h's parts
    const int l = token_adapter(p, t);
    u32x4_t bs[kW];
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      bs[w] = u32x4_t{0, 0, 0, 0};
      if (p.base && live && nl + 8 * w < p.N)
        bs[w] = *reinterpret_cast<const u32x4_t *>(reinterpret_cast<const one *>(p.base) + t * p.ldb + nl + 8 * w);
    }
    float h[RS][8];
#pragma unroll
    for (int s = 0; s < RS; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) h[s][e] = 0.f;
    for (int i = 0; i < p.splits; ++i) {
#pragma unroll
      for (int s = 0; s < RS; ++s) {
        const int k = 32 * s + 8 * g;
        if (l >= 0 && k < p.r) {
          const f32x4 *q = reinterpret_cast<const f32x4 *>(p.part + ((int64_t)i * p.T + t) * p.r16 + k);
          const f32x4 a = q[0], b = q[1];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            h[s][e] += a[e];
            h[s][4 + e] += b[e];
          }
        }
      }
    }
    // h of token lr, ranks 32 s + 8 g + 0..7, as two 16-bit terms
    const float sc = l >= 0 && p.scaling ? p.scaling[l] : 1.0f;
    float top = 0.f;
#pragma unroll
    for (int s = 0; s < RS; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[s][e] = __fmul_rn(h[s][e], sc);
        if constexpr (DT == 1) top = fmaxf(top, fabsf(h[s][e]));
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
    vec hi[RS], lo[RS];
#pragma unroll
    for (int s = 0; s < RS; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = DT == 1 ? __builtin_ldexpf(h[s][e], ex) : h[s][e];
        const one a = Half<DT>::round(v);
        hi[s][e] = a;
        lo[s][e] = Half<DT>::round(__builtin_isfinite((float)a) ? __fsub_rn(v, (float)a) : 0.f);
      }

    f32x4 d[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) d[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    unsigned long long left = __ballot(l >= 0) & 0xFFFFull;
    while (left) {
      int a[D];
#pragma unroll
      for (int k = 0; k < D; ++k) a[k] = next_adapter(left, l);
#pragma unroll
      for (int k = 0; k < D; ++k) {
        if (a[k] < 0 || (k == 0 && a[0] == held)) continue;
        const uint16_t *bm = reinterpret_cast<const uint16_t *>(p.B) + (int64_t)a[k] * p.N * p.r;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const int n = min(n0 + (int)col + 4 * j, p.N - 1);  // columns past N: dropped below
#pragma unroll
          for (int s = 0; s < RS; ++s) {
            const int kk = 32 * s + 8 * g;
            bv[k][j][s] = kk < p.r ? *reinterpret_cast<const u32x4_t *>(bm + (int64_t)n * p.r + kk)
                                   : u32x4_t{0, 0, 0, 0};
          }
        }
      }
      held = a[0];
#pragma unroll
      for (int k = 0; k < D; ++k) {
        if (a[k] < 0) continue;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < RS; ++s) {
            acc = Half<DT>::mma(__builtin_bit_cast(vec, bv[k][j][s]), lo[s], acc);
            acc = Half<DT>::mma(__builtin_bit_cast(vec, bv[k][j][s]), hi[s], acc);
          }
          if (l == a[k]) d[j] = acc;
        }
      }
    }
    if (!live) continue;
    // lane: columns nl + 4 j + r of token lr (N is a multiple of 8: a word is all in or all out)
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      if (nl + 8 * w >= p.N) continue;
      if (l >= 0) {
        one v[8];
        const one *b = reinterpret_cast<const one *>(&bs[w]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float add = d[2 * w + e / 4][e % 4];
          v[e] = Half<DT>::round(__fadd_rn((float)b[e], DT == 1 ? __builtin_ldexpf(add, -ex) : add));
        }
        bs[w] = *reinterpret_cast<const u32x4_t *>(v);
      }
      *reinterpret_cast<u32x4_t *>(reinterpret_cast<one *>(p.out) + t * p.ldo + nl + 8 * w) = bs[w];
    }
  }
}

// The first kernel's shape: blocks of 16 tokens per workgroup and its waves
constexpr int64_t kWide = 4096;  // from this many tokens on: 32 tokens, 8 waves
int down_tokens(int64_t T) { return T >= kWide ? 32 : 16; }
int down_waves(int64_t T) { return T >= kWide ? 8 : 4; }

// Parts of K: enough workgroups to fill the card where tokens are few, of 2 steps a wave at
// least, and no more than the second kernel can add up at ease.
int split_count(int64_t T, int64_t K) {
  const int64_t tiles = (T + down_tokens(T) - 1) / down_tokens(T), steps = (K + 31) / 32;
  int64_t s = (T >= kWide ? 256 : 512) / tiles;
  const int64_t most = steps / (2 * down_waves(T));
  if (s > most) s = most;
  return (int)(s < 1 ? 1 : s > 16 ? 16 : s);
}

template <int DT, int RB>
hipError_t launch(AdapterArgs a, hipStream_t s) {
  // adapters at a time and steps in flight: about 20 loads of a wave on their way
  constexpr int D = RB == 1 ? 4 : RB <= 4 ? 2 : 1;
  constexpr int U = RB == 1 ? 4 : RB == 2 ? 4 : RB <= 8 ? 2 : 1;
  constexpr int UW = RB == 1 ? 8 : RB <= 4 ? 4 : RB == 8 ? 2 : 1;
  const unsigned tiles = (unsigned)((a.T + down_tokens(a.T) - 1) / down_tokens(a.T));
  constexpr int kWideWaves = RB < 16 ? 8 : 4;  // their parts in LDS: 128 KiB at most
  const dim3 grid(tiles, (unsigned)a.splits);
  if (a.T >= kWide)
    hipLaunchKernelGGL((kq_adapter_down_kernel<DT, RB, 2, kWideWaves, 1, UW>), grid, dim3(kWideWaves * 64), 0,
                       s, a);
  else
    hipLaunchKernelGGL((kq_adapter_down_kernel<DT, RB, 1, 4, D, U>), grid, dim3(4 * 64), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  constexpr int RS = (RB + 1) / 2, NB = RS <= 2 ? 4 : 2, DU = RS == 1 ? 4 : RS <= 4 ? 2 : 1;
  const int64_t t16 = (a.T + 15) / 16;
  const int64_t cols = (a.N + 16 * NB * kUpWaves - 1) / (16 * NB * kUpWaves);
  // some 2048 workgroups, each over a run of tiles whose adapters' B it keeps
  int64_t run = t16 * cols / 2048;
  if (run < 1) run = 1;
  if (run > 64) run = 64;
  while ((t16 + run - 1) / run > 65535) run *= 2;  // the grid's second dimension
  a.tiles_per_group = (int)run;
  hipLaunchKernelGGL((kq_adapter_up_kernel<DT, RS, NB, DU>), dim3((unsigned)cols, (unsigned)((t16 + run - 1) / run)),
                     dim3(kUpWaves * 64), 0, s, a);
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
                         (steps + splits - 1) / splits, 1};
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

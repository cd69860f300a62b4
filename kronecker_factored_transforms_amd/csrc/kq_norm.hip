// kq_norm.hip -- the residual's addition, the root-mean-square norm and INT8 codes with a
// step per row, in one pass over the row.
//
//   h = x + residual,  u = h * w,  r = 1 / sqrt(sum(h^2) / n + eps),  y = u * r,
//   a = max |y|,  s = clip a / 127,  q = clamp(rint(y / s)).
//
// r is positive and rounding is monotone, so max |u * r| = (max |u|) * r to the last bit:
// one reduction over the row, of the pair (sum h^2, max |u|), gives both the norm and the
// quantizer's step, and the row stays in registers (as u) between them.
//
// Bound by memory: x and the residual are read once, the sum and the codes written once (7
// bytes per bf16 value). 16384 x 8192 bf16 with a residual: 163-166 us, 5.7 TB/s, where a
// device-to-device copy of the same size reaches 5.2.
#include "kq_internal.h"
#include "kq_linear.h"

namespace {

constexpr int kMaxRow = 65536;

template <int DT>  // 0: bf16, 1: fp16, 2: fp32
struct Elem;
template <>
struct Elem<0> {
  typedef uint16_t raw;
  static __device__ __forceinline__ float get(raw v) { return __uint_as_float((uint32_t)v << 16); }
  static __device__ __forceinline__ raw put(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
};
template <>
struct Elem<1> {
  typedef uint16_t raw;
  static __device__ __forceinline__ float get(raw v) { return (float)__builtin_bit_cast(_Float16, v); }
  static __device__ __forceinline__ raw put(float v) { return __builtin_bit_cast(uint16_t, half_rne(v)); }
};
template <>
struct Elem<2> {
  typedef float raw;
  static __device__ __forceinline__ float get(raw v) { return v; }
  static __device__ __forceinline__ raw put(float v) { return v; }
};

// A thread's 8 values of a chunk as they stand in memory
template <int DT>
struct Raw8 {
  typename Elem<DT>::raw v[8];
};

// The 16-byte words of a chunk. Rows of any alignment are read and written with the same
// instructions: global memory takes a vector access at any address, and the compiler emits
// it for a type whose alignment is declared as one element's.
template <int DT, bool VEC>
struct Words {
  typedef u32x4_t type;
};
template <>
struct Words<0, false> { typedef u32x4_t type __attribute__((aligned(2))); };
template <>
struct Words<1, false> { typedef u32x4_t type __attribute__((aligned(2))); };
template <>
struct Words<2, false> { typedef u32x4_t type __attribute__((aligned(4))); };

// Where value e of thread t's chunk c stands in its row, NT threads to a row: the threads' words
// follow each other, so that an access covers whole lines (fp32: two words of 4 values; 4096 rows of
// 11008 with a residual 104 us, as 8 neighbours 121; 3000 rows of 1001 at odd addresses, both outputs,
// 10.1, 12.2; 777 of 5121 16.6, 15.7)
template <int DT, int NT>
__device__ __forceinline__ int value_at(int c, int t, int e) {
  constexpr int kV = DT == 2 ? 4 : 8;  // values of a word
  return c * NT * 8 + e / kV * (NT * kV) + t * kV + e % kV;
}

// Thread t's values of chunk c of a row of n. VEC: rows are 16-byte aligned and n is a multiple
// of 8. Otherwise the last word may be cut off; its missing values are 0, and never touched.
template <int DT, int NT, bool VEC>
__device__ __forceinline__ Raw8<DT> load8(const void *p, int c, int t, int n) {
  typedef typename Elem<DT>::raw raw;
  typedef typename Words<DT, VEC>::type word;
  constexpr int kV = 16 / sizeof(raw);
  const raw *q = reinterpret_cast<const raw *>(p);
  Raw8<DT> v = {};
#pragma unroll
  for (int k = 0; k < 8; k += kV) {
    const int i = value_at<DT, NT>(c, t, k);
    if (i + kV <= n) {
      *reinterpret_cast<u32x4_t *>(v.v + k) = *reinterpret_cast<const word *>(q + i);
    } else if constexpr (!VEC) {
#pragma unroll
      for (int e = 0; e < kV; ++e)
        if (i + e < n) v.v[k + e] = q[i + e];
    }
  }
  return v;
}

template <int DT, int NT, bool VEC>
__device__ __forceinline__ void store8(void *p, int c, int t, int n, const float (&v)[8]) {
  typedef typename Elem<DT>::raw raw;
  typedef typename Words<DT, VEC>::type word;
  constexpr int kV = 16 / sizeof(raw);
  raw *q = reinterpret_cast<raw *>(p);
  Raw8<DT> o;
#pragma unroll
  for (int e = 0; e < 8; ++e) o.v[e] = Elem<DT>::put(v[e]);
#pragma unroll
  for (int k = 0; k < 8; k += kV) {
    const int i = value_at<DT, NT>(c, t, k);
    if (i + kV <= n) {
      *reinterpret_cast<word *>(q + i) = *reinterpret_cast<const u32x4_t *>(o.v + k);
    } else if constexpr (!VEC) {
#pragma unroll
      for (int e = 0; e < kV; ++e)
        if (i + e < n) q[i + e] = o.v[k + e];
    }
  }
}

// The codes of such a chunk, the low byte of each b
template <int DT, int NT, bool VEC>
__device__ __forceinline__ void store_codes(uint8_t *q, int c, int t, int n, const uint32_t (&b)[8]) {
  typedef u32x2_t any8 __attribute__((aligned(1)));
  typedef uint32_t any4 __attribute__((aligned(1)));
  constexpr int kV = DT == 2 ? 4 : 8;
  const uint32_t w[2] = {b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24, b[4] | b[5] << 8 | b[6] << 16 | b[7] << 24};
#pragma unroll
  for (int k = 0; k < 8; k += kV) {
    const int i = value_at<DT, NT>(c, t, k);
    if (i + kV <= n) {
      if constexpr (kV == 4 && VEC) *reinterpret_cast<uint32_t *>(q + i) = w[k / 4];
      else if constexpr (kV == 4) *reinterpret_cast<any4 *>(q + i) = w[k / 4];
      else if constexpr (VEC) *reinterpret_cast<u32x2_t *>(q + i) = u32x2_t{w[0], w[1]};
      else *reinterpret_cast<any8 *>(q + i) = u32x2_t{w[0], w[1]};
    } else if constexpr (!VEC) {
#pragma unroll
      for (int e = 0; e < kV; ++e)
        if (i + e < n) q[i + e] = (uint8_t)b[k + e];
    }
  }
}

// The same value, unknown to the compiler: it would otherwise keep every chunk's offsets and
// bounds in registers across the rows, and spill u for them.
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

struct NormArgs {
  const void *x, *res, *w;
  void *res_out, *normed;
  uint8_t *codes;
  void *scales;
  int64_t T, ldx, ldr, ldres, ldy;
  int n;
  float eps, clip;
  int scale_fp16;
};

// One row per NT threads (a workgroup, or a wave or half a wave of a workgroup of four waves);
// CPT chunks of 8 values per thread.
template <int DT, int NT, int CPT, bool VEC>
__global__ __launch_bounds__(NT < 128 ? 256 : NT) void kq_norm_kernel(const NormArgs a) {
  constexpr int kThreads = NT < 128 ? 256 : NT;
  constexpr int kRows = kThreads / NT;  // rows per workgroup
  constexpr int kWaves = NT < 64 ? 1 : NT / 64;       // waves per row
  // a workgroup of 1024 threads has 128 registers for each: there the row comes in parts, and
  // of its longest rows (n > 32768) a quarter of u waits in LDS, each thread's own values
  // (2048 rows of 65536: 218 us; all in registers, with spills, 230; half in LDS 252)
  constexpr int kPart = NT < 1024 || CPT < 2 ? CPT : 2;
  constexpr int kHeld = CPT < 6 ? CPT : 6;
  typedef typename Elem<DT>::raw raw;
  __shared__ float s_red[2][2][kThreads / 64];
  __shared__ f32x4 s_u[CPT > kHeld ? (CPT - kHeld) * 2 : 1][CPT > kHeld ? NT : 1];
  const int tid = threadIdx.x % NT, wave = threadIdx.x / 64;
  int turn = 0;
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < a.T; base += (int64_t)gridDim.x * kRows) {
    const int64_t t = base + threadIdx.x / NT;
    const bool live = t < a.T;
    float u[kHeld][8];
    float sum = 0.f, top = 0.f;
    if (live) {
      const raw *x = reinterpret_cast<const raw *>(a.x) + t * a.ldx;
      const raw *r = a.res ? reinterpret_cast<const raw *>(a.res) + t * a.ldr : nullptr;
      raw *ro = a.res_out ? reinterpret_cast<raw *>(a.res_out) + t * a.ldres : nullptr;
      // a part of the row is on its way before its first value is used (and before any store,
      // which the compiler could not move a load across); kPart chunks at a time are held as
      // they came, beside the u of the whole row
#pragma unroll
      for (int c0 = 0; c0 < CPT; c0 += kPart) {
        const int at = opaque(tid);
        Raw8<DT> xv[kPart], rv[kPart], wv[kPart];
#pragma unroll
        for (int c = 0; c < kPart; ++c) xv[c] = load8<DT, NT, VEC>(x, c0 + c, at, a.n);
        if (r) {
#pragma unroll
          for (int c = 0; c < kPart; ++c) rv[c] = load8<DT, NT, VEC>(r, c0 + c, at, a.n);
        }
#pragma unroll
        for (int c = 0; c < kPart; ++c) wv[c] = load8<DT, NT, VEC>(a.w, c0 + c, at, a.n);
#pragma unroll
        for (int c = 0; c < kPart; ++c) {
          float h[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            h[e] = Elem<DT>::get(xv[c].v[e]);
            if (r) h[e] = __fadd_rn(h[e], Elem<DT>::get(rv[c].v[e]));
          }
          if (ro) store8<DT, NT, VEC>(ro, c0 + c, at, a.n, h);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            sum = fmaf(h[e], h[e], sum);
            h[e] = __fmul_rn(h[e], Elem<DT>::get(wv[c].v[e]));
            top = fmaxf(top, fabsf(h[e]));
          }
          if (c0 + c < kHeld) {
#pragma unroll
            for (int e = 0; e < 8; ++e) u[(c0 + c) % kHeld][e] = h[e];
          } else {
            s_u[(c0 + c - kHeld) * 2][tid] = f32x4{h[0], h[1], h[2], h[3]};
            s_u[(c0 + c - kHeld) * 2 + 1][tid] = f32x4{h[4], h[5], h[6], h[7]};
          }
        }
        if constexpr (CPT > kPart) __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int o = (NT < 64 ? NT : 64) / 2; o >= 1; o >>= 1) {
      sum += __shfl_xor(sum, o, 64);
      top = fmaxf(top, __shfl_xor(top, o, 64));
    }
    if constexpr (kWaves > 1) {  // two halves in turn: one barrier per row
      if (threadIdx.x % 64 == 0) {
        s_red[turn][0][wave] = sum;
        s_red[turn][1][wave] = top;
      }
      __syncthreads();
      sum = 0.f;
      top = 0.f;
#pragma unroll
      for (int k = 0; k < kWaves; ++k) {
        sum += s_red[turn][0][k];
        top = fmaxf(top, s_red[turn][1][k]);
      }
      turn ^= 1;
    }
    if (!live) continue;
    const float root = sqrtf(__fadd_rn(__fdiv_rn(sum, (float)a.n), a.eps));
    const float rstd = root == 0.f ? 0.f : __fdiv_rn(1.0f, root);
    const TokenScale ts = token_scale(__fmul_rn(top, rstd), a.clip, a.scale_fp16, 127.0f);
    if (a.codes && tid == 0) store_scale(a.scales, t, ts, a.scale_fp16);
    raw *yo = a.normed ? reinterpret_cast<raw *>(a.normed) + t * a.ldy : nullptr;
    uint8_t *q = a.codes ? a.codes + t * a.n : nullptr;
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      const int at = opaque(tid);
      float y[8];
      if (c < kHeld) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __fmul_rn(u[c % kHeld][e], rstd);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __fmul_rn(s_u[(c - kHeld) * 2 + e / 4][tid][e % 4], rstd);
      }
      if (yo) store8<DT, NT, VEC>(yo, c, at, a.n, y);
      if (q) {
        // fp32 y * inv plus 1.5 * 2^23 rounds to the nearest integer, ties to even, into the
        // low mantissa bits (|y * inv| < 2^22: at most about 127 / clip, else clamped)
        uint32_t b[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = fminf(fmaxf(__fmul_rn(y[e], ts.inv), -128.0f), 127.0f);
          b[e] = __float_as_uint(__fadd_rn(v, 12582912.0f)) & 0xFFu;
        }
        store_codes<DT, NT, VEC>(q, c, at, a.n, b);
      }
    }
  }
}

template <int DT, int NT, int CPT>
hipError_t launch(const NormArgs &a, bool vec, hipStream_t s) {
  constexpr int kThreads = NT < 128 ? 256 : NT;
  constexpr int kRows = kThreads / NT;
  const int64_t groups = (a.T + kRows - 1) / kRows;
  const dim3 grid((unsigned)(groups < 16384 ? groups : 16384)), block(kThreads);
  if (vec)
    hipLaunchKernelGGL((kq_norm_kernel<DT, NT, CPT, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((kq_norm_kernel<DT, NT, CPT, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

// Threads per row by its length: as few as hold it in 2 to 4 chunks each, so that several rows
// of a compute unit are at different places (reading, reducing, writing). Measured on 16384
// rows of bf16 with a residual: n = 8192 as 256 x 4 chunks 163-166 us, 512 x 2 174, 1024 x 1 182;
// n = 2048 as 128 x 2 44 us, 256 x 1 47; n = 1024 as 64 x 2 24.5 us, 64 x 4 27, 256 x 1 32.5;
// 65536 rows of 256 as 32 lanes 27 us, as 64 (half of them idle) 35. fp32 chunks are twice as
// large: n = 5120 as 512 x 2 9.4 us, 256 x 4 10.3.
template <int DT>
hipError_t dispatch(const NormArgs &a, bool vec, hipStream_t s) {
  if (a.n <= 256) return launch<DT, 32, 1>(a, vec, s);
  if (a.n <= 512) return launch<DT, 64, 1>(a, vec, s);
  if (a.n <= 1024) return launch<DT, 64, 2>(a, vec, s);
  if (a.n <= 2048) return launch<DT, 128, 2>(a, vec, s);
  if (a.n <= 4096) return launch<DT, 256, 2>(a, vec, s);
  if constexpr (DT == 2) {
    if (a.n <= 8192) return launch<DT, 512, 2>(a, vec, s);
    if (a.n <= 16384) return launch<DT, 1024, 2>(a, vec, s);
  }
  if (a.n <= 8192) return launch<DT, 256, 4>(a, vec, s);
  if (a.n <= 16384) return launch<DT, 512, 4>(a, vec, s);
  if (a.n <= 32768) return launch<DT, 1024, 4>(a, vec, s);
  return launch<DT, 1024, 8>(a, vec, s);
}

bool off(const void *p, size_t a) { return ((uintptr_t)p % a) != 0; }

}  // namespace

static kq_status rmsnorm_quant_impl(const void *x, int64_t ldx, const void *residual, int64_t ldr,
                                    const void *w, int64_t T, int64_t n, kq_dtype x_dtype,
                                    float eps, float alpha, kq_dtype scale_dtype, void *res_out,
                                    int64_t ldres, void *normed, int64_t ldy, uint8_t *codes,
                                    void *scales, void *stream) {
  if (T < 0 || n < 1) return KQ_ERR_INVALID_ARG;
  if (x_dtype != KQ_BF16 && x_dtype != KQ_FP16 && x_dtype != KQ_FP32) return KQ_ERR_INVALID_ARG;
  if (scale_dtype != KQ_FP16 && scale_dtype != KQ_FP32) return KQ_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !(eps < __builtin_huge_valf()) || alpha != alpha) return KQ_ERR_INVALID_ARG;
  if (n > kMaxRow) return KQ_ERR_UNSUPPORTED;
  if (T > ((int64_t)1 << 40) / n) return KQ_ERR_INVALID_ARG;
  if (T == 0) return KQ_OK;
  if (!x || !w || (!codes && !normed) || (!codes != !scales)) return KQ_ERR_INVALID_ARG;
  if (!residual && res_out) return KQ_ERR_INVALID_ARG;
  if (ldx < n || (residual && ldr < n) || (res_out && ldres < n) || (normed && ldy < n))
    return KQ_ERR_INVALID_ARG;
  const int64_t kMaxLd = (int64_t)1 << 40;
  for (const int64_t ld : {ldx, ldr, ldres, ldy})  // no product of a row and a stride passes 2^62
    if (ld > kMaxLd || (T > 1 && (double)T * (double)ld > 1e18)) return KQ_ERR_INVALID_ARG;
  const size_t es = x_dtype == KQ_FP32 ? 4 : 2;
  if (off(x, es) || off(residual, es) || off(w, es) || off(res_out, es) || off(normed, es) ||
      off(scales, scale_dtype == KQ_FP32 ? 4 : 2))
    return KQ_ERR_ALIGNMENT;
  const kq_span in[3] = {kq_rows_span(x, T, ldx, n, es), kq_rows_span(residual, T, ldr, n, es),
                         kq_rows_span(w, 1, n, n, es)};
  const kq_span out[4] = {kq_rows_span(res_out, T, ldres, n, es), kq_rows_span(normed, T, ldy, n, es),
                          kq_rows_span(codes, T, n, n, 1),
                          kq_rows_span(scales, 1, T, T, scale_dtype == KQ_FP32 ? 4 : 2)};
  for (int i = 0; i < 4; ++i) {
    for (int j = i + 1; j < 4; ++j)
      if (kq_overlap(out[i], out[j])) return KQ_ERR_INVALID_ARG;
    for (int j = 0; j < 3; ++j) {
      if (!kq_overlap(out[i], in[j])) continue;
      // each thread writes the values it has read: the very same rows may be written in place
      const bool same = (i == 0 && j == 0 && res_out == x && ldres == ldx) ||
                        (i == 0 && j == 1 && res_out == residual && ldres == ldr) ||
                        (i == 1 && j == 0 && normed == x && ldy == ldx);
      if (!same) return KQ_ERR_INVALID_ARG;
    }
  }
  bool vec = n % 8 == 0 && !off(x, 16) && !off(w, 16) && ldx * es % 16 == 0 && !off(codes, 8);
  if (residual) vec = vec && !off(residual, 16) && ldr * es % 16 == 0;
  if (res_out) vec = vec && !off(res_out, 16) && ldres * es % 16 == 0;
  if (normed) vec = vec && !off(normed, 16) && ldy * es % 16 == 0;
  const NormArgs a = {x, residual, w, res_out, normed, codes, scales, T, ldx, ldr, ldres, ldy,
                      (int)n, eps, kq_clip_of_alpha(alpha), scale_dtype == KQ_FP16 ? 1 : 0};
  hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = x_dtype == KQ_BF16   ? dispatch<0>(a, vec, s)
                       : x_dtype == KQ_FP16 ? dispatch<1>(a, vec, s)
                                            : dispatch<2>(a, vec, s);
  return e == hipSuccess ? KQ_OK : KQ_ERR_HIP;
}

extern "C" kq_status kq_rmsnorm_quant(const void *x, int64_t ldx, const void *residual, int64_t ldr,
                                      const void *w, int64_t T, int64_t n, kq_dtype x_dtype,
                                      float eps, float alpha, kq_dtype scale_dtype, void *res_out,
                                      int64_t ldres, void *normed, int64_t ldy, uint8_t *codes,
                                      void *scales, void *stream) {
  const kq_status st = rmsnorm_quant_impl(x, ldx, residual, ldr, w, T, n, x_dtype, eps, alpha,
                                          scale_dtype, res_out, ldres, normed, ldy, codes, scales,
                                          stream);
  if (kq_log_on())
    kq_logf("rmsnorm_quant T=%lld n=%lld: %s", (long long)T, (long long)n, kq_status_string(st));
  return st;
}

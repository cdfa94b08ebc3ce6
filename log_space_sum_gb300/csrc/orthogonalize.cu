// Orthogonalised update: X_0 = G / (|G|_F + eps), transposed when G is taller than wide (so
// that X is M x N with M <= N), then `steps` times
//
//   A = X X^T,   B = b A + c A A,   X <- a X + B X.
//
// The polynomial a s + b s^3 + c s^5 acts on the singular values of X and drives them
// towards one. Compute-bound from a few hundred rows on: M^2 N + M^3 + 2 M^2 N flops a
// step, the symmetric halves of A and A A taken once (tiles on and above the diagonal,
// mirrored by the epilogue).
//
// Operands are float16: the iteration's values are bounded (singular values below about
// 1.3), so its 11 significant bits can be had at the tensor core's 16-bit rate, eight times
// finer than bf16; precision PC_PREC_FP32 keeps hi + lo parts (22 bits) and three products.
// Power-of-two factors keep every operand in float16's range: X is stored as Xs with X =
// 2^-s Xs, 2^s ~ sqrt(N) (a row of X then has entries of about one), A as 2^12 A, B as
// 2^10 B. The first Xs is G times a power of two alone (exact for bf16 G); the rest of
// the norm, nu, enters with the first products in float32. Where |G|_F is small beside eps, so is
// X, and it grows by a step: its matrix then has a further power of two for each step (orth_scales).
//
// Very wide matrices take several steps on the M x M matrix alone: with P = a I + B, X' = P X has
// X' X'^T = P A P, everything commutes, and
//
//   T = A P = a A + A B,   A <- T P = a T + T B,   Q <- Q P = a Q + Q B   (Q = P at first)
//
// are symmetric products of M x M matrices; X <- Q X at the end. An error of A in the direction
// of a small singular value grows by a^2 a step (2e4 over four), so A, B, T and Q are kept in two
// parts here; X itself is then rounded once in all, and bf16 G not at all.
//
// Measured, five steps, bf16: 1024 x 1024 129 us (15 dependent products of 8 us: 2.1 from launch to
// launch, 2.7 of cluster exchange, 1.0 of products), 1024 x 16384 275 us (14 M x M products in two parts of
// 12 us, gram 25, last product 49: 1.40 PF/s); float32, 6 of 770 x 333: 162 us.
#include <cuda_fp16.h>

#include "pc_gemm.cuh"
#include "pc_host.h"

namespace pc {
namespace {

constexpr float kScaleA = 4096.f, kScaleB = 1024.f, kScaleQ = 64.f;

// ------------------------------------------------------------------ norm and operands
constexpr int kNormThreads = 256, kNormBlocks = 608;

__device__ __forceinline__ float orth_value(const float* p) { return *p; }
__device__ __forceinline__ float orth_value(const __nv_bfloat16* p) { return __bfloat162float(*p); }

__device__ __forceinline__ float block_total(float v, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kNormThreads / 32; ++w) s += red[w];
  return s;
}

// 16 bytes of G: 8 bf16 or 4 float values.
template <class T>
constexpr int kPiece = 16 / sizeof(T);
__device__ __forceinline__ void orth_unpack(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void orth_unpack(const uint4& u, float (&v)[4]) {
  v[0] = __uint_as_float(u.x);
  v[1] = __uint_as_float(u.y);
  v[2] = __uint_as_float(u.z);
  v[3] = __uint_as_float(u.w);
}

// part[g][block]: partial sums of squares, in an order that depends on the size alone. G is
// 16-byte aligned; so is every matrix of a stack whose size is a whole number of pieces
// (kVec), the others are read value by value.
template <class T, bool kVec>
__global__ void __launch_bounds__(kNormThreads) k_orth_squares(long long n, const T* __restrict__ g, float* part) {
  grid_dependents_launch();
  __shared__ float red[kNormThreads / 32];
  constexpr int L = kVec ? kPiece<T> : 1, kFlight = kVec ? 4 : 8;
  const T* p = g + static_cast<long long>(blockIdx.y) * n;
  const long long stride = static_cast<long long>(gridDim.x) * kNormThreads;
  float s = 0.f;
  for (long long i = blockIdx.x * static_cast<long long>(kNormThreads) + threadIdx.x; i < n / L;
       i += kFlight * stride) {
    float v[kFlight][L];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const long long at = i + k * stride;
#pragma unroll
      for (int e = 0; e < L; ++e) v[k][e] = 0.f;
      if (at < n / L) {
        if constexpr (kVec)
          orth_unpack(reinterpret_cast<const uint4*>(p)[at], v[k]);
        else
          v[k][0] = orth_value(p + at);
      }
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k)
#pragma unroll
      for (int e = 0; e < L; ++e) s += v[k][e] * v[k][e];
  }
  s = block_total(s, red);
  if (threadIdx.x == 0) part[blockIdx.y * kNormBlocks + blockIdx.x] = s;
}

// A matrix of float16 operands: rows of ld elements, hi, then lo at +lo (0: none).
struct HalfMat {
  __half* ptr;
  long long rows, cols, ld;
  size_t lo;
};

__device__ __forceinline__ void half_split(float v, __half* hi, __half* lo) {
  *hi = __float2half_rn(v);
  *lo = __float2half_rn(v - __half2float(*hi));
}

// The whole block's |G|_F^2 from its matrix's partial sums.
__device__ __forceinline__ float orth_total(int blocks, const float* part, float* red) {
  float s = 0.f;
  for (int i = threadIdx.x; i < blocks; i += kNormThreads) s += part[i];
  return block_total(s, red);
}

// 2^e for Xs = 2^e G: 2^e |G|_F <= 2^15 and the root mean square near one, exponents only.
// Zero (or a norm that is not finite): e = 0, and nu = 2^-e / (|G|_F + eps) carries what
// comes of it.
__device__ __forceinline__ float orth_scale(int rows, int cols, float total, float eps, float* nu) {
  const float norm = sqrtf(total);
  int e = 0;
  if (norm > 0.f && norm < 3e38f) {
    int at;
    frexpf(norm, &at);  // norm = f 2^at, f in [1/2, 1)
    const int spread = (32 - __clz(rows) + 32 - __clz(cols)) / 2;  // sqrt(rows cols) within a factor of two
    e = max(-126, min(min(spread, 15) - at, 126));
  }
  *nu = total == 0.f ? 0.f : ldexpf(1.f, -e) / (norm + eps);
  return ldexpf(1.f, e);
}

// What a matrix's X before each step is held by: X_0 = x Xs, and X_k = 2^-s x Xs with x = 1 / y a power of
// two, from the bound u of |X_k|_F that the polynomial gives: y u <= 1 where u < 1/2, else y = 1.
// scales[step][batch].
struct OrthSteps {
  int steps, batch;
  float a, b, c;
  float2* scales;
};
constexpr int kMaxSteps = 100;
__device__ __forceinline__ void orth_scales(const OrthSteps& p, int m, float total, float eps, float nu) {
  p.scales[m] = make_float2(nu, 1.f);
  float u = sqrtf(total) / (sqrtf(total) + eps);
  for (int k = 1; k < p.steps; ++k) {
    const float u2 = u * u;
    u = fminf(u * (fabsf(p.a) + u2 * (fabsf(p.b) + u2 * fabsf(p.c))), 2.f);
    int t = 0;
    if (u > 0.f && u < 0.5f) frexpf(u, &t);  // u = f 2^t, f in [1/2, 1)
    t = max(t, -126);
    p.scales[static_cast<size_t>(k) * p.batch + m] = make_float2(ldexpf(1.f, t), ldexpf(1.f, -t));
  }
}

// Xs = 2^e G where G is not taller than wide and its rows are whole 16-byte pieces: a stream.
template <class T, int kParts>
__global__ void __launch_bounds__(kNormThreads)
    k_orth_load_rows(int rows, int cols, const T* __restrict__ g, int blocks, const float* part, float eps, HalfMat x,
                     const OrthSteps steps) {
  __shared__ float red[kNormThreads / 32];
  constexpr int L = kPiece<T>, kFlight = 4;
  const int m = blockIdx.y, pieces = cols / L;
  const long long n = static_cast<long long>(rows) * pieces, stride = static_cast<long long>(gridDim.x) * kNormThreads;
  const T* src = g + static_cast<long long>(m) * rows * cols;
  __half* dst = x.ptr + static_cast<size_t>(m) * x.rows * x.ld;
  long long i = blockIdx.x * static_cast<long long>(kNormThreads) + threadIdx.x;
  uint4 raw[kFlight];
  auto fetch = [&]() {
#pragma unroll
    for (int k = 0; k < kFlight; ++k)
      if (i + k * stride < n) raw[k] = reinterpret_cast<const uint4*>(src)[i + k * stride];
  };
  fetch();
  grid_dependency_wait();  // the sums of squares
  grid_dependents_launch();
  float inv;
  const float total = orth_total(blocks, part + m * kNormBlocks, red), up = orth_scale(rows, cols, total, eps, &inv);
  if (blockIdx.x == 0 && threadIdx.x == 0) orth_scales(steps, m, total, eps, inv);
  for (; i < n; i += kFlight * stride, fetch()) {
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const long long at = i + k * stride;
      if (at >= n) break;
      float v[L];
      orth_unpack(raw[k], v);
      uint32_t hi[L / 2], lo[L / 2];
#pragma unroll
      for (int e = 0; e < L / 2; ++e) {
        __half h0, l0, h1, l1;
        half_split(v[2 * e] * up, &h0, &l0);
        half_split(v[2 * e + 1] * up, &h1, &l1);
        const __half2 h = __halves2half2(h0, h1), l = __halves2half2(l0, l1);
        hi[e] = *reinterpret_cast<const uint32_t*>(&h);
        lo[e] = *reinterpret_cast<const uint32_t*>(&l);
      }
      __half* to = dst + (at / pieces) * x.ld + (at % pieces) * L;
      if constexpr (L == 8) {
        *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if constexpr (kParts == 2) *reinterpret_cast<uint4*>(to + x.lo) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      } else {
        *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
        if constexpr (kParts == 2) *reinterpret_cast<uint2*>(to + x.lo) = make_uint2(lo[0], lo[1]);
      }
    }
  }
}

// Xs = 2^e G (or its transpose) over 64 x 64 tiles; any shape and alignment.
template <class T, int kParts>
__global__ void __launch_bounds__(kNormThreads)
    k_orth_load(int rows, int cols, const T* __restrict__ g, int blocks, const float* part, float eps, int tall,
                HalfMat x, const OrthSteps steps) {
  __shared__ float red[kNormThreads / 32];
  __shared__ float tile[64][65];
  const int m = blockIdx.z, t = threadIdx.x;
  const T* src = g + static_cast<long long>(m) * rows * cols;
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
  constexpr int L = kPiece<T>, kPerRow = 64 / L;
#pragma unroll
  for (int i = t; i < 64 * kPerRow; i += kNormThreads) {
    const int rr = i / kPerRow, cc = (i % kPerRow) * L;
    const int r = r0 + rr, c = c0 + cc;
    const T* at = src + static_cast<long long>(r) * cols + c;
    float v[L];
    if (r < rows && c + L <= cols && (reinterpret_cast<uintptr_t>(at) & 15) == 0) {
      orth_unpack(*reinterpret_cast<const uint4*>(at), v);
    } else {
#pragma unroll
      for (int e = 0; e < L; ++e) v[e] = r < rows && c + e < cols ? orth_value(at + e) : 0.f;
    }
#pragma unroll
    for (int e = 0; e < L; ++e) tile[rr][cc + e] = v[e];
  }
  grid_dependency_wait();  // the sums of squares
  grid_dependents_launch();
  float inv;
  const float total = orth_total(blocks, part + m * kNormBlocks, red), up = orth_scale(rows, cols, total, eps, &inv);
  if (blockIdx.x == 0 && blockIdx.y == 0 && t == 0) orth_scales(steps, m, total, eps, inv);
  __half* hi = x.ptr + static_cast<size_t>(m) * x.rows * x.ld;
#pragma unroll
  for (int i = t; i < 64 * 32; i += kNormThreads) {  // pairs of columns of the operand
    const int rr = i >> 5, cc = 2 * (i & 31);
    const int r = (tall ? c0 : r0) + rr, c = (tall ? r0 : c0) + cc;
    if (r >= x.rows || c >= x.cols) continue;
    const float v0 = up * (tall ? tile[cc][rr] : tile[rr][cc]);
    const float v1 = up * (tall ? tile[cc + 1][rr] : tile[rr][cc + 1]);
    __half h0, l0, h1, l1;
    half_split(v0, &h0, &l0);
    half_split(v1, &h1, &l1);
    // the row padding (ld is even) takes the second value of an odd last column
    const size_t at = static_cast<size_t>(r) * x.ld + c;
    *reinterpret_cast<__half2*>(hi + at) = __halves2half2(h0, h1);
    if constexpr (kParts == 2) *reinterpret_cast<__half2*>(hi + x.lo + at) = __halves2half2(l0, l1);
  }
}

// ---------------------------------------------------------------------- the products
enum OrthOp : int { kGram = 0, kPoly = 1, kApply = 2 };

struct OrthArgs {
  int tiles_m, tiles_n, batch;  // kGram, kPoly: tiles_m = tiles_n, pairs m <= n only
  int b_groups;                 // matrix g of the first operand meets g mod b_groups of the second
  int num_kb;
  int M, N;                     // valid rows and columns of the result
  HalfMat prev;                 // added k0 times: kPoly: A; kApply: X (none where the matrix holds a I)
  HalfMat to;                   // the result, in operand form
  int symmetric;                // kPoly in two parts: exactly
  HalfMat also;                 // kPoly: 2^6 (a I + B) goes here, or NULL
  float diag;                   // 2^6 a
  // One part: what rounding took off the diagonal of 2^10 B [group][M]. B is near a multiple of
  // the identity where the singular values are alike, and its diagonal's errors then are too:
  // without them the whole update's error falls from 1.9e-3 to 1.1e-3 (400 x 8192).
  float* off;
  const float2 *scale, *next;   // orth_scales of X (kGram, kApply) and of X' (NULL: the caller's)
  float k0, k1;                 // see the epilogue
  void* out;                    // last kApply: the caller's matrix, else NULL
  int tall;
  unsigned* status;
};

template <int kPa, int kPb, int BN>
struct OrthShape {
  static constexpr uint32_t kA = kBM * 128, kB = BN * 128;  // one part's 64 values of K
  static constexpr uint32_t kStage = kPa * kA + kPb * kB;
};

__device__ __forceinline__ void umma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  umma_bf16(d, a, b, idesc, acc);  // kind::f16: the instruction descriptor names the type
}

// 32 consecutive values of a row of an operand. A lane's run is its own row's, so every access
// of a warp touches 32 rows: 32 bytes at a time halve their number.
__device__ __forceinline__ void ld_32(const void* p, uint32_t (&r)[16], int at) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[at]), "=r"(r[at + 1]), "=r"(r[at + 2]), "=r"(r[at + 3]), "=r"(r[at + 4]), "=r"(r[at + 5]),
                 "=r"(r[at + 6]), "=r"(r[at + 7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void st_32(void* p, const uint32_t (&r)[16], int at) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[at]), "r"(r[at + 1]),
               "r"(r[at + 2]), "r"(r[at + 3]), "r"(r[at + 4]), "r"(r[at + 5]), "r"(r[at + 6]), "r"(r[at + 7])
               : "memory");
}

template <int kParts>
struct HalfRun {
  uint32_t w[kParts][16];
  float off;
  // ld and the column are multiples of 32, so a row's padding is there to be read
  __device__ __forceinline__ void fetch(const HalfMat& x, size_t at) {
#pragma unroll
    for (int part = 0; part < kParts; ++part) {
      ld_32(x.ptr + part * x.lo + at, w[part], 0);
      ld_32(x.ptr + part * x.lo + at + 16, w[part], 8);
    }
  }
  __device__ __forceinline__ float2 pair(int i) const {  // values 2i and 2i + 1
    float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[0][i]));
    if constexpr (kParts == 2) {
      const float2 l = __half22float2(*reinterpret_cast<const __half2*>(&w[1][i]));
      f.x += l.x;
      f.y += l.y;
    }
    return f;
  }
};

// Columns past the matrix hold what the accumulator had there: zeros.
template <int kParts>
__device__ __forceinline__ void store_half_run(const HalfMat& x, size_t at, const float (&v)[32]) {
  uint32_t hi[16], lo[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    hi[i] = *reinterpret_cast<const uint32_t*>(&h);
    if constexpr (kParts == 2) {
      const float2 f = __half22float2(h);
      const __half2 l = __floats2half2_rn(v[2 * i] - f.x, v[2 * i + 1] - f.y);
      lo[i] = *reinterpret_cast<const uint32_t*>(&l);
    }
  }
  st_32(x.ptr + at, hi, 0);
  st_32(x.ptr + at + 16, hi, 8);
  if constexpr (kParts == 2) {
    st_32(x.ptr + x.lo + at, lo, 0);
    st_32(x.ptr + x.lo + at + 16, lo, 8);
  }
}

__device__ __forceinline__ void orth_store(float* p, float v) { *p = v; }
__device__ __forceinline__ void orth_store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// The matrix's scales in one: X = nu Xs, times the power of two of Xs'. Read before the products are
// waited for (beside X's values it took 3 us of the 120 at 1024 x 1024).
template <int kOp>
__device__ __forceinline__ float orth_nu(const OrthArgs& p, int g) {
  if constexpr (kOp == kPoly) return 1.f;
  const float nu = p.scale[g].x;
  return kOp == kApply && p.next ? nu * p.next[g].y : nu;
}

// What the epilogue reads of 32 columns from n of row m: kPoly A, kApply X.
template <int kParts, int kOp, bool kPrev>
__device__ __forceinline__ void orth_fetch(const OrthArgs& p, int g, int m, int n, HalfRun<kParts>& x) {
  if constexpr (kPrev) {
    if (m < p.M && n < p.N) {
      x.fetch(p.prev, static_cast<size_t>(g) * p.prev.rows * p.prev.ld + static_cast<size_t>(m) * p.prev.ld + n);
      if constexpr (kOp == kApply && kParts == 1) x.off = p.off[static_cast<size_t>(g) * p.M + m];
    }
  }
}

// 32 columns from n of row m of D:
//   kGram   2^12 A = k0 nu^2 D
//   kPoly   2^10 B = k0 (2^12 A) + k1 D
//   kApply  X' = k0 nu ((k1 + 2^-10 off) Xs + 2^-10 D), to Xs' or to the caller
// (nu with the power of two of Xs')
template <int kParts, int kOp, bool kPrev, class T>
__device__ __forceinline__ void orth_epilogue(const OrthArgs& p, int g, float nu, int m, int n, bool mirror,
                                              float (&v)[32], const HalfRun<kParts>& x, float* square) {
  if (m >= p.M || n >= p.N) return;
  const int k = min(32, p.N - n);
  const size_t base = static_cast<size_t>(g) * p.to.rows * p.to.ld, at = base + static_cast<size_t>(m) * p.to.ld + n;
  if constexpr (kOp == kGram) {
    const float f = p.k0 * nu * nu;
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= f;
  } else if constexpr (!kPrev) {
    const float f = p.k0 * nu;
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= f;
  } else {
    const float a = kOp == kApply && kParts == 1 ? p.k1 + x.off * (1.f / kScaleB) : p.k1;
    const float k0 = kOp == kPoly ? p.k0 : p.k0 * nu * a, k1 = kOp == kPoly ? p.k1 : p.k0 * nu * (1.f / kScaleB);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 f = x.pair(i);
      v[2 * i] = k0 * f.x + k1 * v[2 * i];
      v[2 * i + 1] = k0 * f.y + k1 * v[2 * i + 1];
    }
  }
  if constexpr (kOp == kApply) {
    if (p.out) {
      T* o = static_cast<T*>(p.out) + static_cast<size_t>(g) * p.M * p.N;
      if (p.tall) {  // lanes hold consecutive m: a store covers a run of one row
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i < k) orth_store(o + static_cast<size_t>(n + i) * p.M + m, v[i]);
      } else {
        T* row = o + static_cast<size_t>(m) * p.N + n;
        if (k == 32 && (reinterpret_cast<uintptr_t>(row) & 15) == 0) {
#pragma unroll
          for (int i = 0; i < 32; i += 16 / sizeof(T)) {
            if constexpr (sizeof(T) == 2)
              *reinterpret_cast<uint4*>(row + i) =
                  make_uint4(pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]),
                             pack_bf16x2(v[i + 4], v[i + 5]), pack_bf16x2(v[i + 6], v[i + 7]));
            else
              *reinterpret_cast<float4*>(row + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i < k) orth_store(row + i, v[i]);
        }
      }
      return;
    }
  }
  // Steps on the Gram matrix mirror the diagonal's tiles too, its squares of 32 x 32 by way of
  // shared memory (two-byte stores along the rows took 6 us): what little A and B do not
  // commute by would otherwise leave an antisymmetric part, which grows by a^2 a step.
  const int above = n - (m & ~31);
  if (kOp == kPoly && kParts == 2 && p.symmetric) {
    if (above < 0) return;  // its mirror image is written
    if (above == 0) {
      const int lane = m & 31, rows = p.M - m + lane;
      const unsigned lanes = rows < 32 ? (1u << rows) - 1 : 0xffffffffu;
#pragma unroll
      for (int i = 0; i < 32; ++i) square[lane * 33 + i] = v[i];
      __syncwarp(lanes);
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i < lane) v[i] = square[i * 33 + lane];
      __syncwarp(lanes);
    } else {
      mirror = true;
    }
  }
  if constexpr (kOp == kPoly && kParts == 1) {
    if (above == 0) {
      float d = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (n + i == m) d = v[i];
      p.off[static_cast<size_t>(g) * p.M + m] = d - __half2float(__float2half_rn(d));
    }
  }
  auto store = [&](const HalfMat& x) {
    store_half_run<kParts>(x, at, v);
    if constexpr (kOp != kApply) {
      if (mirror) {  // lanes hold consecutive m: each store covers a run of row n + i
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i < k) {
            const size_t to = base + static_cast<size_t>(n + i) * x.ld + m;
            __half hi, lo;
            half_split(v[i], &hi, &lo);
            x.ptr[to] = hi;
            if constexpr (kParts == 2) x.ptr[x.lo + to] = lo;
          }
      }
    }
  };
  store(p.to);
  if constexpr (kOp == kPoly && kParts == 2) {
    if (p.also.ptr) {  // rows and columns as p.to
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = v[i] * (kScaleQ / kScaleB) + (n + i == m ? p.diag : 0.f);
      store(p.also);
    }
  }
}

// D = A B^T (kGram, kPoly: both K-major rows) or A B (kApply: B's rows run along K), tiles of
// 128 x BN. kSplit CTAs of a cluster share a tile, each over its part of K, and exchange
// their partial sums through distributed shared memory, each finishing BN / kSplit columns;
// with kSplit = 1 the CTAs are persistent and the accumulator alternates between two
// buffers, so that one tile's epilogue runs under the next one's products.
//   warp 0 TMA, warp 1 MMA, warps 2-9 epilogue (two per lane quarter)
// Two parts (hi + lo): three products a step. A result in two parts is formed in slices of
// kSliceKb blocks of K that are added up in registers, because the accumulator truncates.
// One block of K where both operands have two parts (12 products on one accumulator; with two blocks
// the error of 150 x 700 was 3.4e-6 and is 1.9e-6, of 6 of 770 x 333 1.3e-6 and 0.9e-6, for 2.5% of the
// time), two where they have one.
template <int kPa, int kPb>
constexpr int kSliceKb = kPa == 2 && kPb == 2 ? 1 : 2;
constexpr int kOrthThreads = 64 + 8 * 32;
constexpr int kSquare = 32 * 33;

template <int kPa, int kPb, int BN>
struct OrthRing {
  static constexpr int kFit = (227 * 1024 - 2048) / OrthShape<kPa, kPb, BN>::kStage;
  static constexpr int kStages = kFit < 6 ? kFit : 6;
  // base to 1024 bytes, barriers, and a square for each epilogue warp (two-part results)
  static constexpr uint32_t kBytes = kStages * OrthShape<kPa, kPb, BN>::kStage + 2048 +
                                     (kPa == 2 && kPb == 2 ? 8 * kSquare * 4 : 0);
};

// kPa, kPb: parts of the operands; kParts: of the result and what is added to it.
template <int kPa, int kPb, int kParts, int BN, int kSplit, int kOp, class T>
__global__ void __launch_bounds__(kOrthThreads, 1)
    k_orth_gemm(const __grid_constant__ CUtensorMap a_hi, const __grid_constant__ CUtensorMap a_lo,
                const __grid_constant__ CUtensorMap b_hi, const __grid_constant__ CUtensorMap b_lo,
                const __grid_constant__ OrthArgs p) {
  using S = OrthShape<kPa, kPb, BN>;
  constexpr int kStages = OrthRing<kPa, kPb, BN>::kStages;
  constexpr bool kPairs = kOp != kApply;
  constexpr bool kSliced = kParts == 2;
  constexpr bool kPrev = kOp == kPoly || (kOp == kApply && kPa == kPb);
  constexpr uint32_t kCols = 2 * BN;  // two accumulators
  static_assert(kStages >= 2 && kCols <= 512, "two stages, two accumulators");
  constexpr int kOwn = (BN / 32 + kSplit - 1) / kSplit;  // chunk x of 32 columns belongs to rank x % kSplit
  static_assert(kSplit == 1 || (kSplit - 1) * kOwn * 32 * kBM * 4 <= kStages * S::kStage,
                "the ring holds the partial sums of the other CTAs");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * S::kStage);
  uint64_t *empty = full + kStages, *acc_full = empty + kStages, *acc_empty = acc_full + 2, *mma_done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kSplit > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < kStages; ++i) {
        mbar_init(&full[i], 1);
        mbar_init(&empty[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&acc_full[i], 1);
        mbar_init(&acc_empty[i], 8);
      }
      mbar_init(mma_done, 1);
      fence_barrier_init();
      tma_prefetch_map(&a_hi);
      tma_prefetch_map(&b_hi);
    }
    __syncwarp();
    tmem_alloc(tmem_slot, kCols);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependents_launch();

  const int per_matrix = kPairs ? p.tiles_m * (p.tiles_m + 1) / 2 : p.tiles_m * p.tiles_n;
  const int num_tiles = per_matrix * p.batch;
  const int tile0 = blockIdx.x / kSplit, tile_step = gridDim.x / kSplit;
  auto tile_at = [&](int t, int& g, int& m0, int& n0) {
    g = t / per_matrix;
    int r = t - g * per_matrix;
    if constexpr (kPairs) {  // pairs (i, j >= i), row by row
      int i = 0;
      while (r >= p.tiles_m - i) r -= p.tiles_m - i++;
      m0 = i * kBM;
      n0 = (i + r) * BN;
    } else {  // neighbours share the columns' panel of X
      m0 = (r % p.tiles_m) * kBM;
      n0 = (r / p.tiles_m) * BN;
    }
  };
  const int kb0 = p.num_kb * rank / kSplit, kb1 = p.num_kb * (rank + 1) / kSplit;

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ TMA producer
      grid_dependency_wait();
      int it = 0, issued = 0;
      bool ok = true;
      for (int t = tile0; ok && t < num_tiles; t += tile_step) {
        int g, m0, n0;
        tile_at(t, g, m0, n0);
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % kStages;
          if (!mbar_wait(&empty[s], ((it / kStages) & 1) ^ 1, p.status, kErrTimeoutProducer)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], S::kStage);
          uint8_t* base = smem + s * S::kStage;
#pragma unroll
          for (int part = 0; part < kPa; ++part)
            tma_load_3d(base + part * S::kA, part ? &a_lo : &a_hi, &full[s], kb * 64, m0, g);
          const int gb = g < p.b_groups ? g : g - p.b_groups;
#pragma unroll
          for (int part = 0; part < kPb; ++part) {
            const CUtensorMap* bm = part ? &b_lo : &b_hi;
            uint8_t* bt = base + kPa * S::kA + part * S::kB;
            if constexpr (kOp == kApply) {
#pragma unroll
              for (int c = 0; c < BN; c += 64) tma_load_3d(bt + c * 128, bm, &full[s], n0 + c, kb * 64, gb);
            } else {
              tma_load_3d(bt, bm, &full[s], kb * 64, n0, gb);
            }
          }
          issued = it + 1;
        }
      }
      for (int k = issued > kStages ? issued - kStages : 0; k < issued; ++k)
        mbar_wait(&full[k % kStages], (k / kStages) & 1, p.status, kErrTimeoutDrain);
    }
    if constexpr (kSplit > 1) {
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
  } else if (warp == 1) {
    // ------------------ MMA issuer: the whole warp in step (uniform addresses), one lane issues
    constexpr uint32_t idesc = umma_idesc(0, kBM, BN) | (kOp == kApply ? kIdescBMN : 0u);  // 0: float16
    const bool leader = elect_one();
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      const bool got = __all_sync(0xffffffffu, mbar_wait(bar, parity, p.status, kErrTimeoutMma));
      tc_fence_after();
      return got;
    };
    const uint32_t ring = smem_addr(smem);
    int unit = 0, s = 0;
    uint32_t ph = 0;  // of ring slot s
    bool ok = true;
    for (int t = tile0; ok && t < num_tiles; t += tile_step) {
      for (int kb = kb0; ok && kb < kb1; ++unit) {
        const int end = kSliced ? min(kb + kSliceKb<kPa, kPb>, kb1) : kb1;
        const int buf = unit & 1;
        ok = wait(&acc_empty[buf], ((unit >> 1) & 1) ^ 1);
        if (!ok) break;
        const uint32_t d = tmem + buf * BN;
        uint32_t acc = 0;
        for (; kb < end; ++kb) {
          ok = wait(&full[s], ph);
          if (!ok) break;
          if (leader) {
            const uint32_t at = ring + s * S::kStage;
            const uint64_t a = umma_desc_sw128(at);
            const uint64_t b = kOp == kApply ? umma_desc_sw128_mn(at + kPa * S::kA, 64 * 128)
                                             : umma_desc_sw128(at + kPa * S::kA);
            constexpr uint32_t kBStep = kOp == kApply ? 2048 >> 4 : 32 >> 4;
            auto product = [&](int pa, int pb) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                umma_f16(d, a + ((pa * S::kA) >> 4) + kk * (32 >> 4), b + ((pb * S::kB) >> 4) + kk * kBStep, idesc, acc);
                acc = 1;
              }
            };
            // the small products first
            if constexpr (kPa == 2) product(1, 0);
            if constexpr (kPb == 2) product(0, 1);
            product(0, 0);
            umma_commit(&empty[s]);
          }
          __syncwarp();
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (leader) umma_commit(&acc_full[buf]);  // also after a wait that gave up: the epilogue is released
        __syncwarp();
      }
    }
    if (leader) umma_commit(mma_done);
    __syncwarp();
    mbar_wait(mma_done, 0, p.status, kErrTimeoutDrain);
    if constexpr (kSplit > 1) {
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
  } else {
    // ------------------------------------------------------------------- epilogue
    const int q = warp & 3, part = (warp - 2) >> 2;
    const int row = q * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
    constexpr int kChunks = BN / 64;  // 32-column chunks of this warp: part, part + 2, ..
    // In slices the limit's two registers would cost more than they are worth (6 of 770 x 333: 151.8 us
    // against 150.7): these waits keep the default.
    const unsigned long long wl = kSliced ? kWaitLimitNs : first_wait_limit(p.status);
    grid_dependency_wait();
    int unit = 0;
    bool ok = true;
    auto wait_unit = [&]() {
      const bool got = __all_sync(0xffffffffu, mbar_wait(&acc_full[unit & 1], (unit >> 1) & 1, p.status,
                                                         kErrTimeoutEpilogue, wl));
      tc_fence_after();
      return got;
    };
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[unit & 1]);
      ++unit;
    };
    // the other ranks' sums land at [source][chunk][column][row]
    float* square = reinterpret_cast<float*>(smem + kStages * S::kStage + 1024) + (warp - 2) * kSquare;
    auto slot = [&](int src, int own) { return ((src * kOwn + own) * 32 * kBM + row) * 4; };
    for (int t = tile0; ok && t < num_tiles; t += tile_step) {
      int g, m0, n0;
      tile_at(t, g, m0, n0);
      const bool mirror = kPairs && n0 != m0;
      const float nu = orth_nu<kOp>(p, g);
      if constexpr (kSplit == 1 && !kSliced) {
        HalfRun<kParts> x;
        orth_fetch<kParts, kOp, kPrev>(p, g, m0 + row, n0 + part * 32, x);
        ok = wait_unit();
        if (!ok) break;
#pragma unroll 1
        for (int c = part * 32; c < BN; c += 64) {
          const HalfRun<kParts> now = x;
          if (c + 64 < BN) orth_fetch<kParts, kOp, kPrev>(p, g, m0 + row, n0 + c + 64, x);  // under this chunk's work
          float v[32];
          tmem_ld_32x32(lanes + (unit & 1) * BN + c, v);
          if (c + 64 >= BN) release();
          orth_epilogue<kParts, kOp, kPrev, T>(p, g, nu, m0 + row, n0 + c, mirror, v, now, square);
        }
      } else if constexpr (kSplit > 1 && !kSliced) {
        // straight from tensor memory, one chunk of 32 columns at a time
        static_assert(kChunks == 2, "a warp has the chunks part and part + 2");
        const bool any = kb1 > kb0;  // a share of no blocks: the accumulator was never written
        ok = !any || wait_unit();
        auto load = [&](int xc, float (&v)[32]) {
          if (any) {
            tmem_ld_32x32(lanes + (unit & 1) * BN + xc * 32, v);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.f;
          }
        };
        const int own0 = part % kSplit == rank ? part : (part + 2) % kSplit == rank ? part + 2 : -1;
        HalfRun<kParts> x;
        if (own0 >= 0) orth_fetch<kParts, kOp, kPrev>(p, g, m0 + row, n0 + own0 * 32, x);
        cluster_sync();  // every ring of the cluster is idle
        if (ok) {
#pragma unroll 1
          for (int xc = part; xc < BN / 32; xc += 2) {
            const int owner = xc % kSplit;
            if (owner == rank) continue;
            float v[32];
            load(xc, v);
            const uint32_t to = cluster_map(smem_addr(smem), owner) + slot(rank - (rank > owner), xc / kSplit);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + i * kBM * 4), "f"(v[i]) : "memory");
          }
        }
        cluster_sync();  // the others' sums of this CTA's columns have landed
        if (ok && own0 >= 0) {
#pragma unroll 1
          for (int xc = own0; xc < BN / 32; xc += 2) {
            if (xc % kSplit != rank) continue;
            if (xc != own0) orth_fetch<kParts, kOp, kPrev>(p, g, m0 + row, n0 + xc * 32, x);
            float v[32];
            load(xc, v);
#pragma unroll
            for (int src = 0; src < kSplit - 1; ++src) {
              const float* from = reinterpret_cast<const float*>(smem + slot(src, xc / kSplit));
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] += from[i * kBM];
            }
            orth_epilogue<kParts, kOp, kPrev, T>(p, g, nu, m0 + row, n0 + xc * 32, mirror, v, x, square);
          }
        }
      } else {
        HalfRun<kParts> x[kChunks];  // fetched under the products
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          if (kSplit == 1 || (2 * c + part) % kSplit == rank)
            orth_fetch<kParts, kOp, kPrev>(p, g, m0 + row, n0 + (2 * c + part) * 32, x[c]);
        float acc[kChunks][32];
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[c][i] = 0.f;
        constexpr int kSlice = kSliceKb<kPa, kPb>;
        const int slices = kSliced ? (kb1 - kb0 + kSlice - 1) / kSlice : (kb1 > kb0 ? 1 : 0);
        for (int sl = 0; sl < slices && ok; ++sl) {
          ok = wait_unit();
          if (!ok) break;
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            float v[32];
            tmem_ld_32x32(lanes + (unit & 1) * BN + (2 * c + part) * 32, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[c][i] += v[i];
          }
          release();
        }
        if constexpr (kSplit == 1) {
          if (ok) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
              orth_epilogue<kParts, kOp, kPrev, T>(p, g, nu, m0 + row, n0 + (2 * c + part) * 32, mirror, acc[c], x[c], square);
          }
        } else {
          cluster_sync();  // every ring of the cluster is idle
          if (ok) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              const int xc = 2 * c + part, owner = xc % kSplit;
              if (owner == rank) continue;
              const uint32_t to = cluster_map(smem_addr(smem), owner) + slot(rank - (rank > owner), xc / kSplit);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + i * kBM * 4), "f"(acc[c][i]) : "memory");
            }
          }
          cluster_sync();  // the others' sums of this CTA's columns have landed
          if (ok) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              const int xc = 2 * c + part;
              if (xc % kSplit != rank) continue;
#pragma unroll
              for (int src = 0; src < kSplit - 1; ++src) {
                const float* from = reinterpret_cast<const float*>(smem + slot(src, xc / kSplit));
#pragma unroll
                for (int i = 0; i < 32; ++i) acc[c][i] += from[i * kBM];
              }
              orth_epilogue<kParts, kOp, kPrev, T>(p, g, nu, m0 + row, n0 + xc * 32, mirror, acc[c], x[c], square);
            }
          }
        }
      }
    }
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

// --------------------------------------------------------------------------- launches
inline unsigned blocks_of(long long a, long long b) { return static_cast<unsigned>((a + b - 1) / b); }

template <int kPa, int kPb, int kParts, int BN, int kSplit, int kOp, class T>
pc_status_t launch_orth(const OrthArgs& p, const CUtensorMap (&a)[2], const CUtensorMap (&b)[2], cudaStream_t s,
                        long long tiles, long long flops) {
  constexpr uint32_t smem = OrthRing<kPa, kPb, BN>::kBytes;
  static_assert(smem <= 232448, "shared memory per CTA");
  constexpr auto kernel = k_orth_gemm<kPa, kPb, kParts, BN, kSplit, kOp, T>;
  PC_TRY(allow_smem<kernel>(static_cast<int>(smem)));
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kSplit;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(kSplit > 1 ? tiles * kSplit : (tiles < num_sms() ? tiles : num_sms())));
  cfg.blockDim = dim3(kOrthThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = kSplit > 1 ? 2 : 1;
  const int slot = profile_begin(s);
  PC_CUDA(cudaLaunchKernelEx(&cfg, kernel, a[0], a[1], b[0], b[1], p));
  PC_LAUNCH_CHECK();
  profile_end(slot, s, PC_KIND_ORTHOGONALIZE, flops);
  return PC_OK;
}

// CTAs of a cluster that share a tile of 128 x 128. A cluster lies within one of the GPU's
// eight groups of SMs, so at most 8 floor(SMs / 8 / size) clusters run at once. Sharing costs
// about 1 us (two cluster barriers and the exchange), five blocks of K (measured at 16
// blocks: 7.4 us a product alone, 7.1 shared by three; at 8: 5.8 against 6.4), so each CTA
// keeps at least as many; with two parts a block is three products.
inline int split_of(long long tiles, int num_kb, int products) {
  int best = 1;
  for (int size = 2; size <= 4; ++size)
    if (tiles <= 8 * (num_sms() / 8 / size) && products * num_kb >= 5 * size) best = size;
  return best;
}

template <int kPa, int kPb, int kParts, int kOp, class T>
pc_status_t run_product(OrthArgs p, const CUtensorMap (&a)[2], const CUtensorMap (&b)[2], cudaStream_t s,
                        long long flops) {
  p.tiles_m = static_cast<int>(blocks_of(p.M, kBM));
  const long long wide = static_cast<long long>(p.tiles_m) * blocks_of(p.N, 256) * p.batch;
  if constexpr (kOp == kApply && kPb == 1) {
    if (wide >= num_sms() || kPa == 2) {  // by_gram's matrices have the tiles
      p.tiles_n = static_cast<int>(blocks_of(p.N, 256));
      return launch_orth<kPa, kPb, kParts, 256, 1, kOp, T>(p, a, b, s, wide, flops);
    }
  }
  if constexpr (kPa == kPb) {
    p.tiles_n = static_cast<int>(blocks_of(p.N, 128));
    const long long tiles = (kOp == kApply ? p.tiles_m * static_cast<long long>(p.tiles_n)
                                           : p.tiles_m * (p.tiles_m + 1ll) / 2) * p.batch;
    const int split = split_of(tiles, p.num_kb, kPa == 2 ? 3 : 1);
    switch (split) {
      case 4: return launch_orth<kPa, kPb, kParts, 128, 4, kOp, T>(p, a, b, s, tiles, flops);
      case 3: return launch_orth<kPa, kPb, kParts, 128, 3, kOp, T>(p, a, b, s, tiles, flops);
      case 2: return launch_orth<kPa, kPb, kParts, 128, 2, kOp, T>(p, a, b, s, tiles, flops);
      default: return launch_orth<kPa, kPb, kParts, 128, 1, kOp, T>(p, a, b, s, tiles, flops);
    }
  }
  return PC_OK;
}

// Whether steps are taken on the Gram matrix (see the top). Five steps of it are 14 products of
// M x M matrices in two parts, about 12 us each up to M = 1024, for 4/5 of the gram and 7/10 of
// the apply products. Measured (us, X at every step against this): 512 x 8192 159, 165;
// 1024 x 2048 142, 206; 1024 x 8192 233, 234; 1024 x 16384 345, 277; 2048 x 8192 507, 595;
// 2048 x 16384 862, 715.
inline bool by_gram(long long batch, long long M, long long N, int parts) {
  M = round_up(M, kBM);
  return parts == 1 && N >= 8 * M && static_cast<double>(batch) * M * M * N >= 1.2e10;
}

struct OrthPlan {
  HalfMat X[2], A, Bm;
  HalfMat slots;  // by_gram: five stacks of M x M matrices in two parts, Bm likewise
  float *part, *off;
  float2* scales;
  size_t bytes;
};

// The workspace is 16-byte aligned, the operands' 32-byte accesses want more: its first
// 256-byte boundary is where the plan begins.
OrthPlan plan_orth(void* ws, int batch, int M, int N, int parts) {
  Carver c(reinterpret_cast<void*>(round_up(reinterpret_cast<intptr_t>(ws), 256)));
  OrthPlan p{};
  auto mat = [&](int rows, int cols, int of, int stacks) {
    HalfMat m;
    m.rows = rows;
    m.cols = cols;
    m.ld = round_up(cols, 64);
    const size_t n = static_cast<size_t>(batch) * stacks * rows * m.ld;
    m.lo = of == 2 ? n : 0;
    m.ptr = static_cast<__half*>(c.take(n * of * sizeof(__half)));
    return m;
  };
  p.part = static_cast<float*>(c.take(sizeof(float) * kNormBlocks * batch));
  p.scales = static_cast<float2*>(c.take(sizeof(float2) * batch * kMaxSteps));
  p.off = static_cast<float*>(c.take(sizeof(float) * batch * M));
  p.X[0] = mat(M, N, parts, 1);
  p.X[1] = mat(M, N, parts, 1);
  if (by_gram(batch, M, N, parts)) {
    p.slots = mat(M, M, 2, 5);
    p.Bm = mat(M, M, 2, 1);
    p.A = p.slots;
  } else {
    p.A = mat(M, M, parts, 1);
    p.Bm = mat(M, M, parts, 1);
  }
  p.bytes = c.used + 256 - 16;  // what the boundary may cost
  return p;
}

// Maps of an operand's parts: boxes of 64 columns (128 bytes) x box_rows.
pc_status_t half_maps(CUtensorMap (&map)[2], const HalfMat& x, int batch, int box_rows) {
  for (int part = 0; part < 2; ++part) {
    Operand o;
    o.ptr = x.ptr + (part ? x.lo : 0);
    o.rows = x.rows;
    o.cols = x.cols;
    o.ld = x.ld;
    o.groups = batch;
    PC_TRY(encode_operand_map(&map[part], o, kPrecF16Ops, box_rows, 0));
  }
  return PC_OK;
}

// Steps that are taken on one Gram matrix: Q, a product of polynomials whose largest value on
// the singular values is `growth`, has to fit float16 beside its scale.
inline int gram_steps(float a, float b, float c) {
  auto at = [&](float x) { return fabsf(a + x * (b + x * c)); };  // x: squared singular value, up to 1.5^2
  float growth = fmaxf(at(0.f), at(2.25f));
  if (c != 0.f && -b / (2.f * c) > 0.f && -b / (2.f * c) < 2.25f) growth = fmaxf(growth, at(-b / (2.f * c)));
  int n = 1;
  for (float g = growth * growth; g <= 512.f && n < 16; g *= growth) ++n;
  return n;
}

template <int kParts, class T>
pc_status_t iterate(const OrthPlan& p, int batch, int M, int N, int steps, float a, float b, float c, int tall, T* out,
                    cudaStream_t s) {
  CUtensorMap x_rows[2][2], x_cols[2][2], ma[2], mb[2];  // X as K-major rows, and as rows along K
  for (int i = 0; i < 2; ++i) {
    PC_TRY(half_maps(x_rows[i], p.X[i], batch, kBM));
    PC_TRY(half_maps(x_cols[i], p.X[i], batch, 64));
  }
  PC_TRY(half_maps(ma, p.A, batch, kBM));
  PC_TRY(half_maps(mb, p.Bm, batch, kBM));
  int bits = 0;  // 2^s ~ sqrt(N)
  while ((4ll << (2 * bits)) <= N) ++bits;
  const float up = static_cast<float>(1 << bits), down = 1.f / up;
  const long long mm = static_cast<long long>(batch) * M * M;
  const int m_kb = static_cast<int>(blocks_of(M, 64));
  OrthArgs square{};  // an M x M result
  square.batch = square.b_groups = batch;
  square.M = square.N = M;
  square.num_kb = m_kb;
  square.status = device_status_word();
  const int most = p.slots.ptr ? gram_steps(a, b, c) : 1;
  for (int it = 0, i = 0; it < steps; i ^= 1) {
    const int count = steps - it < most ? steps - it : most;
    const bool last = it + count == steps;
    OrthArgs gram = square;
    gram.num_kb = static_cast<int>(blocks_of(N, 64));
    gram.scale = p.scales + static_cast<size_t>(it) * batch;
    gram.k0 = kScaleA * (it == 0 ? 1.f : down * down);
    OrthArgs poly = square;
    poly.k0 = kScaleB / kScaleA * b;
    poly.k1 = kScaleB / (kScaleA * kScaleA) * c;
    OrthArgs apply = square;
    apply.N = N;
    apply.prev = p.X[i];
    apply.to = p.X[i ^ 1];
    apply.scale = gram.scale;
    apply.next = last ? nullptr : gram.scale + static_cast<size_t>(count) * batch;
    apply.k0 = (it == 0 ? 1.f : down) * (last ? 1.f : up);
    apply.k1 = a;
    apply.out = last ? out : nullptr;
    apply.tall = tall;
    it += count;
    if (count == 1) {
      gram.to = poly.prev = p.A;
      poly.to = p.Bm;
      poly.off = apply.off = p.off;
      PC_TRY((run_product<kParts, kParts, kParts, kGram, float>(gram, x_rows[i], x_rows[i], s, mm * N)));
      PC_TRY((run_product<kParts, kParts, kParts, kPoly, float>(poly, ma, ma, s, mm * M)));
      PC_TRY((run_product<kParts, kParts, kParts, kApply, T>(apply, mb, x_cols[i], s, 2 * mm * N)));
      continue;
    }
    if constexpr (kParts == 1) {
      // the slots hold A in 2, Q in 1 or 3, T in 4 or 0, so that (Q, A) or (A, Q) and the
      // pair that takes their products with P lie side by side
      CUtensorMap at[5][2];
      HalfMat slot[5];
      for (int k = 0; k < 5; ++k) {
        slot[k] = p.slots;
        slot[k].ptr += static_cast<size_t>(k) * batch * M * p.slots.ld;
        PC_TRY(half_maps(at[k], slot[k], k == 1 || k == 2 ? 2 * batch : batch, kBM));
      }
      gram.to = poly.prev = slot[2];
      PC_TRY((run_product<1, 1, 2, kGram, float>(gram, x_rows[i], x_rows[i], s, mm * N)));
      poly.symmetric = 1;
      int q = 1;
      for (int k = 0; k < count; ++k) {
        poly.to = p.Bm;
        poly.also = k == 0 ? slot[q] : HalfMat{};
        poly.diag = kScaleQ * a;
        PC_TRY((run_product<2, 2, 2, kPoly, float>(poly, at[2], at[2], s, mm * M)));
        // products with P: a times the operand and the operand times B
        auto times = [&](int from, int to, int stacks) {
          OrthArgs t = square;
          t.batch = stacks * batch;
          t.prev = slot[from];
          t.to = slot[to];
          t.symmetric = 1;
          t.k0 = a;
          t.k1 = 1.f / kScaleB;
          return run_product<2, 2, 2, kPoly, float>(t, at[from], mb, s, stacks * mm * M);
        };
        if (k + 1 == count) {
          if (k > 0) {
            PC_TRY(times(q, 4 - q, 1));
            q = 4 - q;
          }
          break;
        }
        const int t = k == 0 || q == 1 ? 4 : 0;
        if (k == 0) {
          PC_TRY(times(2, t, 1));
        } else {
          PC_TRY(times(q == 1 ? 1 : 2, q == 1 ? 3 : 0, 2));
          q = 4 - q;
        }
        PC_TRY(times(t, 2, 1));
      }
      apply.k0 *= 1.f / kScaleQ;
      PC_TRY((run_product<2, 1, 1, kApply, T>(apply, at[q], x_cols[i], s, 4 * mm * N)));
    }
  }
  return PC_OK;
}

template <int kParts, class T>
pc_status_t run_orth(int batch, int rows, int cols, const T* G, int steps, float a, float b, float c, float eps,
                     T* out, void* ws, cudaStream_t s) {
  const int tall = rows > cols;
  const int M = tall ? cols : rows, N = tall ? rows : cols;
  const OrthPlan p = plan_orth(ws, batch, M, N, kParts);
  const long long n = static_cast<long long>(rows) * cols;
  const bool vec = n % kPiece<T> == 0;
  const long long want = blocks_of(n, 2 * kNormThreads * (vec ? kPiece<T> : 1));
  const int blocks = static_cast<int>(want < kNormBlocks ? want : kNormBlocks);
  if (vec)
    k_orth_squares<T, true><<<dim3(blocks, batch), kNormThreads, 0, s>>>(n, G, p.part);
  else
    k_orth_squares<T, false><<<dim3(blocks, batch), kNormThreads, 0, s>>>(n, G, p.part);
  PC_LAUNCH_CHECK();
  {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kNormThreads);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const OrthSteps scaled{steps, batch, a, b, c, p.scales};
    if (!tall && cols % kPiece<T> == 0) {
      const long long want_load = blocks_of(n / kPiece<T>, 4 * kNormThreads), most = 4ll * num_sms();
      cfg.gridDim = dim3(static_cast<unsigned>(want_load < most ? want_load : most), batch);
      PC_CUDA(cudaLaunchKernelEx(&cfg, k_orth_load_rows<T, kParts>, rows, cols, G, blocks,
                                 static_cast<const float*>(p.part), eps, p.X[0], scaled));
    } else {
      cfg.gridDim = dim3(blocks_of(cols, 64), blocks_of(rows, 64), batch);
      PC_CUDA(cudaLaunchKernelEx(&cfg, k_orth_load<T, kParts>, rows, cols, G, blocks,
                                 static_cast<const float*>(p.part), eps, tall, p.X[0], scaled));
    }
    PC_LAUNCH_CHECK();
  }
  return iterate<kParts, T>(p, batch, M, N, steps, a, b, c, tall, out, s);
}

pc_status_t check_orth(int batch, int rows, int cols, int steps, pc_precision_t prec, pc_dtype_t dtype) {
  PC_TRY(check_precision(prec));
  PC_TRY(check_dtype(dtype));
  PC_CHECK(batch >= 0 && batch <= 65535, PC_ERR_SHAPE, "batch must be in [0, 65535] (got %d)", batch);
  PC_CHECK(rows >= 1 && cols >= 1, PC_ERR_SHAPE, "rows and columns must be >= 1 (got %d, %d)", rows, cols);
  PC_CHECK(rows <= (1 << 20) && cols <= (1 << 20), PC_ERR_SHAPE, "rows and columns up to 2^20 (got %d, %d)", rows, cols);
  const long long tiles = static_cast<long long>(blocks_of(rows, kBM)) * blocks_of(cols, kBM) * batch;
  PC_CHECK(tiles < (1ll << 29), PC_ERR_SHAPE, "batch * rows * cols too large (%d matrices of %d x %d)", batch, rows, cols);
  PC_CHECK(steps >= 1 && steps <= kMaxSteps, PC_ERR_SHAPE, "steps must be in [1, %d] (got %d)", kMaxSteps, steps);
  return PC_OK;
}

}  // namespace
}  // namespace pc

extern "C" {

pc_status_t pc_orthogonalize_workspace(int batch, int rows, int cols, pc_precision_t prec, size_t* bytes) {
  pc::clear_error();
  PC_CHECK(bytes, PC_ERR_NULL, "bytes must not be NULL");
  PC_TRY(pc::check_orth(batch, rows, cols, 1, prec, PC_F32));
  const int M = rows < cols ? rows : cols, N = rows < cols ? cols : rows;
  *bytes = pc::plan_orth(nullptr, batch, M, N, prec == PC_PREC_FP32 ? 2 : 1).bytes;
  return PC_OK;
}

pc_status_t pc_orthogonalize(int batch, int rows, int cols, const void* G, int steps, float a, float b, float c,
                             float eps, void* out, pc_dtype_t dtype, pc_precision_t prec, void* ws, size_t ws_bytes,
                             cudaStream_t stream) {
  pc::clear_error();
  PC_TRY(pc::check_orth(batch, rows, cols, steps, prec, dtype));
  PC_CHECK(eps >= 0.f, PC_ERR_SHAPE, "eps must not be negative (got %g)", static_cast<double>(eps));
  if (batch == 0) return PC_OK;
  PC_CHECK(G && out, PC_ERR_NULL, "G and out must not be NULL");
  PC_CHECK(pc::aligned16(G) && pc::aligned16(out), PC_ERR_ALIGNMENT, "G and out must be 16-byte aligned");
  size_t need = 0;
  PC_TRY(pc_orthogonalize_workspace(batch, rows, cols, prec, &need));
  PC_CHECK(ws && ws_bytes >= need, PC_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws_bytes, need);
  PC_CHECK(pc::aligned16(ws), PC_ERR_ALIGNMENT, "workspace is not 16-byte aligned");
  const bool two = prec == PC_PREC_FP32;
  using bf16 = __nv_bfloat16;
  if (dtype == PC_BF16) {
    const auto* g = static_cast<const bf16*>(G);
    auto* o = static_cast<bf16*>(out);
    return two ? pc::run_orth<2>(batch, rows, cols, g, steps, a, b, c, eps, o, ws, stream)
               : pc::run_orth<1>(batch, rows, cols, g, steps, a, b, c, eps, o, ws, stream);
  }
  const auto* g = static_cast<const float*>(G);
  auto* o = static_cast<float*>(out);
  return two ? pc::run_orth<2>(batch, rows, cols, g, steps, a, b, c, eps, o, ws, stream)
             : pc::run_orth<1>(batch, rows, cols, g, steps, a, b, c, eps, o, ws, stream);
}

}  // extern "C"

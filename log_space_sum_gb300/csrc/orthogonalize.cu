// Orthogonalised update: the nearest semi-orthogonal matrix direction of G by Newton-Schulz
// products. X_0 = G / (|G|_F + eps), transposed when G is taller than wide (so that X is
// M x N with M <= N), then `steps` times
//
//   A = X X^T,   B = b A + c A A,   X <- a X + B X.
//
// The polynomial a s + b s^3 + c s^5 acts on the singular values of X and drives them to
// one. Compute-bound from a few hundred rows on: M^2 N + M^3 + 2 M^2 N flops a step
// when the symmetric halves of A and A A are taken once.
//
// Every product runs on the tensor-core contraction with X and B in operand form; X is
// kept both as rows (A = X X^T) and transposed (the right operand of B X).
#include "pc_launch.cuh"

namespace pc {
namespace {

constexpr int kNormThreads = 256, kNormBlocks = 64;

__device__ __forceinline__ float orth_value(const float* p) { return *p; }
__device__ __forceinline__ float orth_value(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}

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

// part[g][block]: partial sums of squares, in an order that depends on the size alone.
template <class T>
__global__ void __launch_bounds__(kNormThreads) k_orth_squares(long long n, const T* __restrict__ g, float* part) {
  __shared__ float red[kNormThreads / 32];
  const T* p = g + static_cast<long long>(blockIdx.y) * n;
  float s = 0.f;
  for (long long i = blockIdx.x * static_cast<long long>(kNormThreads) + threadIdx.x; i < n;
       i += static_cast<long long>(gridDim.x) * kNormThreads) {
    const float v = orth_value(p + i);
    s += v * v;
  }
  s = block_total(s, red);
  if (threadIdx.x == 0) part[blockIdx.y * kNormBlocks + blockIdx.x] = s;
}

// inv[g] = 1 / (sqrt(sum of part[g]) + eps)
__global__ void k_orth_inverse(int blocks, const float* part, float eps, float* inv) {
  float s = 0.f;
  for (int i = threadIdx.x; i < blocks; i += 32) s += part[blockIdx.x * kNormBlocks + i];
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (threadIdx.x == 0) inv[blockIdx.x] = 1.f / (sqrtf(s) + eps);
}

// The operand writers of k_transpose64, scaled by inv[g].
template <int P>
struct ScaledStore {
  StoreOperand<P> st;
  const float* inv;
  __device__ void operator()(int g, int c, int r, const float (&v)[8], int n) const {
    const float k = inv[g];
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = v[i] * k;
    st(g, c, r, w, n);
  }
};
template <int P>
struct ScaledRows {
  StoreOperandRows<P> st;
  const float* inv;
  __device__ void operator()(int g, int r, int c, const float4& v, int n) const {
    const float k = inv[g];
    st(g, r, c, make_float4(v.x * k, v.y * k, v.z * k, v.w * k), n);
  }
};

// --------------------------------------------------------------------- epilogues
template <int P>
struct EpiOrthGram : EpiNoHooks {  // A = D
  struct Params {
    void* A;
    long long ld;
    size_t lo;
    int M;
  };
  __device__ static void apply(const Params& p, int g, int m0, int n0, int row, int col0, float (&v)[32], uint8_t*,
                               float*) {
    const int m = m0 + row, n = n0 + col0;
    if (m >= p.M || n >= p.M) return;
    const size_t idx = (static_cast<size_t>(g) * p.M + m) * p.ld + n;
    store_operand_run<P>(p.A, idx, p.lo, v, min(32, p.M - n));
  }
};

template <int P>
struct EpiOrthPoly : EpiNoHooks {  // B = b A + c D
  struct Params {
    const void* A;
    void* Bm;
    long long ld;
    size_t lo;
    int M;
    float b, c;
  };
  __device__ static void apply(const Params& p, int g, int m0, int n0, int row, int col0, float (&v)[32], uint8_t*,
                               float*) {
    const int m = m0 + row, n = n0 + col0;
    if (m >= p.M || n >= p.M) return;
    const size_t idx = (static_cast<size_t>(g) * p.M + m) * p.ld + n;
    const int k = min(32, p.M - n);
    float a[32];
    load_operand_run<P>(p.A, idx, p.lo, a, k);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = p.b * a[i] + p.c * v[i];
    store_operand_run<P>(p.Bm, idx, p.lo, v, k);
  }
};

__device__ __forceinline__ void orth_store(float* p, float v) { *p = v; }
__device__ __forceinline__ void orth_store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <int P, class T>
struct EpiOrthX : EpiNoHooks {  // X' = a X + D, as rows and transposed, or to the caller's matrix
  struct Params {
    const void* X;
    void *Y, *YT;  // NULL on the last step
    long long ld, ldt;
    size_t lo, lot;
    int M, N;
    float a;
    T* out;  // last step: [M][N], or [N][M] when tall
    int tall;
  };
  __device__ static void apply(const Params& p, int g, int m0, int n0, int row, int col0, float (&v)[32], uint8_t*,
                               float*) {
    const int m = m0 + row, n = n0 + col0;
    if (m >= p.M || n >= p.N) return;
    const size_t idx = (static_cast<size_t>(g) * p.M + m) * p.ld + n;
    const int k = min(32, p.N - n);
    float x[32];
    load_operand_run<P>(p.X, idx, p.lo, x, k);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] += p.a * x[i];
    if (p.out) {
      T* o = p.out + static_cast<size_t>(g) * p.M * p.N;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i < k)
          orth_store(o + (p.tall ? static_cast<size_t>(n + i) * p.M + m : static_cast<size_t>(m) * p.N + n + i), v[i]);
    } else {
      store_operand_run<P>(p.Y, idx, p.lo, v, k);
      // lanes hold consecutive m: each store covers one contiguous run of a row of X^T
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i < k) store_operand<P>(p.YT, (static_cast<size_t>(g) * p.N + n + i) * p.ldt + m, p.lot, v[i]);
    }
  }
};

struct OrthPlan {
  Operand X[2], XT[2], A, Bm;
  float *part, *inv;
  size_t bytes;
};

OrthPlan plan_orth(void* ws, int batch, int M, int N, pc_precision_t prec) {
  Carver c(ws);
  OrthPlan p;
  p.part = static_cast<float*>(c.take(sizeof(float) * kNormBlocks * batch));
  p.inv = static_cast<float*>(c.take(sizeof(float) * batch));
  for (int i = 0; i < 2; ++i) {
    p.X[i] = c.operand(prec, batch, M, N);
    p.XT[i] = c.operand(prec, batch, N, M);
  }
  p.A = c.operand(prec, batch, M, M);
  p.Bm = c.operand(prec, batch, M, M);
  p.bytes = c.used;
  return p;
}

// The products' precision: PC_PREC_AUTO takes TF32 operands.
pc_precision_t operand_precision(pc_precision_t prec) { return prec == PC_PREC_AUTO ? PC_PREC_TF32 : prec; }

template <int P, class T>
pc_status_t run_orth(int batch, int rows, int cols, const T* G, int steps, float a, float b, float c, float eps,
                     T* out, pc_precision_t prec, void* ws, cudaStream_t s) {
  using Src = typename std::conditional<sizeof(T) == 2, uint16_t, float>::type;
  const int tall = rows > cols;
  const int M = tall ? cols : rows, N = tall ? rows : cols;
  const OrthPlan p = plan_orth(ws, batch, M, N, prec);
  const Src* src = reinterpret_cast<const Src*>(G);
  const long long n = static_cast<long long>(rows) * cols;
  const int blocks = static_cast<int>(cdiv(n, 4 * kNormThreads) < kNormBlocks ? cdiv(n, 4 * kNormThreads) : kNormBlocks);
  k_orth_squares<Src><<<dim3(blocks, batch), kNormThreads, 0, s>>>(n, src, p.part);
  PC_LAUNCH_CHECK();
  k_orth_inverse<<<batch, 32, 0, s>>>(blocks, p.part, eps, p.inv);
  PC_LAUNCH_CHECK();
  const Operand &same = tall ? p.XT[0] : p.X[0], &turned = tall ? p.X[0] : p.XT[0];
  k_transpose64<ScaledStore<P>, ScaledRows<P>, Src><<<dim3(cdiv(cols, 64), cdiv(rows, 64), batch), 256, 0, s>>>(
      src, cols, n, rows, cols, nullptr,
      ScaledStore<P>{{turned.ptr, turned.ld, turned.lo_elems, static_cast<long long>(cols)}, p.inv},
      ScaledRows<P>{{same.ptr, same.ld, same.lo_elems, static_cast<long long>(rows)}, p.inv});
  PC_LAUNCH_CHECK();
  constexpr int BN = 128;
  OperandMaps mX[2], mXT[2], mA, mB;
  for (int i = 0; i < 2; ++i) {
    PC_TRY(encode_maps(&mX[i], p.X[i], prec, 128));
    PC_TRY(encode_maps(&mXT[i], p.XT[i], prec, 128));
  }
  PC_TRY(encode_maps(&mA, p.A, prec, 128));
  PC_TRY(encode_maps(&mB, p.Bm, prec, 128));
  const dim3 square(cdiv(M, 128), cdiv(M, BN), batch), wide(cdiv(M, 128), cdiv(N, BN), batch);
  const long long mm = static_cast<long long>(batch) * M * M;
  for (int it = 0; it < steps; ++it) {
    const int i = it & 1;
    const bool last = it + 1 == steps;
    PC_TRY((launch_gemm<P, BN, EpiOrthGram<P>>(square, mX[i].hi, mX[i].lo, mX[i].hi, mX[i].lo, num_k_blocks(N, prec),
                                               {p.A.ptr, p.A.ld, p.A.lo_elems, M}, s, PC_KIND_ORTHOGONALIZE,
                                               2 * mm * N)));
    PC_TRY((launch_gemm<P, BN, EpiOrthPoly<P>>(square, mA.hi, mA.lo, mA.hi, mA.lo, num_k_blocks(M, prec),
                                               {p.A.ptr, p.Bm.ptr, p.A.ld, p.A.lo_elems, M, b, c}, s,
                                               PC_KIND_ORTHOGONALIZE, 2 * mm * M)));
    PC_TRY((launch_gemm<P, BN, EpiOrthX<P, T>>(
        wide, mB.hi, mB.lo, mXT[i].hi, mXT[i].lo, num_k_blocks(M, prec),
        {p.X[i].ptr, p.X[i ^ 1].ptr, p.XT[i ^ 1].ptr, p.X[i].ld, p.XT[i].ld, p.X[i].lo_elems, p.XT[i].lo_elems, M, N,
         a, last ? out : nullptr, tall},
        s, PC_KIND_ORTHOGONALIZE, 2 * mm * N)));
  }
  return PC_OK;
}

pc_status_t check_orth(int batch, int rows, int cols, int steps, pc_precision_t prec, pc_dtype_t dtype) {
  PC_TRY(check_precision(prec));
  PC_TRY(check_dtype(dtype));
  PC_CHECK(batch >= 0 && batch <= 65535, PC_ERR_SHAPE, "batch must be in [0, 65535] (got %d)", batch);
  PC_CHECK(rows >= 1 && cols >= 1, PC_ERR_SHAPE, "rows and columns must be >= 1 (got %d, %d)", rows, cols);
  PC_CHECK(rows <= (1 << 20) && cols <= (1 << 20), PC_ERR_SHAPE, "rows and columns up to 2^20 (got %d, %d)", rows, cols);
  PC_CHECK(steps >= 1 && steps <= 100, PC_ERR_SHAPE, "steps must be in [1, 100] (got %d)", steps);
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
  *bytes = pc::plan_orth(nullptr, batch, M, N, pc::operand_precision(prec)).bytes;
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
  const pc_precision_t op = pc::operand_precision(prec);
  using bf16 = __nv_bfloat16;
  if (dtype == PC_BF16) {
    const auto* g = static_cast<const bf16*>(G);
    auto* o = static_cast<bf16*>(out);
    return op == PC_PREC_FP32 ? pc::run_orth<pc::kTF32x3>(batch, rows, cols, g, steps, a, b, c, eps, o, op, ws, stream)
                              : pc::run_orth<pc::kTF32>(batch, rows, cols, g, steps, a, b, c, eps, o, op, ws, stream);
  }
  const auto* g = static_cast<const float*>(G);
  auto* o = static_cast<float*>(out);
  return op == PC_PREC_FP32 ? pc::run_orth<pc::kTF32x3>(batch, rows, cols, g, steps, a, b, c, eps, o, op, ws, stream)
                            : pc::run_orth<pc::kTF32>(batch, rows, cols, g, steps, a, b, c, eps, o, op, ws, stream);
}

}  // extern "C"

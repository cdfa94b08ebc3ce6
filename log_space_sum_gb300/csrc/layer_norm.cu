// Layer norm of rows, forward and backward.
//
//   forward   mean = avg(x), rstd = (avg((x - mean)^2) + eps)^(-1/2), z = (x - mean) rstd,
//             y = z w + b
//   backward  g = dy w,  dx = rstd (g - avg(g) - z avg(g z)),
//             dw = sum over rows of dy z,  db = sum over rows of dy
//
// Memory-bound: x (and dy) are read once and y (dx) written once, about ten flops per
// element. A row lives in the registers of one warp or one CTA between its load and its
// store, so the variance is that of the centred values (no cancellation) at no extra
// traffic. Measured, bf16: forward 32768 x 4096 98 us (5.5 TB/s), gradient 32768 x 1024 37 us on the
// GPU (34 and 5.9 TB/s without the weight's sums). Statistics, sums and the weight's gradients are float32 throughout; the only
// rounding to bf16 is that of y and dx.
#include "pc_device.cuh"
#include "pc_host.h"

namespace pc {
namespace {

template <class T>
constexpr int kLanes = 16 / sizeof(T);  // values of one 16-byte access

__device__ __forceinline__ void unpack(const uint4& u, float (&v)[8]) {  // bf16 x 8
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack(const uint4& u, float (&v)[4]) {
  v[0] = __uint_as_float(u.x);
  v[1] = __uint_as_float(u.y);
  v[2] = __uint_as_float(u.z);
  v[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ uint4 pack(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ uint4 pack(const float (&v)[4]) {
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_float(float v, float* p) { *p = v; }
__device__ __forceinline__ void from_float(float v, __nv_bfloat16* p) { *p = __float2bfloat16_rn(v); }

// kLanes<T> float32 parameters starting at column c (16-byte aligned: c is a multiple of 4).
template <int L>
__device__ __forceinline__ void load_params(const float* p, int c, float (&v)[L]) {
#pragma unroll
  for (int i = 0; i < L; i += 4) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(p + c + i));
    v[i] = f.x;
    v[i + 1] = f.y;
    v[i + 2] = f.z;
    v[i + 3] = f.w;
  }
}

// Sum of a and b over the kWarps warps that share a row (every thread receives both).
// red: kWarps float2 of shared memory per call site, not reused before the next barrier.
template <int kWarps>
__device__ __forceinline__ float2 row_sum(float a, float b, float2* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if constexpr (kWarps > 1) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      a += red[w].x;
      b += red[w].y;
    }
  }
  return make_float2(a, b);
}

// Rows that do not start on 16 bytes, or do not end there (kEdges): the pieces are those of
// memory, and a row's first and last one hold its neighbours' values too. Every piece holds at
// least one value of the row. Rows whose distance is a multiple of kLanes<T> rows start at the
// same place in a piece, so a CTA that walks by such a distance keeps its columns, and the
// parameters that belong to them in registers.
template <class T>
__device__ __forceinline__ int row_shift(const T* row) {  // values of the first piece before the row
  return static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
}
// Bits of a piece from column c that are the row's.
template <class T>
__device__ __forceinline__ uint4 piece_mask(int c, int dim) {
  constexpr int kWord = 4 / sizeof(T);
  uint32_t m[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < kLanes<T>; ++j)
    if (c + j >= 0 && c + j < dim) m[j / kWord] |= (kWord == 2 ? 0xFFFFu : 0xFFFFFFFFu) << (j % kWord * 16);
  return make_uint4(m[0], m[1], m[2], m[3]);
}
__device__ __forceinline__ uint4 masked(const uint4& v, const uint4& m) {
  return make_uint4(v.x & m.x, v.y & m.y, v.z & m.z, v.w & m.w);
}
template <bool kEdges, int L>
__device__ __forceinline__ void params_at(const float* p, int c, int dim, float (&v)[L]) {
  if constexpr (kEdges) {
#pragma unroll
    for (int j = 0; j < L; ++j)
      if (c + j >= 0 && c + j < dim) v[j] = __ldg(p + c + j);
  } else {
    load_params<L>(p, c, v);
  }
}
template <bool kEdges, class T, int L>
__device__ __forceinline__ void store_piece(T* row, int c, int dim, const float (&v)[L]) {
  if (kEdges && (c < 0 || c + L > dim)) {
#pragma unroll
    for (int j = 0; j < L; ++j)
      if (c + j >= 0 && c + j < dim) from_float(v[j], row + c + j);
  } else {
    __stcs(reinterpret_cast<uint4*>(row + c), pack(v));
  }
}

// ------------------------------------------------------------------------ forward
// kWarps = 1: a warp per row, kRows rows per CTA; kWarps > 1: a CTA per row. A thread
// holds kVecs 16-byte pieces of its row (piece i at (i * threads + t)). A CTA per row and no
// loop over rows: CTAs that stay and fetch ahead (as below for rows with edges) were slower (32768 rows
// of 4096 bf16 values: 98.7 us against 96.8, float32 230 against 152; of 1024 bf16: 27.5 against
// 26.2), and so were more threads per row (128 us with 256 threads, 177 with 512).
template <class T, int kWarps, int kVecs, int kRows>
__global__ void __launch_bounds__(32 * kWarps * kRows)
    k_ln_fwd(long long rows, int dim, const T* __restrict__ x, long long x_ld, const float* __restrict__ w,
             const float* __restrict__ b, float eps, T* __restrict__ y, long long y_ld, float* __restrict__ mean,
             float* __restrict__ rstd) {
  constexpr int L = kLanes<T>, kThreads = 32 * kWarps;
  static_assert(kWarps == 1 || kRows == 1, "a warp's row or a CTA's row");
  __shared__ float2 red[2][kWarps];
  const int t = kWarps == 1 ? (threadIdx.x & 31) : threadIdx.x;
  const long long r = static_cast<long long>(blockIdx.x) * kRows + (kWarps == 1 ? threadIdx.x >> 5 : 0);
  if (r >= rows) return;
  const T* xr = x + r * x_ld;
  uint4 raw[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = (i * kThreads + t) * L;
    raw[i] = c < dim ? __ldcs(reinterpret_cast<const uint4*>(xr + c)) : make_uint4(0u, 0u, 0u, 0u);
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    float v[L];
    unpack(raw[i], v);
#pragma unroll
    for (int j = 0; j < L; ++j) s += v[j];
  }
  const float m = row_sum<kWarps>(s, 0.f, red[0]).x / dim;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    float v[L];
    unpack(raw[i], v);
    if ((i * kThreads + t) * L < dim) {
#pragma unroll
      for (int j = 0; j < L; ++j) s += (v[j] - m) * (v[j] - m);
    }
  }
  const float rs = 1.f / sqrtf(row_sum<kWarps>(s, 0.f, red[1]).x / dim + eps);
  if (t == 0) {
    if (mean) mean[r] = m;
    if (rstd) rstd[r] = rs;
  }
  T* yr = y + r * y_ld;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = (i * kThreads + t) * L;
    if (c < dim) {
      float v[L], g[L];
      unpack(raw[i], v);
#pragma unroll
      for (int j = 0; j < L; ++j) v[j] = (v[j] - m) * rs;
      if (w) {
        load_params<L>(w, c, g);
#pragma unroll
        for (int j = 0; j < L; ++j) v[j] *= g[j];
      }
      if (b) {
        load_params<L>(b, c, g);
#pragma unroll
        for (int j = 0; j < L; ++j) v[j] += g[j];
      }
      __stcs(reinterpret_cast<uint4*>(yr + c), pack(v));
    }
  }
}

// The forward of rows with edges: a CTA walks rows gridDim.x (a multiple of kLanes<T>) apart,
// one at a time with the next on its way, its parameters in registers (a CTA for each row would
// read them a value at a time: 55 us for 16384 rows of 1537 bf16 values against 28).
template <class T, int kWarps, int kVecs, int kCtas>
__global__ void __launch_bounds__(32 * kWarps, kCtas)
    k_ln_fwd_edges(long long rows, int dim, const T* __restrict__ x, long long x_ld, const float* __restrict__ w,
                   const float* __restrict__ b, float eps, T* __restrict__ y, long long y_ld,
                   float* __restrict__ mean, float* __restrict__ rstd) {
  constexpr int L = kLanes<T>, kThreads = 32 * kWarps;
  __shared__ float2 red[2][kWarps];
  __shared__ uint4 inside[kVecs][kThreads];
  const int t = threadIdx.x;
  const int shift = row_shift(x + blockIdx.x * x_ld);
  float wv[kVecs][L], bv[kVecs][L];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = (i * kThreads + t) * L - shift;
#pragma unroll
    for (int j = 0; j < L; ++j) {
      wv[i][j] = 1.f;
      bv[i][j] = 0.f;
    }
    if (w && c < dim) params_at<true, L>(w, c, dim, wv[i]);
    if (b && c < dim) params_at<true, L>(b, c, dim, bv[i]);
    inside[i][t] = piece_mask<T>(c, dim);  // read by this thread alone
  }
  uint4 raw[kVecs], next[kVecs];
  auto fetch = [&](long long r) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int c = (i * kThreads + t) * L - shift;
      next[i] = c < dim && r < rows ? __ldcs(reinterpret_cast<const uint4*>(x + r * x_ld + c)) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  fetch(blockIdx.x);
  for (long long r = blockIdx.x; r < rows; r += gridDim.x) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) raw[i] = masked(next[i], inside[i][t]);
    fetch(r + gridDim.x);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      float v[L];
      unpack(raw[i], v);
#pragma unroll
      for (int j = 0; j < L; ++j) s += v[j];
    }
    const float m = row_sum<kWarps>(s, 0.f, red[0]).x / dim;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int c = (i * kThreads + t) * L - shift;
      float v[L];
      unpack(raw[i], v);
      if (c >= 0 && c + L <= dim) {
#pragma unroll
        for (int j = 0; j < L; ++j) s += (v[j] - m) * (v[j] - m);
      } else {
#pragma unroll
        for (int j = 0; j < L; ++j)
          if (c + j >= 0 && c + j < dim) s += (v[j] - m) * (v[j] - m);
      }
    }
    const float rs = 1.f / sqrtf(row_sum<kWarps>(s, 0.f, red[1]).x / dim + eps);
    if (t == 0) {
      if (mean) mean[r] = m;
      if (rstd) rstd[r] = rs;
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int c = (i * kThreads + t) * L - shift;
      if (c < dim) {
        float v[L];
        unpack(raw[i], v);
#pragma unroll
        for (int j = 0; j < L; ++j) v[j] = (v[j] - m) * rs * wv[i][j] + bv[i][j];
        store_piece<true>(y + r * y_ld, c, dim, v);
      }
    }
  }
}

constexpr int kAnyThreads = 256;

// Any row: input and output placed differently, or longer than the registers hold.
// A CTA per row; rows of up to kCols * 256 values are loaded once, longer ones (kCols = 0)
// are read three times (L1 and L2 serve the second and third).
template <class T, int kCols>
__global__ void __launch_bounds__(kAnyThreads)
    k_ln_fwd_any(int dim, const T* __restrict__ x, long long x_ld, const float* __restrict__ w,
                 const float* __restrict__ b, float eps, T* __restrict__ y, long long y_ld, float* __restrict__ mean,
                 float* __restrict__ rstd) {
  __shared__ float2 red[2][kAnyThreads / 32];
  const long long r = blockIdx.x;
  const T* xr = x + r * x_ld;
  T* yr = y + r * y_ld;
  float v[kCols > 0 ? kCols : 1];
  float s = 0.f;
  if constexpr (kCols > 0) {
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      const int c = i * kAnyThreads + threadIdx.x;
      v[i] = c < dim ? to_float(xr[c]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kCols; ++i) s += v[i];
  } else {
    for (int c = threadIdx.x; c < dim; c += kAnyThreads) s += to_float(xr[c]);
  }
  const float m = row_sum<kAnyThreads / 32>(s, 0.f, red[0]).x / dim;
  s = 0.f;
  if constexpr (kCols > 0) {
#pragma unroll
    for (int i = 0; i < kCols; ++i)
      if (i * kAnyThreads + threadIdx.x < dim) s += (v[i] - m) * (v[i] - m);
  } else {
    for (int c = threadIdx.x; c < dim; c += kAnyThreads) {
      const float d = to_float(xr[c]) - m;
      s += d * d;
    }
  }
  const float rs = 1.f / sqrtf(row_sum<kAnyThreads / 32>(s, 0.f, red[1]).x / dim + eps);
  if (threadIdx.x == 0) {
    if (mean) mean[r] = m;
    if (rstd) rstd[r] = rs;
  }
  auto put = [&](int c, float value) {
    float z = (value - m) * rs;
    if (w) z *= w[c];
    if (b) z += b[c];
    from_float(z, yr + c);
  };
  if constexpr (kCols > 0) {
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      const int c = i * kAnyThreads + threadIdx.x;
      if (c < dim) put(c, v[i]);
    }
  } else {
    for (int c = threadIdx.x; c < dim; c += kAnyThreads) put(c, to_float(xr[c]));
  }
}

// ----------------------------------------------------------------------- backward
// A CTA is kGroups groups of kWarps warps; a group walks rows, one at a time with the next on
// its way. A thread keeps its columns' sums of dy z and dy in registers over all its rows; the
// groups' are added up in shared memory and written as one row of the partial sums
// part[2][gridDim.x][dim] (k_ln_reduce adds those rows). Every order is fixed.
template <class T, int kWarps, int kVecs, int kGroups, int kCtas, bool kEdges>
__global__ void __launch_bounds__(32 * kWarps * kGroups, kCtas)
    k_ln_bwd(long long rows, int dim, const T* __restrict__ dy, long long dy_ld, const T* __restrict__ x,
             long long x_ld, const float* __restrict__ w, const float* __restrict__ mean,
             const float* __restrict__ rstd, T* __restrict__ dx, long long dx_ld, float* __restrict__ part) {
  constexpr int L = kLanes<T>, kThreads = 32 * kWarps;
  grid_dependents_launch();
  __shared__ float2 red[2][kGroups][kWarps];
  constexpr int kPitch = kThreads + 4;  // of value j of every thread's piece
  __shared__ float sums[kGroups > 1 ? 2 : 1][kGroups > 1 ? kPitch * kVecs * L : 1];
  __shared__ uint4 inside[kEdges ? kVecs : 1][kEdges ? kThreads : 1];  // the same for every group
  const int group = threadIdx.x / kThreads, t = threadIdx.x % kThreads;
  const long long first = blockIdx.x + static_cast<long long>(group) * gridDim.x;  // a CTA's shifts are alike
  const long long stride = static_cast<long long>(gridDim.x) * kGroups;
  const int shift = kEdges ? row_shift(x + first * x_ld) : 0;
  float wv[kVecs][L], aw[kVecs][L], ab[kVecs][L];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = (i * kThreads + t) * L - shift;
#pragma unroll
    for (int j = 0; j < L; ++j) {
      aw[i][j] = ab[i][j] = 0.f;
      wv[i][j] = 1.f;
    }
    if (w && c < dim) params_at<kEdges, L>(w, c, dim, wv[i]);
    if (kEdges && group == 0) inside[i][t] = piece_mask<T>(c, dim);
  }
  if constexpr (kEdges) __syncthreads();
  int flip = 0;
  uint4 rx[kVecs], rd[kVecs], nx[kVecs], nd[kVecs];
  auto fetch = [&](long long r) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int c = (i * kThreads + t) * L - shift;
      const bool in = c < dim && r < rows;
      nx[i] = in ? __ldcs(reinterpret_cast<const uint4*>(x + r * x_ld + c)) : make_uint4(0u, 0u, 0u, 0u);
      nd[i] = in ? __ldcs(reinterpret_cast<const uint4*>(dy + r * dy_ld + c)) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  fetch(first);
  for (long long r = first; r < rows; r += stride, flip ^= 1) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      if constexpr (kEdges) {
        const uint4 m = inside[i][t];
        rx[i] = masked(nx[i], m);
        rd[i] = masked(nd[i], m);
      } else {
        rx[i] = nx[i];
        rd[i] = nd[i];
      }
    }
    fetch(r + stride);
    const float m = mean[r], rs = rstd[r];
    float sg = 0.f, sz = 0.f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      float xv[L], dv[L];
      unpack(rx[i], xv);
      unpack(rd[i], dv);
#pragma unroll
      for (int j = 0; j < L; ++j) {  // past dim: dy = 0 adds nothing
        const float z = (xv[j] - m) * rs, g = dv[j] * wv[i][j];
        aw[i][j] += dv[j] * z;
        ab[i][j] += dv[j];
        sg += g;
        sz += g * z;
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      sg += __shfl_xor_sync(0xffffffffu, sg, o);
      sz += __shfl_xor_sync(0xffffffffu, sz, o);
    }
    if constexpr (kWarps > 1) {
      if ((t & 31) == 0) red[flip][group][t >> 5] = make_float2(sg, sz);
      // the group's own barrier; the other copy of red is rewritten only after the next one
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kThreads) : "memory");
      sg = sz = 0.f;
#pragma unroll
      for (int q = 0; q < kWarps; ++q) {
        sg += red[flip][group][q].x;
        sz += red[flip][group][q].y;
      }
    }
    const float mg = sg / dim, mz = sz / dim;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int c = (i * kThreads + t) * L - shift;
      if (c < dim) {
        float xv[L], dv[L];
        unpack(rx[i], xv);
        unpack(rd[i], dv);
#pragma unroll
        for (int j = 0; j < L; ++j) dv[j] = rs * (dv[j] * wv[i][j] - mg - (xv[j] - m) * rs * mz);
        store_piece<kEdges>(dx + r * dx_ld, c, dim, dv);
      }
    }
  }
  if (!part) return;
  float* pw = part + static_cast<long long>(blockIdx.x) * dim;
  float* pb = pw + static_cast<long long>(gridDim.x) * dim;
  if constexpr (kGroups == 1) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int c = (i * kThreads + t) * L - shift;
      if (c < dim) {
#pragma unroll
        for (int j = 0; kEdges && j < L; ++j)
          if (c + j >= 0 && c + j < dim) {
            pw[c + j] = aw[i][j];
            pb[c + j] = ab[i][j];
          }
#pragma unroll
        for (int j = 0; !kEdges && j < L; j += 4) {
          *reinterpret_cast<float4*>(pw + c + j) = make_float4(aw[i][j], aw[i][j + 1], aw[i][j + 2], aw[i][j + 3]);
          *reinterpret_cast<float4*>(pb + c + j) = make_float4(ab[i][j], ab[i][j + 1], ab[i][j + 2], ab[i][j + 3]);
        }
      }
    }
  } else {
    for (int g = 0; g < kGroups; ++g) {  // the groups in turn
      if (group == g) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
          for (int j = 0; j < L; ++j) {
            const int at = (i * L + j) * kPitch + t;
            sums[0][at] = g ? sums[0][at] + aw[i][j] : aw[i][j];
            sums[1][at] = g ? sums[1][at] + ab[i][j] : ab[i][j];
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < dim; c += kThreads * kGroups) {
      const int piece = (c + shift) / L, at = (piece / kThreads * L + (c + shift) % L) * kPitch + piece % kThreads;
      pw[c] = sums[0][at];
      pb[c] = sums[1][at];
    }
  }
}

// Any row length and alignment, a CTA per row at a time. Rows of up to kCols * 256 values
// live in registers as above, loaded one value at a time (consecutive lanes, consecutive
// addresses); for longer ones (kCols = 0) the row is read twice and the columns' sums live
// in the CTA's own row of `part` (each column is one thread's: no atomics).
template <class T, int kCols>
__global__ void __launch_bounds__(kAnyThreads)
    k_ln_bwd_any(long long rows, int dim, const T* __restrict__ dy, long long dy_ld, const T* __restrict__ x,
                 long long x_ld, const float* __restrict__ w, const float* __restrict__ mean,
                 const float* __restrict__ rstd, T* __restrict__ dx, long long dx_ld, float* part) {
  grid_dependents_launch();
  __shared__ float2 red[2][kAnyThreads / 32];
  float* pw = part ? part + static_cast<long long>(blockIdx.x) * dim : nullptr;
  float* pb = part ? pw + static_cast<long long>(gridDim.x) * dim : nullptr;
  int flip = 0;
  if constexpr (kCols > 0) {
    float wv[kCols], aw[kCols], ab[kCols];
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      const int c = i * kAnyThreads + threadIdx.x;
      aw[i] = ab[i] = 0.f;
      wv[i] = w && c < dim ? w[c] : 1.f;
    }
    for (long long r = blockIdx.x; r < rows; r += gridDim.x, flip ^= 1) {
      const T *xr = x + r * x_ld, *dr = dy + r * dy_ld;
      float z[kCols], g[kCols];
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const int c = i * kAnyThreads + threadIdx.x;
        z[i] = c < dim ? to_float(xr[c]) : 0.f;
        g[i] = c < dim ? to_float(dr[c]) : 0.f;
      }
      const float m = mean[r], rs = rstd[r];
      float sg = 0.f, sz = 0.f;
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        z[i] = (z[i] - m) * rs;
        aw[i] += g[i] * z[i];
        ab[i] += g[i];
        g[i] *= wv[i];
        sg += g[i];
        sz += g[i] * z[i];
      }
      const float2 sums = row_sum<kAnyThreads / 32>(sg, sz, red[flip]);
      const float mg = sums.x / dim, mz = sums.y / dim;
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const int c = i * kAnyThreads + threadIdx.x;
        if (c < dim) from_float(rs * (g[i] - mg - z[i] * mz), dx + r * dx_ld + c);
      }
    }
    if (part) {
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const int c = i * kAnyThreads + threadIdx.x;
        if (c < dim) {
          pw[c] = aw[i];
          pb[c] = ab[i];
        }
      }
    }
  } else {
    if (part)
      for (int c = threadIdx.x; c < dim; c += kAnyThreads) pw[c] = pb[c] = 0.f;
    for (long long r = blockIdx.x; r < rows; r += gridDim.x, flip ^= 1) {
      const float m = mean[r], rs = rstd[r];
      const T *xr = x + r * x_ld, *dr = dy + r * dy_ld;
      float sg = 0.f, sz = 0.f;
      for (int c = threadIdx.x; c < dim; c += kAnyThreads) {
        const float z = (to_float(xr[c]) - m) * rs, d = to_float(dr[c]), g = w ? d * w[c] : d;
        if (part) {
          pw[c] += d * z;
          pb[c] += d;
        }
        sg += g;
        sz += g * z;
      }
      const float2 sums = row_sum<kAnyThreads / 32>(sg, sz, red[flip]);
      const float mg = sums.x / dim, mz = sums.y / dim;
      for (int c = threadIdx.x; c < dim; c += kAnyThreads) {
        const float z = (to_float(xr[c]) - m) * rs, d = to_float(dr[c]), g = w ? d * w[c] : d;
        from_float(rs * (g - mg - z * mz), dx + r * dx_ld + c);
      }
    }
  }
}

// dweight[c] (+)= sum over n partial rows of part[0][.][c], dbias likewise from part[1].
constexpr int kReduceCols = 16, kReduceRows = 64;
__global__ void __launch_bounds__(kReduceCols* kReduceRows)
    k_ln_reduce(int n, int dim, const float* __restrict__ part, float* __restrict__ dweight,
                float* __restrict__ dbias, int accumulate) {
  grid_dependency_wait();
  __shared__ float s[kReduceRows][kReduceCols + 1];
  float* out = blockIdx.y ? dbias : dweight;
  if (!out) return;
  const int c = blockIdx.x * kReduceCols + threadIdx.x;
  const float* p = part + (blockIdx.y ? static_cast<long long>(n) * dim : 0);
  float a = 0.f;
  if (c < dim) {
    int r = threadIdx.y;
    for (; r + 7 * kReduceRows < n; r += 8 * kReduceRows) {  // eight loads in flight
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = p[static_cast<long long>(r + k * kReduceRows) * dim + c];
#pragma unroll
      for (int k = 0; k < 8; ++k) a += v[k];
    }
#pragma unroll 4
    for (; r < n; r += kReduceRows) a += p[static_cast<long long>(r) * dim + c];
  }
  s[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  const int warp = (threadIdx.y * kReduceCols + threadIdx.x) >> 5, lane = (threadIdx.y * kReduceCols + threadIdx.x) & 31;
  if (warp >= kReduceCols) return;
  a = s[lane][warp] + s[lane + 32][warp];  // a warp sums a column over the rows of s
#pragma unroll
  for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  const int col = blockIdx.x * kReduceCols + warp;
  if (lane == 0 && col < dim) out[col] = accumulate ? out[col] + a : a;
}

// ------------------------------------------------------------------------- launches
// Rows of whole, aligned 16-byte pieces: base and row stride.
inline bool rows_aligned(const void* p, long long ld, int es) { return aligned16(p) && (ld * es) % 16 == 0; }

// Whether rows of both start at the same place in a 16-byte piece.
inline bool same_place(const void* p, long long p_ld, const void* q, long long q_ld, int es) {
  return (reinterpret_cast<uintptr_t>(p) - reinterpret_cast<uintptr_t>(q)) % 16 == 0 && (p_ld - q_ld) * es % 16 == 0;
}

struct LnFwd {
  long long rows;
  int dim;
  const void* x;
  long long x_ld;
  const float *w, *b;
  float eps;
  void* y;
  long long y_ld;
  float *mean, *rstd;
};

template <class T, int kWarps, int kVecs, int kRows>
void fwd_kernel(const LnFwd& a, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((a.rows + kRows - 1) / kRows);
  k_ln_fwd<T, kWarps, kVecs, kRows><<<grid, 32 * kWarps * kRows, 0, s>>>(
      a.rows, a.dim, static_cast<const T*>(a.x), a.x_ld, a.w, a.b, a.eps, static_cast<T*>(a.y), a.y_ld, a.mean,
      a.rstd);
}

template <class T, int kWarps, int kVecs, int kCtas>
void fwd_edges(const LnFwd& a, cudaStream_t s) {
  constexpr int kStep = kLanes<T>;
  const long long want = round_up(a.rows, kStep), most = static_cast<long long>(kCtas) * num_sms() / kStep * kStep;
  k_ln_fwd_edges<T, kWarps, kVecs, kCtas><<<static_cast<unsigned>(want < most ? want : most), 32 * kWarps, 0, s>>>(
      a.rows, a.dim, static_cast<const T*>(a.x), a.x_ld, a.w, a.b, a.eps, static_cast<T*>(a.y), a.y_ld, a.mean,
      a.rstd);
}

template <class T, int kCols>
void fwd_any(const LnFwd& a, cudaStream_t s) {
  k_ln_fwd_any<T, kCols><<<static_cast<unsigned>(a.rows), kAnyThreads, 0, s>>>(
      a.dim, static_cast<const T*>(a.x), a.x_ld, a.w, a.b, a.eps, static_cast<T*>(a.y), a.y_ld, a.mean, a.rstd);
}

template <class T>
void launch_fwd(const LnFwd& a, cudaStream_t s) {
  const bool vec = a.dim % kLanes<T> == 0 && rows_aligned(a.x, a.x_ld, sizeof(T)) &&
                   rows_aligned(a.y, a.y_ld, sizeof(T)) && (!a.w || aligned16(a.w)) && (!a.b || aligned16(a.b));
  const bool place = same_place(a.x, a.x_ld, a.y, a.y_ld, sizeof(T));
  const int pieces = a.dim / kLanes<T>, most = (a.dim + 2 * kLanes<T> - 2) / kLanes<T>;  // pieces that a row can touch
  if (vec && pieces <= 32)
    fwd_kernel<T, 1, 1, 4>(a, s);
  else if (vec && pieces <= 64)
    fwd_kernel<T, 1, 2, 4>(a, s);
  else if (vec && pieces <= 128)
    fwd_kernel<T, 1, 4, 4>(a, s);
  else if (vec && pieces <= 256)
    fwd_kernel<T, 4, 2, 1>(a, s);
  else if (vec && pieces <= 512)
    fwd_kernel<T, 2, 8, 1>(a, s);
  else if (vec && pieces <= 1024)
    fwd_kernel<T, 8, 4, 1>(a, s);
  else if (vec && pieces <= 2048)
    fwd_kernel<T, 16, 4, 1>(a, s);
  else if (place && most <= 64)
    fwd_edges<T, 1, 2, 16>(a, s);
  else if (place && most <= 128)
    fwd_edges<T, 2, 2, 12>(a, s);
  else if (place && most <= 256)
    fwd_edges<T, 4, 2, 6>(a, s);
  else if (place && most <= 512)
    fwd_edges<T, 8, 2, 3>(a, s);
  else if (place && most <= 1024)
    fwd_edges<T, 16, 2, 1>(a, s);
  else if (a.dim <= 4 * kAnyThreads)
    fwd_any<T, 4>(a, s);
  else if (a.dim <= 16 * kAnyThreads)
    fwd_any<T, 16>(a, s);
  else
    fwd_any<T, 0>(a, s);
}

struct LnBwd {
  long long rows;
  int dim;
  const void* dy;
  long long dy_ld;
  const void* x;
  long long x_ld;
  const float *w, *mean, *rstd;
  void* dx;
  long long dx_ld;
  float* part;
  unsigned grid;
};

// CTAs of the backward at most, the rows of partial sums that the workspace holds.
constexpr int kBwdCtas = 6;
unsigned bwd_grid(long long rows) {
  const long long most = static_cast<long long>(kBwdCtas) * num_sms(), want = round_up(rows, 8);
  return static_cast<unsigned>(want < most ? want : most);
}

template <class T, int kWarps, int kVecs, int kGroups, int kCtas, bool kEdges>
void bwd_kernel(LnBwd& a, cudaStream_t s) {
  static_assert(kCtas <= kBwdCtas, "rows of the workspace");
  constexpr int kStep = kEdges ? kLanes<T> : 1;  // of the grid, so that a group's rows start alike
  const long long want = round_up((a.rows + kGroups - 1) / kGroups, kStep);
  const long long most = static_cast<long long>(kCtas) * num_sms() / kStep * kStep;
  a.grid = static_cast<unsigned>(want < most ? want : most);
  k_ln_bwd<T, kWarps, kVecs, kGroups, kCtas, kEdges><<<a.grid, 32 * kWarps * kGroups, 0, s>>>(
      a.rows, a.dim, static_cast<const T*>(a.dy), a.dy_ld, static_cast<const T*>(a.x), a.x_ld, a.w, a.mean, a.rstd,
      static_cast<T*>(a.dx), a.dx_ld, a.part);
}

template <class T, int kCols>
void bwd_any(LnBwd& a, cudaStream_t s) {
  k_ln_bwd_any<T, kCols><<<a.grid, kAnyThreads, 0, s>>>(
      a.rows, a.dim, static_cast<const T*>(a.dy), a.dy_ld, static_cast<const T*>(a.x), a.x_ld, a.w, a.mean, a.rstd,
      static_cast<T*>(a.dx), a.dx_ld, a.part);
}

template <class T, bool kEdges>
void bwd_pieces(LnBwd& a, int pieces, cudaStream_t s) {
  // Two pieces a thread and 512 threads an SM: few warps a row make its sums cheap, and a row on
  // its way for each group covers the latency. 32768 rows of 1024 bf16 values: 38 us; with one
  // piece a thread 44, with two rows at a time 49, with four pieces a thread 76 (spills); without
  // the groups (one row of partial sums each) 42. One CTA an SM has fewer rows of partial sums
  // still, and from 129 pieces on gains by it (16384 rows of 2048: 38 us against 39); below, the
  // groups in turn cost more (32768 rows of 512: 20.5 against 19).
  if (pieces <= 64)
    bwd_kernel<T, 1, 2, 8, 2, kEdges>(a, s);
  else if (pieces <= 128)
    bwd_kernel<T, 2, 2, 4, 2, kEdges>(a, s);
  else if (pieces <= 256)
    bwd_kernel<T, 4, 2, 4, 1, kEdges>(a, s);
  else if (pieces <= 512)
    bwd_kernel<T, 8, 2, 2, 1, kEdges>(a, s);
  else
    bwd_kernel<T, 16, 2, 1, 1, kEdges>(a, s);
}

template <class T>
void launch_bwd(LnBwd& a, cudaStream_t s) {
  const bool vec = a.dim % kLanes<T> == 0 && rows_aligned(a.x, a.x_ld, sizeof(T)) &&
                   rows_aligned(a.dy, a.dy_ld, sizeof(T)) && rows_aligned(a.dx, a.dx_ld, sizeof(T)) &&
                   (!a.w || aligned16(a.w));
  const bool place = same_place(a.x, a.x_ld, a.dy, a.dy_ld, sizeof(T)) && same_place(a.x, a.x_ld, a.dx, a.dx_ld, sizeof(T));
  // pieces that a row can touch
  const int pieces = vec ? a.dim / kLanes<T> : (a.dim + 2 * kLanes<T> - 2) / kLanes<T>;
  if (vec && pieces <= 1024)
    bwd_pieces<T, false>(a, pieces, s);
  else if (place && pieces <= 1024)
    bwd_pieces<T, true>(a, pieces, s);
  else if (a.dim <= 4 * kAnyThreads)
    bwd_any<T, 4>(a, s);
  else if (a.dim <= 8 * kAnyThreads)
    bwd_any<T, 8>(a, s);
  else if (a.dim <= 16 * kAnyThreads)
    bwd_any<T, 16>(a, s);
  else
    bwd_any<T, 0>(a, s);
}

pc_status_t check_shape(long long rows, int dim) {
  PC_CHECK(rows >= 0 && rows < (1ll << 31), PC_ERR_SHAPE, "rows must be in [0, 2^31) (got %lld)", rows);
  PC_CHECK(dim >= 1 && dim <= (1 << 24), PC_ERR_SHAPE, "dim must be in [1, 2^24] (got %d)", dim);
  return PC_OK;
}

pc_status_t check_rows(const char* name, const void* p, long long ld, long long rows, int dim, pc_dtype_t dt) {
  PC_CHECK(p, PC_ERR_NULL, "%s must not be NULL", name);
  PC_CHECK(rows <= 1 || ld >= dim, PC_ERR_SHAPE, "%s: row stride %lld is shorter than a row of %d", name, ld, dim);
  PC_CHECK(reinterpret_cast<uintptr_t>(p) % dtype_bytes(dt) == 0, PC_ERR_ALIGNMENT, "%s is not aligned to its type",
           name);
  return PC_OK;
}

// In place a row is written where it was read: at another stride it would lie on other rows, which
// other CTAs have yet to read.
pc_status_t check_in_place(const char* out_name, const void* out, long long out_ld, const char* in_name, const void* in,
                           long long in_ld, long long rows) {
  PC_CHECK(out != in || rows <= 1 || out_ld == in_ld, PC_ERR_SHAPE, "%s is %s with another row stride (%lld, %lld)",
           out_name, in_name, out_ld, in_ld);
  return PC_OK;
}

}  // namespace
}  // namespace pc

extern "C" {

pc_status_t pc_layer_norm_fwd(long long rows, int dim, const void* x, long long x_ld, const float* weight,
                              const float* bias, float eps, void* y, long long y_ld, float* mean, float* rstd,
                              pc_dtype_t dtype, cudaStream_t stream) {
  pc::clear_error();
  PC_TRY(pc::check_dtype(dtype));
  PC_TRY(pc::check_shape(rows, dim));
  PC_CHECK(eps >= 0.f, PC_ERR_SHAPE, "eps must not be negative (got %g)", static_cast<double>(eps));
  if (rows == 0) return PC_OK;
  PC_TRY(pc::check_rows("x", x, x_ld, rows, dim, dtype));
  PC_TRY(pc::check_rows("y", y, y_ld, rows, dim, dtype));
  PC_TRY(pc::check_in_place("y", y, y_ld, "x", x, x_ld, rows));
  const pc::LnFwd a{rows, dim, x, x_ld, weight, bias, eps, y, y_ld, mean, rstd};
  if (dtype == PC_BF16)
    pc::launch_fwd<__nv_bfloat16>(a, stream);
  else
    pc::launch_fwd<float>(a, stream);
  PC_LAUNCH_CHECK();
  return PC_OK;
}

pc_status_t pc_layer_norm_bwd_workspace(long long rows, int dim, size_t* bytes) {
  pc::clear_error();
  PC_CHECK(bytes, PC_ERR_NULL, "bytes must not be NULL");
  PC_TRY(pc::check_shape(rows, dim));
  *bytes = 2 * sizeof(float) * static_cast<size_t>(pc::bwd_grid(rows)) * dim;
  return PC_OK;
}

pc_status_t pc_layer_norm_bwd(long long rows, int dim, const void* dy, long long dy_ld, const void* x, long long x_ld,
                              const float* weight, const float* mean, const float* rstd, void* dx, long long dx_ld,
                              float* dweight, float* dbias, int accumulate, pc_dtype_t dtype, void* ws,
                              size_t ws_bytes, cudaStream_t stream) {
  pc::clear_error();
  PC_TRY(pc::check_dtype(dtype));
  PC_TRY(pc::check_shape(rows, dim));
  const bool params = dweight || dbias;
  if (rows > 0) {
    PC_TRY(pc::check_rows("dy", dy, dy_ld, rows, dim, dtype));
    PC_TRY(pc::check_rows("x", x, x_ld, rows, dim, dtype));
    PC_TRY(pc::check_rows("dx", dx, dx_ld, rows, dim, dtype));
    PC_TRY(pc::check_in_place("dx", dx, dx_ld, "dy", dy, dy_ld, rows));
    PC_TRY(pc::check_in_place("dx", dx, dx_ld, "x", x, x_ld, rows));
    PC_CHECK(mean && rstd, PC_ERR_NULL, "mean and rstd must not be NULL");
  }
  unsigned grid = pc::bwd_grid(rows);  // of the launch at most
  if (params && rows > 0) {
    PC_CHECK(ws && ws_bytes >= 2 * sizeof(float) * static_cast<size_t>(grid) * dim, PC_ERR_WORKSPACE,
             "workspace of %zu bytes is too small", ws_bytes);
    PC_CHECK(pc::aligned16(ws), PC_ERR_ALIGNMENT, "workspace is not 16-byte aligned");
  }
  if (rows > 0) {
    pc::LnBwd a{rows, dim, dy, dy_ld, x, x_ld, weight, mean, rstd, dx, dx_ld,
                      params ? static_cast<float*>(ws) : nullptr, grid};
    if (dtype == PC_BF16)
      pc::launch_bwd<__nv_bfloat16>(a, stream);
    else
      pc::launch_bwd<float>(a, stream);
    PC_LAUNCH_CHECK();
    grid = a.grid;
  }
  if (params) {  // no rows: the sums are zero
    cudaLaunchAttribute attr;  // set up while the rows are still being read
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((dim + pc::kReduceCols - 1) / pc::kReduceCols, 2);
    cfg.blockDim = dim3(pc::kReduceCols, pc::kReduceRows);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    PC_CUDA(cudaLaunchKernelEx(&cfg, pc::k_ln_reduce, static_cast<int>(grid), dim, static_cast<const float*>(ws),
                               dweight, dbias, accumulate));
    PC_LAUNCH_CHECK();
  }
  return PC_OK;
}

}  // extern "C"

// Linear attention with a decay for each head: per sequence b and head h, with
// l = exp(log_decay[h]) and n = lengths[b] tokens,
//
//   S_t = l S_{t-1} + k_t v_t^T        o_t = scale q_t^T S_t        t = 1 .. n, S_0 given
//
// Every direction is one pass of the same form. With the gradient of S_t,
//   R_t = scale q_t do_t^T + l R_{t+1},  R_n = scale q_n do_n^T + dS_n,
// the backward is  dq_t = scale S_t do_t,  dk_t = R_t v_t,  dv_t = R_t^T k_t,  dS_0 = l R_1:
//   dq = the forward of (do, v, k) with the state transposed,
//   dk = the time-reversed forward of (v, do, q) with the state transposed,
//   dv = the time-reversed forward of (k, q, do).
// A pass runs in chunks of C tokens (i, j: positions in a tile, in order of time):
//   O = (P . L) V + diag(in) Q S,   S' = l^m S + (diag(up) K)^T V,   P = Q K^T,
// with m real tokens in the tile and, in order of time, L_ij = l^(i-j) for i >= j,
// in_i = l^(i-pad+1), up_i = l^(C-1-i); reversed, L_ij = l^(j-i) for j >= i and in, up
// exchanged. No exponent is negative, so nothing overflows for l <= 1. Tiles end at
// the sequence's end: a length that is no multiple of C leaves its `pad` missing rows at
// the front of the first tile (zeros that add nothing), so no row past the length is
// ever read.
#include "linear_attention_tc.cuh"

namespace pc {
namespace {

__device__ __forceinline__ float la_load(const float* p) { return *p; }
__device__ __forceinline__ float la_load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void la_store(float* p, float v) { *p = v; }
__device__ __forceinline__ void la_store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// ------------------------------------------------------------- any type and head size
// All products in float32 on the CUDA cores. A CTA owns one (b, h), kSimtDvs columns of v
// and a segment of the chunks, and walks them with its columns of S in shared memory; the
// scores are formed again for each slice of columns. A thread's outputs are tiles of 2 x 2
// scores, 2 x 4 of O and 4 x 4 of S, fed by 16-byte shared loads (one value at a time the
// loads bound the kernel). A chunk is a few us of latencies on one CTA, so sequences are cut
// until every SM has several: a first launch (kStates) leaves each segment's own
// contribution to the state, the second adds up the ones before its own.
constexpr int kSimtThreads = 256, kSimtC = 32, kSimtDvs = 64;
constexpr int kMaxHeadDim = 256;

// Floats between rows of Q and K: whole 16-byte pieces, an odd number of them (eight lanes'
// rows then lie in different banks).
__host__ __device__ inline int simt_pitch(int dk) { return 4 * (((dk + 3) / 4) | 1); }
constexpr int kSimtPPitch = kSimtC + 4;

size_t simt_smem(int dk) {
  const size_t wide = (dk + 3) / 4 * 4;
  return sizeof(float) * (2 * size_t(kSimtC) * simt_pitch(dk) + 2 * size_t(kSimtC) * kSimtDvs +
                          size_t(kSimtC) * kSimtPPitch + wide * kSimtDvs + kSimtC + 1);
}

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void fma4(float4& a, float k, const float4& v) {
  a.x += k * v.x;
  a.y += k * v.y;
  a.z += k * v.z;
  a.w += k * v.w;
}
__device__ __forceinline__ float dot4(const float4& a, const float4& b, float c) {
  return a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w + c;
}

struct LaSimtArgs {
  LaArgs a;
  float* partial;  // [pass][B*H][segments - 1][dk][dv], spaced for the largest pass
  int passes, segments, chunks_per_segment;
};

template <class T, bool kStates>
__global__ void __launch_bounds__(kSimtThreads) k_la_simt(const __grid_constant__ LaSimtArgs args) {
  extern __shared__ __align__(16) float sm[];
  if constexpr (kStates) grid_dependents_launch();
  const LaArgs& a = args.a;
  const int pass = blockIdx.z % args.passes, seg = blockIdx.z / args.passes;
  const LaPass& p = a.pass[pass];
  const int c0 = blockIdx.y * kSimtDvs;
  if (c0 >= p.dv) return;
  constexpr int C = kSimtC;
  const int b = blockIdx.x / a.H, h = blockIdx.x % a.H, dk = p.dk, pitch = simt_pitch(dk), tid = threadIdx.x;
  const int wide = (dk + 3) / 4 * 4, warp = tid >> 5, lane = tid & 31;
  const int cols = min(kSimtDvs, p.dv - c0);
  float* Q = sm;
  float* K = Q + C * pitch;
  float* V = K + C * pitch;
  float* Vw = V + C * kSimtDvs;  // V times the tokens' weights in the state
  float* P = Vw + C * kSimtDvs;
  float* S = P + C * kSimtPPitch;
  float* pw = S + wide * kSimtDvs;  // l^0 .. l^C
  const float g = a.log_decay[h];
  if (tid <= C) pw[tid] = decay_pow(g, tid);
  const long long bh = blockIdx.x, size = static_cast<long long>(dk) * p.dv;
  const int len = la_length(a, b), nch = (len + C - 1) / C;
  const int first = seg * args.chunks_per_segment, last = min(first + args.chunks_per_segment, nch);
  const int final_seg = nch > 0 ? (nch - 1) / args.chunks_per_segment : 0;
  if (kStates ? seg >= final_seg : seg > final_seg && !(seg == args.segments - 1 && len < a.T)) return;
  float* partial = args.partial + (static_cast<long long>(pass) * a.B * a.H + bh) * (args.segments - 1) * size;
  // decay over a segment before this one; a forward's first one may lack tokens
  const float over = decay_pow(g, args.chunks_per_segment * C);
  const float over0 = p.reverse ? over : decay_pow(g, args.chunks_per_segment * C - (nch * C - len));
  auto load_state = [&]() {  // S before this segment, many loads in flight
    constexpr int kAtOnce = 8;
    const int before = kStates ? 0 : min(seg, final_seg);
    if (before > 0) grid_dependency_wait();
    for (int e0 = tid; e0 < wide * kSimtDvs; e0 += kAtOnce * kSimtThreads) {
      const int c = e0 % kSimtDvs, d0 = e0 / kSimtDvs;  // the others are kSimtThreads / kSimtDvs rows apart
      float v[kAtOnce];
      bool in[kAtOnce];
#pragma unroll
      for (int x = 0; x < kAtOnce; ++x) {
        const int d = d0 + x * (kSimtThreads / kSimtDvs);
        in[x] = !kStates && c < cols && d < dk;
        v[x] = in[x] && p.s_in ? p.s_in[bh * size + (p.s_in_transposed ? static_cast<long long>(c0 + c) * dk + d
                                                                       : static_cast<long long>(d) * p.dv + c0 + c)]
                               : 0.f;
      }
#pragma unroll 2
      for (int y = 0; y < before; ++y) {  // what the segments before this one add
        const float* ps = partial + y * size + static_cast<long long>(d0) * p.dv + c0 + c;
        const float carry = y == 0 ? over0 : over;
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x)
          if (in[x]) v[x] = carry * v[x] + ps[x * (kSimtThreads / kSimtDvs) * p.dv];
      }
#pragma unroll
      for (int x = 0; x < kAtOnce; ++x)
        if (d0 + x * (kSimtThreads / kSimtDvs) < wide) S[e0 + x * kSimtThreads] = v[x];
    }
  };
  if (kStates || first >= last) load_state();
  const T* q = static_cast<const T*>(p.q) + b * p.qs[0] + h * p.qs[2];
  const T* k = static_cast<const T*>(p.k) + b * p.ks[0] + h * p.ks[2];
  const T* v = static_cast<const T*>(p.v) + b * p.vs[0] + h * p.vs[2] + c0;
  T* o = static_cast<T*>(p.o) + b * p.os[0] + h * p.os[2] + c0;
  for (int step = first; step < last; ++step) {
    const int tile = p.reverse ? nch - 1 - step : step;
    const int t0 = len - (nch - tile) * C, pad = max(0, -t0);
    __syncthreads();  // the last chunk's reads are done
#pragma unroll
    for (int r = 0; r < C / 8; ++r) {
      const int i = warp + 8 * r;
      const bool in = i >= pad;
      for (int d = lane; d < wide; d += 32) {
        const bool there = in && d < dk;
        if (!kStates) Q[i * pitch + d] = there ? la_load(q + (t0 + i) * p.qs[1] + d) : 0.f;
        K[i * pitch + d] = there ? la_load(k + (t0 + i) * p.ks[1] + d) : 0.f;
      }
      const float w = pw[p.reverse ? max(i - pad + 1, 0) : C - 1 - i] * p.c_up;
#pragma unroll
      for (int c = lane; c < kSimtDvs; c += 32) {
        const float x = in && c < cols ? la_load(v + (t0 + i) * p.vs[1] + c) : 0.f;
        V[i * kSimtDvs + c] = x;
        Vw[i * kSimtDvs + c] = x * w;
      }
    }
    __syncthreads();
    const int pair = 2 * (tid >> 4), col = tid & 15;  // rows pair, pair + 1; columns 4 col .. of O and S
    if constexpr (!kStates) {
      float score[2][2] = {};
      for (int d = 0; d < wide; d += 4) {
        const float4 q0 = ld4(Q + pair * pitch + d), q1 = ld4(Q + (pair + 1) * pitch + d);
        const float4 k0 = ld4(K + col * pitch + d), k1 = ld4(K + (col + 16) * pitch + d);
        score[0][0] = dot4(q0, k0, score[0][0]);
        score[0][1] = dot4(q0, k1, score[0][1]);
        score[1][0] = dot4(q1, k0, score[1][0]);
        score[1][1] = dot4(q1, k1, score[1][1]);
      }
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int i = pair + r, j = col + 16 * x, gap = p.reverse ? j - i : i - j;
          P[i * kSimtPPitch + j] = gap >= 0 ? score[r][x] * (pw[gap] * p.c_intra) : 0.f;
        }
      if (step == first) {  // the states may have been on their way until now
        load_state();
        __syncthreads();
      } else {
        __syncwarp();  // a warp reads only the rows of P that it wrote
      }
      float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
      auto add = [&](const float* a, int pitch_a, const float* x) {  // four terms of both rows
        const float4 f0 = ld4(a), f1 = ld4(a + pitch_a);
        const float a0[4] = {f0.x, f0.y, f0.z, f0.w}, a1[4] = {f1.x, f1.y, f1.z, f1.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 y = ld4(x + e * kSimtDvs + 4 * col);
          fma4(acc[0], a0[e], y);
          fma4(acc[1], a1[e], y);
        }
      };
      for (int d = 0; d < wide; d += 4) add(Q + pair * pitch + d, pitch, S + d * kSimtDvs);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int i = pair + r;
        const float w = pw[p.reverse ? C - 1 - i : max(i - pad + 1, 0)] * p.c_inter;
        acc[r] = make_float4(acc[r].x * w, acc[r].y * w, acc[r].z * w, acc[r].w * w);
      }
      for (int j = 0; j < C; j += 4) add(P + pair * kSimtPPitch + j, kSimtPPitch, V + j * kSimtDvs);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int i = pair + r;
        const float x[4] = {acc[r].x, acc[r].y, acc[r].z, acc[r].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (i >= pad && 4 * col + e < cols) la_store(o + (t0 + i) * p.os[1] + 4 * col + e, x[e]);
      }
      __syncthreads();  // every read of S, before its update
    }
    const float carry = pw[C - pad];
    for (int d = 4 * (tid >> 4); d < wide; d += 4 * (kSimtThreads / 16)) {
      float4 acc[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 x = ld4(S + (d + e) * kSimtDvs + 4 * col);
        acc[e] = make_float4(carry * x.x, carry * x.y, carry * x.z, carry * x.w);
      }
#pragma unroll 4
      for (int j = 0; j < C; ++j) {
        const float4 x = ld4(K + j * pitch + d), y = ld4(Vw + j * kSimtDvs + 4 * col);
        fma4(acc[0], x.x, y);
        fma4(acc[1], x.y, y);
        fma4(acc[2], x.z, y);
        fma4(acc[3], x.w, y);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) *reinterpret_cast<float4*>(S + (d + e) * kSimtDvs + 4 * col) = acc[e];
    }
  }
  __syncthreads();
  if constexpr (kStates) {
    for (int e = tid; e < dk * kSimtDvs; e += kSimtThreads) {
      const int d = e / kSimtDvs, c = e % kSimtDvs;
      if (c < cols) partial[seg * size + static_cast<long long>(d) * p.dv + c0 + c] = S[e];
    }
    return;
  }
  if (p.s_out && seg == final_seg)
    for (int e = tid; e < dk * kSimtDvs; e += kSimtThreads) {
      const int d = e / kSimtDvs, c = e % kSimtDvs;
      if (c < cols) p.s_out[bh * dk * p.dv + static_cast<long long>(d) * p.dv + c0 + c] = S[e];
    }
  // rows past the length hold zeros
  if (seg == args.segments - 1)
    for (long long e = tid; e < static_cast<long long>(a.T - len) * cols; e += kSimtThreads)
      la_store(o + (len + e / cols) * p.os[1] + e % cols, 0.f);
  la_end_after_states();
}

// Segments: enough that every SM has four CTAs.
int simt_segments(long long heads, int T, int dk, int dv) {
  const int nch = (T + kSimtC - 1) / kSimtC;
  const int wide = dk > dv ? dk : dv;  // a backward has passes of either order
  const long long ctas = heads * ((wide + kSimtDvs - 1) / kSimtDvs), want = (4ll * num_sms() + ctas - 1) / ctas;
  if (nch <= 1 || want <= 1) return 1;
  const int per = static_cast<int>((nch + want - 1) / want);
  return (nch + per - 1) / per;
}
size_t simt_partial_bytes(long long heads, int segments, int dk, int dv) {
  return sizeof(float) * static_cast<size_t>(heads) * (segments - 1) * dk * dv;
}

// Launches a pass, after its states' launch (`dependent`) as its programmatic dependent: CTAs
// start as SMs come free and wait for the states themselves.
template <class Args>
pc_status_t launch_after(void (*kernel)(Args), dim3 grid, int threads, int smem, cudaStream_t s, bool dependent,
                         const Args& args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = dependent ? 1 : 0;
  PC_CUDA(cudaLaunchKernelEx(&cfg, kernel, args));
  PC_LAUNCH_CHECK();
  return PC_OK;
}

template <class T>
pc_status_t launch_simt(const LaArgs& a, int passes, void* ws, cudaStream_t s, int* launches) {
  int dk = 0, dv = 0;
  for (int i = 0; i < passes; ++i) {
    dk = a.pass[i].dk > dk ? a.pass[i].dk : dk;
    dv = a.pass[i].dv > dv ? a.pass[i].dv : dv;
  }
  const int smem = static_cast<int>(simt_smem(dk)), most = static_cast<int>(simt_smem(kMaxHeadDim));
  LaSimtArgs t{};
  t.a = a;
  t.partial = static_cast<float*>(ws);
  t.passes = passes;
  t.segments = simt_segments(static_cast<long long>(a.B) * a.H * passes, a.T, a.pass[0].dk, a.pass[0].dv);
  const int nch = (a.T + kSimtC - 1) / kSimtC;
  t.chunks_per_segment = nch > 0 ? (nch + t.segments - 1) / t.segments : 1;
  const unsigned heads = static_cast<unsigned>(a.B) * a.H, slices = (dv + kSimtDvs - 1) / kSimtDvs;
  if (t.segments > 1) {
    PC_TRY((allow_smem<k_la_simt<T, true>>(most)));
    k_la_simt<T, true><<<dim3(heads, slices, (t.segments - 1) * passes), kSimtThreads, smem, s>>>(t);
    PC_LAUNCH_CHECK();
    ++*launches;
  }
  PC_TRY((allow_smem<k_la_simt<T, false>>(most)));
  PC_TRY(launch_after(k_la_simt<T, false>, dim3(heads, slices, t.segments * passes), kSimtThreads, smem, s,
                      t.segments > 1, t));
  ++*launches;
  return PC_OK;
}

// ------------------------------------------------------------------- tensor cores
// A tensor's map, or false where it has no aligned one. A dimension of one step or of
// stride 0 (shared by all heads or sequences) is left out of the map.
bool tc_map(CUtensorMap* map, int (&ext)[2], const void* base, const long long (&st)[3], int d, int T, int H, int B,
            pc_status_t* status) {
  ext[0] = H > 1 && st[2] != 0;
  ext[1] = B > 1 && st[0] != 0;
  const long long row = T > 1 ? st[1] : 8;
  const long long strides[3] = {row, ext[0] ? st[2] : 8, ext[1] ? st[0] : 8};
  if (!aligned16(base) || d % 8) return false;
  for (const long long s : strides)
    if (s <= 0 || s % 8 || s >= (1ll << 38)) return false;
  const long long dims[4] = {d, T, ext[0] ? H : 1, ext[1] ? B : 1};
  *status = encode_bf16_map4(map, base, dims, strides, 64, kTcC);
  return *status == PC_OK;
}

// Outputs are stored in 16-byte pieces.
bool tc_output(const LaPass& p, int T, int H, int B) {
  return aligned16(p.o) && p.dv % 8 == 0 && (T <= 1 || p.os[1] % 8 == 0) && (H <= 1 || p.os[2] % 8 == 0) &&
         (B <= 1 || p.os[0] % 8 == 0);
}

bool tc_heads(int dk, int dv, pc_dtype_t dt) {
  return dt == PC_BF16 && dk % 8 == 0 && dv % 8 == 0 && dk <= 128 && dv <= 128;
}
int tc_pad(int d) { return d <= 64 ? 64 : 128; }

// How sequences are cut. One CTA per SM takes a segment; cutting a sequence into S makes
// the first launch's states cost about half of a pass's chunks, and each CTA a start of
// about one chunk (measured at head size 128: 3.1 us a chunk, 1.7 us of states alone, 3 us
// from a CTA's launch to its first product), and joining a segment's share 0.3. Where two
// segments of every sequence fit the SMs beside each other, the first ones run beside the
// launch of their states and may be longer than the second ones, which wait for it
// (4 x 2000 tokens, 16 heads: 12 + 4 chunks 48 us, 8 + 8 52; 6 x 2700, 12 heads: 60, 67).
struct TcCut {
  int segments, chunks;  // chunks of every segment but the last
};
TcCut tc_cut(long long heads, int T) {
  const int nch = (T + kTcC - 1) / kTcC;
  const long long sms = num_sms();
  double best = 1e30;
  TcCut cut{1, nch > 0 ? nch : 1};
  for (int s = 1; s <= nch && s <= 64; ++s) {
    const int per = (nch + s - 1) / s;
    if ((nch + per - 1) / per != s) continue;  // the same cut as fewer segments
    double t = static_cast<double>((heads * s + sms - 1) / sms) * (per + 1.0 + 0.3 * (s - 1));
    if (s > 1) t += static_cast<double>((heads * (s - 1) + sms - 1) / sms) * (0.5 * per + 1.0);
    int chunks = per;
    if (s == 2 && 2 * heads <= sms) {
      for (int a = per; a < nch; ++a) {
        const double first = a + 1.0, second = 0.55 * a + 1.0 + 1.3 + (nch - a), both = first > second ? first : second;
        if (both < t) {
          t = both;
          chunks = a;
        }
      }
    }
    if (t < 0.97 * best) {  // a finer cut has to earn its first launch
      best = t;
      cut = {s, chunks};
    }
  }
  return cut;
}

size_t tc_partial_bytes(long long heads, int segments, int dk, int dv) {
  return sizeof(float) * static_cast<size_t>(heads) * (segments - 1) * tc_pad(dk) * tc_pad(dv);
}

template <int DK, int DV>
pc_status_t launch_tc(LaTcArgs& t, int passes, cudaStream_t s, int* launches) {
  constexpr int smem = TcShape<DK, DV, false>::kBytes, states_smem = TcShape<DK, DV, true>::kBytes;
  PC_TRY((allow_smem<k_la_tc<DK, DV, false>>(smem)));
  const unsigned heads = static_cast<unsigned>(t.a.B) * t.a.H;
  t.passes = passes;
  if (t.segments > 1) {
    PC_TRY((allow_smem<k_la_tc<DK, DV, true>>(states_smem)));
    k_la_tc<DK, DV, true><<<dim3(heads * passes, t.segments - 1), kTcThreads, states_smem, s>>>(t);
    PC_LAUNCH_CHECK();
    ++*launches;
  }
  ++*launches;
  return launch_after(k_la_tc<DK, DV, false>, dim3(heads * passes, t.segments), kTcThreads, smem, s, t.segments > 1, t);
}

// Runs the passes on the tensor cores; *done = false (and nothing launched) where a tensor's
// alignment does not allow it.
pc_status_t run_tc(const LaArgs& a, int passes, void* ws, cudaStream_t s, int* launches, bool* done) {
  *done = false;
  LaTcArgs t{};
  t.a = a;
  for (int i = 0; i < passes; ++i) {
    const LaPass& p = a.pass[i];
    LaMaps& m = t.maps[i];
    pc_status_t st = PC_OK;
    if (!tc_output(p, a.T, a.H, a.B) || !tc_map(&m.q, m.q_ext, p.q, p.qs, p.dk, a.T, a.H, a.B, &st) ||
        !tc_map(&m.k, m.k_ext, p.k, p.ks, p.dk, a.T, a.H, a.B, &st) ||
        !tc_map(&m.v, m.v_ext, p.v, p.vs, p.dv, a.T, a.H, a.B, &st) ||
        !tc_map(&m.o, m.o_ext, p.o, p.os, p.dv, a.T, a.H, a.B, &st))
      return st;
  }
  const long long heads = static_cast<long long>(a.B) * a.H;
  const TcCut cut = tc_cut(heads * passes, a.T);
  t.segments = cut.segments;
  t.chunks_per_segment = cut.chunks;
  t.partial = static_cast<float*>(ws);
  t.status = device_status_word();
  *done = true;
  // passes of one padded shape go in one launch
  for (int i = 0; i < passes;) {
    const int dk = tc_pad(a.pass[i].dk), dv = tc_pad(a.pass[i].dv);
    int n = i + 1;
    while (n < passes && tc_pad(a.pass[n].dk) == dk && tc_pad(a.pass[n].dv) == dv) ++n;
    LaTcArgs part = t;
    for (int j = i; j < n; ++j) {
      part.a.pass[j - i] = t.a.pass[j];
      part.maps[j - i] = t.maps[j];
    }
    part.partial = t.partial + tc_partial_bytes(heads * i, t.segments, dk, dv) / sizeof(float);
    if (dk == 64 && dv == 64)
      PC_TRY((launch_tc<64, 64>(part, n - i, s, launches)));
    else if (dk == 64)
      PC_TRY((launch_tc<64, 128>(part, n - i, s, launches)));
    else if (dv == 64)
      PC_TRY((launch_tc<128, 64>(part, n - i, s, launches)));
    else
      PC_TRY((launch_tc<128, 128>(part, n - i, s, launches)));
    i = n;
  }
  return PC_OK;
}

// ------------------------------------------------------------------- a single token
// S <- l S + k v^T and o = scale q^T S, in place. Memory-bound: 8 bytes of state per
// 4 flops. A CTA takes one (b, h). Rows of whole aligned 16-byte pieces (kVecLanes > 0):
// kVecLanes lanes share a row of S, a thread keeps kRows rows in flight; otherwise
// (0) a lane takes one value at a time.
constexpr int kStepThreads = 256;
template <class T, int kVecLanes>
__global__ void __launch_bounds__(kStepThreads)
    k_la_step(int H, int dk, int dv, const T* __restrict__ q, long long q_b, long long q_h, const T* __restrict__ k,
              long long k_b, long long k_h, const T* __restrict__ v, long long v_b, long long v_h,
              const float* __restrict__ log_decay, float scale, float* __restrict__ state, T* __restrict__ o,
              long long o_b, long long o_h) {
  __shared__ float part[kStepThreads / 32][kMaxHeadDim];
  __shared__ float qs[kMaxHeadDim], ks[kMaxHeadDim];
  const int b = blockIdx.x / H, h = blockIdx.x % H;
  const float l = decay_pow(log_decay[h], 1);
  const T *qp = q + b * q_b + h * q_h, *kp = k + b * k_b + h * k_h, *vp = v + b * v_b + h * v_h;
  float* S = state + static_cast<long long>(blockIdx.x) * dk * dv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int d = threadIdx.x; d < dk; d += kStepThreads) {
    qs[d] = la_load(qp + d);
    ks[d] = la_load(kp + d);
  }
  if constexpr (kVecLanes > 0) {
    constexpr int kRows = 8, kGroups = kStepThreads / kVecLanes;  // rows in flight, rows at a time
    const int c = (threadIdx.x % kVecLanes) * 4, first = threadIdx.x / kVecLanes;
    const bool in = c < dv;
    float x[4] = {}, acc[4] = {};
    if (in) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = la_load(vp + c + i);
    }
    __syncthreads();
    for (int d0 = first; d0 < dk; d0 += kRows * kGroups) {
      float4 s[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int d = d0 + i * kGroups;
        if (in && d < dk) s[i] = __ldcs(reinterpret_cast<const float4*>(S + d * dv + c));
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int d = d0 + i * kGroups;
        if (in && d < dk) {
          const float kd = ks[d], qd = qs[d];
          s[i] = make_float4(l * s[i].x + kd * x[0], l * s[i].y + kd * x[1], l * s[i].z + kd * x[2],
                             l * s[i].w + kd * x[3]);
          __stcs(reinterpret_cast<float4*>(S + d * dv + c), s[i]);
          acc[0] += qd * s[i].x;
          acc[1] += qd * s[i].y;
          acc[2] += qd * s[i].z;
          acc[3] += qd * s[i].w;
        }
      }
    }
#pragma unroll
    for (int m = kVecLanes; m < 32; m <<= 1)  // the warp's rows
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], m);
    if (lane < kVecLanes && in) {
#pragma unroll
      for (int i = 0; i < 4; ++i) part[warp][c + i] = acc[i];
    }
  } else {
    __syncthreads();
    for (int c = lane; c < dv; c += 32) {
      const float x = la_load(vp + c);
      float acc = 0.f;
#pragma unroll 4
      for (int d = warp; d < dk; d += kStepThreads / 32) {
        const float s = l * S[d * dv + c] + ks[d] * x;
        S[d * dv + c] = s;
        acc += qs[d] * s;
      }
      part[warp][c] = acc;
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < dv; c += kStepThreads) {
    float acc = 0.f;
#pragma unroll
    for (int w = 0; w < kStepThreads / 32; ++w) acc += part[w][c];
    la_store(o + b * o_b + h * o_h + c, acc * scale);
  }
}

template <class T>
void launch_step(int B, int H, int dk, int dv, const void* q, const void* k, const void* v, const long long* s,
                 const float* log_decay, float scale, float* state, void* o, cudaStream_t stream) {
  auto* kernel = k_la_step<T, 0>;
  if (dv % 4 == 0 && aligned16(state) && dv <= 128)
    kernel = dv <= 32 ? k_la_step<T, 8> : dv <= 64 ? k_la_step<T, 16> : k_la_step<T, 32>;
  kernel<<<static_cast<unsigned>(B) * H, kStepThreads, 0, stream>>>(
      H, dk, dv, static_cast<const T*>(q), s[0], s[1], static_cast<const T*>(k), s[2], s[3],
      static_cast<const T*>(v), s[4], s[5], log_decay, scale, state, static_cast<T*>(o), s[6], s[7]);
}

// ------------------------------------------------------------------------- checks
pc_status_t check_la(int B, int T, int H, int dk, int dv, pc_dtype_t dt) {
  PC_TRY(check_dtype(dt));
  PC_CHECK(B >= 0 && T >= 0 && H >= 1 && static_cast<long long>(B) * H < (1ll << 31) && T < (1 << 30), PC_ERR_SHAPE,
           "B, T >= 0, H >= 1, B * H < 2^31 and T < 2^30 wanted (got %d, %d, %d)", B, T, H);
  PC_CHECK(dk >= 1 && dv >= 1, PC_ERR_SHAPE, "head sizes must be >= 1 (got %d, %d)", dk, dv);
  PC_CHECK(dk <= kMaxHeadDim && dv <= kMaxHeadDim, PC_ERR_UNSUPPORTED, "head sizes up to %d (got %d, %d)",
           kMaxHeadDim, dk, dv);
  return PC_OK;
}

pc_status_t check_tensor(const char* name, const void* p, pc_dtype_t dt) {
  PC_CHECK(p, PC_ERR_NULL, "%s must not be NULL", name);
  PC_CHECK(reinterpret_cast<uintptr_t>(p) % dtype_bytes(dt) == 0, PC_ERR_ALIGNMENT, "%s is not aligned to its type",
           name);
  return PC_OK;
}

// An output may not lie where an input does: CTAs of one call read and write side by side.
pc_status_t check_apart(const char* out_name, const void* out, const char* in_name, const void* in) {
  PC_CHECK(out != in, PC_ERR_UNSUPPORTED, "%s may not be %s itself", out_name, in_name);
  return PC_OK;
}

// An output's elements may not share memory, as a stride of zero makes them.
pc_status_t check_stored_once(const char* name, const long long* strides, const int* dims, int n) {
  for (int i = 0; i < n; ++i)
    PC_CHECK(dims[i] <= 1 || strides[i] != 0, PC_ERR_SHAPE, "%s: stride 0 along a dimension of %d", name, dims[i]);
  return PC_OK;
}

// Workspace: the segments' shares of the state, in whichever variant the tensors' alignment
// will allow.
size_t la_workspace(int B, int T, int H, int dk, int dv, int passes, pc_dtype_t dt) {
  const long long heads = static_cast<long long>(B) * H * passes;
  if (T == 0 || heads == 0) return 0;
  const size_t simt = simt_partial_bytes(heads, simt_segments(heads, T, dk, dv), dk, dv);
  const size_t tc = tc_heads(dk, dv, dt) ? tc_partial_bytes(heads, tc_cut(heads, T).segments, dk, dv) : 0;
  return simt > tc ? simt : tc;
}

pc_status_t run_passes(const LaArgs& a, int passes, pc_dtype_t dt, void* ws, size_t ws_bytes, cudaStream_t s) {
  const LaPass& p = a.pass[0];
  const size_t need = la_workspace(a.B, a.T, a.H, p.dk, p.dv, passes, dt);
  PC_CHECK(need == 0 || (ws && ws_bytes >= need), PC_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws_bytes,
           need);
  PC_CHECK(need == 0 || aligned16(ws), PC_ERR_ALIGNMENT, "workspace is not 16-byte aligned");
  ProfileGroup record(s, PC_KIND_LINEAR_ATTENTION,
                      static_cast<long long>(a.B) * a.T * a.H * (passes == 1 ? 4 : 10) * p.dk * p.dv);
  if (a.T > 0 && tc_heads(p.dk, p.dv, dt)) {
    PC_CHECK(static_cast<long long>(a.B) * a.H * passes < (1ll << 31), PC_ERR_SHAPE,
             "%d passes of B * H = %lld heads: fewer than 2^31 in all wanted", passes, static_cast<long long>(a.B) * a.H);
    bool done = false;
    PC_TRY(run_tc(a, passes, ws, s, &record.launches, &done));
    if (done) return PC_OK;
  }
  return dt == PC_BF16 ? launch_simt<__nv_bfloat16>(a, passes, ws, s, &record.launches)
                       : launch_simt<float>(a, passes, ws, s, &record.launches);
}

LaPass make_pass(const void* q, const long long* qs, const void* k, const long long* ks, const void* v,
                 const long long* vs, void* o, const long long* os, int dk, int dv, const float* s_in,
                 float* s_out, bool s_in_transposed, bool reverse, float scale) {
  LaPass p{};
  p.q = q;
  p.k = k;
  p.v = v;
  p.o = o;
  for (int i = 0; i < 3; ++i) {
    p.qs[i] = qs[i];
    p.ks[i] = ks[i];
    p.vs[i] = vs[i];
    p.os[i] = os[i];
  }
  p.dk = dk;
  p.dv = dv;
  p.s_in = s_in;
  p.s_out = s_out;
  p.s_in_transposed = s_in_transposed;
  p.reverse = reverse;
  // in order of time the state is unscaled and read with the scale; R carries the scale
  p.c_intra = scale;
  p.c_inter = reverse ? 1.f : scale;
  p.c_up = reverse ? scale : 1.f;
  return p;
}

}  // namespace
}  // namespace pc

extern "C" {

pc_status_t pc_linear_attention_workspace(int B, int T, int H, int Dk, int Dv, int with_backward, pc_dtype_t dtype,
                                          size_t* bytes) {
  pc::clear_error();
  PC_CHECK(bytes, PC_ERR_NULL, "bytes must not be NULL");
  PC_TRY(pc::check_la(B, T, H, Dk, Dv, dtype));
  *bytes = pc::la_workspace(B, T, H, Dk, Dv, 1, dtype);
  if (with_backward) {  // three times the heads may be cut less
    const size_t back = pc::la_workspace(B, T, H, Dk, Dv, 3, dtype);
    if (back > *bytes) *bytes = back;
  }
  return PC_OK;
}

pc_status_t pc_linear_attention_fwd(int B, int T, int H, int Dk, int Dv, const void* q, const void* k, const void* v,
                                    const long long* strides, const float* log_decay, float scale,
                                    const float* state, const int32_t* lengths, void* o, float* state_out,
                                    pc_dtype_t dtype, void* ws, size_t ws_bytes, cudaStream_t stream) {
  pc::clear_error();
  PC_TRY(pc::check_la(B, T, H, Dk, Dv, dtype));
  if (B == 0) return PC_OK;
  PC_CHECK(strides && log_decay, PC_ERR_NULL, "strides and log_decay must not be NULL");
  if (T > 0) {
    PC_TRY(pc::check_tensor("q", q, dtype));
    PC_TRY(pc::check_tensor("k", k, dtype));
    PC_TRY(pc::check_tensor("v", v, dtype));
    PC_TRY(pc::check_tensor("o", o, dtype));
    PC_TRY(pc::check_apart("o", o, "q", q));
    PC_TRY(pc::check_apart("o", o, "k", k));
    PC_TRY(pc::check_apart("o", o, "v", v));
    const int dims[3] = {B, T, H};
    PC_TRY(pc::check_stored_once("o", strides + 9, dims, 3));
  }
  if (state) PC_TRY(pc::check_apart("state_out", state_out, "state", state));
  pc::LaArgs a{};
  a.B = B;
  a.T = T;
  a.H = H;
  a.log_decay = log_decay;
  a.lengths = lengths;
  a.pass[0] = pc::make_pass(q, strides, k, strides + 3, v, strides + 6, o, strides + 9, Dk, Dv, state, state_out,
                            false, false, scale);
  return pc::run_passes(a, 1, dtype, ws, ws_bytes, stream);
}

pc_status_t pc_linear_attention_bwd(int B, int T, int H, int Dk, int Dv, const void* q, const void* k, const void* v,
                                    const void* d_o, const long long* strides, const float* log_decay, float scale,
                                    const float* state, const float* dstate_out, const int32_t* lengths, void* dq,
                                    void* dk, void* dv, float* dstate, pc_dtype_t dtype, void* ws, size_t ws_bytes,
                                    cudaStream_t stream) {
  pc::clear_error();
  PC_TRY(pc::check_la(B, T, H, Dk, Dv, dtype));
  if (B == 0) return PC_OK;
  PC_CHECK(strides && log_decay, PC_ERR_NULL, "strides and log_decay must not be NULL");
  if (T > 0) {
    const char* names[7] = {"q", "k", "v", "do", "dq", "dk", "dv"};
    const void* all[7] = {q, k, v, d_o, dq, dk, dv};
    for (int i = 0; i < 7; ++i) PC_TRY(pc::check_tensor(names[i], all[i], dtype));
    for (int i = 4; i < 7; ++i)
      for (int j = 0; j < i; ++j) PC_TRY(pc::check_apart(names[i], all[i], names[j], all[j]));
    const int dims[3] = {B, T, H};
    for (int i = 4; i < 7; ++i) PC_TRY(pc::check_stored_once(names[i], strides + 3 * i, dims, 3));
  }
  if (dstate) {
    PC_TRY(pc::check_apart("dstate", dstate, "dstate_out", dstate_out));
    PC_TRY(pc::check_apart("dstate", dstate, "state", state));
  }
  const long long *qs = strides, *ks = strides + 3, *vs = strides + 6, *gs = strides + 9;
  pc::LaArgs a{};
  a.B = B;
  a.T = T;
  a.H = H;
  a.log_decay = log_decay;
  a.lengths = lengths;
  a.pass[0] = pc::make_pass(d_o, gs, v, vs, k, ks, dq, strides + 12, Dv, Dk, state, nullptr, true, false, scale);
  a.pass[1] = pc::make_pass(v, vs, d_o, gs, q, qs, dk, strides + 15, Dv, Dk, dstate_out, nullptr, true, true, scale);
  a.pass[2] = pc::make_pass(k, ks, q, qs, d_o, gs, dv, strides + 18, Dk, Dv, dstate_out, dstate, false, true, scale);
  return pc::run_passes(a, 3, dtype, ws, ws_bytes, stream);
}

pc_status_t pc_linear_attention_step(int B, int H, int Dk, int Dv, const void* q, const void* k, const void* v,
                                     const long long* strides, const float* log_decay, float scale, float* state,
                                     void* o, pc_dtype_t dtype, cudaStream_t stream) {
  pc::clear_error();
  PC_TRY(pc::check_la(B, 1, H, Dk, Dv, dtype));
  if (B == 0) return PC_OK;
  PC_CHECK(strides && log_decay && state, PC_ERR_NULL, "strides, log_decay and state must not be NULL");
  PC_TRY(pc::check_tensor("q", q, dtype));
  PC_TRY(pc::check_tensor("k", k, dtype));
  PC_TRY(pc::check_tensor("v", v, dtype));
  PC_TRY(pc::check_tensor("o", o, dtype));
  const int dims[2] = {B, H};
  PC_TRY(pc::check_stored_once("o", strides + 6, dims, 2));
  if (dtype == PC_BF16)
    pc::launch_step<__nv_bfloat16>(B, H, Dk, Dv, q, k, v, strides, log_decay, scale, state, o, stream);
  else
    pc::launch_step<float>(B, H, Dk, Dv, q, k, v, strides, log_decay, scale, state, o, stream);
  PC_LAUNCH_CHECK();
  return PC_OK;
}

}  // extern "C"

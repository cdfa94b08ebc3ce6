// One pass of the linear attention (see linear_attention.cu) on the tensor cores: bf16
// elements, head sizes padded to 64 or 128, chunks of C = 128 tokens.
//
// A CTA walks the chunks of one (b, h, segment) with the state in registers:
//
//   scores  P  = Q K^T            A = Q, B = K (both K-major shared memory)
//   inter   O  = Q S              B = S^T, bf16 rows written by the state warps
//   intra   O += (P . L) V        A = the decayed scores in tensor memory, B = V (MN-major)
//   update  D  = (V w)^T K        A = V^T times the tokens' weights in tensor memory,
//                                 B = K (MN-major); S^T <- l^m S^T + D
//
// V w is a float32 product: it enters as three bf16 parts (24 bits), so that the state has
// float32 accuracy; D is summed over one chunk only and added to S in registers with
// round-to-nearest adds, because the tensor core's accumulator truncates. Scores and the S
// that the queries read are rounded to bf16, once each, below the rounding of O.
//
//   warps 0-3    one row of the tile per thread: decay of the scores, O to global memory
//   warps 4-11   one row of S^T per thread, the eight warps splitting the tokens (of V^T)
//                and the columns (of S^T) in two halves
//   warp 12      TMA: Q, K, V tiles of 128 tokens, two stages (96 KB each at head size 128)
//   warp 13      MMA issuer
//   warp 14      TMA store of O, staged in the place of the V tile it was made from
// The state warps hold 64 floats of S^T beside 32 packed products each: setmaxnreg gives them
// 168 registers, out of what the others leave of the launch's 4 x 128 (104, 72).
//
// Segments: with fewer (b, h) than SMs a sequence is cut; a first launch (kStates) leaves
// each segment's own contribution to the state, and each segment of the second adds up the
// ones before it.
#pragma once

#include "linear_attention.cuh"

namespace pc {

constexpr int kTcC = 128;
constexpr int kTcThreads = 16 * 32;
constexpr int kTcStages = 2;

struct LaMaps {
  CUtensorMap q, k, v, o;
  int q_ext[2], k_ext[2], v_ext[2], o_ext[2];  // 1: the map has this head / batch dimension, 0: shared
};

struct LaTcArgs {
  LaArgs a;
  LaMaps maps[3];
  float* partial;      // [pass][B*H][segments - 1][DK][DV]
  int segments, chunks_per_segment;
  unsigned* status;
};

template <int DK, int DV>
struct TcShape {
  static constexpr uint32_t kQBytes = kTcC * DK * 2, kVBytes = kTcC * DV * 2;
  static constexpr uint32_t kStage = 2 * kQBytes + kVBytes;
  static constexpr uint32_t kSBytes = DV * DK * 2;
  static constexpr uint32_t kFixed = kTcStages * kStage + kSBytes;
  static constexpr uint32_t kTables = 2048;
  static constexpr uint32_t kBytes = kFixed + kTables + 1024;
  static_assert(kBytes <= 232448, "shared memory per CTA");
  // tensor memory columns
  static constexpr uint32_t kScore = 0;           // float scores; the decayed ones, packed, in its lower half
  static constexpr uint32_t kLow = 64;            // third part of V w, once the scores have been read
  static constexpr uint32_t kOut = 128;
  static constexpr uint32_t kDelta = 256;
  static constexpr uint32_t kHigh = 384, kMid = 448;
};

template <int kRegs>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Tiles' rows along tokens, first coordinate of the tile of `step`, its missing rows.
struct TcTile {
  int t0, pad;
};
__device__ __forceinline__ TcTile tc_tile(int step, int nch, int len, int reverse) {
  const int tile = reverse ? nch - 1 - step : step;
  const int t0 = len - (nch - tile) * kTcC;
  return {t0, t0 < 0 ? -t0 : 0};
}

template <int DK, int DV, bool kStates>
__global__ void __launch_bounds__(kTcThreads, 1) k_la_tc(const __grid_constant__ LaTcArgs args) {
  using S = TcShape<DK, DV>;
  constexpr int C = kTcC;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_tile = smem + kTcStages * S::kStage;
  float* tables = reinterpret_cast<float*>(smem + S::kFixed);
  float* pw = tables;                // l^n, n = 0 .. C
  float* wt = tables + C + 4;        // weights of a full tile's tokens in the state
  float* near = wt + C;              // c_intra l^(distance) from column j to the block's near edge, j = 0 .. 31
  float* diag = near + 32 + 32;      // c_intra l^|d| at diag[d], d = -31 .. 31 (column - row)
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kFixed + (2 * C + 4 + 128) * sizeof(float));
  uint64_t *qk_full = bars, *v_full = bars + 2, *empty = bars + 4, *sc_full = bars + 6, *oi_full = bars + 7,
           *o_full = bars + 8, *d_full = bars + 9, *p_ready = bars + 10, *sc_read = bars + 11, *o_free = bars + 12,
           *vh_ready = bars + 13, *vl_ready = bars + 14, *s_ready = bars + 15, *mma_done = bars + 16, *o_staged = bars + 17;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 18);

  const LaArgs& a = args.a;
  const LaPass& p = a.pass[blockIdx.z];
  const int bh = blockIdx.x, b = bh / a.H, h = bh % a.H, seg = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = la_length(a, b), nch = (len + C - 1) / C;
  const int first = seg * args.chunks_per_segment;
  const int last = min(first + args.chunks_per_segment, nch);  // the steps [first, last) are this CTA's
  const int final_seg = nch > 0 ? (nch - 1) / args.chunks_per_segment : 0;
  const int n_steps = last - first;
  if constexpr (kStates) {
    if (seg >= final_seg) return;  // nothing follows: not read
  }
  const float g = a.log_decay[h];
  unsigned* status = args.status;

  if constexpr (!kStates) {  // rows past the length hold zeros
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + b * p.os[0] + h * p.os[2];
    const int pieces = p.dv / 8;
    const long long n = static_cast<long long>(a.T - len) * pieces;
    for (long long e = static_cast<long long>(seg) * kTcThreads + threadIdx.x; e < n;
         e += static_cast<long long>(args.segments) * kTcThreads)
      *reinterpret_cast<uint4*>(o + (len + e / pieces) * p.os[1] + (e % pieces) * 8) = make_uint4(0u, 0u, 0u, 0u);
    if (seg > final_seg || (n_steps <= 0 && !p.s_out)) return;
  }

  {
    const int i = threadIdx.x;
    if (i <= C) pw[i] = decay_pow(g, i);
    if (i < C) wt[i] = p.c_up * decay_pow(g, p.reverse ? i + 1 : C - 1 - i);
    if (i < 32) near[i] = p.c_intra * decay_pow(g, p.reverse ? i : 31 - i);
    if (i < 63) diag[i - 31] = p.c_intra * decay_pow(g, i < 31 ? 31 - i : i - 31);
  }
  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < 10; ++i)
        if (kStates || (i != 4 && i != 5)) mbar_init(&bars[i], 1);
      mbar_init(p_ready, 4);
      mbar_init(sc_read, 4);
      mbar_init(o_free, 4);
      mbar_init(vh_ready, 8);
      mbar_init(vl_ready, 8);
      mbar_init(s_ready, 8);
      mbar_init(mma_done, 1);
      mbar_init(o_staged, 4);
      if constexpr (!kStates) {  // a stage is free once its products are done and O has left it
        mbar_init(&empty[0], 2);
        mbar_init(&empty[1], 2);
      }
      fence_barrier_init();
    }
    __syncwarp();
    tmem_alloc(tmem_slot, 512);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto stage = [&](int n) { return smem + (n % kTcStages) * S::kStage; };  // Q, then K, then V

  if (warp < 4) {
    regs_down<104>();
    if constexpr (!kStates) {
      // ----------------------------------------------- scores and outputs, row i per thread
      const int quarter = warp & 3, i = quarter * 32 + lane;
      const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + b * p.os[0] + h * p.os[2];
      for (int n = 0; n < n_steps; ++n) {
        const uint32_t ph = n & 1;
        const TcTile tile = tc_tile(first + n, nch, len, p.reverse);
        if (!__all_sync(0xffffffffu, mbar_wait(sc_full, ph, status, kErrTimeoutEpilogue))) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < C / 32; ++c) {
          uint32_t packed[16];
          const bool past = p.reverse ? c > quarter : c < quarter;
          if (past || c == quarter) {
            float v[32];
            tmem_ld_32x32(lanes + S::kScore + c * 32, v);
            if (c == quarter) {
              const int sign = p.reverse ? 1 : -1;
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const float x = v[j] * diag[j - lane];
                v[j] = (j - lane) * sign >= 0 ? x : 0.f;
              }
            } else {
              // l^gap = l^(from the row to the block's near edge) l^(from there to the column)
              const float edge = pw[p.reverse ? c * 32 - i : i - c * 32 - 31];
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                const float4 w = *reinterpret_cast<const float4*>(near + j);
                mul2(v[j], v[j + 1], edge * w.x, edge * w.y);
                mul2(v[j + 2], v[j + 3], edge * w.z, edge * w.w);
              }
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) packed[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) packed[j] = 0u;
          }
          // columns that this warp has read already
          tmem_st_32x16(lanes + S::kScore + c * 16, packed);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sc_read);
        if (!__all_sync(0xffffffffu, mbar_wait(oi_full, ph, status, kErrTimeoutEpilogue))) break;
        tc_fence_after();
        const float inter = pw[p.reverse ? C - 1 - i : max(i - tile.pad + 1, 0)] * p.c_inter;
#pragma unroll 1
        for (int c = 0; c < DV; c += 32) {
          float v[32];
          tmem_ld_32x32(lanes + S::kOut + c, v);
#pragma unroll
          for (int j = 0; j < 32; j += 2) mul2(v[j], v[j + 1], inter, inter);
          tmem_st_32x32(lanes + S::kOut + c, v);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready);
        if (!__all_sync(0xffffffffu, mbar_wait(o_full, ph, status, kErrTimeoutEpilogue))) break;
        tc_fence_after();
        // a whole tile goes through shared memory in rows of 128 swizzled bytes, one that starts
        // before the sequence (no store may) straight to global memory
        __nv_bfloat16* row = o + (tile.t0 + i) * p.os[1];
        uint8_t* staged = stage(n) + 2 * S::kQBytes + i * 128;
#pragma unroll 1
        for (int c = 0; c < DV; c += 32) {
          float v[32];
          tmem_ld_32x32(lanes + S::kOut + c, v);
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            const uint4 x = make_uint4(pack_bf16x2(v[j], v[j + 1]), pack_bf16x2(v[j + 2], v[j + 3]),
                                       pack_bf16x2(v[j + 4], v[j + 5]), pack_bf16x2(v[j + 6], v[j + 7]));
            if (tile.pad == 0)
              *reinterpret_cast<uint4*>(staged + (c / 64) * C * 128 + (((((c + j) % 64) / 8) ^ (i & 7)) << 4)) = x;
            else if (i >= tile.pad && c + j < p.dv)
              *reinterpret_cast<uint4*>(row + c + j) = x;
          }
        }
        fence_async_shared();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(o_free);
          mbar_arrive(o_staged);
        }
      }
    }
  } else if (warp < 12) {
    regs_up<168>();
    // --------------------------------------------------- the state, row r of S^T per thread
    constexpr int kCols = DK / 2, kToks = C / 2, kUnits = kToks / 16 * 2;
    const int quarter = warp & 3, r = quarter * 32 + lane, part = (warp - 4) >> 2;
    const bool active = quarter * 32 < DV;  // a warp with rows of S^T
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    float s[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) s[c] = 0.f;
    if constexpr (!kStates) {
      const long long size = static_cast<long long>(p.dk) * p.dv;
      if (p.s_in && r < p.dv) {
        const float* in = p.s_in + bh * size;
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const int d = part * kCols + c;
          if (d < p.dk) s[c] = p.s_in_transposed ? in[static_cast<long long>(r) * p.dk + d] : in[d * p.dv + r];
        }
      }
      // what the segments before this one add
      const float* ps = args.partial + (static_cast<long long>(blockIdx.z) * a.B * a.H + bh) *
                                           (args.segments - 1) * (DK * DV);
      for (int e = 0; e < seg; ++e, ps += DK * DV) {
        const int at = e * args.chunks_per_segment;
        int toks = args.chunks_per_segment * C;
        if (!p.reverse && at == 0) toks -= tc_tile(0, nch, len, 0).pad;
        const float carry = decay_pow(g, toks);
        if (active) {
#pragma unroll
          for (int c = 0; c < kCols; ++c) s[c] = carry * s[c] + ps[(part * kCols + c) * DV + r];
        }
      }
    }
    // this lane's row of the four 8 x 8 blocks of a unit: blocks 0, 1 the first eight tokens,
    // 0, 2 the first eight rows of V^T
    const int v_row = (lane & 7) + (lane & 16) / 2, v_piece = (lane >> 3) & 1;
    auto publish = [&]() {  // S^T in bf16, K-major rows of 128 bytes, swizzled
      if (active) {
#pragma unroll
        for (int c = 0; c < kCols; c += 8) {
          const int d = part * kCols + c;
          uint8_t* dst = s_tile + (d / 64) * DV * 128 + r * 128 + ((((d % 64) / 8) ^ (r & 7)) << 4);
          *reinterpret_cast<uint4*>(dst) =
              make_uint4(pack_bf16x2(s[c], s[c + 1]), pack_bf16x2(s[c + 2], s[c + 3]),
                         pack_bf16x2(s[c + 4], s[c + 5]), pack_bf16x2(s[c + 6], s[c + 7]));
        }
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_ready);
    };
    if constexpr (!kStates) publish();
    bool ok = true;
    for (int n = 0; n < n_steps; ++n) {
      const uint32_t ph = n & 1;
      const TcTile tile = tc_tile(first + n, nch, len, p.reverse);
      ok = __all_sync(0xffffffffu, mbar_wait(&v_full[n % kTcStages], (n / kTcStages) & 1, status, kErrTimeoutEpilogue));
      if (!ok) break;
      uint32_t low[kUnits][4];
      if (active) {
        // Units of 16 tokens x 16 rows of V^T: ldmatrix transposes four 8 x 8 blocks into the
        // layout of the 16-lane store, a register holding two consecutive tokens of one row.
        const uint32_t v = smem_addr(stage(n)) + 2 * S::kQBytes + (quarter / 2) * C * 128 + v_row * 128;
        // a reversed tile's missing rows hold zeros, and its weights count from the first real one
        const float* w = wt - (p.reverse ? tile.pad : 0) + part * kToks + 2 * (lane & 3);
        const int first_tok = p.reverse ? tile.pad : 0;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
          const int tok = part * kToks + (u / 2) * 16;  // the unit's first token
          uint32_t x[4];
          ldmatrix_x4_trans(v + tok * 128 + (((quarter & 1) * 4 + (u & 1) * 2 + v_piece) ^ (v_row & 7)) * 16, x);
          float2 ww[2];
          if (tok >= first_tok) {
            ww[0] = make_float2(w[(u / 2) * 16], w[(u / 2) * 16 + 1]);
            ww[1] = make_float2(w[(u / 2) * 16 + 8], w[(u / 2) * 16 + 9]);
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int t = tok + 8 * e + 2 * (lane & 3);
              ww[e].x = t >= first_tok ? w[(u / 2) * 16 + 8 * e] : 0.f;
              ww[e].y = t + 1 >= first_tok ? w[(u / 2) * 16 + 8 * e + 1] : 0.f;
            }
          }
          uint32_t high[4], mid[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float a0 = __uint_as_float(x[e] << 16), a1 = __uint_as_float(x[e] & 0xFFFF0000u);
            mul2(a0, a1, ww[e / 2].x, ww[e / 2].y);
            high[e] = pack_bf16x2(a0, a1);
            sub2_bf16(a0, a1, high[e]);
            mid[e] = pack_bf16x2(a0, a1);
            sub2_bf16(a0, a1, mid[e]);
            low[u][e] = pack_bf16x2(a0, a1);
          }
          const uint32_t at = lanes + (static_cast<uint32_t>((u & 1) * 16) << 16) + tok / 2;
          tmem_st_16x128_x2(at + S::kHigh, high);
          tmem_st_16x128_x2(at + S::kMid, mid);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(vh_ready);
      if constexpr (!kStates) {  // the third part takes the place of scores already read
        ok = __all_sync(0xffffffffu, mbar_wait(sc_read, ph, status, kErrTimeoutEpilogue));
        if (!ok) break;
        tc_fence_after();
      }
      if (active) {
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
          tmem_st_16x128_x2(lanes + (static_cast<uint32_t>((u & 1) * 16) << 16) + S::kLow +
                                (part * kToks + (u / 2) * 16) / 2,
                            low[u]);
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(vl_ready);
      ok = __all_sync(0xffffffffu, mbar_wait(d_full, ph, status, kErrTimeoutEpilogue));
      if (!ok) break;
      tc_fence_after();
      if (active) {
        const float carry = pw[C - tile.pad];
#pragma unroll
        for (int c = 0; c < kCols; c += 32) {
          float d[32];
          tmem_ld_32x32(lanes + S::kDelta + part * kCols + c, d);
#pragma unroll
          for (int j = 0; j < 32; j += 2) fma2(s[c + j], s[c + j + 1], carry, d[j], d[j + 1]);
        }
        tc_fence_before();
      }
      if constexpr (!kStates) {
        if (n + 1 < n_steps) publish();
      }
    }
    if (ok) {
      if constexpr (kStates) {
        float* out = args.partial + ((static_cast<long long>(blockIdx.z) * a.B * a.H + bh) * (args.segments - 1) +
                                     seg) * (DK * DV);
        if (active) {
#pragma unroll
          for (int c = 0; c < kCols; ++c) out[(part * kCols + c) * DV + r] = s[c];
        }
      } else if (p.s_out && seg == final_seg && r < p.dv) {
        float* out = p.s_out + bh * static_cast<long long>(p.dk) * p.dv;
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const int d = part * kCols + c;
          if (d < p.dk) out[d * p.dv + r] = s[c];
        }
      }
    }
  } else {
    regs_down<72>();
    if (warp == 12 && lane == 0) {
      // ------------------------------------------------------------ TMA producer
      const LaMaps& m = args.maps[blockIdx.z];
      int issued = 0;
      for (int n = 0; n < n_steps; ++n) {
        const int st = n % kTcStages;
        const uint32_t ph = (n / kTcStages) & 1;
        if (!mbar_wait(&empty[st], ph ^ 1, status, kErrTimeoutProducer)) break;
        const int t0 = tc_tile(first + n, nch, len, p.reverse).t0;
        uint8_t* base = stage(n);
        mbar_arrive_expect_tx(&qk_full[st], kStates ? S::kQBytes : 2 * S::kQBytes);
#pragma unroll
        for (int x = 0; x < DK; x += 64) {
          if constexpr (!kStates)
            tma_load_4d(base + x * C * 2, &m.q, &qk_full[st], x, t0, h * m.q_ext[0], b * m.q_ext[1]);
          tma_load_4d(base + S::kQBytes + x * C * 2, &m.k, &qk_full[st], x, t0, h * m.k_ext[0], b * m.k_ext[1]);
        }
        mbar_arrive_expect_tx(&v_full[st], S::kVBytes);
#pragma unroll
        for (int x = 0; x < DV; x += 64)
          tma_load_4d(base + 2 * S::kQBytes + x * C * 2, &m.v, &v_full[st], x, t0, h * m.v_ext[0], b * m.v_ext[1]);
        issued = n + 1;
      }
      for (int n = issued > kTcStages ? issued - kTcStages : 0; n < issued; ++n) {
        mbar_wait(&qk_full[n % kTcStages], (n / kTcStages) & 1, status, kErrTimeoutDrain);
        mbar_wait(&v_full[n % kTcStages], (n / kTcStages) & 1, status, kErrTimeoutDrain);
      }
    }
    if (!kStates && warp == 14 && lane == 0) {
      // ------------------------------------------------------------ TMA store of O
      const LaMaps& m = args.maps[blockIdx.z];
      for (int n = 0; n < n_steps; ++n) {
        const TcTile tile = tc_tile(first + n, nch, len, p.reverse);
        if (!mbar_wait(o_staged, n & 1, status, kErrTimeoutEpilogue)) break;
        if (tile.pad == 0) {
#pragma unroll
          for (int x = 0; x < DV; x += 64)
            tma_store_4d(&m.o, stage(n) + 2 * S::kQBytes + x * C * 2, x, tile.t0, h * m.o_ext[0], b * m.o_ext[1]);
          bulk_commit_wait_read();
        }
        mbar_arrive(&empty[n % kTcStages]);
      }
    }
    if (warp == 13) {
      // ----------------- MMA issuer: the whole warp in step (uniform addresses), one lane issues
      constexpr uint32_t idesc_qk = umma_idesc(1, 128, C);
      constexpr uint32_t idesc_qs = umma_idesc(1, 128, DV);
      constexpr uint32_t idesc_pv = umma_idesc(1, 128, DV) | kIdescBMN;
      constexpr uint32_t idesc_up = umma_idesc(1, 128, DK) | kIdescBMN;
      const bool leader = elect_one();
      auto wait = [&](uint64_t* bar, uint32_t ph) {
        const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, ph, status, kErrTimeoutMma));
        tc_fence_after();
        return ok;
      };
      const uint32_t base = smem_addr(smem);
      const uint64_t s_desc = umma_desc_sw128(base + kTcStages * S::kStage);
      for (int n = 0; n < n_steps; ++n) {
        const int st = n % kTcStages;
        const uint32_t ph = n & 1, sph = (n / kTcStages) & 1;
        const uint32_t q_addr = base + st * S::kStage;
        const uint64_t q_desc = umma_desc_sw128(q_addr), k_desc = umma_desc_sw128(q_addr + S::kQBytes);
        const uint64_t k_rows = umma_desc_sw128_mn(q_addr + S::kQBytes, C * 128);
        const uint64_t v_rows = umma_desc_sw128_mn(q_addr + 2 * S::kQBytes, C * 128);
        auto update = [&](uint32_t a_col, bool fresh) {  // D (+)= A K over the chunk's tokens
#pragma unroll
          for (int kk = 0; kk < C / 16; ++kk)
            umma_bf16_ts(tmem + S::kDelta, tmem + a_col + kk * 8, k_rows + kk * (2048 >> 4), idesc_up,
                         fresh && kk == 0 ? 0u : 1u);
        };
        if (!wait(&qk_full[st], sph)) break;
        if constexpr (!kStates) {
          // the score columns hold the last chunk's operands until its products are done
          if (n > 0 && !wait(d_full, ph ^ 1)) break;
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < DK / 16; ++kk) {
              const uint32_t off = ((kk / 4) * C * 128 + (kk % 4) * 32) >> 4;
              umma_bf16(tmem + S::kScore, q_desc + off, k_desc + off, idesc_qk, kk ? 1u : 0u);
            }
            umma_commit(sc_full);
          }
          __syncwarp();
          if (!wait(s_ready, ph) || (n > 0 && !wait(o_free, ph ^ 1))) break;
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < DK / 16; ++kk)
              umma_bf16(tmem + S::kOut, q_desc + (((kk / 4) * C * 128 + (kk % 4) * 32) >> 4),
                        s_desc + (((kk / 4) * DV * 128 + (kk % 4) * 32) >> 4), idesc_qs, kk ? 1u : 0u);
            umma_commit(oi_full);
          }
          __syncwarp();
        }
        if (!wait(vh_ready, ph)) break;
        if constexpr (kStates) {
          if (!wait(vl_ready, ph)) break;
          if (leader) {
            update(S::kLow, true);  // the small part first: its sums lose least
            update(S::kMid, false);
            update(S::kHigh, false);
          }
        } else {
          if (leader) {
            update(S::kMid, true);
            update(S::kHigh, false);
          }
          __syncwarp();
          if (!wait(p_ready, ph) || !wait(&v_full[st], sph)) break;
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < C / 16; ++kk)
              umma_bf16_ts(tmem + S::kOut, tmem + S::kScore + kk * 8, v_rows + kk * (2048 >> 4), idesc_pv, 1u);
            umma_commit(o_full);
          }
          __syncwarp();
          if (!wait(vl_ready, ph)) break;
          if (leader) update(S::kLow, false);
        }
        if (leader) {
          umma_commit(d_full);
          umma_commit(&empty[st]);
        }
        __syncwarp();
      }
      if (leader) umma_commit(mma_done);
      __syncwarp();
      mbar_wait(mma_done, 0, status, kErrTimeoutDrain);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace pc

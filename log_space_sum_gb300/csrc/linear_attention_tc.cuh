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
  CUtensorMap q, k, v;
  int q_ext[2], k_ext[2], v_ext[2];  // 1: the map has this head / batch dimension, 0: shared
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
  float* pw0 = reinterpret_cast<float*>(smem + S::kFixed);  // l^n at pw[n], n = 0 .. C; 1 below
  float* pw = pw0 + C;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kFixed + (2 * C + 4) * sizeof(float));
  uint64_t *qk_full = bars, *v_full = bars + 2, *empty = bars + 4, *sc_full = bars + 6, *oi_full = bars + 7,
           *o_full = bars + 8, *d_full = bars + 9, *p_ready = bars + 10, *sc_read = bars + 11, *o_free = bars + 12,
           *vh_ready = bars + 13, *vl_ready = bars + 14, *s_ready = bars + 15, *mma_done = bars + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 17);

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

  for (int i = threadIdx.x; i < 2 * C + 1; i += kTcThreads) pw0[i] = i < C ? 1.f : decay_pow(g, i - C);
  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < 10; ++i) mbar_init(&bars[i], 1);
      mbar_init(p_ready, 4);
      mbar_init(sc_read, 4);
      mbar_init(o_free, 4);
      mbar_init(vh_ready, 8);
      mbar_init(vl_ready, 8);
      mbar_init(s_ready, 8);
      mbar_init(mma_done, 1);
      fence_barrier_init();
    }
    __syncwarp();
    tmem_alloc(tmem_slot, 512);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int dir = p.reverse ? 1 : -1;  // the direction of time in which exponents grow
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
            if (c == quarter) {  // l^gap at w[j], 1 where the mask gives 0
              const float* w = pw + (p.reverse ? -lane : lane);
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const float x = v[j] * (w[j * dir] * p.c_intra);
                v[j] = (j - lane) * dir >= 0 ? x : 0.f;
              }
            } else {
              // l^gap = l^(distance to the block's near edge) l^(distance within it)
              const float edge = pw[p.reverse ? c * 32 - i : i - c * 32 - 31] * p.c_intra;
              const float* w = pw + (p.reverse ? 0 : 31);
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] *= edge * w[j * dir];
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
        const float inter = pw[p.reverse ? C - 1 - i : i - tile.pad + 1] * p.c_inter;
#pragma unroll 1
        for (int c = 0; c < DV; c += 32) {
          float v[32];
          tmem_ld_32x32(lanes + S::kOut + c, v);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] *= inter;
          tmem_st_32x32(lanes + S::kOut + c, v);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready);
        if (!__all_sync(0xffffffffu, mbar_wait(o_full, ph, status, kErrTimeoutEpilogue))) break;
        tc_fence_after();
        __nv_bfloat16* row = o + (tile.t0 + i) * p.os[1];
#pragma unroll 1
        for (int c = 0; c < DV; c += 32) {
          float v[32];
          tmem_ld_32x32(lanes + S::kOut + c, v);
          if (i >= tile.pad) {
#pragma unroll
            for (int j = 0; j < 32; j += 8)
              if (c + j < p.dv)
                *reinterpret_cast<uint4*>(row + c + j) =
                    make_uint4(pack_bf16x2(v[j], v[j + 1]), pack_bf16x2(v[j + 2], v[j + 3]),
                               pack_bf16x2(v[j + 4], v[j + 5]), pack_bf16x2(v[j + 6], v[j + 7]));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_free);
      }
    }
  } else if (warp < 12) {
    regs_up<168>();
    // --------------------------------------------------- the state, row r of S^T per thread
    constexpr int kCols = DK / 2, kToks = C / 2;
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
      uint32_t low[kToks / 2];
      if (active) {
        // column r of V: row t at t * 128 bytes, its 16-byte piece swizzled by t
        const uint8_t* v = stage(n) + 2 * S::kQBytes + (r / 64) * C * 128 + part * kToks * 128 + (r & 7) * 2;
        const int piece = (r % 64) / 8;
        const float* w = p.reverse ? pw + 1 - tile.pad + part * kToks : pw + C - 1 - part * kToks;
#pragma unroll
        for (int t0 = 0; t0 < kToks; t0 += 32) {
          uint32_t high[16], mid[16];
#pragma unroll
          for (int t = 0; t < 32; t += 2) {
            float x[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int tt = t0 + t + e;
              const uint32_t bits = *reinterpret_cast<const uint16_t*>(v + tt * 128 + ((piece ^ (tt & 7)) << 4));
              x[e] = __uint_as_float(bits << 16) * w[tt * dir];
            }
            const uint32_t hi = pack_bf16x2(x[0], x[1]);
            x[0] -= __uint_as_float(hi << 16);
            x[1] -= __uint_as_float(hi & 0xFFFF0000u);
            const uint32_t mi = pack_bf16x2(x[0], x[1]);
            x[0] -= __uint_as_float(mi << 16);
            x[1] -= __uint_as_float(mi & 0xFFFF0000u);
            high[t / 2] = hi;
            mid[t / 2] = mi;
            low[(t0 + t) / 2] = pack_bf16x2(x[0], x[1]);
          }
          tmem_st_32x16(lanes + S::kHigh + (part * kToks + t0) / 2, high);
          tmem_st_32x16(lanes + S::kMid + (part * kToks + t0) / 2, mid);
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
        for (int t0 = 0; t0 < kToks / 2; t0 += 16) {
          uint32_t x[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = low[t0 + e];
          tmem_st_32x16(lanes + S::kLow + part * (kToks / 2) + t0, x);
        }
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
          for (int j = 0; j < 32; ++j) s[c + j] = carry * s[c + j] + p.c_up * d[j];
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
    if (warp == 13 && lane == 0) {
      // -------------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc_qk = umma_idesc(1, 128, C);
      constexpr uint32_t idesc_qs = umma_idesc(1, 128, DV);
      constexpr uint32_t idesc_pv = umma_idesc(1, 128, DV) | kIdescBMN;
      constexpr uint32_t idesc_up = umma_idesc(1, 128, DK) | kIdescBMN;
      auto wait = [&](uint64_t* bar, uint32_t ph) {
        const bool ok = mbar_wait(bar, ph, status, kErrTimeoutMma);
        tc_fence_after();
        return ok;
      };
      const uint32_t s_addr = smem_addr(s_tile);
      for (int n = 0; n < n_steps; ++n) {
        const int st = n % kTcStages;
        const uint32_t ph = n & 1, sph = (n / kTcStages) & 1;
        const uint32_t q_addr = smem_addr(stage(n)), k_addr = q_addr + S::kQBytes, v_addr = k_addr + S::kQBytes;
        auto update = [&](uint32_t a_col, bool fresh) {  // D (+)= A K over the chunk's tokens
#pragma unroll
          for (int kk = 0; kk < C / 16; ++kk)
            umma_bf16_ts(tmem + S::kDelta, tmem + a_col + kk * 8, umma_desc_sw128_mn(k_addr + kk * 2048, C * 128),
                         idesc_up, fresh && kk == 0 ? 0u : 1u);
        };
        if (!wait(&qk_full[st], sph)) break;
        if constexpr (!kStates) {
          // the score columns hold the last chunk's operands until its products are done
          if (n > 0 && !wait(d_full, ph ^ 1)) break;
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk) {
            const uint32_t off = (kk / 4) * C * 128 + (kk % 4) * 32;
            umma_bf16(tmem + S::kScore, umma_desc_sw128(q_addr + off), umma_desc_sw128(k_addr + off), idesc_qk,
                      kk ? 1u : 0u);
          }
          umma_commit(sc_full);
          if (!wait(s_ready, ph) || (n > 0 && !wait(o_free, ph ^ 1))) break;
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk)
            umma_bf16(tmem + S::kOut, umma_desc_sw128(q_addr + (kk / 4) * C * 128 + (kk % 4) * 32),
                      umma_desc_sw128(s_addr + (kk / 4) * DV * 128 + (kk % 4) * 32), idesc_qs, kk ? 1u : 0u);
          umma_commit(oi_full);
        }
        if (!wait(vh_ready, ph)) break;
        if constexpr (kStates) {
          if (!wait(vl_ready, ph)) break;
          update(S::kLow, true);  // the small part first: its sums lose least
          update(S::kMid, false);
          update(S::kHigh, false);
        } else {
          update(S::kMid, true);
          update(S::kHigh, false);
          if (!wait(p_ready, ph) || !wait(&v_full[st], sph)) break;
#pragma unroll
          for (int kk = 0; kk < C / 16; ++kk)
            umma_bf16_ts(tmem + S::kOut, tmem + S::kScore + kk * 8, umma_desc_sw128_mn(v_addr + kk * 2048, C * 128),
                         idesc_pv, 1u);
          umma_commit(o_full);
          if (!wait(vl_ready, ph)) break;
          update(S::kLow, false);
        }
        umma_commit(d_full);
        umma_commit(&empty[st]);
      }
      umma_commit(mma_done);
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

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
// The weights w are float32, so V w takes four bf16 parts: with w = wh + wm + wl (8 bits each),
// v wh = p1 + r1 and v wm = p2 + r2 exactly for p = rn(v w), r = fma(v, w, -p), and the parts are
// p1, r1, p2 and rn(v wl + r2), one packed bf16 instruction each: the state has float32
// accuracy. D is summed over one chunk only and added to S in registers with round-to-nearest
// adds, because the tensor core's accumulator truncates. Scores and the S
// that the queries read are rounded to bf16, once each, below the rounding of O.
//
//   warps 0-3    one row of the tile per thread: the decay of the scores and of Q S
//   warps 4-7    one row of the tile per thread: O, staged in the place of the V tile it was
//                made from
//   warps 8-15   one row of S^T per thread: the parts of V^T w, in groups of 32 tokens (kStates:
//                64; the first four warps the first half of them), then half of S^T's
//                columns each
//   warp 16      TMA: Q, K, V tiles of 128 tokens, two stages (96 KB each at head size 128),
//                kStates three of K and V
//   warp 17      MMA issuer
//   warp 18      TMA store of O
// The state warps hold 64 floats of S^T each: setmaxnreg gives them 128 registers, out of what
// the others leave of the launch's 5 x 96 (2 x 80, 64; kStates: 168, 2 x 24, 64). A spill would cost more than
// elsewhere: the tiles leave the L1 cache next to nothing.
//
// A chunk of 128 tokens at head size 128 takes 3.1 us (5800 cycles), 4600 cycles of them MMAs: a
// gradient of 8 x 2048 tokens, 16 heads, 163 us on the GPU (384 CTAs in 2.5 waves), 1 x 32771 tokens
// forward 150 us (DRAM at 5.2 TB/s in the pass itself); call after call from Python 167 and 153 to 163.
//
// Segments: with fewer (b, h) than SMs a sequence is cut; a first launch (kStates) leaves
// each segment's own contribution to the state, and each segment of the second adds up the
// ones before it.
#pragma once

#include "linear_attention.cuh"

namespace pc {

constexpr int kTcC = 128;
constexpr int kTcThreads = 20 * 32;

struct LaMaps {
  CUtensorMap q, k, v, o;
  int q_ext[2], k_ext[2], v_ext[2], o_ext[2];  // 1: the map has this head / batch dimension, 0: shared
};

struct LaTcArgs {
  LaArgs a;
  LaMaps maps[3];
  float* partial;      // [pass][B*H][segments - 1][DK][DV]
  int passes, segments, chunks_per_segment;
  unsigned* status;
};

template <int DK, int DV, bool kStates>
struct TcShape {
  static constexpr uint32_t kQBytes = kTcC * DK * 2, kVBytes = kTcC * DV * 2;
  static constexpr uint32_t kK = kStates ? 0 : kQBytes, kV = kK + kQBytes;  // tiles' places in a stage
  static constexpr uint32_t kStage = kV + kVBytes;
  static constexpr int kStages = kStates ? 3 : 2;
  static constexpr uint32_t kSBytes = kStates ? 0 : DV * DK * 2;
  static constexpr uint32_t kFixed = kStages * kStage + kSBytes;
  static constexpr uint32_t kTables = 2064;  // powers and weights (1808 bytes), barriers
  static constexpr uint32_t kBytes = kFixed + kTables + 1008;  // alignment: the base is 16-byte aligned
  static_assert(kBytes <= 232448, "shared memory per CTA");
  // tensor memory columns
  // float scores (128 columns); the decayed ones, packed, then take the first 64
  static constexpr uint32_t kScore = 0;
  static constexpr uint32_t kOut = 128;
  static constexpr uint32_t kDelta = 256;  // kStates: and kOut, in turn
  // the four parts of V^T w for a group of tokens, half a column each per token; two groups in
  // turn (kStates: the second in the scores' place)
  static constexpr uint32_t kParts = 384;
};

// Ends a batch of loads or stores: the addresses of the next are formed after it (all of
// a row's at once would not fit the registers beside the state).
__device__ __forceinline__ void keep_order() { asm volatile("" ::: "memory"); }

template <int kRegs>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Parts wh, wm, wl of the weights of tokens 2i and 2i + 1 of a tile with `pad` missing rows.
__device__ __forceinline__ void weight_parts(uint32_t* wp, int i, float g, const LaPass& p, int pad) {
  float w[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int t = 2 * i + e;
    w[e] = p.c_up * decay_pow(g, p.reverse ? max(t - pad + 1, 0) : kTcC - 1 - t);
  }
#pragma unroll
  for (int part = 0; part < 3; ++part) {
    const uint32_t x = pack_bf16x2(w[0], w[1]);
    sub2_bf16(w[0], w[1], x);
    wp[part * 64 + i] = x;
  }
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
  using S = TcShape<DK, DV, kStates>;
  constexpr int kTcStages = S::kStages;
  constexpr int C = kTcC;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_tile = smem + kTcStages * S::kStage;
  float* tables = reinterpret_cast<float*>(smem + S::kFixed);
  float* pw = tables;                // l^n, n = 0 .. C
  uint32_t* wp = reinterpret_cast<uint32_t*>(tables + C + 4);  // [3][64]: bf16 parts of the tokens' weights, by pairs
  float* near = tables + C + 4 + 192;  // c_intra l^(distance) from column j to the block's near edge, j = 0 .. 31
  float* diag = near + 32 + 32;      // c_intra l^|d| at diag[d], d = -31 .. 31 (column - row)
  uint64_t* spare = reinterpret_cast<uint64_t*>(near + 96);
  auto* limit = reinterpret_cast<unsigned long long*>(spare);  // first_wait_limit
  uint64_t *w_free = spare + 1, *w_ready = spare + 2;          // of a padded tile's weights
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kFixed + (C + 4 + 192 + 128) * sizeof(float));
  auto bar = [&](int at) { return bars + at; };
  uint64_t *q_full = bar(0), *k_full = bar(3), *v_full = bar(6), *q_empty = bar(9), *k_empty = bar(12),
           *v_empty = bar(15), *up_ready = bar(18), *up_free = bar(20), *sc_full = bar(22), *oi_full = bar(23),
           *o_full = bar(24), *d_full = bar(25), *p_ready = bar(26), *o_free = bar(27), *s_ready = bar(28),
           *o_staged = bar(29), *mma_done = bar(30);
  uint64_t* d_free = bar(22);  // kStates: [2], in the place of sc_full and oi_full
  // Of chunk n. kStates: the state warps announce a chunk's operands before they look at the last
  // one's D, so two of these phases can end before a delayed warp looks at the first: two
  // barriers in turn (the other in the place of o_full), of which d_free holds back the next use.
  auto d_done = [&](int n) { return kStates && (n & 1) ? o_full : d_full; };
  auto d_parity = [&](int n) { return static_cast<uint32_t>(kStates ? n >> 1 : n) & 1u; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar(31));

  const LaArgs& a = args.a;
  // the passes of one head run side by side: they read the same tiles, out of L2 but once
  const int pass = blockIdx.x % args.passes, bh = blockIdx.x / args.passes;
  const LaPass& p = a.pass[pass];
  const int b = bh / a.H, h = bh % a.H, seg = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = la_length(a, b), nch = (len + C - 1) / C;
  const int first = seg * args.chunks_per_segment;
  const int last = min(first + args.chunks_per_segment, nch);  // the steps [first, last) are this CTA's
  const int final_seg = nch > 0 ? (nch - 1) / args.chunks_per_segment : 0;
  const int n_steps = last - first;
  if constexpr (kStates) {
    if (seg >= final_seg) return;  // nothing follows: not read
  }
  if constexpr (kStates) grid_dependents_launch();
  const float g = a.log_decay[h];
  unsigned* status = args.status;

  if constexpr (!kStates) {  // rows past the length hold zeros
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + b * p.os[0] + h * p.os[2];
    const int pieces = p.dv / 8;
    const long long n = static_cast<long long>(a.T - len) * pieces;
    for (long long e = static_cast<long long>(seg) * kTcThreads + threadIdx.x; e < n;
         e += static_cast<long long>(args.segments) * kTcThreads)
      *reinterpret_cast<uint4*>(o + (len + e / pieces) * p.os[1] + (e % pieces) * 8) = make_uint4(0u, 0u, 0u, 0u);
    if (seg > final_seg || (n_steps <= 0 && !p.s_out)) {
      la_end_after_states();
      return;
    }
  }

  {
    const int i = threadIdx.x;
    if (i <= C) pw[i] = decay_pow(g, i);
    if (i < C / 2) weight_parts(wp, i, g, p, 0);
    if (i < 32) near[i] = p.c_intra * decay_pow(g, p.reverse ? i : 31 - i);
    if (i < 63) diag[i - 31] = p.c_intra * decay_pow(g, i < 31 ? 31 - i : i - 31);
    if (i == kTcThreads - 1) *limit = first_wait_limit(status);
  }
  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < kTcStages; ++i) {
        mbar_init(&q_full[i], 1);
        mbar_init(&k_full[i], 1);
        mbar_init(&v_full[i], 1);
        mbar_init(&q_empty[i], 1);
        mbar_init(&k_empty[i], 1);
        mbar_init(&v_empty[i], 1);  // its products are done and, where O takes its place, O has left
      }
      mbar_init(sc_full, kStates ? 8 : 1);
      mbar_init(oi_full, kStates ? 8 : 1);
      mbar_init(o_full, 1);
      mbar_init(d_full, 1);
      mbar_init(mma_done, 1);
      mbar_init(p_ready, 4);
      mbar_init(o_free, 4);
      mbar_init(o_staged, 4);
      mbar_init(s_ready, 8);
      mbar_init(&up_ready[0], 8);
      mbar_init(&up_ready[1], 8);
      mbar_init(&up_free[0], 1);
      mbar_init(&up_free[1], 1);
      mbar_init(w_free, 8);
      mbar_init(w_ready, 8);
      fence_barrier_init();
    }
    __syncwarp();
    tmem_alloc(tmem_slot, 512);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  constexpr int kGroup = kStates ? 64 : 32, kGroups = C / kGroup;  // tokens of a group, groups of a tile
  auto d_col = [&](int n) { return kStates && (n & 1) ? S::kOut : S::kDelta; };
  // parity of the use of buffer grp & 1 by group grp of step n
  auto use_parity = [&](int n, int grp) { return static_cast<uint32_t>(n * (kGroups / 2) + (grp >> 1)) & 1u; };
  auto parts = [&](int buf) { return kStates ? (buf ? S::kScore : S::kParts) : S::kParts + buf * 64; };
  auto stage = [&](int n) { return smem + (n % kTcStages) * S::kStage; };  // Q, then K, then V
  // Which waits run out is each warp's own finding: no role waits for another at a barrier without a
  // limit before the CTA's last. The limit that the host may set holds for the waits for products:
  // the roles that they starve run into the default (read by the issuer, it took 8 us of 149 at
  // 1 x 32771 tokens; by every state warp's wait, 3).
  auto wait_products = [&](uint64_t* bar, uint32_t parity) {
    const bool got = __all_sync(0xffffffffu, mbar_wait(bar, parity, status, kErrTimeoutEpilogue, *limit));
    tc_fence_after();
    return got;
  };

  if (warp < 8) {
    regs_down<kStates ? 24 : 80>();
    if constexpr (!kStates) {
      // ----------------------------------------------- scores and outputs, row i per thread
      const int quarter = warp & 3, i = quarter * 32 + lane;
      const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
      if (warp < 4) {
        for (int n = 0; n < n_steps; ++n) {
          const TcTile tile = tc_tile(first + n, nch, len, p.reverse);
          if (!wait_products(sc_full, n & 1)) break;
#pragma unroll 1
          for (int c = 0; c < C / 32; ++c) {
            uint32_t packed[16];
            const bool past = p.reverse ? c > quarter : c < quarter;
            if (past || c == quarter) {
              float v[32];
              tmem_ld_32x32(lanes + S::kScore + c * 32, v);
              if (c == quarter) {
                if (p.reverse) {
#pragma unroll
                  for (int j = 0; j < 32; ++j) v[j] = j >= lane ? v[j] * diag[j - lane] : 0.f;
                } else {
#pragma unroll
                  for (int j = 0; j < 32; ++j) v[j] = j <= lane ? v[j] * diag[j - lane] : 0.f;
                }
              } else {
                // l^gap = l^(from the row to the block's near edge) l^(from there to the column)
                const float edge = pw[p.reverse ? c * 32 - i : i - c * 32 - 31];
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                  const float4 w = *reinterpret_cast<const float4*>(near + j);
                  mul2(v[j], v[j + 1], w.x, w.y);
                  mul2(v[j + 2], v[j + 3], w.z, w.w);
                  mul2(v[j], v[j + 1], edge, edge);
                  mul2(v[j + 2], v[j + 3], edge, edge);
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
          if (!wait_products(oi_full, n & 1)) break;
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
        }
        tmem_wait_st();  // after a wait that ran out
      } else {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + b * p.os[0] + h * p.os[2];
        for (int n = 0; n < n_steps; ++n) {
          const TcTile tile = tc_tile(first + n, nch, len, p.reverse);
          if (!wait_products(o_full, n & 1)) break;
          // a whole tile goes through shared memory in rows of 128 swizzled bytes, one that starts
          // before the sequence (no store may) straight to global memory
          __nv_bfloat16* row = o + (tile.t0 + i) * p.os[1];
          const uint32_t staged = smem_addr(stage(n)) + S::kV + i * 128 + ((i & 7) << 4);
#pragma unroll 1
          for (int c = 0; c < DV; c += 32) {
            float v[32];
            tmem_ld_32x32(lanes + S::kOut + c, v);
            const uint32_t at = (staged + (c / 64) * C * 128) ^ ((c % 64) * 2);
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              const uint4 x = make_uint4(pack_bf16x2(v[j], v[j + 1]), pack_bf16x2(v[j + 2], v[j + 3]),
                                         pack_bf16x2(v[j + 4], v[j + 5]), pack_bf16x2(v[j + 6], v[j + 7]));
              if (tile.pad == 0)
                st_shared_v4(at ^ (j * 2), x.x, x.y, x.z, x.w);
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
    }
  } else if (warp < 16) {
    regs_up<kStates ? 168 : 128>();
    // --------------------------------------------------- the state, row r of S^T per thread
    constexpr int kCols = DK / 2;
    const int quarter = warp & 3, r = quarter * 32 + lane, part = (warp - 8) >> 2;
    const bool active = quarter * 32 < DV;  // a warp with rows of S^T
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    float s[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) s[c] = 0.f;
    if constexpr (!kStates) {
      // S_0; where there is none the reads go to a valid address and their values are dropped
      const bool given = p.s_in && r < p.dv;
      const float* in = !given ? a.log_decay
                               : p.s_in + bh * static_cast<long long>(p.dk) * p.dv + (p.s_in_transposed ? r * p.dk : r);
      const int step = !given ? 0 : p.s_in_transposed ? 1 : p.dv;
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        const int d = part * kCols + c;
        const float x = in[min(d, p.dk - 1) * step];
        s[c] = given && d < p.dk ? x : 0.f;
        if (c % 16 == 15) keep_order();
      }
      // what the segments before this one add
      if (seg > 0) grid_dependency_wait();
      const float* ps = args.partial + (static_cast<long long>(pass) * a.B * a.H + bh) *
                                           (args.segments - 1) * (DK * DV);
      for (int e = 0; e < seg; ++e, ps += DK * DV) {
        const int at = e * args.chunks_per_segment;
        int toks = args.chunks_per_segment * C;
        if (!p.reverse && at == 0) toks -= tc_tile(0, nch, len, 0).pad;
        const float carry = decay_pow(g, toks);
        if (active) {
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            s[c] = carry * s[c] + ps[(part * kCols + c) * DV + r];
            if (c % 16 == 15) keep_order();
          }
        }
      }
    }
    // this lane's row of the four 8 x 8 blocks of a unit: blocks 0, 1 the first eight tokens,
    // 0, 2 the first eight rows of V^T
    const int v_row = (lane & 7) + (lane & 16) / 2, v_piece = (lane >> 3) & 1;
    const uint32_t v_off = S::kV + (quarter / 2) * C * 128 + (part * kGroup / 2 + v_row) * 128 +
                           ((((quarter & 1) * 4 + v_piece) ^ (v_row & 7)) << 4);
    // S^T in bf16: K-major rows of 128 bytes, 16-byte pieces swizzled by the row (an exclusive or
    // with the piece, as the row starts on 128 bytes)
    const uint32_t s_row = smem_addr(s_tile) + (part * kCols / 64) * DV * 128 + r * 128 +
                           ((((part * kCols % 64) / 8) ^ (r & 7)) << 4);
    auto publish = [&]() {
      if (active) {
#pragma unroll
        for (int c = 0; c < kCols; c += 8)
          st_shared_v4(s_row ^ (c * 2), pack_bf16x2(s[c], s[c + 1]), pack_bf16x2(s[c + 2], s[c + 3]),
                       pack_bf16x2(s[c + 4], s[c + 5]), pack_bf16x2(s[c + 6], s[c + 7]));
      }
      fence_async_shared();
    };
    auto arrive = [&](uint64_t* to) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(to);
    };
    if constexpr (!kStates) {
      publish();
      arrive(s_ready);
    }
    // The parts of V^T w for group `grp` of the tile of step n: this warp's half of its tokens.
    auto split = [&](int n, int grp) {
      if (grp == 0) {
        const TcTile tile = tc_tile(first + n, nch, len, p.reverse);
        if (!__all_sync(0xffffffffu, mbar_wait(&v_full[n % kTcStages], (n / kTcStages) & 1, status,
                                               kErrTimeoutEpilogue)))
          return false;
        if (p.reverse && tile.pad > 0) {  // (the last tile) its weights count from its first real row
          auto meet = [&](uint64_t* bar) {  // the eight state warps
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
            return __all_sync(0xffffffffu, mbar_wait(bar, 0, status, kErrTimeoutEpilogue)) != 0;
          };
          if (!meet(w_free)) return false;
          if (threadIdx.x - 256 < C / 2) weight_parts(wp, threadIdx.x - 256, g, p, tile.pad);
          if (!meet(w_ready)) return false;
        }
      }
      const int buf = grp & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(&up_free[buf], use_parity(n, grp) ^ 1, status, kErrTimeoutEpilogue)))
        return false;
      tc_fence_after();
      if (active) {
        const uint32_t v = smem_addr(stage(n)) + v_off + grp * kGroup * 128;
        const uint32_t* w = wp + (grp * kGroup + part * kGroup / 2) / 2 + (lane & 3);
#pragma unroll
        for (int tok = 0; tok < kGroup / 2; tok += 16) {
          uint32_t ww[3][2];
#pragma unroll
          for (int e = 0; e < 3; ++e) {
            ww[e][0] = w[e * 64 + tok / 2];
            ww[e][1] = w[e * 64 + tok / 2 + 4];
          }
          // 16 tokens x 16 rows of V^T at a time: ldmatrix transposes four 8 x 8 blocks into the
          // layout of the 16-lane store, a register holding two consecutive tokens of one row
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t x[4], p1[4], r1[4], p2[4];
            ldmatrix_x4_trans((v ^ (u * 32)) + tok * 128, x);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int k = e / 2;
              p1[e] = bf16x2_mul(x[e], ww[0][k]);
              r1[e] = bf16x2_fms(x[e], ww[0][k], p1[e]);
              p2[e] = bf16x2_mul(x[e], ww[1][k]);
              x[e] = bf16x2_fma(x[e], ww[2][k], bf16x2_fms(x[e], ww[1][k], p2[e]));
            }
            const uint32_t at =
                lanes + (static_cast<uint32_t>(u * 16) << 16) + parts(buf) + (part * kGroup / 2 + tok) / 2;
            tmem_st_16x128_x2(at, p1);
            tmem_st_16x128_x2(at + kGroup / 2, r1);
            tmem_st_16x128_x2(at + kGroup, p2);
            tmem_st_16x128_x2(at + 3 * kGroup / 2, x);
          }
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&up_ready[buf]);
      return true;
    };
    bool ok = true;
    for (int n = 0; ok && n < n_steps; ++n) {
      const bool more = n + 1 < n_steps;
      if constexpr (kStates)  // the next tile is prepared while this one's products run
        ok = (n > 0 || (split(0, 0) && split(0, 1))) && (!more || (split(n + 1, 0) && split(n + 1, 1)));
      else
        ok = split(n, 0) && split(n, 1) && split(n, 2) && split(n, 3);
      ok = ok && wait_products(d_done(n), d_parity(n));
      if (!ok) break;
      if (active) {
        const float carry = pw[C - tc_tile(first + n, nch, len, p.reverse).pad];
#pragma unroll
        for (int c = 0; c < kCols; c += 32) {
          float d[32];
          tmem_ld_32x32(lanes + d_col(n) + part * kCols + c, d);
#pragma unroll
          for (int j = 0; j < 32; j += 2) fma2(s[c + j], s[c + j + 1], carry, d[j], d[j + 1]);
        }
      }
      if constexpr (kStates) {
        arrive(&d_free[n & 1]);  // D may be written again
      } else if (more) {
        publish();
        arrive(s_ready);  // ... and S^T read
      }
    }
    if (ok) {
      if constexpr (kStates) {
        float* out = args.partial + ((static_cast<long long>(pass) * a.B * a.H + bh) * (args.segments - 1) +
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
          if (c % 16 == 15) keep_order();
        }
      }
    }
  } else {
    regs_down<64>();
    if (warp == 16 && lane == 0) {
      // ------------------------------------------------------------ TMA producer
      const LaMaps& m = args.maps[pass];
      int issued[3] = {0, 0, 0};  // tiles of Q, K, V
      uint64_t* full[3] = {q_full, k_full, v_full};
      for (int n = 0; n < n_steps; ++n) {
        const int st = n % kTcStages;
        const uint32_t ph = ((n / kTcStages) & 1) ^ 1;
        const int t0 = tc_tile(first + n, nch, len, p.reverse).t0;
        uint8_t* base = stage(n);
        // each tile as soon as its place is free: Q's is after the first two products
        if constexpr (!kStates) {
          if (!mbar_wait(&q_empty[st], ph, status, kErrTimeoutProducer)) break;
          mbar_arrive_expect_tx(&q_full[st], S::kQBytes);
#pragma unroll
          for (int x = 0; x < DK; x += 64)
            tma_load_4d(base + x * C * 2, &m.q, &q_full[st], x, t0, h * m.q_ext[0], b * m.q_ext[1]);
          issued[0] = n + 1;
        }
        if (!mbar_wait(&k_empty[st], ph, status, kErrTimeoutProducer)) break;
        mbar_arrive_expect_tx(&k_full[st], S::kQBytes);
#pragma unroll
        for (int x = 0; x < DK; x += 64)
          tma_load_4d(base + S::kK + x * C * 2, &m.k, &k_full[st], x, t0, h * m.k_ext[0], b * m.k_ext[1]);
        issued[1] = n + 1;
        if (!mbar_wait(&v_empty[st], ph, status, kErrTimeoutProducer)) break;
        mbar_arrive_expect_tx(&v_full[st], S::kVBytes);
#pragma unroll
        for (int x = 0; x < DV; x += 64)
          tma_load_4d(base + S::kV + x * C * 2, &m.v, &v_full[st], x, t0, h * m.v_ext[0], b * m.v_ext[1]);
        issued[2] = n + 1;
      }
#pragma unroll
      for (int i = 0; i < 3; ++i)  // every copy lands before the CTA leaves
        for (int n = max(issued[i] - kTcStages, 0); n < issued[i]; ++n)
          mbar_wait(&full[i][n % kTcStages], (n / kTcStages) & 1, status, kErrTimeoutDrain);
    }
    if (!kStates && warp == 18 && lane == 0) {
      // ------------------------------------------------------------ TMA store of O
      const LaMaps& m = args.maps[pass];
      for (int n = 0; n < n_steps; ++n) {
        const TcTile tile = tc_tile(first + n, nch, len, p.reverse);
        if (!mbar_wait(o_staged, n & 1, status, kErrTimeoutEpilogue)) break;
        if (tile.pad == 0) {
#pragma unroll
          for (int x = 0; x < DV; x += 64)
            tma_store_4d(&m.o, stage(n) + S::kV + x * C * 2, x, tile.t0, h * m.o_ext[0], b * m.o_ext[1]);
          bulk_commit_wait_read();
        }
        mbar_arrive(&v_empty[n % kTcStages]);
      }
    }
    if (warp == 17) {
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
        const uint64_t q_desc = umma_desc_sw128(q_addr), k_desc = umma_desc_sw128(q_addr + S::kK);
        const uint64_t k_rows = umma_desc_sw128_mn(q_addr + S::kK, C * 128);
        const uint64_t v_rows = umma_desc_sw128_mn(q_addr + S::kV, C * 128);
        auto update = [&](int grp) {  // D (+)= (V w)^T K over a group of tokens, the small parts first
          const uint32_t a = tmem + parts(grp & 1);
#pragma unroll
          for (int part = 3; part >= 0; --part)
#pragma unroll
            for (int kk = 0; kk < kGroup / 16; ++kk)
              umma_bf16_ts(tmem + d_col(n), a + part * kGroup / 2 + kk * 8,
                           k_rows + (grp * (kGroup / 16) + kk) * (2048 >> 4), idesc_up,
                           grp == 0 && part == 3 && kk == 0 ? 0u : 1u);
        };
        auto intra = [&]() {  // O += (P . L) V
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < C / 16; ++kk)
              umma_bf16_ts(tmem + S::kOut, tmem + S::kScore + kk * 8, v_rows + kk * (2048 >> 4), idesc_pv, 1u);
            umma_commit(o_full);
          }
          __syncwarp();
        };
        if ((!kStates && !wait(&q_full[st], sph)) || !wait(&k_full[st], sph)) break;
        if constexpr (!kStates) {
          // The score columns still hold the last chunk's decayed scores, the operands of O's products
          // that were issued just now: these scores may be issued behind them because one thread's
          // MMAs run in the order of their issue. The wait holds the issue back until the last
          // update has ended; it guards nothing.
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
            umma_commit(&q_empty[st]);
          }
          __syncwarp();
        }
        if (kStates && !wait(&d_free[n & 1], ((n >> 1) & 1) ^ 1)) break;
        bool ok = true;
#pragma unroll 1
        for (int grp = 0; ok && grp < kGroups; ++grp) {
          ok = wait(&up_ready[grp & 1], use_parity(n, grp));
          if (!ok) break;
          if (leader) {
            update(grp);
            umma_commit(&up_free[grp & 1]);
            if (grp == kGroups - 1) {
              umma_commit(d_done(n));
              umma_commit(&k_empty[st]);
              if constexpr (kStates) umma_commit(&v_empty[st]);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        if constexpr (!kStates) {  // last: O then takes the place of the V tile
          if (!wait(p_ready, ph)) break;
          intra();
        }
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
  if constexpr (!kStates) la_end_after_states();
}

}  // namespace pc

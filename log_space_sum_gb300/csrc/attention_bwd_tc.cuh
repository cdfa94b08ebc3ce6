// Gradient of causal softmax attention on the tensor cores: bf16 elements, head sizes padded to 64 or 128, packed
// sequences. Three launches: delta and lse in the order of the rows, dk and dv by tiles of 128 keys, dq by tiles
// of 128 rows (a token and a head of the group each).
//
//   dk, dv   S^T = K Q^T, dP^T = V dO^T   A = K, V resident, B = Q, dO streamed (all K-major shared memory)
//            P^T = exp2(S^T scale - lse), dS^T = P^T (dP^T - delta), rounded to bf16 over S^T and dP^T
//            dV += P^T dO, dK += dS^T Q   A in tensor memory, B = the same dO, Q tiles read MN-major
//   dq       S = Q K^T, dP = dO V^T       A = Q, dO resident, B = K, V streamed
//            dQ += dS K                   A = dS in tensor memory (over S), B = the same K tile read MN-major
//
// Keys lie in the lanes of dk, dv's accumulators and rows in those of dq's, so that no tile is transposed and
// nothing is added by atomics: S and dP are formed twice (seven products instead of five) for sums of a fixed order.
// Products of the next tile are issued between those of this one, while the warps form P or dS:
//   dk, dv:  dV(i) S(i+1) | dK(i) dP(i+1)          dq:  dP(j+1) dQ(j) S(j+2)
// Whole tiles of dq are staged in the place of Q and leave by TMA (456 -> 433 us; dk and dv, of fewer and longer CTAs, do not:
// 477 us against 504, with registers spilt).
// Measured: 12 sequences to 4096 (27,873 tokens), 16 / 2 heads of 128, 975 us; under the profiler dk and dv 488 (tensor pipe 62%
// busy; without the warps' arithmetic 423), dq 440 (50%, 3508 CTAs; 413), delta 53. Not kept: four warpgroups of 32
// columns each (1035 us in all), streamed tiles shared by two CTAs through multicast (1119: the pair's lockstep costs more than the
// L2 reads that it saves).
// Warps 0-3 take the columns 0 .. 63 of a tile's lanes, warps 4-7 the others; each writes its bf16 operand over columns that
// it has read itself, so that an operand's second half starts at column 64.
#pragma once

#include "attention_simt.cuh"
#include "attention_tc.cuh"

namespace pc {

struct AttnBwdTcArgs {
  AttnBwdArgs b;
  CUtensorMap q, d_o, k, v, dq;
  int k_ext, v_ext;
  int per;            // tokens of a tile of rows
  float k2;           // scale log2(e)
  float *lse2, *delta;  // [H / pack][T][pack]: lse log2(e) and delta by rows
};

// Eight lanes of 16 bytes (D <= 64) or sixteen a row, four rows a thread at a time: delta and lse in the order of the tiles'
// rows.
constexpr int kAtRowsAtOnce = 4;

template <int kLanesRow>
__global__ void __launch_bounds__(256) k_attn_rows_tc(const __grid_constant__ AttnBwdTcArgs args) {
  const AttnArgs& a = args.b.a;
  constexpr int kRows = 256 / kLanesRow;
  const unsigned all = static_cast<unsigned>(a.T) * a.H;
  const unsigned row0 = blockIdx.x * (kRows * kAtRowsAtOnce) + threadIdx.x / kLanesRow;
  const int d = threadIdx.x % kLanesRow * 8;
  uint4 x[kAtRowsAtOnce], y[kAtRowsAtOnce];
#pragma unroll
  for (int e = 0; e < kAtRowsAtOnce; ++e) {
    const unsigned row = row0 + e * kRows, t = row / a.H, h = row - t * a.H;
    x[e] = y[e] = make_uint4(0u, 0u, 0u, 0u);
    if (row < all && d < a.D) {
      x[e] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.o) + t * a.os[0] + h * a.os[1] + d);
      y[e] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(args.b.d_o) + t * args.b.gs[0] + h * args.b.gs[1] + d);
    }
  }
#pragma unroll
  for (int e = 0; e < kAtRowsAtOnce; ++e) {
    const uint32_t xs[4] = {x[e].x, x[e].y, x[e].z, x[e].w}, ys[4] = {y[e].x, y[e].y, y[e].z, y[e].w};
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v += __uint_as_float(xs[i] << 16) * __uint_as_float(ys[i] << 16);
      v += __uint_as_float(xs[i] & 0xFFFF0000u) * __uint_as_float(ys[i] & 0xFFFF0000u);
    }
#pragma unroll
    for (int w = kLanesRow / 2; w; w >>= 1) v += __shfl_xor_sync(0xffffffffu, v, w);
    const unsigned row = row0 + e * kRows, t = row / a.H, h = row - t * a.H;
    if (row < all && d == 0) {
      const long long at = (static_cast<long long>(h / a.pack) * a.T + t) * a.pack + h % a.pack;
      args.delta[at] = v;
      args.lse2[at] = args.b.lse[static_cast<long long>(h) * a.T + t] * kLog2e;
    }
  }
}

template <int DP>
struct AtBwdShape {
  static constexpr uint32_t kTile = kAtC * DP * 2;
  static constexpr int kSlots = DP == 128 ? 5 : 8;
  static constexpr uint32_t kRing = 2 * kTile;
  static constexpr uint32_t kAux = kRing + kSlots * kTile;  // dk, dv: two stages of lse2 and delta, 128 each
  static constexpr uint32_t kBars = kAux + 2 * 2 * kAtC * 4;
  static constexpr uint32_t kBytes = kBars + 256;  // the tiles fill what there is: the base itself is aligned for them
  static_assert(kBytes <= 232448, "shared memory per CTA");
};

// Zeros rows [from, to) of a tile (by one warp), for products that read it whole.
template <int DP>
__device__ __forceinline__ void at_zero_rows(uint32_t tile, int from, int to) {
  for (int i = from * 8 + (threadIdx.x & 31); i < to * 8; i += 32)
#pragma unroll
    for (int d = 0; d < DP; d += 64) st_shared_v4(tile + d * kAtC * 2 + i * 16, 0u, 0u, 0u, 0u);
  fence_async_shared();
  __syncwarp();
}

// 64 float32 columns of this thread's lane, in two halves.
__device__ __forceinline__ void at_load64(uint32_t col, uint32_t (&v)[2][32]) {
  tmem_ld_32x32_async(col, v[0]);
  tmem_ld_32x32_async(col + 32, v[1]);
  tmem_wait_ld(v[0]);
  tmem_wait_ld(v[1]);
}

// 32 float32 columns of an accumulator, times `by`, as bf16 to a row of D elements.
__device__ __forceinline__ void at_store_row(uint32_t col, int c, int D, float by, bool there, __nv_bfloat16* row) {
  float u[32];
  tmem_ld_32x32(col + c, u);
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    if (there && c + i < D)
      *reinterpret_cast<uint4*>(row + c + i) =
          make_uint4(pack_bf16x2(u[i] * by, u[i + 1] * by), pack_bf16x2(u[i + 2] * by, u[i + 3] * by),
                     pack_bf16x2(u[i + 4] * by, u[i + 5] * by), pack_bf16x2(u[i + 6] * by, u[i + 7] * by));
}

// Products of two K-major tiles (A rows in the lanes), and of a packed operand in tensor memory, whose second half starts
// at column 64, with a tile read MN-major. The descriptors are formed by the whole warp, before one lane issues: in its branch they
// would not be known to be uniform (996 -> 989 us for 12 sequences to 4096).
template <int DP>
__device__ __forceinline__ void at_mma_ss(uint32_t d, uint64_t x, uint64_t y) {
  constexpr uint32_t idesc = umma_idesc(1, 128, kAtC);
#pragma unroll
  for (int kk = 0; kk < DP / 16; ++kk) {
    const uint32_t off = ((kk / 4) * kAtC * 128 + (kk % 4) * 32) >> 4;
    umma_bf16(d, x + off, y + off, idesc, kk ? 1u : 0u);
  }
}
template <int DP>
__device__ __forceinline__ void at_mma_ts(uint32_t d, uint32_t a, uint64_t y, bool add) {
  constexpr uint32_t idesc = umma_idesc(1, 128, DP) | kIdescBMN;
#pragma unroll
  for (int kk = 0; kk < kAtC / 16; ++kk)
    umma_bf16_ts(d, a + (kk / 4) * 64 + (kk % 4) * 8, y + kk * (2048 >> 4), idesc, add || kk > 0 ? 1u : 0u);
}

template <int DP>
__global__ void __launch_bounds__(kAtThreads, 1) k_attn_dkdv_tc(const __grid_constant__ AttnBwdTcArgs args) {
  using S = AtBwdShape<DP>;
  constexpr int C = kAtC;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* aux = reinterpret_cast<float*>(smem + S::kAux);  // [stage][lse2, delta][C]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBars);
  uint64_t *full = bars, *empty = bars + 8, *kv_full = bars + 16, *s_full = bars + 17, *p_ready = bars + 18,
           *dp_full = bars + 19, *ds_ready = bars + 20, *aux_full = bars + 21, *aux_empty = bars + 23, *acc_full = bars + 25,
           *mma_done = bars + 26;
  auto* limit = reinterpret_cast<unsigned long long*>(bars + 27);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 28);

  const AttnArgs& a = args.b.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hk = blockIdx.x % a.Hk, per = args.per, rows = per * a.pack;
  AttnSeq s{0, 0, 0};
  const AttnTile tile = attn_tile_by_cost<true, false>(a, blockIdx.x / a.Hk, C, s);
  if (tile.b < 0) return;
  const int j0 = tile.at * C;
  // rows of the tokens from the tile's first key on, for each `pack` heads of the group in turn
  const int i_first = j0 / per, i_each = (s.n + per - 1) / per - i_first, folds = a.group / a.pack, steps = i_each * folds;
  unsigned* status = a.status;
  auto token0 = [&](int it) { return (i_first + it % i_each) * per; };
  auto fold = [&](int it) { return hk * folds + it / i_each; };

  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < S::kSlots; ++i) {
        mbar_init(&full[i], 1);
        mbar_init(&empty[i], 1);
      }
      mbar_init(kv_full, 1);
      mbar_init(s_full, 1);
      mbar_init(dp_full, 1);
      mbar_init(p_ready, 8);
      mbar_init(ds_ready, 8);
      for (int i = 0; i < 2; ++i) {
        mbar_init(&aux_full[i], 1);
        mbar_init(&aux_empty[i], 8);
      }
      mbar_init(acc_full, 1);
      mbar_init(mma_done, 1);
      *limit = first_wait_limit(status);
      fence_barrier_init();
    }
    __syncwarp();
    tmem_alloc(tmem_slot, 512);
  }
  if (rows < C && warp >= 4) {  // rows that no copy writes
    for (int slot = warp - 4; slot < S::kSlots; slot += 8) at_zero_rows<DP>(smem_addr(smem) + S::kRing + slot * S::kTile, rows, C);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t s_at = tmem, dp_at = tmem + C, dv_at = tmem + 2 * C, dk_at = tmem + 2 * C + DP;

  if (warp < 8) {
    at_regs_up<208>();
    const int part = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane, key = j0 + r;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_col = s_at + lanes + part * 64, dp_col = dp_at + lanes + part * 64;
    const float k2 = args.k2;
    bool ok = at_first_wait(s_full, status, kErrTimeoutEpilogue, *limit);
    for (int it = 0; ok && it < steps; ++it) {
      const float* lse2 = aux + (it & 1) * 2 * C + part * 64;
      const float* delta = lse2 + C;
      ok = at_wait(&aux_full[it & 1], (it >> 1) & 1, status, kErrTimeoutEpilogue) &&
           at_wait(s_full, it & 1, status, kErrTimeoutEpilogue, *limit);
      if (!ok) break;
      uint32_t v[2][32];
      at_load64(s_col, v);
      float p[64];
      // the columns from `low` on see the key
      const int t0 = token0(it);
      if (t0 < j0 + quarter * 32 + 31) {
        const int low = (key - t0) * a.pack - part * 64;
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          float x = __uint_as_float(v[c / 32][c % 32]) * k2 - lse2[c];
          p[c] = c >= low ? at_exp2(x) : 0.f;
        }
      } else {
#pragma unroll
        for (int c = 0; c < 64; c += 4) {
          const float4 z = *reinterpret_cast<const float4*>(lse2 + c);
          p[c] = __uint_as_float(v[c / 32][c % 32]);
          p[c + 1] = __uint_as_float(v[c / 32][c % 32 + 1]);
          p[c + 2] = __uint_as_float(v[c / 32][c % 32 + 2]);
          p[c + 3] = __uint_as_float(v[c / 32][c % 32 + 3]);
          fma2(p[c], p[c + 1], k2, -z.x, -z.y);
          fma2(p[c + 2], p[c + 3], k2, -z.z, -z.w);
#pragma unroll
          for (int e = 0; e < 4; ++e) p[c + e] = at_exp2(p[c + e]);
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(p[c * 32 + 2 * i], p[c * 32 + 2 * i + 1]);
        tmem_st_32x16(s_col + c * 16, w);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_ready);
      ok = at_wait(dp_full, it & 1, status, kErrTimeoutEpilogue, *limit);
      if (!ok) break;
      at_load64(dp_col, v);
#pragma unroll
      for (int c = 0; c < 64; c += 4) {
        const float4 z = *reinterpret_cast<const float4*>(delta + c);
        float e0 = __uint_as_float(v[c / 32][c % 32]), e1 = __uint_as_float(v[c / 32][c % 32 + 1]);
        float e2 = __uint_as_float(v[c / 32][c % 32 + 2]), e3 = __uint_as_float(v[c / 32][c % 32 + 3]);
        at_add2(e0, e1, -z.x, -z.y);
        at_add2(e2, e3, -z.z, -z.w);
        mul2(p[c], p[c + 1], e0, e1);
        mul2(p[c + 2], p[c + 3], e2, e3);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(p[c * 32 + 2 * i], p[c * 32 + 2 * i + 1]);
        tmem_st_32x16(dp_col + c * 16, w);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(ds_ready);
        mbar_arrive(&aux_empty[it & 1]);
      }
    }
    if (ok && at_wait(acc_full, 0, status, kErrTimeoutEpilogue, *limit)) {
      const bool there = key < s.n;
      const long long* st = part ? args.b.dks : args.b.dvs;
      __nv_bfloat16* row =
          static_cast<__nv_bfloat16*>(part ? args.b.dk : args.b.dv) + (s.start + static_cast<long long>(key)) * st[0] + hk * st[1];
      const float by = part ? a.scale : 1.f;
#pragma unroll 1
      for (int c = 0; c < DP; c += 32) at_store_row((part ? dk_at : dv_at) + lanes, c, a.D, by, there, row);
    }
  } else {
    at_regs_down<64>();
    if (warp == 8 && lane == 0) {
      // ------------------------------------------------------------ TMA producer: K, V, then Q, dO, Q, dO, ...
      mbar_arrive_expect_tx(kv_full, 2 * S::kTile);
      for (int d = 0; d < DP; d += 64) {
        tma_load_4d(smem + d * C * 2, &args.k, kv_full, d, s.start + j0, hk * args.k_ext, 0);
        tma_load_4d(smem + S::kTile + d * C * 2, &args.v, kv_full, d, s.start + j0, hk * args.v_ext, 0);
      }
      int issued = 0;
      for (int n = 0; n < 2 * steps; ++n) {
        const int slot = n % S::kSlots, it = n / 2;
        if (!mbar_wait(&empty[slot], ((n / S::kSlots) & 1) ^ 1, status, kErrTimeoutProducer)) break;
        mbar_arrive_expect_tx(&full[slot], rows * DP * 2);
        for (int d = 0; d < DP; d += 64)
          tma_load_4d(smem + S::kRing + slot * S::kTile + d * C * 2, n % 2 ? &args.d_o : &args.q, &full[slot], d, fold(it) * a.pack,
                      s.start + token0(it), 0);
        issued = n + 1;
      }
      mbar_wait(kv_full, 0, status, kErrTimeoutDrain);
      for (int n = max(issued - S::kSlots, 0); n < issued; ++n)  // every copy lands before the CTA leaves
        mbar_wait(&full[n % S::kSlots], (n / S::kSlots) & 1, status, kErrTimeoutDrain);
    } else if (warp == 10) {
      // ------------------------------------------------------------ lse and delta of the rows
      for (int it = 0; it < steps; ++it) {
        if (!__all_sync(0xffffffffu, mbar_wait(&aux_empty[it & 1], ((it >> 1) & 1) ^ 1, status, kErrTimeoutProducer))) break;
        const int t0 = token0(it), have = min(per, s.n - t0) * a.pack;
        const long long at = (static_cast<long long>(fold(it)) * a.T + s.start + t0) * a.pack;
        float z[4], e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = lane + 32 * i;
          z[i] = c < have ? args.lse2[at + c] : INFINITY;  // p of the rows that are not there: 0
          e[i] = c < have ? args.delta[at + c] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          aux[(it & 1) * 2 * C + lane + 32 * i] = z[i];
          aux[(it & 1) * 2 * C + C + lane + 32 * i] = e[i];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&aux_full[it & 1]);
      }
    } else if (warp == 9) {
      // ----------------- MMA issuer: the whole warp in step (uniform addresses), one lane issues
      const bool leader = elect_one();
      const uint32_t base = smem_addr(smem);
      auto slot_addr = [&](int n) { return base + S::kRing + (n % S::kSlots) * S::kTile; };
      // the n-th streamed tile is there; rows behind the sequence are zeros
      auto slot_full = [&](int n) {
        if (!at_wait(&full[n % S::kSlots], (n / S::kSlots) & 1, status, kErrTimeoutMma)) return false;
        const int left = s.n - token0(n / 2);
        if (left < per) at_zero_rows<DP>(slot_addr(n), left * a.pack, rows);
        return true;
      };
      const uint64_t k_desc = umma_desc_sw128(base), v_desc = umma_desc_sw128(base + S::kTile);
      auto scores = [&](int n) {
        const uint64_t q = umma_desc_sw128(slot_addr(n));
        if (leader) {
          at_mma_ss<DP>(s_at, k_desc, q);
          umma_commit(s_full);
        }
        __syncwarp();
      };
      auto products = [&](int n) {
        const uint64_t g = umma_desc_sw128(slot_addr(n));
        if (leader) {
          at_mma_ss<DP>(dp_at, v_desc, g);
          umma_commit(dp_full);
        }
        __syncwarp();
      };
      auto gradient = [&](uint32_t to, uint32_t from, int n, bool add) {
        const uint64_t rows_of = umma_desc_sw128_mn(slot_addr(n), C * 128);
        if (leader) {
          at_mma_ts<DP>(to, from, rows_of, add);
          umma_commit(&empty[n % S::kSlots]);
        }
        __syncwarp();
      };
      bool ok = at_wait(kv_full, 0, status, kErrTimeoutMma) && slot_full(0);
      if (ok) {
        scores(0);
        ok = slot_full(1);
      }
      if (ok) products(1);
      for (int it = 0; ok && it < steps; ++it) {
        const bool more = it + 1 < steps;
        ok = at_wait(p_ready, it & 1, status, kErrTimeoutMma) && (!more || slot_full(2 * it + 2));
        if (!ok) break;
        gradient(dv_at, s_at, 2 * it + 1, it > 0);
        if (more) scores(2 * it + 2);
        ok = at_wait(ds_ready, it & 1, status, kErrTimeoutMma) && (!more || slot_full(2 * it + 3));
        if (!ok) break;
        gradient(dk_at, dp_at, 2 * it, it > 0);
        if (more) products(2 * it + 3);
      }
      if (leader) umma_commit(acc_full);
      __syncwarp();
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

template <int DP>
__global__ void __launch_bounds__(kAtThreads, 1) k_attn_dq_tc(const __grid_constant__ AttnBwdTcArgs args) {
  using S = AtBwdShape<DP>;
  constexpr int C = kAtC;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBars);
  uint64_t *full = bars, *empty = bars + 8, *q_full = bars + 16, *s_full = bars + 17, *dp_full = bars + 19,
           *ds_ready = bars + 20, *acc_full = bars + 21, *mma_done = bars + 22, *staged = bars + 23;
  auto* limit = reinterpret_cast<unsigned long long*>(bars + 24);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 25);

  const AttnArgs& a = args.b.a;
  const int heads = a.H / a.pack, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hp = blockIdx.x % heads, hk = hp * a.pack / a.group, per = args.per;
  // one warp sets up the barriers, another takes the tensor memory, while all find their work
  if (warp == 8 && lane == 0) {
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(dp_full, 1);
    mbar_init(ds_ready, 8);
    mbar_init(acc_full, 1);
    mbar_init(staged, 8);
    mbar_init(mma_done, 1);
    *limit = first_wait_limit(a.status);
    fence_barrier_init();
  }
  AttnSeq s{0, 0, 0};
  const AttnTile tile = attn_tile_by_cost<false, false>(a, blockIdx.x / heads, per, s);
  if (tile.b < 0) return;
  const int t0 = tile.at * per, keys = min(t0 + per, s.n), steps = (keys + C - 1) / C;
  unsigned* status = a.status;

  if (warp == 0) tmem_alloc(tmem_slot, 512);
  if (warp == 8 && lane == 0) {  // the resident operands' copies start before the CTA meets
    mbar_arrive_expect_tx(q_full, 2 * per * a.pack * DP * 2);
    for (int d = 0; d < DP; d += 64) {
      tma_load_4d(smem + d * C * 2, &args.q, q_full, d, hp * a.pack, s.start + t0, 0);
      tma_load_4d(smem + S::kTile + d * C * 2, &args.d_o, q_full, d, hp * a.pack, s.start + t0, 0);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t dp_at = tmem + 2 * C, dq_at = tmem + 3 * C;  // S: two in turn

  const bool whole = t0 + per <= s.n;

  if (warp < 8) {
    at_regs_up<208>();
    const int part = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane, token = t0 + r / a.pack;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const bool there = r < per * a.pack && token < s.n;
    const int see = there ? token : -1, see_all = __reduce_min_sync(0xffffffffu, see);
    const long long at = (static_cast<long long>(hp) * a.T + s.start + t0) * a.pack + r;
    const float lse2 = there ? -args.lse2[at] : 0.f, delta = there ? -args.delta[at] : 0.f, k2 = args.k2;
    bool ok = at_first_wait(&s_full[0], status, kErrTimeoutEpilogue, *limit);
    for (int j = 0; ok && j < steps; ++j) {
      ok = at_wait(&s_full[j & 1], (j >> 1) & 1, status, kErrTimeoutEpilogue, *limit);
      if (!ok) break;
      const uint32_t s_col = tmem + lanes + (j & 1) * C + part * 64;
      uint32_t v[2][32];
      at_load64(s_col, v);
      float p[64];
#pragma unroll
      for (int c = 0; c < 64; c += 2) {
        p[c] = __uint_as_float(v[c / 32][c % 32]);
        p[c + 1] = __uint_as_float(v[c / 32][c % 32 + 1]);
        fma2(p[c], p[c + 1], k2, lse2, lse2);
        p[c] = at_exp2(p[c]);
        p[c + 1] = at_exp2(p[c + 1]);
      }
      ok = at_wait(dp_full, j & 1, status, kErrTimeoutEpilogue, *limit);
      if (!ok) break;
      at_load64(dp_at + lanes + part * 64, v);
      const bool edge = see_all < j * C + part * 64 + 63;
      const int left = see - j * C - part * 64;  // the columns 0 .. left are seen
#pragma unroll
      for (int c = 0; c < 64; c += 2) {
        float e0 = __uint_as_float(v[c / 32][c % 32]), e1 = __uint_as_float(v[c / 32][c % 32 + 1]);
        at_add2(e0, e1, delta, delta);
        mul2(p[c], p[c + 1], e0, e1);
      }
      if (edge) {
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (c > left) p[c] = 0.f;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(p[c * 32 + 2 * i], p[c * 32 + 2 * i + 1]);
        tmem_st_32x16(s_col + c * 16, w);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_ready);
    }
    if (ok && at_wait(acc_full, 0, status, kErrTimeoutEpilogue, *limit)) {
      const int h = hp * a.pack + r % a.pack;
      __nv_bfloat16* row = static_cast<__nv_bfloat16*>(args.b.dq) + (s.start + static_cast<long long>(token)) * args.b.dqs[0] +
                           h * args.b.dqs[1];
#pragma unroll 1
      for (int c = part * (DP / 2); c < (part + 1) * (DP / 2); c += 32) {
        if (whole) {
          float u[32];
          tmem_ld_32x32(dq_at + lanes + c, u);
#pragma unroll
          for (int i = 0; i < 32; ++i) u[i] *= a.scale;
          at_stage(smem_addr(smem), r, c, u);
        } else {
          at_store_row(dq_at + lanes, c, a.D, a.scale, there, row);
        }
      }
      if (whole) {
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(staged);
      }
    }
  } else {
    at_regs_down<64>();
    if (warp == 8 && lane == 0) {
      // ------------------------------------------------------------ TMA producer: Q, dO, then K, V, K, V, ...
      int issued = 0;
      for (int n = 0; n < 2 * steps; ++n) {
        const int slot = n % S::kSlots, j = n / 2;
        if (!mbar_wait(&empty[slot], ((n / S::kSlots) & 1) ^ 1, status, kErrTimeoutProducer)) break;
        mbar_arrive_expect_tx(&full[slot], S::kTile);
        for (int d = 0; d < DP; d += 64)
          tma_load_4d(smem + S::kRing + slot * S::kTile + d * C * 2, n % 2 ? &args.v : &args.k, &full[slot], d, s.start + j * C,
                      hk * (n % 2 ? args.v_ext : args.k_ext), 0);
        issued = n + 1;
      }
      mbar_wait(q_full, 0, status, kErrTimeoutDrain);
      for (int n = max(issued - S::kSlots, 0); n < issued; ++n)  // every copy lands before the CTA leaves
        mbar_wait(&full[n % S::kSlots], (n / S::kSlots) & 1, status, kErrTimeoutDrain);
    } else if (warp == 9) {
      // ----------------- MMA issuer: the whole warp in step (uniform addresses), one lane issues
      const bool leader = elect_one();
      const uint32_t base = smem_addr(smem);
      auto slot_addr = [&](int n) { return base + S::kRing + (n % S::kSlots) * S::kTile; };
      // the n-th streamed tile is there; K's rows behind the keys are zeros (V's give columns that no row sees)
      auto slot_full = [&](int n) {
        if (!at_wait(&full[n % S::kSlots], (n / S::kSlots) & 1, status, kErrTimeoutMma)) return false;
        const int left = keys - n / 2 * C;
        if (n % 2 == 0 && left < C) at_zero_rows<DP>(slot_addr(n), left, C);
        return true;
      };
      const uint64_t q_desc = umma_desc_sw128(base), g_desc = umma_desc_sw128(base + S::kTile);
      auto scores = [&](int j) {
        const uint64_t k = umma_desc_sw128(slot_addr(2 * j));
        if (leader) {
          at_mma_ss<DP>(tmem + (j & 1) * C, q_desc, k);
          umma_commit(&s_full[j & 1]);
        }
        __syncwarp();
      };
      auto products = [&](int j) {  // dP
        const uint64_t v = umma_desc_sw128(slot_addr(2 * j + 1));
        if (leader) {
          at_mma_ss<DP>(dp_at, g_desc, v);
          umma_commit(dp_full);
          umma_commit(&empty[(2 * j + 1) % S::kSlots]);
        }
        __syncwarp();
      };
      bool ok = at_wait(q_full, 0, status, kErrTimeoutMma) && slot_full(0);
      if (ok) {
        scores(0);
        ok = slot_full(1);
      }
      if (ok) {
        products(0);
        ok = steps < 2 || slot_full(2);
      }
      if (ok && steps > 1) scores(1);
      for (int j = 0; ok && j < steps; ++j) {
        ok = (j + 1 >= steps || slot_full(2 * j + 3)) && at_wait(ds_ready, j & 1, status, kErrTimeoutMma);
        if (!ok) break;
        if (j + 1 < steps) products(j + 1);
        const uint64_t k_rows = umma_desc_sw128_mn(slot_addr(2 * j), C * 128);
        if (leader) {
          at_mma_ts<DP>(dq_at, tmem + (j & 1) * C, k_rows, j > 0);
          umma_commit(&empty[(2 * j) % S::kSlots]);
        }
        __syncwarp();
        if (j + 2 < steps) {
          ok = slot_full(2 * j + 4);
          if (ok) scores(j + 2);
        }
      }
      if (leader) umma_commit(acc_full);
      __syncwarp();
      if (leader) umma_commit(mma_done);
      __syncwarp();
      mbar_wait(mma_done, 0, status, kErrTimeoutDrain);
    } else if (warp == 11 && lane == 0 && whole) {
      if (mbar_wait(staged, 0, status, kErrTimeoutEpilogue))
        for (int d = 0; d < DP; d += 64) tma_store_4d(&args.dq, smem + d * C * 2, d, hp * a.pack, s.start + t0, 0);
      bulk_commit_wait_read();
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

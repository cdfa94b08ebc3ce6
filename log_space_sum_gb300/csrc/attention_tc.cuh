// Softmax attention forward on the tensor cores: bf16 elements, head sizes padded to 64 or 128, packed
// prompts or a paged cache.
//
// A CTA takes two tiles of 128 rows (a token and a head of the group each) at a time and walks the keys that they see
// in tiles of 128:
//
//   scores  S = Q K^T     A = Q, B = K (K-major shared memory, by TMA), S in tensor memory
//   softmax               one row per thread: the running maximum m and sum l, P = exp2(S scale - m) rounded to
//                         bf16 and written over S
//   output  O += P V      A = P in tensor memory, B = V (MN-major)
//
//   warps 0-3    softmax of the first tile's rows, warps 4-7 of the second's
//   warp 8       TMA: Q once, then K and V tiles through one ring
//   warp 9       MMA issuer: while one tile's softmax runs, the other's products do; zeros the rows of the last V
//                tile that lie behind the keys, as what is there may be no number
//   warp 10      hands out the work (AtScheduler): CTAs stay, one on each SM
//
// m is raised, and O in tensor memory multiplied by the ratio, only when a row's maximum has grown by more than 2^8:
// P then holds values up to 256, whose relative rounding is the same, and l is summed in float32 from the
// probabilities before their rounding. S of the next tile of keys is issued behind O of this one: MMAs of one thread
// end in the order of their issue, so the arrival of S says that O may be touched.
//
// Bound by the tensor core: 2 x 128 x 128 x D products a tile of rows and keys, 512 cycles each at D = 128.
#pragma once

#include <climits>

#include "attention.cuh"

namespace pc {

constexpr int kAtC = 128;          // rows and keys of a tile
constexpr int kAtThreads = 384;

struct AttnTcArgs {
  AttnArgs a;
  CUtensorMap q, k, v;
  int k_ext, v_ext;         // 1: the map has the heads, 0: they share one
  int box;                  // keys of one TMA box: 128, or a page's where it is smaller
  int per;                  // tokens of a tile of rows
};

template <int DP>
struct AtShape {
  static constexpr uint32_t kTile = kAtC * DP * 2;
  static constexpr int kSlots = DP == 128 ? 5 : 8;  // K and V in turn
  static constexpr uint32_t kRing = 2 * kTile;      // behind the two Q tiles
  static constexpr uint32_t kFixed = kRing + kSlots * kTile;
  static constexpr uint32_t kBytes = kFixed + 1024;  // the base itself is aligned for the tiles
  static_assert(kBytes <= 232448, "shared memory per CTA");
  static constexpr uint32_t kS = 0, kO = 256;  // tensor memory columns: S of both tiles, O of both
};

// One stretch of work of a CTA: tiles [first, end) of the keys that two tiles of rows see.
struct AtSegment {
  int b;                // the sequence; -1: no more work
  int start, n, before; // its first row, its rows, the keys before the first row's own
  int t0, hp;           // first token of the rows, heads
  int keys[2];          // that either tile of rows sees
  int first, end;
  int slot;             // where the part goes that others have to be joined with; -1: the rows' output is whole
};

template <int kRegs>
__device__ __forceinline__ void at_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void at_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
// The lanes of a warp in step at a barrier.
__device__ __forceinline__ bool at_wait(uint64_t* bar, uint32_t parity, unsigned* status, unsigned code,
                                        unsigned long long limit = kWaitLimitNs) {
  const bool got = __all_sync(0xffffffffu, mbar_wait(bar, parity, status, code, limit));
  tc_fence_after();
  return got;
}
__device__ __forceinline__ float at_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void at_add2(float& a0, float& a1, float b0, float b1) {
  add2(a0, a1, __float_as_uint(b0), __float_as_uint(b1));
}

// Tiles of keys of a unit of work: two tiles of rows of one sequence, for one of the heads' groups (one at least: rows
// that see nothing have an output too).
__device__ __forceinline__ int at_cost(const AttnArgs& a, const AttnSeq& s, int at, int per) {
  const int keys = max(attn_keys(a, s, at * 2 * per, per), attn_keys(a, s, (at * 2 + 1) * per, per));
  return max((keys + kAtC - 1) / kAtC, 1);
}

// The work of a CTA, by one warp.
//   packed  whole units, sorted by cost, dealt to the CTAs there and back: neither cuts nor joins
//   paged   all units' tiles in one row, cut into even ranges: a token of one long sequence fills the GPU as many
//           sequences of any lengths do; a unit that a cut goes through is joined afterwards
struct AtScheduler {
  const AttnTcArgs& args;
  int heads, k;                  // packed: the round
  long long left;                // paged: tiles of the range to come
  int b, at, hp, j, cost, tiles; // ... and where it stands
  long long grid, all, pos;
  AttnSeq s;

  __device__ __forceinline__ explicit AtScheduler(const AttnTcArgs& x) : args(x) {
    const AttnArgs& a = x.a;
    heads = a.H / a.pack;
    k = 0;
    left = 0;
    if (!a.page) return;
    if (threadIdx.x % 32 == 0) a.part_head[blockIdx.x].parts = 0;
    all = 0;
    for (int at_b = 0; at_b < a.B; at_b += 32) all += warp_sum(sequence_cost(at_b + threadIdx.x % 32));
    // two tiles a CTA at least
    grid = min(static_cast<long long>(gridDim.x), max(all / 2, 1ll));
    if (all == 0 || blockIdx.x >= grid) return;
    pos = blockIdx.x * all / grid;
    left = (blockIdx.x + 1) * all / grid - pos;
    long long skip = pos;
    for (b = 0;; b += 32) {
      const long long own = sequence_cost(b + threadIdx.x % 32);
      long long sum = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, sum, d);
        if (threadIdx.x % 32 >= d) sum += y;
      }
      const unsigned here = __ballot_sync(0xffffffffu, sum > skip);
      if (here) {
        const int l = __ffs(here) - 1;
        skip -= __shfl_sync(0xffffffffu, sum - own, l);
        b += l;
        break;
      }
      skip -= __shfl_sync(0xffffffffu, sum, 31);
    }
    open(b);
    for (at = 0;; ++at) {
      cost = at_cost(a, s, at, args.per);
      if (skip < static_cast<long long>(cost) * heads) break;
      skip -= static_cast<long long>(cost) * heads;
    }
    hp = static_cast<int>(skip / cost);
    j = static_cast<int>(skip % cost);
  }

  __device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
  }
  __device__ __forceinline__ long long sequence_cost(int seq) {
    if (seq >= args.a.B) return 0;
    const AttnSeq q = attn_seq(args.a, seq);
    long long sum = 0;
    for (int i = 0; i * 2 * args.per < q.n; ++i) sum += at_cost(args.a, q, i, args.per);
    return sum * heads;
  }
  __device__ __forceinline__ void open(int seq) {
    s = attn_seq(args.a, seq);
    tiles = (s.n + 2 * args.per - 1) / (2 * args.per);
  }

  __device__ __forceinline__ AtSegment next() {
    const AttnArgs& a = args.a;
    AtSegment g;
    g.b = -1;
    g.slot = -1;
    if (!a.page) {
      const long long rank = static_cast<long long>(k & 1 ? k + 1 : k) * gridDim.x + (k & 1 ? -1 - static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x));
      ++k;
      if (rank / heads >= INT_MAX) return g;
      const AttnTile tile = attn_tile_by_cost<false>(a, static_cast<int>(rank / heads), 2 * args.per);
      if (tile.b < 0) return g;
      s = attn_seq(a, tile.b);
      g.b = tile.b;
      g.hp = static_cast<int>(rank % heads);
      fill(g, tile.at);
      g.first = 0;
      g.end = (max(g.keys[0], g.keys[1]) + kAtC - 1) / kAtC;
      return g;
    }
    if (left <= 0) return g;
    const int len = static_cast<int>(min(left, static_cast<long long>(cost - j)));
    g.b = b;
    g.hp = hp;
    fill(g, at);
    const int real = (max(g.keys[0], g.keys[1]) + kAtC - 1) / kAtC;
    g.first = min(j, real);
    g.end = min(j + len, real);
    if (len < cost) {
      g.slot = 2 * blockIdx.x + (j == 0 ? 1 : 0);
      if (j == 0 && threadIdx.x % 32 == 0) {
        // the CTAs that hold the rest: tile x is in the range of CTA ((x + 1) grid - 1) / all
        const long long end = pos + cost - 1;
        a.part_head[blockIdx.x] = {static_cast<int>(((end + 1) * grid - 1) / all - blockIdx.x) + 1, s.start + g.t0, s.n - g.t0, hp};
      }
    }
    left -= len;
    pos += len;
    j += len;
    if (j == cost) {
      j = 0;
      if (++hp == heads) {
        hp = 0;
        if (++at == tiles) {
          at = 0;
          do ++b;
          while (b < a.B && attn_seq(a, b).n == 0);
          if (b >= a.B) {
            left = 0;
            return g;
          }
          open(b);
        }
        cost = at_cost(a, s, at, args.per);
      }
    }
    return g;
  }

  __device__ __forceinline__ void fill(AtSegment& g, int tile) {
    g.start = s.start;
    g.n = s.n;
    g.before = s.ctx - s.n;
    g.t0 = tile * 2 * args.per;
    g.keys[0] = attn_keys(args.a, s, g.t0, args.per);
    g.keys[1] = attn_keys(args.a, s, g.t0 + args.per, args.per);
  }
};

template <int DP>
__global__ void __launch_bounds__(kAtThreads, 1) k_attn_tc(const __grid_constant__ AttnTcArgs args) {
  using S = AtShape<DP>;
  constexpr int C = kAtC, kSegs = 4;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kFixed);
  uint64_t *full = bars, *empty = bars + 8, *q_full = bars + 16, *q_empty = bars + 17, *s_full = bars + 18, *p_ready = bars + 20,
           *o_full = bars + 22, *o_free = bars + 24, *seg_full = bars + 26, *seg_empty = bars + 30, *mma_done = bars + 34;
  auto* limit = reinterpret_cast<unsigned long long*>(bars + 35);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 36);
  uint32_t* bad = tmem_slot + 2;  // [16]: missing boxes of the last tiles of keys, a bit for 16 keys each
  AtSegment* segs = reinterpret_cast<AtSegment*>(bad + 16);
  static_assert(37 * 8 + 16 * 4 + kSegs * sizeof(AtSegment) <= 1024, "room behind the tiles");

  const AttnArgs& a = args.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, per = args.per;
  unsigned* status = a.status;

  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < S::kSlots; ++i) {
        mbar_init(&full[i], 1);
        mbar_init(&empty[i], 1);
      }
      mbar_init(q_full, 1);
      mbar_init(q_empty, 1);
      for (int x = 0; x < 2; ++x) {
        mbar_init(&s_full[x], 1);
        mbar_init(&p_ready[x], 4);
        mbar_init(&o_full[x], 1);
        mbar_init(&o_free[x], 4);
      }
      for (int i = 0; i < kSegs; ++i) {
        mbar_init(&seg_full[i], 1);
        mbar_init(&seg_empty[i], 10);
      }
      mbar_init(mma_done, 1);
      *limit = first_wait_limit(status);
      fence_barrier_init();
    }
    __syncwarp();
    tmem_alloc(tmem_slot, 512);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // The k-th segment, for the whole warp; false after a wait that ran out. Tiles of keys are counted over all segments: a
  // ring's place and a barrier's parity follow from the count.
  auto take = [&](int k, AtSegment& g) {
    if (!__all_sync(0xffffffffu, mbar_wait(&seg_full[k % kSegs], (k / kSegs) & 1, status, kErrTimeoutEpilogue))) return false;
    g = segs[k % kSegs];
    __syncwarp();
    if (lane == 0) mbar_arrive(&seg_empty[k % kSegs]);
    return g.b >= 0;
  };
  // tiles of keys [first, last) of tile x of rows
  auto last_of = [&](const AtSegment& g, int x) { return max(min(g.end, (g.keys[x] + C - 1) / C), g.first); };

  if (warp < 8) {
    at_regs_up<208>();
    // ------------------------------------------------------------ softmax, row r of tile x per thread
    const int x = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t s_col = lanes + S::kS + x * C, o_col = lanes + S::kO + x * DP;
    const float k2 = a.scale;  // times log2(e), not zero
    const uint32_t hidden = k2 > 0.f ? 0xff800000u : 0x7f800000u;
    bool ok = true;
    AtSegment g;
    int count = 0, outs = 0, seen = 0;  // tiles of keys of x, outputs of x, tiles of keys of all
    for (int k = 0; ok && take(k, g); ++k) {
      const int last = last_of(g, x), token = g.t0 + x * per + r / a.pack, h = g.hp * a.pack + r % a.pack;
      const bool there = r < per * a.pack && token < g.n;
      const int see = there ? min(g.before + token, g.keys[x] - 1) : -1;  // the last key of the row
      const int see_all = __reduce_min_sync(0xffffffffu, see);
      const bool some = __any_sync(0xffffffffu, there);  // rows are independent: a warp without any has nothing to do
      float m = -INFINITY, l = 0.f;
      for (int j = g.first; j < last; ++j, ++count) {
        ok = at_wait(&s_full[x], count & 1, status, kErrTimeoutEpilogue, *limit);
        if (!ok) break;
        if (some) {
          uint32_t v[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld_32x32_async(s_col + c * 32, v[c]);
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_wait_ld(v[c]);
          auto at = [&](int c) -> float { return __uint_as_float(v[c / 32][c % 32]); };
          const int left = see - j * C;  // the columns 0 .. left are seen
          if (see_all < j * C + C - 1) {
#pragma unroll
            for (int c = 0; c < C; ++c)
              if (c > left) v[c / 32][c % 32] = hidden;
          }
          if (a.page) {
            const uint32_t gone = bad[(seen + j - g.first) & 15];
            if (gone) {
#pragma unroll
              for (int c = 0; c < C; ++c)
                if (gone >> (c / 16) & 1) v[c / 32][c % 32] = hidden;
            }
          }
          float best[4];
          if (k2 > 0.f) {
#pragma unroll
            for (int c = 0; c < 4; ++c) best[c] = at(c);
#pragma unroll
            for (int c = 4; c < C; ++c) best[c % 4] = fmaxf(best[c % 4], at(c));
            best[0] = fmaxf(fmaxf(best[0], best[1]), fmaxf(best[2], best[3])) * k2;
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) best[c] = at(c);
#pragma unroll
            for (int c = 4; c < C; ++c) best[c % 4] = fminf(best[c % 4], at(c));
            best[0] = fminf(fminf(best[0], best[1]), fminf(best[2], best[3])) * k2;
          }
          if (j == g.first) {
            m = best[0];
          } else {
            const bool raise = best[0] > m + 8.f;
            if (__any_sync(0xffffffffu, raise)) {
              const float by = raise ? at_exp2(m - best[0]) : 1.f;  // 0 for the first key that is seen
              if (raise) m = best[0];
              l *= by;
#pragma unroll 1
              for (int c = 0; c < DP; c += 32) {
                float o[32];
                tmem_ld_32x32(o_col + c, o);
#pragma unroll
                for (int i = 0; i < 32; i += 2) mul2(o[i], o[i + 1], by, by);
                tmem_st_32x32(o_col + c, o);
              }
            }
          }
          const float base = m == -INFINITY ? 0.f : -m;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float e0 = __uint_as_float(v[c][2 * i]), e1 = __uint_as_float(v[c][2 * i + 1]);
              fma2(e0, e1, k2, base, base);
              e0 = at_exp2(e0);
              e1 = at_exp2(e1);
              at_add2(sum[(i & 1) * 2], sum[(i & 1) * 2 + 1], e0, e1);
              p[i] = pack_bf16x2(e0, e1);
            }
            tmem_st_32x16(s_col + c * 16, p);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[x]);
      }
      seen += g.end - g.first;
      const bool any = last > g.first;  // (uniform) otherwise O was not written
      if (ok && any) ok = at_wait(&o_full[x], outs++ & 1, status, kErrTimeoutEpilogue, *limit);
      if (!ok) break;
      if (some) {
        const float by = l == 0.f ? 0.f : 1.f / l;
        const long long t = g.start + token;
        const long long row = g.slot < 0 ? 0 : static_cast<long long>(g.slot) * 2 * C + x * C + r;
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + t * a.os[0] + h * a.os[1];
#pragma unroll 1
        for (int c = 0; c < DP; c += 32) {
          float u[32];
          if (any) tmem_ld_32x32(o_col + c, u);
#pragma unroll
          for (int i = 0; i < 32; ++i) u[i] = any && l != 0.f ? u[i] * by : 0.f;
          if (there) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              if (c + i >= a.D) continue;
              if (g.slot >= 0) {
                float4* p = reinterpret_cast<float4*>(a.part_o + row * a.D + c + i);
                p[0] = make_float4(u[i], u[i + 1], u[i + 2], u[i + 3]);
                p[1] = make_float4(u[i + 4], u[i + 5], u[i + 6], u[i + 7]);
              } else {
                *reinterpret_cast<uint4*>(o + c + i) =
                    make_uint4(pack_bf16x2(u[i], u[i + 1]), pack_bf16x2(u[i + 2], u[i + 3]), pack_bf16x2(u[i + 4], u[i + 5]),
                               pack_bf16x2(u[i + 6], u[i + 7]));
              }
            }
          }
        }
        if (there) {
          if (g.slot >= 0) a.part_ml[row] = make_float2(m, l);
          else if (a.lse) a.lse[static_cast<long long>(h) * a.T + t] = (m + log2f(l)) * kLn2;
        }
      }
      if (any) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_free[x]);
      }
    }
  } else {
    at_regs_down<88>();
    AtSegment g;
    if (warp == 8) {
      // ------------------------------------------------------------ TMA producer
      const int boxes = C / args.box;
      int n = 0, filled = 0, issued = 0;  // tiles of K and V, tiles of Q
      bool ok = true;
      for (int k = 0; ok && take(k, g); ++k) {
        if (g.first >= g.end) continue;
        const int top_keys = max(g.keys[0], g.keys[1]), hk = g.hp * a.pack / a.group;
        ok = __all_sync(0xffffffffu, mbar_wait(q_empty, (filled & 1) ^ 1, status, kErrTimeoutProducer));
        if (!ok) break;
        if (lane == 0) {
          const bool two[2] = {last_of(g, 0) > g.first, last_of(g, 1) > g.first};
          mbar_arrive_expect_tx(q_full, (two[0] + two[1]) * per * a.pack * DP * 2);
          for (int x = 0; x < 2; ++x)
            if (two[x])
              for (int d = 0; d < DP; d += 64)
                tma_load_4d(smem + x * S::kTile + d * C * 2, &args.q, q_full, d, g.hp * a.pack, g.start + g.t0 + x * per, 0);
        }
        ++filled;
        int page = a.pages;  // of this lane's box of keys; a.pages: none, whose box is zeros
        auto lookup = [&](int j) {
          if (!a.page || lane >= boxes) return;
          const int key = j * C + lane * args.box;
          page = a.pages;
          if (key < top_keys) {
            const int col = key / a.page;  // (keys end within the table)
            const int id = a.tables[static_cast<long long>(g.b) * a.width + col];
            if (id >= 0 && id < a.pages) page = id;
          }
        };
        lookup(g.first);
        for (int i = 0; i < 2 * (g.end - g.first); ++i, ++n) {  // K, V, K, V, ...
          const int j = g.first + i / 2, slot = n % S::kSlots;
          uint8_t* to = smem + S::kRing + slot * S::kTile;
          ok = __all_sync(0xffffffffu, mbar_wait(&empty[slot], ((n / S::kSlots) & 1) ^ 1, status, kErrTimeoutProducer));
          if (!ok) break;
          if (i % 2 == 0 && a.page) {
            const bool gone = lane < boxes && j * C + lane * args.box < top_keys && page == a.pages;
            if (gone) atomicOr(status, kErrPage);
            uint32_t bits = gone ? ((1u << (args.box / 16)) - 1) << (lane * args.box / 16) : 0u;
            bits = __reduce_or_sync(0xffffffffu, bits);
            if (lane == 0) bad[(n / 2) & 15] = bits;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(&full[slot], S::kTile);
          __syncwarp();
          const CUtensorMap* map = i % 2 ? &args.v : &args.k;
          const int head = hk * (i % 2 ? args.v_ext : args.k_ext);
          if (lane < boxes) {
            for (int d = 0; d < DP; d += 64) {
              if (a.page)
                tma_load_4d(to + d * C * 2 + lane * args.box * 128, map, &full[slot], d, (j * C + lane * args.box) % a.page, head,
                            page);
              else
                tma_load_4d(to + d * C * 2, map, &full[slot], d, g.start + j * C, head, 0);
            }
          }
          issued = n + 1;
          if (i % 2 == 1 && j + 1 < g.end) lookup(j + 1);
        }
      }
      for (n = max(issued - S::kSlots, 0); n < issued; ++n)  // every copy lands before the CTA leaves
        mbar_wait(&full[n % S::kSlots], (n / S::kSlots) & 1, status, kErrTimeoutDrain);
      if (filled) mbar_wait(q_full, (filled - 1) & 1, status, kErrTimeoutDrain);
    } else if (warp == 9) {
      // ----------------- MMA issuer: the whole warp in step (uniform addresses), one lane issues
      constexpr uint32_t idesc_s = umma_idesc(1, 128, C);
      constexpr uint32_t idesc_o = umma_idesc(1, 128, DP) | kIdescBMN;
      const bool leader = elect_one();
      auto wait = [&](uint64_t* bar, uint32_t ph) { return at_wait(bar, ph, status, kErrTimeoutMma); };
      const uint32_t base = smem_addr(smem);
      auto slot_addr = [&](int n) { return base + S::kRing + (n % S::kSlots) * S::kTile; };
      auto slot_full = [&](int n) { return wait(&full[n % S::kSlots], (n / S::kSlots) & 1); };
      auto scores = [&](int x, int n) {  // S of tile x of rows and the K tile at n
        const uint64_t q = umma_desc_sw128(base + x * S::kTile), k = umma_desc_sw128(slot_addr(n));
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < DP / 16; ++kk) {
            const uint32_t off = ((kk / 4) * C * 128 + (kk % 4) * 32) >> 4;
            umma_bf16(tmem + S::kS + x * C, q + off, k + off, idesc_s, kk ? 1u : 0u);
          }
          umma_commit(&s_full[x]);
        }
        __syncwarp();
      };
      auto output = [&](int x, int n, bool add, bool end) {  // O (+)= P V
        const uint64_t v = umma_desc_sw128_mn(slot_addr(n), C * 128);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < C / 16; ++kk)
            umma_bf16_ts(tmem + S::kO + x * DP, tmem + S::kS + x * C + kk * 8, v + kk * (2048 >> 4), idesc_o, add || kk > 0 ? 1u : 0u);
          if (end) umma_commit(&o_full[x]);
        }
        __syncwarp();
      };
      auto release = [&](uint64_t* bar) {
        if (leader) umma_commit(bar);
        __syncwarp();
      };
      bool ok = true;
      int n0 = 0, filled = 0, count[2] = {0, 0}, outs[2] = {0, 0};
      for (int k = 0; ok && take(k, g); ++k) {
        const int n_tiles = g.end - g.first;
        if (n_tiles <= 0) continue;
        const int last[2] = {last_of(g, 0), last_of(g, 1)}, top_keys = max(g.keys[0], g.keys[1]);
        // the tile whose last rows of V are behind the keys, or none
        const int tail = top_keys % C && g.end == (top_keys + C - 1) / C ? g.end - 1 : -1;
        ok = wait(q_full, filled++ & 1) && slot_full(n0);
        if (!ok) break;
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (g.first < last[x]) scores(x, n0);
        release(&empty[n0 % S::kSlots]);
        if (n_tiles == 1) release(q_empty);
        for (int i = 0; ok && i < n_tiles; ++i) {
          const int j = g.first + i, n = n0 + 2 * i;  // K at n, V at n + 1
          ok = slot_full(n + 1);
          if (ok && j == tail) {  // rows behind the keys: zeros (the softmax of this tile runs meanwhile)
            const uint32_t v = slot_addr(n + 1);
            for (int e = (top_keys - j * C) * 8 + lane; e < C * 8; e += 32)
#pragma unroll
              for (int d = 0; d < DP; d += 64) st_shared_v4(v + d * C * 2 + e * 16, 0u, 0u, 0u, 0u);
            fence_async_shared();
            __syncwarp();
          }
          ok = ok && (i + 1 == n_tiles || slot_full(n + 2));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (ok && j < last[x]) {
              ok = wait(&p_ready[x], count[x]++ & 1);
              // O of the segment before has been read
              if (ok && i == 0 && outs[x] > 0) ok = wait(&o_free[x], (outs[x] - 1) & 1);
              if (ok) {
                output(x, n + 1, i > 0, j + 1 == last[x]);
                if (j + 1 < last[x]) scores(x, n + 2);
                else ++outs[x];
              }
            }
          }
          if (ok) {
            release(&empty[(n + 1) % S::kSlots]);
            if (i + 1 < n_tiles) release(&empty[(n + 2) % S::kSlots]);
            if (i + 2 == n_tiles) release(q_empty);  // the last scores have been issued
          }
        }
        n0 += 2 * n_tiles;
      }
      if (leader) umma_commit(mma_done);
      __syncwarp();
      mbar_wait(mma_done, 0, status, kErrTimeoutDrain);
    } else if (warp == 10) {
      // ------------------------------------------------------------ scheduler
      AtScheduler work(args);
      for (int k = 0;; ++k) {
        g = work.next();
        if (!__all_sync(0xffffffffu, mbar_wait(&seg_empty[k % kSegs], ((k / kSegs) & 1) ^ 1, status, kErrTimeoutProducer))) break;
        if (lane == 0) {
          segs[k % kSegs] = g;
          mbar_arrive(&seg_full[k % kSegs]);
        }
        __syncwarp();
        if (g.b < 0) break;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of units that cuts go through: CTA (c, y) the unit whose first part CTA c holds, a warp a row.
__global__ void __launch_bounds__(256) k_attn_tc_join(const __grid_constant__ AttnTcArgs args) {
  const AttnArgs& a = args.a;
  const AttnPart head = a.part_head[blockIdx.x];
  if (head.parts == 0) return;
  const int lane = threadIdx.x & 31;
  for (int row = blockIdx.y * 8 + (threadIdx.x >> 5); row < 2 * kAtC; row += gridDim.y * 8) {
    const int x = row / kAtC, r = row % kAtC, token = x * args.per + r / a.pack;
    if (r >= args.per * a.pack || token >= head.left) continue;
    // the first part lies at CTA c's odd slot, the others at the even ones of those behind it
    auto at = [&](int i) { return (2ll * (blockIdx.x + i) + (i == 0 ? 1 : 0)) * 2 * kAtC + row; };
    float top = -INFINITY;
    for (int i = lane; i < head.parts; i += 32) top = fmaxf(top, a.part_ml[at(i)].x);
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i0 = 0; i0 < head.parts; i0 += 32) {
      const int i = i0 + lane;
      const float2 ml = i < head.parts ? a.part_ml[at(i)] : make_float2(-INFINITY, 0.f);
      const float w = ml.y == 0.f ? 0.f : ml.y * exp2f(ml.x - base);
      sum += w;
      const int some = min(32, head.parts - i0);
#pragma unroll 4
      for (int e = 0; e < some; ++e) {
        const float we = __shfl_sync(0xffffffffu, w, e);
        if (lane * 4 < a.D) {
          const float4 o = *reinterpret_cast<const float4*>(a.part_o + at(i0 + e) * a.D + lane * 4);
          acc[0] += we * o.x;
          acc[1] += we * o.y;
          acc[2] += we * o.z;
          acc[3] += we * o.w;
        }
      }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    const float by = sum == 0.f ? 0.f : 1.f / sum;
    const int h = head.hp * a.pack + r % a.pack;
    const long long t = head.token + token;
    if (lane * 4 < a.D)
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + t * a.os[0] + h * a.os[1] + lane * 4) =
          make_uint2(pack_bf16x2(acc[0] * by, acc[1] * by), pack_bf16x2(acc[2] * by, acc[3] * by));
    if (a.lse && lane == 0) a.lse[static_cast<long long>(h) * a.T + t] = (top + log2f(sum)) * kLn2;
  }
}

}  // namespace pc

// The backward call of the attention on tcgen05: one kernel for the gradients
// of keys and values, one for those of the queries.  Each makes the scores
// again (seven products in all, where one kernel for everything would take
// five but add up dq in an order that is not fixed).
#include "attention_tiles.cuh"

namespace snack {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kHalf = kTile / 2;  // columns of a tile that a warpgroup takes
constexpr int kStatWarp = 10;

// T is the type of the call's tensors and Op that of the operands: T's own, or float16
// for bfloat16 calls of more than 64 columns and some work (halves_take), whose
// tensors are made in it first, times a power of two for each sequence and key head.
// Float16 has 11 bits, so that probabilities and gradients of scores in one part
// leave bfloat16's results as their rounding does, in seven products for both kernels
// where two parts of both take ten.
//
// Else left operands of the second products are in two parts where rounding them
// to one shows in the results.  Gradients of scores: dq and dk would be 1.5 times as far
// off as rounding them alone.  Bfloat16's probabilities: dv 1.4 times (two parts cost 9
// packed sequences at 64 columns 322 -> 334 us, 8192 tokens at 128 1902 -> 2012, forward
// included).  Float16's are in one: 1.4 times, in a type of eight times the precision.
template <typename T, typename Op>
constexpr bool kHalves = std::is_same<T, __nv_bfloat16>::value && std::is_same<Op, __half>::value;
template <typename T, typename Op>
constexpr bool kFineScores = !kHalves<T, Op>;
template <typename Op>
constexpr bool kFineProbs = !std::is_same<Op, __half>::value;

// What brings back a product with a tensor that was made in float16; `sequence`
// numbers the tensor's side as find_tile does.
__device__ __forceinline__ float halves_back(const int32_t *peak, int sequence, int key_heads, int kh) {
  return power_of_two(-power_to_half((uint32_t)__ldg(peak + (int64_t)sequence * key_heads + kh)));
}
__device__ __forceinline__ int other_sequence(int s, bool ragged, bool other_ragged) {
  return s - (ragged ? 1 : 0) + (other_ragged ? 1 : 0);
}

// 32 values of a row, columns [x, x + 32) of a warpgroup's 64 that begin at `at`, as
// the left operand of a product.
template <typename T, bool FINE>
__device__ __forceinline__ void store_row32(uint32_t at, int x, const float *v) {
  if constexpr (FINE) {
    store_parts<typename Operand<T>::type>(at + x, v);
  } else {
    uint32_t out[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) out[e] = pack2<T>(v[2 * e], v[2 * e + 1]);
    tc::store16(at + x / 2, out);
  }
}
template <typename T, int DP, bool FINE>
__device__ __forceinline__ void row_sums(uint32_t d, uint32_t a, uint32_t b, bool add) {
  if constexpr (FINE && !Operand<T>::kSplit)
    fine_sums<T, DP>(d, a, b, add);
  else
    sums<T, DP, kTile>(d, a, b, add);
}

// float16 operands hold neither small probabilities nor small gradients of scores:
// they are taken times powers of two (attention.cuh).  bfloat16 has the range of 32
// bits.
template <typename T>
constexpr bool kScaled = !std::is_same<T, __nv_bfloat16>::value;
template <typename T>
constexpr float kUp = kScaled<T> ? kHalfP : 0.f;  // the power of the probabilities

// The two warps that have a row's 64 columns each tell one another the exponents of
// their largest gradients of scores.
struct Tops {
  uint64_t told[4];  // a pair of warps each
  uint8_t exponent[2][2][kTile];
};
// The row's, of step n; false: the wait has run out.  Whole warps.
__device__ __forceinline__ bool row_exponent(Tops &tops, const float (&t)[kHalf], int n, uint32_t *exponent,
                                             volatile int *failed, int polls) {
  const int warp = threadIdx.x >> 5, w = warp >> 2, pair = warp & 3, row = pair * 32 + (threadIdx.x & 31);
  float top[2] = {};
#pragma unroll
  for (int x = 0; x < kHalf; x += 4) {
    top[0] = tc::max3(top[0], fabsf(t[x]), fabsf(t[x + 1]));
    top[1] = tc::max3(top[1], fabsf(t[x + 2]), fabsf(t[x + 3]));
  }
  *exponent = exponent_bits(fmaxf(top[0], top[1]));
  tops.exponent[n & 1][w][row] = (uint8_t)*exponent;
  tc::bar_arrive_warp(&tops.told[pair]);
  if (!__all_sync(0xffffffffu, tc::bar_wait(&tops.told[pair], n & 1, failed, polls))) return false;
  *exponent = max(*exponent, (uint32_t)tops.exponent[n & 1][w ^ 1][row]);
  return true;
}

// N columns of tensor memory times a factor.  Whole warps.
template <int N>
__device__ __forceinline__ void multiply_sums(uint32_t at, float by) {
#pragma unroll
  for (int c = 0; c < N; c += 32) {
    float v[32];
    tc::load32(at + c, v);
    tc::wait_loads();
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] *= by;
    tc::store32(at + c, reinterpret_cast<const uint32_t *>(v));
  }
}

// ------------------------------------------------------------------ keys and values

struct KeyBars {
  uint64_t kv, q_full[2], q_empty[2], d_full[2], d_empty[2], stat_full[2], stat_empty[2];
  uint64_t scores, probs, dprobs, dscores, done, cut, drain;
  uint32_t tmem;
  int failed, copied;  // copied: tiles of queries and dout whose copies were started
  alignas(16) float lse[2][kTile];
  alignas(16) float delta[2][kTile];
  struct {
    float scores, dprobs, q, dout;
  } by[2];  // what a tile of queries' products are multiplied by
  Tops tops;
};

template <int W>
constexpr size_t keys_smem() { return 1024 + (size_t)6 * tile_bytes<W>(); }

// A block whose wait has given up (as in the forward call).
__device__ __forceinline__ void drain_copies(KeyBars &bars) {
  tc::bar_drain(&bars.kv, 0);
  for (int i = max(0, bars.copied - 4); i < bars.copied; ++i)
    tc::bar_drain(i & 1 ? &bars.d_full[i / 2 & 1] : &bars.q_full[i / 2 & 1], (i / 4) & 1);
}
template <typename T>
__device__ __noinline__ void poison_keys(const AttnCall &c) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, kh = blockIdx.x % c.key_heads;
  if (threadIdx.x == 0) g_attention_failed = 1;
  const Place at = find_tile(c.k_offsets, c.sequences, c.k_tokens, 1, kTile, blockIdx.x / c.key_heads, false);
  const Span ks = own_span(c.k_offsets, c.k_lengths, at.s, c.sequences, c.k_tokens);
  const Strided &to = warp >> 2 ? c.dv : c.dk;
  const int j = at.tile * kTile + (warp & 3) * 32 + lane;
  if (j < ks.cover && to.p)
    poison_row(static_cast<T *>(to.p) + (c.k_offsets ? (ks.row + j) * to.token : ks.seq * to.seq + j * to.token) +
                   kh * to.head, c.d);
}

// A tile of 128 keys (rows of every product: a thread has a key), past which
// the query tiles of all heads that share it stream:
//   S^T = K Q^T,  P^T = exp2(S^T - lse),  dP^T = V dO^T,  dS^T = P^T (dP^T - delta),
//   dV += P^T dO,  dK += dS^T Q.
// Order of the products: dV(n), S(n+1), dK(n), dP(n+1), so that the
// exponentials of n+1 run while dK(n) and dP(n+1) do, and dS(n+1) while dV(n+1)
// does.  Scores, dP and both sums fill the 512 columns of tensor memory.
template <typename T, typename Op, int DP, bool DROP>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_backward_keys(const __grid_constant__ AttnCall c, const __grid_constant__ TileMaps maps) {
  constexpr int W = wide<Op, DP>();
  constexpr bool kSplit = Operand<Op>::kSplit;
  extern __shared__ unsigned char raw[];
  __shared__ KeyBars bars;
  unsigned char *const sk = align1024(raw), *const sv = sk + tile_bytes<W>();
  unsigned char *const sq = sv + tile_bytes<W>(), *const sd = sq + 2 * tile_bytes<W>();
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  volatile int *const failed = &bars.failed;

  // the queries' kernel, which needs nothing of this one, may begin on SMs that this one leaves
  dependency_launch();
  // barriers, tensor memory and the block's place are made ready side by side
  if (warp == kCopyWarp && lane == 0) {
    tc::bar_init(&bars.kv, 2);
    for (int i = 0; i < 4; ++i) tc::bar_init(&bars.tops.told[i], 2);
    for (int i = 0; i < 2; ++i) {
      tc::bar_init(&bars.q_full[i], 1);
      tc::bar_init(&bars.q_empty[i], 1);
      tc::bar_init(&bars.d_full[i], 1);
      tc::bar_init(&bars.d_empty[i], 1);
      tc::bar_init(&bars.stat_full[i], 1);
      tc::bar_init(&bars.stat_empty[i], 8);
    }
    tc::bar_init(&bars.scores, 1);
    tc::bar_init(&bars.probs, 8);
    tc::bar_init(&bars.dprobs, 1);
    tc::bar_init(&bars.dscores, 8);
    tc::bar_init(&bars.done, 1);
    tc::bar_init(&bars.cut, 1);
    tc::bar_init(&bars.drain, 1);
    bars.failed = 0;
    tc::fence_bar_init();
    tc::prefetch_map(&maps.k);
    tc::prefetch_map(&maps.v);
    tc::prefetch_map(&maps.q);
    tc::prefetch_map(&maps.dout);
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(&bars.tmem, 512);
    tc::fence_before();
  }
  const int kh = blockIdx.x % c.key_heads, G = c.group;
  const Place at = find_tile(c.k_offsets, c.sequences, c.k_tokens, 1, kTile, blockIdx.x / c.key_heads, false);
  if (at.s < 0) return leave_block(warp, &bars.tmem);
  const Span ks = own_span(c.k_offsets, c.k_lengths, at.s, c.sequences, c.k_tokens);
  const Span qs = other_span(c.q_offsets, c.q_lengths, at.s, c.k_offsets != nullptr, c.sequences, c.q_tokens);
  const int j0 = at.tile * kTile, nq = qs.valid, nk = ks.valid;
  const int first = first_query(c.causal, j0, nq, nk), tile0 = first / kTile;
  const int tiles = first < nq ? (nq + kTile - 1) / kTile - tile0 : 0;
  const int all = tiles * G;

  const int q_token = c.q_offsets ? (int)qs.row : 0, k_token = c.k_offsets ? (int)ks.row : 0;
  if (warp == kCopyWarp && lane == 0 && all > 0) {
    copy_tile<W>(sk, &maps.k, &bars.kv, kh, k_token + j0, ks.seq);
    copy_tile<W>(sv, &maps.v, &bars.kv, kh, k_token + j0, ks.seq);
  }
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = bars.tmem;  // S, dP, dV, dK

  if (warp >= kCopyWarp) {
    tc::leave_registers<kOtherRegisters>();
    if (warp == kCopyWarp && all > 0) {
      int cut_phase = 0, n = 0, parts = 0;
      bool ok = true;
      for (; n < all && ok; ++n) {
        const int slot = n & 1, g = n / tiles, q0 = (tile0 + n - g * tiles) * kTile, head = kh * G + g;
        for (int side = 0; side < 2 && ok; ++side) {
          uint64_t *const full = side ? &bars.d_full[slot] : &bars.q_full[slot];
          if (n >= 2)
            ok = __all_sync(0xffffffffu, tc::bar_wait(side ? &bars.d_empty[slot] : &bars.q_empty[slot],
                                                      (n / 2 - 1) & 1, failed, c.polls));
          if (!ok) break;
          unsigned char *const to = (side ? sd : sq) + slot * tile_bytes<W>();
          const CUtensorMap *const map = side ? &maps.dout : &maps.q;
          if (q0 + kTile > nq)
            ok = copy_tile_cut<W>(to, map, full, &bars.cut, &cut_phase, head, q_token + q0, qs.seq, nq - q0, failed,
                                   c.polls);
          else if (lane == 0)
            copy_tile<W>(to, map, full, head, q_token + q0, qs.seq);
          __syncwarp();
          ++parts;
        }
      }
      if (lane == 0) bars.copied = parts;
    } else if (warp == kMmaWarp) {
      // the whole warp goes along, so that descriptors stay in uniform registers
      if (all > 0) {
        constexpr uint32_t kStep = tile_bytes<W>() / 16;
        const bool leader = tc::elect_one();
        const uint32_t k0 = tc::desc_rows(tc::smem_addr(sk)), v0 = tc::desc_rows(tc::smem_addr(sv));
        const uint32_t q0 = tc::desc_rows(tc::smem_addr(sq)), d0 = tc::desc_rows(tc::smem_addr(sd));
        const uint32_t q0c = tc::desc_columns(tc::smem_addr(sq), kBlock), d0c = tc::desc_columns(tc::smem_addr(sd), kBlock);
        const uint32_t t_s = tmem, t_dp = tmem + kTile, t_dv = tmem + 2 * kTile, t_dk = t_dv + DP;
        const auto wait = [&](uint64_t *bar, int phase) {
          const bool done = __all_sync(0xffffffffu, tc::bar_wait(bar, phase, failed, c.polls));
          tc::fence_after();
          return done;
        };
        const auto scores = [&](int n) {
          const bool done = wait(&bars.q_full[n & 1], (n / 2) & 1);
          if (done && leader) {
            products<Op, DP>(t_s, k0, q0 + (n & 1) * kStep);
            tc::commit(&bars.scores);
          }
          __syncwarp();
          return done;
        };
        const auto dprobs = [&](int n) {
          const bool done = wait(&bars.d_full[n & 1], (n / 2) & 1);
          if (done && leader) {
            products<Op, DP>(t_dp, v0, d0 + (n & 1) * kStep);
            tc::commit(&bars.dprobs);
          }
          __syncwarp();
          return done;
        };
        bool ok = wait(&bars.kv, 0) && scores(0) && dprobs(0);
        for (int n = 0; n < all && ok; ++n) {
          ok = wait(&bars.probs, n & 1);
          if (!ok) break;
          if (leader) {
            row_sums<Op, DP, kFineProbs<Op>>(t_dv, t_s, d0c + (n & 1) * kStep, n > 0);
            tc::commit(&bars.d_empty[n & 1]);
          }
          __syncwarp();
          if (n + 1 < all) ok = scores(n + 1);
          ok = ok && wait(&bars.dscores, n & 1);
          if (!ok) break;
          if (leader) {
            row_sums<Op, DP, kFineScores<T, Op>>(t_dk, t_dp, q0c + (n & 1) * kStep, n > 0);
            tc::commit(&bars.q_empty[n & 1]);
          }
          __syncwarp();
          if (n + 1 < all) ok = dprobs(n + 1);
        }
        if (leader) {
          tc::commit(&bars.done);
          tc::commit(&bars.drain);
        }
        tc::bar_drain(&bars.drain, 0);
      }
      __syncwarp();
    } else if (warp == kStatWarp) {
      constexpr float up = kUp<Op>;
      float k_back = 1.f, v_back = 1.f;
      if (kSplit && all > 0) {
        k_back = power_back(c.k_power, ks.tile + at.tile, c.key_heads, kh);
        v_back = power_back(c.v_power, ks.tile + at.tile, c.key_heads, kh);
      }
      for (int n = 0; n < all; ++n) {
        const int slot = n & 1, g = n / tiles, q0 = (tile0 + n - g * tiles) * kTile;
        const int64_t place = (int64_t)(kh * G + g) * c.rows + qs.row;
        float lse[4], delta[4], q_back = 1.f, d_back = 1.f;
        if (kSplit) {
          q_back = power_back(c.q_power, qs.tile + q0 / kTile, c.heads, kh * G + g);
          d_back = power_back(c.dout_power, qs.tile + q0 / kTile, c.heads, kh * G + g);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int i = q0 + lane + 32 * x;
          lse[x] = i < nq ? c.lse[place + i] * kLog2e : INFINITY;
          if (lse[x] == -INFINITY) lse[x] = INFINITY;  // a row that sees nothing: its probabilities are zero
          delta[x] = i < nq ? c.delta[place + i] : 0.f;
        }
        if (n >= 2 && !__all_sync(0xffffffffu, tc::bar_wait(&bars.stat_empty[slot], (n / 2 - 1) & 1, failed, c.polls))) break;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          bars.lse[slot][lane + 32 * x] = up - lse[x];  // as they are added
          bars.delta[slot][lane + 32 * x] = -delta[x] * exp2f(-up);  // (times probabilities that are that power up)
        }
        if (lane == 0) bars.by[slot] = {c.scale_log2 * k_back * q_back, v_back * d_back * exp2f(-up), q_back, d_back};
        tc::bar_arrive_warp(&bars.stat_full[slot]);
      }
    }
  } else {
    tc::take_registers<kRowRegisters>();
    const int w = warp >> 2, j = j0 + (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + w * kHalf, dp_at = s_at + kTile;
    float acc[kSplit ? DP : 1] = {};  // split: the sums of dK (first warpgroup) or dV
    float back = 0.f;                 // split: what the last step's are multiplied by
    int power = kMostPower;           // else of the row's sums
    float scores_by = c.scale_log2, dprobs_by = exp2f(-kUp<Op>);
    if (kHalves<T, Op> && all > 0) {
      const int q_at = other_sequence(at.s, c.k_offsets != nullptr, c.q_offsets != nullptr);
      scores_by *= halves_back(c.k_power, at.s, c.key_heads, kh) * halves_back(c.q_power, q_at, c.key_heads, kh);
      dprobs_by *= halves_back(c.v_power, at.s, c.key_heads, kh) * halves_back(c.dout_power, q_at, c.key_heads, kh);
    }
    const bool alone = nk == 1 || (c.causal && j0 == 0 && (warp & 3) == 0);
    const uint64_t seed = DROP ? c.draws() : 0;
    bool ok = true;
    for (int n = 0; n < all; ++n) {
      const int slot = n & 1, g = n / tiles, q0 = (tile0 + n - g * tiles) * kTile + w * kHalf;
      uint64_t kept[4];  // of the four keys whose draws are shared, for 64 queries
      if (DROP) {
        uint64_t own = 0;
#pragma unroll
        for (int x = 0; x < kHalf; x += 4) {
          // this lane draws for one of four queries, for four keys
          const uint64_t z = dropout_draw(
              dropout_row(seed, qs.row + q0 + x + (lane & 3), c.heads, kh * G + g), j);
          uint32_t bits = 0;
#pragma unroll
          for (int y = 0; y < 4; ++y) bits |= draw_lane(z, y) >= c.drop ? 1u << y : 0u;
          own |= (uint64_t)bits << x;
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) kept[y] = __shfl_sync(0xffffffffu, own, (lane & ~3) + y) >> (lane & 3);
      }
      ok = __all_sync(0xffffffffu, tc::bar_wait(&bars.stat_full[slot], (n / 2) & 1, failed, c.polls) &&
                                       tc::bar_wait(&bars.scores, n & 1, failed, c.polls));
      if (!ok) break;
      tc::fence_after();
      if constexpr (kSplit)
        if (w) {
          if (n > 0) add_sums<DP>(acc, tmem + lanes + 2 * kTile, back);  // dV of the tile before
          back = bars.by[slot].dout;
        }
      const float cs = kSplit ? bars.by[slot].scores : scores_by, dprobs = kSplit ? bars.by[slot].dprobs : dprobs_by;
      const float2 cs2 = make_float2(cs, cs);
      float p[kHalf];
      tc::load32(s_at, p);
      tc::load32(s_at + 32, p + 32);
      tc::wait_loads();
#pragma unroll
      for (int x = 0; x < kHalf; x += 4) {
        const float4 l = *reinterpret_cast<const float4 *>(&bars.lse[slot][w * kHalf + x]);
        const float2 a = tc::fma2(make_float2(p[x], p[x + 1]), cs2, make_float2(l.x, l.y));
        const float2 b = tc::fma2(make_float2(p[x + 2], p[x + 3]), cs2, make_float2(l.z, l.w));
        p[x] = tc::exp2_fast(a.x);
        p[x + 1] = tc::exp2_fast(a.y);
        p[x + 2] = tc::exp2_fast(b.x);
        p[x + 3] = tc::exp2_fast(b.y);
      }
      if (c.causal) {
        const int lo = j - (nk - nq) - q0;  // the first query that sees this key
        if (__any_sync(0xffffffffu, lo > 0))
#pragma unroll
          for (int x = 0; x < kHalf; ++x) p[x] = x >= lo ? p[x] : 0.f;
      }
#pragma unroll
      for (int x = 0; x < kHalf; x += 32) {
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = !DROP || (kept[e & 3] >> ((x + e) & ~3) & 1) ? p[x + e] : 0.f;
        store_row32<Op, kFineProbs<Op>>(s_at, x, v);
      }
      tc::wait_stores();
      tc::fence_before();
      tc::bar_arrive_warp(&bars.probs);
      ok = __all_sync(0xffffffffu, tc::bar_wait(&bars.dprobs, n & 1, failed, c.polls));
      if (!ok) break;
      tc::fence_after();
      if constexpr (kSplit)
        if (!w && n > 0) add_sums<DP>(acc, tmem + lanes + 2 * kTile + DP, back);  // dK of the tile before
#pragma unroll
      for (int c0 = 0; c0 < kHalf; c0 += 32) {  // dS takes the probabilities' place
        float t[32];
        tc::load32(dp_at + c0, t);
        tc::wait_loads();
#pragma unroll
        for (int x = 0; x < 32; x += 4) {
          const float4 d = *reinterpret_cast<const float4 *>(&bars.delta[slot][w * kHalf + c0 + x]);
          float v[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            v[y] = t[x + y] * dprobs;
            if (DROP) v[y] = kept[y] >> (c0 + x) & 1 ? v[y] * c.keep_scale : 0.f;
          }
          const float2 u0 = tc::add2(make_float2(v[0], v[1]), make_float2(d.x, d.y));
          const float2 u1 = tc::add2(make_float2(v[2], v[3]), make_float2(d.z, d.w));
          const float2 r0 = tc::mul2(make_float2(p[c0 + x], p[c0 + x + 1]), u0);
          const float2 r1 = tc::mul2(make_float2(p[c0 + x + 2], p[c0 + x + 3]), u1);
          p[c0 + x] = r0.x;
          p[c0 + x + 1] = r0.y;
          p[c0 + x + 2] = r1.x;
          p[c0 + x + 3] = r1.y;
        }
      }
      if (alone) {  // queries that see one key: P = 1 whatever the score, dS is zero
#pragma unroll
        for (int x = 0; x < kHalf; ++x)
          if (nk == 1 || (j == 0 && q0 + x == nq - nk)) p[x] = 0.f;
      }
      if constexpr (kScaled<Op>) {
        uint32_t exponent;
        ok = row_exponent(bars.tops, p, n, &exponent, failed, c.polls);
        if (!ok) break;
        float up;
        if constexpr (kSplit) {
          const int now = row_power(exponent, 14, 0);
          up = power_of_two(now);
          if (!w) back = power_of_two(-now) * bars.by[slot].q;
        } else {  // (the sums so far are complete: these dP come after them)
          const int now = running_power(power, exponent);
          if (n > 0 && __any_sync(0xffffffffu, now != power))
            multiply_sums<DP / 2>(tmem + lanes + 2 * kTile + DP + w * (DP / 2), exp2f((float)(now - power)));
          power = now;
          up = power_of_two(power);
        }
#pragma unroll
        for (int x = 0; x < kHalf; ++x) p[x] *= up;
      }
      store_row32<Op, kFineScores<T, Op>>(dp_at, 0, p);
      store_row32<Op, kFineScores<T, Op>>(dp_at, 32, p + 32);
      tc::wait_stores();
      tc::fence_before();
      tc::bar_arrive_warp(&bars.dscores);
      if (lane == 0) tc::bar_arrive(&bars.stat_empty[slot]);
    }
    if (ok && all > 0) {
      ok = __all_sync(0xffffffffu, tc::bar_wait(&bars.done, 0, failed, c.polls));
      tc::fence_after();
    }
    const Strided &to = w ? c.dv : c.dk;  // a warpgroup each
    if (ok && to.p) {
      T *row = nullptr;
      if (j < ks.cover)
        row = static_cast<T *>(to.p) + (c.k_offsets ? (ks.row + j) * to.token : ks.seq * to.seq + j * to.token) +
              kh * to.head;
      float factor = w ? exp2f(-kUp<Op>) * c.keep_scale : c.scale;
      if (kHalves<T, Op> && all > 0)
        factor *= halves_back(w ? c.dout_power : c.q_power,
                              other_sequence(at.s, c.k_offsets != nullptr, c.q_offsets != nullptr), c.key_heads, kh);
      if constexpr (kSplit) {
        if (all > 0) add_sums<DP>(acc, tmem + lanes + 2 * kTile + (w ? 0 : DP), back);
        store_floats<DP>(row, acc, factor, c.d, j >= nk);
      } else {
        if (kScaled<Op> && !w) factor *= power_of_two(-power);
        store_sums<T, DP>(tmem + lanes + 2 * kTile + (w ? 0 : DP), row, factor, c.d, all > 0, j >= nk);
      }
    }
    tc::fence_before();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::tmem_free(tmem, 512);
  }
  if (bars.failed) {
    if (warp == kCopyWarp) drain_copies(bars);
    if (warp < kCopyWarp) poison_keys<T>(c);
  }
}

// ------------------------------------------------------------------ queries

struct QueryBars {
  uint64_t qd, k_full[3], k_empty[3], v_full[2], v_empty[2];
  uint64_t scores[2], read[2], dprobs[2], dscores[2], done, cut, drain;
  uint32_t tmem;
  int failed, copied_k, copied_v;  // copied: tiles whose copies were started
  Tops tops;
};

template <int W>
constexpr size_t queries_smem() { return 1024 + (size_t)7 * tile_bytes<W>(); }

__device__ __forceinline__ void drain_copies(QueryBars &bars) {
  tc::bar_drain(&bars.qd, 0);
  for (int i = max(0, bars.copied_k - 3); i < bars.copied_k; ++i) tc::bar_drain(&bars.k_full[i % 3], (i / 3) & 1);
  for (int i = max(0, bars.copied_v - 2); i < bars.copied_v; ++i) tc::bar_drain(&bars.v_full[i & 1], (i / 2) & 1);
}
template <typename T>
__device__ __noinline__ void poison_queries(const AttnCall &c) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, head = blockIdx.x % c.heads;
  if (threadIdx.x == 0) g_attention_failed = 1;
  const Place at = find_tile(c.q_offsets, c.sequences, c.q_tokens, 1, kTile, blockIdx.x / c.heads, c.causal);
  const Span qs = own_span(c.q_offsets, c.q_lengths, at.s, c.sequences, c.q_tokens);
  const int i = at.tile * kTile + (warp & 3) * 32 + lane;
  if (warp < 4 && i < qs.cover)
    poison_row(static_cast<T *>(c.dq.p) +
                   (c.q_offsets ? (qs.row + i) * c.dq.token : qs.seq * c.dq.seq + i * c.dq.token) + head * c.dq.head, c.d);
}

// A tile of 128 queries of one head, past which the keys stream:
//   S = Q K^T,  P = exp2(S - lse),  dP = dO V^T,  dS = P (dP - delta),  dQ += dS K.
// Scores and dP take turns in three buffers of tensor memory (S(n) in 2n mod 3,
// dP(n) in 2n+1 mod 3), so that S(n+1) is there before the rows are done with n.
// Order of the products: dP(n+1), dQ(n), S(n+2).
template <typename T, typename Op, int DP, bool DROP>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_backward_queries(const __grid_constant__ AttnCall c, const __grid_constant__ TileMaps maps) {
  constexpr int W = wide<Op, DP>();
  constexpr bool kSplit = Operand<Op>::kSplit;
  extern __shared__ unsigned char raw[];
  __shared__ QueryBars bars;
  unsigned char *const sq = align1024(raw), *const sd = sq + tile_bytes<W>();
  unsigned char *const sk = sd + tile_bytes<W>(), *const sv = sk + 3 * tile_bytes<W>();
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  volatile int *const failed = &bars.failed;

  if (warp == kCopyWarp && lane == 0) {
    tc::bar_init(&bars.qd, 2);
    for (int i = 0; i < 4; ++i) tc::bar_init(&bars.tops.told[i], 2);
    for (int i = 0; i < 3; ++i) {
      tc::bar_init(&bars.k_full[i], 1);
      tc::bar_init(&bars.k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::bar_init(&bars.v_full[i], 1);
      tc::bar_init(&bars.v_empty[i], 1);
      tc::bar_init(&bars.scores[i], 1);
      tc::bar_init(&bars.read[i], 8);
      tc::bar_init(&bars.dprobs[i], 1);
      tc::bar_init(&bars.dscores[i], 8);
    }
    tc::bar_init(&bars.done, 1);
    tc::bar_init(&bars.cut, 1);
    tc::bar_init(&bars.drain, 1);
    bars.failed = 0;
    tc::fence_bar_init();
    tc::prefetch_map(&maps.q);
    tc::prefetch_map(&maps.dout);
    tc::prefetch_map(&maps.k);
    tc::prefetch_map(&maps.v);
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(&bars.tmem, 512);
    tc::fence_before();
  }
  const int head = blockIdx.x % c.heads, kh = head / c.group;
  const Place at = find_tile(c.q_offsets, c.sequences, c.q_tokens, 1, kTile, blockIdx.x / c.heads, c.causal);
  if (at.s < 0) {
    if (blockIdx.x == gridDim.x - 1) dependency_wait();
    return leave_block(warp, &bars.tmem);
  }
  const Span qs = own_span(c.q_offsets, c.q_lengths, at.s, c.sequences, c.q_tokens);
  const Span ks = other_span(c.k_offsets, c.k_lengths, at.s, c.q_offsets != nullptr, c.sequences, c.k_tokens);
  const int i0 = at.tile * kTile, nq = qs.valid, nk = ks.valid;
  const int last = min(i0 + kTile, nq) - 1;
  const int all = i0 < nq ? (max(0, seen_keys(c.causal, last, nq, nk)) + kTile - 1) / kTile : 0;

  const int q_token = c.q_offsets ? (int)qs.row : 0, k_token = c.k_offsets ? (int)ks.row : 0;
  if (warp == kCopyWarp && lane == 0 && all > 0) {
    copy_tile<W>(sq, &maps.q, &bars.qd, head, q_token + i0, qs.seq);
    copy_tile<W>(sd, &maps.dout, &bars.qd, head, q_token + i0, qs.seq);
  }
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = bars.tmem;  // three buffers, dQ

  if (warp >= kCopyWarp) {
    tc::leave_registers<kOtherRegisters>();
    if (warp == kCopyWarp && all > 0) {
      int cut_phase = 0, ks_done = 0, vs_done = 0;
      bool ok = true;
      for (int n = 0; n < all && ok; ++n) {
        if (n >= 3) ok = __all_sync(0xffffffffu, tc::bar_wait(&bars.k_empty[n % 3], (n / 3 - 1) & 1, failed, c.polls));
        if (!ok) break;
        unsigned char *const to = sk + n % 3 * tile_bytes<W>();
        if ((n + 1) * kTile > nk)
          ok = copy_tile_cut<W>(to, &maps.k, &bars.k_full[n % 3], &bars.cut, &cut_phase, kh, k_token + n * kTile,
                                 ks.seq, nk - n * kTile, failed, c.polls);
        else if (lane == 0)
          copy_tile<W>(to, &maps.k, &bars.k_full[n % 3], kh, k_token + n * kTile, ks.seq);
        __syncwarp();
        ++ks_done;
        if (!ok) break;
        if (n >= 2) ok = __all_sync(0xffffffffu, tc::bar_wait(&bars.v_empty[n & 1], (n / 2 - 1) & 1, failed, c.polls));
        if (!ok) break;
        if (lane == 0)
          copy_tile<W>(sv + (n & 1) * tile_bytes<W>(), &maps.v, &bars.v_full[n & 1], kh, k_token + n * kTile, ks.seq);
        __syncwarp();
        ++vs_done;
      }
      if (lane == 0) {
        bars.copied_k = ks_done;
        bars.copied_v = vs_done;
      }
    } else if (warp == kMmaWarp) {
      if (all > 0) {
        constexpr uint32_t kStep = tile_bytes<W>() / 16;
        const bool leader = tc::elect_one();
        const uint32_t q0 = tc::desc_rows(tc::smem_addr(sq)), d0 = tc::desc_rows(tc::smem_addr(sd));
        const uint32_t k0 = tc::desc_rows(tc::smem_addr(sk)), v0 = tc::desc_rows(tc::smem_addr(sv));
        const uint32_t k0c = tc::desc_columns(tc::smem_addr(sk), kBlock);
        const auto wait = [&](uint64_t *bar, int phase) {
          const bool done = __all_sync(0xffffffffu, tc::bar_wait(bar, phase, failed, c.polls));
          tc::fence_after();
          return done;
        };
        const auto scores = [&](int n) {
          const bool done = wait(&bars.k_full[n % 3], (n / 3) & 1);
          if (done && leader) {
            products<Op, DP>(tmem + 2 * n % 3 * kTile, q0, k0 + n % 3 * kStep);
            tc::commit(&bars.scores[n & 1]);
          }
          __syncwarp();
          return done;
        };
        const auto dprobs = [&](int n) {
          const bool done = wait(&bars.v_full[n & 1], (n / 2) & 1);
          if (done && leader) {
            products<Op, DP>(tmem + (2 * n + 1) % 3 * kTile, d0, v0 + (n & 1) * kStep);
            tc::commit(&bars.dprobs[n & 1]);
            tc::commit(&bars.v_empty[n & 1]);
          }
          __syncwarp();
          return done;
        };
        bool ok = wait(&bars.qd, 0) && scores(0) && dprobs(0) && (all < 2 || scores(1));
        for (int n = 0; n < all && ok; ++n) {
          if (n + 1 < all) ok = wait(&bars.read[n & 1], (n / 2) & 1) && dprobs(n + 1);
          ok = ok && wait(&bars.dscores[n & 1], (n / 2) & 1);
          if (!ok) break;
          if (leader) {
            // split: two buffers in turn, each added to the rows' own sums two tiles later
            const uint32_t to = tmem + 3 * kTile + (kSplit ? (n & 1) * DP : 0), ds_at = tmem + (2 * n + 1) % 3 * kTile;
            row_sums<Op, DP, kFineScores<T, Op>>(to, ds_at, k0c + n % 3 * kStep, n > 0);
            tc::commit(&bars.k_empty[n % 3]);
          }
          __syncwarp();
          if (n + 2 < all) ok = scores(n + 2);
        }
        if (leader) {
          tc::commit(&bars.done);
          tc::commit(&bars.drain);
        }
        tc::bar_drain(&bars.drain, 0);
      }
      __syncwarp();
    }
  } else {
    tc::take_registers<kRowRegisters>();
    const int w = warp >> 2, i = i0 + (warp & 3) * 32 + lane;
    const uint32_t at_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    float lse = 0.f, delta = 0.f;
    int lim = 0;
    if (i < nq) {
      const int64_t place = (int64_t)head * c.rows + qs.row + i;
      lse = c.lse[place] * kLog2e;
      delta = c.delta[place];
      if (lse == -INFINITY)
        lse = 0.f;
      else
        lim = max(0, seen_keys(c.causal, i, nq, nk));
      if (lim == 1) lim = 0;  // P = 1 whatever the score: dS is zero
    }
    float acc[kSplit ? DP / 2 : 1] = {};  // split: the sums of this warpgroup's half of the columns
    float back = 0.f, back_before = 0.f;  // split: what the last two steps' are multiplied by
    int power = kMostPower;               // else of the row's sums
    // powers of two of this tile and, one step ahead, of the keys and values
    float q_back = 1.f, d_back = 1.f, k_next = 1.f, v_next = 1.f;
    const auto load_powers = [&](int n) {
      k_next = power_back(c.k_power, ks.tile + n, c.key_heads, kh);
      v_next = power_back(c.v_power, ks.tile + n, c.key_heads, kh);
    };
    if (kSplit && all > 0) {
      q_back = power_back(c.q_power, qs.tile + at.tile, c.heads, head);
      d_back = power_back(c.dout_power, qs.tile + at.tile, c.heads, head);
      load_powers(0);
    }
    if (kHalves<T, Op> && all > 0) {
      const int k_at = other_sequence(at.s, c.q_offsets != nullptr, c.k_offsets != nullptr);
      q_back = halves_back(c.q_power, at.s, c.key_heads, kh);
      d_back = halves_back(c.dout_power, at.s, c.key_heads, kh);
      k_next = halves_back(c.k_power, k_at, c.key_heads, kh);
      v_next = halves_back(c.v_power, k_at, c.key_heads, kh);
    }
    const float2 off2 = make_float2(-lse, -lse);
    const float2 delta2 = make_float2(-delta, -delta);
    const uint64_t draw = DROP ? dropout_row(c.draws(), qs.row + i, c.heads, head) : 0;
    bool ok = true;
    for (int n = 0; n < all; ++n) {
      const int b = n & 1, phase = (n / 2) & 1, key0 = n * kTile + w * kHalf;
      ok = __all_sync(0xffffffffu, tc::bar_wait(&bars.scores[b], phase, failed, c.polls));
      if (!ok) break;
      tc::fence_after();
      if constexpr (kSplit)
        if (n > 1)  // of two tiles before
          add_sums<DP / 2>(acc, at_lane + 3 * kTile + b * DP + w * (DP / 2), back_before);
      const float k_back = k_next, cs = c.scale_log2 * q_back * k_back, dprobs = d_back * v_next;
      const float2 cs2 = make_float2(cs, cs);
      if (kSplit && n + 1 < all) load_powers(n + 1);
      const uint32_t s_at = at_lane + 2 * n % 3 * kTile + w * kHalf, dp_at = at_lane + (2 * n + 1) % 3 * kTile + w * kHalf;
      float p[kHalf];
      tc::load32(s_at, p);
      tc::load32(s_at + 32, p + 32);
      tc::wait_loads();
      tc::fence_before();
      tc::bar_arrive_warp(&bars.read[b]);
#pragma unroll
      for (int x = 0; x < kHalf; x += 2) {
        const float2 a = tc::fma2(make_float2(p[x], p[x + 1]), cs2, off2);
        p[x] = tc::exp2_fast(a.x);
        p[x + 1] = tc::exp2_fast(a.y);
      }
      const int left = lim - key0;
      const bool cut = __any_sync(0xffffffffu, left < kHalf);
      ok = __all_sync(0xffffffffu, tc::bar_wait(&bars.dprobs[b], phase, failed, c.polls));
      if (!ok) break;
      tc::fence_after();
      float t[kHalf];
      tc::load32(dp_at, t);
      tc::load32(dp_at + 32, t + 32);
      tc::wait_loads();
      if (DROP) {
#pragma unroll
        for (int x = 0; x < kHalf; x += 4) {
          const uint64_t z = dropout_draw(draw, key0 + x);
#pragma unroll
          for (int y = 0; y < 4; ++y) t[x + y] = draw_lane(z, y) >= c.drop ? t[x + y] * c.keep_scale : 0.f;
        }
      }
#pragma unroll
      for (int x = 0; x < kHalf; x += 2) {
        float2 a = tc::fma2(make_float2(t[x], t[x + 1]), make_float2(dprobs, dprobs), delta2);
        a = tc::mul2(a, make_float2(p[x], p[x + 1]));
        t[x] = a.x;
        t[x + 1] = a.y;
      }
      if (cut)
#pragma unroll
        for (int x = 0; x < kHalf; ++x) t[x] = x < left ? t[x] : 0.f;
      if constexpr (kScaled<Op>) {
        uint32_t exponent;
        ok = row_exponent(bars.tops, t, n, &exponent, failed, c.polls);
        if (!ok) break;
        float up;
        if constexpr (kSplit) {
          const int now = row_power(exponent, 14, 0);
          up = power_of_two(now);
          back_before = back;
          back = power_of_two(-now) * k_back;
        } else {
          const int now = running_power(power, exponent);
          if (n > 0 && __any_sync(0xffffffffu, now != power)) {  // once the sums so far are complete
            ok = __all_sync(0xffffffffu, tc::bar_wait(&bars.k_empty[(n - 1) % 3], ((n - 1) / 3) & 1, failed, c.polls));
            if (!ok) break;
            tc::fence_after();
            multiply_sums<DP / 2>(at_lane + 3 * kTile + w * (DP / 2), exp2f((float)(now - power)));
          }
          power = now;
          up = power_of_two(power);
        }
#pragma unroll
        for (int x = 0; x < kHalf; ++x) t[x] *= up;
      }
      store_row32<Op, kFineScores<T, Op>>(dp_at, 0, t);
      store_row32<Op, kFineScores<T, Op>>(dp_at, 32, t + 32);
      tc::wait_stores();
      tc::fence_before();
      tc::bar_arrive_warp(&bars.dscores[b]);
    }
    if (ok && all > 0) {
      ok = __all_sync(0xffffffffu, tc::bar_wait(&bars.done, 0, failed, c.polls));
      tc::fence_after();
    }
    if (ok) {
      T *row = nullptr;
      const int from = w * (DP / 2);  // a warpgroup stores half of the columns
      if (i < qs.cover)
        row = static_cast<T *>(c.dq.p) +
              (c.q_offsets ? (qs.row + i) * c.dq.token : qs.seq * c.dq.seq + i * c.dq.token) + head * c.dq.head + from;
      if constexpr (kSplit) {
        for (int n = max(0, all - 2); n < all; ++n)
          add_sums<DP / 2>(acc, at_lane + 3 * kTile + (n & 1) * DP + from,
                           n == all - 1 ? back : back_before);
        store_floats<DP / 2>(row, acc, c.scale, c.d - from, lim == 0);
      } else {
        const float factor = (kScaled<Op> ? c.scale * power_of_two(-power) : c.scale) * k_next;
        store_sums<T, DP / 2>(at_lane + 3 * kTile + from, row, factor, c.d - from, all > 0, lim == 0);
      }
    }
    tc::fence_before();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::tmem_free(tmem, 512);
  }
  if (bars.failed) {
    if (warp == kCopyWarp) drain_copies(bars);
    if (warp < kCopyWarp) poison_queries<T>(c);
  }
  // what follows in the stream waits for this kernel only: its last block waits for the keys'
  if (blockIdx.x == gridDim.x - 1) dependency_wait();
}

template <typename T, typename Op, int DP, bool DROP>
cudaError_t backward_launch(const AttnCall &c, const TileMaps &m, cudaStream_t s) {
  constexpr int W = wide<Op, DP>();
  if (c.dk.p || c.dv.p) {
    const auto kern = tile_backward_keys<T, Op, DP, DROP>;
    cudaError_t e = allow_smem(kern, keys_smem<W>());
    if (e != cudaSuccess) return e;
    const int64_t blocks = tiles_of(c.k_offsets != nullptr, c.sequences, c.k_tokens, 1, kTile) * c.key_heads;
    e = launch_kernel(kern, dim3((unsigned)blocks), kTileThreads, keys_smem<W>(), false, s, c, m);
    if (e != cudaSuccess) return e;
  }
  if (!c.dq.p) return cudaSuccess;
  const auto kern = tile_backward_queries<T, Op, DP, DROP>;
  const cudaError_t e = allow_smem(kern, queries_smem<W>());
  if (e != cudaSuccess) return e;
  const int64_t blocks = tiles_of(c.q_offsets != nullptr, c.sequences, c.q_tokens, 1, kTile) * c.heads;
  return launch_kernel(kern, dim3((unsigned)blocks), kTileThreads, queries_smem<W>(), c.dk.p || c.dv.p, s, c, m);
}

template <typename T, typename Op, int DP>
cudaError_t backward_typed(const AttnCall &c, const TileMaps &m, cudaStream_t s) {
  return c.drop ? backward_launch<T, Op, DP, true>(c, m, s) : backward_launch<T, Op, DP, false>(c, m, s);
}

}  // namespace

cudaError_t tile_backward_launch(const AttnCall &c, int type, const SplitParts &parts, cudaStream_t s) {
  using Bf16 = __nv_bfloat16;
  TileMaps m = {};
  if (!maps_of(&m, c, type, parts, true)) return cudaErrorInvalidValue;
  if (type == SNACK_F32) return backward_typed<float, float, 64>(c, m, s);
  if (type == SNACK_F16)
    return c.d > 64 ? backward_typed<__half, __half, 128>(c, m, s) : backward_typed<__half, __half, 64>(c, m, s);
  if (parts.halves) return backward_typed<Bf16, __half, 128>(c, m, s);
  return c.d > 64 ? backward_typed<Bf16, Bf16, 128>(c, m, s) : backward_typed<Bf16, Bf16, 64>(c, m, s);
}

cudaError_t tile_backward_failed(int *flag, cudaStream_t s) { return read_flag(g_attention_failed, flag, s); }

}  // namespace snack

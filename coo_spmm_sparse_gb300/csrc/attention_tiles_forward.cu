// The forward call of the attention on tcgen05.
#include "attention_tiles.cuh"

namespace snack {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kForwardSlots = 4;  // tiles of keys and values in flight, in turn

template <int W>
constexpr size_t tile_forward_smem() { return 1024 + (size_t)(2 + kForwardSlots) * tile_bytes<W>(); }

struct ForwardBars {
  uint64_t q[2], full[kForwardSlots], empty[kForwardSlots], scores[2], probs[2][2], done[2], cut, drain;
  uint32_t tmem;
  int failed, copied, copied_q;  // tiles of keys and values whose copies were started; a bit for each of queries
};

// A block's part of the queries: two tiles of 128 rows.
struct ForwardPlace {
  Place at;
  Span qs;
  int head0, first[2];
};
__device__ __forceinline__ ForwardPlace forward_place(const AttnCall &c) {
  const bool by_heads = c.group % 2 == 0;
  const int units = by_heads ? c.heads / 2 : c.heads, u = blockIdx.x % units, rows = by_heads ? kTile : 2 * kTile;
  ForwardPlace p;
  p.at = find_tile(c.q_offsets, c.sequences, c.q_tokens, 1, rows, blockIdx.x / units, c.causal);
  p.head0 = by_heads ? 2 * u : u;
  if (p.at.s < 0) return p;
  p.qs = own_span(c.q_offsets, c.q_lengths, p.at.s, c.sequences, c.q_tokens);
  p.first[0] = p.at.tile * rows;
  p.first[1] = p.first[0] + (by_heads ? 0 : kTile);
  return p;
}

// The copies of a block whose wait has given up end before it does.
__device__ __forceinline__ void drain_copies(ForwardBars &bars) {
  for (int t = 0; t < 2; ++t)
    if (bars.copied_q >> t & 1) tc::bar_drain(&bars.q[t], 0);
  for (int i = max(0, bars.copied - kForwardSlots); i < bars.copied; ++i)
    tc::bar_drain(&bars.full[i % kForwardSlots], (i / kForwardSlots) & 1);
}
// The flag, and NaN for its results, by the warps that have rows.  (A call of its own,
// and what it needs made again, so that the kernel keeps no registers for it: they
// cost the long prompt 3 %.)
template <typename T>
__device__ __noinline__ void poison_forward(const AttnCall &c) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) g_attention_failed = 1;
  const ForwardPlace p = forward_place(c);
  const int t = warp >> 2, i = p.first[t] + (warp & 3) * 32 + lane, head = p.head0 + (c.group % 2 == 0 ? t : 0);
  if (i >= p.qs.cover) return;
  const int64_t slot = (blockIdx.y * c.rows + p.qs.row + i) * c.heads + head;
  if (c.splits > 1) {
    poison_row(c.part + slot * c.d, c.d);
    poison_row(c.part + (int64_t)c.splits * c.rows * c.heads * c.d + slot, 1);
  } else {
    poison_row(static_cast<T *>(c.out.p) + head * c.out.head +
                   (c.q_offsets ? (p.qs.row + i) * c.out.token : p.qs.seq * c.out.seq + i * c.out.token), c.d);
    poison_row(c.lse + (int64_t)head * c.rows + p.qs.row + i, 1);
  }
}

// Two tiles of 128 query rows share the keys: two heads of a group over the
// same tokens where the group is even, else neighbouring tokens of one head.
// While the rows of one tile are exponentiated, the products of the other run.
//
// The accumulated row is multiplied down only when the maximum has grown by
// more than 2^8 since the last time: until then probabilities are up to 2^8
// fold, which the 32-bit sums hold as well.
template <typename T, int DP, bool DROP>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_forward(const __grid_constant__ AttnCall c, const __grid_constant__ TileMaps maps) {
  constexpr int W = wide<T, DP>();
  constexpr bool kSplit = Operand<T>::kSplit;
  extern __shared__ unsigned char raw[];
  __shared__ ForwardBars bars;
  unsigned char *const sq = align1024(raw), *const ring = sq + 2 * tile_bytes<W>();
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  volatile int *const failed = &bars.failed;

  // barriers, tensor memory and the block's place are made ready side by side
  if (warp == kCopyWarp && lane == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::bar_init(&bars.q[i], 1);
      tc::bar_init(&bars.scores[i], 1);
      tc::bar_init(&bars.probs[i][0], 4);
      tc::bar_init(&bars.probs[i][1], 4);
      tc::bar_init(&bars.done[i], 1);
    }
    for (int i = 0; i < kForwardSlots; ++i) {
      tc::bar_init(&bars.full[i], 1);
      tc::bar_init(&bars.empty[i], 1);
    }
    tc::bar_init(&bars.cut, 1);
    tc::bar_init(&bars.drain, 1);
    bars.failed = 0;
    tc::fence_bar_init();
    tc::prefetch_map(&maps.q);
    tc::prefetch_map(&maps.k);
    tc::prefetch_map(&maps.v);
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(&bars.tmem, 512);
    tc::fence_before();
  }
  const ForwardPlace place = forward_place(c);
  const Place at = place.at;
  if (at.s < 0) return leave_block(warp, &bars.tmem);
  const Span qs = place.qs;
  const bool by_heads = c.group % 2 == 0;
  const Span ks = other_span(c.k_offsets, c.k_lengths, at.s, c.q_offsets != nullptr, c.sequences, c.k_tokens);
  const int nq = qs.valid, nk = ks.valid;
  const int first[2] = {place.first[0], place.first[1]}, head0 = place.head0, kh = head0 / c.group;
  int steps[2];
  const int begin = c.splits > 1 ? (int)blockIdx.y * (c.chunk / kTile) : 0;  // the first tile of keys
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int last = min(first[t] + kTile, nq) - 1;
    int end = first[t] < nq ? (max(0, seen_keys(c.causal, last, nq, nk)) + kTile - 1) / kTile : 0;
    if (c.splits > 1) end = min(end, begin + c.chunk / kTile);
    steps[t] = max(0, end - begin);
  }
  const int all = max(steps[0], steps[1]);

  const int q_token = c.q_offsets ? (int)qs.row : 0, k_token = (c.k_offsets ? (int)ks.row : 0) + begin * kTile;
  if (warp == kCopyWarp && lane == 0 && all > 0) {
    for (int t = 0; t < 2; ++t)
      if (steps[t])
        copy_tile<W>(sq + t * tile_bytes<W>(), &maps.q, &bars.q[t], head0 + (by_heads ? t : 0), q_token + first[t],
                     qs.seq);
    copy_tile<W>(ring, &maps.k, &bars.full[0], kh, k_token, ks.seq);
  }
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = bars.tmem;  // scores of the two tiles, then their sums
  if (warp >= kCopyWarp) {
  tc::leave_registers<kOtherRegisters>();
  if (warp == kCopyWarp) {
    int cut_phase = 0, item = 0;
    bool ok = true;
    for (int j = 0; j < all && ok; ++j) {
      for (int kv = 0; kv < 2 && ok; ++kv, ++item) {
        if (item == 0) continue;  // on its way since the start
        const int slot = item % kForwardSlots;
        if (item >= kForwardSlots)
          ok = __all_sync(0xffffffffu,
                          tc::bar_wait(&bars.empty[slot], (item / kForwardSlots - 1) & 1, failed, c.polls));
        if (!ok) break;
        unsigned char *const to = ring + slot * tile_bytes<W>();
        const int token = k_token + j * kTile;
        const int left = nk - (begin + j) * kTile;
        if (kv && left < kTile)
          ok = copy_tile_cut<W>(to, &maps.v, &bars.full[slot], &bars.cut, &cut_phase, kh, token, ks.seq, left, failed,
                                 c.polls);
        else if (lane == 0)
          copy_tile<W>(to, kv ? &maps.v : &maps.k, &bars.full[slot], kh, token, ks.seq);
        __syncwarp();
      }
    }
    if (lane == 0) {
      bars.copied = item;
      bars.copied_q = (steps[0] > 0) + 2 * (steps[1] > 0);
    }
  } else if (warp == kMmaWarp) {
    // the whole warp goes along, so that descriptors stay in uniform registers
    if (all > 0) {
      const bool leader = tc::elect_one();
      const uint32_t q0 = tc::desc_rows(tc::smem_addr(sq)), k0 = tc::desc_rows(tc::smem_addr(ring));
      const uint32_t v0 = tc::desc_columns(tc::smem_addr(ring), kBlock);
      constexpr uint32_t kStep = tile_bytes<W>() / 16;
      const auto wait = [&](uint64_t *bar, int phase) {
        const bool done = __all_sync(0xffffffffu, tc::bar_wait(bar, phase, failed, c.polls));
        tc::fence_after();
        return done;
      };
      const auto wait_item = [&](int item) {
        return wait(&bars.full[item % kForwardSlots], (item / kForwardSlots) & 1);
      };
      bool ok = wait_item(0);
      for (int t = 0; t < 2 && ok; ++t)
        if (steps[t]) {
          ok = wait(&bars.q[t], 0);
          if (ok && leader) {
            products<T, DP>(tmem + t * kTile, q0 + t * kStep, k0);
            tc::commit(&bars.scores[t]);
          }
        }
      if (leader) tc::commit(&bars.empty[0]);
      for (int j = 0; j < all && ok; ++j) {
        const uint32_t v_at = v0 + (2 * j + 1) % kForwardSlots * kStep, k_at = k0 + (2 * j + 2) % kForwardSlots * kStep;
        ok = wait_item(2 * j + 1) && (j + 1 >= all || wait_item(2 * j + 2));
        for (int t = 0; t < 2 && ok; ++t) {
          if (j >= steps[t]) continue;
          const uint32_t s_at = tmem + t * kTile, o_at = tmem + 2 * kTile + t * DP;
          ok = wait(&bars.probs[t][0], j & 1);
          if (ok && leader) sums<T, DP, kTile / 2>(o_at, s_at, v_at, j > 0);
          ok = ok && wait(&bars.probs[t][1], j & 1);
          if (ok && leader) {
            sums<T, DP, kTile / 2>(o_at, s_at, v_at, true, kTile / 2);
            if (j + 1 < steps[t]) {
              products<T, DP>(s_at, q0 + t * kStep, k_at);
              tc::commit(&bars.scores[t]);
            } else {
              tc::commit(&bars.done[t]);
            }
          }
          __syncwarp();
        }
        if (leader) {
          tc::commit(&bars.empty[(2 * j + 1) % kForwardSlots]);
          if (j + 1 < all) tc::commit(&bars.empty[(2 * j + 2) % kForwardSlots]);
        }
        __syncwarp();
      }
      if (leader) tc::commit(&bars.drain);
      tc::bar_drain(&bars.drain, 0);
    }
    __syncwarp();
  }
  } else {
    tc::take_registers<kRowRegisters>();
    const int t = warp >> 2, head = head0 + (by_heads ? t : 0);
    const int i = first[t] + (warp & 3) * 32 + lane;  // token of this thread's row
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + t * kTile, o_at = tmem + lanes + 2 * kTile + t * DP;
    // keys that the row sees from the block's first on; a block with a part of the keys leaves a part
    const int lim = i < nq ? max(0, seen_keys(c.causal, i, nq, nk) - begin * kTile) : 0;
    const int64_t slot = (blockIdx.y * c.rows + qs.row + i) * c.heads + head;
    float *const part_lse = c.part + (int64_t)c.splits * c.rows * c.heads * c.d + slot;
    uint64_t draw = 0;
    if (DROP) draw = dropout_row(c.draws(), qs.row + i, c.heads, head);
    float m = -INFINITY, sum = 0.f;
    bool ok = true;
    if constexpr (kSplit) {
      // Two passes over the scores in tensor memory, 64 at a time: a row's sums
      // stay in registers beside them.
      float o[DP] = {};
      // powers of two of this tile of queries, of the keys' (one tile ahead) and of the values before
      const float q_back = steps[t] ? power_back(c.q_power, qs.tile + first[t] / kTile, c.heads, head) : 0.f;
      float k_back = 0.f, v_back = 0.f, v_before = 0.f;
      const auto load_powers = [&](int j) {
        k_back = power_back(c.k_power, ks.tile + begin + j, c.key_heads, kh);
        v_back = power_back(c.v_power, ks.tile + begin + j, c.key_heads, kh);
      };
      if (steps[t]) load_powers(0);
      for (int j = 0; j < steps[t]; ++j) {
        ok = __all_sync(0xffffffffu, tc::bar_wait(&bars.scores[t], j & 1, failed, c.polls));
        if (!ok) break;
        tc::fence_after();
        if (j > 0) add_sums<DP>(o, o_at, v_before);  // of the tile before: complete when these scores are
        const float cs = fmaxf(c.scale_log2 * q_back * k_back, 1e-37f);
        v_before = v_back;
        if (j + 1 < steps[t]) load_powers(j + 1);
        const int left = lim - j * kTile;  // keys of this tile that the row sees
        const bool cut = __any_sync(0xffffffffu, left < kTile);
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < kTile; x += 64) {
          float s[64];
          tc::load32(s_at + x, s);
          tc::load32(s_at + x + 32, s + 32);
          tc::wait_loads();
          if (cut)
#pragma unroll
            for (int e = 0; e < 64; ++e) s[e] = x + e < left ? s[e] : -INFINITY;
#pragma unroll
          for (int e = 0; e < 64; e += 8)
#pragma unroll
            for (int y = 0; y < 4; ++y) top[y] = tc::max3(top[y], s[e + y], s[e + 4 + y]);
        }
        const float grown = fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * cs);
        const float shrink = grown == -INFINITY ? 1.f : tc::exp2_fast(m - grown);
        m = grown;
        sum *= shrink;
        if (__any_sync(0xffffffffu, shrink != 1.f))
#pragma unroll
          for (int e = 0; e < DP; ++e) o[e] *= shrink;
        const float off = m == -INFINITY ? kHalfP : kHalfP - m;
        float part[4] = {};
#pragma unroll
        for (int x = 0; x < kTile; x += 64) {
          float s[64];
          tc::load32(s_at + x, s);
          tc::load32(s_at + x + 32, s + 32);
          tc::wait_loads();
#pragma unroll
          for (int e = 0; e < 64; ++e) s[e] = tc::exp2_fast(fmaf(s[e], cs, off));
          if (cut)
#pragma unroll
            for (int e = 0; e < 64; ++e) s[e] = x + e < left ? s[e] : 0.f;
#pragma unroll
          for (int e = 0; e < 64; ++e) part[e & 3] += s[e];
          if (DROP)
#pragma unroll
            for (int e = 0; e < 64; e += 4) {
              const uint64_t z = dropout_draw(draw, (begin + j) * kTile + x + e);
#pragma unroll
              for (int y = 0; y < 4; ++y) s[e + y] = draw_lane(z, y) >= c.drop ? s[e + y] : 0.f;
            }
          store_parts<__half>(s_at + x, s);
          store_parts<__half>(s_at + x + 32, s + 32);
          tc::wait_stores();
          tc::fence_before();
          tc::bar_arrive_warp(&bars.probs[t][x / 64]);
        }
        sum += (part[0] + part[1]) + (part[2] + part[3]);
      }
      if (ok && steps[t]) {
        ok = __all_sync(0xffffffffu, tc::bar_wait(&bars.done[t], 0, failed, c.polls));
        tc::fence_after();
        if (ok) add_sums<DP>(o, o_at, v_before);
      }
      if (ok && i < qs.cover) {
        float *const row = c.splits > 1 ? c.part + slot * c.d
                                        : static_cast<float *>(c.out.p) + head * c.out.head +
                                              (c.q_offsets ? (qs.row + i) * c.out.token
                                                           : qs.seq * c.out.seq + i * c.out.token);
        store_floats<DP>(row, o, c.keep_scale / sum, c.d, sum == 0.f);
        *(c.splits > 1 ? part_lse : c.lse + (int64_t)head * c.rows + qs.row + i) =
            sum == 0.f ? -INFINITY : m * kLn2 + (logf(sum) - kHalfP * kLn2);
      }
    } else {
    const float cs = c.scale_log2;
    for (int j = 0; j < steps[t]; ++j) {
      ok = __all_sync(0xffffffffu, tc::bar_wait(&bars.scores[t], j & 1, failed, c.polls));
      if (!ok) break;
      tc::fence_after();
      float s[kTile];
#pragma unroll
      for (int x = 0; x < kTile; x += 32) tc::load32(s_at + x, s + x);
      tc::wait_loads();
      const int left = lim - j * kTile;  // keys of this tile that the row sees
      if (__any_sync(0xffffffffu, left < kTile)) {
#pragma unroll
        for (int x = 0; x < kTile; ++x) s[x] = x < left ? s[x] : -INFINITY;
      }
      float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int x = 4; x < kTile - 4; x += 8)
#pragma unroll
        for (int y = 0; y < 4; ++y) top[y] = tc::max3(top[y], s[x + y], s[x + 4 + y]);
#pragma unroll
      for (int y = 0; y < 4; ++y) top[y] = fmaxf(top[y], s[kTile - 4 + y]);
      const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
      const float grown = fmaxf(m, most);
      const bool up = j == 0 || (grown - m) * cs > 8.f;
      if (j > 0 && __any_sync(0xffffffffu, up)) {
        const float shrink = up ? tc::exp2_fast((m - grown) * cs) : 1.f;
        sum *= shrink;
#pragma unroll
        for (int x = 0; x < DP; x += 32) {
          float o[32];
          tc::load32(o_at + x, o);
          tc::wait_loads();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= shrink;
          tc::store32(o_at + x, reinterpret_cast<const uint32_t *>(o));
        }
      }
      if (up) m = grown;
      const float off = m == -INFINITY ? 0.f : -m * cs;
      const float2 cs2 = make_float2(cs, cs), off2 = make_float2(off, off);
      float2 part[2] = {};
#pragma unroll
      for (int x = 0; x < kTile; x += 64) {
        uint32_t p[32];
#pragma unroll
        for (int e = 0; e < 64; e += 2) {
          float2 a = tc::fma2(make_float2(s[x + e], s[x + e + 1]), cs2, off2);
          a.x = tc::exp2_fast(a.x);
          a.y = tc::exp2_fast(a.y);
          part[e / 2 & 1] = tc::add2(part[e / 2 & 1], a);
          if (DROP) {
            s[x + e] = a.x;
            s[x + e + 1] = a.y;
          } else {
            p[e / 2] = pack2<T>(a.x, a.y);
          }
        }
        if (DROP) {
#pragma unroll
          for (int e = 0; e < 64; e += 4) {
            const uint64_t z = dropout_draw(draw, (begin + j) * kTile + x + e);
            float k[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) k[y] = draw_lane(z, y) >= c.drop ? s[x + e + y] : 0.f;
            p[e / 2] = pack2<T>(k[0], k[1]);
            p[e / 2 + 1] = pack2<T>(k[2], k[3]);
          }
        }
        tc::store32(s_at + x, p);
        tc::wait_stores();
        tc::fence_before();
        tc::bar_arrive_warp(&bars.probs[t][x / 64]);
      }
      sum += (part[0].x + part[0].y) + (part[1].x + part[1].y);
    }
    if (ok && steps[t]) {
      ok = __all_sync(0xffffffffu, tc::bar_wait(&bars.done[t], 0, failed, c.polls));
      tc::fence_after();
    }
    if (ok) {
      const bool mine = i < qs.cover;
      const float factor = c.keep_scale / sum;
      if (c.splits > 1) {
#pragma unroll
        for (int x = 0; x < DP; x += 32) {
          float v[32];
          if (steps[t] > 0) {
            tc::load32(o_at + x, v);
            tc::wait_loads();
          }
          store_floats<32>(mine ? c.part + slot * c.d + x : nullptr, v, factor, c.d - x, sum == 0.f);
          __syncwarp();
        }
      } else {
        T *row = nullptr;
        if (mine)
          row = static_cast<T *>(c.out.p) +
                (c.q_offsets ? (qs.row + i) * c.out.token : qs.seq * c.out.seq + i * c.out.token) + head * c.out.head;
        store_sums<T, DP>(o_at, row, factor, c.d, steps[t] > 0, sum == 0.f);
      }
      if (mine)
        *(c.splits > 1 ? part_lse : c.lse + (int64_t)head * c.rows + qs.row + i) =
            sum == 0.f ? -INFINITY : m * cs * kLn2 + logf(sum);
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
    if (warp < kCopyWarp) poison_forward<T>(c);
  }
}

}  // namespace

bool tiles_take(const AttnCall &c, int type) {
  return (type != SNACK_F32 || c.d <= 64) && c.scale > 0.f && c.k_tokens > 0 && c.q_tokens > 0 && c.sequences > 0;
}

bool tiles_read(const AttnCall &c) {
  const int64_t qn = c.q_offsets ? 1 : c.sequences, kn = c.k_offsets ? 1 : c.sequences;
  return c.d % 8 == 0 && even(c.q, c.heads, c.q_tokens, qn) && even(c.k, c.key_heads, c.k_tokens, kn) &&
         even(c.v, c.key_heads, c.k_tokens, kn) && (!c.dout.p || even(c.dout, c.heads, c.q_tokens, qn));
}

int64_t tile_forward_blocks(const AttnCall &c) {
  const bool by_heads = c.group % 2 == 0;
  return tiles_of(c.q_offsets != nullptr, c.sequences, c.q_tokens, 1, by_heads ? kTile : 2 * kTile) *
         (by_heads ? c.heads / 2 : c.heads);
}

template <typename T, int DP, bool DROP>
static cudaError_t forward_launch(const AttnCall &c, const TileMaps &m, cudaStream_t s) {
  const auto kern = tile_forward<T, DP, DROP>;
  constexpr size_t smem = tile_forward_smem<wide<T, DP>()>();
  const cudaError_t e = allow_smem(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3((unsigned)tile_forward_blocks(c), (unsigned)c.splits), kTileThreads, smem, false, s, c, m);
}

template <typename T>
static cudaError_t forward_typed(const AttnCall &c, const TileMaps &m, cudaStream_t s) {
  if constexpr (!Operand<T>::kSplit)
    if (c.d > 64)
      return c.drop ? forward_launch<T, 128, true>(c, m, s) : forward_launch<T, 128, false>(c, m, s);
  return c.drop ? forward_launch<T, 64, true>(c, m, s) : forward_launch<T, 64, false>(c, m, s);
}

cudaError_t tile_forward_launch(const AttnCall &c, int type, const SplitParts &parts, cudaStream_t s) {
  TileMaps m = {};
  if (!maps_of(&m, c, type, parts, false)) return cudaErrorInvalidValue;
  return type == SNACK_F32    ? forward_typed<float>(c, m, s)
         : type == SNACK_BF16 ? forward_typed<__nv_bfloat16>(c, m, s)
                              : forward_typed<__half>(c, m, s);
}

cudaError_t tile_forward_failed(int *flag, cudaStream_t s) { return read_flag(g_attention_failed, flag, s); }

}  // namespace snack

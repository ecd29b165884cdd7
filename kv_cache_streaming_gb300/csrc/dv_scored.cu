// dv_scored_attention: causal attention that also adds up, for each cache row and key head,
// the weight that the new tokens gave it,
//   mass[b][h][j] += sum_i sum_g w_{i,g,j},  w_{i,g,j} = exp2(c s_{i,g,j} - lse_{i,g}).
//
// A weight is known only once its row's softmax is complete, so the sums are a second pass.
// The attention kernel (dv_attention.cuh, form kScored) leaves lse = log2 sum_j exp2(c s_j) of
// each (token, query head); then
//   few rows (a decode step): it has left the scores too, 4 bytes each, and few_kernel reads
//     them back: 8 bytes a row of the cache beside the 4 D of K and V;
//   else mass_kernel computes S^T = K Q^T again on the tensor cores, with the keys as rows, so
//     that a thread that owns a key sums along its row of tensor memory and nothing is reduced
//     across threads.
//
// mass_kernel: a unit of work is 256 cache rows of a (sequence, key head), two tiles of keys,
// against the counted (token, head of the group) rows that attend some of them, in tiles of
// 128: with one tile of keys, fetching the queries again for each bound it by L2.  The units
// form one line, each as long as its tiles and unit cost, cut into equal stretches, one a CTA
// (one CTA an SM); a unit that a cut divides leaves partial sums, which mass_join_kernel adds in
// order (no atomics: the same bits each time).  Warps 0-7 and 8-15 sum the unit's two tiles of
// keys, two to a quarter of the rows with half of the columns each; 16 loads (and walks over the
// units), 17 issues the products into two buffers of tensor memory for each tile, 18 fetches lse.
//
// A group that does not divide 128 leaves columns of each tile without a token, which takes the
// masked sums for its last 32 columns: 8 prompts of 64 to 1536 tokens at groups of 4, 5, 6, 7, 8
// give 430, 422, 416, 413, 440 TFLOP/s attended.  (Two spilled registers of mass_kernel are stored and
// loaded a few times a unit, not in the loop over its tiles.)
//
// Every wait gives up after a number of tries, as in the attention kernel.
//
// Measured (bf16, heads of 128): a decode step of 32 sequences of 64 to 1791 rows, 112 heads, 300
// us, of which few_kernel takes 14 to 16 (6.3 TB/s); two contexts of 115000, 64 query heads on 8, 160
// us (few_kernel 19); 32 prompts of 64 to 1536 tokens, 112 heads, 1387 us in a short loop: attention
// 925, its join 13, mass_kernel 447, its join 3; under the power cap of a long one 1477: 988, 14, 471,
// 3.  mass_kernel takes about 1000 cycles a tile of 128 x 128, where its products and its
// exponentials take 512 each.  It is bound by the instructions around them (2400 a tile for 1170 of loads, sums and
// exponentials), with the tensor cores 47% and the special functions 42% active.  On the way:
// units of 128 keys 582 us (560 without products, 404 without exponentials: L2, which then fetched
// the queries twice as often), of 256 552, hidden columns skipped 501, sixteen warps 464, one wait
// and one arrival a tile 448.
#include <algorithm>

#include "dv_attention.cuh"

namespace dv {

cudaError_t scored_waits(void** address) { return waits_address(address); }

namespace {

// Rows (new tokens x heads of a group) up to which the scores are kept: beyond, writing and
// reading them costs more than K again.  Two contexts of 115000, 64 query heads on 8, with 1, 2, 4, 8
// tokens: 169, 188, 230, 321 us kept, 218 to 220 computed again; 16 sequences of 64 to 1791 rows, 56
// heads, with 16, 32, 64 tokens: 87, 109, 158 and 102, 106, 118.
constexpr int kFewRows = 16;
constexpr int kFewThreads = kJoinThreads, kFewPer = 4;
// Blocks of the sums, an SM, up to which they also join what the cuts divided.  One launch less
// (8 short sequences, 25 heads of 64: 17.4 us, 20.3 with two), but every block of a divided
// unit goes through its pieces' statistics (two contexts of 115000, 8 key heads: 165 us, 160 with
// two launches; 32 sequences, 112 heads: 309 and 304).
constexpr int kFewWave = 8;
constexpr int kUnit = 2 * kTile;  // rows of a unit of mass_kernel
constexpr int kSumWarps = 16;
constexpr int kMassThreads = 32 * (kSumWarps + 3);
// What a unit costs besides its tiles (its keys' fetch, the sums' exchange), in tiles of keys: 32
// ragged prompts, 112 heads, 490, 464, 473 us at 1, 2, 3 (and one wait a tile more than now).
constexpr int kMassUnitCost = 2;

struct MassDivided {
  int64_t at;    // of the unit's first row in mass
  int32_t rows;  // of the unit (0: none here)
  int32_t last;  // the last CTA with a piece
};

template <int MAXB>
struct MassParams {
  CUtensorMap q_map;  // as in AttnBase
  CUtensorMap k_map;
  const uint4* k;
  const float* lse;  // [H][T][G]
  float* mass;       // [B][H][S]
  float* part;       // two slots of kUnit sums a CTA: of the piece it goes on with, and begins
  MassDivided* divided;
  int32_t share, extra;
  int32_t H, G, C, S;
  int32_t k_rows, tile_tok;
  int32_t tokens, last;  // T; the counted tokens of a sequence (0: all)
  uint32_t tries;
  float c;
  SeqTable<MAXB> seq;
  int32_t cost_pre[MAXB + 1];
};

// The counted tokens of a sequence of n new ones: [first, n).
__host__ __device__ __forceinline__ int first_counted(int n, int last) {
  return last > 0 && n > last ? n - last : 0;
}
// The first counted token that attends some of the rows from `row` on.
__host__ __device__ __forceinline__ int first_token(int start, int n, int last, int row) {
  const int c0 = first_counted(n, last);
  return row - start > c0 ? row - start : c0;
}

struct MassItem {
  int b, h, row0;   // the unit's rows [row0, row0 + kUnit)
  int row_end;      // of the sequence
  int tok0, n;      // the piece's first token; its tiles of tokens (0: no more items)
  int whole, first;  // the piece is the whole unit; is the unit's first
  int start, n_tok, tok_at;
};

template <int DP>
struct MassSmem {
  static constexpr int kSlot = kTile * DP * 2;
  static constexpr int kK = 4, kQ = DP == 128 ? 3 : 6;  // tiles of K and Q held
  static constexpr int kS = 2, kL = 3;  // sums of each tile of keys, lse
  static constexpr int kQAt = kK * kSlot;
  static constexpr int kCtl = kQAt + kQ * kSlot;
  struct Ctl {
    float lse[kL][kTile];  // negative
    float sum[kUnit];      // of the second half of the columns
    uint64_t k_full[kK], k_empty[kK], q_full[kQ], q_empty[kQ];
    uint64_t s_full[2][kS], s_empty[2][kS], lse_full[kL];
    uint64_t sum_full, sum_empty, item_full[kItems], item_empty[kItems], drained;
    MassItem item[kItems];
    uint32_t tmem;
  };
  static constexpr int kBytes = kCtl + (int)sizeof(Ctl);
  static_assert(kBytes <= 232448, "more shared memory than a CTA has");
};

template <typename P>
struct MassWalk {
  const P& p;
  int pos, end;     // as in Walk
  int b, h, kt, t;  // the next piece: its unit and first tile of tokens

  __device__ int tokens() const { return p.seq.pre[b + 1] - p.seq.pre[b]; }
  __device__ int tiles(int first) const {  // of tokens, from `first` on
    return (tokens() - first + p.tile_tok - 1) / p.tile_tok;
  }
  __device__ int token0() const {
    return first_token(p.seq.start[b], tokens(), p.last, kt * kUnit);
  }
  // Tiles of keys of the unit, what each of its tiles of tokens costs.
  __device__ int keys() const {
    return p.seq.start[b] + tokens() - kt * kUnit > kTile ? 2 : 1;
  }
  // The unit's tiles of tokens before place x of the line (whichever CTA asks).
  __device__ int before(int x, int cnt) const {
    const int w = keys();
    return max(0, min(cnt, (x - pos - kMassUnitCost + w - 1) / w));
  }
  __device__ void next_unit(int cnt) {
    pos += kMassUnitCost + cnt * keys();
    t = 0;
    if (++kt * kUnit >= p.seq.start[b] + tokens()) {
      kt = 0;
      if (++h == p.H) {
        h = 0;
        if (pos < end) do ++b; while (p.seq.pre[b + 1] == p.seq.pre[b]);
      }
    }
  }

  __device__ MassWalk(const P& p_, int lo, int hi) : p(p_), pos(lo), end(hi) {
    b = h = kt = t = 0;
    if (lo >= hi) return;
    int x = 0, y = p.seq.batch;
#pragma unroll 1
    while (y - x > 1) {
      const int m = (x + y) >> 1;
      if (p.cost_pre[m] <= lo) x = m; else y = m;
    }
    b = x;
    int rem = lo - p.cost_pre[b];
    const int head = (p.cost_pre[b + 1] - p.cost_pre[b]) / p.H;
    h = rem / head;
    rem -= h * head;
    // the rows that every counted token attends, but for the last unit of them: of one cost
    const int c0 = first_counted(tokens(), p.last);
    const int flat = (p.seq.start[b] + c0) / kUnit, cost0 = kMassUnitCost + 2 * tiles(c0);
    kt = min(rem / cost0, flat);
    rem -= kt * cost0;
    int cnt = tiles(token0());
    if (kt == flat)
#pragma unroll 1
      while (rem >= kMassUnitCost + cnt * keys()) {
        rem -= kMassUnitCost + cnt * keys();
        ++kt;
        cnt = tiles(token0());
      }
    pos = lo - rem;
    t = before(lo, cnt);
    if (t == cnt) next_unit(cnt);  // (the stretch starts inside its last tile, which is not its own)
  }

  __device__ void next(MassItem* it) {
    it->n = 0;
    if (pos >= end) return;
    const int first = token0(), cnt = tiles(first);
    const int n = before(end, cnt) - t;
    if (n <= 0) return;
    it->b = b;
    it->h = h;
    it->row0 = kt * kUnit;
    it->row_end = p.seq.start[b] + tokens();
    it->tok0 = first + t * p.tile_tok;
    it->n = n;
    it->whole = n == cnt;
    it->first = t == 0;
    it->start = p.seq.start[b];
    it->n_tok = tokens();
    it->tok_at = p.seq.pre[b];
    next_unit(cnt);
  }
};

// The item's first tile of tokens of which some attend the unit's second tile of keys.
template <typename P>
__device__ __forceinline__ int second_from(const P& p, const MassItem& it) {
  // tile j's last token is tok0 + (j + 1) tile_tok - 1, at most n_tok - 1
  const int hidden = it.row0 + kTile - it.start - it.tok0;  // tokens before the first that does
  return max(0, min(hidden / p.tile_tok, it.n - 1));
}

// (a, b) = (a, b) * c + (d, e)
__device__ __forceinline__ void fma2(float& a, float& b, float c, float d, float e) {
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %2};\n"
      " mov.b64 z, {%3, %4};\n fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}"
      : "+f"(a), "+f"(b)
      : "f"(c), "f"(d), "f"(e));
}

template <typename T, int DP, int MAXB>
__global__ __launch_bounds__(kMassThreads, 1) void mass_kernel(
    const __grid_constant__ MassParams<MAXB> p) {
  using SM = MassSmem<DP>;
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t base = smem_u32(sm);
  if ((base & 1023) != 0) {  // the swizzle goes by address bits
    ops_pdl_enter();
    if (threadIdx.x == 0) {
      gave_up();
      if (blockIdx.x > 0) p.divided[blockIdx.x - 1] = MassDivided{};
    }
    return;
  }
  typename SM::Ctl& ctl = *reinterpret_cast<typename SM::Ctl*>(sm + SM::kCtl);
  const int warp = __shfl_sync(~0u, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const auto at = [&](const uint64_t& bar) {
    return base + (uint32_t)(reinterpret_cast<const uint8_t*>(&bar) - sm);
  };
  if (warp == kSumWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     base + (uint32_t)(reinterpret_cast<uint8_t*>(&ctl.tmem) - sm)),
                 "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < SM::kK; ++i) {
      bar_init(at(ctl.k_full[i]), 1);
      bar_init(at(ctl.k_empty[i]), 1);
    }
    for (int i = 0; i < SM::kQ; ++i) {
      bar_init(at(ctl.q_full[i]), 1);
      bar_init(at(ctl.q_empty[i]), 1);
    }
    for (int i = 0; i < 2 * SM::kS; ++i) {
      bar_init(at(ctl.s_full[i / SM::kS][i % SM::kS]), 2);  // the products, and who issued them
      bar_init(at(ctl.s_empty[i / SM::kS][i % SM::kS]), kSumWarps / 2);
    }
    for (int i = 0; i < SM::kL; ++i) bar_init(at(ctl.lse_full[i]), 1);
    for (int i = 0; i < kItems; ++i) {
      bar_init(at(ctl.item_full[i]), 1);
      bar_init(at(ctl.item_empty[i]), kSumWarps + 2);
    }
    bar_init(at(ctl.sum_full), kUnit);
    bar_init(at(ctl.sum_empty), kUnit);
    bar_init(at(ctl.drained), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(~0u, ctl.tmem, 0);
  ops_pdl_enter();

  const int used = p.tile_tok * p.G;  // rows of a tile of Q that hold a token
  const auto wait = [&](uint32_t bar, uint32_t parity) { return bar_wait(bar, parity, p.tries); };
  const auto get_item = [&](uint32_t k, MassItem* it) {
    if (!wait(at(ctl.item_full[k % kItems]), k / kItems & 1)) return false;
    *it = ctl.item[k % kItems];
    return __all_sync(~0u, it->n > 0) != 0;
  };
  const auto done_item = [&](uint32_t k) {
    __syncwarp();
    if (lane == 0) bar_arrive(at(ctl.item_empty[k % kItems]));
  };

  if (warp == kSumWarps) {
    // ---- the walk, and loads ----
    const bool on = elect();
    MassWalk<MassParams<MAXB>> walk(p, cut(p, blockIdx.x), cut(p, blockIdx.x + 1));
    if (blockIdx.x > 0 && on) {
      MassDivided d = {};
      if (walk.t > 0 && cut(p, blockIdx.x - 1) <= walk.pos + kMassUnitCost) {
        const int row0 = walk.kt * kUnit, cnt = walk.tiles(walk.token0());
        const int row_end = p.seq.start[walk.b] + walk.tokens();
        d.at = ((int64_t)walk.b * p.H + walk.h) * p.S + row0;
        d.rows = min(kUnit, row_end - row0);
        d.last = blockIdx.x;
#pragma unroll 1
        while (walk.before(cut(p, d.last + 1), cnt) < cnt) ++d.last;
      }
      p.divided[blockIdx.x - 1] = d;
    }
    Ring<SM::kK> kr;
    Ring<SM::kQ> qr;
    uint32_t nk = 0, nq = 0, n_items = 0;
    bool ok = true;
    while (ok) {
      MassItem it;
      walk.next(&it);
      if (n_items >= kItems)
        ok = wait(at(ctl.item_empty[n_items % kItems]), (n_items / kItems - 1) & 1);
      if (!ok) break;
      if (on) {
        ctl.item[n_items % kItems] = it;
        bar_arrive(at(ctl.item_full[n_items % kItems]));
      }
      ++n_items;
      if (it.n == 0) break;
#pragma unroll 1
      for (int row0 = it.row0; row0 < min(it.row0 + kUnit, it.row_end); row0 += kTile) {
        if (nk >= SM::kK && !(ok = wait(at(ctl.k_empty[kr.slot]), kr.turn ^ 1))) break;
        const uint32_t bar = at(ctl.k_full[kr.slot]), dst = base + kr.slot * SM::kSlot;
        const int head = it.b * p.H + it.h, rows = min(kTile, it.row_end - row0);
        const int pad = p.C & 1;  // zeros for the other half of the last contraction step
        bar_expect(bar, p.C * rows * 16 + pad * (kTile * 16), on);
        if (rows == kTile) {
          tma_load4(dst, &p.k_map, 0, row0 / p.k_rows, 0, head, bar, on);
        } else {
          const uint4* src = p.k + (int64_t)head * p.C * p.S + row0;
#pragma unroll 1
          for (int c = 0; c < p.C; ++c)
            bulk_load(dst + c * (kTile * 16), src + (int64_t)c * p.S, rows * 16, bar, on);
        }
        if (pad) bulk_load(dst + p.C * (kTile * 16), g_zero_rows, kTile * 16, bar, on);
        kr.next();
        ++nk;
      }
      if (!ok) break;
#pragma unroll 1
      for (int j = 0; j < it.n; ++j) {
        if (nq >= SM::kQ && !(ok = wait(at(ctl.q_empty[qr.slot]), qr.turn ^ 1))) break;
        const uint32_t bar = at(ctl.q_full[qr.slot]);
        bar_expect(bar, (DP / 64) * 128 * used, on);
        for (int half = 0; half < DP / 64; ++half)
          tma_load4(base + SM::kQAt + qr.slot * SM::kSlot + half * (kTile * 128), &p.q_map,
                    half * 64, 0, it.h, it.tok_at + it.tok0 + j * p.tile_tok, bar, on);
        qr.next();
        ++nq;
      }
    }
    // No copy is left in flight, whichever warp gave up.
#pragma unroll 1
    for (uint32_t i = 0; i < SM::kK && i < nk; ++i)  // a slot's last use
      bar_wait(at(ctl.k_full[i]), (nk - i - 1) / SM::kK & 1, kSpinLimit);
#pragma unroll 1
    for (uint32_t i = 0; i < SM::kQ && i < nq; ++i)
      bar_wait(at(ctl.q_full[i]), (nq - i - 1) / SM::kQ & 1, kSpinLimit);
    __syncwarp();
  } else if (warp == kSumWarps + 1) {
    // ---- products: S^T = K Q^T ----
    const bool on = elect();
    constexpr uint32_t kType = std::is_same<T, __half>::value ? 0u : 1u;
    constexpr uint32_t kIdesc = 1u << 4 | kType << 7 | kType << 10 | (uint32_t)(kTile >> 3) << 17 |
                                (uint32_t)(kTile >> 4) << 24;
    const int steps = (p.C + 1) / 2;
    Ring<SM::kK> kr;
    Ring<SM::kQ> qr;
    Ring<SM::kS> sr;
    Ring<SM::kL> lr;
    uint32_t n_items = 0;
    bool ok = true;
    MassItem it;
    while (ok && get_item(n_items, &it)) {
      const int n = __shfl_sync(~0u, it.n, 0), row0 = __shfl_sync(~0u, it.row0, 0);
      const int keys = __shfl_sync(~0u, it.row_end, 0) - row0 > kTile ? 2 : 1;
      // the first tile of tokens that attends the second tile of keys
      const int second = keys < 2 ? n : second_from(p, it);
      Ring<SM::kK> kt[2] = {kr, kr};
      kt[1].next();
      for (int i = 0; i < keys; ++i) kr.next();
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        if (!(ok = wait(at(ctl.q_full[qr.slot]), qr.turn))) break;
        // (lse is written once the sums that were in the buffers have been read)
        if (!(ok = wait(at(ctl.lse_full[lr.slot]), lr.turn))) break;
        const uint64_t qd = smem_desc(base + SM::kQAt + qr.slot * SM::kSlot, 0, 1024, 2);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i == 0 || j >= second) {
            if (j == (i ? second : 0) && !(ok = wait(at(ctl.k_full[kt[i].slot]), kt[i].turn))) break;
            fence_after();
            const uint64_t kd = smem_desc(base + kt[i].slot * SM::kSlot, kTile * 16, 128, 0);
#pragma unroll
            for (int s = 0; s < DP / 16; ++s)
              mma_ss(tmem + (i * SM::kS + sr.slot) * kTile, kd + s * (2 * kTile),
                     qd + (s >> 2) * (kTile * 8) + (s & 3) * 2, kIdesc, s > 0, on && s < steps);
          }
          mma_commit(at(ctl.s_full[i][sr.slot]), on);
          if (on) bar_arrive(at(ctl.s_full[i][sr.slot]));
        }
        if (!ok) break;
        mma_commit(at(ctl.q_empty[qr.slot]), on);
        qr.next();
        sr.next();
        lr.next();
      }
      for (int i = 0; i < keys; ++i) mma_commit(at(ctl.k_empty[kt[i].slot]), on);
      done_item(n_items++);
    }
    // the products in flight end before tensor memory is given back
    mma_commit(at(ctl.drained), on);
    bar_wait(at(ctl.drained), 0, kSpinLimit);
    __syncwarp();
  } else if (warp == kSumWarps + 2) {
    // ---- lse of each tile's rows ----
    Ring<SM::kL> lr;
    Ring<SM::kS> sr;
    uint32_t n_items = 0, nl = 0;
    bool ok = true;
    MassItem it;
    while (ok && get_item(n_items, &it)) {
#pragma unroll 1
      for (int j = 0; j < it.n; ++j) {
        const int tok = it.tok0 + j * p.tile_tok, cols = min(p.tile_tok, it.n_tok - tok) * p.G;
        const float* const src = p.lse + ((int64_t)it.h * p.tokens + it.tok_at + tok) * p.G;
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[e] = lane + 32 * e < cols ? -src[lane + 32 * e] : -INFINITY;
        // Once the sums of the tile before the last have been read, a warp is through with the
        // tile before that one, whose place this is.
        if (nl >= SM::kS)
          if (!(ok = wait(at(ctl.s_empty[0][sr.slot]), sr.turn ^ 1) &&
                     wait(at(ctl.s_empty[1][sr.slot]), sr.turn ^ 1))) break;
#pragma unroll
        for (int e = 0; e < 4; ++e) ctl.lse[lr.slot][lane + 32 * e] = x[e];
        __syncwarp();
        if (lane == 0) bar_arrive(at(ctl.lse_full[lr.slot]));
        lr.next();
        sr.next();
        ++nl;
      }
      done_item(n_items++);
    }
  } else {
    // ---- sums: a key per thread, half of the columns ----
    const int set = warp >> 3, half = warp >> 2 & 1, r = set * kTile + (threadIdx.x & (kTile - 1));
    const uint32_t ts =
        tmem + ((uint32_t)(warp & 3) << 21) + set * SM::kS * kTile + half * (kTile / 2);
    Ring<SM::kS> sr;
    Ring<SM::kL> lr;
    uint32_t item = 0;
    bool ok = true;
    MassItem it;
    for (; ok && get_item(item, &it); ++item) {
      const int row = it.row0 + r;
      float* const mass = p.mass + ((int64_t)it.b * p.H + it.h) * p.S + row;
      const float old = half == 0 && row < it.row_end && it.whole ? *mass : 0.f;
      const int from = set == 0 ? 0 : it.row_end - it.row0 > kTile ? second_from(p, it) : it.n;
      float total = 0.f;
#pragma unroll 1
      for (int j = 0, tok = it.tok0; j < it.n; ++j, tok += p.tile_tok, sr.next(), lr.next()) {
        if (!(ok = wait(at(ctl.s_full[set][sr.slot]), sr.turn))) break;
        fence_after();
        const auto read = [&]() {  // the tile's scores: its buffer is free
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(at(ctl.s_empty[set][sr.slot]));
        };
        if (j < from) {
          read();
          continue;
        }
        const uint32_t s0 = ts + sr.slot * kTile;
        const float* const nl = ctl.lse[lr.slot] + half * (kTile / 2);
        const int cols = min(p.tile_tok, it.n_tok - tok) * p.G;
        const int lead = it.row0 + set * kTile - it.start - tok;  // (the first key's own token)
        float sum[4] = {};
        uint32_t x[2][32];
        tmem_ld32(x[0], s0);
        tmem_wait_ld();
        tmem_ld32(x[1], s0 + 32);  // under the first exponentials
        const auto add = [&](int i) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 n4 = *reinterpret_cast<const float4*>(nl + 32 * i + e);
            float a = __uint_as_float(x[i][e]), b = __uint_as_float(x[i][e + 1]);
            float c = __uint_as_float(x[i][e + 2]), d = __uint_as_float(x[i][e + 3]);
            fma2(a, b, p.c, n4.x, n4.y);
            fma2(c, d, p.c, n4.z, n4.w);
            add2(sum[0], sum[1], ex2(a), ex2(b));
            add2(sum[2], sum[3], ex2(c), ex2(d));
          }
        };
        if (cols == kTile && lead <= 1 - kTile) {  // every key's token comes before the tile
          add(0);
          tmem_wait_ld();
          read();
          add(1);
        } else {
          tmem_wait_ld();
          read();
          // columns [lo, hi): tokens from the key's own row on, up to the last (what is past
          // them may hold anything)
          const int lo = max(0, lead + (threadIdx.x & (kTile - 1))) * p.G - half * (kTile / 2);
          const int hi = cols - half * (kTile / 2);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (__all_sync(~0u, lo <= 32 * i && hi >= 32 * i + 32)) {
              add(i);
            } else if (__any_sync(~0u, lo < 32 * i + 32 && hi > 32 * i)) {
#pragma unroll
              for (int e = 32 * i; e < 32 * i + 32; ++e) {
                const float w = ex2(fmaf(__uint_as_float(x[i][e - 32 * i]), p.c, nl[e]));
                if (e >= lo && e < hi) sum[e & 3] += w;
              }
            }
          }
        }
        total += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      }
      if (!ok) break;
      if (half == 1) {
        if (item > 0 && !(ok = wait(at(ctl.sum_empty), (item - 1) & 1))) break;
        ctl.sum[r] = total;
        bar_arrive(at(ctl.sum_full));
      } else {
        if (!(ok = wait(at(ctl.sum_full), item & 1))) break;
        total += ctl.sum[r];
        bar_arrive(at(ctl.sum_empty));
        if (!it.whole)
          p.part[(int64_t)(blockIdx.x * 2 + (it.first ? 1 : 0)) * kUnit + r] = total;
        else if (row < it.row_end)
          *mass = old + total;
      }
      done_item(item);
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kSumWarps)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
}

// Adds the pieces of the unit that the cut after CTA blockIdx.x is the first to divide.
__global__ __launch_bounds__(kUnit) void mass_join_kernel(const MassDivided* divided,
                                                          const float* part, float* mass) {
  ops_pdl_enter();
  const MassDivided d = divided[blockIdx.x];
  const int r = threadIdx.x, i0 = blockIdx.x;
  if (r >= d.rows) return;
  float total = part[(int64_t)(2 * i0 + 1) * kUnit + r];
  for (int i = i0 + 1; i <= d.last; ++i) total += part[(int64_t)(2 * i) * kUnit + r];
  mass[d.at + r] += total;
}

// ---- few rows: from the scores that the attention kernel kept ----------------------

template <int MAXB>
struct FewParams {
  JoinParams join;
  const float* scores;
  float* mass;
  int32_t H, S, last, chunks;
  int32_t join_ctas, join_blocks;  // blocks that join pieces of outputs: a unit's, of each cut
  int32_t share, extra, unit_cost, heads;  // of the attention kernel's schedule
  float c;
  SeqTable<MAXB> seq;
  int32_t block_pre[MAXB + 1];
  int32_t cost_pre[MAXB + 1];
};

// The CTA whose stretch holds place x of the line.
template <typename P>
__device__ __forceinline__ int owner(const P& p, int x) {
  const int longer = p.extra * (p.share + 1);
  return x < longer ? x / (p.share + 1) : p.extra + (x - longer) / p.share;
}

// -lse of row r of a unit that the cuts may have divided: from the attention kernel, or from
// its pieces' statistics.
template <typename T, typename P>
__device__ __forceinline__ float row_lse(const P& p, int b, int h, int r) {
  const int n = p.seq.pre[b + 1] - p.seq.pre[b], G = p.join.G;
  const int tiles = (p.seq.start[b] + n + kTile - 1) / kTile;
  const int pos = p.cost_pre[b] + (p.heads ? h >> 1 : h) * (p.unit_cost + tiles);
  const int row = p.heads ? (h & 1) * kHeadRows + r : r;
  const int i0 = owner(p, pos + p.unit_cost), i1 = owner(p, pos + p.unit_cost + tiles - 1);
  if (i0 == i1) return -p.join.lse[((int64_t)h * p.join.tokens + p.seq.pre[b]) * G + r];
  const int64_t slot = (int64_t)p.join.rows * (p.join.D + 2);
  const int first = cut(p, i0) < pos ? 1 : 0;
  float m = -INFINITY, l = 0.f;
#pragma unroll 1
  for (int i = i0; i <= i1; i += 4) {
    float2 ml[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      ml[k] = i + k <= i1
                  ? reinterpret_cast<const float2*>(
                        p.join.part + slot * (2 * (i + k) + (i + k == i0 ? first : 0)) +
                        (int64_t)p.join.rows * p.join.D)[row]
                  : make_float2(-INFINITY, 0.f);
    const float m_new =
        fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), m);
    l *= m == -INFINITY ? 0.f : ex2(m - m_new);
    m = m_new;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k <= i1)  // (a piece of NaN scores alone has m = -inf and l = NaN)
        l += (ml[k].x == -INFINITY ? 0.f : ex2(ml[k].x - m)) * ml[k].y;
  }
  return (std::is_same<T, __half>::value ? kHalfUp : 0.f) - (m + log2f(l));
}

// Blocks that join the pieces of divided outputs (where that is left to them), then those that sum: kFewPer cache rows a
// thread, kFewThreads apart, whose loads are in flight together; a block for each (sequence,
// key head, kFewThreads * kFewPer rows).
// JOIN: it joins; else lse is complete.
template <typename T, int MAXB, bool JOIN>
__global__ __launch_bounds__(kFewThreads) void few_kernel(
    const __grid_constant__ FewParams<MAXB> p) {
  __shared__ float nlse[kFewRows];
  ops_pdl_enter();
  const int joins = JOIN ? p.join_ctas * p.join_blocks : 0;
  if (JOIN && (int)blockIdx.x < joins) {
    const int i0 = blockIdx.x / p.join_blocks;
    join<T, kPlain>(p.join, i0, blockIdx.x - i0 * p.join_blocks, p.join_blocks);
    return;
  }
  const int id = blockIdx.x - joins, bh = id / p.chunks, chunk = id - bh * p.chunks;
  const int b = bh / p.H, h = bh - b * p.H;
  const int start = p.seq.start[b], n = p.seq.pre[b + 1] - p.seq.pre[b], G = p.join.G;
  const int row_end = start + n;
  if (n == 0 || chunk * (kFewThreads * kFewPer) >= row_end) return;  // (the whole block)
  const int row0 = chunk * (kFewThreads * kFewPer) + threadIdx.x;
  const int64_t pitch = (int64_t)((row_end + kTile - 1) / kTile) * kTile;
  const float* s = p.scores + kTile * (int64_t)p.block_pre[b] * (p.H * G) +
                   (int64_t)h * G * n * pitch + row0;
  float* const mass = p.mass + ((int64_t)b * p.H + h) * p.S + row0;
  const int c0 = first_counted(n, p.last);
  float old[kFewPer], sum[kFewPer] = {};
#pragma unroll
  for (int e = 0; e < kFewPer; ++e)
    old[e] = row0 + e * kFewThreads < row_end ? mass[e * kFewThreads] : 0.f;
  const float* const lse = p.join.lse + ((int64_t)h * p.join.tokens + p.seq.pre[b]) * G;
  if constexpr (JOIN) {
    if ((int)threadIdx.x < n * G) nlse[threadIdx.x] = row_lse<T>(p, b, h, threadIdx.x);
    __syncthreads();
  }
  for (int g = 0; g < G; ++g) {
#pragma unroll 2
    for (int i = c0; i < n; ++i) {
      const float* const x = s + (int64_t)(g * n + i) * pitch;
      const float nl = JOIN ? nlse[i * G + g] : -lse[i * G + g];
      const int end = start + i + 1;  // of the rows that the token attends
#pragma unroll
      for (int e = 0; e < kFewPer; ++e)
        if (row0 + e * kFewThreads < end) sum[e] += ex2(fmaf(x[e * kFewThreads], p.c, nl));
    }
  }
#pragma unroll
  for (int e = 0; e < kFewPer; ++e)
    if (row0 + e * kFewThreads < row_end) mass[e * kFewThreads] = old[e] + sum[e];
}

// ---- host ----------------------------------------------------------------------------

size_t up32(size_t n) { return (n + 31) / 32 * 32; }

// Whether the attention kernel keeps the scores: it runs one row tile a unit, of few rows.
bool keeps_scores(const Plan& p, int group) {
  return p.max_len <= kTile / group && p.max_len * group <= kFewRows &&
         score_blocks(p, nullptr) <= INT32_MAX;
}

// The workspace behind the attention's own: lse, then the scores or the mass kernel's pieces.
size_t lse_bytes(const Plan& p, int group) {
  return up32((size_t)p.tokens * p.H * group * sizeof(float));
}
size_t scored_bytes(const Plan& p, int group) {
  const size_t rest =
      keeps_scores(p, group)
          ? (size_t)score_blocks(p, nullptr) * p.H * group * kTile * sizeof(float)
          : (size_t)sm_count() * (2 * kUnit * sizeof(float) + sizeof(MassDivided));
  return 32 + lse_bytes(p, group) + rest;
}

// Cost of the mass kernel's units, before each sequence in `pre`; in *tiles their tiles.
int64_t mass_cost(const Plan& p, int tile_tok, int32_t last, int32_t* pre, int64_t* tiles) {
  int64_t total = 0;
  *tiles = 0;
  for (int b = 0; b < p.B; ++b) {
    if (pre) pre[b] = (int32_t)total;
    const int n = p.seq_len[b], start = p.seq_start[b];
    if (n == 0) continue;
    const auto count = [&](int first) { return (n - first + tile_tok - 1) / tile_tok; };
    // (the rows that all counted tokens attend, but for the last unit of them: of one cost)
    const int c0 = first_counted(n, last);
    int64_t units = (start + c0) / kUnit, t = units * 2 * count(c0);
    for (int64_t row = units * kUnit; row < (int64_t)start + n; row += kUnit, ++units)
      t += count(first_token(start, n, last, (int)row)) * ((int64_t)start + n - row > kTile ? 2 : 1);
    *tiles += t * p.H;
    total += (t + units * kMassUnitCost) * p.H;
  }
  if (pre) pre[p.B] = (int32_t)total;
  return total;
}

// Blocks of rows of a (sequence, key head) in few_kernel.
int64_t few_chunks(const Plan& p) {
  int64_t rows = 0;
  for (int b = 0; b < p.B; ++b)
    if (p.seq_len[b] > 0) rows = std::max<int64_t>(rows, (int64_t)p.seq_start[b] + p.seq_len[b]);
  return (rows + kFewThreads * kFewPer - 1) / (kFewThreads * kFewPer);
}

template <typename T, int DP, int MAXB>
cudaError_t launch_mass(const MassParams<MAXB>& kp, int ctas, cudaStream_t stream) {
  void (*const kernel)(MassParams<MAXB>) = mass_kernel<T, DP, MAXB>;
  constexpr int kBytes = MassSmem<DP>::kBytes;
  const cudaError_t err =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (err != cudaSuccess) return err;
  return ops_launch(kernel, dim3((unsigned)ctas), kMassThreads, kBytes, stream, kp);
}

template <typename T, int MAXB>
dv_status add_mass(const Plan& p, const dv_queries& q, const Extra& x, int32_t last, uint8_t* ws,
                   uint8_t* rest, cudaStream_t stream) {
  const int group = q.q_heads / p.H;
  if (x.scores) {
    FewParams<MAXB> fp;
    const Schedule sch = schedule<kScored>(p, group, x, fp.cost_pre);
    fp.join = join_params(p, q, sch, x, reinterpret_cast<const float*>(ws));
    fp.join_ctas = x.join_later ? sch.ctas - 1 : 0;
    fp.join_blocks = (int32_t)join_blocks(p, q, sch);
    fp.share = (int32_t)(sch.total / sch.ctas);
    fp.extra = (int32_t)(sch.total % sch.ctas);
    fp.unit_cost = sch.unit_cost;
    fp.heads = sch.heads ? 1 : 0;
    fp.scores = x.scores;
    fp.mass = x.mass;
    fp.H = p.H;
    fp.S = p.S;
    fp.last = last;
    fp.c = q.scale * 1.4426950408889634f;
    fill_table(p, &fp.seq);
    score_blocks(p, fp.block_pre);
    fp.chunks = (int32_t)few_chunks(p);
    const unsigned blocks = (unsigned)(fp.join_ctas * fp.join_blocks + fp.chunks * p.H * p.B);
    const cudaError_t err =
        x.join_later
            ? ops_launch(few_kernel<T, MAXB, true>, dim3(blocks), kFewThreads, 0, stream, fp)
            : ops_launch(few_kernel<T, MAXB, false>, dim3(blocks), kFewThreads, 0, stream, fp);
    return err == cudaSuccess ? DV_OK : cuda_fail(err, "scored attention's sums launch");
  }
  MassParams<MAXB> kp;
  kp.tile_tok = kTile / group;
  int64_t tiles = 0;
  const int64_t total = mass_cost(p, kp.tile_tok, last, kp.cost_pre, &tiles);
  int64_t ctas = sm_count();
  if (ctas > tiles / 2) ctas = std::max<int64_t>(1, tiles / 2);  // (two tiles of keys a CTA at least)
  const void* k = static_cast<const uint4*>(p.k) + p.l0 * p.layer_chunks;
  if (!encode_q(&kp.q_map, p, q, group, kp.tile_tok) ||
      !encode_k(&kp.k_map, p, q.dtype == DV_DTYPE_FP16, k))
    return fail(DV_ERR_CUDA, "cuTensorMapEncodeTiled refused the queries or the cache");
  kp.k = static_cast<const uint4*>(k);
  kp.lse = x.lse;
  kp.mass = x.mass;
  kp.part = reinterpret_cast<float*>(rest);
  kp.divided = reinterpret_cast<MassDivided*>(rest + (size_t)ctas * 2 * kUnit * sizeof(float));
  kp.share = (int32_t)(total / ctas);
  kp.extra = (int32_t)(total % ctas);
  kp.H = p.H;
  kp.G = group;
  kp.C = p.C;
  kp.S = p.S;
  kp.k_rows = k_run(p);
  kp.tokens = (int32_t)p.tokens;
  kp.last = last;
  kp.tries = attention_tries();
  kp.c = q.scale * 1.4426950408889634f;
  fill_table(p, &kp.seq);
  cudaError_t err = p.D <= 64 ? launch_mass<T, 64, MAXB>(kp, (int)ctas, stream)
                              : launch_mass<T, 128, MAXB>(kp, (int)ctas, stream);
  if (err == cudaSuccess && ctas > 1)
    err = ops_launch(mass_join_kernel, dim3((unsigned)ctas - 1), kUnit, 0, stream,
                     static_cast<const MassDivided*>(kp.divided),
                     static_cast<const float*>(kp.part), kp.mass);
  return err == cudaSuccess ? DV_OK : cuda_fail(err, "scored attention's sums launch");
}

}  // namespace
}  // namespace dv

extern "C" dv_status dv_scored_attention_workspace(const dv_cache* cache, const int32_t* seq_start,
                                                   const int32_t* seq_end, int32_t q_heads,
                                                   size_t* bytes) {
  if (!bytes) return dv::fail(DV_ERR_INVALID_ARG, "bytes is NULL");
  dv::Plan p;
  dv_status st = dv::plan_ranges(cache, 0, 1, seq_start, seq_end, &p);
  if (st != DV_OK) return st;
  if ((st = dv::check_heads(cache, p, q_heads)) != DV_OK) return st;
  const int group = q_heads / p.H;
  *bytes = p.tokens == 0 ? 0
                         : dv::schedule<dv::kScored>(p, group, {}, nullptr).bytes +
                               dv::scored_bytes(p, group);
  return DV_OK;
}

extern "C" dv_status dv_scored_attention(const dv_cache* cache, int32_t layer,
                                         const int32_t* seq_start, const int32_t* seq_end,
                                         const dv_queries* queries, int32_t last, float* mass,
                                         void* workspace, size_t workspace_bytes,
                                         dv_stream stream) {
  dv::Trace trace("dv_scored_attention");
  if (last < 0) return dv::fail(DV_ERR_INVALID_ARG, "the last %d tokens", last);
  dv_status st = dv::check_max_seq(cache);
  if (st != DV_OK) return st;
  dv::Plan p;
  dv_queries q;
  dv::Extra x;
  x.mass = mass;
  uint8_t* ws = nullptr;
  st = dv::check_call<dv::kScored>(cache, layer, seq_start, seq_end, queries, &x, workspace,
                                   workspace_bytes, dv::scored_bytes, &p, &q, &ws);
  if (st != DV_OK || p.tokens == 0) return st;
  const int group = q.q_heads / p.H;
  uint8_t* const lse = ws + dv::up32(dv::schedule<dv::kScored>(p, group, x, nullptr).bytes);
  uint8_t* const rest = lse + dv::lse_bytes(p, group);
  x.lse = reinterpret_cast<float*>(lse);
  int64_t tiles = 0, work = 0;
  if (dv::keeps_scores(p, group)) {
    x.scores = reinterpret_cast<float*>(rest);
    work = dv::few_chunks(p) * p.H * p.B;
    x.join_later = work <= dv::kFewWave * (int64_t)dv::sm_count();
  } else {
    work = dv::mass_cost(p, dv::kTile / group, last, nullptr, &tiles);
  }
  if (work > INT32_MAX)
    return dv::fail(DV_ERR_UNSUPPORTED, "%lld tiles of weights in one call", (long long)work);
  if ((st = dv::run_call<dv::kScored>(p, q, x, ws, stream)) != DV_OK) return st;
  const bool small = p.B <= dv::kSmallBatch;
  if (q.dtype == DV_DTYPE_FP16)
    return small ? dv::add_mass<__half, dv::kSmallBatch>(p, q, x, last, ws, rest, stream)
                 : dv::add_mass<__half, dv::kMaxBatch>(p, q, x, last, ws, rest, stream);
  return small ? dv::add_mass<__nv_bfloat16, dv::kSmallBatch>(p, q, x, last, ws, rest, stream)
               : dv::add_mass<__nv_bfloat16, dv::kMaxBatch>(p, q, x, last, ws, rest, stream);
}

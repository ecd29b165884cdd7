// dv_prompt_attention and dv_tree_attention: attention of new tokens over the
// cache on the tensor cores (tcgen05).
//
// A unit of work is 128 query rows, (token, head of the group) pairs that share
// a key head, against the sequence's cache rows in tiles of 128.  For a tile
// the kernel keeps S = Q K^T, 128 x 128 sums in tensor memory; a warpgroup
// takes a row per thread through the running maximum and sum of the softmax,
//   m' = max(m, max_j s_j),  p_j = exp2(c (s_j - m')),  l' = l f + sum p,
//   O' = O f + P V,          f = exp2(c (m - m')),      c = scale log2(e),
// writes P (rounded to the 16-bit type, the tensor core's operand) over S in
// tensor memory, from where O += P V reads it as the left operand.  O stays
// in tensor memory over all tiles.  f is applied lazily: as long as no row of
// a warp grows by more than 2^8 the old maximum stays the reference (p up to
// 256; P keeps its relative precision, l is summed in 32 bits).
//
// Two chains of such tiles run at once, one's softmax under the other's
// products:
//   PAIR   two row tiles (256 rows) over the same K/V tiles: prompts.
//   SPLIT  one row tile, the even K/V tiles on one chain and the odd ones on
//          the other, joined at the end: decode steps and small trees, bound
//          by reading K and V once.
//
// Warps: 0-3 and 4-7 the chains' softmax, 8 loads, 9 issues the products.  K
// goes to shared memory chunk row by chunk row (bulk copies): the cache's
// [D/8][S][8] is, per tile, exactly the tensor core's unswizzled layout of
// 8 x 16-byte core matrices, so nothing is transposed.  V goes in by TMA with
// the 128-byte swizzle and is read with its rows as the contraction.  Only rows
// up to the last attended one are fetched (V in 32s).
//
// The tiles of all units form one line, cut into equal stretches, one for
// each CTA (one CTA an SM); a unit that a cut divides leaves partial sums in
// the workspace, which join_kernel adds up.
//
// Rows a mask hides must have no effect, but 0 x NaN is NaN in a product: in
// tiles that hold hidden rows, V's non-finite values are set to zero in shared
// memory (rows past the last attended one altogether), and should there have been any, the
// epilogue adds them to the outputs of the rows that do attend them.
//
// Every wait gives up after kSpinLimit tries: the CTA then drains its copies,
// frees its tensor memory and returns, and dv_attention_check reports it.
#include <cuda.h>

#include "dv_ops.h"

namespace dv {
namespace {

constexpr int kTile = 128;        // rows of Q and of K/V in a tile
constexpr int kThreadsAttn = 320;  // two softmax warpgroups, a load and a product warp
constexpr uint32_t kSpinLimit = 1u << 22;
constexpr float kLazy = 8.f;       // log2 of the growth that is left to the old maximum

// Set when a wait in an attention kernel gave up.
__device__ unsigned int g_attention_timeout;
// The second half of the last contraction step when head_dim is an odd number of chunks.
__device__ uint4 g_zero_rows[kTile];

template <int MAXB>
struct AttnParams {
  CUtensorMap q_map;  // {D, G, H, T}, 64 x G x 1 x tokens of a tile
  CUtensorMap v_map;  // {D, S, B * H}, 64 x 32 x 1
  uint16_t* out;
  const uint4* k;
  const uint16_t* v;
  const uint64_t* tree;
  float* part;
  int64_t out_stride;
  int64_t total;  // tiles of all units
  int32_t H, G, D, C, S;
  int32_t tile_tok;  // tokens of a row tile: 128 / G
  int32_t unit_tok;  // tokens of a unit
  int32_t is_tree;
  float c;  // scale * log2(e)
  SeqTable<MAXB> seq;
  int64_t tile_pre[MAXB + 1];
};

// ---- instructions --------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __noinline__ bool bar_wait_long(uint32_t bar, uint32_t parity, volatile int* abort) {
  for (uint32_t i = 0; i < kSpinLimit; ++i) {
    if (bar_try(bar, parity)) return true;
    if ((i & 31) == 31 && *abort) return false;
  }
  *abort = 1;
  atomicExch(&g_attention_timeout, 1u);
  return false;
}
// Waits for the phase of `parity` to complete; false when it gave up.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (bar_try(bar, parity)) return true;
  return bar_wait_long(bar, parity, abort);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst), "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load4(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                          int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(w),
      "r"(bar)
      : "memory");
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b),
      "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d), "r"(a), "l"(b),
      "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
// Arrives on `bar` once every product issued so far has finished.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

#define DV_R8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), \
                    "=r"(a[i + 5]), "=r"(a[i + 6]), "=r"(a[i + 7])
#define DV_W8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), \
                    "r"(a[i + 5]), "r"(a[i + 6]), "r"(a[i + 7])

// 32 columns of the thread's row of tensor memory.
__device__ __forceinline__ void tmem_ld32(uint32_t* a, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : DV_R8(a, 0), DV_R8(a, 8), DV_R8(a, 16), DV_R8(a, 24)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* a) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      DV_W8(a, 0), DV_W8(a, 8), DV_W8(a, 16), DV_W8(a, 24)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Shared-memory operand descriptors: address, the two byte strides in 16s, the
// fixed bit 46, and the swizzle (2: 128 bytes, 0: none).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride,
                                              uint64_t swizzle) {
  return (uint64_t)((addr >> 4) & 0x3fff) | (uint64_t)((lead >> 4) & 0x3fff) << 16 |
         (uint64_t)((stride >> 4) & 0x3fff) << 32 | (uint64_t)1 << 46 | swizzle << 61;
}

// ---- shared memory -------------------------------------------------------------

template <int DP>
struct Smem {
  static constexpr int kQ = kTile * DP * 2;     // bytes of a row tile
  static constexpr int kSlot = kTile * DP * 2;  // bytes of a K or V tile
  static constexpr int kSlots = DP == 128 ? 5 : 10;
  static constexpr int kKv = 2 * kQ;
  static constexpr int kCtl = kKv + kSlots * kSlot;
  struct Ctl {
    uint64_t q_full[2], q_empty[2];
    uint64_t kv_full[kSlots], kv_empty[kSlots];
    uint64_t s_full[2], p_ready[2], o_done[2];
    uint64_t item_done[2], xchg, drained;
    float2 ml[2][kTile];  // SPLIT: the chains' maxima and sums
    int bad[2];           // the last item of this parity with non-finite values taken out of V
    volatile int abort;
    uint32_t tmem;
  };
  static constexpr int kBytes = kCtl + (int)sizeof(Ctl);
  static_assert(kBytes <= 232448, "more shared memory than a CTA has");
};

// ---- the walk over units ---------------------------------------------------------

struct Item {
  int b, h;
  int tok0;         // the unit's first token in its sequence
  int row_end;      // rows [0, row_end) are attended by some row of the unit
  int t0, t1, cnt;  // tiles of this piece; of the whole unit
};

// K/V tiles of the unit of tokens [tok0, tok0 + unit_tok) of sequence b.
template <typename P>
__device__ __forceinline__ int unit_rows(const P& p, int b, int tok0) {
  const int n = p.seq.pre[b + 1] - p.seq.pre[b];
  return p.seq.start[b] + (p.is_tree ? n : min(tok0 + p.unit_tok, n));
}

template <typename P>
struct Walk {
  const P& p;
  int64_t pos, end;
  int b, h, tok0, t;  // the next piece: its unit and first tile
  bool first;

  __device__ Walk(const P& p_, int64_t lo, int64_t hi) : p(p_), pos(lo), end(hi), first(true) {
    b = h = tok0 = t = 0;
    if (lo >= hi) return;
    int x = 0, y = p.seq.batch;
    while (y - x > 1) {
      const int m = (x + y) >> 1;
      if (p.tile_pre[m] <= lo) x = m; else y = m;
    }
    b = x;
    int64_t rem = lo - p.tile_pre[b];
    const int64_t head = (p.tile_pre[b + 1] - p.tile_pre[b]) / p.H;
    h = (int)(rem / head);
    rem -= h * head;
    for (;;) {
      const int cnt = (unit_rows(p, b, tok0) + kTile - 1) / kTile;
      if (rem < cnt) break;
      rem -= cnt;
      tok0 += p.unit_tok;
    }
    t = (int)rem;
  }

  __device__ bool next(Item* it) {
    if (pos >= end) return false;
    if (!first) {
      tok0 += p.unit_tok;
      if (tok0 >= p.seq.pre[b + 1] - p.seq.pre[b]) {
        tok0 = 0;
        if (++h == p.H) {
          h = 0;
          do ++b; while (p.seq.pre[b + 1] == p.seq.pre[b]);
        }
      }
      t = 0;
    }
    first = false;
    it->b = b;
    it->h = h;
    it->tok0 = tok0;
    it->row_end = unit_rows(p, b, tok0);
    it->cnt = (it->row_end + kTile - 1) / kTile;
    it->t0 = t;
    it->t1 = (int)min((int64_t)it->cnt, t + (end - pos));
    pos += it->t1 - it->t0;
    return true;
  }
};

template <typename P>
__device__ __forceinline__ int64_t cut(const P& p, int i, int n) {
  return p.total / n * i + min((int64_t)i, p.total % n);
}

// The tiles of chain i in a piece: how many, and which is the j-th.
template <bool PAIR, typename P>
__device__ __forceinline__ int chain_tiles(const P& p, const Item& it, int i) {
  if (!PAIR) return (it.t1 - it.t0 + 1 - i) / 2;
  const int n = p.seq.pre[it.b + 1] - p.seq.pre[it.b];
  const int tok = it.tok0 + i * p.tile_tok;
  if (tok >= n) return 0;
  if (p.is_tree) return it.t1 - it.t0;
  const int rows = p.seq.start[it.b] + min(tok + p.tile_tok, n);
  return max(0, min(it.t1, (rows + kTile - 1) / kTile) - it.t0);
}
// The place of the j-th K and V tile in the order of loads: PAIR K0 V0 K1 V1 ...,
// SPLIT K0 K1 V0 K2 V1 K3 ... (the order in which the products take them).
template <bool PAIR>
__device__ __forceinline__ uint32_t k_place(int j) {
  return PAIR ? 2 * j : j == 0 ? 0 : 2 * j - 1;
}
template <bool PAIR>
__device__ __forceinline__ uint32_t v_place(int j, int n) {
  return PAIR ? 2 * j + 1 : j + min(j + 2, n);
}

// ---- the kernel ------------------------------------------------------------------

// Two 64-column masks of the row's attended columns of the tile at row col0.
// Bit c of `bits`: new row c; rows before `start` are always attended.
__device__ __forceinline__ uint64_t tree_mask(uint64_t bits, int rel) {  // rel: column 0 - start
  if (rel <= -64) return ~0ull;
  if (rel < 0) return bits << -rel | ((1ull << -rel) - 1);
  return rel < 64 ? bits >> rel : 0ull;
}
__device__ __forceinline__ uint64_t causal_mask(int last) {  // the last attended column
  return last >= 63 ? ~0ull : last < 0 ? 0ull : (2ull << last) - 1;
}

template <typename T>
__device__ __forceinline__ constexpr uint32_t exp_mask() {
  return sizeof(T) == 2 && std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
}

template <typename T, int DP, bool PAIR, int MAXB>
__global__ __launch_bounds__(kThreadsAttn, 1) void attention_kernel(
    const __grid_constant__ AttnParams<MAXB> p) {
  using SM = Smem<DP>;
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t base = smem_u32(sm);
  if ((base & 1023) != 0) {  // the swizzle goes by address bits
    g_attention_timeout = 1;
    return;
  }
  typename SM::Ctl& ctl = *reinterpret_cast<typename SM::Ctl*>(sm + SM::kCtl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const auto q_full = [&](int i) { return smem_u32(&ctl.q_full[i]); };
  const auto q_empty = [&](int i) { return smem_u32(&ctl.q_empty[i]); };
  const auto kv_full = [&](uint32_t n) { return smem_u32(&ctl.kv_full[n % SM::kSlots]); };
  const auto kv_empty = [&](uint32_t n) { return smem_u32(&ctl.kv_empty[n % SM::kSlots]); };
  const auto kv_addr = [&](uint32_t n) { return base + SM::kKv + (n % SM::kSlots) * SM::kSlot; };
  const auto kv_parity = [&](uint32_t n) { return (n / SM::kSlots) & 1u; };
  volatile int* const abort = &ctl.abort;

  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&ctl.tmem)),
                 "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(q_full(i), 1);
      bar_init(q_empty(i), 1);
      bar_init(smem_u32(&ctl.s_full[i]), 1);
      bar_init(smem_u32(&ctl.p_ready[i]), kTile);
      bar_init(smem_u32(&ctl.o_done[i]), 1);
      bar_init(smem_u32(&ctl.item_done[i]), 2 * kTile);
      ctl.bad[i] = -1;
    }
    for (int i = 0; i < SM::kSlots; ++i) {
      bar_init(kv_full(i), 1);
      bar_init(kv_empty(i), 1);
    }
    bar_init(smem_u32(&ctl.xchg), 2 * kTile);
    bar_init(smem_u32(&ctl.drained), 1);
    ctl.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = ctl.tmem;
  Walk<AttnParams<MAXB>> walk(p, cut(p, blockIdx.x, gridDim.x), cut(p, blockIdx.x + 1, gridDim.x));
  Item it;
  ops_pdl_enter();

  if (warp == 8) {
    // ---- loads ----
    uint32_t n_loads = 0, n_q = 0, base_n = 0;
    uint32_t q_used[2] = {0, 0};
    bool ok = true;
    while (ok && walk.next(&it)) {
      const int n = it.t1 - it.t0;
      const int64_t head = (int64_t)it.b * p.H + it.h;
      for (int i = 0; i < (PAIR ? 2 : 1) && ok; ++i) {
        if (PAIR && chain_tiles<PAIR>(p, it, i) == 0) continue;
        const int qb = PAIR ? i : (int)(n_q & 1);
        if (q_used[qb] > 0) ok = bar_wait(q_empty(qb), (q_used[qb] - 1) & 1, abort);
        if (!ok) break;
        ++q_used[qb];
        ++n_q;
        if (lane == 0) bar_expect(q_full(qb), (DP / 64) * 128 * p.G * p.tile_tok);
        __syncwarp();
        if (lane < DP / 64)
          tma_load4(base + qb * SM::kQ + lane * (kTile * 128), &p.q_map, lane * 64, 0, it.h,
                    p.seq.pre[it.b] + it.tok0 + i * p.tile_tok, q_full(qb));
      }
      for (int m = 0; m < 2 * n && ok; ++m) {
        // the m-th load of the piece: K or V of which tile
        int j;
        bool is_k;
        if (PAIR) {
          j = m >> 1;
          is_k = (m & 1) == 0;
        } else {
          is_k = m == 0 || (m & 1) != 0;
          j = m == 0 ? 0 : is_k ? (m + 1) / 2 : m / 2 - 1;
          if (m >= 2 && is_k && j >= n) {  // past the last K: the last V tile
            is_k = false;
            j = n - 1;
          }
          if (n == 1 && m == 1) {
            is_k = false;
            j = 0;
          }
        }
        const uint32_t ld = base_n + m, bar = kv_full(ld), dst = kv_addr(ld);
        if (ld >= SM::kSlots) ok = bar_wait(kv_empty(ld), kv_parity(ld) ^ 1, abort);
        if (!ok) break;
        n_loads = ld + 1;
        const int row = (it.t0 + j) * kTile, rows = min(kTile, it.row_end - row);
        if (is_k) {
          const int chunks = p.C + (p.C & 1);
          if (lane == 0) bar_expect(bar, p.C * rows * 16 + (p.C & 1) * (kTile * 16));
          __syncwarp();
          if (lane < p.C)
            bulk_load(dst + lane * (kTile * 16), p.k + (head * p.C + lane) * p.S + row, rows * 16,
                      bar);
          else if (lane < chunks)
            bulk_load(dst + lane * (kTile * 16), g_zero_rows, kTile * 16, bar);
        } else {
          const int boxes = (rows + 31) / 32;
          if (lane == 0) bar_expect(bar, boxes * (DP / 64) * 4096);
          __syncwarp();
          const int half = lane & (DP / 64 - 1), box = lane / (DP / 64);
          if (box < boxes)
            tma_load3(dst + half * (kTile * 128) + box * 4096, &p.v_map, half * 64, row + box * 32,
                      (int)head, bar);
        }
      }
      base_n += 2 * n;
    }
    // A CTA that gave up leaves no copy in flight.
    if (!ok) {
      int never = 0;
      for (uint32_t ld = n_loads > SM::kSlots ? n_loads - SM::kSlots : 0; ld < n_loads; ++ld)
        bar_wait(kv_full(ld), kv_parity(ld), &never);
      for (int i = 0; i < 2; ++i)
        if (q_used[i] > 0) bar_wait(q_full(i), (q_used[i] - 1) & 1, &never);
    }
  } else if (warp == 9) {
    // ---- products ----
    if (lane == 0) {
      constexpr uint32_t kType = std::is_same<T, __half>::value ? 0u : 1u;
      constexpr uint32_t kIdesc = 1u << 4 | kType << 7 | kType << 10 | (uint32_t)(kTile >> 4) << 24;
      constexpr uint32_t kIdescS = kIdesc | (uint32_t)(kTile >> 3) << 17;
      constexpr uint32_t kIdescO = kIdesc | 1u << 16 | (uint32_t)(DP >> 3) << 17;
      const int steps = (p.C + 1) / 2;
      uint32_t base_n = 0, n_q = 0, q_used[2] = {0, 0}, p_count[2] = {0, 0};
      bool ok = true;
      while (ok && walk.next(&it)) {
        const int n = it.t1 - it.t0;
        const int nt[2] = {chain_tiles<PAIR>(p, it, 0), chain_tiles<PAIR>(p, it, 1)};
        const int qb_split = (int)(n_q & 1);
        if (PAIR) {
          for (int i = 0; i < 2; ++i)
            if (nt[i] > 0) ++q_used[i];
        } else {
          ++q_used[qb_split];
          ++n_q;
        }
        const int longest = max(nt[0], nt[1]);
        // S_i = Q K_j^T into the chain's S columns
        const auto qk = [&](int i, int j) {
          const int tile = PAIR ? j : 2 * j + i;
          const uint32_t ld = base_n + k_place<PAIR>(tile);
          const int qb = PAIR ? i : qb_split;
          if (j == 0 && !bar_wait(q_full(qb), (q_used[qb] - 1) & 1, abort)) return false;
          if (!bar_wait(kv_full(ld), kv_parity(ld), abort)) return false;
          fence_after();
          const uint32_t qa = base + qb * SM::kQ, ka = kv_addr(ld);
          for (int s = 0; s < steps; ++s)
            mma_ss(tmem + i * kTile,
                   smem_desc(qa + (s >> 2) * (kTile * 128) + (s & 3) * 32, 0, 1024, 2),
                   smem_desc(ka + s * (2 * kTile * 16), kTile * 16, 128, 0), kIdescS, s > 0);
          mma_commit(smem_u32(&ctl.s_full[i]));
          if (!PAIR || i == 1 || j >= nt[1]) mma_commit(kv_empty(ld));
          // the row tile's last use
          if (j == nt[i] - 1 && (PAIR || tile == n - 1)) mma_commit(q_empty(qb));
          return true;
        };
        const auto pv = [&](int i, int j) {
          const int tile = PAIR ? j : 2 * j + i;
          const uint32_t ld = base_n + v_place<PAIR>(tile, n);
          if (!bar_wait(kv_full(ld), kv_parity(ld), abort)) return false;
          if (!bar_wait(smem_u32(&ctl.p_ready[i]), p_count[i] & 1, abort)) return false;
          ++p_count[i];
          fence_after();
          const uint32_t va = kv_addr(ld);
          const int rows = min(kTile, it.row_end - (it.t0 + tile) * kTile);
          for (int s = 0; s * 16 < rows; ++s)
            mma_ts(tmem + 2 * kTile + i * kTile, tmem + i * kTile + s * 8,
                   smem_desc(va + s * 2048, kTile * 128, 1024, 2), kIdescO, j > 0 || s > 0);
          if (!PAIR || i == 1 || j >= nt[1]) mma_commit(kv_empty(ld));
          if (j == nt[i] - 1) mma_commit(smem_u32(&ctl.o_done[i]));
          return true;
        };
        for (int i = 0; i < 2 && ok; ++i)
          if (nt[i] > 0) ok = qk(i, 0);
        for (int j = 0; j < longest && ok; ++j)
          for (int i = 0; i < 2 && ok; ++i) {
            if (j < nt[i]) ok = pv(i, j);
            if (ok && j + 1 < nt[i]) ok = qk(i, j + 1);
          }
        base_n += 2 * n;
      }
      // the products that are in flight end before tensor memory is given back
      int never = 0;
      mma_commit(smem_u32(&ctl.drained));
      bar_wait(smem_u32(&ctl.drained), 0, &never);
    }
    __syncwarp();
  } else {
    // ---- softmax: a chain's warpgroup, a thread per row ----
    const int i = warp >> 2, r = threadIdx.x & (kTile - 1);
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // the warp's 32 lanes of tensor memory
    const uint32_t ts = tmem + lanes + i * kTile, to = tmem + lanes + 2 * kTile;
    const int tr = r / p.G, g = r - tr * p.G;
    uint32_t base_n = 0, s_count = 0, o_count = 0, x_count = 0, item = 0;
    bool ok = true;
    for (; ok && walk.next(&it); ++item) {
      const int n = it.t1 - it.t0;
      const int nt[2] = {chain_tiles<PAIR>(p, it, 0), chain_tiles<PAIR>(p, it, 1)};
      const int tile_tok0 = it.tok0 + (PAIR ? i * p.tile_tok : 0);
      const int start = p.seq.start[it.b], n_tok = p.seq.pre[it.b + 1] - p.seq.pre[it.b];
      const int tok = tile_tok0 + tr;
      const bool valid = tr < p.tile_tok && tok < n_tok;
      const bool any_valid = __any_sync(~0u, valid);
      uint64_t bits = 0;
      if (p.is_tree && valid) {
        bits = p.tree ? __ldg(p.tree + p.seq.pre[it.b] + tok) : causal_mask(tok);
        if (n_tok < 64) bits &= (1ull << n_tok) - 1;
      }
      // the other chain may be an item behind, not more (PAIR: bad[]; SPLIT: O)
      if (PAIR ? item >= 2 : item >= 1) {
        const uint32_t w = item - (PAIR ? 2 : 1);
        ok = bar_wait(smem_u32(&ctl.item_done[w & 1]), (w >> 1) & 1, abort);
        if (!ok) break;
      }
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < nt[i]; ++j) {
        const int tile = PAIR ? j : 2 * j + i;
        const int col0 = (it.t0 + tile) * kTile;
        // whether some row of the tile does not attend every column
        const bool masked = p.is_tree ? col0 + kTile > start : col0 + kTile > start + tile_tok0 + 1;
        if (!(ok = bar_wait(smem_u32(&ctl.s_full[i]), s_count & 1, abort))) break;
        ++s_count;
        fence_after();
        if (masked && (!PAIR || i == 0 || j >= nt[0])) {
          // V's hidden rows: zero past the last attended one, finite elsewhere.  (The wait
          // comes after S's: the products have then taken the slot's previous load, and the
          // barrier is not two phases back.)
          const uint32_t ld = base_n + v_place<PAIR>(tile, n);
          if (!(ok = bar_wait(kv_full(ld), kv_parity(ld), abort))) break;
          uint4* const vrow = reinterpret_cast<uint4*>(sm + (kv_addr(ld) - base) + r * 128);
          if (col0 + r >= it.row_end) {
#pragma unroll
            for (int k = 0; k < DP / 8; ++k)
              vrow[(k >> 3) * (kTile * 8) + ((k + r) & 7)] = make_uint4(0, 0, 0, 0);
          } else {
            constexpr uint32_t M = exp_mask<T>();
            uint32_t bad = 0;
#pragma unroll
            for (int k = 0; k < DP / 8; ++k) {
              const uint4 u = vrow[(k >> 3) * (kTile * 8) + ((k + r) & 7)];
              const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {  // a zero half-word of x: all exponent bits set
                const uint32_t x = (w[e] & M) ^ M;
                bad |= (x - 0x00010001u) & ~x & 0x80008000u;
              }
            }
            if (bad) {
              ctl.bad[item & 1] = (int)item;
              uint16_t* const e = reinterpret_cast<uint16_t*>(vrow);
              for (int k = 0; k < DP; ++k) {
                uint16_t& x = e[(k >> 6) * (kTile * 64) + (k & 63)];
                if ((x & (M & 0xffff)) == (M & 0xffff)) x = 0;
              }
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        if (any_valid) {
          uint32_t x[kTile];
#pragma unroll
          for (int k = 0; k < 4; ++k) tmem_ld32(x + 32 * k, ts + 32 * k);
          tmem_wait_ld();
          if (masked) {
            const uint64_t lo = p.is_tree ? tree_mask(bits, col0 - start)
                                          : causal_mask(start + tok - col0);
            const uint64_t hi = p.is_tree ? tree_mask(bits, col0 + 64 - start)
                                          : causal_mask(start + tok - col0 - 64);
#pragma unroll
            for (int k = 0; k < kTile; ++k)
              if (!((k < 64 ? lo : hi) >> (k & 63) & 1)) x[k] = 0xff800000u;  // -inf
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < kTile; ++k) mx[k & 3] = fmaxf(mx[k & 3], __uint_as_float(x[k]));
          const float m_new = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), m);
          if (__any_sync(~0u, valid && (m_new - m) * p.c > kLazy)) {
            const float f = m == -INFINITY ? 0.f : ex2((m - m_new) * p.c);
            m = m_new;
            l *= f;
            if (j > 0) {
#pragma unroll
              for (int k = 0; k < DP / 32; ++k) {
                uint32_t o[32];
                tmem_ld32(o, to + i * kTile + 32 * k);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st32(to + i * kTile + 32 * k, o);
              }
            }
          }
          const float mb = m == -INFINITY ? 0.f : m * p.c;
          float sum[4] = {};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float a = ex2(fmaf(__uint_as_float(x[64 * k + 2 * e]), p.c, -mb));
              const float b = ex2(fmaf(__uint_as_float(x[64 * k + 2 * e + 1]), p.c, -mb));
              sum[e & 3] += a + b;
              w[e] = Pack2<T>::pack(a, b);
            }
            tmem_st32(ts + 32 * k, w);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_wait_st();
        }
        fence_before();
        bar_arrive(smem_u32(&ctl.p_ready[i]));
      }
      if (!ok) break;
      if (nt[i] > 0) {
        if (!(ok = bar_wait(smem_u32(&ctl.o_done[i]), o_count & 1, abort))) break;
        ++o_count;
        fence_after();
      }
      float w0 = 1.f, w1 = 0.f;  // SPLIT: the chains' weights
      if (!PAIR) {
        ctl.ml[i][r] = make_float2(m, l);
        fence_before();
        bar_arrive(smem_u32(&ctl.xchg));
        if (!(ok = bar_wait(smem_u32(&ctl.xchg), x_count & 1, abort))) break;
        ++x_count;
        fence_after();  // the other chain's O has been waited for by its own threads
        const float2 a = ctl.ml[0][r], b = ctl.ml[1][r];
        m = fmaxf(a.x, b.x);
        w0 = a.x == -INFINITY ? 0.f : ex2((a.x - m) * p.c);
        w1 = b.x == -INFINITY ? 0.f : ex2((b.x - m) * p.c);
        l = a.y * w0 + b.y * w1;
      }
      // ---- the piece's output: SPLIT each chain half of the columns ----
      if (any_valid) {
        const bool whole = it.t0 == 0 && it.t1 == it.cnt;
        const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
        const bool patch = ctl.bad[item & 1] == (int)item;
        constexpr int kCols = PAIR ? DP : DP / 2;
        const int c0 = PAIR ? 0 : i * kCols;
        const int hq = it.h * p.G + g;
        uint16_t* const out =
            p.out + (int64_t)(p.seq.pre[it.b] + tok) * p.out_stride + (int64_t)hq * p.D;
        // slot 0: the CTA's first piece, 1: its last
        constexpr int kRows = PAIR ? 2 * kTile : kTile;
        float* const part = p.part + (int64_t)(blockIdx.x * 2 + (item == 0 ? 0 : 1)) * kRows *
                                         (p.D + 2);
        const int prow = (PAIR ? i * kTile : 0) + r;
        if (!whole && valid && (PAIR || i == 0))
          reinterpret_cast<float2*>(part + kRows * p.D)[prow] = make_float2(m * p.c, l);
#pragma unroll 1
        for (int k = 0; k < kCols; k += 32) {
          uint32_t o[32];
          if (nt[PAIR ? i : 0] > 0) {
            tmem_ld32(o, to + (PAIR ? i * kTile : 0) + c0 + k);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0;
          }
          if (!PAIR) {
            if (w0 != 1.f || w1 != 0.f) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                o[e] = __float_as_uint(w0 == 0.f ? 0.f : __uint_as_float(o[e]) * w0);
            }
            if (nt[1] > 0) {
              uint32_t o1[32];
              tmem_ld32(o1, to + kTile + c0 + k);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (w1 != 0.f)
                  o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), w1, __uint_as_float(o[e])));
            }
          }
          if (valid) {
            if (patch) {
              // the non-finite values that the row does attend, from the cache
              const int first = (p.is_tree ? start : start + it.tok0 + 1) / kTile * kTile;
              const int64_t head = (int64_t)it.b * p.H + it.h;
              for (int row = max(first, it.t0 * kTile); row < min(it.row_end, it.t1 * kTile); ++row) {
                if (row >= start &&
                    !(p.is_tree ? (bits >> (row - start) & 1) != 0 : row <= start + tok))
                  continue;
                const uint16_t* vr = p.v + (head * p.S + row) * p.D + c0 + k;
                for (int e = 0; e < 32; e += 2) {
                  if (c0 + k + e >= p.D) break;
                  const float2 f = Pack2<T>::unpack(*reinterpret_cast<const uint32_t*>(vr + e));
#pragma unroll
                  for (int q = 0; q < 32; q += 2)
                    if (q == e) {
                      if (!isfinite(f.x)) o[q] = __float_as_uint(__uint_as_float(o[q]) + f.x);
                      if (!isfinite(f.y)) o[q + 1] = __float_as_uint(__uint_as_float(o[q + 1]) + f.y);
                    }
                }
              }
            }
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              if (c0 + k + e >= p.D) break;
              if (whole) {
                uint32_t w[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  w[q] = Pack2<T>::pack(__uint_as_float(o[e + 2 * q]) * inv,
                                        __uint_as_float(o[e + 2 * q + 1]) * inv);
                *reinterpret_cast<uint4*>(out + c0 + k + e) = make_uint4(w[0], w[1], w[2], w[3]);
              } else {
                float* const d = part + (int64_t)prow * p.D + c0 + k + e;
                *reinterpret_cast<uint4*>(d) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                *reinterpret_cast<uint4*>(d + 4) = make_uint4(o[e + 4], o[e + 5], o[e + 6], o[e + 7]);
              }
            }
          }
        }
      }
      fence_before();
      bar_arrive(smem_u32(&ctl.item_done[item & 1]));
      base_n += 2 * n;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 8)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
}

// ---- the join ----------------------------------------------------------------------

// Adds up the pieces of the unit that the cut after CTA blockIdx.x divides, if
// that is the unit's first cut:
//   out = sum_i f_i O_i / sum_i f_i l_i,  f_i = exp2(m_i - max m).
template <typename T, int MAXB>
__global__ __launch_bounds__(256) void join_kernel(const __grid_constant__ AttnParams<MAXB> p,
                                                   int ctas, int rows_per_unit) {
  ops_pdl_enter();
  const int i0 = blockIdx.x;
  const int64_t at = cut(p, i0 + 1, ctas);
  const Walk<AttnParams<MAXB>> walk(p, at, at + 1);  // the unit that holds tile `at`
  if (walk.t == 0) return;                           // no unit is divided here
  const int64_t lo = at - walk.t, from = cut(p, i0, ctas);
  if (from > lo) return;  // an earlier cut divides it too
  const int rows_end = unit_rows(p, walk.b, walk.tok0);
  const int64_t hi = lo + (rows_end + kTile - 1) / kTile;
  int i1 = i0 + 1;  // the last CTA with a piece
  while (cut(p, i1 + 1, ctas) < hi) ++i1;
  const int n_tok = min(p.seq.pre[walk.b + 1] - p.seq.pre[walk.b] - walk.tok0, p.unit_tok);
  const int lane = threadIdx.x & 31;
  const int64_t slot = (int64_t)rows_per_unit * (p.D + 2);
  for (int q = blockIdx.y * 8 + (threadIdx.x >> 5); q < n_tok * p.G; q += gridDim.y * 8) {
    const int tok = q / p.G, g = q - tok * p.G;
    const int tile = tok / p.tile_tok;
    const int r = tile * kTile + (tok - tile * p.tile_tok) * p.G + g;
    const auto piece = [&](int i) {
      return p.part + slot * (2 * i + (i == i0 && from < lo ? 1 : 0));
    };
    float m = -INFINITY;
    for (int i = i0; i <= i1; ++i)
      m = fmaxf(m, reinterpret_cast<const float2*>(piece(i) + (int64_t)rows_per_unit * p.D)[r].x);
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = i0; i <= i1; ++i) {
      const float* const pc = piece(i);
      const float2 ml = reinterpret_cast<const float2*>(pc + (int64_t)rows_per_unit * p.D)[r];
      if (ml.x == -INFINITY) continue;
      const float f = ex2(ml.x - m);
      l += f * ml.y;
      if (lane * 4 < p.D) {
        const float4 a = reinterpret_cast<const float4*>(pc + (int64_t)r * p.D)[lane];
        o.x += f * a.x;
        o.y += f * a.y;
        o.z += f * a.z;
        o.w += f * a.w;
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (lane * 4 < p.D) {
      uint16_t* const out = p.out + (int64_t)(p.seq.pre[walk.b] + walk.tok0 + tok) * p.out_stride +
                            (int64_t)(walk.h * p.G + g) * p.D;
      reinterpret_cast<uint2*>(out)[lane] =
          make_uint2(Pack2<T>::pack(o.x * inv, o.y * inv), Pack2<T>::pack(o.z * inv, o.w * inv));
    }
  }
}

// ---- host ---------------------------------------------------------------------------

// How a call is cut into units and CTAs.
struct Schedule {
  bool pair;
  int tile_tok, unit_tok;
  int64_t total;  // tiles
  int64_t units;
  int ctas;
  size_t bytes;  // of workspace
};

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    n = 152;
  }
  return n;
}

constexpr int kMinTiles = 4;  // a CTA's share is not cut below this many tiles

Schedule schedule(const Plan& p, int group, bool is_tree, int64_t* tile_pre) {
  Schedule s;
  s.tile_tok = kTile / group;
  s.pair = p.max_len > s.tile_tok;
  s.unit_tok = s.tile_tok * (s.pair ? 2 : 1);
  s.total = s.units = 0;
  for (int b = 0; b < p.B; ++b) {
    if (tile_pre) tile_pre[b] = s.total;
    const int n = p.seq_len[b], first = p.seq_start[b];
    int64_t tiles = 0;
    for (int64_t u = 0; u < n; u += s.unit_tok) {
      const int64_t rows = first + (is_tree || u + s.unit_tok > n ? n : u + s.unit_tok);
      tiles += (rows + kTile - 1) / kTile;
      s.units += p.H;
    }
    s.total += tiles * p.H;
  }
  if (tile_pre) tile_pre[p.B] = s.total;
  const int64_t sms = sm_count();
  int64_t ctas = s.total / kMinTiles;
  if (ctas < s.units) ctas = s.units;
  if (ctas > sms) ctas = sms;
  if (ctas < 1) ctas = 1;
  s.ctas = (int)ctas;
  s.bytes = ctas > 1 ? (size_t)ctas * 2 * (s.pair ? 2 : 1) * kTile * (p.D + 2) * sizeof(float) : 0;
  return s;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

bool encode(CUtensorMap* map, bool fp16, int rank, const void* base, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  static const EncodeFn fn = reinterpret_cast<EncodeFn>(driver_fn("cuTensorMapEncodeTiled"));
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return fn && fn(map, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                  (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int DP, bool PAIR, int MAXB>
cudaError_t launch_kernel(const AttnParams<MAXB>& kp, int ctas, cudaStream_t stream) {
  void (*const kernel)(AttnParams<MAXB>) = attention_kernel<T, DP, PAIR, MAXB>;
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Smem<DP>::kBytes);
  if (err != cudaSuccess) return err;
  return ops_launch(kernel, dim3((unsigned)ctas), kThreadsAttn, Smem<DP>::kBytes, stream, kp);
}

template <typename T, int MAXB>
dv_status launch_attention(const Plan& p, const dv_queries& q, bool is_tree, const uint64_t* tree,
                           float* part, size_t part_bytes, cudaStream_t stream) {
  AttnParams<MAXB> kp;
  const int group = q.q_heads / p.H;
  const Schedule s = schedule(p, group, is_tree, kp.tile_pre);
  const bool fp16 = q.dtype == DV_DTYPE_FP16;
  const void* k = static_cast<const uint4*>(p.k) + p.l0 * p.layer_chunks;
  const void* v = static_cast<const uint4*>(p.v) + p.l0 * p.layer_chunks;
  const cuuint64_t D = (cuuint64_t)p.D;
  const cuuint64_t qd[4] = {D, (cuuint64_t)group, (cuuint64_t)p.H, (cuuint64_t)p.tokens};
  const cuuint64_t qs[3] = {D * 2, D * 2 * group,
                            (cuuint64_t)(p.tokens > 1 ? q.q_stride : (int64_t)q.q_heads * p.D) * 2};
  const cuuint32_t qb[4] = {64, (cuuint32_t)group, 1, (cuuint32_t)s.tile_tok};
  const cuuint64_t vd[3] = {D, (cuuint64_t)p.S, (cuuint64_t)p.B * p.H};
  const cuuint64_t vs[2] = {D * 2, D * 2 * p.S};
  const cuuint32_t vb[3] = {64, 32, 1};
  if (!encode(&kp.q_map, fp16, 4, q.q, qd, qs, qb) || !encode(&kp.v_map, fp16, 3, v, vd, vs, vb))
    return fail(DV_ERR_CUDA, "cuTensorMapEncodeTiled refused the queries or the cache");
  kp.out = static_cast<uint16_t*>(q.out);
  kp.k = static_cast<const uint4*>(k);
  kp.v = static_cast<const uint16_t*>(v);
  kp.tree = tree;
  kp.part = part;
  kp.out_stride = q.out_stride;
  kp.total = s.total;
  kp.H = p.H;
  kp.G = group;
  kp.D = p.D;
  kp.C = p.C;
  kp.S = p.S;
  kp.tile_tok = s.tile_tok;
  kp.unit_tok = s.unit_tok;
  kp.is_tree = is_tree ? 1 : 0;
  kp.c = q.scale * 1.4426950408889634f;
  fill_table(p, &kp.seq);
  cudaError_t err;
  if (p.D <= 64)
    err = s.pair ? launch_kernel<T, 64, true, MAXB>(kp, s.ctas, stream)
                 : launch_kernel<T, 64, false, MAXB>(kp, s.ctas, stream);
  else
    err = s.pair ? launch_kernel<T, 128, true, MAXB>(kp, s.ctas, stream)
                 : launch_kernel<T, 128, false, MAXB>(kp, s.ctas, stream);
  if (err != cudaSuccess) return cuda_fail(err, "attention launch");
  if (s.ctas > 1) {
    void (*const join)(AttnParams<MAXB>, int, int) = join_kernel<T, MAXB>;
    err = ops_launch(join, dim3((unsigned)s.ctas - 1, 8), 256, 0, stream, kp, (int)s.ctas,
                     (s.pair ? 2 : 1) * kTile);
    if (err != cudaSuccess) return cuda_fail(err, "attention join launch");
  }
  return DV_OK;
}

dv_status check_heads(const dv_cache* cache, const Plan& p, int32_t q_heads) {
  if (cache->elem_bytes != 2)
    return fail(DV_ERR_UNSUPPORTED, "attention needs 2-byte elements (elem_bytes %d)",
                cache->elem_bytes);
  if (p.D > 128) return fail(DV_ERR_UNSUPPORTED, "attention needs head_dim <= 128 (got %d)", p.D);
  if (q_heads <= 0 || q_heads % p.H != 0)
    return fail(DV_ERR_INVALID_ARG, "q_heads %d is not a multiple of num_heads %d", q_heads, p.H);
  if (q_heads / p.H > DV_MAX_GROUP)
    return fail(DV_ERR_UNSUPPORTED, "%d query heads share a key head, more than %d", q_heads / p.H,
                DV_MAX_GROUP);
  return DV_OK;
}

dv_status attention(const dv_cache* cache, int32_t layer, const int32_t* s, const int32_t* e,
                    const dv_queries* queries, bool is_tree, const uint64_t* tree, void* workspace,
                    size_t workspace_bytes, cudaStream_t stream) {
  if (!queries) return fail(DV_ERR_INVALID_ARG, "queries is NULL");
  Plan p;
  dv_status st = plan_layer(cache, layer, s, e, queries->dtype, &p);
  if (st != DV_OK) return st;
  dv_queries q = *queries;
  if ((st = check_heads(cache, p, q.q_heads)) != DV_OK) return st;
  if (!(q.scale > 0.f) || !std::isfinite(q.scale))
    return fail(DV_ERR_INVALID_ARG, "scale must be finite and positive (got %g)", (double)q.scale);
  if (is_tree && p.max_len > DV_MAX_TREE)
    return fail(DV_ERR_UNSUPPORTED, "%d drafted tokens of a sequence, more than %d", p.max_len,
                DV_MAX_TREE);
  if (p.tokens == 0) return DV_OK;
  const size_t need = schedule(p, q.q_heads / p.H, is_tree, nullptr).bytes;
  if (workspace_bytes < need)
    return fail(DV_ERR_BUFFER_TOO_SMALL, "attention needs %zu workspace bytes (got %zu)", need,
                workspace_bytes);
  if ((st = resolve_cache(cache, &p)) != DV_OK) return st;
  void* dev = nullptr;
  size_t nq = 0, no = 0;
  if ((st = resolve_rows(p, q.q, q.q_heads, q.q_stride, "q", &dev, &nq)) != DV_OK) return st;
  q.q = dev;
  if ((st = resolve_rows(p, q.out, q.q_heads, q.out_stride, "out", &dev, &no)) != DV_OK) return st;
  q.out = dev;
  if (overlap(q.out, no, q.q, nq)) return fail(DV_ERR_INVALID_ARG, "out overlaps q");
  if (tree) {
    if ((st = resolve_words(tree, (size_t)p.tokens * 8, 8, "tree", &dev)) != DV_OK) return st;
    tree = static_cast<const uint64_t*>(dev);
  }
  float* part = nullptr;
  if (need > 0) {
    if ((st = resolve(workspace, need, false, "workspace", &dev)) != DV_OK) return st;
    part = static_cast<float*>(dev);
    if (overlap(part, need, q.q, nq) || overlap(part, need, q.out, no))
      return fail(DV_ERR_INVALID_ARG, "workspace overlaps q or out");
  }
  const bool small = p.B <= kSmallBatch;
  if (q.dtype == DV_DTYPE_FP16)
    return small ? launch_attention<__half, kSmallBatch>(p, q, is_tree, tree, part, need, stream)
                 : launch_attention<__half, kMaxBatch>(p, q, is_tree, tree, part, need, stream);
  return small
             ? launch_attention<__nv_bfloat16, kSmallBatch>(p, q, is_tree, tree, part, need, stream)
             : launch_attention<__nv_bfloat16, kMaxBatch>(p, q, is_tree, tree, part, need, stream);
}

}  // namespace
}  // namespace dv

extern "C" dv_status dv_attention_workspace(const dv_cache* cache, const int32_t* seq_start,
                                            const int32_t* seq_end, int32_t q_heads,
                                            size_t* bytes) {
  if (!bytes) return dv::fail(DV_ERR_INVALID_ARG, "bytes is NULL");
  dv::Plan p;
  dv_status st = dv::plan_ranges(cache, 0, 1, seq_start, seq_end, &p);
  if (st != DV_OK) return st;
  if ((st = dv::check_heads(cache, p, q_heads)) != DV_OK) return st;
  *bytes = 0;
  if (p.tokens == 0) return DV_OK;
  const int group = q_heads / p.H;
  const size_t a = dv::schedule(p, group, false, nullptr).bytes;
  const size_t b = p.max_len <= DV_MAX_TREE ? dv::schedule(p, group, true, nullptr).bytes : 0;
  *bytes = a > b ? a : b;
  return DV_OK;
}

extern "C" dv_status dv_attention_check(dv_stream stream) {
  void* flag = nullptr;
  cudaError_t err = cudaGetSymbolAddress(&flag, dv::g_attention_timeout);
  unsigned int v = 0;
  if (err == cudaSuccess)
    err = cudaMemcpyAsync(&v, flag, sizeof(v), cudaMemcpyDeviceToHost, stream);
  if (err == cudaSuccess && (err = cudaStreamSynchronize(stream)) == cudaSuccess && v != 0) {
    err = cudaMemsetAsync(flag, 0, sizeof(v), stream);
    if (err == cudaSuccess)
      return dv::fail(DV_ERR_TIMEOUT, "an attention kernel gave up a wait; its output is not valid");
  }
  return err == cudaSuccess ? DV_OK : dv::cuda_fail(err, "reading the attention kernels' flag");
}

extern "C" dv_status dv_prompt_attention(const dv_cache* cache, int32_t layer,
                                         const int32_t* seq_start, const int32_t* seq_end,
                                         const dv_queries* queries, void* workspace,
                                         size_t workspace_bytes, dv_stream stream) {
  dv::Trace trace("dv_prompt_attention");
  return dv::attention(cache, layer, seq_start, seq_end, queries, false, nullptr, workspace,
                       workspace_bytes, stream);
}

extern "C" dv_status dv_tree_attention(const dv_cache* cache, int32_t layer,
                                       const int32_t* seq_start, const int32_t* seq_end,
                                       const dv_queries* queries, const uint64_t* tree,
                                       void* workspace, size_t workspace_bytes, dv_stream stream) {
  dv::Trace trace("dv_tree_attention");
  return dv::attention(cache, layer, seq_start, seq_end, queries, true, tree, workspace,
                       workspace_bytes, stream);
}

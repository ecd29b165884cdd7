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
// 256; P keeps its relative precision, l is summed in 32 bits; a published
// method).  fp16's p are held 2^7 times as large, in the middle of its range.
//
// Two chains of such tiles run at once, one's softmax under the other's
// products:
//   PAIR   two row tiles (256 rows) over the same K/V tiles: prompts.
//   SPLIT  one row tile, the even K/V tiles on one chain and the odd ones on
//          the other, joined at the end: decode steps and small trees, bound
//          by reading K and V once.
// PAIR where some sequence has more rows than a row tile, SPLIT otherwise, one
// form for a call.  PAIR and SPLIT, us: 8 prompts of 1000, 25 heads of 64, 51 and
// 65, of 129 to 384 within 6% either way; 32 prompts of 256, 40 heads of 128, 67
// and 73, of 1000 339 and 456; 2 x 64 nodes after 131000, 64 query heads on 8,
// 362 and 587.  PAIR runs a sequence of one row tile on one chain: a chunk of
// 2048 with 31 single tokens after 500 to 8000 rows takes 163 where SPLIT takes
// 140, 8 x 64 nodes after 2000 rows 50 and 45.
// P is handed over in two halves, so that the products with V start under the
// second half's exponentials.
//
// Warps: 0-3 and 4-7 the chains' softmax, 8 loads (and walks over the units,
// publishing each in a ring), 9 and 10 issue the chains' products, 11 looks
// after V's hidden rows.  K goes to shared memory by TMA in its own layout: the
// cache's [D/8][S][8] is, per tile, exactly the tensor core's unswizzled layout
// of 8 x 16-byte core matrices, so nothing is transposed.  V goes in with the
// 128-byte swizzle and is read with its rows as the contraction.  A sequence's
// last, partial tile is fetched up to the last attended row (K in bulk copies,
// V in 32s).
//
// The units form one line, each as long as its cost, cut into equal stretches,
// one for each CTA (one CTA an SM); a unit that a cut divides leaves partial
// sums in the workspace, which join_kernel adds up.
//
// Rows a mask hides must have no effect, but 0 x NaN is NaN in a product: in
// tiles that hold hidden rows, warp 11 sets V's non-finite values to zero in
// shared memory (rows past the last attended one altogether), while the tile's
// scores are computed, and should there have been any, the epilogue adds them
// to the outputs of the rows that do attend them.
//
// Every wait gives up after a number of tries (kSpinLimit, unless a test has set fewer):
// the CTA then drains its copies and products, each with a bounded wait too, frees its tensor
// memory and returns, and dv_attention_check reports it.
//
// Measured (bf16, heads of 128 unless said; in a long loop, where the power cap
// counts).  SPLIT is bound by HBM: a decode step of 32 sequences of 64 to 1791
// rows, 112 heads (1.52 GB) 230 to 232 us, 6.5 to 6.6 TB/s.
// PAIR is bound by the chain scores - softmax - products of a tile, about 3100
// cycles for a pair of tiles whose products take 2048 on the tensor cores: 4096
// tokens after 28672, 64 query heads on 8, 2.72 to 2.81 ms, 1.47 to 1.52 PFLOP/s (2.63
// to 2.68 alone); on short prompts the filling and draining of the chains come on
// top, and the half of the diagonal tiles that is hidden: 32 prompts of 64 to 1536
// tokens, 112 heads, 0.85 to 0.86 ms, 0.84 PFLOP/s attended.
// Heads of 64 halve the products but not the softmax: 8 prompts of 1000, 25
// heads (fp16), 54 us.  What was tried and was slower: S in halves of 64
// columns two steps ahead; two buffers of 96 columns for heads of 64; the
// maximum from a second pass over S, or only when a sum grows too large (7 to
// 10% each); one product warp for both chains (28% on ragged prompts); the next
// tile's second half of scores issued as soon as S has been read (4 to 6%).
#include <cuda.h>

#include <atomic>
#include <mutex>
#include <vector>

#include "dv_ops.h"

namespace dv {
namespace {

constexpr int kTile = 128;        // rows of Q and of K/V in a tile
constexpr int kThreadsAttn = 384;  // two softmax warpgroups, and one of the other warps
constexpr uint32_t kSpinLimit = 1u << 22;
constexpr int kJoinThreads = 256;
constexpr int kTurnPolls = 32;     // of another chain's progress, a preference (about 1 us)
constexpr float kLazy = 8.f;       // log2 of the growth that is left to the old maximum
// fp16 holds weights to 2^-25 of the largest and loses bits of those below 2^-14: log2 of a
// factor on all of a row's weights, and on l with them, that takes both down by its share.
// 2^(kLazy + kHalfUp) stays below fp16's 2^16.
constexpr float kHalfUp = 7.f;

// Waits in attention kernels that gave up, one for each lane; only ever grows, so that no
// caller's check takes another's record away.
__device__ unsigned long long g_attention_gave_up;
// The second half of the last contraction step when head_dim is an odd number of chunks.
__device__ uint4 g_zero_rows[kTile];

// A unit that a cut divides (the first cut that does), for the join.
struct Divided {
  int32_t tok, head, tokens;  // first token and query head of its output; tokens (0: none here)
  int32_t last, slot;         // the last CTA with a piece; the first piece's slot
  int32_t pad[3];
};

template <int MAXB>
struct AttnParams {
  CUtensorMap q_map;   // {D, G, H, T}, 64 x G x 1 x tokens of a tile
  CUtensorMap k_map;   // {8 w, S / w, C, B * H}, 8 w x 128 / w x C x 1: w rows of a chunk row in one run
  CUtensorMap v_map;   // {D, S, B * H}, 64 x 128 x 1
  CUtensorMap v_part;  // the same, 64 x 32 x 1
  uint16_t* out;
  const uint4* k;
  const uint16_t* v;
  const uint64_t* tree;
  float* part;       // two slots a CTA for pieces' sums
  Divided* divided;  // of the cut before each CTA but the first
  int64_t out_stride;
  int32_t share, extra;  // a CTA's part of the units' cost; the first `extra` have one more
  int32_t H, G, D, C, S;
  int32_t k_rows;    // w of k_map
  int32_t tile_tok;  // tokens of a row tile: 128 / G
  int32_t unit_tok;  // tokens of a unit
  int32_t unit_cost;  // in tiles, on top of a unit's tiles
  int32_t is_tree;
  uint32_t tries;    // of a wait, before it gives up
  int32_t wide;  // every output row of a head is 32-byte aligned, of whole 32-byte sectors
  float c;  // scale * log2(e)
  SeqTable<MAXB> seq;
  int32_t cost_pre[MAXB + 1];  // cost of the sequences before
};

// ---- instructions --------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
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
// Waits, as a whole warp, for the phase of `parity` to complete; false when it gave up after
// `tries`.  The vote makes it one answer for the warp's lanes, which go on to instructions
// that need all of them: a phase may complete between one lane's last try and another's.
// (It costs 1 to 2% on short and ragged prompts, less on trees.)  Kept short: it stands at
// some thirty places, and the kernel's speed hangs on its size (an instruction cache miss in
// every loop made ragged prompts twice as slow); the record is out of line (3 KB, 0.4%).
__device__ __noinline__ bool gave_up() {
  atomicAdd(&g_attention_gave_up, 1ull);
  return false;
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, uint32_t tries) {
  bool ok = false;
#pragma unroll 1
  for (; tries != 0 && !(ok = bar_try(bar, parity)); --tries) {
  }
  return __all_sync(~0u, ok) || gave_up();
}

// The load and the product warp run their loops as whole warps on uniform
// values, and one elected lane (`on`) issues: descriptors and addresses then
// stay in uniform registers, from where these instructions take them.
__device__ __forceinline__ bool elect() {
  uint32_t on;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(on));
  return on != 0;
}
#define DV_ON(n) "{\n .reg .pred q;\n setp.ne.b32 q, %" #n ", 0;\n @q "
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes, bool on) {
  asm volatile(DV_ON(2) "mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}" ::"r"(bar),
               "r"(bytes), "r"((uint32_t)on)
               : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar, bool on) {
  asm volatile(DV_ON(4)
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n}" ::
          "r"(dst), "l"(src), "r"(bytes), "r"(bar), "r"((uint32_t)on)
      : "memory");
}
__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                          uint32_t bar, bool on) {
  asm volatile(DV_ON(6)
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];\n}" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar),
      "r"((uint32_t)on)
      : "memory");
}
__device__ __forceinline__ void tma_load4(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                          int w, uint32_t bar, bool on) {
  asm volatile(DV_ON(7)
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];\n}" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(w),
      "r"(bar), "r"((uint32_t)on)
      : "memory");
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc,
                                       bool on) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b),
      "r"(idesc), "r"((uint32_t)acc), "r"((uint32_t)on)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc,
                                       bool on) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d), "r"(a), "l"(b),
      "r"(idesc), "r"((uint32_t)acc), "r"((uint32_t)on)
      : "memory");
}
// Arrives on `bar` once every product issued so far has finished.
__device__ __forceinline__ void mma_commit(uint32_t bar, bool on) {
  asm volatile(DV_ON(1)
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar),
      "r"((uint32_t)on)
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
__device__ __forceinline__ void tmem_ld16(uint32_t* a, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : DV_R8(a, 0), DV_R8(a, 8)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* a) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      DV_W8(a, 0), DV_W8(a, 8)
      : "memory");
}

// 32 bytes to a 32-byte aligned place.
__device__ __forceinline__ void st32(void* dst, const uint32_t* a) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), DV_W8(a, 0)
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

// A unit, or the piece of one, that the CTA works on.
struct Item {
  int b, h;
  int tok0;     // the unit's first token in its sequence
  int row_end;  // rows [0, row_end) are attended by some row of the unit
  int t0, n;    // the piece's tiles [t0, t0 + n); n = 0: no more items
  int whole;    // the piece is the whole unit
  int nt0, nt1;  // tiles of each chain
  int masked;   // the first tile that hides a row from some query row
  int start, n_tok, tok_at;  // the sequence's first new row, new tokens, place in packed buffers
  int bad;      // non-finite values were taken out of V
};
constexpr int kItems = 4;

template <int DP>
struct Smem {
  static constexpr int kQ = kTile * DP * 2;     // bytes of a row tile
  static constexpr int kSlot = kTile * DP * 2;  // bytes of a K or V tile
  static constexpr int kK = DP == 128 ? 2 : 5;  // K tiles held
  static constexpr int kV = DP == 128 ? 3 : 5;  // V tiles held (longer: until the softmax is done)
  static constexpr int kKAt = 2 * kQ, kVAt = kKAt + kK * kSlot;
  static constexpr int kCtl = kVAt + kV * kSlot;
  struct Ctl {
    uint64_t q_full[2], q_empty[2];
    uint64_t k_full[kK], k_empty[kK], v_full[kV], v_ok[kV], v_empty[kV];
    uint64_t s_full[2], p_half[2], p_ready[2], o_done[2];
    uint64_t item_full[kItems], item_empty[kItems], o_read[2], xchg, drained;
    Item item[kItems];
    float2 ml[2][kTile];  // SPLIT: the chains' maxima and sums
    uint32_t tmem;
    volatile int turn[2];  // PAIR: tiles whose softmax the chain is through the maximum of
  };
  static constexpr int kBytes = kCtl + (int)sizeof(Ctl);
  static_assert(kBytes <= 232448, "more shared memory than a CTA has");
};

// A place in a ring of N: its slot, and the parity of its turn.
template <int N>
struct Ring {
  uint32_t slot = 0, turn = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      turn ^= 1;
    }
  }
};

// ---- the walk over units ---------------------------------------------------------

// Rows attended by some row of the unit of tokens [tok0, tok0 + unit_tok) of sequence b.
template <typename P>
__device__ __forceinline__ int unit_rows(const P& p, int b, int tok0) {
  const int n = p.seq.pre[b + 1] - p.seq.pre[b];
  return p.seq.start[b] + (p.is_tree ? n : min(tok0 + p.unit_tok, n));
}

template <typename P>
struct Walk {
  const P& p;
  int pos, end;       // where the unit starts on the line of costs; where the CTA's stretch ends
  int b, h, tok0, t;  // the next piece: its unit and first tile

  __device__ Walk(const P& p_, int lo, int hi) : p(p_), pos(lo), end(hi) {
    b = h = tok0 = t = 0;
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
#pragma unroll 1
    for (;;) {
      const int cost = p.unit_cost + (unit_rows(p, b, tok0) + kTile - 1) / kTile;
      if (rem < cost) break;
      rem -= cost;
      tok0 += p.unit_tok;
    }
    pos = lo - rem;
    t = max(0, rem - p.unit_cost);
  }

  template <bool PAIR>
  __device__ void next(Item* it) {
    it->n = 0;
    if (pos >= end) return;
    const int start = p.seq.start[b], at = p.seq.pre[b], n_tok = p.seq.pre[b + 1] - at;
    const int row_end = unit_rows(p, b, tok0), cnt = (row_end + kTile - 1) / kTile;
    const int n = min(cnt, end - pos - p.unit_cost) - t;
    if (n <= 0) return;
    it->b = b;
    it->h = h;
    it->tok0 = tok0;
    it->row_end = row_end;
    it->t0 = t;
    it->n = n;
    it->whole = t == 0 && n == cnt;
    it->start = start;
    it->n_tok = n_tok;
    it->tok_at = at;
    it->bad = 0;
    it->masked = (p.is_tree ? start : start + tok0 + 1) / kTile;
    if (PAIR) {
      // chain 0's row tile may end earlier, chain 1's may be empty
      const int tok1 = tok0 + p.tile_tok;
      const int rows0 = p.is_tree ? row_end : start + min(tok1, n_tok);
      it->nt0 = max(0, min(t + n, (rows0 + kTile - 1) / kTile) - t);
      it->nt1 = tok1 < n_tok ? n : 0;
    } else {
      it->nt0 = (n + 1) / 2;
      it->nt1 = n / 2;
    }
    pos += p.unit_cost + cnt;
    t = 0;
    tok0 += p.unit_tok;
    if (tok0 >= n_tok) {
      tok0 = 0;
      if (++h == p.H) {
        h = 0;
        if (pos < end) do ++b; while (p.seq.pre[b + 1] == p.seq.pre[b]);
      }
    }
  }
};

// Where CTA i's stretch of the line starts.
template <typename P>
__device__ __forceinline__ int cut(const P& p, int i) {
  return p.share * i + min(i, p.extra);
}

// ---- the kernel ------------------------------------------------------------------

// 32-column masks of the columns a row attends.
// Bit c of `bits`: new row c; rows before the new ones are always attended.
__device__ __forceinline__ uint32_t tree_mask(uint64_t bits, int rel) {  // rel: column 0 - start
  if (rel <= -32) return ~0u;
  if (rel < 0) return (uint32_t)bits << -rel | ((1u << -rel) - 1);
  return rel < 64 ? (uint32_t)(bits >> rel) : 0u;
}
__device__ __forceinline__ uint32_t causal_mask(int last) {  // the last attended column
  return last >= 31 ? ~0u : last < 0 ? 0u : (2u << last) - 1;
}

// (a, b) = (a, b) * c + d, and (a, b) += (c, d)
__device__ __forceinline__ void fma2(float& a, float& b, float c, float d) {
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %2};\n"
      " mov.b64 z, {%3, %3};\n fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}"
      : "+f"(a), "+f"(b)
      : "f"(c), "f"(d));
}
__device__ __forceinline__ void add2(float& a, float& b, float c, float d) {
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n"
      " add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
      : "+f"(a), "+f"(b)
      : "f"(c), "f"(d));
}

template <typename T, int DP, bool PAIR, int MAXB>
__global__ __launch_bounds__(kThreadsAttn, 1) void attention_kernel(
    const __grid_constant__ AttnParams<MAXB> p) {
  using SM = Smem<DP>;
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t base = smem_u32(sm);
  if ((base & 1023) != 0) {  // the swizzle goes by address bits
    ops_pdl_enter();
    if (threadIdx.x == 0) {
      gave_up();
      if (blockIdx.x > 0) p.divided[blockIdx.x - 1] = Divided{};  // nothing for the join
    }
    return;
  }
  typename SM::Ctl& ctl = *reinterpret_cast<typename SM::Ctl*>(sm + SM::kCtl);
  const int warp = __shfl_sync(~0u, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  // a barrier's shared-memory address
  const auto at = [&](const uint64_t& bar) {
    return base + (uint32_t)(reinterpret_cast<const uint8_t*>(&bar) - sm);
  };

  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     base + (uint32_t)(reinterpret_cast<uint8_t*>(&ctl.tmem) - sm)),
                 "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (threadIdx.x == 0) {
    ctl.turn[0] = ctl.turn[1] = 0;
    for (int i = 0; i < 2; ++i) {
      bar_init(at(ctl.q_full[i]), 1);
      bar_init(at(ctl.q_empty[i]), PAIR ? 1 : 2);  // the chains that use it
      bar_init(at(ctl.s_full[i]), 1);
      bar_init(at(ctl.p_half[i]), kTile);
      bar_init(at(ctl.p_ready[i]), kTile);
      bar_init(at(ctl.o_done[i]), 1);
      bar_init(at(ctl.o_read[i]), 2 * kTile);
    }
    for (int i = 0; i < SM::kK; ++i) {
      bar_init(at(ctl.k_full[i]), 1);
      bar_init(at(ctl.k_empty[i]), 2);  // both chains
    }
    for (int i = 0; i < SM::kV; ++i) {
      bar_init(at(ctl.v_full[i]), 1);
      bar_init(at(ctl.v_ok[i]), 1);
      bar_init(at(ctl.v_empty[i]), 3);  // both chains, and the look at hidden rows
    }
    for (int i = 0; i < kItems; ++i) {
      bar_init(at(ctl.item_full[i]), 1);
      bar_init(at(ctl.item_empty[i]), 11);  // all warps but the loads'
    }
    bar_init(at(ctl.xchg), 2 * kTile);
    bar_init(at(ctl.drained), 2);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(~0u, ctl.tmem, 0);
  // (Global memory is touched only past this; the load warp finds its first unit before.)
  if (warp != 8) ops_pdl_enter();

  const auto wait = [&](uint32_t bar, uint32_t parity) { return bar_wait(bar, parity, p.tries); };
  // The k-th item, from the ring.
  const auto get_item = [&](uint32_t k, Item* it) {
    if (!wait(at(ctl.item_full[k % kItems]), k / kItems & 1)) return false;
    *it = ctl.item[k % kItems];
    return __all_sync(~0u, it->n > 0) != 0;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    if (warp == 8) {
      // ---- the walk, and loads ----
      {
        const bool on = elect();
        Walk<AttnParams<MAXB>> walk(p, cut(p, blockIdx.x),
                                    cut(p, blockIdx.x + 1));
        ops_pdl_enter();
        if (blockIdx.x > 0 && on) {
          Divided d = {};
          const int from = cut(p, blockIdx.x - 1);
          if (walk.t > 0 && from <= walk.pos + p.unit_cost) {
            const int n_tok = p.seq.pre[walk.b + 1] - p.seq.pre[walk.b] - walk.tok0;
            const int end = walk.pos + p.unit_cost +
                            (unit_rows(p, walk.b, walk.tok0) + kTile - 1) / kTile;
            d.tok = p.seq.pre[walk.b] + walk.tok0;
            d.head = walk.h * p.G;
            d.tokens = min(n_tok, p.unit_tok);
            d.last = blockIdx.x;
#pragma unroll 1
            while (cut(p, d.last + 1) < end) ++d.last;
            d.slot = from < walk.pos ? 1 : 0;
          }
          p.divided[blockIdx.x - 1] = d;
        }
        Item it, after;
        Ring<SM::kK> kr;
        Ring<SM::kV> vr;
        uint32_t nk = 0, nv = 0, q0 = 0, q1 = 0, n_items = 0, n_q = 0;
        bool ok = true;
        const auto publish = [&](const Item& x) {
          if (n_items >= kItems)
            ok = wait(at(ctl.item_empty[n_items % kItems]), (n_items / kItems - 1) & 1);
          if (!ok) return;
          if (on) {
            ctl.item[n_items % kItems] = x;
            bar_arrive(at(ctl.item_full[n_items % kItems]));
          }
          ++n_items;
        };
        const auto load_q = [&](const Item& x, int i) {
          const int qb = PAIR ? i : (int)(n_q & 1);
          const uint32_t used = qb ? q1 : q0;  // the buffer's loads so far
          if (used > 0) ok = wait(at(ctl.q_empty[qb]), (used - 1) & 1);
          if (!ok) return;
          if (qb) ++q1; else ++q0;
          ++n_q;
          const uint32_t bar = at(ctl.q_full[qb]);
          bar_expect(bar, (DP / 64) * 128 * p.G * p.tile_tok, on);
          for (int half = 0; half < DP / 64; ++half)
            tma_load4(base + qb * SM::kQ + half * (kTile * 128), &p.q_map, half * 64, 0, x.h,
                      x.tok_at + x.tok0 + i * p.tile_tok, bar, on);
        };
        // In the order K0 V0 K1 V1 ...; a unit's queries before its first K.
        int j = 0, head = 0, v_row = 0, v_rows = 0;  // the V tile that is due (none: v_rows 0)
        bool fetch = true, step = true;  // the next unit is to be published; to be begun
#pragma unroll 1
        while (ok) {
          if (v_rows > 0) {
            if (nv >= SM::kV) ok = wait(at(ctl.v_empty[vr.slot]), vr.turn ^ 1);
            if (!ok) break;
            // a whole tile in one copy a half, else in boxes of 32 rows
            const uint32_t bar = at(ctl.v_full[vr.slot]);
            const uint32_t dst = base + SM::kVAt + vr.slot * SM::kSlot;
            const int boxes = (v_rows + 31) / 32, copies = boxes == 4 ? 1 : boxes;
            const CUtensorMap* const map = boxes == 4 ? &p.v_map : &p.v_part;
            bar_expect(bar, boxes * (DP / 64) * 4096, on);
#pragma unroll 1
            for (int x = 0; x < copies; ++x)
              for (int half = 0; half < DP / 64; ++half)
                tma_load3(dst + half * (kTile * 128) + x * 4096, map, half * 64, v_row + x * 32,
                          head, bar, on);
            vr.next();
            ++nv;
            v_rows = 0;
          }
          if (fetch) {  // ahead of need, under a unit's first loads: the next unit, SPLIT its queries
            walk.template next<PAIR>(&after);
            publish(after);
            if (!PAIR && ok && after.n > 0) load_q(after, 0);
            fetch = false;
          }
          if (step) {
            it = after;
            if (it.n == 0) break;
            j = 0;
            step = false;
            head = it.b * p.H + it.h;
            // (the row tiles' buffers are free once the unit before has used them up)
            if (PAIR)
#pragma unroll 1
              for (int i = 0; i < 2 && ok; ++i)
                if ((i ? it.nt1 : it.nt0) > 0) load_q(it, i);
          }
          if (!ok) break;
          const int row = (it.t0 + j) * kTile, rows = min(kTile, it.row_end - row);
          if (nk >= SM::kK) ok = wait(at(ctl.k_empty[kr.slot]), kr.turn ^ 1);
          if (!ok) break;
          const uint32_t bar = at(ctl.k_full[kr.slot]);
          const uint32_t dst = base + SM::kKAt + kr.slot * SM::kSlot;
          const int pad = p.C & 1;  // zeros for the other half of the last contraction step
          bar_expect(bar, p.C * rows * 16 + pad * (kTile * 16), on);
          if (rows == kTile) {
            tma_load4(dst, &p.k_map, 0, row / p.k_rows, 0, head, bar, on);
          } else {
            const uint4* src = p.k + (int64_t)head * p.C * p.S + row;
#pragma unroll 1
            for (int c = 0; c < p.C; ++c)
              bulk_load(dst + c * (kTile * 16), src + (int64_t)c * p.S, rows * 16, bar, on);
          }
          if (pad) bulk_load(dst + p.C * (kTile * 16), g_zero_rows, kTile * 16, bar, on);
          kr.next();
          ++nk;
          v_row = row;
          v_rows = rows;
          fetch = j == 0;
          step = ++j == it.n;
        }
        // No copy is left in flight, whichever warp gave up: nobody else may have waited for it.
#pragma unroll 1
        for (uint32_t i = 0; i < SM::kK && i < nk; ++i)  // a slot's last use
          bar_wait(at(ctl.k_full[i]), (nk - i - 1) / SM::kK & 1, kSpinLimit);
#pragma unroll 1
        for (uint32_t i = 0; i < SM::kV && i < nv; ++i)
          bar_wait(at(ctl.v_full[i]), (nv - i - 1) / SM::kV & 1, kSpinLimit);
        if (q0 > 0) bar_wait(at(ctl.q_full[0]), (q0 - 1) & 1, kSpinLimit);
        if (q1 > 0) bar_wait(at(ctl.q_full[1]), (q1 - 1) & 1, kSpinLimit);
      }
      __syncwarp();
    } else if (warp < 11) {
      // ---- products ----
      {
        const bool on = elect();
        constexpr uint32_t kType = std::is_same<T, __half>::value ? 0u : 1u;
        constexpr uint32_t kIdesc =
            1u << 4 | kType << 7 | kType << 10 | (uint32_t)(kTile >> 4) << 24;
        constexpr uint32_t kIdescS = kIdesc | (uint32_t)(kTile >> 3) << 17;
        constexpr uint32_t kIdescO = kIdesc | 1u << 16 | (uint32_t)(DP >> 3) << 17;
        const int i = warp - 9, steps = (p.C + 1) / 2;
        Ring<SM::kK> kr;
        Ring<SM::kV> vr;
        uint32_t n_items = 0, n_q = 0, p_count = 0;
        int other = 0;  // tiles of the other chain in the units before
        bool ok = true;
        Item it;
        while (ok && get_item(n_items, &it)) {
          const int n = __shfl_sync(~0u, it.n, 0), t0 = __shfl_sync(~0u, it.t0, 0);
          const int nt = __shfl_sync(~0u, i ? it.nt1 : it.nt0, 0), row_end = __shfl_sync(~0u, it.row_end, 0);
          const int masked = __shfl_sync(~0u, it.masked, 0);
          const int nt_other = __shfl_sync(~0u, i ? it.nt0 : it.nt1, 0);
          const int qb = PAIR ? i : (int)(n_items & 1);
          const uint32_t q_parity = (PAIR ? n_q : n_items >> 1) & 1;
          if (nt > 0) ++n_q;
          if (!PAIR && nt == 0) {  // (once the buffer's last turn is over for both chains)
            if (!(ok = wait(at(ctl.q_full[qb]), q_parity))) break;
            if (on) bar_arrive(at(ctl.q_empty[qb]));
          }
          const auto mine = [&](int j) { return PAIR ? j < nt : (j & 1) == i; };
          int jk = 0, jv = 0, k_mine = 0, v_mine = 0;
          // Both chains go through every K and V tile in order; one that is not the chain's is
          // let go.  Neither ring is followed past the other (V_j is loaded after K_j+1 and not
          // before K_j-1, V_j-1 are let go).
          // Up to the chain's next K tile: S = Q K^T into the chain's S columns.
          const auto next_k = [&]() {
#pragma unroll 1
            while (jk < n) {
              const bool own = mine(jk);
              if (!own && jk > jv + 1) break;
              if (!wait(at(ctl.k_full[kr.slot]), kr.turn)) return false;
              if (own) {
                if (k_mine == 0 && !wait(at(ctl.q_full[qb]), q_parity)) return false;
                if (PAIR && t0 + jk < masked) {
                  // The chains take turns: a chain's scores are computed once the other's softmax
                  // is at its exponentials, so that one's products run under the other's
                  // softmax (in step, both compete for the one and then for the other: 15% slower
                  // on long prompts).  No more than a preference: after some polls it goes on.
                  const int due = k_mine - 1 + i;  // the other chain's tile that comes before
                  if (due >= 0 && due < nt_other)
#pragma unroll 1
                    for (int w = 0; w < kTurnPolls && ctl.turn[i ^ 1] - other <= due; ++w) {
                    }
                }
                fence_after();
                const uint64_t qd = smem_desc(base + qb * SM::kQ, 0, 1024, 2);
                const uint64_t kd =
                    smem_desc(base + SM::kKAt + kr.slot * SM::kSlot, kTile * 16, 128, 0);
                const uint32_t s0 = tmem + i * kTile;
#pragma unroll
                for (int s = 0; s < DP / 16; ++s)
                  mma_ss(s0, qd + (s >> 2) * (kTile * 8) + (s & 3) * 2, kd + s * (2 * kTile),
                         kIdescS, s > 0, on && s < steps);
                mma_commit(at(ctl.s_full[i]), on);
                mma_commit(at(ctl.k_empty[kr.slot]), on);
                if (++k_mine == nt) mma_commit(at(ctl.q_empty[qb]), on);
              } else if (on) {
                bar_arrive(at(ctl.k_empty[kr.slot]));
              }
              kr.next();
              ++jk;
              if (own) break;
            }
            return true;
          };
          // Up to the chain's next V tile: O += P V.
          const auto next_v = [&]() {
#pragma unroll 1
            while (jv < jk) {
              const bool own = mine(jv);
              // (hidden rows have been looked at where the tile has any)
              if (!wait(at(own && t0 + jv >= masked ? ctl.v_ok[vr.slot] : ctl.v_full[vr.slot]),
                            vr.turn))
                return false;
              if (own) {
                const uint64_t vd =
                    smem_desc(base + SM::kVAt + vr.slot * SM::kSlot, kTile * 128, 1024, 2);
                const uint32_t o = tmem + 2 * kTile + i * kTile, s0 = tmem + i * kTile;
                const int rows = min(kTile, row_end - (t0 + jv) * kTile);
                const bool more = v_mine > 0;
                if (!wait(at(ctl.p_half[i]), p_count & 1)) return false;
                fence_after();
#pragma unroll
                for (int s = 0; s < kTile / 32; ++s)
                  mma_ts(o, s0 + s * 8, vd + s * 128, kIdescO, more || s > 0, on && s * 16 < rows);
                if (!wait(at(ctl.p_ready[i]), p_count & 1)) return false;
                fence_after();
#pragma unroll
                for (int s = kTile / 32; s < kTile / 16; ++s)
                  mma_ts(o, s0 + s * 8, vd + s * 128, kIdescO, true, on && s * 16 < rows);
                ++p_count;
                mma_commit(at(ctl.v_empty[vr.slot]), on);
                if (++v_mine == nt) mma_commit(at(ctl.o_done[i]), on);
              } else if (on) {
                bar_arrive(at(ctl.v_empty[vr.slot]));
              }
              vr.next();
              ++jv;
              if (own) break;
            }
            return true;
          };
#pragma unroll 1
          for (;;) {
            if (!(ok = next_k()) || jv == n) break;
            if (!(ok = next_v())) break;
          }
          if (on) bar_arrive(at(ctl.item_empty[n_items % kItems]));
          ++n_items;
          other += nt_other;
        }
        // the products in flight end before tensor memory is given back
        mma_commit(at(ctl.drained), on);
        bar_wait(at(ctl.drained), 0, kSpinLimit);
      }
      __syncwarp();
    } else {
      // ---- V's hidden rows: zero past the last attended one, finite elsewhere ----
      Ring<SM::kV> vr;
      Item it;
      bool ok = true;
      for (uint32_t k = 0; ok && get_item(k, &it); ++k) {
#pragma unroll 1
        for (int j = 0; j < it.n; ++j, vr.next()) {
          if (!(ok = wait(at(ctl.v_full[vr.slot]), vr.turn))) break;
          const int row0 = (it.t0 + j) * kTile;
          if (it.t0 + j >= it.masked) {
#pragma unroll 1
            for (int r = lane; r < kTile; r += 32) {
              uint4* const vrow = reinterpret_cast<uint4*>(sm + SM::kVAt + vr.slot * SM::kSlot + r * 128);
              if (row0 + r >= it.row_end) {
#pragma unroll
                for (int c = 0; c < DP / 8; ++c)
                  vrow[(c >> 3) * (kTile * 8) + ((c + r) & 7)] = make_uint4(0, 0, 0, 0);
              } else {
                // adding one to the exponent carries to the sign bit where it is all ones
                constexpr uint32_t one = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;
                uint32_t bad = 0;
#pragma unroll
                for (int c = 0; c < DP / 8; ++c) {
                  const uint4 u = vrow[(c >> 3) * (kTile * 8) + ((c + r) & 7)];
                  bad |= ((u.x & 0x7fff7fffu) + one) | ((u.y & 0x7fff7fffu) + one) |
                         ((u.z & 0x7fff7fffu) + one) | ((u.w & 0x7fff7fffu) + one);
                }
                if (bad & 0x80008000u) {
                  ctl.item[k % kItems].bad = 1;
                  uint16_t* const e = reinterpret_cast<uint16_t*>(vrow);
#pragma unroll 1
                  for (int c = 0; c < DP; ++c) {
                    uint16_t& y = e[(c >> 6) * (kTile * 64) + (c & 63)];
                    if (((y & 0x7fffu) + (one & 0xffffu)) & 0x8000u) y = 0;
                  }
                }
              }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          __syncwarp();
          if (lane == 0) {
            bar_arrive(at(ctl.v_ok[vr.slot]));
            bar_arrive(at(ctl.v_empty[vr.slot]));
          }
        }
        if (lane == 0) bar_arrive(at(ctl.item_empty[k % kItems]));
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ---- softmax: a chain's warpgroup, a thread per row ----
    const int i = warp >> 2, r = threadIdx.x & (kTile - 1);
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // the warp's 32 lanes of tensor memory
    const uint32_t ts = tmem + lanes + i * kTile, to = tmem + lanes + 2 * kTile;
    const int tr = r / p.G, g = r - tr * p.G;
    uint32_t s_count = 0, o_count = 0, item = 0;
    bool ok = true;
    Item it;
    for (; ok && get_item(item, &it); ++item) {
      const int tile_tok0 = it.tok0 + (PAIR ? i * p.tile_tok : 0);
      const int tok = tile_tok0 + tr, nt = i ? it.nt1 : it.nt0;
      const bool valid = tr < p.tile_tok && tok < it.n_tok;
      const bool any_valid = __any_sync(~0u, valid);
      uint64_t bits = 1;  // (a prompt's token attends itself)
      if (p.is_tree && valid) {
        bits = p.tree ? __ldg(p.tree + it.tok_at + tok) : (2ull << tok) - 1;
        if (it.n_tok < 64) bits &= (1ull << it.n_tok) - 1;
      }
      // the first tile that hides a column from some row of the chain's tile
      const int masked = p.is_tree ? it.masked : (it.start + tile_tok0 + 1) / kTile;
      if (!PAIR && item > 0) {  // the other chain has read this chain's last O
        const uint32_t w = item - 1;
        if (!(ok = wait(at(ctl.o_read[w & 1]), w >> 1 & 1))) break;
      }
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int j = 0; j < nt; ++j) {
        const int tile = it.t0 + (PAIR ? j : 2 * j + i);
        if (!(ok = wait(at(ctl.s_full[i]), s_count & 1))) break;
        ++s_count;
        fence_after();
        uint32_t x[kTile];
        // Half of the row: p = 2^kUp exp2(c (s - m)), to tensor memory; gives its sum.
        const auto half_row = [&](int half) {
          constexpr float kUp = std::is_same<T, __half>::value ? kHalfUp : 0.f;
          const float mb = m == -INFINITY ? kUp : fmaf(-m, p.c, kUp);
          float sum[4] = {};
#pragma unroll
          for (int k = 2 * half; k < 2 * half + 2; ++k) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float a = __uint_as_float(x[32 * k + 2 * e]);
              float b = __uint_as_float(x[32 * k + 2 * e + 1]);
              fma2(a, b, p.c, mb);
              a = ex2(a);
              b = ex2(b);
              add2(sum[2 * (e & 1)], sum[2 * (e & 1) + 1], a, b);
              w[e] = Pack2<T>::pack(a, b);
            }
            tmem_st16(ts + 16 * k, w);
          }
          return (sum[0] + sum[1]) + (sum[2] + sum[3]);
        };
        if (any_valid) {
          // Hidden columns are set to -inf in tensor memory, 32 at a time and only where the
          // warp has some: a small loop beside the tile's long straight code.
          if (tile >= masked) {
#pragma unroll 1
            for (int k = 0; k < kTile; k += 32) {
              const int col = tile * kTile + k;
              const uint32_t w = p.is_tree ? tree_mask(bits, col - it.start)
                                           : causal_mask(it.start + tok - col);
              if (__all_sync(~0u, w == ~0u)) continue;
              uint32_t y[32];
              tmem_ld32(y, ts + k);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(w & (1u << e))) y[e] = 0xff800000u;
              tmem_st32(ts + k, y);
            }
            tmem_wait_st();
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) tmem_ld32(x + 32 * k, ts + 32 * k);
          tmem_wait_ld();
          const auto row_max = [&]() {
            float mx[4] = {m, m, m, m};
#pragma unroll
            for (int k = 0; k < kTile; k += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                mx[e] = fmaxf(fmaxf(mx[e], __uint_as_float(x[k + 2 * e])),
                              __uint_as_float(x[k + 2 * e + 1]));
            return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          };
          // Takes m_new as the reference where some row of the warp has grown past it by 2^kLazy.
          const auto move_max = [&](float m_new) {
            if (!__any_sync(~0u, valid && (m_new - m) * p.c > kLazy)) return;
            const float f = m == -INFINITY ? 0.f : ex2((m - m_new) * p.c);
            m = m_new;
            l *= f;
            if (j > 0) {
#pragma unroll 1
              for (int k = 0; k < DP; k += 16) {
                uint32_t o[16];
                tmem_ld16(o, to + i * kTile + k);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st16(to + i * kTile + k, o);
              }
            }
          };
          move_max(row_max());
          if (PAIR && r == 0) ctl.turn[i] = (int)s_count;
          l += half_row(0);
          tmem_wait_st();
        }
        fence_before();
        bar_arrive(at(ctl.p_half[i]));
        if (any_valid) {
          l += half_row(1);
          tmem_wait_st();
        }
        fence_before();
        bar_arrive(at(ctl.p_ready[i]));
      }
      if (!ok) break;
      if (nt > 0) {
        if (!(ok = wait(at(ctl.o_done[i]), o_count & 1))) break;
        ++o_count;
        fence_after();
      }
      float w0 = 1.f, w1 = 0.f;  // SPLIT: the chains' weights
      if (!PAIR) {
        ctl.ml[i][r] = make_float2(m, l);
        fence_before();
        bar_arrive(at(ctl.xchg));
        if (!(ok = wait(at(ctl.xchg), item & 1))) break;
        fence_after();  // the other chain's O has been waited for by its own threads
        const float2 a = ctl.ml[0][r], b = ctl.ml[1][r];
        m = fmaxf(a.x, b.x);
        w0 = a.x == -INFINITY ? 0.f : ex2((a.x - m) * p.c);
        w1 = b.x == -INFINITY ? 0.f : ex2((b.x - m) * p.c);
        l = a.y * w0 + b.y * w1;
      }
      // ---- the piece's output: SPLIT each chain half of the columns ----
      if (any_valid) {
        const bool whole = it.whole != 0;
        // A row that attends nothing gives zeros.  One whose every attended score is -inf has
        // l = 0 too: 0 x inf, NaN, as its softmax is.
        const float inv = !whole ? 1.f : it.start == 0 && bits == 0 ? 0.f : 1.f / l;
        constexpr int kCols = PAIR ? DP : DP / 2;
        const int c0 = PAIR ? 0 : i * kCols;
        // slot 0: the CTA's first piece, 1: its last
        constexpr int kRows = PAIR ? 2 * kTile : kTile;
        float* const part =
            p.part + (int64_t)(blockIdx.x * 2 + (item == 0 ? 0 : 1)) * kRows * (p.D + 2);
        const int prow = (PAIR ? i * kTile : 0) + r;
        uint16_t* const out = p.out + (int64_t)(it.tok_at + tok) * p.out_stride +
                              (int64_t)(it.h * p.G + g) * p.D;
        if (!whole && valid && (PAIR || i == 0))
          reinterpret_cast<float2*>(part + kRows * p.D)[prow] = make_float2(m * p.c, l);
#pragma unroll 1
        for (int k = c0; k < c0 + kCols; k += 32) {
          if (k >= p.D) break;
          uint32_t o[32];
          if ((PAIR ? nt : it.nt0) > 0) {
            tmem_ld32(o, to + (PAIR ? i * kTile : 0) + k);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0;
          }
          if (!PAIR) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = __float_as_uint(__uint_as_float(o[e]) * w0);
            if (it.nt1 > 0) {
              uint32_t o1[32];
              tmem_ld32(o1, to + kTile + k);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e)
                o[e] = __float_as_uint(
                    fmaf(__uint_as_float(o1[e]), w1, __uint_as_float(o[e])));
            }
          }
          if (valid) {
            if (whole) {
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e)
                w[e] = Pack2<T>::pack(__uint_as_float(o[2 * e]) * inv,
                                      __uint_as_float(o[2 * e + 1]) * inv);
              if (p.wide) {  // rows of whole, aligned 32-byte sectors: half the store requests
#pragma unroll
                for (int e = 0; e < 16; e += 8)
                  if (k + 2 * e < p.D) st32(out + k + 2 * e, w + e);
              } else {
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                  if (k + 2 * e < p.D)
                    *reinterpret_cast<uint4*>(out + k + 2 * e) =
                        make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
              }
            } else {
              float* const d = part + (int64_t)prow * p.D + k;
#pragma unroll
              for (int e = 0; e < 32; e += 8)
                if (k + e < p.D) st32(d + e, o + e);
            }
          }
        }
      }
      fence_before();
      if (!PAIR) bar_arrive(at(ctl.o_read[item & 1]));
      if (valid && ctl.item[item % kItems].bad != 0) {
        // Rare: the non-finite values taken out of V that the row does attend are added to
        // what it has just written.
        constexpr int kCols = PAIR ? DP : DP / 2;
        const int c0 = PAIR ? 0 : i * kCols, c1 = min(p.D, c0 + kCols);
        const uint16_t* const v = p.v + ((int64_t)it.b * p.H + it.h) * p.S * (int64_t)p.D;
        uint32_t* const out = reinterpret_cast<uint32_t*>(
            p.out + (int64_t)(it.tok_at + tok) * p.out_stride + (int64_t)(it.h * p.G + g) * p.D);
        constexpr int kRows = PAIR ? 2 * kTile : kTile;
        float* const part =
            p.part + (int64_t)(blockIdx.x * 2 + (item == 0 ? 0 : 1)) * kRows * (p.D + 2) +
            (int64_t)((PAIR ? i * kTile : 0) + r) * p.D;
        const int row1 = min(it.row_end, (it.t0 + it.n) * kTile);
#pragma unroll 1
        for (int row = max(it.masked, it.t0) * kTile; row < row1; ++row) {
          if (row >= it.start &&
              !(p.is_tree ? (bits >> (row - it.start) & 1) != 0 : row <= it.start + tok))
            continue;
#pragma unroll 1
          for (int c = c0; c < c1; c += 2) {
            float2 f = Pack2<T>::unpack(
                *reinterpret_cast<const uint32_t*>(v + (int64_t)row * p.D + c));
            if (isfinite(f.x) && isfinite(f.y)) continue;
            f.x = isfinite(f.x) ? 0.f : f.x;
            f.y = isfinite(f.y) ? 0.f : f.y;
            if (it.whole) {
              const float2 o = Pack2<T>::unpack(out[c / 2]);
              out[c / 2] = Pack2<T>::pack(o.x + f.x, o.y + f.y);
            } else {
              part[c] += f.x;
              part[c + 1] += f.y;
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) bar_arrive(at(ctl.item_empty[item % kItems]));
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 8)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
}

// ---- the join ----------------------------------------------------------------------

struct JoinParams {
  uint16_t* out;
  const float* part;
  const Divided* divided;
  int64_t out_stride;
  int32_t G, D, tile_tok, rows;  // rows: of a piece's slot
};

// Adds up the pieces of the unit that the cut after CTA blockIdx.x is the
// first to divide:
//   out = sum_i f_i O_i / sum_i f_i l_i,  f_i = exp2(m_i - max m).
// Bound by latency (a launch of a few microseconds): a thread per 4 output
// values, with no load waiting for another but for the unit's description.
template <typename T>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(const __grid_constant__ JoinParams p) {
  ops_pdl_enter();
  const int i0 = blockIdx.x;
  const Divided d = p.divided[i0];
  const int d4 = p.D / 4, n = d.tokens * p.G * d4, pieces = d.last - i0 + 1;
  const int64_t slot = (int64_t)p.rows * (p.D + 2);
  const auto piece = [&](int i) { return p.part + slot * (2 * (i0 + i) + (i == 0 ? d.slot : 0)); };
#pragma unroll 1
  for (int e = blockIdx.y * kJoinThreads + threadIdx.x; e < n; e += gridDim.y * kJoinThreads) {
    const int q = e / d4, c = e - q * d4;
    const int tok = q / p.G, g = q - tok * p.G;
    const int tile = tok / p.tile_tok;
    const int r = tile * kTile + (tok - tile * p.tile_tok) * p.G + g;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int i = 0; i < pieces; i += 4) {
      float2 ml[4];
      float4 a[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
        if (i + k < pieces) {
          const float* const pc = piece(i + k);
          ml[k] = reinterpret_cast<const float2*>(pc + (int64_t)p.rows * p.D)[r];
          a[k] = reinterpret_cast<const float4*>(pc + (int64_t)r * p.D)[c];
        }
      }
      const float m_new = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), m);
      const float f0 = m == -INFINITY ? 0.f : ex2(m - m_new);
      m = m_new;
      l *= f0;
      o = make_float4(o.x * f0, o.y * f0, o.z * f0, o.w * f0);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k < pieces) {  // (a piece of NaN scores alone has m = -inf and l = NaN)
          const float f = ml[k].x == -INFINITY ? 0.f : ex2(ml[k].x - m);
          l += f * ml[k].y;
          o.x += f * a[k].x;
          o.y += f * a[k].y;
          o.z += f * a[k].z;
          o.w += f * a[k].w;
        }
    }
    // Some row is attended (a token that attends none has at most 64 rows, one tile, which no
    // cut divides): l = 0 means scores of -inf alone, NaN.
    const float inv = 1.f / l;
    uint16_t* const out =
        p.out + (int64_t)(d.tok + tok) * p.out_stride + (int64_t)(d.head + g) * p.D;
    reinterpret_cast<uint2*>(out)[c] =
        make_uint2(Pack2<T>::pack(o.x * inv, o.y * inv), Pack2<T>::pack(o.z * inv, o.w * inv));
  }
}

// ---- host ---------------------------------------------------------------------------

// How a call is cut into units and CTAs.
struct Schedule {
  bool pair;
  int tile_tok, unit_tok;
  int64_t total;  // cost: tiles, and unit_cost for each unit
  int unit_cost;
  int64_t units;
  int ctas;
  size_t part_bytes, bytes;  // of workspace: the pieces' sums, all
};

std::atomic<uint32_t> g_tries{kSpinLimit};

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    n = 152;
  }
  return n;
}

// A CTA's share is not cut below this many tiles, one for each chain, where
// there are fewer units than SMs: a finer cut gains nothing that the join does
// not take (one sequence's decode step over 1000 rows, 8 key heads: 8.7 us at 2
// and at 1, 10.5 at 4, 12.3 at 8; over 2000: 9.3, 9.8, 10.3, 13.5).
constexpr int kMinTiles = 2;
// What a unit costs besides its tiles (fetching its queries, filling and
// draining the two chains, its output), in tiles: without it CTAs with many
// short sequences took twice as long as the others (decode of a ragged batch:
// 346 us at 0, 252 at 1, 232 at 2, 246 at 5; ragged prompts: 902 at 0, 823 at 1,
// 814 at 2, 828 at 3, where prompts of 1000 take 57, 53, 55, 55).
constexpr int kUnitCostPair = 1, kUnitCostSplit = 2;

Schedule schedule(const Plan& p, int group, bool is_tree, int32_t* cost_pre) {
  Schedule s;
  s.tile_tok = kTile / group;
  s.pair = p.max_len > s.tile_tok;
  s.unit_tok = s.tile_tok * (s.pair ? 2 : 1);
  s.unit_cost = s.pair ? kUnitCostPair : kUnitCostSplit;
  s.total = s.units = 0;
  int64_t all_tiles = 0;
  for (int b = 0; b < p.B; ++b) {
    if (cost_pre) cost_pre[b] = (int32_t)s.total;
    const int n = p.seq_len[b], first = p.seq_start[b];
    int64_t tiles = 0;
    for (int64_t u = 0; u < n; u += s.unit_tok) {
      const int64_t rows = first + (is_tree || u + s.unit_tok > n ? n : u + s.unit_tok);
      tiles += (rows + kTile - 1) / kTile;
      s.total += (int64_t)s.unit_cost * p.H;
      s.units += p.H;
    }
    s.total += tiles * p.H;
    all_tiles += tiles * p.H;
  }
  if (cost_pre) cost_pre[p.B] = (int32_t)s.total;
  const int64_t sms = sm_count();
  int64_t ctas = all_tiles / kMinTiles;
  if (ctas < s.units) ctas = s.units;
  if (ctas > sms) ctas = sms;
  if (ctas < 1) ctas = 1;
  s.ctas = (int)ctas;
  s.part_bytes = (size_t)ctas * 2 * (s.pair ? 2 : 1) * kTile * (p.D + 2) * sizeof(float);
  s.bytes = ctas > 1 ? s.part_bytes + (size_t)ctas * sizeof(Divided) : 0;
  return s;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

bool encode(CUtensorMap* map, bool fp16, int rank, const void* base, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box, bool swizzle) {
  static const EncodeFn fn = reinterpret_cast<EncodeFn>(driver_fn("cuTensorMapEncodeTiled"));
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return fn && fn(map, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                  (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
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
  const Schedule s = schedule(p, group, is_tree, kp.cost_pre);
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
  const cuuint32_t vb[3] = {64, kTile, 1}, vp[3] = {64, 32, 1};
  // A chunk row's S rows of 16 bytes are one run, so the copy's innermost run may be several
  // rows: as many as divide S, up to the 256 elements a box may have: 512 bytes where 32 divide
  // it, 16 for an odd S.  (2048 tokens after 14336, 64 query heads on 8, with S a multiple of 32,
  // of 8, of 2, odd: 616, 617, 631, 661 us; a decode step of 16 x 16384 rows: 155, 156, 161, 185.)
  int w = 32;
  while (p.S % w != 0) w /= 2;
  kp.k_rows = w;
  const cuuint64_t kd[4] = {8 * (cuuint64_t)w, (cuuint64_t)p.S / w, (cuuint64_t)p.C,
                            (cuuint64_t)p.B * p.H};
  const cuuint64_t ks[3] = {16 * (cuuint64_t)w, 16 * (cuuint64_t)p.S, 16 * (cuuint64_t)p.S * p.C};
  const cuuint32_t kb[4] = {8 * (cuuint32_t)w, (cuuint32_t)(kTile / w), (cuuint32_t)p.C, 1};
  if (!encode(&kp.q_map, fp16, 4, q.q, qd, qs, qb, true) ||
      !encode(&kp.k_map, fp16, 4, k, kd, ks, kb, false) ||
      !encode(&kp.v_map, fp16, 3, v, vd, vs, vb, true) ||
      !encode(&kp.v_part, fp16, 3, v, vd, vs, vp, true))
    return fail(DV_ERR_CUDA, "cuTensorMapEncodeTiled refused the queries or the cache");
  kp.out = static_cast<uint16_t*>(q.out);
  kp.k = static_cast<const uint4*>(k);
  kp.v = static_cast<const uint16_t*>(v);
  kp.tree = tree;
  kp.part = part;
  kp.divided = reinterpret_cast<Divided*>(reinterpret_cast<uint8_t*>(part) + s.part_bytes);
  kp.out_stride = q.out_stride;
  kp.share = (int32_t)(s.total / s.ctas);
  kp.extra = (int32_t)(s.total % s.ctas);
  kp.H = p.H;
  kp.G = group;
  kp.D = p.D;
  kp.C = p.C;
  kp.S = p.S;
  kp.tile_tok = s.tile_tok;
  kp.unit_tok = s.unit_tok;
  kp.unit_cost = s.unit_cost;
  kp.is_tree = is_tree ? 1 : 0;
  kp.wide = p.D % 16 == 0 && q.out_stride % 16 == 0 && reinterpret_cast<uintptr_t>(q.out) % 32 == 0;
  kp.c = q.scale * 1.4426950408889634f;
  kp.tries = g_tries.load(std::memory_order_relaxed);
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
    JoinParams jp;
    jp.out = kp.out;
    jp.part = part;
    jp.divided = kp.divided;
    jp.out_stride = kp.out_stride;
    jp.G = group;
    jp.D = p.D;
    jp.tile_tok = s.tile_tok;
    jp.rows = (s.pair ? 2 : 1) * kTile;
    const int unit = (s.unit_tok < p.max_len ? s.unit_tok : p.max_len) * group * (p.D / 4);
    err = ops_launch(join_kernel<T>, dim3((unsigned)s.ctas - 1, (unit + kJoinThreads - 1) / kJoinThreads),
                     kJoinThreads, 0, stream, jp);
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
  if (q.tokens != p.tokens)
    return fail(DV_ERR_INVALID_ARG, "q and out hold %lld tokens, the ranges %lld",
                (long long)q.tokens, (long long)p.tokens);
  if (p.tokens == 0) return DV_OK;
  const Schedule sch = schedule(p, q.q_heads / p.H, is_tree, nullptr);
  const size_t need = sch.bytes;
  if (sch.total > INT32_MAX)
    return fail(DV_ERR_UNSUPPORTED, "%lld tiles of attention in one call", (long long)sch.total);
  if (workspace_bytes < need)
    return fail(DV_ERR_BUFFER_TOO_SMALL, "attention needs %zu workspace bytes (got %zu)", need,
                workspace_bytes);
  // What the call writes (out and the workspace) shares no bytes with what it reads.
  size_t nq = 0, no = 0;
  const size_t nt = (size_t)p.tokens * 8;
  if ((st = span_rows(p, q.q_heads, q.q_stride, "q", &nq)) != DV_OK) return st;
  if ((st = span_rows(p, q.q_heads, q.out_stride, "out", &no)) != DV_OK) return st;
  if (overlap(q.out, no, q.q, nq) || overlap(q.out, no, tree, nt) || overlaps_layers(p, q.out, no))
    return fail(DV_ERR_INVALID_ARG, "out overlaps q, tree or the cache's layer");
  if (need > 0 &&
      (overlap(workspace, need, q.q, nq) || overlap(workspace, need, q.out, no) ||
       overlap(workspace, need, tree, nt) || overlaps_layers(p, workspace, need)))
    return fail(DV_ERR_INVALID_ARG, "workspace overlaps q, out, tree or the cache's layer");
  if ((st = resolve_layers(&p)) != DV_OK) return st;
  void* dev = nullptr;
  if ((st = resolve_words(q.q, nq, 16, "q", &dev)) != DV_OK) return st;
  q.q = dev;
  if ((st = resolve_words(q.out, no, 16, "out", &dev)) != DV_OK) return st;
  q.out = dev;
  if (tree) {
    if ((st = resolve_words(tree, nt, 8, "tree", &dev)) != DV_OK) return st;
    tree = static_cast<const uint64_t*>(dev);
  }
  float* part = nullptr;
  if (need > 0) {
    if ((st = resolve_words(workspace, need, 32, "workspace", &dev)) != DV_OK) return st;
    part = static_cast<float*>(dev);
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

extern "C" dv_status dv_debug_attention_tries(int32_t tries) {
  if (tries > (int32_t)dv::kSpinLimit)
    return dv::fail(DV_ERR_INVALID_ARG, "%d tries are more than %u", tries, dv::kSpinLimit);
  dv::g_tries.store(tries < 0 ? dv::kSpinLimit : (uint32_t)tries, std::memory_order_relaxed);
  return DV_OK;
}

namespace {

// The count of waits that gave up as a stream's last check found it; streams without an entry
// have found none.
struct Checked {
  unsigned long long context, stream, count;
};

// Whether `count` is news to the stream; remembers it.
bool count_is_new(unsigned long long context, unsigned long long stream, unsigned long long count) {
  static std::mutex mu;
  static std::vector<Checked> checked;
  if (count == 0) return false;
  std::lock_guard<std::mutex> lock(mu);
  for (Checked& c : checked)
    if (c.context == context && c.stream == stream) {
      const bool news = c.count != count;
      c.count = count;
      return news;
    }
  try {
    checked.push_back({context, stream, count});
  } catch (...) {  // reported again by the next check
  }
  return true;
}

}  // namespace

extern "C" dv_status dv_attention_check(dv_stream stream) {
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  cudaError_t err = cudaStreamIsCapturing(stream, &capture);
  if (err == cudaSuccess && capture != cudaStreamCaptureStatusNone)
    return dv::fail(DV_ERR_INVALID_ARG, "dv_attention_check waits for its stream, which is being "
                    "captured into a graph");
  void* counter = nullptr;
  unsigned long long id = 0, context = 0, count = 0;
  if (err == cudaSuccess) err = cudaStreamGetId(stream, &id);
  if (err == cudaSuccess) err = cudaGetSymbolAddress(&counter, dv::g_attention_gave_up);
  if (err == cudaSuccess)
    err = cudaMemcpyAsync(&count, counter, sizeof(count), cudaMemcpyDeviceToHost, stream);
  if (err == cudaSuccess) err = cudaStreamSynchronize(stream);
  if (err != cudaSuccess) return dv::cuda_fail(err, "reading the attention kernels' count");
  dv::context_id(&context);
  if (count_is_new(context, id, count))
    return dv::fail(DV_ERR_TIMEOUT, "an attention kernel gave up a wait; its output is not valid");
  return DV_OK;
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

// Attention of a chunk of new tokens over a paged cache: the BF16-only pages (oscar_bf16_chunk), and
// the pool's mixed cache before the step's append (oscar_chunk_attend).
//
//   out[t, h] = sum_s softmax_s(q[t, h] . k[s] / sqrt(128)) v[s],  s over the keys token t sees
//
// One pass over the keys with the running maximum and sum of the softmax in base 2. Both products
// run on the tensor cores (tcgen05, fp32 accumulators in tensor memory):
//   S = Q K^T    Q [128 rows x 128] and K [128 keys x 128] in shared memory, K-major
//   O += P V     P [128 rows x 128 keys] from tensor memory, V [128 keys x 128] in shared memory
// A tile's 128 rows are 128/hg tokens x the hg query heads of one KV head, so all of them share
// every K and V block. A CTA works on two tiles at once: while one tile's 128 threads (a thread per
// row) turn S into P, the tensor cores run the other tile's products.
//
// Keys come in blocks of 128 (two half blocks of 64, each a page or a run of rows):
//   pages of the BF16 cache, the pool's sink page and ring pages   tensor copies of a page's two 64-dim
//       halves: the page's own swizzle (chunk c of token t at c ^ (t & 7)) is the 128-byte swizzle the
//       tensor cores read, so a page is used as it lies
//   the chunk's own rows (pool)       tensor copies with the 128-byte swizzle
//   INT2 history (pool)               as fp16 tiles of the same layout: four warps turn the codes into them
//       (mode kDequant), or, where several pairs of tiles go over a history, chunk_tiles.cu has made them
//       before and bulk copies bring them in (mode kTiles)
// The INT2 blocks come first. For them Q is rotated on the tensor cores (Q R_K, R in two bf16 limbs)
// and kept as fp16 with a power of two per row, k^ and v^ = fp16(level * s + z) and P are fp16, and
// O is in the rotated basis: behind the last INT2 block it is split into two bf16 limbs and
// multiplied by R_V^T in place (three products), and the BF16 blocks follow with the plain Q.
//
// Roundings to fewer bits. Weights enter the value product as one bf16 (BF16 keys) or one fp16 (INT2 keys), q R_K, k^ and
// v^ as one fp16, where the decode kernels keep weights and q R_K in two halves (hi + lo, 16 and 22 bits) and
// the codes exact; maxima, sums and O are fp32 in both. A second half would add half as many products again to a loop
// that they bound, for outputs that are rounded to bf16 anyway (the decode's are fp32). Relative error of whole outputs against
// 64 bits: 0.0017 from that last rounding alone, 0.0020 to 0.0024 with the weights over BF16 keys, 0.0019 over INT2
// keys.
//
// Work: the key blocks of the items (sequence, KV head, pair of tiles), counted by what they cost. The
// whole call is one range, cut into equal parts for the CTAs; an item cut by a boundary leaves one
// partial (maximum, sum, unnormalised O) per part, and a second kernel joins them. This keeps every
// SM busy for one long sequence with few rows as for a ragged batch, and needs nothing from the host:
// lengths are read on the device, so a captured call follows them.
//
// What bounds it. 128 keys cost the two tiles 2048 cycles of products and take 2670: work issued ahead
// keeps the tensor cores busy over gaps of 180 cycles only, a wait costs 60, and a tile's own chain (its
// products, 1024; the softmax, 1240; the signals between them, 200) is longer than its turn. Not the
// copies (half of their bytes left out change nothing) and not shared memory (products alone run at
// their full rate beside them). Beside that an item costs 6000 cycles a tile for queries, masked blocks
// and output. With codes dequantised in the kernel a block takes 3800 cycles, the expansion.
// Measured (GB300, 32 query and 8 KV heads unless said; products counted for visible keys only), replayed from a graph ten
// at a time, and in calls one after another, which draw the clock down:
//   8192 new tokens                             369 us, 1490 TFLOP/s; 393 a call
//   1024 new after 64K, 64 query heads          1358 us, 1630 TFLOP/s; 1540 to 1680 a call (the power limit's clock)
//   12 sequences of 1 to 257 after up to 8K     142 us; 157 a call
//   16 sequences of 4 after 1K to 32K           175 us, 6700 GB/s: memory bound, 99% of the copy peak; 181 a call
//   pool, 2048 new after 30000 of INT2          705 us, 1480 TFLOP/s, of it 21 us for the tiles; 775 a call
//   pool, 10 of 1 to 300 after up to 6K, 64 query heads, group 32      259 us, of it 23 us for the tiles; 264 a call
//
// Keys no row may see, and what lies behind a sequence's last key, must not reach a sum even as 0 *
// NaN: such values are zeroed in shared memory before the product. Where some rows of the tile see
// a key and others do not (the diagonal), a non-finite value element is zeroed too, noted, and added
// at the end to the rows that do see it.
#include <atomic>
#include <cstring>
#include <type_traits>

#include "int2_tiles.cuh"
#include "tcgen05.cuh"

namespace oscar {
namespace {

// The BF16-only cache; the pool with INT2 blocks dequantised in the kernel; the pool with their fp16
// tiles made beforehand.
enum { kBf16 = 0, kDequant = 1, kTiles = 2 };

constexpr int kTile = 128;                    // rows of a tile, keys of a block
constexpr int kHalfBytes = kTile * 128;       // 64 dims of 128 rows
constexpr int kTileBytes = 2 * kHalfBytes;    // 128 x 128 16-bit values
template <int MODE>
constexpr int kStages = MODE == kDequant ? 4 : 5;  // K / V tiles in flight
constexpr int kCodeBuf = 3 * 2 * int2_block_bytes(128);  // packed INT2 pages in flight: three blocks (two of groups of 32)
constexpr int kMaxSlots = 3;
constexpr int kMaxCtas = 152;
constexpr int kPageHalfBytes = kPage * 128;   // 64 dims of one page
constexpr float kGrown = 60000.f;             // a block's weights under an old maximum: fp16 holds each of them
// The reference of INT2 scores is set 4 (in powers of two) below their maximum: the largest weight is 2^4, fp16 weights keep their 11
// bits down to 2^-18 of it and are off by 2^-29 of it at most below that, half a step of a bf16 output for 2^20 such keys. With the
// largest at 1 they vanish at 2^-25: 0.3% of the output for a flat history of 130 thousand tokens under one strong key. More
// headroom means more renewals: 2048 after 30000 takes 768 us a call with 4, 771 with 5, 790 with 8 (766 with 0).
constexpr float kHeadroom = 4.f;
constexpr int kDescBytes = 32;
// Work is counted in thousands of SM cycles, as measured on batches of equal items (G = 128, hg = 4):
// a block of BF16 keys takes 3, one of INT2 keys 4; an item takes another 6 a tile (queries in, first
// and masked blocks, output out), and 8 more a tile for its two rotations. Where the fp16 tiles are made
// beforehand the rotations weigh twice as much beside the faster blocks: with 16 the ragged batch of 10
// takes 259 us for 282 with 8, others 0.93 to 1.01 of the time (24 gives 260, and 0.94 to 1.08).
constexpr int kUnitsBf16 = 3, kUnitsInt2 = 4, kUnitsTile = 6, kUnitsRotate = 8, kUnitsRotateTiles = 16;
constexpr int kMinUnits = 4;  // per CTA, at least: a block and a little (64 tokens after 500: 28 us at 12, 20 at 3 to 6)

constexpr uint32_t kIdescBase = (1u << 4) | ((uint32_t)(kTile >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
constexpr uint32_t kIdescBf16 = kIdescBase | (1u << 7) | (1u << 10);  // A, B bf16; fp16 without these bits
constexpr uint32_t kIdescMn = 1u << 16;                               // B with its N axis contiguous

// Lower descriptor words of 128-byte-swizzled tiles: K-major (row r of a 64-dim half at r * 128), and
// the same bytes read with the other axis contiguous (leading offset: the next 64 of N).
__device__ __forceinline__ uint32_t desc_k(uint32_t a) { return (a >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t a) { return (a >> 4) | ((uint32_t)(kHalfBytes >> 4) << 16); }

struct ChunkArgs {
  int32_t Hq, Hkv, hg, lg, n_seqs, n_tokens, rows;  // lg: log2 of a tile pair's tokens; rows: of a partial slot
  int32_t wide;                                 // out starts on a 32-byte boundary
  // BF16-only cache
  const int32_t *page_table, *lengths, *cu;
  const uint8_t* v_pages;
  int32_t max_pages;
  int64_t n_pages_total;
  // pool
  DevPool P;
  int32_t layer, skip_single;
  const __nv_bfloat16* v_new;
  // the history's fp16 tiles (mode kTiles): of sequence i from block tile_base[i] on, [KV head][block][K, V]
  const uint8_t* tiles;
  const int32_t* tile_base;
  __nv_bfloat16* out;
  uint8_t* ws;
  uint32_t* err;
};

struct ChunkMaps {
  CUtensorMap q, k, v;            // k, v: pages of the BF16 cache, or the chunk's rows (pool)
  CUtensorMap sink_k, sink_v, ring_k, ring_v;
};

struct Part {                     // what a CTA's first boundary cuts (one per CTA; parts 0: nothing)
  int32_t parts, row0, rows, head;  // parts of the item, its first q row (token), rows, first query head
  int32_t pad[4];
};
static_assert(sizeof(Part) == kDescBytes, "Part");

// One sequence's work: n new tokens; token t sees `pre` leading blocks and A + t + 1 keys of the
// causal ones.
struct SeqWork {
  int32_t n, A, row0;
  int32_t nI, nB;                 // INT2 blocks, blocks of cached BF16 pages (pool)
  int32_t hist, F, L, sink, seq;  // pool: history tokens, frontier and length before the step
  int32_t tile0;                  // first block of its tiles
  int32_t rotate;                 // units of a tile's two rotations
};

template <int MODE>
__device__ __forceinline__ SeqWork load_seq(const ChunkArgs& C, int i) {
  SeqWork s{};
  if constexpr (MODE != kBf16) {
    const StepSeq& st = C.P.step[i];
    s.n = st.L_new - st.L_old;
    if (C.skip_single && s.n == 1) s.n = 0;
    s.row0 = st.in_offset;
    s.F = st.F_old;
    s.L = st.L_old;
    s.sink = st.sink_page;
    s.seq = st.seq_id;
    s.hist = s.F - kSink;
    s.nI = (s.hist + kTile - 1) / kTile;
    // the sink page, then the ring pages of positions [F, L)
    const int ring = s.L > s.F ? ((s.L - 1) >> 6) - (s.F >> 6) + 1 : 0;
    s.nB = s.L > 0 ? (1 + ring + 1) / 2 : 0;
    s.A = 0;
    if (MODE == kTiles) s.tile0 = C.tile_base[i];
    s.rotate = s.nI <= 0 ? 0 : MODE == kTiles ? kUnitsRotateTiles : kUnitsRotate;
  } else {
    const int a = min(max(C.cu[i], 0), C.n_tokens), b = min(max(C.cu[i + 1], a), C.n_tokens);
    int len = max(C.lengths[i], 0);
    if (len > C.max_pages * kPage) {
      set_err(C.err, OSCAR_DEVERR_PAGE);
      len = C.max_pages * kPage;
    }
    s.n = b - a;
    s.row0 = a;
    s.A = len - s.n;
  }
  return s;
}

// Key blocks that tile pair t of a sequence really has.
__device__ __forceinline__ int real_blocks(const SeqWork& s, int lg, int t) {
  const int keys = s.A + min(s.n, (t + 1) << lg);
  return s.nI + s.nB + (keys > 0 ? (keys + kTile - 1) / kTile : 0);
}

__device__ __forceinline__ int pairs_of(const SeqWork& s, int lg) { return (s.n + (1 << lg) - 1) >> lg; }
__device__ __forceinline__ int item_overhead(const SeqWork& s, int tiles) {
  return tiles * (kUnitsTile + s.rotate);
}
__device__ __forceinline__ int item_tiles(const SeqWork& s, int lg, int t) { return s.n - (t << lg) > (1 << lg) / 2 ? 2 : 1; }
// Units of an item of nb blocks (an item without keys counts one).
__device__ __forceinline__ int64_t item_units(const SeqWork& s, int tiles, int nb) {
  return item_overhead(s, tiles) + (int64_t)s.nI * kUnitsInt2 + (int64_t)(nb - s.nI) * kUnitsBf16;
}
// Units of the tile pairs 0 .. t-1, all of them full (2^lg tokens, 16 to 256): their overheads and
// leading blocks, and the causal blocks sum over u < t of max(1, ceil((A + 2^lg (u + 1)) / 128)).
__device__ __forceinline__ int64_t units_before(const SeqWork& s, int lg, int t) {
  const int bt = 1 << lg;
  const int n0 = s.A < 0 ? min(-s.A >> lg, t) : 0;  // pairs without a key
  const int m = t - n0, c = s.A + (n0 << lg) + bt + kTile - 1;
  int64_t blocks = (int64_t)n0 + (int64_t)m * (c >> 7);
  if (bt >= kTile) {
    blocks += (int64_t)(bt >> 7) * (((int64_t)m * (m - 1)) >> 1);
  } else {
    const int lr = 7 - lg, r = 1 << lr, w0 = (kTile - (c & 127) + bt - 1) >> lg;  // remainders >= w0 carry
    const int64_t M = m >> lr;
    const int rem = m & (r - 1);
    blocks += r * ((M * (M - 1)) >> 1) + M * (r - w0) + rem * M + max(0, rem - w0);
  }
  return t * item_units(s, 2, s.nI + s.nB) + blocks * kUnitsBf16;
}
__device__ __forceinline__ int64_t units_of(const SeqWork& s, int lg) {  // of one KV head
  const int T = pairs_of(s, lg);
  return T ? units_before(s, lg, T - 1) + item_units(s, item_tiles(s, lg, T - 1), max(1, real_blocks(s, lg, T - 1))) : 0;
}
// The block in front of which a boundary x units behind an item's start cuts it (never one block off
// either end).
__device__ __forceinline__ int cut_at(const SeqWork& s, int tiles, int64_t x, int nb) {
  const int64_t y = x - item_overhead(s, tiles) / 2, yi = (int64_t)s.nI * kUnitsInt2;
  const int64_t k = y <= 0 ? 0 : y < yi ? y / kUnitsInt2 : s.nI + (y - yi) / kUnitsBf16;
  return k < 2 ? 0 : k > nb - 2 ? nb : (int)k;
}

// A place in the order (sequence, KV head, tile pair, block), moved segment by segment up to the
// CTA's end.
template <int MODE>
struct Cursor {
  SeqWork s;
  int i, h, t, k0, k1, nb;  // the segment: blocks [k0, k1) of nb
  int lg;
  int64_t end;              // units from the item's start to the CTA's end

  __device__ __forceinline__ void start(const ChunkArgs& C, int i_, int h_, int t_, int64_t x, int64_t n) {
    lg = C.lg;
    i = i_;
    h = h_;
    t = t_;
    end = x + n;
    s = load_seq<MODE>(C, i);
    nb = max(1, real_blocks(s, lg, t));
    k0 = cut_at(s, tiles(), x, nb);
    k1 = cut_at(s, tiles(), end, nb);
    if (k0 >= nb) next(C);
  }
  __device__ __forceinline__ bool valid() const { return k1 > k0; }
  __device__ __forceinline__ void next(const ChunkArgs& C) {
    end -= item_units(s, tiles(), nb);
    k0 = k1 = 0;
    if (end <= 0) return;
    if (++t >= pairs_of(s, lg)) {
      t = 0;
      if (++h >= C.Hkv) {
        h = 0;
        do {
          ++i;
          s = load_seq<MODE>(C, i);
        } while (s.n == 0 && i + 1 < C.n_seqs);
      }
    }
    nb = max(1, real_blocks(s, lg, t));
    k1 = cut_at(s, tiles(), end, nb);
  }
  __device__ __forceinline__ bool empty() const { return real_blocks(s, lg, t) == 0; }
  __device__ __forceinline__ int tokens() const { return min(1 << lg, s.n - (t << lg)); }
  __device__ __forceinline__ int tiles() const { return item_tiles(s, lg, t); }
  __device__ __forceinline__ bool two() const { return tiles() == 2; }  // the second tile has rows
  // Causal keys that every row of the pair sees, and that any does.
  __device__ __forceinline__ int keys_all() const { return max(s.A + (t << lg) + 1, 0); }
  __device__ __forceinline__ int keys_any() const { return s.A + min(s.n, (t + 1) << lg); }
};

// Where one half block of 64 keys comes from, and its slots [lo, hi) that hold keys for anyone.
struct Half {
  int lo, hi;
  int pos;  // BF16 cache: page index; pool: first chunk row, or position of slot 0 in the ring, -1 the sink
};
template <int MODE>
__device__ __forceinline__ Half half_of(const SeqWork& s, int k, int half) {
  Half r;
  if (MODE != kBf16 && k < s.nI) {
    const int j = 2 * k + half;
    r.lo = 0;
    r.hi = min(max(s.hist - j * kPage, 0), kPage);
    r.pos = j;
  } else if (MODE != kBf16 && k < s.nI + s.nB) {
    const int j = 2 * (k - s.nI) + half;
    if (j == 0) {
      r.lo = 0;
      r.hi = min(kSink, s.L);
      r.pos = -1;
    } else {
      r.pos = ((s.F >> 6) + j - 1) << 6;
      r.lo = min(max(s.F - r.pos, 0), kPage);
      r.hi = min(max(s.L - r.pos, r.lo), kPage);
    }
  } else {
    const int j = 2 * (k - s.nI - s.nB) + half;
    r.lo = 0;
    r.hi = min(max(s.A + s.n - j * kPage, 0), kPage);
    r.pos = j;
  }
  return r;
}
__device__ __forceinline__ uint64_t bits(int lo, int hi) {  // bits [lo, hi) of 64
  const uint64_t a = hi >= 64 ? ~0ull : (1ull << max(hi, 0)) - 1ull, b = lo >= 64 ? ~0ull : (1ull << lo) - 1ull;
  return a & ~b;
}

// ------------------------------------------------------------------------------------------------
// A V tile to be cleaned, two halves of 64 rows: rows outside [a, b) of a half are zeroed, rows [lo, hi)
// of the tile searched for non-finite values.
struct Clean {
  int32_t a[2], b[2], lo, hi;
  int32_t stage, slot;  // slot: row of `bad` that takes the keys found; stage -1: no more
};

template <int MODE>
struct Shared {
  uint64_t full[kStages<MODE>], empty[kStages<MODE>], code_full[kMaxSlots], code_empty[kMaxSlots];
  // S of a block is followed by its P, so s_full never runs ahead of the rows' threads; O has a barrier of
  // its own, since nothing answers it before the next S
  uint64_t q_full, q_empty, s_full[2], p_ready[2], o_full[2], done, clean_go, clean_done;
  uint32_t tmem;
  int32_t abort;
  // plan
  int64_t total, st_x, scan[20];
  int32_t st_i, st_h, st_t;
  Clean clean;
  // non-finite values of the diagonal blocks: key bits per block, two segments in turn
  uint32_t bad[2][4][4];
  uint32_t any_bad[2];
  Cursor<MODE> cursors[8];  // of the softmax warps, whose registers hold scores
};
constexpr int kSharedBytes = 2048;
static_assert(sizeof(Shared<kDequant>) <= kSharedBytes && sizeof(Shared<kBf16>) <= kSharedBytes, "Shared");
template <int MODE>
constexpr int kChunkSmem = (2 + kStages<MODE>) * kTileBytes + (MODE == kDequant ? kCodeBuf : 0) + kSharedBytes;
static_assert(kChunkSmem<kDequant> <= 232448 && kChunkSmem<kBf16> <= 232448, "shared memory of an SM");

// One try that sleeps up to ns nanoseconds: a spinning warp takes issue slots from the others.
__device__ __forceinline__ bool mbar_try_wait_for(uint64_t* bar, uint32_t parity, uint32_t ns) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(ns)
      : "memory");
  return ok != 0;
}
// Bounded wait that also ends when another role gave up. SLEEP: for roles with time to spare.
template <bool SLEEP = false, int MODE>
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, Shared<MODE>* sh, uint32_t* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (SLEEP ? mbar_try_wait_for(bar, parity, 2000) : mbar_try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile int32_t*>(&sh->abort)) return false;
    if (clock64() - t0 >= kWaitCycles) break;
  }
  *reinterpret_cast<volatile int32_t*>(&sh->abort) = 1;
  set_err(err, OSCAR_DEVERR_TIMEOUT);
  return false;
}
// The same for a whole warp, which leaves it converged (tensor-memory instructions and aligned
// barriers follow).
template <bool SLEEP = false, int MODE>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Shared<MODE>* sh, uint32_t* err) {
  const bool ok = wait_bar<SLEEP>(bar, parity, sh, err);
  __syncwarp();
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}

// The ring of K / V tiles has two producers in a mixed pool: the tensor-copy warp and the four
// dequantising warps. A parity tells a barrier's phase only to a role that is at most one phase off, so
// both go through every position: a stage is empty again when its tile has been used (one arrival, of
// the tensor cores) and when the producer it does not belong to has passed it (four arrivals).
constexpr int kPassers = 4;
template <int MODE>
struct Ring {  // position in the stream of K / V tiles
  uint32_t pos = 0;
  __device__ __forceinline__ int stage() const { return pos % kStages<MODE>; }
  __device__ __forceinline__ uint32_t parity() const { return (pos / kStages<MODE>) & 1; }
};
// A tile's full barrier counts the four dequantising warps; a tensor copy's lane arrives for all.
template <int MODE>
__device__ __forceinline__ void expect_tile(uint64_t* bar, uint32_t bytes) {
  mbar_expect_tx(bar, bytes);
  if (MODE == kDequant) mbar_arrive_n(bar, 3);
}
// Blocks of packed pages that fit the code buffer.
__device__ __forceinline__ int code_slots(const DevPool& P) { return P.ngroups == 1 ? 3 : 2; }

// The two limb tiles of a rotation matrix.
constexpr int kLimbs = 2;

// ---- tensor-copy warp --------------------------------------------------------------------------
template <int MODE>
__device__ void load_role(const ChunkArgs& C, const ChunkMaps& M, Shared<MODE>* sh, uint8_t* sq, uint8_t* ring, uint8_t* codes,
                          Cursor<MODE> cur) {
  // one lane
  const uint64_t keep = policy_evict_last(), once = policy_evict_first();
  // Of the keys and values: kept in L2 where several pairs of tiles come for them (1K after 64K: 1590 us, 1640
  // without), else let go (16 sequences of 4: 177 us for 182).
  uint64_t policy = keep;
  Ring<MODE> r;
  uint32_t issued = 0, qn = 0;  // bit s: stage s has had a tensor copy
  uint32_t last_parity = 0;
  bool ok = true;
  auto load_q = [&]() {
    if (qn && !wait_bar<true>(&sh->q_empty, (qn - 1) & 1, sh, C.err)) return false;
    const int tiles = cur.two() ? 2 : 1, tok = cur.s.row0 + (cur.t << C.lg);
    mbar_expect_tx(&sh->q_full, tiles * kTileBytes);
    for (int u = 0; u < tiles; ++u)
      for (int d = 0; d < 2; ++d)
        tma_load_3d(sq + u * kTileBytes + d * kHalfBytes, &M.q, d * 64, cur.h * C.hg, tok + u * ((1 << C.lg) / 2), &sh->q_full, once);
    ++qn;
    return true;
  };
  auto stage = [&](uint8_t*& dst, uint64_t*& bar) {
    const int s = r.stage();
    if (!wait_bar<true>(&sh->empty[s], r.parity() ^ 1, sh, C.err)) return false;
    dst = ring + s * kTileBytes;
    bar = &sh->full[s];
    issued |= 1u << s;
    last_parity = (last_parity & ~(1u << s)) | (r.parity() << s);
    ++r.pos;
    return true;
  };
  auto skip = [&](int n) {  // tiles that the dequantising warps fill
    for (; n > 0; --n, ++r.pos) {
      if (!wait_bar<true>(&sh->empty[r.stage()], r.parity() ^ 1, sh, C.err)) return false;
      issued &= ~(1u << r.stage());
      mbar_arrive_n(&sh->empty[r.stage()], 4);
    }
    return true;
  };
  auto load_limbs = [&](int kv) {
    const uint8_t* src = C.P.rlimbs + ((size_t)(C.layer * C.P.Hkv + cur.h) * 2 + kv) * (kLimbs * kTileBytes);
    for (int l = 0; l < kLimbs; ++l) {
      uint8_t* dst;
      uint64_t* bar;
      if (!stage(dst, bar)) return false;
      expect_tile<MODE>(bar, kTileBytes);
      bulk_g2s(dst, src + l * kTileBytes, kTileBytes, bar, keep);
    }
    return true;
  };
  auto load_tiles = [&](int k) {  // the fp16 tiles of INT2 block k
    const uint8_t* src = C.tiles + ((int64_t)cur.s.tile0 * C.Hkv + (int64_t)cur.h * cur.s.nI + k) * (2 * kTileBytes);
    for (int kv = 0; kv < 2; ++kv) {
      uint8_t* dst;
      uint64_t* bar;
      if (!stage(dst, bar)) return false;
      mbar_expect_tx(bar, kTileBytes);
      bulk_g2s(dst, src + kv * kTileBytes, kTileBytes, bar, policy);
    }
    return true;
  };
  // The packed pages of INT2 block k, as they lie.
  uint32_t cpos = 0;
  auto load_codes = [&](int k) {
    const int slots = code_slots(C.P), slot = cpos % slots;
    const int64_t j = 2 * (int64_t)k;
    const bool second = (j + 1) * kPage < cur.s.hist;
    const int32_t* pt = C.P.page_table + (size_t)cur.s.seq * C.P.maxp + j;
    int64_t pid[2] = {pt[0], second ? pt[1] : 0};
    if (!wait_bar<true>(&sh->code_empty[slot], ((cpos / slots) & 1) ^ 1, sh, C.err)) return false;
    mbar_expect_tx(&sh->code_full[slot], (second ? 2 : 1) * C.P.block_bytes);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (x && !second) break;
      if (pid[x] < 0 || pid[x] >= C.P.max_int2_pages) {
        set_err(C.err, OSCAR_DEVERR_PAGE);
        pid[x] = 0;
      }
      bulk_g2s(codes + (size_t)(slot * 2 + x) * C.P.block_bytes,
               C.P.int2 + (size_t)C.layer * C.P.int2_layer_stride + ((size_t)pid[x] * C.Hkv + cur.h) * C.P.block_bytes,
               C.P.block_bytes, &sh->code_full[slot], policy);
    }
    ++cpos;
    return true;
  };
  auto load_block = [&](int k) {
    Half hf[2];
    int row[2];
    const CUtensorMap* map[2][2];
    bool rows3 = false;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      hf[x] = half_of<MODE>(cur.s, k, x);
      if constexpr (MODE != kBf16) {
        rows3 = k >= cur.s.nI + cur.s.nB;
        if (rows3) {
          row[x] = cur.s.row0 + hf[x].pos * kPage;
          map[x][0] = &M.k;
          map[x][1] = &M.v;
        } else if (hf[x].pos < 0) {
          row[x] = (cur.s.sink * C.Hkv + cur.h) * kPage;
          map[x][0] = &M.sink_k;
          map[x][1] = &M.sink_v;
        } else {
          row[x] = (cur.s.seq * C.Hkv + cur.h) * kRecent + (hf[x].pos & (kRecent - 1));
          map[x][0] = &M.ring_k;
          map[x][1] = &M.ring_v;
        }
      } else {
        int64_t pid = 0;
        if (hf[x].hi > 0) pid = C.page_table[(int64_t)cur.i * C.max_pages + hf[x].pos];
        if (pid < 0 || pid >= C.n_pages_total) {
          set_err(C.err, OSCAR_DEVERR_PAGE);
          pid = 0;
        }
        row[x] = (int)((pid * C.Hkv + cur.h) * kPage);
        map[x][0] = &M.k;
        map[x][1] = &M.v;
      }
    }
    const int n = (hf[0].hi > hf[0].lo) + (hf[1].hi > hf[1].lo);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint8_t* dst;
      uint64_t* bar;
      if (!stage(dst, bar)) return false;
      expect_tile<MODE>(bar, n * 2 * kPageHalfBytes);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (hf[x].hi <= hf[x].lo) continue;
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          uint8_t* to = dst + d * kHalfBytes + x * kPageHalfBytes;
          if (MODE != kBf16 && rows3)
            tma_load_3d(to, map[x][kv], d * 64, cur.h, row[x], bar, policy);
          else
            tma_load_2d(to, map[x][kv], d * 64, row[x], bar, policy);
        }
      }
    }
    return true;
  };
  for (; ok && cur.valid(); cur.next(C)) {
    if (cur.empty()) continue;
    const int nI = MODE != kBf16 ? min(cur.k1, cur.s.nI) : 0;
    policy = pairs_of(cur.s, cur.lg) > 1 ? keep : once;
    if (cur.k0 < nI) {
      ok = load_q() && load_limbs(0);
      if constexpr (MODE == kDequant) {
        for (int k = cur.k0; ok && k < nI; ++k) ok = load_codes(k) && (k < cur.k0 + 2 || skip(2));  // packed pages run ahead
        ok = ok && skip(2 * min(2, nI - cur.k0));
      } else if constexpr (MODE == kTiles) {
        for (int k = cur.k0; ok && k < nI; ++k) ok = load_tiles(k);
      }
      ok = ok && (C.P.absorbed || load_limbs(1));
    }
    const int kb = max(cur.k0, nI);
    if (ok && kb < cur.k1) {
      ok = load_q();
      for (int k = kb; ok && k < cur.k1; ++k) ok = load_block(k);
    }
  }
  // Never leave with a copy in flight, whoever gave up: wait for the last lap's tiles, queries and
  // packed pages.
  for (int s = 0; s < kStages<MODE>; ++s)
    if ((issued >> s) & 1) mbar_wait(&sh->full[s], (last_parity >> s) & 1, C.err);
  if (qn) mbar_wait(&sh->q_full, (qn - 1) & 1, C.err);
  if constexpr (MODE == kDequant) {
    const uint32_t slots = code_slots(C.P);
    for (uint32_t c = cpos > slots ? cpos - slots : 0; c < cpos; ++c) mbar_wait(&sh->code_full[c % slots], (c / slots) & 1, C.err);
  }
}

// Bits 15 and 31: which of the two bf16 values of a word are infinite or NaN (all exponent bits set, so
// that one more carries out).
__device__ __forceinline__ uint32_t nonfinite(uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }

// ---- cleaning warps (two): a V tile at a time, 64 rows each, while the tile's scores become P ------
template <int MODE>
__device__ void clean_role(const ChunkArgs& C, Shared<MODE>* sh, uint8_t* ring, int part, int lane) {
  for (uint32_t n = 0;; ++n) {
    if (!wait_warp<true>(&sh->clean_go, n & 1, sh, C.err)) return;
    const Clean w = sh->clean;
    if (w.stage < 0) return;
    const int a = w.a[part], b = w.b[part], lo = min(max(w.lo - 64 * part, 0), 64), hi = min(max(w.hi - 64 * part, 0), 64);
    // a lane takes one 16-byte chunk of every other row
    const int c = lane & 15, odd = lane >> 4;
    uint8_t* base = ring + w.stage * kTileBytes + (c >> 3) * kHalfBytes + part * kPageHalfBytes + (c & 7) * 16;
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 4
    for (int row = odd; row < a; row += 2) *reinterpret_cast<uint4*>(base + row * 128) = zero;
#pragma unroll 4
    for (int row = b + odd; row < 64; row += 2) *reinterpret_cast<uint4*>(base + row * 128) = zero;
    uint32_t found[2] = {0, 0};
    for (int r0 = lo + odd; r0 < hi; r0 += 16) {
      uint4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = r0 + 2 * i < hi ? *reinterpret_cast<const uint4*>(base + (r0 + 2 * i) * 128) : zero;
      uint32_t any = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) any |= nonfinite(v[i].x) | nonfinite(v[i].y) | nonfinite(v[i].z) | nonfinite(v[i].w);
      if (any) {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          const int row = r0 + 2 * i;
          if (row >= hi) break;
          uint32_t* e = reinterpret_cast<uint32_t*>(base + row * 128);
          for (int j = 0; j < 4; ++j) {
            const uint32_t f = nonfinite(e[j]);
            if (f) {
              e[j] &= (f & 0x8000u ? 0u : 0xFFFFu) | (f & 0x80000000u ? 0u : 0xFFFF0000u);
              if (row < 32) found[0] |= 1u << row; else found[1] |= 1u << (row - 32);
            }
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t f = __reduce_or_sync(0xffffffffu, found[i]);
      if (f && lane == 0) {
        sh->bad[w.slot >> 2][w.slot & 3][2 * part + i] = f;
        sh->any_bad[w.slot >> 2] = 1;
      }
    }
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->clean_done);
  }
}

// ---- tensor-core warp --------------------------------------------------------------------------
template <int MODE>
__device__ void mma_role(const ChunkArgs& C, Shared<MODE>* sh, uint8_t* sq, uint8_t* ring, Cursor<MODE> cur, int lane) {
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh->tmem, 0), aq = smem_u32(sq), ar = smem_u32(ring);
  const uint32_t one = elect_one();
  Ring<MODE> r;
  uint32_t qn = 0, pn[2] = {0, 0}, seg = 0, cn = 0;
  bool ok = true;
  auto S = [&](int u) { return tmem + (uint32_t)(u * kTile); };
  auto O = [&](int u) { return tmem + (uint32_t)(2 * kTile + u * kTile); };
  auto wait_full = [&](uint32_t pos) {
    const bool w = wait_warp(&sh->full[pos % kStages<MODE>], (pos / kStages<MODE>) & 1, sh, C.err);
    tc_fence_after();
    return w;
  };
  auto wait_p = [&](int u) {
    const bool w = wait_warp(&sh->p_ready[u], pn[u]++ & 1, sh, C.err);
    tc_fence_after();
    return w;
  };
  auto addr = [&](uint32_t pos) { return ar + (__shfl_sync(0xffffffffu, pos, 0) % kStages<MODE>) * kTileBytes; };
  auto qk = [&](int u, uint32_t b, uint32_t idesc, bool acc) {
    tc_gemm_ss(S(u), desc_k(aq + u * kTileBytes), desc_k(b), idesc, acc, one);
  };
  auto pv = [&](int u, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
    tc_gemm_ts(O(u), a, desc_mn(b), idesc | kIdescMn, acc, one);
  };
  auto commit = [&](uint64_t* bar) { tc_commit_elected(bar, one); };

  for (; ok && cur.valid(); cur.next(C)) {
    if (cur.empty()) continue;
    const int tiles = cur.two() ? 2 : 1, sb = seg++ & 1;
    const int nI = MODE != kBf16 ? min(cur.k1, cur.s.nI) : 0;
    if (lane < 16) sh->bad[sb][lane >> 2][lane & 3] = 0;
    if (lane == 0) sh->any_bad[sb] = 0;
    __syncwarp();
    if (tiles == 1) commit(&sh->s_full[1]);
    bool acc = false;  // O holds something
    // Blocks [a, b) with operands of idesc: S of the next block is issued behind P V of this one,
    // tile by tile, so that one tile's softmax runs beside the other tile's products.
    auto blocks = [&](int a, int b, uint32_t idesc) {
      uint32_t kpos = r.pos;
      if (!wait_full(kpos)) return false;
      for (int u = 0; u < tiles; ++u) {
        qk(u, addr(kpos), idesc, false);
        commit(&sh->s_full[u]);
      }
      commit(&sh->empty[kpos % kStages<MODE>]);
      if (a + 1 == b) commit(&sh->q_empty);
      for (int k = a; k < b; ++k) {
        const uint32_t vpos = kpos + 1;
        if (!wait_full(vpos)) return false;
        bool dirty = false;
        if (idesc == kIdescBf16) {
          Clean w;
          w.lo = w.hi = w.slot = 0;
          if (MODE != kBf16 && k < cur.s.nI + cur.s.nB) {
            const Half h0 = half_of<MODE>(cur.s, k, 0), h1 = half_of<MODE>(cur.s, k, 1);
            w.a[0] = h0.lo, w.b[0] = h0.hi, w.a[1] = h1.lo, w.b[1] = h1.hi;
          } else {  // the diagonal: some rows of the pair see a key and others do not
            const int j = k - cur.s.nI - cur.s.nB;
            w.lo = min(max(cur.keys_all() - j * kTile, 0), kTile);
            w.hi = min(cur.keys_any() - j * kTile, kTile);
            w.a[0] = w.a[1] = 0, w.b[0] = min(w.hi, 64), w.b[1] = max(w.hi - 64, 0);
            w.slot = 4 * sb + j - cur.keys_all() / kTile;
          }
          dirty = w.lo < w.hi || w.a[0] > 0 || w.a[1] > 0 || w.b[0] < 64 || w.b[1] < 64;
          if (dirty && lane == 0) {
            w.stage = vpos % kStages<MODE>;
            sh->clean = w;
            mbar_arrive(&sh->clean_go);
          }
        }
        for (int u = 0; u < tiles; ++u) {
          if (!wait_p(u)) return false;
          if (u == 0 && dirty && !wait_warp(&sh->clean_done, cn++ & 1, sh, C.err)) return false;
          pv(u, S(u), addr(vpos), idesc, acc);
          if (k + 1 < b) {
            if (u == 0 && !wait_full(vpos + 1)) return false;
            qk(u, addr(vpos + 1), idesc, false);
          }
          commit(k + 1 < b ? &sh->s_full[u] : &sh->o_full[u]);  // the next S, or behind the last block O
        }
        acc = true;
        commit(&sh->empty[vpos % kStages<MODE>]);
        kpos = vpos + 1;
        if (k + 1 < b) commit(&sh->empty[kpos % kStages<MODE>]);
        if (k + 2 == b) commit(&sh->q_empty);
      }
      r.pos = kpos;
      return true;
    };
    if (MODE != kBf16 && cur.k0 < nI) {
      ok = wait_warp(&sh->q_full, qn++ & 1, sh, C.err) && wait_full(r.pos) && wait_full(r.pos + 1);
      if (!ok) break;
      for (int u = 0; u < tiles; ++u) {
        qk(u, addr(r.pos), kIdescBf16, false);
        qk(u, addr(r.pos + 1), kIdescBf16, true);
        commit(&sh->s_full[u]);
      }
      commit(&sh->empty[r.pos % kStages<MODE>]);
      commit(&sh->empty[(r.pos + 1) % kStages<MODE>]);
      r.pos += kLimbs;
      for (int u = 0; ok && u < tiles; ++u) ok = wait_p(u);  // Q R_K is in shared memory
      ok = ok && blocks(cur.k0, nI, kIdescBase);
      if (!ok) break;
      if (!C.P.absorbed) {
        ok = wait_full(r.pos) && wait_full(r.pos + 1);
        for (int u = 0; ok && u < tiles; ++u) {
          ok = wait_p(u);  // the limbs of O are in S
          if (!ok) break;
          pv(u, S(u), addr(r.pos), kIdescBf16, false);
          pv(u, S(u), addr(r.pos + 1), kIdescBf16, true);
          pv(u, S(u) + 64, addr(r.pos), kIdescBf16, true);
          if (nI == cur.k1) commit(&sh->o_full[u]);
        }
        commit(&sh->empty[r.pos % kStages<MODE>]);
        commit(&sh->empty[(r.pos + 1) % kStages<MODE>]);
        r.pos += kLimbs;
      }
    }
    const int kb = max(cur.k0, nI);
    if (ok && kb < cur.k1) ok = wait_warp(&sh->q_full, qn++ & 1, sh, C.err) && blocks(kb, cur.k1, kIdescBf16);
    if (ok && tiles == 1) ok = wait_p(1);
  }
  if (lane == 0) {
    sh->clean.stage = -1;
    mbar_arrive(&sh->clean_go);
  }
  // no product in flight when the tensor memory is given back
  commit(&sh->done);
  mbar_wait(&sh->done, 0, C.err);
}

// Two values in a word, fp16 or bf16.
template <bool HALF>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  if (HALF) return pack_half2(x, y);
  const __nv_bfloat162 w = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&w);
}
template <bool HALF>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (HALF) return half2_to_float2(w);
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// ---- softmax warps: one thread per row -----------------------------------------------------------
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 32 bytes of a thread's own row, one sector: in one store where the row starts on such a boundary.
__device__ __forceinline__ void store32(void* p, const uint32_t* w, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
                 "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <int MODE>
__device__ void softmax_role(const ChunkArgs& C, Shared<MODE>* sh, uint8_t* sq, const Cursor<MODE>& start, int u) {
  const int row = threadIdx.x & 127, warp = row >> 5;
  const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
  const uint32_t tS = sh->tmem + lane_off + u * kTile, tO = sh->tmem + lane_off + 2 * kTile + u * kTile;
  uint32_t sn = 0, on = 0, seg = 0;
  bool ok = true;
  const int hg = C.hg, tpt = kTile / hg;
  // this warp's cursor, moved by its first lane
  Cursor<MODE>& cur = sh->cursors[threadIdx.x >> 5];
  if ((threadIdx.x & 31) == 0) cur = start;
  __syncwarp();
  auto next = [&]() {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) cur.next(C);
    __syncwarp();
  };
  auto wait_s = [&]() {
    const bool w = wait_warp(&sh->s_full[u], sn++ & 1, sh, C.err);
    tc_fence_after();
    return w;
  };
  auto wait_o = [&]() {
    const bool w = wait_warp(&sh->o_full[u], on++ & 1, sh, C.err);
    tc_fence_after();
    return w;
  };
  auto ready = [&]() {
    tc_fence_before();
    mbar_arrive(&sh->p_ready[u]);
  };

  for (; ok && cur.valid(); next()) {
    const int tok = (cur.t << C.lg) + u * tpt + row / hg;  // this row's token of the sequence
    const bool live = tok < cur.s.n;
    const bool whole = cur.k0 == 0 && cur.k1 == cur.nb;
    const int head = cur.h * hg + row % hg;
    __nv_bfloat16* dst = C.out + ((int64_t)(cur.s.row0 + tok) * C.Hq + head) * kHeadDim;
    if (cur.empty()) {
      if (live)
        for (int c = 0; c < 16; ++c) reinterpret_cast<uint4*>(dst)[c] = make_uint4(0, 0, 0, 0);
      continue;
    }
    const int sb = seg++ & 1;
    if (u == 1 && !cur.two()) {
      // nothing to do, but the tensor-core warp must know that this tile's threads have left the segment
      // before, and may not be left behind by them
      ok = wait_s();
      ready();
      continue;
    }
    const int lim = min(cur.s.A + tok + 1, cur.s.A + cur.s.n);  // keys of the causal blocks this row sees
    const int nI = MODE != kBf16 ? min(cur.k1, cur.s.nI) : 0;
    float m = -INFINITY, l = 0.f;
    bool have = false;  // O holds something

    auto block = [&](auto half16, int k, float scale) {
      if (!wait_s()) return false;
      // scores of columns this row may not see
      uint64_t b0 = ~0ull, b1 = ~0ull;
      bool masked;
      if (MODE != kBf16 && k < cur.s.nI + cur.s.nB) {
        const Half h0 = half_of<MODE>(cur.s, k, 0), h1 = half_of<MODE>(cur.s, k, 1);
        b0 = bits(h0.lo, h0.hi);
        b1 = bits(h1.lo, h1.hi);
        masked = (b0 & b1) != ~0ull;
      } else {
        const int at = (k - cur.s.nI - cur.s.nB) * kTile;
        masked = __any_sync(0xffffffffu, lim < at + kTile);
        if (masked) {
          b0 = bits(0, min(max(lim - at, 0), 64));
          b1 = bits(0, min(max(lim - at - 64, 0), 64));
        }
      }
      if (masked) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t x[32];
          tc_ld32_issue(tS + 32 * c, x);
          tc_ld_wait1(x);
          const uint32_t b = (uint32_t)((c & 2 ? b1 : b0) >> (32 * (c & 1)));
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!((b >> i) & 1)) x[i] = 0xFF800000u;
          tc_st32(tS + 32 * c, x);
          tc_st_wait();
        }
      }
      // The maximum is taken anew only where it must be: for the rows' first block, and when the weights of
      // 32 (or 128) scores under the last one sum to more than kGrown (each is finite then, or their sum infinite).
      // The weights already made are scaled then, as the sums and O are. The warp goes through it together, but a row
      // takes its new maximum only where it needs it: its bits do not depend on the other rows, of later tokens among them. The loops stay rolled: the warps'
      // instructions come from one cache, and unrolled they waited for it longer than for their data.
      float2 sum = make_float2(0.f, 0.f);
      auto grow = [&](int c0, bool mine) {
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll 1
        for (int c = c0; c < 4; ++c) {
          uint32_t x[32];
          tc_ld32_issue(tS + 32 * c, x);
          tc_ld_wait1(x);
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            mx0 = max3(mx0, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
            mx1 = max3(mx1, __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]));
          }
        }
        const float mb = fmaxf(mx0, mx1) * scale - (decltype(half16)::value ? kHeadroom : 0.f);
        const float mn = mine ? fmaxf(m, mb) : m, alpha = mn > m ? fast_exp2(m - mn) : 1.f;
        m = mn;
        l *= alpha;
        sum.x *= alpha;
        sum.y *= alpha;
        if (c0 > 0) tc_st_wait();  // the weights read back below were stored without a wait
#pragma unroll 1
        for (int c = 0; c < c0; ++c) {
          uint32_t w[16];
          tc_ld16_issue(tS + 16 * c, w);
          tc_ld16_wait(w);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 f = unpack2<decltype(half16)::value>(w[i]);
            w[i] = pack2<decltype(half16)::value>(f.x * alpha, f.y * alpha);
          }
          tc_st16(tS + 16 * c, w);
          tc_st_wait();
        }
        if (have) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tc_ld32_issue(tO + 32 * c, o);
            tc_ld_wait1(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tc_st32(tO + 32 * c, o);
            tc_st_wait();
          }
        }
      };
      bool mine = m == -INFINITY, renewed = false;  // this row: needs a maximum; has taken it in this block
      const float2 sc2 = make_float2(scale, scale);
      if constexpr (MODE == kDequant) {
        bool again = __any_sync(0xffffffffu, mine);
#pragma unroll 1
        for (int c = 0;;) {
          if (again) {
            grow(c, mine);
            renewed |= mine;
            again = false;
          }
          const float nm = m == -INFINITY ? 0.f : -m;
          const float2 nm2 = make_float2(nm, nm);
#pragma unroll 1
          for (; c < 4; ++c) {
            uint32_t x[32], p[16];
            float2 s0 = make_float2(0.f, 0.f), s1 = s0;
            tc_ld32_issue(tS + 32 * c, x);
            tc_ld_wait1(x);
            // two scores an instruction, but for the exponentials
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float2 e = __ffma2_rn(make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), sc2, nm2);
              e.x = fast_exp2(e.x);
              e.y = fast_exp2(e.y);
              if (i & 1) s1 = __fadd2_rn(s1, e); else s0 = __fadd2_rn(s0, e);
              p[i] = pack2<decltype(half16)::value>(e.x, e.y);
            }
            s0 = __fadd2_rn(s0, s1);
            mine = !renewed && s0.x + s0.y > kGrown;
            again = __any_sync(0xffffffffu, mine);
            if (again) break;
            sum = __fadd2_rn(sum, s0);
            tc_st16(tS + 16 * c, p);  // the columns of scores already read
          }
          if (!again) break;
        }
      } else {
        uint32_t p[64];
        for (bool again = __any_sync(0xffffffffu, mine);;) {
          if (again) grow(0, mine);
          renewed |= mine;
          const float nm = m == -INFINITY ? 0.f : -m;
          const float2 nm2 = make_float2(nm, nm);
          float2 s0 = make_float2(0.f, 0.f), s1 = s0;
          uint32_t x[2][16];
          tc_ld16_issue(tS, x[0]);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t(&y)[16] = x[c & 1];
            tc_ld16_wait(y);
            if (c < 7) tc_ld16_issue(tS + 16 * (c + 1), x[(c + 1) & 1]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float2 e = __ffma2_rn(make_float2(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1])), sc2, nm2);
              e.x = fast_exp2(e.x);
              e.y = fast_exp2(e.y);
              if (i & 1) s1 = __fadd2_rn(s1, e); else s0 = __fadd2_rn(s0, e);
              p[8 * c + i] = pack2<decltype(half16)::value>(e.x, e.y);
            }
          }
          sum = __fadd2_rn(s0, s1);
          mine = !renewed && sum.x + sum.y > kGrown;
          again = __any_sync(0xffffffffu, mine);
          if (!again) break;
        }
        tc_st64(tS, p);
      }
      l += sum.x + sum.y;
      tc_st_wait();
      ready();
      have = true;
      return true;
    };

    if (MODE != kBf16 && cur.k0 < nI) {
      // Q R_K: fp16, scaled by the power of two that brings the row's largest value to [1, 2)
      ok = wait_s();
      if (!ok) break;
      float scale = kScoreLog2;
      {
        uint32_t s[32];
        float mx = 0.f;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          tc_ld32_issue(tS + 32 * c, s);
          tc_ld_wait1(s);
#pragma unroll
          for (int i = 0; i < 32; ++i) mx = fmaxf(mx, fabsf(__uint_as_float(s[i])));
        }
        const uint32_t e = __float_as_uint(mx) >> 23;
        float down = 1.f;
        if (e > 0 && e < 254) {
          down = __uint_as_float((254 - e) << 23);
          scale *= __uint_as_float(e << 23);
        }
        uint8_t* q = sq + u * kTileBytes + row * 128;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          tc_ld32_issue(tS + 32 * c, s);
          tc_ld_wait1(s);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = pack_half2(__uint_as_float(s[8 * j + 2 * i]) * down, __uint_as_float(s[8 * j + 2 * i + 1]) * down);
            *reinterpret_cast<uint4*>(q + (c >> 1) * kHalfBytes + (((4 * (c & 1) + j) ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      fence_proxy_async();
      ready();
      for (int k = cur.k0; ok && k < nI; ++k) ok = block(std::true_type{}, k, scale);
      if (!ok) break;
      ok = wait_o();  // O is complete
      if (!ok) break;
      if (!C.P.absorbed) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32], hi[16], lo[16];
          tc_ld32_issue(tO + 32 * c, o);
          tc_ld_wait1(o);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float x = __uint_as_float(o[2 * i]), y = __uint_as_float(o[2 * i + 1]);
            const __nv_bfloat162 a = __floats2bfloat162_rn(x, y);
            const __nv_bfloat162 b = __floats2bfloat162_rn(x - __bfloat162float(a.x), y - __bfloat162float(a.y));
            hi[i] = *reinterpret_cast<const uint32_t*>(&a);
            lo[i] = *reinterpret_cast<const uint32_t*>(&b);
          }
          tc_st16(tS + 16 * c, hi);
          tc_st_wait();
          tc_st16(tS + 64 + 16 * c, lo);
          tc_st_wait();
        }
        ready();
      }
    }
    const int kb = max(cur.k0, nI);
    for (int k = kb; ok && k < cur.k1; ++k) ok = block(std::false_type{}, k, kScoreLog2);
    if (!ok) break;
    // O is complete (behind the last INT2 block of an absorbed pool it was waited for above)
    if (kb < cur.k1 || (MODE != kBf16 && !C.P.absorbed)) ok = wait_o();
    if (!ok) break;

    const bool bad = *reinterpret_cast<volatile uint32_t*>(&sh->any_bad[sb]) != 0;
    float* slot = nullptr;
    float inv = l == 0.f ? 0.f : 1.f / l;
    if (!whole) {
      // a boundary cuts the item in front of this segment (slot 0) or behind it (slot 1)
      slot = reinterpret_cast<float*>(C.ws + (size_t)kMaxCtas * kDescBytes) +
             ((size_t)blockIdx.x * 2 + (cur.k0 > 0 ? 0 : 1)) * C.rows * (kHeadDim + 2);
      const int pr = u * kTile + row;
      if (live) *reinterpret_cast<float2*>(slot + (size_t)C.rows * kHeadDim + 2 * pr) = make_float2(m, l);
      slot += (size_t)pr * kHeadDim;
      inv = 1.f;
    }
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint32_t o[32];
      tc_ld32_issue(tO + 32 * c, o);
      tc_ld_wait1(o);
      if (live) {
        float f[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(o[i]);
        if (bad) {  // non-finite values this row does see
          const int j0 = cur.keys_all() / kTile;
          for (int b = 0; b < kTile * 4; ++b) {
            const int key = j0 * kTile + b;
            if (key >= lim || !((sh->bad[sb][b >> 7][(b >> 5) & 3] >> (b & 31)) & 1)) continue;
            const __nv_bfloat16* v;
            int swz = 0;
            if constexpr (MODE != kBf16) {
              v = C.v_new + ((int64_t)(cur.s.row0 + key) * C.Hkv + cur.h) * kHeadDim;
            } else {
              int64_t pid = C.page_table[(int64_t)cur.i * C.max_pages + (key >> 6)];
              if (pid < 0 || pid >= C.n_pages_total) pid = 0;
              v = reinterpret_cast<const __nv_bfloat16*>(C.v_pages) + (((int64_t)pid * C.Hkv + cur.h) * kPage + (key & 63)) * kHeadDim;
              swz = key & 7;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int d = 32 * c + i;
              const float x = __bfloat162float(v[(((d >> 3) ^ swz) << 3) + (d & 7)]);
              if (!isfinite(x)) f[i] += x;
            }
          }
        }
        if (whole) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const __nv_bfloat162 x = __floats2bfloat162_rn(f[16 * i + 2 * e] * inv, f[16 * i + 2 * e + 1] * inv);
              w[e] = *reinterpret_cast<const uint32_t*>(&x);
            }
            store32(dst + 32 * c + 16 * i, w, C.wide);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) store32(slot + 32 * c + 8 * i, reinterpret_cast<const uint32_t*>(f) + 8 * i, true);
        }
      }
      __syncwarp();  // the next tensor-memory load is the whole warp's
    }
  }
}

// ---- dequantising warps (pool) -------------------------------------------------------------------
__device__ void dequant_role(const ChunkArgs& C, Shared<kDequant>* sh, uint8_t* ring, const uint8_t* codes, Cursor<kDequant> cur) {
  const int x = threadIdx.x & 127, lane = threadIdx.x & 31;
  const DevPool& P = C.P;
  const int ng = P.ngroups, slots = code_slots(P);
  // K: thread x has token x of the block. V: a slice of 16 tokens, of it tokens 8u + 2tq + {0, 1} and
  // one half of the dims.
  const int slice = x >> 4, wh = (x >> 3) & 1, uu = (x >> 2) & 1, tq = x & 3;
  Ring<kDequant> r;
  uint32_t cpos = 0;
  bool ok = true;
  auto done = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  auto skip = [&](int n) {  // tiles of the tensor-copy warp
    for (; n > 0; --n, ++r.pos) {
      if (!wait_warp(&sh->empty[r.stage()], r.parity() ^ 1, sh, C.err)) return false;
      done(&sh->empty[r.stage()]);
    }
    return true;
  };
  for (; ok && cur.valid(); cur.next(C)) {
    if (cur.empty()) continue;
    const int nI = min(cur.k1, cur.s.nI);
    if (cur.k0 < nI) {
      ok = skip(kLimbs);
      const size_t lh = (size_t)C.layer * P.Hkv + cur.h;
      const bool table = P.lloyd != 0;
      const float ak = table ? P.cb_a[lh * 2] : 1.f, av = table ? P.cb_a[lh * 2 + 1] : 1.f;
      for (int k = cur.k0; ok && k < nI; ++k) {
        const int slot = cpos % slots;
        ok = wait_warp(&sh->code_full[slot], (cpos / slots) & 1, sh, C.err);
        if (!ok) break;
        ++cpos;
        // This thread's packed words. Of a token behind the history the value's scale and zero are 0, so the values are;
        // its key is whatever lies there (a page slot that was not loaded, too), and the mask covers its score.
        const uint8_t* kp = codes + (size_t)(slot * 2 + (x >> 6)) * P.block_bytes;
        const uint8_t* vp = codes + (size_t)(slot * 2 + (slice >> 2)) * P.block_bytes;
        const uint4 kc0 = reinterpret_cast<const uint4*>(kp + (x & 63) * kCodeBytes)[0];
        const uint4 kc1 = reinterpret_cast<const uint4*>(kp + (x & 63) * kCodeBytes)[1];
        uint32_t vc[8], ksz[4], vsz[2][2];
        const uint8_t* vw = vp + kPage * kCodeBytes + (slice & 3) * 512 + tq * 16 + 8 * uu + 4 * wh;
#pragma unroll
        for (int g = 0; g < 8; ++g) vc[g] = *reinterpret_cast<const uint32_t*>(vw + g * 64);
        const uint32_t* sz = reinterpret_cast<const uint32_t*>(kp + 2 * kPage * kCodeBytes);
#pragma unroll
        for (int i = 0; i < 4; ++i) ksz[i] = i < ng ? sz[sz_index(x & 63, i, ng)] : 0;
        sz = reinterpret_cast<const uint32_t*>(vp + 2 * kPage * kCodeBytes) + kPage * ng;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int tau = (slice & 3) * 16 + 8 * uu + 2 * tq + e;
          const bool live = k * kTile + (slice >> 2) * kPage + tau < cur.s.hist;
#pragma unroll
          for (int w = 0; w < 2; ++w) vsz[e][w] = live ? sz[sz_index(tau, ng == 1 ? 0 : 2 * wh + w, ng)] : 0;
        }
        done(&sh->code_empty[slot]);
        // K tile
        int s = r.stage();
        ok = wait_warp(&sh->empty[s], r.parity() ^ 1, sh, C.err);
        if (!ok) break;
        {
          // dims 64 wd + 32 sh8 + 8p + 2tq + {0, 1} are slot p of byte sh8 of the halves of word [tq][wd]
          uint8_t* dst = ring + s * kTileBytes + x * 128;
          auto tile = [&](auto tab) {
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {  // 64-dim half wd = i >> 1, byte sh8 = i & 1
              uint32_t W[4] = {i & 2 ? kc0.y : kc0.x, i & 2 ? kc0.w : kc0.z, i & 2 ? kc1.y : kc1.x, i & 2 ? kc1.w : kc1.z};
#pragma unroll
              for (int j = 0; j < 4; ++j) W[j] >>= 8 * (i & 1);
              const Levels t = levels(ng == 1 || i == 0 ? ksz[0] : i == 1 ? ksz[1] : i == 2 ? ksz[2] : ksz[3], ak, decltype(tab)::value);
#pragma unroll
              for (int p = 0; p < 4; ++p)  // chunk 4 sh8 + p of the half wd
                *reinterpret_cast<uint4*>(dst + (i >> 1) * kHalfBytes + (((4 * (i & 1) + p) ^ (x & 7)) << 4)) =
                    make_uint4(expand(W[0], p, t, decltype(tab)::value), expand(W[1], p, t, decltype(tab)::value), expand(W[2], p, t, decltype(tab)::value), expand(W[3], p, t, decltype(tab)::value));
            }
          };
          if (table) tile(std::true_type{}); else tile(std::false_type{});
        }
        fence_proxy_async();
        done(&sh->full[s]);
        ++r.pos;
        // V tile
        s = r.stage();
        ok = wait_warp(&sh->empty[s], r.parity() ^ 1, sh, C.err);
        if (!ok) break;
        {
          // dims 32 (2 wh + w1) + 8p + g of token e are slot p of byte w1 of half e of word g
          uint8_t* half = ring + s * kTileBytes + wh * kHalfBytes;
          auto tile = [&](auto tab) {
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              // token e, byte w1; lanes of odd u start with the odd token: eight rows, eight banks
              const int e = (i >> 1) ^ uu, w1 = i & 1, rowv = slice * 16 + 8 * uu + 2 * tq + e;
              uint8_t* dst = half + rowv * 128;
              const Levels t = levels(ng == 1 || !w1 ? (e ? vsz[1][0] : vsz[0][0]) : (e ? vsz[1][1] : vsz[0][1]), av, decltype(tab)::value);
              const uint32_t sel = (e ? 0x7632u : 0x5410u);
              uint32_t W[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) W[j] = __byte_perm(vc[2 * j], vc[2 * j + 1], sel) >> (8 * w1);
#pragma unroll
              for (int p = 0; p < 4; ++p)
                *reinterpret_cast<uint4*>(dst + (((4 * w1 + p) ^ (rowv & 7)) << 4)) =
                    make_uint4(expand(W[0], p, t, decltype(tab)::value), expand(W[1], p, t, decltype(tab)::value), expand(W[2], p, t, decltype(tab)::value), expand(W[3], p, t, decltype(tab)::value));
            }
          };
          if (table) tile(std::true_type{}); else tile(std::false_type{});
        }
        fence_proxy_async();
        done(&sh->full[s]);
        ++r.pos;
      }
      if (ok && !P.absorbed) ok = skip(kLimbs);
    }
    if (ok) ok = skip(2 * (cur.k1 - max(cur.k0, nI)));
  }
}

// ------------------------------------------------------------------------------------------------
template <int MODE>
constexpr int kChunkThreads = MODE == kDequant ? 512 : 384;

template <int R>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// First unit of CTA c of n.
__device__ __forceinline__ int64_t boundary(int c, int64_t total, int n) {
  if (c >= n) return total;
  return total < (1 << 22) ? (int64_t)((uint32_t)c * (uint32_t)total / (uint32_t)n) : (int64_t)c * total / n;
}

// Units of all sequences, this CTA's range [g0, g1) of them and the item that holds g0; every thread
// of the CTA. Returns the number of CTAs that have a range.
template <int MODE>
__device__ int plan(const ChunkArgs& C, Shared<MODE>* sh, int64_t& g0, int64_t& g1) {
  constexpr int NT = kChunkThreads<MODE>, NW = NT / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // The first NT sequences stay in registers; their scan is the only one of a call without more.
  SeqWork s{};
  if (threadIdx.x < C.n_seqs) s = load_seq<MODE>(C, threadIdx.x);
  int64_t per = units_of(s, C.lg), inc, base, before;
  auto scan = [&]() {  // units before this thread's sequence of the round, and behind the round
    inc = per * C.Hkv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) sh->scan[warp] = inc;
    __syncthreads();
    before = base + inc - per * C.Hkv;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const int64_t y = sh->scan[w];
      if (w < warp) before += y;
      base += y;
    }
  };
  base = 0;
  scan();
  int64_t total = base;
  if (C.n_seqs > NT) {
    int64_t more = 0;
    for (int i = threadIdx.x + NT; i < C.n_seqs; i += NT) more += units_of(load_seq<MODE>(C, i), C.lg) * C.Hkv;
#pragma unroll
    for (int o = 16; o; o >>= 1) more += __shfl_xor_sync(0xffffffffu, more, o);
    __syncthreads();
    if (lane == 0) sh->scan[warp] = more;
    __syncthreads();
    for (int w = 0; w < NW; ++w) total += sh->scan[w];
  }
  const int n = (int)min((int64_t)gridDim.x, max((int64_t)1, total / kMinUnits));
  g0 = boundary(blockIdx.x, total, n);
  g1 = boundary(blockIdx.x + 1, total, n);
  if (g0 >= g1) return n;
  if (threadIdx.x == 0) sh->total = total;
  for (int i = threadIdx.x;; i += NT) {
    if (per > 0 && g0 >= before && g0 < before + per * C.Hkv) {
      int64_t x = g0 - before;
      int h = 0;
      while (x >= per) {
        x -= per;
        ++h;
      }
      int lo = 0, hi = pairs_of(s, C.lg) - 1;
      while (lo < hi) {  // the last pair that starts at or before x
        const int mid = (lo + hi + 1) >> 1;
        if (units_before(s, C.lg, mid) <= x) lo = mid; else hi = mid - 1;
      }
      sh->st_i = i;
      sh->st_h = h;
      sh->st_t = lo;
      sh->st_x = x - units_before(s, C.lg, lo);
    }
    if (base > g0) break;
    s = SeqWork{};
    if (i + NT < C.n_seqs) s = load_seq<MODE>(C, i + NT);
    per = units_of(s, C.lg);
    __syncthreads();  // the last round's sums have been read
    scan();
  }
  return n;
}

template <int MODE>
__global__ void __launch_bounds__(kChunkThreads<MODE>, 1)
    k_chunk(const __grid_constant__ ChunkArgs C, const __grid_constant__ ChunkMaps M) {
  extern __shared__ __align__(1024) uint8_t smem[];  // tiles start on the swizzle's 1024-byte boundaries
  uint8_t *sq = smem, *ring = smem + 2 * kTileBytes, *codes = ring + kStages<MODE> * kTileBytes;
  Shared<MODE>* sh = reinterpret_cast<Shared<MODE>*>(codes + (MODE == kDequant ? kCodeBuf : 0));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages<MODE>; ++s) {
      mbar_init(&sh->full[s], MODE == kDequant ? 4 : 1);
      mbar_init(&sh->empty[s], MODE == kDequant ? 1 + kPassers : 1);
    }
    for (int s = 0; s < kMaxSlots; ++s) {
      mbar_init(&sh->code_full[s], 1);
      mbar_init(&sh->code_empty[s], 4);
    }
    mbar_init(&sh->q_full, 1);
    mbar_init(&sh->q_empty, 1);
    mbar_init(&sh->done, 1);
    mbar_init(&sh->clean_go, 1);
    mbar_init(&sh->clean_done, 2);
    for (int u = 0; u < 2; ++u) {
      mbar_init(&sh->s_full[u], 1);
      mbar_init(&sh->o_full[u], 1);
      mbar_init(&sh->p_ready[u], kTile);
    }
    sh->abort = 0;
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may come up; it waits for this grid's end
  int64_t g0, g1;
  const int n = plan<MODE>(C, sh, g0, g1);
  if (threadIdx.x == 0 && g0 >= g1) reinterpret_cast<Part*>(C.ws)[blockIdx.x].parts = 0;
  if (g0 >= g1) return;
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh->tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  Cursor<MODE> cur;
  const int64_t x0 = sh->st_x;
  cur.start(C, sh->st_i, sh->st_h, sh->st_t, x0, g1 - g0);
  if (threadIdx.x == 0) {
    // The item this CTA's start cuts is joined by merge block blockIdx.x, if the boundary before lies in
    // front of it (else an earlier boundary cuts it too).
    Part d{};
    if (cur.k0 > 0) {
      const int64_t total = sh->total;
      const int64_t first = g0 - x0;
      const int c = blockIdx.x;
      if (cut_at(cur.s, cur.tiles(), boundary(c - 1, total, n) - first, cur.nb) == 0) {
        int e = c;
        while (e + 1 < n && cut_at(cur.s, cur.tiles(), boundary(e + 1, total, n) - first, cur.nb) < cur.nb) ++e;
        d.parts = e - c + 2;
        d.row0 = cur.s.row0 + (cur.t << C.lg);
        d.rows = cur.tokens() * C.hg;
        d.head = cur.h * C.hg;
      }
    }
    reinterpret_cast<Part*>(C.ws)[blockIdx.x] = d;
  }
  if constexpr (MODE == kDequant) {
    // registers of the launch: 512 x 128 = 128 x (2 x 168 + 96 + 80)
    if (warp < 8) {
      reg_inc<168>();
      softmax_role<MODE>(C, sh, sq, cur, warp >> 2);
    } else if (warp < 12) {
      reg_dec<96>();
      dequant_role(C, sh, ring, codes, cur);
    } else {
      reg_dec<80>();
      if (warp == 12) {
        if (lane == 0) load_role<MODE>(C, M, sh, sq, ring, codes, cur);
      } else if (warp == 13) {
        mma_role<MODE>(C, sh, sq, ring, cur, lane);
      } else {
        clean_role<MODE>(C, sh, ring, warp - 14, lane);
      }
    }
  } else {
    // 384 x 168 = 128 x (2 x 208 + 88)
    if (warp < 8) {
      reg_inc<208>();
      softmax_role<MODE>(C, sh, sq, cur, warp >> 2);
    } else {
      reg_dec<88>();
      if (warp == 8) {
        if (lane == 0) load_role<MODE>(C, M, sh, sq, ring, codes, cur);
      } else if (warp == 9) {
        mma_role<MODE>(C, sh, sq, ring, cur, lane);
      } else {
        clean_role<MODE>(C, sh, ring, warp - 10, lane);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sh->tmem));
}

// Join the parts of the items that CTA boundaries cut: block (c, y) takes kJoinRows rows of the item that
// boundary c cuts first. Part 0 is slot 1 of CTA c - 1, part p slot 0 of CTA c - 1 + p.
//
// What bounds it is the wait for its loads: a warp takes two rows, two parts of each in flight. Few registers
// (many blocks at once) count for more than deep loads: four rows and four parts at a time take 9 us more on
// the ragged batch of 12 (142 us), one row and eight parts 6 us; with one part after another, the way from
// 64 tokens after 500 is 7 us longer (21 us).
constexpr int kJoinEach = 2, kJoinDepth = 2, kJoinRows = 8 * kJoinEach;
__global__ void __launch_bounds__(256) k_chunk_join(const __grid_constant__ ChunkArgs C) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while k_chunk still runs
  const Part d = reinterpret_cast<const Part*>(C.ws)[blockIdx.x];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = blockIdx.y * kJoinRows + warp;
  if (d.parts == 0 || row0 >= d.rows) return;
  const float* slots = reinterpret_cast<const float*>(C.ws + (size_t)kMaxCtas * kDescBytes);
  const size_t slot = (size_t)C.rows * (kHeadDim + 2);
  auto part = [&](int p) { return slots + ((size_t)(blockIdx.x - 1 + p) * 2 + (p == 0 ? 1 : 0)) * slot; };
  float M[kJoinEach], l[kJoinEach];
  float4 acc[kJoinEach];
#pragma unroll
  for (int r = 0; r < kJoinEach; ++r) {
    M[r] = -INFINITY;
    l[r] = 0.f;
    acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int p0 = 0; p0 < d.parts; p0 += kJoinDepth) {
    float2 ml[kJoinEach][kJoinDepth];
    float4 o[kJoinEach][kJoinDepth];
#pragma unroll
    for (int i = 0; i < kJoinDepth; ++i) {
#pragma unroll
      for (int r = 0; r < kJoinEach; ++r) {
        const int row = row0 + 8 * r;
        ml[r][i] = make_float2(-INFINITY, 0.f);  // as of a part that saw no key
        o[r][i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p0 + i < d.parts && row < d.rows) {
          const float* s = part(p0 + i);
          ml[r][i] = *reinterpret_cast<const float2*>(s + (size_t)C.rows * kHeadDim + 2 * row);
          o[r][i] = *reinterpret_cast<const float4*>(s + (size_t)row * kHeadDim + 4 * lane);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kJoinEach; ++r) {
      float top = M[r];
#pragma unroll
      for (int i = 0; i < kJoinDepth; ++i) top = fmaxf(top, ml[r][i].x);
      const float old = M[r] == -INFINITY ? 0.f : fast_exp2(M[r] - top);
      M[r] = top;
      l[r] *= old;
      acc[r] = make_float4(acc[r].x * old, acc[r].y * old, acc[r].z * old, acc[r].w * old);
#pragma unroll
      for (int i = 0; i < kJoinDepth; ++i) {
        if (ml[r][i].x == -INFINITY && ml[r][i].y == 0.f) continue;
        const float w = fast_exp2(ml[r][i].x - M[r]);
        l[r] += w * ml[r][i].y;
        acc[r].x += w * o[r][i].x;
        acc[r].y += w * o[r][i].y;
        acc[r].z += w * o[r][i].z;
        acc[r].w += w * o[r][i].w;
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kJoinEach; ++r) {
    const int row = row0 + 8 * r;
    if (row >= d.rows) break;
    const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
    const __nv_bfloat162 a = __floats2bfloat162_rn(acc[r].x * inv, acc[r].y * inv), b = __floats2bfloat162_rn(acc[r].z * inv, acc[r].w * inv);
    __nv_bfloat16* dst = C.out + ((int64_t)(d.row0 + row / C.hg) * C.Hq + d.head + row % C.hg) * kHeadDim + 4 * lane;
    *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}

// ------------------------------------------------------------------------------------------------
bool map_rows(CUtensorMap* m, const void* base, int heads, int64_t tokens, int64_t token_stride, int box_heads, int box_tokens) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)kHeadDim * 2, (cuuint64_t)token_stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens}, estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Swizzled pages as rows of 128 dims, copied as they lie: 64 rows x 64 dims a box.
bool map_pages(CUtensorMap* m, const void* base, int64_t rows) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)kHeadDim, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)kHeadDim * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)kPage}, estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int slot_rows(int hg, int64_t n_tokens) { return n_tokens * hg <= kTile ? kTile : 2 * kTile; }

int log2_of(int x) { return x <= 1 ? 0 : 1 + log2_of(x / 2); }

void set_buffers(ChunkArgs& C, void* workspace, void* out) {
  C.lg = log2_of(2 * kTile / C.hg);
  C.out = static_cast<__nv_bfloat16*>(out);
  C.wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
  C.ws = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(workspace) + 31) & ~(uintptr_t)31);  // slots of 32-byte stores
}

// One CTA per SM of the current device (0: a CUDA call failed); the kernel's shared memory is asked
// for on the first call per device.
template <int MODE>
int chunk_ctas() {
  constexpr int kDevices = 64;
  static std::atomic<int> ctas[kDevices];  // 0: not set up
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < kDevices && (sms = ctas[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaFuncSetAttribute(k_chunk<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kChunkSmem<MODE>) != cudaSuccess)
    return 0;
  sms = sms < kMaxCtas ? sms : kMaxCtas;
  if (dev < kDevices) ctas[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

template <int MODE>
cudaError_t launch_chunk(const ChunkArgs& C, const ChunkMaps& M, cudaStream_t s) {
  const int ctas = chunk_ctas<MODE>();
  if (ctas < 1) return cudaErrorUnknown;
  k_chunk<MODE><<<ctas, kChunkThreads<MODE>, kChunkSmem<MODE>, s>>>(C, M);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || ctas == 1) return e;
  // its launch overlaps the end of k_chunk
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t join{};
  join.gridDim = dim3(ctas, C.rows / kJoinRows);
  join.blockDim = dim3(256);
  join.stream = s;
  join.attrs = &early;
  join.numAttrs = 1;
  return cudaLaunchKernelEx(&join, k_chunk_join, C);
}

}  // namespace

// Partials of a call: two slots per CTA (an item cut in front of the CTA's range, and one behind it).
size_t chunk_workspace_bytes(int hg, int64_t n_tokens) {
  return 32 + (size_t)kMaxCtas * (kDescBytes + 2 * (size_t)slot_rows(hg, n_tokens) * (kHeadDim + 2) * 4);
}

cudaError_t launch_chunk_pool(const DevPool& P, const StepDims& S, int layer, bool skip_single, const ChunkTiles* tiles,
                              const void* q, const void* k_new, const void* v_new, void* workspace, void* out, cudaStream_t s) {
  ChunkArgs C{};
  C.Hq = P.Hq;
  C.Hkv = P.Hkv;
  C.hg = P.hg;
  C.n_seqs = S.n_seqs;
  C.n_tokens = S.total_new;
  C.rows = slot_rows(P.hg, S.total_new);
  C.P = P;
  C.layer = layer;
  C.skip_single = skip_single;
  C.v_new = static_cast<const __nv_bfloat16*>(v_new);
  set_buffers(C, workspace, out);
  C.err = P.err;
  ChunkMaps M;
  std::memset(&M, 0, sizeof(M));
  const int64_t T = S.total_new, sink_rows = (int64_t)P.max_sink_pages * P.Hkv * kPage, ring_rows = (int64_t)P.max_seqs * P.Hkv * kRecent;
  if (!map_rows(&M.q, q, P.Hq, T, (int64_t)P.Hq * kHeadDim, P.hg, kTile / P.hg) ||
      !map_rows(&M.k, k_new, P.Hkv, T, (int64_t)P.Hkv * kHeadDim, 1, kPage) ||
      !map_rows(&M.v, v_new, P.Hkv, T, (int64_t)P.Hkv * kHeadDim, 1, kPage) ||
      !map_pages(&M.sink_k, P.sink_k + (size_t)layer * P.sink_layer_stride, sink_rows) ||
      !map_pages(&M.sink_v, P.sink_v + (size_t)layer * P.sink_layer_stride, sink_rows) ||
      !map_pages(&M.ring_k, P.ring_k + (size_t)layer * P.ring_layer_stride, ring_rows) ||
      !map_pages(&M.ring_v, P.ring_v + (size_t)layer * P.ring_layer_stride, ring_rows))
    return cudaErrorUnknown;
  if (!tiles) return launch_chunk<kDequant>(C, M, s);
  C.tiles = tiles->tiles;
  C.tile_base = tiles->base;
  return launch_chunk<kTiles>(C, M, s);
}

}  // namespace oscar

using namespace oscar;

extern "C" {

size_t oscar_bf16_chunk_workspace_bytes(int32_t num_q_heads, int32_t num_kv_heads, int32_t n_seqs, int32_t n_tokens) {
  if (num_kv_heads < 1 || num_q_heads < 1 || num_q_heads % num_kv_heads || n_seqs < 1 || n_tokens < 0) return 0;
  const int hg = num_q_heads / num_kv_heads;
  if (hg != 1 && hg != 2 && hg != 4 && hg != 8 && hg != 16) return 0;
  return chunk_workspace_bytes(hg, n_tokens);
}

oscar_status oscar_bf16_chunk(int32_t num_q_heads, int32_t num_kv_heads, int32_t n_seqs, int32_t n_tokens,
                              const void* k_pages, const void* v_pages, int64_t n_pages_total, const int32_t* page_table,
                              int32_t max_pages_per_seq, const int32_t* lengths, const int32_t* cu_tokens, const void* q,
                              int64_t q_token_stride, void* workspace, size_t workspace_bytes, void* out, uint32_t* err,
                              void* stream) {
  const size_t need = oscar_bf16_chunk_workspace_bytes(num_q_heads, num_kv_heads, n_seqs, n_tokens);
  if (!need) return OSCAR_EINVAL;
  if (n_tokens == 0) return OSCAR_OK;
  if (!k_pages || !v_pages || !page_table || !lengths || !cu_tokens || !q || !workspace || !out || !err) return OSCAR_EINVAL;
  if (((reinterpret_cast<uintptr_t>(k_pages) | reinterpret_cast<uintptr_t>(v_pages) | reinterpret_cast<uintptr_t>(q) |
        reinterpret_cast<uintptr_t>(workspace) | reinterpret_cast<uintptr_t>(out)) & 15) != 0)
    return OSCAR_EINVAL;  // read and written in 16-byte pieces
  if (((reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(lengths) | reinterpret_cast<uintptr_t>(cu_tokens) |
        reinterpret_cast<uintptr_t>(err)) & 3) != 0)
    return OSCAR_EINVAL;
  if (q_token_stride % 8 || q_token_stride < (int64_t)num_q_heads * kHeadDim || q_token_stride >= (1ll << 38)) return OSCAR_EINVAL;
  // rows of the page buffers are addressed by 31-bit coordinates (549 GB of K)
  if (workspace_bytes < need || n_pages_total < 1 || n_pages_total > INT32_MAX / kPage / num_kv_heads || max_pages_per_seq < 1 ||
      max_pages_per_seq > (INT32_MAX - 4096) / kPage)  // positions and a few tiles beyond them are 32-bit
    return OSCAR_EINVAL;
  ChunkArgs C{};
  C.Hq = num_q_heads;
  C.Hkv = num_kv_heads;
  C.hg = num_q_heads / num_kv_heads;
  C.n_seqs = n_seqs;
  C.n_tokens = n_tokens;
  C.rows = slot_rows(C.hg, n_tokens);
  C.page_table = page_table;
  C.lengths = lengths;
  C.cu = cu_tokens;
  C.v_pages = static_cast<const uint8_t*>(v_pages);
  C.max_pages = max_pages_per_seq;
  C.n_pages_total = n_pages_total;
  set_buffers(C, workspace, out);
  C.err = err;
  ChunkMaps M;
  std::memset(&M, 0, sizeof(M));
  const int64_t rows = n_pages_total * num_kv_heads * kPage;
  if (!map_rows(&M.q, q, num_q_heads, n_tokens, q_token_stride, C.hg, kTile / C.hg) || !map_pages(&M.k, k_pages, rows) ||
      !map_pages(&M.v, v_pages, rows))
    return OSCAR_ECUDA;
  const cudaError_t e = launch_chunk<kBf16>(C, M, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return OSCAR_ECUDA;
  }
  return OSCAR_OK;
}

}  // extern "C"

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
// row) turn S into P, the tensor cores run the other tile's products. A tile costs 2 x 512 cycles of
// tensor core per 128 keys and as many exponentials per row; both bound the long chunks.
//
// Keys come in blocks of 128 (two half blocks of 64, each a page or a run of rows):
//   pages of the BF16 cache, the pool's sink page and ring pages   tensor copies of a page's two 64-dim
//       halves: the page's own swizzle (chunk c of token t at c ^ (t & 7)) is the 128-byte swizzle the
//       tensor cores read, so a page is used as it lies
//   the chunk's own rows (pool)       tensor copies with the 128-byte swizzle
//   INT2 history (pool)               four warps turn the codes into fp16 tiles of the same layout
// The INT2 blocks come first. For them Q is rotated on the tensor cores (Q R_K, R in two bf16 limbs)
// and kept as fp16 with a power of two per row, k^ and v^ = fp16(level * s + z) and P are fp16, and
// O is in the rotated basis: behind the last INT2 block it is split into two bf16 limbs and
// multiplied by R_V^T in place (three products), and the BF16 blocks follow with the plain Q.
//
// Work: unit = one key block of one item (sequence, KV head, pair of tiles). The units of the whole
// call are one range, cut into equal parts for the CTAs; an item cut by a boundary leaves one
// partial (maximum, sum, unnormalised O) per part, and a second kernel joins them. This keeps every
// SM busy for one long sequence with few rows as for a ragged batch, and needs nothing from the host:
// lengths are read on the device, so a captured call follows them.
//
// Keys no row may see, and what lies behind a sequence's last key, must not reach a sum even as 0 *
// NaN: such values are zeroed in shared memory before the product. Where some rows of the tile see
// a key and others do not (the diagonal), a non-finite value element is zeroed too, noted, and added
// at the end to the rows that do see it.
#include <cstring>

#include "tcgen05.cuh"

namespace oscar {
namespace {

constexpr int kTile = 128;                    // rows of a tile, keys of a block
constexpr int kHalfBytes = kTile * 128;       // 64 dims of 128 rows
constexpr int kTileBytes = 2 * kHalfBytes;    // 128 x 128 16-bit values
constexpr int kStages = 5;                    // K / V tiles in flight
constexpr int kMaxCtas = 152;
constexpr int kPageHalfBytes = kPage * 128;   // 64 dims of one page
constexpr float kLazy = 8.f;                  // the maximum may lag by 2^8 before O is rescaled
constexpr int kDescBytes = 32;
constexpr int kMinUnits = 2;                  // key blocks per CTA, at least, before a call is cut further

constexpr uint32_t kIdescBase = (1u << 4) | ((uint32_t)(kTile >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
constexpr uint32_t kIdescBf16 = kIdescBase | (1u << 7) | (1u << 10);  // A, B bf16; fp16 without these bits
constexpr uint32_t kIdescMn = 1u << 16;                               // B with its N axis contiguous

// Lower descriptor words of 128-byte-swizzled tiles: K-major (row r of a 64-dim half at r * 128), and
// the same bytes read with the other axis contiguous (leading offset: the next 64 of N).
__device__ __forceinline__ uint32_t desc_k(uint32_t a) { return (a >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t a) { return (a >> 4) | ((uint32_t)(kHalfBytes >> 4) << 16); }

struct ChunkArgs {
  int32_t Hq, Hkv, hg, n_seqs, n_tokens, rows;  // rows: rows of a partial slot
  // BF16-only cache
  const int32_t *page_table, *lengths, *cu;
  const uint8_t* v_pages;
  int32_t max_pages;
  int64_t n_pages_total;
  // pool
  DevPool P;
  int32_t layer;
  const __nv_bfloat16* v_new;
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
};

template <bool MIXED>
__device__ __forceinline__ SeqWork load_seq(const ChunkArgs& C, int i) {
  SeqWork s{};
  if constexpr (MIXED) {
    const StepSeq& st = C.P.step[i];
    s.n = st.L_new - st.L_old;
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

// Key blocks that tile pair t of a sequence really has, and the units it counts for (at least one).
__device__ __forceinline__ int real_blocks(const SeqWork& s, int bt, int t) {
  const int keys = s.A + min(s.n, bt * (t + 1));
  return s.nI + s.nB + (keys > 0 ? (keys + kTile - 1) / kTile : 0);
}

// Units of the tile pairs 0 .. t-1, all of them full (bt tokens, a power of two up to 256):
// sum over u < t of max(1, pre + ceil((A + bt (u + 1)) / 128)).
__device__ __forceinline__ int64_t units_before(const SeqWork& s, int bt, int64_t t) {
  const int64_t n0 = s.A < 0 ? min((int64_t)(-s.A / bt), t) : 0;  // pairs without a key
  const int64_t m = t - n0, c = s.A + bt * n0 + bt + kTile - 1, q = c >> 7;
  int64_t sum = n0 + m * (s.nI + s.nB + q);
  if (bt >= kTile) return sum + (bt / kTile) * (m * (m - 1) / 2);
  const int r = kTile / bt, d = (int)(c & 127), w0 = (kTile - d + bt - 1) / bt;  // remainders >= w0 carry
  const int64_t M = m / r, rem = m - M * r;
  return sum + r * (M * (M - 1) / 2) + M * (r - w0) + rem * M + max((int64_t)0, rem - w0);
}
__device__ __forceinline__ int pairs_of(const SeqWork& s, int bt) { return (s.n + bt - 1) / bt; }
__device__ __forceinline__ int64_t units_of(const SeqWork& s, int bt) {  // of one KV head
  const int T = pairs_of(s, bt);
  return T ? units_before(s, bt, T - 1) + max(1, real_blocks(s, bt, T - 1)) : 0;
}

// A place in the order (sequence, KV head, tile pair, block), moved segment by segment.
template <bool MIXED>
struct Cursor {
  SeqWork s;
  int i, h, t, k0, k1, nb;  // the segment: blocks [k0, k1) of nb
  int64_t left;             // units from k0 on
  int bt;

  __device__ __forceinline__ void start(const ChunkArgs& C, int i_, int h_, int t_, int k, int64_t n) {
    bt = 2 * kTile / C.hg;
    i = i_;
    h = h_;
    t = t_;
    k0 = k;
    left = n;
    if (left > 0) {
      s = load_seq<MIXED>(C, i);
      fit();
    }
  }
  __device__ __forceinline__ void fit() {
    nb = max(1, real_blocks(s, bt, t));
    k1 = (int)min((int64_t)nb, k0 + left);
  }
  __device__ __forceinline__ bool valid() const { return left > 0; }
  __device__ __forceinline__ void next(const ChunkArgs& C) {
    left -= k1 - k0;
    if (left <= 0) return;
    k0 = 0;
    if (++t >= pairs_of(s, bt)) {
      t = 0;
      if (++h >= C.Hkv) {
        h = 0;
        do {
          ++i;
          s = load_seq<MIXED>(C, i);
        } while (s.n == 0 && i + 1 < C.n_seqs);
      }
    }
    fit();
  }
  __device__ __forceinline__ bool empty() const { return real_blocks(s, bt, t) == 0; }
  __device__ __forceinline__ int tokens() const { return min(bt, s.n - t * bt); }
  __device__ __forceinline__ bool two() const { return tokens() > bt / 2; }  // the second tile has rows
};

// Where one half block of 64 keys comes from, and its slots [lo, hi) that hold keys for anyone.
struct Half {
  int lo, hi;
  int pos;  // BF16 cache: page index; pool: first chunk row, or position of slot 0 in the ring, -1 the sink
};
template <bool MIXED>
__device__ __forceinline__ Half half_of(const SeqWork& s, int k, int half) {
  Half r;
  if (MIXED && k < s.nI) {
    const int j = 2 * k + half;
    r.lo = 0;
    r.hi = min(max(s.hist - j * kPage, 0), kPage);
    r.pos = j;
  } else if (MIXED && k < s.nI + s.nB) {
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
struct Shared {
  uint64_t full[kStages], empty[kStages];
  uint64_t q_full, q_empty, s_full[2], p_ready[2], done;
  uint32_t tmem;
  int32_t abort;
  // plan
  int64_t total, scan[16];
  int32_t st_i, st_h, st_t, st_k;
  // non-finite values of the diagonal blocks: key bits per block, two segments in turn
  uint32_t bad[2][4][4];
  uint32_t any_bad[2];
};
static_assert(sizeof(Shared) <= 1024, "Shared");
constexpr int kChunkSmem = 2 * kTileBytes + kStages * kTileBytes + 1024 + 1024;

// Bounded wait that also ends when another role gave up.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, Shared* sh, uint32_t* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile int32_t*>(&sh->abort)) return false;
    if (clock64() - t0 >= kWaitCycles) break;
  }
  *reinterpret_cast<volatile int32_t*>(&sh->abort) = 1;
  set_err(err, OSCAR_DEVERR_TIMEOUT);
  return false;
}
// The same for a whole warp, which leaves it converged (tensor-memory instructions and aligned
// barriers follow).
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Shared* sh, uint32_t* err) {
  const bool ok = wait_bar(bar, parity, sh, err);
  __syncwarp();
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// AND over the four warps of the dequantising group (named barrier 1).
__device__ __forceinline__ bool and128(bool v) {
  uint32_t out;
  __syncwarp();
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.and.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(out)
      : "r"((uint32_t)v)
      : "memory");
  return out != 0;
}

struct Ring {  // position in the stream of K / V tiles
  uint32_t pos = 0;
  __device__ __forceinline__ int stage() const { return pos % kStages; }
  __device__ __forceinline__ uint32_t parity() const { return (pos / kStages) & 1; }
};

// The two limb tiles of a rotation matrix.
constexpr int kLimbs = 2;

// ---- tensor-copy warp --------------------------------------------------------------------------
template <bool MIXED>
__device__ void load_role(const ChunkArgs& C, const ChunkMaps& M, Shared* sh, uint8_t* sq, uint8_t* ring, Cursor<MIXED> cur) {
  // one lane
  const uint64_t keep = policy_evict_last(), once = policy_evict_first();
  Ring r;
  uint32_t issued = 0, qn = 0;  // bit s: stage s has had a tensor copy
  uint32_t last_parity = 0;
  bool ok = true;
  auto load_q = [&]() {
    if (qn && !wait_bar(&sh->q_empty, (qn - 1) & 1, sh, C.err)) return false;
    const int tiles = cur.two() ? 2 : 1, tok = cur.s.row0 + cur.t * cur.bt;
    mbar_expect_tx(&sh->q_full, tiles * kTileBytes);
    for (int u = 0; u < tiles; ++u)
      for (int d = 0; d < 2; ++d)
        tma_load_3d(sq + u * kTileBytes + d * kHalfBytes, &M.q, d * 64, cur.h * C.hg, tok + u * (cur.bt / 2), &sh->q_full, once);
    ++qn;
    return true;
  };
  auto stage = [&](uint8_t*& dst, uint64_t*& bar) {
    const int s = r.stage();
    if (!wait_bar(&sh->empty[s], r.parity() ^ 1, sh, C.err)) return false;
    dst = ring + s * kTileBytes;
    bar = &sh->full[s];
    issued |= 1u << s;
    last_parity = (last_parity & ~(1u << s)) | (r.parity() << s);
    ++r.pos;
    return true;
  };
  // Tiles that the dequantising warps fill: their stages are waited for all the same, since a parity
  // tells the phase of a barrier only to a role that has seen every phase of it.
  auto skip = [&](int n) {
    for (; n > 0; --n, ++r.pos)
      if (!wait_bar(&sh->empty[r.stage()], r.parity() ^ 1, sh, C.err)) return false;
    return true;
  };
  auto load_limbs = [&](int kv) {
    const uint8_t* src = C.P.rlimbs + ((size_t)(C.layer * C.P.Hkv + cur.h) * 2 + kv) * (kLimbs * kTileBytes);
    for (int l = 0; l < kLimbs; ++l) {
      uint8_t* dst;
      uint64_t* bar;
      if (!stage(dst, bar)) return false;
      mbar_expect_tx(bar, kTileBytes);
      bulk_g2s(dst, src + l * kTileBytes, kTileBytes, bar, keep);
    }
    return true;
  };
  auto load_block = [&](int k) {
    Half hf[2];
    int row[2];
    const CUtensorMap* map[2][2];
    bool rows3 = false;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      hf[x] = half_of<MIXED>(cur.s, k, x);
      if constexpr (MIXED) {
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
      mbar_expect_tx(bar, n * 2 * kPageHalfBytes);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (hf[x].hi <= hf[x].lo) continue;
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          uint8_t* to = dst + d * kHalfBytes + x * kPageHalfBytes;
          if (MIXED && rows3)
            tma_load_3d(to, map[x][kv], d * 64, cur.h, row[x], bar, keep);
          else
            tma_load_2d(to, map[x][kv], d * 64, row[x], bar, keep);
        }
      }
    }
    return true;
  };
  for (; ok && cur.valid(); cur.next(C)) {
    if (cur.empty()) continue;
    const int nI = MIXED ? min(cur.k1, cur.s.nI) : 0;
    if (cur.k0 < nI) {
      ok = load_q() && load_limbs(0) && skip(2 * (nI - cur.k0)) && (C.P.absorbed || load_limbs(1));
    }
    const int kb = max(cur.k0, nI);
    if (ok && kb < cur.k1) {
      ok = load_q();
      for (int k = kb; ok && k < cur.k1; ++k) ok = load_block(k);
    }
  }
  if (!ok) {  // never leave with a copy in flight
    for (int s = 0; s < kStages; ++s)
      if ((issued >> s) & 1) mbar_wait(&sh->full[s], (last_parity >> s) & 1, C.err);
    if (qn) mbar_wait(&sh->q_full, (qn - 1) & 1, C.err);
  }
}

// ---- tensor-core warp --------------------------------------------------------------------------
// Zero the rows of a V tile that nobody may see, and on the diagonal the non-finite values of the
// others, whose keys are returned as bits (per lane group, OR-ed by the caller).
__device__ __forceinline__ void clean_v(uint8_t* tile, uint64_t live0, uint64_t live1, bool diagonal, uint32_t (&bad)[4], int lane) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t live = (uint32_t)((w & 2 ? live1 : live0) >> (32 * (w & 1)));
    uint32_t b = 0;
    if (live != 0xFFFFFFFFu || diagonal) {
#pragma unroll 4
      for (int it = 0; it < 16; ++it) {  // 32 rows x 16 chunks: a lane takes one chunk of 4 rows apart
        const int row = it * 2 + (lane >> 4), c = lane & 15;
        uint4* p = reinterpret_cast<uint4*>(tile + (c >> 3) * kHalfBytes + (w * 32 + row) * 128 + (c & 7) * 16);
        if (!((live >> row) & 1)) {
          *p = make_uint4(0, 0, 0, 0);
        } else if (diagonal) {
          uint4 v = *p;
          uint32_t* e = reinterpret_cast<uint32_t*>(&v);
          bool hit = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if ((e[i] & 0x7F80u) == 0x7F80u) {
              e[i] &= 0xFFFF0000u;
              hit = true;
            }
            if ((e[i] & 0x7F800000u) == 0x7F800000u) {
              e[i] &= 0xFFFFu;
              hit = true;
            }
          }
          if (hit) {
            *p = v;
            b |= 1u << row;
          }
        }
      }
    }
    bad[w] = __reduce_or_sync(0xffffffffu, b);
  }
  fence_proxy_async();
  __syncwarp();
}

template <bool MIXED>
__device__ void mma_role(const ChunkArgs& C, Shared* sh, uint8_t* sq, uint8_t* ring, Cursor<MIXED> cur, int lane) {
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh->tmem, 0), aq = smem_u32(sq), ar = smem_u32(ring);
  const uint32_t one = elect_one();
  Ring r;
  uint32_t qn = 0, pn[2] = {0, 0}, seg = 0;
  bool ok = true;
  auto S = [&](int u) { return tmem + (uint32_t)(u * kTile); };
  auto O = [&](int u) { return tmem + (uint32_t)(2 * kTile + u * kTile); };
  auto wait_full = [&](uint32_t pos) {
    const bool w = wait_warp(&sh->full[pos % kStages], (pos / kStages) & 1, sh, C.err);
    tc_fence_after();
    return w;
  };
  auto wait_p = [&](int u) {
    const bool w = wait_warp(&sh->p_ready[u], pn[u]++ & 1, sh, C.err);
    tc_fence_after();
    return w;
  };
  auto addr = [&](uint32_t pos) { return ar + (__shfl_sync(0xffffffffu, pos, 0) % kStages) * kTileBytes; };
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
    const int nI = MIXED ? min(cur.k1, cur.s.nI) : 0;
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
      commit(&sh->empty[kpos % kStages]);
      if (a + 1 == b) commit(&sh->q_empty);
      for (int k = a; k < b; ++k) {
        const uint32_t vpos = kpos + 1;
        if (!wait_full(vpos)) return false;
        if (idesc == kIdescBf16) {
          // causal blocks are those behind the cached ones; the diagonal starts where the pair's first
          // row ends
          const int j = k - cur.s.nI - cur.s.nB, j0 = max(cur.s.A + cur.t * cur.bt + 1, 0) / kTile;
          const bool diagonal = j >= j0;
          const Half h0 = half_of<MIXED>(cur.s, k, 0), h1 = half_of<MIXED>(cur.s, k, 1);
          const uint64_t l0 = bits(h0.lo, h0.hi), l1 = bits(h1.lo, h1.hi);
          if (diagonal || (l0 & l1) != ~0ull) {
            uint32_t bad[4];
            clean_v(ring + (vpos % kStages) * kTileBytes, l0, l1, diagonal, bad, lane);
            if (diagonal && (bad[0] | bad[1] | bad[2] | bad[3])) {
              if (lane < 4) sh->bad[sb][j - j0][lane] = bad[lane];
              if (lane == 0) sh->any_bad[sb] = 1;
              __syncwarp();
            }
          }
        }
        for (int u = 0; u < tiles; ++u) {
          if (!wait_p(u)) return false;
          pv(u, S(u), addr(vpos), idesc, acc);
          if (k + 1 < b) {
            if (u == 0 && !wait_full(vpos + 1)) return false;
            qk(u, addr(vpos + 1), idesc, false);
          }
          commit(&sh->s_full[u]);  // the next S, or behind the last block O
        }
        acc = true;
        commit(&sh->empty[vpos % kStages]);
        kpos = vpos + 1;
        if (k + 1 < b) commit(&sh->empty[kpos % kStages]);
        if (k + 2 == b) commit(&sh->q_empty);
      }
      r.pos = kpos;
      return true;
    };
    if (MIXED && cur.k0 < nI) {
      ok = wait_warp(&sh->q_full, qn++ & 1, sh, C.err) && wait_full(r.pos) && wait_full(r.pos + 1);
      if (!ok) break;
      for (int u = 0; u < tiles; ++u) {
        qk(u, addr(r.pos), kIdescBf16, false);
        qk(u, addr(r.pos + 1), kIdescBf16, true);
        commit(&sh->s_full[u]);
      }
      commit(&sh->empty[r.pos % kStages]);
      commit(&sh->empty[(r.pos + 1) % kStages]);
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
          if (nI == cur.k1) commit(&sh->s_full[u]);
        }
        commit(&sh->empty[r.pos % kStages]);
        commit(&sh->empty[(r.pos + 1) % kStages]);
        r.pos += kLimbs;
      }
    }
    const int kb = max(cur.k0, nI);
    if (ok && kb < cur.k1) ok = wait_warp(&sh->q_full, qn++ & 1, sh, C.err) && blocks(kb, cur.k1, kIdescBf16);
    if (ok && tiles == 1) ok = wait_p(1);
  }
  // no product in flight when the tensor memory is given back
  commit(&sh->done);
  mbar_wait(&sh->done, 0, C.err);
}

// ---- softmax warps: one thread per row -----------------------------------------------------------
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <bool MIXED>
__device__ void softmax_role(const ChunkArgs& C, Shared* sh, uint8_t* sq, Cursor<MIXED> cur, int u) {
  const int row = threadIdx.x & 127, warp = row >> 5;
  const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
  const uint32_t tS = sh->tmem + lane_off + u * kTile, tO = sh->tmem + lane_off + 2 * kTile + u * kTile;
  uint32_t sn = 0, seg = 0;
  bool ok = true;
  const int hg = C.hg, tpt = kTile / hg;
  auto wait_s = [&]() {
    const bool w = wait_warp(&sh->s_full[u], sn++ & 1, sh, C.err);
    tc_fence_after();
    return w;
  };
  auto ready = [&]() {
    tc_fence_before();
    mbar_arrive(&sh->p_ready[u]);
  };
  auto load_s = [&](uint32_t (&s)[4][32]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) tc_ld32_issue(tS + 32 * c, s[c]);
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int c = 0; c < 4; ++c) tc_ld_wait_pass(s[c]);
  };

  for (; ok && cur.valid(); cur.next(C)) {
    const int tok = cur.t * cur.bt + u * tpt + row / hg;  // this row's token of the sequence
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
    const int nI = MIXED ? min(cur.k1, cur.s.nI) : 0;
    float m = -INFINITY, l = 0.f;
    bool have = false;  // O holds something

    auto block = [&](int k, float scale, bool half16) {
      if (!wait_s()) return false;
      uint32_t s[4][32];
      load_s(s);
      // the columns this row may see
      uint64_t b0 = ~0ull, b1 = ~0ull;
      bool masked;
      if (MIXED && k < cur.s.nI + cur.s.nB) {
        const Half h0 = half_of<MIXED>(cur.s, k, 0), h1 = half_of<MIXED>(cur.s, k, 1);
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
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t b = (uint32_t)((c & 2 ? b1 : b0) >> (32 * (c & 1)));
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!((b >> i) & 1)) s[c][i] = 0xFF800000u;
        }
      }
      float mx[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mx[c] = __uint_as_float(s[c][0]);
#pragma unroll
        for (int i = 1; i < 31; i += 2) mx[c] = max3(mx[c], __uint_as_float(s[c][i]), __uint_as_float(s[c][i + 1]));
        mx[c] = fmaxf(mx[c], __uint_as_float(s[c][31]));
      }
      const float mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
      // the maximum moves only when it would grow by more than 2^kLazy; sums stay far inside fp32
      const bool move = mb > m + kLazy || (m == -INFINITY && mb > m);
      if (__any_sync(0xffffffffu, move)) {
        const float mn = move ? mb : m, alpha = move ? fast_exp2(m - mn) : 1.f;
        m = mn;
        l *= alpha;
        if (have) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tc_ld32_issue(tO + 32 * c, o);
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
            tc_ld_wait_pass(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tc_st32(tO + 32 * c, o);
          }
        }
      }
      const float nm = m == -INFINITY ? 0.f : -m;
      // two scores an instruction, but for the exponentials
      const float2 sc2 = make_float2(scale, scale), nm2 = make_float2(nm, nm);
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t p[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float2 x = __ffma2_rn(make_float2(__uint_as_float(s[c][2 * i]), __uint_as_float(s[c][2 * i + 1])), sc2, nm2);
          x.x = fast_exp2(x.x);
          x.y = fast_exp2(x.y);
          sum[i & 1] = __fadd2_rn(sum[i & 1], x);
          if (MIXED && half16) {
            p[i] = pack_half2(x.x, x.y);
          } else {
            const __nv_bfloat162 w = __floats2bfloat162_rn(x.x, x.y);
            p[i] = *reinterpret_cast<const uint32_t*>(&w);
          }
        }
        tc_st16(tS + 16 * c, p);
      }
      l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
      tc_st_wait();
      ready();
      have = true;
      return true;
    };

    if (MIXED && cur.k0 < nI) {
      // Q R_K: fp16, scaled by the power of two that brings the row's largest value to [1, 2)
      ok = wait_s();
      if (!ok) break;
      float scale = kScoreLog2;
      {
        uint32_t s[4][32];
        load_s(s);
        float mx = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) mx = fmaxf(mx, fabsf(__uint_as_float(s[c][i])));
        const uint32_t e = __float_as_uint(mx) >> 23;
        float down = 1.f;
        if (e > 0 && e < 254) {
          down = __uint_as_float((254 - e) << 23);
          scale *= __uint_as_float(e << 23);
        }
        uint8_t* q = sq + u * kTileBytes + row * 128;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = pack_half2(__uint_as_float(s[c >> 2][(c & 3) * 8 + 2 * i]) * down, __uint_as_float(s[c >> 2][(c & 3) * 8 + 2 * i + 1]) * down);
          *reinterpret_cast<uint4*>(q + (c >> 3) * kHalfBytes + (((c & 7) ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      fence_proxy_async();
      ready();
      for (int k = cur.k0; ok && k < nI; ++k) ok = block(k, scale, true);
      if (!ok) break;
      ok = wait_s();  // O is complete
      if (!ok) break;
      if (!C.P.absorbed) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32], hi[16], lo[16];
          tc_ld32_issue(tO + 32 * c, o);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
          tc_ld_wait_pass(o);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float x = __uint_as_float(o[2 * i]), y = __uint_as_float(o[2 * i + 1]);
            const __nv_bfloat162 a = __floats2bfloat162_rn(x, y);
            const __nv_bfloat162 b = __floats2bfloat162_rn(x - __bfloat162float(a.x), y - __bfloat162float(a.y));
            hi[i] = *reinterpret_cast<const uint32_t*>(&a);
            lo[i] = *reinterpret_cast<const uint32_t*>(&b);
          }
          tc_st16(tS + 16 * c, hi);
          tc_st16(tS + 64 + 16 * c, lo);
        }
        tc_st_wait();
        ready();
      }
    }
    const int kb = max(cur.k0, nI);
    for (int k = kb; ok && k < cur.k1; ++k) ok = block(k, kScoreLog2, false);
    if (!ok) break;
    // O is complete (behind the last INT2 block of an absorbed pool it was waited for above)
    if (kb < cur.k1 || (MIXED && !C.P.absorbed)) ok = wait_s();
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
      asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
      tc_ld_wait_pass(o);
      if (live) {
      float f[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(o[i]);
      if (bad) {  // non-finite values this row does see
        const int j0 = max(cur.s.A + cur.t * cur.bt + 1, 0) / kTile;
        for (int b = 0; b < kTile * 4; ++b) {
          const int key = j0 * kTile + b;
          if (key >= lim || !((sh->bad[sb][b >> 7][(b >> 5) & 3] >> (b & 31)) & 1)) continue;
          const __nv_bfloat16* v;
          int swz = 0;
          if constexpr (MIXED) {
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
        for (int i = 0; i < 4; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(f[8 * i + 2 * e] * inv, f[8 * i + 2 * e + 1] * inv);
            w[e] = *reinterpret_cast<const uint32_t*>(&x);
          }
          reinterpret_cast<uint4*>(dst)[4 * c + i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          reinterpret_cast<float4*>(slot)[8 * c + i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
      }
      }
      __syncwarp();  // the next tensor-memory load is the whole warp's
    }
  }
}

// ---- dequantising warps (pool) -------------------------------------------------------------------
// The four fp16 values a code can stand for in one group, as two words a byte selector picks from.
struct Levels {
  uint32_t a, b;
};
__device__ __forceinline__ Levels levels(uint32_t sz, float l1, float l2) {
  const float s = half_lo(sz), z = half_hi(sz);
  Levels r;
  r.a = pack_half2(z, fmaf(l1, s, z));
  r.b = pack_half2(fmaf(l2, s, z), fmaf(3.f, s, z));
  return r;
}
// Codes 2p of the four bytes of x (elements 0 .. 3) as two f16x2 words.
__device__ __forceinline__ void pick4(uint32_t x, int p, const Levels& t, uint32_t& lo, uint32_t& hi) {
  const uint32_t sel = ((x >> (2 * p)) & 0x03030303u) * 0x22u + 0x10101010u;  // nibbles 2c, 2c + 1 per code
  lo = __byte_perm(t.a, t.b, sel);
  hi = __byte_perm(t.a, t.b, sel >> 16);
}

__device__ void dequant_role(const ChunkArgs& C, Shared* sh, uint8_t* ring, Cursor<true> cur) {
  const int x = threadIdx.x & 127;
  const DevPool& P = C.P;
  const int ng = P.ngroups;
  // K: thread x has token x of the block. V: a slice of 16 tokens, of it tokens 8u + 2tq + {0, 1} and
  // one half of the dims.
  const int slice = x >> 4, tq = (x >> 2) & 3, uu = (x >> 1) & 1, wh = x & 1;
  Ring r;
  bool ok = true;
  auto skip = [&](int n) {  // tiles of the tensor-copy warp (see there)
    for (; n > 0; --n, ++r.pos)
      if (!wait_warp(&sh->empty[r.stage()], r.parity() ^ 1, sh, C.err)) return false;
    return true;
  };
  for (; ok && cur.valid(); cur.next(C)) {
    if (cur.empty()) continue;
    const int nI = min(cur.k1, cur.s.nI);
    if (cur.k0 < nI) {
      ok = and128(skip(kLimbs));
      if (!ok) break;
      const size_t lh = (size_t)C.layer * P.Hkv + cur.h;
      const float ak = P.lloyd ? P.cb_a[lh * 2] : 1.f, av = P.lloyd ? P.cb_a[lh * 2 + 1] : 1.f;
      const float ak2 = 3.f - ak, av2 = 3.f - av;
      const uint8_t* base = P.int2 + (size_t)C.layer * P.int2_layer_stride;
      auto page = [&](int j) -> const uint8_t* {  // page j of the history, null when it has none
        if (j * kPage >= cur.s.hist) return nullptr;
        int64_t pid = P.page_table[(size_t)cur.s.seq * P.maxp + j];
        if (pid < 0 || pid >= P.max_int2_pages) {
          set_err(P.err, OSCAR_DEVERR_PAGE);
          pid = 0;
        }
        return base + ((size_t)pid * P.Hkv + cur.h) * P.block_bytes;
      };
      // the packed words of one block, fetched a block ahead
      uint4 kc[2];
      uint32_t vc[8], ksz[4], vsz[2][2];
      auto fetch = [&](int k) {
        const uint8_t* kp = page(2 * k + (x >> 6));
        const int tau = x & 63;
        kc[0] = kc[1] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) ksz[i] = 0;
        if (kp && (2 * k + (x >> 6)) * kPage + tau < cur.s.hist) {
          kc[0] = reinterpret_cast<const uint4*>(kp + tau * kCodeBytes)[0];
          kc[1] = reinterpret_cast<const uint4*>(kp + tau * kCodeBytes)[1];
          const uint32_t* sz = reinterpret_cast<const uint32_t*>(kp + 2 * kPage * kCodeBytes);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < ng) ksz[i] = sz[sz_index(tau, i, ng)];
        }
        // V: slices 0 .. 3 are the block's first page
        const uint8_t* vp = page(2 * k + (slice >> 2));
#pragma unroll
        for (int i = 0; i < 8; ++i) vc[i] = 0;
        vsz[0][0] = vsz[0][1] = vsz[1][0] = vsz[1][1] = 0;
        if (vp) {
          const uint8_t* c = vp + kPage * kCodeBytes + (slice & 3) * 512 + tq * 16 + 8 * uu + 4 * wh;
#pragma unroll
          for (int g = 0; g < 8; ++g) vc[g] = *reinterpret_cast<const uint32_t*>(c + g * 64);
          const uint32_t* sz = reinterpret_cast<const uint32_t*>(vp + 2 * kPage * kCodeBytes) + kPage * ng;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int tau2 = (slice & 3) * 16 + 8 * uu + 2 * tq + e;
            if ((2 * k + (slice >> 2)) * kPage + tau2 < cur.s.hist) {  // else scale and zero stay 0: zero rows
#pragma unroll
              for (int w = 0; w < 2; ++w) vsz[e][w] = sz[sz_index(tau2, ng == 1 ? 0 : 2 * wh + w, ng)];
            }
          }
        }
      };
      fetch(cur.k0);
      for (int k = cur.k0; ok && k < nI; ++k) {
        // K tile
        int s = r.stage();
        bool w = wait_warp(&sh->empty[s], r.parity() ^ 1, sh, C.err);
        if (w) {
          uint8_t* dst = ring + s * kTileBytes + x * 128;
          const uint32_t W[8] = {kc[0].x, kc[0].y, kc[0].z, kc[0].w, kc[1].x, kc[1].y, kc[1].z, kc[1].w};  // [tq][word]
#pragma unroll
          for (int wd = 0; wd < 2; ++wd)
#pragma unroll
            for (int sh8 = 0; sh8 < 2; ++sh8) {
              const Levels t = levels(ng == 1 ? ksz[0] : ksz[2 * wd + sh8], ak, ak2);
              const uint32_t sel = sh8 ? 0x7531u : 0x6420u;
              const uint32_t xa = __byte_perm(W[wd], W[2 + wd], sel), xb = __byte_perm(W[4 + wd], W[6 + wd], sel);
#pragma unroll
              for (int p = 0; p < 4; ++p) {
                uint4 v;
                pick4(xa, p, t, v.x, v.y);
                pick4(xb, p, t, v.z, v.w);
                const int c = 4 * sh8 + p;  // chunk of the half wd
                *reinterpret_cast<uint4*>(dst + wd * kHalfBytes + ((c ^ (x & 7)) << 4)) = v;
              }
            }
          fence_proxy_async();
        }
        ok = and128(w);
        if (ok && x == 0) mbar_arrive(&sh->full[s]);
        ++r.pos;
        if (!ok) break;
        // V tile
        s = r.stage();
        w = wait_warp(&sh->empty[s], r.parity() ^ 1, sh, C.err);
        if (w) {
          uint8_t* half = ring + s * kTileBytes + wh * kHalfBytes;
#pragma unroll
          for (int ee = 0; ee < 2; ++ee) {
            const int e = ee ^ uu;  // lanes of odd u start with the odd token: eight rows, eight banks
            const int rowv = slice * 16 + 8 * uu + 2 * tq + e;
#pragma unroll
            for (int w1 = 0; w1 < 2; ++w1) {
              const Levels t = levels(e ? vsz[1][w1] : vsz[0][w1], av, av2);
              // byte 2e + w1 of the eight words: elements 0 .. 7 of the chunks
              const uint32_t sel = (uint32_t)(2 * e + w1) * 0x11u + 0x40u;
              const uint32_t x01 = __byte_perm(vc[0], vc[1], sel), x23 = __byte_perm(vc[2], vc[3], sel);
              const uint32_t x45 = __byte_perm(vc[4], vc[5], sel), x67 = __byte_perm(vc[6], vc[7], sel);
              const uint32_t xa = __byte_perm(x01, x23, 0x5410u), xb = __byte_perm(x45, x67, 0x5410u);
#pragma unroll
              for (int p = 0; p < 4; ++p) {
                uint4 v;
                pick4(xa, p, t, v.x, v.y);
                pick4(xb, p, t, v.z, v.w);
                const int c = 4 * w1 + p;
                *reinterpret_cast<uint4*>(half + rowv * 128 + ((c ^ (rowv & 7)) << 4)) = v;
              }
            }
          }
          fence_proxy_async();
        }
        if (k + 1 < nI) fetch(k + 1);
        ok = and128(w);
        if (ok && x == 0) mbar_arrive(&sh->full[s]);
        ++r.pos;
      }
      if (ok && !P.absorbed) ok = and128(skip(kLimbs));
    }
    if (ok) ok = and128(skip(2 * (cur.k1 - max(cur.k0, nI))));
  }
}

// ------------------------------------------------------------------------------------------------
template <bool MIXED>
constexpr int kChunkThreads = MIXED ? 512 : 384;

template <int R>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// Units of all sequences, and the place of unit g0(total) in them; every thread of the CTA.
template <bool MIXED>
__device__ int64_t plan(const ChunkArgs& C, Shared* sh, int bt, int64_t& g0, int64_t& g1, int grid) {
  constexpr int NT = kChunkThreads<MIXED>, NW = NT / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t mine = 0, total = 0;
  for (int i = threadIdx.x; i < C.n_seqs; i += NT) mine += units_of(load_seq<MIXED>(C, i), bt) * C.Hkv;
#pragma unroll
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) sh->scan[warp] = mine;
  __syncthreads();
  for (int w = 0; w < NW; ++w) total += sh->scan[w];
  const int64_t n = min((int64_t)grid, max((int64_t)1, total / kMinUnits));
  g0 = blockIdx.x < n ? (int64_t)blockIdx.x * total / n : total;
  g1 = blockIdx.x < n ? ((int64_t)blockIdx.x + 1) * total / n : total;
  if (g0 >= g1) return n;
  int64_t base = 0;
  for (int i0 = 0; i0 < C.n_seqs; i0 += NT) {
    const int i = i0 + threadIdx.x;
    SeqWork s{};
    if (i < C.n_seqs) s = load_seq<MIXED>(C, i);
    const int64_t per = units_of(s, bt), cnt = per * C.Hkv;
    int64_t inc = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    __syncthreads();
    if (lane == 31) sh->scan[warp] = inc;
    __syncthreads();
    int64_t before = base + inc - cnt;
    for (int w = 0; w < warp; ++w) before += sh->scan[w];
    for (int w = 0; w < NW; ++w) base += sh->scan[w];
    if (cnt > 0 && g0 >= before && g0 < before + cnt) {
      int64_t x = g0 - before;
      const int h = (int)(x / per);
      x -= h * per;
      int lo = 0, hi = pairs_of(s, bt) - 1;
      while (lo < hi) {  // the last pair that starts at or before x
        const int mid = (lo + hi + 1) >> 1;
        if (units_before(s, bt, mid) <= x) lo = mid; else hi = mid - 1;
      }
      sh->st_i = i;
      sh->st_h = h;
      sh->st_t = lo;
      sh->st_k = (int)(x - units_before(s, bt, lo));
    }
    if (base > g0) break;
  }
  sh->total = total;
  return n;
}

template <bool MIXED>
__global__ void __launch_bounds__(kChunkThreads<MIXED>, 1)
    k_chunk(const __grid_constant__ ChunkArgs C, const __grid_constant__ ChunkMaps M) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t *sq = smem, *ring = smem + 2 * kTileBytes;
  Shared* sh = reinterpret_cast<Shared*>(ring + kStages * kTileBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bt = 2 * kTile / C.hg;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], 1);
    }
    mbar_init(&sh->q_full, 1);
    mbar_init(&sh->q_empty, 1);
    mbar_init(&sh->done, 1);
    for (int u = 0; u < 2; ++u) {
      mbar_init(&sh->s_full[u], 1);
      mbar_init(&sh->p_ready[u], kTile);
    }
    sh->abort = 0;
    fence_mbar_init();
  }
  int64_t g0, g1;
  const int64_t n = plan<MIXED>(C, sh, bt, g0, g1, gridDim.x);
  if (threadIdx.x == 0 && g0 >= g1) reinterpret_cast<Part*>(C.ws)[blockIdx.x].parts = 0;
  if (g0 >= g1) return;
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh->tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  Cursor<MIXED> cur;
  cur.start(C, sh->st_i, sh->st_h, sh->st_t, sh->st_k, g1 - g0);
  if (threadIdx.x == 0) {
    // The item this CTA's first boundary cuts is joined by merge block blockIdx.x, if the item starts
    // in the CTA before (else an earlier boundary cuts it too).
    Part d{};
    const int64_t first = g0 - cur.k0, end = first + cur.nb, c = blockIdx.x, total = sh->total;
    if (cur.k0 > 0 && first >= (c - 1) * total / n) {
      int64_t e = c;
      while (e + 1 < n && (e + 1) * total / n < end) ++e;
      d.parts = (int)(e - c + 2);
      d.row0 = cur.s.row0 + cur.t * bt;
      d.rows = cur.tokens() * C.hg;
      d.head = cur.h * C.hg;
    }
    reinterpret_cast<Part*>(C.ws)[blockIdx.x] = d;
  }
  if constexpr (MIXED) {
    // registers of the launch: 512 x 128 = 128 x (2 x 184 + 104 + 40)
    if (warp < 8) {
      reg_inc<184>();
      softmax_role<true>(C, sh, sq, cur, warp >> 2);
    } else if (warp < 12) {
      reg_dec<104>();
      dequant_role(C, sh, ring, cur);
    } else {
      reg_dec<40>();
      if (warp == 12) {
        if (lane == 0) load_role<true>(C, M, sh, sq, ring, cur);
      } else if (warp == 13) {
        mma_role<true>(C, sh, sq, ring, cur, lane);
      }
    }
  } else {
    // 384 x 168 = 128 x (2 x 208 + 88)
    if (warp < 8) {
      reg_inc<208>();
      softmax_role<false>(C, sh, sq, cur, warp >> 2);
    } else {
      reg_dec<88>();
      if (warp == 8) {
        if (lane == 0) load_role<false>(C, M, sh, sq, ring, cur);
      } else if (warp == 9) {
        mma_role<false>(C, sh, sq, ring, cur, lane);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sh->tmem));
}

// Join the parts of the items that CTA boundaries cut: block (c, y) takes 32 rows of the item that
// boundary c cuts first. Part 0 is slot 1 of CTA c - 1, part p slot 0 of CTA c - 1 + p.
constexpr int kJoinRows = 32;
__global__ void __launch_bounds__(256) k_chunk_join(const __grid_constant__ ChunkArgs C) {
  const Part d = reinterpret_cast<const Part*>(C.ws)[blockIdx.x];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (d.parts == 0) return;
  const float* slots = reinterpret_cast<const float*>(C.ws + (size_t)kMaxCtas * kDescBytes);
  const size_t slot = (size_t)C.rows * (kHeadDim + 2);
  auto part = [&](int p) { return slots + ((size_t)(blockIdx.x - 1 + p) * 2 + (p == 0 ? 1 : 0)) * slot; };
  for (int row = blockIdx.y * kJoinRows + warp; row < min(d.rows, (int)(blockIdx.y + 1) * kJoinRows); row += 8) {
    float M = -INFINITY;
    for (int p = lane; p < d.parts; p += 32) M = fmaxf(M, part(p)[(size_t)C.rows * kHeadDim + 2 * row]);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll 4
    for (int p = 0; p < d.parts; ++p) {
      const float* s = part(p);
      const float2 ml = *reinterpret_cast<const float2*>(s + (size_t)C.rows * kHeadDim + 2 * row);
      const float4 o = *reinterpret_cast<const float4*>(s + (size_t)row * kHeadDim + 4 * lane);
      if (ml.x == -INFINITY && ml.y == 0.f) continue;  // saw no key
      const float w = fast_exp2(ml.x - M);
      l += w * ml.y;
      acc.x += w * o.x;
      acc.y += w * o.y;
      acc.z += w * o.z;
      acc.w += w * o.w;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), b = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
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

int chunk_ctas() {  // one CTA per SM of the current device
  int dev = 0, sms = kMaxCtas;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return sms < kMaxCtas ? sms : kMaxCtas;
}

template <bool MIXED>
cudaError_t launch_chunk(const ChunkArgs& C, const ChunkMaps& M, cudaStream_t s) {
  const int ctas = chunk_ctas();
  if (ctas < 1) return cudaErrorUnknown;
  cudaError_t e = cudaFuncSetAttribute(k_chunk<MIXED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kChunkSmem);
  if (e != cudaSuccess) return e;
  k_chunk<MIXED><<<ctas, kChunkThreads<MIXED>, kChunkSmem, s>>>(C, M);
  e = cudaGetLastError();
  if (e != cudaSuccess || ctas == 1) return e;
  k_chunk_join<<<dim3(ctas, C.rows / kJoinRows), 256, 0, s>>>(C);
  return cudaGetLastError();
}

}  // namespace

// Partials of a call: two slots per CTA (an item cut in front of the CTA's range, and one behind it).
size_t chunk_workspace_bytes(int hg, int64_t n_tokens) {
  return (size_t)kMaxCtas * (kDescBytes + 2 * (size_t)slot_rows(hg, n_tokens) * (kHeadDim + 2) * 4);
}

cudaError_t launch_chunk_pool(const DevPool& P, const StepDims& S, int layer, const void* q, const void* k_new,
                              const void* v_new, void* workspace, void* out, cudaStream_t s) {
  ChunkArgs C{};
  C.Hq = P.Hq;
  C.Hkv = P.Hkv;
  C.hg = P.hg;
  C.n_seqs = S.n_seqs;
  C.n_tokens = S.total_new;
  C.rows = slot_rows(P.hg, S.total_new);
  C.P = P;
  C.layer = layer;
  C.v_new = static_cast<const __nv_bfloat16*>(v_new);
  C.out = static_cast<__nv_bfloat16*>(out);
  C.ws = static_cast<uint8_t*>(workspace);
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
  return launch_chunk<true>(C, M, s);
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
      max_pages_per_seq > INT32_MAX / kPage)
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
  C.out = static_cast<__nv_bfloat16*>(out);
  C.ws = static_cast<uint8_t*>(workspace);
  C.err = err;
  ChunkMaps M;
  std::memset(&M, 0, sizeof(M));
  const int64_t rows = n_pages_total * num_kv_heads * kPage;
  if (!map_rows(&M.q, q, num_q_heads, n_tokens, q_token_stride, C.hg, kTile / C.hg) || !map_pages(&M.k, k_pages, rows) ||
      !map_pages(&M.v, v_pages, rows))
    return OSCAR_ECUDA;
  const cudaError_t e = launch_chunk<false>(C, M, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return OSCAR_ECUDA;
  }
  return OSCAR_OK;
}

}  // extern "C"

// What the key/value cache kernels of both element widths share: requests and
// row tiles, how work is cut and found, scores, the join of partial results,
// and on the host the checks and the plan of a call.  Internal linkage: each
// source that includes this has its own instances.
#pragma once

#include <hip/hip_runtime.h>

#include "wq.h"
#include "wq_device.h"
#include "wq_host.h"

using namespace wq;

namespace {

constexpr int KV_THREADS = 256;

// Sum of v over the lower lanes of the wave and this one: within rows of 16 lanes
// by shifts of 1, 2, 4 and 8, then the last lane of a row into the next and of
// the first half into the second (DPP moves; exchanges through LDS take ten times
// as long).  Every lane of the wave has to be active.
template <int CTRL, int ROWS>
__device__ __forceinline__ int64_t scan_step(int64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(v >> 32), CTRL, ROWS, 0xF, false);
  return v + (int64_t)((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ int64_t wave_scan(int64_t v) {
  v = scan_step<0x111, 0xF>(v);
  v = scan_step<0x112, 0xF>(v);
  v = scan_step<0x114, 0xF>(v);
  v = scan_step<0x118, 0xF>(v);
  v = scan_step<0x142, 0xA>(v);
  return scan_step<0x143, 0xC>(v);
}

// Rows of one key/value head are numbered r = query * group + head in group:
// the `group` query heads that share a key/value head share its tiles.
constexpr int TILE = 64;                      // tokens per step
constexpr int PROWS = 128, PTHREADS = 256;    // rows of a prompt tile, threads of its workgroup
// Requests of at most this many rows go through the decode kernel: its tiles of
// 32 read K and V once each, the prompt kernel once for 128, but a prompt
// tile's staging and barriers cost the same however few there are.  24 requests
// on 500-6000 tokens, 8 heads of 128: 48 rows 54 us decoded against 58 in
// prompt tiles, 64 rows 56 against 57, 128 rows 79 against 66.
constexpr int SHORT_ROWS = 64;
// Decode workgroups over all heads: two a CU, as the registers of D = 128 allow
// (256: 2-4 % slower on drafted tokens; 768 and 1024 at D = 64, where they fit:
// 9 and 14 % slower on short windows).
constexpr int DEC_GROUPS = 512;
// A workgroup a row tile where no request can have more tiles than this (few row
// tiles, enough of them for half the CUs) and they fit the chip twice over.  The
// host knows lengths by the table's width and the window only: 1000 tokens take
// 12.8 us on a table of 17 columns of 64, 17.0 us on one of 520, in shares.  8
// heads of 128, calls back to back: 1 x 700 tokens 12.8 us against 18.0 in
// shares and a join, 1 x 2000 17 against 16; 16 x 2000 18.5 against 21.8, 16 x
// 4000 30 against 31.
constexpr int SOLO_TILES = 20, SOLO_TILES_MANY = 40;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

struct KvArgs {
  const uint16_t* q;
  int64_t q_stride;
  const int32_t* cu_q;
  const int32_t* kv_lens;
  int64_t batch, tokens;
  int q_heads, kv_heads, group, window;
  const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  int log_page;
  int64_t num_pages;
  const int32_t* table;
  int64_t max_blocks;
  float sm_scale, softcap;
  uint16_t* out;
  float* lse;
  // x / group = x * group_mul >> 31 + group_shift for x below 2^31: group_mul =
  // floor(2^(31 + s) / group) + 1 with 2^s >= group is above the quotient by at most
  // 2^s / group 2^-(31 + s), which x below 2^31 does not take past the next whole number
  uint32_t group_mul, group_shift;
  __device__ __forceinline__ uint32_t by_group(uint32_t x) const { return (uint32_t)((uint64_t)x * group_mul >> 31 >> group_shift); }
};

// Partial results of the prompt kernel's split rows: `used[0]` slots are in
// use; slot s of head h holds PROWS * D sums and (maximum, sum) pairs.  `rec`
// names the slot's rows in the entry of the first split, with the number of
// splits that follow.
struct KvRec {
  int32_t splits;                             // 0 in the entries of the other splits
  int32_t rows, query0, head0;                // the first row: query row of the tensors, head in its group
};
struct KvPart {
  int64_t splits;                             // aim: items per head, over which the tiles are spread
  int64_t slots;                              // room in the arrays below: nothing is written past it, whatever cu_q holds
  int min_tiles;                              // no split is shorter
  int64_t* used;
  KvRec* rec;
  float* sums;
  float* stats;
};

// Partial results of the decode kernel.  Wave x of a head (4 to a workgroup)
// has two slots: 2 x for a row tile that begins in its share of the work and
// ends behind it, 2 x + 1 for one that began before.  A workgroup inside one
// row tile joins its waves first and uses the slots of its first wave alone.
// chain[x] describes the row tile of slot 2 x; every wave writes its own entry.
// With `by_tile` there is an entry for each row tile instead, which the wave
// that begins it writes: fewer for k_kv_join to look at where row tiles are few.
struct KvChain {
  int32_t rows, query0, head0;                // 0 rows: none
  int32_t first, last;                        // waves that share the row tile
  int32_t first_joined, last_joined;          // whether the workgroups of those joined their waves
};
struct KvShare {
  int groups, rows;                           // workgroups per head (0: one a row tile), rows of a slot
  int chains;                                 // entries of chain: 4 a workgroup, or fewer
  int log_joins;                              // log2 of the workgroups of k_kv_join for a row tile
  bool by_tile;
  KvChain* chain;
  float* sums;
  float* stats;
};

// Which requests a launch takes: all of them, those of at most SHORT_ROWS rows,
// or the others.
enum { REQ_ALL, REQ_SHORT, REQ_LONG };

// One item of work: rows [r0, r0 + rows) of a request, a share of their tiles.
// Uniform over the workgroup (read from one lane, so it lives in scalar registers).
struct KvItem {
  int request, q0, n, len;                    // first query row, queries, tokens in the cache
  int r0, rows, splits, split;
  int64_t slot;                               // partial slot, where splits > 1
};

__device__ __forceinline__ int lane32(int v, int src) { return __builtin_amdgcn_readlane(v, src); }
__device__ __forceinline__ int64_t lane64(int64_t v, int src) {
  return (int64_t)(((uint64_t)(uint32_t)lane32((int)(v >> 32), src) << 32) | (uint32_t)lane32((int)v, src));
}
__device__ __forceinline__ int64_t wave_sum(int64_t v) { return lane64(wave_scan(v), 63); }
// a / b for a >= 0 and b > 0: a division of 64 bits takes five times one of 32.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if ((uint64_t)(a | b) >> 32 == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// The lowest token that position `pos` sees (window 0: the first).
__device__ __forceinline__ int kv_lowest(int pos, int window) { return window > 0 && pos >= window ? pos - window + 1 : 0; }

// Request i (its lengths clamped to what the tensors hold): first query row,
// queries, tokens, tiles that some query sees, row tiles of R rows.
struct KvRequest {
  int q0, n, len, first, tiles, row_tiles;    // first: the first of the tiles
  template <int R, int WHICH>
  __device__ __forceinline__ void load(const KvArgs& A, int64_t i) {
    q0 = n = len = 0;
    if (i < A.batch) {
      const int cap = (int)(A.max_blocks << A.log_page);
      int a = A.cu_q[i], z = A.cu_q[i + 1];
      len = A.kv_lens[i];
      a = a < 0 ? 0 : a;
      z = z > A.tokens ? (int)A.tokens : z;
      q0 = a;
      n = z > a ? z - a : 0;
      len = len < 0 ? 0 : len > cap ? cap : len;
    }
    const int rows = n * A.group;             // below 2^31, as tokens * group is
    if (WHICH == REQ_SHORT ? rows > SHORT_ROWS : WHICH == REQ_LONG ? rows <= SHORT_ROWS : false) n = 0;
    row_tiles = n > 0 ? (int)(((int64_t)rows + R - 1) / R) : 0;
    first = kv_lowest(len - n, A.window) / TILE;
    tiles = len > 0 ? (len - 1) / TILE - first + 1 : 0;
  }
  __device__ __forceinline__ KvRequest from(int src) const {       // another lane's
    return KvRequest{lane32(q0, src), lane32(n, src), lane32(len, src), lane32(first, src), lane32(tiles, src),
                     lane32(row_tiles, src)};
  }
};

// Every wave finds its item itself, from the lengths: the tiles of all
// requests are spread evenly over about part.splits items, a request of
// `tiles` tiles being cut into tiles / share splits per row tile, to the
// nearest (rounding up costs more in partial sums than it evens out).
// False if there is no such item.
template <int R, int WHICH>
__device__ __forceinline__ bool kv_find(const KvArgs& A, const KvPart& part, int64_t item, bool count_all, KvItem& it) {
  const int lane = threadIdx.x & 63;
  KvRequest q;
  int64_t total = 0;
  for (int64_t base = 0; base < A.batch; base += 64) {
    q.load<R, WHICH>(A, base + lane);
    total += (int64_t)q.tiles * q.row_tiles;
  }
  total = wave_sum(total);
  int64_t share = (total + part.splits - 1) / part.splits;
  share = share < part.min_tiles ? part.min_tiles : share;
  const int per = share > 0x7FFFFFFF ? 0x7FFFFFFF : (int)share;
  int64_t items = 0, slots = 0;
  bool found = false;
  for (int64_t base = 0; base < A.batch; base += 64) {
    if (A.batch > 64) q.load<R, WHICH>(A, base + lane);
    const int rounded = (int)((2 * (int64_t)q.tiles + per) / (2 * (int64_t)per)), splits = rounded > 1 ? rounded : 1;
    const int64_t own = (int64_t)q.row_tiles * splits, part_own = splits > 1 ? own : 0;
    const int64_t end = items + wave_scan(own), part_end = slots + wave_scan(part_own);
    const unsigned long long at = __ballot(end > item);
    if (at && !found) {
      const int src = __builtin_ctzll(at);
      const int idx = (int)(item - lane64(end - own, src));
      it.splits = lane32(splits, src);
      it.split = idx % it.splits;
      it.request = (int)base + src;
      it.q0 = lane32(q.q0, src);
      it.n = lane32(q.n, src);
      it.len = lane32(q.len, src);
      it.r0 = (lane32(q.row_tiles, src) - 1 - idx / it.splits) * R;  // the longest rows first
      const int left = it.n * A.group - it.r0;
      it.rows = left < R ? left : R;
      it.slot = lane64(part_end - part_own, src) + idx;
      found = true;
    }
    if (found && !count_all) return true;
    items = lane64(end, 63);
    slots = lane64(part_end, 63);
  }
  if (count_all && threadIdx.x == 0) part.used[0] = slots < part.slots ? slots : part.slots;
  return found;
}

// Queries of a row tile: row r0 is query `first` of the request and head
// `head0` of the group; row r0 + i is i rows on.
struct KvRows {
  int first, head0, pos0;                     // pos0: position of query `first`
  __device__ __forceinline__ KvRows(const KvArgs& A, int r0, int n, int len)
      : first((int)A.by_group((uint32_t)r0)), head0(r0 - first * A.group), pos0(len - n + first) {}
  __device__ __forceinline__ int query(const KvArgs& A, int i) const { return (int)A.by_group((uint32_t)(head0 + i)); }
  __device__ __forceinline__ int head(const KvArgs& A, int i) const { return head0 + i - query(A, i) * A.group; }
};

// Tokens [lo, hi) that the item's rows see between them, and its tiles [t0, t1).
__device__ __forceinline__ void kv_tiles(const KvArgs& A, const KvItem& it, const KvRows& rows, int& lo, int& hi,
                                         int& t0, int& t1) {
  const int last = rows.pos0 + rows.query(A, it.rows - 1);
  hi = last < 0 ? 0 : last + 1;
  lo = kv_lowest(rows.pos0, A.window);
  lo = lo < hi ? lo : hi;
  const int a = lo / TILE, n = hi > lo ? (hi - 1) / TILE + 1 - a : 0;
  t0 = a + (int)((int64_t)n * it.split / it.splits);
  t1 = a + (int)((int64_t)n * (it.split + 1) / it.splits);
}

// Scores to base 2: dot * mul, or, capped, cap * tanh(x) * log2 e with x = dot *
// sm_scale / cap.  Sixteen at a time: where all of a wave's have |x| <= 1/4 (most
// scores are far below their cap), by the series of tanh up to x^7, whose next
// term is under 3.4e-7 of the result; else as cap - 2 cap / (e^2x + 1), off by
// at most cap * 2^-22.  Both take the same time (chunks 560 us); the series
// keeps small scores exact (lse off by 5e-8 instead of 2.5e-7, 2-norm).  It is
// taken in powers of the dot, with k = sm_scale / cap in its coefficients: for k
// from 2^-16 on (softcap 50 at heads of 128 has 2^-9) the squares of dots of up
// to 1 / 4k and the coefficient of k^7 are in fp32's range with 2^20 to spare
// against the bound.  A smaller k leaves it, so its scores all go by the
// exponential.  (A series in x itself holds for every k but takes a
// multiplication more a score: chunks 581 us.)
template <bool CAP>
struct KvScore {
  float mul;                                  // of what `cap` leaves
  float limit, to2x, twice, a0, a1, a2, a3;
  __device__ __forceinline__ explicit KvScore(const KvArgs& A) {
    mul = CAP ? 1.0f : A.sm_scale * LOG2E;
    if constexpr (CAP) {
      const float k = A.sm_scale / A.softcap, k2 = k * k;
      limit = k >= 0x1p-16f ? 0.25f / k : 0.0f;
      to2x = 2.0f * LOG2E * k;
      twice = A.softcap * LOG2E;
      a0 = A.sm_scale * LOG2E;
      a1 = a0 * k2 * (-1.0f / 3.0f);
      a2 = a0 * k2 * k2 * (2.0f / 15.0f);
      a3 = a0 * k2 * k2 * k2 * (-17.0f / 315.0f);
    }
  }
  __device__ __forceinline__ float series(float s) const {
    const float y = s * s;
    return s * __builtin_fmaf(__builtin_fmaf(__builtin_fmaf(a3, y, a2), y, a1), y, a0);
  }
  __device__ __forceinline__ float exponential(float s) const {
    return __builtin_fmaf(__builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(s * to2x) + 1.0f), -2.0f * twice, twice);
  }
  // `edge`: some of the sixteen are of tokens that their row does not see.  The form
  // of one that it does see must not follow their bytes, so each goes by itself then
  // (the series where all are below the limit is what each would take).
  template <typename T>
  __device__ __forceinline__ void cap(T& s, bool edge) const {
    if constexpr (CAP) {
      float big = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; i++) big = __builtin_fmaxf(big, __builtin_fabsf(s[i]));
      if (!__any(big > limit)) {
#pragma unroll
        for (int i = 0; i < 16; i++) s[i] = series(s[i]);
      } else if (!edge) {
#pragma unroll
        for (int i = 0; i < 16; i++) s[i] = exponential(s[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 16; i++) s[i] = __builtin_fabsf(s[i]) > limit ? exponential(s[i]) : series(s[i]);
      }
    }
  }
};

// Joins `parts` partial results of rows [row0, row0 + some) of one head, a wave
// taking every fourth row: its lanes hold 4 channels each, and the groups of
// lanes that this leaves share the parts, 4 of them in flight per lane, since a
// long context alone in its batch has many parts of few rows.  slot_of(i) is
// the place of part i among the slots of `room` rows.
template <int D, typename SLOT>
__device__ __forceinline__ void kv_join(const KvArgs& A, const float* sums, const float* stats, int room, int kvh,
                                        int row0, int some, int rows, int query0, int head0, int parts, SLOT slot_of) {
  constexpr int LANES = D / 4, GROUPS = 64 / LANES, DEEP = 4;
  const int lane = threadIdx.x & 63, grp = lane / LANES, ch = (lane % LANES) * 4;
  for (int row = row0 + threadIdx.x / 64; row < row0 + some && row < rows; row += KV_THREADS / 64) {
    float M = -INFINITY, L = 0.0f;
    f32x4_t acc = {0, 0, 0, 0};
    for (int s0 = grp; s0 < parts; s0 += GROUPS * DEEP) {
      float ms[DEEP], ls[DEEP], top = M;
      f32x4_t v[DEEP];
#pragma unroll
      for (int u = 0; u < DEEP; u++) {
        const int sp = s0 + GROUPS * u;
        const int64_t a = (slot_of(sp < parts ? sp : s0) * A.kv_heads + kvh) * room + row;
        ms[u] = stats[2 * a];
        ls[u] = stats[2 * a + 1];
        v[u] = *reinterpret_cast<const f32x4_t*>(sums + a * D + ch);
        if (sp >= parts) ms[u] = -INFINITY;
        top = __builtin_fmaxf(top, ms[u]);
      }
      const float keep = M == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(M - top);
      M = top;
      L *= keep;
      acc *= keep;
#pragma unroll
      for (int u = 0; u < DEEP; u++) {
        const float f = ms[u] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ms[u] - M);
        L = __builtin_fmaf(f, ls[u], L);
#pragma unroll
        for (int e = 0; e < 4; e++) acc[e] = __builtin_fmaf(f, v[u][e], acc[e]);
      }
    }
#pragma unroll
    for (int o = LANES; o < 64; o <<= 1) {
      const float mo = __shfl_xor(M, o, 64), lo = __shfl_xor(L, o, 64), top = __builtin_fmaxf(M, mo);
      const float a = M == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(M - top);
      const float b = mo == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mo - top);
      L = a * L + b * lo;
#pragma unroll
      for (int e = 0; e < 4; e++) acc[e] = a * acc[e] + b * __shfl_xor(acc[e], o, 64);
      M = top;
    }
    if (grp == 0) {
      const uint32_t rr = (uint32_t)head0 + row, group = A.group;
      const int64_t token = (int64_t)query0 + rr / group, orow = token * A.q_heads + kvh * group + rr % group;
      if (token < 0 || token >= A.tokens) continue;
      const float inv = L == 0.0f ? 0.0f : 1.0f / L;
      *reinterpret_cast<u32x2_t*>(A.out + orow * D + ch) =
          u32x2_t{pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv)};
      if (A.lse && ch == 0) A.lse[orow] = L == 0.0f ? -INFINITY : (M + __builtin_log2f(L)) * LN2;
    }
  }
}

// Workgroups of the decode kernel's waves first, 2^log_joins each, then
// PROWS / 16 for each prompt slot.  8 rows each where more than 8 are likely (24
// requests of 1-7 drafted tokens 10.2 -> 8.2 us), 16 else, since most of these
// workgroups find nothing (64 requests of 4 rows 4.6 us, 5.8 in eights).
template <int D, int NR>
__global__ __launch_bounds__(KV_THREADS) void k_kv_join(const KvArgs A, const KvShare dec, const KvPart pro) {
  const int kvh = (int)(blockIdx.x % (unsigned)A.kv_heads);
  int64_t x = blockIdx.x / (unsigned)A.kv_heads;
  const int64_t decode = (int64_t)dec.chains << dec.log_joins;
  if (x < decode) {
    const KvChain c = dec.chain[x >> dec.log_joins];
    const int some = 16 * NR >> dec.log_joins, row0 = (int)(x & ((1 << dec.log_joins) - 1)) * some;
    // no row tile, or one that lengths changing under the kernel left unwritten
    if (c.rows <= 0 || c.rows > 16 * NR || c.first < 0 || c.last < c.first || c.last >= 4 * dec.groups) return;
    // parts: the first workgroup's, one for each between, the last workgroup's
    const int ga = c.first / 4, gz = c.last / 4;
    const int a = c.first_joined ? 1 : (gz > ga ? 4 * ga + 3 : c.last) - c.first + 1;
    const int mid = gz > ga ? gz - ga - 1 : 0, z = gz > ga ? (c.last_joined ? 1 : c.last - 4 * gz + 1) : 0;
    kv_join<D>(A, dec.sums, dec.stats, dec.rows, kvh, row0, some, c.rows, c.query0, c.head0, a + mid + z,
               [&](int i) -> int64_t {
                 if (i < a) return i == 0 ? 2 * c.first : 2 * (c.first + i) + 1;
                 return i < a + mid ? 8 * (ga + 1 + i - a) + 1 : 2 * (4 * gz + i - a - mid) + 1;
               });
    return;
  }
  x -= decode;
  const int64_t slot = x / (PROWS / 16);
  if (slot >= pro.used[0]) return;
  const KvRec rec = pro.rec[slot];
  // entries that ranges of rows on top of each other left unwritten hold anything
  if (rec.splits <= 0 || slot + rec.splits > pro.slots || rec.rows > PROWS) return;
  kv_join<D>(A, pro.sums, pro.stats, PROWS, kvh, (int)(x % (PROWS / 16)) * 16, 16, rec.rows, rec.query0, rec.head0, rec.splits,
             [&](int i) -> int64_t { return slot + i; });
}

int log2_page(int page) {
  return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : page == 128 ? 7 : -1;
}

// Items aimed at for prompts, over all key/value heads (two workgroups a CU; 256
// leaves 24 x 128 rows at 80 us instead of 66, 1024 slows 4 x 512 queries on
// 4000 tokens from 164 to 190 us by its partial sums), and the fewest tiles of
// a split (1: the same; 16: 72 us instead of 66).
constexpr int64_t PRO_ITEMS = 512;
constexpr int PRO_MIN = 4;

// What a call launches and where its workspace lies.  Prompt items per head are
// at most splits + row tiles; slots (items of requests with two splits or
// more) at most 2 * splits, and no more than the tiles of the table's width
// allow.  The decode kernel has as many workgroups as the chip holds at once
// (two a CU, as its registers allow), or one a head.
struct KvPlan {
  bool prompt, solo;                          // solo: decode only, a workgroup a row tile, nothing to join
  int nr;                                     // 16-row columns of a decode tile
  int groups, rows, log_joins;                // decode workgroups per head, rows of its slots, joins a row tile
  int chains;                                 // row tiles of the decode kernel, at most
  int64_t pro_splits, pro_items, pro_slots;
  size_t dec_sums, dec_stats, pro_used, pro_rec, pro_sums, pro_stats, bytes;
};

KvPlan kv_plan(int64_t batch, int64_t tokens, int64_t max_q, int q_heads, int kv_heads, int head_dim, int page,
               int64_t max_blocks, int64_t window) {
  KvPlan p = {};
  const int64_t group = q_heads / kv_heads, reqs = batch < tokens ? batch : tokens;
  const int64_t tiles = (max_blocks * page + TILE - 1) / TILE;
  const int64_t most_q = max_q > 0 && max_q < tokens ? max_q : tokens;
  p.prompt = most_q * group > SHORT_ROWS;
  p.nr = most_q * group <= 16 ? 1 : 2;
  p.rows = 16 * p.nr;
  p.log_joins = (p.nr == 2) + (!p.prompt && most_q * group > 8);
  const int64_t wgs = DEC_GROUPS / kv_heads, row_tiles = tokens * group / p.rows + reqs;
  const int64_t seen = window > 0 && window < tiles * TILE ? (window + most_q - 2) / TILE + 2 : tiles;
  const int64_t work = row_tiles * kv_heads;
  p.solo = !p.prompt && (seen < tiles ? seen : tiles) <= (work < DEC_GROUPS / 4 ? SOLO_TILES : SOLO_TILES_MANY) &&
           work <= 2 * DEC_GROUPS;
  p.groups = (int)(p.solo ? row_tiles : wgs > 1 ? wgs : 1);
  const int64_t chains = p.prompt ? reqs * (SHORT_ROWS / p.rows) : row_tiles;
  p.chains = (int)(chains < 4 * p.groups ? chains : 4 * p.groups);
  if (p.solo) return p;
  p.pro_splits = (PRO_ITEMS + kv_heads - 1) / kv_heads;
  const int64_t pro_rows = p.prompt ? tokens * group / PROWS + reqs : 0;
  p.pro_items = p.prompt ? pro_rows + p.pro_splits : 0;
  if (p.prompt && tiles > PRO_MIN) {
    const int64_t most = (tiles + PRO_MIN - 1) / PRO_MIN;
    p.pro_slots = pro_rows > 2 * p.pro_splits / most ? 2 * p.pro_splits : pro_rows * most;
  }
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t a = at;
    at += (n + 255) & ~(size_t)255;
    return a;
  };
  const size_t slots = 8 * (size_t)p.groups * kv_heads * p.rows;
  take(4 * (size_t)p.groups * sizeof(KvChain));
  p.dec_sums = take(slots * head_dim * 4);
  p.dec_stats = take(slots * 8);
  p.pro_used = take(8);
  p.pro_rec = take(p.pro_slots * sizeof(KvRec));
  p.pro_sums = take((size_t)p.pro_slots * kv_heads * PROWS * head_dim * 4);
  p.pro_stats = take((size_t)p.pro_slots * kv_heads * PROWS * 8);
  p.bytes = at;
  return p;
}

bool kv_sizes_ok(int64_t batch, int64_t tokens, int64_t max_q, int32_t q_heads, int32_t kv_heads, int32_t page,
                 int64_t max_blocks) {
  return batch >= 0 && batch <= 0x7FFFFFFF && tokens >= 0 && tokens <= 0x7FFFFFFF && max_q >= 0 &&
         max_q <= 0x7FFFFFFF && kv_heads >= 1 && q_heads >= kv_heads && q_heads % kv_heads == 0 && q_heads <= 65535 &&
         tokens * (q_heads / kv_heads) <= 0x7FFFFFFF - PROWS && max_blocks >= 1 && max_blocks <= 0x7FFFFF00 / page;
}
// The arguments of an attention call on either cache.
struct KvCall {
  const void* q;
  int64_t q_stride;
  const int32_t *cu_q, *kv_lens;
  int64_t batch, tokens, max_q;
  int32_t q_heads, kv_heads, head_dim;
  const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  int32_t page;
  int64_t num_pages;
  const int32_t* table;
  int64_t max_blocks;
  float sm_scale, softcap;
  int64_t window;
  uint16_t* out;
  float* lse;
  void* workspace;
  size_t ws_bytes;
};

// What both refuse.
wq_status kv_check(const KvCall& c) {
  if ((c.head_dim != 64 && c.head_dim != 128) || log2_page(c.page) < 0) return WQ_EUNSUPPORTED;
  if (!kv_sizes_ok(c.batch, c.tokens, c.max_q, c.q_heads, c.kv_heads, c.page, c.max_blocks) || c.num_pages < 1 || c.window < 0)
    return WQ_EINVAL;
  if (!(c.sm_scale > 0.0f) || !(c.sm_scale < INFINITY) || !(c.softcap >= 0.0f) || !(c.softcap < INFINITY)) return WQ_EINVAL;
  if (c.sm_scale > 0x1p127f) return WQ_EUNSUPPORTED;         // scores go to base 2: sm_scale * log2 e is finite
  if (c.softcap > 0.0f && (c.softcap < 0x1p-10f || c.softcap > 0x1p10f || !(c.sm_scale / c.softcap < 0x1p14f) ||
                           !(c.sm_scale / c.softcap > 0x1p-100f)))
    return WQ_EUNSUPPORTED;
  const int64_t row = (int64_t)c.q_heads * c.head_dim;
  if (c.q_stride < row || c.q_stride % 8 || c.q_stride > (int64_t(1) << 40) ||
      !wq_numel_ok(c.num_pages, (int64_t)c.kv_heads * c.head_dim * c.page) || !wq_numel_ok(c.tokens ? c.tokens : 1, row) ||
      !wq_numel_ok(c.batch ? c.batch : 1, c.max_blocks))
    return WQ_EINVAL;
  if (!c.k_codes || !c.k_scales || !c.v_codes || !c.v_scales) return WQ_EINVAL;
  if (c.batch > 0 && c.tokens > 0 && (!c.q || !c.cu_q || !c.kv_lens || !c.table || !c.out || c.out == c.q)) return WQ_EINVAL;
  if (!wq_aligned(c.q) || !wq_aligned(c.out) || !wq_aligned(c.k_codes) || !wq_aligned(c.v_codes) || !wq_aligned(c.workspace))
    return WQ_EALIGN;
  return WQ_OK;
}

// The checked call's plan, arguments and places in the workspace.
struct KvLaunch {
  KvPlan plan;
  KvArgs args;
  KvShare dec;
  KvPart pro;
  wq_status lay_out(const KvCall& c) {
    plan = kv_plan(c.batch, c.tokens, c.max_q, c.q_heads, c.kv_heads, c.head_dim, c.page, c.max_blocks, c.window);
    const KvPlan& p = plan;
    if (p.bytes > 0 && (c.ws_bytes < p.bytes || !c.workspace)) return WQ_EINVAL;
    if (p.pro_items * c.kv_heads > 0x7FFFFFFF / PTHREADS) return WQ_EINVAL;
    args = KvArgs{(const uint16_t*)c.q, c.q_stride, c.cu_q, c.kv_lens, c.batch, c.tokens, c.q_heads, c.kv_heads,
                  c.q_heads / c.kv_heads, (int)(c.window < 0x7FFFFFFF ? c.window : 0), c.k_codes, c.k_scales, c.v_codes,
                  c.v_scales, log2_page(c.page), c.num_pages, c.table, c.max_blocks, c.sm_scale, c.softcap, c.out, c.lse, 0, 0};
    while ((1 << args.group_shift) < args.group) args.group_shift++;
    args.group_mul = (uint32_t)((uint64_t(1) << (31 + args.group_shift)) / (uint32_t)args.group + 1);
    uint8_t* ws = (uint8_t*)c.workspace;
    dec = KvShare{p.solo ? 0 : p.groups, p.rows, 4 * p.groups, p.log_joins, false, (KvChain*)ws, (float*)(ws + p.dec_sums),
                  (float*)(ws + p.dec_stats)};
    pro = KvPart{p.pro_splits, p.pro_slots, PRO_MIN, (int64_t*)(ws + p.pro_used), (KvRec*)(ws + p.pro_rec),
                 (float*)(ws + p.pro_sums), (float*)(ws + p.pro_stats)};
    return WQ_OK;
  }
};

}  // namespace

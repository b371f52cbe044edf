// Attention over the 4-bit key/value cache for gfx950 (E2M1 elements, one E8M0
// scale per 32 channels of a token and head).
#include <utility>

#include "wq_kv_common.h"

namespace {

// As over the 8-bit cache, both kernels compute S^T = K q^T and O^T = V^T P^T on
// bf16 matrix cores, so that a row of the query tile is a column of both
// products and a lane's probabilities are the operand elements that it supplies
// to the second.  E2M1 times a power of two is exact in bf16.  Keys have one scale
// for 32 channels of a token, which the conversion takes; values have one for 32
// channels of a token too, while their operand runs along the tokens, so a byte
// of the transposed page holds two channels of one token: it is converted
// with its token's scale, and the pairs are then sorted by channel.

// E8M0 byte i of w as the operand of a scaled conversion, which reads nothing
// but its bits 23 to 30.
__device__ __forceinline__ float scale_of(uint32_t w, int i) {
  return __uint_as_float(i == 3 ? w >> 1 : w << (23 - 8 * i));
}

// Eight E2M1 codes with one scale -> eight bf16.
__device__ __forceinline__ bf16x8_t e2m1_bf16x8(uint32_t w, float scale) {
  u32x4_t v;
  v[0] = dq_fp4_pair<0>(w, scale);
  v[1] = dq_fp4_pair<1>(w, scale);
  v[2] = dq_fp4_pair<2>(w, scale);
  v[3] = dq_fp4_pair<3>(w, scale);
  return __builtin_bit_cast(bf16x8_t, v);
}

// Eight tokens of a pair of channels (a, b: a byte a token; sa, sb: a scale a
// token) -> eight bf16 of either channel.
__device__ __forceinline__ void value_pairs(uint32_t a, uint32_t b, uint32_t sa, uint32_t sb, bf16x8_t& even, bf16x8_t& odd) {
  u32x4_t lo, hi;
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const uint32_t w = i ? b : a, s = i ? sb : sa;
    const uint32_t x0 = dq_fp4_pair<0>(w, scale_of(s, 0)), x1 = dq_fp4_pair<1>(w, scale_of(s, 1));
    const uint32_t x2 = dq_fp4_pair<2>(w, scale_of(s, 2)), x3 = dq_fp4_pair<3>(w, scale_of(s, 3));
    lo[2 * i] = __builtin_amdgcn_perm(x1, x0, 0x05040100u);
    hi[2 * i] = __builtin_amdgcn_perm(x1, x0, 0x07060302u);
    lo[2 * i + 1] = __builtin_amdgcn_perm(x3, x2, 0x05040100u);
    hi[2 * i + 1] = __builtin_amdgcn_perm(x3, x2, 0x07060302u);
  }
  even = __builtin_bit_cast(bf16x8_t, lo);
  odd = __builtin_bit_cast(bf16x8_t, hi);
}

// Scale bytes above 252 (none of which the append writes) made 252, so that
// the values are finite.  Done in tiles whose rows see different tokens: there a
// row's probability of 0 meets values that it does not see, and must stay 0.
__device__ __forceinline__ uint32_t finite_scales(uint32_t w) {
  const uint32_t t = ((w & 0x7F7F7F7Fu) + 0x03030303u) & w & 0x80808080u;     // bytes 253 to 255
  return w & ~((t >> 7) | (t >> 6));
}

// Lane I of the row of 16 that a lane is in.
template <int I>
__device__ __forceinline__ uint32_t row_lane(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x150 + I, 0xF, 0xF, false);
}

template <typename F, int... I>
__device__ __forceinline__ void for_each(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>{}), ...);
}

// The pieces of 16 tokens, at j, that every row of a tile sees alike: those in
// [lo, hi).  Rows at positions first to last see different tokens of the tiles
// before (whose lowest token the last row does not see) and behind.
struct KvAlike {
  int lo, hi;
  __device__ __forceinline__ KvAlike(int first, int last, int window) {
    const int last_lo = kv_lowest(last, window);
    lo = last > first ? (last_lo + TILE - 1) / TILE * TILE : 0;
    hi = last > first ? (first < 0 ? 0 : (first + 1) / TILE * TILE) : 0x7FFFFFFF;
  }
  __device__ __forceinline__ bool operator()(int j) const { return j >= lo && j <= hi - 16; }
};

// Decode, as over the 8-bit cache: 16 or 32 rows a row tile, tiles of 64 tokens cut
// into equal shares, one a wave, K and V from HBM straight into registers.  SOLO:
// a workgroup of WAVES waves has a row tile and nothing is joined, by a kernel
// without shares, whose start is shorter (one request of 1000 tokens 9.8 -> 8.2 us).
//
// Bound by bytes where contexts are long: D / 2 + D / 32 for K and for V a token and
// head, 64 requests of 2048-8192 tokens x 8 heads of 128 (296 MB) 68.5 us in all,
// 4.3 TB/s, of which the joins are 5 and start and end 10; longer ones add 6.0
// TB/s.  One 131072 tokens beside four short (243 MB): 58.5 us, 4.2 TB/s.  Half the
// bytes of the 8-bit cache bring the conversions to the front: vector units are
// busy 0.43 of the cycles, matrix cores 0.15, neither 0.46.  Two waves a SIMD
// with one tile each on its way: two or three tiles on their way took the same
// time, three waves a SIMD 71.5 us instead of 68.
// Short contexts and drafted tokens are bound by latency (33 windows of 1000 tokens,
// 16 heads of 64: 11.0 us; 24 requests of 1-7 queries: 28.8 us).
//
// Lane l = 16 g + m.  K tile a (of 4): operand row m is token
// 16 (m / 4) + 4 a + m % 4, result rows 4 g + i are then tokens 16 g + 4 a + i;
// step h of the products takes channels D / 4 g + 8 h on of each, so that a lane's
// codes of a token are one load and four lanes' make a whole row.  V^T: operand
// row m of tiles 2 b and 2 b + 1 are channels 32 b + 2 m and the next.
template <int D, bool CAP, int WHICH, int NR, bool SOLO, int WAVES = 4>
__global__ __launch_bounds__(64 * WAVES, 2) void k_kv4_decode(const KvArgs A, const KvShare part) {
  constexpr int KH = D / 32, NB = D / 32, DT = D / 16, R = 16 * NR;   // k steps, blocks, channel tiles
  constexpr bool FINE = NR == 1 && !SOLO;     // probabilities in two bf16 terms
  __shared__ __attribute__((aligned(16))) float so[WAVES][R][D + 4];
  __shared__ float sm[WAVES][R], sl[WAVES][R];
  const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = (int)(blockIdx.x / (unsigned)A.kv_heads), kvh = (int)(blockIdx.x % (unsigned)A.kv_heads);
  const int x = WAVES * group + wave;
  const KvChain none = {};

  // all the work, in tiles or in row tiles, and this wave's share [u0, u1) of it
  auto units_of = [&](const KvRequest& r) { return SOLO || r.tiles <= 0 ? 1 : r.tiles; };
  KvRequest lanes;
  int64_t total = 0, tiles = 0, end = 0, tiles_end = 0;     // of all requests; up to and with the lane's
  auto scan = [&](int64_t base, int64_t& before, int64_t& tiles_before) {      // 64 requests from `base` on
    lanes.load<R, WHICH>(A, base + lane);
    end = before + wave_scan((int64_t)units_of(lanes) * lanes.row_tiles);
    tiles_end = tiles_before + wave_scan(lanes.row_tiles);
    before = lane64(end, 63);
    tiles_before = lane64(tiles_end, 63);
  };
  for (int64_t base = 0; base < A.batch; base += 64) scan(base, total, tiles);
  if (!SOLO && part.by_tile && blockIdx.x == 0)        // entries behind the last row tile's
    for (int64_t i = tiles + tid; i < part.chains; i += 64 * WAVES) part.chain[i] = none;
  const bool each = !SOLO && !part.by_tile;   // an entry for each wave
  // the first `extra` shares have one unit more
  const int64_t shares = SOLO ? WAVES * total : total < WAVES * part.groups ? total : WAVES * part.groups;
  const int64_t least = SOLO || total == 0 ? 0 : quotient(total, shares), extra = total - least * shares;
  auto share_at = [&](int64_t y) { return y >= shares ? total : SOLO ? y / WAVES : y * least + (y < extra ? y : extra); };
  const int64_t u0 = share_at(x), u1 = share_at(x + 1), g0 = share_at(WAVES * group), g1 = share_at(WAVES * (group + 1));
  if (g0 >= g1) {                             // an idle workgroup
    if (each && kvh == 0 && lane == 0) part.chain[x] = none;
    return;
  }
  // the request that holds unit u
  KvRequest q = {};
  int request = 0;
  int64_t begin = 0, tile0 = 0;               // its first unit, and row tile
  auto find = [&](int64_t u) {
    int64_t before = 0, tiles_before = 0;
    for (int64_t base = 0; base < A.batch; base += 64) {
      if (A.batch > 64) scan(base, before, tiles_before);
      const unsigned long long at = __ballot(end > u);
      if (at) {
        const int src = __builtin_ctzll(at);
        q = lanes.from(src);
        request = (int)base + src;
        tile0 = lane64(tiles_end, src) - q.row_tiles;
        begin = lane64(end, src) - (int64_t)units_of(q) * q.row_tiles;
        return;
      }
    }
  };
  find(g0);
  auto units = [&]() { return units_of(q); };
  int rt = (int)quotient(g0 - begin, units());     // row tiles in order of their units, the last rows first
  const bool joined = SOLO || g1 <= begin + (int64_t)(rt + 1) * units();
  if (!joined) {
    if (u0 >= u1) {
      if (each && kvh == 0 && lane == 0) part.chain[x] = none;
      return;
    }
    find(u0);
    rt = (int)quotient(u0 - begin, units());
  }
  if (q.row_tiles == 0) {                     // lengths that changed under the kernel
    if (each && kvh == 0 && lane == 0) part.chain[x] = none;
    return;
  }

  const int last_col = (int)A.max_blocks - 1;
  const uint32_t head_bytes = (uint32_t)(D / 2) << A.log_page, page_bytes = head_bytes * A.kv_heads;
  const uint32_t head_scales = (uint32_t)NB << A.log_page, page_scales = head_scales * A.kv_heads;
  const int in_page = (1 << A.log_page) - 1;
  const uint8_t* kbase = A.k_codes + (int64_t)kvh * head_bytes;
  const uint8_t* vbase = A.v_codes + (int64_t)kvh * head_bytes;
  const uint8_t *ksb = A.k_scales + (int64_t)kvh * head_scales, *vsb = A.v_scales + (int64_t)kvh * head_scales;
  const KvScore<CAP> sc(A);
  KvChain chain = none;

  for (int64_t u = u0;;) {
    const int64_t row_begin = begin + (int64_t)rt * units(), row_end = row_begin + units();
    const int64_t stop = u1 < row_end ? u1 : row_end;
    const int step = joined ? WAVES : 1;          // the waves of a joined workgroup take its tiles in turn
    const int r0 = (q.row_tiles - 1 - rt) * R;
    const int n_rows = q.n * A.group - r0 < R ? q.n * A.group - r0 : R;
    const KvRows rows(A, r0, q.n, q.len);
    // tokens [lo, hi) that the rows see between them, tiles [t, t1) of this share
    const int row_max = rows.pos0 + rows.query(A, n_rows - 1);
    const int hi = row_max < 0 ? 0 : row_max + 1;
    int lo = kv_lowest(rows.pos0, A.window);
    lo = lo < hi ? lo : hi;
    const int lo_max = kv_lowest(row_max, A.window);
    auto first_tile = [&]() {
      const int a = q.first + (int)((joined ? g0 : u) - row_begin);
      return a < lo / TILE ? lo / TILE : a;
    };
    int t = first_tile(), t1 = q.first + (SOLO ? q.tiles : (int)((joined ? g1 : stop) - row_begin));
    t1 = t1 > (hi + TILE - 1) / TILE ? (hi + TILE - 1) / TILE : t1;
    t += joined ? wave : 0;

    const int32_t* tab = A.table + (int64_t)request * A.max_blocks;
    // a tile on its way
    uint32_t kr[4][KH], vsc;                  // vsc: scales of four of the lane's 16 values, in block m / 4
    u32x4_t vr[NB], ksc;                      // ksc: scales of 16 keys, this lane's among them
    bool vok;
    int idk, idv;                             // page ids of the next tile to load
    auto load_ids = [&](int t) {
      const int ck = (t * TILE + 16 * (m >> 2)) >> A.log_page, cv = (t * TILE + 16 * g) >> A.log_page;
      idk = tab[ck < last_col ? ck : last_col];
      idv = tab[cv < last_col ? cv : last_col];
    };
    auto load_k = [&](int t) {
      const uint64_t id = idk >= 0 && idk < A.num_pages ? idk : 0;
      const int off = (t * TILE + 16 * (m >> 2)) & in_page;
      ksc = ld16(ksb + (id * page_scales + (((D == 128 ? g : g >> 1) << A.log_page) + off)));
      const uint8_t* p = kbase + (id * page_bytes + (off + (m & 3)) * (D / 2) + 4 * KH * g);
#pragma unroll
      for (int a = 0; a < 4; a++) {
        if constexpr (D == 128) {
          const u32x4_t w = ld16(p + 4 * a * (D / 2));
#pragma unroll
          for (int h = 0; h < KH; h++) kr[a][h] = w[h];
        } else {
          const u32x2_t w = *reinterpret_cast<const u32x2_t*>(p + 4 * a * (D / 2));
#pragma unroll
          for (int h = 0; h < KH; h++) kr[a][h] = w[h];
        }
      }
    };
    auto load_v = [&](int t) {
      vok = idv >= 0 && idv < A.num_pages;
      const uint64_t id = vok ? idv : 0;
      const int off = (t * TILE + 16 * g) & in_page;
      const uint8_t* p = vbase + (id * page_bytes + ((m << A.log_page) + off));
      vsc = *reinterpret_cast<const uint32_t*>(vsb + (id * page_scales + ((((m >> 2) & (NB - 1)) << A.log_page) + off + 4 * (m & 3))));
#pragma unroll
      for (int b = 0; b < NB; b++) vr[b] = ld16(p + ((16 * b) << A.log_page));
    };
    if (t < t1) {
      load_ids(t);
      load_k(t);
      load_v(t);
      if (t + step < t1) load_ids(t + step);
    }

    // query fragments: columns m of q^T, channels D / 4 g + 8 h on in step h; row m's limits
    bf16x8_t qf[NR][KH];
    int pos[NR], rlo[NR];
#pragma unroll
    for (int c = 0; c < NR; c++) {
      const bool live = 16 * c + m < n_rows;
      const int i = live ? 16 * c + m : 0, query = rows.query(A, i);
      pos[c] = rows.pos0 + query;
      rlo[c] = kv_lowest(pos[c], A.window);
      const uint16_t* qp = A.q + (int64_t)(q.q0 + rows.first + query) * A.q_stride + (kvh * A.group + rows.head(A, i)) * D;
#pragma unroll
      for (int h = 0; h < KH; h++) {
        u32x4_t w = ld16(qp + D / 4 * g + 8 * h);
        if (!live) w = u32x4_t{0, 0, 0, 0};
        qf[c][h] = __builtin_bit_cast(bf16x8_t, w);
      }
    }

    f32x4_t o[NR][DT];
    float mx[NR], l[NR];
#pragma unroll
    for (int c = 0; c < NR; c++) {
#pragma unroll
      for (int d = 0; d < DT; d++) o[c][d] = f32x4_t{0, 0, 0, 0};
      mx[c] = -INFINITY;
      l[c] = 0.0f;
    }
    for (; t < t1; t += step) {
      const int j0 = t * TILE + 16 * g;       // this lane's 16 tokens in scores and V^T
      const bool more = t + step < t1;
      f32x4_t s[NR][4];
#pragma unroll
      for (int a = 0; a < 4; a++) {
        // byte m % 4, turned to where the conversion reads a scale
        const float ks = __uint_as_float(__builtin_amdgcn_alignbit(ksc[a], ksc[a], 9 + 8 * (m & 3)));
#pragma unroll
        for (int c = 0; c < NR; c++) s[c][a] = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int h = 0; h < KH; h++) {
          const bf16x8_t k = e2m1_bf16x8(kr[a][h], ks);
#pragma unroll
          for (int c = 0; c < NR; c++) s[c][a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, qf[c][h], s[c][a], 0, 0, 0);
        }
      }
      if (more) load_k(t + step);
      const bool edge = t * TILE + TILE - 1 > rows.pos0 || t * TILE < lo_max || __any(!vok);
      if (edge) vsc = finite_scales(vsc);     // of tokens that not every row sees
      // bf16 for the matrix cores: half a step of 2^-8 per probability, the sum l keeps fp32.  Where
      // contexts are long and the products few (FINE), what that leaves is multiplied too (rest0, rest1): the
      // error against 64 bits is then the output's own rounding, 1.7e-3 instead of 2.3e-3 (2-norm), for
      // half a percent of a ragged batch's time (68.2 us) and 1.8 of one long context's (58.3); row tiles
      // of their own would pay 8 to 9 % (8.19 -> 8.83 us), those of 32 rows 9 (28.8 -> 31.4)
      bf16x8_t p0[NR], p1[NR], rest0[NR], rest1[NR];
#pragma unroll
      for (int c = 0; c < NR; c++) {
        if (c > 0 && 16 * c >= n_rows) {      // a column without rows
          p0[c] = p1[c] = __builtin_bit_cast(bf16x8_t, (u32x4_t{0, 0, 0, 0}));
          continue;
        }
        if constexpr (CAP) {
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; i++) v[i] = s[c][i >> 2][i & 3];
          sc.cap(v, edge);
#pragma unroll
          for (int i = 0; i < 16; i++) s[c][i >> 2][i & 3] = v[i];
        }
        if (edge) {                           // tokens outside the row's limits
          const int z = vok ? pos[c] - j0 : -1, low = rlo[c] - j0;
#pragma unroll
          for (int a = 0; a < 4; a++)
#pragma unroll
            for (int i = 0; i < 4; i++) s[c][a][i] = 4 * a + i <= z && 4 * a + i >= low ? s[c][a][i] : -INFINITY;
        }
        float mt = -INFINITY;
#pragma unroll
        for (int a = 0; a < 4; a++)
#pragma unroll
          for (int i = 0; i < 4; i++) mt = __builtin_fmaxf(mt, s[c][a][i]);
        mt = __builtin_fmaxf(mt, __shfl_xor(mt, 16, 64));
        mt = __builtin_fmaxf(mt, __shfl_xor(mt, 32, 64)) * sc.mul;
        if (__any(mt > mx[c] + 8.0f)) {       // only past 2^8: the sums hold that, and the result is the same
          const float mn = __builtin_fmaxf(mx[c], mt);
          const float f = mx[c] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mx[c] - mn);
          mx[c] = mn;
          l[c] *= f;
#pragma unroll
          for (int d = 0; d < DT; d++) o[c][d] *= f;
        }
        const float off = mx[c] == -INFINITY ? 0.0f : -mx[c];
        uint32_t pw[8], rw[8];
#pragma unroll
        for (int a = 0; a < 4; a++) {
          float p[4];
#pragma unroll
          for (int i = 0; i < 4; i++) {
            p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[c][a][i], sc.mul, off));
            l[c] += p[i];
          }
          pw[2 * a] = pack_bf16x2(p[0], p[1]);
          pw[2 * a + 1] = pack_bf16x2(p[2], p[3]);
          if constexpr (FINE) {
#pragma unroll
            for (int i = 0; i < 2; i++) {
              const uint32_t w = pw[2 * a + i];
              rw[2 * a + i] = pack_bf16x2(p[2 * i] - bf16_lo(w), p[2 * i + 1] - bf16_hi(w));
            }
          }
        }
        p0[c] = __builtin_bit_cast(bf16x8_t, (u32x4_t{pw[0], pw[1], pw[2], pw[3]}));
        p1[c] = __builtin_bit_cast(bf16x8_t, (u32x4_t{pw[4], pw[5], pw[6], pw[7]}));
        if constexpr (FINE) {
          rest0[c] = __builtin_bit_cast(bf16x8_t, (u32x4_t{rw[0], rw[1], rw[2], rw[3]}));
          rest1[c] = __builtin_bit_cast(bf16x8_t, (u32x4_t{rw[4], rw[5], rw[6], rw[7]}));
        }
      }
      for_each(std::make_integer_sequence<int, NB>{}, [&](auto block) {
        constexpr int B = decltype(block)::value;
        bf16x8_t v[2][2];                     // channels 32 B + 2 m and the next, tokens 0-7 and 8-15
        value_pairs(vr[B][0], vr[B][1], row_lane<4 * B>(vsc), row_lane<4 * B + 1>(vsc), v[0][0], v[1][0]);
        value_pairs(vr[B][2], vr[B][3], row_lane<4 * B + 2>(vsc), row_lane<4 * B + 3>(vsc), v[0][1], v[1][1]);
#pragma unroll
        for (int k = 0; k < (FINE ? 4 : 2); k++)
#pragma unroll
          for (int e = 0; e < 2; e++)
#pragma unroll
            for (int c = 0; c < NR; c++)
              o[c][2 * B + e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  v[e][k & 1], k == 0 ? p0[c] : k == 1 ? p1[c] : k == 2 ? rest0[c] : rest1[c], o[c][2 * B + e], 0, 0, 0);
      });
      if (more) {
        load_v(t + step);
        if (t + 2 * step < t1) load_ids(t + 2 * step);
      }
    }
#pragma unroll
    for (int c = 0; c < NR; c++) {
      l[c] += __shfl_xor(l[c], 16, 64);
      l[c] += __shfl_xor(l[c], 32, 64);
    }

    // this wave, or the workgroup, has units [from, to) of the row tile's
    const int64_t from = joined ? g0 : u, to = joined ? g1 : stop;
    const bool whole = SOLO || (from == row_begin && to == row_end);
    const int slot = 2 * (joined ? WAVES * group : x) + (from == row_begin ? 0 : 1);
    if (from == row_begin && !SOLO && (!joined || wave == 0)) {
      KvChain c = none;
      if (!whole) {
        // the last wave: the one whose share holds unit row_end - 1
        const int64_t wide = extra * (least + 1), unit = row_end - 1;
        const int64_t last = unit < wide ? quotient(unit, least + 1) : extra + quotient(unit - wide, least);
        c = KvChain{n_rows, q.q0 + rows.first, rows.head0, joined ? WAVES * group : x, (int)last, joined,
                    share_at((last | (WAVES - 1)) + 1) <= row_end};
        chain = c;
      }
      if (part.by_tile && kvh == 0 && lane == 0 && tile0 + rt < part.chains) part.chain[tile0 + rt] = c;
    }
    auto put = [&](int row, int ch, const f32x4_t& v, float top, float sum) {      // 4 channels of a row
      if (!whole) {
        const int64_t at = ((int64_t)slot * A.kv_heads + kvh) * part.rows + row;
        *reinterpret_cast<f32x4_t*>(part.sums + at * D + ch) = v;
        if (ch == 0) {
          part.stats[2 * at] = top;
          part.stats[2 * at + 1] = sum;
        }
        return;
      }
      const int64_t orow = (int64_t)(q.q0 + rows.first + rows.query(A, row)) * A.q_heads + kvh * A.group + rows.head(A, row);
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      *reinterpret_cast<u32x2_t*>(A.out + orow * D + ch) =
          u32x2_t{pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv)};
      if (A.lse && ch == 0) A.lse[orow] = sum == 0.0f ? -INFINITY : (top + __builtin_log2f(sum)) * LN2;
    };
    // channels 32 b + 8 g + 4 e on of this lane's row, from the tiles of even and odd channels
    auto four = [&](int c, int b, int e) {
      return f32x4_t{o[c][2 * b][2 * e], o[c][2 * b + 1][2 * e], o[c][2 * b][2 * e + 1], o[c][2 * b + 1][2 * e + 1]};
    };
    if (!joined) {
#pragma unroll
      for (int c = 0; c < NR; c++)
        if (16 * c + m < n_rows) {
#pragma unroll
          for (int b = 0; b < NB; b++)
#pragma unroll
            for (int e = 0; e < 2; e++) put(16 * c + m, 32 * b + 8 * g + 4 * e, four(c, b, e), mx[c], l[c]);
        }
      u = stop;
      if (u >= u1) break;
      if (++rt == q.row_tiles) {              // on to the next request that has rows
        begin = row_end;
        tile0 += q.row_tiles;
        rt = 0;
        do {
          request++;
          q.load<R, WHICH>(A, request);
          q = q.from(0);
        } while (q.row_tiles == 0 && request < A.batch);
        if (q.row_tiles == 0) break;
      }
      continue;
    }
#pragma unroll
    for (int c = 0; c < NR; c++) {
      if (g == 0) {
        sm[wave][16 * c + m] = mx[c];
        sl[wave][16 * c + m] = l[c];
      }
#pragma unroll
      for (int b = 0; b < NB; b++)
#pragma unroll
        for (int e = 0; e < 2; e++) *reinterpret_cast<f32x4_t*>(&so[wave][16 * c + m][32 * b + 8 * g + 4 * e]) = four(c, b, e);
    }
    __syncthreads();
    for (int i = tid; i < n_rows * (D / 4); i += 64 * WAVES) {
      const int row = i / (D / 4), ch = i % (D / 4) * 4;
      float top = sm[0][row], sum = 0.0f;
#pragma unroll
      for (int w = 1; w < WAVES; w++) top = __builtin_fmaxf(top, sm[w][row]);
      f32x4_t acc = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < WAVES; w++) {
        const float f = sm[w][row] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(sm[w][row] - top);
        sum = __builtin_fmaf(f, sl[w][row], sum);
        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(&so[w][row][ch]);
#pragma unroll
        for (int e = 0; e < 4; e++) acc[e] = __builtin_fmaf(f, v[e], acc[e]);
      }
      put(row, ch, acc, top, sum);
    }
    break;
  }
  if (each && kvh == 0 && lane == 0) part.chain[x] = chain;
}

// Prompts and chunks, as over the 8-bit cache: 128 rows per workgroup, 32 per
// wave, a tile of 64 tokens converted to bf16 once per workgroup on its way to LDS.
// Bound by the matrix cores and the vector units in turn: three prompts of
// 1500-4096 tokens, 32 heads of 128 on 8 (264 GFLOP) 294-302 us, 875-898 TFLOP/s, where the
// matrix cores are busy 0.38 of the cycles, the vector units 0.50, both 0.16,
// neither 0.28; two chunks on up to 16000 tokens with capped scores 538-543 us with
// four single tokens beside them.  The 8-bit cache's prompts take 304-326 us: what
// halves here is read once per workgroup and was never the bound.
//
// Lane l = 32 h + m.  Within a 32-token half u of the tile, operand row
// 8 (r / 4) + 4 h + r % 4 is token 32 u + 16 h + r: result register r of lane
// half h is that token.  Operand row 16 e + r of V^T tile d is channel 32 d + 2 r + e.
//
// BIG: pages of 64 tokens and more, so that a tile lies in one page and its id
// and addresses are scalars.
template <int D, bool CAP, bool BIG>
__global__ __launch_bounds__(PTHREADS, D == 64 ? 3 : 2) void k_kv4_prompt(const KvArgs A, const KvPart part) {
  constexpr int KS = D / 16, DT = D / 32;     // k steps, channel tiles
  constexpr int XK = D == 128 ? 1 : 2;
  constexpr int W = D / 32;                   // words of K, and of V^T, a thread
  __shared__ __attribute__((aligned(16))) uint8_t sk[3][TILE * D * 2], sv[2][TILE * D * 2];
  const int64_t item = blockIdx.x / (unsigned)A.kv_heads;
  const int kvh = (int)(blockIdx.x % (unsigned)A.kv_heads);
  KvItem it;
  if (!kv_find<PROWS, REQ_LONG>(A, part, item, blockIdx.x == 0, it)) return;
  if (it.splits > 1 && it.slot >= part.slots) return;
  const int tid = threadIdx.x, lane = tid & 63, m = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const KvRows rows(A, it.r0, it.n, it.len);
  int lo, hi, t0, t1;
  kv_tiles(A, it, rows, lo, hi, t0, t1);
  const bool split = it.splits > 1;
  if (split && tid == 0 && kvh == 0)
    part.rec[it.slot] = KvRec{it.split ? 0 : it.splits, it.rows, it.q0 + rows.first, rows.head0};

  const int wrow = wave * 32;                 // first row of the wave in the tile
  const bool live = wrow + m < it.rows;
  const int ri = live ? wrow + m : 0, query = rows.query(A, ri), head = kvh * A.group + rows.head(A, ri);
  const int pos = rows.pos0 + query, rlo = kv_lowest(pos, A.window);
  bf16x8_t qf[KS];
  // limits of the wave's rows; a wave without rows computes nothing
  const int w_rows = it.rows - wrow < 32 ? it.rows - wrow : 32;
  const int w_min = rows.pos0 + rows.query(A, wrow), w_max = rows.pos0 + rows.query(A, wrow + (w_rows > 0 ? w_rows - 1 : 0));
  const int w_lo_max = kv_lowest(w_max, A.window);
  // the table does not change while the kernel runs: scalar loads where the index is uniform
  const __attribute__((address_space(4))) int32_t* tab =
      (const __attribute__((address_space(4))) int32_t*)(A.table + (int64_t)it.request * A.max_blocks);
  const int last_col = (int)A.max_blocks - 1;
  const uint32_t head_bytes = (uint32_t)(D / 2) << A.log_page, page_bytes = head_bytes * A.kv_heads;
  const uint32_t head_scales = (uint32_t)(D / 32) << A.log_page, page_scales = head_scales * A.kv_heads;
  const int in_page = (1 << A.log_page) - 1;
  const uint8_t *ksb = A.k_scales + (int64_t)kvh * head_scales, *vsb = A.v_scales + (int64_t)kvh * head_scales;

  // staging: thread tid takes D / 4 channels of K of token tid / 4, and of V^T the
  // pair of channels vrow at 4 W tokens from vtok
  const int ktok = tid >> 2, kch = D / 4 * (tid & 3);
  const int vrow = D == 128 ? tid >> 2 : tid >> 3, vtok = D == 128 ? 16 * (tid & 3) : 8 * (tid & 7);
  const uint8_t* kbase = A.k_codes + (int64_t)kvh * head_bytes;
  const uint8_t* vbase = A.v_codes + (int64_t)kvh * head_bytes;
  const uint32_t koff = ktok * (D / 2) + kch / 2, kso = ((kch >> 5) << A.log_page) + ktok;
  const uint32_t voff = (vrow << A.log_page) + vtok, vso = ((vrow >> 4) << A.log_page) + vtok;
  uint8_t *kdst[W / 2], *vdst[2];
  {
    const int u = ktok >> 5, th = (ktok >> 4) & 1, tr = ktok & 15, row = 8 * (tr >> 2) + 4 * th + (tr & 3);
#pragma unroll
    for (int i = 0; i < W / 2; i++) {
      const int k = kch / 16 + i;
      kdst[i] = sk[0] + ((u * KS + k) * 64 + (row ^ (XK * k))) * 16;
    }
    const int tg = vtok >> 4;
#pragma unroll
    for (int e = 0; e < 2; e++)
      vdst[e] = sv[0] + (((vrow >> 4) * 4 + 2 * (tg >> 1) + ((vtok >> 3) & 1)) * 64 + 32 * (tg & 1) +
                         (((vrow & 15) + 16 * e) ^ (2 * tg))) * 16;
  }
  constexpr int BUF = TILE * D * 2;
  uint32_t kr[W], vr[W], vsc[W], ksc;
  bool vok;
  // page ids on their way: of the next K, V^T and, in score layout, the masks;
  // with BIG pages of tiles t .. t + 4
  int idk, idv, idm[2], idn[2], ids[5];
  auto page_id = [&](int t, int tok) {        // past t1 the last tile again: loaded, never used
    const int c = ((t < t1 ? t : t1 - 1) * TILE + tok) >> A.log_page;
    return tab[c < last_col ? c : last_col];
  };
  auto there = [&](int id) { return id >= 0 && id < A.num_pages; };
  auto ids_k = [&](int t) {
    if constexpr (!BIG) idk = page_id(t, ktok);
  };
  auto ids_v = [&](int t) {
    if constexpr (!BIG) idv = page_id(t, vtok);
  };
  auto ids_m = [&](int t) {
    if constexpr (!BIG) {
#pragma unroll
      for (int u = 0; u < 2; u++) idn[u] = page_id(t, 32 * u + 16 * h);
    }
  };
  auto words = [&](uint32_t (&w)[W], const uint8_t* p) {
    if constexpr (D == 128) {
      const u32x4_t x = ld16(p);
#pragma unroll
      for (int i = 0; i < W; i++) w[i] = x[i];
    } else {
      const u32x2_t x = *reinterpret_cast<const u32x2_t*>(p);
#pragma unroll
      for (int i = 0; i < W; i++) w[i] = x[i];
    }
  };
  auto load_k = [&](int t, int id) {
    if constexpr (BIG) {
      const uint64_t block = (uint64_t)(uint32_t)(there(id) ? id : 0);
      const uint32_t off = (uint32_t)((t * TILE) & in_page);
      ksc = (ksb + (block * page_scales + off))[kso];
      words(kr, kbase + (block * page_bytes + off * (D / 2)) + koff);
    } else {
      const uint64_t block = (uint64_t)(uint32_t)(there(idk) ? idk : 0);
      const uint32_t off = (uint32_t)((t * TILE + ktok) & in_page);
      ksc = ksb[block * page_scales + ((kch >> 5) << A.log_page) + off];
      words(kr, kbase + (block * page_bytes + off * (D / 2) + kch / 2));
    }
  };
  auto load_v = [&](int t, int id) {
    if constexpr (BIG) {
      vok = there(id);
      const uint64_t block = (uint64_t)(uint32_t)(vok ? id : 0);
      const uint32_t off = (uint32_t)((t * TILE) & in_page);
      words(vsc, vsb + (block * page_scales + off) + vso);
      words(vr, vbase + (block * page_bytes + off) + voff);
    } else {
      vok = there(idv);
      const uint64_t block = (uint64_t)(uint32_t)(vok ? idv : 0);
      const uint32_t off = (uint32_t)((t * TILE + vtok) & in_page);
      words(vsc, vsb + (block * page_scales + ((vrow >> 4) << A.log_page) + off));
      words(vr, vbase + (block * page_bytes + (vrow << A.log_page) + off));
    }
  };
  auto store_k = [&](int at) {
    const float s = scale_of(ksc, 0);
#pragma unroll
    for (int i = 0; i < W; i++)
      *reinterpret_cast<bf16x8_t*>(kdst[i >> 1] + at + 32 * 16 * (i & 1)) = e2m1_bf16x8(kr[i], s);
  };
  KvAlike alike(rows.pos0, rows.pos0 + rows.query(A, it.rows - 1), A.window);
  alike.lo = alike.lo > lo ? alike.lo : lo;   // and nothing of theirs is unseen
  alike.hi = alike.hi < hi ? alike.hi : hi;
  auto store_v = [&](int t, int buf) {
    if (!vok || !alike(t * TILE + (vtok & ~15))) {   // scales of tokens that not every row sees stay finite
#pragma unroll
      for (int i = 0; i < W; i++) vsc[i] = finite_scales(vsc[i]);
    }
#pragma unroll
    for (int i = 0; i < W / 2; i++) {
      bf16x8_t v[2];
      value_pairs(vr[2 * i], vr[2 * i + 1], vsc[2 * i], vsc[2 * i + 1], v[0], v[1]);
#pragma unroll
      for (int e = 0; e < 2; e++) *reinterpret_cast<bf16x8_t*>(vdst[e] + buf * BUF + 64 * 16 * i) = v[e];
    }
  };
  if (t0 < t1) {
    if constexpr (BIG) {
#pragma unroll
      for (int i = 0; i < 5; i++) ids[i] = page_id(t0 + i, 0);
    }
    ids_k(t0);
    ids_v(t0);
    ids_m(t0);
    load_k(t0, ids[0]);
    load_v(t0, ids[0]);
    ids_k(t0 + 1);
    ids_v(t0 + 1);
    if constexpr (!BIG) {
      idm[0] = idn[0];
      idm[1] = idn[1];
    }
    ids_m(t0 + 1);
  }
  {
    const uint16_t* qp = A.q + (int64_t)(it.q0 + rows.first + query) * A.q_stride + head * D;
#pragma unroll
    for (int k = 0; k < KS; k++) {
      u32x4_t w = ld16(qp + 16 * k + 8 * h);
      if (!live) w = u32x4_t{0, 0, 0, 0};
      qf[k] = __builtin_bit_cast(bf16x8_t, w);
    }
  }

  f32x16_t o[DT];
#pragma unroll
  for (int d = 0; d < DT; d++)
#pragma unroll
    for (int i = 0; i < 16; i++) o[d][i] = 0.0f;
  float mx = -INFINITY, l = 0.0f;
  const KvScore<CAP> sc(A);
  const uint8_t* kfrag = sk[0] + (32 * h) * 16;
  const uint8_t* vfrag[2];
#pragma unroll
  for (int u = 0; u < 2; u++) vfrag[u] = sv[0] + (128 * u + 32 * h + (m ^ (2 * (2 * u + h)))) * 16;
  constexpr int HOLD = D == 128 ? 6 : 4;      // fragments read ahead of their use
  bf16x8_t kf[HOLD];
  auto frag_k = [&](int at, int u, int k) {
    return *reinterpret_cast<const bf16x8_t*>(kfrag + at + (u * KS + k) * 1024 + (m ^ (XK * k)) * 16);
  };
  auto fetch = [&](int at, int u) {
#pragma unroll
    for (int k = 0; k < HOLD; k++) kf[k] = frag_k(at, u, k);
  };
  auto scores = [&](int at, int u) {          // of half u of the tile whose K begins at `at`
    f32x16_t z;
#pragma unroll
    for (int i = 0; i < 16; i++) z[i] = 0.0f;
    bf16x8_t rest[KS > HOLD ? KS - HOLD : 1];
#pragma unroll
    for (int k = HOLD; k < KS; k++) rest[k - HOLD] = frag_k(at, u, k);
    __builtin_amdgcn_sched_barrier(0x47F);    // LDS reads stay where they are
#pragma unroll
    for (int k = 0; k < KS; k++)
      z = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k < HOLD ? kf[k] : rest[k - HOLD], qf[k], z, 0, 0, 0);
    return z;
  };
  // caps and masks the scores of half u of tile t and moves the running
  // maximum: only when a score passes it by 2^8, for the sums hold that and
  // the result is the same
  auto settle = [&](int t, int u, f32x16_t& s) {
    const int j0 = t * TILE + 32 * u;
    const bool ok = there(BIG ? ids[0] : idm[u]);
    const bool edge = j0 + 31 > w_min || j0 < w_lo_max || (BIG ? !ok : __any(!ok));
    sc.cap(s, edge);
    if (edge) {
      const int j = j0 + 16 * h, z = ok ? pos - j : -1, b = rlo - j;
#pragma unroll
      for (int i = 0; i < 16; i++) s[i] = i <= z && i >= b ? s[i] : -INFINITY;
    }
    float mt = -INFINITY;
#pragma unroll
    for (int i = 0; i < 16; i++) mt = __builtin_fmaxf(mt, s[i]);
    const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(mt), __float_as_uint(mt), false, false);
    mt = __builtin_fmaxf(__uint_as_float(both[0]), __uint_as_float(both[1])) * sc.mul;
    if (__any(mt > mx + 8.0f)) {
      const float mn = __builtin_fmaxf(mx, mt);
      const float f = mx == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mx - mn);
      mx = mn;
      l *= f;
#pragma unroll
      for (int d = 0; d < DT; d++) o[d] *= f;
    }
  };
  auto weigh = [&](int buf, int u, const f32x16_t& s, int at, int un) {   // probabilities, and their sums of V
    const float off = mx == -INFINITY ? 0.0f : -mx;
    bf16x8_t v0[DT], v1[DT];
#pragma unroll
    for (int d = 0; d < DT; d++) v0[d] = *reinterpret_cast<const bf16x8_t*>(vfrag[u] + buf * BUF + d * 4096);
    __builtin_amdgcn_sched_barrier(0x47F);    // LDS reads stay where they are
    uint32_t pw[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float a = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * i], sc.mul, off));
      const float b = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * i + 1], sc.mul, off));
      l += a + b;
      pw[i] = pack_bf16x2(a, b);              // off by up to 2^-8 of a probability, l keeps fp32 (a second
                                              // term for the rest: 297 -> 388 us, capped 538 -> 701)
    }
#pragma unroll
    for (int d = 0; d < DT; d++) v1[d] = *reinterpret_cast<const bf16x8_t*>(vfrag[u] + buf * BUF + d * 4096 + 1024);
    const bf16x8_t p0 = __builtin_bit_cast(bf16x8_t, (u32x4_t{pw[0], pw[1], pw[2], pw[3]}));
    const bf16x8_t p1 = __builtin_bit_cast(bf16x8_t, (u32x4_t{pw[4], pw[5], pw[6], pw[7]}));
#pragma unroll
    for (int d = 0; d < DT; d++) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v0[d], p0, o[d], 0, 0, 0);
    fetch(at, un);
    __builtin_amdgcn_sched_barrier(0x47F);    // LDS reads stay where they are
#pragma unroll
    for (int d = 0; d < DT; d++) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v1[d], p1, o[d], 0, 0, 0);
  };
  // at the top of a step: first half of tile t settled, K of t and t + 1 and
  // V^T of t in LDS, K of t + 2 and V^T of t + 1 on their way to registers
  f32x16_t s0, s1;
  int k0 = 0, k1 = BUF, k2 = 2 * BUF;         // K of t, t + 1, t + 2
  if (t0 < t1) {
    store_k(k0);
    store_v(t0, 0);
    load_k(t0 + 1, ids[1]);
    load_v(t0 + 1, ids[1]);
    ids_k(t0 + 2);
    ids_v(t0 + 2);
    store_k(k1);
    load_k(t0 + 2, ids[2]);
    ids_k(t0 + 3);
    tile_barrier();
    if (w_rows > 0) {
      fetch(k0, 0);
      s0 = scores(k0, 0);
      fetch(k0, 1);
      settle(t0, 0, s0);
    }
  }
  for (int t = t0; t < t1; t++) {
    const int buf = (t - t0) & 1;
    if (w_rows > 0) {
      s1 = scores(k0, 1);
      weigh(buf, 0, s0, k1, 0);
      settle(t, 1, s1);
      s0 = scores(k1, 0);                     // behind the last tile: not used
      weigh(buf, 1, s1, k1, 1);
    }
    if (t + 1 == t1) break;
    store_k(k2);
    store_v(t + 1, buf ^ 1);
    load_k(t + 3, ids[3]);
    load_v(t + 2, ids[2]);
    ids_k(t + 4);
    ids_v(t + 3);
    tile_barrier();
    if constexpr (BIG) {
#pragma unroll
      for (int i = 0; i < 4; i++) ids[i] = ids[i + 1];
      ids[4] = page_id(t + 5, 0);
    } else {
      idm[0] = idn[0];
      idm[1] = idn[1];
      ids_m(t + 2);
    }
    if (w_rows > 0) settle(t + 1, 0, s0);
    const int k = k0;
    k0 = k1;
    k1 = k2;
    k2 = k;
  }
  l += __shfl_xor(l, 32, 64);
  if (!live) return;
  // channels 32 d + 16 i + 8 h + 2 j and the next: registers 4 i + j and 4 i + 8 + j of tile d
  const int64_t orow = (int64_t)(it.q0 + rows.first + query) * A.q_heads + head;
  if (split) {
    const int64_t at = (it.slot * A.kv_heads + kvh) * PROWS + wrow + m;
#pragma unroll
    for (int d = 0; d < DT; d++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int r = 4 * (i >> 1) + 2 * (i & 1);
        *reinterpret_cast<f32x4_t*>(part.sums + at * D + 32 * d + 16 * (i >> 1) + 8 * h + 4 * (i & 1)) =
            f32x4_t{o[d][r], o[d][r + 8], o[d][r + 1], o[d][r + 9]};
      }
    if (h == 0) {
      part.stats[2 * at] = mx;
      part.stats[2 * at + 1] = l;
    }
    return;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int d = 0; d < DT; d++)
#pragma unroll
    for (int i = 0; i < 2; i++) {
      u32x4_t w;
#pragma unroll
      for (int j = 0; j < 4; j++) w[j] = pack_bf16x2(o[d][4 * i + j] * inv, o[d][4 * i + 8 + j] * inv);
      *reinterpret_cast<u32x4_t*>(A.out + orow * D + 32 * d + 16 * i + 8 * h) = w;
    }
  if (A.lse && h == 0) A.lse[orow] = l == 0.0f ? -INFINITY : (mx + __builtin_log2f(l)) * LN2;
}

// Workgroups of 8 waves for row tiles of their own, where each has a CU (8 heads of 128: 1 x 1000
// tokens 9.3 -> 9.0 us, 16 x 2000 16.3 -> 14.0; 33 x 1000, 264 workgroups, 14.2 -> 17.1).
constexpr unsigned SOLO_WIDE = 256;

template <int D, bool CAP>
void launch_attention(const KvArgs& A, const KvPlan& p, const KvShare& dec, const KvPart& pro, hipStream_t s) {
  const unsigned h = (unsigned)A.kv_heads, groups = (unsigned)p.groups * h;
  if (p.prompt) {
    const unsigned items = (unsigned)p.pro_items * h;
    if (A.log_page >= 6) k_kv4_prompt<D, CAP, true><<<items, PTHREADS, 0, s>>>(A, pro);
    else k_kv4_prompt<D, CAP, false><<<items, PTHREADS, 0, s>>>(A, pro);
    k_kv4_decode<D, CAP, REQ_SHORT, 2, false><<<groups, KV_THREADS, 0, s>>>(A, dec);
  } else if (p.solo) {
    if (p.nr == 2) k_kv4_decode<D, CAP, REQ_ALL, 2, true><<<groups, KV_THREADS, 0, s>>>(A, dec);
    else if (groups <= SOLO_WIDE) k_kv4_decode<D, CAP, REQ_ALL, 1, true, 8><<<groups, 512, 0, s>>>(A, dec);
    else k_kv4_decode<D, CAP, REQ_ALL, 1, true><<<groups, KV_THREADS, 0, s>>>(A, dec);
    return;
  } else if (p.nr == 2) {
    k_kv4_decode<D, CAP, REQ_ALL, 2, false><<<groups, KV_THREADS, 0, s>>>(A, dec);
  } else {
    k_kv4_decode<D, CAP, REQ_ALL, 1, false><<<groups, KV_THREADS, 0, s>>>(A, dec);
  }
  const unsigned joins = ((unsigned)dec.chains * h << dec.log_joins) + (unsigned)(p.pro_slots * (PROWS / 16)) * h;
  if (p.nr == 2) k_kv_join<D, 2><<<joins, KV_THREADS, 0, s>>>(A, dec, pro);
  else k_kv_join<D, 1><<<joins, KV_THREADS, 0, s>>>(A, dec, pro);
}

}  // namespace

extern "C" {

size_t wq_kv4_attention_workspace_size(int64_t batch, int64_t tokens, int64_t max_q, int32_t q_heads, int32_t kv_heads,
                                       int32_t head_dim, int32_t page, int64_t max_blocks, int64_t window) {
  if (window < 0 || (head_dim != 64 && head_dim != 128) || log2_page(page) < 0 ||
      !kv_sizes_ok(batch, tokens, max_q, q_heads, kv_heads, page, max_blocks))
    return 0;
  return batch && tokens ? kv_plan(batch, tokens, max_q, q_heads, kv_heads, head_dim, page, max_blocks, window).bytes : 0;
}

wq_status wq_kv4_attention(const void* q_bf16, int64_t q_stride, const int32_t* cu_q, const int32_t* kv_lens,
                           int64_t batch, int64_t tokens, int64_t max_q, int32_t q_heads, int32_t kv_heads,
                           int32_t head_dim, const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes,
                           const uint8_t* v_scales, int32_t page, int64_t num_pages, const int32_t* block_table,
                           int64_t max_blocks, float sm_scale, float softcap, int64_t window, uint16_t* out,
                           float* lse, void* workspace, size_t ws_bytes, void* stream) {
  const KvCall c = {q_bf16, q_stride, cu_q, kv_lens, batch, tokens, max_q, q_heads, kv_heads, head_dim, k_codes, k_scales,
                    v_codes, v_scales, page, num_pages, block_table, max_blocks, sm_scale, softcap, window, out, lse,
                    workspace, ws_bytes};
  if (const wq_status bad = kv_check(c)) return bad;
  if (!wq_aligned(k_scales) || !wq_aligned(v_scales)) return WQ_EALIGN;
  if (batch == 0 || tokens == 0) return WQ_OK;               // nothing to compute
  KvLaunch l;
  if (const wq_status bad = l.lay_out(c)) return bad;
  if (!l.plan.solo && l.plan.chains < l.dec.chains) {         // row tiles are fewer than waves
    l.dec.chains = l.plan.chains;
    l.dec.by_tile = true;
    // few workgroups to join them then: half the rows each (24 requests of 1-7 drafted tokens 30.2 -> 29.1 us)
    if (l.plan.nr == 2) l.dec.log_joins++;
  }
  hipStream_t s = wq_stream(stream);
  if (head_dim == 128) {
    if (softcap > 0.0f) launch_attention<128, true>(l.args, l.plan, l.dec, l.pro, s);
    else launch_attention<128, false>(l.args, l.plan, l.dec, l.pro, s);
  } else {
    if (softcap > 0.0f) launch_attention<64, true>(l.args, l.plan, l.dec, l.pro, s);
    else launch_attention<64, false>(l.args, l.plan, l.dec, l.pro, s);
  }
  return wq_launch_status();
}

}  // extern "C"

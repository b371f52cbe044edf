// 8-bit key/value cache for gfx950: block tables and slot maps from request
// lengths, the append that quantizes new keys and values into their pages
// (E4M3 elements, one E8M0 scale per page and head), and the attention that
// reads the pages.
#include <hip/hip_runtime.h>

#include "wq.h"
#include "wq_device.h"
#include "wq_host.h"

using namespace wq;

namespace {

constexpr int KV_THREADS = 256;
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------------------
// Block tables and slot maps
// ---------------------------------------------------------------------------
// Sum of v over the lower lanes of the wave and this one.
__device__ __forceinline__ int64_t wave_scan(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t u = __shfl_up(v, o, 64);
    if (lane >= o) v += u;
  }
  return v;
}

// The first of `count` running sums that is above v (the last one is).
__device__ __forceinline__ int first_above(const int64_t* sums, int count, int64_t v) {
  int a = 0, z = count - 1;
  while (a < z) {
    const int mid = (a + z) >> 1;
    if (sums[mid] > v) z = mid;
    else a = mid + 1;
  }
  return a;
}

// Every workgroup scans the lengths of all requests (256 at a time: running
// sums of new tokens and of the pages needed, kept in LDS for the chunk) and
// writes its own rows of the token arrays, found by binary search in the
// chunk's token ends, and its share of the new table entries, found in the
// same way.  Workgroup 0 writes the per-request outputs.  There is no
// dependence between workgroups, so one launch does it all: the new pages of a
// token come from the free list itself, not from the table that another
// workgroup fills.  Bound by latency: 4.4 us for 256 requests of one token,
// 4.0 us for 7 prompts of 16384 tokens (an empty launch takes 2.5 us).
__global__ __launch_bounds__(KV_THREADS) void k_kv_blocks(
    const int32_t* __restrict__ ctx_lens, const int32_t* __restrict__ new_lens, int64_t batch,
    const int32_t* __restrict__ free_pages, int64_t num_free, const int32_t* __restrict__ cursor, int log_page,
    int32_t* __restrict__ table, int64_t max_blocks, int64_t tokens, int64_t* __restrict__ slots,
    int32_t* __restrict__ positions, int32_t* __restrict__ cu_new, int32_t* __restrict__ kv_lens,
    int32_t* __restrict__ state) {
  __shared__ int64_t ends[KV_THREADS];       // token rows up to and with each request of the chunk
  __shared__ int64_t page_ends[KV_THREADS];  // places of free_pages up to and with its new pages
  __shared__ int64_t firsts[KV_THREADS];     // the place of its first new page, -1 if refused
  __shared__ int32_t ctxs[KV_THREADS];
  __shared__ int32_t news[KV_THREADS];
  __shared__ int64_t wave_sum[2][KV_THREADS / 64];
  __shared__ int64_t used_sum[KV_THREADS / 64];
  __shared__ int32_t refused_sum[KV_THREADS / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t page = (int64_t)1 << log_page;
  const int64_t row0 = (int64_t)blockIdx.x * KV_THREADS, row1 = row0 + KV_THREADS < tokens ? row0 + KV_THREADS : tokens;
  const bool lead = blockIdx.x == 0;
  const int64_t start = cursor && cursor[0] > 0 ? cursor[0] : 0;
  int64_t tok_before = 0, page_before = start, used = 0;
  int32_t refused = 0;
  for (int64_t base = 0; base < batch; base += KV_THREADS) {
    const int64_t i = base + tid;
    int32_t c = i < batch ? ctx_lens[i] : 0, n = i < batch ? new_lens[i] : 0;
    c = c > 0 ? c : 0;
    n = n > 0 ? n : 0;
    const int64_t after = (int64_t)c + n;
    const int64_t held = (c + page - 1) >> log_page, total = (after + page - 1) >> log_page;
    const bool fits = total <= max_blocks && after <= 0x7FFFFFFF;
    const int64_t need = fits ? total - held : 0;
    int64_t tok = wave_scan(n, lane), pg = wave_scan(need, lane);
    __syncthreads();                          // the previous chunk's arrays are no longer read
    if (lane == 63) {
      wave_sum[0][wave] = tok;
      wave_sum[1][wave] = pg;
    }
    __syncthreads();
    for (int w = 0; w < wave; w++) {
      tok += wave_sum[0][w];
      pg += wave_sum[1][w];
    }
    const int64_t end = tok_before + tok, first = page_before + pg - need;
    const bool ok = fits && first + need <= num_free + (need ? 0 : first) && end <= tokens;
    ends[tid] = end;
    firsts[tid] = ok ? first : -1;
    ctxs[tid] = c;
    news[tid] = n;
    if (i < batch) {
      used += ok ? need : 0;
      refused += ok ? 0 : 1;
      if (lead) {
        cu_new[i + 1] = (int32_t)(end < tokens ? end : tokens);
        kv_lens[i] = ok ? (int32_t)after : c;
      }
    }
    page_ends[tid] = first + need;
    const int64_t tok_first = tok_before, page_first = page_before;
    for (int w = 0; w < KV_THREADS / 64; w++) {
      tok_before += wave_sum[0][w];
      page_before += wave_sum[1][w];
    }
    __syncthreads();
    const int count = (int)(batch - base < KV_THREADS ? batch - base : KV_THREADS);
    // table entries: the chunk's new pages in turn, each found in the running sums
    const int64_t pages = page_before - page_first;
    for (int64_t j = (int64_t)blockIdx.x * KV_THREADS + tid; j < pages; j += (int64_t)gridDim.x * KV_THREADS) {
      const int a = first_above(page_ends, count, page_first + j);
      const int64_t col = (((int64_t)ctxs[a] + news[a] + page - 1) >> log_page) - (page_ends[a] - (page_first + j));
      if (firsts[a] >= 0) table[(base + a) * max_blocks + col] = free_pages[page_first + j];
    }
    // token rows of this chunk's requests
    const int64_t lo = row0 > tok_first ? row0 : tok_first, hi = row1 < tok_before ? row1 : tok_before;
    for (int64_t row = lo + tid; row < hi; row += KV_THREADS) {
      const int a = first_above(ends, count, row);
      int64_t slot = -1;
      const int64_t pos = ctxs[a] + row - (ends[a] - news[a]);
      if (firsts[a] >= 0) {
        const int64_t h = (ctxs[a] + page - 1) >> log_page, col = pos >> log_page;
        const int64_t id = col < h ? table[(base + a) * max_blocks + col] : free_pages[firsts[a] + col - h];
        if (id >= 0) slot = (id << log_page) + (pos & (page - 1));
      }
      slots[row] = slot;
      positions[row] = slot >= 0 ? (int32_t)pos : -1;
    }
  }
  for (int64_t row = (row0 > tok_before ? row0 : tok_before) + tid; row < row1; row += KV_THREADS) {
    slots[row] = -1;
    positions[row] = -1;
  }
  if (lead) {
    used = wave_scan(used, lane);
    const int64_t ref = wave_scan(refused, lane);
    if (lane == 63) {
      used_sum[wave] = used;
      refused_sum[wave] = (int32_t)ref;
    }
    __syncthreads();
    if (tid == 0) {
      int64_t u = start;
      int32_t r = 0;
      for (int w = 0; w < KV_THREADS / 64; w++) {
        u += used_sum[w];
        r += refused_sum[w];
      }
      cu_new[0] = 0;
      state[0] = (int32_t)u;
      state[1] = r;
    }
  }
}

// ---------------------------------------------------------------------------
// Append
// ---------------------------------------------------------------------------
// Four fp32 -> four E4M3 bytes, RNE, saturating, NaN -> 0x7F with its sign.
__device__ __forceinline__ uint32_t e4m3_word(const float v[4]) {
  uint32_t r = e4m3_pack2<false>(clamp448(v[0]), clamp448(v[1]), 0u);
  r = e4m3_pack2<true>(clamp448(v[2]), clamp448(v[3]), r);
#pragma unroll
  for (int i = 0; i < 4; i++)
    if (v[i] != v[i]) r = (r & ~(0xFFu << (8 * i))) | ((0x7Fu | ((__float_as_uint(v[i]) >> 24) & 0x80u)) << (8 * i));
  return r;
}

// Four E4M3 bytes times 2^shift, rounded again.
__device__ __forceinline__ uint32_t e4m3_word_shifted(uint32_t w, int shift) {
  const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, 1.0f, false);
  const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, 1.0f, true);
  const float v[4] = {__builtin_ldexpf(a[0], shift), __builtin_ldexpf(a[1], shift), __builtin_ldexpf(b[0], shift),
                      __builtin_ldexpf(b[1], shift)};
  return e4m3_word(v);
}

// The least E8M0 code c with amax <= 448 * 2^(c-127), amax as its bits: 448 = 1.75 * 2^8, so
// the biased exponent less 8, one more where the fraction is above .75.
__device__ __forceinline__ int e8m0_cover(uint32_t bits) {
  const int c = (int)(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return c > 0 ? c : 0;
}

// Eight elements as they were loaded.
template <bool BF16>
struct Raw8 {
  uint32_t w[BF16 ? 4 : 8];
  // the larger of m and the magnitudes, as bit patterns: one half word each for
  // bf16 (both halves of m), one word for fp32; NaN and infinity come out largest
  __device__ __forceinline__ uint32_t magnitude(uint32_t m) const {
#pragma unroll
    for (int i = 0; i < (BF16 ? 4 : 8); i++) {
      if constexpr (BF16) {
        const u16x2_t a = __builtin_bit_cast(u16x2_t, w[i] & 0x7FFF7FFFu), b = __builtin_bit_cast(u16x2_t, m);
        m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(a, b));
      } else {
        const uint32_t a = w[i] & 0x7FFFFFFFu;
        m = a > m ? a : m;
      }
    }
    return m;
  }
  __device__ __forceinline__ void widen(float v[8]) const {
#pragma unroll
    for (int i = 0; i < 8; i++)
      v[i] = BF16 ? (i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2])) : __uint_as_float(w[BF16 ? 0 : i]);
  }
  // E4M3 codes of x * 2^(127-c); the finite magnitudes are at most 448 then
  __device__ __forceinline__ u32x2_t codes(float scale_as_e8m0) const {
    u32x2_t out;
#pragma unroll
    for (int h = 0; h < 2; h++) {
      s16x2_t r = {0, 0};
      if constexpr (BF16) {
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, w[2 * h]), scale_as_e8m0, false);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, w[2 * h + 1]), scale_as_e8m0, true);
      } else {
        const uint32_t* f = w + (BF16 ? 0 : 4 * h);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, __uint_as_float(f[0]), __uint_as_float(f[1]), scale_as_e8m0, false);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, __uint_as_float(f[2]), __uint_as_float(f[3]), scale_as_e8m0, true);
      }
      out[h] = __builtin_bit_cast(uint32_t, r);
    }
    return out;
  }
};

// One run (tokens t .. t+n-1 at offsets off .. off+n-1 of one page) of one
// head, keys or values, by the whole workgroup.  A thread takes 8 channels of
// the 4 tokens of an aligned quad of the page and keeps them in registers
// between the run's maximum and its codes: values then leave as words of 4
// tokens, which LDS turns into whole rows of the transposed page.  Bound by
// bytes, so the arithmetic is kept to one and a half instructions an element:
// maxima of bit patterns, two for bf16 at a time, and conversions that take
// the scale; a run that holds a NaN or an infinity goes the long way.  8192
// tokens of prompts, 8 heads of 128, bf16: 13.3 us a call (3.8 TB/s).
template <bool BF16, bool VALUES, int D, int PAGE>
__device__ __forceinline__ void append_run(const void* __restrict__ x, int64_t stride, int64_t t, int n, int off,
                                           uint8_t* __restrict__ codes, uint8_t* __restrict__ scale, uint8_t* lds,
                                           uint32_t* red) {
  constexpr int CH = D / 8, ITEMS = PAGE / 4 * CH, R = (ITEMS + KV_THREADS - 1) / KV_THREADS, LROW = PAGE + 4;
  const int tid = threadIdx.x, end = off + n;
  const int old = off ? (int)*scale : 0;
  Raw8<BF16> v[R][4];
  uint32_t m = 0;
#pragma unroll
  for (int r = 0; r < R; r++) {
    const int p = r * KV_THREADS + tid, o = p / CH * 4;            // o: first offset of the quad
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const bool in = o + i >= off && o + i < end;
      const uint8_t* from = (const uint8_t*)x + ((t + (in ? o + i - off : 0)) * stride + (p % CH) * 8) * (BF16 ? 2 : 4);
#pragma unroll
      for (int e = 0; e < (BF16 ? 1 : 2); e++) {
        const u32x4_t q = in ? ld16(from + 16 * e) : u32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int b = 0; b < 4; b++) v[r][i].w[4 * e + b] = q[b];
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; r++)
#pragma unroll
    for (int i = 0; i < 4; i++) m = v[r][i].magnitude(m);
  if constexpr (BF16) m = (m & 0xFFFFu) > (m >> 16) ? m << 16 : m & 0xFFFF0000u;
  auto join = [&](uint32_t a) {               // the largest over the workgroup
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t b = (uint32_t)__shfl_xor((int)a, o, 64);
      a = a > b ? a : b;
    }
    if ((tid & 63) == 0) red[tid >> 6] = a;
    __syncthreads();
    a = red[0] > red[1] ? red[0] : red[1];
    const uint32_t b = red[2] > red[3] ? red[2] : red[3];
    return a > b ? a : b;
  };
  m = join(m);
  const bool odd = m >= 0x7F800000u;          // NaN or infinity: the maximum of the others, element by element
  if (odd) {
    m = 0;
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        float f[8];
        v[r][i].widen(f);
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const uint32_t a = __float_as_uint(f[e]) & 0x7FFFFFFFu;
          m = a < 0x7F800000u && a > m ? a : m;
        }
      }
    __syncthreads();
    m = join(m);
  }
  const int need = e8m0_cover(m);
  const int c = need > old ? need : old;
  const int moved = off && c > old ? off : 0; // tokens before the run whose codes change
  if (tid == 0 && (!off || c != old)) *scale = (uint8_t)c;
  const float sc = e8m0_as_scale((uint32_t)c);
#pragma unroll
  for (int r = 0; r < R; r++) {
    const int p = r * KV_THREADS + tid, o = p / CH * 4, ch = (p % CH) * 8;
    if (o + 3 < off || o >= end) continue;
    u32x2_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if (!odd) {
        w[i] = v[r][i].codes(sc);
      } else {
        float q[8];
        v[r][i].widen(q);
#pragma unroll
        for (int e = 0; e < 8; e++) q[e] = __builtin_ldexpf(q[e], 127 - c);
        w[i] = u32x2_t{e4m3_word(q), e4m3_word(q + 4)};
      }
    }
    if constexpr (!VALUES) {
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (o + i >= off && o + i < end) *reinterpret_cast<u32x2_t*>(codes + (o + i) * D + ch) = w[i];
    } else {
      // 4 tokens x 4 channels at a time: bytes of one channel into one word
#pragma unroll
      for (int hf = 0; hf < 2; hf++) {
        const uint32_t lo01 = __builtin_amdgcn_perm(w[1][hf], w[0][hf], 0x05010400u);
        const uint32_t hi01 = __builtin_amdgcn_perm(w[1][hf], w[0][hf], 0x07030602u);
        const uint32_t lo23 = __builtin_amdgcn_perm(w[3][hf], w[2][hf], 0x05010400u);
        const uint32_t hi23 = __builtin_amdgcn_perm(w[3][hf], w[2][hf], 0x07030602u);
        uint32_t* l = reinterpret_cast<uint32_t*>(lds + (ch + 4 * hf) * LROW + o);
        l[0] = __builtin_amdgcn_perm(lo23, lo01, 0x05040100u);
        l[LROW / 4] = __builtin_amdgcn_perm(lo23, lo01, 0x07060302u);
        l[2 * (LROW / 4)] = __builtin_amdgcn_perm(hi23, hi01, 0x05040100u);
        l[3 * (LROW / 4)] = __builtin_amdgcn_perm(hi23, hi01, 0x07060302u);
      }
    }
  }
  if constexpr (!VALUES) {
    for (int p = tid; p < moved * D / 4; p += KV_THREADS) {
      uint32_t* w = reinterpret_cast<uint32_t*>(codes) + p;
      *w = e4m3_word_shifted(*w, old - c);
    }
  } else {
    __syncthreads();
    if (n == PAGE) {                          // a whole page: 16-byte stores
      for (int p = tid; p < D * PAGE / 16; p += KV_THREADS) {
        const uint32_t* l = reinterpret_cast<const uint32_t*>(lds + p / (PAGE / 16) * LROW + p % (PAGE / 16) * 16);
        *reinterpret_cast<u32x4_t*>(codes + p * 16) = u32x4_t{l[0], l[1], l[2], l[3]};
      }
    } else {
      const int w0 = moved ? 0 : off >> 2, words = ((end + 3) >> 2) - w0;
      for (int p = tid; p < D * words; p += KV_THREADS) {
        const int d = p / words, w = w0 + p % words;
        uint8_t* g = codes + d * PAGE + 4 * w;
        // bytes [a, z) of the word are this run's
        const int a = off - 4 * w > 0 ? off - 4 * w : 0, z = end - 4 * w < 4 ? end - 4 * w : 4;
        const uint32_t fresh = a < 4 ? *reinterpret_cast<const uint32_t*>(lds + d * LROW + 4 * w) : 0u;
        if (a == 0 && z == 4) {
          *reinterpret_cast<uint32_t*>(g) = fresh;
        } else if (moved && a > 0) {
          const uint32_t had = *reinterpret_cast<const uint32_t*>(g);
          const uint32_t kept = e4m3_word_shifted(had, old - c);
          uint32_t res = 0;
#pragma unroll
          for (int b = 0; b < 4; b++) res |= (b < a ? kept : b < z ? fresh : had) & (0xFFu << (8 * b));
          *reinterpret_cast<uint32_t*>(g) = res;
        } else {
          for (int b = a; b < z; b++) g[b] = (uint8_t)(fresh >> (8 * b));
        }
      }
    }
  }
  __syncthreads();                            // LDS is free for the next run
}

// Runs of one token each (a decode step): `runs` has the chunk's tokens that
// begin one, `slot` the slot of token t0 + lane.  D / 8 lanes a token, many
// tokens at once and no barrier among them; the pages whose scale grew are
// gone over by the whole workgroup afterwards.  64 tokens, 8 heads of 128: 4.2
// us where no scale grows (5.3 as runs), 7.8 us where half of the pages' do and
// 8.5 us where all do; 2048: 66 us, bound by the cache line that each value
// byte of the transposed page touches (76 as runs).
template <bool BF16, bool VALUES, int D, int PAGE>
__device__ __forceinline__ void append_ones(const void* __restrict__ x, int64_t stride, int64_t t0, int chunk,
                                            unsigned long long runs, int64_t slot, int heads, int head,
                                            uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int* grown) {
  constexpr int GL = D / 8, AT_ONCE = KV_THREADS / GL;
  const int tid = threadIdx.x, lane = tid & 63, ch = tid % GL * 8;
  if (tid < 64) grown[tid] = 0;
  __syncthreads();
  for (int base = 0; base < chunk; base += AT_ONCE) {
    const int i = base + tid / GL;
    const int64_t sl = __shfl(slot, i & 63, 64);
    if (i >= chunk || !(runs >> i & 1)) continue;                  // the same for all lanes of a token
    const int off = (int)(sl & (PAGE - 1));
    const int64_t block = sl / PAGE * heads + head;
    const int old = off ? (int)scales[block] : 0;
    Raw8<BF16> v;
    const uint8_t* from = (const uint8_t*)x + ((t0 + i) * stride + ch) * (BF16 ? 2 : 4);
#pragma unroll
    for (int e = 0; e < (BF16 ? 1 : 2); e++) {
      const u32x4_t q = ld16(from + 16 * e);
#pragma unroll
      for (int b = 0; b < 4; b++) v.w[4 * e + b] = q[b];
    }
    auto join = [&](uint32_t a) {
#pragma unroll
      for (int o = 1; o < GL; o <<= 1) {
        const uint32_t b = (uint32_t)__shfl_xor((int)a, o, 64);
        a = a > b ? a : b;
      }
      return a;
    };
    uint32_t m = v.magnitude(0);
    if constexpr (BF16) m = (m & 0xFFFFu) > (m >> 16) ? m << 16 : m & 0xFFFF0000u;
    m = join(m);
    const bool odd = m >= 0x7F800000u;        // NaN or infinity
    float f[8];
    if (odd) {
      v.widen(f);
      m = 0;
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const uint32_t a = __float_as_uint(f[e]) & 0x7FFFFFFFu;
        m = a < 0x7F800000u && a > m ? a : m;
      }
      m = join(m);
    }
    const int need = e8m0_cover(m), c = need > old ? need : old;
    u32x2_t w;
    if (!odd) {
      w = v.codes(e8m0_as_scale((uint32_t)c));
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++) f[e] = __builtin_ldexpf(f[e], 127 - c);
      w = u32x2_t{e4m3_word(f), e4m3_word(f + 4)};
    }
    uint8_t* p = codes + block * PAGE * D;
    if constexpr (!VALUES) {
      *reinterpret_cast<u32x2_t*>(p + off * D + ch) = w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++) p[(ch + e) * PAGE + off] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
    }
    if (ch == 0 && (!off || c != old)) scales[block] = (uint8_t)c;
    if (ch == 0 && off && c > old) grown[i] = c - old;
  }
  __syncthreads();
  const int shift = grown[lane];
  for (unsigned long long todo = __ballot(shift != 0); todo; todo &= todo - 1) {
    const int i = __builtin_ctzll(todo);
    const int64_t sl = __shfl(slot, i, 64);
    const int by = -__shfl(shift, i, 64), off = (int)(sl & (PAGE - 1));
    uint8_t* p = codes + (sl / PAGE * heads + head) * PAGE * D;
    if constexpr (!VALUES) {
      for (int j = tid; j < off * D / 4; j += KV_THREADS) {
        uint32_t* w = reinterpret_cast<uint32_t*>(p) + j;
        *w = e4m3_word_shifted(*w, by);
      }
    } else {
      const int words = (off + 3) >> 2;
      for (int j = tid; j < D * words; j += KV_THREADS) {
        const int k = j % words;
        uint32_t* w = reinterpret_cast<uint32_t*>(p + j / words * PAGE) + k;
        const uint32_t had = *w, keep = off - 4 * k < 4 ? ~0u << (8 * (off - 4 * k)) : 0u;   // bytes from `off` on
        *w = (had & keep) | (e4m3_word_shifted(had, by) & ~keep);
      }
    }
  }
}

// Workgroup (x, head, keys or values) writes the runs that begin in tokens
// [x * chunk, (x + 1) * chunk), chunk <= 64: one token where that gives no more
// than 2048 workgroups, else up to a page, since a workgroup without a run of
// its own costs its start (8192 tokens: 14.7 us at 2048, 17.4 at 4096, 22 at 8192).
template <bool BF16, int D, int PAGE>
__global__ __launch_bounds__(KV_THREADS) void k_kv_append(
    const void* __restrict__ k, int64_t k_stride, const void* __restrict__ v, int64_t v_stride,
    const int64_t* __restrict__ slots, int64_t tokens, int chunk, int64_t num_pages, uint8_t* __restrict__ k_codes,
    uint8_t* __restrict__ k_scales, uint8_t* __restrict__ v_codes, uint8_t* __restrict__ v_scales) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[D * (PAGE + 4)];
  __shared__ uint32_t red[KV_THREADS / 64];
  __shared__ int grown[64];
  const int lane = threadIdx.x & 63, head = blockIdx.y, heads = gridDim.y;
  const int64_t limit = num_pages * PAGE;
  const int64_t t0 = (int64_t)blockIdx.x * chunk;
  // every wave looks at the chunk's slots and those that a run of them may reach
  auto slot_of = [&](int64_t t) { return t < tokens ? slots[t] : (int64_t)-1; };
  const int64_t s0 = slot_of(t0 + lane), s1 = slot_of(t0 + 64 + lane);
  const int64_t before0 = t0 ? slots[t0 - 1] : -1;
  int64_t before = __shfl_up(s0, 1, 64);
  before = lane ? before : before0;
  const bool valid = s0 >= 0 && s0 < limit;
  const bool begins = valid && lane < chunk && !((s0 & (PAGE - 1)) && before == s0 - 1);
  unsigned long long runs = __ballot(begins);
  // follows: the token extends the run of the one before it
  const int64_t last0 = __shfl(s0, 63, 64), up1 = __shfl_up(s1, 1, 64), before1 = lane ? up1 : last0;
  const unsigned long long on0 = __ballot((s0 & (PAGE - 1)) && before == s0 - 1);
  const unsigned long long on1 = __ballot((s1 & (PAGE - 1)) && before1 == s1 - 1);
  const int64_t col = (int64_t)head * D * (BF16 ? 2 : 4);
  // no token of the chunk, nor the one behind it, goes on in another's run
  const unsigned long long behind = chunk < 64 ? on0 & ((2ull << chunk) - 2) : (on0 & ~1ull) | (on1 & 1);
  if (!behind) {
    if (blockIdx.z == 0)
      append_ones<BF16, false, D, PAGE>((const uint8_t*)k + col, k_stride, t0, chunk, runs, s0, heads, head, k_codes,
                                        k_scales, grown);
    else
      append_ones<BF16, true, D, PAGE>((const uint8_t*)v + col, v_stride, t0, chunk, runs, s0, heads, head, v_codes,
                                       v_scales, grown);
    return;
  }
  unsigned long long on2 = 0;
  if constexpr (PAGE == 128) {
    const int64_t s2 = slot_of(t0 + 128 + lane);
    const int64_t last1 = __shfl(s1, 63, 64), up2 = __shfl_up(s2, 1, 64), before2 = lane ? up2 : last1;
    on2 = __ballot((s2 & (PAGE - 1)) && before2 == s2 - 1 && lane < 63);
  }
  while (runs) {
    const int i = __builtin_ctzll(runs);
    runs &= runs - 1;
    const int64_t t = t0 + i, slot = __shfl(s0, i, 64);
    // tokens that follow i without a gap: up to PAGE - 1 of them
    const unsigned long long a = i < 63 ? ~(on0 >> (i + 1)) : ~0ull;
    int n = 1 + (a ? __builtin_ctzll(a) : 64);
    if (n >= 64 - i) {
      n = 64 - i + (~on1 ? __builtin_ctzll(~on1) : 64);
      if (PAGE == 128 && n == 128 - i) n += __builtin_ctzll(~on2);   // a page is at most 128 tokens: ~on2 != 0
    }
    const int off = (int)(slot & (PAGE - 1));
    const int64_t block = slot / PAGE * heads + head;
    if (blockIdx.z == 0)
      append_run<BF16, false, D, PAGE>((const uint8_t*)k + col, k_stride, t, n, off, k_codes + block * PAGE * D,
                                       k_scales + block, lds, red);
    else
      append_run<BF16, true, D, PAGE>((const uint8_t*)v + col, v_stride, t, n, off, v_codes + block * PAGE * D,
                                      v_scales + block, lds, red);
  }
}

// ---------------------------------------------------------------------------
// Attention
// ---------------------------------------------------------------------------
// Both attention kernels compute the transposed products S^T = K q^T and
// O^T = V^T P^T on bf16 matrix cores, the E4M3 bytes converted with their
// page's scale on the way (exact).  A row of the query tile is then a column
// of both products, so that a lane holds scores, probabilities, statistics and
// sums of one row only: the softmax needs no more than one or two exchanges
// between lanes per tile, and the probabilities that a lane computed are
// the very operand elements it has to supply to the second product.  The
// order of the tokens along the second product's inner axis is free as long
// as V^T follows it, so it is chosen such that a lane's probabilities belong to
// 16 consecutive tokens: one page, one scale, and one 16-byte load per
// channel of V^T.
//
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
struct KvChain {
  int32_t rows, query0, head0;                // 0 rows: none
  int32_t first, last;                        // waves that share the row tile
  int32_t first_joined, last_joined;          // whether the workgroups of those joined their waves
};
struct KvShare {
  int groups, rows;                           // workgroups per head (0: one a row tile), rows of a slot
  int log_joins;                              // log2 of the workgroups of k_kv_join for a row tile
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

__device__ __forceinline__ int64_t wave_sum(int64_t v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}
__device__ __forceinline__ int lane32(int v, int src) { return __builtin_amdgcn_readlane(v, src); }
__device__ __forceinline__ int64_t lane64(int64_t v, int src) {
  return (int64_t)(((uint64_t)(uint32_t)lane32((int)(v >> 32), src) << 32) | (uint32_t)lane32((int)v, src));
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
  total = lane64(wave_sum(total), 0);
  int64_t share = (total + part.splits - 1) / part.splits;
  share = share < part.min_tiles ? part.min_tiles : share;
  const int per = share > 0x7FFFFFFF ? 0x7FFFFFFF : (int)share;
  int64_t items = 0, slots = 0;
  bool found = false;
  for (int64_t base = 0; base < A.batch; base += 64) {
    if (A.batch > 64) q.load<R, WHICH>(A, base + lane);
    const int rounded = (int)((2 * (int64_t)q.tiles + per) / (2 * (int64_t)per)), splits = rounded > 1 ? rounded : 1;
    const int64_t own = (int64_t)q.row_tiles * splits, part_own = splits > 1 ? own : 0;
    const int64_t end = items + wave_scan(own, lane), part_end = slots + wave_scan(part_own, lane);
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
      : first((int)((uint32_t)r0 / (uint32_t)A.group)), head0((int)((uint32_t)r0 % (uint32_t)A.group)),
        pos0(len - n + first) {}
  __device__ __forceinline__ int query(const KvArgs& A, int i) const { return (int)((uint32_t)(head0 + i) / (uint32_t)A.group); }
  __device__ __forceinline__ int head(const KvArgs& A, int i) const { return (int)((uint32_t)(head0 + i) % (uint32_t)A.group); }
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

// Eight E4M3 bytes with E8M0 scale operand -> eight bf16.
__device__ __forceinline__ bf16x8_t e4m3_bf16x8(uint32_t a, uint32_t b, float scale) {
  const u32x4_t w = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, true)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, true))};
  return __builtin_bit_cast(bf16x8_t, w);
}

// Keeps the bytes of tokens [lo, hi) of a 16-byte piece that begins at token j.
__device__ __forceinline__ u32x4_t keep_tokens(u32x4_t v, int j, int lo, int hi) {
  const int a = lo > j ? (lo - j < 16 ? lo - j : 16) : 0;
  const int z = hi > j ? (hi - j < 16 ? hi - j : 16) : 0;
#pragma unroll
  for (int w = 0; w < 4; w++) {
    const int aw = a - 4 * w < 0 ? 0 : a - 4 * w > 4 ? 4 : a - 4 * w;
    const int zw = z - 4 * w < 0 ? 0 : z - 4 * w > 4 ? 4 : z - 4 * w;
    v[w] &= (uint32_t)((1ull << (8 * zw)) - 1) & ~(uint32_t)((1ull << (8 * aw)) - 1);
  }
  return v;
}

// Values that are not finite: the NaN code, and what a scale above 2^119 takes
// past bf16's range.  In a tile whose rows see different tokens the product
// would carry them to every row (0 * NaN), so such bytes are taken out there, and
// `add_not_finite` gives them to the rows that see them once the sums are done.
// Where there are none this costs up to 2 % (chunks 543 -> 550 us, window step
// 13.0 -> 13.2 us, drafted tokens the same): the bytes are looked at in those
// tiles only.
// The least magnitude that is not finite with E8M0 code c:
__device__ __forceinline__ uint32_t not_finite_from(uint32_t c) { return c > 246 ? (262 - c) * 8 : 0x7F; }
// What takes the magnitudes from there on, and no other, to bit 7 of their byte.
__device__ __forceinline__ uint32_t not_finite_add(uint32_t c) { return (0x80u - not_finite_from(c)) * 0x01010101u; }
// 16 bytes without those that are not finite; bit 7 of some byte of `found` is set if there were any.
__device__ __forceinline__ u32x4_t take_not_finite(u32x4_t v, uint32_t add, uint32_t& found) {
#pragma unroll
  for (int w = 0; w < 4; w++) {
    const uint32_t t = (v[w] & 0x7F7F7F7Fu) + add;
    found |= t;
    v[w] &= ~__builtin_amdgcn_perm(t, t << 8, 0x0B090A08u);    // bit 7 of each byte of t all over it
  }
  return v;
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
// What was taken out of tiles [t0, t1) in channels ch .. ch + 3 and a row at `pos`
// sees, added to the row's results as they were stored: sums or, if null, outputs.
// Rare, so done afterwards in memory: the loops' registers have no room for it.
template <typename TAB>
__device__ __forceinline__ void add_not_finite(const KvArgs& A, TAB tab, int kvh, int head_dim, int t0, int t1, KvAlike alike,
                                               int pos, int ch, float* sums, uint16_t* outs) {
  const int rlo = kv_lowest(pos, A.window), last = t1 * TILE - 1 < pos ? t1 * TILE - 1 : pos;
  float add[4] = {0, 0, 0, 0};
#pragma unroll 1
  for (int j = t0 * TILE > rlo ? t0 * TILE : rlo; j <= last; j++) {      // below kv_len, as pos is
    if (alike(j & ~15)) {
      j |= 15;
      continue;
    }
    const int id = tab[j >> A.log_page];
    if (id < 0 || id >= A.num_pages) continue;
    const int64_t block = (int64_t)id * A.kv_heads + kvh;
    const uint32_t least = not_finite_from(A.v_scales[block]);
    const uint8_t* p = A.v_codes + (((block * head_dim + ch) << A.log_page) + (j & ((1 << A.log_page) - 1)));
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const uint32_t v = p[e << A.log_page], mag = v & 0x7Fu;
      if (mag >= least) add[e] += mag == 0x7Fu ? __builtin_nanf("") : v & 0x80u ? -INFINITY : INFINITY;
    }
  }
#pragma unroll
  for (int e = 0; e < 4; e++) {
    if (add[e] == 0.0f) continue;
    if (sums) sums[e] += add[e];
    else outs[e] = (uint16_t)(pack_bf16x2(bf16_lo(outs[e]) + add[e], 0.0f) & 0xFFFFu);
  }
}

// Decode: 16 or 32 rows (the query heads of a group, for one token or a few
// drafted ones) per row tile.  Bound by the bytes of K and V: they go from HBM
// straight into the registers that feed v_mfma_f32_16x16x32_bf16, the next
// tile's K loads leaving as soon as this tile's scores are done and its V loads
// after its sums, so that a wave always has 8 to 16 KB in flight.
//
// The launch fills the chip once, and the tiles of all row tiles, one after the
// other, are cut into equal shares, one a wave: no wave waits for another, long
// contexts and short ones may stand side by side, and the shares differ by
// one tile at most.  A share that begins or ends inside a row tile leaves
// partial sums, which k_kv_join puts together; a workgroup whose waves are all
// inside one row tile joins them in LDS first.  A row tile that sees nothing
// counts as one tile, so that its rows are written.  Where no request has more
// than a few tiles and the row tiles fit the chip, each gets a workgroup
// instead (`solo`): the join's launch costs more than the tiles in turn do.
//
// 8 heads of 128, 4 query heads each: 64 x 8192 tokens 187 us (5.76 TB/s, 0.92
// of a streaming read's rate); 64 x 2048-8192 tokens 106 us and 5.0 us joining.
// 32 rows of heads of 128 take 256 registers and spill 6 more (12 capped) outside
// the loop over tiles; the scalars that do not fit lie in lanes of others.
//
// Lane l = 16 g + m.  K tile a (of 4): operand row m is token
// 16 (m / 4) + 4 a + m % 4, result rows 4 g + i are then tokens 16 g + 4 a + i.
template <int D, bool CAP, int WHICH, int NR>
__global__ __launch_bounds__(KV_THREADS, 2) void k_kv_decode(const KvArgs A, const KvShare part) {
  constexpr int KP = D / 64, DT = D / 16, R = 16 * NR;
  __shared__ __attribute__((aligned(16))) float so[4][R][D + 4];
  __shared__ float sm[4][R], sl[4][R];
  __shared__ int st[4];
  const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = (int)(blockIdx.x / (unsigned)A.kv_heads), kvh = (int)(blockIdx.x % (unsigned)A.kv_heads);
  const int x = 4 * group + wave;
  const KvChain none = {};

  // all the work, in tiles or in row tiles, and this wave's share [u0, u1) of it
  const bool solo = part.groups == 0;
  auto units_of = [&](const KvRequest& r) { return solo || r.tiles <= 0 ? 1 : r.tiles; };
  KvRequest lanes;
  int64_t total = 0;
  for (int64_t base = 0; base < A.batch; base += 64) {
    lanes.load<R, WHICH>(A, base + lane);
    total += (int64_t)units_of(lanes) * lanes.row_tiles;
  }
  total = lane64(wave_sum(total), 0);
  const int64_t shares = solo ? 4 * total : total < 4 * part.groups ? total : 4 * part.groups;
  auto share_at = [&](int64_t y) { return y >= shares ? total : solo ? y / 4 : y * total / shares; };
  const int64_t u0 = share_at(x), u1 = share_at(x + 1), g0 = share_at(4 * group), g1 = share_at(4 * group + 4);
  if (g0 >= g1) {                             // an idle workgroup
    if (!solo && kvh == 0 && lane == 0) part.chain[x] = none;
    return;
  }
  // the request that holds unit u, and its first unit
  KvRequest q = {};
  int request = 0;
  int64_t begin = 0;
  auto find = [&](int64_t u) {
    int64_t before = 0;
    for (int64_t base = 0; base < A.batch; base += 64) {
      if (A.batch > 64) lanes.load<R, WHICH>(A, base + lane);
      const int64_t own = (int64_t)units_of(lanes) * lanes.row_tiles;
      const int64_t end = before + wave_scan(own, lane);
      const unsigned long long at = __ballot(end > u);
      if (at) {
        const int src = __builtin_ctzll(at);
        q = lanes.from(src);
        request = (int)base + src;
        begin = lane64(end - own, src);
        return;
      }
      before = lane64(end, 63);
    }
  };
  find(g0);
  auto units = [&]() { return units_of(q); };
  int rt = (int)((g0 - begin) / units());     // row tiles in order of their units, the last rows first
  const bool joined = g1 <= begin + (int64_t)(rt + 1) * units();   // always so if solo
  if (!joined) {
    if (u0 >= u1) {
      if (kvh == 0 && lane == 0) part.chain[x] = none;
      return;
    }
    find(u0);
    rt = (int)((u0 - begin) / units());
  }
  if (q.row_tiles == 0) {                     // lengths that changed under the kernel
    if (!solo && kvh == 0 && lane == 0) part.chain[x] = none;
    return;
  }

  const int last_col = (int)A.max_blocks - 1;
  const uint32_t head_bytes = (uint32_t)D << A.log_page, page_bytes = head_bytes * A.kv_heads;
  const int in_page = (1 << A.log_page) - 1;
  const uint8_t* kbase = A.k_codes + (int64_t)kvh * head_bytes;
  const uint8_t* vbase = A.v_codes + (int64_t)kvh * head_bytes;
  const uint8_t *ksb = A.k_scales + kvh, *vsb = A.v_scales + kvh;
  const KvScore<CAP> sc(A);
  KvChain chain = none;

  for (int64_t u = u0;;) {
    const int64_t row_begin = begin + (int64_t)rt * units(), row_end = row_begin + units();
    const int64_t stop = u1 < row_end ? u1 : row_end;
    const int step = joined ? 4 : 1;          // the waves of a joined workgroup take its tiles in turn
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
    int t = first_tile(), t1 = q.first + (solo ? q.tiles : (int)((joined ? g1 : stop) - row_begin));
    t1 = t1 > (hi + TILE - 1) / TILE ? (hi + TILE - 1) / TILE : t1;
    t += joined ? wave : 0;

    const int32_t* tab = A.table + (int64_t)request * A.max_blocks;
    u32x4_t kr[4][KP], vr[DT];
    uint32_t ksc, vsc;
    bool vok;
    int idk, idv;                             // page ids of the next tile to load
    auto load_ids = [&](int t) {
      const int ck = (t * TILE + 16 * (m >> 2)) >> A.log_page, cv = (t * TILE + 16 * g) >> A.log_page;
      idk = tab[ck < last_col ? ck : last_col];
      idv = tab[cv < last_col ? cv : last_col];
    };
    auto load_k = [&](int t) {
      const uint32_t id = idk >= 0 && idk < A.num_pages ? idk : 0;
      ksc = ksb[(uint64_t)id * (uint32_t)A.kv_heads];
      const uint8_t* p = kbase + ((uint64_t)id * page_bytes + (((t * TILE + 16 * (m >> 2)) & in_page) + (m & 3)) * D + 16 * g);
#pragma unroll
      for (int a = 0; a < 4; a++)
#pragma unroll
        for (int h = 0; h < KP; h++) kr[a][h] = ld16(p + 4 * a * D + 64 * h);
    };
    auto load_v = [&](int t) {
      vok = idv >= 0 && idv < A.num_pages;
      const uint32_t id = vok ? idv : 0;
      vsc = vsb[(uint64_t)id * (uint32_t)A.kv_heads];
      const uint8_t* p = vbase + ((uint64_t)id * page_bytes + (m << A.log_page) + ((t * TILE + 16 * g) & in_page));
#pragma unroll
      for (int d = 0; d < DT; d++) vr[d] = ld16(p + ((16 * d) << A.log_page));
    };
    uint32_t taken = 0;                       // values of this lane's that are not finite
    if (t < t1) {
      load_ids(t);
      load_k(t);
      load_v(t);
      if (t + step < t1) load_ids(t + step);
    }

    // query fragments: columns m of q^T; row m's limits
    bf16x8_t qf[NR][KP][2];
    int pos[NR], rlo[NR];
#pragma unroll
    for (int c = 0; c < NR; c++) {
      const bool live = 16 * c + m < n_rows;
      const int i = live ? 16 * c + m : 0, query = rows.query(A, i);
      pos[c] = rows.pos0 + query;
      rlo[c] = kv_lowest(pos[c], A.window);
      const uint16_t* qp = A.q + (int64_t)(q.q0 + rows.first + query) * A.q_stride + (kvh * A.group + rows.head(A, i)) * D;
#pragma unroll
      for (int p = 0; p < KP; p++)
#pragma unroll
        for (int h = 0; h < 2; h++) {
          u32x4_t w = ld16(qp + 64 * p + 16 * g + 8 * h);
          if (!live) w = u32x4_t{0, 0, 0, 0};
          qf[c][p][h] = __builtin_bit_cast(bf16x8_t, w);
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
      const float ks = e8m0_as_scale(ksc);
#pragma unroll
      for (int a = 0; a < 4; a++) {
#pragma unroll
        for (int c = 0; c < NR; c++) s[c][a] = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int p = 0; p < KP; p++) {
          const u32x4_t w = kr[a][p];
          const bf16x8_t k0 = e4m3_bf16x8(w[0], w[1], ks), k1 = e4m3_bf16x8(w[2], w[3], ks);
#pragma unroll
          for (int c = 0; c < NR; c++) {
            s[c][a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, qf[c][p][0], s[c][a], 0, 0, 0);
            s[c][a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, qf[c][p][1], s[c][a], 0, 0, 0);
          }
        }
      }
      if (more) load_k(t + step);
      float vs = e8m0_as_scale(vsc);
      const bool differs = t * TILE + TILE - 1 > rows.pos0 || t * TILE < lo_max, edge = differs || __any(!vok);
      if (edge) {                             // bytes of V that no row may see
        const int a = vok ? lo : 0, z = vok ? hi : 0;
        if (j0 + 16 <= a || j0 >= z) vs = 1.0f;
        const uint32_t add = hi - 1 > rows.pos0 && differs ? not_finite_add(vsc) : 0;   // 0 takes nothing
#pragma unroll
        for (int d = 0; d < DT; d++) vr[d] = keep_tokens(vr[d], j0, a, z);
        if (__builtin_expect(add != 0, 0))    // by itself, so that V^T keeps its registers
#pragma unroll
          for (int d = 0; d < DT; d++) vr[d] = take_not_finite(vr[d], add, taken);
      }
      bf16x8_t p0[NR], p1[NR];
#pragma unroll
      for (int c = 0; c < NR; c++) {
        if constexpr (CAP) {
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; i++) v[i] = s[c][i >> 2][i & 3];
          sc.cap(v, edge);
#pragma unroll
          for (int i = 0; i < 16; i++) s[c][i >> 2][i & 3] = v[i];
        }
        if (edge) {                           // tokens outside the row's limits
          const int z = vok ? pos[c] - j0 : -1, b = rlo[c] - j0;
#pragma unroll
          for (int a = 0; a < 4; a++)
#pragma unroll
            for (int i = 0; i < 4; i++) s[c][a][i] = 4 * a + i <= z && 4 * a + i >= b ? s[c][a][i] : -INFINITY;
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
        uint32_t pw[8];
#pragma unroll
        for (int a = 0; a < 4; a++) {
          float p[4];
#pragma unroll
          for (int i = 0; i < 4; i++) {
            p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[c][a][i], sc.mul, off));
            l[c] += p[i];
          }
          // bf16 for the matrix cores: half a step of 2^-8 per probability, the sum l keeps fp32
          pw[2 * a] = pack_bf16x2(p[0], p[1]);
          pw[2 * a + 1] = pack_bf16x2(p[2], p[3]);
        }
        p0[c] = __builtin_bit_cast(bf16x8_t, (u32x4_t{pw[0], pw[1], pw[2], pw[3]}));
        p1[c] = __builtin_bit_cast(bf16x8_t, (u32x4_t{pw[4], pw[5], pw[6], pw[7]}));
      }
#pragma unroll
      for (int d = 0; d < DT; d++) {
        const bf16x8_t v0 = e4m3_bf16x8(vr[d][0], vr[d][1], vs), v1 = e4m3_bf16x8(vr[d][2], vr[d][3], vs);
#pragma unroll
        for (int c = 0; c < NR; c++) {
          o[c][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, p0[c], o[c][d], 0, 0, 0);
          o[c][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, p1[c], o[c][d], 0, 0, 0);
        }
      }
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
    const bool whole = from == row_begin && to == row_end;
    const int slot = 2 * (joined ? 4 * group : x) + (from == row_begin ? 0 : 1);
    if (from == row_begin && !whole && (!joined || wave == 0)) {
      // the last wave: the one whose share holds unit row_end - 1
      const int64_t last = (row_end * shares - 1) / total;
      chain = KvChain{n_rows, q.q0 + rows.first, rows.head0, joined ? 4 * group : x, (int)last, joined,
                      share_at((last | 3) + 1) <= row_end};
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
    auto put_not_finite = [&](int row, int ch) {
      const int query = rows.query(A, row);
      const int64_t at = ((int64_t)slot * A.kv_heads + kvh) * part.rows + row;
      const int64_t orow = (int64_t)(q.q0 + rows.first + query) * A.q_heads + kvh * A.group + rows.head(A, row);
      add_not_finite(A, tab, kvh, D, first_tile(), t1, KvAlike(rows.pos0, hi - 1, A.window), rows.pos0 + query, ch,
                     whole ? nullptr : part.sums + at * D + ch, A.out + orow * D + ch);
    };
    if (!joined) {
#pragma unroll
      for (int c = 0; c < NR; c++)
        if (16 * c + m < n_rows) {
#pragma unroll
          for (int d = 0; d < DT; d++) put(16 * c + m, 16 * d + 4 * g, o[c][d], mx[c], l[c]);
        }
      if (__builtin_expect(__any((taken & 0x80808080u) != 0), 0)) {
#pragma unroll 1
        for (int i = 0; i < NR * DT; i++)
          if (16 * (i / DT) + m < n_rows) put_not_finite(16 * (i / DT) + m, 16 * (i % DT) + 4 * g);
      }
      u = stop;
      if (u >= u1) break;
      if (++rt == q.row_tiles) {              // on to the next request that has rows
        begin = row_end;
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
      const bool wave_taken = __any((taken & 0x80808080u) != 0);
      if (lane == 0) st[wave] = wave_taken;
#pragma unroll
      for (int d = 0; d < DT; d++) *reinterpret_cast<f32x4_t*>(&so[wave][16 * c + m][16 * d + 4 * g]) = o[c][d];
    }
    __syncthreads();
    const bool any_taken = (st[0] | st[1] | st[2] | st[3]) != 0;
    for (int i = tid; i < n_rows * (D / 4); i += KV_THREADS) {
      const int row = i / (D / 4), ch = i % (D / 4) * 4;
      float top = sm[0][row], sum = 0.0f;
#pragma unroll
      for (int w = 1; w < 4; w++) top = __builtin_fmaxf(top, sm[w][row]);
      f32x4_t acc = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < 4; w++) {
        const float f = sm[w][row] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(sm[w][row] - top);
        sum = __builtin_fmaf(f, sl[w][row], sum);
        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(&so[w][row][ch]);
#pragma unroll
        for (int e = 0; e < 4; e++) acc[e] = __builtin_fmaf(f, v[e], acc[e]);
      }
      put(row, ch, acc, top, sum);
      if (__builtin_expect(any_taken, 0)) put_not_finite(row, ch);
    }
    break;
  }
  if (!solo && kvh == 0 && lane == 0) part.chain[x] = chain;
}

// Prompts and chunks: 128 rows per workgroup, 32 per wave.  Bound by the
// vector instructions of the softmax and the matrix cores alike, so the loop
// is arranged for the two to overlap: half a tile's scores (32 tokens) are
// multiplied while those of the half before are exponentiated.  A tile of 64 tokens is
// converted to bf16 once per workgroup, on its way from registers (loaded a
// step ahead) to LDS, where it lies in operand order (each fragment 1 KB
// contiguous, its 16-byte units permuted by an xor so that neither the writes
// nor the reads conflict), and feeds v_mfma_f32_32x32x16_bf16.
//
// Lane l = 32 h + m.  Within a 32-token half u of the tile, operand row
// 8 (r / 4) + 4 h + r % 4 is token 32 u + 16 h + r: result register r of lane
// half h is that token.
//
// BIG: pages of 64 tokens and more, so that a tile lies in one page: its id,
// scales and addresses are scalars, which takes a fifth of the loop's vector
// instructions away (330 -> 323 us, capped 688 -> 654 us).
//
// Three prompts of 1500-4096 tokens, 32 heads of 128 on 8: 304-326 us over
// several runs (810-868 TFLOP/s; matrix cores busy 0.36 of the cycles, vector units 0.45,
// both 0.15, neither 0.34; no LDS bank conflicts).  The clock falls under the load
// (a tenth fewer cycles took 3 % off the time); at 2.4 GHz the same cycles would
// take 302 us.  Heads of 64 195 us, pages of 16 341 us (211 us), a cap of 50 371 us
// (251 us).
//
// Registers allow two waves a SIMD at heads of 128 and three at heads of 64, where
// capped scores need that said (the same three prompts: 282 us at two, 251 at three).
template <int D, bool CAP, bool BIG>
__global__ __launch_bounds__(PTHREADS, D == 64 ? 3 : 2) void k_kv_prompt(const KvArgs A, const KvPart part) {
  constexpr int KS = D / 16, DT = D / 32;     // k steps, channel tiles
  constexpr int XK = D == 128 ? 1 : 2;
  constexpr int ST = D / 64;                  // 16-byte pieces of K, and of V^T, a thread
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
  const uint32_t head_bytes = (uint32_t)D << A.log_page, page_bytes = head_bytes * A.kv_heads;
  const int in_page = (1 << A.log_page) - 1;
  const uint8_t *ksb = A.k_scales + kvh, *vsb = A.v_scales + kvh;

  // staging: K piece x is token x / KS, channels 16 (x % KS)..; V^T piece x is
  // channel x / 4, tokens 16 (x % 4)..; a thread's pieces are 256 apart, so that
  // they differ by 256 / KS tokens and by 64 channels
  const int ktok = tid / KS, vtok = 16 * (tid & 3);
  const uint8_t* kbase = A.k_codes + (int64_t)kvh * head_bytes;
  const uint8_t* vbase = A.v_codes + (int64_t)kvh * head_bytes;
  const uint32_t koff = ktok * D + 16 * (tid % KS), voff = ((tid >> 2) << A.log_page) + vtok;
  uint8_t *kdst[ST], *vdst[ST];
#pragma unroll
  for (int i = 0; i < ST; i++) {
    const int tok = ktok + PTHREADS / KS * i, k = tid % KS, u = tok >> 5, th = (tok >> 4) & 1, tr = tok & 15;
    const int row = 8 * (tr >> 2) + 4 * th + (tr & 3);
    kdst[i] = sk[0] + ((u * KS + k) * 64 + (row ^ (XK * k))) * 16;
    const int d = (tid >> 2) + 64 * i, tg = tid & 3;
    vdst[i] = sv[0] + (((d >> 5) * 4 + 2 * (tg >> 1)) * 64 + 32 * (tg & 1) + ((d & 31) ^ (2 * tg))) * 16;
  }
  constexpr int BUF = TILE * D * 2;
  u32x4_t kr[ST], vr[ST];
  uint32_t ksc[ST], vsc;
  bool vok;
  // page ids on their way: of the next K, V^T and, in score layout, the masks;
  // with BIG pages of tiles t .. t + 4
  int idk[ST], idv, idm[2], idn[2], ids[5];
  auto page_id = [&](int t, int tok) {        // past t1 the last tile again: loaded, never used
    const int c = ((t < t1 ? t : t1 - 1) * TILE + tok) >> A.log_page;
    return tab[c < last_col ? c : last_col];
  };
  auto there = [&](int id) { return id >= 0 && id < A.num_pages; };
  auto ids_k = [&](int t) {
    if constexpr (!BIG) {
#pragma unroll
      for (int i = 0; i < ST; i++) idk[i] = page_id(t, ktok + PTHREADS / KS * i);
    }
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
  auto load_k = [&](int t, int id) {
    if constexpr (BIG) {
      const uint64_t block = (uint64_t)(uint32_t)(there(id) ? id : 0);
      const uint8_t* p = kbase + (block * page_bytes + (uint32_t)((t * TILE) & in_page) * D);
      ksc[0] = ksb[block * (uint32_t)A.kv_heads];
#pragma unroll
      for (int i = 0; i < ST; i++) kr[i] = ld16(p + (koff + PTHREADS / KS * D * i));
    } else {
#pragma unroll
      for (int i = 0; i < ST; i++) {
        const uint32_t k = there(idk[i]) ? idk[i] : 0;
        ksc[i] = ksb[(uint64_t)k * (uint32_t)A.kv_heads];
        const uint32_t in = ((t * TILE + ktok + PTHREADS / KS * i) & in_page) * D + 16 * (tid % KS);
        kr[i] = ld16(kbase + ((uint64_t)k * page_bytes + in));
      }
    }
  };
  auto load_v = [&](int t, int id) {
    if constexpr (BIG) {
      vok = there(id);
      const uint64_t block = (uint64_t)(uint32_t)(vok ? id : 0);
      const uint8_t* p = vbase + (block * page_bytes + (uint32_t)((t * TILE) & in_page));
      vsc = vsb[block * (uint32_t)A.kv_heads];
#pragma unroll
      for (int i = 0; i < ST; i++) vr[i] = ld16(p + (voff + ((64u * i) << A.log_page)));
    } else {
      vok = there(idv);
      const uint32_t v = vok ? idv : 0;
      vsc = vsb[(uint64_t)v * (uint32_t)A.kv_heads];
      const uint8_t* p = vbase + ((uint64_t)v * page_bytes + ((t * TILE + vtok) & in_page) + ((tid >> 2) << A.log_page));
#pragma unroll
      for (int i = 0; i < ST; i++) vr[i] = ld16(p + ((64 * i) << A.log_page));
    }
  };
  auto store_k = [&](int at) {
#pragma unroll
    for (int i = 0; i < ST; i++) {
      const float s = e8m0_as_scale(ksc[BIG ? 0 : i]);
      *reinterpret_cast<bf16x8_t*>(kdst[i] + at) = e4m3_bf16x8(kr[i][0], kr[i][1], s);
      *reinterpret_cast<bf16x8_t*>(kdst[i] + at + 32 * 16) = e4m3_bf16x8(kr[i][2], kr[i][3], s);
    }
  };
  KvAlike alike(rows.pos0, rows.pos0 + rows.query(A, it.rows - 1), A.window);
  alike.lo = alike.lo > lo ? alike.lo : lo;   // and nothing of theirs is unseen
  alike.hi = alike.hi < hi ? alike.hi : hi;
  uint32_t taken = 0;                         // whether this lane took values out that are not finite
  auto store_v = [&](int t, int buf) {        // without the bytes that no row may see
    const int j = t * TILE + vtok;
    float s = e8m0_as_scale(vsc);
    if (!vok || !alike(j)) {
      const int a = vok ? lo : 0, z = vok ? hi : 0;
      const uint32_t add = not_finite_add(vsc);
      uint32_t found = 0;
      if (j + 16 <= a || j >= z) s = 1.0f;
#pragma unroll
      for (int i = 0; i < ST; i++) vr[i] = take_not_finite(keep_tokens(vr[i], j, a, z), add, found);
      taken |= found & 0x80808080u;
    }
#pragma unroll
    for (int i = 0; i < ST; i++) {
      *reinterpret_cast<bf16x8_t*>(vdst[i] + buf * BUF) = e4m3_bf16x8(vr[i][0], vr[i][1], s);
      *reinterpret_cast<bf16x8_t*>(vdst[i] + buf * BUF + 64 * 16) = e4m3_bf16x8(vr[i][2], vr[i][3], s);
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
  constexpr int HOLD = 4;                     // fragments read ahead of their use
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
      pw[i] = pack_bf16x2(a, b);              // half a step of 2^-8 per probability, l keeps fp32
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
  bool any_taken = false;
  if (t0 < t1 && !(alike(t0 * TILE) && alike(t1 * TILE - 16))) {
    uint32_t* flags = reinterpret_cast<uint32_t*>(sk[0] + k2);     // free in the last step
    const bool wave_taken = __any(taken != 0);
    if (lane == 0) flags[wave] = wave_taken;
    tile_barrier();
    any_taken = (flags[0] | flags[1] | flags[2] | flags[3]) != 0;
  }
  l += __shfl_xor(l, 32, 64);
  if (!live) return;
  if (split) {
    const int64_t at = (it.slot * A.kv_heads + kvh) * PROWS + wrow + m;
#pragma unroll
    for (int d = 0; d < DT; d++)
#pragma unroll
      for (int i = 0; i < 4; i++)
        *reinterpret_cast<f32x4_t*>(part.sums + at * D + 32 * d + 8 * i + 4 * h) =
            f32x4_t{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
    if (h == 0) {
      part.stats[2 * at] = mx;
      part.stats[2 * at + 1] = l;
    }
  }
  const int64_t orow = (int64_t)(it.q0 + rows.first + query) * A.q_heads + head;
  if (!split) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int d = 0; d < DT; d++)
#pragma unroll
      for (int i = 0; i < 4; i++)
        *reinterpret_cast<u32x2_t*>(A.out + orow * D + 32 * d + 8 * i + 4 * h) =
            u32x2_t{pack_bf16x2(o[d][4 * i] * inv, o[d][4 * i + 1] * inv),
                    pack_bf16x2(o[d][4 * i + 2] * inv, o[d][4 * i + 3] * inv)};
    if (A.lse && h == 0) A.lse[orow] = l == 0.0f ? -INFINITY : (mx + __builtin_log2f(l)) * LN2;
  }
  if (__builtin_expect(any_taken, 0)) {
    float* sums = split ? part.sums + ((it.slot * A.kv_heads + kvh) * PROWS + wrow + m) * D : nullptr;
#pragma unroll 1
    for (int ch = 4 * h; ch < D; ch += 8)
      add_not_finite(A, tab, kvh, D, t0, t1, alike, pos, ch, split ? sums + ch : nullptr, A.out + orow * D + ch);
  }
}

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
  const int64_t decode = 4 * (int64_t)dec.groups << dec.log_joins;
  if (x < decode) {
    const KvChain c = dec.chain[x >> dec.log_joins];
    const int some = 16 * NR >> dec.log_joins, row0 = (int)(x & ((1 << dec.log_joins) - 1)) * some;
    if (c.rows == 0) return;
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

template <bool BF16, int D>
void launch_append(int page, dim3 grid, hipStream_t s, const void* k, int64_t ks, const void* v, int64_t vs,
                   const int64_t* slots, int64_t tokens, int chunk, int64_t num_pages, uint8_t* kc, uint8_t* ksc,
                   uint8_t* vc, uint8_t* vsc) {
#define WQ_APPEND(PAGE) \
  k_kv_append<BF16, D, PAGE><<<grid, KV_THREADS, 0, s>>>(k, ks, v, vs, slots, tokens, chunk, num_pages, kc, ksc, vc, vsc)
  if (page == 16) WQ_APPEND(16);
  else if (page == 32) WQ_APPEND(32);
  else if (page == 64) WQ_APPEND(64);
  else WQ_APPEND(128);
#undef WQ_APPEND
}

}  // namespace

extern "C" {

wq_status wq_kv_blocks(const int32_t* ctx_lens, const int32_t* new_lens, int64_t batch, const int32_t* free_pages,
                       int64_t num_free, const int32_t* cursor, int32_t page, int32_t* block_table, int64_t max_blocks,
                       int64_t tokens, int64_t* slots, int32_t* positions, int32_t* cu_new, int32_t* kv_lens,
                       int32_t* state, void* stream) {
  if (log2_page(page) < 0) return WQ_EUNSUPPORTED;
  if (batch < 0 || batch > 0x7FFFFFFF || num_free < 0 || num_free > 0x7FFFFFFF || tokens < 0 || tokens > 0x7FFFFFFF ||
      max_blocks < 1 || max_blocks > 0x7FFFFFFF || !wq_numel_ok(batch ? batch : 1, max_blocks))
    return WQ_EINVAL;
  if (!cu_new || !state || (batch > 0 && (!ctx_lens || !new_lens || !block_table || !kv_lens)) ||
      (num_free > 0 && !free_pages) || (tokens > 0 && (!slots || !positions)))
    return WQ_EINVAL;
  // the outputs, and behind them the inputs; what has no elements is nowhere
  const void* at[] = {cu_new, state, batch ? kv_lens : nullptr, batch ? block_table : nullptr,
                      tokens ? slots : nullptr, tokens ? positions : nullptr, batch ? ctx_lens : nullptr,
                      batch ? new_lens : nullptr, num_free ? free_pages : nullptr, cursor};
  for (int i = 0; i < 6; i++)
    for (int j = i + 1; j < 10; j++)
      if (at[i] && at[i] == at[j]) return WQ_EINVAL;
  const int64_t groups = (tokens + KV_THREADS - 1) / KV_THREADS;
  k_kv_blocks<<<(unsigned)(groups > 1 ? groups : 1), KV_THREADS, 0, (hipStream_t)stream>>>(
      ctx_lens, new_lens, batch, free_pages, num_free, cursor, log2_page(page), block_table, max_blocks, tokens, slots,
      positions, cu_new, kv_lens, state);
  return wq_launch_status();
}

wq_status wq_kv_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, int x_dtype,
                       const int64_t* slots, int64_t tokens, int32_t heads, int32_t head_dim, int32_t page,
                       int64_t num_pages, uint8_t* k_codes, uint8_t* k_scales, uint8_t* v_codes, uint8_t* v_scales,
                       void* stream) {
  if ((x_dtype != WQ_F32 && x_dtype != WQ_BF16) || (head_dim != 64 && head_dim != 128) || log2_page(page) < 0)
    return WQ_EUNSUPPORTED;
  if (tokens < 0 || tokens > 0x7FFFFFFF || heads < 1 || heads > 65535 || num_pages < 1) return WQ_EINVAL;
  if (!k_codes || !k_scales || !v_codes || !v_scales || (tokens > 0 && (!k || !v || !slots))) return WQ_EINVAL;
  const int64_t row = (int64_t)heads * head_dim;
  if (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8 || k_stride > (int64_t(1) << 40) ||
      v_stride > (int64_t(1) << 40) || !wq_numel_ok(num_pages, row * page) || !wq_numel_ok(tokens ? tokens : 1, row))
    return WQ_EINVAL;
  if (!wq_aligned(k) || !wq_aligned(v) || !wq_aligned(k_codes) || !wq_aligned(v_codes)) return WQ_EALIGN;
  if (tokens == 0) return WQ_OK;
  int chunk = 1;
  while (chunk < 64 && chunk < page && (tokens + chunk - 1) / chunk * heads * 2 > 2048) chunk *= 2;
  const dim3 grid((unsigned)((tokens + chunk - 1) / chunk), (unsigned)heads, 2);
  hipStream_t s = (hipStream_t)stream;
  const bool bf = x_dtype == WQ_BF16;
  if (bf && head_dim == 128)
    launch_append<true, 128>(page, grid, s, k, k_stride, v, v_stride, slots, tokens, chunk, num_pages, k_codes,
                             k_scales, v_codes, v_scales);
  else if (bf)
    launch_append<true, 64>(page, grid, s, k, k_stride, v, v_stride, slots, tokens, chunk, num_pages, k_codes,
                            k_scales, v_codes, v_scales);
  else if (head_dim == 128)
    launch_append<false, 128>(page, grid, s, k, k_stride, v, v_stride, slots, tokens, chunk, num_pages, k_codes,
                              k_scales, v_codes, v_scales);
  else
    launch_append<false, 64>(page, grid, s, k, k_stride, v, v_stride, slots, tokens, chunk, num_pages, k_codes,
                             k_scales, v_codes, v_scales);
  return wq_launch_status();
}

}  // extern "C"

namespace {

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

template <int D, bool CAP>
void launch_attention(const KvArgs& A, const KvPlan& p, const KvShare& dec, const KvPart& pro, hipStream_t s) {
  const unsigned h = (unsigned)A.kv_heads, groups = (unsigned)p.groups * h;
  if (p.prompt) {
    const unsigned items = (unsigned)p.pro_items * h;
    if (A.log_page >= 6) k_kv_prompt<D, CAP, true><<<items, PTHREADS, 0, s>>>(A, pro);
    else k_kv_prompt<D, CAP, false><<<items, PTHREADS, 0, s>>>(A, pro);
    k_kv_decode<D, CAP, REQ_SHORT, 2><<<groups, KV_THREADS, 0, s>>>(A, dec);
  } else if (p.nr == 2) {
    k_kv_decode<D, CAP, REQ_ALL, 2><<<groups, KV_THREADS, 0, s>>>(A, dec);
  } else {
    k_kv_decode<D, CAP, REQ_ALL, 1><<<groups, KV_THREADS, 0, s>>>(A, dec);
  }
  if (p.solo) return;
  const unsigned joins = (4 * groups << p.log_joins) + (unsigned)(p.pro_slots * (PROWS / 16)) * h;
  if (p.nr == 2) k_kv_join<D, 2><<<joins, KV_THREADS, 0, s>>>(A, dec, pro);
  else k_kv_join<D, 1><<<joins, KV_THREADS, 0, s>>>(A, dec, pro);
}

}  // namespace

extern "C" {

size_t wq_kv_attention_workspace_size(int64_t batch, int64_t tokens, int64_t max_q, int32_t q_heads, int32_t kv_heads,
                                      int32_t head_dim, int32_t page, int64_t max_blocks, int64_t window) {
  if (window < 0 || (head_dim != 64 && head_dim != 128) || log2_page(page) < 0 ||
      !kv_sizes_ok(batch, tokens, max_q, q_heads, kv_heads, page, max_blocks))
    return 0;
  return batch && tokens ? kv_plan(batch, tokens, max_q, q_heads, kv_heads, head_dim, page, max_blocks, window).bytes : 0;
}

wq_status wq_kv_attention(const void* q_bf16, int64_t q_stride, const int32_t* cu_q, const int32_t* kv_lens,
                          int64_t batch, int64_t tokens, int64_t max_q, int32_t q_heads, int32_t kv_heads,
                          int32_t head_dim, const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes,
                          const uint8_t* v_scales, int32_t page, int64_t num_pages, const int32_t* block_table,
                          int64_t max_blocks, float sm_scale, float softcap, int64_t window, uint16_t* out,
                          float* lse, void* workspace, size_t ws_bytes, void* stream) {
  if ((head_dim != 64 && head_dim != 128) || log2_page(page) < 0) return WQ_EUNSUPPORTED;
  if (!kv_sizes_ok(batch, tokens, max_q, q_heads, kv_heads, page, max_blocks) || num_pages < 1 || window < 0)
    return WQ_EINVAL;
  if (!(sm_scale > 0.0f) || !(sm_scale < INFINITY) || !(softcap >= 0.0f) || !(softcap < INFINITY)) return WQ_EINVAL;
  if (sm_scale > 0x1p127f) return WQ_EUNSUPPORTED;           // scores go to base 2: sm_scale * log2 e is finite
  if (softcap > 0.0f && (softcap < 0x1p-10f || softcap > 0x1p10f || !(sm_scale / softcap < 0x1p14f) || !(sm_scale / softcap > 0x1p-100f)))
    return WQ_EUNSUPPORTED;
  const int64_t row = (int64_t)q_heads * head_dim;
  if (q_stride < row || q_stride % 8 || q_stride > (int64_t(1) << 40) ||
      !wq_numel_ok(num_pages, (int64_t)kv_heads * head_dim * page) || !wq_numel_ok(tokens ? tokens : 1, row) ||
      !wq_numel_ok(batch ? batch : 1, max_blocks))
    return WQ_EINVAL;
  if (!k_codes || !k_scales || !v_codes || !v_scales) return WQ_EINVAL;
  if (batch > 0 && tokens > 0 && (!q_bf16 || !cu_q || !kv_lens || !block_table || !out || out == q_bf16)) return WQ_EINVAL;
  if (!wq_aligned(q_bf16) || !wq_aligned(out) || !wq_aligned(k_codes) || !wq_aligned(v_codes) || !wq_aligned(workspace))
    return WQ_EALIGN;
  if (batch == 0 || tokens == 0) return WQ_OK;               // nothing to compute
  const KvPlan p = kv_plan(batch, tokens, max_q, q_heads, kv_heads, head_dim, page, max_blocks, window);
  if (p.bytes > 0 && (ws_bytes < p.bytes || !workspace)) return WQ_EINVAL;
  if (p.pro_items * kv_heads > 0x7FFFFFFF / PTHREADS) return WQ_EINVAL;
  const KvArgs A = {(const uint16_t*)q_bf16, q_stride, cu_q, kv_lens, batch, tokens, q_heads, kv_heads,
                    q_heads / kv_heads, (int)(window < 0x7FFFFFFF ? window : 0), k_codes, k_scales, v_codes, v_scales,
                    log2_page(page), num_pages, block_table, max_blocks, sm_scale, softcap, out, lse};
  uint8_t* ws = (uint8_t*)workspace;
  const KvShare dec = {p.solo ? 0 : p.groups, p.rows, p.log_joins, (KvChain*)ws, (float*)(ws + p.dec_sums), (float*)(ws + p.dec_stats)};
  const KvPart pro = {p.pro_splits, p.pro_slots, PRO_MIN, (int64_t*)(ws + p.pro_used), (KvRec*)(ws + p.pro_rec),
                      (float*)(ws + p.pro_sums), (float*)(ws + p.pro_stats)};
  hipStream_t s = (hipStream_t)stream;
  if (head_dim == 128) {
    if (softcap > 0.0f) launch_attention<128, true>(A, p, dec, pro, s);
    else launch_attention<128, false>(A, p, dec, pro, s);
  } else {
    if (softcap > 0.0f) launch_attention<64, true>(A, p, dec, pro, s);
    else launch_attention<64, false>(A, p, dec, pro, s);
  }
  return wq_launch_status();
}

}  // extern "C"

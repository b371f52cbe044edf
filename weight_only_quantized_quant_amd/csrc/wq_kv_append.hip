// What a step adds to a key/value cache on gfx950: new keys and values
// quantized into their slots, of the 8-bit cache (E4M3 elements, one E8M0 scale
// per page and head) or the 4-bit one (E2M1 elements, one E8M0 scale per 32
// channels of a token), with queries and keys rotated by position on the way
// if asked for.
#include <type_traits>

#include "wq_kv_common.h"

namespace {

typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

// Eight elements as they were loaded.
template <bool BF16>
struct Raw8 {
  uint32_t w[BF16 ? 4 : 8];
  __device__ __forceinline__ void load(const void* x, int64_t at) {
#pragma unroll
    for (int e = 0; e < (BF16 ? 1 : 2); e++) {
      const u32x4_t q = ld16((const uint8_t*)x + at * (BF16 ? 2 : 4) + 16 * e);
#pragma unroll
      for (int b = 0; b < 4; b++) w[4 * e + b] = q[b];
    }
  }
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

// ---------------------------------------------------------------------------
// Rotation by position
// ---------------------------------------------------------------------------
// Channels 0 .. rot - 1 of a head are rot / 2 pairs; pair i is turned by the
// angle whose cosine and sine stand at i and rot / 2 + i of the position's row:
//   a' = a cos - b sin,  b' = b cos + a sin.
// A pair is channels (i, i + rot / 2), or (2 i, 2 i + 1) if interleaved; rot is a
// multiple of 16, so that 8 aligned channels are turned whole or not at all and
// their partners are 8 aligned channels too.
struct KvRotary {
  const int32_t* positions;
  const float* cos_sin;                       // max_pos x rot
  int64_t max_pos;
  int rot, interleaved;
  const void* q;
  int64_t q_stride;
  uint16_t* q_out;
  int64_t q_out_stride;
  int q_heads;
  // a token whose position has no angles is left out
  __device__ __forceinline__ bool there(int64_t t) const {
    const int64_t p = positions[t];
    return p >= 0 && p < max_pos;
  }
};

// 8 channels of a row that begins at element `row` of x, token t, turned: keys,
// in fp64, where the products of two fp32 numbers are exact, so that
// the result, rounded once to fp32, is the nearest to what the formula gives, and
// the code that follows from it does not depend on how the sum was made (fp32
// moved 1 code in some thousand to its neighbour, and a scale now and then).
template <bool BF16>
__device__ __forceinline__ void rotate8(const void* x, int64_t row, int ch, const KvRotary& R, int64_t t, float out[8]) {
  float a[8];
  load8<BF16>(x, row + ch, a);
  if (ch >= R.rot) {
#pragma unroll
    for (int e = 0; e < 8; e++) out[e] = a[e];
    return;
  }
  const int half = R.rot >> 1;
  const float* cs = R.cos_sin + (int64_t)R.positions[t] * R.rot;
  if (R.interleaved) {
    const f32x4_t c = *reinterpret_cast<const f32x4_t*>(cs + ch / 2), s = *reinterpret_cast<const f32x4_t*>(cs + half + ch / 2);
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const double u = a[2 * e], v = a[2 * e + 1];
      out[2 * e] = (float)__builtin_elementwise_fma(u, (double)c[e], -(v * (double)s[e]));
      out[2 * e + 1] = (float)__builtin_elementwise_fma(v, (double)c[e], u * (double)s[e]);
    }
  } else {
    const bool lower = ch < half;
    const int i = lower ? ch : ch - half;
    float b[8], c[8], s[8];
    load8<BF16>(x, row + (lower ? ch + half : i), b);
    load8_f32(cs + i, c);
    load8_f32(cs + half + i, s);
#pragma unroll
    for (int e = 0; e < 8; e++)
      out[e] = (float)__builtin_elementwise_fma((double)a[e], (double)c[e], (double)b[e] * (double)(lower ? -s[e] : s[e]));
  }
}

// The queries, rounded once to bf16 (half a step of 2^-8; fp32 before that).  A
// thread takes 16 channels that are turned together (8 and their partners, or 16
// behind `rot`) of QHEADS heads of a token, whose angles it reads once, with all of
// its loads in flight.  It writes what it has read itself, so q_out may be q.
// Bound by bytes: 8192 tokens x 32 heads of 128 take 24 us alone (5.6 TB/s; 8
// channels a thread, one after the other, 40).  One head a thread: the same in
// bf16, 29 us beside the 8-bit append; four: 4.2 us instead of 3.4 for 64 tokens.
constexpr int QHEADS = 2;

template <bool BF16, int D>
__device__ __forceinline__ void rotate_queries(const KvRotary& R, int64_t tokens) {
  const int64_t sets = (R.q_heads + QHEADS - 1) / QHEADS, units = tokens * sets * (D / 16);
  const int64_t groups = (int64_t)gridDim.x * gridDim.y * (gridDim.z - 2);
  const int64_t group = ((int64_t)(blockIdx.z - 2) * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
  const int half = R.rot >> 1;
  for (int64_t u = group * KV_THREADS + threadIdx.x; u < units; u += groups * KV_THREADS) {
    const int64_t set = u / (D / 16), t = set / sets;
    const int i = (int)(u % (D / 16)), head = (int)(set - t * sets) * QHEADS;
    const int64_t pos = R.positions[t];
    if (pos < 0 || pos >= R.max_pos) continue;
    const bool turned = 16 * i < R.rot;
    const int a = turned && !R.interleaved ? 8 * i : 16 * i, b = turned && !R.interleaved ? a + half : a + 8;
    float c[8], s[8];
    Raw8<BF16> x[QHEADS][2];
    const int64_t from = t * R.q_stride + (int64_t)head * D, to = t * R.q_out_stride + (int64_t)head * D;
#pragma unroll
    for (int h = 0; h < QHEADS; h++)
      if (head + h < R.q_heads) {
        x[h][0].load(R.q, from + h * D + a);
        x[h][1].load(R.q, from + h * D + b);
      }
    if (turned) {
      load8_f32(R.cos_sin + pos * R.rot + 8 * i, c);
      load8_f32(R.cos_sin + pos * R.rot + half + 8 * i, s);
    }
#pragma unroll
    for (int h = 0; h < QHEADS; h++)
      if (head + h < R.q_heads) {
        float f[16];
        x[h][0].widen(f);
        x[h][1].widen(f + 8);
        auto turn = [&](float& v, float& w, int e) {
          const float v0 = v, w0 = w;
          v = __builtin_fmaf(v0, c[e], -(w0 * s[e]));
          w = __builtin_fmaf(w0, c[e], v0 * s[e]);
        };
        if (turned && R.interleaved) {
#pragma unroll
          for (int e = 0; e < 8; e++) turn(f[2 * e], f[2 * e + 1], e);
        } else if (turned) {
#pragma unroll
          for (int e = 0; e < 8; e++) turn(f[e], f[8 + e], e);
        }
#pragma unroll
        for (int k = 0; k < 2; k++)
          *reinterpret_cast<u32x4_t*>(R.q_out + to + h * D + (k ? b : a)) =
              u32x4_t{pack_bf16x2(f[8 * k], f[8 * k + 1]), pack_bf16x2(f[8 * k + 2], f[8 * k + 3]),
                      pack_bf16x2(f[8 * k + 4], f[8 * k + 5]), pack_bf16x2(f[8 * k + 6], f[8 * k + 7])};
      }
  }
}

// ---------------------------------------------------------------------------
// 8-bit cache
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

// One run (tokens t .. t+n-1 at offsets off .. off+n-1 of one page) of one
// head, keys or values, by the whole workgroup.  A thread takes 8 channels of
// the 4 tokens of an aligned quad of the page and keeps them in registers
// between the run's maximum and its codes: values then leave as words of 4
// tokens, which LDS turns into whole rows of the transposed page.  Bound by
// bytes, so the arithmetic is kept to one and a half instructions an element:
// maxima of bit patterns, two for bf16 at a time, and conversions that take
// the scale; a run that holds a NaN or an infinity goes the long way.  8192
// tokens of prompts, 8 heads of 128, bf16: 13.3 us a call (3.8 TB/s).
template <bool BF16IN, bool ROT, bool VALUES, int D, int PAGE>
__device__ __forceinline__ void append_run(const void* __restrict__ x, int64_t stride, int64_t t, int n, int off,
                                           uint8_t* __restrict__ codes, uint8_t* __restrict__ scale, uint8_t* lds,
                                           uint32_t* red, const KvRotary& rotary) {
  constexpr bool BF16 = BF16IN && !ROT;       // rotated elements are fp32
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
      if constexpr (ROT) {
        float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (in) rotate8<BF16IN>(x, (t + o + i - off) * stride, (p % CH) * 8, rotary, t + o + i - off, f);
#pragma unroll
        for (int e = 0; e < 8; e++) v[r][i].w[e] = __float_as_uint(f[e]);
      } else {
        const uint8_t* from = (const uint8_t*)x + ((t + (in ? o + i - off : 0)) * stride + (p % CH) * 8) * (BF16 ? 2 : 4);
#pragma unroll
        for (int e = 0; e < (BF16 ? 1 : 2); e++) {
          const u32x4_t q = in ? ld16(from + 16 * e) : u32x4_t{0, 0, 0, 0};
#pragma unroll
          for (int b = 0; b < 4; b++) v[r][i].w[4 * e + b] = q[b];
        }
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
template <bool BF16IN, bool ROT, bool VALUES, int D, int PAGE>
__device__ __forceinline__ void append_ones(const void* __restrict__ x, int64_t stride, int64_t t0, int chunk,
                                            unsigned long long runs, int64_t slot, int heads, int head,
                                            uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int* grown,
                                            const KvRotary& rotary) {
  constexpr bool BF16 = BF16IN && !ROT;
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
    if constexpr (ROT) {
      float r[8];
      rotate8<BF16IN>(x, (t0 + i) * stride, ch, rotary, t0 + i, r);
#pragma unroll
      for (int e = 0; e < 8; e++) v.w[e] = __float_as_uint(r[e]);
    } else {
      const uint8_t* from = (const uint8_t*)x + ((t0 + i) * stride + ch) * (BF16 ? 2 : 4);
#pragma unroll
      for (int e = 0; e < (BF16 ? 1 : 2); e++) {
        const u32x4_t q = ld16(from + 16 * e);
#pragma unroll
        for (int b = 0; b < 4; b++) v.w[4 * e + b] = q[b];
      }
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
// ROT: keys are rotated on the way, and workgroups z >= 2 rotate the queries.
template <bool BF16, bool ROT, int D, int PAGE>
__global__ __launch_bounds__(KV_THREADS) void k_kv_append(
    const void* __restrict__ k, int64_t k_stride, const void* __restrict__ v, int64_t v_stride,
    const int64_t* __restrict__ slots, int64_t tokens, int chunk, int64_t num_pages, uint8_t* __restrict__ k_codes,
    uint8_t* __restrict__ k_scales, uint8_t* __restrict__ v_codes, uint8_t* __restrict__ v_scales, const KvRotary rotary) {
  if constexpr (ROT) {
    if (blockIdx.z >= 2) {
      rotate_queries<BF16, D>(rotary, tokens);
      return;
    }
  }
  __shared__ __attribute__((aligned(16))) uint8_t lds[D * (PAGE + 4)];
  __shared__ uint32_t red[KV_THREADS / 64];
  __shared__ int grown[64];
  const int lane = threadIdx.x & 63, head = blockIdx.y, heads = gridDim.y;
  const int64_t limit = num_pages * PAGE;
  const int64_t t0 = (int64_t)blockIdx.x * chunk;
  // every wave looks at the chunk's slots and those that a run of them may reach
  auto slot_of = [&](int64_t t) {
    int64_t s = -1;
    if (t < tokens) {
      s = slots[t];
      if constexpr (ROT) s = rotary.there(t) ? s : -1;
    }
    return s;
  };
  const int64_t s0 = slot_of(t0 + lane), s1 = slot_of(t0 + 64 + lane);
  const int64_t before0 = t0 ? slot_of(t0 - 1) : -1;
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
      append_ones<BF16, ROT, false, D, PAGE>((const uint8_t*)k + col, k_stride, t0, chunk, runs, s0, heads, head,
                                             k_codes, k_scales, grown, rotary);
    else
      append_ones<BF16, false, true, D, PAGE>((const uint8_t*)v + col, v_stride, t0, chunk, runs, s0, heads, head,
                                              v_codes, v_scales, grown, rotary);
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
      append_run<BF16, ROT, false, D, PAGE>((const uint8_t*)k + col, k_stride, t, n, off, k_codes + block * PAGE * D,
                                            k_scales + block, lds, red, rotary);
    else
      append_run<BF16, false, true, D, PAGE>((const uint8_t*)v + col, v_stride, t, n, off, v_codes + block * PAGE * D,
                                             v_scales + block, lds, red, rotary);
  }
}

// ---------------------------------------------------------------------------
// 4-bit cache
// ---------------------------------------------------------------------------
struct Kv4Append {
  const void *k, *v;
  int64_t k_stride, v_stride;
  const int64_t* slots;
  int64_t tokens, num_pages;
  int chunk, log_page;
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
};

// Workgroup (x, head, keys or values) writes tokens [x * chunk, (x + 1) * chunk),
// chunk <= 64.  A thread takes 8 channels of a token, four threads a block of
// 32: its maximum by two exchanges, its scale, and the codes by the scaled
// conversion.  No code depends on another token, so there are no runs here and
// nothing is read back.  Keys leave as one word a thread; values go through LDS,
// which turns them into the bytes of up to four tokens that lie side by side in
// the transposed page.
// Few tokens are bound by latency (128 tokens x 8 heads of 128: 4.0 us a call), many by
// bytes and by one round of workgroups (8111 tokens x 4 heads of 64, 10.6 MB: 5.8
// us, whose floor is 2.1; 8192 tokens x 8 heads of 128 with 32 query heads turned
// beside them, 181 MB: 43.2 us, 4.2 TB/s).  Keys turned in fp64 are a small part:
// the queries alone take 24 of the 43.
template <bool BF16, bool ROT, int D>
__global__ __launch_bounds__(KV_THREADS) void k_kv4_append(const Kv4Append A, const KvRotary rotary) {
  constexpr int GL = D / 8, AT_ONCE = KV_THREADS / GL, ROWS = D / 2, LROW = 68;
  __shared__ __attribute__((aligned(16))) uint8_t lds[ROWS * LROW];
  __shared__ int list[64];
  if constexpr (ROT) {
    if (blockIdx.z >= 2) {
      rotate_queries<BF16, D>(rotary, A.tokens);
      return;
    }
  }
  const int tid = threadIdx.x, lane = tid & 63, head = blockIdx.y, heads = gridDim.y, ch = tid % GL * 8;
  const bool values = blockIdx.z == 1;
  const int64_t t0 = (int64_t)blockIdx.x * A.chunk, page = (int64_t)1 << A.log_page;
  int64_t slot = -1;                          // of token t0 + lane, in every wave
  if (lane < A.chunk && t0 + lane < A.tokens) {
    slot = A.slots[t0 + lane];
    if constexpr (ROT) slot = rotary.there(t0 + lane) ? slot : -1;
  }
  if (slot >= A.num_pages << A.log_page) slot = -1;
  const void* x = values ? A.v : A.k;
  const int64_t stride = values ? A.v_stride : A.k_stride;
  uint8_t *codes = values ? A.v_codes : A.k_codes, *scales = values ? A.v_scales : A.k_scales;
  for (int base = 0; base < A.chunk; base += AT_ONCE) {
    const int i = base + tid / GL;
    const int64_t sl = __shfl(slot, i & 63, 64);
    if (i >= A.chunk || sl < 0) continue;     // the same for all lanes of a token
    const int64_t row = (t0 + i) * stride + (int64_t)head * D;
    float f[8];
    if (ROT && !values) rotate8<BF16>(x, row, ch, rotary, t0 + i, f);
    else load8<BF16>(x, row + ch, f);
    float m = 0.0f;                           // of the finite elements: E2M1 has no infinity and no NaN
#pragma unroll
    for (int e = 0; e < 8; e++) {
      const float a = __builtin_fabsf(f[e]);
      m = a < INFINITY && a > m ? a : m;
      f[e] = f[e] != f[e] ? 0.0f : __builtin_fminf(__builtin_fmaxf(f[e], -0x1.fffffep127f), 0x1.fffffep127f);
    }
    const uint32_t c0 = e8m0_code(group_max(m, 4)), c = c0 < 252u ? c0 : 252u;
    const float sc = e8m0_as_scale(c);
    uint32_t w = e2m1_pack2<0>(0u, f[0], f[1], sc);
    w = e2m1_pack2<1>(w, f[2], f[3], sc);
    w = e2m1_pack2<2>(w, f[4], f[5], sc);
    w = e2m1_pack2<3>(w, f[6], f[7], sc);
    const int64_t block = (sl >> A.log_page) * heads + head;
    const int off = (int)(sl & (page - 1));
    if ((ch & 31) == 0) scales[((block * (D / 32) + (ch >> 5)) << A.log_page) + off] = (uint8_t)c;
    if (!values) {
      *reinterpret_cast<uint32_t*>(codes + ((block << A.log_page) + off) * ROWS + ch / 2) = w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; e++) lds[(ch / 2 + e) * LROW + i] = (uint8_t)(w >> (8 * e));
    }
  }
  if (!values) return;
  // what to write of each row: four tokens at once where they are an aligned four of a page
  const int64_t next = __shfl_down(slot, 1, 64);
  const unsigned long long on = __ballot(lane < 63 && slot >= 0 && next == slot + 1);
  const unsigned long long four = __ballot(slot >= 0 && (slot & 3) == 0 && lane < 61 && (on >> lane & 7) == 7);
  const bool covered = (four << 1 | four << 2 | four << 3) >> lane & 1;
  const unsigned long long entries = __ballot(slot >= 0 && !covered);
  if (tid < 64 && (entries >> lane & 1))
    list[__popcll(entries & ((1ull << lane) - 1))] = lane | (int)(four >> lane & 1) << 6;
  __syncthreads();
  const int n = __popcll(entries);
  for (int p = tid; p - lane < n * ROWS; p += KV_THREADS) {
    const int r = p / (n > 0 ? n : 1), what = p < n * ROWS ? list[p % n] : 0, i = what & 63;
    const int64_t sl = __shfl(slot, i, 64);
    if (p >= n * ROWS) continue;
    uint8_t* to = codes + ((((sl >> A.log_page) * heads + head) * ROWS + r) << A.log_page) + (sl & (page - 1));
    const uint8_t* from = lds + r * LROW + i;
    if (what >> 6) *reinterpret_cast<uint32_t*>(to) = from[0] | from[1] << 8 | from[2] << 16 | (uint32_t)from[3] << 24;
    else *to = from[0];
  }
}

template <bool BF16, bool ROT, int D>
void launch_append(int page, dim3 grid, hipStream_t s, const void* k, int64_t ks, const void* v, int64_t vs,
                   const int64_t* slots, int64_t tokens, int chunk, int64_t num_pages, uint8_t* kc, uint8_t* ksc,
                   uint8_t* vc, uint8_t* vsc, const KvRotary& rotary) {
#define WQ_APPEND(PAGE)                                                                                             \
  k_kv_append<BF16, ROT, D, PAGE><<<grid, KV_THREADS, 0, s>>>(k, ks, v, vs, slots, tokens, chunk, num_pages, kc, ksc, vc, \
                                                              vsc, rotary)
  if (page == 16) WQ_APPEND(16);
  else if (page == 32) WQ_APPEND(32);
  else if (page == 64) WQ_APPEND(64);
  else WQ_APPEND(128);
#undef WQ_APPEND
}

// One append, into either cache, with or without rotation.
wq_status append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, int x_dtype, const int64_t* slots,
                 int64_t tokens, int32_t heads, int32_t head_dim, int cache, int32_t page, int64_t num_pages,
                 uint8_t* k_codes, uint8_t* k_scales, uint8_t* v_codes, uint8_t* v_scales, const KvRotary* rotary,
                 void* stream) {
  if ((x_dtype != WQ_F32 && x_dtype != WQ_BF16) || (head_dim != 64 && head_dim != 128) || log2_page(page) < 0 ||
      (cache != WQ_E4M3 && cache != WQ_E2M1X2))
    return WQ_EUNSUPPORTED;
  if (tokens < 0 || tokens > 0x7FFFFFFF || heads < 1 || heads > 65535 || num_pages < 1) return WQ_EINVAL;
  if (!k_codes || !k_scales || !v_codes || !v_scales || (tokens > 0 && (!k || !v || !slots))) return WQ_EINVAL;
  const int64_t row = (int64_t)heads * head_dim;
  if (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8 || k_stride > (int64_t(1) << 40) ||
      v_stride > (int64_t(1) << 40) || !wq_numel_ok(num_pages, row * page) || !wq_numel_ok(tokens ? tokens : 1, row))
    return WQ_EINVAL;
  if (!wq_aligned(k) || !wq_aligned(v) || !wq_aligned(k_codes) || !wq_aligned(v_codes)) return WQ_EALIGN;
  if (cache == WQ_E2M1X2 && (!wq_aligned(k_scales) || !wq_aligned(v_scales))) return WQ_EALIGN;
  const bool bf = x_dtype == WQ_BF16;
  KvRotary r = {};
  if (rotary) {
    r = *rotary;
    const int64_t q_row = (int64_t)r.q_heads * head_dim;
    if (r.rot < 16 || r.rot > head_dim || r.rot % 16) return WQ_EUNSUPPORTED;
    if (r.q_heads < 0 || r.q_heads > 65535 || r.max_pos < 1 || !wq_numel_ok(r.max_pos, r.rot)) return WQ_EINVAL;
    if (tokens > 0 && (!r.positions || !r.cos_sin || (r.q_heads > 0 && (!r.q || !r.q_out)))) return WQ_EINVAL;
    if (r.q_heads > 0 && (r.q_stride < q_row || r.q_out_stride < q_row || r.q_stride % 8 || r.q_out_stride % 8 ||
                          r.q_stride > (int64_t(1) << 40) || r.q_out_stride > (int64_t(1) << 40) ||
                          !wq_numel_ok(tokens ? tokens : 1, q_row)))
      return WQ_EINVAL;
    if (r.q_heads > 0 && tokens > 0) {
      // in place row by row only
      if (r.q == r.q_out && (!bf || (r.q_stride != r.q_out_stride && tokens > 1))) return WQ_EINVAL;
      // other workgroups read or write these while the queries are written
      for (const void* p : {k, v, (const void*)slots, (const void*)r.positions, (const void*)r.cos_sin, (const void*)k_codes,
                            (const void*)k_scales, (const void*)v_codes, (const void*)v_scales})
        if (r.q_out == p) return WQ_EINVAL;
    }
    if (!wq_aligned(r.cos_sin) || !wq_aligned(r.q) || !wq_aligned(r.q_out)) return WQ_EALIGN;
  }
  if (tokens == 0) return WQ_OK;
  hipStream_t s = wq_stream(stream);
  const bool eight = cache == WQ_E4M3;
  // tokens a workgroup: few at least, so that a step's are spread over the chip (64 tokens x 8 heads: 4-bit 4.0-4.2 us in
  // fours, 4.3 singly, 5.0 in sixteens; 8-bit with rotation 4.5 in fours, 6.6 singly, where its workgroups are many)
  int chunk = !eight || rotary ? 4 : 1;
  while (chunk < 64 && (chunk < page || !eight) && (tokens + chunk - 1) / chunk * heads * 2 > 2048) chunk *= 2;
  const int64_t gx = (tokens + chunk - 1) / chunk;
  unsigned gz = 2;
  if (r.q_heads > 0) {
    const int64_t groups = (tokens * ((r.q_heads + QHEADS - 1) / QHEADS) * (head_dim / 16) + KV_THREADS - 1) / KV_THREADS;
    const int64_t z = (groups + gx * heads - 1) / (gx * heads);
    gz += (unsigned)(z < 65533 ? z : 65533);
  }
  const dim3 grid((unsigned)gx, (unsigned)heads, gz);
  auto run = [&](auto in, auto dim) {
    constexpr bool BF = decltype(in)::value;
    constexpr int D = decltype(dim)::value;
    if (!eight) {
      const Kv4Append a = {k, v, k_stride, v_stride, slots, tokens, num_pages, chunk, log2_page(page),
                           k_codes, k_scales, v_codes, v_scales};
      if (rotary) k_kv4_append<BF, true, D><<<grid, KV_THREADS, 0, s>>>(a, r);
      else k_kv4_append<BF, false, D><<<grid, KV_THREADS, 0, s>>>(a, r);
    } else if (rotary) {
      launch_append<BF, true, D>(page, grid, s, k, k_stride, v, v_stride, slots, tokens, chunk, num_pages, k_codes,
                                 k_scales, v_codes, v_scales, r);
    } else {
      launch_append<BF, false, D>(page, grid, s, k, k_stride, v, v_stride, slots, tokens, chunk, num_pages, k_codes,
                                  k_scales, v_codes, v_scales, r);
    }
  };
  using std::integral_constant;
  if (bf && head_dim == 128) run(integral_constant<bool, true>{}, integral_constant<int, 128>{});
  else if (bf) run(integral_constant<bool, true>{}, integral_constant<int, 64>{});
  else if (head_dim == 128) run(integral_constant<bool, false>{}, integral_constant<int, 128>{});
  else run(integral_constant<bool, false>{}, integral_constant<int, 64>{});
  return wq_launch_status();
}

}  // namespace

extern "C" {

wq_status wq_kv_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, int x_dtype,
                       const int64_t* slots, int64_t tokens, int32_t heads, int32_t head_dim, int32_t page,
                       int64_t num_pages, uint8_t* k_codes, uint8_t* k_scales, uint8_t* v_codes, uint8_t* v_scales,
                       void* stream) {
  return append(k, k_stride, v, v_stride, x_dtype, slots, tokens, heads, head_dim, WQ_E4M3, page, num_pages, k_codes,
                k_scales, v_codes, v_scales, nullptr, stream);
}

wq_status wq_kv4_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, int x_dtype,
                        const int64_t* slots, int64_t tokens, int32_t heads, int32_t head_dim, int32_t page,
                        int64_t num_pages, uint8_t* k_codes, uint8_t* k_scales, uint8_t* v_codes, uint8_t* v_scales,
                        void* stream) {
  return append(k, k_stride, v, v_stride, x_dtype, slots, tokens, heads, head_dim, WQ_E2M1X2, page, num_pages, k_codes,
                k_scales, v_codes, v_scales, nullptr, stream);
}

wq_status wq_kv_append_rotary(const void* q, int64_t q_stride, int32_t q_heads, const void* k, int64_t k_stride,
                              const void* v, int64_t v_stride, int x_dtype, const int32_t* positions,
                              const float* cos_sin, int64_t max_pos, int32_t rot, int32_t interleaved,
                              const int64_t* slots, int64_t tokens, int32_t heads, int32_t head_dim, int cache_dtype,
                              int32_t page, int64_t num_pages, uint8_t* k_codes, uint8_t* k_scales, uint8_t* v_codes,
                              uint8_t* v_scales, uint16_t* q_out, int64_t q_out_stride, void* stream) {
  const KvRotary r = {positions, cos_sin, max_pos, rot, interleaved != 0, q, q_stride, q_out, q_out_stride, q_heads};
  return append(k, k_stride, v, v_stride, x_dtype, slots, tokens, heads, head_dim, cache_dtype, page, num_pages, k_codes,
                k_scales, v_codes, v_scales, &r, stream);
}

}  // extern "C"

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

// Every workgroup scans the lengths of all requests (256 at a time: running
// sums of new tokens and of the pages needed, kept in LDS for the chunk) and
// writes its own rows of the token arrays, found by binary search in the
// chunk's token ends, and the table rows of the requests i with
// i % workgroups equal to its own number, one wave a row.  Workgroup 0 writes
// the per-request outputs.  There is no dependence between workgroups, so one
// launch does it all: the new pages of a token come from the free list
// itself, not from the table that another workgroup fills.
__global__ __launch_bounds__(KV_THREADS) void k_kv_blocks(
    const int32_t* __restrict__ ctx_lens, const int32_t* __restrict__ new_lens, int64_t batch,
    const int32_t* __restrict__ free_pages, int64_t num_free, const int32_t* __restrict__ cursor, int log_page,
    int32_t* __restrict__ table, int64_t max_blocks, int64_t tokens, int64_t* __restrict__ slots,
    int32_t* __restrict__ positions, int32_t* __restrict__ cu_new, int32_t* __restrict__ kv_lens,
    int32_t* __restrict__ state) {
  __shared__ int64_t ends[KV_THREADS];       // token rows up to and with each request of the chunk
  __shared__ int64_t firsts[KV_THREADS];     // its first new page's place in free_pages, -1 if refused
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
    const int64_t tok_first = tok_before;
    for (int w = 0; w < KV_THREADS / 64; w++) {
      tok_before += wave_sum[0][w];
      page_before += wave_sum[1][w];
    }
    __syncthreads();
    const int count = (int)(batch - base < KV_THREADS ? batch - base : KV_THREADS);
    // table rows
    const int64_t off = base % gridDim.x;
    int r0 = (int)(((int64_t)blockIdx.x + gridDim.x - off) % gridDim.x);
    for (int64_t r = r0 + (int64_t)wave * gridDim.x; r < count; r += (int64_t)gridDim.x * (KV_THREADS / 64)) {
      const int64_t f = firsts[r];
      if (f < 0) continue;
      const int64_t h = (ctxs[r] + page - 1) >> log_page, t = ((int64_t)ctxs[r] + news[r] + page - 1) >> log_page;
      for (int64_t j = h + lane; j < t; j += 64) table[(base + r) * max_blocks + j] = free_pages[f + j - h];
    }
    // token rows of this chunk's requests
    const int64_t lo = row0 > tok_first ? row0 : tok_first, hi = row1 < tok_before ? row1 : tok_before;
    for (int64_t row = lo + tid; row < hi; row += KV_THREADS) {
      int a = 0, z = count - 1;               // the first request whose end is behind the row
      while (a < z) {
        const int mid = (a + z) >> 1;
        if (ends[mid] > row) z = mid;
        else a = mid + 1;
      }
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

// The least E8M0 code c with amax <= 448 * 2^(c-127): 448 = 1.75 * 2^8, so
// the biased exponent less 8, one more where the fraction is above .75.
__device__ __forceinline__ int e8m0_cover(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int c = (int)(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return c > 0 ? c : 0;
}

// One run (tokens t .. t+n-1 at offsets off .. off+n-1 of one page) of one
// head, keys or values, by the whole workgroup.  The run stays in registers
// between its maximum and its codes.
template <bool BF16, bool VALUES, int D, int R>
__device__ __forceinline__ void append_run(const void* __restrict__ x, int64_t stride, int64_t t, int n, int off,
                                           int page, uint8_t* __restrict__ codes, uint8_t* __restrict__ scale,
                                           uint8_t* lds, float* red) {
  constexpr int CH = D / 8;                   // 8-element pieces of a token
  const int tid = threadIdx.x;
  const int old = off ? (int)*scale : 0;
  float v[R][8];
  float m = 0.0f;
#pragma unroll
  for (int r = 0; r < R; r++) {
    const int p = r * KV_THREADS + tid;
    if (p < n * CH) {
      load8<BF16>(x, (t + p / CH) * stride + (p % CH) * 8, v[r]);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float a = __builtin_fabsf(v[r][i]);
        m = a < INFINITY ? __builtin_fmaxf(m, a) : m;
      }
    }
  }
  m = group_max(m, 64);
  if ((tid & 63) == 0) red[tid >> 6] = m;
  __syncthreads();
  m = __builtin_fmaxf(__builtin_fmaxf(red[0], red[1]), __builtin_fmaxf(red[2], red[3]));
  const int need = e8m0_cover(m);
  const int c = need > old ? need : old;
  const int moved = off && c > old ? off : 0; // tokens before the run whose codes change
  if (tid == 0 && (!off || c != old)) *scale = (uint8_t)c;
#pragma unroll
  for (int r = 0; r < R; r++) {
    const int p = r * KV_THREADS + tid;
    if (p < n * CH) {
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; i++) q[i] = __builtin_ldexpf(v[r][i], 127 - c);
      const u32x2_t w = {e4m3_word(q), e4m3_word(q + 4)};
      if constexpr (!VALUES) {
        *reinterpret_cast<u32x2_t*>(codes + (off + p / CH) * D + (p % CH) * 8) = w;
      } else {
        uint8_t* o = lds + (p % CH) * 8 * (page + 4) + off + p / CH;
#pragma unroll
        for (int i = 0; i < 8; i++) o[i * (page + 4)] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
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
    const int w0 = moved ? 0 : off >> 2, words = ((off + n + 3) >> 2) - w0;
    for (int p = tid; p < D * words; p += KV_THREADS) {
      const int d = p / words, w = w0 + p % words;
      uint8_t* g = codes + d * page + 4 * w;
      const uint32_t fresh = *reinterpret_cast<const uint32_t*>(lds + d * (page + 4) + 4 * w);
      // bytes [a, z) of the word are this run's
      const int a = off - 4 * w > 0 ? off - 4 * w : 0, z = off + n - 4 * w < 4 ? off + n - 4 * w : 4;
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
  __syncthreads();                            // LDS is free for the next run
}

// Workgroup (x, head, keys or values) writes the runs that begin in tokens
// [x * chunk, (x + 1) * chunk).
template <bool BF16, int D, int R>
__global__ __launch_bounds__(KV_THREADS) void k_kv_append(
    const void* __restrict__ k, int64_t k_stride, const void* __restrict__ v, int64_t v_stride,
    const int64_t* __restrict__ slots, int64_t tokens, int chunk, int log_page, int64_t num_pages,
    uint8_t* __restrict__ k_codes, uint8_t* __restrict__ k_scales, uint8_t* __restrict__ v_codes,
    uint8_t* __restrict__ v_scales) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[D * (R * KV_THREADS * 8 / D + 4)];
  __shared__ float red[KV_THREADS / 64];
  __shared__ unsigned long long follow[2];
  const int tid = threadIdx.x, head = blockIdx.y, heads = gridDim.y, page = 1 << log_page;
  const int64_t limit = num_pages << log_page;
  const int64_t t1 = ((int64_t)blockIdx.x + 1) * chunk < tokens ? ((int64_t)blockIdx.x + 1) * chunk : tokens;
  for (int64_t t = (int64_t)blockIdx.x * chunk; t < t1; t++) {
    const int64_t slot = slots[t];
    const int off = (int)(slot & (page - 1));
    if (slot < 0 || slot >= limit) continue;
    if (t > 0 && off && slots[t - 1] == slot - 1) continue;
    // the run's length: tokens that follow on in the page
    if (tid < 128) {
      const bool on = tid < page - off && t + tid < tokens && slots[t + tid] == slot + tid;
      const unsigned long long b = __ballot(on);
      if ((tid & 63) == 0) follow[tid >> 6] = b;
    }
    __syncthreads();
    const unsigned long long b0 = ~follow[0], b1 = ~follow[1];
    const int n = b0 ? __builtin_ctzll(b0) : 64 + (b1 ? __builtin_ctzll(b1) : 64);
    const int64_t block = (slot >> log_page) * heads + head;
    const int64_t size = (int64_t)page * D;
    const int64_t col = (int64_t)head * D * (BF16 ? 2 : 4);
    if (blockIdx.z == 0)
      append_run<BF16, false, D, R>((const uint8_t*)k + col, k_stride, t, n, off, page, k_codes + block * size,
                                    k_scales + block, lds, red);
    else
      append_run<BF16, true, D, R>((const uint8_t*)v + col, v_stride, t, n, off, page, v_codes + block * size,
                                   v_scales + block, lds, red);
  }
}

// ---------------------------------------------------------------------------
// Attention
// ---------------------------------------------------------------------------
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  return __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(byte, 1.0f, false)[0];
}
__device__ __forceinline__ float e8m0_value(uint32_t c) { return __builtin_ldexpf(1.0f, (int)c - 127); }

// One wave per (row, query head): 64 tokens at a time, a lane's token in the
// scores, a lane's channels in the sums.
template <int D>
__global__ __launch_bounds__(64) void k_kv_attention(
    const uint16_t* __restrict__ q, int64_t q_stride, const int32_t* __restrict__ cu_q,
    const int32_t* __restrict__ kv_lens, int64_t batch, int64_t tokens, int q_heads, int kv_heads,
    const uint8_t* __restrict__ k_codes, const uint8_t* __restrict__ k_scales, const uint8_t* __restrict__ v_codes,
    const uint8_t* __restrict__ v_scales, int log_page, int64_t num_pages, const int32_t* __restrict__ table,
    int64_t max_blocks, float sm_scale, float softcap, int64_t window, uint16_t* __restrict__ out,
    float* __restrict__ lse) {
  __shared__ float qs[D];
  const int lane = threadIdx.x, head = blockIdx.y, kvh = head / (q_heads / kv_heads);
  const int64_t row = blockIdx.x;
  int64_t a = 0, z = batch;                   // the first request whose end is behind the row
  while (a < z) {
    const int64_t mid = (a + z) >> 1;
    if (cu_q[mid + 1] > row) z = mid;
    else a = mid + 1;
  }
  if (a >= batch || cu_q[a] > row || cu_q[a] < 0) return;
  const int64_t cap = max_blocks << log_page;
  int64_t len = kv_lens[a];
  len = len < 0 ? 0 : len > cap ? cap : len;
  const int64_t end = cu_q[a + 1] < tokens ? cu_q[a + 1] : tokens;
  const int64_t pos = len - end + row;
  const int64_t lo = window > 0 && pos - window + 1 > 0 ? pos - window + 1 : 0;
  for (int d = lane; d < D; d += 64) qs[d] = bf16_to_f32(q[row * q_stride + (int64_t)head * D + d]);
  __syncthreads();
  float m = -INFINITY, l = 0.0f, o[D / 64] = {};
  for (int64_t base = lo & ~(int64_t)63; base <= pos; base += 64) {
    const int64_t j = base + lane;
    const bool in = j >= lo && j <= pos;
    const int64_t id = in ? table[a * max_blocks + (j >> log_page)] : -1;
    const bool seen = id >= 0 && id < num_pages;
    const int64_t block = seen ? id * kv_heads + kvh : 0;
    const int off = (int)(j & ((1 << log_page) - 1));
    float s = -INFINITY;
    if (seen) {
      const uint8_t* kp = k_codes + ((block << log_page) + off) * D;
      float dot = 0.0f;
      for (int d = 0; d < D; d++) dot = __builtin_fmaf(qs[d], e4m3_value(kp[d]), dot);
      s = dot * e8m0_value(k_scales[block]) * sm_scale;
      if (softcap > 0.0f) s = softcap * tanhf(s / softcap);
    }
    const float mt = group_max(s, 64);
    const float mn = __builtin_fmaxf(m, mt);
    const float use = mn == -INFINITY ? 0.0f : mn;
    const float keep = expf(m - use);
    float p = seen ? expf(s - use) : 0.0f;
    float sum = p;
    for (int x = 1; x < 64; x <<= 1) sum += __shfl_xor(sum, x, 64);
    l = l * keep + sum;
    m = mn;
    const float pv = seen ? p * e8m0_value(v_scales[block]) : 0.0f;
    for (int e = 0; e < D / 64; e++) o[e] *= keep;
    for (int i = 0; i < 64; i++) {
      if (!__shfl((int)seen, i, 64)) continue;
      const int64_t bi = __shfl(block, i, 64);
      const int oi = __shfl(off, i, 64);
      const float pi = __shfl(pv, i, 64);
      for (int e = 0; e < D / 64; e++)
        o[e] = __builtin_fmaf(pi, e4m3_value(v_codes[((bi * D + lane + 64 * e) << log_page) + oi]), o[e]);
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
  for (int e = 0; e < D / 64; e++) out[(row * q_heads + head) * D + lane + 64 * e] = (uint16_t)f32_to_bf16_bits(o[e] * inv);
  if (lse && lane == 0) lse[row * q_heads + head] = l == 0.0f ? -INFINITY : m + logf(l);
}

int log2_page(int page) {
  return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : page == 128 ? 7 : -1;
}

template <bool BF16, int D>
void launch_append(int page, dim3 grid, hipStream_t s, const void* k, int64_t ks, const void* v, int64_t vs,
                   const int64_t* slots, int64_t tokens, int chunk, int64_t num_pages, uint8_t* kc, uint8_t* ksc,
                   uint8_t* vc, uint8_t* vsc) {
  const int lp = log2_page(page);
#define WQ_APPEND(PAGE)                                                                                             \
  k_kv_append<BF16, D, (PAGE * D / 8 + KV_THREADS - 1) / KV_THREADS><<<grid, KV_THREADS, 0, s>>>(                    \
      k, ks, v, vs, slots, tokens, chunk, lp, num_pages, kc, ksc, vc, vsc)
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
  if (kv_lens && (kv_lens == ctx_lens || kv_lens == new_lens)) return WQ_EINVAL;
  if (cu_new == ctx_lens || cu_new == new_lens || cu_new == cursor || state == cursor || state == ctx_lens ||
      state == new_lens || (block_table && block_table == free_pages))
    return WQ_EINVAL;
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
  while (chunk < 64 && chunk < page && (tokens + chunk - 1) / chunk * heads * 2 > 4096) chunk *= 2;
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

size_t wq_kv_attention_workspace_size(int64_t batch, int64_t tokens, int64_t max_q, int32_t q_heads, int32_t kv_heads,
                                      int32_t head_dim, int32_t page, int64_t max_blocks) {
  (void)batch, (void)tokens, (void)max_q, (void)q_heads, (void)kv_heads, (void)head_dim, (void)page, (void)max_blocks;
  return 0;
}

wq_status wq_kv_attention(const void* q_bf16, int64_t q_stride, const int32_t* cu_q, const int32_t* kv_lens,
                          int64_t batch, int64_t tokens, int64_t max_q, int32_t q_heads, int32_t kv_heads,
                          int32_t head_dim, const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes,
                          const uint8_t* v_scales, int32_t page, int64_t num_pages, const int32_t* block_table,
                          int64_t max_blocks, float sm_scale, float softcap, int64_t window, uint16_t* out,
                          float* lse, void* workspace, size_t ws_bytes, void* stream) {
  if ((head_dim != 64 && head_dim != 128) || log2_page(page) < 0) return WQ_EUNSUPPORTED;
  if (batch < 0 || batch > 0x7FFFFFFF || tokens < 0 || tokens > 0x7FFFFFFF || max_q < 0 || kv_heads < 1 ||
      q_heads < kv_heads || q_heads % kv_heads || q_heads > 65535 || num_pages < 1 || max_blocks < 1 ||
      max_blocks > 0x7FFFFFFF / page || window < 0)
    return WQ_EINVAL;
  if (!(sm_scale > 0.0f) || !(sm_scale < INFINITY) || !(softcap >= 0.0f) || !(softcap < INFINITY)) return WQ_EINVAL;
  const int64_t row = (int64_t)q_heads * head_dim;
  if (q_stride < row || q_stride % 8 || q_stride > (int64_t(1) << 40) ||
      !wq_numel_ok(num_pages, (int64_t)kv_heads * head_dim * page) || !wq_numel_ok(tokens ? tokens : 1, row) ||
      !wq_numel_ok(batch ? batch : 1, max_blocks))
    return WQ_EINVAL;
  if (!k_codes || !k_scales || !v_codes || !v_scales) return WQ_EINVAL;
  if (batch > 0 && tokens > 0 && (!q_bf16 || !cu_q || !kv_lens || !block_table || !out)) return WQ_EINVAL;
  if (!wq_aligned(q_bf16) || !wq_aligned(out) || !wq_aligned(k_codes) || !wq_aligned(v_codes) || !wq_aligned(workspace))
    return WQ_EALIGN;
  if (ws_bytes < wq_kv_attention_workspace_size(batch, tokens, max_q, q_heads, kv_heads, head_dim, page, max_blocks))
    return WQ_EINVAL;
  if (batch == 0 || tokens == 0) return WQ_OK;
  const dim3 grid((unsigned)tokens, (unsigned)q_heads);
  const int lp = log2_page(page);
  if (head_dim == 128)
    k_kv_attention<128><<<grid, 64, 0, (hipStream_t)stream>>>(
        (const uint16_t*)q_bf16, q_stride, cu_q, kv_lens, batch, tokens, q_heads, kv_heads, k_codes, k_scales, v_codes,
        v_scales, lp, num_pages, block_table, max_blocks, sm_scale, softcap, window, out, lse);
  else
    k_kv_attention<64><<<grid, 64, 0, (hipStream_t)stream>>>(
        (const uint16_t*)q_bf16, q_stride, cu_q, kv_lens, batch, tokens, q_heads, kv_heads, k_codes, k_scales, v_codes,
        v_scales, lp, num_pages, block_table, max_blocks, sm_scale, softcap, window, out, lse);
  return wq_launch_status();
}

}  // extern "C"

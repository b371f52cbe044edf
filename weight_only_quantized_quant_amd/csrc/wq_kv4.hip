// Attention over the 4-bit key/value cache for gfx950 (E2M1 elements, one E8M0
// scale per 32 channels of a token and head).
#include "wq_kv_common.h"

namespace {

// Scale codes above this count as it: the largest value is then 6 * 2^125, finite
// in bf16 and fp32.
constexpr uint32_t KV4_TOP = 252;

// One wave a row and query head: a lane a token for the scores, two channels a
// lane for the sums.
template <int D, bool CAP>
__global__ __launch_bounds__(64) void k_kv4_rows(const KvArgs A) {
  __shared__ float qs[D], ps[64];
  __shared__ int ids[64];
  const int lane = threadIdx.x, head = blockIdx.y, kvh = head / A.group;
  const int64_t t = blockIdx.x;
  int q0 = 0, n = 0, len = 0;
  int64_t request = -1;
  for (int64_t base = 0; base < A.batch && request < 0; base += 64) {
    KvRequest r;
    r.load<1, REQ_ALL>(A, base + lane);
    const unsigned long long at = __ballot(r.n > 0 && t >= r.q0 && t < r.q0 + r.n);
    if (!at) continue;
    const int src = __builtin_ctzll(at);
    request = base + src;
    q0 = lane32(r.q0, src);
    n = lane32(r.n, src);
    len = lane32(r.len, src);
  }
  if (request < 0) return;
  const int pos = len - n + (int)(t - q0), lo = kv_lowest(pos, A.window), last_col = (int)A.max_blocks - 1;
  for (int d = lane; d < D; d += 64) qs[d] = bf16_to_f32(A.q[t * A.q_stride + (int64_t)head * D + d]);
  __syncthreads();
  const KvScore<CAP> sc(A);
  const int in_page = (1 << A.log_page) - 1;
  float mx = -INFINITY, l = 0.0f, o[2] = {0.0f, 0.0f};
  for (int j0 = lo; j0 <= pos; j0 += 64) {
    const int j = j0 + lane, col = j >> A.log_page;
    int id = j <= pos ? A.table[request * A.max_blocks + (col < last_col ? col : last_col)] : -1;
    if (id < 0 || id >= A.num_pages) id = -1;
    float s = -INFINITY;
    if (id >= 0) {
      const int64_t block = (int64_t)id * A.kv_heads + kvh;
      const uint8_t* k = A.k_codes + (((block << A.log_page) + (j & in_page)) * (D / 2));
      s = 0.0f;
      for (int b = 0; b < D / 32; b++) {
        uint32_t c = A.k_scales[((block * (D / 32) + b) << A.log_page) + (j & in_page)];
        c = c < KV4_TOP ? c : KV4_TOP;
        for (int w = 0; w < 4; w++) {
          const uint32_t codes = *reinterpret_cast<const uint32_t*>(k + 16 * b + 4 * w);
          uint32_t v[4];
          dq_fp4_word(codes, e8m0_as_scale(c), v);
          for (int e = 0; e < 4; e++)
            s += qs[32 * b + 8 * w + 2 * e] * bf16_lo(v[e]) + qs[32 * b + 8 * w + 2 * e + 1] * bf16_hi(v[e]);
        }
      }
      s = CAP ? (__builtin_fabsf(s) > sc.limit ? sc.exponential(s) : sc.series(s)) : s * sc.mul;
    }
    float top = s;
    for (int e = 1; e < 64; e <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, e, 64));
    const float mn = __builtin_fmaxf(mx, top);
    if (mn == -INFINITY) continue;
    const float keep = __builtin_amdgcn_exp2f(mx - mn), p = __builtin_amdgcn_exp2f(s - mn);
    float sum = p;
    for (int e = 1; e < 64; e <<= 1) sum += __shfl_xor(sum, e, 64);
    l = l * keep + sum;
    mx = mn;
    o[0] *= keep;
    o[1] *= keep;
    __syncthreads();
    ps[lane] = p;
    ids[lane] = id;
    __syncthreads();
    for (int i = 0; i < 64 && j0 + i <= pos; i++) {
      if (ids[i] < 0 || lane >= D / 2) continue;
      const int64_t block = (int64_t)ids[i] * A.kv_heads + kvh;
      const int off = (j0 + i) & in_page;
      uint32_t c = A.v_scales[((block * (D / 32) + lane / 16) << A.log_page) + off];
      c = c < KV4_TOP ? c : KV4_TOP;
      const uint32_t v = dq_fp4_pair<0>(A.v_codes[((block * (D / 2) + lane) << A.log_page) + off], e8m0_as_scale(c));
      o[0] += ps[i] * bf16_lo(v);
      o[1] += ps[i] * bf16_hi(v);
    }
  }
  const int64_t orow = t * A.q_heads + head;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (lane < D / 2) *reinterpret_cast<uint32_t*>(A.out + orow * D + 2 * lane) = pack_bf16x2(o[0] * inv, o[1] * inv);
  if (A.lse && lane == 0) A.lse[orow] = l == 0.0f ? -INFINITY : (mx + __builtin_log2f(l)) * LN2;
}

}  // namespace

extern "C" {

size_t wq_kv4_attention_workspace_size(int64_t, int64_t, int64_t, int32_t, int32_t, int32_t, int32_t, int64_t, int64_t) {
  return 0;
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
  if (batch == 0 || tokens == 0) return WQ_OK;
  const KvArgs A = {(const uint16_t*)q_bf16, q_stride, cu_q, kv_lens, batch, tokens, q_heads, kv_heads,
                    q_heads / kv_heads, (int)(window < 0x7FFFFFFF ? window : 0), k_codes, k_scales, v_codes, v_scales,
                    log2_page(page), num_pages, block_table, max_blocks, sm_scale, softcap, out, lse};
  const dim3 grid((unsigned)tokens, (unsigned)q_heads);
  hipStream_t s = (hipStream_t)stream;
  if (head_dim == 128) {
    if (softcap > 0.0f) k_kv4_rows<128, true><<<grid, 64, 0, s>>>(A);
    else k_kv4_rows<128, false><<<grid, 64, 0, s>>>(A);
  } else {
    if (softcap > 0.0f) k_kv4_rows<64, true><<<grid, 64, 0, s>>>(A);
    else k_kv4_rows<64, false><<<grid, 64, 0, s>>>(A);
  }
  return wq_launch_status();
}

}  // extern "C"

// kv4_attn.hip -- attention over the paged 4-bit key/value cache.
//
// Mathematics. For a query row, o = sum_j w_j v_j / sum_j w_j with w_j =
// 2^(x_j - m), x_j = scale log2(e) q . k_j and m the running maximum: one pass
// over the keys, the sums being multiplied by 2^(m_old - m_new) whenever the
// maximum moves.
//
// The plain kernel: a workgroup per row and query head; GL = head_dim / 8
// lanes (rounded up to a power of two) hold 8 channels each, so a wave works
// on 64 / GL keys at a time and the dot product is a lane reduction.
#include <algorithm>

#include "gq_device.h"
#include "kv4.h"

namespace gq {

namespace {

constexpr int kThreads = 256;

// The keys that a row sees: lo .. hi - 1 (none: hi <= lo).
struct Seen {
  int lo, hi;
};

__device__ __forceinline__ Seen seen_keys(const AttnArgs& a, int pos, int len) {
  Seen s;
  s.hi = a.causal ? (pos + 1 < len ? pos + 1 : len) : len;
  s.lo = a.window > 0 && pos + 1 > a.window ? pos + 1 - a.window : 0;
  return s;
}

__device__ __forceinline__ int clamped_len(const AttnArgs& a, int len) {
  return len < 0 ? 0 : len > a.max_len ? a.max_len : len;
}

// 8 channels of one key or value: d (n - 8).
__device__ __forceinline__ void load8(const Kv4Args& c, const uint8_t* part, int slot, int sub, float x[8]) {
  const uint32_t code = load_u32(part + slot * (c.hd / 2) + sub * 4);
  const float d = half_bits_to_float(
      load_u16(part + kv4_code_bytes(c.hd, c.page_log2) + 2 * (((sub >> 2) << c.page_log2) + slot)));
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = d * (float)((int)(code >> (4 * ((i >> 1) + 4 * (i & 1))) & 15) - 8);
}

template <int GL>
__global__ __launch_bounds__(kThreads) void attn_plain_kernel(AttnArgs a) {
  constexpr int kKeys = kThreads / GL;  // keys in flight
  __shared__ float sm[kKeys], sl[kKeys], so[kKeys][GL * 8 + 1];
  const int tid = threadIdx.x, sub = tid % GL, g = tid / GL;
  const Kv4Args& c = a.c;
  const int h = blockIdx.y, kvh = h / a.group;
  const bool on = sub * 8 < c.hd;
  const int cl = on ? sub : 0;
  for (int b = 0, t = blockIdx.x; t < c.n_tok; t += gridDim.x) {
    // the row's sequence
    SeqRows s{0, 0, 0};
    if (c.q_start) {
      int lo = 0, hi = c.n_seq;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (c.q_start[mid + 1] <= t) lo = mid + 1;
        else hi = mid;
      }
      b = lo;
    } else {
      b = t;
    }
    if (b >= c.n_seq) continue;
    s = seq_rows(c, b);
    const int64_t i = (int64_t)t - s.first;
    if (i < 0 || i >= s.n || i >= a.max_q) continue;
    const int len = clamped_len(a, s.len);
    const Seen k = seen_keys(a, len - s.n + (int)i, len);
    const float* q = a.q + t * a.q_stride + (int64_t)h * c.hd;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = on ? q[sub * 8 + e] * a.scale : 0.f;
    float m = -INFINITY, l = 0.f, o[8] = {};
    for (int j = k.lo + g; j < k.hi; j += kKeys) {
      const uint8_t* page = page_of(c, b, j);
      const int slot = j & ((1 << c.page_log2) - 1);
      float kx[8], vx[8];
      if (page) {
        load8(c, page + kv4_part(c, kvh, 0), slot, cl, kx);
        load8(c, page + kv4_part(c, kvh, 1), slot, cl, vx);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) kx[e] = vx[e] = __builtin_nanf("");
      }
      float d = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) d = __builtin_fmaf(x[e], kx[e], d);
      if (!on) d = 0.f;
#pragma unroll
      for (int w = GL / 2; w > 0; w /= 2) d += __shfl_xor(d, w, GL);
      const float mn = fmaxf(m, d), base = mn == -INFINITY ? 0.f : mn;
      const float r = exp2f(m - base), p = exp2f(d - base);
      l = l * r + p;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = o[e] * r + p * vx[e];
      m = mn;
    }
    __syncthreads();
    if (sub == 0) sm[g] = m, sl[g] = l;
#pragma unroll
    for (int e = 0; e < 8; ++e) so[g][sub * 8 + e] = o[e];
    __syncthreads();
    float mx = -INFINITY;
    for (int e = 0; e < kKeys; ++e) mx = fmaxf(mx, sm[e]);
    if (mx == -INFINITY) mx = 0.f;
    for (int ch = tid; ch < c.hd; ch += kThreads) {
      float lt = 0.f, ot = 0.f;
      for (int e = 0; e < kKeys; ++e) {
        const float r = exp2f(sm[e] - mx);
        lt += r * sl[e];
        ot += r * so[e][ch];
      }
      a.out[t * a.out_stride + (int64_t)h * c.hd + ch] = k.hi > k.lo ? ot / lt : 0.f;
    }
  }
}

}  // namespace

int kv4_attn_splits(int64_t, int64_t, int64_t, int64_t) { return 1; }

hipError_t launch_kv4_attn(const AttnArgs& a, hipStream_t s) {
  const int gl = a.c.hd <= 32 ? 4 : a.c.hd <= 64 ? 8 : a.c.hd <= 128 ? 16 : 32;
  const dim3 grid(std::min(a.c.n_tok, 1 << 20), a.n_head), block(kThreads);
  if (gl == 4) hipLaunchKernelGGL((attn_plain_kernel<4>), grid, block, 0, s, a);
  else if (gl == 8) hipLaunchKernelGGL((attn_plain_kernel<8>), grid, block, 0, s, a);
  else if (gl == 16) hipLaunchKernelGGL((attn_plain_kernel<16>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((attn_plain_kernel<32>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace gq

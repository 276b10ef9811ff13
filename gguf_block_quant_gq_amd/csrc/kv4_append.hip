// kv4_append.hip -- rotary positions with per-head norms, storing keys and
// values in the paged 4-bit cache, and reading them back.
//
// Mathematics. A head of hd channels is first normed, x_c w_c / sqrt(mean
// x_c^2 + eps), and its first rot channels are turned in pairs by the angle
// pos * freq_p. Keys go on into 4-bit blocks: d = -a / 8 (a: the block's value
// of largest magnitude) rounded to 8 significant bits, codes rint(x / d).
//
// Everything up to the rounding into fp32 or into a block is fp64. The
// kernels move 8 to 10 bytes per element for about 10 fp64 operations, which
// the vector units do well inside the time the bytes take; in return the angle
// of a far position is exact to fp64, and a code or a scale next to a rounding
// border falls on the formula's side of it, so that two evaluations of the
// same formula agree on every held value.
//
// Split. hd / 8 lanes (rounded up to a power of two) own a head, 8 channels
// each; a wave holds whole heads, so the norm's sum and the block's largest
// value are lane exchanges, and a head may be turned in place (its loads all
// precede its stores). A workgroup takes one token at a time: its sines and
// cosines (about 60 fp64 operations a pair) are computed once into LDS and
// kept in registers over the token's heads.
#include <algorithm>

#include "gq_device.h"
#include "kv4.h"

namespace gq {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;  // head_dim / 2

typedef double f64x2 __attribute__((ext_vector_type(2)));

// sin and cos of a: a is brought into [-pi/4, pi/4] by subtracting k pi/2 in
// two parts (pi/2 rounded to fp64, whose multiple leaves an exact difference,
// and the remainder), then the two Taylor series, whose first omitted terms
// are below 1e-19 there.
__device__ __forceinline__ f64x2 sin_cos(double a) {
  const double k = __builtin_rint(a * 0.63661977236758134308);  // 2 / pi
  double r = __builtin_fma(-k, 1.57079632679489661923, a);      // pi / 2
  r = __builtin_fma(-k, 6.12323399573676603587e-17, r);         // pi / 2 - fp64(pi / 2)
  const double z = r * r;
  double s = 1.0 / 355687428096000.0;  // 1 / 17!
  s = __builtin_fma(s, -z, 1.0 / 1307674368000.0);
  s = __builtin_fma(s, -z, 1.0 / 6227020800.0);
  s = __builtin_fma(s, -z, 1.0 / 39916800.0);
  s = __builtin_fma(s, -z, 1.0 / 362880.0);
  s = __builtin_fma(s, -z, 1.0 / 5040.0);
  s = __builtin_fma(s, -z, 1.0 / 120.0);
  s = __builtin_fma(s, -z, 1.0 / 6.0);
  s = __builtin_fma(-r * z, s, r);
  double c = 1.0 / 6402373705728000.0;  // 1 / 18!
  c = __builtin_fma(c, -z, 1.0 / 20922789888000.0);
  c = __builtin_fma(c, -z, 1.0 / 87178291200.0);
  c = __builtin_fma(c, -z, 1.0 / 479001600.0);
  c = __builtin_fma(c, -z, 1.0 / 3628800.0);
  c = __builtin_fma(c, -z, 1.0 / 40320.0);
  c = __builtin_fma(c, -z, 1.0 / 720.0);
  c = __builtin_fma(c, -z, 1.0 / 24.0);
  c = __builtin_fma(c, -z, 1.0 / 2.0);
  c = __builtin_fma(c, -z, 1.0);
  // quadrant: k mod 4 (k is a whole number; fp64 keeps it for any int32 position)
  const double q = k - 4.0 * __builtin_floor(k * 0.25);
  const bool swap = q == 1.0 || q == 3.0;
  const double ss = swap ? c : s, cc = swap ? s : c;
  return f64x2{q >= 2.0 ? -ss : ss, q == 1.0 || q == 2.0 ? -cc : cc};
}

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// The sum over aligned groups of GL lanes, in every lane of the group.
template <int GL>
__device__ __forceinline__ double group_sum_f64(double v) {
  if constexpr (GL >= 2) v += dpp_f64<0xB1>(v);   // quad_perm [1,0,3,2]
  if constexpr (GL >= 4) v += dpp_f64<0x4E>(v);   // quad_perm [2,3,0,1]
  if constexpr (GL >= 8) v += dpp_f64<0x141>(v);  // row_half_mirror
  if constexpr (GL >= 16) v += dpp_f64<0x140>(v); // row_mirror
  if constexpr (GL >= 32) v += __shfl_xor(v, 16);
  return v;
}

// A block's scale from its value of largest magnitude a: -a / 8 rounded to 8
// significant bits (steps no finer than 2^-24), at most 8160 in magnitude.
// Adding 1.5 * 2^52 steps rounds to a whole number of steps, ties to even.
__device__ __forceinline__ double block_scale(double a) {
  const double d = a * -0.125;
  const int e = (int)((__builtin_bit_cast(uint64_t, d) >> 52) & 0x7FF) - 1023;
  const int u = e - 7 < -24 ? -24 : e - 7 > 8 ? 8 : e - 7;  // past 2^15 the bound below decides
  const double big = __builtin_bit_cast(double, (uint64_t)(u + 52 + 1023) << 52) * 1.5;
  const double r = (d + big) - big;
  if (d != d) return d;
  return r > 8160.0 ? 8160.0 : r < -8160.0 ? -8160.0 : r;
}

// rint(x / d), ties to even, clamped to -8 .. 7. x times 1/d may be off by a
// few units of 2^-52, enough to miss an exact tie: the remainder x - r d is
// exact, and is compared with d / 2.
__device__ __forceinline__ int block_code(double x, double d, double inv) {
  double t = x * inv;
  t = t < -8.0 ? -8.0 : t > 7.0 ? 7.0 : t;  // a NaN passes both tests and ends as code 0
  double r = __builtin_rint(t);
  const double rem = __builtin_fma(-r, d, x);  // in units of d: x / d - r
  const double twice = 2.0 * __builtin_fabs(rem), ad = __builtin_fabs(d);
  const double side = (rem < 0) == (d < 0) ? 1.0 : -1.0;
  const bool odd = ((int)r & 1) != 0;
  if (twice > ad || (twice == ad && odd)) r += side;
  r = r < -8.0 ? -8.0 : r > 7.0 ? 7.0 : r;
  return (int)r;
}

struct QkArgs {
  Kv4Args c;           // append only
  HeadArgs part[3];    // queries, keys, values (append: out of keys and values unused)
  RopeArgs r;
  const int32_t* pos;  // gq_qk_rope only
  int n_tok;
  int hd;
  float eps;
};

// GL lanes per head. FAST: whole groups of 8 channels turn with a whole group
// (rot a multiple of 16, or of 8 with interleaved pairs), so partners are one
// more 32-byte load.
template <int GL, bool APPEND, bool FAST>
__global__ __launch_bounds__(kThreads) void qk_rope_kernel(QkArgs a) {
  __shared__ f64x2 turn[kMaxPairs];
  constexpr int kHeads = kThreads / GL;  // heads per pass
  const int tid = threadIdx.x, sub = tid % GL, slot = tid / GL;
  const int hd = a.hd, c0 = sub * 8, half = a.r.half;
  const bool lane_on = c0 < hd;
  const int heads = a.part[0].n_head + (APPEND ? a.part[1].n_head + a.part[2].n_head : 0);

  // this lane's partners: channel c turns with c + half, or with c - half
  // (half layout), or with its neighbour (interleaved)
  const bool low = c0 < half, rot_on = lane_on && c0 < 2 * half;
  const int pc0 = a.r.interleaved || !rot_on ? c0 : low ? c0 + half : c0 - half;

  for (int t = blockIdx.x; t < a.n_tok; t += gridDim.x) {
    int seq = 0, pos = 0;
    if constexpr (APPEND) {
      pos = row_position(a.c, t, &seq);
      if (pos < 0) continue;  // the same for the whole workgroup
    } else {
      pos = half > 0 ? a.pos[t] : 0;
    }
    __syncthreads();  // the pass before has read its turns
    for (int p = tid; p < half; p += kThreads) {
      const f64x2 sc = sin_cos((double)pos * (double)a.r.freqs[p]);
      turn[p] = sc * (double)a.r.mscale;
    }
    __syncthreads();
    uint8_t* page = nullptr;
    if constexpr (APPEND) page = page_of(a.c, seq, pos);

    for (int h0 = blockIdx.y * kHeads; h0 < heads; h0 += gridDim.y * kHeads) {
      int h = h0 + slot, kind = 0;
      if constexpr (APPEND) {
        if (h >= a.part[0].n_head) h -= a.part[0].n_head, kind = 1;
        if (kind == 1 && h >= a.part[1].n_head) h -= a.part[1].n_head, kind = 2;
      }
      const HeadArgs& ha = APPEND ? a.part[kind] : a.part[0];
      const bool on = lane_on && h0 + slot < heads;
      const bool turns = on && rot_on && kind != 2;
      const float* xh = ha.x + t * ha.x_stride + (int64_t)(on ? h : 0) * hd;
      double y[8], z[8];  // this lane's channels and their partners
      const int cl = lane_on ? c0 : 0;
      {
        const f32x4 u = load_f32x4(xh + cl), v = load_f32x4(xh + cl + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = on ? u[i] : 0.f, y[i + 4] = on ? v[i] : 0.f;
      }
      if (turns && !a.r.interleaved) {
        if constexpr (FAST) {
          const f32x4 u = load_f32x4(xh + pc0), v = load_f32x4(xh + pc0 + 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = u[i], z[i + 4] = v[i];
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int c = c0 + i;
            z[i] = xh[c < half ? c + half : c < 2 * half ? c - half : c];
          }
        }
      }
      const float* w = ha.w;
      if (w && kind != 2) {
        double ss = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __builtin_fma(y[i], y[i], ss);
        ss = group_sum_f64<GL>(ss);
        const double rs = 1.0 / __builtin_sqrt(ss / hd + (double)a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[i] *= rs * (double)w[cl + i];
          if (turns && !a.r.interleaved) {
            const int c = c0 + i;
            z[i] *= rs * (double)w[FAST ? pc0 + i : c < half ? c + half : c < 2 * half ? c - half : c];
          }
        }
      }
      if (turns) {
        if (a.r.interleaved) {
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const int p = (c0 + i) >> 1;
            if (FAST || p < half) {
              const f64x2 sc = turn[p];
              const double u = y[i], v = y[i + 1];
              y[i] = u * sc.y - v * sc.x;
              y[i + 1] = v * sc.y + u * sc.x;
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int c = c0 + i;
            const bool lo = FAST ? low : c < half;
            if (FAST || c < 2 * half) {
              const f64x2 sc = turn[lo ? c : c - half];
              y[i] = lo ? y[i] * sc.y - z[i] * sc.x : y[i] * sc.y + z[i] * sc.x;
            }
          }
        }
      }
      if (!APPEND || kind == 0) {
        if (on) {
          float* o = ha.out + t * ha.out_stride + (int64_t)h * hd + c0;
          const f32x4 u = {(float)y[0], (float)y[1], (float)y[2], (float)y[3]};
          const f32x4 v = {(float)y[4], (float)y[5], (float)y[6], (float)y[7]};
          __builtin_memcpy(__builtin_assume_aligned(o, 4), &u, 16);
          __builtin_memcpy(__builtin_assume_aligned(o + 4, 4), &v, 16);
        }
      } else {
        // the block's value of largest magnitude: the lowest channel among
        // equals, a NaN before everything (four lanes share a block)
        double best = y[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) {
          const bool take = best == best && !(__builtin_fabs(y[i]) <= __builtin_fabs(best));
          best = take ? y[i] : best;
        }
        {
          const double o1 = dpp_f64<0xB1>(best);
          const bool up = (tid & 1) != 0;  // the lower lane wins a tie
          bool take = !(__builtin_fabs(o1) <= __builtin_fabs(best)) || (up && __builtin_fabs(o1) == __builtin_fabs(best));
          best = best == best && take ? o1 : best;
          const double o2 = dpp_f64<0x4E>(best);
          const bool up2 = (tid & 2) != 0;
          take = !(__builtin_fabs(o2) <= __builtin_fabs(best)) || (up2 && __builtin_fabs(o2) == __builtin_fabs(best));
          best = best == best && take ? o2 : best;
        }
        const double d = block_scale(best);
        const double inv = d != 0.0 ? 1.0 / d : 0.0;
        uint32_t word = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t n = d != 0.0 && d == d ? (uint32_t)(block_code(y[i], d, inv) + 8) : 8u;
          word |= n << (4 * ((i >> 1) + 4 * (i & 1)));
        }
        if (on && page) {
          const int s = pos & ((1 << a.c.page_log2) - 1);
          uint8_t* part = page + kv4_part(a.c, h, kind - 1);
          *reinterpret_cast<uint32_t*>(part + s * (hd / 2) + sub * 4) = word;
          if (sub % 4 == 0) {
            const _Float16 d16 = (_Float16)(float)d;
            _Float16* scales = reinterpret_cast<_Float16*>(part + kv4_code_bytes(hd, a.c.page_log2));
            scales[((sub / 4) << a.c.page_log2) + s] = d16;
          }
        }
      }
    }
  }
}

// K and V of the token rows: a thread expands one dword of codes.
__global__ __launch_bounds__(kThreads) void kv4_read_kernel(Kv4Args c, float* __restrict__ K, float* __restrict__ V) {
  const int words = c.hd / 8, per_row = 2 * c.n_kv * words;
  for (int t = blockIdx.x; t < c.n_tok; t += gridDim.x) {
    int seq = 0;
    const int pos = row_position(c, t, &seq);
    if (pos < 0) continue;
    const uint8_t* page = page_of(c, seq, pos);
    const int s = pos & ((1 << c.page_log2) - 1);
    for (int i = blockIdx.y * kThreads + threadIdx.x; i < per_row; i += gridDim.y * kThreads) {
      const int kv = i >= c.n_kv * words, j = i - kv * c.n_kv * words;
      const int h = j / words, w = j - h * words;
      float* out = kv ? V : K;
      if (!out) continue;
      f32x4 u, v;
      if (page) {
        const uint8_t* part = page + kv4_part(c, h, kv);
        const uint32_t code = load_u32(part + s * (c.hd / 2) + w * 4);
        const float d = half_bits_to_float(
            load_u16(part + kv4_code_bytes(c.hd, c.page_log2) + 2 * (((w >> 2) << c.page_log2) + s)));
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          u[b] = d * (float)((int)(code >> (4 * ((b >> 1) + 4 * (b & 1))) & 15) - 8);
          v[b] = d * (float)((int)(code >> (4 * (2 + (b >> 1) + 4 * (b & 1))) & 15) - 8);
        }
      } else {
        u = v = f32x4{__builtin_nanf(""), __builtin_nanf(""), __builtin_nanf(""), __builtin_nanf("")};
      }
      float* o = out + ((int64_t)t * c.n_kv + h) * c.hd + w * 8;
      __builtin_memcpy(__builtin_assume_aligned(o, 4), &u, 16);
      __builtin_memcpy(__builtin_assume_aligned(o + 4, 4), &v, 16);
    }
  }
}

template <bool APPEND>
hipError_t launch_qk(const QkArgs& a, int heads, hipStream_t s) {
  const int gl = a.hd <= 32 ? 4 : a.hd <= 64 ? 8 : a.hd <= 128 ? 16 : 32;
  const int passes = (heads * gl + kThreads - 1) / kThreads;
  // few tokens: a workgroup per pass over the heads, each with its own turns
  // (latency counts); many: one workgroup per token computes them once
  const int gy = a.n_tok >= 1024 ? 1 : std::min(passes, 65535);
  const int gx = std::min(a.n_tok, 1 << 20);
  const bool fast = a.r.half == 0 || (a.r.interleaved ? a.r.half % 4 == 0 : a.r.half % 8 == 0);
  const dim3 grid(gx, gy), block(kThreads);
#define GQ_QK_LAUNCH(GL)                                                                               \
  do {                                                                                                 \
    if (fast) hipLaunchKernelGGL((qk_rope_kernel<GL, APPEND, true>), grid, block, 0, s, a);            \
    else hipLaunchKernelGGL((qk_rope_kernel<GL, APPEND, false>), grid, block, 0, s, a);                \
  } while (0)
  if (gl == 4) GQ_QK_LAUNCH(4);
  else if (gl == 8) GQ_QK_LAUNCH(8);
  else if (gl == 16) GQ_QK_LAUNCH(16);
  else GQ_QK_LAUNCH(32);
#undef GQ_QK_LAUNCH
  return hipGetLastError();
}

}  // namespace

hipError_t launch_qk_rope(const HeadArgs& h, int n_tok, int hd, const int32_t* pos, const RopeArgs& r, float eps,
                          hipStream_t s) {
  QkArgs a{};
  a.part[0] = h;
  a.r = r;
  a.pos = pos;
  a.n_tok = n_tok;
  a.hd = hd;
  a.eps = eps;
  return launch_qk<false>(a, h.n_head, s);
}

hipError_t launch_kv4_append(const Kv4Args& c, const HeadArgs& q, const HeadArgs& k, const HeadArgs& v,
                             const RopeArgs& r, float eps, hipStream_t s) {
  QkArgs a{};
  a.c = c;
  a.part[0] = q;
  a.part[1] = k;
  a.part[2] = v;
  a.r = r;
  a.n_tok = c.n_tok;
  a.hd = c.hd;
  a.eps = eps;
  return launch_qk<true>(a, q.n_head + k.n_head + v.n_head, s);
}

hipError_t launch_kv4_read(const Kv4Args& c, float* K, float* V, hipStream_t s) {
  const int passes = (2 * c.n_kv * (c.hd / 8) + kThreads - 1) / kThreads;
  const int gx = std::min(c.n_tok, 1 << 20), gy = c.n_tok >= 1024 ? 1 : std::min(passes, 65535);
  hipLaunchKernelGGL(kv4_read_kernel, dim3(gx, gy), dim3(kThreads), 0, s, c, K, V);
  return hipGetLastError();
}

}  // namespace gq

// Rotary positions (RoPE) on caller tensors: pair (a, b) of a head at position p becomes
//   m (a cos w - b sin w),  m (b cos w + a sin w),   w = 2 pi p f_i,
// with f_i in turns per position and the magnitude m of the plan (struct dllm_rope).
//
// Precision. p f_i is reduced to a fraction of a turn in 64 bits (the product's rounding is
// recovered by an fma), so far positions lose nothing; m cos and m sin are rounded to 32
// bits once, and each product and sum of the rotation is rounded to 32 bits separately (no
// contraction), so the rotation has one result whichever kernel computes it: the cache's
// codes for a key do not depend on whether rope or append rotated it.
#pragma once

#include <algorithm>

#include "common.cuh"
#include "dllm.h"

namespace dllm {

struct RopeParams {
  int rd;                               // rotated dims of a head (0: none)
  int interleaved;                      // pairs (2 i, 2 i + 1) instead of (i, i + rd / 2)
  float sign;                           // -1: the transposed rotation
  double mag;
  double turns[DLLM_ROPE_MAX_PAIRS];
};

DLLM_DEV float2 rope_cos_sin(const RopeParams& r, int pos, int i) {
  const double f = r.turns[i];
  const double n = rint((double)pos * f);
  double s, c;
  sincospi(2.0 * fma((double)pos, f, -n), &s, &c);
  return make_float2((float)(r.mag * c), r.sign * (float)(r.mag * s));
}

DLLM_DEV float rope_first(float a, float b, float2 cs) { return __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y)); }
DLLM_DEV float rope_second(float a, float b, float2 cs) { return __fadd_rn(__fmul_rn(b, cs.x), __fmul_rn(a, cs.y)); }

// Round to nearest even that keeps NaN a NaN (f32_to_bf16 of common.cuh takes finite values).
DLLM_DEV bf16_t f32_to_bf16_any(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }

DLLM_DEV float load1(const float* p) { return *p; }
DLLM_DEV float load1(const bf16_t* p) { return bf16_to_f32(*p); }
DLLM_DEV void store1(float* p, float v) { *p = v; }
DLLM_DEV void store1(bf16_t* p, float v) { *p = f32_to_bf16_any(v); }

DLLM_DEV void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
DLLM_DEV void store8(bf16_t* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = (uint32_t)f32_to_bf16_any(v[2 * i]) | ((uint32_t)f32_to_bf16_any(v[2 * i + 1]) << 16);
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// How a block's threads divide up `tb` tokens of `units` units each (units of rope_kernel, code words
// of kv4_append_kernel): a thread keeps its unit, so that everything that depends on it is computed
// once, and walks over tokens. Small units per token: `tp` tokens side by side; many: `passes` times
// `threads` units.
struct TokenTiling {
  int units, tp, passes, tb;
};
constexpr int kTokenSteps = 8;   // tokens a thread takes, one after the other
inline __host__ __device__ int rope_stride(int rd) { return (rd / 4 + 8) / 8 * 8; }   // 16-byte chunks of a token's cos and sin, in eights
inline TokenTiling token_tiling(int units, int T, int rd, int sms, int* threads) {
  TokenTiling t;
  t.units = units;
  t.passes = (units + 511) / 512;
  t.tp = units <= 128 ? std::min(256 / units, 64) : 1;
  while (t.tp > 1 && (t.tp > T || t.tp * rope_stride(rd) * 16 > 32768)) t.tp /= 2;
  *threads = (units * t.tp + 32 * t.passes - 1) / (32 * t.passes) * 32;
  // few tokens: fewer steps rather than fewer blocks than SMs
  int steps = kTokenSteps;
  while (steps > 1 && ((long)t.tp * steps * sms > T || t.tp * steps * rope_stride(rd) * 16 > 32768)) steps /= 2;
  t.tb = t.tp * steps;
  return t;
}
constexpr int kMaxTokensPerBlock = 256;

// The tokens' cos and sin in shared memory, one 64-bit evaluation per token and pair, shared by all
// heads. Two pairs are a 16-byte chunk (c0, c1, s0, s1), the operands of two-value operations; chunk q
// of a token lies at q ^ (q / 8 % 8) of every eight, so that lanes which take 4 (or 2) chunks each, one
// after the other, read different banks (in order, four lanes met in each: half the kernel's shared
// memory time).
DLLM_DEV int rope_chunk(int q) { return q ^ ((q >> 3) & 7); }
DLLM_DEV void rope_fill(const RopeParams& r, const int32_t* __restrict__ pos, long t0, int nt, float4* cs) {
  const int half = r.rd / 2, stride = rope_stride(r.rd);
  for (int u = threadIdx.x; u < nt * half; u += blockDim.x) {
    const int t = u / half, i = u - t * half;
    const float2 v = rope_cos_sin(r, pos[t0 + t], i);
    float* at = reinterpret_cast<float*>(cs + t * stride + rope_chunk(i >> 1)) + (i & 1);
    at[0] = v.x;
    at[2] = v.y;
  }
}
DLLM_DEV float2 rope_pair(const float4* cs, int i) {
  const float* at = reinterpret_cast<const float*>(cs + rope_chunk(i >> 1)) + (i & 1);
  return make_float2(at[0], at[2]);
}

// Two fp32 operations in one instruction, each rounded by itself.
DLLM_DEV uint64_t pack_f32x2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
DLLM_DEV void unpack_f32x2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
DLLM_DEV uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
DLLM_DEV uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
DLLM_DEV uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// x = x cos + y sin (MINUS: x cos - y sin) for eight pairs from chunk q0 on, y being the partners.
template <int MINUS>
DLLM_DEV void rope_turn8(float (&x)[8], const float (&y)[8], const float4* cs, int q0) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 q = cs[rope_chunk(q0 + i)];
    float a0, a1, b0, b1;
    unpack_f32x2(mul_f32x2(pack_f32x2(x[2 * i], x[2 * i + 1]), pack_f32x2(q.x, q.y)), a0, a1);
    unpack_f32x2(mul_f32x2(pack_f32x2(y[2 * i], y[2 * i + 1]), pack_f32x2(q.z, q.w)), b0, b1);
    // one by one: the compiler joins a two-value product and a two-value sum to fused operations, in
    // spite of their .rn, and the rotation would have another rounding here than elsewhere
    x[2 * i] = MINUS ? __fsub_rn(a0, b0) : __fadd_rn(a0, b0);
    x[2 * i + 1] = MINUS ? __fsub_rn(a1, b1) : __fadd_rn(a1, b1);
  }
}

// Four interleaved pairs from chunk q0 on.
DLLM_DEV void rope_turn4(float (&x)[8], const float4* cs, int q0) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 q = cs[rope_chunk(q0 + i)];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float2 c = e ? make_float2(q.y, q.w) : make_float2(q.x, q.z);
      const float a = x[4 * i + 2 * e], b = x[4 * i + 2 * e + 1];
      x[4 * i + 2 * e] = rope_first(a, b, c);
      x[4 * i + 2 * e + 1] = rope_second(a, b, c);
    }
  }
}

// Eight values as they were loaded.
template <typename T>
struct Raw8;
template <>
struct Raw8<bf16_t> {
  uint4 a;
  DLLM_DEV void load(const bf16_t* p) { a = *reinterpret_cast<const uint4*>(p); }
  DLLM_DEV void flip(uint32_t sign) {   // sign: 0 or 0x80000000
    const uint32_t m = sign | (sign >> 16);
    a = make_uint4(a.x ^ m, a.y ^ m, a.z ^ m, a.w ^ m);
  }
  DLLM_DEV void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  DLLM_DEV void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  DLLM_DEV void flip(uint32_t sign) {
    float* v[8] = {&a.x, &a.y, &a.z, &a.w, &b.x, &b.y, &b.z, &b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) *v[i] = __uint_as_float(__float_as_uint(*v[i]) ^ sign);
  }
  DLLM_DEV void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

// Rotates tb tokens, all heads, in units of a head: VEC, 8 pairs (half layout), 8 elements
// (interleaved) or 8 dims that are only copied; otherwise one pair or one dim. A thread's next load
// is on its way while it works on the last one, the first while cos and sin are computed.
// 32768 tokens of 16 heads of 64 in bf16, half of each rotated: 31.3 us, 4.3 of 6.55 TB/s. Bound by issue (68% while
// SMs are busy) and the L1 pipe (67%), not by memory: the launch bounds leave the bf16 vector form 40 registers, and it
// spills 80 bytes a thread (fp32: 64 registers, 36 bytes); 2048 blocks are 2.3 waves. The bounds are for 512 threads,
// which only tokens of more than 128 units need. 64 tokens of 16 heads of 176 2.6 us, a launch's time.
// In place is fine: a unit reads everything it writes before writing it, and nothing else
// reads it.
template <typename TI, typename TO, bool VEC>
__global__ void __launch_bounds__(512, sizeof(TI) == 2 ? 3 : 2)
rope_kernel(const __grid_constant__ RopeParams r, const TI* x, long x_tok, long x_head,
            const int32_t* __restrict__ pos, int T, int head_units, int rot_units, TO* y, long y_tok, long y_head,
            TokenTiling tl) {
  extern __shared__ float4 cs_smem[];   // [tb][rope_stride]
  pdl_begin();
  const int half = r.rd / 2, stride = rope_stride(r.rd);
  const long t0 = (long)blockIdx.x * tl.tb;
  const int nt = (int)min((long)tl.tb, T - t0);
  const int tl0 = tl.tp > 1 ? threadIdx.x / tl.units : 0;
  const bool real = tl0 < tl.tp;
  bool filled = false;
  for (int unit = threadIdx.x - tl0 * tl.units; (unit < tl.units && real) || !filled; unit += blockDim.x) {
    const bool mine = unit < tl.units && real;
    const int h = unit / head_units, k = unit - h * head_units;
    const bool rot = k < rot_units;
    const bool pair = VEC && rot && !r.interleaved;
    const int d = VEC ? (rot ? 8 * k : r.rd + (k - rot_units) * 8) : 0;
    const TI* xs = x + (t0 + tl0) * x_tok + h * x_head + d;
    TO* ys = y + (t0 + tl0) * y_tok + h * y_head + d;
    const long x_step = tl.tp * x_tok, y_step = tl.tp * y_tok;
    Raw8<TI> a, b;
    if (VEC && mine && tl0 < nt) {
      a.load(xs);
      if (pair) b.load(xs + half);
    }
    if (!filled) {
      rope_fill(r, pos, t0, nt, cs_smem);
      __syncthreads();
      filled = true;
    }
    if (!mine) break;
    const float4* cs = cs_smem + tl0 * stride;
    if (VEC) {
      const int q0 = pair ? d / 2 : d / 4;
      for (int t = tl0; t < nt; t += tl.tp) {
        float v[8], w[8];
        a.get(v);
        if (pair) b.get(w);
        xs += x_step;
        if (t + tl.tp < nt) {
          a.load(xs);
          if (pair) b.load(xs + half);
        }
        if (pair) {
          float q[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) q[e] = v[e];
          rope_turn8<1>(v, w, cs, q0);
          rope_turn8<0>(w, q, cs, q0);
          store8(ys + half, w);
        } else if (rot) {
          rope_turn4(v, cs, q0);
        }
        store8(ys, v);
        ys += y_step;
        cs += tl.tp * stride;
      }
    } else {
      const int i0 = !rot ? r.rd + (k - rot_units) : r.interleaved ? 2 * k : k;
      const int i1 = !rot ? i0 : r.interleaved ? 2 * k + 1 : k + half;
      for (int t = tl0; t < nt; t += tl.tp) {
        const float p = load1(xs + i0), q = load1(xs + i1);
        if (rot) {
          const float2 c = rope_pair(cs, k);
          store1(ys + i0, rope_first(p, q, c));
          store1(ys + i1, rope_second(p, q, c));
        } else {
          store1(ys + i0, p);
        }
        xs += x_step;
        ys += y_step;
        cs += tl.tp * stride;
      }
    }
  }
}

}  // namespace dllm

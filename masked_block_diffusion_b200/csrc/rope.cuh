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

DLLM_DEV void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
DLLM_DEV void load8(const bf16_t* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
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

// One block rotates `tb` tokens, all heads. The block first computes the tokens' cos and
// sin (one 64-bit evaluation per token and pair, shared by all heads), then every thread
// takes units of a head: VEC, 8 pairs (half layout), 8 elements (interleaved) or 8 dims
// that are only copied; otherwise one pair or one dim.
// In place is fine: a unit reads everything it writes before writing it, and nothing else
// reads it.
template <typename TI, typename TO, bool VEC>
__global__ void __launch_bounds__(256)
rope_kernel(const __grid_constant__ RopeParams r, const TI* x, long x_tok, long x_head,
            const int32_t* __restrict__ pos, int T, int H, int hd, TO* y, long y_tok, long y_head, int tb) {
  extern __shared__ float2 cs_smem[];   // [tb][rd / 2]
  pdl_begin();
  const int half = r.rd / 2;
  const long t0 = (long)blockIdx.x * tb;
  const int nt = (int)min((long)tb, T - t0);
  for (int u = threadIdx.x; u < nt * half; u += blockDim.x) {
    const int t = u / half, i = u - t * half;
    cs_smem[u] = rope_cos_sin(r, pos[t0 + t], i);
  }
  __syncthreads();
  const int step = VEC ? 8 : 1;
  const int rot_units = VEC && r.interleaved ? r.rd / 8 : half / step;
  const int units = rot_units + (hd - r.rd) / step;
  const int total = nt * H * units;
  for (int u = threadIdx.x; u < total; u += blockDim.x) {
    const int row = u / units, k = u - row * units;
    const int t = row / H, h = row - t * H;
    const TI* xs = x + (t0 + t) * x_tok + h * x_head;
    TO* ys = y + (t0 + t) * y_tok + h * y_head;
    const float2* cs = cs_smem + t * half;
    if (VEC) {
      float a[8], b[8];
      if (k >= rot_units) {
        const int d = r.rd + (k - rot_units) * 8;
        load8(xs + d, a);
        store8(ys + d, a);
      } else if (r.interleaved) {
        load8(xs + 8 * k, a);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 c = cs[4 * k + i];
          b[2 * i] = rope_first(a[2 * i], a[2 * i + 1], c);
          b[2 * i + 1] = rope_second(a[2 * i], a[2 * i + 1], c);
        }
        store8(ys + 8 * k, b);
      } else {
        load8(xs + 8 * k, a);
        load8(xs + half + 8 * k, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 c = cs[8 * k + i];
          const float p = rope_first(a[i], b[i], c), q = rope_second(a[i], b[i], c);
          a[i] = p;
          b[i] = q;
        }
        store8(ys + 8 * k, a);
        store8(ys + half + 8 * k, b);
      }
    } else if (k >= rot_units) {
      const int d = r.rd + (k - rot_units);
      store1(ys + d, load1(xs + d));
    } else {
      const int i0 = r.interleaved ? 2 * k : k, i1 = r.interleaved ? 2 * k + 1 : k + half;
      const float a = load1(xs + i0), b = load1(xs + i1);
      store1(ys + i0, rope_first(a, b, cs[k]));
      store1(ys + i1, rope_second(a, b, cs[k]));
    }
  }
}

}  // namespace dllm

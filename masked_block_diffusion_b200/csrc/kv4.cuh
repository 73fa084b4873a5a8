// The paged 4-bit KV cache: its format, appending to it and reading it back.
//
// A page holds `page` positions of one layer:
//   codes  [n_pages][2 (K, V)][Hkv][page][hd / 2]    scales [n_pages][2][Hkv][page][hd / 16]
// Sixteen consecutive dims of a position share a scale byte, the upper eight bits of a
// positive fp16 number without its sign (5 exponent and 3 mantissa bits), at most 0xD2 =
// 2560, so that 24 * scale is finite in fp16 (the unpacking needs it). A dim's value is
// scale * (code - 8). Both factors are short (4 and 3 significant bits), so every value
// is exact in bf16 and in fp16: the attention kernels' operands carry no rounding of their
// own.
//
// Eight dims are one 32-bit word: dim 8 w + 2 j in nibble j, dim 8 w + 2 j + 1 in nibble
// j + 4. (word >> 4 j) & 0x000F000F is then an adjacent pair of dims in two 16-bit halves,
// which one OR turns into two floating-point numbers.
//
// Per position and head a page's codes lie together, as do its scales, so 16 positions (the
// smallest page) of one head are one contiguous copy of a multiple of 16 bytes.
#pragma once

#include "common.cuh"
#include "rope.cuh"

namespace dllm {

constexpr int kKv4MaxScale = 0xD2;

struct Kv4 {
  uint8_t* codes;
  uint8_t* scales;
  int n_pages, page_shift, Hkv, hd;
};

struct Kv4Addr {          // which rows of the cache a call's tokens are
  const int32_t* req;     // [T] row of the table, < 0: padding
  const int32_t* pos;     // [T] position
  const int32_t* table;   // [n_req][stride] page ids
  int n_req, stride;
};

DLLM_DEV float kv4_scale(int b) { return __half2float(__ushort_as_half((unsigned short)(b << 7))); }

// (page, offset in the page) of token t: page >= 0, -1 where nothing is stored there, -2 for padding.
DLLM_DEV int kv4_page_of(const Kv4& c, const Kv4Addr& a, long t, int& off) {
  const int r = a.req[t], p = a.pos[t];
  if (r < 0) return -2;
  const int col = p >> c.page_shift;
  off = p & ((1 << c.page_shift) - 1);
  if (r >= a.n_req || p < 0 || col >= a.stride) return -1;
  const int id = a.table[(long)r * a.stride + col];
  return id >= 0 && id < c.n_pages ? id : -1;
}

// Row index of (page id, K or V, head, offset): rows of hd / 2 code bytes and hd / 16 scale bytes.
DLLM_DEV long kv4_row(const Kv4& c, int id, int kv, int head, int off) {
  return ((((long)id * 2 + kv) * c.Hkv + head) << c.page_shift) + off;
}

// The group's scale byte: the least one with 7 * scale >= top, for 0 <= top <= 7 * 2560.
// That is top / 7 rounded up to a scale. The quotient correctly rounded to fp32 does as well as the
// exact one: a scale s has 4 significant bits, 7 s is exact, and the next fp32 number above 7 s
// is (at least 2^-21 / 7 = 1.14 * 2^-24 of s's binade) more than half a step of fp32 away
// from s after the division. Rounding up is an addition to the bits below the scale's; under 2^-14 the
// scales are 2^-17 apart, as they are just above 2^-14.
DLLM_DEV int kv4_scale_byte(float top) {
  const float seventh = 0x1.24924ap-3f;   // 1 / 7 correctly rounded; the quotient as in kv4_pack8
  const float q0 = __fmul_rn(top, seventh);
  const float q = __fmaf_rn(__fmaf_rn(-q0, 7.f, top), seventh, q0);
  const bool small = q < 0x1p-14f;
  const uint32_t bits = __float_as_uint(small ? __fadd_ru(q, 0x1p-14f) : q);
  return (int)((bits + 0xFFFFFu) >> 20) - (small ? 904 : 896);
}

// 1 / s of a scale, correctly rounded: the approximation improved by one Newton step (a test goes
// through all scales).
DLLM_DEV float kv4_reciprocal(float s) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
  return __fmaf_rn(__fmaf_rn(-s, y, 1.f), y, y);
}

DLLM_DEV float max_nan(float a, float b) {   // NaN if either is one
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Eight values, half of a group whose other half the neighbouring lane (lane ^ 1) has, to their code
// word and the group's scale byte. The code is the correctly rounded quotient v / s to the nearest
// integer, ties to even, + 8; beyond 7 scales saturates; NaN counts as 0.
// The quotient: with y = 1 / s correctly rounded, q0 = v y, q = q0 + (v - q0 s) y with fused
// operations is the correctly rounded v / s (Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990): three operations per value and one reciprocal
// per group instead of a division per value. Adding 1.5 * 2^23 rounds q to an integer in the
// number's low bits, and multiplying by 2^(4 nibble) adds it into the word; what the constant's own
// bits contribute is taken off the word's start value.
DLLM_DEV uint32_t kv4_pack8(float (&v)[8], int& byte) {
  float top = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) top = max_nan(top, fabsf(v[i]));
  top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
  if (!(top <= 7.f * 2560.f)) {   // saturation, infinities or NaN: values brought within the codes' range first
    top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = v[i] == v[i] ? fminf(fmaxf(v[i], -7.f * 2560.f), 7.f * 2560.f) : 0.f;
      top = fmaxf(top, fabsf(v[i]));
    }
    // the neighbour took this branch too: both lanes saw the same top
    top = fmaxf(top, __shfl_xor_sync(3u << (threadIdx.x & 30), top, 1));
  }
  byte = kv4_scale_byte(top);
  if (byte == 0) return 0x88888888u;
  const float s = kv4_scale(byte), y = kv4_reciprocal(s);
  const uint32_t magic = 0x4B400000u;   // 1.5 * 2^23
  uint32_t w = 0x88888888u;
#pragma unroll
  for (int i = 0; i < 8; ++i) w -= magic << (4 * (i >> 1) + 16 * (i & 1));
  const uint64_t yy = pack_f32x2(y, y), ms = pack_f32x2(-s, -s), round = pack_f32x2(12582912.f, 12582912.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t x = pack_f32x2(v[2 * i], v[2 * i + 1]);
    const uint64_t q0 = mul_f32x2(x, yy);
    float a, b;
    unpack_f32x2(add_f32x2(fma_f32x2(fma_f32x2(q0, ms, x), yy, q0), round), a, b);
    w += (__float_as_uint(a) << (4 * i)) + (__float_as_uint(b) << (4 * i + 16));
  }
  return w;
}

// Appends T tokens' keys (rotated on the way) and values. One block takes `tb` tokens: their
// cos and sin once; then a thread has 8 dims (a code word) of K or V of one token after the other, two
// neighbouring lanes a group, so that loads of 32 or 16 bytes and stores of 4 are contiguous along
// a warp. The loads of all its tokens go out first, before the page ids (two dependent loads) and the
// cos and sin are there; a rotated chunk's partner comes later, out of the L1 cache, where
// another thread's load has brought it. Bound by instruction issue (68% while SMs are busy): 10 600
// tokens of 8 heads of 176 in bf16, three prompts, 38 us (26 without rotation), 77 MB; 64 tokens 3.3 us.
// Part of the issue is work done twice: both lanes of a group find its scale, a rotated word is loaded by two threads, and at
// the launch bounds' 40 registers the bf16 vector form spills (36 bytes a thread at 176 dims, 20 at 64 and 128).
template <int HD, typename TI, bool VEC>
__global__ void __launch_bounds__(512, sizeof(TI) == 2 ? 3 : 2)
kv4_append_kernel(const __grid_constant__ RopeParams r, Kv4 c, Kv4Addr a, const TI* __restrict__ k, long k_tok,
                  long k_head, const TI* __restrict__ v, long v_tok, long v_head,
                  const int32_t* __restrict__ rope_pos, int T, TokenTiling tl) {
  extern __shared__ float4 cs_smem[];             // [tb][rope_stride]
  __shared__ long row_of[kMaxTokensPerBlock];     // the tokens' row in the cache (K, first head), -1: none
  constexpr int WORDS = HD / 8;
  pdl_begin();
  const int half = r.rd / 2, stride = rope_stride(r.rd);
  const long t0 = (long)blockIdx.x * tl.tb;
  const int nt = (int)min((long)tl.tb, T - t0);
  // lanes past the last word go along with it, since neighbours talk to each other
  const int tl0 = tl.tp > 1 ? min((int)threadIdx.x / tl.units, tl.tp - 1) : 0;
  for (int base = 0; base < tl.units; base += blockDim.x) {
    const int mine = threadIdx.x - tl0 * tl.units + base;
    const int unit = min(mine, tl.units - 2 + (mine & 1));
    const int row = unit / WORDS, w = unit - row * WORDS;     // row: K heads, then V heads
    const int d = 8 * w;
    const bool is_k = row < c.Hkv;
    const long x_step = tl.tp * (is_k ? k_tok : v_tok);
    const TI* xs = (is_k ? k + (t0 + tl0) * k_tok + row * k_head : v + (t0 + tl0) * v_tok + (row - c.Hkv) * v_head) + d;
    const bool rot = is_k && d < r.rd, pair = rot && !r.interleaved;
    const bool first = d < half;
    const int away = first ? half : -half;
    const int q0 = pair ? (first ? d : d - half) / 2 : d / 4;
    const uint32_t flip = first ? 0x80000000u : 0u;           // a cos - b sin in the first half, b cos + a sin in the second
    uint8_t* codes = c.codes + ((long)row << c.page_shift) * (HD / 2) + 4 * w;      // V's heads follow K's
    uint8_t* scales = c.scales + ((long)row << c.page_shift) * (HD / 16) + w / 2;
    const float4* cs = cs_smem + tl0 * stride;
    Raw8<TI> next;
    if (VEC && tl0 < nt) next.load(xs);
    if (base == 0) {
      for (int t = threadIdx.x; t < nt; t += blockDim.x) {
        int off = 0;
        const int id = kv4_page_of(c, a, t0 + t, off);
        row_of[t] = id < 0 ? -1 : kv4_row(c, id, 0, 0, off);
      }
      rope_fill(r, rope_pos, t0, nt, cs_smem);
      __syncthreads();
    }
    for (int step = 0; step < nt; step += tl.tp) {            // the same for the whole block
      const int t = tl0 + step;
      const long at = t < nt ? row_of[t] : -1;
      const Raw8<TI> raw = next;
      if (VEC && t + tl.tp < nt) next.load(xs + x_step);
      float x[8];
      if (at < 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.f;
      } else if (VEC) {
        raw.get(x);
        if (pair) {
          Raw8<TI> xb;
          float y[8];
          xb.load(xs + away);
          xb.flip(flip);
          xb.get(y);
          rope_turn8<0>(x, y, cs, q0);
        } else if (rot) {
          rope_turn4(x, cs, q0);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int dd = d + e;
          const float own = load1(xs + e);
          if (!is_k || dd >= r.rd) {
            x[e] = own;
          } else if (r.interleaved) {
            const float2 q = rope_pair(cs, dd >> 1);
            const float other = load1(xs + (dd & 1 ? e - 1 : e + 1));
            x[e] = dd & 1 ? rope_second(other, own, q) : rope_first(own, other, q);
          } else {
            const bool lo = dd < half;
            const float2 q = rope_pair(cs, lo ? dd : dd - half);
            const float other = load1(xs + e + (lo ? half : -half));
            x[e] = lo ? rope_first(own, other, q) : rope_second(other, own, q);
          }
        }
      }
      int byte;
      const uint32_t word = kv4_pack8(x, byte);
      if (at >= 0 && mine < tl.units) {
        *reinterpret_cast<uint32_t*>(codes + at * (HD / 2)) = word;
        if ((w & 1) == 0) scales[at * (HD / 16)] = (uint8_t)byte;
      }
      xs += x_step;
      cs += tl.tp * stride;
    }
  }
}

// Two bf16 values (adjacent dims) of nibble pair j of a code word. The nibble u goes to the
// mantissa bits of weight 1 of 16 + u (exponent 2^4, 7 mantissa bits); then
// (16 + u) s - 24 s = (u - 8) s, exact: 24 s has 6 significant bits and the product is
// not rounded inside the fma.
DLLM_DEV uint32_t kv4_bf16x2(uint32_t w, int j, __nv_bfloat162 s, __nv_bfloat162 ms24) {
  const uint32_t sh = j == 0 ? w << 3 : w >> (4 * j - 3);
  const uint32_t u = (sh & 0x00780078u) | 0x41804180u;
  const __nv_bfloat162 v = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&u), s, ms24);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The scale byte as bf16 in both halves: byte << 4 is scale * 2^-112 there (the exponent
// biases differ by 112), subnormal bytes included.
DLLM_DEV __nv_bfloat162 kv4_scale_bf16x2(uint32_t byte) {
  const uint32_t b = (byte << 4) * 0x00010001u;
  const uint32_t up = 0x77807780u;   // 2^112
  return __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&b), *reinterpret_cast<const __nv_bfloat162*>(&up));
}

// Reads T tokens' rows back as bf16 [T][Hkv][hd]. One warp per token, lanes along its groups of 16
// dims (K's heads, then V's), whose loads are all issued before the first is used. A token with no
// page reads NaN; a padding token's rows are zeroed or left as they are. Bound by its writes: 52 600
// positions of 8 heads of 176 80 us, 4.7 TB/s (a torch fill of what it writes takes 77 us).
template <int HD>
__global__ void __launch_bounds__(256)
kv4_read_kernel(Kv4 c, Kv4Addr a, int T, bf16_t* __restrict__ k_out, bf16_t* __restrict__ v_out, int zero_padding) {
  constexpr int G = HD / 16, UNROLL = 6;
  pdl_begin();
  const long t = (long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= T) return;
  const int lane = threadIdx.x & 31;
  int off = 0;
  const int id = kv4_page_of(c, a, t, off);
  if (id == -2 && !zero_padding) return;
  const int per_kv = c.Hkv * G;
  const int first = k_out != nullptr ? 0 : per_kv, last = v_out != nullptr ? 2 * per_kv : per_kv;
  const long row0 = id >= 0 ? kv4_row(c, id, 0, 0, off) : 0;
  for (int u0 = first + lane; u0 < last; u0 += 32 * UNROLL) {
    uint2 w[UNROLL];
    uint32_t b[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      const int u = u0 + 32 * i;
      if (u < last && id >= 0) {
        const int h = u / G, g = u - h * G;              // V's heads follow K's
        const long row = row0 + ((long)h << c.page_shift);
        w[i] = *reinterpret_cast<const uint2*>(c.codes + row * (HD / 2) + 8 * g);
        b[i] = c.scales[row * (HD / 16) + g];
      }
    }
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      const int u = u0 + 32 * i;
      if (u >= last) continue;
      uint32_t o[8];
      if (id < 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = id == -1 ? 0x7FC07FC0u : 0u;
      } else {
        const __nv_bfloat162 s = kv4_scale_bf16x2(b[i]);
        const __nv_bfloat162 ms24 = __hmul2(s, __float2bfloat162_rn(-24.f));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          o[j] = kv4_bf16x2(w[i].x, j, s, ms24);
          o[4 + j] = kv4_bf16x2(w[i].y, j, s, ms24);
        }
      }
      bf16_t* out = u < per_kv ? k_out + t * (c.Hkv * HD) + u * 16 : v_out + t * (c.Hkv * HD) + (u - per_kv) * 16;
      reinterpret_cast<uint4*>(out)[0] = make_uint4(o[0], o[1], o[2], o[3]);
      reinterpret_cast<uint4*>(out)[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

}  // namespace dllm

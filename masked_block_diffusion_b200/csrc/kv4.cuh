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

// The group's scale byte: the least one with 7 * scale >= top (0xD2 at most; top is not NaN).
DLLM_DEV int kv4_scale_byte(float top) {
  if (!(top > 0.f)) return 0;
  if (top >= 7.f * 2560.f) return kKv4MaxScale;
  // a guess from the quotient's bits, put right by exact products (7 * scale has 7 bits)
  int b = min((int)(__half_as_ushort(__float2half_rd(top * (1.f / 7.f))) >> 7), kKv4MaxScale);
  if (b > 0 && 7.f * kv4_scale(b - 1) >= top) --b;
  if (7.f * kv4_scale(b) < top) ++b;
  return b;
}

// Sixteen values to two code words and the scale byte. Nearest code, ties to even of the
// correctly rounded quotient; beyond 7 scales saturates; NaN counts as 0.
DLLM_DEV uint2 kv4_pack(const float (&v)[16], int& byte) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(v[i]));   // fmaxf drops a NaN
  byte = kv4_scale_byte(top);
  const float s = kv4_scale(byte);
  uint32_t w[2] = {0x88888888u, 0x88888888u};
  if (byte > 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w[h] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float q = fminf(fmaxf(rintf(__fdiv_rn(v[8 * h + i], s)), -7.f), 7.f);
        const uint32_t u = v[8 * h + i] == v[8 * h + i] ? (uint32_t)((int)q + 8) : 8u;
        w[h] |= u << (4 * (i >> 1) + 16 * (i & 1));
      }
    }
  }
  return make_uint2(w[0], w[1]);
}

// Sixteen dims d0 .. d0 + 15 of a head at xs, rotated by cs (null: as they are).
template <typename TI, bool VEC>
DLLM_DEV void kv4_load16(const TI* xs, int d0, const RopeParams& r, const float2* cs, float (&v)[16]) {
  const int half = r.rd / 2;
  if (VEC) {
    // rd and half are multiples of 8: each 8-dim chunk lies on one side of every border
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int d = d0 + 8 * h;
      float a[8];
      load8(xs + d, a);
      if (cs != nullptr && d < r.rd) {
        if (r.interleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 c = cs[d / 2 + i];
            v[8 * h + 2 * i] = rope_first(a[2 * i], a[2 * i + 1], c);
            v[8 * h + 2 * i + 1] = rope_second(a[2 * i], a[2 * i + 1], c);
          }
        } else {
          float b[8];
          const bool first = d < half;
          load8(xs + (first ? d + half : d - half), b);
          const float2* c = cs + (first ? d : d - half);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[8 * h + i] = first ? rope_first(a[i], b[i], c[i]) : rope_second(b[i], a[i], c[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * h + i] = a[i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int d = d0 + i;
      const float a = load1(xs + d);
      if (cs == nullptr || d >= r.rd) {
        v[i] = a;
      } else if (r.interleaved) {
        const float b = load1(xs + (d ^ 1));
        v[i] = d & 1 ? rope_second(b, a, cs[d >> 1]) : rope_first(a, b, cs[d >> 1]);
      } else {
        const bool first = d < half;
        const float b = load1(xs + (first ? d + half : d - half));
        v[i] = first ? rope_first(a, b, cs[d]) : rope_second(b, a, cs[d - half]);
      }
    }
  }
}

// Appends T tokens' keys (rotated on the way) and values. One block takes `tb` tokens: their
// cos and sin once, then one thread per 16-dim group of K or V.
template <typename TI, bool VEC>
__global__ void __launch_bounds__(256)
kv4_append_kernel(const __grid_constant__ RopeParams r, Kv4 c, Kv4Addr a, const TI* __restrict__ k, long k_tok,
                  long k_head, const TI* __restrict__ v, long v_tok, long v_head,
                  const int32_t* __restrict__ rope_pos, int T, int tb) {
  extern __shared__ float2 cs_smem[];   // [tb][rd / 2]
  pdl_begin();
  const int half = r.rd / 2;
  const long t0 = (long)blockIdx.x * tb;
  const int nt = (int)min((long)tb, T - t0);
  for (int u = threadIdx.x; u < nt * half; u += blockDim.x) {
    const int t = u / half, i = u - t * half;
    if (a.req[t0 + t] >= 0) cs_smem[u] = rope_cos_sin(r, rope_pos[t0 + t], i);
  }
  __syncthreads();
  const int groups = c.hd / 16;
  const int per_tok = 2 * c.Hkv * groups;
  for (int u = threadIdx.x; u < nt * per_tok; u += blockDim.x) {
    const int t = u / per_tok;
    int rest = u - t * per_tok;
    const int g = rest % groups;
    rest /= groups;
    const int kv = rest / c.Hkv, h = rest - kv * c.Hkv;
    int off;
    const int id = kv4_page_of(c, a, t0 + t, off);
    if (id < 0) continue;
    float x[16];
    if (kv == 0)
      kv4_load16<TI, VEC>(k + (t0 + t) * k_tok + h * k_head, 16 * g, r, r.rd > 0 ? cs_smem + t * half : nullptr, x);
    else
      kv4_load16<TI, VEC>(v + (t0 + t) * v_tok + h * v_head, 16 * g, r, nullptr, x);
    int byte;
    const uint2 w = kv4_pack(x, byte);
    const long row = kv4_row(c, id, kv, h, off);
    *reinterpret_cast<uint2*>(c.codes + row * (c.hd / 2) + 8 * g) = w;
    c.scales[row * (c.hd / 16) + g] = (uint8_t)byte;
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

// Reads T tokens' rows back as bf16 [T][Hkv][hd]: one thread per 16-dim group. A token
// with no page reads NaN; a padding token's rows stay as they are.
__global__ void __launch_bounds__(256)
kv4_read_kernel(Kv4 c, Kv4Addr a, long T, bf16_t* __restrict__ k_out, bf16_t* __restrict__ v_out) {
  pdl_begin();
  const int groups = c.hd / 16;
  const long per_kv = T * c.Hkv * groups;
  const long u = (long)blockIdx.x * blockDim.x + threadIdx.x;
  if (u >= per_kv) return;
  const int kv = blockIdx.y;
  bf16_t* out = kv ? v_out : k_out;
  if (out == nullptr) return;
  const long row_out = u / groups;
  const int g = (int)(u - row_out * groups);
  const long t = row_out / c.Hkv;
  const int h = (int)(row_out - t * c.Hkv);
  int off = 0;
  const int id = kv4_page_of(c, a, t, off);
  if (id == -2) return;
  uint32_t o[8];
  if (id < 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = 0x7FC07FC0u;
  } else {
    const long row = kv4_row(c, id, kv, h, off);
    const uint2 w = *reinterpret_cast<const uint2*>(c.codes + row * (c.hd / 2) + 8 * g);
    const __nv_bfloat162 s = kv4_scale_bf16x2(c.scales[row * (c.hd / 16) + g]);
    const __nv_bfloat162 ms24 = __hmul2(s, __float2bfloat162_rn(-24.f));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o[j] = kv4_bf16x2(w.x, j, s, ms24);
      o[4 + j] = kv4_bf16x2(w.y, j, s, ms24);
    }
  }
  uint4* dst = reinterpret_cast<uint4*>(out + row_out * c.hd + 16 * g);
  dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
  dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

}  // namespace dllm

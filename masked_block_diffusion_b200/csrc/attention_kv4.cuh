// Attention over the paged 4-bit KV cache for few query rows per KV head (single tokens, a
// few tokens to verify, small canvases), and the merge of key splits. What both attention kernels share is here.
//
// Row R of request b and KV head g is query R / group, head g * group + R % group. Row R
// sees the keys below lim = kv_len (causal: kv_len - n + R / group + 1 for n queries):
//   s_t = scale * q . k_t,   o = sum_t e^(s_t - m) v_t / sum_t e^(s_t - m),   lse = m + log(sum).
// A row that sees no key has o = 0 and lse = -inf.
//
// With few rows the packed cache's bytes bound the time, if unpacking them does not: both
// products are taken transposed, S^T = K Q^T and O^T = V^T P^T, so that the packed operand
// fills the 16-row side of mma.m16n8k16 and eight query rows its 8-column side. (The 5th-
// generation tensor instruction reads its operands from shared or tensor memory only; with
// rows this few, writing the unpacked values there and reading them back would cost more
// than the multiplication.) Unpacking is what costs, mostly on the integer pipe: per word of eight
// codes two shifts, four AND-ORs and four exact fmas (kv4_sixteenth). Both operands are unpacked to
// sixteenths of their values in fp16, for which two nibbles need one shift; Q goes to fp16 with a
// power of two per row that keeps its largest value near the top of the range (a bf16 value
// has 8 bits, fp16 11, so only values 2^-28 of the row's largest lose any). Thread (r, c) =
// (lane / 4, lane % 4):
//   K: token r's and token r + 8's dims 64 i + 16 c .. + 15 (8 code bytes and their scale) are
//      its A fragments of four k16 steps; Q's fragments carry the same dims.
//   V: tokens 2c, 2c + 1, 2c + 8, 2c + 9, dims 8 w .. 8 w + 7 with w = 8 i + r: a byte permute
//      pairs two tokens' words, and nibble pair j gives the two tokens' dim 8 w + 2 j (+ 1).
// P is rounded to fp16 (11 bits) for O^T; the running maximum is kept 6 octaves low, so that
// P up to 2^14 uses fp16's range and weights down to 2^-30 of the largest survive. Scores,
// sums and accumulators are fp32.
// Measured: one token of 64 requests over up to 4352 keys (16 heads, 8 KV heads of 176) 111 us, 3.0 TB/s of packed
// cache; two tokens over 131072 keys (16 heads, 4 KV heads of 64) 37.1 us, 1.8 TB/s; one token over 4352
// keys 12.4 us with the join. Issue (59% while SMs are busy) and the latency of dependent instructions with
// 16 warps per SM bound the long calls.
#pragma once

#include "common.cuh"
#include "attention_tc.cuh"
#include "kv4.cuh"

namespace dllm {

constexpr float kKv4Low = 6.f;    // the softmax reference lies this many octaves below the maximum seen

struct AttnKv4Params {
  Kv4 c;
  const bf16_t* q;
  long q_tok, q_head;
  bf16_t* out;
  long o_tok, o_head;
  float* lse;               // [T][H] or null
  const int* q_start;       // [B + 1]
  const int* kv_len;        // [B]
  const int* table;         // [B][stride]
  int stride, B, T, H, group;
  int max_q, max_kv, causal;
  int n_splits;             // few rows: blocks that a request's keys are shared out to, in equal parts
  float scale_log2;         // scale * log2(e)
  float* part_o;            // [n_splits][T][H][hd]
  float* part_lse;          // [n_splits][T][H], log2 domain
  // On tcgen05 instead, two per block of the grid: part_o [2 blocks][hd / 4][256 rows][4], part_lse [2 blocks][256], and
  // parts[i] = (request, KV head, tile, 1: goes on in the next block, 2: ends here; 0: no such part)
  int4* parts;
  int cut;                  // 0: tiles stay whole, and there are no parts
  int unit_shift;           // Kv4Walk
  uint32_t mask_low, mask_high;   // Kv4Masks
  uint32_t mask_bf16;             // 0x00780078
};

// The largest score for which the reference m may stay: its weight is 2^14. Rounded down, since where numbers
// are 16 apart m + 14 would become m + 16, and a weight of 2^16 is infinite in fp16.
DLLM_DEV float kv4_above(float m) { return __fadd_rd(m, kKv4Low + 8.f); }

// A request's queries and keys. bad: its row range holds, but not its lengths: every row becomes NaN.
struct Kv4Req {
  int q0, n, kv;
  bool skip, bad;
};

DLLM_DEV Kv4Req kv4_request(const AttnKv4Params& p, int b) {
  Kv4Req r;
  r.q0 = p.q_start[b];
  const int q1 = p.q_start[b + 1];
  r.kv = p.kv_len[b];
  r.skip = r.q0 < 0 || q1 < r.q0 || q1 > p.T;
  r.n = r.skip ? 0 : q1 - r.q0;
  const long room = (long)p.stride << p.c.page_shift;
  r.bad = r.n > p.max_q || r.kv < 0 || r.kv > p.max_kv || r.kv > room;
  return r;
}

// Row R's keys end here.
DLLM_DEV int kv4_row_limit(const AttnKv4Params& p, const Kv4Req& r, int query) {
  return p.causal ? max(0, min(r.kv, r.kv - r.n + query + 1)) : r.kv;
}

// Every row of a bad request's head range [h0, h0 + nh) becomes NaN: 8, 16 or 32 lanes a row, 16 bytes each, by thread
// `first` of `step` (whole warps). Other warps of the block may wait meanwhile for its next tile, and a bad request may
// have as many rows as the call, so this must not take long: 240 000 rows of 2 heads of 176 9.9 ms, 17 GB/s from
// one block, of which the limit of those waits (2 s) leaves room for 34 GB per KV head (123 ms with two bytes a thread and
// divisions for each, where 3 GB were too many).
template <int HD>
DLLM_DEV void kv4_poison(const AttnKv4Params& p, const Kv4Req& r, int h0, int nh, int first, int step) {
  constexpr int LANES = HD <= 64 ? 8 : HD <= 128 ? 16 : 32;
  const unsigned rows = (unsigned)r.n * nh, by = step / LANES;   // at most T H, below 2^31
  const unsigned by_i = by / nh, by_h = by - by_i * nh;
  unsigned row = first / LANES, i = row / nh, h = row - i * nh;
  const int d = 8 * (first % LANES);
  const uint4 nan = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
#pragma unroll 1
  for (; row < rows; row += by) {
    const long t = r.q0 + (long)i;
    if (d < HD) *reinterpret_cast<uint4*>(p.out + t * p.o_tok + (h0 + (int)h) * p.o_head + d) = nan;
    if (d == 0 && p.lse != nullptr) p.lse[t * p.H + h0 + h] = __int_as_float(0x7FC00000);
    i += by_i;
    h += by_h;
    if (h >= (unsigned)nh) {
      h -= nh;
      ++i;
    }
  }
}

DLLM_DEV void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"((uint64_t)__cvta_generic_to_global(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

DLLM_DEV void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit values held two per thread.
DLLM_DEV uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

DLLM_DEV __half2 kv4_half2(uint32_t bits) { return *reinterpret_cast<const __half2*>(&bits); }

// The four nibble pairs of a code word as sixteenths, pair j holding dims 2 j and 2 j + 1 (or two keys'
// same dim). A nibble u at bits 2..5 of an fp16 number of exponent 2^4 is 16 + u / 16, at bits 6..9
// of one of exponent 2^0 it is 1 + u / 16, so one shift serves two neighbouring nibbles; then
// (16 + u / 16) s - 16.5 s = (u - 8) s / 16, and likewise with 1.5 s: exact, since 16.5 s and 1.5 s
// have at most 10 bits and the fma rounds once (scales up to 2560: 16.5 s < 65504).
struct Kv4Scale2 {
  __half2 s, m16, m1;   // the scale, -16.5 and -1.5 times it
};
// (a & mask) | bits in one operation. An instruction takes one constant: the masks come as kernel
// parameters, which the compiler keeps in registers, where with two constants it splits the operation.
template <uint32_t BITS>
DLLM_DEV uint32_t and_or(uint32_t a, uint32_t mask) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(mask), "n"(BITS));
  return d;
}
struct Kv4Masks {
  uint32_t low, high;   // 0x003C003C, 0x03C003C0
};
DLLM_DEV Kv4Scale2 kv4_scale2(uint32_t bits) {
  Kv4Scale2 r;
  r.s = kv4_half2(bits);
  r.m16 = __hmul2(r.s, __float2half2_rn(-16.5f));
  r.m1 = __hmul2(r.s, __float2half2_rn(-1.5f));
  return r;
}
DLLM_DEV void kv4_sixteenth(uint32_t w, const Kv4Scale2& s, const Kv4Masks& m, uint32_t (&o)[4]) {
  const uint32_t a = w * 4, b = w >> 6;   // (bits of the other half that a shift brings along are masked)
  const uint32_t u[4] = {and_or<0x4C004C00u>(a, m.low), and_or<0x3C003C00u>(a, m.high), and_or<0x4C004C00u>(b, m.low),
                         and_or<0x3C003C00u>(b, m.high)};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2 v = __hfma2(kv4_half2(u[j]), s.s, j & 1 ? s.m1 : s.m16);
    o[j] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

// Shared memory of a block: `STAGES` stages of 128 keys' packed K and V, 32 keys for each of four
// warps. Each warp has two 16-key tiles under way at a time, which are independent until the products
// with V. The first warp also issues the copies, so that no warp's registers are spent on that
// alone and four blocks of one 8-row column share an SM; they hold 100 KB of copies in flight.
template <int HD, int NR>
struct AttnKv4Cfg {
  static constexpr int KEYS = 128;
  static constexpr int WARPS = 4;
  static constexpr int TILES = KEYS / WARPS / 16;
  static constexpr int kCodes = KEYS * HD / 2;
  static constexpr int kScales = KEYS * HD / 16;
  static constexpr int kStage = 2 * (kCodes + kScales);
  static constexpr int STAGES = HD == 64 ? 4 : 2;
  static constexpr int kRows = 8 * NR;
  static constexpr int kRed = WARPS * kRows * (HD + 2) * 4;     // the warps' results, over the stages
  static constexpr int kBody = STAGES * kStage > kRed ? STAGES * kStage : kRed;
  static constexpr int kOffBar = (kBody + 15) / 16 * 16;
  static constexpr int kTotal = kOffBar + 2 * STAGES * 8 + 16;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int BLOCKS = NR == 1 ? 4 : HD == 176 ? 2 : 3;   // per SM
};

// Grid (n_splits, Hkv * row tiles, B). A block takes 8 NR rows of one KV head over one split.
template <int HD, int NR>
__global__ void __launch_bounds__(AttnKv4Cfg<HD, NR>::THREADS, AttnKv4Cfg<HD, NR>::BLOCKS)
attn_kv4_kernel(const __grid_constant__ AttnKv4Params p) {
  using G = AttnKv4Cfg<HD, NR>;
  constexpr int KI = (HD + 63) / 64;
  constexpr int WORDS = HD / 8;
  constexpr int TI = G::TILES;
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::kOffBar);
  uint64_t* empty = full + G::STAGES;
  volatile int* flags = reinterpret_cast<volatile int*>(empty + G::STAGES);   // [0] abort, [1] a page that is none

  pdl_begin();
  const int g = blockIdx.y % p.c.Hkv, tile = blockIdx.y / p.c.Hkv, sp = blockIdx.x, b = blockIdx.z;
  const Kv4Req rq = kv4_request(p, b);
  const int R0 = tile * G::kRows, n_rows = rq.n * p.group;
  if (rq.skip) return;
  if (rq.bad) {
    if (tile == 0 && sp == 0) kv4_poison<HD>(p, rq, g * p.group, p.group, threadIdx.x, blockDim.x);
    return;
  }
  if (R0 >= n_rows) return;
  const int last = min(n_rows - 1, R0 + G::kRows - 1);
  // equal splits of the request's own keys, in whole stages: max_kv may lie far above them
  const int chunk = max(1, ((rq.kv + p.n_splits - 1) / p.n_splits + G::KEYS - 1) / G::KEYS) * G::KEYS;
  const int ks = sp * chunk;
  const int ke = min(kv4_row_limit(p, rq, last / p.group), ks + chunk);
  const int nst = ke > ks ? (ke - ks + G::KEYS - 1) / G::KEYS : 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < G::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], G::WARPS);
    }
    flags[0] = flags[1] = 0;
    fence_mbar_init();
  }
  __syncthreads();

  // Copies stage `it` (first warp): lane i takes piece i, a page's share of it. False if its stage did
  // not come free. The page ids of a stage are asked for when the one before is copied.
  const int shift = min(p.c.page_shift, 7), keys = 1 << shift;
  auto piece = [&](int t) -> bool { return lane < (G::KEYS >> shift) && t < ke; };
  auto ask = [&](int it) -> int {
    const int t = ks + it * G::KEYS + lane * keys;
    return piece(t) ? p.table[(long)b * p.stride + (t >> p.c.page_shift)] : 0;
  };
  int id_next = warp == 0 ? ask(0) : 0;
  auto copy_stage = [&](int it) -> bool {
    const int t = ks + it * G::KEYS + lane * keys;
    int id = piece(t) ? id_next : -1;
    if (piece(t) && (id < 0 || id >= p.c.n_pages)) {
      id = -1;
      flags[1] = 1;
    }
    id_next = ask(it + 1);
    const uint32_t codes = keys * (HD / 2), scales = keys * (HD / 16);
    const uint32_t n = __popc(__ballot_sync(0xffffffffu, id >= 0));
    const int st = it % G::STAGES;
    if (!__all_sync(0xffffffffu, mbar_wait(&empty[st], ((it / G::STAGES) & 1) ^ 1, flags))) return false;
    if (lane == 0) mbar_arrive_expect_tx(&full[st], n * 2 * (codes + scales));
    __syncwarp();
    if (id >= 0) {
      uint8_t* dst = smem + st * G::kStage;
      const int off = t & ((1 << p.c.page_shift) - 1);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const long r = kv4_row(p.c, id, kv, g, off);
        uint8_t* d = dst + kv * (G::kCodes + G::kScales);
        bulk_load(d + lane * codes, p.c.codes + r * (HD / 2), codes, &full[st]);
        bulk_load(d + G::kCodes + lane * scales, p.c.scales + r * (HD / 16), scales, &full[st]);
      }
    }
    __syncwarp();
    return true;
  };
  int copied = 0;
  bool ok = true;
  if (warp == 0)
    while (copied < min(nst, G::STAGES) && (ok = copy_stage(copied))) ++copied;

  const int r = lane >> 2, c = lane & 3;
  uint32_t qf[NR][KI][8];               // fp16, scaled by a power of two per row
  int lim[NR][2];                       // columns 2c, 2c + 1: keys the row sees end here
  float fac[NR][2];                     // and what turns their sums into log2 weights
  float m[NR][2], l[NR][2];
  float o[NR][KI][4][4];
#pragma unroll
  for (int nr = 0; nr < NR; ++nr) {
    const int R = R0 + 8 * nr + r;
    const bool real = R < n_rows;
    const bf16_t* qr = p.q + (long)(rq.q0 + (real ? R / p.group : 0)) * p.q_tok + (g * p.group + (real ? R % p.group : 0)) * p.q_head;
#pragma unroll
    for (int i = 0; i < KI; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int d = 64 * i + 16 * c + 8 * h;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (real && d < HD) v = *reinterpret_cast<const uint4*>(qr + d);
        qf[nr][i][4 * h] = v.x;
        qf[nr][i][4 * h + 1] = v.y;
        qf[nr][i][4 * h + 2] = v.z;
        qf[nr][i][4 * h + 3] = v.w;
      }
    // the row's largest magnitude to [2^14, 2^15): bf16 bits compare like their magnitudes
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < KI; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, max(qf[nr][i][e] & 0x7FFFu, (qf[nr][i][e] >> 16) & 0x7FFFu));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // exponent field e: times 2^(141 - e), in two factors that are normal numbers for every e
    const int up = 141 - max((int)(top >> 7), 15);          // -114 .. 126
    const float scale_q = __uint_as_float((uint32_t)(127 + up) << 23);
#pragma unroll
    for (int i = 0; i < KI; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const __half2 v = __floats2half2_rn(__uint_as_float(qf[nr][i][e] << 16) * scale_q,
                                            __uint_as_float(qf[nr][i][e] & 0xFFFF0000u) * scale_q);
        qf[nr][i][e] = *reinterpret_cast<const uint32_t*>(&v);
      }
    const float down = __uint_as_float((uint32_t)(127 - up) << 23);   // 2^-up: normal
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int Rc = R0 + 8 * nr + 2 * c + e;
      lim[nr][e] = Rc < n_rows ? min(ke, kv4_row_limit(p, rq, Rc / p.group)) : 0;
      fac[nr][e] = __shfl_sync(0xffffffffu, down, 4 * (2 * c + e)) * 16.f * p.scale_log2;
      m[nr][e] = -INFINITY;
      l[nr][e] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < KI; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nr][i][j][e] = 0.f;
  }

  const int all_see = min(ke, kv4_row_limit(p, rq, R0 / p.group));   // every row of the tile sees the keys below
  const bool rows_full = R0 + G::kRows <= n_rows;
  const Kv4Masks masks{p.mask_low, p.mask_high};
  for (int it = 0; it < nst && ok; ++it) {
    const int st = it % G::STAGES;
    // the stage that was read last is filled again while this one is being read
    if (warp == 0 && it > 0 && copied < nst) {
      ok = copy_stage(copied);
      if (!ok) break;
      ++copied;
    }
    if (!__all_sync(0xffffffffu, mbar_wait(&full[st], (it / G::STAGES) & 1, flags))) { ok = false; break; }
    const int t0 = ks + it * G::KEYS + 16 * TI * warp;
    if (t0 < ke) {
      const uint8_t* kc = smem + st * G::kStage + 16 * TI * warp * (HD / 2);
      const uint8_t* kS = smem + st * G::kStage + G::kCodes + 16 * TI * warp * (HD / 16);
      const uint8_t* vc = kc + G::kCodes + G::kScales;
      const uint8_t* vS = kS + G::kCodes + G::kScales;
      float s[TI][NR][4];
#pragma unroll
      for (int u = 0; u < TI; ++u)
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[u][nr][e] = 0.f;
#pragma unroll
      for (int i = 0; i < KI; ++i) {
        const int grp = 4 * i + c;
        const bool in = 64 * (i + 1) <= HD || 16 * grp < HD;
#pragma unroll
        for (int u = 0; u < TI; ++u) {
          const int ra = 16 * u + r, rb = ra + 8;
          uint2 wa = make_uint2(0, 0), wb = wa;
          uint32_t ba = 0, bb = 0;
          if (in) {
            wa = *reinterpret_cast<const uint2*>(kc + ra * (HD / 2) + 8 * grp);
            wb = *reinterpret_cast<const uint2*>(kc + rb * (HD / 2) + 8 * grp);
            ba = kS[ra * (HD / 16) + grp];
            bb = kS[rb * (HD / 16) + grp];
          }
          const Kv4Scale2 sa = kv4_scale2(ba * 0x00800080u), sb = kv4_scale2(bb * 0x00800080u);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t xa[4], xb[4];
            kv4_sixteenth(h ? wa.y : wa.x, sa, masks, xa);
            kv4_sixteenth(h ? wb.y : wb.x, sb, masks, xb);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t a[4] = {xa[2 * k], xb[2 * k], xa[2 * k + 1], xb[2 * k + 1]};
#pragma unroll
              for (int nr = 0; nr < NR; ++nr)
                mma_f16_16816(s[u][nr], a, qf[nr][i][4 * h + 2 * k], qf[nr][i][4 * h + 2 * k + 1]);
            }
          }
        }
      }
      uint32_t pf[TI][NR][2];
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int u = 0; u < TI; ++u) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[u][nr][e] *= fac[nr][e & 1];
          if (t0 + 16 * TI > all_see || !rows_full) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (t0 + 16 * u + r + 8 * (e >> 1) >= lim[nr][e & 1]) s[u][nr][e] = -INFINITY;
          }
          mx0 = fmaxf(mx0, fmaxf(s[u][nr][0], s[u][nr][2]));
          mx1 = fmaxf(mx1, fmaxf(s[u][nr][1], s[u][nr][3]));
        }
        // a new reference only when a score is more than 2^14 above it (the first visible key always is)
        if (__any_sync(0xffffffffu, mx0 > kv4_above(m[nr][0]) || mx1 > kv4_above(m[nr][1]))) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = e ? mx1 : mx0;
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float mn = fmaxf(m[nr][e], mx - kKv4Low);
            f[e] = mn == -INFINITY ? 1.f : exp2f(m[nr][e] - mn);
            m[nr][e] = mn;
            l[nr][e] *= f[e];
          }
#pragma unroll
          for (int i = 0; i < KI; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[nr][i][j][e] *= f[e & 1];
        }
        const float b0 = m[nr][0] == -INFINITY ? 0.f : m[nr][0], b1 = m[nr][1] == -INFINITY ? 0.f : m[nr][1];
#pragma unroll
        for (int u = 0; u < TI; ++u) {
          const float p0 = ex2_approx(s[u][nr][0] - b0), p1 = ex2_approx(s[u][nr][1] - b1);
          const float p2 = ex2_approx(s[u][nr][2] - b0), p3 = ex2_approx(s[u][nr][3] - b1);
          l[nr][0] += p0 + p2;
          l[nr][1] += p1 + p3;
          const __half2 h01 = __floats2half2_rn(p0, p1), h23 = __floats2half2_rn(p2, p3);
          pf[u][nr][0] = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&h01));
          pf[u][nr][1] = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&h23));
        }
      }
      const bool tail = t0 + 16 * TI > ke;   // keys past the end: what their bytes hold is not used, not even times 0
#pragma unroll
      for (int i = 0; i < KI; ++i) {
        const int w = 8 * i + r;
        const bool in = 8 * (i + 1) <= WORDS || w < WORDS;
#pragma unroll
        for (int u = 0; u < TI; ++u) {
          uint32_t x[4] = {0, 0, 0, 0}, sc[4] = {0, 0, 0, 0};
          if (in) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int t = 16 * u + 2 * c + (e & 1) + 8 * (e >> 1);
              x[e] = *reinterpret_cast<const uint32_t*>(vc + t * (HD / 2) + 4 * w);
              sc[e] = vS[t * (HD / 16) + w / 2];
            }
          }
          if (tail) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (t0 + 16 * u + 2 * c + (e & 1) + 8 * (e >> 1) >= ke) sc[e] = 0;
          }
          const Kv4Scale2 s0 = kv4_scale2((sc[1] * 65536u + sc[0]) * 128u), s1 = kv4_scale2((sc[3] * 65536u + sc[2]) * 128u);
          uint32_t e0[4], d0[4], e1[4], d1[4];   // even and odd dims of the two pairs of tokens
          kv4_sixteenth(__byte_perm(x[0], x[1], 0x5410), s0, masks, e0);
          kv4_sixteenth(__byte_perm(x[0], x[1], 0x7632), s0, masks, d0);
          kv4_sixteenth(__byte_perm(x[2], x[3], 0x5410), s1, masks, e1);
          kv4_sixteenth(__byte_perm(x[2], x[3], 0x7632), s1, masks, d1);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t a[4] = {e0[j], d0[j], e1[j], d1[j]};
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) mma_f16_16816(o[nr][i][j], a, pf[u][nr][0], pf[u][nr][1]);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
  }
  if (!ok) flags[0] = 1;
  // whatever became of the waits, the copies already issued land before the stages are used otherwise
  if (warp == 0)
    for (int i = max(0, copied - G::STAGES); i < copied; ++i) mbar_drain(&full[i % G::STAGES], (i / G::STAGES) & 1);
  __syncthreads();   // every copy has landed and every stage is read: the stages' memory is free
  // ---------------- each warp's reference, sum and O of its rows
  float* red = reinterpret_cast<float*>(smem) + warp * G::kRows * (HD + 2);
#pragma unroll
  for (int nr = 0; nr < NR; ++nr)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float sum = l[nr][e];
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      float* row = red + (8 * nr + 2 * c + e) * (HD + 2);
      if (r == 0) {
        row[HD] = m[nr][e];
        row[HD + 1] = sum;
      }
#pragma unroll
      for (int i = 0; i < KI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (8 * i + r < WORDS)
            *reinterpret_cast<float2*>(row + 8 * (8 * i + r) + 2 * j) = make_float2(o[nr][i][j][e], o[nr][i][j][2 + e]);
    }
  __syncthreads();
  // ---------------- the warps' results joined
  const bool lost = flags[0] != 0 || flags[1] != 0;
  const float* all = reinterpret_cast<const float*>(smem);
  for (int u = threadIdx.x; u < G::kRows * (HD / 2); u += G::THREADS) {
    const int rr = u / (HD / 2), d = 2 * (u - rr * (HD / 2));
    const int R = R0 + rr;
    if (R >= n_rows) continue;
    float mw[G::WARPS], mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < G::WARPS; ++w) {
      mw[w] = all[(w * G::kRows + rr) * (HD + 2) + HD];
      mx = fmaxf(mx, mw[w]);
    }
    float sum = 0.f, a0 = 0.f, a1 = 0.f;
#pragma unroll
    for (int w = 0; w < G::WARPS; ++w) {
      const float* row = all + (w * G::kRows + rr) * (HD + 2);
      if (row[HD + 1] == 0.f) continue;   // no key seen
      // a reference at -inf with a sum: every score was NaN, and so is the sum
      const float f = mw[w] == -INFINITY ? 1.f : exp2f(mw[w] - mx);
      sum += f * row[HD + 1];
      a0 += f * row[d];
      a1 += f * row[d + 1];
    }
    const float inv = sum == 0.f ? 0.f : 16.f / sum;   // V came in sixteenths
    float lse2 = sum == 0.f ? -INFINITY : mx + log2f(sum);
    a0 *= inv;
    a1 *= inv;
    if (lost) a0 = a1 = lse2 = __int_as_float(0x7FC00000);
    const long t = rq.q0 + R / p.group;
    const int h = g * p.group + R % p.group;
    if (p.n_splits == 1) {
      *reinterpret_cast<uint32_t*>(p.out + t * p.o_tok + h * p.o_head + d) =
          (uint32_t)f32_to_bf16_any(a0) | ((uint32_t)f32_to_bf16_any(a1) << 16);
      if (d == 0 && p.lse != nullptr) p.lse[t * p.H + h] = lse2 * 0.6931471805599453f;
    } else {
      const long at = ((long)sp * p.T + t) * p.H + h;
      *reinterpret_cast<float2*>(p.part_o + at * HD + d) = make_float2(a0, a1);
      if (d == 0) p.part_lse[at] = lse2;
    }
  }
}

// Joins the splits of one query and head per block: grid (max_q * H, B). Every split of every row
// has written its partial (0 with lse = -inf where it saw no key), so the loads depend on nothing:
// warp w takes splits w, w + 4, ... with all lanes' loads in flight, and the warps' sums are added in
// shared memory. (One warp per head that looked at each split's lse first took 20 us for 34 splits.)
template <int HD>
__global__ void __launch_bounds__(128)
attn_kv4_merge_kernel(const __grid_constant__ AttnKv4Params p) {
  constexpr int VI = (HD + 63) / 64;
  __shared__ float sh[4][HD + 2];
  pdl_begin();
  const int i = blockIdx.x / p.H, h = blockIdx.x - i * p.H;
  const Kv4Req rq = kv4_request(p, blockIdx.y);
  if (rq.skip || rq.bad || i >= rq.n) return;
  const long t = rq.q0 + i;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float* lse = p.part_lse + t * p.H + h;
  const float* po = p.part_o + (t * p.H + h) * HD + 2 * lane;
  const long row = (long)p.T * p.H;
  float mx = -INFINITY;
  bool nan = false;
  for (int s = lane; s < p.n_splits; s += 32) {
    const float v = lse[s * row];
    nan |= v != v;
    mx = fmaxf(mx, v);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  nan = __any_sync(0xffffffffu, nan);
  const float ref = mx == -INFINITY ? 0.f : mx;
  float acc[VI][2], sum = 0.f;
#pragma unroll
  for (int v = 0; v < VI; ++v) acc[v][0] = acc[v][1] = 0.f;
#pragma unroll 4
  for (int s = warp; s < p.n_splits; s += 4) {
    const float w = exp2f(lse[s * row] - ref);
    float2 x[VI];
#pragma unroll
    for (int v = 0; v < VI; ++v)
      x[v] = 64 * v + 2 * lane < HD ? *reinterpret_cast<const float2*>(po + s * row * HD + 64 * v) : make_float2(0.f, 0.f);
    sum += w;
#pragma unroll
    for (int v = 0; v < VI; ++v) {
      acc[v][0] += w * x[v].x;
      acc[v][1] += w * x[v].y;
    }
  }
#pragma unroll
  for (int v = 0; v < VI; ++v)
    if (64 * v + 2 * lane < HD) {
      sh[warp][64 * v + 2 * lane] = acc[v][0];
      sh[warp][64 * v + 2 * lane + 1] = acc[v][1];
    }
  if (lane == 0) sh[warp][HD] = sum;
  __syncthreads();
  const float all = sh[0][HD] + sh[1][HD] + sh[2][HD] + sh[3][HD];
  const float inv = mx == -INFINITY ? 0.f : 1.f / all;
  const float qnan = __int_as_float(0x7FC00000);
  for (int d = 2 * threadIdx.x; d < HD; d += 256) {
    const float a = (sh[0][d] + sh[1][d] + sh[2][d] + sh[3][d]) * inv;
    const float b = (sh[0][d + 1] + sh[1][d + 1] + sh[2][d + 1] + sh[3][d + 1]) * inv;
    *reinterpret_cast<uint32_t*>(p.out + t * p.o_tok + h * p.o_head + d) =
        (uint32_t)f32_to_bf16_any(nan ? qnan : a) | ((uint32_t)f32_to_bf16_any(nan ? qnan : b) << 16);
  }
  if (threadIdx.x == 0 && p.lse != nullptr)
    p.lse[t * p.H + h] = nan ? qnan : mx == -INFINITY ? -INFINITY : (mx + log2f(all)) * 0.6931471805599453f;
}

}  // namespace dllm

// Tensor-core (tcgen05 / TMEM) attention over the paged 4-bit KV cache, for canvases and
// prompt pieces: many query rows per KV head. The rows, masks and results are those of
// attention_kv4.cuh.
//
// One block takes 256 query rows (two tiles of 128) of one KV head over one split of the
// keys. Unpacking 64 keys costs about as many issue slots as one tile's softmax, so both
// tiles read the same unpacked K and V; the two tiles' softmaxes alternate with each other's
// products on the tensor pipe.
//
// Roles (512 threads):
//   warp 0       TMEM; lane 0 issues the products: S_t = Q_t K^T (bf16) into tile t's S columns,
//                O_t += P_t V (fp16) with P_t read from TMEM, where the softmax wrote it over S_t;
//   warp 1       copies packed keys page by page into a ring (bulk copies, one lane per piece);
//   warps 4..7   softmax of tile 0, warps 8..11 of tile 1: one row per thread (TMEM lane), 64
//                scores in registers, lazy reference as in attention_kv4.cuh; O is rescaled in
//                TMEM when the reference moves (rare), and read and written out at the end;
//   warps 12..15 unpack: K to bf16 and V to fp16, both exact, as 64-dim atoms of 128-byte
//                rows with the 128-byte swizzle (K's rows are keys, K-major; V's are the same
//                rows read as the MN-major operand). Eight consecutive lanes write 4 groups
//                of 2 adjacent keys: 8 different 16-byte columns, no bank conflict.
//   warps 2, 3   only help to load Q.
// TMEM: S_t at 64 t, O_t at 128 + HD t: 480 of 512 columns at head_dim 176.
// Every wait is bounded, as in gemm_tc.cuh; a block that gives one up writes NaN.
#pragma once

#include "attention_kv4.cuh"

namespace dllm {

// Instruction descriptor: fp16 A (K-major) x fp16 B (MN-major), fp32 D.
__host__ __device__ constexpr uint32_t idesc_f16_f32_bmn(int M, int N) {
  return (1u << 4) | (1u << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

template <int HD>
struct AttnKv4TcCfg {
  static constexpr int BK = 64;
  static constexpr int ATOMS = (HD + 63) / 64;
  static constexpr int STAGES = 2;                       // unpacked K and V
  static constexpr int RAW = HD == 176 ? 2 : 4;          // packed stages
  static constexpr int kQTile = ATOMS * 128 * 128;
  static constexpr int kAtom = BK * 128;
  static constexpr int kKV = ATOMS * kAtom;
  static constexpr int kCodes = BK * HD / 2;
  static constexpr int kScales = BK * HD / 16;
  static constexpr int kRawStage = 2 * (kCodes + kScales);
  static constexpr int kOffK = 2 * kQTile;
  static constexpr int kOffV = kOffK + STAGES * kKV;
  static constexpr int kOffRaw = kOffV + STAGES * kKV;
  static constexpr int kOffBar = kOffRaw + RAW * kRawStage;
  static constexpr int kTotal = kOffBar + 256 + 1024;
  static constexpr int kOCol = 2 * BK;
  static constexpr int kTmemCols = 512;
  static constexpr int THREADS = 512;
  static_assert(kOCol + 2 * HD <= kTmemCols, "TMEM");
  static_assert(kTotal <= 232448, "shared memory");
  static_assert(kOffBar % 16 == 0, "barriers");
};

// Tile t's softmax: thread (warp w, lane) owns row 32 (w % 4) + lane of the tile.
template <int HD>
DLLM_DEV void kv4_softmax_tile(const AttnKv4Params& p, const Kv4Req& rq, uint32_t tmem_base, uint64_t* s_full,
                               uint64_t* p_full, uint64_t* o_final, volatile int* flags, int t, int R0, int g, int sp,
                               int ks, int ke, int nblk) {
  using G = AttnKv4TcCfg<HD>;
  constexpr int BK = G::BK;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = 32 * (warp & 3) + lane;
  const uint32_t lane_base = tmem_base + ((uint32_t)(32 * (warp & 3)) << 16);
  const uint32_t s_col = lane_base + t * BK;
  const uint32_t o_col = lane_base + G::kOCol + t * HD;
  const int R = R0 + 128 * t + row;
  const bool real = R < rq.n * p.group;
  const int lim = real ? min(ke, kv4_row_limit(p, rq, R / p.group)) : ke;
  float m = -INFINITY, l = 0.f;
  bool ok = true;
  for (int j = 0; j < nblk; ++j) {
    if (!__all_sync(0xffffffffu, mbar_wait(&s_full[t], j & 1, flags))) { ok = false; break; }
    tc_fence_after();
    float s[BK];
    tmem_ld64(s_col, s);
    const int seen = lim - (ks + j * BK);
    if (seen < BK) {
#pragma unroll
      for (int c = 0; c < BK; ++c)
        if (c >= seen) s[c] = -INFINITY;
    }
    const float mx = tree_max<BK>(s) * p.scale_log2;
    if (j == 0) {
      m = mx - kKv4Low;
    } else {
      const bool need = mx > m + (kKv4Low + 8.f);
      if (__any_sync(0xffffffffu, need)) {
        // tile t's O is stable here: S_t(j) was issued only after P_t V(j - 1) completed
        const float mn = need ? mx - kKv4Low : m;
        const float f = need ? exp2f(m - mn) : 1.0f;
#pragma unroll 1
        for (int c = 0; c < HD; c += 16) {
          float v[16];
          tmem_ld16(o_col + c, v);
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] *= f;
          tmem_st16(o_col + c, v);
        }
        l *= f;
        m = mn;
      }
    }
    const float mb = m == -INFINITY ? 0.f : m;
    uint32_t pk[BK / 2];
#pragma unroll
    for (int c = 0; c < BK; c += 2) {
      s[c] = ex2_approx(fmaf(s[c], p.scale_log2, -mb));
      s[c + 1] = ex2_approx(fmaf(s[c + 1], p.scale_log2, -mb));
      const __half2 h = __floats2half2_rn(s[c], s[c + 1]);
      pk[c / 2] = *reinterpret_cast<const uint32_t*>(&h);
    }
    tmem_st32_nowait(s_col, pk);
    l += tree_sum<BK>(s);
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&p_full[t]);
  }
  if (ok) ok = __all_sync(0xffffffffu, mbar_wait(o_final, 0, flags));
  if (!ok) flags[0] = 1;
  tc_fence_after();
  const bool lost = flags[0] != 0 || flags[1] != 0;
  const float nan = __int_as_float(0x7FC00000);
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  const float lse2 = lost ? nan : l == 0.f ? -INFINITY : m + log2f(l);
  const long tok = rq.q0 + R / p.group;
  const int h = g * p.group + R % p.group;
  const long at = ((long)sp * p.T + tok) * p.H + h;
#pragma unroll 1
  for (int c = 0; c < HD; c += 16) {
    float v[16];
    if (nblk > 0) {
      tmem_ld16(o_col + c, v);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = 0.f;
    }
    if (!real) continue;
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = lost ? nan : l == 0.f ? 0.f : v[e] * inv;
    if (p.n_splits == 1) {
      uint32_t w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        w[e] = (uint32_t)f32_to_bf16_any(v[2 * e]) | ((uint32_t)f32_to_bf16_any(v[2 * e + 1]) << 16);
      uint4* dst = reinterpret_cast<uint4*>(p.out + tok * p.o_tok + h * p.o_head + c);
      dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
      dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
      float4* dst = reinterpret_cast<float4*>(p.part_o + at * HD + c);
#pragma unroll
      for (int e = 0; e < 4; ++e) dst[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
    }
  }
  if (real) {
    if (p.n_splits > 1) p.part_lse[at] = lse2;
    else if (p.lse != nullptr) p.lse[tok * p.H + h] = lse2 * 0.6931471805599453f;
  }
}

// Grid (row tiles, n_splits, Hkv * B); the last query tiles, which see the most keys when
// causal, come first.
template <int HD>
__global__ void __launch_bounds__(AttnKv4TcCfg<HD>::THREADS, 1)
attn_kv4_tc_kernel(const __grid_constant__ AttnKv4Params p) {
  using G = AttnKv4TcCfg<HD>;
  constexpr int BK = G::BK, AT = G::ATOMS, ST = G::STAGES;
  constexpr uint32_t kIdQK = idesc_bf16_f32(128, BK);
  constexpr uint32_t kIdPV = idesc_f16_f32_bmn(128, HD);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem + G::kOffK;
  uint8_t* sV = smem + G::kOffV;
  uint8_t* sR = smem + G::kOffRaw;
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + G::kOffBar);
  uint64_t* raw_empty = raw_full + G::RAW;
  uint64_t* k_full = raw_empty + G::RAW;
  uint64_t* k_empty = k_full + ST;
  uint64_t* v_full = k_empty + ST;
  uint64_t* v_empty = v_full + ST;
  uint64_t* s_full = v_empty + ST;   // [2]: S_t(j) is in its columns
  uint64_t* p_full = s_full + 2;     // [2]: P_t(j) is written over it
  uint64_t* pv_done = p_full + 2;    // [2]: P_t V(j) completed
  uint64_t* o_final = pv_done + 2;
  uint64_t* drain = o_final + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* flags = reinterpret_cast<volatile int*>(tmem_slot + 1);   // [0] abort, [1] a page that is none

  pdl_wait();
  const int sp = blockIdx.y, g = blockIdx.z % p.c.Hkv, b = blockIdx.z / p.c.Hkv;
  const int tile = gridDim.x - 1 - blockIdx.x;
  const Kv4Req rq = kv4_request(p, b);
  const int n_rows = rq.n * p.group, R0 = 256 * tile;
  if (rq.skip) return;
  if (rq.bad) {
    if (tile == 0 && sp == 0) kv4_poison(p, rq, g * p.group, p.group, HD);
    return;
  }
  if (R0 >= n_rows) return;
  const int nt = n_rows - R0 > 128 ? 2 : 1;
  const int last = min(n_rows, R0 + 256) - 1;
  const int ks = sp * p.chunk;
  const int ke = min(kv4_row_limit(p, rq, last / p.group), ks + p.chunk);
  const int nblk = ke > ks ? (ke - ks + BK - 1) / BK : 0;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < G::RAW; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], 4);
    }
    for (int s = 0; s < ST; ++s) {
      mbar_init(&k_full[s], 4);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 4);
      mbar_init(&v_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 4);
      mbar_init(&pv_done[t], 1);
    }
    mbar_init(o_final, 1);
    mbar_init(drain, 1);
    flags[0] = flags[1] = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, G::kTmemCols);
    tmem_relinquish();
  }
  // Q: 16-byte chunk c of row r at column c ^ (r % 8) of its atom's 128-byte row; rows past the last are 0
  for (int u = threadIdx.x; u < nt * 128 * (HD / 8); u += G::THREADS) {
    const int r = u / (HD / 8), c = u - r * (HD / 8);
    const int R = R0 + r;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (R < n_rows)
      v = *reinterpret_cast<const uint4*>(p.q + (long)(rq.q0 + R / p.group) * p.q_tok + (g * p.group + R % p.group) * p.q_head + 8 * c);
    *reinterpret_cast<uint4*>(smem + (r >> 7) * G::kQTile + (c >> 3) * 128 * 128 + (r & 127) * 128 + (((c ^ r) & 7) << 4)) = v;
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();   // after the TMEM allocation
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- MMA issuer
      bool ok = true;
      auto issue_s = [&](int t, int j) -> bool {
        const int st = j % ST;
        if (!mbar_wait(&k_full[st], (j / ST) & 1, flags)) return false;
        tc_fence_after();
        const uint32_t d = tmem_base + t * BK;
        const uint32_t qb = smem_u32(smem + t * G::kQTile), kb = smem_u32(sK + st * G::kKV);
#pragma unroll
        for (int k = 0; k < HD / 16; ++k)
          umma_bf16(d, sdesc_k_sw128(qb + (k >> 2) * 128 * 128 + (k & 3) * 32),
                    sdesc_k_sw128(kb + (k >> 2) * G::kAtom + (k & 3) * 32), kIdQK, k != 0);
        umma_commit(&s_full[t]);
        if (t == nt - 1) umma_commit(&k_empty[st]);
        return true;
      };
      auto issue_pv = [&](int t, int j) -> bool {
        const int st = j % ST;
        if (!mbar_wait(&v_full[st], (j / ST) & 1, flags)) return false;
        if (!mbar_wait(&p_full[t], j & 1, flags)) return false;
        tc_fence_after();
        const uint32_t vb = smem_u32(sV + st * G::kKV);
#pragma unroll
        for (int k = 0; k < BK / 16; ++k)
          umma_bf16_ts(tmem_base + G::kOCol + t * HD, tmem_base + t * BK + k * 8,
                       sdesc_mn_sw128(vb + k * 16 * 128, G::kAtom), kIdPV, (j | k) != 0);
        umma_commit(&pv_done[t]);
        if (t == nt - 1) umma_commit(&v_empty[st]);
        return true;
      };
      for (int t = 0; t < nt && ok && nblk > 0; ++t) ok = issue_s(t, 0);
      for (int j = 0; j < nblk && ok; ++j)
        for (int t = 0; t < nt && ok; ++t) {
          ok = issue_pv(t, j);
          // S_t(j + 1) goes over the columns that P_t V(j) reads
          if (ok && j + 1 < nblk) ok = mbar_wait(&pv_done[t], j & 1, flags) && issue_s(t, j + 1);
        }
      if (ok) umma_commit(o_final);
      else flags[0] = 1;
      umma_commit(drain);
      mbar_drain(drain, 0);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- packed keys: lane i copies piece i of a block (a page's share of it)
    const int shift = min(p.c.page_shift, 6);
    const int pieces = BK >> shift, keys = 1 << shift;
    const uint32_t codes = keys * HD / 2, scales = keys * HD / 16;
    const int* trow = p.table + (long)b * p.stride;
    bool ok = true;
    int j = 0;
    for (; j < nblk; ++j) {
      const int t = ks + j * BK + lane * keys;
      int id = -1;
      if (lane < pieces && t < ke) {
        id = trow[t >> p.c.page_shift];
        if (id < 0 || id >= p.c.n_pages) {
          id = -1;
          flags[1] = 1;
        }
      }
      const uint32_t n = __popc(__ballot_sync(0xffffffffu, id >= 0));
      const int st = j % G::RAW;
      if (!mbar_wait(&raw_empty[st], ((j / G::RAW) & 1) ^ 1, flags)) ok = false;
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) mbar_arrive_expect_tx(&raw_full[st], n * 2 * (codes + scales));
      __syncwarp();
      if (id >= 0) {
        const int off = t & ((1 << p.c.page_shift) - 1);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const long r = kv4_row(p.c, id, kv, g, off);
          uint8_t* d = sR + st * G::kRawStage + kv * (G::kCodes + G::kScales);
          bulk_load(d + lane * codes, p.c.codes + r * (HD / 2), codes, &raw_full[st]);
          bulk_load(d + G::kCodes + lane * scales, p.c.scales + r * (HD / 16), scales, &raw_full[st]);
        }
      }
    }
    if (!__all_sync(0xffffffffu, ok)) flags[0] = 1;
    // the copies already issued land before the block's shared memory goes away
    for (int i = max(0, j - G::RAW); i < j; ++i) mbar_drain(&raw_full[i % G::RAW], (i / G::RAW) & 1);
  } else if (warp >= 12) {
    // ---------------- unpacking: a warp's turn is 8 keys of one 64-dim atom
    const int w = warp - 12;
    const int grp = lane & 3, k8 = lane >> 2;
    bool ok = true;
    for (int j = 0; j < nblk && ok; ++j) {
      const int rs = j % G::RAW, st = j % ST;
      const int left = ke - (ks + j * BK);   // keys past the end become 0, whatever their bytes hold
      if (!__all_sync(0xffffffffu, mbar_wait(&raw_full[rs], (j / G::RAW) & 1, flags))) { ok = false; break; }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        uint64_t* empty = kv ? v_empty : k_empty;
        uint64_t* full = kv ? v_full : k_full;
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[st], ((j / ST) & 1) ^ 1, flags))) { ok = false; break; }
        const uint8_t* rc = sR + rs * G::kRawStage + kv * (G::kCodes + G::kScales);
        const uint8_t* rsc = rc + G::kCodes;
        uint8_t* dst = (kv ? sV : sK) + st * G::kKV;
#pragma unroll
        for (int i = 0; i < 2 * AT; ++i) {
          const int key = 8 * (w + 4 * (i & 1)) + k8, a = i >> 1;
          const int gg = 4 * a + grp;
          if (16 * gg < HD) {
            const uint2 c = *reinterpret_cast<const uint2*>(rc + key * (HD / 2) + 8 * gg);
            const uint32_t byte = key < left ? rsc[key * (HD / 16) + gg] : 0;
            uint32_t o[8];
            if (kv == 0) {
              const __nv_bfloat162 s = kv4_scale_bf16x2(byte);
              const __nv_bfloat162 n = __hmul2(s, __float2bfloat162_rn(-24.f));
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                o[e] = kv4_bf16x2(c.x, e, s, n);
                o[4 + e] = kv4_bf16x2(c.y, e, s, n);
              }
            } else {
              const __half2 s = kv4_half2((byte << 7) * 0x00010001u);
              const __half2 n = __hmul2(s, __float2half2_rn(-24.f));
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                o[e] = kv4_f16x2(c.x, e, s, n);
                o[4 + e] = kv4_f16x2(c.y, e, s, n);
              }
            }
            uint8_t* r = dst + a * G::kAtom + key * 128;
            *reinterpret_cast<uint4*>(r + (((2 * grp) ^ (key & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(r + (((2 * grp + 1) ^ (key & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
      }
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(&raw_empty[rs]);
    }
    if (!ok) flags[0] = 1;
  } else if (warp >= 4) {
    const int t = (warp - 4) >> 2;
    if (t < nt)
      kv4_softmax_tile<HD>(p, rq, tmem_base, s_full, p_full, o_final, flags, t, R0, g, sp, ks, ke, nblk);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) {
    __syncwarp();
    tmem_dealloc(tmem_base, G::kTmemCols);
  }
}

}  // namespace dllm

// Tensor-core (tcgen05 / TMEM) attention over the paged 4-bit KV cache, for canvases and
// prompt pieces: many query rows per KV head. The rows, masks and results are those of
// attention_kv4.cuh.
//
// The work is cut into tiles of 256 query rows of one KV head, two halves of 128 (below: tile 0 and tile 1
// of the tensor cores). Both read the same unpacked K and V, which halves the unpacking, and while
// one's softmax turns its scores into weights the tensor pipe runs the other's products. One block
// per SM goes through its share of all tiles (Kv4Walk); its unpacking warps begin the next tile while
// the softmax still writes the last one out.
//
// Roles (512 threads):
//   warps 0, 1   each issues one tile's products (warp 0 holds the TMEM allocation): S_t = Q_t K^T
//                (bf16) into tile t's S columns, and O_t += P_t V (fp16) with P_t read from
//                TMEM. A wait and an issue cost such a warp 150 to 200 cycles each among the
//                busy warps of its scheduler, so one warp for both tiles was the bottleneck.
//                With two buffers of scores per tile (head_dim 64 and 128) S_t(j + 2) goes out when
//                O_t(j) is done, whose P_t(j) lay in the same columns; with one, S_t(j + 1) goes out as
//                soon as the softmax has read S_t(j). Either way a tile's next scores are there
//                when its softmax is.
//   warps 2..5   softmax of tile 0, warps 6..9 of tile 1: one row per thread (TMEM lane), 48
//                scores in registers, lazy reference as in attention_kv4.cuh; O is rescaled in
//                TMEM when the reference moves (rare). They copy their rows of Q first, and
//                write O out through the same shared memory in the end, both along the rows;
//                a part of a tile leaves in fp32 straight from TMEM, [hd / 4][row][4].
//   warps 10..15 unpack 8 (of 96 keys: 16) keys of each block, K to bf16 and V to sixteenths in
//                fp16 (both exact), as 64-dim atoms of 128-byte rows with the 128-byte swizzle
//                (K's rows are keys, K-major; V's are the same rows read as the MN-major operand).
//                Eight consecutive lanes write 4 groups of 2 adjacent keys: 8 different 16-byte
//                columns, no bank conflict. The packed bytes come straight into registers, a block
//                of keys ahead, and the page ids two blocks ahead.
// TMEM: S_0, S_1 (BK columns each, or two times BK), P_0, P_1 (BK / 2, or in S), O_0, O_1 (head_dim). Keys per
// block: what fits, in multiples of 48, so that six warps unpack: 96 at head_dim 64, else 48.
// The code has to stay within the instruction cache: three roles run different loops at a time, and
// with the unrolled forms of loading Q and writing O (150 KB of code in all) every loop ran a
// quarter slower, and code that runs once waits for its own fetching. What runs once per tile is
// therefore small loops. At head_dim 176 a block of 48 keys takes 1.1 us, of which the products alone need
// 0.8 (Q is read from shared memory again for every 48 keys); at head_dim 64 a block of 96 keys takes 1.4,
// and 256 x 96 exponentials alone 0.8.
// 37 requests of 128 queries over 2048 keys at head_dim 176: 110 us, 990 TFLOP/s. 16 canvases of 256
// queries over 2200 to 4350 keys: 164 us, 915 TFLOP/s; at head_dim 64, 139 us, 525 TFLOP/s
// (148 with one buffer of scores per tile; head_dim 128: 176 and 188).
// Every wait is bounded, as in gemm_tc.cuh; a block that gives one up writes NaN from there on.
#pragma once

#include "attention_kv4.cuh"

namespace dllm {

// Instruction descriptor: fp16 A and B, both K-major, fp32 D.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// True in one lane of a converged warp, always the same one. The warp that issues the products
// runs its loop as a whole and lets the elected lane issue: descriptors, addresses and loop
// state are then the same in every lane, and stay in uniform registers, which is where the
// tensor instructions take them from. (In a branch that only lane 0 enters, each product cost
// about 150 cycles to issue, more than it took to run.)
DLLM_DEV bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r));
  return r != 0;
}

// What parts cost on their way to memory and back, in blocks of keys: 2 us and 180 KB each way per
// part of head_dim 176, 4 TB/s.
__host__ __device__ constexpr int kv4_cut_cost(int parts, int hd) { return 2 + parts * hd / 2600; }

template <int HD>
struct AttnKv4TcCfg {
  static constexpr int BK = HD == 64 ? 96 : 48;          // keys of a block
  static constexpr int CH = 48;                          // of which the softmax has this many in registers at a time
  static constexpr int ATOMS = (HD + 63) / 64;
  static constexpr int KST = 3, VST = 2;                 // unpacked stages of K and of V
  static constexpr int kQTile = ATOMS * 128 * 128;
  static constexpr int kAtom = BK * 128;
  static constexpr int kKV = ATOMS * kAtom;
  static constexpr int kOffK = 2 * kQTile;
  static constexpr int kOffV = kOffK + KST * kKV;
  static constexpr int kOffBar = kOffV + VST * kKV;
  static constexpr int kOffShare = kOffBar + 256;        // Kv4Walk::begin's
  static constexpr int kTotal = kOffShare + 256 + 1024;
  // Two buffers of scores per tile, P in place of the scores it came from, where TMEM has room; else one, and P
  // in columns of its own.
  static constexpr bool TWO = 4 * BK + 2 * HD <= 512;
  static constexpr int kOCol = (TWO ? 4 : 3) * BK;
  __host__ __device__ static constexpr int s_col(int t, uint32_t c) { return TWO ? (2 * t + (int)(c & 1)) * BK : t * BK; }
  // the column of a tile's P from key `key` of a block on (a multiple of 16)
  __host__ __device__ static constexpr int p_col(int t, uint32_t c, int key) {
    return TWO ? s_col(t, c) + key / CH * CH + key % CH / 2 : 2 * BK + t * (BK / 2) + key / 2;
  }
  // which of a tile's two barriers counts block c, and its phase's parity
  __host__ __device__ static constexpr int bar(int t, uint32_t c) { return 2 * t + (TWO ? (int)(c & 1) : 0); }
  __host__ __device__ static constexpr uint32_t par(uint32_t c) { return TWO ? (c >> 1) & 1 : c & 1; }
  static constexpr int kTmemCols = 512;
  static constexpr int UNPACK = 6;                       // unpacking warps
  static constexpr int GPW = BK / 8 / UNPACK;            // groups of 8 keys of a block that each takes
  static constexpr int THREADS = 32 * (2 + 8 + UNPACK);
  static constexpr int START = 4;                        // what starting a tile costs, in blocks of keys
  static_assert(kOCol + 2 * HD <= kTmemCols, "TMEM");
  static_assert(kTotal <= 232448, "shared memory");
  static_assert(kOffBar % 16 == 0, "barriers");
};

DLLM_DEV void tmem_st8_nowait(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// 48 columns of scores into registers, and 24 columns of weights out of them (not waited for).
DLLM_DEV void kv4_load_scores(uint32_t taddr, float (&s)[48]) {
  tmem_ld32(taddr, reinterpret_cast<float(&)[32]>(s[0]));
  tmem_ld16(taddr + 32, reinterpret_cast<float(&)[16]>(s[32]));
}
DLLM_DEV void kv4_store_weights(uint32_t taddr, const uint32_t (&w)[24]) {
  tmem_st16_nowait(taddr, reinterpret_cast<const uint32_t(&)[16]>(w[0]));
  tmem_st8_nowait(taddr + 16, w + 16);
}

// kv4_bf16x2 with the AND-OR in one operation (and_or).
DLLM_DEV uint32_t kv4_bf16x2_masked(uint32_t w, int j, __nv_bfloat162 s, __nv_bfloat162 ms24, uint32_t mask) {
  const uint32_t u = and_or<0x41804180u>(j == 0 ? w << 3 : w >> (4 * j - 3), mask);
  const __nv_bfloat162 v = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&u), s, ms24);
  return *reinterpret_cast<const uint32_t*>(&v);
}

DLLM_DEV uint32_t kv4_bf16_pair(float lo, float hi) {   // to nearest even, NaN stays one
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 16 bytes from global to shared memory, `n` of them (0 or 16) read and the others 0.
DLLM_DEV void copy16(void* dst, const void* src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)),
               "l"((uint64_t)__cvta_generic_to_global(src)), "r"(n)
               : "memory");
}

// 16-byte chunk c of row r of a 128-row tile of atoms (64 dims of 2 bytes) under the 128-byte swizzle.
DLLM_DEV uint8_t* kv4_chunk(uint8_t* tile, int r, int c) {
  return tile + (c >> 3) * 128 * 128 + r * 128 + (((c ^ r) & 7) << 4);
}

// A row tile over key blocks j0 .. j1 - 1.
struct Kv4Work {
  int b, h, tile, j0, j1;
  bool starts, ends;        // with the tile's first, last key block
  Kv4Req rq;
};

// The work of a thread block, the same in all its threads: a share of all tiles, which lie request by
// request, head by head, from the last tile (which sees the most keys when causal) to the first.
// Lengths are known on the device only, so each block adds up the requests' work by itself (begin).
// The shares have either equal numbers of whole tiles or equal numbers of key blocks, and then some
// tiles are cut into parts that attn_kv4_parts_kernel joins. A cut is worth its two parts' way to
// memory and back if whole tiles would leave more SMs idle than that, which `begin` estimates (in key
// blocks of 1.1 us at head_dim 176, 1.4 at 64). Measured, head_dim 176, whole against cut: one canvas of
// 256 queries (16 tiles) over 256 keys 16.5 us and 18.1, 768 keys 26.4 and 19.7; 37 requests of 128 queries over
// 500 to 1000 keys (296 tiles) 63 and 76; 16 canvases over 2200 to 4350 keys (256 tiles) 209 and 164.
// With fewer tiles than SMs, every tile has as many shares as fit.
template <int HD>
struct Kv4Walk {
  using G = AttnKv4TcCfg<HD>;
  int b, h, i, x;           // the next tile, and how far into it the share begins
  int left, tiles;
  bool cut;                 // shares may begin and end inside a tile
  Kv4Req rq;

  DLLM_DEV int blocks(const AttnKv4Params& p, int tile) const {
    if (rq.bad) return 0;
    const int last = min(rq.n * p.group, 256 * (tile + 1)) - 1;
    return (kv4_row_limit(p, rq, last / p.group) + G::BK - 1) / G::BK;
  }
  DLLM_DEV void request(const AttnKv4Params& p, int b_) {
    b = b_;
    rq = kv4_request(p, b);
    tiles = rq.bad ? rq.n > 0 : (rq.n * p.group + 255) / 256;   // a bad request is answered with its first tile
  }
  // in units of 2^unit_shift key blocks, so that all of a call's fit 32 bits
  DLLM_DEV int cost(const AttnKv4Params& p, int tile) const {
    return cut ? G::START + ((blocks(p, tile) + (1 << p.unit_shift) - 1) >> p.unit_shift) : 1;
  }
  DLLM_DEV int costs(const AttnKv4Params& p, int& most) const {
    if (!cut) return tiles;
    int c = 0;
    for (int t = 0; t < tiles; ++t) {
      const int c1 = cost(p, t);
      c += c1;
      most = max(most, c1);
    }
    return c;
  }
  // All threads; mem: MEM ints that stay as they are until the next barrier. Half of the time of a kernel that
  // has little to do is code that is fetched to run once, so 32 bits, few divisions and one barrier, which
  // serves as the kernel's too.
  static constexpr int WARPS = G::THREADS / 32, MEM = 3 * WARPS + 8;
  DLLM_DEV void begin(const AttnKv4Params& p, int* mem) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r0 = p.B * tid / G::THREADS, r1 = p.B * (tid + 1) / G::THREADS;
    int work = 0, some = 0, most = 0;
    cut = p.cut;
    for (int r = r0; r < r1; ++r) {
      request(p, r);
      work += p.c.Hkv * costs(p, most);
      some += p.c.Hkv * tiles;
    }
    int upto_work = work, upto_some = some;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto_work, o), u = __shfl_up_sync(0xffffffffu, upto_some, o);
      if (lane >= o) {
        upto_work += v;
        upto_some += u;
      }
    }
    most = __reduce_max_sync(0xffffffffu, most);
    int* found = mem + 3 * WARPS;
    if (tid == 0) found[0] = -1;
    if (lane == 31) {
      mem[warp] = upto_work;
      mem[WARPS + warp] = upto_some;
      mem[2 * WARPS + warp] = most;
    }
    __syncthreads();
    // lane w of every warp has what warp w added up
    const int sum = lane < WARPS ? mem[lane] : 0, tile_sum = lane < WARPS ? mem[WARPS + lane] : 0;
    const int count = __reduce_add_sync(0xffffffffu, tile_sum);
    int all = __reduce_add_sync(0xffffffffu, sum), n = gridDim.x;
    if (cut) {
      most = __reduce_max_sync(0xffffffffu, lane < WARPS ? mem[2 * WARPS + lane] : 0);
      // tiles that are cut have to be worth it: parts are written and read again
      cut = (count + n - 1) / n * most > all / n + (kv4_cut_cost(count < n ? n : 2 * n, HD) >> p.unit_shift);
    }
    if (!cut) all = count;
    const int mine = cut ? work : some;
    const int upto = (cut ? upto_work : upto_some) + __reduce_add_sync(0xffffffffu, lane < warp ? (cut ? sum : tile_sum) : 0);
    // no share is empty but the last blocks', so that a tile's parts lie in consecutive blocks
    int lo = 0;
    n = min(all, n);
    left = 0;
    if (count > 0 && count < n) n = n / count * count;
    if ((int)blockIdx.x < n) {
      const int each = all / n, more = all - each * n, k = blockIdx.x;
      lo = each * k + more * k / n;
      left = each * (k + 1) + more * (k + 1) / n - lo;
    }
    if (left > 0 && lo >= upto - mine && lo < upto) {
      int rest = lo - (upto - mine);
      for (int r = r0; r < r1; ++r) {
        request(p, r);
        const int c = costs(p, most);
        if (rest >= p.c.Hkv * c) {
          rest -= p.c.Hkv * c;
          continue;
        }
        found[0] = r;
        found[1] = rest / c;
        rest -= rest / c * c;
        int t = tiles - 1;
        for (int c1 = cost(p, t); rest >= c1; c1 = cost(p, --t)) rest -= c1;
        found[2] = t;
        found[3] = rest;
        found[4] = tiles;
        found[5] = rq.q0;
        found[6] = rq.n;
        found[7] = rq.bad ? -1 : rq.kv;
        break;
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    b = found[0];
    if (b < 0) left = 0;   // no work (or row ranges that overlap, in numbers beyond 32 bits)
    h = found[1];
    i = found[2];
    x = found[3];
    tiles = found[4];
    rq = Kv4Req{found[5], found[6], found[7], false, found[7] < 0};
  }
  DLLM_DEV bool next(const AttnKv4Params& p, Kv4Work& w) {
    while (left > 0) {
      if (i < 0) {
        if (++h == p.c.Hkv) {   // the next request with rows: a padded batch may have many without
          h = 0;
          const int lane = threadIdx.x & 31;
          unsigned some = 0;
          for (++b; some == 0; b += 32) {
            if (b >= p.B) return false;
            const int r = min(b + lane, p.B - 1);
            some = __ballot_sync(0xffffffffu, b + lane < p.B && p.q_start[r + 1] > p.q_start[r]);
          }
          request(p, b - 32 + __ffs(some) - 1);
        }
        i = tiles - 1;
        continue;
      }
      const int all = blocks(p, i), take = min(left, cost(p, i) - x);
      const int j0 = cut ? max(0, x - G::START) << p.unit_shift : 0;
      const int j1 = cut ? min(all, max(0, x + take - G::START) << p.unit_shift) : all;
      const bool begun = x == 0;
      w = Kv4Work{b, h, i, j0, j1, j0 == 0, j1 == all, rq};
      left -= take;
      --i;
      x = 0;
      if (j1 > j0 || (all == 0 && begun)) return true;
    }
    return false;
  }
};

// The blocks of keys of a tile from j on, one row per thread; m and l are the row's reference and sum so far. `lim` is
// where the row's keys end, counted from the first block's first. False once a wait was given up.
// A weight is 2^(s fac - m), with one fma. That takes the rounded reference off the exact product, which shifts all of
// a row's weights alike and is nothing while the rounding is far below 1. With a reference of 2^25 it is not: the
// largest weight would leave fp16's range, or vanish. So this loop leaves before the weights of a block whose
// reference is above 2^22 in any row of the warp, and FAR's, which rounds the products first as the reference is
// rounded, goes on from there. (Rounding them where needed in one loop: prompt pieces at head_dim 64 93.4 us
// instead of 88.9.)
template <int HD, bool FAR>
DLLM_DEV bool kv4_softmax_blocks(float scale, int lim, int nblk, uint32_t lane_base, uint64_t* s_full, uint64_t* s_read,
                                 uint64_t* p_full, uint64_t* pv_done, volatile int* flags, int t, uint32_t done, int& j,
                                 float& m, float& l) {
  using G = AttnKv4TcCfg<HD>;
  constexpr int BK = G::BK, CH = G::CH, NCH = BK / CH;
  const int lane = threadIdx.x & 31;
  const uint32_t o_col = lane_base + G::kOCol + t * HD;
  const float fac = FAR ? 1.f : scale;
#pragma unroll 1
  for (; j < nblk; ++j) {
    if (!__all_sync(0xffffffffu, mbar_wait(&s_full[G::bar(t, done + j)], G::par(done + j), flags))) return false;
    tc_fence_after();
    const uint32_t s_col = lane_base + G::s_col(t, done + j);
    float s[CH];
    const int seen = lim - j * BK;
    auto load = [&](int q) {
      kv4_load_scores(s_col + q * CH, s);
      if (FAR) {
#pragma unroll
        for (int c = 0; c < CH; ++c) s[c] *= scale;
      }
      if (seen < (q + 1) * CH) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
          if (q * CH + c >= seen) s[c] = -INFINITY;
      }
    };
    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int q = 0; q < NCH; ++q) {
      load(q);
#pragma unroll
      for (int c = 0; c < CH; ++c) top[c & 3] = fmaxf(top[c & 3], s[c]);
    }
    const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * fac;
    bool moved = j == 0;
    if (j == 0) {
      m = mx - kKv4Low;
    } else {
      const bool need = mx > kv4_above(m);
      moved = __any_sync(0xffffffffu, need);
      if (moved) {
        // O is stable once the product of the block before is done
        if (!__all_sync(0xffffffffu, mbar_wait(&pv_done[G::bar(t, done + j - 1)], G::par(done + j - 1), flags))) return false;
        tc_fence_after();
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
    if (!FAR && moved && __any_sync(0xffffffffu, fabsf(m) > 0x1p22f && m != -INFINITY)) return true;
    const float mb = m == -INFINITY ? 0.f : m;
    const uint64_t sc2 = pack_f32x2(fac, fac), mb2 = pack_f32x2(-mb, -mb);
    uint64_t sum[4] = {0, 0, 0, 0};   // pairs of fp32 sums
#pragma unroll
    for (int q = NCH - 1; q >= 0; --q) {   // the last chunk is still in registers
      if (q < NCH - 1) load(q);
      if (q == 0 && !G::TWO) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_read[t]);
      }
      uint32_t pk[CH / 2];
#pragma unroll
      for (int c = 0; c < CH; c += 2) {
        float a, b;
        unpack_f32x2(fma_f32x2(pack_f32x2(s[c], s[c + 1]), sc2, mb2), a, b);
        a = ex2_approx(a);
        b = ex2_approx(b);
        sum[(c / 2) & 3] = add_f32x2(sum[(c / 2) & 3], pack_f32x2(a, b));
        const __half2 h = __floats2half2_rn(a, b);
        pk[c / 2] = *reinterpret_cast<const uint32_t*>(&h);
      }
      if (q == NCH - 1 && j > 0 && !G::TWO) {   // P's columns are free once the product of the block before is done
        if (!__all_sync(0xffffffffu, mbar_wait(&pv_done[G::bar(t, done + j - 1)], G::par(done + j - 1), flags))) return false;
        tc_fence_after();
      }
      kv4_store_weights(lane_base + G::p_col(t, done + j, q * CH), pk);
    }
    float l0, l1;
    unpack_f32x2(add_f32x2(add_f32x2(sum[0], sum[1]), add_f32x2(sum[2], sum[3])), l0, l1);
    l += l0 + l1;
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&p_full[G::bar(t, done + j)]);
  }
  return true;
}

// Tile t's softmax: thread (warp w, lane) owns row 32 (w % 4) + lane of the tile. `done` counts the blocks of
// keys that went through the tile's barriers before.
template <int HD>
DLLM_DEV void kv4_softmax_tile(const AttnKv4Params& p, const Kv4Work& w, const uint32_t* tmem_slot, uint64_t* s_full,
                               uint64_t* s_read, uint64_t* p_full, uint64_t* pv_done, uint64_t* q_full,
                               uint8_t* q_smem, volatile int* flags, int t, uint32_t done) {
  using G = AttnKv4TcCfg<HD>;
  constexpr int BK = G::BK, CHUNKS = HD / 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = 32 * (warp & 3), row = row0 + lane;
  const int R = 256 * w.tile + 128 * t + row;
  const Kv4Req& rq = w.rq;
  const int g = w.h, nblk = w.j1 - w.j0, ks = w.j0 * BK, ke = w.j1 * BK;
  const bool real = R < rq.n * p.group;
  const int lim = real ? min(ke, kv4_row_limit(p, rq, R / p.group)) : ke;
  // Q: the warp's 32 rows, copied along the rows; rows past the last are 0. A tile without keys needs none, and
  // must not arrive: the issuer counts a phase of q_full for each work with keys and waits for every one.
  if (nblk > 0) {
    const long src = real ? (long)(rq.q0 + R / p.group) * p.q_tok + (g * p.group + R % p.group) * p.q_head : -1;
#pragma unroll 2
    for (int i = 0; i < CHUNKS; ++i) {
      const int u = 32 * i + lane, r = u / CHUNKS, c = u - r * CHUNKS;
      const long from = __shfl_sync(0xffffffffu, src, r);
      copy16(kv4_chunk(q_smem, row0 + r, c), p.q + (from >= 0 ? from + 8 * c : 0), from >= 0 ? 16 : 0);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&q_full[t]);
  }
  const uint32_t lane_base = *tmem_slot + ((uint32_t)row0 << 16);
  const uint32_t o_col = lane_base + G::kOCol + t * HD;
  float m = -INFINITY, l = 0.f;
  int j = 0;
  bool ok = kv4_softmax_blocks<HD, false>(p.scale_log2, lim - ks, nblk, lane_base, s_full, s_read, p_full, pv_done, flags, t,
                                          done, j, m, l);
  if (ok && j < nblk)
    ok = kv4_softmax_blocks<HD, true>(p.scale_log2, lim - ks, nblk, lane_base, s_full, s_read, p_full, pv_done, flags, t, done,
                                      j, m, l);
  if (ok && nblk > 0) ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[G::bar(t, done + nblk - 1)], G::par(done + nblk - 1), flags));
  if (!ok) flags[0] = 1;
  tc_fence_after();
  const bool lost = flags[0] != 0;
  const float nan = __int_as_float(0x7FC00000);
  const float inv = lost ? nan : l == 0.f ? 0.f : 16.0f / l;   // V came in sixteenths
  const float lse2 = lost ? nan : l == 0.f ? -INFINITY : m + log2f(l);
  // (where the row goes is worked out again, rather than kept in registers through the loop)
  int row_now = R;
  asm volatile("" : "+r"(row_now));
  const long tok = rq.q0 + row_now / p.group;
  const int h = g * p.group + row_now % p.group;
  // a part of a tile: the block's second one if it is the tile's first (then it is the block's last work)
  const int part = 2 * blockIdx.x + w.starts;
  if (!(w.starts && w.ends)) {
    p.part_lse[part * 256 + 128 * t + row] = lse2;
    if (t == 0 && row == 0) p.parts[part] = make_int4(w.b, w.h, w.tile, w.ends ? 2 : 1);
    float4* to = reinterpret_cast<float4*>(p.part_o) + (long)part * 64 * HD + 128 * t + row;
#pragma unroll 1
    for (int c = 0; c < HD; c += 16) {
      float v[16];
      tmem_ld16(o_col + c, v);
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        to[(c + e) * 64] = make_float4(v[e] * inv, v[e + 1] * inv, v[e + 2] * inv, v[e + 3] * inv);
    }
    return;
  }
  if (real && p.lse != nullptr) p.lse[tok * p.H + h] = lse2 * 0.6931471805599453f;
  // O through the tile's Q, which no product reads any more, so that rows leave along the rows
#pragma unroll 1
  for (int c = 0; c < HD; c += 16) {
    float v[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = 0.f;
    if (nblk > 0) tmem_ld16(o_col + c, v);   // (without a block O was never written)
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      o[e] = kv4_bf16_pair(v[2 * e] * inv, v[2 * e + 1] * inv);
    *reinterpret_cast<uint4*>(kv4_chunk(q_smem, row, c / 8)) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(kv4_chunk(q_smem, row, c / 8 + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
  }
  __syncwarp();
  bf16_t* to = real ? p.out + tok * p.o_tok + h * p.o_head : nullptr;
#pragma unroll 2
  for (int i = 0; i < CHUNKS; ++i) {
    const int u = 32 * i + lane, r = u / CHUNKS, c = u - r * CHUNKS;
    bf16_t* dst = reinterpret_cast<bf16_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), r));
    if (dst != nullptr)
      *reinterpret_cast<uint4*>(dst + 8 * c) = *reinterpret_cast<const uint4*>(kv4_chunk(q_smem, row0 + r, c));
  }
  __syncwarp();
}

// Grid: any number of blocks; Kv4Walk says what each does.
template <int HD>
__global__ void __launch_bounds__(AttnKv4TcCfg<HD>::THREADS, 1)
attn_kv4_tc_kernel(const __grid_constant__ AttnKv4Params p) {
  using G = AttnKv4TcCfg<HD>;
  constexpr int BK = G::BK, AT = G::ATOMS, KST = G::KST, VST = G::VST;
  constexpr uint32_t kIdQK = idesc_bf16_f32(128, BK);
  constexpr uint32_t kIdPV = idesc_f16_f32(128, HD) | (1u << 16);   // B MN-major
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem + G::kOffK;
  uint8_t* sV = smem + G::kOffV;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + G::kOffBar);
  uint64_t* k_empty = k_full + KST;
  uint64_t* v_full = k_empty + KST;
  uint64_t* v_empty = v_full + VST;
  // two per tile, of even and odd blocks, with two buffers (G::bar)
  uint64_t* s_full = v_empty + VST;  // [4]: S_t(j) is in its columns
  uint64_t* p_full = s_full + 4;     // [4]: P_t(j) is in its columns
  uint64_t* pv_done = p_full + 4;    // [4]: P_t V(j) completed
  uint64_t* s_read = pv_done + 4;    // [2]: the softmax has S_t(j) in registers (one buffer only)
  // [2]: tile t's Q is in shared memory. One phase per work that has keys and rows in the tile, arrived on by the
  // softmax's warps and waited for by the issuer; were one left out on either side, the wait of a later work would
  // pass on an older phase's parity, and its scores would come from another work's Q.
  uint64_t* q_full = s_read + 2;
  uint64_t* drain = q_full + 2;      // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
  volatile int* flags = reinterpret_cast<volatile int*>(tmem_slot + 1);   // [0] abort

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < KST; ++s) {
      mbar_init(&k_full[s], G::UNPACK);
      mbar_init(&k_empty[s], 2);
    }
    for (int s = 0; s < VST; ++s) {
      mbar_init(&v_full[s], G::UNPACK);
      mbar_init(&v_empty[s], 2);
    }
    for (int t = 0; t < 2; ++t) {
      for (int k = 2 * t; k < 2 * t + 2; ++k) {
        mbar_init(&s_full[k], 1);
        mbar_init(&p_full[k], 4);
        mbar_init(&pv_done[k], 1);
      }
      mbar_init(&s_read[t], 4);
      mbar_init(&q_full[t], 4);
      mbar_init(&drain[t], 1);
    }
    flags[0] = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    __syncwarp();
    tmem_alloc(tmem_slot, G::kTmemCols);
    tmem_relinquish();
  }
  pdl_wait();
  if (p.cut && threadIdx.x < 2) p.parts[2 * blockIdx.x + threadIdx.x] = make_int4(0, 0, 0, 0);
  Kv4Walk<HD> walk;
  static_assert(4 * Kv4Walk<HD>::MEM <= 256, "share");
  walk.begin(p, reinterpret_cast<int*>(smem + G::kOffShare));   // barriers and TMEM are there after it
  pdl_trigger();                                                // after the TMEM allocation
  Kv4Work w;

  if (warp < 2) {
    // ---------------- MMA issuer of tile `warp`: the warp waits as one, an elected lane issues
    const int t = __shfl_sync(0xffffffffu, warp, 0);
    const uint32_t tm = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const uint32_t o_col = tm + G::kOCol + t * HD;
    const uint64_t qd = sdesc_k_sw128(smem_u32(smem + t * G::kQTile));
    const uint64_t kd0 = sdesc_k_sw128(smem_u32(sK)), vd0 = sdesc_mn_sw128(smem_u32(sV), G::kAtom);
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, flags));
    };
    int kst = 0, vst = 0;        // stages and their parities
    uint32_t kph = 0, vph = 0;
    uint32_t done = 0, loads = 0;
    bool live = true;            // the work has rows in this tile; otherwise the stages are only passed on
    auto issue_s = [&](int j) -> bool {
      if (!wait(&k_full[kst], kph)) return false;
      tc_fence_after();
      if (elect_one()) {
        if (live) {
          const uint64_t kd = kd0 + kst * (G::kKV >> 4);   // descriptors count 16-byte units
#pragma unroll
          for (int k = 0; k < HD / 16; ++k)
            umma_bf16(tm + G::s_col(t, done + j), qd + (((k >> 2) * 128 * 128 + (k & 3) * 32) >> 4),
                      kd + (((k >> 2) * G::kAtom + (k & 3) * 32) >> 4), kIdQK, k != 0);
          umma_commit(&s_full[G::bar(t, done + j)]);
          umma_commit(&k_empty[kst]);
        } else {
          mbar_arrive(&k_empty[kst]);
        }
      }
      __syncwarp();
      if (++kst == KST) { kst = 0; kph ^= 1; }
      return true;
    };
    bool ok = true;
    while (ok && walk.next(p, w)) {
      const int nblk = w.j1 - w.j0;
      live = t == 0 || w.rq.n * p.group - 256 * w.tile > 128;
      if (nblk == 0) continue;   // no key in sight: there is nothing to multiply, and no Q to wait for
      ok = (!live || wait(&q_full[t], loads & 1)) && issue_s(0) && (!G::TWO || nblk == 1 || issue_s(1));
#pragma unroll 1
      for (int j = 0; j < nblk && ok; ++j) {
        if (!G::TWO && j + 1 < nblk && !((!live || wait(&s_read[t], (done + j) & 1)) && issue_s(j + 1))) { ok = false; break; }
        if (!wait(&v_full[vst], vph) || (live && !wait(&p_full[G::bar(t, done + j)], G::par(done + j)))) { ok = false; break; }
        tc_fence_after();
        if (elect_one()) {
          if (live) {
            const uint64_t vd = vd0 + vst * (G::kKV >> 4);
#pragma unroll
            for (int k = 0; k < BK / 16; ++k)
              umma_bf16_ts(o_col, tm + G::p_col(t, done + j, 16 * k), vd + ((k * 16 * 128) >> 4), kIdPV, (j | k) != 0);
            umma_commit(&pv_done[G::bar(t, done + j)]);
            umma_commit(&v_empty[vst]);
          } else {
            mbar_arrive(&v_empty[vst]);
          }
        }
        __syncwarp();
        if (++vst == VST) { vst = 0; vph ^= 1; }
        // the next scores of this buffer once P_t(j), which lies in it, has been read
        if (G::TWO && j + 2 < nblk)
          ok = (!live || wait(&pv_done[G::bar(t, done + j)], G::par(done + j))) && issue_s(j + 2);
      }
      if (live) {
        done += nblk;
        ++loads;
      }
    }
    if (!ok) flags[0] = 1;
    if (elect_one()) umma_commit(&drain[t]);
    __syncwarp();
    mbar_drain(&drain[t], 0);
    __syncwarp();
  } else if (warp >= 10) {
    // ---------------- unpacking: GPW times 8 keys of each block, lane / 4 the key, lane % 4 the group of an atom
    constexpr int GPW = G::GPW;
    const int k8 = lane >> 2, grp = lane & 3;
    const int key0 = 8 * (warp - 10) + k8;                      // and key0 + 48
    const int mask = (1 << p.c.page_shift) - 1;
    const long v_rows = (long)p.c.Hkv << p.c.page_shift, page_rows = 2 * v_rows;
    const int* trow = nullptr;
    int head_row = 0, ks = 0, ke = 0, nblk = 0;
    uint2 code[2][GPW][AT];
    uint32_t byte[2][GPW][AT];
    int id_k[GPW], id_v[GPW];
    // table entry of a key in block j, -2 past the end
    auto ask = [&](int j, int (&id)[GPW]) {
#pragma unroll
      for (int i = 0; i < GPW; ++i) {
        const int t = ks + j * BK + key0 + 48 * i;
        id[i] = j < nblk && t < ke ? trow[t >> p.c.page_shift] : -2;
      }
    };
    // an entry that is no page becomes -1
    auto check = [&](int (&id)[GPW]) {
#pragma unroll
      for (int i = 0; i < GPW; ++i)
        if (id[i] != -2 && (id[i] < 0 || id[i] >= p.c.n_pages)) id[i] = -1;
    };
    // a block's bytes of K or V; a key that does not exist has scale 0 and becomes 0; one in no page has an
    // infinite scale in K, which makes it NaN (infinity - infinity), and with it the rows that see it
    auto fetch = [&](int kv, int j, const int (&id)[GPW]) {
#pragma unroll
      for (int i = 0; i < GPW; ++i) {
        const long r = max(id[i], 0) * page_rows + (head_row + ((ks + j * BK + key0 + 48 * i) & mask)) + (kv ? v_rows : 0);
        const uint8_t* pc = p.c.codes + r * (HD / 2) + 8 * grp;
        const uint8_t* ps = p.c.scales + r * (HD / 16) + grp;
#pragma unroll
        for (int a = 0; a < AT; ++a) {
          code[kv][i][a] = make_uint2(0, 0);
          byte[kv][i][a] = kv == 0 && id[i] == -1 ? 0x7F8 : 0;
          if (id[i] >= 0 && 16 * (4 * a + grp) < HD) {
            code[kv][i][a] = *reinterpret_cast<const uint2*>(pc + 32 * a);
            byte[kv][i][a] = ps[4 * a];
          }
        }
      }
    };
    const uint32_t at0 = key0 * 128 + (((2 * grp) ^ k8) << 4);
    const Kv4Masks masks{p.mask_low, p.mask_high};
    bool ok = true;
    // the next work's first page ids
    auto open = [&]() -> bool {
      do {
        if (!walk.next(p, w)) return false;
      } while (w.j1 == w.j0);
      nblk = w.j1 - w.j0;
      ks = w.j0 * BK;
      ke = min(w.j1 * BK, kv4_row_limit(p, w.rq, (min(w.rq.n * p.group, 256 * (w.tile + 1)) - 1) / p.group));
      trow = p.table + (long)w.b * p.stride;
      head_row = w.h << p.c.page_shift;
      ask(0, id_v);
      ask(1, id_k);
      return true;
    };
    int kst = 0, vst = 0;            // stages, and the parities of their being empty
    uint32_t kph = 1, vph = 1;
    bool more = open();
    while (more) {
      // K runs a block ahead of V, as S runs ahead of P V: the turns are K(0), K(1), V(0), K(2), V(1), ...
      check(id_v);
      fetch(0, 0, id_v);
      fetch(1, 0, id_v);
#pragma unroll 1
      for (int j = -1; j < nblk && ok; ++j) {
        // this turn's bytes have had a block's time to arrive; all loads of the next one are issued
        // together before any is waited for again
        uint2 now[2][GPW][AT];
        uint32_t scale[2][GPW][AT];
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
#pragma unroll
          for (int i = 0; i < GPW; ++i)
#pragma unroll
            for (int a = 0; a < AT; ++a) {
              if (kv == 1 && j < 0) continue;
              now[kv][i][a] = code[kv][i][a];
              scale[kv][i][a] = byte[kv][i][a];
              asm volatile("" : "+r"(now[kv][i][a].x), "+r"(now[kv][i][a].y), "+r"(scale[kv][i][a]));
            }
        check(id_k);
        fetch(0, j + 2, id_k);
        if (j >= 0) fetch(1, j + 1, id_v);
#pragma unroll
        for (int i = 0; i < GPW; ++i) id_v[i] = id_k[i];
        ask(j + 3, id_k);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int jb = kv ? j : j + 1;
          if (jb < 0 || jb >= nblk) continue;
          const int st = kv ? vst : kst;
          if (!__all_sync(0xffffffffu, mbar_wait(&(kv ? v_empty : k_empty)[st], kv ? vph : kph, flags))) {
            ok = false;
            break;
          }
          if (kv == 0 && ++kst == KST) { kst = 0; kph ^= 1; }
          if (kv == 1 && ++vst == VST) { vst = 0; vph ^= 1; }
          uint8_t* dst = (kv ? sV : sK) + st * G::kKV + at0;
          uint8_t* dst2 = (kv ? sV : sK) + st * G::kKV + (at0 ^ 16);
#pragma unroll
          for (int i = 0; i < GPW; ++i)
#pragma unroll
            for (int a = 0; a < AT; ++a) {
              if (16 * (4 * a + grp) < HD) {
                uint32_t o[8];
                if (kv == 0) {
                  const __nv_bfloat162 sc = kv4_scale_bf16x2(scale[kv][i][a]);
                  const __nv_bfloat162 m24 = __hmul2(sc, __float2bfloat162_rn(-24.f));
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    o[e] = kv4_bf16x2_masked(now[kv][i][a].x, e, sc, m24, p.mask_bf16);
                    o[4 + e] = kv4_bf16x2_masked(now[kv][i][a].y, e, sc, m24, p.mask_bf16);
                  }
                } else {
                  const Kv4Scale2 sc = kv4_scale2(scale[kv][i][a] * 0x00800080u);
                  kv4_sixteenth(now[kv][i][a].x, sc, masks, reinterpret_cast<uint32_t(&)[4]>(o[0]));
                  kv4_sixteenth(now[kv][i][a].y, sc, masks, reinterpret_cast<uint32_t(&)[4]>(o[4]));
                }
                *reinterpret_cast<uint4*>(dst + a * G::kAtom + i * 48 * 128) = make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4*>(dst2 + a * G::kAtom + i * 48 * 128) = make_uint4(o[4], o[5], o[6], o[7]);
              }
            }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&(kv ? v_full : k_full)[st]);
        }
      }
      more = ok && open();
    }
    if (!ok) flags[0] = 1;
  } else {
    const int t = (warp - 2) >> 2;
    uint32_t done = 0;
    while (walk.next(p, w)) {
      if (w.rq.bad) {
        if (t == 0) kv4_poison<HD>(p, w.rq, w.h * p.group, p.group, threadIdx.x - 64, 128);
      } else if (t == 0 || w.rq.n * p.group - 256 * w.tile > 128) {
        kv4_softmax_tile<HD>(p, w, tmem_slot, s_full, s_read, p_full, pv_done, q_full, smem + t * G::kQTile, flags, t, done);
        done += w.j1 - w.j0;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) {
    __syncwarp();
    tmem_dealloc(*tmem_slot, G::kTmemCols);
  }
}

constexpr int kKv4MaxBlocks = 160;   // of attn_kv4_tc_kernel: what attn_kv4_parts_kernel has room for

// Joins the parts of tiles that several of `blocks` blocks shared. One wave of blocks (256 threads each),
// which look up which tiles there are and deal out pieces of 8 dims of one, a row per thread. What
// bounds it is the latency of loads that depend on one another, so a thread has up to four parts' loads
// under way. (A block per tile and piece, most of which ended at once: as long as the joins.)
template <int HD>
__global__ void __launch_bounds__(256, 4)
attn_kv4_parts_kernel(const __grid_constant__ AttnKv4Params p, int blocks) {
  constexpr int PIECES = HD / 8, WORDS = kKv4MaxBlocks / 32, K = 4;
  __shared__ unsigned begun[WORDS], ended[WORDS];   // a bit per block: it began a tile that goes on, it ended one
  __shared__ int4 tile[kKv4MaxBlocks];              // (request, KV head, tile, first block and number of blocks << 16)
  pdl_begin();
  const int row = threadIdx.x, lane = row & 31;
  int4 what = make_int4(0, 0, 0, 0);
  if (row < kKv4MaxBlocks) {
    int end = 0;
    if (row < blocks) {
      what = p.parts[2 * row + 1];
      end = p.parts[2 * row].w;
    }
    const unsigned x = __ballot_sync(0xffffffffu, what.w != 0), y = __ballot_sync(0xffffffffu, end == 2);
    if (lane == 0) {
      begun[row >> 5] = x;
      ended[row >> 5] = y;
    }
  }
  __syncthreads();
  int tiles = 0, before = 0;
#pragma unroll
  for (int i = 0; i < WORDS; ++i) {
    const unsigned x = begun[i];
    tiles += __popc(x);
    if (32 * i < row) before += __popc(row - 32 * i < 32 ? x & ((1u << (row - 32 * i)) - 1) : x);
  }
  if (what.w != 0) {   // the block that ends the tile: the next one that ends any
    int j = (row + 1) >> 5;
    unsigned rest = j < WORDS ? ended[j] & (0xffffffffu << ((row + 1) & 31)) : 0;
    while (rest == 0 && j < WORDS - 1) rest = ended[++j];
    tile[before] = make_int4(what.x, what.y, what.z, row | (rest == 0 ? 1 : 32 * j + __ffs(rest) - row) << 16);
  }
  __syncthreads();
  for (int item = blockIdx.x; item < tiles * PIECES; item += gridDim.x) {
    const int piece = item % PIECES;
    what = tile[item / PIECES];
    const int first = what.w & 0xFFFF, n = what.w >> 16;
    const float4* o = reinterpret_cast<const float4*>(p.part_o) + 2 * piece * 256 + row;
    const Kv4Req rq = kv4_request(p, what.x);
    float mx = -INFINITY, all = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    for (int s = 0; s < n; s += K) {
      float lse[K];
      float4 x[K], y[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (s + k >= n) continue;
        const long part = 2 * (first + s + k) + (s + k == 0);
        lse[k] = p.part_lse[part * 256 + row];
        x[k] = o[part * 64 * HD];
        y[k] = o[part * 64 * HD + 256];
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (s + k >= n) continue;
        const float top = fmaxf(mx, lse[k]);
        const float base = top == -INFINITY ? 0.f : top;
        const float f = exp2f(mx - base), w = exp2f(lse[k] - base);   // a part with NaN makes all NaN
        mx = top;
        all = all * f + w;
        a = make_float4(a.x * f + w * x[k].x, a.y * f + w * x[k].y, a.z * f + w * x[k].z, a.w * f + w * x[k].w);
        b = make_float4(b.x * f + w * y[k].x, b.y * f + w * y[k].y, b.z * f + w * y[k].z, b.w * f + w * y[k].w);
      }
    }
    const int R = 256 * what.z + row;
    if (R >= rq.n * p.group) continue;
    const long t = rq.q0 + R / p.group;
    const int h = what.y * p.group + R % p.group;
    const float inv = all == 0.f ? 0.f : 1.f / all;
    uint4 out;
    out.x = kv4_bf16_pair(a.x * inv, a.y * inv);
    out.y = kv4_bf16_pair(a.z * inv, a.w * inv);
    out.z = kv4_bf16_pair(b.x * inv, b.y * inv);
    out.w = kv4_bf16_pair(b.z * inv, b.w * inv);
    *reinterpret_cast<uint4*>(p.out + t * p.o_tok + h * p.o_head + 8 * piece) = out;
    if (piece == 0 && p.lse != nullptr)
      p.lse[t * p.H + h] = all == 0.f ? -INFINITY : (mx + log2f(all)) * 0.6931471805599453f;
  }
}

}  // namespace dllm
